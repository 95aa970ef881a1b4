// fd_keep.cu -- the rows of a cache that stay, moved together: place start + j of a
// sequence gets what place start + index[j] held, for a rising list index.
//
// The list rises, so index[j] >= j and a row never moves up.  A CTA takes a slice
// of the rows of one (sequence, KV head) of K or V and works through the list in
// order, a chunk at a time: all rows of a chunk are loaded before the first of
// them is stored, and a chunk's sources lie at or past its first place, so no store
// of an earlier chunk has reached them.  Slices of different channels share nothing.
//
// The drafts of a step (up to 64 entries) are one chunk of whole rows in registers: bound by a chain
// of loads (count, index, page, row).  Long lists go through shared memory, five chunks of 16 KB on their way
// (loads may run ahead of the stores of earlier chunks).  Where the first row that moves comes from behind
// the last place that is written, as when the latest part of a sequence stays, no row is both read and written: the CTAs
// of a (sequence, KV head) share the list and take whole rows.  Otherwise each takes the whole list
// and a 32-byte slice of the rows, if there are fewer (sequence, KV head)s than SMs.
// Measured, bf16, D = 128: the 5 rows of a step 1.7 us, 64 paths of up to 8 rows 4.4 us; 65536 rows of 8 heads 99.8 us (5.4 TB/s)
// from behind what is written, of which every CTA's look at the list is some 8, 250 us (2.1 TB/s) where they overlap; 16 such lists of 4096 rows 97 us (5.5 TB/s).
#include "../../include/fdecode.h"
#include "fd_tree.cuh"

namespace fdk {
namespace {

constexpr int kThreads = 256;

// Up to 64 entries.  Lanes: 16-byte pieces of a row; Loads: rows a thread holds.
template <int Lanes, int Loads>
__global__ void __launch_bounds__(kThreads) fd_keep_kernel(const KeepParams p) {
  constexpr int kStep = kThreads / Lanes;   // rows side by side
  static_assert(kStep * Loads == kMaxDrafts, "one chunk");
  __shared__ int32_t stop;                  // first entry of the list that does not count
  pdl_launch_dependents();
  pdl_wait();
  int64_t c = blockIdx.x;
  uint4* base = static_cast<uint4*>(c % 2 ? p.kv.v : p.kv.k);
  c /= 2;
  const int32_t h = (int32_t)(c % p.kv.Hkv), b = (int32_t)(c / p.kv.Hkv);
  const int32_t count = p.counts ? clamp_len(__ldg(p.counts + b), p.n) : p.n;
  const int32_t start = p.starts ? __ldg(p.starts + b) : 0;
  const int32_t* index = p.index + (int64_t)b * p.n;
  const int32_t at = threadIdx.x % Lanes, row = threadIdx.x / Lanes;
  if (threadIdx.x == 0) stop = count;
  // 16-byte piece of place t, or -1
  auto piece = [&](int64_t t) -> int64_t {
    if (!p.kv.paged) return (((int64_t)b * p.kv.Hkv + h) * p.kv.capacity + t) * Lanes + at;
    const int32_t page = __ldg(p.kv.block_table + (int64_t)b * p.kv.max_pages + t / p.kv.page_size);
    if (page < 0 || page >= p.kv.num_pages) return -1;
    return (((int64_t)page * p.kv.Hkv + h) * p.kv.page_size + t % p.kv.page_size) * Lanes + at;
  };
  uint4 x[Loads];
  bool moves[Loads];
  int32_t bad = INT32_MAX;
  bool lost = false;
#pragma unroll
  for (int i = 0; i < Loads; ++i) {
    const int32_t j = row + i * kStep;
    moves[i] = false;
    if (j >= count) continue;
    const int32_t from = __ldg(index + j), before = j > 0 ? __ldg(index + j - 1) : -1;
    if (from <= before || before < -1 || start < 0 || (int64_t)start + from >= p.max_len) {
      bad = j < bad ? j : bad;
      continue;
    }
    if (from == j) continue;
    const int64_t src = piece((int64_t)start + from);
    moves[i] = src >= 0;
    lost = lost || src < 0;
    if (moves[i]) x[i] = base[src];
  }
  if (lost) atomicOr(p.err, kErrBadIndex);
  // every row is loaded
  if (__syncthreads_or(bad != INT32_MAX)) {
    if (bad != INT32_MAX) atomicMin(&stop, bad);
    __syncthreads();
    if (threadIdx.x == 0) atomicOr(p.err, kErrBadIndex);
  }
  const int32_t last = stop;
#pragma unroll
  for (int i = 0; i < Loads; ++i) {
    const int32_t j = row + i * kStep;
    if (!moves[i] || j >= last) continue;
    const int64_t dst = piece((int64_t)start + j);
    if (dst >= 0)
      base[dst] = x[i];
    else
      atomicOr(p.err, kErrBadIndex);
  }
}

// ------------------------------------------------------------------ long lists
constexpr int kLongLoads = 4, kStages = 6, kScan = 8;
constexpr int kStageBytes = kThreads * kLongLoads * 16;

// The cache rows of one (sequence, KV head) of K or V, in 16-byte pieces.
struct Rows {
  uint4* base;
  const int32_t* table;  // paged: the sequence's
  int64_t first;         // piece 0 of place 0 (contiguous)
  int32_t Hkv, h, page_size, num_pages, width;

  // Piece `at` of place t, or -1.
  __device__ __forceinline__ int64_t piece(int64_t t, int32_t at) const {
    if (!table) return first + t * width + at;
    const int32_t page = __ldg(table + t / page_size);
    if (page < 0 || page >= num_pages) return -1;
    return (((int64_t)page * Hkv + h) * page_size + t % page_size) * width + at;
  }
};

// Entries [j0, j1) of a rising list, all of them in range: piece `at` + (thread % Lanes) of their rows.  A thread stores
// what it has loaded itself, so a barrier a chunk is all that the threads share.
template <int Lanes>
__device__ __forceinline__ void move_rows(const Rows& r, const int32_t* index, int32_t start, int32_t j0, int32_t j1,
                                          int32_t at, uint32_t ring, unsigned* err) {
  constexpr int kStep = kThreads / Lanes;
  constexpr int kChunk = kStep * kLongLoads;
  const int32_t row = threadIdx.x / Lanes;
  at += threadIdx.x % Lanes;
  const uint32_t mine = ring + threadIdx.x * 16u;
  const int32_t chunks = (j1 - j0 + kChunk - 1) / kChunk;
  int32_t from[kLongLoads];  // entries of the next chunk to be loaded
  auto entries = [&](int32_t k) {
#pragma unroll
    for (int i = 0; i < kLongLoads; ++i) {
      const int32_t j = j0 + k * kChunk + row + i * kStep;
      from[i] = k < chunks && j < j1 ? __ldg(index + j) : -1;
    }
  };
  uint64_t moves = 0;  // eight bits a stage: rows on their way
  auto load = [&](int32_t k) {
    if (k < chunks) {
      const int32_t s = k % kStages;
      uint64_t bits = 0;
      bool lost = false;
#pragma unroll
      for (int i = 0; i < kLongLoads; ++i) {
        if (from[i] < 0) continue;
        const int64_t src = r.piece((int64_t)start + from[i], at);
        lost = lost || src < 0;
        if (src < 0) continue;
        bits |= 1ull << i;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(mine + (uint32_t)(s * kStageBytes + i * (kThreads * 16))),
                     "l"(r.base + src)
                     : "memory");
      }
      moves = (moves & ~(0xffull << (8 * s))) | bits << (8 * s);
      if (lost) atomicOr(err, kErrBadIndex);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    entries(k + 1);
  };
  entries(0);
  for (int32_t k = 0; k < kStages - 1; ++k) load(k);
  for (int32_t k = 0; k < chunks; ++k) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncthreads();  // every row of the chunk is loaded
    const int32_t s = k % kStages;
#pragma unroll
    for (int i = 0; i < kLongLoads; ++i) {
      if (!(moves >> (8 * s + i) & 1)) continue;
      const int64_t dst = r.piece((int64_t)start + j0 + k * kChunk + row + i * kStep, at);
      if (dst >= 0)
        r.base[dst] = lds128u(mine + (uint32_t)(s * kStageBytes + i * (kThreads * 16)));
      else
        atomicOr(err, kErrBadIndex);
    }
    load(k + kStages - 1);
  }
}

// Wide: 16-byte pieces of a row; Narrow: of a slice.  parts: CTAs of a (sequence, KV head), Wide / Narrow at least.
template <int Wide, int Narrow>
__global__ void __launch_bounds__(kThreads) fd_keep_long_kernel(const KeepParams p, int32_t parts) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ int32_t s_stop, s_moves;
  pdl_launch_dependents();
  pdl_wait();
  int64_t c = blockIdx.x;
  const int32_t part = (int32_t)(c % parts);
  c /= parts;
  Rows r;
  r.base = static_cast<uint4*>(c % 2 ? p.kv.v : p.kv.k);
  c /= 2;
  const int32_t h = (int32_t)(c % p.kv.Hkv), b = (int32_t)(c / p.kv.Hkv);
  r.table = p.kv.paged ? p.kv.block_table + (int64_t)b * p.kv.max_pages : nullptr;
  r.first = ((int64_t)b * p.kv.Hkv + h) * p.kv.capacity * Wide;
  r.Hkv = p.kv.Hkv;
  r.h = h;
  r.page_size = p.kv.page_size;
  r.num_pages = p.kv.num_pages;
  r.width = Wide;
  const int32_t count = p.counts ? clamp_len(__ldg(p.counts + b), p.n) : p.n;
  const int32_t start = p.starts ? __ldg(p.starts + b) : 0;
  const int32_t* index = p.index + (int64_t)b * p.n;
  // The whole list: its first entry that does not count, and the first that moves its row.  (index[j] - j never falls.)
  if (threadIdx.x == 0) s_stop = s_moves = count;
  __syncthreads();
  int32_t bad = count, moves = count;
  const int64_t room = start < 0 ? 0 : (int64_t)p.max_len - start;  // entries from there on point past the end
  const int32_t lead = (int32_t)((reinterpret_cast<uintptr_t>(index) / 4) & 3);  // index - lead is at a 16-byte boundary
  const int lane = threadIdx.x & 31;
  for (int32_t j0 = -lead; j0 < count; j0 += 4 * kScan * kThreads) {
    int4 at[kScan];
    int32_t before[kScan];  // lane 0's first
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      const int32_t j = j0 + 4 * (i * kThreads + (int32_t)threadIdx.x);
      before[i] = lane == 0 && j > 0 && j < count ? __ldg(index + j - 1) : -1;
      if (j >= 0 && j + 4 <= count) {
        at[i] = __ldg(reinterpret_cast<const int4*>(index + j));
      } else {
        auto one = [&](int32_t k) { return k >= 0 && k < count ? __ldg(index + k) : -1; };
        at[i] = make_int4(one(j), one(j + 1), one(j + 2), one(j + 3));
      }
    }
#pragma unroll
    for (int i = 0; i < kScan; ++i) {
      const int32_t j = j0 + 4 * (i * kThreads + (int32_t)threadIdx.x);
      const int4 a = at[i];
      const int32_t up = __shfl_up_sync(0xffffffffu, a.w, 1), prev = lane == 0 ? before[i] : up;
      const bool whole = j >= 0 && j + 4 <= count;
      // four that rise, in range, and stay (as all before them do) or are behind one that moves: most are
      if (whole && prev < a.x && a.x < a.y && a.y < a.z && a.z < a.w && a.w < room && (a.w == j + 3 || j >= moves)) continue;
      const int32_t v[5] = {prev, a.x, a.y, a.z, a.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if (j + x < 0 || j + x >= count) continue;
        if (v[x + 1] <= v[x] || v[x + 1] >= room) bad = min(bad, j + x);
        if (v[x + 1] != j + x) moves = min(moves, j + x);
      }
    }
  }
  if (bad < count) atomicMin(&s_stop, bad);
  if (moves < count) atomicMin(&s_moves, moves);
  __syncthreads();
  const int32_t stop = s_stop, first = s_moves;
  if (stop < count && threadIdx.x == 0) atomicOr(p.err, kErrBadIndex);
  if (first >= stop) return;
  if (parts > 1 && __ldg(index + first) >= stop) {
    // no row is both read and written
    const int32_t per = (stop - first + parts - 1) / parts;
    const int64_t j0 = first + (int64_t)part * per, j1 = stop - j0 < per ? stop : j0 + per;
    if (j0 < j1) move_rows<Wide>(r, index, start, (int32_t)j0, (int32_t)j1, 0, smem_addr(ring), p.err);
  } else if (part < Wide / Narrow) {
    move_rows<Narrow>(r, index, start, first, stop, part * Narrow, smem_addr(ring), p.err);
  }
}

template <int Wide, int Narrow>
cudaError_t launch_long(const KeepParams& p, int64_t parts, cudaStream_t stream) {
  const int64_t grid = (int64_t)p.B * p.kv.Hkv * 2 * parts;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  const cudaError_t e = allow_smem<fd_keep_long_kernel<Wide, Narrow>>(kStages * kStageBytes);
  if (e != cudaSuccess) return e;
  return launch_early(fd_keep_long_kernel<Wide, Narrow>, (unsigned)grid, kThreads, (size_t)kStages * kStageBytes, stream, p,
                      (int32_t)parts);
}

template <int Wide>
cudaError_t launch_long(const KeepParams& p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t pairs = (int64_t)p.B * p.kv.Hkv * 2;
  if (pairs >= sms) return launch_long<Wide, Wide>(p, 1, stream);
  const int64_t parts = 2 * (int64_t)sms / pairs;  // two CTAs an SM
  return launch_long<Wide, 2>(p, parts > Wide / 2 ? parts : Wide / 2, stream);
}

template <int Lanes, int Loads>
cudaError_t launch(const KeepParams& p, cudaStream_t stream) {
  const int64_t grid = (int64_t)p.B * p.kv.Hkv * 2;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_early(fd_keep_kernel<Lanes, Loads>, (unsigned)grid, kThreads, 0, stream, p);
}

}  // namespace

cudaError_t launch_keep(int row_bytes, const KeepParams& p, cudaStream_t stream) {
  if (p.n <= kMaxDrafts) {
    if (row_bytes == 128) return launch<8, 2>(p, stream);
    if (row_bytes == 256) return launch<16, 4>(p, stream);
    return launch<32, 8>(p, stream);
  }
  if (row_bytes == 128) return launch_long<8>(p, stream);
  if (row_bytes == 256) return launch_long<16>(p, stream);
  return launch_long<32>(p, stream);
}

}  // namespace fdk
