// fd_keep.cu -- the rows of a cache that stay, moved together: place start + j of a
// sequence gets what place start + index[j] held, for a rising list index.
//
// The list rises, so index[j] >= j and a row never moves up.  A CTA takes a slice
// of the rows of one (sequence, KV head) of K or V and works through the list in
// order, a chunk at a time: all rows of a chunk are in registers before the first of
// them is stored, and a chunk's sources lie at or past its first place, so no store
// of an earlier chunk has reached them.  Slices of different channels share nothing.
#include "../../include/fdecode.h"
#include "fd_tree.cuh"

namespace fdk {
namespace {

constexpr int kThreads = 256;

// Lanes: 16-byte pieces of a row that a CTA takes; Loads: rows a thread holds.
template <int Lanes, int Loads>
__global__ void __launch_bounds__(kThreads) fd_keep_kernel(const KeepParams p, int32_t slices) {
  constexpr int kStep = kThreads / Lanes;   // rows side by side
  constexpr int kChunk = kStep * Loads;
  __shared__ int32_t stop;                  // first entry of the list that does not count
  pdl_launch_dependents();
  pdl_wait();
  int64_t c = blockIdx.x;
  const int32_t slice = (int32_t)(c % slices);
  c /= slices;
  uint4* base = static_cast<uint4*>(c % 2 ? p.kv.v : p.kv.k);
  c /= 2;
  const int32_t h = (int32_t)(c % p.kv.Hkv), b = (int32_t)(c / p.kv.Hkv);
  const int32_t count = p.counts ? clamp_len(__ldg(p.counts + b), p.n) : p.n;
  const int32_t start = p.starts ? __ldg(p.starts + b) : 0;
  const int32_t* index = p.index + (int64_t)b * p.n;
  const int32_t at = slice * Lanes + threadIdx.x % Lanes, row = threadIdx.x / Lanes;
  const int32_t width = slices * Lanes;     // 16-byte pieces of a row
  if (threadIdx.x == 0) stop = count;
  // 16-byte piece of place t, or -1
  auto piece = [&](int64_t t) -> int64_t {
    if (!p.kv.paged) return (((int64_t)b * p.kv.Hkv + h) * p.kv.capacity + t) * width + at;
    const int32_t page = __ldg(p.kv.block_table + (int64_t)b * p.kv.max_pages + t / p.kv.page_size);
    if (page < 0 || page >= p.kv.num_pages) return -1;
    return (((int64_t)page * p.kv.Hkv + h) * p.kv.page_size + t % p.kv.page_size) * width + at;
  };
  for (int32_t j0 = 0; j0 < count; j0 += kChunk) {
    uint4 x[Loads];
    bool moves[Loads];
    int32_t bad = INT32_MAX;
    bool lost = false;
#pragma unroll
    for (int i = 0; i < Loads; ++i) {
      const int32_t j = j0 + row + i * kStep;
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
    // every row of the chunk is loaded
    if (__syncthreads_or(bad != INT32_MAX)) {
      if (bad != INT32_MAX) atomicMin(&stop, bad);
      __syncthreads();
      if (threadIdx.x == 0) atomicOr(p.err, kErrBadIndex);
    }
    const int32_t last = stop;
#pragma unroll
    for (int i = 0; i < Loads; ++i) {
      const int32_t j = j0 + row + i * kStep;
      if (!moves[i] || j >= last) continue;
      const int64_t dst = piece((int64_t)start + j);
      if (dst >= 0)
        base[dst] = x[i];
      else
        atomicOr(p.err, kErrBadIndex);
    }
    if (last < count) return;
  }
}

template <int Lanes, int Loads>
cudaError_t launch(const KeepParams& p, int slices, cudaStream_t stream) {
  const int64_t grid = (int64_t)p.B * p.kv.Hkv * 2 * slices;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  return launch_early(fd_keep_kernel<Lanes, Loads>, (unsigned)grid, kThreads, 0, stream, p, (int32_t)slices);
}

}  // namespace

cudaError_t launch_keep(int row_bytes, const KeepParams& p, cudaStream_t stream) {
  // the drafts of a step: whole rows, all of them at once
  if (p.n <= 64) {
    if (row_bytes == 128) return launch<8, 2>(p, 1, stream);
    if (row_bytes == 256) return launch<16, 4>(p, 1, stream);
    return launch<32, 8>(p, 1, stream);
  }
  // long lists: slices of a sector, as only they run side by side
  return launch<2, 8>(p, row_bytes / 32, stream);
}

}  // namespace fdk
