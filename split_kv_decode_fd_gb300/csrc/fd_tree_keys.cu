// fd_tree_keys.cu -- attention of a tree of drafted tokens over a bf16 cache, up to 64
// rows a KV head: keys on the rows of the matrix products, query rows on their columns.
//
//     S^T = K Q^T   (128 keys x rows, over D)       O^T = V^T P   (D x rows, over 128 keys)
//
// so that K and V are read from shared memory where they land, as the first operands, and a
// product's work goes with the rows there are (N = 32 or 64), not with 128 (fd_tree_mma.cu).
//
// Precision: K and V are exact in bf16.  q and p (fp32) are cut into three bf16 numbers of eight
// bits each by truncation, which is exact, so all products are, and fp32 sums are what rounds.
// The parts of q lie side by side as 3 N columns of one product, so that K is read once for
// all of them, and their columns are added in registers, small parts first; of p the first two parts, and
// the third is added to the columns of the second.  (A product for each part read 400 KB of shared memory a
// tile, 3100 cycles of its bandwidth.)  O is taken out of tensor memory every tile, since
// the adds of the matrix unit drop bits.
//
// Bound by memory where the rows are few: with 32 rows 131072 keys stream at 6.4 to 6.7 TB/s; with 64 a tile takes some 2930 cycles,
// S, softmax, P and O one after another through one place for P, against 2890 at an SM's share of the memory rate.  Measured: 64
// rows, 131072 keys of 8 heads 96 us (5.6 TB/s; 4 more with P's place given back as one, not the first two parts before the
// third); 64 paged sequences of 512 to 16384 tokens, 64 rows, 230 us (5.5 TB/s), of
// which a piece's start and end are some 4 us together and a CTA has 4 of them.  Code that a piece runs once is rolled: it comes from
// behind the instruction cache (with q's cut and the mask unrolled the paged sequences took 12 us more; 640 sequences of 512 tokens take 407).
//
// A row's reference (what its scores are taken relative to) is the same for all keys, and moves only when a score of a
// tile exceeds it by 2^kTau: a vote of the threads says so, and then the tile's maxima are found.
//
// Sixteen warps:
//   0-7   softmax: thread = key, two groups of four warps for half of the rows each.  Reads S, masks, writes
//         P to shared memory; cuts q at the start of a piece.
//   8-11  sums, thread = channel: O of each tile times what the references have moved by; writes the rows
//         at the end of a piece.
//   12    walks the share, announces its pieces, copies q and K;   13  copies V;
//   14, 15  products, one thread of each: S, and O.
#include "fd_tree_tc.cuh"

namespace fdk {
namespace {

constexpr int kKeys = kPlanTile;
constexpr int kThreads = 512, kRegs = 128;  // registers a thread at launch
constexpr int kSoftmaxRegs = 136, kSumsRegs = 152, kOtherRegs = 88;
static_assert(256 * kSoftmaxRegs + 128 * kSumsRegs + 128 * kOtherRegs == kThreads * kRegs, "shares");
constexpr int kSums = 8, kCopyK = 12, kCopyV = 13, kSWarp = 14;  // first of the sums' warps; S, and O: 15
constexpr uint32_t kMiscBytes = 3 * 1024;
constexpr int kMoves = 4;              // tiles whose moves of the references are kept
constexpr float kTau = 8.f;            // p stays below 2^kTau
constexpr float kNoRef = -3.0e38f;     // the reference of a row that has seen no key

template <int D, int N>
struct Layout {
  static constexpr int kNB = D / 64;                        // 128-byte column blocks of a row
  static constexpr uint32_t kTile = kNB * kTileBlock;       // a K or V tile
  static constexpr uint32_t kQPart = N * 128u;              // rows of a part of q in a column block
  static constexpr uint32_t kQBlock = kParts * kQPart;
  static constexpr uint32_t kPPart = kKeys * N * 2u;        // a part of p: [N / 8][128 keys][8 rows]
  static constexpr uint32_t kP = kNB * kQBlock;             // q first
  static constexpr uint32_t kRing = kP + kParts * kPPart;
  static constexpr uint32_t kK = D == 64 ? 4 : N == 32 ? 3 : 2, kV = D == 64 ? 4 : 2;  // slots
  static constexpr uint32_t kVRing = kRing + kK * kTile;
  static constexpr uint32_t kMisc = kVRing + kV * kTile;
  static constexpr uint32_t kBytes = kMisc + kMiscBytes;
  static_assert(kBytes <= 232448, "shared memory");
  static_assert(N * D * 4 <= kTile, "a slot holds the rows of q");
};

// Behind the rings.
template <int N>
struct Misc {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t q_full[2];                  // of even and odd pieces
  uint64_t s_full[2], s_empty[2], o_full, o_empty, moves_full[kMoves];
  uint64_t piece_full[2], piece_empty[2];
  uint64_t p_full, p_empty[2], q_ready, fin_full, fin_empty, drain[2];
  uint32_t tmem;
  volatile int abort;
  TreePiece piece[2];
  alignas(16) float move[kMoves][N];   // what the sums so far are multiplied by; move[.][half] < 0: they are not
  alignas(16) float ref[N];            // references, base 2, with the other sign
  float part[8][N / 2];                // by warp: maxima of a tile, sums of a piece
  uint64_t unfit[8];                   // tokens whose values are not finite, as the softmax warps met them
};

// An MMA's A operand in rows (of K) of 128 bytes with the 128-byte swizzle, its M along the rows: as b_desc_rows.
constexpr uint32_t kAlongRows = 1u << 15;  // of the instruction descriptor: A is M-major

__device__ __forceinline__ bool group_or(bool pred, uint32_t id) {
  uint32_t r;
  __syncwarp();
  asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, %2, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
               : "=r"(r)
               : "r"((uint32_t)pred), "r"(id)
               : "memory");
  return r != 0;
}

// One of v[0 .. R) in each lane of a warp: lane l gets that of index l % R over all lanes, by halving.
template <int R, class F>
__device__ __forceinline__ float across(float (&v)[R], F f) {
  const uint32_t lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= R) {
#pragma unroll
      for (int i = 0; i < R; ++i) v[i] = f(v[i], __shfl_xor_sync(0xffffffffu, v[i], o));
    } else {
      const bool up = (lane & (uint32_t)o) != 0;
#pragma unroll
      for (int i = 0; i < o; ++i) {
        const float mine = up ? v[i + o] : v[i], other = up ? v[i] : v[i + o];
        v[i] = f(mine, __shfl_xor_sync(0xffffffffu, other, o));
      }
    }
  }
  return v[0];
}

// What does not fit the registers spills to L2, as shared memory leaves L1 nothing (64 paged sequences: 255 us with 128
// for every thread, 239 with these shares).
template <int N>
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs)); }

template <int D, int N>
__global__ void __launch_bounds__(kThreads, 1)
    fd_tree_keys_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                        const __grid_constant__ TreeParams p) {
  using Lay = Layout<D, N>;
  constexpr uint32_t kTile = Lay::kTile;
  constexpr int kHalf = N / 2;  // rows of a softmax group
  static_assert(sizeof(Misc<N>) <= kMiscBytes, "Misc");
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc<N>& s = *reinterpret_cast<Misc<N>*>(smem + Lay::kMisc);
  const uint32_t sq = smem_addr(smem), sp = sq + Lay::kP, k_ring = sq + Lay::kRing, v_ring = sq + Lay::kVRing;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t range = blockIdx.x / p.nsub, sub = blockIdx.x % p.nsub;
  const int32_t row0 = sub * N;
  const int32_t live = p.rows - row0 < N ? p.rows - row0 : N;

  if ((sq & 1023u) != 0) {  // the swizzle goes by address; no room is left to align here
    if (tid == 0) atomicOr(p.err, kErrTimeout);
    return;
  }
  if (tid == 0) {
    for (int i = 0; i < 4; ++i) {
      mbar_init(s.k_full + i, 1);
      mbar_init(s.k_empty + i, 1);
      mbar_init(s.v_full + i, 1);
      mbar_init(s.v_empty + i, 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s.q_full + i, 1);
      mbar_init(s.s_full + i, 1);
      mbar_init(s.s_empty + i, 8);
      mbar_init(s.piece_full + i, 1);
      mbar_init(s.piece_empty + i, 3 + 8 + 4);
      mbar_init(s.drain + i, 1);
    }
    for (int i = 0; i < kMoves; ++i) mbar_init(s.moves_full + i, 8);
    mbar_init(&s.o_full, 1);
    mbar_init(&s.o_empty, 4);
    mbar_init(&s.p_full, 8);
    mbar_init(s.p_empty, 1);
    mbar_init(s.p_empty + 1, 1);
    mbar_init(&s.q_ready, 8);
    mbar_init(&s.fin_full, 8);
    mbar_init(&s.fin_empty, 4);
    s.abort = 0;
    fence_barrier_init();
  }
  if (warp == kCopyK && lane == 0) prefetch_tensormap(&tmap_k);
  if (warp == kCopyV && lane == 0) prefetch_tensormap(&tmap_v);
  if (warp == kSWarp) tmem_alloc_all(smem_addr(&s.tmem));
  pdl_launch_dependents();
  tmem_fence_before();
  cta_sync();
  tmem_fence_after();
  // Tensor memory: two buffers of S^T of 3 N columns (with one, K's slot waited for the softmax), then O^T, 2 N columns.
  const uint32_t tmem = s.tmem;
  pdl_wait();
  Waits w{&s.abort, kWaitLimitNs};

  // The next piece, for a warp; false at the end.
  auto take = [&](uint32_t e, TreePiece& pc) -> bool {
    w.on(s.piece_full + (e & 1), (e >> 1) & 1);
    if (!w.all()) return false;
    pc = s.piece[e & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(s.piece_empty + (e & 1));
    return pc.b >= 0;
  };
  const TileCopy copy(p);

  if (warp >= kCopyK) {
    give_registers();  // a warpgroup at one place, as the instruction wants it
    if (warp == kCopyK) {
      // ------------------------------------------------------------ pieces, q, K
      uint32_t u = 0, f = 0;
      Ring<Lay::kK> r;
      TreeWalk<0> walk(p, range);
      if (lane == 0 && sub == 0) walk.say_none();
      for (uint32_t e = 0;; ++e) {
        TreePiece pc;
        if (!walk.next(pc)) pc.b = -1;
        if (e >= 2) w.on(s.piece_empty + (e & 1), ((e >> 1) - 1) & 1);
        if (!w.all()) break;
        if (lane == 0) {
          s.piece[e & 1] = pc;
          mbar_arrive(s.piece_full + (e & 1));
        }
        if (pc.b < 0) break;
        const int32_t n = ceil_div(pc.end - pc.begin, kKeys);
        int32_t page = copy.page_of(pc, 0);
        w.on(s.k_empty + r.slot, r.phase ^ 1u);
        if (!w.all()) break;
        // The rows of q lie side by side.  They have barriers of their own, as the softmax waits for them without
        // having waited for the slot's other uses; two, as q of the next piece may come before the softmax looks (not
        // that of the one after: no ring has five slots).
        if (lane == 0) {
          mbar_arrive_expect_tx(s.q_full + (e & 1), (uint32_t)live * D * 4);
          bulk_load(smem + Lay::kRing + r.slot * kTile, p.q + (((int64_t)pc.b * p.Hkv + pc.h) * p.rows + row0) * D,
                    (uint32_t)live * D * 4, s.q_full + (e & 1));
          mbar_arrive(s.k_full + r.slot);
        }
        __syncwarp();
        ++f;
        ++u;
        r.next();
        for (int32_t j = 0; j < n; ++j, ++u, r.next()) {
          const int32_t next = copy.page_of(pc, j + 1);
          w.on(s.k_empty + r.slot, r.phase ^ 1u);
          if (!w.all()) break;
          copy.start<Lay::kNB>(&tmap_k, pc, j, page, smem + Lay::kRing + r.slot * kTile, s.k_full + r.slot);
          page = next;
          if (j == 0 && lane == 0 && sub == 0) walk.say(pc);
        }
        if (!w.ok) break;
      }
      if (!w.ok) {
        s.abort = 1;
        atomicOr(p.err, kErrTimeout);
      }
      if (lane == 0) {
        land(s.k_full, u, Lay::kK, w.limit);
        for (uint32_t e = f > 2 ? f - 2 : 0; e < f; ++e) mbar_wait_for(s.q_full + (e & 1), (e >> 1) & 1, w.limit);
      }
    } else if (warp == kCopyV) {
      // ------------------------------------------------------------ V
      uint32_t u = 0;
      Ring<Lay::kV> r;
      TreePiece pc;
      for (uint32_t e = 0; take(e, pc); ++e) {
        const int32_t n = ceil_div(pc.end - pc.begin, kKeys);
        int32_t page = copy.page_of(pc, 0);
        for (int32_t j = 0; j < n; ++j, ++u, r.next()) {
          const int32_t next = copy.page_of(pc, j + 1);
          w.on(s.v_empty + r.slot, r.phase ^ 1u);
          if (!w.all()) break;
          copy.start<Lay::kNB>(&tmap_v, pc, j, page, smem + Lay::kVRing + r.slot * kTile, s.v_full + r.slot);
          page = next;
        }
        if (!w.ok) break;
      }
      if (!w.ok) {
        s.abort = 1;
        atomicOr(p.err, kErrTimeout);
      }
      if (lane == 0) land(s.v_full, u, Lay::kV, w.limit);
    } else {
      // ------------------------------------------------------------ products
      // Every branch and operand is uniform over the warp as the compiler sees it (votes and shuffles), so that the
      // products take their operands from uniform registers as they are.
      constexpr uint32_t idS = bf16_instr_desc(kKeys, kParts * N), idO = bf16_instr_desc(D, 2 * N, true) | kAlongRows,
                         idLast = bf16_instr_desc(D, N, true) | kAlongRows;
      const uint32_t base = uniform(tmem), q0 = uniform(sq), p0 = uniform(sp), k0 = uniform(k_ring), v0 = uniform(v_ring);
      const bool is_s = uniform((uint32_t)warp) == kSWarp;
      Ring<Lay::kK> rk;
      Ring<Lay::kV> rv;
      uint32_t g = 0, f = 0;  // tiles and pieces so far
      TreePiece pc;
      for (uint32_t e = 0; take(e, pc); ++e) {
        const uint32_t n = uniform((uint32_t)ceil_div(pc.end - pc.begin, kKeys));
        if (is_s) {
          w.on(&s.q_ready, f & 1);
          if (!w.all()) break;
          if (elect_one()) mbar_arrive(s.k_empty + rk.slot);  // the slot that q came in
          __syncwarp();
          rk.next();
          for (uint32_t j = 0; j < n; ++j, rk.next()) {
            const uint32_t t = g + j;
            w.on(s.k_full + rk.slot, rk.phase);
            if (t >= 2) w.on(s.s_empty + (t & 1), ((t - 2) >> 1) & 1);
            if (!w.all()) break;
            tmem_fence_after();
            if (elect_one()) {
              const uint32_t d = base + (t & 1) * (kParts * N), k = k0 + rk.slot * kTile;
#pragma unroll
              for (int i = 0; i < D / 16; ++i) {
                const uint32_t block = (uint32_t)(i >> 2), off = (uint32_t)(i & 3) * 32u;
                mma_ss(d, b_desc(k + block * kTileBlock + off), b_desc(q0 + block * Lay::kQBlock + off), idS, i != 0);
              }
              mma_commit(smem_addr(s.s_full + (t & 1)));
              mma_commit(smem_addr(s.k_empty + rk.slot));
            }
            __syncwarp();
          }
        } else {
          for (uint32_t j = 0; j < n; ++j, rv.next()) {
            const uint32_t t = g + j;
            w.on(s.v_full + rv.slot, rv.phase);
            w.on(&s.p_full, t & 1);
            if (t > 0) w.on(&s.o_empty, (t - 1) & 1);
            if (!w.all()) break;
            tmem_fence_after();
            if (elect_one()) {
              const uint32_t d = base + 2 * kParts * N, v = v0 + rv.slot * kTile;
#pragma unroll
              for (int i = 0; i < kKeys / 16; ++i)
                mma_ss(d, b_desc_rows(v + (uint32_t)i * 2048u, kTileBlock), b_desc_n<kKeys * 16>(p0 + (uint32_t)i * 256u), idO,
                       i != 0);
              mma_commit(smem_addr(s.p_empty));  // the first two parts' places
#pragma unroll
              for (int i = 0; i < kKeys / 16; ++i)
                mma_ss(d + N, b_desc_rows(v + (uint32_t)i * 2048u, kTileBlock),
                       b_desc_n<kKeys * 16>(p0 + 2 * Lay::kPPart + (uint32_t)i * 256u), idLast, 1);
              mma_commit(smem_addr(&s.o_full));
              mma_commit(smem_addr(s.p_empty + 1));
              mma_commit(smem_addr(s.v_empty + rv.slot));
            }
            __syncwarp();
          }
        }
        if (!w.ok) break;
        g += n;
        ++f;
      }
      if (!w.ok) {
        s.abort = 1;
        atomicOr(p.err, kErrTimeout);
      }
      // every product has completed before tensor memory is given back
      if (elect_one()) {
        uint64_t* done = s.drain + (is_s ? 0 : 1);
        mma_commit(smem_addr(done));
        if (!mbar_wait_for(done, 0, w.limit)) atomicOr(p.err, kErrTimeout);
      }
      __syncwarp();
    }
  } else if (warp < kSums) {
    take_registers<kSoftmaxRegs>();
    // ------------------------------------------------------------ softmax
    // The four warps of a group meet at barriers: they stay together, whatever a wait of one of them says, and leave
    // together.
    const uint32_t group = (uint32_t)warp >> 2, id = 1 + group;
    const int32_t key = (warp & 3) * 32 + lane;  // of a tile = lane of tensor memory
    const int32_t r0 = (int32_t)group * kHalf;   // this group's first row
    // A scale of either sign, or 0, goes into q, so that scores rise with S.
    const float f = p.qk_scale == 0.f ? 1.f : fabsf(p.qk_scale);
    const uint32_t flip = p.qk_scale < 0.f ? 0x80000000u : 0u, keepq = p.qk_scale == 0.f ? 0u : 0xffffffffu;
    uint32_t g = 0, uk = 0;  // tiles and uses of K's slots so far
    TreePiece pc;
    for (uint32_t e = 0;; ++e) {
      const bool more = take(e, pc);
      if (group_or(!more, id)) break;
      const int32_t n = ceil_div(pc.end - pc.begin, kKeys), P = pc.len - pc.m;
      // q: three bf16 parts of each row in the swizzled layout of an operand, by 256 / N threads a row.  The products
      // of the piece before have read theirs: every thread has seen its last S.
      w.on(s.q_full + (e & 1), (e >> 1) & 1);
      {
        constexpr int kPer = 256 / N, kC = D / 4 / kPer;  // threads a row, their 16-byte chunks
        const int32_t row = tid % N;
        const uint32_t c0 = (uint32_t)(tid / N * kC);
        const uint32_t from = k_ring + uk % Lay::kK * kTile + (uint32_t)row * (D * 4);
#pragma unroll 1
        for (int i = 0; i < kC; ++i) {  // a lane starts at a chunk of its own, off the others' banks
          const uint32_t c = c0 + (uint32_t)((i + lane) % kC), c8 = c >> 1;  // c8: chunk of eight bf16
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          if (row < live) x = lds128u(from + c * 16u);
          uint32_t a[kParts], b[kParts];
          cut3(__uint_as_float((x.x & keepq) ^ flip), __uint_as_float((x.y & keepq) ^ flip), a);
          cut3(__uint_as_float((x.z & keepq) ^ flip), __uint_as_float((x.w & keepq) ^ flip), b);
          const uint32_t to = sq + (c8 >> 3) * Lay::kQBlock + (uint32_t)row * 128u + (((c8 ^ (uint32_t)row) & 7u) << 4) + (c & 1u) * 8u;
#pragma unroll
          for (int part = 0; part < kParts; ++part) sts64(to + (uint32_t)part * Lay::kQPart, a[part], b[part]);
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_ready);
      uint64_t anc = 0, unfit = 0;  // of the token of row r0 + lane: its ancestors and itself
      if (pc.end > P) {
        const Ancestors all = tree_ancestors(p.tree, pc.b, pc.m, p.err);
        anc = all.of((row0 + r0 + lane) % p.tree.n - (p.tree.n - pc.m));
      }
      // The references of the piece before have been read.
      if (e >= 1) w.on(&s.fin_empty, (e - 1) & 1);
      if ((warp & 3) == 0 && lane < kHalf) s.ref[r0 + lane] = -kNoRef;
      group_or(false, id);
      uint64_t l[kHalf / 2];  // this key's sums of the rows, in pairs
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) l[i] = 0;
      for (int32_t j = 0; j < n; ++j) {
        const uint32_t t = g + (uint32_t)j;
        const int32_t t0 = pc.begin + j * kKeys;
        const bool some_hidden = t0 + kKeys > P;
        w.on(s.s_full + (t & 1), (t >> 1) & 1);
        tmem_fence_after();
        uint64_t x[kHalf / 2];  // scores of two rows
        {
          const uint32_t at = tmem + (t & 1) * (kParts * N) + group * kHalf + ((uint32_t)((warp & 3) * 32) << 16);
          uint32_t v0[kHalf], v1[kHalf];
          TmemRow<kHalf>::load(at + 2 * N, v0);
          TmemRow<kHalf>::load(at + N, v1);
          tmem_wait_loads();
          TmemRow<kHalf>::tie(v0);
          TmemRow<kHalf>::tie(v1);
          auto pair = [](const uint32_t* v) { return pack2(__uint_as_float(v[0]), __uint_as_float(v[1])); };
#pragma unroll
          for (int i = 0; i < kHalf / 2; ++i) x[i] = add2(pair(v0 + 2 * i), pair(v1 + 2 * i));
          TmemRow<kHalf>::load(at, v0);
          tmem_wait_loads();
          TmemRow<kHalf>::tie(v0);
#pragma unroll
          for (int i = 0; i < kHalf / 2; ++i) x[i] = add2(x[i], pair(v0 + 2 * i));
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s.s_empty + (t & 1));
        if (some_hidden) {
          // the rows that see this key
          const int32_t a = t0 + key - P;  // its token
          uint32_t sees = a < 0 ? 0xffffffffu : 0u;
          if (__any_sync(0xffffffffu, a >= 0 && a < 64)) {
#pragma unroll 2
            for (int i = 0; i < kHalf; ++i) {
              const uint32_t low = __shfl_sync(0xffffffffu, (uint32_t)anc, i), high = __shfl_sync(0xffffffffu, (uint32_t)(anc >> 32), i);
              if (a >= 0 && a < 64) sees |= ((a < 32 ? low : high) >> (a & 31) & 1u) << i;
            }
          }
#pragma unroll
          for (int i = 0; i < kHalf; i += 2) {
            float x0, x1;
            unpack2(x[i / 2], x0, x1);
            x[i / 2] = pack2(sees >> i & 1 ? x0 : -INFINITY, sees >> (i + 1) & 1 ? x1 : -INFINITY);
          }
        }
        // relative to the references (kept with the other sign); a NaN does not vote
        uint64_t y[kHalf / 2];
        const uint64_t f2 = pack2(f, f);
        auto relative = [&] {
#pragma unroll
          for (int i = 0; i < kHalf / 2; i += 2) {
            const float4 ref = lds128(smem_addr(s.ref + r0 + 2 * i));
            y[i] = fma2(x[i], f2, pack2(ref.x, ref.y));
            y[i + 1] = fma2(x[i + 1], f2, pack2(ref.z, ref.w));
          }
        };
        relative();
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kHalf / 2; ++i) {
          float y0, y1;
          unpack2(y[i], y0, y1);
          top = max3(top, y0, y1);
        }
        const bool moved = group_or(top > kTau, id);
        float* move = s.move[t % kMoves] + r0;
        if (moved) {
          // the tile's largest score of each row: of a warp's keys in lane i % kHalf, then of the four warps
          float best[kHalf];
#pragma unroll
          for (int i = 0; i < kHalf / 2; ++i) {
            float x0, x1;
            unpack2(x[i], x0, x1);
            best[2 * i] = x0 * f;
            best[2 * i + 1] = x1 * f;
          }
          const float most = across(best, [](float a, float b) { return fmaxf(a, b); });
          if (lane < kHalf) s.part[warp][lane] = most;
          group_or(false, id);
          if ((warp & 3) == 0 && lane < kHalf) {
            const float old = -s.ref[r0 + lane];
            float m = old;
#pragma unroll
            for (int i = 0; i < 4; ++i) m = fmaxf(m, s.part[4 * group + i][lane]);
            s.ref[r0 + lane] = -m;
            move[lane] = old == m ? 1.f : ex2(old - m);
          }
          group_or(false, id);
          relative();
#pragma unroll
          for (int i = 0; i < kHalf / 2; ++i) l[i] = mul2(l[i], pack2(move[2 * i], move[2 * i + 1]));
        } else if ((warp & 3) == 0 && lane == 0) {
          move[0] = -1.f;
        }
        uint32_t a[kParts][kHalf / 2];
#pragma unroll
        for (int i = 0; i < kHalf / 2; ++i) {
          float e0, e1;
          unpack2(y[i], e0, e1);
          e0 = ex2(e0);
          e1 = ex2(e1);
          l[i] = add2(l[i], pack2(e0, e1));
          uint32_t part[kParts];
          cut3(e0, e1, part);
#pragma unroll
          for (int k = 0; k < kParts; ++k) a[k][i] = part[k];
        }
        // P's places are free once O of the tile before has read them, the first two parts' before the third's
        const uint32_t to = sp + (uint32_t)(r0 / 8) * (kKeys * 16u) + (uint32_t)key * 16u;
#pragma unroll
        for (int k = 0; k < kParts; ++k) {
          if (k != 1 && t > 0) w.on(s.p_empty + k / 2, (t - 1) & 1);
#pragma unroll
          for (int c = 0; c < kHalf / 8; ++c)
            sts128(to + (uint32_t)k * Lay::kPPart + (uint32_t)c * (kKeys * 16u), a[k][4 * c], a[k][4 * c + 1], a[k][4 * c + 2],
                   a[k][4 * c + 3]);
        }
        if (some_hidden) {
          // V's rows at or past the length may hold anything, and so may those of the drafts, which not every
          // row sees: 0 * NaN is not 0.  Values that are no numbers become 0 here and are added to the rows that
          // see them at the end.  (The slot's use before this one has landed: O of the tile before is done.)
          const uint32_t slot = t % Lay::kV, v = v_ring + slot * kTile;
          w.on(s.v_full + slot, (t / Lay::kV) & 1);
          constexpr int kChunks = D / 8;
          const int32_t first = P > t0 ? P - t0 : 0, end = pc.len - t0 < kKeys ? pc.len - t0 : kKeys;
          for (int32_t i = tid; i < (kKeys - first) * kChunks; i += 256) {
            const int32_t v_row = first + i / kChunks;
            const uint32_t c = (uint32_t)(i % kChunks);
            const uint32_t a = v + (c >> 3) * kTileBlock + (uint32_t)v_row * 128u + ((c & 7u) << 4);
            if (v_row >= end) {
              sts128(a, 0u, 0u, 0u, 0u);
              continue;
            }
            const uint4 x4 = lds128u(a);
            uint32_t v4[4] = {x4.x, x4.y, x4.z, x4.w};
            bool any = false;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if ((v4[k] & 0x7f80u) == 0x7f80u) v4[k] &= 0xffff0000u, any = true;
              if ((v4[k] & 0x7f800000u) == 0x7f800000u) v4[k] &= 0x0000ffffu, any = true;
            }
            if (any) {
              sts128(a, v4[0], v4[1], v4[2], v4[3]);
              unfit |= 1ull << (t0 + v_row - P);
            }
          }
        }
        fence_async();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(s.moves_full + t % kMoves);
          mbar_arrive(&s.p_full);
        }
      }
      g += (uint32_t)n;
      uk += 1 + (uint32_t)n;
      // the rows' sums over this warp's keys
      float mine[kHalf];
#pragma unroll
      for (int i = 0; i < kHalf / 2; ++i) unpack2(l[i], mine[2 * i], mine[2 * i + 1]);
      const float sum = across(mine, [](float a, float b) { return a + b; });
      group_or(false, id);  // the maxima of the last tile have been read
      if (lane < kHalf) s.part[warp][lane] = sum;
      unfit = ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(unfit >> 32)) << 32) |
              __reduce_or_sync(0xffffffffu, (uint32_t)unfit);
      if (lane == 0) s.unfit[warp] = unfit;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.fin_full);
      if (group_or(!w.ok, id)) {
        w.ok = false;
        break;
      }
    }
    if (!w.ok) {
      s.abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
  } else {
    take_registers<kSumsRegs>();
    // ------------------------------------------------------------ sums
    // D = 128: lane of tensor memory = channel; D = 64: a warp's lanes 0-15 hold sixteen channels.
    constexpr int kLanes = D / 4;
    const int32_t channel = (warp & 3) * kLanes + lane % kLanes;
    const bool holds = lane < kLanes;
    const uint32_t at = tmem + 2 * kParts * N + ((uint32_t)((warp & 3) * 32) << 16);
    tree_no_rows<D, N, 0>(p, range, sub, tid - kSums * 32, 128);
    uint32_t g = 0;
    TreePiece pc;
    for (uint32_t e = 0; take(e, pc); ++e) {
      const int32_t n = ceil_div(pc.end - pc.begin, kKeys);
      float acc[N];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = 0.f;
      for (int32_t j = 0; j < n; ++j) {
        const uint32_t t = g + (uint32_t)j;
        w.on(s.moves_full + t % kMoves, (t / kMoves) & 1);
        const float* move = s.move[t % kMoves];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (move[h * kHalf] >= 0.f) {
#pragma unroll
            for (int i = 0; i < kHalf; ++i) acc[h * kHalf + i] *= move[h * kHalf + i];
          }
        }
        w.on(&s.o_full, t & 1);
        tmem_fence_after();
#pragma unroll
        for (int c = 0; c < N; c += 32) {
          float o[32], small[32];
          tmem_load<32>(at + (uint32_t)(N + c), small);
          tmem_load<32>(at + (uint32_t)c, o);
#pragma unroll
          for (int i = 0; i < 32; ++i) acc[c + i] += o[i] + small[i];
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s.o_empty);
      }
      g += (uint32_t)n;
      w.on(&s.fin_full, e & 1);
      // lane i: the sums and the references of rows i and i + 32
      float l[N / 32], m[N / 32];
#pragma unroll
      for (int k = 0; k < N / 32; ++k) {
        const int32_t r = lane + 32 * k, of = r / kHalf, in = r % kHalf;
        l[k] = (s.part[4 * of][in] + s.part[4 * of + 1][in]) + (s.part[4 * of + 2][in] + s.part[4 * of + 3][in]);
        m[k] = -s.ref[r];
      }
      uint64_t unfit = 0;
      for (int i = 0; i < 8; ++i) unfit |= s.unfit[i];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.fin_empty);
      if (w.all() && unfit) {  // (of a piece that was given up it may be anything)
        const Ancestors all = tree_ancestors(p.tree, pc.b, pc.m, p.err);
        uint64_t anc[N / 32];
#pragma unroll
        for (int k = 0; k < N / 32; ++k) anc[k] = all.of((row0 + lane + 32 * k) % p.tree.n - (p.tree.n - pc.m));
        for (uint64_t u = unfit; u; u &= u - 1) {
          const int32_t a = __ffsll((long long)u) - 1, place = pc.len - pc.m + a;
          int64_t v_row = ((int64_t)pc.b * p.Hkv + pc.h) * p.kv.capacity + place;
          if (p.kv.paged) {
            const int32_t page = __ldg(p.kv.block_table + (int64_t)pc.b * p.kv.max_pages + place / p.kv.page_size);
            if (page < 0 || page >= p.kv.num_pages) continue;
            v_row = ((int64_t)page * p.Hkv + pc.h) * p.kv.page_size + place % p.kv.page_size;
          }
          const uint32_t bits = (uint32_t)__ldg(static_cast<const uint16_t*>(p.kv.v) + v_row * D + channel) << 16;
          const bool bad = (bits & 0x7f800000u) == 0x7f800000u;
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const uint64_t see = __shfl_sync(0xffffffffu, anc[i / 32], i % 32);
            if (bad && (see >> a & 1)) acc[i] += __uint_as_float(bits);
          }
        }
      }
      // rows that are tokens' (a division for each of them, unrolled, was 64 KB of code to fetch: 15 us a piece)
      const int32_t pad = p.tree.n - pc.m;
      uint32_t writes[N / 32];
      float inv[N / 32];
#pragma unroll
      for (int k = 0; k < N / 32; ++k) {
        const int32_t r = lane + 32 * k;
        writes[k] = __ballot_sync(0xffffffffu, r < live && (row0 + r) % p.tree.n >= pad && w.ok);
        inv[k] = pc.slot >= 0 ? 1.f : (l[k] == 0.f ? 0.f : 1.f / l[k]);
      }
      const int64_t out = ((int64_t)pc.b * p.Hkv + pc.h) * p.rows + row0;
      const int64_t state = ((int64_t)pc.slot * p.nsub + sub) * N;
      float* to = (pc.slot < 0 ? p.out + out * D : p.o_part + state * D) + channel;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float x = acc[i] * __shfl_sync(0xffffffffu, inv[i / 32], i % 32);
        if (holds && (writes[i / 32] >> (i % 32) & 1u)) to[i * D] = x;
      }
      if (warp == kSums && w.ok) {
#pragma unroll
        for (int k = 0; k < N / 32; ++k) {
          const int32_t r = lane + 32 * k;
          if (!(writes[k] >> lane & 1u)) continue;
          if (pc.slot >= 0) {
            p.m_part[state + r] = m[k];
            p.l_part[state + r] = l[k];
          } else if (p.lse) {
            p.lse[out + r] = l[k] == 0.f ? -INFINITY : (m[k] + log2f(l[k])) * kTreeLn2;
          }
        }
      }
      if (!w.all()) break;
    }
    if (!w.ok) {
      s.abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
  }
  tmem_fence_before();
  cta_sync();
  if (warp == kSWarp) {
    tmem_fence_after();
    tmem_free_all(tmem);
  }
}

template <int D, int N>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  constexpr uint32_t bytes = Layout<D, N>::kBytes;
  const cudaError_t e = allow_smem<fd_tree_keys_kernel<D, N>, kRegs>((int)bytes);
  if (e != cudaSuccess) return e;
  return launch_early(fd_tree_keys_kernel<D, N>, (unsigned)(p.ranges * p.nsub), kThreads, bytes, stream, tk, tv, p);
}

}  // namespace

cudaError_t launch_tree_keys(int D, int rows, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                             cudaStream_t stream) {
  if (D == 128 && rows == 64) return launch<128, 64>(tk, tv, p, stream);
  if (D == 128 && rows == 32) return launch<128, 32>(tk, tv, p, stream);
  if (D == 64 && rows == 64) return launch<64, 64>(tk, tv, p, stream);
  if (D == 64 && rows == 32) return launch<64, 32>(tk, tv, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fdk
