// fd_tree_mma.cu -- attention of a tree of drafted tokens over a bf16 cache on the
// 5th-generation tensor cores, for more than 64 rows a KV head.
//
// The rows of a KV head's group (heads x tokens, 128 a CTA) are the rows of
// both products: S = Q K^T (128 x 128 keys, over D) and O = P V (128 x D, over the 128
// keys of a tile).  Blocks of rows of a KV head run side by side on the same keys, which come from memory once
// and from L2 for the others.
//
// Precision: K and V are exact in bf16.  q and p (fp32) are cut into three bf16
// numbers of eight bits each by truncation, which is exact, so all products are, and
// fp32 sums are what rounds: S sums its small parts first, and O is taken out of
// tensor memory every tile and added up in registers, since the adds of the matrix
// unit drop bits.  Six products of 8 k-steps make some 3100 cycles a tile of 128 channels, and a
// tile's 64 KB at an SM's share of the memory rate some 3000: the products bind.
//
// Measured: 256 rows a KV head on 131072 keys, 8 KV heads: 250 us, 1.65 PFLOP/s of exact products (the chip at its power limit, at
// 1.87 GHz; a long run of large bf16 matrix products in a library reaches 1.73).
//
// Twelve warps:
//   0-3  softmax, thread = row: reads S, masks, keeps the running max and sum, writes P
//        over S; cuts q at the start of a piece.
//   4-7  sums, thread = row: O of each tile times what the max has moved by; writes the
//        rows at the end of a piece.
//   8    walks the share, announces its pieces, copies q (its first 64 rows) and K;
//   9    copies (the other rows of q and) V.  K and V have a ring of slots each, as only one warp may wait for a slot to
//        be free: a barrier tells a phase from the one before, not from the one before that.  A warp starts a copy in
//        some 100 cycles, so a copy brings up to 64 rows of a page and 64 channels (128-byte swizzle), and K and V have
//        a warp each (with copies of 16 rows by one warp a tile took 4300 cycles);
//   10   products, one thread: S of the next tile, then O of this one.  While the softmax of a tile runs, the tensor
//        core has the S of the next and the O of the one before.  (With a warp for S and one for O, 8 % slower.)
//   11   nothing: registers are given back by four warps together.
#include "fd_tree_tc.cuh"

namespace fdk {
namespace {

constexpr int kRows = kTreeRowsMma;
constexpr int kKeys = kPlanTile;
constexpr int kThreads = 384, kRegs = 168;  // registers a thread at launch
constexpr int kMoreRegs = 200, kLessRegs = 104;  // of the softmax and the sums, and of the other roles
static_assert(256 * kMoreRegs + 128 * kLessRegs == kThreads * kRegs, "shares");
constexpr int kCopyK = 8, kCopyV = 9, kProducts = 10;
constexpr uint32_t kMiscBytes = 3 * 1024;
constexpr int kPBufs = 4;                // barriers of P and places for a tile's max
// Tensor memory: two S / P buffers and O.  P takes 8 columns for each part of 16 keys, 192 in
// all, and S the last 128 of them: a chunk of P never reaches an unread chunk of S.
constexpr uint32_t kBuf = 192, kSOff = 64, kOCol = 384;

template <int D>
struct Layout {
  static constexpr int kNB = D / 64;                          // 128-byte column blocks of a row
  static constexpr uint32_t kBlock = 16384;                   // [128 rows][128 bytes]
  static constexpr uint32_t kTile = kNB * kBlock;             // a K or V tile
  static constexpr uint32_t kQBlock = kRows * 128u;           // a column block of a part of q
  static constexpr uint32_t kQPart = kNB * kQBlock;
  static constexpr uint32_t kRing = kParts * kQPart;          // q first
  static constexpr uint32_t kK = D == 64 ? 4 : 2, kV = D == 64 ? 4 : 2;  // slots
  static constexpr uint32_t kVRing = kRing + kK * kTile;
  static constexpr uint32_t kMisc = kVRing + kV * kTile;
  static constexpr uint32_t kQRowsPerSlot = kTile / (D * 4);  // fp32 rows of q
  static constexpr uint32_t kBytes = kMisc + kMiscBytes;
  static_assert(kBytes <= 232448, "shared memory");
};

// Behind the ring.
struct Misc {
  uint64_t k_full[4], k_empty[4], v_full[4], v_empty[4];
  uint64_t q_full[2][2];                               // of even and odd pieces, of each 64 rows
  uint64_t s_full[2], p_empty[2], o_empty[2], p_full[kPBufs];
  uint64_t piece_full[2], piece_empty[2];
  uint64_t o_full, q_ready, fin_full, fin_empty, drain;
  uint32_t tmem;
  volatile int abort;
  TreePiece piece[2];
  float m[kPBufs][kRows]; // running max of the last tiles
  float l[kRows];         // a piece's sums
  uint64_t unfit[4];      // tokens whose values are not finite, as the softmax warps met them
};
static_assert(sizeof(Misc) <= kMiscBytes, "Misc");

// What does not fit the registers spills to L2, as shared memory leaves L1 nothing: 64 drafts (256 rows) on 131072 keys took 8 heads
// 316 us with 168 for every thread, 268 with 200 for those with much to hold, 250 with less code in the loops and S read twice.
__device__ __forceinline__ void take_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kMoreRegs)); }
__device__ __forceinline__ void give_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLessRegs)); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    fd_tree_mma_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                       const __grid_constant__ TreeParams p) {
  using Lay = Layout<D>;
  constexpr uint32_t kBlock = Lay::kBlock, kTile = Lay::kTile;
  extern __shared__ __align__(1024) uint8_t smem[];
  Misc& s = *reinterpret_cast<Misc*>(smem + Lay::kMisc);
  const uint32_t sq = smem_addr(smem), k_ring = sq + Lay::kRing, v_ring = sq + Lay::kVRing;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int32_t range = blockIdx.x / p.nsub, sub = blockIdx.x % p.nsub;
  const int32_t row0 = sub * kRows;
  const int32_t live = p.rows - row0 < kRows ? p.rows - row0 : kRows;
  const uint32_t nq = ((uint32_t)live + Lay::kQRowsPerSlot - 1) / Lay::kQRowsPerSlot;
  const uint32_t warps = ((uint32_t)live + 31) / 32;  // of the softmax and of the sums that have rows

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
      mbar_init(s.s_full + i, 1);
      for (int k = 0; k < 2; ++k) mbar_init(&s.q_full[i][k], 1);
      mbar_init(s.p_empty + i, 1);
      mbar_init(s.o_empty + i, warps);
      mbar_init(s.piece_full + i, 1);
      mbar_init(s.piece_empty + i, 2 + 2 * warps);
    }
    for (int i = 0; i < kPBufs; ++i) mbar_init(s.p_full + i, warps);
    mbar_init(&s.o_full, 1);
    mbar_init(&s.drain, 1);
    mbar_init(&s.q_ready, warps);
    mbar_init(&s.fin_full, warps);
    mbar_init(&s.fin_empty, warps);
    s.abort = 0;
    fence_barrier_init();
  }
  if (warp == kCopyK && lane == 0) prefetch_tensormap(&tmap_k);
  if (warp == kCopyV && lane == 0) prefetch_tensormap(&tmap_v);
  if (warp == kProducts) tmem_alloc_all(smem_addr(&s.tmem));
  if (warp < 4 && warp >= (int)warps) {  // rows of q that are none are 0
    for (uint32_t i = 0; i < kParts * Lay::kNB * 8u; ++i)
      sts128(sq + (i >> 3) * Lay::kQBlock + (uint32_t)tid * 128u + (i & 7u) * 16u, 0u, 0u, 0u, 0u);
    fence_async();
  }
  pdl_launch_dependents();
  tmem_fence_before();
  cta_sync();
  tmem_fence_after();
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
  // Rows [64 i, 64 (i + 1)) of the q of piece e, which lie side by side, into a slot.  They have barriers of their own, as
  // the softmax waits for them without having waited for the slot's other uses; two, as q of the next piece may come
  // before the softmax looks (not that of the one after: no ring has five slots).
  auto copy_q = [&](const TreePiece& pc, uint32_t e, int32_t i, uint8_t* to, uint64_t* full) {
    if (lane == 0) {
      uint64_t* landed = &s.q_full[e & 1][i];
      const int32_t first = i * (int32_t)Lay::kQRowsPerSlot;
      const int32_t rows = live - first < (int32_t)Lay::kQRowsPerSlot ? live - first : (int32_t)Lay::kQRowsPerSlot;
      mbar_arrive_expect_tx(landed, (uint32_t)rows * D * 4);
      bulk_load(to, p.q + (((int64_t)pc.b * p.Hkv + pc.h) * p.rows + row0 + first) * D, (uint32_t)rows * D * 4, landed);
      mbar_arrive(full);
    }
    __syncwarp();
  };
  auto leave = [&](uint64_t* full, uint32_t u, uint32_t n, uint32_t i, uint32_t f) {
    if (!w.ok) {
      s.abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
    if (lane != 0) return;
    land(full, u, n, w.limit);
    for (uint32_t e = f > 2 ? f - 2 : 0; e < f; ++e) mbar_wait_for(&s.q_full[e & 1][i], (e >> 1) & 1, w.limit);
  };

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
          if (pc.b >= 0 && sub == 0) walk.say(pc);
        }
        if (pc.b < 0) break;
        const int32_t n = ceil_div(pc.end - pc.begin, kKeys);
        int32_t page = copy.page_of(pc, 0);
        w.on(s.k_empty + r.slot, r.phase ^ 1u);
        if (!w.all()) break;
        copy_q(pc, e, 0, smem + Lay::kRing + r.slot * kTile, s.k_full + r.slot);
        ++f;
        ++u;
        r.next();
        for (int32_t j = 0; j < n; ++j, ++u, r.next()) {
          const int32_t next = copy.page_of(pc, j + 1);
          w.on(s.k_empty + r.slot, r.phase ^ 1u);
          if (!w.all()) break;
          copy.start<Lay::kNB>(&tmap_k, pc, j, page, smem + Lay::kRing + r.slot * kTile, s.k_full + r.slot);
          page = next;
        }
        if (!w.ok) break;
      }
      leave(s.k_full, u, Lay::kK, 0, f);
    } else if (warp == kCopyV) {
      // ------------------------------------------------------------ q, V
      uint32_t u = 0, f = 0;
      Ring<Lay::kV> r;
      TreePiece pc;
      for (uint32_t e = 0; take(e, pc); ++e) {
        const int32_t n = ceil_div(pc.end - pc.begin, kKeys);
        int32_t page = copy.page_of(pc, 0);
        if (nq == 2) {
          w.on(s.v_empty + r.slot, r.phase ^ 1u);
          if (!w.all()) break;
          copy_q(pc, e, 1, smem + Lay::kVRing + r.slot * kTile, s.v_full + r.slot);
          ++f;
          ++u;
          r.next();
        }
        for (int32_t j = 0; j < n; ++j, ++u, r.next()) {
          const int32_t next = copy.page_of(pc, j + 1);
          w.on(s.v_empty + r.slot, r.phase ^ 1u);
          if (!w.all()) break;
          copy.start<Lay::kNB>(&tmap_v, pc, j, page, smem + Lay::kVRing + r.slot * kTile, s.v_full + r.slot);
          page = next;
        }
        if (!w.ok) break;
      }
      leave(s.v_full, u, Lay::kV, 1, f);
    } else if (warp == kProducts) {
      // ------------------------------------------------------------ products
      // Every branch and operand is uniform over the warp as the compiler sees it (votes and shuffles), so that the
      // products take their operands from uniform registers as they are.
      constexpr uint32_t idS = bf16_instr_desc(kRows, kKeys), idO = bf16_instr_desc(kRows, D, true);
      const uint32_t base = uniform(tmem), q0 = uniform(sq), k0 = uniform(k_ring), v0 = uniform(v_ring);
      Ring<Lay::kK> rk;
      Ring<Lay::kV> rv;
      uint32_t g = 0, f = 0;  // tiles and pieces so far
      TreePiece pc;
      for (uint32_t e = 0; take(e, pc); ++e) {
        const uint32_t n = uniform((uint32_t)ceil_div(pc.end - pc.begin, kKeys));
        w.on(&s.q_ready, f & 1);
        if (!w.all()) break;
        if (elect_one()) {  // the slots that q came in
          mbar_arrive(s.k_empty + rk.slot);
          if (nq == 2) mbar_arrive(s.v_empty + rv.slot);
        }
        __syncwarp();
        rk.next();
        if (nq == 2) rv.next();
        for (uint32_t j = 0; j <= n; ++j) {
          if (j < n) {
            const uint32_t t = g + j;
            w.on(s.k_full + rk.slot, rk.phase);
            if (!w.all()) break;
            tmem_fence_after();
            if (elect_one()) {
              const uint32_t d = base + (t & 1) * kBuf + kSOff, k = k0 + rk.slot * kTile;
#pragma unroll 1
              for (int part = kParts - 1; part >= 0; --part) {
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                  const uint32_t block = (uint32_t)(i >> 2), off = (uint32_t)(i & 3) * 32u;
                  mma_ss(d, b_desc(q0 + (uint32_t)part * Lay::kQPart + block * Lay::kQBlock + off),
                         b_desc(k + block * kBlock + off), idS, part != kParts - 1 || i != 0);
                }
              }
              mma_commit(smem_addr(s.s_full + (t & 1)));
              mma_commit(smem_addr(s.k_empty + rk.slot));
            }
            __syncwarp();
            rk.next();
          }
          if (j > 0) {
            const uint32_t t = g + j - 1;
            w.on(s.v_full + rv.slot, rv.phase);
            w.on(s.p_full + t % kPBufs, (t / kPBufs) & 1);
            if (t > 0) w.on(s.o_empty + ((t - 1) & 1), ((t - 1) >> 1) & 1);
            if (!w.all()) break;
            tmem_fence_after();
            if (elect_one()) {
              const uint32_t a = base + (t & 1) * kBuf, v = v0 + rv.slot * kTile;
#pragma unroll 1
              for (int part = kParts - 1; part >= 0; --part) {
#pragma unroll
                for (int i = 0; i < kKeys / 16; ++i)
                  mma_ts(base + kOCol, a + (uint32_t)i * (8u * kParts) + (uint32_t)part * 8u,
                         b_desc_rows(v + (uint32_t)i * 2048u, kBlock), idO, part != kParts - 1 || i != 0);
              }
              mma_commit(smem_addr(&s.o_full));
              mma_commit(smem_addr(s.p_empty + (t & 1)));
              mma_commit(smem_addr(s.v_empty + rv.slot));
            }
            __syncwarp();
            rv.next();
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
        mma_commit(smem_addr(&s.drain));
        if (!mbar_wait_for(&s.drain, 0, w.limit)) atomicOr(p.err, kErrTimeout);
      }
      __syncwarp();
    }
  } else if (warp < 4) {
    take_registers();
    if (warp < (int)warps) {
    // ------------------------------------------------------------ softmax
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const int32_t row = warp * 32 + lane;  // of the block = lane of tensor memory
    // A scale of either sign, or 0, goes into q, so that scores rise with S.
    const float f = p.qk_scale == 0.f ? 1.f : fabsf(p.qk_scale);
    const uint32_t flip = p.qk_scale < 0.f ? 0x80000000u : 0u, keepq = p.qk_scale == 0.f ? 0u : 0xffffffffu;
    const uint64_t f2 = pack2(f, f);
    uint32_t g = 0, uk = 0, uv = 0;  // tiles and uses of the rings so far
    TreePiece pc;
    for (uint32_t e = 0; take(e, pc); ++e) {
      const int32_t n = ceil_div(pc.end - pc.begin, kKeys), P = pc.len - pc.m;
      // q: three bf16 parts of the row in the swizzled layout of an MMA operand.  The products of the piece before
      // have read theirs: its last S has been seen.  A lane starts at a 16-byte chunk of its own, off the others' banks.
      for (uint32_t i = 0; i < nq; ++i) w.on(&s.q_full[e & 1][i], (e >> 1) & 1);
      if (row < live || e == 0) {  // rows that are none stay 0
        constexpr uint32_t kC = D / 4, kStep = 8;  // fp32 chunks of a row, at a time
        const uint32_t from = (row < (int32_t)Lay::kQRowsPerSlot ? k_ring + uk % Lay::kK * kTile : v_ring + uv % Lay::kV * kTile) +
                              (uint32_t)row % Lay::kQRowsPerSlot * (D * 4);
#pragma unroll 1
        for (uint32_t i0 = 0; i0 < kC; i0 += kStep) {
          uint4 x[kStep];
#pragma unroll
          for (uint32_t i = 0; i < kStep; ++i) {
            x[i] = make_uint4(0u, 0u, 0u, 0u);
            if (row < live) x[i] = lds128u(from + ((i0 + i + (uint32_t)lane) % kC) * 16u);
          }
#pragma unroll
          for (uint32_t i = 0; i < kStep; ++i) {
            const uint32_t c = (i0 + i + (uint32_t)lane) % kC, c8 = c >> 1;  // c8: chunk of eight bf16
            uint32_t a[kParts], b[kParts];
            cut3(__uint_as_float((x[i].x & keepq) ^ flip), __uint_as_float((x[i].y & keepq) ^ flip), a);
            cut3(__uint_as_float((x[i].z & keepq) ^ flip), __uint_as_float((x[i].w & keepq) ^ flip), b);
            const uint32_t to = sq + (c8 >> 3) * Lay::kQBlock + (uint32_t)row * 128u + (((c8 ^ (uint32_t)row) & 7u) << 4) + (c & 1u) * 8u;
#pragma unroll
            for (int part = 0; part < kParts; ++part) sts64(to + (uint32_t)part * Lay::kQPart, a[part], b[part]);
          }
        }
      }
      fence_async();
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.q_ready);
      uint64_t anc = 0, unfit = 0;
      if (pc.end > P) {
        const Ancestors all = tree_ancestors(p.tree, pc.b, pc.m, p.err);
        anc = all.of((row0 + row) % p.tree.n - (p.tree.n - pc.m));
      }
      float m = -INFINITY, l = 0.f;
      for (int32_t j = 0; j < n; ++j) {
        const uint32_t t = g + (uint32_t)j, buf = t & 1;
        const int32_t t0 = pc.begin + j * kKeys;
        const uint32_t at = tmem + buf * kBuf + lanes;
        w.on(s.s_full + buf, (t >> 1) & 1);
        tmem_fence_after();
        const bool some_hidden = t0 + kKeys > P;
        TileMask mask;
        if (some_hidden) mask = tile_mask(P, anc, t0);
        // S twice: for its maximum, and for P a chunk at a time (held in registers it took all of them, 255 us for 250)
        float top4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          float x[64];
          uint32_t* xr = reinterpret_cast<uint32_t*>(x);
          TmemRow<32>::load(at + kSOff + 64u * h, xr);
          TmemRow<32>::load(at + kSOff + 64u * h + 32u, xr + 32);
          tmem_wait_loads();
          TmemRow<32>::tie(xr);
          TmemRow<32>::tie(xr + 32);
          if (some_hidden) {
            const uint32_t w0 = h ? mask.w[2] : mask.w[0], w1 = h ? mask.w[3] : mask.w[1];
#pragma unroll
            for (int c = 0; c < 64; ++c) x[c] = (c < 32 ? w0 : w1) >> (c & 31) & 1u ? x[c] : -INFINITY;
          }
#pragma unroll
          for (int c = 0; c < 64; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) top4[i] = max3(top4[i], x[c + 2 * i], x[c + 2 * i + 1]);
        }
        const float top = max3(fmaxf(top4[0], top4[1]), top4[2], top4[3]);
        const float mn = fmaxf(m, top == -INFINITY ? -INFINITY : top * f);
        const float alpha = m == mn ? 1.f : ex2(m - mn);  // 0 from -inf
        const float base = mn == -INFINITY ? 0.f : mn;
        const uint64_t base2 = pack2(-base, -base);
        uint64_t sum2[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};
        uint32_t next[16];
        TmemRow<16>::load(at + kSOff, next);
#pragma unroll 2
        for (int c = 0; c < kKeys / 16; ++c) {
          uint32_t x[16];
          tmem_wait_loads();
          TmemRow<16>::tie(next);
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = next[i];
          if (c + 1 < kKeys / 16) TmemRow<16>::load(at + kSOff + 16u * (c + 1), next);
          if (some_hidden) {
            const uint32_t two = c < 4 ? (c < 2 ? mask.w[0] : mask.w[1]) : (c < 6 ? mask.w[2] : mask.w[3]), w16 = two >> (16 * (c & 1));
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = w16 >> i & 1u ? x[i] : 0xff800000u;
          }
          uint32_t a[8 * kParts];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float y0, y1;
            unpack2(fma2(pack2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), f2, base2), y0, y1);
            y0 = ex2(y0);
            y1 = ex2(y1);
            sum2[i & 1] = add2(sum2[i & 1], pack2(y0, y1));
            uint32_t part[kParts];
            cut3(y0, y1, part);
#pragma unroll
            for (int k = 0; k < kParts; ++k) a[8 * k + i] = part[k];
          }
          TmemRow<16>::store(at + (uint32_t)c * 24u, a);
          TmemRow<8>::store(at + (uint32_t)c * 24u + 16u, a + 16);
        }
        float s0, s1, s2, s3;
        unpack2(sum2[0], s0, s1);
        unpack2(sum2[1], s2, s3);
        l = fmaf(l, alpha, (s0 + s1) + (s2 + s3));
        m = mn;
        // the sums are past the tile that had this place: S of this one came after O of the tile before the last, which
        // waited for the sums of the one before that
        s.m[t % kPBufs][row] = m;
        if (t0 + kKeys > P) {
          // V's rows at or past the length may hold anything, and so may those of the drafts, which not every
          // row sees: 0 * NaN is not 0.  Values that are no numbers become 0 here and are added to the rows that
          // see them at the end.
          const uint32_t use = uv + nq - 1 + (uint32_t)j, v = v_ring + use % Lay::kV * kTile;
          // The slot's use before this one must have landed for the wait to tell them apart.  It is that of a tile
          // whose O is done (S of this tile came after it), but for the first tile where q has a slot too: there it is the
          // tile before.
          if (nq == 2 && j == 0 && t > 0) w.on(s.p_empty + ((t - 1) & 1), ((t - 1) >> 1) & 1);
          w.on(s.v_full + use % Lay::kV, (use / Lay::kV) & 1);
          constexpr int kChunks = D / 8;
          const int32_t first = P > t0 ? P - t0 : 0, end = pc.len - t0 < kKeys ? pc.len - t0 : kKeys;
          for (int32_t i = row; i < (kKeys - first) * kChunks; i += (int32_t)warps * 32) {
            const int32_t v_row = first + i / kChunks;
            const uint32_t c = (uint32_t)(i % kChunks);
            const uint32_t a = v + (c >> 3) * kBlock + (uint32_t)v_row * 128u + ((c & 7u) << 4);
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
          fence_async();
        }
        tmem_wait_stores();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s.p_full + t % kPBufs);
      }
      if (e >= 1) w.on(&s.fin_empty, (e - 1) & 1);
      s.l[row] = l;
      unfit = ((uint64_t)__reduce_or_sync(0xffffffffu, (uint32_t)(unfit >> 32)) << 32) |
              __reduce_or_sync(0xffffffffu, (uint32_t)unfit);
      if (lane == 0) s.unfit[warp] = unfit;
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.fin_full);
      g += (uint32_t)n;
      uk += 1 + (uint32_t)n;
      uv += nq - 1 + (uint32_t)n;
      if (!w.all()) break;
    }
    if (!w.ok) {
      s.abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
    }
  } else if (warp < 8) {
    take_registers();
    if (warp < 4 + (int)warps) {
    // ------------------------------------------------------------ sums
    const uint32_t at = tmem + kOCol + ((uint32_t)((warp - 4) * 32) << 16);
    const int32_t row = (warp - 4) * 32 + lane;
    tree_no_rows<D, kRows, 0>(p, range, sub, row, (int)warps * 32);
    uint32_t g = 0;
    TreePiece pc;
    for (uint32_t e = 0; take(e, pc); ++e) {
      const int32_t n = ceil_div(pc.end - pc.begin, kKeys);
      uint64_t acc[D / 2];
#pragma unroll
      for (int i = 0; i < D / 2; ++i) acc[i] = 0;
      float m = -INFINITY;
      for (int32_t j = 0; j < n; ++j) {
        const uint32_t t = g + (uint32_t)j, buf = t & 1;
        w.on(s.p_full + t % kPBufs, (t / kPBufs) & 1);
        const float mn = s.m[t % kPBufs][row];
        const float alpha = m == mn ? 1.f : ex2(m - mn);
        m = mn;
        const uint64_t alpha2 = pack2(alpha, alpha);
        w.on(&s.o_full, t & 1);
        tmem_fence_after();
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          float o[32];
          tmem_load<32>(at + 32u * c, o);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[16 * c + i] = fma2(acc[16 * c + i], alpha2, pack2(o[2 * i], o[2 * i + 1]));
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(s.o_empty + buf);
      }
      g += (uint32_t)n;
      w.on(&s.fin_full, e & 1);
      const float l = s.l[row];
      uint64_t unfit = 0;
      for (uint32_t i = 0; i < warps; ++i) unfit |= s.unfit[i];
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.fin_empty);
      const bool writes = row < live && (row0 + row) % p.tree.n >= p.tree.n - pc.m;
      float o[D];
#pragma unroll
      for (int i = 0; i < D / 2; ++i) unpack2(acc[i], o[2 * i], o[2 * i + 1]);
      if (w.all() && unfit) {  // (of a piece that was given up it may be anything)
        const Ancestors all = tree_ancestors(p.tree, pc.b, pc.m, p.err);
        unfit &= all.of((row0 + row) % p.tree.n - (p.tree.n - pc.m));
        while (unfit) {
          const int32_t place = pc.len - pc.m + __ffsll((long long)unfit) - 1;
          unfit &= unfit - 1;
          int64_t v_row = ((int64_t)pc.b * p.Hkv + pc.h) * p.kv.capacity + place;
          if (p.kv.paged) {
            const int32_t page = __ldg(p.kv.block_table + (int64_t)pc.b * p.kv.max_pages + place / p.kv.page_size);
            if (page < 0 || page >= p.kv.num_pages) continue;
            v_row = ((int64_t)page * p.Hkv + pc.h) * p.kv.page_size + place % p.kv.page_size;
          }
          const uint32_t* v = static_cast<const uint32_t*>(p.kv.v) + v_row * (D / 2);
#pragma unroll
          for (int i = 0; i < D / 2; ++i) {
            const uint32_t x = __ldg(v + i);
            if ((x & 0x7f80u) == 0x7f80u) o[2 * i] += bf16_lo(x);
            if ((x & 0x7f800000u) == 0x7f800000u) o[2 * i + 1] += bf16_hi(x);
          }
        }
      }
      if (writes && w.ok) {
        const int64_t out = ((int64_t)pc.b * p.Hkv + pc.h) * p.rows + row0 + row;
        const int64_t state = ((int64_t)pc.slot * p.nsub + sub) * kRows + row;
        float* to = pc.slot < 0 ? p.out + out * D : p.o_part + state * D;
        const float inv = pc.slot >= 0 ? 1.f : (l == 0.f ? 0.f : 1.f / l);
#pragma unroll
        for (int i = 0; i < D; i += 8) {
#pragma unroll
          for (int k = 0; k < 8; ++k) o[i + k] *= inv;
          store32(to + i, o + i);
        }
        if (pc.slot >= 0) {
          p.m_part[state] = m;
          p.l_part[state] = l;
        } else if (p.lse) {
          p.lse[out] = l == 0.f ? -INFINITY : (m + log2f(l)) * kTreeLn2;
        }
      }
      if (!w.all()) break;
    }
    if (!w.ok) {
      s.abort = 1;
      atomicOr(p.err, kErrTimeout);
    }
    }
  }
  tmem_fence_before();
  cta_sync();
  if (warp == kProducts) {
    tmem_fence_after();
    tmem_free_all(tmem);
  }
}

template <int D>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p, cudaStream_t stream) {
  constexpr uint32_t bytes = Layout<D>::kBytes;
  const cudaError_t e = allow_smem<fd_tree_mma_kernel<D>, kRegs>((int)bytes);
  if (e != cudaSuccess) return e;
  return launch_early(fd_tree_mma_kernel<D>, (unsigned)(p.ranges * p.nsub), kThreads, bytes, stream, tk, tv, p);
}

}  // namespace

cudaError_t launch_tree_mma(int D, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                            cudaStream_t stream) {
  if (D == 128) return launch<128>(tk, tv, p, stream);
  if (D == 64) return launch<64>(tk, tv, p, stream);
  return cudaErrorInvalidValue;
}

}  // namespace fdk
