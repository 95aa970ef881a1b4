// fd_kv4_decode.cu -- decode attention over a 4-bit cache on the tcgen05 tensor
// cores.
//
// A piece of work is a run of keys of one (sequence, KV head) and the up to 16
// query heads (or heads x rows) of its group; the balanced plan of fd_plan.h
// gives every SM's CTA an equal share of pieces.  Per tile of 128 keys:
//
//     S^T[key, head] = K[key, :] . q[head, :]        M = 128 keys, K = D
//     p = exp2(S - m),  l += p                       thread = key
//     O^T[d, head] += V^T[d, :] . p[:, head]         M = 128 channels, K = 128 keys
//
// Both products take their A operand (K, V^T) from tensor memory as fp16, where a
// lane is a row: the thread that owns the row widens its codes in registers
// and stores them there.  code * scale has six significant bits and is exact in
// fp16.  The B operands are small: q (once per piece) and p (per tile) in shared
// memory, each as the sum of two fp16 numbers, hi and lo (p's lo held 2^11 times up), that
// sit in columns of their own; so the products are exact, and they add up in fp32.  q is K-major in
// swizzled rows; p is N-major, so that a key's thread stores its heads as they lie
// in registers, eight columns a 16-byte store.
//
// What bounds it: 9/16 byte per element from HBM (18 KB per tile for D = 128, 414 ns or
// 857 cycles of an SM's share of a copy's rate, at 2070 MHz) and, next to it, instruction issue:
// a tile is 1300 instructions of widening (one conversion and one product for two elements) and,
// with all waits and the softmax, some 3200, which is 800 of a scheduler's slots.  A tile
// takes 1060 cycles with 4 heads a group, so each is busy for some 80 % of it.  The
// MMAs cost hardly any (mma.sync costs as many as the widening: measured 8.4 slots for
// a 16x8x16 step), and with heads on the N axis their time does not grow with the group.
// Measured, D = 128, 8 KV heads, as the slope of the time from 131072 to 1048576 tokens: 1060 cycles
// a tile with 4 heads a group (5.5 TB/s, 81 % of a copy's rate), 1160 with 8, 1810 with 16 (the
// softmax of half the heads takes a group of warps that long); with pages of 16 tokens 1070 and 1160.
// What does not grow with the length (launch, a CTA's start, join) is 13 us with 4 heads, 14 with
// 8, 20 with 16, so that 131072 tokens take 40.5 us (3.7 TB/s), 524288 tokens 123 (4.9 TB/s, 72 %), 135
// and 209, 16 ragged sequences of 1024 to 16384 tokens 32.5.
//
// Twenty-eight warps:
//   0      walks the plan, announces pieces, copies tiles into a ring of stages: all of
//          a contiguous cache (one bulk copy each), the even ones of a paged one;
//   1, 2   one thread of each issues MMAs: S, and O (each MMA takes 18
//          cycles to issue, and a tile needs eight of each kind); the latter also
//          counts the pieces that the CTA goes on after;
//   3      q of the next piece: scaled to the fp16 range by a power of two per
//          head, split hi / lo, written in the B layout; the odd tiles of a paged cache;
//   4-11   K, two groups of four warps: lane = key;
//   12-19  V, two groups: lane = channel;
//   20-27  softmax, two groups: lane = key; lane = channel where O is taken.
// Group 0 of each role takes the even tiles and group 1 the odd ones (with 16 heads the
// softmax groups take half of the heads each), so that a tile's latency (shared memory, conversions, tensor-memory stores, barriers)
// may be two tiles long.  The softmax groups share nothing within a piece:
// each has its reference, its sums and its O, and the two states are joined at the
// piece's end.  More groups (64 registers a thread) were slower, and so was a
// split of the registers between roles (setmaxnreg does not compile for them).
// Every mbarrier wait is bounded; a wait that runs out raises the error word and
// the CTA still counts its pieces, so that the workspace stays valid.
#include <cuda_fp16.h>

#include <atomic>
#include <type_traits>

#include "fd_internal.h"
#include "fd_kv4.cuh"
#include "fd_split.cuh"
#include "fd_tcgen05.cuh"

namespace fdk {
namespace {

constexpr int kTile = kPlanTile;                       // keys per tile: the M of S^T
constexpr int kTileBlocks = kTile / kKv4Tokens;
constexpr int kDescs = 4;                              // pieces announced ahead
constexpr int kSoftmax0 = 20;                          // first softmax warp
// p is held in fp16: the reference of the exponent lies kRefDown below the
// running maximum and moves when a score exceeds that maximum by kTau, so p <=
// 2^(kRefDown + kTau) = 2^15.  Its lower half is held kLoUp times up, in the same range: the
// smallest fp16 number there stands for 2^-44 of the maximum's weight, and p has its 22 bits
// down to 2^-23 of it.  (Not scaled, a weight below 2^-34 was 0 in O and not in l: 131072 such keys
// put out 8e-6 off.)
constexpr float kRefDown = 9.f, kTau = 6.f;
constexpr float kLoUp = 2048.f, kLoDown = 1.f / kLoUp;
// Tiles of a group whose O products add up in tensor memory before their sum moves to
// fp32 adds in shared memory.  An MMA's add drops bits instead of rounding, some 2^-25.6
// of the sum each and all one way: with 27 tiles in a row the outputs of 128k tokens were
// 4.2e-6 off (2-norm), with four 7.7e-7.  It costs 0.5 us of 40.
constexpr uint32_t kFlush = 4;
constexpr float kNoRef = -3.402823466e38f;  // of a head that has seen no key: no score lies below it

// Position in a ring of NB buffers: tile g is in buffer g % NB, its phase (g / NB) & 1.
template <uint32_t NB>
struct Ring {
  uint32_t i = 0, ph = 0;
  __device__ __forceinline__ void next() {
    if (++i == NB) {
      i = 0;
      ph ^= 1u;
    }
  }
  __device__ __forceinline__ void skip() {  // two tiles on
    i += 2;
    if (i >= NB) {
      i -= NB;
      ph ^= 1u;
    }
  }
};

struct KvPiece {
  int32_t b, vkv, tok_begin, tok_end, slot, len;
  int32_t more;  // the CTA goes on after it
  int32_t pad;
};

// Lengths and tile counts as in CtaTiles, with this kernel's charge for a piece:
// its end and the next one's start take a CTA about as long as four tiles (16 ragged
// sequences 35.9 us with the bf16 kernel's charge of 1.25 tiles, 32.2 so, 33.3 with
// three; 64 paged sequences of 8 heads a group 113 us, with a charge of six 116).
constexpr int kKv4PieceUnits = 4 * kTileUnits;
struct Kv4Tiles {
  const int32_t* pre;
  const int32_t* ln;
  int32_t ut, ul;
  int uniform;
  FD_HD int32_t piece() const { return uniform ? 0 : kKv4PieceUnits; }
  FD_HD int64_t prefix(int32_t b) const { return uniform ? (int64_t)b * pair_units(ut, 0) : pre[b]; }
  FD_HD int32_t tiles(int32_t b) const { return uniform ? ut : ceil_div(ln[b], kPlanTile); }
  FD_HD int32_t len(int32_t b) const { return uniform ? ul : ln[b]; }
};

// A piece to count, from the softmax warps to the O warp; whether it was its sequence's
// last, from the O warp back.
struct JoinPiece {
  int32_t last, b, vkv, npieces, first;
};

template <int D, int G>
struct K4 {
  static constexpr int kN = G <= 8 ? 16 : 2 * G;  // columns: hi of the G heads, then lo; the rest is not used
  // Buffers: K and V in tensor memory (64 columns each for D = 128), S there and p
  // in shared memory.  With two of each, a group's next tile waited for the
  // whole chain of its last one (S, softmax, O): 128k tokens 43 us, 41 so.
  // The softmax groups take alternate tiles, or, with 16 heads, whose scores, references
  // and sums do not fit in a thread's 72 registers, half of the heads of each tile
  // (131072 tokens of 4 KV heads 57.6 us by tiles, 48.6 by heads; 8 windows of 4 rows 37
  // and 30.5).
  static constexpr bool kByHead = G == 16;
  static constexpr uint32_t kStep = kByHead ? 1 : 2;  // from one tile of a group to its next
  static constexpr int kHeads = kByHead ? G / 2 : G;  // heads of a group
  static constexpr int kSGroups = 2, kSThreads = 128 * kSGroups, kThreads = 32 * kSoftmax0 + kSThreads;
  static constexpr uint32_t kKBufs = 3, kVBufs = G <= 8 ? 3 : 2, kSBufs = 4;
  static constexpr uint32_t kColK = 0, kColV = kColK + kKBufs * (D / 2), kColS = kColV + kVBufs * (kTile / 2),
                            kColO = kColS + kSBufs * kN;  // O: one per softmax group, or one of both
  static_assert(kColO + kSGroups * kN <= 512, "tensor memory");
  static constexpr int kStageBytes = kTileBlocks * kv4_block_bytes(D);
  static constexpr int kStages = D == 128 ? 8 : 16;  // a power of two
  static constexpr int kVWarps = D / 32;
  static constexpr int kQBytes = kN * D * 2;
  static constexpr int kPBytes = kN * kTile * 2;
  // byte offsets from a 1024-aligned base
  static constexpr int kQOff = 0;
  static constexpr int kPOff = kQOff + 2 * kQBytes;
  static constexpr int kStageOff = kPOff + kSBufs * kPBytes;
  static constexpr int kVsOff = kStageOff + kStages * kStageBytes;   // V scales as fp16: [8 warps][2][128]
  static constexpr int kRedOff = kVsOff + 8 * 2 * kTile * 2;          // [groups][16][4 warps] maxima, [16] references
  static constexpr int kFacOff = kRedOff + kSGroups * 80 * 4;         // [groups][16] score factors, [16] limits
  static constexpr int kEndOff = kFacOff + kSGroups * 32 * 4;         // a piece's end: see the softmax
  static constexpr int kJoinOff = kEndOff + 16 * 10 * 4;          // the groups' O: [groups][G][D]
  static constexpr int kMetaOff = kJoinOff + kSGroups * G * D * 4;    // per q buffer: factor[16], limit[16], least limit
  static constexpr int kMetaBytes = 2 * 16 * 4 + 16;  // ... and the sequence's pieces, their first CTA
  static constexpr int kDescOff = kMetaOff + 2 * kMetaBytes;
  static constexpr int kLenOff = kDescOff + kDescs * (int)sizeof(KvPiece);
  static constexpr int kPreOff = kLenOff + (kAutoMaxBatch + 4) * 4;
  static constexpr int kBarOff = kPreOff + (kAutoMaxBatch + 4) * 4;
  static constexpr int kBars = 2 * kStages + 2 * kDescs + 2 * kKBufs + 2 * kVBufs + 3 * kSBufs + 4 + 3;
  static constexpr int kFlagOff = kBarOff + kBars * 8;
  static constexpr int kLastOff = kFlagOff + 16;                      // two JoinPieces in turn
  static constexpr int kSmem = kLastOff + 48 + 1024;
  static_assert(kSmem <= 232448 && kSmem > 118784, "one CTA per SM: each takes all of tensor memory");
  static_assert(kStageOff % 128 == 0 && kQBytes % 1024 == 0 && kPBytes % 1024 == 0, "operand alignment");
  static_assert(kDescOff % 16 == 0 && kBarOff % 8 == 0, "alignment");
};

struct Kv4Params {
  SplitParams p;
  Kv4View kv;
};

// Byte offset of fp16 element (n, k) of a B operand: rows n of 64 k (128 bytes,
// swizzled), column blocks of N rows.
template <int N>
__device__ __forceinline__ uint32_t b_off(int n, int k) {
  return (uint32_t)(k >> 6) * (N * 128) + (uint32_t)n * 128 + (((uint32_t)(k >> 3) & 7u) ^ ((uint32_t)n & 7u)) * 16 +
         ((uint32_t)k & 7u) * 2;
}

__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<const __half2*>(&x); }
__device__ __forceinline__ uint32_t hmul2(uint32_t a, __half2 b) {
  const __half2 r = __hmul2(as_half2(a), b);
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Eight codes times their scales (s0 for the first two codes ...).
__device__ __forceinline__ void widen8(uint32_t w, __half2 s0, __half2 s1, __half2 s2, __half2 s3, uint32_t* out) {
  out[0] = hmul2(e2m1x2_f16x2<0>(w), s0);
  out[1] = hmul2(e2m1x2_f16x2<1>(w), s1);
  out[2] = hmul2(e2m1x2_f16x2<2>(w), s2);
  out[3] = hmul2(e2m1x2_f16x2<3>(w), s3);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t lds16u(uint32_t at) {
  unsigned short v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(at));
  return v;
}
__device__ __forceinline__ void sts128u(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// (x0, x1) = hi + lo / up in fp16, as packed pairs (x0 in the low half).  kPacked: the
// difference and its product two at a time, the same numbers (8 heads a group, 64 paged sequences
// 104.8 us against 107.1; 16 heads, 524288 tokens 217.7 against 209.0).
template <bool kPacked>
__device__ __forceinline__ void split_f16x2(float x0, float x1, uint32_t& hi, uint32_t& lo, float up = 1.f) {
  const __half2 h = __floats2half2_rn(x0, x1);
  const float2 f = __half22float2(h);
  float2 d;
  if constexpr (kPacked)
    d = fma2(fma2(f, make_float2(-1.f, -1.f), make_float2(x0, x1)), make_float2(up, up), make_float2(0.f, 0.f));
  else
    d = make_float2((x0 - f.x) * up, (x1 - f.y) * up);
  const __half2 r = __floats2half2_rn(d.x, d.y);
  hi = *reinterpret_cast<const uint32_t*>(&h);
  lo = *reinterpret_cast<const uint32_t*>(&r);
}

// Reductions over the warp of G values a lane, G a power of two: result h is in
// v[0] of the lanes [h * 32 / G, (h + 1) * 32 / G).  Each step halves the values as
// well as the lanes that a result is spread over.
template <int G, int NV, class Op>
__device__ __forceinline__ void warp_reduce(float (&v)[NV], int lane, Op op) {
  int off = 16;
#pragma unroll
  for (int n = G / 2; n > 0; n /= 2, off /= 2) {
    const bool upper = lane & off;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const float send = upper ? v[i] : v[i + n], keep = upper ? v[i + n] : v[i];
      v[i] = op(keep, __shfl_xor_sync(0xffffffffu, send, off));
    }
  }
#pragma unroll
  for (; off > 0; off /= 2) v[0] = op(v[0], __shfl_xor_sync(0xffffffffu, v[0], off));
}

// Barrier of a softmax group (ids from 2, 128 threads) or of all of them (id 1)
// that counts raised predicates.
__device__ __forceinline__ uint32_t vote(uint32_t id, uint32_t threads, bool pred) {
  uint32_t n;
  __syncwarp();
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.popc.u32 %0, %2, %3, p;\n\t}"
               : "=r"(n)
               : "r"((uint32_t)pred), "r"(id), "r"(threads)
               : "memory");
  return n;
}

// One lane of a converged warp, known as such to the compiler: the operands of
// the MMAs then stay in uniform registers (with a lane test each MMA took 70
// issue cycles to set up, 128k tokens 70 us against 52).
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Join of the partial states of one head by one warp: M = max m, weights
// exp(m_k - M) over the states with l > 0, out = sum w O / L, lse = M + ln L.
// State k is partial index base + k * stride.  Thirty-two states' weights at a
// time, their O slices in batches of eight loads, in a fixed order.  The first
// thirty-two states' m and l and the first batch are asked for at once: one
// trip to L2 for few states (16 heads of 9 states on 8 warps took 14000 cycles with the loads one after another, 10000 so).
template <int D>
__device__ __forceinline__ void join_states(const SplitParams& p, size_t base, size_t stride, int count, float* out,
                                            float* lse, int lane) {
  constexpr int E = D / 32;
  float v[8][E];
  const auto load_batch = [&](int k0) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
#pragma unroll
      for (int i = 0; i < E; ++i) v[j][i] = 0.f;
      if (k0 + j < count) load_slice<D>(p.o_part + (base + (k0 + j) * stride) * D + lane * E, v[j]);
    }
  };
  float m = -INFINITY, l = 0.f;
  if (lane < count) {
    m = __ldcg(p.m_part + base + lane * stride);
    l = __ldcg(p.l_part + base + lane * stride);
  }
  load_batch(0);
  float mx = l > 0.f ? m : -INFINITY;
  for (int k = lane + 32; k < count; k += 32)
    if (__ldcg(p.l_part + base + k * stride) > 0.f) mx = fmaxf(mx, __ldcg(p.m_part + base + k * stride));
  mx = warp_max(mx);
  float acc[E], L = 0.f;
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = 0.f;
  if (mx != -INFINITY) {
#pragma unroll 1
    for (int k0 = 0; k0 < count; k0 += 8) {
      if (k0 > 0) {
        if (k0 % 32 == 0) {
          l = 0.f;
          if (k0 + lane < count) {
            m = __ldcg(p.m_part + base + (k0 + lane) * stride);
            l = __ldcg(p.l_part + base + (k0 + lane) * stride);
          }
        }
        load_batch(k0);
      }
      float w = 0.f;
      if (l > 0.f) w = exp2f((m - mx) * kLog2e);
      if (k0 % 32 == 0) L = fmaf(w, l, L);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float wj = __shfl_sync(0xffffffffu, w, (k0 + j) & 31);
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = fmaf(wj, v[j][i], acc[i]);
      }
    }
    L = warp_sum(L);
  }
#pragma unroll
  for (int i = 0; i < E; ++i) acc[i] = mx == -INFINITY ? 0.f : acc[i] / L;
  if constexpr (E == 4)
    *reinterpret_cast<float4*>(out + lane * E) = make_float4(acc[0], acc[1], acc[2], acc[3]);
  else
    *reinterpret_cast<float2*>(out + lane * E) = make_float2(acc[0], acc[1]);
  if (lse && lane == 0) *lse = mx == -INFINITY ? -INFINITY : mx + logf(L);
}

// try_wait that lets the hardware suspend the warp for up to 20 us: with many
// warps waiting at any time, polling took a fifth of the issue slots.
__device__ __forceinline__ bool mbar_sleep_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity), "r"(20000u)
      : "memory");
  return ok != 0;
}

// The part of a wait that is not complete at once, out of the way of the tile loops.
// One that runs out ends the CTA's others.
__device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, volatile int* abort_flag, unsigned long long limit) {
  const unsigned long long t0 = global_ns();
  while (!*abort_flag) {
    if (mbar_sleep_wait(bar, parity)) return true;
    if (global_ns() - t0 > limit) *abort_flag = 1;
  }
  return false;
}

// Waits of one warp (all lanes together): false when the CTA aborts or the limit passes.
struct Waiter {
  volatile int* abort_flag;
  unsigned long long limit;
  __device__ __forceinline__ bool one(uint64_t* bar, uint32_t parity) const {
    return mbar_sleep_wait(bar, parity) || wait_slow(bar, parity, abort_flag, limit);
  }
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) const {
    return __all_sync(0xffffffffu, one(bar, parity));
  }
  // Two barriers, one vote.  (The phase before a barrier's first counts as complete: a
  // buffer that nothing has used yet is free.)
  __device__ __forceinline__ bool both(uint64_t* a, uint32_t pa, uint64_t* b, uint32_t pb) const {
    return __all_sync(0xffffffffu, one(a, pa) && one(b, pb));
  }
};

// Copies of every second tile j, j + 2, ... of a paged piece, by one warp; tile j is the
// CTA's tile g.  Returns how many it dealt with: a wait for a free stage may run out.
// A warp starts a bulk copy in some 90 cycles, and pages of sixteen tokens need eight
// a tile, so two warps take turns (524288 tokens of 8 heads 126 us, with one warp 168, with one
// warp's lanes and 16-byte copies 182; 64 sequences of 512 to 16384 tokens 105, 114 with one).
// Blocks of a tile that follow one another in the pool go in one copy.
template <int D, int kStages>
__device__ __forceinline__ int32_t copy_paged(const Kv4View& kv, unsigned* err, uint8_t* stages, uint64_t* full, Waiter wait,
                                           int32_t stall_it, int32_t b, int32_t kvh, int32_t tok_begin, int32_t tok_end,
                                           uint32_t g, int32_t j) {
  constexpr int kBytes = kv4_block_bytes(D);
  const int lane = threadIdx.x & 31;
  uint64_t* empty = full + kStages;
  const uint8_t* pool = kv.kv;
  const int32_t n = ceil_div(tok_end - tok_begin, kTile), num_pages = kv.num_pages, Hkv = kv.Hkv;
  const int32_t blk0 = tok_begin / kKv4Tokens, blk1 = ceil_div(tok_end, kKv4Tokens);
  // Lane k has block k of this warp's next four tiles at hand (its number in the pool, kNoBlock
  // for a page outside it), and the table entry of its block of the four after is in flight.
  constexpr uint32_t kNoBlock = 0xffffffffu;  // a pool has fewer: 2^32 blocks are 4.9 TB
  uint32_t cur = 0, firsts = 0, bads = 0;     // of four tiles: blocks that start a copy, blocks outside the pool
  const int32_t* trow = kv.block_table + (size_t)b * kv.max_pages;
  int32_t blk = blk0 + (j + 2 * (lane / kTileBlocks)) * kTileBlocks + lane % kTileBlocks;
  // the entry's place in the table, the block in the page; sixty-four blocks on
  const int32_t ppb = kv.page_size / kKv4Tokens, step_q = 64 / ppb, step_r = 64 - step_q * ppb;
  int32_t at = blk / ppb, rem = blk - at * ppb, page = 0;
  const auto load_page = [&] { page = blk < blk1 ? __ldg(trow + at) : 0; };
  const auto take_page = [&] {
    cur = page >= 0 && page < num_pages ? ((uint32_t)page * (uint32_t)Hkv + kvh) * ppb + rem : kNoBlock;
    const uint32_t before = __shfl_up_sync(0xffffffffu, cur, 1);
    firsts = __ballot_sync(0xffffffffu, lane % kTileBlocks == 0 || cur != before + 1);
    bads = __ballot_sync(0xffffffffu, cur == kNoBlock && blk < blk1);
    blk += 64;
    at += step_q;
    rem += step_r;
    if (rem >= ppb) {
      rem -= ppb;
      ++at;
    }
    load_page();
  };
  load_page();
  take_page();
  int32_t done = 0;
  for (; j < n; j += 2, g += 2, ++done) {
    const int32_t left = blk1 - (blk0 + j * kTileBlocks), nblk = left < kTileBlocks ? left : kTileBlocks;
    const uint32_t st = g % kStages;
    if (!wait.warp(empty + st, ((g / kStages) & 1) ^ 1)) break;
    if (g != (uint32_t)stall_it) {
      uint8_t* dst = stages + st * (kTileBlocks * kBytes);
      const int k0 = (done & 3) * kTileBlocks;
      const uint32_t valid = (1u << nblk) - 1, bad = bads >> k0 & valid;
      const int k = lane - k0;  // this lane's block of the tile
      uint32_t starts = firsts >> k0 & valid;
      if (__builtin_expect(bad != 0, 0)) {
        // keys of score 0 and value 0 in its place
        if (k >= 0 && k < kTileBlocks && bad >> k & 1) {
          raise_error(err, kErrBadIndex);
          for (int i = 0; i < kBytes; i += 16) sts128u(smem_addr(dst) + k * kBytes + i, make_uint4(0, 0, 0, 0));
          // before a later copy into this stage
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        starts = (starts | bad << 1) & valid & ~bad;  // a block after a bad one starts a copy
        __syncwarp();
      }
      const uint8_t* from = pool + (uint64_t)cur * kBytes;
      if (starts == valid) {  // one a block: a constant size is quicker to issue
        if (k >= 0 && k < nblk) bulk_load(dst + k * kBytes, from, kBytes, full + st);
      } else if (k >= 0 && k < kTileBlocks && starts >> k & 1) {
        const uint32_t stops = starts | bad | ~valid;  // the next copy, a bad block, the tile's end
        bulk_load(dst + k * kBytes, from, __ffs(stops >> (k + 1)) * kBytes, full + st);
      }
      if (lane == 0) mbar_arrive_expect_tx(full + st, __popc(valid & ~bad) * kBytes);
      __syncwarp();
    }
    if ((done & 3) == 3) take_page();
  }
  return done;
}

// The tiles that a warp copied last: bit i of `mine` is tile last - i.
struct Copied {
  uint32_t last = 0, mine = 0;
  // `count` tiles g, g + step, ...
  __device__ __forceinline__ void add(uint32_t g, uint32_t step, int32_t count) {
    if (count <= 0) return;
    const uint32_t to = g + step * (uint32_t)(count - 1), by = to - last, span = to - g;
    mine = (by < 32 ? mine << by : 0u) | ((step == 1 ? 0xffffffffu : 0x55555555u) & (span < 31 ? (2u << span) - 1 : 0xffffffffu));
    last = to;
  }
  // Stay until those in flight have landed; `end` tiles were copied by all warps.
  template <int kStages>
  __device__ __forceinline__ void land(uint64_t* full, uint32_t end, int32_t stall_it, unsigned long long limit, unsigned* err) const {
    for (uint32_t i = 0; i < (uint32_t)kStages && i <= last; ++i) {
      const uint32_t g = last - i;
      if (!(mine >> i & 1) || g + kStages < end || g == (uint32_t)stall_it) continue;
      if (!mbar_wait_for(full + g % kStages, (g / kStages) & 1, limit)) raise_error(err, kErrTimeout);
    }
  }
};

template <int D, int G>
__global__ void __launch_bounds__(K4<D, G>::kThreads, 1) fd_kv4_kernel(const __grid_constant__ Kv4Params pp) {
  using C = K4<D, G>;
  constexpr int N = C::kN;
  constexpr uint32_t kSG = C::kSGroups, kStep = C::kStep;
  const SplitParams& p = pp.p;
  const Kv4View& kv = pp.kv;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kBarOff);
  uint64_t* empty = full + C::kStages;
  uint64_t* desc_full = empty + C::kStages;
  uint64_t* desc_empty = desc_full + kDescs;
  uint64_t* k_ready = desc_empty + kDescs;  // [kKBufs] K is in tensor memory
  uint64_t* k_free = k_ready + C::kKBufs;   // S of it has been computed
  uint64_t* v_ready = k_free + C::kKBufs;   // [kVBufs]
  uint64_t* v_free = v_ready + C::kVBufs;
  uint64_t* s_full = v_free + C::kVBufs;    // [kSBufs]
  uint64_t* p_ready = s_full + C::kSBufs;   // [kSBufs] p is there, and S has been read
  uint64_t* p_free = p_ready + C::kSBufs;   // [kSBufs] O with it has been computed
  uint64_t* q_ready = p_free + C::kSBufs;   // [2]
  uint64_t* q_free = q_ready + 2;           // [2]
  uint64_t* drain = q_free + 2;
  uint64_t* part_done = drain + 1;          // a piece's partial state is written
  uint64_t* join_known = part_done + 1;     // ... and counted: whether it was its sequence's last
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kFlagOff);
  volatile int* last_flag = abort_flag + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kFlagOff + 8);
  KvPiece* descs = reinterpret_cast<KvPiece*>(smem + C::kDescOff);
  int32_t* lens = reinterpret_cast<int32_t*>(smem + C::kLenOff);
  int32_t* pre = reinterpret_cast<int32_t*>(smem + C::kPreOff);

  if (warp == 3) {  // arrivals that each barrier counts, one barrier a lane
    constexpr uint32_t kV = C::kVWarps;
    for (int i = lane; i < C::kBars; i += 32) {
      uint64_t* at = full + i;
      uint32_t n = 1;
      if (at >= empty && at < desc_full) n = 4 + kV;
      if (at >= desc_empty && at < k_ready) n = 2 + 1 + 8 + 2 * kV + 4 * C::kSGroups;
      if (at >= k_ready && at < k_free) n = 4;
      if (at >= v_ready && at < v_free) n = kV;
      if (at >= p_ready && at < p_free) n = C::kByHead ? 8 : 4;
      if (at >= q_free && at < drain) n = 1 + 4 * C::kSGroups;
      if (at == drain) n = 2;
      if (at == part_done) n = 4 * C::kSGroups;
      mbar_init(at, n);
    }
    if (lane == 0) *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) tmem_alloc_all(smem_addr(tmem_slot));
  pdl_launch_dependents();
  if (p.seq_lens != nullptr) pdl_wait();
  Kv4Tiles tl;
  tl.pre = pre;
  tl.ln = lens;
  tl.ul = p.max_len;
  tl.ut = ceil_div(p.max_len, kPlanTile);
  tl.uniform = 1;
  if (p.n_splits == 0 && p.seq_lens != nullptr) {
    tl.uniform = 0;
    for (int b = tid; b < p.B; b += C::kThreads) lens[b] = clamp_len(__ldg(p.seq_lens + b), p.max_len);
    cta_sync();
    if (warp == 0) {
      const int per = ceil_div(p.B, 32);
      const int lo = lane * per;
      const int hi = lo + per < p.B ? lo + per : p.B;
      int sum = 0;
      for (int b = lo; b < hi; ++b) sum += (int)pair_units(ceil_div(lens[b], kPlanTile), kKv4PieceUnits);
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      int run = incl - sum;
      for (int b = lo; b < hi; ++b) {
        pre[b] = run;
        run += (int)pair_units(ceil_div(lens[b], kPlanTile), kKv4PieceUnits);
      }
      if (lane == 31) pre[p.B] = incl;
    }
  }
  // The producer (warp 0, which has the prefix sums) walks to its first piece
  // before it meets the others here.
  uint32_t tmem = 0;
  if (warp != 0) {
    tmem_fence_before();
    cta_sync();
    tmem_fence_after();
    tmem = *tmem_slot;
  } else {
    __syncwarp();
  }
  const int64_t total = (int64_t)p.hv * tl.prefix(p.B);
  const Waiter wait{abort_flag, wait_limit(p)};
  // Pieces are announced, counted and joined after an abort, too, or the workspace's
  // counters would be left set: these waits outlast the one that ran out.
  const unsigned long long patience = 4 * wait.limit;
  bool ok = true;

  // Every role but the producer takes the announced pieces in order.
  const auto next_piece = [&](uint32_t e, KvPiece& pc) {
    const uint32_t sl = e % kDescs;
    const bool got = __all_sync(0xffffffffu, mbar_wait_for(desc_full + sl, (e / kDescs) & 1, patience));
    if (got) pc = descs[sl];
    __syncwarp();
    if (got && lane == 0) mbar_arrive(desc_empty + sl);
    return got && pc.b >= 0;
  };
  // Pieces of the piece's sequence over all CTAs, and the first CTA that holds one.
  const auto pieces_of = [&](const KvPiece& pc, int32_t& first) {
    first = 0;
    if (p.n_splits != 0) return p.n_splits;
    int32_t last;
    balanced_pair_ctas(tl, p.hv, total, balanced_ctas(total, (int32_t)gridDim.x), pc.b, pc.vkv, &first, &last);
    return last - first + 1;
  };
  // Count the piece (one thread); true for the last of its sequence.
  const auto arrive_last = [&](const KvPiece& pc, int32_t npieces) {
    return atomic_add_acq_rel(p.counters + pc.b * p.hv + pc.vkv, 1) == npieces - 1;
  };
  // Join the sequence's states: heads first, first + step, ...; one warp each.
  const auto join_piece = [&](int32_t b, int32_t vkv, int32_t npieces, int32_t first, int h0, int step) {
    Groups gr;
    gr.g = p.g;
    gr.gpad = p.gpad;
    gr.nsub = p.nsub;
    gr.hv = p.hv;
    int32_t head0, nh;
    vkv_heads(gr, vkv, &head0, &nh);
    const bool balanced = p.n_splits == 0;
    const size_t base = balanced ? (size_t)(b * p.hv + vkv + first) * p.gpad : ((size_t)b * p.Hq + head0) * p.n_splits;
    const size_t hs = balanced ? 1 : (size_t)p.n_splits, stride = balanced ? p.gpad : 1;
    for (int h = h0; h < nh; h += step) {
      const size_t row = (size_t)b * p.Hq + head0 + h;
      join_states<D>(p, base + h * hs, stride, npieces, p.out + row * D, p.lse ? p.lse + row : nullptr, lane);
    }
    if (h0 == 0 && lane == 0) p.counters[b * p.hv + vkv] = 0;  // ready for the next call
  };
  JoinPiece* counted = reinterpret_cast<JoinPiece*>(smem + C::kLastOff);
  const auto tiles_of = [](const KvPiece& pc) { return ceil_div(pc.tok_end - pc.tok_begin, kTile); };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    Groups gr;
    gr.g = p.g;
    gr.gpad = p.gpad;
    gr.nsub = p.nsub;
    gr.hv = p.hv;
    const uint64_t stream_policy = policy_evict_first();
    const bool balanced = p.n_splits == 0;
    const int32_t used = balanced ? balanced_ctas(total, (int32_t)gridDim.x) : 0;
    const bool part = balanced && (int32_t)blockIdx.x < used;  // this CTA has a share of the plan
    BalancedWalk<Kv4Tiles> walk(tl, p.B, p.hv, part ? total : 0, part ? used : 1, part ? (int32_t)blockIdx.x : 0);
    Piece pc;
    bool have;
    if (balanced) {
      have = walk.next(pc);
    } else {
      have = true;
      pc.b = blockIdx.x / p.hv;
      pc.vkv = blockIdx.x % p.hv;
      pc.slot = blockIdx.y;
      pc.len = p.seq_lens ? clamp_len(__ldg(p.seq_lens + pc.b), p.max_len) : p.max_len;
      const int64_t lo = (int64_t)pc.slot * p.split_tokens, hi = lo + p.split_tokens;
      pc.tok_begin = (int32_t)(lo < pc.len ? lo : pc.len);
      pc.tok_end = (int32_t)(hi < pc.len ? hi : pc.len);
    }
    cta_sync();
    uint32_t it = 0, e = 0;  // tiles, pieces
    Ring<C::kStages> st;  // of a contiguous cache
    Copied copied;
    bool live = true;  // the other roles still take pieces
    pdl_wait();
    const auto announce = [&](const KvPiece& d) {
      const uint32_t sl = e % kDescs;
      bool r = true;
      if (lane == 0) {
        r = mbar_wait_for(desc_empty + sl, ((e / kDescs) & 1) ^ 1, patience);
        if (r) {
          descs[sl] = d;
          mbar_arrive(desc_full + sl);
        }
      }
      ++e;
      return (bool)__shfl_sync(0xffffffffu, r, 0);
    };
    for (; have; have = balanced && walk.next(pc)) {
      KvPiece d;
      d.b = pc.b;
      d.vkv = pc.vkv;
      d.tok_begin = pc.tok_begin;
      d.tok_end = pc.tok_end;
      d.slot = pc.slot;
      d.len = pc.len;
      d.more = balanced && !walk.done() ? 1 : 0;
      live = announce(d);
      if (!live) break;
      if (!ok) continue;
      const int32_t kvh = kv_head_of_vkv(gr, pc.vkv), n = tiles_of(d);
      if (kv.paged) {  // the even tiles; the q warp copies the odd ones
        const int32_t mine = (n + 1) / 2;
        const int32_t done = copy_paged<D, C::kStages>(kv, p.err, smem + C::kStageOff, full, wait, p.stall_it, pc.b, kvh,
                                                       pc.tok_begin, pc.tok_end, it, 0);
        copied.add(it, 2, done);
        if (done != mine) ok = false;
        it += n;
        continue;
      }
      const uint8_t* base =
          kv.kv + (((int64_t)pc.b * kv.Hkv + kvh) * kv.cap_blocks + pc.tok_begin / kKv4Tokens) * kv4_block_bytes(D);
      const int32_t blocks = ceil_div(pc.tok_end, kKv4Tokens) - pc.tok_begin / kKv4Tokens;
      const uint32_t it0 = it;
      for (int32_t j = 0; j < n; ++j, ++it, st.next()) {
        const int32_t nblk = blocks - j * kTileBlocks < kTileBlocks ? blocks - j * kTileBlocks : kTileBlocks;
        if (!wait.warp(empty + st.i, st.ph ^ 1)) {
          ok = false;
          break;
        }
        if (lane == 0 && it != (uint32_t)p.stall_it) {
          const uint32_t bytes = (uint32_t)nblk * kv4_block_bytes(D);
          mbar_arrive_expect_tx(full + st.i, bytes);
          const uint8_t* src = base + (int64_t)j * C::kStageBytes;
          asm volatile(
              "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(
                  sbase + C::kStageOff + st.i * C::kStageBytes),
              "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(full + st.i)), "l"(stream_policy)
              : "memory");
        }
      }
      copied.add(it0, 1, (int32_t)(it - it0));
    }
    if (live) {
      KvPiece d;
      d.b = -1;
      live = announce(d);
    }
    if (!ok || !live) {
      raise_error(p.err, kErrTimeout);
      *abort_flag = 1;
    }
    if (lane == 0) copied.land<C::kStages>(full, ok && live ? it : 0, p.stall_it, wait.limit, p.err);
  } else if (warp < 3) {
    // ------------------------------------------------------------ MMA issue
    // Every branch and operand here is uniform over the warp as the compiler sees it
    // (votes and shuffles): only then do the MMAs take their operands from uniform
    // registers as they are (18 cycles each to issue; 70 to 130 otherwise).
    constexpr uint32_t s_desc = f16_instr_desc(kTile, N), o_desc = f16_instr_desc(kTile, N, true);
    const uint32_t base = uniform(tmem), sb = uniform(sbase);
    const bool is_s = uniform(warp) == 1;
    uint32_t g = 0, f = 0;  // tiles, pieces with tiles
    Ring<C::kKBufs> kr;
    Ring<C::kVBufs> vr;
    Ring<C::kSBufs> sr;
    uint32_t sg = 0;  // the softmax group of tile g
    // The O warp counts the pieces that the CTA goes on after, so that the softmax warps need
    // not wait for the atomic: they join a sequence at their next piece's end.  Their first p
    // of that piece comes later than the end of the last.
    bool due = false;
    uint32_t parts = 0;
    const auto count_piece = [&] {
      const bool done = __all_sync(0xffffffffu, mbar_wait_for(part_done, parts & 1, patience));
      if (!done) ok = false;
      if (lane == 0) {
        JoinPiece& j = counted[parts & 1];
        j.last = done && j.npieces != 1 &&
                 atomic_add_acq_rel(p.counters + j.b * p.hv + j.vkv, 1) == j.npieces - 1;
        mbar_arrive(join_known);
      }
      __syncwarp();
      ++parts;
    };
    for (uint32_t e = 0;; ++e) {
      KvPiece pc;
      const bool got = __all_sync(0xffffffffu, next_piece(e, pc));
      const int32_t n = got && ok ? (int32_t)uniform(tiles_of(pc)) : 0;
      if (due) count_piece();
      if (!got) break;
      due = !is_s && p.counters != nullptr && uniform(pc.more) != 0;
      if (n == 0) continue;
      if (is_s && !wait.warp(q_ready + (f & 1), (f >> 1) & 1)) ok = false;
      for (int32_t j = 0; ok && j < n; ++j, ++g) {
        if (is_s) {
          // K is there, and the softmax has read what the S buffer held
          if (!wait.both(k_ready + kr.i, kr.ph, p_ready + sr.i, sr.ph ^ 1)) {
            ok = false;
            break;
          }
          tmem_fence_after();
          const uint32_t qb = f & 1;
          if (elect_one()) {
            // A is eight columns on per K = 16 step, B 32 bytes within a swizzled row, then
            // the next column block
            const uint32_t d = base + C::kColS + sr.i * N, a = base + C::kColK + kr.i * (D / 2),
                           b = sb + C::kQOff + qb * C::kQBytes;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
              mma_ts(d, a + kk * 8, b_desc(b + (kk >> 2) * (N * 128) + (kk & 3) * 32), s_desc, kk > 0);
            mma_commit(smem_addr(s_full + sr.i));
            mma_commit(smem_addr(k_free + kr.i));
            if (j == n - 1) mma_commit(smem_addr(q_free + qb));
          }
        } else {
          if (!wait.both(v_ready + vr.i, vr.ph, p_ready + sr.i, sr.ph)) {
            ok = false;
            break;
          }
          tmem_fence_after();
          if (elect_one()) {
            const bool fresh = j / (int32_t)kStep % (int32_t)kFlush == 0;  // a new sum
            const uint32_t d = base + C::kColO + sg * N, a = base + C::kColV + vr.i * (kTile / 2),
                           b = sb + C::kPOff + sr.i * C::kPBytes;
#pragma unroll
            for (int kk = 0; kk < kTile / 16; ++kk)
              mma_ts(d, a + kk * 8, b_desc_n<16 * kTile>(b + kk * 256), o_desc, kk > 0 || !fresh);
            mma_commit(smem_addr(p_free + sr.i));
            mma_commit(smem_addr(v_free + vr.i));
          }
        }
        __syncwarp();
        kr.next();
        vr.next();
        sr.next();
        if (++sg == kStep) sg = 0;
      }
      ++f;
    }
    if (!ok) {
      raise_error(p.err, kErrTimeout);
      *abort_flag = 1;
    }
    // every MMA has finished before tensor memory goes back
    if (elect_one()) {
      mma_commit(smem_addr(drain));
      if (!mbar_wait_for(drain, 0, wait.limit)) raise_error(p.err, kErrTimeout);
    }
    __syncwarp();
  } else if (warp < 4) {
    // ------------------------------------------------------------ q
    Groups gr;
    gr.g = p.g;
    gr.gpad = p.gpad;
    gr.nsub = p.nsub;
    gr.hv = p.hv;
    uint32_t f = 0, it = 0;
    Copied copied;
    const auto prepare = [&](const KvPiece& pc) {
      const uint32_t qb = f & 1;
      if (f >= 2 && !wait.warp(q_free + qb, ((f >> 1) & 1) ^ 1)) return false;
      int32_t head0, nh;
      vkv_heads(gr, pc.vkv, &head0, &nh);
      const RowLimits rl{head0, nh, pc.len, p.n_q, p.causal};
      float* factor = reinterpret_cast<float*>(smem + C::kMetaOff + qb * C::kMetaBytes);
      const uint32_t qs = sbase + C::kQOff + qb * C::kQBytes;
      // A lane holds eight channels, so a pass of the warp takes 256 / D heads; two passes'
      // loads at a time, one pair of passes ahead (one head a pass and one ahead: 16 heads
      // took 10000 cycles before the first S).
      constexpr int kLanes = D / 8, kHeads = 32 / kLanes;
      const int c8 = lane % kLanes * 8, hl = lane / kLanes;
      float x[2][8], nx[2][8];
      const auto load_heads = [&](int h0, float (&to)[2][8]) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          const int h = h0 + a * kHeads + hl;
          float4 lo = make_float4(0.f, 0.f, 0.f, 0.f), hi = lo;
          if (h < nh) {
            const float4* row = reinterpret_cast<const float4*>(p.q + ((size_t)pc.b * p.Hq + head0 + h) * D + c8);
            lo = __ldcg(row);
            hi = __ldcg(row + 1);
          }
          to[a][0] = lo.x; to[a][1] = lo.y; to[a][2] = lo.z; to[a][3] = lo.w;
          to[a][4] = hi.x; to[a][5] = hi.y; to[a][6] = hi.z; to[a][7] = hi.w;
        }
      };
      const auto put_heads = [&](int h, float (&x)[8]) {
        uint32_t big = 0;  // a NaN is the largest
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[i] *= p.qk_scale;
          big = max(big, __float_as_uint(fabsf(x[i])));
        }
#pragma unroll
        for (int o = kLanes / 2; o > 0; o /= 2) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
        // 2^e <= big < 2^(e + 1): q times 2^(13 - e) fills fp16's range.  The factor of a
        // score is then a power of two, so the product with it is exact: its difference
        // from a reference may be fused, and is never above zero for the largest score.
        int ex = (int)(big >> 23) - 127;
        if (big == 0 || ex > 127) ex = 13;
        ex = ex < -80 ? -80 : ex;  // 2^(13 - ex) is a float
        const float up = pow2i(13 - ex);
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) split_f16x2<!C::kByHead>(x[2 * i] * up, x[2 * i + 1] * up, hi[i], lo[i]);
        if (G % kHeads == 0 || h < G) {
          sts128u(qs + b_off<N>(h, c8), make_uint4(hi[0], hi[1], hi[2], hi[3]));
          sts128u(qs + b_off<N>(G + h, c8), make_uint4(lo[0], lo[1], lo[2], lo[3]));
          if (c8 == 0) factor[h] = h < nh ? pow2i(kv.k_exp) * pow2i(ex - 13) : 0.f;
        }
      };
      load_heads(0, x);
#pragma unroll 1
      for (int h0 = 0; h0 < G; h0 += 2 * kHeads) {
        if (h0 + 2 * kHeads < G) load_heads(h0 + 2 * kHeads, nx);
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          if (h0 + a * kHeads < G) put_heads(h0 + a * kHeads + hl, x[a]);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[a][i] = nx[a][i];
        }
      }
      {  // the keys that each head sees, and the fewest
        const int32_t limit = lane < nh ? rl(lane) : 0x7fffffff;
        if (lane < 16) reinterpret_cast<int32_t*>(factor + 16)[lane] = limit;
        int32_t least = limit;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) least = min(least, __shfl_xor_sync(0xffffffffu, least, o));
        if (lane == 0) {
          int32_t first;
          int32_t* meta = reinterpret_cast<int32_t*>(factor + 32);
          meta[1] = pieces_of(pc, first);
          meta[2] = first;
          meta[0] = least;
        }
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(q_ready + qb);
      ++f;
      return true;
    };
    pdl_wait();
    KvPiece pc;
    for (uint32_t e = 0; next_piece(e, pc); ++e) {
      const int32_t n = tiles_of(pc);
      if (ok && n > 0 && !prepare(pc)) ok = false;
      if (ok && kv.paged && n > 1) {  // the odd tiles
        const int32_t done = copy_paged<D, C::kStages>(kv, p.err, smem + C::kStageOff, full, wait, p.stall_it, pc.b,
                                                       kv_head_of_vkv(gr, pc.vkv), pc.tok_begin, pc.tok_end, it + 1, 1);
        copied.add(it + 1, 2, done);
        if (done != n / 2) ok = false;
      }
      it += n;
    }
    if (!ok) {
      raise_error(p.err, kErrTimeout);
      *abort_flag = 1;
    }
    if (lane == 0) copied.land<C::kStages>(full, ok ? it : 0, p.stall_it, wait.limit, p.err);
  } else if (warp < 12) {
    // ------------------------------------------------------------ K
    const int quad = warp & 3;
    const uint32_t group = (uint32_t)(warp - 4) >> 2;
    const int row = lane & 15;
    const uint32_t krow = (uint32_t)(quad * 2 + (lane >> 4)) * kv4_block_bytes(D);
    const uint32_t sw = kv4_swizzle(D, row);
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    uint32_t g = group, e = 0, g1 = 0;  // this group's next tile, the end of the piece
    Ring<C::kKBufs> kr;
    if (group) kr.next();
    KvPiece pc;
    for (; next_piece(e, pc); ++e) {
      if (ok) g1 += tiles_of(pc);
      for (; ok && g < g1; g += 2, kr.skip()) {
        const uint32_t st = g % C::kStages;
        if (!wait.both(full + st, g / C::kStages & 1, k_free + kr.i, kr.ph ^ 1)) {
          ok = false;
          break;
        }
        tmem_fence_after();
        const uint32_t base = sbase + C::kStageOff + st * C::kStageBytes + krow;
#pragma unroll 1
        for (int c = 0; c < D / 32; ++c) {
          const uint4 w = lds128u(base + row * (D / 2) + ((c ^ sw) << 4));
          const uint32_t b2 = e4m3x2_f16x2(lds16u(base + kv4_ks_off(D) + row * (D / 16) + 2 * c));
          const __half2 sc = *reinterpret_cast<const __half2*>(&b2);
          const __half2 s0 = __low2half2(sc), s1 = __high2half2(sc);
          uint32_t r[16];
          widen8(w.x, s0, s0, s0, s0, r);
          widen8(w.y, s0, s0, s0, s0, r + 4);
          widen8(w.z, s1, s1, s1, s1, r + 8);
          widen8(w.w, s1, s1, s1, s1, r + 12);
          tmem_store16(tmem + lanes + C::kColK + kr.i * (D / 2) + c * 16, r);
        }
        tmem_wait_stores();
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(k_ready + kr.i);
          mbar_arrive(empty + st);
        }
      }
    }
    if (!ok) {
      raise_error(p.err, kErrTimeout);
      *abort_flag = 1;
    }
  } else if (warp < 20) {
    // ------------------------------------------------------------ V
    const int quad = warp & 3;
    const uint32_t group = (uint32_t)(warp - 12) >> 2;
    if (quad < C::kVWarps) {
      const int d = quad * 32 + lane;
      const uint32_t lanes = (uint32_t)(quad * 32) << 16;
      const uint32_t vs = sbase + C::kVsOff + (warp - 12) * (2 * kTile * 2);
      const int sblk = (lane >> 1) & 7, stok = sblk * 16 + (lane & 1) * 8;  // the scales that this lane converts
      uint32_t g = group, e = 0, g1 = 0;
      Ring<C::kVBufs> vr;
      if (group) vr.next();
      KvPiece pc;
      for (; next_piece(e, pc); ++e) {
        const uint32_t g0 = g1;
        if (ok) g1 += tiles_of(pc);
        for (; ok && g < g1; g += 2, vr.skip()) {
          const uint32_t st = g % C::kStages;
          if (!wait.both(full + st, g / C::kStages & 1, v_free + vr.i, vr.ph ^ 1)) {
            ok = false;
            break;
          }
          tmem_fence_after();
          const uint32_t base = sbase + C::kStageOff + st * C::kStageBytes;
          {
            // The warp's two groups of sixteen channels, 128 tokens: scales to fp16,
            // 0 for tokens past the valid ones (0 * anything finite is 0, and codes are finite).
            const uint2 b = lds64u(base + sblk * kv4_block_bytes(D) + kv4_vs_off(D) + (quad * 2 + (lane >> 4)) * 16 +
                                   (lane & 1) * 8);
            uint32_t x[4] = {e4m3x2_f16x2(b.x), e4m3x2_f16x2(b.x >> 16), e4m3x2_f16x2(b.y), e4m3x2_f16x2(b.y >> 16)};
            const int32_t left = pc.tok_end - (pc.tok_begin + (int32_t)(g - g0) * kTile) - stok;  // valid tokens of these eight
            if (left < 8) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                if (left <= 2 * i) x[i] = 0;
                if (left == 2 * i + 1) x[i] &= 0xffffu;
              }
            }
            sts128u(vs + (lane >> 4) * (kTile * 2) + stok * 2, make_uint4(x[0], x[1], x[2], x[3]));
          }
          __syncwarp();
          const uint32_t vsl = vs + (lane >> 4) * (kTile * 2);
#pragma unroll 1
          for (int c = 0; c < kTileBlocks / 2; ++c) {
            uint32_t r[16];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int blk = 2 * c + i;
              const uint2 w = lds64u(base + blk * kv4_block_bytes(D) + kv4_v_off(D) + d * 8);
              const uint4 s0 = lds128u(vsl + blk * 32), s1 = lds128u(vsl + blk * 32 + 16);
              widen8(w.x, as_half2(s0.x), as_half2(s0.y), as_half2(s0.z), as_half2(s0.w), r + 8 * i);
              widen8(w.y, as_half2(s1.x), as_half2(s1.y), as_half2(s1.z), as_half2(s1.w), r + 8 * i + 4);
            }
            tmem_store16(tmem + lanes + C::kColV + vr.i * (kTile / 2) + c * 16, r);
          }
          tmem_wait_stores();
          tmem_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(v_ready + vr.i);
            mbar_arrive(empty + st);
          }
        }
      }
      if (!ok) {
        raise_error(p.err, kErrTimeout);
        *abort_flag = 1;
      }
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int quad = warp & 3;
    const uint32_t group = (uint32_t)(warp - kSoftmax0) >> 2;
    const int st = tid - 32 * kSoftmax0;  // thread among the softmax warps
    const uint32_t bar = 2 + group;  // this group's barrier
    const int key = quad * 32 + lane;  // of the tile; the channel at the end of a piece
    const uint32_t lanes = (uint32_t)(quad * 32) << 16;
    constexpr int H = C::kHeads;
    const int hb = C::kByHead ? (int)group * H : 0;  // this group's first head
    const uint32_t o_col = C::kColO + (C::kByHead ? 0 : group * N) + hb;
    float* red = reinterpret_cast<float*>(smem + C::kRedOff) + group * 80;
    float* fac = reinterpret_cast<float*>(smem + C::kFacOff) + group * 32;
    const float* fac_h = fac + hb;
    const int32_t* lims = reinterpret_cast<const int32_t*>(fac + 16) + hb;
    // A piece's end.  Per head, the sums [groups][4 warps], then [16][groups]
    // references; and the groups' O.
    float* ends = reinterpret_cast<float*>(smem + C::kEndOff);
    float* join = reinterpret_cast<float*>(smem + C::kJoinOff);
    // This thread's key in a p buffer: eight columns, the next eight 16 * kTile bytes on.
    const uint32_t p_at = sbase + C::kPOff + key * 16 + (C::kByHead ? group * (16 * kTile) : 0);
    Groups gr;
    gr.g = p.g;
    gr.gpad = p.gpad;
    gr.nsub = p.nsub;
    gr.hv = p.hv;
    const bool balanced = p.n_splits == 0, fused = p.counters != nullptr;
    pdl_wait();  // before the first write
    // Balanced plan: sequences with no keys own no tile; CTA b % grid writes their outputs.
    if (balanced) {
      for (int32_t b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (tl.len(b) != 0) continue;
        for (int i = st; i < p.Hq * D; i += C::kSThreads) p.out[(size_t)b * p.Hq * D + i] = 0.f;
        if (p.lse)
          for (int i = st; i < p.Hq; i += C::kSThreads) p.lse[(size_t)b * p.Hq + i] = -INFINITY;
      }
    }
    uint32_t g = C::kByHead ? 0 : group, e = 0, f = 0, g1 = 0;  // this group's next tile, the end of the piece
    bool owed = false;                         // the O warp counts the last piece
    uint32_t joins = 0;
    const auto join_owed = [&] {
      const bool known = __all_sync(0xffffffffu, mbar_wait_for(join_known, joins & 1, patience));
      const JoinPiece& j = counted[joins++ & 1];
      if (known && j.last) join_piece(j.b, j.vkv, j.npieces, j.first, warp - kSoftmax0, 4 * kSG);
      ok = ok && known;
    };
    KvPiece pc;
    for (;; ++e) {
      const bool more = next_piece(e, pc);
      if (vote(1, C::kSThreads, !more) != 0) {  // together: the last piece, or a wait that ran out
        if (owed) join_owed();
        break;
      }
      int32_t head0, nh;
      vkv_heads(gr, pc.vkv, &head0, &nh);
      const int32_t n = tiles_of(pc);
      float mr[H], l[H];
#pragma unroll
      for (int h = 0; h < H; ++h) {
        // idle columns have S = 0 and never move their reference
        mr[h] = hb + h < nh ? kNoRef : 0.f;
        l[h] = 0.f;
      }
      int32_t npieces = 0, first = 0;
      bool run = ok && n > 0;
      int32_t whole_end = 0;  // keys below it are seen by every head
      if (run) {
        const uint32_t qb = f & 1;
        const bool got = wait.warp(q_ready + qb, (f >> 1) & 1);
        const float* factor = reinterpret_cast<const float*>(smem + C::kMetaOff + qb * C::kMetaBytes);
        const int32_t* meta = reinterpret_cast<const int32_t*>(factor + 32);
        whole_end = min(pc.tok_end, meta[0]);
        npieces = meta[1];
        first = meta[2];
        if (quad == 0) fac[lane] = factor[lane];  // factors, then limits
        __syncwarp();
        if (lane == 0) mbar_arrive(q_free + qb);
        ++f;
        if (vote(bar, 128, !got) != 0) ok = run = false;
      }
      if (!run) npieces = pieces_of(pc, first);
      const uint32_t g0 = g1;
      if (run) g1 += n;
      const uint32_t g_first = g;
      float* sums = join + (C::kByHead ? hb : (int)group * G) * D + key;  // this thread's channel of O
      for (; run; g += kStep) {
        const uint32_t jj = (g - g_first) / kStep;  // the group's tile
        if (jj > 0 && (g >= g1 || jj % kFlush == 0)) {  // O of the last tiles joins the sums in shared memory
          const bool got = wait.warp(p_free + (g - kStep) % C::kSBufs, (g - kStep) / C::kSBufs & 1);
          if (vote(bar, 128, !got) != 0) {
            ok = run = false;
            break;
          }
          tmem_fence_after();
          constexpr int W = H < 2 ? 2 : H;
          float hi[W], lo[W];
          tmem_load<W>(tmem + lanes + o_col, hi);
          tmem_load<W>(tmem + lanes + o_col + G, lo);
          if (key < D) {
#pragma unroll
            for (int h = 0; h < H; ++h) sums[h * D] = (jj > kFlush ? sums[h * D] : 0.f) + fmaf(lo[h], kLoDown, hi[h]);
          }
          tmem_fence_before();
        }
        if (g >= g1) break;
        const uint32_t i = g % C::kSBufs, ph = g / C::kSBufs & 1;
        const int32_t t0 = pc.tok_begin + (int32_t)(g - g0) * kTile;
        const bool whole = t0 + kTile <= whole_end;
        const bool got = wait.warp(s_full + i, ph);
        tmem_fence_after();
        float x[H < 2 ? 2 : H];
        const auto load_scores = [&] {  // hi + lo, not yet times their factors
          if constexpr (G < 16) {
            float s[2 * G];
            tmem_load<2 * G>(tmem + lanes + C::kColS + i * N, s);
#pragma unroll
            for (int h = 0; h < H; ++h) x[h] = s[h] + s[G + h];
          } else {
            float lo[H];
            tmem_load<H>(tmem + lanes + C::kColS + i * N + hb, x);
            tmem_load<H>(tmem + lanes + C::kColS + i * N + G + hb, lo);
#pragma unroll
            for (int h = 0; h < H; ++h) x[h] += lo[h];
          }
        };
        for (bool again = false;; again = true) {
          // exponents relative to the references; almost always none lies too far above
          bool up = false;
          load_scores();
#pragma unroll
          for (int h = 0; h < H; ++h) x[h] = fmaf(x[h], fac_h[h], -mr[h]);
          if (__builtin_expect(!whole, 0)) {
            const int32_t t = t0 + key < pc.tok_end ? t0 + key : 0x7fffffff;
#pragma unroll
            for (int h = 0; h < H; ++h)
              if (t >= lims[h]) x[h] = -INFINITY;
          }
          if (__builtin_expect(again, 0)) {
            // Once is enough.  Scores of 2^27 and more are further apart than kTau: a reference
            // that was rounded down by more than that stays, and the exponent is cut.
#pragma unroll
            for (int h = 0; h < H; ++h) x[h] = x[h] > kRefDown + kTau ? kRefDown + kTau : x[h];
            break;
          }
#pragma unroll
          for (int h = 0; h < H; ++h) up |= x[h] > kRefDown + kTau;
          // one vote a warp for such a score, 24 for a wait that ran out
          const bool any_up = __any_sync(0xffffffffu, up);
          const uint32_t votes = vote(bar, 128, got ? any_up && lane == 0 : lane >= 8);
          if (__builtin_expect(votes == 0, 1)) break;
          bool moved = votes < 24;
          if (moved) {
            // the reference moves: maxima of the tile, then l and O on the new one
            uint32_t seen = 0;
#pragma unroll
            for (int h = 0; h < H; ++h) seen |= (x[h] == -INFINITY ? 0u : 1u) << h;
            load_scores();
#pragma unroll
            for (int h = 0; h < H; ++h) x[h] = seen >> h & 1 ? x[h] * fac_h[h] : -INFINITY;
            warp_reduce<H>(x, lane, [](float a, float b) { return fmaxf(a, b); });
            if (lane % (32 / H) == 0) red[lane / (32 / H) * 4 + quad] = x[0];
            named_barrier(bar, 128);
            if (key < H) {
              const float4 m = reinterpret_cast<const float4*>(red)[key];
              const float top = fmaxf(fmaxf(m.x, m.y), fmaxf(m.z, m.w)) - kRefDown;
              red[64 + key] = top == INFINITY ? NAN : top;  // a score past the range of floats shows as NaN
            }
            named_barrier(bar, 128);
            float (&alpha)[H < 2 ? 2 : H] = x;
#pragma unroll
            for (int h = 0; h < H; ++h) {
              const float mn = red[64 + h] <= mr[h] ? mr[h] : red[64 + h];
              alpha[h] = ex2(mr[h] - mn);
              mr[h] = mn;
              l[h] *= alpha[h];
            }
            if (jj >= kFlush && key < D) {
#pragma unroll
              for (int h = 0; h < H; ++h) sums[h * D] *= alpha[h];
            }
            if (g != g_first) {
              moved = wait.warp(p_free + (g - kStep) % C::kSBufs, (g - kStep) / C::kSBufs & 1);  // O of this group's last tile
              if (moved) {
                tmem_fence_after();
#pragma unroll
                for (int part = 0; part < 2; ++part) {  // hi, lo
                  constexpr int W = H < 2 ? 2 : H;
                  if (G == 1 && part == 1) break;
                  float o[W];
                  tmem_load<W>(tmem + lanes + o_col + part * G, o);
#pragma unroll
                  for (int h = 0; h < W; ++h) o[h] *= alpha[h % H];
                  tmem_store<W>(tmem + lanes + o_col + part * G, o);
                }
                tmem_wait_stores();
              }
            }
          }
          if (vote(bar, 128, !moved) != 0) {  // red is free again, too
            ok = run = false;
            break;
          }
        }
        if (!run) break;
        // p's buffer: O of what it held has been computed
        if (g < C::kSBufs || wait.warp(p_free + i, ph ^ 1)) {
          const uint32_t ps = p_at + i * C::kPBytes;
#pragma unroll
          for (int h = 0; h < H; ++h) {
            x[h] = ex2(x[h]);
            l[h] += x[h];
          }
          uint32_t w[H < 2 ? 1 : H];  // columns of hi, then of lo, in pairs
          if constexpr (G == 1) {
            uint32_t hi, lo;
            split_f16x2<!C::kByHead>(x[0], 0.f, hi, lo, kLoUp);
            w[0] = hi | lo << 16;
          } else {
#pragma unroll
            for (int h = 0; h < H; h += 2) split_f16x2<!C::kByHead>(x[h], x[h + 1], w[h / 2], w[(H + h) / 2], kLoUp);
          }
          if constexpr (G == 1) {
            asm volatile("st.shared.u32 [%0], %1;" ::"r"(ps), "r"(w[0]) : "memory");
          } else if constexpr (G == 2) {
            asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(ps), "r"(w[0]), "r"(w[1]) : "memory");
          } else {
#pragma unroll
            for (int c = 0; c < H; c += 4)  // hi, lo: G / 8 places on with 8 heads and more
              sts128u(ps + c / 4 * (G / 8) * (16 * kTile), make_uint4(w[c], w[c + 1], w[c + 2], w[c + 3]));
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        } else {
          raise_error(p.err, kErrTimeout);  // the abort ends this group at its next wait
        }
        tmem_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(p_ready + i);
      }
      // ---- end of the piece: sums over the keys, O by channel, the groups joined.
      // (Rolled loops over shared memory: code that runs once a piece is not in the
      // instruction cache, and its length was what a piece's end took.)
      if ((!run || g == g_first) && key < D) {
#pragma unroll
        for (int h = 0; h < H; ++h) sums[h * D] = 0.f;
      }
      warp_reduce<H>(l, lane, [](float a, float b) { return a + b; });
      if (lane % (32 / H) == 0) {
        float* to = ends + (hb + lane / (32 / H)) * 8 + quad;
        to[C::kByHead ? 0 : group * 4] = l[0];
        if (C::kByHead) to[4] = 0.f;
      }
      if (key == 0) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
          ends[128 + (hb + h) * 2 + (C::kByHead ? 0 : group)] = mr[h];
          if (C::kByHead) ends[128 + (hb + h) * 2 + 1] = mr[h];
        }
      }
      named_barrier(1, C::kSThreads);
      const bool final_here = fused && npieces == 1;
#pragma unroll 1
      for (int idx = st; idx < nh * (D / 4); idx += C::kSThreads) {
        const int h = idx / (D / 4), d = idx % (D / 4) * 4;
        // the groups' states on the largest reference; one without keys has l = 0
        const float4 la = reinterpret_cast<const float4*>(ends)[2 * h], lb = reinterpret_cast<const float4*>(ends)[2 * h + 1];
        const float2 ms = reinterpret_cast<const float2*>(ends + 128)[h];
        const float4 oa = *reinterpret_cast<const float4*>(join + h * D + d);
        const float4 ob = C::kByHead ? make_float4(0.f, 0.f, 0.f, 0.f) : *reinterpret_cast<const float4*>(join + (G + h) * D + d);
        const float l0 = (la.x + la.y) + (la.z + la.w), l1 = (lb.x + lb.y) + (lb.z + lb.w), mm = fmaxf(ms.x, ms.y);
        const float w0 = l0 == 0.f ? 0.f : ex2(ms.x - mm), w1 = l1 == 0.f ? 0.f : ex2(ms.y - mm);
        const float L = fmaf(w0, l0, w1 * l1), up = pow2i(kv.v_exp);
        float4 acc = make_float4(fmaf(w0, oa.x, w1 * ob.x) * up, fmaf(w0, oa.y, w1 * ob.y) * up,
                                 fmaf(w0, oa.z, w1 * ob.z) * up, fmaf(w0, oa.w, w1 * ob.w) * up);
        const size_t row = (size_t)pc.b * p.Hq + head0 + h;
        if (final_here) {
          acc.x = L == 0.f ? 0.f : acc.x / L;
          acc.y = L == 0.f ? 0.f : acc.y / L;
          acc.z = L == 0.f ? 0.f : acc.z / L;
          acc.w = L == 0.f ? 0.f : acc.w / L;
          *reinterpret_cast<float4*>(p.out + row * D + d) = acc;
          if (p.lse && d == 0) p.lse[row] = L == 0.f ? -INFINITY : (mm + log2f(L)) * kLn2;
        } else {
          const size_t i = balanced ? (size_t)pc.slot * p.gpad + h : row * p.n_splits + pc.slot;
          *reinterpret_cast<float4*>(p.o_part + i * D + d) = acc;
          if (d == 0) {
            // The join passes over states whose l is not above zero.  A NaN sum goes in as
            // m = inf: the weight exp(inf - inf) then makes out and lse NaN, as the formula does.
            p.m_part[i] = isnan(L) ? INFINITY : (L == 0.f ? -INFINITY : mm * kLn2);
            p.l_part[i] = isnan(L) ? 1.f : L;
          }
        }
      }
      if (owed) join_owed();
      owed = fused && pc.more;
      if (owed) {
        if (st == 0) counted[joins & 1] = JoinPiece{0, pc.b, pc.vkv, npieces, first};
        __syncwarp();
        if (lane == 0) mbar_arrive(part_done);
      } else if (fused && !final_here) {
        named_barrier(1, C::kSThreads);  // every thread's partial stores come before the release
        if (st == 0) *last_flag = arrive_last(pc, npieces) ? 1 : 0;
        named_barrier(1, C::kSThreads);
        if (*last_flag) join_piece(pc.b, pc.vkv, npieces, first, warp - kSoftmax0, 4 * kSG);
      }
    }
    if (!ok) {
      raise_error(p.err, kErrTimeout);
      *abort_flag = 1;
    }
  }
  tmem_fence_before();
  cta_sync();
  if (warp == 1) {
    tmem_fence_after();
    tmem_free_all(tmem);
  }
}

template <int D, int G>
cudaError_t launch_t(const Kv4View& kv, const SplitParams& p, dim3 grid, cudaStream_t stream) {
  using C = K4<D, G>;
  static std::atomic<int> configured_device{-1};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (configured_device.load(std::memory_order_acquire) != dev) {
    e = cudaFuncSetAttribute(fd_kv4_kernel<D, G>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    if (e != cudaSuccess) return e;
    configured_device.store(dev, std::memory_order_release);
  }
  Kv4Params pp;
  pp.p = p;
  pp.kv = kv;
  // Programmatic dependent launch: set-up overlaps the kernel before; every role
  // waits for it before its first access to global memory.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(C::kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fd_kv4_kernel<D, G>, pp);
}

}  // namespace

cudaError_t launch_kv4_split(int D, const Kv4View& kv, const SplitParams& p, dim3 grid, cudaStream_t stream) {
#define FD_CASE(DD, GG) \
  if (D == DD && p.gpad == GG) return launch_t<DD, GG>(kv, p, grid, stream);
  FD_CASE(128, 1) FD_CASE(128, 2) FD_CASE(128, 4) FD_CASE(128, 8) FD_CASE(128, 16)
  FD_CASE(64, 1) FD_CASE(64, 2) FD_CASE(64, 4) FD_CASE(64, 8) FD_CASE(64, 16)
#undef FD_CASE
  return cudaErrorInvalidValue;
}

}  // namespace fdk
