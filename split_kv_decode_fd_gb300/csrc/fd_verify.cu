// fd_verify.cu -- which tokens of a drafted tree stay, by the target's and the
// draft's probabilities and given random numbers, and the token that follows.
//
// The walk starts at token 0.  At a token, whose row of the target is p and of the
// draft q, its children are asked in the order of their numbers.  Refusing one
// leaves of the target what the draft had not offered: norm(max(p - q, 0)), and so on for
// the next.  Not normalised, after some refusals this is
//     r = max(p - c q, 0),   mass Z = sum r,   c' = c + Z when one more is refused,
// from c = 0, Z = 1, as max(max(a, 0) - b, 0) = max(a - b, 0) for b >= 0.  So nothing but c
// is kept.  Child x with random number u stays when u Z q(x) < r(x).  Without a draft's
// probabilities the children are given, not drawn: q is 1 at the child, r is p without
// the refused words, Z is 1 less their mass.  Where the walk ends, the next token is
// the first v with r(0) + ... + r(v) > u_0 sum r.
//
// Sums decide on whole numbers, so they are held in about 48 bits, as pairs of floats with
// the errors of their additions (Knuth's two-sum), from a thread's up to the cluster's.  An
// instruction in 64 bits takes a warp 16 cycles of the SM's pipe for them, so only one warp of a CTA
// walks the tree (when all sixteen did, 64 sequences of 131072 words took 131 us).
//
// Bound by the latency of the passes over a row (its sum when a child is refused, or at the end), one after
// another: some 6 us each once few sequences are left, two thirds of it the sum (its arithmetic in dependent steps, two warps a
// scheduler), the rest the exchange of sums and the walk.
// Measured: 64 sequences of 16 drafts, 131072 words in fp32, up to five passes, 44 us (reading the rows once takes 10); 32
// sequences of 32 drafts, 65521 words in bf16, 11.6; one sequence of 8, 32000 words, 8.1.  (All refused words looked for in every
// group of words 14.2 in place of 11.6; six groups in flight instead of four 45.6 in place of 43.7.)
//
// A cluster takes a sequence, each of its CTAs a part of the vocabulary; CTAs exchange
// their sums through shared memory and decide alike.  The numbers that decide on a child
// without a sum (p, q at its word) are loaded for all tokens at the start.
#include <cuda_bf16.h>

#include "../../include/fdecode.h"
#include "fd_tree.cuh"

namespace fdk {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kCtas = 4;        // CTAs an SM

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// A sum as two floats, hi + lo.
struct Sum {
  float hi, lo;
  __device__ __forceinline__ double value() const { return (double)hi + (double)lo; }
  __device__ __forceinline__ bool positive() const { return hi + lo > 0.f; }
};
__device__ __forceinline__ void add(Sum& s, float hi, float lo) {
  const float t = __fadd_rn(s.hi, hi), b = __fsub_rn(t, s.hi);
  s.lo += __fadd_rn(__fsub_rn(s.hi, __fsub_rn(t, b)), __fsub_rn(hi, b)) + lo;
  s.hi = t;
}
// The sum over the warp's lanes, the same in each: a step's partners add in one order.
__device__ __forceinline__ Sum warp_sum(Sum s) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const Sum other{__shfl_xor_sync(0xffffffffu, s.hi, o), __shfl_xor_sync(0xffffffffu, s.lo, o)};
    Sum low = lane & o ? other : s;
    const Sum high = lane & o ? s : other;
    add(low, high.hi, high.lo);
    s = low;
  }
  return s;
}
__device__ __forceinline__ Sum minus(Sum a, const Sum& b) {
  add(a, -b.hi, -b.lo);
  return a;
}
// The sum over lanes 0 to this one.
__device__ __forceinline__ Sum warp_upto(Sum s) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    Sum before{__shfl_up_sync(0xffffffffu, s.hi, o), __shfl_up_sync(0xffffffffu, s.lo, o)};
    add(before, s.hi, s.lo);
    if (lane >= o) s = before;
  }
  return s;
}
__device__ __forceinline__ Sum from_lane(const Sum& s, int lane) {
  return Sum{__shfl_sync(0xffffffffu, s.hi, lane), __shfl_sync(0xffffffffu, s.lo, lane)};
}
// The lane that holds t when the lanes' sums lie end to end, the last with a sum if rounding leaves none (-1 if none
// has), and the rest of t within it.
__device__ __forceinline__ int holds(const Sum& own, Sum& t) {
  const Sum upto = warp_upto(own);
  const unsigned some = __ballot_sync(0xffffffffu, own.positive());
  const unsigned over = __ballot_sync(0xffffffffu, minus(upto, t).positive()) & some;
  const int l = over ? __ffs(over) - 1 : 31 - __clz(some);
  if (l < 0) return -1;
  t = minus(t, from_lane(minus(upto, own), l));
  return l;
}
// `v` to the same place in the shared memory of CTA `rank`.
__device__ __forceinline__ void store_remote(Sum* at, uint32_t rank, const Sum& v) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.v2.f32 [a], {%2, %3};\n\t}" ::"r"(
                   smem_addr(at)),
               "r"(rank), "f"(v.hi), "f"(v.lo)
               : "memory");
}

template <class T>
constexpr int kGroup = 16 / (int)sizeof(T);  // probabilities in 16 bytes
constexpr int kAhead = 4;                                  // groups of each of p and q that a thread has in flight
constexpr int kRingBytes = 2 * kAhead * kThreads * 16;     // where they land

// The probabilities of 16 bytes.
__device__ __forceinline__ void widen(const uint4& w, float (&x)[4]) {
  x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
}
__device__ __forceinline__ void widen(const uint4& w, float (&x)[8]) {
  x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
  x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
}

template <class T>
__device__ __forceinline__ float at(const T* row, int32_t i);
template <>
__device__ __forceinline__ float at<float>(const float* row, int32_t i) { return __ldg(row + i); }
template <>
__device__ __forceinline__ float at<__nv_bfloat16>(const __nv_bfloat16* row, int32_t i) {
  return __bfloat162float(row[i]);
}

// Group g of a row of V probabilities: entries [g E - off, (g + 1) E - off), `off` making them 16-byte loads (entries
// before or past the row are 0).  vec: they are.
template <class T>
__device__ __forceinline__ void load_group(const T* row, int32_t g, int32_t V, int32_t off, bool vec, float (&x)[kGroup<T>]) {
  constexpr int E = kGroup<T>;
  const int32_t first = g * E - off;
  if (vec && first >= 0 && first + E <= V) {
    widen(__ldg(reinterpret_cast<const uint4*>(row + first)), x);
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = first + e >= 0 && first + e < V ? at(row, first + e) : 0.f;
  }
}

// What is left of the target at the token where the walk stands.
template <class T, bool kDraft>
struct Left {
  const T *p, *q;
  int32_t V, off;
  bool vec;                   // both rows are at the same place of 16 bytes
  float c_hi, c_lo;           // c as a sum of two floats
  const int32_t* refused;     // without a draft: words that are out
  int32_t n_refused;
  uint64_t near;              // those of them that lie in the groups at hand, by their number

  // Before groups [g0, g1), a warp's, are looked at.
  __device__ __forceinline__ void range(int32_t g0, int32_t g1) {
    near = 0;
    if constexpr (!kDraft) {
      const int lane = threadIdx.x & 31;
      const int32_t first = g0 * kGroup<T> - off, end = g1 * kGroup<T> - off;
      uint32_t in[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int32_t x = lane + 32 * i < n_refused ? refused[lane + 32 * i] : -1;
        in[i] = __ballot_sync(0xffffffffu, x >= 0 && x >= first && x < end);
      }
      near = (uint64_t)in[1] << 32 | in[0];
    }
  }
  // Without the words of group g that are out.
  __device__ __forceinline__ void refuse(float (&x)[kGroup<T>], int32_t g) const {
    for (uint64_t some = near; some; some &= some - 1) {
      const int32_t e = refused[__ffsll((long long)some) - 1] - (g * kGroup<T> - off);
#pragma unroll
      for (int k = 0; k < kGroup<T>; ++k)
        if (k == e) x[k] = 0.f;
    }
  }

  // What is not above 0 counts as 0 in the draft's row too (fmaxf gives 0 for NaN).
  static __device__ __forceinline__ void clean(float (&y)[kGroup<T>]) {
    if constexpr (kDraft) {
#pragma unroll
      for (int e = 0; e < kGroup<T>; ++e) y[e] = fmaxf(y[e], 0.f);
    }
  }

  // r of group g as sums hi + lo
  __device__ __forceinline__ void group(const float (&x)[kGroup<T>], const float (&y)[kGroup<T>], int32_t g,
                                        float (&hi)[kGroup<T>], float (&lo)[kGroup<T>]) const {
#pragma unroll
    for (int e = 0; e < kGroup<T>; ++e) {
      float d = x[e], t = 0.f;
      if constexpr (kDraft) {
        const float m = __fmul_rn(c_hi, y[e]);
        const float m_lo = fmaf(c_lo, y[e], fmaf(c_hi, y[e], -m));
        d = __fsub_rn(x[e], m);
        const float b = __fsub_rn(d, x[e]);
        t = __fsub_rn(__fsub_rn(x[e], __fsub_rn(d, b)), __fadd_rn(m, b)) - m_lo;
      }
      const bool some = d + t > 0.f;  // NaN counts as nothing
      hi[e] = some ? d : 0.f;
      lo[e] = some ? t : 0.f;
    }
    if constexpr (!kDraft) refuse(hi, g);
  }

  // r of two words, added to two sums.
  __device__ __forceinline__ void add_pair(uint64_t x, uint64_t y, uint64_t& s_hi, uint64_t& s_lo) const {
    uint64_t d = x, t = 0;
    if constexpr (kDraft) {
      const uint64_t c = pack2(c_hi, c_hi), m = mul2(pack2(-c_hi, -c_hi), y);  // m: - c q
      const uint64_t m_lo = fma2(pack2(c_lo, c_lo), y, fma2(c, y, m));
      d = add2(x, m);
      const uint64_t b = sub2(d, x);
      t = sub2(sub2(sub2(x, sub2(d, b)), sub2(b, m)), m_lo);
    }
    float d0, d1, t0, t1;
    unpack2(d, d0, d1);
    unpack2(t, t0, t1);
    const bool some0 = d0 + t0 > 0.f, some1 = d1 + t1 > 0.f;  // NaN counts as nothing
    d = pack2(some0 ? d0 : 0.f, some1 ? d1 : 0.f);
    const uint64_t n = add2(s_hi, d), b = sub2(n, s_hi);
    uint64_t e = add2(sub2(s_hi, sub2(n, b)), sub2(d, b));
    if constexpr (kDraft) e = add2(e, pack2(some0 ? t0 : 0.f, some1 ? t1 : 0.f));
    s_lo = add2(s_lo, e);
    s_hi = n;
  }

  // The sum over groups [g0, g1), one warp; the same value in every lane.  mine: this thread's 16 bytes of the ring's first row.
  __device__ __forceinline__ Sum sum(int32_t g0, int32_t g1, uint32_t mine) {
    constexpr int E = kGroup<T>;
    constexpr uint32_t kRow = kThreads * 16u;
    const int32_t n = ceil_div(g1 - g0, 32), first = g0 + (int32_t)(threadIdx.x & 31);
    range(g0, g1);
    auto whole = [&](int32_t g) { return vec && g < g1 && g * E - off >= 0 && g * E - off + E <= V; };
    auto load = [&](int32_t i) {
      const int32_t g = first + 32 * i;
      if (i < n && whole(g)) {
        const uint32_t to = mine + (uint32_t)(i % kAhead) * (2 * kRow);
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p + (g * E - off)) : "memory");
        if constexpr (kDraft)
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + kRow), "l"(q + (g * E - off)) : "memory");
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint64_t s_hi = 0, s_lo = 0;
#pragma unroll 1
    for (int32_t i = 0; i < kAhead - 1; ++i) load(i);
#pragma unroll 1
    for (int32_t i = 0; i < n; ++i) {
      load(i + kAhead - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead - 1) : "memory");
      const int32_t g = first + 32 * i;
      float x[E], y[E] = {};
      if (whole(g)) {
        const uint32_t from = mine + (uint32_t)(i % kAhead) * (2 * kRow);
        widen(lds128u(from), x);
        if constexpr (kDraft) widen(lds128u(from + kRow), y);
      } else if (g < g1) {
        load_group(p, g, V, off, vec, x);
        if constexpr (kDraft) load_group(q, g, V, off, vec, y);
      } else {
        continue;
      }
      clean(y);
      if constexpr (!kDraft) refuse(x, g);
#pragma unroll
      for (int e = 0; e < E; e += 2) add_pair(pack2(x[e], x[e + 1]), pack2(y[e], y[e + 1]), s_hi, s_lo);
    }
    Sum s, odd;
    unpack2(s_hi, s.hi, odd.hi);
    unpack2(s_lo, s.lo, odd.lo);
    add(s, odd.hi, odd.lo);
    return warp_sum(s);
  }

  // The first word of groups [g0, g1) up to which the sum is over t; the last with r > 0 if rounding leaves none.
  __device__ __forceinline__ int32_t find(int32_t g0, int32_t g1, Sum t) {
    constexpr int E = kGroup<T>;
    range(g0, g1);
    const int lane = threadIdx.x & 31;
    int32_t word = -1;
    for (int32_t gb = g0; gb < g1; gb += 32) {
      const int32_t g = gb + lane;
      float x[E] = {}, y[E] = {}, hi[E], lo[E];
      if (g < g1) {
        load_group(p, g, V, off, vec, x);
        if constexpr (kDraft) load_group(q, g, V, off, vec, y);
      }
      clean(y);
      group(x, y, g, hi, lo);
      Sum own{0.f, 0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) add(own, hi[e], lo[e]);
      Sum rest = t;
      const int l = holds(own, rest);
      if (l < 0) continue;
      const Sum all = warp_sum(own);
      const bool here = minus(all, t).positive();  // t lies in these groups, not behind them
      // the first of lane l's entries that goes over the rest, its last with r > 0 if rounding leaves none
      int32_t mine = -1;
      bool over = false;
      Sum upto{0.f, 0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        add(upto, hi[e], lo[e]);
        if (hi[e] + lo[e] > 0.f && !over) {
          mine = g * E - off + e;
          over = minus(upto, rest).positive();
        }
      }
      word = __shfl_sync(0xffffffffu, mine, l);
      if (here) return word;
      t = minus(t, all);
    }
    return word;
  }
};

// What the warp that walks tells the others.
struct Order {
  int32_t node;       // sum what is left at this token; -1: the walk has ended
  float c_hi, c_lo;
  int32_t n_refused;  // of the refused words of this CTA's part
  int32_t part;       // the warp whose groups hold the next token, or -1
};

template <class T, bool kDraft>
__global__ void __launch_bounds__(kThreads, kCtas) fd_verify_kernel(const VerifyParams v) {
  __shared__ int32_t s_parent[kMaxDrafts], s_token[kMaxDrafts], s_refused[kMaxDrafts];
  __shared__ float s_p[kMaxDrafts], s_q[kMaxDrafts], s_u[kMaxDrafts];
  __shared__ Sum s_warp[kWarps], s_cta[2][kMaxCluster];
  __shared__ Order s_order;
  __shared__ Sum s_rest;
  extern __shared__ __align__(16) uint8_t ring[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t own = smem_addr(ring) + (uint32_t)tid * 16u;
  uint32_t C;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const uint32_t rank = cluster_rank();
  const int32_t b = blockIdx.x / C;
  pdl_launch_dependents();
  pdl_wait();
  const int32_t n = v.tree.n, m = tree_tokens(v.tree, b), pad = n - m;
  const T* target = static_cast<const T*>(v.target) + b * v.ts[0] + pad * v.ts[1];
  const T* draft = kDraft ? static_cast<const T*>(v.draft) + b * v.ds[0] + pad * v.ds[1] : nullptr;
  if (tid < kMaxDrafts) {
    int32_t up = -1, x = 0;
    bool child = false;
    if (tid < m) {
      up = __ldg(v.tree.parents + b * v.tree.parents_stride + pad + tid);
      x = __ldg(v.tokens + (int64_t)b * n + pad + tid);
      s_u[tid] = __ldg(v.uniforms + (int64_t)b * n + pad + tid);
      const bool wrong = up < -1 || up >= tid;
      child = tid > 0 && !wrong && up >= 0 && x >= 0 && x < v.V;
      if (wrong || (tid > 0 && up >= 0 && !child)) atomicOr(v.err, kErrBadIndex);
    }
    s_parent[tid] = child ? up : -1;
    s_token[tid] = x;
    s_p[tid] = child ? fmaxf(at(target + up * v.ts[1], x), 0.f) : 0.f;
    s_q[tid] = kDraft && child ? fmaxf(at(draft + up * v.ds[1], x), 0.f) : 0.f;
  }
  int32_t* path = v.path + (int64_t)b * n;
  if (rank == 0 && tid < n) path[tid] = tid == 0 && m > 0 ? 0 : -1;
  cluster_sync();  // the tables are written, and every CTA of the cluster runs
  if (m == 0) {    // the same in every CTA of the cluster
    if (rank == 0 && tid == 0) {
      v.count[b] = 0;
      v.next_token[b] = -1;
    }
    return;
  }

  Left<T, kDraft> left;
  left.V = v.V;
  left.refused = s_refused;
  int buf = 0;
  int32_t g0 = 0, g1 = 0, cta0 = 0, cta1 = 0, per_warp = 0;  // groups of this warp and of this CTA

  // The walk, by warp 0 of every CTA alike
  int32_t node = 0, count = 1;
  double c = 0.0, Z = 1.0;
  uint64_t children = 0, refused = 0;
  bool fresh = true;      // at a token whose children have not been looked for
  bool pending = false;   // a sum has been asked for, for the next child or for the end
  bool last = false;      // ... for the end: no child is left
  for (;;) {
    if (warp == 0) {
      if (pending) {
        Sum s{0.f, 0.f};
        if (lane < (int)C) s = s_cta[buf][lane];
        Z = warp_sum(s).value();
      }
      bool sums = pending;  // Z and the sums are those of this token and c
      pending = false;
      Order o{-1, 0.f, 0.f, 0, -1};
      for (;;) {
        if (last) {
          if (!(Z > 0.0) && (c != 0.0 || refused != 0)) {  // nothing left: the target itself
            c = 0.0;
            refused = 0;
            o.node = node;
          }
          break;
        }
        if (fresh) {
          children = __ballot_sync(0xffffffffu, s_parent[lane] == node);
          children |= (uint64_t)__ballot_sync(0xffffffffu, s_parent[lane + 32] == node) << 32;
          c = 0.0;
          Z = 1.0;
          refused = 0;
          fresh = false;
          sums = false;
        }
        if (children == 0) {
          last = true;
          if (sums) continue;
          o.node = node;
          break;
        }
        const int32_t k = __ffsll((long long)children) - 1;
        children &= children - 1;
        bool stays;
        if constexpr (kDraft) {
          const double q = s_q[k];
          stays = (double)s_u[k] * Z * q < fmax((double)s_p[k] - c * q, 0.0);
          if (!stays) {
            c += Z;
            o.node = node;
            break;
          }
        } else {
          // a word that was refused before has nothing left
          const bool again = __any_sync(0xffffffffu, (refused >> lane & 1 && s_token[lane] == s_token[k]) ||
                                                         (refused >> (lane + 32) & 1 && s_token[lane + 32] == s_token[k]));
          const double r = again ? 0.0 : (double)s_p[k];
          stays = (double)s_u[k] * Z < r;
          if (!stays) {
            Z -= r;
            refused |= 1ull << k;
          }
        }
        if (stays) {
          if (rank == 0 && lane == 0) path[count] = k;
          ++count;
          node = k;
          fresh = true;
        }
      }
      pending = o.node >= 0;
      o.c_hi = (float)c;
      o.c_lo = (float)(c - (double)o.c_hi);
      if (!kDraft && pending) {
        // the refused words, for those that have them in their part
        int32_t kept = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const bool out = refused >> (lane + 32 * i) & 1;
          const unsigned who = __ballot_sync(0xffffffffu, out);
          if (out) s_refused[kept + __popc(who & ((1u << lane) - 1u))] = s_token[lane + 32 * i];
          kept += __popc(who);
        }
        o.n_refused = kept;
      }
      if (lane == 0) s_order = o;
    }
    __syncthreads();
    const Order o = s_order;
    if (o.node < 0) break;
    left.p = target + o.node * v.ts[1];
    // Where nothing has been refused (c = 0) the draft's row is not read, as a leaf may have none: p, which is at hand, stands
    // for it (64 sequences of 131072 words: 43.2 us; with q's loads left out by a branch 45.9).
    left.q = kDraft && o.c_hi != 0.f ? draft + o.node * v.ds[1] : left.p;
    left.c_hi = o.c_hi;
    left.c_lo = o.c_lo;
    left.n_refused = o.n_refused;
    constexpr int E = kGroup<T>;
    const uint32_t byte = (uint32_t)(reinterpret_cast<uintptr_t>(left.p) & 15u);
    left.vec = !kDraft || byte == (uint32_t)(reinterpret_cast<uintptr_t>(left.q) & 15u);
    left.off = (int32_t)(byte / sizeof(T));
    const int32_t groups = (v.V + left.off + E - 1) / E, per_cta = ceil_div(groups, (int32_t)C);
    per_warp = ceil_div(per_cta, kWarps);
    cta0 = min(groups, (int32_t)rank * per_cta);
    cta1 = min(groups, cta0 + per_cta);
    g0 = min(cta1, cta0 + warp * per_warp);
    g1 = min(cta1, g0 + per_warp);
    const Sum mine = left.sum(g0, g1, own);
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    buf ^= 1;
    if (warp == 0) {
      Sum s{0.f, 0.f};
      if (lane < kWarps) s = s_warp[lane];
      s = warp_sum(s);
      if (lane < (int)C) store_remote(&s_cta[buf][rank], (uint32_t)lane, s);
    }
    cluster_sync();
  }

  // The word at u_0 of what is left, by the CTA and the warp that have it
  if (warp == 0) {
    const double target_sum = (double)s_u[0] * Z;
    Sum t{(float)target_sum, 0.f};
    t.lo = (float)(target_sum - (double)t.hi);
    const int owner = holds(lane < (int)C ? s_cta[buf][lane] : Sum{0.f, 0.f}, t);
    const int w = holds(lane < kWarps ? s_warp[lane] : Sum{0.f, 0.f}, t);
    if (lane == 0) {
      s_order.part = owner == (int)rank ? w : -1;
      s_rest = t;
      if (rank == 0) v.count[b] = count;
      if (owner < 0 ? rank == 0 : owner == (int)rank && w < 0) v.next_token[b] = -1;
    }
  }
  __syncthreads();
  const int32_t w = s_order.part;
  if (w >= 0) {
    // that warp's groups once more, a part to each warp
    const int32_t h0 = min(cta1, cta0 + w * per_warp), h1 = min(cta1, h0 + per_warp);
    const int32_t per = ceil_div(h1 - h0, kWarps);
    const int32_t i0 = min(h1, h0 + warp * per), i1 = min(h1, i0 + per);
    const Sum mine = left.sum(i0, i1, own);
    if (lane == 0) s_warp[warp] = mine;
    __syncthreads();
    if (warp == 0) {
      Sum t = s_rest;
      const int x = holds(lane < kWarps ? s_warp[lane] : Sum{0.f, 0.f}, t);
      if (lane == 0) {
        s_order.part = x;
        s_rest = t;
        if (x < 0) v.next_token[b] = -1;
      }
    }
    __syncthreads();
    if (s_order.part == warp) {
      const int32_t word = left.find(i0, i1, s_rest);
      if (lane == 0) v.next_token[b] = word;
    }
  }
  if (C > 1) cluster_sync();  // no CTA leaves while another may write its shared memory
}

template <class T, bool kDraft>
cudaError_t launch(const VerifyParams& v, cudaStream_t stream) {
  // Parts of 1024 words at least, and no more CTAs than run at once.
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)cluster * 1024 < v.V && 2 * (int64_t)v.B * cluster <= kCtas * (int64_t)sms)
    cluster *= 2;
  if ((int64_t)v.B * cluster > INT32_MAX) return cudaErrorInvalidValue;
  e = allow_smem<fd_verify_kernel<T, kDraft>>(kRingBytes);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(v.B * cluster));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kRingBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, fd_verify_kernel<T, kDraft>, v);
}

}  // namespace

cudaError_t launch_verify(bool f32, const VerifyParams& v, cudaStream_t stream) {
  if (f32) return v.draft ? launch<float, true>(v, stream) : launch<float, false>(v, stream);
  return v.draft ? launch<__nv_bfloat16, true>(v, stream) : launch<__nv_bfloat16, false>(v, stream);
}

}  // namespace fdk
