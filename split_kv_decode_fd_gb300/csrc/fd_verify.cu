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
// Sums decide on whole numbers, so they are held in about 48 bits: a thread sums in
// pairs of floats with the errors of its additions (Knuth's two-sum), and threads are
// joined in 64 bits.  (In 64 bits throughout, the conversions and additions of the
// slow pipe would take longer than the loads.)
//
// A cluster takes a sequence, each of its CTAs a part of the vocabulary; CTAs exchange
// their sums through shared memory and decide alike.  The numbers that decide on a child
// without a sum (p, q at its word) are loaded for all tokens at the start.
#include <cuda_bf16.h>

#include "../../include/fdecode.h"
#include "fd_tree.cuh"

namespace fdk {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// `v` to the same place in the shared memory of CTA `rank`.
__device__ __forceinline__ void store_remote(double* at, uint32_t rank, double v) {
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\tst.shared::cluster.f64 [a], %2;\n\t}" ::"r"(
                   smem_addr(at)),
               "r"(rank), "d"(v)
               : "memory");
}

template <class T>
constexpr int kGroup = 16 / (int)sizeof(T);  // probabilities in 16 bytes
template <class T>
constexpr int kGroupsAhead = (int)sizeof(T);  // loads a thread has in flight, of each of p and q: 16 probabilities

template <class T>
__device__ __forceinline__ float at(const T* row, int32_t i);
template <>
__device__ __forceinline__ float at<float>(const float* row, int32_t i) { return __ldg(row + i); }
template <>
__device__ __forceinline__ float at<__nv_bfloat16>(const __nv_bfloat16* row, int32_t i) {
  return __bfloat162float(row[i]);
}

// Group g of a row of V probabilities; zeros past its end.
template <class T>
__device__ __forceinline__ void load_group(const T* row, int32_t g, int32_t V, bool aligned, float (&x)[kGroup<T>]) {
  constexpr int E = kGroup<T>;
  if (aligned && (g + 1) * E <= V) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(row) + g);
    if constexpr (E == 4) {
      x[0] = __uint_as_float(w.x), x[1] = __uint_as_float(w.y), x[2] = __uint_as_float(w.z), x[3] = __uint_as_float(w.w);
    } else {
      x[0] = bf16_lo(w.x), x[1] = bf16_hi(w.x), x[2] = bf16_lo(w.y), x[3] = bf16_hi(w.y);
      x[4] = bf16_lo(w.z), x[5] = bf16_hi(w.z), x[6] = bf16_lo(w.w), x[7] = bf16_hi(w.w);
    }
  } else {
#pragma unroll
    for (int e = 0; e < E; ++e) x[e] = g * E + e < V ? at(row, g * E + e) : 0.f;
  }
}

// What is left of the target at the token where the walk stands.
template <class T, bool kDraft>
struct Left {
  const T *p, *q;
  int32_t V;
  bool aligned;
  float c_hi, c_lo;           // c as a sum of two floats
  const int32_t* refused;     // without a draft: words that are out, those of this CTA's part
  int32_t n_refused;

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
    if constexpr (!kDraft) {
      for (int32_t i = 0; i < n_refused; ++i) {
        const int32_t e = refused[i] - g * kGroup<T>;
#pragma unroll
        for (int k = 0; k < kGroup<T>; ++k)
          if (k == e) hi[k] = 0.f;
      }
    }
  }

  // The sum over groups [g0, g1), one warp; the same value in every lane.
  __device__ __forceinline__ double sum(int32_t g0, int32_t g1) const {
    constexpr int E = kGroup<T>, kAhead = kGroupsAhead<T>;
    const int lane = threadIdx.x & 31;
    float s = 0.f, err = 0.f;
    for (int32_t g = g0 + lane; g < g1; g += 32 * kAhead) {
      float x[kAhead][E], y[kAhead][E] = {};
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        const int32_t ga = g + 32 * a;
        if (ga < g1) {
          load_group(p, ga, V, aligned, x[a]);
          if constexpr (kDraft) load_group(q, ga, V, aligned, y[a]);
        } else {
#pragma unroll
          for (int e = 0; e < E; ++e) x[a][e] = 0.f;
        }
      }
#pragma unroll
      for (int a = 0; a < kAhead; ++a) {
        float hi[E], lo[E];
        group(x[a], y[a], g + 32 * a, hi, lo);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float t = __fadd_rn(s, hi[e]), b = __fsub_rn(t, s);
          err += __fadd_rn(__fsub_rn(s, __fsub_rn(t, b)), __fsub_rn(hi[e], b)) + lo[e];
          s = t;
        }
      }
    }
    double all = (double)s + (double)err;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) all += __shfl_xor_sync(0xffffffffu, all, o);
    return all;
  }

  // The first word of groups [g0, g1) up to which the sum is over t; the last with r > 0 if rounding leaves none.
  __device__ __forceinline__ int32_t find(int32_t g0, int32_t g1, double t) const {
    constexpr int E = kGroup<T>;
    const int lane = threadIdx.x & 31;
    double before = 0.0;
    int32_t last = -1;
    for (int32_t gb = g0; gb < g1; gb += 32) {
      const int32_t g = gb + lane;
      float x[E] = {}, y[E] = {}, hi[E], lo[E];
      if (g < g1) {
        load_group(p, g, V, aligned, x);
        if constexpr (kDraft) load_group(q, g, V, aligned, y);
      }
      group(x, y, g, hi, lo);
      double own = 0.0;
      int32_t some = -1;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        own += (double)hi[e] + (double)lo[e];
        if (hi[e] + lo[e] > 0.f) some = g * E + e;
      }
      double upto = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const double v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      const unsigned over = __ballot_sync(0xffffffffu, before + upto > t && some >= 0);
      if (over) {
        const int l = __ffs(over) - 1;
        int32_t word = some;  // of lane l, if its own words do not reach t by rounding
        double cum = before + (upto - own);
#pragma unroll
        for (int e = E - 1; e >= 0; --e) {
          double c = cum;
#pragma unroll
          for (int k = 0; k <= e; ++k) c += (double)hi[k] + (double)lo[k];
          if (c > t && hi[e] + lo[e] > 0.f) word = g * E + e;
        }
        return __shfl_sync(0xffffffffu, word, l);
      }
      const unsigned any = __ballot_sync(0xffffffffu, some >= 0);
      if (any) last = __shfl_sync(0xffffffffu, some, 31 - __clz(any));
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
    return last;
  }
};

// The part of `parts` that holds t when their sums lie end to end; the last with a sum if rounding leaves none.  t
// becomes the rest within the part.
__device__ __forceinline__ int32_t part_of(const double* parts, int32_t count, double& t) {
  double before = 0.0, rest = 0.0;
  int32_t last = -1;
  for (int32_t i = 0; i < count; ++i) {
    if (parts[i] > 0.0) {
      last = i;
      rest = t - before;
      if (before + parts[i] > t) break;
    }
    before += parts[i];
  }
  t = rest;
  return last;
}

template <class T, bool kDraft>
__global__ void __launch_bounds__(kThreads, 2) fd_verify_kernel(const VerifyParams v) {
  __shared__ int32_t s_parent[kMaxDrafts], s_token[kMaxDrafts], s_refused[kMaxDrafts];
  __shared__ float s_p[kMaxDrafts], s_q[kMaxDrafts], s_u[kMaxDrafts];
  __shared__ double s_warp[kWarps], s_cta[2][kMaxCluster];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  uint32_t C;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(C));
  const uint32_t rank = cluster_rank();
  const int32_t b = blockIdx.x / C;
  pdl_launch_dependents();
  pdl_wait();
  const int32_t n = v.tree.n, m = tree_tokens(v.tree, b), pad = n - m;
  const T* target = static_cast<const T*>(v.target) + b * v.ts[0] + pad * v.ts[1];
  const T* draft = kDraft ? static_cast<const T*>(v.draft) + b * v.ds[0] + pad * v.ds[1] : nullptr;
  if (tid < m) {
    int32_t up = __ldg(v.tree.parents + b * v.tree.parents_stride + pad + tid);
    const int32_t x = __ldg(v.tokens + (int64_t)b * n + pad + tid);
    s_u[tid] = __ldg(v.uniforms + (int64_t)b * n + pad + tid);
    const bool wrong = up < -1 || up >= tid;
    const bool child = tid > 0 && !wrong && up >= 0 && x >= 0 && x < v.V;
    if (wrong || (tid > 0 && up >= 0 && !child)) atomicOr(v.err, kErrBadIndex);
    if (!child) up = -1;
    s_parent[tid] = up;
    s_token[tid] = x;
    s_p[tid] = child ? fmaxf(at(target + up * v.ts[1], x), 0.f) : 0.f;
    if constexpr (kDraft) s_q[tid] = child ? at(draft + up * v.ds[1], x) : 0.f;
  }
  int32_t* path = v.path + (int64_t)b * n;
  if (rank == 0 && tid < n) path[tid] = tid == 0 && m > 0 ? 0 : -1;
  cluster_sync();  // the tables are written, and every CTA of the cluster runs
  if (m == 0) {  // the same in every CTA of the cluster
    if (rank == 0 && tid == 0) {
      v.count[b] = 0;
      v.next_token[b] = -1;
    }
    return;
  }

  // groups of this CTA and of this warp
  constexpr int E = kGroup<T>;
  const int32_t groups = (v.V + E - 1) / E;
  const int32_t per_cta = ceil_div(groups, (int32_t)C), per_warp = ceil_div(per_cta, kWarps);
  const int32_t cta0 = min(groups, (int32_t)rank * per_cta), cta1 = min(groups, cta0 + per_cta);
  const int32_t g0 = min(cta1, cta0 + warp * per_warp), g1 = min(cta1, g0 + per_warp);

  Left<T, kDraft> left;
  left.V = v.V;
  left.refused = s_refused;
  left.n_refused = 0;
  int buf = 0;
  // The mass of what is left, the parts of the warps and CTAs on the way
  auto mass_of = [&](int32_t node, double c) -> double {
    left.p = target + node * v.ts[1];
    left.q = kDraft ? draft + node * v.ds[1] : nullptr;
    left.aligned = ((reinterpret_cast<uintptr_t>(left.p) | (kDraft ? reinterpret_cast<uintptr_t>(left.q) : 0)) & 15) == 0;
    left.c_hi = (float)c;
    left.c_lo = (float)(c - (double)left.c_hi);
    const double s = left.sum(g0, g1);
    if (lane == 0) s_warp[warp] = s;
    __syncthreads();
    buf ^= 1;
    if (tid < (int)C) {
      double all = 0.0;
      for (int i = 0; i < kWarps; ++i) all += s_warp[i];
      store_remote(&s_cta[buf][rank], (uint32_t)tid, all);
    }
    cluster_sync();
    double all = 0.0;
    for (uint32_t i = 0; i < C; ++i) all += s_cta[buf][i];
    return all;
  };

  int32_t node = 0, count = 1;
  double c = 0.0, Z = 1.0;
  bool summed = false;
  for (bool on = true; on;) {
    on = false;
    c = 0.0;
    Z = 1.0;
    summed = false;
    uint64_t children = __ballot_sync(0xffffffffu, lane < m && s_parent[lane] == node);
    children |= (uint64_t)__ballot_sync(0xffffffffu, lane + 32 < m && s_parent[(lane + 32) & 63] == node) << 32;
    uint64_t refused = 0;
    while (children) {
      const int32_t k = __ffsll((long long)children) - 1;
      children &= children - 1;
      bool stays;
      if constexpr (kDraft) {
        const double q = s_q[k];
        const double r = fmax((double)s_p[k] - c * q, 0.0);
        stays = (double)s_u[k] * Z * q < r;
        if (!stays) {
          c += Z;
          Z = mass_of(node, c);
          summed = true;
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
        if (rank == 0 && tid == 0) path[count] = k;
        ++count;
        node = k;
        on = true;
        break;
      }
    }
    if (!on && !kDraft) {
      // the refused words of this CTA's part, for the sum
      if (warp == 0) {
        int32_t kept = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int32_t x = s_token[lane + 32 * i];
          const bool mine = (refused >> (lane + 32 * i) & 1) && x >= cta0 * E && x < cta1 * E;
          const unsigned who = __ballot_sync(0xffffffffu, mine);
          if (mine) s_refused[kept + __popc(who & ((1u << lane) - 1u))] = x;
          kept += __popc(who);
        }
        if (lane == 0) s_warp[0] = (double)kept;
      }
      __syncthreads();
      left.n_refused = (int32_t)s_warp[0];
      __syncthreads();
    }
  }
  if (!summed) Z = mass_of(node, c);
  if (!(Z > 0.0)) {  // nothing left: the target itself
    left.n_refused = 0;
    Z = mass_of(node, 0.0);
  }
  int32_t word = -1;
  double t = (double)s_u[0] * Z;
  const int32_t owner = part_of(s_cta[buf], (int32_t)C, t);
  if (owner == (int32_t)rank) {
    const int32_t w = part_of(s_warp, kWarps, t);
    if (w >= 0) {
      // that warp's groups once more, a part to each warp
      const int32_t h0 = min(cta1, cta0 + w * per_warp), h1 = min(cta1, h0 + per_warp);
      const int32_t per = ceil_div(h1 - h0, kWarps);
      const int32_t i0 = min(h1, h0 + warp * per), i1 = min(h1, i0 + per);
      const double s = left.sum(i0, i1);
      __syncthreads();
      if (lane == 0) s_warp[warp] = s;
      __syncthreads();
      const int32_t mine = part_of(s_warp, kWarps, t);
      if (mine == warp) {
        word = left.find(i0, i1, t);
        if (lane == 0) v.next_token[b] = word;
      } else if (mine < 0 && tid == 0) {
        v.next_token[b] = -1;
      }
    }
  } else if (owner < 0 && rank == 0 && tid == 0) {
    v.next_token[b] = -1;
  }
  if (rank == 0 && tid == 0) v.count[b] = count;
  if (C > 1) cluster_sync();  // no CTA leaves while another may write its shared memory
}

template <class T, bool kDraft>
cudaError_t launch(const VerifyParams& v, cudaStream_t stream) {
  int cluster = 1;
  while (cluster < kMaxCluster && (int64_t)cluster * 4096 < v.V) cluster *= 2;
  if ((int64_t)v.B * cluster > INT32_MAX) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(v.B * cluster));
  cfg.blockDim = dim3(kThreads);
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
