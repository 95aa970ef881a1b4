// fd_kv4_decode.cu -- decode attention over a 4-bit cache: partial states of
// the explicit plan.
//
// One CTA per (b, virtual KV head, split): 128 keys at a time, lane = key for
// q.k, then lane = channel for p.V, with an online softmax per head.
#include "fd_internal.h"
#include "fd_kv4.cuh"
#include "fd_split.cuh"

namespace fdk {
namespace {

constexpr int kTile = 128;
constexpr int kHeads = kMaxGroupBf16;

template <int D>
__global__ void __launch_bounds__(128) fd_kv4_split_kernel(const Kv4View kv, const SplitParams p) {
  __shared__ float q[kHeads][D];
  __shared__ float pr[kHeads][kTile];
  __shared__ float red[4];
  __shared__ int64_t blocks[kTile / kKv4Tokens];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int32_t pair = blockIdx.x, s = blockIdx.y;
  const int32_t b = pair / p.hv, vkv = pair % p.hv;
  Groups gr;
  gr.g = p.g;
  gr.gpad = p.gpad;
  gr.nsub = p.nsub;
  gr.hv = p.hv;
  int32_t head0, nh;
  vkv_heads(gr, vkv, &head0, &nh);
  const int32_t kvh = kv_head_of_vkv(gr, vkv);
  const int32_t L = p.seq_lens ? clamp_len(__ldg(p.seq_lens + b), p.max_len) : p.max_len;
  const int64_t lo = (int64_t)s * p.split_tokens;
  const int32_t t_end = (int32_t)(lo + p.split_tokens < L ? lo + p.split_tokens : L);
  const RowLimits lim{head0, nh, L, p.n_q, p.causal};
  const float up = p.qk_scale * pow2i(kv.k_exp);
  for (int i = tid; i < nh * D; i += 128) q[i / D][i % D] = p.q[((size_t)b * p.Hq + head0) * D + i] * up;
  float m[kHeads], l[kHeads], o[kHeads];
  for (int h = 0; h < kHeads; ++h) {
    m[h] = -INFINITY;
    l[h] = 0.f;
    o[h] = 0.f;
  }
  for (int32_t t0 = (int32_t)(lo < L ? lo : L); t0 < t_end; t0 += kTile) {
    __syncthreads();
    if (tid < kTile / kKv4Tokens) {
      blocks[tid] = -1;
      if (t0 + 16 * tid < t_end) {
        blocks[tid] = kv4_block_index(kv, b, kvh, t0 + 16 * tid);
        if (blocks[tid] < 0) raise_error(p.err, kErrBadIndex);
      }
    }
    __syncthreads();
    const int32_t t = t0 + tid;
    const int64_t idx = blocks[tid / 16];
    const bool in = t < t_end;
    float sc[kHeads];
    for (int h = 0; h < kHeads; ++h) sc[h] = 0.f;
    if (in && idx >= 0) {
      const uint8_t* blk = kv.kv + idx * kv4_block_bytes(D);
      for (int c = 0; c < D / 16; ++c) {
        const int at = (tid & 15) * (D / 2) + (((c >> 1) ^ kv4_swizzle(D, tid & 15)) << 4) + (c & 1) * 8;
        const uint2 w = *reinterpret_cast<const uint2*>(blk + at);
        const float f = e4m3_f32(blk[kv4_ks_off(D) + (tid & 15) * (D / 16) + c]);
        const uint32_t x[8] = {e2m1x2_f16x2<0>(w.x), e2m1x2_f16x2<1>(w.x), e2m1x2_f16x2<2>(w.x), e2m1x2_f16x2<3>(w.x),
                               e2m1x2_f16x2<0>(w.y), e2m1x2_f16x2<1>(w.y), e2m1x2_f16x2<2>(w.y), e2m1x2_f16x2<3>(w.y)};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float2 k2 = __half22float2(*reinterpret_cast<const __half2*>(&x[j]));
          for (int h = 0; h < nh; ++h)
            sc[h] = fmaf(k2.y * f, q[h][16 * c + 2 * j + 1], fmaf(k2.x * f, q[h][16 * c + 2 * j], sc[h]));
        }
      }
    }
    for (int h = 0; h < nh; ++h) {
      const float v = in && t < lim(h) ? sc[h] : -INFINITY;
      const float wm = warp_max(v);
      if (lane == 0) red[warp] = wm;
      __syncthreads();
      const float mn = fmaxf(fmaxf(m[h], fmaxf(red[0], red[1])), fmaxf(red[2], red[3]));
      const float ref = mn == -INFINITY ? 0.f : mn;
      const float e = exp2f(v - ref), alpha = exp2f(m[h] - ref);
      pr[h][tid] = e;
      const float ws = warp_sum(e);
      __syncthreads();
      if (lane == 0) red[warp] = ws;
      __syncthreads();
      l[h] = fmaf(l[h], alpha, (red[0] + red[1]) + (red[2] + red[3]));
      o[h] *= alpha;
      m[h] = mn;
      __syncthreads();
    }
    if (tid < D) {
      const int n = t_end - t0 < kTile ? t_end - t0 : kTile;
      for (int j = 0; j < n; ++j) {
        if (blocks[j / 16] < 0) continue;
        const uint8_t* blk = kv.kv + blocks[j / 16] * kv4_block_bytes(D);
        const uint32_t byte = blk[kv4_v_off(D) + tid * 8 + (j & 15) / 2];
        const uint32_t x = e2m1x2_f16x2<0>(j & 1 ? byte >> 4 : byte & 15);
        const float v = __half2float(__ushort_as_half((unsigned short)(x & 0xffff))) *
                        e4m3_f32(blk[kv4_vs_off(D) + (tid / 16) * 16 + (j & 15)]);
        for (int h = 0; h < nh; ++h) o[h] = fmaf(pr[h][j], v, o[h]);
      }
    }
  }
  const float vup = pow2i(kv.v_exp);
  for (int h = 0; h < nh; ++h) {
    const size_t i = ((size_t)b * p.Hq + head0 + h) * p.n_splits + s;
    if (tid < D) p.o_part[i * D + tid] = o[h] * vup;
    if (tid == 0) {
      // The merge passes over states whose l is not above zero.  A NaN sum goes in as
      // m = inf: the weight exp(inf - inf) then makes out and lse NaN, as the formula does.
      p.m_part[i] = isnan(l[h]) ? INFINITY : m[h] == -INFINITY ? m[h] : m[h] * kLn2;
      p.l_part[i] = isnan(l[h]) ? 1.f : l[h];
    }
  }
}

}  // namespace

cudaError_t launch_kv4_split(int D, const Kv4View& kv, const SplitParams& p, dim3 grid, cudaStream_t stream) {
  if (D == 128)
    fd_kv4_split_kernel<128><<<grid, 128, 0, stream>>>(kv, p);
  else
    fd_kv4_split_kernel<64><<<grid, 128, 0, stream>>>(kv, p);
  return cudaGetLastError();
}

}  // namespace fdk
