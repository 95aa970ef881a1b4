// fd_append.cu -- new tokens into a KV cache, with the position rotation of
// queries and keys applied on the way.
//
// A pair (a, b) of channels turned by the angle of the row's position p and
// the pair's index i (cos and sin read from fp32 tables):
//     a' = a cos - b sin,   b' = b cos + a sin,
// in fp32 (one rounding of the second product, one of the fused sum), rounded
// once to the cache's type; q comes out in fp32, the layout of the attention
// calls.  Pairs are (i, i + rot/2), or neighbours (2i, 2i + 1) when interleaved.
//
// The work is bound by memory: each thread takes sixteen channels of one row,
// as the two 8-channel chunks that hold both halves of its eight pairs; no
// shared memory for bf16 and fp32 caches.  Two things count:
//   - whole 32-byte sectors a store.  fp32 rows in 16-byte stores sent each
//     sector to L2 twice: 8192 tokens of 32 + 8 heads of 128 channels took 51.9 us,
//     46.9 to 48.5 with 32-byte stores; a read-back of 32768 tokens 31.8, now 29.8.
//   - rows are loaded before the chain of lengths, pages and positions that says
//     where they go, but after the length that says whether they are padding (55 %
//     live of 8192 tokens: 36.8 us, 32.0 when padding is not loaded).
// Measured on the device: 8192 tokens into bf16 48 us (5.7 TB/s, 84 % of a copy's rate), the
// same into 4 bits 52 us, 64 tokens into bf16 2.4 us, 96 into 4 bits 3.2 us, a read-back
// of 32768 tokens of 8 heads to bf16 29.8 us (5.8 TB/s, 85 %).
#include "../../include/fdecode.h"
#include "fd_kv4.cuh"

namespace fdk {
namespace {

// Whether row i is in front of the sequence's new tokens.
__device__ __forceinline__ bool padding(const NewRows& r, int32_t b, int32_t i) {
  return r.new_lens && i < r.n - clamp_len(__ldg(r.new_lens + b), r.n);
}

// Where a token goes: row j of the padded n rows of sequence b.
struct Place {
  bool live;      // the row is a token, and its position is in the tables
  int32_t t;      // its place in the sequence
  int32_t pos;    // its row of the tables
};

__device__ __forceinline__ Place place_of(const NewRows& r, int32_t b, int32_t i) {
  Place p;
  const int32_t L = clamp_len(r.seq_lens ? __ldg(r.seq_lens + b) : r.max_len, r.max_len);
  const int32_t nl = r.new_lens ? clamp_len(__ldg(r.new_lens + b), r.n) : r.n;
  const int32_t j = i - (r.n - nl);
  p.live = j >= 0;
  p.t = L + (j < 0 ? 0 : j);
  p.pos = p.t;
  if (p.live && r.rot > 0) {
    if (r.positions) p.pos = __ldg(r.positions + (size_t)b * r.n + i);
    if (p.pos < 0 || p.pos >= r.max_pos) {
      p.live = false;
      atomicOr(r.err, kErrBadIndex);
    }
  }
  return p;
}

__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4*>(p));
  v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
  v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
}
// 32 bytes in one store where the address allows it: a warp's two 16-byte stores
// with gaps of 16 bytes would send each sector to L2 twice.
__device__ __forceinline__ void store32(void* p, uint4 a, uint4 b) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
                 "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
                 : "memory");
  } else {
    static_cast<uint4*>(p)[0] = a;
    static_cast<uint4*>(p)[1] = b;
  }
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  store32(p, *reinterpret_cast<const uint4*>(&v[0]), *reinterpret_cast<const uint4*>(&v[4]));
}
__device__ __forceinline__ uint4 bf16x8(const float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
// Two chunks of a row, at channels c0 and c1.
__device__ __forceinline__ void store_chunks(float* row, int c0, int c1, const float (&x)[8], const float (&y)[8]) {
  store8(row + c0, x);
  store8(row + c1, y);
}
__device__ __forceinline__ void store_chunks(__nv_bfloat16* row, int c0, int c1, const float (&x)[8],
                                             const float (&y)[8]) {
  if (c1 == c0 + 8) {
    store32(row + c0, bf16x8(x), bf16x8(y));
  } else {
    *reinterpret_cast<uint4*>(row + c0) = bf16x8(x);
    *reinterpret_cast<uint4*>(row + c1) = bf16x8(y);
  }
}

// The two 8-channel chunks of thread `s` of a row (D / 16 threads a row): the
// halves of eight pairs, or sixteen neighbours where nothing (or neighbours) is
// turned.
struct Chunks {
  int c0, c1;    // first channel of each
  bool turned;
};
template <int D>
__device__ __forceinline__ Chunks chunks_of(int s, int rot, bool interleaved, bool rotate) {
  Chunks c;
  c.turned = rotate && (interleaved ? 16 * s < rot : 8 * s < rot / 2);
  const bool apart = c.turned && !interleaved;
  c.c0 = apart ? 8 * s : 16 * s;
  c.c1 = apart ? 8 * s + rot / 2 : 16 * s + 8;
  return c;
}

// Sixteen channels turned in place; cos and sin of pairs 8s .. 8s + 7.
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const float* cs, const float* sn, bool interleaved) {
  float c[8], s[8];
  load8(cs, c);
  load8(sn, s);
  if (!interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = a[i], y = b[i];
      a[i] = fmaf(x, c[i], -(y * s[i]));
      b[i] = fmaf(y, c[i], x * s[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float x = a[2 * i], y = a[2 * i + 1];
      a[2 * i] = fmaf(x, c[i], -(y * s[i]));
      a[2 * i + 1] = fmaf(y, c[i], x * s[i]);
      x = b[2 * i];
      y = b[2 * i + 1];
      b[2 * i] = fmaf(x, c[4 + i], -(y * s[4 + i]));
      b[2 * i + 1] = fmaf(y, c[4 + i], x * s[4 + i]);
    }
  }
}

// One thread's sixteen channels of row (b, i) of head `h`, as they are.
template <int D, class T>
__device__ __forceinline__ Chunks load_chunks(const void* base, const int64_t (&st)[3], int32_t b, int32_t i, int32_t h,
                                              int s, int rot, bool interleaved, bool rotate, float (&x)[8], float (&y)[8]) {
  const T* row = static_cast<const T*>(base) + (int64_t)b * st[0] + (int64_t)i * st[1] + (int64_t)h * st[2];
  const Chunks c = chunks_of<D>(s, rot, interleaved, rotate);
  load8(row + c.c0, x);
  load8(row + c.c1, y);
  return c;
}
__device__ __forceinline__ void turn_chunks(const NewRows& r, const Chunks& c, int s, const Place& pl, float (&x)[8],
                                            float (&y)[8]) {
  if (c.turned) {
    const int64_t at = (int64_t)pl.pos * (r.rot / 2) + 8 * s;
    turn(x, y, r.cos + at, r.sin + at, r.interleaved);
  }
}

// The same, turned when `rotate`.
template <int D, class T>
__device__ __forceinline__ Chunks load_turned(const NewRows& r, const void* base, const int64_t (&st)[3], int32_t b,
                                              int32_t i, int32_t h, int s, const Place& pl, bool rotate, float (&x)[8],
                                              float (&y)[8]) {
  const Chunks c = load_chunks<D, T>(base, st, b, i, h, s, r.rot, r.interleaved, rotate, x, y);
  turn_chunks(r, c, s, pl, x, y);
  return c;
}

template <int D, class T>
__device__ __forceinline__ void query_row(const NewRows& r, int32_t b, int32_t i, int32_t h, int s) {
  if (padding(r, b, i)) return;
  float x[8], y[8];
  const Chunks c = load_chunks<D, T>(r.q, r.qs, b, i, h, s, r.rot, r.interleaved, true, x, y);
  const Place pl = place_of(r, b, i);
  if (!pl.live) return;
  turn_chunks(r, c, s, pl, x, y);
  float* out = r.q_out + (((int64_t)b * r.Hq + h) * r.n + i) * D;
  store_chunks(out, c.c0, c.c1, x, y);
}

// bf16 and fp32 caches: D / 16 threads a row, the rows of one token (q heads,
// then k, then v) side by side so that they share its row of the tables.
template <int D, class T, class C>
__global__ void __launch_bounds__(256) fd_append_kernel(const NewRows r, const KvView kv, int32_t items) {
  constexpr int TPR = D / 16;
  const int32_t item = (int32_t)(((int64_t)blockIdx.x * 256 + threadIdx.x) / TPR);
  const int s = threadIdx.x % TPR;
  if (item >= items) return;
  const int32_t heads = r.Hq + 2 * kv.Hkv;
  const int32_t tok = item / heads, slot = item - tok * heads;
  const int32_t b = tok / r.n, i = tok - b * r.n;
  if (slot < r.Hq) {
    query_row<D, T>(r, b, i, slot, s);
    return;
  }
  const bool is_v = slot >= r.Hq + kv.Hkv;
  const int32_t h = slot - r.Hq - (is_v ? kv.Hkv : 0);
  if (padding(r, b, i)) return;
  float x[8], y[8];
  const Chunks c = load_chunks<D, T>(is_v ? r.v : r.k, is_v ? r.vs : r.ks, b, i, h, s, r.rot, r.interleaved, !is_v, x, y);
  const Place pl = place_of(r, b, i);
  if (!pl.live) return;
  int64_t row;
  if (kv.paged) {
    const int32_t page = __ldg(kv.block_table + (size_t)b * kv.max_pages + pl.t / kv.page_size);
    if (page < 0 || page >= kv.num_pages) {
      atomicOr(r.err, kErrBadIndex);
      return;
    }
    row = ((int64_t)page * kv.Hkv + h) * kv.page_size + pl.t % kv.page_size;
  } else {
    row = ((int64_t)b * kv.Hkv + h) * kv.capacity + pl.t;
  }
  turn_chunks(r, c, s, pl, x, y);
  C* out = static_cast<C*>(is_v ? kv.v : kv.k) + row * D;
  store_chunks(out, c.c0, c.c1, x, y);
}

// ------------------------------------------------------------------ 4 bits
__device__ __forceinline__ float amax8(const float (&v)[8]) {
  float m = fabsf(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(v[i]));
  return m;
}

// Eight codes of v / scale, channel order from the low nibble.  The quotient is
// a true one: bf16 values lie exactly halfway between two codes often.
__device__ __forceinline__ uint32_t codes8(const float (&v)[8], float scale) {
  float r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) r[i] = scale == 0.f ? copysignf(0.f, v[i]) : __fdiv_rn(v[i], scale);
  return f32_e2m1x8(r);
}

// A CTA of D threads takes one block of sixteen tokens of one (sequence, KV
// head), or D / (D / 16) = 16 query rows.  Thread (t, s) quantises sixteen
// channels of token t; V's codes go through shared memory so that thread d then
// writes the eight bytes of channel d.  Tokens of the block that the call does
// not bring keep their nibbles.
template <int D, class T>
__global__ void __launch_bounds__(D) fd_append_kv4_kernel(const NewRows r, const Kv4View kv, int32_t nblk,
                                                          int32_t kv_ctas) {
  constexpr int TPR = D / 16;
  const int tid = threadIdx.x;
  const int s = tid % TPR, tt = tid / TPR;
  if ((int32_t)blockIdx.x >= kv_ctas) {
    const int64_t item = (int64_t)(blockIdx.x - kv_ctas) * 16 + tt;
    if (item >= (int64_t)r.B * r.n * r.Hq) return;
    const int32_t tok = (int32_t)(item / r.Hq), h = (int32_t)(item - (int64_t)tok * r.Hq);
    query_row<D, T>(r, tok / r.n, tok % r.n, h, s);
    return;
  }
  __shared__ __align__(16) uint8_t vcodes[16][D];
  const int32_t pair = blockIdx.x / nblk, k = blockIdx.x % nblk;
  const int32_t b = pair / kv.Hkv, h = pair % kv.Hkv;
  const int32_t L = clamp_len(r.seq_lens ? __ldg(r.seq_lens + b) : r.max_len, r.max_len);
  const int32_t nl = r.new_lens ? clamp_len(__ldg(r.new_lens + b), r.n) : r.n;
  const int32_t blk0 = (L / 16 + k) * 16;       // first token of this block
  if (blk0 >= L + nl || nl == 0) return;
  const int64_t idx = kv4_block_index(kv, b, h, blk0);
  if (idx < 0) {
    if (tid == 0) atomicOr(r.err, kErrBadIndex);
    return;
  }
  uint8_t* blk = kv.kv + idx * kv4_block_bytes(D);
  const int32_t t = blk0 + tt;
  const int32_t i = t - L + (r.n - nl);  // the row that brings it
  bool live = t >= L && t < L + nl;
  Place pl;
  pl.live = false;
  pl.t = t;
  pl.pos = 0;
  if (live) pl = place_of(r, b, i);
  live = pl.live;
  const uint2 old = *reinterpret_cast<const uint2*>(blk + kv4_v_off(D) + tid * 8);

  float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  Chunks c = chunks_of<D>(s, r.rot, r.interleaved, true);
  if (live) load_turned<D, T>(r, r.k, r.ks, b, i, h, s, pl, true, x, y);
  const float kdown = pow2i(-kv.k_exp), vdown = pow2i(-kv.v_exp);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    x[e] *= kdown;
    y[e] *= kdown;
  }
  // A scale covers sixteen neighbours: this thread's own, or (halves apart) its
  // eight low channels with the next thread's eight, and the same for the high ones.
  float mx = amax8(x), my = amax8(y);
  const float ox = __shfl_xor_sync(0xffffffffu, mx, 1), oy = __shfl_xor_sync(0xffffffffu, my, 1);
  const bool apart = c.turned && !r.interleaved;
  const float sx = apart ? max_nan(mx, ox) : max_nan(mx, my), sy = apart ? max_nan(my, oy) : sx;
  const uint32_t bx = f32_e4m3(__fdiv_rn(sx, 6.f)), by = f32_e4m3(__fdiv_rn(sy, 6.f));
  if (live) {
    const uint32_t wx = codes8(x, e4m3_f32(bx)), wy = codes8(y, e4m3_f32(by));
    const int sw = kv4_swizzle(D, tt);
    uint8_t* row = blk + tt * (D / 2);
    *reinterpret_cast<uint32_t*>(row + (((c.c0 >> 5) ^ sw) << 4) + ((c.c0 & 31) >> 1)) = wx;
    *reinterpret_cast<uint32_t*>(row + (((c.c1 >> 5) ^ sw) << 4) + ((c.c1 & 31) >> 1)) = wy;
    uint8_t* sc = blk + kv4_ks_off(D) + tt * (D / 16);
    if (!apart) {
      sc[c.c0 >> 4] = (uint8_t)bx;
    } else if ((s & 1) == 0) {
      sc[c.c0 >> 4] = (uint8_t)bx;
      sc[c.c1 >> 4] = (uint8_t)by;
    }
    load_turned<D, T>(r, r.v, r.vs, b, i, h, s, pl, false, x, y);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[e] *= vdown;
      y[e] *= vdown;
    }
    const uint32_t bv = f32_e4m3(__fdiv_rn(max_nan(amax8(x), amax8(y)), 6.f));
    const float sv = e4m3_f32(bv);
    blk[kv4_vs_off(D) + s * 16 + tt] = (uint8_t)bv;
    const uint32_t v0 = codes8(x, sv), v1 = codes8(y, sv);
    uint32_t q[4];  // one code a byte
    q[0] = (v0 & 0xfu) | (v0 & 0xf0u) << 4 | (v0 & 0xf00u) << 8 | (v0 & 0xf000u) << 12;
    q[1] = (v0 >> 16 & 0xfu) | (v0 >> 16 & 0xf0u) << 4 | (v0 >> 16 & 0xf00u) << 8 | (v0 >> 16 & 0xf000u) << 12;
    q[2] = (v1 & 0xfu) | (v1 & 0xf0u) << 4 | (v1 & 0xf00u) << 8 | (v1 & 0xf000u) << 12;
    q[3] = (v1 >> 16 & 0xfu) | (v1 >> 16 & 0xf0u) << 4 | (v1 >> 16 & 0xf00u) << 8 | (v1 >> 16 & 0xf000u) << 12;
    *reinterpret_cast<uint4*>(&vcodes[tt][s * 16]) = make_uint4(q[0], q[1], q[2], q[3]);
  }
  // which of the sixteen tokens were written (a bad position leaves its row out)
  __shared__ uint32_t mask;
  if (tid == 0) mask = 0;
  __syncthreads();
  if (live && s == 0) atomicOr(&mask, 1u << tt);
  __syncthreads();
  uint32_t w[2] = {old.x, old.y};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (mask >> j & 1) {
      const uint32_t sh = 4 * (j & 7);
      w[j >> 3] = (w[j >> 3] & ~(0xfu << sh)) | (uint32_t)vcodes[j][tid] << sh;
    }
  *reinterpret_cast<uint2*>(blk + kv4_v_off(D) + tid * 8) = make_uint2(w[0], w[1]);
}

// The largest size of the sixteen lanes' values, NaN if one is.
__device__ __forceinline__ float amax16(float v) {
  float m = fabsf(v);
#pragma unroll
  for (int o = 8; o > 0; o /= 2) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}
__device__ __forceinline__ float load1(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// The same for few tokens a sequence: a CTA of D threads takes a (sequence, KV head)
// and its tokens one after another, a channel a thread; the bytes are the same.  Above,
// eight threads would quantise a lone token, sixteen channels each, while the others wait.
// 1, 2, 3, 4, 8 tokens of 96 sequences: 3.2, 4.6, 5.9, 7.4, 12.8 us; above 5.9, 7.4, 7.7,
// 7.7, 8.6.  Of one sequence: 2.6, 3.5, 4.4, 5.5, 9.4; above 4.9 to 5.0.  D = 64, 96 sequences: 3.0, 4.2,
// 5.5, 6.5, 10.8 against 5.5, 6.3, 6.4, 6.4, 6.8; one: 2.4, 3.3, 4.3, 5.5, 9.2 against 4.6 to 4.9.  1500
// sequences of 3 and 4 tokens, D = 128: 68 and 87 against 78 and 85.
constexpr int32_t kFewRows = 3;
template <int D, class T>
__global__ void __launch_bounds__(D) fd_append_kv4_few_kernel(const NewRows r, const Kv4View kv, int32_t kv_ctas) {
  constexpr int TPR = D / 16;
  const int d = threadIdx.x;
  if ((int32_t)blockIdx.x >= kv_ctas) {
    const int64_t item = (int64_t)(blockIdx.x - kv_ctas) * 16 + d / TPR;
    if (item >= (int64_t)r.B * r.n * r.Hq) return;
    const int32_t tok = (int32_t)(item / r.Hq), h = (int32_t)(item - (int64_t)tok * r.Hq);
    query_row<D, T>(r, tok / r.n, tok % r.n, h, d % TPR);
    return;
  }
  const int32_t b = blockIdx.x / kv.Hkv, h = blockIdx.x % kv.Hkv;
  // this channel's pair, and its place in it
  const int half = r.rot / 2;
  const bool turned = d < r.rot, second = r.interleaved ? d & 1 : d >= half;
  const int pair = r.interleaved ? d / 2 : (second ? d - half : d);
  const int other = !turned ? d : r.interleaved ? d ^ 1 : (second ? d - half : d + half);
  const float kdown = pow2i(-kv.k_exp), vdown = pow2i(-kv.v_exp);
#pragma unroll 1
  for (int32_t i = 0; i < r.n; ++i) {
    if (padding(r, b, i)) continue;
    const T* krow = static_cast<const T*>(r.k) + (int64_t)b * r.ks[0] + (int64_t)i * r.ks[1] + (int64_t)h * r.ks[2];
    const T* vrow = static_cast<const T*>(r.v) + (int64_t)b * r.vs[0] + (int64_t)i * r.vs[1] + (int64_t)h * r.vs[2];
    float k = load1(krow + d), v = load1(vrow + d);
    const float o = load1(krow + other);
    const Place pl = place_of(r, b, i);
    if (!pl.live) continue;
    const int64_t idx = kv4_block_index(kv, b, h, pl.t);
    if (idx < 0) {
      if (d == 0) atomicOr(r.err, kErrBadIndex);
      continue;
    }
    if (turned) {
      const int64_t at = (int64_t)pl.pos * half + pair;
      const float c = __ldg(r.cos + at), sn = __ldg(r.sin + at);
      k = second ? fmaf(k, c, o * sn) : fmaf(k, c, -(o * sn));
    }
    uint8_t* blk = kv.kv + idx * kv4_block_bytes(D);
    const int tt = pl.t % kKv4Tokens;
    uint8_t* vbyte = blk + kv4_v_off(D) + d * 8 + (tt >> 1);
    const uint32_t old = *vbyte;
    k *= kdown;
    v *= vdown;
    const uint32_t bk = f32_e4m3(__fdiv_rn(amax16(k), 6.f)), bv = f32_e4m3(__fdiv_rn(amax16(v), 6.f));
    const float sk = e4m3_f32(bk), sv = e4m3_f32(bv);
    const float qk = sk == 0.f ? copysignf(0.f, k) : __fdiv_rn(k, sk);
    const float qv = sv == 0.f ? copysignf(0.f, v) : __fdiv_rn(v, sv);
    const uint32_t code = f32_e2m1x2(qv, 0.f);
    *vbyte = (uint8_t)(tt & 1 ? (old & 0x0fu) | code << 4 : (old & 0xf0u) | code);
    const uint32_t two = f32_e2m1x2(qk, __shfl_down_sync(0xffffffffu, qk, 1));
    if ((d & 1) == 0) blk[tt * (D / 2) + (((d >> 5) ^ kv4_swizzle(D, tt)) << 4) + ((d & 31) >> 1)] = (uint8_t)two;
    if (d % 16 == 0) {
      blk[kv4_ks_off(D) + tt * (D / 16) + d / 16] = (uint8_t)bk;
      blk[kv4_vs_off(D) + d / 16 * 16 + tt] = (uint8_t)bv;
    }
  }
}

// ------------------------------------------------------------------ read-back
template <class O>
__device__ __forceinline__ void store_values(O* out, uint32_t lo, uint32_t hi, float scale) {
  // lo, hi: eight codes each
  float x[8], y[8];
  uint32_t h[8] = {e2m1x2_f16x2<0>(lo), e2m1x2_f16x2<1>(lo), e2m1x2_f16x2<2>(lo), e2m1x2_f16x2<3>(lo),
                   e2m1x2_f16x2<0>(hi), e2m1x2_f16x2<1>(hi), e2m1x2_f16x2<2>(hi), e2m1x2_f16x2<3>(hi)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h[4 + i]));
    x[2 * i] = a.x * scale;
    x[2 * i + 1] = a.y * scale;
    y[2 * i] = b.x * scale;
    y[2 * i + 1] = b.y * scale;
  }
  store_chunks(out, 0, 8, x, y);
}

template <int D, class O>
__global__ void __launch_bounds__(D) fd_kv4_read_kernel(const Kv4Read r, const Kv4View kv, int32_t nblk) {
  constexpr int TPR = D / 16;
  __shared__ __align__(16) uint8_t vcodes[16][D];
  const int tid = threadIdx.x;
  const int s = tid % TPR, tt = tid / TPR;
  const int32_t pair = blockIdx.x / nblk, k = blockIdx.x % nblk;
  const int32_t b = pair / kv.Hkv, h = pair % kv.Hkv;
  const int32_t L = clamp_len(r.seq_lens ? __ldg(r.seq_lens + b) : r.max_len, r.max_len);
  const int32_t start = r.starts ? clamp_len(__ldg(r.starts + b), r.max_len) : 0;
  const int32_t end = L - start < r.n ? L : start + r.n;
  const uint32_t first = ((uint32_t)start / 16 + k) * 16;  // may pass the largest int32
  if (first >= (uint32_t)end) return;
  const int32_t blk0 = (int32_t)first;
  const int64_t idx = kv4_block_index(kv, b, h, blk0);
  if (idx < 0) {
    if (tid == 0) atomicOr(r.err, kErrBadIndex);
    return;
  }
  const uint8_t* blk = kv.kv + idx * kv4_block_bytes(D);
  const uint2 vw = *reinterpret_cast<const uint2*>(blk + kv4_v_off(D) + tid * 8);
#pragma unroll
  for (int j = 0; j < 16; ++j) vcodes[j][tid] = (uint8_t)((j < 8 ? vw.x >> 4 * j : vw.y >> 4 * (j - 8)) & 0xfu);
  const int32_t t = blk0 + tt;
  const bool live = t >= start && t < end;
  const int64_t row = (((int64_t)b * kv.Hkv + h) * r.n + (t - start)) * D + s * 16;
  if (live) {
    const int sw = kv4_swizzle(D, tt);
    const uint2 kw = *reinterpret_cast<const uint2*>(blk + tt * (D / 2) + (((s >> 1) ^ sw) << 4) + (s & 1) * 8);
    const float sc = e4m3_f32(blk[kv4_ks_off(D) + tt * (D / 16) + s]) * pow2i(kv.k_exp);
    store_values(static_cast<O*>(r.k_out) + row, kw.x, kw.y, sc);
  }
  __syncthreads();
  if (live) {
    const uint4 c = *reinterpret_cast<const uint4*>(&vcodes[tt][s * 16]);
    const auto pack = [](uint32_t a) { return (a & 0xfu) | (a >> 4 & 0xf0u) | (a >> 8 & 0xf00u) | (a >> 12 & 0xf000u); };
    const float sc = e4m3_f32(blk[kv4_vs_off(D) + s * 16 + tt]) * pow2i(kv.v_exp);
    store_values(static_cast<O*>(r.v_out) + row, pack(c.x) | pack(c.y) << 16, pack(c.z) | pack(c.w) << 16, sc);
  }
}

// Blocks of sixteen tokens that n consecutive tokens can touch; n is at most a cache's longest
// sequence, so the sum fits.
int32_t blocks_touched(int32_t n) { return (n + 14) / 16 + 1; }

template <int D, class T>
cudaError_t append_t(bool cache_f32, const NewRows& r, const KvView& kv, cudaStream_t stream) {
  const int64_t items = (int64_t)r.B * r.n * (r.Hq + 2 * kv.Hkv);
  const int64_t ctas = (items * (D / 16) + 255) / 256;
  if (items > INT32_MAX || ctas > INT32_MAX) return cudaErrorInvalidValue;
  if (cache_f32)
    fd_append_kernel<D, T, float><<<(unsigned)ctas, 256, 0, stream>>>(r, kv, (int32_t)items);
  else
    fd_append_kernel<D, T, __nv_bfloat16><<<(unsigned)ctas, 256, 0, stream>>>(r, kv, (int32_t)items);
  return cudaGetLastError();
}

template <int D, class T>
cudaError_t append_kv4_t(const NewRows& r, const Kv4View& kv, cudaStream_t stream) {
  const int32_t nblk = r.n <= kFewRows ? 1 : blocks_touched(r.n);
  const int64_t kv_ctas = (int64_t)r.B * kv.Hkv * nblk;
  const int64_t ctas = kv_ctas + ((int64_t)r.B * r.n * r.Hq + 15) / 16;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  if (r.n <= kFewRows) {
    fd_append_kv4_few_kernel<D, T><<<(unsigned)ctas, D, 0, stream>>>(r, kv, (int32_t)kv_ctas);
    return cudaGetLastError();
  }
  fd_append_kv4_kernel<D, T><<<(unsigned)ctas, D, 0, stream>>>(r, kv, nblk, (int32_t)kv_ctas);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_append(int D, bool rows_f32, bool cache_f32, const NewRows& r, const KvView& kv,
                          cudaStream_t stream) {
  if (D == 128)
    return rows_f32 ? append_t<128, float>(cache_f32, r, kv, stream)
                    : append_t<128, __nv_bfloat16>(cache_f32, r, kv, stream);
  return rows_f32 ? append_t<64, float>(cache_f32, r, kv, stream)
                  : append_t<64, __nv_bfloat16>(cache_f32, r, kv, stream);
}

cudaError_t launch_append_kv4(int D, bool rows_f32, const NewRows& r, const Kv4View& kv, cudaStream_t stream) {
  if (D == 128)
    return rows_f32 ? append_kv4_t<128, float>(r, kv, stream) : append_kv4_t<128, __nv_bfloat16>(r, kv, stream);
  return rows_f32 ? append_kv4_t<64, float>(r, kv, stream) : append_kv4_t<64, __nv_bfloat16>(r, kv, stream);
}

cudaError_t launch_kv4_read(int D, bool out_f32, const Kv4Read& r, const Kv4View& kv, cudaStream_t stream) {
  // r.n rows of the output may be more than there are tokens
  const int32_t nblk = blocks_touched(r.n < r.max_len ? r.n : r.max_len);
  const int64_t ctas = (int64_t)r.B * kv.Hkv * nblk;
  if (ctas > INT32_MAX) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)ctas;
  if (D == 128) {
    if (out_f32)
      fd_kv4_read_kernel<128, float><<<grid, 128, 0, stream>>>(r, kv, nblk);
    else
      fd_kv4_read_kernel<128, __nv_bfloat16><<<grid, 128, 0, stream>>>(r, kv, nblk);
  } else {
    if (out_f32)
      fd_kv4_read_kernel<64, float><<<grid, 64, 0, stream>>>(r, kv, nblk);
    else
      fd_kv4_read_kernel<64, __nv_bfloat16><<<grid, 64, 0, stream>>>(r, kv, nblk);
  }
  return cudaGetLastError();
}

}  // namespace fdk
