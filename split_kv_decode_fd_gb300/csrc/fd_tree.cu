// fd_tree.cu -- attention of a tree of drafted tokens over an fp32 cache, and the join
// of the states that the shares of a sequence leave.
//
// A row sees the places before the drafts, its token's ancestors and itself:
//     out = sum_t exp(x_t - m) v_t / sum_t exp(x_t - m),   x_t = scale q . k_t,
// over what it sees, with the running m and sum of an online softmax.
//
// A CTA of four warps serves 32 rows of a KV head (16 where it has no more) from tiles of 64 keys in shared
// memory; a thread has four rows (two), of which it takes four keys for q . k and D / 16
// channels for p . V: sixteen products for eight values read, so that both keep the
// arithmetic busy rather than shared memory.  K and V have one buffer each: V's next tile
// comes in under q . k, K's under p . V, and the other CTAs of the SM fill what is left.
// Blocks of rows are made of tokens' rows alone and are pairs of their own in the shares: padding costs nothing.
//
// Measured: 6 sequences of 2099 to 3000 tokens, 12 heads on 4, D = 64, 2 to 10 tokens each: 28.6 us, of which the join has some 4,
// the start (walk, q, ancestors, first tile) 4 and a tile with three CTAs on the SM 5, where its 64 x 32 x 64 x 2 products could
// take 1 at the rate of the fp32 units (shares in tiles of 128 keys 33).  Two rows a thread, tiles loaded and then used, and padding's rows too: 58.
#include "fd_tree.cuh"

namespace fdk {
namespace {

constexpr int kKeys = kTreeTileCore;
constexpr int kCoreThreads = 128;

// R: rows a thread has, of those of its half warp; 8 R a CTA.
template <int D, int R>
struct CoreSmem {
  static constexpr int kRows = 8 * R;
  static constexpr int kStride = D + 4;     // rows of q and k: eight rows in a row of banks
  static constexpr int kPStride = kRows + 4;
  float q[kRows * kStride];
  float k[kKeys * kStride];
  float v[kKeys * D];
  float p[kKeys * kPStride];                // weights, key by key
  TreePiece piece;
  int32_t more;
};

__device__ __forceinline__ void cp_async16(uint32_t to, const float* from, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
__device__ __forceinline__ void cp_async_wait_older() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

// Rows [t0, t0 + 64) of K or V to shared memory.  Rows past the piece's end and those of pages that are none hold nothing
// that counts: they come in as zeros.
template <int D, int Stride>
__device__ __forceinline__ void copy_tile(const TreeParams& p, const TreePiece& pc, const void* cache, int32_t t0, uint32_t to) {
  constexpr int kStep = kCoreThreads / (D / 4);  // rows side by side
  const int c = threadIdx.x % (D / 4) * 4, r0 = threadIdx.x / (D / 4);
  const float* base = static_cast<const float*>(cache);
  to += (uint32_t)(r0 * Stride + c) * 4;
  if (t0 >= pc.end) {
    // nothing
  } else if (!p.kv.paged) {
    const float* from = base + (((int64_t)pc.b * p.Hkv + pc.h) * p.kv.capacity + t0 + r0) * D + c;
#pragma unroll
    for (int i = 0; i < kKeys / kStep; ++i) {
      const bool there = t0 + r0 + i * kStep < pc.end;
      cp_async16(to + (uint32_t)(i * kStep * Stride) * 4, there ? from + i * kStep * D : base, there);
    }
  } else {
#pragma unroll 4
    for (int i = 0; i < kKeys / kStep; ++i) {
      const int32_t t = t0 + r0 + i * kStep;
      int64_t at = -1;
      if (t < pc.end) {
        const int32_t page = __ldg(p.kv.block_table + (int64_t)pc.b * p.kv.max_pages + t / p.kv.page_size);
        if (page >= 0 && page < p.kv.num_pages)
          at = ((int64_t)page * p.Hkv + pc.h) * p.kv.page_size + t % p.kv.page_size;
        else
          atomicOr(p.err, kErrBadIndex);
      }
      cp_async16(to + (uint32_t)(i * kStep * Stride) * 4, at < 0 ? base : base + at * D + c, at >= 0);
    }
  }
  cp_async_commit();
}

// Row i of the tokens of a KV head, head by head, as a row of q and out: m of every n rows are tokens, the last.
__device__ __forceinline__ int32_t tree_row(const TreeParams& p, int32_t m, int32_t i) {
  return i / m * p.tree.n + (p.tree.n - m) + i % m;
}

template <int D, int R>
__global__ void __launch_bounds__(kCoreThreads, tree_ctas(true, D)) fd_tree_core_kernel(const TreeParams p) {
  using S = CoreSmem<D, R>;
  constexpr int kRows = S::kRows;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ty = tid / 16, tx = tid % 16;
  const int32_t range = blockIdx.x;
  constexpr int kCols = D / 64;  // float4 of output a row and thread
  constexpr int kStep = kCoreThreads / (D / 4);  // rows side by side in a copy
  const uint32_t to_q = smem_addr(s.q), to_k = smem_addr(s.k), to_v = smem_addr(s.v);
  pdl_launch_dependents();
  pdl_wait();
  tree_no_rows<D, kRows, kRows>(p, range, 0, tid, kCoreThreads);
  TreeWalk<kRows> walk(p, range, warp == 0);
  if (tid == 0) walk.say_none();
  for (;;) {
    if (warp == 0) {
      TreePiece pc;
      const bool found = walk.next(pc);
      if (lane == 0) {
        s.piece = pc;
        s.more = found;
        if (found) walk.say(pc);
      }
    }
    __syncthreads();
    if (!s.more) return;
    const TreePiece pc = s.piece;
    const int64_t row0 = ((int64_t)pc.b * p.Hkv + pc.h) * p.rows;  // of q and out
    const int32_t first = pc.sub * kRows, rows = p.g * pc.m - first;  // of the tokens' rows; how many there are from there
#pragma unroll
    for (int i = 0; i < kRows / kStep; ++i) {
      const int r = tid / (D / 4) + i * kStep, c = tid % (D / 4) * 4;
      const bool there = r < rows;
      cp_async16(to_q + (uint32_t)(r * S::kStride + c) * 4, p.q + (there ? (row0 + tree_row(p, pc.m, first + r)) * D + c : 0), there);
    }
    copy_tile<D, S::kStride>(p, pc, p.kv.k, pc.begin, to_k);  // (and q, which comes with it)
    copy_tile<D, D>(p, pc, p.kv.v, pc.begin, to_v);
    const int32_t P = pc.len - pc.m;
    const Ancestors all = tree_ancestors(p.tree, pc.b, pc.m, p.err);
    uint64_t anc[R];
    float mx[R], l[R];
    uint64_t o[R][kCols][2];  // pairs of channels
#pragma unroll
    for (int i = 0; i < R; ++i) {
      anc[i] = all.of((first + R * ty + i) % pc.m);
      mx[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[i][c][0] = o[i][c][1] = 0;
    }
    for (int32_t t0 = pc.begin; t0 < pc.end; t0 += kKeys) {
      cp_async_wait_older();
      __syncthreads();  // K's tile is there
      // q . k of rows 4 ty .. 4 ty + 3 and keys tx, tx + 16, tx + 32, tx + 48
      uint64_t y[R][4] = {};  // sums of the even and of the odd channels
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        ulonglong2 a[R], k[4];
#pragma unroll
        for (int i = 0; i < R; ++i) a[i] = *reinterpret_cast<const ulonglong2*>(s.q + (R * ty + i) * S::kStride + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const ulonglong2*>(s.k + (tx + 16 * j) * S::kStride + c);
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i][j] = fma2(a[i].y, k[j].y, fma2(a[i].x, k[j].x, y[i][j]));
      }
      __syncthreads();  // K's tile is read
      copy_tile<D, S::kStride>(p, pc, p.kv.k, t0 + kKeys, to_k);
      const bool some_hidden = t0 + kKeys > P;
      uint32_t w[R][2];  // what the rows see of the tile
      float x[R][4];
#pragma unroll
      for (int i = 0; i < R; ++i) {
        w[i][0] = w[i][1] = 0xffffffffu;
        if (some_hidden) {
          const TileMask mask = tile_mask(P, anc[i], t0);
          w[i][0] = mask.w[0];
          w[i][1] = mask.w[1];
        }
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float even, odd;
          unpack2(y[i][j], even, odd);
          x[i][j] = w[i][j >> 1] >> (tx + 16 * (j & 1)) & 1u ? (even + odd) * p.qk_scale : -INFINITY;
          top = fmaxf(top, x[i][j]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float mn = fmaxf(mx[i], top);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float alpha = mx[i] == -INFINITY ? 0.f : ex2(mx[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i][j] = ex2(x[i][j] - base);
          sum += x[i][j];
        }
        l[i] = fmaf(l[i], alpha, sum);
        mx[i] = mn;
        const uint64_t a2 = pack2(alpha, alpha);
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          o[i][c][0] = mul2(o[i][c][0], a2);
          o[i][c][1] = mul2(o[i][c][1], a2);
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float* at = s.p + (tx + 16 * j) * S::kPStride + R * ty;
        if constexpr (R == 4)
          *reinterpret_cast<float4*>(at) = make_float4(x[0][j], x[1][j], x[2][j], x[3][j]);
        else
          *reinterpret_cast<float2*>(at) = make_float2(x[0][j], x[1][j]);
      }
      cp_async_wait_older();
      __syncthreads();  // V's tile is there, and the weights
      auto weights = [&](int t, uint64_t (&weight)[R]) {  // those of this thread's rows for key t
        const float* at = s.p + t * S::kPStride + R * ty;
        if constexpr (R == 4) {
          const float4 e = *reinterpret_cast<const float4*>(at);
          weight[0] = pack2(e.x, e.x), weight[1] = pack2(e.y, e.y), weight[2] = pack2(e.z, e.z), weight[3] = pack2(e.w, e.w);
        } else {
          const float2 e = *reinterpret_cast<const float2*>(at);
          weight[0] = pack2(e.x, e.x), weight[1] = pack2(e.y, e.y);
        }
      };
      // A value that a row does not see may be anything, and 0 * NaN is not 0: drafts whose values are no numbers take
      // the second form.  (With that for every tile with drafts, 26 short sequences of 880 rows a head took 396 us in
      // place of 329.)
      bool odd = false;
      if (some_hidden) {
        const int32_t first = P > t0 ? P - t0 : 0, end = pc.end - t0 < kKeys ? pc.end - t0 : kKeys;
        for (int32_t i = first * (D / 4) + tid; i < end * (D / 4); i += kCoreThreads) {
          const float4 v = *reinterpret_cast<const float4*>(s.v + 4 * i);
          odd = odd || !(fabsf(v.x) < INFINITY && fabsf(v.y) < INFINITY && fabsf(v.z) < INFINITY && fabsf(v.w) < INFINITY);
        }
        odd = __syncthreads_or(odd);
      }
      if (!odd) {
#pragma unroll 4
        for (int t = 0; t < kKeys; ++t) {
          uint64_t weight[R];
          weights(t, weight);
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(s.v + t * D + 64 * c + 4 * tx);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              o[i][c][0] = fma2(weight[i], v.x, o[i][c][0]);
              o[i][c][1] = fma2(weight[i], v.y, o[i][c][1]);
            }
          }
        }
      } else {
#pragma unroll 1
        for (int t = 0; t < kKeys; ++t) {
          uint64_t weight[R];
          weights(t, weight);
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(s.v + t * D + 64 * c + 4 * tx);
#pragma unroll
            for (int i = 0; i < R; ++i) {
              const bool seen = (t < 32 ? w[i][0] : w[i][1]) >> (t & 31) & 1u;
              o[i][c][0] = fma2(weight[i], seen ? v.x : 0, o[i][c][0]);
              o[i][c][1] = fma2(weight[i], seen ? v.y : 0, o[i][c][1]);
            }
          }
        }
      }
      __syncthreads();  // V's tile is read
      copy_tile<D, D>(p, pc, p.kv.v, t0 + kKeys, to_v);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      const int r = R * ty + i;
      if (r >= rows) continue;
      const int64_t row = row0 + tree_row(p, pc.m, first + r);
      const int64_t state = (int64_t)pc.slot * kRows + r;
      float* to = pc.slot < 0 ? p.out + row * D : p.o_part + state * D;
      const float f = pc.slot >= 0 ? 1.f : (l[i] == 0.f ? 0.f : 1.f / l[i]);
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const uint64_t f2 = pack2(f, f);
        *reinterpret_cast<ulonglong2*>(to + 64 * c + 4 * tx) = make_ulonglong2(mul2(o[i][c][0], f2), mul2(o[i][c][1], f2));
      }
      if (tx == 0) {
        if (pc.slot >= 0) {
          p.m_part[state] = mx[i];
          p.l_part[state] = l[i];
        } else if (p.lse) {
          p.lse[row] = l[i] == 0.f ? -INFINITY : (mx[i] + log2f(l[i])) * kTreeLn2;
        }
      }
    }
    // (the last tile's barriers part this piece's reads of s.piece and s.q from the next one's writes)
  }
}

// Joins the states of a pair: a warp a row, the m and l of 32 shares at a time in its lanes.
// With M the largest m so far,
//     out = sum_k 2^(m_k - M) O_k / sum_k 2^(m_k - M) l_k.
template <int D, int Rows>
__global__ void __launch_bounds__(256, 4) fd_tree_join_kernel(const TreeParams p) {
  constexpr int kPer = D / 32;   // channels a lane
  constexpr int kAhead = 8;      // states whose O is on its way
  pdl_launch_dependents();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int32_t w = (int32_t)(blockIdx.x * 8 + (threadIdx.x >> 5));
  const int32_t r = w % Rows, sub = w / Rows % p.nsub, f = w / Rows / p.nsub;
  if (f >= p.n_joins) return;
  const TreeJoin j = p.joins[f];
  int32_t row = (j.sub + sub) * Rows + r;
  // (a call that gave up may have left an entry of an earlier one)
  if (j.b < 0 || j.b >= p.B || j.h < 0 || j.h >= p.Hkv || j.sub < 0 || j.sub >= p.blocks || j.first < 0 || j.last < j.first || j.last >= p.ranges) return;
  const int32_t m = tree_tokens(p.tree, j.b);
  if (p.packed) {
    if (row >= p.g * m) return;
    row = tree_row(p, m, row);
  } else if (row >= p.rows || row % p.tree.n < p.tree.n - m) {
    return;
  }
  const int32_t count = j.last - j.first + 1;
  auto state = [&](int32_t k) {
    return ((int64_t)(2 * (j.first + k) + (k == 0 ? 1 : 0)) * p.nsub + sub) * Rows + r;
  };
  auto load = [&](int32_t k, float (&v)[kPer]) {
    const float* o = p.o_part + state(k) * D + lane * kPer;
    if constexpr (kPer == 4) {
      const float4 x = __ldcg(reinterpret_cast<const float4*>(o));
      v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
    } else {
      const float2 x = __ldcg(reinterpret_cast<const float2*>(o));
      v[0] = x.x, v[1] = x.y;
    }
  };
  float M = -INFINITY, L = 0.f, acc[kPer] = {};
  for (int32_t k0 = 0; k0 < count; k0 += 32) {
    float l = 0.f, m = -INFINITY;
    if (k0 + lane < count) {
      l = __ldcg(p.l_part + state(k0 + lane));
      m = __ldcg(p.m_part + state(k0 + lane));
    }
    const int32_t stop = count - k0 < 32 ? count - k0 : 32;
    float v[kAhead][kPer];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (i < stop) load(k0 + i, v[i]);
    const float top = fmaxf(M, warp_max(l != 0.f ? m : -INFINITY));
    const float alpha = M == top ? 1.f : exp2f(M - top);
    const float e = l != 0.f ? exp2f(m - top) : 0.f;  // a state that has seen nothing has l = 0
    M = top;
    L = fmaf(L, alpha, e * l);
#pragma unroll
    for (int i = 0; i < kPer; ++i) acc[i] *= alpha;
    for (int32_t k = 0; k < stop; k += kAhead) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        const float wk = __shfl_sync(0xffffffffu, e, k + i);
        if (k + i < stop) {
#pragma unroll
          for (int c = 0; c < kPer; ++c) acc[c] = fmaf(wk, v[i][c], acc[c]);
          if (k + i + kAhead < stop) load(k0 + k + i + kAhead, v[i]);
        }
      }
    }
  }
  L = warp_sum(L);
  const float inv = L == 0.f ? 0.f : 1.f / L;
  const int64_t at = ((int64_t)j.b * p.Hkv + j.h) * p.rows + row;
  float* out = p.out + at * D + lane * kPer;
  if constexpr (kPer == 4)
    *reinterpret_cast<float4*>(out) = make_float4(acc[0] * inv, acc[1] * inv, acc[2] * inv, acc[3] * inv);
  else
    *reinterpret_cast<float2*>(out) = make_float2(acc[0] * inv, acc[1] * inv);
  if (p.lse && lane == 0) p.lse[at] = L == 0.f ? -INFINITY : (M + log2f(L)) * kTreeLn2;
}

template <int D, int R>
cudaError_t launch_core(const TreeParams& p, cudaStream_t stream) {
  using S = CoreSmem<D, R>;
  const cudaError_t e = allow_smem<fd_tree_core_kernel<D, R>>((int)sizeof(S));
  if (e != cudaSuccess) return e;
  return launch_early(fd_tree_core_kernel<D, R>, (unsigned)(p.ranges * p.nsub), kCoreThreads, sizeof(S), stream, p);
}

template <int D, int Rows>
cudaError_t launch_join(const TreeParams& p, cudaStream_t stream) {
  return launch_early(fd_tree_join_kernel<D, Rows>, (unsigned)(p.n_joins * p.nsub * (Rows / 8)), 256, 0, stream, p);
}

}  // namespace

cudaError_t launch_tree_core(int D, int rows, const TreeParams& p, cudaStream_t stream) {
  if (D == 128 && rows == 16) return launch_core<128, 2>(p, stream);
  if (D == 128 && rows == 32) return launch_core<128, 4>(p, stream);
  if (D == 64 && rows == 16) return launch_core<64, 2>(p, stream);
  if (D == 64 && rows == 32) return launch_core<64, 4>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_tree_join(int D, int rows, const TreeParams& p, cudaStream_t stream) {
  if (D == 128) {
    if (rows == 16) return launch_join<128, 16>(p, stream);
    if (rows == 32) return launch_join<128, 32>(p, stream);
    if (rows == 64) return launch_join<128, 64>(p, stream);
    if (rows == 128) return launch_join<128, 128>(p, stream);
  } else if (D == 64) {
    if (rows == 16) return launch_join<64, 16>(p, stream);
    if (rows == 32) return launch_join<64, 32>(p, stream);
    if (rows == 64) return launch_join<64, 64>(p, stream);
    if (rows == 128) return launch_join<64, 128>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fdk
