// fd_tree.cu -- attention of a tree of drafted tokens over an fp32 cache, and the join
// of the states that the shares of a sequence leave.
//
// A row sees the places before the drafts, its token's ancestors and itself:
//     out = sum_t exp(x_t - m) v_t / sum_t exp(x_t - m),   x_t = scale q . k_t,
// over what it sees, with the running m and sum of an online softmax.
//
// A CTA serves 32 rows of a KV head from tiles of 64 keys in shared memory, and
// each thread two rows: four keys a row for q . k, D / 16 channels a row for p . V.
#include "fd_tree.cuh"

namespace fdk {
namespace {

constexpr int kRows = kTreeRowsCore;
constexpr int kKeys = 64;
constexpr int kCoreThreads = 256;

template <int D>
struct CoreSmem {
  static constexpr int kStride = D + 4;  // rows of q and k: sixteen rows apart by 16 bytes in the banks
  float q[kRows * kStride];
  float k[kKeys * kStride];
  float v[kKeys * D];
  float p[kRows * (kKeys + 4)];
  TreePiece piece;
  int32_t more;
};

__device__ __forceinline__ float4 load4(const float* p) { return __ldg(reinterpret_cast<const float4*>(p)); }

template <int D>
__global__ void __launch_bounds__(kCoreThreads, kTreeCtasCore) fd_tree_core_kernel(const TreeParams p) {
  using S = CoreSmem<D>;
  extern __shared__ __align__(16) uint8_t smem_raw[];
  S& s = *reinterpret_cast<S*>(smem_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ty = tid / 16, tx = tid % 16;
  const int32_t range = blockIdx.x / p.nsub, sub = blockIdx.x % p.nsub;
  constexpr int kCols = D / 64;  // float4 of output a row and thread
  pdl_launch_dependents();
  pdl_wait();
  tree_no_rows<D, kRows>(p, range, sub, tid, kCoreThreads);  // thread 0 also says what its pieces leave to join
  TreeWalk walk(p, range);  // every warp walks; the pieces that count are those of warp 0
  for (;;) {
    if (warp == 0) {
      TreePiece pc;
      const bool found = walk.next(pc);
      if (lane == 0) {
        s.piece = pc;
        s.more = found;
        if (found && sub == 0) walk.say(pc);
      }
    }
    __syncthreads();
    if (!s.more) return;
    const TreePiece pc = s.piece;
    const int64_t row0 = ((int64_t)pc.b * p.Hkv + pc.h) * p.rows + sub * kRows;  // of q and out
    const int32_t live = p.rows - sub * kRows < kRows ? p.rows - sub * kRows : kRows;
    for (int i = tid; i < kRows * (D / 4); i += kCoreThreads) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      const float4 x = r < live ? load4(p.q + (row0 + r) * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      *reinterpret_cast<float4*>(s.q + r * S::kStride + c) = x;
    }
    const int32_t P = pc.len - pc.m;
    const Ancestors all = tree_ancestors(p.tree, pc.b, pc.m, p.err);
    uint64_t anc[2];
    float mx[2], l[2];
    float4 o[2][kCols];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      anc[i] = all.of((sub * kRows + 2 * ty + i) % p.tree.n - (p.tree.n - pc.m));
      mx[i] = -INFINITY;
      l[i] = 0.f;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    for (int32_t t0 = pc.begin; t0 < pc.end; t0 += kKeys) {
      // rows past the piece's end hold nothing that counts: they come in as zeros
      for (int i = tid; i < kKeys * (D / 4); i += kCoreThreads) {
        const int r = i / (D / 4), c = i % (D / 4) * 4;
        const int32_t t = t0 + r;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
        if (t < pc.end) {
          int64_t at = -1;
          if (p.kv.paged) {
            const int32_t page = __ldg(p.kv.block_table + (int64_t)pc.b * p.kv.max_pages + t / p.kv.page_size);
            if (page >= 0 && page < p.kv.num_pages)
              at = ((int64_t)page * p.Hkv + pc.h) * p.kv.page_size + t % p.kv.page_size;
            else
              atomicOr(p.err, kErrBadIndex);
          } else {
            at = ((int64_t)pc.b * p.Hkv + pc.h) * p.kv.capacity + t;
          }
          if (at >= 0) {
            x = load4(static_cast<const float*>(p.kv.k) + at * D + c);
            y = load4(static_cast<const float*>(p.kv.v) + at * D + c);
          }
        }
        *reinterpret_cast<float4*>(s.k + r * S::kStride + c) = x;
        *reinterpret_cast<float4*>(s.v + r * D + c) = y;
      }
      __syncthreads();
      // q . k of rows 2 ty, 2 ty + 1 and keys tx, tx + 16, tx + 32, tx + 48
      float x[2][4] = {};
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        float4 a[2], k[4];
#pragma unroll
        for (int i = 0; i < 2; ++i) a[i] = *reinterpret_cast<const float4*>(s.q + (2 * ty + i) * S::kStride + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = *reinterpret_cast<const float4*>(s.k + (tx + 16 * j) * S::kStride + c);
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[i][j] = fmaf(a[i].x, k[j].x, x[i][j]);
            x[i][j] = fmaf(a[i].y, k[j].y, x[i][j]);
            x[i][j] = fmaf(a[i].z, k[j].z, x[i][j]);
            x[i][j] = fmaf(a[i].w, k[j].w, x[i][j]);
          }
      }
      uint32_t w[2][2];  // what the two rows see of the tile
      bool all_seen = true;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const TileMask mask = tile_mask(P, anc[i], t0);
        w[i][0] = mask.w[0];
        w[i][1] = mask.w[1];
        all_seen = all_seen && (w[i][0] & w[i][1]) == 0xffffffffu;
        float top = -INFINITY;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[i][j] = w[i][j >> 1] >> (tx + 16 * (j & 1)) & 1u ? x[i][j] * p.qk_scale : -INFINITY;
          top = fmaxf(top, x[i][j]);
        }
#pragma unroll
        for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        const float mn = fmaxf(mx[i], top);
        const float base = mn == -INFINITY ? 0.f : mn;
        const float alpha = mx[i] == -INFINITY ? 0.f : exp2f(mx[i] - base);
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float e = exp2f(x[i][j] - base);
          s.p[(2 * ty + i) * (kKeys + 4) + tx + 16 * j] = e;
          sum += e;
        }
        l[i] = fmaf(l[i], alpha, sum);
        mx[i] = mn;
#pragma unroll
        for (int c = 0; c < kCols; ++c) {
          o[i][c].x *= alpha;
          o[i][c].y *= alpha;
          o[i][c].z *= alpha;
          o[i][c].w *= alpha;
        }
      }
      __syncwarp();  // a row's weights are written and read by one half of a warp
      auto add = [&](int i, float e, int c, const float4& v) {
        o[i][c].x = fmaf(e, v.x, o[i][c].x);
        o[i][c].y = fmaf(e, v.y, o[i][c].y);
        o[i][c].z = fmaf(e, v.z, o[i][c].z);
        o[i][c].w = fmaf(e, v.w, o[i][c].w);
      };
      if (all_seen) {
#pragma unroll 4
        for (int t = 0; t < kKeys; ++t) {
          const float e0 = s.p[2 * ty * (kKeys + 4) + t], e1 = s.p[(2 * ty + 1) * (kKeys + 4) + t];
#pragma unroll
          for (int c = 0; c < kCols; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(s.v + t * D + 64 * c + 4 * tx);
            add(0, e0, c, v);
            add(1, e1, c, v);
          }
        }
      } else {
        // a value that a row does not see may be anything: 0 * NaN is not 0
#pragma unroll 1
        for (int t = 0; t < kKeys; ++t) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if (!(w[i][t >> 5] >> (t & 31) & 1u)) continue;
            const float e = s.p[(2 * ty + i) * (kKeys + 4) + t];
#pragma unroll
            for (int c = 0; c < kCols; ++c) add(i, e, c, *reinterpret_cast<const float4*>(s.v + t * D + 64 * c + 4 * tx));
          }
        }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) l[i] += __shfl_xor_sync(0xffffffffu, l[i], d);
      const int r = 2 * ty + i;
      if (r >= live || (sub * kRows + r) % p.tree.n < p.tree.n - pc.m) continue;
      const int64_t state = ((int64_t)pc.slot * p.nsub + sub) * kRows + r;
      float* to = pc.slot < 0 ? p.out + (row0 + r) * D : p.o_part + state * D;
      const float f = pc.slot >= 0 ? 1.f : (l[i] == 0.f ? 0.f : 1.f / l[i]);
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        *reinterpret_cast<float4*>(to + 64 * c + 4 * tx) =
            make_float4(o[i][c].x * f, o[i][c].y * f, o[i][c].z * f, o[i][c].w * f);
      if (tx == 0) {
        if (pc.slot >= 0) {
          p.m_part[state] = mx[i];
          p.l_part[state] = l[i];
        } else if (p.lse) {
          p.lse[row0 + r] = l[i] == 0.f ? -INFINITY : (mx[i] + log2f(l[i])) * kTreeLn2;
        }
      }
    }
    __syncthreads();  // s.piece and s.q are read
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
  const int32_t row = sub * Rows + r;
  // (a call that gave up may have left an entry of an earlier one)
  if (j.b < 0 || j.b >= p.B || j.h < 0 || j.h >= p.Hkv || j.first < 0 || j.last < j.first || j.last >= p.ranges) return;
  if (row >= p.rows || row % p.tree.n < p.tree.n - tree_tokens(p.tree, j.b)) return;
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

template <int D>
cudaError_t launch_core(const TreeParams& p, cudaStream_t stream) {
  const cudaError_t e = allow_smem<fd_tree_core_kernel<D>>((int)sizeof(CoreSmem<D>));
  if (e != cudaSuccess) return e;
  return launch_early(fd_tree_core_kernel<D>, (unsigned)(p.ranges * p.nsub), kCoreThreads, sizeof(CoreSmem<D>), stream, p);
}

template <int D, int Rows>
cudaError_t launch_join(const TreeParams& p, cudaStream_t stream) {
  return launch_early(fd_tree_join_kernel<D, Rows>, (unsigned)(p.n_joins * p.nsub * (Rows / 8)), 256, 0, stream, p);
}

}  // namespace

cudaError_t launch_tree_core(int D, const TreeParams& p, cudaStream_t stream) {
  if (D == 128) return launch_core<128>(p, stream);
  if (D == 64) return launch_core<64>(p, stream);
  return cudaErrorInvalidValue;
}

cudaError_t launch_tree_join(int D, int rows, const TreeParams& p, cudaStream_t stream) {
  if (D == 128) {
    if (rows == 32) return launch_join<128, 32>(p, stream);
    if (rows == 64) return launch_join<128, 64>(p, stream);
    if (rows == 128) return launch_join<128, 128>(p, stream);
  } else if (D == 64) {
    if (rows == 32) return launch_join<64, 32>(p, stream);
    if (rows == 64) return launch_join<64, 64>(p, stream);
    if (rows == 128) return launch_join<64, 128>(p, stream);
  }
  return cudaErrorInvalidValue;
}

}  // namespace fdk
