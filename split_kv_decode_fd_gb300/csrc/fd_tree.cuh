// fd_tree.cuh -- what the tree attention kernels share: what a row sees, the
// walk over a share of the keys, and where a piece's states go.
#pragma once

#include <atomic>

#include "fd_device.cuh"
#include "fd_tree.h"

namespace fdk {

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
  return d;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t sub2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Cost units (kTileUnits = 4 a tile of 128 keys) that a piece costs a CTA besides its tiles: q and the first tile's way
// through the roles, some 4 us or three tiles of 64 rows.  64 paged sequences of 512 to 16384 tokens, with 6, 12 and 20: 64 rows of a
// KV head 248, 229, 233 us; 32 rows 186, 189, 192; D = 64, 64 rows 230, 214, 217 and 32 rows 142, 132, 136; with the query rows on the products' rows,
// 128 of them 312, 308, 316 and 256 626, 620, 655.  One value serves all but 128 rows of D = 64 (238, 254, 254), where a tile is short beside the piece.
constexpr int kTreePieceUnits = 12;
// The same of the fp32 kernel, in units of four a tile of 64 keys (32 sequences of up to 4096 tokens, with 2, 4 and 8: 64 rows of D = 128
// 586, 591, 603 us, 32 of D = 64 147, 150, 153).
constexpr int kTreePieceUnitsCore = 4;

__device__ __forceinline__ int32_t tree_len(const TreeParams& p, int32_t b) {
  return p.seq_lens ? clamp_len(__ldg(p.seq_lens + b), p.max_len) : p.max_len;
}
__device__ __forceinline__ int32_t tree_tokens(const TreeView& t, int32_t b) {
  return t.new_lens ? clamp_len(__ldg(t.new_lens + b), t.n) : t.n;
}

// The ancestors of every token and itself, as words of bits: lane l of the warp
// holds those of tokens l and l + 32.  Twice as far up in each round, as a chain of
// 64 tokens would otherwise be 64 loads one after another.  A parent that is not
// below its token counts as none and is reported; m: the sequence's tokens.
struct Ancestors {
  uint64_t lo, hi;
  // token j's, for any j of any lane (a warp-collective call)
  __device__ __forceinline__ uint64_t of(int32_t j) const {
    const uint64_t a = __shfl_sync(0xffffffffu, lo, j & 31), b = __shfl_sync(0xffffffffu, hi, j & 31);
    return j < 0 ? 0 : (j < 32 ? a : b);
  }
};
__device__ __forceinline__ Ancestors tree_ancestors(const TreeView& t, int32_t b, int32_t m, unsigned* err) {
  const int32_t lane = threadIdx.x & 31;
  const int32_t* parents = t.parents + b * t.parents_stride + (t.n - m);
  int32_t x[2];
  Ancestors a;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int32_t j = lane + 32 * i;
    x[i] = j < m ? __ldg(parents + j) : -1;
    if (x[i] < -1 || x[i] >= j) {
      if (x[i] != -1) atomicOr(err, kErrBadIndex);
      x[i] = -1;
    }
  }
  a.lo = lane < m ? 1ull << lane : 0;
  a.hi = lane + 32 < m ? 1ull << (lane + 32) : 0;
  while (__any_sync(0xffffffffu, x[0] >= 0 || x[1] >= 0)) {
    const uint64_t up0 = a.of(x[0]), up1 = a.of(x[1]);
    int32_t y[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int32_t s = __shfl_sync(0xffffffffu, x[0], x[i] & 31), l = __shfl_sync(0xffffffffu, x[1], x[i] & 31);
      y[i] = x[i] < 0 ? -1 : (x[i] < 32 ? s : l);
    }
    a.lo |= up0;
    a.hi |= up1;
    x[0] = y[0];
    x[1] = y[1];
  }
  return a;
}

// Bits [0, 128) of a tile of keys that starts at place t0: which of them a row sees
// that sees every place below P, and place P + a for each bit a of `anc`.  The bits
// of places at or past the sequence's end are 0, as anc has none there.
struct TileMask {
  uint32_t w[4];
};
__device__ __forceinline__ TileMask tile_mask(int32_t P, uint64_t anc, int32_t t0) {
  TileMask t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int32_t d = P - (t0 + 32 * i);  // where bit 0 of anc falls in this word
    const uint32_t before = d <= 0 ? 0u : (d >= 32 ? 0xffffffffu : (1u << d) - 1u);
    uint32_t own;
    if (d >= 32 || d <= -64)
      own = 0u;
    else if (d >= 0)
      own = (uint32_t)(anc << d);
    else
      own = (uint32_t)(anc >> -d);
    t.w[i] = before | own;
  }
  return t;
}

// A run of keys of one (sequence, KV head).
struct TreePiece {
  int32_t b, h, sub;
  int32_t begin, end;  // places, `end` clipped to the length
  int32_t len, m;      // the sequence's length and its tokens
  int32_t slot;        // -1: the piece is the whole pair
  int32_t tiles;       // of the pair
  int64_t v;           // the pair's first cost unit
};

// Blocks of `Packed` rows of a KV head of a sequence of m tokens, each a pair of its own; 0: not packed.
template <int Packed>
__device__ __forceinline__ int32_t tree_blocks(const TreeParams& p, int32_t m) {
  if constexpr (Packed == 0) return 1;
  else return ceil_div(p.g * m, Packed);
}

// The pieces of one share, walked by one warp (all lanes alike).  Sequences
// without keys or without tokens cost nothing and have no piece.  Lane l holds length and
// tokens of sequence base + l.
template <int Packed>
struct TreeWalk {
  static constexpr int kTile = Packed > 0 ? kTreeTileCore : kPlanTile;
  const TreeParams& p;
  int64_t units;
  int32_t used, range;
  int64_t pos, end;
  int32_t b, len, m, tiles;
  int32_t i, heads;      // number of the pair in its sequence, and of those
  int64_t v;             // first unit of the pair
  int32_t u;             // units of a pair of its sequence
  int32_t base, my_len, my_m;

  __device__ __forceinline__ bool uniform() const { return !p.seq_lens && !p.tree.new_lens; }
  __device__ __forceinline__ int32_t piece_units() const { return p.seq_lens ? (Packed > 0 ? kTreePieceUnitsCore : kTreePieceUnits) : 0; }
  __device__ __forceinline__ int32_t units_of(int32_t n, int32_t tokens) const {
    return tokens > 0 ? (int32_t)pair_units(ceil_div(n, kTile), piece_units()) : 0;
  }
  __device__ __forceinline__ void block(int32_t b0) {
    const int32_t i = b0 + (int32_t)(threadIdx.x & 31);
    base = b0;
    my_len = i < p.B ? tree_len(p, i) : 0;
    my_m = i < p.B ? tree_tokens(p.tree, i) : 0;
  }
  __device__ __forceinline__ void load(int32_t bb) {
    if (!uniform() && (bb < base || bb >= base + 32)) block(bb & ~31);
    b = bb;
    len = uniform() ? p.max_len : __shfl_sync(0xffffffffu, my_len, bb & 31);
    m = uniform() ? p.tree.n : __shfl_sync(0xffffffffu, my_m, bb & 31);
    tiles = m > 0 ? ceil_div(len, kTile) : 0;
    u = units_of(len, m);
    heads = p.Hkv * tree_blocks<Packed>(p, m);
  }

  __device__ __forceinline__ TreeWalk(const TreeParams& p_, int32_t range_, bool walks = true) : p(p_), range(range_) {
    const int lane = threadIdx.x & 31;
    pos = end = 0;
    b = i = base = my_len = my_m = 0;
    v = 0;
    if (!walks) return;
    if (uniform()) {
      load(0);
      units = (int64_t)p.B * heads * u;
    } else {
      int64_t sum = 0;
      for (int32_t b0 = (p.B - 1) & ~31; b0 >= 0; b0 -= 32) {  // the first block stays at hand
        block(b0);
        sum += (int64_t)units_of(my_len, my_m) * tree_blocks<Packed>(p, my_m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      units = sum * p.Hkv;
    }
    used = units > 0 ? balanced_ctas(units, p.ranges) : 0;
    if (range >= used) return;
    pos = range_begin(units, used, range);
    end = range_begin(units, used, range + 1);
    // the sequence that holds `pos`
    if (uniform()) {
      const int64_t pair = div_floor(pos, u);
      b = (int32_t)div_floor(pair, heads);
      i = (int32_t)(pair - (int64_t)b * heads);
      v = pair * u;
      return;
    }
    int64_t before = 0;
    for (int32_t i0 = 0; i0 < p.B; i0 += 32) {
      if (i0 != base) block(i0);
      const int64_t mine = (int64_t)units_of(my_len, my_m) * tree_blocks<Packed>(p, my_m);
      int64_t incl = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      const unsigned past = __ballot_sync(0xffffffffu, (before + incl) * p.Hkv > pos);
      if (past) {
        const int l = __ffs(past) - 1;
        const int64_t start = (before + __shfl_sync(0xffffffffu, incl - mine, l)) * p.Hkv;
        load(i0 + l);
        i = (int32_t)div_floor(pos - start, u);
        v = start + (int64_t)i * u;
        return;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    pos = end;  // not reached: pos is below the units in all
  }

  // The next piece; false when none is left.
  __device__ __forceinline__ bool next(TreePiece& pc) {
    while (pos < end) {
      const int64_t pend = v + u;
      const int64_t stop = end < pend ? end : pend;
      const int32_t lo = first_tile_at(pos, v, piece_units());
      int32_t hi = first_tile_at(stop, v, piece_units());
      hi = hi < tiles ? hi : tiles;
      const bool found = hi > lo;
      if (found) {
        pc.b = b;
        pc.h = i;
        pc.sub = 0;
        if constexpr (Packed > 0) {
          const int32_t per = tree_blocks<Packed>(p, m);
          pc.h = i / per;
          pc.sub = i % per;
        }
        pc.begin = lo * kTile;
        pc.end = hi < tiles ? hi * kTile : len;
        pc.len = len;
        pc.m = m;
        pc.slot = lo == 0 && hi == tiles ? -1 : 2 * range + (lo == 0 ? 1 : 0);
        pc.tiles = tiles;
        pc.v = v;
      }
      pos = stop;
      if (pos == pend) {
        v = pend;
        if (++i == heads) {
          i = 0;
          if (uniform()) {
            ++b;
          } else if (pos < end) {  // the walk ends inside the units in all, so a sequence with units follows
            int32_t bb = b + 1;
            load(bb);
            while (u == 0 && bb < p.B - 1) load(++bb);
          }
        }
      }
      if (found) return true;
    }
    return false;
  }

  // Before the first piece: the share begins no pair that goes on, for the join.  One lane, the one that says what its pieces
  // leave: it writes the same entry, and nothing else orders the two stores.
  __device__ __forceinline__ void say_none() const {
    if (!p.join_pairs) p.joins[range].b = -1;
  }
  // Says of the pair that `pc` begins (if it does) whether it goes on.
  __device__ __forceinline__ void say(const TreePiece& pc) const {
    if (pc.begin != 0 || (pc.slot < 0 && !p.join_pairs)) return;
    TreeJoin j{-1, pc.h, pc.sub, range, range};
    if (pc.slot >= 0) {
      j.b = pc.b;
      j.last = cta_of_unit(units, used, pc.v + piece_units() + (int64_t)kTileUnits * (pc.tiles - 1));
    }
    p.joins[p.join_pairs ? ((int64_t)pc.b * p.Hkv + pc.h) * p.blocks + pc.sub : range] = j;
  }
};

// Sequences without keys or tokens: no share holds them.  The rows of their tokens get
// out = 0, lse = -inf, and their pairs nothing to join, from the CTAs of share b % ranges.  (Entries of pairs alone, which no
// piece has: an entry of a share is written by the walk.)
template <int D, int Rows, int Packed>
__device__ __forceinline__ void tree_no_rows(const TreeParams& p, int32_t range, int32_t sub, int tid, int threads) {
  for (int32_t b = range; b < p.B; b += p.ranges) {
    const int32_t len = tree_len(p, b), m = tree_tokens(p.tree, b);
    if (p.join_pairs && sub == 0) {
      const int32_t live = len == 0 || m == 0 ? 0 : tree_blocks<Packed>(p, m);
      if (live < p.blocks)
        for (int32_t i = tid; i < p.Hkv * p.blocks; i += threads)
          if (i % p.blocks >= live) p.joins[(int64_t)b * p.Hkv * p.blocks + i].b = -1;
    }
    if (len != 0) continue;
    const int32_t pad = p.tree.n - m;
    const int32_t r0 = sub * Rows, r1 = Packed == 0 && r0 + Rows < p.rows ? r0 + Rows : p.rows;
    for (int64_t i = tid; i < (int64_t)p.Hkv * (r1 - r0); i += threads) {
      const int32_t row = r0 + (int32_t)(i % (r1 - r0));
      if (row % p.tree.n < pad) continue;
      const int64_t at = ((int64_t)b * p.Hkv + i / (r1 - r0)) * p.rows + row;
#pragma unroll 1
      for (int d = 0; d < D; d += 4) *reinterpret_cast<float4*>(p.out + at * D + d) = make_float4(0.f, 0.f, 0.f, 0.f);
      if (p.lse) p.lse[at] = -INFINITY;
    }
  }
}

constexpr float kTreeLn2 = 0.6931471805599453f;

// Lets a kernel take `bytes` of dynamic shared memory, once per device.  Regs: a kernel whose roles share its registers
// out anew waits forever if it was not launched with as many a thread as the shares add up to: any other build of it is refused.
template <auto Kernel, int Regs = 0>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  if constexpr (Regs > 0) {
    cudaFuncAttributes of;
    e = cudaFuncGetAttributes(&of, Kernel);
    if (e != cudaSuccess) return e;
    if ((of.numRegs + 7) / 8 * 8 != Regs) return cudaErrorInvalidConfiguration;  // they are given out by eights
  }
  e = cudaFuncSetAttribute(Kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// A launch whose set-up overlaps the end of the kernel before: the kernel waits for that one
// (griddepcontrol.wait) before its first access to memory.
template <class... A>
cudaError_t launch_early(void (*kernel)(A...), unsigned grid, int threads, size_t smem, cudaStream_t stream, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace fdk
