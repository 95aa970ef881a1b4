// fd_tree_tc.cuh -- what the two tensor-core kernels of the tree attention share: waits, rings, and the
// cut of fp32 numbers into three bf16 ones.
#pragma once

#include "fd_tcgen05.cuh"
#include "fd_tree.cuh"

namespace fdk {

constexpr int kParts = 3;  // bf16 numbers that q and p are cut into

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Pairs of floats in one register pair: the packed arithmetic rounds each as the scalar one does.
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
// 32 bytes in one store where the address allows it: 16-byte stores of rows far apart send each sector to L2 twice.
__device__ __forceinline__ void store32(float* to, const float* v) {
  if ((reinterpret_cast<uintptr_t>(to) & 31) == 0) {
    asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  } else {
    reinterpret_cast<float4*>(to)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(to)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// The upper 16 bits of both, x's in the low half: their bf16 truncations.
__device__ __forceinline__ uint32_t trunc2(float x, float y) {
  return __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
}
__device__ __forceinline__ float trunc1(float x) { return __uint_as_float(__float_as_uint(x) & 0xffff0000u); }

// x and y as sums of three bf16 numbers each, exactly (24 bits = 3 x 8).
__device__ __forceinline__ void cut3(float x, float y, uint32_t (&w)[kParts]) {
  w[0] = trunc2(x, y);
  float a, b;
  unpack2(sub2(pack2(x, y), pack2(trunc1(x), trunc1(y))), a, b);
  w[1] = trunc2(a, b);
  float c, d;
  unpack2(sub2(pack2(a, b), pack2(trunc1(a), trunc1(b))), c, d);
  w[2] = trunc2(c, d);
}

// One lane of a converged warp, known as such to the compiler.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ uint32_t uniform(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

// Waits of all roles: false when the CTA gives up or the limit runs out.
struct Waits {
  volatile int* abort;
  unsigned long long limit;
  bool ok = true;
  __device__ __forceinline__ void on(uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_try_wait(bar, parity)) ok = !*abort && mbar_wait_for(bar, parity, limit);
  }
  // The warp's lanes alike.
  __device__ __forceinline__ bool all() {
    ok = __all_sync(0xffffffffu, ok);
    return ok;
  }
};

// Uses of the ring: slot u % n in phase u / n.
template <uint32_t N>
struct Ring {
  uint32_t slot = 0, phase = 0;
  __device__ __forceinline__ void next(uint32_t by = 1) {
    slot += by;
    if (slot >= N) {
      slot -= N;
      phase ^= 1u;
    }
  }
};

// Copies of K or V tiles by one warp: lane l holds the place of the tile's rows [box l, box (l + 1)), a run of a page.
// A tile lies in NB blocks of 64 channels, [128 rows][128 bytes] with the 128-byte swizzle.
// The lanes start their copies side by side: with a loop of one elected lane, and a second form of the copy for paged
// caches, 64 paged sequences took 301 us, and 273 so.
constexpr uint32_t kTileBlock = 16384;
struct TileCopy {
  const TreeParams& p;
  int32_t box, boxes;
  uint64_t once;  // read by CTAs of the same time: the lines leave L2 first

  __device__ __forceinline__ explicit TileCopy(const TreeParams& p_)
      : p(p_), box(p_.box_rows), boxes(kPlanTile / p_.box_rows), once(policy_evict_first()) {}

  // This lane's page of tile j.
  __device__ __forceinline__ int32_t page_of(const TreePiece& pc, int32_t j) const {
    const int32_t lane = threadIdx.x & 31, t = pc.begin + j * kPlanTile + box * lane;
    return p.kv.paged && lane < boxes && t < pc.end
               ? __ldg(p.kv.block_table + (int64_t)pc.b * p.kv.max_pages + t / p.kv.page_size)
               : -1;
  }
  template <int NB>
  __device__ __forceinline__ void start(const CUtensorMap* map, const TreePiece& pc, int32_t j, int32_t page, uint8_t* to,
                                        uint64_t* full) const {
    const int32_t lane = threadIdx.x & 31, t = pc.begin + j * kPlanTile + box * lane;
    bool mine = lane < boxes && t < pc.end;
    int32_t row = t, z = pc.b * p.Hkv + pc.h;
    if (p.kv.paged) {
      if (mine && (page < 0 || page >= p.kv.num_pages)) {
        atomicOr(p.err, kErrBadIndex);
        mine = false;
      }
      row = t % p.kv.page_size;
      z = page * p.Hkv + pc.h;
    }
    const uint32_t which = __ballot_sync(0xffffffffu, mine);
    if (elect_one()) mbar_arrive_expect_tx(full, (uint32_t)(__popc(which) * box) * NB * 128u);
    __syncwarp();
    if (mine) {
      uint8_t* dst = to + (uint32_t)(lane * box) * 128u;
#pragma unroll 1
      for (int blk = 0; blk < NB; ++blk) tma_load_3d_hint(dst + blk * kTileBlock, map, full, blk * 64, row, z, once);
    }
    __syncwarp();
  }
};

// Waits for the last use of each of a ring's n slots (u uses so far), so that the CTA does not leave while a copy may still be
// landing.  A warp that copies does so at its end in any case: the products wait for every copy, but another role may give up
// after this warp has ended well.
__device__ __forceinline__ void land(uint64_t* full, uint32_t u, uint32_t n, unsigned long long limit) {
  for (uint32_t x = u > n ? u - n : 0; x < u; ++x) mbar_wait_for(full + x % n, (x / n) & 1, limit);
}

}  // namespace fdk
