// fd_kv4.cuh -- device helpers of the 4-bit cache: conversions between fp32 /
// fp16 and the e2m1 codes and e4m3 scales, and block addresses.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fd_device.cuh"
#include "fd_kv4.h"

namespace fdk {

// Two e2m1 codes (low and high nibble of the byte `B` of w) as an fp16 pair, exact.
template <int B>
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t w) {
  uint32_t r;
  if constexpr (B == 0)
    asm("{\n\t.reg .b8 x, y, z, t;\n\tmov.b32 {x, y, z, t}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, x;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (B == 1)
    asm("{\n\t.reg .b8 x, y, z, t;\n\tmov.b32 {x, y, z, t}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, y;\n\t}" : "=r"(r) : "r"(w));
  else if constexpr (B == 2)
    asm("{\n\t.reg .b8 x, y, z, t;\n\tmov.b32 {x, y, z, t}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, z;\n\t}" : "=r"(r) : "r"(w));
  else
    asm("{\n\t.reg .b8 x, y, z, t;\n\tmov.b32 {x, y, z, t}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Two e4m3 values (the 16 bits of w, low byte first) as an fp16 pair, exact; 0x7f is NaN.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 x, y;\n\tmov.b32 {x, y}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
  const uint32_t h = e4m3x2_f16x2(byte & 0xffu);
  return __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
}

// x rounded to the nearest e4m3 (halfway: even), at most 448; NaN stays NaN (0x7f).
__device__ __forceinline__ uint32_t f32_e4m3(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}

// Eight values rounded to the nearest e2m1 (halfway: even), at most 6 in size; v[0] in the low nibble.
__device__ __forceinline__ uint32_t f32_e2m1x8(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 x, y, z, t;\n\tcvt.rn.satfinite.e2m1x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 y, %4, "
      "%3;\n\tcvt.rn.satfinite.e2m1x2.f32 z, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %8, %7;\n\tmov.b32 %0, {x, y, "
      "z, t};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Two values to codes: a in the low nibble of a byte, b in the high one.
__device__ __forceinline__ uint32_t f32_e2m1x2(float a, float b) {
  uint32_t r;
  asm("{\n\t.reg .b8 x;\n\tcvt.rn.satfinite.e2m1x2.f32 x, %2, %1;\n\tmov.b32 %0, {x, x, x, x};\n\t}" : "=r"(r) : "f"(a), "f"(b));
  return r & 0xffu;
}

// The larger of two, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 2^e for |e| <= kKv4MaxExp.
__device__ __forceinline__ float pow2i(int e) { return __int_as_float((e + 127) << 23); }

// Block number of token t of sequence b, KV head h; -1 for a page outside the pool.
__device__ __forceinline__ int64_t kv4_block_index(const Kv4View& kv, int32_t b, int32_t h, int32_t t) {
  if (!kv.paged) return ((int64_t)b * kv.Hkv + h) * kv.cap_blocks + t / kKv4Tokens;
  const int32_t page = __ldg(kv.block_table + (size_t)b * kv.max_pages + t / kv.page_size);
  if (page < 0 || page >= kv.num_pages) return -1;
  return ((int64_t)page * kv.Hkv + h) * (kv.page_size / kKv4Tokens) + t % kv.page_size / kKv4Tokens;
}

}  // namespace fdk
