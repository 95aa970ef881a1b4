// fd_tcgen05.cuh -- the tcgen05 instructions of the 4-bit decode kernel and of the
// tree attention: fp16 and bf16 MMAs with A in tensor or shared memory and B in
// shared memory, and moves between registers and tensor memory (lane = row, one
// 32-bit column a register).
#pragma once

#include <stdint.h>

namespace fdk {

// Shared-memory matrix descriptor of a K-major B operand in rows of 128 bytes
// with the 128-byte swizzle: bits 0-13 start address / 16, 32-45 distance of
// eight-row groups / 16 (1024 bytes), 46 version, 61-63 swizzle (2 = 128 bytes).
__device__ __forceinline__ uint64_t b_desc(uint32_t saddr) {
  constexpr uint32_t kHi = (1024u >> 4) | (1u << 14) | (2u << 29);
  return ((uint64_t)kHi << 32) | ((saddr >> 4) & 0x3FFFu);
}

// The same of an N-major B operand without a swizzle: 16 bytes hold eight n of one
// k, consecutive k are 16 bytes apart (bits 16-29: distance of eight k / 16), the next
// eight n `n_stride` bytes on (bits 32-45).
template <int NStride>
__device__ __forceinline__ uint64_t b_desc_n(uint32_t saddr) {
  constexpr uint32_t kHi = ((uint32_t)NStride >> 4) | (1u << 14);
  return ((uint64_t)kHi << 32) | ((128u >> 4) << 16) | ((saddr >> 4) & 0x3FFFu);
}

// Instruction descriptor of kind::f16: fp32 accumulator, A and B fp16, A K-major, B
// K-major or (bit 16) N-major.
__host__ __device__ constexpr uint32_t f16_instr_desc(int M, int N, bool b_n_major = false) {
  return (1u << 4) | ((b_n_major ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The same with A and B bf16.
__host__ __device__ constexpr uint32_t bf16_instr_desc(int M, int N, bool b_n_major = false) {
  return f16_instr_desc(M, N, b_n_major) | (1u << 7) | (1u << 10);
}

// The descriptor of an N-major B operand in rows (of K) of 128 bytes with the 128-byte
// swizzle: eight rows are 1024 bytes apart, the next 64 n `n_stride` bytes on.
__device__ __forceinline__ uint64_t b_desc_rows(uint32_t saddr, uint32_t n_stride) {
  return b_desc(saddr) | ((uint64_t)(n_stride >> 4) << 16);
}

// D[tmem] (+)= A[smem] B: 128 rows, 16 of K; A's descriptor is as b_desc's.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// D[tmem] (+)= A[tmem] B: 128 rows, 16 of K.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

// The barrier's phase completes once every MMA this thread issued before has.
__device__ __forceinline__ void mma_commit(uint32_t bar_saddr) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar_saddr)
               : "memory");
}

__device__ __forceinline__ void tmem_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_loads() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_stores() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// All 512 columns, their address to shared memory; one warp.
__device__ __forceinline__ void tmem_alloc_all(uint32_t slot_saddr) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(slot_saddr) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_all(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base) : "memory");
}

// NC consecutive columns of this thread's lane: a power of two up to 32.
template <int NC>
struct TmemRow;
template <>
struct TmemRow<2> {
  static __device__ __forceinline__ void load(uint32_t at, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0, %1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(at));
  }
  static __device__ __forceinline__ void tie(uint32_t* r) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]));
  }
  static __device__ __forceinline__ void store(uint32_t at, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1, %2};" ::"r"(at),
                 "r"(r[0]), "r"(r[1])
                 : "memory");
  }
};
template <>
struct TmemRow<4> {
  static __device__ __forceinline__ void load(uint32_t at, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at));
  }
  static __device__ __forceinline__ void tie(uint32_t* r) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]));
  }
  static __device__ __forceinline__ void store(uint32_t at, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3])
                 : "memory");
  }
};
template <>
struct TmemRow<8> {
  static __device__ __forceinline__ void load(uint32_t at, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "r"(at));
  }
  static __device__ __forceinline__ void tie(uint32_t* r) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]));
  }
  static __device__ __forceinline__ void store(uint32_t at, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
  }
};
template <>
struct TmemRow<16> {
  static __device__ __forceinline__ void load(uint32_t at, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
                 : "r"(at));
  }
  static __device__ __forceinline__ void tie(uint32_t* r) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
  }
  static __device__ __forceinline__ void store(uint32_t at, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
                 : "memory");
  }
};
template <>
struct TmemRow<32> {
  static __device__ __forceinline__ void load(uint32_t at, uint32_t* r) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
                 : "r"(at));
  }
  static __device__ __forceinline__ void tie(uint32_t* r) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]));
  }
  static __device__ __forceinline__ void store(uint32_t at, const uint32_t* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(at),
                 "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
                 : "memory");
  }
};

// Complete on return (the empty asm ties the registers to the point after the wait).
template <int NC>
__device__ __forceinline__ void tmem_load(uint32_t at, float* v) {
  uint32_t r[NC];
  TmemRow<NC>::load(at, r);
  tmem_wait_loads();
  TmemRow<NC>::tie(r);
#pragma unroll
  for (int i = 0; i < NC; ++i) v[i] = __uint_as_float(r[i]);
}

// Not waited for.
template <int NC>
__device__ __forceinline__ void tmem_store(uint32_t at, const float* v) {
  uint32_t r[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) r[i] = __float_as_uint(v[i]);
  TmemRow<NC>::store(at, r);
}
__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) { TmemRow<16>::store(at, r); }

}  // namespace fdk
