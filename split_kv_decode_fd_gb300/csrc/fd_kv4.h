// fd_kv4.h -- the 4-bit KV cache: its block format, and the parameters of the
// kernels that write, read and attend it.
//
// A cache holds e2m1 codes (sign, two exponent bits, one mantissa bit: 0, 0.5,
// 1, 1.5, 2, 3, 4, 6) with one e4m3 scale for every sixteen consecutive
// channels of a token; a value is code * scale * 2^exp, exp being one number
// per cache for K and one for V.  (code * scale) has at most six significant
// bits and lies in [2^-10, 2688] or is 0, so it is exact in fp16 and bf16.
//
// Storage unit: the block of sixteen consecutive tokens of one KV head,
// kv4_block_bytes(D) = 18 D contiguous bytes:
//
//   K codes   [16 tokens][D / 2]   two channels a byte, the even one in the low
//             nibble; the 16-byte chunk c (channels 32c .. 32c+31) of row t sits
//             at chunk c ^ kv4_swizzle(D, t), so that eight lanes reading chunk c
//             of eight consecutive rows meet eight different bank groups;
//   V codes   [D][8]               transposed, two tokens a byte, the even one in
//             the low nibble: a lane that owns a channel reads its tokens in
//             pairs, the order in which a tensor-memory operand holds them;
//   K scales  [16 tokens][D / 16]
//   V scales  [D / 16][16 tokens]
//
// One bulk copy of 18 D bytes per block (and one for all blocks of a page or of
// a contiguous run) brings everything that attention needs.  Contiguous caches
// are [B, Hkv, capacity / 16] blocks, paged ones [num_pages, Hkv, page_size / 16].
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "fd_plan.h"

namespace fdk {

constexpr int kKv4Tokens = 16;   // tokens per block
constexpr int kKv4Channels = 16; // channels per scale
constexpr int kKv4MaxExp = 64;   // |k_exp|, |v_exp|

FD_HD constexpr int kv4_block_bytes(int D) { return 18 * D; }
FD_HD constexpr int kv4_v_off(int D) { return 8 * D; }
FD_HD constexpr int kv4_ks_off(int D) { return 16 * D; }
FD_HD constexpr int kv4_vs_off(int D) { return 17 * D; }
// 64-byte rows (D = 128): rows 2j and 2j + 1 fill 128 bytes; 32-byte rows: four of them do.
FD_HD constexpr int kv4_swizzle(int D, int t) { return D == 128 ? (t >> 1) & 3 : (t >> 2) & 1; }

// A 4-bit cache as the kernels see it.
struct Kv4View {
  uint8_t* kv;
  const int32_t* block_table;  // paged: [B, max_pages]
  int64_t cap_blocks;          // contiguous: blocks per (b, KV head)
  int32_t Hkv, paged;
  int32_t page_size, max_pages, num_pages;
  int32_t k_exp, v_exp;
};

// A bf16 or fp32 cache, for the append.
struct KvView {
  void *k, *v;
  const int32_t* block_table;
  int64_t capacity;
  int32_t Hkv, paged;
  int32_t page_size, max_pages, num_pages;
};

// The rows that an append brings (strides in elements: batch, token, head).
struct NewRows {
  const void *q, *k, *v;
  int64_t qs[3], ks[3], vs[3];
  const int32_t* new_lens;   // [B] rows that are tokens (the last ones of the n), or null
  const int32_t* positions;  // [B, n] rows of cos / sin, or null (the token's place in the sequence)
  const float *cos, *sin;    // [max_pos, rot / 2]
  int32_t max_pos, rot, interleaved;
  const int32_t* seq_lens;   // [B] lengths before the append, or null
  int32_t max_len, B, n, Hq;
  float* q_out;              // [B, Hq, n, D]
  unsigned* err;
};

cudaError_t launch_append(int D, bool rows_f32, bool cache_f32, const NewRows& r, const KvView& kv,
                          cudaStream_t stream);
cudaError_t launch_append_kv4(int D, bool rows_f32, const NewRows& r, const Kv4View& kv, cudaStream_t stream);

// Rows [start_b, start_b + n) of every sequence, as far as they lie below L_b.
struct Kv4Read {
  void *k_out, *v_out;       // [B, Hkv, n, D]
  const int32_t* starts;     // [B] or null (0)
  const int32_t* seq_lens;   // [B] or null (max_len)
  int32_t max_len, B, n;
  unsigned* err;
};
cudaError_t launch_kv4_read(int D, bool out_f32, const Kv4Read& r, const Kv4View& kv, cudaStream_t stream);

struct SplitParams;
// Decode attention: the explicit plan (grid of virtual KV heads x splits) or the balanced one (one CTA
// per SM).  With counters the last piece of a sequence joins its states into the output; without, the
// states are left for launch_combine.
cudaError_t launch_kv4_split(int D, const Kv4View& kv, const SplitParams& p, dim3 grid, cudaStream_t stream);

}  // namespace fdk
