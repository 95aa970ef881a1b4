// fd_tree.h -- a step with a tree of drafted tokens: parameters and launches of
// the kernels that attend the drafts, decide which stay and move the rows of
// those together in the cache.
//
// Every sequence b brings n rows of drafts; with new_lens only the last
// m_b = new_lens[b] of them are tokens, and row n - m_b + j is token j.  The
// tokens' keys and values are the last m_b places of the sequence: token j has
// place P_b + j, P_b = L_b - m_b.  parents gives, row by row, the number of a
// token's parent, which is below its own, or -1.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fd_kv4.h"
#include "fd_plan.h"

namespace fdk {

constexpr int kMaxDrafts = 64;  // rows of a window: an ancestor set is one 64-bit word

struct TreeView {
  const int32_t* parents;
  int64_t parents_stride;    // elements from sequence to sequence (0: one tree for all)
  const int32_t* new_lens;   // [B] or null (n)
  int32_t n;
};

// Attention: the g * n rows of a KV head (head by head, token rows within a head,
// as q [B, Hq, n, D] has them) share its keys and values.  They are cut into
// `nsub` blocks of tree_rows() rows, and the keys of all (b, KV head) pairs into
// `ranges` shares of equal cost (BalancedWalk's line of cost units): CTA
// r * nsub + s takes share r for block s, so that the blocks of a KV head read the
// same keys at the same time, from memory once and then from L2.
//
// A pair that lies within a share is finished there.  Otherwise its states go
// to o_part, m_part (base 2) and l_part, and a second kernel joins them.  A
// share has at most two unfinished pieces: one that goes on with a pair begun in
// an earlier share (slot 2 r), and one that begins a pair (slot 2 r + 1).  Their number does not
// grow with the batch.  Where a pair begins, joins says whether and how far it goes on: an
// entry for each pair, or for each share where these are fewer.
//
// `packed` (fp32 caches): a block's rows are those of tokens alone, and each (b, KV head, block) is a pair of
// its own, so that padded batches cost what their tokens need; nsub is 1 then, and `blocks` the
// blocks of a KV head whose rows are all tokens.
struct TreeJoin {
  int32_t b, h, sub;    // sequence (-1: nothing to join), KV head, block of its rows (packed)
  int32_t first, last;  // shares that hold the pair
};

struct TreeParams {
  const float* q;              // [B, Hq, n, D]
  float* out;                  // [B, Hq, n, D]
  float* lse;                  // [B, Hq, n] natural log, or null
  const int32_t* seq_lens;     // [B] or null (max_len)
  KvView kv;
  TreeView tree;
  float* o_part;               // [2 ranges][nsub][tree_rows()][D]
  float* m_part;               // [2 ranges][nsub][tree_rows()]
  float* l_part;
  TreeJoin* joins;             // [n_joins]
  unsigned* err;
  int32_t B, Hq, Hkv, g;
  int32_t rows;                // g * n
  int32_t nsub, ranges;
  int32_t n_joins, join_pairs; // join_pairs: an entry for each pair
  int32_t packed, blocks;
  int32_t max_len;
  int32_t box_rows;            // rows that a copy of K or V brings (bf16 caches)
  float qk_scale;              // scale * log2(e)
};

// Rows per CTA and CTAs per SM: fp32 caches on CUDA cores; bf16 ones on tensor cores, up to 64 rows of a KV head with the
// keys on the rows of the products, more in blocks of 128 with the query rows there.  Measured both ways, 131072 keys of 8
// heads: 32 rows 89 us against 130, 64 rows 97 against 131 (64 paged sequences 230 against 307), 80 rows 165 us against 136, 256 rows
// 321 against 257.  A block of 128 costs the same however many of its rows there are: 65 to 128 rows 136 to 140 us, 129 to 256 rows 248 to
// 257 (blocks of 64 would be even with that from 129 to 192).  fp32, 10 rows of 16 KV heads on 2751 to 5502 keys, D = 128: blocks of 16
// rows 53 us, of 32 61.
constexpr int kTreeTileCore = 64;  // keys of a tile of the fp32 kernel
constexpr int kTreeRowsMma = 128;
constexpr int tree_rows(bool f32, int rows) {
  if (f32) return rows <= 16 ? 16 : 32;
  return rows <= 32 ? 32 : rows <= 64 ? 64 : kTreeRowsMma;
}
constexpr int tree_ctas(bool f32, int D) { return !f32 ? 1 : D == 64 ? 3 : 2; }
// Rows of a copy: as many of 64, 32, 16 as lie in a page.  A copy takes a warp some 100 cycles to start.
constexpr int tree_box_rows(int page) { return page % 64 == 0 ? 64 : page % 32 == 0 ? 32 : 16; }

cudaError_t launch_tree_core(int D, int rows, const TreeParams& p, cudaStream_t stream);
cudaError_t launch_tree_mma(int D, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                            cudaStream_t stream);
cudaError_t launch_tree_keys(int D, int rows, const CUtensorMap& tk, const CUtensorMap& tv, const TreeParams& p,
                             cudaStream_t stream);
// Joins what any of them left; rows: those of a CTA.
cudaError_t launch_tree_join(int D, int rows, const TreeParams& p, cudaStream_t stream);

// Which drafts stay (fd_verify_tree).
struct VerifyParams {
  TreeView tree;
  const int32_t* tokens;     // [B, n]
  const float* uniforms;     // [B, n]
  const void* target;        // row of token j: target + b * ts[0] + (n - m + j) * ts[1]
  const void* draft;         // likewise, or null
  int64_t ts[2], ds[2];
  int32_t* path;             // [B, n]
  int32_t* count;            // [B]
  int32_t* next_token;       // [B]
  int32_t B, V;
  unsigned* err;
};
cudaError_t launch_verify(bool f32, const VerifyParams& p, cudaStream_t stream);

// Rows together (fd_keep_rows): place start + j gets the row of place start + index[j].
struct KeepParams {
  KvView kv;
  const int32_t* index;      // [B, n]
  const int32_t* counts;     // [B] or null (n)
  const int32_t* starts;     // [B] or null (0)
  int32_t B, n, max_len;
  unsigned* err;
};
cudaError_t launch_keep(int row_bytes, const KeepParams& p, cudaStream_t stream);

}  // namespace fdk
