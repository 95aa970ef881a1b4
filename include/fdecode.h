/*
 * fdecode.h -- C ABI of libfdecode: split-KV decode attention (Flash-Decoding)
 * for NVIDIA GB300 (sm_103a).
 *
 * What is computed (per batch b and query head h, one query row each):
 *
 *     out[b,h,:] = softmax(scale * q[b,h,:] . K_b^T) . V_b     over keys t < L_b
 *     lse[b,h]   = ln sum_t exp(scale * q[b,h,:] . k_t)
 *
 * The KV sequence is cut into splits; each split runs an online softmax and
 * leaves an unnormalised partial output O_s with its running max m_s and sum
 * l_s; a log-sum-exp merge rescales each partial by exp(m_s - M), sums, and
 * divides once by the global sum.  Sources, by page and section:
 *   - "Kernel visualization: Flash Decoding" (tinyvolt.com): the fd_split
 *     walkthrough (per-split online softmax, partials written unnormalised)
 *     and "Combine kernel -- one thread block per (batch, head)" (the merge);
 *   - "attn-flash-decoding" (zenaique.com): "What decode looks like" (shapes
 *     Q (batch, n_heads, 1, d_head), K/V (batch, n_kv_heads, T, d_head)) and
 *     the answer on why the log-sum-exp combine is exact;
 *   - "FlashDecoding and split-KV" (guide.dupenodi.dev), "Walking through it":
 *     paged or ragged KV layouts and GQA head grouping.
 *
 * Conventions fixed by this library where the pages are silent:
 *   - GQA: g = Hq / Hkv; query head h reads KV head h / g (integer division).
 *   - lse is a natural log; m_part is in the natural units of scale*q.k.
 *   - L_b == 0 gives out = 0 and lse = -inf.  Keys at t >= L_b (padding, and
 *     block-table entries at index >= ceil(L_b / page_size)) are never read.
 *   - Paged pool layout [num_pages, Hkv, page_size, D]: token t of sequence b
 *     is row t % page_size of page block_table[b * max_pages_per_seq + t / page_size].
 *
 * General rules for every call:
 *   - Pointers are DEVICE pointers unless the name ends in _host.
 *   - All memory is owned by the caller; the library allocates nothing.  The
 *     one exception is the fixed FD_STATIC_SCRATCH_BYTES device array that
 *     fd_decode_static uses in place of a workspace (see there).
 *   - Calls enqueue work on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) and return without waiting, except fd_decode_host and
 *     fd_workspace_status, which synchronise the stream.
 *   - Arguments are checked on the host before anything is enqueued; on an
 *     error no kernel is launched and no memory is touched.
 *   - Supported: D in {64, 128}; K/V in FD_BF16 or FD_F32; q, out, lse, partials
 *     in fp32; Hq % Hkv == 0; page_size a multiple of 16.  q, out, o_part, k, v
 *     must be 16-byte aligned; q/out/partials are dense row-major.
 *   - Results are deterministic: no floating-point atomics; repeated calls
 *     give bit-identical outputs.
 */
#ifndef FDECODE_H_
#define FDECODE_H_

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define FD_API __attribute__((visibility("default")))
#else
#define FD_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef enum fd_status {
  FD_OK = 0,
  FD_ERR_INVALID_ARG = 1,         /* null pointer, bad size, misalignment, Hq % Hkv != 0 ... */
  FD_ERR_UNSUPPORTED = 2,         /* head_dim, dtype or size outside what this build handles */
  FD_ERR_WORKSPACE_TOO_SMALL = 3, /* workspace_bytes < fd_workspace_bytes(...) */
  FD_ERR_BAD_INDEX = 4,           /* a kernel met a block-table entry outside [0, num_pages), or another index outside its range */
  FD_ERR_CUDA = 5,                /* a CUDA runtime/driver call failed (launch, copy, ...) */
  FD_ERR_TIMEOUT = 6              /* a kernel's internal wait gave up (never expected) */
} fd_status;

typedef enum fd_dtype { FD_F32 = 0, FD_BF16 = 1 } fd_dtype;

typedef enum fd_kv_layout { FD_KV_CONTIGUOUS = 0, FD_KV_PAGED = 1 } fd_kv_layout;

/* n_splits value asking the library to plan the split itself (balanced over the SMs). */
#define FD_SPLITS_AUTO 0

/*
 * Largest batch the balanced (FD_SPLITS_AUTO) plan handles in one fused
 * launch; larger batches, or more than 65536 (batch, KV head) pairs, are run
 * with a fixed split count chosen by the library instead.
 */
#define FD_AUTO_MAX_BATCH 1024

/*
 * The KV cache.  All pointers are device pointers.
 *   contiguous: k, v are [B, Hkv, capacity, D]; block_table etc. are ignored.
 *   paged:      k, v are [num_pages, Hkv, page_size, D]; block_table is
 *               [B, max_pages_per_seq] int32, row-major; capacity is ignored.
 */
typedef struct fd_kv_desc {
  fd_kv_layout layout;
  fd_dtype dtype;               /* element type of k and v */
  const void* k;
  const void* v;
  int64_t capacity;             /* contiguous: padded length T_cap of every sequence */
  const int32_t* block_table;   /* paged only */
  int32_t max_pages_per_seq;    /* paged only: row length of block_table */
  int32_t page_size;            /* paged only: tokens per page, multiple of 16 */
  int32_t num_pages;            /* paged only: pages in the pool */
} fd_kv_desc;

/*
 * Bytes of device workspace needed by fd_decode and fd_decode_host.
 * n_splits: FD_SPLITS_AUTO or the explicit split count that will be passed.
 * num_sms:  SM count of the device that will run the call; 0 = query the
 *           current device.  Returns 0 for invalid arguments.
 * The workspace must be zero-filled once after allocation (fd_workspace_init);
 * every successful call, of any shape, leaves it valid for the next call (the
 * merge's arrival counters sit in a fixed-size region and end each call at
 * zero).  One workspace serves one call at a time: calls that share a
 * workspace must be ordered (same stream, or synchronised).
 */
FD_API size_t fd_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t n_splits,
                          int32_t num_sms);

/* Zero-fill a workspace (cudaMemsetAsync on `stream`). */
FD_API fd_status fd_workspace_init(void* workspace, size_t workspace_bytes, void* stream);

/*
 * Synchronise `stream`, then report (and clear) the error word that kernels
 * of earlier calls on this workspace may have raised: FD_OK, FD_ERR_BAD_INDEX
 * or FD_ERR_TIMEOUT.  Kernels never trap; they record and skip instead.
 */
FD_API fd_status fd_workspace_status(void* workspace, size_t workspace_bytes, void* stream);

/*
 * Tokens per split when the caller fixes n_splits > 0:
 *   S = 16 * ceil(ceil(max_seq_len / n_splits) / 16);
 * split s of sequence b covers tokens [s*S, min((s+1)*S, L_b)).
 * (The fd_split sketch takes the split size S as a parameter with
 * n_start = s*S, n_end = min(n_start + S, N).)  Returns 0 on bad arguments.
 */
FD_API int32_t fd_split_size(int32_t max_seq_len, int32_t n_splits);

/*
 * Full decode attention: split + merge, enqueued on `stream`.
 *   q        [B, Hq, D] fp32.
 *   out      [B, Hq, D] fp32 (written).
 *   lse      [B, Hq] fp32 natural-log softmax denominator, or NULL.
 *   seq_lens [B] int32 valid lengths L_b, or NULL (= every L_b is max_seq_len).
 *            Values are clamped to [0, max_seq_len] on the device.
 *   max_seq_len  upper bound of every L_b; contiguous: <= capacity;
 *            paged: <= max_pages_per_seq * page_size.
 *   scale    multiplies q.k (callers usually pass 1/sqrt(D)).
 *   n_splits FD_SPLITS_AUTO (the library balances the keys of all
 *            sequences over one CTA per SM) or the number of splits per sequence.
 *   workspace/workspace_bytes  zero-initialised device scratch of at least
 *            fd_workspace_bytes(B, Hq, Hkv, D, n_splits, 0) bytes.
 * One kernel launch (split with the merge fused in: the last CTA to finish a
 * sequence merges it); two launches only when more than 65536 (batch, KV head)
 * pairs need merging.  Errors in arguments return before any launch.
 */
FD_API fd_status fd_decode(const float* q, const fd_kv_desc* kv, float* out, float* lse, int32_t B,
                    int32_t Hq, int32_t Hkv, const int32_t* seq_lens, int32_t max_seq_len, int32_t D,
                    float scale, int32_t n_splits, void* workspace, size_t workspace_bytes,
                    void* stream);

/*
 * Decode with n_q query rows per (batch, head) sharing one read of K/V, for a
 * few new tokens per sequence (e.g. verifying speculative tokens): the page
 * "FlashDecoding and split-KV", section "Walking through it", lets decode carry
 * n_q slightly above one and leaves the masking of those rows open.
 *   q    [B, Hq, n_q, D] fp32; out [B, Hq, n_q, D]; lse [B, Hq, n_q] or NULL.
 *   causal = 1: the n_q rows are the last n_q tokens, already in the cache, and
 *            row i attends keys t < L_b - (n_q - 1 - i); causal = 0: every row
 *            attends all L_b keys.  A row with no key gives out = 0, lse = -inf.
 *   1 <= n_q <= 64.  Other arguments as in fd_decode; the workspace is
 *   fd_workspace_bytes(B, Hq * n_q, Hkv, D, n_splits, 0).  The rows of a GQA
 *   group are served together (up to 16 rows x heads per bf16 K/V read, 8 per
 *   fp32 read).
 */
FD_API fd_status fd_decode_rows(const float* q, int32_t n_q, int32_t causal, const fd_kv_desc* kv, float* out,
                                float* lse, int32_t B, int32_t Hq, int32_t Hkv, const int32_t* seq_lens,
                                int32_t max_seq_len, int32_t D, float scale, int32_t n_splits, void* workspace,
                                size_t workspace_bytes, void* stream);

/*
 * Fused append-KV + decode (the "fused append-KV" path named in "FlashDecoding
 * and split-KV", section "Walking through it"; the operation is this
 * library's reading of it): for every sequence b the new token's key and
 * value are written into the cache at position L_b and the decode then
 * attends the L_b + 1 keys, in one launch.  The result equals writing the row
 * first and calling fd_decode with lengths L_b + 1 (bit for bit).
 *   k_new, v_new  [B, Hkv, D] device, in the cache dtype (kv->dtype), 16-byte
 *                 aligned; their bits are stored unchanged.
 *   seq_lens / max_seq_len  the lengths BEFORE the append (seq_lens is read,
 *                 not updated: the caller advances its lengths).
 *   kv            kv->k and kv->v are written (one row per (b, KV head)).
 *                 Contiguous: capacity >= max_seq_len + 1.  Paged: the page
 *                 holding position L_b must already be in the block table;
 *                 an entry outside [0, num_pages) skips the cache write and
 *                 is reported as FD_ERR_BAD_INDEX by fd_workspace_status (the
 *                 output still includes the new token).
 *   Other arguments as in fd_decode; the workspace is the same size.
 */
FD_API fd_status fd_append_decode(const float* q, const void* k_new, const void* v_new, const fd_kv_desc* kv,
                                  float* out, float* lse, int32_t B, int32_t Hq, int32_t Hkv,
                                  const int32_t* seq_lens, int32_t max_seq_len, int32_t D, float scale,
                                  int32_t n_splits, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Attention for many query rows per sequence (prefill, or a long window of new
 * tokens): the same operation as fd_decode_rows -- q [B, Hq, n_q, D], the rows
 * are the last n_q tokens of each sequence, causal or not -- computed with
 * query tiles of 128 rows on the tensor cores (tcgen05.mma, TMEM
 * accumulators) instead of rows-as-heads.  "FlashDecoding and split-KV",
 * section "Walking through it": prefill has many query rows and wants
 * FlashAttention's tiling along them; decode has one.
 *   Supports D = 64 and 128 with a bf16 cache (contiguous or paged); any n_q >= 1.
 *   workspace: at least 256 bytes, zero-filled once (its first word is the
 *   kernels' error word, read by fd_workspace_status; bytes 128-135 hold the
 *   kernel's work-queue counters, which every call leaves at zero, so calls
 *   that share a workspace must not overlap in time).  out, lse as in
 *   fd_decode_rows.  One launch, asynchronous on `stream`.
 *   FD_ERR_CUDA, with nothing launched, also when the kernel variant for an odd
 *   group size (one query head per CTA, which redistributes registers between
 *   its warps) was not compiled with the register count it assumes.
 */
FD_API fd_status fd_prefill(const float* q, int32_t n_q, int32_t causal, const fd_kv_desc* kv, float* out,
                            float* lse, int32_t B, int32_t Hq, int32_t Hkv, const int32_t* seq_lens,
                            int32_t max_seq_len, int32_t D, float scale, void* workspace, size_t workspace_bytes,
                            void* stream);

/*
 * Phase dispatch ("FlashDecoding and split-KV", "Walking through it": serving
 * engines pick a kernel per phase and should log which one ran).  fd_attend
 * picks the backend for n_q query rows per sequence and reports it:
 *   FD_BACKEND_DECODE       n_q == 1                      -> fd_decode
 *   FD_BACKEND_DECODE_ROWS  n_q * (Hq / Hkv) <= 16, or no prefill kernel for
 *                           this D / dtype and n_q <= 64  -> fd_decode_rows
 *   FD_BACKEND_PREFILL      otherwise (D = 64 or 128, bf16) -> fd_prefill
 * fd_attend_backend returns the choice without running anything (-1: no
 * backend); fd_backend_name names it.  The workspace must fit the chosen
 * backend: fd_workspace_bytes(B, Hq * n_q, Hkv, D, n_splits, 0) for the decode
 * backends, 256 bytes for prefill.  *backend (may be NULL) receives the choice.
 */
#define FD_BACKEND_DECODE 0
#define FD_BACKEND_DECODE_ROWS 1
#define FD_BACKEND_PREFILL 2
FD_API int32_t fd_attend_backend(int32_t n_q, int32_t Hq, int32_t Hkv, int32_t D, int32_t kv_dtype);
FD_API const char* fd_backend_name(int32_t backend);
FD_API fd_status fd_attend(const float* q, int32_t n_q, int32_t causal, const fd_kv_desc* kv, float* out,
                           float* lse, int32_t B, int32_t Hq, int32_t Hkv, const int32_t* seq_lens,
                           int32_t max_seq_len, int32_t D, float scale, int32_t n_splits, void* workspace,
                           size_t workspace_bytes, void* stream, int32_t* backend);

/* ------------------------------------------------------------------ rotating append
 *
 * New rows of every sequence into a KV cache, their keys (and the queries)
 * rotated by position on the way.  The sources name appending to paged caches
 * ("FlashDecoding and split-KV", section "Walking through it") without a
 * format; these calls are this library's reading, and what stands before
 * fd_decode, fd_decode_rows, fd_prefill or fd_decode_kv4 in a serving loop.
 *
 * A pair (a, b) of channels of a q or k row at position p turns into
 *     a cos[p, i] - b sin[p, i],   b cos[p, i] + a sin[p, i],
 * in fp32, for the rot_dim / 2 pairs i of the first rot_dim channels: (i, i +
 * rot_dim / 2), or (2i, 2i + 1) when interleaved.  The other channels, and v,
 * are taken as they are.  k and v are rounded once to the cache's type; q comes
 * out in fp32 as [B, Hq, n, D], which the attention calls take.
 *
 * Every sequence brings n rows; with new_lens, only the last new_lens[b] of them
 * are tokens (the convention of fd_decode_rows, whose rows are the last ones of
 * the sequence), and the padding rows before them are neither read nor written,
 * in q_out too.  Token j of sequence b goes to place L_b + j of its cache, L_b being
 * the length before the call (seq_lens is read, not updated).  Its row of the
 * tables is that place, or positions[b, i] of its row i when given (a tree of drafts, a
 * sequence whose positions do not start at zero).
 */
typedef struct fd_new_rows {
  fd_dtype dtype;               /* of q, k and v: FD_BF16 or FD_F32 */
  const void* q;                /* [B, n, Hq, D] by strides; unused when Hq = 0 */
  const void* k;                /* [B, n, Hkv, D] by strides */
  const void* v;
  int64_t q_stride[3];          /* elements from batch to batch, row to row, head to head; the D */
  int64_t k_stride[3];          /*   channels of a head are contiguous.  Bases and strides are */
  int64_t v_stride[3];          /*   multiples of 16 bytes; a stride may be 0 (a broadcast input) */
  const int32_t* new_lens;      /* [B] rows that are tokens, or NULL (= n); clamped to [0, n] */
  const int32_t* positions;     /* [B, n] or NULL */
  const float* cos;             /* [max_pos, rot_dim / 2]; may be NULL when rot_dim = 0 */
  const float* sin;
  int32_t max_pos;              /* rows of the tables */
  int32_t rot_dim;              /* 0 (no rotation) or a multiple of 32 up to D */
  int32_t interleaved;          /* 0 or 1 */
} fd_new_rows;

/*
 * Append into a bf16 or fp32 cache (kv->k and kv->v are written).
 *   seq_lens / max_seq_len  lengths BEFORE the append, or NULL (= every L_b is
 *             max_seq_len); the cache must hold max_seq_len + n tokens, and without
 *             `positions` so must the tables.
 *   workspace at least 256 bytes, zero-filled once: its first word is the
 *             error word that fd_workspace_status reads; nothing else of it is used,
 *             so a call may share it with any other.  A page outside [0, num_pages)
 *             (that k and v row is not written) or a position outside [0, max_pos)
 *             (nor is that q row) is reported as FD_ERR_BAD_INDEX.
 * One launch.  Two sequences of one call must not bring tokens to the same place
 * of the same page: which of the two stays is not defined.
 */
FD_API fd_status fd_append_rope(const fd_new_rows* rows, const fd_kv_desc* kv, float* q_out, int32_t B, int32_t n,
                                int32_t Hq, int32_t Hkv, const int32_t* seq_lens, int32_t max_seq_len, int32_t D,
                                void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ 4-bit KV cache
 *
 * e2m1 codes (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4,
 * 6) with one e4m3 scale for every sixteen consecutive channels of a token:
 *     value = code * scale * 2^exp,     exp = k_exp for K, v_exp for V.
 * Writing x: y = x * 2^-exp; scale = the largest |y| of the sixteen / 6, rounded to
 * nearest (even) and held to 448; code = y / scale rounded to nearest (even) and
 * held to 6 in size (0 where the scale is 0).  An infinity so becomes 6 * 448 * 2^exp; a NaN
 * makes the scale, and with it the sixteen values, NaN.
 *
 * The unit of storage is the block of sixteen consecutive tokens of one KV head,
 * fd_kv4_block_bytes(D) = 18 D bytes:
 *     K codes  [16 tokens][D / 2], two channels a byte, the even one in the low
 *              nibble; 16-byte chunk c of row t sits at chunk c ^ ((t / 2) % 4) for
 *              D = 128, c ^ ((t / 4) % 2) for D = 64;
 *     V codes  [D][8], two tokens a byte, the even one in the low nibble;
 *     K scales [16][D / 16];   V scales [D / 16][16].
 * Contiguous: [B, Hkv, capacity / 16] blocks.  Paged: [num_pages, Hkv, page_size /
 * 16] blocks.  kv must be 16-byte aligned.  Bytes of a block that no token was
 * written to are read but never reach a result.
 */
typedef struct fd_kv4_desc {
  fd_kv_layout layout;
  void* kv;
  int64_t capacity;             /* contiguous: tokens per sequence, a multiple of 16 */
  const int32_t* block_table;   /* paged only: [B, max_pages_per_seq] */
  int32_t max_pages_per_seq;
  int32_t page_size;            /* a multiple of 16 */
  int32_t num_pages;
  int32_t k_exp, v_exp;         /* in [-64, 64] */
} fd_kv4_desc;

/* 18 D for D = 64 or 128, else 0. */
FD_API int32_t fd_kv4_block_bytes(int32_t D);

/*
 * fd_append_rope into a 4-bit cache.  The sixteen channels of a scale are taken
 * after the rotation.  A block is written by one sequence at a time: besides
 * the rule above, two sequences of one call must not bring tokens to the same
 * block.  A page outside [0, num_pages) leaves out the block's tokens.
 */
FD_API fd_status fd_append_rope_kv4(const fd_new_rows* rows, const fd_kv4_desc* kv, float* q_out, int32_t B, int32_t n,
                                    int32_t Hq, int32_t Hkv, const int32_t* seq_lens, int32_t max_seq_len, int32_t D,
                                    void* workspace, size_t workspace_bytes, void* stream);

/*
 * Rows of a 4-bit cache as bf16 or fp32 values: for every sequence the tokens
 * t = starts[b] + i, i < n, that lie below L_b, to row i of k_out and v_out [B, Hkv,
 * n, D] (16-byte aligned).  Rows at or past L_b are left as they were.  starts NULL
 * = 0; starts and lengths are clamped to [0, max_seq_len].  bf16 holds every value exactly
 * (fp32 too).  A page outside the pool leaves its rows out and is reported as
 * FD_ERR_BAD_INDEX.  Workspace as for fd_append_rope.
 */
FD_API fd_status fd_kv4_read(const fd_kv4_desc* kv, void* k_out, void* v_out, fd_dtype dtype, int32_t B, int32_t n,
                             int32_t Hkv, const int32_t* starts, const int32_t* seq_lens, int32_t max_seq_len,
                             int32_t D, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Decode attention over a 4-bit cache, 1 <= n_q <= 64 query rows per (batch,
 * head): fd_decode_rows (n_q = 1: fd_decode) on the cache's values, with the same layouts of
 * q, out and lse, the same masking, lengths and split arguments, and a workspace of
 * fd_workspace_bytes(B, Hq * n_q, Hkv, D, n_splits, 0) bytes.  A page outside the pool
 * counts as keys with score 0 and value 0, and is reported as FD_ERR_BAD_INDEX.
 * q is held to 22 bits of each head's largest channel, a softmax weight to 22 bits of
 * itself down to 2^-23 of the largest and to 2^-45 of the largest below; products and sums
 * are fp32.  Scores may have any size that fp32 holds.  A NaN key shows in the rows that see it; a NaN
 * value of one of the last n_q tokens in every row of the window, those before the
 * token too (its weight there is 0, and 0 * NaN is NaN), and of an older token in all
 * rows, as it should.
 */
FD_API fd_status fd_decode_kv4(const float* q, int32_t n_q, int32_t causal, const fd_kv4_desc* kv, float* out,
                               float* lse, int32_t B, int32_t Hq, int32_t Hkv, const int32_t* seq_lens,
                               int32_t max_seq_len, int32_t D, float scale, int32_t n_splits, void* workspace,
                               size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------ trees of drafted tokens
 *
 * A step that checks several drafted tokens at once, arranged in a tree: each
 * sequence brings n rows, and with new_lens only the last m_b = new_lens[b] of
 * them are tokens (as in fd_append_rope): row n - m_b + j is token j.  Token 0 is
 * usually the last accepted token and the root of the drafts.  The tokens' keys and
 * values are the last m_b places of the sequence in the cache: with P_b = L_b - m_b,
 * token j has place P_b + j (fd_append_rope, with the depths as `positions`, writes
 * them there).  Places below 0 do not exist.
 *
 * fd_decode_tree attends them, fd_verify_tree says which stay, fd_keep_rows moves
 * the rows of those together in the cache.
 */
#define FD_MAX_DRAFTS 64

typedef struct fd_tree_desc {
  const int32_t* parents;       /* row by row: the number of the token's parent, below its own, or -1 */
  int64_t parents_stride;       /* elements from sequence to sequence; 0: one tree for all */
  const int32_t* new_lens;      /* [B] or NULL (= n); clamped to [0, n] */
  int32_t n;                    /* rows of every sequence, 1 to FD_MAX_DRAFTS */
} fd_tree_desc;

/*
 * Attention of the drafted tokens: token j sees every place below P_b, its
 * ancestors in the tree, and itself.  (With parents j - 1 this is fd_decode_rows with
 * causal = 1.)
 *   q    [B, Hq, n, D] fp32; out [B, Hq, n, D]; lse [B, Hq, n] or NULL.  Rows of
 *        padding are not written.  A token that sees no place gives out = 0, lse = -inf.
 *   seq_lens / max_seq_len  L_b, the drafts included, as in fd_decode.
 *   workspace  zero-filled once, fd_tree_workspace_bytes(B, Hq, Hkv, D, n, 0) bytes.
 * Keys and values that a token does not see may be anything, NaN included.  Over a bf16
 * cache an infinite key that a token sees, or an infinite value before the drafts, may give NaN
 * where the sums in fp32 give an infinity, or (a key that makes a score of -inf) a number: there q and
 * the weights are sums of bf16 numbers, some of them 0, and 0 times an infinity is NaN.  It
 * touches the rows of its sequence and KV head, a value its channel alone.  A
 * parent that is not below its token counts as -1 and is reported as FD_ERR_BAD_INDEX
 * by fd_workspace_status, and so is a page outside the pool, which leaves the
 * sequence's output undefined.  One launch, and a second one that joins the states
 * where a sequence may be longer than a tile of 128 keys (64 over an fp32 cache).
 */
FD_API size_t fd_tree_workspace_bytes(int32_t B, int32_t Hq, int32_t Hkv, int32_t D, int32_t n, int32_t num_sms);
FD_API fd_status fd_decode_tree(const float* q, const fd_tree_desc* tree, const fd_kv_desc* kv, float* out, float* lse,
                                int32_t B, int32_t Hq, int32_t Hkv, const int32_t* seq_lens, int32_t max_seq_len,
                                int32_t D, float scale, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Which drafts stay.  The walk starts at token 0, which stays.  Where it stands at a
 * token with the target's probabilities p and the draft's q (those of the word after the
 * token), the token's children are asked in the order of their numbers: the child with word x and
 * random number u stays, and the walk goes on there, if
 *     u Z q(x) < r(x),    r = max(p - c q, 0),   c = 0, Z = 1 at first;
 * when it does not, c grows by Z and Z becomes the sum of r.  That is the rule that
 * keeps the target's distribution when the children are drawn from q one by one: r / Z is what is
 * left of the target.  Without `draft` the children are given, not drawn: u Z < r(x), with
 * r = p but 0 at refused words, and Z = 1 less their probabilities.  Where no child
 * stays, the next token is the first word v with r(0) + ... + r(v) > u_0 * sum r (of p
 * itself if nothing is left), u_0 being token 0's random number.
 *   tokens     [B, n] int32 words of the drafts, row by row (token 0's is not used).
 *   uniforms   [B, n] fp32 random numbers in [0, 1).
 *   target     p of token j is V probabilities in FD_F32 or FD_BF16 (dtype) at element
 *              b * target_stride[0] + (n - m_b + j) * target_stride[1]; draft likewise, or
 *              NULL.  They need not be normalised to the last bit; what is not above 0, NaN too,
 *              counts as 0.  Rows need no alignment beyond their type's (16 bytes are
 *              faster).  The draft's rows of tokens without children are not read.
 *   path       [B, n]: the numbers of the tokens that stay, token 0 first, then -1.
 *   count      [B]: how many they are.   next_token [B].  A sequence without tokens gets 0 and -1,
 *              and -1 stands for a target row without a positive probability.
 *   Sums are pairs of fp32 numbers, of which an accumulator adds up to N = V / 512 + 8 words, in small batches
 *   V / 4096 + 8.  They are off by at most (N^2 + 128 N + 2000) 2^-48 times the sum of p + c q, and as a rule by
 *   2^-48 times that for V = 131072 and 2^-42 for 2^22: only a random number that close to the border
 *   between two words, or to a child's, can have another outcome than exact sums give.
 *   workspace  at least 256 bytes, zero-filled once, of which only the error word is used.
 * A child whose word is outside [0, V), or a token whose parent is not below it, is left out
 * (FD_ERR_BAD_INDEX).  One launch.
 */
FD_API fd_status fd_verify_tree(const fd_tree_desc* tree, const int32_t* tokens, const float* uniforms,
                                const void* target, const int64_t target_stride[2], const void* draft,
                                const int64_t draft_stride[2], fd_dtype dtype, int32_t* path, int32_t* count,
                                int32_t* next_token, int32_t B, int32_t V, void* workspace, size_t workspace_bytes,
                                void* stream);

/*
 * Rows that stay, moved together in a bf16 or fp32 cache: for every sequence b and j <
 * counts[b], place starts[b] + j gets the keys and values that place starts[b] + index[b, j] held
 * before the call.  index [B, n] int32 rises along a sequence (index[b, j] <
 * index[b, j + 1], from 0).  counts NULL = n, else clamped to [0, n]; starts NULL = 0.  With
 * fd_verify_tree: index = path, counts = count, starts = P_b (the lengths before the drafts).
 *   max_seq_len  places at or past it are not touched; as in fd_decode.
 * An entry that does not rise, or whose place lies at or past max_seq_len, ends the list
 * there, for all heads alike: it and those after it are left out (a negative start: all).  A page outside the
 * pool leaves out its rows.  Both are reported as FD_ERR_BAD_INDEX.  Two sequences of one call must
 * not share pages that a row moves from or to.  Workspace as for fd_append_rope.  One launch.
 */
FD_API fd_status fd_keep_rows(const fd_kv_desc* kv, const int32_t* index, int32_t n, const int32_t* counts,
                              const int32_t* starts, int32_t B, int32_t Hkv, int32_t max_seq_len, int32_t D,
                              void* workspace, size_t workspace_bytes, void* stream);

/*
 * Split step only ("fd_split" of the walkthrough), with n_splits > 0 splits
 * per sequence of fd_split_size(max_seq_len, n_splits) tokens each.  Writes:
 *   o_part [B, Hq, n_splits, D]  unnormalised sum_t exp(s_t - m_s) v_t
 *   m_part [B, Hq, n_splits]     running max m_s of scale*q.k (natural units)
 *   l_part [B, Hq, n_splits]     sum_t exp(s_t - m_s)
 * A split with no keys holds O = 0, m = -inf, l = 0.  Other arguments as in
 * fd_decode.  Needs no workspace.
 */
FD_API fd_status fd_split_partial(const float* q, const fd_kv_desc* kv, int32_t B, int32_t Hq, int32_t Hkv,
                           const int32_t* seq_lens, int32_t max_seq_len, int32_t D, float scale,
                           int32_t n_splits, float* o_part, float* m_part, float* l_part,
                           void* stream);

/*
 * Merge step only (the combine walkthrough): per (b, h), over splits with
 * l > 0:  M = max m_s,  L = sum exp(m_s - M) l_s,
 *         out = sum exp(m_s - M) O_s / L,  lse = M + ln L  (lse may be NULL).
 * If no split has keys: out = 0, lse = -inf.  Layouts as in fd_split_partial.
 */
FD_API fd_status fd_combine(const float* o_part, const float* m_part, const float* l_part, float* out,
                     float* lse, int32_t B, int32_t Hq, int32_t D, int32_t n_splits, void* stream);

/*
 * fd_decode with the per-step inputs and outputs in HOST memory: q_host
 * [B,Hq,D], seq_lens_host [B] (or NULL), out_host [B,Hq,D] and lse_host
 * [B,Hq] (or NULL).  Pinned (page-locked, device-mapped) buffers are used in
 * place: the kernels read q and the lengths and write out and lse over the
 * host link, with no staging copy (q_host and out_host must then start on a
 * 16-byte boundary, else they are staged).  Pageable buffers are copied
 * through the staging area inside `workspace` (q and lengths in, out and lse
 * back).  Synchronises `stream` before returning, so the host may rewrite
 * q_host and seq_lens_host as soon as the call returns.  The KV cache (kv)
 * stays device-resident.  Workspace as for fd_decode.
 */
FD_API fd_status fd_decode_host(const float* q_host, const fd_kv_desc* kv, float* out_host, float* lse_host,
                         int32_t B, int32_t Hq, int32_t Hkv, const int32_t* seq_lens_host,
                         int32_t max_seq_len, int32_t D, float scale, int32_t n_splits,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * fd_decode without a workspace, for callers that cannot allocate device
 * memory: code handed only its input and output buffers by a host framework
 * (plugin or custom-operator interfaces that own every allocation), and code
 * that must not call cudaMalloc on its path because cudaMalloc can synchronise
 * the device and stall work running on other streams.  The pages have no
 * counterpart to this call; it is a deployment variant of fd_decode.
 *   Arguments as in fd_decode, minus the workspace.  The scratch (error word,
 *   merge counters, split partials) is one file-scope device array of
 *   FD_STATIC_SCRATCH_BYTES inside the library; every GPU that loads the
 *   library holds it until the process exits.
 *   Every call looks the array's device address up on the current device
 *   (cudaGetSymbolAddress); the first call on a device also loads the
 *   library's module there, so make that first call before any stream capture.
 *   Returns FD_ERR_WORKSPACE_TOO_SMALL, before any launch, when the problem
 *   needs more scratch than the array holds (fd_workspace_bytes of the same
 *   problem, minus its host-staging part, is the amount needed).
 *   Allocates nothing: no cudaMalloc or cudaFree.  Each call clears the error
 *   word and the counters (cudaMemsetAsync) and then launches as fd_decode.
 *   All calls share the one array, and it keeps the last call's contents:
 *   calls that overlap on the GPU (different streams, other host threads)
 *   race on it and must be ordered by the caller.
 *   Kernel-side errors (a block-table entry outside the pool, a wait that
 *   gave up) are recorded in the array's error word: read them with
 *   fd_static_status after the call and before the next fd_decode_static
 *   call on that device, which clears the word.
 */
#define FD_STATIC_SCRATCH_BYTES (16u << 20)

FD_API fd_status fd_decode_static(const float* q, const fd_kv_desc* kv, float* out, float* lse, int32_t B,
                                  int32_t Hq, int32_t Hkv, const int32_t* seq_lens, int32_t max_seq_len,
                                  int32_t D, float scale, int32_t n_splits, void* stream);

/*
 * fd_workspace_status for fd_decode_static: synchronise `stream`, then report
 * (and clear) the error word in the library's static scratch array on the
 * current device -- FD_OK, FD_ERR_BAD_INDEX or FD_ERR_TIMEOUT, raised by the
 * kernels of the most recent fd_decode_static call there.  Like that call it
 * has no counterpart on the pages and allocates nothing.
 */
FD_API fd_status fd_static_status(void* stream);

/*
 * Host-side description of the work decomposition, for inspection and tests
 * (touches no GPU).  Enumerates every split piece that fd_decode would run
 * for these lengths on `grid` CTAs (FD_SPLITS_AUTO) or for n_splits > 0, for
 * a cache of dtype kv_dtype (an fd_dtype).
 * Each piece is 7 int32: {cta, b, virtual_kv_head, tok_begin, tok_end, slot,
 * pieces_of_its_sequence} (the last is the arrival count that triggers the
 * fused merge).  A virtual KV head is a KV head with up to 16 (bf16 cache) or
 * 8 (fp32 cache) of its query heads; when Hq / Hkv is at most that, it is the
 * KV head itself.
 * Writes at most `capacity` pieces and returns the total count (negative on
 * bad arguments).  seq_lens_host may be NULL (every L_b = max_seq_len).
 */
FD_API int64_t fd_plan_pieces(int32_t B, int32_t Hq, int32_t Hkv, int32_t kv_dtype, const int32_t* seq_lens_host,
                              int32_t max_seq_len, int32_t n_splits, int32_t grid, int32_t* pieces,
                              int64_t capacity);

/*
 * Testing hook for the kernels' bounded waits; off by default.  Every
 * mbarrier wait of the split and prefill kernels gives up after a time limit
 * (2 s by default), records FD_ERR_TIMEOUT in the error word, lets the copies
 * it issued land and exits, so the context stays usable.  With stage >= 0, the
 * kernels launched afterwards skip, in every CTA that reaches it, the copies of
 * stage number `stage` (split kernels: fd_decode and every call built on it,
 * fd_split_partial; fd_decode_kv4) or K/V tile copy number `stage` (fd_prefill, K and V
 * counted separately), so the waits for it run out; wait_limit_ns > 0 shortens
 * every wait of those kernels to that many nanoseconds (0 keeps the default).  The
 * call's output is then undefined and fd_workspace_status (or
 * fd_static_status) reports FD_ERR_TIMEOUT; the workspace stays valid for the
 * next call.  stage < 0 switches the hook off and restores the default limit.
 * A process-wide setting, read when a call is made.
 */
FD_API void fd_debug_stall(int32_t stage, int64_t wait_limit_ns);

/* Static description of a status code. */
FD_API const char* fd_status_string(fd_status status);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
FD_API int32_t fd_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FDECODE_H_ */
