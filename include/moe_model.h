/*
 * moe_model.h - C ABI of the sequence-side operators of the decoder that the
 * MoE layer (moe.h) belongs to: the per-head norm and rotation of queries and
 * keys, a quantised paged key/value cache with the attention that reads it,
 * and sampling of the next token.
 *
 * Conventions are those of moe.h: every call returns a moe_status_t and
 * nothing throws or exits; calls are asynchronous, ordered by `cuda_stream`
 * (a cudaStream_t; NULL = the legacy default stream), run on the current
 * device, allocate nothing and can be captured in a CUDA graph.  A call keeps
 * no state: two calls may run at once on different streams when neither
 * writes what the other reads or writes (a workspace included).
 * On an error nothing is launched.  All are forward operators.
 */
#ifndef MOE_MODEL_GB300_H
#define MOE_MODEL_GB300_H

#include "moe.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types of activations. */
enum { MOE_BF16 = 0, MOE_FP16 = 1, MOE_FP32 = 2 };

/*
 * Rows of heads, [token][head][D]: the elements of a head are contiguous;
 * strides count elements and are multiples of 8, data is 16-byte aligned.
 * A slice of a packed projection (q, k and v of a token side by side) is one.
 * Inputs may repeat rows (a stride of 0); rows of an output may not overlap
 * (INVALID_ARG).
 */
typedef struct {
  void* data; /* device */
  int64_t token_stride;
  int64_t head_stride;
} moe_heads_t;

/*
 * Per-head RMSNorm and rotation, one pass:
 *   n = x / sqrt(mean(x^2) + eps) * (weight + weight_offset)     (over the D elements of a head)
 *   (a, b) -> (a cos - b sin, b cos + a sin)                     (over pairs of the first rot_dim elements)
 * in fp32, rounded once to the activations' type.  Pair i is (i, i + rot_dim/2),
 * or (2i, 2i + 1) when interleaved; its angle is the table's entry i of the
 * token's position.  weight_offset 1 serves zero-centred weights.
 * moe_rope_table fills a table; its angles are computed in binary64, so far
 * positions keep their accuracy.
 */
typedef struct {
  const void* q_weight; /* device [D] in the activations' type, 16-byte aligned, or NULL: 1 (weight_offset is then not added) */
  const void* k_weight; /* likewise */
  const float* table;   /* device fp32 [n_positions][rot_dim/2][2] (cos, sin), 16-byte aligned; may be NULL when rot_dim is 0 */
  int32_t n_positions;
  int32_t rot_dim;      /* a multiple of 16, 0..D */
  int32_t interleaved;  /* 0 or 1 */
  float eps;            /* >= 0 */
  float weight_offset;
} moe_norm_rope_t;

/*
 * Host: cos and sin of position * base^(-2 i / rot_dim) for positions
 * 0 .. n_positions - 1, into host memory fp32 [n_positions][rot_dim/2][2].
 * Errors: INVALID_ARG (NULL, n_positions < 1, rot_dim not a positive multiple of 16, base not positive and finite).
 */
MOE_API moe_status_t moe_rope_table(int32_t n_positions, int32_t rot_dim, double base, float* table_host);

/*
 * Norm and rotation of n_q query heads and n_kv key heads of n_tokens
 * tokens.  head_dim: a multiple of 8, 8..256.  q_out may be q and k_out may
 * be k (in place); other overlaps are not allowed.  n_q or n_kv may be 0.
 * positions: device int32 [n_tokens], or NULL when rot_dim is 0.  A token of
 * negative position is padding: its rows of q_out and k_out stay as they
 * were.  A position of n_positions or more has no angle: its rows are NaN.
 * dtype: MOE_BF16 or MOE_FP16.
 * Errors: INVALID_ARG (NULL or misaligned pointers, bad sizes, strides or eps), UNSUPPORTED (dtype MOE_FP32, over 65535 heads), CUDA.
 */
MOE_API moe_status_t moe_qk_norm_rope(const moe_norm_rope_t* desc, int32_t dtype, int32_t n_tokens, int32_t head_dim,
                                      int32_t n_q, const moe_heads_t* q, const moe_heads_t* q_out, int32_t n_kv,
                                      const moe_heads_t* k, const moe_heads_t* k_out, const int32_t* positions,
                                      void* cuda_stream);

/*
 * The quantised paged cache.  Keys and values are held in blocks of 32
 * elements along D with one fp16 scale each (the block size and quantiser of
 * the expert weights):
 *   bits 8: d = fp16(amax / 127), value = d * (u - 128), u - 128 = clamp(round_half_even(x / d), -127, 127)
 *   bits 4: d = fp16(amax / 7),   value = d * (u - 8),   u - 8   = clamp(round_half_even(x / d), -8, 7)
 * A block whose d is 0 holds zeros.  A block with a NaN or with a magnitude
 * above 65024 (infinity among them) reads back as NaN: its d is NaN.
 *
 * Layout (a page of the pool; a program that moves pages needs no more than
 * moe_kv_page_bytes): [kv head][page_size / 32 tiles]; a tile holds 32
 * consecutive tokens of one head, R = D * bits / 8:
 *   K values [32][R], K scales fp16 [D/32][32], V values [32][R], V scales fp16 [D/32][32]
 * Element i of a 4-bit row is in byte i/2, low nibble for even i.  The
 * 16-byte chunk c of value row r is stored as chunk c ^ (f(r) & (R/16 - 1)),
 * f(r) = ((r >> 2 ^ r) & 1) << 2 | (r & 2) | (r >> 2 & 1), which spreads the
 * attention's shared-memory reads over the banks.
 *
 * The status word collects what a call's own bounds checks found on the
 * device (bits below, set by atomic or, never cleared by a call).
 */
enum {
  MOE_KV_BAD_PAGE = 1,   /* a block-table entry outside 0..n_pages-1, or a length beyond the table's width, was met */
  MOE_KV_BAD_BATCH = 2,  /* cu_tokens not ascending or beyond n_tokens, or a sequence with more new tokens than its length or than max_tokens */
  MOE_KV_TIMEOUT = 4     /* a wait inside a kernel (two seconds) ran out: outputs are invalid */
};

typedef struct {
  void* data;         /* device, 16-byte aligned, n_pages * moe_kv_page_bytes(); caller-owned */
  size_t data_bytes;
  int32_t n_pages;    /* >= 1 */
  int32_t page_size;  /* tokens a page: a multiple of 32, 32..4096 */
  int32_t n_kv_heads; /* 1..1024 */
  int32_t head_dim;   /* D: 64, 128 or 256 */
  int32_t bits;       /* 8 or 4 */
  int32_t* status;    /* device, one word; caller-owned, zeroed by the caller */
} moe_kv_cache_t;

/*
 * A ragged batch.  Sequence b's new tokens are rows cu_tokens[b] ..
 * cu_tokens[b+1] - 1 of q, k, v and the outputs, and they are the last of its
 * seq_lens[b] positions: row cu_tokens[b] + i has position seq_lens[b] -
 * (cu_tokens[b+1] - cu_tokens[b]) + i.  Position p lives in page
 * block_table[b][p / page_size], row p % page_size.  Rows behind
 * cu_tokens[n_seqs] (a padded batch) have no effect and are not written.
 * The arrays are read on the device when the call runs, so a captured graph
 * follows their contents.
 */
typedef struct {
  const int32_t* block_table; /* device [n_seqs][table_stride] */
  const int32_t* seq_lens;    /* device [n_seqs]: positions that hold tokens, the new ones included */
  const int32_t* cu_tokens;   /* device [n_seqs + 1], ascending from 0 */
  int32_t n_seqs;             /* 1..65536 */
  int32_t table_stride;       /* entries from one row of block_table to the next, >= max_pages */
  int32_t max_pages;          /* entries of a row, >= 1; max_pages * page_size < 2^31 */
  int32_t n_tokens;           /* rows of q, k, v and the outputs, >= cu_tokens[n_seqs], < 2^31 - 256; 0: the call does nothing */
  int32_t max_tokens;         /* the most new tokens of one sequence, 1..n_tokens; the attention is planned for it: a loose bound
                                 is right, but takes a decode batch to the kernel for prompts, at about twice the time */
} moe_kv_batch_t;

/* Bytes of one page, 0 when the arguments are not a cache's. */
MOE_API size_t moe_kv_page_bytes(int32_t page_size, int32_t n_kv_heads, int32_t head_dim, int32_t bits);

/*
 * Quantise the batch's new k and v [n_tokens][n_kv_heads][D] into their
 * pages.  The pages that two sequences write must be distinct: rows written
 * twice by one call hold a mixture of both.  New tokens of negative position
 * and those whose page is bad are not stored (status).
 * Errors: INVALID_ARG, UNSUPPORTED (dtype MOE_FP32), CUDA.
 */
MOE_API moe_status_t moe_kv_append(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t dtype,
                                   const moe_heads_t* k, const moe_heads_t* v, void* cuda_stream);

/*
 * moe_qk_norm_rope of q and k and moe_kv_append of the result and v in one
 * pass (k never makes the round trip through memory); bit-identical to the
 * two calls.  positions: the tokens' positions for the rotation, NULL: their cache positions.
 * A token of negative position is padding: it is skipped altogether.  q_out may be q.
 */
MOE_API moe_status_t moe_kv_append_norm_rope(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch,
                                             const moe_norm_rope_t* desc, int32_t dtype, int32_t n_q,
                                             const moe_heads_t* q, const moe_heads_t* q_out, const moe_heads_t* k,
                                             const moe_heads_t* v, const int32_t* positions, void* cuda_stream);

/*
 * Read the batch's tokens back: row cu_tokens[b] + i of k_out and v_out
 * becomes d * (u - bias), rounded once to dtype, at that row's position (a
 * batch whose token counts are its lengths reads whole sequences).  Rows of
 * negative position or of a bad page are NaN.
 */
MOE_API moe_status_t moe_kv_read(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t dtype,
                                 const moe_heads_t* k_out, const moe_heads_t* v_out, void* cuda_stream);

/*
 * Attention of the batch's new tokens over their sequences' cached
 * positions, the new ones included (append first):
 *   out = softmax(scale * q k^T over positions <= the token's) v
 * Query head j reads kv head j / (n_q / n_kv_heads).  Scores, softmax
 * statistics and sums are fp32; probabilities and dequantised values enter
 * the products as fp16, and so do, with many rows or behind a shared prefix,
 * dequantised keys.  With fp16 activations only the values are rounded there,
 * and otherwise only the probabilities: what the other roundings leave is a
 * second operand.  lse (fp32 [n_tokens][n_q], or NULL): the natural
 * logarithm of the sum of exp(score).  A token of negative position sees
 * nothing: its out is 0 and its lse -infinity.  A row that sees a bad page, or
 * a position behind the table's width, is NaN.  One that sees a value block of
 * NaN is NaN in the block's elements at least, and may be in all, its lse
 * included.  What lies behind the position a row sees never reaches that row.
 * out may be q; other overlaps are not allowed.
 * shared_tokens (a multiple of page_size, 0 = off) says that the block tables
 * of all sequences begin with the same pages up to that position, so that
 * those keys may be read once for the whole batch, which is done where it
 * spares reading a million keys.  Results equal those of shared_tokens = 0 up
 * to rounding.
 * workspace: device, 16-byte aligned, of moe_kv_attend_workspace bytes; its
 * contents need no preparation and mean nothing afterwards.  Calls that
 * overlap need workspaces of their own.
 * Errors: INVALID_ARG, UNSUPPORTED (dtype MOE_FP32, max_tokens * n_q / n_kv_heads
 * over 2^24, or more than 2^31 - 1 groups of 16 rows), OUT_OF_MEMORY (workspace too small), CUDA.
 */
MOE_API moe_status_t moe_kv_attend_workspace(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t n_q,
                                             int32_t shared_tokens, size_t* bytes);
MOE_API moe_status_t moe_kv_attend(const moe_kv_cache_t* cache, const moe_kv_batch_t* batch, int32_t dtype, int32_t n_q,
                                   const moe_heads_t* q, const moe_heads_t* out, float* lse, float scale,
                                   int32_t shared_tokens, void* workspace, size_t workspace_bytes, void* cuda_stream);

/*
 * Sample one token a row from logits [rows][vocab] (row_stride elements
 * apart) and one uniform number u in [0, 1) a row.
 *   order  by logit descending, ties by index ascending; NaN ranks below
 *          every number and is never sampled
 *   w_i  = exp((logit_i - max) / temperature)
 *   top-k  keeps the first top_k of the order (0 or less, or >= vocab: all)
 *   top-p  then keeps the shortest prefix of the order whose mass reaches
 *          top_p of what top-k kept (>= 1: all; the first is always kept)
 *   min-p  then keeps w_i >= min_p (0 or less: all; the first is always kept)
 *   token  the first kept index, ascending, at which the running sum of w
 *          exceeds u times the kept sum
 * temperature <= 0 is greedy: the first of the order.  A NaN parameter is
 * taken as off (temperature: greedy).  Weights are evaluated to about 2^-31
 * relative and summed as integers (units of 2^-45 of the largest), so results
 * do not depend on the order of execution.  Temperatures are clamped to
 * 1e-30..1e30.  A maximum of +infinity: equal weight for every infinite
 * logit, none for the rest.  A row without a number above -infinity has no
 * token: -1, probability 0.
 * temperature, top_k, top_p, min_p: device arrays of one value a row, or
 * NULL (1, all, all, all).  u outside [0, 1) is clamped; NaN counts as 0.
 * tokens: device int32 [rows]; probs: device fp32 [rows] or NULL, w of the
 * token over the kept sum.
 * dtype: MOE_BF16, MOE_FP16 or MOE_FP32; logits aligned to the element.
 * Errors: INVALID_ARG (NULL, rows < 0, vocab < 1, row_stride < vocab, misaligned, unknown dtype),
 * UNSUPPORTED (vocab over 262144, rows over 2^28), CUDA.  rows = 0 does nothing.
 */
MOE_API moe_status_t moe_sample(const void* logits, int32_t dtype, int32_t rows, int32_t vocab, int64_t row_stride,
                                const float* u, const float* temperature, const int32_t* top_k, const float* top_p,
                                const float* min_p, int32_t* tokens, float* probs, void* cuda_stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_MODEL_GB300_H */
