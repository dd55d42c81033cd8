/*
 * moe_attention.h — C ABI of the attention half of a decoder layer (one GB300
 * GPU, sm_103a): a paged key/value cache held in 4 bits, attention over it, and
 * causal attention over whole prompts.
 *
 * The conventions are those of moe_cache.h: a return code per call (MOE_OK or
 * MOE_ERR_*), device pointers owned by the caller, work stream-ordered on the
 * caller's stream, no allocation and no host synchronisation.  These entry
 * points have no handle: they may be called from several threads and streams at
 * once, as long as no two calls in flight share a workspace or write the same
 * tokens.  Every call may be captured into a CUDA graph.
 *
 * Cache layout.  A page holds page_size tokens (a multiple of 32) of every
 * key/value head: [n_kv_heads][page_size / 32 tiles][tile], a tile of head width
 * D being 36 D bytes,
 *   key codes    [D/32 blocks][32 tokens][16 bytes]
 *   key scales   [32 tokens][D/32 blocks] fp16
 *   value codes, value scales likewise,
 * every block the Q4_0 block of moe_cache.h with its scale kept apart: low
 * nibbles of the 16 bytes are values 0..15, high nibbles values 16..31,
 * w = (q - 8) * d.  A tile is contiguous, so one bulk copy brings 32 tokens of a
 * head into shared memory.
 * Quantising a block x[0..31] (fp32): m = the value of largest magnitude (+ when
 * both signs tie), d = m / -8, q = min(15, trunc(x / d + 8.5)), 8 where d == 0;
 * the stored scale is d rounded to fp16, limited to +-65504.  A block with a
 * value that is not finite stores scale NaN and codes 0, so that whatever reads
 * it shows it.
 *
 * Sequences.  page_table[s][i] is the page of tokens [i page_size, (i + 1)
 * page_size) of sequence s.  Entries past a sequence's tokens are not read.  A call
 * of no sequences and no tokens does nothing.
 *
 * Bad contents of device arrays (page numbers, lengths, positions) cannot be
 * refused by the host.  The kernels check them before every access, touch
 * nothing out of range, give the rows concerned NaN (an append writes nothing into
 * the cache for such a token; its rotated rows, which do not depend on the page,
 * are NaN where its length or position is bad), and set bits in *status when status
 * is not NULL:
 */
#ifndef MOE_ATTENTION_H
#define MOE_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include "moe_cache.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_KV_BAD_PAGE 1      /* a page number outside [0, n_pages) was met             */
#define MOE_KV_BAD_LENGTH 2    /* a length or offset is negative, decreasing or past the
                                  page table or the tensor                               */
#define MOE_KV_BAD_POSITION 4  /* a position past the rotation table                     */
#define MOE_KV_TIMED_OUT 8     /* a bounded device wait gave up                          */

#define MOE_KV_COUNTER_BYTES 4096

#define MOE_F32 0
#define MOE_BF16 1
#define MOE_F16 2

typedef struct {
  void *pages;               /* device, 16-byte aligned                                  */
  int64_t page_stride;       /* bytes from page to page, a multiple of 16, at least
                                moe_kv_page_bytes                                        */
  const int32_t *page_table; /* device [n_seqs][table_stride]                            */
  int64_t table_stride;      /* entries from row to row, >= table_width                  */
  int32_t *status;           /* device word the bits above are set in, or NULL           */
  int32_t n_pages, page_size, n_kv_heads, head_dim; /* head_dim 64, 128 or 256           */
  int32_t n_seqs, table_width;
} moe_kv_cache;

/* A token-major tensor [tokens][heads][head_dim], the last dimension contiguous.
 * Base and strides (elements) are multiples of 16 bytes. */
typedef struct {
  const void *data;
  int64_t token_stride, head_stride;
} moe_tensor;

/* Bytes of one page, or 0 for sizes that are not supported. */
int64_t moe_kv_page_bytes(int32_t n_kv_heads, int32_t head_dim, int32_t page_size);

/*
 * Append the keys and values of n_tokens new tokens, rotating keys (and queries)
 * by their positions on the way.
 * Tokens [cu_tokens[s], cu_tokens[s+1]) belong to sequence s (device int32
 * [n_seqs + 1], cu_tokens[0] = 0, cu_tokens[n_seqs] = n_tokens) and take the
 * positions starts[s], starts[s] + 1, ... (device int32 [n_seqs]: tokens cached
 * before).
 * Rotation of the first rot_dim values of a head by position p, in fp32 without
 * contraction: (a, b) -> (a cos[p][i] - b sin[p][i], b cos[p][i] + a sin[p][i]),
 * the pair i being (i, i + rot_dim/2), or (2i, 2i + 1) when interleaved.
 * cos, sin: device fp32 [n_positions][rot_dim/2] contiguous, 16-byte aligned.
 * rot_dim: a multiple of 16, at most head_dim; 0 = no rotation (cos, sin unused).
 * q (NULL data: none): n_q_heads heads, rotated into q_out [tokens][n_q_heads]
 * [head_dim] contiguous.  k_out, where not NULL, receives the rotated keys in
 * dtype, contiguous.  q_out == q.data and k_out == k.data are allowed where the
 * input is contiguous; no other overlap.
 * The cache receives the keys quantised from their rotated fp32 values.
 * dtype: MOE_F32, MOE_BF16 or MOE_F16, of q, k, v and the outputs.
 */
int moe_kv_append(const moe_kv_cache *c, const int32_t *starts, const int32_t *cu_tokens, int32_t n_tokens,
                  const moe_tensor *q, int32_t n_q_heads, const moe_tensor *k, const moe_tensor *v,
                  const float *cos, const float *sin, int32_t rot_dim, int32_t n_positions, int32_t interleaved,
                  void *q_out, void *k_out, int32_t dtype, void *cuda_stream);

/*
 * The values that cached tokens stand for: k_out, v_out [n_tokens][n_kv_heads]
 * [head_dim] contiguous in dtype, for tokens starts[s] + (i - cu_tokens[s]).
 * Either output may be NULL.
 */
int moe_kv_read(const moe_kv_cache *c, const int32_t *starts, const int32_t *cu_tokens, int32_t n_tokens,
                void *k_out, void *v_out, int32_t dtype, void *cuda_stream);

/*
 * Attention of the last q_tokens tokens of every sequence over the cache.
 * seq_lens: device int32 [n_seqs], cached tokens of each sequence, the queried
 * ones among them.  q: [n_seqs * q_tokens] tokens of n_q_heads heads (a multiple
 * of n_kv_heads; query head h reads key/value head h / (n_q_heads / n_kv_heads)).
 * Token j of a sequence of n tokens stands at position p = n - q_tokens + j and
 * sees the positions [max(0, p - window + 1), p], or [0, p] when window == 0; a
 * row that sees nothing gives 0 (and lse -inf).  scale: positive, at most 2.3e38.
 * out: [n_seqs * q_tokens][n_q_heads][head_dim] contiguous, in dtype (MOE_BF16
 * or MOE_F16, q's too).  lse: fp32 [n_seqs * q_tokens][n_q_heads], the natural
 * logarithm of the sum of exponentials, or NULL.
 * workspace: device memory of moe_kv_attention_workspace bytes, 256-byte
 * aligned, its first MOE_KV_COUNTER_BYTES zero before its first use; every call
 * leaves it ready for the next one on the same stream.
 * A NaN or infinity that a row does not see does not reach it.
 */
int64_t moe_kv_attention_workspace(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t q_tokens);
int moe_kv_attention(const moe_kv_cache *c, const int32_t *seq_lens, const moe_tensor *q, int32_t n_q_heads,
                     int32_t q_tokens, float scale, int32_t window, void *out, float *lse, int32_t dtype,
                     void *workspace, int64_t workspace_bytes, void *cuda_stream);

/*
 * Causal attention over whole prompts, packed one after another.
 * Queries [cu_q[s], cu_q[s+1]) and keys [cu_k[s], cu_k[s+1]) are sequence s's
 * (device int32 [n_seqs + 1], not decreasing, from 0 to the tensors' tokens).  A
 * sequence's queries stand at its last positions (keys before them: tokens that
 * an earlier call has seen): query i of n_q, with n_k keys, stands at p = n_k -
 * n_q + i and sees the keys [max(0, p - window + 1), p], or [0, p] when window
 * == 0; a row that sees nothing gives 0 (and lse -inf).  scale: positive, at most 2.3e38.
 * q [n_q_tokens][n_q_heads][head_dim]; k, v [n_k_tokens][n_kv_heads][head_dim];
 * n_q_heads a multiple of n_kv_heads, at most 64 times it.  out: contiguous, q's
 * shape; lse: fp32 [n_q_tokens][n_q_heads], the natural logarithm of the sum of
 * exponentials, or NULL.  dtype: MOE_BF16 or MOE_F16, of q, k, v and out; weights
 * are rounded to it before they meet the values, sums are fp32.  Strides are not 0.
 * A NaN or infinity that a row does not see does not reach it.
 * status: as above, or NULL.  Rows that no sequence holds give NaN, and so do those of
 * a sequence whose cu_k makes no sense; a sequence whose cu_q makes none (out of range,
 * decreasing, or within an earlier sequence) holds no rows.  Nothing is written when
 * n_q_tokens or n_seqs is 0.
 */
int moe_prompt_attention(const moe_tensor *q, int32_t n_q_tokens, int32_t n_q_heads, const moe_tensor *k,
                         const moe_tensor *v, int32_t n_k_tokens, int32_t n_kv_heads, int32_t head_dim,
                         const int32_t *cu_q, const int32_t *cu_k, int32_t n_seqs, float scale, int32_t window,
                         void *out, float *lse, int32_t dtype, int32_t *status, void *cuda_stream);

/*
 * The same with a workspace, for calls whose rows are few and whose keys are many
 * (a chunk of a long prompt): what would leave part of the GPU idle then shares its
 * keys out over more of it.  moe_prompt_attention_workspace gives the bytes for a
 * call's sizes, on the current device, 0 where a workspace would not be used.
 * workspace: device memory of at least as many bytes, 256-byte aligned, its first
 * MOE_KV_COUNTER_BYTES zero before its first use; every call leaves it ready for
 * the next one on the same stream.  NULL: as moe_prompt_attention.
 */
int64_t moe_prompt_attention_workspace(int32_t n_q_tokens, int32_t n_q_heads, int32_t n_k_tokens, int32_t n_kv_heads,
                                       int32_t head_dim, int32_t n_seqs, int32_t window);
int moe_prompt_attention_shared(const moe_tensor *q, int32_t n_q_tokens, int32_t n_q_heads, const moe_tensor *k,
                                const moe_tensor *v, int32_t n_k_tokens, int32_t n_kv_heads, int32_t head_dim,
                                const int32_t *cu_q, const int32_t *cu_k, int32_t n_seqs, float scale, int32_t window,
                                void *out, float *lse, int32_t dtype, int32_t *status, void *workspace,
                                int64_t workspace_bytes, void *cuda_stream);

#ifdef __cplusplus
}
#endif
#endif /* MOE_ATTENTION_H */
