/* moe_attn8.h -- more attention operators of a decoder layer (next to
 * moe_attn.h, whose types, handle, statuses and errors they share): norms of
 * queries and keys for each head with the rotary positions in the same pass and
 * their gradient, a paged cache of 8-bit keys and values that is quantised as it
 * is written and read back, attention over that cache, and attention with a
 * sliding window and a few first tokens that stay visible.
 *
 * Norm. Of each head of each token, with R_p the rotary positions of moe_attn.h,
 *   n = x / sqrt(mean(x^2) + eps),  y = R_p(n * (weight + offset)).
 * The weight is one per value of a head, for all heads (head stride 0) or for
 * each; offset is 1 in models that store it as its distance from one. fp32
 * throughout, one rounding at the end. Its gradient, with u = R_p^T dy (the
 * opposite rotation) and h = u * (weight + offset):
 *   dx = (h - n mean(h n)) / sqrt(mean(x^2) + eps),  dweight = sum of u n
 * over the tokens, and the heads that share the weight.
 *
 * 8-bit cache. K and V are e4m3 codes [pages, kv_heads, page_size, head_dim] in
 * the strides of moe_attn.h's cache (bytes, multiples of 16; head_dim a multiple
 * of 16), and each 16 tokens of a page and head (a block) have a scale for K and
 * one for V, fp32 [pages, kv_heads, page_size / 16]: a value is code * scale.
 * moe_attn_append8 writes scales that are powers of two in 2^-64 .. 2^64: a new
 * value x raises its block's to the least one with |x| <= 448 scale, and is held as
 * x / scale rounded to the nearest code (ties to even, saturating at 448; NaN stays
 * NaN and infinities, which do not count for the scale, saturate). Codes that the
 * block holds already go by the new scale, rounded again: exactly, but for codes that
 * become subnormal. The token in a block's first row begins the block, whose old
 * scale and codes do not count any more. (A fraction in the scale would buy a
 * floating-point code nothing but range that it has.) Caches that others filled may
 * have any scales in 2^-64 .. 2^64; appending to their blocks raises them the same way.
 *
 * Attention over it is that of moe_attn.h with k = code * scale and v = code *
 * scale: scores and sums in fp32, codes times queries exact (bf16 queries are
 * brought to fp16 by a power of two for each row, which loses what is below 2^-39 of
 * the row's largest value), and the softmax's numerators, times the scales of V,
 * rounded to fp16 with all bits down to 2^-26 of the largest. (A weight may be lost to
 * the softmax's sum where it is below 2^(d - 126) of that of a key whose scale of V is
 * 2^d times its own: nothing that counts while a row's scales are within 2^80.) Where a
 * call has scratch and brings the keys to 16 bits, it is moe_attn_forward over those,
 * whose numerators are rounded to the handle's type: in bf16 the same batch then has other
 * last bits than without. What lies behind kv_len is never used; a NaN in a code or scale
 * before it may reach other rows of its sequence.
 *
 * Sinks. With a window and sinks > 0, query i at p also sees key j where j <= p and
 * j < sinks. Without a window they change nothing.
 */
#ifndef MOE_ATTN8_H
#define MOE_ATTN8_H

#include "moe_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define MOE_ATTN8_BLOCK 16  /* tokens of a block */

enum moe_attn_weight_type { MOE_ATTN_WEIGHT_SAME = 0, MOE_ATTN_WEIGHT_F32 = 1 };

typedef struct moe_attn_norm {
  const void* q_weight;   /* [head_dim] or [q_heads, head_dim]                        */
  const void* k_weight;
  int64_t q_head_stride;  /* elements from one head's weights to the next, 0: one for all */
  int64_t k_head_stride;
  float eps;              /* not negative                                             */
  float offset;           /* added to the weights                                     */
  int32_t weight_type;    /* moe_attn_weight_type: the type of x, or fp32             */
} moe_attn_norm;

/* Codes and scales share their strides between K and V (codes: bytes, scales:
 * elements, not negative; 0, one scale for all, where the cache is only read). Code
 * pointers are 16-byte aligned. */
typedef struct moe_attn_cache8 {
  void* k;
  void* v;
  float* k_scales;
  float* v_scales;
  int64_t num_pages;      /* 1..2^31 - 2                                              */
  int64_t page_stride;
  int64_t token_stride;
  int64_t head_stride;
  int64_t scale_page_stride;
  int64_t scale_head_stride;
  int64_t scale_block_stride;
} moe_attn_cache8;

/* Rows of the cache to be read back: those of sequence s are [cu_rows[s],
 * cu_rows[s+1]), its tokens from first[s] on. */
typedef struct moe_attn_extent {
  const int32_t* cu_rows;    /* [num_seqs + 1], ascending                              */
  const int32_t* first;      /* [num_seqs]                                             */
  const int32_t* page_table; /* [num_seqs, columns], rows table_stride apart           */
  int64_t table_stride;
  int32_t columns;           /* first[s] + rows of s <= columns * page_size <= 2^29    */
  int32_t num_seqs;
  int32_t num_rows;          /* of the outputs, up to 2^30                             */
} moe_attn_extent;

/* q_out = norm and rotary positions of q [num_tokens, q_heads, head_dim], k_out of k
 * [num_tokens, kv_heads, head_dim], in one launch; q and q_out, or k and k_out, may
 * both be NULL. num_tokens up to 2^30, head_dim 1..256, heads 0..65536, any element
 * strides (16-byte multiples, and rotations of a multiple of 16 values, are fastest); an
 * output may be its input, other overlaps are refused, as are outputs whose rows lie on
 * each other. */
int moe_attn_norm_rope(const moe_attn_rows* q, const moe_attn_rows* q_out, const moe_attn_rows* k,
                       const moe_attn_rows* k_out, const int32_t* positions, int32_t num_tokens,
                       int32_t q_heads, int32_t kv_heads, int32_t head_dim, int32_t dtype,
                       const moe_attn_norm* norm, const moe_attn_rotation* rotation, void* stream);

/* Device bytes that moe_attn_norm_rope_backward works on. */
int moe_attn_norm_rope_backward_bytes(int32_t num_tokens, int32_t q_heads, int32_t kv_heads,
                                      int32_t head_dim, size_t* bytes);

/* The gradient of moe_attn_norm_rope: dq and dk are the gradients of its results,
 * q and k its inputs; dx_q and dx_k get the gradients of q and k, dw_q and dw_k
 * (fp32, contiguous, of the weights' shape: [head_dim] where the head stride is 0)
 * those of the weights, which are overwritten (zeros without tokens, or heads). The q or
 * the k arguments may all be NULL. dx may be dq or q in place. workspace: as many bytes
 * as above, 16-byte aligned; it keeps nothing between calls. Sums are in an order that
 * depends on the sizes alone: repeats are equal bit by bit. */
int moe_attn_norm_rope_backward(const moe_attn_rows* dq, const moe_attn_rows* q,
                                const moe_attn_rows* dx_q, float* dw_q, const moe_attn_rows* dk,
                                const moe_attn_rows* k, const moe_attn_rows* dx_k, float* dw_k,
                                const int32_t* positions, int32_t num_tokens, int32_t q_heads,
                                int32_t kv_heads, int32_t head_dim, int32_t dtype,
                                const moe_attn_norm* norm, const moe_attn_rotation* rotation,
                                void* workspace, size_t workspace_bytes, void* stream);

/* moe_attn_append with norms of q and k before their rotation. */
int moe_attn_append_norm(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* q_out,
                         const moe_attn_rows* k, const moe_attn_rows* v, const int32_t* positions,
                         const int64_t* slots, int32_t num_tokens, const moe_attn_norm* norm,
                         const moe_attn_rotation* rotation, const moe_attn_cache* cache,
                         void* stream);

/* The same into an 8-bit cache, whose scales and codes do not lie on each other (each
 * stride reaches past what lies within it); norm NULL: none. New tokens of one block
 * follow each other in the call, in the order of their slots; a block that the call comes
 * to twice (or a slot given twice) is left with parts of both. Slots that are negative or
 * past the cache as in moe_attn_append. */
int moe_attn_append8(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* q_out,
                     const moe_attn_rows* k, const moe_attn_rows* v, const int32_t* positions,
                     const int64_t* slots, int32_t num_tokens, const moe_attn_norm* norm,
                     const moe_attn_rotation* rotation, const moe_attn_cache8* cache,
                     void* stream);

/* k_out and v_out [num_rows, kv_heads, head_dim] of the handle's type = the cache's
 * values, code * scale rounded once; fp16 takes what is above 65504 as that. Rows of no
 * sequence, and rows whose position or page leaves its range (MOE_ATTN_DEVERR_RANGE), are
 * not written. */
int moe_attn_read8(moe_attn_handle* h, const moe_attn_cache8* cache, const moe_attn_extent* extent,
                   const moe_attn_rows* k_out, const moe_attn_rows* v_out, void* stream);

/* Device bytes that moe_attn_forward8 works faster with: room for the batch's keys and
 * values in 16 bits, as far as its page table goes, where its sequences have many new
 * tokens (more than 512 query rows to a kv head on average; else, and where that were
 * more than 8 GiB, 0). */
int moe_attn_forward8_scratch_bytes(const moe_attn_handle* h, const moe_attn_batch* batch,
                                    size_t* bytes);

/* moe_attn_forward over an 8-bit cache; sinks: see above (0: none). scratch: as many
 * bytes as above, 256-byte aligned, or NULL; it keeps nothing between calls. With it, the
 * keys and values that queries see are brought to the handle's type first, as
 * moe_attn_read8 gives them: exactly, where scales are powers of two and values in the
 * type's range. (Keys above 65504, which norms in an fp16 layer can make, count in full
 * only without it.) */
int moe_attn_forward8(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* out,
                      float* lse, const moe_attn_cache8* cache, const moe_attn_batch* batch,
                      const moe_attn_scores* scores, int32_t sinks, void* scratch,
                      size_t scratch_bytes, void* stream);

/* moe_attn_forward with sinks. */
int moe_attn_forward_sinks(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* out,
                           float* lse, const moe_attn_cache* cache, const moe_attn_batch* batch,
                           const moe_attn_scores* scores, int32_t sinks, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTN8_H */
