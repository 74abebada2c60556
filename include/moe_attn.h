/* moe_attn.h -- the attention operators a decoder layer runs in front of its
 * routed-expert layer (moe_w4a16.h), for GB300 (sm_103a): rotary positions,
 * appending rotated keys and values to a paged cache, and attention of new
 * tokens over that cache.
 *
 * Rotary positions. Pair i of a head turns by the angle
 *   2 pi frac(p * freq[i] / 2^64)
 * at position p: freq[i] is the pair's speed in units of 2^-64 turns per
 * position, so p * freq[i] wraps as a 64-bit integer and the angle is exact to
 * 2^-32 turns at every 32-bit position, negative ones included.
 *   (a, b) -> magnitude * (a cos - b sin, b cos + a sin)
 * The pairs of the first rot_dim values of a head are (i, i + rot_dim/2) in
 * the half layout, (2i, 2i + 1) in the interleaved one; the rest of the head
 * is copied. `inverse` turns the other way, which is the gradient of the
 * output with respect to the input (the map is linear, and its transpose is
 * magnitude times the opposite rotation).
 *
 * The cache holds, for each page and kv head, page_size rows of head_dim
 * values of K and as many of V; page, token and head strides are the caller's,
 * so pages of [kv_heads, page_size, head_dim] and of [page_size, kv_heads,
 * head_dim] both work. Slot = page id * page_size + offset in the page.
 *
 * Attention. Sequence s has its last n_s tokens in rows [cu_q[s], cu_q[s+1])
 * of q, and kv_len[s] keys, key j in row j % page_size of page
 * page_table[s][j / page_size]. Query i stands at p = kv_len[s] - n_s + i and
 * sees key j < kv_len[s] where
 *   (j <= p and (window == 0 or j > p - window)) or j < prefix[s].
 * Query head h reads kv head h / (q_heads / kv_heads). With
 *   x = scale * q.k;  x = softcap * tanh(x / softcap) if softcap > 0;
 *   x = x - slopes[h] * |p - j| if slopes
 * the output is sum_j softmax(x)_j v_j, and lse = log sum_j exp(x_j). A row
 * that sees no key gives zeros and lse = -inf. Scores, sums and softmax statistics
 * are fp32 (under a cap of 64 or less, to 2^-22 of the cap; under larger ones, to
 * 2^-21 of the score); the softmax's numerators are rounded to the cache's type
 * before they are multiplied with V, in fp16 from units in which weights down to
 * 2^-26 of a row's largest keep all their bits. Keys at and after kv_len, and pages behind them, are
 * never used, whatever they hold; a NaN or an infinity in a V row before
 * kv_len may reach other rows of its sequence that do not see that key (a
 * masked weight is an exact zero, and zero times infinity is NaN).
 *
 * Types: bf16 or fp16, one type for q, k, v, the cache and the outputs; lse
 * and slopes fp32. All pointers are device pointers owned by the caller. A
 * handle owns its workspace, is bound to one device, and serves one stream at
 * a time; its calls run on that device and leave the caller's current device as
 * it is. Calls are asynchronous on `stream` (a cudaStream_t; NULL = legacy
 * default stream), allocate nothing and can be captured into a CUDA graph;
 * lengths, positions, slots and page tables are read on the device, so a graph
 * replays with new ones. They must not change while a call runs: its parts read
 * them at different times.
 *
 * Errors: MOE_ATTN_OK or a negative status (the values and meanings of
 * moe_w4a16_status); invalid arguments are rejected on the host and nothing is
 * launched. Kernels check what they read on the device (cu_q, kv_len, page
 * ids, slots) and bound their waits; a failure sets a bit of the handle's
 * device error word and what it concerns is left out, never accessed.
 */
#ifndef MOE_ATTN_H
#define MOE_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum moe_attn_status {
  MOE_ATTN_OK = 0,
  MOE_ATTN_ERR_INVALID_ARG = -1,       /* null pointer, bad count, layout or type   */
  MOE_ATTN_ERR_UNSUPPORTED_SHAPE = -2, /* sizes outside the supported ranges        */
  MOE_ATTN_ERR_TOO_MANY_TOKENS = -3,   /* more tokens or sequences than the handle's */
  MOE_ATTN_ERR_MISALIGNED = -4,        /* pointer or stride not a 16-byte multiple  */
  MOE_ATTN_ERR_CUDA = -5,              /* a CUDA runtime/driver call failed         */
  MOE_ATTN_ERR_DEVICE = -6,            /* a kernel recorded an error flag           */
  MOE_ATTN_ERR_NO_DEVICE = -7          /* no usable sm_103 device                   */
};

enum moe_attn_dtype { MOE_ATTN_BF16 = 0, MOE_ATTN_FP16 = 1 };
enum moe_attn_layout { MOE_ATTN_ROPE_HALF = 0, MOE_ATTN_ROPE_INTERLEAVED = 1 };

/* device error flag bits (moe_attn_check_device_errors) */
#define MOE_ATTN_DEVERR_TIMEOUT 0x1u /* a bounded wait gave up                      */
#define MOE_ATTN_DEVERR_RANGE 0x2u   /* a length, page id or slot left its range    */

/* rows [tokens, heads, head_dim]; head_dim is contiguous, strides in elements */
typedef struct moe_attn_rows {
  void* data;
  int64_t token_stride;
  int64_t head_stride;
} moe_attn_rows;

typedef struct moe_attn_rotation {
  const int64_t* freq;  /* [rot_dim / 2], units of 2^-64 turns per position (wrapping) */
  int32_t rot_dim;      /* even, 0..head_dim (0: nothing turns)                       */
  int32_t layout;       /* moe_attn_layout                                            */
  float magnitude;      /* factor on the turned values                                */
  int32_t inverse;      /* 0 or 1                                                     */
} moe_attn_rotation;

typedef struct moe_attn_config {
  int32_t q_heads;      /* multiple of kv_heads, at most 64 per kv head               */
  int32_t kv_heads;     /* 1..1024                                                    */
  int32_t head_dim;     /* multiple of 8, 8..128                                      */
  int32_t page_size;    /* 16, 32, 64, 128 or 256                                     */
  int32_t max_tokens;   /* new tokens of one call, 1..2^20                            */
  int32_t max_seqs;     /* sequences of one call, 1..16384                            */
  int32_t dtype;        /* moe_attn_dtype                                             */
  uint32_t flags;       /* must be 0                                                  */
} moe_attn_config;

/* K and V share their strides (in elements); head_dim is contiguous. Base
 * pointers are 16-byte aligned and strides multiples of 8 elements. */
typedef struct moe_attn_cache {
  void* k;
  void* v;
  int64_t num_pages;    /* 1..2^31 - 2                                                */
  int64_t page_stride;
  int64_t token_stride;
  int64_t head_stride;
} moe_attn_cache;

typedef struct moe_attn_batch {
  const int32_t* cu_q;       /* [num_seqs + 1] first q row of each sequence, ascending */
  const int32_t* kv_len;     /* [num_seqs] keys of each sequence, new tokens included  */
  const int32_t* page_table; /* [num_seqs, columns], rows table_stride apart           */
  int64_t table_stride;      /* elements                                               */
  int32_t columns;           /* pages listed per sequence: kv_len <= columns * page_size,
                                which is at most 2^29                                  */
  int32_t num_seqs;
  int32_t num_tokens;        /* rows of q                                              */
  int32_t max_q;             /* no sequence has more new tokens than this              */
} moe_attn_batch;

typedef struct moe_attn_scores {
  float scale;               /* usually 1 / sqrt(head_dim)                             */
  float softcap;             /* 0: none                                                */
  int32_t window;            /* keys a query sees, itself included; 0: all             */
  const float* slopes;       /* [q_heads] or NULL                                      */
  const int32_t* prefix;     /* [num_seqs] or NULL; negative counts as 0               */
} moe_attn_scores;

typedef struct moe_attn_handle moe_attn_handle;

/* Frequencies of rotary positions with base `base` (theta_i = base^(-2i/rot_dim)
 * radians per position), on the host, in fp64. factor > 1 stretches them for
 * contexts longer than original_len:
 *   by_parts == 0: every theta_i / factor (positions interpolated);
 *   by_parts == 1: pairs with fewer than beta_slow turns in original_len are
 *     divided by factor, pairs with more than beta_fast are kept, and between them
 *     the part kept is linear in the number of turns (not in the pair's index, as
 *     some programs have it); the magnitude is 1 + 0.1 log(factor). A model made
 *     with another ramp brings its own frequencies: freq is any table.
 * freq: [rot_dim / 2]; magnitude: one float. */
int moe_attn_rope_frequencies(int32_t rot_dim, double base, double factor, int32_t by_parts,
                              double original_len, double beta_fast, double beta_slow,
                              int64_t* freq, float* magnitude);

/* out = rotary positions of x, [num_tokens, heads, head_dim] each; positions
 * [num_tokens]. head_dim 1..256, heads 0..65536. Any element strides (16-byte multiples are
 * fastest); out == x with equal strides is allowed, other overlaps are not, nor is
 * an output whose rows lie on each other (broadcast). */
int moe_attn_rope(const moe_attn_rows* x, const moe_attn_rows* out, const int32_t* positions,
                  int32_t num_tokens, int32_t heads, int32_t head_dim, int32_t dtype,
                  const moe_attn_rotation* rotation, void* stream);

/* Device bytes of a handle's workspace. */
int moe_attn_workspace_bytes(const moe_attn_config* cfg, size_t* bytes);
/* Validates cfg, binds to `device`, allocates the workspace. Synchronous. */
int moe_attn_create(const moe_attn_config* cfg, int device, moe_attn_handle** out);
/* Frees the workspace and the handle (synchronises the device). NULL is OK. */
int moe_attn_destroy(moe_attn_handle* h);

/* One launch: q_out = rotary(q); for each token, rotary(k) and v go to its slot
 * of the cache. positions [num_tokens]; slots int64 [num_tokens], a negative
 * slot leaves the cache alone (padding), one past the cache sets
 * MOE_ATTN_DEVERR_RANGE. q and q_out may both be NULL (keys and values only);
 * q_out == q is allowed. Two tokens with one slot leave a row with parts of both. */
int moe_attn_append(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* q_out,
                    const moe_attn_rows* k, const moe_attn_rows* v, const int32_t* positions,
                    const int64_t* slots, int32_t num_tokens, const moe_attn_rotation* rotation,
                    const moe_attn_cache* cache, void* stream);

/* Attention of the batch's new tokens, whose keys are in the cache already.
 * q: [num_tokens, q_heads, head_dim] (16-byte aligned, strides multiples of 8
 * elements); out: the same form, not overlapping q; lse: fp32 [num_tokens,
 * q_heads] contiguous, or NULL. Rows of no sequence are not written. */
int moe_attn_forward(moe_attn_handle* h, const moe_attn_rows* q, const moe_attn_rows* out,
                     float* lse, const moe_attn_cache* cache, const moe_attn_batch* batch,
                     const moe_attn_scores* scores, void* stream);

/* Synchronises the device, returns the error flag bits in *flags and clears
 * them; MOE_ATTN_ERR_DEVICE when any was set. Once a wait has given up, the
 * results of all launches until this call are worthless; after it the handle is
 * as good as new. */
int moe_attn_check_device_errors(moe_attn_handle* h, uint32_t* flags);

#ifdef __cplusplus
}
#endif

#endif /* MOE_ATTN_H */
