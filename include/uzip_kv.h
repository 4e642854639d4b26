/*
 * uzip_kv.h -- C ABI of libuzip's operators on a KV cache: rotary positions,
 * attention for a tree of drafted tokens, the attention weight each cached
 * token collects, and eviction by that weight into a packed buffer that the
 * codec of uzip.h then encodes: a BF16 cache by uzip_encode, an E5M2 one by
 * uzip_e5m2_encode. FP16 has no format of its own there: uzip_encode takes its
 * bits and gives them back, but its codebook is for BF16's exponent field.
 *
 * Conventions are those of uzip.h: d_* is device memory of the caller, the
 * library allocates nothing and keeps nothing between calls, work is enqueued
 * on `stream`, a stream of the current device, and is asynchronous, errors found
 * on the host return at once (enum uzip_status) and enqueue nothing.
 *
 * One layer's cache is two pools of pages, K and V, of shape
 * [pages][kv_heads][page_tokens][head_dim], a page table of page numbers
 * [sequences][pages_per_sequence] and the length of each sequence. Token j of
 * sequence b is row j % page_tokens of page table[b][j / page_tokens]; the
 * table is read for tokens in use only. Pages of the whole sequence
 * (page_tokens = its capacity) describe a contiguous cache. The new tokens of
 * a call take the slots lengths[b] .. lengths[b] + counts[b] - 1 of their
 * sequence; the caller advances lengths when it accepts them.
 *
 * Rules that only the device can check: 0 <= lengths[b], 0 <= counts[b] <=
 * new_tokens, lengths[b] + counts[b] <= page_tokens * pages_per_sequence, and
 * page numbers of tokens in use below `pages`. A cache that breaks one is read
 * and written as far as it is in bounds (lengths and counts are clamped, a
 * page that does not exist reads as zeros and is not written), its outputs are
 * not trustworthy, and *d_status, if given, is set to UZIP_ERR_CORRUPT. Attention
 * and mass wait on barriers in shared memory, each wait bounded; if one ran out,
 * which no input brings about, it is set to UZIP_ERR_TIMEOUT. (The other kernels
 * meet at the hardware's own barriers only.) No call sets it to anything else, or
 * clears it.
 */
#ifndef UZIP_KV_H
#define UZIP_KV_H

#include "uzip.h"

#ifdef __cplusplus
extern "C" {
#endif

enum uzkv_dtype { UZKV_BF16 = 0, UZKV_FP16 = 1, UZKV_FP32 = 2, UZKV_E5M2 = 3 };
enum uzkv_layout {
    UZKV_HALF = 0,       /* pair i is elements i and i + rotary_dim / 2 */
    UZKV_INTERLEAVED = 1 /* pair i is elements 2 i and 2 i + 1          */
};

#define UZKV_MAX_HEAD_DIM 256
#define UZKV_MAX_NEW_TOKENS 256 /* of uzkv_tree_attention and uzkv_attention_mass */

typedef struct {
    void *d_k, *d_v; /* 16-byte aligned */
    /* Strides in elements, each a multiple of 16 bytes (any along a dimension of one); elements of a row are contiguous. */
    int64_t k_page_stride, k_head_stride, k_token_stride;
    int64_t v_page_stride, v_head_stride, v_token_stride;
    const int32_t *d_table; /* [sequences] rows of pages_per_sequence, table_stride apart */
    int64_t table_stride;
    const int32_t *d_lengths; /* [sequences] */
    uint32_t *d_status;       /* NULL or one device word */
    uint32_t pages, kv_heads, page_tokens, head_dim;
    uint32_t sequences, pages_per_sequence;
    uint32_t dtype; /* UZKV_BF16, UZKV_FP16 or UZKV_E5M2 */
    uint32_t reserved;
} uzkv_cache_t;

/* A tensor [sequences][tokens][heads][head_dim] with contiguous rows. */
typedef struct {
    void *d;
    int64_t stride_b, stride_t, stride_h; /* in elements */
} uzkv_rows_t;

/* Rotary positions. Pair i of each head turns by positions * turns[i]:
 *   y_a = m (x_a cos - x_b sin),  y_b = m (x_b cos + x_a sin),
 * with m = magnitude; elements rotary_dim .. head_dim - 1 are copied. backward
 * != 0 turns the other way, which is the gradient: dx = m R^T dy. d_turns holds
 * rotary_dim / 2 rates in turns a position, as 64-bit fixed point (2^64 is one
 * turn), so that a phase is one wrapping product and exact at any position.
 *   x, y           dtype BF16, FP16 or FP32; y may be x.
 *   d_positions    [sequences][tokens] int32, rows position_stride apart.
 *   head_dim       1 .. UZKV_MAX_HEAD_DIM; rotary_dim even, 0 < rotary_dim <= head_dim.
 * Returns UZIP_ERR_ARG / UZIP_ERR_CUDA, else UZIP_OK. Async. */
UZIP_API int uzkv_rotary(const uzkv_rows_t *x, const uzkv_rows_t *y, uint32_t dtype, uint32_t sequences,
                         uint32_t tokens, uint32_t heads, uint32_t head_dim, const int32_t *d_positions,
                         int64_t position_stride, const uint64_t *d_turns, uint32_t rotary_dim, uint32_t layout,
                         float magnitude, int backward, uzip_stream_t stream);

/* Rotate the queries and keys of new tokens and store the keys and values in
 * the cache, rounded once to its type, in one launch.
 *   q, q_out       [sequences][tokens][q_heads][head_dim], dtype BF16 or FP16; q_out may be q.
 *   k, v           [sequences][tokens][kv_heads][head_dim] of the same type.
 *   cache          of that type or E5M2; k and v go to the slots of the new tokens.
 *   d_counts       NULL (all tokens) or [sequences]; q_out of later tokens is zero,
 *                  their k and v are not stored.
 * Other arguments as uzkv_rotary. Async. */
UZIP_API int uzkv_rotary_append(const uzkv_rows_t *q, const uzkv_rows_t *k, const uzkv_rows_t *v,
                                const uzkv_rows_t *q_out, uint32_t dtype, uint32_t tokens, uint32_t q_heads,
                                const int32_t *d_positions, int64_t position_stride, const uint64_t *d_turns,
                                uint32_t rotary_dim, uint32_t layout, float magnitude, const int32_t *d_counts,
                                const uzkv_cache_t *cache, uzip_stream_t stream);

/* Attention of new tokens, a tree of drafted ones or a single one, over the
 * cache that already holds their keys and values. Token t of sequence b sees
 * the slots below lengths[b] and, of the new tokens, those whose bit is set in
 * its mask row (bit u % 64 of word u / 64); without a mask, the tokens up to
 * itself. Query head h reads KV head h / (q_heads / kv_heads).
 *   s_j = scale q . k_j,  lse = ln sum exp s_j,  out = sum exp(s_j - lse) v_j;
 * a row that sees nothing (and each token at or past counts[b]) gives out = 0
 * and lse = -inf. What a row does not see, NaN and infinities among it, has no
 * part in its output.
 *   q, out         [sequences][tokens][q_heads][head_dim], dtype BF16 or FP16;
 *                  16-byte aligned rows; out may be q.
 *   d_lse          NULL or [sequences][tokens][q_heads] floats, contiguous.
 *   tokens         1 .. UZKV_MAX_NEW_TOKENS; sequences * tokens * q_heads below 2^31.
 *   d_mask         NULL or [sequences][tokens][ceil(tokens / 64)] words, a
 *                  sequence's rows mask_stride_b words apart (0: one tree for all).
 *   cache          dtype of q or E5M2; head_dim a multiple of 16 bytes' worth of
 *                  elements, up to UZKV_MAX_HEAD_DIM.
 *   d_workspace    uzkv_tree_attention_workspace_bytes bytes, 16-byte aligned, any
 *                  contents; not shared with a call that may overlap.
 * The result does not depend on the launch's timing. Async. */
UZIP_API size_t uzkv_tree_attention_workspace_bytes(uint32_t sequences, uint32_t tokens, uint32_t q_heads,
                                                    uint32_t kv_heads, uint32_t head_dim);
UZIP_API int uzkv_tree_attention(const uzkv_rows_t *q, const uzkv_rows_t *out, float *d_lse, uint32_t dtype,
                                 uint32_t tokens, uint32_t q_heads, const int64_t *d_mask, int64_t mask_stride_b,
                                 const int32_t *d_counts, float scale, const uzkv_cache_t *cache,
                                 void *d_workspace, size_t workspace_bytes, uzip_stream_t stream);

/* The attention weight that each cached token collects from the new tokens,
 * given their log-sum-exp from uzkv_tree_attention on the same arguments:
 *   mass_out[b][g][j] = decay * mass_in[b][g][j]   (j < lengths[b]; 0 without mass_in)
 *                     + sum over the group's heads and the tokens t that see j of
 *                       weights[b][t] * exp(scale q . k_j - lse),
 * 0 for slots that are not in use.
 *   d_lse          [sequences][tokens][q_heads], contiguous; -inf rows add nothing.
 *   d_weights      NULL (ones) or [sequences][tokens] floats, contiguous, >= 0.
 *   d_mass_in      NULL or [sequences][kv_heads][>= slots] floats with the strides of
 *                  mass_out; may be mass_out.
 *   slots          width of mass_out, at most page_tokens * pages_per_sequence; slots
 *                  past it are not weighed.
 * Other arguments as uzkv_tree_attention. Each sum has one order, whatever the
 * launch's timing. Async. */
UZIP_API int uzkv_attention_mass(const uzkv_rows_t *q, const float *d_lse, uint32_t dtype, uint32_t tokens,
                                 uint32_t q_heads, const int64_t *d_mask, int64_t mask_stride_b,
                                 const int32_t *d_counts, const float *d_weights, float scale,
                                 const uzkv_cache_t *cache, const float *d_mass_in, float decay, float *d_mass_out,
                                 int64_t mass_stride_b, int64_t mass_stride_h, uint32_t slots, uzip_stream_t stream);

/* Keep `keep` tokens of each sequence and KV head and pack them. Kept are the
 * first `sink` slots, the last `recent` ones and those of the largest mass
 * (equal masses: the lowest slot first; NaN below every number); a sequence of
 * at most `keep` tokens keeps all. Kept tokens stay in slot order.
 *   d_mass         [sequences][kv_heads][slots] floats; lengths above slots are clamped as
 *                  corrupt.
 *   out_k, out_v   [sequences][kv_heads][keep][head_dim] of the cache's type; rows past
 *                  a sequence's kept tokens are zero. stride_t is the head's stride and
 *                  stride_h the token's. Not part of the cache's pools.
 *   d_kept         [sequences][kv_heads][keep] int32 slots, contiguous, -1 past the kept.
 *   d_mass_out     [sequences][kv_heads][keep] floats, contiguous, 0 past the kept.
 *   d_lengths_out  [sequences] int32: min(lengths[b], keep).
 *   keep           at least max(1, sink + recent), below 2^27.
 * sequences * kv_heads is at most 65,535. Async. */
UZIP_API int uzkv_evict(const uzkv_cache_t *cache, const float *d_mass, int64_t mass_stride_b, int64_t mass_stride_h,
                        uint32_t slots, uint32_t keep, uint32_t sink, uint32_t recent, const uzkv_rows_t *out_k,
                        const uzkv_rows_t *out_v, int32_t *d_kept, float *d_mass_out, int32_t *d_lengths_out,
                        uzip_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* UZIP_KV_H */
