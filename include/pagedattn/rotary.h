/*
 * libpagedattn -- rotary positions: the rotation of query and key heads, with
 * the norm of each head before it in the same pass, alone or on the way of new
 * keys and values into the paged cache. Ownership, streams, errors, layouts and
 * tracing are as pagedattn.h describes.
 */
#ifndef PAGEDATTN_ROTARY_H
#define PAGEDATTN_ROTARY_H

#include "../pagedattn.h"

#ifdef __cplusplus
extern "C" {
#endif

#define PA_ROTARY_MAX_PAIRS 64

/*
 * A rotation: the first rot_dim of a head's 128 dims are rotated in
 * rot_dim / 2 pairs, the others pass. Pair i is dims (2 i, 2 i + 1) when
 * interleaved, dims (i, i + rot_dim / 2) otherwise; at position p
 *   (a, b) -> amplitude * (a cos x - b sin x, b cos x + a sin x),  x = p * frequency of pair i.
 * turns[i] is that frequency, a double in radians per token, in turns modulo one
 * turn, in units of 2^-64 and to half a unit: its product with a 32-bit position is
 * the angle modulo one turn to 2^-34 turns. Sine and cosine are taken in fp32, of the
 * angle rounded to 24 bits (2^-26 turns at most). Host memory, filled by one of the two
 * calls below and read during the calls that take it.
 */
typedef struct {
    int32_t rot_dim;
    int32_t interleaved;
    float amplitude;
    int32_t reserved;
    uint64_t turns[PA_ROTARY_MAX_PAIRS];
} pa_rotary_t;

/*
 * Frequencies: theta_i = base^(-2 i / rot_dim) radians per token, changed for
 * contexts longer than the one the model was trained on by
 *   PLAIN   nothing (factor is not read);
 *   LINEAR  theta_i / factor;
 *   NTK     a base of base * factor^(rot_dim / (rot_dim - 2));
 *   YARN    by parts ("YaRN: Efficient Context Window Extension of Large
 *           Language Models", by-parts interpolation): pairs that turn more than
 *           `high` times in original_context tokens keep theta_i, those that
 *           turn less than `low` times get theta_i / factor, and between the
 *           two indices (rounded outwards) the mix is linear in i;
 *   BANDED  as YARN, but the mix is linear in the number of turns between low
 *           and high.
 */
typedef enum {
    PA_ROTARY_PLAIN = 0,
    PA_ROTARY_LINEAR = 1,
    PA_ROTARY_NTK = 2,
    PA_ROTARY_YARN = 3,
    PA_ROTARY_BANDED = 4
} pa_rotary_scaling_t;

/*
 * Fill *rotary. rot_dim is a multiple of 16 from 16 to 128; base > 1; factor >= 1;
 * YARN and BANDED take original_context >= 1 and 0 < low < high (the others do
 * not read the three). amplitude 0 stands for the scaling's own: 1 + 0.1 ln(factor)
 * for YARN, 1 for the others. No CUDA call; PA_ERR_INVALID_ARG for values
 * outside these, PA_ERR_UNSUPPORTED for another rot_dim.
 */
PA_API pa_status_t pa_rotary_init(pa_rotary_t *rotary, int rot_dim, int interleaved, double base,
                                  pa_rotary_scaling_t scaling, double factor,
                                  double original_context, double low, double high,
                                  double amplitude);

/* The same from given frequencies, radians per token [rot_dim / 2] in host
 * memory, finite and of at most 2^20 in size; amplitude finite. */
PA_API pa_status_t pa_rotary_init_frequencies(pa_rotary_t *rotary, int rot_dim, int interleaved,
                                              const double *frequencies, double amplitude);

/*
 * Rotate the heads of queries and keys by their tokens' positions, after the norm
 * of each head's row where a weight is given:
 *   y = x * weight / sqrt(mean(x^2) + eps)  (or x),  out = the rotation of y,
 * computed in fp32 and rounded to bf16 once. Head h of token t of q lies at element
 * t * q_token_stride + h * q_head_stride, the same for k and for the outputs, whose
 * strides are their own; the 128 dims of a head are contiguous.
 *
 * q or k may be absent (num_q_heads or num_kv_heads 0). rotary NULL rotates
 * nothing (positions are not read); q_weight, k_weight [128] bf16 NULL norm
 * nothing. What is neither normed nor rotated is copied bit by bit. positions
 * [num_tokens] int32 may be any value. An output may be its input (the same address
 * and strides); other overlaps give unspecified results.
 *
 * Requirements: head_dim == 128; addresses 16-byte aligned; strides not negative
 * and multiples of 8; of an output's two strides one is 128 or more and the other
 * steps over all rows that the first one leads to (heads inside tokens or tokens
 * inside heads; rows in turn from both are refused, also where none overlap); eps
 * finite, not negative; heads of both together at most 2^20; num_tokens below 2^31.
 */
PA_API pa_status_t pa_rotate(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                             void *q_out, int64_t q_out_token_stride, int64_t q_out_head_stride,
                             int num_q_heads, const void *k, int64_t k_token_stride,
                             int64_t k_head_stride, void *k_out, int64_t k_out_token_stride,
                             int64_t k_out_head_stride, int num_kv_heads, int head_dim,
                             const int32_t *positions, int64_t num_tokens,
                             const pa_rotary_t *rotary, const void *q_weight,
                             const void *k_weight, float eps, void *stream);

/*
 * Append a step's tokens to the paged cache: the keys rotated (and normed) as by
 * pa_rotate, the values as they are, into slot slot_mapping[t] of k_cache and
 * v_cache as by pa_store_kvcache_layout; and, with num_q_heads > 0, the queries
 * rotated (and normed) into q_out, in the same launch. A row with slot -1 (batch
 * padding) stores nothing, and a slot outside the pool is skipped and recorded (code
 * 3); its queries are rotated like the others. Two rows with the same slot: the
 * value left there is unspecified.
 *
 * Slots and positions are separate: a drafted token's position is the length before
 * the draft plus its depth in the tree, its slot the place of its node
 * (pagedattn/decode_tree.h).
 *
 * Requirements: pa_rotate's and pa_store_kvcache_layout's.
 */
PA_API pa_status_t pa_append_kvcache(const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                     void *q_out, int64_t q_out_token_stride,
                                     int64_t q_out_head_stride, int num_q_heads, const void *k,
                                     int64_t k_token_stride, int64_t k_head_stride, const void *v,
                                     int64_t v_token_stride, int64_t v_head_stride,
                                     int num_kv_heads, int head_dim, void *k_cache, void *v_cache,
                                     const int64_t *slot_mapping, int block_size,
                                     int64_t num_blocks, pa_layout_t layout,
                                     const int32_t *positions, int64_t num_tokens,
                                     const pa_rotary_t *rotary, const void *q_weight,
                                     const void *k_weight, float eps, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGEDATTN_ROTARY_H */
