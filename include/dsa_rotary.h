/*
 * dsa_rotary.h -- C ABI of the rotary positions in the GB300 (sm_103a) library
 * libdsa_cb.so: queries and keys turned by their positions before they go into
 * a cache and its attention (dsa_attention.h, dsa_quant.h). Status codes and
 * the conventions on device pointers and streams are those of dsa_cb.h;
 * element types are dsa_dtype of dsa_dcp_attn.h.
 *
 * The first 2 * pairs elements of every head are `pairs` pairs (a, b). At
 * position p, with f_i radians per token for pair i and t = p * f_i:
 *   a' = factor * (a cos t - b sin t)
 *   b' = factor * (b cos t + a sin t)
 * and with t = -p * f_i where `transpose` is set: the transposed map, which
 * takes the gradient of the outputs to that of the inputs (with factor 1 it
 * is also the inverse). The elements behind the pairs are copied as they are
 * (factor does not touch them).
 *
 * Frequencies come as turns per token in fixed point, 2^64 to a turn:
 *   turns[i] = round(f_i / (2 pi) * 2^64) mod 2^64   (as int64)
 * so that the fraction of a turn, p * turns[i] mod 2^64, is exact at any
 * position (32-bit, negative ones included) but for the rounding of turns[i].
 * Context scaling (slower or mixed frequencies) is a choice of the turns.
 *
 * Arithmetic: cosines, sines, products and sums in fp32, each output rounded
 * once to `dtype` (to nearest even).
 */
#ifndef DSA_ROTARY_H
#define DSA_ROTARY_H

#include <stdint.h>

#include "dsa_cb.h"
#include "dsa_dcp_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * dsa_rotary -- one launch for queries and keys.
 *
 *   q, q_out    [tokens, heads, head_dim] of `dtype` (DSA_DTYPE_F32, _BF16 or
 *               _F16): element (t, h, d) at q + t*q_st + h*q_sh + d, strides
 *               in elements; q_out alike with its own strides.
 *   k, k_out    [tokens, kv_heads, head_dim] likewise; kv_heads 0 for none.
 *   positions   [tokens] device int32.
 *   turns       [pairs] device int64; 2 * pairs <= head_dim.
 *   interleaved 0: pair i is elements i and i + pairs; nonzero: elements 2i
 *               and 2i + 1.
 *
 * An output may be its input (same address and strides), and overlaps nothing
 * else; rows of an output do not overlap. Any strides from 0 on and any
 * address that is a multiple of the element's size will do; addresses and
 * strides that are multiples of 16 bytes are fastest.
 *
 * tokens == 0, head_dim == 0 or heads == kv_heads == 0: DSA_OK, nothing
 * written. DSA_EINVAL for an unknown dtype, negative sizes or strides, pairs
 * beyond head_dim / 2, a factor that is not finite, a NULL required pointer
 * or an address that is no multiple of the element's size. DSA_EUNSUPPORTED
 * for tokens from 2^31, head_dim over 4096, or more than 65535 heads in all.
 */
dsa_status dsa_rotary(const void *q, void *q_out, int32_t heads, int64_t q_st,
                      int64_t q_sh, int64_t qo_st, int64_t qo_sh, const void *k,
                      void *k_out, int32_t kv_heads, int64_t k_st, int64_t k_sh,
                      int64_t ko_st, int64_t ko_sh, int32_t dtype,
                      int64_t tokens, int32_t head_dim,
                      const int32_t *positions, const int64_t *turns,
                      int32_t pairs, int32_t interleaved, float factor,
                      int32_t transpose, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_ROTARY_H */
