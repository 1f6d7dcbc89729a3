/*
 * dsa_quant.h -- C ABI of the 8-bit cache in the GB300 (sm_103a) library
 * libdsa_cb.so: keys and values written into pages as e4m3 codes with a scale
 * for each block of tokens and head, read back as packed rows, and attended to
 * by single tokens. Status codes and the conventions on device pointers and
 * streams are those of dsa_cb.h; element types are dsa_dtype of
 * dsa_dcp_attn.h. dsa_cache.h forks, frees and compacts these pages too.
 *
 * A pool of pages (one for keys, one for values, of one layer):
 *   codes   [num_pages, page_size, kv_heads, head_dim] bytes, e4m3 (sign, four
 *           exponent bits of bias 7, three mantissa bits; 0x7f and 0xff are
 *           NaN, there are no infinities): token t of page n, head h at codes
 *           + n*sn + t*st + h*sh, strides in bytes.
 *   scales  [num_pages, page_size / block, kv_heads] fp32, each page's
 *           contiguous: page n's at scales + n*ssn (in elements).
 *   The value of a code is code * scale of its page, token / block and head.
 * page_size is a power of two, at least 16; block a power of two that divides
 * it. head_dim is a multiple of 16 up to 128; codes are 16-byte aligned, with
 * strides that are multiples of 16; kv_heads is at most 2^20.
 *
 *   tables  [seqs, max_pages] device int32 at tables + s*ld_tables + i: token
 *           t of sequence s lies on page tables[s][t / page_size]. Entries
 *           outside [0, num_pages) (such as -1) stand for no page.
 */
#ifndef DSA_QUANT_H
#define DSA_QUANT_H

#include <stddef.h>
#include <stdint.h>

#include "dsa_cb.h"
#include "dsa_dcp_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The pages of one layer's keys and values, and the sequences on them, as above. */
typedef struct {
    void *k_codes, *v_codes;
    float *k_scales, *v_scales;
    int64_t num_pages;
    int64_t kc_sn, kc_st, kc_sh; /* bytes */
    int64_t vc_sn, vc_st, vc_sh;
    int64_t ks_sn, vs_sn; /* floats */
    const int32_t *tables;
    int64_t max_pages, ld_tables;
    int32_t page_size, block, kv_heads, head_dim;
} dsa_quant_pages;

/*
 * dsa_quant_cache_write -- appends tokens to sequences.
 *
 *   k, v    [total, kv_heads, head_dim] of `dtype` (DSA_DTYPE_BF16 or
 *           DSA_DTYPE_F16), strides in elements.
 *   cu      [seqs + 1] device int32: sequence s's new tokens are rows
 *           [cu[s], cu[s+1]); nondecreasing, and rows behind cu[seqs] are
 *           not read. Offsets are clamped to [0, total]. Those that decrease
 *           leave the blocks of these sequences unspecified, and nothing else.
 *   lens    [seqs] device int32: tokens that each sequence held before. They
 *           are not changed. (Negative ones count as 0.)
 * Row cu[s] + i becomes token lens[s] + i of sequence s. Tokens that have no
 * page, or lie behind max_pages * page_size, are dropped.
 *
 * For each block, head, and keys or values alike, with A the largest finite
 * |x| of the new tokens:
 *   scale = the least power of two, from 2^-126 on, that is not below A / 448,
 *           and, where the block held tokens already, not below its old scale
 *           (a negative or NaN one counts as 0, one over 2^126 as 2^126);
 *   code  = x / scale rounded to nearest even; NaN where x is not finite.
 * Where a block that held tokens gets another scale, their codes become
 * (code * old scale) / scale, rounded likewise (to 448 what passes it). Those
 * are the tokens in front of lens[s]; codes behind the new tokens are left as
 * they were.
 *
 * No two sequences of a call may write to the same block (pages that hold new
 * tokens are not shared).
 *
 * total == 0, seqs == 0 or kv_heads == 0: DSA_OK, nothing written. DSA_EINVAL
 * for an unknown dtype, negative sizes, page_size, block or head_dim < 1, a
 * block that does not divide page_size, ld_tables below max_pages, NULL pages or a
 * NULL required pointer. DSA_EUNSUPPORTED for DSA_DTYPE_F32, layouts and sizes
 * other than above, k or v not 16-byte aligned or with strides that are no
 * multiples of 8 elements, a block over 256, and sizes from 2^31 (seqs from
 * 2^28).
 */
dsa_status dsa_quant_cache_write(const dsa_quant_pages *pages, const void *k,
                                 const void *v, int32_t dtype, int64_t total,
                                 int64_t k_st, int64_t k_sh, int64_t v_st,
                                 int64_t v_sh, const int32_t *cu, int32_t seqs,
                                 const int32_t *lens, void *stream);

/*
 * dsa_quant_cache_read -- the first tokens of each sequence as packed rows
 * (the k and v of dsa_prompt_attention in dsa_attention.h).
 *
 *   cu      [seqs + 1] device int32: token i of sequence s becomes row cu[s] +
 *           i, for i < cu[s+1] - cu[s]. Offsets are clamped to [0, total];
 *           rows of no sequence are left as they were. Offsets that decrease
 *           leave the rows unspecified, and nothing else.
 *   k, v    [total, kv_heads, head_dim] of `dtype` (DSA_DTYPE_BF16 or
 *           DSA_DTYPE_F16): code * scale, rounded once. Rows of tokens that
 *           have no page, or lie behind max_pages * page_size, are 0.
 * Both may not overlap. Errors as for dsa_quant_cache_write.
 */
dsa_status dsa_quant_cache_read(const dsa_quant_pages *pages, const int32_t *cu,
                                int32_t seqs, int64_t total, int32_t dtype,
                                void *k, int64_t k_st, int64_t k_sh, void *v,
                                int64_t v_st, int64_t v_sh, void *stream);

/*
 * Bytes of device workspace of a dsa_quant_attention call with these sizes on
 * the current device (0 where it needs none, and for sizes that it refuses or
 * has nothing to do for). The contents need no initialisation and mean
 * nothing after the call; two calls that may run at the same time must not
 * share a workspace.
 */
size_t dsa_quant_attention_workspace_bytes(int64_t batch, int32_t heads,
                                           int32_t kv_heads, int32_t head_dim,
                                           int64_t max_pages,
                                           int32_t page_size);

/*
 * dsa_quant_attention -- one query token for each of `batch` sequences.
 *
 * Query head h reads key/value head h / (heads / kv_heads). Over the tokens j
 * that a sequence sees, with sk and sv the scales of their blocks:
 *   x_j = scale * log2(e) * sk_j * <q, kcode_j>;   m = max_j x_j;
 *   l   = sum_j 2^(x_j - m);
 *   out = (sum_j 2^(x_j - m) * sv_j * vcode_j) / l;   lse = m + log2(l).
 * A row that sees no token has out = 0 and lse = -inf, and so has one all of
 * whose scores are -inf. Tokens that are not seen have no influence, whatever
 * their codes and scales hold; a NaN in a key (or its scale) that is seen
 * makes the row NaN, one in a value that dimension of it. Scales may be any
 * numbers from 0 on. (out, lse) is a partial output for dsa_merge_attn_out and
 * dsa_correct_attn_out of dsa_dcp_attn.h.
 *
 *   q       [batch, heads, head_dim] of `dtype` (DSA_DTYPE_BF16 or
 *           DSA_DTYPE_F16) at q + b*q_sb + h*q_sh, strides in elements.
 *   lens    [batch] device int32: sequence b sees its tokens [0, lens[b]),
 *           clamped to [0, max_pages * page_size]; tokens on no page are not
 *           seen.
 *   scale   > 0: the factor of <q, k>; scale * log2(e) is finite in fp32.
 *   out     [batch, heads, head_dim] of `dtype`.
 *   lse     [batch, heads] fp32 at lse + b*l_sb + h*l_sh, or NULL.
 *   workspace     dsa_quant_attention_workspace_bytes(...) bytes, 256-byte
 *           aligned (NULL when that is 0).
 *
 * Arithmetic: products of q and codes exact, summed in fp32; scores, maxima,
 * exponentials and sums in fp32; the weights 2^(x_j - m) * sv_j go into the
 * product with the codes of V as two fp16 numbers (rounded to 2^-22 of
 * themselves, or 2^-32 of the largest one); out is rounded once from fp32. Where
 * scale * log2(e) * sk_j, or that times the largest |q| of a row, passes 2^127,
 * the row may be NaN; where scale * log2(e) * sk_j lies below 2^-126 it is
 * rounded to a multiple of 2^-149. Results are held to 2^-149 at the least.
 *
 * batch == 0 or heads == 0: DSA_OK, nothing written. DSA_EINVAL for kv_heads
 * < 1 or no divisor of heads, a scale that is not as above, a workspace that
 * is too small or not aligned, and as for dsa_quant_cache_write.
 * DSA_EUNSUPPORTED as there, for heads / kv_heads > 128, q and out not 16-byte
 * aligned or with strides that are no multiples of 8, and where batch *
 * kv_heads times the 32-token tiles that a row of `tables` has room for passes
 * 2.5 * 10^8, or batch * heads 10^9.
 */
dsa_status dsa_quant_attention(const dsa_quant_pages *pages, const void *q,
                               int32_t dtype, int64_t batch, int32_t heads,
                               int64_t q_sb, int64_t q_sh, const int32_t *lens,
                               float scale, void *out, int64_t o_sb,
                               int64_t o_sh, float *lse, int64_t l_sb,
                               int64_t l_sh, void *workspace,
                               size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_QUANT_H */
