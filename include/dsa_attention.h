/*
 * dsa_attention.h -- C ABI of the attention operators in the GB300 (sm_103a)
 * library libdsa_cb.so (status codes and the conventions on device pointers
 * and streams are those of dsa_cb.h; element types are dsa_dtype of
 * dsa_dcp_attn.h).
 *
 * Both operators compute, for every query row q of `heads` query heads that
 * share `kv_heads` key/value heads in groups of G = heads / kv_heads (query
 * head h reads key/value head h / G), over the keys j that the row sees:
 *   x_j = scale * log2(e) * <q, k_j>;   m = max_j x_j;
 *   l   = sum_j 2^(x_j - m);
 *   out = (sum_j 2^(x_j - m) v_j) / l;  lse = m + log2(l)   (base 2).
 * A row that sees no key has out = 0 and lse = -inf, and so has one all of
 * whose scores are -inf (of infinities in q or k). Keys that a row does not
 * see have no influence on it, whatever they hold, not on a bit; a NaN in a key
 * that it sees makes the row NaN, one in a value that dimension of it.
 * (An output that is not finite, of a row that does not see all of its block's
 * keys, costs about the block's time once more.)
 *
 * (out, lse) is a partial output for dsa_merge_attn_out and
 * dsa_correct_attn_out of dsa_dcp_attn.h: runs over disjoint sets of keys
 * merge into the run over their union. Those two take bf16 and fp32: an fp16
 * out is widened to fp32 for them (which loses nothing).
 *
 * Arithmetic: products of bf16 or fp16 operands summed in fp32; maxima,
 * exponentials and sums in fp32; the weights 2^(x_j - m) are rounded to the
 * operands' type for the product with V; out is rounded once from fp32 (to
 * nearest even).
 *
 * Layouts: element (t, h, d) of a [tokens, heads, head_dim] tensor lies at
 * base + t*st + h*sh + d, strides in elements. Bases are 16-byte aligned and
 * strides are multiples of 8 elements for q, k, v and out (other layouts
 * return DSA_EUNSUPPORTED); the LSEs may have any strides. out and lse
 * overlap no input.
 */
#ifndef DSA_ATTENTION_H
#define DSA_ATTENTION_H

#include <stddef.h>
#include <stdint.h>

#include "dsa_cb.h"
#include "dsa_dcp_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

/*
 * Bytes of device workspace of a dsa_prompt_attention call with these sizes
 * on the current device (0 where it needs none, and for sizes that it refuses
 * or has nothing to do for). The contents need no initialisation and mean
 * nothing after the call; two calls that may run at the same time must not
 * share a workspace.
 */
size_t dsa_prompt_workspace_bytes(int64_t total_q, int64_t total_k,
                                  int32_t heads, int32_t kv_heads,
                                  int32_t head_dim, int32_t seqs);

/*
 * dsa_prompt_attention -- attention of whole prompts, packed.
 *
 *   q      [total_q, heads, head_dim] of `dtype` (DSA_DTYPE_BF16 or
 *          DSA_DTYPE_F16).
 *   k, v   [total_k, kv_heads, head_dim] of `dtype`.
 *   cu_q   [seqs + 1] device int32: sequence i's queries are rows
 *          [cu_q[i], cu_q[i+1]); nondecreasing.
 *   cu_k   [seqs + 1] device int32: its keys are rows [cu_k[i], cu_k[i+1]).
 *   causal 0: every query of a sequence sees all of its keys; nonzero: query
 *          t of n sees the keys j <= t + (keys - n), so that the last query
 *          sees all of them (the keys before the first query are cached ones).
 *   scale  > 0: the factor of <q, k>; scale * log2(e) is finite in fp32
 *          (scale up to 2.35e38).
 *   out    [total_q, heads, head_dim] of `dtype`.
 *   lse    [total_q, heads] fp32 at lse + t*l_st + h*l_sh, or NULL.
 *   workspace     dsa_prompt_workspace_bytes(...) bytes, 256-byte aligned
 *          (NULL when that is 0).
 *
 * Offsets are clamped to [0, total]; a sequence whose end is below its start
 * is empty. Rows that belong to no sequence (behind the last one, as in a
 * padded batch) are left as they were. Offsets that decrease leave the rows
 * of out and lse unspecified, and nothing else.
 *
 * total_q == 0, heads == 0 or seqs == 0: DSA_OK, nothing written. DSA_EINVAL
 * for an unknown dtype, negative sizes, kv_heads < 1 or no divisor of heads,
 * head_dim < 1, a scale that is not as above, or a NULL q, cu_q, cu_k or
 * out (or k or v with total_k > 0), or a workspace that is too small.
 * DSA_EUNSUPPORTED for
 * DSA_DTYPE_F32, head_dim over 128 or no multiple of 8, heads / kv_heads >
 * 128, layouts other than above, and sizes from 2^31 (total_k from 2^31 -
 * 4096).
 */
dsa_status dsa_prompt_attention(const void *q, const void *k, const void *v,
                                int32_t dtype, int64_t total_q, int64_t total_k,
                                int32_t heads, int32_t kv_heads,
                                int32_t head_dim, int64_t q_st, int64_t q_sh,
                                int64_t k_st, int64_t k_sh, int64_t v_st,
                                int64_t v_sh, const int32_t *cu_q,
                                const int32_t *cu_k, int32_t seqs,
                                int32_t causal, float scale, void *out,
                                int64_t o_st, int64_t o_sh, float *lse,
                                int64_t l_st, int64_t l_sh, void *workspace,
                                size_t workspace_bytes, void *stream);

/*
 * Bytes of device workspace of a dsa_shared_prefix_attention call with these
 * sizes on the current device (0 for sizes that it refuses or has nothing to
 * do for). The contents need no initialisation and mean nothing after the
 * call; two calls that may run at the same time must not share a workspace.
 */
size_t dsa_shared_prefix_workspace_bytes(int64_t batch, int32_t heads,
                                         int32_t kv_heads, int32_t head_dim,
                                         int64_t prefix_len, int64_t max_pages,
                                         int32_t page_size);

/*
 * dsa_shared_prefix_attention -- one query token for each of `batch`
 * sequences on a paged cache, whose first prefix_len tokens are the same for
 * all: those keys and values are read once for the whole batch.
 *
 *   q        [batch, heads, head_dim] of `dtype` at q + b*q_sb + h*q_sh.
 *   k_pages, v_pages  [num_pages, page_size, kv_heads, head_dim] of `dtype`:
 *            token t of page n, head h at k_pages + n*k_sn + t*k_st + h*k_sh.
 *   tables   [batch, max_pages] device int32 at tables + b*ld_tables + i:
 *            token t of sequence b lies on page tables[b][t / page_size].
 *   lens     [batch] device int32: sequence b sees its tokens
 *            [0, lens[b]), clamped to [0, max_pages * page_size].
 *   prefix_len    a multiple of page_size, 0 for no shared prefix: for t <
 *            prefix_len the page is prefix_pages[t / page_size] for every
 *            sequence and the tables' first prefix_len / page_size columns
 *            are not read (a sequence with fewer tokens sees what it has).
 *   prefix_pages  [prefix_len / page_size] device int32; NULL when
 *            prefix_len == 0. May be a row of `tables`; `tables` itself stands
 *            for the first row whose slot is not empty (its length is over 0
 *            or its first entry not negative; row 0 if all are empty).
 *   out      [batch, heads, head_dim] of `dtype`.
 *   lse      [batch, heads] fp32 at lse + b*l_sb + h*l_sh, or NULL.
 *   workspace     dsa_shared_prefix_workspace_bytes(...) bytes, 256-byte
 *            aligned (NULL when that is 0).
 *
 * Tokens on a page whose id is not in [0, num_pages) (such as -1) are not
 * seen. page_size is a power of two, at least 16.
 *
 * batch == 0 or heads == 0: DSA_OK, nothing written. DSA_EINVAL and
 * DSA_EUNSUPPORTED as for dsa_prompt_attention, and DSA_EINVAL for a
 * prefix_len that is negative, no multiple of page_size or over max_pages *
 * page_size, a NULL required pointer or a workspace that is too small or not
 * aligned, and for ld_tables below max_pages; DSA_EUNSUPPORTED for another
 * page_size, and where batch * kv_heads times the 128-token tiles that a row of
 * `tables` has room for passes 10^8, or batch * heads 8 * 10^9.
 */
dsa_status dsa_shared_prefix_attention(
    const void *q, const void *k_pages, const void *v_pages, int32_t dtype,
    int64_t batch, int32_t heads, int32_t kv_heads, int32_t head_dim,
    int64_t num_pages, int32_t page_size, int64_t q_sb, int64_t q_sh,
    int64_t k_sn, int64_t k_st, int64_t k_sh, int64_t v_sn, int64_t v_st,
    int64_t v_sh, const int32_t *prefix_pages, int64_t prefix_len,
    const int32_t *tables, int64_t max_pages, int64_t ld_tables,
    const int32_t *lens, float scale, void *out, int64_t o_sb, int64_t o_sh,
    float *lse, int64_t l_sb, int64_t l_sh, void *workspace,
    size_t workspace_bytes, void *stream);

/*
 * dsa_attention_error -- whether a wait inside an attention kernel has given
 * up (after some ten seconds without any progress) since the process started
 * or the last clear; such a call's outputs are not valid. Returns the wait's nonzero site code, 0 for
 * none, or -1 if the flag could not be read. clear != 0 resets it after
 * reading. Waits for all of the current device's streams first; not for use
 * while one of them is captured.
 */
int dsa_attention_error(int clear);

#ifdef __cplusplus
}
#endif

#endif /* DSA_ATTENTION_H */
