/*
 * dsa_cache.h -- C ABI of the paged cache's bookkeeping in the GB300
 * (sm_103a) library libdsa_cb.so: forking, freeing and compacting sequences
 * whose tokens lie on pages (the cache that dsa_shared_prefix_attention of
 * dsa_attention.h reads). Status codes and the conventions on device pointers
 * and streams are those of dsa_cb.h. All of the state is on the device and
 * no call waits for it:
 *
 *   cache   `planes` pools of num_pages pages (the keys and the values of
 *           every layer, say), each page page_size tokens of token_bytes:
 *           token t of page n in plane p at cache + p*plane_stride +
 *           n*page_stride + t*token_bytes, all in bytes and multiples of 16
 *           (the base 16-byte aligned), or DSA_EUNSUPPORTED. A page has the
 *           same number in all planes.
 *   refs    [num_pages] int32: how many tables hold the page; 0: free.
 *   tables  [seqs, max_pages] int32 at tables + s*ld_tables + i: token t of
 *           sequence slot s lies on page tables[s][t / page_size]; -1: none.
 *           A slot owns a reference to each page of its row.
 *   lens    [seqs] int32: tokens of each slot. A slot is empty when its
 *           length is 0 and its row's first entry is negative.
 *
 * Results do not depend on the order in which the GPU does the work. Entries
 * of tables outside [0, num_pages) stand for no page: they are copied and
 * cleared like -1, never followed. Calls on the same state are ordered by the
 * caller (one stream, or events).
 */
#ifndef DSA_CACHE_H
#define DSA_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "dsa_cb.h"

#ifdef __cplusplus
extern "C" {
#endif

/* What dsa_cache_fork writes for each pair. */
enum {
    DSA_FORK_OK = 0,
    DSA_FORK_NO_PAGE = 1, /* no free page left for its last, partial page */
    DSA_FORK_REFUSED = 2  /* bad slot numbers, a child that is not empty or
                             named before, or a parent whose partial page is
                             missing; the child is left as it was */
};

/*
 * Bytes of device workspace of dsa_cache_fork (pairs, num_pages) and of
 * dsa_cache_compact (pairs = 0); 0 for negative sizes. No initialisation is
 * needed; calls that may overlap must not share one.
 */
size_t dsa_cache_workspace_bytes(int64_t pairs, int64_t num_pages);

/*
 * dsa_cache_fork -- makes slot children[i] a copy of slot parents[i].
 *
 * The pages that the parent fills whole (lens / page_size of them) are shared:
 * the child's row holds them too and their refs go up by one. When its last
 * page is partly filled, the child gets a page of its own, with the used
 * tokens copied in all planes: the free pages go to the pairs that need one
 * in the order of i, lowest page first. Parents are taken as they were before
 * the call. Behind its pages the child's row is -1.
 *
 *   parents, children  [pairs] device int32.
 *   status  [pairs] device int32, DSA_FORK_* of each pair. A pair that is
 *           refused or finds no page changes nothing (a later pair that
 *           needs no page may still succeed).
 *
 * pairs == 0: DSA_OK. DSA_EINVAL for negative sizes, page_size < 1,
 * max_pages < 1 with pairs > 0, NULL pointers or a workspace that is too
 * small; DSA_EUNSUPPORTED for layouts other than above and for sizes from
 * 2^31 (pairs from 2^16).
 */
dsa_status dsa_cache_fork(void *cache, int64_t planes, int64_t plane_stride,
                          int64_t num_pages, int64_t page_stride,
                          int32_t page_size, int64_t token_bytes, int32_t *refs,
                          int32_t *tables, int64_t seqs, int64_t max_pages,
                          int64_t ld_tables, int32_t *lens,
                          const int32_t *parents, const int32_t *children,
                          int64_t pairs, int32_t *status, void *workspace,
                          size_t workspace_bytes, void *stream);

/*
 * dsa_cache_fork_scaled -- dsa_cache_fork for pages that have scales beside them
 * (those of dsa_quant.h): `scale_bytes` of each page n in plane p at scales +
 * p*scale_plane_stride + n*scale_page_stride, in bytes and multiples of 4.
 * With a partial page that is copied go all of its scales.
 *
 * Errors as for dsa_cache_fork, and DSA_EINVAL for negative scale sizes or NULL
 * scales with scale_bytes > 0, DSA_EUNSUPPORTED for other multiples and for
 * scale_bytes from 2^31.
 */
dsa_status dsa_cache_fork_scaled(
    void *cache, int64_t planes, int64_t plane_stride, int64_t num_pages,
    int64_t page_stride, int32_t page_size, int64_t token_bytes, void *scales,
    int64_t scale_plane_stride, int64_t scale_page_stride, int64_t scale_bytes,
    int32_t *refs, int32_t *tables, int64_t seqs, int64_t max_pages,
    int64_t ld_tables, int32_t *lens, const int32_t *parents,
    const int32_t *children, int64_t pairs, int32_t *status, void *workspace,
    size_t workspace_bytes, void *stream);

/*
 * dsa_cache_free -- empties the slots named in seqs_list: the refs of the
 * pages of their rows go down by one (not below 0), their rows become -1 and
 * their lengths 0. Numbers outside [0, seqs) are passed over; a slot named
 * twice is freed once. Errors as for dsa_cache_fork.
 */
dsa_status dsa_cache_free(int32_t *refs, int64_t num_pages, int32_t *tables,
                          int64_t seqs, int64_t max_pages, int64_t ld_tables,
                          int32_t *lens, const int32_t *seqs_list,
                          int64_t count, void *stream);

/*
 * dsa_cache_compact -- moves the pages in use (refs > 0) to the lowest
 * numbers: with n of them, the used pages numbered n or more go, in order, to
 * the free pages below n, in order (no other page moves). Contents (whole
 * pages, all planes), refs and the entries of all tables follow.
 *
 *   remap   [num_pages] device int32: where the contents of each used page
 *           now are; -1 for pages that were free.
 *   live    [1] device int32: n.
 *
 * The old places of moved pages keep their bytes. A table entry that names a
 * free page becomes -1. num_pages == 0: DSA_OK, live = 0. Errors as for
 * dsa_cache_fork.
 */
dsa_status dsa_cache_compact(void *cache, int64_t planes, int64_t plane_stride,
                             int64_t num_pages, int64_t page_stride,
                             int32_t page_size, int64_t token_bytes,
                             int32_t *refs, int32_t *tables, int64_t seqs,
                             int64_t max_pages, int64_t ld_tables,
                             int32_t *remap, int32_t *live, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * dsa_cache_compact_scaled -- dsa_cache_compact for pages that have scales
 * beside them, which follow the pages. Scales and errors as for
 * dsa_cache_fork_scaled.
 */
dsa_status dsa_cache_compact_scaled(
    void *cache, int64_t planes, int64_t plane_stride, int64_t num_pages,
    int64_t page_stride, int32_t page_size, int64_t token_bytes, void *scales,
    int64_t scale_plane_stride, int64_t scale_page_stride, int64_t scale_bytes,
    int32_t *refs, int32_t *tables, int64_t seqs, int64_t max_pages,
    int64_t ld_tables, int32_t *remap, int32_t *live, void *workspace,
    size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* DSA_CACHE_H */
