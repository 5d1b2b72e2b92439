/*
 * polar_cache.h -- C ABI of the paged KV cache itself: the pool whose pages
 * polar_attn_decode_paged() and its relatives read.  Rows (sequences) grow,
 * share pages, give them back and are moved together, all on the device and
 * without a host synchronisation, so that a serving loop can be captured into
 * a CUDA graph.  The paper has no counterpart; its paged decode ("GQA-Grouped
 * Paged Decode Kernel", section 2.2 of the technical summary) takes such a
 * cache as given.
 *
 * Conventions as in polar_attn.h: device pointers on the current device, the
 * caller owns all memory, calls are asynchronous on `stream`, host-detected
 * errors return at once with nothing launched, device-detected errors go to
 * the status word that polar_attn_get_status() reads and the kernel skips the
 * row, page or entry in question.  kv_pages, bounds, k, v and workspaces are
 * 16-byte aligned, int32 arrays 4-byte aligned.
 *
 * A page is live while refs[page] > 0: refs[page] is the number of page-table
 * entries that name it.  A table entry counts only below ceil(seqlen / 64).
 * New pages are the free pages with the lowest ids.
 *
 * Every result is determined by the arguments alone (the order in which
 * threads run plays no part).
 */
#ifndef POLAR_CACHE_H
#define POLAR_CACHE_H

#include <stddef.h>
#include <stdint.h>

#include "polar_attn.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
    void *kv_pages;  /* [num_pages, 2, Hkv, 64, 64] dtype: as polar_attn_decode_paged */
    void *bounds;    /* [num_pages, Hkv, 2, 64] dtype, or NULL: per page and kv head the
                        smallest [0] and largest [1] key of each dimension over the page's
                        valid rows, what polar_attn_decode_paged_sparse scores pages by */
    int32_t *refs;   /* [num_pages]: table entries that name the page; 0: free.  NULL only
                        for polar_attn_cache_append (a caller with its own allocator) */
    int num_pages, Hkv;
    int head_dim;    /* must be 64 */
    int dtype;       /* POLAR_BF16 (else POLAR_ERR_UNSUPPORTED) */
} polar_cache_t;

/*
 * Bytes of device scratch that polar_attn_cache_reserve and
 * polar_attn_cache_compact need for this pool and up to num_seqs rows (0 for
 * arguments they reject).  Contents on entry are ignored; calls that share a
 * workspace must not overlap.
 */
size_t polar_attn_cache_workspace_size(const polar_cache_t *cache, int num_seqs);

/*
 * Room for new tokens: row i grows by grow[i] tokens.
 *
 *  page_table [num_seqs, max_pages] int32, in place: entries of new pages
 *  seqlens    [num_seqs] int32, in place: grown by granted[i]
 *  grow       [num_seqs] int32, >= 0
 *  granted    [num_seqs] int32, out: grow[i] where the row was served, else 0
 *
 * Row i takes ceil((len + grow) / 64) - ceil(len / 64) free pages.  A partly
 * filled last page that other entries name too (refs > 1) is first replaced by
 * a copy of its valid rows (keys, values, bounds), so that the row may be
 * written; where all the entries that name it belong to growing rows of this
 * call, the last of those rows keeps the page itself.  Rows are served in
 * order: from the first row whose pages are not there on, no row is served
 * (granted 0, nothing changed) and POLAR_ERR_NO_PAGES is recorded.  A length
 * outside [0, 64 * max_pages], before or after growing, or grow < 0 records
 * POLAR_ERR_BAD_SEQLEN, a last page outside the pool POLAR_ERR_BAD_PAGE; such
 * a row is passed over.
 */
polar_status_t polar_attn_cache_reserve(const polar_cache_t *cache, int32_t *page_table,
                                        int max_pages, int32_t *seqlens, const int32_t *grow,
                                        int num_seqs, int32_t *granted, void *workspace,
                                        size_t ws_bytes, void *stream);

/*
 * Writes the newest tokens of each row into its pages.
 *
 *  k, v       [num_seqs, src_tokens, Hkv, 64] dtype
 *  counts     [num_seqs] int32 in [0, tokens], or NULL: every row gets `tokens`
 *  pick       [num_seqs, tokens] int32, or NULL: token t of a row comes from
 *             source row pick[i][t] (the accepted path of a drafted tree), or
 *             from source row t (then tokens <= src_tokens)
 *  seqlens    [num_seqs] int32: the lengths with the new tokens counted
 *
 * Token t < counts[i] of row i goes to position seqlens[i] - counts[i] + t.
 * With cache->bounds, the bounds of every page that got a token are set from
 * all its valid rows (positions below seqlens[i]).  With cache->refs, a page
 * that is not named by exactly one entry is not written (POLAR_ERR_BAD_PAGE).  A count
 * or length out of range records POLAR_ERR_BAD_SEQLEN and the row is skipped;
 * a source row out of range records POLAR_ERR_BAD_SLOT and that token is
 * skipped; a page outside the pool records POLAR_ERR_BAD_PAGE.  Two rows must
 * not share a page that they write.
 */
polar_status_t polar_attn_cache_append(const polar_cache_t *cache, const void *k, const void *v,
                                       int src_tokens, const int32_t *pick, int tokens,
                                       const int32_t *counts, const int32_t *page_table,
                                       int max_pages, const int32_t *seqlens, int num_seqs,
                                       void *stream);

/*
 * Row i of the destination becomes a copy of source row src_rows[i] that
 * shares its pages (refs + 1 for each entry); nothing is copied but the table.
 *
 *  src_table [num_src, max_pages], src_lens [num_src]: read only
 *  src_rows  [num_dst] int32; negative: the destination row is left alone;
 *            >= num_src records POLAR_ERR_BAD_SLOT and does the same
 *  dst_table [num_dst, max_pages], dst_lens [num_dst]: written up to each
 *            row's ceil(len / 64) entries; what they held before is overwritten
 *            without being given back.  They may not overlap the source's
 *            (POLAR_ERR_INVALID_ARG); one table's rows may serve as both when
 *            the ranges passed are disjoint.
 *
 * A source length outside [0, 64 * max_pages] records POLAR_ERR_BAD_SEQLEN and
 * leaves the row alone; a page outside the pool records POLAR_ERR_BAD_PAGE and
 * its entry is copied as it is.
 */
polar_status_t polar_attn_cache_fork(const polar_cache_t *cache, const int32_t *src_table,
                                     const int32_t *src_lens, int num_src,
                                     const int32_t *src_rows, int num_dst, int32_t *dst_table,
                                     int32_t *dst_lens, int max_pages, void *stream);

/*
 * Gives pages back: row i keeps its first keep[i] tokens.
 *
 *  keep  [num_seqs] int32, or NULL: every row is emptied.  Negative, or at
 *        least the row's length: the row is left alone.
 *
 * Entries from ceil(keep / 64) up to ceil(len / 64) lose their reference and
 * become -1; seqlens[i] becomes keep[i].  A page outside the pool, or one with
 * no reference left to give, records POLAR_ERR_BAD_PAGE (its entry still
 * becomes -1); a length outside [0, 64 * max_pages] records
 * POLAR_ERR_BAD_SEQLEN and the row is left alone.
 */
polar_status_t polar_attn_cache_free(const polar_cache_t *cache, int32_t *page_table,
                                     int max_pages, int32_t *seqlens, const int32_t *keep,
                                     int num_seqs, void *stream);

/*
 * Moves the live pages to the front of the pool.  With n live pages, the k-th
 * live page of id >= n moves to the k-th free id < n; pages below n stay.
 * Keys, values, bounds and references move along, and the entries of the rows
 * passed follow them (every row that names a page of this pool must be among
 * them).  Afterwards pages 0 .. n - 1 are live and the others free.
 *
 *  used  [1] int32, out: n
 *
 * An entry outside the pool, or one that names a free page, records
 * POLAR_ERR_BAD_PAGE and is left as it is; a length outside
 * [0, 64 * max_pages] records POLAR_ERR_BAD_SEQLEN and leaves the row's
 * entries alone.
 */
polar_status_t polar_attn_cache_compact(const polar_cache_t *cache, int32_t *page_table,
                                        int max_pages, const int32_t *seqlens, int num_seqs,
                                        int32_t *used, void *workspace, size_t ws_bytes,
                                        void *stream);

#ifdef __cplusplus
}
#endif

#endif /* POLAR_CACHE_H */
