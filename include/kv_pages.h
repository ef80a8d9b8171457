/* Ownership and data of the pages of a paged cache: reserve, fork, free, compact, copy; and
 * what a step needs to know of them: its tokens' places, and the prefixes that rows share.
 *
 * State, all on the device and owned by the caller:
 *   block_table  int32 [n_tables, table_ld]: row t holds the page ids of one sequence,
 *                page i for its positions [i * page_size, (i + 1) * page_size); an
 *                entry < 0 holds none
 *   refs         int32 [num_pages]: how many owners a page has (table entries of this
 *                table, and any the caller adds for itself); a page with 0 is free
 *   planes       the tensors that hold the pages' data (codes and scales of every
 *                layer, indexer keys, ...): page p of a plane is the page_bytes bytes at
 *                base + p * page_bytes
 *
 * Sequences share pages. Fork makes a child row share its parent's pages and copies
 * nothing; reserve makes the positions about to be written writable, which gives a
 * sequence the pages that it lacks and a copy of a page that it shares; free drops the
 * pages past a kept length (a rejected draft's, a finished sequence's); compact moves
 * live pages into the lowest ids. Free pages are given out lowest id first, in the
 * order of the rows named and of their pages, so every result is determined by the
 * arguments. Nothing here waits on the host or allocates.
 *
 * Each call is enqueued on `stream`. The two launches of a reserve or a compact use the
 * workspace together: host threads that share one enqueue their calls one after another.
 * A row id may be named once per call; rows, parents and children that break this, or a
 * contract below, race on the table and the counts, but every access stays inside the
 * arrays. */
#ifndef KV_PAGES_H
#define KV_PAGES_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* kvpages_stream_t; /* identical to cudaStream_t */

/* One tensor of page data (a host struct, copied by the call). */
typedef struct {
  void* base;         /* device; 4-byte aligned */
  int64_t page_bytes; /* a positive multiple of 4 */
} kvpages_plane;

#define KVPAGES_MAX_PLANES 240

/* Host-side return codes (negative: nothing was enqueued). */
enum {
  KVPAGES_OK = 0,
  KVPAGES_ERR_NULL = -1,      /* a required pointer is NULL */
  KVPAGES_ERR_SHAPE = -2,     /* n < 0, n_tables < 1, table_ld < 1 or > 2^31 - 1, page_size < 1,
                                 num_pages < 0, n_planes outside [0, KVPAGES_MAX_PLANES],
                                 page_bytes not a positive multiple of 4 */
  KVPAGES_ERR_ALIGN = -3,     /* a plane or an int32 array not 4-byte aligned, workspace not
                                 16-byte aligned */
  KVPAGES_ERR_CUDA = -4,      /* a launch or a device query failed */
  KVPAGES_ERR_WORKSPACE = -5  /* workspace smaller than kvpages_workspace_bytes */
};

/* Device status bits, OR-ed into *status (NULL: not reported). */
enum {
  KVPAGES_STATUS_ROW = 1,       /* a row id outside [0, n_tables): skipped */
  KVPAGES_STATUS_LEN = 2,       /* a length < 0, old > new, or past the table row: skipped */
  KVPAGES_STATUS_PAGE = 4,      /* a page id >= num_pages (or a pair's id < 0 on one side
                                   only): that entry is skipped */
  KVPAGES_STATUS_NO_PAGE = 8,   /* reserve: too few free pages for a row; it and the rows
                                   named after it that need pages get none; step: a
                                   position without a page: its slot is -1 */
  KVPAGES_STATUS_CHILD = 16,    /* fork: the child row still holds pages: skipped */
  KVPAGES_STATUS_REFS = 32,     /* free: a page without an owner: its count stays; compact:
                                   a table entry that names a free page: left as it is */
  KVPAGES_STATUS_TOKENS = 64    /* step: more tokens than places: the last ones have none */
};

/* Bytes of device workspace for reserve and compact (pure). 0 for invalid arguments. */
size_t kvpages_workspace_bytes(int n, int num_pages);

/* Makes positions [old_lens[i], new_lens[i]) of row rows[i] writable: of the pages they
 * lie in, a missing one becomes a free page, one that others own too becomes a free page
 * (holding a copy of the data if it has positions < old_lens[i]). Rows are served in
 * order; one that cannot be served whole gets nothing. Two launches. */
int kvpages_reserve(const int32_t* rows, const int32_t* old_lens, const int32_t* new_lens, int n,
                    int32_t* block_table, int n_tables, int64_t table_ld, int page_size,
                    int32_t* refs, int num_pages, const kvpages_plane* planes, int n_planes,
                    void* workspace, size_t ws_bytes, int32_t* status, kvpages_stream_t stream);

/* Row children[i] := the entries of row parents[i] for its first ceil(lens[i] /
 * page_size) pages (placeholders < 0 as they are); the pages get one more owner. The
 * child row must hold no page; a row may be the parent of many children, but not parent
 * and child in one call. One launch. */
int kvpages_fork(const int32_t* parents, const int32_t* children, const int32_t* lens, int n,
                 int32_t* block_table, int n_tables, int64_t table_ld, int page_size,
                 int32_t* refs, int num_pages, int32_t* status, kvpages_stream_t stream);

/* Row rows[i] keeps its first ceil(keep_lens[i] / page_size) pages (none where keep_lens
 * is NULL); the other entries become -1 and their pages lose an owner. One launch. */
int kvpages_free(const int32_t* rows, const int32_t* keep_lens, int n, int32_t* block_table,
                 int n_tables, int64_t table_ld, int page_size, int32_t* refs, int num_pages,
                 int32_t* status, kvpages_stream_t stream);

/* With L live pages (refs > 0): the k-th live page with id >= L moves, data and count, to
 * the k-th free id < L, and every table entry follows. Two launches.
 *   new_ids  device int32 [num_pages] (written): the new id of each page, -1 of a free one
 *   counts   device int32 [2] or NULL (written): L, pages moved */
int kvpages_compact(int32_t* block_table, int n_tables, int64_t table_ld, int32_t* refs,
                    int num_pages, const kvpages_plane* planes, int n_planes, int32_t* new_ids,
                    int32_t* counts, void* workspace, size_t ws_bytes, int32_t* status,
                    kvpages_stream_t stream);

/* Page src[i] of every plane is copied to page dst[i]; a pair of two negative ids is
 * padding. No page may be the destination of two pairs, or the source of one and the
 * destination of another. One launch. */
int kvpages_copy(const int32_t* src, const int32_t* dst, int n, int num_pages,
                 const kvpages_plane* planes, int n_planes, int32_t* status,
                 kvpages_stream_t stream);

/* The places of a step's new tokens. Request i (row rows[i]) brings positions [old_lens[i],
 * new_lens[i]); the tokens stand one after another in the order of the requests, token t of
 * request i from starts[i] on. With pos its position:
 *   positions    device int32 [tokens] (written): pos
 *   token_table  device int32 [tokens] (written): rows[i], as kv8_store, indexer_k_prologue and
 *                (for rows of one query) kv8_attention's group_table take it
 *   slots        device int32 [tokens] (written): table[rows[i]][pos / page_size] * page_size +
 *                pos % page_size; -1 where the entry is negative (KVPAGES_STATUS_NO_PAGE) or
 *                not below num_pages (KVPAGES_STATUS_PAGE)
 *   lens         device int32 [tokens] (written): pos + 1, what a causal query row sees
 *   starts       device int32 [n + 1] (written): min(tokens, tokens of the requests before)
 * `tokens` is the number of places, for graphs a bound on the step's tokens: the places behind
 * the last token hold -1, -1, -1 and 0 (an attention row of length 0 attends to nothing, a
 * store skips a token of row -1; both set their status bits for that row). A request that fails a
 * check brings no tokens. num_pages * page_size < 2^31. One launch. */
int kvpages_step(const int32_t* rows, const int32_t* old_lens, const int32_t* new_lens, int n,
                 const int32_t* block_table, int n_tables, int64_t table_ld, int page_size,
                 int num_pages, int tokens, int32_t* positions, int32_t* token_table,
                 int32_t* slots, int32_t* lens, int32_t* starts, int32_t* status,
                 kvpages_stream_t stream);

/* How long a prefix the rows of each set share. Set s is the requests set_starts[s] ..
 * set_starts[s + 1] - 1 of (rows[i], lens[i]), i < n; those of length 0 are left out.
 *   set_starts   device int32 [n_sets + 1], rising, within [0, n]
 *   prefix_lens  device int32 [n_sets] (written): page_size times the number of leading pages,
 *                all inside the least length of the set, that are the same page (of [0,
 *                num_pages)) in every row of the set; 0 for a set of fewer than two rows,
 *                and where a row or a length of the set fails a check
 * What kv8_attention_shared takes as prefix_lens. One launch. */
int kvpages_shared(const int32_t* rows, const int32_t* lens, int n, const int32_t* set_starts,
                   int n_sets, const int32_t* block_table, int n_tables, int64_t table_ld,
                   int page_size, int num_pages, int32_t* prefix_lens, int32_t* status,
                   kvpages_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* KV_PAGES_H */
