/*
 * spec_cache.h -- C ABI of the paged key-value cache of a speculative decoding round, and
 * of the attention that reads it (MI355X, gfx950).
 *
 * A round scores N new tokens of every sequence at once and keeps the part of them that the
 * verification (spec_verify.h) accepts:
 *   spec_cache_resize      room in the pool for the sequences' next N slots
 *   spec_cache_append      per layer: the new tokens' keys and values into their slots
 *   spec_paged_attention   per layer: the new tokens' attention over the cache and, for a
 *                          draft tree, over their own ancestors
 *   spec_verify / spec_tree_verify / ...   accepted_len and, for trees, path_nodes
 *   spec_cache_commit      every layer: the accepted path's entries moved together, and
 *                          the new lengths
 *   spec_cache_resize      the pages behind the new lengths given back
 *   spec_cache_fork        continuations of one sequence that share its pages
 *
 * New tokens ("nodes").  Node 0 is the last token emitted (the tree verification's root,
 * whose key and value are not cached yet); nodes 1 .. N-1 are the drafted tokens.  With
 * parent == NULL they are a chain (node i follows node i-1; N = G + 1 for spec_verify with
 * G drafts), otherwise the tree of spec_tree_verify's parent array (parent[b, 0] = -1,
 * 0 <= parent[b, n] < n).  depth(n) is the number of n's ancestors.
 *
 * Cache layout.  A pool holds P pages of page_size slots (a power of two, 16 .. 256); slot s
 * of sequence b lies in page p = page_table[b, s / page_size] at t = s % page_size.  With
 * E = 16 / element size (8 for bf16, 4 for f32):
 *   k_pages [P, Hkv, D / E, page_size, E]  key element d of the slot: [p, h, d / E, t, d % E]
 *   v_pages [P, Hkv, page_size / E, D, E]  value element d:           [p, h, t / E, d, t % E]
 * so that the 16 bytes a lane feeds to a matrix instruction (E consecutive d of one key, E
 * consecutive slots of one value element) lie together.  One layer's pool is one such array;
 * the calls that work on every layer take L of them, one behind the other.  Committed tokens
 * occupy slots 0 .. cache_len[b]-1, node i slot cache_len[b] + i.
 *
 * Conventions are those of spec_verify.h: device pointers to contiguous row-major memory
 * (unless strides are given), the caller owns every buffer, nothing is allocated, kept or
 * synchronised, work is enqueued on `stream`, and a status other than SV_OK means that
 * nothing was enqueued.  Every call may be captured into a HIP graph: no kernel waits for
 * another workgroup, and workspaces need no particular contents.  Outputs do not overlap a
 * call's inputs unless it is stated that they may.  Calls that overlap in time need
 * workspaces of their own, and calls that change a cache or its tables have to be ordered
 * with every other call on them.  Page indexes, lengths, trees and paths are checked on the
 * device: memory outside the pool is never touched, and a sequence with a code in row_status
 * has the outputs stated at each call.
 *
 * Refused sequences.  A sequence that spec_cache_resize refuses (SV_ROW_NO_PAGES, or another
 * code) keeps the pages it has, and the last of them may be one that other sequences hold too:
 * what is written to it is written to theirs.  The calls that follow in the round therefore
 * take the resize's row_status as `prior` (the _after variants below, which are the calls
 * themselves with prior == NULL): prior [B] int32, and a sequence with prior[b] < 0 is left
 * alone, before anything else of it is tested.  Its row_status is prior[b]; nothing of it is
 * written or moved, its attention rows are NaN, and it keeps its length.  prior does not
 * overlap a call's outputs (SV_ERR_PARAM).  It is read on the device, so that a captured round
 * follows refusals too.
 */
#ifndef SPEC_CACHE_H
#define SPEC_CACHE_H

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Codes in row_status (SV_ROW_BAD_TREE of spec_verify.h besides). */
#define SV_ROW_BAD_PAGE (-7)    /* a page index that the call needs lies outside [0, P), or  */
                                /* its reference count is not positive (resize, fork)        */
#define SV_ROW_BAD_LENGTH (-8)  /* a length, count or path that does not fit the tables       */
#define SV_ROW_NO_PAGES (-9)    /* spec_cache_resize: not enough free pages                   */
#define SV_ROW_BAD_FORK (-10)   /* spec_cache_fork: not a pair it can make                    */

#define SV_CACHE_MAX_NEW 1024   /* most new tokens N of a sequence in one call                */
#define SV_CACHE_MAX_SEQS 4096  /* most sequences of spec_cache_resize and spec_cache_fork    */

/* ---- attention of the new tokens over a paged cache ----
 *
 * For node i of sequence b and query head h (key head h / (Hq / Hkv)):
 *   out[b, i, h] = sum_t softmax_t(scale * q[b, i, h] . k_t) v_t
 * over the slots t that the node sees: committed tokens, itself and its ancestors.  With
 * window > 0 a token at position pos is seen only if pos(i) - pos < window or pos < sinks,
 * where pos is a committed token's slot and cache_len[b] + depth for a node.
 *   q            [B, N, Hq, D] dtype; q_stride_b and q_stride_n elements between sequences
 *                and nodes, heads and D contiguous
 *   k_pages, v_pages  one layer's pool
 *   page_table   [B, table_width] int32; entries behind a sequence's slots are not read
 *   cache_len    [B] int32 committed tokens; cache_len + n_new <= table_width * page_size
 *   n_new        [B] int32 new tokens of each sequence, 0 .. N (NULL: N)
 *   parent       [B, N] int32 or NULL, see above (entries behind n_new are not read)
 *   D            64, 128 or 256;  Hq a multiple of Hkv;  N at most SV_CACHE_MAX_NEW;  rows
 *                B * N * Hq, those of a sequence and key head padded to a multiple of 128 at
 *                most, fewer than 2^26
 *   scale        finite;  window >= 0 (0: none);  sinks >= 0 (needs window)
 *   out          [B, N, Hq, D] dtype out; rows of nodes behind n_new are zero
 *   row_status   [B] int32 out: 0, or SV_ROW_BAD_LENGTH, SV_ROW_BAD_TREE, SV_ROW_BAD_PAGE
 *                (tested in this order); the sequence's output rows are then NaN
 *   workspace    sv_attention_workspace_bytes(...) bytes, 256-byte aligned, any contents
 * q, k_pages, v_pages and out start at multiples of 16 bytes, and the strides of q are
 * multiples of 16 bytes (else SV_ERR_ALIGN).  Products are taken in matrix instructions of
 * the inputs' type with f32 sums; scores, softmax statistics and the output's sum are f32,
 * the weights are rounded to the inputs' type for the second product and divided by the sum
 * of the rounded ones.  Weighted values are summed before that division, with weights of up to
 * 2^8: values whose sum over the slots seen passes 2^119 in size may give infinities. */
size_t sv_attention_workspace_bytes(int32_t B, int32_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                    int32_t page_size, int32_t table_width, sv_dtype dtype);
sv_status spec_paged_attention(const void *q, int64_t q_stride_b, int64_t q_stride_n,
                               const void *k_pages, const void *v_pages, sv_dtype dtype,
                               const int32_t *page_table, const int32_t *cache_len,
                               const int32_t *n_new, const int32_t *parent, int32_t B, int32_t N,
                               int32_t Hq, int32_t Hkv, int32_t D, int32_t page_size,
                               int32_t num_pages, int32_t table_width, float scale,
                               int32_t window, int32_t sinks, void *out, int32_t *row_status,
                               void *workspace, size_t workspace_bytes, void *stream);

/* spec_paged_attention with each kernel dispatch bracketed by caller-owned HIP events, as
 * in spec_verify_timed. */
sv_status spec_paged_attention_timed(const void *q, int64_t q_stride_b, int64_t q_stride_n,
                                     const void *k_pages, const void *v_pages, sv_dtype dtype,
                                     const int32_t *page_table, const int32_t *cache_len,
                                     const int32_t *n_new, const int32_t *parent, int32_t B,
                                     int32_t N, int32_t Hq, int32_t Hkv, int32_t D,
                                     int32_t page_size, int32_t num_pages, int32_t table_width,
                                     float scale, int32_t window, int32_t sinks, void *out,
                                     int32_t *row_status, void *workspace,
                                     size_t workspace_bytes, void *stream, void *const *events,
                                     int32_t n_events, int32_t *n_launched);

/* spec_paged_attention (with events as in spec_paged_attention_timed where they are given)
 * behind a call that may have refused sequences: see `prior` above. */
sv_status spec_paged_attention_after(const void *q, int64_t q_stride_b, int64_t q_stride_n,
                                     const void *k_pages, const void *v_pages, sv_dtype dtype,
                                     const int32_t *page_table, const int32_t *cache_len,
                                     const int32_t *n_new, const int32_t *parent,
                                     const int32_t *prior, int32_t B, int32_t N, int32_t Hq,
                                     int32_t Hkv, int32_t D, int32_t page_size,
                                     int32_t num_pages, int32_t table_width, float scale,
                                     int32_t window, int32_t sinks, void *out,
                                     int32_t *row_status, void *workspace,
                                     size_t workspace_bytes, void *stream, void *const *events,
                                     int32_t n_events, int32_t *n_launched);

/* Names of the kernels spec_paged_attention launches, ';'-separated (static storage). */
const char *sv_attention_launch_plan(int32_t N, int32_t Hq, int32_t Hkv, int32_t D, sv_dtype dtype);

/* ---- the new tokens' keys and values into the cache ----
 *
 * Writes k[b, i] and v[b, i] into slot cache_len[b] + i for i < n_new[b], in one layer's pool.
 *   k, v         [B, N, Hkv, D] dtype; strides as for q above, 16-byte aligned
 *   row_status   [B] int32 out: 0, SV_ROW_BAD_LENGTH or SV_ROW_BAD_PAGE; nothing of the
 *                sequence is then written
 * D is a multiple of 16 up to 512.  The slots' pages must be the sequence's own (as
 * spec_cache_resize leaves them for the sequences that it serves; the others are told by
 * `prior` above): two sequences that write to one page race. */
sv_status spec_cache_append(const void *k, int64_t k_stride_b, int64_t k_stride_n, const void *v,
                            int64_t v_stride_b, int64_t v_stride_n, sv_dtype dtype, void *k_pages,
                            void *v_pages, const int32_t *page_table, const int32_t *cache_len,
                            const int32_t *n_new, int32_t B, int32_t N, int32_t Hkv, int32_t D,
                            int32_t page_size, int32_t num_pages, int32_t table_width,
                            int32_t *row_status, void *stream);
sv_status spec_cache_append_after(const void *k, int64_t k_stride_b, int64_t k_stride_n,
                                  const void *v, int64_t v_stride_b, int64_t v_stride_n,
                                  sv_dtype dtype, void *k_pages, void *v_pages,
                                  const int32_t *page_table, const int32_t *cache_len,
                                  const int32_t *n_new, const int32_t *prior, int32_t B,
                                  int32_t N, int32_t Hkv, int32_t D, int32_t page_size,
                                  int32_t num_pages, int32_t table_width, int32_t *row_status,
                                  void *stream);

/* ---- the accepted path's entries moved together, and the new lengths ----
 *
 * After a verification node 0 and the accepted nodes stay: the entry of node
 * path_nodes[b, j] moves from slot cache_len[b] + path_nodes[b, j] to cache_len[b] + 1 + j,
 * j < accepted_len[b], in every layer, and new_len[b] = cache_len[b] + 1 + accepted_len[b].
 *   k_pages, v_pages  L pools, one behind the other (num_pages pages each)
 *   accepted_len [B] int32 as the verification left it; negative (a row code): the sequence
 *                keeps its length, and the code is handed on in row_status
 *   path_nodes   [B, N] int32 as spec_tree_verify left it (increasing nodes 1 .. N-1), or
 *                NULL for chains, whose accepted entries lie together already
 *   new_len      [B] int32 out; may be cache_len itself for chains (with path_nodes, outputs
 *                that overlap cache_len or accepted_len are SV_ERR_PARAM)
 *   row_status   [B] int32 out: 0, the verification's code, SV_ROW_BAD_LENGTH (accepted_len
 *                beyond N - 1, or slots beyond the table), SV_ROW_BAD_TREE (path_nodes not
 *                increasing in 1 .. N-1) or SV_ROW_BAD_PAGE; new_len is then cache_len and
 *                nothing of the sequence is moved
 * D is a multiple of 16 up to 512.  The slots' pages must be the sequence's own, as for the
 * append. */
sv_status spec_cache_commit(void *k_pages, void *v_pages, sv_dtype dtype,
                            const int32_t *page_table, const int32_t *cache_len,
                            const int32_t *accepted_len, const int32_t *path_nodes, int32_t L,
                            int32_t B, int32_t N, int32_t Hkv, int32_t D, int32_t page_size,
                            int32_t num_pages, int32_t table_width, int32_t *new_len,
                            int32_t *row_status, void *stream);
sv_status spec_cache_commit_after(void *k_pages, void *v_pages, sv_dtype dtype,
                                  const int32_t *page_table, const int32_t *cache_len,
                                  const int32_t *accepted_len, const int32_t *path_nodes,
                                  const int32_t *prior, int32_t L, int32_t B, int32_t N,
                                  int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages,
                                  int32_t table_width, int32_t *new_len, int32_t *row_status,
                                  void *stream);

/* ---- pages taken, given back and copied on write ----
 *
 * The pool's books: page_table [S, table_width] with seq_pages[b] pages held by sequence b
 * (the rest of its row is -1), ref_count[p] the number of rows that hold page p, and free_map
 * with bit p % 32 of word p / 32 set where ref_count[p] == 0 (bits of no page are 0).  An
 * empty pool has seq_pages 0, page_table -1, ref_count 0 and every page's bit set.
 *
 * For every sequence with want_len[b] >= 0, in this order:
 *   1. pages behind the first ceil(want_len / page_size) are given back (their entries
 *      become -1); a page that nobody holds then is free;
 *   2. where want_len > keep_len: pages are added up to ceil(want_len / page_size), and held
 *      pages at or behind slot keep_len that others hold too are replaced by fresh ones, so
 *      that slots keep_len .. want_len - 1 are the sequence's own to write.  Where such a page
 *      holds kept slots (keep_len % page_size > 0), those slots are copied, in all L layers.
 * Fresh pages are the free pages of lowest index, in the order of the sequences and of their
 * slots.  A sequence is served only if the free pages cover its need and the needs of all
 * sequences before it; one that is not, and every later one that needs a page, keeps the pages
 * it has after step 1 (SV_ROW_NO_PAGES).  Pages that step 2 replaces become free after the
 * call's allocation, when nobody else holds them.
 *   keep_len     [S] int32 tokens whose entries stay, within the pages held
 *   want_len     [S] int32 slots to have room for; -1 leaves the sequence as it is
 *   k_pages, v_pages  L pools (NULL with L = 0: the caller copies, or shares no pages)
 *   row_status   [S] int32 out: 0, SV_ROW_BAD_LENGTH, SV_ROW_BAD_PAGE (neither changes the
 *                sequence's row) or SV_ROW_NO_PAGES
 *   workspace    sv_resize_workspace_bytes(S, num_pages) bytes, 256-byte aligned
 * S * table_width fits 31 bits (else SV_ERR_SHAPE). */
size_t sv_resize_workspace_bytes(int32_t S, int32_t num_pages);
sv_status spec_cache_resize(int32_t *page_table, int32_t *seq_pages, int32_t *ref_count,
                            int32_t *free_map, const int32_t *keep_len, const int32_t *want_len,
                            void *k_pages, void *v_pages, sv_dtype dtype, int32_t L, int32_t S,
                            int32_t Hkv, int32_t D, int32_t page_size, int32_t num_pages,
                            int32_t table_width, int32_t *row_status, void *workspace,
                            size_t workspace_bytes, void *stream);

/* ---- continuations that share a sequence's pages ----
 *
 * For pair i: sequence dst[i], which holds no pages, becomes a continuation of src[i]: its
 * table row, seq_pages and cache_len are copied, and every page it then holds counts one
 * holder more.  Nothing is copied until one of them writes (spec_cache_resize).
 *   cache_len    [S] int32, read at src and written at dst
 *   src, dst     [F] int32
 *   pair_status  [F] int32 out: 0, SV_ROW_BAD_FORK (an index outside [0, S), dst already
 *                holding pages, a dst that is some pair's src, or that an earlier pair
 *                names), SV_ROW_BAD_LENGTH (seq_pages[src] outside [0, table_width]) or
 *                SV_ROW_BAD_PAGE; such a pair changes nothing */
sv_status spec_cache_fork(int32_t *page_table, int32_t *seq_pages, int32_t *ref_count,
                          int32_t *cache_len, const int32_t *src, const int32_t *dst, int32_t F,
                          int32_t S, int32_t num_pages, int32_t table_width,
                          int32_t *pair_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_CACHE_H */
