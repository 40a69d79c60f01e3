/*
 * sv_tree.h -- C ABI of the tree operators of libspecverify.so: a decoding
 * step that drafts a TREE of tokens per request instead of a chain.
 *
 *   sv_tree_attention   the drafted nodes' keys and values go to a paged
 *                       cache, and every node attends to the cached prefix
 *                       and to its own ancestors;
 *   sv_tree_verify      lossless verification of the tree from given
 *                       uniforms (spec_verify is its chain form);
 *   sv_cache_commit     the accepted path's cache rows move behind the prefix;
 *   sv_cache_resize     a slot gets or gives back pages to match a length;
 *   sv_cache_fork       a cached sequence is forked into others.
 *
 * The tree.  A request has counts[b] nodes (0 <= counts[b] <= N; NULL = N
 * each).  Node 0 is the root: the last token the request has committed, whose
 * key and value are not cached yet.  parents[b][i] < i is the parent of node
 * i >= 1 (parents[b][0] is not read); parents == NULL is a chain.  A request
 * with counts[b] = 0 is an idle slot.
 *
 * The cache.  Keys and values live in pages of page_size rows; row t of
 * request b is row t % page_size of page page_table[b][t / page_size].
 * Entries of the table that no row needs are never used as page ids (they
 * hold -1 by convention, see sv_cache_resize).  All strides are in elements;
 * the head dimension is contiguous.
 *
 * Ownership, streams and errors are those of spec_verify.h: device memory of
 * the caller, nothing allocated, work enqueued on `stream`, argument errors
 * found on the host before anything is enqueued.  Values that only the device
 * can check never cause an access out of bounds; what happens to such a
 * request is said at each function.
 */
#ifndef SV_TREE_H
#define SV_TREE_H

#include <stddef.h>
#include <stdint.h>

#include "spec_verify.h"

#ifdef __cplusplus
extern "C" {
#endif

#define SV_MAX_NODES 256    /* largest N */
#define SV_MAX_SLOTS 8192   /* largest number of slots (or forks) of one cache call */
#define SV_F16 2            /* sv_dtype of caches only: IEEE half */

/* Keys and values of a paged cache; k and v have the same layout. */
typedef struct {
    void *k, *v;            /* [layers][pages][page_size][heads][head_dim] by the strides below */
    int32_t layers, pages, page_size, heads, head_dim;
    int32_t dtype;          /* SV_F32, SV_BF16 or SV_F16 */
    int64_t layer_stride, page_stride, row_stride, head_stride;
} sv_cache;

/* ------------------------------------------------------------------------
 * Attention of the nodes over a paged cache (one layer).
 *
 *   row lens[b] + i of the cache  <-  k[b][i], v[b][i]          (i < counts[b])
 *   out[b][i][h] = sum_t p_t v_t,  p = softmax_t(scale q[b][i][h] . k_t)
 *
 * over t < lens[b] and t = lens[b] + a, a an ancestor of node i or i itself;
 * query head h reads key/value head h / (q_heads / heads).  Rows
 * i >= counts[b] of out are left as they are.  The cached keys and values of
 * rows t < lens[b] + counts[b] must be finite; rows past them may hold
 * anything.  Scores are held in 32 bits, which scale q.k log2(e) must not
 * overflow.
 *
 * Supported: SV_BF16 and SV_F16, head_dim 64 and 128, page_size 16, 32, 64
 * and 128, q_heads a multiple of heads with at most 64 query heads per key
 * head; q, k, v, out and the cache 16-byte aligned with strides that are
 * multiples of 8 elements.
 *
 * A request with lens[b] < 0, counts[b] outside [0, N], a parent that is not
 * in [0, i), more rows than max_pages pages hold, or a page id outside
 * [0, pages) among those it needs writes nothing to the cache, and its out
 * rows (i < counts[b], none if counts[b] is out of range) are NaN.  So are
 * the rows of a request whose data were lost to a device-side wait that ran
 * out.  Pages that requests share must hold rows before lens[b] only. */
typedef struct {
    int32_t B, N, q_heads, max_pages;
    int64_t table_stride;                       /* of page_table rows; 0 = max_pages */
    int64_t q_stride_b, q_stride_n, q_stride_h;
    int64_t k_stride_b, k_stride_n, k_stride_h; /* of the new keys */
    int64_t v_stride_b, v_stride_n, v_stride_h; /* of the new values */
    int64_t o_stride_b, o_stride_n, o_stride_h;
} sv_tree_attention_shape;

SV_API size_t sv_tree_attention_workspace_bytes(const sv_tree_attention_shape *shape, const sv_cache *cache);
SV_API sv_status sv_tree_attention(const sv_tree_attention_shape *shape, const sv_cache *cache, const void *q,
                                   const void *k, const void *v, const int32_t *page_table, const int32_t *lens,
                                   const int32_t *parents, const int32_t *counts, float scale, void *out,
                                   void *workspace, size_t workspace_bytes, void *stream);

/* ------------------------------------------------------------------------
 * Verification of the trees.
 *
 *   target_logits [B][N][row_stride]  row i: the target after node i
 *   draft_logits  [B][N][row_stride]  row i: the distribution q_i that node
 *                                     i's children were drawn from,
 *                                     independently; NULL = the drafter gave
 *                                     ids only (each child a point mass)
 *   tokens        [B][N]              node i's token (tokens[b][0] is not read)
 *   uniforms      [B][N] in [0, 1)    node i's test; slot 0 is the final draw
 *
 * From the root, the children of the current node are tried in index order;
 * the first one accepted becomes the current node, and a node none of whose
 * children is accepted ends the walk with one more token.  With
 * p = softmax(Z / T) at the current node:
 *   ids only: child c is accepted iff u_c R < p(x_c), R = 1 - the p of the
 *     distinct earlier siblings' tokens (a repeated token is never accepted);
 *     the last token is drawn from p without the children's tokens;
 *   draft logits: with (l, n) = (0, 1) before the first child, c is accepted
 *     iff u_c n q(x_c) < max(0, p(x_c) - l q(x_c)); each rejection sets
 *     l += n, n = sum_v max(0, p(v) - l q(v)); the last token is drawn from
 *     max(0, p - l q).  (This is the residual after r independent draws from
 *     q, each rejected by the rule of spec_verify.)
 *   greedy: the first child whose token is the argmax (lowest index on ties)
 *     of the target's row; the last token is that argmax.
 * The last token is the smallest t whose running weight sum exceeds u W (W:
 * all weight); no weight at all falls back to p.  A leaf draws from p.
 * Only rows of nodes on the accepted path are read.  Sums that a draw or a
 * residual is made of are held in 64 bits; an acceptance test is settled by
 * sums in 32 bits where it clears their error bound, else by sums in 64.  A
 * chain of k drafts follows the rule of spec_verify with its uniforms moved by
 * one slot; near ties spec_verify, whose sums are in 32 bits, may answer with a
 * neighbour.
 *
 *   out_accept_len [B]     accepted drafts j
 *   out_tokens     [B][N]  their tokens, the last token at index j, then -1
 *   out_path       [B][N]  0, the accepted nodes in order (j of them), then -1
 *
 * An idle slot gets 0, -1s and -1s.  A request with counts[b] outside [0, N],
 * a parent not in [0, i) or a token outside [0, V) gets -1 in all outputs.
 * Logits of -inf are tokens of no probability; a row without a finite logit,
 * NaN and +inf give unspecified (but in-bounds) results. */
typedef struct {
    int32_t B, N, V;
    int32_t dtype;      /* SV_F32 or SV_BF16 */
    int64_t row_stride; /* >= V; 0 = V */
} sv_tree_shape;

SV_API sv_status sv_tree_verify(const sv_tree_shape *shape, const void *target_logits, const void *draft_logits,
                                const int32_t *tokens, const int32_t *parents, const int32_t *counts,
                                const float *uniforms, double temperature, int32_t greedy, int32_t *out_accept_len,
                                int32_t *out_tokens, int32_t *out_path, void *stream);

/* ------------------------------------------------------------------------
 * Compaction to the accepted path (all layers of `cache` at once): with n the
 * number of leading entries >= 0 of path[b] (width entries per row), row
 * lens[b] + path[b][i] moves to row lens[b] + i for i < n, and
 * out_lens[b] = lens[b] + n.  out_lens must not overlap lens.  A request with
 * lens[b] < 0, a path that does not increase strictly, rows past max_pages
 * pages, or a page id outside [0, pages) among those it touches moves nothing
 * and gets out_lens[b] = -1. */
SV_API sv_status sv_cache_commit(const sv_cache *cache, const int32_t *page_table, int64_t table_stride,
                                 int32_t B, int32_t max_pages, const int32_t *lens, const int32_t *path,
                                 int64_t path_stride, int32_t width, int32_t *out_lens, void *stream);

/* Pages.  page_table[slot] lists a slot's pages in its leading entries, -1
 * behind them; refcount[page] counts the slots that list a page, 0 = free.
 *
 * Every slot comes to hold exactly ceil(lens[slot] / page_size) pages: first
 * all slots give back what they have too much (lens 0 frees the sequence),
 * then the missing pages are taken, free pages in increasing order of their
 * id, slots in order.  out_status[slot] = 0, or -1 (the slot unchanged) when
 * lens[slot] < 0, max_pages is too small, an entry is not in [-1, pages) or
 * pages follow a -1; or when the free pages do not suffice for the slot and
 * all before it that miss some.  out_status must not overlap lens. */
SV_API sv_status sv_cache_resize(int32_t *page_table, int64_t table_stride, int32_t slots, int32_t max_pages,
                                 const int32_t *lens, int32_t page_size, int32_t *refcount, int32_t pages,
                                 int32_t *out_status, void *stream);

/* Fork i makes slot dst[i] a copy of slot src[i]: what dst holds is given
 * back, the full pages of src are shared, the ragged last one (the
 * lens % page_size rows that it holds, in all layers) is copied to a page
 * taken as above, and lens[dst] = lens[src].  Pages past src's length (kept
 * for rows to come) are not taken over.  out_status[i] = 0, or -1 when src or dst is
 * not in [0, slots), dst is named twice or is also a src, src's length or
 * pages are not valid as above, or dst's entries are not (all unchanged); or
 * -2 when no free page is left for the ragged page (dst is left empty, its
 * length 0).  Rows of shared pages must not be written: a forked slot is
 * extended, not rewound below the length it was forked at.  lens, src (or
 * dst) and out_status must not overlap. */
SV_API sv_status sv_cache_fork(const sv_cache *cache, int32_t *page_table, int64_t table_stride, int32_t slots,
                               int32_t max_pages, int32_t *lens, int32_t *refcount, const int32_t *src,
                               const int32_t *dst, int32_t forks, int32_t *out_status, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* SV_TREE_H */
