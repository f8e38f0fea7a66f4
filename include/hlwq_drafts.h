/*
 * hlwq_drafts.h — C ABI of libhlwq's operators for trees of drafted tokens over
 * the paged cache of include/hlwq_attention.h.
 *
 * A step of a generation loop that drafts tokens ahead gives each request a tree
 * of new rows: request b owns rows cu_rows[b] .. cu_rows[b + 1] - 1, its nodes 0,
 * 1, .. in that order.  Node 0 is the root, the last token the request is known
 * to have (not yet in the cache); parents[row] is the index, within its request,
 * of the node that the row's token follows, less than its own, or -1 where it
 * follows the cached tokens.  Any other value counts as -1.  The step is
 *   hlwq_kv_tree_attention  attention of the rows over the cache and their own
 *                           ancestors, once a layer;
 *   hlwq_verify_drafts      which rows the target model keeps, and the token that
 *                           follows them;
 *   hlwq_kv_page_plan and hlwq_kv_paged_append (include/hlwq_attention.h) put the
 *                           rows that were kept into the cache.
 *
 * Ownership, execution, errors and overlap are those of include/hlwq.h; lengths,
 * trees and probabilities are read on the device when the call runs, so a call
 * can be captured into a graph and replayed on new contents of the same buffers.
 * Values in device arrays that name something out of range never make a call
 * read or write outside the buffers it was given.
 */
#ifndef HLWQ_DRAFTS_H
#define HLWQ_DRAFTS_H

#include "hlwq_attention.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Attention of trees of rows: as hlwq_kv_paged_attention (whose arguments,
 * layouts, arithmetic and limits these are), but of the step's own rows a row
 * attends to itself and its ancestors alone; it attends to every token held
 * before the step.  parents i32 [rows], 4-byte aligned.  Positions are the
 * caller's: q and k_new come rotated for the depth of each node.  A request of
 * more than HLWQ_TREE_NODES rows is passed over, its rows left as they were.
 *
 * All requests are worked on in tiles of 16 query rows of one KV head: with
 * g = q_heads / kv_heads, T = kv_heads * min(rows * g / 16 + requests, rows * g).
 * HLWQ_ERR_LIMIT where T reaches 2^20, or T * max_pages * page_size / 128 reaches
 * 2^31.  `workspace`: hlwq_kv_tree_attention_workspace bytes, about 17 MB and 33
 * KB for each of the T tiles; where requests have 48 rows of a KV head and more on
 * average (tiles of 64 rows, if the table is wide as well), up to 34 MB, 132 KB for
 * each of those tiles and 516 bytes for each row and query head. */
enum { HLWQ_TREE_NODES = 8192 };
int hlwq_kv_tree_attention(const hlwq_kv_cache* cache, const void* q_bf16, int64_t q_stride, int64_t q_heads,
                           const void* k_new_bf16, int64_t k_stride, const void* v_new_bf16, int64_t v_stride,
                           const int32_t* parents, const int32_t* cu_rows, const int32_t* lens,
                           const int32_t* block_table, int64_t max_pages, int64_t rows, float scale, void* out_bf16,
                           void* workspace, size_t workspace_bytes, void* hip_stream);

/* Workspace of hlwq_kv_tree_attention for these sizes; 0 if they are invalid or
 * past its limits, or there is nothing to do. */
size_t hlwq_kv_tree_attention_workspace(int64_t requests, int64_t rows, int64_t q_heads, int64_t kv_heads);

/* Types of probabilities. */
enum { HLWQ_F32 = 0, HLWQ_BF16 = 1, HLWQ_F16 = 2 };

typedef struct hlwq_drafts {
  const int32_t* tokens;    /* [rows] */
  const int32_t* parents;   /* [rows] */
  const int32_t* cu_rows;   /* [requests + 1] */
  const void* target;       /* [rows][vocab]: row r is the target's distribution of the token after row r */
  const void* draft;        /* [rows][vocab], or NULL: row r is what the tokens of r's children were drawn from */
  const float* uniforms;    /* [rows] in [0, 1): row r's decides on its own token */
  const float* next_uniforms; /* [requests] in [0, 1): for the token that follows */
  int32_t* n_kept;          /* [requests], written: rows kept, the root among them; 0 for a request of no rows */
  int32_t* next_token;      /* [requests], written: -1 for a request of no rows or a row of p without mass */
  int32_t* kept;            /* [rows], written: kept[cu_rows[b] + j] is the row of request b's j-th kept node, -1 past
                               the last and in rows of no request (may be NULL where there are no requests) */
  int64_t requests, rows, vocab;
  int64_t target_stride, draft_stride; /* elements from row to row, at least vocab */
  int dtype;                /* of target and draft */
} hlwq_drafts;

/* Verify drafted tokens against the target's probabilities, so that what is
 * kept and the token that follows are distributed as the target's own samples.
 * From the root on, the children of the node reached are looked at in order of
 * index.  With p and q the node's rows of target and draft, after j of its
 * children were refused the residual is
 *   r_j = (p - s_j q)+ / W_j,  s_0 = 0, W_0 = 1,
 *   s_{j+1} = s_j + W_j, W_{j+1} = sum over the vocabulary of (p - s_{j+1} q)+
 * (the recursive rejection r_{j+1} = (r_j - q)+ / |(r_j - q)+|, without its
 * divisions; children are independent draws from q).  A child of token x and
 * uniform u is kept if u q(x) W_j < (p(x) - s_j q(x))+; the walk goes on from it.
 * Where no child is kept, the next token is the lowest i at which the running
 * sum of r_j passes next_uniform times its total; of p if r_j has no mass left.
 * Without `draft` a child's q is one at its token: W_{j+1} = W_j - p(x), and p(x)
 * counts as 0 from then on.
 *
 * p need not sum to one.  Probabilities below 0 and NaN, of target and draft,
 * count as 0.  A token outside [0, vocab) is passed over, as are a request's rows
 * from the 4096th on.  Sums and products are in 64 bits.  vocab from 1 to 2^24, at most
 * 2^20 requests, rows below 2^31, strides at most 2^40; target and draft aligned
 * to their type, the others to 4 bytes. */
int hlwq_verify_drafts(const hlwq_drafts* drafts, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* HLWQ_DRAFTS_H */
