/*
 * hlwq_attention.h — C ABI of libhlwq's serving operators: a paged KV cache of
 * HLWQ codes and the attention that reads it.
 *
 * One step of a generation loop over a batch of requests is
 *   hlwq_kv_page_plan        pages, slots and positions of the step's tokens;
 *   hlwq_kv_paged_attention  attention of the new tokens over pages, window and
 *                            themselves (hlwq_prompt_attention where nothing is
 *                            cached yet);
 *   hlwq_kv_paged_append     the new keys and values into the window, the tokens
 *                            they push out encoded into pages.
 * The cache is the streaming cache of hlwq_kv_append (include/hlwq.h) with its
 * packed part cut into pages: of a request that holds T tokens, tokens
 * t < T - n_residual are encoded, exactly as hlwq_kv_quantize encodes them, and
 * the newest min(T, n_residual) are kept in bf16 in a ring ("Qwopus3.6-27B-v2 ·
 * HLWQ Q5", "Methodology notes", KV bullet: H256, 8 centroids, 128-token
 * residual buffer).
 *
 * Ownership, execution, errors and overlap are those of include/hlwq.h: the
 * caller allocates every buffer in device memory of the current device, every
 * call validates its host arguments, enqueues on `hip_stream` and returns
 * without synchronising; nothing is enqueued on an error; calls on different
 * streams may run concurrently (each with a workspace of its own).  Lengths,
 * tables and slots are read on the device when the call runs, so a call can be
 * captured into a graph and replayed on new contents of the same buffers.
 *
 * Values in device arrays that name something out of range (a page id, a slot,
 * a request, a length) never make a call read or write outside the buffers it
 * was given: row ranges are cut to [0, rows), a prefix sum that falls makes the
 * attention do nothing, and what the others cause is stated at each call.
 *
 * Limits, past which a call gives HLWQ_ERR_LIMIT, beside those stated at each: 2^20
 * requests, sequences and table entries a request, 2^12 heads, a row stride of
 * 2^22 elements, and below 2^31 rows, rows * q_heads, ring slots a request and
 * n_pages * page_size.
 *
 * Layouts (row-major, contiguous unless a stride is given):
 *   packed u8   [n_pages][kv_heads][page_size][32 * bits]
 *   norms  fp16 [n_pages][kv_heads][page_size]
 *   window bf16 [requests][kv_heads][ring][256], token t in slot t mod ring;
 *               ring >= n_residual (a ring of n_residual + n slots keeps a step
 *               of up to n tokens off the slots it encodes, so that the step can
 *               be repeated)
 *   block_table i32 [requests][max_pages]: entry p of a request is the page of
 *               its encoded tokens [p * page_size, (p + 1) * page_size)
 *   rows        the step's new tokens of all requests, one after the other:
 *               request b owns rows cu_new[b] .. cu_new[b + 1] - 1, in order of
 *               position; rows from cu_new[requests] on belong to nobody and
 *               are neither read nor written
 *   lens        i32 [requests]: tokens of each request, the step's included;
 *               row i of request b stands at position
 *               lens[b] - (cu_new[b + 1] - cu_new[b]) + (i - cu_new[b])
 */
#ifndef HLWQ_ATTENTION_H
#define HLWQ_ATTENTION_H

#include "hlwq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Keys or values of a paged cache. */
typedef struct hlwq_kv_store {
  void* packed; /* u8   [n_pages][kv_heads][page_size][32 * bits], 16-byte aligned */
  void* norms;  /* fp16 [n_pages][kv_heads][page_size], 16-byte aligned */
  void* window; /* bf16 [requests][kv_heads][ring][256], 16-byte aligned; may be NULL when ring = 0 */
} hlwq_kv_store;

typedef struct hlwq_kv_cache {
  hlwq_kv_store k, v;
  int64_t n_pages;
  int64_t requests;   /* slots of the batch */
  int64_t kv_heads;
  int64_t page_size;  /* 16, 32, 64, 128 or 256; n_pages * page_size < 2^31 */
  int64_t n_residual; /* newest tokens kept in bf16 */
  int64_t ring;       /* window slots per request, at least n_residual */
  int head_dim;       /* 256 */
  int bits;           /* 3 or 2 */
} hlwq_kv_cache;

typedef struct hlwq_kv_plan {
  /* read */
  const int32_t* tokens;   /* [requests] tokens held before the step */
  const int32_t* n_new;    /* [requests] tokens of the step */
  const uint8_t* reset;    /* [requests], or NULL: nonzero where the slot's request has ended; its pages go
                              back on the stack first and the slot starts from no tokens */
  const int32_t* n_free;   /* [1] free pages before the step */
  /* read and written */
  int32_t* free_pages;     /* [n_pages] stack of free page ids, the top at n_free - 1 */
  int32_t* block_table;    /* [requests][max_pages] */
  /* written */
  int32_t* cu_new;         /* [requests + 1] prefix sum of n_new */
  int32_t* lens;           /* [requests] tokens after the step */
  int32_t* row_request;    /* [rows] request of each row, -1 past the last */
  int32_t* positions;      /* [rows] position of each row, -1 past the last */
  int32_t* slots;          /* [rows] page * page_size + offset of the token the row pushes out of the
                              window (position - n_residual), -1 if it pushes none */
  int32_t* n_free_after;   /* [1] */
  int32_t* status;         /* [1], see below */
  int64_t requests, rows, max_pages, n_pages, page_size, n_residual;
} hlwq_kv_plan;

/* Plan one step: from the requests' lengths, the pages they need, taken from
 * the stack and entered into the block table, and for every row its request,
 * its position and the slot of the token it pushes out of the window.  Pages
 * given back are pushed in order of (slot, page); pages are popped in order of
 * (request, page).  tokens, n_new and n_free are left as they are (lens and
 * n_free_after are the next step's), so the same step can be planned again
 * unless a reset slot takes pages in it.  A page may stand in several tables (a
 * common beginning read by several requests) once all its tokens are encoded: a
 * request's next tokens go on in its last page.  The plan keeps no count of that,
 * so only one of them may be reset.
 *
 * *status afterwards: 0; or the number of pages missing from the stack; or -1
 * where a device value is out of range (a negative length, more new tokens than
 * rows, a request longer than its table row, a free count or a given-back page
 * id outside the pool).  With a nonzero status the stack, the table and the
 * free count are left as they were, cu_new is all 0, lens = tokens and every
 * row is -1, so that the step's other calls do nothing.
 *
 * All buffers 4-byte aligned (reset: any); requests and max_pages at most
 * 2^20, rows below 2^31. */
int hlwq_kv_page_plan(const hlwq_kv_plan* plan, void* hip_stream);

/* Put the step's keys and values k_new, v_new (bf16 [rows][kv_heads][256],
 * consecutive rows k_stride / v_stride elements apart: a multiple of 8, at
 * least 256 * kv_heads, at most 2^22) into the cache: row i, at position t of its request,
 * pushes out token t - n_residual, whose codes and norm go to slots[i]; the new
 * tokens that stay among the newest n_residual go to their ring slots.
 * cu_new, lens, row_request and slots as hlwq_kv_page_plan wrote them.  Rows
 * whose request is out of range are passed over; a slot out of range stores
 * nothing.  HLWQ_ERR_LIMIT where rows * kv_heads passes 2^29 - 32. */
int hlwq_kv_paged_append(const hlwq_kv_cache* cache, const void* k_new_bf16, int64_t k_stride,
                         const void* v_new_bf16, int64_t v_stride, const int32_t* cu_new, const int32_t* lens,
                         const int32_t* row_request, const int32_t* slots, int64_t rows, void* hip_stream);

/* Attention of the step's rows, before its append: row i at position t of
 * request b attends to tokens 0 .. t of the request,
 *   out = sum_j p_j v_j,  p = softmax_j(scale q . k_j),
 * where with T = lens[b] - (its new tokens) tokens j < T - n_residual are read
 * from pages (the vector n16 / 256 * H256 c[codes], not rounded to bf16), those
 * below T from the window, and the rest from k_new, v_new.  Query head h reads
 * KV head h / (q_heads / kv_heads).  q and out bf16 [rows][q_heads][256], out
 * contiguous, q with a row stride as k_new's.  scale finite.
 *
 * The rotation is symmetric, q . (H c) = (H q) . c, so the codes are never
 * rotated back: q is rotated once, the sum over encoded tokens runs over
 * centroids in fp16 (2^-11 relative) and its fp32 result is rotated once.
 * Scores, softmax and sums are fp32; probabilities enter the products rounded
 * to 16 bits; the output is rounded once.  A row whose q . k, before the scale,
 * or score passes fp32's range is NaN.
 *
 * A token whose page id lies outside [0, n_pages), or past max_pages, is left
 * out of the sum.  lens[b] below the number of new tokens counts as equal to it.
 * Norms of encoded tokens must be finite and not negative; k_new, v_new and window may hold NaN
 * and infinities, which reach only rows that attend to them.
 *
 * Requests of few rows (rows times query heads of a KV head: up to 64, of a
 * single request 256) are worked on in tiles of 16 such rows of one KV head.
 * What the sizes say of their number T, whatever the lengths on the device: with
 * g = q_heads / kv_heads at most kv_heads * min(rows * g / 16 + requests, rows * g)
 * and, where rows * g passes 64 * requests (256 for a single one), at most
 * kv_heads * ceil(64 / 16) for each request (none for a single one or where g
 * passes 64).  HLWQ_ERR_LIMIT where T reaches 2^20, or T * max_pages * page_size
 * / 128 reaches 2^31.
 *
 * `workspace` holds partial sums: hlwq_kv_paged_attention_workspace bytes,
 * 16-byte aligned, contents immaterial before and after.  That is about 17 MB and
 * 33 KB for each of the T tiles (if there are any), and 135 MB more where rows * g
 * passes 64 * requests (256 for a single one).  Calls in turn on one stream may
 * share it. */
int hlwq_kv_paged_attention(const hlwq_kv_cache* cache, const void* q_bf16, int64_t q_stride, int64_t q_heads,
                            const void* k_new_bf16, int64_t k_stride, const void* v_new_bf16, int64_t v_stride,
                            const int32_t* cu_new, const int32_t* lens, const int32_t* block_table,
                            int64_t max_pages, int64_t rows, float scale, void* out_bf16, void* workspace,
                            size_t workspace_bytes, void* hip_stream);

/* Workspace of hlwq_kv_paged_attention for these sizes; 0 if they are invalid or
 * past its limits (2^20 requests, 2^12 query heads, rows * q_heads below 2^31, T
 * below 2^20), or there is nothing to do. */
size_t hlwq_kv_paged_attention_workspace(int64_t requests, int64_t rows, int64_t q_heads, int64_t kv_heads);

/* Causal attention over whole prompts packed one after the other: sequence b
 * owns rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1 of q, k, v and out, and row i
 * attends to the rows of its sequence up to itself.  q, out bf16
 * [rows][q_heads][256], k, v bf16 [rows][kv_heads][256], strides, heads, scale
 * and arithmetic as above (no token is encoded).  Rows from
 * cu_seqlens[sequences] on are neither read nor written.  NaN and infinities reach
 * only rows that attend to them.  HLWQ_ERR_LIMIT where kv_heads * min(rows * g /
 * 256 + sequences, rows * g), with g = q_heads / kv_heads, reaches 2^23. */
int hlwq_prompt_attention(const void* q_bf16, int64_t q_stride, const void* k_bf16, int64_t k_stride,
                          const void* v_bf16, int64_t v_stride, const int32_t* cu_seqlens, int64_t sequences,
                          int64_t rows, int64_t q_heads, int64_t kv_heads, int head_dim, float scale,
                          void* out_bf16, void* hip_stream);

#ifdef __cplusplus
}
#endif

#endif /* HLWQ_ATTENTION_H */
