/*
 * hlwq_moe.h — C ABI of libhlwq's mixture-of-experts layer for a few tokens,
 * computed straight from banks of HLWQ codes.
 *
 * The banks are what hlwq_quantize (include/hlwq.h) makes of an expert bank
 * [experts][out][in] ("Gemma-4-26B-A4B-it-HLWQ-Q5", "Technical Details":
 * gate_up and down banks, each expert quantized independently):
 *   gate_up  [experts][2 * inner][hidden], the first `inner` rows of an expert
 *            its gate, the others its up projection;
 *   down     [experts][hidden][inner];
 * packed u8 [experts][out][ceil(in / 128)][16 * bits] and norms fp16
 * [experts][out][ceil(in / 128)].  For token t with experts e_k and weights w_k
 *   y_t = sum_k w_k D_{e_k} (act(G_{e_k} x_t) * (U_{e_k} x_t)),
 * where a block of a matrix is n16 / 128 * H128 c[codes], not rounded to bf16.
 *
 * H is symmetric, so a block's product is n16 / 128 * c . (H x): activations are
 * rotated once, by blocks of 128, and the codes are never rotated back.  The
 * rotated activations and the centroids enter the products as fp16 (2^-11
 * relative; a row of activations is taken over a power of two of its own), sums
 * are fp32 and the output is rounded once.
 *
 * Ownership, execution, errors and overlap are those of include/hlwq.h: the
 * caller allocates every buffer in device memory of the current device, every
 * call validates its host arguments, enqueues on `hip_stream` and returns
 * without synchronising; nothing is enqueued on an error; calls on different
 * streams may run concurrently (each with a workspace of its own).  Nothing on
 * the device is read by the host, so a call can be captured into a graph.
 *
 * Made for decode steps.  Tokens are taken 4096 / top_k at a time, and an expert's
 * codes are gone through once for so many of its pairs (tokens that chose it) among
 * these: 16, or, where large banks are streamed, min(16, 192 / blocks of a row), 12
 * at 2048 values, 6 at 4096; for a handful of pairs in all once for each.
 */
#ifndef HLWQ_MOE_H
#define HLWQ_MOE_H

#include "hlwq.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  HLWQ_ACT_SILU = 0,     /* g / (1 + exp(-g)) */
  HLWQ_ACT_GELU_TANH = 1 /* g / 2 (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3))) */
};

typedef struct hlwq_moe_banks {
  const void* gate_up_packed; /* 4-byte aligned */
  const void* gate_up_norms;  /* 2-byte aligned */
  const void* down_packed;    /* 4-byte aligned */
  const void* down_norms;     /* 2-byte aligned */
  int64_t experts;            /* at most 1024 */
  int64_t hidden, inner;      /* each at most 2^20; an expert's matrix below 2^31 bytes of codes */
  int bits;                   /* 5 or 3 */
  int activation;             /* HLWQ_ACT_* */
} hlwq_moe_banks;

/* The experts of tokens whose routing is known: x bf16 [tokens][hidden], rows
 * x_stride elements apart (at least hidden, at most 2^20), experts i32 and weights fp32
 * [tokens][top_k], out bf16 [tokens][hidden].  top_k at most 32.  An expert
 * outside [0, banks->experts) adds nothing; one named twice adds twice.  NaN and
 * infinities in a token's row make only its own output NaN.
 *
 * `workspace`: hlwq_moe_workspace bytes, 16-byte aligned, contents immaterial
 * before and after.  x and out 2-byte aligned, experts and weights 4.
 * HLWQ_ERR_LIMIT: sizes past those stated, or more than 2^24 tokens. */
int hlwq_moe_experts(const hlwq_moe_banks* banks, const void* x_bf16, int64_t x_stride, int64_t tokens, int64_t top_k,
                     const int32_t* experts, const float* weights, void* out_bf16, void* workspace,
                     size_t workspace_bytes, void* hip_stream);

/* The whole layer: logits = router x with router bf16 [banks->experts][hidden],
 * summed in 64 bits in a fixed order; the top_k experts of each token (top_k at most
 * banks->experts) by falling logit, equal ones by rising index, NaN below all;
 * their weights softmax(logits), over all experts, or, with renormalize, over
 * the chosen ones; then as hlwq_moe_experts, which gets them in experts and
 * weights, written here. */
int hlwq_moe_layer(const hlwq_moe_banks* banks, const void* x_bf16, int64_t x_stride, int64_t tokens,
                   const void* router_bf16, int64_t top_k, int renormalize, int32_t* experts, float* weights,
                   void* out_bf16, void* workspace, size_t workspace_bytes, void* hip_stream);

/* Workspace of either call for these sizes; 0 if they are invalid or past the
 * limits, or there is nothing to do. */
size_t hlwq_moe_workspace(int64_t experts, int64_t hidden, int64_t inner, int64_t tokens, int64_t top_k);

#ifdef __cplusplus
}
#endif

#endif /* HLWQ_MOE_H */
