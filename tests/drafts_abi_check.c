/* Plain C client of libhlwq's operators for drafted tokens and experts:
 * compiles against include/hlwq_drafts.h and include/hlwq_moe.h with a C
 * compiler and exercises the argument checks, size arithmetic, overlap checks
 * and workspace helpers (no kernel is launched, no address is read).  Exit
 * status 0 on success; prints the first failed check otherwise. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "hlwq_drafts.h"
#include "hlwq_moe.h"

#define CHECK(cond)                                                     \
  do {                                                                  \
    if (!(cond)) {                                                      \
      fprintf(stderr, "check failed: %s (line %d)\n", #cond, __LINE__); \
      return 1;                                                         \
    }                                                                   \
  } while (0)

/* addresses far apart */
static void* at(int k) { return (void*)(uintptr_t)(((uint64_t)1 << 32) + ((uint64_t)k << 40)); }

static hlwq_kv_cache cache(void) {
  hlwq_kv_cache c;
  c.k.packed = at(0);
  c.k.norms = at(1);
  c.k.window = at(2);
  c.v.packed = at(3);
  c.v.norms = at(4);
  c.v.window = at(5);
  c.n_pages = 8;
  c.requests = 2;
  c.kv_heads = 4;
  c.page_size = 64;
  c.n_residual = 128;
  c.ring = 128;
  c.head_dim = 256;
  c.bits = 3;
  return c;
}

static int tree(const hlwq_kv_cache* c, int64_t qs, int64_t heads, int64_t ks, void* parents, int64_t width, int64_t rows,
                float scale, void* out, size_t bytes) {
  return hlwq_kv_tree_attention(c, at(12), qs, heads, at(6), ks, at(7), ks, (const int32_t*)parents, (const int32_t*)at(8),
                                (const int32_t*)at(9), (const int32_t*)at(13), width, rows, scale, out, at(15), bytes, NULL);
}

static hlwq_drafts drafts(void) {
  hlwq_drafts d;
  d.tokens = (const int32_t*)at(0);
  d.parents = (const int32_t*)at(1);
  d.cu_rows = (const int32_t*)at(2);
  d.target = at(3);
  d.draft = at(4);
  d.uniforms = (const float*)at(5);
  d.next_uniforms = (const float*)at(6);
  d.n_kept = (int32_t*)at(7);
  d.next_token = (int32_t*)at(8);
  d.kept = (int32_t*)at(9);
  d.requests = 2;
  d.rows = 9;
  d.vocab = 1000;
  d.target_stride = 1000;
  d.draft_stride = 1000;
  d.dtype = HLWQ_F32;
  return d;
}

static hlwq_moe_banks banks(void) {
  hlwq_moe_banks b;
  b.gate_up_packed = at(0);
  b.gate_up_norms = at(1);
  b.down_packed = at(2);
  b.down_norms = at(3);
  b.experts = 16;
  b.hidden = 640;
  b.inner = 200;
  b.bits = 5;
  b.activation = HLWQ_ACT_SILU;
  return b;
}

static int layer(const hlwq_moe_banks* b, int64_t xs, int64_t tokens, int64_t k, void* out, size_t bytes) {
  return hlwq_moe_layer(b, at(4), xs, tokens, at(5), k, 1, (int32_t*)at(6), (float*)at(7), out, at(9), bytes, NULL);
}
static int experts(const hlwq_moe_banks* b, int64_t xs, int64_t tokens, int64_t k, void* out, size_t bytes) {
  return hlwq_moe_experts(b, at(4), xs, tokens, k, (const int32_t*)at(6), (const float*)at(7), out, at(9), bytes, NULL);
}

int main(void) {
  const int64_t big = INT64_MAX, small = INT64_MIN;
  const size_t all = (size_t)1 << 38;
  hlwq_kv_cache c = cache();
  hlwq_drafts d = drafts();
  hlwq_moe_banks b = banks();
  size_t need;

  /* attention of trees; out over the parents, sizes at and past the ends */
  need = hlwq_kv_tree_attention_workspace(2, 5, 24, 4);
  CHECK(need > 0);
  CHECK(tree(NULL, 6144, 24, 1024, at(16), 9, 5, 1.0f, at(14), all) == HLWQ_ERR_NULL);
  CHECK(tree(&c, 6144, 24, 1024, NULL, 9, 5, 1.0f, at(14), all) == HLWQ_ERR_NULL);
  CHECK(tree(&c, 6144, 24, 1024, at(16), 9, 5, 1.0f, at(16), need) == HLWQ_ERR_OVERLAP);
  CHECK(tree(&c, 6144, 24, 1024, at(16), 9, 5, 1.0f, at(16), need - 1) == HLWQ_ERR_SHAPE);
  CHECK(tree(&c, 6144, 24, 1024, (char*)at(16) + 2, 9, 5, 1.0f, at(14), all) == HLWQ_ERR_ALIGN);
  CHECK(tree(&c, 6144, 24, 1024, at(16), big, 5, 1.0f, at(14), all) == HLWQ_ERR_LIMIT);
  CHECK(tree(&c, 6144, 24, 1024, at(16), 9, big, 1.0f, at(14), all) == HLWQ_ERR_LIMIT);
  CHECK(tree(&c, 6144, big, 1024, at(16), 9, 5, 1.0f, at(14), all) != HLWQ_OK);
  CHECK(tree(&c, small, 24, 1024, at(16), 9, 5, 1.0f, at(14), all) == HLWQ_ERR_SHAPE);
  CHECK(tree(&c, 6144, 24, 1024, at(16), small, 5, 1.0f, at(14), all) == HLWQ_ERR_SHAPE);
  CHECK(tree(&c, 6144, 24, 1024, at(16), 9, 5, NAN, at(14), all) == HLWQ_ERR_SHAPE);
  /* tiles of 64 rows within their limits where those of sixteen are past theirs */
  CHECK(hlwq_kv_tree_attention_workspace(2, (1 << 20) - 1, 64, 4) == 0 ||
        hlwq_kv_tree_attention_workspace(2, (1 << 20) - 1, 64, 4) > ((size_t)1 << 34));
  CHECK(hlwq_kv_tree_attention_workspace(2, 1 << 20, 64, 4) == 0);
  CHECK(tree(&c, 16384, 64, 1024, at(16), 64, 1 << 20, 1.0f, at(14), (size_t)1 << 39) == HLWQ_ERR_LIMIT);
  CHECK(tree(&c, 16384, 64, 1024, at(16), 1 << 20, 1 << 18, 1.0f, at(14), (size_t)1 << 39) == HLWQ_ERR_LIMIT);
  CHECK(hlwq_kv_tree_attention_workspace(big, 5, 24, 4) == 0);
  CHECK(hlwq_kv_tree_attention_workspace(2, big, 24, 4) == 0);
  CHECK(hlwq_kv_tree_attention_workspace(2, 5, big, 1) == 0);
  CHECK(hlwq_kv_tree_attention_workspace(small, small, small, small) == 0);
  c.n_pages = big;
  CHECK(tree(&c, 6144, 24, 1024, at(16), 9, 5, 1.0f, at(14), all) == HLWQ_ERR_LIMIT);

  /* verification: each buffer, each output over each input */
  CHECK(hlwq_verify_drafts(NULL, NULL) == HLWQ_ERR_NULL);
  d.kept = (int32_t*)at(0);
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_OVERLAP);
  d = drafts();
  d.next_token = (int32_t*)at(7);
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_OVERLAP);
  d = drafts();
  d.n_kept = (int32_t*)((char*)at(4) + 4 * 8999);
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_OVERLAP);
  d = drafts();
  d.uniforms = NULL;
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_NULL);
  d = drafts();
  d.draft = (const char*)at(4) + 2;
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_ALIGN);
  d = drafts();
  d.rows = big;
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_LIMIT);
  d = drafts();
  d.requests = big;
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_LIMIT);
  d = drafts();
  d.vocab = d.target_stride = d.draft_stride = big;
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_LIMIT);
  d = drafts();
  d.target_stride = big;
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_LIMIT);
  d = drafts();
  d.rows = 0x7fffffff; /* rows of 2^40 elements: past the address space in a product of 64 bits */
  d.target_stride = d.draft_stride = (int64_t)1 << 40;
  d.kept = (int32_t*)at(0);
  CHECK(hlwq_verify_drafts(&d, NULL) != HLWQ_OK);
  d = drafts();
  d.rows = small;
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_SHAPE);
  d = drafts();
  d.vocab = small;
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_ERR_SHAPE);
  d = drafts();
  d.dtype = 3;
  CHECK(hlwq_verify_drafts(&d, NULL) != HLWQ_OK);
  memset(&d, 0, sizeof d);
  d.vocab = d.target_stride = 1;
  CHECK(hlwq_verify_drafts(&d, NULL) == HLWQ_OK);

  /* experts: every buffer, out over the codes' last byte, sizes at and past the ends */
  need = hlwq_moe_workspace(16, 640, 200, 7, 4);
  CHECK(need > 0);
  CHECK(layer(NULL, 640, 7, 4, at(8), all) == HLWQ_ERR_NULL);
  CHECK(experts(NULL, 640, 7, 4, at(8), all) == HLWQ_ERR_NULL);
  CHECK(layer(&b, 640, 7, 4, NULL, all) == HLWQ_ERR_NULL);
  CHECK(layer(&b, 640, 7, 4, at(8), need - 1) == HLWQ_ERR_SHAPE);
  CHECK(layer(&b, 640, 7, 4, at(6), need) == HLWQ_ERR_OVERLAP);
  CHECK(experts(&b, 640, 7, 4, (char*)at(0) + 16 * 400 * 5 * 80 - 2, need) == HLWQ_ERR_OVERLAP);
  CHECK(experts(&b, 640, 7, 4, (char*)at(3) + 16 * 640 * 2 * 2 - 2, need) == HLWQ_ERR_OVERLAP);
  CHECK(experts(&b, 640, 7, 4, (char*)at(9) + need - 2, need) == HLWQ_ERR_OVERLAP);
  CHECK(experts(&b, 640, 7, 4, (char*)at(8) + 1, need) == HLWQ_ERR_ALIGN);
  CHECK(layer(&b, 639, 7, 4, at(8), all) == HLWQ_ERR_SHAPE);
  CHECK(layer(&b, big, 7, 4, at(8), all) == HLWQ_ERR_LIMIT);
  CHECK(layer(&b, small, 7, 4, at(8), all) == HLWQ_ERR_SHAPE);
  CHECK(layer(&b, 640, big, 4, at(8), all) == HLWQ_ERR_LIMIT);
  CHECK(layer(&b, 640, small, 4, at(8), all) == HLWQ_ERR_SHAPE);
  CHECK(layer(&b, 640, 7, 17, at(8), all) == HLWQ_ERR_SHAPE);
  CHECK(experts(&b, 640, 7, 33, at(8), all) == HLWQ_ERR_LIMIT);
  CHECK(experts(&b, 640, 7, big, at(8), all) == HLWQ_ERR_LIMIT);
  CHECK(experts(&b, 640, 0, 4, NULL, 0) == HLWQ_OK);
  b.bits = 4;
  CHECK(layer(&b, 640, 7, 4, at(8), all) == HLWQ_ERR_BITS);
  b = banks();
  b.activation = 2;
  CHECK(layer(&b, 640, 7, 4, at(8), all) == HLWQ_ERR_SHAPE);
  b = banks();
  b.experts = big;
  CHECK(layer(&b, 640, 7, 4, at(8), all) == HLWQ_ERR_LIMIT);
  b = banks();
  b.hidden = big;
  CHECK(layer(&b, big, 7, 4, at(8), all) == HLWQ_ERR_LIMIT);
  b = banks();
  b.hidden = b.inner = 1 << 20; /* a matrix of more than 2^31 bytes */
  CHECK(layer(&b, 1 << 20, 7, 4, at(8), all) == HLWQ_ERR_LIMIT);
  b = banks();
  b.inner = small;
  CHECK(layer(&b, 640, 7, 4, at(8), all) == HLWQ_ERR_SHAPE);
  CHECK(hlwq_moe_workspace(big, 640, 200, 7, 4) == 0);
  CHECK(hlwq_moe_workspace(16, big, 200, 7, 4) == 0);
  CHECK(hlwq_moe_workspace(16, 640, big, 7, 4) == 0);
  CHECK(hlwq_moe_workspace(16, 640, 200, big, 4) == 0);
  CHECK(hlwq_moe_workspace(16, 640, 200, 7, big) == 0);
  CHECK(hlwq_moe_workspace(small, small, small, small, small) == 0);
  CHECK(hlwq_moe_workspace(1024, 1 << 20, 1 << 20, 1 << 23, 32) > 0);

  puts("drafts abi ok");
  return 0;
}
