/* Plain C client of libhlwq's serving operators: compiles against
 * include/hlwq_attention.h with a C compiler and exercises the argument checks,
 * size arithmetic, overlap checks and the workspace helper (no kernel is
 * launched, no address is read).  Exit status 0 on success; prints the first
 * failed check otherwise. */
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "hlwq_attention.h"

#define CHECK(cond)                                                     \
  do {                                                                  \
    if (!(cond)) {                                                      \
      fprintf(stderr, "check failed: %s (line %d)\n", #cond, __LINE__); \
      return 1;                                                         \
    }                                                                   \
  } while (0)

/* addresses far apart */
static void* at(int k) { return (void*)(uintptr_t)(((uint64_t)1 << 32) + ((uint64_t)k << 36)); }

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

static int append(const hlwq_kv_cache* c, void* k, int64_t ks, int64_t vs, void* slots, int64_t rows) {
  return hlwq_kv_paged_append(c, k, ks, at(7), vs, (const int32_t*)at(8), (const int32_t*)at(9), (const int32_t*)at(10),
                              (const int32_t*)slots, rows, NULL);
}

static int attention(const hlwq_kv_cache* c, int64_t qs, int64_t heads, int64_t ks, int64_t width, int64_t rows, float scale,
                     void* out, size_t bytes) {
  return hlwq_kv_paged_attention(c, at(12), qs, heads, at(6), ks, at(7), ks, (const int32_t*)at(8), (const int32_t*)at(9),
                                 (const int32_t*)at(13), width, rows, scale, out, at(15), bytes, NULL);
}

static int prompt(int64_t qs, int64_t ks, int64_t sequences, int64_t rows, int64_t q_heads, int64_t kv_heads, float scale,
                  void* out) {
  return hlwq_prompt_attention(at(0), qs, at(1), ks, at(2), ks, (const int32_t*)at(3), sequences, rows, q_heads, kv_heads,
                               256, scale, out, NULL);
}

static hlwq_kv_plan plan(void) {
  hlwq_kv_plan p;
  p.tokens = (const int32_t*)at(0);
  p.n_new = (const int32_t*)at(1);
  p.reset = (const uint8_t*)at(2);
  p.n_free = (const int32_t*)at(3);
  p.free_pages = (int32_t*)at(4);
  p.block_table = (int32_t*)at(5);
  p.cu_new = (int32_t*)at(6);
  p.lens = (int32_t*)at(7);
  p.row_request = (int32_t*)at(8);
  p.positions = (int32_t*)at(9);
  p.slots = (int32_t*)at(10);
  p.n_free_after = (int32_t*)at(11);
  p.status = (int32_t*)at(12);
  p.requests = 3;
  p.rows = 7;
  p.max_pages = 5;
  p.n_pages = 11;
  p.page_size = 64;
  p.n_residual = 128;
  return p;
}

int main(void) {
  hlwq_kv_cache c = cache();
  hlwq_kv_plan p = plan();
  size_t need;
  const int64_t big = INT64_MAX;

  /* plan: every buffer named, the last of them written over the first; sizes at and past the ends */
  CHECK(hlwq_kv_page_plan(NULL, NULL) == HLWQ_ERR_NULL);
  p.status = (int32_t*)at(0);
  CHECK(hlwq_kv_page_plan(&p, NULL) == HLWQ_ERR_OVERLAP);
  p.requests = (int64_t)1 << 20;
  p.max_pages = (int64_t)1 << 20;
  p.rows = 0x7fffffff;
  p.n_pages = 0x7fffffff / 64;
  p.n_residual = big;
  CHECK(hlwq_kv_page_plan(&p, NULL) == HLWQ_ERR_OVERLAP);
  p.max_pages = big;
  CHECK(hlwq_kv_page_plan(&p, NULL) == HLWQ_ERR_LIMIT);
  p = plan();
  p.rows = big;
  CHECK(hlwq_kv_page_plan(&p, NULL) == HLWQ_ERR_LIMIT);
  p = plan();
  p.requests = INT64_MIN;
  CHECK(hlwq_kv_page_plan(&p, NULL) == HLWQ_ERR_SHAPE);
  p = plan();
  p.page_size = INT64_MIN;
  CHECK(hlwq_kv_page_plan(&p, NULL) == HLWQ_ERR_SHAPE);
  p = plan();
  p.n_free = NULL;
  CHECK(hlwq_kv_page_plan(&p, NULL) == HLWQ_ERR_NULL);

  /* append */
  CHECK(append(NULL, at(6), 1024, 1024, at(11), 5) == HLWQ_ERR_NULL);
  CHECK(append(&c, at(6), 1024, 1024, at(5), 5) == HLWQ_ERR_OVERLAP);
  CHECK(append(&c, at(6), big, 1024, at(11), 5) == HLWQ_ERR_SHAPE); /* not a multiple of 8 */
  CHECK(append(&c, at(6), big - 7, 1024, at(11), 5) == HLWQ_ERR_LIMIT);
  CHECK(append(&c, at(6), INT64_MIN, 1024, at(11), 5) == HLWQ_ERR_SHAPE);
  CHECK(append(&c, at(6), 1024, 1024, at(11), big) == HLWQ_ERR_LIMIT);
  CHECK(append(&c, at(6), 1024, 1024, at(11), INT64_MIN) == HLWQ_ERR_SHAPE);
  CHECK(append(&c, (char*)at(6) + 8, 1024, 1024, at(11), 5) == HLWQ_ERR_ALIGN);
  CHECK(append(&c, at(6), 1 << 22, 1 << 22, at(11), 0x7fffffff / 4) == HLWQ_ERR_LIMIT);
  CHECK(append(&c, at(6), 1 << 22, 1 << 22, at(5), (1 << 27) - 8) == HLWQ_ERR_OVERLAP); /* rows of 2^50 bytes */
  CHECK(append(&c, NULL, 0, 0, NULL, 0) == HLWQ_OK);

  /* caches whose byte counts pass int64 or the address space */
  c.requests = 1 << 20;
  c.kv_heads = 1 << 12;
  c.ring = 0x7fffffff;
  CHECK(append(&c, at(6), 1 << 20, 1 << 20, at(11), 5) == HLWQ_ERR_SHAPE);
  c.ring = 1 << 20;
  c.n_pages = 0x7fffffff / 64;
  CHECK(append(&c, at(6), 1 << 20, 1 << 20, at(11), 5) == HLWQ_ERR_OVERLAP);
  c = cache();
  c.n_pages = big;
  CHECK(append(&c, at(6), 1024, 1024, at(11), 5) == HLWQ_ERR_LIMIT);
  c = cache();
  c.kv_heads = big;
  CHECK(attention(&c, 1024, 4, 1024, 9, 5, 1.0f, at(14), 0) == HLWQ_ERR_LIMIT);
  c = cache();
  c.ring = big;
  c.n_residual = big;
  CHECK(attention(&c, 1024, 4, 1024, 9, 5, 1.0f, at(14), 0) == HLWQ_ERR_LIMIT);
  c = cache();

  /* attention: all its buffers, out over the cache's last window */
  need = hlwq_kv_paged_attention_workspace(2, 5, 24, 4);
  CHECK(need > 0);
  CHECK(attention(&c, 6144, 24, 1024, 9, 5, 0.0625f, at(5), need) == HLWQ_ERR_OVERLAP);
  CHECK(attention(&c, 6144, 24, 1024, 9, 5, 0.0625f, at(14), need - 1) == HLWQ_ERR_SHAPE);
  CHECK(attention(&c, 6144, 24, 1024, 9, 5, NAN, at(14), need) == HLWQ_ERR_SHAPE);
  CHECK(attention(&c, 6144, 24, 1024, big, 5, 0.0625f, at(14), need) == HLWQ_ERR_LIMIT);
  CHECK(attention(&c, 6144, 24, 1024, 9, big, 0.0625f, at(14), need) == HLWQ_ERR_LIMIT);
  CHECK(attention(&c, 6144, big, 1024, 9, 5, 0.0625f, at(14), need) == HLWQ_ERR_SHAPE); /* not a multiple of 4 */
  CHECK(attention(&c, 6144, big - 3, 1024, 9, 5, 0.0625f, at(14), need) == HLWQ_ERR_LIMIT);
  CHECK(attention(&c, big, 24, 1024, 9, 5, 0.0625f, at(14), need) == HLWQ_ERR_SHAPE);
  CHECK(attention(&c, 1 << 22, 24, 1 << 22, 1 << 20, 0x7fffffff / 24, 0.0625f, at(14), SIZE_MAX) == HLWQ_ERR_OVERLAP);
  CHECK(attention(&c, 6144, 24, 1024, 9, 0, 0.0625f, NULL, 0) == HLWQ_OK);

  /* the workspace helper takes anything */
  CHECK(hlwq_kv_paged_attention_workspace(big, big, big, big) == 0);
  CHECK(hlwq_kv_paged_attention_workspace(INT64_MIN, INT64_MIN, INT64_MIN, INT64_MIN) == 0);
  CHECK(hlwq_kv_paged_attention_workspace(1, big, 4096, 1) == 0);
  CHECK(hlwq_kv_paged_attention_workspace(1 << 20, 0x7fffffff / 4096, 4096, 1) > 0);
  CHECK(hlwq_kv_paged_attention_workspace(1 << 20, 0x7fffffff / 4096, 4096, 4096) == 0);
  CHECK(hlwq_kv_paged_attention_workspace(1, 0x7fffffff, 1, 1) > 0);

  /* prompts */
  CHECK(prompt(6144, 1024, 2, 5, 24, 4, 0.0625f, at(0)) == HLWQ_ERR_OVERLAP);
  CHECK(prompt(6144, 1024, big, 5, 24, 4, 0.0625f, at(4)) == HLWQ_ERR_LIMIT);
  CHECK(prompt(6144, 1024, 2, big, 24, 4, 0.0625f, at(4)) == HLWQ_ERR_LIMIT);
  CHECK(prompt(big - 7, 1024, 2, 5, 24, 4, 0.0625f, at(4)) == HLWQ_ERR_LIMIT);
  CHECK(prompt(6144, 1024, 2, 5, 24, big, 0.0625f, at(4)) == HLWQ_ERR_SHAPE);
  CHECK(prompt(6144, 1024, 2, 5, 24, 4, INFINITY, at(4)) == HLWQ_ERR_SHAPE);
  CHECK(prompt(1 << 20, 1 << 20, 1 << 20, 0x7fffffff / 4096, 4096, 4096, 1.0f, at(4)) == HLWQ_ERR_OVERLAP);
  CHECK(prompt(0, 0, 0, 0, 0, 0, 1.0f, NULL) == HLWQ_OK);

  printf("serving abi ok\n");
  return 0;
}
