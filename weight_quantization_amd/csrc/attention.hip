// attention.hip — attention over the paged cache of HLWQ codes and over whole
// prompts (include/hlwq_attention.h).

#include "attention_chunk.h"

#include <cmath>

namespace hlwq_kv {
namespace {

// Heads and rows of an attention call.  *nothing: valid, with no work.
int check_heads(int64_t rows, int64_t q_heads, int64_t kv_heads, bool* nothing) {
  if (rows < 0 || q_heads < 0 || kv_heads < 0) return HLWQ_ERR_SHAPE;
  *nothing = rows == 0 || q_heads == 0;
  if (*nothing) return HLWQ_OK;
  if (kv_heads == 0 || q_heads % kv_heads) return HLWQ_ERR_SHAPE;
  // (out alone would pass the memory there is)
  if (q_heads > kMaxHeads || rows > 0x7fffffff / q_heads) return HLWQ_ERR_LIMIT;
  return HLWQ_OK;
}

// Tiles of m rows of a call: at most one more per request than whole ones,
// every tile holding a row.
int64_t tiles_of(int64_t requests, int64_t rows, int64_t group, int64_t kv_heads, int64_t m) {
  return std::min(rows * group / m + requests, rows * group) * kv_heads;
}

int64_t prompt_groups(const AttnArgs& a, int64_t tile) {
  return tiles_of(a.requests, a.rows, a.group, a.kv_heads, tile);
}

// Tiles of 256 rows read K and V half as often as tiles of 128, but need twice
// the rows to fill the device's 256 CUs; and where not even two tiles of 128
// meet on a CU, what a tile waits for counts, so eight waves split its keys.
// Measured (24 query heads on 4, one sequence, us):
//   tokens                100    517    900   1500   2500   4000   8000  16384
//   256 rows               19     36     52     79    124    214    731   2930
//   128 rows               13     29     43     71    117    210    727   3023
//   128 rows, keys halved  16     26     37     55    106    235    767
// Four sequences of 1500 (568 tiles of 256 rows): 140, 130 and 165; nine of 1 to
// 2500 on 2 KV heads (720 tiles): 196 and 207.  The lengths are on the device,
// so the host goes by their mean.
int launch_prompt(const AttnArgs& a, hipStream_t stream) {
  const int64_t wide = prompt_groups(a, 256), narrow = prompt_groups(a, 128);
  const bool halved = narrow <= 512 && a.rows >= int64_t{384} * a.requests;
  const int64_t groups = wide >= 640 ? wide : narrow;
  if (groups > 0x7fffff) return HLWQ_ERR_LIMIT;
  const dim3 grid(static_cast<uint32_t>(groups));
  if (wide >= 640) return launch(hlwq_prompt_attention_kernel<8, 64, 1>, grid, dim3(512), stream, a);
  if (halved) return launch(hlwq_prompt_attention_kernel<8, 64, 2>, grid, dim3(512), stream, a);
  return launch(hlwq_prompt_attention_kernel<4, 32, 1>, grid, dim3(256), stream, a);
}

// How a paged call is shared among the kernels: requests of few query rows to a
// KV head go to the split kernel, the others to the chunk kernel, which unpacks
// each code once for 256 rows but takes 40 us however little it has to do.  The
// lengths are on the device, so the host goes by the mean: where it is few rows
// the split kernel takes every request; else both are called, except for a
// single request.  Measured, split and chunk kernel (24 query heads on 4, 3
// bits, us):
//   one request over 16000 tokens, 36 rows     33   76;  120 rows   48   84;
//                                  240 rows    70  100;  480 rows  112  112
//   8 requests over 4000 tokens, 36 rows each  44   59;   60 rows   50   61;
//                                  120 rows    79   67;  240 rows  128   91
//   32 requests over 1000 tokens, 60 rows      67   70;  240 rows  224  106
// The mean misses one chunk among many slots, which then is the split kernel's
// alone: 512 tokens over 16000 beside 63 single tokens over 4000 take 673 us (312
// and 80 by themselves; 1024 tokens, where both kernels are called, 587), 300
// over 4000 in one of 32 slots 121 (105 alone).
constexpr int64_t few_rows(int64_t requests) { return requests == 1 ? 256 : 64; }
// Workgroups that the device holds at once: two to a CU of the split kernel
// (256 registers a work-item), one of the chunk kernel.
constexpr int64_t kSplitResident = 512, kChunkWorkers = 256;
struct PagedPlan {
  bool split, chunk;      // which kernels are called
  int64_t split_tiles, split_workers;
  int64_t split_slots;    // of partial sums
  size_t split_bytes, chunk_bytes;  // of workspace, each its own
};
PagedPlan paged_plan(int64_t requests, int64_t rows, int64_t q_heads, int64_t kv_heads) {
  PagedPlan p{};
  const int64_t group = q_heads / kv_heads;
  const int64_t few = few_rows(requests);
  p.chunk = rows * group > few * requests;
  p.split_tiles = tiles_of(requests, rows, group, kv_heads, kSplitRows);
  // Beside the chunk kernel the split kernel takes requests of whole tokens, at
  // most `few` rows, whatever the call's rows are.
  if (p.chunk)
    p.split_tiles = requests > 1 ? std::min(p.split_tiles, std::min(requests, rows) * ceil_div(few / group * group, kSplitRows) * kv_heads) : 0;
  p.split = p.split_tiles > 0;
  if (p.split) {
    // The workgroups of the tiles' windows come after the pages' and end early.
    // Where they are few all fit the device at once; where they are more, places
    // kept free for them would stand empty most of the time, and it is better
    // that they follow the first pages' workgroups.  Measured (4 KV heads, 3
    // bits, 4000 tokens a request, us), with places kept and without: 4 requests
    // 19.8 and 22.5, 8 26.4 and 25.3, 16 35.8 and 33.6, 64 87 and 74, 128 183
    // and 154.
    p.split_workers = kSplitResident - (p.split_tiles < kSplitResident / 16 ? p.split_tiles : 0);
    p.split_slots = 2 * (p.split_workers + p.split_tiles);
    p.split_bytes = partial_floats(p.split_slots, kSplitRows) * sizeof(float);
  }
  p.chunk_bytes = p.chunk ? partial_floats(2 * kChunkWorkers, kChunkRows) * sizeof(float) : 0;
  return p;
}

// Tiles of the split kernel's launches: sixteen workgroups of 256 to a tile in
// its join, 2^32 - 1 work-items to a launch.
constexpr int64_t kMaxSplitTiles = 0xffffff / kSplitRows;

size_t workspace_bytes_of(int64_t requests, int64_t rows, int64_t q_heads, int64_t kv_heads) {
  bool nothing;
  if (requests <= 0 || requests > kMaxRequests || check_heads(rows, q_heads, kv_heads, &nothing) != HLWQ_OK || nothing) return 0;
  const PagedPlan p = paged_plan(requests, rows, q_heads, kv_heads);
  return p.split_tiles > kMaxSplitTiles ? 0 : p.split_bytes + p.chunk_bytes;
}

template <int BITS>
int launch_split(const AttnArgs& a, int64_t tiles, hipStream_t stream) {
  const int st = launch(hlwq_split_attention_kernel<BITS>, dim3(static_cast<uint32_t>(a.workers + tiles)), dim3(kSplitThreads), stream, a);
  if (st != HLWQ_OK) return st;
  return launch(hlwq_split_join_kernel, dim3(static_cast<uint32_t>(tiles * kSplitRows)), dim3(kSplitThreads), stream, a);
}

// The shift that keeps the sum of the costs of tiles of m rows and blocks of kt
// tokens below 2^31 (Work): 0 unless millions of tiles meet millions of tokens.
int32_t cost_shift_of(const AttnArgs& a, int64_t m, int64_t kt) {
  const int64_t rows = static_cast<int64_t>(a.rows) * a.group;
  const double tiles = static_cast<double>(std::min(rows / m + a.requests, rows)) * a.kv_heads;
  const double blocks = (static_cast<double>(static_cast<int64_t>(a.width) << a.page_shift) + a.n_res + a.rows) / kt + 4;
  const double grow = (kBlockCost * m / kt / a.group + 1.0) * (rows / m + 1);
  if (tiles * (blocks * kBlockCost + grow) < 0x1p30) return 0;
  int32_t shift = 1;
  while (tiles * (blocks / (1 << shift) + 2) > 0x1p30 && shift < 30) ++shift;
  return shift;
}

// (run_paged has refused what passes the launches' sizes)
int launch_paged(int bits, AttnArgs a, const PagedPlan& p, void* ws, hipStream_t stream) {
  a.most = 0x7fffffff;
  const int32_t few = static_cast<int32_t>(few_rows(a.requests));
  if (p.split) {
    a.partial = static_cast<float*>(ws);
    a.workers = static_cast<int32_t>(p.split_workers);
    a.slots = static_cast<int32_t>(p.split_slots);
    a.least = 1;
    if (p.chunk) a.most = few;
    const int st = bits == 3 ? launch_split<3>(a, p.split_tiles, stream) : launch_split<2>(a, p.split_tiles, stream);
    if (st != HLWQ_OK || !p.chunk) return st;
    a.most = 0x7fffffff;
  }
  a.partial = reinterpret_cast<float*>(static_cast<char*>(ws) + p.split_bytes);
  a.workers = kChunkWorkers;
  a.slots = 2 * kChunkWorkers;
  a.cost_shift = cost_shift_of(a, kChunkRows, kChunkBlock);
  a.least = p.split ? few + 1 : 1;
  const int st = launch(bits == 3 ? hlwq_chunk_attention_kernel<3> : hlwq_chunk_attention_kernel<2>,
                        dim3(static_cast<uint32_t>(a.workers)), dim3(512), stream, a);
  if (st != HLWQ_OK) return st;
  // up to 2^29 workgroups: rows * q_heads below 2^31, more than 64 rows a request
  const int64_t groups = tiles_of(a.requests, a.rows, a.group, a.kv_heads, kChunkRows) * (kChunkRows / kChunkJoinRows);
  const dim3 grid(static_cast<uint32_t>(std::min(groups, kChunkJoinWide)), static_cast<uint32_t>(ceil_div(groups, kChunkJoinWide)));
  return launch(hlwq_chunk_join_kernel, grid, dim3(256), stream, a);
}

int run_paged(const hlwq_kv_cache* c, const void* q, int64_t q_stride, int64_t q_heads, const void* k, int64_t k_stride,
              const void* v, int64_t v_stride, const int32_t* cu, const int32_t* lens, const int32_t* table,
              int64_t max_pages, int64_t rows, float scale, void* out, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!c) return HLWQ_ERR_NULL;
  Spans spans;
  int st = check_cache(*c, false, spans);
  if (st != HLWQ_OK) return st;
  bool nothing;
  if ((st = check_heads(rows, q_heads, c->kv_heads, &nothing)) != HLWQ_OK) return st;
  if (max_pages < 0 || !std::isfinite(scale)) return HLWQ_ERR_SHAPE;
  if (max_pages > kMaxTable) return HLWQ_ERR_LIMIT;
  if (nothing || c->requests == 0) return HLWQ_OK;
  int64_t qe, ke, ve;
  if ((st = check_rows(q, q_stride, rows, q_heads, &qe)) != HLWQ_OK ||
      (st = check_rows(k, k_stride, rows, c->kv_heads, &ke)) != HLWQ_OK ||
      (st = check_rows(v, v_stride, rows, c->kv_heads, &ve)) != HLWQ_OK)
    return st;
  const PagedPlan plan = paged_plan(c->requests, rows, q_heads, c->kv_heads);
  // (the split kernel counts its tiles' blocks in 32 bits)
  if (plan.split_tiles > kMaxSplitTiles || plan.split_tiles * ceil_div(max_pages * c->page_size, kSplitBlock) > 0x7fffffff)
    return HLWQ_ERR_LIMIT;
  const size_t need = plan.split_bytes + plan.chunk_bytes;
  if (!cu || !lens || !out || !ws || (max_pages > 0 && !table)) return HLWQ_ERR_NULL;
  if (ws_bytes < need) return HLWQ_ERR_SHAPE;
  if (misaligned(cu, 4) || misaligned(lens, 4) || misaligned(table, 4) || misaligned(out, 16) || misaligned(ws, 16))
    return HLWQ_ERR_ALIGN;
  add_span(spans, q, qe, 2, false);
  add_span(spans, k, ke, 2, false);
  add_span(spans, v, ve, 2, false);
  add_span(spans, cu, c->requests + 1, 4, false);
  add_span(spans, lens, c->requests, 4, false);
  add_span(spans, table, c->requests * max_pages, 4, false);
  add_span(spans, out, rows * q_heads, 2 * kDim, true);
  add_span(spans, ws, static_cast<int64_t>(need), 1, true);
  if (check_disjoint(spans) != HLWQ_OK) return HLWQ_ERR_OVERLAP;
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.k_new = static_cast<const uint16_t*>(k);
  a.v_new = static_cast<const uint16_t*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.k_packed = static_cast<const uint8_t*>(c->k.packed);
  a.v_packed = static_cast<const uint8_t*>(c->v.packed);
  a.k_norms = static_cast<const uint16_t*>(c->k.norms);
  a.v_norms = static_cast<const uint16_t*>(c->v.norms);
  a.k_window = static_cast<const uint16_t*>(c->k.window);
  a.v_window = static_cast<const uint16_t*>(c->v.window);
  a.cu = cu;
  a.lens = lens;
  a.table = table;
  a.out = static_cast<uint16_t*>(out);
  a.n_res = c->n_residual;
  a.ring = c->ring;
  a.width = static_cast<int32_t>(max_pages);
  a.requests = static_cast<int32_t>(c->requests);
  a.rows = static_cast<int32_t>(rows);
  a.q_heads = static_cast<int32_t>(q_heads);
  a.kv_heads = static_cast<int32_t>(c->kv_heads);
  a.group = static_cast<int32_t>(q_heads / c->kv_heads);
  a.n_pages = static_cast<int32_t>(c->n_pages);
  a.page_shift = __builtin_ctzll(static_cast<uint64_t>(c->page_size));
  a.scale = scale;
  a.factor = std::fmax(std::fabs(scale) * kLog2e, __FLT_DENORM_MIN__);
  return launch_paged(c->bits, a, plan, ws, stream);
}

int run_prompt(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
               const int32_t* cu, int64_t sequences, int64_t rows, int64_t q_heads, int64_t kv_heads, int head_dim,
               float scale, void* out, hipStream_t stream) {
  if (head_dim != kDim) return HLWQ_ERR_BLOCK;
  bool nothing;
  int st = check_heads(rows, q_heads, kv_heads, &nothing);
  if (st != HLWQ_OK) return st;
  if (sequences < 0 || !std::isfinite(scale)) return HLWQ_ERR_SHAPE;
  if (sequences > kMaxRequests) return HLWQ_ERR_LIMIT;
  if (nothing || sequences == 0) return HLWQ_OK;
  int64_t qe, ke, ve;
  if ((st = check_rows(q, q_stride, rows, q_heads, &qe)) != HLWQ_OK ||
      (st = check_rows(k, k_stride, rows, kv_heads, &ke)) != HLWQ_OK ||
      (st = check_rows(v, v_stride, rows, kv_heads, &ve)) != HLWQ_OK)
    return st;
  if (!cu || !out) return HLWQ_ERR_NULL;
  if (misaligned(cu, 4) || misaligned(out, 16)) return HLWQ_ERR_ALIGN;
  Spans spans;
  add_span(spans, q, qe, 2, false);
  add_span(spans, k, ke, 2, false);
  add_span(spans, v, ve, 2, false);
  add_span(spans, cu, sequences + 1, 4, false);
  add_span(spans, out, rows * q_heads, 2 * kDim, true);
  if (check_disjoint(spans) != HLWQ_OK) return HLWQ_ERR_OVERLAP;
  AttnArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.q_stride = q_stride;
  a.k_new = static_cast<const uint16_t*>(k);
  a.v_new = static_cast<const uint16_t*>(v);
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.cu = cu;
  a.out = static_cast<uint16_t*>(out);
  a.requests = static_cast<int32_t>(sequences);
  a.rows = static_cast<int32_t>(rows);
  a.q_heads = static_cast<int32_t>(q_heads);
  a.kv_heads = static_cast<int32_t>(kv_heads);
  a.group = static_cast<int32_t>(q_heads / kv_heads);
  a.scale = scale;
  a.factor = std::fmax(std::fabs(scale) * kLog2e, __FLT_DENORM_MIN__);
  return launch_prompt(a, stream);
}

}  // namespace
}  // namespace hlwq_kv

extern "C" {

int hlwq_kv_paged_attention(const hlwq_kv_cache* cache, const void* q_bf16, int64_t q_stride, int64_t q_heads,
                            const void* k_new_bf16, int64_t k_stride, const void* v_new_bf16, int64_t v_stride,
                            const int32_t* cu_new, const int32_t* lens, const int32_t* block_table,
                            int64_t max_pages, int64_t rows, float scale, void* out_bf16, void* workspace,
                            size_t workspace_bytes, void* hip_stream) {
  return hlwq_kv::run_paged(cache, q_bf16, q_stride, q_heads, k_new_bf16, k_stride, v_new_bf16, v_stride, cu_new, lens,
                            block_table, max_pages, rows, scale, out_bf16, workspace, workspace_bytes,
                            static_cast<hipStream_t>(hip_stream));
}

size_t hlwq_kv_paged_attention_workspace(int64_t requests, int64_t rows, int64_t q_heads, int64_t kv_heads) {
  return hlwq_kv::workspace_bytes_of(requests, rows, q_heads, kv_heads);
}

int hlwq_prompt_attention(const void* q_bf16, int64_t q_stride, const void* k_bf16, int64_t k_stride,
                          const void* v_bf16, int64_t v_stride, const int32_t* cu_seqlens, int64_t sequences,
                          int64_t rows, int64_t q_heads, int64_t kv_heads, int head_dim, float scale, void* out_bf16,
                          void* hip_stream) {
  return hlwq_kv::run_prompt(q_bf16, q_stride, k_bf16, k_stride, v_bf16, v_stride, cu_seqlens, sequences, rows, q_heads,
                             kv_heads, head_dim, scale, out_bf16, static_cast<hipStream_t>(hip_stream));
}

}  // extern "C"
