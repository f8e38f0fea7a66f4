// attention.hip — attention over the paged cache of HLWQ codes and over whole
// prompts (include/hlwq_attention.h).

#include "attention_tile.h"

#include <cmath>

namespace hlwq_kv {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float wave_sum(float s) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) s += lane_xor(s, d);
  return s;
}

__device__ __forceinline__ void load4(const uint16_t* p, int lane, float (&x)[4]) {
  const uint2 w = *reinterpret_cast<const uint2*>(p + 4 * lane);
  x[0] = bf16_lo(w.x);
  x[1] = bf16_hi(w.x);
  x[2] = bf16_lo(w.y);
  x[3] = bf16_hi(w.y);
}

template <int BITS>
__device__ __forceinline__ void load4_codes(const uint8_t* p, const float* cent, int lane, float (&x)[4]) {
  uint32_t f;
  if constexpr (BITS == 2) {
    f = p[lane];
  } else {
    const uint8_t* q = p + (3 * lane >> 1);
    f = (static_cast<uint32_t>(q[0]) | (static_cast<uint32_t>(q[1]) << 8)) >> (4 * (lane & 1));
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) x[j] = cent[(f >> (BITS * j)) & ((1 << BITS) - 1)];
}

// Running softmax of one row: largest score, sum and weighted values.
struct Running {
  float m = -FLT_MAX, l = 0;
  float nat[4] = {0, 0, 0, 0}, rot[4] = {0, 0, 0, 0};
  __device__ __forceinline__ float weight(float s) {
    if (s > m) {
      const float f = expf(m - s);
      m = s;
      l *= f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        nat[j] *= f;
        rot[j] *= f;
      }
    }
    const float p = expf(s - m);
    l += p;
    return p;
  }
};

// One wave per row and query head, four values to a lane.
template <int BITS>
__global__ void __launch_bounds__(kThreads) hlwq_attention_kernel(const AttnArgs a) {
  constexpr float cent3[8] = HLWQ_CENTROIDS_3;
  constexpr float cent2[4] = HLWQ_CENTROIDS_2;
  __shared__ float cent[8];
  if constexpr (BITS > 0) {
    if (threadIdx.x < (1 << BITS)) cent[threadIdx.x] = BITS == 3 ? cent3[threadIdx.x & 7] : cent2[threadIdx.x & 3];
    __syncthreads();
  }
  const int lane = threadIdx.x & 63;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kThreads / 64) + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row64 = unit / a.q_heads;
  if (row64 >= a.rows) return;
  const int32_t row = static_cast<int32_t>(row64), head = static_cast<int32_t>(unit - row64 * a.q_heads);
  const int32_t kvh = head / (a.q_heads / a.kv_heads);
  // the last request that begins at or before the row
  int32_t lo = 0, hi = a.requests - 1;
  while (lo < hi) {
    const int32_t mid = (lo + hi + 1) >> 1;
    if (a.cu[mid] <= row)
      lo = mid;
    else
      hi = mid - 1;
  }
  const RowRange rr = row_range(a.cu, lo, a.rows);
  if (row < rr.begin || row >= rr.end) return;
  const int64_t n = rr.end - rr.begin;
  const int64_t held = a.lens ? max(static_cast<int64_t>(a.lens[lo]), n) - n : 0;
  const int64_t enc = BITS ? max(held - a.n_res, int64_t{0}) : 0;

  float q[4], qr[4];
  load4(a.q + row * a.q_stride + head * kDim, lane, q);
#pragma unroll
  for (int j = 0; j < 4; ++j) qr[j] = q[j];
  wave_fwht(qr, lane);
  Running st;
  if constexpr (BITS > 0) {
    for (int64_t t = 0; t < enc; ++t) {
      const int64_t p = t >> a.page_shift;
      const int32_t id = p < a.width ? a.table[lo * a.width + p] : -1;
      if (id < 0 || id >= a.n_pages) continue;
      const int64_t vec = ((static_cast<int64_t>(id) * a.kv_heads + kvh) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
      float x[4];
      load4_codes<BITS>(a.k_packed + vec * 32 * BITS, cent, lane, x);
      float s = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) s = __builtin_fmaf(qr[j], x[j], s);
      s = wave_sum(s) * (f16_value(a.k_norms[vec]) * (1.0f / kDim)) * a.scale;
      const float w = st.weight(s) * (f16_value(a.v_norms[vec]) * (1.0f / kDim));
      load4_codes<BITS>(a.v_packed + vec * 32 * BITS, cent, lane, x);
#pragma unroll
      for (int j = 0; j < 4; ++j) st.rot[j] = __builtin_fmaf(w, x[j], st.rot[j]);
    }
  }
  const int64_t last = held + (row - rr.begin);
  for (int64_t t = enc; t <= last; ++t) {
    const uint16_t *kp, *vp;
    if (t < held) {
      const int64_t o = ((static_cast<int64_t>(lo) * a.kv_heads + kvh) * a.ring + t % a.ring) * kDim;
      kp = a.k_window + o;
      vp = a.v_window + o;
    } else {
      kp = a.k_new + (rr.begin + (t - held)) * a.k_stride + kvh * kDim;
      vp = a.v_new + (rr.begin + (t - held)) * a.v_stride + kvh * kDim;
    }
    float x[4];
    load4(kp, lane, x);
    float s = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) s = __builtin_fmaf(q[j], x[j], s);
    const float w = st.weight(wave_sum(s) * a.scale);
    load4(vp, lane, x);
#pragma unroll
    for (int j = 0; j < 4; ++j) st.nat[j] = __builtin_fmaf(w, x[j], st.nat[j]);
  }
  wave_fwht(st.rot, lane);
  const float inv = 1.0f / st.l;
  float o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = (st.nat[j] + st.rot[j]) * inv;
  uint2 v;
  v.x = pack_bf16x2(o[0], o[1]);
  v.y = pack_bf16x2(o[2], o[3]);
  *reinterpret_cast<uint2*>(a.out + (static_cast<int64_t>(row) * a.q_heads + head) * kDim + 4 * lane) = v;
}

// Heads and rows of an attention call.  *nothing: valid, with no work.
int check_heads(int64_t rows, int64_t q_heads, int64_t kv_heads, bool* nothing) {
  if (rows < 0 || q_heads < 0 || kv_heads < 0) return HLWQ_ERR_SHAPE;
  *nothing = rows == 0 || q_heads == 0;
  if (*nothing) return HLWQ_OK;
  if (kv_heads == 0 || q_heads % kv_heads) return HLWQ_ERR_SHAPE;
  if (q_heads > kMaxHeads || rows > 0x7fffffff) return HLWQ_ERR_LIMIT;
  return HLWQ_OK;
}

int launch_attention(int bits, const AttnArgs& a, hipStream_t stream) {
  const int64_t groups = ceil_div(static_cast<int64_t>(a.rows) * a.q_heads, kThreads / 64);
  if (groups > 0x7fffff) return HLWQ_ERR_LIMIT;
  return launch(bits == 3 ? hlwq_attention_kernel<3> : bits == 2 ? hlwq_attention_kernel<2> : hlwq_attention_kernel<0>,
                dim3(static_cast<uint32_t>(groups)), dim3(kThreads), stream, a);
}

// Workgroups of a prompt call with `tile` rows to each: at most one tile more
// per sequence than whole ones.
int64_t prompt_groups(const AttnArgs& a, int64_t tile) {
  const int64_t rows = static_cast<int64_t>(a.rows) * a.group;
  return std::min(rows / tile + a.requests, rows) * a.kv_heads;
}

int launch_prompt(const AttnArgs& a, hipStream_t stream) {
  const bool wide = prompt_groups(a, 256) >= 512;
  const int64_t groups = prompt_groups(a, wide ? 256 : 128);
  if (groups > 0x7fffff) return HLWQ_ERR_LIMIT;
  return launch(wide ? hlwq_prompt_attention_kernel<8, 64> : hlwq_prompt_attention_kernel<4, 32>,
                dim3(static_cast<uint32_t>(groups)), dim3(wide ? 512 : 256), stream, a);
}

size_t workspace_bytes_of(int64_t requests, int64_t rows, int64_t q_heads, int64_t kv_heads) {
  bool nothing;
  if (requests <= 0 || requests > kMaxRequests || check_heads(rows, q_heads, kv_heads, &nothing) != HLWQ_OK || nothing) return 0;
  return 16;
}

int run_paged(const hlwq_kv_cache* c, const void* q, int64_t q_stride, int64_t q_heads, const void* k, int64_t k_stride,
              const void* v, int64_t v_stride, const int32_t* cu, const int32_t* lens, const int32_t* table,
              int64_t max_pages, int64_t rows, float scale, void* out, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!c) return HLWQ_ERR_NULL;
  std::vector<Span> spans;
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
  const size_t need = workspace_bytes_of(c->requests, rows, q_heads, c->kv_heads);
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
  a.width = max_pages;
  a.requests = static_cast<int32_t>(c->requests);
  a.rows = static_cast<int32_t>(rows);
  a.q_heads = static_cast<int32_t>(q_heads);
  a.kv_heads = static_cast<int32_t>(c->kv_heads);
  a.n_pages = static_cast<int32_t>(c->n_pages);
  a.page_shift = __builtin_ctzll(static_cast<uint64_t>(c->page_size));
  a.scale = scale;
  return launch_attention(c->bits, a, stream);
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
  std::vector<Span> spans;
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
