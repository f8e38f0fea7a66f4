// kv_paged.hip — the paged KV cache's bookkeeping and writes: page planning and
// the append of a step's tokens (include/hlwq_attention.h).  Compiled with
// -ffp-contract=off, so the encoder follows the operation order documented in
// include/hlwq.h bit for bit.

#include "kv_common.h"

namespace hlwq_kv {
namespace {

// ---------------------------------------------------------------------------
// Page plan.  One workgroup plans the tables (the prefix sums over the
// requests, the stack and the block table are one dependent chain), then a
// grid over the rows fills the maps.  Latency bounds both: 4.3 + 2.2 us for 64
// requests of a token, 17.4 + 4.4 us for 1000 requests of which some are reset
// and some begin.
// ---------------------------------------------------------------------------

constexpr int kPlanThreads = 1024;
constexpr int kPlanWaves = kPlanThreads / 64;
constexpr int kRowThreads = 256;
constexpr int kFewPages = 64;  // that a lane takes by itself

struct PlanArgs {
  const int32_t* tokens;
  const int32_t* n_new;
  const uint8_t* reset;
  const int32_t* n_free;
  int32_t* free_pages;
  int32_t* table;
  int32_t* cu;
  int32_t* lens;
  int32_t* row_request;
  int32_t* positions;
  int32_t* slots;
  int32_t* n_free_after;
  int32_t* status;
  int32_t requests, rows, width, n_pages, page_shift;
  int64_t n_res;
};

// What one request asks of a step.
struct Need {
  int64_t held, n;    // tokens before (0 after a reset) and new
  int64_t back;       // pages given back
  int64_t had, want;  // pages before and after
  bool bad;
};
__device__ __forceinline__ int64_t pages_of(const PlanArgs& a, int64_t tokens) {
  const int64_t e = tokens - a.n_res;
  return e > 0 ? (e + (int64_t{1} << a.page_shift) - 1) >> a.page_shift : 0;
}
__device__ __forceinline__ Need need_of(const PlanArgs& a, int32_t b) {
  Need d;
  const int32_t t = a.tokens[b], n = a.n_new[b];
  const bool ended = a.reset && a.reset[b];
  const int64_t before = pages_of(a, t);
  d.held = ended ? 0 : t;
  d.n = n;
  d.back = ended ? before : 0;
  d.had = ended ? 0 : before;
  d.want = pages_of(a, d.held + n);
  d.bad = t < 0 || n < 0 || before > a.width || d.want > a.width || d.held + n > 0x7fffffff;
  if (d.bad) d.n = d.back = d.had = d.want = 0;
  return d;
}

__global__ void __launch_bounds__(kPlanThreads) hlwq_kv_plan_tables_kernel(const PlanArgs a) {
  __shared__ int64_t sums[3][kPlanWaves];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t per = (a.requests + kPlanThreads - 1) / kPlanThreads;
  const int32_t b0 = static_cast<int32_t>(min(static_cast<int64_t>(threadIdx.x) * per, static_cast<int64_t>(a.requests)));
  const int32_t b1 = min(b0 + per, a.requests);
  const int32_t nf = a.n_free[0];

  // totals and exclusive prefixes of new rows, pages given back, pages taken
  int64_t own[3] = {0, 0, 0};
  bool bad = nf < 0 || nf > a.n_pages;
  for (int32_t b = b0; b < b1; ++b) {
    const Need d = need_of(a, b);
    bad |= d.bad;
    own[0] += d.n;
    own[1] += d.back;
    own[2] += d.want - d.had;
  }
  int64_t pre[3], total[3];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int64_t s = wave_scan(own[k]);
    pre[k] = s - own[k];
    if (lane == 63) sums[k][wave] = s;
  }
  bad = __syncthreads_or(bad);
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    total[k] = 0;
    for (int w = 0; w < kPlanWaves; ++w) {
      if (w == wave) pre[k] += total[k];
      total[k] += sums[k][w];
    }
  }
  bad |= total[0] > a.rows || nf + total[1] > a.n_pages;

  // Pages given back: a wave goes through its lanes' requests one by one, 256
  // pages at a time.  All are looked at before any is moved.
  const auto for_back = [&](auto run) {
    int64_t at = pre[1];
    for (int32_t k = 0; k < per; ++k) {
      const int32_t b = b0 + k;
      const int32_t own = b < b1 ? static_cast<int32_t>(need_of(a, b).back) : 0;
      uint64_t todo = __ballot(own > 0);
      while (todo) {
        const int l = __builtin_ctzll(todo);
        todo &= todo - 1;
        const int32_t n = __builtin_amdgcn_readlane(own, l);
        const int32_t to = __builtin_amdgcn_readlane(static_cast<int32_t>(at), l);
        const int32_t* from = a.table + static_cast<int64_t>(__builtin_amdgcn_readlane(b, l)) * a.width;
        for (int32_t p0 = 0; p0 < n; p0 += 256) {
          int32_t id[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) id[i] = p0 + 64 * i + lane < n ? from[p0 + 64 * i + lane] : 0;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (p0 + 64 * i + lane < n) run(id[i], to + p0 + 64 * i + lane);
        }
      }
      at += own;
    }
  };
  if (!bad && total[1] > 0) {
    bool off = false;
    for_back([&](int32_t id, int32_t) { off |= id < 0 || id >= a.n_pages; });
    bad = __syncthreads_or(off);
  }
  const int64_t top = nf + total[1];
  const int64_t missing = total[2] - top;
  if (bad || missing > 0) {
    for (int32_t b = b0; b < b1; ++b) {
      a.cu[b] = 0;
      a.lens[b] = a.tokens[b];
    }
    if (threadIdx.x == 0) {
      a.cu[a.requests] = 0;
      *a.n_free_after = nf;
      *a.status = bad ? -1 : static_cast<int32_t>(min(missing, int64_t{0x7fffffff}));
    }
    return;
  }
  if (total[1] > 0) {
    for_back([&](int32_t id, int32_t to) { a.free_pages[nf + to] = id; });
    __syncthreads();
  }
  // Pages taken: up to kFewPages by the request's own lane, more by the whole
  // wave.  A lane alone waits for each load: one request's 4096 pages made a plan
  // of 427 us, which a wave does in 19; but 64 requests' 62 pages each, which the
  // lanes take side by side (19 us), take a wave 25.
  int64_t row = pre[0], taken = pre[2];
  for (int32_t k = 0; k < per; ++k) {
    const int32_t b = b0 + k;
    int32_t had = 0, n = 0;
    if (b < b1) {
      const Need d = need_of(a, b);
      a.cu[b] = static_cast<int32_t>(row);
      a.lens[b] = static_cast<int32_t>(d.held + d.n);
      row += d.n;
      had = static_cast<int32_t>(d.had);
      n = static_cast<int32_t>(d.want - d.had);
    }
    const int32_t first = static_cast<int32_t>(top - 1 - taken);
    if (n <= kFewPages)
      for (int32_t p = 0; p < n; ++p) a.table[static_cast<int64_t>(b) * a.width + had + p] = a.free_pages[first - p];
    uint64_t todo = __ballot(n > kFewPages);
    while (todo) {
      const int l = __builtin_ctzll(todo);
      todo &= todo - 1;
      const int32_t many = __builtin_amdgcn_readlane(n, l);
      const int32_t* from = a.free_pages + __builtin_amdgcn_readlane(first, l);
      int32_t* to = a.table + static_cast<int64_t>(__builtin_amdgcn_readlane(b, l)) * a.width + __builtin_amdgcn_readlane(had, l);
      for (int32_t p0 = 0; p0 < many; p0 += 256) {
        int32_t id[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) id[i] = p0 + 64 * i + lane < many ? from[-(p0 + 64 * i + lane)] : 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (p0 + 64 * i + lane < many) to[p0 + 64 * i + lane] = id[i];
      }
    }
    taken += n;
  }
  if (threadIdx.x == 0) {
    a.cu[a.requests] = static_cast<int32_t>(total[0]);
    *a.n_free_after = static_cast<int32_t>(top - total[2]);
    *a.status = 0;
  }
}

__global__ void __launch_bounds__(kRowThreads) hlwq_kv_plan_rows_kernel(const PlanArgs a) {
  const int64_t i64 = static_cast<int64_t>(blockIdx.x) * kRowThreads + threadIdx.x;
  if (i64 >= a.rows) return;
  const int32_t i = static_cast<int32_t>(i64);
  int32_t req = -1, pos = -1, slot = -1;
  if (i < a.cu[a.requests]) {
    // the last request that begins at or before row i (empty ones begin where
    // the next one does, so the last is the one that owns it)
    int32_t lo = 0, hi = a.requests - 1;
    while (lo < hi) {
      const int32_t mid = (lo + hi + 1) >> 1;
      if (a.cu[mid] <= i)
        lo = mid;
      else
        hi = mid - 1;
    }
    req = lo;
    pos = a.lens[lo] - (a.cu[lo + 1] - i);
    const int64_t old = pos - a.n_res;
    if (old >= 0) {
      const int32_t id = a.table[static_cast<int64_t>(lo) * a.width + (old >> a.page_shift)];
      if (id >= 0 && id < a.n_pages)
        slot = static_cast<int32_t>((static_cast<int64_t>(id) << a.page_shift) + (old & ((1 << a.page_shift) - 1)));
    }
  }
  a.row_request[i] = req;
  a.positions[i] = pos;
  a.slots[i] = slot;
}

// ---------------------------------------------------------------------------
// Append.  Eight lanes take one head vector of one row, K or V, 32 values a
// lane: they encode the token that the row pushes out of the window (from the
// ring, or from the step's own row n_residual before it) into its slot, and put
// a new token that stays into the ring.  A ring slot that is read and rewritten
// in the same call has the same lanes do both, in that order, so nobody waits
// for anybody.
//
// What bounds a long append is the VALU (about 125 instructions a vector, 69%
// busy; a whole wave to a vector, four values a lane, takes 320), what bounds a
// decode step the chain of three loads behind one another.  Measured: a prompt
// of 16383 tokens on 4 KV heads, 80 MB, 29 us (2.7 TB/s); a token of each of 32
// requests 5.8 us.
// ---------------------------------------------------------------------------

struct AppendArgs {
  const uint16_t* src[2];
  int64_t stride[2];
  uint8_t* packed[2];
  uint16_t* norms[2];
  uint16_t* window[2];
  const int32_t* cu;
  const int32_t* lens;
  const int32_t* row_request;
  const int32_t* slots;
  int64_t n_slots;  // n_pages * page_size
  int32_t requests, rows, heads, page_shift;
  int64_t n_res;
  int32_t ring;
};

constexpr int kAppendThreads = 256;
constexpr int kAppendLanes = 8;  // to a vector

__device__ __forceinline__ int32_t floor_mod(int64_t a, int32_t m) {
  const int32_t r = static_cast<int32_t>(a < 0 ? ~a : a) % m;  // positions and their differences fit 31 bits
  return a < 0 ? m - 1 - r : r;
}

// 8 codes of y[0 .. 7], first in the lowest bits: the number of thresholds
// strictly below y, found by halves, each comparison's bit shifted in.
template <int BITS>
__device__ __forceinline__ uint32_t eight_codes(const float* y) {
  constexpr float t3[7] = HLWQ_THRESHOLDS_3;
  constexpr float t2[3] = HLWQ_THRESHOLDS_2;
  uint32_t v = 0;
#pragma unroll
  for (int i = 7; i >= 0; --i) {
    if constexpr (BITS == 3) {
      const bool c2 = y[i] > t3[3];
      const bool c1 = y[i] > (c2 ? t3[5] : t3[1]);
      const float lo = c1 ? t3[2] : t3[0], hi = c1 ? t3[6] : t3[4];
      const bool c0 = y[i] > (c2 ? hi : lo);
      v = v + v + c2;
      v = v + v + c1;
      v = v + v + c0;
    } else {
      const bool c1 = y[i] > t2[1];
      const bool c0 = y[i] > (c1 ? t2[2] : t2[0]);
      v = v + v + c1;
      v = v + v + c0;
    }
  }
  return v;
}

// Codes and norm of the vector whose values 32 i .. 32 i + 31 are lane i's (of
// eight), to `packed` (the vector's bytes) and *norm.
template <int BITS>
__device__ __forceinline__ void encode(const u32x4 (&w)[4], uint8_t* packed, uint16_t* norm, int i) {
  float x[32];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    x[2 * k] = bf16_lo(w[k >> 2][k & 3]);
    x[2 * k + 1] = bf16_hi(w[k >> 2][k & 3]);
  }
  // the norm's adjacent-pair tree, five levels in the lane, three across
  float s[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) s[k] = __builtin_fmaf(x[2 * k], x[2 * k], x[2 * k + 1] * x[2 * k + 1]);
#pragma unroll
  for (int n = 8; n >= 1; n >>= 1)
#pragma unroll
    for (int k = 0; k < n; ++k) s[k] = s[2 * k] + s[2 * k + 1];
  float sum = s[0];
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) sum = sum + lane_xor(sum, d);
  const float n = sqrtf(sum);
  const float r = n >= FLT_MIN ? 1.0f / n : 0.0f;
  // butterflies at strides 1 .. 16 in the lane, 32 .. 128 across: a + b below,
  // a - b above, each one rounding (the product by +-1 is exact)
#pragma unroll
  for (int h = 1; h < 32; h <<= 1)
#pragma unroll
    for (int k = 0; k < 32; ++k)
      if ((k & h) == 0) {
        const float a = x[k], b = x[k + h];
        x[k] = a + b;
        x[k + h] = a - b;
      }
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) {
    const float sign = (i & d) ? -1.0f : 1.0f;
#pragma unroll
    for (int k = 0; k < 32; ++k) x[k] = __builtin_fmaf(x[k], sign, lane_xor(x[k], d));
  }
#pragma unroll
  for (int k = 0; k < 32; ++k) x[k] *= r;
  uint32_t g[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) g[k] = eight_codes<BITS>(x + 8 * k);
  if constexpr (BITS == 3) {
    u32x3 out;
    out[0] = g[0] | (g[1] << 24);
    out[1] = (g[1] >> 8) | (g[2] << 16);
    out[2] = (g[2] >> 16) | (g[3] << 8);
    uint32_t* to = reinterpret_cast<uint32_t*>(packed + 12 * i);
    to[0] = out[0];
    to[1] = out[1];
    to[2] = out[2];
  } else {
    *reinterpret_cast<u32x2*>(packed + 8 * i) = u32x2{g[0] | (g[1] << 16), g[2] | (g[3] << 16)};
  }
  if (i == 0) *norm = f16_bits(n);
}

template <int BITS>
__global__ void __launch_bounds__(kAppendThreads) hlwq_kv_paged_append_kernel(const AppendArgs a) {
  const int i = threadIdx.x & (kAppendLanes - 1);
  const int side = blockIdx.y;
  const uint32_t unit = blockIdx.x * (kAppendThreads / kAppendLanes) + threadIdx.x / kAppendLanes;
  const int32_t row = static_cast<int32_t>(unit / static_cast<uint32_t>(a.heads));
  if (row >= a.rows) return;
  const int32_t head = static_cast<int32_t>(unit - static_cast<uint32_t>(row) * static_cast<uint32_t>(a.heads));
  const int32_t b = a.row_request[row];
  if (b < 0 || b >= a.requests) return;
  const RowRange rr = row_range(a.cu, b, a.rows);
  if (row < rr.begin || row >= rr.end) return;
  const int64_t n = rr.end - rr.begin;
  const int64_t total = max(static_cast<int64_t>(a.lens[b]), n), held = total - n;
  const int64_t t = held + (row - rr.begin), old = t - a.n_res;
  const int64_t stay = max(held, total - a.n_res);  // first new token that stays in the window
  const uint16_t* src = a.src[side] + head * kDim + 32 * i;
  uint16_t* ring = a.window[side] + (static_cast<int64_t>(b) * a.heads + head) * a.ring * kDim + 32 * i;
  const auto load = [](const uint16_t* p, u32x4(&w)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = reinterpret_cast<const u32x4*>(p)[k];
  };
  const auto store = [](uint16_t* p, const u32x4(&w)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) reinterpret_cast<u32x4*>(p)[k] = w[k];
  };

  if (old >= 0) {
    const bool ringed = old < held;
    uint16_t* place = ringed ? ring + static_cast<int64_t>(floor_mod(old, a.ring)) * kDim : nullptr;
    const int64_t slot = a.slots[row];
    if (slot >= 0 && slot < a.n_slots) {
      u32x4 w[4];
      load(ringed ? place : src + (row - a.n_res) * a.stride[side], w);
      const int64_t vec = (((slot >> a.page_shift) * a.heads + head) << a.page_shift) + (slot & ((1 << a.page_shift) - 1));
      encode<BITS>(w, a.packed[side] + vec * (32 * BITS), a.norms[side] + vec, i);
    }
    if (ringed) {
      // the token that stays in the slot just read, if one does
      const int64_t t2 = stay + floor_mod(old - stay, a.ring);
      if (t2 < total) {
        u32x4 w[4];
        load(src + (rr.begin + (t2 - held)) * a.stride[side], w);
        store(place, w);
      }
    }
  }
  if (t >= stay) {
    // its slot's last token before the step; if that one leaves the window
    // now, the row that encodes it writes this one
    const int64_t u = held - 1 - floor_mod(held - 1 - t, a.ring);
    const bool other = u >= 0 && u >= held - a.n_res && u < total - a.n_res;
    if (!other) {
      u32x4 w[4];
      load(src + row * a.stride[side], w);
      store(ring + static_cast<int64_t>(floor_mod(t, a.ring)) * kDim, w);
    }
  }
}

int run_plan(const hlwq_kv_plan* p, hipStream_t stream) {
  if (!p) return HLWQ_ERR_NULL;
  if (p->requests < 0 || p->rows < 0 || p->max_pages < 0 || p->n_pages < 0 || p->n_residual < 0) return HLWQ_ERR_SHAPE;
  if (p->page_size < 16 || p->page_size > 256 || (p->page_size & (p->page_size - 1))) return HLWQ_ERR_SHAPE;
  if (p->requests > kMaxRequests || p->max_pages > kMaxTable || p->rows > 0x7fffffff ||
      p->n_pages > 0x7fffffff / p->page_size)
    return HLWQ_ERR_LIMIT;
  const int64_t table = p->requests * p->max_pages;
  if (!p->n_free || !p->cu_new || !p->n_free_after || !p->status ||
      (p->requests > 0 && (!p->tokens || !p->n_new || !p->lens)) ||
      (p->rows > 0 && (!p->row_request || !p->positions || !p->slots)) || (p->n_pages > 0 && !p->free_pages) ||
      (table > 0 && !p->block_table))
    return HLWQ_ERR_NULL;
  Spans spans;
  const struct {
    const void* p;
    int64_t count;
    bool written;
  } words[] = {{p->tokens, p->requests, false},      {p->n_new, p->requests, false},  {p->n_free, 1, false},
               {p->free_pages, p->n_pages, true},    {p->block_table, table, true},   {p->cu_new, p->requests + 1, true},
               {p->lens, p->requests, true},         {p->row_request, p->rows, true}, {p->positions, p->rows, true},
               {p->slots, p->rows, true},            {p->n_free_after, 1, true},      {p->status, 1, true}};
  for (const auto& w : words) {
    if (misaligned(w.p, 4)) return HLWQ_ERR_ALIGN;
    add_span(spans, w.p, w.count, 4, w.written);
  }
  add_span(spans, p->reset, p->requests, 1, false);
  if (check_disjoint(spans) != HLWQ_OK) return HLWQ_ERR_OVERLAP;
  PlanArgs a;
  a.tokens = p->tokens;
  a.n_new = p->n_new;
  a.reset = p->reset;
  a.n_free = p->n_free;
  a.free_pages = p->free_pages;
  a.table = p->block_table;
  a.cu = p->cu_new;
  a.lens = p->lens;
  a.row_request = p->row_request;
  a.positions = p->positions;
  a.slots = p->slots;
  a.n_free_after = p->n_free_after;
  a.status = p->status;
  a.requests = static_cast<int32_t>(p->requests);
  a.rows = static_cast<int32_t>(p->rows);
  a.width = static_cast<int32_t>(p->max_pages);
  a.n_pages = static_cast<int32_t>(p->n_pages);
  a.page_shift = __builtin_ctzll(static_cast<uint64_t>(p->page_size));
  a.n_res = p->n_residual;
  const int st = launch(hlwq_kv_plan_tables_kernel, dim3(1), dim3(kPlanThreads), stream, a);
  if (st != HLWQ_OK || p->rows == 0) return st;
  return launch(hlwq_kv_plan_rows_kernel, dim3(static_cast<uint32_t>(ceil_div(p->rows, kRowThreads))), dim3(kRowThreads),
                stream, a);
}

int run_append(const hlwq_kv_cache* c, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
               const int32_t* cu, const int32_t* lens, const int32_t* row_request, const int32_t* slots, int64_t rows,
               hipStream_t stream) {
  if (!c) return HLWQ_ERR_NULL;
  Spans spans;
  int st = check_cache(*c, true, spans);
  if (st != HLWQ_OK) return st;
  if (rows < 0) return HLWQ_ERR_SHAPE;
  if (rows == 0 || c->requests == 0 || c->kv_heads == 0) return HLWQ_OK;
  int64_t units;
  // (a launch has at most 2^32 - 1 work-items)
  if (rows > 0x7fffffff || !mul_ok(rows, c->kv_heads, &units) ||
      ceil_div(units, kAppendThreads / kAppendLanes) > 0xffffffff / kAppendThreads)
    return HLWQ_ERR_LIMIT;
  int64_t ke, ve;
  if ((st = check_rows(k, k_stride, rows, c->kv_heads, &ke)) != HLWQ_OK ||
      (st = check_rows(v, v_stride, rows, c->kv_heads, &ve)) != HLWQ_OK)
    return st;
  if (!cu || !lens || !row_request || !slots) return HLWQ_ERR_NULL;
  if (misaligned(cu, 4) || misaligned(lens, 4) || misaligned(row_request, 4) || misaligned(slots, 4)) return HLWQ_ERR_ALIGN;
  add_span(spans, k, ke, 2, false);
  add_span(spans, v, ve, 2, false);
  add_span(spans, cu, c->requests + 1, 4, false);
  add_span(spans, lens, c->requests, 4, false);
  add_span(spans, row_request, rows, 4, false);
  add_span(spans, slots, rows, 4, false);
  if (check_disjoint(spans) != HLWQ_OK) return HLWQ_ERR_OVERLAP;
  AppendArgs a;
  const hlwq_kv_store* s[2] = {&c->k, &c->v};
  const void* src[2] = {k, v};
  const int64_t stride[2] = {k_stride, v_stride};
  for (int i = 0; i < 2; ++i) {
    a.src[i] = static_cast<const uint16_t*>(src[i]);
    a.stride[i] = stride[i];
    a.packed[i] = static_cast<uint8_t*>(s[i]->packed);
    a.norms[i] = static_cast<uint16_t*>(s[i]->norms);
    a.window[i] = static_cast<uint16_t*>(s[i]->window);
  }
  a.cu = cu;
  a.lens = lens;
  a.row_request = row_request;
  a.slots = slots;
  a.n_slots = c->n_pages * c->page_size;
  a.requests = static_cast<int32_t>(c->requests);
  a.rows = static_cast<int32_t>(rows);
  a.heads = static_cast<int32_t>(c->kv_heads);
  a.page_shift = __builtin_ctzll(static_cast<uint64_t>(c->page_size));
  a.n_res = c->n_residual;
  a.ring = static_cast<int32_t>(c->ring);
  const dim3 grid(static_cast<uint32_t>(ceil_div(units, kAppendThreads / kAppendLanes)), 2);
  return launch(c->bits == 3 ? hlwq_kv_paged_append_kernel<3> : hlwq_kv_paged_append_kernel<2>, grid, dim3(kAppendThreads),
                stream, a);
}

}  // namespace
}  // namespace hlwq_kv

extern "C" {

int hlwq_kv_page_plan(const hlwq_kv_plan* plan, void* hip_stream) {
  return hlwq_kv::run_plan(plan, static_cast<hipStream_t>(hip_stream));
}

int hlwq_kv_paged_append(const hlwq_kv_cache* cache, const void* k_new_bf16, int64_t k_stride, const void* v_new_bf16,
                         int64_t v_stride, const int32_t* cu_new, const int32_t* lens, const int32_t* row_request,
                         const int32_t* slots, int64_t rows, void* hip_stream) {
  return hlwq_kv::run_append(cache, k_new_bf16, k_stride, v_new_bf16, v_stride, cu_new, lens, row_request, slots, rows,
                             static_cast<hipStream_t>(hip_stream));
}

}  // extern "C"
