// verify.hip — which drafted tokens stand against the target's probabilities,
// and the token that follows them (include/hlwq_drafts.h).
//
// One workgroup walks a request's tree.  Each wave holds 64 nodes at a time, a
// node a lane, with the entries of both distributions that decide on it, so the
// next child of the node reached is a ballot away and no memory is waited for
// between decisions.  A row is read whole only where a child is refused (for the
// residual's mass) and for the token that follows.  All waves decide alike, from
// the same values, so that the sums may hold barriers.

#include "kv_common.h"

#include "hlwq_drafts.h"

#include <type_traits>

namespace hlwq_kv {
namespace {

constexpr int kVerifyThreads = 1024, kVerifyWaves = kVerifyThreads / 64;
constexpr int kMaxNodes = 4096;  // of a request
constexpr int64_t kMaxVocab = 1 << 24, kMaxRowStride = int64_t{1} << 40;

struct VerifyArgs {
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* cu;
  const void* target;
  const void* draft;
  const float* uniforms;
  const float* next_uniforms;
  int32_t* n_kept;
  int32_t* next_token;
  int32_t* kept;
  int64_t target_stride, draft_stride;
  int32_t requests, rows, vocab;
};

struct F32 {
  typedef float type;
  static constexpr int kWide = 4;  // values to a load
  __device__ __forceinline__ static float value(float v) { return v; }
};
struct Bf16 {
  typedef uint16_t type;
  static constexpr int kWide = 8;
  __device__ __forceinline__ static float value(uint16_t v) { return bf16_lo(v); }
};
struct F16 {
  typedef uint16_t type;
  static constexpr int kWide = 8;
  __device__ __forceinline__ static float value(uint16_t v) { return f16_value(v); }
};

// A row's residual weights: with DRAFT (p - s q)+, without p but for the refused
// tokens.  Probabilities below 0 and NaN are 0: p's by the positive part, which
// is 0 of a NaN, q's before they are taken from p, where a NaN would lose p and a
// negative one raise it.  (Where q is in 64 bits that is one instruction, which 48
// trees over 131072 fp32 do not notice, 39.8 us, and 23 over 59670 fp16 do, 28.6
// where 26.8 were taken without it; in 32 bits it is two, and 42.1 us for the 48.)
template <class T, bool DRAFT>
struct Residual {
  const typename T::type* p;
  const typename T::type* q;
  double s;                // 0: of p alone
  const int32_t* refused;  // in LDS
  int32_t n_refused;
};

template <class T>
struct Wide {
  typedef typename T::type type __attribute__((ext_vector_type(T::kWide), aligned(sizeof(typename T::type))));
};

// A lane's sum of weights of [lo, hi), over the wave's share of it, W values to a
// load.  Sixteen waves keep enough loads on their way; several to a wave make the
// code longer, and most of it runs once: four took 25 us for 250 rows of 100003
// bf16 where one takes 19.  Where a draft's refusals read row after row, two at a
// time are worth it: 39.4 us for 48 trees over 131072 where one takes 43.4 (four
// 38.9).
template <class T, bool DRAFT>
__device__ __forceinline__ double lane_sum(const Residual<T, DRAFT>& r, int32_t lo, int32_t hi, int lane) {
  typedef typename Wide<T>::type wide;
  constexpr int W = T::kWide;
  double sum = 0;
  const int32_t whole = lo + (hi - lo) / W * W;
  const auto over = [&](auto weight, bool both) {
    constexpr int kTogether = DRAFT ? 2 : 1;
    int32_t i = lo + lane * W;
    const auto step = [&](auto loads) {
      wide p[loads], q[loads];
#pragma unroll
      for (int k = 0; k < loads; ++k) {
        p[k] = *reinterpret_cast<const wide*>(r.p + i + 64 * W * k);
        q[k] = wide{};
        if (both) q[k] = *reinterpret_cast<const wide*>(r.q + i + 64 * W * k);
      }
#pragma unroll
      for (int k = 0; k < loads; ++k)
#pragma unroll
        for (int j = 0; j < W; ++j) sum += weight(i + 64 * W * k + j, T::value(p[k][j]), T::value(q[k][j]));
      i += 64 * W * loads;
    };
    if constexpr (kTogether > 1)
#pragma clang loop unroll(disable)
      while (i + 64 * W * (kTogether - 1) < whole) step(std::integral_constant<int, kTogether>{});
#pragma clang loop unroll(disable)
    while (i < whole) step(std::integral_constant<int, 1>{});
    for (i = whole + lane; i < hi; i += 64) sum += weight(i, T::value(r.p[i]), both ? T::value(r.q[i]) : 0.0f);
  };
  const auto alone = [](int32_t, float p, float) { return static_cast<double>(fmaxf(p, 0.0f)); };
  if constexpr (DRAFT) {
    if (r.s == 0)
      over(alone, false);
    else if (r.s == 1)
      over([](int32_t, float p, float q) { return fmax(static_cast<double>(p) - fmax(static_cast<double>(q), 0.0), 0.0); }, true);
    else
      over([s = r.s](int32_t, float p, float q) { return fmax(p - s * fmax(static_cast<double>(q), 0.0), 0.0); }, true);
  } else {
    // the refused tokens that lie here: none in most waves' shares
    int32_t here[2] = {-1, -1}, some = 0;
    for (int32_t k = 0; k < r.n_refused; ++k) {
      const int32_t x = __builtin_amdgcn_readfirstlane(r.refused[k]);
      if (x < lo || x >= hi) continue;
      if (some < 2) (some ? here[1] : here[0]) = x;
      ++some;
    }
    if (some == 0)
      over(alone, false);
    else if (some <= 2)
      over([here](int32_t i, float p, float) { return i == here[0] || i == here[1] ? 0.0 : static_cast<double>(fmaxf(p, 0.0f)); }, false);
    else
      over([&](int32_t i, float p, float) {
        for (int32_t k = 0; k < r.n_refused; ++k) p = r.refused[k] == i ? 0.0f : p;
        return static_cast<double>(fmaxf(p, 0.0f));
      }, false);
  }
  return sum;
}

// The range k of sixteen equal ones of [lo, hi), multiples of `unit` long.
struct Range {
  int32_t lo, hi;
};
__device__ __forceinline__ Range part_of(Range a, int32_t k, int32_t unit) {
  const int32_t size = static_cast<int32_t>(ceil_div(a.hi - a.lo, kVerifyWaves * unit)) * unit;
  Range r;
  r.lo = min(a.lo + k * size, a.hi);  // (2^24 and a part more)
  r.hi = min(r.lo + size, a.hi);
  return r;
}

// Sums of the sixteen parts of a range, one a wave, in LDS; returns their sum.
template <class T, bool DRAFT>
__device__ __forceinline__ double part_sums(const Residual<T, DRAFT>& r, Range all, int32_t unit, double* lds, int lane, int wave) {
  const Range mine = part_of(all, wave, unit);
  const double s = wave_sum(lane_sum(r, mine.lo, mine.hi, lane));
  __syncthreads();
  if (lane == 0) lds[wave] = s;
  __syncthreads();
  double total = 0;
#pragma unroll
  for (int k = 0; k < kVerifyWaves; ++k) total += lds[k];
  return total;
}

// The part in which the running sum passes `rest`, which becomes what of it lies
// in the part; where rounding leaves none, the last part with any weight.
__device__ __forceinline__ int32_t find_part(const double* lds, double& rest) {
  int32_t last = -1;
  double before = 0, last_before = 0;
  bool passed = false;
#pragma unroll
  for (int k = 0; k < kVerifyWaves; ++k) {
    const double v = lds[k];
    if (!passed && v > 0) {
      last = k;
      last_before = before;
      passed = before + v > rest;
    }
    before += v;
  }
  rest -= last_before;
  return last;
}

constexpr int32_t kPartUnit = 512;  // of the first parts, a multiple of what a wave loads at once

// The lowest index at which the running sum of the weights passes `rest`; -1 if they
// have none.  The sums of the row's sixteen parts, in LDS, are known: the part that
// holds it, a sixteenth of that, and so on down to 64 values, a lane each.
template <class T, bool DRAFT>
__device__ __forceinline__ int32_t sample(const Residual<T, DRAFT>& r, Range all, double rest, double* lds, int lane, int wave) {
  int32_t unit = kPartUnit;
  for (;;) {
    const int32_t k = find_part(lds, rest);
    if (k < 0) return -1;
    all = part_of(all, k, unit);
    if (all.hi - all.lo <= 64) break;
    unit = 64;
    part_sums(r, all, unit, lds, lane, wave);
  }
  const int32_t i = all.lo + lane;
  const double own = lane_sum(r, i, min(i + 1, all.hi), 0);
  double upto = own;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const double other = __shfl_up(upto, d);
    if (lane >= d) upto += other;
  }
  const uint64_t any = __ballot(own > 0), past = __ballot(own > 0 && upto > rest);
  if (!any) return -1;
  return all.lo + (past ? __builtin_ctzll(past) : 63 - __builtin_clzll(any));
}

template <class T, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads) hlwq_verify_kernel(const VerifyArgs a) {
  typedef typename T::type type;
  __shared__ double sums[kVerifyWaves];
  __shared__ int32_t kept[kMaxNodes], refused[kMaxNodes];
  __shared__ int32_t node_parent[64], node_token[64];
  __shared__ float node_u[64], node_p[64], node_q[64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t b = blockIdx.x;
  const auto not_kept = [&](int64_t from, int64_t to) {
    for (int64_t i = from + threadIdx.x; i < to; i += kVerifyThreads) a.kept[i] = -1;
  };
  if (a.requests == 0) return not_kept(0, a.rows);
  const RowRange rr = row_range(a.cu, b, a.rows);
  if (b == 0) {  // rows before the first request and past the last
    not_kept(0, rr.begin);
    not_kept(row_range(a.cu, a.requests - 1, a.rows).end, a.rows);
  }
  const int32_t count = min(rr.end - rr.begin, kMaxNodes);
  if (count <= 0) {
    if (threadIdx.x == 0) {
      a.n_kept[b] = 0;
      a.next_token[b] = -1;
    }
    return;
  }
  const type* target = static_cast<const type*>(a.target);
  const type* draft = static_cast<const type*>(a.draft);
  const auto p_row = [&](int32_t node) { return target + (rr.begin + static_cast<int64_t>(node)) * a.target_stride; };
  const auto q_row = [&](int32_t node) { return draft + (rr.begin + static_cast<int64_t>(node)) * a.draft_stride; };
  const Range all{0, a.vocab};

  int32_t cur = 0, n_kept = 1, n_refused = 0;
  double mass = 1, taken = 0;
  bool summed = false;  // `sums` holds the parts' sums of the present residual
  const auto residual = [&] { return Residual<T, DRAFT>{p_row(cur), DRAFT ? q_row(cur) : nullptr, taken, refused, n_refused}; };
  if (threadIdx.x == 0) kept[0] = 0;
  for (int32_t base = 0; base < count; base += 64) {
    __syncthreads();
    if (wave == 0) {
      const int32_t node = base + lane;
      int32_t parent = -1, token = -1;
      float u = 0, p = 0, q = 0;
      if (node > 0 && node < count) {
        const int64_t row = rr.begin + static_cast<int64_t>(node);
        parent = a.parents[row];
        token = a.tokens[row];
        u = a.uniforms[row];
        if (parent >= node || token < 0 || token >= a.vocab) parent = -1;
        if (parent >= 0) {
          p = T::value(p_row(parent)[token]);
          q = DRAFT ? fmaxf(T::value(q_row(parent)[token]), 0.0f) : 1.0f;
        }
      }
      node_parent[lane] = parent;
      node_token[lane] = token;
      node_u[lane] = u;
      node_p[lane] = p;
      node_q[lane] = q;
    }
    __syncthreads();
    const int32_t parent = node_parent[lane];
    uint64_t left = ~uint64_t{0};
    for (;;) {
      const uint64_t child = __ballot(parent == cur) & left;
      if (!child) break;
      const int at = __builtin_ctzll(child);
      left = at == 63 ? 0 : ~uint64_t{0} << (at + 1);
      const int32_t token = node_token[at];
      const double u = node_u[at], p = node_p[at], q = node_q[at];
      double value = p;
      if constexpr (DRAFT)
        value = p - taken * q;
      else
        for (int32_t k = 0; k < n_refused; ++k) value = refused[k] == token ? 0.0 : value;
      if (u * q * mass < (value > 0 ? value : 0.0)) {
        cur = base + at;
        if (threadIdx.x == 0) kept[n_kept] = cur;
        ++n_kept;
        mass = 1;
        taken = 0;
        n_refused = 0;
        summed = false;
      } else if (DRAFT) {
        taken += mass;
        mass = part_sums(residual(), all, kPartUnit, sums, lane, wave);
        summed = true;
      } else {
        mass -= value > 0 ? value : 0.0;
        __syncthreads();
        if (threadIdx.x == 0) refused[n_refused] = token;
        __syncthreads();
        ++n_refused;
      }
    }
  }

  Residual<T, DRAFT> r = residual();
  double total = summed ? mass : part_sums(r, all, kPartUnit, sums, lane, wave);
  if (!(total > 0)) {  // nothing left of p: p itself
    r.s = 0;
    r.n_refused = 0;
    total = part_sums(r, all, kPartUnit, sums, lane, wave);
  }
  const int32_t next = sample(r, all, a.next_uniforms[b] * total, sums, lane, wave);
  if (threadIdx.x == 0) {
    a.n_kept[b] = n_kept;
    a.next_token[b] = next;
  }
  for (int32_t i = threadIdx.x; i < rr.end - rr.begin; i += kVerifyThreads) a.kept[rr.begin + i] = i < n_kept ? rr.begin + kept[i] : -1;
}

int run_verify(const hlwq_drafts* d, hipStream_t stream) {
  if (!d) return HLWQ_ERR_NULL;
  if (d->dtype != HLWQ_F32 && d->dtype != HLWQ_BF16 && d->dtype != HLWQ_F16) return HLWQ_ERR_SHAPE;
  if (d->requests < 0 || d->rows < 0 || d->vocab < 1 || d->target_stride < d->vocab || (d->draft && d->draft_stride < d->vocab))
    return HLWQ_ERR_SHAPE;
  if (d->requests > kMaxRequests || d->rows > 0x7fffffff || d->vocab > kMaxVocab || d->target_stride > kMaxRowStride ||
      (d->draft && d->draft_stride > kMaxRowStride))
    return HLWQ_ERR_LIMIT;
  if (d->requests == 0 && (d->rows == 0 || !d->kept)) return HLWQ_OK;
  const uintptr_t size = d->dtype == HLWQ_F32 ? 4 : 2;
  if (d->requests > 0 && (!d->cu_rows || !d->n_kept || !d->next_token || !d->next_uniforms ||
                          (d->rows > 0 && (!d->tokens || !d->parents || !d->target || !d->uniforms || !d->kept))))
    return HLWQ_ERR_NULL;
  int64_t te, de, bytes;
  if (!mul_ok(d->rows, d->target_stride, &te) || !mul_ok(te, 4, &bytes) ||
      (d->draft && (!mul_ok(d->rows, d->draft_stride, &de) || !mul_ok(de, 4, &bytes))))
    return HLWQ_ERR_SHAPE;
  const struct {
    const void* p;
    int64_t count;
    bool written;
  } words[] = {{d->tokens, d->rows, false},       {d->parents, d->rows, false},       {d->cu_rows, d->requests + 1, false},
               {d->uniforms, d->rows, false},     {d->next_uniforms, d->requests, false}, {d->n_kept, d->requests, true},
               {d->next_token, d->requests, true}, {d->kept, d->rows, true}};
  Spans spans;
  for (const auto& w : words) {
    if (misaligned(w.p, 4)) return HLWQ_ERR_ALIGN;
    add_span(spans, w.p, w.count, 4, w.written);
  }
  if (misaligned(d->target, size) || misaligned(d->draft, size)) return HLWQ_ERR_ALIGN;
  if (d->rows > 0) {
    add_span(spans, d->target, (d->rows - 1) * d->target_stride + d->vocab, static_cast<int64_t>(size), false);
    if (d->draft) add_span(spans, d->draft, (d->rows - 1) * d->draft_stride + d->vocab, static_cast<int64_t>(size), false);
  }
  if (check_disjoint(spans) != HLWQ_OK) return HLWQ_ERR_OVERLAP;
  VerifyArgs a;
  a.tokens = d->tokens;
  a.parents = d->parents;
  a.cu = d->cu_rows;
  a.target = d->target;
  a.draft = d->draft;
  a.uniforms = d->uniforms;
  a.next_uniforms = d->next_uniforms;
  a.n_kept = d->n_kept;
  a.next_token = d->next_token;
  a.kept = d->kept;
  a.target_stride = d->target_stride;
  a.draft_stride = d->draft_stride;
  a.requests = static_cast<int32_t>(d->requests);
  a.rows = static_cast<int32_t>(d->rows);
  a.vocab = static_cast<int32_t>(d->vocab);
  const dim3 grid(static_cast<uint32_t>(std::max<int64_t>(d->requests, 1)));
  const auto go = [&](auto type) {
    using T = decltype(type);
    return d->draft ? launch(hlwq_verify_kernel<T, true>, grid, dim3(kVerifyThreads), stream, a)
                    : launch(hlwq_verify_kernel<T, false>, grid, dim3(kVerifyThreads), stream, a);
  };
  return d->dtype == HLWQ_F32 ? go(F32{}) : d->dtype == HLWQ_BF16 ? go(Bf16{}) : go(F16{});
}

}  // namespace
}  // namespace hlwq_kv

extern "C" int hlwq_verify_drafts(const hlwq_drafts* drafts, void* hip_stream) {
  return hlwq_kv::run_verify(drafts, static_cast<hipStream_t>(hip_stream));
}
