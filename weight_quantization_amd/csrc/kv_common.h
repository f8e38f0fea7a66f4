// kv_common.h — what the paged-cache and attention kernels share: conversions,
// cross-lane exchanges and the wave-wide Walsh-Hadamard transform on the
// device; size checks, overlap checks and launches on the host.
#pragma once

#include <hip/hip_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cstdint>

#include "hlwq_attention.h"
#include "hlwq_tables.inc"

namespace hlwq_kv {

constexpr int kDim = 256;  // head vector length

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x3 __attribute__((ext_vector_type(3)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// device
// ---------------------------------------------------------------------------

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two floats to a pair of bf16, round to nearest even, NaN kept.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
  const bf16x2 v = {static_cast<__bf16>(lo), static_cast<__bf16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

__device__ __forceinline__ uint16_t f16_bits(float f) { return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f)); }
__device__ __forceinline__ float f16_value(uint16_t b) { return static_cast<float>(__builtin_bit_cast(_Float16, b)); }

// Value of lane l ^ d (d a compile-time power of two after unrolling), all in
// the VALU: quad permutations for d = 1 and 2; two mirrors for 4 and 8 (l ^ 3
// then l ^ 7, l ^ 7 then l ^ 15); for 16 and 32 the swaps of half rows and half
// waves between two copies.  A swizzle through LDS takes ten times as long.
__device__ __forceinline__ uint32_t lane_xor(uint32_t v, int d) {
  const int i = static_cast<int>(v);
  if (d == 1) return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(i, 0xB1, 0xF, 0xF, true));
  if (d == 2) return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(i, 0x4E, 0xF, 0xF, true));
  if (d == 4) {
    const int j = __builtin_amdgcn_mov_dpp(i, 0x1B, 0xF, 0xF, true);
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(j, 0x141, 0xF, 0xF, true));
  }
  if (d == 8) {
    const int j = __builtin_amdgcn_mov_dpp(i, 0x141, 0xF, 0xF, true);
    return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(j, 0x140, 0xF, 0xF, true));
  }
  if (d == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    return (threadIdx.x & 16) ? r[0] : r[1];
  }
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return (threadIdx.x & 32) ? r[0] : r[1];
}
__device__ __forceinline__ float lane_xor(float v, int d) { return __uint_as_float(lane_xor(__float_as_uint(v), d)); }

__device__ __forceinline__ double lane_xor(double v, int d) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = lane_xor(static_cast<uint32_t>(u), d), hi = lane_xor(static_cast<uint32_t>(u >> 32), d);
  return __builtin_bit_cast(double, lo | static_cast<uint64_t>(hi) << 32);
}

// The value of one lane, in all.
__device__ __forceinline__ double lane_value(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = __builtin_amdgcn_readlane(static_cast<uint32_t>(u), lane);
  const uint32_t hi = __builtin_amdgcn_readlane(static_cast<uint32_t>(u >> 32), lane);
  return __builtin_bit_cast(double, lo | static_cast<uint64_t>(hi) << 32);
}

// Inclusive prefix sum over the wave: within rows of sixteen, then the rows'
// last values on.
template <int CTRL, int ROWS>
__device__ __forceinline__ int64_t scan_step(int64_t v) {
  const int lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xF, false);
  const int hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(v >> 32), CTRL, ROWS, 0xF, false);
  return v + static_cast<int64_t>((static_cast<uint64_t>(static_cast<uint32_t>(hi)) << 32) | static_cast<uint32_t>(lo));
}
__device__ __forceinline__ int64_t wave_scan(int64_t v) {
  v = scan_step<0x111, 0xF>(v);
  v = scan_step<0x112, 0xF>(v);
  v = scan_step<0x114, 0xF>(v);
  v = scan_step<0x118, 0xF>(v);
  v = scan_step<0x142, 0xA>(v);
  return scan_step<0x143, 0xC>(v);
}
__device__ __forceinline__ int32_t wave_scan(int32_t v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);
  return v + __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);
}
// Largest value and sum over the wave, in every lane.
__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, lane_xor(v, d));
  return v;
}
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += lane_xor(v, d);
  return v;
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += lane_xor(v, d);
  return v;
}

// Unnormalised butterflies of a 256-vector held four values to a lane (lane l
// holds 4l .. 4l + 3), strides 1, 2, 4, .. 128, each sum one fp32 rounding.
__device__ __forceinline__ void wave_fwht(float (&x)[4], int lane) {
  const float a0 = x[0] + x[1], a1 = x[0] - x[1], a2 = x[2] + x[3], a3 = x[2] - x[3];
  x[0] = a0 + a2;
  x[2] = a0 - a2;
  x[1] = a1 + a3;
  x[3] = a1 - a3;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const bool upper = (lane & d) != 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float q = lane_xor(x[j], d);
      x[j] = upper ? q - x[j] : x[j] + q;
    }
  }
}

// The rows of request b: [begin, end) cut to the rows there are.
struct RowRange {
  int32_t begin, end;
};
__device__ __forceinline__ RowRange row_range(const int32_t* __restrict__ cu, int64_t b, int32_t rows) {
  RowRange r;
  r.begin = min(max(cu[b], 0), rows);
  r.end = min(max(cu[b + 1], r.begin), rows);
  return r;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

inline bool mul_ok(int64_t a, int64_t b, int64_t* r) { return !__builtin_mul_overflow(a, b, r); }
__host__ __device__ inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// One buffer of a call: its bytes [lo, hi), and whether the call writes it (a
// size past the address space counts as reaching its end).
struct Span {
  uintptr_t lo, hi;
  bool written;
};
// Of one call: at most fifteen (an entry point allocates nothing, so that
// nothing is thrown through it).
struct Spans {
  Span at[16];
  int count = 0;
};
inline void add_span(Spans& v, const void* p, int64_t count, int64_t unit, bool written) {
  int64_t bytes;
  if (!p || count <= 0) return;
  if (!mul_ok(count, unit, &bytes)) bytes = INT64_MAX;
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  uintptr_t hi;
  if (__builtin_add_overflow(lo, static_cast<uintptr_t>(bytes), &hi)) hi = UINTPTR_MAX;
  v.at[v.count++] = Span{lo, hi, written};
}

// HLWQ_ERR_OVERLAP if a written buffer shares a byte with any other buffer.
inline int check_disjoint(Spans& v) {
  std::sort(v.at, v.at + v.count, [](const Span& a, const Span& b) { return a.lo < b.lo; });
  uintptr_t end_any = 0, end_written = 0;
  for (int i = 0; i < v.count; ++i) {
    const Span& x = v.at[i];
    if (x.lo < end_written || (x.written && x.lo < end_any)) return HLWQ_ERR_OVERLAP;
    end_any = std::max(end_any, x.hi);
    if (x.written) end_written = std::max(end_written, x.hi);
  }
  return HLWQ_OK;
}

template <typename T>
struct same_type {
  using type = T;
};

// Launch a kernel and return the status of this launch itself.
template <typename... P>
int launch(void (*kernel)(P...), dim3 grid, dim3 block, hipStream_t stream, typename same_type<P>::type... args) {
  void* params[] = {static_cast<void*>(&args)...};
  return hipLaunchKernel(reinterpret_cast<const void*>(kernel), grid, block, params, 0, stream) == hipSuccess
             ? HLWQ_OK
             : HLWQ_ERR_DEVICE;
}

// Sizes a step may have.
constexpr int64_t kMaxRequests = 1 << 20;
constexpr int64_t kMaxTable = 1 << 20;
constexpr int64_t kMaxHeads = 1 << 12;
constexpr int64_t kMaxStride = 1 << 22;  // elements: 64 rows stay below 2^31 bytes

// Rows of `heads` 256-vectors, `stride` elements apart: the extent in
// elements, or a status.
inline int check_rows(const void* p, int64_t stride, int64_t rows, int64_t heads, int64_t* extent) {
  if (stride < heads * kDim || (stride & 7)) return HLWQ_ERR_SHAPE;
  if (stride > kMaxStride) return HLWQ_ERR_LIMIT;
  int64_t bytes;
  if (!mul_ok(rows - 1, stride, extent) || __builtin_add_overflow(*extent, heads * kDim, extent) ||
      !mul_ok(*extent, 2, &bytes))
    return HLWQ_ERR_SHAPE;
  if (!p) return HLWQ_ERR_NULL;
  return misaligned(p, 16) ? HLWQ_ERR_ALIGN : HLWQ_OK;
}

// Validate a cache and add its buffers to `spans` (written or read by the call).
inline int check_cache(const hlwq_kv_cache& c, bool written, Spans& spans) {
  if (c.head_dim != kDim) return HLWQ_ERR_BLOCK;
  if (c.bits != 3 && c.bits != 2) return HLWQ_ERR_BITS;
  if (c.n_pages < 0 || c.requests < 0 || c.kv_heads < 0 || c.n_residual < 0 || c.ring < c.n_residual)
    return HLWQ_ERR_SHAPE;
  if (c.page_size < 16 || c.page_size > 256 || (c.page_size & (c.page_size - 1))) return HLWQ_ERR_SHAPE;
  if (c.requests > kMaxRequests || c.kv_heads > kMaxHeads || c.n_pages > 0x7fffffff / c.page_size ||
      c.ring > 0x7fffffff)
    return HLWQ_ERR_LIMIT;
  int64_t vecs, ring, bytes;
  if (!mul_ok(c.n_pages * c.page_size, c.kv_heads, &vecs) || !mul_ok(vecs, 32 * c.bits, &bytes) ||
      !mul_ok(c.requests * c.kv_heads, c.ring, &ring) || !mul_ok(ring, 2 * kDim, &bytes))
    return HLWQ_ERR_SHAPE;
  for (const hlwq_kv_store* s : {&c.k, &c.v}) {
    if ((vecs > 0 && (!s->packed || !s->norms)) || (ring > 0 && !s->window)) return HLWQ_ERR_NULL;
    if (misaligned(s->packed, 16) || misaligned(s->norms, 16) || misaligned(s->window, 16)) return HLWQ_ERR_ALIGN;
    add_span(spans, s->packed, vecs, 32 * c.bits, written);
    add_span(spans, s->norms, vecs, 2, written);
    add_span(spans, s->window, ring, 2 * kDim, written);
  }
  return HLWQ_OK;
}

}  // namespace hlwq_kv
