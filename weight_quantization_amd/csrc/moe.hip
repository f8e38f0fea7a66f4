// moe.hip — a mixture-of-experts layer of a few tokens, from the codes of its
// banks (include/hlwq_moe.h).

#include "staging.h"

#include "hlwq_moe.h"

namespace hlwq_kv {
namespace {

typedef uint32_t u32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x3_4 __attribute__((ext_vector_type(3), aligned(4)));
typedef uint32_t u32x4_2 __attribute__((ext_vector_type(4), aligned(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));

constexpr int kBlock = 128;
constexpr int64_t kMaxExperts = 1024, kMaxTopK = 32, kMaxSize = 1 << 20, kMaxTokens = 1 << 24;
constexpr int kMaxPairs = 4096;  // (token, expert) pairs of one pass over the banks
constexpr int kTile = 16;        // rows of a matrix, and pairs, to a product

__device__ __forceinline__ int32_t quotient(int32_t a, int32_t b) {
  return static_cast<int32_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const f16x2 v = {static_cast<_Float16>(lo), static_cast<_Float16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

// ---------------------------------------------------------------------------
// Activations: rotated by blocks of 128 and rounded to fp16, a row over a power
// of two that brings its largest value to [1, 2) before the rotation; a rotated
// value is at most 128 times that, so it is held times 2^7 and stays below 2^15.
// ---------------------------------------------------------------------------

constexpr int kRotateThreads = 256;

// Largest magnitude of a row's n values, NaN and infinities left out, in every
// thread; at(i): values i and i + 1, i even.
template <class F>
__device__ __forceinline__ float row_top(F at, int32_t n, float* lds) {
  float top = 0;
#pragma unroll 4
  for (int32_t i = 2 * threadIdx.x; i < n; i += 2 * kRotateThreads) {
    const f32x2 v = at(i);
    const float x = fabsf(v[0]), y = fabsf(v[1]);
    top = fmaxf(top, fmaxf(x <= FLT_MAX ? x : 0.0f, y <= FLT_MAX ? y : 0.0f));
  }
  top = wave_max(top);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = top;
  __syncthreads();
  return fmaxf(fmaxf(lds[0], lds[1]), fmaxf(lds[2], lds[3]));
}

// A block of 128 held two values to a lane (2 l and 2 l + 1), unnormalised.
__device__ __forceinline__ void block_fwht(float (&x)[2], int lane) {
  const float a = x[0] + x[1], b = x[0] - x[1];
  x[0] = a;
  x[1] = b;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const bool upper = (lane & d) != 0;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float q = lane_xor(x[j], d);
      x[j] = upper ? q - x[j] : x[j] + q;
    }
  }
}

// (at least -110: the factors 2^(7 - e) and 2^(e - 14) are normal numbers, and exact)
__device__ __forceinline__ int scale_exponent(float top) { return top > 0 ? max(__builtin_amdgcn_frexp_expf(top) - 1, -110) : 0; }

template <class F>
__device__ __forceinline__ void rotate_row(F at, int32_t n, uint16_t* __restrict__ to, float* __restrict__ scale) {
  __shared__ float lds[kRotateThreads / 64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = scale_exponent(row_top(at, n, lds));
  const float f = __builtin_ldexpf(1.0f, 7 - e);
  if (threadIdx.x == 0) *scale = __builtin_ldexpf(1.0f, e - 7 - 7);  // and the blocks' 1 / 128
  const int32_t nb = static_cast<int32_t>(ceil_div(n, kBlock));
  for (int32_t b = wave; b < nb; b += kRotateThreads / 64) {
    const int32_t i = b * kBlock + 2 * lane;
    const f32x2 v = i < n ? at(i) : f32x2{0, 0};
    float x[2] = {v[0] * f, v[1] * f};
    block_fwht(x, lane);
    *reinterpret_cast<uint32_t*>(to + i) = pack_f16x2(x[0], x[1]);
  }
}

struct PrepareArgs {
  const uint16_t* x;
  int64_t x_stride;
  const uint16_t* router;  // null: the routing is known
  double* logits;          // [tokens][experts]
  uint16_t* rotated;       // [tokens][nb * 128]
  float* scale;            // [tokens]
  int32_t tokens, hidden, experts, expert_groups;
  int32_t rotating;  // workgroups that rotate: one a token, or none
};

// Router logits of some experts and tokens a wave, lanes along the row, eight
// values to a load.  Products of bf16 are exact in 64 bits, where they are summed:
// experts whose logits differ by less than fp32 resolves are told apart.
constexpr int kRouterWaves = kRotateThreads / 64;

template <int EXPERTS, int TOKENS>
__device__ __forceinline__ void router_logits(const PrepareArgs& a, int32_t e0, int32_t t0) {
  const int lane = threadIdx.x & 63;
  const uint16_t *r[EXPERTS], *x[TOKENS];
#pragma unroll
  for (int k = 0; k < EXPERTS; ++k) r[k] = a.router + static_cast<int64_t>(min(e0 + k, a.experts - 1)) * a.hidden;
#pragma unroll
  for (int j = 0; j < TOKENS; ++j) x[j] = a.x + min(t0 + j, a.tokens - 1) * a.x_stride;
  double sum[EXPERTS][TOKENS] = {};
  const int32_t whole = a.hidden & ~7;
#pragma unroll 2
  for (int32_t i = 8 * lane; i < whole; i += 512) {
    u32x4_2 rv[EXPERTS], xv[TOKENS];
#pragma unroll
    for (int k = 0; k < EXPERTS; ++k) rv[k] = *reinterpret_cast<const u32x4_2*>(r[k] + i);
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) xv[j] = *reinterpret_cast<const u32x4_2*>(x[j] + i);
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      double xd[TOKENS];
#pragma unroll
      for (int j = 0; j < TOKENS; ++j) xd[j] = w & 1 ? bf16_hi(xv[j][w >> 1]) : bf16_lo(xv[j][w >> 1]);
#pragma unroll
      for (int k = 0; k < EXPERTS; ++k) {
        const double rd = w & 1 ? bf16_hi(rv[k][w >> 1]) : bf16_lo(rv[k][w >> 1]);
#pragma unroll
        for (int j = 0; j < TOKENS; ++j) sum[k][j] = __builtin_fma(rd, xd[j], sum[k][j]);
      }
    }
  }
  if (const int32_t i = whole + lane; i < a.hidden)
#pragma unroll
    for (int k = 0; k < EXPERTS; ++k)
#pragma unroll
      for (int j = 0; j < TOKENS; ++j) sum[k][j] = __builtin_fma(static_cast<double>(bf16_lo(r[k][i])), static_cast<double>(bf16_lo(x[j][i])), sum[k][j]);
#pragma unroll
  for (int k = 0; k < EXPERTS; ++k)
#pragma unroll
    for (int j = 0; j < TOKENS; ++j) {
      const double s = wave_sum(sum[k][j]);
      if (lane == 0 && e0 + k < a.experts && t0 + j < a.tokens) a.logits[static_cast<int64_t>(t0 + j) * a.experts + e0 + k] = s;
    }
}
// Experts and tokens to a wave: more of them read and widen each value less often,
// fewer make more waves.  Measured (hidden 2048, the whole kernel, us; a layer of
// few experts loses up to 2.5 from 97 tokens on):
//   256 experts, tokens    2    8   17   32   48   64    96   128   192   512
//   1 x 2                3.6  4.3  4.8  6.4  7.9 10.0  13.0  15.8  21.9  51.8
//   2 x 2                4.1  4.4  5.0  5.7  6.8  8.7  10.7  13.0  17.4  38.7
//   4 x 4                6.8  7.1  7.0  7.2  7.9  8.3  10.1  10.5  13.7  27.9
//   128 experts
//   1 x 2                3.5  4.2  4.2  4.8  5.4  6.6   8.3  10.7  12.9  29.2
//   2 x 2                4.2  4.2  4.4  5.1  5.5  6.0   7.4   8.8  10.6  23.1
//   4 x 4                6.6  7.0  7.1  7.1  7.8  7.8   8.1   8.5  11.0  17.9
//   8 experts
//   1 x 2                3.6  4.3  4.1  4.2  4.2  4.3   4.5   4.4   4.5   5.8
//   2 x 2                3.6  4.3  4.5  4.3  4.2  4.2   5.0   4.4   4.8   6.2
//   4 x 4                5.8  6.2  6.6  6.7  6.7  6.8   6.8   6.9   6.8   9.0
struct RouterTile {
  int experts, tokens;
};
__host__ __device__ inline RouterTile router_tile(int64_t tokens) {
  if (tokens == 1) return {1, 1};
  if (tokens <= 32) return {1, 2};
  return tokens <= 96 ? RouterTile{2, 2} : RouterTile{4, 4};
}

// The first workgroups rotate a token each, the others take the router's.
__global__ void __launch_bounds__(kRotateThreads) hlwq_moe_prepare_kernel(const PrepareArgs a) {
  if (static_cast<int32_t>(blockIdx.x) < a.rotating) {
    const int32_t t = blockIdx.x;
    const uint16_t* row = a.x + t * a.x_stride;
    const int64_t pitch = ceil_div(a.hidden, kBlock) * kBlock;
    rotate_row(
        [row, n = a.hidden](int32_t i) {
          const float next = bf16_lo(row[min(i + 1, n - 1)]);
          return f32x2{bf16_lo(row[i]), i + 1 < n ? next : 0.0f};
        },
        a.hidden, a.rotated + t * pitch, a.scale + t);
    return;
  }
  const int32_t w = blockIdx.x - a.rotating;
  const RouterTile tile = router_tile(a.tokens);
  const int32_t e0 = (w % a.expert_groups * kRouterWaves + (threadIdx.x >> 6)) * tile.experts, t0 = w / a.expert_groups * tile.tokens;
  if (e0 >= a.experts) return;
  if (tile.tokens == 1)
    router_logits<1, 1>(a, e0, t0);
  else if (tile.experts == 1)
    router_logits<1, 2>(a, e0, t0);
  else if (tile.experts == 2)
    router_logits<2, 2>(a, e0, t0);
  else
    router_logits<4, 4>(a, e0, t0);
}

// ---------------------------------------------------------------------------
// The best experts of a token, a wave each: lane l holds experts l, l + 64, ..;
// top_k times the largest of the wave's, by the upper halves of the logits first.
// 4 to 5.4 us for 5 to 192 tokens, most of it a kernel's start.
// ---------------------------------------------------------------------------

struct TopArgs {
  const double* logits;
  int32_t* ids;
  float* weights;
  int32_t tokens, experts, top_k, renormalize;
};

// Order of 64-bit floats as that of unsigned numbers; NaN lowest, then minus infinity; never 0.
__device__ __forceinline__ uint64_t order_of(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 counts as 0
  if (v != v) return 1;
  return u >> 63 ? ~u : u | (uint64_t{1} << 63);
}
__device__ __forceinline__ double value_of(uint64_t key) {
  if (key == 1) return __builtin_nan("");
  return __builtin_bit_cast(double, key >> 63 ? key & ~(uint64_t{1} << 63) : ~key);
}
// The largest of the wave's, in every lane (running maxima towards the last lane).
__device__ __forceinline__ uint32_t top_of_wave(uint32_t v) {
  const auto step = [&](int from) { return static_cast<uint32_t>(from); };
  v = max(v, step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x111, 0xF, 0xF, false)));
  v = max(v, step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x112, 0xF, 0xF, false)));
  v = max(v, step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x114, 0xF, 0xF, false)));
  v = max(v, step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x118, 0xF, 0xF, false)));
  v = max(v, step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x142, 0xA, 0xF, false)));
  v = max(v, step(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0x143, 0xC, 0xF, false)));
  return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), 63));
}

// A wave finds a token's best: lane j < top_k gets the j-th.
struct Chosen {
  int32_t id;
  float weight;
};
template <int PER>
__device__ __forceinline__ Chosen choose(const double* __restrict__ row, int32_t experts, int32_t top_k, bool renormalize) {
  const int lane = threadIdx.x & 63;
  uint64_t key[PER], left[PER];
#pragma unroll
  for (int k = 0; k < PER; ++k) {
    key[k] = lane + 64 * k < experts ? order_of(row[lane + 64 * k]) : 0;
    left[k] = key[k];
  }
  uint64_t mine = 0;
  int32_t id = 0;
  for (int32_t j = 0; j < top_k; ++j) {
    uint64_t best = left[0];
    int32_t at = 0;
#pragma unroll
    for (int k = 1; k < PER; ++k) {
      at = left[k] > best ? k : at;
      best = max(best, left[k]);
    }
    const uint32_t hi = static_cast<uint32_t>(best >> 32);
    const uint32_t top = top_of_wave(hi);
    uint64_t who = __ballot(hi == top);
    int32_t lowest = 64 * at + lane;
    if (who & (who - 1)) {  // several: by their lower halves, then by index
      const uint32_t lo = hi == top ? static_cast<uint32_t>(best) : 0;
      const uint32_t low_top = top_of_wave(lo);
      who = __ballot(hi == top && lo == low_top);
      lowest = static_cast<int32_t>(~top_of_wave(who >> lane & 1 ? ~static_cast<uint32_t>(lowest) : 0u));
    } else {
      lowest = __builtin_amdgcn_readlane(lowest, __builtin_ctzll(who));
    }
    const int from = lowest & 63;
#pragma unroll
    for (int k = 0; k < PER; ++k) left[k] = lane == from && k == lowest >> 6 ? 0 : left[k];
    const uint64_t b = static_cast<uint64_t>(static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(hi), from))) << 32 |
                       static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(best)), from));
    if (lane == j) {
      mine = b;
      id = lowest;
    }
  }
  const double top = lane_value(value_of(mine), 0);
  const double w = lane < top_k ? exp(value_of(mine) - top) : 0.0;
  double total = w;
  if (!renormalize) {
    total = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k)
      if (key[k]) total += exp(value_of(key[k]) - top);
  }
  total = wave_sum(total);
  return Chosen{id, static_cast<float>(w / total)};
}

constexpr int kTopThreads = 256;
template <int PER>
__global__ void __launch_bounds__(kTopThreads) hlwq_moe_top_kernel(const TopArgs a) {
  const int lane = threadIdx.x & 63;
  const int32_t t = blockIdx.x * (kTopThreads / 64) + (threadIdx.x >> 6);
  if (t >= a.tokens) return;
  const Chosen c = choose<PER>(a.logits + static_cast<int64_t>(t) * a.experts, a.experts, a.top_k, a.renormalize);
  if (lane < a.top_k) {
    const int64_t p = static_cast<int64_t>(t) * a.top_k + lane;
    a.ids[p] = c.id;
    a.weights[p] = c.weight;
  }
}

// Tokens of no hidden values: all logits are 0.
__global__ void __launch_bounds__(kTopThreads) hlwq_moe_even_kernel(const TopArgs a) {
  const int64_t p = static_cast<int64_t>(blockIdx.x) * kTopThreads + threadIdx.x;
  if (p >= static_cast<int64_t>(a.tokens) * a.top_k) return;
  a.ids[p] = static_cast<int32_t>(p % a.top_k);
  a.weights[p] = static_cast<float>(1.0 / (a.renormalize ? a.top_k : a.experts));
}

// ---------------------------------------------------------------------------
// Products with an expert's codes, where the named experts are not many.  A
// workgroup takes the a-th of the experts that some pair names and some tiles of
// sixteen rows of its matrix (with GATED the same tile of gate and up); its waves
// split the blocks of a row, KS ways with BW at a time, or the tiles.  Per block and tile a lane
// holds 32 codes of one row, looks them up two at a time, and they meet sixteen
// pairs' activations in four matrix products; the norm of a row and block
// multiplies the result, where it is one value to a lane.  What bounds it are the
// loads, 20 bytes of another row to each lane, an address a cycle: all 256 experts of
// 2048 x 512 would take 143 + 62 us (64 tokens), where streaming takes 83 + 44.
// ---------------------------------------------------------------------------

constexpr int kProductThreads = 512, kProductWaves = kProductThreads / 64;

struct ProductArgs {
  const uint8_t* packed;
  const uint16_t* norms;
  const uint16_t* act;     // fp16 [.][nb * 128]
  const float* act_scale;  // [.]
  const int32_t* ids;      // [pairs]
  const float* weights;    // [pairs] (GATED)
  float* out;              // [pairs][n_out]
  uint16_t* rotated;       // [pairs][blocks of n_out * 128], where a workgroup rotates what it has
  float* rotated_scale;    // [pairs][blocks of n_out]
  int32_t pairs, experts, top_k;
  int32_t rows;   // of an expert's matrix
  int32_t n_out;  // of them outputs: rows, or half of them
  int32_t nb;     // blocks to a row
  int32_t tiles;  // of outputs, a pair of row tiles each
  int32_t activation;
};

template <int BITS>
struct RowCodes;
template <>
struct RowCodes<5> {
  u32x4_4 a;
  uint32_t b;
};
template <>
struct RowCodes<3> {
  u32x3_4 a;
};
__device__ __forceinline__ void load_row(RowCodes<5>& c, const uint8_t* p) {
  c.a = *reinterpret_cast<const u32x4_4*>(p);
  c.b = *reinterpret_cast<const uint32_t*>(p + 16);
}
__device__ __forceinline__ void load_row(RowCodes<3>& c, const uint8_t* p) { c.a = *reinterpret_cast<const u32x3_4*>(p); }
__device__ __forceinline__ uint32_t word_of(const RowCodes<5>& c, int i) { return i < 4 ? c.a[i] : c.b; }
__device__ __forceinline__ uint32_t word_of(const RowCodes<3>& c, int i) { return c.a[i]; }
__device__ __forceinline__ void set_word(RowCodes<5>& c, int i, uint32_t v) {
  if (i < 4)
    c.a[i] = v;
  else
    c.b = v;
}
__device__ __forceinline__ void set_word(RowCodes<3>& c, int i, uint32_t v) { c.a[i] = v; }

// The book in LDS: pairs of centroids, looked up by two codes at once.  Of 3-bit
// codes 64 of them, in 32 copies side by side, one for each bank; of 5-bit codes
// 1024 in two copies, whose look-ups meet in the banks: 7.5 cycles of the CU each
// (4.5 with sixteen copies, 64 KB; single codes, 32 values whose 16 words meet
// never, under 3, but two of them and their packing take longer).
template <int BITS>
struct Book {
  static constexpr int kShift = BITS == 5 ? 1 : 5;  // 2^this copies
  static constexpr uint32_t kBytes = (4u << (2 * BITS)) << kShift;
  static constexpr int kTo = 2 + kShift;  // where a look-up's bits begin in an address
  static constexpr uint32_t kMask = ((1u << (2 * BITS)) - 1) << kTo;
};

// The bits of a row's codes from `bit` on (at least `count` of them), from bit `to`
// of the result on.
template <int BITS>
__device__ __forceinline__ uint32_t bits_at(const RowCodes<BITS>& c, int bit, int count, int to) {
  const int at = bit >> 5, s = bit & 31;
  if (s + count > 32) return __builtin_amdgcn_alignbit(word_of(c, at + 1), word_of(c, at), s - to);
  return s >= to ? word_of(c, at) >> (s - to) : word_of(c, at) << (to - s);
}

// Four 5-bit codes, the low 20 bits of v, to four centroids without LDS: spread to
// bytes, each the place k of its size among sixteen (k counted from the middle, so
// downwards below it); the high and the low bytes of the fp16 sizes picked from two
// eights each, and the sign put to the high ones.
struct Sizes5 {
  static constexpr float c[32] = HLWQ_CENTROIDS_5;
  static constexpr uint32_t word(int first, int shift) {
    uint32_t w = 0;
    for (int i = 0; i < 4; ++i) w |= ((__builtin_bit_cast(uint16_t, static_cast<_Float16>(c[16 + first + i])) >> shift) & 0xffu) << (8 * i);
    return w;
  }
};
__device__ __forceinline__ u32x2 four_centroids(uint32_t v) {
  const uint32_t t = __builtin_amdgcn_bitop3_b32(v, v << 6, 0x3ffu, 0xE4);       // c ? a : b
  const uint32_t k = __builtin_amdgcn_bitop3_b32(t, t << 3, 0x00ff00ffu, 0xE4);  // a code a byte, above it bits of others
  const uint32_t upper = k & 0x10101010u;
  const uint32_t size = __builtin_amdgcn_bitop3_b32(k, upper - (upper >> 4), 0x0f0f0f0fu, 0x82);  // ~(a ^ b) & c
  const uint32_t in8 = size & 0x07070707u;
  const uint32_t which = __builtin_amdgcn_bitop3_b32(size >> 1, 0x04040404u, 0x03020100u, 0xEA);  // (a & b) | c
  uint32_t hi = __builtin_amdgcn_perm(__builtin_amdgcn_perm(Sizes5::word(12, 8), Sizes5::word(8, 8), in8),
                                      __builtin_amdgcn_perm(Sizes5::word(4, 8), Sizes5::word(0, 8), in8), which);
  const uint32_t lo = __builtin_amdgcn_perm(__builtin_amdgcn_perm(Sizes5::word(12, 0), Sizes5::word(8, 0), in8),
                                            __builtin_amdgcn_perm(Sizes5::word(4, 0), Sizes5::word(0, 0), in8), which);
  hi = __builtin_amdgcn_bitop3_b32(hi, upper << 3, 0x80808080u, 0xF2);  // a | (~b & c)
  return u32x2{__builtin_amdgcn_perm(hi, lo, 0x05010400u), __builtin_amdgcn_perm(hi, lo, 0x07030602u)};
}

// Two 3-bit codes, the low six bits of v, to two centroids.
struct Values3 {
  static constexpr float c[8] = HLWQ_CENTROIDS_3;
  static constexpr uint32_t word(int first, int shift) {
    uint32_t w = 0;
    for (int i = 0; i < 4; ++i) w |= ((__builtin_bit_cast(uint16_t, static_cast<_Float16>(c[first + i])) >> shift) & 0xffu) << (8 * i);
    return w;
  }
};
__device__ __forceinline__ uint32_t two_centroids(uint32_t v) {
  const uint32_t at = (v & 7u) | (v << 5 & 0x700u);
  const uint32_t hi = __builtin_amdgcn_perm(Values3::word(4, 8), Values3::word(0, 8), at);
  const uint32_t lo = __builtin_amdgcn_perm(Values3::word(4, 0), Values3::word(0, 0), at);
  return __builtin_amdgcn_perm(hi, lo, 0x05010400u);
}

// 32 codes to four operands of eight centroids.
template <int BITS, int WITHOUT = 0>
__device__ __forceinline__ void decode(const RowCodes<BITS>& c, const uint8_t* book, uint32_t copy, u32x4 (&w)[4]) {
  using K = Book<BITS>;
#pragma unroll
  for (int p = 2 * WITHOUT; p < 16; ++p)
    w[p >> 2][p & 3] = *reinterpret_cast<const uint32_t*>(book + ((bits_at<BITS>(c, 2 * BITS * p, 2 * BITS, K::kTo) & K::kMask) | copy));
#pragma unroll
  for (int g = 0; g < WITHOUT; ++g) {
    const u32x2 v = four_centroids(bits_at<BITS>(c, 4 * BITS * g, 4 * BITS, 0));
    w[g >> 1][2 * (g & 1)] = v[0];
    w[g >> 1][2 * (g & 1) + 1] = v[1];
  }
}

template <int BITS>
__device__ __forceinline__ uint32_t book_copy(int lane) {
  return (lane & ((1 << Book<BITS>::kShift) - 1)) * 4;
}

__device__ __forceinline__ float sigmoid_times(float g, float z) { return g / (1.0f + __builtin_amdgcn_exp2f(-1.44269504088896340736f * z)); }
__device__ __forceinline__ float activate(float g, int32_t kind) {
  // gelu's g / 2 (1 + tanh(z)) is g / (1 + exp(-2 z))
  return sigmoid_times(g, kind == HLWQ_ACT_SILU ? g : 1.5957691216057308f * (g + 0.044715f * g * g * g));
}

// The book filled, from registers: with tables read from memory the banks' kernels
// took 0.4 us more.
template <int BITS>
__device__ __forceinline__ void fill_book(uint8_t* book) {
  static_assert(Book<BITS>::kBytes == 16 * kProductThreads, "four words a thread");
  if constexpr (BITS == 5) {
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) {
      const uint32_t p = i * kProductThreads + threadIdx.x, v = four_centroids(p)[0];
      reinterpret_cast<u32x2*>(book)[p] = u32x2{v, v};
    }
  } else {
    const uint32_t v = two_centroids(threadIdx.x >> 3);
    reinterpret_cast<u32x4*>(book)[threadIdx.x] = u32x4{v, v, v, v};
  }
}

// The a-th expert that some pair names, or -1; its pairs, in any order, to `list`.
struct Expert {
  int32_t id, count;
};
__device__ __forceinline__ Expert find_expert(const ProductArgs& a, int32_t slot, int32_t* list, uint32_t* named, int32_t* count_of) {
  const int lane = threadIdx.x & 63;
  if (threadIdx.x < kMaxExperts / 32) named[threadIdx.x] = 0;
  if (threadIdx.x == 0) *count_of = 0;
  __syncthreads();
  int32_t id[kMaxPairs / kProductThreads];
#pragma unroll
  for (int k = 0; k < kMaxPairs / kProductThreads; ++k) {
    const int32_t p = threadIdx.x + k * kProductThreads;
    id[k] = p < a.pairs ? a.ids[p] : -1;
    if (id[k] >= a.experts) id[k] = -1;
    if (id[k] >= 0) atomicOr(&named[id[k] >> 5], 1u << (id[k] & 31));
  }
  __syncthreads();
  uint32_t word = lane < kMaxExperts / 32 ? named[lane] : 0;
  const int32_t upto = wave_scan(static_cast<int32_t>(__builtin_popcount(word)));
  const uint64_t past = __ballot(upto > slot);
  if (!past) return Expert{-1, 0};
  const int at = __builtin_ctzll(past);
  word = __builtin_amdgcn_readlane(word, at);
  int32_t skip = slot - (__builtin_amdgcn_readlane(upto, at) - __builtin_popcount(word));
  for (; skip > 0; --skip) word &= word - 1;
  const int32_t expert = 32 * at + __builtin_ctz(word);
#pragma unroll
  for (int k = 0; k < kMaxPairs / kProductThreads; ++k)
    if (id[k] == expert) list[atomicAdd(count_of, 1)] = threadIdx.x + k * kProductThreads;
  __syncthreads();
  return Expert{expert, *count_of};
}

template <int BITS, int KS, int BW, bool GATED>
__global__ void __launch_bounds__(kProductThreads) hlwq_moe_product_kernel(const ProductArgs a) {
  constexpr int kGroups = kProductWaves / KS;  // of waves, a tile each
  constexpr int kPitch = 20;                   // floats to a pair's sums of a tile
  __shared__ __attribute__((aligned(16))) uint8_t book[Book<BITS>::kBytes];
  __shared__ int32_t list[kMaxPairs];
  __shared__ uint32_t named[kMaxExperts / 32];
  __shared__ int32_t count_of;
  __shared__ float sums[kProductWaves][2][kTile * kPitch];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);

  fill_book<BITS>(book);
  const Expert ex = find_expert(a, blockIdx.y, list, named, &count_of);
  if (ex.id < 0) return;
  const int32_t expert = ex.id, count = ex.count;

  const int r = lane & 15, h4 = lane >> 4;
  const int ks = wave % KS, group = wave / KS;
  const uint32_t copy = book_copy<BITS>(lane);
  const uint8_t* packed = a.packed + static_cast<int64_t>(expert) * a.rows * a.nb * (16 * BITS);
  const uint16_t* norms = a.norms + static_cast<int64_t>(expert) * a.rows * a.nb;
  const int32_t pitch = a.nb * kBlock;

  for (int32_t c0 = 0; c0 < count; c0 += kTile) {
    const int32_t pair = c0 + r < count ? list[c0 + r] : -1;
    const uint16_t* act = a.act + static_cast<int64_t>(GATED ? max(pair, 0) / a.top_k : max(pair, 0)) * pitch + 32 * h4;
    for (int32_t tile0 = blockIdx.x * kGroups; tile0 < a.tiles; tile0 += gridDim.x * kGroups) {
      const int32_t tile = tile0 + group;
      f32x4 acc[2] = {};
      if (tile < a.tiles) {
        const int32_t first[2] = {GATED ? tile * kTile : 2 * tile * kTile, GATED ? a.n_out + tile * kTile : (2 * tile + 1) * kTile};
        uint32_t row[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) row[m] = min(first[m] + r, a.rows - 1) * a.nb;
        for (int32_t b0 = ks * BW; b0 < a.nb; b0 += KS * BW) {
          RowCodes<BITS> codes[BW][2];
          float norm[BW][2];
          u32x4 x[BW][4];
#pragma unroll
          for (int k = 0; k < BW; ++k)
            if (b0 + k < a.nb) {
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                load_row(codes[k][m], packed + static_cast<uint64_t>(row[m] + b0 + k) * (16 * BITS) + 4 * BITS * h4);
                norm[k][m] = f16_value(norms[row[m] + b0 + k]);
              }
#pragma unroll
              for (int j = 0; j < 4; ++j)
                x[k][j] = pair >= 0 ? *reinterpret_cast<const u32x4*>(act + (b0 + k) * kBlock + 8 * j) : u32x4{0, 0, 0, 0};
            }
#pragma unroll
          for (int k = 0; k < BW; ++k)
            if (b0 + k < a.nb) {
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                u32x4 w[4];
                decode<BITS>(codes[k][m], book, copy, w);
                f32x4 d = {0, 0, 0, 0};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                  d = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x[k][j]), __builtin_bit_cast(f16x8, w[j]), d, 0, 0, 0);
                acc[m] += d * norm[k][m];
              }
            }
        }
      }
      // pairs 4 h4 + i of row r: the waves that split the blocks join
      __syncthreads();
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i) sums[wave][m][(4 * h4 + i) * kPitch + r] = acc[m][i];
      __syncthreads();
      for (int32_t i = threadIdx.x; i < kGroups * kTile * kTile; i += kProductThreads) {
        const int32_t g = i / (kTile * kTile), c = i / kTile % kTile, rr = i % kTile;
        if (tile0 + g >= a.tiles || c0 + c >= count) continue;
        const int32_t p = list[c0 + c];
        float s[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int m = 0; m < 2; ++m) s[m] += sums[g * KS + k][m][c * kPitch + rr];
        const float scale = a.act_scale[GATED ? p / a.top_k : p];
        float* out = a.out + static_cast<int64_t>(p) * a.n_out;
        if constexpr (GATED) {
          const int32_t o = (tile0 + g) * kTile + rr;
          if (o < a.n_out) out[o] = activate(s[0] * scale, a.activation) * (s[1] * scale) * a.weights[p];
        } else {
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const int32_t o = (2 * (tile0 + g) + m) * kTile + rr;
            if (o < a.n_out) out[o] = s[m] * scale;
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The same where the touched experts are many.  A workgroup a CU takes an equal
// run of (expert, 128 rows of gate and of up, or 256 of down), a wave a pair of
// row tiles of each, whose blocks it goes through from first to last, so that no
// sums are joined.  The codes come straight to LDS, four blocks of both tiles at a
// time, the next four as soon as these are in registers: four lanes fetch 64
// bytes of a row side by side (each lane its own 20 bytes of another row, straight
// to registers, is an address a cycle, and took twice as long), and 16-byte pieces
// are turned by the row so that the dwords that the lanes then read lie in
// different banks.  Inner values are rotated before they leave, over a power of
// two for each block (act_scale [.][nb]).
//
// Measured (256 experts, hidden 2048, inner 512, 5 bits): gate and up 83 us for 64
// tokens (298 MB of codes and norms) and 104 for 192 (344 MB), down 44 and 50: 5 TB/s
// while every CU has a set, of which LDS look-ups take a third of the cycles and
// VALU another; without work the kernel takes 4.  17 tokens at 3 bits 33 and 20.
// ---------------------------------------------------------------------------

constexpr int kWorkgroups = 256;
constexpr int kMaxInnerBlocks = 64;  // whose scales a workgroup keeps
// Of activations in LDS.  (40 KB, and four copies of the pairs of 5-bit codes, took 2%
// less for 64 and 192 tokens of 256 experts; but busier experts take passes more.)
constexpr int kActBytes = 48 << 10;
// Pairs of a pass over an expert's codes, of rows of nb blocks: sixteen up to 1536
// values, 12 at 2048, 6 at 4096, 4 at 5120, one past 12288.
__host__ __device__ inline int32_t pass_pairs(int64_t nb) { return static_cast<int32_t>(nb * 256 * kTile <= kActBytes ? kTile : kActBytes / (nb * 256)); }
constexpr int kChunk = 4;            // blocks that are staged together
constexpr int kWithoutBook = 1;      // fours of 32 5-bit codes whose centroids come from registers

template <int BITS>
struct StreamLds {
  static constexpr uint32_t codes = 1024 * BITS, norms = 2 * codes, wave = norms + 2 * 256;  // of a wave: two tiles' codes, their norms
  static constexpr uint32_t book = 0, stage = Book<BITS>::kBytes, act = stage + kProductWaves * wave,
                            inner = act + kActBytes, list = inner + kTile * (kBlock + 4) * 4, bytes = list + kMaxPairs * 2;
};

template <int BITS, bool GATED>
__global__ void __launch_bounds__(kProductThreads, 2) hlwq_moe_stream_kernel(const ProductArgs a) {
  using L = StreamLds<BITS>;
  constexpr int kPitch = kBlock + 4;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[L::bytes];
  __shared__ __attribute__((aligned(16))) uint32_t named[kMaxExperts / 2];  // pairs of two experts
  __shared__ int32_t counts[64];
  static_assert(kMaxPairs == 64 * 64, "a count for each wave's ballot");
  static_assert(kMaxInnerBlocks * kTile <= kTile * kPitch, "scales lie where inner values do");
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
  float* const inner = reinterpret_cast<float*>(lds + L::inner);
  uint16_t* const list = reinterpret_cast<uint16_t*>(lds + L::list);
  const int r = lane & 15, h4 = lane >> 4;
  const uint32_t copy = book_copy<BITS>(lane);

  const int32_t sets = a.tiles;  // of 128 or 256 rows
  const int32_t capacity = pass_pairs(a.nb);

  // The experts' pairs, and this workgroup's run of (expert, pass over as many of
  // its pairs as fit, set): passes cost the same whatever their pairs.
  static_assert(kMaxExperts == 64 * 16 && kMaxPairs < 0x10000, "sixteen experts a lane, two counts a word");
  int32_t id[kMaxPairs / kProductThreads];
#pragma unroll
  for (int k = 0; k < kMaxPairs / kProductThreads; ++k) {
    const int32_t p = threadIdx.x + k * kProductThreads;
    id[k] = p < a.pairs ? a.ids[p] : -1;
  }
  for (int i = threadIdx.x; i < kMaxExperts / 2; i += kProductThreads) named[i] = 0;
  fill_book<BITS>(lds + L::book);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kMaxPairs / kProductThreads; ++k) {
    if (id[k] >= a.experts) id[k] = -1;
    if (id[k] >= 0) atomicAdd(&named[id[k] >> 1], 1u << 16 * (id[k] & 1));
  }
  __syncthreads();
  const float per_pass = 1.0f / capacity;
  // (counts are small: the quotient's error stays under the half that is added)
  const auto passes_of = [&](uint32_t count) { return static_cast<int32_t>((count + (capacity - 0.5f)) * per_pass); };
  const auto count_at = [&](int32_t e) { return named[e >> 1] >> 16 * (e & 1) & 0xffffu; };
  int32_t own = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t both = named[8 * lane + i];
    own += passes_of(both & 0xffffu) + passes_of(both >> 16);
  }
  const int32_t upto = wave_scan(own);
  const uint64_t total = static_cast<uint64_t>(__builtin_amdgcn_readlane(upto, 63)) * static_cast<uint32_t>(sets);
  static_assert(kWorkgroups == 256, "");
  int32_t q = static_cast<int32_t>(total * blockIdx.x >> 8);
  const int32_t q_end = static_cast<int32_t>(total * (blockIdx.x + 1) >> 8);

  const uint32_t row_bytes = a.nb * (16 * BITS);
  const int32_t chunks = static_cast<int32_t>(ceil_div(a.nb, kChunk)), pitch = a.nb * kBlock;
  const uint32_t my = base + L::stage + wave * L::wave;
  // where dword d of a lane's codes of block k lies in a tile's stage
  uint32_t place[kChunk][BITS];
#pragma unroll
  for (int k = 0; k < kChunk; ++k)
#pragma unroll
    for (int d = 0; d < BITS; ++d) {
      const int g = 4 * BITS * k + BITS * h4 + d;
      place[k][d] = my + (g >> 4) * 1024 + r * 64 + (((g >> 2) & 3) ^ (r >> 2)) * 16 + (g & 3) * 4;
    }
  const auto row_of = [&](int32_t set, int m, int i) {
    const int32_t o = (set * kProductWaves + wave) * (GATED ? kTile : 2 * kTile);
    return min(o + i + (GATED ? m * a.n_out : m * kTile), a.rows - 1);
  };

  int32_t listed = -1;
  while (q < q_end) {
    const int32_t slot = q / sets, set0 = q - slot * sets, set1 = min(sets, set0 + q_end - q);
    q += set1 - set0;
    const int at = __builtin_ctzll(__ballot(upto > slot));
    const int32_t rest = slot - __builtin_amdgcn_readlane(upto - own, at);
    const int32_t its = lane < 16 ? passes_of(count_at(16 * at + lane)) : 0, its_upto = wave_scan(its);
    const int within = __builtin_ctzll(__ballot(its_upto > rest));
    const int32_t expert = 16 * at + within, c0 = (rest - __builtin_amdgcn_readlane(its_upto - its, within)) * capacity;
    const int32_t columns = min(capacity, static_cast<int32_t>(count_at(expert)) - c0);
    const int64_t first = static_cast<int64_t>(expert) * a.rows * a.nb, blocks = static_cast<int64_t>(a.rows) * a.nb;
    const u32x4 codes = buffer_of(a.packed + first * (16 * BITS), blocks * (16 * BITS)), norms = buffer_of(a.norms + first, 2 * blocks);
    const auto stage = [&](int32_t set, int32_t chunk) {
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t row = row_of(set, m, lane >> 2);
        const uint32_t from = row * row_bytes + chunk * (kChunk * 16 * BITS) + 16 * ((lane & 3) ^ (lane >> 4));
#pragma unroll
        for (int i = 0; i < BITS; ++i) stage16(codes, from + 64 * i, my + m * L::codes + i * 1024);
        stage4(norms, ((2 * (row * a.nb + chunk * kChunk)) & ~3u) + 4 * (lane & 3), my + L::norms + m * 256);
      }
    };
    const auto idle = [&](int32_t set) { return (set * kProductWaves + wave) * (GATED ? kTile : 2 * kTile) >= a.n_out; };
    if (!idle(set0)) stage(set0, 0);

    // the expert's pairs in order, as other workgroups may take other passes of them
    barrier();
    if (expert != listed) {
      uint64_t mine[kMaxPairs / kProductThreads];
#pragma unroll
      for (int k = 0; k < kMaxPairs / kProductThreads; ++k) {
        mine[k] = __ballot(id[k] == expert);
        if (lane == 0) counts[k * kProductWaves + wave] = __builtin_popcountll(mine[k]);
      }
      wait_lds();
      barrier();
      const int32_t all = counts[lane], before = wave_scan(all) - all;
#pragma unroll
      for (int k = 0; k < kMaxPairs / kProductThreads; ++k)
        if (id[k] == expert)
          list[__builtin_amdgcn_readlane(before, k * kProductWaves + wave) + __builtin_popcountll(mine[k] & ((uint64_t{1} << lane) - 1))] =
              static_cast<uint16_t>(threadIdx.x + k * kProductThreads);
      wait_lds();
      barrier();
      listed = expert;
    }
    for (int32_t c = wave; c < columns; c += kProductWaves) {
      const int32_t pair = __builtin_amdgcn_readfirstlane(list[c0 + c]);
      const uint16_t* from = a.act + static_cast<int64_t>(GATED ? quotient(pair, a.top_k) : pair) * pitch;
      for (int32_t piece = lane; piece < a.nb * 16; piece += 64) {
        const int32_t at_j = (piece & ~15) + (piece & 3) * 4 + (piece >> 2 & 3);  // pieces of 16 bytes: block, h4, j to block, j, h4
        lds_put<u32x4>(base + L::act + (at_j * columns + c) * 16, *reinterpret_cast<const u32x4*>(from + 8 * piece));
      }
    }
    float pair_scale[4], pair_weight[4];  // of the lane's four
    if constexpr (GATED)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int32_t pair = list[c0 + min(4 * h4 + i, columns - 1)];
        pair_scale[i] = a.act_scale[quotient(pair, a.top_k)];
        pair_weight[i] = a.weights[pair];
      }
    if constexpr (!GATED)
      for (int32_t i = threadIdx.x; i < a.nb * kTile; i += kProductThreads) {
        const int32_t c = i & (kTile - 1);
        inner[i] = c < columns ? a.act_scale[static_cast<int64_t>(list[c0 + c]) * a.nb + (i >> 4)] : 0.0f;
      }
    wait_lds();
    barrier();
    const uint32_t act = base + L::act + (h4 * columns + min(r, columns - 1)) * 16;

    for (int32_t set = set0; set < set1; ++set) {
      f32x4 acc[2] = {};
      if (!idle(set)) {
        uint32_t norm_at[2];
#pragma unroll
        for (int m = 0; m < 2; ++m) norm_at[m] = my + L::norms + m * 256 + r * 16 + 2 * ((row_of(set, m, r) * a.nb) & 1);
        for (int32_t chunk = 0; chunk < chunks; ++chunk) {
          wait_staged();
          RowCodes<BITS> code[2][kChunk];
          float norm[2][kChunk];
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int k = 0; k < kChunk; ++k) {
#pragma unroll
              for (int d = 0; d < BITS; ++d) set_word(code[m][k], d, lds_at<uint32_t>(place[k][d] + m * L::codes));
              norm[m][k] = f16_value(lds_at<uint16_t>(norm_at[m] + 2 * k));
            }
          wait_lds();
          if (chunk + 1 < chunks)
            stage(set, chunk + 1);
          else if (set + 1 < set1 && !idle(set + 1))
            stage(set + 1, 0);
          // Unit u: block u / 2, tile u % 2.  The look-ups of the next unit are under
          // way while one is multiplied.
          u32x4 x[2][4], w[2][4];
          f32x4 scale[2];
          const auto look = [&](int u) {
            const int k = u >> 1;
            if ((u & 1) == 0) {
              const int32_t b = chunk * kChunk + k;
#pragma unroll
              for (int j = 0; j < 4; ++j) x[k & 1][j] = lds_at<u32x4>(act + (b * 4 + j) * 64 * columns);
              if constexpr (!GATED) scale[k & 1] = *reinterpret_cast<const f32x4*>(inner + b * kTile + 4 * h4);
            }
            decode<BITS, BITS == 5 ? kWithoutBook : 0>(code[u & 1][k], lds + L::book, copy, w[u & 1]);
            __builtin_amdgcn_sched_barrier(0);
          };
          const auto multiply = [&](int u) {
            const int k = u >> 1, m = u & 1;
            f32x4 d = {0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              d = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, x[k & 1][j]), __builtin_bit_cast(f16x8, w[m][j]), d, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[m][i] = __builtin_fmaf(d[i], GATED ? norm[m][k] : scale[k & 1][i] * norm[m][k], acc[m][i]);
            __builtin_amdgcn_sched_barrier(0);
          };
          const int32_t there = min(a.nb - chunk * kChunk, kChunk);
          if (there == kChunk) {
            look(0);
#pragma unroll
            for (int u = 0; u < 2 * kChunk; ++u) {
              if (u + 1 < 2 * kChunk) look(u + 1);
              multiply(u);
            }
          } else {
#pragma unroll
            for (int u = 0; u < 2 * (kChunk - 1); ++u)
              if (u < 2 * there) {
                look(u);
                multiply(u);
              }
          }
        }
      }
      const int32_t out0 = (set * kProductWaves + wave) * (GATED ? kTile : 2 * kTile);
      if constexpr (GATED) {
        barrier();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int32_t c = 4 * h4 + i;
          float v = 0;
          if (c < columns && out0 + r < a.n_out)
            v = activate(acc[0][i] * pair_scale[i], a.activation) * (acc[1][i] * pair_scale[i]) * pair_weight[i];
          inner[c * kPitch + wave * kTile + r] = v;
        }
        wait_lds();
        barrier();
        for (int32_t c = wave; c < columns; c += kProductWaves) {
          const float2 v = *reinterpret_cast<const float2*>(inner + c * kPitch + 2 * lane);
          float y[2] = {v.x, v.y};
          const float y0 = fabsf(y[0]) <= FLT_MAX ? fabsf(y[0]) : 0.0f, y1 = fabsf(y[1]) <= FLT_MAX ? fabsf(y[1]) : 0.0f;
          const int e = scale_exponent(wave_max(fmaxf(y0, y1)));
          const float f = __builtin_ldexpf(1.0f, 7 - e);
          y[0] *= f;
          y[1] *= f;
          block_fwht(y, lane);
          const int64_t to = static_cast<int64_t>(list[c0 + c]) * sets + set;
          *reinterpret_cast<uint32_t*>(a.rotated + to * kBlock + 2 * lane) = pack_f16x2(y[0], y[1]);
          if (lane == 0) a.rotated_scale[to] = __builtin_ldexpf(1.0f, e - 14);
        }
      } else {
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int32_t o = out0 + m * kTile + r;
          if (o >= a.n_out) continue;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int32_t c = 4 * h4 + i;
            if (c < columns) a.out[static_cast<int64_t>(list[c0 + c]) * a.n_out + o] = acc[m][i];
          }
        }
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The same for a few pairs, where what counts is how many kernels follow each
// other and what each waits for: the first finds its token's experts by itself
// (every workgroup again, from the logits) and rotates its activations while it
// does, the second rotates the inner values and joins a token's pairs.  A
// workgroup takes sixteen rows; its waves split the blocks of one pair, or the
// pairs.  All sixteen rows of the activations' operand are the same pair's.
//
// Measured (one token, 8 of 256 experts, hidden 2048, inner 512, 5 bits, 16 MB): 11.7
// us, of which 2.9 are the choice and 4.1 the start, and 7.5.  What bounds them is
// latency and the fetching of code that runs once: centroids from registers
// instead of the book, and loops instead of unrolled blocks, change nothing.
// ---------------------------------------------------------------------------

constexpr int kFewPairs = 32, kFewBlocks = 64;

struct FewArgs {
  ProductArgs p;
  const uint16_t* x;
  int64_t x_stride;
  const double* logits;  // null: the routing is known
  int32_t* ids;
  float* weights;
  float* h;       // [pairs][inner]
  uint16_t* out;  // [tokens][hidden]
  int32_t hidden, inner, renormalize, tokens;
};

// A block of values v[2 l], v[2 l + 1] rotated to LDS as fp16 over a power of two,
// which is returned (with the blocks' 1 / 128).
__device__ __forceinline__ float rotate_block(float (&v)[2], uint16_t* to, int lane) {
  const float a = fabsf(v[0]) <= FLT_MAX ? fabsf(v[0]) : 0.0f, b = fabsf(v[1]) <= FLT_MAX ? fabsf(v[1]) : 0.0f;
  const int e = scale_exponent(wave_max(fmaxf(a, b)));
  const float f = __builtin_ldexpf(1.0f, 7 - e);
  v[0] *= f;
  v[1] *= f;
  block_fwht(v, lane);
  *reinterpret_cast<uint32_t*>(to + 2 * lane) = pack_f16x2(v[0], v[1]);
  return __builtin_ldexpf(1.0f, e - 14);
}

// A block's products of a row tile with the activations at `act`: lane r has row r's.
template <int BITS>
__device__ __forceinline__ float few_product(const RowCodes<BITS>& c, const uint8_t* book, uint32_t copy, const uint16_t* act) {
  u32x4 w[4];
  decode<BITS>(c, book, copy, w);
  f32x4 d = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 4; ++j)
    d = __builtin_amdgcn_mfma_f32_16x16x32_f16(*reinterpret_cast<const f16x8*>(act + 8 * j), __builtin_bit_cast(f16x8, w[j]), d, 0, 0, 0);
  return d[0];
}

template <int BITS, int PER>
__global__ void __launch_bounds__(kProductThreads) hlwq_moe_few_up_kernel(const FewArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t book[Book<BITS>::kBytes];
  __shared__ __attribute__((aligned(16))) uint16_t act[kFewBlocks * kBlock];
  __shared__ float scales[kFewBlocks];
  __shared__ Chosen chosen;
  __shared__ float sums[kProductWaves][2][kTile];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h4 = lane >> 4;
  const int32_t pair = blockIdx.y, t = quotient(pair, a.p.top_k), j = pair - t * a.p.top_k;
  if (a.logits) {
    if (wave == kProductWaves - 1) {
      const Chosen c = choose<PER>(a.logits + static_cast<int64_t>(t) * a.p.experts, a.p.experts, a.p.top_k, a.renormalize);
      if (lane == j) chosen = c;
      if (blockIdx.x == 0 && j == 0 && lane < a.p.top_k) {
        a.ids[pair + lane] = c.id;
        a.weights[pair + lane] = c.weight;
      }
    }
  } else if (threadIdx.x == 0) {
    chosen = Chosen{a.ids[pair], a.weights[pair]};
  }
  fill_book<BITS>(book);
  const uint16_t* x = a.x + t * a.x_stride;
  for (int32_t b = wave; b < a.p.nb; b += kProductWaves) {
    const int32_t i = b * kBlock + 2 * lane;
    float v[2] = {i < a.hidden ? bf16_lo(x[i]) : 0.0f, i + 1 < a.hidden ? bf16_lo(x[i + 1]) : 0.0f};
    const float scale = rotate_block(v, act + b * kBlock, lane);
    if (lane == 0) scales[b] = scale;
  }
  __syncthreads();
  const Chosen c = chosen;
  const int32_t expert = __builtin_amdgcn_readfirstlane(c.id);
  if (expert < 0 || expert >= a.p.experts) return;
  const int32_t out0 = blockIdx.x * kTile;
  const uint32_t copy = book_copy<BITS>(lane);
  const uint8_t* codes[2];
  const uint16_t* norms[2];
#pragma unroll
  for (int m = 0; m < 2; ++m) {
    const int64_t at = (static_cast<int64_t>(expert) * a.p.rows + min(out0 + r + m * a.p.n_out, a.p.rows - 1)) * a.p.nb;
    codes[m] = a.p.packed + at * (16 * BITS) + 4 * BITS * h4;
    norms[m] = a.p.norms + at;
  }
  float acc[2] = {0, 0};
  constexpr int kAhead = 3;  // blocks whose codes are under way together
  for (int32_t b0 = wave; b0 < a.p.nb; b0 += kAhead * kProductWaves) {
    RowCodes<BITS> code[kAhead][2];
    float norm[kAhead][2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int32_t b = b0 + k * kProductWaves;
      if (b >= a.p.nb) break;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        load_row(code[k][m], codes[m] + b * (16 * BITS));
        norm[k][m] = f16_value(norms[m][b]);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int32_t b = b0 + k * kProductWaves;
      if (b >= a.p.nb) break;
#pragma unroll
      for (int m = 0; m < 2; ++m)
        acc[m] = __builtin_fmaf(few_product<BITS>(code[k][m], book, copy, act + b * kBlock + 32 * h4), norm[k][m] * scales[b], acc[m]);
    }
  }
  if (lane < kTile) {
    sums[wave][0][lane] = acc[0];
    sums[wave][1][lane] = acc[1];
  }
  __syncthreads();
  if (threadIdx.x < kTile && out0 + static_cast<int32_t>(threadIdx.x) < a.p.n_out) {
    float s[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < kProductWaves; ++k)
#pragma unroll
      for (int m = 0; m < 2; ++m) s[m] += sums[k][m][threadIdx.x];
    a.h[static_cast<int64_t>(pair) * a.inner + out0 + threadIdx.x] = activate(s[0], a.p.activation) * s[1] * c.weight;
  }
}

template <int BITS>
__global__ void __launch_bounds__(kProductThreads) hlwq_moe_few_down_kernel(const FewArgs a) {
  __shared__ __attribute__((aligned(16))) uint8_t book[Book<BITS>::kBytes];
  __shared__ __attribute__((aligned(16))) uint16_t act[kProductWaves][kChunk * kBlock];
  __shared__ float sums[kFewPairs][kTile];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r = lane & 15, h4 = lane >> 4;
  const int32_t out0 = blockIdx.x * kTile;
  const uint32_t copy = book_copy<BITS>(lane);
  fill_book<BITS>(book);
  __syncthreads();
  for (int32_t pair = wave; pair < a.p.pairs; pair += kProductWaves) {
    const int32_t expert = a.ids[pair];
    float acc = 0;
    if (expert >= 0 && expert < a.p.experts) {
      const int64_t at = (static_cast<int64_t>(expert) * a.p.rows + min(out0 + r, a.p.rows - 1)) * a.p.nb;
      const uint8_t* codes = a.p.packed + at * (16 * BITS) + 4 * BITS * h4;
      const uint16_t* norms = a.p.norms + at;
      const float* h = a.h + static_cast<int64_t>(pair) * a.inner;
      for (int32_t b0 = 0; b0 < a.p.nb; b0 += kChunk) {
        RowCodes<BITS> code[kChunk];
        float norm[kChunk], v[kChunk][2], scale[kChunk];
#pragma unroll
        for (int k = 0; k < kChunk; ++k) {
          const int32_t b = b0 + k, i = b * kBlock + 2 * lane;
          if (b >= a.p.nb) break;
          load_row(code[k], codes + b * (16 * BITS));
          norm[k] = f16_value(norms[b]);
          v[k][0] = i < a.inner ? h[i] : 0.0f;
          v[k][1] = i + 1 < a.inner ? h[i + 1] : 0.0f;
        }
#pragma unroll
        for (int k = 0; k < kChunk; ++k)
          if (b0 + k < a.p.nb) scale[k] = rotate_block(v[k], act[wave] + k * kBlock, lane);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int k = 0; k < kChunk; ++k)
          if (b0 + k < a.p.nb)
            acc = __builtin_fmaf(few_product<BITS>(code[k], book, copy, act[wave] + k * kBlock + 32 * h4), norm[k] * scale[k], acc);
        __builtin_amdgcn_wave_barrier();
      }
    }
    if (lane < kTile) sums[pair][lane] = acc;
  }
  __syncthreads();
  const int32_t t = threadIdx.x / kTile, row = threadIdx.x % kTile;
  if (t < a.tokens && out0 + row < a.hidden) {
    float s = 0;
    for (int32_t j = 0; j < a.p.top_k; ++j) s += sums[t * a.p.top_k + j][row];
    a.out[static_cast<int64_t>(t) * a.hidden + out0 + row] = static_cast<uint16_t>(pack_bf16x2(s, 0));
  }
}

// ---------------------------------------------------------------------------
// Between the two: a pair's inner activations rotated; after them: a token's
// pairs joined.
// ---------------------------------------------------------------------------

struct RotateArgs {
  const float* in;  // [pairs][n]
  const int32_t* ids;
  uint16_t* rotated;
  float* scale;
  int32_t n, experts;
};
__global__ void __launch_bounds__(kRotateThreads) hlwq_moe_rotate_kernel(const RotateArgs a) {
  const int32_t p = blockIdx.x;
  if (a.ids[p] < 0 || a.ids[p] >= a.experts) return;
  const float* row = a.in + static_cast<int64_t>(p) * a.n;
  const int64_t pitch = ceil_div(a.n, kBlock) * kBlock;
  rotate_row(
      [row, n = a.n](int32_t i) {
        const float next = row[min(i + 1, n - 1)];
        return f32x2{row[i], i + 1 < n ? next : 0.0f};
      },
      a.n, a.rotated + p * pitch, a.scale + p);
}

struct JoinArgs {
  const float* in;  // [pairs][n]
  const int32_t* ids;
  uint16_t* out;  // [tokens][n]
  int32_t n, experts, top_k;
};
__global__ void __launch_bounds__(256) hlwq_moe_join_kernel(const JoinArgs a) {
  const int32_t i = blockIdx.x * 256 + threadIdx.x;
  if (i >= a.n) return;
  const int64_t t = blockIdx.y;
  float s = 0;
  for (int32_t k = 0; k < a.top_k; ++k) {
    const int64_t p = t * a.top_k + k;
    if (a.ids[p] >= 0 && a.ids[p] < a.experts) s += a.in[p * a.n + i];
  }
  a.out[t * a.n + i] = static_cast<uint16_t>(pack_bf16x2(s, 0));
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------

struct Sizes {
  int64_t experts, hidden, inner, tokens, top_k;
  int64_t hidden_blocks, inner_blocks;
  int64_t pass;  // tokens to a pass
};

// *nothing: valid, with no work but the routing's.
int check_sizes(Sizes& s, bool* nothing) {
  if (s.experts < 0 || s.hidden < 0 || s.inner < 0 || s.tokens < 0 || s.top_k < 0) return HLWQ_ERR_SHAPE;
  if (s.experts > kMaxExperts || s.hidden > kMaxSize || s.inner > kMaxSize || s.top_k > kMaxTopK || s.tokens > kMaxTokens)
    return HLWQ_ERR_LIMIT;
  *nothing = s.tokens == 0 || s.hidden == 0;
  s.hidden_blocks = ceil_div(s.hidden, kBlock);
  s.inner_blocks = ceil_div(s.inner, kBlock);
  s.pass = std::min(s.tokens, kMaxPairs / std::max<int64_t>(s.top_k, 1));
  return HLWQ_OK;
}

// The workspace's parts, each a multiple of 16 bytes.
struct Parts {
  size_t logits, x, x_scale, h, h_rotated, h_scale, y, total;
};
Parts parts_of(const Sizes& s) {
  Parts p;
  size_t at = 0;
  const auto take = [&at](int64_t count, int64_t unit) {
    const size_t here = at;
    at += (static_cast<size_t>(count * unit) + 15) & ~size_t{15};
    return here;
  };
  const int64_t pairs = s.pass * s.top_k;
  p.logits = take(s.pass * s.experts, 8);
  p.x = take(s.pass * s.hidden_blocks * kBlock, 2);
  p.x_scale = take(s.pass, 4);
  p.h = take(pairs * s.inner, 4);
  p.h_rotated = take(pairs * s.inner_blocks * kBlock, 2);
  p.h_scale = take(pairs * s.inner_blocks, 4);
  p.y = take(pairs * s.hidden, 4);
  p.total = at;
  return p;
}

// Four waves to a row's blocks, or eight with two blocks each at a time.  Measured
// (5 bits, us, a kernel's time for gate and up, four waves and eight; x1: a pair or
// two to an expert, 16 tokens x 2 of 32 experts, 1024 values out from 20 blocks on):
//   2 blocks of a row, x1     5.6, 6.5      12, x1    23, 32
//   4, x1                     7.4, 10.7     16, x1    40, 53
//   6, x1                     8.6, 13.4     24, x1    33, 36
//   8, x1                    14.6, 19.4     40, x1    51, 46
// and the whole layer, all blocks with four or all with eight:
//   100 tokens x 4 of 8, 2048 x 512 (16 and 4 blocks)      73, 59
//   100 x 2 of 8, 4096 x 1408 (32 and 11)                 134, 118
//   33 x 1 of 2, 768 x 2048 (6 and 16)                     42, 34
//   1 x 2 of 8, 4096 x 14336 (32 and 112)                 132, 113
//   12 x 4 of 12, 640 x 1920 (5 and 15)                    31, 37
// Long rows are those of few large experts as a rule, to which many pairs come;
// where they are not, eight waves lose.  (Four with two blocks at a time and
// eight with three took as long or longer at every size.)
template <int BITS, bool GATED>
int launch_product(const ProductArgs& a, hipStream_t stream) {
  const auto go = [&](auto kernel, int groups) {
    const uint32_t wide = static_cast<uint32_t>(ceil_div(a.tiles, groups));
    return launch(kernel, dim3(wide, static_cast<uint32_t>(std::min(a.experts, a.pairs))), dim3(kProductThreads), stream, a);
  };
  if (a.nb <= 8) return go(hlwq_moe_product_kernel<BITS, 4, 1, GATED>, 2);
  return go(hlwq_moe_product_kernel<BITS, 8, 2, GATED>, 1);
}

// Whether the pairs are few enough for the two kernels that do the most by
// themselves, but read an expert's codes again for each pair, and whose second one
// gives a pair's row of inner values to a wave: up to 16 blocks of them, and one
// token's pairs, a wave each, or of little to read.  Measured (all kernels of a
// layer with 5 bits, us; tokens x experts of each, hidden x inner, blocks of codes
// read for all pairs; by these, by the kernels of many pairs):
//   1 x 8 of 256, 2048 x 512, 197 thousand     22.4, 28.0
//   8 x 4 of 256, 2048 x 128, 197 thousand     22.1, 30.0
//   32 x 1 of 128, 1024 x 256, 197 thousand    22.7, 23.2
//   1 x 8 of 128, 2816 x 704, 383 thousand     28.1, 34.4
//   2 x 8 of 256, 2048 x 512, 393 thousand     30.1, 32.8
//   8 x 4 of 64, 2048 x 256, 393 thousand      28.9, 32.8
//   1 x 2 of 8, 4096 x 2048, 393 thousand      35.1, 33.0
//   16 x 2 of 64, 1024 x 512, 393 thousand     37.3, 27.3
//   1 x 8 of 64, 4096 x 1024, 786 thousand     38.1, 45.1
//   1 x 4 of 16, 4096 x 2048, 786 thousand     44.0, 44.6
//   1 x 8 of 64, 4096 x 2048, 1.6 million      69.3, 70.4
//   1 x 8 of 256, 7168 x 2048, 2.8 million      102, 108
// more pairs or tokens, which may name the same experts:
//   2 x 10 of 512, 2048 x 512, 492 thousand    49.5, 44.2
//   3 x 8 of 256, 2048 x 512, 590 thousand     42.6, 39.3
//   2 x 8 of 128, 2816 x 704, 766 thousand     43.0, 41.6
//   1 x 16 of 256, 2048 x 1024, 786 thousand   53.5, 49.7
//   2 x 4 of 32, 4096 x 1408, 1.1 million      49.5, 53.9
//   2 x 4 of 8, 4096 x 2048, 1.6 million       64.1, 57.9
//   2 x 8 of 8, 4096 x 2048, 3.1 million        120, 71
//   2 x 8 of 256, 7168 x 2048, 5.5 million      186, 127
// more than 16 blocks of inner values:
//   1 x 2 of 8, 1024 x 4096, 197 thousand      40.7, 30.5
//   1 x 1 of 8, 4096 x 4096, 393 thousand      47.0, 36.6
//   1 x 2 of 8, 4096 x 8192, 1.6 million        108, 73
constexpr int64_t kFewCodes = 3 << 17, kFewInner = 16;  // blocks
bool few(const Sizes& s, int64_t tokens, int64_t pairs) {
  return pairs <= kFewPairs && s.hidden_blocks <= kFewBlocks && s.inner_blocks <= kFewInner &&
         ((tokens == 1 && pairs <= kProductWaves) || pairs * (2 * s.inner * s.hidden_blocks + s.hidden * s.inner_blocks) <= kFewCodes);
}
template <int BITS>
int launch_few(const FewArgs& up, const ProductArgs& down, hipStream_t stream) {
  const dim3 grid(static_cast<uint32_t>(ceil_div(up.inner, kTile)), static_cast<uint32_t>(up.p.pairs));
  const int st = up.p.experts <= 256 ? launch(hlwq_moe_few_up_kernel<BITS, 4>, grid, dim3(kProductThreads), stream, up)
                                     : launch(hlwq_moe_few_up_kernel<BITS, 16>, grid, dim3(kProductThreads), stream, up);
  if (st != HLWQ_OK) return st;
  FewArgs a = up;
  a.p = down;
  return launch(hlwq_moe_few_down_kernel<BITS>, dim3(static_cast<uint32_t>(ceil_div(up.hidden, kTile))), dim3(kProductThreads), stream, a);
}

// Whether the touched experts' sets of rows give the CUs work enough, the banks lie
// as the loads to LDS take them, and these do not go through the codes much more
// often than the product kernels, which take sixteen pairs of an expert at a time.
// Measured (as above; streamed, by the product kernels; sets of gate and up, if no
// expert is named twice):
//   4 tokens x 8 of 256, 2048 x 512, 128 sets     48.5, 47.3
//   8 x 8 of 64, 1024 x 256, 128                  34.9, 31.4
//   32 x 2 of 8, 4096 x 2048, 128                 80.4, 78.6
//   16 x 8 of 256, 2048 x 128, 128                51.8, 56.6
//   40 x 8 of 160, 512 x 128, 160                 35.5, 33.2
//   40 x 2 of 20, 2048 x 1024, 160                50.7, 55.4
//   24 x 8 of 256, 2048 x 128, 192                55.6, 71.7
//   64 x 8 of 256, 2048 x 512, 1024                141, 225
// Passes: a touched expert has pairs / touched pairs, more or less, so what is left
// over takes half a pass of its own; two thirds of the codes are gate and up.  A
// pass here is worth half of one of theirs.  Pairs of an expert, pairs of a pass
// over either bank, us as above:
//   512 x 4 of 16, 2048 x 2048: 128, 12 and 12     350, 575
//   200 x 4 of 32, 4096 x 1408: 25, 6 and 16       323, 378
//   256 x 8 of 64, 3584 x 512: 32, 6 and 16        261, 280
//   100 x 4 of 16, 1024 x 4096: 25, 16 and 6       142, 139
//   64 x 4 of 8, 2880 x 2880: 32, 8 and 8          173, 150
//   32 x 4 of 32, 5120 x 1000: 4, 4 and 16         140, 139
// and past it:
//   300 x 2 of 16, 4096 x 2048: 38, 6 and 12       332, 376
//   100 x 2 of 8, 4096 x 2560: 25, 6 and 9         186, 183
//   200 x 2 of 8, 4096 x 4096: 50, 6 and 6         477, 448
//   100 x 8 of 32, 5120 x 1000: 25, 4 and 16       365, 331; with 3 bits 257, 256
//   100 x 4 of 16, 6144 x 2560: 25, 4 and 9        572, 467
//   100 x 4 of 16, 1024 x 8192: 25, 16 and 3       297, 261
//   100 x 2 of 8, 8192 x 4096: 25, 3 and 6         752, 495
//   256 x 8 of 64, 7168 x 2048: 32, 3 and 12      3117, 1978
constexpr int64_t kStreamSets = 160;
bool streams(const hlwq_moe_banks& b, const Sizes& s, int64_t pairs) {
  const int64_t touched = std::min(s.experts, pairs);
  if (s.inner_blocks > kMaxInnerBlocks || s.hidden_blocks > kActBytes / 256 || touched * s.inner_blocks < kStreamSets ||
      misaligned(b.gate_up_packed, 16) || misaligned(b.down_packed, 16) || misaligned(b.gate_up_norms, 4) ||
      misaligned(b.down_norms, 4) || (s.hidden * s.inner_blocks) % 2 != 0)
    return false;
  const double each = static_cast<double>(pairs) / static_cast<double>(touched);
  const auto passes = [each](int32_t of) { return std::max(1.0, each / of + 0.5); };
  return 2 * passes(pass_pairs(s.hidden_blocks)) + passes(pass_pairs(s.inner_blocks)) < 2 * 3 * passes(kTile);
}
template <int BITS, bool GATED>
int launch_stream(ProductArgs a, hipStream_t stream) {
  a.tiles = static_cast<int32_t>(ceil_div(a.n_out, GATED ? kBlock : 2 * kBlock));
  return launch(hlwq_moe_stream_kernel<BITS, GATED>, dim3(kWorkgroups), dim3(kProductThreads), stream, a);
}

int run_moe(const hlwq_moe_banks* b, const void* x, int64_t x_stride, int64_t tokens, const void* router, bool route, int64_t top_k,
            int renormalize, int32_t* ids, float* weights, void* out, void* ws, size_t ws_bytes, hipStream_t stream) {
  if (!b) return HLWQ_ERR_NULL;
  if (b->bits != 5 && b->bits != 3) return HLWQ_ERR_BITS;
  if (b->activation != HLWQ_ACT_SILU && b->activation != HLWQ_ACT_GELU_TANH) return HLWQ_ERR_SHAPE;
  Sizes s{b->experts, b->hidden, b->inner, tokens, top_k, 0, 0, 0};
  bool nothing;
  int st = check_sizes(s, &nothing);
  if (st != HLWQ_OK) return st;
  if (x_stride < s.hidden || (route && top_k > s.experts)) return HLWQ_ERR_SHAPE;
  const int64_t block = 16 * b->bits;
  if (x_stride > kMaxSize || 2 * s.inner * s.hidden_blocks > 0x7fffffff / block || s.hidden * s.inner_blocks > 0x7fffffff / block)
    return HLWQ_ERR_LIMIT;
  const int64_t pairs = tokens * top_k;
  if (nothing) {
    if (!route || pairs == 0) return HLWQ_OK;
    if (!ids || !weights) return HLWQ_ERR_NULL;
    if (misaligned(ids, 4) || misaligned(weights, 4)) return HLWQ_ERR_ALIGN;
    Spans spans;
    add_span(spans, ids, pairs, 4, true);
    add_span(spans, weights, pairs, 4, true);
    if (check_disjoint(spans) != HLWQ_OK) return HLWQ_ERR_OVERLAP;
    const TopArgs a{nullptr, ids, weights, static_cast<int32_t>(tokens), static_cast<int32_t>(s.experts), static_cast<int32_t>(top_k),
                    renormalize != 0};
    return launch(hlwq_moe_even_kernel, dim3(static_cast<uint32_t>(ceil_div(pairs, kTopThreads))), dim3(kTopThreads), stream, a);
  }
  const int64_t up = s.experts * 2 * s.inner * s.hidden_blocks, down = s.experts * s.hidden * s.inner_blocks;
  const Parts parts = parts_of(s);
  if (!x || !out || !ws || (route && s.experts > 0 && !router) || (pairs > 0 && (!ids || !weights)) ||
      (up > 0 && (!b->gate_up_packed || !b->gate_up_norms)) || (down > 0 && (!b->down_packed || !b->down_norms)))
    return HLWQ_ERR_NULL;
  if (ws_bytes < parts.total) return HLWQ_ERR_SHAPE;
  if (misaligned(x, 2) || misaligned(out, 2) || misaligned(router, 2) || misaligned(ids, 4) || misaligned(weights, 4) ||
      misaligned(ws, 16) || misaligned(b->gate_up_packed, 4) || misaligned(b->down_packed, 4) ||
      misaligned(b->gate_up_norms, 2) || misaligned(b->down_norms, 2))
    return HLWQ_ERR_ALIGN;
  Spans spans;
  add_span(spans, x, (tokens - 1) * x_stride + s.hidden, 2, false);
  if (route) add_span(spans, router, s.experts * s.hidden, 2, false);
  add_span(spans, b->gate_up_packed, up, block, false);
  add_span(spans, b->gate_up_norms, up, 2, false);
  add_span(spans, b->down_packed, down, block, false);
  add_span(spans, b->down_norms, down, 2, false);
  add_span(spans, ids, pairs, 4, route);
  add_span(spans, weights, pairs, 4, route);
  add_span(spans, out, tokens * s.hidden, 2, true);
  add_span(spans, ws, static_cast<int64_t>(parts.total), 1, true);
  if (check_disjoint(spans) != HLWQ_OK) return HLWQ_ERR_OVERLAP;

  char* const at = static_cast<char*>(ws);
  const auto i32 = [](int64_t v) { return static_cast<int32_t>(v); };
  for (int64_t t0 = 0; t0 < tokens; t0 += s.pass) {
    const int64_t n = std::min(s.pass, tokens - t0), m = n * top_k;
    int32_t* const my_ids = ids ? ids + t0 * top_k : nullptr;
    float* const my_weights = weights ? weights + t0 * top_k : nullptr;
    uint16_t* const my_out = static_cast<uint16_t*>(out) + t0 * s.hidden;
    const bool empty = m == 0 || s.inner == 0 || s.experts == 0;
    PrepareArgs pa{};
    pa.x = static_cast<const uint16_t*>(x) + t0 * x_stride;
    pa.x_stride = x_stride;
    pa.router = static_cast<const uint16_t*>(router);
    pa.logits = reinterpret_cast<double*>(at + parts.logits);
    pa.rotated = reinterpret_cast<uint16_t*>(at + parts.x);
    pa.scale = reinterpret_cast<float*>(at + parts.x_scale);
    pa.tokens = i32(n);
    pa.hidden = i32(s.hidden);
    pa.experts = i32(s.experts);
    pa.expert_groups = i32(ceil_div(s.experts, router_tile(n).experts * kRouterWaves));
    const bool is_few = !empty && few(s, n, m);
    pa.rotating = empty || is_few ? 0 : i32(n);
    const int64_t preparing = pa.rotating + (route && m > 0 ? pa.expert_groups * ceil_div(n, router_tile(n).tokens) : 0);
    if (preparing > 0 &&
        (st = launch(hlwq_moe_prepare_kernel, dim3(static_cast<uint32_t>(preparing)), dim3(kRotateThreads), stream, pa)) != HLWQ_OK)
      return st;
    if (route && m > 0 && !is_few) {
      TopArgs ta{pa.logits, my_ids, my_weights, i32(n), i32(s.experts), i32(top_k), renormalize != 0};
      const dim3 grid(static_cast<uint32_t>(ceil_div(n, kTopThreads / 64)));
      st = s.experts <= 256 ? launch(hlwq_moe_top_kernel<4>, grid, dim3(kTopThreads), stream, ta)
                            : launch(hlwq_moe_top_kernel<16>, grid, dim3(kTopThreads), stream, ta);
      if (st != HLWQ_OK) return st;
    }
    if (!empty) {
      ProductArgs g{};
      g.packed = static_cast<const uint8_t*>(b->gate_up_packed);
      g.norms = static_cast<const uint16_t*>(b->gate_up_norms);
      g.act = pa.rotated;
      g.act_scale = pa.scale;
      g.ids = my_ids;
      g.weights = my_weights;
      g.out = reinterpret_cast<float*>(at + parts.h);
      g.rotated = reinterpret_cast<uint16_t*>(at + parts.h_rotated);
      g.rotated_scale = reinterpret_cast<float*>(at + parts.h_scale);
      g.pairs = i32(m);
      g.experts = i32(s.experts);
      g.top_k = i32(top_k);
      g.rows = i32(2 * s.inner);
      g.n_out = i32(s.inner);
      g.nb = i32(s.hidden_blocks);
      g.tiles = i32(ceil_div(s.inner, kTile));
      g.activation = b->activation;
      ProductArgs d = g;
      d.packed = static_cast<const uint8_t*>(b->down_packed);
      d.norms = static_cast<const uint16_t*>(b->down_norms);
      d.act = g.rotated;
      d.act_scale = g.rotated_scale;
      d.weights = nullptr;
      d.out = reinterpret_cast<float*>(at + parts.y);
      d.rows = d.n_out = i32(s.hidden);
      d.nb = i32(s.inner_blocks);
      d.tiles = i32(ceil_div(s.hidden, 2 * kTile));
      if (is_few) {
        const FewArgs f{g, pa.x, x_stride, route ? pa.logits : nullptr, my_ids, my_weights, g.out, my_out, i32(s.hidden), i32(s.inner),
                        renormalize != 0, i32(n)};
        if ((st = b->bits == 5 ? launch_few<5>(f, d, stream) : launch_few<3>(f, d, stream)) != HLWQ_OK) return st;
        continue;
      }
      const bool stream_banks = streams(*b, s, m);
      if (stream_banks)
        st = b->bits == 5 ? launch_stream<5, true>(g, stream) : launch_stream<3, true>(g, stream);
      else
        st = b->bits == 5 ? launch_product<5, true>(g, stream) : launch_product<3, true>(g, stream);
      if (st != HLWQ_OK) return st;
      const RotateArgs ra{g.out, my_ids, g.rotated, g.rotated_scale, i32(s.inner), i32(s.experts)};
      if (!stream_banks && (st = launch(hlwq_moe_rotate_kernel, dim3(static_cast<uint32_t>(m)), dim3(kRotateThreads), stream, ra)) != HLWQ_OK)
        return st;
      if (stream_banks)
        st = b->bits == 5 ? launch_stream<5, false>(d, stream) : launch_stream<3, false>(d, stream);
      else
        st = b->bits == 5 ? launch_product<5, false>(d, stream) : launch_product<3, false>(d, stream);
      if (st != HLWQ_OK) return st;
    }
    JoinArgs ja{reinterpret_cast<const float*>(at + parts.y), my_ids, my_out, i32(s.hidden), i32(s.experts), empty ? 0 : i32(top_k)};
    const dim3 grid(static_cast<uint32_t>(ceil_div(s.hidden, 256)), static_cast<uint32_t>(n));
    if ((st = launch(hlwq_moe_join_kernel, grid, dim3(256), stream, ja)) != HLWQ_OK) return st;
  }
  return HLWQ_OK;
}

}  // namespace
}  // namespace hlwq_kv

extern "C" {

int hlwq_moe_experts(const hlwq_moe_banks* banks, const void* x_bf16, int64_t x_stride, int64_t tokens, int64_t top_k,
                     const int32_t* experts, const float* weights, void* out_bf16, void* workspace,
                     size_t workspace_bytes, void* hip_stream) {
  return hlwq_kv::run_moe(banks, x_bf16, x_stride, tokens, nullptr, false, top_k, 0, const_cast<int32_t*>(experts),
                          const_cast<float*>(weights), out_bf16, workspace, workspace_bytes, static_cast<hipStream_t>(hip_stream));
}

int hlwq_moe_layer(const hlwq_moe_banks* banks, const void* x_bf16, int64_t x_stride, int64_t tokens,
                   const void* router_bf16, int64_t top_k, int renormalize, int32_t* experts, float* weights,
                   void* out_bf16, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return hlwq_kv::run_moe(banks, x_bf16, x_stride, tokens, router_bf16, true, top_k, renormalize, experts, weights, out_bf16,
                          workspace, workspace_bytes, static_cast<hipStream_t>(hip_stream));
}

size_t hlwq_moe_workspace(int64_t experts, int64_t hidden, int64_t inner, int64_t tokens, int64_t top_k) {
  hlwq_kv::Sizes s{experts, hidden, inner, tokens, top_k, 0, 0, 0};
  bool nothing;
  if (hlwq_kv::check_sizes(s, &nothing) != HLWQ_OK || nothing) return 0;
  return hlwq_kv::parts_of(s).total;
}

}  // extern "C"
