// attention_wide.h — attention of trees of some dozens of query rows over long
// caches: the split kernel's arithmetic with tiles of 64 rows.
//
// The split kernel unpacks every code once for sixteen rows, about 400 VALU
// instructions for 32 tokens, twice what their softmax takes; with 64 rows to a
// tile four waves share one unpacking.  A block is 64 tokens, 32 for each half of
// the eight waves; of a half's four waves two unpack K's operands (sixteen tokens
// each) and two V's (half the values each) into LDS as the lanes read them back,
// 16 bytes side by side, for the next block while this one is multiplied, and each
// takes sixteen of the rows.  The halves' sums are joined at the end.
//
// A block takes 256 KB of LDS reads and 64 KB of writes (2500 cycles at 128 bytes
// each) and about 300 VALU instructions and 32 products a wave (2400 and 1000
// cycles of a SIMD that holds two): what bounds it is LDS and VALU alike.  One
// request of 64 rows over 32767 tokens (3 bits, 24 query and 4 KV heads) takes 135
// us (on another card 144) with the rotation and the joining, tiles of sixteen rows
// 154 to 167; 24 ragged requests of up to 16384 tokens (2 bits) 177 and 226.  Of
// the 144 the unpacking is 51 (so much less without it), the products and the
// softmax 37; with a single block to a workgroup 40 are left: the launches, and the
// window's and the step's own tokens, which otherwise are done beside the pages.
#pragma once

#include "attention_split.h"
#include "staging.h"

#include <type_traits>

namespace hlwq_kv {

constexpr int kWideThreads = 512;
constexpr int kWideRows = 64;
constexpr int kWideBlock = 64;                     // tokens to a block
constexpr uint32_t kWideHalf = 32 << 10;           // of LDS: operands of 32 tokens, K's two sixteens, then V's
constexpr uint32_t kWideStage = 2 * kWideHalf;     // of a block
constexpr int kWideStats = 8 * 16 * 2;             // floats

// Beside a block's operands, for each half: K's norms (-1: the token is not there),
// V's over the power of two that no norm met so far exceeds (0), that exponent, and
// whether some token is not there.
struct WideSide {
  float k[32], v[32];
  int32_t exponent, missing, unused[2];
};

constexpr int kWideFloats = 8 * 16 * kSplitPitch + kWideStats;  // the sums' phase
constexpr uint32_t kWideBytes = 2 * kWideStage + 4 * sizeof(WideSide);
constexpr int kWideLds = kWideFloats * 4 > static_cast<int>(kWideBytes) ? kWideFloats : kWideBytes / 4;  // floats
static_assert(kWideLds * 4 >= Kin::bytes(kWideRows), "all phases fit");

// Query rows rotated once for all that read them: fp16 over a power of two that
// brings a row's largest value to [1, 2), as the products' operands, [row][x][lane
// group] 16 bytes; and the factors of their scores.
constexpr int kRotatedRow = 2 * kDim;  // bytes
template <int BITS>
__global__ void __launch_bounds__(256) hlwq_rotate_queries_kernel(const AttnArgs a) {
  __shared__ __attribute__((aligned(16))) uint16_t lds[4][kDim];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 4 + wave;
  const int32_t row = static_cast<int32_t>(at / a.q_heads), head = static_cast<int32_t>(at - static_cast<int64_t>(row) * a.q_heads);
  if (row >= min(a.rows, a.cu[a.requests])) return;
  const uint2 v = *reinterpret_cast<const uint2*>(a.q + row * a.q_stride + head * kDim + 4 * lane);
  float x[4] = {bf16_lo(v.x) * kQueryScale, bf16_hi(v.x) * kQueryScale, bf16_lo(v.y) * kQueryScale, bf16_hi(v.y) * kQueryScale};
  wave_fwht(x, lane);
  const float mx = wave_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
  const int ex = row_exponent(mx);
  const float f = __builtin_ldexpf(a.scale < 0 ? -1.0f : 1.0f, -ex);
  *reinterpret_cast<uint2*>(lds[wave] + 4 * lane) = uint2{pack_f16x2(x[0] * f, x[1] * f), pack_f16x2(x[2] * f, x[3] * f)};
  if (lane == 0) a.rotated_factor[at] = fmaxf(__builtin_ldexpf(a.factor, ex), __FLT_DENORM_MIN__);
  __builtin_amdgcn_wave_barrier();
  if (lane >= 32) return;
  const int op = lane >> 2, h4 = lane & 3;
  uint32_t d[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    d[k] = *reinterpret_cast<const uint32_t*>(lds[wave] + 64 * h4 + (BITS == 3 ? 32 * (op >> 2) + 8 * k + 2 * (op & 3) : 16 * (op >> 1) + 4 * k + 2 * (op & 1)));
  *reinterpret_cast<u32x4*>(a.rotated + at * (kRotatedRow / 2) + 8 * lane) =
      u32x4{__builtin_amdgcn_perm(d[1], d[0], 0x05040100u), __builtin_amdgcn_perm(d[3], d[2], 0x05040100u),
            __builtin_amdgcn_perm(d[1], d[0], 0x07060302u), __builtin_amdgcn_perm(d[3], d[2], 0x07060302u)};
}

// The two halves' sums of the tile's rows joined and given to write(row, sums of
// lane's four values, maximum, sum of weights).
template <class F>
__device__ __forceinline__ void join_halves(SplitRows& r, bool enc, int there, float* lds, int lane, int wave, F write) {
  const int c = lane & 15, h4 = lane >> 4;
  const float f = enc ? __builtin_ldexpf(1.0f / kTopWeight, r.exponent - 8) : 1.0f;  // H c n / 256
  float* stat = lds + 8 * 16 * kSplitPitch;
  const float l = group_sum(r.l);
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      f32x4 v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = r.o[4 * x + k][i] * f;
      *reinterpret_cast<f32x4*>(lds + (wave * 16 + c) * kSplitPitch + 16 * (4 * h4 + i) + 4 * x) = v;
    }
  if (h4 == 0) {
    stat[(wave * 16 + c) * 2] = r.m;
    stat[(wave * 16 + c) * 2 + 1] = l;
  }
  __syncthreads();
#pragma clang loop unroll(disable)
  for (int row = wave; row < min(there, kWideRows); row += 8) {
    float2 s[2];
#pragma unroll
    for (int w = 0; w < 2; ++w) s[w] = *reinterpret_cast<const float2*>(stat + (64 * w + row) * 2);
    const float m = fmaxf(s[0].x, s[1].x);
    float o[4] = {0, 0, 0, 0}, sum = 0;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const float g = fast_exp2(s[w].x - m);
      sum += s[w].y * g;
      const f32x4 v = *reinterpret_cast<const f32x4*>(lds + (64 * w + row) * kSplitPitch + 4 * lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += v[e] * g;
    }
    write(row, f32x4{o[0], o[1], o[2], o[3]}, m, sum);
  }
}

// What a wave loads of 32 tokens' codes: as Codes, of which it uses K's of one
// sixteen or V's.
template <int BITS>
__device__ __forceinline__ void load_part(Codes<BITS>& c, const AttnArgs& a, int part, int64_t vec_a, int64_t vec_b, int lane) {
  const int r = lane & 15, h4 = lane >> 4;
  if (part < 2) {
    const uint8_t* kp = a.k_packed + (part == 0 ? vec_a : vec_b) * (32 * BITS);
    if constexpr (BITS == 3) {
#pragma unroll
      for (int u = 0; u < 2; ++u) c.k[0][u] = *reinterpret_cast<const u32x3_4*>(kp + r * 96 + 24 * h4 + 12 * u);
    } else {
      c.k[0] = *reinterpret_cast<const u32x4*>(kp + r * 64 + 16 * h4);
    }
    return;
  }
#pragma unroll
  for (int sub = 0; sub < 2; ++sub) {
    const uint8_t* vp = a.v_packed + (sub == 0 ? vec_a : vec_b) * (32 * BITS);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (BITS == 3)
        c.v[4 * sub + i] = *reinterpret_cast<const u32x2_4*>(vp + (4 * h4 + i) * 96 + 12 * (r >> 1) + 4 * (r & 1));
      else
        c.v[4 * sub + i] = *reinterpret_cast<const uint32_t*>(vp + (4 * h4 + i) * 64 + 4 * r);
    }
  }
}

// Unpacked to LDS: operand x of K's sixteen `part`, or of V's half `part` - 2, a KB each.
// (The codes pass through empty assembly, so that no part of this is done ahead of
// the branches it stands in, for all parts, and kept in registers.)
__device__ __forceinline__ uint32_t held(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
}
__device__ __forceinline__ u32x2 held(u32x2 v) { return u32x2{held(v[0]), held(v[1])}; }
__device__ __forceinline__ u32x3 held(u32x3 v) { return u32x3{held(v[0]), held(v[1]), held(v[2])}; }
__device__ __forceinline__ u32x4 held(u32x4 v) { return u32x4{held(v[0]), held(v[1]), held(v[2]), held(v[3])}; }
template <int BITS>
__device__ __forceinline__ void unpack_part(Codes<BITS>& c, int part, uint8_t* to, int lane) {
  u32x4* at = reinterpret_cast<u32x4*>(to + part * 8192) + lane;
  if (part < 2) {
    if constexpr (BITS == 3) {
      c.k[0][0] = held(c.k[0][0]);
      c.k[0][1] = held(c.k[0][1]);
    } else {
      c.k[0] = held(c.k[0]);
    }
    u32x4 f[8];
    k_fragments<BITS>(c, 0, f);
#pragma unroll
    for (int x = 0; x < 8; ++x) at[64 * x] = f[x];
    return;
  }
  const bool odd = lane & 1;
  const auto half = [&](auto h) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c.v[i] = held(c.v[i]);
    uint32_t ca[8], cb[8];
    v_codes<BITS>(c, 0, h, odd, ca);
    v_codes<BITS>(c, 1, h, odd, cb);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const u32x2 p = look_up<BITS>(ca[x]), q = look_up<BITS>(cb[x]);
      at[64 * x] = u32x4{p[0], p[1], q[0], q[1]};
    }
  };
  if (part == 2)
    half(std::integral_constant<int, 0>{});
  else
    half(std::integral_constant<int, 1>{});
}

// The weights of 32 encoded tokens from their products with the query, as the
// operand of V's products: as in code_step, with the norms that lie in LDS.
__device__ __forceinline__ u32x4 wide_weights(SplitRows& r, f32x4 (&s)[2], float factor, const WideSide& side, int h4) {
  const int32_t exponent = __builtin_amdgcn_readfirstlane(side.exponent);
  if (exponent != r.exponent) {
    const float f = __builtin_ldexpf(1.0f, max(r.exponent - exponent, -126));
    r.exponent = exponent;
#pragma unroll
    for (int x = 0; x < 16; ++x) r.o[x] *= f;
  }
  f32x4 vn[2];
#pragma unroll
  for (int sub = 0; sub < 2; ++sub) {
    s[sub] *= *reinterpret_cast<const f32x4*>(side.k + 16 * sub + 4 * h4);
    vn[sub] = *reinterpret_cast<const f32x4*>(side.v + 16 * sub + 4 * h4);
  }
  if (__builtin_amdgcn_readfirstlane(side.missing)) {
    keep_branch();
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i >> 2][i & 3] = side.k[16 * (i >> 2) + 4 * h4 + (i & 3)] < 0 ? -HUGE_VALF : s[i >> 2][i & 3];
  }
  float t[8], p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = s[i >> 2][i & 3];
  weigh(r, t, factor, false, [](int) { return false; }, p);
  u32x4 pf;
#pragma unroll
  for (int i = 0; i < 4; ++i) pf[i] = pack_f16x2(p[2 * i] * vn[i >> 1][2 * (i & 1)], p[2 * i + 1] * vn[i >> 1][2 * (i & 1) + 1]);
  return pf;
}

// Pages [u0, u1) of a tile; their sums are over centroids.
template <int BITS, class F>
__device__ __forceinline__ void wide_pages(const AttnArgs& a, const Extent& e, int32_t b, int32_t head, int32_t r0, int32_t u0,
                                           int32_t u1, float* lds, int lane, int wave, F write) {
  const int c = lane & 15, h4 = lane >> 4, part = wave & 3, half = wave >> 2;
  const int32_t rows = e.n * a.group;
  const bool idle = r0 + 16 * part >= rows;
  // lane 2 i + s holds the page of sixteen s of the half's 32 tokens of block u0 +
  // i, for 32 blocks at a time and the next 32 ahead
  const auto pages = [&](int32_t u) {
    const int64_t t = static_cast<int64_t>(u + (lane >> 1)) * kWideBlock + 32 * half + 16 * (lane & 1);
    const int32_t id = t < e.paged ? a.table[static_cast<int64_t>(b) * a.width + (t >> a.page_shift)] : -1;
    return id < a.n_pages ? id : -1;
  };
  int32_t ids = pages(u0), ids_ahead = u0 + 32 < u1 ? pages(u0 + 32) : -1;
  // What the wave loads of a block: its part of the codes, and the norms that go
  // with it: K's of its sixteen (a lane each), or V's of all 32 (part 2).
  Codes<BITS> codes;
  uint16_t norm = 0;
  int there_a = 0, there_b = 0;
  const auto fetch = [&](int32_t u) {
    const int at = (u - u0) & 31;
    if (at == 0 && u > u0) {
      ids = ids_ahead;
      if (u + 32 < u1) ids_ahead = pages(u + 32);
    }
    const int32_t t = u * kWideBlock + 32 * half;  // at most 2^20 pages of 2^8 tokens
    const int32_t id_a = __builtin_amdgcn_readlane(ids, 2 * at), id_b = __builtin_amdgcn_readlane(ids, 2 * at + 1);
    there_a = id_a < 0 ? 0 : min(static_cast<int32_t>(e.paged) - t, 16);
    there_b = id_b < 0 ? 0 : min(static_cast<int32_t>(e.paged) - t - 16, 16);
    const auto vector_of = [&](int32_t id, int32_t t) {
      return ((static_cast<int64_t>(max(id, 0)) * a.kv_heads + head) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
    };
    const int64_t vec_a = vector_of(id_a, t), vec_b = vector_of(id_b, t + 16);
    load_part<BITS>(codes, a, part, vec_a, vec_b, lane);
    if (part < 2)
      norm = a.k_norms[(part ? vec_b : vec_a) + c];
    else if (part == 2)
      norm = a.v_norms[(lane & 16 ? vec_b : vec_a) + c];
  };
  int exponent = -64;  // of V's norms, in part 2's wave
  uint8_t* const stage = reinterpret_cast<uint8_t*>(lds) + half * kWideHalf;
  WideSide* const sides = reinterpret_cast<WideSide*>(reinterpret_cast<uint8_t*>(lds) + 2 * kWideStage) + half;  // two apart
  const auto unpack = [&](int buffer) {
    unpack_part<BITS>(codes, part, stage + buffer * kWideStage, lane);
    WideSide& side = sides[2 * buffer];
    const float n = f16_value(norm);
    if (part < 2) {
      const int mine = part ? there_b : there_a;
      if (lane < 16) side.k[16 * part + lane] = lane < mine ? n : -1.0f;
    } else if (part == 2) {
      // as in code_step: over a power of two that no norm met so far exceeds
      const bool in = c < (lane & 16 ? there_b : there_a);
      const float top = wave_max(in ? n : 0.0f);
      if (top > __builtin_ldexpf(1.0f, exponent)) exponent = __builtin_amdgcn_readfirstlane(__builtin_amdgcn_frexp_expf(top));
      if (lane < 32) side.v[lane] = in ? n * __builtin_ldexpf(kTopWeight, -exponent) : 0.0f;
      if (lane == 0) {
        side.exponent = exponent;
        side.missing = there_a < 16 || there_b < 16;
      }
    }
  };
  fetch(u0);
  u32x4 q[8];
  float factor;
  {
    const int32_t row = min(r0 + 16 * part + c, rows - 1), token = token_of(row, a.group);
    const int64_t at = (e.begin + static_cast<int64_t>(token)) * a.q_heads + head * a.group + (row - token * a.group);
    const u32x4* from = reinterpret_cast<const u32x4*>(a.rotated + at * (kRotatedRow / 2)) + h4;
#pragma unroll
    for (int x = 0; x < 8; ++x) q[x] = from[4 * x];
    factor = a.rotated_factor[at];
  }
  SplitRows r;
  clear(r);
  unpack(0);
  if (u0 + 1 < u1) fetch(u0 + 1);
  // Block u from LDS; u + 1 unpacked beside it, and then u + 2 on its way.  The
  // upper half's waves, on the same SIMDs as the lower's, multiply first.
#pragma clang loop unroll(disable)
  for (int32_t u = u0; u < u1; ++u) {
    wait_lds();
    barrier();
    const int buffer = (u - u0) & 1;
#pragma clang loop unroll(disable)
    for (int turn = 0; turn < 2; ++turn) {
      if ((half == 0) == (turn == 0)) {
        if (u + 1 < u1) unpack(buffer ^ 1);
        if (u + 2 < u1) fetch(u + 2);
        continue;
      }
      if (idle) continue;
      // its chain of products and softmax is the longer one (3 us of 144)
      __builtin_amdgcn_s_setprio(1);
      // kDeep operands on their way while one is multiplied
      constexpr int kDeep = 6;
      const u32x4* f = reinterpret_cast<const u32x4*>(stage + buffer * kWideStage) + lane;
      u32x4 g[kDeep];
      f32x4 s[2] = {};
#pragma unroll
      for (int x = 0; x < kDeep; ++x) g[x] = f[64 * x];
      __builtin_amdgcn_sched_group_barrier(0x100, kDeep, 0);
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        s[x >> 3] = mfma16<true>(g[x % kDeep], q[x & 7], s[x >> 3]);
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if (x + kDeep < 16) {
          g[x % kDeep] = f[64 * (x + kDeep)];
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
      }
      // V's first operands on their way during the softmax
#pragma unroll
      for (int x = 0; x < kDeep; ++x) g[x] = f[64 * (16 + x)];
      __builtin_amdgcn_sched_barrier(0);
      const u32x4 pf = wide_weights(r, s, factor, sides[2 * buffer], h4);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        r.o[x] = mfma16<true>(g[x % kDeep], pf, r.o[x]);
        __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
        if (x + kDeep < 16) {
          g[x % kDeep] = f[64 * (16 + x + kDeep)];
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        }
      }
      __builtin_amdgcn_s_setprio(0);
    }
  }
  join_halves(r, true, rows - r0, lds, lane, wave, write);
}

// The window's and the step's own tokens of a tile.
template <class F>
__device__ __forceinline__ void wide_tokens(const AttnArgs& a, const Extent& e, int32_t b, int32_t head, int32_t r0, float* lds,
                                            int lane, int wave, F write) {
  constexpr int M = kWideRows;
  const int c = lane & 15, h4 = lane >> 4, part = wave & 3, half = wave >> 2;
  const int32_t rows = e.n * a.group;
  const Tokens tokens(a, e, b, head);
  const int64_t last = tokens.near + token_of(min(r0 + M, rows) - 1, a.group);
  u32x4 q[8];
  const int32_t row = min(r0 + 16 * part + c, rows - 1), token = token_of(row, a.group);
  const int32_t q_head = head * a.group + (row - token * a.group);
  const uint16_t* p = a.q + (e.begin + static_cast<int64_t>(token)) * a.q_stride + q_head * kDim + 8 * h4;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    q[x] = *reinterpret_cast<const u32x4*>(p + 32 * x);
    if (a.scale < 0) q[x] ^= 0x80008000u;
  }
  SplitRows r;
  const Kin kin = find_kin<M, kWideThreads>(a, e, tokens.near, r0, rows, static_cast<int32_t>(last - tokens.near) + 1, lds, 16 * part + c);
  clear(r);
  if (r0 + 16 * part < rows)
    for (int64_t k0 = 32 * half; k0 <= last; k0 += 64) {
      const uint32_t seen = kin.word(k0);
      if (!__any(seen != 0)) continue;
      const bool masked = k0 + 31 >= tokens.near;
      token_step(r, q, a.factor, k0, last, [&](int64_t k) { return seen >> (k - k0) & 1; }, masked, masked, tokens, lane);
    }
  join_halves(r, false, rows - r0, lds, lane, wave, write);
}

template <int BITS>
__global__ void __launch_bounds__(kWideThreads) __attribute__((amdgpu_waves_per_eu(2, 2))) hlwq_wide_attention_kernel(const AttnArgs a) {
  constexpr int M = kWideRows;
  using Wide = SplitWork<M, kWideBlock>;
  __shared__ __attribute__((aligned(16))) float lds[kWideLds];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const auto tiles = [&](const Extent& e) { return Wide(a, e).tiles * a.kv_heads; };
  const auto cost = [&](const Extent& e) {
    const Wide w(a, e);
    return w.tiles * w.blocks * a.kv_heads;
  };
  const auto to_slot = [&](int32_t slot) {
    return [&a, slot, lane](int row, f32x4 o, float m, float l) {
      *reinterpret_cast<f32x4*>(partial_row<M>(a, slot, row) + 4 * lane) = o;
      if (lane == 0) *partial_stat<M>(a, slot, row) = float2{m, l};
    };
  };

  if (static_cast<int32_t>(blockIdx.x) >= a.workers) {
    // a tile's window and own tokens
    const int32_t x = blockIdx.x - a.workers;
    Finder<decltype(tiles), Nothing> finder(a, tiles, Nothing{});
    if (x >= finder.total) return;
    const Found f = finder.find(x);
    const Wide w(a, f.e);
    const int32_t head = quotient(f.rest, w.tiles), r0 = (f.rest - head * w.tiles) * M;
    const int32_t slot = tile_slot(a, x, 1);
    wide_tokens(a, w.e, f.b, head, r0, lds, lane, wave, [&](int row, f32x4 o, float m, float l) {
      if (w.blocks == 0)
        write_row(a, w.e.begin, head, r0 + row, o, l, lane);
      else
        to_slot(slot)(row, o, m, l);
    });
    return;
  }

  Finder<decltype(cost), decltype(tiles)> finder(a, cost, tiles);
  const Share share(finder.total, a.workers, 1);
  const int32_t worker = blockIdx.x;
  if (finder.total == 0 || worker >= share.workers) return;
  const Found first = finder.find(share.bound(worker));
  int32_t left = share.bound(worker + 1) - share.bound(worker), b = first.b, rest = first.rest, before = first.before;
#pragma clang loop unroll(disable)
  while (left > 0 && b < a.requests) {
    const Wide w(a, b == first.b ? first.e : extent_of(a, b));
    const int32_t tile = w.blocks ? quotient(rest, w.blocks) : 0;  // of all KV heads'
    if (w.blocks == 0 || tile >= w.tiles * a.kv_heads) {            // past the request's last
      before += w.tiles * a.kv_heads;
      rest = 0;
      ++b;
      continue;
    }
    const int32_t u0 = rest - tile * w.blocks, u1 = min(u0 + left, w.blocks);
    const int32_t head = quotient(tile, w.tiles);
    const int32_t slot = u0 == 0 && u1 == w.blocks ? tile_slot(a, before + tile, 0) : 2 * worker + (u0 > 0 ? 0 : 1);
    wide_pages<BITS>(a, w.e, b, head, (tile - head * w.tiles) * M, u0, u1, lds, lane, wave, to_slot(slot));
    __syncthreads();
    left -= u1 - u0;
    rest += u1 - u0;
  }
}

// Joins the rows of a tile, a wave each: the partial sums of its pages, rotated
// then, and of its other tokens.
constexpr int kWideJoinRows = 4;  // of a workgroup
__global__ void __launch_bounds__(64 * kWideJoinRows) hlwq_wide_join_kernel(const AttnArgs a) {
  constexpr int M = kWideRows;
  using Wide = SplitWork<M, kWideBlock>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const auto tiles = [&](const Extent& e) { return Wide(a, e).tiles * a.kv_heads; };
  const auto cost = [&](const Extent& e) {
    const Wide w(a, e);
    return w.tiles * w.blocks * a.kv_heads;
  };
  Finder<decltype(tiles), decltype(cost)> finder(a, tiles, cost);
  const int32_t x = blockIdx.x / (M / kWideJoinRows), row = blockIdx.x % (M / kWideJoinRows) * kWideJoinRows + wave;
  if (x >= finder.total) return;
  const Found f = finder.find(x);
  const Wide w(a, f.e);
  const int32_t head = quotient(f.rest, w.tiles), r0 = (f.rest - head * w.tiles) * M;
  if (w.blocks == 0 || r0 + row >= w.e.n * a.group) return;
  const Share share(Finder<decltype(cost), Nothing>(a, cost, Nothing{}).total, a.workers, 1);
  const int32_t x0 = f.before + f.rest * w.blocks;
  const int32_t w0 = share.worker_at(x0), w1 = share.worker_at(x0 + w.blocks - 1), parts = w1 - w0 + 1;
  const auto slot_of = [&](int32_t k) { return w0 == w1 ? tile_slot(a, x, 0) : 2 * (w0 + k) + (k == 0 ? 1 : 0); };
  const float2 other = *partial_stat<M>(a, tile_slot(a, x, 1), row);
  const f32x4 tokens = *reinterpret_cast<const f32x4*>(partial_row<M>(a, tile_slot(a, x, 1), row) + 4 * lane);
  float m = -FLT_MAX, l = 0;
  f32x4 o = {0, 0, 0, 0};
  for (int32_t k0 = 0; k0 < parts; k0 += 64) {
    float2 s{-FLT_MAX, 0};
    if (k0 + lane < parts) s = *partial_stat<M>(a, slot_of(k0 + lane), row);
    const float mn = fmaxf(m, wave_max(s.x)), old = fast_exp2(m - mn), g = fast_exp2(s.x - mn);
    m = mn;
    l = l * old + wave_sum(s.y * g);
    o *= old;
    const int count = min(parts - k0, 64);
    for (int i = 0; i < count; i += 4) {
      f32x4 v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = *reinterpret_cast<const f32x4*>(partial_row<M>(a, slot_of(k0 + min(i + j, count - 1)), row) + 4 * lane);
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (i + j < count) o += v[j] * __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), i + j));
    }
  }
  float y[4] = {o[0], o[1], o[2], o[3]};
  wave_fwht(y, lane);
  const float mn = fmaxf(m, other.x), g0 = fast_exp2(m - mn), g1 = fast_exp2(other.x - mn);
#pragma unroll
  for (int k = 0; k < 4; ++k) o[k] = y[k] * g0 + tokens[k] * g1;
  write_row(a, w.e.begin, head, r0 + row, o, l * g0 + other.y * g1, lane);
}

}  // namespace hlwq_kv
