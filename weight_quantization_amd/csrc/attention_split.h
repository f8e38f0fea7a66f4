// attention_split.h — attention of few query rows over long caches (single
// tokens, drafts), and the joining of partial sums.
//
// A decode step reads every code of the cache once for a handful of rows (the
// query heads of a group), so memory bounds it if the codes are turned into
// centroids quickly enough.  Nothing is staged: a wave takes 32 tokens, each
// lane loads the bytes that its matrix operand needs, 24 bytes (3 bits) of one
// key for K, six bytes of eight tokens for V, and unpacks them in registers.
//   - Codes are spread to one a byte across several vectors at once (the same
//     code of four groups, or of four tokens, in a register), so that one shift
//     and one mask extract four codes, and looked up with byte permutes: 57
//     instructions for 32 codes.
//   - The products sum over dimensions (K) and tokens (V) in any order, so the
//     operands take the order the bytes come in, and q is laid out to match.
//   - q is rotated once: q . H c = (H q) . c; the sum over tokens of p n c is
//     rotated once at the end.
// A workgroup is four waves with 32 tokens each to a block of 128; sums are
// joined over the waves in LDS, and over workgroups in the workspace.
#pragma once

#include "attention_common.h"

namespace hlwq_kv {

typedef uint32_t u32x2_4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32x3_4 __attribute__((ext_vector_type(3), aligned(4)));

constexpr int kSplitThreads = 256;
constexpr int kSplitBlock = 128;  // tokens to a block
constexpr int kSplitPitch = kDim + 4;  // floats to a row of sums in LDS: rows 4 banks apart
constexpr int kSplitLeast = 1;    // blocks that are worth a workgroup of their own

// Eight code registers, code i of four 3-byte groups each, from the groups'
// first, second and third bytes.
__device__ __forceinline__ void spread3(uint32_t a, uint32_t b, uint32_t c, uint32_t* out) {
  out[0] = a & 0x07070707u;
  out[1] = (a >> 3) & 0x07070707u;
  out[2] = ((a >> 6) & 0x03030303u) | ((b << 2) & 0x04040404u);
  out[3] = (b >> 1) & 0x07070707u;
  out[4] = (b >> 4) & 0x07070707u;
  out[5] = ((b >> 7) & 0x01010101u) | ((c << 1) & 0x06060606u);
  out[6] = (c >> 2) & 0x07070707u;
  out[7] = (c >> 5) & 0x07070707u;
}
__device__ __forceinline__ void spread2(uint32_t w, uint32_t* out) {
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = (w >> (2 * i)) & 0x03030303u;
}

// What a lane loads for 32 tokens (two sixteens, each within a page).
template <int BITS>
struct Codes;
template <>
struct Codes<3> {
  u32x3_4 k[2][2];  // key lane % 16 of each sixteen, bytes 24 (lane / 16) ..
  u32x2_4 v[8];     // tokens 4 (lane / 16) + i of each sixteen: the two words that hold bytes 6 (lane % 16) ..
  u32x2 kn[2], vn[2];  // norms of tokens 4 (lane / 16) ..
};
template <>
struct Codes<2> {
  u32x4 k[2];
  uint32_t v[8];
  u32x2 kn[2], vn[2];
};

template <int BITS>
__device__ __forceinline__ void load_codes(Codes<BITS>& c, const AttnArgs& a, int sub, int64_t vec, int lane) {
  const int r = lane & 15, h4 = lane >> 4;
  const uint8_t* kp = a.k_packed + vec * (32 * BITS);
  const uint8_t* vp = a.v_packed + vec * (32 * BITS);
  c.kn[sub] = *reinterpret_cast<const u32x2*>(a.k_norms + vec + 4 * h4);
  if constexpr (BITS == 3) {
#pragma unroll
    for (int u = 0; u < 2; ++u) c.k[sub][u] = *reinterpret_cast<const u32x3_4*>(kp + r * 96 + 24 * h4 + 12 * u);
  } else {
    c.k[sub] = *reinterpret_cast<const u32x4*>(kp + r * 64 + 16 * h4);
  }
  c.vn[sub] = *reinterpret_cast<const u32x2*>(a.v_norms + vec + 4 * h4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BITS == 3)
      c.v[4 * sub + i] = *reinterpret_cast<const u32x2_4*>(vp + (4 * h4 + i) * 96 + 12 * (r >> 1) + 4 * (r & 1));
    else
      c.v[4 * sub + i] = *reinterpret_cast<const uint32_t*>(vp + (4 * h4 + i) * 64 + 4 * r);
  }
}

// K fragments of one sixteen: eight products' operands.  Product x sums the
// lane group's dimensions dim_of(x, j), j = 0 .. 7.
template <int BITS>
__device__ __forceinline__ void k_fragments(const Codes<BITS>& c, int sub, u32x4 (&f)[8]) {
  if constexpr (BITS == 3) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const u32x3_4 w = c.k[sub][u];
      const uint32_t a = __builtin_amdgcn_perm(w[2], __builtin_amdgcn_perm(w[1], w[0], 0x00060300u), 0x05020100u);
      const uint32_t b = __builtin_amdgcn_perm(w[2], __builtin_amdgcn_perm(w[1], w[0], 0x00070401u), 0x06020100u);
      const uint32_t d = __builtin_amdgcn_perm(w[2], __builtin_amdgcn_perm(w[1], w[0], 0x00000502u), 0x07040100u);
      uint32_t code[8];
      spread3(a, b, d, code);
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const u32x2 lo = look_up<3>(code[2 * x]), hi = look_up<3>(code[2 * x + 1]);
        f[4 * u + x] = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t code[4];
      spread2(c.k[sub][u], code);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const u32x2 lo = look_up<2>(code[2 * x]), hi = look_up<2>(code[2 * x + 1]);
        f[2 * u + x] = u32x4{lo[0], lo[1], hi[0], hi[1]};
      }
    }
  }
}
// The even one of the two dimensions, relative to the lane group's 64, that
// slots j and j + 4 of product x stand for (j < 4; slot j + 4 is the odd one).
template <int BITS>
__device__ __forceinline__ constexpr int dim_of(int x, int j) {
  return BITS == 3 ? 32 * (x >> 2) + 8 * j + 2 * (x & 3) : 16 * (x >> 1) + 4 * j + 2 * (x & 1);
}

// Codes of dimensions 16 (lane % 16) + 8 half + 0 .. 7 of the sixteen's four
// tokens, one register a dimension.
template <int BITS>
__device__ __forceinline__ void v_codes(const Codes<BITS>& c, int sub, int half, bool odd, uint32_t (&code)[8]) {
  if constexpr (BITS == 3) {
    const uint32_t near = odd ? 0x07030602u : 0x05010400u, far = odd ? 0x05010400u : 0x07030602u;
    uint32_t p[2][2];  // byte pairs (0, 1), (2, 3) or (4, 5) of tokens (0, 1) and (2, 3)
    uint32_t by[3];
    const auto pair = [&](int which, uint32_t (&q)[2]) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const u32x2_4 x = c.v[4 * sub + 2 * t], y = c.v[4 * sub + 2 * t + 1];
        if (which == 0) q[t] = __builtin_amdgcn_perm(y[0], x[0], near);
        if (which == 1) q[t] = __builtin_amdgcn_perm(odd ? y[1] : y[0], odd ? x[1] : x[0], far);
        if (which == 2) q[t] = __builtin_amdgcn_perm(y[1], x[1], near);
      }
    };
    if (half == 0) {
      pair(0, p[0]);
      pair(1, p[1]);
      by[0] = __builtin_amdgcn_perm(p[0][1], p[0][0], 0x05040100u);
      by[1] = __builtin_amdgcn_perm(p[0][1], p[0][0], 0x07060302u);
      by[2] = __builtin_amdgcn_perm(p[1][1], p[1][0], 0x05040100u);
    } else {
      pair(1, p[0]);
      pair(2, p[1]);
      by[0] = __builtin_amdgcn_perm(p[0][1], p[0][0], 0x07060302u);
      by[1] = __builtin_amdgcn_perm(p[1][1], p[1][0], 0x05040100u);
      by[2] = __builtin_amdgcn_perm(p[1][1], p[1][0], 0x07060302u);
    }
    spread3(by[0], by[1], by[2], code);
  } else {
    const uint32_t sel = half ? 0x07030602u : 0x05010400u;
    const uint32_t p = __builtin_amdgcn_perm(c.v[4 * sub + 1], c.v[4 * sub], sel);
    const uint32_t q = __builtin_amdgcn_perm(c.v[4 * sub + 3], c.v[4 * sub + 2], sel);
    spread2(__builtin_amdgcn_perm(q, p, 0x05040100u), code);
    spread2(__builtin_amdgcn_perm(q, p, 0x07060302u), code + 4);
  }
}

template <bool ENC>
__device__ __forceinline__ f32x4 mfma16(u32x4 a, u32x4 b, f32x4 c) {
  if constexpr (ENC)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Largest value over the four lane groups.
__device__ __forceinline__ float group_max(float v) {
  v = fmaxf(v, lane_xor(v, 16));
  return fmaxf(v, half_swap(v));
}
__device__ __forceinline__ float group_sum(float v) {
  v += lane_xor(v, 16);
  return v + half_swap(v);
}

// One wave's sums over its tokens: o[n][s][i] is value 16 (4 (lane / 16) + i) +
// s of row 16 n + lane % 16.
template <int NR>
struct SplitRows {
  f32x4 o[NR][16];
  float m[NR], l[NR];
  int exponent;  // of the pages' values: sums are over p n 2^-exponent
};

template <int NR>
__device__ __forceinline__ void clear(SplitRows<NR>& r) {
#pragma unroll
  for (int n = 0; n < NR; ++n) {
#pragma unroll
    for (int s = 0; s < 16; ++s) r.o[n][s] = f32x4{0, 0, 0, 0};
    r.m[n] = -FLT_MAX;
    r.l[n] = 0;
  }
  r.exponent = -64;
}

// Softmax weights of eight scores a lane and row set, s[..] times factor[n];
// gone[i]: the token is not seen by the row.
template <int NR, class G>
__device__ __forceinline__ void weigh(SplitRows<NR>& r, int n, float (&s)[8], float factor, bool masked, G gone, float (&p)[8]) {
  if (masked) {
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = gone(i) ? -FLT_MAX : s[i];
  }
  float mx = s[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
  mx = group_max(mx) * factor;
  if (__any(mx - r.m[n] > kLazy)) {
    const float mn = fmaxf(r.m[n], mx);
    const float f = fast_exp2(r.m[n] - mn);
    r.m[n] = mn;
    r.l[n] *= f;
#pragma unroll
    for (int x = 0; x < 16; ++x) r.o[n][x] *= f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = fast_exp2(__builtin_fmaf(s[i], factor, -r.m[n]));
    if (masked) p[i] = gone(i) ? 0.0f : p[i];
    r.l[n] += p[i];
  }
}

// 32 encoded tokens; there: how many of each sixteen exist.
template <int BITS, int NR>
__device__ __forceinline__ void code_step(SplitRows<NR>& r, const u32x4 (&q)[NR][8], const float (&factor)[NR],
                                          const Codes<BITS>& c, int there_a, int there_b, int lane) {
  const int h4 = lane >> 4;
  const bool odd = lane & 1, masked = there_a < 16 || there_b < 16;
  f32x4 s[NR][2];
#pragma unroll
  for (int sub = 0; sub < 2; ++sub) {
    u32x4 f[8];
    k_fragments<BITS>(c, sub, f);
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      s[n][sub] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < 8; ++x) s[n][sub] = mfma16<true>(f[x], q[n][x], s[n][sub]);
    }
  }
  float kn[8], vn[8];
  const auto gone = [&](int i) { return 4 * h4 + (i & 3) >= (i < 4 ? there_a : there_b); };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t kw = c.kn[i >> 2][(i >> 1) & 1], vw = c.vn[i >> 2][(i >> 1) & 1];
    kn[i] = f16_value(static_cast<uint16_t>(i & 1 ? kw >> 16 : kw));
    vn[i] = f16_value(static_cast<uint16_t>(i & 1 ? vw >> 16 : vw));
    if (masked && gone(i)) vn[i] = 0;
  }
  // The weights p n are products' operands in fp16, so n is taken over a power
  // of two that no norm met so far exceeds: p n 2^-exponent is at most 2^kLazy,
  // and a weight is rounded to a subnormal only where it is below 2^-14 of
  // that.
  float top = vn[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) top = fmaxf(top, vn[i]);
  if (__any(top > __builtin_ldexpf(1.0f, r.exponent))) {
    top = group_max(top);
    int e = __builtin_amdgcn_frexp_expf(top);
    e = __builtin_amdgcn_readfirstlane(e);
    const float f = __builtin_ldexpf(1.0f, max(r.exponent - e, -126));
    r.exponent = e;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int x = 0; x < 16; ++x) r.o[n][x] *= f;
  }
  const float over = __builtin_ldexpf(1.0f, -r.exponent);
  u32x4 pf[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    float t[8], p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = s[n][i >> 2][i & 3] * kn[i];
    weigh<NR>(r, n, t, factor[n], masked, gone, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) pf[n][i] = pack_f16x2(p[2 * i] * (vn[2 * i] * over), p[2 * i + 1] * (vn[2 * i + 1] * over));
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t ca[8], cb[8];
    v_codes<BITS>(c, 0, half, odd, ca);
    v_codes<BITS>(c, 1, half, odd, cb);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const u32x2 a = look_up<BITS>(ca[x]), b = look_up<BITS>(cb[x]);
      const u32x4 f{a[0], a[1], b[0], b[1]};
#pragma unroll
      for (int n = 0; n < NR; ++n) r.o[n][8 * half + x] = mfma16<true>(f, pf[n], r.o[n][8 * half + x]);
    }
  }
}

// 32 bf16 tokens from k0 on; row(side, k): token k's vector; lim[n]: last
// token that the lane's row of set n sees; last: the last one there is.
template <int NR, class F>
__device__ __forceinline__ void token_step(SplitRows<NR>& r, const u32x4 (&q)[NR][8], float factor, int64_t k0, int64_t last,
                                           const int64_t (&lim)[NR], bool masked, F row, int lane) {
  const int c = lane & 15, h4 = lane >> 4;
  f32x4 s[NR][2];
#pragma unroll
  for (int sub = 0; sub < 2; ++sub) {
    const uint16_t* p = row(0, min(k0 + 16 * sub + c, last)) + 8 * h4;
    u32x4 f[8];
#pragma unroll
    for (int x = 0; x < 8; ++x) f[x] = *reinterpret_cast<const u32x4*>(p + 32 * x);
#pragma unroll
    for (int n = 0; n < NR; ++n) {
      s[n][sub] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int x = 0; x < 8; ++x) s[n][sub] = mfma16<false>(f[x], q[n][x], s[n][sub]);
    }
  }
  const auto token = [&](int i) { return k0 + 16 * (i >> 2) + 4 * h4 + (i & 3); };
  u32x4 pf[NR];
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    float t[8], p[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) t[i] = s[n][i >> 2][i & 3];
    weigh<NR>(r, n, t, factor, masked, [&](int i) { return token(i) > lim[n]; }, p);
#pragma unroll
    for (int i = 0; i < 4; ++i) pf[n][i] = pack_bf16x2(p[2 * i], p[2 * i + 1]);
  }
  uint32_t left = 0;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    u32x4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = *reinterpret_cast<const u32x4*>(row(1, min(token(i), last)) + 16 * c + 8 * half);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const uint32_t sel = x & 1 ? 0x07060302u : 0x05040100u;
      u32x4 f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = __builtin_amdgcn_perm(v[2 * i + 1][x >> 1], v[2 * i][x >> 1], sel);
        // as in key_step: 0 times what a row does not see must stay 0
        if (masked) f[i] = finite_pair(f[i], left);
      }
#pragma unroll
      for (int n = 0; n < NR; ++n) r.o[n][8 * half + x] = mfma16<false>(f, pf[n], r.o[n][8 * half + x]);
    }
  }
  if (__any(left != 0)) {
    for (int k = 0; k < 32 && k0 + k <= last; ++k) {
      const uint16_t* p = row(1, k0 + k) + 64 * h4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float v = bf16_lo(p[16 * i + x]);
#pragma unroll
          for (int n = 0; n < NR; ++n) r.o[n][x][i] += k0 + k <= lim[n] && !__builtin_isfinite(v) ? v : 0.0f;
        }
    }
  }
}

// Rows of a segment joined over the waves: wave w owns rows 4 w .. 4 w + 3 of
// each set, four values to a lane.
template <int NR>
struct Joined {
  float o[NR][4][4], m[NR][4], l[NR][4];
};
constexpr int kSplitStats = 4 * 16 * 2;  // floats

// Adds the waves' sums to the joined ones, rotated if they are over centroids.
template <int NR>
__device__ __forceinline__ void join(Joined<NR>& j, SplitRows<NR>& r, bool enc, float* lds, int lane, int wave) {
  const int c = lane & 15, h4 = lane >> 4;
  const float f = enc ? __builtin_ldexpf(1.0f, r.exponent - 8) : 1.0f;  // H c n / 256
  float* stat = lds + 4 * 16 * kSplitPitch;
#pragma unroll
  for (int n = 0; n < NR; ++n) {
    const float l = group_sum(r.l[n]);
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        f32x4 v;
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = r.o[n][4 * x + k][i] * f;
        *reinterpret_cast<f32x4*>(lds + (wave * 16 + c) * kSplitPitch + 16 * (4 * h4 + i) + 4 * x) = v;
      }
    if (h4 == 0) {
      stat[(wave * 16 + c) * 2] = r.m[n];
      stat[(wave * 16 + c) * 2 + 1] = l;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int row = 4 * wave + k;
      float m = j.m[n][k];
#pragma unroll
      for (int w = 0; w < 4; ++w) m = fmaxf(m, stat[(w * 16 + row) * 2]);
      const float old = fast_exp2(j.m[n][k] - m);
      float o[4] = {0, 0, 0, 0}, sum = 0;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float g = fast_exp2(stat[(w * 16 + row) * 2] - m);
        sum += stat[(w * 16 + row) * 2 + 1] * g;
        const f32x4 v = *reinterpret_cast<const f32x4*>(lds + (w * 16 + row) * kSplitPitch + 4 * lane);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] += v[e] * g;
      }
      if (enc) wave_fwht(o, lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) j.o[n][k][e] = j.o[n][k][e] * old + o[e];
      j.l[n][k] = j.l[n][k] * old + sum;
      j.m[n][k] = m;
    }
  }
}

template <int BITS, int NR>
__global__ void __launch_bounds__(kSplitThreads) __attribute__((amdgpu_waves_per_eu(NR == 1 ? 2 : 1, NR == 1 ? 2 : 1)))
hlwq_split_attention_kernel(const AttnArgs a) {
  constexpr int M = 16 * NR;
  constexpr int kQPitch = kDim + 8;  // fp16 to a row of rotated q in LDS
  __shared__ __attribute__((aligned(16))) float lds[4 * 16 * kSplitPitch + kSplitStats];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h4 = lane >> 4;
  const auto cost = [&](int32_t b) {
    const Work<M, kSplitBlock> w(a, b);
    return w.head_cost() * a.kv_heads;
  };
  const int64_t total = sum_over(a.requests, cost);
  const Share share(total, a.workers, kSplitLeast);
  const int64_t worker = blockIdx.x;
  if (total == 0 || worker >= share.workers) return;
  const Found first = find(a.requests, share.bound(worker), cost, [](int32_t) { return int64_t{0}; });

  for_segments<M, kSplitBlock>(a, share, first, worker, [&](const Work<M, kSplitBlock>& w, const Segment& g) {
    const Extent& e = w.e;
    const int32_t r0 = static_cast<int32_t>(g.tile * M), rows = w.rows(a);
    const int64_t blocks = w.blocks(a, g.tile);
    const int64_t u0 = w.block_at(g.from, blocks, g.cost), u1 = w.block_at(g.to, blocks, g.cost);
    const int64_t near = e.held - e.enc;  // tokens in the window
    Joined<NR> all;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        all.m[n][k] = -FLT_MAX;
        all.l[n][k] = 0;
#pragma unroll
        for (int x = 0; x < 4; ++x) all.o[n][k][x] = 0;
      }
    // token (of the step) and q vector of a row of the tile
    const auto q_row = [&](int32_t row, int32_t& token) {
      token = token_of(row, a.group);
      return a.q + (e.begin + static_cast<int64_t>(token)) * a.q_stride + (g.head * a.group + (row - token * a.group)) * kDim;
    };

    if (u0 < w.page_blocks && u0 < u1) {
      const int64_t end = min(u1, w.page_blocks);
      // Pages: lane 2 i + s holds that of sixteen s of the wave's 32 tokens of
      // block u0 + i, for 32 blocks at a time and the next 32 ahead.
      const auto pages = [&](int64_t u) {
        const int64_t t = (u + (lane >> 1)) * kSplitBlock + 32 * wave + 16 * (lane & 1);
        const int32_t id = t < e.paged ? a.table[static_cast<int64_t>(g.b) * a.width + (t >> a.page_shift)] : -1;
        return id < a.n_pages ? id : -1;
      };
      int32_t ids = pages(u0), ids_ahead = u0 + 32 < end ? pages(u0 + 32) : -1;
      const auto fetch = [&](int64_t u, Codes<BITS>& to, int (&there)[2]) {
        const int at = static_cast<int>(u - u0) & 31;
        if (at == 0 && u > u0) {
          ids = ids_ahead;
          if (u + 32 < end) ids_ahead = pages(u + 32);
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int64_t t = u * kSplitBlock + 32 * wave + 16 * s;
          const int32_t id = __builtin_amdgcn_readlane(ids, 2 * at + s);
          there[s] = id < 0 ? 0 : static_cast<int>(min(e.paged - t, int64_t{16}));
          const int64_t vec = ((static_cast<int64_t>(max(id, 0)) * a.kv_heads + g.head) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
          load_codes<BITS>(to, a, s, vec, lane);
        }
      };
      Codes<BITS> cur, next;
      int there[2], there_next[2] = {0, 0};
      fetch(u0, cur, there);

      // q rotated, each row over a power of two that brings its largest value
      // to [1, 2), as fp16
      uint16_t* ql = reinterpret_cast<uint16_t*>(lds);
      float* qf = lds + M * kQPitch / 2;
      for (int row = wave; row < M; row += 4) {
        float x[4] = {0, 0, 0, 0};
        if (r0 + row < rows) {
          int32_t token;
          const uint2 v = *reinterpret_cast<const uint2*>(q_row(r0 + row, token) + 4 * lane);
          x[0] = bf16_lo(v.x);
          x[1] = bf16_hi(v.x);
          x[2] = bf16_lo(v.y);
          x[3] = bf16_hi(v.y);
        }
        wave_fwht(x, lane);
        float mx = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) mx = fmaxf(mx, lane_xor(mx, d));
        const int ex = mx > 0 ? __builtin_amdgcn_frexp_expf(mx) - 1 : 0;
        const float f = __builtin_ldexpf(a.scale < 0 ? -1.0f : 1.0f, -ex);
        *reinterpret_cast<uint2*>(ql + row * kQPitch + 4 * lane) = uint2{pack_f16x2(x[0] * f, x[1] * f), pack_f16x2(x[2] * f, x[3] * f)};
        if (lane == 0) qf[row] = __builtin_ldexpf(fabsf(a.scale) * kLog2e, ex - 8);
      }
      __syncthreads();
      u32x4 q[NR][8];
      float factor[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        factor[n] = qf[16 * n + c];
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          uint32_t d[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            d[k] = *reinterpret_cast<const uint32_t*>(ql + (16 * n + c) * kQPitch + 64 * h4 + dim_of<BITS>(x, k));
          q[n][x] = u32x4{__builtin_amdgcn_perm(d[1], d[0], 0x05040100u), __builtin_amdgcn_perm(d[3], d[2], 0x05040100u),
                          __builtin_amdgcn_perm(d[1], d[0], 0x07060302u), __builtin_amdgcn_perm(d[3], d[2], 0x07060302u)};
        }
      }
      SplitRows<NR> r;
      clear(r);
      for (int64_t u = u0; u < end; ++u) {
        if (u + 1 < end) fetch(u + 1, next, there_next);
        if (there[0] + there[1] > 0) code_step<BITS, NR>(r, q, factor, cur, there[0], there[1], lane);
        cur = next;
        there[0] = there_next[0];
        there[1] = there_next[1];
      }
      join<NR>(all, r, true, lds, lane, wave);
      __syncthreads();
    }

    if (u1 > w.page_blocks) {
      const int64_t from = max(u0, w.page_blocks) - w.page_blocks, to = u1 - w.page_blocks;
      const int32_t first_token = w.first_token(a, g.tile);
      const int64_t last = near + w.last_token(a, g.tile);
      u32x4 q[NR][8];
      int64_t lim[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        int32_t token;
        const uint16_t* p = q_row(min(r0 + 16 * n + c, rows - 1), token) + 8 * h4;
        lim[n] = near + token;
#pragma unroll
        for (int x = 0; x < 8; ++x) {
          q[n][x] = *reinterpret_cast<const u32x4*>(p + 32 * x);
          if (a.scale < 0) q[n][x] ^= 0x80008000u;
        }
      }
      const int64_t ring0 = a.ring > 0 ? e.enc % a.ring : 0;
      const auto row = [&](int side, int64_t k) {
        if (k < near) {
          int64_t slot = ring0 + k;
          if (slot >= a.ring) slot -= a.ring;
          return (side ? a.v_window : a.k_window) + ((static_cast<int64_t>(g.b) * a.kv_heads + g.head) * a.ring + slot) * kDim;
        }
        return (side ? a.v_new : a.k_new) + (e.begin + (k - near)) * (side ? a.v_stride : a.k_stride) + g.head * kDim;
      };
      SplitRows<NR> r;
      clear(r);
      for (int64_t u = from; u < to; ++u) {
        const int64_t k0 = u * kSplitBlock + 32 * wave;
        if (k0 <= last) token_step<NR>(r, q, fabsf(a.scale) * kLog2e, k0, last, lim, k0 + 31 > near + first_token, row, lane);
      }
      join<NR>(all, r, false, lds, lane, wave);
      __syncthreads();
    }

    const bool whole = g.from == 0 && g.to == g.cost;
    const int slot = g.from > 0 ? 0 : 1;
#pragma unroll
    for (int n = 0; n < NR; ++n)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int row = 16 * n + 4 * wave + k;
        if (r0 + row >= rows) continue;
        if (whole) {
          const float inv = 1.0f / all.l[n][k];
          const int32_t token = token_of(r0 + row, a.group);
          const int64_t at = (e.begin + static_cast<int64_t>(token)) * a.q_heads + g.head * a.group + (r0 + row - token * a.group);
          *reinterpret_cast<uint2*>(a.out + at * kDim + 4 * lane) =
              uint2{pack_bf16x2(all.o[n][k][0] * inv, all.o[n][k][1] * inv), pack_bf16x2(all.o[n][k][2] * inv, all.o[n][k][3] * inv)};
        } else {
          *reinterpret_cast<f32x4*>(partial_row<M>(a, worker, slot, row) + 4 * lane) =
              f32x4{all.o[n][k][0], all.o[n][k][1], all.o[n][k][2], all.o[n][k][3]};
          if (lane == 0) *partial_stat<M>(a, worker, slot, row) = float2{all.m[n][k], all.l[n][k]};
        }
      }
  });
}

// ---------------------------------------------------------------------------
// Tiles that several workgroups shared.  Where tiles are narrow and many
// workgroups share one (few rows over a long cache), a workgroup joins one row
// and each wave every fourth partial sum; where they are wide (WAVE_ROWS > 0)
// a wave joins that many rows by itself.
// ---------------------------------------------------------------------------

template <int M, int KT, int LEAST, int WAVE_ROWS>
__global__ void __launch_bounds__(kSplitThreads) hlwq_join_attention_kernel(const AttnArgs a) {
  constexpr int kRows = WAVE_ROWS ? 4 * WAVE_ROWS : 1;  // of a workgroup
  __shared__ __attribute__((aligned(16))) float lds[4 * (kDim + 4)];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const auto cost = [&](int32_t b) {
    const Work<M, KT> w(a, b);
    return w.head_cost() * a.kv_heads;
  };
  const auto tiles = [&](int32_t b) {
    const Work<M, KT> w(a, b);
    return w.tiles * a.kv_heads;
  };
  const int64_t total = sum_over(a.requests, cost);
  if (total == 0) return;
  const Found f = find(a.requests, blockIdx.x / (M / kRows), tiles, cost);
  if (f.b < 0) return;
  const Work<M, KT> w(a, f.b);
  const int32_t head = static_cast<int32_t>(quotient(f.rest, w.tiles));
  const int64_t tile = f.rest - head * w.tiles;
  const int32_t row0 = (blockIdx.x % (M / kRows)) * kRows, r0 = static_cast<int32_t>(tile * M), rows = w.rows(a);
  if (r0 + row0 >= rows) return;
  const int64_t x0 = f.also + head * w.head_cost() + w.cost_before(tile), x1 = x0 + w.cost(tile);
  const Share share(total, a.workers, LEAST);
  const int64_t w0 = share.worker_at(x0), w1 = share.worker_at(x1 - 1);
  if (w0 == w1) return;  // one workgroup did it all

  const auto write = [&](int32_t at_row, f32x4 o, float l) {
    const float inv = 1.0f / l;
    const int32_t token = token_of(at_row, a.group);
    const int64_t at = (w.e.begin + static_cast<int64_t>(token)) * a.q_heads + head * a.group + (at_row - token * a.group);
    *reinterpret_cast<uint2*>(a.out + at * kDim + 4 * lane) = uint2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
  };
  const auto add = [&](int64_t k, int row, f32x4& o, float& m, float& l) {
    const int slot = k == w0 ? 1 : 0;
    const float2 s = *partial_stat<M>(a, k, slot, row);
    const f32x4 v = *reinterpret_cast<const f32x4*>(partial_row<M>(a, k, slot, row) + 4 * lane);
    const float mn = fmaxf(m, s.x);
    const float f0 = fast_exp2(m - mn), f1 = fast_exp2(s.x - mn);
    m = mn;
    l = l * f0 + s.y * f1;
    o = o * f0 + v * f1;
  };
  if constexpr (WAVE_ROWS > 0) {
    float m[WAVE_ROWS], l[WAVE_ROWS];
    f32x4 o[WAVE_ROWS];
#pragma unroll
    for (int i = 0; i < WAVE_ROWS; ++i) {
      m[i] = -FLT_MAX;
      l[i] = 0;
      o[i] = f32x4{0, 0, 0, 0};
    }
    const int row = row0 + wave * WAVE_ROWS;
    for (int64_t k = w0; k <= w1; ++k)
#pragma unroll
      for (int i = 0; i < WAVE_ROWS; ++i)
        if (r0 + row + i < rows) add(k, row + i, o[i], m[i], l[i]);
#pragma unroll
    for (int i = 0; i < WAVE_ROWS; ++i)
      if (r0 + row + i < rows) write(r0 + row + i, o[i], l[i]);
  } else {
    float m = -FLT_MAX, l = 0;
    f32x4 o = {0, 0, 0, 0};
    for (int64_t k = w0 + wave; k <= w1; k += 4) add(k, row0, o, m, l);
    *reinterpret_cast<f32x4*>(lds + wave * (kDim + 4) + 4 * lane) = o;
    if (lane == 0) {
      lds[wave * (kDim + 4) + kDim] = m;
      lds[wave * (kDim + 4) + kDim + 1] = l;
    }
    __syncthreads();
    if (wave != 0) return;
    float mx = -FLT_MAX;
#pragma unroll
    for (int k = 0; k < 4; ++k) mx = fmaxf(mx, lds[k * (kDim + 4) + kDim]);
    l = 0;
    o = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float g = fast_exp2(lds[k * (kDim + 4) + kDim] - mx);
      l += lds[k * (kDim + 4) + kDim + 1] * g;
      o += *reinterpret_cast<const f32x4*>(lds + k * (kDim + 4) + 4 * lane) * g;
    }
    write(r0 + row0, o, l);
  }
}

}  // namespace hlwq_kv
