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
// A workgroup is four waves with 32 tokens each to a block of 128.  Some
// workgroups share the pages' blocks of all requests in equal stretches, one
// more per tile (sixteen rows of a KV head) takes the window's and the step's
// own tokens; each joins its waves' sums in LDS and leaves them in the
// workspace, and a second kernel joins a tile's.  A workgroup runs through its
// code once or twice, so what bounds a short call is the fetching of
// instructions: what is not in the loop over blocks is kept small, not unrolled.
//
// Sixteen rows take 256 registers, so that two workgroups share a CU; 32 rows
// read each code half as often but take all 512 and leave one, which took 28.5
// us for 24 rows over 16000 tokens (24.7) and 47 for 8 requests over 4000 (34).
//
// Measured (24 query heads on 4, kernel and join): one token over 500, 9.7 + 4.0
// us; over 32767, 18.7 + 5.2 us for 26 MB, of which 5.5 us are memory's and the
// rest a chain of latencies (lengths, pages, codes, partial sums).  48 ragged
// requests, 2 bits, 115 MB: 48.6 + 7.4 us, VALU issue 46% busy and the matrix
// cores 9%; a step of 32 tokens takes about 600 VALU instructions a wave, four
// tenths of them look-ups.
#pragma once

#include "attention_common.h"

namespace hlwq_kv {

typedef uint32_t u32x2_4 __attribute__((ext_vector_type(2), aligned(4)));
typedef uint32_t u32x3_4 __attribute__((ext_vector_type(3), aligned(4)));

constexpr int kSplitThreads = 256;
constexpr int kSplitRows = 16;
constexpr int kSplitBlock = 128;  // tokens to a block
constexpr int kSplitPitch = kDim + 4;  // floats to a row of sums in LDS: rows 4 banks apart

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

// One wave's sums over its tokens: o[s][i] is value 16 (4 (lane / 16) + i) + s
// of row lane % 16.
struct SplitRows {
  f32x4 o[16];
  float m, l;
  int exponent;  // of the pages' values: sums are over p n 2^-exponent
};

__device__ __forceinline__ void clear(SplitRows& r) {
#pragma unroll
  for (int s = 0; s < 16; ++s) r.o[s] = f32x4{0, 0, 0, 0};
  r.m = -FLT_MAX;
  r.l = 0;
  r.exponent = -64;
}

// Softmax weights of a lane's eight scores, s[..] times factor;
// gone[i]: the token is not seen by the row.
template <class G>
__device__ __forceinline__ void weigh(SplitRows& r, float (&s)[8], float factor, bool masked, G gone, float (&p)[8]) {
  if (masked) {
    keep_branch();
#pragma unroll
    for (int i = 0; i < 8; ++i) s[i] = gone(i) ? -HUGE_VALF : s[i];
  }
  float mx = s[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, s[i]);
  mx = group_max(mx) * factor;
  if (__any(mx - r.m > kLazy)) {
    const float mn = fmaxf(r.m, mx);
    const float f = fast_exp2(r.m - mn);
    r.m = mn;
    r.l *= f;
#pragma unroll
    for (int x = 0; x < 16; ++x) r.o[x] *= f;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = fast_exp2(__builtin_fmaf(s[i], factor, -r.m));
    r.l += p[i];
  }
}

// 32 encoded tokens; there: how many of each sixteen exist.
template <int BITS>
__device__ __forceinline__ void code_step(SplitRows& r, const u32x4 (&q)[8], float factor, const Codes<BITS>& c, int there_a,
                                          int there_b, int lane) {
  const int h4 = lane >> 4;
  const bool odd = lane & 1, masked = there_a < 16 || there_b < 16;
  f32x4 s[2];
#pragma unroll
  for (int sub = 0; sub < 2; ++sub) {
    u32x4 f[8];
    k_fragments<BITS>(c, sub, f);
    s[sub] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < 8; ++x) s[sub] = mfma16<true>(f[x], q[x], s[sub]);
  }
  float kn[8], vn[8];
  const auto gone = [&](int i) { return 4 * h4 + (i & 3) >= (i < 4 ? there_a : there_b); };
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t kw = c.kn[i >> 2][(i >> 1) & 1], vw = c.vn[i >> 2][(i >> 1) & 1];
    kn[i] = f16_value(static_cast<uint16_t>(i & 1 ? kw >> 16 : kw));
    vn[i] = f16_value(static_cast<uint16_t>(i & 1 ? vw >> 16 : vw));
  }
  if (masked) {
    keep_branch();
#pragma unroll
    for (int i = 0; i < 8; ++i) vn[i] = gone(i) ? 0.0f : vn[i];
  }
  // The weights p n are products' operands in fp16, so n is taken over a power
  // of two that no norm met so far exceeds, times kTopWeight: a weight is at most
  // 2^15 and keeps its 2^-11 down to 2^-29 of that.  A token with the row's
  // largest score thus does up to norms 2^21 times its own.
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
    for (int x = 0; x < 16; ++x) r.o[x] *= f;
  }
  const float over = __builtin_ldexpf(kTopWeight, -r.exponent);
  u32x4 pf;
  float t[8], p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = s[i >> 2][i & 3] * kn[i];
  weigh(r, t, factor, masked, gone, p);
#pragma unroll
  for (int i = 0; i < 4; ++i) pf[i] = pack_f16x2(p[2 * i] * (vn[2 * i] * over), p[2 * i + 1] * (vn[2 * i + 1] * over));
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint32_t ca[8], cb[8];
    v_codes<BITS>(c, 0, half, odd, ca);
    v_codes<BITS>(c, 1, half, odd, cb);
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const u32x2 a = look_up<BITS>(ca[x]), b = look_up<BITS>(cb[x]);
      const u32x4 f{a[0], a[1], b[0], b[1]};
      r.o[8 * half + x] = mfma16<true>(f, pf, r.o[8 * half + x]);
    }
  }
}

__constant__ uint16_t c_zero_vector[kDim] = {};

// Where the window's and the step's tokens of a KV head lie, K and V: token k
// below `near` in ring slot ring0 + k (mod ring), the others in the step's rows.
struct Tokens {
  const uint16_t *window[2], *rows[2];
  uint32_t stride[2];  // of the rows; the window's is kDim
  int64_t near, ring0, ring;
  __device__ __forceinline__ Tokens(const AttnArgs& a, const Extent& e, int32_t b, int32_t head) {
    const int64_t w = (static_cast<int64_t>(b) * a.kv_heads + head) * a.ring * kDim;
    window[0] = a.k_window + w;
    window[1] = a.v_window + w;
    stride[0] = static_cast<uint32_t>(a.k_stride);
    stride[1] = static_cast<uint32_t>(a.v_stride);
    rows[0] = a.k_new + e.begin * a.k_stride + head * kDim;
    rows[1] = a.v_new + e.begin * a.v_stride + head * kDim;
    near = e.held - e.enc;
    ring = a.ring;
    ring0 = near > 0 ? static_cast<uint32_t>(e.enc) % static_cast<uint32_t>(a.ring) : 0;  // both below 2^31
  }
  // Token k's vector: selects and one multiply, no branch, so that loads of
  // several tokens are in flight together.  Past `last`, a vector of zeros.
  __device__ __forceinline__ const uint16_t* at(int side, int64_t k, int64_t last) const {
    if (k > last) return c_zero_vector;
    const bool in = k < near;
    const int64_t slot = ring0 + k >= ring ? ring0 + k - ring : ring0 + k;
    const uint32_t index = static_cast<uint32_t>(in ? slot : k - near);
    return (in ? window[side] : rows[side]) + static_cast<uint64_t>(index) * (in ? static_cast<uint32_t>(kDim) : stride[side]);
  }
};

// 32 bf16 tokens from k0 on; lim: last token that the lane's row sees; last:
// the last one there is.  masked: some row does not see some token; mixed: nor
// do all that are there see the same.
__device__ __forceinline__ void token_step(SplitRows& r, const u32x4 (&q)[8], float factor, int64_t k0, int64_t last,
                                           int64_t lim, bool masked, bool mixed, const Tokens& tokens, int lane) {
  const int c = lane & 15, h4 = lane >> 4;
  const auto token = [&](int i) { return k0 + 16 * (i >> 2) + 4 * h4 + (i & 3); };
  // every load before the first use
  u32x4 f[2][8], v[2][8];
#pragma unroll
  for (int sub = 0; sub < 2; ++sub) {
    const uint16_t* p = tokens.at(0, k0 + 16 * sub + c, last) + 8 * h4;
#pragma unroll
    for (int x = 0; x < 8; ++x) f[sub][x] = *reinterpret_cast<const u32x4*>(p + 32 * x);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint16_t* p = tokens.at(1, token(i), last) + 16 * c;
    v[0][i] = *reinterpret_cast<const u32x4*>(p);
    v[1][i] = *reinterpret_cast<const u32x4*>(p + 8);
  }
#pragma unroll
  for (int sub = 0; sub < 2; ++sub)
#pragma unroll
    for (int x = 0; x < 8; ++x) asm volatile("" : "+v"(f[sub][x]));
  f32x4 s[2];
#pragma unroll
  for (int sub = 0; sub < 2; ++sub) {
    s[sub] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int x = 0; x < 8; ++x) s[sub] = mfma16<false>(f[sub][x], q[x], s[sub]);
  }
  u32x4 pf;
  float t[8], p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = s[i >> 2][i & 3];
  weigh(r, t, factor, masked, [&](int i) { return token(i) > lim; }, p);
#pragma unroll
  for (int i = 0; i < 4; ++i) pf[i] = pack_bf16x2(p[2 * i], p[2 * i + 1]);
  // as in key_step: where some rows see a token and others do not, 0 times its
  // value must stay 0
  uint32_t left = 0;
  if (mixed) {
#pragma unroll
    for (int half = 0; half < 2; ++half)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) v[half][i][x] = finite_pair(v[half][i][x], left);
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const uint32_t sel = x & 1 ? 0x07060302u : 0x05040100u;
      u32x4 f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        f[i] = __builtin_amdgcn_perm(v[half][2 * i + 1][x >> 1], v[half][2 * i][x >> 1], sel);
      }
      r.o[8 * half + x] = mfma16<false>(f, pf, r.o[8 * half + x]);
    }
  }
  if (mixed && __any(left != 0)) {
    for (int k = 0; k < 32 && k0 + k <= last; ++k) {
      const uint16_t* p = tokens.at(1, k0 + k, last) + 64 * h4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const float v = bf16_lo(p[16 * i + x]);
          r.o[x][i] += k0 + k <= lim && !__builtin_isfinite(v) ? v : 0.0f;
        }
    }
  }
}

// An output row from its sums.
__device__ __forceinline__ void write_row(const AttnArgs& a, int32_t begin, int32_t head, int32_t row, f32x4 o, float l, int lane) {
  const float inv = 1.0f / l;
  const int32_t token = token_of(row, a.group);
  const int64_t at = (begin + static_cast<int64_t>(token)) * a.q_heads + head * a.group + (row - token * a.group);
  *reinterpret_cast<uint2*>(a.out + at * kDim + 4 * lane) = uint2{pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv)};
}

constexpr int kSplitStats = 4 * 16 * 2;  // floats

// The four waves' sums of a tile's `there` rows joined, rotated if they are
// over centroids, and given to write(row, sums of lane's four values, maximum,
// sum of weights).
template <class F>
__device__ __forceinline__ void join_waves(SplitRows& r, bool enc, int there, float* lds, int lane, int wave, F write) {
  const int c = lane & 15, h4 = lane >> 4;
  const float f = enc ? __builtin_ldexpf(1.0f / kTopWeight, r.exponent - 8) : 1.0f;  // H c n / 256
  float* stat = lds + 4 * 16 * kSplitPitch;
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
  for (int row = wave; row < min(there, kSplitRows); row += 4) {
    float2 s[4];
    float m = -FLT_MAX;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      s[w] = *reinterpret_cast<const float2*>(stat + (w * 16 + row) * 2);
      m = fmaxf(m, s[w].x);
    }
    float o[4] = {0, 0, 0, 0}, sum = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      const float g = fast_exp2(s[w].x - m);
      sum += s[w].y * g;
      const f32x4 v = *reinterpret_cast<const f32x4*>(lds + (w * 16 + row) * kSplitPitch + 4 * lane);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] += v[e] * g;
    }
    if (enc) wave_fwht(o, lane);
    write(row, f32x4{o[0], o[1], o[2], o[3]}, m, sum);
  }
}

// What a request asks of the split kernel.
struct SplitWork {
  Extent e;
  int32_t tiles, blocks;  // tiles of a KV head, page blocks of each
  __device__ __forceinline__ SplitWork(const AttnArgs& a, const Extent& x) {
    e = x;
    const int32_t r = e.n * a.group;
    tiles = r >= a.least && r <= a.most ? static_cast<int32_t>(ceil_div(r, kSplitRows)) : 0;
    blocks = static_cast<int32_t>(ceil_div(e.paged, kSplitBlock));
  }
};
// Slots of partial sums (attention_common.h): after the workers' come two to a
// tile, for pages that one workgroup took whole and for the other tokens.
__device__ __forceinline__ int32_t tile_slot(const AttnArgs& a, int32_t tile, int which) { return 2 * (a.workers + tile) + which; }

// A query row is rotated as q / 256: exact for every bf16, subnormals too, and a
// sum of 256 values then never passes fp32.
constexpr float kQueryScale = 1.0f / 256;

// The exponent of a rotated query row's largest value: the row over 2^that lies in
// [1, 2), or below 1 where 1 / 2^that would pass fp32 (rows under 2^-126).
__device__ __forceinline__ int row_exponent(float top) {
  return top > 0 ? max(__builtin_amdgcn_frexp_expf(top) - 1, -126) : 0;
}

// Pages [u0, u1) of a tile.
template <int BITS, class F>
__device__ __forceinline__ void attend_pages(const AttnArgs& a, const Extent& e, int32_t b, int32_t head, int32_t r0, int32_t u0,
                                             int32_t u1, float* lds, int lane, int wave, F write) {
  constexpr int M = kSplitRows;
  constexpr int kQPitch = kDim + 8;  // fp16 to a row of rotated q in LDS
  const int c = lane & 15, h4 = lane >> 4;
  const int32_t rows = e.n * a.group;
  // Pages: lane 2 i + s holds that of sixteen s of the wave's 32 tokens of
  // block u0 + i, for 32 blocks at a time and the next 32 ahead.
  const auto pages = [&](int32_t u) {
    const int64_t t = static_cast<int64_t>(u + (lane >> 1)) * kSplitBlock + 32 * wave + 16 * (lane & 1);
    const int32_t id = t < e.paged ? a.table[static_cast<int64_t>(b) * a.width + (t >> a.page_shift)] : -1;
    return id < a.n_pages ? id : -1;
  };
  int32_t ids = pages(u0), ids_ahead = u0 + 32 < u1 ? pages(u0 + 32) : -1;

  const auto q_load = [&](int row) {
    const int32_t token = token_of(min(r0 + row, rows - 1), a.group);
    return *reinterpret_cast<const uint2*>(a.q + (e.begin + static_cast<int64_t>(token)) * a.q_stride +
                                           (head * a.group + (min(r0 + row, rows - 1) - token * a.group)) * kDim + 4 * lane);
  };
  uint2 v = q_load(wave);

  const auto fetch = [&](int32_t u, Codes<BITS>& to, int (&there)[2]) {
    const int at = (u - u0) & 31;
    if (at == 0 && u > u0) {
      ids = ids_ahead;
      if (u + 32 < u1) ids_ahead = pages(u + 32);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int64_t t = static_cast<int64_t>(u) * kSplitBlock + 32 * wave + 16 * s;
      const int32_t id = __builtin_amdgcn_readlane(ids, 2 * at + s);
      there[s] = id < 0 ? 0 : static_cast<int>(min(e.paged - t, int64_t{16}));
      const int64_t vec = ((static_cast<int64_t>(max(id, 0)) * a.kv_heads + head) << a.page_shift) + (t & ((1 << a.page_shift) - 1));
      load_codes<BITS>(to, a, s, vec, lane);
    }
  };
  Codes<BITS> codes[2];
  int there[2][2];
  fetch(u0, codes[0], there[0]);

  // q rotated, each row over a power of two that brings its largest value to
  // [1, 2), as fp16, while the codes are on their way
  uint16_t* ql = reinterpret_cast<uint16_t*>(lds);
  float* qf = lds + M * kQPitch / 2;
#pragma clang loop unroll(disable)
  for (int row = wave; row < M; row += 4) {
    float x[4] = {bf16_lo(v.x) * kQueryScale, bf16_hi(v.x) * kQueryScale, bf16_lo(v.y) * kQueryScale, bf16_hi(v.y) * kQueryScale};
    if (r0 + row + 4 < rows && row + 4 < M) v = q_load(row + 4);
    if (r0 + row >= rows) {  // rows that are not there: zeros, and no more to load
      *reinterpret_cast<uint2*>(ql + row * kQPitch + 4 * lane) = uint2{0, 0};
      if (lane == 0) qf[row] = 1;
      continue;
    }
    wave_fwht(x, lane);
    const float mx = wave_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3]))));
    const int ex = row_exponent(mx);
    const float f = __builtin_ldexpf(a.scale < 0 ? -1.0f : 1.0f, -ex);
    *reinterpret_cast<uint2*>(ql + row * kQPitch + 4 * lane) = uint2{pack_f16x2(x[0] * f, x[1] * f), pack_f16x2(x[2] * f, x[3] * f)};
    if (lane == 0) qf[row] = fmaxf(__builtin_ldexpf(a.factor, ex), __FLT_DENORM_MIN__);
  }
  __syncthreads();
  u32x4 q[8];
  const float factor = qf[c];
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    uint32_t d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      d[k] = *reinterpret_cast<const uint32_t*>(ql + c * kQPitch + 64 * h4 + dim_of<BITS>(x, k));
    q[x] = u32x4{__builtin_amdgcn_perm(d[1], d[0], 0x05040100u), __builtin_amdgcn_perm(d[3], d[2], 0x05040100u),
                 __builtin_amdgcn_perm(d[1], d[0], 0x07060302u), __builtin_amdgcn_perm(d[3], d[2], 0x07060302u)};
  }
  SplitRows r;
  clear(r);
  // block u while the codes of u + 1 are on their way; by twos, as moving them
  // from one set of registers to the other took a tenth of the step
  for (int32_t u = u0; u < u1; u += 2)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (u + k >= u1) break;
      if (u + k + 1 < u1) fetch(u + k + 1, codes[k ^ 1], there[k ^ 1]);
      if (there[k][0] + there[k][1] > 0) code_step<BITS>(r, q, factor, codes[k], there[k][0], there[k][1], lane);
    }
  join_waves(r, true, rows - r0, lds, lane, wave, write);
}

// The window's and the step's own tokens of a tile.
template <class F>
__device__ __forceinline__ void attend_tokens(const AttnArgs& a, const Extent& e, int32_t b, int32_t head, int32_t r0, float* lds,
                                              int lane, int wave, F write) {
  constexpr int M = kSplitRows;
  const int c = lane & 15, h4 = lane >> 4;
  const int32_t rows = e.n * a.group;
  const Tokens tokens(a, e, b, head);
  const int64_t first = tokens.near + token_of(r0, a.group), last = tokens.near + token_of(min(r0 + M, rows) - 1, a.group);
  u32x4 q[8];
  const int32_t row = min(r0 + c, rows - 1), token = token_of(row, a.group);
  const int32_t q_head = head * a.group + (row - token * a.group);
  const uint16_t* p = a.q + (e.begin + static_cast<int64_t>(token)) * a.q_stride + q_head * kDim + 8 * h4;
  const int64_t lim = tokens.near + token;
#pragma unroll
  for (int x = 0; x < 8; ++x) {
    q[x] = *reinterpret_cast<const u32x4*>(p + 32 * x);
    if (a.scale < 0) q[x] ^= 0x80008000u;
  }
  SplitRows r;
  clear(r);
  for (int64_t k0 = 32 * wave; k0 <= last; k0 += kSplitBlock)
    token_step(r, q, a.factor, k0, last, lim, k0 + 31 > first, k0 + 31 > first && first < last, tokens, lane);
  join_waves(r, false, rows - r0, lds, lane, wave, write);
}

template <int BITS>
__global__ void __launch_bounds__(kSplitThreads) __attribute__((amdgpu_waves_per_eu(2, 2)))
hlwq_split_attention_kernel(const AttnArgs a) {
  constexpr int M = kSplitRows;
  __shared__ __attribute__((aligned(16))) float lds[4 * 16 * kSplitPitch + kSplitStats];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const auto tiles = [&](const Extent& e) { return SplitWork(a, e).tiles * a.kv_heads; };
  const auto cost = [&](const Extent& e) {
    const SplitWork w(a, e);
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
    const SplitWork w(a, f.e);
    const int32_t head = quotient(f.rest, w.tiles), r0 = (f.rest - head * w.tiles) * M;
    const int32_t slot = tile_slot(a, x, 1);
    attend_tokens(a, w.e, f.b, head, r0, lds, lane, wave, [&](int row, f32x4 o, float m, float l) {
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
    const SplitWork w(a, b == first.b ? first.e : extent_of(a, b));
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
    attend_pages<BITS>(a, w.e, b, head, (tile - head * w.tiles) * M, u0, u1, lds, lane, wave, to_slot(slot));
    __syncthreads();
    left -= u1 - u0;
    rest += u1 - u0;
  }
}

// Joins a row of a tile from the partial sums of its pages and its other
// tokens, each wave every fourth.
__global__ void __launch_bounds__(kSplitThreads) hlwq_split_join_kernel(const AttnArgs a) {
  constexpr int M = kSplitRows;
  __shared__ __attribute__((aligned(16))) float lds[4 * kSplitPitch];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const auto tiles = [&](const Extent& e) { return SplitWork(a, e).tiles * a.kv_heads; };
  const auto cost = [&](const Extent& e) {
    const SplitWork w(a, e);
    return w.tiles * w.blocks * a.kv_heads;
  };
  Finder<decltype(tiles), decltype(cost)> finder(a, tiles, cost);
  const int32_t x = blockIdx.x / M, row = blockIdx.x % M;
  if (x >= finder.total) return;
  const Found f = finder.find(x);
  const SplitWork w(a, f.e);
  const int32_t head = quotient(f.rest, w.tiles), r0 = (f.rest - head * w.tiles) * M;
  if (w.blocks == 0 || r0 + row >= w.e.n * a.group) return;
  const Share share(Finder<decltype(cost), Nothing>(a, cost, Nothing{}).total, a.workers, 1);
  const int32_t x0 = f.before + f.rest * w.blocks;
  const int32_t w0 = share.worker_at(x0), w1 = share.worker_at(x0 + w.blocks - 1);
  const int32_t parts = w1 - w0 + 2;  // the pages', then the other tokens'
  const auto slot_of = [&](int32_t k) {
    return k == parts - 1 ? tile_slot(a, x, 1) : w0 == w1 ? tile_slot(a, x, 0) : 2 * (w0 + k) + (k == 0 ? 1 : 0);
  };

  // 64 partial sums at a time: a lane reads each one's maximum and sum, then
  // the weighted rows, several in flight
  float m = -FLT_MAX, l = 0;
  f32x4 o = {0, 0, 0, 0};
  for (int32_t k0 = wave; k0 < parts; k0 += 256) {
    float2 s{-FLT_MAX, 0};
    if (k0 + 4 * lane < parts) s = *partial_stat<M>(a, slot_of(k0 + 4 * lane), row);
    const float mn = fmaxf(m, wave_max(s.x)), old = fast_exp2(m - mn), g = fast_exp2(s.x - mn);
    m = mn;
    l = l * old + wave_sum(s.y * g);
    o *= old;
    const int count = min((parts - k0 + 3) / 4, 64);
    for (int i = 0; i < count; i += 8) {
      f32x4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        v[j] = *reinterpret_cast<const f32x4*>(partial_row<M>(a, slot_of(k0 + 4 * min(i + j, count - 1)), row) + 4 * lane);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (i + j < count) o += v[j] * __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(g), i + j));
    }
  }
  *reinterpret_cast<f32x4*>(lds + wave * kSplitPitch + 4 * lane) = o;
  if (lane == 0) {
    lds[wave * kSplitPitch + kDim] = m;
    lds[wave * kSplitPitch + kDim + 1] = l;
  }
  __syncthreads();
  if (wave != 0) return;
  float mx = -FLT_MAX;
#pragma unroll
  for (int k = 0; k < 4; ++k) mx = fmaxf(mx, lds[k * kSplitPitch + kDim]);
  l = 0;
  o = f32x4{0, 0, 0, 0};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float g = fast_exp2(lds[k * kSplitPitch + kDim] - mx);
    l += lds[k * kSplitPitch + kDim + 1] * g;
    o += *reinterpret_cast<const f32x4*>(lds + k * kSplitPitch + 4 * lane) * g;
  }
  write_row(a, w.e.begin, head, r0 + row, o, l, lane);
}

}  // namespace hlwq_kv
