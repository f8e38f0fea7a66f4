// attention_tile.h — the matrix-core attention for many query rows: a
// workgroup takes 32 rows a wave and streams keys and values through LDS.
//
// A row is a (token, query head) pair of one KV head, row r of a request being
// token r / group, head r % group, so that grouped heads fill the same tile and
// share every key and value that is read.  Per 32 keys and wave: 16 products of
// 32x32x16 for S^T, the softmax of 16 scores a lane, 16 products for O^T.  The
// sums O^T stay in 128 registers, Q in 64.
//
// What bounds it: per 32 keys a wave's products take 1024 cycles of its SIMD's
// matrix core, its softmax and addresses about 200 VALU instructions (1000
// cycles with the exponentials), and it reads 32 KB from LDS.  With two waves a
// SIMD the CU reads 256 KB in 2048 matrix cycles, half of what LDS gives (K as
// b128, V transposed on the way by ds_read_tr16).  The two waves stand at the
// same barrier once a block, so their softmaxes meet more often than they pass
// each other: over 16384 tokens (24 heads on 4) the matrix cores are 60% busy
// and VALU issue 33%, 2.78 ms, 1.19 PFLOP/s (1.36 to 1.56 in a large library
// product).  517 tokens take 26 us, nine packed prompts of 1 to 2500 tokens
// (16 heads on 2) 196 us.
//
// A load from scratch memory in the loop over blocks waits for all loads under
// way, those of the next block among them (a single spilled register took 6%).
// The two kernels with blocks of 64 keys have none there; the one of four waves
// and 32 keys still reloads one register a block.
#pragma once

#include "attention_common.h"
#include "staging.h"

namespace hlwq_kv {

// LDS tile of keys (or values): key k's 256 values in 32 chunks of 16 bytes at
// 512 k, chunk c in place c ^ swizzle(k).  Sixteen lanes that read the same
// chunk of sixteen keys then hit different banks, and so do the four keys by
// 64 bytes of a transposed read of V.
__device__ __forceinline__ int swizzle(int key) { return ((key & 3) << 2) | ((key >> 2) & 3); }

// One wave's 32 rows.
struct Rows {
  f32x16 o[8];  // o[t][i]: value 32 t + 8 (i / 4) + 4 (lane / 32) + i % 4 of row lane % 32
  float m, l;   // running maximum (of scores times log2 e) and this lane's share of the sum
};

__device__ __forceinline__ void clear(Rows& r) {
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) r.o[t][i] = 0;
}

__device__ __forceinline__ void scale_rows(Rows& r, float f) {
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) r.o[t][i] *= f;
}

template <bool ENC>
__device__ __forceinline__ f32x16 mfma32(u32x4 a, u32x4 b, f32x16 c) {
  if constexpr (ENC)
    return __builtin_amdgcn_mfma_f32_32x32x16_f16(__builtin_bit_cast(f16x8, a), __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// The lane's number, which the compiler takes for a new one each time: what it
// computes from it stays in no register from one use to the next.
__device__ __forceinline__ int lane_now() {
  int lane;
  asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(lane));
  return lane;
}

// Lane constants of the LDS reads.  What distinguishes the reads of a step is
// three bits of the address, to be exclusive-ored in (they meet the swizzle),
// and an offset that the instruction adds.
struct TileLane {
  uint32_t k;  // chunk 0 (or 1, upper half) of key lane % 32
  uint32_t v;  // transposed read of value block 0, keys 0 .. 3 (4 .. 7, upper half)
};
__device__ __forceinline__ TileLane tile_lane(int lane) {
  const int col = lane & 31, h = lane >> 5, l16 = lane & 15, g2 = (lane >> 4) & 1;
  TileLane t;
  t.k = col * 512 + ((h ^ swizzle(col)) * 16);
  t.v = (4 * h + (l16 >> 2)) * 512 + ((((2 * g2 + ((l16 >> 1) & 1)) ^ h) + ((l16 >> 2) << 2)) * 16) + 8 * (l16 & 1);
  return t;
}

// Fragment x of K for S^T's products over values 16 x .. of the 32 keys at `k`.
__device__ __forceinline__ u32x4 k_fragment(uint32_t k, int x) {
  return lds_at<u32x4>((k ^ ((x & 7) * 32)) + (x >> 3) * 256);
}

// Fragment x = 2 t + s of V^T for O^T's rows 32 t .. and keys 16 s .. of the 32
// at `v`: ds_read_tr16_b64 gives lane i of sixteen the element i % 4 of the
// four lanes i / 4 + 4 j, so with lane r pointing at key r / 4, values 4 (r %
// 4) .. the lane gets value i of four keys.
__device__ __forceinline__ u32x4 v_fragment(uint32_t v, int x) {
  const int t = x >> 1, off = (t >> 2) * 256 + (x & 1) * 8192;
  const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)static_cast<uintptr_t>((v ^ ((t & 3) * 64)) + off));
  const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)static_cast<uintptr_t>((v ^ ((t & 3) * 64 + 32)) + (off + 4096)));
  return __builtin_bit_cast(u32x4, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

// One step of 32 keys whose K and V lie in LDS at k and v (lane addresses), for
// rows that see keys 0 .. lim of them.
//   ENC: centroids in fp16; kn, vn: LDS addresses of the 32 keys' norms (kn < 0
//   where a key is not there; vn over the tile's scale), masked: some key is
//   not.
//   otherwise bf16, masked: some row does not see some key.
// factor turns a product into a score times log2 e.
template <bool ENC>
__device__ __forceinline__ void key_step(Rows& r, const u32x4 (&q)[16], uint32_t k, uint32_t v, float factor,
                                         int lim, bool masked, uint32_t kn, uint32_t vn) {
  constexpr int PK = 4, PV = 4;  // fragments in flight: what fits the registers beside the sums
  f32x16 s;
#pragma unroll
  for (int i = 0; i < 16; ++i) s[i] = 0;
  u32x4 kf[PK];
  const auto k_read = [&](int x) { kf[x % PK] = k_fragment(k, x); };
#pragma unroll
  for (int x = 0; x < PK; ++x) k_read(x);
  __builtin_amdgcn_sched_group_barrier(0x100, PK, 0);
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    s = mfma32<ENC>(kf[x % PK], q[x], s);
    __builtin_amdgcn_sched_group_barrier(0x8, 1, 0);
    if (x + PK < 16) {
      k_read(x + PK);
      __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    }
  }
  // score i of a lane is key 8 (i / 4) + 4 h + i % 4
  if constexpr (ENC) {
    const int h = lane_now() >> 5;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 n = lds_at<f32x4>(kn + 32 * i + 16 * h);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[4 * i + j] *= n[j];
      }
    }
    if (masked) {
      keep_branch();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 n = lds_at<f32x4>(kn + 32 * i + 16 * h);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[4 * i + j] = n[j] < 0 ? -HUGE_VALF : s[4 * i + j];
      }
    }
  } else if (masked) {
    const int mine = lim - 4 * (lane_now() >> 5);
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] = 8 * (i / 4) + i % 4 > mine ? -HUGE_VALF : s[i];
  }
  float mx = s[0];
#pragma unroll
  for (int i = 1; i < 16; ++i) mx = fmaxf(mx, s[i]);
  mx = fmaxf(mx, half_swap(mx)) * factor;
  if (__any(mx - r.m > kLazy)) {
    const float mn = fmaxf(r.m, mx);
    const float f = fast_exp2(r.m - mn);
    r.m = mn;
    r.l *= f;
    scale_rows(r, f);
  }
  float p[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) p[i] = fast_exp2(__builtin_fmaf(s[i], factor, -r.m));
  float sum = 0;
#pragma unroll
  for (int i = 0; i < 16; i += 4) sum += (p[i] + p[i + 1]) + (p[i + 2] + p[i + 3]);
  r.l += sum;
  asm volatile("" : "+v"(r.l));  // now, so that the sixteen end here
  u32x4 pf[2];
  if constexpr (ENC) {
    const int h = lane_now() >> 5;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 n = lds_at<f32x4>(vn + 32 * i + 16 * h);
      pf[i >> 1][2 * (i & 1)] = pack_f16x2(p[4 * i] * n[0], p[4 * i + 1] * n[1]);
      pf[i >> 1][2 * (i & 1) + 1] = pack_f16x2(p[4 * i + 2] * n[2], p[4 * i + 3] * n[3]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) pf[i >> 2][i & 3] = pack_bf16x2(p[2 * i], p[2 * i + 1]);
  }
  u32x4 vf[PV];
#pragma unroll
  for (int x = 0; x < PV; ++x) vf[x] = v_fragment(v, x);
#pragma unroll
  for (int x = 0; x < 16; ++x) {
    __builtin_amdgcn_sched_barrier(0);  // else each read would move to right before its product
    r.o[x >> 1] = mfma32<ENC>(vf[x % PV], pf[x & 1], r.o[x >> 1]);
    if (x + PV < 16) vf[x % PV] = v_fragment(v, x + PV);
  }
}

// A masked key's value times its probability 0 is NaN where the value is
// infinite or NaN.  So before a block of `keys` values of which some row does
// not see some is worked on, the workgroup's T threads set such values in LDS
// to zero, with a note at `flag`; they are added at the end to the rows that
// see them (add_nonfinite).  (A branch to that work at each fragment of the
// products takes longer: few of the blocks are masked, but none of the others
// could then be scheduled as a whole.)
template <int T, int KEYS>
__device__ __forceinline__ void leave_out_nonfinite(uint32_t values, uint32_t flag) {
#pragma unroll
  for (int i = 0; i < KEYS * 32 / T; ++i) {
    const uint32_t at = values + (i * T + threadIdx.x) * 16;
    u32x4 v = lds_at<u32x4>(at);
    uint32_t any = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = finite_pair(v[j], any);
    if (any != 0) {
      lds_put<u32x4>(at, v);
      lds_put<uint32_t>(flag, 1);
    }
  }
  wait_lds();
  barrier();
}

// The infinite and NaN values that were left out, of keys [from, to]: added to
// the row if it sees their key (key <= lim).  value(key): the key's 256 values
// in memory.
template <class F>
__device__ __forceinline__ void add_nonfinite(Rows& r, uint32_t flag, int64_t from, int64_t to, int64_t lim, int h, F value) {
  if (__builtin_amdgcn_readfirstlane(lds_at<uint32_t>(flag)) == 0) return;
  for (int64_t key = from; key <= to; ++key) {
    const uint16_t* p = value(key);
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 w = *reinterpret_cast<const uint2*>(p + 32 * t + 8 * i + 4 * h);
        const float x[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
#pragma unroll
        for (int j = 0; j < 4; ++j) r.o[t][4 * i + j] += key <= lim && !__builtin_isfinite(x[j]) ? x[j] : 0.0f;
      }
  }
}

// ---------------------------------------------------------------------------
// Whole prompts.  A workgroup takes one tile of one KV head's rows, of NW waves
// with 32 each and blocks of KT keys; PARTS 2: half the waves take the first 32
// keys of each block and half the others, for the same rows, and their sums are
// joined at the end.  A causal tile costs as many keys as its last token has
// before it, so the longest start first: of up to 64 sequences the longest of
// all (212 us to 206 for nine packed prompts), else each sequence's.
// Consecutive workgroups take different KV heads, so that an XCD's L2 serves as
// few heads as there are.
// ---------------------------------------------------------------------------

template <int NW, int KT, int PARTS>
__global__ void __launch_bounds__(64 * NW) __attribute__((amdgpu_waves_per_eu(2, 2))) hlwq_prompt_attention_kernel(const AttnArgs a) {
  constexpr int kRows = 32 * NW / PARTS;
  constexpr uint32_t kStage = KT * 1024;  // K and V of one stage
  constexpr uint32_t kFlag = 2 * kStage, kStats = kFlag + 16;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kStats + (PARTS > 1 ? NW / 2 * 512 : 0)];
  static_assert(PARTS == 1 || (PARTS == 2 && KT == 64 && NW / 2 * 32768 <= 2 * kStage));
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, h = lane >> 5;
  const int head = blockIdx.x % a.kv_heads;
  const int g = a.group;

  const auto tiles = [&](const Extent& e) { return static_cast<int32_t>(ceil_div(e.n * g, kRows)); };
  Finder<decltype(tiles), Nothing> finder(a, tiles, Nothing{});
  if (static_cast<int32_t>(blockIdx.x / a.kv_heads) >= finder.total) return;
  const int32_t x = blockIdx.x / a.kv_heads;
  Found f;
  if (a.requests <= 64) {
    f = finder.find_from_last(x);
  } else {
    f = finder.find(x);
    f.rest = tiles(f.e) - 1 - f.rest;
  }
  const int32_t begin = f.e.begin, n = f.e.n, rows = n * g;
  const int32_t r0 = f.rest * kRows;  // the tile's first row
  const int strip = wave % (NW / PARTS), part = wave / (NW / PARTS);
  const int32_t w0 = r0 + 32 * strip;  // the wave's
  // tokens of the lane's row, of the wave's first and last, of the tile's last
  const int32_t tok = token_of(min(w0 + col, rows - 1), g);
  const auto q_head = [&]() { return head * g + (min(w0 + col, rows - 1) - tok * g); };
  const int32_t seen = token_of(r0, g) + 1;  // keys that every row of the tile sees
  const int32_t first = token_of(min(w0, rows - 1), g), last = w0 < rows ? token_of(min(w0 + 31, rows - 1), g) : -1;
  const int32_t end = token_of(min(r0 + kRows - 1, rows - 1), g) + 1;

  u32x4 q[16];
  {
    const uint16_t* qp = a.q + (begin + static_cast<int64_t>(tok)) * a.q_stride + q_head() * kDim + 8 * h;
#pragma unroll
    for (int s = 0; s < 16; ++s) q[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
  }
  Rows r;
  clear(r);
  r.m = -FLT_MAX;
  r.l = 0;
  const float factor = a.factor;

  // Stage i of a wave's KT / (2 NW): keys 2 NW i + 2 wave and the one after,
  // 512 bytes each, lane l the chunk that belongs in place l % 32.  Rows past
  // the sequence read as zeros.
  const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
  const auto stage = [&](int buf, int32_t t0) {
    const int64_t at = begin + static_cast<int64_t>(t0);
    const u32x4 kb = buffer_of(a.k_new + at * a.k_stride + head * kDim, ((n - t0 - 1) * a.k_stride + kDim) * 2);
    const u32x4 vb = buffer_of(a.v_new + at * a.v_stride + head * kDim, ((n - t0 - 1) * a.v_stride + kDim) * 2);
    const int now = lane_now(), key = 2 * wave + (now >> 5);
    const uint32_t place = ((now & 31) ^ swizzle(key)) * 16;
    const uint32_t ko = key * static_cast<uint32_t>(a.k_stride) * 2, vo = key * static_cast<uint32_t>(a.v_stride) * 2;
#pragma unroll
    for (int i = 0; i < KT / (2 * NW); ++i) {
      const int pair = 2 * NW * i + 2 * wave;
      // 8 keys on, the swizzle differs in one bit; 16 keys on, it is the same
      const uint32_t c = place ^ (swizzle(2 * NW * i) * 16);
      stage16(kb, ko + 2 * NW * i * static_cast<uint32_t>(a.k_stride) * 2 + c, base + buf * kStage + pair * 512);
      stage16(vb, vo + 2 * NW * i * static_cast<uint32_t>(a.v_stride) * 2 + c, base + buf * kStage + KT * 512 + pair * 512);
    }
  };
  const TileLane at = tile_lane(lane);
  const uint32_t flag = base + kFlag;
  if (threadIdx.x == 0) lds_put<uint32_t>(flag, 0);
  wait_lds();
  stage(0, 0);
  // settle Q before the loop (and turn it round for a negative scale), so that
  // no wait on its loads stands inside
#pragma unroll
  for (int s = 0; s < 16; ++s) {
    if (a.scale < 0) q[s] ^= 0x80008000u;
    asm volatile("" : "+v"(q[s]));
  }
  for (int32_t t0 = 0, buf = 0; t0 < end; t0 += KT, buf ^= 1) {
    wait_staged();
    barrier();
    if (t0 + KT < end) stage(buf ^ 1, t0 + KT);
    if (t0 + KT > seen) leave_out_nonfinite<64 * NW, KT>(base + buf * kStage + KT * 512, flag);
#pragma unroll
    for (int u = 0; u < KT / 32 / PARTS; ++u) {
      const int step = PARTS > 1 ? part : u;
      const int32_t k0 = t0 + 32 * step;
      if (k0 > last) continue;
      const uint32_t kb = base + buf * kStage + step * 16384, vb = kb + KT * 512;
      key_step<false>(r, q, kb + at.k, vb + at.v, factor, tok - k0, k0 + 31 > first, 0, 0);
    }
  }
  add_nonfinite(r, flag, seen / KT * KT, part > 0 ? -1 : last, tok, h, [&](int64_t key) {
    return a.v_new + (begin + key) * a.v_stride + head * kDim;
  });
  if constexpr (PARTS > 1) {
    // the second part's sums to the first, through the stages
#pragma unroll
    for (int t = 0; t < 8; ++t) asm volatile("" : "+v"(r.o[t]));  // the loop's registers end here
    barrier();
    const uint32_t to = base + strip * 32768 + lane_now() * 16, stat = base + kStats + strip * 512 + lane_now() * 8;
    if (part > 0) {
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          lds_put<f32x4>(to + (4 * t + i) * 1024, f32x4{r.o[t][4 * i], r.o[t][4 * i + 1], r.o[t][4 * i + 2], r.o[t][4 * i + 3]});
      lds_put<f32x2>(stat, f32x2{r.m, r.l});
    }
    wait_lds();
    barrier();
    if (part > 0) return;
    const f32x2 s = lds_at<f32x2>(stat);
    // above 0, as an infinite value times 0 would be NaN
    const float m = fmaxf(r.m, s[0]), f0 = fmaxf(fast_exp2(r.m - m), FLT_MIN), f1 = fast_exp2(s[0] - m);
    r.l = r.l * f0 + s[1] * f1;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x4 o = lds_at<f32x4>(to + (4 * t + i) * 1024);
#pragma unroll
        for (int j = 0; j < 4; ++j) r.o[t][4 * i + j] = r.o[t][4 * i + j] * f0 + o[j] * f1;
        __builtin_amdgcn_sched_barrier(0);  // few of the other's sums in registers at once
      }
  }
  r.l += half_swap(r.l);
  const float inv = 1.0f / r.l;
  if (w0 + col < rows) {
    uint16_t* op = a.out + ((begin + static_cast<int64_t>(tok)) * a.q_heads + q_head()) * kDim;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint2 w = {pack_bf16x2(r.o[t][4 * i] * inv, r.o[t][4 * i + 1] * inv),
                         pack_bf16x2(r.o[t][4 * i + 2] * inv, r.o[t][4 * i + 3] * inv)};
        *reinterpret_cast<uint2*>(op + 32 * t + 8 * i + 4 * h) = w;
      }
  }
}

}  // namespace hlwq_kv
