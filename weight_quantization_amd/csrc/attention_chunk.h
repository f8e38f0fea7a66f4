// attention_chunk.h — attention of many new tokens over a paged cache: the tile
// kernel of attention_tile.h with a first phase over pages of codes.
//
// Pages are worked on in the rotated domain (attention_split.h): the 512
// work-items unpack 64 tokens' codes into LDS as fp16 centroids while the
// previous 64 are multiplied, so that 256 query rows share one unpacking; then
// the sums are rotated in registers and the window's and the step's own tokens
// follow in bf16.
#pragma once

#include "attention_split.h"
#include "attention_tile.h"

namespace hlwq_kv {

constexpr int kChunkRows = 256;
constexpr int kChunkBlock = 64;   // tokens to a block
constexpr int kChunkLeast = 4 * kBlockCost;  // cost that is worth a workgroup of its own

// Butterflies over the 256 values of a row whose lanes hold 128 each, v[x] of
// the lower half and of the upper half differing in one bit of their index,
// any order of the others in x.
__device__ __forceinline__ void fwht_halves(float (&v)[128]) {
#pragma unroll
  for (int d = 1; d < 128; d <<= 1)
#pragma unroll
    for (int x = 0; x < 128; ++x)
      if ((x & d) == 0) {
        const float a = v[x], b = v[x + d];
        v[x] = a + b;
        v[x + d] = a - b;
      }
#pragma unroll
  for (int x = 0; x < 128; x += 2) {
    // halves swapped between two registers, added there, and swapped back
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[x]), __float_as_uint(v[x + 1]), false, false);
    const float lo = __uint_as_float(s[0]), hi = __uint_as_float(s[1]);
    const auto t = __builtin_amdgcn_permlane32_swap(__float_as_uint(lo + hi), __float_as_uint(lo - hi), false, false);
    v[x] = __uint_as_float(t[0]);
    v[x + 1] = __uint_as_float(t[1]);
  }
}

// 32 codes of a token, in order, to fp16 centroids: four chunks of eight.
__device__ __forceinline__ uint32_t spread_run3(uint32_t v) {  // 12 bits to four bytes
  const uint32_t a = (v | (v << 10)) & 0x003f003fu;
  return (a | (a << 5)) & 0x07070707u;
}
__device__ __forceinline__ uint32_t spread_run2(uint32_t v) {  // 8 bits to four bytes
  const uint32_t a = (v | (v << 12)) & 0x000f000fu;
  return (a | (a << 6)) & 0x03030303u;
}
template <int BITS>
struct Run {
  uint32_t w[BITS];
};
template <int BITS>
__device__ __forceinline__ u32x4 run_chunk(const Run<BITS>& r, int g) {
  uint32_t lo, hi;
  if constexpr (BITS == 3) {
    const uint32_t x = g == 0 ? r.w[0] : g == 1 ? __builtin_amdgcn_alignbit(r.w[1], r.w[0], 24)
                     : g == 2 ? __builtin_amdgcn_alignbit(r.w[2], r.w[1], 16) : r.w[2] >> 8;
    lo = spread_run3(x & 0xfffu);
    hi = spread_run3((x >> 12) & 0xfffu);
  } else {
    const uint32_t x = r.w[g >> 1] >> (16 * (g & 1));
    lo = spread_run2(x & 0xffu);
    hi = spread_run2((x >> 8) & 0xffu);
  }
  const u32x2 a = look_up<BITS>(lo), b = look_up<BITS>(hi);
  return u32x4{a[0], a[1], b[0], b[1]};
}

template <int BITS>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) hlwq_chunk_attention_kernel(const AttnArgs a) {
  constexpr int M = kChunkRows, KT = kChunkBlock;
  constexpr uint32_t kStage = KT * 1024;
  // two stages of K and V, then for each: K norms, V norms, {some token missing, V's exponent}
  constexpr uint32_t kSide = 2 * KT * 4 + 16;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * kStage + 2 * kSide];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int col = lane & 31, h = lane >> 5;
  const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));
  const TileLane at = tile_lane(lane);

  const auto cost = [&](const Extent& e) { return Work<M, KT>(a, e).head_cost() * a.kv_heads; };
  Finder<decltype(cost), Nothing> finder(a, cost, Nothing{});
  const Share share(finder.total, a.workers, kChunkLeast);
  if (finder.total == 0 || blockIdx.x >= share.workers) return;
  // Workgroups of one XCD (every eighth) take neighbouring stretches, which
  // share a KV head's keys in its L2.
  const int32_t worker = share.workers % 8 == 0 ? (blockIdx.x % 8) * (share.workers / 8) + blockIdx.x / 8 : blockIdx.x;
  const Found first = finder.find(share.bound(worker));

  for_segments<M, KT>(a, share, first, worker, [&](const Work<M, KT>& w, const Segment& g) {
    const Extent& e = w.e;
    const int32_t rows = w.rows(a), w0 = g.tile * M + 32 * wave;
    const int32_t blocks = w.blocks(a, g.tile);
    const int32_t u0 = w.block_at(g.from, blocks, g.cost), u1 = w.block_at(g.to, blocks, g.cost);
    const int64_t near = e.held - e.enc;
    const int32_t tok = token_of(min(w0 + col, rows - 1), a.group);
    const auto q_head = [&]() { return g.head * a.group + (min(w0 + col, rows - 1) - tok * a.group); };
    const auto q_ptr = [&]() { return a.q + (e.begin + static_cast<int64_t>(tok)) * a.q_stride + q_head() * kDim + 8 * h; };
    Rows r;
    r.m = -FLT_MAX;
    r.l = 0;
    r.left = 0;
    const bool idle = w0 >= rows;  // none of the wave's rows exists: it only stages

    if (u0 < w.page_blocks && u0 < u1) {
      const int64_t end = min(u1, w.page_blocks);
      // lane = token of the block, wave = which 32 of its 256 codes; wave 0 has
      // the K norms, wave 1 the V norms
      const auto page_of = [&](int64_t u) {
        const int64_t t = u * KT + lane;
        return t < e.paged ? a.table[static_cast<int64_t>(g.b) * a.width + (t >> a.page_shift)] : -1;
      };
      Run<BITS> ck, cv;
      uint16_t norm = 0;
      bool there = false;
      const auto fetch = [&](int64_t u, int32_t id) {
        there = id >= 0 && id < a.n_pages;
        const int64_t vec = (((there ? static_cast<int64_t>(id) : 0) * a.kv_heads + g.head) << a.page_shift) +
                            ((u * KT + lane) & ((1 << a.page_shift) - 1));
        const uint32_t* kp = reinterpret_cast<const uint32_t*>(a.k_packed + vec * (32 * BITS)) + BITS * wave;
        const uint32_t* vp = reinterpret_cast<const uint32_t*>(a.v_packed + vec * (32 * BITS)) + BITS * wave;
        if constexpr (BITS == 3) {
          const u32x3_4 k = *reinterpret_cast<const u32x3_4*>(kp), v = *reinterpret_cast<const u32x3_4*>(vp);
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            ck.w[i] = k[i];
            cv.w[i] = v[i];
          }
        } else {
          const u32x2 k = *reinterpret_cast<const u32x2*>(kp), v = *reinterpret_cast<const u32x2*>(vp);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ck.w[i] = k[i];
            cv.w[i] = v[i];
          }
        }
        if (wave == 0) norm = a.k_norms[vec];
        if (wave == 1) norm = a.v_norms[vec];
      };
      int exponent = -64;  // wave 1's
      const auto unpack = [&](int buf) {
        const uint32_t k = base + buf * kStage + lane * 512, v = k + KT * 512;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const uint32_t c = ((4 * wave + x) ^ swizzle(lane)) * 16;
          *reinterpret_cast<lds_u32x4*>(static_cast<uintptr_t>(k + c)) = run_chunk<BITS>(ck, x);
          *reinterpret_cast<lds_u32x4*>(static_cast<uintptr_t>(v + c)) = run_chunk<BITS>(cv, x);
        }
        const uint32_t side = base + 2 * kStage + buf * kSide;
        if (wave == 0) {
          *reinterpret_cast<lds_f32*>(static_cast<uintptr_t>(side + 4 * lane)) = there ? f16_value(norm) : -1.0f;
          const bool all = __all(there);
          if (lane == 0) *reinterpret_cast<lds_u32*>(static_cast<uintptr_t>(side + 8 * KT)) = !all;
        }
        if (wave == 1) {
          // as in code_step: norms over a power of two that none met so far exceeds
          const float n = there ? f16_value(norm) : 0.0f;
          const float top = wave_max(n);
          if (top > __builtin_ldexpf(1.0f, exponent)) exponent = __builtin_amdgcn_frexp_expf(top);
          *reinterpret_cast<lds_f32*>(static_cast<uintptr_t>(side + 4 * KT + 4 * lane)) = __builtin_ldexpf(n, -exponent);
          if (lane == 0) *reinterpret_cast<lds_u32*>(static_cast<uintptr_t>(side + 8 * KT + 4)) = exponent;
        }
      };
      fetch(u0, page_of(u0));
      int32_t id = u0 + 1 < end ? page_of(u0 + 1) : -1;

      // q rotated, over a power of two that brings the row's largest value to
      // [1, 2), as fp16
      u32x4 q[16];
      float factor;
      {
        float x[128];
        const uint16_t* qp = q_ptr();
#pragma unroll
        for (int s = 0; s < 16; ++s) {
          const u32x4 v = *reinterpret_cast<const u32x4*>(qp + 16 * s);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            x[8 * s + 2 * j] = bf16_lo(v[j]);
            x[8 * s + 2 * j + 1] = bf16_hi(v[j]);
          }
        }
        fwht_halves(x);
        float mx = 0;
#pragma unroll
        for (int i = 0; i < 128; ++i) mx = fmaxf(mx, fabsf(x[i]));
        mx = fmaxf(mx, half_swap(mx));
        const int ex = mx > 0 ? __builtin_amdgcn_frexp_expf(mx) - 1 : 0;
        const float f = __builtin_ldexpf(a.scale < 0 ? -1.0f : 1.0f, -ex);
#pragma unroll
        for (int s = 0; s < 16; ++s)
#pragma unroll
          for (int j = 0; j < 4; ++j) q[s][j] = pack_f16x2(x[8 * s + 2 * j] * f, x[8 * s + 2 * j + 1] * f);
        factor = __builtin_ldexpf(fabsf(a.scale) * kLog2e, ex - 8);
      }
      unpack(0);
      clear(r);
      int scaled = -64;
      for (int64_t u = u0; u < end; ++u) {
        const int buf = (u - u0) & 1;
        if (u + 1 < end) {
          fetch(u + 1, id);
          if (u + 2 < end) id = page_of(u + 2);
        }
        wait_lds();
        barrier();
        if (!idle) {
          const uint32_t side = base + 2 * kStage + buf * kSide;
          const u32x2 info = *reinterpret_cast<const lds_u32x2*>(static_cast<uintptr_t>(side + 8 * KT));
          const bool masked = __builtin_amdgcn_readfirstlane(info[0]) != 0;
          const int ex = __builtin_amdgcn_readfirstlane(info[1]);
          if (ex != scaled) {
            scale_rows(r, __builtin_ldexpf(1.0f, max(scaled - ex, -126)));
            scaled = ex;
          }
#pragma unroll
          for (int s = 0; s < KT / 32; ++s) {
            const uint32_t kb = base + buf * kStage + s * 16384;
            key_step<true>(r, q, kb + at.k, kb + KT * 512 + at.v, factor, 0, masked, side + 128 * s, side + 4 * KT + 128 * s, lane);
          }
        }
        if (u + 1 < end) unpack(buf ^ 1);
      }
      // the sums over centroids, rotated
      float x[128];
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) x[16 * t + i] = r.o[t][i];
      fwht_halves(x);
      const float f = __builtin_ldexpf(1.0f, scaled - 8);
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i) r.o[t][i] = x[16 * t + i] * f;
      barrier();  // every wave is done with LDS
    } else {
      clear(r);
    }

    if (u1 > w.page_blocks) {
      const int64_t from = max(u0, w.page_blocks) - w.page_blocks, to = u1 - w.page_blocks;
      const int64_t first_key = near + token_of(min(w0, rows - 1), a.group);               // the last that the wave's first row sees
      const int64_t last_key = idle ? -1 : near + token_of(min(w0 + 31, rows - 1), a.group);  // and its last
      const int64_t end_key = near + w.last_token(a, g.tile);                      // and the tile's last
      const Tokens tokens(a, e, g.b, g.head);
      const auto stage = [&](int buf, int64_t t0) {
#pragma unroll
        for (int i = 0; i < KT / 16; ++i) {
          const int pair = 16 * i + 2 * wave;
          const int64_t k = t0 + pair + h;
          const uint32_t c = (col ^ swizzle(2 * wave + h)) * 8;
          stage16(tokens.at(0, k, end_key) + c, base + buf * kStage + pair * 512);
          stage16(tokens.at(1, k, end_key) + c, base + buf * kStage + KT * 512 + pair * 512);
        }
      };
      u32x4 q[16];
      const uint16_t* qp = q_ptr();
#pragma unroll
      for (int s = 0; s < 16; ++s) q[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
      stage(0, from * KT);
#pragma unroll
      for (int s = 0; s < 16; ++s) {
        if (a.scale < 0) q[s] ^= 0x80008000u;
        asm volatile("" : "+v"(q[s]));
      }
      for (int64_t u = from; u < to; ++u) {
        const int buf = (u - from) & 1;
        wait_staged();
        barrier();
        if (u + 1 < to) stage(buf ^ 1, (u + 1) * KT);
#pragma unroll
        for (int s = 0; s < KT / 32; ++s) {
          const int64_t k0 = u * KT + 32 * s;
          if (k0 > last_key) continue;
          const uint32_t kb = base + buf * kStage + s * 16384;
          key_step<false>(r, q, kb + at.k, kb + KT * 512 + at.v, fabsf(a.scale) * kLog2e,
                          static_cast<int>(min(near + tok - k0, int64_t{64})), k0 + 31 > first_key, 0, 0, lane);
        }
      }
      add_nonfinite(r, max((first_key + 1) / 32 * 32, from * KT), min(last_key, to * KT - 1), near + tok, h,
                    [&](int64_t key) { return tokens.at(1, key, end_key); });
      barrier();
    }

    r.l += half_swap(r.l);
    if (w0 + col < rows) {
      if (g.from == 0 && g.to == g.cost) {
        const float inv = 1.0f / r.l;
        uint16_t* op = a.out + ((e.begin + static_cast<int64_t>(tok)) * a.q_heads + q_head()) * kDim;
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 v = {pack_bf16x2(r.o[t][4 * i] * inv, r.o[t][4 * i + 1] * inv),
                             pack_bf16x2(r.o[t][4 * i + 2] * inv, r.o[t][4 * i + 3] * inv)};
            *reinterpret_cast<uint2*>(op + 32 * t + 8 * i + 4 * h) = v;
          }
      } else {
        const int slot = g.from > 0 ? 0 : 1, at_row = 32 * wave + col;
        float* op = partial_row<M>(a, 2 * worker + slot, at_row);
#pragma unroll
        for (int t = 0; t < 8; ++t)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<f32x4*>(op + 32 * t + 8 * i + 4 * h) = f32x4{r.o[t][4 * i], r.o[t][4 * i + 1], r.o[t][4 * i + 2], r.o[t][4 * i + 3]};
        if (h == 0) *partial_stat<M>(a, 2 * worker + slot, at_row) = float2{r.m, r.l};
      }
    }
  });
}

// Joins the tiles that several workgroups shared, four rows to a wave.
constexpr int kChunkJoinRows = 16;  // of a workgroup
__global__ void __launch_bounds__(256) hlwq_chunk_join_kernel(const AttnArgs a) {
  constexpr int M = kChunkRows, KT = kChunkBlock;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const auto cost = [&](const Extent& e) { return Work<M, KT>(a, e).head_cost() * a.kv_heads; };
  const auto tiles = [&](const Extent& e) { return Work<M, KT>(a, e).tiles * a.kv_heads; };
  Finder<decltype(tiles), decltype(cost)> finder(a, tiles, cost);
  const int32_t x = blockIdx.x / (M / kChunkJoinRows);
  if (x >= finder.total) return;
  const Found f = finder.find(x);
  const Work<M, KT> w(a, f.e);
  const int32_t head = quotient(f.rest, w.tiles), tile = f.rest - head * w.tiles;
  const int32_t row0 = (blockIdx.x % (M / kChunkJoinRows)) * kChunkJoinRows + 4 * wave, rows = w.rows(a) - tile * M;
  if (row0 >= rows) return;
  const int32_t x0 = f.before + head * w.head_cost() + w.cost_before(tile), x1 = x0 + w.cost(tile);
  const Share share(Finder<decltype(cost), Nothing>(a, cost, Nothing{}).total, a.workers, kChunkLeast);
  const int32_t w0 = share.worker_at(x0), w1 = share.worker_at(x1 - 1);
  if (w0 == w1) return;  // one workgroup did it all
  float m[4], l[4];
  f32x4 o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -FLT_MAX;
    l[i] = 0;
    o[i] = f32x4{0, 0, 0, 0};
  }
  for (int32_t k = w0; k <= w1; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (row0 + i >= rows) continue;
      const int32_t slot = 2 * k + (k == w0 ? 1 : 0);
      const float2 s = *partial_stat<M>(a, slot, row0 + i);
      const f32x4 v = *reinterpret_cast<const f32x4*>(partial_row<M>(a, slot, row0 + i) + 4 * lane);
      const float mn = fmaxf(m[i], s.x);
      const float f0 = fast_exp2(m[i] - mn), f1 = fast_exp2(s.x - mn);
      m[i] = mn;
      l[i] = l[i] * f0 + s.y * f1;
      o[i] = o[i] * f0 + v * f1;
    }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row0 + i < rows) write_row(a, w.e.begin, head, tile * M + row0 + i, o[i], l[i], lane);
}

}  // namespace hlwq_kv
