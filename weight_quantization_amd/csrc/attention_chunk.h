// attention_chunk.h — attention of many new tokens over a paged cache: the tile
// kernel of attention_tile.h with a first phase over pages of codes.
//
// Pages are worked on in the rotated domain (attention_split.h): the codes of 64
// tokens go to LDS as they are, the 512 work-items unpack them there to fp16
// centroids while the 64 before are multiplied, so that 256 query rows share
// one unpacking; then the sums are rotated in registers and the window's and
// the step's own tokens follow in bf16.
//
// Measured: 1024 tokens over 16000 (24 query heads on 4, 3 bits, 415 GFLOP)
// take 535 to 580 us (the card slows its clock within ten calls) and the join
// 21.  About 90 us of that are there however few the pages: two rotations of
// 256 x 256 sums a stretch, 92 MB of partial sums, and 80 KB of instructions
// that run once.  A block of 64 tokens takes about 4.1 us, of which the products
// are 1.8; matrix cores 36% busy, VALU issue 42%.
#pragma once

#include "attention_split.h"
#include "attention_tile.h"

namespace hlwq_kv {

constexpr int kChunkRows = 256;
constexpr int kChunkBlock = 64;   // tokens to a block
// Cost that is worth a workgroup of its own.  One block against four (24 query
// heads on 4, us): 8 requests of 40 over 500 tokens 60 and 75, of 20 over 4000
// 68 and 68, one of 100 over 200 42 and 64, one of 80 over 4000 75 and 73.
constexpr int kChunkLeast = kBlockCost;

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

// Where a lane's row of the tile stands: the wave's 32 rows begin at w0 of the
// request's `rows`.  Worked out anew for each phase from a lane number that the
// compiler cannot follow, as what it would keep between them costs registers
// that the loops need.
struct ChunkRow {
  int lane, col, h;
  int32_t tok, q_head;
  __device__ __forceinline__ ChunkRow(const AttnArgs& a, int32_t head, int32_t w0, int32_t rows) {
    lane = threadIdx.x & 63;
    asm volatile("" : "+v"(lane));
    col = lane & 31;
    h = lane >> 5;
    const int32_t row = min(w0 + col, rows - 1);
    tok = token_of(row, a.group);
    q_head = head * a.group + (row - tok * a.group);
  }
  __device__ __forceinline__ const uint16_t* q(const AttnArgs& a, int32_t begin) const {
    return a.q + (begin + static_cast<int64_t>(tok)) * a.q_stride + q_head * kDim + 8 * h;
  }
};

// Zeros that no other code takes a zero from: the compiler would keep sixteen
// of them for the upper half of a 64-bit address.
__device__ __forceinline__ void clear_apart(Rows& r) {
  clear(r);
#pragma unroll
  for (int t = 0; t < 8; ++t) asm volatile("" : "+v"(r.o[t]));
}

// LDS of the chunk kernel: two stages of 64 tokens' K and V (fp16 or bf16), two
// of their packed codes, and of their norms as they are in memory, four of the
// ids of their pages, and for each stage the K norms, the V norms, whether some
// token is missing and the V norms' exponent.
template <int BITS>
struct ChunkLds {
  static constexpr uint32_t kStage = kChunkBlock * 1024, kCodes = kChunkBlock * 32 * BITS, kLine = kChunkBlock * 4;
  static constexpr uint32_t kSide = 2 * kLine + 16;
  static constexpr uint32_t raw = 2 * kStage, norms = raw + 4 * kCodes, ids = norms + 4 * kLine, side = ids + 4 * kLine,
                            flag = side + 2 * kSide, bytes = flag + 16;
};

// Vector of token t, which lies in page `id` of its request.
__device__ __forceinline__ int64_t place(const AttnArgs& a, int32_t head, int32_t id, int32_t t) {
  int32_t within = t & ((1 << a.page_shift) - 1);
  asm volatile("" : "+v"(within));  // its upper half is computed: a register with a zero for it would be kept, and spilled
  return ((static_cast<int64_t>(id) * a.kv_heads + head) << a.page_shift) + within;
}

// Pages [u0, u1) of 64 tokens.  At block u the page ids of u + 3 and the codes
// and norms of u + 2 are on their way to LDS, those of u + 1 are unpacked, and
// u is multiplied; the lower waves unpack before they multiply, the upper ones
// (on the same SIMDs) after, so that one's VALU work meets the other's products.
// Whatever a lane would keep from block to block is in LDS: the sums, the query
// and the step's operands fill the registers, and one reload from scratch
// memory waits for every load that is under way.
template <int BITS>
__device__ __forceinline__ void chunk_pages(Rows& r, const AttnArgs& a, const Extent& e, int32_t b, int32_t head, int32_t w0, int32_t u0,
                                            int32_t u1, uint32_t base, int wave) {
  using L = ChunkLds<BITS>;
  constexpr int KT = kChunkBlock, kWaves = 2 * BITS;  // waves that fetch codes: 16 bytes a lane
  const int32_t rows = e.n * a.group;
  const int32_t paged = static_cast<int32_t>(e.paged);  // at most 2^20 pages of 2^8 tokens
  const int32_t* const table = a.table + static_cast<int64_t>(b) * a.width;
  // lane = token of the block
  const auto ids = [&](int32_t u) {
    if (u < u1 && wave == 6)
      stage4(table + (min(u * KT + lane_now(), paged - 1) >> a.page_shift), base + L::ids + (u & 3) * L::kLine);
  };
  const auto id_of = [&](int32_t u, int token) {
    const int32_t id = lds_at<int32_t>(base + L::ids + (u & 3) * L::kLine + 4 * token);
    return u * KT + token < paged && id < a.n_pages ? id : -1;
  };
  // Waves 0 .. 2 BITS - 1 fetch 1 KB of K codes and of V codes each, lane by
  // lane 16 bytes of a token; waves 6 and 7 the norms of token `lane`, K and V.
  // Of a page that is not there the first one's, which no row comes to see.
  const auto fetch = [&](int32_t u) {
    if (u >= u1) return;
    const int lane = lane_now();
    if (wave < kWaves) {
      const int piece = wave * 64 + lane, token = piece / (2 * BITS), part = piece - token * (2 * BITS);
      const int64_t vec = place(a, head, max(id_of(u, token), 0), u * KT + token) * (32 * BITS) + 16 * part;
      const uint32_t to = base + L::raw + (u & 1) * 2 * L::kCodes + wave * 1024;
      stage16(a.k_packed + vec, to);
      stage16(a.v_packed + vec, to + L::kCodes);
    }
    if (wave >= 6)
      stage2((wave == 6 ? a.k_norms : a.v_norms) + place(a, head, max(id_of(u, lane), 0), u * KT + lane),
             base + L::norms + ((u & 1) * 2 + wave - 6) * L::kLine);
  };
  const auto norms = [&](int32_t u, int exponent) {
    if (u >= u1 || wave < 6) return;
    const int lane = lane_now();
    const uint32_t side = base + L::side + (u & 1) * L::kSide;
    const bool there = id_of(u, lane) >= 0;
    const float n = f16_value(static_cast<uint16_t>(lds_at<uint32_t>(base + L::norms + ((u & 1) * 2 + wave - 6) * L::kLine + 4 * lane)));
    if (wave == 6) {
      lds_put<float>(side + 4 * lane, there ? n : -1.0f);
      const bool all = __all(there);
      if (lane == 0) lds_put<uint32_t>(side + 2 * L::kLine, !all);
    } else {
      // as in code_step: norms over a power of two that none met so far exceeds
      const float top = wave_max(there ? n : 0.0f);
      if (top > __builtin_ldexpf(1.0f, exponent)) exponent = __builtin_amdgcn_frexp_expf(top);
      lds_put<float>(side + L::kLine + 4 * lane, there ? __builtin_ldexpf(kTopWeight * n, -exponent) : 0.0f);
      if (lane == 0) lds_put<int32_t>(side + 2 * L::kLine + 4, exponent);
    }
  };
  const auto exponent_of = [&](int32_t u) {
    return __builtin_amdgcn_readfirstlane(lds_at<int32_t>(base + L::side + (u & 1) * L::kSide + 2 * L::kLine + 4));
  };
  // lane = token of the block; which 32 of its 256 codes is turned by lane / 8,
  // so that the reads (24 or 16 words apart) fall on all banks, and with them
  // the writes
  const auto unpack = [&](int32_t u) {
    if (u >= u1) return;
    const int lane = lane_now(), run = (wave + (lane >> 3)) & 7;
    const uint32_t raw = base + L::raw + (u & 1) * 2 * L::kCodes + lane * 32 * BITS + run * 4 * BITS;
    const uint32_t to = base + (u & 1) * L::kStage + lane * 512 + ((4 * run) ^ swizzle(lane)) * 16;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      Run<BITS> codes;
#pragma unroll
      for (int i = 0; i < BITS; ++i) codes.w[i] = lds_at<uint32_t>(raw + side * L::kCodes + 4 * i);
#pragma unroll
      for (int x = 0; x < 4; ++x) lds_put<u32x4>((to ^ (x * 16)) + side * KT * 512, run_chunk<BITS>(codes, x));
    }
  };
  ids(u0);
  ids(u0 + 1);
  ids(u0 + 2);
  wait_staged();
  barrier();
  fetch(u0);
  fetch(u0 + 1);
  // q rotated, over a power of two that brings the row's largest value to
  // [1, 2), as fp16
  u32x4 q[16];
  float factor;
  {
    float x[128];
    const uint16_t* qp = ChunkRow(a, head, w0, rows).q(a, e.begin);
#pragma unroll
    for (int s = 0; s < 16; ++s) {
      const u32x4 v = *reinterpret_cast<const u32x4*>(qp + 16 * s);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[8 * s + 2 * j] = bf16_lo(v[j]) * kQueryScale;
        x[8 * s + 2 * j + 1] = bf16_hi(v[j]) * kQueryScale;
      }
    }
    fwht_halves(x);
    float mx = 0;
#pragma unroll
    for (int i = 0; i < 128; ++i) mx = fmaxf(mx, fabsf(x[i]));
    mx = fmaxf(mx, half_swap(mx));
    const int ex = row_exponent(mx);
    const float f = __builtin_ldexpf(a.scale < 0 ? -1.0f : 1.0f, -ex);
#pragma unroll
    for (int s = 0; s < 16; ++s)
#pragma unroll
      for (int j = 0; j < 4; ++j) q[s][j] = pack_f16x2(x[8 * s + 2 * j] * f, x[8 * s + 2 * j + 1] * f);
    factor = fmaxf(__builtin_ldexpf(a.factor, ex), __FLT_DENORM_MIN__);
  }
  clear_apart(r);
  wait_staged();
  barrier();
  norms(u0, -64);
  unpack(u0);
  int scaled = -64;
  const bool first_half = wave < 4, idle = w0 >= rows;
  TileLane at = tile_lane(lane_now());
  asm volatile("" : "+v"(at.k), "+v"(at.v));
  for (int32_t u = u0; u < u1; ++u) {
    wait_staged();
    wait_lds();
    barrier();
    const int ex = exponent_of(u);
    norms(u + 1, ex);
    fetch(u + 2);
    ids(u + 3);
#pragma clang loop unroll(disable)
    for (int turn = 0; turn < 2; ++turn) {
      if (first_half == (turn == 0)) {
        unpack(u + 1);
        continue;
      }
      if (idle) continue;
      const uint32_t side = base + L::side + (u & 1) * L::kSide;
      const bool masked = __builtin_amdgcn_readfirstlane(lds_at<uint32_t>(side + 2 * L::kLine)) != 0;
      if (ex != scaled) {
        scale_rows(r, __builtin_ldexpf(1.0f, max(scaled - ex, -126)));
        scaled = ex;
      }
#pragma unroll
      for (int s = 0; s < KT / 32; ++s) {
        uint32_t kb = base + (u & 1) * L::kStage + s * 16384;
        asm volatile("" : "+s"(kb));  // 16 addresses of each step are not kept
        key_step<true>(r, q, kb + at.k, kb + KT * 512 + at.v, factor, 0, masked, side + 128 * s, side + L::kLine + 128 * s);
      }
    }
  }
  // the sums over centroids, rotated
  float x[128];
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) x[16 * t + i] = r.o[t][i];
  fwht_halves(x);
  const float f = __builtin_ldexpf(1.0f / kTopWeight, scaled - 8);
#pragma unroll
  for (int t = 0; t < 8; ++t)
#pragma unroll
    for (int i = 0; i < 16; ++i) r.o[t][i] = x[16 * t + i] * f;
}

// The window's and the step's own tokens, blocks [from, to) of 64 of them.  (Blocks
// that are staged or masked reload a register from scratch memory each.)
template <int BITS>
__device__ __forceinline__ void chunk_tokens(Rows& r, const AttnArgs& a, const Extent& e, int32_t b, int32_t head, int32_t w0,
                                             int64_t end_key, int32_t from, int32_t to, uint32_t base, int wave) {
  using L = ChunkLds<BITS>;
  constexpr int KT = kChunkBlock;
  const int32_t rows = e.n * a.group;
  const Tokens tokens(a, e, b, head);
  // the keys that all rows see; the last that the wave's first row sees, and its last row
  const int64_t seen = tokens.near + token_of(w0 - 32 * wave, a.group) + 1;
  const int64_t first_key = tokens.near + token_of(min(w0, rows - 1), a.group);
  const int64_t last_key = w0 >= rows ? -1 : tokens.near + token_of(min(w0 + 31, rows - 1), a.group);
  // Tokens t0 .. t0 + 63, from window and step; the last one again for what is
  // past it, which is masked.
  const auto stage = [&](int buf, int64_t t0) {
    const int lane = lane_now(), pair = 2 * wave + (lane >> 5);
    const int32_t c = ((lane & 31) ^ swizzle(pair)) * 16;
    const int window = static_cast<int>(max(min(tokens.near - t0, int64_t{KT}), int64_t{0}));
    const int last = static_cast<int>(min(end_key - t0, int64_t{KT - 1}));
    // where token t0 would be in the ring, in the ring after its end, among the step's
    const int64_t slot = tokens.ring0 + t0;
    const int until = static_cast<int>(min(tokens.ring - slot, int64_t{KT}));  // may be below 0: all after the end
    const char* from[2][3];
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      from[side][0] = reinterpret_cast<const char*>(tokens.window[side] + slot * kDim);
      from[side][1] = reinterpret_cast<const char*>(tokens.window[side] + (slot - tokens.ring) * kDim);
      from[side][2] = reinterpret_cast<const char*>(tokens.rows[side] + (t0 - tokens.near) * tokens.stride[side]);
    }
#pragma unroll
    for (int i = 0; i < KT / 16; ++i) {
      const int j = min(16 * i + pair, last);
      const uint32_t to = base + buf * L::kStage + (16 * i + 2 * wave) * 512;
#pragma unroll
      for (int side = 0; side < 2; ++side) {
        // below 2^29 + 2^9: strides are at most 2^22
        const int32_t off = j * (j < window ? kDim * 2 : static_cast<int32_t>(2 * tokens.stride[side])) + c;
        stage16((j < window ? j < until ? from[side][0] : from[side][1] : from[side][2]) + off, to + side * KT * 512);
      }
    }
  };
  if (threadIdx.x == 0) lds_put<uint32_t>(base + L::flag, 0);
  wait_lds();
  stage(0, static_cast<int64_t>(from) * KT);
  u32x4 q[16];
  const uint16_t* qp = ChunkRow(a, head, w0, rows).q(a, e.begin);
#pragma unroll
  for (int s = 0; s < 16; ++s) q[s] = *reinterpret_cast<const u32x4*>(qp + 16 * s);
#pragma unroll
  for (int s = 0; s < 16; ++s) {
    if (a.scale < 0) q[s] ^= 0x80008000u;
    asm volatile("" : "+v"(q[s]));
  }
  TileLane at = tile_lane(lane_now());
  asm volatile("" : "+v"(at.k), "+v"(at.v));
  int32_t tok = ChunkRow(a, head, w0, rows).tok;
  asm volatile("" : "+v"(tok));
  for (int32_t u = from; u < to; ++u) {
    const int buf = (u - from) & 1;
    wait_staged();
    barrier();
    if (u + 1 < to) stage(buf ^ 1, static_cast<int64_t>(u + 1) * KT);
    if (static_cast<int64_t>(u + 1) * KT > seen) leave_out_nonfinite<512, KT>(base + buf * L::kStage + KT * 512, base + L::flag);
#pragma clang loop unroll(disable)
    for (int s = 0; s < KT / 32; ++s) {
      const int64_t k0 = static_cast<int64_t>(u) * KT + 32 * s;
      if (k0 > last_key) continue;
      const uint32_t kb = base + buf * L::kStage + s * 16384;
      key_step<false>(r, q, kb + at.k, kb + KT * 512 + at.v, a.factor,
                      static_cast<int>(min(tokens.near - k0 + tok, int64_t{64})), k0 + 31 > first_key, 0, 0);
    }
  }
  add_nonfinite(r, base + L::flag, max(seen / KT * KT, static_cast<int64_t>(from) * KT), min(last_key, static_cast<int64_t>(to) * KT - 1),
                tokens.near + tok, lane_now() >> 5, [&](int64_t key) { return tokens.at(1, key, end_key); });
}

template <int BITS>
__global__ void __launch_bounds__(512) __attribute__((amdgpu_waves_per_eu(2, 2))) hlwq_chunk_attention_kernel(const AttnArgs a) {
  constexpr int M = kChunkRows, KT = kChunkBlock;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[ChunkLds<BITS>::bytes];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t base = static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t*)lds));

  const auto cost = [&](const Extent& e) { return Work<M, KT>(a, e).head_cost() * a.kv_heads; };
  Finder<decltype(cost), Nothing> finder(a, cost, Nothing{});
  const Share share(finder.total, a.workers, kChunkLeast);
  if (finder.total == 0) return;
  // Workgroups of one XCD (every eighth) take neighbouring stretches, which
  // share a KV head's keys in its L2.
  const int32_t of_xcd = (share.workers + 7) / 8;
  const int32_t worker = (blockIdx.x % 8) * of_xcd + blockIdx.x / 8;
  if (static_cast<int32_t>(blockIdx.x / 8) >= of_xcd || worker >= share.workers) return;
  const Found first = finder.find(share.bound(worker));

  for_segments<M, KT>(a, share, first, worker, [&](const Work<M, KT>& w, const Segment& g) {
    const int32_t rows = w.rows(a), w0 = g.tile * M + 32 * wave;
    const int32_t blocks = w.blocks(a, g.tile);
    const int32_t u0 = w.block_at(g.from, blocks, g.cost), u1 = w.block_at(g.to, blocks, g.cost);
    Rows r;
    r.m = -FLT_MAX;
    r.l = 0;
    if (u0 < w.page_blocks && u0 < u1) {
      chunk_pages<BITS>(r, a, w.e, g.b, g.head, w0, u0, min(u1, w.page_blocks), base, wave);
      barrier();  // every wave is done with LDS
    } else {
      clear_apart(r);
    }
    if (u1 > w.page_blocks) {
      chunk_tokens<BITS>(r, a, w.e, g.b, g.head, w0, w.e.held - w.e.enc + w.last_token(a, g.tile),
                         max(u0, w.page_blocks) - w.page_blocks, u1 - w.page_blocks, base, wave);
      barrier();
    }
    r.l += half_swap(r.l);
    const ChunkRow row(a, g.head, w0, rows);
    if (w0 + row.col >= rows) return;
    if (g.from == 0 && g.to == g.cost) {
      const float inv = 1.0f / r.l;
      uint16_t* op = a.out + ((w.e.begin + static_cast<int64_t>(row.tok)) * a.q_heads + row.q_head) * kDim + 4 * row.h;
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint2 v = {pack_bf16x2(r.o[t][4 * i] * inv, r.o[t][4 * i + 1] * inv),
                           pack_bf16x2(r.o[t][4 * i + 2] * inv, r.o[t][4 * i + 3] * inv)};
          *reinterpret_cast<uint2*>(op + 32 * t + 8 * i) = v;
        }
    } else {
      const int slot = 2 * worker + (g.from > 0 ? 0 : 1), at_row = 32 * wave + row.col;
      float* op = partial_row<M>(a, slot, at_row) + 4 * row.h;
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<f32x4*>(op + 32 * t + 8 * i) = f32x4{r.o[t][4 * i], r.o[t][4 * i + 1], r.o[t][4 * i + 2], r.o[t][4 * i + 3]};
      if (row.h == 0) *partial_stat<M>(a, slot, at_row) = float2{r.m, r.l};
    }
  });
}

// Joins the tiles that several workgroups shared, four rows to a wave.
constexpr int kChunkJoinRows = 16;  // of a workgroup
constexpr int64_t kChunkJoinWide = 1 << 20;  // workgroups along the grid's first dimension; the rest along its second
__global__ void __launch_bounds__(256) hlwq_chunk_join_kernel(const AttnArgs a) {
  constexpr int M = kChunkRows, KT = kChunkBlock;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const auto cost = [&](const Extent& e) { return Work<M, KT>(a, e).head_cost() * a.kv_heads; };
  const auto tiles = [&](const Extent& e) { return Work<M, KT>(a, e).tiles * a.kv_heads; };
  Finder<decltype(tiles), decltype(cost)> finder(a, tiles, cost);
  const uint32_t at = blockIdx.y * static_cast<uint32_t>(kChunkJoinWide) + blockIdx.x;
  const int32_t x = at / (M / kChunkJoinRows);
  if (x >= finder.total) return;
  const Found f = finder.find(x);
  const Work<M, KT> w(a, f.e);
  const int32_t head = quotient(f.rest, w.tiles), tile = f.rest - head * w.tiles;
  const int32_t row0 = (at % (M / kChunkJoinRows)) * kChunkJoinRows + 4 * wave, rows = w.rows(a) - tile * M;
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
  // four parts of four rows in flight: a part at a time, 480 rows over 16000
  // tokens, four KV heads' two tiles of 32 parts each, took 133 us instead of 112
  for (int32_t k0 = w0; k0 <= w1; k0 += 4) {
    float2 s[4][4];
    f32x4 v[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int32_t k = min(k0 + j, w1), slot = 2 * k + (k == w0 ? 1 : 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = min(row0 + i, rows - 1);
        s[j][i] = *partial_stat<M>(a, slot, row);
        v[j][i] = *reinterpret_cast<const f32x4*>(partial_row<M>(a, slot, row) + 4 * lane);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (k0 + j <= w1)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float mn = fmaxf(m[i], s[j][i].x);
          const float f0 = fast_exp2(m[i] - mn), f1 = fast_exp2(s[j][i].x - mn);
          m[i] = mn;
          l[i] = l[i] * f0 + s[j][i].y * f1;
          o[i] = o[i] * f0 + v[j][i] * f1;
        }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row0 + i < rows) write_row(a, w.e.begin, head, tile * M + row0 + i, o[i], l[i], lane);
}

}  // namespace hlwq_kv
