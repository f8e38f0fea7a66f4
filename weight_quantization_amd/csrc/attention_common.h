// attention_common.h — what the attention kernels share: arguments, the
// requests' extents, the matrix-core fragments and the unpacking of codes.
//
// Every kernel computes S^T = K Q^T and O^T = V^T P^T, so that a query row is
// a column of both results: its softmax statistics are one register of the
// lanes that hold the column, the probabilities come out of the first product
// in the layout that the second takes them in (up to an order of the keys,
// which V's operand follows), and nothing is exchanged across lanes but the
// row maximum.
#pragma once

#include "kv_common.h"

namespace hlwq_kv {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) u32x4 lds_u32x4;
typedef __attribute__((address_space(3))) u32x2 lds_u32x2;
typedef __attribute__((address_space(3))) f32x4 lds_f32x4;
typedef __attribute__((address_space(3))) float lds_f32;
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
typedef __attribute__((address_space(3))) uint32_t lds_u32;

constexpr float kLog2e = 1.44269504088896340736f;
// A row's running maximum is raised, and its sums rescaled, only once a score
// passes it by this much (in powers of two): probabilities then reach 2^8,
// far inside the range of bf16, fp16 and fp32, and the rescale of 256 sums is
// paid a few times per row instead of once per tile.
constexpr float kLazy = 8.0f;

struct AttnArgs {
  const uint16_t* q;
  const uint16_t* k_new;
  const uint16_t* v_new;
  int64_t q_stride, k_stride, v_stride;
  const uint8_t* k_packed;
  const uint8_t* v_packed;
  const uint16_t* k_norms;
  const uint16_t* v_norms;
  const uint16_t* k_window;
  const uint16_t* v_window;
  const int32_t* cu;
  const int32_t* lens;  // null: nothing is cached
  const int32_t* table;
  uint16_t* out;
  float* partial;  // workspace: partial sums, then their statistics
  int64_t n_res, ring;
  int32_t requests, rows, q_heads, kv_heads, group, n_pages, page_shift, width;
  int32_t workers;  // workgroups that share the work
  int32_t least, most;  // requests with rows * group in [least, most] are this kernel's
  float scale;
};

// One request's part of a step.
struct Extent {
  int32_t begin, n;   // rows
  int64_t held, enc;  // tokens before the step, those of them encoded
  int64_t paged;      // encoded tokens that have a table entry
};
__device__ __forceinline__ Extent extent_of(const AttnArgs& a, int32_t b) {
  Extent e;
  const RowRange r = row_range(a.cu, b, a.rows);
  e.begin = r.begin;
  e.n = r.end - r.begin;
  e.held = a.lens ? max(static_cast<int64_t>(a.lens[b]) - e.n, int64_t{0}) : 0;
  e.enc = a.lens ? max(e.held - a.n_res, int64_t{0}) : 0;
  e.paged = a.n_pages > 0 ? min(e.enc, static_cast<int64_t>(a.width) << a.page_shift) : 0;
  return e;
}

// The token that row r of a request belongs to.
__device__ __forceinline__ int32_t token_of(int32_t r, int32_t group) {
  return static_cast<int32_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(group));
}

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

// Value of lane l ^ 32.
__device__ __forceinline__ float half_swap(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// Two floats rounded to a pair of fp16, to nearest.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const f16x2 v = {static_cast<_Float16>(lo), static_cast<_Float16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

// The pair of bf16 with infinities and NaN replaced by zero; `any` gets a bit
// set if there was one.  (Adding one to an exponent of all ones carries into
// the sign's place.)
__device__ __forceinline__ uint32_t finite_pair(uint32_t w, uint32_t& any) {
  const uint32_t m = ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
  any |= m;
  return w & ~(m | (m - (m >> 15)));
}

// ---------------------------------------------------------------------------
// Codes to centroids.  The centroids enter the products as fp16; their bytes
// are looked up by v_perm_b32, which picks each byte of its result from eight
// bytes in two registers: one permute gives the high bytes of four centroids,
// one the low bytes, and two more interleave them to four fp16.
// ---------------------------------------------------------------------------

constexpr uint16_t f16_of(float f) { return __builtin_bit_cast(uint16_t, static_cast<_Float16>(f)); }
template <int BITS>
struct Book {
  static constexpr float c3[8] = HLWQ_CENTROIDS_3;
  static constexpr float c2[4] = HLWQ_CENTROIDS_2;
  static constexpr uint32_t word(int first, int shift) {
    uint32_t w = 0;
    for (int i = 0; i < 4; ++i) {
      const uint16_t h = BITS == 3 ? f16_of(c3[(first + i) & 7]) : f16_of(c2[i]);
      w |= static_cast<uint32_t>((h >> shift) & 0xff) << (8 * i);
    }
    return w;
  }
  static constexpr uint32_t hi0 = word(0, 8), hi1 = word(4, 8), lo0 = word(0, 0), lo1 = word(4, 0);
};

// Four codes, one a byte, to four fp16 centroids.
template <int BITS>
__device__ __forceinline__ u32x2 look_up(uint32_t c) {
  const uint32_t hi = __builtin_amdgcn_perm(Book<BITS>::hi1, Book<BITS>::hi0, c);
  const uint32_t lo = __builtin_amdgcn_perm(Book<BITS>::lo1, Book<BITS>::lo0, c);
  return u32x2{__builtin_amdgcn_perm(hi, lo, 0x05010400u), __builtin_amdgcn_perm(hi, lo, 0x07030602u)};
}

// ---------------------------------------------------------------------------
// Finding work.  The requests' lengths are on the device, so every wave sums
// what the requests ask for and finds its workgroup's share of it, without
// LDS or a barrier: lane i takes requests i, i + 64, ..
// ---------------------------------------------------------------------------

// a / b for a, b >= 0, in 32 bits where they fit (64 take ten times as long).
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

__device__ __forceinline__ int64_t uniform64(int64_t v) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(static_cast<uint64_t>(v) >> 32));
  return static_cast<int64_t>((static_cast<uint64_t>(hi) << 32) | lo);
}

// The sum of a quantity over the requests.
template <class F>
__device__ __forceinline__ int64_t sum_over(int32_t requests, F of) {
  int64_t v = 0;
  for (int32_t b = threadIdx.x & 63; b < requests; b += 64) v += of(b);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return uniform64(v);
}

// The request that holds unit x of the quantity (0 <= x < its sum), x's place
// in it, and the sum of `also` over the requests before it.
struct Found {
  int32_t b;
  int64_t rest, also;
};
template <class F, class G>
__device__ __forceinline__ Found find(int32_t requests, int64_t x, F of, G also) {
  const int lane = threadIdx.x & 63;
  Found f{0, 0, 0};
  for (int32_t b0 = 0; b0 < requests; b0 += 64) {
    const bool in = b0 + lane < requests;
    const int64_t own = in ? of(b0 + lane) : 0, other = in ? also(b0 + lane) : 0;
    int64_t v = own, w = other;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int64_t p = __shfl_up(v, d, 64), q = __shfl_up(w, d, 64);
      if (lane >= d) {
        v += p;
        w += q;
      }
    }
    const uint64_t past = __ballot(x < v);
    if (past) {
      const int at = __builtin_ctzll(past);
      f.b = b0 + at;
      f.rest = uniform64(x - __shfl(v - own, at, 64));
      f.also += uniform64(__shfl(w - other, at, 64));
      return f;
    }
    x -= uniform64(__shfl(v, 63, 64));
    f.also += uniform64(__shfl(w, 63, 64));
  }
  f.b = -1;
  return f;
}

// How the paged kernels share their work out.  A tile is M consecutive rows of
// one request and KV head; it costs its key blocks of KT tokens: those of the
// pages, then those of the window and of the step's own tokens up to the
// tile's last row.  The tiles lie one after the other, by request, KV head and
// row, and every workgroup takes an equal stretch of their cost, so that
// requests of any lengths load the workgroups alike; a tile that several
// workgroups share is joined from their partial sums afterwards.
template <int M, int KT>
struct Work {
  Extent e;
  int64_t tiles, base, step, page_blocks;
  __device__ __forceinline__ Work(const AttnArgs& a, int32_t b) {
    e = extent_of(a, b);
    const int32_t rows = e.n * a.group;
    tiles = rows >= a.least && rows <= a.most ? ceil_div(rows, M) : 0;
    page_blocks = ceil_div(e.paged, KT);
    base = page_blocks + ceil_div(e.held - e.enc + 1, KT);
    // at least the blocks by which a tile's tokens pass those of the one before
    step = M <= KT ? 1 : (static_cast<uint32_t>(M - 1) / static_cast<uint32_t>(a.group) + KT) / KT;
  }
  // of one KV head
  __device__ __forceinline__ int64_t cost_before(int64_t j) const { return j * base + step * (j * (j - 1) / 2); }
  __device__ __forceinline__ int64_t cost(int64_t j) const { return base + step * j; }
  __device__ __forceinline__ int64_t head_cost() const { return cost_before(tiles); }
  // the tile that holds place x of a KV head's cost
  __device__ __forceinline__ int64_t tile_at(int64_t x) const {
    if (tiles == 1) return 0;
    const double b = 2.0 * base - step, s = step;
    int64_t j = static_cast<int64_t>((sqrt(b * b + 8.0 * s * x) - b) / (2.0 * s));
    j = max(min(j, tiles - 1), int64_t{0});
    while (j > 0 && cost_before(j) > x) --j;
    while (j + 1 < tiles && cost_before(j + 1) <= x) ++j;
    return j;
  }
  __device__ __forceinline__ int32_t rows(const AttnArgs& a) const { return e.n * a.group; }
  // tokens (of the step) of the tile's first row and last row
  __device__ __forceinline__ int32_t first_token(const AttnArgs& a, int64_t j) const {
    return static_cast<uint32_t>(j * M) / static_cast<uint32_t>(a.group);
  }
  __device__ __forceinline__ int32_t last_token(const AttnArgs& a, int64_t j) const {
    return static_cast<uint32_t>(min((j + 1) * M, static_cast<int64_t>(rows(a))) - 1) / static_cast<uint32_t>(a.group);
  }
  // key blocks of tile j: the pages', then the others
  __device__ __forceinline__ int64_t blocks(const AttnArgs& a, int64_t j) const {
    return page_blocks + ceil_div(e.held - e.enc + last_token(a, j) + 1, KT);
  }
  // the block at place x of a tile's cost: its blocks spread evenly over it
  __device__ __forceinline__ static int64_t block_at(int64_t x, int64_t blocks, int64_t cost) {
    return blocks == cost ? x : quotient(x * blocks, cost);
  }
};

// The stretches: worker w of `workers` takes cost [bound(w), bound(w + 1)),
// the first `more` one unit more than the others.  Fewer workgroups than there
// are share a small total, at least least_blocks to each.
struct Share {
  int64_t workers, each, more;
  __device__ __forceinline__ Share(int64_t total, int64_t most, int64_t least_blocks) {
    workers = max(min(most, total / least_blocks), int64_t{1});
    each = quotient(total, workers);
    more = total - each * workers;
  }
  __device__ __forceinline__ int64_t bound(int64_t w) const { return w * each + min(w, more); }
  // the worker whose stretch holds x
  __device__ __forceinline__ int64_t worker_at(int64_t x) const {
    const int64_t cut = more * (each + 1);
    return x < cut ? quotient(x, each + 1) : more + quotient(x - cut, each);
  }
};

// A worker's partial sums of a tile: slot 0 if its stretch begins inside the
// tile, 1 if it begins with or before it.  M rows of 256 floats to a slot, then for
// all slots the rows' maxima and sums.
template <int M>
__device__ __forceinline__ float* partial_row(const AttnArgs& a, int64_t worker, int slot, int row) {
  return a.partial + ((worker * 2 + slot) * M + row) * kDim;
}
template <int M>
__device__ __forceinline__ float2* partial_stat(const AttnArgs& a, int64_t worker, int slot, int row) {
  return reinterpret_cast<float2*>(a.partial + static_cast<int64_t>(a.workers) * 2 * M * kDim) + (worker * 2 + slot) * M + row;
}
constexpr int64_t partial_floats(int64_t workers, int64_t m) { return workers * 2 * m * (kDim + 2); }

// One worker's segments, one after the other.
struct Segment {
  int32_t b, head;
  int64_t tile, from, to, cost;  // places [from, to) of the tile's cost
};
template <int M, int KT, class F>
__device__ __forceinline__ void for_segments(const AttnArgs& a, const Share& s, const Found& first, int64_t worker, F run) {
  int64_t left = s.bound(worker + 1) - s.bound(worker);
  int64_t rest = first.rest;
  for (int32_t b = first.b; left > 0 && b < a.requests; ++b, rest = 0) {
    const Work<M, KT> w(a, b);
    if (w.tiles == 0) continue;
    const int64_t head_cost = w.head_cost();
    int32_t head = static_cast<int32_t>(quotient(rest, head_cost));
    rest -= head * head_cost;
    for (; head < a.kv_heads && left > 0; ++head, rest = 0) {
      int64_t j = w.tile_at(rest);
      rest -= w.cost_before(j);
      for (; j < w.tiles && left > 0; ++j, rest = 0) {
        Segment g{b, head, j, rest, min(rest + left, w.cost(j)), w.cost(j)};
        left -= g.to - g.from;
        run(w, g);
      }
    }
  }
}

}  // namespace hlwq_kv
