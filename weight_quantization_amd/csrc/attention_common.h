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
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr float kLog2e = 1.44269504088896340736f;
// A row's running maximum is raised, and its sums rescaled, only once a score
// passes it by this much (in powers of two): probabilities then reach 2^8,
// far inside the range of bf16, fp16 and fp32, and the rescale of 256 sums is
// paid a few times per row instead of once per tile.
constexpr float kLazy = 8.0f;
constexpr float kTopWeight = 128;  // times 2^kLazy still below fp16's largest, 65504

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
  int32_t slots;    // of partial sums
  int32_t least, most;  // requests with rows * group in [least, most] are this kernel's
  int32_t cost_shift;
  float scale;   // its sign is given to the queries
  float factor;  // |scale| log2 e, above 0: a masked score, minus infinity, stays that
};

// One request's part of a step.
struct Extent {
  int32_t begin, n;   // rows
  int64_t held, enc;  // tokens before the step, those of them encoded
  int64_t paged;      // encoded tokens that have a table entry
};
__device__ __forceinline__ Extent extent_of(const AttnArgs& a, int32_t begin, int32_t n, int32_t len) {
  Extent e;
  e.begin = begin;
  e.n = n;
  e.held = len > n ? len - n : 0;  // a length may be anything: len - n alone could pass 32 bits
  e.enc = a.lens ? max(e.held - a.n_res, int64_t{0}) : 0;
  e.paged = a.n_pages > 0 ? min(e.enc, static_cast<int64_t>(a.width) << a.page_shift) : 0;
  return e;
}
__device__ __forceinline__ Extent extent_of(const AttnArgs& a, int32_t b) {
  const RowRange r = row_range(a.cu, b, a.rows);
  return extent_of(a, r.begin, r.end - r.begin, a.lens ? a.lens[b] : 0);
}

// The token that row r of a request belongs to.
__device__ __forceinline__ int32_t token_of(int32_t r, int32_t group) {
  return static_cast<int32_t>(static_cast<uint32_t>(r) / static_cast<uint32_t>(group));
}

__device__ __forceinline__ float fast_exp2(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ float half_swap(float v) { return lane_xor(v, 32); }

// Two floats rounded to a pair of fp16, to nearest.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const f16x2 v = {static_cast<_Float16>(lo), static_cast<_Float16>(hi)};
  return __builtin_bit_cast(uint32_t, v);
}

// In a rare branch: keeps the compiler from doing its work always and selecting.
__device__ __forceinline__ void keep_branch() { asm volatile(""); }

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
// LDS or a barrier: lane i takes requests i, i + 64, ..  Sums stay below 2^31
// (cost_shift), as 64-bit divisions cost hundreds of instructions.
// ---------------------------------------------------------------------------

// A quantity of each request, its sum, and the request that holds a place of
// it.  (Of up to 64 requests everything stays in registers between the two.)
struct Found {
  int32_t b;
  int32_t rest, before;  // the place's within the request, the sum of `other` over the requests before it
  Extent e;              // of the request
};
template <class F, class G>
struct Finder {
  F of;
  G other;
  int32_t requests;
  int32_t own, prefix, total;
  Extent mine;
  const AttnArgs& args;
  __device__ __forceinline__ Finder(const AttnArgs& a, F f, G g) : of(f), other(g), requests(a.requests), args(a) {
    const int lane = threadIdx.x & 63;
    total = 0;
    bool falls = false;
    for (int32_t b0 = 0; b0 < requests; b0 += 64) {
      const int32_t b = min(b0 + lane, requests - 1);
      mine = extent_of(a, b);
      own = b0 + lane < requests ? of(mine) : 0;
      falls |= a.cu[b + 1] < a.cu[b];
      prefix = wave_scan(own);
      total += __builtin_amdgcn_readlane(prefix, 63);
    }
    // where cu falls, rows could belong to several requests and the sums pass
    // what the host has allowed for: such a call does nothing
    if (__any(falls)) total = 0;
  }
  // place x, 0 <= x < total
  __device__ __forceinline__ Found find(int32_t x) {
    const int lane = threadIdx.x & 63;
    Found f{-1, 0, 0, {}};
    for (int32_t b0 = 0; b0 < requests; b0 += 64) {
      const bool in = b0 + lane < requests;
      if (requests > 64) {
        mine = extent_of(args, min(b0 + lane, requests - 1));
        own = in ? of(mine) : 0;
        prefix = wave_scan(own);
      }
      const int32_t aside = wave_scan(in ? other(mine) : 0);
      const uint64_t past = __ballot(x < prefix);
      if (past) {
        const int at = __builtin_ctzll(past);
        f.b = b0 + at;
        f.rest = x - __builtin_amdgcn_readlane(prefix - own, at);
        if (at > 0) f.before += __builtin_amdgcn_readlane(aside, at - 1);
        f.e = extent_at(at);
        return f;
      }
      x -= __builtin_amdgcn_readlane(prefix, 63);
      f.before += __builtin_amdgcn_readlane(aside, 63);
    }
    return f;
  }
  // Place x of up to 64 requests' places taken from the last to the first: all
  // those of rest >= j come before those of rest = j - 1.
  __device__ __forceinline__ Found find_from_last(int32_t x) const {
    const auto beyond = [&](int32_t j) { return __builtin_amdgcn_readlane(wave_scan(max(own - j, 0)), 63); };
    int32_t j = 0, none = total;  // beyond(j) > x >= beyond(none)
    while (none - j > 1) {
      const int32_t mid = j + (none - j) / 2;
      (beyond(mid) > x ? j : none) = mid;
    }
    x -= beyond(j + 1);
    uint64_t having = __ballot(own > j);
    for (; x > 0; --x) having &= having - 1;
    const int at = __builtin_ctzll(having);
    return Found{at, j, 0, extent_at(at)};
  }
  // of lane `at`'s request
  __device__ __forceinline__ Extent extent_at(int at) const {
    return extent_of(args, __builtin_amdgcn_readlane(mine.begin, at), __builtin_amdgcn_readlane(mine.n, at),
                     static_cast<int32_t>(__builtin_amdgcn_readlane(static_cast<int32_t>(mine.held), at)) +
                         __builtin_amdgcn_readlane(mine.n, at));
  }
};
struct Nothing {
  __device__ __forceinline__ int32_t operator()(const Extent&) const { return 0; }
};

__device__ __forceinline__ int32_t quotient(int32_t a, int32_t b) {
  return static_cast<int32_t>(static_cast<uint32_t>(a) / static_cast<uint32_t>(b));
}

// How the paged kernels share their work out.  A tile is M consecutive rows of
// one request and KV head; it costs its key blocks of KT tokens: those of the
// pages, then those of the window and of the step's own tokens up to the
// tile's last row.  The tiles lie one after the other, by request, KV head and
// row, and every workgroup takes an equal stretch of their cost, so that
// requests of any lengths load the workgroups alike; a tile that several
// workgroups share is joined from their partial sums afterwards.  (The cost
// need only be near the blocks' number: it is counted in eighths of one, so
// that it grows by as little as a tile's tokens do, or, where its sum could pass
// 2^31, in units of 2^cost_shift blocks.)
constexpr int32_t kBlockCost = 8;
template <int M, int KT>
struct Work {
  Extent e;
  int32_t tiles, page_blocks, base, step;
  __device__ __forceinline__ Work(const AttnArgs& a, const Extent& x) {
    e = x;
    const int32_t r = rows(a);
    tiles = r >= a.least && r <= a.most ? static_cast<int32_t>(ceil_div(r, M)) : 0;
    page_blocks = static_cast<int32_t>(ceil_div(e.paged, KT));
    base = page_blocks + static_cast<int32_t>(ceil_div(e.held - e.enc + 1, KT));
    if (a.cost_shift) {
      base = (base >> a.cost_shift) + 1;
      step = 0;
    } else {
      base *= kBlockCost;
      step = quotient(kBlockCost * M / KT, a.group) + 1;  // what a tile's tokens come to, rounded up
    }
  }
  // of one KV head
  // (unsigned: j (j - 1) may pass 2^31, but only where step is 0)
  __device__ __forceinline__ int32_t cost_before(int32_t j) const {
    const uint32_t u = static_cast<uint32_t>(j);
    return static_cast<int32_t>(u * static_cast<uint32_t>(base) + static_cast<uint32_t>(step) * (u * (u - 1) / 2));
  }
  __device__ __forceinline__ int32_t cost(int32_t j) const { return base + step * j; }
  __device__ __forceinline__ int32_t head_cost() const { return cost_before(tiles); }
  // the tile that holds place x of a KV head's cost: from an estimate of the
  // root of cost_before(j) = x
  __device__ __forceinline__ int32_t tile_at(int32_t x) const {
    if (tiles == 1) return 0;
    const float b = 2.0f * base - step, s = step;
    int32_t j = step ? static_cast<int32_t>((__builtin_amdgcn_sqrtf(b * b + 8.0f * s * x) - b) * 0.5f * __builtin_amdgcn_rcpf(s))
                     : quotient(x, base);
    j = max(min(j, tiles - 1), 0);
    while (j > 0 && cost_before(j) > x) --j;
    while (j + 1 < tiles && cost_before(j + 1) <= x) ++j;
    return j;
  }
  __device__ __forceinline__ int32_t rows(const AttnArgs& a) const { return e.n * a.group; }
  // tokens (of the step) of the tile's first row and last row
  __device__ __forceinline__ int32_t first_token(const AttnArgs& a, int32_t j) const { return token_of(j * M, a.group); }
  __device__ __forceinline__ int32_t last_token(const AttnArgs& a, int32_t j) const {
    return token_of(min(M, rows(a) - j * M) + j * M - 1, a.group);
  }
  // key blocks of tile j: the pages', then the others
  __device__ __forceinline__ int32_t blocks(const AttnArgs& a, int32_t j) const {
    return page_blocks + static_cast<int32_t>(ceil_div(e.held - e.enc + last_token(a, j) + 1, KT));
  }
  // the block at place x of a tile's cost: its blocks spread evenly over it
  __device__ __forceinline__ static int32_t block_at(int32_t x, int32_t blocks, int32_t cost) {
    if (cost == blocks * kBlockCost) return x / kBlockCost;
    if (x == cost) return blocks;
    return __builtin_amdgcn_readfirstlane(static_cast<int32_t>(static_cast<double>(x) * blocks / cost));
  }
};

// The stretches: worker w of `workers` takes cost [bound(w), bound(w + 1)), all
// but the last the same, at least `least`.  Where that is a few blocks, fewer
// workers than there could be take as long as all of them and leave fewer
// partial sums to join.
struct Share {
  int32_t total, each, workers;
  __device__ __forceinline__ Share(int32_t cost, int32_t most, int32_t least) : total(cost) {
    each = max(quotient(cost - 1, most) + 1, least);
    workers = quotient(cost - 1, each) + 1;
  }
  __device__ __forceinline__ int32_t bound(int32_t w) const {
    return static_cast<int32_t>(min(static_cast<uint32_t>(w) * static_cast<uint32_t>(each), static_cast<uint32_t>(total)));
  }
  // the worker whose stretch holds x
  __device__ __forceinline__ int32_t worker_at(int32_t x) const { return quotient(x, each); }
};

// Partial sums lie in slots of M rows of 256 floats, followed for all slots by
// the rows' maxima and sums.  Worker w has slot 2 w for a stretch that begins
// inside a tile and 2 w + 1 for one that begins with the tile and ends inside it.
template <int M>
__device__ __forceinline__ float* partial_row(const AttnArgs& a, int32_t slot, int row) {
  return a.partial + (slot * static_cast<int64_t>(M) + row) * kDim;
}
template <int M>
__device__ __forceinline__ float2* partial_stat(const AttnArgs& a, int32_t slot, int row) {
  return reinterpret_cast<float2*>(a.partial + static_cast<int64_t>(a.slots) * M * kDim) + slot * static_cast<int64_t>(M) + row;
}
constexpr int64_t partial_floats(int64_t slots, int64_t m) { return slots * m * (kDim + 2); }

// One worker's segments, one after the other.
struct Segment {
  int32_t b, head;
  int32_t tile, from, to, cost;  // places [from, to) of the tile's cost
};
template <int M, int KT, class F>
__device__ __forceinline__ void for_segments(const AttnArgs& a, const Share& s, const Found& first, int32_t worker, F run) {
  int32_t left = s.bound(worker + 1) - s.bound(worker);
  int32_t b = first.b, rest = first.rest;
#pragma clang loop unroll(disable)
  while (left > 0 && b < a.requests) {
    const Work<M, KT> w(a, b == first.b ? first.e : extent_of(a, b));
    const int32_t head_cost = w.head_cost();
    Segment g;
    g.b = b;
    g.head = head_cost ? quotient(rest, head_cost) : a.kv_heads;
    if (g.head >= a.kv_heads) {  // past the request's last
      ++b;
      rest = 0;
      continue;
    }
    const int32_t x = rest - g.head * head_cost;
    g.tile = __builtin_amdgcn_readfirstlane(w.tile_at(x));
    g.cost = w.cost(g.tile);
    g.from = x - w.cost_before(g.tile);
    g.to = min(g.from + left, g.cost);
    left -= g.to - g.from;
    rest += g.to - g.from;
    run(w, g);
  }
}

}  // namespace hlwq_kv
