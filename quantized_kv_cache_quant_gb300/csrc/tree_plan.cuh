// How tree attention's work is cut, and how the pieces of one result are
// joined; shared by its kernels.
//
// The query rows of request b and kv head h are its T nodes x gq query heads
// (row r: node r / gq, head r % gq), in tiles of R rows. A (b, h, tile) is a
// "pair"; its work is ceil((len + T) / unit) units of tokens. The units of all
// pairs follow one another (b, then h, then tile: tiles that read the same
// keys run next to one another and meet in L2) and are cut into equal slices,
// one per thread block, whatever the requests' lengths; a cut that would leave
// fewer than `snap` units of a pair on one of its sides moves to the pair's
// nearer end, since a piece costs a partial result and a change of segments
// whatever its length. Lengths live on the device, so every thread block finds
// its slice itself with one scan over the requests. A block that holds only part
// of a pair leaves a partial result, its first segment's in slot 2c, a later
// one's in 2c + 1, and a second kernel joins them, always in the same order. A
// block begins at most one pair that it does not end: that pair is the one it
// describes to the second kernel, and the pair's other parts are the following
// blocks' first segments.
#pragma once

#include <climits>

#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "spec_internal.h"

namespace kvq {

// Lengths go up to the longest table, 16 below 2^31: neither of these leaves 31 bits there.
constexpr int kTreeLongest = INT_MAX / 16 * 16;
// Units of n tokens (n > 0).
__host__ __device__ constexpr int tree_units(int n, int unit) { return (n - 1) / unit + 1; }
// Whether the n tokens from tok on reach beyond the first len.
__host__ __device__ constexpr bool tree_beyond(int tok, int n, int len) { return tok > len - n; }
static_assert(tree_units(1, 64) == 1 && tree_units(64, 64) == 1 && tree_units(65, 64) == 2);
static_assert(tree_units(kTreeLongest, 64) == 1 << 25 && tree_units(kTreeLongest, 16) == INT_MAX / 16);
static_assert(!tree_beyond(0, 16, 16) && tree_beyond(1, 16, 16) && tree_beyond(0, 64, 0));
static_assert(tree_beyond(((1 << 25) - 1) * 64, 64, kTreeLongest) && !tree_beyond(((1 << 25) - 2) * 64, 64, kTreeLongest));
static_assert(!tree_beyond(kTreeLongest - 16, 16, kTreeLongest) && tree_beyond(kTreeLongest - 16, 16, kTreeLongest - 1));

struct TreeRequest {
  int first, nodes, len;  // first row, rows, tokens before them
  int units, tiles;       // per (head, tile); tiles of R rows
};

template <int R, int UNIT>
__device__ __forceinline__ TreeRequest tree_request(const TreeArgs& a, int b) {
  TreeRequest r;
  const int gq = a.q_heads / a.kv_heads, cap = min(a.max_blocks * 16, a.max_seq_len);
  r.first = min(max(a.tree_offsets[b], 0), a.n_tokens);
  const long long rows = static_cast<long long>(a.tree_offsets[b + 1]) - r.first;
  r.nodes = static_cast<int>(min(max(rows, 0ll), static_cast<long long>(min(min(a.max_tree, cap), a.n_tokens - r.first))));
  r.len = min(max(a.seq_lens[b], 0), cap - r.nodes);
  r.tiles = (r.nodes * gq + R - 1) / R;
  r.units = r.nodes > 0 ? tree_units(r.len + r.nodes, UNIT) : 0;
  return r;
}

struct TreeSlice {
  long long total;   // units of all pairs
  int blocks;        // slices that share them
  int snap;
  long long begin, end;  // (an empty slice: begin >= end)
  int b;             // request of the first unit
  long long before;  // units of the requests before b

  __device__ __forceinline__ long long cut(int c) const { return static_cast<long long>(c) * total / blocks; }
  // blocks that share the pair of units [begin, begin + units)
  __device__ __forceinline__ int parts_of(long long pair_begin, int units) const {
    // cut(c) >= u for c >= ceil(u * blocks / total)
    const long long lo = pair_begin + snap, hi = pair_begin + units - snap;
    if (lo > hi) return 1;
    auto first = [&](long long u) { return (u * blocks + total - 1) / total; };
    return 1 + static_cast<int>(first(hi + 1) - first(lo));
  }
};

// u / v for 0 <= u, 0 < v
__device__ __forceinline__ int tree_div(long long u, int v) {
  const unsigned long long x = static_cast<unsigned long long>(u);
  return x >> 32 ? static_cast<int>(x / v) : static_cast<int>(static_cast<uint32_t>(x) / static_cast<uint32_t>(v));
}

// The slice of thread block blockIdx.x. sm: 32 + 4 words of 8 bytes of shared
// memory that nothing else uses until the next __syncthreads after the call.
// shortest(u): the units that slices get at least, where a pair has about u;
// snap(u): the snap, 1 or more, of slices of u units.
template <int R, int UNIT, class Shortest, class Snap>
__device__ __forceinline__ TreeSlice tree_slice(const TreeArgs& a, unsigned long long* sm, Shortest shortest, Snap snap_of) {
  TreeSlice s;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  auto units_of = [&](int b) -> unsigned long long {
    if (b >= a.batch) return 0ull;
    const TreeRequest r = tree_request<R, UNIT>(a, b);
    return static_cast<unsigned long long>(r.units) * r.tiles * a.kv_heads;
  };
  // one chunk of blockDim.x requests: exclusive prefix of v, the chunk's sum in `sum`
  auto scan = [&](unsigned long long v, unsigned long long& sum) -> unsigned long long {
    unsigned long long inc = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long u = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += u;
    }
    if (lane == 31) sm[warp] = inc;
    __syncthreads();
    unsigned long long w = lane < warps ? sm[lane] : 0ull, before = 0ull;
    sum = 0ull;
    for (int i = 0; i < warps; ++i) {
      const unsigned long long x = __shfl_sync(0xffffffffu, w, i);
      if (i < warp) before += x;
      sum += x;
    }
    __syncthreads();
    return before + inc - v;
  };
  const unsigned long long mine = units_of(threadIdx.x);
  unsigned long long sum;
  const unsigned long long mine_at = scan(mine, sum);
  unsigned long long total = sum;
  for (int b0 = blockDim.x; b0 < a.batch; b0 += blockDim.x) {
    (void)scan(units_of(b0 + threadIdx.x), sum);
    total += sum;
  }
  s.total = static_cast<long long>(total);
  // (the pairs that requests of equal trees would have)
  const int rows = min((a.n_tokens - 1) / a.batch + 1, a.max_tree) * (a.q_heads / a.kv_heads);
  const int per = shortest(s.total / (static_cast<long long>(a.batch) * a.kv_heads * ((rows + R - 1) / R)));
  s.blocks = static_cast<int>(min(static_cast<long long>(gridDim.x), (s.total + per - 1) / per));
  const int snap = s.blocks > 0 ? snap_of(s.total / s.blocks) : 1;
  s.snap = snap;
  s.begin = s.end = s.before = 0;
  s.b = 0;
  if (static_cast<int>(blockIdx.x) >= s.blocks) return s;
  const unsigned long long u0 = static_cast<unsigned long long>(s.cut(blockIdx.x));
  const unsigned long long u1 = static_cast<unsigned long long>(s.cut(blockIdx.x + 1));  // == total for the last one
  auto claim = [&](int b, unsigned long long at, unsigned long long n) {
    if (at <= u0 && u0 < at + n) {
      sm[32] = static_cast<unsigned long long>(b);
      sm[33] = at;
    }
    if (at <= u1 && u1 < at + n) {
      sm[34] = static_cast<unsigned long long>(b);
      sm[35] = at;
    }
  };
  claim(threadIdx.x, mine_at, mine);
  unsigned long long carry = 0;
  if (a.batch > static_cast<int>(blockDim.x)) {
    (void)scan(mine, carry);
    for (int b0 = blockDim.x; b0 < a.batch; b0 += blockDim.x) {
      const unsigned long long n = units_of(b0 + threadIdx.x);
      const unsigned long long at = carry + scan(n, sum);
      claim(b0 + threadIdx.x, at, n);
      carry += sum;
    }
  }
  __syncthreads();
  // the cut at unit u of request b, whose units begin at `before`
  auto snapped = [&](long long u, int b, long long before) -> long long {
    const TreeRequest r = tree_request<R, UNIT>(a, b);
    const long long pair_begin = before + static_cast<long long>(tree_div(u - before, r.units)) * r.units;
    const int in = static_cast<int>(u - pair_begin);
    if (in >= snap && r.units - in >= snap) return u;
    return 2 * in <= r.units ? pair_begin : pair_begin + r.units;
  };
  s.b = static_cast<int>(sm[32]);
  s.before = static_cast<long long>(sm[33]);
  s.begin = snapped(u0, s.b, s.before);
  s.end = static_cast<int>(blockIdx.x) + 1 == s.blocks ? s.total : snapped(u1, static_cast<int>(sm[34]), static_cast<long long>(sm[35]));
  __syncthreads();
  return s;
}

// One pair's share of a slice.
struct TreeSegment {
  int b, h, tile;
  TreeRequest r;
  long long pair_begin;    // the pair's first unit in the range of all
  int u0, u1;              // units of the pair in this slice
  int slot;                // 2 * block (+ 1): where a partial result goes
  int parts;               // blocks that share the pair
};

struct TreeWalk {
  long long at, before;
  int b;
  TreeSegment seg;

  __device__ __forceinline__ void start(const TreeSlice& s) {
    at = s.begin;
    before = s.before;
    b = s.b;
    seg.b = -1;
  }
};

// Walks a slice's segments: w.at is the unit to go on from, w.b and w.before
// its request, w.seg.r that request once w.seg.b names it. Out of line: the
// roles of a thread block share one copy (their hot loops and five inlined
// copies together did not fit the instruction cache). Between two segments every
// role waits for this, so it reads a request once, not once a pair, and divides
// in 64 bits only for pairs that blocks share.
template <int R, int UNIT>
__device__ __noinline__ bool next_segment(const TreeArgs& a, const TreeSlice& s, TreeWalk& w) {
  long long at = w.at, before = w.before;
  int b = w.b;
  TreeSegment& g = w.seg;
  if (at >= s.end) return false;
  if (g.b != b) g.r = tree_request<R, UNIT>(a, b);
  long long n = static_cast<long long>(g.r.units) * g.r.tiles * a.kv_heads;
  while (at >= before + n) {  // requests without nodes have no units
    before += n;
    ++b;
    g.r = tree_request<R, UNIT>(a, b);
    n = static_cast<long long>(g.r.units) * g.r.tiles * a.kv_heads;
  }
  const int pair = tree_div(at - before, g.r.units);
  g.b = b;
  g.h = pair / g.r.tiles;
  g.tile = pair % g.r.tiles;
  g.pair_begin = before + static_cast<long long>(pair) * g.r.units;
  g.u0 = static_cast<int>(at - g.pair_begin);
  g.u1 = static_cast<int>(min(s.end - g.pair_begin, static_cast<long long>(g.r.units)));
  g.slot = 2 * static_cast<int>(blockIdx.x) + (at == s.begin ? 0 : 1);
  g.parts = g.u0 == 0 && g.u1 == g.r.units ? 1 : s.parts_of(g.pair_begin, g.r.units);
  w.at = g.pair_begin + g.u1;
  w.before = before;
  w.b = b;
  return true;
}

// Whether node `node`'s mask (row of words) lets it see the token at `tok`:
// every one before the tree, nodes by their bits, none behind the last node.
__device__ __forceinline__ bool tree_sees(const uint64_t* mask, int tok, int len, int total) {
  if (tok < len) return true;
  if (tok >= total) return false;
  const int j = tok - len;
  return (mask[j >> 6] >> (j & 63)) & 1;
}

// Bytes of four FP8 codes that are NaN (or an E5M2 infinity, which no cast of this library writes): 0xFF each.
template <int FMT>
__device__ __forceinline__ uint32_t fp8_nonfinite(uint32_t w) {
  const uint32_t mag = w & 0x7F7F7F7Fu;
  return FMT == 0 ? __vcmpeq4(mag, 0x7F7F7F7Fu) : __vcmpgeu4(mag, 0x7C7C7C7Cu);
}

// Output channels 4 c4 .. +3 of a pair's row.
template <int D>
__device__ __forceinline__ void tree_store4(const TreeArgs& a, const TreeSegment& g, int gq, int row, int c4, float4 v) {
  const long long at = (static_cast<long long>(g.r.first + row / gq) * a.q_heads + g.h * gq + row % gq) * D + 4 * c4;
  if (a.out_fp32)
    *reinterpret_cast<float4*>(reinterpret_cast<float*>(a.out) + at) = v;
  else
    *reinterpret_cast<uint2*>(reinterpret_cast<__half*>(a.out) + at) = make_uint2(pack_rn_f16x2(v.x, v.y), pack_rn_f16x2(v.z, v.w));
}

// The products take NaN codes of the tree's own value rows as 0 (a weight of 0
// times NaN would reach rows that do not see the token). Where any was met,
// this puts NaN into channels [c0, c1) of row `row` that such a code reaches
// through a node the row sees; by the thread that stored them.
template <int D, int FMT>
__device__ __noinline__ void tree_put_nan(const TreeArgs& a, int b, int h, int first, int nodes, int len, int row, int c0,
                                          int c1) {
  const int gq = a.q_heads / a.kv_heads, n = first + row / gq;
  const uint64_t* mask = a.tree_mask + static_cast<long long>(n) * a.mask_words;
  const long long at = (static_cast<long long>(n) * a.q_heads + h * gq + row % gq) * D;
#pragma unroll 1
  for (int j = 0; j < nodes; ++j) {
    if (!((mask[j >> 6] >> (j & 63)) & 1)) continue;
    const int tok = len + j, t = tok % 16;
    const int blk = min(max(a.block_table[static_cast<long long>(b) * a.max_blocks + tok / 16], 0), a.num_blocks - 1);
    const uint8_t* vb = a.v_pool + (static_cast<long long>(blk) * a.kv_heads + h) * (16 * D);
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      const uint32_t code = vb[(c / 32 * 32 + 4 * (c % 8) + t % 8 / 2) * 16 + c % 32 / 8 * 4 + t / 8 * 2 + t % 2];
      if (fp8_nonfinite<FMT>(code) & 0xFFu) {
        if (a.out_fp32) reinterpret_cast<float*>(a.out)[at + c] = NAN;
        else reinterpret_cast<uint16_t*>(a.out)[at + c] = 0x7FFFu;
      }
    }
  }
}

// What a block leaves for the joining kernel: the pair it began and did not
// end (parts 0: none). A block begins at most one such pair.
__device__ __forceinline__ void tree_leave_none(const TreeArgs& a) {
  a.joins[blockIdx.x].parts = 0;
}
__device__ __forceinline__ void tree_leave_join(const TreeArgs& a, const TreeSegment& g, int rows, int row0) {
  TreeJoin j;
  j.parts = g.parts;
  j.slot0 = g.slot;
  j.rows = rows;
  j.row0 = row0;
  j.b = g.b;
  j.h = g.h;
  j.first = g.r.first;
  j.nodes = g.r.nodes;
  j.len = g.r.len;
  a.joins[blockIdx.x] = j;
}

}  // namespace kvq
