// How group attention's work is cut (by tree_plan.cuh) and where its kernels
// leave their results.
//
// The sequences of a group share leading blocks. The work has two kinds of
// pairs: (group, kv head, tile of the group's query rows) over the shared
// blocks, and (sequence, kv head, tile) over the blocks behind them; no row of a
// pair is masked. A launch takes one kind or both, the shared ones first. Every
// pair leaves sums and outputs of its rows, not yet divided, as multiples of
// 2^m with m the number that it leaves beside them (the kernels' weights carry
// different factors), and a last kernel joins what a row has of each kind.
#pragma once

#include "beam_internal.h"
#include "tree_plan.cuh"

namespace kvq {

struct GroupRequest {
  int first, nodes, len;  // first sequence (row of q), sequences, tokens
  int units, tiles;       // per (head, tile); tiles of R rows
  int seq, block0;        // row of the block table and its first column
  int kind, index;        // kind of pair, number among the requests of its kind
};

// The shared blocks of group g, as far as the table and max_seq_len reach.
__device__ __forceinline__ int group_shared(const GroupArgs& a, int g) {
  return min(max(a.shared_blocks[g], 0), min(a.max_blocks, a.max_seq_len / 16));
}

template <int R, int UNIT>
__device__ __forceinline__ GroupRequest tree_request(const GroupArgs& a, int b) {
  GroupRequest r;
  const int gq = a.q_heads / a.kv_heads, groups = a.batch / a.width;
  const bool shared = (a.kinds & 1) != 0 && b < groups;
  if (shared) {
    r.kind = 0;
    r.index = b;
    r.first = b * a.width;
    // the table row of a sequence that is not empty (an empty one's row names no blocks)
    int live = 0;
    while (live < a.width && a.seq_lens[r.first + live] <= 0) ++live;
    r.nodes = live < a.width ? a.width : 0;
    r.seq = r.first + (live < a.width ? live : 0);
    r.block0 = 0;
    r.len = group_shared(a, b) * 16;
  } else {
    const int i = (a.kinds & 1) != 0 ? b - groups : b;
    r.kind = 1;
    r.index = i;
    r.first = i;
    r.nodes = 1;
    r.seq = i;
    r.block0 = group_shared(a, i / a.width);
    r.len = min(max(a.seq_lens[i], 0), min(a.max_blocks * 16, a.max_seq_len)) - r.block0 * 16;
  }
  r.tiles = (r.nodes * gq + R - 1) / R;
  r.units = r.nodes > 0 && r.len > 0 ? tree_units(r.len, UNIT) : 0;
  return r;
}

__device__ __forceinline__ int plan_requests(const GroupArgs& a) {
  return ((a.kinds & 1) != 0 ? a.batch / a.width : 0) + ((a.kinds & 2) != 0 ? a.batch : 0);
}
template <int R>
__device__ __forceinline__ long long plan_pairs(const GroupArgs& a) {
  const int gq = a.q_heads / a.kv_heads;
  long long n = 0;
  if ((a.kinds & 1) != 0) n += static_cast<long long>(a.batch / a.width) * ((a.width * gq + R - 1) / R);
  if ((a.kinds & 2) != 0) n += static_cast<long long>(a.batch) * ((gq + R - 1) / R);
  return n * a.kv_heads;
}

using GroupSegment = PlanSegment<GroupRequest>;
using GroupWalk = PlanWalk<GroupRequest>;

// Where partial row f of the segment's row `row` (of the tile) goes: its output, its maximum and sum. `tile_row`: the
// kernel's row that computed it; `tile_rows`: how many those are.
struct GroupPlace {
  float* o;
  float* ml;
};
template <int D>
__device__ __forceinline__ GroupPlace group_place(const GroupArgs& a, const GroupSegment& g, int gq, int row0, int row, int f,
                                                  int tile_row, int tile_rows) {
  const GroupPartials& p = a.part[g.r.kind];
  long long at;
  if (g.parts == 1) {
    const int r = row0 + row;
    at = static_cast<long long>(f) * a.batch * a.q_heads + static_cast<long long>(g.r.first + r / gq) * a.q_heads + g.h * gq + r % gq;
    return {p.whole_o + at * D, p.whole_ml + at * 2};
  }
  at = static_cast<long long>(g.slot) * tile_rows + tile_row;
  return {p.o + at * D, p.ml + at * 2};
}

// By one thread: what the last kernel has to know of a pair that begins in this segment.
__device__ __forceinline__ void group_record(const GroupArgs& a, const GroupSegment& g) {
  if (g.u0 != 0) return;
  GroupRecord* r = a.part[g.r.kind].records + (static_cast<long long>(g.r.index) * a.kv_heads + g.h) * g.r.tiles + g.tile;
  *r = GroupRecord{g.parts, g.slot};
}

}  // namespace kvq
