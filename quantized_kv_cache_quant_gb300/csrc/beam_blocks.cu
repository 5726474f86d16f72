// Blocks that several sequences share, for sm_103a: tables that follow their
// parents, copies of blocks, compaction of a pool (kvq_beam.h).
#include <climits>
#include <cooperative_groups.h>

#include "beam_internal.h"
#include "block_scan.cuh"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "spec_internal.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// Fork, first launch: the entries. A thread block takes a request, a warp 32 of
// its columns at a time: it reads the old entries of all sequences, then writes
// the parents' ones, so that the tables can change in place. An entry that
// changes adds a reference to the new block and takes one from the old block.
// All of a column's additions come before its subtractions, and no other request
// adds a reference to a block without holding one itself, so a count falls below
// 0 only when the last reference has gone, and for one thread only: that thread
// marks the block as free.
// Both launches, called in a row: 64 requests of 8 sequences over 32K tokens 15.9
// us, 8 requests of 4 over 1000 tokens 9.0. That is latency, a chain of loads,
// atomics and barriers in each of them.
// ---------------------------------------------------------------------------
constexpr int kForkWarps = 4;

__global__ void __launch_bounds__(32 * kForkWarps) fork_entries_kernel(const BlocksForkArgs a) {
  extern __shared__ int old_all[];  // [kForkWarps][width][32]
  __shared__ int parent_s[kBeamMaxWidth], held_s[kBeamMaxWidth], len_s[kBeamMaxWidth], want_s[kBeamMaxWidth];
  __shared__ int most_s, full_s;
  const int g = blockIdx.x, w = a.width, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    most_s = 0;
    full_s = INT_MAX;
  }
  for (int i = threadIdx.x; i < w; i += blockDim.x) {
    const int b = g * w + i;
    parent_s[i] = a.parents[b];
    held_s[i] = min(max(a.n_held[b], 0), a.max_blocks);
    len_s[i] = max(a.seq_lens[b], 0);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < w; i += blockDim.x) {
    const int p = parent_s[i];
    int want = 0;
    if (p >= 0 && p < w) {
      const long long len = min(static_cast<long long>(len_s[p]), static_cast<long long>(held_s[p]) * a.block_tokens);
      want = static_cast<int>((len + a.block_tokens - 1) / a.block_tokens);
    } else {
      parent_s[i] = -1;  // (read by this thread alone until the barrier)
    }
    want_s[i] = want;
  }
  __syncthreads();
  if (threadIdx.x < w) {
    atomicMax(&most_s, max(held_s[threadIdx.x], want_s[threadIdx.x]));
    if (want_s[threadIdx.x] > 0) atomicMin(&full_s, want_s[threadIdx.x]);
  }
  __syncthreads();
  const int most = most_s, full = full_s;
  int* old_s = old_all + warp * w * 32;
  int32_t* table = a.block_table + static_cast<long long>(g) * w * a.max_blocks;
  auto counted = [&](int block) { return block >= 0 && block < a.num_blocks; };
  int first_differing = INT_MAX;
  for (int c0 = (blockIdx.y * kForkWarps + warp) * 32; c0 < most; c0 += gridDim.y * kForkWarps * 32) {
    const int c = c0 + lane;
#pragma unroll 8
    for (int i = 0; i < w; ++i) old_s[i * 32 + lane] = c < held_s[i] ? table[static_cast<long long>(i) * a.max_blocks + c] : -1;
    bool alike = true;
    int lead = -1;
    bool any = false;
    for (int i = 0; i < w; ++i) {
      const int old = old_s[i * 32 + lane], now = c < want_s[i] ? old_s[parent_s[i] * 32 + lane] : -1;
      if (want_s[i] > 0) {
        if (!any) lead = now;
        alike &= now == lead;
        any = true;
      }
      // (entries behind the held ones become -1 too)
      if (now != old) {
        table[static_cast<long long>(i) * a.max_blocks + c] = now;
        if (counted(now)) atomicAdd(a.shares + now, 1);
      }
    }
    for (int i = 0; i < w; ++i) {
      const int old = old_s[i * 32 + lane], now = c < want_s[i] ? old_s[parent_s[i] * 32 + lane] : -1;
      if (now != old && counted(old) && atomicSub(a.shares + old, 1) == 0) {
        a.shares[old] = 0;
        atomicOr(a.bits + word_at(old >> 5), 1u << (old & 31));
      }
    }
    if (!alike && c < full) first_differing = min(first_differing, c);
  }
  // (columns from `full` on cannot be shared, so they need no look)
  first_differing = __reduce_min_sync(0xffffffffu, first_differing);
  if (lane == 0 && first_differing < a.max_blocks) atomicMax(a.alike + g, a.max_blocks - first_differing);
}

// ---------------------------------------------------------------------------
// Fork, second launch, one cluster: the freed blocks go to the stack, the
// sequences with a partly filled shared last block take blocks from it.
//   A = blocks free after the push; freed block number e (ascending) of n goes
//   to place count + n - 1 - e, copy r takes place A - 1 - r.
// Every block of the cluster counts its part of the bits; the first one knows
// the sequences. It starts while the first launch runs and reads the sequences'
// lengths meanwhile; what that launch writes (entries, counts, bits) it reads
// after it.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(1024) fork_tails_kernel(const BlocksForkArgs a) {
  extern __shared__ int sm[];
  int* len_s = sm;                 // [batch] new length
  int* tail_s = len_s + a.batch;   // [batch] last block if partly filled, else -1
  __shared__ unsigned long long scan_ws[32], freed_s;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
  const int words = (a.num_blocks + 31) / 32;
  const int per = (words + ranks - 1) / ranks, w0 = min(words, rank * per), w1 = min(words, w0 + per);
  const int count = min(max(*a.free_count, 0), a.num_blocks);
  if (rank == 0) {
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
      const int first = b / a.width * a.width, p = a.parents[b];
      int len = 0;
      if (p >= 0 && p < a.width) {
        const int held = min(max(a.n_held[first + p], 0), a.max_blocks);
        len = static_cast<int>(min(static_cast<long long>(max(a.seq_lens[first + p], 0)), static_cast<long long>(held) * a.block_tokens));
      }
      len_s[b] = len;
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // the last blocks (each thread's own lengths), and the freed blocks of this part
  if (rank == 0) {
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
      const int len = len_s[b], column = len / a.block_tokens;
      int tail = -1;
      if (len != column * a.block_tokens) tail = __ldcg(a.block_table + static_cast<long long>(b) * a.max_blocks + column);
      tail_s[b] = tail >= 0 && tail < a.num_blocks ? tail : -1;
    }
  }
  unsigned long long mine = 0, ignore;
  for (int i = w0 + threadIdx.x; i < w1; i += blockDim.x) mine += __popc(__ldcg(a.bits + word_at(i)));
  (void)block_scan(mine, scan_ws, ignore);
  long long before = 0, freed = static_cast<long long>(ignore);
  if (ranks > 1) {
    if (threadIdx.x == 0) freed_s = ignore;
    cluster.sync();
    freed = 0;
    for (int r = 0; r < ranks; ++r) {
      const long long n = static_cast<long long>(*cluster.map_shared_rank(&freed_s, r));
      if (r < rank) before += n;
      freed += n;
    }
  }
  const int top = static_cast<int>(min(count + freed, static_cast<long long>(a.num_blocks)));
  if (freed > 0) {
    for (int i0 = w0; i0 < w1; i0 += blockDim.x) {
      const int i = i0 + threadIdx.x;
      uint32_t word = i < w1 ? __ldcg(a.bits + word_at(i)) : 0u;
      __syncthreads();
      unsigned long long total;
      long long e = before + static_cast<long long>(block_scan(__popc(word), scan_ws, total));
      before += static_cast<long long>(total);
      if (word != 0) a.bits[word_at(i)] = 0u;
      for (; word != 0; word &= word - 1, ++e) {
        const long long place = count + freed - 1 - e;
        if (place >= 0 && place < a.num_blocks) a.free_blocks[place] = 32 * i + __ffs(word) - 1;
      }
    }
  }
  if (ranks > 1) cluster.sync();  // the pushes are done, nobody reads another block's count any more
  else __syncthreads();
  if (rank != 0) return;
  int copies = 0;  // of the sequences before
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    bool copier = false;
    int tail = -1;
    if (b < a.batch && (tail = tail_s[b]) >= 0) {
      const int shares = __ldcg(a.shares + tail);
      const int first = b / a.width * a.width;
      int among = 0;
      bool earlier = false;
      for (int i = first; i < first + a.width; ++i) {
        among += tail_s[i] == tail;
        earlier |= tail_s[i] == tail && i < b;
      }
      copier = earlier || shares + 1 != among;
    }
    unsigned long long total;
    const int r = copies + static_cast<int>(block_scan(copier ? 1ull : 0ull, scan_ws, total));
    copies += static_cast<int>(total);
    if (b < a.batch) {
      const int len = len_s[b];
      const bool made = copier && r < top;
      if (made) {
        const int fresh = __ldcg(a.free_blocks + (top - 1 - r));
        a.block_table[static_cast<long long>(b) * a.max_blocks + len / a.block_tokens] = fresh;
        a.copy_src[r] = tail;
        a.copy_dst[r] = fresh;
      }
      // the old block's count falls once all sequences have looked at it: a copy is marked in its length
      if (made) len_s[b] = -1 - len;
      if (a.granted != nullptr) a.granted[b] = !copier || made;
    }
    __syncthreads();
  }
  for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
    int len = len_s[b];
    if (len < 0) {
      len = -1 - len;
      atomicSub(a.shares + tail_s[b], 1);
      len_s[b] = len;
    }
    a.seq_lens[b] = len;
    a.n_held[b] = static_cast<int>((static_cast<long long>(len) + a.block_tokens - 1) / a.block_tokens);
  }
  __syncthreads();
  for (int g = threadIdx.x; g < a.batch / a.width; g += blockDim.x) {
    const int alike = __ldcg(a.alike + g);
    int full = INT_MAX;
    for (int i = 0; i < a.width; ++i)
      if (len_s[g * a.width + i] > 0) full = min(full, len_s[g * a.width + i] / a.block_tokens);
    if (alike != 0) a.alike[g] = 0;
    if (a.shared_blocks != nullptr)
      a.shared_blocks[g] = full == INT_MAX ? 0 : min(full, alike == 0 ? a.max_blocks : a.max_blocks - alike);
  }
  if (threadIdx.x == 0) {
    const int made = min(copies, top);
    *a.copy_count = made;
    *a.free_count = top - made;
  }
}

// ---------------------------------------------------------------------------
// Copies. A warp takes pieces of 4 KB: 8 loads of 16 bytes a lane in flight,
// then the stores. Pieces of one pair follow one another through all buffers.
// Bound by memory: 448 pairs in 32 buffers of 16 KB blocks in 70 us (76 where
// calls follow each other), 6.2 TB/s read and written. Four blocks an SM are as
// many as their registers let in.
// ---------------------------------------------------------------------------
constexpr int kCopyThreads = 256;

__global__ void __launch_bounds__(kCopyThreads) blocks_copy_kernel(const __grid_constant__ BlocksCopyArgs a) {
  constexpr int kUnits = kCopyPiece / 512;  // 16-byte units a lane
  const int lane = threadIdx.x & 31;
  const int pieces = a.first_piece[a.n_buffers];
  int n = a.n_pairs;
  if (a.count != nullptr) n = min(n, max(*a.count, 0));
  const long long items = static_cast<long long>(n) * pieces;
  for (long long it = (static_cast<long long>(blockIdx.x) * kCopyThreads + threadIdx.x) >> 5; it < items;
       it += static_cast<long long>(gridDim.x) * (kCopyThreads / 32)) {
    const int pair = it >> 32 ? static_cast<int>(it / pieces) : static_cast<int>(static_cast<uint32_t>(it) / static_cast<uint32_t>(pieces));
    const int piece = static_cast<int>(it - static_cast<long long>(pair) * pieces);
    const int from = a.src[pair], to = a.dst[pair];
    int lo = 0, hi = a.n_buffers;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (a.first_piece[mid] <= piece) lo = mid;
      else hi = mid;
    }
    if (from < 0 || from >= a.num_blocks || to < 0 || to >= a.num_blocks) continue;
    const long long bytes = a.block_bytes[lo], at = static_cast<long long>(piece - a.first_piece[lo]) * kCopyPiece;
    const uint4* src = reinterpret_cast<const uint4*>(a.base[lo] + from * bytes + at) + lane;
    uint4* dst = reinterpret_cast<uint4*>(a.base[lo] + to * bytes + at) + lane;
    const int units = static_cast<int>(min(bytes - at, static_cast<long long>(kCopyPiece)) / 16) - lane;
    uint4 v[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      if (32 * u < units) v[u] = src[32 * u];
#pragma unroll
    for (int u = 0; u < kUnits; ++u)
      if (32 * u < units) dst[32 * u] = v[u];
  }
}

// ---------------------------------------------------------------------------
// Compaction: the free blocks as bits (mark), their ranks (rank: one cluster,
// "targets" are the free blocks below keep, "movers" the used ones from keep on),
// the lists (lists: mover r goes to target r, the targets left form the stack),
// and what follows the moves (follow: map, shares, tables). Five launches, each
// of which starts under the one before. 1M blocks and 512 tables: 32 us for 13 MB,
// of which the launches' dependences on each other are some 11 and the scattered
// atomics, reads and writes the rest.
// ---------------------------------------------------------------------------
constexpr int kCompactThreads = 256;

// Bits of word i that are blocks below keep, and those that are blocks of the pool from keep on.
__device__ __forceinline__ uint32_t low_bits(int n) { return n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u; }
__device__ __forceinline__ uint32_t target_bits(const BlocksCompactArgs& a, int i, uint32_t word) {
  return word & low_bits(a.keep - 32 * i);
}
__device__ __forceinline__ uint32_t mover_bits(const BlocksCompactArgs& a, int i, uint32_t word) {
  return ~word & low_bits(a.num_blocks - 32 * i) & ~low_bits(a.keep - 32 * i);
}
// What a pass of the same launch has written is read past L1 (SAME), that of a launch before through it.
template <bool SAME, class T>
__device__ __forceinline__ T passed(const T* p) {
  return SAME ? __ldcg(p) : *p;
}
// Rank of mover x among the movers.
template <bool SAME>
__device__ __forceinline__ int mover_rank(const BlocksCompactArgs& a, int x, uint32_t word) {
  const int i = x >> 5;
  // (the word that keep cuts counts the targets before it; it is the first with movers)
  return (i > a.keep >> 5 ? passed<SAME>(a.before + word_at(i)) : 0) + __popc(mover_bits(a, i, word) & ((1u << (x & 31)) - 1u));
}

// The four passes, by thread `me` of `threads`.
__device__ __forceinline__ void compact_mark(const BlocksCompactArgs& a, long long me, long long threads) {
  const int count = min(max(*a.free_count, 0), a.num_blocks);
  for (long long i = me; i < count; i += threads) {
    const int x = a.free_blocks[i];
    if (x >= 0 && x < a.num_blocks) atomicOr(a.bits + word_at(x >> 5), 1u << (x & 31));
  }
}

// By a cluster: each block ranks its part of the words.
__device__ __forceinline__ void compact_rank(const BlocksCompactArgs& a, unsigned long long* scan_ws, unsigned long long* sums) {
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = cluster.block_rank(), ranks = cluster.num_blocks();
  const int words = (a.num_blocks + 31) / 32, cut = a.keep >> 5;
  const int per = ((words + ranks - 1) / ranks + 3) & ~3, w0 = min(words, rank * per), w1 = min(words, w0 + per);
  // low half: targets, high half: movers
  auto both = [&](int i, uint32_t word) -> unsigned long long {
    return static_cast<unsigned long long>(__popc(target_bits(a, i, word))) |
           (static_cast<unsigned long long>(__popc(mover_bits(a, i, word))) << 32);
  };
  // a thread's four words from i on (i a multiple of 4: they lie side by side), and their counts
  auto four = [&](int i, unsigned long long (&n)[4]) -> unsigned long long {
    uint4 w = make_uint4(0u, 0u, 0u, 0u);
    if (i < w1) w = __ldcg(reinterpret_cast<const uint4*>(a.bits + word_at(i)));
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) n[e] = i + e < w1 ? both(i + e, word[e]) : 0ull;
    return (n[0] + n[1]) + (n[2] + n[3]);
  };
  unsigned long long mine = 0, total, n[4];
  for (int i = w0 + 4 * threadIdx.x; i < w1; i += 4 * blockDim.x) mine += four(i, n);
  (void)block_scan(mine, scan_ws, total);
  if (threadIdx.x == 0) *sums = total;
  cluster.sync();
  unsigned long long before = 0, all = 0;
  for (int r = 0; r < ranks; ++r) {
    const unsigned long long n = *cluster.map_shared_rank(sums, r);
    if (r < rank) before += n;
    all += n;
  }
  for (int i0 = w0; i0 < w1; i0 += 4 * blockDim.x) {
    const int i = i0 + 4 * threadIdx.x;
    __syncthreads();
    const unsigned long long sum = four(i, n);
    unsigned long long at = before + block_scan(sum, scan_ws, total);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (i + e < w1) a.before[word_at(i) + e] = static_cast<int32_t>(i + e <= cut ? at & 0xffffffffu : at >> 32);
      at += n[e];
    }
    before += total;
  }
  if (rank == 0 && threadIdx.x == 0) {
    const int targets = static_cast<int>(all & 0xffffffffu), movers = static_cast<int>(all >> 32);
    const bool done = movers <= targets && movers <= a.max_copies;
    a.state->movers = movers;
    a.state->targets = targets;
    a.state->done = done;
    *a.done = done;
    *a.copy_count = done ? movers : 0;
    if (done) *a.free_count = targets - movers;
  }
  cluster.sync();  // (no block ends while another reads its sums)
}

template <bool SAME>
__device__ __forceinline__ void compact_lists(const BlocksCompactArgs& a, long long me, long long threads) {
  const int movers = passed<SAME>(&a.state->movers), targets = passed<SAME>(&a.state->targets);
  if (passed<SAME>(&a.state->done) == 0) return;
  const int lane = threadIdx.x & 31, words = (a.num_blocks + 31) / 32;
  const uint32_t below = (1u << lane) - 1u;
  for (long long i = me >> 5; i < words; i += threads >> 5) {
    const uint32_t word = passed<SAME>(a.bits + word_at(static_cast<int>(i))), to = target_bits(a, i, word), from = mover_bits(a, i, word);
    const int x = 32 * static_cast<int>(i) + lane;
    if (to >> lane & 1u) {
      const int r = passed<SAME>(a.before + word_at(static_cast<int>(i))) + __popc(to & below);
      if (r < movers) a.copy_dst[r] = x;
      else a.free_blocks[targets - 1 - r] = x;
    }
    if (from >> lane & 1u) a.copy_src[mover_rank<SAME>(a, x, word)] = x;
  }
}

template <bool SAME>
__device__ __forceinline__ void compact_follow(const BlocksCompactArgs& a, long long me, long long threads) {
  const bool done = passed<SAME>(&a.state->done) != 0;
  // where block x is now
  auto now = [&](int x) -> int {
    if (!done || x < a.keep) return x;
    const uint32_t word = passed<SAME>(a.bits + word_at(x >> 5));
    return word >> (x & 31) & 1u ? x : passed<SAME>(a.copy_dst + mover_rank<SAME>(a, x, word));
  };
  for (long long x = me; x < a.num_blocks; x += threads) {
    const int to = now(static_cast<int>(x));
    a.moved_to[x] = to;
    if (to != x) {
      a.shares[to] = a.shares[x];
      a.shares[x] = 0;
    }
  }
  if (!done) return;
  // table rows: a warp takes 128 entries of a row at a time
  const int lane = threadIdx.x & 31, chunks = (a.max_blocks + 127) / 128;
  for (long long item = me >> 5; item < static_cast<long long>(a.batch) * chunks; item += threads >> 5) {
    const int b = static_cast<int>(item / chunks), c0 = static_cast<int>(item % chunks) * 128;
    const int held = min(max(a.n_held[b], 0), a.max_blocks);
    if (c0 >= held) continue;
    int32_t* row = a.block_table + static_cast<long long>(b) * a.max_blocks;
    int x[4], to[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = c0 + 32 * e + lane < held ? row[c0 + 32 * e + lane] : -1;
#pragma unroll
    for (int e = 0; e < 4; ++e) to[e] = x[e] >= a.keep && x[e] < a.num_blocks ? now(x[e]) : x[e];
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (to[e] != x[e]) row[c0 + 32 * e + lane] = to[e];
  }
}

// Each launch but the last lets the next one in at once, which waits for it.
__device__ __forceinline__ void compact_begin() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ long long grid_thread() { return static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; }
__device__ __forceinline__ long long grid_threads() { return static_cast<long long>(gridDim.x) * blockDim.x; }

__global__ void __launch_bounds__(kCompactThreads) compact_clear_kernel(const BlocksCompactArgs a) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  for (long long i = grid_thread(); i < (a.num_blocks + 31) / 32; i += grid_threads()) a.bits[word_at(static_cast<int>(i))] = 0u;
}
__global__ void __launch_bounds__(kCompactThreads) compact_mark_kernel(const BlocksCompactArgs a) {
  compact_begin();
  compact_mark(a, grid_thread(), grid_threads());
}
__global__ void __launch_bounds__(1024) compact_rank_kernel(const BlocksCompactArgs a) {
  __shared__ unsigned long long scan_ws[32], sums_s;
  compact_begin();
  compact_rank(a, scan_ws, &sums_s);
}
__global__ void __launch_bounds__(kCompactThreads) compact_lists_kernel(const BlocksCompactArgs a) {
  compact_begin();
  compact_lists<false>(a, grid_thread(), grid_threads());
}
__global__ void __launch_bounds__(kCompactThreads) compact_follow_kernel(const BlocksCompactArgs a) {
  // (the last launch: what comes behind it may read the tables before it waits, so it is not let in early)
  asm volatile("griddepcontrol.wait;" ::: "memory");
  compact_follow<false>(a, grid_thread(), grid_threads());
}
// Small pools: all of it in one cluster.
__global__ void __launch_bounds__(1024) compact_cluster_kernel(const BlocksCompactArgs a) {
  __shared__ unsigned long long scan_ws[32], sums_s;
  cg::cluster_group cluster = cg::this_cluster();
  for (long long i = grid_thread(); i < (a.num_blocks + 31) / 32; i += grid_threads()) a.bits[word_at(static_cast<int>(i))] = 0u;
  cluster.sync();
  compact_mark(a, grid_thread(), grid_threads());
  cluster.sync();
  compact_rank(a, scan_ws, &sums_s);
  compact_lists<true>(a, grid_thread(), grid_threads());
  cluster.sync();
  compact_follow<true>(a, grid_thread(), grid_threads());
}

int blocks_for(long long items, int per_block, int per_sm) {
  const long long want = (items + per_block - 1) / per_block, full = static_cast<long long>(per_sm) * device_sm_count();
  return static_cast<int>(want < 1 ? 1 : want < full ? want : full);
}

// One cluster of `ranks` blocks (8 is the portable most); ranks 0: `blocks` blocks without clusters. `early`: it may start
// while the launch before runs, for which it waits itself.
template <class Args>
cudaError_t launch(void (*kern)(Args), const Args& a, int ranks, int blocks, int threads, int smem, bool early, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(ranks > 0 ? ranks : blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 0;
  if (ranks > 0) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = ranks;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (early) {
    attr[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_blocks_fork(const BlocksForkArgs& a, cudaStream_t s) {
  const int groups = a.batch / a.width;
  const int smem = kForkWarps * a.width * 32 * static_cast<int>(sizeof(int));  // 32 KB at the widest
  const long long spans = (static_cast<long long>(a.max_blocks) + 32 * kForkWarps - 1) / (32 * kForkWarps);
  const long long room = (8ll * device_sm_count() + groups - 1) / groups;
  fork_entries_kernel<<<dim3(groups, static_cast<unsigned>(spans < room ? spans : room)), 32 * kForkWarps, smem, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int words = (a.num_blocks + 31) / 32;
  static_assert(2 * kSpecMaxBatch * sizeof(int) <= 48 * 1024, "no more shared memory than a kernel has without asking");
  // (8 requests of 4 sequences, a pool of 64K blocks: 10.2 us with one block, 10.2 to 12.3 with 8; of 1M 32.8 and 14.3)
  return launch(fork_tails_kernel, a, words <= 4096 ? 1 : 8, 0, 1024, 2 * a.batch * static_cast<int>(sizeof(int)), true, s);
}

cudaError_t launch_blocks_copy(const BlocksCopyArgs& a, cudaStream_t s) {
  const long long items = static_cast<long long>(a.n_pairs) * a.first_piece[a.n_buffers];
  blocks_copy_kernel<<<blocks_for(items, kCopyThreads / 32, 4), kCopyThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_blocks_compact(const BlocksCompactArgs& a, cudaStream_t s) {
  const int words = (a.num_blocks + 31) / 32;
  const long long entries = static_cast<long long>(a.batch) * a.max_blocks;
  // (one launch or five, with the tables put back before it: 4096 blocks 16.5 us both on the device, 20 and 29 from the
  // host; 16384 blocks 18.6 both; 65536 blocks 33 and 25)
  if (a.num_blocks <= 16384 && entries <= 65536) return launch(compact_cluster_kernel, a, 8, 0, 1024, 0, false, s);
  auto grid = [&](long long items, int per_thread) { return blocks_for(items, per_thread * kCompactThreads, 8); };
  cudaError_t e = launch(compact_clear_kernel, a, 0, grid(words, 1), kCompactThreads, 0, false, s);
  if (e == cudaSuccess) e = launch(compact_mark_kernel, a, 0, grid(a.num_blocks, 4), kCompactThreads, 0, true, s);
  if (e == cudaSuccess) e = launch(compact_rank_kernel, a, 8, 0, 1024, 0, true, s);
  if (e == cudaSuccess) e = launch(compact_lists_kernel, a, 0, grid(32ll * words, 2), kCompactThreads, 0, true, s);
  if (e == cudaSuccess)
    e = launch(compact_follow_kernel, a, 0, grid(entries > a.num_blocks ? entries : a.num_blocks, 4), kCompactThreads, 0, true, s);
  return e;
}

}  // namespace kvq
