// Serving-step kernels of the paged caches for sm_103a: block tables and slot
// maps from request lengths, the append of new tokens into the FP8 pools by
// slot, and the move of an accepted path (kvq_spec.h).
#include <climits>
#include <cooperative_groups.h>

#include "block_scan.cuh"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "spec_internal.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kBlock = 16;  // tokens of an FP8 pool block

// The last index b in [0, n) with start(b) <= i, start ascending and start(0) <= i.
template <class F>
__device__ __forceinline__ int owner_of(int n, int i, F start) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start(mid) <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

// ---------------------------------------------------------------------------
// Block tables. One cluster of thread blocks: each scans all requests (a few
// words each) into its own shared memory, so every block knows each request's
// place among the released and the granted entries; the entries themselves are
// spread over all threads of the cluster. The cluster barrier between the
// releases and the growth, in place of a second launch, lets the growth take
// blocks that this call released.
//   A = blocks free after the releases; released entry r goes to stack place
//   A-1-r, granted entry i comes from place A-1-i.
// Bound by latency: 3.1 us for 8 requests with nothing to change, 8 us for 135
// thousand changed entries (scan, scattered table rows, the barrier).
// ---------------------------------------------------------------------------
// SHARED: a request that would release an entry whose block others hold is
// refused; its warp looks through those entries together, one such request after
// another (512 requests that all shrink: 16 us with the growth that undoes it in
// turn, 8 without; nothing to release: 0.5 us more, the second barrier).
template <bool SHARED>
__global__ void __launch_bounds__(1024) blocks_resize_kernel(BlocksResizeArgs a) {
  extern __shared__ int sm[];
  int* held_s = sm;                       // [B] blocks held before
  int* want_s = held_s + a.batch;         // [B] blocks held after the shrink or, if granted, the growth
  int* drop_s = want_s + a.batch;         // [B] released entries of the requests before
  int* ask_s = drop_s + a.batch;          // [B] growth asked for by the requests before
  __shared__ unsigned long long scan_ws[32];
  __shared__ int grown_s;                 // blocks granted in all
  cg::cluster_group cluster = cg::this_cluster();
  const int n_free = min(max(*a.free_count, 0), a.num_blocks);

  // low half: released entries, high half: growth asked for (each sum < 2^31)
  unsigned long long carry = 0;
  for (int b0 = 0; b0 < a.batch; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int held = 0, need = 0;
    if (b < a.batch) {
      held = min(max(a.n_held[b], 0), a.max_blocks);
      const int t = a.target_tokens[b];
      const long long n = t < 0 ? -1 : (static_cast<long long>(t) + a.block_tokens - 1) / a.block_tokens;
      need = (n < 0 || n > a.max_blocks) ? -1 : static_cast<int>(n);
    }
    if constexpr (SHARED) {
      const int lane = threadIdx.x & 31;
      for (unsigned who = __ballot_sync(0xffffffffu, need >= 0 && need < held); who != 0; who &= who - 1) {
        const int l = __ffs(who) - 1;
        const int32_t* row = a.block_table + static_cast<long long>(__shfl_sync(0xffffffffu, b, l)) * a.max_blocks;
        const unsigned from = __shfl_sync(0xffffffffu, need, l), to = __shfl_sync(0xffffffffu, held, l);
        bool others = false;
        for (unsigned j = from + lane; j < to; j += 32) {
          const int x = row[j];
          if (x >= 0 && x < a.num_blocks) others |= a.shares[x] > 0;
        }
        if (__any_sync(0xffffffffu, others) && lane == l) need = -1;
      }
    }
    const int now = need < 0 ? held : need;
    const unsigned long long v = static_cast<unsigned long long>(max(held - now, 0)) |
                                 (static_cast<unsigned long long>(max(now - held, 0)) << 32);
    unsigned long long total;
    const unsigned long long before = carry + block_scan(v, scan_ws, total);
    if (b < a.batch) {
      held_s[b] = held;
      want_s[b] = need;  // -1: refused
      drop_s[b] = static_cast<int>(before & 0xffffffffu);
      ask_s[b] = static_cast<int>(before >> 32);
    }
    carry += total;
    __syncthreads();
  }
  if constexpr (SHARED) cluster.sync();  // (no block releases entries that another looks through)
  const int released = static_cast<int>(carry & 0xffffffffu);
  // (free list and tables that agree never hold more than num_blocks blocks)
  const int top = static_cast<int>(min(static_cast<long long>(n_free) + released, static_cast<long long>(a.num_blocks)));
  if (threadIdx.x == 0) grown_s = 0;
  __syncthreads();
  for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
    const int grow = max(want_s[b] - held_s[b], 0);
    if (grow > 0) {
      if (static_cast<long long>(ask_s[b]) + grow <= top)
        atomicMax(&grown_s, ask_s[b] + grow);
      else
        want_s[b] = -1;
    }
  }
  __syncthreads();
  const int grown = grown_s;

  const int threads = blockDim.x * cluster.num_blocks(), me = cluster.block_rank() * blockDim.x + threadIdx.x;
  // A warp takes 128 neighbouring entries, a lane four of them 32 apart: their reads are in flight together.
  // (entries count up to 2^31 - 1: unsigned, so that the last step passes that number without wrapping)
  const unsigned first = (me & ~31) * 4 + (me & 31), n_drop = released, n_grow = grown;
  for (unsigned i0 = first; i0 < n_drop; i0 += 4 * threads) {
    int b = owner_of(a.batch, static_cast<int>(i0), [&](int m) { return drop_s[m]; });
    int32_t* entry[4];
    int32_t block[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      entry[e] = nullptr;
      const unsigned i = i0 + 32 * e;
      if (i < n_drop) {
        while (b + 1 < a.batch && static_cast<int>(i) >= drop_s[b + 1]) ++b;
        entry[e] = a.block_table + static_cast<long long>(b) * a.max_blocks + want_s[b] + (static_cast<int>(i) - drop_s[b]);
        block[e] = *entry[e];
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (entry[e] == nullptr) continue;
      const int place = top - 1 - static_cast<int>(i0 + 32 * e);
      if (place >= 0) a.free_blocks[place] = block[e];
      *entry[e] = -1;
    }
  }
  cluster.sync();
  for (unsigned i0 = first; i0 < n_grow; i0 += 4 * threads) {
    // growth is granted in order until it is refused for good: what the granted requests asked for is their place
    int b = owner_of(a.batch, static_cast<int>(i0), [&](int m) { return min(ask_s[m], grown); });
    int32_t* entry[4];
    int32_t block[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      entry[e] = nullptr;
      const unsigned i = i0 + 32 * e;
      if (i < n_grow) {
        while (b + 1 < a.batch && static_cast<int>(i) >= ask_s[b + 1]) ++b;
        entry[e] = a.block_table + static_cast<long long>(b) * a.max_blocks + held_s[b] + (static_cast<int>(i) - ask_s[b]);
        block[e] = __ldcg(a.free_blocks + (top - 1 - static_cast<int>(i)));
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (entry[e] != nullptr) *entry[e] = block[e];
  }
  // every block has read the old counts before the barrier
  if (cluster.block_rank() == 0) {
    for (int b = threadIdx.x; b < a.batch; b += blockDim.x) {
      const int want = want_s[b];
      if (want >= 0) a.n_held[b] = want;
      if (a.granted != nullptr) a.granted[b] = want >= 0;
    }
    if (threadIdx.x == 0) *a.free_count = top - grown;
  }
}

// ---------------------------------------------------------------------------
// Slot map: every thread block scans the requests' new lengths itself (no
// second launch), then takes its share of the rows, four to a thread. 16 bytes
// are written a row: 2.16 million rows in 10.7 us, 3.2 TB/s (the output stays in
// L2); a few rows in 3.7 us, the scan and two dependent reads.
// ---------------------------------------------------------------------------
constexpr int kMapThreads = 256;

__global__ void __launch_bounds__(kMapThreads) slot_map_kernel(SlotMapArgs a) {
  __shared__ int off_s[kSpecMaxBatch + 1];
  __shared__ unsigned long long scan_ws[32];
  unsigned long long carry = 0;
  const unsigned long long cap = static_cast<unsigned long long>(a.n_rows);
  for (int b0 = 0; b0 < a.batch; b0 += kMapThreads) {
    const int b = b0 + threadIdx.x;
    unsigned long long total;
    const unsigned long long before =
        carry + block_scan(b < a.batch ? static_cast<unsigned long long>(max(a.new_lens[b], 0)) : 0ull, scan_ws, total);
    if (b < a.batch) off_s[b] = static_cast<int>(before < cap ? before : cap);
    carry += total;
    __syncthreads();
  }
  const int n = static_cast<int>(carry < cap ? carry : cap);
  if (threadIdx.x == 0) off_s[a.batch] = n;
  __syncthreads();
  if (blockIdx.x == 0)
    for (int b = threadIdx.x; b <= a.batch; b += kMapThreads) a.offsets[b] = off_s[b];

  const int lane = threadIdx.x & 31;
  // (64 bits: the last step may pass 2^31)
  for (long long first = 4ll * (blockIdx.x * kMapThreads + (threadIdx.x & ~31)); first < a.n_rows;
       first += 4ll * gridDim.x * kMapThreads) {
    const int i0 = static_cast<int>(min(first + 4 * lane, static_cast<long long>(a.n_rows)));
    long long slot[4];
    int seq[4], pos[4];
    int b = i0 < n ? owner_of(a.batch, i0, [&](int m) { return off_s[m]; }) : 0;
    int next = i0 < n ? off_s[b + 1] : 0, j = 0, block = -1;
    long long p = 0;
    int row = 0;  // p's row in its block
    bool fresh = true;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      slot[e] = seq[e] = pos[e] = -1;
      if (e < n - i0) {
        const int i = i0 + e;
        while (i >= next) {
          next = off_s[++b + 1];
          fresh = true;
        }
        p = fresh ? static_cast<long long>(a.seq_lens[b]) + (i - off_s[b]) : p + 1;
        if (p < 0 || p > INT_MAX) {  // outside every table
          block = -1;
        } else if (fresh || p == 0 || ++row == a.block_tokens) {
          // the one division of most threads; behind a position outside, 0 begins the table, behind a block the next one
          j = fresh ? static_cast<int>(p) / a.block_tokens : p == 0 ? 0 : j + 1;
          row = fresh ? static_cast<int>(p) - j * a.block_tokens : 0;
          block = j < a.max_blocks ? a.block_table[static_cast<long long>(b) * a.max_blocks + j] : -1;
        }
        fresh = false;
        seq[e] = b;
        pos[e] = p <= INT_MAX ? static_cast<int>(p) : -1;
        if (block >= 0 && block < a.num_blocks) slot[e] = static_cast<long long>(block) * a.block_tokens + row;
      }
    }
    if (first + 127 < a.n_rows) {
      // slots change lanes so that each store covers 512 neighbouring bytes (a thread's own 32 would be written as
      // two halves of its sector: 2.2 million rows in 11.9 us, so in 10.9)
      longlong2* s2 = reinterpret_cast<longlong2*>(a.slots + first);
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int from = 16 * half + (lane >> 1);
        const long long lo0 = __shfl_sync(0xffffffffu, slot[0], from), lo1 = __shfl_sync(0xffffffffu, slot[1], from);
        const long long hi0 = __shfl_sync(0xffffffffu, slot[2], from), hi1 = __shfl_sync(0xffffffffu, slot[3], from);
        s2[32 * half + lane] = (lane & 1) ? make_longlong2(hi0, hi1) : make_longlong2(lo0, lo1);
      }
      if (a.seq_ids) *reinterpret_cast<int4*>(a.seq_ids + i0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      if (a.positions) *reinterpret_cast<int4*>(a.positions + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (e >= a.n_rows - i0) break;
        a.slots[i0 + e] = slot[e];
        if (a.seq_ids) a.seq_ids[i0 + e] = seq[e];
        if (a.positions) a.positions[i0 + e] = pos[e];
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Append. Tokens that follow one another in the call and in one block form a
// run; a warp takes (run, head, K or V): it stages the run's rows in shared
// memory and writes the block's fragment-ordered bytes, whole 16-byte units
// where the run covers them (a key unit is 16 channels of one token, a value
// unit 4 tokens of 4 channels). A value row alone is single bytes, each in a
// 32-byte sector of its own, so writing whole runs at once is what keeps long
// appends at the memory's rate. 65536 tokens (8 heads, D = 128, rows of a fused
// projection) in 73.8 us, 80 % of the measured copy rate; 2112 tokens in runs of
// 33 in 6.1 us; 8 tokens in 3.6 us, one chain of dependent reads.
// ---------------------------------------------------------------------------
constexpr int kAppendWarps = 4;

template <int D, int FMT, int ROLE, int MODE>
__device__ __forceinline__ void append_run(const __half* xs, int r0, int n, float scale, uint8_t* block) {
  constexpr int RS = D + 8;
  const int lane = threadIdx.x & 31, gg = lane >> 2, tg = lane & 3;
  const float y = (MODE == 0) ? 0.0f : __frcp_rn(scale);
  auto in_run = [&](int tok) { return tok >= r0 && tok < r0 + n; };
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    uint8_t* unit = block + (c * 32 + lane) * 16;
    if constexpr (ROLE == 0) {
      const int nt = c / (D / 64), kh = c % (D / 64), tok = 8 * nt + gg;
      if (!in_run(tok)) continue;
      uint32_t w[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {  // word e: channels 64kh + 16e + 4tg .. +3
        const uint2 x = *reinterpret_cast<const uint2*>(xs + tok * RS + 64 * kh + 16 * e + 4 * tg);
        const float2 lo = scaled_pair<MODE>(x.x, scale, y), hi = scaled_pair<MODE>(x.y, scale, y);
        w[e] = f32x2_to_fp8x2<FMT>(lo.x, lo.y) | (static_cast<uint32_t>(f32x2_to_fp8x2<FMT>(hi.x, hi.y)) << 16);
      }
      *reinterpret_cast<uint4*>(unit) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      uint32_t pr[8];  // pair 2e + r: tokens 8r + 2tg, +1 of channel 8 (4c + e) + gg
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t t4[4];
        ldsm_x4_trans(t4, xs + (8 * r + (lane & 7)) * RS + 8 * (4 * c + (lane >> 3)));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 q = scaled_pair<MODE>(t4[e], scale, y);
          pr[2 * e + r] = f32x2_to_fp8x2<FMT>(q.x, q.y);
        }
      }
      const bool in[4] = {in_run(2 * tg), in_run(2 * tg + 1), in_run(8 + 2 * tg), in_run(9 + 2 * tg)};
      if (in[0] && in[1] && in[2] && in[3]) {
        *reinterpret_cast<uint4*>(unit) = make_uint4(pr[0] | (pr[1] << 16), pr[2] | (pr[3] << 16),
                                                     pr[4] | (pr[5] << 16), pr[6] | (pr[7] << 16));
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          if (in[2 * r] && in[2 * r + 1]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) *reinterpret_cast<uint16_t*>(unit + 4 * e + 2 * r) = static_cast<uint16_t>(pr[2 * e + r]);
          } else if (in[2 * r]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) unit[4 * e + 2 * r] = static_cast<uint8_t>(pr[2 * e + r]);
          } else if (in[2 * r + 1]) {
#pragma unroll
            for (int e = 0; e < 4; ++e) unit[4 * e + 2 * r + 1] = static_cast<uint8_t>(pr[2 * e + r] >> 8);
          }
        }
      }
    }
  }
}

template <int D, int FMT, int ROLE>
__device__ __forceinline__ void append_role(const Fp8AppendArgs& a, __half* xs, long long tok0, int r0, int n, int h,
                                            long long blk) {
  constexpr int RS = D + 8;
  const int lane = threadIdx.x & 31;
  const uint16_t* src = (ROLE == 0 ? a.k_new : a.v_new) + static_cast<long long>(h) * D;
  const long long stride = ROLE == 0 ? a.k_stride : a.v_stride;
  for (int i = lane; i < n * (D / 8); i += 32) {
    const int t = i / (D / 8), c8 = i % (D / 8);
    cp_async16(xs + (r0 + t) * RS + 8 * c8, src + (tok0 + t) * stride + 8 * c8);
  }
  cp_async_commit();
  const float scale = (ROLE == 0 ? a.k_scale : a.v_scale)[a.per_head ? h : 0];
  uint8_t* block = (ROLE == 0 ? a.k_pool : a.v_pool) + (blk * a.kv_heads + h) * (kBlock * D);
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  if (scale >= 0x1p-96f && scale <= 0x1p96f)
    append_run<D, FMT, ROLE, 1>(xs, r0, n, scale, block);
  else
    append_run<D, FMT, ROLE, 0>(xs, r0, n, scale, block);
  __syncwarp();
}

// Warp (x, y): tokens [x * window, + window) and the (head, role) items y, y + ny, ...
template <int D, int FMT>
__global__ void __launch_bounds__(32 * kAppendWarps) fp8_append_kernel(Fp8AppendArgs a, int window, int item_warps) {
  __shared__ __align__(16) __half bufs[kAppendWarps][kBlock * (D + 8)];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long id = static_cast<long long>(blockIdx.x) * kAppendWarps + warp;
  const long long i0 = id / item_warps * window;
  if (i0 >= a.n_tokens) return;
  const int item0 = static_cast<int>(id % item_warps);
  __half* xs = bufs[warp];
  const long long n_slots = static_cast<long long>(a.num_blocks) * kBlock;
  // this lane's token (of the window and of the run that may reach beyond it) and the one before
  const long long i = i0 + lane;
  const long long slot = i < a.n_tokens ? a.slots[i] : -1;
  long long prev = __shfl_up_sync(0xffffffffu, slot, 1);
  if (lane == 0) prev = i0 > 0 ? a.slots[i0 - 1] : -1;
  const bool ok = slot >= 0 && slot < n_slots;
  const bool follows = ok && prev >= 0 && slot == prev + 1 && (slot & (kBlock - 1)) != 0;
  const uint32_t cont = __ballot_sync(0xffffffffu, follows);
  uint32_t leaders = __ballot_sync(0xffffffffu, ok && !follows && lane < window);
  while (leaders != 0) {
    const int l = __ffs(leaders) - 1;
    leaders &= leaders - 1;
    const long long s = __shfl_sync(0xffffffffu, slot, l);
    const uint32_t after = l < 31 ? cont >> (l + 1) : 0u;
    const int n = __ffs(~after);  // the leader and the tokens that follow it
    const int r0 = static_cast<int>(s & (kBlock - 1));
    for (int it = item0; it < 2 * a.kv_heads; it += item_warps) {
      if (it < a.kv_heads)
        append_role<D, FMT, 0>(a, xs, i0 + l, r0, n, it, s / kBlock);
      else
        append_role<D, FMT, 1>(a, xs, i0 + l, r0, n, it - a.kv_heads, s / kBlock);
    }
  }
}

// ---------------------------------------------------------------------------
// Accept. One thread block per request. A path ascends, so row i's place seq_len
// + i is at or before its source and before every later source: moving rows in
// order never reads what has been overwritten.
//   keys  : a thread owns one column (a 16-byte unit of one head) of every row
//   values: a unit holds 4 tokens of 4 channels, so a row alone is 4 single
//           bytes a unit; a warp takes one 512-byte chunk (32 channels of a head,
//           16 tokens) of a place block at a time, each lane gathers its unit's
//           bytes from the units of their sources (of the same channels, so the
//           same warp's) and writes the unit whole. Byte by byte this took 18 us
//           for 256 requests x 8 rows: 2.1 million writes of parts of sectors.
// One request: 4.5 us, a chain of dependent reads (length, path, table, rows).
// 256 requests x 12 rows: 14.2 us; a value row touches all 64 sectors of its
// block and head, 16 times its bytes, and that is what is moved.
// ---------------------------------------------------------------------------
constexpr int kAcceptBatch = 8;

template <int D>
__global__ void __launch_bounds__(512) fp8_accept_kernel(Fp8AcceptArgs a) {
  // of row i: source block (-1: stays), place block, source row | place row << 8
  __shared__ int src_blk[kTreeMax], dst_blk[kTreeMax], rows[kTreeMax];
  const int b = blockIdx.x;
  const int len = a.seq_lens[b];
  const int n = min(max(a.n_accepted[b], 0), a.path_len);
  const int32_t* table = a.block_table + static_cast<long long>(b) * a.max_blocks;
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int node = a.path[static_cast<long long>(b) * a.path_len + i];
    int sb = -1, db = -1, r = 0;
    const long long from = static_cast<long long>(len) + node, to = static_cast<long long>(len) + i;
    if (len >= 0 && node >= 0 && node < kTreeMax && node != i && from / kBlock < a.max_blocks && to / kBlock < a.max_blocks) {
      sb = table[from / kBlock];
      db = table[to / kBlock];
      if (sb >= a.num_blocks || db < 0 || db >= a.num_blocks) sb = -1;
      r = static_cast<int>(from % kBlock) | (static_cast<int>(to % kBlock) << 8);
    }
    src_blk[i] = sb;
    dst_blk[i] = db;
    rows[i] = r;
  }
  __syncthreads();
  // (this block alone reads seq_lens[b]; a length near 2^31 wraps)
  if (threadIdx.x == 0) a.new_lens[b] = static_cast<int>(static_cast<unsigned>(len) + n);
  if (len < 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  constexpr int KU = D / 16, CH = D / 32;
  const long long end = min(static_cast<long long>(len) + n, static_cast<long long>(a.max_blocks) * kBlock);
  const int k_tasks = (a.kv_heads * KU + 31) / 32, tasks = k_tasks + a.kv_heads * CH;
  for (int task = warp; task < tasks; task += warps) {
    if (task < k_tasks) {
      const int col = task * 32 + lane, h = col / KU, u = col % KU;
      if (h >= a.kv_heads) continue;
      auto unit = [&](int blk, int t) {
        return reinterpret_cast<uint4*>(a.k_pool + (static_cast<long long>(blk) * a.kv_heads + h) * (kBlock * D) +
                                        ((t / 8 * (D / 64) + u / 4) * 32 + 4 * (t % 8) + u % 4) * 16);
      };
      for (int i0 = 0; i0 < n; i0 += kAcceptBatch) {
        uint4 v[kAcceptBatch];
#pragma unroll
        for (int e = 0; e < kAcceptBatch; ++e)
          if (i0 + e < n && src_blk[i0 + e] >= 0) v[e] = *unit(src_blk[i0 + e], rows[i0 + e] & 255);
#pragma unroll
        for (int e = 0; e < kAcceptBatch; ++e)
          if (i0 + e < n && src_blk[i0 + e] >= 0) *unit(dst_blk[i0 + e], rows[i0 + e] >> 8) = v[e];
      }
    } else {
      const int h = (task - k_tasks) / CH, c = (task - k_tasks) % CH, tig = lane & 3;
      auto unit = [&](int blk, int in_chunk) {
        return reinterpret_cast<uint4*>(a.v_pool + (static_cast<long long>(blk) * a.kv_heads + h) * (kBlock * D) +
                                        (c * 32 + in_chunk) * 16);
      };
      // place blocks in order: what a later one's rows come from lies behind every place of an earlier one
      for (long long p0 = len / kBlock * kBlock; p0 < end; p0 += kBlock) {
        uint4 src[4];
        int shift[4], place = -1;
#pragma unroll
        for (int e = 0; e < 4; ++e) {  // the unit's tokens: byte e of each word is token 8 (e / 2) + 2 tig + e % 2
          const int i = static_cast<int>(p0 - len) + 8 * (e >> 1) + 2 * tig + (e & 1);
          shift[e] = -1;
          if (i >= 0 && i < n && src_blk[i] >= 0) {
            const int from = rows[i] & 255;
            shift[e] = 8 * (from / 8 * 2 + from % 2);
            src[e] = *unit(src_blk[i], (lane & ~3) + from % 8 / 2);
            place = dst_blk[i];
          }
        }
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (place >= 0) w = *unit(place, lane);
        __syncwarp();  // every lane has read before one writes
        if (place >= 0) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (shift[e] < 0) continue;
            const uint32_t sel = 0x3210u ^ ((e ^ 4u) << (4 * e));  // byte e from the second word's byte 0
            w.x = __byte_perm(w.x, src[e].x >> shift[e], sel);
            w.y = __byte_perm(w.y, src[e].y >> shift[e], sel);
            w.z = __byte_perm(w.z, src[e].z >> shift[e], sel);
            w.w = __byte_perm(w.w, src[e].w >> shift[e], sel);
          }
          *unit(place, lane) = w;
        }
        __syncwarp();
      }
    }
  }
}

template <bool SHARED>
cudaError_t launch_resize(const BlocksResizeArgs& a, cudaStream_t s) {
  auto kern = blocks_resize_kernel<SHARED>;
  const int smem = 4 * a.batch * static_cast<int>(sizeof(int));
  static SharedMemoryOnce once;
  cudaError_t e = once.set(kern, 4 * kSpecMaxBatch * static_cast<int>(sizeof(int)));
  if (e != cudaSuccess) return e;
  const bool small = static_cast<long long>(a.batch) * a.max_blocks <= 16384;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  // tables of more than 16K entries: 16 blocks (7.4 us for 135K changed entries; 8, the portable most, take 10.5)
  attr.val.clusterDim.x = small ? 1 : 16;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(attr.val.clusterDim.x);
  cfg.blockDim = dim3(small ? 256 : 1024);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (!small) {
    static std::atomic<int> fits[SharedMemoryOnce::kDevices] = {};  // 16 blocks: 1 they do, -1 they do not
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int f = dev < SharedMemoryOnce::kDevices ? fits[dev].load(std::memory_order_relaxed) : 0;
    if (f == 0) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      cudaLaunchConfig_t most = cfg;
      most.dynamicSmemBytes = 4 * kSpecMaxBatch * sizeof(int);
      int clusters = 0;
      f = cudaOccupancyMaxActiveClusters(&clusters, kern, &most) == cudaSuccess && clusters > 0 ? 1 : -1;
      if (f < 0) (void)cudaGetLastError();
      if (dev < SharedMemoryOnce::kDevices) fits[dev].store(f, std::memory_order_relaxed);
    }
    if (f < 0) {
      attr.val.clusterDim.x = 8;
      cfg.gridDim = dim3(8);
    }
  }
  e = cudaLaunchKernelEx(&cfg, kern, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_blocks_resize(const BlocksResizeArgs& a, cudaStream_t s) {
  return a.shares != nullptr ? launch_resize<true>(a, s) : launch_resize<false>(a, s);
}

cudaError_t launch_slot_map(const SlotMapArgs& a, cudaStream_t s) {
  const long long want = (static_cast<long long>(a.n_rows) + 4 * kMapThreads - 1) / (4 * kMapThreads);
  const long long full = 4LL * device_sm_count();
  slot_map_kernel<<<static_cast<int>(want < full ? want : full), kMapThreads, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_fp8_append(const Fp8AppendArgs& a, cudaStream_t s) {
  // One warp per (16-token window, head, role) when those fill the GPU; with
  // fewer tokens one warp per (token, head, role), of which only the first
  // token of a run works.
  const long long items = 2LL * a.kv_heads;
  const int window = static_cast<long long>(a.n_tokens) * items > 64LL * device_sm_count() ? kBlock : 1;
  const long long windows = (static_cast<long long>(a.n_tokens) + window - 1) / window;
  const long long want = (windows * items + kAppendWarps - 1) / kAppendWarps;
  if (want > 0x7fffffffLL) return cudaErrorInvalidValue;
  const int grid = static_cast<int>(want);
  switch (a.head_dim * 10 + a.fmt) {
    case 1280: fp8_append_kernel<128, 0><<<grid, 32 * kAppendWarps, 0, s>>>(a, window, static_cast<int>(items)); break;
    case 1281: fp8_append_kernel<128, 1><<<grid, 32 * kAppendWarps, 0, s>>>(a, window, static_cast<int>(items)); break;
    case 640: fp8_append_kernel<64, 0><<<grid, 32 * kAppendWarps, 0, s>>>(a, window, static_cast<int>(items)); break;
    case 641: fp8_append_kernel<64, 1><<<grid, 32 * kAppendWarps, 0, s>>>(a, window, static_cast<int>(items)); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_fp8_accept(const Fp8AcceptArgs& a, cudaStream_t s) {
  const long long tasks = (static_cast<long long>(a.kv_heads) * (a.head_dim / 16) + 31) / 32 +
                          static_cast<long long>(a.kv_heads) * (a.head_dim / 32);
  const int threads = static_cast<int>(32 * (tasks < 16 ? tasks : 16));
  if (a.head_dim == 128)
    fp8_accept_kernel<128><<<a.batch, threads, 0, s>>>(a);
  else
    fp8_accept_kernel<64><<<a.batch, threads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kvq
