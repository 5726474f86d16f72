// Group attention over shared blocks on the fifth-generation tensor cores
// (tcgen05), for groups with more query rows per kv head than one mma.sync tile.
//
// A thread block per SM walks its slice of (group, kv head, row tile) pairs in
// tiles of 64 tokens. The tensor core's 128 rows hold the query rows of a tile
// once, or those of a group with up to 64 of them twice: copy f of a row then has
// the weights of the f-th half of a tile's tokens and zeros elsewhere. The
// products cost what they did, each softmax thread has half of the work, and the
// copies are partial results like those of different thread blocks.
// Two streams take alternate token tiles, each with
// its own scores, weights and outputs, so that the tensor core works for one
// while the other one's softmax runs:
//   S = Q K^T : A = Q (fp16, exact) in tensor memory (WIDE: in shared memory),
//               B = the keys as fp16 in shared memory, 128 x 64 fp32 accumulators
//   O += P V  : A = P in tensor memory (fp16; WIDE, for fp32 output: and the
//               rounding's remainder), B = the values as fp16
// Tensor memory's 512 columns (D = 128): O 2 x 128, S 2 x 64, P 2 x 32 and Q 64,
// or with WIDE P 2 x 64 and no Q.
// Roles, operand orders and the lazily renewed maxima are those of tree
// attention's kernel: one warp copies pool blocks, four turn FP8 bytes into fp16
// operand tiles, three threads issue the MMAs, eight warps do the softmax, a
// thread per row (and copy).
//
// 4 x 8 sequences over 128K tokens (64 rows a kv head): 253 us, 4.3 TB/s. What
// bounds it is the loop through the four fp16 places: conversion (930 clocks),
// scores (600), softmax (1390) and products (1400) of a tile take some 4300 / 4
// clocks a tile with all of them at work; DRAM is at half its rate, the tensor core busy
// 38 % of the time. Shared memory has no fifth place at D = 128; with 6 and 8 at
// D = 64 the copies are what the conversion waits for. No faster: a second
// copying warp (277 us), a place handed on through shared memory (274), weights
// made before the wait for the products before (265).
// WIDE, by fp32 output: 347 us (1.37 times as long; 1.2 to 1.3 with 64 channels and
// up to 64 rows, 1.7 with 128 channels and rows): twice the value products and, with
// 128 channels, two places for the copies in place of four. With fp16 output one part leaves 2.24e-4
// of error against 64 bits there, of which the output's rounding is 2.05e-4.
#include "group_plan.cuh"
#include "tc_device.cuh"

namespace kvq {
namespace {

constexpr int kBlock = 16;
constexpr int kTile = 64;             // tokens of a tile (and of a work unit)
constexpr int kBufs = 4;              // fp16 tiles (keys and values)
constexpr float kBias = 7.0f;
constexpr float kMostSum = 32768.0f;  // of a tile's weights in a row: each is within fp16 then
constexpr int kThreads = 512;
constexpr int kLanes = kGroupTcRows;  // rows of the tensor core
// warps: 0-3 and 4-7 softmax of stream 0 and 1, 8-11 conversion, 12 copies, 13 the scores' MMAs, 14 and 15 the outputs'
// MMAs of stream 0 and 1
constexpr int kConvertWarp = 8, kCopyWarp = 12, kScoreWarp = 13, kOutputWarp = 14;
constexpr int kMaxStages = 6;

template <int D, bool WIDE>
struct TcPlan {
  static constexpr int STAGE = 2 * kTile * D;       // pool bytes of a tile: keys, then values
  static constexpr int TILE = kTile * D * 2;        // one fp16 tile of keys or values
  static constexpr int Q_TILE = WIDE ? kLanes * D * 2 : 0;
  // Both rings have an even number of places: the converting pairs take tiles of alternate parity, and so a place
  // always belongs to one pair, which sees each phase of its barriers.
  static constexpr int FIXED = kBufs * 2 * TILE + Q_TILE;
  static constexpr int FIT = (221184 - FIXED) / STAGE;  // 227 KB without what TcShared takes
  static constexpr int STAGES = (FIT < kMaxStages ? FIT : kMaxStages) & ~1;
  static_assert(STAGES >= 2, "room for the copies");
  static_assert(STAGES % 2 == 0 && kBufs % 2 == 0, "a place of a ring belongs to one converting pair");
  static constexpr int K_OFF = STAGES * STAGE, V_OFF = K_OFF + kBufs * TILE, Q_OFF = V_OFF + kBufs * TILE;
  static constexpr int BYTES = Q_OFF + Q_TILE;
  // tensor memory columns
  static constexpr int P_COLS = (WIDE ? 2 : 1) * kTile / 2;
  static constexpr int TM_O = 0, TM_S = 2 * D, TM_P = TM_S + 2 * kTile, TM_Q = TM_P + 2 * P_COLS;
  static_assert((WIDE ? TM_Q : TM_Q + D / 2) <= 512, "tensor memory");
};

struct TcShared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t ready[kBufs], free[kBufs];
  uint64_t qready[2], sready[2], sfree[2], pready[2], pdone[2], drain[3];
  unsigned long long plan[36];
  uint32_t tmem;
  int dead;
  float ml[2][kLanes][2];
  // the arguments, for functions out of line (a reference to a kernel's parameters is read from global memory there)
  GroupArgs args;
  // each warp's place in the slice: in shared memory, not in registers that the roles' loops need
  TreeSlice slice;
  GroupWalk walk[kThreads / 32];
};

// Token of column c of a tile.
__host__ __device__ constexpr int column_token(int c) {
  return (c & ~15) + 8 * ((c >> 1) & 1) + 2 * ((c >> 2) & 3) + (c & 1);
}

template <int D, int FMT, bool WIDE, int FOLD>
__global__ void __launch_bounds__(kThreads, 1) group_tc_kernel(const __grid_constant__ GroupArgs a) {
  using S = TcPlan<D, WIDE>;
  constexpr int R = kLanes / FOLD;          // query rows of a tile
  constexpr int COLS = kTile / FOLD;        // tokens of a tile that a softmax thread has
  constexpr int UPB = kTile / kBlock;       // pool blocks of a tile
  constexpr unsigned kStages = S::STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ TcShared sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform for the compiler too
  const int gq = a.q_heads / a.kv_heads;
  // the own pairs' kernel comes in where blocks of this one have left
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 2);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sh.ready[i], 2);
      mbar_init(&sh.free[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.qready[i], 4);
      mbar_init(&sh.sready[i], 1);
      mbar_init(&sh.sfree[i], 4);
      mbar_init(&sh.pready[i], 4);
      mbar_init(&sh.pdone[i], 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&sh.drain[i], 1);
    sh.dead = 0;
    sh.args = a;
    fence_mbar_init();
  }
  {
    // slices and cuts as tree attention's
    const TreeSlice s = tree_slice<R, kTile>(
        a, sh.plan, [](long long pair) { return static_cast<int>(min(max(pair, 2ll), 4ll)); },
        [](long long u) { return static_cast<int>(min(max(u, 4ll), 8ll)); });
    if (s.begin >= s.end) return;
    if (tid == 0) sh.slice = s;
    if (lane == 0) sh.walk[warp].start(s);
  }
  if (warp == kScoreWarp) {
    __syncwarp();
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* dead = &sh.dead;

  GroupWalk& walk = sh.walk[warp];
  const GroupSegment& seg = walk.seg;
  auto next_here = [&]() { return next_segment<R, kTile>(sh.args, sh.slice, walk); };
  // the warp's next segment: one lane finds it, all read it
  auto next = [&]() -> bool {
    __syncwarp();
    bool more = false;
    if (elect_one()) more = next_here();
    __syncwarp();  // (a vote alone does not order memory)
    return __any_sync(0xffffffffu, more);
  };

  if (warp == kCopyWarp) {
    // ---- copies: one thread issues those of a tile's blocks. (A copy from each of eight lanes at once is a loop over
    // the lanes of some 100 clocks a copy: 830 of a tile's 1020 clocks, which was what bounded the kernel.) ----
    unsigned n = 0;  // tiles issued
    bool ok = true;
    while (ok && next()) {
      const int nblk = tree_units(seg.r.len, kBlock);
      const int32_t* table = a.block_table + static_cast<long long>(seg.r.seq) * a.max_blocks + seg.r.block0;
      const long long head = static_cast<long long>(seg.h) * (kBlock * D), stride = static_cast<long long>(a.kv_heads) * (kBlock * D);
      const int u0 = seg.u0, u1 = seg.u1;
      // table entries come 32 at a time, a load ahead
      auto entries = [&](int j) -> int { return j + lane < nblk ? min(max(table[j + lane], 0), a.num_blocks - 1) : 0; };
      int here32 = entries(u0 * UPB), next32 = entries(u0 * UPB + 32);
      for (int t = u0; t < u1; ++t, ++n) {
        const int off = (t - u0) * UPB & 31;
        if (off == 0 && t > u0) {
          here32 = next32;
          next32 = entries(t * UPB + 32);
        }
        int blk[UPB];
#pragma unroll
        for (int i = 0; i < UPB; ++i) blk[i] = __shfl_sync(0xffffffffu, here32, off + i);
        const int s = n % kStages;
        if (n >= kStages) ok = role_wait_warp(&sh.empty[s], (n / kStages - 1) & 1, dead, a.status);
        if (!ok) break;
        if (elect_one()) {
          const int here = min(UPB, nblk - t * UPB);
          mbar_arrive_expect_tx(&sh.full[s], here * 2 * kBlock * D);
          uint8_t* to = smem + s * S::STAGE;
#pragma unroll
          for (int i = 0; i < UPB; ++i) {
            if (i >= here) break;
            const long long at = head + blk[i] * stride;
            bulk_g2s(to + i * (kBlock * D), a.k_pool + at, kBlock * D, &sh.full[s]);
            bulk_g2s(to + kTile * D + i * (kBlock * D), a.v_pool + at, kBlock * D, &sh.full[s]);
          }
        }
        __syncwarp();
      }
    }
    // no copy of this block is in flight when it ends, whichever role gave up
    for (unsigned k = n > kStages ? n - kStages : 0; k < n; ++k)
      (void)mbar_wait_bounded(&sh.full[k % kStages], (k / kStages) & 1);
  } else if (warp == kScoreWarp) {
    // ---- scores: one thread; S_i = Q K(tile)^T once the scores before are read ----
    if (elect_one()) {
      constexpr uint32_t ID_S = tc_idesc_f16(kLanes, kTile);
      const uint32_t kbase = smem_addr(smem + S::K_OFF), qbase = smem_addr(smem + S::Q_OFF);
      unsigned n = 0, n_s[2] = {0, 0}, segs = 0;  // tiles, tiles of each stream, segments
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && role_wait(bar, parity, dead, a.status);
        return ok;
      };
      auto scores = [&](int i, uint32_t kt, bool read) {
        if (!read && !wait(&sh.sfree[i], (n_s[i] - 1) & 1)) return;
        ++n_s[i];
        tc_fence_after();
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t bd = smem_desc_kmajor(kt + ks * (2 * kTile * 16), kTile * 16, 128);
          if constexpr (WIDE)
            tc_mma_f16_ss(tmem + S::TM_S + i * kTile, smem_desc_kmajor(qbase + ks * (2 * kLanes * 16), kLanes * 16, 128), bd, ID_S, ks > 0);
          else
            tc_mma_f16(tmem + S::TM_S + i * kTile, tmem + S::TM_Q + 8 * ks, bd, ID_S, ks > 0);
        }
        tc_commit(&sh.sready[i]);
      };
      while (ok && next_here()) {
        if (!wait(&sh.qready[0], segs & 1) || !wait(&sh.qready[1], segs & 1)) break;
        ++segs;
        const int tiles = seg.u1 - seg.u0;
        for (int t = 0; t < tiles; ++t, ++n) {
          const unsigned k = n % kBufs;
          // (asked together: each answer takes some 100 clocks)
          auto read = [&](int i) { return n_s[i] == 0 || mbar_test(&sh.sfree[i], (n_s[i] - 1) & 1); };
          const bool here = mbar_test(&sh.ready[k], (n / kBufs) & 1);
          const bool free_now = read(t & 1);
          if (!here && !wait(&sh.ready[k], (n / kBufs) & 1)) break;
          scores(t & 1, kbase + k * S::TILE, free_now);
          if (!ok) break;
        }
      }
      // no MMA of this thread is in flight when the block frees its tensor memory, whichever role gave up
      tc_commit(&sh.drain[0]);
      (void)mbar_wait_bounded(&sh.drain[0], 0);
    }
    __syncwarp();
  } else if (warp >= kOutputWarp) {
    // ---- outputs of stream i: one thread; O_i += P_i V(tile) ----
    const int i = warp - kOutputWarp;
    if (elect_one()) {
      constexpr uint32_t ID_O = tc_idesc_f16(kLanes, D);
      const uint32_t vbase = smem_addr(smem + S::V_OFF);
      const uint32_t o = tmem + S::TM_O + i * D, pt = tmem + S::TM_P + i * S::P_COLS;
      unsigned n = 0, n_p = 0;  // tiles, tiles of this stream
      bool ok = true;
      while (ok && next_here()) {
        const int tiles = seg.u1 - seg.u0;
        for (int t = i; t < tiles; t += 2, ++n_p) {
          const unsigned k = (n + t) % kBufs;
          // (weights are ready after the tile's scores, so its values are there too)
          ok = role_wait(&sh.pready[i], n_p & 1, dead, a.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t vt = vbase + k * S::TILE;
#pragma unroll
          for (int part = 0; part < (WIDE ? 2 : 1); ++part)
#pragma unroll
            for (int ks = 0; ks < kTile / 16; ++ks)
              tc_mma_f16(o, pt + part * (kTile / 2) + 8 * ks, smem_desc_kmajor(vt + ks * (2 * D * 16), D * 16, 128), ID_O,
                         t != i || part != 0 || ks != 0);
          tc_commit(&sh.pdone[i]);
          tc_commit(&sh.free[k]);
        }
        n += tiles;
      }
      tc_commit(&sh.drain[1 + i]);
      (void)mbar_wait_bounded(&sh.drain[1 + i], 0);
    }
    __syncwarp();
  } else if (warp >= kConvertWarp) {
    // ---- conversion: warps 2p and 2p + 1 take the tiles of parity p, two blocks each ----
    const int cw = warp - kConvertWarp, pair = cw >> 1, w0 = 2 * (cw & 1);
    unsigned n = 0;
    bool ok = true;
    while (ok && next()) {
      const int total = seg.r.len, u0 = seg.u0, u1 = seg.u1;
      for (int t = u0; t < u1; ++t, ++n) {
        if (static_cast<int>(n & 1) != pair) continue;
        const int s = n % kStages, k = n % kBufs;
        const bool room = n < kBufs || mbar_test(&sh.free[k], (n / kBufs - 1) & 1);
        ok = role_wait_warp(&sh.full[s], (n / kStages) & 1, dead, a.status);
        // unit (nt, kh, g, tig): 16 channels of token 8nt + g; a quarter of the warp takes 8 tokens of one
        // core matrix, their tig rotated so that neither the reads nor the writes meet in a bank
        const int g3 = lane & 3, nt = (lane >> 2) & 1, ktig = ((lane >> 3) + (g3 >> 1) + 2 * nt) & 3;
        const uint8_t* ksrc = smem + s * S::STAGE + w0 * (kBlock * D) + (nt * (D / 64) * 32 + 4 * g3 + ktig) * 16;
        uint4 x[2][D / 64][2];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int kh = 0; kh < D / 64; ++kh)
#pragma unroll
            for (int gs = 0; gs < 2; ++gs)
              x[w][kh][gs] = *reinterpret_cast<const uint4*>(ksrc + w * (kBlock * D) + kh * 512 + gs * 256);
        // unit (c, g, tig): tokens 2tig, 2tig + 1, 8 + 2tig, 9 + 2tig of channels 8 (4c + j) + g
        const int g = (lane >> 1) & 7, tig = 2 * ((lane >> 4) ^ ((g >> 1) & 1)) + (lane & 1);
        const uint8_t* vsrc = smem + s * S::STAGE + kTile * D + w0 * (kBlock * D) + (4 * g + tig) * 16;
        uint4 y[2][D / 32];
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int c = 0; c < D / 32; ++c) y[w][c] = *reinterpret_cast<const uint4*>(vsrc + w * (kBlock * D) + c * 512);
        // (the warp's answer, not the lane's: the barrier may complete between two lanes' tests)
        if (ok && !__all_sync(0xffffffffu, room)) ok = role_wait_warp(&sh.free[k], (n / kBufs - 1) & 1, dead, a.status);
        if (!ok) break;
        // row of the core matrix: 4 (g3 / 2) + 2nt + g3 % 2
        uint8_t* kdst = smem + S::K_OFF + k * S::TILE + ktig * 2 * (kTile * 16) + 2 * w0 * 128 +
                        (4 * (g3 >> 1) + 2 * nt + (g3 & 1)) * 16;
#pragma unroll
        for (int w = 0; w < 2; ++w)
#pragma unroll
          for (int kh = 0; kh < D / 64; ++kh)
#pragma unroll
            for (int gs = 0; gs < 2; ++gs) {
              const uint4 u = x[w][kh][gs];
              uint8_t* d = kdst + kh * 8 * (kTile * 16) + (2 * w + gs) * 128;
              *reinterpret_cast<uint4*>(d) =
                  make_uint4(fp8_lo_pair<FMT>(u.x), fp8_hi_pair<FMT>(u.x), fp8_lo_pair<FMT>(u.y), fp8_hi_pair<FMT>(u.y));
              *reinterpret_cast<uint4*>(d + kTile * 16) =
                  make_uint4(fp8_lo_pair<FMT>(u.z), fp8_hi_pair<FMT>(u.z), fp8_lo_pair<FMT>(u.w), fp8_hi_pair<FMT>(u.w));
            }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          // (the shared blocks are full: a block of the tile has all its tokens or none, and then its values are 0)
          const uint32_t keep = tree_beyond(t * kTile + (w0 + w) * kBlock, kBlock, total) ? 0u : 0xFFFFFFFFu;
          uint8_t* vdst = smem + S::V_OFF + k * S::TILE + (2 * (w0 + w) + (tig >> 1)) * (D * 16) + g * 16 + (tig & 1) * 8;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const uint32_t word[4] = {y[w][c].x & keep, y[w][c].y & keep, y[w][c].z & keep, y[w][c].w & keep};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint2*>(vdst + (4 * c + j) * 128) = make_uint2(fp8_lo_pair<FMT>(word[j]), fp8_hi_pair<FMT>(word[j]));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_if(&sh.ready[k], lane == 0);
        // released once what was read has been used: released after the loads alone, the next copy would overwrite
        // bytes that are still on their way
        mbar_arrive_if(&sh.empty[s], lane == 0);
      }
    }
  } else {
    // ---- softmax: stream `i`, a thread per lane of the tensor memory: copy `fold` of query row `row` ----
    const int i = warp >> 2, tm_lane = tid & (kLanes - 1);
    const int row = tm_lane % R, fold = tm_lane / R;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tm_s = tmem + lanes + S::TM_S + i * kTile + fold * COLS;
    const uint32_t tm_p = tmem + lanes + S::TM_P + i * S::P_COLS;
    if constexpr (FOLD > 1) {
      // weights of the other copies' tokens: 0, once
      uint32_t zero[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) zero[c] = 0u;
#pragma unroll
      for (int c = 0; c < S::P_COLS; c += 16) tmem_st16(tm_p + c, zero);
      tmem_wait_st();
    }
    unsigned n = 0, n_both[2] = {0, 0};  // tiles of this stream; tiles of each stream at the segment's end
    bool ok = true;
    while (next()) {
      const int h = seg.h, total = seg.r.len, row0 = seg.tile * R;
      const int rows = min(R, seg.r.nodes * gq - row0);
      const bool live = row < rows;
      const bool warp_live = (tm_lane & ~31) % R < rows;  // (a warp's lanes are rows of one copy)
      const int node = live ? (row0 + row) / gq : 0, head = live ? row0 + row - node * gq : 0;
      const float k_scale = a.k_scale[a.per_head ? h : 0];
      // a negative scale turns the query's signs, so that larger scores stay larger
      float kmul = fabsf(k_scale) * a.scale_log2;
      if (kmul == 0.0f) kmul = 1e-37f;
      const uint32_t flip = k_scale < 0.0f ? 0x80008000u : 0u;

      if (ok) {  // the query row, its channels in the key units' order (each stream brings half of them)
        const __half* q = reinterpret_cast<const __half*>(a.q) + (seg.r.first + node) * a.q_stride +
                          static_cast<long long>(h * gq + head) * D;
        constexpr bool HALVES = D == 128;
        if (HALVES || i == 0) {
#pragma unroll 1
          for (int kh = HALVES ? i : 0; kh < (HALVES ? i + 1 : D / 64); ++kh) {
            uint32_t w[32];
#pragma unroll
            for (int c8 = 0; c8 < 8; ++c8) {  // channels 64kh + 8 c8 .. +7: places 16 (c8 % 2) + 4 (c8 / 2), and 16 behind them
              uint4 x = make_uint4(0u, 0u, 0u, 0u);
              if (live) x = *reinterpret_cast<const uint4*>(q + 64 * kh + 8 * c8);
              const int at = 2 * (8 * (c8 % 2) + c8 / 2);
              w[at] = x.x ^ flip;
              w[at + 1] = x.y ^ flip;
              w[at + 8] = x.z ^ flip;
              w[at + 9] = x.w ^ flip;
            }
            __syncwarp();  // lanes without a row loaded nothing
            if constexpr (WIDE) {
              uint8_t* d = smem + S::Q_OFF + kh * 8 * (kLanes * 16) + tm_lane * 16;
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(d + c * (kLanes * 16)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
            } else {
              tmem_st32(tmem + lanes + S::TM_Q + 32 * kh, w);
            }
          }
          if constexpr (WIDE) fence_proxy_async_smem();
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&sh.qready[i], lane == 0);
      }

      float m = -INFINITY, msub = -kBias, l = 0.0f;  // m in log2 units; weights are 2^(s * kmul - msub)
      const int u0 = seg.u0, u1 = seg.u1;
      for (int t = u0 + i; ok && t < u1; t += 2, ++n) {
        ok = role_wait_warp(&sh.sready[i], n & 1, dead, a.status);
        if (!ok) break;
        tc_fence_after();
        const bool pv_done = n > 0 && mbar_test(&sh.pdone[i], (n - 1) & 1);  // answers while the scores load
        uint32_t sr[COLS];
        if (warp_live) {
#pragma unroll
          for (int c = 0; c < COLS; c += 32) tmem_ld32(tm_s + c, sr + c);
        }
        const int left = total - t * kTile;  // tokens from the tile's first on
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&sh.sfree[i], lane == 0);
        // the products of the tile before have read P and written O
        if (n > 0 && !__all_sync(0xffffffffu, pv_done)) ok = role_wait_warp(&sh.pdone[i], (n - 1) & 1, dead, a.status);
        if (!ok) break;
        if (warp_live) {
          if (left < kTile) {
#pragma unroll
            for (int c = 0; c < COLS; ++c)
              if (fold * COLS + column_token(c) >= left) sr[c] = 0xFF800000u;
          }
          // Weights against the maximum so far; a tile needs no maximum of its own while their sum shows that none
          // has left fp16's range. Where one has (and in a row without a maximum), the second pass follows a new one.
          bool fresh = t < u0 + 2;  // the stream's first tile: O is empty
          float tile_sum = 0.0f;
#pragma unroll 1
          for (int pass = fresh ? 1 : 0; pass < 2; ++pass) {
            if (pass == 1) {
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < COLS; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(sr[c]));
              const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kmul;
              const bool grow = top > m && (m == -INFINITY || !(tile_sum <= kMostSum));
              const float m_new = grow ? top : m;
              const float alpha = grow ? fast_exp2(m - m_new) : 1.0f;
              l *= alpha;
              m = m_new;
              msub = (m == -INFINITY ? 0.0f : m) - kBias;
              if (!fresh) {
                tmem_wait_st();  // the first pass's weights, which this one overwrites
                tc_fence_after();
#pragma unroll 1
                for (int c0 = 0; c0 < D; c0 += 16) {
                  uint32_t o[16];
                  tmem_ld16(tmem + lanes + S::TM_O + i * D + c0, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                  tmem_st16(tmem + lanes + S::TM_O + i * D + c0, o);
                }
              }
            }
            float2 sum[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
            const float2 mul2 = make_float2(kmul, kmul), sub2 = make_float2(-msub, -msub);
#pragma unroll
            for (int c0 = 0; c0 < COLS; c0 += 32) {
              uint32_t hi[16], lo[WIDE ? 16 : 1];
#pragma unroll
              for (int c = 0; c < 32; c += 2) {
                float2 p = __ffma2_rn(make_float2(__uint_as_float(sr[c0 + c]), __uint_as_float(sr[c0 + c + 1])), mul2, sub2);
                p.x = fast_exp2(p.x);
                p.y = fast_exp2(p.y);
                sum[(c >> 1) & 1] = __fadd2_rn(sum[(c >> 1) & 1], p);
                const __half2 hp = __floats2half2_rn(p.x, p.y);
                hi[c / 2] = h2_bits(hp);
                if constexpr (WIDE) {
                  const float2 f = __half22float2(hp);
                  lo[c / 2] = pack_rn_f16x2(p.x - f.x, p.y - f.y);
                }
              }
              const uint32_t to = tm_p + (fold * COLS + c0) / 2;
              tmem_st16(to, hi);
              if constexpr (WIDE) tmem_st16(to + kTile / 2, lo);
            }
            tile_sum = (sum[0].x + sum[0].y) + (sum[1].x + sum[1].y);
            if (!__any_sync(0xffffffffu, m == -INFINITY || !(tile_sum <= kMostSum))) break;
          }
          l += tile_sum;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&sh.pready[i], lane == 0);
      }

      // ---- the segment's result ----
      const bool have1 = seg.u1 - seg.u0 > 1;  // stream 1 had tiles
      // A stream writes ml only where it had tiles: their scores waited for the queries of both streams, which each brings
      // once it has read the segment before. Without tiles nothing would order its write behind the other stream's reads.
      if (i == 0 || have1) {
        sh.ml[i][tm_lane][0] = m;
        sh.ml[i][tm_lane][1] = l;
      }
      // the last products of both streams
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int its = (seg.u1 - seg.u0 + 1 - e) / 2;
        n_both[e] += its;
        if (its > 0) ok = ok && role_wait_warp(&sh.pdone[e], (n_both[e] - 1) & 1, dead, a.status);
      }
      ok = barrier_and(1, 256, ok);
      if (ok) {
        tc_fence_after();
        // columns [c_begin, c_begin + D / 2) of this thread's row, 16 at a time
        const int c_begin = i * (D / 2);
        const float m0 = sh.ml[0][tm_lane][0], l0 = sh.ml[0][tm_lane][1];
        const float m1 = have1 ? sh.ml[1][tm_lane][0] : -INFINITY, l1 = have1 ? sh.ml[1][tm_lane][1] : 0.0f;
        const float M = fmaxf(m0, m1);
        // (a stream without a maximum has the sum 0, or NaN, which stays)
        const float f0 = M == -INFINITY ? 1.0f : fast_exp2(m0 - M), f1 = M == -INFINITY ? 1.0f : fast_exp2(m1 - M);
        const GroupPlace to = group_place<D>(sh.args, seg, gq, row0, live ? row : 0, fold, tm_lane, kLanes);
        if (warp_live) {
#pragma unroll 1
          for (int c0 = c_begin; c0 < c_begin + D / 2; c0 += 16) {
            uint32_t o[16], o1[16];
            __syncwarp();  // lanes without a row have come round early
            tmem_ld16(tmem + lanes + S::TM_O + c0, o);
            if (have1) tmem_ld16(tmem + lanes + S::TM_O + D + c0, o1);
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float v = __uint_as_float(o[c]) * f0;
              if (have1) v = fmaf(__uint_as_float(o1[c]), f1, v);
              o[c] = __float_as_uint(v);
            }
            if (!live) continue;
#pragma unroll
            for (int c = 0; c < 16; c += 4) reinterpret_cast<uint4*>(to.o + c0)[c / 4] = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
          }
          if (live && i == 0) *reinterpret_cast<float2*>(to.ml) = make_float2(M - kBias, l0 * f0 + l1 * f1);
        }
        tc_fence_before();
      }
      if (tid == 0) group_record(sh.args, seg);
    }
  }
  __syncthreads();
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int FMT, bool WIDE, int FOLD>
cudaError_t launch_tc(const GroupArgs& a, cudaStream_t s) {
  constexpr int smem = TcPlan<D, WIDE>::BYTES;
  static_assert(smem + sizeof(TcShared) <= 232448, "shared memory of a thread block");
  auto kern = group_tc_kernel<D, FMT, WIDE, FOLD>;
  static SharedMemoryOnce once;
  const cudaError_t e = once.set(kern, smem);
  if (e != cudaSuccess) return e;
  const int sms = device_sm_count(), grid = sms < kGroupTcMaxBlocks ? sms : kGroupTcMaxBlocks;
  kern<<<grid, kThreads, smem, s>>>(a);
  return cudaGetLastError();
}

template <int FOLD>
cudaError_t dispatch_tc(const GroupArgs& a, cudaStream_t s) {
  switch (a.head_dim * 100 + a.fmt * 10 + (a.out_fp32 ? 1 : 0)) {
    case 12800: return launch_tc<128, 0, false, FOLD>(a, s);
    case 12801: return launch_tc<128, 0, true, FOLD>(a, s);
    case 12810: return launch_tc<128, 1, false, FOLD>(a, s);
    case 12811: return launch_tc<128, 1, true, FOLD>(a, s);
    case 6400: return launch_tc<64, 0, false, FOLD>(a, s);
    case 6401: return launch_tc<64, 0, true, FOLD>(a, s);
    case 6410: return launch_tc<64, 1, false, FOLD>(a, s);
    case 6411: return launch_tc<64, 1, true, FOLD>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_group_tc(const GroupArgs& a, cudaStream_t s) {
  switch (a.part[0].fold) {
    case 1: return dispatch_tc<1>(a, s);
    case 2: return dispatch_tc<2>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
