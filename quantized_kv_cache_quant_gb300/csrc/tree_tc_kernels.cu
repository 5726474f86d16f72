// Tree attention on the fifth-generation tensor cores (tcgen05), for requests
// with more query rows per kv head than one mma.sync tile.
//
// A thread block per SM walks its slice of (request, kv head, row tile) pairs in
// tiles of 64 tokens. Two streams of 128 query rows each share the tensor core:
//   R = 256: the streams hold different rows and both take every token tile;
//   R = 128: they hold the same rows and take alternate token tiles, each with
//            its own running maximum, sum and outputs, joined at the end.
// While one stream's softmax runs on the CUDA cores the tensor core works for
// the other one.
//   S = Q K^T : A = Q (fp16, exact) in tensor memory, or in shared memory where
//               tensor memory has no room, B = the keys as fp16 in shared
//               memory, accumulators 128 x 64 fp32 in tensor memory
//   O += P V  : A = P in tensor memory (fp16; WIDE, for fp32 output: and the
//               rounding's remainder), B = the values as fp16
// Tensor memory's 512 columns (D = 128): O 2 x 128, S 2 x 64, P 2 x 32 and Q 64,
// or with WIDE P 2 x 64 and no Q. P beside S, not over it, is what lets a
// stream's next scores run under its softmax: with P over S a tile took 1220
// clocks (R = 128) and 2200 (R = 256) instead of 1050 and 1900.
// Roles: one warp copies pool blocks (bulk copies, some tiles ahead), four warps
// turn FP8 bytes into fp16 operand tiles (each byte once per thread block, for
// all its rows), three threads issue the MMAs (scores, and each stream's outputs:
// a wait costs an issuing thread some 100 clocks even when it is over, and one
// thread with all the waits of a tile was what bounded the kernel), two groups of
// four warps do the softmax, a thread per query row. Weights are 2^(score - m + kBias), m a maximum of
// the row that is renewed (and the row's outputs rescaled) only when a tile's
// weights sum to more than 2^15: all of them are within fp16 until then, those
// down to 2^-21 of the largest are normal fp16 numbers, and a tile in which
// nothing grows needs no maximum.
//
// Orders that the products do not see: the channels of Q and K follow the key
// bytes' order, the tokens of a block that of the value bytes (column 4t + 2r +
// e is token 8r + 2t + e), so that both conversions read 16-byte units and
// write 16- and 8-byte pieces, all without bank conflicts.
//
// What bounds it: the chain within a stream. P has one buffer, so a stream's
// weights of a tile wait for the product of its tile before: 1380 clocks of
// softmax and 700 of product and commit with R = 128, 2080 a tile of the stream
// and, with two streams on alternate tiles, 1040 a tile, whatever D; the memory
// needs 745, the products 512. (Six places in the fp16 ring in place of four, at
// D = 64, changed nothing.) R = 256: 1430 and 500, 1930 a tile; the products need
// 1024. Weights in two parts (WIDE) take 1.5 to 1.8 times as long. Measured on
// random pages, cold caches, 8 kv heads, E4M3 at D = 128, E5M2 per head at D = 64:
//   32 requests x 32768 tokens, trees of 16, 64 rows   512 us  4.2 TB/s (WIDE 875)
//   4 requests x 131072 tokens, chains of 4, 32 rows   259 us  4.1 TB/s (WIDE 424)
//   16 requests x 16384 tokens, 63 nodes, 504 rows     505 us  1075 TFLOP/s (WIDE 885)
//   32 requests x 512 to 16384 tokens, 1 to 40 nodes, D = 64   195 us (WIDE 287)
// Between segments: about 8000 clocks from the last scores of one to the first
// of the next (outputs 4000, queries 2000, the next segment 1500).
#include "tc_device.cuh"
#include "tree_plan.cuh"

namespace kvq {
namespace {

constexpr int kBlock = 16;
constexpr int kTile = 64;             // tokens of a tile (and of a work unit)
constexpr int kMaxBufs = 4;           // fp16 tiles (keys and values)
constexpr float kBias = 7.0f;
constexpr float kMostSum = 32768.0f;  // of a tile's weights in a row: each is within fp16 then
constexpr int kThreads = 512;
// warps: 0-3 and 4-7 softmax of stream 0 and 1, 8-11 conversion, 12 copies, 13 the scores' MMAs, 14 and 15 the outputs'
// MMAs of stream 0 and 1
constexpr int kConvertWarp = 8, kCopyWarp = 12, kScoreWarp = 13, kOutputWarp = 14;
constexpr int kMaxStages = 6;

template <int D, bool WIDE, int R>
struct TcPlan {
  static constexpr bool SPLIT_ROWS = R == 256;      // the streams' rows differ (else their tokens do)
  static constexpr int Q_SMEM = (WIDE ? 1 : 0) + (SPLIT_ROWS ? 1 : 0);  // Q tiles in shared memory
  // shared memory
  static constexpr int STAGE = 2 * kTile * D;       // pool bytes of a tile: keys, then values
  static constexpr int TILE = kTile * D * 2;        // one fp16 tile of keys or values
  static constexpr int Q_TILE = 128 * D * 2;
  // Both rings have an even number of places: the converting pairs take tiles of alternate parity, and so a place
  // always belongs to one pair, which sees each phase of its barriers. (In an odd ring a pair meets a place every second
  // time round, and its wait for a phase's parity is over while the phase before still runs.)
  // (2 places in place of 4 where 4 fit: 690, 536 and 340 us for 492, 448 and 244 of an earlier state)
  static constexpr int BUFS = Q_SMEM == 2 ? 2 : kMaxBufs;
  static constexpr int FIXED = BUFS * 2 * TILE + Q_SMEM * Q_TILE;
  static constexpr int FIT = (221184 - FIXED) / STAGE;  // 227 KB without what TcShared takes
  static constexpr int STAGES = (FIT < kMaxStages ? FIT : kMaxStages) & ~1;
  static_assert(STAGES >= 2, "room for the copies");
  static_assert(STAGES % 2 == 0 && BUFS % 2 == 0, "a place of a ring belongs to one converting pair");
  static constexpr int K_OFF = STAGES * STAGE, V_OFF = K_OFF + BUFS * TILE, Q_OFF = V_OFF + BUFS * TILE;
  static constexpr int BYTES = Q_OFF + Q_SMEM * Q_TILE;
  // tensor memory columns
  static constexpr int P_COLS = (WIDE ? 2 : 1) * kTile / 2;
  static constexpr int TM_O = 0, TM_S = 2 * D, TM_P = TM_S + 2 * kTile, TM_Q = TM_P + 2 * P_COLS;
  static_assert((WIDE ? TM_Q : TM_Q + D / 2) <= 512, "tensor memory");
};

struct TcShared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t ready[kMaxBufs], free[kMaxBufs];
  uint64_t qready[2], sready[2], sfree[2], pready[2], pdone[2], drain[3];
  unsigned long long plan[36];
  uint32_t tmem;
  int dead, nan_met;
  float ml[2][128][2];
  // the arguments, for functions out of line (a reference to a kernel's parameters is read from global memory there)
  TreeArgs args;
  // each warp's place in the slice: in shared memory, not in registers that the roles' loops need
  TreeSlice slice;
  TreeWalk walk[kThreads / 32];
};

// Bits of the tokens tok .. tok + 63 that a row with these mask words sees.
__device__ __forceinline__ uint64_t tree_window(const uint64_t* mask, int words, int tok, int len, int total) {
  const int j0 = tok - len;
  uint64_t w;
  if (j0 <= -64) return ~0ull;
  if (j0 < 0) {
    const int ctx = -j0;  // 1 .. 63 tokens before the tree
    w = ((1ull << ctx) - 1) | (mask[0] << ctx);
  } else {
    const int i = j0 >> 6, sh = j0 & 63;
    w = i < words ? mask[i] >> sh : 0ull;
    if (sh != 0 && i + 1 < words) w |= mask[i + 1] << (64 - sh);
  }
  const int n = total - tok;  // tokens of the request from here on
  return n >= 64 ? w : (n <= 0 ? 0ull : w & ((1ull << n) - 1));
}

// Token of column c of a tile.
__host__ __device__ constexpr int column_token(int c) {
  return (c & ~15) + 8 * ((c >> 1) & 1) + 2 * ((c >> 2) & 3) + (c & 1);
}

template <int D, int FMT, bool WIDE, int R>
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(const __grid_constant__ TreeArgs a) {
  using S = TcPlan<D, WIDE, R>;
  constexpr bool SPLIT_ROWS = S::SPLIT_ROWS;
  constexpr int UPB = kTile / kBlock;  // pool blocks of a tile
  constexpr unsigned kStages = S::STAGES, kBufs = S::BUFS;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ TcShared sh;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);  // uniform for the compiler too
  const int gq = a.q_heads / a.kv_heads;

  if (tid == 0) {
    for (int i = 0; i < kMaxStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 2);
    }
    for (int i = 0; i < kMaxBufs; ++i) {
      mbar_init(&sh.ready[i], 2);
      mbar_init(&sh.free[i], SPLIT_ROWS ? 2 : 1);  // from each stream that reads the tile
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.qready[i], 4);
      mbar_init(&sh.sready[i], 1);
      mbar_init(&sh.sfree[i], 4);
      mbar_init(&sh.pready[i], 4);
      mbar_init(&sh.pdone[i], 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&sh.drain[i], 1);
    sh.dead = sh.nan_met = 0;
    sh.args = a;
    fence_mbar_init();
  }
  if (tid == 0) tree_leave_none(a);
  {
    // Slices of 2 to 4 tiles at least: a pair of 2 tiles (one request of 100 tokens) takes 11 us alone in its block and
    // 16 with another one, a request of 2500 tokens 20 us in slices of 2 and 17 in slices of 4. Cuts keep 4 to 8 tiles
    // from a pair's ends: 16 requests of 1000 tokens and 64 rows 31 us with cuts anywhere, 23 with 8.
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

  TreeWalk& walk = sh.walk[warp];
  const TreeSegment& seg = walk.seg;
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
    // ---- copies: lane 2i + r takes block i of a tile, r = 0 keys, 1 values ----
    unsigned n = 0;  // tiles issued
    bool ok = true;
    while (ok && next()) {
      const int nblk = tree_units(seg.r.len + seg.r.nodes, kBlock);
      const int32_t* table = a.block_table + static_cast<long long>(seg.b) * a.max_blocks;
      const uint8_t* pool = ((lane & 1) ? a.v_pool : a.k_pool) + static_cast<long long>(seg.h) * (kBlock * D);
      const int i = lane >> 1, u0 = seg.u0, u1 = seg.u1;
      auto entry = [&](int t) -> int { return (i < UPB && t * UPB + i < nblk) ? table[t * UPB + i] : 0; };
      int ahead = entry(u0);
      for (int t = u0; t < u1; ++t, ++n) {
        const int blk = ahead;
        if (t + 1 < u1) ahead = entry(t + 1);
        const int s = n % kStages;
        if (n >= kStages) ok = role_wait_warp(&sh.empty[s], (n / kStages - 1) & 1, dead, a.status);
        if (!ok) break;
        const int here = min(UPB, nblk - t * UPB);
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], here * 2 * kBlock * D);
        __syncwarp();
        if (i < here) {
          const long long p = min(max(blk, 0), a.num_blocks - 1);
          bulk_g2s(smem + s * S::STAGE + (lane & 1) * (kTile * D) + i * (kBlock * D),
                   pool + p * a.kv_heads * (kBlock * D), kBlock * D, &sh.full[s]);
        }
      }
    }
    // no copy of this block is in flight when it ends, whichever role gave up
    for (unsigned k = n > kStages ? n - kStages : 0; k < n; ++k)
      (void)mbar_wait_bounded(&sh.full[k % kStages], (k / kStages) & 1);
  } else if (warp == kScoreWarp) {
    // ---- scores: one thread; S_i = Q_i K(tile)^T once the scores before are read ----
    if (elect_one()) {
      constexpr uint32_t ID_S = tc_idesc_f16(128, kTile);
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
        const bool q_smem = WIDE || (SPLIT_ROWS && i == 1);
        const uint32_t qt = qbase + ((WIDE && SPLIT_ROWS) ? i * S::Q_TILE : 0);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t bd = smem_desc_kmajor(kt + ks * (2 * kTile * 16), kTile * 16, 128);
          if (q_smem)
            tc_mma_f16_ss(tmem + S::TM_S + i * kTile, smem_desc_kmajor(qt + ks * (2 * 128 * 16), 128 * 16, 128), bd, ID_S, ks > 0);
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
          const bool read0 = (SPLIT_ROWS || !(t & 1)) && read(0), read1 = (SPLIT_ROWS || (t & 1)) && read(1);
          if (!here && !wait(&sh.ready[k], (n / kBufs) & 1)) break;
          const uint32_t kt = kbase + k * S::TILE;
          if constexpr (SPLIT_ROWS) {
            scores(0, kt, read0);
            scores(1, kt, read1);
          } else {
            if (t & 1) scores(1, kt, read1);
            else scores(0, kt, read0);
          }
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
      constexpr uint32_t ID_O = tc_idesc_f16(128, D);
      const uint32_t vbase = smem_addr(smem + S::V_OFF);
      const uint32_t o = tmem + S::TM_O + i * D, pt = tmem + S::TM_P + i * S::P_COLS;
      unsigned n = 0, n_p = 0;  // tiles, tiles of this stream
      bool ok = true;
      while (ok && next_here()) {
        const int first = SPLIT_ROWS ? 0 : i, step = SPLIT_ROWS ? 1 : 2, tiles = seg.u1 - seg.u0;
        for (int t = first; t < tiles; t += step, ++n_p) {
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
                         t != first || part != 0 || ks != 0);
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
    // ---- conversion: warps 2p and 2p + 1 take the tiles of parity p, two blocks each. (All four warps on
    // one tile left the tensor core waiting: a tile's waits, fences and load latencies are a fixed cost of
    // each warp, so two tiles are converted at a time.) ----
    const int cw = warp - kConvertWarp, pair = cw >> 1, w0 = 2 * (cw & 1);
    unsigned n = 0;
    bool ok = true;
    while (ok && next()) {
      const int len = seg.r.len, total = len + seg.r.nodes, u0 = seg.u0, u1 = seg.u1;
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
          const int tok0 = t * kTile + (w0 + w) * kBlock;
          uint32_t keep = 0xFFFFFFFFu;
          if (tree_beyond(tok0, kBlock, len)) {  // the tree's own tokens, and rows behind them
            uint32_t tree_bytes = 0;
            keep = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = tok0 + 8 * (i >> 1) + 2 * tig + (i & 1);
              if (tok < total) keep |= 0xFFu << (8 * i);
              if (tok >= len) tree_bytes |= 0xFFu << (8 * i);
            }
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {
              uint32_t* word = &y[w][c].x;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t bad = fp8_nonfinite<FMT>(word[j]) & tree_bytes & keep;
                if (bad != 0) sh.nan_met = 1;
                word[j] &= keep & ~bad;
              }
            }
          }
          uint8_t* vdst = smem + S::V_OFF + k * S::TILE + (2 * (w0 + w) + (tig >> 1)) * (D * 16) + g * 16 + (tig & 1) * 8;
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const uint32_t word[4] = {y[w][c].x, y[w][c].y, y[w][c].z, y[w][c].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint2*>(vdst + (4 * c + j) * 128) = make_uint2(fp8_lo_pair<FMT>(word[j]), fp8_hi_pair<FMT>(word[j]));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        mbar_arrive_if(&sh.ready[k], lane == 0);
        // released once what was read has been used: released after the loads alone, the next copy overwrote bytes
        // that were still on their way
        mbar_arrive_if(&sh.empty[s], lane == 0);
      }
    }
  } else {
    // ---- softmax: stream `i`, a thread per query row ----
    const int i = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tm_s = tmem + lanes + S::TM_S + i * kTile, tm_p = tmem + lanes + S::TM_P + i * S::P_COLS;
    unsigned n = 0, n_both[2] = {0, 0};  // tiles of this stream; tiles of each stream at the segment's end
    bool ok = true;
    while (next()) {
      const int h = seg.h, len = seg.r.len, total = len + seg.r.nodes, row0 = seg.tile * R;
      const int rows = min(R, seg.r.nodes * gq - row0);       // of the tile
      const int my_rows = SPLIT_ROWS ? min(128, rows - 128 * i) : rows;  // of this stream (may be below 1)
      const int trow = SPLIT_ROWS ? row + 128 * i : row;      // row of the tile
      const bool live = row < my_rows;
      const bool warp_live = (row & ~31) < my_rows;
      const int node = live ? (row0 + trow) / gq : 0, head = live ? row0 + trow - node * gq : 0;
      const float k_scale = a.k_scale[a.per_head ? h : 0], v_scale = a.v_scale[a.per_head ? h : 0];
      // a negative scale turns the query's signs, so that larger scores stay larger
      float kmul = fabsf(k_scale) * a.scale_log2;
      if (kmul == 0.0f) kmul = 1e-37f;
      const uint32_t flip = k_scale < 0.0f ? 0x80008000u : 0u;
      const uint64_t* mask = a.tree_mask + static_cast<long long>(seg.r.first + node) * a.mask_words;

      if (ok) {  // the query row, its channels in the key units' order (R = 128: each stream brings half of them)
        const __half* q = reinterpret_cast<const __half*>(a.q) + (seg.r.first + node) * a.q_stride +
                          static_cast<long long>(h * gq + head) * D;
        constexpr bool HALVES = !SPLIT_ROWS && D == 128;
        if (SPLIT_ROWS || HALVES || i == 0) {
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
            if (WIDE || (SPLIT_ROWS && i == 1)) {  // (uniform per warp)
              uint8_t* d = smem + S::Q_OFF + ((WIDE && SPLIT_ROWS) ? i * S::Q_TILE : 0) + kh * 8 * (128 * 16) + row * 16;
#pragma unroll
              for (int c = 0; c < 8; ++c)
                *reinterpret_cast<uint4*>(d + c * (128 * 16)) = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
            } else {
              tmem_st32(tmem + lanes + S::TM_Q + 32 * kh, w);
            }
          }
          if (WIDE || (SPLIT_ROWS && i == 1)) fence_proxy_async_smem();
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&sh.qready[i], lane == 0);
      }

      float m = -INFINITY, msub = -kBias, l = 0.0f;  // m in log2 units; weights are 2^(s * kmul - msub)
      const int step = SPLIT_ROWS ? 1 : 2;
      const int u0 = seg.u0, u1 = seg.u1;
      for (int t = u0 + (SPLIT_ROWS ? 0 : i); ok && t < u1; t += step, ++n) {
        ok = role_wait_warp(&sh.sready[i], n & 1, dead, a.status);
        if (!ok) break;
        tc_fence_after();
        const bool pv_done = n > 0 && mbar_test(&sh.pdone[i], (n - 1) & 1);  // answers while the scores load
        uint32_t sr[kTile];
        if (warp_live) {
          tmem_ld32(tm_s, sr);
          tmem_ld32(tm_s + 32, sr + 32);
        }
        const int tok0 = t * kTile;
        uint64_t vis = ~0ull;
        const bool edge = tree_beyond(tok0, kTile, len);
        if (edge && warp_live) vis = tree_window(mask, a.mask_words, tok0, len, total);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        mbar_arrive_if(&sh.sfree[i], lane == 0);
        // the products of the tile before have read P and written O
        if (n > 0 && !__all_sync(0xffffffffu, pv_done)) ok = role_wait_warp(&sh.pdone[i], (n - 1) & 1, dead, a.status);
        if (!ok) break;
        if (warp_live) {
          if (edge) {
#pragma unroll
            for (int c = 0; c < kTile; ++c)
              if (!((vis >> column_token(c)) & 1)) sr[c] = 0xFF800000u;
          }
          // Weights against the maximum so far; a tile needs no maximum of its own while their sum shows that none
          // has left fp16's range. Where one has (and in a row without a maximum), the second pass follows a new one.
          bool fresh = t < u0 + step;  // the stream's first tile: O is empty
          float tile_sum = 0.0f;
#pragma unroll 1
          for (int pass = fresh ? 1 : 0; pass < 2; ++pass) {
            if (pass == 1) {
              float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
              for (int c = 0; c < kTile; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(sr[c]));
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
            for (int c0 = 0; c0 < kTile; c0 += 32) {
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
              tmem_st16(tm_p + c0 / 2, hi);
              if constexpr (WIDE) tmem_st16(tm_p + kTile / 2 + c0 / 2, lo);
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
      const bool have1 = SPLIT_ROWS || seg.u1 - seg.u0 > 1;  // stream 1 had tiles
      // A stream writes ml only where it had tiles: their scores waited for the queries of both streams, which each brings
      // once it has read the segment before. Without tiles nothing would order its write behind the other stream's reads.
      if (!SPLIT_ROWS && (i == 0 || have1)) {
        sh.ml[i][row][0] = m;
        sh.ml[i][row][1] = l;
      }
      // the last products of the streams whose outputs this thread reads
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int tiles = seg.u1 - seg.u0, its = SPLIT_ROWS ? tiles : (tiles + 1 - e) / 2;
        n_both[e] += its;
        if (its > 0 && (!SPLIT_ROWS || e == i)) ok = ok && role_wait_warp(&sh.pdone[e], (n_both[e] - 1) & 1, dead, a.status);
      }
      ok = barrier_and(1, 256, ok);
      const bool whole = seg.parts == 1;
      if (ok) {
        tc_fence_after();
        const bool nan_met = sh.nan_met != 0;
        // columns [c_begin, c_begin + COLS) of this thread's row, 16 at a time
        constexpr int COLS = SPLIT_ROWS ? D : D / 2;
        const int c_begin = SPLIT_ROWS ? 0 : i * COLS;
        float M = m, L = l, f0 = 1.0f, f1 = 0.0f;
        if constexpr (!SPLIT_ROWS) {
          const float m0 = sh.ml[0][row][0], l0 = sh.ml[0][row][1];
          const float m1 = have1 ? sh.ml[1][row][0] : -INFINITY, l1 = have1 ? sh.ml[1][row][1] : 0.0f;
          M = fmaxf(m0, m1);
          // (a stream without a maximum has the sum 0, or NaN, which stays)
          f0 = M == -INFINITY ? 1.0f : fast_exp2(m0 - M);
          f1 = M == -INFINITY ? 1.0f : fast_exp2(m1 - M);
          L = l0 * f0 + l1 * f1;
        }
        const float f = whole ? (L == 0.0f ? 0.0f : v_scale / L) : 1.0f;
        const long long prow = static_cast<long long>(seg.slot) * R + trow;
        const long long orow = static_cast<long long>(seg.r.first + node) * a.q_heads + h * gq + head;
        const bool halves = whole && !WIDE;  // fp16 output, else fp32 output or a partial result
        float* const dst = (whole ? reinterpret_cast<float*>(a.out) + orow * D : a.part_o + prow * D);
        if (warp_live) {
#pragma unroll 1
          for (int c0 = c_begin; c0 < c_begin + COLS; c0 += 16) {
            uint32_t o[16], o1[SPLIT_ROWS ? 1 : 16];
            __syncwarp();  // lanes without a row have come round early
            tmem_ld16(tmem + lanes + S::TM_O + (SPLIT_ROWS ? i * D : 0) + c0, o);
            if constexpr (!SPLIT_ROWS) {
              if (have1) tmem_ld16(tmem + lanes + S::TM_O + D + c0, o1);
            }
            tmem_wait_ld();
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              float v = __uint_as_float(o[c]) * f0;
              if constexpr (!SPLIT_ROWS) {
                if (have1) v = fmaf(__uint_as_float(o1[c]), f1, v);
              }
              o[c] = __float_as_uint(v * f);
            }
            if (!live) continue;
            if (halves) {
              uint4* d = reinterpret_cast<uint4*>(reinterpret_cast<__half*>(a.out) + orow * D + c0);
#pragma unroll
              for (int c = 0; c < 16; c += 8) {
                auto two = [&](int e) { return pack_rn_f16x2(__uint_as_float(o[c + e]), __uint_as_float(o[c + e + 1])); };
                d[c / 8] = make_uint4(two(0), two(2), two(4), two(6));
              }
            } else {
#pragma unroll
              for (int c = 0; c < 16; c += 4) reinterpret_cast<uint4*>(dst + c0)[c / 4] = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
            }
          }
          if (whole && live && nan_met)
            tree_put_nan<D, FMT>(sh.args, seg.b, h, seg.r.first, seg.r.nodes, len, row0 + trow, c_begin, c_begin + COLS);
        if (!whole && live && (SPLIT_ROWS || i == 0))
            *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(M, L);
        }
        tc_fence_before();
      }
      if (!whole && tid == 0) {
        a.part_flag[seg.slot] = sh.nan_met;
        if (seg.u0 == 0) tree_leave_join(sh.args, seg, ok ? rows : 0, row0);
      }
    }
  }
  __syncthreads();
  if (warp == kScoreWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int FMT, bool WIDE, int R>
cudaError_t launch_tc(const TreeArgs& a, cudaStream_t s) {
  constexpr int smem = TcPlan<D, WIDE, R>::BYTES;
  static_assert(smem + sizeof(TcShared) <= 232448, "shared memory of a thread block");
  auto kern = tree_tc_kernel<D, FMT, WIDE, R>;
  static SharedMemoryOnce once;
  cudaError_t e = once.set(kern, smem);
  if (e != cudaSuccess) return e;
  constexpr int kMost = kTreePartRows / (2 * R);  // blocks whose partial results fit the workspace
  static_assert(kMost <= kTreeMaxBlocks, "and what describes them");
  const int sms = device_sm_count(), grid = sms < kMost ? sms : kMost;
  kern<<<grid, kThreads, smem, s>>>(a);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_tree_join(a, grid, R, s);
}

template <int R>
cudaError_t dispatch_tc(const TreeArgs& a, cudaStream_t s) {
  switch (a.head_dim * 100 + a.fmt * 10 + (a.out_fp32 ? 1 : 0)) {
    case 12800: return launch_tc<128, 0, false, R>(a, s);
    case 12801: return launch_tc<128, 0, true, R>(a, s);
    case 12810: return launch_tc<128, 1, false, R>(a, s);
    case 12811: return launch_tc<128, 1, true, R>(a, s);
    case 6400: return launch_tc<64, 0, false, R>(a, s);
    case 6401: return launch_tc<64, 0, true, R>(a, s);
    case 6410: return launch_tc<64, 1, false, R>(a, s);
    case 6411: return launch_tc<64, 1, true, R>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_tree_tc(const TreeArgs& a, cudaStream_t s) {
  // 256 rows a tile read and convert the keys once for twice the rows, but a request with fewer rows pays for both
  // streams: it takes an average (host's knowledge: the rows of all requests) above one stream's rows. And it takes more
  // tiles of 128 rows than SMs (one request, 252 rows, 1000 tokens: 23 us with 128, 29 with 256; four requests, 512 rows,
  // 2500 tokens: 49 and 51; 16 requests: 131 and 116).
  const int gq = a.q_heads / a.kv_heads;
  const long long rows = static_cast<long long>(a.n_tokens) * gq, row_tiles = (rows + 127) / 128;
  const bool wide_tile = rows > 128ll * a.batch && a.max_tree * gq > 128 && row_tiles * a.kv_heads > device_sm_count();
  return wide_tile ? dispatch_tc<256>(a, s) : dispatch_tc<128>(a, s);
}

}  // namespace kvq
