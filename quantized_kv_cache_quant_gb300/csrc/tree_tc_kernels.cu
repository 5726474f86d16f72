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
//   S = Q K^T : A = Q in tensor memory (fp16, exact), B = the keys as fp16 in
//               shared memory, accumulators 128 x 64 fp32 in tensor memory
//   O += P V  : A = P in tensor memory (fp16, over S's columns; WIDE: and the
//               rounding's remainder), B = the values as fp16
// Roles: one warp copies pool blocks (bulk copies, 6 tiles ahead), four warps turn
// FP8 bytes into fp16 operand tiles (each byte once per thread block, for all
// its rows), one thread issues the MMAs, two groups of four warps do the
// softmax, a thread per query row. A row's outputs are rescaled only when its
// maximum has grown by more than 2^kSlack: weights then reach 2^(kBias +
// kSlack) = 2^15, within fp16, and those down to 2^-21 of the largest stay
// normal fp16 numbers.
//
// Orders that the products do not see: the channels of Q and K follow the key
// bytes' order, the tokens of a block that of the value bytes (column 4t + 2r +
// e is token 8r + 2t + e), so that both conversions read 16-byte units and
// write 16- and 8-byte pieces, all without bank conflicts.
#include "tc_device.cuh"
#include "tree_plan.cuh"

namespace kvq {
namespace {

constexpr int kBlock = 16;
constexpr int kTile = 64;             // tokens of a tile (and of a work unit)
constexpr int kStages = 6;            // tiles of pool bytes in flight
constexpr int kBufs = 3;              // fp16 tiles of keys and of values
constexpr float kBias = 7.0f;
constexpr float kSlack = 8.0f;
constexpr int kThreads = 448;
// warps: 0-3 and 4-7 softmax of stream 0 and 1, 8-11 conversion, 12 copies, 13 MMA
constexpr int kConvertWarp = 8, kCopyWarp = 12, kMmaWarp = 13;

template <int D>
struct TcSmem {
  static constexpr int STAGE = 2 * kTile * D;      // key bytes, then value bytes
  static constexpr int KTILE = kTile * D * 2;      // one fp16 tile
  static constexpr int K_OFF = kStages * STAGE;
  static constexpr int V_OFF = K_OFF + kBufs * KTILE;
  static constexpr int BYTES = V_OFF + kBufs * KTILE;
};

struct TcShared {
  uint64_t full[kStages], empty[kStages];
  uint64_t kready[kBufs], kfree[kBufs], vready[kBufs], vfree[kBufs];
  uint64_t qready[2], sready[2], pready[2], oready[2], drain;
  unsigned long long plan[34];
  uint32_t tmem;
  int dead, nan_met, last;
  float ml[2][128][2];
  float merge[2 * 256 + 1];
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
__global__ void __launch_bounds__(kThreads, 1) tree_tc_kernel(TreeArgs a) {
  using S = TcSmem<D>;
  constexpr bool SPLIT_ROWS = R == 256;  // the streams' rows differ (else their tokens do)
  constexpr int UPB = kTile / kBlock;    // pool blocks of a tile
  constexpr uint32_t TM_O = 0, TM_Q = 2 * D, TM_S = 2 * D + D;  // columns: O, Q, S of stream 0; stream 1 follows each
  constexpr uint32_t S_COLS = kTile, Q_COLS = D / 2;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ TcShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int gq = a.q_heads / a.kv_heads;

  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sh.full[i], 1);
      mbar_init(&sh.empty[i], 4);
    }
    for (int i = 0; i < kBufs; ++i) {
      mbar_init(&sh.kready[i], 4);
      mbar_init(&sh.vready[i], 4);
      mbar_init(&sh.kfree[i], 1);
      mbar_init(&sh.vfree[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh.qready[i], 4);
      mbar_init(&sh.sready[i], 1);
      mbar_init(&sh.pready[i], 4);
      mbar_init(&sh.oready[i], 1);
    }
    mbar_init(&sh.drain, 1);
    sh.dead = sh.nan_met = 0;
    fence_mbar_init();
  }
  const TreeSlice slice = tree_slice<R, kTile>(a, sh.plan, 2);
  if (static_cast<int>(blockIdx.x) >= slice.blocks) return;
  if (warp == kMmaWarp) {
    tmem_alloc(&sh.tmem, 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sh.tmem;
  volatile int* dead = &sh.dead;

  long long at = slice.begin, before = slice.before;
  int b = slice.b;
  TreeSegment seg;

  if (warp == kCopyWarp) {
    // ---- copies: lane 2i + r takes block i of a tile, r = 0 keys, 1 values ----
    unsigned n = 0;  // tiles issued
    bool ok = true;
    while (ok && next_segment<R, kTile>(a, slice, at, b, before, seg)) {
      const int nblk = (seg.r.len + seg.r.nodes + kBlock - 1) / kBlock;
      const int32_t* table = a.block_table + static_cast<long long>(seg.b) * a.max_blocks;
      const uint8_t* pool = (lane & 1) ? a.v_pool : a.k_pool;
      const int i = lane >> 1;
      auto entry = [&](int t) -> int { return (i < UPB && t * UPB + i < nblk) ? table[t * UPB + i] : 0; };
      int next = entry(seg.u0);
      for (int t = seg.u0; t < seg.u1; ++t, ++n) {
        const int blk = next;
        if (t + 1 < seg.u1) next = entry(t + 1);
        const int s = n % kStages;
        if (n >= kStages) ok = role_wait(&sh.empty[s], (n / kStages - 1) & 1, dead, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const int here = min(UPB, nblk - t * UPB);
        if (lane == 0) mbar_arrive_expect_tx(&sh.full[s], here * 2 * kBlock * D);
        __syncwarp();
        if (i < here) {
          const long long p = min(max(blk, 0), a.num_blocks - 1);
          bulk_g2s(smem + s * S::STAGE + (lane & 1) * (kTile * D) + i * (kBlock * D),
                   pool + (p * a.kv_heads + seg.h) * (kBlock * D), kBlock * D, &sh.full[s]);
        }
      }
    }
    if (!ok || *dead) {  // no copy of this block is in flight when it ends
      for (unsigned k = n > kStages ? n - kStages : 0; k < n; ++k)
        (void)mbar_wait_bounded(&sh.full[k % kStages], (k / kStages) & 1);
    }
  } else if (warp == kMmaWarp) {
    // ---- MMA: one thread ----
    if (lane == 0) {
      constexpr uint32_t ID_S = tc_idesc_f16(128, kTile), ID_O = tc_idesc_f16(128, D);
      const uint32_t kbase = smem_addr(smem + S::K_OFF), vbase = smem_addr(smem + S::V_OFF);
      unsigned n = 0;                    // tiles whose keys are in use or done
      unsigned n_s[2] = {0, 0};          // tiles of each stream whose weights were used
      unsigned segs = 0;
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        ok = ok && role_wait(bar, parity, dead, a.status);
        return ok;
      };
      auto scores = [&](int i, unsigned k) {  // S_i = Q_i K(tile k)^T
        const uint32_t kt = kbase + (k % kBufs) * S::KTILE;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          tc_mma_f16(tmem + TM_S + i * S_COLS, tmem + TM_Q + i * Q_COLS + 8 * ks,
                     smem_desc_kmajor(kt + ks * (2 * kTile * 16), kTile * 16, 128), ID_S, ks > 0);
        tc_commit(&sh.sready[i]);
      };
      auto outputs = [&](int i, unsigned k, bool first) {  // O_i += P_i V(tile k)
        const uint32_t vt = vbase + (k % kBufs) * S::KTILE;
#pragma unroll
        for (int part = 0; part < (WIDE ? 2 : 1); ++part)
#pragma unroll
          for (int ks = 0; ks < kTile / 16; ++ks)
            tc_mma_f16(tmem + TM_O + i * D, tmem + TM_S + i * S_COLS + part * (kTile / 2) + 8 * ks,
                       smem_desc_kmajor(vt + ks * (2 * D * 16), D * 16, 128), ID_O, !(first && part == 0 && ks == 0));
      };
      while (ok && next_segment<R, kTile>(a, slice, at, b, before, seg)) {
        const int tiles = seg.u1 - seg.u0;
        if (!wait(&sh.qready[0], segs & 1) || !wait(&sh.qready[1], segs & 1)) break;
        ++segs;
        tc_fence_after();
        if constexpr (SPLIT_ROWS) {
          if (!wait(&sh.kready[n % kBufs], (n / kBufs) & 1)) break;
          tc_fence_after();
          scores(0, n);
          scores(1, n);
          tc_commit(&sh.kfree[n % kBufs]);
          for (int t = 0; t < tiles && ok; ++t, ++n) {
            const bool more = t + 1 < tiles;
            if (more && !wait(&sh.kready[(n + 1) % kBufs], ((n + 1) / kBufs) & 1)) break;
            if (!wait(&sh.vready[n % kBufs], (n / kBufs) & 1)) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!wait(&sh.pready[i], n_s[i] & 1)) break;
              ++n_s[i];
              tc_fence_after();
              outputs(i, n, t == 0);
              if (i == 1) tc_commit(&sh.vfree[n % kBufs]);
              if (more) {
                scores(i, n + 1);  // after P_i V(n) on the tensor core, which reads the columns this writes
                if (i == 1) tc_commit(&sh.kfree[(n + 1) % kBufs]);
              } else {
                tc_commit(&sh.oready[i]);
              }
            }
          }
        } else {
          for (int t = 0; t <= tiles && ok; ++t) {
            if (t < tiles) {
              const unsigned k = n + t;
              if (!wait(&sh.kready[k % kBufs], (k / kBufs) & 1)) break;
              tc_fence_after();
              scores(t & 1, k);
              tc_commit(&sh.kfree[k % kBufs]);
            }
            if (t > 0) {
              const int i = (t - 1) & 1;
              const unsigned k = n + t - 1;
              if (!wait(&sh.vready[k % kBufs], (k / kBufs) & 1) || !wait(&sh.pready[i], n_s[i] & 1)) break;
              ++n_s[i];
              tc_fence_after();
              outputs(i, k, t <= 2);
              tc_commit(&sh.vfree[k % kBufs]);
              if (t - 1 + 2 >= tiles) tc_commit(&sh.oready[i]);
            }
          }
          n += tiles;
        }
      }
      if (!ok) {  // no MMA of this block is in flight when it frees its tensor memory
        tc_commit(&sh.drain);
        (void)mbar_wait_bounded(&sh.drain, 0);
      }
    }
    __syncwarp();
  } else if (warp >= kConvertWarp) {
    // ---- conversion: warp w takes block w of a tile ----
    const int w = warp - kConvertWarp;
    unsigned n = 0;
    bool ok = true;
    while (ok && next_segment<R, kTile>(a, slice, at, b, before, seg)) {
      const int len = seg.r.len, total = len + seg.r.nodes;
      for (int t = seg.u0; t < seg.u1; ++t, ++n) {
        const int s = n % kStages, k = n % kBufs;
        ok = role_wait(&sh.full[s], (n / kStages) & 1, dead, a.status);
        if (ok && n >= kBufs) ok = role_wait(&sh.kfree[k], (n / kBufs - 1) & 1, dead, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        {
          const uint8_t* src = smem + s * S::STAGE + w * (kBlock * D);
          uint8_t* dst = smem + S::K_OFF + k * S::KTILE;
          // unit (nt, kh, g, tig): 16 channels of token 8nt + g; a quarter of the warp takes 8 tokens of one
          // core matrix, their tig rotated so that neither the reads nor the writes meet in a bank
          const int q4 = lane >> 3, g3 = lane & 3, nt = (lane >> 2) & 1, tig = (q4 + (g3 >> 1) + 2 * nt) & 3;
          const int v8 = 4 * (g3 >> 1) + 2 * nt + (g3 & 1);  // row of the core matrix
#pragma unroll
          for (int kh = 0; kh < D / 64; ++kh)
#pragma unroll
            for (int gs = 0; gs < 2; ++gs) {
              const int g = g3 + 4 * gs;
              const uint4 x = *reinterpret_cast<const uint4*>(src + ((nt * (D / 64) + kh) * 32 + 4 * g + tig) * 16);
              uint8_t* d = dst + ((kh * 4 + tig) * 2) * (kTile * 16) + (2 * w + gs) * 128 + v8 * 16;
              *reinterpret_cast<uint4*>(d) =
                  make_uint4(fp8_lo_pair<FMT>(x.x), fp8_hi_pair<FMT>(x.x), fp8_lo_pair<FMT>(x.y), fp8_hi_pair<FMT>(x.y));
              *reinterpret_cast<uint4*>(d + kTile * 16) =
                  make_uint4(fp8_lo_pair<FMT>(x.z), fp8_hi_pair<FMT>(x.z), fp8_lo_pair<FMT>(x.w), fp8_hi_pair<FMT>(x.w));
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.kready[k]);
        if (n >= kBufs) ok = role_wait(&sh.vfree[k], (n / kBufs - 1) & 1, dead, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        {
          const uint8_t* src = smem + s * S::STAGE + kTile * D + w * (kBlock * D);
          uint8_t* dst = smem + S::V_OFF + k * S::KTILE;
          // unit (c, g, tig): tokens 2tig, 2tig + 1, 8 + 2tig, 9 + 2tig of channels 8 (4c + j) + g
          const int half = lane >> 4, g = (lane >> 1) & 7, tig = 2 * (half ^ ((g >> 1) & 1)) + (lane & 1);
          const int tok0 = t * kTile + w * kBlock;
          const bool edge = tok0 + kBlock > len;  // the tree's own tokens, and rows behind them
          uint32_t keep = 0xFFFFFFFFu, tree_bytes = 0;
          if (edge) {
            keep = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int tok = tok0 + 8 * (i >> 1) + 2 * tig + (i & 1);
              if (tok < total) keep |= 0xFFu << (8 * i);
              if (tok >= len) tree_bytes |= 0xFFu << (8 * i);
            }
          }
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            const uint4 x = *reinterpret_cast<const uint4*>(src + (c * 32 + 4 * g + tig) * 16);
            uint32_t word[4] = {x.x, x.y, x.z, x.w};
            if (edge) {
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t bad = fp8_nonfinite<FMT>(word[j]) & tree_bytes & keep;
                if (bad != 0) sh.nan_met = 1;
                word[j] &= keep & ~bad;
              }
            }
            uint8_t* d = dst + (2 * w + (tig >> 1)) * (D * 16) + (4 * c) * 128 + g * 16 + (tig & 1) * 8;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              *reinterpret_cast<uint2*>(d + j * 128) = make_uint2(fp8_lo_pair<FMT>(word[j]), fp8_hi_pair<FMT>(word[j]));
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh.vready[k]);
          mbar_arrive(&sh.empty[s]);
        }
      }
    }
  } else {
    // ---- softmax: stream `i`, a thread per query row ----
    const int i = warp >> 2, row = tid & 127;
    const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t tm_s = tmem + lanes + TM_S + i * S_COLS;
    unsigned n = 0, o_seen[2] = {0, 0};  // tiles of this stream; results of each stream waited for
    bool ok = true;
    while (next_segment<R, kTile>(a, slice, at, b, before, seg)) {
      const int h = seg.h, len = seg.r.len, total = len + seg.r.nodes, row0 = seg.tile * R;
      const int rows = min(R, seg.r.nodes * gq - row0);       // of the tile
      const int my_rows = SPLIT_ROWS ? min(128, rows - 128 * i) : rows;  // of this stream (may be below 1)
      const int trow = SPLIT_ROWS ? row + 128 * i : row;      // row of the tile
      const bool live = row < my_rows;
      const bool warp_live = (row & ~31) < my_rows;
      const int node = live ? (row0 + trow) / gq : 0;
      const float k_scale = a.k_scale[a.per_head ? h : 0], v_scale = a.v_scale[a.per_head ? h : 0];
      // a negative scale turns the query's signs, so that larger scores stay larger
      float kmul = fabsf(k_scale) * a.scale_log2;
      if (kmul == 0.0f) kmul = 1e-37f;
      const uint32_t flip = k_scale < 0.0f ? 0x80008000u : 0u;
      const uint64_t* mask = a.tree_mask + static_cast<long long>(seg.r.first + node) * a.mask_words;

      if (ok) {  // the query row, its channels in the key units' order
        const __half* q = reinterpret_cast<const __half*>(a.q) + (seg.r.first + node) * a.q_stride +
                          static_cast<long long>(h * gq + (live ? (row0 + trow) % gq : 0)) * D;
#pragma unroll
        for (int kh = 0; kh < D / 64; ++kh) {
          uint32_t w[32];
#pragma unroll
          for (int c4 = 0; c4 < 16; ++c4) {  // place 4 c4 of this half: channels 64kh + 16 (c4 % 4) + 4 (c4 / 4) .. +3
            uint2 x = make_uint2(0u, 0u);
            if (live) x = *reinterpret_cast<const uint2*>(q + 64 * kh + 16 * (c4 % 4) + 4 * (c4 / 4));
            w[2 * c4] = x.x ^ flip;
            w[2 * c4 + 1] = x.y ^ flip;
          }
          tmem_st32(tmem + lanes + TM_Q + i * Q_COLS + 32 * kh, w);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.qready[i]);
      }

      float m = -INFINITY, msub = -kBias, l = 0.0f;  // m in log2 units; weights are 2^(s * kmul - msub)
      const int step = SPLIT_ROWS ? 1 : 2;
      for (int t = seg.u0 + (SPLIT_ROWS ? 0 : i); ok && t < seg.u1; t += step, ++n) {
        ok = role_wait(&sh.sready[i], n & 1, dead, a.status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (warp_live) {
          uint32_t sr[kTile];
          tmem_ld32(tm_s, sr);
          tmem_ld32(tm_s + 32, sr + 32);
          const int tok0 = t * kTile;
          const bool edge = tok0 + kTile > len;
          uint64_t vis = ~0ull;
          if (edge) vis = tree_window(mask, a.mask_words, tok0, len, total);
          tmem_wait_ld();
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if (edge) {
#pragma unroll
            for (int c = 0; c < kTile; ++c)
              if (!((vis >> column_token(c)) & 1)) sr[c] = 0xFF800000u;
          }
#pragma unroll
          for (int c = 0; c < kTile; ++c) mx[c & 3] = fmaxf(mx[c & 3], __uint_as_float(sr[c]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * kmul;
          // grown beyond the slack (or from nothing): take the new maximum, bring what was summed to it
          const bool grow = top > m + kSlack || (m == -INFINITY && top > m);
          if (__any_sync(0xffffffffu, grow)) {
            const float m_new = grow ? top : m;
            const float alpha = grow ? fast_exp2(m - m_new) : 1.0f;
            l *= alpha;
            m = m_new;
            msub = (m == -INFINITY ? 0.0f : m) - kBias;
            if (t >= seg.u0 + step) {  // O holds something; the scores of this tile came after its last product
#pragma unroll 1
              for (int c0 = 0; c0 < D; c0 += 16) {
                uint32_t o[16];
                tmem_ld16(tmem + lanes + TM_O + i * D + c0, o);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 16; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                tmem_st16(tmem + lanes + TM_O + i * D + c0, o);
              }
            }
          }
          float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          // (all scores are in registers: the weights may go over their columns)
#pragma unroll
          for (int c0 = 0; c0 < kTile; c0 += 32) {
            uint32_t hi[16], lo[WIDE ? 16 : 1];
#pragma unroll
            for (int c = 0; c < 32; c += 2) {
              const float p0 = fast_exp2(fmaf(__uint_as_float(sr[c0 + c]), kmul, -msub));
              const float p1 = fast_exp2(fmaf(__uint_as_float(sr[c0 + c + 1]), kmul, -msub));
              sum[c & 2] += p0;
              sum[(c & 2) + 1] += p1;
              const __half2 p = __floats2half2_rn(p0, p1);
              hi[c / 2] = h2_bits(p);
              if constexpr (WIDE) {
                const float2 f = __half22float2(p);
                lo[c / 2] = pack_rn_f16x2(p0 - f.x, p1 - f.y);
              }
            }
            tmem_st16(tm_s + c0 / 2, hi);
            if constexpr (WIDE) tmem_st16(tm_s + kTile / 2 + c0 / 2, lo);
          }
          l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh.pready[i]);
      }

      // ---- the segment's result ----
      const bool have1 = SPLIT_ROWS || seg.u1 - seg.u0 > 1;  // stream 1 had tiles
      if constexpr (!SPLIT_ROWS) {
        sh.ml[i][row][0] = m;
        sh.ml[i][row][1] = l;
      }
      // (with rows split a stream reads its own outputs only)
      if (!SPLIT_ROWS || i == 0) {
        ok = ok && role_wait(&sh.oready[0], o_seen[0] & 1, dead, a.status);
        ++o_seen[0];
      }
      if (have1 && (!SPLIT_ROWS || i == 1)) {
        ok = ok && role_wait(&sh.oready[1], o_seen[1] & 1, dead, a.status);
        ++o_seen[1];
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
          const float m0 = sh.ml[0][row][0], l0 = sh.ml[0][row][1], m1 = sh.ml[1][row][0], l1 = sh.ml[1][row][1];
          M = fmaxf(m0, m1);
          // (a stream without a maximum has the sum 0, or NaN, which stays)
          f0 = M == -INFINITY ? 1.0f : fast_exp2(m0 - M);
          f1 = M == -INFINITY ? 1.0f : fast_exp2(m1 - M);
          L = l0 * f0 + l1 * f1;
        }
        const float f = whole ? (L == 0.0f ? 0.0f : v_scale / L) : 1.0f;
        const long long prow = static_cast<long long>(seg.slot) * R + trow;
        if (warp_live) {
#pragma unroll 1
          for (int c0 = c_begin; c0 < c_begin + COLS; c0 += 16) {
            uint32_t o[16], o1[SPLIT_ROWS ? 1 : 16];
            tmem_ld16(tmem + lanes + TM_O + (SPLIT_ROWS ? i * D : 0) + c0, o);
            if constexpr (!SPLIT_ROWS) {
              if (have1) tmem_ld16(tmem + lanes + TM_O + D + c0, o1);
            }
            tmem_wait_ld();
            if (!live) continue;
#pragma unroll
            for (int c = 0; c < 16; c += 4) {
              float v[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                v[e] = __uint_as_float(o[c + e]) * f0;
                if constexpr (!SPLIT_ROWS) {
                  if (have1) v[e] = fmaf(__uint_as_float(o1[c + e]), f1, v[e]);
                }
                v[e] *= f;
              }
              const float4 x = make_float4(v[0], v[1], v[2], v[3]);
              if (whole)
                tree_store4<D>(a, seg, gq, row0 + trow, (c0 + c) / 4, x);
              else
                *reinterpret_cast<float4*>(a.part_o + prow * D + c0 + c) = x;
            }
          }
          if (whole && live && nan_met) tree_put_nan<D, FMT>(a, seg, gq, row0 + trow, c_begin, c_begin + COLS);
          if (!whole && live && (SPLIT_ROWS || i == 0))
            *reinterpret_cast<float2*>(a.part_ml + prow * 2) = make_float2(M, L);
        }
        tc_fence_before();
      }
      if (!whole) {
        if (tid == 0) a.part_flag[seg.slot] = sh.nan_met;
        __threadfence();
        named_barrier(1, 256);
        if (tid == 0) {
          const bool last = atomicAdd(a.counters + seg.first_block, 1u) == static_cast<uint32_t>(seg.parts - 1);
          if (last) a.counters[seg.first_block] = 0u;
          sh.last = last;
        }
        named_barrier(1, 256);
        if (sh.last && ok) {
          __threadfence();
          tree_merge<R, D, FMT>(a, seg, slice, gq, rows, v_scale, sh.merge, tid, 256, [] { named_barrier(1, 256); });
        }
        named_barrier(1, 256);  // sh.last and sh.merge are free again
      }
    }
  }
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int FMT, bool WIDE, int R>
cudaError_t launch_tc(const TreeArgs& a, cudaStream_t s) {
  constexpr int smem = TcSmem<D>::BYTES;
  auto kern = tree_tc_kernel<D, FMT, WIDE, R>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  constexpr int kMost = kTreePartRows / (2 * R);  // blocks whose partial results fit the workspace
  static_assert(kMost <= kTreeMaxBlocks, "their counters too");
  const int sms = device_sm_count();
  kern<<<sms < kMost ? sms : kMost, kThreads, smem, s>>>(a);
  return cudaGetLastError();
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
  return a.max_tree * (a.q_heads / a.kv_heads) <= 128 ? dispatch_tc<128>(a, s) : dispatch_tc<256>(a, s);
}

}  // namespace kvq
