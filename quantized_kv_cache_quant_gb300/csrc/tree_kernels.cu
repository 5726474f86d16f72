// Attention of a tree of drafted tokens over the paged FP8 cache (kvq_spec.h).
#include "tree_plan.cuh"

namespace kvq {
namespace {

constexpr int kBlock = 16;  // tokens of an FP8 pool block

// ---------------------------------------------------------------------------
// Few rows: 16 query rows a tile on mma.sync m16n8k16, the rows on the MMA's
// 16-row side. Four warps; warp w takes every fourth block of the segment
// through its own ring of bulk copies, with its own running maximum, sum and
// outputs, joined at the end of the segment.
//   q.k^T: A = q (channels permuted as the keys' order), B = the keys as fp16
//   p.V  : A = p rounded to fp16 and, on a second product, what the rounding
//          left (2^-22 of p, as the decode of one token), B = the values as fp16
// p carries a factor 2^kBias so that weights down to 2^-24 of the largest stay
// normal fp16 numbers.
// Bound by the memory: 32 requests x 32768 tokens, 8 heads, D = 128, 16 rows in
// 370 us on random pages, 5.8 TB/s, 85 % of the measured copy rate (383 us with
// cold caches, 375 with p in one part); three blocks an SM (168 registers) keep
// four copies of 4 KB a warp in flight. A tile of 32 rows on this layout spilled
// and took a third longer than tcgen05 for chains of 4 over 128K tokens.
// ---------------------------------------------------------------------------
constexpr int kRows = 16;
constexpr int kUnit = 64;    // tokens of a unit: one block a warp
constexpr int kStages = 4;
constexpr float kBias = 10.0f;

template <int D>
struct TreeSmem {
  static constexpr int BAR_BYTES = 128;
  static constexpr int STAGE = 2 * kBlock * D;
  static constexpr int RING = 4 * kStages * STAGE;
  static constexpr int COMBINE = 4 * kRows * (D + 2) * 4;
  static constexpr int AREA = RING > COMBINE ? RING : COMBINE;
  static constexpr int BYTES = BAR_BYTES + AREA;
};

template <int D, int FMT>
__global__ void __launch_bounds__(128) tree_rows16_kernel(const __grid_constant__ TreeArgs a) {
  using S = TreeSmem<D>;
  constexpr int KS = D / 16, NT = D / 8, CH = D / 32;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ unsigned long long plan_s[36];
  __shared__ int nan_s;
  // the arguments and the slice, for functions out of line (a reference to a kernel's parameters is read from global
  // memory there)
  __shared__ TreeArgs args_s;
  __shared__ TreeSlice slice_s;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
  uint8_t* area = smem + S::BAR_BYTES;
  float* o_s = reinterpret_cast<float*>(area);   // [4][16][D]
  float* m_s = o_s + 4 * kRows * D;              // [4][16]
  float* l_s = m_s + 4 * kRows;                  // [4][16]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
  const int gq = a.q_heads / a.kv_heads;
  uint64_t* bar = bars + warp * kStages;
  uint8_t* ring = area + warp * kStages * S::STAGE;
  if (lane == 0) {
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(&bar[s], 1);
    fence_mbar_init();
  }
  if (tid == 0) tree_leave_none(a);
  // (one request of 2500 tokens: slices of 4 units 15.5 us, of 2 18.1; of 400 tokens: 13.5 and 12.4)
  const TreeSlice slice = tree_slice<kRows, kUnit>(
      a, plan_s, [](long long pair) { return pair >= 32 ? 4 : 2; }, [](long long u) { return u >= 4 ? 4 : 2; });
  if (slice.begin >= slice.end) return;

  if (tid == 0) {
    args_s = a;
    slice_s = slice;
  }
  __syncthreads();
  TreeWalk walk;
  walk.start(slice);
  const TreeSegment& seg = walk.seg;
  unsigned it = 0;         // blocks this warp has taken through its ring
  bool dead = false;       // a wait ran out: no more copies
  while (next_segment<kRows, kUnit>(args_s, slice_s, walk)) {
    const int h = seg.h, len = seg.r.len, total = len + seg.r.nodes, row0 = seg.tile * kRows;
    const int rows = min(kRows, seg.r.nodes * gq - row0);
    const int nblk = tree_units(total, kBlock);
    const int j_begin = seg.u0 * 4, j_end = min(seg.u1 * 4, nblk);
    const int n_mine = (!dead && j_end - j_begin > warp) ? (j_end - j_begin - warp + 3) / 4 : 0;
    const int32_t* table = a.block_table + static_cast<long long>(seg.b) * a.max_blocks;
    auto phys = [&](int j) -> long long {
      return min(max(table[j_begin + warp + 4 * j], 0), a.num_blocks - 1);
    };
    auto issue = [&](int j, long long blk) {
      const long long off = (blk * a.kv_heads + h) * (kBlock * D);
      const int s = (it + j) % kStages;
      uint8_t* dst = ring + s * S::STAGE;
      mbar_arrive_expect_tx(&bar[s], S::STAGE);
      bulk_g2s(dst, a.k_pool + off, kBlock * D, &bar[s]);
      bulk_g2s(dst + kBlock * D, a.v_pool + off, kBlock * D, &bar[s]);
    };
    if (lane == 0) {
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      for (int j = 0; j < kStages && j < n_mine; ++j) issue(j, phys(j));
    }
    if (tid == 0) nan_s = 0;

    // query rows g and g + 8 of the tile, A fragments of m16n8k16
    uint32_t qa[KS][4];
    const uint64_t* mask[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = row0 + g + 8 * e;
      const bool ok = g + 8 * e < rows;
      const int n = seg.r.first + (ok ? r / gq : 0);
      mask[e] = a.tree_mask + static_cast<long long>(n) * a.mask_words;
      const __half* qrow = reinterpret_cast<const __half*>(a.q) + n * a.q_stride +
                           static_cast<long long>(h * gq + (ok ? r % gq : 0)) * D;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint2 w = ok ? *reinterpret_cast<const uint2*>(qrow + 16 * ks + 4 * tig) : make_uint2(0u, 0u);
        qa[ks][e] = w.x;
        qa[ks][2 + e] = w.y;
      }
    }
    const float kmul = a.k_scale[a.per_head ? h : 0] * a.scale_log2;
    const float vscale = a.v_scale[a.per_head ? h : 0];

    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};
    float o_acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) o_acc[i][0] = o_acc[i][1] = o_acc[i][2] = o_acc[i][3] = 0.0f;
    bool nan_met = false;

    int j = 0;
    bool timed_out = false;
    for (; j < n_mine; ++j) {
      const int s = (it + j) % kStages;
      const long long next_blk = (lane == 0 && j + kStages < n_mine) ? phys(j + kStages) : 0;
      if (__any_sync(0xffffffffu, !mbar_wait_bounded(&bar[s], ((it + j) / kStages) & 1))) {
        timed_out = true;
        break;
      }
      const uint4* kb = reinterpret_cast<const uint4*>(ring + s * S::STAGE);
      const uint4* vb = reinterpret_cast<const uint4*>(ring + s * S::STAGE + kBlock * D);
      const int tok_base = (j_begin + warp + 4 * j) * kBlock;
      uint32_t kw[2 * KS];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint4 x = kb[c * 32 + lane];
        kw[4 * c] = x.x;
        kw[4 * c + 1] = x.y;
        kw[4 * c + 2] = x.z;
        kw[4 * c + 3] = x.w;
      }
      float sacc[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt) {
        sacc[nt][0] = sacc[nt][1] = sacc[nt][2] = sacc[nt][3] = 0.0f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          const uint32_t w = kw[nt * KS + ks];
          mma16816(sacc[nt], qa[ks][0], qa[ks][1], qa[ks][2], qa[ks][3], fp8_lo_pair<FMT>(w), fp8_hi_pair<FMT>(w));
        }
      }
      uint32_t vw[NT];
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const uint4 x = vb[c * 32 + lane];
        vw[4 * c] = x.x;
        vw[4 * c + 1] = x.y;
        vw[4 * c + 2] = x.z;
        vw[4 * c + 3] = x.w;
      }
      // scores of rows g (sc[0]) and g + 8 (sc[1]): tokens 2tig, 2tig + 1, 8 + 2tig, 9 + 2tig
      float sc[2][4];
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[e][i] = sacc[i >> 1][2 * e + (i & 1)] * kmul;
      if (tree_beyond(tok_base, kBlock, len)) {  // the tree's own tokens, and rows behind them
        uint32_t keep = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = tok_base + 8 * (i >> 1) + 2 * tig + (i & 1);
          if (tok < total) keep |= 0xFFu << (8 * i);
#pragma unroll
          for (int e = 0; e < 2; ++e)
            if (!tree_sees(mask[e], tok, len, total)) sc[e][i] = -INFINITY;
        }
        // context tokens are seen by every row: their NaN codes stay as they are
        uint32_t tree_bytes = keep;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (tok_base + 8 * (i >> 1) + 2 * tig + (i & 1) < len) tree_bytes &= ~(0xFFu << (8 * i));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t bad = fp8_nonfinite<FMT>(vw[nt]) & tree_bytes;
          nan_met |= bad != 0;
          vw[nt] &= keep & ~bad;
        }
      }
      uint32_t A[4], L[4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float mx = quad_max(fmaxf(fmaxf(sc[e][0], sc[e][1]), fmaxf(sc[e][2], sc[e][3])));
        const float m_new = fmaxf(m_run[e], mx);
        if (m_new != m_run[e]) {
          const float alpha = fast_exp2(m_run[e] - m_new);
          l_run[e] *= alpha;
#pragma unroll
          for (int i = 0; i < NT; ++i) {
            o_acc[i][2 * e] *= alpha;
            o_acc[i][2 * e + 1] *= alpha;
          }
          m_run[e] = m_new;
        }
        const float sub = (m_new == -INFINITY ? 0.0f : m_new) - kBias;
        float p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = fast_exp2(sc[e][i] - sub);
        l_run[e] += (p[0] + p[1]) + (p[2] + p[3]);
        const __half2 h0 = __floats2half2_rn(p[0], p[1]), h1 = __floats2half2_rn(p[2], p[3]);
        A[e] = h2_bits(h0);
        A[2 + e] = h2_bits(h1);
        const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
        L[e] = pack_rn_f16x2(p[0] - f0.x, p[1] - f0.y);
        L[2 + e] = pack_rn_f16x2(p[2] - f1.x, p[3] - f1.y);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint32_t b0 = fp8_lo_pair<FMT>(vw[nt]), b1 = fp8_hi_pair<FMT>(vw[nt]);
        mma16816(o_acc[nt], A[0], A[1], A[2], A[3], b0, b1);
        mma16816(o_acc[nt], L[0], L[1], L[2], L[3], b0, b1);
      }
      __syncwarp();
      if (lane == 0 && j + kStages < n_mine) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        issue(j + kStages, next_blk);
      }
    }
    if (timed_out) {
      if (lane == 0) report_timeout(a.status);
      for (int jj = j; jj < n_mine && jj < j + kStages; ++jj)
        (void)mbar_wait_bounded(&bar[(it + jj) % kStages], ((it + jj) / kStages) & 1);
      dead = true;
      m_run[0] = m_run[1] = -INFINITY;
      l_run[0] = l_run[1] = 0.0f;
#pragma unroll
      for (int i = 0; i < NT; ++i) o_acc[i][0] = o_acc[i][1] = o_acc[i][2] = o_acc[i][3] = 0.0f;
    }
    it += n_mine;
    l_run[0] = quad_sum(l_run[0]);
    l_run[1] = quad_sum(l_run[1]);

    __syncthreads();  // all rings are drained: their memory takes the warps' results
    if (nan_met) nan_s = 1;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = warp * kRows + g + 8 * e;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<float2*>(o_s + r * D + 8 * nt + 2 * tig) = make_float2(o_acc[nt][2 * e], o_acc[nt][2 * e + 1]);
      if (tig == 0) {
        m_s[r] = m_run[e];
        l_s[r] = l_run[e];
      }
    }
    __syncthreads();
    constexpr int V = D / 4;
    const bool whole = seg.parts == 1;
    for (int i = tid; i < rows * V; i += 128) {
      const int r = i / V, c4 = i % V;
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < 4; ++w) M = fmaxf(M, m_s[w * kRows + r]);
      float L = 0.0f;
      float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        // (a warp without a maximum has the sum 0, or NaN, which stays)
        const float f = M == -INFINITY ? 1.0f : fast_exp2(m_s[w * kRows + r] - M);
        const float4 x = *reinterpret_cast<const float4*>(o_s + (w * kRows + r) * D + 4 * c4);
        L = fmaf(l_s[w * kRows + r], f, L);
        o.x = fmaf(x.x, f, o.x);
        o.y = fmaf(x.y, f, o.y);
        o.z = fmaf(x.z, f, o.z);
        o.w = fmaf(x.w, f, o.w);
      }
      if (whole) {
        const float f = L == 0.0f ? 0.0f : vscale / L;
        tree_store4<D>(a, seg, gq, row0 + r, c4, make_float4(o.x * f, o.y * f, o.z * f, o.w * f));
        if (nan_s) tree_put_nan<D, FMT>(args_s, seg.b, h, seg.r.first, seg.r.nodes, len, row0 + r, 4 * c4, 4 * c4 + 4);
      } else {
        const long long row = static_cast<long long>(seg.slot) * kRows + r;
        *reinterpret_cast<float4*>(a.part_o + row * D + 4 * c4) = o;
        if (c4 == 0) *reinterpret_cast<float2*>(a.part_ml + row * 2) = make_float2(M, L);
      }
    }
    if (!whole && tid == 0) {
      a.part_flag[seg.slot] = nan_s;
      if (seg.u0 == 0) tree_leave_join(args_s, seg, rows, row0);
    }
    __syncthreads();  // the next segment's copies overwrite what was read here
  }
}

template <int D, int FMT>
cudaError_t launch_rows16(const TreeArgs& a, cudaStream_t s) {
  constexpr int smem = TreeSmem<D>::BYTES;
  auto kern = tree_rows16_kernel<D, FMT>;
  static SharedMemoryOnce once;
  int per_sm = 0;
  cudaError_t e = once.set(kern, smem, 128, &per_sm);
  if (e != cudaSuccess) return e;
  int grid = device_sm_count() * per_sm;
  if (grid > kTreeMaxBlocks) grid = kTreeMaxBlocks;
  kern<<<grid, 128, smem, s>>>(a);
  e = cudaGetLastError();
  return e != cudaSuccess ? e : launch_tree_join(a, grid, kRows, s);
}

// ---------------------------------------------------------------------------
// Joining of partial results: block (c, y) takes what block c of the attention
// left, rows 32 y .. +31, a warp four of them. Lanes weigh a row's parts (log2
// units), then the rows' outputs are added up part by part, all four rows and
// two parts in flight. A second launch costs some 4 us; the last block of a pair
// joining its parts inside the attention (fence, counter, then cold reads) took
// 8 to 16.
// ---------------------------------------------------------------------------
template <int D, int FMT>
__global__ void __launch_bounds__(256) tree_join_kernel(const __grid_constant__ TreeArgs a, int tile_rows) {
  constexpr int V = D / 32;  // floats of a row a lane holds
  constexpr int kJoinRows = 4;
  const TreeJoin j = a.joins[blockIdx.x];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r0 = 32 * blockIdx.y + kJoinRows * warp;
  if (j.parts == 0 || r0 >= j.rows) return;
  const int gq = a.q_heads / a.kv_heads;
  const float v_scale = a.v_scale[a.per_head ? j.h : 0];
  auto slot_of = [&](int i) { return i == 0 ? j.slot0 : (j.slot0 & ~1) + 2 * i; };
  // (a part without a maximum has the sum 0, or NaN, which stays)
  float M[kJoinRows], L[kJoinRows], w[kJoinRows], acc[kJoinRows][V];
#pragma unroll
  for (int k = 0; k < kJoinRows; ++k) {
    M[k] = -INFINITY;
    L[k] = 0.0f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[k][e] = 0.0f;
  }
  bool nan_met = false;
  for (int i0 = 0; i0 < j.parts; i0 += 32) {
    const int i = i0 + lane, n = min(32, j.parts - i0);
    float2 ml[kJoinRows];
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {  // (rows behind the last one are within the slot: tiles hold a multiple of 4)
      ml[k] = make_float2(-INFINITY, 0.0f);
      if (i < j.parts)
        ml[k] = reinterpret_cast<const float2*>(a.part_ml)[static_cast<long long>(slot_of(i)) * tile_rows + r0 + k];
    }
    if (i < j.parts) nan_met |= a.part_flag[slot_of(i)] != 0;
#pragma unroll
    for (int k = 0; k < kJoinRows; ++k) {
      const float Mn = fmaxf(M[k], warp_max(ml[k].x));
      const float old = Mn == -INFINITY ? 1.0f : fast_exp2(M[k] - Mn);
      w[k] = Mn == -INFINITY ? 1.0f : fast_exp2(ml[k].x - Mn);
      L[k] = L[k] * old + warp_sum(ml[k].y * w[k]);
      M[k] = Mn;
#pragma unroll
      for (int e = 0; e < V; ++e) acc[k][e] *= old;
    }
#pragma unroll 2
    for (int p = 0; p < n; ++p) {
      const float* o = a.part_o + (static_cast<long long>(slot_of(i0 + p)) * tile_rows + r0) * D + V * lane;
      float v[kJoinRows][V];
#pragma unroll
      for (int k = 0; k < kJoinRows; ++k) {
        if constexpr (V == 4) {
          const float4 x = *reinterpret_cast<const float4*>(o + k * D);
          v[k][0] = x.x, v[k][1] = x.y, v[k][2] = x.z, v[k][3] = x.w;
        } else {
          const float2 x = *reinterpret_cast<const float2*>(o + k * D);
          v[k][0] = x.x, v[k][1] = x.y;
        }
      }
#pragma unroll
      for (int k = 0; k < kJoinRows; ++k) {
        const float wp = __shfl_sync(0xffffffffu, w[k], p);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[k][e] = fmaf(v[k][e], wp, acc[k][e]);
      }
    }
  }
  nan_met = __any_sync(0xffffffffu, nan_met);
#pragma unroll
  for (int k = 0; k < kJoinRows; ++k) {
    if (r0 + k < j.rows) {
      const float f = L[k] == 0.0f ? 0.0f : v_scale / L[k];
      const int row = j.row0 + r0 + k, node = row / gq;
      const long long at = (static_cast<long long>(j.first + node) * a.q_heads + j.h * gq + (row - node * gq)) * D + V * lane;
#pragma unroll
      for (int e = 0; e < V; e += 2) {
        if (a.out_fp32)
          *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at + e) = make_float2(acc[k][e] * f, acc[k][e + 1] * f);
        else
          *reinterpret_cast<uint32_t*>(reinterpret_cast<__half*>(a.out) + at + e) = pack_rn_f16x2(acc[k][e] * f, acc[k][e + 1] * f);
      }
      if (nan_met) tree_put_nan<D, FMT>(a, j.b, j.h, j.first, j.nodes, j.len, row, V * lane, V * lane + V);
    }
  }
}

}  // namespace

cudaError_t launch_tree_join(const TreeArgs& a, int blocks, int tile_rows, cudaStream_t s) {
  // rows that a tile of these requests can have
  const int most = a.max_tree * (a.q_heads / a.kv_heads), rows = most < tile_rows ? most : tile_rows;
  const dim3 grid(blocks, (rows + 31) / 32);
  switch (a.head_dim * 10 + a.fmt) {
    case 1280: tree_join_kernel<128, 0><<<grid, 256, 0, s>>>(a, tile_rows); break;
    case 1281: tree_join_kernel<128, 1><<<grid, 256, 0, s>>>(a, tile_rows); break;
    case 640: tree_join_kernel<64, 0><<<grid, 256, 0, s>>>(a, tile_rows); break;
    case 641: tree_join_kernel<64, 1><<<grid, 256, 0, s>>>(a, tile_rows); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t s) {
  // Up to 16 rows a kv head, and little work altogether: few tiles of 16 rows over at most 2560 tokens, where the wider
  // kernel's longer change of segments decides (8 heads, one request: trees of 5 at 1000 tokens 14.0 us here and 15.7
  // there, of 32 17.8 and 24.4, at 2500 tokens 24.5 and 24.7, at 5000 32.1 and 29.9; 16 requests at 1000 27 and 23).
  const int rows = a.max_tree * (a.q_heads / a.kv_heads);
  const long long tiles = static_cast<long long>(a.batch) * a.kv_heads * ((rows + kRows - 1) / kRows);
  if (rows > kRows && (tiles > 64 || a.max_seq_len > 2560)) return launch_tree_tc(a, s);
  static_assert(2 * kTreeMaxBlocks * kRows <= kTreePartRows, "partial results fit the workspace");
  switch (a.head_dim * 10 + a.fmt) {
    case 1280: return launch_rows16<128, 0>(a, s);
    case 1281: return launch_rows16<128, 1>(a, s);
    case 640: return launch_rows16<64, 0>(a, s);
    case 641: return launch_rows16<64, 1>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
