// Decode attention of sequences that share leading blocks, over the paged FP8
// cache (kvq_beam.h): few query rows a kv head, and the joining of results.
#include "group_plan.cuh"

namespace kvq {
namespace {

constexpr int kBlock = 16;  // tokens of an FP8 pool block

// ---------------------------------------------------------------------------
// 16 query rows a tile on mma.sync m16n8k16, the rows on the MMA's 16-row side:
// as tree attention's kernel of few rows, without a mask. Four warps; warp w
// takes every fourth block of the segment, with its own running maximum, sum and
// outputs, joined at the segment's end. A block's bytes are in operand order, so
// that each lane needs 16-byte units of its own: it copies them into its part of
// a ring in shared memory, some blocks ahead, and nobody waits for anyone else.
//   q.k^T: A = q (channels permuted as the keys' order), B = the keys as fp16
//   p.V  : A = p rounded to fp16 and, on a second product, what the rounding
//          left (2^-22 of p), B = the values as fp16
// p carries a factor 2^kBias so that weights down to 2^-24 of the largest stay
// normal fp16 numbers.
//
// 8 x 4 sequences over 32K shared tokens (16 rows a kv head, 128 channels): 113 us
// with the joining, 4.8 TB/s; 64 own sequences of 8K tokens 197 us, 5.4 TB/s;
// lengths of all kinds with 64 channels 84 us, 3.1 TB/s. Long segments run at the
// memory's rate; what is added to that are each wave's start (3 us of plan, then
// three dependent reads: request, table, block, some 5 us, which a thread block
// has at every segment) and the waves' last thread blocks, which end 10 us after
// the mean. Six stages (92 us in place of 86) and five blocks an SM at 96
// registers (96) cost more than they hide; bulk copies and barriers for all four
// warps took 94, cuts that keep off a pair's ends by 1 or 2 units in place of 4
// the same or 2 us more.
// ---------------------------------------------------------------------------
constexpr int kRows = kGroupRows16;
constexpr int kUnit = 64;    // tokens of a unit: one block a warp
constexpr int kStages = 4;
constexpr float kBias = 10.0f;

template <int D>
struct GroupSmem {
  static constexpr int STAGE = 2 * kBlock * D;
  // blocks a warp takes at a time: with 64 channels there are registers for two, which share a maximum and its shuffles
  // (lengths of all kinds 86 -> 84 us; long segments alone as before)
  static constexpr int AT_ONCE = D == 64 ? 2 : 1;
  static_assert(kStages % AT_ONCE == 0, "the blocks taken at once lie behind each other in the ring");
  static constexpr int RING = 4 * kStages * STAGE;
  static constexpr int COMBINE = 4 * kRows * (D + 2) * 4;
  static constexpr int AREA = RING > COMBINE ? RING : COMBINE;
  static constexpr int BYTES = AREA;
};

// A launch lets the next one in at once: the own pairs start where the tcgen05 kernel's thread blocks have left, which
// they do not depend on, and the joining kernel has its rows' places ready. Each waits for the launch before it at its
// end (or where it needs its results), so that the last one's end is that of all.
__device__ __forceinline__ void let_next_in() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void wait_for_launch_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <int D, int FMT>
__global__ void __launch_bounds__(128) group_rows16_kernel(const __grid_constant__ GroupArgs a) {
  using S = GroupSmem<D>;
  constexpr int KS = D / 16, NT = D / 8, CH = D / 32, AT = S::AT_ONCE;
  let_next_in();
  const int kind = a.kinds == 3 ? static_cast<int>(blockIdx.y) : a.kinds - 1;  // (shared pairs first: they are the long ones)
  if (static_cast<int>(blockIdx.x) >= a.blocks[kind]) {
    wait_for_launch_before();
    return;
  }
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ unsigned long long plan_s[36];
  // the arguments and the slice, for functions out of line (a reference to a kernel's parameters is read from global
  // memory there)
  __shared__ GroupArgs args_s;
  __shared__ TreeSlice slice_s;
  uint8_t* area = smem;
  float* o_s = reinterpret_cast<float*>(area);   // [4][16][D]
  float* m_s = o_s + 4 * kRows * D;              // [4][16]
  float* l_s = m_s + 4 * kRows;                  // [4][16]

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, tig = lane & 3;
  const int gq = a.q_heads / a.kv_heads;
  uint8_t* ring = area + warp * kStages * S::STAGE + lane * 16;  // this lane's units
  // Thread blocks of their own for each kind, cut into slices of their own: own pairs are many and short, and a few blocks
  // would have nothing else if both kinds were cut as one (8 groups of 4 over 32K shared tokens: 267 us so, 121 apart).
  if (tid == 0) {
    args_s = a;
    args_s.kinds = 1 << kind;
  }
  __syncthreads();
  const TreeSlice slice = tree_slice<kRows, kUnit>(
      args_s, plan_s, [](long long pair) { return pair >= 32 ? 4 : 2; }, [](long long u) { return u >= 4 ? 4 : 2; });
  if (slice.begin >= slice.end) {
    wait_for_launch_before();
    return;
  }
  if (tid == 0) slice_s = slice;
  __syncthreads();
  GroupWalk walk;
  walk.start(slice);
  const GroupSegment& seg = walk.seg;
  int turn = 0;            // the warp whose turn it is to take a short segment alone
  while (next_segment<kRows, kUnit>(args_s, slice_s, walk)) {
    const int h = seg.h, total = seg.r.len, row0 = seg.tile * kRows;
    const int rows = min(kRows, seg.r.nodes * gq - row0);
    const int nblk = tree_units(total, kBlock);
    const int j_begin = seg.u0 * 4, j_end = min(seg.u1 * 4, nblk);
    // A short segment among others is one warp's alone, beside the other warps' segments, with no barriers: 2048 pairs of
    // 20 to 100 tokens took 47 us with all four warps at each of them.
    const int units = seg.u1 - seg.u0;
    const bool alone = units <= 4 && slice.end - slice.begin >= 3 * units;
    if (alone) {
      turn = (turn + 1) & 3;
      if (turn != warp) continue;
    }
    const int first = alone ? 0 : warp, step = alone ? 1 : 4;
    const int n_mine = j_end - j_begin > first ? (j_end - j_begin - first + step - 1) / step : 0;
    const int32_t* table = a.block_table + static_cast<long long>(seg.r.seq) * a.max_blocks + seg.r.block0;
    auto phys = [&](int j) -> long long {
      return j < n_mine ? min(max(table[j_begin + first + step * j], 0), a.num_blocks - 1) : 0;
    };
    auto issue = [&](int j, long long blk, uint8_t* dst) {
      if (j < n_mine) {
        const long long off = (blk * a.kv_heads + h) * (kBlock * D) + lane * 16;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          cp_async16(dst + c * 512, a.k_pool + off + c * 512);
          cp_async16(dst + kBlock * D + c * 512, a.v_pool + off + c * 512);
        }
      }
      cp_async_commit();
    };
    {
      long long blk[kStages];
#pragma unroll
      for (int j = 0; j < kStages; ++j) blk[j] = phys(j);
#pragma unroll
      for (int j = 0; j < kStages; ++j) issue(j, blk[j], ring + j * S::STAGE);
    }
    long long next_blk[AT];
#pragma unroll
    for (int b = 0; b < AT; ++b) next_blk[b] = phys(kStages + b);

    // query rows g and g + 8 of the tile, A fragments of m16n8k16
    uint32_t qa[KS][4];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int r = row0 + g + 8 * e;
      const bool ok = g + 8 * e < rows;
      const __half* qrow = reinterpret_cast<const __half*>(a.q) + (seg.r.first + (ok ? r / gq : 0)) * a.q_stride +
                           static_cast<long long>(h * gq + (ok ? r % gq : 0)) * D;
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        const uint2 w = ok ? *reinterpret_cast<const uint2*>(qrow + 16 * ks + 4 * tig) : make_uint2(0u, 0u);
        qa[ks][e] = w.x;
        qa[ks][2 + e] = w.y;
      }
    }
    const float kmul = a.k_scale[a.per_head ? h : 0] * a.scale_log2;

    float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};
    float o_acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i) o_acc[i][0] = o_acc[i][1] = o_acc[i][2] = o_acc[i][3] = 0.0f;

    for (int j = 0; j < n_mine; j += AT) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - AT) : "memory");
      uint8_t* const here = ring + j % kStages * S::STAGE;
      // scores of rows g (sc[0]) and g + 8 (sc[1]): tokens 2tig, 2tig + 1, 8 + 2tig, 9 + 2tig of each block
      float sc[2][4 * AT];
#pragma unroll
      for (int b = 0; b < AT; ++b) {
        const uint8_t* kb = here + b * S::STAGE;
        uint32_t kw[2 * KS];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(kb + c * 512);
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
#pragma unroll
        for (int e = 0; e < 2; ++e)
#pragma unroll
          for (int i = 0; i < 4; ++i) sc[e][4 * b + i] = sacc[i >> 1][2 * e + (i & 1)] * kmul;
      }
      uint32_t vw[AT][NT];
#pragma unroll
      for (int b = 0; b < AT; ++b) {
        const uint8_t* vb = here + b * S::STAGE + kBlock * D;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(vb + c * 512);
          vw[b][4 * c] = x.x;
          vw[b][4 * c + 1] = x.y;
          vw[b][4 * c + 2] = x.z;
          vw[b][4 * c + 3] = x.w;
        }
        // rows of the block behind the last token, and of a block that the warp does not have: not seen, values as 0
        const int tok_base = j + b < n_mine ? (j_begin + first + step * (j + b)) * kBlock : total;
        if (tree_beyond(tok_base, kBlock, total)) {
          uint32_t keep = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (tok_base + 8 * (i >> 1) + 2 * tig + (i & 1) < total) keep |= 0xFFu << (8 * i);
            else sc[0][4 * b + i] = sc[1][4 * b + i] = -INFINITY;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) vw[b][nt] &= keep;
        }
      }
      uint32_t A[AT][4], L[AT][4];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = fmaxf(fmaxf(sc[e][0], sc[e][1]), fmaxf(sc[e][2], sc[e][3]));
#pragma unroll
        for (int i = 4; i < 4 * AT; i += 2) mx = fmaxf(mx, fmaxf(sc[e][i], sc[e][i + 1]));
        mx = quad_max(mx);
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
#pragma unroll
        for (int b = 0; b < AT; ++b) {
          float p[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) p[i] = fast_exp2(sc[e][4 * b + i] - sub);
          l_run[e] += (p[0] + p[1]) + (p[2] + p[3]);
          const __half2 h0 = __floats2half2_rn(p[0], p[1]), h1 = __floats2half2_rn(p[2], p[3]);
          A[b][e] = h2_bits(h0);
          A[b][2 + e] = h2_bits(h1);
          const float2 f0 = __half22float2(h0), f1 = __half22float2(h1);
          L[b][e] = pack_rn_f16x2(p[0] - f0.x, p[1] - f0.y);
          L[b][2 + e] = pack_rn_f16x2(p[2] - f1.x, p[3] - f1.y);
        }
      }
#pragma unroll
      for (int b = 0; b < AT; ++b)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const uint32_t b0 = fp8_lo_pair<FMT>(vw[b][nt]), b1 = fp8_hi_pair<FMT>(vw[b][nt]);
          mma16816(o_acc[nt], A[b][0], A[b][1], A[b][2], A[b][3], b0, b1);
          mma16816(o_acc[nt], L[b][0], L[b][1], L[b][2], L[b][3], b0, b1);
        }
      // (the lane has used what it read there)
#pragma unroll
      for (int b = 0; b < AT; ++b) {
        issue(j + b + kStages, next_blk[b], here + b * S::STAGE);
        next_blk[b] = phys(j + AT + b + kStages);
      }
    }
    l_run[0] = quad_sum(l_run[0]);
    l_run[1] = quad_sum(l_run[1]);

    if (alone) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = g + 8 * e;
        if (r >= rows) continue;
        const GroupPlace to = group_place<D>(args_s, seg, gq, row0, r, 0, r, kRows);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          *reinterpret_cast<float2*>(to.o + 8 * nt + 2 * tig) = make_float2(o_acc[nt][2 * e], o_acc[nt][2 * e + 1]);
        if (tig == 0) *reinterpret_cast<float2*>(to.ml) = make_float2(m_run[e] - kBias, l_run[e]);
      }
      if (lane == 0) group_record(args_s, seg);
      __syncwarp();
      continue;
    }
    __syncthreads();  // all rings are drained: their memory takes the warps' results
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
      const GroupPlace to = group_place<D>(args_s, seg, gq, row0, r, 0, r, kRows);
      *reinterpret_cast<float4*>(to.o + 4 * c4) = o;
      if (c4 == 0) *reinterpret_cast<float2*>(to.ml) = make_float2(M - kBias, L);
    }
    if (tid == 0) group_record(args_s, seg);
    __syncthreads();  // the next segment's copies overwrite what was read here
  }
  wait_for_launch_before();
}

// ---------------------------------------------------------------------------
// Joining: a warp per output row. What it has to know of the row's two pairs is
// read at once, then lanes weigh the partial results (log2 units), 32 at a time
// and the shared ones first, then the outputs are added up in that order: three
// dependent reads in all. 16384 rows of 128 channels: 17 us (24 where the two
// pairs were looked at one after the other).
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) group_join_kernel(const __grid_constant__ GroupArgs a) {
  constexpr int V = D / 32;  // floats of a row a lane holds
  const int lane = threadIdx.x & 31;
  const unsigned row = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);  // (below 2^31)
  if (row >= static_cast<unsigned>(a.batch) * a.q_heads) return;
  const int b = row / a.q_heads, hq = row - b * a.q_heads;
  const int gq = a.q_heads / a.kv_heads, h = hq / gq, group = b / a.width;
  const GroupPartials &p0 = a.part[0], &p1 = a.part[1];
  // the row's place in its pair, and that pair's record
  const int in0 = (b - group * a.width) * gq + hq - h * gq, in1 = hq - h * gq;
  const int tile0 = in0 / p0.tile_rows, tile1 = in1 / p1.tile_rows;
  const int tiles0 = (a.width * gq + p0.tile_rows - 1) / p0.tile_rows, tiles1 = (gq + p1.tile_rows - 1) / p1.tile_rows;
  const GroupRecord* const at0 = p0.records + (static_cast<long long>(group) * a.kv_heads + h) * tiles0 + tile0;
  const GroupRecord* const at1 = p1.records + (static_cast<long long>(b) * a.kv_heads + h) * tiles1 + tile1;
  const int len = min(a.seq_lens[b], min(a.max_blocks * 16, a.max_seq_len)), shared = group_shared(a, group);
  const float v_scale = a.v_scale[a.per_head ? h : 0];
  wait_for_launch_before();
  const GroupRecord r0 = *at0, r1 = *at1;
  // (a pair without tokens has no record)
  const int n0 = len > 0 && shared > 0 ? r0.parts * p0.fold : 0, n1 = len > 0 && len > shared * 16 ? r1.parts : 0;
  // partial result i: its place, shared ones first
  auto part_of = [&](int i, const float*& ml, const float*& o) {
    const bool first = i < n0;
    const GroupPartials& p = first ? p0 : p1;
    const GroupRecord r = first ? r0 : r1;
    const int fold = first ? p.fold : 1, at = first ? i : i - n0, part = at / fold, f = at - part * fold;
    const int tile_row = first ? in0 - tile0 * p.tile_rows : in1 - tile1 * p.tile_rows;
    if (r.parts == 1) {
      const long long place = static_cast<long long>(f) * a.batch * a.q_heads + row;
      ml = p.whole_ml + place * 2;
      o = p.whole_o + place * D;
    } else {
      const int slot = part == 0 ? r.slot0 : (r.slot0 & ~1) + 2 * part;
      const long long place = (static_cast<long long>(slot) * fold + f) * p.tile_rows + tile_row;
      ml = p.ml + place * 2;
      o = p.o + place * D;
    }
  };
  float acc[V], M = -INFINITY, L = 0.0f;
#pragma unroll
  for (int e = 0; e < V; ++e) acc[e] = 0.0f;
  const int n = n0 + n1;
  for (int i0 = 0; i0 < n; i0 += 32) {
    const int here = min(32, n - i0);
    float2 x = make_float2(-INFINITY, 0.0f);
    const float *ml = nullptr, *o = nullptr;
    if (i0 + lane < n) {
      part_of(i0 + lane, ml, o);
      x = *reinterpret_cast<const float2*>(ml);
    }
    // (a part without a maximum has the sum 0, or NaN, which stays)
    const float Mn = fmaxf(M, warp_max(x.x));
    const float old = Mn == -INFINITY ? 1.0f : fast_exp2(M - Mn);
    const float w = Mn == -INFINITY ? 1.0f : fast_exp2(x.x - Mn);
    L = L * old + warp_sum(x.y * w);
    M = Mn;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= old;
#pragma unroll 4
    for (int q = 0; q < here; ++q) {
      const float wq = __shfl_sync(0xffffffffu, w, q);
      const float* from = reinterpret_cast<const float*>(__shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), q)) + V * lane;
      float v[V];
      if constexpr (V == 4) {
        const float4 y = *reinterpret_cast<const float4*>(from);
        v[0] = y.x, v[1] = y.y, v[2] = y.z, v[3] = y.w;
      } else {
        const float2 y = *reinterpret_cast<const float2*>(from);
        v[0] = y.x, v[1] = y.y;
      }
#pragma unroll
      for (int e = 0; e < V; ++e) acc[e] = fmaf(v[e], wq, acc[e]);
    }
  }
  const float f = L == 0.0f ? 0.0f : v_scale / L;
  const long long at = static_cast<long long>(row) * D + V * lane;
#pragma unroll
  for (int e = 0; e < V; e += 2) {
    if (a.out_fp32)
      *reinterpret_cast<float2*>(reinterpret_cast<float*>(a.out) + at + e) = make_float2(acc[e] * f, acc[e + 1] * f);
    else
      *reinterpret_cast<uint32_t*>(reinterpret_cast<__half*>(a.out) + at + e) = pack_rn_f16x2(acc[e] * f, acc[e + 1] * f);
  }
}

// `early`: the launch may begin while the one before runs.
cudaError_t launch_next(void (*kern)(const GroupArgs), const GroupArgs& a, dim3 grid, int threads, int smem, bool early, cudaStream_t s) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = early ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <int D, int FMT>
cudaError_t launch_rows16(const GroupArgs& a, cudaStream_t s) {
  constexpr int smem = GroupSmem<D>::BYTES;
  auto kern = group_rows16_kernel<D, FMT>;
  static SharedMemoryOnce once;
  int per_sm = 0;
  cudaError_t e = once.set(kern, smem, 128, &per_sm);
  if (e != cudaSuccess) return e;
  const int most = device_sm_count() * per_sm < kGroupMaxBlocks ? device_sm_count() * per_sm : kGroupMaxBlocks;
  // no more thread blocks than the longest sequences would have work for (slices have two units at least), so that few
  // requests' pairs of both kinds run side by side
  GroupArgs b = a;
  const int gq = a.q_heads / a.kv_heads;
  const long long units = (a.max_seq_len + kUnit - 1ll) / kUnit;
  const long long pairs[2] = {static_cast<long long>(a.batch / a.width) * a.kv_heads * ((a.width * gq + kRows - 1) / kRows),
                              static_cast<long long>(a.batch) * a.kv_heads * ((gq + kRows - 1) / kRows)};
  int grid = 0;
  for (int kind = 0; kind < 2; ++kind) {
    const long long want = (pairs[kind] * units + 1) / 2;
    b.blocks[kind] = static_cast<int>(want < most ? want : most);
    if ((a.kinds >> kind & 1) != 0 && b.blocks[kind] > grid) grid = b.blocks[kind];
  }
  return launch_next(kern, b, dim3(grid, a.kinds == 3 ? 2 : 1), 128, smem, a.kinds != 3, s);
}

}  // namespace

cudaError_t launch_group_attention(const GroupArgs& args, cudaStream_t s) {
  GroupArgs a = args;
  cudaError_t e = cudaSuccess;
  a.kinds = 3;
  if (a.part[0].tile_rows != kRows) {
    a.kinds = 1;
    e = launch_group_tc(a, s);
    if (e != cudaSuccess) return e;
    a.kinds = 2;
  }
  switch (a.head_dim * 10 + a.fmt) {
    case 1280: e = launch_rows16<128, 0>(a, s); break;
    case 1281: e = launch_rows16<128, 1>(a, s); break;
    case 640: e = launch_rows16<64, 0>(a, s); break;
    case 641: e = launch_rows16<64, 1>(a, s); break;
    default: e = cudaErrorInvalidValue;
  }
  if (e != cudaSuccess) return e;
  const long long rows = static_cast<long long>(a.batch) * a.q_heads;
  const unsigned grid = static_cast<unsigned>((rows + kJoinWarps - 1) / kJoinWarps);
  return launch_next(a.head_dim == 128 ? group_join_kernel<128> : group_join_kernel<64>, a, dim3(grid), 32 * kJoinWarps, 0, true, s);
}

}  // namespace kvq
