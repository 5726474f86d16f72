// Attention of a tree of drafted tokens over the paged FP8 cache (kvq_spec.h).
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "spec_internal.h"

namespace kvq {
namespace {

constexpr int kBlock = 16;  // tokens of an FP8 pool block
constexpr int kThreads = 128;

// One thread block per (query row, query head): chunks of 128 tokens, a thread
// per token for the scores, a thread per channel for the value sums, running
// maximum and sum of the softmax.
template <int D, int FMT>
__global__ void __launch_bounds__(kThreads) tree_simple_kernel(TreeArgs a) {
  __shared__ float qs[D], ps[kThreads], red[8];
  __shared__ int blk_s[kThreads / kBlock + 1];
  const int n = blockIdx.x, hq = blockIdx.y, tid = threadIdx.x;
  const int gq = a.q_heads / a.kv_heads, h = hq / gq;
  if (n < a.tree_offsets[0] || n >= a.tree_offsets[a.batch]) return;
  int lo = 0, hi = a.batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a.tree_offsets[mid] <= n) lo = mid;
    else hi = mid;
  }
  const int b = lo, first = a.tree_offsets[b];
  const int nodes = min(min(a.tree_offsets[b + 1] - first, a.max_tree), a.max_blocks * kBlock);
  if (n - first >= nodes) return;
  const int len = min(max(a.seq_lens[b], 0), a.max_blocks * kBlock - nodes);
  const int total = len + nodes;
  const __half* q = reinterpret_cast<const __half*>(a.q) + n * a.q_stride + hq * D;
  if (tid < D) qs[tid] = __half2float(q[tid]) * (a.k_scale[a.per_head ? h : 0] * a.scale_log2);
  const uint64_t* mask = a.tree_mask + static_cast<long long>(n) * a.mask_words;
  float m_run = -INFINITY, l_run = 0.0f, o = 0.0f;
  for (int t0 = 0; t0 < total; t0 += kThreads) {
    __syncthreads();
    if (tid < kThreads / kBlock && t0 + tid * kBlock < total) {
      const int e = a.block_table[static_cast<long long>(b) * a.max_blocks + t0 / kBlock + tid];
      blk_s[tid] = min(max(e, 0), a.num_blocks - 1);
    }
    __syncthreads();
    const int t = t0 + tid;
    bool sees = t < total;
    if (t >= len && t < total) sees = (mask[(t - len) >> 6] >> ((t - len) & 63)) & 1;
    float s = -INFINITY;
    if (sees) {
      const int row = t % kBlock;
      const uint8_t* kb = a.k_pool + (static_cast<long long>(blk_s[tid / kBlock]) * a.kv_heads + h) * (kBlock * D);
      s = 0.0f;
      for (int c = 0; c < D; c += 2) {
        const int byte = ((row / 8 * (D / 64) + c / 64) * 32 + 4 * (row % 8) + c % 16 / 4) * 16 + c % 64 / 16 * 4 + c % 4;
        const float2 kf = __half22float2(bits_h2(fp8x2_to_f16x2<FMT>(*reinterpret_cast<const uint16_t*>(kb + byte))));
        s = fmaf(qs[c], kf.x, s);
        s = fmaf(qs[c + 1], kf.y, s);
      }
    }
    const float wm = warp_max(s);
    if ((tid & 31) == 0) red[tid >> 5] = wm;
    __syncthreads();
    const float m_new = fmaxf(m_run, fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])));
    const float alpha = m_run == -INFINITY ? 0.0f : fast_exp2(m_run - m_new);
    const float p = sees ? fast_exp2(s - m_new) : 0.0f;
    ps[tid] = sees ? p : -1.0f;  // -1: not seen (its value bytes are not read)
    const float ws = warp_sum(p);
    if ((tid & 31) == 0) red[4 + (tid >> 5)] = ws;
    __syncthreads();
    l_run = l_run * alpha + (red[4] + red[5]) + (red[6] + red[7]);
    m_run = m_new;
    if (tid < D) {
      o *= alpha;
      const int c = tid;
      for (int i = 0; i < kThreads && t0 + i < total; ++i) {
        if (ps[i] < 0.0f) continue;
        const int row = i % kBlock;
        const uint8_t* vb = a.v_pool + (static_cast<long long>(blk_s[i / kBlock]) * a.kv_heads + h) * (kBlock * D);
        const int byte = (c / 32 * 32 + 4 * (c % 8) + row % 8 / 2) * 16 + c % 32 / 8 * 4 + row / 8 * 2 + row % 2;
        o = fmaf(ps[i], __low2float(bits_h2(fp8x2_to_f16x2<FMT>(vb[byte]))), o);
      }
    }
  }
  if (tid < D) {
    const float r = l_run == 0.0f ? 0.0f : o / l_run * a.v_scale[a.per_head ? h : 0];
    const long long at = (static_cast<long long>(n) * a.q_heads + hq) * D + tid;
    if (a.out_fp32) reinterpret_cast<float*>(a.out)[at] = r;
    else reinterpret_cast<__half*>(a.out)[at] = __float2half_rn(r);
  }
}

}  // namespace

cudaError_t launch_tree_attention(const TreeArgs& a, cudaStream_t s) {
  const dim3 grid(a.n_tokens, a.q_heads);
  switch (a.head_dim * 10 + a.fmt) {
    case 1280: tree_simple_kernel<128, 0><<<grid, kThreads, 0, s>>>(a); break;
    case 1281: tree_simple_kernel<128, 1><<<grid, kThreads, 0, s>>>(a); break;
    case 640: tree_simple_kernel<64, 0><<<grid, kThreads, 0, s>>>(a); break;
    case 641: tree_simple_kernel<64, 1><<<grid, kThreads, 0, s>>>(a); break;
    default: return cudaErrorInvalidValue;
  }
  return cudaGetLastError();
}

}  // namespace kvq
