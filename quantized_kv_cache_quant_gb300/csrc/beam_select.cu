// Selection of beam candidates for sm_103a (kvq_beam.h): log-softmax over the
// vocabulary and the n best (beam, token) of each request in one pass over the
// logits and one launch.
//
// A cluster of thread blocks takes one request; its rows are cut into parts, and
// block r of C takes parts r, r + C, ... The warps of a block go through a part on
// their own, 2 KB at a time, the next 2 KB on their way. Rows may start on any
// boundary of their type: loads are of aligned 16 bytes, and a thread puts its 8
// or 4 elements together from two of them, so that a row's sum does not depend on
// where the row lies.
//   sum    every thread keeps a maximum and a sum of exp(x - maximum) of its own
//          (fp32, rescaled when the maximum grows, with many steps folded into
//          fp64); they meet at the part's end
//   best   within a row the order of the scores is that of the logits, so a part
//          needs its k = n_out largest logits only. A value that k of the threads'
//          maxima reach is one that at least k elements reach, and only the threads
//          whose maximum reaches it have such elements, some 3 k of 256: the 64 bytes
//          with the maximum are read once more, from L2 (all of a thread's bytes where
//          its next best step reaches it too). Every warp keeps a list of (value,
//          token) keys, which is cut down to its k largest where it runs full; in the
//          end the lists are ranked together.
// Then the first block of the cluster has every part's maximum, sum and sorted
// list (read through distributed shared memory), turns them into scores in fp64,
// and one warp takes the largest head of all lists n_out times.
//
// (Lists that elements enter on the way cost more than the sums: one list a block,
// with barriers between chunks of 32 KB in shared memory, 134 us for 512 rows of
// 128000 bf16 logits, 67 with one barrier a chunk; a list a warp 184. Looking for the
// k-th of the maxima, so that fewer steps are read again, 51.4 against 52, but with
// fp32 logits 69.5 against 64.3 and 152 against 133 us for one request of 64 beams.)
//
// 512 rows of 128000 bf16 logits (one in five ended): 46 us, 2.3 TB/s; fp32, all
// alive, 60 us, 4.3 TB/s; one request of 4 x 32000: 9.5 us. The large calls are bound
// by instructions on the SMs that have four rows at once (of 128000: some 28 us; the
// mean row takes 18), then comes a part's end (bound, second look, ranking: 5 us)
// and the first block's scores (5), which other clusters' reading hides in part. The
// small ones are a chain of such steps, some 10 us of waits. One request is one
// cluster, 16 blocks at most: alone with 64 beams it has a tenth of the SMs.
#include <cfloat>
#include <climits>
#include <cooperative_groups.h>
#include <cuda_bf16.h>

#include "beam_internal.h"
#include "kvq_device.cuh"
#include "kvq_internal.h"
#include "spec_internal.h"

namespace kvq {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kVecs = 4;                       // 16-byte vectors a thread holds of a warp's 2 KB
constexpr int kStep = 32 * kVecs;              // vectors of them
constexpr int kMaxParts = 128;                 // parts of a request: four heads a lane
constexpr int kMaxSplits = 32;                 // parts of a row: a lane's heads, 32 parts apart, are of different beams
constexpr int kFold = 64;                      // steps whose terms a thread adds up in float32
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLog2eLow = 1.925963033500e-8f;  // log2(e) - kLog2e
constexpr unsigned long long kNone = 0ull;     // no key: below every one (a key's low half is never 0)

// Order-preserving code of a float (no NaN, no -0): larger float, larger code.
__device__ __forceinline__ uint32_t float_code(float x) {
  const uint32_t u = __float_as_uint(x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float code_float(uint32_t c) {
  return __uint_as_float(c & 0x80000000u ? c & 0x7fffffffu : ~c);
}
// Larger value first, then the lower token (below 2^31).
__device__ __forceinline__ unsigned long long make_key(float x, int token) {
  return (static_cast<unsigned long long>(float_code(x)) << 32) | ~static_cast<uint32_t>(token);
}
__device__ __forceinline__ int key_token(unsigned long long key) { return static_cast<int>(~static_cast<uint32_t>(key)); }

// NaN counts as -inf, +inf as the largest float; -0 becomes +0.
__device__ __forceinline__ float clean(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX) + 0.0f; }

// A vector of 16 bytes as floats, its largest element (NaN passed over), and -inf in every place.
template <int TYPE>
struct Logits;
template <>
struct Logits<0> {  // fp16
  static constexpr int SIZE = 2;
  static constexpr uint32_t LOW = 0xfc00fc00u;
  __device__ static __forceinline__ float largest(const uint4& v) {
    const __half2 m = __hmax2(__hmax2(bits_h2(v.x), bits_h2(v.y)), __hmax2(bits_h2(v.z), bits_h2(v.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  __device__ static __forceinline__ float at(const void* p, long long i) { return __half2float(static_cast<const __half*>(p)[i]); }
  __device__ static __forceinline__ void unpack(const uint4& v, float2 (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = __half22float2(bits_h2(w[e]));
  }
};
template <>
struct Logits<1> {  // fp32
  static constexpr int SIZE = 4;
  static constexpr uint32_t LOW = 0xff800000u;
  __device__ static __forceinline__ float largest(const uint4& v) {
    return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
  }
  __device__ static __forceinline__ float at(const void* p, long long i) { return static_cast<const float*>(p)[i]; }
  __device__ static __forceinline__ void unpack(const uint4& v, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
};
template <>
struct Logits<2> {  // bf16
  static constexpr int SIZE = 2;
  static constexpr uint32_t LOW = 0xff80ff80u;
  __device__ static __forceinline__ float largest(const uint4& v) {
    auto pair = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 m = __hmax2(__hmax2(pair(v.x), pair(v.y)), __hmax2(pair(v.z), pair(v.w)));
    return fmaxf(__low2float(m), __high2float(m));
  }
  __device__ static __forceinline__ float at(const void* p, long long i) {
    return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p)[i]) << 16);
  }
  __device__ static __forceinline__ void unpack(const uint4& v, float2 (&x)[4]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = make_float2(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
  }
};

// What a part leaves for the first block of its cluster, beside its sorted list: its maximum and the sum of exp(x -
// maximum) in units of 2^-32 (below 2^62: whole numbers add up to the same whatever the order, and without fp64's waits).
struct PartSum {
  unsigned long long sum;
  float max;
};
constexpr float kSumUnits = 4294967296.0f;

// Bytes of the sums and lists of a request's parts.
__host__ __device__ constexpr int list_bytes(int parts, int k) {
  return (parts * static_cast<int>(sizeof(PartSum) + k * sizeof(unsigned long long)) + 15) / 16 * 16;
}

// Keys of a warp's list: it is cut down to k before 32 more might not fit.
__host__ __device__ constexpr int list_cap(int k) { return (2 * k + 64 + 31) / 32 * 32; }
// Two lists a warp: cutting down writes the other one.
__host__ __device__ constexpr int warp_list_bytes(int k) { return 2 * kWarps * list_cap(k) * static_cast<int>(sizeof(unsigned long long)); }

struct SelectShared {
  uint32_t top[kWarps], low[kWarps];  // codes of the warps' largest and j-th largest thread maxima
  int ones[kThreads];      // first vectors of threads' only steps with elements that reach the bound
  uint8_t rich[kThreads];  // threads that have several such steps
  unsigned long long sum;  // of the part
  uint32_t bound;          // code of a value that at least k of the part's elements reach
  int n_ones, riches, count;  // of `ones`, of `rich`; keys in the common list
  float score[kBeamMaxWidth];
  uint8_t kind[kBeamMaxWidth];  // of each beam
};
// Each thread's sum of the steps folded so far, relative to the maximum then.
struct LongSums {
  double sum[kThreads];
  float max[kThreads];
};
constexpr uint8_t kLive = 0, kDead = 1, kEnded = 2;

// exp(x - m) for x <= m: d = x - m rounds relative to d alone, and log2(e) in two parts keeps the product's
// error from pointing one way over a whole row.
__device__ __forceinline__ float exp_below(float x, float m) {
  const float d = x - m;
  return fast_exp2(fmaf(d, kLog2eLow, d * kLog2e));
}

// A thread's sum s of exp(x - m) joins that of its steps before. Out of line: seldom called, and in fp64.
__device__ __noinline__ void fold_sum(LongSums& sums, float s, float m) {
  const int tid = threadIdx.x;
  if (m == -INFINITY) return;
  const float before = sums.max[tid];
  if (before < m) {
    sums.sum[tid] = before == -INFINITY ? 0.0 : sums.sum[tid] * exp(static_cast<double>(before) - static_cast<double>(m));
    sums.max[tid] = m;
  }
  sums.sum[tid] += static_cast<double>(s);
}

// The k largest keys of list[0, n) to out[0, k), largest first (kNone behind the n-th): eight threads count those above a
// key. All threads, synchronised before and after.
__device__ __forceinline__ void rank_list(const unsigned long long* list, int n, int k, unsigned long long* out) {
  for (int i = n + threadIdx.x; i < k; i += kThreads) out[i] = kNone;
  for (int i0 = 0; i0 + static_cast<int>(threadIdx.x & ~31u) / 8 < n; i0 += kThreads / 8) {
    const int i = i0 + threadIdx.x / 8;
    const unsigned long long key = i < n ? list[i] : kNone;
    int larger = 0;
    for (int j = threadIdx.x % 8; j < n; j += 8) larger += list[j] > key;
    larger += __shfl_xor_sync(0xffffffffu, larger, 1);
    larger += __shfl_xor_sync(0xffffffffu, larger, 2);
    larger += __shfl_xor_sync(0xffffffffu, larger, 4);
    if (threadIdx.x % 8 == 0 && i < n && larger < k) out[larger] = key;
  }
}

// The k largest of a warp's n keys (k <= n), largest first, into the other list.
__device__ __noinline__ void cut_list(const unsigned long long* from, int n, int k, unsigned long long* to) {
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < n; i += 32) {
    const unsigned long long key = from[i];
    int larger = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) larger += from[j] > key;
    if (larger < k) to[larger] = key;
  }
  __syncwarp();
}

// The k best candidates where scores of different logits of one beam may have rounded to one number: a row's parts are cut
// by the size of the call, so that in such a beam the keys decide and not the lists' order. By warp 0 of the first block.
__device__ __noinline__ void put_by_keys(int parts, int splits, int k, float* out_scores, int32_t* out_parents, int32_t* out_tokens) {
  extern __shared__ __align__(16) uint8_t dyn[];
  const unsigned long long* lists = reinterpret_cast<const unsigned long long*>(dyn + parts * sizeof(PartSum));
  const unsigned long long* code = reinterpret_cast<const unsigned long long*>(dyn + list_bytes(parts, k));
  const int* token = reinterpret_cast<const int*>(code + parts * k);
  const int lane = threadIdx.x & 31, beam_keys = splits * k;
  auto put = [&](int o, int i) {  // candidate i is the o-th best
    const unsigned long long u = code[i];
    const double x = __longlong_as_double(static_cast<long long>(u >> 63 ? u & ~(1ull << 63) : ~u));
    out_scores[o] = static_cast<float>(x);
    out_parents[o] = i / k / splits;
    out_tokens[o] = token[i];
  };
  // lane l's lists are l, l + 32, ...: a head each
  constexpr int kLists = kMaxParts / 32;
  int at[kLists];
#pragma unroll
  for (int q = 0; q < kLists; ++q) at[q] = 0;
  for (int o = 0; o < k; ++o) {
    unsigned long long best = 0ull;
    int best_q = 0, best_at = INT_MAX;
#pragma unroll
    for (int q = 0; q < kLists; ++q) {
      const int part = lane + 32 * q;
      if (part >= parts || at[q] >= k) continue;
      const unsigned long long c = code[part * k + at[q]];
      if (c > best) {
        best = c;
        best_q = q;
        best_at = part * k + at[q];
      }
    }
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(best >> 32));
    const bool in_hi = static_cast<uint32_t>(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xffffffffu, in_hi ? static_cast<uint32_t>(best) : 0u);
    uint32_t who = __ballot_sync(0xffffffffu, in_hi && static_cast<uint32_t>(best) == lo && best != 0ull);
    if (who & (who - 1)) {  // (a lane's own lists are of different beams, and it has the lower one)
      const bool tie = who >> lane & 1u;
      const uint32_t beam = tie ? best_at / beam_keys : 0xffffffffu, low_beam = __reduce_min_sync(0xffffffffu, beam);
      const bool lowest = tie && beam == low_beam;
      const unsigned long long key = lowest ? lists[best_at] : kNone;
      const uint32_t key_hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(key >> 32));
      const bool in_key = lowest && static_cast<uint32_t>(key >> 32) == key_hi;
      const uint32_t key_lo = __reduce_max_sync(0xffffffffu, in_key ? static_cast<uint32_t>(key) : 0u);
      who = __ballot_sync(0xffffffffu, in_key && static_cast<uint32_t>(key) == key_lo);
    }
    if (who >> lane & 1u) {
      put(o, best_at);
#pragma unroll
      for (int q = 0; q < kLists; ++q) at[q] += q == best_q;
    }
    __syncwarp();
  }
}

// LONG: some part has more than kFold steps (rows of 262144 float32 logits and more). A sum of so many terms would drift, by
// up to 2^-24 of it at each addition (a row of 2^22 equal logits but for every fourth: 1.5e-5), so these threads fold theirs
// into fp64 every kFold steps. A kernel of its own: the other one has no registers for it (with the fold in the same loop,
// 64 x 8 x 128000 bf16 logits took 6 % longer).
template <int TYPE, bool LONG>
__global__ void __launch_bounds__(kThreads, 4) beam_select_kernel(const BeamSelectArgs a, int splits) {
  using L = Logits<TYPE>;
  constexpr int E = 16 / L::SIZE;  // elements of a vector
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ SelectShared sh;
  __shared__ LongSums folded;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int group = blockIdx.x / ranks, k = a.n_out, parts = a.width * splits;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, cap = list_cap(k);
  // the parts' sums and lists, in the first block's memory, where all blocks write them; the warps' lists, and after the
  // last part the scores of all lists
  PartSum* const sums = reinterpret_cast<PartSum*>(cluster.map_shared_rank(dyn, 0));  // [parts]
  unsigned long long* const lists = reinterpret_cast<unsigned long long*>(sums + parts);  // [parts][k]
  uint8_t* const area = dyn + list_bytes(parts, k);
  unsigned long long* const warp_lists = reinterpret_cast<unsigned long long*>(area);  // [2][kWarps][cap]

  // (all blocks have to run before one writes into the first's memory)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  for (int i = tid; i < a.width; i += kThreads) {
    const long long row = static_cast<long long>(group) * a.width + i;
    const float score = a.scores[row];
    sh.score[i] = isfinite(score) ? score : -INFINITY;
    // A beam without a finite score is a dead one, ended or not: its tokens go by their index. (The compiler's registers for
    // the loop below hang on this line: with the score asked first it spills twice as much, and 64 x 8 x 128000 bf16 logits
    // take 49.7 us in place of 46.2.)
    sh.kind[i] = a.finished != nullptr && a.finished[row] != 0 && isfinite(score) ? kEnded : isfinite(score) ? kLive : kDead;
  }
  __syncthreads();
  bool all_run = false;
  for (int part = rank; part < parts; part += ranks) {
    const int beam = part / splits, split = part % splits;
    const long long row = static_cast<long long>(group) * a.width + beam;
    // a beam that has ended or is dead: its candidates follow without a look at the logits
    if (sh.kind[beam] != kLive) continue;
    const uint8_t* base = static_cast<const uint8_t*>(a.logits) + row * a.row_stride * L::SIZE;
    // aligned vector i holds elements i * E - lead .. of the row; a thread's vector j is elements j * E .., from aligned
    // vectors j and, where the row does not start on 16 bytes, j + 1
    const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(base) & 15u) / L::SIZE;
    const uint4* vecs = reinterpret_cast<const uint4*>(base - lead * L::SIZE);
    const int nv = (a.vocab + E - 1) / E;
    const int v0 = static_cast<int>(static_cast<long long>(nv) * split / splits);
    const int v1 = static_cast<int>(static_cast<long long>(nv) * (split + 1) / splits);
    if (tid == 0) {
      sh.n_ones = sh.riches = sh.count = 0;
      sh.sum = 0ull;
      sh.bound = 0u;
    }
    __syncthreads();  // (the part before is done with the lists too)

    // vector j of elements by single loads; what lies outside the row becomes -inf
    auto edge = [&](int j) -> uint4 {
      const long long e0 = static_cast<long long>(j) * E;
      uint32_t w[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (L::SIZE == 4) {
          w[q] = e0 + q < a.vocab ? reinterpret_cast<const uint32_t*>(base)[e0 + q] : L::LOW;
        } else {
          const uint16_t* p = reinterpret_cast<const uint16_t*>(base);
          w[q] = e0 + 2 * q < a.vocab ? p[e0 + 2 * q] : L::LOW & 0xffffu;
          w[q] |= (e0 + 2 * q + 1 < a.vocab ? p[e0 + 2 * q + 1] : L::LOW & 0xffffu) << 16;
        }
      }
      return make_uint4(w[0], w[1], w[2], w[3]);
    };
    // 16 bytes of elements from two aligned vectors
    const int lead_words = lead * L::SIZE / 4, lead_bits = lead * L::SIZE % 4 * 8;
    auto join = [&](const uint4& x, const uint4& y) -> uint4 {
      uint32_t w[5] = {x.x, x.y, x.z, x.w, y.x};
      if (lead_words == 1) w[0] = x.y, w[1] = x.z, w[2] = x.w, w[3] = y.x, w[4] = y.y;
      else if (lead_words == 2) w[0] = x.z, w[1] = x.w, w[2] = y.x, w[3] = y.y, w[4] = y.z;
      else if (lead_words == 3) w[0] = x.w, w[1] = y.x, w[2] = y.y, w[3] = y.z, w[4] = y.w;
      return make_uint4(__funnelshift_r(w[0], w[1], lead_bits), __funnelshift_r(w[1], w[2], lead_bits),
                        __funnelshift_r(w[2], w[3], lead_bits), __funnelshift_r(w[3], w[4], lead_bits));
    };
    // vector j of elements (behind the part's last: -inf)
    auto vec = [&](int j) -> uint4 {
      if (j >= v1) return make_uint4(L::LOW, L::LOW, L::LOW, L::LOW);
      if (lead == 0 ? (j + 1) * static_cast<long long>(E) > a.vocab : j == 0 || (j + 2) * static_cast<long long>(E) - lead > a.vocab)
        return edge(j);
      if (lead == 0) return __ldg(vecs + j);
      const uint4 x = __ldg(vecs + j), y = __ldg(vecs + j + 1);
      return join(x, y);
    };
    // A step, vectors c + 32 u + lane, as it is loaded: the aligned vectors and the one behind them where all of that
    // lies within the row (`whole`; neighbours exchange what they need when the step's turn comes), else the elements.
    struct Step {
      uint4 v[kVecs], behind;
      bool whole;
    };
    auto load = [&](int c, Step& x) {
      x.whole = c + kStep <= v1 && (lead == 0 ? (c + kStep) * static_cast<long long>(E) <= a.vocab
                                              : c > 0 && (c + kStep + 1) * static_cast<long long>(E) - lead <= a.vocab);
#pragma unroll
      for (int u = 0; u < kVecs; ++u) x.v[u] = x.whole ? __ldg(vecs + c + 32 * u + lane) : vec(c + 32 * u + lane);
      if (x.whole && lead != 0) x.behind = __ldg(vecs + c + kStep);
    };
    auto elements = [&](const Step& x, uint4 (&v)[kVecs]) {
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        v[u] = x.v[u];
        if (lead != 0 && x.whole) {
          // the vector behind comes from the next lane, lane 31's from lane 0 of the next 32
          const uint4 from = lane == 0 ? (u + 1 < kVecs ? x.v[u + 1 < kVecs ? u + 1 : 0] : x.behind) : x.v[u];
          const int next_lane = (lane + 1) & 31;
          const uint4 y = make_uint4(__shfl_sync(0xffffffffu, from.x, next_lane), __shfl_sync(0xffffffffu, from.y, next_lane),
                                     __shfl_sync(0xffffffffu, from.z, next_lane), __shfl_sync(0xffffffffu, from.w, next_lane));
          v[u] = join(x.v[u], y);
        }
      }
    };

    float m = -INFINITY, s = 0.0f;  // of this thread
    float second = -INFINITY;       // the largest element of its steps but the one with the maximum,
    int at = v1;                    // whose first vector (lane 0's) this is
    if constexpr (LONG) {
      folded.sum[tid] = 0.0;
      folded.max[tid] = -INFINITY;
    }
    Step next;
    int c = v0 + warp * kStep;
    if (c < v1) load(c, next);
    for (; c < v1; c += kWarps * kStep) {
      uint4 v[kVecs];
      elements(next, v);
      if (c + kWarps * kStep < v1) load(c + kWarps * kStep, next);
      float top = L::largest(v[0]);
#pragma unroll
      for (int u = 1; u < kVecs; ++u) top = fmaxf(top, L::largest(v[u]));
      const bool infinite = top == INFINITY;
      top = clean(top);
      if (top > m) {
        s = m == -INFINITY ? 0.0f : s * exp_below(m, top);
        second = m;
        m = top;
        at = c;
      } else {
        second = fmaxf(second, top);
      }
      if (m > -INFINITY) {
        // (a step's terms first: fewer roundings at the sum's size)
        float2 add = make_float2(0.0f, 0.0f);
        // exp(x - m) is 2^(x log2(e) - m'), m' = m log2(e) rounded, times what that rounding left, which all terms have in
        // common: one rounding a term, relative to its distance from m', and of log2(e)'s own error (1.3e-8) only the
        // part at x - m counts. (A difference first, and log2(e) in two parts, were three operations.) What is left is
        // exp(y), |y| < 2^-8 below 65536: the series' next term is below 2^-26.
        const float top2 = m * kLog2e, y = -0.693147181f * fmaf(m, kLog2e, -top2);
        const float left = fabsf(m) < 65536.0f ? 1.0f + fmaf(0.5f * y, y, y) : NAN;
        const float2 log2e = make_float2(kLog2e, kLog2e), less = make_float2(-top2, -top2);
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
          float2 x[E / 2];
          L::unpack(v[u], x);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            float2 p = __ffma2_rn(x[e], log2e, less);
            p.x = fast_exp2(p.x);
            p.y = fast_exp2(p.y);
            add = __fadd2_rn(add, p);
          }
        }
        float sum = (add.x + add.y) * left;
        if (infinite || sum != sum) {  // infinities and NaN, as their values count; a maximum of any size
          sum = 0.0f;
#pragma unroll
          for (int u = 0; u < kVecs; ++u) {
            float2 x[E / 2];
            L::unpack(v[u], x);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) sum += exp_below(clean(x[e].x), m) + exp_below(clean(x[e].y), m);
          }
        }
        s += sum;
      }
      if constexpr (LONG) {
        if ((c - v0) / (kWarps * kStep) % kFold == kFold - 1) {
          fold_sum(folded, s, m);
          s = 0.0f;
        }
      }
    }
    if constexpr (LONG) fold_sum(folded, s, m);

    // The largest of the threads' maxima, and a bound that k of them reach: each warp's j-th largest one (8 j >= k), the
    // smallest of the warps' ones; some 3 k do. (The k-th itself took 1.8 us to find by bisection, 0.7 among these.)
    const uint32_t mine = m > -INFINITY ? float_code(m) : 0u;
    {
      uint32_t code = mine, best = __reduce_max_sync(0xffffffffu, code);
      if (lane == 0) sh.top[warp] = best;
      for (int left = (k + kWarps - 1) / kWarps - 1; left > 0; --left) {
        const uint32_t who = __ballot_sync(0xffffffffu, code == best);
        if (lane == __ffs(who) - 1) code = 0u;
        best = __reduce_max_sync(0xffffffffu, code);
      }
      if (lane == 0) sh.low[warp] = best;
    }
    __syncthreads();
    const uint32_t bound = __reduce_min_sync(0xffffffffu, sh.low[lane % kWarps]);
    if (mine != 0u && mine >= bound) {
      // (nearly all of them have one step with such elements)
      if (second > -INFINITY && float_code(second) >= bound) sh.rich[atomicAdd(&sh.riches, 1)] = static_cast<uint8_t>(tid);
      else sh.ones[atomicAdd(&sh.n_ones, 1)] = at + lane;
    }
    const uint32_t most = __reduce_max_sync(0xffffffffu, sh.top[lane % kWarps]);  // (0: nothing above -inf)
    const float part_max = most == 0u ? -INFINITY : code_float(most);
    {
      unsigned long long units;
      if constexpr (LONG)
        units = mine != 0u ? __double2ull_rn(folded.sum[tid] * static_cast<double>(exp_below(m, part_max)) * kSumUnits) : 0ull;
      else
        units = mine != 0u ? __float2ull_rn(s * exp_below(m, part_max) * kSumUnits) : 0ull;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) units += __shfl_xor_sync(0xffffffffu, units, o);
      if (lane == 0) atomicAdd(&sh.sum, units);
    }
    __syncthreads();

    // their steps once more: eight threads' step with the maximum a warp and load, or all steps of one thread, 32 vectors a
    // load
    unsigned long long* list = warp_lists + warp * cap;
    unsigned long long* other = warp_lists + (kWarps + warp) * cap;
    unsigned long long own = kNone;  // the warp's k-th largest key (kNone: fewer than k so far)
    int n = 0;                       // keys in the warp's list
    auto cut = [&]() {
      __syncwarp();
      cut_list(list, n, k, other);
      unsigned long long* const x = list;
      list = other;
      other = x;
      n = k;
      own = list[k - 1];
    };
    const int steps = (v1 - v0 + kWarps * kStep - 1) / (kWarps * kStep), ones = (sh.n_ones + 7) / 8, riches = sh.riches;
    int r = warp, q0 = 0;  // the load that comes next
    auto place = [&]() -> int {
      int j = v1;
      if (r < ones) {
        const int i = r * 8 + lane / kVecs;
        if (i < sh.n_ones) j = sh.ones[i] + 32 * (lane % kVecs);
        r += kWarps;
      } else if (r - ones < riches) {
        const int thread = sh.rich[r - ones], q = q0 + lane;
        if (q < steps * kVecs) j = v0 + (q / kVecs * kWarps + thread / 32) * kStep + q % kVecs * 32 + thread % 32;
        q0 += 32;
        if (q0 >= steps * kVecs) {
          q0 = 0;
          r += kWarps;
        }
      }
      return j;
    };
    bool more = r < ones + riches;
    int j = place();
    uint4 w = vec(j);
    while (more) {
      more = r < ones + riches;
      const int j_next = place();
      const uint4 w_next = vec(j_next);
      const float high = clean(L::largest(w));
      if (__any_sync(0xffffffffu, high > -INFINITY && float_code(high) >= bound)) {
        float2 x[E / 2];
        L::unpack(w, x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float y = clean(e % 2 ? x[e / 2].y : x[e / 2].x);
          const unsigned long long key = make_key(y, j * E + e);
          const bool wanted = y > -INFINITY && static_cast<uint32_t>(key >> 32) >= bound && key > own;
          const uint32_t who = __ballot_sync(0xffffffffu, wanted);
          if (who == 0) continue;
          if (wanted) list[n + __popc(who & ((1u << lane) - 1u))] = key;
          n += __popc(who);
          if (n > cap - 32) cut();
        }
      }
      j = j_next;
      w = w_next;
    }
    if (n > max(k, 32)) cut();
    if (lane == 0 && own != kNone) atomicMax(&sh.bound, static_cast<uint32_t>(own >> 32));  // (k elements reach it)
    __syncthreads();
    // keys that reach the bound, of all warps, into one list (the warps' other lists, which nobody reads any more)
    {
      const uint32_t reach = sh.bound;
      unsigned long long keys[(kBeamMaxOut + 31) / 32];
#pragma unroll
      for (int q = 0; q < (kBeamMaxOut + 31) / 32; ++q) keys[q] = lane + 32 * q < n ? list[lane + 32 * q] : kNone;
      __syncthreads();
#pragma unroll
      for (int q = 0; q < (kBeamMaxOut + 31) / 32; ++q)
        if (static_cast<uint32_t>(keys[q] >> 32) >= reach && keys[q] != kNone) warp_lists[atomicAdd(&sh.count, 1)] = keys[q];
    }
    __syncthreads();
    const int found = sh.count;
    if (!all_run) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    all_run = true;
    unsigned long long* const out = lists + part * k;
    rank_list(warp_lists, found, k, out);
    if (tid == 0) sums[part] = PartSum{sh.sum, part_max};
    if (found < k) {  // tokens at -inf, by their index
      __syncthreads();
      if (warp == 0) {
        int need = k - found;
        const int t0 = v0 * E, t1 = min(v1 * E, a.vocab);
        for (int t = t0; need > 0 && t < t1; t += 32) {
          const bool low = t + lane < t1 && clean(L::at(base, t + lane)) == -INFINITY;
          const uint32_t all = __ballot_sync(0xffffffffu, low);
          const int at = __popc(all & ((1u << lane) - 1u));
          if (low && at < need) out[k - need + at] = make_key(-INFINITY, t + lane);
          need -= __popc(all);
        }
      }
    }
    __syncthreads();
  }
  if (!all_run) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  cluster.sync();
  if (rank != 0) return;

  // ---- the first block: scores of all lists, and the best of them ----
  unsigned long long* code = reinterpret_cast<unsigned long long*>(area);  // [parts][k]
  int* token = reinterpret_cast<int*>(code + parts * k);                   // [parts][k]
  __shared__ double log_sum[kBeamMaxWidth];
  __shared__ float row_max[kBeamMaxWidth];
  // order-preserving code of a score; 0: none
  auto score_code = [](double x) -> unsigned long long {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
    return u >> 63 ? ~u : u | (1ull << 63);
  };
  for (int beam = tid; beam < a.width; beam += kThreads) {
    double sum = 0.0;
    float most = -INFINITY;
    if (sh.kind[beam] == kLive) {
      for (int split = 0; split < splits; ++split) most = fmaxf(most, sums[beam * splits + split].max);
      for (int split = 0; most > -INFINITY && split < splits; ++split) {
        const PartSum p = sums[beam * splits + split];
        if (p.max > -INFINITY) sum += static_cast<double>(p.sum) * static_cast<double>(exp_below(p.max, most));
      }
    }
    // 2^e f, f in [1, 2): the logarithm of f is below 1, so that in fp32 it is off by some 2^-24, as f is
    const unsigned long long bits = static_cast<unsigned long long>(__double_as_longlong(sum));
    const int e = static_cast<int>(bits >> 52) - 1023 - 32;
    const float f = static_cast<float>(__longlong_as_double(static_cast<long long>((bits & 0xfffffffffffffull) | 0x3ff0000000000000ull)));
    log_sum[beam] = most == -INFINITY ? 0.0 : fma(static_cast<double>(e), 0.69314718055994530942, static_cast<double>(logf(f)));
    row_max[beam] = most;
  }
  __syncthreads();
  bool by_keys = false;
  for (int i = tid; i < parts * k; i += kThreads) {
    const int part = i / k, at = i % k, beam = part / splits;
    const float score = sh.score[beam];
    unsigned long long c = 0ull;
    int t = 0;
    if (sh.kind[beam] != kLive) {
      // the end token first, then the others by their index, all in the row's first part
      const bool end = sh.kind[beam] == kEnded;
      if (part % splits == 0) {
        t = !end ? at : at == 0 ? a.end_token : at - 1 + (at - 1 >= a.end_token);
        c = score_code(end && at == 0 ? static_cast<double>(score) : -INFINITY);
      }
    } else {
      const unsigned long long key = lists[i];
      if (key != kNone) {
        const float x = code_float(static_cast<uint32_t>(key >> 32));
        t = key_token(key);
        // Two float32 x differ by 2^-24 of the larger one; where that is more than the roundings of a score (three, of 2^-53
        // of what it is made of), their scores differ too.
        by_keys |= fabsf(x) * 0x1p26f < fabsf(x - row_max[beam]) + fabsf(score) + fabsf(static_cast<float>(log_sum[beam]));
        c = score_code(x == -INFINITY ? -INFINITY
                                      : static_cast<double>(score) + ((static_cast<double>(x) - static_cast<double>(row_max[beam])) - log_sum[beam]));
      }
    }
    code[i] = c;
    token[i] = t;
  }
  if (__syncthreads_or(by_keys)) {
    const long long to = static_cast<long long>(group) * k;
    if (warp == 0) put_by_keys(parts, splits, k, a.out_scores + to, a.out_parents + to, a.out_tokens + to);
    return;
  }
  auto put = [&](int o, int i) {  // candidate i is the o-th best
    const unsigned long long u = code[i];
    const double x = __longlong_as_double(static_cast<long long>(u >> 63 ? u & ~(1ull << 63) : ~u));
    const long long to = static_cast<long long>(group) * k + o;
    a.out_scores[to] = static_cast<float>(x);
    a.out_parents[to] = i / k / splits;
    a.out_tokens[to] = token[i];
  };
  // Equal scores: the lower beam, then the lower token, as the logits are equal (the lists' order: parts of a row go up in
  // tokens).
  const int total = parts * k;
  if (total <= kThreads) {
    // few: eight threads count those before a candidate
    for (int i0 = 0; i0 + (warp << 2) < total; i0 += kThreads / 8) {
      const int i = i0 + tid / 8;
      const unsigned long long c = i < total ? code[i] : 0ull;
      int before = 0;
      for (int j = tid % 8; j < total; j += 8) before += code[j] >= c + (j >= i);
      before += __shfl_xor_sync(0xffffffffu, before, 1);
      before += __shfl_xor_sync(0xffffffffu, before, 2);
      before += __shfl_xor_sync(0xffffffffu, before, 4);
      if (tid % 8 == 0 && i < total && c != 0ull && before < k) put(before, i);
    }
    return;
  }
  if (warp != 0) return;
  // lane l's lists are l, l + 32, ...: a head each
  constexpr int kLists = kMaxParts / 32;
  int at[kLists];
#pragma unroll
  for (int q = 0; q < kLists; ++q) at[q] = 0;
  for (int o = 0; o < k; ++o) {
    unsigned long long best = 0ull;
    int best_q = 0, best_at = INT_MAX;
#pragma unroll
    for (int q = 0; q < kLists; ++q) {
      const int part = lane + 32 * q;
      if (part >= parts || at[q] >= k) continue;
      const unsigned long long c = code[part * k + at[q]];
      if (c > best) {
        best = c;
        best_q = q;
        best_at = part * k + at[q];
      }
    }
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(best >> 32));
    const bool in_hi = static_cast<uint32_t>(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xffffffffu, in_hi ? static_cast<uint32_t>(best) : 0u);
    const bool tie = in_hi && static_cast<uint32_t>(best) == lo && best != 0ull;
    const uint32_t first = __reduce_min_sync(0xffffffffu, tie ? static_cast<uint32_t>(best_at) : 0xffffffffu);
    if (tie && static_cast<uint32_t>(best_at) == first) {
      put(o, best_at);
#pragma unroll
      for (int q = 0; q < kLists; ++q) at[q] += q == best_q;
    }
    __syncwarp();
  }
}

// Shared memory of a request of `parts` parts, k candidates each.
constexpr int shared_bytes(int parts, int k) {
  const int scores = parts * k * static_cast<int>(sizeof(unsigned long long) + sizeof(int));
  return list_bytes(parts, k) + (scores > warp_list_bytes(k) ? scores : warp_list_bytes(k));
}
// Of the widest request with the most candidates in one block, rows whole.
constexpr int kMostShared = shared_bytes(kBeamMaxWidth, kBeamMaxOut);
static_assert(kWarps * kBeamMaxOut <= 2 * kWarps * list_cap(kBeamMaxOut), "the keys of all warps, cut down, fit where their lists were");
static_assert(kMostShared + sizeof(SelectShared) + sizeof(LongSums) + 2048 <= 232448, "shared memory of a thread block");

struct SelectPlan {
  int ranks, splits, smem;
};

// Blocks of a cluster (up to 16: one request is one cluster), as many as have room at once where four fit an SM, and parts
// of a row, so that the block with the most to do has little of it; a part costs what `fixed` bytes of logits do beside its
// own. (64 requests of 8 rows of 128000: clusters of 2, 4, 8 and 16 blocks 88, 57, 51 and 67 us; four blocks an SM allow 8.)
// Four blocks fit while a request's lists are small. Those of 64 beams with 128 candidates take 161 KB, which the other
// blocks of its cluster hold too without a use for it: one block an SM, and many such requests run in several waves (64
// requests of 64 rows of 32000 fp16 logits: 119 us with 16 candidates, 887 with 128).
SelectPlan plan_select(const BeamSelectArgs& a, int size, int most_ranks) {
  SelectPlan best{1, 1, 0};
  const long long fixed = 16384;
  int ranks = 1;
  while (ranks < most_ranks && static_cast<long long>(a.groups) * ranks * 2 <= 4ll * device_sm_count()) ranks *= 2;
  long long best_cost = LLONG_MAX;
  for (int splits = 1; splits <= kMaxSplits && a.width * splits <= kMaxParts; ++splits) {
    const int parts = a.width * splits;
    const long long rounds = (parts + ranks - 1) / ranks;
    const long long cost = rounds * (static_cast<long long>(a.vocab) * size / splits + fixed);
    const int smem = shared_bytes(parts, a.n_out);
    if (cost < best_cost && (splits == 1 || smem <= kMostShared)) {
      best_cost = cost;
      best = SelectPlan{ranks, splits, smem};
    }
  }
  return best;
}

// Steps of the longest part.
int most_steps(const BeamSelectArgs& a, int size, int splits) {
  const int nv = static_cast<int>((static_cast<long long>(a.vocab) * size + 15) / 16);
  return ((nv + splits - 1) / splits + kWarps * kStep - 1) / (kWarps * kStep);
}

template <int TYPE, bool LONG>
cudaError_t launch_select(const BeamSelectArgs& a, cudaStream_t s) {
  auto kern = beam_select_kernel<TYPE, LONG>;
  static SharedMemoryOnce once;
  cudaError_t e = once.set(kern, kMostShared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attrs[2];
  cudaLaunchAttribute& attr = attrs[0];
  // (ended beams leave blocks idle: SMs with fewer busy ones take the next cluster; 52 -> 48 us with one beam in five ended)
  attrs[1].id = cudaLaunchAttributeClusterSchedulingPolicyPreference;
  attrs[1].val.clusterSchedulingPolicyPreference = cudaClusterSchedulingPolicyLoadBalancing;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 16;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kMostShared;
  cfg.stream = s;
  cfg.attrs = attrs;
  cfg.numAttrs = 1;
  // clusters of 16 blocks, asked for once per device: 1 they fit, -1 they do not (8 are the portable most)
  static std::atomic<int> fits[SharedMemoryOnce::kDevices] = {};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int f = dev < SharedMemoryOnce::kDevices ? fits[dev].load(std::memory_order_relaxed) : 0;
  if (f == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    int clusters = 0;
    f = cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) == cudaSuccess && clusters > 0 ? 1 : -1;
    if (f < 0) (void)cudaGetLastError();
    if (dev < SharedMemoryOnce::kDevices) fits[dev].store(f, std::memory_order_relaxed);
  }
  const SelectPlan p = plan_select(a, Logits<TYPE>::SIZE, f > 0 ? 16 : 8);
  if constexpr (!LONG) {
    if (most_steps(a, Logits<TYPE>::SIZE, p.splits) > kFold) return launch_select<TYPE, true>(a, s);
  }
  attr.val.clusterDim.x = p.ranks;
  cfg.gridDim = dim3(static_cast<unsigned>(a.groups) * p.ranks);
  cfg.dynamicSmemBytes = p.smem;
  cfg.numAttrs = 2;
  e = cudaLaunchKernelEx(&cfg, kern, a, p.splits);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_beam_select(const BeamSelectArgs& a, cudaStream_t s) {
  switch (a.type) {
    case 0: return launch_select<0, false>(a, s);
    case 1: return launch_select<1, false>(a, s);
    case 2: return launch_select<2, false>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
