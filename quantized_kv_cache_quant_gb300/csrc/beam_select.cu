// Selection of beam candidates for sm_103a (kvq_beam.h): log-softmax over the
// vocabulary and the n best (beam, token) of each request in one pass over the
// logits and one launch.
//
// A cluster of thread blocks takes one request; its rows are cut into parts, and
// block r of C takes parts r, r + C, ... A part streams through shared memory in
// chunks of 16 KB, the next ones' copies in flight. Rows may start on any
// boundary of their type: copies are of aligned 16 bytes, and a thread puts its
// 8 or 4 elements together from two of them, so that a row's sum does not depend
// on where the row lies.
//   sum    every thread keeps a maximum and a sum of exp(x - maximum) of its own
//          (fp32, rescaled when the maximum grows); they meet at the part's end
//   best   within a row the order of the scores is that of the logits, so a part
//          needs its k = n_out largest logits only. Of the 8 warps' maxima of the first
//          chunk (their j-th largest lane maxima, 8 j >= k) the smallest is a bound that at
//          least k elements reach and few do; the threads whose own maximum reaches it
//          put those elements into a list of (value, token) keys. Chunks after the
//          first have to exceed it. A list that runs full is cut down to its k
//          largest, found bit by bit where even one chunk does not fit.
// Then the first block of the cluster has every part's maximum, sum and sorted
// list (read through distributed shared memory), turns them into scores in fp64,
// and one warp takes the largest head of all lists n_out times.
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
constexpr int kVecs = 4;                       // 16-byte vectors a thread holds of a chunk
constexpr int kChunk = kThreads * kVecs;       // vectors of a chunk
constexpr int kStages = 3;                     // chunks in shared memory
constexpr int kStageBytes = (kChunk + 1) * 16; // and one vector more, where elements reach into it
constexpr int kCap = 512;                      // keys of a part's list
constexpr int kMaxParts = 128;                 // parts of a request: four heads a lane
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

// What a part leaves for the first block of its cluster.
struct PartSum {
  double sum;
  float max;
};

// Bytes of the sums and lists of `mine` parts.
__host__ __device__ constexpr int list_bytes(int mine, int k) {
  return (mine * static_cast<int>(sizeof(PartSum) + k * sizeof(unsigned long long)) + 15) / 16 * 16;
}

struct SelectShared {
  unsigned long long list[kCap];
  uint32_t bound[kWarps];
  float warp_max[kWarps];
  double warp_sum[kWarps];
  int added[3], hits;  // keys that chunk it has added: [it % 3]
};

// exp(x - m) for x <= m: d = x - m rounds relative to d alone, and log2(e) in two parts keeps the product's
// error from pointing one way over a whole row.
__device__ __forceinline__ float exp_below(float x, float m) {
  const float d = x - m;
  return fast_exp2(fmaf(d, kLog2eLow, d * kLog2e));
}

// The k largest keys of list[0, n) to out[0, k), largest first (kNone behind the n-th): eight threads count those above a
// key. All threads, synchronised before and after.
__device__ __forceinline__ void rank_list(const unsigned long long* list, int n, int k, unsigned long long* out) {
  for (int i = n + threadIdx.x; i < k; i += kThreads) out[i] = kNone;
  for (int i0 = 0; i0 < n; i0 += kThreads / 8) {
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

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 4) beam_select_kernel(const BeamSelectArgs a, int splits) {
  using L = Logits<TYPE>;
  constexpr int E = 16 / L::SIZE;  // elements of a vector
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ SelectShared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int ranks = cluster.num_blocks(), rank = cluster.block_rank();
  const int group = blockIdx.x / ranks, k = a.n_out, parts = a.width * splits;
  const int mine = (parts + ranks - 1) / ranks;  // parts of a block at most
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the ring, and after the last part the scores of all lists
  uint8_t* const ring = dyn + list_bytes(mine, k);
  PartSum* sums = reinterpret_cast<PartSum*>(dyn);                                          // [mine]
  unsigned long long* lists = reinterpret_cast<unsigned long long*>(dyn + mine * sizeof(PartSum));  // [mine][k]

  for (int slot = 0, part = rank; part < parts; ++slot, part += ranks) {
    const int beam = part / splits, split = part % splits;
    const long long row = static_cast<long long>(group) * a.width + beam;
    const float score = a.scores[row];
    unsigned long long* out = lists + slot * k;
    // a beam that has ended or is dead: its candidates follow without a look at the logits
    if ((a.finished != nullptr && a.finished[row] != 0) || !isfinite(score)) continue;
    const uint8_t* base = static_cast<const uint8_t*>(a.logits) + row * a.row_stride * L::SIZE;
    // aligned vector i holds elements i * E - lead .. of the row; a thread's vector j is elements j * E .., from aligned
    // vectors j and, where the row does not start on 16 bytes, j + 1
    const int lead = static_cast<int>(reinterpret_cast<uintptr_t>(base) & 15u) / L::SIZE;
    const uint4* vecs = reinterpret_cast<const uint4*>(base - lead * L::SIZE);
    const int nv = (a.vocab + E - 1) / E;
    const int v0 = static_cast<int>(static_cast<long long>(nv) * split / splits);
    const int v1 = static_cast<int>(static_cast<long long>(nv) * (split + 1) / splits);
    if (tid < 3) sh.added[tid] = 0;

    auto copy = [&](uint8_t* stage, int c, int i) {  // aligned vector c + i; what lies outside the row becomes -inf
      const long long e0 = static_cast<long long>(c + i) * E - lead;
      uint4* to = reinterpret_cast<uint4*>(stage) + i;
      if (e0 >= 0 && e0 + E <= a.vocab) {
        cp_async16(to, vecs + c + i);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if constexpr (L::SIZE == 4) {
            w[q] = e0 + q >= 0 && e0 + q < a.vocab ? reinterpret_cast<const uint32_t*>(base)[e0 + q] : 0xff800000u;
          } else {
            constexpr uint32_t kLow = TYPE == 0 ? 0xfc00u : 0xff80u;
            const uint16_t* p = reinterpret_cast<const uint16_t*>(base);
            const long long x = e0 + 2 * q;
            w[q] = x >= 0 && x < a.vocab ? p[x] : kLow;
            w[q] |= (x + 1 >= 0 && x + 1 < a.vocab ? p[x + 1] : kLow) << 16;
          }
        }
        *to = make_uint4(w[0], w[1], w[2], w[3]);
      }
    };
    const int reach = v1 + (lead > 0);  // aligned vectors up to here
    auto issue = [&](int it) {
      const int c = v0 + it * kChunk;
      if (c < v1) {
        uint8_t* stage = ring + it % kStages * kStageBytes;
        if (c * static_cast<long long>(E) >= lead && c + kChunk < reach &&
            (static_cast<long long>(c) + kChunk + 1) * E - lead <= a.vocab) {  // all within the row
#pragma unroll
          for (int u = 0; u < kVecs; ++u)
            cp_async16(reinterpret_cast<uint4*>(stage) + u * kThreads + tid, vecs + c + u * kThreads + tid);
          if (tid == 0) cp_async16(reinterpret_cast<uint4*>(stage) + kChunk, vecs + c + kChunk);
        } else {
          for (int i = tid; i <= kChunk && c + i < reach; i += kThreads) copy(stage, c, i);
        }
      }
      cp_async_commit();
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

    float m = -INFINITY, s = 0.0f;  // of this thread
    float bound = -INFINITY;        // at least k elements so far reach it (-inf: not yet)
    int held = 0;                   // keys in the list before the chunk (at most 2 k + 32)
    float top = -INFINITY;          // of this thread's elements of the chunk

    // Vector u of chunk it; behind the part's last one: -inf.
    auto vec = [&](int it, int u) -> uint4 {
      if (v0 + it * kChunk + u * kThreads + tid >= v1) return make_uint4(L::LOW, L::LOW, L::LOW, L::LOW);
      const uint4* here = reinterpret_cast<const uint4*>(ring + it % kStages * kStageBytes) + u * kThreads + tid;
      return lead == 0 ? here[0] : join(here[0], here[1]);
    };
    // f(value, token) of every element of chunk it: the less frequent passes, a vector at a time, in little code
    auto each = [&](int it, auto f) {
#pragma unroll 1
      for (int u = 0; u < kVecs; ++u) {
        float2 x[E / 2];
        L::unpack(vec(it, u), x);
#pragma unroll
        for (int e = 0; e < E; ++e)
          f(clean(e % 2 ? x[e / 2].y : x[e / 2].x), (v0 + it * kChunk + u * kThreads + tid) * E + e);
      }
    };
    // A bound of a chunk: each warp's j-th largest lane maximum, the smallest of the warps' ones.
    auto chunk_bound = [&]() {
      uint32_t code = float_code(top), best = 0u;
      const int times = (k + kWarps - 1) / kWarps;
      for (int t = 0; t < times; ++t) {
        best = __reduce_max_sync(0xffffffffu, code);
        const uint32_t who = __ballot_sync(0xffffffffu, code == best);
        if (lane == __ffs(who) - 1) code = 0u;
      }
      if (lane == 0) sh.bound[warp] = best;
      __syncthreads();
      const uint32_t low = sh.bound[lane % kWarps];
      return code_float(max(__reduce_min_sync(0xffffffffu, low), float_code(-INFINITY)));
    };
    // (in chunks after the first tokens are higher, so an equal value does not displace one in the list)
    auto wanted = [&](float x, float limit, bool equal) { return x > limit || (equal && x == limit && x > -INFINITY); };
    auto collect = [&](int it, float limit, bool equal) {
      if (!wanted(top, limit, equal)) return;
#pragma unroll 1
      for (int u = 0; u < kVecs; ++u) {
        const uint4 w = vec(it, u);
        if (!wanted(L::largest(w), limit, equal)) continue;
        float2 x[E / 2];
        L::unpack(w, x);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          const float y = e % 2 ? x[e / 2].y : x[e / 2].x;
          if (wanted(y, limit, equal)) {
            const int i = held + atomicAdd(&sh.added[it % 3], 1);
            if (i < kCap) sh.list[i] = make_key(clean(y), (v0 + it * kChunk + u * kThreads + tid) * E + e);
          }
        }
      }
    };
    // What chunk it added, once all threads have collected: the list is cut down where it has grown.
    auto settle = [&](int it, bool last) {
      const int had = held;
      held += sh.added[it % 3];
      if (tid == 0) sh.added[(it + 2) % 3] = 0;  // (of chunk it - 1, which all have read)
      if (held > kCap && it > 0) {  // a bound of this chunk's own may let fewer through
        const float tight = chunk_bound();
        if (tight > bound) {
          if (tid == 0) sh.added[it % 3] = 0;
          __syncthreads();
          held = had;
          collect(it, tight, true);
          __syncthreads();
          held += sh.added[it % 3];
        }
      }
      if (held > kCap) {
        // the k-th largest key of what was had and this chunk, bit by bit
        unsigned long long kth = 0ull;
        for (int bit = 63; bit >= 0; --bit) {
          const unsigned long long trial = kth | (1ull << bit);
          int reach = 0;
          if (make_key(top, 0) >= trial)
            each(it, [&](float x, int token) { reach += x > -INFINITY && make_key(x, token) >= trial; });
          for (int i = tid; i < had; i += kThreads) reach += sh.list[i] >= trial;
          if (tid == 0) sh.hits = 0;
          __syncthreads();
          reach = __reduce_add_sync(0xffffffffu, reach);
          if (lane == 0) atomicAdd(&sh.hits, reach);
          __syncthreads();
          if (sh.hits >= k) kth = trial;
          __syncthreads();
        }
        constexpr int kHad = (2 * kBeamMaxOut + 32 + kThreads - 1) / kThreads;
        unsigned long long keep[kHad];
#pragma unroll
        for (int q = 0; q < kHad; ++q) keep[q] = tid + q * kThreads < had ? sh.list[tid + q * kThreads] : kNone;
        if (tid == 0) sh.hits = 0;
        __syncthreads();
        auto put = [&](unsigned long long key) {
          if (key >= kth) sh.list[atomicAdd(&sh.hits, 1)] = key;  // (k keys, they are distinct)
        };
#pragma unroll
        for (int q = 0; q < kHad; ++q)
          if (keep[q] != kNone) put(keep[q]);
        each(it, [&](float x, int token) {
          if (x > -INFINITY) put(make_key(x, token));
        });
        __syncthreads();
        held = k;
        bound = code_float(static_cast<uint32_t>(kth >> 32));
      } else if (!last && held > (it == 0 ? k : 2 * k + 32)) {
        // Few elements of later chunks exceed the k-th so far, and a warp without one has nothing to collect.
        rank_list(sh.list, held, k, out);
        __syncthreads();
        for (int i = tid; i < k; i += kThreads) sh.list[i] = out[i];
        held = k;
        bound = code_float(static_cast<uint32_t>(out[k - 1] >> 32));
        // (keys that the next chunk adds go behind these)
      }
    };

    __syncthreads();  // the part before is done with the ring
#pragma unroll
    for (int it = 0; it < kStages - 1; ++it) issue(it);
    int it = 0;
    for (int c = v0; c < v1; ++it, c += kChunk) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncthreads();  // this chunk has landed; what the one before has added is complete
      if (it > 0) settle(it - 1, false);
      issue(it + kStages - 1);  // (where the chunk before was; settle reads it again between barriers only)
      uint4 v[kVecs];
#pragma unroll
      for (int u = 0; u < kVecs; ++u) v[u] = vec(it, u);
      top = L::largest(v[0]);
#pragma unroll
      for (int u = 1; u < kVecs; ++u) top = fmaxf(top, L::largest(v[u]));
      const bool infinite = top == INFINITY;
      top = clean(top);
      if (top > m) {
        s = m == -INFINITY ? 0.0f : s * exp_below(m, top);
        m = top;
      }
      if (m > -INFINITY) {
        // (a chunk's terms first: fewer roundings at the sum's size)
        float2 add = make_float2(0.0f, 0.0f);
        const float2 m2 = make_float2(-m, -m), high = make_float2(kLog2e, kLog2e), low = make_float2(kLog2eLow, kLog2eLow);
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
          if (c + u * kThreads >= v1) break;
          float2 x[E / 2];
          L::unpack(v[u], x);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            const float2 d = __fadd2_rn(x[e], m2);
            float2 p = __ffma2_rn(d, low, __fmul2_rn(d, high));
            p.x = fast_exp2(p.x);
            p.y = fast_exp2(p.y);
            add = __fadd2_rn(add, p);
          }
        }
        float sum = add.x + add.y;
        if (infinite || sum != sum) {  // infinities and NaN, as their values count
          sum = 0.0f;
          each(it, [&](float x, int) { sum += exp_below(x, m); });
        }
        s += sum;
      }
      if (it == 0) bound = chunk_bound();
      collect(it, bound, it == 0);
    }
    __syncthreads();
    if (it > 0) settle(it - 1, true);  // (a part of a short row may have no vector)

    // the part's maximum and sum, its sorted list
    const float wm = code_float(__reduce_max_sync(0xffffffffu, float_code(m)));
    double ws = m == -INFINITY ? 0.0 : static_cast<double>(s) * static_cast<double>(exp_below(m, wm));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, o);
    __syncthreads();
    if (lane == 0) {
      sh.warp_max[warp] = wm;
      sh.warp_sum[warp] = ws;
    }
    const int n = held;
    rank_list(sh.list, n, k, out);
    __syncthreads();
    if (warp == 0) {
      const float v = lane < kWarps ? sh.warp_max[lane] : -INFINITY;
      const float pm = code_float(__reduce_max_sync(0xffffffffu, float_code(v)));
      double ps = v == -INFINITY ? 0.0 : sh.warp_sum[lane] * static_cast<double>(exp_below(v, pm));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, o);
      if (lane == 0) {
        sums[slot].max = pm;
        sums[slot].sum = ps;
      }
      // fewer than k finite values: tokens at -inf, by their index
      const int have = min(n, k);
      int need = k - have;
      const int t0 = v0 * E;
      const int t1 = min(v1 * E, a.vocab);
      for (int t = t0; need > 0 && t < t1; t += 32) {
        const bool low = t + lane < t1 && clean(L::at(base, t + lane)) == -INFINITY;
        const uint32_t all = __ballot_sync(0xffffffffu, low);
        const int at = __popc(all & ((1u << lane) - 1u));
        if (low && at < need) out[k - need + at] = make_key(-INFINITY, t + lane);
        need -= __popc(all);
      }
    }
    __syncthreads();
  }
  cluster.sync();

  // ---- the first block: scores of all lists, and the best of them ----
  unsigned long long* code = reinterpret_cast<unsigned long long*>(ring);  // [parts][k]
  int* token = reinterpret_cast<int*>(code + parts * k);                   // [parts][k]
  __shared__ double log_sum[kBeamMaxWidth];
  __shared__ float row_max[kBeamMaxWidth];
  // order-preserving code of a score; 0: none
  auto score_code = [](double x) -> unsigned long long {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
    return u >> 63 ? ~u : u | (1ull << 63);
  };
  auto ended = [&](int beam) {
    const long long row = static_cast<long long>(group) * a.width + beam;
    return a.finished != nullptr && a.finished[row] != 0;
  };
  if (rank == 0) {
    for (int beam = tid; beam < a.width; beam += kThreads) {
      const float score = a.scores[static_cast<long long>(group) * a.width + beam];
      double sum = 0.0;
      float most = -INFINITY;
      if (!ended(beam) && isfinite(score)) {
        for (int split = 0; split < splits; ++split) {
          const int part = beam * splits + split;
          most = fmaxf(most, cluster.map_shared_rank(sums, part % ranks)[part / ranks].max);
        }
        for (int split = 0; most > -INFINITY && split < splits; ++split) {
          const int part = beam * splits + split;
          const PartSum p = cluster.map_shared_rank(sums, part % ranks)[part / ranks];
          if (p.max > -INFINITY) sum += p.sum * static_cast<double>(exp_below(p.max, most));
        }
      }
      log_sum[beam] = most == -INFINITY ? 0.0 : log(sum);
      row_max[beam] = most;
    }
    __syncthreads();
    for (int i = tid; i < parts * k; i += kThreads) {
      const int part = i / k, at = i % k, beam = part / splits;
      const float score = a.scores[static_cast<long long>(group) * a.width + beam];
      unsigned long long c = 0ull;
      int t = 0;
      const bool end = ended(beam);
      if (end || !isfinite(score)) {
        // the end token first, then the others by their index, all in the row's first part
        if (part % splits == 0) {
          if (end && at == 0) {
            t = a.end_token;
            c = score_code(isfinite(score) ? static_cast<double>(score) : -INFINITY);
          } else {
            t = end ? at - 1 + (at - 1 >= a.end_token) : at;
            c = score_code(-INFINITY);
          }
        }
      } else {
        const unsigned long long key = cluster.map_shared_rank(lists, part % ranks)[(part / ranks) * k + at];
        if (key != kNone) {
          const float x = code_float(static_cast<uint32_t>(key >> 32));
          t = key_token(key);
          c = score_code(x == -INFINITY ? -INFINITY
                                        : static_cast<double>(score) + ((static_cast<double>(x) - static_cast<double>(row_max[beam])) - log_sum[beam]));
        }
      }
      code[i] = c;
      token[i] = t;
    }
  }
  cluster.sync();  // (no block ends while the first one reads its lists)
  if (rank != 0 || warp != 0) return;
  // lane l's lists are l, l + 32, ...: a head each
  constexpr int kLists = kMaxParts / 32;
  int at[kLists];
#pragma unroll
  for (int q = 0; q < kLists; ++q) at[q] = 0;
  for (int o = 0; o < k; ++o) {
    unsigned long long best = 0ull;
    int best_q = 0, best_part = INT_MAX, best_token = INT_MAX;
#pragma unroll
    for (int q = 0; q < kLists; ++q) {
      const int part = lane + 32 * q;
      if (part >= parts || at[q] >= k) continue;
      const unsigned long long c = code[part * k + at[q]];
      // (a lane's lists go up in beams and, within one, in tokens)
      if (c > best) {
        best = c;
        best_q = q;
        best_part = part;
        best_token = token[part * k + at[q]];
      }
    }
    const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(best >> 32));
    const bool in_hi = static_cast<uint32_t>(best >> 32) == hi;
    const uint32_t lo = __reduce_max_sync(0xffffffffu, in_hi ? static_cast<uint32_t>(best) : 0u);
    const bool tie = in_hi && static_cast<uint32_t>(best) == lo && best != 0ull;
    // equal scores: the lower beam, then the lower token (parts of a row go up in tokens, but equal values in two parts
    // of one row follow the parts)
    const uint32_t part = __reduce_min_sync(0xffffffffu, tie ? static_cast<uint32_t>(best_part) : 0xffffffffu);
    if (tie && static_cast<uint32_t>(best_part) == part) {
      const unsigned long long u = best;
      const double x = __longlong_as_double(static_cast<long long>(u >> 63 ? u & ~(1ull << 63) : ~u));
      const long long to = static_cast<long long>(group) * k + o;
      a.out_scores[to] = static_cast<float>(x);
      a.out_parents[to] = best_part / splits;
      a.out_tokens[to] = best_token;
#pragma unroll
      for (int q = 0; q < kLists; ++q) at[q] += q == best_q;
    }
    __syncwarp();
  }
}

// Shared memory of `mine` parts a block, `parts` in all, k candidates each.
constexpr int shared_bytes(int mine, int parts, int k) {
  const int scores = parts * k * static_cast<int>(sizeof(unsigned long long) + sizeof(int));
  return list_bytes(mine, k) + (scores > kStages * kStageBytes ? scores : kStages * kStageBytes);
}
// Of the widest request with the most candidates in one block, rows whole.
constexpr int kMostShared = shared_bytes(kBeamMaxWidth, kBeamMaxWidth, kBeamMaxOut);
static_assert(2 * kBeamMaxOut + 32 <= kCap, "a list that is not cut down leaves room");
static_assert(kMostShared + sizeof(SelectShared) + 2048 <= 232448, "shared memory of a thread block");

struct SelectPlan {
  int ranks, splits, smem;
};

// Blocks of a cluster and parts of a row. Small batches take large clusters (up to 16 blocks, one request is one
// cluster), so that up to four blocks an SM work; a row is cut so that the parts spread evenly over them, where a part
// costs what `fixed` bytes of logits do beside its own.
SelectPlan plan_select(const BeamSelectArgs& a, int size, int most_ranks) {
  SelectPlan best{1, 1, 0};
  const long long fixed = 16384;
  int ranks = 1;
  while (ranks < most_ranks && static_cast<long long>(a.groups) * ranks * 2 <= 4ll * device_sm_count()) ranks *= 2;
  long long best_cost = LLONG_MAX;
  for (int splits = 1; splits <= 32 && a.width * splits <= kMaxParts; ++splits) {
    const long long rounds = (a.width * splits + ranks - 1) / ranks;
    const long long cost = rounds * (static_cast<long long>(a.vocab) * size / splits + fixed);
    const int parts = a.width * splits;
    const int smem = shared_bytes(static_cast<int>(rounds), parts, a.n_out);
    if (cost < best_cost && (splits == 1 || smem <= kMostShared)) {
      best_cost = cost;
      best.splits = splits;
      best.smem = smem;
    }
  }
  best.ranks = ranks;
  return best;
}

template <int TYPE>
cudaError_t launch_select(const BeamSelectArgs& a, cudaStream_t s) {
  auto kern = beam_select_kernel<TYPE>;
  static SharedMemoryOnce once;
  cudaError_t e = once.set(kern, kMostShared);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  const SelectPlan p = plan_select(a, Logits<TYPE>::SIZE, 16);
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = p.ranks;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(a.groups) * p.ranks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, kern, a, p.splits);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

cudaError_t launch_beam_select(const BeamSelectArgs& a, cudaStream_t s) {
  switch (a.type) {
    case 0: return launch_select<0>(a, s);
    case 1: return launch_select<1>(a, s);
    case 2: return launch_select<2>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace kvq
