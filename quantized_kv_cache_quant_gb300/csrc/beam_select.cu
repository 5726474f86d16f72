// Selection of beam candidates for sm_103a (kvq_beam.h): log-softmax over the
// vocabulary and the n best (beam, token) of each request in one pass over the
// logits and one launch.
//
// A cluster of thread blocks takes one request; its rows are cut into parts, and
// block r of C takes parts r, r + C, ... A part streams through shared memory in
// chunks of 32 KB, the next ones' copies in flight. Rows may start on any
// boundary of their type: copies are of aligned 16 bytes, and a thread puts its
// 8 or 4 elements together from two of them, so that a row's sum does not depend
// on where the row lies.
//   sum    every thread keeps a maximum and a sum of exp(x - maximum) of its own
//          (fp32, rescaled when the maximum grows); they meet at the part's end
//   best   within a row the order of the scores is that of the logits, so a part
//          needs its k = n_out largest logits only. Of the 16 warps' chunk maxima
//          (their j-th largest lane maxima, 16 j >= k) the smallest is a bound that at
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

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kVecs = 4;                       // 16-byte vectors a thread holds of a chunk
constexpr int kChunk = kThreads * kVecs;       // vectors of a chunk
constexpr int kStages = 3;                     // chunks in shared memory
constexpr int kStageBytes = (kChunk + 1) * 16; // and one vector more, where elements reach into it
constexpr int kCap = 1024;                     // keys of a part's list
constexpr int kCut = 512;                      // cut down to k beyond this many
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

template <int TYPE>
struct Logits;
template <>
struct Logits<0> {  // fp16
  static constexpr int SIZE = 2;
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
  __device__ static __forceinline__ float at(const void* p, long long i) { return static_cast<const float*>(p)[i]; }
  __device__ static __forceinline__ void unpack(const uint4& v, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
};
template <>
struct Logits<2> {  // bf16
  static constexpr int SIZE = 2;
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
  int count, hits;
};

// exp(x - m) for x <= m: d = x - m rounds relative to d alone, and log2(e) in two parts keeps the product's
// error from pointing one way over a whole row.
__device__ __forceinline__ float exp_below(float x, float m) {
  const float d = x - m;
  return fast_exp2(fmaf(d, kLog2eLow, d * kLog2e));
}

// The k largest keys of sh.list[0, n) to out[0, k), largest first (kNone behind the n-th). All threads, synchronised
// before and after.
__device__ __forceinline__ void rank_list(const unsigned long long* list, int n, int k, unsigned long long* out) {
  for (int i = threadIdx.x; i < k; i += kThreads)
    if (i >= n) out[i] = kNone;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    const unsigned long long key = list[i];
    int larger = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) larger += list[j] > key;
    if (larger < k) out[larger] = key;
  }
}

template <int TYPE>
__global__ void __launch_bounds__(kThreads, 2) beam_select_kernel(const BeamSelectArgs a, int splits) {
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
    if (tid == 0) sh.count = 0;

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
#pragma unroll
        for (int u = 0; u < kVecs; ++u)
          if (c + u * kThreads + tid < reach) copy(stage, c, u * kThreads + tid);
        if (tid == 0 && lead > 0 && c + kChunk < reach) copy(stage, c, kChunk);
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
    __syncthreads();  // the part before is done with the ring
#pragma unroll
    for (int it = 0; it < kStages - 1; ++it) issue(it);
    for (int it = 0, c = v0; c < v1; ++it, c += kChunk) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncthreads();  // this chunk has landed, the one before has been read
      issue(it + kStages - 1);
      uint4 v[kVecs];
      const uint4* here = reinterpret_cast<const uint4*>(ring + it % kStages * kStageBytes) + tid;
      if (lead == 0) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) v[u] = here[u * kThreads];
      } else {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) v[u] = join(here[u * kThreads], here[u * kThreads + 1]);
      }
      const int held = min(kVecs, (v1 - c - tid + kThreads - 1) / kThreads);  // vectors of this thread (may be below 1)
      // f(value, token) of every element
      auto each = [&](auto f) {
#pragma unroll
        for (int u = 0; u < kVecs; ++u) {
          if (u >= held) continue;
          float2 x[E / 2];
          L::unpack(v[u], x);
#pragma unroll
          for (int e = 0; e < E / 2; ++e) {
            f(clean(x[e].x), (c + u * kThreads + tid) * E + 2 * e);
            f(clean(x[e].y), (c + u * kThreads + tid) * E + 2 * e + 1);
          }
        }
      };
      float top = -INFINITY;  // (fmaxf passes over NaN)
#pragma unroll
      for (int u = 0; u < kVecs; ++u) {
        if (u >= held) continue;
        float2 x[E / 2];
        L::unpack(v[u], x);
#pragma unroll
        for (int e = 0; e < E / 2; ++e) top = fmaxf(top, fmaxf(x[e].x, x[e].y));
      }
      const bool infinite = top == INFINITY;
      top = clean(top);
      if (top > m) {
        s = m == -INFINITY ? 0.0f : s * exp_below(m, top);
        m = top;
      }
      if (m > -INFINITY) {
        // (a chunk's terms first: fewer roundings at the sum's size)
        if (infinite) {
          float add = 0.0f;
          each([&](float x, int) { add += exp_below(x, m); });
          s += add;
        } else {
          float2 add = make_float2(0.0f, 0.0f);
          const float2 m2 = make_float2(-m, -m), high = make_float2(kLog2e, kLog2e), low = make_float2(kLog2eLow, kLog2eLow);
#pragma unroll
          for (int u = 0; u < kVecs; ++u) {
            if (u >= held) continue;
            float2 x[E / 2];
            L::unpack(v[u], x);
#pragma unroll
            for (int e = 0; e < E / 2; ++e) {
              const float2 d = __fadd2_rn(x[e], m2);
              float2 p = __ffma2_rn(d, low, __fmul2_rn(d, high));
              // (NaN and -inf: below every normal number)
              p.x = fast_exp2(fmaxf(p.x, -200.0f));
              p.y = fast_exp2(fmaxf(p.y, -200.0f));
              add = __fadd2_rn(add, p);
            }
          }
          s += add.x + add.y;
        }
      }

      // the bound of this chunk: each warp's j-th largest lane maximum, the smallest of the warps' ones
      const bool first = c == v0;
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
        uint32_t low = sh.bound[lane % kWarps];
        return code_float(max(__reduce_min_sync(0xffffffffu, low), float_code(-INFINITY)));
      };
      if (first) bound = chunk_bound();
      // (in later chunks tokens are higher, so an equal value does not displace one in the list)
      auto wanted = [&](float x, float limit, bool equal) { return x > limit || (equal && x == limit && x > -INFINITY); };
      auto collect = [&](float limit, bool equal) {
        if (!wanted(top, limit, equal)) return;
        each([&](float x, int token) {
          if (wanted(x, limit, equal)) {
            const int i = atomicAdd(&sh.count, 1);
            if (i < kCap) sh.list[i] = make_key(x, token);
          }
        });
      };
      __syncthreads();
      const int had = sh.count;  // (at most kCut)
      __syncthreads();
      collect(bound, first);
      __syncthreads();
      int n = sh.count;
      if (n > kCap && !first) {  // a bound of this chunk's own may let fewer through
        const float tight = chunk_bound();
        if (tight > bound) {
          __syncthreads();
          if (tid == 0) sh.count = had;
          __syncthreads();
          collect(tight, true);
          __syncthreads();
          n = sh.count;
        }
      }
      if (n > kCap) {
        // the k-th largest key of what was had and this chunk, bit by bit
        unsigned long long kth = 0ull;
        for (int bit = 63; bit >= 0; --bit) {
          const unsigned long long trial = kth | (1ull << bit);
          int reach = 0;
          if (make_key(top, 0) >= trial)
            each([&](float x, int token) { reach += x > -INFINITY && make_key(x, token) >= trial; });
          for (int i = tid; i < had; i += kThreads) reach += sh.list[i] >= trial;
          if (tid == 0) sh.hits = 0;
          __syncthreads();
          reach = __reduce_add_sync(0xffffffffu, reach);
          if (lane == 0) atomicAdd(&sh.hits, reach);
          __syncthreads();
          if (sh.hits >= k) kth = trial;
          __syncthreads();
        }
        unsigned long long keep = kNone;
        if (tid < had) keep = sh.list[tid];
        if (tid == 0) sh.count = 0;
        __syncthreads();
        auto put = [&](unsigned long long key) {
          if (key >= kth) sh.list[atomicAdd(&sh.count, 1)] = key;  // (k keys, they are distinct)
        };
        if (keep != kNone) put(keep);
        each([&](float x, int token) {
          if (x > -INFINITY) put(make_key(x, token));
        });
        __syncthreads();
        bound = code_float(static_cast<uint32_t>(kth >> 32));
      } else if (n > kCut) {
        rank_list(sh.list, n, k, out);
        __syncthreads();
        for (int i = tid; i < k; i += kThreads) sh.list[i] = out[i];
        if (tid == 0) sh.count = min(n, k);
        bound = code_float(static_cast<uint32_t>(out[k - 1] >> 32));  // (n > kCut >= k)
        __syncthreads();
      }
    }

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
    const int n = min(sh.count, kCap);
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
static_assert(kMostShared + sizeof(SelectShared) + 2048 <= 232448, "shared memory of a thread block");

struct SelectPlan {
  int ranks, splits, smem;
};

// Blocks of a cluster and parts of a row. Small batches take large clusters (up to 16 blocks, one request is one
// cluster), so that about two blocks an SM work; a row is cut so that the parts spread evenly over them, where a part
// costs what `fixed` bytes of logits do beside its own.
SelectPlan plan_select(const BeamSelectArgs& a, int size, int most_ranks) {
  SelectPlan best{1, 1, 0};
  const long long fixed = 32768;
  int ranks = 1;
  while (ranks < most_ranks && static_cast<long long>(a.groups) * ranks * 2 <= 2ll * device_sm_count()) ranks *= 2;
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
