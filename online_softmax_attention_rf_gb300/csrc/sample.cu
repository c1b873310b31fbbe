// sample.cu -- a token drawn from each row of logits by temperature, top-k,
// top-p and min-p, from given random numbers.
//
// The row softmax cascade (maximum, then sum of exponentials; RedFuser: An
// Automatic Operator Fusion Framework for Cascaded Reductions on AI
// Accelerators, section 1) with a selection between the sum and the draw. With
// m the row's maximum, t_j = (m - x_j) / T * log2 e and w_j = 2^-t_j:
//   top-k keeps the k largest x_j, top-p of those the shortest run from the
//   largest down whose weights reach top_p of their sum (equal logits: lower
//   index first), min-p of those w_j >= min_p; the draw is argmax w_j / e_j.
// Both cuts fall at one place in the order by (x descending, index ascending),
// and neither needs the row sorted.
//  - A histogram of counts by t, in steps of 1/16, gives the step that top-k's cut
//    falls into, and the few steps that top-p's is to be expected in; a second one,
//    of weights, tells whether it is there, and divides those steps finely.
//  - bf16 logits have few values: a histogram by value does for them at once, where
//    the cut lies within the 1023 values below the largest.
//  - Where no more than 512 logits lie above the cut's step, as is usual, these alone
//    go on: one CTA puts them in order and finishes the row. Otherwise what lies in
//    the cut's part of a step, a few logits, is put in order at the row's end. Equal
//    logits in great numbers: histograms of the logits' bits down to one value, then
//    a count of it in the order of the indices.
// Weights are added as integers where atomics do it (to 20 bits below the power of
// two of their step, which is off by 2^-20 of them at most), and else in a fixed
// order, so that the order of the additions cannot move a cut.
//
// A cluster of CTAs takes a row: as many as leave all rows' CTAs resident, so
// that one row has many and many rows have one each. A CTA reads its share once if
// that fits shared memory beside another CTA's, else in each pass, out of L2.
// Histograms and few logits are joined through distributed shared memory.
//
// Measured (replayed, float32, top-k and top-p of one row of 32000: 7.5 us; 200 rows
// of 50001: top-k 21 us, top-p 55, no limit 23; 512 rows of 131072: min-p 71 us, top-k
// 111, top-p 207, no limit 142; bf16, 64 rows of 131072: top-k 16, top-p 45). One row
// is bound by latency: dependent loads, cluster barriers (about 0.6 us each) and the
// searches of the histograms. Many rows are bound by the passes' chains of dependent
// instructions, about 17 a logit and pass, with 16 to 32 warps an SM to run them (64
// registers a thread, two CTAs an SM): 40 to 44 % of the issue slots are used. (The bf16
// forms spill: 96 bytes where rows are held, 140 where they are read again, 0.3 % of
// the instructions of 64 rows of 131072; the float32 forms do not.)
// Memory does 10 to 25 % of its rate, and telling L2 or L1 of what comes next costs time
// (top-p 55 to 58, no limit 147 to 179).
#include <cooperative_groups.h>

#include <cfloat>

#include "paged_device.cuh"

namespace cg = cooperative_groups;

namespace rf {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kCtas = 2;  // of an SM
constexpr int kMaxCluster = 8;
constexpr int kBuckets = 1024;
constexpr int kPerUnit = 16;   // buckets of the first histogram per unit of t
constexpr int kFracBits = 42;  // of the row's sum of weights: up to 2^20 of them, of at most 1
constexpr int kFineBits = 20;  // of a weight, below the power of two of its interval
constexpr int kHalf = 17;      // of them in the lower half
// Logits that a CTA adds to its histogram before the sums are taken out of it: a
// count and the upper three bits of its weights then share a word, and the lower
// bits fit another.
constexpr int kWindow = 32 * kThreads;
static_assert((uint64_t(kWindow) << kHalf) < (1ull << 32) && kWindow * 7ull < (1ull << kHalf),
              "a window's sums fit their places");
constexpr int kMaxBlocks = 128;  // of a CTA's share, a group of 16 bytes a thread each
constexpr int kFew = kThreads;  // logits that one CTA finishes, one a thread
constexpr uint32_t kAll = 0xffffffffu;
// A weight of 1 in units of 2^-kFracBits, less 2^-20 of it (as fine_of has it).
constexpr float kWeightOne = 4398042316800.f;
constexpr float kInf = __builtin_huge_valf();
static_assert(kBuckets == 2 * kThreads, "the scan takes two buckets a thread");
static_assert(2 * kFew <= kBuckets, "a histogram's place holds the few logits");

// max(a, b, c), NaN if one of them is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float d;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
__device__ __forceinline__ uint32_t max_bf16x2_nan(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

template <typename T>
struct Elem;

template <>
struct Elem<float> {
  static constexpr int N = 4;  // in 16 bytes
  static constexpr uint32_t kLowest = 0x007fffffu;  // key of -inf
  static __device__ __forceinline__ uint4 none() {
    return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u);
  }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&y)[4]) {
    y[0] = __uint_as_float(w.x); y[1] = __uint_as_float(w.y);
    y[2] = __uint_as_float(w.z); y[3] = __uint_as_float(w.w);
  }
  // The group's maximum (NaN if one is) with m.
  static __device__ __forceinline__ float max_of(const uint4& w, float m) {
    m = max3_nan(m, __uint_as_float(w.x), __uint_as_float(w.y));
    return max3_nan(m, __uint_as_float(w.z), __uint_as_float(w.w));
  }
  // An order of unsigned numbers that is the logits' (the two zeros are one).
  static __device__ __forceinline__ uint32_t key(float x) {
    const uint32_t u = __float_as_uint(x + 0.f);
    return u ^ (static_cast<uint32_t>(static_cast<int>(u) >> 31) | 0x80000000u);
  }
  static __device__ __forceinline__ float value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
  }
};

template <>
struct Elem<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kLowest = 0x007fu;
  static __device__ __forceinline__ uint4 none() {
    return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u);
  }
  static __device__ __forceinline__ void unpack(const uint4& w, float (&y)[8]) {
    const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[2 * i] = __uint_as_float(r[i] << 16);
      y[2 * i + 1] = __uint_as_float(r[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ float max_of(const uint4& w, float m) {
    const uint32_t p = max_bf16x2_nan(max_bf16x2_nan(w.x, w.y), max_bf16x2_nan(w.z, w.w));
    return max3_nan(m, __uint_as_float(p << 16), __uint_as_float(p & 0xffff0000u));
  }
  static __device__ __forceinline__ uint32_t key(float x) { return Elem<float>::key(x) >> 16; }
  static __device__ __forceinline__ float value(uint32_t k) {
    return Elem<float>::value(k << 16 | (k & 0x8000u ? 0u : 0xffffu));
  }
};

struct Best {
  float score;
  int idx;
  float t;
};
constexpr int kNoIdx = 0x7fffffff;
__device__ __forceinline__ void take(Best& a, const Best& b) {
  if (b.score > a.score || (b.score == a.score && b.idx < a.idx)) a = b;
}

struct Shared {
  // This CTA's histogram: counts above the upper halves of the weights, and the
  // lower halves. In the cluster's first CTA few logits and their indices take
  // its place as they come.
  alignas(16) uint32_t upper[kBuckets];
  uint32_t lower[kBuckets];
  // What the others see of it, of two histograms in turn; few logits in order.
  uint64_t val[2][kBuckets];
  uint32_t num[2][kBuckets];
  uint64_t part[2];  // and of a sum of weights
  uint64_t wsum[kWarps], wlow[kWarps];
  uint32_t wcnt[kWarps];
  // a value of each CTA of the cluster
  float cmax[kMaxCluster];
  uint32_t cties[kMaxCluster];
  float csum[kMaxCluster];
  Best cbest[kMaxCluster];
  // of each warp
  float wf[kWarps];
  Best wbest[kWarps];
  // the bucket that a sum falls into
  int found, found2, found_low;
  uint32_t found_num, found_count;  // logits in it, and up to its end
  uint64_t found_rest;
  int tie_limit;
  uint32_t block_ties[kMaxBlocks];
  // few logits: of this CTA, their first place in the first CTA, and all that arrived there
  uint32_t mine, place, pushed;
  float cut_x;      // the cut among them
  int cut_limit;
};

// What a selection left: the logits above x, and of those equal to x the ones
// before an index. -inf has no probability.
struct Kept {
  float x = kNegInf;
  int limit = 0;
  __device__ __forceinline__ bool has(float y, int v) const {
    return y > x || (y == x && v < limit);
  }
};

// Where a cut falls: `kept` where that is known, else among the few logits of it up
// to x whose kPerUnit * t is in [from, to): the row's last step takes them in until
// their counts or weights reach `rest`.
struct Cut {
  Kept kept;
  float from = kInf, to = kInf, x = kInf;
  uint64_t rest = 0;  // 0: the cut is known
  bool weights = false;
};

// A thread's two buckets of the cluster's histogram.
struct Sums {
  uint64_t v[2];
  uint32_t n[2];
};

// share * total, rounded up, at least 1 (0 <= share < 1).
__device__ __forceinline__ uint64_t times_up(uint64_t total, float share) {
  const uint32_t bits = __float_as_uint(share);
  const int shift = 150 - static_cast<int>(bits >> 23);  // share = m * 2^-shift
  if (shift >= 128) return 1;  // a total below 2^63 times less than 2^-104
  const uint64_t m = (bits & 0x7fffffu) | 0x800000u;
  const uint64_t hi = __umul64hi(total, m), lo = total * m;
  if (shift >= 64) return (hi >> (shift - 64)) + 1;
  const uint64_t q = hi << (64 - shift) | lo >> shift;
  return q + ((lo << (64 - shift)) != 0 || q == 0 ? 1 : 0);
}

template <typename T, bool kHeld>
struct Row {
  using E = Elem<T>;
  const SampleArgs& a;
  Shared& sh;
  cg::cluster_group cluster;
  int rank, size;
  int tid, warp, lane;
  const T* base;     // the row's start rounded down to 16 bytes (groups are read from here)
  uint4* held;       // this CTA's groups in shared memory
  int first;         // the row's first element, counted from base
  int end;           // one past its last
  int g0, ng;        // this CTA's groups of 16 bytes
  float max, c16;    // maximum, kPerUnit * log2(e) / temperature
  int turn = 0;      // of the two places that others read

  __device__ __forceinline__ Row(const SampleArgs& a_, Shared& s)
      : a(a_), sh(s), cluster(cg::this_cluster()) {}

  // What a selection kept: everything without kPart.
  template <bool kPart>
  static __device__ __forceinline__ bool in(const Kept& kept, float x, int v) {
    return kPart ? kept.has(x, v) : x > kNegInf;
  }

  // A group's logits; what lies outside the row counts as -inf.
  __device__ __forceinline__ uint4 load_group(int g) const {
    const int v = g * E::N;
    if (v >= first && v + E::N <= end) return __ldg(reinterpret_cast<const uint4*>(base) + g);
    T y[E::N];
#pragma unroll
    for (int i = 0; i < E::N; ++i)
      y[i] = v + i >= first && v + i < end ? base[v + i] : T(kNegInf);
    uint4 w;
    memcpy(&w, y, 16);
    return w;
  }

  // U of this thread's groups, g and those kThreads behind each other, from where
  // the row is; groups that there are not count as -inf.
  template <int U, bool kFromShared>
  __device__ __forceinline__ void fetch(uint4 (&w)[U], int g) const {
    const uint4* from = kFromShared ? held : reinterpret_cast<const uint4*>(base) + g0;
    // the first and the last group may not lie wholly in the row
    const int f0 = !kFromShared && g0 == 0 && first > 0 ? 1 : 0;
    const int f1 = kFromShared ? ng : min(ng, end / E::N - g0);
    if (g >= f0 && g + (U - 1) * kThreads < f1) {
#pragma unroll
      for (int j = 0; j < U; ++j)
        w[j] = kFromShared ? from[g + j * kThreads] : __ldg(from + g + j * kThreads);
    } else {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int h = g + j * kThreads;
        w[j] = E::none();
        if (h < ng) w[j] = kFromShared ? from[h] : load_group(g0 + h);
      }
    }
  }

  // Reads the row; this thread's maximum (NaN if one is).
  __device__ __forceinline__ float read() const {
    constexpr int U = 6;
    float m = kNegInf;
    for (int g = tid; g < ng; g += U * kThreads) {
      uint4 w[U];
      fetch<U, false>(w, g);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (kHeld && g + j * kThreads < ng) held[g + j * kThreads] = w[j];
        m = E::max_of(w[j], m);
      }
    }
    return m;
  }

  // f(x, index from base) for this thread's logits of at least `least` and some
  // others, in ascending order.
  template <typename F>
  __device__ __forceinline__ void each_from(float least, F&& f) const {
    constexpr int U = 4;
    for (int g = tid; g < ng; g += U * kThreads) {
      uint4 w[U];
      fetch<U, kHeld>(w, g);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (E::max_of(w[j], kNegInf) < least) continue;
        float y[E::N];
        E::unpack(w[j], y);
#pragma unroll
        for (int i = 0; i < E::N; ++i) f(y[i], (g0 + g + j * kThreads) * E::N + i);
      }
    }
  }

  // f(group, index of its first logit from base, sum) for this thread's groups with
  // a logit of at least `least` (kAllGroups: for all of them, and for groups of -inf
  // behind them); the sum of what f adds to `sum` (weights, a few at a time in
  // float32, so with 15 roundings at most, and these as integers) in units of
  // 2^-kFracBits.
  template <bool kAllGroups, typename F>
  __device__ __forceinline__ uint64_t groups_sum(float least, int g, int batches, F&& f) const {
    constexpr int U = 4, kRun = 16 / E::N;
    uint64_t sum = 0;
#pragma unroll 1
    for (int k = 0; k < batches; ++k, g += U * kThreads) {
      uint4 w[U];
      fetch<U, kHeld>(w, g);
#pragma unroll
      for (int j = 0; j < U; j += kRun) {
        float run = 0.f;
#pragma unroll
        for (int i = j; i < j + kRun; ++i)
          if (kAllGroups || E::max_of(w[i], kNegInf) >= least)
            f(w[i], (g0 + g + i * kThreads) * E::N, run);
        sum += __float2ull_rn(run * kWeightOne);
      }
    }
    return sum;
  }
  // Batches of groups of a thread: of all, and of a window.
  __device__ __forceinline__ int batches() const {
    return (ng + 4 * kThreads - 1) / (4 * kThreads);
  }
  static constexpr int kWindowBatches = kWindow / kThreads / (4 * E::N);

  // kPerUnit * t: not below 0; +inf for -inf
  __device__ __forceinline__ float t16_of(float x) const { return __fmul_rn(max - x, c16); }
  static __device__ __forceinline__ int bucket_at(float t16) {  // t16 in [0, kBuckets)
    return __float_as_int(__fadd_rz(t16, 8388608.f)) & (kBuckets - 1);
  }
  __device__ __forceinline__ int bucket_of(float x) const {
    return bucket_at(fminf(t16_of(x), kBuckets - 1.f));
  }
  // A weight over 2^-e, e the power of its interval, as an integer: less than 2^20
  // (the weight is taken 2^-20 of it smaller).
  static __device__ __forceinline__ uint32_t fine_of(float t16) {
    const float e16 = __fadd_rz(t16, 134217728.f) - 134217728.f;  // to a multiple of 16
    const float f = ex2_approx(fmaf(e16 - t16, 1.f / kPerUnit, -1.3758e-6f));
    return __float_as_uint(f + 8.f) - 0x41000000u;
  }

  // The least of the logits' type whose t16 is below `from` (all of the warp): there is
  // none for 0, which is the maximum's own.
  __device__ float least_below(float from) const {
    uint32_t lo = E::kLowest + 1, hi = E::key(max);
    while (lo < hi) {
      const uint32_t step = (hi - lo) / 32 + 1;
      const uint32_t is = __ballot_sync(kAll, t16_of(E::value(min(hi, lo + lane * step))) < from);
      const int f = is != 0 ? __ffs(is) - 1 : 32;
      if (f < 32) hi = min(hi, lo + f * step);
      lo = f > 0 ? lo + (f - 1) * step + 1 : hi;
    }
    return from > 0.f ? E::value(hi) : kInf;
  }

  // A logit that no logit up to the end of step hi lies below.
  __device__ __forceinline__ float reach(int hi) const {
    return hi < kBuckets - 1 ? max - (hi + 2) / c16 : kNegInf;
  }

  // The CTA's histogram in this thread's two buckets, and the sum of groups_sum():
  // f(group, index, sum, add) adds logits by add(bucket, t16).
  template <bool kWeights, typename F>
  __device__ Sums histogram(float least, uint64_t* sum, F&& f) const {
    uint2* upper = reinterpret_cast<uint2*>(sh.upper);
    uint2* lower = reinterpret_cast<uint2*>(sh.lower);
    upper[tid] = lower[tid] = make_uint2(0, 0);
    __syncthreads();
    Sums s{};
    auto add = [&](int b, float t16) {
      const uint32_t f = kWeights ? fine_of(t16) : 0u;
      atomicAdd(&sh.upper[b], (1u << kHalf) + (f >> kHalf));
      if (kWeights) atomicAdd(&sh.lower[b], f & ((1u << kHalf) - 1));
    };
    for (int k = 0; k < batches(); k += kWindowBatches) {
      *sum += groups_sum<false>(least, tid + k * 4 * kThreads, min(kWindowBatches, batches() - k),
                         [&](const uint4& w, int v, float& run) { f(w, v, run, add); });
      __syncthreads();
      const uint2 u = upper[tid], l = lower[tid];
      upper[tid] = lower[tid] = make_uint2(0, 0);
      const uint32_t us[2] = {u.x, u.y}, ls[2] = {l.x, l.y};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        s.n[i] += us[i] >> kHalf;
        s.v[i] += (uint64_t(us[i] & ((1u << kHalf) - 1)) << kHalf) + ls[i];
      }
      __syncthreads();
    }
    if (!kWeights) {
      s.v[0] = s.n[0];
      s.v[1] = s.n[1];
    }
    return s;
  }

  // The cluster's histogram from its CTAs', and the sum over all of their threads
  // of a weight each.
  template <bool kWeights, bool kPart>
  __device__ uint64_t join(Sums& s, uint64_t part) {
    if (kPart) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) part += __shfl_xor_sync(kAll, part, o);
      if (lane == 0) sh.wsum[warp] = part;
      __syncthreads();
      part = sh.wsum[lane & (kWarps - 1)];
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) part += __shfl_xor_sync(kAll, part, o);
      __syncthreads();
    }
    if (size == 1) return part;
    if (kWeights)
      *reinterpret_cast<ulonglong2*>(&sh.val[turn][2 * tid]) = make_ulonglong2(s.v[0], s.v[1]);
    *reinterpret_cast<uint2*>(&sh.num[turn][2 * tid]) = make_uint2(s.n[0], s.n[1]);
    if (kPart && tid == 0) sh.part[turn] = part;
    cluster.sync();
#pragma unroll
    for (int q = 1; q < kMaxCluster; ++q) {
      if (q >= size) break;
      const int other = (rank + q) & (size - 1);
      if (kWeights) {
        const ulonglong2 v =
            *reinterpret_cast<ulonglong2*>(cluster.map_shared_rank(&sh.val[turn][2 * tid], other));
        s.v[0] += v.x;
        s.v[1] += v.y;
      }
      const uint2 n =
          *reinterpret_cast<uint2*>(cluster.map_shared_rank(&sh.num[turn][2 * tid], other));
      s.n[0] += n.x;
      s.n[1] += n.y;
      if (kPart) part += *cluster.map_shared_rank(&sh.part[turn], other);
    }
    if (!kWeights) {
      s.v[0] = s.n[0];
      s.v[1] = s.n[1];
    }
    turn ^= 1;  // this place is written again only behind the next histogram's barrier
    return part;
  }

  // Inclusive sum over the warp's lanes.
  template <typename U>
  __device__ __forceinline__ U scan(U s) const {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const U u = __shfl_up_sync(kAll, s, o);
      if (lane >= o) s += u;
    }
    return s;
  }

  // The bucket in which the running sum of h.v reaches the target, aim(sum of all), and
  // what the target is behind the sum before it; none: -1. Each warp adds up its 64
  // buckets; the one that the target falls into looks closer.
  template <typename F>
  __device__ int find_by(const Sums& h, uint64_t* rest, F&& aim) const {
    const uint64_t v = sum_of_warp(h.v[0] + h.v[1]);
    const uint32_t n = __reduce_add_sync(kAll, h.n[0] + h.n[1]);
    if (lane == 0) {
      sh.wsum[warp] = v;
      sh.wcnt[warp] = n;
    }
    if (tid == 0) sh.found = -1;
    __syncthreads();
    const uint64_t s = scan(lane < kWarps ? sh.wsum[lane] : 0);
    const uint64_t target = aim(__shfl_sync(kAll, s, 31));
    if (warp == __popc(__ballot_sync(kAll, s < target))) {
      const uint64_t before = before_lane(s, h);
      const uint32_t count = __reduce_add_sync(kAll, lane < warp ? sh.wcnt[lane] : 0u) +
                             scan(h.n[0] + h.n[1]);
      const bool odd = target > before + h.v[0];
      if (before < target && target <= before + h.v[0] + h.v[1]) {
        sh.found = 2 * tid + odd;
        sh.found_num = odd ? h.n[1] : h.n[0];
        sh.found_count = odd ? count : count - h.n[1];
        sh.found_rest = target - before - (odd ? h.v[0] : 0);
      }
    }
    __syncthreads();
    const int b = sh.found;
    *rest = sh.found_rest;
    __syncthreads();
    return b;
  }
  // clamp: the last bucket with anything in it where all of them do not reach it.
  __device__ int find(const Sums& h, uint64_t target, uint64_t* rest, bool clamp = false) const {
    return find_by(h, rest, [&](uint64_t all) { return clamp ? min(target, all) : target; });
  }
  __device__ __forceinline__ uint64_t sum_of_warp(uint64_t s) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    return s;
  }
  // Sum before a lane's buckets, s the warps' running sums.
  __device__ __forceinline__ uint64_t before_lane(uint64_t s, const Sums& h) const {
    const uint64_t before = __shfl_sync(kAll, s, warp > 0 ? warp - 1 : 0);
    return (warp > 0 ? before : 0) + scan(h.v[0] + h.v[1]) - h.v[0] - h.v[1];
  }

  // The steps [*lo, *hi] that a cut of `kept` (everything without kPart) falls
  // into: the one with the target'th logit, and *rest to go in it; or, with
  // kWeights, those that in all likelihood have the place where the weights reach
  // *rest, which is the share of their sum *total. *enough: the step whose end is
  // certainly behind the cut. False: there is no cut. sh.found_num, sh.found_count:
  // the logits in step *enough, and up to its end.
  template <bool kWeights, bool kPart>
  __device__ bool steps(uint64_t target, float share, const Kept& kept, int* lo, int* hi,
                        uint64_t* total, uint64_t* rest, int* enough) {
    *reinterpret_cast<uint2*>(&sh.upper[2 * tid]) = make_uint2(0, 0);
    __syncthreads();
    const uint64_t sum =
        groups_sum<!kPart>(kPart ? kept.x : kNegInf, tid, batches(),
                           [&](const uint4& w, int v, float& run) {
          float y[E::N];
          E::unpack(w, y);
#pragma unroll
          for (int i = 0; i < E::N; ++i) {
            const float t16 = t16_of(y[i]);
            const bool is = in<kPart>(kept, y[i], v + i);
            if (kWeights) {
              const float q = ex2_approx(t16 * (-1.f / kPerUnit));
              run += kPart && !is ? 0.f : q;  // -inf weighs nothing
            }
            // the step in the bits from 2 on: a byte offset
            const uint32_t at = __float_as_uint(__fadd_rz(fminf(t16, kBuckets - 1.f), 2097152.f)) &
                                (4 * kBuckets - 4);
            if (is)
              atomicAdd(reinterpret_cast<uint32_t*>(reinterpret_cast<char*>(sh.upper) + at), 1u);
          }
        });
    __syncthreads();
    Sums s{};
    s.n[0] = sh.upper[2 * tid];
    s.n[1] = sh.upper[2 * tid + 1];
    *total = join<false, kWeights>(s, sum);
    if (!kWeights) {
      s.v[0] = s.n[0];
      s.v[1] = s.n[1];
      *lo = *hi = *enough = find(s, target, rest);
      return *lo >= 0;
    }
    *rest = times_up(*total, share);
    // Where it is to be expected: a logit's weight is the step's middle one, give or
    // take 1.3 % (the spread of a number within 4.4 %), so that the sum is off by 1.3
    // % of the root of the sum of the weights' squares; five times that, and some.
    // The logits that are certainly enough: the least that a step's weights can be
    // reaches the sum with them. 2^-18 covers the roundings of the sums, the weights
    // and t. Both searches go together, as in find_by().
    float squares = 0.f;
    Sums low{};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float w = ex2_approx((2 * tid + i + 0.5f) * (-1.f / kPerUnit));
      squares += s.n[i] * w * w;
      s.v[i] = s.n[i] * __float2ull_rn(w * kWeightOne);
      low.v[i] = s.n[i] * __float2ull_rn(ex2_approx((2 * tid + i + 1) * (-1.f / kPerUnit)) *
                                         (kWeightOne * (1.f - 0x1p-18f)));
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) squares += __shfl_xor_sync(kAll, squares, o);
    const uint64_t v = sum_of_warp(s.v[0] + s.v[1]), l = sum_of_warp(low.v[0] + low.v[1]);
    const uint32_t n = __reduce_add_sync(kAll, s.n[0] + s.n[1]);
    if (lane == 0) {
      sh.wsum[warp] = v;
      sh.wlow[warp] = l;
      sh.wcnt[warp] = n;
      sh.wf[warp] = squares;
    }
    if (tid == 0) {
      sh.found_low = -1;
      sh.found_count = kAll;
    }
    __syncthreads();
    squares = sh.wf[lane & (kWarps - 1)];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) squares += __shfl_xor_sync(kAll, squares, o);
    const uint64_t off = __float2ull_rn(kWeightOne * 0.065f * sqrtf(squares)) + (*total >> 11);
    const uint64_t mid = scan(lane < kWarps ? sh.wsum[lane] : 0);
    const uint64_t least = scan(lane < kWarps ? sh.wlow[lane] : 0);
    const uint64_t all = __shfl_sync(kAll, mid, 31);
    const uint64_t one = min(*rest > off ? *rest - off : 1, all), two = min(*rest + off, all);
    if (warp == __popc(__ballot_sync(kAll, mid < one)) ||
        warp == __popc(__ballot_sync(kAll, mid < two))) {
      const uint64_t before = before_lane(mid, s), end = before + s.v[0] + s.v[1];
      if (before < one && one <= end) sh.found = 2 * tid + (one > before + s.v[0]);
      if (before < two && two <= end) sh.found2 = 2 * tid + (two > before + s.v[0]);
    }
    if (warp == __popc(__ballot_sync(kAll, least < *rest))) {
      const uint64_t before = before_lane(least, low);
      const uint32_t count = __reduce_add_sync(kAll, lane < warp ? sh.wcnt[lane] : 0u) +
                             scan(s.n[0] + s.n[1]);
      const bool odd = *rest > before + low.v[0];
      if (before < *rest && *rest <= before + low.v[0] + low.v[1]) {
        sh.found_low = 2 * tid + odd;
        sh.found_count = odd ? count : count - s.n[1];
      }
    }
    __syncthreads();
    *lo = min(sh.found, kBuckets - 2);
    *hi = min(sh.found2, kBuckets - 2);
    *enough = sh.found_low;
    __syncthreads();
    return true;
  }

  // A cut of `kept` (everything without kPart) at the target'th logit, or, with
  // kWeights, where the weights reach a share of their sum *total, by a histogram of
  // the largest logit's 1023 next values: with 8 bits of a value (bf16) they span far
  // enough for most rows, a value's logits weigh the same, and nothing has to be
  // divided further. False: the cut lies below these values, or there is none.
  // sh.found_count: the logits down to the cut's value.
  template <bool kWeights, bool kPart>
  __device__ bool by_value(uint64_t target, float share, const Kept& kept, bool last, Cut* cut,
                           uint64_t* total) {
    *reinterpret_cast<uint2*>(&sh.upper[2 * tid]) = make_uint2(0, 0);
    __syncthreads();
    const uint32_t top = E::key(max);
    uint64_t sum =
        groups_sum<!kPart>(kPart ? kept.x : kNegInf, tid, batches(),
                           [&](const uint4& w, int v, float& run) {
          float y[E::N];
          E::unpack(w, y);
          uint32_t below[E::N];
          bool rest = false;  // of the weights: each by itself
#pragma unroll
          for (int i = 0; i < E::N; ++i) {
            below[i] = in<kPart>(kept, y[i], v + i) ? top - E::key(y[i]) : kAll;
            rest |= below[i] >= kBuckets - 1;
            if (below[i] < kBuckets - 1) atomicAdd(&sh.upper[below[i]], 1u);
          }
          if (kWeights && rest) {
#pragma unroll
            for (int i = 0; i < E::N; ++i)
              if (below[i] >= kBuckets - 1 && below[i] != kAll)
                run += ex2_approx(t16_of(y[i]) * (-1.f / kPerUnit));
          }
        });
    __syncthreads();
    Sums s{};
    s.n[0] = sh.upper[2 * tid];
    s.n[1] = sh.upper[2 * tid + 1];
    sum = join<false, kWeights>(s, sum);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (kWeights) s.v[i] = s.n[i] == 0 ? 0 : s.n[i] * weight_of(E::value(top - (2 * tid + i)));
    uint64_t rest;
    const int b = find_by(s, &rest, [&](uint64_t all) {
      if (!kWeights) return target;
      *total = all + sum;
      return times_up(*total, share);
    });
    if (b < 0) return false;
    *cut = at_value<kWeights, kPart>(E::value(top - b), rest, kept, last);
    return true;
  }
  // Whether by_value() reaches weights of 2^-16, below which a top-p's cut seldom lies.
  __device__ __forceinline__ bool values_suffice() const {
    const uint32_t top = E::key(max);
    return top - E::kLowest < kBuckets || t16_of(E::value(top - (kBuckets - 2))) >= 16.f * kPerUnit;
  }
  // A value's weight in units of 2^-kFracBits.
  __device__ __forceinline__ uint64_t weight_of(float x) const {
    return __float2ull_rn(ex2_approx(t16_of(x) * (-1.f / kPerUnit)) * kWeightOne);
  }
  // The cut of `kept` that takes the logits above x, and of the sh.found_num equal to
  // it the first whose counts, or weights in units of 2^-kFracBits, reach rest. last:
  // as for narrow().
  template <bool kWeights, bool kPart>
  __device__ Cut at_value(float x, uint64_t rest, const Kept& kept, bool last) const {
    if (kWeights) {
      const uint64_t w = weight_of(x);
      rest = w > 0 ? (rest + w - 1) / w : kAll;
    }
    const uint32_t n = sh.found_num;
    const int limit = kPart && x == kept.x ? kept.limit : kNoIdx;
    if (rest >= n) return Cut{Kept{x, limit}};
    // the row's last step takes the first `rest` of few
    if (n <= kFew && last) return Cut{Kept{x, limit}, 0.f, kInf, x, rest, false};
    return Cut{Kept{x, min(limit, tie_limit(x, static_cast<uint32_t>(rest)))}};
  }

  // Few logits go to the cluster's first CTA: collected in the CTA (a counter of the
  // cluster's that all of them add to costs its way there and back each time), then
  // sent together. What others read of this CTA's last histogram is not touched.
  __device__ __forceinline__ void push_one(float x, int v) const {
    const uint32_t at = atomicAdd(&sh.mine, 1u);
    if (at < kFew) {
      sh.num[turn][at] = __float_as_uint(x);
      sh.num[turn][kFew + at] = static_cast<uint32_t>(v);
    }
  }
  __device__ __forceinline__ void send() const {
    __syncthreads();
    const uint32_t n = min(sh.mine, static_cast<uint32_t>(kFew));
    if (tid == 0 && n > 0) sh.place = atomicAdd(cluster.map_shared_rank(&sh.pushed, 0), n);
    __syncthreads();
    if (tid == 0) sh.mine = 0;
    if (tid < n) {
      const uint32_t at = sh.place + tid;
      if (at < kFew) {
        *cluster.map_shared_rank(&sh.upper[at], 0) = sh.num[turn][tid];
        *cluster.map_shared_rank(&sh.lower[at], 0) = sh.num[turn][kFew + tid];
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void push(float least, F&& is) const {
    each_from(least, [&](float x, int v) {
      if (is(x, v)) push_one(x, v);
    });
    send();
    cluster.sync();
  }

  // This thread's logit and index of the few, in order (one CTA); how many.
  __device__ int in_order(float* x, int* v) const {
    const int n = min(static_cast<int>(sh.pushed), kFew);
    // (x descending, index ascending) as one number; its rank by counting
    uint64_t* all = sh.val[0];
    uint64_t* sorted = sh.val[1];
    const uint64_t mine =
        tid < n ? uint64_t(Elem<float>::key(__uint_as_float(sh.upper[tid]))) << 32 | ~sh.lower[tid]
                : 0;
    if (tid < (n + 7) / 8 * 8) all[tid] = mine;
    __syncthreads();
    if (tid < n) {
      int r = 0;
      for (int j = 0; j < n; j += 8) {
        ulonglong2 o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = *reinterpret_cast<const ulonglong2*>(all + j + 2 * i);
#pragma unroll
        for (int i = 0; i < 4; ++i) r += (o[i].x > mine) + (o[i].y > mine);
      }
      sorted[r] = mine;
    }
    __syncthreads();
    const uint64_t got = tid < n ? sorted[tid] : 0;
    *x = tid < n ? Elem<float>::value(static_cast<uint32_t>(got >> 32)) : kNegInf;
    *v = tid < n ? static_cast<int>(~static_cast<uint32_t>(got)) : kNoIdx;
    return n;
  }

  // Sum over the threads before this one, and over all.
  __device__ uint64_t sum_before(uint64_t u, uint64_t* all) const {
    const uint64_t s = scan(u);
    if (lane == 31) sh.wsum[warp] = s;
    __syncthreads();
    const uint64_t w = scan(lane < kWarps ? sh.wsum[lane] : 0);
    *all = __shfl_sync(kAll, w, 31);
    const uint64_t before = __shfl_sync(kAll, w, warp > 0 ? warp - 1 : 0);
    __syncthreads();
    return (warp > 0 ? before : 0) + s - u;
  }

  // What is left of `kept` when the running sum of counts, or of weights (rest: of
  // them in units of 2^-kFracBits), in the order of the logits, is cut within the
  // steps [lo, hi] by `rest`: counted from lo on, or, with kWeights, from the first
  // logit on. n: the logits in these steps, or more. last: nothing is cut after it,
  // so that few logits may be left to the row's last step.
  template <bool kWeights, bool kPart>
  __device__ Cut narrow(int lo, int hi, uint32_t n, uint64_t rest, const Kept& kept, bool last) {
    // The steps divided by a power of two: a part lies within one unit of t, and
    // what is subtracted and multiplied here is exact.
    int parts, part;  // log2 of the parts of a step; the one with the cut (-1: all)
    float scale, top, bottom;
    auto part_of = [&](float t16) { return bucket_at(fminf((t16 - top) * scale, kBuckets - 1.f)); };
    for (const uint64_t whole = rest;; lo = 0, hi = kBuckets - 2) {
      parts = 0;
      part = -1;
      while ((hi - lo + 1) << (parts + 1) <= kBuckets) ++parts;
      scale = static_cast<float>(1 << parts);
      top = lo;
      bottom = hi < kBuckets - 1 ? hi + 1.f : kInf;
      if (!kWeights && (n <= kFew || hi == kBuckets - 1)) break;
      if constexpr (sizeof(T) == 2) {  // no more values than buckets: by value
        const uint32_t upto = lo > 0 ? E::key(max - top / c16 * (1.f - 0x1p-21f)) : E::key(max);
        if (upto - E::key(max - bottom / c16 * (1.f + 0x1p-21f)) < kBuckets) {
          uint64_t above = 0;
          Sums h = histogram<false>(
              reach(hi), &above, [&](const uint4& w, int v, float& run, auto&& add) {
                float y[E::N];
                E::unpack(w, y);
#pragma unroll
                for (int i = 0; i < E::N; ++i) {
                  const float t16 = t16_of(y[i]);
                  if (!in<kPart>(kept, y[i], v + i)) continue;
                  if (kWeights && t16 < top) run += ex2_approx(t16 * (-1.f / kPerUnit));
                  const uint32_t below = upto - E::key(y[i]);
                  if (t16 >= top && t16 < bottom && below < kBuckets) add(below, t16);
                }
              });
          above = join<false, kWeights>(h, above);
          if (kWeights) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
              h.v[i] = h.n[i] == 0 ? 0 : h.n[i] * weight_of(E::value(upto - (2 * tid + i)));
          }
          const bool all = !kWeights || (lo == 0 && hi == kBuckets - 2);
          if (kWeights && whole <= above && !all) continue;
          const uint64_t target = !kWeights ? whole : whole > above ? whole - above : 1;
          part = find(h, target, &rest, all);
          if (part < 0 && !all) continue;  // not in these steps, against all likelihood
          if (part < 0) return Cut{kept};  // what is left weighs nothing
          return at_value<kWeights, kPart>(E::value(upto - part), rest, kept, last);
        }
      }
      uint64_t above = 0;
      Sums h = histogram<kWeights>(
          reach(hi), &above, [&](const uint4& w, int v, float& run, auto&& add) {
            float y[E::N], t16[E::N];
            E::unpack(w, y);
            bool any = false;
#pragma unroll
            for (int i = 0; i < E::N; ++i) {
              t16[i] = t16_of(y[i]);
              if (kPart && !kept.has(y[i], v + i)) t16[i] = kInf;
              if (kWeights) run += t16[i] < top ? ex2_approx(t16[i] * (-1.f / kPerUnit)) : 0.f;
              any |= t16[i] >= top && t16[i] < bottom;
            }
            if (!any) return;
#pragma unroll
            for (int i = 0; i < E::N; ++i)
              if (t16[i] >= top && t16[i] < bottom) add(part_of(t16[i]), t16[i]);
          });
      above = join<kWeights, kWeights>(h, above);
      if (kWeights) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int e = kFracBits - kFineBits - (lo + ((2 * tid + i) >> parts)) / kPerUnit;
          h.v[i] = e >= 0 ? h.v[i] << e : h.v[i] >> -e;
        }
        // not in these steps, against all likelihood: in any of them
        const bool all = lo == 0 && hi == kBuckets - 2;
        if (whole <= above && !all) continue;
        part = find(h, whole > above ? whole - above : 1, &rest, all);
        if (part < 0 && !all) continue;
      } else {
        part = find(h, whole, &rest, true);
      }
      n = sh.found_num;
      break;
    }
    const int step = lo + (part > 0 ? part >> parts : 0);
    if (kWeights) {  // in units of the part's weights
      const int e = kFracBits - kFineBits - step / kPerUnit;
      rest = e >= 0 ? (rest + (uint64_t(1) << e) - 1) >> e : rest << -e;
    }
    // The part's keys lie in [klo, khi]: max - x is between its ends over c16, up to
    // rounding; 2^-21 of it is more than that.
    const float from = part < 0 ? top : top + part / scale;
    const float to = part < 0 ? bottom : top + (part + 1) / scale;
    uint32_t khi = from > 0.f ? E::key(max - from / c16 * (1.f - 0x1p-21f)) : E::key(max);
    uint32_t klo = E::kLowest;
    if (to < kInf) klo = umax(klo, E::key(max - to / c16 * (1.f + 0x1p-21f)));
    bool narrowed = false;
    auto is = [&](float x, int v) {
      const float t16 = t16_of(x);
      return x >= E::value(klo) && x <= E::value(khi) && t16 >= from && (t16 < to || to == kInf) &&
             in<kPart>(kept, x, v);
    };
    while (n > kFew && khi > klo) {
      int s = 0;
      while (((khi - klo) >> s) >= kBuckets) ++s;
      uint64_t none = 0;
      Sums h = histogram<kWeights>(E::value(klo), &none,
                                   [&](const uint4& w, int v, float&, auto&& add) {
                                     float y[E::N];
                                     E::unpack(w, y);
#pragma unroll
                                     for (int e = 0; e < E::N; ++e)
                                       if (is(y[e], v + e))
                                         add((khi - E::key(y[e])) >> s, t16_of(y[e]));
                                   });
      join<kWeights, false>(h, 0);
      narrowed = true;
      const int i = find(h, rest, &rest, true);
      n = sh.found_num;
      khi -= static_cast<uint32_t>(i) << s;
      klo = s > 0 ? umax(klo, khi - ((1u << s) - 1)) : khi;
    }
    if (n > kFew) {  // one value
      const float x = E::value(klo);
      if (kWeights) {
        const uint64_t f = fine_of(t16_of(x));
        rest = (rest + f - 1) / f;
      }
      const int limit = tie_limit(x, static_cast<uint32_t>(rest < kAll ? rest : kAll));
      return Cut{Kept{x, x == kept.x ? min(limit, kept.limit) : limit}};
    }
    if (last)  // (nothing below the lowest key is left; of kept what it was)
      return Cut{kPart && kept.x >= E::value(klo) ? kept : Kept{E::value(klo), kNoIdx}, from, to,
                 narrowed ? E::value(khi) : kInf, rest, kWeights};
    push(E::value(klo), is);
    if (rank == 0) {
      float x;
      int v;
      const int m = in_order(&x, &v);
      uint64_t all;
      const uint64_t u = tid < m ? (kWeights ? fine_of(t16_of(x)) : 1) : 0;
      const uint64_t before = sum_before(u, &all);
      // the last one that is in; all of them if rounding leaves the sum short
      if (tid < m && before < rest && (before + u >= rest || tid == m - 1))
        for (int q = 0; q < size; ++q) {
          *cluster.map_shared_rank(&sh.cut_x, q) = x;
          *cluster.map_shared_rank(&sh.cut_limit, q) = v + 1;
        }
      if (tid == 0) sh.pushed = 0;
    }
    cluster.sync();
    return Cut{Kept{sh.cut_x, sh.cut_limit}};
  }
  static __device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

  // Of the logits equal to x the first `ties` are those before the returned index.
  __device__ int tie_limit(float x, uint32_t ties) const {
    if (tid < kMaxBlocks) sh.block_ties[tid] = 0;
    if (tid == 0) sh.tie_limit = kNoIdx;
    __syncthreads();
    each_from(x, [&](float y, int v) {
      if (y == x) atomicAdd(&sh.block_ties[(v / E::N - g0) / kThreads], 1u);
    });
    __syncthreads();
    uint32_t n = 0;  // of the CTA, and before each of a lane's blocks
    uint32_t before[kMaxBlocks / 32];
#pragma unroll
    for (int i = 0; i < kMaxBlocks / 32; ++i) {
      const uint32_t s = scan(sh.block_ties[32 * i + lane]);
      before[i] = n + s;
      n += __shfl_sync(kAll, s, 31);
    }
    if (tid < size) *cluster.map_shared_rank(&sh.cties[rank], tid) = n;
    cluster.sync();
    uint32_t others = 0;
    for (int q = 0; q < rank; ++q) others += sh.cties[q];
    if (ties <= others) return 0;
    uint32_t left = ties - others;
    if (left >= n) return kNoIdx;
    // the block with the left'th of this CTA's, and in it the one
    int block = 0;
#pragma unroll
    for (int i = 0; i < kMaxBlocks / 32; ++i)
      block += __popc(__ballot_sync(kAll, before[i] < left));
#pragma unroll
    for (int i = 0; i < kMaxBlocks / 32; ++i) {
      const uint32_t s = __shfl_sync(kAll, before[i], (block - 1) & 31);
      if (block > 0 && (block - 1) / 32 == i) left -= s;
    }
    uint4 w[1];
    fetch<1, kHeld>(w, block * kThreads + tid);
    float y[E::N];
    E::unpack(w[0], y);
    uint32_t mine = 0;
#pragma unroll
    for (int i = 0; i < E::N; ++i) mine += y[i] == x;
    const uint32_t s = scan(mine);
    if (lane == 31) sh.wcnt[warp] = s;
    __syncthreads();
    uint32_t ahead = __reduce_add_sync(kAll, lane < warp ? sh.wcnt[lane] : 0u) + s - mine;
    if (ahead < left && left <= ahead + mine) {
#pragma unroll
      for (int i = 0; i < E::N; ++i)
        if (y[i] == x && ++ahead == left)
          sh.tie_limit = (g0 + block * kThreads + tid) * E::N + i + 1;
    }
    __syncthreads();
    return sh.tie_limit;
  }

  // The best and the sum of the CTA's threads, in a fixed order, in warp 0.
  __device__ __forceinline__ void reduce(Best& best, float& sum) const {
    auto step = [&](int o) {
      const Best other{__shfl_xor_sync(kAll, best.score, o), __shfl_xor_sync(kAll, best.idx, o),
                       __shfl_xor_sync(kAll, best.t, o)};
      take(best, other);
      sum += __shfl_xor_sync(kAll, sum, o);
    };
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) step(o);
    __syncthreads();
    if (lane == 0) {
      sh.wbest[warp] = best;
      sh.wf[warp] = sum;
    }
    __syncthreads();
    if (warp == 0) {
      best = sh.wbest[lane & (kWarps - 1)];
      sum = sh.wf[lane & (kWarps - 1)];
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) step(o);
    }
  }

  __device__ __forceinline__ void answer(int b, const Best& best, float sum, bool bad,
                                         bool greedy) const {
    const bool none = bad || best.idx == kNoIdx;
    if (none) record_status(a.status, dev_code(kDevBadList, kKerSample, 1));
    a.token[b] = none ? -1 : best.idx - first;
    if (a.logprob != nullptr)
      a.logprob[b] = none     ? __int_as_float(0x7fc00000)
                     : greedy ? 0.f
                              : -(best.t + log2f(sum)) * kLn2;
  }

  // The few logits that the last cut falls into (one CTA): those that are in join
  // the others' best and sum, which thread 0 has.
  __device__ __forceinline__ void last_few(int b, uint64_t rest, bool weights, Best& best,
                                           float& sum) const {
    float x;
    int v;
    const int n = in_order(&x, &v);
    const float t16 = t16_of(x);
    uint64_t all;
    const uint64_t u = tid < n ? (weights ? fine_of(t16) : 1) : 0;
    if (sum_before(u, &all) < rest && tid < n) {
      const float w = ex2_approx(t16 * (-1.f / kPerUnit));
      take(best, Best{__fdividef(w, __ldg(a.expo + int64_t(b) * a.V + (v - first))), v,
                      t16 * (1.f / kPerUnit)});
      sum += w;
    }
    reduce(best, sum);
  }

  // The row from its few logits (one CTA): both cuts and the draw. total: the row's
  // sum of weights, where top-k does not cut.
  __device__ void finish(int b, bool cut_k, int k, float p, float t_max, uint64_t total) const {
    float x;
    int v;
    const int n = in_order(&x, &v);
    bool in = tid < n && (!cut_k || tid < k);
    const float ev = in ? __ldg(a.expo + int64_t(b) * a.V + (v - first)) : 1.f;
    const float t = in ? t16_of(x) * (1.f / kPerUnit) : kInf;
    const float w = ex2_approx(-t);
    if (!(p >= 1.f)) {
      uint64_t all;
      const uint64_t before = sum_before(__float2ull_rn(w * kWeightOne), &all);
      in = in && before < times_up(cut_k ? all : total, p > 0.f ? p : 0.f);
    }
    in = in && (t <= t_max || tid == 0);
    Best best{-1.f, kNoIdx, 0.f};
    if (in) take(best, Best{__fdividef(w, ev), v, t});
    float sum = in ? w : 0.f;
    reduce(best, sum);
    if (tid == 0) answer(b, best, sum, false, false);
  }
};

template <typename T, bool kHeld>
__global__ void __launch_bounds__(kThreads, kCtas) sample_kernel(const SampleArgs a) {
  using E = Elem<T>;
  extern __shared__ __align__(16) unsigned char smem_raw[];
  __shared__ Shared sh;
  Row<T, kHeld> r(a, sh);
  r.rank = static_cast<int>(r.cluster.block_rank());
  r.size = static_cast<int>(r.cluster.num_blocks());
  r.tid = threadIdx.x;
  r.warp = r.tid >> 5;
  r.lane = r.tid & 31;
  const int b = blockIdx.x / r.size;
  if (r.tid == 0) sh.pushed = sh.mine = 0;
  r.cluster.barrier_arrive();  // waited for before any CTA's memory is written by another
  pdl_wait();
  pdl_trigger();
  const T* x0 = static_cast<const T*>(a.logits) + int64_t(b) * a.stride;
  r.first = static_cast<int>((reinterpret_cast<uintptr_t>(x0) & 15) / sizeof(T));
  r.end = r.first + a.V;
  r.base = x0 - r.first;
  const int groups = (r.end + E::N - 1) / E::N;
  const int per = (groups + r.size - 1) / r.size;
  r.g0 = r.rank * per;
  r.ng = max(0, min(groups - r.g0, per));
  r.held = reinterpret_cast<uint4*>(smem_raw);
  const float temp = a.temperature != nullptr ? a.temperature[b] : 1.f;
  const int k = a.top_k != nullptr ? a.top_k[b] : 0;
  const float p = a.top_p != nullptr ? a.top_p[b] : 1.f;
  const float mp = a.min_p != nullptr ? a.min_p[b] : 0.f;
  const bool greedy = !(temp > 0.f);
  // 1 / T overflows for small T: any finite number in its place leaves the
  // maximum its weight 1 and takes all others' away
  r.c16 = greedy ? 0.f : fminf(kPerUnit * kLog2e / temp, FLT_MAX);

  // the row's maximum; a NaN or +inf in it, or nothing finite, refuses it
  auto max2 = [](float x, float y) { return max3_nan(x, y, y); };
  float m = r.read();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = max2(m, __shfl_xor_sync(kAll, m, o));
  if (r.lane == 0) sh.wf[r.warp] = m;
  __syncthreads();
  m = sh.wf[r.lane & (kWarps - 1)];
#pragma unroll
  for (int o = kWarps / 2; o > 0; o >>= 1) m = max2(m, __shfl_xor_sync(kAll, m, o));
  r.cluster.barrier_wait();
  if (r.size > 1) {
    if (r.tid < r.size) *r.cluster.map_shared_rank(&sh.cmax[r.rank], r.tid) = m;
    r.cluster.sync();
    m = kNegInf;
    for (int q = 0; q < r.size; ++q) m = max2(m, sh.cmax[q]);
  }
  const bool bad = !(m <= FLT_MAX) || m == kNegInf;
  r.max = m;

  Best best{-1.f, kNoIdx, 0.f};
  float sum = 0.f;
  Cut cut;
  // w >= min_p as t <= -log2(min_p); the maximum always stays
  const float t_max = mp > 0.f ? fmaxf(0.f, -log2f(mp)) : kInf;
  const bool cut_k = k > 0 && k < a.V, cut_p = !(p >= 1.f);
  if (!bad && greedy) {
    r.each_from(m, [&](float x, int v) {
      if (x == m) take(best, Best{1.f, v, 0.f});
    });
  } else if (!bad) {
    uint32_t left = kAll;  // no more logits than these are kept
    const float share = p > 0.f ? p : 0.f;
    if (cut_k || cut_p) {
      int lo, hi, enough;
      uint64_t total, rest;
      // by values where they are few, else, or below them, by steps of t
      bool is = false, steps = true;
      if constexpr (sizeof(T) == 2) {
        const Kept all;
        if (cut_k)
          is = r.template by_value<false, false>(k, 0.f, all, !cut_p, &cut, &total);
        else if (r.values_suffice())
          is = r.template by_value<true, false>(0, share, all, true, &cut, &total);
        steps = !is;
        if (is && sh.found_count <= kFew) {
          r.push(cut.kept.x, [&](float x, int) { return x >= cut.kept.x; });
          if (r.rank == 0) r.finish(b, cut_k, k, p, t_max, total);
          return;
        }
        if (is) left = sh.found_count;
      }
      if (steps) {
        cut = Cut{};
        if (cut_k)
          is = r.template steps<false, false>(k, 0.f, cut.kept, &lo, &hi, &total, &rest, &enough);
        else
          is = r.template steps<true, false>(0, share, cut.kept, &lo, &hi, &total, &rest, &enough);
        if (is && sh.found_count <= kFew) {
          r.push(r.reach(enough),
                 [&](float x, int) { return x > kNegInf && r.bucket_of(x) <= enough; });
          if (r.rank == 0) r.finish(b, cut_k, k, p, t_max, total);
          return;
        }
        if (is) {
          left = sh.found_count;
          if (cut_k)
            cut = r.template narrow<false, false>(lo, hi, sh.found_num, rest, cut.kept, !cut_p);
          else
            cut = r.template narrow<true, false>(lo, hi, kAll, rest, cut.kept, true);
        }
      }
      if (cut_k && cut_p) {
        const Kept first = cut.kept;
        bool found = false;
        if constexpr (sizeof(T) == 2)
          found = r.values_suffice() &&
                  r.template by_value<true, true>(0, share, first, true, &cut, &total);
        if (found) {
          left = min(left, sh.found_count);
        } else if (r.template steps<true, true>(0, share, first, &lo, &hi, &total, &rest,
                                                &enough)) {
          left = min(left, sh.found_count);
          cut = r.template narrow<true, true>(lo, hi, kAll, rest, first, true);
        }
      }
    }
    const float* e = a.expo + int64_t(b) * a.V - r.first;
    auto draw = [&](float t, int v, float ev) {
      const float q = ex2_approx(-t);
      sum += q;
      // a thread's indices ascend: the first of equal scores stays
      const float score = __fdividef(q, ev);
      if (score > best.score) best = Best{score, v, t};
    };
    // whether a logit is in; what the row's last step looks at goes to the first CTA
    auto taken = [&](float y, float t16, int v) {
      if (!cut.kept.has(y, v)) return false;
      if (t16 < cut.from || y > cut.x) return true;
      if (t16 < cut.to) r.push_one(y, v);  // (t = inf has no weight)
      return false;
    };
    // a bound for what is looked at, a little low; t decides
    const float least = fmaxf(fmaxf(cut.kept.x, -FLT_MAX), m - (t_max * kPerUnit + 1.f) / r.c16);
    constexpr int U = 4;
    if (left > static_cast<uint32_t>(a.V) / 8 && t_max == kInf) {
      // Many are left: group by group, the random numbers in 16 bytes where they lie
      // so. From `sure` on a logit is in; what little lies between is looked at.
      const float sure =
          cut.rest > 0 ? (cut.x < kInf ? E::value(E::key(cut.x) + 1) : r.least_below(cut.from))
          : cut.kept.limit == kNoIdx ? least
                                     : fmaxf(least, E::value(E::key(cut.kept.x) + 1));
      // A known cut's equal logits are all in before its limit, and none behind it: only
      // one group has to look at them.
      const bool known = cut.rest == 0;
      const int all_before = known ? cut.kept.limit : 0;
      const int none_from = known ? cut.kept.limit : kNoIdx;
      const float c = r.c16 * (1.f / kPerUnit);
      const bool wide = reinterpret_cast<uintptr_t>(e) % 16 == 0;
      constexpr int kPair = 8 / E::N;
      for (int g = r.tid; g < r.ng; g += U * kThreads) {
        uint4 w[U];
        r.template fetch<U, kHeld>(w, g);
#pragma unroll
        for (int j0 = 0; j0 < U; j0 += kPair) {
          if (g + j0 * kThreads >= r.ng) break;
          // the random numbers of a few groups are on their way together
          float ev[kPair][E::N];
#pragma unroll
          for (int j = 0; j < kPair; ++j) {
            const int v = (r.g0 + g + (j0 + j) * kThreads) * E::N;
            if (wide && v >= r.first && v + E::N <= r.end) {
#pragma unroll
              for (int i = 0; i < E::N; i += 4) {
                const float4 q = __ldg(reinterpret_cast<const float4*>(e + v + i));
                ev[j][i] = q.x; ev[j][i + 1] = q.y; ev[j][i + 2] = q.z; ev[j][i + 3] = q.w;
              }
            } else {
              float y[E::N];
              E::unpack(w[j0 + j], y);
#pragma unroll
              for (int i = 0; i < E::N; ++i) {
                ev[j][i] = 1.f;
                if (y[i] >= least) ev[j][i] = __ldg(e + v + i);
              }
            }
          }
#pragma unroll
          for (int j = 0; j < kPair; ++j) {
            const int v = (r.g0 + g + (j0 + j) * kThreads) * E::N;
            float y[E::N];
            E::unpack(w[j0 + j], y);
            float in_from = sure, look_from = least;
            if constexpr (sizeof(T) == 2) {
              if (v + E::N <= all_before) in_from = least;
              if (v >= none_from) look_from = sure;
            }
            bool look = false;
#pragma unroll
            for (int i = 0; i < E::N; ++i) {
              const float q = ex2_approx((y[i] - m) * c);
              const bool is = y[i] >= in_from;
              sum += is ? q : 0.f;
              const float score = __fdividef(q, ev[j][i]);
              if (is && score > best.score) {
                best.score = score;
                best.idx = v + i;
              }
              look |= !is && y[i] >= look_from;
            }
            if (look) {
#pragma unroll
              for (int i = 0; i < E::N; ++i) {
                const float t16 = r.t16_of(y[i]);
                if (y[i] >= look_from && y[i] < in_from && taken(y[i], t16, v + i)) {
                  const float q = ex2_approx(t16 * (-1.f / kPerUnit));
                  sum += q;
                  take(best, Best{__fdividef(q, ev[j][i]), v + i, 0.f});
                }
              }
            }
          }
        }
      }
      if (best.idx != kNoIdx)
        best.t = r.t16_of(to_f32(r.base[best.idx])) * (1.f / kPerUnit);
    } else {
      // Few are left: a bit for each of a thread's next logits that is, then those,
      // four at a time.
      for (int g = r.tid; g < r.ng; g += U * kThreads) {
        uint4 w[U];
        r.template fetch<U, kHeld>(w, g);
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < U; ++j) {
          float y[E::N];
          E::unpack(w[j], y);
#pragma unroll
          for (int i = 0; i < E::N; ++i) bits |= (y[i] >= least ? 1u : 0u) << (j * E::N + i);
        }
        while (bits != 0) {
          constexpr int W = 4;
          float t[W], ev[W];
          int at[W];
#pragma unroll
          for (int u = 0; u < W; ++u) {
            t[u] = -1.f;
            ev[u] = 1.f;
            at[u] = 0;
            if (bits == 0) continue;
            const int bit = __ffs(bits) - 1, gk = g + bit / E::N * kThreads;
            bits &= bits - 1;
            at[u] = (r.g0 + gk) * E::N + bit % E::N;
            const float y = to_f32(kHeld ? reinterpret_cast<const T*>(r.held + gk)[bit % E::N]
                                         : r.base[at[u]]);
            const float t16 = r.t16_of(y);
            if (t16 * (1.f / kPerUnit) <= t_max && taken(y, t16, at[u])) {
              t[u] = t16 * (1.f / kPerUnit);
              ev[u] = __ldg(e + at[u]);
            }
          }
#pragma unroll
          for (int u = 0; u < W; ++u)
            if (t[u] >= 0.f) draw(t[u], at[u], ev[u]);
        }
      }
    }
  }
  // the cluster's best and sum, joined in a fixed order
  if (cut.rest > 0) r.send();
  r.reduce(best, sum);
  if (r.tid == 0) {
    *r.cluster.map_shared_rank(&sh.cbest[r.rank], 0) = best;
    *r.cluster.map_shared_rank(&sh.csum[r.rank], 0) = sum;
  }
  r.cluster.sync();
  if (r.rank != 0) return;
  best = Best{-1.f, kNoIdx, 0.f};
  sum = 0.f;
  if (r.tid == 0) {
    for (int q = 0; q < r.size; ++q) {
      take(best, sh.cbest[q]);
      sum += sh.csum[q];
    }
  }
  if (cut.rest > 0) r.last_few(b, cut.rest, cut.weights, best, sum);
  if (r.tid == 0) r.answer(b, best, sum, bad, greedy);
}

// Of a row's share, beside the SM's other CTA's, and both histograms.
constexpr size_t kMostHeld = (227 * 1024 / kCtas - sizeof(Shared) - 1024) / 16 * 16;

template <typename T, bool kHeld>
cudaError_t launch_k(const SampleArgs& a, int cluster, size_t smem, cudaStream_t s) {
  if (kHeld) {  // the most that any row needs: calls of two threads set the same
    const cudaError_t e =
        cudaFuncSetAttribute(sample_kernel<T, kHeld>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             static_cast<int>(kMostHeld));
    if (e != cudaSuccess) return e;
  }
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<T, kHeld>, a);
}

template <typename T>
cudaError_t launch_t(const SampleArgs& a, cudaStream_t s) {
  constexpr int kResident = kCtas * 152;
  constexpr int64_t kL2 = 100 << 20;
  // As many CTAs a row as leave all rows' CTAs resident, with a few logits a thread.
  int cluster = 1;
  while (cluster < kMaxCluster && int64_t(a.B) * cluster * 2 <= kResident &&
         a.V > cluster * kThreads * 4)
    cluster *= 2;
  const int groups = (a.V + 2 * Elem<T>::N - 2) / Elem<T>::N;  // with any lead
  static_assert((kMaxSampleVocab / 4 + 2) / kMaxCluster + 1 <= kMaxBlocks * kThreads &&
                    kL2 / kResident / 16 + 1 <= kMaxBlocks * kThreads,
                "a share has no more blocks");
  auto share = [&] { return size_t((groups + cluster - 1) / cluster) * 16; };
  // rows that are read again, and resident at one time, fit L2; a thread has no more
  // than 200 logits as far as eight CTAs go, V = 819200 (200 / 512 rows of 131072 in bf16
  // with one CTA a row and with two: top-k 61 / 125 and 46 / 93 us, top-p 122 / 226 and
  // 90 / 194, no limit 50 / 108 and 50 / 108; rows of 70000 want one where there are no
  // cuts: 64 and 75)
  while (cluster < kMaxCluster && share() > kMostHeld &&
         (kResident * int64_t(share()) > kL2 || a.V > cluster * kThreads * 200))
    cluster *= 2;
  if (share() <= kMostHeld) return launch_k<T, true>(a, cluster, share(), s);
  return launch_k<T, false>(a, cluster, 0, s);
}

}  // namespace

cudaError_t launch_sample_rows(const SampleArgs& a, rf_dtype dt, cudaStream_t s) {
  return dt == RF_F32 ? launch_t<float>(a, s) : launch_t<__nv_bfloat16>(a, s);
}

}  // namespace rf
