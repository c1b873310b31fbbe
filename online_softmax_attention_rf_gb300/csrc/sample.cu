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
// and neither needs the row sorted. A histogram of t in steps of 1/16, of counts
// for top-k and of weights for top-p, gives the interval that the cut falls into.
// Where no more than 512 logits lie above the interval's lower end, as is usual,
// these alone go on: one CTA puts them in order and finishes the row. Otherwise
// histograms of the logits' bits inside the interval narrow it down to one value,
// and a count of that value's occurrences settles which of them are in.
// Counts and weights are added as integers (a weight to 22 bits below the power
// of two of its interval, about what float32 carries), so that the order of the
// additions cannot move a cut.
//
// A cluster of CTAs holds a row in shared memory, read once from global memory;
// each pass goes over it there. Histograms are joined through distributed shared
// memory: each CTA adds up its share of the buckets and hands the sums to all.
#include <cooperative_groups.h>

#include <cfloat>

#include "paged_device.cuh"

namespace cg = cooperative_groups;

namespace rf {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBuckets = 1024;
constexpr int kPerUnit = 16;   // buckets of the first histogram per unit of t
constexpr int kFracBits = 42;  // of the row's sum of weights: up to 2^20 of them, of at most 1
constexpr int kFineBits = 22;  // of a weight, below the power of two of its interval
constexpr int kHalf = 11;      // of them in the lower half: 2^20 weights fit 32 bits
constexpr int kFew = kThreads; // logits that one CTA finishes, one a thread
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kInf = __builtin_huge_valf();
static_assert(kBuckets == 2 * kThreads, "the scan takes two buckets a thread");
static_assert(kFew <= kBuckets, "a histogram's place holds the few logits");

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
  // this CTA's histogram: counts, and weights in two halves. In the cluster's
  // first CTA the few logits and their indices take the place of the first two,
  // sorted ones that of the cluster's sums.
  alignas(16) uint32_t cnt[kBuckets];
  uint32_t hi[kBuckets], lo[kBuckets];
  // the cluster's
  uint64_t val[kBuckets];
  uint32_t num[kBuckets];
  uint64_t wsum[kWarps];
  uint32_t wcnt[kWarps];
  // a value of each CTA of the cluster
  float cmax[kMaxCluster];
  uint32_t cties[kMaxCluster];
  float csum[kMaxCluster];
  Best cbest[kMaxCluster];
  // of each warp
  float wf[kWarps];
  Best wbest[kWarps];
  uint64_t found_rest;
  uint64_t total;
  int found;
  uint32_t found_count;  // logits in the buckets up to the found one
  int tie_limit;
  uint32_t pushed;       // few logits that arrived
};

// Where a selection ends: every logit above x is in, and of those equal to x
// the first `ties` (kAll: all).
struct Cut {
  float x;
  uint32_t ties;
};

// What a selection left of this CTA's logits. -inf has no probability.
struct Kept {
  float x = kNegInf;
  int limit = 0;  // of those equal to x, the ones before this index
  __device__ __forceinline__ bool has(float y, int v) const { return y > x || (y == x && v < limit); }
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

  __device__ __forceinline__ Row(const SampleArgs& a_, Shared& s)
      : a(a_), sh(s), cluster(cg::this_cluster()) {}

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

  // Reads the row; this thread's maximum (NaN if one is).
  __device__ float read() const {
    float m = kNegInf;
    // groups that lie wholly in the row; the first and the last one may not
    const int f0 = g0 == 0 && first > 0 ? 1 : 0;
    const int f1 = min(ng, end / E::N - g0);
    const uint4* from = reinterpret_cast<const uint4*>(base) + g0;
    constexpr int U = 4;
    int g = f0 + tid;
    for (; g + (U - 1) * kThreads < f1; g += U * kThreads) {
      uint4 w[U];
#pragma unroll
      for (int j = 0; j < U; ++j) w[j] = __ldg(from + g + j * kThreads);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        if (kHeld) held[g + j * kThreads] = w[j];
        m = E::max_of(w[j], m);
      }
    }
    for (; g < f1; g += kThreads) {
      const uint4 w = __ldg(from + g);
      if (kHeld) held[g] = w;
      m = E::max_of(w, m);
    }
    // ragged ends: group 0, and those from max(f0, f1) on (one at most)
    const int e = tid == 0 ? (f0 > 0 && ng > 0 ? 0 : -1) : tid == 1 ? f1 : -1;
    if (e >= 0 && e < ng && (tid == 0 || e >= f0)) {
      const uint4 w = load_group(g0 + e);
      if (kHeld) held[e] = w;
      m = E::max_of(w, m);
    }
    return m;
  }

  // f(group, index of its first logit from base), over this thread's groups with
  // a logit of at least `least`, in ascending order.
  template <typename F>
  __device__ __forceinline__ void groups_from(float least, F&& f) const {
#pragma unroll 2
    for (int g = tid; g < ng; g += kThreads) {
      const uint4 w = kHeld ? held[g] : load_group(g0 + g);
      if (E::max_of(w, kNegInf) >= least) f(w, (g0 + g) * E::N);
    }
  }
  template <typename F>
  __device__ __forceinline__ void each_from(float least, F&& f) const {
    groups_from(least, [&](const uint4& w, int v) {
      float y[E::N];
      E::unpack(w, y);
#pragma unroll
      for (int i = 0; i < E::N; ++i) f(y[i], v + i);
    });
  }

  // kPerUnit * t: not below 0; +inf for -inf
  __device__ __forceinline__ float t16_of(float x) const { return __fmul_rn(max - x, c16); }
  __device__ __forceinline__ int bucket_of(float x) const {
    const float t = fminf(t16_of(x), kBuckets - 1.f);
    return __float_as_int(__fadd_rz(t, 8388608.f)) & (kBuckets - 1);
  }
  // A weight over 2^-e, e the power of its interval, as an integer.
  static __device__ __forceinline__ uint32_t fine_of(float t16) {
    const float e16 = __fadd_rz(t16, 134217728.f) - 134217728.f;  // to a multiple of 16
    const float f = ex2_approx((e16 - t16) * (1.f / kPerUnit));   // in (0.5, 1]
    return __float_as_uint(f + 2.f) - 0x40000000u;                // f * 2^22
  }
  __device__ __forceinline__ void add_fine(int b, uint32_t f) const {
    atomicAdd(&sh.hi[b], f >> kHalf);
    atomicAdd(&sh.lo[b], f & ((1u << kHalf) - 1));
  }

  __device__ __forceinline__ void clear() const {
    uint4* h = reinterpret_cast<uint4*>(sh.cnt);  // cnt, hi, lo
    for (int i = tid; i < 3 * kBuckets / 4; i += kThreads) h[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
  }

  // Joins the CTAs' histograms: val (counts, or weights; weights of the first
  // histogram in units of 2^-kFracBits) and num (counts), the same in each CTA.
  template <bool kWeights>
  __device__ void join(bool by_unit) const {
    cluster.sync();
    const int share = kBuckets / size;
    for (int i = tid; i < share; i += kThreads) {
      const int b = rank * share + i;
      uint32_t n = 0, hi = 0;
      uint64_t lo = 0;
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        if (q >= size) break;
        n += *cluster.map_shared_rank(&sh.cnt[b], q);
        if (kWeights) {
          hi += *cluster.map_shared_rank(&sh.hi[b], q);
          lo += *cluster.map_shared_rank(&sh.lo[b], q);
        }
      }
      uint64_t v = n;
      if (kWeights) {
        v = (uint64_t(hi) << kHalf) + lo;
        if (by_unit) {
          const int s = kFracBits - kFineBits - b / kPerUnit;
          v = s >= 0 ? v << s : v >> -s;
        }
      }
      for (int q = 0; q < size; ++q) {
        *cluster.map_shared_rank(&sh.val[b], q) = v;
        *cluster.map_shared_rank(&sh.num[b], q) = n;
      }
    }
    cluster.sync();
  }

  // The bucket in which the running sum of val reaches the target (share < 0:
  // `target`, else that share of the whole), what the target is behind the sum
  // before it, and the logits up to it; none: -1. Each warp adds up its 64
  // buckets; the one that the target falls into looks closer.
  __device__ int find(uint64_t target, float share, uint64_t* rest) const {
    const uint64_t v0 = sh.val[2 * tid], v1 = sh.val[2 * tid + 1];
    const uint32_t n0 = sh.num[2 * tid], n1 = sh.num[2 * tid + 1];
    uint64_t s = v0 + v1;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    const uint32_t n = __reduce_add_sync(kAll, n0 + n1);
    if (lane == 0) {
      sh.wsum[warp] = s;
      sh.wcnt[warp] = n;
    }
    if (tid == 0) sh.found = -1;
    __syncthreads();
    s = scan(lane < kWarps ? sh.wsum[lane] : 0);
    const uint64_t total = __shfl_sync(kAll, s, 31);
    if (share >= 0.f) target = times_up(total, share);
    if (warp == __popc(__ballot_sync(kAll, s < target))) {
      uint64_t before = __shfl_sync(kAll, s, warp > 0 ? warp - 1 : 0);
      if (warp == 0) before = 0;
      const uint32_t count = __reduce_add_sync(kAll, lane < warp ? sh.wcnt[lane] : 0u) +
                             scan(n0 + n1);
      before += scan(v0 + v1) - v0 - v1;
      int b = -1;
      if (before < target && target <= before + v0)
        b = 2 * tid;
      else if (before + v0 < target && target <= before + v0 + v1)
        b = 2 * tid + 1;
      if (b >= 0) {
        sh.found = b;
        sh.found_rest = target - before - (b & 1 ? v0 : 0);
        sh.found_count = b & 1 ? count : count - n1;
        sh.total = total;
      }
    }
    __syncthreads();
    *rest = sh.found_rest;
    return sh.found;
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

  // The first histogram of what `in` keeps (everything without kPart), and the
  // bucket that the cut falls into, as find().
  template <bool kWeights, bool kPart>
  __device__ int first_histogram(uint64_t target, float share, const Kept& in, uint64_t* rest) const {
    clear();
    each_from(kPart ? in.x : kNegInf, [&](float x, int v) {
      if (kPart && !in.has(x, v)) return;
      const float t = t16_of(x);
      if (kWeights) {
        if (t < kBuckets - 1.f) {  // the weights behind, below 2^-63, count for nothing
          const int b = __float_as_int(__fadd_rz(t, 8388608.f)) & (kBuckets - 1);
          atomicAdd(&sh.cnt[b], 1u);
          add_fine(b, fine_of(t));
        }
      } else if (x > kNegInf) {
        const int b = __float_as_int(__fadd_rz(fminf(t, kBuckets - 1.f), 8388608.f)) & (kBuckets - 1);
        atomicAdd(&sh.cnt[b], 1u);
      }
    });
    join<kWeights>(true);
    return find(target, share, rest);
  }

  // The place where the running sum over (x descending, index ascending) of
  // counts, or of weights, goes on from bucket b of the first histogram by
  // `rest`.
  template <bool kWeights>
  __device__ Cut narrow(int b, uint64_t rest, const Kept& in) const {
    if (kWeights) {  // in units of the interval's weights
      const int s = kFracBits - kFineBits - b / kPerUnit;
      rest = s >= 0 ? (rest + (uint64_t(1) << s) - 1) >> s : rest << -s;
    }
    // The interval's keys lie in [klo, khi] (max - x is between b and b + 1 over
    // c16, up to rounding: 2^-21 of it is more than that); from `inside` on they
    // are in it or above it.
    const float d_hi = (b + 1) / c16;
    uint32_t khi = b > 0 ? E::key(max - b / c16 * (1.f - 0x1p-21f)) : E::key(max);
    uint32_t klo = E::kLowest;
    float inside = kNegInf;
    if (b < kBuckets - 1) {
      klo = umax(klo, E::key(max - d_hi * (1.f + 0x1p-21f)));
      inside = max - d_hi * (1.f - 0x1p-21f);
    }
    while (true) {
      const uint32_t span = khi - klo;
      if (span == 0) break;
      int s = 0;
      while ((span >> s) >= kBuckets) ++s;
      clear();
      const float xlo = E::value(klo), xhi = E::value(khi);
      each_from(xlo, [&](float x, int v) {
        if (!(x >= xlo && x <= xhi) || bucket_of(x) != b || !in.has(x, v)) return;
        const int i = static_cast<int>((khi - E::key(x)) >> s);
        atomicAdd(&sh.cnt[i], 1u);
        if (kWeights) add_fine(i, fine_of(t16_of(x)));
      });
      join<kWeights>(false);
      const int i = find(rest, -1.f, &rest);  // the interval's sum is at least the rest
      const uint32_t n = sh.num[i];
      khi -= static_cast<uint32_t>(i) << s;
      klo = s > 0 ? umax(klo, khi - ((1u << s) - 1)) : khi;
      // a single logit is in, whichever it is, and nothing below it
      if (n == 1 && E::value(klo) > inside) return Cut{E::value(klo), kAll};
    }
    const float x = E::value(klo);
    if (kWeights) {
      const uint64_t f = fine_of(t16_of(x));
      rest = (rest + f - 1) / f;
    }
    return Cut{x, static_cast<uint32_t>(rest < kAll ? rest : kAll)};
  }
  static __device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }

  // What the cut leaves of `in`.
  __device__ Kept settle(const Cut& cut, const Kept& in) const {
    if (cut.x < in.x) return in;  // the lower end of an interval with one logit in it
    const int last = cut.x == in.x ? in.limit : kNoIdx;
    return Kept{cut.x, cut.ties == kAll ? last : min(last, tie_limit(cut))};
  }

  // Of the elements equal to the cut, the first cut.ties are those before the
  // returned index.
  __device__ int tie_limit(const Cut& cut) const {
    uint32_t n = 0;
    each_from(cut.x, [&](float x, int) { n += x == cut.x; });
    n = __reduce_add_sync(kAll, n);
    __syncthreads();
    if (lane == 0) sh.wcnt[warp] = n;
    if (tid == 0) sh.tie_limit = kNoIdx;
    __syncthreads();
    n = 0;
    for (int w = 0; w < kWarps; ++w) n += sh.wcnt[w];
    if (tid < size) *cluster.map_shared_rank(&sh.cties[rank], tid) = n;
    cluster.sync();
    uint32_t before = 0;
    for (int q = 0; q < rank; ++q) before += sh.cties[q];
    if (cut.ties <= before) return 0;
    uint32_t left = cut.ties - before;
    if (left >= n) return kNoIdx;
    // the left'th of this CTA's, in order
    for (int g = 0; g < ng; g += kThreads) {
      uint32_t mine = 0;
      float y[E::N];
      if (g + tid < ng) {
        E::unpack(kHeld ? held[g + tid] : load_group(g0 + g + tid), y);
#pragma unroll
        for (int i = 0; i < E::N; ++i) mine += y[i] == cut.x;
      }
      uint32_t s = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t u = __shfl_up_sync(kAll, s, o);
        if (lane >= o) s += u;
      }
      __syncthreads();
      if (lane == 31) sh.wcnt[warp] = s;
      __syncthreads();
      uint32_t total = 0, ahead = s - mine;
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) ahead += sh.wcnt[w];
        total += sh.wcnt[w];
      }
      if (ahead < left && left <= ahead + mine) {
#pragma unroll
        for (int i = 0; i < E::N; ++i)
          if (y[i] == cut.x && ++ahead == left) sh.tie_limit = (g0 + g + tid) * E::N + i + 1;
      }
      if (left <= total) break;
      left -= total;
    }
    __syncthreads();
    return sh.tie_limit;
  }

  // The best and the sum of the CTA's threads, in a fixed order, in thread 0.
  __device__ __forceinline__ void reduce(Best& best, float& sum) const {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Best other{__shfl_xor_sync(kAll, best.score, o), __shfl_xor_sync(kAll, best.idx, o),
                       __shfl_xor_sync(kAll, best.t, o)};
      take(best, other);
      sum += __shfl_xor_sync(kAll, sum, o);
    }
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
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        const Best other{__shfl_xor_sync(kAll, best.score, o), __shfl_xor_sync(kAll, best.idx, o),
                         __shfl_xor_sync(kAll, best.t, o)};
        take(best, other);
        sum += __shfl_xor_sync(kAll, sum, o);
      }
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

  // The few logits from bucket b up go to the cluster's first CTA.
  __device__ __forceinline__ void push(int b) const {
    // a bound for the prefilter, a little low; bucket_of decides
    const float least = fmaxf(kNegInf, max - (b + 2) / c16);
    each_from(least, [&](float x, int v) {
      if (!(x > kNegInf) || bucket_of(x) > b) return;
      const uint32_t at = atomicAdd(cluster.map_shared_rank(&sh.pushed, 0), 1u);
      if (at < kFew) {
        *cluster.map_shared_rank(&sh.cnt[at], 0) = __float_as_uint(x);
        *cluster.map_shared_rank(&sh.hi[at], 0) = static_cast<uint32_t>(v);
      }
    });
  }

  // The row from its few logits (one CTA): in order, then both cuts and the draw.
  // total: the row's sum of weights, where top-k does not cut.
  __device__ void finish(int b, int k, float p, float t_max, uint64_t total) const {
    const int n = min(static_cast<int>(sh.pushed), kFew);
    float* sx = reinterpret_cast<float*>(sh.val);  // sorted
    int* sv = reinterpret_cast<int*>(sh.val) + kFew;
    if (tid < n) {
      const float x = __uint_as_float(sh.cnt[tid]);
      const int v = static_cast<int>(sh.hi[tid]);
      int r = 0;
#pragma unroll 8
      for (int j = 0; j < n; ++j) {
        const float y = __uint_as_float(sh.cnt[j]);
        r += y > x || (y == x && static_cast<int>(sh.hi[j]) < v);
      }
      sx[r] = x;
      sv[r] = v;
    }
    __syncthreads();
    const bool cut_k = k > 0 && k < a.V;
    bool in = tid < n && (!cut_k || tid < k);
    const int v = in ? sv[tid] : 0;
    const float ev = in ? a.expo[int64_t(b) * a.V + (v - first)] : 1.f;
    const float t = in ? t16_of(sx[tid]) * (1.f / kPerUnit) : kInf;
    const float w = ex2_approx(-t);
    if (!(p >= 1.f)) {
      // weights in units of 2^-kFracBits
      const uint64_t u = __float2ull_rn(w * 4398046511104.f);
      uint64_t s = u;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t q = __shfl_up_sync(kAll, s, o);
        if (lane >= o) s += q;
      }
      if (lane == 31) sh.wsum[warp] = s;
      __syncthreads();
      uint64_t before = s - u, all = 0;
      for (int q = 0; q < kWarps; ++q) {
        if (q < warp) before += sh.wsum[q];
        all += sh.wsum[q];
      }
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
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const SampleArgs a) {
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
  if (r.tid == 0) sh.pushed = 0;
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
  float m = r.read();
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float q = __shfl_xor_sync(kAll, m, o);
    m = max3_nan(m, q, q);
  }
  if (r.lane == 0) sh.wf[r.warp] = m;
  __syncthreads();
  m = sh.wf[0];
#pragma unroll
  for (int w = 1; w < kWarps; w += 3)
    m = max3_nan(m, max3_nan(sh.wf[w], sh.wf[min(w + 1, kWarps - 1)], sh.wf[min(w + 2, kWarps - 1)]),
                 kNegInf);
  r.cluster.barrier_wait();
  if (r.tid < r.size) *r.cluster.map_shared_rank(&sh.cmax[r.rank], r.tid) = m;
  r.cluster.sync();
  m = kNegInf;
  for (int q = 0; q < r.size; ++q) m = max3_nan(m, sh.cmax[q], kNegInf);
  const bool bad = !(m <= FLT_MAX) || m == kNegInf;
  r.max = m;

  Best best{-1.f, kNoIdx, 0.f};
  float sum = 0.f;
  if (!bad && greedy) {
    r.each_from(m, [&](float x, int v) {
      if (x == m) take(best, Best{1.f, v, 0.f});
    });
  } else if (!bad) {
    // w >= min_p as t <= -log2(min_p); the maximum always stays
    const float t_max = mp > 0.f ? fmaxf(0.f, -log2f(mp)) : kInf;
    Kept kept;
    const bool cut_k = k > 0 && k < a.V, cut_p = !(p >= 1.f);
    const float share = p > 0.f ? p : 0.f;
    if (cut_k || cut_p) {
      uint64_t rest;
      const int at = cut_k ? r.template first_histogram<false, false>(k, -1.f, kept, &rest)
                           : r.template first_histogram<true, false>(0, share, kept, &rest);
      if (at >= 0 && sh.found_count <= kFew) {
        r.push(at);
        r.cluster.sync();
        if (r.rank == 0) r.finish(b, k, p, t_max, sh.total);
        return;
      }
      if (at >= 0)
        kept = r.settle(cut_k ? r.template narrow<false>(at, rest, kept)
                              : r.template narrow<true>(at, rest, kept), kept);
      if (cut_k && cut_p) {
        const int at_p = r.template first_histogram<true, true>(0, share, kept, &rest);
        if (at_p >= 0) kept = r.settle(r.template narrow<true>(at_p, rest, kept), kept);
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
    if (kept.x == kNegInf && t_max == kInf) {
      // nothing is cut off: group by group
      r.groups_from(kNegInf, [&](const uint4& w, int v) {
        float y[E::N], ev[E::N];
        E::unpack(w, y);
#pragma unroll
        for (int i = 0; i < E::N; ++i) ev[i] = y[i] > kNegInf ? __ldg(e + v + i) : 1.f;
#pragma unroll
        for (int i = 0; i < E::N; ++i)
          if (y[i] > kNegInf) draw(r.t16_of(y[i]) * (1.f / kPerUnit), v + i, ev[i]);
      });
    } else {
      // Mostly few are left: a bit for each of a thread's next 32 logits that is,
      // then those, four at a time. The bound is a little low; t decides.
      const float least = fmaxf(fmaxf(kept.x, -FLT_MAX), m - (t_max * kPerUnit + 1.f) / r.c16);
      constexpr int kGroups = 32 / E::N;
      for (int g = r.tid; g < r.ng; g += kGroups * kThreads) {
        uint32_t left = 0;
#pragma unroll
        for (int j = 0; j < kGroups; ++j) {
          if (g + j * kThreads >= r.ng) break;
          float y[E::N];
          E::unpack(kHeld ? r.held[g + j * kThreads] : r.load_group(r.g0 + g + j * kThreads), y);
#pragma unroll
          for (int i = 0; i < E::N; ++i) left |= (y[i] >= least ? 1u : 0u) << (j * E::N + i);
        }
        while (left != 0) {
          constexpr int U = 4;
          float t[U], ev[U];
          int at[U];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            t[u] = -1.f;
            ev[u] = 1.f;
            at[u] = 0;
            if (left == 0) continue;
            const int k = __ffs(left) - 1, gk = g + k / E::N * kThreads;
            left &= left - 1;
            at[u] = (r.g0 + gk) * E::N + k % E::N;
            const float y = kHeld ? to_f32(reinterpret_cast<const T*>(r.held + gk)[k % E::N])
                                  : to_f32(r.base[at[u]]);
            const float ty = r.t16_of(y) * (1.f / kPerUnit);
            if (kept.has(y, at[u]) && ty <= t_max) {
              t[u] = ty;
              ev[u] = __ldg(e + at[u]);
            }
          }
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (t[u] >= 0.f) draw(t[u], at[u], ev[u]);
        }
      }
    }
  }
  // the cluster's best and sum, joined in a fixed order
  r.reduce(best, sum);
  if (r.tid == 0) {
    *r.cluster.map_shared_rank(&sh.cbest[r.rank], 0) = best;
    *r.cluster.map_shared_rank(&sh.csum[r.rank], 0) = sum;
  }
  r.cluster.sync();
  if (r.rank == 0 && r.tid == 0) {
    best = sh.cbest[0];
    sum = sh.csum[0];
    for (int q = 1; q < r.size; ++q) {
      take(best, sh.cbest[q]);
      sum += sh.csum[q];
    }
    r.answer(b, best, sum, bad, greedy);
  }
}

template <typename T, bool kHeld>
cudaError_t launch_k(const SampleArgs& a, int cluster, size_t smem, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(sample_kernel<T, kHeld>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
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
  constexpr int kMostHeld = 160 * 1024;
  // a row goes to as many CTAs as it takes to have few of its logits a thread
  int cluster = 1;
  while (cluster < kMaxCluster && a.V > cluster * kThreads * 4) cluster *= 2;
  const int groups = (a.V + 2 * Elem<T>::N - 2) / Elem<T>::N;  // with any lead
  const size_t bytes = size_t((groups + cluster - 1) / cluster) * 16;
  if (bytes <= kMostHeld) return launch_k<T, true>(a, cluster, bytes, s);
  return launch_k<T, false>(a, cluster, 0, s);
}

}  // namespace

cudaError_t launch_sample_rows(const SampleArgs& a, rf_dtype dt, cudaStream_t s) {
  return dt == RF_F32 ? launch_t<float>(a, s) : launch_t<__nv_bfloat16>(a, s);
}

}  // namespace rf
