// draft_verify.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Per sequence, with p_i = softmax(target_i / T), q_i = softmax(draft_i / T)
// (or all of q_i on the drafted token x_i when there are no draft logits):
// drafts are accepted in order while u_i q_i(x_i) < p_i(x_i); the first
// refused position a draws from max(p_a - q_a, 0), and a fully accepted draft
// draws one more token from p. A draw is argmax_j w_j / e_j over given
// exponential variates e_j, which picks j with probability w_j / sum w, needs
// no running sum over the vocabulary, and cannot be tipped by the order of a
// sum: only by two contenders within rounding of each other.
//
// It is the row-softmax cascade (maximum, then sum of exponentials) followed
// by a third reduction that needs both: stats_kernel takes (max, sum) of every
// logit row in one pass, split over CTAs; choose_kernel joins the pieces,
// walks the acceptance chain and takes the third reduction over the one row
// per sequence that needs it, with a cluster of CTAs per sequence (most of
// that row's logits are in L2 by then).
#include <cooperative_groups.h>

#include <cfloat>

#include "paged_device.cuh"

namespace rf {
namespace {

namespace cg = cooperative_groups;

constexpr int kStatThreads = 128;
constexpr int kStatWarps = kStatThreads / 32;
constexpr int kMaxSplits = 32;
constexpr int kCluster = 8;
constexpr int kNone = 0x7fffffff;

// State of one row piece: maximum, sum of exp((x - max) / T), lowest index of
// the maximum (filled in greedy rows only, whose sum is 0, or NaN where the row
// has a NaN). Read as one int4.
struct alignas(16) Stat {
  float m, l;
  int arg, pad;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// exp((x - m) / T) with c = log2(e) / T. The difference is taken before the
// scaling, so that it is exact or nearly so for the entries that matter.
__device__ __forceinline__ float weight(float x, float m, float c) { return ex2_approx((x - m) * c); }

// log2(e) / T. Below a temperature of 4.3e-39 it would be infinite, and the
// largest logit's 0 * inf a NaN; the largest finite number still leaves nothing
// of any logit that is 2^-120 below the largest.
__device__ __forceinline__ float log2e_over(float t, bool* greedy) {
  *greedy = !(t > 0.f);
  return *greedy ? kLog2e : fminf(kLog2e / t, FLT_MAX);
}

__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int n) { return max(0, min(a.S, n)); }

__device__ __forceinline__ void merge(float& m, float& l, float m2, float l2, float c) {
  const float mn = fmaxf(m, m2);
  // an empty side (m = -inf) has l = 0, or NaN where it met one; its weight
  // would be inf - inf
  l = (m == kNegInf ? l : l * weight(m, mn, c)) + (m2 == kNegInf ? l2 : l2 * weight(m2, mn, c));
  m = mn;
}

// Where a row's numbers come from: 16 bytes at a time.
template <typename T>
struct Vec16;
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  static constexpr uint32_t kNone = 0xff800000u;  // -inf
  static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
};
template <>
struct Vec16<__nv_bfloat16> {
  static constexpr int N = 8;
  static constexpr uint32_t kNone = 0xff80ff80u;  // two -inf
  static __device__ __forceinline__ void unpack(const uint4& v, float* x) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};

// A thread's running state over the numbers it reads.
struct Running {
  float m = kNegInf, l = 0.f;
  int arg = kNone;
};

// n numbers x of consecutive indices from v0 on. Probabilities: the maximum of
// the batch first, so that the state is rescaled at most once a batch. Greedy
// rows: the lowest index of the maximum.
template <int n>
__device__ __forceinline__ void take_batch(Running& st, const float* x, float c) {
  float mx = x[0];
#pragma unroll
  for (int i = 1; i < n; ++i) mx = fmaxf(mx, x[i]);
  if (mx > st.m) {
    if (st.m != kNegInf) st.l *= weight(st.m, mx, c);
    st.m = mx;
  }
  // all of the thread's numbers so far -inf: a finite stand-in keeps their
  // weights 0 rather than NaN
  const float m = st.m == kNegInf ? 0.f : st.m;
  const float2 nm = make_float2(-m, -m), cc = make_float2(c, c);
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int i = 0; i + 1 < n; i += 2) {
    const float2 d = __fmul2_rn(fadd2(make_float2(x[i], x[i + 1]), nm), cc);
    s = fadd2(s, make_float2(ex2_approx(d.x), ex2_approx(d.y)));
  }
  if (n & 1) s.x += weight(x[n - 1], m, c);
  st.l += s.x + s.y;
}

__device__ __forceinline__ void take_greedy(Running& st, float x, int v) {
  if (x > st.m || (x == st.m && v < st.arg)) {
    st.m = x;
    st.arg = v;
  }
  if (x != x) st.l = x;  // a NaN shows in the sum
}

// One CTA: piece `split` of one logit row. Rows of sequence b: its S + 1
// target rows, then its S draft rows. Bound by the loads in flight (16 bytes,
// four a thread, each logit read once): 29.9 us for the 151 MB of 64 sequences of
// 4 drafts at V = 131072 in bf16, 5.06 TB/s, with 47 % of the issue slots; packed
// float32 arithmetic; rows of any alignment (a row of an odd vocabulary starts
// anywhere) by single numbers up to the first 16-byte boundary and after the
// last.
template <typename T>
__global__ void __launch_bounds__(kStatThreads) stats_kernel(const VerifyArgs a, Stat* stats,
                                                             int nsplit, int piece) {
  using V = Vec16<T>;
  constexpr int N = V::N, U = 2;
  const int per = a.draft != nullptr ? 2 * a.S + 1 : a.S + 1;
  const int row = blockIdx.x / nsplit, split = blockIdx.x % nsplit;
  const int b = row / per, r = row % per;
  const bool is_draft = r > a.S;
  const int i = is_draft ? r - a.S - 1 : r;
  pdl_wait();
  pdl_trigger();
  bool greedy;
  const float c = log2e_over(a.temperature != nullptr ? a.temperature[b] : 1.f, &greedy);
  const int nd = drafts_of(a, a.n_draft != nullptr ? a.n_draft[b] : a.S);
  if (is_draft ? (i >= nd || greedy) : i > nd) return;  // never looked at
  const T* x = is_draft ? static_cast<const T*>(a.draft) + (int64_t(b) * a.S + i) * a.V
                        : static_cast<const T*>(a.target) + (int64_t(b) * (a.S + 1) + i) * a.V;
  const int v0 = min(a.V, split * piece), v1 = min(a.V, v0 + piece);
  const int tid = threadIdx.x;
  // [v0, h) single, [h, h + N * nv) by 16 bytes, [.., v1) single
  const int lead = static_cast<int>((16 - (reinterpret_cast<uintptr_t>(x + v0) & 15)) & 15) /
                   static_cast<int>(sizeof(T));
  const int h = min(v1, v0 + lead);
  const int nv = (v1 - h) / N;
  const int tail = h + nv * N;
  const uint4* xv = reinterpret_cast<const uint4*>(x + h);
  Running st;
  if (!greedy) {
    // Whole batches of U groups a thread, two register sets in turn, each
    // loaded while the other is worked on; then one batch with what is left,
    // whose missing groups count as -inf.
    const uint4* at = xv + tid;
    auto load = [&](uint4 (&w)[U], int batch) {
#pragma unroll
      for (int j = 0; j < U; ++j) w[j] = at[(batch * U + j) * kStatThreads];
    };
    auto work = [&](const uint4 (&w)[U]) {
      float y[U * N];
#pragma unroll
      for (int j = 0; j < U; ++j) V::unpack(w[j], y + j * N);
      take_batch<U * N>(st, y, c);
    };
    const int whole = nv / (U * kStatThreads);
    uint4 wa[U], wb[U], rest[U];
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int k = (whole * U + j) * kStatThreads;
      rest[j] = make_uint4(V::kNone, V::kNone, V::kNone, V::kNone);
      if (k + tid < nv) rest[j] = at[k];
    }
    if (whole > 0) load(wa, 0);
    int i = 0;
    for (; i + 2 <= whole; i += 2) {
      load(wb, i + 1);
      work(wa);
      if (i + 2 < whole) load(wa, i + 2);
      work(wb);
    }
    if (i < whole) work(wa);
    work(rest);
    for (int v = v0 + tid; v < h; v += kStatThreads) {
      const float y = to_f32(x[v]);
      take_batch<1>(st, &y, c);
    }
    for (int v = tail + tid; v < v1; v += kStatThreads) {
      const float y = to_f32(x[v]);
      take_batch<1>(st, &y, c);
    }
  } else {
    for (int k = tid; k < nv; k += kStatThreads) {
      float y[N];
      V::unpack(xv[k], y);
#pragma unroll
      for (int j = 0; j < N; ++j) take_greedy(st, y[j], h + k * N + j);
    }
    for (int v = v0 + tid; v < h; v += kStatThreads) take_greedy(st, to_f32(x[v]), v);
    for (int v = tail + tid; v < v1; v += kStatThreads) take_greedy(st, to_f32(x[v]), v);
  }
  float m = st.m, l = st.l;
  int arg = st.arg;
  __shared__ Stat part[kStatWarps];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    const int a2 = __shfl_xor_sync(0xffffffffu, arg, o);
    arg = m2 > m ? a2 : m2 == m ? min(arg, a2) : arg;
    merge(m, l, m2, l2, c);
  }
  if ((tid & 31) == 0) part[tid >> 5] = Stat{m, l, arg, 0};
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < kStatWarps; ++w) {
      const Stat s = part[w];
      arg = s.m > m ? s.arg : s.m == m ? min(arg, s.arg) : arg;
      merge(m, l, s.m, s.l, c);
    }
    stats[int64_t(row) * nsplit + split] = Stat{m, l, arg, 0};
  }
}

struct Best {
  float score;
  int idx;
};
__device__ __forceinline__ void take(Best& a, float score, int idx) {
  if (score > a.score || (score == a.score && idx < a.idx)) a = Best{score, idx};
}

// W consecutive numbers, loaded as one or two words.
template <typename T, int W>
struct alignas(W * sizeof(T) < 16 ? W * sizeof(T) : 16) Pack {
  T x[W];
};

// One cluster per sequence. W: the numbers a thread loads at a time from each
// row; every row starts on a boundary of W numbers. Bound by the latency of its
// few rounds of loads: 21.5 us alone on cold caches for 64 sequences at
// V = 131072 in bf16, which read 64 MB, 38 % of the memory's rate; behind
// stats_kernel, with part of that in L2, about 12. Measured when both kernels took
// 46.7 us there: the exponentials prefetched into L2 under stats_kernel, 47.9 (they
// take their bandwidth from it). Two register sets against the compiler's
// unrolled loads, both kernels of 16 sequences at an odd V = 50001 (9.3 us today):
// 12.3 us against 13.7.
template <typename T, int W, int kThreads>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads, 1024 / kThreads)
    choose_kernel(const VerifyArgs a, const Stat* stats, int nsplit) {
  constexpr int kWarps = kThreads / 32;
  __shared__ float rm[2 * kMaxDrafts + 1], rl[2 * kMaxDrafts + 1];
  __shared__ int rarg[2 * kMaxDrafts + 1];
  __shared__ uint8_t accept[kMaxDrafts];
  __shared__ Best wbest[kWarps];
  __shared__ Best cbest[2][kCluster];
  __shared__ int chosen_pass[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / kCluster;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int per = a.draft != nullptr ? 2 * a.S + 1 : a.S + 1;
  cluster.barrier_arrive();  // waited for before any CTA's memory is written by another
  const T* target = static_cast<const T*>(a.target) + int64_t(b) * (a.S + 1) * a.V;
  const T* draft = static_cast<const T*>(a.draft) + (a.draft != nullptr ? int64_t(b) * a.S * a.V : 0);
  // stats_kernel lets this grid start only when all of its CTAs have seen the
  // work before it complete, so the call's inputs are complete in L2 by now; only
  // pdl_wait makes them visible through L1, so what is read before it is read past
  // L1. What stats_kernel writes has to be waited for, and this grid writes
  // nothing before.
  bool greedy;
  const float c =
      log2e_over(a.temperature != nullptr ? __ldcg(a.temperature + b) : 1.f, &greedy);
  const int nd = drafts_of(a, a.n_draft != nullptr ? __ldcg(a.n_draft + b) : a.S);
  // the drafted tokens' logits, on their way while the statistics are joined
  int x = 0;
  bool in_range = false;
  float xt = 0.f, xd = 0.f, xu = 0.f;
  if (tid < nd) {
    x = __ldcg(a.tokens + int64_t(b) * a.S + tid);
    xu = __ldcg(a.u + int64_t(b) * a.S + tid);
    in_range = x >= 0 && x < a.V;
    if (in_range && !greedy) {
      xt = to_f32(__ldcg(target + int64_t(tid) * a.V + x));
      if (a.draft != nullptr) xd = to_f32(__ldcg(draft + int64_t(tid) * a.V + x));
    }
  }
  pdl_wait();
  // The row statistics, joined from their pieces in a fixed order. stats_kernel
  // may write them while this grid runs, so they are neither __restrict__ (read
  // as data that never changes) nor taken from L1.
  for (int r = warp; r < per; r += kWarps) {
    const bool is_draft = r > a.S;
    const int i = is_draft ? r - a.S - 1 : r;
    if (is_draft ? (i >= nd || greedy) : i > nd) continue;
    float m = kNegInf, l = 0.f;
    int arg = kNone;
    if (lane < nsplit) {
      const int4 s = __ldcg(reinterpret_cast<const int4*>(stats + (int64_t(b) * per + r) * nsplit + lane));
      m = __int_as_float(s.x);
      l = __int_as_float(s.y);
      arg = s.z;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
      const int a2 = __shfl_xor_sync(0xffffffffu, arg, o);
      arg = m2 > m ? a2 : m2 == m ? min(arg, a2) : arg;
      merge(m, l, m2, l2, c);
    }
    if (lane == 0) {
      rm[r] = m;
      rl[r] = l;
      // the greedy choice, of a row with a finite maximum and without NaN
      rarg[r] = l == 0.f && fabsf(m) <= FLT_MAX ? arg : -1;
    }
  }
  __syncthreads();
  if (tid < nd) {
    bool acc = false;
    if (!in_range) {
      record_status(a.status, dev_code(kDevBadList, kKerVerify, 1));
    } else if (greedy) {
      acc = x == rarg[tid];
    } else {
      const float p = weight(xt, rm[tid], c) / rl[tid];
      const int rd = a.S + 1 + tid;
      const float q = a.draft != nullptr ? weight(xd, rm[rd], c) / rl[rd] : 1.f;
      acc = xu * q < p;
    }
    accept[tid] = acc;
  }
  __syncthreads();
  int at = 0;
  while (at < nd && accept[at]) ++at;  // nd <= kMaxDrafts, shared memory broadcast
  // the choice at position `at`
  int chosen;
  cluster.barrier_wait();
  if (greedy) {
    chosen = rarg[at];
  } else {
    const bool refused = at < nd;
    const T* pt = target + int64_t(at) * a.V;
    const T* qt = draft + int64_t(at) * a.V;
    const bool has_q = refused && a.draft != nullptr;
    const float* e = a.expo + int64_t(b) * a.V;
    // p = exp2((x - m) c - log2 l): the sum's logarithm rides in the exponent
    const float pm = rm[at], pk = -log2f(rl[at]);
    const float qm = has_q ? rm[a.S + 1 + at] : 0.f, qk = has_q ? -log2f(rl[a.S + 1 + at]) : 0.f;
    const int out_of_race = refused && !has_q ? a.tokens[int64_t(b) * a.S + at] : -1;
    chosen = -1;
    // pass 0: the remainder max(p - q, 0) (p itself when everything was
    // accepted); pass 1, only when rounding leaves nothing of the remainder: p.
    // None when the draft row has no probabilities (its sum is 0 or NaN).
    const bool draws = !has_q || rl[a.S + 1 + at] > 0.f;
    for (int pass = 0; draws && pass < (refused ? 2 : 1); ++pass) {
      Best best{0.f, kNone};
      const int skip = pass == 0 ? out_of_race : -1;
      // w / e as w * (1 / e): two steps of error, below what the weights carry.
      // A thread's indices ascend, so the first of equal scores stays.
      auto one = [&](float w, float ev, int v) {
        const float score = w * rcp_approx(ev);
        if (score > best.score) best = Best{score, v};
      };
      auto p_of = [&](float x) { return ex2_approx(fmaf(x - pm, c, pk)); };
      auto q_of = [&](float x) { return ex2_approx(fmaf(x - qm, c, qk)); };
      // two register sets in turn: one loads while the other is worked on
      constexpr int U = W == 1 ? 4 : 1;
      constexpr int kStep = kCluster * kThreads * W;
      const bool two = has_q && pass == 0;
      struct Set {
        Pack<T, W> p[U], q[U];
        Pack<float, W> e[U];
      };
      auto load = [&](Set& k, int v) {
#pragma unroll
        for (int j = 0; j < U; ++j, v += kStep) {
          if (v >= a.V) break;
          k.p[j] = *reinterpret_cast<const Pack<T, W>*>(pt + v);
          if (two) k.q[j] = *reinterpret_cast<const Pack<T, W>*>(qt + v);
          k.e[j] = *reinterpret_cast<const Pack<float, W>*>(e + v);
        }
      };
      auto work = [&](const Set& k, int v) {
#pragma unroll
        for (int j = 0; j < U; ++j, v += kStep) {
          if (v >= a.V) break;
#pragma unroll
          for (int i = 0; i < W; ++i) {
            const float w = v + i == skip ? 0.f : p_of(to_f32(k.p[j].x[i]));
            one(two ? w - q_of(to_f32(k.q[j].x[i])) : w, k.e[j].x[i], v + i);
          }
        }
      };
      Set ka, kb;
      int v = (rank * kThreads + tid) * W;
      load(ka, v);
      while (v < a.V) {
        load(kb, v + U * kStep);
        work(ka, v);
        v += U * kStep;
        load(ka, v + U * kStep);
        work(kb, v);
        v += U * kStep;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        take(best, __shfl_xor_sync(0xffffffffu, best.score, o),
             __shfl_xor_sync(0xffffffffu, best.idx, o));
      if (lane == 0) wbest[warp] = best;
      __syncthreads();
      if (warp == 0) {
        best = lane < kWarps ? wbest[lane] : Best{0.f, kNone};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
          take(best, __shfl_xor_sync(0xffffffffu, best.score, o),
               __shfl_xor_sync(0xffffffffu, best.idx, o));
        if (lane < kCluster) *cluster.map_shared_rank(&cbest[pass][rank], lane) = best;
      }
      cluster.sync();
      // every CTA joins the cluster's bests, so that all agree on a second pass
      if (tid == 0) {
        Best all = cbest[pass][0];
        for (int k = 1; k < kCluster; ++k) take(all, cbest[pass][k].score, cbest[pass][k].idx);
        chosen_pass[pass] = all.score > 0.f ? all.idx : -1;
      }
      __syncthreads();
      chosen = chosen_pass[pass];
      if (chosen >= 0) break;
    }
  }
  if (rank != 0) return;
  if (tid == 0) {
    if (chosen < 0) record_status(a.status, dev_code(kDevBadList, kKerVerify, 2));
    a.n_accepted[b] = at;
  }
  for (int i = tid; i <= a.S; i += kThreads)
    a.out[int64_t(b) * (a.S + 1) + i] =
        i < at ? a.tokens[int64_t(b) * a.S + i] : i == at ? chosen : -1;
}

template <typename T, int W>
cudaError_t launch_choose(const VerifyArgs& a, const Stat* stats, int nsplit, cudaStream_t s) {
  // as many threads a CTA as keep all clusters resident at once: with few
  // sequences a sweep over the vocabulary then takes few rounds of loads, with
  // many there is no second wave. Both kernels, replayed, at 512 threads and at
  // 256: one sequence, V = 32000, float32: 5.7 us and 6.5; 64 sequences,
  // V = 131072, bf16: 46.0 and 42.0.
  const int ctas = a.B * kCluster;
  const bool few = ctas <= 2 * 152;
  return launch_pdl(few ? choose_kernel<T, W, 512> : choose_kernel<T, W, 256>, dim3(ctas),
                    dim3(few ? 512 : 256), 0, s, a, stats, nsplit);
}

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, void* ws, cudaStream_t s) {
  Stat* stats = static_cast<Stat*>(ws);
  const int64_t rows = int64_t(a.B) * (a.draft != nullptr ? 2 * a.S + 1 : a.S + 1);
  // enough pieces that the rows fill the SMs a few times over, but pieces of at
  // least 2048 logits. Both kernels, replayed, at 3, 6, 8 and 16 times over: 64
  // sequences of 4 drafts, V = 131072, bf16: 48.0, 42.0, 45.1, 44.9 us (4 and 5
  // times give the same pieces as 6; more pieces pay their start more often); 16
  // sequences of up to 7 copied drafts, V = 50001, float32: 9.7, 9.3, 8.8, 10.4.
  int64_t nsplit = (152 * 6 + rows - 1) / rows;
  nsplit = min64(min64(nsplit, kMaxSplits), (int64_t(a.V) + 2047) / 2048);
  // pieces of whole 16-byte groups
  const int piece = static_cast<int>(((a.V + nsplit - 1) / nsplit + 7) / 8 * 8);
  if (rows * nsplit > 0x7fffffffLL || int64_t(a.B) * kCluster > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  const int ns = static_cast<int>(nsplit);
  cudaError_t e = launch_pdl(stats_kernel<T>, dim3(static_cast<unsigned>(rows * nsplit)),
                             dim3(kStatThreads), 0, s, a, stats, ns, piece);
  if (e != cudaSuccess) return e;
  const auto at = [](const void* p) { return reinterpret_cast<uintptr_t>(p); };
  const auto fits = [&](int w) {
    return a.V % w == 0 && at(a.target) % (w * sizeof(T)) == 0 &&
           at(a.draft) % (w * sizeof(T)) == 0 && at(a.expo) % 16 == 0;
  };
  if constexpr (sizeof(T) == 2)
    if (fits(8)) return launch_choose<T, 8>(a, stats, ns, s);
  if (fits(4)) return launch_choose<T, 4>(a, stats, ns, s);
  return launch_choose<T, 1>(a, stats, ns, s);
}

}  // namespace

int64_t draft_verify_stats(int B, int S) { return int64_t(B) * (2 * S + 1) * kMaxSplits * sizeof(Stat); }

cudaError_t launch_draft_verify(const VerifyArgs& a, rf_dtype dt, void* ws, cudaStream_t s) {
  return dt == RF_F32 ? launch_t<float>(a, ws, s) : launch_t<__nv_bfloat16>(a, ws, s);
}

}  // namespace rf
