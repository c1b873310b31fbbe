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
// per sequence that needs it, with a cluster of CTAs per sequence.
#include <cooperative_groups.h>

#include "rf_device.cuh"

namespace rf {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSplits = 32;
constexpr int kCluster = 8;
constexpr int kNone = 0x7fffffff;

// State of one row piece: maximum, sum of exp((x - max) / T), lowest index of
// the maximum (filled in greedy rows only).
struct Stat {
  float m, l;
  int arg, pad;
};

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// exp((x - m) / T) with c = log2(e) / T. The difference is taken before the
// scaling, so that it is exact or nearly so for the entries that matter.
__device__ __forceinline__ float weight(float x, float m, float c) { return ex2_approx((x - m) * c); }

__device__ __forceinline__ float log2e_over(const float* temperature, int b, bool* greedy) {
  const float t = temperature != nullptr ? temperature[b] : 1.f;
  *greedy = !(t > 0.f);
  return *greedy ? kLog2e : kLog2e / t;
}

__device__ __forceinline__ int drafts_of(const VerifyArgs& a, int b) {
  return a.n_draft != nullptr ? max(0, min(a.S, a.n_draft[b])) : a.S;
}

__device__ __forceinline__ void merge(float& m, float& l, float m2, float l2, float c) {
  const float mn = fmaxf(m, m2);
  // an empty side (m = -inf) has weight 0; its exponent would be inf - inf
  l = (m == kNegInf ? 0.f : l * weight(m, mn, c)) + (m2 == kNegInf ? 0.f : l2 * weight(m2, mn, c));
  m = mn;
}

// One CTA: piece `split` of one logit row. Rows of sequence b: its S + 1
// target rows, then its S draft rows.
template <typename T>
__global__ void __launch_bounds__(kThreads) stats_kernel(const VerifyArgs a, Stat* stats, int nsplit,
                                                         int piece) {
  const int per = a.draft != nullptr ? 2 * a.S + 1 : a.S + 1;
  const int row = blockIdx.x / nsplit, split = blockIdx.x % nsplit;
  const int b = row / per, r = row % per;
  const bool is_draft = r > a.S;
  const int i = is_draft ? r - a.S - 1 : r;
  bool greedy;
  const float c = log2e_over(a.temperature, b, &greedy);
  const int nd = drafts_of(a, b);
  if (is_draft ? (i >= nd || greedy) : i > nd) return;  // never looked at
  const T* x = is_draft ? static_cast<const T*>(a.draft) + (int64_t(b) * a.S + i) * a.V
                        : static_cast<const T*>(a.target) + (int64_t(b) * (a.S + 1) + i) * a.V;
  const int v0 = min(a.V, split * piece), v1 = min(a.V, v0 + piece);
  float m = kNegInf, l = 0.f;
  int arg = kNone;
  for (int v = v0 + threadIdx.x; v < v1; v += kThreads) {
    const float xv = to_f32(x[v]);
    if (xv > m) {
      l = m == kNegInf ? 0.f : l * weight(m, xv, c);
      m = xv;
      arg = v;
    }
    if (xv != kNegInf) l += weight(xv, m, c);
  }
  __shared__ Stat part[kWarps];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float m2 = __shfl_xor_sync(0xffffffffu, m, o), l2 = __shfl_xor_sync(0xffffffffu, l, o);
    const int a2 = __shfl_xor_sync(0xffffffffu, arg, o);
    arg = m2 > m ? a2 : m2 == m ? min(arg, a2) : arg;
    merge(m, l, m2, l2, c);
  }
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = Stat{m, l, arg, 0};
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kWarps; ++w) {
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

// One cluster per sequence.
template <typename T>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kThreads)
    choose_kernel(const VerifyArgs a, const Stat* __restrict__ stats, int nsplit) {
  __shared__ float rm[2 * kMaxDrafts + 1], rl[2 * kMaxDrafts + 1];
  __shared__ int rarg[2 * kMaxDrafts + 1];
  __shared__ uint8_t accept[kMaxDrafts];
  __shared__ Best wbest[2][kWarps];
  __shared__ Best cbest[2][kCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int b = blockIdx.x / kCluster;
  cluster.barrier_arrive();  // waited for before rank 0's memory is written
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = a.draft != nullptr ? 2 * a.S + 1 : a.S + 1;
  bool greedy;
  const float c = log2e_over(a.temperature, b, &greedy);
  const int nd = drafts_of(a, b);
  // the row statistics, joined from their pieces in a fixed order
  for (int r = warp; r < per; r += kWarps) {
    const bool is_draft = r > a.S;
    const int i = is_draft ? r - a.S - 1 : r;
    if (is_draft ? (i >= nd || greedy) : i > nd) continue;
    float m = kNegInf, l = 0.f;
    int arg = kNone;
    if (lane < nsplit) {
      const Stat s = stats[(int64_t(b) * per + r) * nsplit + lane];
      m = s.m;
      l = s.l;
      arg = s.arg;
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
      rarg[r] = arg;
    }
  }
  __syncthreads();
  const T* target = static_cast<const T*>(a.target) + int64_t(b) * (a.S + 1) * a.V;
  const T* draft = static_cast<const T*>(a.draft) + (a.draft != nullptr ? int64_t(b) * a.S * a.V : 0);
  for (int i = threadIdx.x; i < nd; i += kThreads) {
    const int x = a.tokens[int64_t(b) * a.S + i];
    bool acc = false;
    if (x < 0 || x >= a.V) {
      record_status(a.status, dev_code(kDevBadList, kKerVerify, 1));
    } else if (greedy) {
      acc = x == rarg[i];
    } else {
      const float p = weight(to_f32(target[int64_t(i) * a.V + x]), rm[i], c) / rl[i];
      float q = 1.f;
      if (a.draft != nullptr) {
        const int rd = a.S + 1 + i;
        q = weight(to_f32(draft[int64_t(i) * a.V + x]), rm[rd], c) / rl[rd];
      }
      acc = a.u[int64_t(b) * a.S + i] * q < p;
    }
    accept[i] = acc;
  }
  __syncthreads();
  int at = 0;
  while (at < nd && accept[at]) ++at;  // nd <= kMaxDrafts, shared memory broadcast
  // the choice at position `at`
  int chosen;
  if (greedy) {
    cluster.barrier_wait();
    chosen = rarg[at] == kNone ? -1 : rarg[at];
  } else {
    const bool refused = at < nd;
    const T* pt = target + int64_t(at) * a.V;
    const T* qt = draft + int64_t(at) * a.V;
    const bool has_q = refused && a.draft != nullptr;
    const float* e = a.expo + int64_t(b) * a.V;
    const float pm = rm[at], pl = 1.f / rl[at];
    const float qm = has_q ? rm[a.S + 1 + at] : 0.f, ql = has_q ? 1.f / rl[a.S + 1 + at] : 0.f;
    const int xd = refused && a.draft == nullptr ? a.tokens[int64_t(b) * a.S + at] : -1;
    // best over the remainder max(p - q, 0), and over p itself for the case
    // that rounding leaves nothing of the remainder
    Best rest{0.f, kNone}, full{0.f, kNone};
    for (int v = rank * kThreads + threadIdx.x; v < a.V; v += kCluster * kThreads) {
      const float p = weight(to_f32(pt[v]), pm, c) * pl;
      float w = p;
      if (has_q) w = p - weight(to_f32(qt[v]), qm, c) * ql;
      if (v == xd) w = 0.f;
      const float ev = e[v];
      take(rest, w > 0.f ? w / ev : 0.f, v);
      take(full, p / ev, v);
    }
    Best two[2] = {rest, full};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        take(two[k], __shfl_xor_sync(0xffffffffu, two[k].score, o),
             __shfl_xor_sync(0xffffffffu, two[k].idx, o));
      if (lane == 0) wbest[k][warp] = two[k];
    }
    __syncthreads();
    cluster.barrier_wait();
    if (threadIdx.x < 2) {
      Best best = wbest[threadIdx.x][0];
      for (int w = 1; w < kWarps; ++w) take(best, wbest[threadIdx.x][w].score, wbest[threadIdx.x][w].idx);
      *cluster.map_shared_rank(&cbest[threadIdx.x][rank], 0) = best;
    }
    cluster.sync();
    if (rank != 0) return;
    Best r = cbest[0][0], f = cbest[1][0];
    for (int k = 1; k < kCluster; ++k) {
      take(r, cbest[0][k].score, cbest[0][k].idx);
      take(f, cbest[1][k].score, cbest[1][k].idx);
    }
    const Best best = r.score > 0.f ? r : f;
    chosen = best.score > 0.f ? best.idx : -1;
  }
  if (rank != 0) return;
  if (threadIdx.x == 0) {
    if (chosen < 0) record_status(a.status, dev_code(kDevBadList, kKerVerify, 2));
    a.n_accepted[b] = at;
  }
  for (int i = threadIdx.x; i <= a.S; i += kThreads)
    a.out[int64_t(b) * (a.S + 1) + i] =
        i < at ? a.tokens[int64_t(b) * a.S + i] : i == at ? chosen : -1;
}

template <typename T>
cudaError_t launch_t(const VerifyArgs& a, void* ws, cudaStream_t s) {
  Stat* stats = static_cast<Stat*>(ws);
  const int64_t rows = int64_t(a.B) * (a.draft != nullptr ? 2 * a.S + 1 : a.S + 1);
  // enough pieces that the rows fill the SMs a few times over, but pieces of
  // at least 2048 logits
  int64_t nsplit = (152 * 8 + rows - 1) / rows;
  nsplit = min64(min64(nsplit, kMaxSplits), (int64_t(a.V) + 2047) / 2048);
  const int piece = static_cast<int>((a.V + nsplit - 1) / nsplit);
  if (rows * nsplit > 0x7fffffffLL || int64_t(a.B) * kCluster > 0x7fffffffLL)
    return cudaErrorInvalidConfiguration;
  stats_kernel<T><<<static_cast<unsigned>(rows * nsplit), kThreads, 0, s>>>(
      a, stats, static_cast<int>(nsplit), piece);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  choose_kernel<T><<<static_cast<unsigned>(a.B) * kCluster, kThreads, 0, s>>>(
      a, stats, static_cast<int>(nsplit));
  return cudaGetLastError();
}

}  // namespace

int64_t draft_verify_stats(int B, int S) { return int64_t(B) * (2 * S + 1) * kMaxSplits * sizeof(Stat); }

cudaError_t launch_draft_verify(const VerifyArgs& a, rf_dtype dt, void* ws, cudaStream_t s) {
  return dt == RF_F32 ? launch_t<float>(a, ws, s) : launch_t<__nv_bfloat16>(a, ws, s);
}

}  // namespace rf
