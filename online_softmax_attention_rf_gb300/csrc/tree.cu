// tree.cu -- trees of drafted tokens: the attention mask of a tree's nodes, and
// the walk down it along the tokens that the target drew.
//
// A step's nodes are packed like a step's tokens: sequence b has the rows
// cu_q[b] .. cu_q[b + 1] - 1, in an order in which a node follows its parent;
// parents are numbered within the sequence. A CTA takes a sequence. Bound by
// latency, a few dependent loads and the steps of the walk: one tree of 32 nodes,
// replayed, mask 2.8 us, walk 1.9.
#include "paged_device.cuh"

namespace rf {
namespace {

constexpr int kThreads = 128;
constexpr int kStaged = 1024;  // nodes of a sequence kept in shared memory

// Rows of sequence b; none (and reported) when the offsets are not ascending
// within [0, T].
__device__ __forceinline__ bool rows_of(const int32_t* cu_q, int b, int T, int* first, int* n) {
  const int c0 = cu_q[b], c1 = cu_q[b + 1];
  *first = c0;
  *n = c0 >= 0 && c1 >= c0 ? c1 - c0 : 0;
  return c0 >= 0 && c1 >= c0 && c1 <= T;
}

// The rows of [lo, hi) that no sequence with good offsets has, f(row) for each. All
// threads call. A look at all offsets finds either how far the rows from the present one
// on are some sequence's, or how far they are none's; sequences behind each other
// count as one there, so that a few looks do unless most offsets are bad.
template <typename F>
__device__ void unowned(const int32_t* cu_q, int B, int T, int lo, int hi, F&& f) {
  __shared__ int end, next;
  const int each = (B + kThreads - 1) / kThreads;
  const int s0 = min(int64_t(B), int64_t(threadIdx.x) * each), s1 = min(B, s0 + each);
  for (int at = lo; at < hi;) {
    if (threadIdx.x == 0) {
      end = at;
      next = hi;
    }
    __syncthreads();
    for (int s = s0; s < s1;) {
      int n, first, last;
      if (!rows_of(cu_q, s++, T, &first, &n) || n == 0) continue;
      last = first + n;
      for (int more; s < s1 && rows_of(cu_q, s, T, &more, &n); ++s) last = more + n;
      if (first > at)
        atomicMin(&next, first);
      else if (last > at)
        atomicMax(&end, last);
    }
    __syncthreads();
    const int to = end > at ? end : min(next, hi);
    if (end <= at)
      for (int r = at + threadIdx.x; r < to; r += kThreads) f(r);
    __syncthreads();
    at = to;
  }
}

// The rows outside every sequence, f(row) for each: those before the first and
// behind the last, by the CTAs of these two, and those between a sequence's offsets
// where these are not good, by its CTA. (From any row a step in the offsets leads past,
// or it lies before the first or behind the last.)
template <typename F>
__device__ __forceinline__ void outside(const int32_t* cu_q, int b, int B, int T, bool good,
                                        F&& f) {
  if (b == 0)
    for (int r = threadIdx.x; r < min(min(cu_q[0], cu_q[1]), T); r += kThreads) f(r);
  if (b == B - 1)
    for (int64_t r = int64_t(max(0, max(cu_q[B], cu_q[B - 1]))) + threadIdx.x; r < T; r += kThreads)
      f(static_cast<int>(r));
  if (!good)
    unowned(cu_q, B, T, max(0, min(cu_q[b], cu_q[b + 1])), min(T, max(cu_q[b], cu_q[b + 1])), f);
}

// Node i's bits are those of the nodes on its way up, itself among them. Parents
// come before their children, so that the way meets a row's words from the
// highest used one down, and each is written once.
__global__ void __launch_bounds__(kThreads) tree_mask_kernel(const TreeMaskArgs a) {
  __shared__ int parent[kStaged];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  int c0, n;
  const bool good = rows_of(a.cu_q, b, a.T, &c0, &n);
  outside(a.cu_q, b, a.B, a.T, good, [&](int r) {
    for (int w = 0; w < a.words; ++w) a.mask[int64_t(r) * a.words + w] = 0;
    if (a.pos != nullptr) a.pos[r] = 0;
  });
  if (!good || n > 64 * a.words) {  // more nodes than the words have bits for
    if (threadIdx.x == 0) record_status(a.status, dev_code(kDevBadList, kKerTree, 1));
    if (good)
      for (int64_t r = c0 + threadIdx.x; r < int64_t(c0) + n; r += kThreads) {
        for (int w = 0; w < a.words; ++w) a.mask[r * a.words + w] = 0;
        if (a.pos != nullptr) a.pos[r] = 0;
      }
    return;
  }
  const int ctx = a.kv_len != nullptr ? a.kv_len[b] - n : 0;
  for (int i = threadIdx.x; i < n; i += kThreads) {
    int p = a.parent[c0 + i];
    if (p < -1 || p >= i) {  // not before its child: the node stands alone
      record_status(a.status, dev_code(kDevBadList, kKerTree, 2));
      p = -1;
    }
    parent[i] = p;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) {
    uint64_t* row = a.mask + int64_t(c0 + i) * a.words;
    for (int w = a.words - 1; w > i / 64; --w) row[w] = 0;
    int at = i / 64, depth = -1;
    uint64_t bits = 0;
    for (int p = i; p >= 0; p = parent[p]) {
      while (at > p / 64) {
        row[at--] = bits;
        bits = 0;
      }
      bits |= uint64_t(1) << (p % 64);
      ++depth;
    }
    for (; at >= 0; --at) {
      row[at] = bits;
      bits = 0;
    }
    if (a.pos != nullptr) a.pos[c0 + i] = max(0, ctx + depth);
  }
}

// One warp walks; the other warps only help to fetch the nodes.
__global__ void __launch_bounds__(kThreads) tree_accept_kernel(const TreeAcceptArgs a) {
  __shared__ int parent[kStaged], token[kStaged], drawn[kStaged];
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x, lane = threadIdx.x & 31;
  int c0, n;
  const bool good = rows_of(a.cu_q, b, a.T, &c0, &n);
  if (!good) {
    if (threadIdx.x == 0) record_status(a.status, dev_code(kDevBadList, kKerTree, 3));
    n = 0;
  }
  const int kv = a.kv_len[b];
  for (int i = threadIdx.x; i < min(n, kStaged); i += kThreads) {
    parent[i] = a.parent[c0 + i];
    token[i] = a.tokens[c0 + i];
    drawn[i] = a.sampled[c0 + i];
  }
  outside(a.cu_q, b, a.B, a.T, good, [&](int r) { a.path[r] = a.out[r] = -1; });
  __syncthreads();
  __shared__ int walked;
  if (threadIdx.x < 32) {
    int len = 0;
    for (int at = 0; at < n;) {
      const int s = at < kStaged ? drawn[at] : a.sampled[c0 + at];
      if (lane == 0) {
        a.path[c0 + len] = at;
        a.out[c0 + len] = s;
      }
      ++len;
      // the first child, by number, that holds the drawn token (-1: no draw)
      int next = n;
      for (int j0 = at + 1; s >= 0 && j0 < n; j0 += 32) {
        const int j = j0 + lane;
        bool is = false;
        if (j < n) {
          const bool st = j < kStaged;
          is = (st ? parent[j] : a.parent[c0 + j]) == at && (st ? token[j] : a.tokens[c0 + j]) == s;
        }
        const uint32_t hit = __ballot_sync(0xffffffffu, is);
        if (hit != 0) {
          next = j0 + __ffs(hit) - 1;
          break;
        }
      }
      at = next;
    }
    if (lane == 0) {
      walked = len;
      a.n_path[b] = len;
      a.base[b] = kv - n;
      a.new_len[b] = kv - n + len;
    }
  }
  __syncthreads();
  for (int i = walked + threadIdx.x; i < n; i += kThreads) a.path[c0 + i] = a.out[c0 + i] = -1;
}

}  // namespace

cudaError_t launch_tree_mask(const TreeMaskArgs& a, cudaStream_t s) {
  static_assert(64 * kMaxTreeWords <= kStaged, "a tree's parents fit shared memory");
  return launch_pdl(tree_mask_kernel, dim3(a.B), dim3(kThreads), 0, s, a);
}

cudaError_t launch_tree_accept(const TreeAcceptArgs& a, cudaStream_t s) {
  return launch_pdl(tree_accept_kernel, dim3(a.B), dim3(kThreads), 0, s, a);
}

}  // namespace rf
