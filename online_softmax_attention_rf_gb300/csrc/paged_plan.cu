// paged_plan.cu -- rf_paged_plan: a step's attention over a paged cache,
// divided into one span of equal cost per CTA (paged_plan.h has the terms).
//
// One CTA. The lengths stay on the device: a serving loop's lengths change
// every step, and a captured step has to follow them. The plan is made once a
// step and used by the attention of every layer.
#include "paged_plan.h"
#include "rf_device.cuh"

namespace rf {
namespace {

constexpr int kThreads = 1024;
// Cost of an item: a fixed part (filling the pipeline and writing the output),
// plus per step kPairCost when it has two tiles and kSingleCost when it has
// one. Measured at d = 128: 5 us, 1.7 us and 1.2 us. With fewer items than
// CTAs every CTA pays the fixed part about once whatever the cuts are, and only
// the steps are shared out.
constexpr int kItemCost = 8;
constexpr int kItemCostFew = 1;
constexpr int kPairCost = 3;
constexpr int kSingleCost = 2;
// A span is worth at least this much. Two cuts of one item are then more than
// a step apart: no CTA inside an item is left without steps.
constexpr int kMinSpan = 4;
static_assert(kMinSpan - 1 >= kPairCost && kPairCost >= kSingleCost, "cuts may coincide");

struct Item {
  int rows, steps, cost;
};

// Item `pair` of a sequence with n new and kv cached tokens.
__device__ __forceinline__ Item item_of(int pair, int n, int kv, int causal, int G, int fixed) {
  const int tt = plan_tile_tokens(G);
  const int i0 = pair * 2 * tt, i1 = min(n, i0 + 2 * tt);
  Item it;
  it.rows = (i1 - i0) * G;
  it.steps = (plan_visible(i1 - 1, n, kv, causal) + kPlanTile - 1) / kPlanTile;
  it.cost = fixed + it.steps * (i1 - i0 > tt ? kPairCost : kSingleCost);
  return it;
}

__device__ PlanStart locate(int64_t x, const int64_t* cost, const int32_t* cu, const int32_t* kvl,
                            const PagedPlanArgs& a, int fixed) {
  int lo = 0, hi = a.B;  // the first b with cost[b + 1] > x
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cost[mid + 1] <= x) lo = mid + 1; else hi = mid;
  }
  PlanStart st{lo, 0, 0, 0};
  if (lo == a.B) return st;
  const int G = a.H / a.Hkv, tt = plan_tile_tokens(G);
  const int n = cu[lo + 1] - cu[lo], kv = kvl[lo];
  const int pairs = (n + 2 * tt - 1) / (2 * tt);
  int64_t rem = x - cost[lo];
  const int64_t per_head = (cost[lo + 1] - cost[lo]) / a.Hkv;
  st.head = static_cast<int>(rem / per_head);
  rem -= st.head * per_head;
  for (; st.pair < pairs; ++st.pair) {
    const Item it = item_of(st.pair, n, kv, a.causal, G, fixed);
    if (rem < it.cost) {
      const int w = it.rows > tt * G ? kPairCost : kSingleCost;
      const int step = rem <= fixed ? 0 : static_cast<int>((rem - fixed + w - 1) / w);
      if (step < it.steps || step == 0) {
        st.step = step;
        return st;
      }
      ++st.pair;  // past the item's last step: the next item
      break;
    }
    rem -= it.cost;
  }
  if (st.pair < pairs) return st;
  st.pair = 0;
  if (++st.head < a.Hkv) return st;
  st.head = 0;
  do ++st.seq;
  while (st.seq < a.B && cu[st.seq + 1] == cu[st.seq]);
  return st;
}

__device__ __forceinline__ bool same_item(const PlanStart& a, const PlanStart& b) {
  return a.seq == b.seq && a.head == b.head && a.pair == b.pair;
}

__global__ void __launch_bounds__(kThreads) paged_plan_kernel(const PagedPlanArgs a) {
  __shared__ PlanStart start[kPlanCtas + 1];
  __shared__ int flag[kPlanCtas + 1], units[kPlanCtas + 1];
  __shared__ int64_t wsum[32];
  __shared__ int64_t carry;
  PlanHeader* h = static_cast<PlanHeader*>(a.plan);
  int32_t* cu = const_cast<int32_t*>(plan_cu_q(a.plan));
  int32_t* kvl = const_cast<int32_t*>(plan_kv_len(a.plan, a.B));
  int64_t* cost = reinterpret_cast<int64_t*>(static_cast<char*>(a.plan) + plan_cost_offset(a.B));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t max_kv = int64_t(a.max_pages) * a.page;
  bool bad = false;
  for (int b = tid; b <= a.B; b += kThreads) {
    const int c = a.cu_q[b];
    bad |= c < 0 || c > a.T;
    cu[b] = c;
    if (b < a.B) {
      const int kv = a.kv_len[b];
      bad |= kv < 0 || kv > max_kv || a.cu_q[b + 1] < c;
      kvl[b] = kv;
    }
  }
  if (tid == 0) {
    h->magic = kPlanMagic;
    h->B = a.B; h->T = a.T; h->H = a.H; h->Hkv = a.Hkv;
    h->page = a.page; h->max_pages = a.max_pages; h->causal = a.causal;
    carry = 0;
    cost[0] = 0;
  }
  if (__syncthreads_or(bad)) {
    // lengths that contradict themselves or the table: nothing is computed
    if (tid == 0) {
      h->ctas = h->n_merge = h->merge_units = 0;
      record_status(a.status, dev_code(kDevBadList, kKerPaged, 1));
    }
    return;
  }
  const int G = a.H / a.Hkv, tt = plan_tile_tokens(G);
  // the number of items
  int64_t items = 0;
  for (int b = tid; b < a.B; b += kThreads) items += (cu[b + 1] - cu[b] + 2 * tt - 1) / (2 * tt);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) items += __shfl_xor_sync(0xffffffffu, items, o);
  if (lane == 0) wsum[warp] = items;
  __syncthreads();
  items = 0;
  for (int w = 0; w < kThreads / 32; ++w) items += wsum[w];
  const int fixed = items * a.Hkv > kPlanCtas ? kItemCost : kItemCostFew;
  __syncthreads();
  // costs of the sequences, a warp each
  for (int b = warp; b < a.B; b += kThreads / 32) {
    const int n = cu[b + 1] - cu[b], kv = kvl[b];
    const int pairs = (n + 2 * tt - 1) / (2 * tt);
    int64_t sum = 0;
    for (int p = lane; p < pairs; p += 32) sum += item_of(p, n, kv, a.causal, G, fixed).cost;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) cost[b + 1] = sum * a.Hkv;
  }
  __syncthreads();
  // inclusive prefix sums
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid;
    int64_t v = b < a.B ? cost[b + 1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += u;
    }
    if (lane == 31) wsum[warp] = v;
    __syncthreads();
    if (warp == 0) {
      int64_t s = wsum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += u;
      }
      wsum[lane] = s;
    }
    __syncthreads();
    v += carry + (warp > 0 ? wsum[warp - 1] : 0);
    if (b < a.B) cost[b + 1] = v;
    __syncthreads();
    if (tid == kThreads - 1) carry = v;
    __syncthreads();
  }
  const int64_t total = cost[a.B];
  const int ctas = total == 0 ? 0 : static_cast<int>(min64(kPlanCtas, max64(1, total / kMinSpan)));
  if (tid <= ctas) start[tid] = locate(ctas > 0 ? total * tid / ctas : 0, cost, cu, kvl, a, fixed);
  __syncthreads();
  // items that a cut falls into: found by the first cut inside each
  PlanMerge m{};
  bool first = false;
  if (tid <= ctas) {
    const PlanStart s = start[tid];
    if (tid > 0 && tid < ctas && s.step > 0) {
      const PlanStart p = start[tid - 1];
      first = !same_item(p, s) || p.step == 0;
      if (first) {
        int parts = 1;
        while (tid + parts <= ctas && start[tid + parts - 1].step > 0 &&
               same_item(start[tid + parts - 1], s))
          ++parts;
        const int rows = item_of(s.pair, cu[s.seq + 1] - cu[s.seq], kvl[s.seq], a.causal, G, fixed).rows;
        m = PlanMerge{s.seq, s.head, s.pair, tid - 1, parts, rows, 0, 0};
      }
    }
    flag[tid] = first;
    units[tid] = first ? plan_units(m.rows / G, 0, G) + plan_units(m.rows / G, 1, G) : 0;
    h->start[tid] = s;
  }
  __syncthreads();
  if (tid <= ctas) {
    int idx = 0;
    for (int c = 0; c < tid; ++c) {
      idx += flag[c];
      m.unit0 += units[c];
    }
    if (first) h->merge[idx] = m;
    if (tid == ctas) {
      h->ctas = ctas;
      h->n_merge = idx;
      h->merge_units = m.unit0;
    }
  }
}

}  // namespace

cudaError_t launch_paged_plan(const PagedPlanArgs& a, cudaStream_t s) {
  paged_plan_kernel<<<1, kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace rf
