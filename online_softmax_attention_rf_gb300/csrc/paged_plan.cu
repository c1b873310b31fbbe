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
// Cost of an item, in units of 0.28 us: a fixed part (filling the pipeline and
// writing the output) and a part per step. Set at d = 128. Two tiles: a step
// measured at 1.7 us, the fixed part at 5 us (18 units); 22 units stand between
// what the spans of six ragged chunks showed, 92 us on average: the longest 106
// us at 18 units, 98 at 28 with the shortest down to 74. One tile: 3.4 us, and
// 1.45 a step (memory bounds the step of a decode item). At d = 64, for which the
// same costs are used, steps take 1.45 and 0.85 us: a one-tile step is charged
// too much there, and by those times the longest span of a batch that mixes
// chunks and single tokens is 16 % above the mean.
constexpr int kPairFixed = 22;
constexpr int kPairCost = 6;
constexpr int kSingleFixed = 12;
constexpr int kSingleCost = 5;
// A span is worth at least this much. Two cuts of one item are then more than
// a step apart: no CTA inside an item is left without steps.
constexpr int kMinSpan = 8;
static_assert(kMinSpan - 1 >= kPairCost && kPairCost >= kSingleCost, "cuts may coincide");
// With no more items than CTAs an item is cut by itself, into equal parts of at
// least this cost (both softmax groups have a step of a one-tile item then): a
// span that held the end of one item and the start of the next would pay two
// fixed parts one after the other (8 items of 5 steps: 10.6 us, against 7.5).
constexpr int kMinPart = 10;

struct Item {
  int rows, steps, cost;
  int fixed, per_step;
};

// Item `pair` of a sequence with n new and kv cached tokens.
__device__ __forceinline__ Item item_of(int pair, int n, int kv, int causal, int G) {
  const int tt = plan_tile_tokens(G);
  const int i0 = pair * 2 * tt, i1 = min(n, i0 + 2 * tt);
  Item it;
  it.rows = (i1 - i0) * G;
  it.steps = plan_steps(plan_visible(i1 - 1, n, kv, causal));
  const bool two = i1 - i0 > tt;
  it.per_step = two ? kPairCost : kSingleCost;
  it.fixed = two ? kPairFixed : kSingleFixed;
  it.cost = it.fixed + it.steps * it.per_step;
  return it;
}

__device__ PlanStart locate_item(int64_t x, const int64_t* cost, const int32_t* cu, const int32_t* kvl,
                            const PagedPlanArgs& a) {
  int lo = 0, hi = a.B;  // the first b with cost[b + 1] > x
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cost[mid + 1] <= x) lo = mid + 1; else hi = mid;
  }
  PlanStart st{lo, 0, 0, 0, 0, 0, 0, 0};
  if (lo == a.B) return st;
  const int G = a.H / a.Hkv, tt = plan_tile_tokens(G);
  const int n = cu[lo + 1] - cu[lo], kv = kvl[lo];
  const int pairs = (n + 2 * tt - 1) / (2 * tt);
  int64_t rem = x - cost[lo];
  const int64_t per_head = (cost[lo + 1] - cost[lo]) / a.Hkv;
  st.head = static_cast<int>(rem / per_head);
  rem -= st.head * per_head;
  for (; st.pair < pairs; ++st.pair) {
    const Item it = item_of(st.pair, n, kv, a.causal, G);
    if (rem < it.cost) {
      const int step =
          rem <= it.fixed ? 0 : static_cast<int>((rem - it.fixed + it.per_step - 1) / it.per_step);
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

// The start at cost x, with its sequence's lengths.
__device__ PlanStart locate(int64_t x, const int64_t* cost, const int32_t* cu, const int32_t* kvl,
                            const PagedPlanArgs& a) {
  PlanStart st = locate_item(x, cost, cu, kvl, a);
  if (st.seq < a.B) {
    st.row0 = cu[st.seq];
    st.row1 = cu[st.seq + 1];
    st.kv = kvl[st.seq];
  }
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
  const bool few = items * a.Hkv <= kPlanCtas;
  __syncthreads();
  // prefix sums over the sequences of their costs, or of their items
  auto scan = [&](bool count) {
    for (int b = warp; b < a.B; b += kThreads / 32) {
      const int n = cu[b + 1] - cu[b], kv = kvl[b];
      const int pairs = (n + 2 * tt - 1) / (2 * tt);
      int64_t sum = count ? (lane == 0 ? pairs : 0) : 0;
      if (!count)
        for (int p = lane; p < pairs; p += 32) sum += item_of(p, n, kv, a.causal, G).cost;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (lane == 0) cost[b + 1] = sum * a.Hkv;
    }
    if (tid == 0) carry = 0;
    __syncthreads();
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
    return cost[a.B];
  };
  const int64_t total = scan(few);
  int ctas = 0;
  bool by_item = few;
  if (few) {
    // thread i has item i
    PlanStart st{};
    Item it{};
    int worth = 0;
    if (tid < total) {
      int lo = 0, hi = a.B;  // the first b with cost[b + 1] > tid
      while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (cost[mid + 1] <= tid) lo = mid + 1; else hi = mid;
      }
      const int per_head = static_cast<int>(cost[lo + 1] - cost[lo]) / a.Hkv;
      const int rem = tid - static_cast<int>(cost[lo]);
      st = PlanStart{lo, rem / per_head, rem % per_head, 0, cu[lo], cu[lo + 1], kvl[lo], 0};
      it = item_of(st.pair, st.row1 - st.row0, st.kv, a.causal, G);
      worth = it.steps * it.per_step;
    }
    if (tid < kPlanCtas) units[tid] = worth;
    __syncthreads();
    // the least part worth (a warp, by bisection) with which all parts fit
    if (warp == 0) {
      auto parts_at = [&](int part) {
        int sum = 0;
        for (int i = lane; i < total; i += 32) sum += max(1, (units[i] + part - 1) / part);
        return __reduce_add_sync(0xffffffffu, sum);
      };
      int lo = kMinPart, hi = kMinPart;
      for (int i = lane; i < total; i += 32) hi = max(hi, units[i]);
      hi = __reduce_max_sync(0xffffffffu, hi);
      while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (parts_at(mid) <= kPlanCtas) hi = mid; else lo = mid + 1;
      }
      int64_t sum = 0;
      for (int i = lane; i < total; i += 32) sum += units[i];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      // unless the largest part is longer than an even span and its second
      // fixed part: items of unequal length, about as many as CTAs
      if (lane == 0) carry = lo <= sum / kPlanCtas + kSingleFixed || lo == kMinPart ? lo : -1;
    }
    __syncthreads();
    const int part = static_cast<int>(carry);
    by_item = part > 0;
    __syncthreads();
    if (by_item) {
      const int parts = tid < total ? max(1, min(it.steps, (worth + part - 1) / part)) : 0;
      if (tid < kPlanCtas) flag[tid] = parts;
      __syncthreads();
      int cta0 = 0;
      ctas = 0;
      for (int i = 0; i < total; ++i) {
        if (i < tid) cta0 += flag[i];
        ctas += flag[i];
      }
      for (int j = 0; j < parts; ++j) {
        st.step = static_cast<int>(int64_t(it.steps) * j / parts);
        start[cta0 + j] = st;
      }
      if (tid == 0) start[ctas] = PlanStart{a.B, 0, 0, 0, 0, 0, 0, 0};
    }
  }
  if (!by_item) {
    const int64_t sum = few ? scan(false) : total;
    ctas = static_cast<int>(min64(kPlanCtas, max64(1, sum / kMinSpan)));
    if (tid <= ctas) start[tid] = locate(sum * tid / ctas, cost, cu, kvl, a);
  }
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
        const int rows = item_of(s.pair, cu[s.seq + 1] - cu[s.seq], kvl[s.seq], a.causal, G).rows;
        m = PlanMerge{s.seq, s.head, s.pair, tid - 1, parts, rows, 0, s.row0 + s.pair * 2 * tt};
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
