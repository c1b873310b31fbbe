// attn_paged.cu -- attention of a ragged batch's new tokens over a paged
// key/value cache. Simple form: one warp per (token, head).
#include "paged_plan.h"
#include "rf_device.cuh"

namespace rf {
namespace {

__device__ __forceinline__ bool plan_matches(const PlanHeader* h, const PagedAttnArgs& a) {
  return h->magic == kPlanMagic && h->B == a.B && h->T == a.T && h->H == a.H && h->Hkv == a.Hkv &&
         h->page == a.page && h->max_pages == a.max_pages;
}

template <int D>
__global__ void __launch_bounds__(128) attn_paged_simple(const PagedAttnArgs a) {
  constexpr int E = D / 32;
  const PlanHeader* h = static_cast<const PlanHeader*>(a.plan);
  if (!plan_matches(h, a)) {
    record_status(a.status, dev_code(kDevBadList, kKerPaged, 2));
    return;
  }
  if (h->ctas == 0) return;
  const int lane = threadIdx.x & 31;
  const int64_t row = int64_t(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (row >= int64_t(a.T) * a.H) return;
  const int t = static_cast<int>(row / a.H), hd = static_cast<int>(row % a.H);
  const int32_t* cu = plan_cu_q(a.plan);
  const int32_t* kvl = plan_kv_len(a.plan, a.B);
  int lo = 0, hi = a.B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid + 1] <= t) lo = mid + 1; else hi = mid;
  }
  if (lo >= a.B || cu[lo] > t) return;
  const int n = cu[lo + 1] - cu[lo], kv = kvl[lo];
  const int lim = plan_visible(t - cu[lo], n, kv, h->causal);
  const int hk = hd / (a.H / a.Hkv);
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + t * a.q_stride + hd * D + lane * E;
  float qv[E], acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) {
    qv[e] = __bfloat162float(q[e]) * a.scale * kLog2e;
    acc[e] = 0.f;
  }
  float m = kNegInf, l = 0.f;
  for (int j = 0; j < lim; ++j) {
    const int id = a.table[lo * a.table_stride + j / a.page];
    if (id < 0 || id >= a.num_pages) {
      record_status(a.status, dev_code(kDevBadList, kKerPaged, 3));
      return;
    }
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.k_cache) + id * a.k_page_stride +
                             (j % a.page) * a.k_token_stride + hk * a.k_head_stride + lane * E;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.v_cache) + id * a.v_page_stride +
                             (j % a.page) * a.v_token_stride + hk * a.v_head_stride + lane * E;
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) s += qv[e] * __bfloat162float(k[e]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float mn = fmaxf(m, s);
    const float al = m == kNegInf ? 0.f : ex2_approx(m - mn);
    const float p = s == kNegInf ? 0.f : ex2_approx(s - mn);
    m = mn;
    l = l * al + p;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = acc[e] * al + p * __bfloat162float(v[e]);
  }
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + row * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = __float2bfloat16(l > 0.f ? acc[e] / l : 0.f);
  if (lane == 0 && a.lse != nullptr) a.lse[row] = l > 0.f ? (m + log2f(l)) * kLn2 : kNegInf;
}

}  // namespace

cudaError_t launch_attn_paged(const PagedAttnArgs& a, cudaStream_t s, const char** why) {
  const int64_t grid = (int64_t(a.T) * a.H + 3) / 4;
  if (grid > 0x7fffffffLL) {
    *why = "too many rows";
    return cudaErrorInvalidConfiguration;
  }
  if (a.d == 128)
    attn_paged_simple<128><<<static_cast<unsigned>(grid), 128, 0, s>>>(a);
  else
    attn_paged_simple<64><<<static_cast<unsigned>(grid), 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace rf
