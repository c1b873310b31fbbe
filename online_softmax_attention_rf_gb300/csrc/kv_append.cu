// kv_append.cu -- the write side of a paged key/value cache.
//
// rf_paged_slots: where each new token of a ragged batch goes. Token i of
// sequence b (n_b new tokens, kv_len[b] cached ones including them) has
// position kv_len[b] - n_b + i and lands in row position % page of page
// table[b][position / page].
//
// rf_kv_append_paged: per (token, head) row x of q or k, in float32,
//   y = x * rsqrt(mean(x^2) + eps) * w            (when the head norm is on)
//   y_i, y_j <- y_i c - y_j s, y_j c + y_i s      for the rotated pairs (i, j)
// with one rounding at the store; q goes to q_out, k and (unchanged) v to the
// token's slot. A row is read once and written once, so memory traffic bounds
// it. A lane holds two 16-byte pieces of a row chosen so that both members of
// every rotated pair are in it: pieces p and p + rot/2 for half-split pairs,
// neighbouring pieces otherwise. The rotation then needs no exchange between
// lanes, and only the norm's sum does.
#include "rf_device.cuh"

namespace rf {
namespace {

constexpr int kThreads = 256;

template <typename T>
struct Piece;  // 16 bytes of a row

template <>
struct Piece<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const float* p, float (&x)[N]) {
    const float4 v = *reinterpret_cast<const float4*>(p);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[N]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};

template <>
struct Piece<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const __nv_bfloat16* p, float (&x)[N]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[N]) {
    uint4 v;
    v.x = pack_bf16x2(x[0], x[1]);
    v.y = pack_bf16x2(x[2], x[3]);
    v.z = pack_bf16x2(x[4], x[5]);
    v.w = pack_bf16x2(x[6], x[7]);
    *reinterpret_cast<uint4*>(p) = v;
  }
};

// L lanes per row (a power of two >= pieces / 2).
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a, int64_t rows) {
  using P = Piece<T>;
  constexpr int N = P::N;
  const int lane = threadIdx.x & (L - 1);
  const int64_t row = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / L;
  // rows run token-major: H query heads (when q is given), then Hkv key heads
  // and Hkv value heads
  const int heads = a.H + 2 * a.Hkv;
  const bool live = row < rows;
  const int64_t t = live ? row / heads : 0;
  const int h = static_cast<int>(row - t * heads);
  const int64_t slot = live ? a.slots[t] : -1;
  bool ok = live && slot >= 0;
  if (ok && slot >= int64_t(a.num_pages) * a.page) {
    record_status(a.status, dev_code(kDevBadList, kKerAppend, 1));
    ok = false;
  }
  int pos = 0;
  if (ok && a.rot > 0) {
    pos = a.pos[t];
    if (pos < 0 || pos >= a.max_pos) {
      record_status(a.status, dev_code(kDevBadList, kKerAppend, 2));
      ok = false;
    }
  }
  const bool is_q = h < a.H, is_v = h >= a.H + a.Hkv;
  const int hk = is_q ? h : is_v ? h - a.H - a.Hkv : h - a.H;
  const T* src = static_cast<const T*>(is_q ? a.q : is_v ? a.v : a.k) +
                 t * (is_q ? a.q_stride : is_v ? a.v_stride : a.k_stride) + int64_t(hk) * a.d;
  T* dst;
  if (is_q) {
    dst = static_cast<T*>(a.q_out) + (t * a.H + hk) * a.d;
  } else {
    const int s = ok ? static_cast<int>(slot) : 0;
    dst = static_cast<T*>(is_v ? a.v_cache : a.k_cache) +
          (s / a.page) * (is_v ? a.v_page_stride : a.k_page_stride) +
          (s % a.page) * (is_v ? a.v_token_stride : a.k_token_stride) +
          hk * (is_v ? a.v_head_stride : a.k_head_stride);
  }
  // this lane's pieces c0, c1 and the first angle of each
  const int half = a.rot / 2;
  const int rot_lanes = a.rot / (2 * N);
  const bool mine = ok && lane < a.d / (2 * N);
  const bool split = !a.interleaved && lane < rot_lanes;
  const int c0 = split ? lane * N : 2 * lane * N;
  const int c1 = split ? c0 + half : c0 + N;
  float x0[N], x1[N];
#pragma unroll
  for (int i = 0; i < N; ++i) x0[i] = x1[i] = 0.f;
  if (mine) {
    P::load(src + c0, x0);
    P::load(src + c1, x1);
  }
  const T* w = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
  if (a.norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    if (mine && !is_v && w != nullptr) {
      const float r = 1.f / sqrtf(ss / a.d + a.eps);
      float w0[N], w1[N];
      P::load(w + c0, w0);
      P::load(w + c1, w1);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        x0[i] = x0[i] * r * w0[i];
        x1[i] = x1[i] * r * w1[i];
      }
    }
  }
  if (!mine) return;
  if (!is_v && lane < rot_lanes) {
    const float* cs = a.cos_sin + int64_t(pos) * a.rot;
    float c[N], s[N];
    const int a0 = split ? c0 : c0 / 2;  // N angles from here on
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 cv = *reinterpret_cast<const float4*>(cs + a0 + i);
      const float4 sv = *reinterpret_cast<const float4*>(cs + half + a0 + i);
      c[i] = cv.x; c[i + 1] = cv.y; c[i + 2] = cv.z; c[i + 3] = cv.w;
      s[i] = sv.x; s[i + 1] = sv.y; s[i + 2] = sv.z; s[i + 3] = sv.w;
    }
    if (split) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float u = x0[i], v = x1[i];
        x0[i] = u * c[i] - v * s[i];
        x1[i] = v * c[i] + u * s[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const float u = x0[2 * i], v = x0[2 * i + 1];
        x0[2 * i] = u * c[i] - v * s[i];
        x0[2 * i + 1] = v * c[i] + u * s[i];
        const float y = x1[2 * i], z = x1[2 * i + 1];
        x1[2 * i] = y * c[N / 2 + i] - z * s[N / 2 + i];
        x1[2 * i + 1] = z * c[N / 2 + i] + y * s[N / 2 + i];
      }
    }
  }
  P::store(dst + c0, x0);
  P::store(dst + c1, x1);
}

__global__ void paged_slots_kernel(const int32_t* __restrict__ cu_q,
                                   const int32_t* __restrict__ kv_len,
                                   const int32_t* __restrict__ table, int64_t table_stride, int B,
                                   int T, int max_pages, int page, int num_pages,
                                   int32_t* __restrict__ pos, int64_t* __restrict__ slots,
                                   int* status) {
  const int t = blockIdx.x * blockDim.x + threadIdx.x;
  if (t >= T) return;
  // the last b with cu_q[b] <= t; tokens outside every sequence get no slot
  int lo = 0, hi = B;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (cu_q[mid + 1] <= t) lo = mid + 1; else hi = mid;
  }
  int p = 0;
  int64_t slot = -1;
  if (lo < B && cu_q[lo] <= t) {
    const int n = cu_q[lo + 1] - cu_q[lo];
    const int at = kv_len[lo] - n + (t - cu_q[lo]);
    if (at >= 0) {
      p = at;
      const int pi = at / page;
      const int id = pi < max_pages ? table[int64_t(lo) * table_stride + pi] : -1;
      if (id >= 0 && id < num_pages)
        slot = int64_t(id) * page + at % page;
      else
        record_status(status, dev_code(kDevBadList, kKerAppend, 3));
    }
  }
  pos[t] = p;
  slots[t] = slot;
}

template <typename T, int L>
cudaError_t launch_l(const KvAppendArgs& a, cudaStream_t s) {
  const int64_t rows = int64_t(a.T) * (a.H + 2 * a.Hkv);
  const int64_t grid = (rows * L + kThreads - 1) / kThreads;
  if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  kv_append_kernel<T, L><<<static_cast<unsigned>(grid), kThreads, 0, s>>>(a, rows);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_t(const KvAppendArgs& a, cudaStream_t s) {
  const int need = a.d / (2 * Piece<T>::N);
  if (need <= 1) return launch_l<T, 1>(a, s);
  if (need <= 2) return launch_l<T, 2>(a, s);
  if (need <= 4) return launch_l<T, 4>(a, s);
  if (need <= 8) return launch_l<T, 8>(a, s);
  if (need <= 16) return launch_l<T, 16>(a, s);
  return launch_l<T, 32>(a, s);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs& a, rf_dtype dt, cudaStream_t s) {
  return dt == RF_F32 ? launch_t<float>(a, s) : launch_t<__nv_bfloat16>(a, s);
}

cudaError_t launch_paged_slots(const int32_t* cu_q, const int32_t* kv_len, const int32_t* table,
                               int64_t table_stride, int B, int T, int max_pages, int page,
                               int num_pages, int32_t* pos, int64_t* slots, cudaStream_t s,
                               int* status) {
  paged_slots_kernel<<<(T + 127) / 128, 128, 0, s>>>(cu_q, kv_len, table, table_stride, B, T,
                                                     max_pages, page, num_pages, pos, slots,
                                                     status);
  return cudaGetLastError();
}

}  // namespace rf
