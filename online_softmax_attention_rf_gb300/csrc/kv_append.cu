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
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[N]) {
    x[0] = __uint_as_float(v.x); x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z); x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[N]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};

template <>
struct Piece<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[N]) {
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

template <typename T>
__device__ __forceinline__ uint4 raw(const T* p) {
  return *reinterpret_cast<const uint4*>(p);
}

// L lanes per row (a power of two >= pieces / 2), kThreads / L rows at a time.
// A block takes one token: its slot, position, angles and norm weights are
// read once and stay in registers while the token's rows pass, kRows of them
// in flight per lane (the loads of all are issued before the first is used).
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) kv_append_kernel(const KvAppendArgs a) {
  using P = Piece<T>;
  constexpr int N = P::N;
  constexpr int kRows = 3;
  constexpr int kStep = kThreads / L;
  const int lane = threadIdx.x & (L - 1), first = threadIdx.x / L;
  const int t = blockIdx.x;
  // rows of a token: H query heads (when q is given), then Hkv key heads and
  // Hkv value heads
  const int heads = a.H + 2 * a.Hkv;
  const bool mine = lane < a.d / (2 * N);
  // this lane's pieces c0 and c1 of a row that is rotated, and of one that is not
  const int half = a.rot / 2;
  const int rot_lanes = a.rot / (2 * N);
  const bool rotates = lane < rot_lanes;
  const bool split = !a.interleaved && rotates;
  const int c0 = split ? lane * N : 2 * lane * N;
  const int c1 = split ? c0 + half : c0 + N;
  pdl_wait();
  pdl_trigger();
  const int64_t slot = a.slots[t];
  if (slot < 0) return;
  const int pos = a.rot > 0 ? a.pos[t] : 0;
  const bool bad_slot = slot >= int64_t(a.num_pages) * a.page;
  if (bad_slot || (a.rot > 0 && (pos < 0 || pos >= a.max_pos))) {
    if (threadIdx.x == 0)
      record_status(a.status, dev_code(kDevBadList, kKerAppend, bad_slot ? 1 : 2));
    return;
  }
  const int page = static_cast<int>(slot) / a.page, in_page = static_cast<int>(slot) - page * a.page;
  const T* q_row = static_cast<const T*>(a.q) + t * a.q_stride;
  const T* k_row = static_cast<const T*>(a.k) + t * a.k_stride;
  const T* v_row = static_cast<const T*>(a.v) + t * a.v_stride;
  T* q_to = static_cast<T*>(a.q_out) + int64_t(t) * a.H * a.d;
  T* k_to = static_cast<T*>(a.k_cache) + page * a.k_page_stride + in_page * a.k_token_stride;
  T* v_to = static_cast<T*>(a.v_cache) + page * a.v_page_stride + in_page * a.v_token_stride;
  float c[N], s[N];
  if (rotates) {
    const float* cs = a.cos_sin + int64_t(pos) * a.rot + (split ? c0 : c0 / 2);  // N angles
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 cv = *reinterpret_cast<const float4*>(cs + i);
      const float4 sv = *reinterpret_cast<const float4*>(cs + half + i);
      c[i] = cv.x; c[i + 1] = cv.y; c[i + 2] = cv.z; c[i + 3] = cv.w;
      s[i] = sv.x; s[i + 1] = sv.y; s[i + 2] = sv.z; s[i + 3] = sv.w;
    }
  }
  // every lane runs every round: the norm's sum is taken by whole warps
  for (int h0 = first; h0 - first < heads; h0 += kRows * kStep) {
    uint4 raw0[kRows], raw1[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int h = h0 + j * kStep;
      const T* src = h < a.H ? q_row + h * a.d
                             : h < a.H + a.Hkv ? k_row + (h - a.H) * a.d
                                               : v_row + (h - a.H - a.Hkv) * a.d;
      raw0[j] = raw1[j] = make_uint4(0, 0, 0, 0);
      if (mine && h < heads) {
        raw0[j] = raw(src + c0);
        raw1[j] = raw(src + c1);
      }
    }
#pragma unroll
    for (int j = 0; j < kRows; ++j) {
      const int h = h0 + j * kStep;
      const bool is_q = h < a.H, is_v = h >= a.H + a.Hkv;
      const T* w = static_cast<const T*>(is_q ? a.q_weight : a.k_weight);
      float x0[N], x1[N];
      P::unpack(raw0[j], x0);
      P::unpack(raw1[j], x1);
      if (a.norm) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < N; ++i) ss += x0[i] * x0[i] + x1[i] * x1[i];
#pragma unroll
        for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        if (mine && !is_v && w != nullptr) {
          const float r = 1.f / sqrtf(ss / a.d + a.eps);
          float w0[N], w1[N];
          P::unpack(raw(w + c0), w0);
          P::unpack(raw(w + c1), w1);
#pragma unroll
          for (int i = 0; i < N; ++i) {
            x0[i] = x0[i] * r * w0[i];
            x1[i] = x1[i] * r * w1[i];
          }
        }
      }
      if (!is_v && rotates) {
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
      if (mine && h < heads) {
        T* dst = is_q ? q_to + h * a.d
                      : is_v ? v_to + (h - a.H - a.Hkv) * a.v_head_stride
                             : k_to + (h - a.H) * a.k_head_stride;
        P::store(dst + c0, x0);
        P::store(dst + c1, x1);
      }
    }
  }
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
  return launch_pdl(kv_append_kernel<T, L>, dim3(static_cast<unsigned>(a.T)), dim3(kThreads), 0, s,
                    a);
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
