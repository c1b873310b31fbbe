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
// it, if enough reads are in flight and the arithmetic stays out of the way. A
// producer lane keeps a ring of 16 KB stages filled with bulk copies (the heads
// of a token lie back to back), and four warps take rows from it with packed
// float32 arithmetic: 56 us for 8192 tokens of 80 heads of 128, 6.04 TB/s, which
// is what the same kernel takes to copy the rows. (Rows loaded into registers by
// a block a token: 80 us, the reads in flight and the issue slots both short;
// eight consumer warps, whose registers spill at three CTAs an SM: 79 us, and 64
// at two.) A lane holds two 16-byte pieces of a row chosen so that both
// members of every rotated pair are in it: pieces p and p + rot/2 for half-split
// pairs, neighbouring pieces otherwise. The rotation then needs no exchange
// between lanes, and only the norm's sum does.
#include "paged_device.cuh"

namespace rf {
namespace {

constexpr int kWarps = 4;                       // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kStageBytes = 16384;
constexpr int kStages = 4;                      // three CTAs are resident per SM
constexpr int kMaxDim = 256;

// 16 bytes of a row as N / 2 pairs of float32.
template <typename T>
struct Piece;

template <>
struct Piece<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float2 (&x)[N / 2]) {
    x[0] = make_float2(__uint_as_float(v.x), __uint_as_float(v.y));
    x[1] = make_float2(__uint_as_float(v.z), __uint_as_float(v.w));
  }
  static __device__ __forceinline__ uint4 pack(const float2 (&x)[N / 2]) {
    return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x),
                      __float_as_uint(x[1].y));
  }
};

template <>
struct Piece<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ void unpack(const uint4& v, float2 (&x)[N / 2]) {
    x[0] = two(v.x); x[1] = two(v.y); x[2] = two(v.z); x[3] = two(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float2 (&x)[N / 2]) {
    return make_uint4(pack_bf16x2(x[0].x, x[0].y), pack_bf16x2(x[1].x, x[1].y),
                      pack_bf16x2(x[2].x, x[2].y), pack_bf16x2(x[3].x, x[3].y));
  }
};

// What a stage holds: rows of one kind of one token, and where they go.
enum Kind : int { kQ = 0, kK = 1, kV = 2, kEnd = 3 };
struct Unit {
  char* dst;
  int64_t stride;  // bytes between rows there
  int rows, kind;
};

struct Smem {
  alignas(128) unsigned char rows[kStages][kStageBytes];
  alignas(16) float cs[kStages][kMaxDim];   // the token's cosines, then its sines
  alignas(16) unsigned char w[2][kMaxDim * 4];  // norm weights of q and k
  Unit unit[kStages];
  uint64_t full[kStages];
  uint64_t empty[kStages];
  int abort_flag;
};

// L lanes per row (a power of two >= pieces / 2), kWarps * 32 / L rows at a time.
template <typename T, int L, bool kNorm, bool kInter>
__global__ void __launch_bounds__(kThreads, 3) kv_append_kernel(const KvAppendArgs a) {
  using P = Piece<T>;
  constexpr int N = P::N, N2 = N / 2;
  extern __shared__ unsigned char smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 127) & ~uintptr_t(127));
  const int warp = threadIdx.x >> 5, lane32 = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kWarps);
    }
    sm.abort_flag = 0;
    fence_barrier_init();
  }
  pdl_wait();
  pdl_trigger();
  if constexpr (kNorm) {
    for (int i = threadIdx.x; i < 2 * a.d; i += kThreads) {
      const T* w = static_cast<const T*>(i < a.d ? a.q_weight : a.k_weight);
      const int e = i < a.d ? i : i - a.d;
      if (w != nullptr) reinterpret_cast<T*>(sm.w[i < a.d ? 0 : 1])[e] = w[e];
    }
  }
  __syncthreads();

  if (warp == kWarps) {
    // ---------------- producer: this block's tokens, 32 slots and positions at a time
    int n = 0;  // units put into the ring
    bool ok = true;
    const int row_bytes = a.d * static_cast<int>(sizeof(T));
    const int chunk = kStageBytes / row_bytes;  // rows a stage holds
    // heads [0, heads) from src to dst, in chunks (lane 0)
    const uint64_t stream = policy_evict_first(), keep = policy_evict_last();
    auto put = [&](int kind, const void* src, void* dst, int64_t stride, int heads, int pos) {
      for (int h = 0; ok && h < heads; h += chunk, ++n) {
        const int s = n % kStages, rows = min(chunk, heads - h);
        ok = mbar_wait(&sm.empty[s], ((n / kStages) & 1) ^ 1, a.status,
                       dev_code(kDevTimeout, kKerAppend, 10), &sm.abort_flag);
        if (!ok) return;
        sm.unit[s] = Unit{static_cast<char*>(dst) + h * stride, stride, rows, kind};
        const uint32_t bytes = static_cast<uint32_t>(rows) * row_bytes;
        const uint32_t cs_bytes = kind != kV ? static_cast<uint32_t>(a.rot) * 4 : 0;
        mbar_arrive_expect_tx(&sm.full[s], bytes + cs_bytes);
        bulk_load(sm.rows[s], static_cast<const char*>(src) + int64_t(h) * row_bytes, bytes,
                  &sm.full[s], stream);
        if (cs_bytes > 0)
          bulk_load(sm.cs[s], a.cos_sin + int64_t(pos) * a.rot, cs_bytes, &sm.full[s],
                    keep);
      }
    };
    for (int64_t base = blockIdx.x; ok && base < a.T; base += int64_t(32) * gridDim.x) {
      const int64_t mine = base + int64_t(lane32) * gridDim.x;
      int64_t slot = mine < a.T ? a.slots[mine] : -1;
      int pos = mine < a.T && a.rot > 0 ? a.pos[mine] : 0;
      const bool bad_slot = slot >= int64_t(a.num_pages) * a.page;
      const bool bad_pos = slot >= 0 && a.rot > 0 && (pos < 0 || pos >= a.max_pos);
      if (bad_slot || bad_pos) {
        record_status(a.status, dev_code(kDevBadList, kKerAppend, bad_slot ? 1 : 2));
        slot = -1;
      }
      for (int i = 0; i < 32 && base + int64_t(i) * gridDim.x < a.T; ++i) {
        const int64_t sl = __shfl_sync(0xffffffffu, slot, i);
        const int po = __shfl_sync(0xffffffffu, pos, i);
        if (sl < 0 || lane32 != 0 || !ok) continue;
        const int64_t t = base + int64_t(i) * gridDim.x;
        const int page = static_cast<int>(sl) / a.page;
        const int in_page = static_cast<int>(sl) - page * a.page;
        if (a.H > 0)
          put(kQ, static_cast<const T*>(a.q) + t * a.q_stride,
              static_cast<T*>(a.q_out) + t * a.H * a.d, row_bytes, a.H, po);
        put(kK, static_cast<const T*>(a.k) + t * a.k_stride,
            static_cast<T*>(a.k_cache) + page * a.k_page_stride + in_page * a.k_token_stride,
            a.k_head_stride * static_cast<int64_t>(sizeof(T)), a.Hkv, po);
        put(kV, static_cast<const T*>(a.v) + t * a.v_stride,
            static_cast<T*>(a.v_cache) + page * a.v_page_stride + in_page * a.v_token_stride,
            a.v_head_stride * static_cast<int64_t>(sizeof(T)), a.Hkv, po);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
    if (lane32 == 0) {
      const int s = n % kStages;
      int oldest = max(0, n - kStages);
      if (ok && mbar_wait(&sm.empty[s], ((n / kStages) & 1) ^ 1, a.status,
                          dev_code(kDevTimeout, kKerAppend, 11), &sm.abort_flag)) {
        sm.unit[s].kind = kEnd;
        mbar_arrive(&sm.full[s]);
        // the end took over the stage of unit n - kStages, which was consumed;
        // that stage's barrier is a phase further now
        oldest = max(0, n - kStages + 1);
      }
      // never leave with copies in flight
      for (int u = oldest; u < n; ++u)
        mbar_wait(&sm.full[u % kStages], (u / kStages) & 1, a.status,
                  dev_code(kDevTimeout, kKerAppend, 12), nullptr);
    }
    return;
  }

  // ---------------- consumers
  const int lane = threadIdx.x & (L - 1);
  constexpr int kStep = kWarps * 32 / L;
  const bool mine = lane < a.d / (2 * N);
  // this lane's pieces c0 and c0 + c1 of a row that is rotated, and of one that is not
  const int half = a.rot / 2;
  const bool rotates = lane < a.rot / (2 * N);
  const bool split = !kInter && rotates;
  const int c0 = split ? lane * N : 2 * lane * N;
  const int c1 = split ? half : N;
  const float inv_d = 1.f / a.d;
  for (int n = 0;; ++n) {
    const int st = n % kStages;
    if (!mbar_wait_warp(&sm.full[st], (n / kStages) & 1, a.status,
                        dev_code(kDevTimeout, kKerAppend, 13), &sm.abort_flag))
      break;
    const Unit u = sm.unit[st];
    if (u.kind == kEnd) break;
    // a unit of few rows keeps few warps busy: other ones each time
    const int vwarp = (warp + 3 * n) & (kWarps - 1);
    const int first = (vwarp * 32 + lane32) / L, warp_first = vwarp * 32 / L;
    const T* src = reinterpret_cast<const T*>(sm.rows[st]) + c0;
    char* const dst = u.dst + c0 * sizeof(T);
    if (u.kind == kV) {
      for (int r = first; r < u.rows; r += kStep) {
        if (!mine) continue;
        const uint4 x = *reinterpret_cast<const uint4*>(src + r * a.d);
        const uint4 y = *reinterpret_cast<const uint4*>(src + r * a.d + c1);
        *reinterpret_cast<uint4*>(dst + r * u.stride) = x;
        *reinterpret_cast<uint4*>(dst + r * u.stride + c1 * sizeof(T)) = y;
      }
    } else {
      const bool norm = kNorm && (u.kind == kQ ? a.q_weight : a.k_weight) != nullptr;
      const T* w = reinterpret_cast<const T*>(sm.w[u.kind]) + c0;
      uint4 w0 = make_uint4(0, 0, 0, 0), w1 = w0;
      if (norm && mine) {
        w0 = *reinterpret_cast<const uint4*>(w);
        w1 = *reinterpret_cast<const uint4*>(w + c1);
      }
      float2 c[N2], s[N2];
      if (rotates) {
        const float* cs = sm.cs[st] + (split ? c0 : c0 / 2);  // N angles
#pragma unroll
        for (int i = 0; i < N2; i += 2) {
          const float4 cv = *reinterpret_cast<const float4*>(cs + 2 * i);
          const float4 sv = *reinterpret_cast<const float4*>(cs + half + 2 * i);
          c[i] = make_float2(cv.x, cv.y);
          c[i + 1] = make_float2(cv.z, cv.w);
          s[i] = make_float2(sv.x, sv.y);
          s[i + 1] = make_float2(sv.z, sv.w);
        }
      }
      // whole warps go round: the norm's sum is taken by all their lanes
#pragma unroll 2
      for (int r0 = 0; r0 + warp_first < u.rows; r0 += kStep) {
        const int r = r0 + first;
        const bool live = mine && r < u.rows;
        uint4 raw0 = make_uint4(0, 0, 0, 0), raw1 = raw0;
        if (live) {
          raw0 = *reinterpret_cast<const uint4*>(src + r * a.d);
          raw1 = *reinterpret_cast<const uint4*>(src + r * a.d + c1);
        }
        float2 x0[N2], x1[N2];
        P::unpack(raw0, x0);
        P::unpack(raw1, x1);
        if (norm) {
          float2 s2 = __fmul2_rn(x0[0], x0[0]);
#pragma unroll
          for (int i = 1; i < N2; ++i) s2 = ffma2(x0[i], x0[i], s2);
#pragma unroll
          for (int i = 0; i < N2; ++i) s2 = ffma2(x1[i], x1[i], s2);
          float ss = s2.x + s2.y;
#pragma unroll
          for (int o = L / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float q = rsqrtf(ss * inv_d + a.eps);
          const float2 qq = make_float2(q, q);
          float2 y[N2];
          P::unpack(w0, y);
#pragma unroll
          for (int i = 0; i < N2; ++i) x0[i] = __fmul2_rn(__fmul2_rn(x0[i], qq), y[i]);
          P::unpack(w1, y);
#pragma unroll
          for (int i = 0; i < N2; ++i) x1[i] = __fmul2_rn(__fmul2_rn(x1[i], qq), y[i]);
        }
        if (rotates) {
          if constexpr (!kInter) {
#pragma unroll
            for (int i = 0; i < N2; ++i) {
              const float2 y = x0[i], z = x1[i];
              const float2 zs = __fmul2_rn(z, s[i]);
              x0[i] = ffma2(y, c[i], make_float2(-zs.x, -zs.y));
              x1[i] = ffma2(z, c[i], __fmul2_rn(y, s[i]));
            }
          } else {
            // neighbours: (y, z) -> (y c - z s, z c + y s), one angle a pair
            auto turn = [](float2 p, float co, float si) {
              return make_float2(fmaf(p.x, co, -(p.y * si)), fmaf(p.y, co, p.x * si));
            };
#pragma unroll
            for (int i = 0; i < N2; ++i) {
              const float2 ca = c[i / 2], sa = s[i / 2];
              const float2 cb = c[N2 / 2 + i / 2], sb = s[N2 / 2 + i / 2];
              x0[i] = (i & 1) ? turn(x0[i], ca.y, sa.y) : turn(x0[i], ca.x, sa.x);
              x1[i] = (i & 1) ? turn(x1[i], cb.y, sb.y) : turn(x1[i], cb.x, sb.x);
            }
          }
        }
        if (live) {
          *reinterpret_cast<uint4*>(dst + r * u.stride) = P::pack(x0);
          *reinterpret_cast<uint4*>(dst + r * u.stride + c1 * sizeof(T)) = P::pack(x1);
        }
      }
    }
    __syncwarp();
    if (lane32 == 0) mbar_arrive(&sm.empty[st]);
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

template <typename T, int L, bool kNorm, bool kInter>
cudaError_t launch_v(const KvAppendArgs& a, cudaStream_t s) {
  constexpr int smem = sizeof(Smem) + 128;
  cudaError_t e = cudaFuncSetAttribute(kv_append_kernel<T, L, kNorm, kInter>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int grid = a.T < 3 * 152 ? a.T : 3 * 152;
  return launch_pdl(kv_append_kernel<T, L, kNorm, kInter>, dim3(static_cast<unsigned>(grid)),
                    dim3(kThreads), smem, s, a);
}

template <typename T, int L>
cudaError_t launch_l(const KvAppendArgs& a, cudaStream_t s) {
  if (a.norm) return a.interleaved ? launch_v<T, L, true, true>(a, s) : launch_v<T, L, true, false>(a, s);
  return a.interleaved ? launch_v<T, L, false, true>(a, s) : launch_v<T, L, false, false>(a, s);
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
