// attn_paged.cu -- attention of a ragged batch's new tokens over a paged
// key/value cache, on the tcgen05 tensor cores.
//
// The cascade max -> sum exp -> normalised P.V in the incremental form of
// attn_tc.cu (RedFuser: An Automatic Operator Fusion Framework for Cascaded
// Reductions on AI Accelerators, section 2), with the multi-segment strategy
// of section 3 across CTAs. Differences that the paged cache and the ragged
// batch ask for:
//  - Query rows are packed: the G query heads of one key head at one token are
//    G neighbouring rows, so that a tile of 128 rows holds floor(128 / G)
//    tokens and the keys of a group are read once for all its heads. A decode
//    step is a tile with G live rows, drafted tokens one with a few times G.
//  - Work is dealt by the step's plan (paged_plan.h): one persistent CTA per
//    span of key tiles. A whole item is written by the CTA itself; a part goes
//    to the workspace and attn_paged_merge joins the parts by log-sum-exp.
//  - A key tile of 128 keys comes in boxes of R = gcd(page, 128) rows, one TMA
//    copy per box and 64 columns, each lane of a producer warp looking up one
//    box's page. A page of 16 takes 32 copies a step; one warp's issue of them
//    would bound a decode step at 5.5 TB/s, so K and V have a producer each.
//    Boxes that start past the cache's end are not copied; the rows of V between
//    the end and the tile's edge are zeroed in shared memory before P.V (their
//    weights are 0, but 0 * NaN is not).
//  - An item of one tile (up to 128 packed rows) is either split: both softmax
//    groups take alternate key tiles and join their states at the end (with one
//    group the chain Q K^T -> softmax -> P.V of a tile would not keep up with
//    memory); or, when it is short, solo: the groups take whole items in turn,
//    and one's epilogue runs under the other's softmax.
//
// Roles of the 384 threads: warps 0-3 and 4-7 softmax groups, warp 8 walks the
// span, publishes a descriptor of each segment (an item or a part of one) and
// copies Q and K, warp 11 copies V, warps 9 and 10 issue the two groups' MMAs.
// Tensor memory, the lock and the reuse of S by P are those of attn_tc.cu.
// Every wait is bounded; on expiry the kernel records a status code and the CTA
// unwinds, the five warps of a group together at a reducing named barrier.
//
// Measured: decode of 8 sequences x 8 key heads x 65536 keys 6.74 TB/s of cache
// at d = 128 (pages of 16 to 128) and 5.64 at d = 64, memory and the chain
// scores -> softmax -> P.V of a one-tile step bounding them; a chunk of 2048
// tokens at 32768 keys, 64 heads, d = 128, 1.38 to 1.52 ms (1547 to 1400
// TFLOP/s), bound as attn_tc.cu is; one token over 515 keys 12.7 us, launches
// and dependent loads.
//
// P is rounded to bf16 for the tensor cores (scores, maxima, sums and
// accumulators stay in float32): half a step, 2^-8, of each weight. The row
// sum takes the unrounded weights.
#include <cudaTypedefs.h>

#include <mutex>

#include "paged_plan.h"
#include "paged_device.cuh"

namespace rf {
namespace {

constexpr float kRescaleThreshold = 8.0f;  // log2 units: rescale when the max grows > 256x
constexpr int kBM = kPlanTile;             // packed query rows per tile
constexpr int kBN = kPlanTile;             // keys per tile
constexpr int kThreads = 384;
constexpr int kWarpK = 8;                  // spans, Q, K; TMEM allocator
constexpr int kWarpIssue = 9;              // warps 9 and 10
constexpr int kWarpV = 11;
constexpr int kSegs = 4;                   // segment descriptors in flight
constexpr int kSoloSteps = 4;              // a one-tile segment up to this long is solo
constexpr int kChunk = 16384;              // one 128-row x 64-column bf16 swizzle block

template <int D>
struct Layout {
  static constexpr int kTileBytes = kBM * D * 2;
  // Two rings, of K and of V tiles, as many slots as fit. One ring of five for
  // both (d = 128) was not sound: behind a K producer that is late, a table
  // entry coming from memory, the V producer would wait for a phase two ahead of
  // the slot's barrier, and the parity of that wait passes at once
  // (tests/test_paged_protocol.py). With a wait for the K tile it cost 2 % of a
  // chunk. Measured before the issuers' release and test became one walk: 2 + 3
  // slots: 2048 tokens at 32768 keys 1.41 ms, 3 + 2: 1.45, one ring of 5: 1.43.
  // d = 64, 8 x 8 heads of 65536 keys: 6 + 6 slots 5.39 TB/s (5.64 since), 4 + 8
  // 5.22, 5 + 7 5.19, 4 + 4 5.09.
  static constexpr int kSlotsK = (D == 128) ? 2 : 6;
  static constexpr int kSlotsV = (D == 128) ? 3 : 6;
  static constexpr int kStages = kSlotsK + kSlotsV;
  static constexpr int kOffQ = 0;
  static constexpr int kOffKV = kOffQ + 2 * kTileBytes;
  static constexpr int kOffBar = kOffKV + kStages * kTileBytes;
  static constexpr int kBarBytes = 640;
  static constexpr int kOffXch = kOffBar + kBarBytes;  // group 1's m and l for group 0
  static constexpr int kXchBytes = 2 * kBM * 4;
  static constexpr int kBytes = kOffXch + kXchBytes + 1024;  // + alignment slack
  static constexpr uint32_t kTmemS = 0;
  static constexpr uint32_t kTmemO = 2 * kBN;
  __host__ __device__ static constexpr uint32_t tmem_p(int t) {
    return D == 128 ? kTmemS + t * kBN : kTmemO + 2 * D + t * 64;
  }
};

// One CTA's part of one item: steps [kb, ke). Group t's query tile is t in a
// pair and 0 otherwise; its steps are the first n[t] (pair), every second one
// from kb + t on (split), or all or none (solo).
enum SegMode : int { kPair = 0, kSplit = 1, kSolo0 = 2, kSolo1 = 3 };
struct Seg {
  int seq;         // -1: the span's end
  int head;
  int row0, ntok;  // the item's first token among the packed tokens, and its tokens
  int kv;          // cached tokens of the sequence
  int lim0;        // keys that the item's first token sees (may be below 0; kv when not causal)
  int kb, ke;
  int n[2];
  int slot;        // partial slot, -1: the whole item
  int mode;
  int q;           // Q ring number of the first tile
  int pad[3];
};
static_assert(sizeof(Seg) == 64, "descriptor size");

// The slots of a step's K and V tiles and the parities of their uses, carried
// from step to step: the division that slot n % kSlotsK asks for is on the
// issuers' path.
template <int D>
struct Slots {
  int k = 0, v = Layout<D>::kSlotsK;
  uint32_t kp = 0, vp = 0;
  __device__ __forceinline__ void next() {
    if (++k == Layout<D>::kSlotsK) {
      k = 0;
      kp ^= 1;
    }
    if (++v == Layout<D>::kStages) {
      v = Layout<D>::kSlotsK;
      vp ^= 1;
    }
  }
};

struct Bars {
  Seg seg[kSegs];
  uint64_t seg_full[kSegs];
  uint64_t seg_empty[kSegs];
  uint64_t kv_full[12];
  uint64_t kv_empty[12];
  uint64_t q_full[2];
  uint64_t q_empty[2];
  uint64_t s_full[2];
  uint64_t o_done[2];
  uint64_t mma_idle[2];
  uint64_t split_ready;
  uint64_t split_read;
  uint32_t tmem_base;
  int abort_flag;
  int issue_lock;
};
static_assert(sizeof(Bars) <= Layout<64>::kBarBytes && sizeof(Bars) <= Layout<128>::kBarBytes,
              "barrier block overflows its shared-memory slot");
static_assert(Layout<64>::kBytes <= 227 * 1024 && Layout<128>::kBytes <= 227 * 1024,
              "attention shared memory exceeds a CTA's limit");

struct Params {
  const PlanHeader* plan;
  const int32_t* table;
  int64_t table_stride;
  int B, T, H, Hkv, page, max_pages, num_pages;
  int G, tt;            // heads of a group, tokens of a tile
  int box;              // rows of one copied box
  int k_token_first, v_token_first;  // the map's dimension 1 is the token (else the head)
  float scale_log2;
  __nv_bfloat16* o;
  float* lse;
  int o_wide;       // o is 32-byte aligned
  // Partial states. A slot holds two tiles; O of a tile is stored by groups of
  // four columns, [D / 4][128 rows][4], so that the warp that owns 32 rows
  // writes 512 contiguous bytes at a time (a row-major tile would take 32
  // half-written sectors a store: 8 us a pair of tiles).
  float* o_part;    // [2 * kPlanCtas][2][D / 4][128][4]
  float* lse_part;  // [2 * kPlanCtas][2][128]
  int* status;
};

__device__ __forceinline__ bool plan_matches(const PlanHeader* h, const Params& p) {
  return h->magic == kPlanMagic && h->B == p.B && h->T == p.T && h->H == p.H && h->Hkv == p.Hkv &&
         h->page == p.page && h->max_pages == p.max_pages;
}

__device__ __forceinline__ bool same_item(const PlanStart& a, const PlanStart& b) {
  return a.seq == b.seq && a.head == b.head && a.pair == b.pair;
}

// Walks a CTA's span (the K producer warp, all lanes alike). The next
// sequence's lengths are on their way while the current one is worked on.
struct Span {
  PlanStart cur, end;
  const int32_t* cu;
  const int32_t* kvl;
  int B, Hkv, tt, causal;
  int t0, t1, kv, t2, kv1;  // cu[seq], cu[seq + 1], kvl[seq], and the next ones
  int q, solo;              // Q ring numbers and solo segments handed out

  __device__ __forceinline__ void fetch() {
    t2 = cu[min(cur.seq + 2, B)];
    kv1 = kvl[min(cur.seq + 1, B - 1)];
  }
  __device__ __forceinline__ void init(const Params& p, const PlanStart& first,
                                       const PlanStart& last) {
    cur = first;
    end = last;
    cu = plan_cu_q(p.plan);
    kvl = plan_kv_len(p.plan, p.B);
    B = p.B;
    Hkv = p.Hkv;
    tt = p.tt;
    causal = p.plan->causal;
    q = solo = 0;
    if (cur.seq < B) {
      t0 = cur.row0;
      t1 = cur.row1;
      kv = cur.kv;
      fetch();
    }
  }
  __device__ __forceinline__ bool next(Seg& s) {
    if (cur.seq >= B || (same_item(cur, end) && cur.step == end.step)) {
      s = Seg{};
      s.seq = -1;
      return false;
    }
    const int n = t1 - t0, tok0 = cur.pair * 2 * tt;
    s.seq = cur.seq;
    s.head = cur.head;
    s.ntok = min(2 * tt, n - tok0);
    s.row0 = t0 + tok0;
    s.kv = kv;
    s.lim0 = causal ? kv - n + tok0 + 1 : kv;
    const int steps = steps_of(s.ntok - 1, s);
    s.kb = cur.step;
    const int cta = static_cast<int>(blockIdx.x);
    if (same_item(cur, end)) {
      s.ke = min(steps, end.step);
      cur = end;
    } else {
      s.ke = steps;
      cur.step = 0;
      if (tok0 + s.ntok < n) {
        ++cur.pair;
      } else {
        cur.pair = 0;
        if (++cur.head == Hkv) {
          cur.head = 0;
          do {
            ++cur.seq;
            t0 = t1;
            t1 = t2;
            kv = kv1;
            if (cur.seq < B) fetch();
          } while (cur.seq < B && t1 == t0);
        }
      }
    }
    s.slot = s.kb > 0 ? 2 * cta : s.ke < steps ? 2 * cta + 1 : -1;
    const int len = s.ke - s.kb;
    const bool last = cur.seq >= B || (same_item(cur, end) && cur.step == end.step);
    s.q = q;
    if (s.ntok > tt) {
      s.mode = kPair;
      s.n[0] = max(0, min(s.ke, steps_of(tt - 1, s)) - s.kb);
      s.n[1] = len;
      q += len > 0 ? 2 : 0;
    } else {
      if (len > kSoloSteps || last) {
        s.mode = kSplit;
        s.n[0] = (len + 1) / 2;
        s.n[1] = len / 2;
      } else {
        const int t = solo++ & 1;
        s.mode = kSolo0 + t;
        s.n[0] = t == 0 ? len : 0;
        s.n[1] = t == 1 ? len : 0;
      }
      q += len > 0 ? 1 : 0;
    }
    return true;
  }
  // Steps that the item's token i needs.
  __device__ __forceinline__ int steps_of(int i, const Seg& s) const {
    return plan_steps(causal ? max(0, s.lim0 + i) : s.kv);
  }
};

// Named barrier of one group -- its four softmax warps and its issuer warp --
// that also ORs a predicate over the group: after each step's P, and once at the
// end of the span. A warp that fails calls it once with true and leaves, and the
// others leave at whichever of their calls it meets. Every warp thus makes its
// last call together with the four others, and none waits at a barrier that the
// rest have abandoned.
__device__ __forceinline__ bool group_sync_or(int t, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, 160, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "r"(1 + t)
      : "memory");
  return r != 0;
}

// The MMA issue lock (attn_tc.cu): a block of MMAs reaches the pipe whole.
__device__ __forceinline__ bool issue_lock(int* lk, int* status, int code,
                                           volatile int* abort_flag) {
  if (atomicCAS(lk, 0, 1) == 0) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    __nanosleep(32);
    if (atomicCAS(lk, 0, 1) == 0) return true;
    if (*abort_flag || globaltimer_ns() - t0 > RF_WAIT_LIMIT_NS) {
      record_status(status, code);
      *abort_flag = 1;
      return false;
    }
  }
}
__device__ __forceinline__ void issue_unlock(int* lk) { atomicExch(lk, 0); }

template <int D>
__device__ __forceinline__ void issue_qk(uint32_t tm_s, uint64_t q_desc, uint64_t k_desc) {
  constexpr uint32_t idesc = idesc_bf16_f32(kBM, kBN, 0);
#pragma unroll
  for (int kk = 0; kk < D / 16; ++kk) {
    const uint64_t off = static_cast<uint64_t>(((kk >> 2) * kChunk + (kk & 3) * 32) >> 4);
    mma_bf16(tm_s, q_desc + off, k_desc + off, idesc, kk > 0 ? 1u : 0u);
  }
}

template <int D>
__device__ __forceinline__ void issue_pv(uint32_t tm_o, uint32_t tm_p, uint64_t v_desc,
                                         bool accumulate) {
  constexpr uint32_t idesc = idesc_bf16_f32(kBM, D, 1);
#pragma unroll
  for (int kk = 0; kk < kBN / 16; ++kk) {
    const uint64_t off = static_cast<uint64_t>((kk * 16 * 128) >> 4);
    mma_bf16_ts(tm_o, tm_p + kk * 8, v_desc + off, idesc, (kk > 0 || accumulate) ? 1u : 0u);
  }
}

// Where a packed row's result goes: O and LSE of the call, or a partial slot.
struct RowOut {
  __nv_bfloat16* o;
  float* part;  // the row's first four columns; the next four are 4 * kBM floats on
  float* lse;
};

template <int D>
__device__ __forceinline__ RowOut row_out(const Params& p, const Seg& s, int t, int r, int row_tok,
                                          int row_head) {
  RowOut w{nullptr, nullptr, nullptr};
  if (s.slot >= 0) {
    const int64_t tile = int64_t(s.slot) * 2 + t;
    w.part = p.o_part + (tile * (D / 4) * kBM + r) * 4;
    w.lse = p.lse_part + tile * kBM + r;
  } else {
    const int64_t row = int64_t(s.row0 + t * p.tt + row_tok) * p.H + (s.head * p.G + row_head);
    w.o = p.o + row * D;
    w.lse = p.lse != nullptr ? p.lse + row : nullptr;
  }
  return w;
}

// 16 columns of a row of O.
__device__ __forceinline__ void put_bf16x16(__nv_bfloat16* o, const float* v, int wide) {
  uint32_t x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = pack_bf16x2(v[2 * e], v[2 * e + 1]);
  if (wide) {
    st_global_v8(o, x);
  } else {
    *reinterpret_cast<uint4*>(o) = make_uint4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<uint4*>(o + 8) = make_uint4(x[4], x[5], x[6], x[7]);
  }
}

// 32 columns of a finished row from column c on.
__device__ __forceinline__ void put32(const RowOut& w, int c, const float (&v)[32], int wide) {
  if (w.part != nullptr) {
#pragma unroll
    for (int e = 0; e < 32; e += 4)
      *reinterpret_cast<float4*>(w.part + (c + e) * kBM) =
          make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
  } else {
    put_bf16x16(w.o + c, v, wide);
    put_bf16x16(w.o + c + 16, v + 16, wide);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_paged_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using L = Layout<D>;
  constexpr int NS = L::kStages;
  extern __shared__ unsigned char smem_raw[];
  unsigned char* smem = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars& bar = *reinterpret_cast<Bars*>(smem + L::kOffBar);
  const uint32_t s_base = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&bar.seg_full[i], 1);
      mbar_init(&bar.seg_empty[i], 11);  // softmax and issuer warps, V producer
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(&bar.kv_full[i], 1);
      mbar_init(&bar.kv_empty[i], 2);  // one release per softmax group
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bar.q_full[t], 1);
      mbar_init(&bar.q_empty[t], 2);   // one release per softmax group
      mbar_init(&bar.s_full[t], 1);
      mbar_init(&bar.o_done[t], 1);
      mbar_init(&bar.mma_idle[t], 1);
    }
    mbar_init(&bar.split_ready, 4);
    mbar_init(&bar.split_read, 4);
    bar.abort_flag = 0;
    bar.issue_lock = 0;
    fence_barrier_init();
  }
  if (warp == kWarpK) {
    tmem_alloc(&bar.tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == kWarpK && lane == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = bar.tmem_base;
  // Up to here nothing of the call's memory was read or written. The plan's
  // header and this CTA's starts are read together.
  pdl_wait();
  pdl_trigger();
  const PlanStart first = p.plan->start[blockIdx.x], last = p.plan->start[blockIdx.x + 1];
  const bool matches = plan_matches(p.plan, p);
  if (!matches && blockIdx.x == 0 && threadIdx.x == 0)
    record_status(p.status, dev_code(kDevBadList, kKerPaged, 2));
  const bool busy = matches && static_cast<int>(blockIdx.x) < p.plan->ctas;
  volatile int* abort_flag = &bar.abort_flag;
#define RF_WAIT(b, par, site)                                                         \
  mbar_wait(&bar.b, (par), p.status, dev_code(kDevTimeout, kKerPaged, site), abort_flag)
#define RF_WAIT_WARP(b, par, site)                                                    \
  mbar_wait_warp(&bar.b, (par), p.status, dev_code(kDevTimeout, kKerPaged, site), abort_flag)

  if (!busy) {
    // no span
  } else if (warp == kWarpK || warp == kWarpV) {
    // ------------------------------------------------------------ producers
    // K producer, per segment: the first K tile, then Q (once the Q ring has
    // room: after the second K tile at the latest), then the other K tiles. It
    // publishes each segment while it works on the one before. Lane l copies
    // box l % boxes, columns 64 (l / boxes) .. + 63, of a tile.
    const bool is_k = warp == kWarpK;
    const CUtensorMap* map = is_k ? &tm_k : &tm_v;
    const bool token_first = is_k ? p.k_token_first : p.v_token_first;
    const int boxes = kBN / p.box;
    const int my_key = lane % boxes * p.box, my_chunk = lane / boxes;
    const bool has_box = my_chunk < D / 64;
    unsigned char* const my_dst = smem + L::kOffKV + my_chunk * kChunk + my_key * 128;
    int step = 0;               // steps copied
    Slots<D> at;
    int q_loads = 0;
    bool ok = true;
    // this lane's page of step u of a segment and the box's first row in it
    auto page_of = [&](const Seg& s, int u, int& in_page) -> int {
      in_page = 0;
      if (u >= s.ke || !has_box) return -1;
      const int key = u * kBN + my_key;
      if (key >= s.kv) return -1;
      const int pi = key / p.page;
      in_page = key - pi * p.page;
      return p.table[int64_t(s.seq) * p.table_stride + pi];
    };
    Span span;
    Seg s, nxt;
    int id = -1, in_page = 0;
    auto publish = [&](int k, const Seg& d) {
      if (lane == 0) {
        ok = RF_WAIT(seg_empty[k % kSegs], ((k / kSegs) & 1) ^ 1, 14);
        if (ok) {
          bar.seg[k % kSegs] = d;
          mbar_arrive(&bar.seg_full[k % kSegs]);
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    };
    if (is_k) {
      span.init(p, first, last);
      span.next(s);
      publish(0, s);
      if (s.seq >= 0) id = page_of(s, s.kb, in_page);
    }
    for (int k = 0; ok; ++k) {
      int id_seg = -1, in_seg = 0;  // the next segment's first page
      if (is_k) {
        if (s.seq < 0) break;
        span.next(nxt);
        publish(k + 1, nxt);
        if (!ok) break;
        if (nxt.seq >= 0) id_seg = page_of(nxt, nxt.kb, in_seg);
      } else {
        ok = RF_WAIT_WARP(seg_full[k % kSegs], (k / kSegs) & 1, 15);
        if (!ok) break;
        s = bar.seg[k % kSegs];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.seg_empty[k % kSegs]);
        if (s.seq < 0) break;
        id = page_of(s, s.kb, in_page);
      }
      bool q_due = is_k && s.ke > s.kb;
      for (int u = s.kb; ok && u < s.ke; ++u, ++step, at.next()) {
        int in_next = 0;
        const int id_next = page_of(s, u + 1, in_next);
        const bool mine = has_box && u * kBN + my_key < s.kv;
        if (mine && (id < 0 || id >= p.num_pages)) {
          record_status(p.status, dev_code(kDevBadList, kKerPaged, 3));
          id = p.num_pages;  // past the pool: the copy fills with zeros
        }
        const int slot = is_k ? at.k : at.v;
        if (lane == 0) {
          const int n_box = (min(kBN, s.kv - u * kBN) + p.box - 1) / p.box;
          ok = RF_WAIT(kv_empty[slot], (is_k ? at.kp : at.vp) ^ 1, 10);
          if (ok) mbar_arrive_expect_tx(&bar.kv_full[slot], n_box * p.box * D * 2);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (mine)
          tma_load_4d(my_dst + slot * L::kTileBytes, map, &bar.kv_full[slot], my_chunk * 64,
                      token_first ? in_page : s.head, token_first ? s.head : in_page, id);
        if (q_due && lane == 0) {
          const int tiles = s.mode == kPair ? 2 : 1;
          // the ring has two tiles: the last number's release is the later one
          const int lq = s.q + tiles - 1;
          const bool must = u > s.kb || u + 1 == s.ke;
          if (must || mbar_test_wait(&bar.q_empty[lq & 1], ((lq >> 1) & 1) ^ 1)) {
            for (int i = 0; i < tiles && ok; ++i) {
              const int qs = s.q + i, b = qs & 1;
              ok = RF_WAIT(q_empty[b], ((qs >> 1) & 1) ^ 1, 12);
              if (!ok) break;
              mbar_arrive_expect_tx(&bar.q_full[b], p.G * p.tt * D * 2);
              for (int c = 0; c < D / 64; ++c)
                tma_load_4d(smem + L::kOffQ + b * L::kTileBytes + c * kChunk, &tm_q,
                            &bar.q_full[b], c * 64, 0, s.head, s.row0 + i * p.tt);
              q_loads = qs + 1;
            }
            q_due = false;
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        id = id_next;
        in_page = in_next;
      }
      if (is_k) {
        s = nxt;
        id = id_seg;
        in_page = in_seg;
      }
    }
    // never leave with copies in flight: this warp's last copies, one per slot
    if (lane == 0) {
      const int ring = is_k ? L::kSlotsK : L::kSlotsV;
      for (int n = max(0, step - ring); n < step; ++n)
        mbar_wait(&bar.kv_full[(is_k ? 0 : L::kSlotsK) + n % ring], (n / ring) & 1, p.status,
                  dev_code(kDevTimeout, kKerPaged, 11), nullptr);
      for (int qs = max(0, q_loads - 2); qs < q_loads; ++qs)
        mbar_wait(&bar.q_full[qs & 1], (qs >> 1) & 1, p.status,
                  dev_code(kDevTimeout, kKerPaged, 13), nullptr);
    }
    __syncwarp();
  } else if (warp >= kWarpIssue) {
    // ------------------------------------------------------------ MMA issuers
    const int t = warp - kWarpIssue;
    bool ok = true;
    const uint64_t q_desc0 = sdesc_sw128(s_base + L::kOffQ, 16, 1024);
    const uint64_t k_desc0 = sdesc_sw128(s_base + L::kOffKV, 16, 1024);
    const uint64_t v_desc0 = sdesc_sw128(s_base + L::kOffKV, kChunk, 1024);
    const uint32_t mm_s = tmem + L::kTmemS + t * kBN;
    const uint32_t mm_o = tmem + L::kTmemO + t * D;
    const uint32_t mm_p = tmem + L::tmem_p(t);
    Slots<D> at;              // of the next step
    Slots<D> cur;             // of the step whose QK was issued last
    int n_iss = 0, n_seg = 0; // steps of the started segment issued so far, and all of them
    int started = -1;         // last segment whose Q was waited for
    bool issued_any = false;
    // the segment being started (lane 0), this group's Q tile in it
    int a_kb = 0, a_ke = 0, a_mode = 0, u_next = 0, q_slot = 0;
#define RF_SLOT(slot) (static_cast<uint64_t>(((slot) * L::kTileBytes) >> 4))
#define RF_LOCK() issue_lock(&bar.issue_lock, p.status, dev_code(kDevTimeout, kKerPaged, 23), abort_flag)
    auto needs = [&](int u) {
      if (a_mode == kPair) return u < a_kb + n_seg;
      if (a_mode == kSplit) return ((u - a_kb) & 1) == t;
      return n_seg > 0;
    };
    // The next step this group takes; steps that only the other group takes are
    // released (both slots) once they have landed. False at the segment's end.
    auto advance = [&](Slots<D>& mine) -> bool {
      while (u_next < a_ke) {
        const bool own = needs(u_next++);
        const Slots<D> w = at;
        at.next();
        if (own) {
          mine = w;
          return true;
        }
        if (!(ok = RF_WAIT(kv_full[w.k], w.kp, 20))) return false;
        mbar_arrive(&bar.kv_empty[w.k]);
        if (!(ok = RF_WAIT(kv_full[w.v], w.vp, 20))) return false;
        mbar_arrive(&bar.kv_empty[w.v]);
      }
      return false;
    };
    auto next_k = [&](Slots<D>& mine) -> bool {
      if (!advance(mine)) return false;
      return (ok = RF_WAIT(kv_full[mine.k], mine.kp, 21));
    };
    // next_k without waiting: whether everything up to the K tile of this group's
    // next step has landed. Between this group's steps lies at most one of the
    // other's (a split item), so each barrier tested is at most one phase behind.
    auto try_k = [&](Slots<D>& mine) -> bool {
      while (u_next < a_ke) {
        if (!mbar_test_wait(&bar.kv_full[at.k], at.kp)) return false;
        const bool own = needs(u_next);
        if (!own) {
          if (!mbar_test_wait(&bar.kv_full[at.v], at.vp)) return false;
          mbar_arrive(&bar.kv_empty[at.k]);
          mbar_arrive(&bar.kv_empty[at.v]);
        }
        mine = at;
        at.next();
        ++u_next;
        if (own) return true;
      }
      return false;
    };
    auto qk_commits = [&](const Slots<D>& w) {
      mma_commit(&bar.s_full[t]);
      mma_commit(&bar.kv_empty[w.k]);
      if (++n_iss == n_seg) mma_commit(&bar.q_empty[q_slot]);  // the segment's last read of Q
      cur = w;
    };
    auto issue_s = [&](const Slots<D>& w) {
      issue_qk<D>(mm_s, q_desc0 + static_cast<uint64_t>((q_slot * L::kTileBytes) >> 4),
                  k_desc0 + RF_SLOT(w.k));
    };
    // Segment k (lane 0): wait for its Q tiles, release the ones this group does
    // not read, and issue the first QK; without steps of its own, release all.
    // Every phase of every barrier is observed, in order, by both groups.
    auto start_segment = [&](int k) {
      started = k;
      n_seg = n_iss = 0;
      if (!(ok = RF_WAIT(seg_full[k % kSegs], (k / kSegs) & 1, 25))) return;
      const Seg& a = bar.seg[k % kSegs];
      if (a.seq < 0 || a.kb == a.ke) return;
      a_kb = u_next = a.kb;
      a_ke = a.ke;
      a_mode = a.mode;
      n_seg = a.n[t];
      const int q0 = a.q, tiles = a.mode == kPair ? 2 : 1;
      for (int i = 0; i < tiles; ++i) {
        const int qs = q0 + i, b = qs & 1;
        if (!(ok = RF_WAIT(q_full[b], (qs >> 1) & 1, 22))) return;
        if (n_seg > 0 && (tiles == 1 || i == t))
          q_slot = b;
        else
          mbar_arrive(&bar.q_empty[b]);
      }
      Slots<D> first;
      if (n_seg == 0) {
        advance(first);  // releases every step; returns false
        return;
      }
      if (next_k(first) && (ok = RF_LOCK())) {
        tc_fence_after_sync();
        issue_s(first);
        issue_unlock(&bar.issue_lock);
        issued_any = true;
        qk_commits(first);
      }
    };

    for (int k = 0;; ++k) {
      if (ok) ok = RF_WAIT_WARP(seg_full[k % kSegs], (k / kSegs) & 1, 26);
      if (!ok) {
        group_sync_or(t, true);
        break;
      }
      const Seg& d = bar.seg[k % kSegs];
      const int n = d.n[t], kb = d.kb, kv = d.kv, mode = d.mode;
      const bool end = d.seq < 0;
      if (lane == 0 && !end && started < k) start_segment(k);
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (lane == 0) mbar_arrive(&bar.seg_empty[k % kSegs]);
      if (end) {
        group_sync_or(t, false);
        break;
      }
      if (mode >= kSolo0 && mode != kSolo0 + t) continue;  // the other group's
      bool left = false;
      for (int jj = 0; jj < n; ++jj) {
        // While the softmax runs: wait for V_u, zero its rows past the cache's
        // end, and see whether the next step's K tile is there. If it is, its
        // Q K^T goes out in one block with this step's P.V. If it is not (memory
        // bounds a decode step), P.V goes first: it frees V_u's slot, without
        // which the rings could not run ahead of the two groups.
        const bool last = jj + 1 == n;
        const int u = kb + (mode == kSplit ? 2 * jj + t : jj);
        Slots<D> k2;
        bool fast = false;
        if (lane == 0 && ok) ok = RF_WAIT(kv_full[cur.v], cur.vp, 24);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        const int rows = kv - u * kBN;
        if (ok && rows < kBN) {
          const int vs = __shfl_sync(0xffffffffu, cur.v, 0);
          unsigned char* v = smem + L::kOffKV + vs * L::kTileBytes;
          for (int i = rows * 8 + lane; i < kBN * 8; i += 32)
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
              *reinterpret_cast<uint4*>(v + c * kChunk + i * 16) = make_uint4(0, 0, 0, 0);
          fence_proxy_async_smem();
          __syncwarp();
        }
        if (lane == 0 && ok && !last) fast = try_k(k2);
        ok = __shfl_sync(0xffffffffu, ok, 0);
        // P_t is in tensor memory
        if (group_sync_or(t, !ok)) {
          left = true;
          break;
        }
        if (lane == 0 && (ok = RF_LOCK())) {
          tc_fence_after_sync();
          const int v_slot = cur.v;
          issue_pv<D>(mm_o, mm_p, v_desc0 + RF_SLOT(v_slot), jj > 0);
          if (fast) issue_s(k2);
          issue_unlock(&bar.issue_lock);
          if (fast) qk_commits(k2);
          mma_commit(&bar.kv_empty[v_slot]);
          if (last) {
            mma_commit(&bar.o_done[t]);
          } else if (!fast && next_k(k2) && (ok = RF_LOCK())) {
            tc_fence_after_sync();
            issue_s(k2);
            issue_unlock(&bar.issue_lock);
            qk_commits(k2);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      if (left) break;
      // while the softmax warps write this segment's output: release the steps
      // after this group's last, and start this group's next segment (the one
      // after the next, when the next is the other group's alone)
      if (lane == 0 && ok && n > 0) {
        Slots<D> none;
        advance(none);
        if (ok) start_segment(k + 1);
        if (ok && n_seg == 0 && bar.seg[(k + 1) % kSegs].seq >= 0) start_segment(k + 2);
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
    }
#undef RF_SLOT
#undef RF_LOCK
    // never leave with MMAs in flight (their operands live in this CTA)
    if (lane == 0 && issued_any) {
      mma_commit(&bar.mma_idle[t]);
      mbar_wait(&bar.mma_idle[t], 0, p.status, dev_code(kDevTimeout, kKerPaged, 28), nullptr);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax groups
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;     // row within the tile == TMEM lane
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tm_s = tmem + L::kTmemS + t * kBN + lane_off;
    const uint32_t tm_o = tmem + L::kTmemO + t * D + lane_off;
    const uint32_t tm_p = tmem + L::tmem_p(t) + lane_off;
    const int row_tok = r / p.G, row_head = r - row_tok * p.G;
    const int causal = p.plan->causal;
    int j = 0;                           // S tiles consumed (all segments)
    int o_segs = 0;                      // segments whose final P.V was waited for
    int n_split = 0;                     // split segments so far
    bool ok = true;
    for (int k = 0;; ++k) {
      if (ok) ok = RF_WAIT_WARP(seg_full[k % kSegs], (k / kSegs) & 1, 31);
      if (!ok) {
        group_sync_or(t, true);
        break;
      }
      const Seg s = bar.seg[k % kSegs];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.seg_empty[k % kSegs]);
      if (s.seq < 0) {
        group_sync_or(t, false);
        break;
      }
      bool left = false;
      if (s.mode >= kSolo0 && s.mode != kSolo0 + t) continue;  // the other group's
      const int tile = s.mode == kPair ? t : 0;      // the group's query tile
      const int tok = tile * p.tt + row_tok;         // token within the item
      const bool row_ok = row_tok < p.tt && tok < s.ntok;
      // a warp without live rows leaves the softmax to the others
      const bool warp_ok = __any_sync(0xffffffffu, row_ok);
      const int n = t == 0 ? s.n[0] : s.n[1];
      // keys this row sees, and the fewest any row of the tile sees; a row that
      // holds no token computes on whatever is there and is not written
      const int row_lim = !row_ok || !causal ? s.kv : max(0, s.lim0 + tok);
      const int first_lim = causal ? max(0, s.lim0 + tile * p.tt) : s.kv;
      float m_run = kNegInf, l_run = 0.f;
      for (int jj = 0; jj < n; ++jj, ++j) {
        const int u = s.kb + (s.mode == kSplit ? 2 * jj + t : jj);
        if (ok && warp_ok)
          ok = mbar_wait_warp(&bar.s_full[t], j & 1, p.status,
                              dev_code(kDevTimeout, kKerPaged, 30), abort_flag);
        if (ok && warp_ok) {
          tc_fence_after_sync();
          const int k0 = u * kBN;
          const int lim = (first_lim - k0 < kBN) ? max(0, min(kBN, row_lim - k0)) : kBN;
          float mx;
          {
            uint32_t sr[128];
            tmem_ld128_wait(tm_s, sr);
            if (lim < kBN) {
#pragma unroll
              for (int c = 0; c < kBN; ++c)
                if (c >= lim) sr[c] = __float_as_uint(kNegInf);
            }
            float m8[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) m8[i] = kNegInf;
#pragma unroll
            for (int c = 0; c < kBN; c += 2)
              m8[(c >> 1) & 7] = fmax3(m8[(c >> 1) & 7], __uint_as_float(sr[c]),
                                       __uint_as_float(sr[c + 1]));
            mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]),
                       fmaxf(m8[6], m8[7]));
          }
          const float m_new = (mx == kNegInf) ? m_run : fmaxf(m_run, mx * p.scale_log2);
          const bool resc = m_new > m_run + kRescaleThreshold;
          const float m_use = resc ? m_new : m_run;
          const float alpha = resc ? ex2_approx(m_run - m_new) : 1.f;
          const float sh = (m_use == kNegInf) ? 0.f : m_use;
          const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
          const float2 nsh2 = make_float2(-sh, -sh);
          float2 s4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) s4[i] = make_float2(0.f, 0.f);
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint32_t sh1[64];
            tmem_ld64_wait(tm_s + 64 * h, sh1);
            if (lim < kBN) {
#pragma unroll
              for (int c = 0; c < 64; ++c)
                if (64 * h + c >= lim) sh1[c] = __float_as_uint(kNegInf);
            }
#pragma unroll
            for (int c = 0; c < 64; c += 2) {
              const float2 x = ffma2(
                  make_float2(__uint_as_float(sh1[c]), __uint_as_float(sh1[c + 1])), sc2, nsh2);
              const float2 pp = make_float2(ex2_approx(x.x), ex2_approx(x.y));
              s4[(c >> 1) & 3] = fadd2(s4[(c >> 1) & 3], pp);
              sh1[c >> 1] = pack_bf16x2(pp.x, pp.y);
            }
            tmem_st32(tm_p + 32 * h, *reinterpret_cast<const uint32_t(*)[32]>(&sh1[0]));
          }
          tmem_wait_st();
          const float2 st = fadd2(fadd2(s4[0], s4[1]), fadd2(s4[2], s4[3]));
          l_run = l_run * alpha + (st.x + st.y);
          m_run = m_use;
          if (jj > 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t ov[32];
              tmem_ld32_wait(tm_o + c, ov);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
              tmem_st32_wait(tm_o + c, ov);
            }
          }
          tc_fence_before_sync();
        }
        if (group_sync_or(t, !ok)) {
          left = true;
          break;
        }
      }
      if (left) break;
      // epilogue: O = acc / l, LSE = (m + log2 l) ln 2
      if (n > 0) {
        ok = mbar_wait_warp(&bar.o_done[t], o_segs & 1, p.status,
                            dev_code(kDevTimeout, kKerPaged, 32), abort_flag);
        ++o_segs;
      }
      if (s.mode == kSplit) {
        // Group 1's state over the odd steps goes to group 0 (m and l through
        // shared memory, O_1 read from tensor memory in the same lanes), which
        // joins it with its own and writes the rows. Group 1 then waits until
        // group 0 has read them before its next segment can overwrite O_1.
        float* xm = reinterpret_cast<float*>(smem + L::kOffXch);
        float* xl = xm + kBM;
        const uint32_t sp = n_split & 1;
        ++n_split;
        if (t == 1) {
          if (ok) {
            tc_fence_after_sync();
            xm[r] = m_run;
            xl[r] = l_run;
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.split_ready);
            ok = mbar_wait_warp(&bar.split_read, sp, p.status,
                                dev_code(kDevTimeout, kKerPaged, 34), abort_flag);
          }
        } else {
          if (ok)
            ok = mbar_wait_warp(&bar.split_ready, sp, p.status,
                                dev_code(kDevTimeout, kKerPaged, 35), abort_flag);
          if (ok) {
            tc_fence_after_sync();
            if (warp_ok) {
              const float m1 = xm[r], l1 = xl[r];
              const float m = fmaxf(m_run, m1);
              const float a0 = m_run == kNegInf ? 0.f : ex2_approx(m_run - m);
              const float a1 = m1 == kNegInf ? 0.f : ex2_approx(m1 - m);
              const float l = a0 * l_run + a1 * l1;
              const float inv = l == 0.f ? 0.f : __frcp_rn(l);  // NaN stays NaN
              // a group without steps leaves its O columns unwritten: its
              // weight is 0 and its values are never used
              const float w0 = a0 * inv, w1 = a1 * inv;
              const uint32_t tm_o1 = tmem + L::kTmemO + D + lane_off;
              const RowOut out = row_out<D>(p, s, 0, r, row_tok, row_head);
#pragma unroll 1
              for (int c = 0; c < D; c += 32) {
                uint32_t o0[32], o1[32];
                tmem_ld32_wait(tm_o + c, o0);
                tmem_ld32_wait(tm_o1 + c, o1);
                if (row_ok) {
                  float v[32];
#pragma unroll
                  for (int e = 0; e < 32; ++e)
                    v[e] = (w0 != 0.f ? w0 * __uint_as_float(o0[e]) : 0.f) +
                           (w1 != 0.f ? w1 * __uint_as_float(o1[e]) : 0.f);
                  put32(out, c, v, p.o_wide);
                }
              }
              if (row_ok && out.lse != nullptr)
                *out.lse = l == 0.f ? kNegInf : (m + __log2f(l)) * kLn2;
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.split_read);
          }
        }
      } else if (ok && warp_ok) {
        const RowOut out = row_out<D>(p, s, tile, r, row_tok, row_head);
        const float inv = l_run == 0.f ? 0.f : __frcp_rn(l_run);  // NaN stays NaN
        tc_fence_after_sync();
        if (n > 0) {
#pragma unroll 1
          for (int c = 0; c < D; c += 64) {
            uint32_t ov[64];
            tmem_ld64_wait(tm_o + c, ov);
            if (row_ok) {
              // a row without keys has P = 0 in every step: O is 0 as it stands
#pragma unroll
              for (int h = 0; h < 64; h += 32) {
                float v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(ov[h + e]) * inv;
                put32(out, c + h, v, p.o_wide);
              }
            }
          }
          tc_fence_before_sync();
        } else if (row_ok) {
          const float v[32] = {};
          for (int c = 0; c < D; c += 32) put32(out, c, v, p.o_wide);
        }
        if (row_ok && out.lse != nullptr)
          *out.lse = l_run == 0.f ? kNegInf : (m_run + __log2f(l_run)) * kLn2;
      }
    }
  }
#undef RF_WAIT
#undef RF_WAIT_WARP

  // ------------------------------------------------------------ teardown
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kWarpK) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
}

// Running softmax state of one row over parts: m, l and 16 columns.
struct MergeState {
  float m = kNegInf, l = 0.f;
  float acc[16] = {};
  // joined with another state; one without keys (m = -inf) adds nothing, NaN
  // passes through
  __device__ __forceinline__ void add(float m2, float l2, const float (&v)[16]) {
    const float mn = fmaxf(m, m2);
    const float a = m == kNegInf ? 0.f : __expf(m - mn);
    const float b = m2 == kNegInf ? 0.f : __expf(m2 - mn);
    l = l * a + l2 * b;
#pragma unroll
    for (int e = 0; e < 16; ++e) acc[e] = acc[e] * a + (b != 0.f ? b * v[e] : 0.f);
    m = mn;
  }
};

// Joins the parts of the items that several CTAs share: LSE = log sum_s
// exp(lse_s), O = sum_s exp(lse_s - LSE) O_s, in a fixed order. A warp takes 32
// rows of an item and 16 columns, a lane a row; where the rows are few the lanes
// share the parts too and join their states by shuffles. Two blocks an SM, each
// of which reads the plan once: with more, smaller blocks their reads of the
// same few lines of it queue up in L2 (1216 blocks whose warps read it each:
// 21 us for 8 items of 3 parts).
constexpr int kMergeThreads = 512;
constexpr int kMergeBlocks = 2 * kPlanCtas;

template <int D>
__global__ void __launch_bounds__(kMergeThreads, 2) attn_paged_merge(const Params p) {
  constexpr int kGroups = D / 16;
  __shared__ alignas(16) int4 table[kPlanCtas * 2];
  __shared__ int head[16];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // The plan was complete before the attention kernel let this one start, so it
  // is read (past L1, which may hold an older one) while that kernel runs; the
  // partial states have to be waited for. Every block waits, tasks or not: what
  // follows in the stream may rely on this kernel's end alone.
  if (threadIdx.x < 16) head[threadIdx.x] = __ldcg(reinterpret_cast<const int*>(p.plan) + threadIdx.x);
  for (int i = threadIdx.x; i < 2 * kPlanCtas; i += kMergeThreads)
    table[i] = __ldcg(reinterpret_cast<const int4*>(p.plan->merge) + i);
  __syncthreads();
  const PlanMerge* merge = reinterpret_cast<const PlanMerge*>(table);
  const bool matches = head[0] == kPlanMagic && head[1] == p.B && head[2] == p.T && head[3] == p.H &&
                       head[4] == p.Hkv && head[5] == p.page && head[6] == p.max_pages;
  const int n_merge = matches ? head[9] : 0;
  const int tasks = matches ? head[10] * kGroups : 0;
  pdl_wait();
  // neighbouring warps take the column groups of one unit: a row's sectors are
  // written by one block
  for (int task = blockIdx.x * (kMergeThreads / 32) + warp; task < tasks;
       task += kMergeBlocks * (kMergeThreads / 32)) {
    const int unit = task / kGroups, c = task % kGroups * 16;
    int e = -1;  // the item: the last one with unit0 <= unit
    for (int k = lane; k - lane < n_merge; k += 32)
      e += __popc(__ballot_sync(0xffffffffu, k < n_merge && merge[k].unit0 <= unit));
    const PlanMerge g = merge[e];
    const int ntok = g.rows / p.G;
    const int u0 = plan_units(ntok, 0, p.G);
    const int tile = unit - g.unit0 >= u0 ? 1 : 0;
    const int r0 = (unit - g.unit0 - tile * u0) * 32;
    const int live = min(32, min(p.tt, ntok - tile * p.tt) * p.G - r0);  // rows of the 32
    const int pad = live > 16 ? 32 : live > 8 ? 16 : 8;
    const int row = lane & (pad - 1);
    const int r = r0 + row;
    MergeState st;
    if (row < live) {
#pragma unroll 2
      for (int i = lane / pad; i < g.parts; i += 32 / pad) {
        const int cta = g.cta + i;
        const int64_t at = int64_t(i == 0 ? 2 * cta + 1 : 2 * cta) * 2 + tile;
        const float ls = __ldcg(p.lse_part + at * kBM + r);
        const float* from = p.o_part + (at * (D / 4) * kBM + r) * 4 + c * kBM;
        float v[16];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 x = __ldcg(reinterpret_cast<const float4*>(from + q * 4 * kBM));
          v[4 * q] = x.x; v[4 * q + 1] = x.y; v[4 * q + 2] = x.z; v[4 * q + 3] = x.w;
        }
        st.add(ls, 1.f, v);
      }
    }
    for (int o = pad; o < 32; o <<= 1) {
      float v[16];
      const float m2 = __shfl_xor_sync(0xffffffffu, st.m, o);
      const float l2 = __shfl_xor_sync(0xffffffffu, st.l, o);
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = __shfl_xor_sync(0xffffffffu, st.acc[i], o);
      st.add(m2, l2, v);
    }
    if (lane < pad && row < live) {
      const int64_t to = int64_t(g.row0 + tile * p.tt + r / p.G) * p.H + g.head * p.G + r % p.G;
      const float inv = st.l == 0.f ? 0.f : __fdividef(1.f, st.l);
#pragma unroll
      for (int i = 0; i < 16; ++i) st.acc[i] *= inv;
      put_bf16x16(p.o + to * D + c, st.acc, p.o_wide);
      if (c == 0 && p.lse != nullptr) p.lse[to] = st.l == 0.f ? kNegInf : st.m + __logf(st.l);
    }
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, []() {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult q{};
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  return fn;
}

// A 4-D bf16 map, 128-byte swizzle; extents, strides and box of dimensions
// 1..3 in elements (dimension 0: D contiguous elements, boxes of 64). L2 fetches
// what a row holds: 256 bytes at d = 64 would bring in the neighbouring head,
// which another CTA reads much later (4.02 TB/s of cache instead of 5.24, one ring of 12 slots).
bool make_map(CUtensorMap* m, const void* base, int D, const int64_t (&ext)[3],
              const int64_t (&stride)[3], const int (&box)[3]) {
  auto fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(ext[0]),
                              static_cast<cuuint64_t>(ext[1]), static_cast<cuuint64_t>(ext[2])};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(stride[0]) * 2,
                                 static_cast<cuuint64_t>(stride[1]) * 2,
                                 static_cast<cuuint64_t>(stride[2]) * 2};
  const cuuint32_t b[4] = {64, static_cast<cuuint32_t>(box[0]), static_cast<cuuint32_t>(box[1]),
                           static_cast<cuuint32_t>(box[2])};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, b, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            D == 64 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// One cache's map: dimensions (token, head) in the order of their strides,
// then the page; *token_first tells which.
bool make_cache_map(CUtensorMap* m, const void* base, const PagedAttnArgs& a, int64_t page_stride,
                    int64_t token_stride, int64_t head_stride, int box, int* token_first) {
  *token_first = token_stride <= head_stride ? 1 : 0;
  if (*token_first)
    return make_map(m, base, a.d, {a.page, a.Hkv, a.num_pages},
                    {token_stride, head_stride, page_stride}, {box, 1, 1});
  return make_map(m, base, a.d, {a.Hkv, a.page, a.num_pages},
                  {head_stride, token_stride, page_stride}, {1, box, 1});
}

int gcd(int a, int b) { return b == 0 ? a : gcd(b, a % b); }

template <int D>
cudaError_t launch_d(const PagedAttnArgs& a, cudaStream_t s, const char** why) {
  Params p{};
  p.plan = static_cast<const PlanHeader*>(a.plan);
  p.table = a.table;
  p.table_stride = a.table_stride;
  p.B = a.B; p.T = a.T; p.H = a.H; p.Hkv = a.Hkv;
  p.page = a.page; p.max_pages = a.max_pages; p.num_pages = a.num_pages;
  p.G = a.H / a.Hkv;
  p.tt = plan_tile_tokens(p.G);
  p.box = gcd(a.page, kBN);
  p.scale_log2 = a.scale * kLog2e;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.o_wide = reinterpret_cast<uintptr_t>(a.o) % 32 == 0;
  p.o_part = a.ws;
  p.lse_part = a.ws + size_t(2) * kPlanCtas * kPlanRows * D;
  p.status = a.status;
  CUtensorMap mq, mk, mv;
  // query rows packed (head in group, key head, token): strides ascend
  if (!make_map(&mq, a.q, D, {p.G, a.Hkv, a.T}, {D, int64_t(p.G) * D, a.q_stride},
                {p.G, 1, p.tt}) ||
      !make_cache_map(&mk, a.k_cache, a, a.k_page_stride, a.k_token_stride, a.k_head_stride, p.box,
                      &p.k_token_first) ||
      !make_cache_map(&mv, a.v_cache, a, a.v_page_stride, a.v_token_stride, a.v_head_stride, p.box,
                      &p.v_token_first)) {
    *why = "tensor map encoding failed";
    return cudaErrorInvalidValue;
  }
  constexpr int smem = Layout<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(attn_paged_kernel<D>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) {
    *why = "shared memory attribute";
    return e;
  }
  e = launch_pdl(attn_paged_kernel<D>, dim3(kPlanCtas), dim3(kThreads), smem, s, mq, mk, mv, p);
  if (e != cudaSuccess) return e;
  return launch_pdl(attn_paged_merge<D>, dim3(kMergeBlocks), dim3(kMergeThreads), 0, s, p);
}

}  // namespace

cudaError_t launch_attn_paged(const PagedAttnArgs& a, cudaStream_t s, const char** why) {
  return a.d == 128 ? launch_d<128>(a, s, why) : launch_d<64>(a, s, why);
}

}  // namespace rf
