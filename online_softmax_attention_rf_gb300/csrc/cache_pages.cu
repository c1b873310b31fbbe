// cache_pages.cu -- housekeeping of a paged key/value cache: kept rows moved
// together, pages copied, and the pages of sequences shared, handed out and
// taken back by their counts of owners.
//
// No arithmetic but whole numbers and copies. The copies are bound by memory
// (each byte read and written once), the page numbers by the latency of a few
// dependent loads.
#include <cooperative_groups.h>

#include "paged_device.cuh"

namespace cg = cooperative_groups;

namespace rf {
namespace {

// ------------------------------------------------------------------ rows

// Rows move towards the front: row i of a sequence's list comes from a place at
// or behind i, and the list ascends. A cluster of CTAs takes a share of one
// sequence's heads in some of the planes (K and V of the layers) and goes through
// the list in rounds of a chunk a CTA: in each plane a round is read whole before
// any of it is written, and what it overwrites lies before every later round's
// rows. Loads and stores of one CTA take turns; the four CTAs of an SM overlap. Half
// of 8 caches of up to 8000 tokens, 8 heads, d = 128, 4 layers dropped: 137 us, 5.4
// TB/s, bound by memory and by the longest cache's CTAs, which end last (with the
// next chunk's loads under this one's stores in a CTA there were two CTAs an SM, and
// not all resident: 166 us).
constexpr int kMoveThreads = 256;
constexpr int kMoveUnits = 8;  // rows of a chunk a thread has 16 bytes of
constexpr int kMoveRows = kMoveThreads;  // rows of a chunk at most: a thread looks one up

// kCluster: more than one CTA a cluster.
template <bool kCluster>
__global__ void __launch_bounds__(kMoveThreads, 4) kv_compact_kernel(const CompactArgs a) {
  // places (page, row in it) of a CTA's three chunks in turn, -1: stays
  __shared__ int2 from[3][kMoveRows], to[3][kMoveRows];
  pdl_wait();
  pdl_trigger();
  cg::cluster_group cluster = cg::this_cluster();
  const int size = kCluster ? static_cast<int>(cluster.num_blocks()) : 1;
  const int rank = kCluster ? static_cast<int>(cluster.block_rank()) : 0;
  const int b = blockIdx.x / size / a.head_splits, split = blockIdx.x / size % a.head_splits;
  const int plane0 = blockIdx.y * a.planes, plane1 = min(plane0 + a.planes, 2 * a.pool.layers);
  const int c0 = a.cu_keep[b], room = a.cu_keep[b + 1] - c0;
  const int n = a.n_keep != nullptr ? a.n_keep[b] : room;
  const bool head = split == 0 && blockIdx.y == 0;  // the CTA that reports
  if (c0 < 0 || room < 0 || c0 > a.N - room || n < 0 || n > room) {
    if (head && threadIdx.x == 0) record_status(a.status, dev_code(kDevBadList, kKerPages, 1));
    return;
  }
  const int64_t base = a.base != nullptr ? a.base[b] : 0;
  const int32_t* keep = a.keep + c0;
  const int32_t* table = a.table + int64_t(b) * a.table_stride;
  const int h0 = split * a.heads, heads = min(a.heads, a.pool.Hkv - h0);
  const int ru = heads * a.pool.row16;  // units of 16 bytes of a row, at most the threads
  const int pass = kMoveThreads / ru;   // rows that the threads have at a time
  const int rows = min(pass * kMoveUnits, kMoveRows);

  auto slot = [&](int64_t pos) -> int {  // page * tokens of a page + row, -1: nowhere
    if (pos < 0 || pos >= int64_t(a.max_pages) * a.pool.page) return -1;
    const int pi = static_cast<int>(pos / a.pool.page);
    const int id = table[pi];
    if (id < 0 || id >= a.pool.num_pages) return -1;
    return id * a.pool.page + static_cast<int>(pos - int64_t(pi) * a.pool.page);
  };
  auto locate = [&](int chunk, int buf) {
    const int i = chunk * rows + threadIdx.x;
    if (threadIdx.x < static_cast<unsigned>(rows)) {
      int f = -1, t = -1;
      if (i < n) {
        const int k = keep[i];
        const int prev = i > 0 ? keep[i - 1] : -1;
        if (k <= prev || k < i) {
          if (head) record_status(a.status, dev_code(kDevBadList, kKerPages, 2));
        } else if (k > i) {
          f = slot(base + k);
          t = slot(base + i);
          if (f < 0 || t < 0) {
            if (head) record_status(a.status, dev_code(kDevBadList, kKerPages, 3));
            f = t = -1;
          }
        }
      }
      from[buf][threadIdx.x] = make_int2(f < 0 ? -1 : f / a.pool.page, f % a.pool.page);
      to[buf][threadIdx.x] = make_int2(t < 0 ? -1 : t / a.pool.page, t % a.pool.page);
    }
  };
  // this thread's rows of a chunk, r0 + j * pass, and its place in them
  const int r0 = threadIdx.x / ru, u = threadIdx.x - r0 * ru, h = u / a.pool.row16;
  const int chunks = (n + rows - 1) / rows;
  locate(rank, 0);
  __syncthreads();
  for (int c = rank, buf = 0; c - rank < chunks; c += size) {
    const int next = buf < 2 ? buf + 1 : 0;
    for (int plane = plane0; plane < plane1; ++plane) {
      const PoolSide& side = (plane & 1) ? a.pool.v : a.pool.k;
      char* const mine = side.base + (plane >> 1) * side.layer + (h0 + h) * side.head +
                         (u - h * a.pool.row16) * 16;
      auto at = [&](const int2& p) {
        return reinterpret_cast<uint4*>(mine + p.x * side.page + p.y * side.token);
      };
      uint4 w[kMoveUnits];
#pragma unroll
      for (int j = 0; j < kMoveUnits; ++j) {
        const int r = r0 + j * pass;
        if (r0 < pass && r < rows && from[buf][r].x >= 0) w[j] = *at(from[buf][r]);
      }
      // a warp that is behind may still have to write the chunk before this one: the
      // next one's places go to the third buffer
      if (plane == plane0 && c - rank + size < chunks) locate(c + size, next);
      // the round is read by all
      if (kCluster) cluster.sync(); else __syncthreads();
#pragma unroll
      for (int j = 0; j < kMoveUnits; ++j) {
        const int r = r0 + j * pass;
        if (r0 < pass && r < rows && to[buf][r].x >= 0) *at(to[buf][r]) = w[j];
      }
    }
    buf = next;
  }
}

// ------------------------------------------------------------------ pages

// A CTA has 32 KB of a page in flight (pages of less: one CTA each). Bound by memory:
// 186 pages of 64 KB in 8 planes, as a step of forks copies them, in 27 us of its
// 36, 7.2 TB/s with what L2 holds of the last step.
constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = 8;  // 16-byte units in flight a thread

__global__ void __launch_bounds__(kCopyThreads) kv_copy_pages_kernel(const CopyPagesArgs a) {
  pdl_wait();
  pdl_trigger();
  const int pair = blockIdx.x / a.splits, split = blockIdx.x % a.splits;
  const int s = a.src[pair], d = a.dst[pair];
  if (s < 0 || d < 0 || s == d) return;
  if (s >= a.pool.num_pages || d >= a.pool.num_pages) {
    if (threadIdx.x == 0 && split == 0 && blockIdx.y == 0)
      record_status(a.status, dev_code(kDevBadList, kKerPages, 4));
    return;
  }
  const PoolSide& side = (blockIdx.y & 1) ? a.pool.v : a.pool.k;
  char* cache = side.base + (blockIdx.y >> 1) * side.layer;
  const char* from = cache + s * side.page;
  char* to = cache + d * side.page;
  const int units = a.pool.page * a.pool.Hkv * a.pool.row16;
  const int u0 = split * a.per_split, u1 = min(units, u0 + a.per_split);
  const bool token_major = side.head <= side.token;
  const int inner = token_major ? a.pool.Hkv : a.pool.page;
  const int64_t so = token_major ? side.token : side.head, si = token_major ? side.head : side.token;
  auto place = [&](int u) -> int64_t {
    if (side.dense) return int64_t(u) * 16;
    const int r = u / a.pool.row16, o = r / inner;
    return o * so + (r - o * inner) * si + (u - r * a.pool.row16) * 16;
  };
  for (int u = u0 + threadIdx.x; u < u1; u += kCopyThreads * kCopyUnits) {
    uint4 w[kCopyUnits];
#pragma unroll
    for (int i = 0; i < kCopyUnits; ++i)
      if (u + i * kCopyThreads < u1)
        w[i] = *reinterpret_cast<const uint4*>(from + place(u + i * kCopyThreads));
#pragma unroll
    for (int i = 0; i < kCopyUnits; ++i)
      if (u + i * kCopyThreads < u1)
        *reinterpret_cast<uint4*>(to + place(u + i * kCopyThreads)) = w[i];
  }
}

// ------------------------------------------------------------------ owners

constexpr int kOwnThreads = 256;

__device__ __forceinline__ int pages_of(int len, int page) {  // len >= 0
  return len / page + (len % page != 0 ? 1 : 0);
}

// A row of the new table is a row of the old one; its pages have one owner more, but
// for those without one, which are free and stay so: nothing adds to a count of 0, so
// that all rows that read it find it as it was. (Four rows of 32 pages 1.7 us replayed, 1.3
// without the look; 192 of 40 2.3; 16384 rows of one prompt's 16 pages 35 to 42, 25
// without, 57 where each looks in L2 and not in L1.)
__global__ void __launch_bounds__(kOwnThreads) pages_fork_kernel(const PagesForkArgs a) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int s = a.src[i];
  int len = 0;
  bool bad = s < 0 || s >= a.B;
  if (!bad) {
    len = a.len[s];
    bad = len < 0 || len > int64_t(a.max_pages) * a.page;
    if (bad) len = 0;
  }
  const int n = pages_of(len, a.page);
  for (int j = blockIdx.y * kOwnThreads + threadIdx.x; j < n; j += gridDim.y * kOwnThreads) {
    const int id = a.table[int64_t(s) * a.table_stride + j];
    a.out[int64_t(i) * a.out_stride + j] = id;
    if (id < 0 || id >= a.num_pages || a.refs[id] < 1)
      bad = true;
    else
      atomicAdd(a.refs + id, 1);
  }
  if (bad) record_status(a.status, dev_code(kDevBadList, kKerPages, 5));
  if (threadIdx.x == 0 && blockIdx.y == 0) a.len_out[i] = len;
}

// The pages of a row behind its new length lose an owner.
__global__ void __launch_bounds__(kOwnThreads) pages_release_kernel(const PagesReleaseArgs a) {
  pdl_wait();
  pdl_trigger();
  const int i = blockIdx.x;
  const int old_len = a.len[i], new_len = a.new_len != nullptr ? a.new_len[i] : 0;
  bool bad = old_len < 0 || new_len < 0 || max(old_len, new_len) > int64_t(a.max_pages) * a.page;
  if (!bad) {
    const int n = pages_of(old_len, a.page);
    for (int j = pages_of(new_len, a.page) + blockIdx.y * kOwnThreads + threadIdx.x; j < n;
         j += gridDim.y * kOwnThreads) {
      const int id = a.table[int64_t(i) * a.table_stride + j];
      if (id < 0 || id >= a.num_pages) {
        bad = true;
      } else if (atomicSub(a.refs + id, 1) <= 0) {  // had no owner: left as it was
        atomicAdd(a.refs + id, 1);
        bad = true;
      }
    }
  }
  if (bad) record_status(a.status, dev_code(kDevBadList, kKerPages, 6));
}

// New pages for rows that grow: the free pages (without owners) of the lowest
// numbers, row after row. A partly filled last page with several owners is
// written to by none of them: each of the rows that write to it gets a page of
// its own in its place and a pair (page, copy) to copy, but for the last of them
// when they are all the owners there are.
//
// One cluster: each CTA works out all rows' needs, and has a share of the pages.
// It counts the free ones of its share, and once all counts are known hands its
// own out. Bound by latency (lengths, table and owners, two cluster barriers, two
// reads of the owners) up to a few hundred rows: four rows that grow in a pool of 64
// pages 3.7 us, replayed. Many rows that write to one page are counted one by one, which
// goes with their square: in a pool of 20000 pages 5.4 us for four of them, 6.5 for 192,
// 18 for 1024, 182 for 4096, 2650 for 16384.
constexpr int kGrowThreads = 1024;
constexpr int kGrowCluster = 8;

struct GrowRow {
  int start;   // pages needed by the rows before
  int first;   // first page index that is filled in
  int shared;  // the page that is replaced, -1: none
};

// Exclusive sum over the CTA's threads, and the total; all threads call.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* warps, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  auto up = [&](T s) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const T u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += u;
    }
    return s;
  };
  const T s = up(v);
  __syncthreads();  // the sums of a call before are read
  if (lane == 31) warps[warp] = s;
  __syncthreads();
  const T w = up(warps[lane]);
  *total = __shfl_sync(0xffffffffu, w, 31);
  const T before = __shfl_sync(0xffffffffu, w, warp > 0 ? warp - 1 : 0);
  return (warp > 0 ? before : T(0)) + s - v;
}

__global__ void __cluster_dims__(kGrowCluster, 1, 1) __launch_bounds__(kGrowThreads)
    pages_grow_kernel(const PagesGrowArgs a) {
  extern __shared__ GrowRow rows[];  // [n]
  __shared__ int warps[kGrowThreads / 32];
  __shared__ int64_t wide_warps[kGrowThreads / 32];
  __shared__ int frees[kGrowCluster];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = static_cast<int>(cluster.block_rank());
  const int tid = threadIdx.x;
  cluster.barrier_arrive();
  pdl_wait();
  pdl_trigger();
  bool bad = false;
  constexpr int kNothing = -2;  // in the place of a shared page: the row gets nothing
  auto shared_page = [&](int i) -> int {
    const int len = a.len[i], to = a.new_len[i];
    if (len < 0 || to <= len || to > int64_t(a.max_pages) * a.page || len % a.page == 0) return -1;
    const int id = a.table[int64_t(i) * a.table_stride + len / a.page];
    if (id < 0 || id >= a.num_pages) {
      bad = true;
      return -1;
    }
    const int owners = a.refs[id];
    if (owners < 1) {  // a free page: it may be handed out, so that nobody can write to it
      bad = true;
      return kNothing;
    }
    return owners > 1 ? id : -1;
  };
  for (int i = tid; i < a.n; i += kGrowThreads) rows[i].shared = shared_page(i);
  __syncthreads();
  // of the rows that write to one page, all but as many as it has owners besides
  // (the sum may pass 32 bits; then there are not enough pages, and no starts needed)
  int64_t need = 0;
  for (int i0 = 0; i0 < a.n; i0 += kGrowThreads) {
    const int i = i0 + tid;
    int count = 0, first = 0;
    if (i < a.n) {
      const int len = a.len[i], to = a.new_len[i];
      if (len < 0 || to < 0 || max(len, to) > int64_t(a.max_pages) * a.page) {
        bad = true;
      } else if (rows[i].shared != kNothing) {
        const int id = rows[i].shared;
        int ahead = 0;
        if (id >= 0)
          for (int j = 0; j < i; ++j) ahead += rows[j].shared == id;
        const bool copied = id >= 0 && ahead < a.refs[id] - 1;
        first = pages_of(len, a.page) - (copied ? 1 : 0);
        count = max(0, pages_of(to, a.page) - first);
        rows[i].first = copied ? -1 - first : first;  // the sign marks a copy until all have looked
      }
    }
    int64_t total;
    const int64_t before = block_scan<int64_t>(count, wide_warps, &total);
    if (i < a.n) {
      rows[i].start = static_cast<int>(need + before);
      if (count == 0) rows[i].first = 0;
    }
    need += total;
  }
  __syncthreads();
  for (int i = tid; i < a.n; i += kGrowThreads) {
    const int f = rows[i].first;
    rows[i].first = f < 0 ? -1 - f : f;
    if (f >= 0) rows[i].shared = -1;
  }
  if (bad && rank == 0) record_status(a.status, dev_code(kDevBadList, kKerPages, 7));
  // free pages of this CTA's share: [p0, p1)
  const int share = ((a.num_pages + kGrowCluster - 1) / kGrowCluster + 3) / 4 * 4;
  const int p0 = static_cast<int>(min64(a.num_pages, int64_t(rank) * share));
  const int p1 = static_cast<int>(min64(a.num_pages, int64_t(p0) + share));
  auto group = [&](int p, int4& r) -> int {  // of four pages, how many are free
    r = make_int4(1, 1, 1, 1);
    if (p + 4 <= p1 && a.wide) {
      r = *reinterpret_cast<const int4*>(a.refs + p);
    } else {
      if (p < p1) r.x = a.refs[p];
      if (p + 1 < p1) r.y = a.refs[p + 1];
      if (p + 2 < p1) r.z = a.refs[p + 2];
      if (p + 3 < p1) r.w = a.refs[p + 3];
    }
    return (r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0);
  };
  int mine = 0;
  for (int p = p0 + tid * 4; p < p1; p += kGrowThreads * 4) {
    int4 r;
    mine += group(p, r);
  }
  int total;
  block_scan(mine, warps, &total);
  cluster.barrier_wait();
  if (tid < kGrowCluster) *cluster.map_shared_rank(&frees[rank], tid) = total;
  cluster.sync();  // all have read the table and the owners
  int have = 0, at = 0;
  for (int q = 0; q < kGrowCluster; ++q) {
    if (q < rank) at += frees[q];
    have += frees[q];
  }
  const bool enough = need <= have;
  if (rank == 0) {
    if (tid == 0) a.left[0] = static_cast<int>(max64(have - need, -int64_t(0x7fffffff)));
    for (int i = tid; i < a.n; i += kGrowThreads)
      if (!enough || rows[i].shared < 0) a.copy_src[i] = a.copy_dst[i] = -1;
  }
  if (!enough) return;
  for (int p = p0; p < p1 && at < need; p += kGrowThreads * 4) {
    int4 r;
    const int q = p + tid * 4;
    const int n = q < p1 ? group(q, r) : 0;
    int k = at + block_scan(n, warps, &total);
    at += total;
    if (n == 0) continue;
    const int refs[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (refs[e] != 0 || k >= need) continue;
      // the row: the last one that starts at or before k
      int lo = 0, hi = a.n - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (rows[mid].start <= k) lo = mid; else hi = mid - 1;
      }
      const int j = rows[lo].first + (k - rows[lo].start);
      a.table[int64_t(lo) * a.table_stride + j] = q + e;
      a.refs[q + e] = 1;
      if (rows[lo].shared >= 0 && k == rows[lo].start) {
        a.copy_src[lo] = rows[lo].shared;
        a.copy_dst[lo] = q + e;
        atomicSub(a.refs + rows[lo].shared, 1);
      }
      ++k;
    }
  }
}

}  // namespace

cudaError_t launch_kv_compact(CompactArgs a, cudaStream_t s) {
  // As many CTAs as are resident: with many planes a CTA has several (64 sequences,
  // 16 layers: 14.9 us with one each), with few the heads are shared out, then the
  // list. (One sequence of 8000 tokens, 8 heads, 8 layers, half kept: 103 us without
  // clusters, 54 with. Lists before heads: the eight sequences above 151 us.)
  constexpr int kResident = 4 * 152, kMaxCluster = 8;
  const int64_t planes = int64_t(a.B) * a.pool.layers * 2;
  int cluster = 1, splits = 1;
  while (splits < a.pool.Hkv && planes * splits < kResident) splits *= 2;
  a.planes = static_cast<int>(min64(2 * a.pool.layers, (planes + kResident - 1) / kResident));
  a.heads = (a.pool.Hkv + splits - 1) / splits;
  const int most = kMoveThreads / a.pool.row16;  // the threads hold a row
  a.heads = a.heads < most ? a.heads : most;
  a.head_splits = (a.pool.Hkv + a.heads - 1) / a.heads;
  // (a list of a few rows is one chunk)
  while (cluster < kMaxCluster && planes * a.head_splits * cluster * 2 <= kResident &&
         a.N / a.B > 64 * cluster)
    cluster *= 2;
  const dim3 grid(a.B * a.head_splits * cluster, (2 * a.pool.layers + a.planes - 1) / a.planes);
  if (cluster == 1) return launch_pdl(kv_compact_kernel<false>, grid, dim3(kMoveThreads), 0, s, a);
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kMoveThreads);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kv_compact_kernel<true>, a);
}

cudaError_t launch_kv_copy_pages(CopyPagesArgs a, cudaStream_t s) {
  // A long list of large pages: no more than 2^22 CTAs a plane, which take several
  // batches of a page each then: pairs and parts of a page fit 32 bits, and an empty
  // list of 2^20 pairs of 134 MB costs 8.4 ms (one such page among them: 9.8).
  constexpr int64_t kMost = 1 << 22;
  const int64_t units = int64_t(a.pool.page) * a.pool.Hkv * a.pool.row16;
  const int64_t batch = kCopyThreads * kCopyUnits;
  const int64_t most = kMost / a.n, batches = (units + batch - 1) / batch;  // n <= 2^20
  const int64_t per = (batches + most - 1) / most * batch;
  a.per_split = static_cast<int>(min64(units, per));
  a.splits = static_cast<int>((units + a.per_split - 1) / a.per_split);
  return launch_pdl(kv_copy_pages_kernel, dim3(a.n * a.splits, 2 * a.pool.layers),
                    dim3(kCopyThreads), 0, s, a);
}

namespace {
dim3 own_grid(int n, int max_pages) {
  const int most = (max_pages + kOwnThreads - 1) / kOwnThreads;
  return dim3(n, most < 64 ? most : 64);
}
}  // namespace

cudaError_t launch_pages_fork(const PagesForkArgs& a, cudaStream_t s) {
  return launch_pdl(pages_fork_kernel, own_grid(a.n, a.max_pages), dim3(kOwnThreads), 0, s, a);
}

cudaError_t launch_pages_release(const PagesReleaseArgs& a, cudaStream_t s) {
  return launch_pdl(pages_release_kernel, own_grid(a.n, a.max_pages), dim3(kOwnThreads), 0, s, a);
}

cudaError_t launch_pages_grow(PagesGrowArgs a, cudaStream_t s) {
  const size_t smem = size_t(a.n) * sizeof(GrowRow);
  if (smem > 40 * 1024) {  // more than a kernel has by itself
    const cudaError_t e = cudaFuncSetAttribute(
        pages_grow_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>(kMaxGrowRows * sizeof(GrowRow)));  // all calls set the same
    if (e != cudaSuccess) return e;
  }
  a.wide = reinterpret_cast<uintptr_t>(a.refs) % 16 == 0;
  return launch_pdl(pages_grow_kernel, dim3(kGrowCluster), dim3(kGrowThreads), smem, s, a);
}

}  // namespace rf
