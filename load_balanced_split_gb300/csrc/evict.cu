// Eviction from the paged cache by accumulated attention weight: which keys each KV head
// keeps (evict_select_kernel), and the move of their rows to the front (evict_compact_kernel).
//
// Selection.  A request longer than its budget keeps its first `sinks` keys, its last
// `recent` keys and, of the others, the budget - sinks - recent with the largest weight,
// ties to the lower index.  One block per (request, KV head): a radix select over an
// order-preserving integer image of the weights (digits of 11, 11 and 10 bits: three
// histograms instead of a sort) finds the last weight that stays, T, and how many keys of
// weight T stay; a pass with ballots and one scan over the block then writes the kept
// indices in ascending order.  The weights are read from memory once and kept in shared
// memory (up to kKeyCap of them; a longer request's rest is read again in each pass).
//
// Compaction.  Row t of the new cache is row kept[t] of the old one, and kept is
// ascending, so kept[t] >= t: a block that takes the rows of one (request, head) in order,
// a chunk at a time, and writes a chunk after all of its rows are read never overwrites a
// row that is still needed.  Columns of a row are independent, so with few (request, head)
// pairs a row is split over several blocks; a move to other pages also splits the rows.
#include "hpa_internal.cuh"

namespace hpa {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kKeyCap = 48 * 1024;  // weights held in shared memory
constexpr int kBins = 2048;
constexpr int kSelSmem = kKeyCap * 4 + kBins * 4;

// Integers in the order of the weights: NaN above every number, -0 equal to +0.
__device__ __forceinline__ uint32_t weight_key(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The bin that holds the k-th largest entry (k >= 1, k <= the entries counted), and the
// number of entries in higher bins.  All threads of the block call it.
__device__ void find_bin(const int *hist, int k, int *wsum, int &bin, int &above) {
  __shared__ int s_bin, s_above;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  // thread t owns bins kBins - 1 - 2 t and the one below: a scan from the top
  const int b0 = kBins - 1 - 2 * tid, h0 = hist[b0], h1 = hist[b0 - 1];
  int v = h0 + h1;
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) wsum[wid] = v;
  __syncthreads();
  if (wid == 0) {
    int s = wsum[lane];
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(kFull, s, o);
      if (lane >= o) s += n;
    }
    wsum[lane] = s;
  }
  __syncthreads();
  const int before = v - h0 - h1 + (wid ? wsum[wid - 1] : 0);
  if (before < k && before + h0 >= k) {
    s_bin = b0;
    s_above = before;
  } else if (before + h0 < k && before + h0 + h1 >= k) {
    s_bin = b0 - 1;
    s_above = before + h0;
  }
  __syncthreads();
  bin = s_bin;
  above = s_above;
  __syncthreads();
}

__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t sel_smem[];
  uint32_t *keys = sel_smem;
  int *hist = reinterpret_cast<int *>(sel_smem + kKeyCap);
  __shared__ int wsum[kSelWarps], s_bad;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int r = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  if (tid == 0) s_bad = 0;
  for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
  __syncthreads();
  const int L = p.seq_lens[r], budget = p.budgets[r];
  const int pstart = p.page_indptr[r], pcount = p.page_indptr[r + 1] - pstart;
  const int n = min(L, budget);
  int bad = 0;
  if (L < 1) bad = HPA_STATUS_BAD_SEQLEN;
  else if (budget < 1 || n > p.kept_stride ||
           (L > budget && static_cast<int64_t>(p.sinks) + p.recent > budget))
    bad = HPA_STATUS_BAD_BUDGET;
  else if ((L - 1) / PAGE + 1 > pcount)
    bad = HPA_STATUS_BAD_PAGE;
  int32_t *kept = p.kept + static_cast<int64_t>(blockIdx.x) * p.kept_stride;
  const bool cut = !bad && L > budget;
  const int lo = p.sinks, hi = L - p.recent;  // candidates [lo, hi) when the request is cut
  const int npages = bad ? 0 : (L - 1) / PAGE + 1;

  // page pg's two weights of this lane, as order-preserving integers
  auto load_page = [&](int pg) {
    const int id = p.page_indices[pstart + pg];
    uint2 x = make_uint2(0u, 0u);
    if (id < 0 || id >= p.num_pages) s_bad = HPA_STATUS_BAD_PAGE;
    else
      x = reinterpret_cast<const uint2 *>(p.acc + (static_cast<int64_t>(id) * p.Hkv + h) * PAGE)[lane];
    return make_uint2(weight_key(x.x), weight_key(x.y));
  };
  // every candidate's key in turn, a page per warp and turn
  auto each = [&](bool first, auto f) {
    for (int pg = wid; pg < npages; pg += kSelWarps) {
      const int i = pg * PAGE + 2 * lane;
      uint2 k;
      if (!first && pg < kKeyCap / PAGE) {
        k = *reinterpret_cast<const uint2 *>(keys + i);
      } else {
        k = load_page(pg);
        if (pg < kKeyCap / PAGE) *reinterpret_cast<uint2 *>(keys + i) = k;
      }
      if (i >= lo && i < hi) f(k.x);
      if (i + 1 >= lo && i + 1 < hi) f(k.y);
    }
  };

  if (!cut && !bad) {  // nothing leaves: the pages are checked, as below
    for (int pg = tid; pg < npages; pg += kSelThreads) {
      const int id = p.page_indices[pstart + pg];
      if (id < 0 || id >= p.num_pages) s_bad = HPA_STATUS_BAD_PAGE;
    }
  }
  uint32_t T = 0xffffffffu;
  int need = 0, take = cut ? budget - p.sinks - p.recent : 0;
  if (cut) {
    each(true, [&](uint32_t k) { atomicAdd(&hist[k >> 21], 1); });
    __syncthreads();
    if (take > 0) {  // uniform over the block
      int b1, b2, b3, above;
      find_bin(hist, take, wsum, b1, above);
      need = take - above;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      each(false, [&](uint32_t k) { if (k >> 21 == b1) atomicAdd(&hist[(k >> 10) & 2047], 1); });
      __syncthreads();
      find_bin(hist, need, wsum, b2, above);
      need -= above;
      for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      const uint32_t top = (static_cast<uint32_t>(b1) << 11) | b2;
      each(false, [&](uint32_t k) { if (k >> 10 == top) atomicAdd(&hist[k & 1023], 1); });
      __syncthreads();
      find_bin(hist, need, wsum, b3, above);
      need -= above;  // keys equal to T that stay
      T = (top << 10) | b3;
    }
  }
  __syncthreads();
  if (!bad) bad = s_bad;
  if (bad) {
    if (tid == 0) {
      if (p.status) atomicOr(reinterpret_cast<int *>(p.status), bad);
      if (h == 0) p.new_lens[r] = -1;
    }
    return;
  }
  if (tid == 0 && h == 0) p.new_lens[r] = n;
  if (!cut) {
    for (int i = tid; i < n; i += kSelThreads) kept[i] = i;
    return;
  }
  // a contiguous range of pages per warp: keys above T (and the fixed ones) and equal to T
  __shared__ int s_gt[kSelWarps], s_eq[kSelWarps];
  const int per = (npages + kSelWarps - 1) / kSelWarps;
  const int p0 = min(npages, wid * per), p1 = min(npages, p0 + per);
  auto classify = [&](int pg, int half, bool &gt, bool &eq) {
    const int i = pg * PAGE + 32 * half + lane;
    gt = eq = false;
    if (i >= L) return;
    if (i < lo || i >= hi) {
      gt = true;
      return;
    }
    uint32_t k;
    if (pg < kKeyCap / PAGE) {
      k = keys[i];
    } else {
      const int id = p.page_indices[pstart + pg];  // in range: checked when it was first read
      k = weight_key(__float_as_uint(p.acc[(static_cast<int64_t>(id) * p.Hkv + h) * PAGE + i % PAGE]));
    }
    gt = take > 0 && k > T;
    eq = take > 0 && k == T;
  };
  int gt_n = 0, eq_n = 0;
  for (int pg = p0; pg < p1; ++pg)
    for (int half = 0; half < 2; ++half) {
      bool gt, eq;
      classify(pg, half, gt, eq);
      gt_n += __popc(__ballot_sync(kFull, gt));
      eq_n += __popc(__ballot_sync(kFull, eq));
    }
  if (lane == 0) s_gt[wid] = gt_n, s_eq[wid] = eq_n;
  __syncthreads();
  int gt_at = 0, eq_at = 0;
  for (int x = 0; x < wid; ++x) gt_at += s_gt[x], eq_at += s_eq[x];
  const uint32_t below = (1u << lane) - 1u;
  for (int pg = p0; pg < p1; ++pg)
    for (int half = 0; half < 2; ++half) {
      bool gt, eq;
      classify(pg, half, gt, eq);
      const uint32_t mg = __ballot_sync(kFull, gt), me = __ballot_sync(kFull, eq);
      const int eq_rank = eq_at + __popc(me & below);
      if (gt || (eq && eq_rank < need))
        kept[gt_at + __popc(mg & below) + min(eq_rank, need)] = pg * PAGE + 32 * half + lane;
      gt_at += __popc(mg);
      eq_at += __popc(me);
    }
}

// ----------------------------------------------------------------------------- compaction
constexpr int kCmpThreads = 256;
constexpr int kCmpRows = 4;  // rows in flight per thread

// Moves the T-wide column `col` of rows [t0, t1) of one (request, head); `lanes` threads
// share a row.  base: the pool as T; row_ts: Ts per row.
template <typename T>
__device__ void move_rows(const CompactParams &p, T *base, int row_ts, int col, int lanes, int r,
                          int h, int t0, int t1) {
  const int32_t *kept = p.kept + (static_cast<int64_t>(r) * p.Hkv + h) * p.kept_stride;
  const bool in_place = p.dst_indptr == nullptr;
  const int ps = p.page_indptr[r], pn = p.page_indptr[r + 1] - ps;
  const int ds = in_place ? ps : p.dst_indptr[r];
  const int dn = in_place ? pn : p.dst_indptr[r + 1] - ds;
  const int32_t *didx = in_place ? p.page_indices : p.dst_indices;
  const int per = kCmpThreads / lanes, row = threadIdx.x / lanes;
  const int c = col + threadIdx.x % lanes;
  auto place = [&](const int32_t *idx, int start, int count, int t) -> int64_t {
    const int id = t >= 0 && t / PAGE < count ? idx[start + t / PAGE] : -1;
    if (id < 0 || id >= p.num_pages) {
      if (p.status) atomicOr(reinterpret_cast<int *>(p.status), HPA_STATUS_BAD_PAGE);
      return -1;
    }
    return ((static_cast<int64_t>(id) * p.Hkv + h) * PAGE + t % PAGE) * row_ts + c;
  };
  for (int b = t0; b < t1; b += kCmpRows * per) {
    T x[kCmpRows];
    int64_t to[kCmpRows];
#pragma unroll
    for (int u = 0; u < kCmpRows; ++u) {
      const int t = b + u * per + row;
      to[u] = -1;
      if (t < t1) {
        const int src = kept[t];
        if (!(in_place && src == t)) {
          const int64_t from = place(p.page_indices, ps, pn, src);
          if (from >= 0) {
            to[u] = place(didx, ds, dn, t);
            x[u] = base[from];
          }
        }
      }
    }
    if (in_place) __syncthreads();  // the chunk is read before any of it is written
#pragma unroll
    for (int u = 0; u < kCmpRows; ++u)
      if (to[u] >= 0) base[to[u]] = x[u];
  }
}

__global__ void __launch_bounds__(kCmpThreads)
    evict_compact_kernel(const CompactParams p, int slices, int t_split) {
  const int r = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
  const int n = p.new_lens[r];
  if (n <= 0 || n > p.kept_stride) return;  // left as it is (new_lens -1: a bad request)
  int t0 = 0, t1 = n;
  if (t_split > 1) {
    const int64_t z = blockIdx.z;
    t0 = static_cast<int>(n * z / t_split);
    t1 = static_cast<int>(n * (z + 1) / t_split);
  }
  const int part = blockIdx.y, row_ts = p.row_bytes / 16;
  if (part < 2 * slices) {
    uint4 *base = static_cast<uint4 *>(part & 1 ? p.v_pool : p.k_pool);
    const int lanes = row_ts / slices;
    move_rows<uint4>(p, base, row_ts, (part >> 1) * lanes, lanes, r, h, t0, t1);
  } else {
    move_rows<float>(p, p.acc, 1, 0, 1, r, h, t0, t1);
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictParams &p, cudaStream_t s) {
  static int configured[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSelSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = 1;
  }
  evict_select_kernel<<<static_cast<unsigned>(p.B * p.Hkv), kSelThreads, kSelSmem, s>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_evict_compact(const CompactParams &p, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t pairs = static_cast<int64_t>(p.B) * p.Hkv;
  int slices = 1;  // at least 32 bytes of a row
  while (slices < p.row_bytes / 32 && pairs * 2 * slices < 4 * sms) slices *= 2;
  int t_split = 1;
  if (p.dst_indptr != nullptr)
    while (t_split < 64 && pairs * 2 * slices * t_split < 8 * sms) t_split *= 2;
  const dim3 grid(static_cast<unsigned>(pairs), 2 * slices + (p.acc ? 1 : 0), t_split);
  evict_compact_kernel<<<grid, kCmpThreads, 0, s>>>(p, slices, t_split);
  return cudaGetLastError();
}

}  // namespace hpa
