// Eviction from the paged cache by accumulated attention weight: which keys each KV head
// keeps (evict_select_kernel), and the move of their rows to the front.
//
// Selection.  A request longer than its budget keeps its first `sinks` keys, its last
// `recent` keys and, of the others, the budget - sinks - recent with the largest weight,
// ties to the lower index.  One cluster of 1 to 8 blocks per (request, KV head): a radix
// select over an order-preserving integer image of the weights (digits of 11, 10 and 11
// bits: three histograms instead of a sort) finds the last weight that stays, T, and how
// many keys of weight T stay; the blocks add up one another's histograms through
// distributed shared memory.  A pass with ballots and a scan over the warps and blocks
// then writes the kept indices in ascending order.  The weights are read from memory once,
// eight pages in flight per warp, and stay in the shared memory of the cluster (24 K keys
// a block, 192 K a cluster; a longer request's rest is read again in each pass, from L2).
// The third digit's pass also counts what lies above and lists the few keys that share
// both digits before, so the final counts go over that list.
// Bound by instructions (44 % of the issue slots busy over the whole launch, the wait for
// their fetch the first stall) and the barriers between the passes, not by memory: 15 us for
// 32 requests of 8 heads and about 8192 keys cut to 2048, 54 for 64 of about 24000 cut to
// 4096, 23 for one of 196608 cut to 16384.
//
// Compaction (evict_copy_kernel to other pages, evict_shift_kernel in place).  Row t of the
// new cache is row kept[t] of the old one, and kept is ascending, so kept[t] >= t: in place,
// a cluster that takes the rows of one (request, head) in order, a step at a time, and
// writes a step after all of its rows are read never overwrites a row that is still needed.
// Columns of a row are independent, so with few (request, head) pairs a row is split over
// several blocks.  Bound by DRAM: to other pages 0.54 GB read and written in 86 us (6.2
// TB/s) for the first of those, 1.09 GB (E4M3 rows) in 174 us, 68 MB in 14.3 for the last.
// In place the same rows take 94, 187 and 28 us: a step's reads end before its writes
// begin.  One block per (pair, slice) with no cluster took 108, 271 and 180.
#include <cooperative_groups.h>

#include <climits>
#include <type_traits>

#include "hpa_internal.cuh"

namespace hpa {
namespace {

namespace cg = cooperative_groups;

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kWarpPages = 24;                               // pages a warp holds in shared memory
constexpr int kBlockPages = kSelWarps * kWarpPages;
constexpr int kBins = 2048, kBins2 = 1024;                    // first and third digit; second
constexpr int kList = 1024;                                  // keys that share two digits
constexpr int kMaxCluster = 8;
constexpr int kMaxLen = INT_MAX - 65536;  // the loops over keys run past the end by less
// Keys per block before a cluster grows, half of what a block holds: each of a cluster's
// barriers costs a microsecond (72 pairs of 12000 keys: 16 us in one block each, 21 in four;
// 8 of 16384: 17 in two and in four; 8 of 1024: 6 in one, 18 in eight)
constexpr int64_t kMinKeys = 12288;
constexpr int kSelSmem = kBlockPages * PAGE * 4 + (kBins + kBins2 + kList) * 4;
constexpr int kSelBlocks = 2;                                // per SM: 112 KB of shared memory each
constexpr int kFlight = 4;                                   // page pairs in flight per warp
// Keys that are no candidates: beyond the request, and those that stay in any case
constexpr uint32_t kAbsent = 0u, kFixed = 0xffffffffu;

// Integers in the order of the weights, between kAbsent and kFixed: NaN above every
// number, -0 equal to +0.
__device__ __forceinline__ uint32_t weight_key(uint32_t u) {
  if ((u & 0x7fffffffu) > 0x7f800000u) return kFixed - 1;
  if (u == 0x80000000u) u = 0u;
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Over the n blocks of the cluster that take part: the bin of the k-th largest entry (1 <= k
// <= the entries counted) and the number of entries in higher bins.  The caller has
// synchronised the cluster after the last count into `hist`.
template <int BINS>
__device__ void find_bin(cg::cluster_group &cl, int n, int *hist, int k, int &bin, int &above) {
  constexpr int N = BINS / kSelThreads;  // bins per thread: 4 or 2
  typedef typename std::conditional<N == 4, int4, int2>::type Bins;
  static_assert(sizeof(Bins) == 4 * N, "one load per block");
  __shared__ int wsum[kSelWarps], s_bin, s_above;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  // thread t owns bins [low, low + N), low = BINS - N (t + 1): a scan from the highest bin
  const int low = BINS - N * (tid + 1);
  int c[N];
  auto add = [&](const int *from, bool first) {
    const Bins o = *reinterpret_cast<const Bins *>(from + low);
    const int *x = reinterpret_cast<const int *>(&o);
#pragma unroll
    for (int i = 0; i < N; ++i) c[i] = (first ? 0 : c[i]) + x[i];
  };
  add(hist, true);
  if (n > 1) {
    const int me = cl.block_rank();
#pragma unroll
    for (int x = 1; x < kMaxCluster; ++x)  // all the others' loads in flight
      if (x < n) add(cl.map_shared_rank(hist, (me + x) & (n - 1)), false);
  }
  int mine = 0;
#pragma unroll
  for (int i = 0; i < N; ++i) mine += c[i];
  int v = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) wsum[wid] = v;
  __syncthreads();
  const int before = v - mine + __reduce_add_sync(kFull, lane < wid ? wsum[lane] : 0);
  if (before < k && before + mine >= k) {
    int up = before;  // entries in the bins above bin x
    bool found = false;
#pragma unroll
    for (int x = N - 1; x >= 0; --x) {
      if (!found && up + c[x] >= k) {
        s_bin = low + x;
        s_above = up;
        found = true;
      }
      up += c[x];
    }
  }
  __syncthreads();
  bin = s_bin;
  above = s_above;
}

__global__ void __launch_bounds__(kSelThreads, kSelBlocks)
    evict_select_kernel(const EvictParams p) {
  extern __shared__ __align__(16) uint32_t sel_smem[];
  __shared__ int s_bad, s_listed, s_total[2], s_gt[kSelWarps], s_eq[kSelWarps];
  cg::cluster_group cl = cg::this_cluster();
  int ranks = cl.num_blocks();
  const int rank = cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  int *hist0 = reinterpret_cast<int *>(sel_smem + kBlockPages * PAGE), *hist1 = hist0 + kBins;
  // keys that share the first two digits: their other 11 bits, and the warp above them
  uint32_t *list = reinterpret_cast<uint32_t *>(hist1 + kBins2);
  uint32_t *keys = sel_smem + wid * (kWarpPages * PAGE);   // this warp's first pages
  const int pair = blockIdx.x / ranks, slot = pair / p.Hkv, h = pair % p.Hkv;
  // No early launch of the kernel after this one: compaction blocks that wait on the SMs
  // settle unevenly around these (174 -> 251 us of compaction on 64 requests cut to 4096).
  pdl_wait();
  int r = slot;
  if (p.longest_first) {  // the request that has `slot` longer ones; four threads count for each
    __shared__ int s_r;
    int *lens = reinterpret_cast<int *>(sel_smem);
    for (int i = tid; i < p.B; i += kSelThreads) lens[i] = p.seq_lens[i];
    __syncthreads();
    const int q = tid >> 2;
    int longer = 0;
    if (q < p.B)
      for (int u = tid & 3; u < p.B; u += 4)
        longer += lens[u] > lens[q] || (lens[u] == lens[q] && u < q);
    longer += __shfl_xor_sync(kFull, longer, 1);
    longer += __shfl_xor_sync(kFull, longer, 2);
    if (q < p.B && (tid & 3) == 0 && longer == slot) s_r = q;
    __syncthreads();
    r = s_r;
  }
  const int L = p.seq_lens[r], budget = p.budgets[r];
  const int pstart = p.page_indptr[r], pcount = p.page_indptr[r + 1] - pstart;
  // hpa_evict to other pages: their list is checked here, before anything is moved
  const int dstart = p.dst_indptr ? p.dst_indptr[r] : 0;
  const int dcount = p.dst_indptr ? p.dst_indptr[r + 1] - dstart : 0;
  const int n = min(L, budget);
  if (tid == 0) s_bad = s_listed = 0;
  if (tid < kSelWarps) s_gt[tid] = s_eq[tid] = 0;
  for (int i = tid; i < (kBins + kBins2) / 4; i += kSelThreads)  // both histograms
    reinterpret_cast<int4 *>(hist0)[i] = make_int4(0, 0, 0, 0);
  int bad = 0;  // the same in every block of the cluster
  if (L < 1) bad = HPA_STATUS_BAD_SEQLEN;
  else if (L > kMaxLen) bad = HPA_STATUS_OVERFLOW;
  else if (budget < 1 || n > p.kept_stride ||
           (L > budget && static_cast<int64_t>(p.sinks) + p.recent > budget))
    bad = HPA_STATUS_BAD_BUDGET;
  else if ((L - 1) / PAGE + 1 > pcount)
    bad = HPA_STATUS_BAD_PAGE;
  else if (p.dst_indptr && (n - 1) / PAGE + 1 > dcount)
    bad = HPA_STATUS_BAD_PAGE;
  const bool lead = rank == 0 && tid == 0;
  auto refuse = [&](int why) {
    if (lead) {
      if (p.status) atomicOr(reinterpret_cast<int *>(p.status), why);
      if (h == 0) p.new_lens[r] = -1;
    }
  };
  if (bad) {
    refuse(bad);
    return;
  }
  // A short request is the first blocks' alone (4 of 1024 keys in a large pool: 27 us in
  // eight blocks each, 11 so); the cluster's barrier does not wait for blocks that have left.
  while (ranks > 1 && static_cast<int64_t>(ranks / 2) * kMinKeys >= L) ranks /= 2;
  if (rank >= ranks) return;
  __syncthreads();
  int32_t *kept = p.kept + (static_cast<int64_t>(r) * p.Hkv + h) * p.kept_stride;
  const int32_t *pidx = p.page_indices + pstart;
  const bool cut = L > budget;
  const int npages = (L - 1) / PAGE + 1;
  // contiguous pages: per block, and within it per warp
  const int per_block = (npages + ranks - 1) / ranks;
  const int b0 = min(npages, rank * per_block), b1 = min(npages, b0 + per_block);
  const int per_warp = (b1 - b0 + kSelWarps - 1) / kSelWarps;
  const int w0 = min(b1, b0 + wid * per_warp), w1 = min(b1, w0 + per_warp);
  const int held = min(w1, w0 + kWarpPages);  // pages [w0, held) stay in shared memory
  const int lo = p.sinks, hi = L - p.recent;  // candidates [lo, hi) of a request that is cut
  const int take = cut ? budget - p.sinks - p.recent : 0;

  // Reads pages [from, to), two per turn (lane: 4 consecutive keys), and gives f each
  // turn's keys in order; KEEP stores them as well.
  auto read_pages = [&](int from, int to, auto keep, auto f) {
    constexpr bool KEEP = decltype(keep)::value;
    for (int g = from; g < to; g += 32) {
      const int cnt = min(32, to - g);
      int id = 0;
      if (lane < cnt) {
        id = pidx[g + lane];
        if (id < 0 || id >= p.num_pages) {
          s_bad = 1;
          id = 0;
        }
      }
      for (int u0 = 0; u0 < cnt; u0 += 2 * kFlight) {
        uint4 k[kFlight];
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          const int at = u0 + 2 * u + (lane >> 4);
          const int pid = __shfl_sync(kFull, id, at & 31);
          k[u] = make_uint4(0u, 0u, 0u, 0u);
          if (at < cnt)
            k[u] = reinterpret_cast<const uint4 *>(
                p.acc + (static_cast<int64_t>(pid) * p.Hkv + h) * PAGE)[lane & 15];
        }
#pragma unroll
        for (int u = 0; u < kFlight; ++u) {
          const int at = u0 + 2 * u, i = (g + at) * PAGE + 4 * lane;
          if (at >= cnt) break;
          auto key = [&](uint32_t x, int j) {
            return j >= hi || j < lo ? (j < L ? kFixed : kAbsent) : weight_key(x);
          };
          const bool there = at + (lane >> 4) < cnt;  // an odd last page
          const int key0 = (g + at) * PAGE;
          const bool plain = at + 1 < cnt && key0 >= lo && hi - key0 >= 2 * PAGE;
          uint4 x = make_uint4(kAbsent, kAbsent, kAbsent, kAbsent);
          // the usual turn: candidates alone, none of them negative or NaN
          const bool usual =
              plain &&
              __all_sync(kFull, max(max(k[u].x, k[u].y), max(k[u].z, k[u].w)) <= 0x7f800000u);
          if (usual) {
            x = make_uint4(k[u].x | 0x80000000u, k[u].y | 0x80000000u, k[u].z | 0x80000000u,
                           k[u].w | 0x80000000u);
            if (KEEP) *reinterpret_cast<uint4 *>(keys + (g + at - w0) * PAGE + 4 * lane) = x;
          } else if (there) {
            x = make_uint4(key(k[u].x, i), key(k[u].y, i + 1), key(k[u].z, i + 2),
                           key(k[u].w, i + 3));
            if (KEEP) *reinterpret_cast<uint4 *>(keys + (g + at - w0) * PAGE + 4 * lane) = x;
          }
          f(i, x);
        }
      }
    }
  };
  // All keys of the warp again, in order: those held, then the rest from memory.
  auto each = [&](auto f) {
    for (int pg = w0; pg < held; pg += 2) {
      uint4 x = make_uint4(kAbsent, kAbsent, kAbsent, kAbsent);
      if (pg + (lane >> 4) < held)
        x = *reinterpret_cast<const uint4 *>(keys + (pg - w0) * PAGE + 4 * lane);
      f(pg * PAGE + 4 * lane, x);
    }
    read_pages(held, w1, std::false_type(), f);
  };

  // Ids of the new cache's pages come while the weights are read: one per thread into the
  // list, which is not in use yet (32 x 8192 cut to 2048: 15.5 us, 15.7 with a wait here,
  // 14.9 in place).
  const int dpages = p.dst_indptr ? (n - 1) / PAGE + 1 : 0, g0 = rank * kSelThreads + tid;
  if (g0 < dpages)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(list + tid)),
                 "l"(p.dst_indices + dstart + g0)
                 : "memory");

  if (cut) {
    auto first = [&](int, uint4 x) {
      auto add = [&](uint32_t k) {
        if (k - 1u < kFixed - 1u) atomicAdd(&hist0[k >> 21], 1);
      };
      add(x.x), add(x.y), add(x.z), add(x.w);
    };
    read_pages(w0, held, std::true_type(), first);
    read_pages(held, w1, std::false_type(), first);
    __syncwarp();
  } else {  // nothing leaves, but the pages are checked in the same way
    for (int g = w0 + lane; g < w1; g += 32)
      if (pidx[g] < 0 || pidx[g] >= p.num_pages) s_bad = 1;
  }
  if (g0 < dpages) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    int id = static_cast<int>(list[tid]);
    for (int g = g0;; id = p.dst_indices[dstart + g]) {
      if (id < 0 || id >= p.num_pages) s_bad = 1;
      g += ranks * kSelThreads;
      if (g >= dpages) break;
    }
  }
  auto cluster_sync = [&]() {
    if (ranks > 1) cl.sync();
    else __syncthreads();
  };
  cluster_sync();
  if (ranks > 1) {
#pragma unroll
    for (int x = 0; x < kMaxCluster; ++x)
      if (x < ranks) bad |= *cl.map_shared_rank(&s_bad, x);
  } else {
    bad = s_bad;
  }
  if (bad || !cut) {
    if (bad) refuse(HPA_STATUS_BAD_PAGE);
    else {
      if (lead && h == 0) p.new_lens[r] = n;
      for (int i = rank * kSelThreads + tid; i < n; i += ranks * kSelThreads) kept[i] = i;
    }
    cluster_sync();  // no block leaves while another reads its shared memory
    return;
  }
  uint32_t T = kFixed - 1;  // with nothing to take, only the fixed keys are above
  int need = 0, gt_n = 0, eq_n = 0;
  if (take > 0) {
    int d1, d2, d3, above;
    find_bin<kBins>(cl, ranks, hist0, take, d1, above);
    need = take - above;
    const uint32_t top1 = d1;
    const uint32_t low1 = top1 << 21, end1 = top1 == 2047 ? kFixed : low1 + (1u << 21);
    each([&](int, uint4 x) {
      auto see = [&](uint32_t k) {
        if (k - low1 < end1 - low1) atomicAdd(&hist1[(k >> 11) & 1023], 1);
      };
      see(x.x), see(x.y), see(x.z), see(x.w);
    });
    cluster_sync();
    find_bin<kBins2>(cl, ranks, hist1, need, d2, above);
    need -= above;
    // every block has read hist0 (before the barrier above): it takes the last digit
    for (int i = tid; i < kBins / 4; i += kSelThreads)
      reinterpret_cast<int4 *>(hist0)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    // keys above both digits are counted; the few that share them go on the list
    const uint32_t top2 = top1 << 10 | static_cast<uint32_t>(d2), low2 = top2 << 11;
    const uint32_t end2 = top2 == 0x1fffffu ? kFixed : low2 + 2048u;
    each([&](int, uint4 x) {
      auto see = [&](uint32_t k) {
        gt_n += k >= end2;  // the fixed ones among them
        if (k - low2 < end2 - low2) {
          atomicAdd(&hist0[k & 2047], 1);
          const int at = atomicAdd(&s_listed, 1);
          if (at < kList) list[at] = (k & 2047u) | static_cast<uint32_t>(wid) << 11;
        }
      };
      see(x.x), see(x.y), see(x.z), see(x.w);
    });
    cluster_sync();
    const int listed = s_listed;  // of this block: beyond kList its keys are walked again
    find_bin<kBins>(cl, ranks, hist0, need, d3, above);
    need -= above;  // keys equal to T that stay
    T = low2 | static_cast<uint32_t>(d3);
    if (listed <= kList) {
      for (int i = tid; i < listed; i += kSelThreads) {
        const int k = list[i] & 2047u, w = list[i] >> 11;
        if (k > d3) atomicAdd(&s_gt[w], 1);
        else if (k == d3) atomicAdd(&s_eq[w], 1);
      }
    } else {
      each([&](int, uint4 x) {
        auto see = [&](uint32_t k) {
          gt_n += k > T && k < end2;
          eq_n += k == T;
        };
        see(x.x), see(x.y), see(x.z), see(x.w);
      });
    }
  } else {
    each([&](int, uint4 x) {
      gt_n += (x.x == kFixed) + (x.y == kFixed) + (x.z == kFixed) + (x.w == kFixed);
    });
  }
  gt_n = __reduce_add_sync(kFull, gt_n);
  eq_n = __reduce_add_sync(kFull, eq_n);
  if (lane == 0) atomicAdd(&s_gt[wid], gt_n), atomicAdd(&s_eq[wid], eq_n);
  __syncthreads();
  const int gt_w = lane < kSelWarps ? s_gt[lane] : 0, eq_w = lane < kSelWarps ? s_eq[lane] : 0;
  int gt_at = __reduce_add_sync(kFull, lane < wid ? gt_w : 0);  // before this warp
  int eq_at = __reduce_add_sync(kFull, lane < wid ? eq_w : 0);
  if (ranks > 1) {
    if (wid == 0) {
      const int gt_all = __reduce_add_sync(kFull, gt_w), eq_all = __reduce_add_sync(kFull, eq_w);
      if (lane == 0) s_total[0] = gt_all, s_total[1] = eq_all;
    }
    cl.sync();
#pragma unroll
    for (int x = 0; x < kMaxCluster - 1; ++x)
      if (x < rank) {
        const int *o = cl.map_shared_rank(s_total, x);
        gt_at += o[0], eq_at += o[1];
      }
  }
  const uint32_t below = (1u << lane) - 1u;
  each([&](int i, uint4 x) {
    const uint32_t k[4] = {x.x, x.y, x.z, x.w};
    int mine = 0, gts = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t m = __ballot_sync(kFull, k[e] > T);
      gts += __popc(m & below);
      mine += __popc(m);
    }
    int gr = gt_at + gts;
    if (__any_sync(kFull, k[0] == T || k[1] == T || k[2] == T || k[3] == T)) {
      int eqs = 0, all = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t m = __ballot_sync(kFull, k[e] == T);
        eqs += __popc(m & below);
        all += __popc(m);
      }
      int er = eq_at + eqs;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (k[e] > T || (k[e] == T && er < need)) kept[gr + min(er, need)] = i + e;
        gr += k[e] > T, er += k[e] == T;
      }
      eq_at += all;
    } else {
      gr += min(eq_at, need);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (k[e] > T) kept[gr++] = i + e;
    }
    gt_at += mine;
  });
  if (lead && h == 0) p.new_lens[r] = n;
  if (ranks > 1) cl.sync();  // no block leaves while another reads its shared memory
}

// ----------------------------------------------------------------------------- compaction
constexpr int kCmpThreads = 256;  // also the rows of a tile
constexpr int kCmpFlight = 8;     // 16-byte pieces in flight per thread

// Where row t of a cache lives: (page, slot) as page * PAGE + slot, or -1 without a valid page.
__device__ __forceinline__ int64_t row_place(const CompactParams &p, const int32_t *idx, int start,
                                             int count, int t) {
  const int id = t >= 0 && t / PAGE < count ? idx[start + t / PAGE] : -1;
  if (id < 0 || id >= p.num_pages) {
    if (p.status) atomicOr(reinterpret_cast<int *>(p.status), HPA_STATUS_BAD_PAGE);
    return -1;
  }
  return static_cast<int64_t>(id) * p.Hkv * PAGE + t % PAGE;
}

// A request's two page tables: its own, and the one the new cache goes to.
struct Places {
  const int32_t *src_idx, *dst_idx;
  int ps, pn, ds, dn;
  __device__ Places(const CompactParams &p, int r, bool in_place) {
    src_idx = p.page_indices;
    ps = p.page_indptr[r], pn = p.page_indptr[r + 1] - ps;
    dst_idx = in_place ? src_idx : p.dst_indices;
    ds = in_place ? ps : p.dst_indptr[r];
    dn = in_place ? pn : p.dst_indptr[r + 1] - ds;
  }
};

// To other pages.  Block (pair, slice, z): tiles z, z + gridDim.z, ... of 256 rows of one
// (request, head), columns [slice * lanes, (slice + 1) * lanes) of 16 bytes of K and V.  A
// thread finds one row's source and destination (the next tile's while this one moves: an
// index, a page id and the row are three dependent reads), then the block moves the tile
// in batches of 8 pieces per thread.
// Moving the rows in the selection's own blocks, to overlap one request's selection with
// another's move, was slower: 108 -> 121 and 263 -> 302 us (32 x 8192 cut to 2048, 64 x
// 24000 to 4096), the blocks that a selection wants being too few and too large to move.
__global__ void __launch_bounds__(kCmpThreads)
    evict_copy_kernel(const CompactParams p, int lanes) {
  __shared__ int64_t s_src[kCmpThreads], s_dst[kCmpThreads];
  const int r = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv, tid = threadIdx.x;
  pdl_wait();  // the selection is usually the kernel just before
  const int n = p.new_lens[r];
  if (n <= 0 || n > p.kept_stride) return;  // left as it is (new_lens -1: a bad request)
  const int32_t *kept = p.kept + static_cast<int64_t>(blockIdx.x) * p.kept_stride;
  const Places at(p, r, false);
  const int row_ts = p.row_bytes / 16, col = blockIdx.y * lanes;
  const int sh = 31 - __clz(lanes);  // lanes is a power of two
  const int64_t head = static_cast<int64_t>(h) * PAGE;
  const int64_t step = static_cast<int64_t>(gridDim.z) * kCmpThreads;

  int64_t src = -1, dst = -1;
  auto resolve = [&](int64_t t) {  // rows that are not there have src -1
    src = dst = -1;
    if (t < n) {
      src = row_place(p, at.src_idx, at.ps, at.pn, kept[t]);
      dst = row_place(p, at.dst_idx, at.ds, at.dn, static_cast<int>(t));
      if (dst < 0) src = -1;
    }
  };
  int64_t t0 = static_cast<int64_t>(blockIdx.z) * kCmpThreads;
  resolve(t0 + tid);
  for (; t0 < n; t0 += step) {
    __syncthreads();  // the previous tile's places are no longer needed
    s_src[tid] = src < 0 ? -1 : src + head;
    s_dst[tid] = dst + head;
    if (p.acc && blockIdx.y == 0 && src >= 0) p.acc[dst + head] = p.acc[src + head];
    __syncthreads();
    if (t0 + step < n) resolve(t0 + step + tid);
    const int pieces = static_cast<int>(n - t0 < kCmpThreads ? n - t0 : kCmpThreads) << sh;
#pragma unroll 1
    for (int kv = 0; kv < 2; ++kv) {
      uint4 *pool = static_cast<uint4 *>(kv ? p.v_pool : p.k_pool);
      for (int b = 0; b < pieces; b += kCmpFlight * kCmpThreads) {
        uint4 x[kCmpFlight];
#pragma unroll
        for (int u = 0; u < kCmpFlight; ++u) {
          const int e = b + u * kCmpThreads + tid;
          const int64_t from = e < pieces ? s_src[e >> sh] : -1;
          if (from >= 0) x[u] = pool[from * row_ts + col + (e & (lanes - 1))];
        }
#pragma unroll
        for (int u = 0; u < kCmpFlight; ++u) {
          const int e = b + u * kCmpThreads + tid;
          if (e < pieces && s_src[e >> sh] >= 0)
            pool[s_dst[e >> sh] * row_ts + col + (e & (lanes - 1))] = x[u];
        }
      }
    }
  }
}

// In place.  A cluster takes the rows of one (request, head) and column slice in order, a
// step of `rows` rows for each of its blocks at a time: every block reads its rows of K, V
// and the weights into registers, the cluster's barrier follows, and only then are they
// written.  A row that is written at t is the source of no row after this step (kept[t'] >=
// t' > t), and the sources of this step have been read.
__global__ void __launch_bounds__(kCmpThreads, 2)
    evict_shift_kernel(const CompactParams p, int lanes, int rows) {
  __shared__ int64_t s_src[kCmpThreads], s_dst[kCmpThreads];
  cg::cluster_group cl = cg::this_cluster();
  const int r = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv, tid = threadIdx.x;
  pdl_wait();
  const int n = p.new_lens[r];
  if (n <= 0 || n > p.kept_stride) return;  // the whole cluster
  const int32_t *kept = p.kept + static_cast<int64_t>(blockIdx.x) * p.kept_stride;
  const Places at(p, r, true);
  const int row_ts = p.row_bytes / 16, col = blockIdx.y * lanes;
  const int sh = 31 - __clz(lanes);
  const int64_t head = static_cast<int64_t>(h) * PAGE;
  const int64_t step = static_cast<int64_t>(cl.num_blocks()) * rows;
  const int pieces = rows << sh;  // per pool, at most 8 per thread
  uint4 *const kp = static_cast<uint4 *>(p.k_pool), *const vp = static_cast<uint4 *>(p.v_pool);

  int64_t src = -1, dst = -1;
  auto resolve = [&](int64_t t) {  // rows that stay where they are, and none, have src -1
    src = dst = -1;
    if (tid < rows && t < n) {
      const int k = kept[t];
      if (k != t) {
        src = row_place(p, at.src_idx, at.ps, at.pn, k);
        dst = row_place(p, at.dst_idx, at.ds, at.dn, static_cast<int>(t));
        if (dst < 0) src = -1;
      }
    }
  };
  int64_t t0 = static_cast<int64_t>(cl.block_rank()) * rows;
  resolve(t0 + tid);
  for (int64_t first = 0; first < n; first += step, t0 += step) {
    __syncthreads();  // the previous step's places are no longer needed
    s_src[tid] = src < 0 ? -1 : src + head;
    s_dst[tid] = dst + head;
    const int64_t as = src + head, ad = dst + head;
    const bool weigh = p.acc && blockIdx.y == 0 && src >= 0;
    const float a = weigh ? p.acc[as] : 0.f;
    __syncthreads();
    uint4 k[kCmpFlight], v[kCmpFlight];
#pragma unroll
    for (int u = 0; u < kCmpFlight; ++u) {
      const int e = u * kCmpThreads + tid;
      const int64_t from = e < pieces ? s_src[e >> sh] : -1;
      if (from >= 0) {
        k[u] = kp[from * row_ts + col + (e & (lanes - 1))];
        v[u] = vp[from * row_ts + col + (e & (lanes - 1))];
      }
    }
    resolve(t0 + step + tid);
    cl.sync();
    if (weigh) p.acc[ad] = a;
#pragma unroll
    for (int u = 0; u < kCmpFlight; ++u) {
      const int e = u * kCmpThreads + tid;
      if (e < pieces && s_src[e >> sh] >= 0) {
        const int64_t to = s_dst[e >> sh] * row_ts + col + (e & (lanes - 1));
        kp[to] = k[u];
        vp[to] = v[u];
      }
    }
  }
}

}  // namespace

cudaError_t launch_evict_select(const EvictParams &p, cudaStream_t s) {
  static int configured[64] = {0};
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSelSmem);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = 1;
  }
  // Blocks per (request, head).  The lengths are on the device; the launch goes by the pool's
  // average and not by the budget, which says nothing of the length (one request of 196608
  // cut to 64 by one block each: 138 us, by eight 27), and blocks that a shorter request does
  // not need leave.  More blocks as long as the clusters find room on the GPU together and a
  // block has kMinKeys; past that room (up to 1.4 times) only where the weights are far more
  // than the blocks hold (160 pairs of 196608: 171 us in two blocks each, 195 in one; 160 of
  // 55000: 60 and 56; 64 of 191721: 74 in eight, 58 in four; 256 of 30000: 46 in two, 33 in
  // one).
  const int64_t pairs = static_cast<int64_t>(p.B) * p.Hkv;
  const int64_t share = p.num_pages * PAGE / p.B, room = kSelBlocks * sms;
  const int64_t held = kBlockPages * PAGE;
  int ranks = 1;
  while (ranks < kMaxCluster &&
         ((pairs * ranks * 2 <= room && ranks * kMinKeys < share) ||
          (pairs * ranks * 2 <= room * 7 / 5 && ranks * held * 3 < share)))
    ranks *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(pairs * ranks));
  cfg.blockDim = dim3(kSelThreads);
  cfg.dynamicSmemBytes = kSelSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  EvictParams q = p;
  // More blocks than the GPU holds: the longest requests first, or one of them begins last
  // (64 x 24000, lognormal: 74 -> 65 us; 58 -> 61 if all are of one length).
  q.longest_first = p.B > 1 && p.B <= kSelThreads / 4 && pairs * ranks > room;
  return cudaLaunchKernelEx(&cfg, evict_select_kernel, q);
}

cudaError_t launch_evict_compact(const CompactParams &p, cudaStream_t s) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int64_t pairs = static_cast<int64_t>(p.B) * p.Hkv;
  const int row_ts = p.row_bytes / 16;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kCmpThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int slices = 1;
  if (p.dst_indptr != nullptr) {
    // rows: as many tiles as the kept lists can hold, up to 32 blocks per SM (8 per SM: 174
    // -> 183 us for 512 pairs of 4096 rows); with few of them, columns of 64 bytes or more
    const int64_t tiles = (p.kept_stride + kCmpThreads - 1) / kCmpThreads;
    const int64_t most = 1 + 32 * static_cast<int64_t>(sms) / pairs;
    const int split = static_cast<int>(tiles < most ? tiles : most);
    while (slices < row_ts / 4 && pairs * split * slices < 2 * sms) slices *= 2;
    cfg.gridDim = dim3(static_cast<unsigned>(pairs), slices, split);
    return cudaLaunchKernelEx(&cfg, evict_copy_kernel, p, row_ts / slices);
  }
  // Blocks of a cluster as far as the kept lists have rows for them: 8 with few pairs (16384
  // rows of 8 pairs: 28 us in 8, 42 in 4, 147 in one), 4 where these fill the GPU (512
  // pairs of 4096 rows: 187 us in 4, 200 in 8, 192 in one); then columns of 32 bytes or
  // more.
  auto rows_of = [&](int lanes) { return lanes > kCmpFlight ? kCmpThreads / 2 : kCmpThreads; };
  int ranks = 1;
  while (ranks < (pairs * 4 < 2 * sms ? kMaxCluster : 4) &&
         static_cast<int64_t>(ranks) * rows_of(row_ts) < p.kept_stride)
    ranks *= 2;
  while (slices < row_ts / 2 && pairs * slices * ranks < 2 * sms) slices *= 2;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = ranks;
  cfg.numAttrs = 2;
  cfg.gridDim = dim3(static_cast<unsigned>(pairs), slices, ranks);
  const int lanes = row_ts / slices;
  return cudaLaunchKernelEx(&cfg, evict_shift_kernel, p, lanes, rows_of(lanes));
}

}  // namespace hpa
