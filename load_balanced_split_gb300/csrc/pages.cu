// Page tables and slot maps from request lengths, on the device (hpa_assign_pages).
//
// With n_r = ceil(L_r / 64) the pages that request r is to have and h_r those that it holds:
//   back_r = max(h_r - n_r, 0),   take_r = max(n_r - h_r, 0),
//   the returned pages go on the free stack in the order of the requests (and of their pages),
//   request r is served if take_r = 0 or sum_{q <= r} take_q <= free + sum back,
//   and its i-th new page is the stack's entry free + sum back - 1 - (sum_{q < r} take_q + i).
// All of it follows from running sums over the requests, so the result is the same on every run.
//
// Two launches (one for a few short requests).  scan_kernel, one block, makes the sums and a record
// per request; fill_kernel, a few blocks per request, moves page ids and writes the token slots.  A
// returned page that is given out in the same step is read from the row that returns it, so no
// block of the second waits for another.  Both are bound by latency, of launches and of loads that
// follow from one another (the largest case reads and writes 5 MB): one request takes 3.9 us, 128
// that take a token each 6.3 to 7.2, 1000 with chunks of 256 tokens 13, 4000 with a token each 26.
// The second starts while the first still runs (programmatic dependent launch) and waits for its
// records.  One block for the sums because a step of 1000 requests is then one load and two scans,
// without a meeting of blocks; its scattered accesses (a row per request) are what it spends most
// on, so the owners of rows are in shared memory where they fit (1000 requests 17 -> 13 us with
// records in two arrays, 4000 60 -> 26).
#include <climits>

#include "hpa_internal.cuh"

namespace hpa {
namespace {

constexpr int kFillThreads = 256;

// What fill_kernel needs of a request, two 16-byte words in arrays of their own (a warp's then lie
// together).
struct __align__(16) Pages {
  int row;     // its row of the table, -1: none
  int held;    // pages it holds before the step
  int pages;   // pages it holds after the step
  int served;  // its tokens get slots
};
struct __align__(16) Places {
  int take_off;  // pages that requests before it take
  int back_off;  // pages that requests before it return
  int tok_off;   // tokens of the requests before it
  int len;
};

// Workspace: totals (16 words), Pages and Places of each request, the owner of each row.
enum { WS_FREE = 0, WS_AVAIL, WS_TOKENS, WS_HEADER_WORDS = 16 };
constexpr int kSharedRows = 8192;  // up to so many rows have their owners in shared memory

__device__ __forceinline__ Pages *pages_at(const AssignParams &p) {
  return reinterpret_cast<Pages *>(p.ws + WS_HEADER_WORDS);
}
__device__ __forceinline__ Places *places_at(const AssignParams &p) {
  return reinterpret_cast<Places *>(p.ws + WS_HEADER_WORDS) + p.B;
}

struct Sum2 {
  long long a, b;
};

// Inclusive scan of pairs over the block; `total` receives the sums.
__device__ Sum2 block_scan2(Sum2 v, Sum2 *wbuf, Sum2 &total) {
  const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5, warps = blockDim.x >> 5;
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, v.a, o);
    const long long b = __shfl_up_sync(0xffffffffu, v.b, o);
    if (lane >= o) v.a += a, v.b += b;
  }
  if (warps == 1) {
    total.a = __shfl_sync(0xffffffffu, v.a, 31);
    total.b = __shfl_sync(0xffffffffu, v.b, 31);
    return v;
  }
  if (lane == 31) wbuf[wid] = v;
  __syncthreads();
  if (wid == 0) {
    Sum2 s = lane < warps ? wbuf[lane] : Sum2{0, 0};
    for (int o = 1; o < 32; o <<= 1) {
      const long long a = __shfl_up_sync(0xffffffffu, s.a, o);
      const long long b = __shfl_up_sync(0xffffffffu, s.b, o);
      if (lane >= o) s.a += a, s.b += b;
    }
    if (lane < warps) wbuf[lane] = s;
  }
  __syncthreads();
  if (wid > 0) v.a += wbuf[wid - 1].a, v.b += wbuf[wid - 1].b;
  total = wbuf[warps - 1];
  __syncthreads();
  return v;
}

__device__ __forceinline__ int clip(long long x) {
  return x > INT_MAX ? INT_MAX : static_cast<int>(x);
}

// Page i of a request after the step: from its own row, or from the stack.
__device__ __forceinline__ int page_of(const AssignParams &p, const Pages &x, const Places &at,
                                       int i, int free, int avail) {
  if (i < x.held) return p.table[static_cast<int64_t>(x.row) * p.stride + i];
  const int v = avail - 1 - (at.take_off + i - x.held);
  if (v < free) return p.free_pages[v];
  // returned in this step: the last request with back_off <= v - free that returns any
  const int want = v - free;
  int lo = 0, hi = p.B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (places_at(p)[mid].back_off <= want) lo = mid;
    else hi = mid - 1;
  }
  const Pages q = pages_at(p)[lo];
  return p.table[static_cast<int64_t>(q.row) * p.stride + q.pages + want -
                 places_at(p)[lo].back_off];
}

// What follows from the sums for one request, by `step` threads of which this is number `first`.
__device__ __forceinline__ void fill_request(const AssignParams &p, int r, int first, int step) {
  const int free = p.ws[WS_FREE], avail = p.ws[WS_AVAIL];
  const Pages x = pages_at(p)[r];
  const Places at = places_at(p)[r];
  int bad = 0;
  // the request's page list, and its new pages into the table
  const int begin = p.page_indptr[r], room = p.page_indptr[r + 1] - begin;
  int32_t *row = p.table + static_cast<int64_t>(x.row < 0 ? 0 : x.row) * p.stride;
  for (int i = first; i < x.pages; i += step) {
    const int id = page_of(p, x, at, i, free, avail);
    if (id < 0 || id >= p.num_pages) bad = HPA_STATUS_BAD_PAGE;
    if (i >= x.held) row[i] = id;
    if (i < room) p.page_indices[begin + i] = id;
  }
  // the pages it returns
  for (int i = x.pages + first; i < x.held; i += step) {
    const long long to = static_cast<long long>(free) + at.back_off + i - x.pages;
    if (to < p.num_pages) p.free_pages[to] = row[i];
    else bad |= HPA_STATUS_BAD_MAP;  // more pages than there are: a damaged state
  }
  if (p.new_tokens) {
    const int nt = p.new_tokens[r], offset = p.pos_offset ? p.pos_offset[r] : 0;
    const int end = min(max(nt, 0), max(p.max_tokens - at.tok_off, 0));
    const long long before = static_cast<long long>(at.len) - nt;  // of a bad request below 0
    for (int t = first; t < end; t += step) {
      const int pos = static_cast<int>(max(before + t, 0ll));
      long long slot = -1;
      if (x.served) {
        const int id = page_of(p, x, at, pos / PAGE, free, avail);
        if (id >= 0 && id < p.num_pages) slot = static_cast<long long>(id) * PAGE + pos % PAGE;
      }
      p.slots[at.tok_off + t] = slot;
      const long long text = static_cast<long long>(pos) + offset;
      p.positions[at.tok_off + t] =
          static_cast<int32_t>(text > INT_MAX ? INT_MAX : text < INT_MIN ? INT_MIN : text);
    }
  }
  if (bad && p.status) atomicOr(reinterpret_cast<int *>(p.status), bad);
}

// The places behind the last token.
__device__ __forceinline__ void fill_rest(const AssignParams &p, long long first, long long step) {
  if (!p.new_tokens) return;
  for (long long t = p.ws[WS_TOKENS] + first; t < p.max_tokens; t += step) {
    p.slots[t] = -1;
    p.positions[t] = 0;
  }
}

__global__ void __launch_bounds__(kFillThreads) fill_kernel(const AssignParams p) {
  pdl_wait();
  const int first = blockIdx.y * kFillThreads + threadIdx.x, step = gridDim.y * kFillThreads;
  fill_request(p, blockIdx.x, first, step);
  fill_rest(p, static_cast<long long>(blockIdx.x) * step + first,
            static_cast<long long>(gridDim.x) * step);
}

// What a request says and has, its loads started together.
struct Request {
  int row, L, nt, held;
};
__device__ __forceinline__ Request load_request(const AssignParams &p, int r) {
  Request q;
  q.row = p.rows ? p.rows[r] : r;
  q.L = p.seq_lens[r];
  q.nt = p.new_tokens ? p.new_tokens[r] : 0;
  q.held = q.row >= 0 && q.row < p.num_rows ? p.held_in[q.row] : 0;
  return q;
}

// spread: threads a request for the whole step in this one block; 0: fill_kernel follows.
template <bool kOwnersShared>
__global__ void __launch_bounds__(1024) scan_kernel(const AssignParams p, int spread) {
  if (spread == 0) pdl_launch_dependents();  // fill_kernel waits for this grid before it reads
  pdl_wait();
  __shared__ Sum2 wbuf[32];
  __shared__ int s_bad;
  extern __shared__ int32_t s_owner[];
  const int tid = threadIdx.x, n = blockDim.x;
  Pages *pages_ws = pages_at(p);
  Places *places_ws = places_at(p);
  int32_t *owner =
      kOwnersShared ? s_owner : p.ws + WS_HEADER_WORDS + 8 * static_cast<int64_t>(p.B);
  if (tid == 0) s_bad = 0;
  int free = *p.free_in;
  Request req = {-1, 0, 0, 0};
  if (tid < p.B) req = load_request(p, tid);
  __syncthreads();
  if (free < 0 || free > p.num_pages) {  // a damaged state: nothing is given out
    if (tid == 0) atomicOr(&s_bad, HPA_STATUS_BAD_MAP);
    free = free < 0 ? 0 : p.num_pages;
  }
  if (p.rows) {  // a row listed twice belongs to the first request that lists it
    for (int r = tid; r < p.B; r += n) {
      const int row = r == tid ? req.row : p.rows[r];
      if (row >= 0 && row < p.num_rows) owner[row] = INT_MAX;
    }
    __syncthreads();
    for (int r = tid; r < p.B; r += n) {
      const int row = r == tid ? req.row : p.rows[r];
      if (row >= 0 && row < p.num_rows) atomicMin(owner + row, r);
    }
    if (!kOwnersShared) __threadfence_block();
    __syncthreads();
  }
  // returned and wanted pages
  Sum2 carry = {0, 0}, total;
  Pages mine = {-1, 0, 0, 0};
  Places mine_at = {0, 0, 0, 0};
  for (int base = 0; base < p.B; base += n) {
    const int r = base + tid;
    Pages x = {-1, 0, 0, 0};
    Places at = {0, 0, 0, 0};
    long long back = 0, take = 0;
    if (r < p.B) {
      if (base > 0) req = load_request(p, r);
      int row = req.row, held = req.held;
      const int L = req.L, nt = req.nt;
      int bad = 0;
      if (row < 0 || row >= p.num_rows ||
          (p.rows && *reinterpret_cast<volatile int32_t *>(owner + row) != r)) {
        bad = HPA_STATUS_BAD_MAP;
        row = -1;
        held = 0;
      }
      if (held < 0 || held > p.stride) {
        bad |= HPA_STATUS_BAD_MAP;
        row = -1;
        held = 0;
      }
      if (L < 0 || nt < 0 || nt > L) bad |= HPA_STATUS_BAD_SEQLEN;
      const int need = L <= 0 ? 0 : (L - 1) / PAGE + 1;
      if (need > p.stride) bad |= HPA_STATUS_OVERFLOW;
      if (bad) atomicOr(&s_bad, bad);
      x.row = row;
      x.held = held;
      x.pages = bad ? held : need;
      x.served = !bad;
      at.len = L;
      back = max(held - x.pages, 0);
      take = max(x.pages - held, 0);
    }
    const Sum2 s = block_scan2({back, take}, wbuf, total);
    if (r < p.B) {
      at.back_off = clip(carry.a + s.a - back);
      at.take_off = clip(carry.b + s.b - take);
      if (p.B <= n) {  // one round: they stay in registers
        mine = x;
        mine_at = at;
      } else {
        pages_ws[r] = x;
        places_ws[r] = at;
      }
    }
    carry.a += total.a;
    carry.b += total.b;
  }
  const long long avail = free + carry.a;
  // who is served, their pages and tokens
  Sum2 done = {0, 0};
  long long given = 0;
  for (int base = 0; base < p.B; base += n) {
    const int r = base + tid;
    long long pages = 0, tokens = 0;
    Pages x = mine;
    Places at = mine_at;
    int nt = req.nt;
    if (r < p.B) {
      if (p.B > n) {
        x = pages_ws[r];
        at = places_ws[r];
        nt = p.new_tokens ? p.new_tokens[r] : 0;
      }
      const int take = x.pages - x.held;
      if (take > 0 && static_cast<long long>(at.take_off) + take > avail) {
        x.pages = x.held;
        x.served = 0;
        atomicOr(&s_bad, HPA_STATUS_NO_PAGES);
      }
      if (take > 0 && x.served) given = max(given, static_cast<long long>(at.take_off) + take);
      pages = x.pages;
      tokens = max(nt, 0);
      if (x.row >= 0) p.held_out[x.row] = x.pages;
    }
    const Sum2 s = block_scan2({pages, tokens}, wbuf, total);
    if (r < p.B) {
      at.tok_off = clip(done.b + s.b - tokens);
      pages_ws[r] = x;
      places_ws[r] = at;
      // what passes the list's end is cut, for the attention calls trust these offsets
      const long long end = done.a + s.a;
      p.page_indptr[r + 1] = static_cast<int32_t>(end < p.indices_cap ? end : p.indices_cap);
    }
    done.a += total.a;
    done.b += total.b;
  }
  // requests are served from the first on while the pages last: the last one's end is the sum
  for (int o = 16; o > 0; o >>= 1) given = max(given, __shfl_xor_sync(0xffffffffu, given, o));
  if ((tid & 31) == 0) wbuf[tid >> 5].a = given;
  __syncthreads();
  if (tid == 0) {
    for (int w = 1; w < (n >> 5); ++w) given = max(given, wbuf[w].a);
    if (done.a > p.indices_cap || (p.new_tokens && done.b > p.max_tokens))
      s_bad |= HPA_STATUS_OVERFLOW;
    p.page_indptr[0] = 0;
    const long long left = avail - given;
    *p.free_out = static_cast<int32_t>(left < p.num_pages ? left : p.num_pages);
    p.ws[WS_FREE] = free;
    p.ws[WS_AVAIL] = clip(avail);
    p.ws[WS_TOKENS] = clip(done.b);
    if (p.status && s_bad) atomicOr(reinterpret_cast<int *>(p.status), s_bad);
  }
  if (spread > 0) {
    __syncthreads();
    if (tid / spread < p.B) fill_request(p, tid / spread, tid % spread, spread);
    fill_rest(p, tid, n);
  }
}

}  // namespace

int64_t assign_workspace_words(int64_t B, int64_t num_rows) {
  return WS_HEADER_WORDS + 8 * B + num_rows;
}

cudaError_t launch_assign_pages(const AssignParams &p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.stream = s;
  cfg.gridDim = dim3(1);
  // A few requests of short lists are done in the first launch, whose one block then has no more
  // than 4 places a thread to fill: one of 900 tokens 4.3 -> 3.8 us, and 2 of the 12 that the host
  // takes.  (With 8 to 12 a thread, 8 requests of 8192 tokens 4.2 -> 4.9 and 32 4.9 -> 8.1; with
  // 32 requests and 3 a thread 5.4 -> 6.0.)
  int slots = 1;
  while (slots < p.B) slots *= 2;
  const int threads = slots <= 8 ? 256 : 32 * slots;
  const int spread = slots <= 16 && p.stride <= 4 * (threads / slots) &&
                             p.max_tokens <= 4 * (threads / slots)
                         ? threads / slots
                         : 0;
  cfg.blockDim = dim3(spread ? threads : p.B >= 1024 ? 1024 : (p.B + 31) / 32 * 32);
  const bool shared = p.rows && p.num_rows <= kSharedRows;
  cfg.dynamicSmemBytes = shared ? 4 * p.num_rows : 0;
  cudaError_t e = shared ? cudaLaunchKernelEx(&cfg, scan_kernel<true>, p, spread)
                         : cudaLaunchKernelEx(&cfg, scan_kernel<false>, p, spread);
  if (e != cudaSuccess || spread) return e;
  cfg.dynamicSmemBytes = 0;
  const int y = (p.stride + 4 * kFillThreads - 1) / (4 * kFillThreads);
  cfg.gridDim = dim3(p.B, y < 64 ? y : 64);
  cfg.blockDim = dim3(kFillThreads);
  return cudaLaunchKernelEx(&cfg, fill_kernel, p);
}

}  // namespace hpa
