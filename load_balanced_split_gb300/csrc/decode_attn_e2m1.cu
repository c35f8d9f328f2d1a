// Split-KV GQA decode attention over a paged KV cache held in 4 bits (HPA_KV_E2M1), driven by
// the same task maps as the 16- and 8-bit kernels.
//
// A page of one KV head is one block of 4608 bytes: 64 rows of 64 bytes of E2M1 codes (the even
// element of a pair in the low nibble), then 64 x 8 E4M3 scales, one for every 16 elements of a
// row.  With c the code's value, b its block's scale and s_h the head's scale,
//   x = c * b * s_h,   out = sum_i softmax(sm_scale * q . k_i) v_i   over the keys a token sees.
//
// What bounds it: at 4.5 bits an element the DRAM delivers 42 elements a clock to each SM, so
// the widening to f16 has about three instruction slots an element before it, not the memory,
// is what the kernel waits for; and an MMA takes 8 of them, in which little else issues (an FFMA
// beside it costs 1 more, a conversion half of one).  With 8 rows the memory still sets the pace
// (5.6 TB/s over 32 x 8192 keys, starts and ends included), with 16 the slots (4.7 TB/s).  The
// layout:
//  * the products run as m16n8k16 MMAs with the KEYS (S = K Q^T) and the HEAD DIMS (O^T = V^T P^T)
//    as the 16 rows and 8 query rows as the 8 columns, so an MMA takes 256 cache elements for 8
//    query rows, where queries on the 16 rows would take 128 and leave half of the tile empty
//    (9 to 16 rows fill it and stand there in the first product);
//  * a thread reads 32 consecutive dims of a key with one 16-byte load and widens two codes per
//    conversion; the head dims are permuted alike in Q and K, so nothing is shuffled.  The
//    product of a code and its block scale has 6 significant bits and is exact in f16;
//  * V needs its pairs along the keys.  Two keys' words are interleaved by nibbles (four logic
//    operations for 16 elements), so that a converted byte already is a pair of keys;
//  * P moves from the first product's accumulator layout to the second's operand by movmatrix;
//  * the softmax's running maximum moves only when a score passes it by 2^8 (as in the 8-bit
//    kernel), so a page costs one vote and no exchange of maxima;
//  * a warp takes 32 keys of a page at a time, with one wait, vote and release.  One producer
//    warp keeps a ring of pages in flight with bulk copies, two a page (codes and scales lie
//    together).
// Sums, softmax statistics and outputs are fp32.  Queries enter as f16, each row scaled by a power
// of two that puts its largest element into [2^14, 2^15) (exact down to 2^-28 of it), and the
// probabilities are rounded to f16 as the second product's operand: 2^-11 of each, and of those
// below 2^-21 of the row's largest 2^-32 of that one.
//
// Windows with sink tokens (WIN): the producer maps the map's compact pages to real ones
// (WinSpan), and pages at the window's ends mask by position.  Pages without a hidden key run a
// copy of the loop without masks.  A code cannot be NaN but a block scale can: V scales of keys
// that no token sees are taken as zero, and a key that some tokens see and others do not marks
// the rows that see it alone if its scales hold a NaN.
#include <math_constants.h>

#include <type_traits>

#include "e2m1.cuh"

namespace hpa {
namespace {

// Query rows in tiles of 8 columns (1 or 2), and what was measured best for each number of them, in
// us (32 x 8192 keys with 8 rows and 128 windows of 4096 with 16 sinks; 64 x 20000 with 16 rows and
// 64 x 8000 in a window of 2000):
//   1 tile:  4 consumer warps in pairs that share a page, three CTAs per SM at 128 registers, 59
//            and 111 (5 warps with a page each, two CTAs: 62 and 127; four to a page: 72 and 127);
//   2 tiles: the same pairs, two CTAs at 168 registers, query fragments in shared memory, 332
//            and 48 (a page each gains 1 %, but takes 95 in the window: a segment's last pages,
//            and its start, then leave warps idle for a page's time; 12 warps in one CTA 315
//            for 317 on 64 requests of equal length, and 63 for 48 in the window).
// The warps of an SM come in fours: with 10 in a CTA the schedulers that have three set the pace.
// More rows go to decode_attn_e2m1_tc.cu (as 3 tiles here, 8 warps at 232 registers, 13 x 20011
// keys with 20 rows took 102 where it takes 92).
template <int NT>
struct Cfg {
  static constexpr int kWarps = 4;                   // consumer warps
  static constexpr int kShare = 2;                   // warps of a team, which share a page
  static constexpr int kTeams = kWarps / kShare;
  static constexpr int kBlocks = NT == 1 ? 3 : 2;    // CTAs per SM
  static constexpr int kStages = NT == 1 ? 6 : 8;
  // A team meets the same stages again.  Copies may land out of order, so a warp that came to a
  // stage whose page before it, another team's, had not landed would take that page's phase for
  // the end of its own.
  static_assert(kWarps % kShare == 0 && kStages % kTeams == 0, "each stage belongs to one team");
  static constexpr int kThreads = (kWarps + 1) * 32;
  static constexpr int kMine = 4 / kShare;           // a page's groups of 16 keys for a warp
  static constexpr int kGroups = 2;                  // groups that share a softmax step
  static constexpr int kSide = NT == 1 ? 1 : 2;      // groups whose MMA chains run side by side
  // With 16 rows they fill the MMA's 16: S = Q K^T has P in the layout that the second product
  // wants, without movmatrix, and a lane has 2 rows' statistics, not 4 (351 -> 343 us).  The query
  // fragments lie in shared memory then.
  static constexpr bool kRowsOnM = NT == 2;
  static constexpr int kStats = kRowsOnM ? 2 : 2 * NT;
};
constexpr int kStageBytes = 2 * kUnit;
constexpr int kQRowBytes = 272;  // 256 of a query row, padded against bank conflicts
constexpr int kMergeStride = HEAD_DIM + 4;

template <int NT>
struct Smem {
  static constexpr int kWarps = Cfg<NT>::kWarps, kStages = Cfg<NT>::kStages;
  static constexpr int kRows = 8 * NT;
  static constexpr int kBufs = 2;  // merge buffers
  static constexpr int kQSlot = kRows * kQRowBytes;
  static constexpr int kMerge = kStages * kStageBytes;               // float[kBufs][kRows][stride]
  static constexpr int kStats = kMerge + kBufs * kRows * kMergeStride * 4;  // m, l: [warps][kRows]
  static constexpr int kQ = kStats + 2 * kWarps * kRows * 4;         // two query slots
  static constexpr int kInfo = kQ + 2 * kQSlot;                      // int4[2]
  static constexpr int kFrag = kInfo + 2 * 16;                       // query fragments, factors
  // full[stages], empty[stages], qfull[2], qempty[2]
  static constexpr int kBars = kFrag + (Cfg<NT>::kRowsOnM ? NT * 8 * 256 + kRows * 4 : 0);
  static constexpr int kFlag = kBars + (2 * kStages + 4) * 8;
  static constexpr int kAlloc = kFlag + 16;
};

// Which of a group's 8 keys stands at index k of the MMAs' key dimension: the keys that the
// four lanes of a quad read together for V (k = 0, 2, 4, 6 and 1, 3, 5, 7) then lie in both
// halves of the 128 bytes that shared memory serves at once.
__device__ __forceinline__ constexpr int key_at(int k) { return k ^ ((k >> 1) & 1); }

__device__ __forceinline__ void sts32(uint32_t addr, uint32_t a) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(a) : "memory");
}

// Transpose of an 8x8 matrix of 16-bit elements held a row of pairs per lane quad.
__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ float absmax8_bf16(uint4 v) {
  float m = 0.f;
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(w[i] << 16)),
                       fabsf(__uint_as_float(w[i] & 0xffff0000u))));
  return m;
}

// ----------------------------------------------------------------------------- producer
// One warp.  Reading a segment's row, its request's page list and its page ids are round trips to
// L2 that follow from one another, so a lane each reads the rows of 32 segments at once, and the
// next 32 page ids are on their way while the last are used.  A lane copies the page whose id it
// holds, and a segment's query rows are bulk copies too, so that the warp waits for nothing but
// stages to become free.  (With each segment's loads before its pages this warp was what the others
// waited for: 343 us where this takes 335, 64 x 20000 keys with 16 rows, and 52 for 48 in a window
// of 2000.)
template <int NT, bool WIN>
__device__ void producer(const AttnParams &p, const uint8_t *k_pool, const uint8_t *v_pool,
                         uint8_t *smem, const MapHead &head) {
  using S = Smem<NT>;
  constexpr int kStages = S::kStages;
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const uint32_t base = smem_u32(smem);
  const uint32_t full0 = base + S::kBars, empty0 = full0 + 8 * kStages;
  const uint32_t qfull0 = empty0 + 8 * kStages, qempty0 = qfull0 + 16;
  const volatile int *abort_flag = reinterpret_cast<const volatile int *>(smem + S::kFlag);
  const uint64_t pol = l2_policy_evict_first();
  const int rows = group_rows(p), rb = row_base(p);
  // where this lane's query row lies behind its request's first
  const int64_t q_at =
      (static_cast<int64_t>((rb + lane) / p.G) * p.Hq + h * p.G + (rb + lane) % p.G) * HEAD_DIM;
  int n0 = 0, nq = 0;  // pages and segments on their way
  bool ok = true;
  for (int s0 = head.s_begin; s0 < head.s_end && ok; s0 += 32) {
    Seg mine = {0, 0, 0, 0, 0, 0};
    int list = 0, listed = 0;  // its request's page list
    if (s0 + lane < head.s_end) {
      mine = read_seg<WIN>(p, s0 + lane, head.tile, true);
      list = p.page_indptr[mine.r];
      listed = p.page_indptr[mine.r + 1] - list;
    }
    struct Walk {
      Seg f;
      int list, listed;
      WinSpan win;
    };
    auto segment = [&](int j) {
      Walk x = {};
      x.f.r = __shfl_sync(kFull, mine.r, j);
      x.f.L = __shfl_sync(kFull, mine.L, j);
      x.f.klo = __shfl_sync(kFull, mine.klo, j);
      x.f.khi = __shfl_sync(kFull, mine.khi, j);
      x.f.pg0 = x.f.klo / PAGE;
      x.f.pg1 = (x.f.khi + PAGE - 1) / PAGE;
      x.list = __shfl_sync(kFull, list, j);
      x.listed = __shfl_sync(kFull, listed, j);
      if (WIN && x.f.pg0 < x.f.pg1) x.win = WinSpan::make(x.f.L, p.q_len, head.window, head.sinks);
      return x;
    };
    auto load_id = [&](const Walk &x, int pb) {
      if (pb + lane >= x.f.pg1) return 0;
      const int pg = WIN ? x.win.real_page(pb + lane) : pb + lane;
      return pg < x.listed ? p.page_indices[x.list + pg] : -1;
    };
    const int n_seg = min(32, head.s_end - s0);
    Walk cur = segment(0);
    int next_id = load_id(cur, cur.f.pg0);
    for (int j = 0; j < n_seg && ok; ++j) {
      const Walk nxt = segment(j + 1 < n_seg ? j + 1 : j);
      {  // the segment's place and query rows, two segments ahead of the consumers at most
        const int slot = nq & 1;
        bool good = true;
        if (lane == 0) good = wait_phase(qempty0 + 8 * slot, ((nq >> 1) & 1) ^ 1, abort_flag);
        if (!__shfl_sync(kFull, good, 0)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          reinterpret_cast<int4 *>(smem + S::kInfo)[slot] =
              make_int4(cur.f.r, cur.f.L, cur.f.klo, cur.f.khi);
          mbar_arrive_expect_tx(qfull0 + 8 * slot, rows * HEAD_DIM * 2);
        }
        __syncwarp();
        if (lane < rows)
          bulk_load(base + S::kQ + slot * S::kQSlot + lane * kQRowBytes,
                    p.q + static_cast<int64_t>(cur.f.r) * p.q_len * p.Hq * HEAD_DIM + q_at,
                    HEAD_DIM * 2, qfull0 + 8 * slot);
        ++nq;
      }
      if (cur.f.pg0 >= cur.f.pg1) next_id = load_id(nxt, nxt.f.pg0);
      for (int pb = cur.f.pg0; pb < cur.f.pg1 && ok; pb += 32) {
        const int cnt = min(32, cur.f.pg1 - pb);
        int id = next_id;
        next_id = pb + 32 < cur.f.pg1 ? load_id(cur, pb + 32) : load_id(nxt, nxt.f.pg0);
        if (lane < cnt && (id < 0 || id >= p.num_pages)) {  // bad id or too short a page list
          status_or(p.tm, HPA_STATUS_BAD_PAGE);
          id = 0;
        }
        const int n = n0 + lane, stage = n % kStages;
        const uint32_t phase = (n / kStages) & 1;
        const uint32_t fb = full0 + 8 * stage, dst = base + stage * kStageBytes;
        const int64_t at = (static_cast<int64_t>(id) * p.Hkv + h) * kUnit;
        for (int i = 0; i < cnt; ++i) {
          bool good = true;
          if (lane == i) {
            good = wait_phase(empty0 + 8 * stage, phase ^ 1, abort_flag);
            if (good) {
              mbar_arrive_expect_tx(fb, kStageBytes);
              bulk_load_hint(dst, k_pool + at, kUnit, fb, pol);
              bulk_load_hint(dst + kUnit, v_pool + at, kUnit, fb, pol);
            }
          }
          if (!__all_sync(kFull, good)) {
            n0 += i;
            ok = false;
            break;
          }
        }
        if (ok) n0 += cnt;
      }
      cur = nxt;
    }
  }
  if (!ok || *abort_flag) {
    if (lane == 0) {
      status_or(p.tm, HPA_STATUS_TIMEOUT);
      *reinterpret_cast<volatile int *>(smem + S::kFlag) = 1;
    }
    // never leave the CTA with copies still landing in its shared memory: the last page of each
    // stage, and the last query rows of each slot
    if (lane < kStages && n0 > lane) {
      const int last = n0 - 1 - (n0 - 1 - lane) % kStages;
      mbar_wait_bounded_rolled(full0 + 8 * lane, (last / kStages) & 1, 1000000000ull);
    }
    if (lane < 2 && nq > lane) {
      const int last = nq - 1 - (nq - 1 - lane) % 2;
      mbar_wait_bounded_rolled(qfull0 + 8 * lane, (last >> 1) & 1, 1000000000ull);
    }
  }
}

// ----------------------------------------------------------------------------- consumer
// V^T operand of 16 keys for one k half (8 keys: a pair per lane): the words of two keys, both
// 16 dims of the lane, as f16 pairs along the keys; r[2 t] belongs to dim 16 g + 2 t, r[2 t + 1]
// to the next.
__device__ __forceinline__ void v_pairs(uint32_t lo_key, uint32_t hi_key, uint32_t scale,
                                        uint32_t (&even)[4], uint32_t (&odd)[4]) {
  widen8((lo_key & 0x0f0f0f0fu) | ((hi_key << 4) & 0xf0f0f0f0u), even);
  widen8(((lo_key >> 4) & 0x0f0f0f0fu) | (hi_key & 0xf0f0f0f0u), odd);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    even[i] = mul_f16x2(even[i], scale);
    odd[i] = mul_f16x2(odd[i], scale);
  }
}

template <int NT, bool WIN>
__device__ void consumer(const AttnParams &p, uint8_t *smem, const MapHead &head) {
  using S = Smem<NT>;
  constexpr int kStages = S::kStages, kWarps = S::kWarps;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, h = blockIdx.y;
  const int g = lane >> 2, c = lane & 3;
  const uint32_t base = smem_u32(smem);
  const uint32_t full0 = base + S::kBars, empty0 = full0 + 8 * kStages;
  const uint32_t qfull0 = empty0 + 8 * kStages, qempty0 = qfull0 + 16;
  float *mbuf = reinterpret_cast<float *>(smem + S::kMerge);
  float *sm_m = reinterpret_cast<float *>(smem + S::kStats);
  float *sm_l = sm_m + kWarps * S::kRows;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kFlag);

  const int G = p.G, q_len = p.q_len, rows = group_rows(p), rb = row_base(p);
  const float sl2 = p.scale_log2 * p.k_scale[h], vsc = p.v_scale[h];
  // the two accumulator columns of each n-tile: query rows 8 nt + 2 c + {0, 1}, their tokens
  int tok[2 * NT];
#pragma unroll
  for (int i = 0; i < 2 * NT; ++i) {
    const int row = 8 * (i >> 1) + 2 * c + (i & 1);
    tok[i] = row < rows ? (rb + row) / G : q_len - 1;
  }
  // The rows of the softmax's statistics, and of score e of x[.][i]: those columns, or with the
  // rows on M 8 i + g; the key of that score, in its group of 16
  constexpr bool RM = Cfg<NT>::kRowsOnM;
  constexpr int NS = Cfg<NT>::kStats;
  auto stat_row = [&](int i) { return RM ? 8 * i + g : 8 * (i >> 1) + 2 * c + (i & 1); };
  auto stat_of = [](int i, int e) { return RM ? e >> 1 : 2 * i + (e & 1); };
  int stat_tok[NS];
#pragma unroll
  for (int i = 0; i < NS; ++i)
    stat_tok[i] = !RM ? tok[i % (2 * NT)] : stat_row(i) < rows ? (rb + stat_row(i)) / G : q_len - 1;
  // where this lane's shares of a page lie: K rows key_at(g) (+8), dims 32 c..; V keys of the
  // quad's lane c, dims 16 g..; their scales
  const int k_off = key_at(g) * 64 + c * 16;
  const int ks_off = 4096 + key_at(g) * 8 + 2 * c;
  const int vk0 = key_at(2 * c), vk1 = key_at(2 * c + 1);
  auto key_of = [&](int i, int e) {
    return RM ? 8 * i + (e & 1 ? vk1 : vk0) : key_at(g) + 8 * (e >> 1);
  };

  int count = 0;  // pages of this CTA so far: page n goes to team n % kTeams, stage n % kStages
  const int n_items = head.s_end - head.s_begin;
  for (int k = 0; k < n_items; ++k) {
    const int s = head.s_begin + k, slot = k & 1;
    bool ok = wait_phase(qfull0 + 8 * slot, (k >> 1) & 1, abort_flag);
    ok = __all_sync(kFull, ok);
    Seg f;
    {
      const int4 inf = reinterpret_cast<const int4 *>(smem + S::kInfo)[slot];
      f.r = inf.x;
      f.L = inf.y;
      f.klo = inf.z;
      f.khi = inf.w;
      f.pg0 = f.klo / PAGE;
      f.pg1 = ok ? (f.khi + PAGE - 1) / PAGE : f.pg0;  // no pages if the wait gave up
    }
    if (ok && f.L < q_len && w == 0 && lane == 0) status_or(p.tm, HPA_STATUS_BAD_SEQLEN);
    // Row of token j sees key i < lim_min + j, and with a window i < sinks or i >= start + j.
    // Pages [clear0, clear1) of the map hold no key that some row does not see.
    const int lim_min = f.L - q_len + 1;
    WinSpan win = {};
    int clear0 = 0, clear1 = lim_min / PAGE;
    if (WIN && f.pg0 < f.pg1) {
      win = WinSpan::make(f.L, q_len, head.window, head.sinks);
      const int first = win.start + q_len - 1;  // where the last row's window starts
      clear0 = first > 0 ? (first - 1) / PAGE + 1 - win.hidden : 0;
      clear1 = lim_min / PAGE - win.hidden;
    }

    // Query rows as the B operand: lane (g, c) holds dims [32 c, 32 c + 32) of rows 8 nt + g,
    // scaled by 2^e of the row; sl holds what takes the scores of its columns to log2 units.
    // From 9 rows on the fragments lie in shared memory, one warp's work for all.
    uint32_t qf[RM ? 1 : NT][8][2];
    const uint32_t frag = base + S::kFrag + lane * 16;
    float *factor = reinterpret_cast<float *>(smem + S::kFrag + NT * 8 * 256);
    float sl[NS];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (RM && w != nt) continue;
      const int row = 8 * nt + g, at = RM ? 0 : nt;
      const uint32_t qa = base + S::kQ + slot * S::kQSlot + row * kQRowBytes + c * 64;
      uint4 raw[4];
      float am = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        raw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (row < rows) lds128(qa + 16 * i, raw[i].x, raw[i].y, raw[i].z, raw[i].w);
        am = fmaxf(am, absmax8_bf16(raw[i]));
      }
      am = fmaxf(am, __shfl_xor_sync(kFull, am, 1));
      am = fmaxf(am, __shfl_xor_sync(kFull, am, 2));
      const int e = f16_row_exponent(am);
      // the sign of the score factor goes to the query, so that the larger score is the larger sum
      const float up = sl2 == 0.f ? 0.f : copysignf(exp2i(e), sl2);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t x[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int u = 0; u < 4; ++u)  // elements 8 i + 2 u, + 1: k-step 2 i + u / 2, register u % 2
          qf[at][2 * i + (u >> 1)][u & 1] = pack_f16(__uint_as_float(x[u] << 16) * up,
                                                     __uint_as_float(x[u] & 0xffff0000u) * up);
      }
      // never zero, which would make NaN of a hidden key's -inf; at 2^-126 all scores are nothing
      float down = sl2 == 0.f ? 1.f : fabsf(sl2) * exp2i(-e);
      if (down < exp2i(-126)) down = exp2i(-126);
      if (RM) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {  // registers nt and nt + 2 of the A operand
          sts32(frag + ks * 512 + 4 * nt, qf[0][ks][0]);
          sts32(frag + ks * 512 + 8 + 4 * nt, qf[0][ks][1]);
        }
        if (c == 0) factor[row] = down;
      } else {
        sl[(2 * nt) % NS] = __shfl_sync(kFull, down, 8 * c);
        sl[(2 * nt + 1) % NS] = __shfl_sync(kFull, down, 8 * c + 4);
      }
    }
    if (RM) {
      named_barrier(1, kWarps * 32);
#pragma unroll
      for (int i = 0; i < NS; ++i) sl[i] = factor[stat_row(i)];
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(qempty0 + 8 * slot);  // the slot may be refilled

    float m[NS], l[NS], o[NT][8][4];
#pragma unroll
    for (int i = 0; i < NS; ++i) m[i] = -CUDART_INF_F, l[i] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[nt][t][e] = 0.f;

    // One page of this warp; EDGE looks for keys that some row does not see.
    auto page = [&](int pg, int stage, uint32_t phase, auto edge_tag) {
      constexpr bool EDGE = decltype(edge_tag)::value;
      constexpr int KG = Cfg<NT>::kGroups, KP = Cfg<NT>::kSide;
      const bool got = wait_phase(full0 + 8 * stage, phase, abort_flag);
      if (!__all_sync(kFull, got)) {
        ok = false;
        return;
      }
      const uint8_t *kt = smem + stage * kStageBytes, *vt = kt + kUnit;
      const int key0 = (WIN ? win.real_page(pg) : pg) * PAGE;

#pragma unroll
      for (int kc = 0; kc < Cfg<NT>::kMine; kc += KG) {
        const int k0 = (w % Cfg<NT>::kShare) * Cfg<NT>::kMine + kc;
        // S = K Q^T, 16 keys at a time
        float x[KG][NT][4];
#pragma unroll
        for (int kg = 0; kg < KG; ++kg)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[kg][nt][e] = 0.f;
#pragma unroll
        for (int kp = 0; kp < KG; kp += KP) {  // groups whose chains of MMAs run side by side
          uint4 kw[KP][2];
          uint32_t sc[KP][2][2];
#pragma unroll
          for (int kq = 0; kq < KP; ++kq)
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // keys key_at(g) and key_at(g) + 8 of the group
              const int row = 16 * (k0 + kp + kq) + 8 * u;
              kw[kq][u] = *reinterpret_cast<const uint4 *>(kt + k_off + row * 64);
              const uint32_t two =
                  e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(kt + ks_off + row * 8));
              sc[kq][u][0] = both_halves<0>(two);
              sc[kq][u][1] = both_halves<1>(two);
            }
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // a word: 8 dims, two k-steps
            uint32_t qb[2][NT][2], qm[2][4];  // one of them: rows as B, or on M
#pragma unroll
            for (int st = 0; st < 2; ++st) {
              if constexpr (RM) {
                lds128(frag + (2 * i + st) * 512, qm[st][0], qm[st][1], qm[st][2], qm[st][3]);
              } else {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  qb[st][nt][0] = qf[nt][2 * i + st][0];
                  qb[st][nt][1] = qf[nt][2 * i + st][1];
                }
              }
            }
#pragma unroll
            for (int kq = 0; kq < KP; ++kq) {
              uint32_t a[2][4];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const uint4 v = kw[kq][u];
                widen8(i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w, a[u]);
#pragma unroll
                for (int b = 0; b < 4; ++b) a[u][b] = mul_f16x2(a[u][b], sc[kq][u][i >> 1]);
              }
#pragma unroll
              for (int st = 0; st < 2; ++st) {
                const uint32_t af[4] = {a[0][2 * st], a[1][2 * st], a[0][2 * st + 1],
                                        a[1][2 * st + 1]};
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  if (RM) mma_f16(x[kp + kq][nt], qm[st], a[nt & 1][2 * st], a[nt & 1][2 * st + 1]);
                  else mma_f16(x[kp + kq][nt], af, qb[st][nt][0], qb[st][nt][1]);
                }
              }
            }
          }
        }
        // what a row does not see to -inf (x is the plain sum; x * sl the score in log2 units)
        if (EDGE) {
#pragma unroll
          for (int kg = 0; kg < KG; ++kg)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int key = key0 + 16 * (k0 + kg) + key_of(nt, e), j = stat_tok[stat_of(nt, e)];
                if (!(key < lim_min + j && (!WIN || key < head.sinks || key >= win.start + j)))
                  x[kg][nt][e] = -CUDART_INF_F;
              }
        }
        // running maximum, of the plain sums: moves when a score passes it by more than the slack
        bool over = false;
        float top[NS];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int kg = 0; kg < KG; ++kg)
#pragma unroll
            for (int u = 0; u < 2; ++u) {  // the two scores of one row
              const float a = x[kg][nt][RM ? 2 * u : u], b = x[kg][nt][RM ? 2 * u + 1 : u + 2];
              const int i = stat_of(nt, RM ? 2 * u : u);
              const bool fresh = kg == 0 && (!RM || nt == 0);
              top[i] = fresh ? fmaxf(a, b) : fmaxf(top[i], fmaxf(a, b));
            }
#pragma unroll
        for (int i = 0; i < NS; ++i) over |= (top[i] - m[i]) * sl[i] > kRescaleSlack;
        if (__any_sync(kFull, over)) {
          float a[NS];
#pragma unroll
          for (int i = 0; i < NS; ++i) {
#pragma unroll
            for (int d = RM ? 1 : 4; d < (RM ? 4 : 32); d <<= 1)
              top[i] = fmaxf(top[i], __shfl_xor_sync(kFull, top[i], d));
            const float mn = (top[i] - m[i]) * sl[i] > kRescaleSlack ? top[i] : m[i];
            a[i] = mn == -CUDART_INF_F ? 1.f : exp2f((m[i] - mn) * sl[i]);
            m[i] = mn;
            l[i] *= a[i];
          }
#pragma unroll
          for (int i = 0; i < 2 * NT; ++i) {  // the columns of o
            const float f = RM ? __shfl_sync(kFull, a[(i >> 1) % NS], 8 * c + 4 * (i & 1))
                               : a[i % NS];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
              o[i >> 1][t][i & 1] *= f;
              o[i >> 1][t][2 + (i & 1)] *= f;
            }
          }
        }
        // Probabilities; their sums in fp32 before the rounding to f16.  The exponent is the plain
        // sum less the maximum's, then the factor: however large the scores, the largest one's own
        // is the lift and none passes it by more than the slack.  (The product less a rounded
        // maximum, one instruction less, is off by half a step of fp32 at that maximum: from 2^26 on
        // the weight of the largest score itself went to zero or beyond f16.)
        uint32_t pb[KG][NT][2];
        float less[NS];
#pragma unroll
        for (int i = 0; i < NS; ++i) less[i] = m[i] == -CUDART_INF_F ? 0.f : -m[i];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int kg = 0; kg < KG; ++kg) {
            float pr[4];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const int i = stat_of(nt, 2 * u), j = stat_of(nt, 2 * u + 1);
              const f32x2 d = add2(pk(x[kg][nt][2 * u], x[kg][nt][2 * u + 1]), pk(less[i], less[j]));
              upk(fma2(d, pk(sl[i], sl[j]), pk(kLift, kLift)), pr[2 * u], pr[2 * u + 1]);
              pr[2 * u] = exp2f(pr[2 * u]);
              pr[2 * u + 1] = exp2f(pr[2 * u + 1]);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u)
              l[stat_of(nt, RM ? 2 * u : u)] += pr[RM ? 2 * u : u] + pr[RM ? 2 * u + 1 : u + 2];
            const uint32_t lo = pack_f16(pr[0], pr[1]), hi = pack_f16(pr[2], pr[3]);
            if constexpr (RM) {  // lo: rows 0 to 7, hi: rows 8 to 15; nt: the half of the 16 keys
              pb[kg][0][nt] = lo;
              pb[kg][1][nt] = hi;
            } else {
              pb[kg][nt][0] = transpose8(lo);
              pb[kg][nt][1] = transpose8(hi);
            }
          }
        // O^T += V^T P^T
#pragma unroll
        for (int kg = 0; kg < KG; ++kg) {
          const int kb = 16 * (k0 + kg);
          auto words = [&](int key) {
            return *reinterpret_cast<const uint2 *>(vt + key * 64 + 8 * g);
          };
          const uint2 v0 = words(kb + vk0), v1 = words(kb + vk1);
          const uint2 v2 = words(kb + 8 + vk0), v3 = words(kb + 8 + vk1);
          const uint8_t *sb = vt + 4096 + g;
          uint32_t b0 = sb[(kb + vk0) * 8], b1 = sb[(kb + vk1) * 8];
          uint32_t b2 = sb[(kb + 8 + vk0) * 8], b3 = sb[(kb + 8 + vk1) * 8];
          const int keys[4] = {key0 + kb + vk0, key0 + kb + vk1, key0 + kb + 8 + vk0,
                               key0 + kb + 8 + vk1};
          auto scales = [](uint32_t lo, uint32_t hi) {
            return e4m3x2_to_f16x2(static_cast<uint16_t>(lo | (hi << 8)));
          };
          auto sees = [&](int key, int j) {
            return key < lim_min + j && (!WIN || key < head.sinks || key >= win.start + j);
          };
          if (EDGE) {
            auto hide = [&](int key, uint32_t b) {  // seen by no token: the scale is taken as zero
              return key >= f.L || (WIN && key >= head.sinks && key < win.low) ? 0u : b;
            };
            b0 = hide(keys[0], b0), b1 = hide(keys[1], b1);
            b2 = hide(keys[2], b2), b3 = hide(keys[3], b3);
            if (q_len > 1) {
              // A NaN that some tokens see and others do not: 0 * NaN would reach every row, so
              // the scale is taken as zero and the block's 16 dims, which are this quad's o, become
              // NaN for the rows that see the key.
              uint32_t odd = 0;
              auto take = [&](int u, uint32_t b) {
                if (!e4m3_nan(b) || (sees(keys[u], 0) && sees(keys[u], q_len - 1))) return b;
                odd |= 1u << u;
                return 0u;
              };
              b0 = take(0, b0), b1 = take(1, b1), b2 = take(2, b2), b3 = take(3, b3);
              if (__any_sync(kFull, odd != 0)) {
#pragma unroll 1
                for (int v = 0; v < 16; ++v) {  // the quad's 16 keys
                  const uint32_t bits = __shfl_sync(kFull, odd, (lane & 28) | (v >> 2));
                  if (!((bits >> (v & 3)) & 1)) continue;
                  const int at = key0 + kb + key_at(2 * (v >> 2) + (v & 1)) + 8 * ((v & 3) >> 1);
#pragma unroll
                  for (int i = 0; i < 2 * NT; ++i)
                    if (sees(at, tok[i]))
#pragma unroll
                      for (int t = 0; t < 8; ++t)
                        o[i >> 1][t][i & 1] = o[i >> 1][t][2 + (i & 1)] = CUDART_NAN_F;
                }
              }
            }
          }
          const uint32_t s01 = scales(b0, b1), s23 = scales(b2, b3);
#pragma unroll
          for (int hw = 0; hw < 2; ++hw) {
            uint32_t a0[4], a1[4], a2[4], a3[4];
            v_pairs(hw ? v0.y : v0.x, hw ? v1.y : v1.x, s01, a0, a1);
            v_pairs(hw ? v2.y : v2.x, hw ? v3.y : v3.x, s23, a2, a3);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              const uint32_t af[4] = {a0[t], a1[t], a2[t], a3[t]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(o[nt][4 * hw + t], af, pb[kg][nt][0], pb[kg][nt][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * stage);
    };
    // this team's pages of the segment: page n of the CTA with n % kTeams == team
    constexpr int kTeams = Cfg<NT>::kTeams;
    const int skip = (w / Cfg<NT>::kShare + kTeams - count % kTeams) % kTeams;
    const int n_pages = f.pg1 - f.pg0;
    for (int i = skip; i < n_pages && ok; i += kTeams) {
      const int n = count + i, stage = n % kStages, pg = f.pg0 + i;
      const uint32_t phase = (n / kStages) & 1;
      if (pg >= clear0 && pg < clear1) page(pg, stage, phase, std::false_type());
      else page(pg, stage, phase, std::true_type());
    }
    count += n_pages;
    // A warp that gave up flags the map and raises the CTA's abort flag; it still takes part
    // in the named barriers below.  Later waits see the flag and fail at once.
    if (!ok && lane == 0) {
      status_or(p.tm, HPA_STATUS_TIMEOUT);
      *abort_flag = 1;
    }

    // ---- segment end: merge the warps' (m, l, O) and store the partial
#pragma unroll
    for (int i = 0; i < NS; ++i) {
#pragma unroll
      for (int d = RM ? 1 : 4; d < (RM ? 4 : 32); d <<= 1) l[i] += __shfl_xor_sync(kFull, l[i], d);
      if (RM ? c == 0 : g == 0) {
        sm_m[w * S::kRows + stat_row(i)] = m[i] * sl[i];
        sm_l[w * S::kRows + stat_row(i)] = l[i];
      }
    }
    named_barrier(1, kWarps * 32);
    auto row_stats = [&](int row, float &M, float &Lsum) {
      M = -CUDART_INF_F;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) M = fmaxf(M, sm_m[v * S::kRows + row]);
      M = M == -CUDART_INF_F ? 0.f : M;
      Lsum = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v)
        Lsum += sm_l[v * S::kRows + row] * exp2f(sm_m[v * S::kRows + row] - M);
    };
    float fs[2 * NT];
#pragma unroll
    for (int i = 0; i < 2 * NT; ++i) {
      const int row = 8 * (i >> 1) + 2 * c + (i & 1);
      float M, Lsum;
      row_stats(row, M, Lsum);
      fs[i] = Lsum == 0.f ? 0.f : exp2f(sm_m[w * S::kRows + row] - M) / Lsum * vsc;
    }
    float *mine = mbuf + (w % S::kBufs) * (S::kRows * kMergeStride);
    auto merge = [&](auto add_tag) {  // warps 0 / 1 store, then warps 2 / 3 add
      constexpr bool ADD = decltype(add_tag)::value;
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i) {
        const int row = 8 * (i >> 1) + 2 * c + (i & 1);
        float4 *d = reinterpret_cast<float4 *>(mine + row * kMergeStride + 16 * g);
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const float(&oa)[4] = o[i >> 1][2 * t], (&ob)[4] = o[i >> 1][2 * t + 1];
          const int e = i & 1;
          float4 nv = make_float4(oa[e] * fs[i], oa[2 + e] * fs[i],
                                  ob[e] * fs[i], ob[2 + e] * fs[i]);
          if (ADD) {
            const float4 old = d[t];
            nv.x += old.x, nv.y += old.y, nv.z += old.z, nv.w += old.w;
          }
          d[t] = nv;
        }
      }
    };
    if (w < S::kBufs) merge(std::false_type());
    named_barrier(1, kWarps * 32);
#pragma unroll
    for (int v = S::kBufs; v < kWarps; v += S::kBufs) {
      if (w >= v && w < v + S::kBufs) merge(std::true_type());
      named_barrier(1, kWarps * 32);
    }
    const int tid = threadIdx.x;
    for (int v = tid; v < rows * (HEAD_DIM / 4); v += kWarps * 32) {
      const int row = v / (HEAD_DIM / 4), c4 = v % (HEAD_DIM / 4);
      const int j = (rb + row) / G, gq = (rb + row) % G;
      const int64_t dst = (static_cast<int64_t>(s) * q_len + j) * p.Hq + h * G + gq;
      float4 a = reinterpret_cast<const float4 *>(mbuf + row * kMergeStride)[c4];
#pragma unroll
      for (int u = 1; u < S::kBufs; ++u) {
        const float4 b =
            reinterpret_cast<const float4 *>(mbuf + (u * S::kRows + row) * kMergeStride)[c4];
        a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
      }
      reinterpret_cast<float4 *>(p.partial_o + dst * HEAD_DIM)[c4] = a;
    }
    if (tid < rows) {
      float M, Lsum;
      row_stats(tid, M, Lsum);
      const int j = (rb + tid) / G, gq = (rb + tid) % G;
      // a row that sees a NaN has no sum: +inf, beside which no other partial counts, makes the
      // combine's result NaN (it passes over -inf and NaN)
      p.partial_lse[(static_cast<int64_t>(s) * q_len + j) * p.Hq + h * G + gq] =
          Lsum == 0.f ? -CUDART_INF_F
          : Lsum > 0.f ? (M - kLift + log2f(Lsum)) * 0.69314718055994531f
                       : CUDART_INF_F;
    }
    named_barrier(1, kWarps * 32);
  }
}

template <int NT, bool WIN>
__global__ void __launch_bounds__(Cfg<NT>::kThreads, Cfg<NT>::kBlocks)
    decode_attn_e2m1_kernel(const uint8_t *__restrict__ k_pool, const uint8_t *__restrict__ v_pool,
                            const AttnParams p) {
  using S = Smem<NT>;
  constexpr int kStages = S::kStages, kWarps = S::kWarps;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ MapHead head;
  const int c = blockIdx.x;
  const uint32_t base = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(base + S::kBars + 8 * st, 1);
      mbar_init(base + S::kBars + 8 * (kStages + st), Cfg<NT>::kShare);
    }
    for (int sl = 0; sl < 2; ++sl) {
      mbar_init(base + S::kBars + 8 * (2 * kStages + sl), 1);            // qfull
      mbar_init(base + S::kBars + 8 * (2 * kStages + 2 + sl), kWarps);   // qempty
    }
    *reinterpret_cast<int *>(smem + S::kFlag) = 0;
    fence_barrier_init();
  }
  // Nothing above reads memory that an earlier kernel writes: the prologue overlaps it.
  pdl_wait();
  if (threadIdx.x == 0) {
    MapHead m = read_map_head(p.tm, p.lay, p.B, p.C, c, p.q_len, WIN, c == 0 && blockIdx.y == 0);
    if (!WIN && m.windowed) {  // a map of hpa_plan_window belongs to hpa_decode_attn_window
      status_or(p.tm, HPA_STATUS_BAD_MAP);
      m.go = 0;
    }
    head = m;
  }
  __syncthreads();
  pdl_launch_dependents();  // the combine kernel may be scheduled; it waits for this grid
  if (!head.go) return;     // bad map, or a partition with no tiles
  const MapHead m = head;
  if (threadIdx.x >= kWarps * 32) producer<NT, WIN>(p, k_pool, v_pool, smem, m);
  else consumer<NT, WIN>(p, smem, m);
}

template <int NT, bool WIN>
cudaError_t configure() {
  static int configured[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && configured[dev]) return cudaSuccess;
  e = cudaFuncSetAttribute(decode_attn_e2m1_kernel<NT, WIN>,
                           cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<NT>::kAlloc);
  if (e == cudaSuccess && dev < 64) configured[dev] = 1;
  return e;
}

template <int NT, bool WIN>
cudaError_t launch(const AttnParams &p, const void *k_pool, const void *v_pool, cudaStream_t s) {
  cudaError_t e = configure<NT, WIN>();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.C, p.Hkv, (p.rows + p.group - 1) / p.group);
  cfg.blockDim = dim3(Cfg<NT>::kThreads);
  cfg.dynamicSmemBytes = Smem<NT>::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_attn_e2m1_kernel<NT, WIN>,
                            static_cast<const uint8_t *>(k_pool),
                            static_cast<const uint8_t *>(v_pool), p);
}

template <int NT>
int occupancy(int *ctas) {
  if (configure<NT, false>() != cudaSuccess) return -1;
  const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(
      ctas, decode_attn_e2m1_kernel<NT, false>, Cfg<NT>::kThreads, Smem<NT>::kAlloc);
  return e == cudaSuccess ? 0 : -1;
}

}  // namespace

// Query rows of a KV head in groups of equal size: CTAs that share pages keep pace and find them in
// L2.
int attn_e2m1_group(int rows) {
  const int groups = (rows + E2M1_MAX_ROWS - 1) / E2M1_MAX_ROWS;
  return (rows + groups - 1) / groups;
}

cudaError_t launch_decode_attn_e2m1(const AttnParams &p, const void *k_pool, const void *v_pool,
                                    cudaStream_t s) {
  if (p.group > 16) return launch_decode_attn_e2m1_tc(p, k_pool, v_pool, s);
  const auto run = p.group <= 8 ? (p.window ? launch<1, true> : launch<1, false>)
                                : (p.window ? launch<2, true> : launch<2, false>);
  return run(p, k_pool, v_pool, s);
}

int attn_e2m1_ctas_per_sm(int rows, int *ctas) {
  const int group = attn_e2m1_group(rows);
  if (group > 16) {  // a CTA takes an SM's tensor memory
    *ctas = 1;
    return 0;
  }
  return group <= 8 ? occupancy<1>(ctas) : occupancy<2>(ctas);
}

}  // namespace hpa
