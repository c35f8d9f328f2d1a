// Accumulated attention weight of every cached key, the score a cache eviction goes by.
//
// For request r, KV head h and key i, over the query rows (token j, head g of h) that see
// i, with the rows' log-sum-exp known from the attention step:
//   acc_out[i] = (i < L - q_len ? decay * acc_in[i] : 0) + sum_rows exp(s_i - lse_row),
//   s_i = sm_scale * q_row . k_i.
// No value is read and no softmax statistic is carried from key to key, so keys are
// independent: the task map of the attention step only serves as a balanced work list.
//
// GB300 design:
//  * a step is two pages (128 keys) of one KV head: S[128 keys][rows] = K . Q^T runs as
//    tcgen05.mma with the accumulators in tensor memory.  Keys sit on the TMEM lanes, so
//    a compute thread owns one key: it sums its rows' exponentials alone, without an
//    exchange between lanes, and neighbouring threads read and write neighbouring
//    accumulators.  The sums are in the same order on every run;
//  * E4M3 pages enter the MMA as they are, the query rows as two E4M3 terms side by side
//    in N (as in decode_attn_tc.cu), so nothing is widened;
//  * roles: a TMA producer warp, one thread issuing MMAs, eight compute warps in two groups
//    that take every other step, and one to four warps that stage each segment's query rows
//    ahead.  With the staging in the producer warp, 64 rows took 17 us before the first page
//    was asked for (16 E4M3 rows 8, 8 rows 3), at every segment.  A stage is free as soon
//    as its MMAs are done; the accumulators of a step's pages (256 bytes each) come with it
//    into a ring of their own;
//  * up to 16 rows two CTAs share an SM, above one with a deeper ring: the partition
//    counts of hpa_default_num_ctas for these row counts.
// Bound by DRAM.  Plan and weights together: 0.89 GB (32 requests of about 24000 E4M3 keys,
// two tokens) in 141 us, 6.4 TB/s; 0.27 GB (16 of about 8192, bf16, one token) in 47, of
// which 41 stream the pages; 0.14 GB (one of 65536, bf16, 64 rows a KV head) in 30, of
// which 18 do.  On mma.sync, where a key's rows lie in four
// lanes and 16 rows make a pass: 219, 52 and 72 us.
// Every wait is bounded in time, as in the attention kernels.
#include <math_constants.h>

#include <type_traits>

#include "tcgen05.cuh"

namespace hpa {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kGroupWarps = 4;  // compute warps that share a step: one key per thread
constexpr int kGroups = 2;
constexpr int kCompute = kGroups * kGroupWarps;
constexpr int kStepPages = 2;
constexpr int kAccBytes = PAGE * 4;
// The lse of a row that adds nothing, and its token: one that sees no key at all
constexpr float kNoWeight = 3.402823466e38f;
constexpr int kNoToken = -(1 << 30);

// RP: query rows, padded to 8, 16, 32, 48 or 64.
template <int KV, int RP>
struct KwCfg {
  static constexpr bool kSmall = RP <= 16;
  static constexpr int kStagers = RP <= 8 ? 1 : RP <= 16 ? 2 : 4;  // warps, 8 rows at a time each
  static constexpr int kThreads = (kCompute + 2 + kStagers) * 32;
  static constexpr int kPageBytes = KV == HPA_KV_BF16 ? 16384 : 8192;
  static constexpr int kStageBytes = kStepPages * kPageBytes;
  static constexpr int kN = KV == HPA_KV_E4M3 ? 2 * RP : RP < 16 ? 16 : RP;  // MMA columns
  // Two CTAs share an SM with 64 KB of pages in flight each: with 96 KB, CTAs of equal
  // budgets ended further apart (148 -> 154 us at 32 x 24000 E4M3, 49.5 -> 51 at 16 x 8192).
  static constexpr int kStages = (kSmall ? 64 : 160) * 1024 / kStageBytes;
  static constexpr int kBufs = KV == HPA_KV_E4M3 && kSmall ? 2 : 4;  // S buffers in TMEM
  // Slots of the accumulator ring.  The copy for step n is issued once the MMAs of step
  // n - kStages are done, and these once the scores of step n - kStages - kBufs have left
  // TMEM.  The group of that step reads its accumulators only after it has released the
  // scores, but its step before, n - kStages - kBufs - kGroups, it has finished: a slot may
  // be taken again that many steps later.
  static constexpr int kAccs = kSmall ? 8 : 16;
  static_assert(kStages + kBufs + kGroups <= kAccs && kAccs % kGroups == 0, "accumulator ring");
  static constexpr int kTmem = kBufs * kN <= 32    ? 32
                               : kBufs * kN <= 64  ? 64
                               : kBufs * kN <= 128 ? 128
                               : kBufs * kN <= 256 ? 256
                                                   : 512;
  static_assert(kBufs * kN <= 512, "TMEM");
  static constexpr int kQSlot = kN * (KV == HPA_KV_BF16 ? 256 : 128);
  static constexpr int kQ = kStages * kStageBytes;              // two slots
  static constexpr int kAcc = kQ + 2 * kQSlot;                  // float[kAccs][2][64]
  static constexpr int kRow = kAcc + kAccs * kStepPages * kAccBytes;  // float2[2][RP]
  static constexpr int kJRow = kRow + 2 * RP * 8;               // int[RP]: token j of a row
  static constexpr int kJSee = kJRow + RP * 4;                  // int[2][RP]: the same, or kNoToken
  static constexpr int kInfo = (kJSee + 2 * RP * 4 + 15) & ~15;  // int4[2]: none adds, L, pages
  static constexpr int kPid = kInfo + 32;                       // int2[kAccs]
  // kv_full[kStages] kv_empty[kStages] s_full[kBufs] s_free[kBufs] acc_full[kAccs]
  // q_full[2] q_empty[2] drain
  static constexpr int kBars = kPid + kAccs * 8;
  static constexpr int kKvFull = kBars, kKvEmpty = kKvFull + 8 * kStages,
                       kSFull = kKvEmpty + 8 * kStages, kSFree = kSFull + 8 * kBufs,
                       kAccFull = kSFree + 8 * kBufs, kQFull = kAccFull + 8 * kAccs,
                       kQEmpty = kQFull + 16, kDrain = kQEmpty + 16;
  static constexpr int kTmemAt = kDrain + 8;
  static constexpr int kAbort = kTmemAt + 4;
  static constexpr int kAlloc = kAbort + 4 + 1024;              // room to align the base
};

// Segment s of this partition: request, length, compact pages [pg0, pg1).  The keys of a
// request shorter than q_len are not followed.
struct KwSeg {
  int r, L, pg0, pg1;
};
__device__ __forceinline__ KwSeg kw_seg(const KeyWeightsParams &p, const MapHead &m, int s,
                                        bool report) {
  const SegRow sr =
      m.windowed ? read_seg_row<true, true>(p.tm, p.lay, p.B, s, blockIdx.x, m.tile, report)
                 : read_seg_row<false, true>(p.tm, p.lay, p.B, s, blockIdx.x, m.tile, report);
  KwSeg f = {sr.r, sr.L, sr.klo / PAGE, (sr.khi + PAGE - 1) / PAGE};
  if (sr.L < p.q_len) {
    if (report) status_raise(p.tm, HPA_STATUS_BAD_SEQLEN);
    f.pg1 = f.pg0;
  }
  return f;
}

// ----------------------------------------------------------------------------- stagers
// Each segment's query rows as the MMA's B operand (K-major, 128-byte swizzle), and each
// row's score factor and log-sum-exp in base 2: a weight is 2^(factor * S - lse).
// Rows that pad the tile and rows of lse -inf add nothing.  They are copies of the first row
// that does add, with an lse of kNoWeight: a query of zeros would make NaN of an infinite
// key (0 inf), and the key's weight with it.  A copy's score is not finite only where the
// row's own is not, and 2^(factor * S - kNoWeight) is then 0, infinite or NaN as the row's
// own weight is.  That holds where the row sees the key; the compute warps' masked path
// takes copies out by their token, and runs for every key if no row of the segment adds.
// Four lanes share a row.  With every lane in all of a warp's eight rows, twice the code,
// which a launch fetches cold, 16 E4M3 rows were staged 8.5 us after the map was there and
// 64 bf16 ones 7.5; so 3.7 and 3.1, before the first pages land.
template <int KV, int RP>
__device__ void kw_stager(const KeyWeightsParams &p, uint8_t *smem, const MapHead &m, int ws) {
  using S = KwCfg<KV, RP>;
  const int lane = threadIdx.x & 31, G = p.G, h = blockIdx.y;
  const uint32_t base = smem_u32(smem);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kAbort);
  const int *jrow = reinterpret_cast<const int *>(smem + S::kJRow);
  constexpr int kHalves = RP > 32 ? 2 : 1;
  using Rows = typename std::conditional<(RP > 32), unsigned long long, uint32_t>::type;
  float factor = p.scale_log2;
  if (KV == HPA_KV_E4M3) factor *= p.k_scale[h];
  for (int k = 0; k < m.s_end - m.s_begin; ++k) {
    const int slot = k & 1;
    const KwSeg f = kw_seg(p, m, m.s_begin + k, false);
    int good = 1;
    if (lane == 0)
      good = !*abort_flag &&
             mbar_wait_bounded_rolled(base + S::kQEmpty + 8 * slot, ((k >> 1) & 1) ^ 1);
    if (!__shfl_sync(kFull, good, 0)) {
      if (lane == 0) {
        status_or(p.tm, HPA_STATUS_TIMEOUT);
        *abort_flag = 1;
      }
      return;
    }
    uint8_t *qs = smem + S::kQ + slot * S::kQSlot;
    float2 *rc = reinterpret_cast<float2 *>(smem + S::kRow) + slot * RP;
    int *jsee = reinterpret_cast<int *>(smem + S::kJSee) + slot * RP;
    const int64_t row_at = static_cast<int64_t>(f.r) * p.q_len * p.Hq + h * G;
    auto place = [&](int row) {
      const int j = jrow[row];
      return row_at + static_cast<int64_t>(j) * p.Hq + (row - j * G);
    };
    float z[kHalves];  // every row's lse, a row (or two) per lane
#pragma unroll
    for (int u = 0; u < kHalves; ++u)
      z[u] = lane + 32 * u < p.rows ? p.lse[place(lane + 32 * u)] : -CUDART_INF_F;
    Rows adds = 0;  // rows that add a weight
#pragma unroll 1
    for (int row0 = 8 * ws; row0 < (KV == HPA_KV_BF16 ? S::kN : RP); row0 += 8 * S::kStagers) {
      // four lanes to a row: 32 dims each, in 16-byte pieces of the operand
      const int row = row0 + (lane >> 2), qd = lane & 3;
      uint4 x[4] = {};
      float mine = factor;
      int src = row < p.rows ? row : 0;
#pragma unroll 1
      while (row0 < RP) {  // columns beyond RP are not read back
        const uint4 *from = reinterpret_cast<const uint4 *>(p.q + place(src) * HEAD_DIM);
#pragma unroll
        for (int c = 0; c < 4; ++c)
          x[c] = from[KV == HPA_KV_BF16 ? 4 * c + qd : 8 * (c >> 1) + 2 * qd + (c & 1)];
        adds = __ballot_sync(kFull, z[0] != -CUDART_INF_F);
        if constexpr (kHalves > 1)
          adds |= static_cast<Rows>(__ballot_sync(kFull, z[1] != -CUDART_INF_F)) << 32;
        const int want = adds == 0 || (adds >> src & 1) ? src : __ffsll(adds) - 1;
        if (__all_sync(kFull, want == src)) break;
        src = want;
      }
      const float lse = __shfl_sync(kFull, kHalves > 1 && row0 >= 32 ? z[kHalves - 1] : z[0],
                                    row & 31);
      if (KV == HPA_KV_BF16) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *reinterpret_cast<uint4 *>(qs + kmaj(row, 16 * (4 * c + qd), S::kN * 128)) = x[c];
      } else {
        float2 f[4][4];
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t u[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            f[c][e] = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[e]));
            amax = fmaxf(amax, fmaxf(fabsf(f[c][e].x), fabsf(f[c][e].y)));
          }
        }
        amax = fmaxf(amax, __shfl_xor_sync(kFull, amax, 1));
        const float sq = pow2_to_128(fmaxf(amax, __shfl_xor_sync(kFull, amax, 2)));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 a = f[2 * half + (e >> 1)][2 * (e & 1)];
            const float2 b = f[2 * half + (e >> 1)][2 * (e & 1) + 1];
            const float v[4] = {a.x, a.y, b.x, b.y};
            e4m3_two_terms(v, sq, hi[e], lo[e]);
          }
          uint8_t *to = qs + kmaj(row, 16 * (4 * half + qd), 0);
          *reinterpret_cast<uint4 *>(to) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4 *>(to + RP * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        }
        mine = factor / sq;
      }
      if (qd == 0 && row < RP) {
        const bool add = adds >> row & 1;
        rc[row] = make_float2(mine, add ? lse * 1.4426950408889634f : kNoWeight);
        jsee[row] = add ? jrow[row] : kNoToken;
      }
    }
    if (ws == 0 && lane == 0)
      reinterpret_cast<int4 *>(smem + S::kInfo)[slot] = make_int4(adds == 0, f.L, f.pg0, f.pg1);
    fence_proxy_async_smem();  // the MMA reads the slot through the async proxy
    mbar_arrive(base + S::kQFull + 8 * slot);  // every lane publishes its own stores
  }
}

// ----------------------------------------------------------------------------- producer
template <int KV, int RP>
__device__ void kw_producer(const KeyWeightsParams &p, const CUtensorMap *tmk, uint8_t *smem,
                            const MapHead &m) {
  using S = KwCfg<KV, RP>;
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const uint32_t base = smem_u32(smem);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kAbort);
  volatile int2 *pids = reinterpret_cast<volatile int2 *>(smem + S::kPid);
  const bool windowed = m.windowed;
  uint64_t pol = 0;
  if (lane == 0) pol = l2_policy_evict_first();
  int st = 0, slot_a = 0;
  uint32_t phase = 0, issued = 0, parity_bits = 0, acc_issued = 0, acc_parity = 0, acc_phase = 0;
  bool ok = true;
  for (int s = m.s_begin; s < m.s_end && ok; ++s) {
    const KwSeg f = kw_seg(p, m, s, lane == 0);
    WinSpan win = {};
    if (windowed && f.pg0 < f.pg1) win = WinSpan::make(f.L, p.q_len, m.window, m.sinks);
    const int pstart = p.page_indptr[f.r];
    const int pcount = p.page_indptr[f.r + 1] - pstart;
    for (int pb = f.pg0; pb < f.pg1 && ok; pb += 32 * kStepPages) {
      int id[kStepPages];
#pragma unroll
      for (int u = 0; u < kStepPages; ++u) {
        const int v = pb + kStepPages * lane + u;
        id[u] = 0;
        if (v < f.pg1) {
          const int pg = windowed ? win.real_page(v) : v;
          id[u] = pg < pcount ? p.page_indices[pstart + pg] : -1;
          if (id[u] < 0 || id[u] >= p.num_pages) {
            status_raise(p.tm, HPA_STATUS_BAD_PAGE);
            id[u] = -1;  // page 0 is read in its place and nothing is written
          }
        }
      }
      const int steps = min(32, (f.pg1 - pb + kStepPages - 1) / kStepPages);
      for (int i = 0; i < steps; ++i) {
        const int n = min(kStepPages, f.pg1 - (pb + kStepPages * i));
        const int i0 = __shfl_sync(kFull, id[0], i), i1 = __shfl_sync(kFull, id[1], i);
        int good = 1;
        if (lane == 0) {
          if (*abort_flag || !mbar_wait_bounded_rolled(base + S::kKvEmpty + 8 * st, phase ^ 1)) {
            good = 0;
          } else {
            const uint32_t fb = base + S::kKvFull + 8 * st, dst = base + st * S::kStageBytes;
            const uint32_t ab = base + S::kAccFull + 8 * slot_a;
            pids[slot_a].x = i0;
            pids[slot_a].y = n > 1 ? i1 : -1;
            mbar_arrive_expect_tx(fb, n * S::kPageBytes);
            if (p.acc_in) mbar_arrive_expect_tx(ab, n * kAccBytes);
            else mbar_arrive(ab);
#pragma unroll
            for (int u = 0; u < kStepPages; ++u) {
              if (u >= n) break;
              const int z = max(u ? i1 : i0, 0) * p.Hkv + h;
              tma_load_3d(dst + u * 8192, tmk, fb, 0, 0, z, pol);
              if (KV == HPA_KV_BF16)  // [dim block][128 keys][128 B]
                tma_load_3d(dst + kStepPages * 8192 + u * 8192, tmk, fb, 64, 0, z, pol);
              if (p.acc_in)
                bulk_load(base + S::kAcc + (slot_a * kStepPages + u) * kAccBytes,
                          p.acc_in + static_cast<int64_t>(z) * PAGE, kAccBytes, ab);
            }
            issued |= 1u << st;
            parity_bits = (parity_bits & ~(1u << st)) | (phase << st);
            acc_issued |= 1u << slot_a;
            acc_parity = (acc_parity & ~(1u << slot_a)) | (acc_phase << slot_a);
          }
        }
        ok = __shfl_sync(kFull, good, 0) != 0;
        if (!ok) break;
        if (++st == S::kStages) st = 0, phase ^= 1;
        if (++slot_a == S::kAccs) slot_a = 0, acc_phase ^= 1;
      }
    }
  }
  __syncwarp();
  if (lane == 0) raised_done(p.tm, gridDim.x * gridDim.y);  // this warp alone raises errors
  if (!ok && lane == 0) {
    status_or(p.tm, HPA_STATUS_TIMEOUT);
    *abort_flag = 1;
    // no copy may land after the CTA has left
    for (int i = 0; i < S::kStages; ++i)
      if (issued >> i & 1u)
        mbar_wait_bounded_rolled(base + S::kKvFull + 8 * i, parity_bits >> i & 1u, 1000000000ull);
    for (int i = 0; i < S::kAccs; ++i)
      if (acc_issued >> i & 1u)
        mbar_wait_bounded_rolled(base + S::kAccFull + 8 * i, acc_parity >> i & 1u, 1000000000ull);
  }
}

// ----------------------------------------------------------------------------- MMA issuer
template <int KV, int RP>
__device__ void kw_issuer(const KeyWeightsParams &p, uint8_t *smem, int n_seg, uint32_t tmem) {
  using S = KwCfg<KV, RP>;
  const uint32_t base = smem_u32(smem);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kAbort);
  const uint32_t idesc = tc_idesc(KV == HPA_KV_BF16 ? 1 : 0, S::kN, 0, 0);
  int st = 0, buf = 0;
  uint32_t phase = 0, sphase = 0;
  bool ok = true;
  for (int k = 0; k < n_seg && ok; ++k) {
    const int slot = k & 1;
    if (*abort_flag || !mbar_wait_bounded_rolled(base + S::kQFull + 8 * slot, (k >> 1) & 1)) {
      ok = false;
      break;
    }
    const int4 info = reinterpret_cast<const int4 *>(smem + S::kInfo)[slot];
    const int steps = (info.w - info.z + kStepPages - 1) / kStepPages;
    const uint32_t q = base + S::kQ + slot * S::kQSlot;
    for (int i = 0; i < steps; ++i) {
      if (*abort_flag || !mbar_wait_bounded_rolled(base + S::kKvFull + 8 * st, phase) ||
          !mbar_wait_bounded_rolled(base + S::kSFree + 8 * buf, sphase ^ 1)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t kb = base + st * S::kStageBytes, d = tmem + buf * S::kN;
      if (KV == HPA_KV_BF16) {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)  // 16 dims per MMA
          tc_mma<KV>(d, tc_desc(kb + (kk >> 2) * (kStepPages * 8192) + (kk & 3) * 32, 16, 1024),
                     tc_desc(q + (kk >> 2) * (S::kN * 128) + (kk & 3) * 32, 16, 1024), idesc,
                     kk > 0);
      } else {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // 32 dims per MMA
          tc_mma<KV>(d, tc_desc(kb + kk * 32, 16, 1024), tc_desc(q + kk * 32, 16, 1024), idesc,
                     kk > 0);
      }
      tc_commit(base + S::kSFull + 8 * buf);
      tc_commit(base + S::kKvEmpty + 8 * st);
      if (i == steps - 1) tc_commit(base + S::kQEmpty + 8 * slot);
      if (++st == S::kStages) st = 0, phase ^= 1;
      if (++buf == S::kBufs) buf = 0, sphase ^= 1;
    }
    if (steps == 0) mbar_arrive(base + S::kQEmpty + 8 * slot);
  }
  if (!ok) {
    status_or(p.tm, HPA_STATUS_TIMEOUT);
    *abort_flag = 1;
  }
  tc_commit(base + S::kDrain);  // every MMA completes before the CTA frees its TMEM
}

// ----------------------------------------------------------------------------- compute
template <int KV, int RP>
__device__ void kw_compute(const KeyWeightsParams &p, uint8_t *smem, const MapHead &head,
                           uint32_t tmem) {
  using S = KwCfg<KV, RP>;
  constexpr int kPart = RP < 16 ? RP : 16;  // rows read from TMEM at a time
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, h = blockIdx.y;
  const int w = warp % kGroupWarps, group = warp / kGroupWarps, t = 32 * w + lane;
  const uint32_t base = smem_u32(smem);
  const uint32_t lane_t = tmem + (static_cast<uint32_t>(32 * w) << 16);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kAbort);
  const bool windowed = head.windowed;
  const int sinks = head.sinks, q_len = p.q_len, n_seg = head.s_end - head.s_begin;
  int n = 0;  // step of the CTA
  bool ok = true;
  for (int k = 0; k < n_seg && ok; ++k) {
    const int slot = k & 1;
    ok = __all_sync(kFull, !*abort_flag && mbar_wait_bounded_rolled(base + S::kQFull + 8 * slot,
                                                                    (k >> 1) & 1));
    if (!ok) break;
    const int4 info = reinterpret_cast<const int4 *>(smem + S::kInfo)[slot];
    const int L = info.y, pg0 = info.z, pg1 = info.w;
    const int steps = (pg1 - pg0 + kStepPages - 1) / kStepPages;
    WinSpan win = {};
    if (windowed && steps > 0) win = WinSpan::make(L, q_len, head.window, sinks);
    // first key hidden from some row (from all of them if no row adds a weight)
    const int lim_min = info.x ? 0 : L - q_len + 1;
    const uint32_t rows = base + S::kRow + slot * RP * 8;
    const int *jsee = reinterpret_cast<const int *>(smem + S::kJSee) + slot * RP;
    for (int i = (group + kGroups - n % kGroups) % kGroups; i < steps; i += kGroups) {
      const int m = n + i, buf = m % S::kBufs, sa = m % S::kAccs;
      ok = __all_sync(kFull,
                      !*abort_flag &&
                          mbar_wait_bounded_rolled(base + S::kAccFull + 8 * sa, m / S::kAccs & 1) &&
                          mbar_wait_bounded_rolled(base + S::kSFull + 8 * buf, m / S::kBufs & 1));
      if (!ok) break;
      tc_fence_after();
      const int v = pg0 + kStepPages * i + t / PAGE;  // compact page of this thread's key
      const int key = (windowed ? win.real_page(v) : v) * PAGE + t % PAGE;
      const int2 pid2 = const_cast<const int2 *>(reinterpret_cast<int2 *>(smem + S::kPid))[sa];
      const int pid = t < PAGE ? pid2.x : pid2.y;
      // some rows do not see this key: the causal end, a window's start
      const bool part =
          key >= lim_min || (windowed && key >= sinks && key < win.start + q_len - 1);
      const bool any_part = __any_sync(kFull, part);
      f32x2 sum = pk(0.f, 0.f);
#pragma unroll
      for (int r0 = 0; r0 < RP; r0 += kPart) {
        float s[kPart], u[KV == HPA_KV_E4M3 ? kPart : 8];
#pragma unroll
        for (int c = 0; c < kPart; c += 8) {
          const uint32_t col = lane_t + buf * S::kN + r0 + c;
          tc_ld8(col, *reinterpret_cast<float(*)[8]>(s + c));
          if (KV == HPA_KV_E4M3) tc_ld8(col + RP, *reinterpret_cast<float(*)[8]>(u + c));
        }
        tc_wait_ld();
        if (r0 + kPart >= RP) {  // every score of the step is in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(base + S::kSFree + 8 * buf);
        }
#pragma unroll
        for (int e = 0; e < kPart; e += 2) {
          uint32_t c0, l0, c1, l1;  // two rows' score factor and lse
          lds128(rows + (r0 + e) * 8, c0, l0, c1, l1);
          f32x2 x = pk(s[e], s[e + 1]);
          if (KV == HPA_KV_E4M3) x = fma2(pk(u[e], u[e + 1]), pk(0.0625f, 0.0625f), x);
          float a, b;
          upk(fma2(x, pk(__uint_as_float(c0), __uint_as_float(c1)),
                   pk(-__uint_as_float(l0), -__uint_as_float(l1))),
              a, b);
          a = exp2f(a), b = exp2f(b);
          if (any_part) {
            auto hidden = [&](int j) {
              return key >= lim_min + j || (windowed && key >= sinks && key < win.start + j);
            };
            if (hidden(jsee[r0 + e])) a = 0.f;
            if (hidden(jsee[r0 + e + 1])) b = 0.f;
          }
          sum = add2(sum, pk(a, b));
        }
      }
      float wt, w1;
      upk(sum, wt, w1);
      wt += w1;
      if (pid >= 0 && key < L && !(windowed && key >= sinks && key < win.low)) {
        if (p.acc_in && key < L - q_len)
          wt += p.decay * reinterpret_cast<const float *>(smem + S::kAcc)[sa * 128 + t];
        p.acc_out[(static_cast<int64_t>(pid) * p.Hkv + h) * PAGE + t % PAGE] = wt;
      }
    }
    n += steps;
    __syncwarp();
    if (lane == 0) mbar_arrive(base + S::kQEmpty + 8 * slot);
  }
  if (!ok && lane == 0) {
    status_or(p.tm, HPA_STATUS_TIMEOUT);
    *abort_flag = 1;
  }
}

// ----------------------------------------------------------------------------- kernel
template <int KV, int RP>
__global__ void __launch_bounds__(KwCfg<KV, RP>::kThreads, RP <= 16 ? 2 : 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmk, const KeyWeightsParams p) {
  using S = KwCfg<KV, RP>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int c = blockIdx.x, warp = threadIdx.x >> 5;
  __shared__ MapHead head;  // read once, for all threads
  const uint32_t base = smem_u32(smem);
  if (threadIdx.x == 32) prefetch_tmap(&tmk);
  pdl_wait();  // nothing above reads what an earlier kernel writes
  if (threadIdx.x == 0) {
    head = read_map_head(p.tm, p.lay, p.B, p.C, c, p.q_len, false, c == 0 && blockIdx.y == 0, true);
    for (int i = 0; i < S::kStages; ++i) {
      mbar_init(base + S::kKvFull + 8 * i, 1);   // TMA bytes
      mbar_init(base + S::kKvEmpty + 8 * i, 1);  // MMA commit
    }
    for (int i = 0; i < S::kBufs; ++i) {
      mbar_init(base + S::kSFull + 8 * i, 1);            // MMA commit
      mbar_init(base + S::kSFree + 8 * i, kGroupWarps);  // the step's compute warps
    }
    for (int i = 0; i < S::kAccs; ++i) mbar_init(base + S::kAccFull + 8 * i, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(base + S::kQFull + 8 * i, 32 * S::kStagers);
      mbar_init(base + S::kQEmpty + 8 * i, 1 + kCompute);
    }
    mbar_init(base + S::kDrain, 1);
    *reinterpret_cast<int *>(smem + S::kAbort) = 0;
    fence_barrier_init();
  }
  if (threadIdx.x < RP) reinterpret_cast<int *>(smem + S::kJRow)[threadIdx.x] = threadIdx.x / p.G;
  __syncthreads();
  pdl_launch_dependents();
  if (!head.go) {
    if (threadIdx.x == 0) raised_done(p.tm, gridDim.x * gridDim.y);
    return;
  }
  if (warp == 0) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     base + S::kTmemAt),
                 "r"(S::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + S::kTmemAt);
  const MapHead m = head;
  if (warp < kCompute)
    kw_compute<KV, RP>(p, smem, m, tmem);
  else if (warp == kCompute)
    kw_producer<KV, RP>(p, &tmk, smem, m);
  else if (warp >= kCompute + 2)
    kw_stager<KV, RP>(p, smem, m, warp - kCompute - 2);
  else if ((threadIdx.x & 31) == 0)
    kw_issuer<KV, RP>(p, smem, m.s_end - m.s_begin, tmem);
  tc_fence_before();
  __syncthreads();
  mbar_wait_bounded_rolled(base + S::kDrain, 0, 1000000000ull);
  if (warp == 0) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(S::kTmem)
                 : "memory");
  }
}

template <int KV, int RP>
cudaError_t launch(const KeyWeightsParams &p, const CUtensorMap &tmk, cudaStream_t s) {
  using S = KwCfg<KV, RP>;
  static int configured[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(key_weights_kernel<KV, RP>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, S::kAlloc);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.C, p.Hkv);
  cfg.blockDim = dim3(S::kThreads);
  cfg.dynamicSmemBytes = S::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, key_weights_kernel<KV, RP>, tmk, p);
}

template <int KV>
cudaError_t launch_kv(const KeyWeightsParams &p, const CUtensorMap &tmk, cudaStream_t s) {
  return p.rows <= 8    ? launch<KV, 8>(p, tmk, s)
         : p.rows <= 16 ? launch<KV, 16>(p, tmk, s)
         : p.rows <= 32 ? launch<KV, 32>(p, tmk, s)
         : p.rows <= 48 ? launch<KV, 48>(p, tmk, s)
                        : launch<KV, 64>(p, tmk, s);
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsParams &p, const CUtensorMap &tmk, int kv_dtype,
                               cudaStream_t s) {
  return kv_dtype == HPA_KV_BF16 ? launch_kv<HPA_KV_BF16>(p, tmk, s)
                                 : launch_kv<HPA_KV_E4M3>(p, tmk, s);
}

}  // namespace hpa
