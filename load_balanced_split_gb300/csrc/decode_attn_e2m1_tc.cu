// Attention over 4-bit pages (HPA_KV_E2M1) for more than 16 query rows a KV head, on tcgen05.
//
// The products and their precision are those of decode_attn_e2m1.cu.  There an m16n8k16 MMA holds
// its scheduler for 8 cycles, so that the time grows with the rows.  Here a tile is 128 keys (two
// pages) and what a warp does for it depends on the rows in the softmax alone:
//   widen K, a key a thread, into tensor memory (f16, a key a lane): operand A of S^T = K Q^T;
//   S^T[128 keys][rows] in tensor memory, a key a thread: P = 2^(S - m), rounded to f16 into shared
//   memory, over the tile's own K codes;
//   widen V, a key a thread, into shared memory (f16, 128-byte swizzle), operand A (MN-major) of
//   O^T[128 dims][rows] += V^T P^T, which stays in tensor memory for the segment.
// Three teams of four warps take tiles in turn, each with its own S, O, running maxima and V
// buffer; K of a team's next tile is widened while the votes on the maximum come in, so that the
// first product runs under the softmax and V.  One thread per team issues both products: an MMA
// costs its thread some 87 cycles whatever its width (16 a tile: 1400), but three threads' overlap.
//
// What bounds it: a tile takes 1370 cycles of an SM (64 x 20000 keys with 24 rows: 369 us, 4.0
// TB/s), where the DRAM would allow 790 and shared memory's banks are taken for some 1100 (V as f16
// goes through it twice, 512; then P, codes and queries).  Neither less arithmetic (-6 % without
// any) nor fewer MMAs (0 %) change that much; the steps' meetings do: the fence between the stores
// and the second product is 10 %, a barrier for the votes was as much.  Against passes of up to 24
// rows in the other kernel, in us: 64 x 8000 keys with 32 rows 184 (260), with 64 rows 372 (564),
// 13 x 20011 with 20 rows 92 (102), in a window of 2000 with 24 rows 77 (76); but a short segment
// costs more here (Q, the first product and the teams' merge follow one another): 64 x 500 with 24
// rows 39 (33).  With 16 rows that kernel is ahead at every length.
//
// Tensor memory of a team, in columns: K 64, S 2 x 32, O 32.
#include <math_constants.h>

#include "e2m1.cuh"
#include "tcgen05.cuh"

namespace hpa {
namespace {

constexpr int kTeams = 3;
constexpr int kTeamThreads = 128;
constexpr int kConsumers = kTeams * kTeamThreads;
constexpr int kProducerWarp = kConsumers / 32;
constexpr int kIssuerWarp = kProducerWarp + 1;  // one for each team
constexpr int kThreads = (kIssuerWarp + kTeams) * 32;
// Rings of tiles.  K of a tile is widened while the team is at the tile before, and its place then
// holds P until the second product is done: three places a team.  V is needed an iteration later
// and free as soon as it is widened: one place a team, which the team's issuer fills (from L2,
// where the producer has asked for it with K).  With two places a team for K and V together the
// copies of a tile began when it was nearly needed (64 x 20000 with 24 rows 461 us, then 385; the
// issuers' copies gained most in windows, 80 to 75).
constexpr int kStages = 9, kVStages = 3;
// Copies may land out of order: a team that came to a stage whose tile before, another team's,
// had not landed would take that tile's phase for the end of its own.
static_assert(kStages % kTeams == 0 && kVStages % kTeams == 0, "each stage belongs to one team");
constexpr int kStageBytes = 2 * kUnit;  // two pages of K or of V
constexpr int kTileKeys = 2 * PAGE;
static_assert(kThreads == 512, "128 registers a thread");

// NG: groups of 8 query rows that hold one (3 or 4 of the MMAs' 4)
template <int NG>
struct Tc {
  static constexpr int N = 32;        // columns of an MMA
  static constexpr int kRows = 8 * NG;
  static_assert(kRows <= N && N == E2M1_MAX_ROWS, "a group's rows, and the buffers of N rows");
  static constexpr int kPRow = 2 * N;  // bytes of P of one key
  static constexpr int kPSwz = 4;      // descriptor mode of a 64-byte swizzle
  static_assert(kTileKeys * kPRow <= 2 * kUnit, "P lies over the tile's K");
  static constexpr int kTeamCols = 64 + 3 * N;
  static_assert(kTeams * kTeamCols <= 512, "tensor memory");
  static constexpr int kPacked = kStages * kStageBytes;  // V as it comes
  static constexpr int kV = kPacked + kVStages * kStageBytes;  // f16 V of each team's tile
  static constexpr int kVBytes = kTileKeys * HEAD_DIM * 2;
  static constexpr int kQ = kV + kTeams * kVBytes;    // query operand
  static constexpr int kRaw = kQ + N * HEAD_DIM * 2;  // query rows as they come
  static constexpr int kPair = kRaw + N * HEAD_DIM * 2;          // float2[teams][32]: sl, lift - m
  static constexpr int kMax = kPair + kTeams * 32 * 8;           // float[teams][32]
  static constexpr int kTop = kMax + kTeams * 32 * 4;            // float[teams][4][32]
  static constexpr int kFac = kTop + kTeams * 4 * 32 * 4;        // float[teams][32]
  static constexpr int kFactor = kFac + kTeams * 32 * 4;         // float[32]: sl of each row
  static constexpr int kTok = kFactor + 32 * 4;                  // int[32]: token of each row
  static constexpr int kNan = kTok + 32 * 4;                     // uint32[2][32]: NaN blocks
  static constexpr int kIds = kNan + 2 * 32 * 4;                   // int2[16]: pages of tiles
  static constexpr int kVotes = kIds + 16 * 8;                   // int4[teams][2]
  static constexpr int kInfo = kVotes + kTeams * 2 * 16;         // int4
  static constexpr int kBars = kInfo + 16;
  // full[9] empty[9] vfull[3] qfull qempty drain, and for each team: K ready, S ready, P
  // ready, PV done, votes
  static constexpr int kNumBars = 2 * kStages + kVStages + 3 + 5 * kTeams;
  static constexpr int kTmem = kBars + 8 * kNumBars;
  static constexpr int kFlag = kTmem + 4;
  static constexpr int kBytes = kFlag + 4;
  static constexpr int kAlloc = kBytes + 1024;  // room to align the base
  static_assert(kAlloc + 64 <= 232448, "shared memory of one CTA");
};
enum {
  B_FULL = 0,
  B_EMPTY = kStages,
  B_VFULL = 2 * kStages,
  B_QFULL = B_VFULL + kVStages,
  B_QEMPTY,
  B_DRAIN,
  B_TEAM
};
enum { T_K = 0, T_S, T_P, T_PV, T_VOTE };

__device__ __forceinline__ void tc_mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// A from tensor memory: a row a lane, two elements a column
__device__ __forceinline__ void tc_mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                              uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
__device__ __forceinline__ float warp_max_nan(float v) {
  float r;
  asm volatile("redux.sync.max.NaN.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}

// Barrier of a team, with the OR of its threads' predicates.
__device__ __forceinline__ bool team_any(int team, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(2 + team), "r"(kTeamThreads)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ bool all_consumers(bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
      "barrier.cta.red.and.pred p, 1, %2, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(x)), "r"(kConsumers)
      : "memory");
  return r != 0;
}

// Sums over the warp of its lanes' R values; lane r gets that of value r (r < R).
template <int R>
__device__ __forceinline__ float column_sum(const float (&v)[R], int lane) {
  float a[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) a[i] = i < R ? v[i] : 0.f;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const bool hi = lane & d;
#pragma unroll
    for (int i = 0; i < d; ++i) {
      const float give = hi ? a[i] : a[i + d], keep = hi ? a[i + d] : a[i];
      a[i] = keep + __shfl_xor_sync(kFull, give, d);
    }
  }
  return a[0];
}

// Tiles of a segment and those of one team: tile i of the segment is tile count + i of the CTA.
__device__ __forceinline__ int first_of_team(int team, int count) {
  return (team + kTeams - count % kTeams) % kTeams;
}

// ----------------------------------------------------------------------------- producer
template <int NG, bool WIN>
__device__ void producer(const AttnParams &p, const uint8_t *k_pool, const uint8_t *v_pool,
                         uint8_t *smem, const MapHead &head) {
  using S = Tc<NG>;
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const uint32_t base = smem_u32(smem), bars = base + S::kBars;
  const volatile int *abort_flag = reinterpret_cast<const volatile int *>(smem + S::kFlag);
  const uint64_t pol = l2_policy_evict_first();
  const int rows = group_rows(p), rb = row_base(p);
  // where this lane's query row lies behind its request's first
  const int64_t q_at =
      (static_cast<int64_t>((rb + lane) / p.G) * p.Hq + h * p.G + (rb + lane) % p.G) * HEAD_DIM;
  int2 *ids = reinterpret_cast<int2 *>(smem + S::kIds);
  int n0 = 0, nq = 0;  // tiles whose K, and segments, are on their way
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
      {  // the segment's place and query rows, once the last ones have been taken up
        bool good = true;
        if (lane == 0) good = wait_phase(bars + 8 * B_QEMPTY, (nq & 1) ^ 1, abort_flag);
        if (!__shfl_sync(kFull, good, 0)) {
          ok = false;
          break;
        }
        if (lane == 0) {
          *reinterpret_cast<int4 *>(smem + S::kInfo) =
              make_int4(cur.f.r, cur.f.L, cur.f.klo, cur.f.khi);
          mbar_arrive_expect_tx(bars + 8 * B_QFULL, rows * HEAD_DIM * 2);
        }
        __syncwarp();
        if (lane < rows)
          bulk_load(base + S::kRaw + lane * HEAD_DIM * 2,
                    p.q + static_cast<int64_t>(cur.f.r) * p.q_len * p.Hq * HEAD_DIM + q_at,
                    HEAD_DIM * 2, bars + 8 * B_QFULL);
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
        const int n = n0 + lane / 2, stage = n % kStages;  // lanes 2 i and 2 i + 1: tile i
        const uint32_t phase = (n / kStages) & 1;
        const uint32_t fb = bars + 8 * (B_FULL + stage);
        const uint32_t dst = base + stage * kStageBytes + (lane & 1) * kUnit;
        const int64_t at = (static_cast<int64_t>(id) * p.Hkv + h) * kUnit;
        const int tiles = (cnt + 1) / 2, second = __shfl_down_sync(kFull, id, 1);
        for (int i = 0; i < tiles; ++i) {
          bool good = true;
          if (lane == 2 * i) {
            good = wait_phase(bars + 8 * (B_EMPTY + stage), phase ^ 1, abort_flag);
            if (good) {
              ids[n & 15] = make_int2(id, lane + 1 < cnt ? second : -1);
              mbar_arrive_expect_tx(fb, (lane + 1 < cnt ? 2 : 1) * kUnit);
            }
          }
          if (!__all_sync(kFull, good)) {
            n0 += i;
            ok = false;
            break;
          }
          if (lane / 2 == i && lane < cnt) {
            bulk_load_hint(dst, k_pool + at, kUnit, fb, pol);
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(v_pool + at), "r"(kUnit)
                         : "memory");
          }
        }
        if (ok) n0 += tiles;
      }
      cur = nxt;
    }
  }
  if (!ok || *abort_flag) {
    if (lane == 0) {
      status_or(p.tm, HPA_STATUS_TIMEOUT);
      *reinterpret_cast<volatile int *>(smem + S::kFlag) = 1;
    }
    // never leave the CTA with copies still landing in its shared memory
    if (lane < kStages && n0 > lane) {
      const int last = n0 - 1 - (n0 - 1 - lane) % kStages;
      mbar_wait_bounded_rolled(bars + 8 * (B_FULL + lane), (last / kStages) & 1, 1000000000ull);
    }
    if (lane == 0 && nq > 0)
      mbar_wait_bounded_rolled(bars + 8 * B_QFULL, (nq - 1) & 1, 1000000000ull);
  }
}

// ----------------------------------------------------------------------------- MMA issue
// One thread for each team: S = K Q^T of its next tile, then O += V P of this one; and the copies
// of V, whose place is free when P of the tile before is there.
template <int NG>
__device__ void issuer(const AttnParams &p, const uint8_t *v_pool, uint8_t *smem,
                       const MapHead &head, uint32_t tmem, int team) {
  using S = Tc<NG>;
  constexpr int N = S::N;
  const uint32_t base = smem_u32(smem), bars = base + S::kBars;
  const uint32_t mine = bars + 8 * (B_TEAM + 5 * team);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kFlag);
  const uint32_t t0 = tmem + team * S::kTeamCols, o_t = t0 + 64 + 2 * N;
  const uint32_t vb = base + S::kV + team * S::kVBytes, qb = base + S::kQ;
  const uint32_t id_qk = tc_idesc(0, N, 0, 0), id_pv = tc_idesc(0, N, 1, 1);
  const int2 *ids = reinterpret_cast<const int2 *>(smem + S::kIds);
  const uint64_t pol = l2_policy_evict_first();
  const uint32_t vfull = bars + 8 * (B_VFULL + team);
  int count = 0, nk = 0, np = 0, nv = 0;  // tiles of the CTA; products and copies of this team
  bool ok = true;
  auto copy_v = [&](int n) {  // its K has come, so its pages are known
    const int2 id = ids[n & 15];
    const uint32_t dst = base + S::kPacked + team * kStageBytes;
    const int64_t h = blockIdx.y;
    mbar_arrive_expect_tx(vfull, (id.y < 0 ? 1 : 2) * kUnit);
    bulk_load_hint(dst, v_pool + (static_cast<int64_t>(id.x) * p.Hkv + h) * kUnit, kUnit, vfull,
                   pol);
    if (id.y >= 0)
      bulk_load_hint(dst + kUnit, v_pool + (static_cast<int64_t>(id.y) * p.Hkv + h) * kUnit, kUnit,
                     vfull, pol);
    ++nv;
  };
  auto qk = [&]() {
    if (!wait_phase(mine + 8 * T_K, nk & 1, abort_flag)) return false;
    tc_fence_after();
    const uint32_t s_t = t0 + 64 + (nk & 1) * N;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk)  // 16 dims
      tc_mma_f16_ts(s_t, t0 + 8 * kk, tc_desc(qb + (kk >> 2) * (N * 128) + (kk & 3) * 32, 16, 1024),
                    id_qk, kk > 0);
    tc_commit(mine + 8 * T_S);
    ++nk;
    return true;
  };
  for (int k = 0; k < head.s_end - head.s_begin && ok; ++k) {
    if (!wait_phase(bars + 8 * B_QFULL, k & 1, abort_flag)) {
      ok = false;
      break;
    }
    const int4 inf = *reinterpret_cast<const int4 *>(smem + S::kInfo);
    mbar_arrive(bars + 8 * B_QEMPTY);
    const int pg0 = inf.z / PAGE, pg1 = (inf.w + PAGE - 1) / PAGE, tiles = (pg1 - pg0 + 1) / 2;
    const int first = first_of_team(team, count);
    if (first < tiles) {
      ok = qk();
      if (ok) copy_v(count + first);
    }
    for (int i = first; i < tiles && ok; i += kTeams) {
      if (i + kTeams < tiles && !qk()) {
        ok = false;
        break;
      }
      if (!wait_phase(mine + 8 * T_P, np & 1, abort_flag)) {
        ok = false;
        break;
      }
      tc_fence_after();
      if (i + kTeams < tiles) copy_v(count + i + kTeams);
      const int stage = (count + i) % kStages;
      const uint32_t pb = base + stage * kStageBytes;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)  // 16 keys
        tc_mma_f16(o_t, tc_desc(vb + kk * 2048, kTileKeys * 128, 1024),
                   tc_desc(pb + kk * 16 * S::kPRow, 16, 8 * S::kPRow, S::kPSwz), id_pv,
                   i > first || kk > 0);
      tc_commit(bars + 8 * (B_EMPTY + stage));
      tc_commit(mine + 8 * T_PV);
      ++np;
    }
    count += tiles;
  }
  if (!ok) {
    status_or(p.tm, HPA_STATUS_TIMEOUT);
    *abort_flag = 1;
  }
  // never leave the CTA with copies still landing in its shared memory
  if ((!ok || *abort_flag) && nv > 0) mbar_wait_bounded_rolled(vfull, (nv - 1) & 1, 1000000000ull);
  tc_commit(bars + 8 * B_DRAIN);  // everything issued is done before the CTA frees its memory
}

// ----------------------------------------------------------------------------- consumer
template <int NG, bool WIN>
__device__ void consumer(const AttnParams &p, uint8_t *smem, const MapHead &head, uint32_t tmem) {
  using S = Tc<NG>;
  constexpr int N = S::N, R8 = S::kRows;
  const int tid = threadIdx.x, w = tid >> 5, lane = tid & 31, h = blockIdx.y;
  const int team = w >> 2, quarter = w & 3, kt = tid & 127;  // this thread's key of a tile
  const uint32_t base = smem_u32(smem), bars = base + S::kBars;
  const uint32_t mine = bars + 8 * (B_TEAM + 5 * team);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kFlag);
  // A wait that gives up raises the flag, so that no other lasts; the thread still takes part in
  // everything that follows, barriers among them.
  auto wait = [&](uint32_t bar, uint32_t parity) {
    const bool good = wait_phase(bar, parity, abort_flag);
    if (!good) *abort_flag = 1;
    __syncwarp();
    return good;
  };
  const uint32_t t0 = tmem + team * S::kTeamCols + (static_cast<uint32_t>(32 * quarter) << 16);
  const uint32_t o_t = t0 + 64 + 2 * N;
  const uint32_t vb = base + S::kV + team * S::kVBytes;
  const uint32_t pair = base + S::kPair + team * 256;
  float *pair_f = reinterpret_cast<float *>(smem + S::kPair) + team * 64;
  float *max_f = reinterpret_cast<float *>(smem + S::kMax);
  float *top_f = reinterpret_cast<float *>(smem + S::kTop) + team * 128;
  float *fac_f = reinterpret_cast<float *>(smem + S::kFac) + team * 32;
  int4 *votes = reinterpret_cast<int4 *>(smem + S::kVotes) + 2 * team;
  const float *factor = reinterpret_cast<const float *>(smem + S::kFactor);
  const int *tok = reinterpret_cast<const int *>(smem + S::kTok);
  const int G = p.G, q_len = p.q_len, rows = group_rows(p), rb = row_base(p);
  const float sl2 = p.scale_log2 * p.k_scale[h], vsc = p.v_scale[h];
  const int half = kt >> 6, row = kt & 63;   // which page of the tile, and where in it
  const int rot = (lane >> 1) & 3;           // chunk that this lane starts a row with

  int count = 0, n_s = 0;  // tiles of the CTA; of this team
  const int n_items = head.s_end - head.s_begin;
  for (int k = 0; k < n_items; ++k) {
    uint32_t *nan_rows = reinterpret_cast<uint32_t *>(smem + S::kNan) + 32 * (k & 1);
    bool ok = wait(bars + 8 * B_QFULL, k & 1);
    const int4 inf = *reinterpret_cast<const int4 *>(smem + S::kInfo);
    // Query rows as the B operand, f16, each scaled by 2^e; factor takes its scores to log2 units.
    for (int r = w; r < N; r += kConsumers / 32) {
      uint2 raw = make_uint2(0u, 0u);
      if (r < rows) raw = *reinterpret_cast<const uint2 *>(smem + S::kRaw + r * 256 + lane * 8);
      const float x[4] = {__uint_as_float(raw.x << 16), __uint_as_float(raw.x & 0xffff0000u),
                          __uint_as_float(raw.y << 16), __uint_as_float(raw.y & 0xffff0000u)};
      const float am = warp_max(fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])),
                                      fmaxf(fabsf(x[2]), fabsf(x[3]))));
      const int e = f16_row_exponent(am);
      // the sign of the score factor goes to the query, so that the larger score is the larger sum
      const float up = sl2 == 0.f ? 0.f : copysignf(exp2i(e), sl2);
      // never zero, which would make NaN of a hidden key's -inf; at 2^-126 all scores are nothing
      float down = sl2 == 0.f ? 1.f : fabsf(sl2) * exp2i(-e);
      if (down < exp2i(-126)) down = exp2i(-126);
      *reinterpret_cast<uint2 *>(smem + S::kQ + kmaj(r, 8 * lane, N * 128)) =
          make_uint2(pack_f16(x[0] * up, x[1] * up), pack_f16(x[2] * up, x[3] * up));
      if (lane == 0) {
        reinterpret_cast<float *>(smem + S::kFactor)[r] = down;
        reinterpret_cast<int *>(smem + S::kTok)[r] = r < rows ? (rb + r) / G : q_len - 1;
        nan_rows[r] = 0;
      }
    }
    fence_proxy_async_smem();  // the MMAs read them
    ok = all_consumers(ok);    // all go the same way from here on
    if (lane == 0) mbar_arrive(bars + 8 * B_QEMPTY);
    Seg f;
    f.r = inf.x, f.L = inf.y, f.klo = inf.z, f.khi = inf.w;
    f.pg0 = f.klo / PAGE;
    f.pg1 = ok ? (f.khi + PAGE - 1) / PAGE : f.pg0;  // no pages if the wait gave up
    if (ok && f.L < q_len && tid == 0) status_or(p.tm, HPA_STATUS_BAD_SEQLEN);
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
    auto sees = [&](int key, int j) {
      return key < lim_min + j && (!WIN || key < head.sinks || key >= win.start + j);
    };
    if (kt < 32) {
      pair_f[2 * kt] = kt < R8 ? factor[kt] : 1.f;
      pair_f[2 * kt + 1] = 0.f;
      max_f[team * 32 + kt] = -CUDART_INF_F;
    }
    float l[R8];
#pragma unroll
    for (int r = 0; r < R8; ++r) l[r] = 0.f;
    team_any(team, false);

    const int tiles = (f.pg1 - f.pg0 + 1) / 2, first = first_of_team(team, count);
    // K of a tile: this thread's key into its lane of tensor memory
    auto widen_k = [&](int i) {
      const int n = count + i, stage = n % kStages;
      ok = wait(bars + 8 * (B_FULL + stage), (n / kStages) & 1) && ok;
      const uint8_t *unit = smem + stage * kStageBytes + half * kUnit;
      const uint2 sc = *reinterpret_cast<const uint2 *>(unit + 4096 + row * 8);
      uint4 c[4];  // chunk (u + rot) % 4 of the key's 64 bytes: lanes 64 bytes apart would collide
#pragma unroll
      for (int u = 0; u < 4; ++u)
        c[u] = *reinterpret_cast<const uint4 *>(unit + row * 64 + ((u + rot) & 3) * 16);
      auto pick = [](bool s, const uint4 &a, const uint4 &b) {
        return make_uint4(s ? a.x : b.x, s ? a.y : b.y, s ? a.z : b.z, s ? a.w : b.w);
      };
      uint4 d[4], q[4];  // back in order
#pragma unroll
      for (int u = 0; u < 4; ++u) d[u] = pick(rot & 1, c[(u + 3) & 3], c[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u) q[u] = pick(rot & 2, d[(u + 2) & 3], d[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u) {  // 32 dims, two blocks
        const uint32_t two = e4m3x2_to_f16x2(
            static_cast<uint16_t>((u < 2 ? sc.x : sc.y) >> (16 * (u & 1))));
        const uint32_t s0 = both_halves<0>(two), s1 = both_halves<1>(two);
        const uint32_t word[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
        uint32_t out[16];
#pragma unroll
        for (int v = 0; v < 4; ++v) {
          uint32_t e[4];
          widen8(word[v], e);
#pragma unroll
          for (int b = 0; b < 4; ++b) out[4 * v + b] = mul_f16x2(e[b], v < 2 ? s0 : s1);
        }
        tc_st16(t0 + 16 * u, out);
      }
      tc_wait_st();
      tc_fence_before();
      mbar_arrive(mine + 8 * T_K);
    };

    if (first < tiles) widen_k(first);
    bool unset = true;  // a row of the team has met no key yet: it has no maximum to compare with
    for (int i = first; i < tiles; i += kTeams) {
      ok = wait(mine + 8 * T_S, n_s & 1) && ok;
      tc_fence_after();
      const int n = count + i, stage = n % kStages;
      const int pg = f.pg0 + 2 * i + half;
      const bool here = pg < f.pg1;  // the segment's last tile may lack a page
      const int key = (WIN ? win.real_page(pg) : pg) * PAGE + row;
      const bool edge = f.pg0 + 2 * i < clear0 || f.pg0 + 2 * i + 2 > clear1 ||
                        f.pg0 + 2 * i + 2 > f.pg1;
      float x[R8];
#pragma unroll
      for (int g = 0; g < NG; ++g)
        tc_ld8(t0 + 64 + (n_s & 1) * N + 8 * g, *reinterpret_cast<float(*)[8]>(&x[8 * g]));
      tc_wait_ld();
      if (edge) {
#pragma unroll
        for (int r = 0; r < R8; ++r)
          if (!here || !sees(key, tok[r])) x[r] = -CUDART_INF_F;
      }
      // running maximum: moves when a score passes it by more than the slack
      float most = -CUDART_INF_F;
#pragma unroll
      for (int r = 0; r < R8; r += 2) {
        uint32_t a, b, c, d;
        lds128(pair + 8 * r, a, b, c, d);
        x[r] = fmaf(x[r], __uint_as_float(a), __uint_as_float(b));  // less the maximum, plus lift
        x[r + 1] = fmaf(x[r + 1], __uint_as_float(c), __uint_as_float(d));
        most = fmaxf(most, fmaxf(x[r], x[r + 1]));
      }
      // The warps' votes; while they come in, K of the next tile.  Every warp of the team gets here
      // within its waits' limits, so this wait always ends, and all read the same votes.
      const bool over = unset || __any_sync(kFull, most > kRescaleSlack + kLift);
      if (lane == 0) {
        reinterpret_cast<int *>(votes + (n_s & 1))[quarter] = over;
        mbar_arrive(mine + 8 * T_VOTE);
      }
      if (i + kTeams < tiles) widen_k(i + kTeams);
      mbar_wait_bounded_rolled(mine + 8 * T_VOTE, n_s & 1, 60000000000ull);
      __syncwarp();
      const int4 vote = votes[n_s & 1];
      if (vote.x | vote.y | vote.z | vote.w) {
#pragma unroll
        for (int g = 0; g < NG; ++g) {  // the scores themselves again
          float v[8];
          tc_ld8(t0 + 64 + (n_s & 1) * N + 8 * g, v);
          tc_wait_ld();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int r = 8 * g + e;
            x[r] = x[r] == -CUDART_INF_F ? x[r] : __fmul_rn(v[e], pair_f[2 * r]);
            const float t = warp_max_nan(x[r]);
            if (lane == 0) top_f[quarter * 32 + r] = t;
          }
        }
        team_any(team, false);
        bool none = false;
        if (kt < R8) {
          const float m = max_f[team * 32 + kt];
          const float t = max_nan(max_nan(top_f[kt], top_f[32 + kt]),
                                  max_nan(top_f[64 + kt], top_f[96 + kt]));
          // (a NaN becomes the maximum: its row is NaN whatever that is, and not without one)
          const float mn = t - m <= kRescaleSlack ? m : t;
          fac_f[kt] = mn == -CUDART_INF_F ? 1.f : exp2f(m - mn);
          max_f[team * 32 + kt] = mn;
          none = mn == -CUDART_INF_F;
          // rounded down: with the slack it must not pass what f16 holds where a step of fp32 at the
          // maximum is as large as the lift (the scores are rounded products here)
          pair_f[2 * kt + 1] = none ? 0.f : __fsub_rd(kLift, mn);
        }
        unset = team_any(team, none);
        if (i > first) {  // O of the tiles before is at rest once their products are done
          ok = wait(mine + 8 * T_PV, (n_s - 1) & 1) && ok;
          tc_fence_after();
#pragma unroll
          for (int g = 0; g < NG; ++g) {
            float o[8];
            tc_ld8(o_t + 8 * g, o);
            tc_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] *= fac_f[8 * g + e];
            tc_st8(o_t + 8 * g, o);
          }
          tc_wait_st();
        }
#pragma unroll
        for (int r = 0; r < R8; ++r) {
          l[r] *= fac_f[r];
          x[r] += pair_f[2 * r + 1];  // a row still without a key has -inf alone
        }
      }
      // probabilities; their sums in fp32 before the rounding to f16
      uint32_t pk2[R8 / 2];
#pragma unroll
      for (int r = 0; r < R8; r += 2) {
        const float a = exp2f(x[r]), b = exp2f(x[r + 1]);
        l[r] += a;
        l[r + 1] += b;
        pk2[r / 2] = pack_f16(a, b);
      }
      // The tile's K is read, and the products of the tile before are done with V: P over the one,
      // V over the other.
      if (i > first) ok = wait(mine + 8 * T_PV, (n_s - 1) & 1) && ok;
      const uint32_t pb = base + stage * kStageBytes;
#pragma unroll
      for (int g = 0; g < NG; ++g)
        sts128(pb + mnmaj(kt, 16 * g, S::kPRow), pk2[4 * g], pk2[4 * g + 1], pk2[4 * g + 2],
               pk2[4 * g + 3]);
      {
        const int vst = n % kVStages;
        ok = wait(bars + 8 * (B_VFULL + vst), (n / kVStages) & 1) && ok;
        const uint8_t *unit = smem + S::kPacked + vst * kStageBytes + half * kUnit;
        uint2 sc = *reinterpret_cast<const uint2 *>(unit + 4096 + row * 8);
        if (edge) {
          // a key that no token sees: its scales are taken as zero
          const bool hidden = !here || key >= f.L ||
                              (WIN && key >= head.sinks && key < win.low);
          if (hidden) sc = make_uint2(0u, 0u);
          if (q_len > 1 && !hidden && !(sees(key, 0) && sees(key, q_len - 1))) {
            // A NaN that some tokens see and others do not: 0 * NaN would reach every row, so the
            // scale is taken as zero and the rows that see the key lose the block's 16 dims.
            uint32_t blocks = 0;
#pragma unroll
            for (int b = 0; b < 8; ++b)
              if (e4m3_nan((b < 4 ? sc.x : sc.y) >> (8 * (b & 3)))) blocks |= 1u << b;
            if (blocks) {
#pragma unroll 1
              for (int r = 0; r < rows; ++r)
                if (sees(key, tok[r])) atomicOr(nan_rows + r, blocks);
#pragma unroll
              for (int b = 0; b < 4; ++b) {
                if ((blocks >> b) & 1) sc.x &= ~(0xffu << (8 * b));
                if ((blocks >> (b + 4)) & 1) sc.y &= ~(0xffu << (8 * b));
              }
            }
          }
        }
        const uint32_t at = vb + kt * 128;
#pragma unroll
        for (int u = 0; u < 4; ++u) {  // chunks in the lane's order: no two lanes collide
          const int c = (u + rot) & 3;
          const uint4 q = *reinterpret_cast<const uint4 *>(unit + row * 64 + c * 16);
          const uint32_t two =
              e4m3x2_to_f16x2(static_cast<uint16_t>((c & 2 ? sc.y : sc.x) >> (16 * (c & 1))));
          const uint32_t s0 = both_halves<0>(two), s1 = both_halves<1>(two);
          const uint32_t word[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int v = 0; v < 4; ++v) {  // 8 dims: 16-byte chunk 4 (c % 2) + v of block c / 2
            uint32_t e[4];
            widen8(word[v], e);
#pragma unroll
            for (int b = 0; b < 4; ++b) e[b] = mul_f16x2(e[b], v < 2 ? s0 : s1);
            sts128(at + (c >> 1) * (kTileKeys * 128) + (((4 * (c & 1) + v) ^ (kt & 7)) << 4), e[0],
                   e[1], e[2], e[3]);
          }
        }
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(mine + 8 * T_P);
      ++n_s;
    }
    count += tiles;
    const bool started = first < tiles;

    // ---- segment end: the teams' (m, l, O) together, and the partial
    if (started) {
      ok = wait(mine + 8 * T_PV, (n_s - 1) & 1) && ok;
      tc_fence_after();
    }
    top_f[quarter * 32 + lane] = column_sum<R8>(l, lane);  // the warp's sum of row `lane`
    if (!ok && lane == 0) status_or(p.tm, HPA_STATUS_TIMEOUT);
    all_consumers(true);
    auto row_stats = [&](int r, float &M, float &sum) {
      const float *tops = reinterpret_cast<const float *>(smem + S::kTop);
      M = -CUDART_INF_F;
#pragma unroll
      for (int t = 0; t < kTeams; ++t) M = fmaxf(M, max_f[t * 32 + r]);
      M = M == -CUDART_INF_F ? 0.f : M;
      sum = 0.f;
#pragma unroll
      for (int t = 0; t < kTeams; ++t) {
        const float *v = tops + t * 128 + r;
        sum += (v[0] + v[32] + v[64] + v[96]) * exp2f(max_f[t * 32 + r] - M);
      }
    };
    float fac = 0.f;  // row `lane`: what takes this team's O to the partial's
    if (lane < R8) {
      float M, sum;
      row_stats(lane, M, sum);
      fac = sum == 0.f ? 0.f : exp2f(max_f[team * 32 + lane] - M) / sum * vsc;
    }
    float *buf = reinterpret_cast<float *>(smem + S::kV);
    float *mybuf = buf + team * (S::kVBytes / 4);  // [rows][128], over the team's V
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (started) {
        tc_ld8(o_t + 8 * g, o);
        tc_wait_ld();
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = o[e] * __shfl_sync(kFull, fac, 8 * g + e);
        mybuf[(8 * g + e) * HEAD_DIM + kt] = started ? x : 0.f;
      }
    }
    tc_fence_before();
    all_consumers(true);
    const int s = head.s_begin + k;
    for (int v = tid; v < rows * (HEAD_DIM / 4); v += kConsumers) {
      const int r = v / (HEAD_DIM / 4), c4 = v % (HEAD_DIM / 4);
      const int j = (rb + r) / G, gq = (rb + r) % G;
      const int64_t dst = (static_cast<int64_t>(s) * q_len + j) * p.Hq + h * G + gq;
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int t = 0; t < kTeams; ++t) {
        const float4 b =
            reinterpret_cast<const float4 *>(buf + t * (S::kVBytes / 4) + r * HEAD_DIM)[c4];
        a = make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w);
      }
      if ((nan_rows[r] >> (c4 / 4)) & 1)
        a = make_float4(CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F, CUDART_NAN_F);
      reinterpret_cast<float4 *>(p.partial_o + dst * HEAD_DIM)[c4] = a;
    }
    if (tid < rows) {
      float M, sum;
      row_stats(tid, M, sum);
      const int j = (rb + tid) / G, gq = (rb + tid) % G;
      // a row that sees a NaN has no sum: +inf, beside which no other partial counts, makes the
      // combine's result NaN (it passes over -inf and NaN)
      p.partial_lse[(static_cast<int64_t>(s) * q_len + j) * p.Hq + h * G + gq] =
          sum == 0.f  ? -CUDART_INF_F
          : sum > 0.f ? (M - kLift + log2f(sum)) * 0.69314718055994531f
                      : CUDART_INF_F;
    }
    // the next segment's first barrier stands before all that would write over what is read here
  }
}

template <int NG, bool WIN>
__global__ void __launch_bounds__(kThreads, 1)
    decode_attn_e2m1_tc_kernel(const uint8_t *__restrict__ k_pool,
                               const uint8_t *__restrict__ v_pool, const AttnParams p) {
  using S = Tc<NG>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ MapHead head;
  const int c = blockIdx.x, w = threadIdx.x >> 5;
  const uint32_t base = smem_u32(smem), bars = base + S::kBars;
  if (threadIdx.x == 0) {
    for (int st = 0; st < kStages; ++st) {
      mbar_init(bars + 8 * (B_FULL + st), 1);
      mbar_init(bars + 8 * (B_EMPTY + st), 1);
    }
    for (int st = 0; st < kVStages; ++st) mbar_init(bars + 8 * (B_VFULL + st), 1);
    mbar_init(bars + 8 * B_QFULL, 1);
    mbar_init(bars + 8 * B_QEMPTY, kConsumers / 32 + kTeams);
    mbar_init(bars + 8 * B_DRAIN, kTeams);
    for (int t = 0; t < kTeams; ++t) {
      mbar_init(bars + 8 * (B_TEAM + 5 * t + T_K), kTeamThreads);
      mbar_init(bars + 8 * (B_TEAM + 5 * t + T_S), 1);
      mbar_init(bars + 8 * (B_TEAM + 5 * t + T_P), kTeamThreads);
      mbar_init(bars + 8 * (B_TEAM + 5 * t + T_PV), 1);
      mbar_init(bars + 8 * (B_TEAM + 5 * t + T_VOTE), 4);
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
  if (w == kProducerWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                     base + S::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + S::kTmem);
  const MapHead m = head;
  if (w < kProducerWarp) {
    consumer<NG, WIN>(p, smem, m, tmem);
  } else if (w == kProducerWarp) {
    producer<NG, WIN>(p, k_pool, v_pool, smem, m);
  } else {
    if ((threadIdx.x & 31) == 0) issuer<NG>(p, v_pool, smem, m, tmem, w - kIssuerWarp);
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (w == kProducerWarp) {
    if ((threadIdx.x & 31) == 0 && !mbar_wait_bounded_rolled(bars + 8 * B_DRAIN, 0))
      status_or(p.tm, HPA_STATUS_TIMEOUT);
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
  }
}

template <int NG, bool WIN>
cudaError_t launch(const AttnParams &p, const void *k_pool, const void *v_pool, cudaStream_t s) {
  static int configured[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(decode_attn_e2m1_tc_kernel<NG, WIN>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, Tc<NG>::kAlloc);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = 1;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(p.C, p.Hkv, (p.rows + p.group - 1) / p.group);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Tc<NG>::kAlloc;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, decode_attn_e2m1_tc_kernel<NG, WIN>,
                            static_cast<const uint8_t *>(k_pool),
                            static_cast<const uint8_t *>(v_pool), p);
}

}  // namespace

cudaError_t launch_decode_attn_e2m1_tc(const AttnParams &p, const void *k_pool, const void *v_pool,
                                       cudaStream_t s) {
  const auto run = p.group <= 24 ? (p.window ? launch<3, true> : launch<3, false>)
                                 : (p.window ? launch<4, true> : launch<4, false>);
  return run(p, k_pool, v_pool, s);
}

}  // namespace hpa
