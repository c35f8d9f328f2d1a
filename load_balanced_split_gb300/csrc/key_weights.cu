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
//  * one CTA per (partition, KV head): a TMA producer warp and groups of four consumer
//    warps; a page of K (16 KB bf16 / 8 KB E4M3) and the page's 256 bytes of acc_in are
//    one pipeline stage, so the read of the accumulators needs no latency of its own;
//  * keys are the M dimension of the m16n8k16 MMAs and query rows the N dimension: the 8
//    rows of a usual GQA group fill N exactly, where rows as M would pad them to 16;
//  * a warp owns 16 keys and all rows, so it sums its exponentials in registers and two
//    lane exchanges, and writes 16 accumulators: no exchange between warps, no atomics,
//    the same sums in the same order on every run;
//  * up to 16 rows the query fragments stay in registers; above, they are read from
//    shared memory for every 16 keys, in fragment order (8-byte conflict-free loads);
//  * the producer warp stages each segment's query rows ahead: fragment order, for E4M3
//    pages converted to f16 after a power-of-two scale per row (exact, as in
//    decode_attn.cu), with each row's score factor and log-sum-exp in base 2.
#include <math_constants.h>

#include "hpa_internal.cuh"

namespace hpa {
namespace {

constexpr uint32_t kFull = 0xffffffffu;
constexpr int kGroupWarps = 4;      // consumer warps that share a page: 16 keys each
constexpr int kQStride = 288;       // bytes per staged query row: 64-bit loads hit all banks
constexpr int kAccBytes = PAGE * 4;

// RT: n-tiles of 8 query rows kept in registers (1 or 2); 0: 3 to 8 tiles, from shared memory.
template <int KV, int RT>
struct KwCfg {
  static constexpr int kGroups = RT ? 1 : 2;
  static constexpr int kConsumers = kGroups * kGroupWarps;
  static constexpr int kThreads = (kConsumers + 1) * 32;
  static constexpr int kRows = RT ? 8 * RT : MAX_ROWS_TOTAL;
  static constexpr int kKBytes = KV == HPA_KV_BF16 ? 16384 : 8192;
  static constexpr int kStages = KV == HPA_KV_BF16 ? 5 : 10;
  static constexpr int kAcc = kStages * kKBytes;            // float[kStages][64]
  static constexpr int kQ = kAcc + kStages * kAccBytes;     // two slots of query rows
  static constexpr int kQSlot = kRows * kQStride;
  static constexpr int kRow = kQ + 2 * kQSlot;              // float2[2][kRows]: factor, lse
  static constexpr int kInfo = kRow + 2 * kRows * 8;        // int4[2]
  static constexpr int kPid = kInfo + 32;                   // int[kStages]
  static constexpr int kBars = (kPid + kStages * 4 + 15) & ~15;
  static constexpr int kFlag = kBars + (2 * kStages + 4) * 8;
  static constexpr int kAlloc = kFlag + 16 + 1024;          // room to align the base
};

// A segment's walk: real pages of request r over the compact (or plain) key range.
struct KwSeg {
  int r, L, pg0, pg1;
  WinSpan win;
};

__device__ __forceinline__ KwSeg kw_seg(const KeyWeightsParams &p, bool windowed, int window,
                                        int sinks, int s, int tile, bool report) {
  const int c = blockIdx.x;
  const SegRow sr = windowed ? read_seg_row<true>(p.tm, p.lay, p.B, s, c, tile, report)
                             : read_seg_row<false>(p.tm, p.lay, p.B, s, c, tile, report);
  KwSeg f;
  f.r = sr.r;
  f.L = sr.L;
  f.pg0 = sr.klo / PAGE;
  f.pg1 = (sr.khi + PAGE - 1) / PAGE;
  f.win = WinSpan{};
  if (sr.L < p.q_len) {
    if (report) status_or(p.tm, HPA_STATUS_BAD_SEQLEN);
    f.pg1 = f.pg0;
  } else if (windowed && f.pg0 < f.pg1) {
    f.win = WinSpan::make(sr.L, p.q_len, window, sinks);
  }
  return f;
}

// (score factor, lse in base 2) of a row; a row that sees no key (lse -inf) weighs nothing.
__device__ __forceinline__ float2 row_consts(float factor, float lse) {
  const float l2 = lse * 1.4426950408889634f;
  return make_float2(factor, l2 == -CUDART_INF_F ? CUDART_INF_F : l2);
}

// ----------------------------------------------------------------------------- producer
template <int KV, int RT>
__device__ void kw_stage_rows(const KeyWeightsParams &p, uint8_t *smem, int slot, int r, int h) {
  using S = KwCfg<KV, RT>;
  const int lane = threadIdx.x & 31, G = p.G;
  uint8_t *qs = smem + S::kQ + slot * S::kQSlot;
  float2 *rc = reinterpret_cast<float2 *>(smem + S::kRow) + slot * S::kRows;
  const int padded = RT ? S::kRows : (p.rows + 7) & ~7;
  float factor = p.scale_log2;
  if (KV == HPA_KV_E4M3) factor *= p.k_scale[h];
  for (int row0 = 0; row0 < padded; row0 += 8) {
    uint2 x[8];
    float lse = 0.f;  // lane i < 8: of row row0 + i
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // eight rows' loads in flight; lane: dims [4 lane, 4 lane + 4)
      const int row = row0 + i;
      x[i] = make_uint2(0u, 0u);
      if (row < p.rows) {
        const int64_t at = (static_cast<int64_t>(r) * p.q_len + row / G) * p.Hq + h * G + row % G;
        x[i] = reinterpret_cast<const uint2 *>(p.q + at * HEAD_DIM)[lane];
        if (lane == i) lse = p.lse[at];
      }
    }
    float mine = 0.f;  // lane i: row i's score factor
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint8_t *dst = qs + (row0 + i) * kQStride;
      if (KV == HPA_KV_BF16) {
        // k-step lane / 4; its thread qd holds dims 2 qd, 2 qd + 1, 2 qd + 8, 2 qd + 9
        const int in = 4 * (lane & 3), at = (lane >> 2) * 32 + (in & 4) * 4 + (in >> 3) * 4;
        *reinterpret_cast<uint32_t *>(dst + at) = x[i].x;
        *reinterpret_cast<uint32_t *>(dst + at + 8) = x[i].y;
        if (lane == i) mine = factor;
      } else {
        const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x[i].x));
        const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&x[i].y));
        float m = fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y)));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        const int e = f16_row_exponent(m);
        const float sc = exp2i(e);
        // k-step ks of thread qd is dims 32 qd + 4 ks + [0, 4): lane = 8 qd + ks
        uint2 v;
        v.x = pack_f16(a.x * sc, a.y * sc);
        v.y = pack_f16(b.x * sc, b.y * sc);
        *reinterpret_cast<uint2 *>(dst + (lane & 7) * 32 + (lane >> 3) * 8) = v;
        if (lane == i) mine = factor * exp2i(-e);
      }
    }
    if (lane < 8)
      rc[row0 + lane] = row0 + lane < p.rows ? row_consts(mine, lse)
                                             : make_float2(0.f, CUDART_INF_F);
  }
}

template <int KV, int RT>
__device__ void kw_producer(const KeyWeightsParams &p, const CUtensorMap *tmk, uint8_t *smem,
                            int s_begin, int s_end, int tile, bool windowed) {
  using S = KwCfg<KV, RT>;
  const int lane = threadIdx.x & 31, h = blockIdx.y;
  const uint32_t base = smem_u32(smem);
  const uint32_t full0 = base + S::kBars, empty0 = full0 + 8 * S::kStages;
  const uint32_t qfull0 = empty0 + 8 * S::kStages, qempty0 = qfull0 + 16;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kFlag);
  volatile int *pids = reinterpret_cast<volatile int *>(smem + S::kPid);
  const int window = windowed ? p.tm[TM_WINDOW] : 0, sinks = windowed ? p.tm[TM_SINKS] : 0;
  uint64_t pol = 0;
  if (lane == 0) {
    pol = l2_policy_evict_first();
    prefetch_tmap(tmk);
  }
  int stage = 0;
  uint32_t phase = 0, issued = 0, parity_bits = 0;
  bool ok = true;
  for (int k = 0; k < s_end - s_begin && ok; ++k) {
    const KwSeg f = kw_seg(p, windowed, window, sinks, s_begin + k, tile, lane == 0);
    const int slot = k & 1;
    int good = 1;
    if (lane == 0) good = !*abort_flag && mbar_wait_bounded(qempty0 + 8 * slot, ((k >> 1) & 1) ^ 1);
    if (!__shfl_sync(kFull, good, 0)) {
      ok = false;
      break;
    }
    kw_stage_rows<KV, RT>(p, smem, slot, f.r, h);
    if (lane == 0)
      reinterpret_cast<int4 *>(smem + S::kInfo)[slot] = make_int4(f.r, f.L, f.pg0, f.pg1);
    mbar_arrive(qfull0 + 8 * slot);  // every lane publishes its own stores
    const int pstart = p.page_indptr[f.r];
    const int pcount = p.page_indptr[f.r + 1] - pstart;
    for (int pb = f.pg0; pb < f.pg1 && ok; pb += 32) {
      const int cnt = min(32, f.pg1 - pb);
      int id = 0;
      if (lane < cnt) {
        const int pg = windowed ? f.win.real_page(pb + lane) : pb + lane;
        id = pg < pcount ? p.page_indices[pstart + pg] : -1;
        if (id < 0 || id >= p.num_pages) {
          status_or(p.tm, HPA_STATUS_BAD_PAGE);
          id = -1;  // page 0 is read in its place and nothing is written
        }
      }
      for (int i = 0; i < cnt; ++i) {
        const int pid = __shfl_sync(kFull, id, i);
        good = 1;
        if (lane == 0) {
          if (*abort_flag || !mbar_wait_bounded(empty0 + 8 * stage, phase ^ 1)) {
            good = 0;
          } else {
            const uint32_t fb = full0 + 8 * stage, dst = base + stage * S::kKBytes;
            const int z = max(pid, 0) * p.Hkv + h;
            pids[stage] = pid;
            mbar_arrive_expect_tx(fb, S::kKBytes + (p.acc_in ? kAccBytes : 0));
            tma_load_3d(dst, tmk, fb, 0, 0, z, pol);
            if (KV == HPA_KV_BF16) tma_load_3d(dst + 8192, tmk, fb, 64, 0, z, pol);
            if (p.acc_in)
              bulk_load(base + S::kAcc + stage * kAccBytes,
                        p.acc_in + static_cast<int64_t>(z) * PAGE, kAccBytes, fb);
            issued |= 1u << stage;
            parity_bits = (parity_bits & ~(1u << stage)) | (phase << stage);
          }
        }
        ok = __shfl_sync(kFull, good, 0) != 0;
        if (!ok) break;
        if (++stage == S::kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
  }
  if (!ok && lane == 0) {
    status_or(p.tm, HPA_STATUS_TIMEOUT);
    *abort_flag = 1;
    for (int st = 0; st < S::kStages; ++st)  // no copy may land after the CTA has left
      if (issued & (1u << st))
        mbar_wait_bounded(full0 + 8 * st, (parity_bits >> st) & 1u, 1000000000ull);
  }
}

// ----------------------------------------------------------------------------- consumer
// A fragments (16 keys x 128 dims) of the warp's keys of the page at kt.
template <int KV>
__device__ __forceinline__ void kw_load_keys(uint32_t (&a)[8][4], uint32_t kt, int w, int lane) {
  if (KV == HPA_KV_BF16) {
    const int mi = lane >> 3, key = 16 * w + (mi & 1) * 8 + (lane & 7);
    const uint32_t row = kt + key * 128;
#pragma unroll
    for (int ks = 0; ks < 8; ++ks) {
      const int chunk = (ks & 3) * 2 + (mi >> 1);
      ldsm_x4(row + (ks >> 2) * 8192 + ((chunk ^ (lane & 7)) << 4), a[ks][0], a[ks][1], a[ks][2],
              a[ks][3]);
    }
  } else {
    // thread (r8, qd) widens dims [32 qd, 32 qd + 32) of keys r8 and r8 + 8; k-step ks
    // is dims 32 qd + 4 ks + [0, 4), as the query rows are staged
    const int r8 = lane >> 2, qd = lane & 3;
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const uint32_t row = kt + (16 * w + 8 * hf + r8) * 128;
      uint32_t u[8];
      lds128(row + (((2 * qd) ^ r8) << 4), u[0], u[1], u[2], u[3]);
      lds128(row + (((2 * qd + 1) ^ r8) << 4), u[4], u[5], u[6], u[7]);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks) {
        a[ks][hf] = e4m3x2_to_f16x2(static_cast<uint16_t>(u[ks] & 0xffffu));
        a[ks][2 + hf] = e4m3x2_to_f16x2(static_cast<uint16_t>(u[ks] >> 16));
      }
    }
  }
}

__device__ __forceinline__ void kw_load_rows(uint32_t (&b)[8][2], uint32_t qrow, int lane) {
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    lds64(qrow + (lane >> 2) * kQStride + ks * 32 + (lane & 3) * 8, b[ks][0], b[ks][1]);
}

template <int KV, int RT>
__device__ void kw_consumer(const KeyWeightsParams &p, uint8_t *smem, int s_begin, int s_end,
                            bool windowed) {
  using S = KwCfg<KV, RT>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int w = warp % kGroupWarps, group = warp / kGroupWarps;
  const int r8 = lane >> 2, qd = lane & 3, h = blockIdx.y;
  const uint32_t base = smem_u32(smem);
  const uint32_t full0 = base + S::kBars, empty0 = full0 + 8 * S::kStages;
  const uint32_t qfull0 = empty0 + 8 * S::kStages, qempty0 = qfull0 + 16;
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + S::kFlag);
  volatile int *pids = reinterpret_cast<volatile int *>(smem + S::kPid);
  const int window = windowed ? p.tm[TM_WINDOW] : 0, sinks = windowed ? p.tm[TM_SINKS] : 0;
  const int q_len = p.q_len, n_tiles = RT ? RT : (p.rows + 7) / 8;
  int stage = 0, turn = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int k = 0; k < s_end - s_begin && ok; ++k) {
    const int slot = k & 1;
    ok = __all_sync(kFull, !*abort_flag && mbar_wait_bounded(qfull0 + 8 * slot, (k >> 1) & 1));
    if (!ok) break;
    const int4 info = reinterpret_cast<const int4 *>(smem + S::kInfo)[slot];
    const int L = info.y, pg0 = info.z, pg1 = info.w;
    WinSpan win = {};
    if (windowed && pg0 < pg1) win = WinSpan::make(L, q_len, window, sinks);
    const int lim_min = L - q_len + 1;  // first key hidden from some row
    const uint32_t qs = base + S::kQ + slot * S::kQSlot;
    const float4 *rc = reinterpret_cast<const float4 *>(smem + S::kRow) + slot * (S::kRows / 2);
    uint32_t qb[RT ? RT : 1][8][2];
    float4 qc[RT ? RT : 1];
    if (RT) {
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        kw_load_rows(qb[t], qs + t * 8 * kQStride, lane);
        qc[t] = rc[4 * t + qd];
      }
    }
    for (int pg = pg0; pg < pg1; ++pg) {
      const bool mine = S::kGroups == 1 || turn == group;
      if (S::kGroups > 1 && ++turn == S::kGroups) turn = 0;
      if (mine) {
        ok = __all_sync(kFull, !*abort_flag && mbar_wait_bounded(full0 + 8 * stage, phase));
        if (!ok) break;
        const int key0 = (windowed ? win.real_page(pg) : pg) * PAGE, wk = key0 + 16 * w;
        uint32_t a[8][4];
        kw_load_keys<KV>(a, base + stage * S::kKBytes, w, lane);
        // some rows do not see some of the warp's keys: the causal end, a window's start
        const bool part = wk + 16 > lim_min ||
                          (windowed && wk < win.start + q_len - 1 && wk + 16 > sinks);
        float w0 = 0.f, w1 = 0.f;  // keys wk + r8 and wk + r8 + 8, rows 8 t + 2 qd + {0, 1}
        auto tile = [&](const uint32_t(&b)[8][2], float4 c, int t) {
          float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            if (KV == HPA_KV_BF16) mma_bf16(s, a[ks], b[ks][0], b[ks][1]);
            else mma_f16(s, a[ks], b[ks][0], b[ks][1]);
          }
          float e[4];
          e[0] = exp2f(fmaf(s[0], c.x, -c.y));
          e[1] = exp2f(fmaf(s[1], c.z, -c.w));
          e[2] = exp2f(fmaf(s[2], c.x, -c.y));
          e[3] = exp2f(fmaf(s[3], c.z, -c.w));
          if (part) {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const int j = (8 * t + 2 * qd + (x & 1)) / p.G, key = wk + r8 + 8 * (x >> 1);
              if (key >= lim_min + j || (windowed && key >= sinks && key < win.start + j)) e[x] = 0.f;
            }
          }
          w0 += e[0] + e[1];
          w1 += e[2] + e[3];
        };
        if (RT) {
#pragma unroll
          for (int t = 0; t < RT; ++t) tile(qb[t], qc[t], t);
        } else {
          for (int t = 0; t < n_tiles; ++t) {
            kw_load_rows(qb[0], qs + t * 8 * kQStride, lane);
            tile(qb[0], rc[4 * t + qd], t);
          }
        }
        w0 += __shfl_xor_sync(kFull, w0, 1);
        w0 += __shfl_xor_sync(kFull, w0, 2);
        w1 += __shfl_xor_sync(kFull, w1, 1);
        w1 += __shfl_xor_sync(kFull, w1, 2);
        const int pid = pids[stage], at = 16 * w + r8 + 8 * qd, key = key0 + at;
        if (qd < 2 && pid >= 0 && key < L && !(windowed && key >= sinks && key < win.low)) {
          float v = qd ? w1 : w0;
          if (p.acc_in && key < L - q_len)
            v += p.decay * reinterpret_cast<const float *>(smem + S::kAcc + stage * kAccBytes)[at];
          p.acc_out[(static_cast<int64_t>(pid) * p.Hkv + h) * PAGE + at] = v;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty0 + 8 * stage);
      }
      if (++stage == S::kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(qempty0 + 8 * slot);
  }
  if (!ok && lane == 0) {
    status_or(p.tm, HPA_STATUS_TIMEOUT);
    *abort_flag = 1;
  }
}

// ----------------------------------------------------------------------------- kernel
template <int KV, int RT>
__global__ void __launch_bounds__(KwCfg<KV, RT>::kThreads, RT ? 2 : 1)
    key_weights_kernel(const __grid_constant__ CUtensorMap tmk, const KeyWeightsParams p) {
  using S = KwCfg<KV, RT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int c = blockIdx.x;
  __shared__ int hdr[5];  // go, tile, s_begin, s_end, windowed
  const uint32_t base = smem_u32(smem);
  pdl_wait();  // nothing above reads what an earlier kernel writes
  if (threadIdx.x == 0) {
    const int32_t *tm = p.tm;
    const int tile = tm[TM_TILE];
    const bool windowed = tm[TM_KIND] == KIND_WINDOW;
    int go = tm[TM_STATUS] == 0;
    if (go && (tm[TM_B] != p.B || tm[TM_C] != p.C || tile <= 0 || tile % PAGE != 0 ||
               (windowed && tm[TM_QLEN] != p.q_len))) {
      if (c == 0 && blockIdx.y == 0) status_or(p.tm, HPA_STATUS_MISMATCH);
      go = 0;
    }
    if (go && !(windowed ? map_ranges_ok<true>(tm, p.lay, p.B, p.C, c)
                         : map_ranges_ok<false>(tm, p.lay, p.B, p.C, c))) {
      status_or(p.tm, HPA_STATUS_BAD_MAP);
      go = 0;
    }
    hdr[1] = tile;
    hdr[2] = go ? tm[p.lay.cta_seg + c] : 0;
    hdr[3] = go ? tm[p.lay.cta_seg + c + 1] : 0;
    hdr[0] = go && hdr[2] < hdr[3];
    hdr[4] = windowed;
    for (int st = 0; st < S::kStages; ++st) {
      mbar_init(base + S::kBars + 8 * st, 1);
      mbar_init(base + S::kBars + 8 * (S::kStages + st), kGroupWarps);
    }
    for (int sl = 0; sl < 2; ++sl) {
      mbar_init(base + S::kBars + 8 * (2 * S::kStages + sl), 32);                     // qfull
      mbar_init(base + S::kBars + 8 * (2 * S::kStages + 2 + sl), S::kConsumers);      // qempty
    }
    *reinterpret_cast<int *>(smem + S::kFlag) = 0;
    fence_barrier_init();
  }
  __syncthreads();
  pdl_launch_dependents();
  if (!hdr[0]) return;
  if (threadIdx.x >= S::kConsumers * 32)
    kw_producer<KV, RT>(p, &tmk, smem, hdr[2], hdr[3], hdr[1], hdr[4]);
  else
    kw_consumer<KV, RT>(p, smem, hdr[2], hdr[3], hdr[4]);
}

template <int KV, int RT>
cudaError_t launch(const KeyWeightsParams &p, const CUtensorMap &tmk, cudaStream_t s) {
  using S = KwCfg<KV, RT>;
  static int configured[64] = {0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !configured[dev]) {
    e = cudaFuncSetAttribute(key_weights_kernel<KV, RT>,
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
  return cudaLaunchKernelEx(&cfg, key_weights_kernel<KV, RT>, tmk, p);
}

}  // namespace

cudaError_t launch_key_weights(const KeyWeightsParams &p, const CUtensorMap &tmk, int kv_dtype,
                               cudaStream_t s) {
  if (kv_dtype == HPA_KV_BF16)
    return p.rows <= 8    ? launch<HPA_KV_BF16, 1>(p, tmk, s)
           : p.rows <= 16 ? launch<HPA_KV_BF16, 2>(p, tmk, s)
                          : launch<HPA_KV_BF16, 0>(p, tmk, s);
  return p.rows <= 8    ? launch<HPA_KV_E4M3, 1>(p, tmk, s)
         : p.rows <= 16 ? launch<HPA_KV_E4M3, 2>(p, tmk, s)
                        : launch<HPA_KV_E4M3, 0>(p, tmk, s);
}

}  // namespace hpa
