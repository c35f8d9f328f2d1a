// Queries and the cache from a token's projections in one pass (hpa_store_qkv): RMSNorm per head,
// position rotation, optional Walsh-Hadamard transform; queries leave as bf16, keys and values go
// to the paged cache as bf16, E4M3 or E2M1 with block scales.
//
// For a head's row x of 128 dims at position t, w the norm's weights:
//   norm:   y = x / sqrt(mean(x^2) + eps) * w      (before or after the rotation)
//   turn:   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first rot_dim dims,
//           pair i at table entry t, i
//   H:      the orthonormal Sylvester transform of order 128.
// 1 / rms is one factor per row and passes through the linear steps, so it is applied once, with
// the cache's scale, where the row is written; nothing is rounded before that.
//
// Every row is read once and written once.  Without the transform the DRAM bounds it: 32768 tokens
// of 64/8 heads, normed and rotated into a bf16 cache, take 211 us, 6.4 TB/s or 0.95 of the copy
// peak.  With it the issue slots do, two thirds of which are taken (48 shuffles and 24 additions
// of pairs for four rows, beside some 130 others): 297 us into a 4-bit cache, 4.3 TB/s.  A small
// batch is one launch (3.7 us for a token, 4.3 for 128).
//
// A warp takes items of up to 8 rows (one token, heads of q, of k or of v), four rows at a time, 8
// lanes to a row: lane k holds dims [8k, 8k + 8) and [64 + 8k, 64 + 8k + 8), so that the pairs of a
// full rotation of halves and of adjacent dims lie in one lane, and loads and stores are 16 bytes
// wide.  The next item's rows are on their way to shared memory while one is worked on.
#include "hpa_internal.cuh"

namespace hpa {
namespace {

constexpr int kWarps = 10;  // two blocks at 96 registers (8 at 108 take 311 us, 12 at 80 300)
constexpr uint32_t kFull = 0xffffffffu;
constexpr int kLanesPerHead = 8;
constexpr int kHeadsPerPass = 32 / kLanesPerHead;
constexpr int kChunkHeads = 8;
constexpr int kRowBytes = HEAD_DIM * 2;
constexpr int kCosOff = kChunkHeads * kRowBytes;       // the token's table row behind the rows
constexpr int kSlotBytes = kCosOff + HEAD_DIM * 4;
constexpr int kSlots = 2;
constexpr int kNormBytes = 2 * HEAD_DIM * 4;           // q and k weights
constexpr int kSmem = kNormBytes + kWarps * kSlots * kSlotBytes;

enum { ROPE_NONE, ROPE_HALVES, ROPE_HALVES_PART, ROPE_PAIRS };
enum { KIND_Q, KIND_K, KIND_V };

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Eight fp32 values -> four bytes of E2M1 codes, the even element in the low nibble (round to
// nearest even, saturating at +-6).
__device__ __forceinline__ uint32_t pack_e2m1(const float (&v)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
      "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// A warp's items follow one another: token by token, its chunks of q, k and v heads in turn.
struct Item {
  int tok, ch;            // token, chunk of it
  int kind, h0, nh;       // q / k / v, first head, heads
  int pos, place;         // position; slot % PAGE
  int page;               // -1: the token is skipped
  bool fresh;             // the warp's first item of its token: it brings the table row
};

struct Chunks {
  int cq, ck, n;  // chunks of q and of k (or v) heads, and of a token
};

__device__ __forceinline__ void set_chunk(const StoreQkvParams &p, const Chunks &w, Item &x) {
  x.kind = x.ch < w.cq ? KIND_Q : x.ch < w.cq + w.ck ? KIND_K : KIND_V;
  const int c = x.ch - (x.kind == KIND_Q ? 0 : x.kind == KIND_K ? w.cq : w.cq + w.ck);
  x.h0 = c * kChunkHeads;
  x.nh = min(kChunkHeads, (x.kind == KIND_Q ? p.Hq : p.Hkv) - x.h0);
}

__device__ __forceinline__ void set_token(const StoreQkvParams &p, Item &x, bool report) {
  const long long slot = p.slots[x.tok];
  x.pos = p.positions[x.tok];
  x.place = static_cast<int>(slot & (PAGE - 1));
  const bool page_ok = slot >= 0 && slot / PAGE < p.num_pages;
  const bool pos_ok = p.rot_dim == 0 || (x.pos >= 0 && x.pos < p.max_pos);
  x.page = page_ok && pos_ok ? static_cast<int>(slot / PAGE) : -1;
  x.fresh = true;
  if (report && x.ch == 0 && p.status && slot != -1 && x.page < 0)
    atomicOr(reinterpret_cast<int *>(p.status),
             page_ok ? HPA_STATUS_BAD_SEQLEN : HPA_STATUS_BAD_PAGE);
}

// Start an item's rows and, with its token's first, the table row on their way into a slot.
template <int ROPE>
__device__ __forceinline__ void fetch(const StoreQkvParams &p, const Item &x, uint32_t slot,
                                      int lane) {
  if (x.page < 0) return;
  const __nv_bfloat16 *src = (x.kind == KIND_Q   ? p.q + x.tok * p.q_stride
                              : x.kind == KIND_K ? p.k + x.tok * p.k_stride
                                                 : p.v + x.tok * p.v_stride) +
                             x.h0 * HEAD_DIM + 8 * lane;
  if (x.nh == kChunkHeads) {
#pragma unroll
    for (int u = 0; u < 4; ++u) cp_async16(slot + 16 * lane + 512 * u, src + 256 * u);
  } else {
    for (int c = lane; c < x.nh * (kRowBytes / 16); c += 32)
      cp_async16(slot + 16 * c, src + 8 * (c - lane));
  }
  if (ROPE != ROPE_NONE && x.fresh && x.kind != KIND_V && lane < p.rot_dim / 4)
    cp_async16(slot + kCosOff + 16 * lane,
               p.cos_sin + static_cast<int64_t>(x.pos) * p.rot_dim + 4 * lane);
}

__device__ __forceinline__ void lds_f32x8(uint32_t addr, f32x2 (&x)[4]) {
  uint32_t w[8];
  lds128(addr, w[0], w[1], w[2], w[3]);
  lds128(addr + 16, w[4], w[5], w[6], w[7]);
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = pk(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
}

// The table entries of a lane: what its dims' cosine and sine are, pair by pair of registers.
// ROPE_HALVES: c[j], s[j] for dims 8k + 2j, + 1 and their partners 64 further on.
// ROPE_HALVES_PART: the same for dims below rot_dim, the sine negated in the lower half.
// ROPE_PAIRS: entry i for dims 2i, 2i + 1: c[j] = (cos, cos), s[j] = (-sin, sin), j over 8 pairs.
template <int ROPE>
struct Turn {
  static constexpr int kPairs = ROPE == ROPE_PAIRS ? 8 : 4;
  f32x2 c[kPairs], s[kPairs];
};

template <int ROPE>
__device__ __forceinline__ void load_turn(Turn<ROPE> &t, uint32_t row, int k, int rot) {
  const int half = rot / 2;
  if (ROPE == ROPE_HALVES || ROPE == ROPE_HALVES_PART) {
    const int i = (8 * k) & (half - 1);  // halves are powers of two of at least 8
    f32x2 c[4], s[4];
    lds_f32x8(row + 4 * i, c);
    lds_f32x8(row + 4 * (half + i), s);
    const float sg = ROPE == ROPE_HALVES_PART && 8 * k < half ? -1.f : 1.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) t.c[j] = c[j], t.s[j] = mul2(s[j], pk(sg, sg));
  }
  if (ROPE == ROPE_PAIRS) {
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int i = 32 * hf + 4 * k;  // entries of dims 64 hf + 8 k ..
      float c[4] = {1.f, 1.f, 1.f, 1.f}, s[4] = {0.f, 0.f, 0.f, 0.f};
      if (i < half) {
        uint32_t w[4];
        lds128(row + 4 * i, w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = __uint_as_float(w[j]);
        lds128(row + 4 * (half + i), w[0], w[1], w[2], w[3]);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = __uint_as_float(w[j]);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        t.c[4 * hf + j] = pk(c[j], c[j]);
        t.s[4 * hf + j] = pk(-s[j], s[j]);
      }
    }
  }
}

// y[j]: dims 8k + 2j, + 1 (j < 4) and 64 + 8k + 2(j - 4), + 1.
template <int ROPE>
__device__ __forceinline__ void turn(f32x2 (&y)[8], const Turn<ROPE> &t, int k, int rot) {
  if (ROPE == ROPE_HALVES) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x2 lo = y[j], hi = y[4 + j], ns = mul2(t.s[j], pk(-1.f, -1.f));
      y[j] = fma2(hi, ns, mul2(lo, t.c[j]));
      y[4 + j] = fma2(lo, t.s[j], mul2(hi, t.c[j]));
    }
  } else if (ROPE == ROPE_HALVES_PART) {  // the partner dim lies rot / 16 lanes away
    const int m = rot / 16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float a, b;
      upk(y[j], a, b);
      const f32x2 other = pk(__shfl_xor_sync(kFull, a, m), __shfl_xor_sync(kFull, b, m));
      const f32x2 z = fma2(other, t.s[j], mul2(y[j], t.c[j]));
      if (8 * k < rot) y[j] = z;
    }
  } else if (ROPE == ROPE_PAIRS) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a, b;
      upk(y[j], a, b);
      y[j] = fma2(pk(b, a), t.s[j], mul2(y[j], t.c[j]));
    }
  }
}

__device__ __forceinline__ float row_sum_squares(const f32x2 (&y)[8]) {
  f32x2 s2 = mul2(y[0], y[0]);
#pragma unroll
  for (int j = 1; j < 8; ++j) s2 = fma2(y[j], y[j], s2);
  float a, b;
  upk(s2, a, b);
  float ss = a + b;
  ss += __shfl_xor_sync(kFull, ss, 1);
  ss += __shfl_xor_sync(kFull, ss, 2);
  ss += __shfl_xor_sync(kFull, ss, 4);
  return ss;
}

// Sylvester butterflies over the 128 dims (unscaled): dim bits 0 in a pair, 1, 2 and 6 between
// registers, 3 to 5 between lanes.
__device__ __forceinline__ void hadamard128(f32x2 (&y)[8], int lane) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float a, b;
    upk(y[j], a, b);
    y[j] = pk(a + b, a - b);
  }
#pragma unroll
  for (int st = 1; st < 8; st <<= 1)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!(j & st)) {
        const f32x2 a = y[j], b = y[j | st];
        y[j] = add2(a, b);
        y[j | st] = sub2(a, b);
      }
#pragma unroll
  for (int m = 1; m < kLanesPerHead; m <<= 1) {
    const float sgn = (lane & m) ? -1.f : 1.f;  // partner + sign * own
    const f32x2 sg2 = pk(sgn, sgn);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float a, b;
      upk(y[j], a, b);
      y[j] = fma2(sg2, y[j], pk(__shfl_xor_sync(kFull, a, m), __shfl_xor_sync(kFull, b, m)));
    }
  }
}

__device__ __forceinline__ void store_bf16(__nv_bfloat16 *row, int k, const float (&v)[16]) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
  reinterpret_cast<uint4 *>(row + 8 * k)[0] = make_uint4(w[0], w[1], w[2], w[3]);
  reinterpret_cast<uint4 *>(row + 64 + 8 * k)[0] = make_uint4(w[4], w[5], w[6], w[7]);
}

// One cache row, 16 dims in this lane, in units of the head's scale.  All lanes of the warp
// call it (E2M1 exchanges maxima); those without a row pass active = false.
__device__ __forceinline__ void store_row(void *pool, int kv_dtype, int64_t unit, int place, int k,
                                          const float (&v)[16], bool active) {
  if (kv_dtype == HPA_KV_BF16) {
    if (active)
      store_bf16(static_cast<__nv_bfloat16 *>(pool) + (unit * PAGE + place) * HEAD_DIM, k, v);
  } else if (kv_dtype == HPA_KV_E4M3) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = f32x2_to_e4m3x2(v[4 * i], v[4 * i + 1]);
      const uint32_t hi = f32x2_to_e4m3x2(v[4 * i + 2], v[4 * i + 3]);
      q[i] = lo | (hi << 16);
    }
    uint8_t *row = static_cast<uint8_t *>(pool) + (unit * PAGE + place) * HEAD_DIM;
    if (active) {
      reinterpret_cast<uint2 *>(row + 8 * k)[0] = make_uint2(q[0], q[1]);
      reinterpret_cast<uint2 *>(row + 64 + 8 * k)[0] = make_uint2(q[2], q[3]);
    }
  } else {
    // a block of 16 dims is two neighbouring lanes' eights: scale = E4M3 of its largest / 6,
    // codes = E2M1 of the quotients.  A quotient on the border of two codes is common (bf16
    // inputs, scales of 4 bits) and has to fall to the even one, which v * (1 / s) alone may miss
    // by its last bit: its exact remainder, times 1 / s, puts that right (Markstein, IBM J. Res.
    // Dev. 34, 1990; a division each takes 30 us more, 32768 tokens of 64/8 heads).  The remainder
    // is taken negative, so that a quotient of zero keeps its sign.
    uint8_t *base = static_cast<uint8_t *>(pool) + unit * E2M1_UNIT;
    uint32_t codes[2], sb[2];
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      float am = fabsf(v[8 * hf]);
#pragma unroll
      for (int i = 1; i < 8; ++i) am = max_nan(am, fabsf(v[8 * hf + i]));
      am = max_nan(am, __shfl_xor_sync(kFull, am, 1));
      sb[hf] = f32x2_to_e4m3x2(__fdiv_rn(am, 6.f), 0.f) & 0xffu;
      const uint32_t h2 = e4m3x2_to_f16x2(static_cast<uint16_t>(sb[hf]));
      const float s = __half2float(__ushort_as_half(static_cast<unsigned short>(h2 & 0xffffu)));
      const float r = s == 0.f ? 0.f : __frcp_rn(s);
      float z[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = v[8 * hf + i] * r;
        z[i] = fmaf(fmaf(q, s, -v[8 * hf + i]), -r, q);
      }
      if (am > 3e38f) {  // an infinity has no remainder
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = v[8 * hf + i] * r;
      }
      codes[hf] = s == 0.f ? 0u : pack_e2m1(z);
      // the row's four scales of this half, gathered into a word
      sb[hf] = (k & 1) ? 0u : sb[hf] << (4 * k);
      sb[hf] |= __shfl_xor_sync(kFull, sb[hf], 2);
      sb[hf] |= __shfl_xor_sync(kFull, sb[hf], 4);
    }
    if (active) {
      uint32_t *row = reinterpret_cast<uint32_t *>(base + place * (HEAD_DIM / 2));
      row[k] = codes[0];
      row[8 + k] = codes[1];
      if (k == 0)
        *reinterpret_cast<uint2 *>(base + PAGE * HEAD_DIM / 2 + place * (HEAD_DIM / E2M1_BLOCK)) =
            make_uint2(sb[0], sb[1]);
    }
  }
}

// One item, with the table entries that a lane keeps from one to the next of a token.  Norm weights
// are read again for every four rows: kept too, their 16 registers cost two warps a block.
template <int ROPE>
__device__ __forceinline__ void work(const StoreQkvParams &p, const Item &x, Turn<ROPE> &t,
                                     uint32_t slot, uint32_t norms, int lane) {
  const int k = lane % kLanesPerHead, hp = lane / kLanesPerHead;
  const bool key_like = x.kind != KIND_V;
  const bool has_norm = x.kind == KIND_Q ? p.q_norm != nullptr : p.k_norm != nullptr;
  if (key_like && x.fresh) load_turn<ROPE>(t, slot + kCosOff, k, p.rot_dim);
  const uint32_t wat = norms + (x.kind == KIND_K) * (HEAD_DIM * 4) + 32 * k;
#pragma unroll 1
  for (int ps = 0; ps * kHeadsPerPass < x.nh; ++ps) {
    const int hh = ps * kHeadsPerPass + hp, h = x.h0 + hh;
    const bool active = hh < x.nh;  // lanes without a head still take the shuffles
    f32x2 y[8];
    {
      uint32_t r[8] = {0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u};
      if (active) {
        const uint32_t a = slot + hh * kRowBytes + 16 * k;
        lds128(a, r[0], r[1], r[2], r[3]);
        lds128(a + 128, r[4], r[5], r[6], r[7]);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
        y[i] = pk(__uint_as_float(r[i] << 16), __uint_as_float(r[i] & 0xffff0000u));
    }
    float f = 1.f;
    if (key_like) {
      if (has_norm && !p.norm_after) {
        f = rsqrtf(row_sum_squares(y) / HEAD_DIM + p.eps);
        f32x2 w[8];
        lds_f32x8(wat, reinterpret_cast<f32x2(&)[4]>(w[0]));
        lds_f32x8(wat + 256, reinterpret_cast<f32x2(&)[4]>(w[4]));
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = mul2(y[j], w[j]);
      }
      turn<ROPE>(y, t, k, p.rot_dim);
      if (has_norm && p.norm_after) {
        f = rsqrtf(row_sum_squares(y) / HEAD_DIM + p.eps);
        f32x2 w[8];
        lds_f32x8(wat, reinterpret_cast<f32x2(&)[4]>(w[0]));
        lds_f32x8(wat + 256, reinterpret_cast<f32x2(&)[4]>(w[4]));
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = mul2(y[j], w[j]);
      }
      if (p.use_hadamard) {
        hadamard128(y, lane);
        f *= 0.08838834764831845f;  // 1 / sqrt(128)
      }
    }
    if (x.kind != KIND_Q && p.kv_dtype != HPA_KV_BF16 && active)
      f *= __frcp_rn(x.kind == KIND_K ? p.k_scale[h] : p.v_scale[h]);
    float v[16];
    const f32x2 f2 = pk(f, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) upk(mul2(y[i], f2), v[2 * i], v[2 * i + 1]);
    if (x.kind == KIND_Q) {
      if (active) store_bf16(p.q_out + x.tok * p.q_out_stride + h * HEAD_DIM, k, v);
    } else {
      store_row(x.kind == KIND_K ? p.k_pool : p.v_pool, p.kv_dtype,
                static_cast<int64_t>(x.page) * p.Hkv + h, x.place, k, v, active);
    }
  }
}

template <int ROPE>
__global__ void __launch_bounds__(kWarps * 32, 2) store_qkv_kernel(const StoreQkvParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  pdl_wait();
  if (threadIdx.x < HEAD_DIM) {
    float *n = reinterpret_cast<float *>(smem);
    if (p.q_norm) n[threadIdx.x] = p.q_norm[threadIdx.x];
    if (p.k_norm) n[HEAD_DIM + threadIdx.x] = p.k_norm[threadIdx.x];
  }
  __syncthreads();
  const uint32_t norms = smem_u32(smem);
  const uint32_t slots = norms + kNormBytes + warp * kSlots * kSlotBytes;
  Chunks w;
  w.cq = p.q ? (p.Hq + kChunkHeads - 1) / kChunkHeads : 0;
  w.ck = p.k ? (p.Hkv + kChunkHeads - 1) / kChunkHeads : 0;
  w.n = w.cq + 2 * w.ck;
  // equal shares of the items, each a run of its own: a token's table row, place and weights are
  // then read once for its (usually ten) items
  const int64_t n_items = static_cast<int64_t>(p.num_tokens) * w.n;
  const int64_t n_warps = static_cast<int64_t>(gridDim.x) * kWarps;
  const int64_t mine = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
  const int64_t begin = n_items * mine / n_warps;
  const int count = static_cast<int>(n_items * (mine + 1) / n_warps - begin);
  if (count <= 0) return;
  Item cur;
  cur.tok = static_cast<int>(begin / w.n);
  cur.ch = static_cast<int>(begin % w.n);
  set_chunk(p, w, cur);
  set_token(p, cur, lane == 0);
  fetch<ROPE>(p, cur, slots, lane);
  cp_async_commit();
  Turn<ROPE> kept;
  for (int i = 0, buf = 0; i < count; ++i, buf ^= 1) {
    Item nxt = cur;
    if (i + 1 < count) {
      nxt.fresh = false;
      if (++nxt.ch == w.n) {
        nxt.ch = 0;
        ++nxt.tok;
        set_token(p, nxt, lane == 0);
      }
      set_chunk(p, w, nxt);
      fetch<ROPE>(p, nxt, slots + (buf ^ 1) * kSlotBytes, lane);
    }
    cp_async_commit();
    cp_async_wait<1>();  // this item's group has landed (the next one may still fly)
    __syncwarp();
    if (cur.page >= 0) work<ROPE>(p, cur, kept, slots + buf * kSlotBytes, norms, lane);
    __syncwarp();  // every lane is done with this slot before it is refilled
    cur = nxt;
  }
  cp_async_wait<0>();
}

template <int ROPE>
cudaError_t launch(const StoreQkvParams &p, cudaStream_t s) {
  static int wave[64] = {0};  // blocks that fill the device once
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  int blocks = dev < 64 ? wave[dev] : 0;
  if (blocks == 0) {
    int sms = 0, per_sm = 0;
    e = cudaFuncSetAttribute(store_qkv_kernel<ROPE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kSmem);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, store_qkv_kernel<ROPE>,
                                                        kWarps * 32, kSmem);
    if (e != cudaSuccess) return e;
    blocks = sms * (per_sm > 0 ? per_sm : 1);
    if (dev < 64) wave[dev] = blocks;
  }
  const int chunks = (p.q ? (p.Hq + kChunkHeads - 1) / kChunkHeads : 0) +
                     (p.k ? 2 * ((p.Hkv + kChunkHeads - 1) / kChunkHeads) : 0);
  const int64_t want = (static_cast<int64_t>(p.num_tokens) * chunks + kWarps - 1) / kWarps;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(want < blocks ? want : blocks));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  return cudaLaunchKernelEx(&cfg, store_qkv_kernel<ROPE>, p);
}

}  // namespace

cudaError_t launch_store_qkv(const StoreQkvParams &p, cudaStream_t s) {
  if (p.rot_dim == 0) return launch<ROPE_NONE>(p, s);
  if (p.interleaved) return launch<ROPE_PAIRS>(p, s);
  return p.rot_dim == HEAD_DIM ? launch<ROPE_HALVES>(p, s) : launch<ROPE_HALVES_PART>(p, s);
}

}  // namespace hpa
