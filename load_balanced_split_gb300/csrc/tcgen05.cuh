// tcgen05 (5th-generation tensor core) wrappers and operand layouts shared by the
// attention kernel (decode_attn_tc.cu) and the key-weight kernel (key_weights.cu).
#pragma once

#include "hpa_internal.cuh"

namespace hpa {
namespace {

// ---- tcgen05 wrappers ---------------------------------------------------------------
// Shared-memory matrix descriptor (sm_100 family): start, leading and stride byte
// offsets in 16-byte units, version 1, swizzle mode (2 = 128-byte, 4 = 64-byte,
// 6 = 32-byte).
__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo,
                                            uint32_t swz = 2) {
  return static_cast<uint64_t>((addr >> 4) & 0x3FFFu) |
         (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>((sbo >> 4) & 0x3FFFu) << 32) | (1ull << 46) |
         (static_cast<uint64_t>(swz) << 61);
}

// Instruction descriptor: fp32 accumulate, M = 128, N = n; A/B formats (bf16 = 1 for
// kind::f16, E4M3 = 0 for kind::f8f6f4) and major-ness (0 = K-major, 1 = MN-major).
__device__ __forceinline__ uint32_t tc_idesc(int fmt, int n, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(fmt) << 7) | (static_cast<uint32_t>(fmt) << 10) |
         (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(128 >> 4) << 24);
}

template <int KV>
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                       uint32_t acc) {
  if (KV == HPA_KV_BF16)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

// Arrive on `bar` once every MMA this thread has issued so far has completed.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
      : "memory");
}

__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

// 8 consecutive 32-bit TMEM columns of this thread's lane.
__device__ __forceinline__ void tc_ld8(uint32_t taddr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]),
                 "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}

__device__ __forceinline__ void tc_st8(uint32_t taddr, const float (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
               "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7]))
               : "memory");
}

__device__ __forceinline__ void tc_wait_ld() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Two f16 (element 0 in the low half) -> two E4M3 codes, round to nearest even,
// saturating.
__device__ __forceinline__ uint16_t f16x2_to_e4m3x2(uint32_t v) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ void sts64(uint32_t addr, uint32_t a, uint32_t b) {
  asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(addr), "r"(a), "r"(b) : "memory");
}
__device__ __forceinline__ void sts128(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                       uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}

// 2^k with a * 2^k in [128, 256) for a > 0 (1 for a == 0), k clamped to keep it an
// fp32 normal.
__device__ __forceinline__ float pow2_to_128(float a) {
  int ea = static_cast<int>((__float_as_uint(a) >> 23) & 0xffu) - 127;
  ea = min(max(ea, -119), 126);
  return a > 0.f ? __uint_as_float(static_cast<uint32_t>(127 + 7 - ea) << 23) : 1.f;
}

// Four values times sq (a power of two from pow2_to_128 of their row) as two E4M3 terms,
// one byte each: hi = e4m3(x sq), lo = e4m3(16 (x sq - hi)).  Residuals are at most half
// an E4M3 step of [128, 256), i.e. 8, so lo never saturates, and hi + lo / 16 carries a
// bf16 element to its 8 significant bits down to 2^-12 of the row's largest (without the
// 16, residuals of small elements fall under E4M3's smallest step).
__device__ __forceinline__ void e4m3_two_terms(const float (&x)[4], float sq, uint32_t &hi,
                                               uint32_t &lo) {
  float res[4];
  hi = lo = 0;
#pragma unroll
  for (int e = 0; e < 4; e += 2) {
    const float v0 = x[e] * sq, v1 = x[e + 1] * sq;
    const uint16_t h2 = f32x2_to_e4m3x2(v0, v1);
    const uint32_t hh = e4m3x2_to_f16x2(h2);
    const float2 hf = __half22float2(*reinterpret_cast<const __half2 *>(&hh));
    res[e] = v0 - hf.x;  // exact: both have at most 8 significant bits
    res[e + 1] = v1 - hf.y;
    hi |= static_cast<uint32_t>(h2) << (8 * e);
  }
#pragma unroll
  for (int e = 0; e < 4; e += 2)
    lo |= static_cast<uint32_t>(f32x2_to_e4m3x2(16.f * res[e], 16.f * res[e + 1])) << (8 * e);
}

__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// Byte offset of byte n of key k's row in an MN-major operand whose rows are one
// swizzle width sw (32, 64 or 128 bytes) long, from a 1024-byte aligned base: the
// 16-byte chunk index XOR address bits 7.. (as many bits as the row has chunks - 1).
__device__ __forceinline__ uint32_t mnmaj(int k, int n, int sw) {
  const uint32_t row = static_cast<uint32_t>(k) * sw;
  return row + ((((n >> 4) ^ (row >> 7)) & (sw / 16 - 1)) << 4) + (n & 15);
}

// Byte offset of (row r, byte kb) in a K-major operand with 128-byte swizzle:
// 8-row atoms of 8 x 128 B, 16-byte chunk index XOR (row % 8).  Rows beyond the
// first 128-byte column block live in the next block, `blk` bytes further on.
__device__ __forceinline__ uint32_t kmaj(int r, int kb, uint32_t blk) {
  return (kb >> 7) * blk + (r >> 3) * 1024 + (r & 7) * 128 + ((((kb & 127) >> 4) ^ (r & 7)) << 4) +
         (kb & 15);
}

}  // namespace
}  // namespace hpa
