// What the attention kernels of 4-bit pages share: widening of codes, waits, segments.
#pragma once

#include "hpa_internal.cuh"

namespace hpa {
namespace {

constexpr int kUnit = E2M1_UNIT;  // bytes of one page and KV head of K or V
constexpr float kRescaleSlack = 8.f;
// Probabilities are held times 2^7: with the slack up to 2^15 in f16, whose smallest step is then
// 2^-31 of the row's largest, so that a million small ones beside it are not lost to rounding.
constexpr float kLift = 7.f;
constexpr uint32_t kFull = 0xffffffffu;

// The four bytes of w, two E2M1 codes each, as f16 pairs (low nibble in the low half; exact).
__device__ __forceinline__ void widen8(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// One half of an f16 pair in both halves (written so that a multiplication can take it in place).
template <int HI>
__device__ __forceinline__ uint32_t both_halves(uint32_t a) {
  uint32_t d;
  if (HI)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {h, h};\n\t}"
        : "=r"(d) : "r"(a));
  else
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tmov.b32 %0, {l, l};\n\t}"
        : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ void bulk_load_hint(uint32_t dst, const void *src, uint32_t bytes,
                                               uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ bool e4m3_nan(uint32_t byte) { return (byte & 0x7fu) == 0x7fu; }

struct Seg {
  int r, L, klo, khi, pg0, pg1;
};

template <bool WIN>
__device__ __forceinline__ Seg read_seg(const AttnParams &p, int s, int tile, bool report) {
  const SegRow sr = read_seg_row<WIN>(p.tm, p.lay, p.B, s, blockIdx.x, tile, report);
  return Seg{sr.r, sr.L, sr.klo, sr.khi, sr.klo / PAGE, (sr.khi + PAGE - 1) / PAGE};
}

__device__ __forceinline__ int row_base(const AttnParams &p) {
  return p.group * static_cast<int>(blockIdx.z);
}
__device__ __forceinline__ int group_rows(const AttnParams &p) {
  return min(p.group, p.rows - row_base(p));
}

// mbarrier.try_wait that may sleep for up to 20 us before it answers no.
__device__ __forceinline__ bool try_wait_long(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(20000)
      : "memory");
  return ok != 0;
}

// Wait for a phase; false if it took too long, or if another warp of the CTA gave up.
__device__ __forceinline__ bool wait_phase(uint32_t bar, uint32_t parity,
                                           const volatile int *abort_flag) {
  if (try_wait_long(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (try_wait_long(bar, parity)) return true;
    if (*abort_flag || globaltimer_ns() - t0 > 2000000000ull) return false;
  }
}

}  // namespace
}  // namespace hpa
