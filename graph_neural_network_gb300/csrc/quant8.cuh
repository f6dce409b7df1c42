// Rounding to 8 bits that the exact quotient decides, shared by the checkpoints and the
// 8-bit norms.
#pragma once

#include "device.cuh"

namespace gnn {

constexpr float kWhole = 12582912.f;  // 1.5 * 2^23: adding it rounds to a whole number

// max(top / kTop, 2^-126).  The quotient is correctly rounded (Markstein 1990,
// "Computation of elementary functions on the IBM RISC System/6000": with c the
// rounded reciprocal and q within one step, q + (a - b q) c rounds to a / b);
// quotients below 2^-126, where the residue is not exact, give way to the bound.
template <int kTop>
__device__ __forceinline__ float scale_of(float top) {
  constexpr float c = float(1.0 / kTop);
  const float q = __fmul_rn(top, c);
  return fmaxf(__fmaf_rn(__fmaf_rn(-float(kTop), q, top), c, q), 1.17549435e-38f);
}

__device__ __forceinline__ float reciprocal(float s) {
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(s));
  return inv;
}

// ---- int8 ---------------------------------------------------------------------

// Candidates t[k] (whole numbers plus kWhole) for the quotients x / s, and the
// largest residue.
template <int V>
__device__ __forceinline__ float candidates(const float (&x)[V], float s, float inv,
                                            float (&t)[V], float (&r)[V]) {
  float most = 0.f;
#pragma unroll
  for (int c = 0; c < V; c += 2) {
    t[c] = t[c + 1] = kWhole;
    fma2(t[c], t[c + 1], x[c], x[c + 1], inv, inv);
    float q0, q1;
    add2(q0, q1, t[c], t[c + 1], -kWhole, -kWhole);
    r[c] = x[c];
    r[c + 1] = x[c + 1];
    fma2(r[c], r[c + 1], q0, q1, -s, -s);
    most = fmaxf(most, fmaxf(fabsf(r[c]), fabsf(r[c + 1])));
  }
  return most;
}

// Corrects the candidates whose residue is half a scale or more.
template <int V>
__device__ __forceinline__ void settle(float half, float (&t)[V], const float (&r)[V]) {
#pragma unroll
  for (int c = 0; c < V; ++c) {
    const float a = fabsf(r[c]);
    if (a > half || (a == half && (__float_as_uint(t[c]) & 1))) t[c] += r[c] > 0.f ? 1.f : -1.f;
  }
}

// The low byte of whole + kWhole is the whole number's: four of them.
__device__ __forceinline__ uint32_t low_bytes(const float* t) {
  const uint32_t a = __byte_perm(__float_as_uint(t[0]), __float_as_uint(t[1]), 0x0040);
  const uint32_t b = __byte_perm(__float_as_uint(t[2]), __float_as_uint(t[3]), 0x0040);
  return __byte_perm(a, b, 0x5410);
}

// ---- e4m3 ---------------------------------------------------------------------
//
// The float32 quotient r = x inv is within three units of its last place of x / s.  Its
// rounding to three bits behind the leading one, by the hardware's conversion, is
// that of x / s unless r lies next to a border, whose 20 dropped bits are a one and
// zeros.  Below 2^-6 the steps are 2^-9 throughout; r + 2^-6 has its borders at the
// same bits.  An r within eight units of a border (one in 60,000) takes the branch
// that compares x with border * s, exact in 64 bits, and steps off the border
// towards x / s (an exact tie stays on it: the conversion rounds it to even).

constexpr float kSmallest = 0.015625f;  // 2^-6, the least normal e4m3

__device__ __forceinline__ bool near_border(float r) {
  const float a = fabsf(r);
  const uint32_t low = __float_as_uint(a < kSmallest ? a + kSmallest : a) & 0xfffffu;
  return low - (0x80000u - 8u) <= 16u;
}

static __device__ __noinline__ float off_border(float r, float x, float s) {
  const float a = fabsf(r);
  const bool small = a < kSmallest;
  const uint32_t bits = __float_as_uint(small ? a + kSmallest : a);
  const float border = __uint_as_float((bits & ~0xfffffu) | 0x80000u) - (small ? kSmallest : 0.f);
  const double want = fabs(double(x)), at = double(border) * double(s);
  const uint32_t b = __float_as_uint(border);
  const float to = want > at   ? __uint_as_float(b + 1)
                   : want < at ? __uint_as_float(b - 1)
                               : border;
  return copysignf(to, r);
}

// Two floats as two e4m3 bytes, `lo` in the low one.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t v;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(v) : "f"(hi), "f"(lo));
  return v;
}

// The two e4m3 bytes of v (16 bits) as floats, exactly.
__device__ __forceinline__ void widen_e4m3(uint32_t v, float& lo, float& hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(uint16_t(v)));
  asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.f32.f16 %0, a;\n cvt.f32.f16 %1, b;\n}"
      : "=f"(lo), "=f"(hi)
      : "r"(h));
}

}  // namespace gnn
