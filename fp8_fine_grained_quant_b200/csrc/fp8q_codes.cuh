// fp8q_codes.cuh -- E4M3 codes and scales of groups of bf16 or FP32 values by a
// corrected FP32 quotient: the arithmetic that the dispatch and checkpoint
// kernels share.  The same codes as the IEEE quotient gives, bit for bit.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "fp8q_ptx.cuh"
#include "fp8q_quant.cuh"

namespace fp8q {

// ------------------------------------------------------------ packed FP32
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t join_f32x2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void split_f32x2(uint64_t p, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(p));
}
// max(|a|, |b|, |c|) in one instruction.
__device__ __forceinline__ float max3_abs(float a, float b, float c) {
  float r;
  asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Four E4M3 codes -> their values (exact), two packed pairs.
__device__ __forceinline__ void e4m3x4_to_f32x2(uint32_t c, uint64_t& p0, uint64_t& p1) {
  uint32_t h0, h1;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(h0), "=r"(h1)
      : "r"(c));
  const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  p0 = join_f32x2(f0.x, f0.y);
  p1 = join_f32x2(f1.x, f1.y);
}

// ------------------------------------------------------------ codes by a corrected quotient
// The code of fl32(x / s) without a division, a bracket or a branch: with
// y = RN(1/s), q0 = x y, q1 = q0 + (x - q0 s) y, the remainder step of P. W.
// Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", IBM J. Res. Dev. 34 (1990).  What follows is only that the code is
// right, which needs less than the quotient's own last bit.  Away from the E4M3 midpoints
// q1 and fl32(x / s) are on the same side of each.  They could part only where
// x / s is next to an FP32 rounding midpoint beside an E4M3 midpoint; there q0
// is one of the two floats around it (x y is off by less than an ulp), x - q0 s
// is exact, and what is left of y's error is below 2^-25 ulp, while x / s, a
// quotient of two 24-bit numbers, is at least 2^-24 ulp away.  The same holds
// for bf16 and for FP32 values x.  Needs y within half an ulp of 1/s, checked
// exactly (1 - s y is a float), and s far from the ends of the range, so that no
// remainder underflows where a code is decided; else the IEEE division.
//
// y is kept negated: with -q0 and -q1 a zero keeps its sign, and one XOR turns
// four codes' signs back.  Three packed FP32 operations and one conversion a
// pair of elements, against two products, two conversions and a comparison for
// the bracket, and no element is ever redone.
struct DivScale {
  uint64_t ny2, s2;  // {-y, -y} and {s, s}
  bool ok;
};
__device__ __forceinline__ bool corrected_reciprocal(float s, float& y) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  y = __fmaf_rn(r, __fmaf_rn(-s, r, 1.0f), r);
  const float half_ulp = __uint_as_float(__float_as_uint(y) & 0x7F800000u) * 0x1p-24f;
  return fabsf(__fmaf_rn(-s, y, 1.0f)) <= s * half_ulp && s >= 0x1p-80f && s <= 0x1p+120f;
}
__device__ __forceinline__ DivScale div_scale(float s) {
  float y;
  const bool ok = corrected_reciprocal(s, y);
  return {pack_f32x2(-y), pack_f32x2(s), ok};
}
// -(x / s), corrected, for a pair.
__device__ __forceinline__ uint64_t neg_quotient(uint64_t x, uint64_t ny2, uint64_t s2) {
  const uint64_t q0 = mul_f32x2(x, ny2);
  return fma_f32x2(fma_f32x2(q0, s2, x), ny2, q0);
}
__device__ __forceinline__ uint32_t codes4(uint64_t x0, uint64_t x1, const DivScale& d) {
  return e4m3x4_from_f32x2(neg_quotient(x0, d.ny2, d.s2), neg_quotient(x1, d.ny2, d.s2)) ^ 0x80808080u;
}
// Codes of fl32(x / s) for four FP32 values by IEEE division.
__device__ __noinline__ uint32_t codes4_exact(uint64_t x0, uint64_t x1, float s) {
  float a, b, c, d;
  split_f32x2(x0, a, b);
  split_f32x2(x1, c, d);
  return cvt_e4m3x2(__fdiv_rn(a, s), __fdiv_rn(b, s)) | (cvt_e4m3x2(__fdiv_rn(c, s), __fdiv_rn(d, s)) << 16);
}
// 16 bf16 (eight words) -> 16 codes, low byte first.
__device__ __forceinline__ uint4 codes16_bf16(const uint32_t (&w)[8], float s) {
  const DivScale d = div_scale(s);
  if (!d.ok) return quantize16_exact(w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7], s);
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = codes4(bf16x2_to_f32x2(w[2 * i]), bf16x2_to_f32x2(w[2 * i + 1]), d);
  return make_uint4(c[0], c[1], c[2], c[3]);
}
// 16 FP32 values (eight pairs) -> 16 codes.
__device__ __forceinline__ uint4 codes16_f32(const uint64_t (&v)[8], float s) {
  const DivScale d = div_scale(s);
  uint32_t c[4];
  if (d.ok) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = codes4(v[2 * i], v[2 * i + 1], d);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = codes4_exact(v[2 * i], v[2 * i + 1], s);
  }
  return make_uint4(c[0], c[1], c[2], c[3]);
}

// s = fl32(amax / 448), 1 when that is 0, for any finite FP32 amax.
__device__ __forceinline__ float group_scale_f32(float amax) {
  const float s = __fdiv_rn(amax, 448.0f);
  return s == 0.0f ? 1.0f : s;
}

}  // namespace fp8q
