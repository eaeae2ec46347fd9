// fp8q_ckpt.cuh -- activation checkpoints in 8 bits and their use in the
// backward pass.
//
// The forward pass already quantizes every GEMM input in 1x128 tiles ("The
// Insider Secrets Of Deepseek Discovered", Figure 7 (a)).  Kept until the
// backward pass in place of the bf16 activation, those codes and scales are
// what Fprop multiplied, at half the memory.  Three kernels make that usable:
// the SwiGLU between the two expert GEMMs saves its input as 1x128 tiles
// beside the tiles of its output, its backward reads the saved tiles, and the
// weight gradient, which contracts over tokens (Figure 6), gets its 128x1
// operand from saved 1x128 tiles.
#pragma once

#include <cstdint>

#include "fp8q_codes.cuh"
#include "fp8q_ptx.cuh"
#include "fp8q_quant.cuh"

namespace fp8q {

// ------------------------------------------------------------ 1 / (1 + exp(-g))
// For bf16 g in [-88, 2^126], a pair.  With log2 e = H + l, H its first 16 bits:
// exp(-g) = 2^(-g H) e^(-g l ln 2), where g H is exact (8 bits by 16) and the
// second factor is 1 - g l ln 2 to (g l ln 2)^2 / 2 <= 2^-23.3.  With ex2.approx
// (2^-22), the factor's and the sum's roundings (2^-24 each) and rcp.approx.ftz
// (2^-23): below 5.7e-7.  At -88 the result is 0 (flushed).
__device__ __forceinline__ uint64_t sigmoid_bf16x2(uint64_t g) {
  constexpr float kH = 47274.0f / 32768.0f;     // log2 e = 1.44269504089 to 16 bits
  constexpr float kLowLn2 = 4.8884952e-6f;      // (log2 e - H) ln 2
  float t0, t1, e0, e1;
  split_f32x2(mul_f32x2(g, pack_f32x2(-kH)), t0, t1);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t0));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t1));
  const uint64_t one = pack_f32x2(1.0f);
  float a, b, x, y;
  split_f32x2(fma_f32x2(join_f32x2(e0, e1), fma_f32x2(g, pack_f32x2(-kLowLn2), one), one), a, b);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(a));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(b));
  return join_f32x2(x, y);
}
// 1 / (1 + e) by rcp.approx.ftz (1 ulp).
__device__ __forceinline__ uint64_t rcp_one_plus(uint64_t e) {
  float a, b, x, y;
  split_f32x2(add_f32x2(e, pack_f32x2(1.0f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(a));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(b));
  return join_f32x2(x, y);
}

// h = bf16(silu(g) u), correctly rounded, for the 16 elements of a lane; the
// same values as swiglu16.  FP32: 5.7e-7 from p (above) and 1.2e-7 from two
// products.  Where h (1 -+ 7.75e-7), whose own roundings are 0.6e-7, give one
// bf16, that is it; elements they leave open (about one in 2500), and those outside [2^-99, 2^119], are evaluated in
// double, their words read again at gp and up.  Gates below -88 enter as -88,
// where h comes out as 0 and is evaluated in double; lanes with a gate above
// 2^126 (g_max, the lane's largest magnitude) are too.  Returns the largest |h|.
__device__ __forceinline__ float swiglu16_f32x2(const uint32_t (&gw)[8], const uint32_t (&uw)[8], uint32_t (&hw)[8],
                                                float g_max, const uint8_t* gp, const uint8_t* up) {
  uint32_t d[8];
  uint32_t any = 0u, most = 0u, least = 0x7F807F80u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t g = bf16x2_to_f32x2(max_bf16x2(gw[i], 0xC2B0C2B0u)), u = bf16x2_to_f32x2(uw[i]);  // -88
    const uint64_t h = mul_f32x2(mul_f32x2(g, sigmoid_bf16x2(g)), u);
    hw[i] = bf16x2_from_pair(mul_f32x2(h, pack_f32x2(1.0f - 0x1.ap-21f)));
    d[i] = hw[i] ^ bf16x2_from_pair(mul_f32x2(h, pack_f32x2(1.0f + 0x1.ap-21f)));
    any |= d[i];
    const uint32_t m = hw[i] & 0x7FFF7FFFu;
    most = max_bf16x2(most, m);
    least = min_bf16x2(least, m);
  }
  const uint32_t top = max(most & 0xFFFFu, most >> 16);
  const bool in_range = top <= 0x7B00u && min(least & 0xFFFFu, least >> 16) >= 0x0E00u && g_max < 0x1p+126f;
  if (any == 0u && in_range) return __uint_as_float(top << 16);
  uint32_t redo = 0u;  // bit 2i + j: half j of word i
  if (in_range) {      // the usual case: only what the bracket left open
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t x = ((d[i] & 0x7FFF7FFFu) + 0x7FFF7FFFu) | d[i];  // bits 15 and 31: halves that differ
      redo |= ((x >> 15) & 1u) << (2 * i) | (x >> 31) << (2 * i + 1);
    }
  } else {
    const bool all = !(g_max < 0x1p+126f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t m = (hw[i] >> (16 * j)) & 0x7FFFu;
        const uint32_t g = (gw[i] >> (16 * j)) & 0x7FFFu, u = (uw[i] >> (16 * j)) & 0x7FFFu;
        // a zero factor makes an exact zero, and rows that nobody wrote (not finite) are not worth the time
        const bool worth = g != 0u && u != 0u && max(g, u) < 0x7F80u;
        const bool open = all || ((d[i] >> (16 * j)) & 0xFFFFu) != 0u || m < 0x0E00u || m > 0x7B00u;
        redo |= static_cast<uint32_t>(open && worth) << (2 * i + j);
      }
    }
  }
  for (; redo != 0u; redo &= redo - 1u) {
    const int b = __ffs(redo) - 1, i = b >> 1, sh = (b & 1) * 16;
    const uint32_t g = __ldg(reinterpret_cast<const uint32_t*>(gp) + i) >> sh << 16;
    const uint32_t u = __ldg(reinterpret_cast<const uint32_t*>(up) + i) >> sh << 16;
    const uint32_t x = swiglu_bf16_exact(__uint_as_float(g), __uint_as_float(u)) << sh;
#pragma unroll
    for (int k = 0; k < 8; ++k) hw[k] = i == k ? (hw[k] & (0xFFFF0000u >> sh)) | x : hw[k];
  }
  return abs_max16(hw);
}

// ---------------------------------------------------------------------------
// SwiGLU with its checkpoint: c1 [rows, 2 inter] bf16, [gate | up] ->
//   qh [rows, inter], sh      the tiles of h = bf16(silu(gate) * up), as
//                             swiglu_quant_1x128_kernel writes them;
//   qc [rows, 2 inter], sc    the tiles of c1 itself, as
//                             quant_act_1x128_kernel writes them.
// One pass over c1 instead of two.  Eight lanes own one tile of h and the gate
// and up tiles it comes from.  Bound by instruction issue (about 600 a warp for
// 512 elements of h, a fifth of them packed FP32, which take two slots): 35072 x
// 2048 take 110 us on a B200, 4.6 TB/s, 78 us for their bytes at a copy's rate.
// (With quantize16 and swiglu16 185 us; 48 or 80 registers 117 and 112.)
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256, 4) swiglu_ckpt_1x128_kernel(const uint8_t* __restrict__ c1,
                                                                   uint8_t* __restrict__ qh, float* __restrict__ sh,
                                                                   uint8_t* __restrict__ qc, float* __restrict__ sc,
                                                                   int64_t inter, int64_t num_tiles) {
  const int sub = threadIdx.x & 7;
  const int64_t grp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
  const int64_t ngrp = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 3;
  const uint32_t per_row = static_cast<uint32_t>(inter >> 7);
  // tile t of h is tile kb of row `row`; a step moves (row, kb) by a constant, with a carry
  const uint32_t step_row = static_cast<uint32_t>(ngrp) / per_row, step_kb = static_cast<uint32_t>(ngrp) % per_row;
  uint32_t row = static_cast<uint32_t>(grp) / per_row, kb = static_cast<uint32_t>(grp) % per_row;
  for (int64_t t = grp; (t & ~int64_t(3)) < num_tiles; t += ngrp) {
    const bool valid = t < num_tiles;
    const uint64_t gate = static_cast<uint64_t>(row) * (2 * per_row) + kb, up = gate + per_row;  // tiles of c1
    uint32_t gw[8], uw[8], hw[8];
    float ah = 0.0f;
    uint32_t agu = 0u;  // largest |gate| (low half) and |up| as bf16
    if (valid) {
      const uint8_t* gp = c1 + gate * 256 + sub * 32;
      const uint8_t* upp = c1 + up * 256 + sub * 32;
      ld_nc_v8(gp, gw);
      ld_nc_v8(upp, uw);
      const float ag = abs_max16(gw), au = abs_max16(uw);
      agu = (__float_as_uint(ag) >> 16) | __float_as_uint(au);
      ah = swiglu16_f32x2(gw, uw, hw, ag, gp, upp);
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) {
      ah = fmaxf(ah, __shfl_xor_sync(0xFFFFFFFFu, ah, off));
      agu = max_bf16x2(agu, __shfl_xor_sync(0xFFFFFFFFu, agu, off));
    }
    if (valid) {
      const float s_h = group_scale(ah), s_g = group_scale(__uint_as_float(agu << 16)),
                  s_u = group_scale(__uint_as_float(agu & 0xFFFF0000u));
      *reinterpret_cast<uint4*>(qh + t * 128 + sub * 16) = codes16_bf16(hw, s_h);
      *reinterpret_cast<uint4*>(qc + gate * 128 + sub * 16) = codes16_bf16(gw, s_g);
      *reinterpret_cast<uint4*>(qc + up * 128 + sub * 16) = codes16_bf16(uw, s_u);
      if (sub == 0) {
        sh[t] = s_h;
        sc[gate] = s_g;
        sc[up] = s_u;
      }
    }
    row += step_row;
    kb += step_kb;
    if (kb >= per_row) {
      kb -= per_row;
      ++row;
    }
  }
}

// ---------------------------------------------------------------------------
// SwiGLU backward from the checkpoint.  With g = fl32(qc sc) of the gate half,
// u of the up half and p = 1 / (1 + exp(-g)):
//   d gate = dh u p (1 + g (1 - p)),   d up = dh g p
// in FP32.  dc [rows, 2 inter] is their bf16 rounding, for the weight gradient's
// token-axis quantizer; q and s are their 1x128 tiles, the operand of the
// activation gradient's GEMM, taken from the FP32 values: s = fl32(amax / 448),
// codes of fl32(d / s).  The FP32 values are good to 17 units of 2^-24 of their
// terms, not to the last bit, so about 7 codes in a million, next to an E4M3
// midpoint, come out a step from those of another FP32 evaluation.  35072 x 2048
// take 123 us on a B200 in a burst and up to 139 back to back (729 MB in three
// read and four written streams, 5.2 to 5.9 TB/s); by scalar FP32 and the bracket
// 162 us.
// ---------------------------------------------------------------------------
// Gradients of a pair: dg = dh (u (p (1 + g (1 - p)))), du = dh (g p).  With
// E = exp(-|g|) and r = 1 / (1 + E), p and 1 - p are r and E r, the other way
// round for negative gates: both keep their digits, and a p below FP32's normal
// range is not flushed (E is the square of e^(-|g|/2), which stays normal: twice
// ex2's error, E within 2^-20.9).  |g| beyond 104 makes E 0 either way.  In units
// of 2^-24, relative: E 8.6; r 7.3 at most (2 from rcp, 1 from the sum, the rest
// E's); E r 12.6; so dg 17 of |dh u| p (|g| (1 - p) + |1 + g (1 - p)|), du 15.
// (exp(-|g|) by one ex2.approx with subnormal results, E 5 and E r 9: 134.7 us
// against 122.3, and codes no nearer to the exact ones: 6.6 to 9.1 in a million off,
// against 7.4 to 9.1.)
__device__ __forceinline__ void swiglu_bwd_f32x2(uint64_t g, uint64_t u, uint64_t dh, uint64_t& dg, uint64_t& du) {
  float g0, g1;
  split_f32x2(g, g0, g1);
  const uint64_t x = join_f32x2(fminf(fabsf(g0), 104.0f), fminf(fabsf(g1), 104.0f));
  // e^(-x / 2) = 2^(-x L / 2) with L = log2 e: t = fl(x L' / 2), L' the FP32 below L by 1.925963e-8, and
  // what t lacks, x L / 2 - t = fma(x, L' / 2, -t) + x (L - L') / 2, enters squared as 1 - 2 ln 2 times it
  constexpr float kHalfL = 0.72134752f;  // L' / 2
  const uint64_t nt = mul_f32x2(x, pack_f32x2(-kHalfL));
  uint64_t lack = fma_f32x2(x, pack_f32x2(kHalfL), nt);
  lack = fma_f32x2(x, pack_f32x2(0.5f * 1.925963e-8f), lack);
  float t0, t1, e0, e1;
  split_f32x2(nt, t0, t1);
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e0) : "f"(t0));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e1) : "f"(t1));
  const uint64_t h = join_f32x2(e0, e1);
  const uint64_t E = mul_f32x2(fma_f32x2(h, mul_f32x2(lack, pack_f32x2(-2.0f * 0.693147181f)), h), h);
  const uint64_t r = rcp_one_plus(E), w = mul_f32x2(E, r);
  float r0, r1, w0, w1;
  split_f32x2(r, r0, r1);
  split_f32x2(w, w0, w1);
  const bool n0 = g0 < 0.0f, n1 = g1 < 0.0f;
  const uint64_t p = join_f32x2(n0 ? w0 : r0, n1 ? w1 : r1), q = join_f32x2(n0 ? r0 : w0, n1 ? r1 : w1);
  du = mul_f32x2(dh, mul_f32x2(g, p));
  dg = mul_f32x2(dh, mul_f32x2(u, mul_f32x2(p, fma_f32x2(g, q, pack_f32x2(1.0f)))));
}

__device__ __forceinline__ float abs_max16_f32x2(const uint64_t (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float a, b;
    split_f32x2(v[i], a, b);
    m = max3_abs(m, a, b);
  }
  return m;
}

__global__ void __launch_bounds__(256, 4) swiglu_bwd_1x128_kernel(const uint8_t* __restrict__ dh,
                                                                  const uint8_t* __restrict__ qc,
                                                                  const float* __restrict__ sc,
                                                                  uint8_t* __restrict__ dc, uint8_t* __restrict__ q,
                                                                  float* __restrict__ s, int64_t inter,
                                                                  int64_t num_tiles) {
  const int sub = threadIdx.x & 7;
  const int64_t grp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
  const int64_t ngrp = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 3;
  const uint32_t per_row = static_cast<uint32_t>(inter >> 7);
  const uint32_t step_row = static_cast<uint32_t>(ngrp) / per_row, step_kb = static_cast<uint32_t>(ngrp) % per_row;
  uint32_t row = static_cast<uint32_t>(grp) / per_row, kb = static_cast<uint32_t>(grp) % per_row;
  for (int64_t t = grp; (t & ~int64_t(3)) < num_tiles; t += ngrp) {
    const bool valid = t < num_tiles;
    const uint64_t gate = static_cast<uint64_t>(row) * (2 * per_row) + kb;  // tile of the gate half
    row += step_row;
    kb += step_kb;
    if (kb >= per_row) {
      kb -= per_row;
      ++row;
    }
    uint64_t dg[8], du[8];
    float ag = 0.0f, au = 0.0f;
    if (valid) {
      uint32_t dw[8];
      ld_nc_v8(dh + t * 256 + sub * 32, dw);
      const uint4 cg = ld_nc_v4(qc + gate * 128 + sub * 16), cu = ld_nc_v4(qc + (gate + per_row) * 128 + sub * 16);
      const uint32_t gc[4] = {cg.x, cg.y, cg.z, cg.w}, uc[4] = {cu.x, cu.y, cu.z, cu.w};
      const uint64_t s_g = pack_f32x2(__ldg(sc + gate)), s_u = pack_f32x2(__ldg(sc + gate + per_row));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint64_t g0, g1, u0, u1;
        e4m3x4_to_f32x2(gc[i], g0, g1);
        e4m3x4_to_f32x2(uc[i], u0, u1);
        swiglu_bwd_f32x2(mul_f32x2(g0, s_g), mul_f32x2(u0, s_u), bf16x2_to_f32x2(dw[2 * i]), dg[2 * i], du[2 * i]);
        swiglu_bwd_f32x2(mul_f32x2(g1, s_g), mul_f32x2(u1, s_u), bf16x2_to_f32x2(dw[2 * i + 1]), dg[2 * i + 1],
                         du[2 * i + 1]);
      }
      ag = abs_max16_f32x2(dg);
      au = abs_max16_f32x2(du);
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) {
      ag = fmaxf(ag, __shfl_xor_sync(0xFFFFFFFFu, ag, off));
      au = fmaxf(au, __shfl_xor_sync(0xFFFFFFFFu, au, off));
    }
    if (!valid) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const uint64_t(&d)[8] = half ? du : dg;
      const float sv = group_scale_f32(half ? au : ag);
      uint32_t o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = bf16x2_from_pair(d[i]);
      const uint64_t at = gate + half * per_row;
      *reinterpret_cast<uint4*>(dc + at * 256 + sub * 32) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(dc + at * 256 + sub * 32 + 16) = make_uint4(o[4], o[5], o[6], o[7]);
      *reinterpret_cast<uint4*>(q + at * 128 + sub * 16) = codes16_f32(d, sv);
      if (sub == 0) s[at] = sv;
    }
  }
}

// ---------------------------------------------------------------------------
// Weight-gradient operand from a checkpoint: q [M, K], s [M, K/128] (1x128
// tiles) -> qt [K, Mp], st [Mp/128, K] (128x1 tiles, codes token-contiguous,
// Mp >= M padded with code 0, as quant_act_128x1_t writes them).  The values
// v = fl32(code * s) are regrouped along tokens: st = fl32(amax / 448) (1 when
// 0), codes E4M3(fl32(v / st)).
//
// A 256-thread CTA takes 128 tokens x 64 channels: thread t owns channels
// 4 (t % 16) .. +3 of tokens 8 (t / 16) .. +7 and keeps their 32 values in
// registers.  The per-channel maxima are combined over the CTA, one thread per
// channel computes its scale and reciprocal, every thread quantizes its values
// (codes by the corrected quotient, a scale a column), and the code bytes are
// transposed in registers and through a swizzled shared tile, to leave as full
// 128-byte rows.  Half a block of channels a CTA keeps five CTAs on an SM and
// the last wave short.  4096 x 7168 take 18.3 us on a B200 (3.3 TB/s; 9.3 us for
// the bytes), bound by instruction issue and the five waves of 740 CTAs; with 64
// values a thread 18.8, with four CTAs an SM 19.7 and with six, which spill, 18.8.
// With an IEEE division an element 51 us.
// ---------------------------------------------------------------------------
constexpr int kCkptChannels = 64;
constexpr int kCkptThreads = 256;

__global__ void __launch_bounds__(kCkptThreads, 5) ckpt_128x1_t_kernel(const uint8_t* __restrict__ q,
                                                                       const float* __restrict__ s,
                                                                       uint8_t* __restrict__ qt,
                                                                       float* __restrict__ st, int64_t M, int64_t K,
                                                                       int64_t Mp) {
  __shared__ __align__(16) uint8_t tile[kCkptChannels * 128];
  __shared__ __align__(16) float col_max[kCkptThreads / 32][kCkptChannels];
  __shared__ __align__(16) float ch_scale[kCkptChannels];
  __shared__ __align__(16) float ch_ny[kCkptChannels];  // -1/s; NaN: the channel takes the division
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cg = tid & 15, rg = tid >> 4;
  const int64_t nkc = K / kCkptChannels;
  const int64_t mb = static_cast<uint32_t>(blockIdx.x) / static_cast<uint32_t>(nkc);
  const int64_t kc = static_cast<uint32_t>(blockIdx.x) - mb * nkc;
  const int64_t tok0 = mb * 128 + rg * 8;
  uint32_t c[8];
  float sr[8];
  const uint8_t* qp = q + tok0 * K + kc * kCkptChannels + cg * 4;
  const float* sp = s + tok0 * (K >> 7) + (kc >> 1);
  const int left = M - tok0 < 8 ? static_cast<int>(M - tok0) : 8;
#pragma unroll
  for (int r = 0; r < 8; ++r, qp += K, sp += K >> 7) {
    c[r] = 0u;
    sr[r] = 1.0f;
    if (r < left) {
      c[r] = __ldg(reinterpret_cast<const uint32_t*>(qp));
      sr[r] = __ldg(sp);
    }
  }
  uint64_t v[8][2];  // [token][channel pair]
  float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int r = 0; r < 8; r += 2) {
#pragma unroll
    for (int k = r; k < r + 2; ++k) {
      const uint64_t s2 = pack_f32x2(sr[k]);
      e4m3x4_to_f32x2(c[k], v[k][0], v[k][1]);
      v[k][0] = mul_f32x2(v[k][0], s2);
      v[k][1] = mul_f32x2(v[k][1], s2);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float a, b, x, y;
      split_f32x2(v[r][i], a, b);
      split_f32x2(v[r + 1][i], x, y);
      m[2 * i] = max3_abs(m[2 * i], a, x);
      m[2 * i + 1] = max3_abs(m[2 * i + 1], b, y);
    }
  }
  // lanes l and l ^ 16 hold the same channels (the warp's two token groups)
#pragma unroll
  for (int i = 0; i < 4; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], 16));
  if (lane < 16) *reinterpret_cast<float4*>(&col_max[warp][cg * 4]) = make_float4(m[0], m[1], m[2], m[3]);
  __syncthreads();
  if (tid < kCkptChannels) {
    float a = col_max[0][tid];
#pragma unroll
    for (int w = 1; w < kCkptThreads / 32; ++w) a = fmaxf(a, col_max[w][tid]);
    const float sv = group_scale_f32(a);
    float y;
    const bool ok = corrected_reciprocal(sv, y);
    ch_scale[tid] = sv;
    ch_ny[tid] = ok ? -y : __int_as_float(0x7FC00000);
    st[mb * K + kc * kCkptChannels + tid] = sv;
  }
  __syncthreads();
  const float4 y4 = *reinterpret_cast<const float4*>(&ch_ny[cg * 4]);
  const float4 x4 = *reinterpret_cast<const float4*>(&ch_scale[cg * 4]);
  const uint64_t ny2[2] = {join_f32x2(y4.x, y4.y), join_f32x2(y4.z, y4.w)};
  const uint64_t s2[2] = {join_f32x2(x4.x, x4.y), join_f32x2(x4.z, x4.w)};
  const bool ok = y4.x < 0.0f && y4.y < 0.0f && y4.z < 0.0f && y4.w < 0.0f;
  uint32_t code[8];  // token r's four channels
  if (ok) {
#pragma unroll
    for (int r = 0; r < 8; ++r)
      code[r] = e4m3x4_from_f32x2(neg_quotient(v[r][0], ny2[0], s2[0]), neg_quotient(v[r][1], ny2[1], s2[1])) ^
                0x80808080u;
  } else {
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      uint64_t d[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float a, b, x, y;
        split_f32x2(v[r][i], a, b);
        split_f32x2(s2[i], x, y);
        d[i] = join_f32x2(__fdiv_rn(a, x), __fdiv_rn(b, y));
      }
      code[r] = e4m3x4_from_f32x2(d[0], d[1]);
    }
  }
  // now channel i: tokens 0-3 in code[i], 4-7 in code[4 + i]
  transpose4x4_bytes(code[0], code[1], code[2], code[3]);
  transpose4x4_bytes(code[4], code[5], code[6], code[7]);
  // channel row cg*4 + i of the tile, logical 8-byte slot rg, physical slot rg ^ cg: a half
  // warp's sixteen stores fall in sixteen slots
#pragma unroll
  for (int i = 0; i < 4; ++i)
    *reinterpret_cast<uint2*>(tile + (cg * 4 + i) * 128 + ((rg ^ cg) << 3)) = make_uint2(code[i], code[4 + i]);
  __syncthreads();
  uint8_t* dst = qt + kc * kCkptChannels * Mp + mb * 128;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int row = (tid >> 3) + 32 * i, ch = tid & 7;
    const int swz = row >> 2;
    // logical slots 2ch and 2ch + 1 sit in physical 16-byte chunk ch ^ (swz / 2), their
    // halves swapped when swz is odd
    uint4 o = *reinterpret_cast<const uint4*>(tile + row * 128 + ((ch ^ (swz >> 1)) << 4));
    if (swz & 1) o = make_uint4(o.z, o.w, o.x, o.y);
    *reinterpret_cast<uint4*>(dst + row * Mp + ch * 16) = o;
  }
}

}  // namespace fp8q
