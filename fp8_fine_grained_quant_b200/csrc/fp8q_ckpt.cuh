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

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>

#include "fp8q_ptx.cuh"
#include "fp8q_quant.cuh"

namespace fp8q {

// Four E4M3 codes -> their values (exact).
__device__ __forceinline__ void e4m3x4_to_f32(uint32_t c, float (&v)[4]) {
  uint32_t h0, h1;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(h0), "=r"(h1)
      : "r"(c));
  const float2 f0 = __half22float2(*reinterpret_cast<const __half2*>(&h0));
  const float2 f1 = __half22float2(*reinterpret_cast<const __half2*>(&h1));
  v[0] = f0.x;
  v[1] = f0.y;
  v[2] = f1.x;
  v[3] = f1.y;
}

// s = fl32(amax / 448), 1 when that is 0, for any finite FP32 amax.
__device__ __forceinline__ float group_scale_f32(float amax) {
  const float s = __fdiv_rn(amax, 448.0f);
  return s == 0.0f ? 1.0f : s;
}

// E4M3 codes of fl32(x / s) for four FP32 values, by the bracket of 1/s where
// it decides (see quantize16) and by IEEE division where it does not.
__device__ __forceinline__ uint32_t quantize4_f32(const float (&x)[4], float s, float rlo, float rhi, bool exact_only) {
  uint32_t lo = cvt_e4m3x2(__fmul_rn(x[0], rlo), __fmul_rn(x[1], rlo)) |
                (cvt_e4m3x2(__fmul_rn(x[2], rlo), __fmul_rn(x[3], rlo)) << 16);
  const uint32_t hi = cvt_e4m3x2(__fmul_rn(x[0], rhi), __fmul_rn(x[1], rhi)) |
                      (cvt_e4m3x2(__fmul_rn(x[2], rhi), __fmul_rn(x[3], rhi)) << 16);
  uint32_t m = exact_only ? 0x80808080u : nonzero_bytes(lo ^ hi);
  for (; m != 0u; m &= m - 1u) {
    const int j = (__ffs(m) - 1) >> 3;
    const float v = j == 0 ? x[0] : (j == 1 ? x[1] : (j == 2 ? x[2] : x[3]));
    lo = with_exact_code(lo, j, v, s);
  }
  return lo;
}

// ---------------------------------------------------------------------------
// SwiGLU with its checkpoint: c1 [rows, 2 inter] bf16, [gate | up] ->
//   qh [rows, inter], sh      the tiles of h = bf16(silu(gate) * up), as
//                             swiglu_quant_1x128_kernel writes them;
//   qc [rows, 2 inter], sc    the tiles of c1 itself, as
//                             quant_act_1x128_kernel writes them.
// One pass over c1 instead of two.  Eight lanes own one tile of h and the gate
// and up tiles it comes from.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256, 4) swiglu_ckpt_1x128_kernel(const uint8_t* __restrict__ c1,
                                                                   uint8_t* __restrict__ qh, float* __restrict__ sh,
                                                                   uint8_t* __restrict__ qc, float* __restrict__ sc,
                                                                   int64_t inter, int64_t num_tiles) {
  const int sub = threadIdx.x & 7;
  const int64_t grp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
  const int64_t ngrp = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 3;
  const uint32_t per_row = static_cast<uint32_t>(inter >> 7);
  for (int64_t t = grp; (t & ~int64_t(3)) < num_tiles; t += ngrp) {
    const bool valid = t < num_tiles;
    const uint32_t row = valid ? static_cast<uint32_t>(t) / per_row : 0u;
    const uint32_t kb = valid ? static_cast<uint32_t>(t) - row * per_row : 0u;
    const int64_t gate = static_cast<int64_t>(row) * 2 * inter + static_cast<int64_t>(kb) * 128 + sub * 16;
    uint32_t gw[8], uw[8], hw[8];
    if (valid) {
      ld_nc_v8(c1 + gate * 2, gw);
      ld_nc_v8(c1 + (gate + inter) * 2, uw);
      swiglu16(gw, uw, hw, c1 + gate * 2, c1 + (gate + inter) * 2);
    } else {
      zero8(gw);
      zero8(uw);
      zero8(hw);
    }
    float ah = abs_max16(hw), ag = abs_max16(gw), au = abs_max16(uw);
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) {
      ah = fmaxf(ah, __shfl_xor_sync(0xFFFFFFFFu, ah, off));
      ag = fmaxf(ag, __shfl_xor_sync(0xFFFFFFFFu, ag, off));
      au = fmaxf(au, __shfl_xor_sync(0xFFFFFFFFu, au, off));
    }
    if (valid) {
      const float s_h = group_scale(ah), s_g = group_scale(ag), s_u = group_scale(au);
      *reinterpret_cast<uint4*>(qh + t * 128 + sub * 16) = quantize16(hw, s_h, recip_pair(s_h), s_h < kMinFastScale);
      *reinterpret_cast<uint4*>(qc + gate) = quantize16(gw, s_g, recip_pair(s_g), s_g < kMinFastScale);
      *reinterpret_cast<uint4*>(qc + gate + inter) = quantize16(uw, s_u, recip_pair(s_u), s_u < kMinFastScale);
      if (sub == 0) {
        sh[t] = s_h;
        const int64_t g = static_cast<int64_t>(row) * 2 * per_row + kb;
        sc[g] = s_g;
        sc[g + per_row] = s_u;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// SwiGLU backward from the checkpoint.  With g = fl32(qc sc) of the gate half,
// u of the up half and p = 1 / (1 + exp(-g)):
//   d gate = dh u p (1 + g (1 - p)),   d up = dh g p
// in FP32 (1 - p as exp(-g) p, which keeps its digits).  dc [rows, 2 inter] is
// their bf16 rounding, for the weight gradient's token-axis quantizer; q and s
// are their 1x128 tiles, the operand of the activation gradient's GEMM, taken
// from the FP32 values: s = fl32(amax / 448), codes of fl32(d / s).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void swiglu_bwd1(float g, float u, float dh, float& dg, float& du) {
  const float e = expf(-g);
  float p = div_full(1.0f, 1.0f + e);
  // 1 - p = e / (1 + e); for g below -88 e overflows and p is 0
  const float q = e > 0x1.fffffep+127f ? 1.0f : __fmul_rn(e, p);
  du = dh * (g * p);
  dg = dh * (u * (p * fmaf(g, q, 1.0f)));
}

__global__ void __launch_bounds__(256) swiglu_bwd_1x128_kernel(const uint8_t* __restrict__ dh,
                                                               const uint8_t* __restrict__ qc,
                                                               const float* __restrict__ sc, uint8_t* __restrict__ dc,
                                                               uint8_t* __restrict__ q, float* __restrict__ s,
                                                               int64_t inter, int64_t num_tiles) {
  const int sub = threadIdx.x & 7;
  const int64_t grp = (static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x) >> 3;
  const int64_t ngrp = (static_cast<int64_t>(gridDim.x) * blockDim.x) >> 3;
  const uint32_t per_row = static_cast<uint32_t>(inter >> 7);
  for (int64_t t = grp; (t & ~int64_t(3)) < num_tiles; t += ngrp) {
    const bool valid = t < num_tiles;
    const uint32_t row = valid ? static_cast<uint32_t>(t) / per_row : 0u;
    const uint32_t kb = valid ? static_cast<uint32_t>(t) - row * per_row : 0u;
    const int64_t gate = static_cast<int64_t>(row) * 2 * inter + static_cast<int64_t>(kb) * 128 + sub * 16;
    const int64_t si = static_cast<int64_t>(row) * 2 * per_row + kb;
    float dg[16], du[16];
    float ag = 0.0f, au = 0.0f;
    if (valid) {
      uint32_t dw[8];
      ld_nc_v8(dh + t * 256 + sub * 32, dw);
      const uint4 cg = ld_nc_v4(qc + gate), cu = ld_nc_v4(qc + gate + inter);
      const uint32_t gc[4] = {cg.x, cg.y, cg.z, cg.w}, uc[4] = {cu.x, cu.y, cu.z, cu.w};
      const float s_g = __ldg(sc + si), s_u = __ldg(sc + si + per_row);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float g[4], u[4];
        e4m3x4_to_f32(gc[i], g);
        e4m3x4_to_f32(uc[i], u);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t w = dw[2 * i + (j >> 1)];
          const float d = __uint_as_float((j & 1) ? (w & 0xFFFF0000u) : (w << 16));
          swiglu_bwd1(__fmul_rn(g[j], s_g), __fmul_rn(u[j], s_u), d, dg[4 * i + j], du[4 * i + j]);
          ag = fmaxf(ag, fabsf(dg[4 * i + j]));
          au = fmaxf(au, fabsf(du[4 * i + j]));
        }
      }
    }
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) {
      ag = fmaxf(ag, __shfl_xor_sync(0xFFFFFFFFu, ag, off));
      au = fmaxf(au, __shfl_xor_sync(0xFFFFFFFFu, au, off));
    }
    if (!valid) continue;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const float(&d)[16] = half ? du : dg;
      const float sv = group_scale_f32(half ? au : ag);
      float rlo, rhi;
      const bool ok = recip_bracket(sv, rlo, rhi);
      const bool exact_only = !ok || sv < kMinFastScale;
      uint32_t o[8], c[4];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = bf16x2_rn(d[2 * i], d[2 * i + 1]);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x[4] = {d[4 * i], d[4 * i + 1], d[4 * i + 2], d[4 * i + 3]};
        c[i] = quantize4_f32(x, sv, rlo, rhi, exact_only);
      }
      const int64_t at = gate + half * inter;
      *reinterpret_cast<uint4*>(dc + at * 2) = make_uint4(o[0], o[1], o[2], o[3]);
      *reinterpret_cast<uint4*>(dc + at * 2 + 16) = make_uint4(o[4], o[5], o[6], o[7]);
      *reinterpret_cast<uint4*>(q + at) = make_uint4(c[0], c[1], c[2], c[3]);
      if (sub == 0) s[si + half * per_row] = sv;
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
// A 256-thread CTA takes one 128-token x 128-channel block: thread t owns
// channels 8 (t % 16) .. +7 of tokens 8 (t / 16) .. +7.  The per-channel
// maxima are combined over the CTA, then every thread quantizes its 8 x 8
// values; the code bytes are transposed in registers and through a swizzled
// shared tile, and leave as full 128-byte rows.
// ---------------------------------------------------------------------------
__global__ void __launch_bounds__(256, 3) ckpt_128x1_t_kernel(const uint8_t* __restrict__ q,
                                                              const float* __restrict__ s, uint8_t* __restrict__ qt,
                                                              float* __restrict__ st, int64_t M, int64_t K, int64_t Mp,
                                                              int64_t num_blocks) {
  __shared__ __align__(16) uint8_t tile[128 * 128];
  __shared__ __align__(16) float col_max[8][128];
  __shared__ __align__(16) float ch_scale[128];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cg = tid & 15, rg = tid >> 4;
  const int64_t nkc = K >> 7;
  for (int64_t b = blockIdx.x; b < num_blocks; b += gridDim.x) {
    const int64_t mb = b / nkc, kc = b - mb * nkc;
    float v[8][8];  // [token][channel]
    float m[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int r = 0; r < 8; ++r) {
      const int64_t tok = mb * 128 + rg * 8 + r;
      uint2 c = make_uint2(0u, 0u);
      float sr = 1.0f;
      if (tok < M) {
        c = __ldg(reinterpret_cast<const uint2*>(q + tok * K + kc * 128 + cg * 8));
        sr = __ldg(s + tok * nkc + kc);
      }
      float x[4];
      e4m3x4_to_f32(c.x, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[r][i] = __fmul_rn(x[i], sr);
      e4m3x4_to_f32(c.y, x);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[r][4 + i] = __fmul_rn(x[i], sr);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = fmaxf(m[i], fabsf(v[r][i]));
    }
    // lanes l and l ^ 16 hold the same channels (two token groups of the warp)
#pragma unroll
    for (int i = 0; i < 8; ++i) m[i] = fmaxf(m[i], __shfl_xor_sync(0xFFFFFFFFu, m[i], 16));
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) col_max[warp][cg * 8 + i] = m[i];
    }
    __syncthreads();
    if (tid < 128) {
      float a = col_max[0][tid];
#pragma unroll
      for (int w = 1; w < 8; ++w) a = fmaxf(a, col_max[w][tid]);
      const float sv = group_scale_f32(a);
      ch_scale[tid] = sv;
      st[mb * K + kc * 128 + tid] = sv;
    }
    __syncthreads();
    uint32_t clo[8], chi[8];
#pragma unroll
    for (int r = 0; r < 8; ++r) clo[r] = chi[r] = 0u;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sv = ch_scale[cg * 8 + i];
#pragma unroll
      for (int r = 0; r < 8; ++r) {
        const uint32_t code = cvt_e4m3x2(__fdiv_rn(v[r][i], sv), 0.0f) & 0xFFu;
        if (i < 4)
          clo[r] |= code << (8 * i);
        else
          chi[r] |= code << (8 * (i - 4));
      }
    }
    transpose8x8_bytes(clo, chi);  // now channel c: tokens 0-3 in clo[c], 4-7 in chi[c]
    // channel row cg*8 + c of the tile, logical 8-byte slot rg, physical slot rg ^ cg
#pragma unroll
    for (int c = 0; c < 8; ++c)
      *reinterpret_cast<uint2*>(tile + (cg * 8 + c) * 128 + ((rg ^ cg) << 3)) = make_uint2(clo[c], chi[c]);
    __syncthreads();
    uint8_t* dst = qt + (kc * 128) * Mp + mb * 128;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int c = tid + 256 * i, row = c >> 3, ch = c & 7;
      const int swz = row >> 3;
      // logical slots 2ch, 2ch+1 sit in physical 16-byte chunk ch ^ (swz / 2),
      // their halves swapped when swz is odd
      uint4 o = *reinterpret_cast<const uint4*>(tile + row * 128 + ((ch ^ (swz >> 1)) << 4));
      if (swz & 1) o = make_uint4(o.z, o.w, o.x, o.y);
      *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(row) * Mp + ch * 16) = o;
    }
    __syncthreads();  // tile, col_max and ch_scale are reused
  }
}

}  // namespace fp8q
