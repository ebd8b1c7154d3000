// 4-bit floating point shared by the FP4 kernels: E2M1 elements, two per byte
// (the element of the even column in the low half), with
//   MXFP4  one E8M0 scale 2^X per 32 elements along the row,
//          X = floor(log2 amax) - 2 (6 = 1.5 * 2^2 is the largest element);
//   NVFP4  one E4M3 scale s per 16 elements and one fp32 tensor scale g:
//          s = E4M3(fl(amax * fl(1 / fl(6 g)))), element E2M1(fl(x * fl(1 / fl(s g)))).
// The NVFP4 steps are single-precision operations rounded one by one (never
// fused), so that a value next to a rounding border is the same wherever the
// matrix is made. A block that holds a NaN or an infinity gets the scale's NaN
// code. Scales lie in the layout of mx_sf_offset.
#pragma once

#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "kernels.h"
#include "ptx.cuh"

namespace h3 {

template <int FMT>
struct Fp4 {
  static constexpr int BLOCK = FMT == kFp4Mx ? 32 : 16;  // elements per scale
  static constexpr uint32_t NAN_SCALE = FMT == kFp4Mx ? 0xffu : 0x7fu;
};

// What the NVFP4 scales of one tensor are computed with (unused by MXFP4).
struct Fp4Tensor {
  float g, r6;  // tensor scale, fl(1 / fl(6 g))
  bool ok;      // g is positive and finite
};
H3_DEV Fp4Tensor fp4_tensor(const float *g_ptr) {
  Fp4Tensor t;
  t.g = g_ptr ? __ldg(g_ptr) : 1.f;
  t.ok = t.g > 0.f && t.g < INFINITY;
  t.r6 = __frcp_rn(__fmul_rn(6.f, t.g));
  return t;
}

H3_DEV float e4m3_to_float(uint32_t b) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
  return __half2float(__half(h));
}

// Scale byte of a block whose largest magnitude is amax (NaN or infinite if
// the block holds such a value), and in *inv what its elements are multiplied by.
template <int FMT>
H3_DEV uint32_t fp4_scale(float amax, const Fp4Tensor &t, float *inv) {
  if constexpr (FMT == kFp4Mx) {
    const int eb = static_cast<int>(__float_as_uint(amax) >> 23);
    if (eb >= 255) {
      *inv = 0.f;
      return Fp4<FMT>::NAN_SCALE;
    }
    const uint32_t sb = eb > 2 ? static_cast<uint32_t>(eb - 2) : 0u;  // X + 127
    *inv = __uint_as_float((254u - sb) << 23);                        // 2^-X
    return sb;
  } else {
    if (!(amax < INFINITY) || !t.ok) {
      *inv = 0.f;
      return Fp4<FMT>::NAN_SCALE;
    }
    // amax 0 is kept from 0 * infinity where 6 g is below the normal range
    const float want = amax > 0.f ? __fmul_rn(amax, t.r6) : 0.f;
    const uint32_t sb = __nv_cvt_float_to_fp8(want, __NV_SATFINITE, __NV_E4M3);
    const float d = __fmul_rn(e4m3_to_float(sb), t.g);
    *inv = d >= 1.17549435e-38f ? __frcp_rn(d) : 0.f;  // a scale of 0, or below 2^-126: the block is zero
    return sb;
  }
}

// Four consecutive elements, already multiplied by the inverse scale, as 16 bits.
H3_DEV uint32_t fp4_pack4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest);
  const uint32_t hi = __nv_cvt_float2_to_fp4x2(make_float2(c, d), __NV_E2M1, cudaRoundNearest);
  return lo | (hi << 8);
}
H3_DEV uint32_t fp4_pack8(const float *v, float inv) {
  return fp4_pack4(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv), __fmul_rn(v[2], inv),
                   __fmul_rn(v[3], inv)) |
         (fp4_pack4(__fmul_rn(v[4], inv), __fmul_rn(v[5], inv), __fmul_rn(v[6], inv),
                    __fmul_rn(v[7], inv))
          << 16);
}

// The larger magnitude; NaN if either is NaN (fmaxf would drop it).
H3_DEV float amax_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 32 consecutive values of a row: packed elements and the scale byte(s) of
// their one (MXFP4) or two (NVFP4) blocks.
template <int FMT>
H3_DEV void fp4_quant32(const float (&v)[32], const Fp4Tensor &t, uint32_t (&q)[4],
                        uint32_t (&sb)[2]) {
  constexpr int B = Fp4<FMT>::BLOCK;
#pragma unroll
  for (int b = 0; b < 32 / B; ++b) {
    float amax = 0.f, inv;
#pragma unroll
    for (int i = 0; i < B; ++i) amax = amax_nan(amax, fabsf(v[B * b + i]));
    sb[b] = fp4_scale<FMT>(amax, t, &inv);
#pragma unroll
    for (int i = 0; i < B / 8; ++i) q[B / 8 * b + i] = fp4_pack8(v + B * b + 8 * i, inv);
  }
}

// What a scale byte stands for.
template <int FMT>
H3_DEV float fp4_scale_value(uint32_t sb) {
  if constexpr (FMT == kFp4Mx)
    return sb == 0 ? __uint_as_float(0x00400000u) : __uint_as_float(sb == 255u ? 0x7fc00000u : sb << 23);
  else
    return e4m3_to_float(sb);
}

}  // namespace h3
