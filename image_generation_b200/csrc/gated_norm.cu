// The norms on either side of a branch's residual addition, in one pass over
// the rows: with x the fp32 residual stream and y a branch's output,
//   x' = r x + gate * (post ? RMSNorm(y) post_weight : y)
//   out = RMSNorm(x') pre_weight (1 + scale) + shift
// where RMSNorm(v) = v / sqrt(mean(v^2) + eps), x' is kept in fp32 and out is
// rounded once, to bf16, MXFP8, MXFP4 or NVFP4. gate, shift and scale have one
// row per image of a batch (rows_per_group rows share one).
//
// Bound by HBM: 4 + 2 bytes read and 4 + 2 written per element with bf16 y and
// out. One CTA owns a row, a thread V units of 8 consecutive elements: x' stays
// in registers between its sum of squares and its use, and a scale block of the
// output (16 or 32 elements) spans two or four neighbouring lanes.
#include "fp4.cuh"

namespace h3 {
namespace {

constexpr int kMaxThreads = 256;  // V units each: d <= 8 * 256 * 4

H3_DEV void load8(const float *p, float (&v)[8]) {
  const float4 a = __ldcs(reinterpret_cast<const float4 *>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4 *>(p) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
H3_DEV void load8(const uint16_t *p, float (&v)[8]) {
  const uint4 a = __ldcs(reinterpret_cast<const uint4 *>(p));
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// Eight floats of a vector that every row reads (`other` where there is none).
H3_DEV void vec8(const float *p, int at, float other, float (&v)[8]) {
  if (!p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = other;
    return;
  }
  const float4 a = __ldg(reinterpret_cast<const float4 *>(p + at));
  const float4 b = __ldg(reinterpret_cast<const float4 *>(p + at) + 1);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Sum over the block; `red` is not reused before another barrier has passed.
H3_DEV float block_sum(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < static_cast<int>(blockDim.x >> 5); ++w) t += red[w];
  return t;
}

// Eight elements of unit `u` of a row, in the output's type. Every lane of the
// warp calls it; `on` is the same for the lanes that share a scale block.
template <int OUT>
H3_DEV void store_unit(const GatedNormParams &p, const Fp4Tensor &t, int row, int u, bool on,
                       const float (&v)[8]) {
  const size_t at = static_cast<size_t>(row) * p.d + 8 * u;
  if constexpr (OUT == kNormBf16) {
    if (on)
      st_global_v4(static_cast<uint16_t *>(p.out) + at, pack_bf16x2(v[0], v[1]),
                   pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  } else if constexpr (OUT == kNormMxfp8) {
    float am = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) am = fmaxf(am, fabsf(v[i]));
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 1));
    am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, 2));
    const uint32_t sb = mx_scale_byte(am);
    const float m = mx_inv_scale(sb);
    if (!on) return;
    *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(p.out) + at) =
        make_uint2(mx_pack4(v[0] * m, v[1] * m, v[2] * m, v[3] * m),
                   mx_pack4(v[4] * m, v[5] * m, v[6] * m, v[7] * m));
    if ((u & 3) == 0) p.out_sf[mx_sf_offset(row, u >> 2, p.d / 128)] = static_cast<uint8_t>(sb);
  } else {
    constexpr int FMT = OUT == kNormFp4Mx ? kFp4Mx : kFp4Nv;
    float am = 0.f, inv;
#pragma unroll
    for (int i = 0; i < 8; ++i) am = amax_nan(am, fabsf(v[i]));
    am = amax_nan(am, __shfl_xor_sync(0xffffffffu, am, 1));
    if constexpr (FMT == kFp4Mx) am = amax_nan(am, __shfl_xor_sync(0xffffffffu, am, 2));
    const uint32_t sb = fp4_scale<FMT>(am, t, &inv);
    if (!on) return;
    *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.out) + at / 2) = fp4_pack8(v, inv);
    constexpr int PER = Fp4<FMT>::BLOCK / 8;
    if ((u & (PER - 1)) == 0) {
      const int s = u / PER, chunks = (p.d / Fp4<FMT>::BLOCK + 3) / 4;
      uint8_t *sf = p.out_sf + mx_sf_offset(row, s, chunks);
      *sf = static_cast<uint8_t>(sb);
      // a row that ends with two of its last four scales: the others are 0
      if (FMT == kFp4Mx && 8 * (u + PER) == p.d && (s & 3) == 1)
        *reinterpret_cast<uint16_t *>(sf + 1) = 0;
    }
  }
}

template <typename TB, int OUT, int V>
__global__ void __launch_bounds__(kMaxThreads)
    gated_norm_kernel(const GatedNormParams p, bool post) {
  __shared__ float red[2][kMaxThreads / 32];
  const int units = p.d / 8, step = blockDim.x;
  const float inv_d = 1.f / static_cast<float>(p.d);
  const TB *branch = static_cast<const TB *>(p.branch);
  Fp4Tensor t{};
  if constexpr (OUT == kNormFp4Nv) t = fp4_tensor(p.out_scale);
  for (int row = blockIdx.x; row < p.n; row += gridDim.x) {
    const size_t at = static_cast<size_t>(row) * p.d;
    const size_t mod = static_cast<size_t>(row / p.rows_per_group) * p.ld_mod;
    float x[V][8], y[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int u = threadIdx.x + j * step;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = y[j][i] = 0.f;
      if (u < units) {
        load8(p.x + at + 8 * u, x[j]);
        if (branch) load8(branch + at + 8 * u, y[j]);
      }
    }
    float rinv_y = 1.f;
    if (post) {
      float ss = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(y[j][i], y[j][i], ss);
      rinv_y = rsqrtf(block_sum(ss, red[0]) * inv_d + p.eps);
    }
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int u = threadIdx.x + j * step;
      if (u < units) {
        float w[8], g[8];
        if (post) {
          vec8(p.post_weight, 8 * u, 1.f, w);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[j][i] = y[j][i] * rinv_y * w[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] *= p.residual_scale;
        if (branch) {
          vec8(p.gate ? p.gate + mod : nullptr, 8 * u, 1.f, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) x[j][i] = fmaf(g[i], y[j][i], x[j][i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(x[j][i], x[j][i], ss);
        if (p.x_out) {
          float4 *o = reinterpret_cast<float4 *>(p.x_out + at + 8 * u);
          __stcs(o, make_float4(x[j][0], x[j][1], x[j][2], x[j][3]));
          __stcs(o + 1, make_float4(x[j][4], x[j][5], x[j][6], x[j][7]));
        }
      }
    }
    const float rinv = rsqrtf(block_sum(ss, red[1]) * inv_d + p.eps);
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int u = threadIdx.x + j * step;
      if (j * step >= units) break;  // the same for the whole block
      const bool on = u < units;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.f;
      if (on) {
        float w[8], sc[8], sh[8];
        vec8(p.pre_weight, 8 * u, 1.f, w);
        vec8(p.scale ? p.scale + mod : nullptr, 8 * u, 0.f, sc);
        vec8(p.shift ? p.shift + mod : nullptr, 8 * u, 0.f, sh);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = fmaf(x[j][i] * rinv * w[i], 1.f + sc[i], sh[i]);
      }
      store_unit<OUT>(p, t, row, u, on, v);
    }
    if (!post) __syncthreads();  // red[1] is read above; the next row writes it with no other barrier
  }
}

template <typename TB, int OUT, int V>
cudaError_t launch(const GatedNormParams &p, bool post, int threads, int num_sms, cudaStream_t s) {
  static PerDevice occupancy;
  int per_sm = 0;
  cudaError_t e = per_device(
      occupancy,
      [&](int *v) {
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(v, gated_norm_kernel<TB, OUT, V>,
                                                             kMaxThreads, 0);
      },
      &per_sm);
  if (e != cudaSuccess) return e;
  // full CTAs hold kMaxThreads; narrower ones fit more often
  const long long most = static_cast<long long>(num_sms) * (per_sm > 0 ? per_sm : 1) *
                         (kMaxThreads / threads);
  const int grid = static_cast<int>(p.n < most ? p.n : most);
  gated_norm_kernel<TB, OUT, V><<<grid, threads, 0, s>>>(p, post);
  return cudaGetLastError();
}

template <typename TB, int OUT>
cudaError_t launch_v(const GatedNormParams &p, bool post, int num_sms, cudaStream_t s) {
  const int units = p.d / 8;
  const int v = (units + kMaxThreads - 1) / kMaxThreads;
  const int threads = ((units + v - 1) / v + 31) / 32 * 32;
  switch (v) {
    case 1:
      return launch<TB, OUT, 1>(p, post, threads, num_sms, s);
    case 2:
      return launch<TB, OUT, 2>(p, post, threads, num_sms, s);
    case 3:
      return launch<TB, OUT, 3>(p, post, threads, num_sms, s);
    case 4:
      return launch<TB, OUT, 4>(p, post, threads, num_sms, s);
    default:
      return cudaErrorInvalidValue;
  }
}

template <typename TB>
cudaError_t launch_out(const GatedNormParams &p, bool post, int kind, int num_sms, cudaStream_t s) {
  switch (kind) {
    case kNormBf16:
      return launch_v<TB, kNormBf16>(p, post, num_sms, s);
    case kNormMxfp8:
      return launch_v<TB, kNormMxfp8>(p, post, num_sms, s);
    case kNormFp4Mx:
      return launch_v<TB, kNormFp4Mx>(p, post, num_sms, s);
    case kNormFp4Nv:
      return launch_v<TB, kNormFp4Nv>(p, post, num_sms, s);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_gated_norm(const GatedNormParams &p, bool branch_f32, bool post, int out_kind,
                              int num_sms, cudaStream_t s) {
  return branch_f32 ? launch_out<float>(p, post, out_kind, num_sms, s)
                    : launch_out<uint16_t>(p, post, out_kind, num_sms, s);
}

}  // namespace h3
