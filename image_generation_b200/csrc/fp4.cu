// FP4 matrices from and to wider types (next to mx_quantize): the tensor scale
// of an NVFP4 matrix, quantisation, and the values that a quantised matrix
// stands for.
//
// All three are bound by HBM: 2 bytes read per bf16 element and 1/2 byte plus
// 1/32 or 1/16 written (the tensor scale only reads). One lane owns 16
// consecutive elements, so an NVFP4 block needs no exchange between lanes and
// an MXFP4 block one shuffle; four lanes (64 elements, what rows are a multiple
// of) join their scale bytes into one store.
#include "fp4.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;

// 16 consecutive elements as fp32.
H3_DEV void load16(const uint16_t *p, float (&v)[16]) {
  const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
  const uint4 b = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
H3_DEV void load16(const float *p, float (&v)[16]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p) + q);
    v[4 * q] = a.x;
    v[4 * q + 1] = a.y;
    v[4 * q + 2] = a.z;
    v[4 * q + 3] = a.w;
  }
}

// Unit u (16 elements) of a [rows, k] matrix: its row and its place in it.
struct Unit {
  long long row;
  int at;
};
H3_DEV Unit unit_of(long long u, int per_row) {
  Unit r;
  r.row = u / per_row;
  r.at = static_cast<int>(u - r.row * per_row);
  return r;
}

template <int FMT, typename T>
__global__ void __launch_bounds__(kThreads)
    fp4_quantize_kernel(const T *__restrict__ src, long long ld, long long units, int k,
                        const float *__restrict__ g, uint8_t *__restrict__ dst,
                        uint8_t *__restrict__ sf) {
  const Fp4Tensor t = fp4_tensor(FMT == kFp4Nv ? g : nullptr);
  const int per_row = k / 16;
  const int chunks = (k / Fp4<FMT>::BLOCK + 3) / 4;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  // units is a multiple of 4, so the four lanes that share a scale store stay together
  for (long long u = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; u < units;
       u += step) {
    const unsigned live = __activemask();
    const Unit at = unit_of(u, per_row);
    float v[16];
    load16(src + at.row * ld + 16 * at.at, v);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = amax_nan(amax, fabsf(v[i]));
    if (FMT == kFp4Mx) amax = amax_nan(amax, __shfl_xor_sync(live, amax, 1));
    float inv;
    const uint32_t sb = fp4_scale<FMT>(amax, t, &inv);
    *reinterpret_cast<uint2 *>(dst + at.row * (k / 2) + 8 * at.at) =
        make_uint2(fp4_pack8(v, inv), fp4_pack8(v + 8, inv));
    const int row = static_cast<int>(at.row);
    if (FMT == kFp4Nv) {
      uint32_t w = sb << (8 * (at.at & 3));
      w |= __shfl_xor_sync(live, w, 1);
      w |= __shfl_xor_sync(live, w, 2);
      if ((at.at & 3) == 0) *reinterpret_cast<uint32_t *>(sf + mx_sf_offset(row, at.at, chunks)) = w;
    } else {
      const int s = at.at >> 1;
      uint32_t w = sb << (8 * (s & 1));
      w |= __shfl_xor_sync(live, w, 2);
      if ((at.at & 3) == 0) {
        *reinterpret_cast<uint16_t *>(sf + mx_sf_offset(row, s, chunks)) = static_cast<uint16_t>(w);
        // the last group of four scales of a row with 64 elements left over
        if (at.at + 4 == per_row && (s & 2) == 0)
          *reinterpret_cast<uint16_t *>(sf + mx_sf_offset(row, s + 2, chunks)) = 0;
      }
    }
  }
}

template <int FMT>
__global__ void __launch_bounds__(kThreads)
    fp4_dequantize_kernel(const uint8_t *__restrict__ q, const uint8_t *__restrict__ sf,
                          long long units, int k, const float *__restrict__ g,
                          uint16_t *__restrict__ out) {
  const float gv = g ? __ldg(g) : 1.f;
  const int per_row = k / 16;
  const int chunks = (k / Fp4<FMT>::BLOCK + 3) / 4;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  for (long long u = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; u < units;
       u += step) {
    const Unit at = unit_of(u, per_row);
    const uint2 w = __ldg(reinterpret_cast<const uint2 *>(q + at.row * (k / 2) + 8 * at.at));
    const int s = FMT == kFp4Nv ? at.at : at.at >> 1;
    const float d =
        fp4_scale_value<FMT>(__ldg(sf + mx_sf_offset(static_cast<int>(at.row), s, chunks)), gv);
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = ((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xffu;
      const __half2_raw h =
          __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(b), __NV_E2M1);
      const float2 f = __half22float2(__half2(h));
      o[i] = pack_bf16x2(__fmul_rn(f.x, d), __fmul_rn(f.y, d));
    }
    uint16_t *dst = out + at.row * k + 16 * at.at;
    st_global_v4(dst, o[0], o[1], o[2], o[3]);
    st_global_v4(dst + 8, o[4], o[5], o[6], o[7]);
  }
}

// Largest finite magnitude of the matrix over 2688 = 6 * 448 (1 for a matrix
// of zeros). Each block leaves its maximum in `part`; the block that finds
// itself last (by `done`, which it sets back to 0) joins them. A maximum does
// not depend on the order, so neither does the result.
template <typename T>
__global__ void __launch_bounds__(kThreads)
    fp4_tensor_scale_kernel(const T *__restrict__ src, long long ld, long long units, int k,
                            float *__restrict__ part, unsigned *__restrict__ done,
                            float *__restrict__ out) {
  __shared__ float red[kThreads / 32];
  __shared__ bool last;
  const int per_row = k / 16;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  float m = 0.f;
  for (long long u = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; u < units;
       u += step) {
    const Unit at = unit_of(u, per_row);
    float v[16];
    load16(src + at.row * ld + 16 * at.at, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = fabsf(v[i]);
      m = a < INFINITY ? fmaxf(m, a) : m;
    }
  }
  auto block_max = [&](float x) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    float r = red[0];
#pragma unroll
    for (int w = 1; w < kThreads / 32; ++w) r = fmaxf(r, red[w]);
    return r;
  };
  m = block_max(m);
  if (threadIdx.x == 0) {
    part[blockIdx.x] = m;
    __threadfence();
    last = atomicAdd(done, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  m = 0.f;
  for (int i = threadIdx.x; i < static_cast<int>(gridDim.x); i += kThreads)
    m = fmaxf(m, __ldcg(part + i));
  __syncthreads();  // red[] is read above by every thread
  m = block_max(m);
  if (threadIdx.x == 0) {
    *out = m > 0.f ? __fdiv_rn(m, 2688.f) : 1.f;
    *done = 0;
  }
}

int grid_for(long long units, int num_sms) {
  const long long want = (units + kThreads - 1) / kThreads;
  return static_cast<int>(want < 8LL * num_sms ? want : 8LL * num_sms);
}

}  // namespace

cudaError_t launch_fp4_quantize(int fmt, const void *src, bool f32, long long ld, int rows, int k,
                                const float *g, uint8_t *dst, uint8_t *sf, int num_sms,
                                cudaStream_t s) {
  const long long units = static_cast<long long>(rows) * (k / 16);
  const int grid = grid_for(units, num_sms);
  auto run = [&](auto kernel, auto *p) {
    kernel<<<grid, kThreads, 0, s>>>(p, ld, units, k, g, dst, sf);
    return cudaGetLastError();
  };
  const float *pf = static_cast<const float *>(src);
  const uint16_t *pb = static_cast<const uint16_t *>(src);
  if (fmt == kFp4Mx)
    return f32 ? run(fp4_quantize_kernel<kFp4Mx, float>, pf)
               : run(fp4_quantize_kernel<kFp4Mx, uint16_t>, pb);
  return f32 ? run(fp4_quantize_kernel<kFp4Nv, float>, pf)
             : run(fp4_quantize_kernel<kFp4Nv, uint16_t>, pb);
}

cudaError_t launch_fp4_dequantize(int fmt, const uint8_t *q, const uint8_t *sf, int rows, int k,
                                  const float *g, void *out, int num_sms, cudaStream_t s) {
  const long long units = static_cast<long long>(rows) * (k / 16);
  const int grid = grid_for(units, num_sms);
  uint16_t *o = static_cast<uint16_t *>(out);
  if (fmt == kFp4Mx)
    fp4_dequantize_kernel<kFp4Mx><<<grid, kThreads, 0, s>>>(q, sf, units, k, g, o);
  else
    fp4_dequantize_kernel<kFp4Nv><<<grid, kThreads, 0, s>>>(q, sf, units, k, g, o);
  return cudaGetLastError();
}

cudaError_t launch_fp4_tensor_scale(const void *src, bool f32, long long ld, int rows, int k,
                                    float *part, unsigned *done, float *out, int num_sms,
                                    cudaStream_t s) {
  const long long units = static_cast<long long>(rows) * (k / 16);
  int grid = grid_for(units, num_sms);
  if (grid > kFp4ScaleParts) grid = kFp4ScaleParts;
  if (f32)
    fp4_tensor_scale_kernel<<<grid, kThreads, 0, s>>>(static_cast<const float *>(src), ld, units,
                                                      k, part, done, out);
  else
    fp4_tensor_scale_kernel<<<grid, kThreads, 0, s>>>(static_cast<const uint16_t *>(src), ld,
                                                      units, k, part, done, out);
  return cudaGetLastError();
}

}  // namespace h3
