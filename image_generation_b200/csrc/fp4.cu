// FP4 matrices from and to wider types (next to mx_quantize): the tensor scale
// of an NVFP4 matrix, quantisation, and the values that a quantised matrix
// stands for.
//
// All three are bound by HBM: 2 bytes read per bf16 element and 1/2 byte plus
// 1/32 or 1/16 written (the tensor scale only reads, the values are written as 2
// bytes). One lane owns 16 consecutive elements (32 bytes of bf16 in one access),
// so an NVFP4 block needs no exchange between lanes and an MXFP4 block one
// shuffle; four lanes (64 elements, what rows are a multiple of) join their scale
// bytes into one store. The quantization goes from the matrix's end to its
// beginning: what the tensor scale's pass read last is still in L2, and what it
// writes last is what a reader from the beginning wants first. 16896 x 5376 of
// bf16, NVFP4: tensor scale 29 us (6.2 TB/s), quantization 42 (5.5), values 38
// (6.1); one after another 118.
#include "fp4.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;

// 32 bytes; `wide`: the address is a multiple of 32 (else of 16).
H3_DEV Words8 load32(const void *p, bool wide) {
  if (wide) return ld_global_v8(p);
  const uint4 a = __ldg(static_cast<const uint4 *>(p));
  const uint4 b = __ldg(static_cast<const uint4 *>(p) + 1);
  return {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// 16 consecutive elements as loaded, and as fp32.
template <typename T>
struct Unit {
  Words8 w[sizeof(T) / 2];
};
template <typename T>
H3_DEV void load16(const T *p, bool wide, Unit<T> &u) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T) / 2); ++i)
    u.w[i] = load32(reinterpret_cast<const uint8_t *>(p) + 32 * i, wide);
}
H3_DEV void values16(const Unit<uint16_t> &u, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(u.w[0].v[i] << 16);
    v[2 * i + 1] = __uint_as_float(u.w[0].v[i] & 0xffff0000u);
  }
}
H3_DEV void values16(const Unit<float> &u, float (&v)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(u.w[i / 8].v[i % 8]);
}
bool is_wide(const void *p, long long row_bytes) {
  return (reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(row_bytes)) % 32 == 0;
}

// Units (16 elements) of a [rows, k] matrix that one thread passes over, `step`
// apart: the row and the place in it, kept without a division per unit.
struct Walk {
  long long row, dr;
  int at, da, per_row;
  H3_DEV Walk(long long u, long long step, int n) : per_row(n) {
    row = u / n;
    at = static_cast<int>(u - row * n);
    dr = step / n;
    da = static_cast<int>(step - dr * n);
  }
  H3_DEV void next() {
    row += dr;
    at += da;
    if (at >= per_row) at -= per_row, ++row;
  }
};

template <int FMT, typename T>
__global__ void __launch_bounds__(kThreads)
    fp4_quantize_kernel(const T *__restrict__ src, long long ld, bool wide, long long rows, int k,
                        const float *__restrict__ g, uint8_t *__restrict__ dst,
                        uint8_t *__restrict__ sf) {
  const Fp4Tensor t = fp4_tensor(FMT == kFp4Nv ? g : nullptr);
  const int per_row = k / 16;
  const int chunks = (k / Fp4<FMT>::BLOCK + 3) / 4;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  // rows count from the last one; a row is a multiple of four units, so the four
  // lanes that share a scale store stay together
  Walk at(static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x, step, per_row);
  Walk ahead = at;  // the next unit is loaded before this one's arithmetic
  Unit<T> here{};
  if (at.row < rows) load16(src + (rows - 1 - at.row) * ld + 16 * at.at, wide, here);
  for (; at.row < rows; at.next()) {
    const unsigned live = 0xfu << (threadIdx.x & 28);  // these four lanes
    const long long r = rows - 1 - at.row;
    float v[16];
    values16(here, v);
    ahead.next();
    if (ahead.row < rows) load16(src + (rows - 1 - ahead.row) * ld + 16 * ahead.at, wide, here);
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) amax = amax_nan(amax, fabsf(v[i]));
    if (FMT == kFp4Mx) amax = amax_nan(amax, __shfl_xor_sync(live, amax, 1));
    float inv;
    const uint32_t sb = fp4_scale<FMT>(amax, t, &inv);
    *reinterpret_cast<uint2 *>(dst + r * (k / 2) + 8 * at.at) =
        make_uint2(fp4_pack8(v, inv), fp4_pack8(v + 8, inv));
    const int row = static_cast<int>(r);
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
                          long long rows, int k, const float *__restrict__ g,
                          uint16_t *__restrict__ out, bool wide) {
  const float gv = g ? __ldg(g) : 1.f;
  const int per_row = k / 16;
  const int chunks = (k / Fp4<FMT>::BLOCK + 3) / 4;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  Walk at(static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x, step, per_row);
  Walk ahead = at;  // the next unit is loaded before this one's arithmetic
  uint2 w = make_uint2(0, 0);
  uint32_t sb = 0;
  auto load = [&](const Walk &u) {
    w = __ldg(reinterpret_cast<const uint2 *>(q + u.row * (k / 2) + 8 * u.at));
    sb = __ldg(sf + mx_sf_offset(static_cast<int>(u.row), FMT == kFp4Nv ? u.at : u.at >> 1, chunks));
  };
  if (at.row < rows) load(at);
  for (; at.row < rows; at.next()) {
    const uint2 codes = w;
    const float scale = fp4_scale_value<FMT>(sb), d = __fmul_rn(scale, gv);
    ahead.next();
    if (ahead.row < rows) load(ahead);
    Words8 o;
    auto values = [&](auto &&value) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t b = ((i < 4 ? codes.x : codes.y) >> (8 * (i & 3))) & 0xffu;
        const __half2_raw h =
            __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(b), __NV_E2M1);
        const float2 f = __half22float2(__half2(h));
        o.v[i] = pack_bf16x2(value(f.x), value(f.y));
      }
    };
    if (!isinf(d))
      values([&](float e) { return __fmul_rn(e, d); });
    else  // the first product is exact, or infinite where g > 1 makes the whole so: 0 stays 0
      values([&](float e) { return __fmul_rn(__fmul_rn(e, scale), gv); });
    uint16_t *dst = out + at.row * k + 16 * at.at;
    if (wide) {
      st_global_v8(dst, o);
    } else {
      st_global_v4(dst, o.v[0], o.v[1], o.v[2], o.v[3]);
      st_global_v4(dst + 8, o.v[4], o.v[5], o.v[6], o.v[7]);
    }
  }
}

// Largest finite magnitude of the matrix over 2688 = 6 * 448, at least 2^-149 (1
// for a matrix of zeros): a scale of 0 would make NaN of a matrix whose quotient
// rounds to 0, where 2^-149 gives zeros, as the scales just above it do. Each block
// leaves its maximum in `part`, and a block of a second launch joins them: a maximum
// does not depend on the order, so neither does the result, and nothing that an
// earlier call left in `part` is read. (A counter by which the last block of one launch
// joins them makes every later scale wrong once it is off 0, by a call cut short or,
// against the rule, overlapped by another of its context. 16896 x 5376 of bf16: 29.5 us;
// with such a counter 30.2, and 33.9 where it is set to 0 before each launch.)
H3_DEV float block_max(float x, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
  __syncthreads();
  float r = red[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) r = fmaxf(r, red[w]);
  return r;
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    fp4_amax_kernel(const T *__restrict__ src, long long ld, bool wide, long long rows, int k,
                    float *__restrict__ part) {
  __shared__ float red[kThreads / 32];
  const int per_row = k / 16;
  const long long step = static_cast<long long>(gridDim.x) * kThreads;
  float m = 0.f;
  for (Walk at(static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x, step, per_row);
       at.row < rows; at.next()) {
    Unit<T> here;
    load16(src + at.row * ld + 16 * at.at, wide, here);
    float v[16];
    values16(here, v);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float a = fabsf(v[i]);
      m = a < INFINITY ? fmaxf(m, a) : m;
    }
  }
  m = block_max(m, red);
  if (threadIdx.x == 0) part[blockIdx.x] = m;
}

// Launched while the kernel above still runs: its block is in place when that ends.
__global__ void __launch_bounds__(kThreads)
    fp4_tensor_scale_kernel(const float *__restrict__ part, int parts, float *__restrict__ out) {
  __shared__ float red[kThreads / 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");  // until the parts are written
  float m = 0.f;
  for (int i = threadIdx.x; i < parts; i += kThreads) m = fmaxf(m, __ldcg(part + i));
  m = block_max(m, red);
  if (threadIdx.x == 0)
    *out = m > 0.f ? fmaxf(__fdiv_rn(m, 2688.f), __uint_as_float(1u)) : 1.f;
}

int grid_for(long long units, int num_sms, int per_sm) {
  const long long want = (units + kThreads - 1) / kThreads, most = static_cast<long long>(per_sm) * num_sms;
  return static_cast<int>(want < most ? want : most);
}

}  // namespace

cudaError_t launch_fp4_quantize(int fmt, const void *src, bool f32, long long ld, int rows, int k,
                                const float *g, uint8_t *dst, uint8_t *sf, int num_sms,
                                cudaStream_t s) {
  const long long units = static_cast<long long>(rows) * (k / 16);
  const int grid = grid_for(units, num_sms, 8);
  const bool wide = is_wide(src, ld * (f32 ? 4 : 2));
  auto run = [&](auto kernel, auto *p) {
    kernel<<<grid, kThreads, 0, s>>>(p, ld, wide, rows, k, g, dst, sf);
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
  // more CTAs than fit at once: 38.3 against 45.9 us with 8 per SM (16896 x 5376)
  const int grid = grid_for(units, num_sms, 64);
  uint16_t *o = static_cast<uint16_t *>(out);
  const bool wide = is_wide(out, 2LL * k);
  if (fmt == kFp4Mx)
    fp4_dequantize_kernel<kFp4Mx><<<grid, kThreads, 0, s>>>(q, sf, rows, k, g, o, wide);
  else
    fp4_dequantize_kernel<kFp4Nv><<<grid, kThreads, 0, s>>>(q, sf, rows, k, g, o, wide);
  return cudaGetLastError();
}

cudaError_t launch_fp4_tensor_scale(const void *src, bool f32, long long ld, int rows, int k,
                                    float *part, float *out, int num_sms, cudaStream_t s) {
  const long long units = static_cast<long long>(rows) * (k / 16);
  int grid = grid_for(units, num_sms, 8);
  if (grid > kFp4ScaleParts) grid = kFp4ScaleParts;
  const bool wide = is_wide(src, ld * (f32 ? 4 : 2));
  if (f32)
    fp4_amax_kernel<<<grid, kThreads, 0, s>>>(static_cast<const float *>(src), ld, wide, rows, k, part);
  else
    fp4_amax_kernel<<<grid, kThreads, 0, s>>>(static_cast<const uint16_t *>(src), ld, wide, rows, k,
                                              part);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(1, 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fp4_tensor_scale_kernel, static_cast<const float *>(part), grid, out);
}

}  // namespace h3
