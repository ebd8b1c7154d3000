// The norms on either side of a branch's residual addition, in one pass over
// the rows: with x the fp32 residual stream and y a branch's output,
//   x' = r x + gate * (post ? RMSNorm(y) post_weight : y)
//   out = RMSNorm(x') pre_weight (1 + scale) + shift
// where RMSNorm(v) = v / sqrt(mean(v^2) + eps), x' is kept in fp32 and out is
// rounded once, to bf16, MXFP8, MXFP4 or NVFP4. gate, shift and scale have one
// row per image of a batch (rows_per_group rows share one).
//
// Bound by HBM: 4 + 2 bytes read and 4 + 2 written per element with bf16 y and
// out. A CTA owns a row at a time, a thread two chunks of 4 columns of every row
// the CTA takes (16 bytes of x a lane: whole lines per warp), so it holds its part
// of the modulation in registers and x' stays there between its sum of squares
// and its use; a scale block of the output (16 or 32 elements) spans four or
// eight neighbouring lanes. The next rows are on their way to shared memory
// meanwhile (cp.async, each thread its own columns, so nobody waits for
// another's copy). 16896 x 5376 with a bf16 branch and output: 161 us replayed on the
// same buffers, 167 on three sets in turn, 184 called with new ones each time (5.9 TB/s
// of the 1.09 GB that it cannot do without); MXFP8 rows 198, MXFP4 198, NVFP4 215, where a
// chunk of 4 elements takes up to 3 shuffles and a scale. What was tried, on the same
// buffers: 306 with loads to registers and the modulation read for every row; 260 with 32
// bytes per lane instead of 16; 209 and 189 with twice and one and a half times the
// instructions of now; two rows in hand per barrier 273, out of registers.
#include "fp4.cuh"

namespace h3 {
namespace {

constexpr int kMaxThreads = 1024;  // 8 columns each: d <= 8192
constexpr int kMaxWarps = kMaxThreads / 32;
constexpr int kRows = 4;                  // rows in shared memory per CTA, fewer where wide
constexpr int kSmemBytes = 200 * 1024;    // of one SM, for all its CTAs

// Four values as two packed pairs.
struct Four {
  uint64_t lo, hi;
};
H3_DEV Four four(float a, float b, float c, float d) { return {f2_pack(a, b), f2_pack(c, d)}; }
H3_DEV Four four(float4 v) { return four(v.x, v.y, v.z, v.w); }
H3_DEV float4 unpack(const Four &v) {
  float4 r;
  f2_unpack(v.lo, r.x, r.y);
  f2_unpack(v.hi, r.z, r.w);
  return r;
}
H3_DEV Four mul(const Four &a, const Four &b) { return {f2_mul(a.lo, b.lo), f2_mul(a.hi, b.hi)}; }
H3_DEV Four fma(const Four &a, const Four &b, const Four &c) {
  return {f2_fma(a.lo, b.lo, c.lo), f2_fma(a.hi, b.hi, c.hi)};
}
H3_DEV Four all(float v) { return four(v, v, v, v); }
H3_DEV float sum_squares(const Four &a, const Four &b) {
  float x, y;
  f2_unpack(f2_fma(a.lo, a.lo, f2_fma(a.hi, a.hi, f2_fma(b.lo, b.lo, f2_mul(b.hi, b.hi)))), x, y);
  return x + y;
}
// Four floats of a vector (`other` where there is none).
H3_DEV Four vec4(const float *p, int at, float other) {
  return p ? four(__ldg(reinterpret_cast<const float4 *>(p + at))) : all(other);
}
// Four elements in shared memory.
H3_DEV Four chunk4(uint32_t at, const float *) { return four(ld_shared_v4(at)); }
H3_DEV Four chunk4(uint32_t at, const uint16_t *) {
  const uint2 a = ld_shared_v2(at);
  return four(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xffff0000u),
              __uint_as_float(a.y << 16), __uint_as_float(a.y & 0xffff0000u));
}

// Sum over the block; `red` (zero past the block's warps) is not written again
// before another barrier has passed. Each warp adds the warps' sums up by itself.
H3_DEV float block_sum(float v, float *red) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[threadIdx.x & 31];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Chunk `c` of a row in the output's type. Every lane of the warp calls it; `on`
// is the same for the lanes that share a scale block.
template <int OUT>
H3_DEV void store_chunk(const GatedNormParams &p, const Fp4Tensor &t, int row, int c, bool on,
                        const Four &value) {
  const size_t at = static_cast<size_t>(row) * p.d + 4 * c;
  const float4 f = unpack(value);
  const float v[4] = {f.x, f.y, f.z, f.w};
  if constexpr (OUT == kNormBf16) {
    if (on)
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
          make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
  } else if constexpr (OUT == kNormMxfp8) {
    float am = fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
    const uint32_t sb = mx_scale_byte(am);
    const float m = mx_inv_scale(sb);
    if (!on) return;
    *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.out) + at) =
        mx_pack4(v[0] * m, v[1] * m, v[2] * m, v[3] * m);
    if ((c & 7) == 0) p.out_sf[mx_sf_offset(row, c >> 3, p.d / 128)] = static_cast<uint8_t>(sb);
  } else {
    constexpr int FMT = OUT == kNormFp4Mx ? kFp4Mx : kFp4Nv;
    constexpr int PER = Fp4<FMT>::BLOCK / 4;  // chunks per scale block
    float am = 0.f, inv;
#pragma unroll
    for (int i = 0; i < 4; ++i) am = amax_nan(am, fabsf(v[i]));
#pragma unroll
    for (int o = 1; o < PER; o <<= 1) am = amax_nan(am, __shfl_xor_sync(0xffffffffu, am, o));
    const uint32_t sb = fp4_scale<FMT>(am, t, &inv);
    if (!on) return;
    *reinterpret_cast<uint16_t *>(static_cast<uint8_t *>(p.out) + at / 2) =
        static_cast<uint16_t>(fp4_pack4(__fmul_rn(v[0], inv), __fmul_rn(v[1], inv),
                                        __fmul_rn(v[2], inv), __fmul_rn(v[3], inv)));
    if ((c & (PER - 1)) == 0) {
      const int s = c / PER, chunks = (p.d / Fp4<FMT>::BLOCK + 3) / 4;
      uint8_t *sf = p.out_sf + mx_sf_offset(row, s, chunks);
      *sf = static_cast<uint8_t>(sb);
      // a row that ends with two of its last four scales: the others are 0
      if (FMT == kFp4Mx && 4 * (c + PER) == p.d && (s & 3) == 1)
        *reinterpret_cast<uint16_t *>(sf + 1) = 0;
    }
  }
}

// FULL: every thread has both of its chunks.
template <typename TB, int OUT, bool FULL>
__global__ void __launch_bounds__(kMaxThreads, 1)
    gated_norm_kernel(const GatedNormParams p, bool post, int depth) {
  extern __shared__ __align__(16) uint8_t rows_smem[];
  __shared__ __align__(16) float red[2][kMaxWarps];
  const int c0 = threadIdx.x, c1 = threadIdx.x + blockDim.x;  // chunks of this thread
  const bool on0 = FULL || c0 < p.d / 4, on1 = FULL || c1 < p.d / 4;
  const float inv_d = 1.f / static_cast<float>(p.d);
  const TB *branch = static_cast<const TB *>(p.branch);
  Fp4Tensor t{};
  if constexpr (OUT == kNormFp4Nv) t = fp4_tensor(p.out_scale);
  if (threadIdx.x < 2 * kMaxWarps) red[threadIdx.x / kMaxWarps][threadIdx.x % kMaxWarps] = 0.f;
  if (blockDim.x < 2 * kMaxWarps && threadIdx.x + 32 < 2 * kMaxWarps)
    red[(threadIdx.x + 32) / kMaxWarps][(threadIdx.x + 32) % kMaxWarps] = 0.f;
  __syncthreads();

  const uint32_t row_bytes = p.d * (4 + sizeof(TB));
  const uint32_t rows0 = smem_u32(rows_smem);
  // one group of copies per row, empty past the last: this CTA's rows in turn
  const long long apart = static_cast<long long>(gridDim.x) * p.d;
  const long long begin = static_cast<long long>(blockIdx.x) * p.d + 4 * c0;
  const int second = 4 * static_cast<int>(blockDim.x);  // from a row's first chunk to its second
  const float *next_x = p.x + begin;
  const TB *next_y = branch ? branch + begin : nullptr;
  long long next_row = blockIdx.x;
  uint32_t next_at = rows0;
  const uint32_t rows_end = rows0 + depth * row_bytes, branch_at = 4 * p.d;
  auto fetch = [&] {
    if (next_row < p.n) {
      const uint32_t at = next_at + 16 * c0, by = next_at + branch_at + 4 * sizeof(TB) * c0;
      if (on0) cp_async16(at, next_x);
      if (on1) cp_async16(at + 4 * second, next_x + second);
      if (branch) {
        if (on0) cp_async<4 * sizeof(TB)>(by, next_y);
        if (on1) cp_async<4 * sizeof(TB)>(by + sizeof(TB) * second, next_y + second);
      }
    }
    cp_async_commit();
    next_row += gridDim.x;
    next_x += apart;
    if (branch) next_y += apart;
    next_at += row_bytes;
    if (next_at == rows_end) next_at = rows0;
  };
  for (int i = 0; i < depth - 1; ++i) fetch();

  // gate post_weight, pre_weight (1 + scale), shift of the columns of this thread
  Four gw[2] = {all(0.f), all(0.f)}, up[2] = {all(0.f), all(0.f)}, add[2] = {all(0.f), all(0.f)};
  const Four rs = all(p.residual_scale);
  long long group_end = 0;  // first row past the modulation in hand
  uint32_t at = rows0;
  float4 *x_out = p.x_out ? reinterpret_cast<float4 *>(p.x_out + begin) : nullptr;
  for (int row = blockIdx.x; row < p.n; row += gridDim.x) {
    if (row >= group_end) {
      const int g = row / p.rows_per_group;
      group_end = (g + 1LL) * p.rows_per_group;
      const size_t mod = static_cast<size_t>(g) * p.ld_mod;
      auto load = [&](int j, int c) {
        gw[j] = mul(vec4(p.gate ? p.gate + mod : nullptr, 4 * c, 1.f), vec4(p.post_weight, 4 * c, 1.f));
        const Four w = vec4(p.pre_weight, 4 * c, 1.f);
        const Four one = all(1.f);
        const Four sc = vec4(p.scale ? p.scale + mod : nullptr, 4 * c, 0.f);
        up[j] = mul(w, fma(sc, one, one));
        add[j] = vec4(p.shift ? p.shift + mod : nullptr, 4 * c, 0.f);
      };
      if (on0) load(0, c0);
      if (on1) load(1, c1);
    }
    fetch();  // to the slot that the row before this one left
    cp_async_wait_but(depth - 1);
    Four x[2], y[2] = {all(0.f), all(0.f)};
    if (!FULL) x[0] = x[1] = all(0.f);
    {
      const uint32_t ax = at + 16 * c0, ay = at + branch_at + 4 * sizeof(TB) * c0;
      if (on0) x[0] = chunk4(ax, p.x);
      if (on1) x[1] = chunk4(ax + 4 * second, p.x);
      if (branch && on0) y[0] = chunk4(ay, branch);
      if (branch && on1) y[1] = chunk4(ay + sizeof(TB) * second, branch);
    }
    at += row_bytes;
    if (at == rows_end) at = rows0;
    if (post) {
      const Four r = all(rsqrtf(block_sum(sum_squares(y[0], y[1]), red[0]) * inv_d + p.eps));
      y[0] = mul(y[0], r);
      y[1] = mul(y[1], r);
    }
    // without a branch y is 0
    x[0] = fma(gw[0], y[0], mul(x[0], rs));
    x[1] = fma(gw[1], y[1], mul(x[1], rs));
    if (x_out) {
      if (on0) __stcs(x_out, unpack(x[0]));
      if (on1) __stcs(x_out + blockDim.x, unpack(x[1]));
      x_out += apart / 4;
    }
    const Four r = all(rsqrtf(block_sum(sum_squares(x[0], x[1]), red[1]) * inv_d + p.eps));
    store_chunk<OUT>(p, t, row, c0, on0, fma(mul(x[0], r), up[0], add[0]));
    store_chunk<OUT>(p, t, row, c1, on1, fma(mul(x[1], r), up[1], add[1]));
    if (!post) __syncthreads();  // red[1] is read above; the next row writes it with no other barrier
  }
  cp_async_wait_all();
}

template <typename TB, int OUT, bool FULL>
cudaError_t launch_full(const GatedNormParams &p, bool post, int num_sms, cudaStream_t s) {
  static PerDevice attr;
  const int threads = (p.d / 8 + 31) / 32 * 32;
  const int row_bytes = p.d * (4 + static_cast<int>(sizeof(TB)));
  // threads of an SM at 64 registers; rows in flight as far as shared memory goes
  int per_sm = 1024 / threads;
  if (per_sm > 16) per_sm = 16;
  int depth = kSmemBytes / (per_sm * row_bytes);
  if (depth > kRows) depth = kRows;
  if (depth < 2) depth = 2;
  const long long most = static_cast<long long>(num_sms) * per_sm;
  if (p.n <= most) depth = 2;  // a CTA has one row
  cudaError_t e = set_smem_once(attr, gated_norm_kernel<TB, OUT, FULL>, kSmemBytes);
  if (e != cudaSuccess) return e;
  const int grid = static_cast<int>(p.n < most ? p.n : most);
  gated_norm_kernel<TB, OUT, FULL><<<grid, threads, depth * row_bytes, s>>>(p, post, depth);
  return cudaGetLastError();
}

template <typename TB, int OUT>
cudaError_t launch(const GatedNormParams &p, bool post, int num_sms, cudaStream_t s) {
  return p.d % 256 == 0 ? launch_full<TB, OUT, true>(p, post, num_sms, s)
                        : launch_full<TB, OUT, false>(p, post, num_sms, s);
}

template <typename TB>
cudaError_t launch_out(const GatedNormParams &p, bool post, int kind, int num_sms, cudaStream_t s) {
  switch (kind) {
    case kNormBf16:
      return launch<TB, kNormBf16>(p, post, num_sms, s);
    case kNormMxfp8:
      return launch<TB, kNormMxfp8>(p, post, num_sms, s);
    case kNormFp4Mx:
      return launch<TB, kNormFp4Mx>(p, post, num_sms, s);
    case kNormFp4Nv:
      return launch<TB, kNormFp4Nv>(p, post, num_sms, s);
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
