// Rotary positions on three axes (frame, row, column) applied to the rows of Q
// and K, with an optional RMSNorm of each head before: for head vector h of the
// token at (p0, p1, p2),
//   u = norm ? h / sqrt(mean(h^2) + eps) weight : h
//   pair j of axis i turns by a = p_i theta^(-j / s_i):
//     (u_lo, u_hi) -> (u_lo cos a - u_hi sin a, u_hi cos a + u_lo sin a)
// s_i pairs per axis, the axes one after another; a pair is two neighbours
// (interleaved) or elements j and s_i + j of the axis's section (split). What
// is left of the head passes through. The inverse turns by -a, which is also
// the gradient of the rotation.
//
// Bound by HBM: every element is read and written once. Positions are fp32, so
// the angle is formed and reduced to a half turn in fp64 (far positions), and
// its sine and cosine are computed once per token in shared memory for all
// heads. A group of G lanes (a power of two >= head_dim / 16) owns one head,
// each lane 8 pairs, so the head's sum of squares is log2(G) shuffles.
#include "kernels.h"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;
constexpr int kMaxTokens = 8;  // tokens per CTA and pass

H3_DEV void load8(const uint16_t *p, float (&v)[8]) {
  const uint4 a = *reinterpret_cast<const uint4 *>(p);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
H3_DEV void load8(const float *p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
H3_DEV void store8(uint16_t *p, const float (&v)[8]) {
  st_global_v4(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
               pack_bf16x2(v[6], v[7]));
}
H3_DEV void store8(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
H3_DEV float load1(const uint16_t *p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
H3_DEV float load1(const float *p) { return *p; }
H3_DEV void store1(uint16_t *p, float v) { *p = static_cast<uint16_t>(pack_bf16x2(v, 0.f)); }
H3_DEV void store1(float *p, float v) { *p = v; }

// Where the two elements of a pair lie in a head.
struct Pair {
  int lo, hi;
};
H3_DEV Pair split_pair(const RopeAxesParams &p, int pair) {
  int first = 0, s = p.sec[0];
  if (pair >= first + s) first += s, s = p.sec[1];
  if (pair >= first + s) first += s, s = p.sec[2];
  if (pair >= first + s) first += s, s = p.head_dim / 2 - first;  // what passes through
  return {first + pair, first + pair + s};
}

enum Order { kInterleaved, kSplit8, kSplitAny };  // kSplit8: every section a multiple of 8 pairs

// The 8 pairs of one lane as (a, b).
template <typename T, int ORDER>
H3_DEV void load_pairs(const RopeAxesParams &p, const T *h, int u, const Pair &at, float (&a)[8],
                       float (&b)[8]) {
  if constexpr (ORDER == kInterleaved) {
    float x[8], y[8];
    load8(h + 16 * u, x);
    load8(h + 16 * u + 8, y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = x[2 * i], b[i] = x[2 * i + 1];
      a[4 + i] = y[2 * i], b[4 + i] = y[2 * i + 1];
    }
  } else if constexpr (ORDER == kSplit8) {
    load8(h + at.lo, a);
    load8(h + at.hi, b);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Pair q = split_pair(p, 8 * u + i);
      a[i] = load1(h + q.lo);
      b[i] = load1(h + q.hi);
    }
  }
}
template <typename T, int ORDER>
H3_DEV void store_pairs(const RopeAxesParams &p, T *h, int u, const Pair &at, const float (&a)[8],
                        const float (&b)[8]) {
  if constexpr (ORDER == kInterleaved) {
    float x[8], y[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = a[i], x[2 * i + 1] = b[i];
      y[2 * i] = a[4 + i], y[2 * i + 1] = b[4 + i];
    }
    store8(h + 16 * u, x);
    store8(h + 16 * u + 8, y);
  } else if constexpr (ORDER == kSplit8) {
    store8(h + at.lo, a);
    store8(h + at.hi, b);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Pair q = split_pair(p, 8 * u + i);
      store1(h + q.lo, a[i]);
      store1(h + q.hi, b[i]);
    }
  }
}

template <typename T, int ORDER>
__global__ void __launch_bounds__(kThreads)
    rope_axes_kernel(const __grid_constant__ RopeAxesParams p, int tokens, int g_log2) {
  // cosines, then sines of the pairs of each token; 1 and 0 where nothing turns
  __shared__ __align__(16) float cs[kMaxTokens][2][kRopeMaxPairs];
  const int half = p.head_dim / 2, units = p.head_dim / 16;
  const int turning = p.sec[0] + p.sec[1] + p.sec[2];
  const int u = threadIdx.x & ((1 << g_log2) - 1);
  const int group = threadIdx.x >> g_log2, groups = kThreads >> g_log2;
  const bool on = u < units;
  Pair at{0, 0};
  if (ORDER == kSplit8 && on) at = split_pair(p, 8 * u);
  const float inv_dh = 1.f / static_cast<float>(p.head_dim);
  for (long long t0 = static_cast<long long>(blockIdx.x) * tokens; t0 < p.n;
       t0 += static_cast<long long>(gridDim.x) * tokens) {
    const int tn = static_cast<int>(p.n - t0 < tokens ? p.n - t0 : tokens);
    for (int i = threadIdx.x; i < tn * half; i += kThreads) {
      const int tok = i / half, pair = i - tok * half;
      float c = 1.f, s = 0.f;
      if (pair < turning) {
        const int axis = pair < p.sec[0] ? 0 : pair < p.sec[0] + p.sec[1] ? 1 : 2;
        // in half turns, reduced to [-1, 1] where fp32 is exact enough
        double a = static_cast<double>(__ldg(p.pos + 3 * (t0 + tok) + axis)) * p.half_turns[pair];
        a -= 2.0 * rint(0.5 * a);
        sincospif(static_cast<float>(a), &s, &c);
        if (p.inverse) s = -s;
      }
      cs[tok][0][pair] = c;
      cs[tok][1][pair] = s;
    }
    __syncthreads();
#pragma unroll 1
    for (int w = 0; w < 2; ++w) {
      const int heads = p.heads[w], items = tn * heads;
      const T *src = static_cast<const T *>(p.src[w]) + t0 * p.ld_src[w];
      T *dst = static_cast<T *>(p.dst[w]) + t0 * p.ld_dst[w];
      float wa[8], wb[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) wa[i] = wb[i] = 1.f;
      if (p.weight[w] && on && items) load_pairs<float, ORDER>(p, p.weight[w], u, at, wa, wb);
      // every lane takes the same number of turns: the shuffles need whole warps
      for (int first = 0; first < items; first += groups) {
        const int it = first + group;
        const bool live = on && it < items;
        const int tok = live ? it / heads : 0, head = live ? it - tok * heads : 0;
        float a[8], b[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.f;
        if (live)
          load_pairs<T, ORDER>(p, src + tok * p.ld_src[w] + head * p.head_dim, u, at, a, b);
        if (p.norm) {
          float ss = 0.f;
#pragma unroll
          for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
          for (int o = (1 << g_log2) >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float r = rsqrtf(ss * inv_dh + p.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) a[i] *= r * wa[i], b[i] *= r * wb[i];
        }
        if (live) {
          const float4 *c4 = reinterpret_cast<const float4 *>(&cs[tok][0][8 * u]);
          const float4 *s4 = reinterpret_cast<const float4 *>(&cs[tok][1][8 * u]);
          const float4 c0 = c4[0], c1 = c4[1], s0 = s4[0], s1 = s4[1];
          const float c[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
          const float s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float x = a[i], y = b[i];
            a[i] = x * c[i] - y * s[i];
            b[i] = y * c[i] + x * s[i];
          }
          store_pairs<T, ORDER>(p, dst + tok * p.ld_dst[w] + head * p.head_dim, u, at, a, b);
        }
      }
    }
    __syncthreads();  // cs[] is rewritten for the next tokens
  }
}

template <typename T, int ORDER>
cudaError_t launch(const RopeAxesParams &p, int num_sms, cudaStream_t s) {
  int g = 0;
  while ((16 << g) < p.head_dim) ++g;
  // several tokens per pass where there are enough of them to fill the SMs
  int tokens = static_cast<int>(p.n / (4LL * num_sms));
  tokens = tokens < 1 ? 1 : tokens > kMaxTokens ? kMaxTokens : tokens;
  const long long want = (static_cast<long long>(p.n) + tokens - 1) / tokens;
  const int grid = static_cast<int>(want < 8LL * num_sms ? want : 8LL * num_sms);
  rope_axes_kernel<T, ORDER><<<grid, kThreads, 0, s>>>(p, tokens, g);
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_order(const RopeAxesParams &p, bool interleaved, int num_sms, cudaStream_t s) {
  if (interleaved) return launch<T, kInterleaved>(p, num_sms, s);
  if (p.sec[0] % 8 == 0 && p.sec[1] % 8 == 0 && p.sec[2] % 8 == 0)
    return launch<T, kSplit8>(p, num_sms, s);
  return launch<T, kSplitAny>(p, num_sms, s);
}

}  // namespace

cudaError_t launch_rope_axes(const RopeAxesParams &p, bool f32, bool interleaved, int num_sms,
                             cudaStream_t s) {
  return f32 ? launch_order<float>(p, interleaved, num_sms, s)
             : launch_order<uint16_t>(p, interleaved, num_sms, s);
}

}  // namespace h3
