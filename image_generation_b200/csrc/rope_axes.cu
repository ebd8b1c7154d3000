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
// Bound by HBM: every element is read and written once. A warp takes a token (or
// a share of its heads where there are few tokens): a group of G lanes (a power of
// two >= head_dim / 16) owns one head at a time, each lane the same 8 pairs of
// every head, so a head's sum of squares is log2(G) shuffles and the lane keeps
// cosine and sine, times the norm's weights, in registers for all heads of the
// token. Positions are fp32, so the angle is formed and reduced to a half turn in
// fp64 (far positions). The warp's next heads are on their way to shared memory
// (cp.async, whole lines at a time).
// 16896 tokens x 112 heads x 96: 118 us replayed, 129 called on new rows each time, 5.6
// TB/s (replayed, 181 with cosines in shared memory per head, 164 with loads to
// registers); 20736 x 64 x 128, neighbours: 112 and 123. Sections that are not multiples of
// 8 pairs, split, are another matter: 2-byte accesses and a pair's place worked out per
// head, 967 us where neighbours take 154 (16896 x 112 x 128).
#include <type_traits>

#include "kernels.h"
#include "ptx.cuh"

namespace h3 {
namespace {

constexpr int kThreads = 256;
constexpr int kPerSm = 3;  // CTAs: 80 registers a thread
constexpr int kDepth = 4;  // rounds of heads of a warp in shared memory

// Eight values as four packed pairs.
struct Eight {
  uint64_t v[4];
};
// Eight elements in shared memory.
H3_DEV void load8(uint32_t at, const uint16_t *, float (&v)[8]) {
  const float4 f = ld_shared_v4(at);
  const uint32_t w[4] = {__float_as_uint(f.x), __float_as_uint(f.y), __float_as_uint(f.z),
                         __float_as_uint(f.w)};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
H3_DEV void load8(uint32_t at, const float *, float (&v)[8]) {
  const float4 a = ld_shared_v4(at), b = ld_shared_v4(at + 16);
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
H3_DEV Eight eight(const float (&v)[8]) {
  return {f2_pack(v[0], v[1]), f2_pack(v[2], v[3]), f2_pack(v[4], v[5]), f2_pack(v[6], v[7])};
}
H3_DEV void floats(const Eight &e, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) f2_unpack(e.v[i], v[2 * i], v[2 * i + 1]);
}
H3_DEV Eight shared8(const float *p) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  return {f2_pack(a.x, a.y), f2_pack(a.z, a.w), f2_pack(b.x, b.y), f2_pack(b.z, b.w)};
}
H3_DEV void store8(uint16_t *p, const float (&v)[8]) {
  st_global_v4(p, pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
               pack_bf16x2(v[6], v[7]));
}
H3_DEV void store8(float *p, const float (&v)[8]) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
H3_DEV float load1(uint32_t at, const uint16_t *) { return __uint_as_float(ld_shared_u16(at) << 16); }
H3_DEV float load1(uint32_t at, const float *) { return __uint_as_float(ld_shared_u32(at)); }
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

// The 8 pairs (a, b) of one lane, from two pieces of 8 elements.
template <int ORDER>
H3_DEV void pairs_of(const float (&x)[8], const float (&y)[8], Eight &a, Eight &b) {
  if constexpr (ORDER == kInterleaved) {
    const float ea[8] = {x[0], x[2], x[4], x[6], y[0], y[2], y[4], y[6]};
    const float eb[8] = {x[1], x[3], x[5], x[7], y[1], y[3], y[5], y[7]};
    a = eight(ea), b = eight(eb);
  } else {
    a = eight(x), b = eight(y);
  }
}
template <typename T, int ORDER>
H3_DEV void store_pairs(const RopeAxesParams &p, T *h, int u, int lo, int hi, const Eight &ea,
                        const Eight &eb) {
  float a[8], b[8];
  floats(ea, a);
  floats(eb, b);
  if constexpr (ORDER == kInterleaved) {
    const float x[8] = {a[0], b[0], a[1], b[1], a[2], b[2], a[3], b[3]};
    const float y[8] = {a[4], b[4], a[5], b[5], a[6], b[6], a[7], b[7]};
    store8(h + lo, x);
    store8(h + hi, y);
  } else if constexpr (ORDER == kSplit8) {
    store8(h + lo, a);
    store8(h + hi, b);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const Pair q = split_pair(p, 8 * u + i);
      store1(h + q.lo, a[i]);
      store1(h + q.hi, b[i]);
    }
  }
}

// PARTIAL: part of the head passes through.
template <typename T, int ORDER, int G_LOG2, bool PARTIAL>
__global__ void __launch_bounds__(kThreads, kPerSm)
    rope_axes_kernel(const __grid_constant__ RopeAxesParams p, int parts) {
  __shared__ __align__(16) float cs[kThreads / 32][2][kRopeMaxPairs];  // of each warp's token
  constexpr int GROUPS = 32 >> G_LOG2;
  constexpr uint32_t ROUND = GROUPS * (16 << G_LOG2) * sizeof(T);  // bytes of GROUPS heads, at most
  extern __shared__ __align__(16) uint8_t ring_smem[];  // of each warp: kDepth rounds
  const int half = p.head_dim / 2;
  const int turning = p.sec[0] + p.sec[1] + p.sec[2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u = lane & ((1 << G_LOG2) - 1), group = lane >> G_LOG2;
  const bool on = u < p.head_dim / 16;
  // the lane's two pieces of 8 elements in a head
  int lo = 16 * u, hi = 16 * u + 8;
  if (ORDER == kSplit8 && on) {
    const Pair at = split_pair(p, 8 * u);
    lo = at.lo, hi = at.hi;
  }
  const float inv_dh = 1.f / static_cast<float>(p.head_dim);
  const int stride = GROUPS * p.head_dim;
  const uint32_t ring = smem_u32(ring_smem) + warp * kDepth * ROUND;
  const uint32_t head_at = group * p.head_dim * sizeof(T);
  const int round_units = stride * static_cast<int>(sizeof(T)) / 16;  // 16-byte pieces
  const long long tasks = static_cast<long long>(p.n) * parts;
  const long long task = static_cast<long long>(blockIdx.x) * (kThreads / 32) + warp;
  if (task >= tasks) return;
  const long long t = task / parts;
  const int part = static_cast<int>(task - t * parts);
  // this part's rounds of GROUPS heads: q's, then k's
  auto rounds_of = [&](int heads) { return (heads + GROUPS - 1) / GROUPS; };
  auto first_of = [&](int heads, int i) { return rounds_of(heads) * i / parts; };
  // on their way to shared memory one after another, whole lines at a time
  uint32_t to = ring;
  int which = 0, ahead = 0, left = 0;  // of the matrix being fetched: rounds, 16-byte pieces
  const uint8_t *from = nullptr;
  auto begin = [&](int w) {
    const int heads = w ? p.heads[1] : p.heads[0];
    const int r0 = first_of(heads, part), r1 = first_of(heads, part + 1);
    const T *src = w ? static_cast<const T *>(p.src[1]) + t * p.ld_src[1]
                     : static_cast<const T *>(p.src[0]) + t * p.ld_src[0];
    which = w;
    ahead = r1 - r0;
    from = reinterpret_cast<const uint8_t *>(src + r0 * stride) + 16 * lane;
    left = (min(r1 * GROUPS, heads) - r0 * GROUPS) * p.head_dim * static_cast<int>(sizeof(T)) / 16 -
           lane;
  };
  auto fetch = [&] {
    if (ahead == 0 && which == 0) begin(1);
    if (ahead > 0) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(ROUND / 512); ++i)
        if (32 * i + lane < round_units && 32 * i < left)
          cp_async16(to + 16 * lane + 512 * i, from + 512 * i);
      from += stride * sizeof(T);
      left -= round_units;
      --ahead;
    }
    cp_async_commit();
    to = to == ring + (kDepth - 1) * ROUND ? ring : to + ROUND;
  };
  begin(0);
#pragma unroll
  for (int i = 0; i < kDepth - 1; ++i) fetch();
  for (int pair = lane; pair < half; pair += 32) {
    float c = 1.f, s = 0.f;  // where nothing turns
    if (pair < turning) {
      const int axis = pair < p.sec[0] ? 0 : pair < p.sec[0] + p.sec[1] ? 1 : 2;
      // in half turns, reduced to [-1, 1] where fp32 is exact enough
      double a = static_cast<double>(__ldg(p.pos + 3 * t + axis)) * p.half_turns[pair];
      a -= 2.0 * rint(0.5 * a);
      sincospif(static_cast<float>(a), &s, &c);
      if (p.inverse) s = -s;
    }
    cs[warp][0][pair] = c;
    cs[warp][1][pair] = s;
  }
  __syncwarp();
  uint32_t at = ring;
#pragma unroll 1
  for (int w = 0; w < 2; ++w) {
    const int heads = w ? p.heads[1] : p.heads[0];
    const int r0 = first_of(heads, part), r1 = first_of(heads, part + 1);
    if (r0 >= r1) continue;
    int head = r0 * GROUPS + group;  // of this lane in the round at hand
    const int end = on ? min(r1 * GROUPS, heads) : 0;
    T *dst = w ? static_cast<T *>(p.dst[1]) + t * p.ld_dst[1]
               : static_cast<T *>(p.dst[0]) + t * p.ld_dst[0];
    dst += head * p.head_dim;
    // x = a (wa c) - b (wb s), y = b (wb c) + a (wa s)
    Eight ac = shared8(&cs[warp][0][on ? 8 * u : 0]), as = shared8(&cs[warp][1][on ? 8 * u : 0]);
    Eight bc = ac, bs = as;
    if (const float *weight = w ? p.weight[1] : p.weight[0]; weight && on) {
      float wa[8], wb[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        Pair q{16 * u + 2 * i, 16 * u + 2 * i + 1};
        if (ORDER == kSplit8) q = {lo + i, hi + i};
        if (ORDER == kSplitAny) q = split_pair(p, 8 * u + i);
        wa[i] = __ldg(weight + q.lo);
        wb[i] = __ldg(weight + q.hi);
      }
      const Eight va = eight(wa), vb = eight(wb);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        ac.v[i] = f2_mul(ac.v[i], va.v[i]);
        as.v[i] = f2_mul(as.v[i], va.v[i]);
        bc.v[i] = f2_mul(bc.v[i], vb.v[i]);
        bs.v[i] = f2_mul(bs.v[i], vb.v[i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) bs.v[i] = f2_mul(bs.v[i], f2_pack(-1.f, -1.f));
#pragma unroll 1
    for (int r = r0; r < r1; ++r) {
      __syncwarp();  // the round before has been read: its place is free
      fetch();
      cp_async_wait_but<kDepth - 1>();
      __syncwarp();  // the other lanes' copies too
      const bool live = head < end;
      Eight a{}, b{};
      if (live) {
        float x[8], y[8];
        if constexpr (ORDER == kSplitAny) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const Pair q = split_pair(p, 8 * u + i);
            x[i] = load1(at + head_at + q.lo * sizeof(T), static_cast<const T *>(nullptr));
            y[i] = load1(at + head_at + q.hi * sizeof(T), static_cast<const T *>(nullptr));
          }
        } else {
          load8(at + head_at + lo * sizeof(T), static_cast<const T *>(nullptr), x);
          load8(at + head_at + hi * sizeof(T), static_cast<const T *>(nullptr), y);
        }
        pairs_of<ORDER>(x, y, a, b);
      }
      const uint32_t here = at + head_at;
      at = at == ring + (kDepth - 1) * ROUND ? ring : at + ROUND;
      float rinv = 1.f;
      if (p.norm) {
        uint64_t ss = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) ss = f2_fma(a.v[i], a.v[i], f2_fma(b.v[i], b.v[i], ss));
        float s0, s1;
        f2_unpack(ss, s0, s1);
        s0 += s1;
#pragma unroll
        for (int o = 1 << G_LOG2 >> 1; o > 0; o >>= 1) s0 += __shfl_xor_sync(0xffffffffu, s0, o);
        rinv = rsqrtf(s0 * inv_dh + p.eps);
        const uint64_t scale = f2_pack(rinv, rinv);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a.v[i] = f2_mul(a.v[i], scale);
          b.v[i] = f2_mul(b.v[i], scale);
        }
      }
      if (live) {
        Eight x, y;
        if (PARTIAL && 8 * u >= turning) {
          // passes through, and stays out of its neighbour, an infinity too
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x.v[i] = f2_mul(a.v[i], ac.v[i]);
            y.v[i] = f2_mul(b.v[i], bc.v[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            x.v[i] = f2_fma(a.v[i], ac.v[i], f2_mul(b.v[i], bs.v[i]));
            y.v[i] = f2_fma(b.v[i], bc.v[i], f2_mul(a.v[i], as.v[i]));
          }
        }
        if (PARTIAL && ORDER != kSplit8 && turning % 8 && u == turning / 8) {
          // the lane in which the rotation ends: its other pairs from the ring again, so
          // that the rest keeps no registers for this
          float fx[8], fy[8];
          floats(x, fx);
          floats(y, fy);
          const float *weight = w ? p.weight[1] : p.weight[0];
#pragma unroll 1
          for (int i = turning % 8; i < 8; ++i) {
            Pair q{16 * u + 2 * i, 16 * u + 2 * i + 1};
            if (ORDER != kInterleaved) q = split_pair(p, 8 * u + i);
            const T *type = nullptr;
            float va = load1(here + q.lo * sizeof(T), type) * rinv;
            float vb = load1(here + q.hi * sizeof(T), type) * rinv;
            if (weight) va *= __ldg(weight + q.lo), vb *= __ldg(weight + q.hi);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (j == i) fx[j] = va, fy[j] = vb;
          }
          x = eight(fx);
          y = eight(fy);
        }
        store_pairs<T, ORDER>(p, dst, u, lo, hi, x, y);
      }
      head += GROUPS;
      dst += stride;
    }
  }
  cp_async_wait_all();  // empty groups
}

template <typename T, int ORDER, int G_LOG2, bool PARTIAL>
cudaError_t launch_kernel(const RopeAxesParams &p, int num_sms, cudaStream_t s) {
  static PerDevice attr;
  constexpr int kBytes = kDepth * (32 >> G_LOG2) * (16 << G_LOG2) * static_cast<int>(sizeof(T)) *
                         (kThreads / 32);
  cudaError_t e = set_smem_once(attr, rope_axes_kernel<T, ORDER, G_LOG2, PARTIAL>, kBytes);
  if (e != cudaSuccess) return e;
  const int groups = 32 >> G_LOG2;
  const int rounds = ((p.heads[0] > p.heads[1] ? p.heads[0] : p.heads[1]) + groups - 1) / groups;
  // a token's heads go to several warps where there are fewer tokens than warps
  const long long warps = static_cast<long long>(kPerSm) * num_sms * (kThreads / 32);
  long long parts = warps / p.n;
  parts = parts < 1 ? 1 : parts > rounds ? rounds : parts;
  // one task per warp: in persistent CTAs the last round was uneven (129 against 123 us)
  const int grid = static_cast<int>((p.n * parts + kThreads / 32 - 1) / (kThreads / 32));
  rope_axes_kernel<T, ORDER, G_LOG2, PARTIAL><<<grid, kThreads, kBytes, s>>>(p, static_cast<int>(parts));
  return cudaGetLastError();
}

template <typename T, int ORDER, int G_LOG2>
cudaError_t launch_groups(const RopeAxesParams &p, int num_sms, cudaStream_t s) {
  return 2 * (p.sec[0] + p.sec[1] + p.sec[2]) < p.head_dim
             ? launch_kernel<T, ORDER, G_LOG2, true>(p, num_sms, s)
             : launch_kernel<T, ORDER, G_LOG2, false>(p, num_sms, s);
}

template <typename T, int ORDER>
cudaError_t launch(const RopeAxesParams &p, int num_sms, cudaStream_t s) {
  if (p.head_dim <= 64) return launch_groups<T, ORDER, 2>(p, num_sms, s);
  if (p.head_dim <= 128) return launch_groups<T, ORDER, 3>(p, num_sms, s);
  return launch_groups<T, ORDER, 4>(p, num_sms, s);
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
