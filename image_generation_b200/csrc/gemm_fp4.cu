// Block-scaled FP4 tcgen05 GEMM: acc[m, n] = sum_k A[m, k] W[n, k] with A and W
// in E2M1 (two per byte) and a scale per 32 (MXFP4, E8M0) or per 16 (NVFP4,
// E4M3) consecutive k of every row, fp32 accumulate in tensor memory; then
// alpha = (A's tensor scale) (W's tensor scale), the bias, and one of
//   STORE            out bf16 = v
//   GELU             out bf16 = GELU(v), or the same rounded to FP4
//   GATED_RESIDUAL   out fp32 = resid + gate * v
// with v = alpha acc + bias.
//
// Two kernels: 256 x 256 tiles on pairs of CTAs, persistent, for products that
// fill the SMs with them; 128 x 128 tiles with k split over a cluster for the
// rest. In both one warp loads (128 bytes = 256 k of each row per k-block, in
// 128-byte swizzle, and that k-block's scale blocks, into a ring of stages), one
// warp copies the scales into tensor memory (tcgen05.cp) and issues the MMAs, one
// per 64 k, and the others run the epilogue. The loading and the issuing warp
// stay converged and elect a lane around their instructions: from a single
// lane's branch, the operands' way into uniform registers took twice the MMAs' time.
//
// Bound, large: by what the tensor cores and L2 give at the card's power. NVFP4
// 8192^3 196 us (5.6 PFLOP/s; MMAs and loads alone 154, with the scales' copies 179),
// MXFP4 16896 x 14336 x 5376 with GELU 486 us in a short run (5.4; 412 without an
// epilogue), 564 in a long one at the power limit and 539 with FP4 rows, NVFP4 4608 x
// 5376 x 14336 into the residual 157, 189 called with new operands each time (that
// instance spills, 60 bytes stored and 224 loaded by ptxas's count, with 16 warps 132 and
// 136). Few rows: by reading W. One row x 32256
// x 5376 13.8 us with W partly in L2, 21 from HBM (97.5 MB).
//
// k is a multiple of 64: a last k-block with fewer than four groups of 64 reads
// zeros past the row (TMA fill) and issues only the MMAs whose k exist, so the
// padding of the scale blocks is never multiplied.
#include "fp4.cuh"
#include "gemm_epilogue.cuh"
#include "kernels.h"
#include "ptx.cuh"

namespace h3 {
namespace {

using namespace gemm_detail;

constexpr int BM = 128;
constexpr int BKB = 128;       // bytes of a row per k-block
constexpr int BK = 2 * BKB;    // elements
constexpr int SF = 512;        // bytes of a scale block: 128 rows x 4 scales
constexpr uint32_t TMEM_COLS = 512;

template <int FMT>
struct Kb {  // scale blocks per k-block, and MMAs that share one
  static constexpr int CHUNKS = BK / (4 * Fp4<FMT>::BLOCK);
  static constexpr int PER_CHUNK = 4 / CHUNKS;
};

// alpha = ga * gw, as a factor and a second one, applied first, that is 1 unless
// the product leaves the normal range of fp32. Then it is the larger of the two: a sum
// times the smaller may be subnormal, and lose its bits, where the whole is not.
struct Alpha {
  float a, b;
};
H3_DEV Alpha tensor_alpha(const float *ga, const float *gw) {
  const float x = ga ? __ldg(ga) : 1.f, y = gw ? __ldg(gw) : 1.f;
  const float p = x * y;
  if (fabsf(p) >= 1.17549435e-38f && fabsf(p) < INFINITY) return {p, 1.f};
  return fabsf(x) < fabsf(y) ? Alpha{x, y} : Alpha{y, x};
}

// erf GELU of two values, x Phi(x) = max(x, 0) - |x| q with q = erfc(|x| / sqrt 2) / 2
// by Abramowitz & Stegun, Handbook of Mathematical Functions, 7.1.26 (|error| of
// erf <= 1.5e-7): q = t (b1 + ... + b5 t^4) e^(-x^2 / 2), t = 1 / (1 + p |x| / sqrt 2).
// In packed fp32 pairs: one value at a time, the epilogue of a product
// 16896 x 14336 x 5376 took 97 of its 514 us. |x| is kept finite, so that its
// product with an e of 0 is 0 (a NaN stays one by way of e).
H3_DEV void gelu2(float &a, float &b) {
  auto c2 = [](float c) { return f2_pack(c, c); };
  const uint64_t x = f2_pack(a, b);
  const uint64_t ax = f2_pack(fminf(fabsf(a), 3e38f), fminf(fabsf(b), 3e38f));
  float d0, d1, t0, t1, e0, e1;
  f2_unpack(f2_fma(ax, c2(0.3275911f * 0.70710678118654752f), c2(1.f)), d0, d1);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t0) : "f"(d0));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t1) : "f"(d1));
  f2_unpack(f2_mul(f2_mul(x, c2(-0.5f * 1.4426950408889634f)), x), e0, e1);
  const uint64_t t = f2_pack(t0, t1), e = f2_pack(ex2_approx(e0), ex2_approx(e1));
  uint64_t q = f2_fma(c2(0.5f * 1.061405429f), t, c2(0.5f * -1.453152027f));
  q = f2_fma(q, t, c2(0.5f * 1.421413741f));
  q = f2_fma(q, t, c2(0.5f * -0.284496736f));
  q = f2_fma(q, t, c2(0.5f * 0.254829592f));
  q = f2_mul(f2_mul(q, t), f2_mul(e, ax));
  float q0, q1;
  f2_unpack(q, q0, q1);
  a = fmaxf(a, 0.f) - q0;
  b = fmaxf(b, 0.f) - q1;
}

// N accumulators of a row, as values: alpha acc + bias, then GELU, or the
// gated addition to the residual (resid(q): columns 4 q .. 4 q + 3 of it).
template <int EPI, int N, typename Resid>
H3_DEV void values(const Fp4GemmParams &p, const Alpha &al, const uint32_t (&acc)[N], int col,
                   Resid &&resid, float (&v)[N]) {
  // in packed pairs
  uint64_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i)
    w[i] = f2_pack(__uint_as_float(acc[2 * i]), __uint_as_float(acc[2 * i + 1]));
  if (al.b != 1.f) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = f2_mul(w[i], f2_pack(al.b, al.b));
  }
  const uint64_t alpha = f2_pack(al.a, al.a);
  if (p.bias) {
    const float4 *b = reinterpret_cast<const float4 *>(p.bias + col);
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const float4 bb = __ldg(b + q);
      w[2 * q] = f2_fma(w[2 * q], alpha, f2_pack(bb.x, bb.y));
      w[2 * q + 1] = f2_fma(w[2 * q + 1], alpha, f2_pack(bb.z, bb.w));
    }
  } else {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = f2_mul(w[i], alpha);
  }
  if constexpr (EPI == kEpiGatedResidual) {
    const float4 *g = reinterpret_cast<const float4 *>(p.gate + col);
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      const float4 gg = __ldg(g + q), x = resid(q);
      w[2 * q] = f2_fma(f2_pack(gg.x, gg.y), w[2 * q], f2_pack(x.x, x.y));
      w[2 * q + 1] = f2_fma(f2_pack(gg.z, gg.w), w[2 * q + 1], f2_pack(x.z, x.w));
    }
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) f2_unpack(w[i], v[2 * i], v[2 * i + 1]);
  if constexpr (EPI == kEpiGelu || EPI == kEpiGeluFp4) {
    // one branch for all, not one each
    if (p.gelu_tanh) {
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = gelu_f(v[i], 1);
    } else {
#pragma unroll
      for (int i = 0; i < N; i += 2) gelu2(v[i], v[i + 1]);
    }
  }
}

// 32 values of a row rounded to the operands' FP4 format.
template <int FMT>
H3_DEV void store_fp4(const Fp4GemmParams &p, const Fp4Tensor &t, const float (&v)[32], int row,
                      int col) {
  uint32_t q[4], sb[2];
  fp4_quant32<FMT>(v, t, q, sb);
  st_global_v4(static_cast<uint8_t *>(p.out) + (static_cast<size_t>(row) * p.n + col) / 2, q[0],
               q[1], q[2], q[3]);
  const int chunks = (p.n / Fp4<FMT>::BLOCK + 3) / 4;
  uint8_t *sf = p.out_sf + mx_sf_offset(row, col / Fp4<FMT>::BLOCK, chunks);
  if constexpr (FMT == kFp4Nv) {
    *reinterpret_cast<uint16_t *>(sf) = static_cast<uint16_t>(sb[0] | (sb[1] << 8));
  } else {
    *sf = static_cast<uint8_t>(sb[0]);
    // a row that ends with two of its last four scales: the others are 0
    if (col + 32 == p.n && p.n % 128 == 64) *reinterpret_cast<uint16_t *>(sf + 1) = 0;
  }
}

// The same with 8 values in a lane: two or four neighbouring lanes share a scale
// block, and four lanes from a multiple of four on call this together.
template <int FMT>
H3_DEV void store_fp4_by8(const Fp4GemmParams &p, const Fp4Tensor &t, const float (&v)[8], int row,
                          int col) {
  const unsigned live = 0xfu << (threadIdx.x & 28);
  float am = 0.f, inv;
#pragma unroll
  for (int i = 0; i < 8; ++i) am = amax_nan(am, fabsf(v[i]));
  am = amax_nan(am, __shfl_xor_sync(live, am, 1));
  if constexpr (FMT == kFp4Mx) am = amax_nan(am, __shfl_xor_sync(live, am, 2));
  const uint32_t sb = fp4_scale<FMT>(am, t, &inv);
  *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(p.out) +
                                (static_cast<size_t>(row) * p.n + col) / 2) = fp4_pack8(v, inv);
  constexpr int B = Fp4<FMT>::BLOCK;
  if (col % B) return;
  uint8_t *sf = p.out_sf + mx_sf_offset(row, col / B, (p.n / B + 3) / 4);
  *sf = static_cast<uint8_t>(sb);
  // a row that ends with two of its last four scales: the others are 0
  if (FMT == kFp4Mx && col + B == p.n && p.n % 128 == 64) *reinterpret_cast<uint16_t *>(sf + 1) = 0;
}

// ---------------------------------------------------------- few tiles: split k
// Output tiles of 128 x 128, one per CTA or per cluster of up to eight CTAs that
// share its k-blocks: for few rows (where reading W bounds the call) and for
// products with too few 256 x 256 tiles to fill the SMs. Two CTAs fit on an SM, so
// one's epilogue runs beside the other's loads.
//   warp 0 TMA and bulk loads, warp 1 MMAs (M128 N128 K64), warps 2..5 epilogue.
// In a cluster CTA r finishes a slice of the tile's rows: the others store their
// partial sums of those rows into its shared memory (the stages, free once every
// CTA of the cluster has no MMA left), and it adds them up in the order of their
// k, so a result does not depend on which CTA was first. (Reading the partial
// tiles from the other CTAs instead waits for each load: 40 us for 128 rows.)
namespace split {
constexpr int BN = 128;
constexpr int THREADS = 192;
constexpr int MAX_SPLIT = 8;
constexpr int B_BYTES = BN * BKB;
constexpr uint32_t TCOLS = 256;  // of each CTA's tensor memory
constexpr uint32_t SF_COL0 = BN;

// ROWS: rows of A that are loaded, BM or, for up to 32, fewer: then a stage is
// smaller and there is one more of them on the way. (The MMA reads BM rows of
// shared memory; those past ROWS give rows that nobody reads.)
template <int FMT, int ROWS>
struct Tile {
  static constexpr int STAGES = ROWS == BM ? 3 : 4;
  static constexpr int A_BYTES = ROWS * BKB;
  static constexpr int SF_BYTES = Kb<FMT>::CHUNKS * SF;  // of A or W, one k-block
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + 2 * SF_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 1;
  static constexpr int SMEM_BYTES = STAGES * STAGE_BYTES + 1024 + NUM_BARS * 8 + 16;
  static constexpr uint32_t SF_COLS = 8 * Kb<FMT>::CHUNKS;  // per stage: A, then W
};
constexpr int FEW = 32;
constexpr int SLOTS_BYTES = (BM + MAX_SPLIT) * BN * 4;  // the parts of a slice of rows
template <int FMT, int ROWS>
constexpr bool tile_ok() {
  using T = Tile<FMT, ROWS>;
  return SF_COL0 + T::STAGES * T::SF_COLS <= TCOLS &&       // tensor memory
         T::STAGE_BYTES % 1024 == 0 &&                      // stages start on swizzle atoms
         BM * BKB <= T::STAGE_BYTES &&                      // the MMA's A rows lie in the stage
         2 * (T::SMEM_BYTES + 1024) <= 228 * 1024 &&        // two CTAs per SM
         SLOTS_BYTES + 4 * 4096 <= T::STAGES * T::STAGE_BYTES;  // slots and boxes fit
}
static_assert(tile_ok<kFp4Nv, BM>() && tile_ok<kFp4Mx, BM>() && tile_ok<kFp4Nv, FEW>() &&
                  tile_ok<kFp4Mx, FEW>(),
              "tile sizes");

// A row's 32 values to global memory.
template <int FMT, int EPI>
H3_DEV void store32(const Fp4GemmParams &p, const Fp4Tensor &to, const float (&v)[32], int row,
                    int col) {
  const size_t at = static_cast<size_t>(row) * p.n + col;
  if constexpr (EPI == kEpiGatedResidual) {
    float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
#pragma unroll
    for (int q = 0; q < 8; ++q) o[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
  } else if constexpr (EPI == kEpiGeluFp4) {
    store_fp4<FMT>(p, to, v, row, col);
  } else {
    store_bf16_row<32>(static_cast<uint16_t *>(p.out) + at, v);
  }
}

template <int FMT, int EPI, int ROWS>
__global__ void __launch_bounds__(THREADS, 2)
    gemm_fp4_split(const __grid_constant__ CUtensorMap tma_a,
                   const __grid_constant__ CUtensorMap tma_b, const Fp4GemmParams p, int splits,
                   int a_rows) {
  using T = Tile<FMT, ROWS>;
  constexpr bool NV = FMT == kFp4Nv;
  constexpr int STAGES = T::STAGES, A_BYTES = T::A_BYTES;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + STAGES * T::STAGE_BYTES);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + T::NUM_BARS);
  __shared__ int entry_status;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = smem_u32(bars);
  auto FULL = [&](int s) { return bar0 + 8u * s; };
  auto EMPTY = [&](int s) { return bar0 + 8u * (STAGES + s); };
  const uint32_t TFULL = bar0 + 8u * (2 * STAGES);

  if (threadIdx.x == 0) {
    entry_status = *reinterpret_cast<const volatile int *>(p.status);
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(FULL(s), 1);
      mbar_init(EMPTY(s), 1);
    }
    mbar_init(TFULL, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tma_a);
    tma_prefetch_desc(&tma_b);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), TCOLS);
    tmem_relinquish();
  }
  __syncwarp();
  tc_fence_before();
  if (splits > 1)
    cluster_sync();
  else
    __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  // whether to run at all is decided for the cluster as a whole, by its first CTA
  const bool skip =
      (splits > 1 ? static_cast<int>(ld_shared_cluster_u32(map_to_cta(smem_u32(&entry_status), 0)))
                  : entry_status) != 0;

  const int part = splits > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int tile = blockIdx.x / splits;
  int tm, tn;
  tile_coords(tile, p.tiles_m, p.tiles_n, tm, tn);
  const int kblocks = (p.k + BK - 1) / BK;
  const int kb0 = static_cast<int>(static_cast<long long>(kblocks) * part / splits);
  const int kb1 = static_cast<int>(static_cast<long long>(kblocks) * (part + 1) / splits);

  if (!skip && warp == 0) {
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_warp(EMPTY(stage), phase ^ 1, p.status)) break;
      ++issued;
      if (elect_one()) {
        const int c0 = kb * Kb<FMT>::CHUNKS;
        const uint32_t sf_bytes = min(Kb<FMT>::CHUNKS, p.chunks - c0) * SF;
        // a box counts whole, also where it reads past the matrix
        mbar_arrive_expect_tx(FULL(stage), a_rows * BKB + B_BYTES + 2 * sf_bytes);
        const uint32_t sa = sbase + stage * T::STAGE_BYTES;
        tma_load_2d(sa + A_BYTES, &tma_b, kb * BKB, tn * BN, FULL(stage));
        bulk_load(sa + A_BYTES + B_BYTES + T::SF_BYTES,
                  p.b_sf + (static_cast<size_t>(tn) * p.chunks + c0) * SF, sf_bytes, FULL(stage));
        tma_load_2d(sa, &tma_a, kb * BKB, tm * BM, FULL(stage));
        bulk_load(sa + A_BYTES + B_BYTES,
                  p.a_sf + (static_cast<size_t>(tm) * p.chunks + c0) * SF, sf_bytes, FULL(stage));
      }
      __syncwarp();
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    // every load has landed before the CTA may leave (the MMA warp may have given up)
    for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
      mbar_wait(FULL(i % STAGES), (i / STAGES) & 1, p.status, false);
  } else if (!skip && warp == 1) {
    int stage = 0;
    uint32_t phase = 0;
    for (int kb = kb0; kb < kb1; ++kb) {
      if (!mbar_wait_warp(FULL(stage), phase, p.status)) break;
      tc_fence_after();
      const uint32_t sa = sbase + stage * T::STAGE_BYTES;
      const uint64_t da = desc_sw128(sa, 16, 1024), db = desc_sw128(sa + A_BYTES, 16, 1024);
      const uint64_t dsf = desc_sf_copy(sa + A_BYTES + B_BYTES);
      const uint32_t sfa = tmem + SF_COL0 + T::SF_COLS * stage;
      const uint32_t sfb = sfa + 4 * Kb<FMT>::CHUNKS;
      const int groups = min(4, (p.k - kb * BK) / 64);
      if (elect_one()) {
#pragma unroll
        for (int c = 0; c < Kb<FMT>::CHUNKS; ++c) {
          if (c * Kb<FMT>::PER_CHUNK >= groups) break;
          tmem_cp_sf(sfa + 4 * c, dsf + c * SF / 16);
          tmem_cp_sf(sfb + 4 * c, dsf + (T::SF_BYTES + c * SF) / 16);
        }
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          if (g >= groups) break;
          const int c = g / Kb<FMT>::PER_CHUNK, id = 2 * (g % Kb<FMT>::PER_CHUNK);
          umma_fp4<NV>(tmem, da + 2 * g, db + 2 * g, idesc_fp4(BM, BN, NV, id), sfa + 4 * c,
                       sfb + 4 * c, (kb != kb0 || g != 0) ? 1u : 0u);
        }
        umma_commit(EMPTY(stage));
      }
      __syncwarp();
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (elect_one()) umma_commit(TFULL);
    __syncwarp();
    mbar_wait(TFULL, 0, p.status, false);  // no MMA is left when tensor memory is released
  } else if (!skip) {
    const int sub = warp & 3;
    const int in_tile = sub * 32 + lane;
    const int rows = min(BM, p.m - tm * BM);
    const bool ok = mbar_wait(TFULL, 0, p.status, false);
    tc_fence_after();
    if (__all_sync(0xffffffffu, ok) && sub * 32 < rows) {
      const uint32_t tbase = tmem + (static_cast<uint32_t>(sub * 32) << 16);
      if (splits == 1) {
        const Alpha al = tensor_alpha(p.a_scale, p.b_scale);
        Fp4Tensor to{};
        if constexpr (EPI == kEpiGeluFp4) to = fp4_tensor(FMT == kFp4Nv ? p.out_scale : nullptr);
        const int row = tm * BM + in_tile;
#pragma unroll 1
        for (int c = 0; c < BN && tn * BN + c < p.n; c += 32) {
          const int col = tn * BN + c;
          float4 x[8] = {};  // loaded before the first store: out may be resid
          if (EPI == kEpiGatedResidual && in_tile < rows) {
#pragma unroll
            for (int q = 0; q < 8; ++q)
              x[q] = reinterpret_cast<const float4 *>(p.resid + static_cast<size_t>(row) * p.n + col)[q];
          }
          uint32_t r[32];
          tmem_ld32(tbase + c, r);
          float v[32];
          values<EPI>(p, al, r, col, [&](int q) { return x[q]; }, v);
          if (in_tile < rows) store32<FMT, EPI>(p, to, v, row, col);
        }
      }
    }
  }
  if (splits > 1) {
    __syncwarp();
    cluster_sync();  // no MMA or load of the cluster uses the stages any more
    const int rows = min(BM, p.m - tm * BM);
    const int slice = (rows + splits - 1) / splits;  // rows that one CTA finishes
    const int sub = warp & 3;
    if (!skip && warp >= 2 && sub * 32 < rows) {
      // this CTA's part of a row to the row's CTA: slot `part` of its slots of
      // `slice` rows of BN floats, 16-byte unit q of row i at q ^ (i % 8). By way of
      // a box of 32 rows x 32 columns of its own, so that 8 lanes store a line.
      const uint32_t box = sbase + SLOTS_BYTES + sub * 4096;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < BN; c += 32) {
        uint32_t r[32];
        tmem_ld32(tmem + (static_cast<uint32_t>(sub * 32) << 16) + c, r);
#pragma unroll
        for (int q = 0; q < 8; ++q)
          st_shared_v4(box + lane * 128 + 16 * (q ^ (lane & 7)), r[4 * q], r[4 * q + 1],
                       r[4 * q + 2], r[4 * q + 3]);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int l = 4 * j + (lane >> 3), q = lane & 7, in_tile = sub * 32 + l;
          if (in_tile < rows) {
            const float4 v = ld_shared_v4(box + l * 128 + 16 * (q ^ (l & 7)));
            const int owner = in_tile / slice, i = in_tile - owner * slice;
            st_shared_cluster_v4(map_to_cta(sbase, owner) + (part * slice + i) * (BN * 4) +
                                     16 * ((c / 4 + q) ^ (i & 7)),
                                 __float_as_uint(v.x), __float_as_uint(v.y), __float_as_uint(v.z),
                                 __float_as_uint(v.w));
          }
        }
        __syncwarp();  // the box is written again
      }
    }
    __syncwarp();
    tc_fence_before();
    cluster_sync();  // every part has arrived
    if (!skip && warp >= 2) {
      const Alpha al = tensor_alpha(p.a_scale, p.b_scale);
      Fp4Tensor to{};
      if constexpr (EPI == kEpiGeluFp4) to = fp4_tensor(FMT == kFp4Nv ? p.out_scale : nullptr);
      const int r0 = min(rows, part * slice), mine = min(rows, r0 + slice) - r0;
      // 8 columns at a time; lanes that share a scale block of an FP4 output stay
      // together (n is a multiple of 32)
      const int groups = min(BN, p.n - tn * BN) / 8;
      for (int it = threadIdx.x - 64; it < mine * groups; it += 128) {
        const int i = it / groups, g = it - i * groups;
        const int row = tm * BM + r0 + i, col = tn * BN + 8 * g;
        const size_t at = static_cast<size_t>(row) * p.n + col;
        float4 x[2] = {};
        if (EPI == kEpiGatedResidual) {
          x[0] = reinterpret_cast<const float4 *>(p.resid + at)[0];
          x[1] = reinterpret_cast<const float4 *>(p.resid + at)[1];
        }
        float sum[8] = {};
        for (int s = 0; s < splits; ++s) {
          const uint32_t o = sbase + (s * slice + i) * (BN * 4);
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const float4 v = ld_shared_v4(o + 16 * ((2 * g + q) ^ (i & 7)));
            sum[4 * q + 0] += v.x;
            sum[4 * q + 1] += v.y;
            sum[4 * q + 2] += v.z;
            sum[4 * q + 3] += v.w;
          }
        }
        uint32_t r[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) r[q] = __float_as_uint(sum[q]);
        float v[8];
        values<EPI>(p, al, r, col, [&](int q) { return x[q]; }, v);
        if constexpr (EPI == kEpiGatedResidual) {
          float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at);
          o[0] = make_float4(v[0], v[1], v[2], v[3]);
          o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else if constexpr (EPI == kEpiGeluFp4) {
          store_fp4_by8<FMT>(p, to, v, row, col);
        } else {
          store_bf16_row<8>(static_cast<uint16_t *>(p.out) + at, v);
        }
      }
    }
    __syncwarp();
  } else {
    tc_fence_before();
    __syncthreads();
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TCOLS);
  }
}

template <int FMT, int EPI, int ROWS>
cudaError_t launch_tile(const Fp4GemmMaps &t, const Fp4GemmParams &p, const Fp4GemmPlan &plan,
                        cudaStream_t s) {
  static PerDevice smem_attr;
  constexpr int kSmem = Tile<FMT, ROWS>::SMEM_BYTES;
  cudaError_t e = set_smem_once(smem_attr, gemm_fp4_split<FMT, EPI, ROWS>, kSmem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(plan.grid, 1, 1);
  cfg.blockDim = dim3(THREADS, 1, 1);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = plan.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemm_fp4_split<FMT, EPI, ROWS>, t.a, t.b, p, plan.splits,
                            plan.box_a);
}

template <int FMT, int EPI>
cudaError_t launch(const Fp4GemmMaps &t, const Fp4GemmParams &p, const Fp4GemmPlan &plan,
                   cudaStream_t s) {
  return plan.box_a <= FEW ? launch_tile<FMT, EPI, FEW>(t, p, plan, s)
                           : launch_tile<FMT, EPI, BM>(t, p, plan, s);
}
}  // namespace split

// ------------------------------------------------------- a pair of CTAs per tile
// Output tiles of 256 x 256 on clusters of two CTAs (M256 N256 K64): each CTA
// loads its own 128 rows of A and 128 of W's 256, so a byte from L2 feeds twice
// the MACs of a one-CTA tile. (256 x 192, with two whole accumulators in tensor
// memory, ran the products a fifth slower.)
//
// Tensor memory: one accumulator in columns 0..255, and in 256..511 the scales of
// every stage. The epilogue first reads the whole accumulator into registers (128
// columns of a row per thread) and then lets the next tile's MMAs start; its
// arithmetic and stores run beside them. Overlapping the accumulators of
// successive tiles instead, for a shorter pause between them, leaves the scales of
// NVFP4 two k-blocks of columns; waiting for those cost more than the pause.
//
// The epilogue's rows go through shared memory (boxes of 32 rows x 128 bytes per
// warp, 64 bytes with FP4 rows) and leave by TMA stores. With SHORT sums the
// epilogue is what a tile waits for, and its warps wait for their loads and stores:
// then it has 16 of them instead of 8, 64 columns each, and the ring one stage less.
// NVFP4 8192 x 8192, 8 and 16 warps: GELU k 1024 89 and 73 us, 2048 94 and 87, 3584
// 113 and 119; into the residual (5376 columns) 98 and 84, 101 and 91, 105 and 109;
// stores 58 and 57, 75 and 83.
namespace pair {
constexpr int BN = 256;
// k-blocks up to which a sum is short.
constexpr int short_blocks(int epi) { return epi == kEpiStore ? 4 : 8; }
constexpr int A_BYTES = BM * BKB, B_BYTES = BN / 2 * BKB;
constexpr int OUT_BYTES = 4096;  // per epilogue warp: a box of 32 rows x 128 bytes
constexpr uint32_t SF_COL0 = BN;
constexpr uint16_t kBothCtas = 0x3, kFirstCta = 0x1;

template <int FMT, bool SHORT>
struct Tile {
  static constexpr int STAGES = SHORT ? 4 : 5;
  static constexpr int PARTS = SHORT ? 4 : 2;  // epilogue warps per TMEM lane quarter
  static constexpr int CHUNKS = BN / 32 / PARTS;  // 32 columns each, of one of them
  static constexpr int THREADS = 64 + 128 * PARTS;
  static constexpr int SFA_BYTES = Kb<FMT>::CHUNKS * SF, SFB_BYTES = 2 * SFA_BYTES;
  static constexpr int STAGE_BYTES = A_BYTES + B_BYTES + SFA_BYTES + SFB_BYTES;
  static constexpr int NUM_BARS = 2 * STAGES + 3;
  static constexpr int OUT_AT = STAGES * STAGE_BYTES;
  static constexpr int BARS_AT = OUT_AT + 4 * PARTS * OUT_BYTES;
  static constexpr int SMEM_BYTES = BARS_AT + 1024 + NUM_BARS * 8 + 16;
  static constexpr uint32_t SF_COLS = 12 * Kb<FMT>::CHUNKS;
};
template <int FMT, bool SHORT>
constexpr bool tile_ok() {
  using T = Tile<FMT, SHORT>;
  return SF_COL0 + T::STAGES * T::SF_COLS <= TMEM_COLS &&  // tensor memory
         T::STAGE_BYTES % 1024 == 0 &&                     // stages start on swizzle atoms
         T::SMEM_BYTES <= 227 * 1024;
}
static_assert(tile_ok<kFp4Nv, true>() && tile_ok<kFp4Nv, false>() && tile_ok<kFp4Mx, true>() &&
                  tile_ok<kFp4Mx, false>(),
              "tile sizes");

template <int FMT, int EPI, bool SHORT>
__global__ void __launch_bounds__(Tile<FMT, SHORT>::THREADS, 1)
    gemm_fp4_pair(const __grid_constant__ CUtensorMap tma_a,
                  const __grid_constant__ CUtensorMap tma_b,
                  const __grid_constant__ CUtensorMap tma_sfa,
                  const __grid_constant__ CUtensorMap tma_sfb,
                  const __grid_constant__ CUtensorMap tma_out, const Fp4GemmParams p) {
  using T = Tile<FMT, SHORT>;
  constexpr bool NV = FMT == kFp4Nv;
  constexpr int STAGES = T::STAGES, PARTS = T::PARTS, CHUNKS = T::CHUNKS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + T::BARS_AT);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + T::NUM_BARS);
  __shared__ int entry_status;
  __shared__ int loads_issued;

  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const uint32_t peer = rank ^ 1u;
  const bool leader = rank == 0;
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = smem_u32(bars);
  auto FULL = [&](int s) { return bar0 + 8u * s; };
  auto EMPTY = [&](int s) { return bar0 + 8u * (STAGES + s); };
  const uint32_t TFULL = bar0 + 8u * (2 * STAGES);       // a tile is accumulated
  const uint32_t TEMPTY = bar0 + 8u * (2 * STAGES + 1);  // it is in registers
  const uint32_t DRAIN = bar0 + 8u * (2 * STAGES + 2);

  if (threadIdx.x == 0) {
    entry_status = *reinterpret_cast<const volatile int *>(p.status);
    loads_issued = 0;
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(FULL(s), 2);  // one arrival per producer of the pair
      mbar_init(EMPTY(s), 1);
    }
    mbar_init(TFULL, 1);
    mbar_init(TEMPTY, 2 * 4 * PARTS);  // both CTAs' epilogue warps
    mbar_init(DRAIN, 1);
    fence_mbar_init();
    tma_prefetch_desc(&tma_a);
    tma_prefetch_desc(&tma_b);
    tma_prefetch_desc(&tma_sfa);
    tma_prefetch_desc(&tma_sfb);
  }
  cluster_sync();  // barriers initialised and entry status visible pair-wide
  const int peer_status =
      static_cast<int>(ld_shared_cluster_u32(map_to_cta(smem_u32(&entry_status), peer)));
  const bool skip = (entry_status | peer_status) != 0;
  if (!skip && warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync();  // the peer has read our status word; TMEM allocated in both
  if (skip) return;
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  const int num_tiles = p.tiles_m * p.tiles_n;
  const int kblocks = (p.k + BK - 1) / BK;
  const int pair_id = blockIdx.x >> 1;
  const int pairs = gridDim.x >> 1;

  if (warp == 0) {
    const uint32_t full_leader = map_to_cta(FULL(0), 0);
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;
    bool ok = true;
    for (int t = pair_id; t < num_tiles && ok; t += pairs) {
      int tm, tn;
      tile_coords(t, p.tiles_m, p.tiles_n, tm, tn);
      const int block_a = 2 * tm + static_cast<int>(rank);
      const int row_b = tn * BN + static_cast<int>(rank) * (BN / 2);
      for (int kb = 0; kb < kblocks; ++kb) {
        ok = mbar_wait_warp(EMPTY(stage), phase ^ 1, p.status);
        if (!ok) break;
        const uint32_t full = full_leader + 8u * stage;
        const uint32_t sa = sbase + stage * T::STAGE_BYTES;
        if (elect_one()) {
          // boxes count whole, also where they read past a matrix
          if (leader)
            mbar_arrive_expect_tx(FULL(stage), T::STAGE_BYTES);
          else
            mbar_arrive_expect_tx_cluster(full, T::STAGE_BYTES);
          const int sf_x = kb * (T::SFA_BYTES / 8);  // 8-byte elements
          tma_load_2d_pair(sa, &tma_a, kb * BKB, block_a * BM, full);
          tma_load_2d_pair(sa + A_BYTES, &tma_b, kb * BKB, row_b, full);
          tma_load_2d_pair(sa + A_BYTES + B_BYTES, &tma_sfa, sf_x, block_a, full);
          tma_load_2d_pair(sa + A_BYTES + B_BYTES + T::SFA_BYTES, &tma_sfb, sf_x, tn * (BN / 128),
                           full);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (lane == 0) loads_issued = issued;
  } else if (warp == 1) {
    if (leader) {
      int stage = 0;
      uint32_t phase = 0;
      uint32_t empty_phase = 1;  // the first tile waits for no epilogue
      bool ok = true;
      for (int t = pair_id; t < num_tiles && ok; t += pairs) {
        ok = mbar_wait_cluster(TEMPTY, empty_phase, p.status);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int kb = 0; kb < kblocks; ++kb) {
          ok = mbar_wait_warp(FULL(stage), phase, p.status);
          if (!ok) break;
          tc_fence_after();
          const uint32_t sa = sbase + stage * T::STAGE_BYTES;
          const uint64_t da = desc_sw128(sa, 16, 1024), db = desc_sw128(sa + A_BYTES, 16, 1024);
          const uint64_t dsf = desc_sf_copy(sa + A_BYTES + B_BYTES);
          const uint32_t sfa = tmem + SF_COL0 + T::SF_COLS * stage;
          const uint32_t sfb = sfa + 4 * Kb<FMT>::CHUNKS;
          const int groups = min(4, (p.k - kb * BK) / 64);
          if (elect_one()) {
            // descriptors count in 16 bytes; nothing here carries out of the address
#pragma unroll
            for (int c = 0; c < Kb<FMT>::CHUNKS; ++c) {
              if (c * Kb<FMT>::PER_CHUNK >= groups) break;
              tmem_cp_sf_pair(sfa + 4 * c, dsf + c * SF / 16);
              tmem_cp_sf_pair(sfb + 8 * c, dsf + (T::SFA_BYTES + c * SF) / 16);
              tmem_cp_sf_pair(sfb + 8 * c + 4, dsf + (2 * T::SFA_BYTES + c * SF) / 16);
            }
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              if (g >= groups) break;
              const int c = g / Kb<FMT>::PER_CHUNK, id = 2 * (g % Kb<FMT>::PER_CHUNK);
              umma_fp4_pair<NV>(tmem, da + 2 * g, db + 2 * g, idesc_fp4(2 * BM, BN, NV, id),
                                sfa + 4 * c, sfb + 8 * c, (kb | g) != 0 ? 1u : 0u);
            }
            umma_commit_pair(EMPTY(stage), kBothCtas);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        if (elect_one()) umma_commit_pair(TFULL, kBothCtas);
        __syncwarp();
        empty_phase ^= 1;
      }
      // Every pair MMA (and the arrivals its commits make) completes before
      // either CTA may release TMEM or exit.
      if (elect_one()) umma_commit_pair(DRAIN, kFirstCta);
      __syncwarp();
      mbar_wait(DRAIN, 0, p.status, false);
    }
  } else {
    const int sub = warp & 3;  // TMEM lane quarter this warp may access
    const int part = (warp - 2) >> 2;
    const Alpha al = tensor_alpha(p.a_scale, p.b_scale);
    Fp4Tensor to{};
    if constexpr (EPI == kEpiGeluFp4) to = fp4_tensor(FMT == kFp4Nv ? p.out_scale : nullptr);
    const uint32_t tempty = map_to_cta(TEMPTY, 0);
    const uint32_t out0 = sbase + T::OUT_AT + (warp - 2) * OUT_BYTES;
    const uint32_t lanes = tmem + (static_cast<uint32_t>(sub * 32) << 16);
    uint32_t full_phase = 0;
    for (int t = pair_id; t < num_tiles; t += pairs) {
      int tm, tn;
      tile_coords(t, p.tiles_m, p.tiles_n, tm, tn);
      const int row0 = (2 * tm + static_cast<int>(rank)) * BM + sub * 32;
      const int row = row0 + lane;
      const int col0 = tn * BN + 32 * CHUNKS * part;  // this warp's columns, by 32
      uint32_t scales = 0;                    // of an FP4 output, being gathered
      // 32 columns of the warp's rows of the residual into its box, whole lines at
      // a time (a thread's own row at a time, the warps' lines did not fit into L1)
      auto fetch = [&](int j) {
        if (EPI != kEpiGatedResidual || col0 + 32 * j >= p.n || row0 >= p.m) return;
        if (lane == 0) bulk_wait_read<0>();
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3), u = lane & 7;
          if (row0 + r < p.m)
            cp_async16(out0 + r * 128 + 16 * (u ^ (r & 7)),
                       p.resid + static_cast<size_t>(row0 + r) * p.n + col0 + 32 * j + 4 * u);
        }
      };
      auto finish = [&](int j, const uint32_t (&r)[32]) {
        const int col = col0 + 32 * j;
        if (col >= p.n || row0 >= p.m) return;  // the same for the whole warp
        const uint32_t o = out0 + lane * 128;  // 128-byte swizzle: 16-byte unit q at q ^ (row % 8)
        if constexpr (EPI == kEpiGatedResidual) {
          cp_async_wait_all();
          __syncwarp();
        }
        float v[32];
        values<EPI>(p, al, r, col, [&](int q) { return ld_shared_v4(o + 16 * (q ^ (lane & 7))); }, v);
        if constexpr (EPI == kEpiGeluFp4) {
          static_assert(CHUNKS == 4, "a box of 64 bytes a row");
          // the warp's 128 columns as one box of 64 bytes a row, and a row's scales as words
          const bool last = j == 3 || col + 32 >= p.n;
          uint32_t c[4], sb[2];
          fp4_quant32<FMT>(v, to, c, sb);
          if (j == 0) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
          }
          // 64-byte swizzle: 16-byte unit j at j ^ (row / 2 % 4)
          st_shared_v4(out0 + lane * 64 + 16 * (j ^ ((lane >> 1) & 3)), c[0], c[1], c[2], c[3]);
          constexpr int PER = 32 / Fp4<FMT>::BLOCK;  // scales of 32 columns
          scales |= (PER == 2 ? sb[0] | (sb[1] << 8) : sb[0]) << (8 * PER * (j % (4 / PER)));
          if (j % (4 / PER) == 4 / PER - 1 || last) {
            // a row that ends inside a group of four scales: the others are 0
            if (row < p.m)
              *reinterpret_cast<uint32_t *>(
                  p.out_sf + mx_sf_offset(row, (col / Fp4<FMT>::BLOCK) & ~3,
                                          (p.n / Fp4<FMT>::BLOCK + 3) / 4)) = scales;
            scales = 0;
          }
          if (last) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tma_out, col0 / 2, row0, out0);
              bulk_commit();
            }
          }
        } else if constexpr (EPI == kEpiGatedResidual) {
#pragma unroll
          for (int q = 0; q < 8; ++q)
            st_shared_v4(o + 16 * (q ^ (lane & 7)), __float_as_uint(v[4 * q]),
                         __float_as_uint(v[4 * q + 1]), __float_as_uint(v[4 * q + 2]),
                         __float_as_uint(v[4 * q + 3]));
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            tma_store_2d(&tma_out, col, row0, out0);
            bulk_commit();
          }
          if (j + 1 < CHUNKS) fetch(j + 1);
        } else {
          if ((j & 1) == 0) {
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
          }
#pragma unroll
          for (int q = 0; q < 4; ++q)
            st_shared_v4(o + 16 * ((q + 4 * (j & 1)) ^ (lane & 7)),
                         pack_bf16x2(v[8 * q], v[8 * q + 1]),
                         pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                         pack_bf16x2(v[8 * q + 4], v[8 * q + 5]),
                         pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
          // the box is whole with its second half, or where the matrix ends
          if ((j & 1) == 1 || col + 32 >= p.n) {
            fence_async_smem();
            __syncwarp();
            if (lane == 0) {
              tma_store_2d(&tma_out, col & ~63, row0, out0);
              bulk_commit();
            }
          }
        }
      };
      fetch(0);
      const bool ok = mbar_wait(TFULL, full_phase, p.status);
      if (!__all_sync(0xffffffffu, ok)) break;
      tc_fence_after();
      uint32_t r[CHUNKS][32];
#pragma unroll
      for (int j = 0; j < CHUNKS; ++j) tmem_ld32_async(lanes + 32 * (CHUNKS * part + j), r[j]);
      tmem_wait_ld(r);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader)
          mbar_arrive(TEMPTY);
        else
          mbar_arrive_cluster(tempty);
      }
#pragma unroll
      for (int j = 0; j < CHUNKS; ++j) finish(j, r[j]);
      full_phase ^= 1;
    }
    cp_async_wait_all();
    if (lane == 0) bulk_wait_all();
  }

  // Drain: every load either producer issued must land before its CTA exits.
  // A stage's FULL phase completes once both producers arrived and all bytes
  // landed; where one producer stopped early (after a failure elsewhere) the
  // first CTA arrives in its place, then waits out the last STAGES loads.
  __syncwarp();
  tc_fence_before();
  cluster_sync();
  if (leader && threadIdx.x == 0) {
    const int mine = loads_issued;
    const int theirs =
        static_cast<int>(ld_shared_cluster_u32(map_to_cta(smem_u32(&loads_issued), peer)));
    const int lo = mine < theirs ? mine : theirs;
    const int hi = mine < theirs ? theirs : mine;
    for (int i = lo; i < hi; ++i) mbar_arrive(FULL(i % STAGES));
    for (int i = hi - STAGES > 0 ? hi - STAGES : 0; i < hi; ++i)
      mbar_wait(FULL(i % STAGES), (i / STAGES) & 1, p.status, false);
  }
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
}

template <int FMT, int EPI, bool SHORT>
cudaError_t launch_tile(const Fp4GemmMaps &t, const Fp4GemmParams &p, int grid, cudaStream_t s) {
  static PerDevice smem_attr;
  using T = Tile<FMT, SHORT>;
  cudaError_t e = set_smem_once(smem_attr, gemm_fp4_pair<FMT, EPI, SHORT>, T::SMEM_BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(T::THREADS, 1, 1);
  cfg.dynamicSmemBytes = T::SMEM_BYTES;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, gemm_fp4_pair<FMT, EPI, SHORT>, t.a, t.b, t.a_sf, t.b_sf, t.out,
                            p);
}

template <int FMT, int EPI>
cudaError_t launch(const Fp4GemmMaps &t, const Fp4GemmParams &p, int grid, cudaStream_t s) {
  // an FP4 row's box is as wide as 128 columns, so these stay with eight warps
  if constexpr (EPI != kEpiGeluFp4)
    if (p.k <= short_blocks(EPI) * BK) return launch_tile<FMT, EPI, true>(t, p, grid, s);
  return launch_tile<FMT, EPI, false>(t, p, grid, s);
}
}  // namespace pair

template <int FMT, int EPI>
cudaError_t launch_epi(const Fp4GemmMaps &t, const Fp4GemmParams &p, const Fp4GemmPlan &plan,
                       cudaStream_t s) {
  return plan.pair ? pair::launch<FMT, EPI>(t, p, plan.grid, s)
                   : split::launch<FMT, EPI>(t, p, plan, s);
}

template <int FMT>
cudaError_t launch_fmt(int epi, const Fp4GemmMaps &t, const Fp4GemmParams &p,
                       const Fp4GemmPlan &plan, cudaStream_t s) {
  switch (epi) {
    case kEpiStore:
      return launch_epi<FMT, kEpiStore>(t, p, plan, s);
    case kEpiGelu:
      return launch_epi<FMT, kEpiGelu>(t, p, plan, s);
    case kEpiGatedResidual:
      return launch_epi<FMT, kEpiGatedResidual>(t, p, plan, s);
    case kEpiGeluFp4:
      return launch_epi<FMT, kEpiGeluFp4>(t, p, plan, s);
    default:
      return cudaErrorInvalidValue;
  }
}

}  // namespace

Fp4GemmPlan fp4_gemm_plan(int fmt, Fp4GemmParams *p, int num_sms) {
  Fp4GemmPlan plan{};
  p->chunks = fp4_chunks(fmt, p->k);
  const int kblocks = (p->k + BK - 1) / BK;
  const auto tiles = [&](int bm, int bn) {
    p->tiles_m = (p->m + bm - 1) / bm;
    p->tiles_n = (p->n + bn - 1) / bn;
    return static_cast<long long>(p->tiles_m) * p->tiles_n;
  };
  plan.splits = 1;
  plan.box_a = BM;
  plan.box_b = split::BN;
  static_assert(split::BN == pair::BN / 2, "one box of W for both");
  // 128 x 128 tiles where there is a multiprocessor for each (or no second block
  // of rows): 512 x 2048 x 4096 9.4 against 12.2 us on pairs, 2304 x 768 x 768 6.4
  // against 8.2. With two on some, pairs win: 2048 x 2048 x 8192 18.0 against 20.0.
  const long long small = tiles(BM, split::BN);
  plan.pair = p->m > BM && small > num_sms;
  if (plan.pair) {
    const long long t = tiles(2 * BM, pair::BN);
    plan.grid = 2 * static_cast<int>(t < num_sms / 2 ? t : num_sms / 2);
    return plan;
  }
  if (p->m < BM) plan.box_a = (p->m + 7) / 8 * 8;  // no rows that are not there
  // k shared by as many CTAs as have a multiprocessor, where that saves more than
  // joining the parts costs. A k-block takes a CTA about 0.28 us; the join 2 us and
  // 3.5 for 128 rows: 1 x 5376 x 14336 19.6 us in one part, 11.3 in three; 512 x
  // 1024 x 14336 20.2 and 14.0 in four; 128 x 5376 x 5376 11.4 and 12.0 in three.
  int parts = static_cast<int>(num_sms / small);
  if (parts > split::MAX_SPLIT) parts = split::MAX_SPLIT;
  if (parts > kblocks / 2) parts = kblocks / 2;
  const int rows = p->m < BM ? p->m : BM;
  if (parts > 1 && 0.28 * (kblocks - kblocks / parts) > 2.0 + 3.5 * rows / BM) plan.splits = parts;
  plan.grid = static_cast<int>(small * plan.splits);
  return plan;
}

cudaError_t launch_gemm_fp4(int fmt, int epilogue, const Fp4GemmMaps &t, const Fp4GemmParams &p,
                            const Fp4GemmPlan &plan, cudaStream_t s) {
  return fmt == kFp4Mx ? launch_fmt<kFp4Mx>(epilogue, t, p, plan, s)
                       : launch_fmt<kFp4Nv>(epilogue, t, p, plan, s);
}

}  // namespace h3
