// ep_small.cuh -- the epilogue and expert matmuls for a few rows per expert (warp MMA).
//
// Item: an expert's chunk of up to 8 T rows x 16 RH weight rows, the whole of K.  KS warps of
// a CTA share an item, taking its units of 128 k in turn; their f32 sums meet in shared
// memory, are added in warp order and go through the epilogue.
//
// Both operands come straight from global memory into registers: weights (read once, so kept
// out of L1) two or more units ahead, activations (read by every warp, so from L1) when they
// are needed.  Lane (g, c) of mma.sync m16n8k16 takes weight rows g, g + 8, ... and, in each
// 32-byte sector of a row, bytes [8c, 8c + 8); the codes in there and the activations they
// meet are the same k for every row, so no data is moved between lanes.
//
// A word of codes becomes bf16 pairs of whole numbers: one lop3 sets an exponent over a field
// (base + q), one subtraction takes off the base and the centre, q - 1 (ternary) or q - 8
// (4-bit).  Products with bf16 activations are exact; per 128 (64) weights the f32 sum is
// scaled, and 4-bit adds the zero point by the sum of the activations (an MMA with ones):
//   ternary  acc += d * sum (q - 1) x
//   4-bit    acc += s * (sum (q - 8) x - (z - 8) sum x)
#pragma once

#include "common.cuh"
#include "ep_tc.cuh"
#include "epilogue.cuh"
#include "gemv_stream.cuh"

namespace tgemm {

constexpr int kEsWarps = 8;
constexpr int kEsPitch = 36;  // floats per token row of a warp's sums: no bank conflicts

struct EsParams {
  int N, K, E, R, x_rows;
  int U;                  // units of 128 k
  int KS;                 // warps per item: 1, 2, 4 or 8
  int tiles_n;            // row blocks
  const uint16_t* x;
  const uint8_t* wq;
  const uint16_t* scales;
  const int* offsets;
  const int* rows;
  EpArgs ep;
};

__host__ __device__ constexpr int es_smem_bytes(int T, bool grouped) {
  return kEsWarps * 8 * T * kEsPitch * 4 + (grouped ? 2 * (kEtMaxExperts + 2) * 4 : 0);
}

__device__ __forceinline__ uint2 ld_stream_v2(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

__device__ __forceinline__ uint32_t bsub2_u32(uint32_t a, uint32_t b) {
  __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

// A lane's share of one unit of 16 RH weight rows: its codes of rows g + 8 j, and the scales
// of row (lane % (8 * 2 RH)) (Q2: d; 4-bit: the (s, z) pairs of the unit's two groups).
template <int FMT, int RH>
struct EsUnit {
  static constexpr int kW = FMT == 0 ? 2 : 4;  // 32-bit words of codes per row
  uint32_t w[2 * RH][kW];
  uint32_t sc[FMT == 0 ? 1 : 2];
};

template <int FMT, int T, int RH>
__global__ void __launch_bounds__(kEsWarps * 32, 2) ep_small_kernel(const EsParams p) {
  constexpr int kTok = 8 * T, kRows = 16 * RH, kJ = 2 * RH;
  constexpr int kUnitBytes = FMT == 0 ? 32 : 64;
  constexpr int kD = FMT == 0 ? 3 : 2;  // units in flight ahead
  using Unit = EsUnit<FMT, RH>;
  extern __shared__ __align__(16) float es_red[];  // [warp][token][kEsPitch]
  int* tab_off = reinterpret_cast<int*>(es_red + kEsWarps * kTok * kEsPitch);
  int* tab_tp = tab_off + kEtMaxExperts + 2;
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
  const int KS = p.KS, grp = warp / KS, wk = warp - grp * KS;
  const int groups = kEsWarps / KS, stride = gridDim.x * groups;
  const int row_bytes = FMT == 0 ? p.K / 4 : p.K / 2;
  const int nscale = FMT == 0 ? p.K / 128 : p.K / 64;

  pdl_trigger();
  int num_items;
  if (p.offsets) {
    pdl_wait();
    if (warp == 0) et_build_table(p.offsets, p.E, p.R, kTok, tab_off, tab_tp);
    __syncthreads();
    num_items = tab_tp[p.E] * p.tiles_n;
  } else {
    num_items = (p.R + kTok - 1) / kTok * p.tiles_n;
  }
  // item t: expert, first weight row, first row, rows
  auto item_at = [&](int t, int& e, int& n0, int& m0, int& mt) {
    int tt = 0, r = t, lo = 0, hi = p.R;
    e = 0;
    if (p.offsets) {
      e = et_find(tab_tp, p.E, t / p.tiles_n);
      tt = tab_tp[e + 1] - tab_tp[e];
      r = t - tab_tp[e] * p.tiles_n;
      lo = tab_off[e];
      hi = tab_off[e + 1];
    } else {
      tt = (p.R + kTok - 1) / kTok;
    }
    const int tn = r / tt, ti = r - tn * tt;
    n0 = tn * kRows;
    m0 = lo + ti * kTok;
    mt = min(kTok, hi - m0);
  };

  // ---- the loads run kD units ahead of the products
  int lt = blockIdx.x * groups + grp, lu = wk;  // next unit to load
  const uint8_t* lbase = nullptr;
  const uint16_t* sbase = nullptr;
  uint32_t loff[kJ];
  auto load_item = [&]() {
    if (lt >= num_items) return;
    int e, n0, m0, mt;
    item_at(lt, e, n0, m0, mt);
    lbase = p.wq + (static_cast<int64_t>(e) * p.N + n0) * row_bytes + 8 * c;
    // rows past N read row N - 1 (their sums are not stored)
#pragma unroll
    for (int j = 0; j < kJ; ++j) loff[j] = static_cast<uint32_t>(min(g + 8 * j, p.N - 1 - n0)) * row_bytes;
    const int srow = min(g + 8 * (c % kJ), p.N - 1 - n0);
    sbase = p.scales + (static_cast<int64_t>(e) * p.N + n0 + srow) * nscale * (FMT == 0 ? 1 : 2);
  };
  auto load_unit = [&](Unit& b) {
    if (lt >= num_items) return;
    const uint8_t* src = lbase + static_cast<int64_t>(lu) * kUnitBytes;
    const bool second = FMT == 1 && 2 * lu + 1 < nscale;  // K may end on half a unit
#pragma unroll
    for (int j = 0; j < kJ; ++j) {
      const uint2 a = ld_stream_v2(src + loff[j]);
      b.w[j][0] = a.x;
      b.w[j][1] = a.y;
      if (FMT == 1) {
        const uint2 h = second ? ld_stream_v2(src + loff[j] + 32) : make_uint2(0u, 0u);
        b.w[j][Unit::kW - 2] = h.x;
        b.w[j][Unit::kW - 1] = h.y;
      }
    }
    if (FMT == 0) {
      b.sc[0] = __ldg(sbase + lu);
    } else {
      const uint32_t* sp = reinterpret_cast<const uint32_t*>(sbase) + 2 * lu;
      b.sc[0] = __ldg(sp);
      b.sc[FMT] = second ? __ldg(sp + 1) : 0u;
    }
    lu += KS;
    if (lu >= p.U) {
      lu = wk;
      lt += stride;
      load_item();
    }
  };
  Unit buf[kD];
  load_item();
#pragma unroll
  for (int d = 0; d < kD; ++d) load_unit(buf[d]);
  if (!p.offsets) pdl_wait();

  float* red = es_red + static_cast<size_t>(warp) * kTok * kEsPitch;
  const float* red_grp = es_red + static_cast<size_t>(grp) * KS * kTok * kEsPitch;
  for (int t = blockIdx.x * groups + grp; t < num_items; t += stride) {
    int e, n0, m0, mt;
    item_at(t, e, n0, m0, mt);
    // the lane's token rows: row g + 8 t of the chunk (past its end: its last), elements of
    // the lane's 64 (Q2) or 2 x 32 (4-bit) bytes of a unit
    const uint16_t* xp[T];
    bool xok[T];
#pragma unroll
    for (int i = 0; i < T; ++i) {
      int64_t m = m0 + min(g + 8 * i, mt - 1);
      if (p.rows) m = __ldg(p.rows + m);
      xok[i] = m >= 0 && m < p.x_rows;  // else a row of zeros
      xp[i] = p.x + (xok[i] ? m : 0) * p.K + (FMT == 0 ? 32 : 16) * c;
    }
    float acc[RH][T][4];
#pragma unroll
    for (int h = 0; h < RH; ++h)
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[h][i][k] = 0.f;

    for (int u = wk; u < p.U; u += KS) {
      const Unit cur = buf[0];
#pragma unroll
      for (int d = 0; d + 1 < kD; ++d) buf[d] = buf[d + 1];
      load_unit(buf[kD - 1]);
      // FMT 0: two half units (words) under one scale; FMT 1: two groups with their own
      float pacc[RH][T][4];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (FMT == 1 && 2 * u + hf >= nscale) break;
        if (FMT == 1 || hf == 0) {
#pragma unroll
          for (int h = 0; h < RH; ++h)
#pragma unroll
            for (int i = 0; i < T; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k) pacc[h][i][k] = 0.f;
        }
        float xsum[T][4];
        uint32_t a[kJ][8];  // bf16 pairs of 16 codes per row
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          if (FMT == 0) {
            gs_q2_pairs(cur.w[j][hf], a[j]);
            constexpr uint32_t kOne[3] = {0x43014301u, 0x42044204u, 0x41104110u};  // 129, 33, 9
#pragma unroll
            for (int i = 0; i < 8; ++i) a[j][i] = bsub2_u32(a[j][i], kOne[i % 3]);
          } else {
#pragma unroll
            for (int wd = 0; wd < 2; ++wd)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                a[j][4 * wd + i] =
                    bsub2_u32(lop3_and_or(cur.w[j][(2 * hf + wd) % Unit::kW] >> (4 * i), 0x000F000Fu, 0x43004300u),
                              0x43084308u);  // 136
          }
        }
#pragma unroll
        for (int i = 0; i < T; ++i) {
          // 16 activations of token g + 8 i: x[0..15] as 8 pairs of neighbours
          const uint4* xs = reinterpret_cast<const uint4*>(xp[i] + u * 128 + (FMT == 0 ? 16 : 64) * hf);
          uint4 r0 = __ldg(xs), r1 = __ldg(xs + 1);
          if (!xok[i]) r0 = r1 = make_uint4(0u, 0u, 0u, 0u);
          const uint32_t r[8] = {r0.x, r0.y, r0.z, r0.w, r1.x, r1.y, r1.z, r1.w};
          uint32_t b[8];  // b[k] meets the code pair k: codes (i, i + 8), or (i, i + 4) of each word
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int lo = FMT == 0 ? k / 2 : 4 * (k / 4) + (k & 3) / 2;
            b[k] = prmt(r[lo], r[lo + (FMT == 0 ? 4 : 2)], (k & 1) ? 0x7632u : 0x5410u);
          }
          if (FMT == 1) {
#pragma unroll
            for (int k = 0; k < 4; ++k) xsum[i][k] = 0.f;
          }
#pragma unroll
          for (int s = 0; s < 4; ++s) {
#pragma unroll
            for (int h = 0; h < RH; ++h) {
              const uint32_t af[4] = {a[2 * h][2 * s], a[2 * h + 1][2 * s], a[2 * h][2 * s + 1], a[2 * h + 1][2 * s + 1]};
              mma_bf16_16816(pacc[h][i], af, b[2 * s], b[2 * s + 1]);
            }
            if (FMT == 1) {
              const uint32_t ones[4] = {0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u};
              mma_bf16_16816(xsum[i], ones, b[2 * s], b[2 * s + 1]);
            }
          }
        }
        if (FMT == 0 && hf == 0) continue;
        // scale: rows g + 8 j; the lane with c = j (mod kJ) of this g holds row j's
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          const uint32_t sv = __shfl_sync(0xFFFFFFFFu, cur.sc[FMT == 0 ? 0 : hf], 4 * g + j);
          const float s = __half2float(__ushort_as_half(static_cast<uint16_t>(sv & 0xFFFFu)));
          const int h = j >> 1, k0 = 2 * (j & 1);
          if (FMT == 0) {
#pragma unroll
            for (int i = 0; i < T; ++i) {
              acc[h][i][k0] = fmaf(s, pacc[h][i][k0], acc[h][i][k0]);
              acc[h][i][k0 + 1] = fmaf(s, pacc[h][i][k0 + 1], acc[h][i][k0 + 1]);
            }
          } else {
            const float z = __half2float(__ushort_as_half(static_cast<uint16_t>(sv >> 16))) - 8.f;
#pragma unroll
            for (int i = 0; i < T; ++i) {
              acc[h][i][k0] = fmaf(s, fmaf(-z, xsum[i][0], pacc[h][i][k0]), acc[h][i][k0]);
              acc[h][i][k0 + 1] = fmaf(s, fmaf(-z, xsum[i][1], pacc[h][i][k0 + 1]), acc[h][i][k0 + 1]);
            }
          }
        }
      }
    }
    // ---- sums of the KS warps -> epilogue.  acc[h][i][k]: weight row 16 h + g (+ 8 for
    // k >= 2), token 8 i + 2 c + (k & 1)
#pragma unroll
    for (int h = 0; h < RH; ++h)
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          red[(8 * i + 2 * c + (k & 1)) * kEsPitch + 16 * h + g + 8 * (k >> 1)] = acc[h][i][k];
    if (KS == 1)
      __syncwarp();
    else
      named_barrier_sync(1 + grp, 32 * KS);
    {
      constexpr int kPer = 32 / kRows;  // tokens a warp stores at once
      const int nn = lane % kRows, n = n0 + nn;
      float bias = 0.f;
      if (p.ep.bias && n < p.N) bias = ep_load(p.ep.bias, static_cast<int64_t>(e) * p.N + n, p.ep.bias_f32);
      for (int m = wk * kPer + lane / kRows; m < mt; m += KS * kPer) {
        if (n >= p.N) continue;
        float v[1] = {0.f};
        for (int w = 0; w < KS; ++w) v[0] += red_grp[(w * kTok + m) * kEsPitch + nn];
        v[0] += bias;
        ep_act_all(v, p.ep.act);
        ep_store1(p.ep, m0 + m, n, p.N, v[0]);
      }
    }
    if (KS == 1)
      __syncwarp();
    else
      named_barrier_sync(1 + grp, 32 * KS);
  }
}

}  // namespace tgemm
