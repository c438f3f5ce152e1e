// ep_tc.cuh -- tensor-core kernel of the epilogue and expert matmuls:
//   y[m] = residual[m] + gate[m] * act(x[m] W_e^T + bias_e),   rows m of expert e
// with W packed (ternary or 4-bit).  A dense call is one expert that owns every row.
//
// Tile: 128 weight rows (MMA M) x up to 128 tokens (MMA N, in steps of 16), 128 k per stage,
// A (the dequantized weights) in tensor memory, B (the activations, an f16 copy in the
// dequantizers' k order) in shared memory, f32 accumulators in tensor memory.
#pragma once

#include "common.cuh"
#include "epilogue.cuh"
#include "gemm_tc.cuh"
#include "prep.cuh"

namespace tgemm {

constexpr int kEtRows = 128;
constexpr int kEtTok = 128;
constexpr int kEtBK = 128;
constexpr int kEtStages = 4;
constexpr int kEtGroups = 2;                    // dequant groups of 4 warps, stages in turn
constexpr int kEtDeqWarp0 = 2;
constexpr int kEtEpiWarp0 = kEtDeqWarp0 + 4 * kEtGroups;
constexpr int kEtWProdWarp = kEtEpiWarp0 + 8;
constexpr int kEtThreads = (kEtWProdWarp + 1) * 32;
constexpr int kEtXBox = kEtTok * 128;           // 128 tokens x 64 k of f16
constexpr int kEtXBytes = 2 * kEtXBox;
constexpr int kEtMaxExperts = 1024;
constexpr int kEtBoxPitch = kEtRows + 4;        // floats per token row of an output box
constexpr int kEtBoxFloats = 16 * kEtBoxPitch;

template <int FMT>
struct EtFmt {
  static constexpr int kWqRowBytes = FMT == 0 ? 32 : 64;
  static constexpr int kWStages = FMT == 0 ? 8 : 6;
  static constexpr int kWBytes = kEtRows * kWqRowBytes;
  static constexpr int kXOff = 0;
  static constexpr int kWOff = kEtStages * kEtXBytes;
  static constexpr int kBoxOff = kWOff + kWStages * kWBytes;
  static constexpr int kTabOff = kBoxOff + 4 * kEtBoxFloats * 4;
  static constexpr int kBarOff = kTabOff + 2 * (kEtMaxExperts + 2) * 4;
  static constexpr int kNumBars = 2 * kEtStages + 2 * kWStages + 4 + 1 + 4;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

struct EtParams {
  int N, K, E, R;
  int nt;                 // tokens per tile, a multiple of 16
  int tiles_n;            // ceil(N / 128)
  int ksteps;             // units per tile: ceil(K / 128), twice that with the low parts
  const int* offsets;     // [E + 1] row ranges, or null: one expert, rows [0, R)
  const uint16_t* scales;
  EpArgs ep;
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Row ranges and token-tile counts of the experts, in shared memory: off[e], off[e + 1]
// bound expert e's rows, tp[e] is the number of token tiles before it.
struct EtTable {
  const int* off;
  const int* tp;
};
struct EtTile {
  int e, n0, m0, mt;  // expert, first weight row, first token row, tokens
};
// The expert with token tile tt: the largest e with tp[e] <= tt (and so tt < tp[e + 1]).
__device__ __forceinline__ int et_find(const int* tp, int E, int tt) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (tp[mid] <= tt)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}
// Tile t of the walk (e is the walk's position, looked up again once t leaves that expert).
__device__ __forceinline__ EtTile et_tile(const EtParams& p, const EtTable& tb, int t, int& e) {
  if (t >= tb.tp[e + 1] * p.tiles_n) e = et_find(tb.tp, p.E, t / p.tiles_n);
  const int tt = tb.tp[e + 1] - tb.tp[e];
  const int r = t - tb.tp[e] * p.tiles_n;
  const int tn = r / tt, ti = r - tn * tt;
  EtTile x;
  x.e = e;
  x.n0 = tn * kEtRows;
  x.m0 = tb.off[e] + ti * p.nt;
  x.mt = min(p.nt, tb.off[e + 1] - x.m0);
  return x;
}

// Group offsets come from the device and are not trusted: each is clamped to [previous, R],
// so that every row range lies inside the caller's buffers.
__device__ __forceinline__ void et_build_table(const int* offsets, int E, int R, int nt, int* off, int* tp) {
  const int lane = threadIdx.x & 31;
  if (!offsets) {
    if (lane == 0) {
      off[0] = 0;
      off[1] = R;
      tp[0] = 0;
      tp[1] = (R + nt - 1) / nt;
    }
    return;
  }
  int tiles = 0;
  int run = min(max(__ldg(offsets), 0), R);
  if (lane == 0) {
    off[0] = run;
    tp[0] = 0;
  }
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    int v = e < E ? min(max(__ldg(offsets + e + 1), 0), R) : 0;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, v, s);
      if (lane >= s) v = max(v, o);
    }
    v = max(v, run);
    int prev = __shfl_up_sync(0xFFFFFFFFu, v, 1);
    if (lane == 0) prev = run;
    int c = (v - prev + nt - 1) / nt;
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, c, s);
      if (lane >= s) c += o;
    }
    c += tiles;
    if (e < E) {
      off[e + 1] = v;
      tp[e + 1] = c;
    }
    run = __shfl_sync(0xFFFFFFFFu, v, 31);
    tiles = __shfl_sync(0xFFFFFFFFu, c, 31);
  }
}

// 4-bit codes as an f16 pair: the high part f16(w) or the low part f16(w - f16(w)) of
// w = (q - z) s in f32.  Pairs as q4_word_to_f16.
template <bool LOW>
__device__ __forceinline__ void q4_word_split(uint32_t w, float s, float z, uint32_t* o) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = (static_cast<float>((w >> (4 * i)) & 15u) - z) * s;
    const float b = (static_cast<float>((w >> (4 * i + 16)) & 15u) - z) * s;
    const uint32_t h = pack_f16x2(a, b);
    if (LOW) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
      o[i] = pack_f16x2(a - f.x, b - f.y);
    } else {
      o[i] = h;
    }
  }
}

// SPLIT (4-bit weights, f32 y): every 128-k stage runs twice, with the weights' high and low
// f16 parts, since f16 weights alone are 2^-12 relative off.
//
// SUMS (f32 y): the tensor core adds each K = 16 step to the f32 accumulator with truncation,
// 1.5e-8 of the sum per step towards zero (2.3e-6 at K = 2560), so after every kSeg units the
// accumulator goes into a running sum in tensor memory, rounded to nearest.  That leaves room
// for two A stages instead of four.
constexpr int kEtSumCol0 = 2 * kEtTok;
template <int FMT, bool SPLIT, bool SUMS>
__global__ void __launch_bounds__(kEtThreads, 1)
    ep_tc_kernel(const __grid_constant__ CUtensorMap tm_x128,
                 const __grid_constant__ CUtensorMap tm_x16,
                 const __grid_constant__ CUtensorMap tm_w, const EtParams p) {
  using F = EtFmt<FMT>;
  constexpr int kA = SUMS ? 2 : 4;                                 // A stages
  constexpr int kACol0 = SUMS ? kEtSumCol0 + kEtTok : 2 * kEtTok;  // their columns
  static_assert(kACol0 + 64 * kA <= 512, "TMEM budget");
  constexpr int kSeg = 4;
  extern __shared__ uint8_t et_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(et_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + F::kBarOff;
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kEtStages + s); };
  auto wfull_bar = [&](int w) { return bar0 + 8u * (2 * kEtStages + w); };
  auto wempty_bar = [&](int w) { return bar0 + 8u * (2 * kEtStages + F::kWStages + w); };
  auto accfull_bar = [&](int a) { return bar0 + 8u * (2 * kEtStages + 2 * F::kWStages + a); };
  auto accempty_bar = [&](int a) { return bar0 + 8u * (2 * kEtStages + 2 * F::kWStages + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kEtStages + 2 * F::kWStages + 4);
  // output boxes: two per set of 4 epilogue warps
  auto box_bar = [&](int h, int b) { return bar0 + 8u * (2 * kEtStages + 2 * F::kWStages + 5 + 2 * h + b); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + F::kMiscOff);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + F::kMiscOff + 4);
  int* tab_off = reinterpret_cast<int*>(smem + F::kTabOff);
  int* tab_tp = tab_off + kEtMaxExperts + 2;

  // warp index as a warp-uniform value, so that the single-thread roles below issue from
  // uniform registers
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kEtStages; ++s) {
      mbar_init(full_bar(s), 1 + 4);  // the producer's expect_tx + a dequant group
      mbar_init(empty_bar(s), 1);     // MMA commit
    }
    for (int w = 0; w < F::kWStages; ++w) {
      mbar_init(wfull_bar(w), 1);
      mbar_init(wempty_bar(w), 4);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accfull_bar(a), 1);
      mbar_init(accempty_bar(a), 8);
      for (int b = 0; b < 2; ++b) mbar_init(box_bar(a, b), 4);
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm_x128);
    tma_prefetch_desc(&tm_x16);
    tma_prefetch_desc(&tm_w);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_trigger();
  // With device offsets every role needs them first; a dense call's weights are read early,
  // and only the activation producer and the epilogue wait.
  if (p.offsets || warp == 0 || (warp >= kEtEpiWarp0 && warp < kEtWProdWarp)) pdl_wait();
  if (warp == kEtWProdWarp) et_build_table(p.offsets, p.E, p.R, p.nt, tab_off, tab_tp);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const EtTable tb{tab_off, tab_tp};
  const int num_tiles = tab_tp[p.E] * p.tiles_n;
  const int ksteps = p.ksteps;

  if (warp == 0) {
    // ------------------------------------------------------------ activation producer
    if (elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      int e = 0;
      for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        const EtTile tl = et_tile(p, tb, t, e);
        const int nb = (tl.mt + 15) >> 4;  // boxes of 16 tokens
        for (int u = 0; u < ksteps; ++u, ++it) {
          const uint32_t s = it % kEtStages, ph = (it / kEtStages) & 1u;
          if (!mbar_wait(empty_bar(s), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t dst = sbase + F::kXOff + s * kEtXBytes;
          const int k0 = (SPLIT ? u >> 1 : u) * kEtBK;
          mbar_arrive_expect_tx(full_bar(s), nb * 4096u);
          if (nb == kEtTok / 16) {
            tma_load_2d(dst, &tm_x128, full_bar(s), k0, tl.m0);
            tma_load_2d(dst + kEtXBox, &tm_x128, full_bar(s), k0 + 64, tl.m0);
          } else {
            for (int j = 0; j < nb; ++j) {
              tma_load_2d(dst + 2048 * j, &tm_x16, full_bar(s), k0, tl.m0 + 16 * j);
              tma_load_2d(dst + kEtXBox + 2048 * j, &tm_x16, full_bar(s), k0 + 64, tl.m0 + 16 * j);
            }
          }
        }
      }
      // every load issued must land before the CTA may exit
      for (uint32_t j = (it > kEtStages ? it - kEtStages : 0); j < it; ++j)
        mbar_wait_drain(full_bar(j % kEtStages), (j / kEtStages) & 1u);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMA issuer
    if (elect_one()) {
      uint32_t it = 0, sc = 0;  // units, accumulator segments
      bool ok = true;
      int e = 0;
      for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        const EtTile tl = et_tile(p, tb, t, e);
        const uint32_t idesc = make_idesc_f16(0u, kEtRows, static_cast<uint32_t>((tl.mt + 15) & ~15));
        for (int u0 = 0; ok && u0 < ksteps; u0 += kSeg, ++sc) {
          const int u1 = SUMS ? min(u0 + kSeg, ksteps) : ksteps;
          const uint32_t a = sc & 1u;
          if (!mbar_wait(accempty_bar(a), ((sc >> 1) & 1u) ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + a * kEtTok;
          for (int u = u0; u < u1; ++u, ++it) {
            const uint32_t s = it % kEtStages, ph = (it / kEtStages) & 1u;
            if (!mbar_wait(full_bar(s), ph, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_tmem = tmem_base + kACol0 + (it % kA) * 64;
            const uint64_t b0 = smem_desc_sw128(sbase + F::kXOff + s * kEtXBytes);
            const uint64_t b1 = smem_desc_sw128(sbase + F::kXOff + s * kEtXBytes + kEtXBox);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_f16_ts(d_tmem, a_tmem + 8u * kk, (kk < 4 ? b0 : b1) + 2u * (kk & 3), idesc,
                         (u > u0 || kk > 0) ? 1u : 0u);
            mma_commit(empty_bar(s));
          }
          if (!ok) break;
          mma_commit(accfull_bar(a));
          if (!SUMS) {
            ++sc;
            break;
          }
        }
      }
      mma_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0u);
    }
  } else if (warp < kEtEpiWarp0) {
    // ------------------------------------------------------------ dequantizers
    const int q = warp & 3;                        // TMEM lane quarter
    const int grp = (warp - kEtDeqWarp0) >> 2;     // which stages: it % kEtGroups == grp
    const int rt = 32 * q + lane;                  // weight row within the tile
    const int nscale = FMT == 0 ? p.K / 128 : p.K / 64;
    const uint32_t a_lane = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + kACol0;
    const uint32_t w_mine = sbase + F::kWOff + rt * F::kWqRowBytes;
    // 16-byte chunk c of the row sits at chunk c ^ swz (TMA's 32- or 64-byte swizzle)
    const uint32_t swz = FMT == 0 ? (rt >> 2) & 1 : (rt >> 1) & 3;
    bool ok = true;
    uint32_t it = 0;  // units before this tile
    int e = 0;
    for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x, it += ksteps) {
      const EtTile tl = et_tile(p, tb, t, e);
      const int n = tl.n0 + rt;
      const bool valid = n < p.N;
      const uint16_t* srow = p.scales + (static_cast<int64_t>(tl.e) * p.N + (valid ? n : 0)) * nscale * (FMT == 0 ? 1 : 2);
      int u = static_cast<int>((grp + kEtGroups - it % kEtGroups) % kEtGroups);
      // scales of one unit: Q2 d, 4-bit the (s, z) pairs of its two groups
      auto scales_of = [&](int uu, uint32_t (&sc)[2]) {
        const int ks = SPLIT ? uu >> 1 : uu;
        sc[0] = sc[1] = 0u;
        if (!valid || uu >= ksteps) return;
        if (FMT == 0) {
          sc[0] = __ldg(srow + ks);
        } else {
          const uint32_t* sp = reinterpret_cast<const uint32_t*>(srow) + 2 * ks;
          sc[0] = __ldg(sp);
          if (2 * ks + 1 < nscale) sc[1] = __ldg(sp + 1);
        }
      };
      uint32_t sc_next[2];
      scales_of(u, sc_next);
      for (; u < ksteps; u += kEtGroups) {
        const uint32_t i = it + u;
        uint32_t sc[2] = {sc_next[0], sc_next[1]};
        scales_of(u + kEtGroups, sc_next);
        const uint32_t w = i % F::kWStages, wph = (i / F::kWStages) & 1u;
        if (!mbar_wait_warp(wfull_bar(w), wph, abort_flag)) {
          ok = false;
          break;
        }
        constexpr int kWords = F::kWqRowBytes / 4;
        uint32_t cw[kWords];
#pragma unroll
        for (int c = 0; c < kWords / 4; ++c) {
          const uint4 v = ld_shared_v4(w_mine + w * F::kWBytes + ((c ^ swz) << 4));
          cw[4 * c] = v.x;
          cw[4 * c + 1] = v.y;
          cw[4 * c + 2] = v.z;
          cw[4 * c + 3] = v.w;
        }
        // the slot is refilled by TMA (the async proxy) once the group has released it
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(wempty_bar(w));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t o[32];
          if (FMT == 0) {
            const uint32_t d2 = sc[0] | (sc[0] << 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) q2_word_to_f16(cw[4 * h + j], d2, o + 8 * j);
          } else if (!SPLIT) {
            const uint32_t s2 = (sc[h] & 0xFFFFu) | (sc[h] << 16);
            const uint32_t z2 = (sc[h] >> 16) | (sc[h] & 0xFFFF0000u);
#pragma unroll
            for (int j = 0; j < 8; ++j) q4_word_to_f16(cw[(8 * h + j) % kWords], s2, z2, o + 4 * j);
          } else {
            const float sf = __half2float(__ushort_as_half(static_cast<uint16_t>(sc[h] & 0xFFFFu)));
            const float zf = __half2float(__ushort_as_half(static_cast<uint16_t>(sc[h] >> 16)));
            if (u & 1) {
#pragma unroll
              for (int j = 0; j < 8; ++j) q4_word_split<true>(cw[(8 * h + j) % kWords], sf, zf, o + 4 * j);
            } else {
#pragma unroll
              for (int j = 0; j < 8; ++j) q4_word_split<false>(cw[(8 * h + j) % kWords], sf, zf, o + 4 * j);
            }
          }
          if (h == 0) {
            // the A stage is free once unit i - kA, which had it before, is multiplied
            const uint32_t j = i - kA;
            if (i >= kA && !mbar_wait_warp(empty_bar(j % kEtStages), (j / kEtStages) & 1u, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
          }
          tmem_st_32x32b_x32(a_lane + (i % kA) * 64 + 32 * h, o);
        }
        if (!ok) break;
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(full_bar(i % kEtStages));
      }
    }
  } else if (warp < kEtWProdWarp) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;                      // TMEM lane quarter
    const int set = (warp - kEtEpiWarp0) >> 2;   // 16-token chunks of this parity
    const EpArgs& a = p.ep;
    const bool vec = (p.N & 3) == 0;             // 4 outputs at a time stay aligned
    float* boxes = reinterpret_cast<float*>(smem + F::kBoxOff) + 2 * set * kEtBoxFloats;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    uint32_t sc = 0, bc = 0;  // segments done, boxes filled by this set
    bool ok = true;
    int e = 0;
    auto release = [&](uint32_t ab) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(accempty_bar(ab));
    };
    for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
      const EtTile tl = et_tile(p, tb, t, e);
      const int n = tl.n0 + 32 * q + lane;       // this thread's weight row
      const int n4 = tl.n0 + 4 * lane;           // its 4 rows in the copy-out
      float bias = 0.f;
      if (a.bias && n < p.N) bias = ep_load(a.bias, static_cast<int64_t>(tl.e) * p.N + n, a.bias_f32);
      uint2 gate_n = make_uint2(0u, 0u);
      if (vec && a.gate && !a.gate_rows && n4 < p.N) gate_n = *reinterpret_cast<const uint2*>(a.gate + n4);
      const int chunks = (tl.mt + 15) >> 4;
      // running sum += a segment, in f32 rounded to nearest
      for (int u = kSeg; SUMS && ok && u < ksteps; u += kSeg, ++sc) {
        const uint32_t ab = sc & 1u;
        if (!mbar_wait_warp(accfull_bar(ab), (sc >> 1) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int cc = set; cc < chunks; cc += 2) {
          uint32_t v[16], w[16];
          tmem_ld_32x32b_x16(t_lane + ab * kEtTok + 16 * cc, v);
          if (u > kSeg) tmem_ld_32x32b_x16(t_lane + kEtSumCol0 + 16 * cc, w);
          tmem_wait_ld();
          if (u > kSeg) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
          }
          tmem_st_32x32b_x16(t_lane + kEtSumCol0 + 16 * cc, v);
        }
        tmem_wait_st();
        release(ab);
      }
      if (!ok) break;
      const uint32_t ab = sc & 1u;
      if (!mbar_wait_warp(accfull_bar(ab), (sc >> 1) & 1u, abort_flag)) {
        ok = false;
        break;
      }
      ++sc;
      tc_fence_after();
      if (set >= chunks) release(ab);
      for (int cc = set; cc < chunks; cc += 2, ++bc) {
        const int m0 = tl.m0 + 16 * cc + 4 * q;  // this warp's 4 tokens in the copy-out
        const int mt = min(4, tl.mt - 16 * cc - 4 * q);
        const int64_t i0 = static_cast<int64_t>(m0) * p.N + n4;
        EpOperands4 in[4];
        if (vec && n4 < p.N) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i < mt) ep_fetch4(a, i0 + static_cast<int64_t>(i) * p.N, in[i]);
        }
        uint32_t v[16];
        tmem_ld_32x32b_x16(t_lane + ab * kEtTok + 16 * cc, v);
        float f[16];
        if (SUMS && ksteps > kSeg) {
          uint32_t w[16];
          tmem_ld_32x32b_x16(t_lane + kEtSumCol0 + 16 * cc, w);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(w[i]) + __uint_as_float(v[i]);
        } else {
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]);
        }
        if (cc + 2 >= chunks) release(ab);  // the accumulator is read out
#pragma unroll
        for (int i = 0; i < 16; ++i) f[i] += bias;
        ep_act_all(f, a.act);
        float* box = boxes + (bc & 1u) * kEtBoxFloats;
#pragma unroll
        for (int i = 0; i < 16; ++i) box[i * kEtBoxPitch + 32 * q + lane] = f[i];
        __syncwarp();
        if (lane == 0) mbar_arrive(box_bar(set, bc & 1u));
        if (!mbar_wait_warp(box_bar(set, bc & 1u), (bc >> 1) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        // this warp's 4 tokens of the chunk, 128 weight rows each.  With two boxes one
        // meeting per chunk is enough: a box is written again only after every warp has
        // come to the next meeting, and so has read this one.
        if (vec) {
          if (n4 < p.N) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < mt)
                ep_store4(a, i0 + static_cast<int64_t>(i) * p.N, in[i], gate_n,
                          *reinterpret_cast<const float4*>(box + (4 * q + i) * kEtBoxPitch + 4 * lane));
          }
        } else {
          for (int i = 0; i < mt; ++i) {
            const float* src = box + (4 * q + i) * kEtBoxPitch;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int nn = tl.n0 + 32 * j + lane;
              if (nn < p.N) ep_store1(a, m0 + i, nn, p.N, src[32 * j + lane]);
            }
          }
        }
      }
    }
  } else {
    // ------------------------------------------------------------ packed-weight producer
    if (elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      int e = 0;
      for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        const EtTile tl = et_tile(p, tb, t, e);
        const int row = tl.e * p.N + tl.n0;
        for (int u = 0; u < ksteps; ++u, ++it) {
          const uint32_t w = it % F::kWStages, ph = (it / F::kWStages) & 1u;
          if (!mbar_wait(wempty_bar(w), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(wfull_bar(w), F::kWBytes);
          tma_load_2d(sbase + F::kWOff + w * F::kWBytes, &tm_w, wfull_bar(w),
                      (SPLIT ? u >> 1 : u) * F::kWqRowBytes, row);
        }
      }
      for (uint32_t j = (it > F::kWStages ? it - F::kWStages : 0); j < it; ++j)
        mbar_wait_drain(wfull_bar(j % F::kWStages), (j / F::kWStages) & 1u);
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512);
  }
}

// The f16 copy of the activations in the dequantizers' k order, row by row: row r of the copy
// is row rows[r] of x (or r), for the rows some expert has; an index outside x gives zeros.
template <int FMT>
__global__ void __launch_bounds__(256) ep_prep_kernel(const uint16_t* __restrict__ x,
                                                      uint16_t* __restrict__ x16,
                                                      const int* __restrict__ rows,
                                                      const int* __restrict__ offsets, int E,
                                                      int x_rows, int R, int K) {
  pdl_trigger_and_wait();
  const int lim = offsets ? min(max(__ldg(offsets + E), 0), R) : R;
  const int gk = K / 16;
  const int64_t total = static_cast<int64_t>(lim) * gk;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t r = i / gk;
    const int g = static_cast<int>(i - r * gk);
    int64_t src = r;
    if (rows) src = __ldg(rows + r);
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    if (src >= 0 && src < x_rows) {
      const uint4* xp = reinterpret_cast<const uint4*>(x + src * K) + 2 * g;
      a = __ldg(xp);
      b = __ldg(xp + 1);
    }
    x16_group<FMT>(a, b, reinterpret_cast<uint4*>(x16 + r * K) + 2 * g);
  }
}

}  // namespace tgemm
