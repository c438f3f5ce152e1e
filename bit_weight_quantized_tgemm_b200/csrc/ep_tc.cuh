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
constexpr int kEtSumTok = 80;                   // most tokens of a tile with running sums
constexpr int kEtBK = 128;
constexpr int kEtGroups = 3;                    // dequant groups of 4 warps, stages in turn
constexpr int kEtWProdWarp = 2;
constexpr int kEtDeqWarp0 = 3;
constexpr int kEtEpiWarp0 = kEtDeqWarp0 + 4 * kEtGroups;
constexpr int kEtThreads = (kEtEpiWarp0 + 8) * 32;
constexpr int kEtXRing = 4 * kEtTok * 256;      // activation ring: 4 slots of 128 tokens or 8 of 64
constexpr int kEtXSlots = 8;
constexpr int kEtA = 4;                         // A stages in tensor memory
constexpr int kEtACol0 = 256;                   // their columns, behind the accumulators
constexpr int kEtMaxExperts = 1024;
static_assert(3 * kEtSumTok <= kEtACol0 && 2 * kEtTok <= kEtACol0 && kEtACol0 + 64 * kEtA <= 512, "TMEM budget");

template <int FMT>
struct EtFmt {
  static constexpr int kWqRowBytes = FMT == 0 ? 32 : 64;
  static constexpr int kWStages = FMT == 0 ? 16 : 8;
  static constexpr int kWBytes = kEtRows * kWqRowBytes;
  static constexpr int kXOff = 0;
  static constexpr int kWOff = kEtXRing;
  static constexpr int kTabOff = kWOff + kWStages * kWBytes;
  static constexpr int kBarOff = kTabOff + 2 * (kEtMaxExperts + 2) * 4;
  static constexpr int kNumBars = 2 * kEtXSlots + 2 * kWStages + 4 + 1;
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

// TMA maps.  Activations: the f16 copy as [k block of 64][row][64], boxes of two k blocks
// (a stage) and 16, 32, 64 or 128 rows, so that one copy brings a tile's stage.
struct EtMaps {
  CUtensorMap x[4];
  CUtensorMap w;
};
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, uint32_t bar,
                                            int32_t x, int32_t y, int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// log2 of the box rows / 16 for a tile of mt tokens
__device__ __forceinline__ int et_box(int mt) { return mt <= 16 ? 0 : mt <= 32 ? 1 : mt <= 64 ? 2 : 3; }

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// mbar_wait with a suspend hint: the waiting warp sleeps in the barrier unit instead of
// polling, and leaves its issue slots to the dequantizers.  Bounded as mbar_wait is.
__device__ __forceinline__ bool mbar_try_sleep(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity), "r"(1000000u)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool et_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  if (mbar_try_sleep(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_try_sleep(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1u;
      atomicOr(&g_device_error, kDevErrTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool et_wait_warp(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  return __all_sync(0xFFFFFFFFu, et_wait(bar, parity, abort_flag));
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
// accumulator goes into a running sum in tensor memory, rounded to nearest.
template <int FMT, bool SPLIT, bool SUMS>
__global__ void __launch_bounds__(kEtThreads, 1)
    ep_tc_kernel(const __grid_constant__ EtMaps tm, const EtParams p) {
  using F = EtFmt<FMT>;
  constexpr int kSeg = 4;
  constexpr int kAccCols = SUMS ? kEtSumTok : kEtTok;  // columns of an accumulator
  constexpr int kSumCol0 = 2 * kAccCols;
  extern __shared__ uint8_t et_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(et_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + F::kBarOff;
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (kEtXSlots + s); };
  auto wfull_bar = [&](uint32_t w) { return bar0 + 8u * (2 * kEtXSlots + w); };
  auto wempty_bar = [&](uint32_t w) { return bar0 + 8u * (2 * kEtXSlots + F::kWStages + w); };
  auto accfull_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kEtXSlots + 2 * F::kWStages + a); };
  auto accempty_bar = [&](uint32_t a) { return bar0 + 8u * (2 * kEtXSlots + 2 * F::kWStages + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (2 * kEtXSlots + 2 * F::kWStages + 4);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + F::kMiscOff);
  volatile uint32_t* abort_flag = reinterpret_cast<volatile uint32_t*>(smem + F::kMiscOff + 4);
  int* tab_off = reinterpret_cast<int*>(smem + F::kTabOff);
  int* tab_tp = tab_off + kEtMaxExperts + 2;

  // warp index as a warp-uniform value, so that the single-thread roles below issue from
  // uniform registers (an MMA issued from per-thread registers takes 125 cycles whatever its
  // size; from uniform ones N / 2 cycles)
  const int warp = __shfl_sync(0xFFFFFFFFu, static_cast<int>(threadIdx.x) >> 5, 0);
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kEtXSlots; ++s) {
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
    }
    mbar_init(drain_bar, 1);
    *abort_flag = 0u;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tm.x[et_box(p.nt)]);
    tma_prefetch_desc(&tm.w);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_trigger();
  // With device offsets every role needs them first; a dense call's weights are read early,
  // and only the activation producer and the epilogue wait.
  if (p.offsets || warp == 0 || warp >= kEtEpiWarp0) pdl_wait();
  if (warp == kEtWProdWarp) et_build_table(p.offsets, p.E, p.R, p.nt, tab_off, tab_tp);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const EtTable tb{tab_off, tab_tp};
  const int num_tiles = tab_tp[p.E] * p.tiles_n;
  const int ksteps = p.ksteps;
  // activation slots: unit i uses slot i & (nx - 1); deeper when the tiles are small
  const int lx = p.nt <= kEtTok / 2 ? 3 : 2;
  const uint32_t nx = 1u << lx, xslot = kEtXRing >> lx;

  if (warp == 0) {
    // ------------------------------------------------------------ activation producer
    if (elect_one()) {
      uint32_t it = 0;
      bool ok = true;
      int e = 0;
      for (int t = blockIdx.x; ok && t < num_tiles; t += gridDim.x) {
        const EtTile tl = et_tile(p, tb, t, e);
        const int box = et_box(tl.mt);
        const CUtensorMap* map = &tm.x[box];
        const uint32_t bytes = 4096u << box;
        for (int u = 0; u < ksteps; ++u, ++it) {
          const uint32_t s = it & (nx - 1), ph = (it >> lx) & 1u;
          if (!et_wait(empty_bar(s), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(full_bar(s), bytes);
          tma_load_3d(sbase + F::kXOff + s * xslot, map, full_bar(s), 0, tl.m0, 2 * (SPLIT ? u >> 1 : u));
        }
      }
      // every load issued must land before the CTA may exit
      for (uint32_t j = (it > nx ? it - nx : 0); j < it; ++j)
        mbar_wait_drain(full_bar(j & (nx - 1)), (j >> lx) & 1u);
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
        const uint32_t half = 2048u << et_box(tl.mt);  // bytes of a k block's box
        for (int u0 = 0; ok && u0 < ksteps; ++sc) {
          const int u1 = SUMS ? min(u0 + kSeg, ksteps) : ksteps;
          const uint32_t a = sc & 1u;
          if (!et_wait(accempty_bar(a), ((sc >> 1) & 1u) ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + a * kAccCols;
          for (int u = u0; u < u1; ++u, ++it) {
            const uint32_t s = it & (nx - 1), ph = (it >> lx) & 1u;
            if (!et_wait(full_bar(s), ph, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a_tmem = tmem_base + kEtACol0 + (it % kEtA) * 64;
            const uint32_t xs = sbase + F::kXOff + s * xslot;
            const uint64_t b0 = smem_desc_sw128(xs);
            const uint64_t b1 = smem_desc_sw128(xs + half);
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              mma_f16_ts(d_tmem, a_tmem + 8u * kk, (kk < 4 ? b0 : b1) + 2u * (kk & 3), idesc,
                         (u > u0 || kk > 0) ? 1u : 0u);
            mma_commit(empty_bar(s));
          }
          if (!ok) break;
          mma_commit(accfull_bar(a));
          u0 = u1;
        }
      }
      mma_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0u);
    }
  } else if (warp == kEtWProdWarp) {
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
          if (!et_wait(wempty_bar(w), ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(wfull_bar(w), F::kWBytes);
          tma_load_2d(sbase + F::kWOff + w * F::kWBytes, &tm.w, wfull_bar(w),
                      (SPLIT ? u >> 1 : u) * F::kWqRowBytes, row);
        }
      }
      for (uint32_t j = (it > F::kWStages ? it - F::kWStages : 0); j < it; ++j)
        mbar_wait_drain(wfull_bar(j % F::kWStages), (j / F::kWStages) & 1u);
    }
  } else if (warp < kEtEpiWarp0) {
    // ------------------------------------------------------------ dequantizers
    // Group grp takes the units i = grp (mod kEtGroups) of the CTA's stream of units; each of
    // its threads unpacks one weight row's 128 codes of the unit.
    const int q = warp & 3;                        // TMEM lane quarter
    const int grp = (warp - kEtDeqWarp0) >> 2;
    const int rt = 32 * q + lane;                  // weight row within the tile
    const int nscale = FMT == 0 ? p.K / 128 : p.K / 64;
    const uint32_t a_lane = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + kEtACol0;
    const uint32_t w_mine = sbase + F::kWOff + rt * F::kWqRowBytes;
    // 16-byte chunk c of the row sits at chunk c ^ swz (TMA's 32- or 64-byte swizzle)
    const uint32_t swz = FMT == 0 ? (rt >> 2) & 1 : (rt >> 1) & 3;
    // The scales are loaded two of the group's units ahead, across tiles: position (lt, lu).
    // They alternate between two sets of registers, never moved: a move would wait for its load.
    constexpr int kSc = FMT == 0 ? 1 : 2;
    int lt = blockIdx.x, lu = grp, le = 0;
    const uint16_t* lrow = nullptr;
    auto locate = [&]() {  // the row's scales of tile lt (null: no such tile or row)
      while (lu >= ksteps) {
        lu -= ksteps;
        lt += gridDim.x;
        lrow = nullptr;
        if (lt >= num_tiles) return;
      }
      if (!lrow && lt < num_tiles) {
        const EtTile tl = et_tile(p, tb, lt, le);
        if (tl.n0 + rt < p.N)
          lrow = p.scales + (static_cast<int64_t>(tl.e) * p.N + tl.n0 + rt) * nscale * (FMT == 0 ? 1 : 2);
      }
    };
    auto load_scales = [&](uint32_t (&sc)[kSc]) {
      sc[0] = sc[kSc - 1] = 0u;
      if (lt < num_tiles) {
        const int ks = SPLIT ? lu >> 1 : lu;
        if (lrow) {
          if (FMT == 0) {
            sc[0] = __ldg(lrow + ks);
          } else {
            const uint32_t* sp = reinterpret_cast<const uint32_t*>(lrow) + 2 * ks;
            sc[0] = __ldg(sp);
            if (2 * ks + 1 < nscale) sc[kSc - 1] = __ldg(sp + 1);
          }
        }
        lu += kEtGroups;
        locate();
      }
    };
    locate();
    uint32_t sa[kSc], sb[kSc];
    load_scales(sa);
    load_scales(sb);
    const int my_tiles = num_tiles > static_cast<int>(blockIdx.x)
                             ? (num_tiles - static_cast<int>(blockIdx.x) + gridDim.x - 1) / gridDim.x : 0;
    const uint32_t units = static_cast<uint32_t>(my_tiles) * ksteps;
    // one unit; false at the end
    auto unit = [&](uint32_t i, uint32_t (&sn)[kSc]) -> bool {
      if (i >= units) return false;
      uint32_t sc[kSc];
#pragma unroll
      for (int j = 0; j < kSc; ++j) sc[j] = sn[j];
      load_scales(sn);
      const uint32_t w = i % F::kWStages, wph = (i / F::kWStages) & 1u;
      if (!et_wait_warp(wfull_bar(w), wph, abort_flag)) return false;
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
      for (int h = 0; h < 4; ++h) {  // 32 codes each
        uint32_t o[16];
        if (FMT == 0) {
          const uint32_t d2 = sc[0] | (sc[0] << 16);
#pragma unroll
          for (int j = 0; j < 2; ++j) q2_word_to_f16(cw[2 * h + j], d2, o + 8 * j);
        } else if (!SPLIT) {
          const uint32_t s1 = sc[(h >> 1) % kSc];
          const uint32_t s2 = (s1 & 0xFFFFu) | (s1 << 16);
          const uint32_t z2 = (s1 >> 16) | (s1 & 0xFFFF0000u);
#pragma unroll
          for (int j = 0; j < 4; ++j) q4_word_to_f16(cw[(4 * h + j) % kWords], s2, z2, o + 4 * j);
        } else {
          const uint32_t s1 = sc[(h >> 1) % kSc];
          const float sf = __half2float(__ushort_as_half(static_cast<uint16_t>(s1 & 0xFFFFu)));
          const float zf = __half2float(__ushort_as_half(static_cast<uint16_t>(s1 >> 16)));
          if (i & 1) {  // ksteps is even: odd units are the low parts
#pragma unroll
            for (int j = 0; j < 4; ++j) q4_word_split<true>(cw[(4 * h + j) % kWords], sf, zf, o + 4 * j);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) q4_word_split<false>(cw[(4 * h + j) % kWords], sf, zf, o + 4 * j);
          }
        }
        if (h == 0) {
          // the A stage is free once unit i - kEtA, which had it before, is multiplied
          const uint32_t j = i - kEtA;
          if (i >= kEtA && !et_wait_warp(empty_bar(j & (nx - 1)), (j >> lx) & 1u, abort_flag)) return false;
          tc_fence_after();
        }
        tmem_st_32x32b_x16(a_lane + (i % kEtA) * 64 + 16 * h, o);
      }
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(full_bar(i & (nx - 1)));
      return true;
    };
    for (uint32_t i = grp; unit(i, sa) && unit(i + kEtGroups, sb); i += 2 * kEtGroups) {
    }
  } else {
    // ------------------------------------------------------------ epilogue
    // A thread has one weight row n and 16 tokens of a chunk; its warp's loads and stores take
    // 32 neighbouring n of a token row.
    const int q = warp & 3;                      // TMEM lane quarter
    const int set = (warp - kEtEpiWarp0) >> 2;   // 16-token chunks of this parity
    const EpArgs& a = p.ep;
    const uint32_t t_lane = tmem_base + (static_cast<uint32_t>(32 * q) << 16);
    uint32_t sc = 0;  // segments done
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
      const bool nv = n < p.N;
      float bias = 0.f, gate_n = 1.f;
      if (a.bias && nv) bias = ep_load(a.bias, static_cast<int64_t>(tl.e) * p.N + n, a.bias_f32);
      if (a.gate && !a.gate_rows && nv) gate_n = bf16_bits_to_f32(a.gate[n]);
      const int chunks = (tl.mt + 15) >> 4;
      // running sum += a segment, in f32 rounded to nearest
      for (int u = kSeg; SUMS && ok && u < ksteps; u += kSeg, ++sc) {
        const uint32_t ab = sc & 1u;
        if (!et_wait_warp(accfull_bar(ab), (sc >> 1) & 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after();
        for (int cc = set; cc < chunks; cc += 2) {
          uint32_t v[16], w[16];
          tmem_ld_32x32b_x16(t_lane + ab * kAccCols + 16 * cc, v);
          if (u > kSeg) tmem_ld_32x32b_x16(t_lane + kSumCol0 + 16 * cc, w);
          tmem_wait_ld();
          if (u > kSeg) {
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + __uint_as_float(w[i]));
          }
          tmem_st_32x32b_x16(t_lane + kSumCol0 + 16 * cc, v);
        }
        tmem_wait_st();
        release(ab);
      }
      if (!ok) break;
      const uint32_t ab = sc & 1u;
      if (!et_wait_warp(accfull_bar(ab), (sc >> 1) & 1u, abort_flag)) {
        ok = false;
        break;
      }
      ++sc;
      tc_fence_after();
      if (set >= chunks) release(ab);
      for (int cc = set; cc < chunks; cc += 2) {
        const int mt = tl.mt - 16 * cc;  // tokens of the chunk, at least one
        const int64_t i0 = static_cast<int64_t>(tl.m0 + 16 * cc) * p.N + n;
        // the tokens' gates and residuals, on their way while the sums are read
        float g[16], r[16];
        if (a.gate && a.gate_rows) {
          const uint16_t* src = a.gate + i0;
#pragma unroll
          for (int i = 0; i < 16; ++i, src += p.N) g[i] = nv && i < mt ? bf16_bits_to_f32(*src) : 0.f;
        }
        if (a.residual) {
          if (a.residual_f32) {
            const float* src = static_cast<const float*>(a.residual) + i0;
#pragma unroll
            for (int i = 0; i < 16; ++i, src += p.N) r[i] = nv && i < mt ? *src : 0.f;
          } else {
            const uint16_t* src = static_cast<const uint16_t*>(a.residual) + i0;
#pragma unroll
            for (int i = 0; i < 16; ++i, src += p.N) r[i] = nv && i < mt ? bf16_bits_to_f32(*src) : 0.f;
          }
        }
        uint32_t v[16];
        tmem_ld_32x32b_x16(t_lane + ab * kAccCols + 16 * cc, v);
        float f[16];
        if (SUMS && ksteps > kSeg) {
          uint32_t w[16];
          tmem_ld_32x32b_x16(t_lane + kSumCol0 + 16 * cc, w);
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
        if (a.gate) {
          if (a.gate_rows) {
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] *= g[i];
          } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] *= gate_n;
          }
        }
        if (a.residual) {
#pragma unroll
          for (int i = 0; i < 16; ++i) f[i] += r[i];
        }
        if (a.out_f32) {
          float* dst = static_cast<float*>(a.y) + i0;
#pragma unroll
          for (int i = 0; i < 16; ++i, dst += p.N)
            if (nv && i < mt) *dst = f[i];
        } else {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.y) + i0;
#pragma unroll
          for (int i = 0; i < 16; ++i, dst += p.N)
            if (nv && i < mt) *dst = __float2bfloat16_rn(f[i]);
        }
      }
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
