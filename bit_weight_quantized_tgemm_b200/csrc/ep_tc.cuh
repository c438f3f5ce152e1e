// ep_tc.cuh -- tensor-core kernel of the epilogue and expert matmuls:
//   y[m] = residual[m] + gate[m] * act(x[m] W_e^T + bias_e),   rows m of expert e
// with W packed (ternary or 4-bit).  A dense call is one expert that owns every row.
//
// Tile: 128 weight rows (MMA M) x up to 128 tokens (MMA N, in steps of 16), in units of 128 k.
// A, the dequantized weights, is in tensor memory; B, the activations (an f16 copy in the
// dequantizers' k order), in shared memory; the f32 accumulators are in tensor memory, two, so
// that the epilogue of a tile runs under the next tile's products.  Persistent, one CTA an SM:
//   warp 0      activations -> shared memory, one TMA copy a unit
//   warp 1      the MMAs, 8 a unit
//   warp 2      packed weights -> shared memory by TMA; before that the experts' tile table
//   warp 3      scales -> shared memory by asynchronous copies
//   warps 4-15  dequantizers, three groups of 4, units in turn: a thread unpacks one weight row
//               of a unit from shared memory into tensor memory
//   warps 16-23 the epilogue, two sets of 4, chunks of 16 tokens in turn
// Weight rows are MMA M, and few tokens a small N, since most calls have many weights and few
// tokens an expert; an expert's own rows fill the token tiles, so no row is multiplied twice.
//
// What bounds it.  A unit of few tokens takes 0.27 us whatever its format (76 units of 17 x 2560
// x 9728), which is the dequantizers' arithmetic (256 to 384 cycles of the half-rate pipes) with
// the MMA thread's waits and issue (some 460 cycles) beside it; a fourth group, units of 64 k
// or tests of the barriers ahead of the waits change nothing or cost.  A unit of 128 tokens
// takes 0.45 us or 790 cycles, of which the tensor core is busy for 512 (1536 x 12288 x 2560
// ternary, 81 us in a replayed graph: 1190 TFLOP/s, tensor pipe 68 % of active cycles, 11 TB/s out
// of L2).  It is not L2: pairs of CTAs
// that each load half of the tokens take 80 us.  The dequantizers' stores and the accumulators
// share tensor memory, and the issue slots are 66 % full.  The kernels are held to 80 registers a
// thread and spill: 20 to 48 bytes for a bf16 y, 260 to 280 for an f32 one, whose running sums take
// 48 registers of the epilogue's threads.  About 8 us a call are the copy of x, the
// start of both kernels, the first unit and the last epilogue (148 tiles of 17 tokens x 16 units:
// 13.0 us; five rounds of them 33.9 us).
#pragma once

#include "common.cuh"
#include "epilogue.cuh"
#include "gemm_tc.cuh"
#include "prep.cuh"

namespace tgemm {

constexpr int kEtRows = 128;
constexpr int kEtTok = 128;
constexpr int kEtSumTok = 96;                   // most tokens of a tile with running sums
constexpr int kEtGroups = 3;                    // dequant groups of 4 warps, stages in turn
constexpr int kEtWProdWarp = 2;
constexpr int kEtScaleWarp = 3;
constexpr int kEtDeqWarp0 = 4;
constexpr int kEtEpiWarp0 = kEtDeqWarp0 + 4 * kEtGroups;
constexpr int kEtThreads = (kEtEpiWarp0 + 8) * 32;
constexpr int kEtRing = 192 * 1024;             // activation slots, then weight stages
constexpr int kEtXSlots = 8, kEtWStages = 16;   // the most of each
constexpr int kEtChunk = 16;                    // scale blocks of a chunk
constexpr int kEtScBufs = 3;                    // chunks of scales in shared memory
constexpr int kEtMaxExperts = 1024;
// Every ring has a power of two of places, so that place and phase of unit i come from its bits.
// Activation slots hold 32, 64 or 128 tokens.  Large tiles bring 32 KB of activations a unit; with
// small ones many weights are to be on their way from memory.
__host__ __device__ constexpr int et_slot_tok(int nt) { return nt <= 32 ? 32 : nt <= 64 ? 64 : kEtTok; }
// log2 of the slots, for units of bk
__host__ __device__ constexpr int et_lx(int nt, int bk) { return nt * bk <= 64 * 128 || bk < 128 ? 3 : 2; }
// log2 of the weight stages of wbytes each, in the rest of the ring
__host__ __device__ constexpr int et_lw(int nt, int bk, int wbytes) {
  const int n = (kEtRing - (et_slot_tok(nt) * bk * 2 << et_lx(nt, bk))) / wbytes;
  return n >= 16 ? 4 : n >= 8 ? 3 : 2;
}
static_assert(et_lw(128, 128, 8192) == 3 && et_lw(64, 128, 8192) == 3 && et_lw(32, 128, 8192) == 4 &&
                  et_lw(128, 128, 4096) == 4 && et_lw(128, 64, 4096) == 4,
              "weight stages");
// Tensor memory: two accumulators and from column 256 four A stages of 64 columns.
// The A stages hold no more units than there are activation slots: a dequant group reports unit
// i on its slot's barrier once it may write its A stages, that is when the unit that had them
// before is multiplied, and the barrier must then be done with unit i - slots.
constexpr int kEtLA = 2;  // log2 of the A stages
static_assert(2 * kEtTok <= 256 && 256 + (64 << kEtLA) <= 512 && 2 * kEtSumTok <= 256 && kEtLA <= et_lx(128, 128), "TMEM");

template <int FMT, bool SPLIT>
struct EtFmt {
  // k of a unit.  With two f16 parts a weight, 64: an A stage then holds both, and four units
  // instead of two are between the dequantizers and the tensor core.
  static constexpr int kBK = SPLIT ? 64 : 128;
  static constexpr int kWqRowBytes = FMT == 0 ? kBK / 4 : kBK / 2;
  static constexpr CUtensorMapSwizzle kWSwizzle = kWqRowBytes == 32 ? CU_TENSOR_MAP_SWIZZLE_32B : CU_TENSOR_MAP_SWIZZLE_64B;
  static constexpr int kWBytes = kEtRows * kWqRowBytes;
  // A chunk's scales as 32-bit words [word][row] (Q2: two blocks' d, 4-bit: a block's (s, z)):
  // the pitch keeps the scale warp's writes and the dequantizers' reads free of bank conflicts.
  static constexpr int kScWords = FMT == 0 ? kEtChunk / 2 : kEtChunk;
  static constexpr int kScPitch = 4 * kEtRows + (FMT == 0 ? 16 : 8);
  static constexpr int kScBytes = kScWords * kScPitch;
  static constexpr int kScOff = kEtRing;
  static constexpr int kTabOff = kScOff + kEtScBufs * kScBytes;
  static constexpr int kBarOff = kTabOff + 2 * (kEtMaxExperts + 2) * 4;
  static constexpr int kNumBars = 2 * kEtXSlots + 2 * kEtWStages + 4 + 1 + 2 * kEtScBufs;
  static constexpr int kMiscOff = kBarOff + kNumBars * 8;
  static constexpr int kSmemBytes = kMiscOff + 16 + 1024;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

constexpr int kEtMaxSplit = 8;
// The units [first, end) that CTA `rank` of a tile's `split` takes: whole pairs, since a pair of
// ternary scales is one word.
__host__ __device__ constexpr int et_first_unit(int ksteps, int split, int rank) {
  return rank >= split ? ksteps : (ksteps + 1) / 2 * rank / split * 2;
}

struct EtParams {
  int N, K, E, R;
  int nt;                 // tokens per tile, a multiple of 16
  int tiles_n;            // ceil(N / 128)
  int ksteps;             // units of a tile: K / kBK, rounded up
  int split;              // CTAs of a cluster that share a tile's units (dense calls)
  int nblocks;            // scale blocks of a row: K / 128 or K / 64
  const int* offsets;     // [E + 1] row ranges, or null: one expert, rows [0, R)
  const uint16_t* scales;
  EpArgs ep;
};

// TMA maps.  Activations: the f16 copy as [k block of 64][row][64], boxes of a unit's one or two
// k blocks and 16, 32, 64, 96 or 128 rows (no more than nt), so that one copy brings a tile's unit.
constexpr int kEtBoxes = 5;
struct EtMaps {
  CUtensorMap x[kEtBoxes];
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
// the map for a tile of mt tokens, and its box's rows
__host__ __device__ constexpr int et_box(int mt) { return mt <= 16 ? 0 : mt <= 32 ? 1 : (mt + 31) / 32; }
__host__ __device__ constexpr int et_box_most(int box) { return box == 0 ? 16 : 32 * box; }
__host__ __device__ constexpr int et_box_rows(int box, int nt) { return et_box_most(box) < nt ? et_box_most(box) : nt; }
static_assert(et_box(kEtTok) == kEtBoxes - 1 && et_box(33) == 2 && et_box(64) == 2 && et_box(65) == 3, "boxes");

// Every thread of a cluster, the warps each from where they are.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire;" ::: "memory"); }
__device__ __forceinline__ void cluster_sync() {
  cluster_arrive();
  cluster_wait();
}
// A store to shared memory of CTA `rank` of the cluster, at the place `addr` has in this one.
__device__ __forceinline__ void st_cluster_f32(uint32_t addr, uint32_t rank, float v) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "st.shared::cluster.f32 [a], %2;\n\t}" ::"r"(addr), "r"(rank), "f"(v)
      : "memory");
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}

// Wait for a phase.  The common case is one try_wait (39 cycles); a warp that has to wait
// sleeps in the barrier unit and leaves its issue slots to others.  Bounded: after
// kWaitLimitNs it records a timeout and raises the CTA's abort flag, and every later wait of
// the CTA that is not satisfied returns false at once.  A thread whose wait failed issues no
// more copies or MMAs and arrives on no more barriers, so the kernel runs out with the device
// error word set.
__device__ __noinline__ bool et_wait_slow(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity), "r"(100000u)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      *abort_flag = 1u;
      atomicOr(&g_device_error, kDevErrTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool et_wait(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  return mbar_try_wait(bar, parity) || et_wait_slow(bar, parity, abort_flag);
}
// By a whole warp, which goes on together; each lane gets its own answer.
__device__ __forceinline__ bool et_wait_warp(uint32_t bar, uint32_t parity, volatile uint32_t* abort_flag) {
  const bool ok = et_wait(bar, parity, abort_flag);
  __syncwarp();
  return ok;
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
  const int tt = tb.tp[e + 1] - tb.tp[e], rows = tb.off[e + 1] - tb.off[e];
  const int step = ((rows + tt - 1) / tt + 15) & ~15;  // the rows in equal parts, as nt would make
  const int r = t - tb.tp[e] * p.tiles_n;
  const int tn = r / tt, ti = r - tn * tt;
  EtTile x;
  x.e = e;
  x.n0 = tn * kEtRows;
  x.m0 = tb.off[e] + ti * step;
  x.mt = min(step, tb.off[e + 1] - x.m0);
  return x;
}

// From L2: the line may be in this SM's L1 from an earlier call.
__device__ __forceinline__ int ld_relaxed(const int* p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
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
  int run = min(max(ld_relaxed(offsets), 0), R);
  if (lane == 0) {
    off[0] = run;
    tp[0] = 0;
  }
  for (int e0 = 0; e0 < E; e0 += 32) {
    const int e = e0 + lane;
    int v = e < E ? min(max(ld_relaxed(offsets + e + 1), 0), R) : 0;
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

__device__ __forceinline__ uint32_t hadd2_u32(uint32_t a, uint32_t b) {
  __half2 r = __hadd2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmin2_u32(uint32_t a, uint32_t b) {
  __half2 r = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hfma2_u32(uint32_t a, uint32_t b, uint32_t c) {
  __half2 r = __hfma2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b), *reinterpret_cast<__half2*>(&c));
  return *reinterpret_cast<uint32_t*>(&r);
}

// 4-bit weights for a bf16 y: f16((q - c) s - f16((z - c) s)), pairs as q4_word_to_f16, with c the
// whole number next to z.  q - c is exact, and z - c as good as q - z (exact for 0 <= z <= 1024).
// The rounding of (z - c) s, which all weights of a group share, is one of at most s / 2, and
// nothing leaves f16's range unless a weight does.  Shared roundings matter because activations of
// one sign add them up: relative to y, at K = 2560 with z in [7, 8] and activations around one,
// this form is 4.4e-4 off, c = 0 (that is f16(z s)) 2.5e-3, f16(f16(q - z) s) 4.5e-4; with z in
// [0, 15] 9e-5, and c = 8 for every z 2.6e-4 (computed).  Three instructions a pair, as c = 0;
// five more a group (12 x 9728 x 2560: 12.4 -> 12.7 us; 366 rows of 64 experts: 38.9 -> 39.6 us).
struct Q4Centre {
  uint32_t base[2];  // 1024 + c and 64 + c, twice each: the unpacked codes are 1024 + q and 64 + q
  uint32_t zs;       // f16((c - z) s) twice
};
__device__ __forceinline__ Q4Centre q4_centre(uint32_t s2, uint32_t z2) {
  Q4Centre c;
  // at 1024 an f16 step is 1; the limit keeps a z near the end of f16's range finite
  c.base[0] = hmin2_u32(hadd2_u32(z2, 0x64006400u), 0x78007800u);
  c.base[1] = hsub2_u32(c.base[0], 0x63806380u);                                    // 960 less
  c.zs = hmul2_u32(hsub2_u32(hsub2_u32(c.base[0], 0x64006400u), z2), s2);
  return c;
}
__device__ __forceinline__ void q4_word_centred(uint32_t w, uint32_t s2, const Q4Centre& c, uint32_t* o) {
  constexpr uint32_t kMagic[2] = {0x64006400u, 0x54005400u};  // 1024, 64
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = i & 1;
    const uint32_t q = hsub2_u32(lop3_and_or(i < 2 ? w : (w >> 8), 0x000F000Fu << (4 * j), kMagic[j]), c.base[j]);
    o[i] = hfma2_u32(q, s2, c.zs);
  }
}

// 4-bit weights w = (q - z) s as a high and a low f16 part, pairs as q4_word_to_f16: with
// t = f16(q - z), hi = f16(t s) and lo = f16(t s - hi), which one fma gives.  EXACT: q - z is an
// f16 value for every code; otherwise its rounding error (two-sum), times s, joins lo.
template <bool EXACT>
__device__ __forceinline__ void q4_word_split(uint32_t w, uint32_t s2, uint32_t z2, uint32_t* hi, uint32_t* lo) {
  constexpr uint32_t kMagic[2] = {0x64006400u, 0x54005400u};  // 1024, 64
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int j = i & 1;
    const uint32_t q = hsub2_u32(lop3_and_or(i < 2 ? w : (w >> 8), 0x000F000Fu << (4 * j), kMagic[j]), kMagic[j]);
    const uint32_t t = hsub2_u32(q, z2);
    hi[i] = hmul2_u32(t, s2);
    lo[i] = hfma2_u32(t, s2, hi[i] ^ 0x80008000u);
    if (!EXACT) {
      const uint32_t b = hsub2_u32(q, t);  // z, up to rounding
      const uint32_t err = hadd2_u32(hsub2_u32(q, hadd2_u32(t, b)), hsub2_u32(b, z2));
      lo[i] = hfma2_u32(err, s2, lo[i]);
    }
  }
}
// Whether q - z has at most 11 bits for every code q: z a multiple of 2^-7 in [0, 16], or of
// 2^-8 (as every f16 is there) in [7, 8].
__device__ __forceinline__ bool q4_zero_exact(uint32_t z16) {
  const float z = __half2float(__ushort_as_half(static_cast<uint16_t>(z16)));
  const float z128 = z * 128.f;
  return (z >= 7.f && z <= 8.f) || (z >= 0.f && z <= 16.f && z128 == rintf(z128));
}

// SPLIT (4-bit weights, f32 y): a unit's weights are a high and a low f16 part in one A stage,
// since f16 weights alone are 2^-12 relative off.  The low part is subnormal for weights below
// 2^-3 and so off by up to 2^-25: y is 1e-6 off with scales around 0.01, 4e-5 with 0.0001.  (One
// power of two over all weights would shift that floor, but only at the cost of large weights.)
//
// SUMS (f32 y): the tensor core adds each K = 16 step to the f32 accumulator with truncation,
// 1.5e-8 of the sum per step towards zero (2.3e-6 at K = 2560), so after every 48 steps the
// epilogue warps take the accumulator into running sums in registers, rounded to nearest: 5e-7 of
// the norm of y at K = 2560, 6.7e-7 at 9728.  They hold 96 tokens a tile.
template <int FMT, bool SPLIT, bool SUMS, bool SHARE>
__global__ void __launch_bounds__(kEtThreads, 1)
    ep_tc_kernel(const __grid_constant__ EtMaps tm, const EtParams p) {
  using F = EtFmt<FMT, SPLIT>;
  constexpr int kSeg = 6;  // units (of 8 steps) of an accumulator segment
  static_assert(FMT == 1 || !SPLIT, "ternary weights are exact in f16");
  static_assert(!SPLIT || SUMS, "the low parts are for f32 y");
  constexpr int kCU = FMT == 1 && !SPLIT ? 8 : 16;  // units of a chunk of scales
  extern __shared__ uint8_t et_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(et_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar0 = sbase + F::kBarOff;
  auto full_bar = [&](uint32_t s) { return bar0 + 8u * s; };
  auto empty_bar = [&](uint32_t s) { return bar0 + 8u * (kEtXSlots + s); };
  auto wfull_bar = [&](uint32_t w) { return bar0 + 8u * (2 * kEtXSlots + w); };
  auto wempty_bar = [&](uint32_t w) { return bar0 + 8u * (2 * kEtXSlots + kEtWStages + w); };
  constexpr uint32_t kBar1 = 2 * kEtXSlots + 2 * kEtWStages;
  auto accfull_bar = [&](uint32_t a) { return bar0 + 8u * (kBar1 + a); };
  auto accempty_bar = [&](uint32_t a) { return bar0 + 8u * (kBar1 + 2 + a); };
  const uint32_t drain_bar = bar0 + 8u * (kBar1 + 4);
  auto sfull_bar = [&](uint32_t b) { return bar0 + 8u * (kBar1 + 5 + b); };
  auto sempty_bar = [&](uint32_t b) { return bar0 + 8u * (kBar1 + 5 + kEtScBufs + b); };
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
    for (int w = 0; w < kEtWStages; ++w) {
      mbar_init(wfull_bar(w), 1);
      mbar_init(wempty_bar(w), 4);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accfull_bar(a), 1);
      mbar_init(accempty_bar(a), 8);
    }
    for (int b = 0; b < kEtScBufs; ++b) {
      mbar_init(sfull_bar(b), 32);  // the scale warp's lanes
      mbar_init(sempty_bar(b), 4 * kEtGroups);
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
  // The activation producer and the epilogue wait for the copy of x, and the barrier below for
  // them, so that the other roles too start behind the copy.  Only the experts' table is built
  // meanwhile: offsets come from before the copy's kernel, which waits for what is ahead of it before
  // it lets this one start.
  if (warp == 0 || warp >= kEtEpiWarp0) pdl_wait();
  if (warp == kEtWProdWarp) et_build_table(p.offsets, p.E, p.R, p.nt, tab_off, tab_tp);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const EtTable tb{tab_off, tab_tp};
  const int num_tiles = tab_tp[p.E] * p.tiles_n;
  // A cluster of p.split CTAs shares a tile: each has its own units and some of the outputs.
  const int split = SHARE ? p.split : 1, rank = static_cast<int>(blockIdx.x) % split;
  const int cta = static_cast<int>(blockIdx.x) / split, ctas = static_cast<int>(gridDim.x) / split;
  const int ub0 = et_first_unit(p.ksteps, split, rank);
  const int ksteps = et_first_unit(p.ksteps, split, rank + 1) - ub0, nchunks = (ksteps + kCU - 1) / kCU;
  constexpr int kAcc = SUMS ? kEtSumTok : kEtTok, kA0 = 2 * kEtTok;  // an accumulator's columns, the first A column
  // activation slots and weight stages
  const int lx = et_lx(p.nt, F::kBK), lw = et_lw(p.nt, F::kBK, F::kWBytes);
  const uint32_t nx = 1u << lx, xslot = et_slot_tok(p.nt) * F::kBK * 2;
  const uint32_t nw = 1u << lw, w_ring = sbase + nx * xslot;

  // Every role walks the same stream of units: tile by tile, unit by unit along k.
  if (warp == 0) {
    // ------------------------------------------------------------ activation producer
    if (elect_one()) {
      uint32_t it = 0;
      int e = 0;
      bool ok = true;
      for (int t = cta; ok && t < num_tiles; t += ctas) {
        const EtTile tl = et_tile(p, tb, t, e);
        const int box = et_box(tl.mt);
        const uint32_t bytes = 2u * F::kBK * et_box_rows(box, p.nt);
        for (int u = 0; u < ksteps; ++u, ++it) {
          const uint32_t s = it & (nx - 1);
          ok = et_wait(empty_bar(s), ((it >> lx) & 1u) ^ 1u, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(full_bar(s), bytes);
          tma_load_3d(sbase + s * xslot, &tm.x[box], full_bar(s), 0, tl.m0, (ub0 + u) * (F::kBK / 64));
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
      int e = 0;
      bool ok = true;
      for (int t = cta; ok && t < num_tiles; t += ctas) {
        const EtTile tl = et_tile(p, tb, t, e);
        const uint32_t ncols = static_cast<uint32_t>((tl.mt + 15) & ~15);
        const uint32_t idesc = make_idesc_f16(0u, kEtRows, ncols);
        const uint32_t half = 128u * et_box_rows(et_box(tl.mt), p.nt);  // bytes of a k block's box
        uint32_t d_tmem = 0;
        for (int u = 0; u < ksteps; ++u, ++it) {
          const bool first = u == 0 || (SUMS && u % kSeg == 0);  // of an accumulator segment
          if (first) {
            if (SUMS && u > 0) mma_commit(accfull_bar(sc++ & 1u));
            ok = et_wait(accempty_bar(sc & 1u), ((sc >> 1) & 1u) ^ 1u, abort_flag);
            if (!ok) break;
            d_tmem = tmem_base + (sc & 1u) * kAcc;
          }
          const uint32_t s = it & (nx - 1);
          const uint32_t xs = sbase + s * xslot;
          const uint64_t b0 = smem_desc_sw128(xs);
          const uint64_t b1 = SPLIT ? b0 : smem_desc_sw128(xs + half);  // SPLIT: the low parts meet the same x
          ok = et_wait(full_bar(s), (it >> lx) & 1u, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t a_tmem = tmem_base + kA0 + (it & ((1u << kEtLA) - 1)) * 64;
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            mma_f16_ts(d_tmem, a_tmem + 8u * kk, (kk < 4 ? b0 : b1) + 2u * (kk & 3), idesc,
                       (kk > 0 || !first) ? 1u : 0u);
          mma_commit(empty_bar(s));
        }
        if (ok) mma_commit(accfull_bar(sc++ & 1u));
      }
      mma_commit(drain_bar);
      mbar_wait_drain(drain_bar, 0u);
    }
  } else if (warp == kEtWProdWarp) {
    // ------------------------------------------------------------ packed-weight producer
    if (elect_one()) {
      uint32_t it = 0;
      int e = 0;
      bool ok = true;
      for (int t = cta; ok && t < num_tiles; t += ctas) {
        const EtTile tl = et_tile(p, tb, t, e);
        const int row = tl.e * p.N + tl.n0;
        for (int u = 0; u < ksteps; ++u, ++it) {
          const uint32_t w = it & (nw - 1);
          ok = et_wait(wempty_bar(w), ((it >> lw) & 1u) ^ 1u, abort_flag);
          if (!ok) break;
          mbar_arrive_expect_tx(wfull_bar(w), F::kWBytes);
          tma_load_2d(w_ring + w * F::kWBytes, &tm.w, wfull_bar(w), (ub0 + u) * F::kWqRowBytes, row);
        }
      }
      for (uint32_t j = (it > nw ? it - nw : 0); j < it; ++j) mbar_wait_drain(wfull_bar(j & (nw - 1)), (j >> lw) & 1u);
    }
  } else if (warp == kEtScaleWarp) {
    // ------------------------------------------------------------ scales -> shared memory
    // A row's scales of a chunk are 32 (Q2) or 64 neighbouring bytes, so a warp's copy of 32
    // words touches 4 or 2 lines.  (One thread per weight row reading its own scale each unit
    // touches 32, 32 cycles of the load unit per warp and unit, which bound the kernel.)
    // Asynchronous copies, as far ahead as the buffers go.
    constexpr int kW = F::kScWords, kR = 32 / kW;  // words of a row, rows a copy takes
    const int wd = lane % kW, rl = lane / kW;
    const int kb0 = ub0 * kEtChunk / kCU;          // the first unit's block
    // pairs of Q2 scales are words only where the rows start on words
    const bool words = FMT == 1 || ((p.nblocks & 1) == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 3) == 0);
    uint32_t cidx = 0;
    int e = 0;
    bool ok = true;
    for (int t = cta; t < num_tiles; t += ctas) {
      const EtTile tl = et_tile(p, tb, t, e);
      const int rows = min(kEtRows, p.N - tl.n0);
      const int64_t row0 = static_cast<int64_t>(tl.e) * p.N + tl.n0 + rl;
      for (int c = 0; c < nchunks; ++c, ++cidx) {
        const uint32_t b = cidx % kEtScBufs;
        const int k = kb0 + c * kEtChunk + wd * (kEtChunk / kW);  // the word's (first) block
        const uint32_t off = F::kScOff + b * F::kScBytes + wd * F::kScPitch + 4 * rl;
        ok = et_wait_warp(sempty_bar(b), ((cidx / kEtScBufs) & 1u) ^ 1u, abort_flag) && ok;
        if (!ok) continue;
        if (words) {
          // rows past N and blocks past K: zeros, no weight
          const uint32_t* src = reinterpret_cast<const uint32_t*>(p.scales) + (row0 * p.nblocks + k) / (FMT == 0 ? 2 : 1);
          const int64_t step = static_cast<int64_t>(kR) * p.nblocks / (FMT == 0 ? 2 : 1);
#pragma unroll 8
          for (int r = 0; r < kEtRows; r += kR, src += step) {
            const bool in = r + rl < rows && k < p.nblocks;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(sbase + off + 4 * r),
                         "l"(in ? static_cast<const void*>(src) : static_cast<const void*>(p.scales)), "r"(in ? 4u : 0u)
                         : "memory");
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(sfull_bar(b)) : "memory");
        } else {
#pragma unroll 8
          for (int r = 0; r < kEtRows; r += kR) {
            uint32_t v = 0u;
            if (r + rl < rows) {
              const uint16_t* src = p.scales + (row0 + r) * p.nblocks + k;
              if (k < p.nblocks) v = ld_scale(src);
              if (k + 1 < p.nblocks) v |= static_cast<uint32_t>(ld_scale(src + 1)) << 16;
            }
            *reinterpret_cast<uint32_t*>(smem + off + 4 * r) = v;
          }
          mbar_arrive(sfull_bar(b));
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  } else if (warp < kEtEpiWarp0) {
    // ------------------------------------------------------------ dequantizers
    // Group grp takes every third unit of the stream; each of its threads unpacks one weight
    // row's codes of the unit.
    const int q = warp & 3;                        // TMEM lane quarter
    const int grp = (warp - kEtDeqWarp0) >> 2;
    const int rt = 32 * q + lane;                  // weight row within the tile
    const uint32_t a_lane = tmem_base + (static_cast<uint32_t>(32 * q) << 16) + kA0;
    const uint32_t w_mine = w_ring + rt * F::kWqRowBytes;
    const uint8_t* s_mine = smem + F::kScOff + 4 * rt;
    // 16-byte chunk c of the row sits at chunk c ^ swz (TMA's 32- or 64-byte swizzle)
    const uint32_t swz = F::kWqRowBytes == 32 ? (rt >> 2) & 1 : (rt >> 1) & 3;
    const int my_tiles = num_tiles > cta ? (num_tiles - cta + ctas - 1) / ctas : 0;
    uint32_t i = grp, i0 = 0, cidx = 0;  // the group's next unit; the chunk's first; chunks
    bool ok = true;
    for (int t = 0; t < my_tiles; ++t)
    for (int c = 0; c < nchunks; ++c, ++cidx) {
      const uint32_t i1 = i0 + min(kCU, ksteps - c * kCU);
      const uint32_t sb = cidx % kEtScBufs;
      const uint8_t* s_chunk = s_mine + sb * F::kScBytes;
      // also when none of the units is ours: the release below must not run ahead of the fill
      ok = et_wait_warp(sfull_bar(sb), (cidx / kEtScBufs) & 1u, abort_flag) && ok;
      for (; i < i1; i += kEtGroups) {
        const uint32_t m = i - i0, w = i & (nw - 1);
        const uint32_t a_dst = a_lane + (i & ((1u << kEtLA) - 1)) * 64;
        // the unit's A stage is free once the unit that had it before is multiplied
        auto slot_wait = [&]() {
          constexpr uint32_t kBack = 1u << kEtLA;
          const uint32_t j = i - kBack;
          if (i >= kBack) ok = et_wait_warp(empty_bar(j & (nx - 1)), (j >> lx) & 1u, abort_flag) && ok;
          tc_fence_after();
        };
        {
          constexpr int kChunks = F::kWqRowBytes / 16;      // 16 bytes of codes each
          constexpr int kRegs = FMT == 0 ? 32 : 16;         // f16 pairs of a chunk
          const uint32_t src = w_mine + w * F::kWBytes;
          constexpr int kSc = FMT == 1 && !SPLIT ? 2 : 1;   // scale words
          uint32_t sc[kSc];
          if (FMT == 0) {
            sc[0] = *reinterpret_cast<const uint32_t*>(s_chunk + (m >> 1) * F::kScPitch);
            sc[0] = m & 1 ? sc[0] >> 16 : sc[0] & 0xFFFFu;
          } else {
#pragma unroll
            for (int k = 0; k < kSc; ++k) sc[k] = *reinterpret_cast<const uint32_t*>(s_chunk + (kSc * m + k) * F::kScPitch);
          }
          const bool exact = SPLIT && __all_sync(0xFFFFFFFFu, q4_zero_exact(sc[0] >> 16));
          ok = et_wait_warp(wfull_bar(w), (i >> lw) & 1u, abort_flag) && ok;
          uint4 cw[kChunks];
#pragma unroll
          for (int k = 0; k < kChunks; ++k) cw[k] = ld_shared_v4(src + ((k ^ swz) << 4));
          // the slot is refilled by TMA (the async proxy) once the group has released it
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(wempty_bar(w));
#pragma unroll
          for (int k = 0; k < kChunks; ++k) {
            const uint32_t wd[4] = {cw[k].x, cw[k].y, cw[k].z, cw[k].w};
            uint32_t o[kRegs];
            const uint32_t s1 = sc[kSc == 1 ? 0 : k >> 1];
            const uint32_t s2 = (s1 & 0xFFFFu) | (s1 << 16);
            uint32_t lo[SPLIT ? kRegs : 1];
            (void)lo;
            if constexpr (SPLIT) {
              const uint32_t z2 = (s1 >> 16) | (s1 & 0xFFFF0000u);
              if (exact) {
#pragma unroll
                for (int j = 0; j < 4; ++j) q4_word_split<true>(wd[j], s2, z2, o + 4 * j, lo + 4 * j);
              } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) q4_word_split<false>(wd[j], s2, z2, o + 4 * j, lo + 4 * j);
              }
            } else if (FMT == 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j) q2_word_to_f16(wd[j], s2, o + 8 * j);
            } else {
              const Q4Centre ce = q4_centre(s2, (s1 >> 16) | (s1 & 0xFFFF0000u));
#pragma unroll
              for (int j = 0; j < 4; ++j) q4_word_centred(wd[j], s2, ce, o + 4 * j);
            }
            if (k == 0) slot_wait();
            if constexpr (kRegs == 32)
              tmem_st_32x32b_x32(a_dst + 32 * k, o);
            else
              tmem_st_32x32b_x16(a_dst + 16 * k, o);
            if constexpr (SPLIT) tmem_st_32x32b_x16(a_dst + 32 + 16 * k, lo);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(full_bar(i & (nx - 1)));
      }
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(sempty_bar(sb));
      i0 = i1;
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
      if (lane == 0 && ok) mbar_arrive(accempty_bar(ab));
    };
    for (int t = cta; t < num_tiles; t += ctas) {
      const EtTile tl = et_tile(p, tb, t, e);
      const int n = tl.n0 + 32 * q + lane;       // this thread's weight row
      const bool nv = n < p.N;
      float bias = 0.f, gate_n = 1.f;
      if (a.bias && nv) bias = ep_load(a.bias, static_cast<int64_t>(tl.e) * p.N + n, a.bias_f32);
      if (a.gate && !a.gate_rows && nv) gate_n = bf16_bits_to_f32(a.gate[n]);
      // While the tile is multiplied, its gates and residuals come into L2: a lane a token, this
      // warp's 32 weight rows (64 or 128 bytes), tokens shared between the two sets.
      if (n - lane < p.N) {
        for (int k = lane + 32 * set; k < tl.mt; k += 64) {
          const int64_t i = static_cast<int64_t>(tl.m0 + k) * p.N + n - lane;
          if (a.gate && a.gate_rows) prefetch_l2(a.gate + i);
          if (a.residual)
            prefetch_l2(a.residual_f32 ? static_cast<const void*>(static_cast<const float*>(a.residual) + i)
                                       : static_cast<const void*>(static_cast<const uint16_t*>(a.residual) + i));
        }
      }
      // The outputs of the kN tokens from token m of the tile on, whose sums f gets from sums().
      // Loads are unconditional, from clamped places: a load behind a branch of its own is waited
      // for before the next one (13000 cycles a chunk instead of 700).  bf16 outputs leave in
      // pairs: neighbouring lanes trade, so that one has (n, n + 1) of an even token and the
      // other of the odd one.
      const int64_t tile0 = static_cast<int64_t>(tl.m0) * p.N;
      auto finish = [&](auto& f, int m, auto&& sums) {
        constexpr int kN = sizeof(f) / sizeof(float);
        const int mt = min(kN, tl.mt - m);
        const int64_t row0 = tile0 + static_cast<uint32_t>(m) * static_cast<uint32_t>(p.N);
        const int64_t i0 = row0 + (nv ? n : p.N - 1);
        auto at = [&](int i) { return static_cast<uint32_t>(min(i, mt - 1)) * static_cast<uint32_t>(p.N); };
        uint16_t g[kN];
        uint32_t r[kN];
        if (a.gate && a.gate_rows) {
          const uint16_t* src = a.gate + i0;
#pragma unroll
          for (int i = 0; i < kN; ++i) g[i] = src[at(i)];
        }
        if (a.residual) {
          if (a.residual_f32) {
            const uint32_t* src = static_cast<const uint32_t*>(a.residual) + i0;
#pragma unroll
            for (int i = 0; i < kN; ++i) r[i] = src[at(i)];
          } else {
            const uint16_t* src = static_cast<const uint16_t*>(a.residual) + i0;
#pragma unroll
            for (int i = 0; i < kN; ++i) r[i] = src[at(i)];
          }
        }
        sums();
#pragma unroll
        for (int i = 0; i < kN; ++i) f[i] += bias;
        ep_act_all(f, a.act);
        if (a.gate) {
          if (a.gate_rows) {
#pragma unroll
            for (int i = 0; i < kN; ++i) f[i] *= bf16_bits_to_f32(g[i]);
          } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) f[i] *= gate_n;
          }
        }
        if (a.residual) {
          if (a.residual_f32) {
#pragma unroll
            for (int i = 0; i < kN; ++i) f[i] += __uint_as_float(r[i]);
          } else {
#pragma unroll
            for (int i = 0; i < kN; ++i) f[i] += __uint_as_float(r[i] << 16);
          }
        }
        if (a.out_f32) {
          float* dst = static_cast<float*>(a.y) + i0;
          if (nv && mt == kN) {
#pragma unroll
            for (int i = 0; i < kN; ++i) dst[static_cast<uint32_t>(i) * static_cast<uint32_t>(p.N)] = f[i];
          } else if (nv) {
#pragma unroll
            for (int i = 0; i < kN; ++i)
              if (i < mt) dst[at(i)] = f[i];
          }
        } else if ((p.N & 1) == 0) {
          const int odd = lane & 1;
          uint32_t v[kN / 2];
#pragma unroll
          for (int i = 0; i < kN / 2; ++i) {
            const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? f[2 * i] : f[2 * i + 1], 1);
            v[i] = odd ? pack_bf16x2(got, f[2 * i + 1]) : pack_bf16x2(f[2 * i], got);
          }
          // both lanes of a pair are inside N, or neither
          uint16_t* dst = static_cast<uint16_t*>(a.y) + row0 + (n - odd) + (odd ? p.N : 0);
          if (nv && mt == kN) {
#pragma unroll
            for (int i = 0; i < kN / 2; ++i)
              *reinterpret_cast<uint32_t*>(dst + static_cast<uint32_t>(2 * i) * static_cast<uint32_t>(p.N)) = v[i];
          } else if (nv) {
#pragma unroll
            for (int i = 0; i < kN / 2; ++i)
              if (2 * i + odd < mt)
                *reinterpret_cast<uint32_t*>(dst + static_cast<uint32_t>(2 * i) * static_cast<uint32_t>(p.N)) = v[i];
          }
        } else if (nv) {
          __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(a.y) + i0;
#pragma unroll
          for (int i = 0; i < kN; ++i)
            if (i < mt) dst[at(i)] = __float2bfloat16_rn(f[i]);
        }
      };
      const int chunks = (tl.mt + 15) >> 4;
      if constexpr (SUMS) {
        // running sums of this set's chunks += a segment, rounded to nearest; the whole sums go
        // back into the last segment's accumulator
        constexpr int kMine = (kEtSumTok / 16 + 1) / 2;
        float sum[kMine][16];
#pragma unroll
        for (int k = 0; k < kMine; ++k)
#pragma unroll
          for (int i = 0; i < 16; ++i) sum[k][i] = 0.f;
#pragma unroll 1
        for (int u = 0; u < ksteps; u += kSeg) {
          const uint32_t ab = sc & 1u, tsrc = t_lane + ab * kAcc + 16 * set;
          ok = et_wait_warp(accfull_bar(ab), (sc >> 1) & 1u, abort_flag) && ok;
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < kMine; ++k) {
            if (2 * k + set >= chunks) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t v[8];
              tmem_ld_32x32b_x8(tsrc + 32 * k + 8 * h, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 8; ++i) sum[k][8 * h + i] += __uint_as_float(v[i]);
            }
          }
          if (u + kSeg < ksteps) {
            release(ab);
            ++sc;
          }
        }
        const uint32_t tdst = t_lane + (sc & 1u) * kAcc + 16 * set;
#pragma unroll
        for (int k = 0; k < kMine; ++k) {
          if (2 * k + set >= chunks) break;
          uint32_t v[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(sum[k][i]);
          tmem_st_32x32b_x16(tdst + 32 * k, v);
        }
        tmem_wait_st();
      }
      {
        const uint32_t ab = sc & 1u;
        auto accumulated = [&] {
          if (SUMS) return;
          ok = et_wait_warp(accfull_bar(ab), (sc >> 1) & 1u, abort_flag) && ok;
          tc_fence_after();
        };
        // Chunk cc of a shared tile belongs to CTA cc % split.  Once the cluster is done with its
        // rings, each CTA puts its sums of the chunk there, and the owner adds them in CTA order.
        const int first = rank + split * set, step = 2 * split;
        const uint32_t part = 4u * (32 * q + lane);  // [chunk / split][CTA][16 tokens][128 rows]
        if constexpr (SHARE) {
          accumulated();
          cluster_sync();
          for (int cc = set; cc < chunks; cc += 2) {
            const int own = cc % split;
            const uint32_t dst = sbase + part + 8192u * static_cast<uint32_t>(cc - own + rank);
            uint32_t v[16];
            tmem_ld_32x32b_x16(t_lane + ab * kAcc + 16 * cc, v);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) st_cluster_f32(dst + 512u * i, own, __uint_as_float(v[i]));
          }
          cluster_sync();
        }
        if (first >= chunks) {
          if (!SHARE) accumulated();
          release(ab);
        }
        for (int cc = first; cc < chunks; cc += step) {
          float f[16];
          finish(f, 16 * cc, [&] {
            if constexpr (SHARE) {
              const float* src = reinterpret_cast<const float*>(smem + part + 8192u * static_cast<uint32_t>(cc - rank));
#pragma unroll
              for (int i = 0; i < 16; ++i) f[i] = src[128 * i];
              for (int r = 1; r < split; ++r) {
                src += 2048;
#pragma unroll
                for (int i = 0; i < 16; ++i) f[i] += src[128 * i];
              }
            } else {
              if (cc == set) accumulated();  // the first chunk's operands are on their way already
              uint32_t v[16];
              tmem_ld_32x32b_x16(t_lane + ab * kAcc + 16 * cc, v);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[i]);
            }
            if (cc + step >= chunks) release(ab);  // the accumulator is read out
          });
        }
        ++sc;
      }
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  // With the epilogue warps of the cluster: rings free, sums there.  Each thread of a cluster comes
  // to both barriers once: the grid of a shared call has one cluster for each tile.
  if (SHARE && warp < kEtEpiWarp0) {
    cluster_sync();
    cluster_sync();
  }
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
__global__ void __launch_bounds__(256) ep_prep_kernel(const uint16_t* x, uint16_t* x16, const int* rows,
                                                      const int* offsets, int E, int x_rows, int R, int K) {
  if (offsets) {
    pdl_wait();  // the matmul reads the offsets as soon as it may start
    pdl_trigger();
  } else {
    pdl_trigger_and_wait();
  }
  const int lim = offsets ? min(max(offsets[E], 0), R) : R;
  const int gk = K / 16;
  const int64_t total = static_cast<int64_t>(lim) * gk;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t r = i / gk;
    const int g = static_cast<int>(i - r * gk);
    int64_t src = r;
    if (rows) src = rows[r];
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    if (src >= 0 && src < x_rows) {
      const uint4* xp = reinterpret_cast<const uint4*>(x + src * K) + 2 * g;
      a = xp[0];
      b = xp[1];
    }
    x16_group<FMT>(a, b, reinterpret_cast<uint4*>(x16 + r * K) + 2 * g);
  }
}

}  // namespace tgemm
