// ep_host.cuh -- host side of the epilogue and expert matmuls, the expert sort and combine:
// argument checks, workspace layout, dispatch.  Part of tgemm.cu (uses its launch helpers).
#pragma once

namespace tgemm {
namespace {

// [a, a + na) and [b, b + nb) share a byte.
bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + nb && y < x + na;
}

// Let a kernel use `bytes` of dynamic shared memory, once per device (`done`: a bit for each).
template <typename Kernel>
int allow_smem(Kernel kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return TGEMM_ECUDA;
  const uint64_t bit = uint64_t{1} << dev;
  if (done.load(std::memory_order_acquire) & bit) return TGEMM_OK;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) return TGEMM_ECUDA;
  done.fetch_or(bit, std::memory_order_release);
  return TGEMM_OK;
}
static_assert(kMaxDevices <= 64, "a bit for each device");

struct EpCall {
  int fmt;
  const uint16_t* x;
  const uint8_t* wq;
  const uint16_t* scales;
  const int* offsets;  // null: dense
  const int* rows;
  int E, x_rows, R, N, K;
  const tgemm_epilogue* ep;
  void* y;
  int out_dtype;
  void* workspace;
  size_t ws_bytes;
  void* stream;
};

bool dtype_ok(int dt) { return dt == TGEMM_OUT_F32 || dt == TGEMM_OUT_BF16; }

// Workspace of the tensor-core path: the f16 copy of the activations.
size_t ep_ws_bytes(int R, int K) { return round_up(static_cast<size_t>(R) * K * 2, 256); }

// The most row chunks of `nt` that R rows in E groups can make (one group: exactly those).
int64_t max_chunks(int R, int E, int nt) {
  return (R + static_cast<int64_t>(std::min(R, E)) * (nt - 1)) / nt;
}

// Tokens per tile and CTAs per tile of a dense call: the pair whose fullest CTA has the least to
// do.  A unit costs 4 cycles per token on the tensor core, and no less than 350, which the
// dequantizers need (0.27 us in all).  Few tiles leave SMs idle, so that clusters of up to 8 CTAs
// share the units of one.  Meeting costs them 2 to 3 us and more with each; another 2 us where the
// clusters nearly fill the device, since one starts when an SM is free for each of its CTAs.
// Measured (us, chains of calls, by CTAs a tile):
//   17 x 2560 x 9728 ternary, 20 tiles: 1 27.3, 2 19.8, 3 16.5, 4 15.0, 5 14.5, 6 14.3
//   17 x 2560 x 2560 ternary, 20 tiles: 1 11.1, 2 10.5, 3 9.9, 4 9.6, 5 9.7, 6 10.0
//   256 x 1408 x 2048 ternary, 44 tiles (of 45 clusters of 3): 1 11.5, 2 11.8, 3 14.4
//   17 x 2560 x 9728 4-bit, f32 y, 20 tiles: 1 51.5, 2 31.7, 3 25.1, 4 21.4, 5 19.7, 6 18.8
struct EtPlan {
  int nt, split;
};
template <typename Held>  // held(s): clusters of s CTAs that the device runs at once
EtPlan et_plan(int M, int tiles_n, int units, int most, int sms, Held&& held) {
  EtPlan best{most, 1};
  int64_t best_cost = INT64_MAX;
  for (int nt = 16; nt <= most; nt += 16) {
    const int64_t tiles = static_cast<int64_t>((M + nt - 1) / nt) * tiles_n;
    const int64_t unit = std::max(4 * nt, 350);
    const int64_t cost = (tiles + sms - 1) / sms * units * unit;
    if (cost <= best_cost) {
      best_cost = cost;
      best = {nt, 1};
    }
    for (int s = 2; s <= kEtMaxSplit && tiles * s <= sms && 4 * s <= units; ++s) {
      int64_t c = static_cast<int64_t>((units + 2 * s - 1) / (2 * s)) * 2 * unit + 3600 + 400 * (s - 2);
      if (c >= best_cost) continue;
      const int64_t n = held(s);
      if (5 * tiles > 4 * n) c += 2600;
      if (c < best_cost && tiles <= n) {
        best_cost = c;
        best = {nt, s};
      }
    }
  }
  return best;
}

template <int FMT, bool SPLIT, bool SUMS>
int launch_ep_tc(const EpCall& c, EtParams p, int sms, cudaStream_t st) {
  using F = EtFmt<FMT, SPLIT>;
  static std::atomic<uint64_t> done{0};
  static std::atomic<uint64_t> done_share{0};
  if (int e = allow_smem(ep_tc_kernel<FMT, SPLIT, SUMS, false>, F::kSmemBytes, done)) return e;
  if (int e = allow_smem(ep_tc_kernel<FMT, SPLIT, SUMS, true>, F::kSmemBytes, done_share)) return e;
  p.ksteps = (c.K + F::kBK - 1) / F::kBK;
  constexpr int kMost = SUMS ? kEtSumTok : kEtTok;  // tokens of a tile
  p.split = 1;
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {1, 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = kEtThreads;
  cfg.dynamicSmemBytes = F::kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  if (c.offsets) {
    // Room for twice an expert's rows on average, of which 32 or 64 leave shared memory for more
    // weights on their way (an expert with more rows takes more tiles).
    const int64_t twice = 2 * static_cast<int64_t>(c.R) / c.E;
    p.nt = twice <= 32 ? 32 : twice <= 64 ? 64 : kMost;
  } else {
    // clusters of s that the current device holds at once, asked once (0: not yet)
    static std::atomic<int> held[kMaxDevices][kEtMaxSplit + 1];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return TGEMM_ECUDA;
    const EtPlan plan = et_plan(c.R, p.tiles_n, p.ksteps, kMost, sms, [&](int s) {
      int n = held[dev][s].load(std::memory_order_relaxed);
      if (n == 0) {
        cudaLaunchConfig_t q = cfg;
        q.gridDim = s * sms;
        attr[1].val.clusterDim.x = s;
        q.attrs = attr + 1;
        q.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, ep_tc_kernel<FMT, SPLIT, SUMS, true>, &q) != cudaSuccess || n < 1) {
          cudaGetLastError();
          n = -1;
        }
        held[dev][s].store(n, std::memory_order_relaxed);
      }
      return n;
    });
    const int tt = (c.R + plan.nt - 1) / plan.nt;
    p.nt = ((c.R + tt - 1) / tt + 15) & ~15;  // the step that the kernel takes
    p.split = plan.split;
  }
  // the most tiles there can be: an expert with rows has at most one partly filled tile
  const int64_t tiles = max_chunks(c.R, c.E, p.nt) * p.tiles_n;
  if (tiles > INT32_MAX / 2) return TGEMM_ETOOLARGE;
  // a shared call has exactly one cluster a tile: the kernel's cluster barriers count on it
  attr[1].val.clusterDim.x = static_cast<unsigned>(p.split);
  cfg.numAttrs = p.split > 1 ? 2 : 1;
  cfg.gridDim = static_cast<unsigned>(p.split > 1 ? tiles * p.split : std::min<int64_t>(tiles, sms));
  EtMaps tm;
  PFN_cuTensorMapEncodeTiled_v12000 enc;
  if (int e = encoder(&enc)) return e;
  for (int i = 0; i < kEtBoxes; ++i) {
    // the boxes that tiles of up to nt tokens use; a dense call has full tiles and one rest
    const int lo = i ? et_box_most(i - 1) : 0, hi = et_box_most(i), rest = c.R % p.nt;
    const bool used = c.offsets ? lo < p.nt : (c.R >= p.nt && p.nt > lo && p.nt <= hi) || (rest > lo && rest <= hi);
    if (!used) continue;
    const cuuint64_t dims[3] = {64, static_cast<cuuint64_t>(c.R), static_cast<cuuint64_t>(c.K) / 64};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(c.K) * 2, 128};
    const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(et_box_rows(i, p.nt)), F::kBK / 64};
    const cuuint32_t estr[3] = {1, 1, 1};
    if (enc(&tm.x[i], CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, c.workspace, dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return TGEMM_ECUDA;
  }
  const uint64_t row_bytes = static_cast<uint64_t>(c.K) / (FMT == 0 ? 4 : 2);
  if (int e = make_map_2d(&tm.w, c.wq, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, row_bytes,
                          static_cast<uint64_t>(c.E) * c.N, F::kWqRowBytes, kEtRows,
                          F::kWSwizzle))
    return e;
  return launch(FMT == 0 ? TGEMM_KIND_TC_Q2 : TGEMM_KIND_TC_Q4, st, [&] {
    return p.split > 1 ? cudaLaunchKernelEx(&cfg, ep_tc_kernel<FMT, SPLIT, SUMS, true>, tm, p)
                       : cudaLaunchKernelEx(&cfg, ep_tc_kernel<FMT, SPLIT, SUMS, false>, tm, p);
  });
}

constexpr int kEsMost = 225 * 1024, kEsHalf = 112 * 1024;  // shared memory of one CTA or two on an SM

// CTAs that share the K of an item of the small path (a dense call with few items and long rows):
// a warp's units take 0.6 to 1.4 us each, half more with two CTAs on an SM; meeting takes 1 us and
// a little for each CTA (tenths of a us here).  Measured (us, chains of calls, by CTAs an item):
//   1 x 1408 x 9728 ternary, 44 items: 1 8.7, 2 6.4, 3 5.8, 4 5.6, 6 6.5;  4-bit: 14.1, 8.1, 8.1, 7.1, 7.5
//   1 x 2560 x 9728 ternary, 80 items: 1 9.1, 2 8.5, 3 7.8;  4-bit: 1 15.5, 3 9.7
//   1 x 2560 x 2560 ternary, 80 items: 1 3.8, 2 4.4, 3 4.1
int es_pick_split(int fmt, int T, int U, int64_t items, int sms) {
  const int unit = T == 1 ? (fmt == 0 ? 6 : 9) : (fmt == 0 ? 11 : 14);
  int best = 1, best_cost = 2 * unit * ((U + kEsWarps - 1) / kEsWarps);
  for (int s = 2; s <= kEtMaxSplit; ++s) {
    const int nu = (U + s * kEsWarps - 1) / (s * kEsWarps);
    const int room = es_smem_bytes(fmt, T, true, nu, true, 1, false) <= kEsHalf ? 2 * sms : sms;
    if (10 * items * s > 9 * room) continue;
    const int cost = nu * unit * (items * s > sms ? 3 : 2) + 2 * (10 + 2 * s);
    if (cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

template <int FMT, int T, bool SHARE>
int launch_ep_small(EsParams p, int64_t chunks, int sms, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  if (int e = allow_smem(ep_small_kernel<FMT, T, SHARE>, kEsMost, done)) return e;
  p.tiles_n = (p.N + kEsRows - 1) / kEsRows;
  const int64_t items = chunks * p.tiles_n;
  if (items > INT32_MAX / 2) return TGEMM_ETOOLARGE;
  const bool grouped = p.offsets != nullptr;
  p.nu_max = (p.U + p.split * kEsWarps - 1) / (p.split * kEsWarps);
  p.staged = es_smem_bytes(FMT, T, SHARE, p.nu_max, true, p.E, grouped) <= kEsMost ? 1 : 0;
  const int smem = es_smem_bytes(FMT, T, SHARE, p.nu_max, p.staged != 0, p.E, grouped);
  if (smem > kEsMost) return TGEMM_ETOOLARGE;
  // shared items: exactly one cluster each, which the kernel's cluster barriers count on
  const int grid = SHARE ? static_cast<int>(items) * p.split
                         : static_cast<int>(std::min<int64_t>(items, smem <= kEsHalf ? 2 * sms : sms));
  cudaLaunchAttribute attr[2] = {};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim = {static_cast<unsigned>(p.split), 1, 1};
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = kEsWarps * 32;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = SHARE ? 2 : 1;
  return launch(FMT == 0 ? TGEMM_KIND_GEMV_Q2 : TGEMM_KIND_GEMV_Q4, st, [&] {
    return cudaLaunchKernelEx(&cfg, ep_small_kernel<FMT, T, SHARE>, p);
  });
}

int run_ep_small(const EpCall& c, const EpArgs& a, int sms, cudaStream_t st) {
  EsParams p = {};
  p.N = c.N;
  p.K = c.K;
  p.E = c.E;
  p.R = c.R;
  p.x_rows = c.x_rows;
  p.U = (c.K + 127) / 128;
  p.x = c.x;
  p.wq = c.wq;
  p.scales = c.scales;
  p.offsets = c.offsets;
  p.rows = c.rows;
  p.ep = a;
  const int per = c.offsets ? (c.R + c.E - 1) / c.E : c.R;  // rows of an expert, on average
  const int64_t chunks = max_chunks(c.R, c.E, per <= 8 ? 8 : 16);
  p.split = c.offsets ? 1 : es_pick_split(c.fmt, per <= 8 ? 1 : 2, p.U, chunks * ((c.N + kEsRows - 1) / kEsRows), sms);
  auto go = [&](auto fmt_c) {
    constexpr int kF = decltype(fmt_c)::value;
    if (p.split > 1)
      return per <= 8 ? launch_ep_small<kF, 1, true>(p, chunks, sms, st) : launch_ep_small<kF, 2, true>(p, chunks, sms, st);
    return per <= 8 ? launch_ep_small<kF, 1, false>(p, chunks, sms, st) : launch_ep_small<kF, 2, false>(p, chunks, sms, st);
  };
  return c.fmt == 0 ? go(std::integral_constant<int, 0>{}) : go(std::integral_constant<int, 1>{});
}

constexpr int kEsMaxK = 32768;  // a warp's scales of K fit in shared memory
static_assert(es_smem_bytes(0, 2, false, kEsMaxK / 128 / kEsWarps, false, kEtMaxExperts, true) <= 225 * 1024 &&
                  es_smem_bytes(1, 2, false, kEsMaxK / 128 / kEsWarps, false, kEtMaxExperts, true) <= 225 * 1024,
              "shared memory of the small path");

// Whether the small path serves a call; tgemm_set_path overrides it.  Measured in chains of calls
// (us, small path / tensor path):
//   dense, ternary   8 tokens  9728 x 2560  8.1 / 11.7;  2560 x 9728  8.6 / 14.2;  4-bit 10.0 / 15.4
//                   16 tokens  1408 x 2048  4.7 / 9.7;  2560 x 2560  5.8 / 9.6;  2560 x 4864  8.3 / 11.1;
//                              9728 x 2560 13.3 / 11.6;  2560 x 9728 18.1 / 14.3;  1408 x 9728  8.9 / 12.4
//                   32 tokens  1408 x 2048  5.0 / 10.0;  2560 x 2560  9.9 / 9.8;  4864 x 2560 13.0 / 11.1
//   64 experts 1408 x 2048, ternary: 24 rows 14.4 / 20.3, 192 rows 32.5 / 35.6, 384 rows 41.6 / 36.1
//   8 experts 4864 x 2560, 4-bit: 32 rows 29.7 / 30.2, 64 rows 39.2 / 32.9
// Up to 8 tokens the weights meet one MMA tile of tokens.  Beyond, the small path's time grows with
// weights times chunks of 16 tokens, while the tensor path spreads few tiles over clusters.
bool ep_is_small(int R, int E, int N, int K, bool grouped) {
  const int p = g_path.load();
  if (K > kEsMaxK) return false;
  if (p == TGEMM_PATH_TENSOR) return false;
  if (p != TGEMM_PATH_AUTO) return true;
  if (grouped) return R <= 16 || R <= 4 * E;
  return R <= 8 || (R <= 64 && static_cast<int64_t>((R + 15) / 16) * N * K <= 14 << 20);
}

int run_ep(const EpCall& c) {
  const int kblock = c.fmt == 0 ? 128 : 64;
  if (!c.x || !c.wq || !c.scales || !c.y) return TGEMM_EINVAL;
  if (c.R < 1 || c.x_rows < 1 || c.N < 1 || c.K < kblock || c.K % kblock) return TGEMM_EINVAL;
  if (c.E < 1 || c.E > kEtMaxExperts) return TGEMM_EINVAL;
  if (static_cast<int64_t>(c.E) * c.N > INT32_MAX - kEtRows) return TGEMM_ETOOLARGE;
  if (c.N > (1 << 24)) return TGEMM_ETOOLARGE;  // a tile of y within 32-bit offsets
  if (!dtype_ok(c.out_dtype)) return TGEMM_EINVAL;
  if (!aligned(c.x, 16) || !aligned(c.wq, 16) || !aligned(c.y, 16)) return TGEMM_EALIGN;
  if (!aligned(c.scales, c.fmt == 0 ? 2 : 4)) return TGEMM_EALIGN;
  if (!aligned(c.offsets, 4) || !aligned(c.rows, 4)) return TGEMM_EALIGN;
  const int out_f32 = c.out_dtype == TGEMM_OUT_F32 ? 1 : 0;
  EpArgs a = {};
  a.y = c.y;
  a.out_f32 = out_f32;
  const size_t outs = static_cast<size_t>(c.R) * c.N;
  const size_t y_bytes = outs * (out_f32 ? 4 : 2);
  if (c.ep) {
    const tgemm_epilogue& e = *c.ep;
    if (e.act < TGEMM_ACT_NONE || e.act > TGEMM_ACT_RELU) return TGEMM_EINVAL;
    if (e.bias && !dtype_ok(e.bias_dtype)) return TGEMM_EINVAL;
    if (e.residual && !dtype_ok(e.residual_dtype)) return TGEMM_EINVAL;
    if (e.gate && e.gate_rows != 0 && e.gate_rows != 1) return TGEMM_EINVAL;
    if (e.gate && !e.gate_rows && c.offsets) return TGEMM_EINVAL;
    a.bias = e.bias;
    a.bias_f32 = e.bias_dtype == TGEMM_OUT_F32;
    a.act = e.act;
    a.gate = e.gate;
    a.gate_rows = e.gate_rows;
    a.residual = e.residual;
    a.residual_f32 = e.residual_dtype == TGEMM_OUT_F32;
    if (!aligned(e.bias, a.bias_f32 ? 4 : 2) || !aligned(e.gate, 16) || !aligned(e.residual, 16)) return TGEMM_EALIGN;
    // y may be the residual or the gate (the same elements), but not a part of one
    const size_t res_bytes = outs * (a.residual_f32 ? 4 : 2);
    if (overlaps(c.y, y_bytes, e.residual, e.residual ? res_bytes : 0) &&
        !(e.residual == c.y && a.residual_f32 == out_f32))
      return TGEMM_EINVAL;
    if (overlaps(c.y, y_bytes, e.gate, e.gate ? (e.gate_rows ? outs : c.N) * 2 : 0) &&
        !(static_cast<const void*>(e.gate) == c.y && e.gate_rows && !out_f32))
      return TGEMM_EINVAL;
    if (overlaps(c.y, y_bytes, e.bias, e.bias ? static_cast<size_t>(c.E) * c.N * (a.bias_f32 ? 4 : 2) : 0))
      return TGEMM_EINVAL;
  }
  const size_t wrows = static_cast<size_t>(c.E) * c.N;
  if (overlaps(c.y, y_bytes, c.x, static_cast<size_t>(c.x_rows) * c.K * 2) ||
      overlaps(c.y, y_bytes, c.wq, wrows * (c.K / (c.fmt == 0 ? 4 : 2))) ||
      overlaps(c.y, y_bytes, c.scales, wrows * (c.fmt == 0 ? c.K / 128 * 2 : c.K / 64 * 4)) ||
      overlaps(c.y, y_bytes, c.offsets, c.offsets ? (static_cast<size_t>(c.E) + 1) * 4 : 0) ||
      overlaps(c.y, y_bytes, c.rows, c.rows ? static_cast<size_t>(c.R) * 4 : 0))
    return TGEMM_EINVAL;
  const bool small = ep_is_small(c.R, c.E, c.N, c.K, c.offsets != nullptr);
  const size_t need = small ? 0 : ep_ws_bytes(c.R, c.K);
  if (need && (!c.workspace || c.ws_bytes < need)) return TGEMM_EWORKSPACE;
  if (need && !aligned(c.workspace, 256)) return TGEMM_EALIGN;
  auto in_ws = [&](const void* p, size_t n) { return need && overlaps(c.workspace, need, p, n); };
  if (in_ws(c.y, y_bytes) || in_ws(c.x, static_cast<size_t>(c.x_rows) * c.K * 2) ||
      in_ws(c.wq, wrows * (c.K / (c.fmt == 0 ? 4 : 2))) ||
      in_ws(c.scales, wrows * (c.fmt == 0 ? c.K / 128 * 2 : c.K / 64 * 4)) ||
      in_ws(c.offsets, (static_cast<size_t>(c.E) + 1) * 4) || in_ws(c.rows, static_cast<size_t>(c.R) * 4) ||
      in_ws(a.bias, static_cast<size_t>(c.E) * c.N * (a.bias_f32 ? 4 : 2)) ||
      in_ws(a.gate, (a.gate_rows ? outs : c.N) * 2) || in_ws(a.residual, outs * (a.residual_f32 ? 4 : 2)))
    return TGEMM_EINVAL;
  DeviceInfo di;
  if (int e = current_device_info(&di)) return e;
  const cudaStream_t st = as_stream(c.stream);
  if (small) return run_ep_small(c, a, di.sms, st);

  uint16_t* x16 = static_cast<uint16_t*>(c.workspace);
  const int pgrid = grid_for(static_cast<int64_t>(c.R) * (c.K / 16), 256, di.sms);
  if (int e = launch(TGEMM_KIND_PREP, st, [&] {
        if (c.fmt == 0)
          return pdl_launch(ep_prep_kernel<0>, pgrid, 256, 0, st, c.x, x16, c.rows, c.offsets, c.E, c.x_rows, c.R, c.K);
        return pdl_launch(ep_prep_kernel<1>, pgrid, 256, 0, st, c.x, x16, c.rows, c.offsets, c.E, c.x_rows, c.R, c.K);
      }))
    return e;

  EtParams p = {};
  p.N = c.N;
  p.K = c.K;
  p.E = c.E;
  p.R = c.R;
  p.tiles_n = (c.N + kEtRows - 1) / kEtRows;
  p.nblocks = c.K / (c.fmt == 0 ? 128 : 64);
  p.offsets = c.offsets;
  p.scales = c.scales;
  p.ep = a;
  if (c.fmt == 0) return out_f32 ? launch_ep_tc<0, false, true>(c, p, di.sms, st) : launch_ep_tc<0, false, false>(c, p, di.sms, st);
  return out_f32 ? launch_ep_tc<1, true, true>(c, p, di.sms, st) : launch_ep_tc<1, false, false>(c, p, di.sms, st);
}

// ---- expert sort and combine ---------------------------------------------------------------

constexpr int64_t kSortMaxPairs = int64_t{1} << 26;
// One CTA sorts up to 4096 pairs alone (64 experts: 4092 pairs 6.2 us, 4098 pairs over three CTAs
// 6.9 us).  Beyond that 2048 pairs each, and no more CTAs than keep the table of counts, which
// every CTA reads, at 256 KB (261992 pairs over 1024 experts: 64 CTAs 20.4 us, 144 22.8 us, 32
// 22.7 us; over 128 experts 64 to 144 CTAs take the same time).
constexpr int kSortOneCta = 4096;

int sort_grid(int64_t n, int E) {
  if (n <= kSortOneCta) return 1;
  const int64_t most = std::min<int64_t>(144, 65536 / E);
  return static_cast<int>(std::min<int64_t>((n + 2047) / 2048, most));
}

size_t sort_workspace(int64_t n, int E) {
  const int G = sort_grid(n, E);
  return G > 1 ? round_up(static_cast<size_t>(G) * sort_pitch(E) * 4, 256) : 0;
}

int run_sort(const int* ids, int T, int k, int E, int* offsets, int* rows, int* pos, void* workspace,
             size_t ws_bytes, void* stream) {
  if (!ids || !offsets || !rows || !pos) return TGEMM_EINVAL;
  if (T < 1 || k < 1 || E < 1 || E > kEtMaxExperts) return TGEMM_EINVAL;
  const int64_t n = static_cast<int64_t>(T) * k;
  if (n > kSortMaxPairs) return TGEMM_ETOOLARGE;
  if (!aligned(ids, 4) || !aligned(offsets, 4) || !aligned(rows, 4) || !aligned(pos, 4)) return TGEMM_EALIGN;
  const size_t nb = static_cast<size_t>(n) * 4, ob = (static_cast<size_t>(E) + 1) * 4;
  if (overlaps(rows, nb, ids, nb) || overlaps(pos, nb, ids, nb) || overlaps(offsets, ob, ids, nb) ||
      overlaps(rows, nb, pos, nb) || overlaps(rows, nb, offsets, ob) || overlaps(pos, nb, offsets, ob))
    return TGEMM_EINVAL;
  const size_t need = sort_workspace(n, E);
  if (need && (!workspace || ws_bytes < need)) return TGEMM_EWORKSPACE;
  if (need && !aligned(workspace, 256)) return TGEMM_EALIGN;
  if (need && (overlaps(workspace, need, ids, nb) || overlaps(workspace, need, rows, nb) ||
               overlaps(workspace, need, pos, nb) || overlaps(workspace, need, offsets, ob)))
    return TGEMM_EINVAL;
  DeviceInfo di;
  if (int e = current_device_info(&di)) return e;
  static std::atomic<uint64_t> done{0};
  if (int e = allow_smem(sort_place_kernel, (kSortWarps + 2) * kEtMaxExperts * 4, done)) return e;
  const cudaStream_t st = as_stream(stream);
  const int G = sort_grid(n, E);
  SortParams p;
  p.ids = ids;
  p.offsets = offsets;
  p.rows = rows;
  p.pos = pos;
  p.hist = G > 1 ? static_cast<int*>(workspace) : nullptr;
  p.n = static_cast<int>(n);
  p.k = k;
  p.E = E;
  const int64_t runs = static_cast<int64_t>(G) * kSortWarps;
  p.run = static_cast<int>(((n + runs - 1) / runs + 31) / 32 * 32);
  if (G > 1) {
    if (int e = launch(TGEMM_KIND_PREP, st, [&] {
          return pdl_launch(sort_count_kernel, G, kSortWarps * 32, static_cast<size_t>(E) * 4, st, p);
        }))
      return e;
  }
  return launch(TGEMM_KIND_PREP, st, [&] {
    return pdl_launch(sort_place_kernel, G, kSortWarps * 32, (static_cast<size_t>(kSortWarps) + 2) * E * 4, st, p);
  });
}

int run_combine(const void* h, int h_dtype, const int* pos, const float* weights, const void* residual,
                int residual_dtype, void* y, int T, int k, int N, int R, int out_dtype, void* stream) {
  if (!h || !pos || !weights || !y) return TGEMM_EINVAL;
  if (T < 1 || k < 1 || N < 1 || R < 1) return TGEMM_EINVAL;
  if (!dtype_ok(h_dtype) || !dtype_ok(out_dtype) || (residual && !dtype_ok(residual_dtype))) return TGEMM_EINVAL;
  if (!aligned(h, 16) || !aligned(y, 16) || !aligned(residual, 16) || !aligned(pos, 4) || !aligned(weights, 4))
    return TGEMM_EALIGN;
  const size_t outs = static_cast<size_t>(T) * N;
  const size_t y_bytes = outs * (out_dtype == TGEMM_OUT_F32 ? 4 : 2);
  const size_t pairs = static_cast<size_t>(T) * k * 4;
  if (overlaps(y, y_bytes, h, static_cast<size_t>(R) * N * (h_dtype == TGEMM_OUT_F32 ? 4 : 2)) ||
      overlaps(y, y_bytes, pos, pairs) || overlaps(y, y_bytes, weights, pairs))
    return TGEMM_EINVAL;
  if (residual && overlaps(y, y_bytes, residual, outs * (residual_dtype == TGEMM_OUT_F32 ? 4 : 2)) &&
      !(residual == y && residual_dtype == out_dtype))
    return TGEMM_EINVAL;
  DeviceInfo di;
  if (int e = current_device_info(&di)) return e;
  CombineParams p;
  p.h = h;
  p.pos = pos;
  p.weights = weights;
  p.residual = residual;
  p.y = y;
  p.T = T;
  p.k = k;
  p.N = N;
  p.R = R;
  p.residual_f32 = residual_dtype == TGEMM_OUT_F32;
  p.out_f32 = out_dtype == TGEMM_OUT_F32;
  const cudaStream_t st = as_stream(stream);
  const bool vec = N % 8 == 0;
  const int64_t blocks = (static_cast<int64_t>(T) * (vec ? N / 8 : N) + 255) / 256;
  if (blocks > INT32_MAX) return TGEMM_ETOOLARGE;
  const dim3 grid(static_cast<unsigned>(blocks));
  return launch(TGEMM_KIND_PREP, st, [&] {
    if (h_dtype == TGEMM_OUT_F32)
      return vec ? pdl_launch(combine_kernel<true, 8>, grid, 256, 0, st, p) : pdl_launch(combine_kernel<true, 1>, grid, 256, 0, st, p);
    return vec ? pdl_launch(combine_kernel<false, 8>, grid, 256, 0, st, p) : pdl_launch(combine_kernel<false, 1>, grid, 256, 0, st, p);
  });
}

}  // namespace
}  // namespace tgemm
