// expert.cuh -- the expert sort (the grouped matmul's plan) and the expert combine.
#pragma once

#include "common.cuh"
#include "epilogue.cuh"

namespace tgemm {

// ---- expert sort -------------------------------------------------------------------------
// A stable counting sort of n (token, choice) pairs by expert.  The pairs are cut into one
// contiguous run per warp (warp w of CTA g takes run 32 g + w), so a pair's place is
//   start of its expert + pairs of that expert in earlier runs + earlier ones in its own run,
// which needs no atomics on global memory and does not depend on timing.
constexpr int kSortWarps = 32;

struct SortParams {
  const int* ids;
  int* offsets;  // [E + 1]
  int* rows;     // [n] source token of each sorted row, -1 behind the last
  int* pos;      // [n] sorted row of each pair, -1 for an id outside [0, E)
  int* hist;     // [G][E] pairs of each CTA by expert (G > 1)
  int n, k, E, run;  // run: pairs per warp
};

__device__ __forceinline__ void sort_run_bounds(const SortParams& p, int cta, int warp, int& lo, int& hi) {
  const int64_t a = (static_cast<int64_t>(cta) * kSortWarps + warp) * p.run;
  lo = static_cast<int>(a < p.n ? a : p.n);
  hi = static_cast<int>(a + p.run < p.n ? a + p.run : p.n);
}

// The warp's pairs by expert, added into cnt[e] (the warp's own counters).
__device__ __forceinline__ void sort_count(const SortParams& p, int lo, int hi, int* cnt) {
  const int lane = threadIdx.x & 31;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    int id = i < hi ? __ldg(p.ids + i) : -1;
    if (id >= p.E) id = -1;
    if (id < 0) id = -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
    if (id >= 0 && lane == __ffs(same) - 1) cnt[id] += __popc(same);
    __syncwarp();
  }
}

__global__ void __launch_bounds__(kSortWarps * 32) sort_count_kernel(const SortParams p) {
  extern __shared__ int st_cnt[];  // [E]
  pdl_trigger_and_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) st_cnt[e] = 0;
  __syncthreads();
  int lo, hi;
  sort_run_bounds(p, blockIdx.x, warp, lo, hi);
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    int id = i < hi ? __ldg(p.ids + i) : -1;
    if (id >= p.E || id < 0) id = -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
    if (id >= 0 && lane == __ffs(same) - 1) atomicAdd(st_cnt + id, __popc(same));
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.E; e += blockDim.x)
    p.hist[static_cast<int64_t>(blockIdx.x) * p.E + e] = st_cnt[e];
}

// Places the CTA's pairs.  With one CTA (G = 1) it needs no counts from before.
__global__ void __launch_bounds__(kSortWarps * 32) sort_place_kernel(const SortParams p) {
  extern __shared__ int st_base[];  // [warps][E], then the experts' starts [E + 1]
  __shared__ int part[kSortWarps];
  int* start = st_base + kSortWarps * p.E;
  pdl_trigger_and_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = gridDim.x, g = blockIdx.x;
  for (int i = tid; i < kSortWarps * p.E; i += blockDim.x) st_base[i] = 0;
  __syncthreads();
  int lo, hi;
  sort_run_bounds(p, g, warp, lo, hi);
  sort_count(p, lo, hi, st_base + warp * p.E);
  __syncthreads();
  // E <= blockDim.x: thread e owns expert e
  int total = 0, before = 0;
  if (tid < p.E) {
    if (G > 1) {
      for (int c = 0; c < G; ++c) {
        const int v = __ldg(p.hist + static_cast<int64_t>(c) * p.E + tid);
        total += v;
        if (c < g) before += v;
      }
    } else {
      for (int w = 0; w < kSortWarps; ++w) total += st_base[w * p.E + tid];
    }
  }
  int incl = total;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int o = __shfl_up_sync(0xFFFFFFFFu, incl, s);
    if (lane >= s) incl += o;
  }
  if (lane == 31) part[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int v = part[lane];
#pragma unroll
    for (int s = 1; s < 32; s <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, v, s);
      if (lane >= s) v += o;
    }
    part[lane] = v;
  }
  __syncthreads();
  if (warp > 0) incl += part[warp - 1];
  if (tid < p.E) {
    int at = incl - total + before;
    for (int w = 0; w < kSortWarps; ++w) {
      const int v = st_base[w * p.E + tid];
      st_base[w * p.E + tid] = at;
      at += v;
    }
    if (tid == p.E - 1) start[0] = incl;  // pairs kept in all
    if (g == 0) {
      p.offsets[tid] = incl - total;
      if (tid == p.E - 1) p.offsets[p.E] = incl;
    }
  }
  __syncthreads();
  int* base = st_base + warp * p.E;
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    int id = i < hi ? __ldg(p.ids + i) : -1;
    if (id >= p.E || id < 0) id = -1;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, id);
    int at = -1;
    if (id >= 0) at = base[id] + __popc(same & ((1u << lane) - 1u));
    __syncwarp();
    if (id >= 0 && lane == __ffs(same) - 1) base[id] += __popc(same);
    __syncwarp();
    if (i < hi) {
      p.pos[i] = at;
      if (at >= 0) p.rows[at] = i / p.k;
    }
  }
  // rows behind the last expert's
  for (int64_t i = start[0] + static_cast<int64_t>(g) * blockDim.x + tid; i < p.n; i += static_cast<int64_t>(G) * blockDim.x)
    p.rows[i] = -1;
}

// ---- expert combine ----------------------------------------------------------------------
//   y[t] = residual[t] + sum_j weights[t][j] h[pos[t][j]],  pairs with pos outside [0, R) left out
// in f32, in the order of j.  Bound by reading h once.
struct CombineParams {
  const void* h;
  const int* pos;
  const float* weights;
  const void* residual;
  void* y;
  int T, k, N, R;
  int residual_f32, out_f32;
};

template <bool HF32>
__global__ void __launch_bounds__(256) combine_kernel(const CombineParams p) {
  pdl_trigger_and_wait();
  const int64_t total = static_cast<int64_t>(p.T) * p.N;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * blockDim.x;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const int64_t t = i / p.N;
    const int n = static_cast<int>(i - t * p.N);
    float v = 0.f;
    for (int j = 0; j < p.k; ++j) {
      const int r = __ldg(p.pos + t * p.k + j);
      if (r < 0 || r >= p.R) continue;
      v = fmaf(__ldg(p.weights + t * p.k + j), ep_load(p.h, static_cast<int64_t>(r) * p.N + n, HF32), v);
    }
    if (p.residual)
      v += p.residual_f32 ? static_cast<const float*>(p.residual)[i]
                          : bf16_bits_to_f32(static_cast<const uint16_t*>(p.residual)[i]);
    if (p.out_f32)
      static_cast<float*>(p.y)[i] = v;
    else
      static_cast<__nv_bfloat16*>(p.y)[i] = __float2bfloat16_rn(v);
  }
}

}  // namespace tgemm
