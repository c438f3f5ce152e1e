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
//
// Bound by latencies: 261992 pairs over 128 experts are 3 MB, 0.5 us of traffic, and take 9.5 us
// in a chain of calls, two launches (3 us) of which the second has four steps that wait for each
// other (counts of all CTAs, own counts, prefix sums, places); 366 pairs take 3.1 us, one launch.
constexpr int kSortWarps = 32;

struct SortParams {
  const int* ids;
  int* offsets;  // [E + 1]
  int* rows;     // [n] source token of each sorted row, -1 behind the last
  int* pos;      // [n] sorted row of each pair, -1 for an id outside [0, E)
  int* hist;     // [G][sort_pitch(E)] pairs of each CTA by expert (G > 1)
  int n, k, E, run;  // run: pairs per warp
};

__host__ __device__ constexpr int sort_pitch(int E) { return (E + 3) & ~3; }

__device__ __forceinline__ void sort_run_bounds(const SortParams& p, int cta, int warp, int& lo, int& hi) {
  const int64_t a = (static_cast<int64_t>(cta) * kSortWarps + warp) * p.run;
  lo = static_cast<int>(a < p.n ? a : p.n);
  hi = static_cast<int>(a + p.run < p.n ? a + p.run : p.n);
}

// Four batches of 32 pairs: their experts, -1 past the run's end or outside [0, E).
__device__ __forceinline__ void sort_load(const SortParams& p, int i0, int hi, int (&id)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = i0 + 32 * j + lane;
    id[j] = i < hi ? p.ids[i] : -1;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (id[j] < 0 || id[j] >= p.E) id[j] = -1;
}

// The lanes with this lane's expert, for each of four batches: a vote on each bit of the ids (a
// match of the ids takes some 200 cycles a warp, one vote and its two instructions 10).  `bits`
// holds E, so that -1 is no expert.
__device__ __forceinline__ void sort_peers(const int (&id)[4], int bits, uint32_t (&same)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) same[j] = 0xFFFFFFFFu;
  for (int b = 0; b < bits; ++b) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t one = (static_cast<uint32_t>(id[j]) >> b) & 1u;
      same[j] &= __ballot_sync(0xFFFFFFFFu, one) ^ (one - 1u);
    }
  }
}

// Pairs of each CTA by expert.
__global__ void __launch_bounds__(kSortWarps * 32) sort_count_kernel(const SortParams p) {
  extern __shared__ int st_cnt[];  // [E]
  const int warp = threadIdx.x >> 5;
  for (int e = threadIdx.x; e < p.E; e += blockDim.x) st_cnt[e] = 0;
  __syncthreads();
  pdl_trigger_and_wait();
  int lo, hi;
  sort_run_bounds(p, blockIdx.x, warp, lo, hi);
  for (int i0 = lo; i0 < hi; i0 += 128) {
    int id[4];
    sort_load(p, i0, hi, id);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (id[j] >= 0) atomicAdd(st_cnt + id[j], 1);
  }
  __syncthreads();
  const int pitch = sort_pitch(p.E);
  for (int e = threadIdx.x; e < pitch; e += blockDim.x)
    p.hist[static_cast<int64_t>(blockIdx.x) * pitch + e] = e < p.E ? st_cnt[e] : 0;
}

// Places the CTA's pairs.  With one CTA (G = 1) it needs no counts from before.
__global__ void __launch_bounds__(kSortWarps * 32) sort_place_kernel(const SortParams p) {
  extern __shared__ int st_base[];  // [warps][E], then totals [E] and the counts of earlier CTAs [E]
  __shared__ int part[kSortWarps];
  int* s_total = st_base + kSortWarps * p.E;
  int* s_before = s_total + p.E;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int G = gridDim.x, g = blockIdx.x;
  for (int i = tid; i < (kSortWarps + 2) * p.E; i += blockDim.x) st_base[i] = 0;
  __syncthreads();
  pdl_trigger_and_wait();
  if (G > 1) {
    // every CTA's counts: thread (seg, e4) adds up every nseg-th CTA's for four experts; the
    // order does not matter, they are whole numbers
    const int quads = sort_pitch(p.E) / 4, nseg = static_cast<int>(blockDim.x) / quads;
    const int seg = tid / quads, e4 = 4 * (tid - seg * quads);
    if (seg < nseg) {
      int sum[4] = {0, 0, 0, 0}, before[4] = {0, 0, 0, 0};
#pragma unroll 4
      for (int c = seg; c < G; c += nseg) {
        const int4 q = *reinterpret_cast<const int4*>(p.hist + static_cast<int64_t>(c) * sort_pitch(p.E) + e4);
        const int v[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          sum[i] += v[i];
          if (c < g) before[i] += v[i];
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (e4 + i < p.E) {
          atomicAdd(s_total + e4 + i, sum[i]);
          if (before[i]) atomicAdd(s_before + e4 + i, before[i]);
        }
    }
  }
  int lo, hi;
  sort_run_bounds(p, g, warp, lo, hi);
  int* base = st_base + warp * p.E;  // the warp's own counters
  for (int i0 = lo; i0 < hi; i0 += 128) {
    int id[4];
    sort_load(p, i0, hi, id);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (id[j] >= 0) atomicAdd(base + id[j], 1);
  }
  __syncthreads();
  // E <= blockDim.x: thread e owns expert e
  int mine = 0, cnt[kSortWarps];
  if (tid < p.E) {
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) cnt[w] = st_base[w * p.E + tid];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) mine += cnt[w];
  }
  const int total = tid < p.E ? (G > 1 ? s_total[tid] : mine) : 0;
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
    int at = incl - total + s_before[tid];
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) {
      st_base[w * p.E + tid] = at;
      at += cnt[w];
    }
    if (g == 0) {
      p.offsets[tid] = incl - total;
      if (tid == p.E - 1) p.offsets[p.E] = incl;
    }
  }
  const int bits = 32 - __clz(p.E);
  const int kept = part[kSortWarps - 1];
  __syncthreads();
  for (int i0 = lo; i0 < hi; i0 += 128) {
    int id[4];
    sort_load(p, i0, hi, id);
    uint32_t same[4];
    sort_peers(id, bits, same);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (i0 + 32 * j >= hi) break;
      const int i = i0 + 32 * j + lane;
      int at = -1;
      if (id[j] >= 0) at = base[id[j]] + __popc(same[j] & ((1u << lane) - 1u));
      __syncwarp();
      if (id[j] >= 0 && lane == __ffs(same[j]) - 1) base[id[j]] += __popc(same[j]);
      __syncwarp();
      if (i < hi) {
        p.pos[i] = at;
        if (at >= 0) p.rows[at] = i / p.k;
      }
    }
  }
  // rows behind the last expert's
  for (int64_t i = kept + static_cast<int64_t>(g) * blockDim.x + tid; i < p.n; i += static_cast<int64_t>(G) * blockDim.x)
    p.rows[i] = -1;
}

// ---- expert combine ----------------------------------------------------------------------
//   y[t] = residual[t] + sum_j weights[t][j] h[pos[t][j]],  pairs with pos outside [0, R) left out
// in f32, in the order of j.  Bound by memory: 8191 x 8 rows of 2560 bf16 and an f32 residual take
// 87.6 us, 5.75 TB/s, with the rows of h gathered in pieces of 16 bytes a thread.
struct CombineParams {
  const void* h;
  const int* pos;
  const float* weights;
  const void* residual;
  void* y;
  int T, k, N, R;
  int residual_f32, out_f32;
};

// Predicated loads, 0 where !in: the loads of several pairs go out together, which ordinary ones
// behind branches of their own do not (61 x 6 x 2048: 2.7 us instead of 2.3).
__device__ __forceinline__ uint4 ld_if_v4(const void* p, bool in) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
      : "l"(p), "r"(static_cast<int>(in)));
  return v;
}
__device__ __forceinline__ uint32_t ld_if_b32(const void* p, bool in) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.b32 %0, [%1];\n\t}"
               : "=&r"(v)
               : "l"(p), "r"(static_cast<int>(in)));
  return v;
}
__device__ __forceinline__ uint32_t ld_if_u16(const void* p, bool in) {
  uint32_t v;
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.u16 %0, [%1];\n\t}"
               : "=&r"(v)
               : "l"(p), "r"(static_cast<int>(in)));
  return v;
}

// One thread: V neighbouring columns of one token (V = 8, or 1 where N is no multiple of 8 and
// the rows of h are not 16-byte aligned).  Up to 8 pairs' rows are on their way at once.
template <bool HF32, int V>
__global__ void __launch_bounds__(256) combine_kernel(const CombineParams p) {
  constexpr int kB = HF32 && V == 8 ? 4 : 8;  // pairs loaded together
  const int nv = p.N / V;
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  pdl_trigger_and_wait();
  if (i >= static_cast<int64_t>(p.T) * nv) return;
  const int64_t t = i / nv;
  const int n = static_cast<int>(i - t * nv) * V;
  const int64_t o = t * p.N + n;
  const int* pos = p.pos + t * p.k;
  const float* wts = p.weights + t * p.k;
  float acc[V];
#pragma unroll
  for (int c = 0; c < V; ++c) acc[c] = 0.f;
  for (int j0 = 0; j0 < p.k; j0 += kB) {
    int r[kB];
    float w[kB];
#pragma unroll
    for (int j = 0; j < kB; ++j) {
      const bool in = j0 + j < p.k;
      r[j] = static_cast<int>(ld_if_b32(pos + j0 + j, in));
      w[j] = __uint_as_float(ld_if_b32(wts + j0 + j, in));
      if (!in || r[j] >= p.R) r[j] = -1;
    }
    if (V == 8) {
      uint4 v[kB][HF32 ? 2 : 1];
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.h) +
                                                          (static_cast<int64_t>(r[j]) * p.N + n) * (HF32 ? 4 : 2));
        v[j][0] = ld_if_v4(src, r[j] >= 0);
        if (HF32) v[j][HF32 ? 1 : 0] = ld_if_v4(src + 1, r[j] >= 0);
      }
#pragma unroll
      for (int j = 0; j < kB; ++j)
        if (r[j] >= 0) {
          const uint32_t a[4] = {v[j][0].x, v[j][0].y, v[j][0].z, v[j][0].w};
          const uint4 b4 = v[j][HF32 ? 1 : 0];
          const uint32_t b[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            if (HF32) {
              acc[c % V] = fmaf(w[j], __uint_as_float(a[c]), acc[c % V]);
              acc[(4 + c) % V] = fmaf(w[j], __uint_as_float(b[c]), acc[(4 + c) % V]);
            } else {
              acc[(2 * c) % V] = fmaf(w[j], __uint_as_float(a[c] << 16), acc[(2 * c) % V]);
              acc[(2 * c + 1) % V] = fmaf(w[j], __uint_as_float(a[c] & 0xFFFF0000u), acc[(2 * c + 1) % V]);
            }
          }
        }
    } else {
      uint32_t v[kB];
#pragma unroll
      for (int j = 0; j < kB; ++j) {
        const int64_t at = static_cast<int64_t>(r[j]) * p.N + n;
        v[j] = HF32 ? ld_if_b32(static_cast<const float*>(p.h) + at, r[j] >= 0)
                    : ld_if_u16(static_cast<const uint16_t*>(p.h) + at, r[j] >= 0) << 16;
      }
#pragma unroll
      for (int j = 0; j < kB; ++j)
        if (r[j] >= 0) acc[0] = fmaf(w[j], __uint_as_float(v[j]), acc[0]);
    }
  }
  // the residual may be y itself: the same elements, read before they are written
#pragma unroll
  for (int c0 = 0; c0 < V; c0 += 4) {
    if (p.residual) {
      if (V == 8) {
        if (p.residual_f32) {
          const float4 r = *reinterpret_cast<const float4*>(static_cast<const float*>(p.residual) + o + c0);
          acc[c0 % V] += r.x;
          acc[(c0 + 1) % V] += r.y;
          acc[(c0 + 2) % V] += r.z;
          acc[(c0 + 3) % V] += r.w;
        } else {
          const uint2 r = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.residual) + o + c0);
          acc[c0 % V] += __uint_as_float(r.x << 16);
          acc[(c0 + 1) % V] += __uint_as_float(r.x & 0xFFFF0000u);
          acc[(c0 + 2) % V] += __uint_as_float(r.y << 16);
          acc[(c0 + 3) % V] += __uint_as_float(r.y & 0xFFFF0000u);
        }
      } else {
        acc[0] += p.residual_f32 ? static_cast<const float*>(p.residual)[o]
                                 : bf16_bits_to_f32(static_cast<const uint16_t*>(p.residual)[o]);
      }
    }
  }
  if (V == 8) {
    if (p.out_f32) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.y) + o);
      dst[0] = make_float4(acc[0], acc[1 % V], acc[2 % V], acc[3 % V]);
      dst[1] = make_float4(acc[4 % V], acc[5 % V], acc[6 % V], acc[7 % V]);
    } else {
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.y) + o) =
          make_uint4(pack_bf16x2(acc[0], acc[1 % V]), pack_bf16x2(acc[2 % V], acc[3 % V]),
                     pack_bf16x2(acc[4 % V], acc[5 % V]), pack_bf16x2(acc[6 % V], acc[7 % V]));
    }
  } else if (p.out_f32) {
    static_cast<float*>(p.y)[o] = acc[0];
  } else {
    static_cast<__nv_bfloat16*>(p.y)[o] = __float2bfloat16_rn(acc[0]);
  }
}

}  // namespace tgemm
