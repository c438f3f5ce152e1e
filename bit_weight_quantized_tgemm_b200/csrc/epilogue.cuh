// epilogue.cuh -- the fused epilogue of the epilogue and expert matmuls:
//   y = residual + gate * act(v + bias),  v = x W^T in f32
// Every step is f32; the one rounding is the store of a bf16 y.
#pragma once

#include "common.cuh"

namespace tgemm {

constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3, kActRelu = 4;

struct EpArgs {
  const void* bias;      // [N] (one row of N per expert), or null
  const uint16_t* gate;  // bf16: [N], or [M][N] when gate_rows; or null
  const void* residual;  // [M][N], or null
  void* y;               // [M][N]
  int bias_f32, gate_rows, residual_f32, out_f32, act;
};

// What another kernel may have written just before (activations, plans, epilogue operands) is read by
// ordinary loads after the wait for that kernel: this grid may be resident while it is written,
// and the read-only path is for memory that nobody writes meanwhile.  Packed weights and scales,
// which are read ahead of the wait, take the read-only path.
__device__ __forceinline__ uint16_t ld_scale(const uint16_t* p) { return __ldg(p); }

__device__ __forceinline__ float ep_exp2(float t) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t));
  return r;
}
// v / (1 + 2^-t), from the exponential and quotient units: the exponential is within 2^-22, the
// quotient within 2 f32 steps, and the rounding of t, at most 2^-24 of it, moves the exponential by
// 2^-24 ln(2) |t|: for v below 0 in all up to 1.5e-6 of the result at v = -20, where that is 4e-8,
// and 5e-6 at v = -87.  A denominator past 2^126 gives 0: results below 1e-36 are flushed.
// 1536 x 9472 x 1280 ternary with a tanh GELU: 56 us with expf, 50 us.
__device__ __forceinline__ float ep_logistic(float v, float t) { return __fdividef(v, 1.f + ep_exp2(-t)); }

constexpr float kLog2E = 1.4426950408889634f;

template <int ACT>
__device__ __forceinline__ float ep_act(float v) {
  if (ACT == kActSilu) return ep_logistic(v, kLog2E * v);
  if (ACT == kActGelu) return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
  // (1 + tanh(u)) / 2 = 1 / (1 + exp(-2 u)),  2 u = 2 sqrt(2 / pi) v (1 + 0.044715 v^2)
  if (ACT == kActGeluTanh) {
    constexpr float kC = 1.5957691216057308f * kLog2E;
    return ep_logistic(v, v * fmaf(0.044715f * kC, v * v, kC));
  }
  if (ACT == kActRelu) return v < 0.f ? 0.f : v;  // keeps a NaN
  return v;
}

// f(v) for each of n values, the activation chosen once.
template <int n>
__device__ __forceinline__ void ep_act_all(float (&v)[n], int act) {
#define TGEMM_EP_ALL(A)                            \
  case A: {                                        \
    _Pragma("unroll") for (int i = 0; i < n; ++i) v[i] = ep_act<A>(v[i]); \
    break;                                         \
  }
  switch (act) {
    TGEMM_EP_ALL(kActSilu)
    TGEMM_EP_ALL(kActGelu)
    TGEMM_EP_ALL(kActGeluTanh)
    TGEMM_EP_ALL(kActRelu)
    default: break;
  }
#undef TGEMM_EP_ALL
}

__device__ __forceinline__ float ep_load(const void* p, int64_t i, int f32) {
  return f32 ? static_cast<const float*>(p)[i] : bf16_bits_to_f32(static_cast<const uint16_t*>(p)[i]);
}

// gate and residual of one element, and its store.  The residual is read with a plain load:
// it may be y itself (the same element, read by the thread that writes it).
__device__ __forceinline__ void ep_store1(const EpArgs& a, int64_t m, int n, int N, float v) {
  const int64_t i = m * N + n;
  if (a.gate) v *= bf16_bits_to_f32(a.gate[a.gate_rows ? i : n]);
  if (a.residual)
    v += a.residual_f32 ? static_cast<const float*>(a.residual)[i]
                        : bf16_bits_to_f32(static_cast<const uint16_t*>(a.residual)[i]);
  if (a.out_f32)
    static_cast<float*>(a.y)[i] = v;
  else
    static_cast<__nv_bfloat16*>(a.y)[i] = __float2bfloat16_rn(v);
}

}  // namespace tgemm
