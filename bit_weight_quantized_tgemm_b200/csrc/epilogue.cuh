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

__device__ __forceinline__ float ep_act(float v, int act) {
  switch (act) {
    case kActSilu: return v / (1.f + expf(-v));
    case kActGelu: return 0.5f * v * (1.f + erff(v * 0.70710678118654752f));
    case kActGeluTanh: return 0.5f * v * (1.f + tanhf(0.79788456080286536f * fmaf(0.044715f * v * v, v, v)));
    case kActRelu: return v < 0.f ? 0.f : v;  // keeps a NaN
    default: return v;
  }
}

__device__ __forceinline__ float ep_load(const void* p, int64_t i, int f32) {
  return f32 ? __ldg(static_cast<const float*>(p) + i)
             : bf16_bits_to_f32(__ldg(static_cast<const uint16_t*>(p) + i));
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
