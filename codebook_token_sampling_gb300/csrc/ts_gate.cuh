// ts_gate.cuh -- a gated activation (ts_gate): out = act(gate) * up, or only the
// rounding of `up` to 8-bit rows.
#pragma once

#include "ts_kv_common.cuh"
#include "ts_rows.cuh"

namespace ts {

constexpr int kGateThreads = 256;
constexpr int kGateUnits = 2;  // per thread
constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3;

struct GateParams {
  const void *up, *gate;
  void *out;
  float *scale;
  int64_t up_stride, gate_stride, out_stride, scale_stride;
  int64_t units;   // of all rows: whole blocks of 128 elements each
  int32_t dim, act;
  FastDiv by_row;  // units per row
};

// 1 / x and 2^x within two units in the last place, subnormal results as zeros
__device__ __forceinline__ float reciprocal(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float power_of_2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr float kLog2E = 1.44269504f;

// g / (1 + exp(-z))
__device__ __forceinline__ float logistic(float g, float z) { return g * reciprocal(1.0f + power_of_2(-kLog2E * z)); }

// g (1 + erf(g / sqrt 2)) / 2 = max(g, 0) - |g| erfc(|g| / sqrt 2) / 2, with Hastings's
// erfc(x) = t (a1 + t (a2 + .. t a5)) exp(-x x), t = 1 / (1 + p x), to 1.5e-7 ("Approximations
// for digital computers", 1955; 7.1.26 in Abramowitz and Stegun).  A third of the
// instructions of erff, which took longer than the loads (273 us for 16,384 x 11,008).
__device__ __forceinline__ float gelu(float g) {
  const float a = fabsf(g);
  const float t = reciprocal(fmaf(0.3275911f * 0.70710678f, a, 1.0f));
  float w = fmaf(t, 0.5f * 1.061405429f, -0.5f * 1.453152027f);
  w = fmaf(t, w, 0.5f * 1.421413741f);
  w = fmaf(t, w, -0.5f * 0.284496736f);
  w = fmaf(t, w, 0.5f * 0.254829592f);
  w = w * t * power_of_2(-0.5f * kLog2E * a * a);
  return fmaf(-fminf(a, 3e38f), w, fmaxf(g, 0.0f));
}

template <int E>
__device__ __forceinline__ void gated(float (&y)[E], const float (&g)[E], int act) {
  if (act == kActSilu) {
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] *= logistic(g[e], g[e]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] *= gelu(g[e]);
  } else {  // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
#pragma unroll
    for (int e = 0; e < E; ++e)
      y[e] *= logistic(g[e], 1.5957691f * fmaf(0.044715f * g[e] * g[e], g[e], g[e]));
  }
}

// The rows' units end to end, kGateUnits per thread, a CTA's next to one another:
// bound by DRAM.
template <class Src, class Out, bool WIDE>
__global__ void __launch_bounds__(kGateThreads) gate_kernel(const GateParams p) {
  using U = RowUnit<WIDE>;
  constexpr int E = U::kElems;
  constexpr int kUnits = kGateUnits;
  pdl_wait_and_release();
  const int64_t base = static_cast<int64_t>(blockIdx.x) * (kGateThreads * kUnits);
  const int64_t r0 = base / p.by_row.d;
  const uint32_t off0 = static_cast<uint32_t>(base - r0 * p.by_row.d) + threadIdx.x;
  const bool act = p.act != kActNone;
  float y[kUnits][E], g[kUnits][E];
  int64_t row[kUnits];
  int32_t at[kUnits];
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    const uint32_t u = off0 + j * kGateThreads;
    const uint32_t r = p.by_row.div(u), c = u - r * p.by_row.d;
    row[j] = r0 + r;
    at[j] = WIDE ? static_cast<int32_t>(c * 8) : static_cast<int32_t>((c >> 5) * kScaleBlock + (c & 31));
    const bool there = base + threadIdx.x + j * kGateThreads < p.units;
    const int32_t dim = there ? p.dim : 0;  // no elements
    load_unit<WIDE>(static_cast<const Src *>(p.up) + row[j] * p.up_stride, at[j], dim, y[j]);
    if (act) load_unit<WIDE>(static_cast<const Src *>(p.gate) + row[j] * p.gate_stride, at[j], dim, g[j]);
    if (!there) at[j] = p.dim + kScaleBlock;
  }
#pragma unroll
  for (int j = 0; j < kUnits; ++j) {
    if (act) gated<E>(y[j], g[j], p.act);
    if constexpr (sizeof(Out) == 1) {
      const float scale = scaled_block<WIDE>(y[j]);
      const int first = static_cast<int>(lane_id()) & (U::kLanes - 1);
      if (first == 0 && at[j] < p.dim) p.scale[row[j] * p.scale_stride + at[j] / kScaleBlock] = scale;
    }
    store_unit<WIDE>(static_cast<Out *>(p.out) + row[j] * p.out_stride, at[j], p.dim, y[j]);
  }
}

}  // namespace ts
