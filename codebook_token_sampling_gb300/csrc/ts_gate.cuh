// ts_gate.cuh -- a gated activation (ts_gate): out = act(gate) * up, or only the
// rounding of `up` to 8-bit rows.
#pragma once

#include "ts_kv_common.cuh"
#include "ts_rows.cuh"

namespace ts {

constexpr int kGateThreads = 256;
constexpr int kGateUnits = 1;  // per thread at once
constexpr int kGateCtas = 6;   // per SM
constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3;

struct GateParams {
  const void *up, *gate;
  void *out;
  float *scale;
  int64_t up_stride, gate_stride, out_stride, scale_stride;
  int64_t step_rows;   // from a CTA's units to its next ones: rows, and units of a row
  uint32_t step_units;
  int32_t n_rows, dim, act;
  FastDiv by_row;  // units per row: whole blocks of 128 elements
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

// y g (1 + erf(g / sqrt 2)) / 2 of two elements: g (1 + erf) / 2 = max(g, 0) - |g| erfc(|g| /
// sqrt 2) / 2, with Hastings's erfc(x) = t (a1 + t (a2 + .. t a5)) exp(-x x), t = 1 / (1 + p x),
// to 1.5e-7 ("Approximations for digital computers", 1955; 7.1.26 in Abramowitz and
// Stegun).  erff took longer than the loads (16,384 x 11,008: 273 us; this one element by
// element 193).
__device__ __forceinline__ uint64_t gelu2(uint64_t y, float g0, float g1) {
  // |g|, but for +inf, whose product with erfc's zero is no part of the result; a NaN stays
  const float a0 = max_nan(-g0, min_nan(g0, 3e38f)), a1 = max_nan(-g1, min_nan(g1, 3e38f));
  const uint64_t a = pair_of(a0, a1);
  float u0, u1, e0, e1;
  parts_of(fma2(a, both_of(0.3275911f * 0.70710678f), both_of(1.0f)), u0, u1);
  parts_of(mul2(mul2(a, a), both_of(-0.5f * kLog2E)), e0, e1);
  const uint64_t t = pair_of(reciprocal(u0), reciprocal(u1)), e = pair_of(power_of_2(e0), power_of_2(e1));
  uint64_t w = fma2(t, both_of(-0.5f * 1.061405429f), both_of(0.5f * 1.453152027f));
  w = fma2(t, w, both_of(-0.5f * 1.421413741f));
  w = fma2(t, w, both_of(0.5f * 0.284496736f));
  w = fma2(t, w, both_of(-0.5f * 0.254829592f));  // minus the half of it
  w = mul2(mul2(w, t), e);
  return mul2(y, fma2(a, w, pair_of(fmaxf(g0, 0.0f), fmaxf(g1, 0.0f))));
}

template <int E>
__device__ __forceinline__ void gated(float (&y)[E], const float (&g)[E], int act) {
  if (act == kActSilu) {
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] *= logistic(g[e], g[e]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int e = 0; e < E; e += 2) parts_of(gelu2(pair_of(y[e], y[e + 1]), g[e], g[e + 1]), y[e], y[e + 1]);
  } else {  // (1 + tanh z) / 2 = 1 / (1 + exp(-2 z))
#pragma unroll
    for (int e = 0; e < E; ++e)
      y[e] *= logistic(g[e], 1.5957691f * fmaf(0.044715f * g[e] * g[e], g[e], g[e]));
  }
}

// The rows' units end to end, kGateUnits of a thread at once, its next ones' loads on
// their way while it works on these (six CTAs to an SM: 175 us for gelu on 16,384 x 11,008
// to 8 bits, 5.2 TB/s; 178 with five, 209 with eight, 193 with a CTA for each two units).
// Bound by instructions there (eight elements take 226, 73% of the issue slots, and
// 16 of the special functions), with silu and without a gate by DRAM.
template <class Src, class Out, bool WIDE>
__global__ void __launch_bounds__(kGateThreads, kGateCtas) gate_kernel(const GateParams p) {
  using U = RowUnit<WIDE>;
  constexpr int E = U::kElems;
  constexpr int N = kGateUnits;
  pdl_wait_and_release();
  const bool act = p.act != kActNone;
  const uint32_t per_row = p.by_row.d;
  int64_t row[N];
  uint32_t in[N];  // unit of the row
  {
    const int64_t base = static_cast<int64_t>(blockIdx.x) * (kGateThreads * N);
    const int64_t r0 = base / per_row;
    const uint32_t off0 = static_cast<uint32_t>(base - r0 * per_row) + threadIdx.x;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t u = off0 + j * kGateThreads, r = p.by_row.div(u);
      row[j] = r0 + r;
      in[j] = u - r * per_row;
    }
  }
  RawUnit<Src, WIDE> up[N], gate[N];
  const auto at = [&](uint32_t c) {
    return WIDE ? static_cast<int32_t>(c * 8) : static_cast<int32_t>((c >> 5) * kScaleBlock + (c & 31));
  };
  const auto fetch = [&]() {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int32_t dim = row[j] < p.n_rows ? p.dim : 0;  // behind the last row: no elements
      up[j].load(static_cast<const Src *>(p.up) + row[j] * p.up_stride, at(in[j]), dim);
      if (act) gate[j].load(static_cast<const Src *>(p.gate) + row[j] * p.gate_stride, at(in[j]), dim);
    }
  };
  fetch();
  while (__any_sync(0xFFFFFFFFu, row[0] < p.n_rows)) {
    float y[N][E], g[N][E];
    int64_t now[N];
    int32_t here[N];
#pragma unroll
    for (int j = 0; j < N; ++j) {
#pragma unroll
      for (int e = 0; e < E; ++e) {
        y[j][e] = up[j].at(e);
        g[j][e] = gate[j].at(e);
      }
      now[j] = row[j];
      here[j] = row[j] < p.n_rows ? at(in[j]) : p.dim + kScaleBlock;
      row[j] += p.step_rows;
      in[j] += p.step_units;
      if (in[j] >= per_row) {
        in[j] -= per_row;
        ++row[j];
      }
    }
    fetch();
#pragma unroll
    for (int j = 0; j < N; ++j) {
      if (act) gated<E>(y[j], g[j], p.act);
      if constexpr (sizeof(Out) == 1) {
        const float scale = scaled_block<WIDE>(y[j]);
        const int first = static_cast<int>(lane_id()) & (U::kLanes - 1);
        if (first == 0 && here[j] < p.dim) p.scale[now[j] * p.scale_stride + here[j] / kScaleBlock] = scale;
      }
      store_unit<WIDE>(static_cast<Out *>(p.out) + now[j] * p.out_stride, here[j], p.dim, y[j]);
    }
  }
}

}  // namespace ts
