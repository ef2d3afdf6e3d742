// ts_gate.cuh -- a gated activation (ts_gate): out = act(gate) * up, or only the
// rounding of `up` to 8-bit rows.
#pragma once

#include "ts_kv_common.cuh"
#include "ts_rows.cuh"

namespace ts {

constexpr int kGateThreads = 256;
// CTAs per SM: three of sixteen elements a lane (bf16 to 8 bits, gelu on 16,384 x 11,008: 140
// us, 225 with four and spills), four where elements of 32 bits are on their way (fp32 to 8
// bits 242 us, 383 with five and spills; bf16 to fp32 213, 251), else five (bf16 to bf16 159,
// 167 with four).
constexpr int gate_ctas(int in_bytes, int out_bytes, int width) {
  return width == 16 ? 3 : in_bytes == 4 || out_bytes == 4 ? 4 : 5;
}
constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3;

struct GateParams {
  const void *up, *gate;
  void *out;
  float *scale;
  int64_t up_stride, gate_stride, out_stride, scale_stride;
  // from a thread's unit to its next one: rows, elements along a row, and what the
  // addresses move by, with what that is off by where the row's end is passed
  struct Move {
    int64_t up, gate, out, scale;
  } step, wrap;
  uint32_t step_rows;
  int32_t step_elems, row_elems;  // row_elems: a row's, up to whole blocks
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

// The rows' units end to end, a thread's next one's loads on their way while it works on
// this one; addresses move along by additions.  16,384 x 11,008 bf16 to 8 bits, sixteen
// elements a lane: gelu 140 us, 6.5 TB/s, bound by DRAM like silu (134 us) and no gate (94).
// With eight elements a lane 174 us, bound by instructions (about 210 for eight, half of them
// for the block's scale, addresses and the loop); a CTA for each two units 193.
template <class Src, class Out, int W>
__global__ void __launch_bounds__(kGateThreads, gate_ctas(sizeof(Src), sizeof(Out), W)) gate_kernel(const GateParams p) {
  using U = RowUnit<W>;
  pdl_wait_and_release();
  const bool act = p.act != kActNone;
  const uint32_t per_row = p.by_row.d;
  uint32_t row;    // of the unit that is fetched next
  int32_t at;      // its (lane's) first element
  const Src *up_at, *gate_at;
  Out *out_next;
  float *scale_next;
  {
    const int64_t base = static_cast<int64_t>(blockIdx.x) * kGateThreads, r0 = base / per_row;
    const uint32_t u = static_cast<uint32_t>(base - r0 * per_row) + threadIdx.x, r = p.by_row.div(u), c = u - r * per_row;
    row = static_cast<uint32_t>(r0) + r;
    at = U::kWide ? static_cast<int32_t>(c * W) : static_cast<int32_t>((c >> 5) * kScaleBlock + (c & 31));
    up_at = static_cast<const Src *>(p.up) + row * p.up_stride + at;
    gate_at = static_cast<const Src *>(p.gate) + row * p.gate_stride + at;
    out_next = static_cast<Out *>(p.out) + row * p.out_stride + at;
    scale_next = p.scale + row * p.scale_stride + at / kScaleBlock;
  }
  const uint32_t n_rows = static_cast<uint32_t>(p.n_rows);
  RawUnit<Src, W> up, gate;
  const auto fetch = [&]() {
    const int32_t left = row < n_rows ? p.dim - at : 0;  // behind the last row: no elements
    up.load(up_at, 0, left);
    if (act) gate.load(gate_at, 0, left);
  };
  fetch();
  while (__any_sync(0xFFFFFFFFu, row < n_rows)) {
    float y[W], g[W];
#pragma unroll
    for (int e = 0; e < W; ++e) {
      y[e] = up.at(e);
      g[e] = gate.at(e);
    }
    const int32_t left = row < n_rows ? p.dim - at : 0;
    Out *out = out_next;
    float *scale_at = scale_next;
    row += p.step_rows;
    at += p.step_elems;
    up_at += p.step.up;
    gate_at += p.step.gate;
    out_next += p.step.out;
    scale_next += p.step.scale;
    if (at >= p.row_elems) {
      ++row;
      at -= p.row_elems;
      up_at += p.wrap.up;
      gate_at += p.wrap.gate;
      out_next += p.wrap.out;
      scale_next += p.wrap.scale;
    }
    fetch();
    if (act) gated<W>(y, g, p.act);
    if constexpr (sizeof(Out) == 1) {
      const float scale = scaled_block<W>(y);
      if ((lane_id() & (U::kLanes - 1)) == 0 && left > 0) *scale_at = scale;
    }
    store_unit<W>(out, 0, left, y);
  }
}

}  // namespace ts
