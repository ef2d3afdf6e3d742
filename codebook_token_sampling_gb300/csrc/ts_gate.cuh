// ts_gate.cuh -- a gated activation (ts_gate): out = act(gate) * up, or only the
// rounding of `up` to 8-bit rows.
#pragma once

#include "ts_kv_common.cuh"
#include "ts_rows.cuh"

namespace ts {

constexpr int kGateThreads = 256;
// CTAs per SM: three of sixteen elements a lane (bf16 to 8 bits, gelu on 16,384 x 11,008: 142
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
constexpr float kLog2E = 1.44269504f, kLn2 = 0.693147181f;

// Two elements at once: g / (1 + exp(-z)).  exp(-z) = 2^t exp(d) with t = -z log2 e rounded
// and d = -z - t ln 2 what that rounding left, so the exponential is right to its size at
// any z; the quotient is within 2^-20 of it (13 roundings at most; the exponential of the
// rounded exponent alone: 2^-23 |z| more).  Beyond 88 the quotient is g, below -88 it is
// less than 2^-119 and counts as 0.
__device__ __forceinline__ uint64_t logistic2(float g0, float g1, float z0, float z1) {
  const uint64_t n = pair_of(fmaxf(fminf(-z0, 88.0f), -88.0f), fmaxf(fminf(-z1, 88.0f), -88.0f));
  const uint64_t t = mul2(n, both_of(kLog2E)), d = fma2(t, both_of(-kLn2), n);
  float t0, t1, u0, u1;
  parts_of(t, t0, t1);
  const uint64_t e = pair_of(power_of_2(t0), power_of_2(t1));
  parts_of(add2(fma2(e, d, e), both_of(1.0f)), u0, u1);
  return mul2(pair_of(g0, g1), pair_of(reciprocal(u0), reciprocal(u1)));
}

// g (1 + erf(g / sqrt 2)) / 2 of two elements: max(g, 0) - a Q(a) with a = |g| and Q(a) =
// erfc(a / sqrt 2) / 2 = exp(-a a / 2) R(a).  R falls from 1/2 to 1 / (a sqrt(2 pi)) and is
// taken as a quotient of two polynomials of positive terms in the manner of Cody, "Rational
// Chebyshev approximations for the error function" (1969), with coefficients of our own
// (least largest relative error over 0 .. 13.3: 3.8e-7).  So the result is right relative to
// its size wherever that is not below 2^-126: FULL within 2^-19, with the exponential's
// argument kept as above (and SQUARES: what the square's rounding left); else 1.1 g g 2^-24
// more, far below the rounding to 16 or 8 bits (kept for those too and with a term more in the
// numerator, gelu on 16,384 x 11,008 bf16 to 8 bits took 161 us instead of 142).  For gates of normal distribution the error's
// norm is 3.2e-8, 3.5e-8 by fp32's erf; a polynomial that is right to 1.5e-7 of one would be
// off by 1% at -8, and erff took longer than the loads (273 us).
template <bool FULL, bool SQUARES>
__device__ __forceinline__ uint64_t gelu2(float g0, float g1) {
  // nothing is left of Q at 16; zeros, NaN and -inf times zero come from the first term
  const uint64_t a = pair_of(fminf(fabsf(g0), 16.0f), fminf(fabsf(g1), 16.0f));
  const uint64_t first = mul2(pair_of(g0, g1), pair_of(g0 > 0.0f ? 1.0f : 0.0f, g1 > 0.0f ? 1.0f : 0.0f));
  const uint64_t half = mul2(a, both_of(-0.5f)), n = mul2(half, a);
  const uint64_t t = FULL ? mul2(n, both_of(kLog2E)) : mul2(mul2(a, a), both_of(-0.5f * kLog2E));
  float t0, t1, u0, u1;
  parts_of(t, t0, t1);
  uint64_t e = pair_of(power_of_2(t0), power_of_2(t1));
  if constexpr (FULL) {
    uint64_t d = fma2(t, both_of(-kLn2), n);
    if constexpr (SQUARES) d = add2(d, fma2(half, a, mul2(n, both_of(-1.0f))));
    e = fma2(e, d, e);
  }
  uint64_t q = fma2(a, both_of(0.0422765017f), both_of(0.297457546f));
  q = fma2(a, q, both_of(0.949712813f));
  q = fma2(a, q, both_of(1.51909733f));
  parts_of(fma2(a, q, both_of(1.0f)), u0, u1);
  uint64_t p = fma2(a, both_of(-0.016863713f), both_of(-0.118754119f));  // minus the numerator
  p = fma2(a, p, both_of(-0.360615194f));
  p = fma2(a, p, both_of(-0.499999821f));
  return fma2(a, mul2(mul2(p, pair_of(reciprocal(u0), reciprocal(u1))), e), first);
}

template <int E, bool FULL, bool SQUARES>
__device__ __forceinline__ void gated(float (&y)[E], const float (&g)[E], int act) {
  if (act == kActSilu) {
#pragma unroll
    for (int e = 0; e < E; e += 2)
      parts_of(mul2(pair_of(y[e], y[e + 1]), logistic2(g[e], g[e + 1], g[e], g[e + 1])), y[e], y[e + 1]);
  } else if (act == kActGelu) {
#pragma unroll
    for (int e = 0; e < E; e += 2)
      parts_of(mul2(pair_of(y[e], y[e + 1]), gelu2<FULL, SQUARES>(g[e], g[e + 1])), y[e], y[e + 1]);
  } else {  // (1 + tanh(z / 2)) / 2 = 1 / (1 + exp(-z))
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      const uint64_t v = pair_of(g[e], g[e + 1]);
      float z0, z1;
      parts_of(mul2(v, fma2(mul2(v, v), both_of(1.5957691216f * 0.044715f), both_of(1.5957691216f))), z0, z1);
      parts_of(mul2(pair_of(y[e], y[e + 1]), logistic2(g[e], g[e + 1], z0, z1)), y[e], y[e + 1]);
    }
  }
}

// The rows' units end to end, a thread's next one's loads on their way while it works on
// this one; addresses move along by additions.  16,384 x 11,008 bf16 to 8 bits, sixteen
// elements a lane: gelu 142 us, 6.4 TB/s, bound by DRAM like silu (134 us) and no gate (94).
// With eight elements a lane 181 us, bound by instructions (about 210 for eight, half of them
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
    if (act) gated<W, sizeof(Out) == 4, sizeof(Src) == 4>(y, g, p.act);
    if constexpr (sizeof(Out) == 1) {
      const float scale = scaled_block<W>(y);
      if ((lane_id() & (U::kLanes - 1)) == 0 && left > 0) *scale_at = scale;
    }
    store_unit<W>(out, 0, left, y);
  }
}

}  // namespace ts
