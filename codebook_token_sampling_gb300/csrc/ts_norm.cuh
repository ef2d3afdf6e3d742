// ts_norm.cuh -- root-mean-square norm of the residual's sum (ts_rms_norm):
//   h = x + residual,   y = h / sqrt(mean(h h) + eps) * (weight + weight_offset).
#pragma once

#include "ts_rows.cuh"

namespace ts {

struct NormParams {
  const void *x, *residual, *weight;
  void *residual_out, *out;
  float *scale;
  int64_t x_stride, residual_stride, residual_out_stride, out_stride, scale_stride;
  int32_t n_rows, dim, weight_f32;
  float eps, weight_offset;
};

// One row per CTA (or, for one-warp rows, one per warp: blockDim.y of them), its V
// units per thread held in registers between the sum of squares and the output, so
// every element is read once and written once.
template <class Src, class Out, int V, bool WIDE>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const NormParams p) {
  using U = RowUnit<WIDE>;
  constexpr int E = U::kElems;
  __shared__ float part[32];
  const int t = static_cast<int>(threadIdx.x), lane = t & 31, warp = t >> 5, nt = static_cast<int>(blockDim.x);
  const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  pdl_wait_and_release();
  if (r >= p.n_rows) return;  // whole warps, of CTAs whose rows are warps

  const auto at = [&](int j) {
    return WIDE ? (t + j * nt) * 8 : (warp + j * (nt >> 5)) * kScaleBlock + lane;
  };
  const Src *x = static_cast<const Src *>(p.x) + r * p.x_stride;
  float h[V][E];
#pragma unroll
  for (int j = 0; j < V; ++j) load_unit<WIDE>(x, at(j), p.dim, h[j]);
  if (p.residual) {
    const Src *res = static_cast<const Src *>(p.residual) + r * p.residual_stride;
    float s[V][E];
#pragma unroll
    for (int j = 0; j < V; ++j) load_unit<WIDE>(res, at(j), p.dim, s[j]);
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) h[j][e] += s[j][e];
  }
  if (p.residual_out) {
    Src *ro = static_cast<Src *>(p.residual_out) + r * p.residual_out_stride;
#pragma unroll
    for (int j = 0; j < V; ++j) store_unit<WIDE>(ro, at(j), p.dim, h[j]);
  }

  // f's sum or largest value over the row's threads, in a fixed order
  const auto over_row = [&](float v, auto f) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (nt == 32) return v;
    if (lane == 0) part[warp] = v;
    __syncthreads();
    v = lane < (nt >> 5) ? part[lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  };
  const auto add = [](float a, float b) { return a + b; };
  const auto squares = [&]() {
    float ss = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) ss = fmaf(h[j][e], h[j][e], ss);
    return over_row(ss, add);
  };
  float ss = squares();
  float rstd;
  if (ss > 0x1p-90f && ss < 0x1p127f) {
    rstd = __frsqrt_rn(__fdiv_rn(ss, static_cast<float>(p.dim)) + p.eps);
  } else {
    // Squares outside fp32's range (or a row of zeros, or one that is not finite):
    // with h = 2^e g, 1 / sqrt(mean(h h) + eps) = 2^-e / sqrt(mean(g g) + eps 4^-e).
    float a = 0.0f;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int e = 0; e < E; ++e) a = max_nan(a, fabsf(h[j][e]));
    if (nt > 32) __syncthreads();  // part is read
    a = over_row(a, [](float u, float v) { return max_nan(u, v); });
    float down = 1.0f;
    if (a > 0.0f && a < INFINITY) {
      const int up = static_cast<int>(__float_as_uint(a) >> 23) - 127;
      down = __uint_as_float(static_cast<uint32_t>(127 - max(up, -126)) << 23);
      if (up == 127) down = 0x1p-126f;  // two powers more than needed, to stay normal
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) h[j][e] *= down;
    }
    if (nt > 32) __syncthreads();
    ss = squares();
    const float scaled_eps = p.eps * down * down;
    if (scaled_eps < INFINITY) {
      rstd = __frsqrt_rn(__fdiv_rn(ss, static_cast<float>(p.dim)) + scaled_eps);
    } else {  // eps is all that counts
      rstd = __frsqrt_rn(p.eps);
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < E; ++e) h[j][e] = __fdiv_rn(h[j][e], down);
    }
  }

  Out *out = static_cast<Out *>(p.out) + r * p.out_stride;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    float y[E];
    if (p.weight) {
      float w[E];
      if (p.weight_f32) load_unit<WIDE>(static_cast<const float *>(p.weight), at(j), p.dim, w);
      else load_unit<WIDE>(static_cast<const uint16_t *>(p.weight), at(j), p.dim, w);
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = h[j][e] * rstd * (w[e] + p.weight_offset);
    } else {
#pragma unroll
      for (int e = 0; e < E; ++e) y[e] = h[j][e] * rstd;
    }
    if constexpr (sizeof(Out) == 1) {
      const float scale = scaled_block<WIDE>(y);
      if ((lane & (U::kLanes - 1)) == 0 && at(j) < p.dim)
        p.scale[r * p.scale_stride + at(j) / kScaleBlock] = scale;
    }
    store_unit<WIDE>(out, at(j), p.dim, y);
  }
}

}  // namespace ts
