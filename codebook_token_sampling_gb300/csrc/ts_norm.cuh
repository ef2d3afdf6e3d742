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

// A CTA walks over rows (or, of one-warp rows, each of its blockDim.y warps does), its V
// units per thread held in registers between the sum of squares and the output, so every
// element is read once and written once.  AHEAD: a thread has the next row's on their way
// meanwhile (one or two units, up to 512 threads).  Bound by DRAM: 32,768 rows of 4096 with
// residual and 8-bit outputs take 144 us, 6.6 TB/s (186 us with a CTA for each row); without a
// residual by instructions too (83 us, floor 60; 125 with eight elements a lane).  A frame
// of 32 x 1024 takes a launch and two trips to memory, 1.9 us; rows of odd width their
// single elements' loads and stores (5000 x 1001 fp32 9.0 us, floor 4.4).  Rows above 8192
// are not AHEAD (8192 x 16,384 fp32 to 8 bits 316 us; with the next row's loads held beside
// this one's sums and spills 458).
template <class Src, class Out, int V, int W, bool AHEAD>
__global__ void __launch_bounds__(W == 16 ? 256 : AHEAD ? 512 : 1024, W == 16 ? 3 : AHEAD ? 2 : 1) rms_norm_kernel(const NormParams p) {
  using U = RowUnit<W>;
  __shared__ float part[2][32];
  // a thread's weights with their offset, where it keeps its elements over many rows: four
  // pieces [4][threads]
  extern __shared__ float4 norm_factors[];
  const int t = static_cast<int>(threadIdx.x), lane = t & 31, warp = t >> 5, nt = static_cast<int>(blockDim.x);
  const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
  int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
  pdl_wait_and_release();
  if (r >= p.n_rows) return;  // whole warps, of CTAs whose rows are warps

  const auto at = [&](int j) {
    return U::kWide ? (t + j * nt) * W : (warp + j * (nt >> 5)) * kScaleBlock + lane;
  };
  // (rows that are not AHEAD: a unit's sum at once, so that no more is held than their sums)
  RawUnit<Src, W> x[AHEAD ? V : 1], res[AHEAD ? V : 1];
  const auto fetch = [&](int64_t row) {
#pragma unroll
    for (int j = 0; j < (AHEAD ? V : 0); ++j) x[j].load(static_cast<const Src *>(p.x) + row * p.x_stride, at(j), p.dim);
    if (p.residual) {
#pragma unroll
      for (int j = 0; j < (AHEAD ? V : 0); ++j)
        res[j].load(static_cast<const Src *>(p.residual) + row * p.residual_stride, at(j), p.dim);
    }
  };
  const auto weights = [&](int j, float (&w)[W]) {
    if (p.weight_f32) load_unit<W>(static_cast<const float *>(p.weight), at(j), p.dim, w);
    else load_unit<W>(static_cast<const uint16_t *>(p.weight), at(j), p.dim, w);
  };
  int flip = 0;
  // f's sum or largest value over the row's threads, in a fixed order
  const auto over_row = [&](float v, auto f) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    if (nt == 32) return v;
    flip ^= 1;
    if (lane == 0) part[flip][warp] = v;
    __syncthreads();  // the other half may still be read, this one is no longer
    v = lane < (nt >> 5) ? part[flip][lane] : 0.0f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v = f(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    return v;
  };

  if constexpr (AHEAD) fetch(r);
  float4 *own = norm_factors + threadIdx.y * nt + t;
  const int apart = nt * static_cast<int>(blockDim.y);
  if constexpr (W == 16) {
    if (p.weight) {
      float w[W];
      weights(0, w);
#pragma unroll
      for (int i = 0; i < 4; ++i)
        own[i * apart] = make_float4(w[4 * i] + p.weight_offset, w[4 * i + 1] + p.weight_offset,
                                      w[4 * i + 2] + p.weight_offset, w[4 * i + 3] + p.weight_offset);
    }
  }
  for (; r < p.n_rows; r += step) {
    float h[V][W];
    if constexpr (AHEAD) {
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < W; ++e) h[j][e] = x[j].at(e);
      if (p.residual) {
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int e = 0; e < W; ++e) h[j][e] += res[j].at(e);
      }
    } else {
      const Src *from = static_cast<const Src *>(p.x) + r * p.x_stride;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        x[0].load(from, at(j), p.dim);
#pragma unroll
        for (int e = 0; e < W; ++e) h[j][e] = x[0].at(e);
      }
      if (p.residual) {
        from = static_cast<const Src *>(p.residual) + r * p.residual_stride;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          res[0].load(from, at(j), p.dim);
#pragma unroll
          for (int e = 0; e < W; ++e) h[j][e] += res[0].at(e);
        }
      }
    }
    if constexpr (AHEAD) {
      if (r + step < p.n_rows) fetch(r + step);
    }
    if (p.residual_out) {
      Src *ro = static_cast<Src *>(p.residual_out) + r * p.residual_out_stride;
#pragma unroll
      for (int j = 0; j < V; ++j) store_unit<W>(ro, at(j), p.dim, h[j]);
    }

    const auto squares = [&]() {
      uint64_t two = 0;
#pragma unroll
      for (int j = 0; j < V; ++j)
#pragma unroll
        for (int e = 0; e < W; e += 2) {
          const uint64_t v = pair_of(h[j][e], h[j][e + 1]);
          two = fma2(v, v, two);
        }
      float even, odd;
      parts_of(two, even, odd);
      return over_row(even + odd, [](float u, float v) { return u + v; });
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
        for (int e = 0; e < W; ++e) a = max_nan(a, fabsf(h[j][e]));
      a = over_row(a, [](float u, float v) { return max_nan(u, v); });
      float down = 1.0f;
      if (a > 0.0f && a < INFINITY) {
        // 2^-e, at most two powers off where it would not be normal
        const int up = static_cast<int>(__float_as_uint(a) >> 23) - 127;
        down = __uint_as_float(static_cast<uint32_t>(127 - min(max(up, -126), 126)) << 23);
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int e = 0; e < W; ++e) h[j][e] *= down;
      }
      ss = squares();
      const float scaled_eps = p.eps * down * down;
      if (scaled_eps < INFINITY) {
        rstd = __frsqrt_rn(__fdiv_rn(ss, static_cast<float>(p.dim)) + scaled_eps);
      } else {  // eps is all that counts
        rstd = __frsqrt_rn(p.eps);
#pragma unroll
        for (int j = 0; j < V; ++j)
#pragma unroll
          for (int e = 0; e < W; ++e) h[j][e] = __fdiv_rn(h[j][e], down);
      }
    }

    Out *out = static_cast<Out *>(p.out) + r * p.out_stride;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float y[W];
      if (p.weight) {
        uint64_t f[W / 2];
        if constexpr (W == 16) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 v = own[i * apart];
            f[2 * i] = pair_of(v.x, v.y);
            f[2 * i + 1] = pair_of(v.z, v.w);
          }
        } else {
          float w[W];
          weights(j, w);
#pragma unroll
          for (int e = 0; e < W; e += 2)
            f[e / 2] = fma2(pair_of(w[e], w[e + 1]), both_of(1.0f), both_of(p.weight_offset));
        }
#pragma unroll
        for (int e = 0; e < W; e += 2)
          parts_of(mul2(mul2(pair_of(h[j][e], h[j][e + 1]), both_of(rstd)), f[e / 2]), y[e], y[e + 1]);
      } else {
#pragma unroll
        for (int e = 0; e < W; ++e) y[e] = h[j][e] * rstd;
      }
      if constexpr (sizeof(Out) == 1) {
        const float scale = scaled_block<W>(y);
        if ((lane & (U::kLanes - 1)) == 0 && at(j) < p.dim)
          p.scale[r * p.scale_stride + at(j) / kScaleBlock] = scale;
      }
      store_unit<W>(out, at(j), p.dim, y);
    }
  }
}

}  // namespace ts
