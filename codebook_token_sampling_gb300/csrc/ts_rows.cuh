// ts_rows.cuh -- rows of a decode layer as the layer operators read and write them:
// a thread's piece of a row in fp32, and 8-bit rows with a scale for each 128
// elements.
#pragma once

#include <cuda_bf16.h>

#include "ts_e4m3.cuh"

namespace ts {

constexpr int kScaleBlock = 128;

// A lane's W elements of a block of 128: 8 or 16 neighbours (moved in pieces of 16 bytes,
// sixteen in pieces of 32), or with W 4 elements l, l + 32, l + 64 and l + 96 of lane l (any
// alignment and width, still one row segment per load).
template <int W>
struct RowUnit {
  static constexpr int kElems = W;
  static constexpr int kLanes = kScaleBlock / W;  // that share a block
  static constexpr bool kWide = W > 4;
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  uint32_t w;
  memcpy(&w, &v, 4);
  return w;
}
__device__ __forceinline__ uint16_t bf16_of(float x) { return __bfloat16_as_ushort(__float2bfloat16_rn(x)); }
__device__ __forceinline__ float value_of(float x) { return x; }
__device__ __forceinline__ float value_of(uint16_t bits) { return __uint_as_float(static_cast<uint32_t>(bits) << 16); }

// Eight neighbours from a 16-byte aligned address.
__device__ __forceinline__ void load8(const uint16_t *p, float *v) {
  const uint4 w = *reinterpret_cast<const uint4 *>(p);
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_lo(u[i]);
    v[2 * i + 1] = bf16_hi(u[i]);
  }
}
__device__ __forceinline__ void load8(const float *p, float *v) {
  const float4 a = reinterpret_cast<const float4 *>(p)[0], b = reinterpret_cast<const float4 *>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
  v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(uint16_t *p, const float *v) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(bf16x2_of(v[0], v[1]), bf16x2_of(v[2], v[3]), bf16x2_of(v[4], v[5]), bf16x2_of(v[6], v[7]));
}
__device__ __forceinline__ void store8(float *p, const float *v) {
  reinterpret_cast<float4 *>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4 *>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void store8(uint8_t *p, const float *v) {
  *reinterpret_cast<uint2 *>(p) =
      make_uint2(e4m3x4_of(v[0], v[1], v[2], v[3]), e4m3x4_of(v[4], v[5], v[6], v[7]));
}
// Sixteen, from 32-byte aligned addresses (8 bits: 16).
__device__ __forceinline__ void store16(uint16_t *p, const float *v) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = bf16x2_of(v[2 * i], v[2 * i + 1]);
  ulonglong4_32a q;
  memcpy(&q, w, 32);
  *reinterpret_cast<ulonglong4_32a *>(p) = q;
}
__device__ __forceinline__ void store16(float *p, const float *v) {
  ulonglong4_32a q[2];
  memcpy(q, v, 64);
  reinterpret_cast<ulonglong4_32a *>(p)[0] = q[0];
  reinterpret_cast<ulonglong4_32a *>(p)[1] = q[1];
}
__device__ __forceinline__ void store16(uint8_t *p, const float *v) {
  *reinterpret_cast<uint4 *>(p) =
      make_uint4(e4m3x4_of(v[0], v[1], v[2], v[3]), e4m3x4_of(v[4], v[5], v[6], v[7]),
                 e4m3x4_of(v[8], v[9], v[10], v[11]), e4m3x4_of(v[12], v[13], v[14], v[15]));
}
__device__ __forceinline__ void store1(float *p, float v) { *p = v; }
__device__ __forceinline__ void store1(uint16_t *p, float v) { *p = bf16_of(v); }
__device__ __forceinline__ void store1(uint8_t *p, float v) { *p = e4m3_of(v); }

// Two fp32 products and sums at once.
__device__ __forceinline__ uint64_t pair_of(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void parts_of(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t both_of(float a) { return pair_of(a, a); }

// A unit at element `at` of a row (its first neighbour, or its lane's first of four, 32
// apart); elements from `dim` on are 0 and not read.
template <int W, class T>
__device__ __forceinline__ void load_unit(const T *row, int64_t at, int64_t dim, float (&v)[W]) {
  if constexpr (RowUnit<W>::kWide) {
    if (at < dim) {
#pragma unroll
      for (int e = 0; e < W; e += 8) load8(row + at + e, v + e);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) v[e] = 0.0f;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = at + 32 * e < dim ? value_of(row[at + 32 * e]) : 0.0f;
  }
}
template <int W, class T>
__device__ __forceinline__ void store_unit(T *row, int64_t at, int64_t dim, const float (&v)[W]) {
  if constexpr (W == 16) {
    if (at < dim) store16(row + at, v);
  } else if constexpr (W == 8) {
    if (at < dim) store8(row + at, v);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (at + 32 * e < dim) store1(row + at + 32 * e, v[e]);
  }
}

// A unit as it is stored, on its way while the one before it is worked on.
template <class T, int W>
struct RawUnit {
  uint32_t w[W * sizeof(T) / 4];
  __device__ __forceinline__ void load(const T *row, int at, int dim) {
    if constexpr (W == 16) {
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) {
        ulonglong4_32a v = {0, 0, 0, 0};
        if (at < dim) v = reinterpret_cast<const ulonglong4_32a *>(row + at)[i];
        memcpy(w + 8 * i, &v, 32);
      }
    } else if constexpr (W == 8) {
#pragma unroll
      for (int i = 0; i < W * static_cast<int>(sizeof(T)) / 16; ++i) {
        const uint4 v = at < dim ? reinterpret_cast<const uint4 *>(row + at)[i] : make_uint4(0, 0, 0, 0);
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else {
      T e[W];
#pragma unroll
      for (int i = 0; i < W; ++i) e[i] = at + 32 * i < dim ? row[at + 32 * i] : T(0);
      memcpy(w, e, sizeof w);
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
};

// The larger one, keeping a NaN; the latter of three sizes.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max_size(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The scale of the block that a unit belongs to (the lanes that share it take
// part), and the unit's elements over it.
template <int W>
__device__ __forceinline__ float scaled_block(float (&v)[W]) {
  float a = max_size(v[0], v[1], v[2]);
#pragma unroll
  for (int e = 3; e + 1 < W; e += 2) a = max_size(a, v[e], v[e + 1]);
  a = max_size(a, v[W - 1], 0.0f);
#pragma unroll
  for (int o = RowUnit<W>::kLanes / 2; o; o >>= 1) a = max_nan(a, __shfl_xor_sync(0xFFFFFFFFu, a, o));
  // a / 448 correctly rounded (the quotient and one correction by its remainder, as above)
  const float top = fmaxf(a, 0x1p-64f), q = top * (1.0f / 448.0f);
  float scale = fmaf(fmaf(-q, 448.0f, top), 1.0f / 448.0f, q);
  if (!(a < INFINITY)) scale = __int_as_float(0x7FC00000);  // a NaN or an infinity in the block
  const uint64_t inv = both_of(__frcp_rn(scale));
#pragma unroll
  for (int e = 0; e < W; e += 2) parts_of(mul2(pair_of(v[e], v[e + 1]), inv), v[e], v[e + 1]);
  return scale;
}

}  // namespace ts
