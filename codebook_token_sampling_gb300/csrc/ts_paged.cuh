// ts_paged.cuh -- attention of one new token per request over a paged
// key-value cache.  For query head h of request r, with key head h / G and the
// attended tokens t (t < len_r, inside the window, not masked):
//   s_t = scale * q . k_t,  optionally  cap * tanh(s_t / cap)
//   o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m),  m = max_t s_t,
//   lse = m + ln sum_t e^(s_t - m).
// Every key and value row is read once and serves the G query heads that
// share it: 4 G flops per 2-byte element, so the bound is DRAM.
//
// Work.  An item is one (request, key head, piece of at most kRows query
// heads); its tokens are cut into tiles of 64 (32 for fp32 rows of 1 KB), and the tiles of all items,
// laid end to end, are dealt to the CTAs in equal runs.  Every CTA finds its
// run by summing the lengths itself, so ragged batches balance with nothing
// planned on the host and no launch before this one.  A run holds whole items
// and at most two pieces of items, which go to a workspace and are joined by
// paged_join_kernel.
//
// A CTA is four warps; warp w takes the w-th quarter of a tile's tokens with a
// running maximum and sum of its own and a private ring of cp.async stages (a
// quarter's K and V each), so no warp waits for another inside an item.
// The ring runs on across items.  At an item's end the four warps' results
// are joined in shared memory.
#pragma once

#include <type_traits>

#include "ts_kv.cuh"
#include "ts_lmhead.cuh"

namespace ts {

constexpr int kPagedThreads = 128;
constexpr int kPagedWarps = 4;
constexpr int kPagedPage = 16;                       // a stage's tokens divide this
constexpr int kPagedRows = 16;                       // most query heads per item
constexpr int kPagedMaxDim = 256;

// A piece of an item in the workspace: kPagedRows rows of kPagedMaxDim sums,
// and each row's maximum and sum.
struct PagedDesc {
  int32_t request, head, parts, pad;  // parts > 1: the item starts in this CTA
};
constexpr size_t kPagedAccBytes = sizeof(float) * kPagedRows * kPagedMaxDim;
constexpr size_t paged_workspace_bytes(int ctas) {
  return static_cast<size_t>(ctas) *
         (sizeof(PagedDesc) + 2 * (kPagedAccBytes + sizeof(float2) * kPagedRows));
}

struct PagedParams {
  const void *q;
  int64_t q_req, q_head;    // elements
  void *out;
  int64_t o_req, o_head;
  float *lse;               // [n_requests][n_heads] or null
  const uint8_t *mask;      // or null
  int64_t mask_stride;
  const int32_t *table;
  int64_t table_stride;
  int32_t max_blocks;
  const int32_t *lens;
  int32_t n_requests;
  const void *k, *v;
  int64_t k_block, k_token, k_head;  // bytes
  int64_t v_block, v_token, v_head;
  const float *k_scale, *v_scale;
  int32_t n_blocks, block_size, kv_heads, dim;
  int32_t group;            // query heads per key head
  int32_t pieces;           // items per (request, key head)
  int32_t rows;             // query heads of a full item
  float scale, softcap;
  int32_t window;           // 0: none
  FastDiv by_block;
  PagedDesc *desc;
  float *acc;               // [2 ctas][kPagedRows][kPagedMaxDim]
  float2 *ml;               // [2 ctas][kPagedRows]
  int32_t ctas;             // of the main launch
  int32_t out_f32;
  uint32_t *status;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// 2^(m - top), 0 for an empty part
__device__ __forceinline__ float exp2_from(float m, float top) {
  return m == -INFINITY ? 0.0f : exp2f(m - top);
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void *gmem, bool real) {
  const int n = real ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem), "l"(gmem), "r"(n)
               : "memory");
}

__device__ __forceinline__ void ldmatrix_x4_at(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans_at(uint32_t (&r)[4], uint32_t a) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                              uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
      "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two e4m3 values as two f16 values (exact)
__device__ __forceinline__ uint32_t f16x2_of_e4m3x2(uint32_t x) {
  uint32_t d;
  const uint16_t h = static_cast<uint16_t>(x);
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(h));
  return d;
}
__device__ __forceinline__ uint32_t bf16x2_of(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t f16x2_of(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// A stage row's 16-byte chunk c sits at chunk c ^ (a function of the row), so
// that the eight rows of a matrix load (or the lanes of a vector load) fall on
// different banks.
// LANES: lanes that read one row side by side (0: matrix loads).
template <int ROW_BYTES, int LANES>
__device__ __forceinline__ uint32_t stage_at(int row, int chunk) {
  constexpr int kChunks = ROW_BYTES / 16;
  int c;
  if constexpr (LANES > 0) c = chunk ^ (LANES * (row & (8 / LANES - 1)));
  else if constexpr (kChunks >= 8) c = chunk ^ (row & 7);
  else c = chunk ^ ((row >> 1) & 3);
  return static_cast<uint32_t>(row * ROW_BYTES + c * 16);
}

// --------------------------------------------------------------------------
// One warp's arithmetic on the tensor cores (bf16 and e4m3 caches): 16 query
// heads x 16 tokens x DP elements.  Rows past the item's heads are zero.
// --------------------------------------------------------------------------
template <bool E4M3, int DP>
struct MmaCore {
  static constexpr int kRows = 16;
  static constexpr int kTok = 16;
  static constexpr int kPer = 0;
  static constexpr bool kFma = false;
  static constexpr int kElemBytes = E4M3 ? 1 : 2;
  static constexpr int kRowBytes = DP * kElemBytes;
  static constexpr uint32_t kQBytes = 0;     // shared memory of the CTA's queries
  static constexpr uint32_t kWarpBytes = 0;  // of a warp's own
  static constexpr int kKSteps = DP / 16;

  uint32_t qf[kKSteps][4];
  float o[DP / 8][4];
  float m[2], l[2];  // rows g and g + 8; l: this lane's tokens only
  float sc[2];       // score factor of the rows

  __device__ __forceinline__ void begin(const PagedParams &p, const uint16_t *q, int rows,
                                        float k_scale, void *) {
    const int lane = static_cast<int>(lane_id()), g = lane >> 2, tg = lane & 3;
    const float unit = p.softcap > 0.0f ? p.scale * k_scale : p.scale * k_scale * kLog2e;
    const uint16_t *row[2] = {q + g * p.q_head, q + (g + 8) * p.q_head};
    const bool real[2] = {g < rows, g + 8 < rows};
    if constexpr (!E4M3) {
#pragma unroll
      for (int kk = 0; kk < kKSteps; ++kk) {
#pragma unroll
        for (int a = 0; a < 4; ++a) {
          const int c = kk * 16 + 2 * tg + (a >> 1) * 8;
          qf[kk][a] = real[a & 1] && c < p.dim
                          ? *reinterpret_cast<const uint32_t *>(row[a & 1] + c) : 0u;
        }
      }
      sc[0] = sc[1] = unit;
    } else {
      // The cache's values are exact in f16, a bf16 query is not in f16's
      // range: each row is divided by a power of two that brings its largest
      // element into [1, 2).  What f16 then drops is below 2^-25 of that.
      // Elements 4 tg .. 4 tg + 3 of a 16-element step stand in the places
      // 2 tg, 2 tg + 1, 2 tg + 8, 2 tg + 9, as the keys' bytes do.
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint2 raw[kKSteps];
        float big = 0.0f;
#pragma unroll
        for (int kk = 0; kk < kKSteps; ++kk) {
          const int c = kk * 16 + 4 * tg;
          raw[kk] = real[h] && c < p.dim ? *reinterpret_cast<const uint2 *>(row[h] + c)
                                         : make_uint2(0u, 0u);
          big = fmaxf(big, fmaxf(fmaxf(fabsf(__uint_as_float(raw[kk].x << 16)),
                                       fabsf(__uint_as_float(raw[kk].x & 0xFFFF0000u))),
                                 fmaxf(fabsf(__uint_as_float(raw[kk].y << 16)),
                                       fabsf(__uint_as_float(raw[kk].y & 0xFFFF0000u)))));
        }
        big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
        const int e = big > 0.0f && big < INFINITY ? ilogbf(big) : 0;
        const auto half_of = [&](uint32_t w) {
          return f16x2_of(scalbnf(__uint_as_float(w << 16), -e),
                          scalbnf(__uint_as_float(w & 0xFFFF0000u), -e));
        };
#pragma unroll
        for (int kk = 0; kk < kKSteps; ++kk) {
          qf[kk][h] = half_of(raw[kk].x);
          qf[kk][2 + h] = half_of(raw[kk].y);
        }
        sc[h] = scalbnf(unit, e);
      }
    }
#pragma unroll
    for (int n = 0; n < DP / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.0f;
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.0f;
  }

  __device__ __forceinline__ void poison() { l[0] = l[1] = __int_as_float(0x7FC00000); }

  // 16 tokens: K rows at shared address ks, V rows at vs, bit t of `valid` set
  // where token t is attended (the others' rows are zero)
  __device__ __forceinline__ void step(const PagedParams &p, uint32_t ks, uint32_t vs,
                                       uint32_t valid, void *) {
    const int lane = static_cast<int>(lane_id()), tg = lane & 3;
    float s[2][4] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    if constexpr (!E4M3) {
      const int row = (lane & 7) + ((lane >> 4) << 3), half = (lane >> 3) & 1;
#pragma unroll
      for (int kk = 0; kk < kKSteps; ++kk) {
        uint32_t b[4];
        ldmatrix_x4_at(b, ks + stage_at<kRowBytes, 0>(row, 2 * kk + half));
        mma_bf16_16816(s[0], qf[kk], b[0], b[1]);
        mma_bf16_16816(s[1], qf[kk], b[2], b[3]);
      }
    } else {
      const int row = (lane & 7) + (((lane >> 3) & 1) << 3), half = lane >> 4;
#pragma unroll
      for (int k2 = 0; k2 < kKSteps / 2; ++k2) {
        uint32_t b[4];
        ldmatrix_x4_at(b, ks + stage_at<kRowBytes, 0>(row, 2 * k2 + half));
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mma_f16_16816(s[e & 1], qf[2 * k2 + (e >> 1)], f16x2_of_e4m3x2(b[e]),
                        f16x2_of_e4m3x2(b[e] >> 16));
      }
    }
    // scores in units of ln 2, unattended ones at -inf
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float x = s[n][e] * sc[e >> 1];
        if (p.softcap > 0.0f) x = p.softcap * tanhf(x / p.softcap) * kLog2e;
        s[n][e] = x;
      }
    if (valid != 0xFFFFu) {
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (!((valid >> (n * 8 + 2 * tg + (e & 1))) & 1u)) s[n][e] = -INFINITY;
    }
    float base[2];
    bool moved = false;
    float drop[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
      x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 1));
      x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 2));
      const float top = fmaxf(m[h], x);
      base[h] = top == -INFINITY ? 0.0f : top;  // a row with nothing yet
      drop[h] = exp2_from(m[h], base[h]);
      moved |= top != m[h];
      m[h] = top;
    }
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
      for (int n = 0; n < DP / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] *= drop[e >> 1];
      l[0] *= drop[0];
      l[1] *= drop[1];
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s[n][e] = exp2f(s[n][e] - base[e >> 1]);
        l[e >> 1] += s[n][e];
      }
    // The weights as the products' left side.  bf16 values carry V: a weight
    // goes in as the sum of two bf16 numbers, its upper half and what is left,
    // so that less than 2^-16 of it is lost and the output's own rounding stays
    // the largest error.  The second number is kept above zero (by 2^-20 of the
    // weight): an attended infinity in V then comes out as one, not as the NaN
    // of 0 times it.  An f16 weight (e4m3 values) keeps 11 bits, enough for the
    // same, and e4m3 has no infinities.
    uint32_t a[4], a2[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = s[i >> 1][2 * (i & 1)], y = s[i >> 1][2 * (i & 1) + 1];
      if constexpr (E4M3) {
        a[i] = f16x2_of(x, y);
      } else {
        const uint32_t ux = __float_as_uint(x), uy = __float_as_uint(y);
        a[i] = __byte_perm(ux, uy, 0x7632);
        a2[i] = bf16x2_of(fmaf(x, 0x1p-20f, x - __uint_as_float(ux & 0xFFFF0000u)),
                          fmaf(y, 0x1p-20f, y - __uint_as_float(uy & 0xFFFF0000u)));
      }
    }
    const int vrow = (lane & 7) + (((lane >> 3) & 1) << 3), vhalf = lane >> 4;
    if constexpr (!E4M3) {
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) {
        uint32_t b[4];
        ldmatrix_x4_trans_at(b, vs + stage_at<kRowBytes, 0>(vrow, 2 * d + vhalf));
        mma_bf16_16816(o[2 * d], a, b[0], b[1]);
        mma_bf16_16816(o[2 * d + 1], a, b[2], b[3]);
        mma_bf16_16816(o[2 * d], a2, b[0], b[1]);
        mma_bf16_16816(o[2 * d + 1], a2, b[2], b[3]);
      }
    } else {
      // A transposed load of 16-bit units hands a lane elements 2 g, 2 g + 1
      // of tokens 2 tg, 2 tg + 1: the even elements make one product's column
      // g, the odd ones another's.
#pragma unroll
      for (int d2 = 0; d2 < DP / 32; ++d2) {
        uint32_t b[4];
        ldmatrix_x4_trans_at(b, vs + stage_at<kRowBytes, 0>(vrow, 2 * d2 + vhalf));
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __byte_perm(b[i], 0u, 0x3120);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mma_f16_16816(o[4 * d2 + 2 * h], a, f16x2_of_e4m3x2(b[2 * h]), f16x2_of_e4m3x2(b[2 * h + 1]));
          mma_f16_16816(o[4 * d2 + 2 * h + 1], a, f16x2_of_e4m3x2(b[2 * h] >> 16),
                        f16x2_of_e4m3x2(b[2 * h + 1] >> 16));
        }
      }
    }
  }

  // Each row's maximum and sum to the warp's places.
  __device__ __forceinline__ void give_ml(float *sm, float *sl) {
    const int lane = static_cast<int>(lane_id()), g = lane >> 2, tg = lane & 3;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x = l[h];
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 1);
      x += __shfl_xor_sync(0xFFFFFFFFu, x, 2);
      if (tg == 0) {
        sm[g + 8 * h] = m[h];
        sl[g + 8 * h] = x;
      }
    }
  }

  // Adds the warp's scaled sums to the buffer (rows of DP + 8 floats).  In
  // round i the warps work on different quarters of the columns, each quarter
  // being begun by one warp and added to by the others in a fixed order.
  static constexpr int kPitch = DP + 8;
  __device__ __forceinline__ void add_round(float *buf, int round, int warp, const float *top,
                                            int rows) {
    const int lane = static_cast<int>(lane_id()), g = lane >> 2, tg = lane & 3;
    const int mine = (warp + round) & 3;
    const float f[2] = {exp2_from(m[0], top[g]), exp2_from(m[1], top[g + 8])};
#pragma unroll
    for (int qd = 0; qd < 4; ++qd) {
      if (qd != mine) continue;
#pragma unroll
      for (int n = qd * DP / 32; n < (qd + 1) * DP / 32; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (g + 8 * h >= rows) continue;
          float *b = buf + (g + 8 * h) * kPitch;
          if constexpr (!E4M3) {
            float2 *at = reinterpret_cast<float2 *>(b + n * 8 + 2 * tg);
            float2 x = make_float2(o[n][2 * h] * f[h], o[n][2 * h + 1] * f[h]);
            if (round) {
              const float2 y = *at;
              x.x += y.x;
              x.y += y.y;
            }
            *at = x;
          } else if ((n & 1) == 0) {
            float4 *at = reinterpret_cast<float4 *>(b + n * 8 + 4 * tg);
            float4 x = make_float4(o[n][2 * h] * f[h], o[n + 1][2 * h] * f[h],
                                   o[n][2 * h + 1] * f[h], o[n + 1][2 * h + 1] * f[h]);
            if (round) {
              const float4 y = *at;
              x.x += y.x;
              x.y += y.y;
              x.z += y.z;
              x.w += y.w;
            }
            *at = x;
          }
        }
      }
    }
  }
};

// --------------------------------------------------------------------------
// One warp's arithmetic in 32 bits (f32 cache): GR query heads, fused
// multiply-adds.  Scores: kPer lanes share a token, each taking every kPer-th
// 16-byte chunk of its key.  Outputs: a lane holds 4-element columns of all GR
// rows.
// --------------------------------------------------------------------------
template <int GR, int DP>
struct FmaCore {
  static constexpr int kRows = GR;
  static constexpr int kTok = DP > 128 ? 8 : 16;  // three stages fit beside each other
  static constexpr int kPer = 32 / kTok;
  static constexpr bool kFma = true;
  static constexpr int kElemBytes = 4;
  static constexpr int kRowBytes = DP * kElemBytes;
  static constexpr uint32_t kQBytes = GR * DP * 4;
  static constexpr uint32_t kWarpBytes = kTok * GR * 4;
  static constexpr int kLanes = DP / 4 < 32 ? DP / 4 : 32;  // lanes across a row
  static constexpr int kSplit = 32 / kLanes;                // tokens side by side
  static constexpr int kCols = DP / 128 > 0 ? DP / 128 : 1; // chunks per lane
  static constexpr int kPitch = DP;

  float o[GR][kCols * 4];
  float m[GR], l[GR];
  float sc;
  const float *q;

  __device__ __forceinline__ void begin(const PagedParams &p, const float *src, int rows,
                                        float k_scale, void *shared) {
    float *sq = static_cast<float *>(shared);
    q = sq;
    sc = p.softcap > 0.0f ? p.scale * k_scale : p.scale * k_scale * kLog2e;
    for (int i = static_cast<int>(threadIdx.x); i < GR * DP / 4; i += kPagedThreads) {
      const int r = i / (DP / 4), c = 4 * (i % (DP / 4));
      reinterpret_cast<float4 *>(sq)[i] = r < rows && c < p.dim
          ? *reinterpret_cast<const float4 *>(src + r * p.q_head + c)
          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    __syncthreads();
#pragma unroll
    for (int g = 0; g < GR; ++g) {
      m[g] = -INFINITY;
      l[g] = 0.0f;
#pragma unroll
      for (int c = 0; c < kCols * 4; ++c) o[g][c] = 0.0f;
    }
  }

  __device__ __forceinline__ void poison() {
#pragma unroll
    for (int g = 0; g < GR; ++g) l[g] = __int_as_float(0x7FC00000);
  }

  static __device__ __forceinline__ float4 lds4(uint32_t a) {
    float4 v;
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
    return v;
  }

  __device__ __forceinline__ void step(const PagedParams &p, uint32_t ks, uint32_t vs,
                                       uint32_t valid, void *own) {
    const int lane = static_cast<int>(lane_id()), t = lane / kPer, part = lane % kPer;
    float *sp = static_cast<float *>(own);  // [kTok][GR] weights
    float s[GR];
#pragma unroll
    for (int g = 0; g < GR; ++g) s[g] = 0.0f;
#pragma unroll 4
    for (int c = part; c < DP / 4; c += kPer) {
      const float4 k = lds4(ks + stage_at<kRowBytes, kPer>(t, c));
#pragma unroll
      for (int g = 0; g < GR; ++g) {
        const float4 x = reinterpret_cast<const float4 *>(q)[g * (DP / 4) + c];
        s[g] = fmaf(x.x, k.x, s[g]);
        s[g] = fmaf(x.y, k.y, s[g]);
        s[g] = fmaf(x.z, k.z, s[g]);
        s[g] = fmaf(x.w, k.w, s[g]);
      }
    }
    const bool on = (valid >> t) & 1u;
    bool moved = false;
    float drop[GR];
#pragma unroll
    for (int g = 0; g < GR; ++g) {
      float x = s[g];
#pragma unroll
      for (int w = 1; w < kPer; w <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
      x *= sc;
      if (p.softcap > 0.0f) x = p.softcap * tanhf(x / p.softcap) * kLog2e;
      if (!on) x = -INFINITY;
      s[g] = x;
#pragma unroll
      for (int w = kPer; w < 32; w <<= 1) x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, w));
      const float top = fmaxf(m[g], x);
      const float base = top == -INFINITY ? 0.0f : top;
      drop[g] = exp2_from(m[g], base);
      moved |= top != m[g];
      m[g] = top;
      s[g] = exp2f(s[g] - base);
    }
    if (moved) {  // the same in all lanes
#pragma unroll
      for (int g = 0; g < GR; ++g) {
        l[g] *= drop[g];
#pragma unroll
        for (int c = 0; c < kCols * 4; ++c) o[g][c] *= drop[g];
      }
    }
#pragma unroll
    for (int g = 0; g < GR; ++g) {
      if (part == 0) {
        l[g] += s[g];
        sp[t * GR + g] = s[g];
      }
    }
    __syncwarp();
    const int col = lane % kLanes, sub = lane / kLanes;
#pragma unroll 4
    for (int u = sub; u < kTok; u += kSplit) {
      float w[GR];
#pragma unroll
      for (int g = 0; g < GR; ++g) w[g] = sp[u * GR + g];
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        const float4 v = lds4(vs + stage_at<kRowBytes, kPer>(u, col + c * 32));
#pragma unroll
        for (int g = 0; g < GR; ++g) {
          o[g][4 * c] = fmaf(w[g], v.x, o[g][4 * c]);
          o[g][4 * c + 1] = fmaf(w[g], v.y, o[g][4 * c + 1]);
          o[g][4 * c + 2] = fmaf(w[g], v.z, o[g][4 * c + 2]);
          o[g][4 * c + 3] = fmaf(w[g], v.w, o[g][4 * c + 3]);
        }
      }
    }
    __syncwarp();  // the weights are read before the next step writes them
  }

  __device__ __forceinline__ void give_ml(float *sm, float *sl) {
    const int lane = static_cast<int>(lane_id());
#pragma unroll
    for (int g = 0; g < GR; ++g) {
      float x = l[g];
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
      if (lane == 0) {
        sm[g] = m[g];
        sl[g] = x;
      }
    }
  }

  // In round i warp i adds.
  __device__ __forceinline__ void add_round(float *buf, int round, int warp, const float *top, int) {
    const int lane = static_cast<int>(lane_id()), col = lane % kLanes;
    if (round != warp) return;
#pragma unroll
    for (int g = 0; g < GR; ++g) {
      const float f = exp2_from(m[g], top[g]);
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        float x[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = o[g][4 * c + e] * f;
          if constexpr (kSplit == 2) x[e] += __shfl_xor_sync(0xFFFFFFFFu, x[e], 16);
        }
        if (lane < kLanes) {
          float4 *at = reinterpret_cast<float4 *>(buf + g * kPitch + 4 * (col + c * 32));
          float4 y = make_float4(x[0], x[1], x[2], x[3]);
          if (round) {
            const float4 z = *at;
            y.x += z.x;
            y.y += z.y;
            y.z += z.z;
            y.w += z.w;
          }
          *at = y;
        }
      }
    }
  }
};

// --------------------------------------------------------------------------
// The kernel
// --------------------------------------------------------------------------
template <class Core, int NS>
struct PagedShape {
  static constexpr int kTile = Core::kTok * kPagedWarps;  // tokens
  static constexpr uint32_t kHalf = Core::kTok * Core::kRowBytes;  // K or V of a stage
  static constexpr uint32_t kRing = NS * 2 * kHalf;               // of a warp
  static constexpr uint32_t kBuf = Core::kRows * Core::kPitch * 4;
  static constexpr uint32_t kSmem =
      kPagedWarps * (kRing + Core::kWarpBytes) + Core::kQBytes + kBuf;
};

// Tiles of request r's items, 0 where nothing is attended; `bad`: its length
// is outside the table.
struct PagedSpan {
  int32_t len, first, t0, tiles;
};
template <int TILE>
__device__ __forceinline__ PagedSpan paged_span(const PagedParams &p, int32_t len, bool &bad) {
  PagedSpan s;
  bad = len < 0 || len > static_cast<int64_t>(p.max_blocks) * p.block_size;
  s.len = bad ? 0 : len;
  s.first = p.window > 0 && s.len > p.window ? s.len - p.window : 0;
  s.t0 = s.first & ~(kPagedPage - 1);
  s.tiles = (s.len - s.t0 + TILE - 1) / TILE;
  return s;
}

__device__ __forceinline__ void paged_store4(const PagedParams &p, int64_t at, float4 x) {
  if (p.out_f32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = x;
  } else {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
        make_uint2(bf16x2_of(x.x, x.y), bf16x2_of(x.z, x.w));
  }
}

// PAGE16: the block size is a multiple of 16, so that a stage's tokens lie in
// one block and one table entry is looked up per stage instead of one per
// token.
template <class Core, int NS, bool PAGE16>
__global__ void __launch_bounds__(kPagedThreads) paged_attention_kernel(const PagedParams p) {
  using Shape = PagedShape<Core, NS>;
  using Elem = std::conditional_t<Core::kFma, float, uint16_t>;  // of the queries
  extern __shared__ __align__(128) unsigned char paged_smem[];
  __shared__ uint32_t valid_ring[kPagedWarps][NS];
  __shared__ float sm[kPagedWarps][kPagedRows], sl[kPagedWarps][kPagedRows];
  __shared__ float s_top[kPagedRows], s_sum[kPagedRows];
  __shared__ int64_t s_part[kPagedWarps];
  __shared__ int64_t s_before;
  __shared__ int32_t s_request;

  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  unsigned char *ring = paged_smem + warp * Shape::kRing;
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  unsigned char *own = paged_smem + kPagedWarps * Shape::kRing + warp * Core::kWarpBytes;
  unsigned char *sq = paged_smem + kPagedWarps * (Shape::kRing + Core::kWarpBytes);
  float *buf = reinterpret_cast<float *>(sq + Core::kQBytes);
  pdl_wait_and_release();

  // ---- this CTA's run of tiles ----
  const int per_request = p.kv_heads * p.pieces;
  const int n_heads = p.kv_heads * p.group;
  uint32_t bits = 0;
  int64_t total = 0;
  for (int r = tid; r < p.n_requests; r += kPagedThreads) {
    bool bad;
    total += static_cast<int64_t>(paged_span<Shape::kTile>(p, p.lens[r], bad).tiles) * per_request;
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  if (lane == 0) s_part[warp] = total;
  __syncthreads();
  total = s_part[0] + s_part[1] + s_part[2] + s_part[3];
  const int64_t run = (total + p.ctas - 1) / p.ctas;
  const int64_t u0 = run * blockIdx.x;
  const int64_t u1 = min(u0 + run, total);
  __syncthreads();

  // requests with nothing to attend to are answered here
  for (int r = static_cast<int>(blockIdx.x); r < p.n_requests; r += p.ctas) {
    bool bad;
    const PagedSpan s = paged_span<Shape::kTile>(p, p.lens[r], bad);
    if (s.tiles > 0) continue;
    if (bad) bits |= kRowBadShape;
    const float x = bad ? __int_as_float(0x7FC00000) : 0.0f;
    for (int i = tid; i < n_heads * (p.dim / 4); i += kPagedThreads) {
      const int h = i / (p.dim / 4), c = 4 * (i - h * (p.dim / 4));
      paged_store4(p, r * p.o_req + h * p.o_head + c, make_float4(x, x, x, x));
    }
    if (p.lse)
      for (int h = tid; h < n_heads; h += kPagedThreads)
        p.lse[static_cast<int64_t>(r) * n_heads + h] = bad ? x : -INFINITY;
  }
  if (tid == 0) p.desc[blockIdx.x].parts = 0;
  if (u0 >= u1) {
    if (bits && tid == 0) atomicOr(p.status, bits);
    return;
  }

  // the request that holds tile u0
  for (int64_t seen = 0, r0 = 0; r0 < p.n_requests; r0 += kPagedThreads) {
    const int64_t r = r0 + tid;
    bool bad;
    int64_t mine = 0;
    if (r < p.n_requests)
      mine = static_cast<int64_t>(paged_span<Shape::kTile>(p, p.lens[r], bad).tiles) * per_request;
    int64_t in = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xFFFFFFFFu, in, o);
      if (lane >= o) in += x;
    }
    if (lane == 31) s_part[warp] = in;
    __syncthreads();
    int64_t before = seen + in - mine;
    for (int w = 0; w < warp; ++w) before += s_part[w];
    if (before <= u0 && u0 < before + mine) {
      s_request = static_cast<int32_t>(r);
      s_before = before;
    }
    seen += s_part[0] + s_part[1] + s_part[2] + s_part[3];
    __syncthreads();
    if (seen > u0) break;
  }

  // ---- cursors over the run ----
  struct Cursor {
    int64_t left;     // tiles of the run, this one included
    int32_t request, head, tile;  // head: key head * pieces + piece
    PagedSpan span;
  };
  const auto next = [&](Cursor &c) {
    --c.left;
    if (++c.tile == c.span.tiles) {
      c.tile = 0;
      if (++c.head == per_request) {
        c.head = 0;
        if (c.left > 0) {
          bool bad;
          do c.span = paged_span<Shape::kTile>(p, p.lens[++c.request], bad);
          while (c.span.tiles == 0);
        }
      }
    }
  };
  Cursor use;
  use.left = u1 - u0;
  use.request = s_request;
  {
    bool bad;
    use.span = paged_span<Shape::kTile>(p, p.lens[use.request], bad);
    const int64_t in = u0 - s_before;
    use.head = static_cast<int32_t>(in / use.span.tiles);
    use.tile = static_cast<int32_t>(in - static_cast<int64_t>(use.head) * use.span.tiles);
  }
  Cursor get = use;

  // ---- loading: a stage's table entry and mask byte are fetched one stage
  // before its rows ----
  int32_t entry = -1;
  bool keep = false;
  const auto look_up = [&]() {
    if (get.left <= 0) return;
    const int32_t base = get.span.t0 + get.tile * Shape::kTile + warp * Core::kTok;
    const int32_t t = base + lane % Core::kTok;
    keep = t >= get.span.first && t < get.span.len;
    entry = -1;
    if (PAGE16 ? base < get.span.len : keep)
      entry = p.table[get.request * p.table_stride +
                      p.by_block.div(static_cast<uint32_t>(PAGE16 ? base : t))];
    if (keep && p.mask) keep = p.mask[get.request * p.mask_stride + t] != 0;
  };
  const auto fetch = [&](int stage) {
    const int32_t base = get.span.t0 + get.tile * Shape::kTile + warp * Core::kTok;
    const bool inside = entry >= 0 && entry < p.n_blocks;
    constexpr uint32_t kAll = (1u << Core::kTok) - 1;
    const uint32_t want = __ballot_sync(0xFFFFFFFFu, keep) & kAll;
    const uint32_t valid = __ballot_sync(0xFFFFFFFFu, keep && inside) & kAll;
    // bit 31: a wanted token's block is outside the cache
    if (lane == 0) valid_ring[warp][stage] = valid | (want != valid ? 0x80000000u : 0u);
    const uint32_t ks = ring_at + stage * 2 * Shape::kHalf, vs = ks + Shape::kHalf;
    const int32_t kvh = get.head / p.pieces;
    const char *kb = static_cast<const char *>(p.k) + kvh * p.k_head;
    const char *vb = static_cast<const char *>(p.v) + kvh * p.v_head;
    constexpr int kChunks = Core::kRowBytes / 16;
    const int chunks = p.dim * Core::kElemBytes / 16;
    if constexpr (PAGE16) {
      const int32_t b = static_cast<int32_t>(p.by_block.div(static_cast<uint32_t>(base)));
      const int32_t off = base - b * p.block_size;
      const int64_t e = inside ? entry : 0;
      kb += e * p.k_block + off * p.k_token;
      vb += e * p.v_block + off * p.v_token;
    }
#pragma unroll
    for (int i = 0; i < Core::kTok * kChunks / 32; ++i) {
      const int c = lane + 32 * i, row = c / kChunks, ch = c % kChunks;
      const bool real = ((valid >> row) & 1u) && ch < chunks;
      const char *ka = kb, *va = vb;
      if constexpr (PAGE16) {
        if (real) {
          ka += row * p.k_token + ch * 16;
          va += row * p.v_token + ch * 16;
        }
      } else {
        const int64_t e = __shfl_sync(0xFFFFFFFFu, entry, row);
        if (real) {
          const uint32_t t = static_cast<uint32_t>(base + row);
          const int64_t off = t - p.by_block.div(t) * p.by_block.d;
          ka += e * p.k_block + off * p.k_token + ch * 16;
          va += e * p.v_block + off * p.v_token + ch * 16;
        }
      }
      const uint32_t at = stage_at<Core::kRowBytes, Core::kPer>(row, ch);
      cp_async16_or_zero(ks + at, ka, real);
      cp_async16_or_zero(vs + at, va, real);
    }
  };

  look_up();
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    if (get.left > 0) {
      fetch(s);
      next(get);
      look_up();
    }
    cp_async_commit();
  }

  // ---- the run ----
  Core core;
  int stage = 0, fill = NS - 1;
  bool fresh = true;      // the item's queries are not loaded yet
  bool from_start = true; // the run holds the item's first tile
  while (use.left > 0) {
    const int32_t kvh = use.head / p.pieces, h0 = (use.head - kvh * p.pieces) * p.rows;
    const int rows = min(p.rows, p.group - h0);
    if (fresh) {
      const Elem *q = static_cast<const Elem *>(p.q) + use.request * p.q_req +
                      (static_cast<int64_t>(kvh) * p.group + h0) * p.q_head;
      core.begin(p, q, rows, p.k_scale ? p.k_scale[kvh] : 1.0f, sq);
      from_start = use.tile == 0;
      fresh = false;
    }
    cp_async_wait_group<NS - 2>();
    __syncwarp();  // the stage is in, and the one before it is no longer read
    if (get.left > 0) {
      fetch(fill);
      next(get);
      look_up();
    }
    cp_async_commit();
    const uint32_t valid = valid_ring[warp][stage];
    const uint32_t ks = ring_at + stage * 2 * Shape::kHalf;
    if (valid & 0xFFFFu) core.step(p, ks, ks + Shape::kHalf, valid & 0xFFFFu, own);
    if (valid >> 31) {
      core.poison();
      bits |= kRowBadBlock;
    }
    stage = stage + 1 == NS ? 0 : stage + 1;
    fill = fill + 1 == NS ? 0 : fill + 1;

    const bool item_end = use.tile == use.span.tiles - 1;
    if (item_end || use.left == 1) {
      // ---- the four warps' parts as one ----
      core.give_ml(sm[warp], sl[warp]);
      __syncthreads();
      if (tid < Core::kRows) {
        float top = sm[0][tid];
#pragma unroll
        for (int w = 1; w < kPagedWarps; ++w) top = fmaxf(top, sm[w][tid]);
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kPagedWarps; ++w) sum += exp2_from(sm[w][tid], top) * sl[w][tid];
        s_top[tid] = top;
        s_sum[tid] = sum;
      }
      __syncthreads();
#pragma unroll 1
      for (int i = 0; i < kPagedWarps; ++i) {
        core.add_round(buf, i, warp, s_top, rows);
        __syncthreads();
      }
      const int quads = p.dim / 4;
      if (from_start && item_end) {
        const float vscale = p.v_scale ? p.v_scale[kvh] : 1.0f;
        const int64_t head = static_cast<int64_t>(kvh) * p.group + h0;
        for (int i = tid; i < rows * quads; i += kPagedThreads) {
          const int r = i / quads, c = 4 * (i - r * quads);
          const float sum = s_sum[r], f = sum == 0.0f ? 0.0f : vscale / sum;
          float4 x = *reinterpret_cast<const float4 *>(buf + r * Core::kPitch + c);
          x.x *= f;
          x.y *= f;
          x.z *= f;
          x.w *= f;
          paged_store4(p, use.request * p.o_req + (head + r) * p.o_head + c, x);
        }
        if (p.lse && tid < rows)
          p.lse[static_cast<int64_t>(use.request) * n_heads + head + tid] =
              s_top[tid] == -INFINITY && s_sum[tid] == 0.0f
                  ? -INFINITY : (s_top[tid] + log2f(s_sum[tid])) * kLn2;
      } else {
        // a piece: the item's first one goes to slot 1, the others are the
        // first thing in their CTA's run and go to slot 0
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (from_start ? 1 : 0);
        float *acc = p.acc + slot * kPagedRows * kPagedMaxDim;
        for (int i = tid; i < rows * quads; i += kPagedThreads) {
          const int r = i / quads, c = 4 * (i - r * quads);
          *reinterpret_cast<float4 *>(acc + r * kPagedMaxDim + c) =
              *reinterpret_cast<const float4 *>(buf + r * Core::kPitch + c);
        }
        if (tid < rows) p.ml[slot * kPagedRows + tid] = make_float2(s_top[tid], s_sum[tid]);
        if (from_start && tid == 0) {
          const int64_t more = use.span.tiles - 1 - use.tile;  // tiles in the CTAs after this one
          PagedDesc d;
          d.request = use.request;
          d.head = use.head;
          d.parts = static_cast<int32_t>(1 + (more + run - 1) / run);
          d.pad = 0;
          p.desc[blockIdx.x] = d;
        }
      }
      __syncthreads();  // the buffers are read before the next item's end writes them
      fresh = true;
    }
    next(use);
  }
  cp_async_wait_group<0>();
  if (bits && lane == 0) atomicOr(p.status, bits);
}

// Joins the items that are spread over several CTAs: block (c, h) takes row h
// of the item whose first piece is CTA c's last.  Each warp sums every fourth
// part, then the four are added up.
__global__ void __launch_bounds__(kPagedThreads) paged_join_kernel(const PagedParams p) {
  __shared__ float s_acc[kPagedWarps][kPagedMaxDim];
  __shared__ float s_top[kPagedWarps], s_sum[kPagedWarps];
  pdl_wait_and_release();
  const int c = static_cast<int>(blockIdx.x), row = static_cast<int>(blockIdx.y);
  const PagedDesc d = p.desc[c];
  if (d.parts < 2) return;
  const int32_t kvh = d.head / p.pieces, h0 = (d.head - kvh * p.pieces) * p.rows;
  if (row >= min(p.rows, p.group - h0)) return;
  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  const auto slot_of = [&](int j) { return 2 * static_cast<int64_t>(c + j) + (j == 0 ? 1 : 0); };

  float top = -INFINITY;
  for (int j = tid; j < d.parts; j += kPagedThreads)
    top = fmaxf(top, p.ml[slot_of(j) * kPagedRows + row].x);
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
  top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));

  float4 x[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
  float sum = 0.0f;
#pragma unroll 4
  for (int j = warp; j < d.parts; j += kPagedWarps) {
    const int64_t s = slot_of(j);
    const float2 ml = p.ml[s * kPagedRows + row];
    const float f = exp2_from(ml.x, top);
    sum += f * ml.y;
    const float *a = p.acc + (s * kPagedRows + row) * kPagedMaxDim;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = 4 * lane + 128 * i;
      if (col < p.dim) {
        const float4 y = *reinterpret_cast<const float4 *>(a + col);
        x[i].x = fmaf(f, y.x, x[i].x);
        x[i].y = fmaf(f, y.y, x[i].y);
        x[i].z = fmaf(f, y.z, x[i].z);
        x[i].w = fmaf(f, y.w, x[i].w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 2; ++i)
    *reinterpret_cast<float4 *>(&s_acc[warp][4 * lane + 128 * i]) = x[i];
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();
  sum = s_sum[0] + s_sum[1] + s_sum[2] + s_sum[3];
  const int64_t head = static_cast<int64_t>(kvh) * p.group + h0 + row;
  const float f = sum == 0.0f ? 0.0f : (p.v_scale ? p.v_scale[kvh] : 1.0f) / sum;
  for (int col = 4 * tid; col < p.dim; col += 4 * kPagedThreads) {
    float4 y = make_float4(0, 0, 0, 0);
#pragma unroll
    for (int w = 0; w < kPagedWarps; ++w) {
      y.x += s_acc[w][col];
      y.y += s_acc[w][col + 1];
      y.z += s_acc[w][col + 2];
      y.w += s_acc[w][col + 3];
    }
    paged_store4(p, d.request * p.o_req + head * p.o_head + col,
                 make_float4(y.x * f, y.y * f, y.z * f, y.w * f));
  }
  if (p.lse && tid == 0)
    p.lse[static_cast<int64_t>(d.request) * p.kv_heads * p.group + head] =
        top == -INFINITY && sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

}  // namespace ts
