// ts_rotary.cuh -- rotary positions (ts_rotary), and the same on the way into the
// paged cache (ts_kv_append_rotary).
#pragma once

#include "ts_kv_common.cuh"
#include "ts_rows.cuh"

namespace ts {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryTokens = 64;       // of a CTA at most
constexpr int kRotaryTableFloats = 8192;  // cosines and sines of a CTA's tokens, at most

struct RotaryParams {
  const void *x;                   // queries
  void *out;
  int64_t x_token, x_head, out_token, out_head;  // strides in elements
  const int32_t *positions;
  const int32_t *rows;             // or null
  const double *freqs;
  float amplitude;
  int32_t n_tokens, n_rows, heads, dim, half;  // half: pairs of a head
  int32_t interleaved, in_place;
  int32_t tokens_per_cta;
  FastDiv by_token, by_head;       // units of 2 P elements per token and per head
  uint32_t *status;
  // the cache's part
  const void *src[2];              // keys and values of the new tokens
  int64_t src_token[2], src_head[2];
  void *dst[2];
  int64_t dst_block[2], dst_token[2], dst_head[2];
  const float *scale[2];           // or null
  const int64_t *slots;
  int64_t n_slots, block_size;
  int32_t kv_heads;
};

// P elements as they are stored.
template <class T, int P>
struct Piece {
  static constexpr int kBytes = P * static_cast<int>(sizeof(T));
  static constexpr int kWords = (kBytes + 3) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const T *p) {
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = reinterpret_cast<const uint4 *>(p)[i];
        w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
      }
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2 *>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t *>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t *>(p);
    }
  }
  __device__ __forceinline__ void store(T *p) const {
    if constexpr (kBytes % 16 == 0) {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else if constexpr (kBytes == 8) {
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else if constexpr (kBytes == 4) {
      *reinterpret_cast<uint32_t *>(p) = w[0];
    } else {
      *reinterpret_cast<uint16_t *>(p) = static_cast<uint16_t>(w[0]);
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    else return (i & 1) ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
  }
  __device__ __forceinline__ void set(const float (&v)[P]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < P; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (P == 1) {
      w[0] = bf16_of(v[0]);
    } else {
#pragma unroll
      for (int i = 0; i < P / 2; ++i) w[i] = bf16x2_of(v[2 * i], v[2 * i + 1]);
    }
  }
};

// P quotients by a scale, rounded to e4m3 (as ts_kv_append rounds them).
template <int P>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&v)[P], float scale, float inv) {
  float y[P];
  bool fine = inv != 0.0f;
#pragma unroll
  for (int i = 0; i < P; ++i) fine &= quotient(v[i], scale, inv, y[i]);
  if (!fine) {
#pragma unroll 1
    for (int i = 0; i < P; ++i) p[i] = e4m3_of(__fdiv_rn(v[i], scale));
    return;
  }
  if constexpr (P == 8) {
    *reinterpret_cast<uint2 *>(p) = make_uint2(e4m3x4_of(y[0], y[1], y[2], y[3]), e4m3x4_of(y[4], y[5], y[6], y[7]));
  } else if constexpr (P == 4) {
    *reinterpret_cast<uint32_t *>(p) = e4m3x4_of(y[0], y[1], y[2], y[3]);
  } else {
    p[0] = e4m3_of(y[0]);
  }
}

// A frequency (radians per position) as turns in units of 2^-64, modulo a turn: the
// product with a position, modulo 2^64, is then the angle's exact fraction of a turn.
__device__ __forceinline__ uint64_t turns_of(double freq) {
  const double t = freq * 0.15915494309189535;  // 1 / (2 pi)
  return static_cast<uint64_t>((t - floor(t)) * 18446744073709551616.0);
}

// A CTA takes whole tokens.  Each angle's cosine and sine are computed once for all
// of a token's heads and go through shared memory; a unit is P elements and the P
// that they are paired with (or 2 P that are only copied).  Bound by DRAM for
// prompts, by latency for a frame.  CACHE: Dst is the cache's type.
template <class Src, class Dst, int P, bool CACHE>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const RotaryParams p) {
  constexpr int kUnroll = P == 8 && sizeof(Src) == 4 ? 2 : 4;
  extern __shared__ __align__(16) float rotary_smem[];
  __shared__ int64_t row_of[kRotaryTokens];
  __shared__ int32_t block_of[kRotaryTokens], off_of[kRotaryTokens];
  const int t = static_cast<int>(threadIdx.x);
  const int32_t t0 = static_cast<int32_t>(blockIdx.x) * p.tokens_per_cta;
  const int nt = min(p.tokens_per_cta, p.n_tokens - t0);
  float *cosines = rotary_smem, *sines = rotary_smem + p.tokens_per_cta * p.half;
  pdl_wait_and_release();

  uint32_t bits = 0;
  if (t < nt) {
    const int32_t pos = p.positions[t0 + t];
    int64_t slot = 0, row = t0 + t;
    if constexpr (CACHE) slot = p.slots[t0 + t];
    bool skip = pos < 0 || slot < 0;
    if (!skip && p.rows) {
      row = p.rows[t0 + t];
      if (row < 0 || row >= p.n_rows) {
        skip = true;
        bits |= kRowBadSlot;
      }
    }
    if constexpr (CACHE) {
      if (!skip && slot >= p.n_slots) {
        skip = true;
        bits |= kRowBadSlot;
      }
    }
    row_of[t] = skip ? -1 : row;
    if constexpr (CACHE) {
      const int64_t blk = skip ? 0 : slot / p.block_size;
      block_of[t] = static_cast<int32_t>(blk);
      off_of[t] = static_cast<int32_t>(skip ? 0 : slot - blk * p.block_size);
    }
  }
  for (int i0 = 0; i0 < p.half; i0 += kRotaryThreads) {
    const int width = min(kRotaryThreads, p.half - i0), groups = kRotaryThreads / width;
    const int g = t / width, i = i0 + t - g * width;
    if (g < groups) {
      const uint64_t f = turns_of(p.freqs[i]);
      for (int k = g; k < nt; k += groups) {
        const uint64_t turn = f * static_cast<uint64_t>(static_cast<int64_t>(p.positions[t0 + k]));
        // the nearest 2^-32 of a turn, as half turns from -1 to 1
        const int32_t top = static_cast<int32_t>((turn + 0x80000000ull) >> 32);
        float s, c;
        sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
        cosines[k * p.half + i] = p.amplitude * c;
        sines[k * p.half + i] = p.amplitude * s;
      }
    }
  }
  __syncthreads();

  const uint32_t units = static_cast<uint32_t>(nt) * p.by_token.d;
  const int rot_units = p.half / P;
  struct Unit {
    int token, head, u, which, a, b;  // which: 0 queries, 1 keys, 2 values
    bool rotates;
  };
  const auto unit_of = [&](uint32_t x) {
    Unit n;
    n.token = static_cast<int>(p.by_token.div(x));
    const uint32_t in = x - static_cast<uint32_t>(n.token) * p.by_token.d;
    n.head = static_cast<int>(p.by_head.div(in));
    n.u = static_cast<int>(in) - n.head * static_cast<int>(p.by_head.d);
    n.which = 0;
    if constexpr (CACHE) {
      if (n.head >= p.heads) {
        n.head -= p.heads;
        n.which = 1;
        if (n.head >= p.kv_heads) {
          n.head -= p.kv_heads;
          n.which = 2;
        }
      }
    }
    n.rotates = n.which != 2 && n.u < rot_units;
    if (n.rotates && !p.interleaved) {
      n.a = n.u * P;
      n.b = p.half + n.a;
    } else {  // neighbours, rotated or copied
      n.a = n.u * 2 * P;
      n.b = n.a + P;
    }
    return n;
  };

  for (uint32_t x0 = t; x0 < units; x0 += kRotaryThreads * kUnroll) {
    Piece<Src, P> va[kUnroll], vb[kUnroll];
    bool there[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t x = x0 + j * kRotaryThreads;
      there[j] = x < units;
      if (!there[j]) continue;
      const Unit n = unit_of(x);
      const int64_t row = row_of[n.token];
      there[j] = row >= 0 && !(n.which == 0 && p.in_place && !n.rotates);
      if (!there[j]) continue;
      const Src *from;
      if (!CACHE || n.which == 0) from = static_cast<const Src *>(p.x) + row * p.x_token + n.head * p.x_head;
      else from = static_cast<const Src *>(p.src[n.which - 1]) + row * p.src_token[n.which - 1] + n.head * p.src_head[n.which - 1];
      va[j].load(from + n.a);
      if (n.b < p.dim) vb[j].load(from + n.b);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (!there[j]) continue;
      const Unit n = unit_of(x0 + j * kRotaryThreads);
      const bool both = n.b < p.dim;
      float a[P], b[P];
      if (n.rotates || (CACHE && n.which != 0 && sizeof(Dst) == 1)) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          a[i] = va[j].at(i);
          b[i] = both ? vb[j].at(i) : 0.0f;
        }
      }
      if (n.rotates) {
        const float *c = cosines + n.token * p.half + n.u * P, *s = sines + n.token * p.half + n.u * P;
        if (P == 1 || !p.interleaved) {
#pragma unroll
          for (int i = 0; i < P; ++i) {
            const float u = a[i], v = b[i];
            a[i] = fmaf(u, c[i], -v * s[i]);
            b[i] = fmaf(v, c[i], u * s[i]);
          }
        } else if constexpr (P > 1) {
#pragma unroll
          for (int i = 0; i < P; i += 2) {
            const float u = a[i], v = a[i + 1], y = b[i], z = b[i + 1];
            const float ca = c[i / 2], sa = s[i / 2], cb = c[P / 2 + i / 2], sb = s[P / 2 + i / 2];
            a[i] = fmaf(u, ca, -v * sa);
            a[i + 1] = fmaf(v, ca, u * sa);
            b[i] = fmaf(y, cb, -z * sb);
            b[i + 1] = fmaf(z, cb, y * sb);
          }
        }
      }
      if (CACHE && n.which != 0) {
        const int kv = n.which - 1;
        Dst *to = static_cast<Dst *>(p.dst[kv]) + block_of[n.token] * p.dst_block[kv] + off_of[n.token] * p.dst_token[kv] +
                  n.head * p.dst_head[kv];
        if constexpr (sizeof(Dst) == 1) {
          float scale = 1.0f, inv = 1.0f;
          if (p.scale[kv]) {
            scale = p.scale[kv][n.head];
            inv = quotient_inverse(scale);
          }
          store_e4m3<P>(reinterpret_cast<uint8_t *>(to) + n.a, a, scale, inv);
          if (both) store_e4m3<P>(reinterpret_cast<uint8_t *>(to) + n.b, b, scale, inv);
        } else {
          if (n.rotates) {
            va[j].set(a);
            vb[j].set(b);
          }
          va[j].store(reinterpret_cast<Src *>(to) + n.a);
          if (both) vb[j].store(reinterpret_cast<Src *>(to) + n.b);
        }
      } else {
        Src *to = static_cast<Src *>(p.out) + row_of[n.token] * p.out_token + n.head * p.out_head;
        if (n.rotates) {
          va[j].set(a);
          vb[j].set(b);
        }
        va[j].store(to + n.a);
        if (both) vb[j].store(to + n.b);
      }
    }
  }
  if (bits) atomicOr(p.status, bits);
}

}  // namespace ts
