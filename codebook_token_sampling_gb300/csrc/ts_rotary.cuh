// ts_rotary.cuh -- rotary positions (ts_rotary), and the same on the way into the
// paged cache (ts_kv_append_rotary).
#pragma once

#include "ts_kv_common.cuh"
#include "ts_rows.cuh"

namespace ts {

constexpr int kRotaryThreads = 256;
constexpr int kRotaryTokens = 64;         // of a CTA at most
constexpr int kRotaryTableFloats = 8192;  // cosines and sines of a CTA's tokens, at most
constexpr int kRotaryRuns = 5;

// Units of one kind of a CTA's tokens: of the queries (which 0), keys (1) or values (2).
struct RotaryRun {
  uint32_t first;            // a multiple of 32
  FastDiv by_token, by_head;  // units per token and per head
  int32_t which, rotates;
  int32_t from;              // first element that is copied
};

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
  uint32_t units;                  // of a CTA: the end of the last run
  RotaryRun run[kRotaryRuns];
  uint32_t *status;
  // the cache's part
  const void *src[2];              // keys and values of the new tokens
  int64_t src_token[2], src_head[2];
  void *dst[2];
  int64_t dst_block[2], dst_token[2], dst_head[2];
  const float *scale[2];           // or null
  const int64_t *slots;
  int64_t n_slots;
  FastDiv by_block;
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
// By whole numbers (64-bit floating point arithmetic would take longer than the rest of a
// frame): freq = m 2^e, and 2^66 / (2 pi) to 64 bits.
__device__ __forceinline__ uint64_t turns_of(double freq) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(freq));
  const int exponent = static_cast<int>((bits >> 52) & 0x7FF);
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (exponent ? 1ull << 52 : 0);
  const uint64_t per_radian = 0xA2F9836E4E441529ull;
  const uint64_t high = __umul64hi(m, per_radian), low = m * per_radian;
  const int right = 1075 + 2 - max(exponent, 1);  // (high, low) 2^-right
  uint64_t turns;
  if (right >= 128) turns = 0;
  else if (right > 64) turns = high >> (right - 64);
  else if (right == 64) turns = high;
  else if (right > 0) turns = (low >> right) | (high << (64 - right));
  else turns = right > -64 ? low << -right : 0;
  return bits >> 63 ? 0 - turns : turns;
}

// The cosine and sine of a position's angle, times the amplitude.
__device__ __forceinline__ void angle_of(uint64_t freq, int32_t pos, float amplitude, float &cosine, float &sine) {
  const uint64_t turn = freq * static_cast<uint64_t>(static_cast<int64_t>(pos));
  // the nearest 2^-32 of a turn, as half turns from -1 to 1
  const int32_t top = static_cast<int32_t>((turn + 0x80000000ull) >> 32);
  float s, c;
  sincospif(static_cast<float>(top) * 0x1p-31f, &s, &c);
  cosine = amplitude * c;
  sine = amplitude * s;
}

// A CTA takes whole tokens.  Each angle's cosine and sine are computed once for all of a
// token's heads and go through shared memory; a unit is P elements and the P that they
// are paired with, or 2 P that are only copied.  The CTA's units lie in runs of one kind
// (queries' and keys' pairs, their copied elements, values), each from a multiple of 32
// on, so that a warp's 32 units go the same way (dealt as they lie in a token, half of
// the lanes waited for the others: 370 instructions a unit, 252 us for 32,768 tokens).
// Bound by DRAM for prompts, by latency for a frame.  CACHE: Dst is the cache's type.
template <class Src, class Dst, int P, bool CACHE>
__global__ void __launch_bounds__(kRotaryThreads, P == 8 ? 3 : 4) rotary_kernel(const RotaryParams p) {
  constexpr int kUnroll = 2;
  extern __shared__ __align__(16) float rotary_smem[];
  __shared__ int64_t row_of[kRotaryTokens];
  __shared__ int64_t slot_of[CACHE ? 2 : 1][kRotaryTokens];  // where keys and values go
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
      skip = row < 0 || row >= p.n_rows;
      if (skip) bits |= kRowBadSlot;
    }
    if constexpr (CACHE) {
      if (!skip && slot >= p.n_slots) {
        skip = true;
        bits |= kRowBadSlot;
      }
      // a cache of 2^31 slots and more takes the 64-bit division
      const int64_t blk = skip ? 0 : p.n_slots <= 0x7FFFFFFF ? static_cast<int64_t>(p.by_block.div(static_cast<uint32_t>(slot)))
                                                             : slot / p.by_block.d;
      const int64_t off = skip ? 0 : slot - blk * p.by_block.d;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv) slot_of[kv][t] = blk * p.dst_block[kv] + off * p.dst_token[kv];
    }
    row_of[t] = skip ? -1 : row;
  }
  for (int i0 = 0; i0 < p.half; i0 += kRotaryThreads) {
    const int width = min(kRotaryThreads, p.half - i0), groups = kRotaryThreads / width;
    const int g = t / width, i = i0 + t - g * width;
    if (g < groups) {
      const uint64_t f = turns_of(p.freqs[i]);
      for (int k = g; k < nt; k += groups)
        angle_of(f, p.positions[t0 + k], p.amplitude, cosines[k * p.half + i], sines[k * p.half + i]);
    }
  }
  __syncthreads();

  struct Unit {
    int64_t to;                // element of the output or the cache
    int token, head, u, a, b;  // token < 0: nothing to do
  };
  const auto run_of = [&](uint32_t x) {  // the same for a warp
    int r = 0;
#pragma unroll
    for (int k = 1; k < kRotaryRuns; ++k) r += x >= p.run[k].first;
    return r;
  };
  const auto unit_of = [&](uint32_t x, const RotaryRun &run, const void *&from) {
    Unit n;
    x -= run.first;
    n.token = static_cast<int>(run.by_token.div(x));
    if (n.token >= nt) {
      n.token = -1;
      return n;
    }
    const uint32_t in = x - static_cast<uint32_t>(n.token) * run.by_token.d;
    n.head = static_cast<int>(run.by_head.div(in));
    n.u = static_cast<int>(in - static_cast<uint32_t>(n.head) * run.by_head.d);
    if (run.rotates && !p.interleaved) {
      n.a = n.u * P;
      n.b = p.half + n.a;
    } else {  // neighbours, rotated or copied
      n.a = run.from + n.u * 2 * P;
      n.b = n.a + P;
    }
    const int64_t row = row_of[n.token];
    if (row < 0) {
      n.token = -1;
      return n;
    }
    if (!CACHE || run.which == 0) {
      from = static_cast<const Src *>(p.x) + row * p.x_token + n.head * p.x_head;
      n.to = row * p.out_token + n.head * p.out_head;
    } else {
      const int kv = run.which - 1;
      from = static_cast<const Src *>(p.src[kv]) + row * p.src_token[kv] + n.head * p.src_head[kv];
      n.to = slot_of[CACHE ? kv : 0][n.token] + n.head * p.dst_head[kv];
    }
    return n;
  };

  const uint32_t units = p.units;
  for (uint32_t x0 = t; x0 < units; x0 += kRotaryThreads * kUnroll) {
    Piece<Src, P> va[kUnroll], vb[kUnroll];
    Unit n[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t x = x0 + j * kRotaryThreads;
      n[j].token = -1;
      if (x >= units) continue;
      const void *from = nullptr;
      n[j] = unit_of(x, p.run[run_of(x & ~31u)], from);
      if (n[j].token < 0) continue;
      va[j].load(static_cast<const Src *>(from) + n[j].a);
      if (n[j].b < p.dim) vb[j].load(static_cast<const Src *>(from) + n[j].b);
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t x = x0 + j * kRotaryThreads;
      if (x >= units) continue;
      const RotaryRun &run = p.run[run_of(x & ~31u)];
      if (n[j].token < 0) continue;
      const bool both = n[j].b < p.dim;
      float a[P], b[P];
      if (run.rotates || (CACHE && run.which != 0 && sizeof(Dst) == 1)) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          a[i] = va[j].at(i);
          b[i] = both ? vb[j].at(i) : 0.0f;
        }
      }
      if (run.rotates) {
        const float *c = cosines + n[j].token * p.half + n[j].u * P, *s = sines + n[j].token * p.half + n[j].u * P;
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
      if (CACHE && run.which != 0) {
        const int kv = run.which - 1;
        Dst *to = static_cast<Dst *>(p.dst[kv]) + n[j].to;
        if constexpr (sizeof(Dst) == 1) {
          float scale = 1.0f, inv = 1.0f;
          if (p.scale[kv]) {
            scale = p.scale[kv][n[j].head];
            inv = quotient_inverse(scale);
          }
          store_e4m3<P>(reinterpret_cast<uint8_t *>(to) + n[j].a, a, scale, inv);
          if (both) store_e4m3<P>(reinterpret_cast<uint8_t *>(to) + n[j].b, b, scale, inv);
        } else {
          if (run.rotates) {
            va[j].set(a);
            vb[j].set(b);
          }
          va[j].store(reinterpret_cast<Src *>(to) + n[j].a);
          if (both) vb[j].store(reinterpret_cast<Src *>(to) + n[j].b);
        }
      } else {
        Src *to = static_cast<Src *>(p.out) + n[j].to;
        if (run.rotates) {
          va[j].set(a);
          vb[j].set(b);
        }
        va[j].store(to + n[j].a);
        if (both) vb[j].store(to + n[j].b);
      }
    }
  }
  if (bits) atomicOr(p.status, bits);
}

}  // namespace ts
