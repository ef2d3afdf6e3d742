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

// A token's units of one kind: of the queries (which 0), keys (1) or values (2).
struct RotaryRun {
  int32_t first;             // a multiple of 32
  int32_t units;
  FastDiv by_head;           // units per head
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
  int32_t units;                   // of a token: the end of the last run
  int32_t group;                   // threads that share a token: a multiple of 32
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

// P quotients by a scale, rounded to e4m3 as ts_kv_append rounds them: a quotient of 2^20
// and more (or infinite, or NaN) is 448 (or NaN) without its correction too; a scale
// that has no inverse here takes divisions.
template <int P>
__device__ __forceinline__ void store_e4m3(uint8_t *p, const float (&v)[P], float scale, float inv) {
  float y[P];
  if (inv == 0.0f) {
#pragma unroll
    for (int i = 0; i < P; ++i) y[i] = __fdiv_rn(v[i], scale);
  } else if constexpr (P == 1) {
    if (!quotient(v[0], scale, inv, y[0])) y[0] = v[0] * inv;
  } else {  // two at once
#pragma unroll
    for (int i = 0; i < P; i += 2) {
      const uint64_t x = pair_of(v[i], v[i + 1]), r = both_of(inv), q = mul2(x, r);
      float q0, q1, y0, y1;
      parts_of(q, q0, q1);
      parts_of(fma2(fma2(q, both_of(-scale), x), r, q), y0, y1);
      y[i] = fabsf(q0) < 0x1p20f ? copysignf(y0, q0) : q0;
      y[i + 1] = fabsf(q1) < 0x1p20f ? copysignf(y1, q1) : q1;
    }
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
// frame): freq = m 2^e, and 2 / pi to 128 bits, so that below 2^64 radians what is cut off
// is no more than 1.4 units.
__device__ __forceinline__ uint64_t turns_of(double freq) {
  const uint64_t bits = static_cast<uint64_t>(__double_as_longlong(freq));
  const int exponent = static_cast<int>((bits >> 52) & 0x7FF);
  const uint64_t m = (bits & 0xFFFFFFFFFFFFFull) | (exponent ? 1ull << 52 : 0);
  const uint64_t first = 0xA2F9836E4E441529ull, next = 0xFC2757D1F534DDC0ull;
  // the product's 64-bit words, the lowest first
  const uint64_t w0 = m * next, low = m * first, w1 = low + __umul64hi(m, next);
  const uint64_t w2 = __umul64hi(m, first) + (w1 < low);
  const int right = 1075 + 66 - max(exponent, 1);  // the product 2^-right
  const uint64_t at = right < 64 ? w0 : right < 128 ? w1 : w2, above = right < 64 ? w1 : right < 128 ? w2 : 0;
  const int by = right & 63;
  uint64_t turns;
  if (right >= 192) turns = 0;
  else if (right >= 0) turns = (at >> by) | (by ? above << (64 - by) : 0);
  else turns = right > -64 ? w0 << -right : 0;
  return bits >> 63 ? 0 - turns : turns;
}

// The cosine and sine of a position's angle, times the amplitude: within 2^-23 of 1 before
// that (the nearest 2^-32 of a turn; what is left of it beside whole quarters, 1 / 8 at most,
// in 24 bits; one step of the functions).
__device__ __forceinline__ void angle_of(uint64_t freq, int32_t pos, float amplitude, float &cosine, float &sine) {
  const uint64_t turn = freq * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const uint32_t top = static_cast<uint32_t>((turn + 0x80000000ull) >> 32);
  const uint32_t quarters = (top + 0x20000000u) >> 30;
  float s, c;
  sincospif(static_cast<float>(static_cast<int32_t>(top - (quarters << 30))) * 0x1p-31f, &s, &c);
  // a quarter turn: (c, s) -> (-s, c), two: both with the other sign
  const float x = quarters & 1 ? -s : c, y = quarters & 1 ? c : s, signed_amplitude = quarters & 2 ? -amplitude : amplitude;
  cosine = signed_amplitude * x;
  sine = signed_amplitude * y;
}

// One, two or four values side by side.
__device__ __forceinline__ void read_side(const float *p, float (&v)[1]) { v[0] = p[0]; }
__device__ __forceinline__ void read_side(const float *p, float (&v)[2]) {
  const float2 f = *reinterpret_cast<const float2 *>(p);
  v[0] = f.x, v[1] = f.y;
}
__device__ __forceinline__ void read_side(const float *p, float (&v)[4]) {
  const float4 f = *reinterpret_cast<const float4 *>(p);
  v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
}

// A CTA takes whole tokens.  Each angle's cosine and sine are computed once for all of a
// token's heads and go through shared memory; a unit is P elements and the P that they
// are paired with, or 2 P that are only copied.  A token's units lie in runs of one kind
// (queries' and keys' pairs, their copied elements, values), each from a multiple of 32
// on, so that a warp's 32 units go the same way, and a thread keeps its unit from token to
// token, so that it is found once (found for every token it took 294 instructions a unit,
// 192 us for 32,768 tokens; with lanes of several kinds 370 and 252).
// The next two tokens' pieces are on their way meanwhile (three CTAs to an SM).  Bound by
// DRAM and latency for prompts: 32,768 tokens of 32 + 8 + 8 heads into an e4m3 cache take
// 136 us, 5.4 TB/s; by latency for a frame (128 tokens of 16 + 8 + 8 heads: 2.8 us).
// CACHE: Dst is the cache's type.
template <class Src, class Dst, int P, bool CACHE>
__global__ void __launch_bounds__(kRotaryThreads, P == 1 ? 4 : 3) rotary_kernel(const RotaryParams p) {
  constexpr int kAhead = 2;
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
      // a unit's eight pairs in two places, so that lanes read 16 bytes side by side
      const int place = P == 8 && !p.interleaved ? ((i >> 2) & 1) * (p.half / 2) + (i >> 3) * 4 + (i & 3) : i;
      for (int k = g; k < nt; k += groups)
        angle_of(f, p.positions[t0 + k], p.amplitude, cosines[k * p.half + place], sines[k * p.half + place]);
    }
  }
  __syncthreads();

  // groups of threads take tokens in turn where a token's units are few
  const int width = p.group, group = t / width, groups = kRotaryThreads / width;
  if (group < groups) {
    for (int x = t - group * width; x < p.units; x += width) {
      int r = 0;
#pragma unroll
      for (int k = 1; k < kRotaryRuns; ++k) r += (x & ~31) >= p.run[k].first;  // the same for a warp
      const int rotates = p.run[r].rotates, which = p.run[r].which;
      const uint32_t in = static_cast<uint32_t>(x - p.run[r].first);
      const int head = static_cast<int>(p.run[r].by_head.div(in));
      const int u = static_cast<int>(in) - head * static_cast<int>(p.run[r].by_head.d);
      if (static_cast<int>(in) >= p.run[r].units) continue;
      // a piece and the one half of the run's width behind it: the halves' pairs; neighbours'
      // pairs and copied elements lie in a piece of their own, and lanes side by side
      const bool single = P == 1 && rotates && p.interleaved;  // but for single elements
      const int apart = single ? 1 : static_cast<int>(p.run[r].by_head.d) * P;
      const int a_at = p.run[r].from + (single ? 2 : P) * u, b_at = a_at + apart;
      const bool both = b_at < p.dim;
      const bool queries = !CACHE || which == 0;
      const int kv = queries ? 0 : which - 1;
      const Src *src = queries ? static_cast<const Src *>(p.x) + head * p.x_head
                               : static_cast<const Src *>(p.src[kv]) + head * p.src_head[kv];
      const int64_t src_token = queries ? p.x_token : p.src_token[kv];
      Src *out = static_cast<Src *>(p.out) + head * p.out_head;
      Dst *cache = queries ? nullptr : static_cast<Dst *>(p.dst[kv]) + head * p.dst_head[kv];
      float scale = 1.0f, inv = 1.0f;
      if (CACHE && sizeof(Dst) == 1 && !queries && p.scale[kv]) {
        scale = p.scale[kv][head];
        inv = quotient_inverse(scale);
      }
      // the next kAhead tokens' pieces are on their way
      Piece<Src, P> va[kAhead], vb[kAhead];
      int64_t row[kAhead];
      const auto fetch = [&](int j, int k) {
        row[j] = k < nt ? row_of[k] : -1;
        if (row[j] < 0) return;
        const Src *from = src + row[j] * src_token;
        va[j].load(from + a_at);
        if (both) vb[j].load(from + b_at);
      };
#pragma unroll
      for (int j = 0; j < kAhead; ++j) fetch(j, group + j * groups);
      for (int k0 = group; k0 < nt; k0 += groups * kAhead) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const int k = k0 + j * groups;
          const int64_t here = row[j];
          Piece<Src, P> pa = va[j], pb = vb[j];
          fetch(j, k + kAhead * groups);
          if (here < 0) continue;
          float a[P], b[P];
          if (rotates || (CACHE && !queries && sizeof(Dst) == 1)) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
              a[i] = pa.at(i);
              b[i] = both ? pb.at(i) : 0.0f;
            }
          }
          if (rotates) {
            const float *c = cosines + k * p.half, *s = sines + k * p.half;
            if (P == 1 || !p.interleaved) {
              constexpr int kSide = P == 1 ? 1 : 4;  // read at once
#pragma unroll
              for (int h = 0; h < P / kSide; ++h) {
                float cs[kSide], sn[kSide];
                read_side(c + h * (p.half / 2) + u * kSide, cs);
                read_side(s + h * (p.half / 2) + u * kSide, sn);
#pragma unroll
                for (int i = 0; i < kSide; ++i) {
                  const float v = a[kSide * h + i], w = b[kSide * h + i];
                  a[kSide * h + i] = fmaf(v, cs[i], -w * sn[i]);
                  b[kSide * h + i] = fmaf(w, cs[i], v * sn[i]);
                }
              }
            } else if constexpr (P > 1) {
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float cs[P / 2], sn[P / 2];
                read_side(c + h * (p.half / 2) + u * (P / 2), cs);
                read_side(s + h * (p.half / 2) + u * (P / 2), sn);
#pragma unroll
                for (int i = 0; i < P / 2; ++i) {
                  float &v = h ? b[2 * i] : a[2 * i], &w = h ? b[2 * i + 1] : a[2 * i + 1];
                  const float v0 = v;
                  v = fmaf(v0, cs[i], -w * sn[i]);
                  w = fmaf(w, cs[i], v0 * sn[i]);
                }
              }
            }
          }
          if (CACHE && sizeof(Dst) == 1 && !queries) {
            uint8_t *to = reinterpret_cast<uint8_t *>(cache + slot_of[CACHE ? kv : 0][k]);
            store_e4m3<P>(to + a_at, a, scale, inv);
            if (both) store_e4m3<P>(to + b_at, b, scale, inv);
          } else {
            if (rotates) {
              pa.set(a);
              pb.set(b);
            }
            Src *to = out + here * p.out_token;
            if (!queries) to = reinterpret_cast<Src *>(cache + slot_of[CACHE ? kv : 0][k]);
            pa.store(to + a_at);
            if (both) pb.store(to + b_at);
          }
        }
      }
    }
  }
  if (bits) atomicOr(p.status, bits);
}

}  // namespace ts
