// ts_paged.cuh -- attention of one new token per request over a paged
// key-value cache.  For query head h of request r, with key head h / G and the
// attended tokens t (t < len_r, inside the window, not masked):
//   s_t = scale * q . k_t,  optionally  cap * tanh(s_t / cap)
//   o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m),  m = max_t s_t,
//   lse = m + ln sum_t e^(s_t - m).
// Every key and value row is read once and serves the G query heads that
// share it: 2 G flops per element (54 TFLOP/s for G = 8 and 2 bytes at the rate
// of DRAM), so the bound is DRAM: 128 requests of up to 8000 tokens, 8 x 4 heads
// of 128 in bf16, 2.1 GB, take 308 us, 7.0 TB/s.  More than 16 query heads (fp32:
// 8) read it once per 16 (8).
//
// Work.  An item is one (request, key head, piece of at most kRows query
// heads); its tokens are cut into tiles of 16 to 128 (a step of every warp), and
// the tiles of all items, laid end to end, are dealt to the CTAs in runs of equal
// cost.  Every CTA finds its run by summing the lengths itself, so ragged batches
// balance with nothing planned on the host and no launch before this one.  (The
// lengths stay as they are while the call runs; should they change, its loops
// still end inside the arrays.)  A run holds whole items
// and at most two parts of items that other runs share: those go to a
// workspace, and the CTA that brings an item's last part joins them; where
// items have many parts, paged_join_kernel does.  The parts' order in the sums
// is always the same.
//
// A CTA is four warps (six or two where rows are wide); each takes its share of
// a tile's tokens with a running maximum and sum of its own and a private ring
// of cp.async stages (a share's K and V each), so no warp waits for another
// inside an item.  The ring runs on across items.  At an item's end the warps'
// results are joined in shared memory.
#pragma once

#include <type_traits>

#include "ts_kv_common.cuh"
#include "ts_lmhead.cuh"

namespace ts {

constexpr int kPagedPage = 16;                       // a stage's tokens divide this
constexpr int kPagedRows = 16;                       // most query heads per item
constexpr int kPagedMaxDim = 256;

// The workspace: two places per CTA for parts of items (place 0 for an item
// that began in an earlier CTA, place 1 for one that it begins and does not
// end), each of kPagedRows rows of kPagedMaxDim sums, the rows' maxima and sums
// and what it is a part of; and two counters per CTA, of the calls so far and of
// the parts that have come of the item that it begins.
//
// The parts' counters need no known state at a call's start: they count from the
// call's number times 2^kCallShift, to which the first part to come lifts them, so
// what a call leaves behind that lost parts (its lengths changed while it ran, or
// two calls ran at once) is below all that the next one counts.  Every call that
// counts adds one to every entry of `calls`, CTA b to entries b, b + ctas, ..; with
// all calls done the entries are equal, whatever ran at once and however many CTAs
// each had.  (It costs up to 2%: 22.4 to 22.5 us for 32 streams, 25.7 to 26.0 for a
// window over rows of 256.)
struct PagedParts {
  int32_t first, parts;  // the CTA of the item's first part; their number, 0: nothing here
  int32_t request, head, piece;
};
constexpr size_t kPagedAccBytes = sizeof(float) * kPagedRows * kPagedMaxDim;
constexpr size_t paged_workspace_bytes(int ctas) {
  return static_cast<size_t>(ctas) *
         (2 * (kPagedAccBytes + sizeof(float2) * kPagedRows + sizeof(PagedParts) + sizeof(uint64_t)));
}
constexpr int kCallShift = 16;  // more than the parts of an item

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
  int32_t room;             // tokens of a table row
  const int32_t *lens;
  int32_t n_requests;
  const void *k, *v;
  int64_t k_head, v_head;   // bytes
  int32_t k_block, k_token, v_block, v_token;  // bytes, below 2^31: products of 32 bits
  const float *k_scale, *v_scale;
  int32_t n_blocks, block_size, kv_heads, dim;
  int32_t group;            // query heads per key head
  int32_t pieces;           // items per (request, key head)
  int32_t rows;             // query heads of a full item
  float scale, softcap;
  int32_t window;           // 0: none
  FastDiv by_block;
  PagedParts *parts;        // [2 ctas]
  unsigned long long *arrived;  // [all_ctas]
  unsigned long long *calls;    // [all_ctas], null where no item is joined here
  float *acc;               // [2 ctas][kPagedRows][kPagedMaxDim]
  float2 *ml;               // [2 ctas][kPagedRows]
  int32_t ctas;             // of the main launch
  int32_t all_ctas;         // that the workspace is for
  int32_t join_here;        // 1: the last CTA to come joins, 0: paged_join_kernel does
  FastDiv by_ctas;
  int32_t tiles_fit;        // all tiles, and what a search adds to them, stay below 2^31
  int32_t out_f32;
  uint32_t *status;
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ int64_t wide_product(int32_t a, int32_t b) {
  return static_cast<int64_t>(a) * b;
}

// 2^x to 2^-22 of itself; below 2^-126 zero
__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 2^(m - top), 0 for an empty part
__device__ __forceinline__ float exp2_from(float m, float top) {
  return m == -INFINITY ? 0.0f : exp2_of(m - top);
}

__device__ __forceinline__ void cp_async16_or_zero(uint32_t smem, const void *gmem, bool real,
                                                   uint64_t policy) {
  const int n = real ? 16 : 0;
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(smem),
               "l"(gmem), "r"(n), "l"(policy)
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
// an 8 x 8 piece of 16-bit values, transposed
__device__ __forceinline__ uint32_t transposed_8x8(uint32_t x) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(x));
  return d;
}
// four e4m3 values as f16 values (exact): the lower two and the upper two
__device__ __forceinline__ void f16_of_e4m3x4(uint32_t x, uint32_t &lower, uint32_t &upper) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lower), "=r"(upper) : "r"(x));
}
// two fp32 values side by side
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t pair_of(float x) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %1};" : "=l"(d) : "f"(x));
  return d;
}
__device__ __forceinline__ float low_of(uint64_t x) {
  return __uint_as_float(static_cast<uint32_t>(x));
}
__device__ __forceinline__ float high_of(uint64_t x) {
  return __uint_as_float(static_cast<uint32_t>(x >> 32));
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

// A stage row's 16-byte chunk c sits at chunk c ^ stage_xor(row), so that the
// eight rows of a matrix load (or the lanes of a vector load) fall on different
// banks.  stage_xor(a + b) = stage_xor(a) ^ stage_xor(b) where a and b share no
// bits.  LANES: lanes that read one row side by side (0: matrix loads).
template <int ROW_BYTES, int LANES>
__host__ __device__ __forceinline__ constexpr int stage_xor(int row) {
  if constexpr (LANES > 0) return LANES * (row & (8 / LANES - 1));
  else if constexpr (ROW_BYTES % 128 == 0) return row & 7;
  else if constexpr (ROW_BYTES % 64 == 0) return (row >> 1) & 3;  // two rows share a 128-byte line's phase
  else return (row >> 2) & 1;                                     // rows of 96 bytes
}
template <int ROW_BYTES, int LANES>
__device__ __forceinline__ uint32_t stage_at(int row, int chunk) {
  return static_cast<uint32_t>(row * ROW_BYTES + ((chunk ^ stage_xor<ROW_BYTES, LANES>(row)) << 4));
}

// --------------------------------------------------------------------------
// One warp's arithmetic on the tensor cores (bf16 and e4m3 caches).  Tokens
// are the products' rows and query heads their columns, eight at a time (NT
// groups of eight): S^T = K Q^T, then O^T = V^T P^T, so that up to eight query
// heads per key head cost one product each and few registers.  A step takes 16
// KT tokens.  Columns past the item's heads are zero.
// --------------------------------------------------------------------------
template <bool E4M3, int DP, int NT, int KT>
struct MmaCore {
  static constexpr int kRows = 8 * NT;
  static constexpr int kTok = 16 * KT;
  static constexpr int kPer = 0;
  static constexpr bool kFma = false;
  static constexpr float kLift = E4M3 ? 15.0f : 0.0f;  // weights count from 2^kLift (see step)
  static constexpr int kElemBytes = E4M3 ? 1 : 2;
  static constexpr int kRowBytes = DP * kElemBytes;
  static constexpr int kDim = DP;
  // stages of 16 KB: six warps with two stages each (56 us), not four with
  // three (59 us: 48 requests of up to 6000 tokens, 2 x 8 bf16 heads of 256)
  static constexpr int kWarps = kTok * kRowBytes > 6144 ? 6 : 4;
  static constexpr int kSteps = DP / 16;
  // wide rows leave no registers for the queries: one copy in shared memory
  static constexpr bool kSharedQ = DP > 128;
  static constexpr uint32_t kQBytes = kSharedQ ? NT * kSteps * 32 * 8 : 0;
  static constexpr uint32_t kWarpBytes = 0;  // shared memory of a warp's own

  // lane = 4 g + tg
  uint32_t qf[NT][kSharedQ ? 1 : kSteps][2];  // head 8 n + g
  uint32_t q_at;                   // of this lane's share of the shared copy
  float o[NT][kSteps][4];          // heads 8 n + 2 tg + (0, 1)
  // of those heads; l: this lane's tokens only; o and l hold 2^kLift times theirs
  float m[NT][2], l[NT][2], sc[NT][2];

  // The queries' words of group n, step kk.
  __device__ __forceinline__ void query(int n, int kk, uint32_t (&x)[2]) const {
    if constexpr (kSharedQ)
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                   : "=r"(x[0]), "=r"(x[1]) : "r"(q_at + (n * kSteps + kk) * 256) : "memory");
    else
      x[0] = qf[n][kk][0], x[1] = qf[n][kk][1];
  }

  __device__ __forceinline__ void begin(const PagedParams &p, const uint16_t *q, int rows,
                                        float k_scale, void *shared) {
    const int lane = static_cast<int>(lane_id()), g = lane >> 2, tg = lane & 3;
    const int warp = static_cast<int>(threadIdx.x) >> 5;
    const float unit = p.softcap > 0.0f ? p.scale * k_scale : p.scale * k_scale * kLog2e;
    if constexpr (kSharedQ)
      q_at = static_cast<uint32_t>(__cvta_generic_to_shared(shared)) + lane * 8;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const uint16_t *row = q + (8 * n + g) * p.q_head;
      const bool real = 8 * n + g < rows;
      const auto keep = [&](int kk, uint32_t x, uint32_t y) {
        if constexpr (kSharedQ) {
          if (kk % kWarps == warp)
            *reinterpret_cast<uint2 *>(static_cast<char *>(shared) + (n * kSteps + kk) * 256 + lane * 8) =
                make_uint2(x, y);
        } else {
          qf[n][kk][0] = x;
          qf[n][kk][1] = y;
        }
      };
      if constexpr (!E4M3) {
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          const int c = kk * 16 + 2 * tg;
          keep(kk, real && c < p.dim ? *reinterpret_cast<const uint32_t *>(row + c) : 0u,
               real && c + 8 < p.dim ? *reinterpret_cast<const uint32_t *>(row + c + 8) : 0u);
        }
        sc[n][0] = sc[n][1] = unit;
      } else {
        // The cache's values are exact in f16, a bf16 query is not in f16's
        // range: each row is divided by a power of two that brings its largest
        // element into [1, 2).  What f16 then drops is below 2^-25 of that.
        // Elements 4 tg .. 4 tg + 3 of a 16-element step stand in the places
        // 2 tg, 2 tg + 1, 2 tg + 8, 2 tg + 9, as the keys' bytes do.
        const auto raw_at = [&](int kk) {
          const int c = kk * 16 + 4 * tg;
          return real && c < p.dim ? *reinterpret_cast<const uint2 *>(row + c) : make_uint2(0u, 0u);
        };
        const auto low = [](uint32_t w) { return __uint_as_float(w << 16); };
        const auto high = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
        float big = 0.0f;
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          const uint2 raw = raw_at(kk);
          if constexpr (!kSharedQ) keep(kk, raw.x, raw.y);
          big = fmaxf(big, fmaxf(fmaxf(fabsf(low(raw.x)), fabsf(high(raw.x))),
                                 fmaxf(fabsf(low(raw.y)), fabsf(high(raw.y)))));
        }
        big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 1));
        big = fmaxf(big, __shfl_xor_sync(0xFFFFFFFFu, big, 2));
        const int e = big > 0.0f && big < INFINITY ? ilogbf(big) : 0;
        // 2^-e in two factors: e goes down to that of the smallest bf16 number
        const float f0 = scalbnf(1.0f, -(e / 2)), f1 = scalbnf(1.0f, -(e - e / 2));
#pragma unroll
        for (int kk = 0; kk < kSteps; ++kk) {
          uint2 raw;
          if constexpr (kSharedQ) raw = raw_at(kk);
          else raw = make_uint2(qf[n][kk][0], qf[n][kk][1]);
          keep(kk, f16x2_of(low(raw.x) * f0 * f1, high(raw.x) * f0 * f1),
               f16x2_of(low(raw.y) * f0 * f1, high(raw.y) * f0 * f1));
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
          sc[n][h] = scalbnf(unit, __shfl_sync(0xFFFFFFFFu, e, 4 * (2 * tg + h)));
      }
#pragma unroll
      for (int d = 0; d < kSteps; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][d][e] = 0.0f;
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.0f;
    }
    if constexpr (kSharedQ) __syncthreads();
  }

  __device__ __forceinline__ void poison() {
#pragma unroll
    for (int n = 0; n < NT; ++n) l[n][0] = l[n][1] = __int_as_float(0x7FC00000);
  }

  static __device__ __forceinline__ float weight(float s, float base) {
    if constexpr (kLift != 0.0f) return exp2_of(s - base + kLift);
    else return exp2_of(s - base);
  }

  // kTok tokens: K rows at shared address ks, V rows at vs, bit t of `valid` set
  // where token t is attended (the others' rows are zero)
  __device__ __forceinline__ void step(const PagedParams &p, uint32_t ks, uint32_t vs,
                                       uint32_t valid, void *) {
    const int lane = static_cast<int>(lane_id()), g = lane >> 2;
    // rows 0-7 | 8-15 by lane bit 3, chunk by bit 4
    const int row = (lane & 7) + (((lane >> 3) & 1) << 3), half = lane >> 4;
    float s[KT][NT][4];
    // one chain of products would be as long as the row: two halves of it side
    // by side where there is nothing else to interleave
    constexpr int kChains = KT * NT == 1 ? 2 : 1;
    float s2[NT][4];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][n][e] = s2[n][e] = 0.0f;
    if constexpr (!E4M3) {
#pragma unroll
      for (int kk = 0; kk < kSteps; ++kk) {
        uint32_t x[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) query(n, kk, x[n]);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          uint32_t a[4];
          ldmatrix_x4_at(a, ks + stage_at<kRowBytes, 0>(16 * t + row, 2 * kk + half));
#pragma unroll
          for (int n = 0; n < NT; ++n)
            mma_bf16_16816(kChains == 2 && (kk & 1) ? s2[n] : s[t][n], a, x[n][0], x[n][1]);
        }
      }
    } else {
#pragma unroll
      for (int k2 = 0; k2 < kSteps / 2; ++k2) {
        uint32_t x[2][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) query(n, 2 * k2, x[0][n]), query(n, 2 * k2 + 1, x[1][n]);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          uint32_t b[4];
          ldmatrix_x4_at(b, ks + stage_at<kRowBytes, 0>(16 * t + row, 2 * k2 + half));
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a[4];
            f16_of_e4m3x4(b[2 * h], a[0], a[2]);
            f16_of_e4m3x4(b[2 * h + 1], a[1], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
              mma_f16_16816(kChains == 2 && h ? s2[n] : s[t][n], a, x[h][n][0], x[h][n][1]);
          }
        }
      }
    }
    if constexpr (kChains == 2) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[0][0][e] += s2[0][e];
    }
    // scores in units of ln 2, unattended ones at -inf
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][n][e] *= sc[n][e & 1];
    if (p.softcap > 0.0f) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            s[t][n][e] = p.softcap * tanhf(s[t][n][e] / p.softcap) * kLog2e;
    }
    constexpr uint32_t kAll = kTok == 32 ? 0xFFFFFFFFu : (1u << (kTok & 31)) - 1;
    if (valid != kAll) {
#pragma unroll
      for (int t = 0; t < KT; ++t)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((valid >> (16 * t + g + 8 * (e >> 1))) & 1u)) s[t][n][e] = -INFINITY;
    }
    float base[NT][2], drop[NT][2];
    bool moved = false;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = fmaxf(s[0][n][h], s[0][n][2 + h]);
#pragma unroll
        for (int t = 1; t < KT; ++t) x = fmaxf(x, fmaxf(s[t][n][h], s[t][n][2 + h]));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xFFFFFFFFu, x, 16));
        const float top = fmaxf(m[n][h], x);
        base[n][h] = top == -INFINITY ? 0.0f : top;  // a head with nothing yet
        drop[n][h] = exp2_from(m[n][h], base[n][h]);
        moved |= top != m[n][h];
        m[n][h] = top;
      }
    if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int d = 0; d < kSteps; ++d)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][d][e] *= drop[n][e & 1];
        l[n][0] *= drop[n][0];
        l[n][1] *= drop[n][1];
      }
    }
    // The weights as the second products' right side, transposed in 8 x 8
    // pieces.  bf16 values carry V: a weight goes in as the sum of two bf16
    // numbers, its upper half and what is left, so that less than 2^-16 of it
    // is lost and the output's own rounding stays the largest error.  The
    // second number is kept above zero (by 2^-20 of the weight): an attended
    // infinity in V then comes out as one, not as the NaN of 0 times it (where its
    // weight is above 2^-113 of the largest; below, both can be zero).  An
    // f16 weight (e4m3 values, which have no infinities) keeps 11 bits.  f16's
    // range is short, and many small weights may make up the output beside a
    // large one whose value is zero: so the largest is 2^kLift, at the range's
    // upper end, and 2^-29 of it keeps 11 bits still, 2^-39 is not lost.  (Counted
    // from 1, all below 2^-25 were lost from the output, not from the sums.)
    uint32_t hi[KT][NT][2], lo[KT][NT][2];
#pragma unroll
    for (int t = 0; t < KT; ++t)
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float x = weight(s[t][n][2 * r], base[n][0]), y = weight(s[t][n][2 * r + 1], base[n][1]);
          l[n][0] += x;
          l[n][1] += y;
          if constexpr (E4M3) {
            hi[t][n][r] = transposed_8x8(f16x2_of(x, y));
          } else {
            const uint32_t ux = __float_as_uint(x), uy = __float_as_uint(y);
            hi[t][n][r] = transposed_8x8(__byte_perm(ux, uy, 0x7632));
            lo[t][n][r] = transposed_8x8(
                bf16x2_of(fmaf(x, 0x1p-20f, x - __uint_as_float(ux & 0xFFFF0000u)),
                          fmaf(y, 0x1p-20f, y - __uint_as_float(uy & 0xFFFF0000u))));
          }
        }
    if constexpr (!E4M3) {
      // rows 0-7 | 8-15 by lane bit 4, chunk by bit 3
      const int vrow = (lane & 7) + ((lane >> 4) << 3), vhalf = (lane >> 3) & 1;
#pragma unroll
      for (int d = 0; d < kSteps; ++d)
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          uint32_t a[4];
          ldmatrix_x4_trans_at(a, vs + stage_at<kRowBytes, 0>(16 * t + vrow, 2 * d + vhalf));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            mma_bf16_16816(o[n][d], a, hi[t][n][0], hi[t][n][1]);
            mma_bf16_16816(o[n][d], a, lo[t][n][0], lo[t][n][1]);
          }
        }
    } else {
      // A transposed load of 16-bit units hands a lane elements 2 g, 2 g + 1
      // of tokens 2 tg, 2 tg + 1: the even elements make a product's rows 0-7,
      // the odd ones its rows 8-15.
#pragma unroll
      for (int d2 = 0; d2 < kSteps / 2; ++d2)
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          uint32_t b[4];
          ldmatrix_x4_trans_at(b, vs + stage_at<kRowBytes, 0>(16 * t + row, 2 * d2 + half));
#pragma unroll
          for (int i = 0; i < 4; ++i) b[i] = __byte_perm(b[i], 0u, 0x3120);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t a[4];
            f16_of_e4m3x4(b[2 * h], a[0], a[1]);
            f16_of_e4m3x4(b[2 * h + 1], a[2], a[3]);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma_f16_16816(o[n][2 * d2 + h], a, hi[t][n][0], hi[t][n][1]);
          }
        }
    }
  }

  // Where column c of head h's sums lies in a warp's buffer: heads 2 tg of one
  // column on different banks, four columns from a multiple of four together.
  static __device__ __forceinline__ int at(int h, int c) { return h * DP + (c ^ (((h >> 1) & 3) << 3)); }

  // The warp's maxima, sums and weighted sums of V (the lift's power of two goes
  // off without a rounding).
  __device__ __forceinline__ void give(float *buf, float *sm, float *sl) {
    constexpr float kLower = E4M3 ? 0x1p-15f : 1.0f;  // 2^-kLift
    const int lane = static_cast<int>(lane_id()), g = lane >> 2, tg = lane & 3;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x = l[n][h];
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 4);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 8);
        x += __shfl_xor_sync(0xFFFFFFFFu, x, 16);
        const int head = 8 * n + 2 * tg + h;
        if (g == 0) {
          sm[head] = m[n][h];
          sl[head] = x * kLower;
        }
#pragma unroll
        for (int d = 0; d < kSteps; ++d) {
          if constexpr (E4M3) {
            *reinterpret_cast<float2 *>(buf + at(head, 16 * d + 2 * g)) =
                make_float2(o[n][d][h] * kLower, o[n][d][2 + h] * kLower);
          } else {
            buf[at(head, 16 * d + g)] = o[n][d][h];
            buf[at(head, 16 * d + 8 + g)] = o[n][d][2 + h];
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
  static constexpr int kTok = DP > 64 ? 8 : 16;
  static constexpr int kPer = 32 / kTok;
  static constexpr bool kFma = true;
  static constexpr int kElemBytes = 4;
  static constexpr int kRowBytes = DP * kElemBytes;
  static constexpr uint32_t kQBytes = GR * DP * 4;
  static constexpr uint32_t kWarpBytes = kTok * GR * 4;
  static constexpr int kLanes = DP / 4 < 32 ? DP / 4 : 32;  // lanes across a row
  static constexpr int kSplit = 32 / kLanes;                // tokens side by side
  static constexpr int kCols = (DP + 127) / 128;            // chunks per lane
  static constexpr int kQuads = DP / 4;
  static constexpr int kDim = DP;
  // stages of 16 KB: six warps per SM as three CTAs of two (62 us), not four as
  // one (73 us: 24 requests of up to 3001 tokens, 4 x 4 heads of 256)
  static constexpr int kWarps = DP > 128 ? 2 : 4;

  uint64_t o[GR][kCols * 2];  // pairs of columns
  float m[GR], l[GR];
  float sc;
  uint32_t q_at;

  __device__ __forceinline__ void begin(const PagedParams &p, const float *src, int rows,
                                        float k_scale, void *shared) {
    float *sq = static_cast<float *>(shared);
    q_at = static_cast<uint32_t>(__cvta_generic_to_shared(sq));
    sc = p.softcap > 0.0f ? p.scale * k_scale : p.scale * k_scale * kLog2e;
    for (int i = static_cast<int>(threadIdx.x); i < GR * DP / 4; i += 32 * kWarps) {
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
      for (int c = 0; c < kCols * 2; ++c) o[g][c] = 0;
    }
  }

  __device__ __forceinline__ void poison() {
#pragma unroll
    for (int g = 0; g < GR; ++g) l[g] = __int_as_float(0x7FC00000);
  }

  static __device__ __forceinline__ void lds_pairs(uint64_t (&v)[2], uint32_t a) {
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(v[0]), "=l"(v[1]) : "r"(a) : "memory");
  }

  __device__ __forceinline__ void step(const PagedParams &p, uint32_t ks, uint32_t vs,
                                       uint32_t valid, void *own) {
    const int lane = static_cast<int>(lane_id()), t = lane / kPer, part = lane % kPer;
    float *sp = static_cast<float *>(own);  // [kTok][GR] weights
    uint64_t pair[GR];  // two running sums per head
#pragma unroll
    for (int g = 0; g < GR; ++g) pair[g] = 0;
#pragma unroll 4
    for (int c = part; c < DP / 4; c += kPer) {
      uint64_t k[2];
      lds_pairs(k, ks + stage_at<kRowBytes, kPer>(t, c));
#pragma unroll
      for (int g = 0; g < GR; ++g) {
        uint64_t x[2];
        lds_pairs(x, q_at + g * DP * 4 + c * 16);
        pair[g] = fma_pair(x[0], k[0], pair[g]);
        pair[g] = fma_pair(x[1], k[1], pair[g]);
      }
    }
    float s[GR];
#pragma unroll
    for (int g = 0; g < GR; ++g) s[g] = low_of(pair[g]) + high_of(pair[g]);
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
      s[g] = exp2_of(s[g] - base);
    }
    if (moved) {  // the same in all lanes
#pragma unroll
      for (int g = 0; g < GR; ++g) {
        l[g] *= drop[g];
#pragma unroll
        for (int c = 0; c < kCols * 2; ++c) o[g][c] = mul_pair(o[g][c], pair_of(drop[g]));
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
    const int col = lane % kLanes, sub = kSplit == 1 ? 0 : lane / kLanes;
#pragma unroll 4
    for (int u = sub; u < kTok; u += kSplit) {
      float w[GR];
#pragma unroll
      for (int g = 0; g < GR; ++g) w[g] = sp[u * GR + g];
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        if (kQuads % kLanes && col + c * 32 >= kQuads) continue;
        uint64_t v[2];
        lds_pairs(v, vs + stage_at<kRowBytes, kPer>(u, col + c * 32));
#pragma unroll
        for (int g = 0; g < GR; ++g) {
          o[g][2 * c] = fma_pair(pair_of(w[g]), v[0], o[g][2 * c]);
          o[g][2 * c + 1] = fma_pair(pair_of(w[g]), v[1], o[g][2 * c + 1]);
        }
      }
    }
    __syncwarp();  // the weights are read before the next step writes them
  }

  static __device__ __forceinline__ int at(int h, int c) { return h * DP + c; }

  __device__ __forceinline__ void give(float *buf, float *sm, float *sl) {
    const int lane = static_cast<int>(lane_id()), col = lane % kLanes;
#pragma unroll
    for (int g = 0; g < GR; ++g) {
      float x = l[g];
#pragma unroll
      for (int w = 1; w < 32; w <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, w);
      if (lane == 0) {
        sm[g] = m[g];
        sl[g] = x;
      }
#pragma unroll
      for (int c = 0; c < kCols; ++c) {
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          y[e] = e & 1 ? high_of(o[g][2 * c + e / 2]) : low_of(o[g][2 * c + e / 2]);
          if constexpr (kSplit == 2) y[e] += __shfl_xor_sync(0xFFFFFFFFu, y[e], 16);
        }
        if (lane < kLanes && col + c * 32 < kQuads)
          *reinterpret_cast<float4 *>(buf + at(g, 4 * (col + c * 32))) = make_float4(y[0], y[1], y[2], y[3]);
      }
    }
  }
};

// --------------------------------------------------------------------------
// The kernel
// --------------------------------------------------------------------------
template <class Core, int NS>
struct PagedShape {
  static constexpr int kTile = Core::kTok * Core::kWarps;  // tokens
  static constexpr uint32_t kHalf = Core::kTok * Core::kRowBytes;  // K or V of a stage
  static constexpr uint32_t kRing = NS * 2 * kHalf;               // of a warp
  // an item's end puts the warp's sums where its last stage was
  static_assert(Core::kRows * Core::kDim * 4 <= 2 * kHalf, "a stage holds the sums");
  static constexpr int kThreads = 32 * Core::kWarps;
  static constexpr int kCost = Core::kDim > 128 ? 2 : 1;  // of an item's end, in tiles
  static constexpr uint32_t kSmem = Core::kWarps * (kRing + Core::kWarpBytes) + Core::kQBytes;
  // CTAs per SM that the registers have to allow, of those that shared memory
  // holds.  Of four warps: four for up to eight query heads (128 registers), three
  // for rows of 96 where four spill (72.4 us and 74.9 for e4m3, 123.9 and 124.3 for
  // bf16, 71.0 and 81.0 for eight fp32 heads), three for sixteen heads and rows of
  // 64 (75.8 us, 83.6 with four: e4m3), two for sixteen and wider rows (three fit
  // rows of 96 only, and serve them better: 80.2 us against 87.2 for bf16).  Rows
  // wider than 128 have the registers that their sums need, 168 or 256.
  static constexpr int kFit = static_cast<int>(226 * 1024 / (kSmem + 2048));
  static constexpr int kFour = Core::kDim == 96 && (!Core::kFma || Core::kRows > 4) ? 3 : 4;
  static constexpr int kMost = (Core::kFma || Core::kRows <= 8 ? kFour : Core::kDim > 64 ? 2 : 3) * 4 / Core::kWarps;
  static constexpr int kRegs = Core::kDim <= 128 ? kMost
                               : Core::kElemBytes == 1 && Core::kRows <= 8 ? 3
                               : 65536 / (256 * 32 * Core::kWarps);
  static constexpr int kMin = kFit > kMost ? kMost : kFit;
  static constexpr int kPerSm = kMin > kRegs ? kRegs : kMin;
};

// Tiles of request r's items, 0 where nothing is attended; `bad`: its length
// is outside the table.
struct PagedSpan {
  int32_t len, first, t0, tiles;
};
template <int TILE>
__device__ __forceinline__ PagedSpan paged_span(const PagedParams &p, int32_t len, bool &bad) {
  PagedSpan s;
  bad = len < 0 || len > p.room;
  s.len = bad ? 0 : len;
  s.first = p.window > 0 && s.len > p.window ? s.len - p.window : 0;
  s.t0 = s.first & ~(kPagedPage - 1);
  s.tiles = (s.len - s.t0 + TILE - 1) / TILE;
  return s;
}

// What an item costs beside its tiles, in tiles: its CTA's warps wait for one
// another and join (2.5 to 4.5 us against about 2 us per tile, measured on 128
// requests of up to 8000 tokens).  Runs are cut in these units: an item's tiles,
// then COST units without one.  Against runs of equal tiles: 98 to 92 us for
// 1024 requests of up to 500 tokens, 57 to 54 for 16 of up to 16,000 in e4m3;
// two units serve rows wider than 128 better (28.6 to 25.7 us, 26.7 with one,
// for a window of 1024 over rows of 256), one the others.
template <int COST>
__device__ __forceinline__ int32_t paged_units(const PagedSpan &s) {
  return s.tiles > 0 ? s.tiles + COST : 0;
}

// A CTA's run of units [u0, u1) of all, and where unit u0 is.
struct PagedRun {
  int64_t run, u0, u1;  // run: units of a full run
  int32_t request, len, head, piece, tile;
};

// Every warp finds it for itself, so that none waits: a lane takes four
// requests of 128 at a time, one round of loads and one warp scan where that
// is all of them.  It stands before a call's first load of the cache, and with
// few requests most of what it takes is the latency of its instructions: 32-bit
// sums and a multiplication for the division where the tiles allow.
template <class Int, int TILE, int COST>
__device__ __forceinline__ PagedRun paged_run(const PagedParams &p) {
  const int lane = static_cast<int>(lane_id());
  const Int per_request = static_cast<Int>(p.kv_heads * p.pieces);
  int32_t len[4];
  Int mine[4], sum, in;
  const auto load = [&](int64_t r0) {  // a round's requests: four per lane
    sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t r = r0 + 4 * lane + i;
      len[i] = r < p.n_requests ? p.lens[r] : 0;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      bool bad;
      mine[i] = static_cast<Int>(paged_units<COST>(paged_span<TILE>(p, len[i], bad))) * per_request;
      sum += mine[i];
    }
  };
  const auto scan = [&]() {
    in = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const Int x = __shfl_up_sync(0xFFFFFFFFu, in, o);
      if (lane >= o) in += x;
    }
  };
  Int total = 0;
  for (int64_t r0 = 128; r0 < p.n_requests; r0 += 128) {
    load(r0);
    total += sum;
  }
  if (p.n_requests > 128) {
#pragma unroll
    for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xFFFFFFFFu, total, o);
  }
  load(0);
  scan();
  Int seen = __shfl_sync(0xFFFFFFFFu, in, 31);
  total += seen;

  PagedRun y;
  Int run;
  if constexpr (sizeof(Int) == 4) run = p.by_ctas.div(total + p.ctas - 1);
  else run = (total + p.ctas - 1) / p.ctas;
  const Int u0 = run * static_cast<Int>(blockIdx.x);
  y.run = run;
  y.u0 = u0;
  y.u1 = min(u0 + run, total);
  y.request = y.len = y.head = y.piece = y.tile = 0;
  if (u0 >= total) return y;
  for (int64_t r0 = 0;;) {
    if (u0 < seen) {
      const Int before = seen - __shfl_sync(0xFFFFFFFFu, in, 31) + in - sum;
      const int owner = __ffs(__ballot_sync(0xFFFFFFFFu, u0 < before + sum)) - 1;
      int which = 0;
      Int skip = before;
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (which == i && u0 >= skip + mine[i]) {
          skip += mine[i];
          which = i + 1;
        }
      int32_t l = len[0];
#pragma unroll
      for (int i = 1; i < 4; ++i)
        if (which == i) l = len[i];
      y.request = __shfl_sync(0xFFFFFFFFu, static_cast<int32_t>(r0) + 4 * lane + which, owner);
      y.len = __shfl_sync(0xFFFFFFFFu, l, owner);
      const Int off = u0 - __shfl_sync(0xFFFFFFFFu, skip, owner);
      bool bad;
      const Int units = static_cast<Int>(paged_units<COST>(paged_span<TILE>(p, y.len, bad)));
      const int32_t item = static_cast<int32_t>(off / units);
      y.tile = static_cast<int32_t>(off - item * units);
      y.head = p.pieces == 1 ? item : item / p.pieces;
      y.piece = item - y.head * p.pieces;
      return y;
    }
    r0 += 128;
    if (r0 >= p.n_requests) {  // only if the lengths changed meanwhile
      y.u1 = y.u0;
      return y;
    }
    load(r0);
    scan();
    seen += __shfl_sync(0xFFFFFFFFu, in, 31);
  }
}

__device__ __forceinline__ void paged_store4(const PagedParams &p, int64_t at, float4 x) {
  if (p.out_f32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = x;
  } else {
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) =
        make_uint2(bf16x2_of(x.x, x.y), bf16x2_of(x.z, x.w));
  }
}

__device__ __forceinline__ float paged_lse(float top, float sum) {
  return top == -INFINITY && sum == 0.0f ? -INFINITY : (top + log2f(sum)) * kLn2;
}

// The place of an item's part k: its first part is its CTA's place 1.
__device__ __forceinline__ int64_t place_of(int first, int k) {
  return 2 * (static_cast<int64_t>(first) + k) + (k == 0 ? 1 : 0);
}

// Four columns of a row of one or several parts.
struct PagedSum {
  float4 x;
  float top, sum;
};

__device__ __forceinline__ uint64_t counted(const unsigned long long *p) {
  uint64_t x;
  asm volatile("ld.relaxed.gpu.global.u64 %0, [%1];" : "=l"(x) : "l"(p) : "memory");
  return x;
}
// Parts that have come, by a counter's value; -1 if it is not (yet) this call's.
__device__ __forceinline__ int come_of(uint64_t x, uint64_t base) {
  return (x >> kCallShift) == (base >> kCallShift) ? static_cast<int>(x - base) : -1;
}

__device__ __forceinline__ void take_in(PagedSum &y, float f, const float4 &x, float sum) {
  y.sum = fmaf(f, sum, y.sum);
  y.x.x = fmaf(f, x.x, y.x.x);
  y.x.y = fmaf(f, x.y, y.x.y);
  y.x.z = fmaf(f, x.z, y.x.z);
  y.x.w = fmaf(f, x.w, y.x.w);
}

// Parts k0, k0 + step, .. below k1, AHEAD of them asked for at once, from L2
// (other SMs wrote them).  Part `mine` is not read: it is `own`.
template <int AHEAD>
__device__ __forceinline__ PagedSum join_parts(const PagedParams &p, int first, int row, int col,
                                               int k0, int k1, int step, int mine,
                                               const PagedSum &own) {
  PagedSum y;
  y.x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  y.top = -INFINITY;
  y.sum = 0.0f;
#pragma unroll 1
  for (int k = k0; k < k1; k += step * AHEAD) {
    PagedSum a[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int part = k + i * step;
      a[i].x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      a[i].top = -INFINITY;
      a[i].sum = 0.0f;
      if (part == mine) {
        a[i] = own;
      } else if (part < k1) {
        const int64_t at = place_of(first, part) * kPagedRows + row;
        const float2 ml = __ldcg(p.ml + at);
        a[i].top = ml.x;
        a[i].sum = ml.y;
        a[i].x = __ldcg(reinterpret_cast<const float4 *>(p.acc + at * kPagedMaxDim + col));
      }
    }
    float top = y.top;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) top = fmaxf(top, a[i].top);
    const PagedSum was = y;
    y.x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    y.sum = 0.0f;
    y.top = top;
    take_in(y, exp2_from(was.top, top), was.x, was.sum);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) take_in(y, exp2_from(a[i].top, top), a[i].x, a[i].sum);
  }
  return y;
}

// Four columns of a head's output, and with the first of them its lse.
__device__ __forceinline__ void paged_answer(const PagedParams &p, int request, int kv_head,
                                             int64_t head, int col, const PagedSum &y) {
  const float f = y.sum == 0.0f ? 0.0f : (p.v_scale ? p.v_scale[kv_head] : 1.0f) / y.sum;
  paged_store4(p, request * p.o_req + head * p.o_head + col,
               make_float4(y.x.x * f, y.x.y * f, y.x.z * f, y.x.w * f));
  if (col == 0 && p.lse)
    p.lse[static_cast<int64_t>(request) * p.kv_heads * p.group + head] = paged_lse(y.top, y.sum);
}

// PAGE16: the block size is a multiple of 16, so that every 16 tokens of a
// stage lie in one block, whose rows follow one another: one table entry per
// 16 tokens and addresses by addition, instead of both per token.
template <class Core, int NS, bool PAGE16>
__global__ void __launch_bounds__(PagedShape<Core, NS>::kThreads, PagedShape<Core, NS>::kPerSm)
    paged_attention_kernel(const PagedParams p) {
  using Shape = PagedShape<Core, NS>;
  using Elem = std::conditional_t<Core::kFma, float, uint16_t>;  // of the queries
  constexpr int kPagedWarps = Core::kWarps, kPagedThreads = Shape::kThreads;
  extern __shared__ __align__(128) unsigned char paged_smem[];
  __shared__ uint32_t valid_ring[kPagedWarps][NS], lost_ring[kPagedWarps][NS];
  __shared__ float sm[kPagedWarps][kPagedRows], sl[kPagedWarps][kPagedRows];
  __shared__ int s_come;
  __shared__ uint64_t s_base;  // thread 0's: the call's number times 2^kCallShift

  const int tid = static_cast<int>(threadIdx.x), lane = tid & 31, warp = tid >> 5;
  unsigned char *ring = paged_smem + warp * Shape::kRing;
  const uint32_t ring_at = static_cast<uint32_t>(__cvta_generic_to_shared(ring));
  unsigned char *own = paged_smem + kPagedWarps * Shape::kRing + warp * Core::kWarpBytes;
  unsigned char *sq = paged_smem + kPagedWarps * (Shape::kRing + Core::kWarpBytes);
  pdl_wait_and_release();

  // ---- this CTA's run of tiles ----
  const int n_heads = p.kv_heads * p.group;
  uint32_t bits = 0;
  PagedRun at;
  if (p.tiles_fit)
    at = paged_run<uint32_t, Shape::kTile, Shape::kCost>(p);
  else
    at = paged_run<int64_t, Shape::kTile, Shape::kCost>(p);
  const int64_t run = at.run, u0 = at.u0, u1 = at.u1;

  // requests with nothing to attend to
  const auto answer_empty = [&]() {
    for (int64_t r = blockIdx.x; r < p.n_requests; r += p.ctas) {
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
          p.lse[r * n_heads + h] = bad ? x : -INFINITY;
    }
  };
  if (!p.join_here && tid < 2) p.parts[2 * static_cast<int64_t>(blockIdx.x) + tid].parts = 0;
  uint64_t call = 0;  // thread 0's
  if (p.calls && tid == 0) {
    call = counted(p.calls + blockIdx.x);  // of this CTA alone, one call after the other
    for (int b = static_cast<int>(blockIdx.x); b < p.all_ctas; b += p.ctas) atomicAdd(p.calls + b, 1ull);
  }
  if (u0 >= u1) {
    answer_empty();
    if (bits && tid == 0) atomicOr(p.status, bits);
    return;
  }

  // ---- cursors over the run: requests, their key heads, pieces of the query
  // heads, tiles ----
  struct Cursor {
    int64_t left;  // units of the run, this tile's included
    int32_t request, head, piece, tile;
    PagedSpan span;
  };
  // steps to the next tile; true where that is another item's first
  const auto next = [&](Cursor &c) {
    --c.left;
    if (++c.tile < c.span.tiles) return false;
    c.left -= Shape::kCost - (c.tile - c.span.tiles);
    c.tile = 0;
    if (++c.piece == p.pieces) {
      c.piece = 0;
      if (++c.head == p.kv_heads) {
        c.head = 0;
        if (c.left > 0) {
          bool bad;
          do {
            if (++c.request >= p.n_requests) {
              c.left = 0;
              break;
            }
            c.span = paged_span<Shape::kTile>(p, p.lens[c.request], bad);
          } while (c.span.tiles == 0);
        }
      }
    }
    return true;
  };
  Cursor use;
  use.left = u1 - u0;
  use.request = at.request;
  use.head = at.head;
  use.piece = at.piece;
  use.tile = at.tile;
  {
    bool bad;
    use.span = paged_span<Shape::kTile>(p, at.len, bad);
  }
  if (use.tile >= use.span.tiles) {  // the run begins behind an item's tiles
    ++use.left;
    --use.tile;
    next(use);
  }
  if (use.left <= 0) {
    answer_empty();
    if (bits && tid == 0) atomicOr(p.status, bits);
    return;
  }
  Cursor get = use;

  // ---- loading: a stage's table entry and mask byte are fetched one stage
  // before its rows ----
  constexpr int kChunks = Core::kRowBytes / 16;              // of a row
  // rows that the lanes copy at once (a power of two), copies of a row by all lanes
  constexpr int kRowsAt = kChunks <= 4 ? 8 : kChunks <= 8 ? 4 : kChunks <= 16 ? 2 : 1;
  constexpr int kParts = (kChunks + 31) / 32;
  constexpr uint32_t kAll = Core::kTok == 32 ? 0xFFFFFFFFu : (1u << (Core::kTok & 31)) - 1;
  const int my_row = kChunks <= 32 ? min(lane / kChunks, kRowsAt - 1) : 0;
  const int my_chunk = kChunks <= 32 ? lane - my_row * kChunks : lane;  // kChunks and more: none
  const int chunks = p.dim * Core::kElemBytes / 16;
  const uint32_t my_at = ring_at + stage_at<Core::kRowBytes, Core::kPer>(my_row, my_chunk);
  // the rows are read once per step: in L2 they make way for what every layer
  // and CTA reads again (tables, lengths, queries, parts)
  const uint64_t policy = l2_evict_first();
  const int32_t *table = nullptr;
  const uint8_t *mask = nullptr;
  const char *kh = nullptr, *vh = nullptr;  // the item's rows, for this lane's first chunk
  const auto aim = [&]() {
    table = p.table + get.request * p.table_stride;
    if (p.mask) mask = p.mask + get.request * p.mask_stride;
    kh = static_cast<const char *>(p.k) + get.head * p.k_head;
    vh = static_cast<const char *>(p.v) + get.head * p.v_head;
  };
  aim();
  int32_t entry = -1;
  bool keep = false;
  const auto look_up = [&]() {
    if (get.left <= 0) return;
    const int32_t base = get.span.t0 + get.tile * Shape::kTile + warp * Core::kTok;
    const int32_t t = base + lane % Core::kTok;
    keep = t >= get.span.first && t < get.span.len;
    entry = -1;
    if constexpr (PAGE16) {
      // a lane's entry is that of its token's 16
      const int32_t at = Core::kTok <= kPagedPage ? base : base + (lane & kPagedPage);
      if (at < get.span.len) entry = table[p.by_block.div(static_cast<uint32_t>(at))];
    } else if (keep) {
      entry = table[p.by_block.div(static_cast<uint32_t>(t))];
    }
    if (keep && mask) keep = mask[t] != 0;
  };
  const auto fetch = [&](int stage) {
    const int32_t base = get.span.t0 + get.tile * Shape::kTile + warp * Core::kTok;
    const bool inside = entry >= 0 && entry < p.n_blocks;
    const uint32_t want = __ballot_sync(0xFFFFFFFFu, keep) & kAll;
    const uint32_t valid = __ballot_sync(0xFFFFFFFFu, keep && inside) & kAll;
    if (lane == 0) {
      valid_ring[warp][stage] = valid;
      // a wanted token's block is outside the cache
      lost_ring[warp][stage] = want != valid;
    }
    const uint32_t to = (Core::kRowBytes % 128 ? ring_at + my_row * Core::kRowBytes : my_at) + stage * 2 * Shape::kHalf;
    const int my_place = my_chunk ^ stage_xor<Core::kRowBytes, Core::kPer>(my_row);
    // copies rows r0 .. r0 + n - 1 of the stage from rows that lie a token
    // stride apart, the first at ka and va (this lane's row and chunk)
    const auto copy = [&](int r0, int n, const char *ka, const char *va) {
#pragma unroll
      for (int i = 0; i < n / kRowsAt; ++i) {
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
          const int r = r0 + i * kRowsAt;
          if ((kRowsAt * kChunks) % 32 && my_chunk + 32 * part >= kChunks) continue;
          const bool real = ((valid >> (r + my_row)) & 1u) && my_chunk + 32 * part < chunks;
          constexpr bool kLines = Core::kRowBytes % 128 == 0;  // a row's address has its chunk's bits
          const uint32_t at =
              kLines ? (to ^ (stage_xor<Core::kRowBytes, Core::kPer>(r) << 4)) + r * Core::kRowBytes + 512 * part
                     : to + r * Core::kRowBytes + ((my_place ^ stage_xor<Core::kRowBytes, Core::kPer>(r)) << 4);
          const int skip = my_chunk + 32 * part < chunks ? 16 * (my_chunk + 32 * part) : 0;
          cp_async16_or_zero(at, ka + skip, real, policy);
          cp_async16_or_zero(at + Shape::kHalf, va + skip, real, policy);
        }
        ka += static_cast<int64_t>(kRowsAt) * p.k_token;
        va += static_cast<int64_t>(kRowsAt) * p.v_token;
      }
    };
    if constexpr (PAGE16) {
      // a block holds whole groups of 16 tokens, all of them inside the cache
      constexpr int kGroup = Core::kTok <= kPagedPage ? Core::kTok : kPagedPage;
#pragma unroll
      for (int r0 = 0; r0 < Core::kTok; r0 += kGroup) {
        const int32_t e = Core::kTok <= kPagedPage ? entry : __shfl_sync(0xFFFFFFFFu, entry, r0);
        const uint32_t t = static_cast<uint32_t>(base + r0);
        const int32_t b = e >= 0 && e < p.n_blocks ? e : 0;
        const int32_t off = static_cast<int32_t>(t - p.by_block.div(t) * p.by_block.d) + my_row;
        copy(r0, kGroup, kh + wide_product(b, p.k_block) + wide_product(off, p.k_token),
             vh + wide_product(b, p.v_block) + wide_product(off, p.v_token));
      }
    } else {
      // the lane of a row knows where it lies
      const uint32_t t = static_cast<uint32_t>(base + lane % Core::kTok);
      const int32_t b = keep && inside ? entry : 0;
      const int32_t off = keep && inside ? static_cast<int32_t>(t - p.by_block.div(t) * p.by_block.d) : 0;
      const int64_t ko = wide_product(b, p.k_block) + wide_product(off, p.k_token);
      const int64_t vo = wide_product(b, p.v_block) + wide_product(off, p.v_token);
#pragma unroll
      for (int r = 0; r < Core::kTok; r += kRowsAt)
        copy(r, kRowsAt, kh + __shfl_sync(0xFFFFFFFFu, ko, r + my_row),
             vh + __shfl_sync(0xFFFFFFFFu, vo, r + my_row));
    }
  };
  const auto advance = [&]() {
    if (next(get) && get.left > 0) {
      aim();
      // the item's queries towards L1, a line per lane
      const char *q = reinterpret_cast<const char *>(
          static_cast<const Elem *>(p.q) + get.request * p.q_req +
          (static_cast<int64_t>(get.head) * p.group + get.piece * p.rows) * p.q_head);
      const int rows = min(p.rows, p.group - get.piece * p.rows);
      for (int r = warp; r < rows; r += kPagedWarps)
        if (lane * 128 < p.dim * static_cast<int>(sizeof(Elem)))
          asm volatile("prefetch.global.L1 [%0];" ::"l"(q + r * p.q_head * sizeof(Elem) + lane * 128));
    }
    look_up();
  };

  look_up();
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    if (get.left > 0) {
      fetch(s);
      advance();
    }
    cp_async_commit();
  }

  answer_empty();
  if (tid == 0) s_base = call << kCallShift;

  // ---- the run ----
  Core core;
  int stage = 0, fill = NS - 1;
  bool fresh = true;       // the item's queries are not loaded yet
  bool from_start = true;  // the run holds the item's first tile
  while (use.left > 0) {
    if (fresh) {
      const int64_t head = static_cast<int64_t>(use.head) * p.group + use.piece * p.rows;
      core.begin(p, static_cast<const Elem *>(p.q) + use.request * p.q_req + head * p.q_head,
                 min(p.rows, p.group - use.piece * p.rows), p.k_scale ? p.k_scale[use.head] : 1.0f, sq);
      from_start = use.tile == 0;
      fresh = false;
    }
    cp_async_wait_group<NS - 2>();
    __syncwarp();  // the stage is in, and the one before it is no longer read
    if (get.left > 0) {
      fetch(fill);
      advance();
    }
    cp_async_commit();
    const uint32_t valid = valid_ring[warp][stage];
    const uint32_t ks = ring_at + stage * 2 * Shape::kHalf;
    if (valid) core.step(p, ks, ks + Shape::kHalf, valid, own);
    if (lost_ring[warp][stage]) {
      core.poison();
      bits |= kRowBadBlock;
    }

    const bool item_end = use.tile == use.span.tiles - 1;
    if (item_end || use.left == 1) {
      // ---- the warps' parts as one: each puts its sums where its stage
      // was ----
      __syncwarp();
      const bool whole = from_start && item_end;
      PagedParts d;
      if (!whole) {
        // the item's tiles among all units: from its first to its last
        const int64_t begin = u1 - use.left - use.tile, last = begin + use.span.tiles - 1;
        if (p.tiles_fit) {
          d.first = static_cast<uint32_t>(begin) / static_cast<uint32_t>(run);
          d.parts = static_cast<uint32_t>(last) / static_cast<uint32_t>(run) - d.first + 1;
        } else {
          d.first = static_cast<int32_t>(begin / run);
          d.parts = static_cast<int32_t>(last / run) - d.first + 1;
        }
        d.request = use.request;
        d.head = use.head;
        d.piece = use.piece;
      }
      // whether the others are there is asked before the sums are written
      int come = -1;
      if (!whole && tid == 0 && p.join_here) come = come_of(counted(p.arrived + d.first), s_base);
      core.give(reinterpret_cast<float *>(ring + stage * 2 * Shape::kHalf), sm[warp], sl[warp]);
      if (!whole && tid == 0) {
        if (come == d.parts - 1) __threadfence();
        s_come = come;
      }
      __syncthreads();
      const int rows = min(p.rows, p.group - use.piece * p.rows), quads = p.dim / 4;
      const int64_t head = static_cast<int64_t>(use.head) * p.group + use.piece * p.rows;
      const int64_t place = 2 * static_cast<int64_t>(blockIdx.x) + (from_start ? 1 : 0);
      const int mine = whole ? 0 : static_cast<int>(blockIdx.x) - d.first;
      bool join = !whole && s_come == d.parts - 1;
      const auto each = [&](bool publish, bool joined) {
        for (int i = tid; i < rows * quads; i += kPagedThreads) {
          const int r = i / quads, c = 4 * (i - r * quads);
          PagedSum y;
          y.top = sm[0][r];
#pragma unroll
          for (int w = 1; w < kPagedWarps; ++w) y.top = fmaxf(y.top, sm[w][r]);
          y.sum = 0.0f;
          y.x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
          for (int w = 0; w < kPagedWarps; ++w)
            take_in(y, exp2_from(sm[w][r], y.top),
                    *reinterpret_cast<const float4 *>(
                        reinterpret_cast<const float *>(paged_smem + w * Shape::kRing +
                                                        stage * 2 * Shape::kHalf) + Core::at(r, c)),
                    sl[w][r]);
          if (publish) {
            *reinterpret_cast<float4 *>(p.acc + (place * kPagedRows + r) * kPagedMaxDim + c) = y.x;
            if (c == 0) p.ml[place * kPagedRows + r] = make_float2(y.top, y.sum);
          } else {
            if (joined) y = join_parts<4>(p, d.first, r, c, 0, d.parts, 1, mine, y);
            paged_answer(p, use.request, use.head, head + r, c, y);
          }
        }
      };
      if (whole || join) {
        each(false, join);
      } else {
        each(true, false);
        if (p.join_here) {
          __syncthreads();  // the part is written
          if (tid == 0) {
            __threadfence();
            if (come < 0) atomicMax(p.arrived + d.first, static_cast<unsigned long long>(s_base));
            s_come = come_of(atomicAdd(p.arrived + d.first, 1ull), s_base);
            __threadfence();
          }
          __syncthreads();
          if (s_come == d.parts - 1) each(false, true);  // the others came meanwhile
        } else if (tid == 0) {
          p.parts[place] = d;
        }
      }
      __syncthreads();  // the sums are read before the stage is filled again
      fresh = true;
    }
    stage = stage + 1 == NS ? 0 : stage + 1;
    fill = fill + 1 == NS ? 0 : fill + 1;
    next(use);
  }
  cp_async_wait_group<0>();
  if (bits && lane == 0) atomicOr(p.status, bits);
}

}  // namespace ts
