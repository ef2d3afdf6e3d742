// ts_kv.cuh -- the paged key-value cache's bookkeeping and writes: block
// tables and slot maps built from request lengths (kv_tables_kernel), and the
// write of new tokens' keys and values at their slots (kv_append_kernel).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "ts_e4m3.cuh"
#include "ts_kv_common.cuh"

namespace ts {

// --------------------------------------------------------------------------
// Block tables and slot maps
// --------------------------------------------------------------------------
constexpr int kTablesMaxThreads = 1024;
constexpr int kTablesMaxRequests = 8192;
constexpr int kTablesPerThread = kTablesMaxRequests / kTablesMaxThreads;

struct KvTablesParams {
  int32_t n_requests, block_size, n_blocks, max_blocks, max_tokens, free_len;
  int64_t table_stride;
  int32_t *block_table;
  const int32_t *lens;
  const int32_t *n_new;      // null: one token each
  const uint8_t *finished;   // null: none
  int32_t *free_blocks;
  const int32_t *n_free;
  int32_t *lens_out;         // where this launch leaves them (a scratch array when
  int32_t *n_free_out;       // several blocks work in place)
  int32_t *token_starts;
  int64_t *slots;
  int32_t *positions;        // may be null
  int32_t *requests;         // may be null
  uint32_t *status;
  FastDiv by_block;
  int32_t per_lane;          // map entries a lane fills in a row: 1 or 4
  int32_t wide_maps;         // slots, positions and requests are 16-byte aligned
};

__host__ __device__ constexpr uint32_t kv_tables_smem(int n_requests) {
  return static_cast<uint32_t>(4 * (n_requests + 1)) * 4u;
}

// Exclusive prefix sums of K values per thread over the block's first `warps`
// warps; total[] gets the sums in all threads.  `part` holds K * 32 values.
// Ends with the block in step.
template <int K, class Int>
__device__ __forceinline__ void block_scan(const Int (&x)[K], Int (&before)[K], Int (&total)[K],
                                           Int *part, int warps) {
  const int lane = static_cast<int>(lane_id());
  const int warp = static_cast<int>(threadIdx.x) >> 5;
  Int in[K];
#pragma unroll
  for (int k = 0; k < K; ++k) in[k] = x[k];
  if (warp < warps) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      Int u[K];
#pragma unroll
      for (int k = 0; k < K; ++k) u[k] = __shfl_up_sync(0xFFFFFFFFu, in[k], o);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (lane >= o) in[k] += u[k];
    }
    if (lane == 31) {
#pragma unroll
      for (int k = 0; k < K; ++k) part[k * 32 + warp] = in[k];
    }
  }
  __syncthreads();
  if (warps == 1) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      total[k] = part[k * 32];
      before[k] = in[k] - x[k];
    }
  } else {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      Int v = lane < warps ? part[k * 32 + lane] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const Int u = __shfl_up_sync(0xFFFFFFFFu, v, o);
        if (lane >= o) v += u;
      }
      total[k] = __shfl_sync(0xFFFFFFFFu, v, 31);
      const Int w = __shfl_sync(0xFFFFFFFFu, v, warp > 0 ? warp - 1 : 0);
      before[k] = in[k] - x[k] + (warp > 0 ? w : 0);
    }
  }
  __syncthreads();
}

// The last i in [0, n) with start[i] <= x, for ascending starts and start[0] <= x.
__device__ __forceinline__ int last_start(const int32_t *start, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

// Every block scans all requests (12 bytes each, from L2) into its shared
// memory and then fills its share of the three lists that the scans lay out:
// released blocks, handed-out blocks and new tokens, each entry finding its
// request by bisection.  One launch therefore serves from one request to
// thousands with hundreds of thousands of tokens: scanning again in every
// block costs about as much as one launch boundary, and a second launch that
// read the scans back would cost that and the reading.  Bound by latency (loads,
// a scan, a search, a load) up to some ten thousand tokens, then by the maps'
// 16 bytes per token.  As few warps scan as hold four or eight requests per
// lane: all 32 would take their turns at the shuffles (1.2 us against 0.4 for
// 128 requests).  Int: 32 bits where n_requests * room fits, which bounds every
// sum.
template <class Int>
__global__ void __launch_bounds__(kTablesMaxThreads) kv_tables_kernel(const KvTablesParams p) {
  extern __shared__ int32_t kv_smem[];
  __shared__ Int part[3 * 32];
  const int n = p.n_requests;
  int32_t *tok_start = kv_smem;              // [n + 1] first token of a request
  int32_t *blk_start = tok_start + (n + 1);  // [n + 1] blocks handed out before it
  int32_t *rel_start = blk_start + (n + 1);  // [n + 1] blocks released before it
  int32_t *len_of = rel_start + (n + 1);     // [n] length before the call
  const int t = static_cast<int>(threadIdx.x), nt = static_cast<int>(blockDim.x);
  const int per = n <= 4 * nt ? 4 : kTablesPerThread;
  const int scanning = (n + 32 * per - 1) / (32 * per);  // warps
  const int i0 = t * per;
  const bool first_block = blockIdx.x == 0;
  pdl_wait_and_release();

  uint32_t bits = 0;
  const int32_t free_in = *p.n_free;
  const int32_t free0 = min(max(free_in, 0), p.free_len);
  if (free0 != free_in) bits |= kRowBadShape;
  const int64_t room = static_cast<int64_t>(p.max_blocks) * p.block_size;

  int32_t want[kTablesPerThread], need[kTablesPerThread], out_len[kTablesPerThread];
  uint32_t gone = 0;  // requests that end here (bit j)
  Int sum[3] = {0, 0, 0};
#pragma unroll
  for (int j = 0; j < kTablesPerThread; ++j) {
    want[j] = need[j] = out_len[j] = 0;
    const int i = i0 + j;
    if (j < per && i < n) {
      const int32_t len = p.lens[i];
      const int32_t a = p.n_new ? p.n_new[i] : 1;
      const bool fin = p.finished && p.finished[i];
      const bool bad = len < 0 || len > room || (!fin && (a < 0 || len + static_cast<int64_t>(a) > room));
      out_len[j] = len;
      len_of[i] = bad ? 0 : len;
      int32_t held = 0;
      if (bad) {
        bits |= kRowBadShape;
      } else {
        held = static_cast<int32_t>(p.by_block.div(static_cast<uint32_t>(len)));
        if (held * static_cast<int64_t>(p.block_size) < len) ++held;
        if (fin) {
          gone |= 1u << j;
          sum[2] += held;
          need[j] = held;
        } else {
          want[j] = a;
          const int32_t end = len + a;
          int32_t all = static_cast<int32_t>(p.by_block.div(static_cast<uint32_t>(end)));
          if (all * static_cast<int64_t>(p.block_size) < end) ++all;
          need[j] = all - held;
          sum[0] += need[j];
          sum[1] += a;
        }
      }
    }
  }
  Int before[3], total[3];
  block_scan<3, Int>(sum, before, total, part, scanning);

  // the stack with the released blocks on it; entries past its end are dropped
  const int64_t top64 = static_cast<int64_t>(free0) + total[2];
  const int32_t top = static_cast<int32_t>(min(top64, static_cast<int64_t>(p.free_len)));
  if (top < top64) bits |= kRowBadShape;
  const int32_t released = top - free0;

  Int blocks = before[0], tokens = before[1], rel = before[2];
  Int got[2] = {0, 0};
  bool refused = false;
#pragma unroll
  for (int j = 0; j < kTablesPerThread; ++j) {
    const int i = i0 + j;
    if (j < per && i < n) {
      rel_start[i] = static_cast<int32_t>(min(rel, static_cast<Int>(released)));
      if ((gone >> j) & 1u) {
        rel += need[j];
        need[j] = 0;
        out_len[j] = 0;
      } else {
        blocks += need[j];
        tokens += want[j];
        const bool given = want[j] == 0 || ((need[j] == 0 || blocks <= top) && tokens <= p.max_tokens);
        if (!given) {
          want[j] = need[j] = 0;
          refused = true;
          bits |= kRowNoBlocks;
        }
        got[0] += want[j];
        got[1] += need[j];
      }
    }
  }
  Int at[2] = {before[1], before[0]}, all[2] = {total[1], total[0]};
  if (__syncthreads_or(refused)) block_scan<2, Int>(got, at, all, part, scanning);
  const int32_t n_tokens = static_cast<int32_t>(all[0]), n_given = static_cast<int32_t>(all[1]);
  int32_t tok = static_cast<int32_t>(at[0]), blk = static_cast<int32_t>(at[1]);
#pragma unroll
  for (int j = 0; j < kTablesPerThread; ++j) {
    const int i = i0 + j;
    if (j < per && i < n) {
      tok_start[i] = tok;
      blk_start[i] = blk;
      if (first_block) {
        p.token_starts[i] = tok;
        p.lens_out[i] = out_len[j] + want[j];
      }
      tok += want[j];
      blk += need[j];
    }
  }
  if (t == 0) {
    tok_start[n] = n_tokens;
    blk_start[n] = n_given;
    rel_start[n] = released;
    if (first_block) {
      p.token_starts[n] = n_tokens;
      *p.n_free_out = top - n_given;
    }
  }
  if (!first_block) bits = 0;  // one report per call
  __syncthreads();

  const auto held_of = [&](int32_t len) {
    const int32_t b = static_cast<int32_t>(p.by_block.div(static_cast<uint32_t>(len)));
    return b * static_cast<int64_t>(p.block_size) < len ? b + 1 : b;
  };
  // where entry x of the blocks that the call releases stands
  const auto released_at = [&](int32_t x) {
    const int r = last_start(rel_start, n, x);
    return p.block_table + r * p.table_stride + (x - rel_start[r]);
  };
  // where entry x of the stack as the releases leave it stands (in the tables
  // for the released ones, so that no thread waits for the stores of another)
  const auto stack_at = [&](int32_t x) {
    return x < free0 ? p.free_blocks + x : released_at(x - free0);
  };

  // what the slots of a request's block b come from: its table, or for a new
  // block the stack
  const auto block_at = [&](int r, int32_t b, int32_t held) {
    return b < held ? p.block_table + r * p.table_stride + b
                    : stack_at(top - 1 - (blk_start[r] + b - held));
  };
  const auto slot_of = [&](int32_t id, int32_t off) {
    if (id < 0 || id >= p.n_blocks) {
      bits |= kRowBadBlock;
      return static_cast<int64_t>(-1);
    }
    return static_cast<int64_t>(id) * p.block_size + off;
  };

  // entry y of the token maps, whose request is r or a later one
  const auto map_token = [&](int32_t y, int &r, int64_t &slot, int32_t &pos, int32_t &of) {
    slot = pos = of = -1;
    if (y >= n_tokens) return;
    if (y >= tok_start[r + 1]) r = last_start(tok_start, n, y);
    const int32_t len = len_of[r];
    pos = len + (y - tok_start[r]);
    of = r;
    const int32_t b = static_cast<int32_t>(p.by_block.div(static_cast<uint32_t>(pos)));
    slot = slot_of(*block_at(r, b, held_of(len)), pos - b * p.block_size);
  };

  // A warp's task: 32 entries of the block lists, or 32 times one or four
  // entries of the token maps (four: prompts, whose tokens share blocks and
  // are stored 16 bytes at a time; one: frames, whose tokens would be looked up
  // one after the other).  Nothing that is read here is written here.
  const int64_t moves = static_cast<int64_t>(released) + n_given;
  const int64_t move_tasks = (moves + 31) / 32;
  const int per_task = 32 * p.per_lane;
  const int64_t tasks = move_tasks + (static_cast<int64_t>(p.max_tokens) + per_task - 1) / per_task;
  const int64_t step = static_cast<int64_t>(gridDim.x) * (nt >> 5);
  // the blocks' warps side by side: a block's own tasks are spread over all
  for (int64_t task = static_cast<int64_t>(t >> 5) * gridDim.x + blockIdx.x; task < tasks; task += step) {
    if (task < move_tasks) {
      const int64_t x = task * 32 + (t & 31);
      if (x < released) {
        p.free_blocks[free0 + x] = *released_at(static_cast<int32_t>(x));
      } else if (x < moves) {
        const int32_t y = static_cast<int32_t>(x - released);
        const int r = last_start(blk_start, n, y);
        p.block_table[r * p.table_stride + held_of(len_of[r]) + (y - blk_start[r])] = *stack_at(top - 1 - y);
      }
      continue;
    }
    const int64_t x0 = (task - move_tasks) * per_task + p.per_lane * (t & 31);
    if (x0 >= p.max_tokens) continue;
    const int32_t y0 = static_cast<int32_t>(x0);
    int64_t slot[4];
    int32_t pos[4], of[4];
    const int m = static_cast<int>(min(static_cast<int64_t>(p.per_lane), p.max_tokens - x0));
    int r0 = 0;
    if (m == 1) {
      map_token(y0, r0, slot[0], pos[0], of[0]);
      p.slots[x0] = slot[0];
      if (p.positions) p.positions[x0] = pos[0];
      if (p.requests) p.requests[x0] = of[0];
      continue;
    }
    r0 = y0 < n_tokens ? last_start(tok_start, n, y0) : n - 1;
    const int32_t p0 = y0 < n_tokens ? len_of[r0] + (y0 - tok_start[r0]) : 0;
    const int32_t b0 = static_cast<int32_t>(p.by_block.div(static_cast<uint32_t>(p0)));
    const int32_t off0 = p0 - b0 * p.block_size;
    if (tok_start[r0 + 1] - y0 >= 4 && off0 + 4 <= p.block_size) {  // four tokens of one block
      const int64_t s = slot_of(*block_at(r0, b0, held_of(len_of[r0])), off0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        slot[i] = s < 0 ? -1 : s + i;
        pos[i] = p0 + i;
        of[i] = r0;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) map_token(y0 + i, r0, slot[i], pos[i], of[i]);
    }
    if (p.wide_maps && m == 4) {
      reinterpret_cast<longlong2 *>(p.slots + x0)[0] = make_longlong2(slot[0], slot[1]);
      reinterpret_cast<longlong2 *>(p.slots + x0)[1] = make_longlong2(slot[2], slot[3]);
      if (p.positions) *reinterpret_cast<int4 *>(p.positions + x0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
      if (p.requests) *reinterpret_cast<int4 *>(p.requests + x0) = make_int4(of[0], of[1], of[2], of[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i >= m) continue;
        p.slots[x0 + i] = slot[i];
        if (p.positions) p.positions[x0 + i] = pos[i];
        if (p.requests) p.requests[x0 + i] = of[i];
      }
    }
  }
  if (bits) atomicOr(p.status, bits);
}

// The end of an update in place by several blocks: the new lengths and the
// free count go from the scratch array to their places.
__global__ void kv_tables_store_kernel(const int32_t *lens_new, int32_t *lens, int32_t n,
                                       const int32_t *free_new, int32_t *n_free) {
  pdl_wait_and_release();
  const int i = static_cast<int>(blockIdx.x * blockDim.x + threadIdx.x);
  if (lens && i < n) lens[i] = lens_new[i];
  if (n_free && i == 0) *n_free = *free_new;
}

// --------------------------------------------------------------------------
// Writing new tokens' keys and values
// --------------------------------------------------------------------------
constexpr int kAppendThreads = 256;
// Units per thread and round: 4 of 16 bytes, one of the 32 or 64 bytes that make
// 16 e4m3 values (five CTAs per SM then hide what their arithmetic takes: 65 us
// for 65,536 tokens of 8 x 128 bf16, against 80 with two units and two CTAs;
// three CTAs for the others: 41 us for 32,768 tokens, 46 with two or five).  fp32
// tokens for an e4m3 cache hold twice the words and spill about 100 bytes a thread
// at five CTAs: 63.6 us for 32,768 tokens, 49.4 at the rate of DRAM.
template <class Src, int VEC>
constexpr int kAppendUnroll = sizeof(Src) * VEC == 16 ? 4 : 1;

struct KvAppendParams {
  const void *src[2];               // K and V of the new tokens
  int64_t src_token[2], src_head[2];  // strides in elements
  void *dst[2];
  int64_t dst_block[2], dst_token[2], dst_head[2];
  const float *scale[2];            // one per key head, null: 1 (e4m3 only)
  const int64_t *slots;
  const int32_t *rows;              // ROWS kernels only
  int32_t n_rows;
  int64_t n_slots;                  // n_blocks * block_size
  int64_t block_size;
  int32_t n_tokens;
  int32_t heads;
  int32_t tokens_per_block;         // CTA
  FastDiv by_block, by_token, by_head;        // units of VEC elements per token, per head
  uint32_t *status;
};

// Sixteen e4m3 values of 16 quotients.
__device__ __forceinline__ uint4 e4m3x16_of(const float (&y)[16]) {
  uint32_t o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_fp8x2_storage_t lo =
        __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i], y[4 * i + 1]), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi =
        __nv_cvt_float2_to_fp8x2(make_float2(y[4 * i + 2], y[4 * i + 3]), __NV_SATFINITE, __NV_E4M3);
    o[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// The rare values by division (out of line: the common ones keep the
// instruction cache).
__device__ __noinline__ uint4 divided_e4m3x16(const float *x, float scale) {
  float y[16];
#pragma unroll 1
  for (int i = 0; i < 16; ++i) y[i] = __fdiv_rn(x[i], scale);
  return e4m3x16_of(y);
}

// Eight or sixteen elements as they are stored.
template <class Src, class Dst, int VEC, bool WIDE>
struct AppendUnit {
  static constexpr int kWords = VEC * static_cast<int>(sizeof(Src)) / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const Src *p) {
    if constexpr (WIDE) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
        w[4 * i] = v.x;
        w[4 * i + 1] = v.y;
        w[4 * i + 2] = v.z;
        w[4 * i + 3] = v.w;
      }
    } else {
      // element by element
      Src e[VEC];
#pragma unroll
      for (int i = 0; i < VEC; ++i) e[i] = p[i];
      memcpy(w, e, sizeof w);
    }
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (sizeof(Src) == 2)
      return __uint_as_float((i & 1) ? (w[i / 2] & 0xFFFF0000u) : (w[i / 2] << 16));
    else
      return __uint_as_float(w[i]);
  }
  // `inv`: 1 / scale, or 0 where it does not serve (see quotient)
  __device__ __forceinline__ void store(Dst *p, float scale, float inv) const {
    if constexpr (sizeof(Src) == sizeof(Dst)) {
#pragma unroll
      for (int i = 0; i < kWords / 4; ++i)
        reinterpret_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
      // x / scale in 32 bits, then the nearest e4m3 value (ties to even, at
      // most 448 in size): the only rounding to 8 bits
      static_assert(VEC == 16, "sixteen 8-bit values per 16-byte store");
      float y[16];
      bool fine = inv != 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) fine &= quotient(at(i), scale, inv, y[i]);
      uint4 o = e4m3x16_of(y);
      if (!fine) {
        float x[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = at(i);
        o = divided_e4m3x16(x, scale);
      }
      *reinterpret_cast<uint4 *>(p) = o;
    }
  }
};

// A thread moves a few units of VEC elements, each of K and of V, so that four to
// eight 16-byte loads are in flight; a CTA takes whole tokens.  A skipped
// token's rows are not read.  Bound by DRAM: each element is read once and
// written once.
// ROWS: token x is row rows[x] (its own kernel: the look-up would slow the
// other by a tenth).
template <class Src, class Dst, int VEC, bool WIDE, bool ROWS>
__global__ void __launch_bounds__(kAppendThreads, sizeof(Dst) == 1 ? 5 : 3) kv_append_kernel(const KvAppendParams p) {
  constexpr int kUnroll = kAppendUnroll<Src, VEC>;
  pdl_wait_and_release();
  const int32_t t0 = static_cast<int32_t>(blockIdx.x) * p.tokens_per_block;
  const int32_t nt = min(p.tokens_per_block, p.n_tokens - t0);
  const uint32_t units = static_cast<uint32_t>(nt) * p.by_token.d;
  uint32_t bits = 0;
  for (uint32_t u0 = threadIdx.x; u0 < units; u0 += kAppendThreads * kUnroll) {
    AppendUnit<Src, Dst, VEC, WIDE> k[kUnroll], v[kUnroll];
    int64_t slot[kUnroll];
    int32_t from[ROWS ? kUnroll : 1];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const uint32_t u = u0 + j * kAppendThreads;
      const uint32_t x = t0 + p.by_token.div(u);
      slot[j] = u < units ? p.slots[x] : -1;
      if constexpr (ROWS) from[j] = u < units ? p.rows[x] : 0;
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      bool bad = slot[j] >= p.n_slots;
      if constexpr (ROWS) bad |= slot[j] >= 0 && (from[j] < 0 || from[j] >= p.n_rows);
      if (bad) {
        bits |= kRowBadSlot;
        slot[j] = -1;
      }
      if (slot[j] >= 0) {
        const uint32_t u = u0 + j * kAppendThreads;
        const uint32_t t = p.by_token.div(u), in = u - t * p.by_token.d;
        const uint32_t h = p.by_head.div(in), e = (in - h * p.by_head.d) * VEC;
        int64_t token = t0 + static_cast<int64_t>(t);
        if constexpr (ROWS) token = from[j];
        k[j].load(static_cast<const Src *>(p.src[0]) + token * p.src_token[0] + h * p.src_head[0] + e);
        v[j].load(static_cast<const Src *>(p.src[1]) + token * p.src_token[1] + h * p.src_head[1] + e);
      }
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      if (slot[j] >= 0) {
        const uint32_t u = u0 + j * kAppendThreads;
        const uint32_t in = u - p.by_token.div(u) * p.by_token.d;
        const uint32_t h = p.by_head.div(in), e = (in - h * p.by_head.d) * VEC;
        // a cache of 2^31 slots and more takes the 64-bit division
        const int64_t blk = p.n_slots <= 0x7FFFFFFF
                                ? static_cast<int64_t>(p.by_block.div(static_cast<uint32_t>(slot[j])))
                                : slot[j] / p.block_size;
        const int64_t off = slot[j] - blk * p.block_size;
        Dst *kd = static_cast<Dst *>(p.dst[0]) + blk * p.dst_block[0] + off * p.dst_token[0] + h * p.dst_head[0] + e;
        Dst *vd = static_cast<Dst *>(p.dst[1]) + blk * p.dst_block[1] + off * p.dst_token[1] + h * p.dst_head[1] + e;
        float scale[2] = {1.0f, 1.0f}, inv[2] = {1.0f, 1.0f};
        if constexpr (sizeof(Dst) == 1) {
#pragma unroll
          for (int s = 0; s < 2; ++s)
            if (p.scale[s]) {
              scale[s] = p.scale[s][h];
              inv[s] = quotient_inverse(scale[s]);
            }
        }
        k[j].store(kd, scale[0], inv[0]);
        v[j].store(vd, scale[1], inv[1]);
      }
    }
  }
  if (bits) atomicOr(p.status, bits);
}

}  // namespace ts
