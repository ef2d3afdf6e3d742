// ts_linear.cuh -- the product of 8-bit rows and 8-bit weights with a scale for each
// block of 128 (ts_linear_e4m3):
//   out[m][n] = sum_b xs[m][b] ws[n / 128][b] sum_{k in b} x[m][k] w[n][k].
#pragma once

#include "ts_rows.cuh"
#include "ts_tcgen05.cuh"

namespace ts {

constexpr uint32_t kRowStalled = 128u;

struct LinearParams {
  const float *x_scale, *w_scale;
  int64_t x_scale_stride, w_scale_stride, out_stride;
  void *out;
  int32_t out_f32, n_rows, out_dim;
  int32_t blocks;     // of 128 along in_dim
  int32_t tiles_n;    // tiles along the weight rows
  int32_t split;      // CTAs of a cluster that share a tile along in_dim
  int32_t tiles_m, tiles;  // tiles along the rows, and all (linear_rows_kernel, as the next)
  int32_t columns;    // weight rows of a tile
  int32_t wide_out;   // out's rows can be stored in pieces of 16 bytes
  int32_t wide_scales;  // x_scale's rows can be read in such pieces
  uint32_t wait_cycles;  // of a wait at most
  int32_t lose;       // tests: the block whose copies the first tile never gets, or -1
  uint32_t *status;
};

// Few rows: 128 weight rows are the product's rows and TN tokens its columns, so a
// tile costs no more columns than there are tokens (sixteen at least).  A tensor-copy
// warp streams stages of one block of 128 along in_dim (weights and tokens, 128 bytes
// a row, swizzled) through a ring; a warp issues a stage's four products into an
// accumulator in TMEM; four warps add a group of blocks' sums at a time, times their
// scales, to fp32 sums in registers (row = lane).  CTAs of a cluster may share a tile
// along in_dim; their sums are added in rank order through shared memory.
// Two CTAs to an SM: half of its TMEM each, so that both always get theirs, and a ring
// of which two fit and three do not.  Bound by latency (launch, tensor maps, the first
// copies, the cluster's sums: 32 x 4096 x 1024 4.3 us) and, with enough tiles, by what a
// CTA's chain of copies, products and sums takes for a block, about 250 ns (16 x 11,008 x
// 4096: 11 us for 45 MB).  Other tiles: 64 or 32 weight rows would read the tokens more
// often; eight CTAs a cluster are 1 us slower than four.
template <int TN>
struct FewTile {
  static constexpr int kStageA = 128 * 128, kStageB = TN * 128;
  static constexpr int kStages = TN == 64 ? 4 : 5;
  static constexpr int kGroup = TN == 64 ? 2 : 4;  // blocks that the warps are told of at once
  static constexpr int kBuffers = 2;  // of a group's accumulators
  static constexpr uint32_t kColumns = kBuffers * kGroup * TN;  // of TMEM: a power of two
  static constexpr uint32_t kSmemBytes = kStages * (kStageA + kStageB) + 1024;
  static_assert(kColumns >= 32 && kColumns <= 256, "half of TMEM at most");
  static_assert(kSmemBytes > 76 * 1024 && kSmemBytes < 110 * 1024, "two CTAs to an SM");
};
constexpr int kFewThreads = 192;

template <int TN>
__global__ void __launch_bounds__(kFewThreads, 2)
    linear_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                      const LinearParams p) {
  using Tile = FewTile<TN>;
  constexpr int NS = Tile::kStages, NB = Tile::kBuffers, G = Tile::kGroup;
  constexpr int kPer = (TN + 31) / 32;  // tokens whose scales a lane fetches
  extern __shared__ unsigned char linear_smem[];
  __shared__ __align__(8) uint64_t bars[2 * NS + 2 * NB + 1];
  __shared__ __align__(16) float scales[4][4][TN];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  const int t = static_cast<int>(threadIdx.x), lane = t & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, t >> 5, 0);  // known to be the same in all lanes
  unsigned char *ring =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(linear_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t full = smem_addr(bars), empty = full + 8 * NS, summed = empty + 8 * NS, taken = summed + 8 * NB;
  const uint32_t done = taken + 8 * NB;
  const auto stalled = [&]() { return *static_cast<volatile int *>(&gave_up) != 0; };

  const int rank = p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = static_cast<int>(blockIdx.x) / p.split;
  const int tile_m = tile / p.tiles_n, tile_n = tile - tile_m * p.tiles_n;
  const int32_t n0 = tile_n * 128, m0 = tile_m * TN;
  const int b0 = static_cast<int>(static_cast<int64_t>(p.blocks) * rank / p.split);
  const int nb = static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / p.split) - b0;

  if (warp == 5) {
    tmem_alloc(smem_addr(&tmem_base), Tile::kColumns);
    tc_fence_before();
  } else if (warp == 4) {
    if (lane == 0) {
      tensor_map_prefetch(&map_w);
      tensor_map_prefetch(&map_x);
    }
  } else if (warp == 0) {  // a lane a barrier
    if (lane < 2 * (NS + NB) + 1) mbar_init(full + 8 * lane, lane >= 2 * NS + NB && lane < 2 * (NS + NB) ? 4 : 1);
    if (lane == 0) gave_up = 0;
    mbar_init_fence();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_wait_and_release();

  float acc[TN];
#pragma unroll
  for (int c = 0; c < TN; ++c) acc[c] = 0.0f;

  if (warp == 4) {
    const uint64_t again = l2_evict_normal();
    // weights that no other tile reads leave L2 to the rest
    const uint64_t w_policy = p.n_rows <= TN ? l2_evict_first() : again;
    const int lose = tile == 0 ? p.lose - b0 : -1;
    int s = 0, issued = 0;
    uint32_t phase = 1;
    for (int i = 0; i < nb; ++i) {
      mbar_wait(empty + 8 * s, phase, &gave_up, p.wait_cycles);
      const bool go = !stalled();
      issued += go;
      if (elected() && go && i != lose) {
        const uint32_t a = smem_addr(ring) + s * (Tile::kStageA + Tile::kStageB), bar = full + 8 * s;
        mbar_expect(bar, Tile::kStageA + Tile::kStageB);
        tensor_load_2d(a, &map_w, (b0 + i) * 128, n0, bar, w_policy);
        tensor_load_2d(a + Tile::kStageA, &map_x, (b0 + i) * 128, m0, bar, again);
      }
      __syncwarp();
      if (++s == NS) s = 0, phase ^= 1;
    }
    if (elected() && stalled())
      for (int j = max(0, issued - NS); j < issued; ++j) mbar_drain(full + 8 * (j % NS), (j / NS) & 1, p.wait_cycles);
  } else if (warp == 5) {
    constexpr uint32_t kind = e4m3_product(128, TN);
    const uint64_t ring_a = operand_of(smem_addr(ring)), ring_b = operand_of(smem_addr(ring) + Tile::kStageA);
    int s = 0, b = 0;
    uint32_t s_phase = 0, b_phase = 1;
    for (int g = 0; g < nb; g += G) {
      mbar_wait(taken + 8 * b, b_phase, &gave_up, p.wait_cycles);
      const int count = min(G, nb - g);
      for (int u = 0; u < count; ++u) {
        mbar_wait(full + 8 * s, s_phase, &gave_up, p.wait_cycles);
        tc_fence_after();
        if (elected()) {
          const uint64_t a = ring_a + s * ((Tile::kStageA + Tile::kStageB) >> 4);
          const uint64_t x = ring_b + s * ((Tile::kStageA + Tile::kStageB) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k) mma_e4m3(tmem + (b * G + u) * TN, a + 2 * k, x + 2 * k, kind, k > 0);
          mma_commit(empty + 8 * s);
          if (u == count - 1) mma_commit(summed + 8 * b);
        }
        __syncwarp();
        if (++s == NS) s = 0, s_phase ^= 1;
      }
      if (++b == NB) b = 0, b_phase ^= 1;
    }
    if (elected() && stalled()) {
      mma_commit(done);
      mbar_drain(done, 0, p.wait_cycles);
    }
  } else {
    // four blocks' scales are fetched while the four before them are used
    float xs[4][kPer], ws[4];
    const auto fetch = [&](int i0) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int b = i0 + u;
        ws[u] = b < nb ? p.w_scale[tile_n * p.w_scale_stride + b0 + b] : 0.0f;
#pragma unroll
        for (int q = 0; q < kPer; ++q) {
          const int32_t c = lane + 32 * q, m = m0 + c;
          xs[u][q] = b < nb && c < TN && m < p.n_rows ? p.x_scale[m * p.x_scale_stride + b0 + b] : 0.0f;
        }
      }
    };
    fetch(0);
    for (int i0 = 0; i0 < nb; i0 += 4) {
      float now[4][kPer];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < kPer; ++q) now[u][q] = xs[u][q] * ws[u];
      fetch(i0 + 4);
      for (int u = 0; u < 4; ++u) {
        float *sc = scales[warp][u];
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          if (lane + 32 * q < TN) sc[lane + 32 * q] = now[u][q];
      }
      __syncwarp();
#pragma unroll
      for (int g = 0; g < 4; g += G) {
        if (i0 + g >= nb) continue;
        const int group = (i0 + g) / G, b = group % NB;
        mbar_wait(summed + 8 * b, (group / NB) & 1, &gave_up, p.wait_cycles);
        tc_fence_after();
#pragma unroll
        for (int u = 0; u < G; ++u) {
          if (i0 + g + u >= nb) continue;
          const float *sc = scales[warp][g + u];
          constexpr int C = TN < 32 ? 16 : 32;
#pragma unroll
          for (int c0 = 0; c0 < TN; c0 += C) {
            float v[C];
            tmem_load(tmem + (static_cast<uint32_t>(warp * 32) << 16) + (b * G + u) * TN + c0, v);
            tmem_load_wait(v);
#pragma unroll
            for (int c = 0; c < C; c += 4) {
              const float4 f = *reinterpret_cast<const float4 *>(sc + c0 + c);
              acc[c0 + c] = fmaf(v[c], f.x, acc[c0 + c]);
              acc[c0 + c + 1] = fmaf(v[c + 1], f.y, acc[c0 + c + 1]);
              acc[c0 + c + 2] = fmaf(v[c + 2], f.z, acc[c0 + c + 2]);
              acc[c0 + c + 3] = fmaf(v[c + 3], f.w, acc[c0 + c + 3]);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(taken + 8 * b);
      }
    }
  }
  __syncwarp();

  const auto store = [&](int32_t n, int32_t m, float v) {
    if (n >= p.out_dim || m >= p.n_rows) return;
    if (p.out_f32) static_cast<float *>(p.out)[m * p.out_stride + n] = v;
    else static_cast<uint16_t *>(p.out)[m * p.out_stride + n] = bf16_of(v);
  };
  if (p.split == 1) {
    if (warp < 4 && !stalled()) {
#pragma unroll
      for (int c = 0; c < TN; ++c) store(n0 + t, m0 + c, acc[c]);
    }
  } else {
    // every product has read the ring: it holds the sums now, a column's 128 rows side by side
    float *sums = reinterpret_cast<float *>(ring);
    if (warp < 4) {
#pragma unroll
      for (int c = 0; c < TN; ++c) sums[c * 128 + t] = acc[c];
    }
    cluster_sync_all();
    uint32_t lost = 0;
    for (int q = 0; q < p.split; ++q) lost |= dsmem_ld_u32(dsmem_addr(&gave_up, q));
    if (warp < 4 && !lost) {
      constexpr int G = 4;  // columns whose sums are on their way at once
      for (int c0 = rank * G; c0 < TN; c0 += p.split * G) {
        float v[G];
#pragma unroll
        for (int c = 0; c < G; ++c) v[c] = 0.0f;
        for (int q = 0; q < p.split; ++q) {
          const uint32_t from = dsmem_addr(sums + c0 * 128 + t, q);
#pragma unroll
          for (int c = 0; c < G; ++c) v[c] += __uint_as_float(dsmem_ld_u32(from + c * 512));
        }
#pragma unroll
        for (int c = 0; c < G; ++c) store(n0 + t, m0 + c0 + c, v[c]);
      }
    }
    cluster_sync_all();  // no CTA leaves while another reads its sums
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 5) tmem_free(tmem, Tile::kColumns);
  if (t == 0 && stalled()) atomicOr(p.status, kRowStalled);
}

// More rows.  8192 x 8192 x 4096: 210 us, 2.6 PFLOP/s by pairs, 229 us repeated for
// seconds under the power cap (732 us with tokens as the
// products' columns, 422 us by single CTAs of 128 columns); bound by the chain from a
// block's products to the answer that its accumulator is free, of which a tile of 256
// columns has two.  128 x 11,008 x 4096: 15 us by 115 CTAs, bound by that chain (250 ns a
// block) and by DRAM.
// 128 tokens are the product's rows and `columns` weight rows (a multiple of
// 32) its columns, so a thread's sums belong to one token and a block's scales are one
// number for 32 of them.  Eight warps add the blocks' sums (a warp: 32 tokens, half of
// the columns), one streams, one issues the products.
// PAIR: two CTAs share a tile of 256 tokens by `columns`: each brings its tokens and
// half of the weights, the first one's thread issues the products of both, and the CTAs
// walk over the tiles; otherwise a CTA (or a cluster along in_dim) has one tile, whose
// tokens and weights it brings by itself: L2 gives about 10 TB/s to all SMs together, which
// bounds a call of 128 tokens before DRAM does.  (The
// pair's block as two products of 128 columns with accumulators and a warpgroup each, to
// add one while the other is multiplied: 328 us instead of 243 for 8192 x 8192 x 4096.)
template <int CH, bool PAIR>
struct RowsTile {
  static constexpr int kMaxColumns = 64 * CH;
  static constexpr int kStageA = 128 * 128, kStageB = (PAIR ? kMaxColumns / 2 : kMaxColumns) * 128;
  static constexpr int kStages = 196608 / (kStageA + kStageB);
  // Blocks that the adding warps are told of at once.  Waits, commits and arrivals cost a
  // block about 500 cycles, as much as its products: a tile of 256 columns has no room for
  // more than two blocks' sums, narrower ones have.
  static constexpr int kGroup = PAIR ? 1 : 2;
  static constexpr int kBuffers = 512 / kMaxColumns / kGroup;
  static constexpr int kStaging = PAIR ? 8 * 32 * 32 * 4 : 0;  // a warp's 32 x 32 outputs
  static constexpr int kPitch = kMaxColumns + 4;               // floats from a tile's row to the next
  static constexpr uint32_t kSmemBytes = kStages * (kStageA + kStageB) + kStaging + 1024;
  static_assert(PAIR || 128 * kPitch * 4 <= kStages * (kStageA + kStageB), "a tile's sums fit the ring");
};
// Three warpgroups: two that add, one of which a warp streams and one issues products.
// Pairs: 384 x 168 registers at launch, 256 x 232 + 128 x 40 from then on.
constexpr int kRowsThreads = 384;

template <int CH, bool PAIR>
__global__ void __launch_bounds__(kRowsThreads, 1)
    linear_rows_kernel(const __grid_constant__ CUtensorMap map_x, const __grid_constant__ CUtensorMap map_w,
                       const LinearParams p) {
  using Tile = RowsTile<CH, PAIR>;
  constexpr int NS = Tile::kStages, NB = Tile::kBuffers, G = Tile::kGroup, kStage = Tile::kStageA + Tile::kStageB;
  extern __shared__ unsigned char linear_smem[];
  __shared__ __align__(8) uint64_t bars[2 * NS + 2 * NB + 1];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  const int t = static_cast<int>(threadIdx.x), lane = t & 31;
  const int warp = __shfl_sync(0xFFFFFFFFu, t >> 5, 0);  // known to be the same in all lanes
  unsigned char *ring =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(linear_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t full = smem_addr(bars), empty = full + 8 * NS, summed = empty + 8 * NS, taken = summed + 8 * NB;
  const uint32_t done = taken + 8 * NB;
  const auto stalled = [&]() { return *static_cast<volatile int *>(&gave_up) != 0; };
  const auto any_stalled = [&]() { return __any_sync(0xFFFFFFFFu, stalled()) != 0; };  // the same in all lanes

  const int shared_by = PAIR ? 2 : p.split;  // CTAs of the cluster
  const int rank = shared_by > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int first = static_cast<int>(blockIdx.x) / shared_by, step = static_cast<int>(gridDim.x) / shared_by;
  const int split = PAIR ? 1 : p.split;
  const int b0 = split == 1 ? 0 : static_cast<int>(static_cast<int64_t>(p.blocks) * rank / split);
  const int nb = split == 1 ? p.blocks : static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / split) - b0;
  // neighbouring tiles share their weights: sixteen tiles of tokens before the next columns
  const auto place = [&](int tile, int32_t &m0, int32_t &n0) {
    const int per = p.tiles_n * 16, group = tile / per, in = tile - group * per;
    const int high = min(16, p.tiles_m - group * 16);
    n0 = in / high * p.columns;
    m0 = (group * 16 + in % high) * (PAIR ? 256 : 128) + (PAIR ? rank * 128 : 0);
  };

  if (warp == 9) {
    tmem_alloc<PAIR>(smem_addr(&tmem_base), 512);
    tc_fence_before();
  } else if (warp == 8) {
    if (lane == 0) {
      tensor_map_prefetch(&map_x);
      tensor_map_prefetch(&map_w);
    }
  } else if (warp == 0) {  // a lane a barrier
    static_assert(2 * (NS + NB) + 1 <= 32, "barriers");
    if (lane < 2 * (NS + NB) + 1) {
      const bool is_taken = lane >= 2 * NS + NB && lane < 2 * (NS + NB);
      mbar_init(full + 8 * lane, is_taken ? (PAIR ? 16 : 8) : 1);
    }
    if (lane == 0) gave_up = 0;
    mbar_init_fence();
  }
  if constexpr (PAIR) cluster_sync_all();  // the other's barriers are there
  else __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_wait_and_release();

  if (warp >= 8) {
    if constexpr (PAIR) registers_less<40>();
    if (warp == 8) {
      const uint64_t policy = l2_evict_normal();
      const uint32_t bytes = (PAIR ? 2 * Tile::kStageA : Tile::kStageA) + static_cast<uint32_t>(p.columns) * 128;
      const uint32_t counted = PAIR ? cluster_addr(full, 0) : full;  // the first CTA counts both CTAs' copies
      int s = 0, issued = 0;
      uint32_t phase = 1;
      for (int tile = first; tile < p.tiles && !any_stalled(); tile += step) {
        const int lose = tile == 0 ? p.lose : -1;
        int32_t m0, n0;
        place(tile, m0, n0);
        const int32_t w0 = n0 + (PAIR ? rank * (p.columns / 2) : 0);
        for (int b = b0; b < b0 + nb; ++b) {
          mbar_wait(empty + 8 * s, phase, &gave_up, p.wait_cycles);
          const bool go = !stalled();
          issued += go;
          if (elected() && go && b != lose) {
            const uint32_t a = smem_addr(ring) + s * kStage;
            if (rank == 0 || !PAIR) mbar_expect(full + 8 * s, bytes);
            if constexpr (PAIR) {
              tensor_load_2d_pair(a, &map_x, b * 128, m0, counted + 8 * s, policy);
              tensor_load_2d_pair(a + Tile::kStageA, &map_w, b * 128, w0, counted + 8 * s, policy);
            } else {
              tensor_load_2d(a, &map_x, b * 128, m0, counted + 8 * s, policy);
              tensor_load_2d(a + Tile::kStageA, &map_w, b * 128, w0, counted + 8 * s, policy);
            }
          }
          __syncwarp();
          if (++s == NS) s = 0, phase ^= 1;
        }
      }
      // the last arrivals from the pair's other CTA come before this one leaves
      if constexpr (PAIR)
        for (int j = max(0, issued - NS); j < issued; ++j) mbar_wait(empty + 8 * (j % NS), (j / NS) & 1, &gave_up, p.wait_cycles);
      if (elected() && (rank == 0 || !PAIR) && stalled())
        for (int j = max(0, issued - NS); j < issued; ++j) mbar_drain(full + 8 * (j % NS), (j / NS) & 1, p.wait_cycles);
    }
    if (warp == 9 && (rank == 0 || !PAIR)) {
      const uint32_t kind = e4m3_product(PAIR ? 256 : 128, p.columns);
      const uint64_t ring_a = operand_of(smem_addr(ring)), ring_b = operand_of(smem_addr(ring) + Tile::kStageA);
      int s = 0, buf = 0;
      uint32_t s_phase = 0, buf_phase = 1;
      for (int tile = first; tile < p.tiles && !any_stalled(); tile += step) {
        for (int g = 0; g < nb; g += G) {
          mbar_wait(taken + 8 * buf, buf_phase, &gave_up, p.wait_cycles);
          const int count = G == 1 ? 1 : min(G, nb - g);
          for (int u = 0; u < count; ++u) {
            mbar_wait(full + 8 * s, s_phase, &gave_up, p.wait_cycles);
            tc_fence_after();
            if (elected()) {
              const uint32_t d = tmem + (buf * G + u) * Tile::kMaxColumns;
              const uint64_t a = ring_a + s * (kStage >> 4), w = ring_b + s * (kStage >> 4);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_e4m3<PAIR>(d, a + 2 * k, w + 2 * k, kind, k > 0);
              mma_commit<PAIR>(empty + 8 * s);
              if (u == count - 1) mma_commit<PAIR>(summed + 8 * buf);
            }
            __syncwarp();
            if (++s == NS) s = 0, s_phase ^= 1;
          }
          if (++buf == NB) buf = 0, buf_phase ^= 1;
        }
      }
      if (elected() && stalled()) {
        mma_commit<PAIR>(done);
        mbar_drain(done, 0, p.wait_cycles);
      }
    }
  } else {
    if constexpr (PAIR) registers_more<232>();
    const int quarter = warp & 3, half = warp >> 2;
    const int all = p.columns / 32, c0 = half ? (all + 1) / 2 : 0, chunks = half ? all / 2 : (all + 1) / 2;
    const uint32_t counted = PAIR ? cluster_addr(taken, 0) : taken;
    const int row = quarter * 32 + lane;
    // four blocks' scales are fetched while the four before them are used (registers that
    // moved on with every block would wait for the newest): the row's, and in lane 8 u + j
    // that of the warp's chunk j of the columns in block u
    float xs[4], ws;
    const float *x_from = p.x_scale, *w_from = p.w_scale;
    bool x_there = false, w_there = false, x_wide = false;
    const auto fetch = [&](int i0) {
      if (x_wide && i0 + 4 <= nb) {
        const float4 f = *reinterpret_cast<const float4 *>(x_from + i0);
        xs[0] = f.x, xs[1] = f.y, xs[2] = f.z, xs[3] = f.w;
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) xs[u] = x_there && i0 + u < nb ? x_from[i0 + u] : 0.0f;
      }
      ws = w_there && i0 + (lane >> 3) < nb ? w_from[i0 + (lane >> 3)] : 0.0f;
    };
    const auto release = [&](int buf) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if constexpr (PAIR) mbar_arrive_remote(counted + 8 * buf);
        else mbar_arrive(counted + 8 * buf);
      }
    };
    const auto scales_at = [&](int32_t m0, int32_t n0) {
      const int n = n0 + 32 * (c0 + (lane & 7));
      x_there = m0 + row < p.n_rows;
      x_wide = x_there && p.wide_scales && b0 % 4 == 0;  // a row's four scales by one load
      w_there = (lane & 7) < chunks && n < p.out_dim;
      x_from = p.x_scale + (m0 + row) * p.x_scale_stride + b0;
      w_from = p.w_scale + (n >> 7) * p.w_scale_stride + b0;
      fetch(0);
    };
    int i = 0;
    int32_t m0 = 0, n0 = 0;
    if (first < p.tiles) {
      place(first, m0, n0);
      scales_at(m0, n0);
    }
    for (int tile = first; tile < p.tiles; tile += step) {
      uint64_t acc[CH][16];
#pragma unroll
      for (int j = 0; j < CH; ++j)
#pragma unroll
        for (int c = 0; c < 16; ++c) acc[j][c] = 0;
      for (int g = 0; g < nb; g += 4) {
        float x_now[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) x_now[u] = xs[u];
        const float w_now = ws;
        fetch(g + 4);
#pragma unroll
        for (int u0 = 0; u0 < 4; u0 += G) {
          if (g + u0 >= nb) continue;
          const int buf = i % NB;
          uint64_t scale[G][CH];
#pragma unroll
          for (int u = 0; u < G; ++u)
#pragma unroll
            for (int j = 0; j < CH; ++j) {
              const float f = x_now[u0 + u] * __shfl_sync(0xFFFFFFFFu, w_now, 8 * (u0 + u) + j);
              scale[u][j] = pair_of(f, f);
            }
          mbar_wait(summed + 8 * buf, (i / NB) & 1, &gave_up, p.wait_cycles);
          ++i;
          tc_fence_after();
          const uint32_t from =
              tmem + (static_cast<uint32_t>(quarter * 32) << 16) + buf * G * Tile::kMaxColumns + 32 * c0;
#pragma unroll
          for (int u = 0; u < G; ++u) {
            if (u > 0 && g + u0 + u >= nb) continue;
#pragma unroll
            for (int j = 0; j < CH; ++j) {
              if (j >= chunks) continue;
              float v[32];
              tmem_load(from + u * Tile::kMaxColumns + 32 * j, v);
              tmem_load_wait(v);
              if (PAIR && j == CH - 1) release(buf);  // the last ones have come
#pragma unroll
              for (int c = 0; c < 16; ++c) acc[j][c] = fma2(pair_of(v[2 * c], v[2 * c + 1]), scale[u][j], acc[j][c]);
            }
          }
          if constexpr (!PAIR) release(buf);
        }
      }
      if (any_stalled()) break;
      if constexpr (PAIR) {
        const int32_t m_now = m0, n_now = n0;
        if (tile + step < p.tiles) {
          place(tile + step, m0, n0);
          scales_at(m0, n0);
        }
        // a chunk's 32 x 32 outputs through the warp's own 4 KB, so that rows are stored in
        // segments of 64 or 128 bytes (16-byte columns are swapped by row: no bank twice)
        float4 *staging = reinterpret_cast<float4 *>(ring + NS * kStage) + warp * 256;
        const int32_t m = m_now + quarter * 32;
        const int rows = min(32, p.n_rows - m);
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          if (j >= chunks) continue;
          const int32_t n = n_now + 32 * (c0 + j);
          const bool wide = p.wide_out && n + 32 <= p.out_dim;
          if (wide && !p.out_f32) {
            uint4 *packed = reinterpret_cast<uint4 *>(staging);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float lo, hi;
                parts_of(acc[j][4 * c + e], lo, hi);
                w[e] = bf16x2_of(lo, hi);
              }
              packed[lane * 4 + (c ^ ((lane >> 1) & 3))] = make_uint4(w[0], w[1], w[2], w[3]);
            }
            __syncwarp();
#pragma unroll
            for (int r0 = 0; r0 < 32; r0 += 8) {
              const int r = r0 + (lane >> 2), c = lane & 3;
              if (r < rows)
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(p.out) + (m + r) * p.out_stride + n + 8 * c) =
                    packed[r * 4 + (c ^ ((r >> 1) & 3))];
            }
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              float4 f;
              parts_of(acc[j][2 * c], f.x, f.y);
              parts_of(acc[j][2 * c + 1], f.z, f.w);
              staging[lane * 8 + (c ^ (lane & 7))] = f;
            }
            __syncwarp();
            if (wide) {
#pragma unroll 2
              for (int r0 = 0; r0 < 32; r0 += 4) {
                const int r = r0 + (lane >> 3), c = lane & 7;
                if (r < rows)
                  *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + (m + r) * p.out_stride + n + 4 * c) =
                      staging[r * 8 + (c ^ (r & 7))];
              }
            } else {
#pragma unroll 2
              for (int r = 0; r < rows; ++r) {
                const float f = reinterpret_cast<const float *>(staging)[r * 32 + 4 * ((lane >> 2) ^ (r & 7)) + (lane & 3)];
                if (n + lane < p.out_dim) {
                  if (p.out_f32) static_cast<float *>(p.out)[(m + r) * p.out_stride + n + lane] = f;
                  else static_cast<uint16_t *>(p.out)[(m + r) * p.out_stride + n + lane] = bf16_of(f);
                }
              }
            }
          }
          __syncwarp();
        }
      } else {
        // the tile's products have read the ring: it holds the sums now, row by row
        float *sums = reinterpret_cast<float *>(ring) + row * Tile::kPitch;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
          if (j >= chunks) continue;
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            float4 f;
            parts_of(acc[j][2 * c], f.x, f.y);
            parts_of(acc[j][2 * c + 1], f.z, f.w);
            reinterpret_cast<float4 *>(sums + 32 * (c0 + j))[c] = f;
          }
        }
      }
    }
  }
  __syncwarp();
  if constexpr (!PAIR) {
    if (split > 1) cluster_sync_all();
    else __syncthreads();
    int lost = stalled();
    for (int q = 0; split > 1 && q < split; ++q) lost |= static_cast<int>(dsmem_ld_u32(dsmem_addr(&gave_up, q)));
    if (first < p.tiles && !lost) {
      int32_t m0, n0;
      place(first, m0, n0);
      const float *sums = reinterpret_cast<const float *>(ring);
      // Rows in turn over the warps (of the cluster's CTAs along in_dim, whose sums are
      // added in rank order), lanes along them: four neighbouring sums of a lane where rows
      // lie on 16 bytes, one where they do not, so that stores lie side by side either way.
      constexpr int kWarps = kRowsThreads / 32;
      const int rows = min(128, p.n_rows - m0), w0 = (split > 1 ? rank : 0) * kWarps + warp, warps = kWarps * split;
      if (p.wide_out) {
        const int per_row = p.columns / 4, at_once = 32 / per_row, sub = lane / per_row, c = (lane - sub * per_row) * 4;
#pragma unroll 4
        for (int r0 = w0 * at_once; r0 < rows; r0 += warps * at_once) {
          const int r = r0 + sub;
          if (sub >= at_once || r >= rows) continue;
          float f[4];
          if (split == 1) {
            const float4 v = *reinterpret_cast<const float4 *>(sums + r * Tile::kPitch + c);
            f[0] = v.x, f[1] = v.y, f[2] = v.z, f[3] = v.w;
          } else {
            f[0] = f[1] = f[2] = f[3] = 0.0f;
            uint4 v[8];
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q < split) v[q] = dsmem_ld_v4(dsmem_addr(sums + r * Tile::kPitch + c, q));
#pragma unroll
            for (int q = 0; q < 8; ++q)
              if (q < split) {
                f[0] += __uint_as_float(v[q].x);
                f[1] += __uint_as_float(v[q].y);
                f[2] += __uint_as_float(v[q].z);
                f[3] += __uint_as_float(v[q].w);
              }
          }
          const int32_t n = n0 + c;
          const int64_t at = (m0 + r) * p.out_stride + n;
          if (n + 4 <= p.out_dim) {
            if (p.out_f32) *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = make_float4(f[0], f[1], f[2], f[3]);
            else *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.out) + at) = make_uint2(bf16x2_of(f[0], f[1]), bf16x2_of(f[2], f[3]));
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n + e < p.out_dim) {
                if (p.out_f32) static_cast<float *>(p.out)[at + e] = f[e];
                else static_cast<uint16_t *>(p.out)[at + e] = bf16_of(f[e]);
              }
          }
        }
      } else {
#pragma unroll 2
        for (int r = w0; r < rows; r += warps) {
          const float *at = sums + r * Tile::kPitch + lane;
          float f[2 * CH];
#pragma unroll
          for (int k = 0; k < 2 * CH; ++k) {
            f[k] = 0.0f;
            if (32 * k >= p.columns) continue;
            if (split == 1) {
              f[k] = at[32 * k];
            } else {
              uint32_t v[8];
#pragma unroll
              for (int q = 0; q < 8; ++q)
                if (q < split) v[q] = dsmem_ld_u32(dsmem_addr(at + 32 * k, q));
#pragma unroll
              for (int q = 0; q < 8; ++q)
                if (q < split) f[k] += __uint_as_float(v[q]);
            }
          }
          const int64_t to = (m0 + r) * p.out_stride + n0 + lane;
#pragma unroll
          for (int k = 0; k < 2 * CH; ++k) {
            if (32 * k >= p.columns || n0 + lane + 32 * k >= p.out_dim) continue;
            if (p.out_f32) static_cast<float *>(p.out)[to + 32 * k] = f[k];
            else static_cast<uint16_t *>(p.out)[to + 32 * k] = bf16_of(f[k]);
          }
        }
      }
    }
  }
  tc_fence_before();
  if (shared_by > 1) cluster_sync_all();  // no CTA leaves while another needs its memory
  else __syncthreads();
  tc_fence_after();
  if (warp == 9) tmem_free<PAIR>(tmem, 512);
  if (t == 0 && stalled()) atomicOr(p.status, kRowStalled);
}

}  // namespace ts
