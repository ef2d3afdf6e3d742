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
  int32_t tiles_n;    // of 128 weight rows
  int32_t split;      // CTAs of a cluster that share a tile along in_dim
  uint32_t *status;
};

// Few rows: 128 weight rows are the product's rows and TN tokens its columns, so a
// tile costs no more columns than there are tokens (sixteen at least).  A tensor-copy
// warp streams stages of one block of 128 along in_dim (weights and tokens, 128 bytes
// a row, swizzled) through a ring; one thread of another warp issues a stage's four
// products into one of four accumulators in TMEM; four warps add each block's sums,
// times its scales, to fp32 sums in registers (row = lane).  CTAs of a cluster may
// share a tile along in_dim; their sums are added in rank order through shared memory.
template <int TN>
struct FewTile {
  static constexpr int kStageA = 128 * 128, kStageB = TN * 128;
  static constexpr int kStages = TN == 16 ? 11 : TN == 32 ? 10 : TN == 64 ? 8 : 6;
  static constexpr int kBuffers = 4;
  static constexpr uint32_t kColumns = kBuffers * TN;  // of TMEM: a power of two, 32 at least
  static constexpr uint32_t kSmemBytes = kStages * (kStageA + kStageB) + 1024;
};
constexpr int kFewThreads = 192;

template <int TN>
__global__ void __launch_bounds__(kFewThreads, 1)
    linear_few_kernel(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
                      const LinearParams p) {
  using Tile = FewTile<TN>;
  constexpr int NS = Tile::kStages, NB = Tile::kBuffers;
  constexpr int kPer = (TN + 31) / 32;  // tokens whose scales a lane fetches
  extern __shared__ unsigned char linear_smem[];
  __shared__ __align__(8) uint64_t bars[2 * NS + 2 * NB + 1];
  __shared__ __align__(16) float scales[4][2][TN];
  __shared__ uint32_t tmem_base;
  __shared__ int gave_up;
  const int t = static_cast<int>(threadIdx.x), lane = t & 31, warp = t >> 5;
  unsigned char *ring =
      reinterpret_cast<unsigned char *>((reinterpret_cast<uintptr_t>(linear_smem) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t full = smem_addr(bars), empty = full + 8 * NS, summed = empty + 8 * NS, taken = summed + 8 * NB;
  const uint32_t done = taken + 8 * NB;
  const auto stalled = [&]() { return *static_cast<volatile int *>(&gave_up) != 0; };

  const int rank = p.split > 1 ? static_cast<int>(cluster_rank()) : 0;
  const int tile = static_cast<int>(blockIdx.x);
  const int tile_m = tile / p.tiles_n, tile_n = tile - tile_m * p.tiles_n;
  const int32_t n0 = tile_n * 128, m0 = tile_m * TN;
  const int b0 = static_cast<int>(static_cast<int64_t>(p.blocks) * rank / p.split);
  const int nb = static_cast<int>(static_cast<int64_t>(p.blocks) * (rank + 1) / p.split) - b0;

  if (warp == 5) {
    if (lane == 0) {
      for (int i = 0; i < NS; ++i) {
        mbar_init(full + 8 * i, 1);
        mbar_init(empty + 8 * i, 1);
      }
      for (int i = 0; i < NB; ++i) {
        mbar_init(summed + 8 * i, 1);
        mbar_init(taken + 8 * i, 4);
      }
      mbar_init(done, 1);
      gave_up = 0;
      mbar_init_fence();
    }
    __syncwarp();
    tmem_alloc(smem_addr(&tmem_base), Tile::kColumns);
    tc_fence_before();
  }
  if (warp == 4 && lane == 0) {
    tensor_map_prefetch(&map_w);
    tensor_map_prefetch(&map_x);
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base;
  pdl_wait_and_release();

  float acc[TN];
#pragma unroll
  for (int c = 0; c < TN; ++c) acc[c] = 0.0f;

  if (warp == 4) {
    if (lane == 0) {
      const uint64_t again = l2_evict_normal();
      // weights that no other tile reads leave L2 to the rest
      const uint64_t w_policy = p.n_rows <= TN ? l2_evict_first() : again;
      int i = 0;
      for (; i < nb; ++i) {
        const int s = i % NS;
        if (!mbar_wait(empty + 8 * s, ((i / NS) & 1) ^ 1, &gave_up)) break;
        const uint32_t a = smem_addr(ring) + s * (Tile::kStageA + Tile::kStageB);
        mbar_expect(full + 8 * s, Tile::kStageA + Tile::kStageB);
        tensor_load_2d(a, &map_w, (b0 + i) * 128, n0, full + 8 * s, w_policy);
        tensor_load_2d(a + Tile::kStageA, &map_x, (b0 + i) * 128, m0, full + 8 * s, again);
      }
      if (stalled())
        for (int j = max(0, i - NS); j < i; ++j) mbar_drain(full + 8 * (j % NS), (j / NS) & 1);
    }
  } else if (warp == 5) {
    if (lane == 0) {
      constexpr uint32_t kind = e4m3_product(TN);
      for (int i = 0; i < nb; ++i) {
        const int s = i % NS, b = i % NB;
        if (!mbar_wait(taken + 8 * b, ((i / NB) & 1) ^ 1, &gave_up)) break;
        if (!mbar_wait(full + 8 * s, (i / NS) & 1, &gave_up)) break;
        tc_fence_after();
        const uint32_t a = smem_addr(ring) + s * (Tile::kStageA + Tile::kStageB);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_e4m3(tmem + b * TN, operand_of(a + 32 * k), operand_of(a + Tile::kStageA + 32 * k), kind, k > 0);
        mma_commit(empty + 8 * s);
        mma_commit(summed + 8 * b);
      }
      if (stalled()) {
        mma_commit(done);
        mbar_drain(done, 0);
      }
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
    bool fine = true;
    for (int i0 = 0; i0 < nb && fine; i0 += 4) {
      float now[4][kPer];
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int q = 0; q < kPer; ++q) now[u][q] = xs[u][q] * ws[u];
      fetch(i0 + 4);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + u, b = i % NB;
        if (i >= nb || !fine) continue;
        float *sc = scales[warp][i & 1];
#pragma unroll
        for (int q = 0; q < kPer; ++q)
          if (lane + 32 * q < TN) sc[lane + 32 * q] = now[u][q];
        __syncwarp();
        fine = mbar_wait(summed + 8 * b, (i / NB) & 1, &gave_up);
        fine = __all_sync(0xFFFFFFFFu, fine);
        if (!fine) continue;
        tc_fence_after();
        constexpr int C = TN < 32 ? 16 : 32;
#pragma unroll
        for (int c0 = 0; c0 < TN; c0 += C) {
          float v[C];
          tmem_load(tmem + (static_cast<uint32_t>(warp * 32) << 16) + b * TN + c0, v);
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

}  // namespace ts
