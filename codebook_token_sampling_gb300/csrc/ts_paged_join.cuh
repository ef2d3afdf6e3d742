// ts_paged_join.cuh -- the launch that joins the parts of items spread over many
// CTAs of the paged attention kernel.
#pragma once

#include "ts_paged.cuh"

namespace ts {

// Joins the items that are spread over many CTAs.  Of an item's rows, block
// first + j takes rows j, j + parts, ..: its eight warps share the parts, a
// lane four or eight columns of them, and are added up in shared memory.  Its
// launch waits for all CTAs, which with few parts costs more than the last CTA
// needs to join them (measured: see join_here in ts_kv.cu).
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

__global__ void __launch_bounds__(kJoinThreads) paged_join_kernel(const PagedParams p) {
  __shared__ PagedSum s_sum[kJoinWarps][2][32];
  const int c = static_cast<int>(blockIdx.x);
  const int lane = static_cast<int>(lane_id()), warp = static_cast<int>(threadIdx.x) >> 5;
  pdl_wait_and_release();
  const PagedParts d[2] = {p.parts[2 * static_cast<int64_t>(c)], p.parts[2 * static_cast<int64_t>(c) + 1]};
#pragma unroll 1
  for (int k = 0; k < 2; ++k) {
    if (d[k].parts < 2) continue;
    const int rows = min(p.rows, p.group - d[k].piece * p.rows);
    const int64_t head = static_cast<int64_t>(d[k].head) * p.group + d[k].piece * p.rows;
    for (int row = c - d[k].first; row < rows; row += d[k].parts) {
      for (int h = 0; 4 * lane + 128 * h < p.dim && h < 2; ++h)
        s_sum[warp][h][lane] = join_parts<8>(p, d[k].first, row, 4 * lane + 128 * h, warp, d[k].parts,
                                             kJoinWarps, -1, PagedSum());
      __syncthreads();
      if (warp < 2 && 4 * lane + 128 * warp < p.dim) {
        PagedSum y;
        y.top = s_sum[0][warp][lane].top;
#pragma unroll
        for (int w = 1; w < kJoinWarps; ++w) y.top = fmaxf(y.top, s_sum[w][warp][lane].top);
        y.x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        y.sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) {
          const PagedSum &z = s_sum[w][warp][lane];
          take_in(y, exp2_from(z.top, y.top), z.x, z.sum);
        }
        paged_answer(p, d[k].request, d[k].head, head + row, 4 * lane + 128 * warp, y);
      }
      __syncthreads();
    }
  }
}

}  // namespace ts
