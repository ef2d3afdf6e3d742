// ts_paged_kernels.h -- the paged attention kernels, one translation unit per
// type of cache (they compile side by side).
#pragma once

#include <cstdint>

namespace ts_host {

struct PagedKernel {
  const void *fn;
  uint32_t smem;
  int threads;
  int tile;       // tokens
  int occupancy;  // CTAs per SM (ts_kv.cu fills it in)
};

// kind 0, 1: bf16 cache with up to 8 or 16 query heads per item, 2, 3: e4m3, 4
// .. 7: f32 with up to 1, 2, 4 or 8; width 0 .. 4: up to 64, 96, 128, 192 or 256
// elements per row (the widths between cost code and save what wider ones pad: 24
// masked fp32 requests with rows of 80, 47 us against 53 with room for 128).
PagedKernel paged_kernel_bf16(int kind, int width, bool page16);
PagedKernel paged_kernel_e4m3(int kind, int width, bool page16);
PagedKernel paged_kernel_f32(int kind, int width, bool page16);

}  // namespace ts_host
