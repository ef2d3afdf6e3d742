// ts_paged_bf16.cu -- the paged attention kernels of bf16 caches.
#include "ts_paged_kernels.cuh"

namespace ts_host {

namespace {

struct Make {
  template <int DP>
  static PagedKernel make(int kind, bool page16) {
    // a step takes 4 KB of keys, or 16 tokens
    constexpr int kt = DP <= 64 ? 2 : 1;
    return kind == 0 ? paged_kernel<ts::MmaCore<false, DP, 1, kt>>(page16)
                     : paged_kernel<ts::MmaCore<false, DP, 2, kt>>(page16);
  }
};

}  // namespace

PagedKernel paged_kernel_bf16(int kind, int width, bool page16) {
  return paged_by_width<Make>(kind, width, page16);
}

}  // namespace ts_host
