// ts_paged_e4m3.cu -- the paged attention kernels of e4m3 caches.
#include "ts_paged_kernels.cuh"

namespace ts_host {

namespace {

struct Make {
  template <int DP>
  static PagedKernel make(int kind, bool page16) {
    // steps of 32 tokens (57 us, 63 with 16: 16 requests of up to 16,000 tokens, 8
    // x 8 heads of 128), of 16 where 32 leave too few warps
    return kind == 2 ? paged_kernel<ts::MmaCore<true, DP, 1, DP <= 128 ? 2 : 1>>(page16)
                     : paged_kernel<ts::MmaCore<true, DP, 2, 2>>(page16);
  }
};

}  // namespace

PagedKernel paged_kernel_e4m3(int kind, int width, bool page16) {
  return paged_by_width<Make>(kind, width, page16);
}

}  // namespace ts_host
