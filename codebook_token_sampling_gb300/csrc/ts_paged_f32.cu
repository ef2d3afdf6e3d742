// ts_paged_f32.cu -- the paged attention kernels of fp32 caches.
#include "ts_paged_kernels.cuh"

namespace ts_host {

namespace {

struct Make {
  template <int DP>
  static PagedKernel make(int kind, bool page16) {
    switch (kind) {
      case 4: return paged_kernel<ts::FmaCore<1, DP>>(page16);
      case 5: return paged_kernel<ts::FmaCore<2, DP>>(page16);
      case 6: return paged_kernel<ts::FmaCore<4, DP>>(page16);
      default: return paged_kernel<ts::FmaCore<8, DP>>(page16);
    }
  }
};

}  // namespace

PagedKernel paged_kernel_f32(int kind, int width, bool page16) {
  return paged_by_width<Make>(kind, width, page16);
}

}  // namespace ts_host
