// ts_paged_kernels.cuh -- what the translation units of the paged attention
// kernels share.
#pragma once

#include "ts_paged.cuh"
#include "ts_paged_kernels.h"

namespace ts_host {

// Stages per warp.  Two, and twelve warps per SM, beat three and eight wherever
// the registers allow (128 requests of up to 8000 tokens, bf16, 8 x 4 heads of
// 128: 310 against 321 us; 24 of up to 3001, fp32, 8 x 8 heads: 86 against 102).
// Sixteen query heads of 128 leave room for eight warps: three.
template <class Core>
constexpr int stages_of() {
  return !Core::kFma && Core::kRows > 8 && Core::kDim == 128 ? 3 : 2;
}

template <class Core>
PagedKernel paged_kernel(bool page16) {
  constexpr int ns = stages_of<Core>();
  static_assert(ts::PagedShape<Core, ns>::kSmem <= 226 * 1024, "shared memory of a CTA");
  return {page16 ? reinterpret_cast<const void *>(ts::paged_attention_kernel<Core, ns, true>)
                 : reinterpret_cast<const void *>(ts::paged_attention_kernel<Core, ns, false>),
          ts::PagedShape<Core, ns>::kSmem, ts::PagedShape<Core, ns>::kThreads,
          ts::PagedShape<Core, ns>::kTile, 0};
}

// F::make<DP>(kind, page16) for the row's width.
template <class F>
PagedKernel paged_by_width(int kind, int width, bool page16) {
  switch (width) {
    case 0: return F::template make<64>(kind, page16);
    case 1: return F::template make<96>(kind, page16);
    case 2: return F::template make<128>(kind, page16);
    case 3: return F::template make<192>(kind, page16);
    default: return F::template make<256>(kind, page16);
  }
}

}  // namespace ts_host
