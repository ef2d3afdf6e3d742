// ts_kv_common.cuh -- what the paged cache's kernels share: status bits and the
// division by a block size.
#pragma once

#include "ts_device.cuh"

namespace ts {

constexpr uint32_t kRowBadBlock = 32u;
constexpr uint32_t kRowNoBlocks = 64u;

// n / d for 0 <= n < 2^31 by a multiplication: with l = ceil(log2 d) and
// mul = floor(2^(31 + l) / d) + 1, n * mul / 2^(31 + l) exceeds n / d by less
// than 2^-l <= 1 / d, so its floor is the quotient.
struct FastDiv {
  uint32_t d, mul, shift;
  __host__ static FastDiv of(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    FastDiv f;
    f.d = d;
    f.mul = static_cast<uint32_t>((1ull << (31 + l)) / d + 1);
    f.shift = 31 + l;
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return static_cast<uint32_t>((static_cast<uint64_t>(n) * mul) >> shift);
  }
};

}  // namespace ts
