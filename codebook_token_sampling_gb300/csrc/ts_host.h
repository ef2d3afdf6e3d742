// ts_host.h -- what the translation units of the C ABI share on the host side:
// the sampler handle and the report of a failed CUDA call.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ts_sampler.h"
#include "ts_overlap.h"

struct ts_sampler {
  int device;
  int cap;
  int num_sms;
  int force_path;     // 0 auto, 1 warps per row, 2 CTA/cluster per row, 3 wide cluster, 4 split
  int force_cluster;  // 0 auto, else CTAs per row
  int pdl;            // launch with programmatic stream serialization
  int wide_exact;     // wide path: always take the exact path (testing)
  int force_wpr;      // warp-per-row path: 0 auto, else warps per row (1, 2, 4)
  int fail_launch;    // tests: the split path's launch of this index (2 or 3) fails once
  uint32_t *status;   // device word (first of two: the status word, then the ticket)
  uint32_t *ticket;   // the warp path's fused step advance: blocks done so far
  int occ_warp[2][5][3];  // resident blocks per SM of each warp-path variant
  int occ_seg[2];         // of the segmented 16-column, one-warp-per-row variant
  int occ_seg32;          // of the fp32 32-column variant (16 columns staged at a time)
  void *ws;           // split wide path workspace (ts_reserve), or null
  size_t ws_bytes;
  int ws_rows;        // row records it holds
  int ws_units;       // unit records it holds
  int ws_vocab;       // widest row it was sized for
  struct ts_kv_state *kv;  // the paged cache's workspace (ts_reserve_kv), or null
  int kv_ctas;        // paged attention: 0 auto, else its number of CTAs (testing)
  int kv_join;        // 0 auto, 1 joins by a launch of their own, 2 by the last CTA (testing)
  bool linear_ready;  // ts_linear_e4m3: its set-up succeeded
  int linear_clusters[5][4];  // ts_linear_e4m3: clusters of 1, 2, 4 and 8 CTAs of each kernel
                              // that the GPU holds at once
  int linear_path;    // ts_linear_e4m3: 0 auto, else its kernel (testing)
  int linear_lose;    // ts_linear_e4m3: 0, else one past the block whose copies get lost (testing)
  int linear_split;   // ts_linear_e4m3: 0 auto, else the CTAs that share a tile (testing)
};

namespace ts_host {

// Keeps the error's text for ts_last_error and returns TS_ERR_CUDA.
ts_status cuda_fail(cudaError_t e, const char *what);

// Frees the paged cache's workspace (the device is current).
cudaError_t kv_free(ts_sampler *s);

// Once per ts_create, on the current device: what ts_linear_e4m3 needs of it, or that it
// cannot be had.
void linear_setup(ts_sampler *s);

// One launch, with programmatic dependent launch if `pdl`.
cudaError_t launch(const void *fn, dim3 grid, dim3 block, size_t smem, bool pdl, cudaStream_t st, void **args);

inline int size_of(int dtype) { return dtype == TS_DTYPE_F32 ? 4 : dtype == TS_DTYPE_BF16 ? 2 : 1; }
inline bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// A cache write's sizes, strides and types (ts_kv_append), then its arrays.
ts_status check_append(const ts_kv_cache *c, const ts_kv_tokens *t);
ts_status check_append_arrays(const ts_kv_tokens *t);

}  // namespace ts_host
