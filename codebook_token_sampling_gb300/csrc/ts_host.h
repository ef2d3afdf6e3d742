// ts_host.h -- what the translation units of the C ABI share on the host side:
// the sampler handle and the report of a failed CUDA call.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "../../include/ts_sampler.h"

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
};

namespace ts_host {

// Keeps the error's text for ts_last_error and returns TS_ERR_CUDA.
ts_status cuda_fail(cudaError_t e, const char *what);

// Frees the paged cache's workspace (the device is current).
cudaError_t kv_free(ts_sampler *s);

}  // namespace ts_host
