// ts_linear.cu -- host side of ts_linear_e4m3: argument checks, tensor maps, kernel
// choice and launch on the caller's stream.
#include <algorithm>
#include <cstring>
#include <mutex>
#include <vector>

#include "ts_host.h"
#include "ts_linear.cuh"

static_assert(ts::kRowStalled == TS_ROW_STALLED, "status bits");

namespace {

using ts_host::aligned;
using ts_host::cuda_fail;

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The kernels: tokens as the products' columns (16, 32 or 64), as their rows, and the
// latter by pairs of CTAs.
struct LinearKernel {
  const void *fn;
  uint32_t smem;
  int threads;
};
template <int TN>
LinearKernel few_kernel() {
  return {reinterpret_cast<const void *>(ts::linear_few_kernel<TN>), ts::FewTile<TN>::kSmemBytes, ts::kFewThreads};
}
template <int CH, bool PAIR>
LinearKernel rows_kernel() {
  return {reinterpret_cast<const void *>(ts::linear_rows_kernel<CH, PAIR>), ts::RowsTile<CH, PAIR>::kSmemBytes,
          ts::kRowsThreads};
}
constexpr int kKernels = 5;

// What is the same for all handles (a handle's calls read g_encode only after its own
// linear_setup saw it set).
struct LinearDevice {
  int device, clusters[kKernels][4];
};
std::mutex g_linear_mu;
std::vector<LinearDevice> g_linear_devices;
EncodeTiled g_encode = nullptr;

LinearKernel kernel_for(int i) {
  return i == 0 ? few_kernel<16>() : i == 1 ? few_kernel<32>() : i == 2 ? few_kernel<64>()
       : i == 3 ? rows_kernel<2, false>() : rows_kernel<4, true>();
}

// Rows of bytes in boxes of 128 columns by `box_rows`, swizzled; what lies outside is 0.
bool tensor_map(CUtensorMap *m, const void *p, int64_t columns, int64_t rows, int64_t stride, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, steps[2] = {1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t blocks_of(int64_t dim) { return ceil_div(dim, TS_SCALE_BLOCK); }

// What a call launches: the kernel, its tile (rows of x by weight rows), and the CTAs that
// share one along in_dim.
struct LinearPlan {
  int kernel, rows, columns, split;
};
// How its arrays lie: rows of x and w on whole lines of 128 bytes, rows of out on pieces of 16.
struct Layout {
  bool whole_lines, wide_out;
};

// CTAs of a cluster for `tiles` tiles: as many as leave none waiting for an SM (1 x 4096 x
// 4096: 5.3 us by clusters of four, 6.2 by eight to two CTAs an SM) or for room in a GPC
// (128 x 1024 x 4096: 7.2 us by eleven clusters of eight, 11.8 by sixteen).
int split_for(const ts_sampler *s, int kernel, int64_t tiles, int64_t blocks) {
  int split = 1;
  for (int i = 1; i < 4 && tiles << i <= s->num_sms && tiles <= s->linear_clusters[kernel][i] && (1 << i) <= blocks; ++i)
    split = 1 << i;
  return split;
}

LinearPlan plan_few(const ts_sampler *s, int64_t m, int64_t n, int64_t blocks) {
  LinearPlan plan = {m <= 16 ? 0 : m <= 32 ? 1 : 2, m <= 16 ? 16 : m <= 32 ? 32 : 64, 128, 1};
  plan.split = split_for(s, plan.kernel, ceil_div(n, 128) * ceil_div(m, plan.rows), blocks);
  return plan;
}
// The least cycles by what a tile takes: for each block the chain from its copy to its
// sums (590 for 128 tokens by 96, 1080 for a pair's 256 by 256), or what all CTAs take in
// through L2 together (5000 bytes a cycle; 4000 where rows do not lie on whole lines of 128
// bytes, so that a row's piece is in two of them: 512 x 4096 x 4112 by 128 columns 22 us, by
// pairs 18, x 4096 13.6 and 17); and about 9000 around them, for pairs 7000 more a tile whose
// outputs cannot be stored in pieces of 16 bytes (777 x 2001 x 512 fp32 10.2 us, 5.9 by 96
// columns; x 2048 x 512 6.9 by pairs).  70 sizes of 100 to 3000 rows, 2001 to 11,008 weight
// rows and 512 to 4112 along in_dim: within 6% of the best of 32, 64, 96, 128 columns and
// pairs but for seven, whose best is up to 20% faster.  512 x 4096 x 4096 13.5 us (pairs 17),
// 1024 x 4096 x 4096 17.9 by pairs (26), 777 x 2001 x 1040 fp32 9.6.
LinearPlan plan_rows(const ts_sampler *s, int64_t m, int64_t n, int64_t blocks, const Layout &at, bool pairs) {
  const double pair_waves = static_cast<double>(ceil_div(ceil_div(m, 256) * ceil_div(n, 256), s->linear_clusters[4][1]));
  LinearPlan best = {4, 256, 256, 1};
  double least = pairs ? pair_waves * (blocks * 1080.0 + (at.wide_out ? 0.0 : 7000.0)) + 8000.0 : 1e30;
  for (int columns = 32; columns <= 128; columns += 32) {
    const int64_t tiles = ceil_div(m, 128) * ceil_div(n, columns), held = s->linear_clusters[3][0];
    const int split = split_for(s, 3, tiles, blocks);
    const double waves = static_cast<double>(ceil_div(tiles * split, held));
    const double at_once = static_cast<double>(std::min<int64_t>(tiles * split, held));
    const double block =
        std::max(350.0 + 2.5 * columns, (16384.0 + columns * 128.0) * at_once / (at.whole_lines ? 5000.0 : 4000.0));
    const double cycles = waves * (ceil_div(blocks, split) * block + 5000.0 + 40.0 * columns);
    if (cycles < least) {
      least = cycles;
      best = {3, 128, columns, split};
    }
  }
  return best;
}
LinearPlan plan_for(const ts_sampler *s, int64_t m, int64_t n, int64_t blocks, const Layout &at) {
  const int path = s->linear_path;
  LinearPlan plan = path == 1 || (path == 0 && m <= 64) ? plan_few(s, m, n, blocks)
                  : path == 3 ? LinearPlan{4, 256, 256, 1} : plan_rows(s, m, n, blocks, at, path == 0);
  if (s->linear_split && plan.kernel != 4) {
    plan.split = s->linear_split;
    while (plan.split > blocks) plan.split /= 2;
  }
  return plan;
}

}  // namespace

// Shared-memory limits of the kernels, the clusters that the device holds of each (asked for
// once per device: seventeen queries), and the driver's encoder of tensor maps.  A handle
// for which one of these fails is without ts_linear_e4m3 only.
void ts_host::linear_setup(ts_sampler *s) {
  std::lock_guard<std::mutex> lock(g_linear_mu);
  s->linear_ready = false;
  for (int i = 0; i < kKernels; ++i) {
    const LinearKernel k = kernel_for(i);
    if (cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(k.smem)) != cudaSuccess) {
      cudaGetLastError();
      return;
    }
  }
  LinearDevice *d = nullptr;
  for (LinearDevice &known : g_linear_devices)
    if (known.device == s->device) d = &known;
  if (!d) {
    LinearDevice now;
    now.device = s->device;
    std::memset(now.clusters, 0, sizeof now.clusters);
    for (int i = 0; i < kKernels; ++i)
      for (int j = 0; j < 4; ++j) {
        if (i == 4 && j != 1) continue;  // pairs are clusters of two
        const LinearKernel k = kernel_for(i);
        cudaLaunchConfig_t cfg;
        std::memset(&cfg, 0, sizeof cfg);
        cfg.gridDim = dim3(static_cast<unsigned>(s->num_sms >> j << j));
        cfg.blockDim = dim3(static_cast<unsigned>(k.threads));
        cfg.dynamicSmemBytes = k.smem;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 1u << j;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        int held = 0;
        if (cudaOccupancyMaxActiveClusters(&held, k.fn, &cfg) != cudaSuccess) {
          cudaGetLastError();
          return;
        }
        now.clusters[i][j] = std::max(held, 1);
      }
    g_linear_devices.push_back(now);
    d = &g_linear_devices.back();
  }
  std::memcpy(s->linear_clusters, d->clusters, sizeof s->linear_clusters);
  if (!g_encode) {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return;
    }
    g_encode = reinterpret_cast<EncodeTiled>(fn);
  }
  s->linear_ready = true;
}

extern "C" ts_status ts_linear_e4m3(ts_sampler *s, const ts_linear_args *a, void *stream) {
  if (!s || !a) return TS_ERR_INVALID_ARG;
  if (a->n_rows < 0 || a->in_dim < 1 || a->out_dim < 1) return TS_ERR_INVALID_ARG;
  if (a->out_dtype != TS_DTYPE_F32 && a->out_dtype != TS_DTYPE_BF16) return TS_ERR_INVALID_ARG;
  const int64_t blocks = blocks_of(a->in_dim);
  for (int64_t x : {a->x_stride, a->x_scale_stride, a->w_stride, a->w_scale_stride, a->out_stride})
    if (x < 0) return TS_ERR_INVALID_ARG;
  if (a->n_rows > 1 && (a->x_stride < a->in_dim || a->x_scale_stride < blocks || a->out_stride < a->out_dim))
    return TS_ERR_INVALID_ARG;
  if ((a->out_dim > 1 && a->w_stride < a->in_dim) || (a->out_dim > TS_SCALE_BLOCK && a->w_scale_stride < blocks))
    return TS_ERR_INVALID_ARG;
  if ((a->n_rows > 1 && a->x_stride % 16) || (a->out_dim > 1 && a->w_stride % 16)) return TS_ERR_INVALID_ARG;
  if (a->in_dim > TS_LINEAR_MAX_DIM || a->n_rows > TS_LINEAR_MAX_ROWS || a->out_dim > TS_LINEAR_MAX_ROWS)
    return TS_ERR_UNSUPPORTED;
  for (int64_t x : {a->x_stride, a->x_scale_stride, a->w_stride, a->w_scale_stride, a->out_stride})
    if (x >= (1ll << 40)) return TS_ERR_UNSUPPORTED;
  if (a->n_rows == 0) return TS_OK;
  const int es = a->out_dtype == TS_DTYPE_F32 ? 4 : 2;
  if (!a->x || !a->x_scale || !a->w || !a->w_scale || !a->out || !aligned(a->x, 16) || !aligned(a->w, 16) ||
      !aligned(a->x_scale, 4) || !aligned(a->w_scale, 4) || !aligned(a->out, es))
    return TS_ERR_INVALID_ARG;
  const ts_host::Span out = ts_host::rows_span(a->out, a->n_rows, a->out_dim, a->out_stride, es);
  if (out.meets(ts_host::rows_span(a->x, a->n_rows, a->in_dim, a->x_stride, 1)) ||
      out.meets(ts_host::rows_span(a->x_scale, a->n_rows, blocks, a->x_scale_stride, 4)) ||
      out.meets(ts_host::rows_span(a->w, a->out_dim, a->in_dim, a->w_stride, 1)) ||
      out.meets(ts_host::rows_span(a->w_scale, blocks_of(a->out_dim), blocks, a->w_scale_stride, 4)))
    return TS_ERR_INVALID_ARG;
  if (!s->linear_ready) return TS_ERR_UNSUPPORTED;

  ts::LinearParams p;
  std::memset(&p, 0, sizeof p);
  p.x_scale = a->x_scale;
  p.w_scale = a->w_scale;
  p.x_scale_stride = a->x_scale_stride;
  p.w_scale_stride = a->w_scale_stride;
  p.out = a->out;
  p.out_stride = a->out_stride;
  p.out_f32 = a->out_dtype == TS_DTYPE_F32 ? 1 : 0;
  p.n_rows = a->n_rows;
  p.out_dim = a->out_dim;
  p.blocks = static_cast<int32_t>(blocks);
  p.status = s->status;
  p.wait_cycles = s->linear_lose ? 1u << 24 : ts::kWaitCycles;
  p.lose = s->linear_lose - 1;
  p.wide_scales = aligned(a->x_scale, 16) && (a->n_rows == 1 || a->x_scale_stride % 4 == 0);
  p.wide_out = aligned(a->out, 16) && (a->n_rows == 1 || a->out_stride * es % 16 == 0);

  const int32_t m = a->n_rows;
  const auto whole_lines = [](const void *rows, int64_t n, int64_t stride) {
    return aligned(rows, 128) && (n == 1 || stride % 128 == 0);
  };
  const LinearPlan plan = plan_for(s, m, a->out_dim, blocks, {whole_lines(a->x, m, a->x_stride) && whole_lines(a->w, a->out_dim, a->w_stride), p.wide_out != 0});
  const LinearKernel k = kernel_for(plan.kernel);
  const bool few = plan.kernel < 3, pair = plan.kernel == 4;
  if (pair && s->linear_lose) return TS_ERR_UNSUPPORTED;
  const int64_t tiles_n = ceil_div(a->out_dim, plan.columns), tiles_m = ceil_div(m, plan.rows), tiles = tiles_n * tiles_m;
  if (tiles * plan.split > INT32_MAX / 2) return TS_ERR_UNSUPPORTED;
  p.tiles_n = static_cast<int32_t>(tiles_n);
  p.tiles_m = static_cast<int32_t>(tiles_m);
  p.tiles = static_cast<int32_t>(tiles);
  p.columns = plan.columns;
  p.split = plan.split;

  // one row's stride says nothing
  const auto pitch = [&](int64_t rows, int64_t stride) {
    return rows > 1 ? stride : (static_cast<int64_t>(a->in_dim) + 15) / 16 * 16;
  };
  const int boxes_x = few ? plan.rows : 128, boxes_w = pair ? plan.columns / 2 : plan.columns;
  CUtensorMap map_w, map_x;
  if (!tensor_map(&map_w, a->w, a->in_dim, a->out_dim, pitch(a->out_dim, a->w_stride), boxes_w) ||
      !tensor_map(&map_x, a->x, a->in_dim, m, pitch(m, a->x_stride), boxes_x))
    return TS_ERR_UNSUPPORTED;

  const int cluster = pair ? 2 : plan.split;
  const int64_t grid = pair ? 2 * std::min<int64_t>(tiles, s->linear_clusters[4][1]) : tiles * cluster;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(k.threads));
  cfg.dynamicSmemBytes = k.smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = s->pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  void *few_args[] = {&map_w, &map_x, &p}, *rows_args[] = {&map_x, &map_w, &p};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, k.fn, few ? few_args : rows_args);
  return e == cudaSuccess ? TS_OK : cuda_fail(e, "linear launch");
}
