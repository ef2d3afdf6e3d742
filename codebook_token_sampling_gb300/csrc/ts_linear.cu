// ts_linear.cu -- host side of ts_linear_e4m3: argument checks, tensor maps, kernel
// choice and launch on the caller's stream.
#include <algorithm>
#include <cstring>

#include "ts_host.h"
#include "ts_linear.cuh"

static_assert(ts::kRowStalled == TS_ROW_STALLED, "status bits");

namespace {

using ts_host::aligned;
using ts_host::cuda_fail;

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled g_encode = nullptr;  // set by the first ts_create, the same for all

// Rows of bytes in boxes of 128 columns by `box_rows`, swizzled; what lies outside is 0.
bool tensor_map(CUtensorMap *m, const void *p, int64_t columns, int64_t rows, int64_t stride, int box_rows) {
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(columns), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  const cuuint32_t box[2] = {128, static_cast<cuuint32_t>(box_rows)}, steps[2] = {1, 1};
  return g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void *>(p), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct FewKernel {
  const void *fn;
  uint32_t smem;
  int columns;
};
template <int TN>
FewKernel few_kernel() {
  return {reinterpret_cast<const void *>(ts::linear_few_kernel<TN>), ts::FewTile<TN>::kSmemBytes, TN};
}
FewKernel few_kernel_for(int i) {
  return i == 0 ? few_kernel<16>() : i == 1 ? few_kernel<32>() : i == 2 ? few_kernel<64>() : few_kernel<128>();
}

int64_t blocks_of(int64_t dim) { return (dim + TS_SCALE_BLOCK - 1) / TS_SCALE_BLOCK; }

}  // namespace

// Shared-memory limits of the kernels, and the driver's encoder of tensor maps.
ts_status ts_host::linear_setup() {
  for (int i = 0; i < 4; ++i) {
    const FewKernel k = few_kernel_for(i);
    const cudaError_t e =
        cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(k.smem));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  }
  void *fn = nullptr;
  cudaDriverEntryPointQueryResult found;
  if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &found) == cudaSuccess &&
      found == cudaDriverEntryPointSuccess)
    g_encode = reinterpret_cast<EncodeTiled>(fn);
  else
    cudaGetLastError();  // ts_linear_e4m3 says TS_ERR_UNSUPPORTED
  return TS_OK;
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
  if (a->in_dim > TS_LINEAR_MAX_DIM) return TS_ERR_UNSUPPORTED;
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
  if (!g_encode) return TS_ERR_UNSUPPORTED;

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
  p.tiles_n = static_cast<int32_t>(blocks_of(a->out_dim));
  p.status = s->status;

  const int32_t m = a->n_rows;
  const FewKernel k = few_kernel_for(m <= 16 ? 0 : m <= 32 ? 1 : m <= 64 ? 2 : 3);
  const int64_t tiles = p.tiles_n * ((static_cast<int64_t>(m) + k.columns - 1) / k.columns);
  if (tiles > INT32_MAX) return TS_ERR_UNSUPPORTED;
  int split = s->linear_split;
  if (!split)
    for (split = 1; split < 8 && tiles * split * 2 <= s->num_sms;) split *= 2;
  while (split > blocks) split /= 2;
  p.split = split;

  // one row's stride says nothing
  const auto pitch = [&](int64_t rows, int64_t stride) {
    return rows > 1 ? stride : (static_cast<int64_t>(a->in_dim) + 15) / 16 * 16;
  };
  CUtensorMap map_w, map_x;
  if (!tensor_map(&map_w, a->w, a->in_dim, a->out_dim, pitch(a->out_dim, a->w_stride), 128) ||
      !tensor_map(&map_x, a->x, a->in_dim, m, pitch(m, a->x_stride), k.columns))
    return TS_ERR_UNSUPPORTED;

  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = dim3(static_cast<unsigned>(tiles), 1, static_cast<unsigned>(split));
  cfg.blockDim = dim3(ts::kFewThreads);
  cfg.dynamicSmemBytes = k.smem;
  cfg.stream = static_cast<cudaStream_t>(stream);
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = s->pdl ? 1 : 0;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = static_cast<unsigned>(split);
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  void *args[] = {&map_w, &map_x, &p};
  const cudaError_t e = cudaLaunchKernelExC(&cfg, k.fn, args);
  return e == cudaSuccess ? TS_OK : cuda_fail(e, "linear launch");
}
