// ts_kv.cu -- host side of the paged key-value cache's calls: argument checks,
// kernel choice and launches on the caller's stream (ts_reserve_kv,
// ts_kv_tables, ts_kv_append, ts_paged_attention).
#include <algorithm>
#include <cmath>
#include <cstring>
#include <mutex>
#include <new>

#include "ts_host.h"
#include "ts_kv.cuh"
#include "ts_paged_join.cuh"
#include "ts_paged_kernels.h"

static_assert(ts::kRowBadBlock == TS_ROW_BAD_BLOCK && ts::kRowNoBlocks == TS_ROW_NO_BLOCKS,
              "status bits");
static_assert(ts::kTablesMaxRequests == TS_KV_MAX_REQUESTS && ts::kPagedMaxDim == TS_KV_MAX_HEAD_DIM,
              "limits");

// Workspace of ts_reserve_kv: paged attention's pieces, then the free count of a
// table update in place and the lengths of as many requests as any call may have.
struct ts_kv_state {
  void *mem;
  int ctas;          // pieces for this many CTAs
  int max_requests;  // as reserved: tables of more are refused
  ts::PagedParts *parts;
  unsigned long long *arrived, *calls;
  float *acc;
  float2 *ml;
  int32_t *lens, *n_free;
};

namespace {

using ts_host::cuda_fail;
using ts_host::PagedKernel;
using ts_host::paged_kernel_bf16;
using ts_host::paged_kernel_e4m3;
using ts_host::paged_kernel_f32;

cudaError_t launch(const void *fn, dim3 grid, int threads, size_t smem, bool pdl, cudaStream_t st,
                   void **args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = pdl ? 1 : 0;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

int size_of(int dtype) { return dtype == TS_DTYPE_F32 ? 4 : dtype == TS_DTYPE_BF16 ? 2 : 1; }

bool aligned(const void *p, size_t to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// --------------------------------------------------------------------------
// Paged attention's kernels
// --------------------------------------------------------------------------
constexpr int kPagedKinds = 8, kPagedWidths = 5;
PagedKernel paged_kernel_for(int kind, int width, bool page16) {
  return kind < 2 ? paged_kernel_bf16(kind, width, page16)
       : kind < 4 ? paged_kernel_e4m3(kind, width, page16) : paged_kernel_f32(kind, width, page16);
}

// Items of up to about this many parts are joined by the last CTA to come (32
// streams of up to 1500 tokens: 19.6 us, 23.7 with the launch), those of more by
// a launch of their own (one request of 131,071: 50 us, 75 by the last CTA).  The
// host knows no lengths: it goes by what the table's width allows and by requests
// of equal lengths.  So few requests that are much shorter than their table take
// the launch for nothing (four of up to 40 tokens, a table of 2048: 6.4 us, 4.5
// without it), and one long request among short ones is joined by the last CTA
// (131,071 tokens beside 31 times 500: 75 us, 60 with the launch).
constexpr int kJoinHere = 10;

// Per device, once: the kernels' shared-memory limits and occupancies.
constexpr int kMaxDevices = 64;
std::mutex g_paged_mu;
struct PagedDevice {
  bool ready;
  PagedKernel kernel[kPagedKinds][kPagedWidths][2];
} g_paged[kMaxDevices];

const void *tables_kernel(bool wide) {
  return wide ? reinterpret_cast<const void *>(ts::kv_tables_kernel<int64_t>)
              : reinterpret_cast<const void *>(ts::kv_tables_kernel<int32_t>);
}

ts_status paged_setup(int device) {
  if (device < 0 || device >= kMaxDevices) return TS_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lock(g_paged_mu);
  PagedDevice &d = g_paged[device];
  if (d.ready) return TS_OK;
  for (int kind = 0; kind < kPagedKinds; ++kind)
    for (int width = 0; width < kPagedWidths; ++width)
      for (int page = 0; page < 2; ++page) {
        PagedKernel k = paged_kernel_for(kind, width, page != 0);
        cudaError_t e = cudaFuncSetAttribute(k.fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(k.smem));
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&k.occupancy, k.fn, k.threads,
                                                          k.smem);
        if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveBlocksPerMultiprocessor");
        if (k.occupancy < 1) return TS_ERR_UNSUPPORTED;
        d.kernel[kind][width][page] = k;
      }
  for (int wide = 0; wide < 2; ++wide) {
    const cudaError_t e = cudaFuncSetAttribute(
        tables_kernel(wide != 0), cudaFuncAttributeMaxDynamicSharedMemorySize,
        static_cast<int>(ts::kv_tables_smem(ts::kTablesMaxRequests)));
    if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute");
  }
  d.ready = true;
  return TS_OK;
}

ts_status check_cache(const ts_kv_cache *c) {
  if (!c || !c->k || !c->v) return TS_ERR_INVALID_ARG;
  if (c->dtype != TS_DTYPE_F32 && c->dtype != TS_DTYPE_BF16 && c->dtype != TS_DTYPE_E4M3)
    return TS_ERR_INVALID_ARG;
  if (c->n_blocks < 1 || c->block_size < 1 || c->n_kv_heads < 1 || c->head_dim < 1)
    return TS_ERR_INVALID_ARG;
  const int es = size_of(c->dtype);
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || c->head_dim * static_cast<int64_t>(es) % 16)
    return TS_ERR_INVALID_ARG;
  const int64_t strides[6] = {c->k_block_stride, c->k_token_stride, c->k_head_stride,
                              c->v_block_stride, c->v_token_stride, c->v_head_stride};
  for (int64_t x : strides)
    if (x < 0 || x * es % 16) return TS_ERR_INVALID_ARG;
  if (c->dtype != TS_DTYPE_E4M3 && (c->k_scale || c->v_scale)) return TS_ERR_INVALID_ARG;
  if (c->head_dim > TS_KV_MAX_HEAD_DIM || c->block_size > 65536) return TS_ERR_UNSUPPORTED;
  for (int64_t x : {c->k_block_stride, c->k_token_stride, c->v_block_stride, c->v_token_stride})
    if (x > INT32_MAX / es) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}

// Whether an array that ts_kv_tables writes shares memory with one that it reads
// or with another that it writes.  (Lengths and the free count may be updated in
// place; the table's rows, which may be strided, are not looked at.)
bool tables_overlap(const ts_kv_tables_args *t) {
  struct Range {
    uintptr_t at;
    size_t bytes;
  };
  const size_t n = static_cast<size_t>(t->n_requests), most = static_cast<size_t>(t->max_tokens);
  const auto range = [](const void *p, size_t bytes) {
    return Range{reinterpret_cast<uintptr_t>(p), p ? bytes : 0};
  };
  const bool lens_apart = t->lens_out != t->lens, free_apart = t->n_free_out != t->n_free;
  constexpr int kWritten = 7, kAll = 11;
  const Range r[kAll] = {
      range(lens_apart ? t->lens_out : nullptr, 4 * n), range(free_apart ? t->n_free_out : nullptr, 4),
      range(t->token_starts, 4 * (n + 1)), range(t->slots, 8 * most), range(t->positions, 4 * most),
      range(t->requests, 4 * most), range(t->free_blocks, 4 * static_cast<size_t>(t->free_len)),
      range(t->lens, 4 * n), range(t->n_new, 4 * n), range(t->finished, n), range(t->n_free, 4)};
  for (int i = 0; i < kWritten; ++i)
    for (int j = i + 1; j < kAll; ++j)
      if (r[i].bytes && r[j].bytes && r[i].at < r[j].at + r[j].bytes && r[j].at < r[i].at + r[i].bytes) return true;
  return false;
}

template <class Src, class Dst, int VEC>
const void *append_kernel(bool wide, bool rows) {
  if (rows)
    return wide ? reinterpret_cast<const void *>(ts::kv_append_kernel<Src, Dst, VEC, true, true>)
                : reinterpret_cast<const void *>(ts::kv_append_kernel<Src, Dst, VEC, false, true>);
  return wide ? reinterpret_cast<const void *>(ts::kv_append_kernel<Src, Dst, VEC, true, false>)
              : reinterpret_cast<const void *>(ts::kv_append_kernel<Src, Dst, VEC, false, false>);
}

}  // namespace

cudaError_t ts_host::kv_free(ts_sampler *s) {
  if (!s->kv) return cudaSuccess;
  const cudaError_t e = cudaFree(s->kv->mem);
  delete s->kv;
  s->kv = nullptr;
  return e;
}

extern "C" {

ts_status ts_reserve_kv(ts_sampler *s, int32_t max_requests) {
  if (!s || max_requests < 0) return TS_ERR_INVALID_ARG;
  if (max_requests > 0 && s->kv) {  // the memory stays: captured graphs hold its addresses
    s->kv->max_requests = std::max(s->kv->max_requests, max_requests);
    return TS_OK;
  }
  int prev = 0;
  cudaGetDevice(&prev);
  cudaError_t e = cudaSetDevice(s->device);
  if (e != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  ts_status rc = TS_OK;
  e = ts_host::kv_free(s);
  if (e != cudaSuccess) rc = cuda_fail(e, "cudaFree");
  if (rc == TS_OK && max_requests > 0) rc = paged_setup(s->device);
  if (rc == TS_OK && max_requests > 0) {
    int ctas = 0;
    for (const auto &kind : g_paged[s->device].kernel)
      for (const auto &width : kind)
        for (const PagedKernel &k : width) ctas = std::max(ctas, k.occupancy * s->num_sms);
    const size_t pieces = ts::paged_workspace_bytes(ctas);
    const size_t bytes = pieces + (static_cast<size_t>(TS_KV_MAX_REQUESTS) + 1) * sizeof(int32_t);
    ts_kv_state *kv = new (std::nothrow) ts_kv_state;
    if (!kv) {
      rc = TS_ERR_NO_MEMORY;
    } else {
      e = cudaMalloc(&kv->mem, bytes);
      if (e != cudaSuccess) {
        delete kv;
        rc = e == cudaErrorMemoryAllocation ? TS_ERR_NO_MEMORY : cuda_fail(e, "cudaMalloc");
      } else if ((e = cudaMemset(kv->mem, 0, bytes)) != cudaSuccess ||  // the counters start at zero,
                 (e = cudaStreamSynchronize(nullptr)) != cudaSuccess) {  // for calls on any stream
        cudaFree(kv->mem);
        delete kv;
        rc = cuda_fail(e, "cudaMemset");
      } else {
        kv->ctas = ctas;
        kv->max_requests = max_requests;
        char *at = static_cast<char *>(kv->mem);
        kv->acc = reinterpret_cast<float *>(at);
        at += 2 * static_cast<size_t>(ctas) * ts::kPagedAccBytes;
        kv->ml = reinterpret_cast<float2 *>(at);
        at += 2 * static_cast<size_t>(ctas) * ts::kPagedRows * sizeof(float2);
        kv->parts = reinterpret_cast<ts::PagedParts *>(at);
        at += 2 * static_cast<size_t>(ctas) * sizeof(ts::PagedParts);
        kv->arrived = reinterpret_cast<unsigned long long *>(at);
        kv->calls = kv->arrived + ctas;
        kv->n_free = reinterpret_cast<int32_t *>(static_cast<char *>(kv->mem) + pieces);
        kv->lens = kv->n_free + 1;
        s->kv = kv;
      }
    }
  }
  cudaSetDevice(prev);
  return rc;
}

ts_status ts_kv_debug_lose_parts(ts_sampler *s, int32_t come) {
  if (!s || !s->kv || come < 0 || come > 1000) return TS_ERR_INVALID_ARG;
  const ts_kv_state *kv = s->kv;
  int prev = 0;
  cudaGetDevice(&prev);
  cudaError_t e = cudaSetDevice(s->device);
  if (e == cudaSuccess) e = cudaDeviceSynchronize();
  unsigned long long calls = 0;  // all entries are equal
  if (e == cudaSuccess) e = cudaMemcpy(&calls, kv->calls, sizeof calls, cudaMemcpyDeviceToHost);
  const unsigned long long left = ((calls ? calls - 1 : 0) << ts::kCallShift) + static_cast<unsigned>(come);
  for (int b = 0; b < kv->ctas && e == cudaSuccess; ++b)
    e = cudaMemcpy(kv->arrived + b, &left, sizeof left, cudaMemcpyHostToDevice);
  cudaSetDevice(prev);
  return e == cudaSuccess ? TS_OK : cuda_fail(e, "ts_kv_debug_lose_parts");
}

ts_status ts_kv_tables(ts_sampler *s, const ts_kv_tables_args *t, void *stream) {
  if (!s || !t) return TS_ERR_INVALID_ARG;
  if (t->n_requests < 0 || t->block_size < 1 || t->n_blocks < 0 || t->max_blocks < 0 ||
      t->free_len < 0 || t->max_tokens < 0 || t->table_stride < t->max_blocks)
    return TS_ERR_INVALID_ARG;
  if (t->n_requests == 0) return TS_OK;
  if (!t->block_table || !t->lens || !t->free_blocks || !t->n_free || !t->token_starts ||
      (t->max_tokens > 0 && !t->slots))
    return TS_ERR_INVALID_ARG;
  if (t->n_requests > TS_KV_MAX_REQUESTS || t->block_size > 65536 ||
      static_cast<int64_t>(t->max_blocks) * t->block_size > TS_KV_MAX_LEN)
    return TS_ERR_UNSUPPORTED;
  if (tables_overlap(t)) return TS_ERR_INVALID_ARG;
  if (!s->kv || s->kv->max_requests < t->n_requests) return TS_ERR_INVALID_ARG;

  const bool lens_in_place = !t->lens_out || t->lens_out == t->lens;
  const bool free_in_place = !t->n_free_out || t->n_free_out == t->n_free;
  ts::KvTablesParams p;
  std::memset(&p, 0, sizeof p);
  p.n_requests = t->n_requests;
  p.block_size = t->block_size;
  p.n_blocks = t->n_blocks;
  p.max_blocks = t->max_blocks;
  p.max_tokens = t->max_tokens;
  p.free_len = t->free_len;
  p.table_stride = t->table_stride;
  p.block_table = t->block_table;
  p.lens = t->lens;
  p.n_new = t->n_new;
  p.finished = t->finished;
  p.free_blocks = t->free_blocks;
  p.n_free = t->n_free;
  p.lens_out = lens_in_place ? const_cast<int32_t *>(t->lens) : t->lens_out;
  p.n_free_out = free_in_place ? const_cast<int32_t *>(t->n_free) : t->n_free_out;
  p.token_starts = t->token_starts;
  p.slots = t->slots;
  p.positions = t->positions;
  p.requests = t->requests;
  p.status = s->status;
  p.by_block = ts::FastDiv::of(static_cast<uint32_t>(t->block_size));
  p.per_lane = t->max_tokens > 32768 ? 4 : 1;
  p.wide_maps = aligned(t->slots, 16) && aligned(t->positions, 16) && aligned(t->requests, 16);

  // one block for a frame's few tokens (of 512 threads: 4.8 us for 128 requests,
  // 5.1 with 256 or 1024); for prompts a block per 4096 map entries, as far as
  // the GPU holds them
  const int threads = t->n_requests <= 1024 && t->max_tokens <= 4096 ? 512 : ts::kTablesMaxThreads;
  const int grid = static_cast<int>(
      std::max<int64_t>(1, std::min<int64_t>(s->num_sms, (static_cast<int64_t>(t->max_tokens) + 4095) / 4096)));
  // blocks that still read the old values may run beside block 0: in place,
  // the new ones go through the workspace
  const bool staged_lens = grid > 1 && lens_in_place, staged_free = grid > 1 && free_in_place;
  if (staged_lens) p.lens_out = s->kv->lens;
  if (staged_free) p.n_free_out = s->kv->n_free;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  void *args[] = {&p};
  const bool wide = static_cast<int64_t>(t->n_requests) * t->max_blocks * t->block_size > INT32_MAX;
  cudaError_t e = launch(tables_kernel(wide), dim3(static_cast<unsigned>(grid)), threads,
                         ts::kv_tables_smem(t->n_requests), s->pdl != 0, st, args);
  if (e != cudaSuccess) return cuda_fail(e, "block tables launch");
  if (staged_lens || staged_free) {
    const int32_t *ln = s->kv->lens, *fn = s->kv->n_free;
    int32_t *lo = staged_lens ? const_cast<int32_t *>(t->lens) : nullptr;
    int32_t *fo = staged_free ? const_cast<int32_t *>(t->n_free) : nullptr;
    int32_t n = t->n_requests;
    void *sargs[] = {&ln, &lo, &n, &fn, &fo};
    e = launch(reinterpret_cast<const void *>(ts::kv_tables_store_kernel),
               dim3(static_cast<unsigned>((n + 255) / 256)), 256, 0, s->pdl != 0, st, sargs);
    if (e != cudaSuccess) return cuda_fail(e, "block tables store launch");
  }
  return TS_OK;
}

ts_status ts_kv_append(ts_sampler *s, const ts_kv_cache *c, const ts_kv_tokens *t, void *stream) {
  if (!s || !t) return TS_ERR_INVALID_ARG;
  const ts_status rc = check_cache(c);
  if (rc != TS_OK) return rc;
  if (t->n_tokens < 0 || (t->rows && t->n_rows < 0) || (t->dtype != TS_DTYPE_F32 && t->dtype != TS_DTYPE_BF16))
    return TS_ERR_INVALID_ARG;
  if (t->k_token_stride < 0 || t->k_head_stride < 0 || t->v_token_stride < 0 || t->v_head_stride < 0)
    return TS_ERR_INVALID_ARG;
  if (c->dtype != t->dtype && c->dtype != TS_DTYPE_E4M3) return TS_ERR_UNSUPPORTED;
  if (t->n_tokens == 0) return TS_OK;
  const int es = size_of(t->dtype);
  if (!t->k || !t->v || !t->slots || !aligned(t->k, es) || !aligned(t->v, es))
    return TS_ERR_INVALID_ARG;

  const int vec = c->dtype == TS_DTYPE_E4M3 ? 16 : 16 / es;
  const bool wide = aligned(t->k, 16) && aligned(t->v, 16) && t->k_token_stride * es % 16 == 0 &&
                    t->k_head_stride * es % 16 == 0 && t->v_token_stride * es % 16 == 0 &&
                    t->v_head_stride * es % 16 == 0;
  const bool bf16 = t->dtype == TS_DTYPE_BF16, rows = t->rows != nullptr;
  const void *fn = c->dtype == TS_DTYPE_E4M3
                       ? (bf16 ? append_kernel<uint16_t, uint8_t, 16>(wide, rows)
                               : append_kernel<float, uint8_t, 16>(wide, rows))
                       : (bf16 ? append_kernel<uint16_t, uint16_t, 8>(wide, rows)
                               : append_kernel<float, float, 4>(wide, rows));
  ts::KvAppendParams p;
  std::memset(&p, 0, sizeof p);
  p.src[0] = t->k;
  p.src[1] = t->v;
  p.src_token[0] = t->k_token_stride;
  p.src_token[1] = t->v_token_stride;
  p.src_head[0] = t->k_head_stride;
  p.src_head[1] = t->v_head_stride;
  p.dst[0] = c->k;
  p.dst[1] = c->v;
  p.dst_block[0] = c->k_block_stride;
  p.dst_block[1] = c->v_block_stride;
  p.dst_token[0] = c->k_token_stride;
  p.dst_token[1] = c->v_token_stride;
  p.dst_head[0] = c->k_head_stride;
  p.dst_head[1] = c->v_head_stride;
  p.scale[0] = c->k_scale;
  p.scale[1] = c->v_scale;
  p.slots = t->slots;
  p.rows = t->rows;
  p.n_rows = t->n_rows;
  p.block_size = c->block_size;
  p.n_slots = static_cast<int64_t>(c->n_blocks) * c->block_size;
  p.n_tokens = t->n_tokens;
  p.heads = c->n_kv_heads;
  const int64_t per_head = c->head_dim / vec, per_token = per_head * c->n_kv_heads;
  if (per_token > (1 << 20)) return TS_ERR_UNSUPPORTED;
  // whole tokens, about four units per thread, fewer while SMs would idle
  const int64_t fill = ts::kAppendThreads * 4, n_tokens = t->n_tokens;
  p.tokens_per_block = static_cast<int32_t>(std::max<int64_t>(
      1, std::min<int64_t>(fill / per_token, (n_tokens + s->num_sms - 1) / s->num_sms)));
  p.by_block = ts::FastDiv::of(static_cast<uint32_t>(c->block_size));
  p.by_token = ts::FastDiv::of(static_cast<uint32_t>(per_token));
  p.by_head = ts::FastDiv::of(static_cast<uint32_t>(per_head));
  p.status = s->status;
  const int64_t grid = (n_tokens + p.tokens_per_block - 1) / p.tokens_per_block;
  void *args[] = {&p};
  const cudaError_t e = launch(fn, dim3(static_cast<unsigned>(grid)), ts::kAppendThreads, 0,
                               s->pdl != 0, static_cast<cudaStream_t>(stream), args);
  return e == cudaSuccess ? TS_OK : cuda_fail(e, "cache append launch");
}

ts_status ts_paged_attention(ts_sampler *s, const ts_kv_cache *c, const ts_paged_query *q,
                             void *stream) {
  if (!s || !q) return TS_ERR_INVALID_ARG;
  const ts_status rc = check_cache(c);
  if (rc != TS_OK) return rc;
  if (q->n_requests < 0 || q->n_heads < 1 || q->n_heads % c->n_kv_heads || q->max_blocks < 0 ||
      q->table_stride < q->max_blocks || q->window < 0)
    return TS_ERR_INVALID_ARG;
  if (q->dtype != TS_DTYPE_F32 && q->dtype != TS_DTYPE_BF16) return TS_ERR_INVALID_ARG;
  if (!std::isfinite(q->scale) || !std::isfinite(q->softcap) || q->softcap < 0.0f)
    return TS_ERR_INVALID_ARG;
  const bool f32 = q->dtype == TS_DTYPE_F32;
  if (f32 != (c->dtype == TS_DTYPE_F32)) return TS_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(q->max_blocks) * c->block_size > TS_KV_MAX_LEN || q->n_heads > TS_KV_MAX_HEADS)
    return TS_ERR_UNSUPPORTED;
  if (q->n_requests == 0) return TS_OK;
  const int es = f32 ? 4 : 2;
  if (!q->q || !q->out || !q->lens || (!q->block_table && q->max_blocks > 0) ||
      !aligned(q->q, 16) || !aligned(q->out, 16))
    return TS_ERR_INVALID_ARG;
  const int64_t strides[4] = {q->q_request_stride, q->q_head_stride, q->out_request_stride,
                              q->out_head_stride};
  for (int64_t x : strides)
    if (x < 0 || x * es % 16) return TS_ERR_INVALID_ARG;
  if (q->key_mask && q->mask_stride < static_cast<int64_t>(q->max_blocks) * c->block_size)
    return TS_ERR_INVALID_ARG;
  if (!s->kv) return TS_ERR_INVALID_ARG;

  const int group = q->n_heads / c->n_kv_heads;
  int kind, rows;
  if (!f32) {
    rows = group <= 8 ? 8 : 16;
    kind = (c->dtype == TS_DTYPE_E4M3 ? 2 : 0) + (rows == 16 ? 1 : 0);
  } else {
    const int size = group == 1 ? 0 : group == 2 ? 1 : group <= 4 ? 2 : 3;
    rows = 1 << size;
    kind = 4 + size;
  }
  const int width = c->head_dim <= 64 ? 0 : c->head_dim <= 96 ? 1 : c->head_dim <= 128 ? 2
                  : c->head_dim <= 192 ? 3 : 4;
  const PagedKernel &k = g_paged[s->device].kernel[kind][width][c->block_size % ts::kPagedPage == 0];

  ts::PagedParams p;
  std::memset(&p, 0, sizeof p);
  const int ces = size_of(c->dtype);
  p.q = q->q;
  p.q_req = q->q_request_stride;
  p.q_head = q->q_head_stride;
  p.out = q->out;
  p.o_req = q->out_request_stride;
  p.o_head = q->out_head_stride;
  p.lse = q->lse;
  p.mask = q->key_mask;
  p.mask_stride = q->mask_stride;
  p.table = q->block_table;
  p.table_stride = q->table_stride;
  p.room = q->max_blocks * c->block_size;
  p.lens = q->lens;
  p.n_requests = q->n_requests;
  p.k = c->k;
  p.v = c->v;
  p.k_block = static_cast<int32_t>(c->k_block_stride * ces);
  p.k_token = static_cast<int32_t>(c->k_token_stride * ces);
  p.k_head = c->k_head_stride * ces;
  p.v_block = static_cast<int32_t>(c->v_block_stride * ces);
  p.v_token = static_cast<int32_t>(c->v_token_stride * ces);
  p.v_head = c->v_head_stride * ces;
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.n_blocks = c->n_blocks;
  p.block_size = c->block_size;
  p.kv_heads = c->n_kv_heads;
  p.dim = c->head_dim;
  p.group = group;
  p.rows = rows;
  p.pieces = (group + rows - 1) / rows;
  p.scale = q->scale;
  p.softcap = q->softcap;
  p.window = q->window;
  p.by_block = ts::FastDiv::of(static_cast<uint32_t>(c->block_size));
  p.parts = s->kv->parts;
  p.arrived = s->kv->arrived;
  p.all_ctas = s->kv->ctas;
  p.acc = s->kv->acc;
  p.ml = s->kv->ml;
  const int64_t items = static_cast<int64_t>(p.pieces) * p.kv_heads * q->n_requests;
  const int64_t item_tiles = std::max<int64_t>(1, (p.room + k.tile - 1) / k.tile);
  p.ctas = k.occupancy * s->num_sms;
  if (s->kv_ctas) p.ctas = std::min(p.ctas, s->kv_ctas);
  p.by_ctas = ts::FastDiv::of(static_cast<uint32_t>(p.ctas));
  // a request's units of work, rounded up
  const double tiles = (p.room / k.tile + 4.0) * p.pieces * p.kv_heads * q->n_requests;
  p.tiles_fit = tiles < 2.0e9 ? 1 : 0;
  // Parts of an item, about: the CTAs that share it, no more than its tiles.
  const int64_t parts = std::min<int64_t>(p.ctas / items + 2, item_tiles);
  p.join_here = s->kv_join ? s->kv_join - 1 : parts <= kJoinHere ? 1 : 0;
  p.calls = p.join_here && item_tiles > 1 ? s->kv->calls : nullptr;  // one tile: one part
  p.out_f32 = f32 ? 1 : 0;
  p.status = s->status;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  void *args[] = {&p};
  cudaError_t e = launch(k.fn, dim3(static_cast<unsigned>(p.ctas)), k.threads, k.smem,
                         s->pdl != 0, st, args);
  if (e != cudaSuccess) return cuda_fail(e, "paged attention launch");
  if (p.join_here) return TS_OK;
  e = launch(reinterpret_cast<const void *>(ts::paged_join_kernel),
             dim3(static_cast<unsigned>(p.ctas)), ts::kJoinThreads, 0, s->pdl != 0, st, args);
  return e == cudaSuccess ? TS_OK : cuda_fail(e, "paged attention join launch");
}

}  // extern "C"
