// ts_layer.cu -- host side of the layer operators that work row by row (ts_rms_norm,
// ts_gate, ts_rotary, ts_kv_append_rotary): argument checks, kernel choice and
// launches on the caller's stream; and the rotary frequencies.
#include <algorithm>
#include <cmath>
#include <cstring>

#include "ts_gate.cuh"
#include "ts_host.h"
#include "ts_norm.cuh"
#include "ts_rotary.cuh"

static_assert(ts::kScaleBlock == TS_SCALE_BLOCK, "8-bit rows");
static_assert(ts::kActNone == TS_ACT_NONE && ts::kActSilu == TS_ACT_SILU && ts::kActGelu == TS_ACT_GELU &&
                  ts::kActGeluTanh == TS_ACT_GELU_TANH, "activations");

namespace {

using ts_host::aligned;
using ts_host::cuda_fail;
using ts_host::Heads;
using ts_host::launch;
using ts_host::rows_span;
using ts_host::size_of;
using ts_host::Span;

bool real_type(int32_t dtype) { return dtype == TS_DTYPE_F32 || dtype == TS_DTYPE_BF16; }
bool out_type(int32_t dtype) { return real_type(dtype) || dtype == TS_DTYPE_E4M3; }
int64_t scales_of(int64_t dim) { return (dim + TS_SCALE_BLOCK - 1) / TS_SCALE_BLOCK; }

// An array of rows: where it is, its stride and its elements' size.
struct Rows {
  const void *p;
  int64_t stride;
  int es;
};
// Whether rows can be moved in pieces of `width` elements (8 or 16).
bool in_pieces(const Rows &r, int64_t n_rows, int width) {
  const int64_t to = std::min(2 * width, width * r.es);
  return aligned(r.p, static_cast<size_t>(to)) && (n_rows == 1 || r.stride * r.es % to == 0);
}

// --------------------------------------------------------------------------
// Norm
// --------------------------------------------------------------------------
template <class Src, class Out>
const void *norm_kernel(int v, int width) {
  if constexpr (sizeof(Out) == 1)
    if (width == 16) return reinterpret_cast<const void *>(ts::rms_norm_kernel<Src, Out, 1, 16, true>);
  if (width == 8)
    return v == 1 ? reinterpret_cast<const void *>(ts::rms_norm_kernel<Src, Out, 1, 8, true>)
         : v == 2 ? reinterpret_cast<const void *>(ts::rms_norm_kernel<Src, Out, 2, 8, true>)
                  : reinterpret_cast<const void *>(ts::rms_norm_kernel<Src, Out, 4, 8, false>);
  return v == 1 ? reinterpret_cast<const void *>(ts::rms_norm_kernel<Src, Out, 1, 4, true>)
       : v == 2 ? reinterpret_cast<const void *>(ts::rms_norm_kernel<Src, Out, 2, 4, true>)
       : v == 4 ? reinterpret_cast<const void *>(ts::rms_norm_kernel<Src, Out, 4, 4, false>)
                : reinterpret_cast<const void *>(ts::rms_norm_kernel<Src, Out, 8, 4, false>);
}
template <class Src>
const void *norm_kernel_to(int32_t out, int v, int width) {
  return out == TS_DTYPE_F32 ? norm_kernel<Src, float>(v, width)
       : out == TS_DTYPE_BF16 ? norm_kernel<Src, uint16_t>(v, width) : norm_kernel<Src, uint8_t>(v, width);
}

// --------------------------------------------------------------------------
// Gate
// --------------------------------------------------------------------------
template <class Src>
const void *gate_kernel_to(int32_t out, int width) {
  if constexpr (sizeof(Src) == 2)
    if (width == 16) return reinterpret_cast<const void *>(ts::gate_kernel<Src, uint8_t, 16>);
  if (width == 8)
    return out == TS_DTYPE_F32 ? reinterpret_cast<const void *>(ts::gate_kernel<Src, float, 8>)
         : out == TS_DTYPE_BF16 ? reinterpret_cast<const void *>(ts::gate_kernel<Src, uint16_t, 8>)
                                : reinterpret_cast<const void *>(ts::gate_kernel<Src, uint8_t, 8>);
  return out == TS_DTYPE_F32 ? reinterpret_cast<const void *>(ts::gate_kernel<Src, float, 4>)
       : out == TS_DTYPE_BF16 ? reinterpret_cast<const void *>(ts::gate_kernel<Src, uint16_t, 4>)
                              : reinterpret_cast<const void *>(ts::gate_kernel<Src, uint8_t, 4>);
}

// --------------------------------------------------------------------------
// Rotary positions
// --------------------------------------------------------------------------
template <class Src, class Dst, bool CACHE>
const void *rotary_kernel(int piece) {
  return piece == 8 ? reinterpret_cast<const void *>(ts::rotary_kernel<Src, Dst, 8, CACHE>)
       : piece == 4 ? reinterpret_cast<const void *>(ts::rotary_kernel<Src, Dst, 4, CACHE>)
                    : reinterpret_cast<const void *>(ts::rotary_kernel<Src, Dst, 1, CACHE>);
}

ts_status check_rotary(const ts_rotary_args *a) {
  if (!a || a->n_tokens < 0 || a->head_dim < 1 || a->rotary_dim < 2 || a->rotary_dim % 2 ||
      a->rotary_dim > a->head_dim || !real_type(a->dtype) || (a->rows && a->n_rows < 0) || !std::isfinite(a->amplitude))
    return TS_ERR_INVALID_ARG;
  for (int64_t x : {a->x_token_stride, a->x_head_stride, a->out_token_stride, a->out_head_stride})
    if (x < 0) return TS_ERR_INVALID_ARG;
  if (a->head_dim > TS_ROTARY_MAX_HEAD_DIM || a->n_heads > TS_KV_MAX_HEADS) return TS_ERR_UNSUPPORTED;
  return TS_OK;
}
Heads out_heads(const ts_rotary_args *a) {
  return Heads::of(a->out, a->rows ? a->n_rows : a->n_tokens, a->n_heads, a->out_token_stride, a->out_head_stride, a->head_dim,
                   size_of(a->dtype));
}
ts_status check_rotary_arrays(const ts_rotary_args *a, bool queries) {
  const int es = size_of(a->dtype);
  if (!a->positions || !a->freqs || !aligned(a->freqs, 8)) return TS_ERR_INVALID_ARG;
  if (!queries) return TS_OK;
  if (!a->x || !a->out || !aligned(a->x, es) || !aligned(a->out, es)) return TS_ERR_INVALID_ARG;
  const Heads out = out_heads(a);
  if (out.meets_itself()) return TS_ERR_INVALID_ARG;
  if (a->x == a->out)
    return a->x_token_stride != a->out_token_stride || a->x_head_stride != a->out_head_stride ? TS_ERR_INVALID_ARG : TS_OK;
  return out.meets(Heads::of(a->x, out.rows, a->n_heads, a->x_token_stride, a->x_head_stride, a->head_dim, es)) ? TS_ERR_INVALID_ARG
                                                                                                                : TS_OK;
}
// Queries' outputs on the new keys or values, or within the cache.
bool out_meets_cache(const ts_rotary_args *a, const ts_kv_cache *c, const ts_kv_tokens *t) {
  const Heads out = out_heads(a);
  const int es = size_of(t->dtype);
  if (out.meets(Heads::of(t->k, out.rows, c->n_kv_heads, t->k_token_stride, t->k_head_stride, c->head_dim, es)) ||
      out.meets(Heads::of(t->v, out.rows, c->n_kv_heads, t->v_token_stride, t->v_head_stride, c->head_dim, es)))
    return true;
  const auto within = [&](const void *pool, int64_t block, int64_t token, int64_t head) {
    if (out.none() || c->n_blocks < 1) return false;
    const __int128 from = reinterpret_cast<uintptr_t>(pool);
    const __int128 last = static_cast<__int128>(c->n_blocks - 1) * block + static_cast<__int128>(c->block_size - 1) * token +
                          static_cast<__int128>(c->n_kv_heads - 1) * head;
    return out.end() > from && from + (last + c->head_dim) * size_of(c->dtype) > out.from;
  };
  return within(c->k, c->k_block_stride, c->k_token_stride, c->k_head_stride) ||
         within(c->v, c->v_block_stride, c->v_token_stride, c->v_head_stride);
}
// The largest piece (8, 4 or 1 elements) that divides the pairs and the head and that
// addresses and strides allow.
int piece_of(const ts_rotary_args *a, const ts_kv_tokens *t, bool queries) {
  const int es = size_of(a->dtype);
  const auto fits = [&](int piece) {
    if (a->rotary_dim / 2 % piece || a->head_dim % piece) return false;
    const int64_t to = std::min(16, piece * es);
    const auto ok = [&](const void *p, int64_t token, int64_t head) {
      return aligned(p, static_cast<size_t>(to)) && token * es % to == 0 && head * es % to == 0;
    };
    if (queries && (!ok(a->x, a->x_token_stride, a->x_head_stride) || !ok(a->out, a->out_token_stride, a->out_head_stride)))
      return false;
    return !t || (ok(t->k, t->k_token_stride, t->k_head_stride) && ok(t->v, t->v_token_stride, t->v_head_stride));
  };
  return fits(8) ? 8 : fits(4) ? 4 : 1;
}

// The parts of the parameters that both calls share, and the launch.
ts_status launch_rotary(const ts_sampler *s, const ts_rotary_args *a, ts::RotaryParams &p, const void *fn, int piece,
                        void *stream) {
  const bool queries = a->x != nullptr;
  p.x = a->x;
  p.out = a->out;
  p.x_token = a->x_token_stride;
  p.x_head = a->x_head_stride;
  p.out_token = a->out_token_stride;
  p.out_head = a->out_head_stride;
  p.positions = a->positions;
  p.rows = a->rows;
  p.freqs = a->freqs;
  p.amplitude = a->amplitude;
  p.n_tokens = a->n_tokens;
  p.n_rows = a->n_rows;
  p.heads = queries ? a->n_heads : 0;
  p.dim = a->head_dim;
  p.half = a->rotary_dim / 2;
  p.interleaved = a->interleaved != 0;
  p.in_place = a->x == a->out;
  p.status = s->status;
  const int64_t per_head = (a->head_dim + 2 * piece - 1) / (2 * piece), turned = p.half / piece;
  const int64_t per_token = per_head * (p.heads + 2 * static_cast<int64_t>(p.kv_heads));
  if (per_token > (1 << 23)) return TS_ERR_UNSUPPORTED;
  // whole tokens: eight of a thread's units, twelve tokens at least (138 us with eight, 136),
  // fewer while SMs would idle
  const int64_t n = a->n_tokens;
  int64_t tokens = std::min<int64_t>(std::max<int64_t>(ts::kRotaryThreads * 8 / per_token, 12), (n + 4 * s->num_sms - 1) / (4 * s->num_sms));
  tokens = std::min<int64_t>(tokens, std::min<int64_t>(ts::kRotaryTokens, ts::kRotaryTableFloats / a->rotary_dim));
  tokens = std::max<int64_t>(1, tokens);
  p.tokens_per_cta = static_cast<int32_t>(tokens);
  // runs of units: pairs of queries and keys, their other elements, values
  const auto add = [&](int k, int which, bool rotates, int64_t heads, int64_t units) {
    ts::RotaryRun &r = p.run[k];
    r.first = p.units;
    r.units = static_cast<int32_t>(heads * units);
    r.which = which;
    r.rotates = rotates;
    r.from = which == 2 || rotates ? 0 : a->rotary_dim;
    r.by_head = ts::FastDiv::of(static_cast<uint32_t>(std::max<int64_t>(1, units)));
    p.units += (r.units + 31) / 32 * 32;
  };
  add(0, 0, true, p.heads, turned);
  add(1, 1, true, p.kv_heads, turned);
  add(2, 0, false, p.in_place ? 0 : p.heads, per_head - turned);
  add(3, 1, false, p.kv_heads, per_head - turned);
  add(4, 2, false, p.kv_heads, per_head);
  p.group = std::min(p.units, ts::kRotaryThreads);
  const size_t smem = static_cast<size_t>(tokens) * a->rotary_dim * sizeof(float);
  void *args[] = {&p};
  const cudaError_t e = launch(fn, dim3(static_cast<unsigned>((n + tokens - 1) / tokens)), ts::kRotaryThreads, smem,
                               s->pdl != 0, static_cast<cudaStream_t>(stream), args);
  return e == cudaSuccess ? TS_OK : cuda_fail(e, "rotary launch");
}

}  // namespace

extern "C" {

ts_status ts_rms_norm(ts_sampler *s, const ts_norm_args *a, void *stream) {
  if (!s || !a) return TS_ERR_INVALID_ARG;
  if (a->n_rows < 0 || a->dim < 1 || !real_type(a->dtype) || !out_type(a->out_dtype) ||
      (a->weight && !real_type(a->weight_dtype)) || !std::isfinite(a->eps) || a->eps < 0.0f ||
      !std::isfinite(a->weight_offset))
    return TS_ERR_INVALID_ARG;
  const bool e4m3 = a->out_dtype == TS_DTYPE_E4M3;
  if (a->out_scale ? !e4m3 : e4m3 && a->n_rows > 0) return TS_ERR_INVALID_ARG;
  const int es = size_of(a->dtype), os = size_of(a->out_dtype);
  const int64_t n = a->n_rows, dim = a->dim;
  const Rows x = {a->x, a->x_stride, es}, res = {a->residual, a->residual_stride, es},
             sum = {a->residual_out, a->residual_out_stride, es}, out = {a->out, a->out_stride, os};
  for (const Rows &r : {x, res, sum, out})
    if (r.p && (r.stride < 0 || (n > 1 && r.stride < dim) || !aligned(r.p, static_cast<size_t>(r.es))))
      return TS_ERR_INVALID_ARG;
  if (e4m3 && (a->out_scale_stride < 0 || (n > 1 && a->out_scale_stride < scales_of(dim)) || !aligned(a->out_scale, 4)))
    return TS_ERR_INVALID_ARG;
  if (a->dim > TS_NORM_MAX_DIM) return TS_ERR_UNSUPPORTED;
  if (n == 0) return TS_OK;
  const int ws = a->weight ? size_of(a->weight_dtype) : 0;
  if (!a->x || !a->out || (ws && !aligned(a->weight, static_cast<size_t>(ws)))) return TS_ERR_INVALID_ARG;
  const auto span = [&](const Rows &r) { return rows_span(r.p, n, dim, r.stride, r.es); };
  const auto same = [](const Rows &u, const Rows &v) { return u.p == v.p && u.stride == v.stride && u.es == v.es; };
  const Span scale = rows_span(a->out_scale, n, scales_of(dim), a->out_scale_stride, 4);
  const Span weight = rows_span(a->weight, 1, dim, dim, ws);
  if (span(out).meets(weight) || span(sum).meets(weight) || scale.meets(weight) || span(out).meets(span(sum)) ||
      span(out).meets(scale) || span(sum).meets(scale) || scale.meets(span(x)) || scale.meets(span(res)))
    return TS_ERR_INVALID_ARG;
  if ((!same(out, x) && span(out).meets(span(x))) || (!same(out, res) && span(out).meets(span(res))) ||
      (!same(sum, x) && span(sum).meets(span(x))) || (!same(sum, res) && span(sum).meets(span(res))))
    return TS_ERR_INVALID_ARG;

  // Sixteen elements a lane to 8-bit rows where rows are many: a block's scale by fewer lanes.
  // Without a residual at every width (2^27 elements in rows of 512 to 4096: bf16 74 to 107 us,
  // 116 to 138 with eight; fp32 100 to 124, 141 to 160; 2^22 elements 5 to 6.5, 5.3 to 7.5).
  // With one, bf16: rows of 512 to 1024 37 to 39 us (43 to 45), of 2560 and 3584 140 and 139
  // (148 and 150), 8192 of 4096 36.8 (40.0), but not 32,768 of 4096 (149, 144 with eight; of
  // 1536 and 2048 that many elements take 151, 147 and 143 with eight, fewer 37, 39).  With
  // one, fp32: eight (2^25 elements 68 to 71 us, 72 to 76 with sixteen; 2^22 up to 13.3, 11.1).
  const bool wide_block = !a->residual || (a->dtype == TS_DTYPE_BF16 && (dim < 4096 || n * dim < (1 << 26)));
  const bool half = e4m3 && dim >= 512 && dim <= 4096 && wide_block && n > 4 * s->num_sms;
  const auto fits = [&](int width) {
    bool ok = dim % width == 0 && (!ws || aligned(a->weight, 16));
    for (const Rows &r : {x, res, sum, out}) ok = ok && (!r.p || in_pieces(r, n, width));
    return ok;
  };
  const int width = half && fits(16) ? 16 : fits(8) ? 8 : 4;
  ts::NormParams p;
  std::memset(&p, 0, sizeof p);
  p.x = a->x;
  p.residual = a->residual;
  p.residual_out = a->residual_out;
  p.weight = a->weight;
  p.out = a->out;
  p.scale = a->out_scale;
  p.x_stride = a->x_stride;
  p.residual_stride = a->residual_stride;
  p.residual_out_stride = a->residual_out_stride;
  p.out_stride = a->out_stride;
  p.scale_stride = a->out_scale_stride;
  p.n_rows = a->n_rows;
  p.dim = a->dim;
  p.weight_f32 = a->weight && a->weight_dtype == TS_DTYPE_F32 ? 1 : 0;
  p.eps = a->eps;
  p.weight_offset = a->weight_offset;

  // Threads of a row, 512 at most and the next row's loads on their way: one unit each, two
  // of eight elements where rows are many (32,768 x 4096: 144 us, 151 with one).  The widest
  // rows take up to 1024 threads and more units.
  const int units = static_cast<int>(width > 4 ? (dim + width - 1) / width : scales_of(dim) * 32);
  const bool many = n > 4 * s->num_sms && width == 8 && units > 128;
  const int v = units <= 512 && !many ? 1 : units <= 1024 ? 2 : units <= 4096 ? 4 : 8;
  const int threads = ((units + v - 1) / v + 31) / 32 * 32;
  const int rows = threads == 32 ? 8 : 1;
  // as many CTAs as the GPU holds (64 registers a thread, 85 for sixteen elements)
  const int64_t ctas = std::min<int64_t>((n + rows - 1) / rows,
                                         static_cast<int64_t>(s->num_sms) * std::max(1, (width == 16 ? 768 : 1024) / (threads * rows)));
  const void *fn = a->dtype == TS_DTYPE_F32 ? norm_kernel_to<float>(a->out_dtype, v, width)
                                            : norm_kernel_to<uint16_t>(a->out_dtype, v, width);
  void *args[] = {&p};
  const cudaError_t e =
      launch(fn, dim3(static_cast<unsigned>(ctas)), dim3(static_cast<unsigned>(threads), static_cast<unsigned>(rows)),
             width == 16 && a->weight ? static_cast<size_t>(threads * rows) * 64 : 0, s->pdl != 0, static_cast<cudaStream_t>(stream), args);
  return e == cudaSuccess ? TS_OK : cuda_fail(e, "norm launch");
}

ts_status ts_gate(ts_sampler *s, const ts_gate_args *a, void *stream) {
  if (!s || !a) return TS_ERR_INVALID_ARG;
  if (a->n_rows < 0 || a->dim < 1 || !real_type(a->dtype) || !out_type(a->out_dtype) || a->act < TS_ACT_NONE ||
      a->act > TS_ACT_GELU_TANH)
    return TS_ERR_INVALID_ARG;
  const bool e4m3 = a->out_dtype == TS_DTYPE_E4M3, act = a->act != TS_ACT_NONE;
  if (a->out_scale ? !e4m3 : e4m3 && a->n_rows > 0) return TS_ERR_INVALID_ARG;
  const int es = size_of(a->dtype), os = size_of(a->out_dtype);
  const int64_t n = a->n_rows, dim = a->dim;
  const Rows up = {a->up, a->up_stride, es}, gate = {act ? a->gate : nullptr, a->gate_stride, es},
             out = {a->out, a->out_stride, os};
  for (const Rows &r : {up, gate, out})
    if (r.p && (r.stride < 0 || (n > 1 && r.stride < dim) || !aligned(r.p, static_cast<size_t>(r.es))))
      return TS_ERR_INVALID_ARG;
  if (e4m3 && (a->out_scale_stride < 0 || (n > 1 && a->out_scale_stride < scales_of(dim)) || !aligned(a->out_scale, 4)))
    return TS_ERR_INVALID_ARG;
  if (a->dim > TS_GATE_MAX_DIM) return TS_ERR_UNSUPPORTED;
  if (n == 0) return TS_OK;
  if (!a->up || !a->out || (act && !a->gate)) return TS_ERR_INVALID_ARG;
  const auto span = [&](const Rows &r) { return rows_span(r.p, n, dim, r.stride, r.es); };
  const auto same = [](const Rows &u, const Rows &v) { return u.p == v.p && u.stride == v.stride && u.es == v.es; };
  const Span scale = rows_span(a->out_scale, n, scales_of(dim), a->out_scale_stride, 4);
  if (scale.meets(span(up)) || scale.meets(span(gate)) || scale.meets(span(out)) ||
      (!same(out, up) && span(out).meets(span(up))) || (!same(out, gate) && span(out).meets(span(gate))))
    return TS_ERR_INVALID_ARG;

  const auto fits = [&](int width) {
    bool ok = dim % width == 0;
    for (const Rows &r : {up, gate, out}) ok = ok && (!r.p || in_pieces(r, n, width));
    return ok;
  };
  // sixteen elements a lane to 8-bit rows where every thread of the GPU has some (gelu on
  // 16,384 x 11,008 142 us, x 11,000 with eight 181)
  const bool half = a->dtype == TS_DTYPE_BF16 && e4m3 && n * scales_of(dim) * 8 >= 4ll * s->num_sms * ts::kGateThreads;
  const int width = half && fits(16) ? 16 : fits(8) ? 8 : 4;
  ts::GateParams p;
  std::memset(&p, 0, sizeof p);
  p.up = a->up;
  p.gate = a->gate;
  p.out = a->out;
  p.scale = a->out_scale;
  p.up_stride = a->up_stride;
  p.gate_stride = a->gate_stride;
  p.out_stride = a->out_stride;
  p.scale_stride = a->out_scale_stride;
  p.dim = a->dim;
  p.act = a->act;
  const int64_t per_row = scales_of(dim) * (TS_SCALE_BLOCK / width);
  p.by_row = ts::FastDiv::of(static_cast<uint32_t>(per_row));
  const int64_t all = (n * per_row + ts::kGateThreads - 1) / ts::kGateThreads;
  const int64_t grid = std::min<int64_t>(all, static_cast<int64_t>(ts::gate_ctas(es, os, width)) * s->num_sms), step = grid * ts::kGateThreads;
  // whole blocks: the threads and a row's units are multiples of a block's
  const int64_t step_rows = step / per_row, step_elems = step % per_row * width;
  p.n_rows = a->n_rows;
  p.step_rows = static_cast<uint32_t>(step_rows);
  p.step_elems = static_cast<int32_t>(step_elems);
  p.row_elems = static_cast<int32_t>(scales_of(dim) * TS_SCALE_BLOCK);
  const auto move = [&](int64_t stride, int64_t in_row, int64_t row, int64_t *step_by, int64_t *wrap_by) {
    if (n == 1) stride = 0;  // says nothing
    *step_by = step_rows * stride + in_row;
    *wrap_by = stride - row;
  };
  move(a->up_stride, step_elems, p.row_elems, &p.step.up, &p.wrap.up);
  move(a->gate_stride, step_elems, p.row_elems, &p.step.gate, &p.wrap.gate);
  move(a->out_stride, step_elems, p.row_elems, &p.step.out, &p.wrap.out);
  move(a->out_scale_stride, step_elems / TS_SCALE_BLOCK, scales_of(dim), &p.step.scale, &p.wrap.scale);
  const void *fn = a->dtype == TS_DTYPE_F32 ? gate_kernel_to<float>(a->out_dtype, width)
                                            : gate_kernel_to<uint16_t>(a->out_dtype, width);
  void *args[] = {&p};
  const cudaError_t e = launch(fn, dim3(static_cast<unsigned>(grid)), ts::kGateThreads, 0, s->pdl != 0,
                               static_cast<cudaStream_t>(stream), args);
  return e == cudaSuccess ? TS_OK : cuda_fail(e, "gate launch");
}

ts_status ts_rotary(ts_sampler *s, const ts_rotary_args *a, void *stream) {
  if (!s) return TS_ERR_INVALID_ARG;
  ts_status rc = check_rotary(a);
  if (rc != TS_OK) return rc;
  if (a->n_heads < 1) return TS_ERR_INVALID_ARG;
  if (a->n_tokens == 0) return TS_OK;
  rc = check_rotary_arrays(a, true);
  if (rc != TS_OK) return rc;
  ts::RotaryParams p;
  std::memset(&p, 0, sizeof p);
  const int piece = piece_of(a, nullptr, true);
  const void *fn = a->dtype == TS_DTYPE_F32 ? rotary_kernel<float, float, false>(piece)
                                            : rotary_kernel<uint16_t, uint16_t, false>(piece);
  return launch_rotary(s, a, p, fn, piece, stream);
}

ts_status ts_kv_append_rotary(ts_sampler *s, const ts_kv_cache *c, const ts_kv_tokens *t, const ts_rotary_args *a,
                              void *stream) {
  if (!s || !t) return TS_ERR_INVALID_ARG;
  ts_status rc = ts_host::check_append(c, t);
  if (rc != TS_OK) return rc;
  rc = check_rotary(a);
  if (rc != TS_OK) return rc;
  const bool queries = a->x != nullptr;
  // (an empty batch has heads and no address)
  if (queries ? a->n_heads < 1 : a->n_heads < 0 || (a->n_heads > 0 && a->n_tokens > 0)) return TS_ERR_INVALID_ARG;
  if (a->n_tokens != t->n_tokens || a->rows != t->rows || (a->rows && a->n_rows != t->n_rows) || a->dtype != t->dtype ||
      a->head_dim != c->head_dim)
    return TS_ERR_INVALID_ARG;
  if (t->n_tokens == 0) return TS_OK;
  rc = ts_host::check_append_arrays(t);
  if (rc != TS_OK) return rc;
  rc = check_rotary_arrays(a, queries);
  if (rc != TS_OK) return rc;
  if (queries && out_meets_cache(a, c, t)) return TS_ERR_INVALID_ARG;

  ts::RotaryParams p;
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
  p.by_block = ts::FastDiv::of(static_cast<uint32_t>(c->block_size));
  p.n_slots = static_cast<int64_t>(c->n_blocks) * c->block_size;
  p.kv_heads = c->n_kv_heads;
  const int piece = piece_of(a, t, queries);
  const bool f32 = a->dtype == TS_DTYPE_F32;
  const void *fn = c->dtype == TS_DTYPE_E4M3
                       ? (f32 ? rotary_kernel<float, uint8_t, true>(piece) : rotary_kernel<uint16_t, uint8_t, true>(piece))
                       : (f32 ? rotary_kernel<float, float, true>(piece) : rotary_kernel<uint16_t, uint16_t, true>(piece));
  return launch_rotary(s, a, p, fn, piece, stream);
}

ts_status ts_rotary_frequencies(double *freqs, int32_t rotary_dim, double base, int32_t scaling, double factor,
                                double original_len, double low, double high, float *amplitude) {
  if (!freqs || rotary_dim < 2 || rotary_dim % 2 || !std::isfinite(base) || base <= 0.0 || scaling < TS_ROPE_PLAIN ||
      scaling > TS_ROPE_BY_PARTS)
    return TS_ERR_INVALID_ARG;
  if (scaling != TS_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0)) return TS_ERR_INVALID_ARG;
  if (scaling == TS_ROPE_NTK && rotary_dim < 4) return TS_ERR_INVALID_ARG;
  if (scaling == TS_ROPE_BY_PARTS &&
      (!std::isfinite(original_len) || original_len < 1.0 || !std::isfinite(low) || !std::isfinite(high) || low >= high))
    return TS_ERR_INVALID_ARG;
  const double d = rotary_dim;
  if (scaling == TS_ROPE_NTK) base *= std::pow(factor, d / (d - 2.0));
  const double two_pi = 6.283185307179586;
  for (int32_t i = 0; i < rotary_dim / 2; ++i) {
    const double f = std::pow(base, -2.0 * i / d);
    freqs[i] = f;
    if (scaling == TS_ROPE_LINEAR) freqs[i] = f / factor;
    if (scaling == TS_ROPE_BY_PARTS) {
      const double r = std::min(1.0, std::max(0.0, (original_len * f / two_pi - low) / (high - low)));
      freqs[i] = f * ((1.0 - r) / factor + r);
    }
  }
  if (amplitude) *amplitude = scaling == TS_ROPE_BY_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  return TS_OK;
}

}  // extern "C"
