// C ABI of the norm before the head and of 8-bit activation checkpoints: argument checks and
// launches. See include/dpo.h for the contract of every call.
#include <algorithm>
#include <cmath>
#include <cstdint>

#include <nvtx3/nvToolsExt.h>

#include "dpo.h"
#include "internal.h"
#include "rows8.cuh"

static_assert(DPO_CHECKPOINT_BLOCK == dpo::kQBlock, "one block length");

namespace {

using namespace dpo;

struct NvtxRange {
  explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange&) = delete;
  NvtxRange& operator=(const NvtxRange&) = delete;
};

dpo_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DPO_OK : DPO_ERR_CUDA; }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool aligned4(const void* p) { return reinterpret_cast<uintptr_t>(p) % 4 == 0; }

dpo_status dtype_ok(int32_t t) {
  if (t == DPO_F16) return DPO_ERR_UNSUPPORTED;
  return t == DPO_BF16 || t == DPO_F32 ? DPO_OK : DPO_ERR_INVALID_ARG;
}

int64_t size_of(int32_t t) { return t == DPO_BF16 ? 2 : 4; }

dpo_status shape_ok(int32_t rows, int32_t d) {
  if (rows < 0 || d < 1 || d > 65536) return DPO_ERR_INVALID_ARG;
  return d % 8 == 0 ? DPO_OK : DPO_ERR_UNSUPPORTED;
}

// A buffer of rows: bytes [begin, end) and how its rows lie in them.
struct Span {
  uintptr_t begin = 0, end = 0;
  int64_t stride = 0;       // bytes
  int64_t size = 0;         // of a value
};

// Checks a row buffer and describes it.
dpo_status rows_ok(const void* p, int32_t dtype, int32_t rows, int32_t d, int64_t stride,
                   Span* out) {
  // the bound keeps rows * stride in bytes within 64 bits, far above what memory holds
  if (p == nullptr || stride < d || stride > (1ll << 60) / std::max(rows, 1))
    return DPO_ERR_INVALID_ARG;
  if (stride % 8 != 0) return DPO_ERR_UNSUPPORTED;
  if (!aligned16(p)) return DPO_ERR_INVALID_ARG;
  out->begin = reinterpret_cast<uintptr_t>(p);
  out->size = size_of(dtype);
  out->stride = stride * out->size;
  out->end = out->begin + static_cast<uintptr_t>(rows > 0 ? rows - 1 : 0) * out->stride +
             static_cast<uintptr_t>(d) * out->size;
  return DPO_OK;
}

Span span_of(const void* p, size_t bytes) {
  Span s;
  s.begin = reinterpret_cast<uintptr_t>(p);
  s.end = p != nullptr ? s.begin + bytes : s.begin;
  return s;
}

bool apart(const Span& a, const Span& b) { return a.end <= b.begin || b.end <= a.begin; }
// Row buffers whose rows interleave without touching (column blocks of one wider array) share
// a range of addresses but no value.
bool rows_apart(const Span& a, const Span& b, int64_t row_a, int64_t row_b) {
  if (apart(a, b)) return true;
  if (a.stride != b.stride) return false;
  const int64_t diff = static_cast<int64_t>(b.begin) - static_cast<int64_t>(a.begin);
  const int64_t off = (diff % a.stride + a.stride) % a.stride;   // b's rows start here in a's pitch
  return off >= row_a && off + row_b <= a.stride;
}
bool same_rows(const Span& a, const Span& b) {
  return a.begin == b.begin && a.stride == b.stride && a.size == b.size;
}

dpo_status ckpt_ok(const dpo_checkpoint* c) {
  if (c->codes == nullptr || c->scales == nullptr || !aligned16(c->codes))
    return DPO_ERR_INVALID_ARG;
  return DPO_OK;
}
Span codes_span(const dpo_checkpoint* c, int32_t rows, int32_t d) {
  return span_of(c->codes, static_cast<size_t>(rows) * d);
}
Span scales_span(const dpo_checkpoint* c, int32_t rows, int32_t d) {
  return span_of(c->scales, static_cast<size_t>(rows) * q_blocks(d));
}
bool ckpt_apart(const dpo_checkpoint* c, int32_t rows, int32_t d, const Span& s) {
  return apart(codes_span(c, rows, d), s) && apart(scales_span(c, rows, d), s);
}

// Checks shared by forward and backward; fills the launch's view and x's span.
dpo_status norm_ok(const dpo_norm* n, NormIn* in, Span* x) {
  if (n == nullptr) return DPO_ERR_INVALID_ARG;
  dpo_status s;
  if ((s = dtype_ok(n->dtype)) != DPO_OK) return s;
  if ((s = dtype_ok(n->weight_dtype)) != DPO_OK) return s;
  if (n->kind != DPO_NORM_LAYER && n->kind != DPO_NORM_RMS) return DPO_ERR_INVALID_ARG;
  if ((s = shape_ok(n->rows, n->d)) != DPO_OK) return s;
  if (!aligned16(n->weight) || !aligned16(n->bias)) return DPO_ERR_INVALID_ARG;
  if ((n->x == nullptr) == (n->from == nullptr)) return DPO_ERR_INVALID_ARG;
  if (n->from != nullptr) {
    if ((s = ckpt_ok(n->from)) != DPO_OK) return s;
  } else if ((s = rows_ok(n->x, n->dtype, n->rows, n->d, n->x_stride, x)) != DPO_OK) {
    return s;
  }
  *in = NormIn{n->rows, n->d, n->kind == DPO_NORM_RMS, n->dtype == DPO_BF16,
               n->weight_dtype == DPO_BF16, n->eps, n->x, n->x_stride,
               n->from != nullptr ? n->from->codes : nullptr,
               n->from != nullptr ? n->from->scales : nullptr, n->weight, n->bias};
  return DPO_OK;
}

size_t norm_ws_bytes(int32_t d) {
  return sizeof(float) * 2 * static_cast<size_t>(norm_parts(d)) * static_cast<size_t>(d);
}

}  // namespace

extern "C" {

dpo_status dpo_checkpoint_pack(int32_t dtype, int32_t rows, int32_t d, const void* x,
                               int64_t x_stride, const dpo_checkpoint* out, void* stream) {
  NvtxRange nvtx_range("dpo_checkpoint_pack");
  dpo_status s;
  if ((s = dtype_ok(dtype)) != DPO_OK) return s;
  if ((s = shape_ok(rows, d)) != DPO_OK) return s;
  if (out == nullptr) return DPO_ERR_INVALID_ARG;
  if (rows == 0) return DPO_OK;
  Span xs;
  if ((s = rows_ok(x, dtype, rows, d, x_stride, &xs)) != DPO_OK) return s;
  if ((s = ckpt_ok(out)) != DPO_OK) return s;
  if (!ckpt_apart(out, rows, d, xs) || !apart(codes_span(out, rows, d), scales_span(out, rows, d)))
    return DPO_ERR_INVALID_ARG;
  return cuda_status(launch_ckpt_pack(dtype == DPO_BF16, rows, d, x, x_stride, out->codes,
                                      out->scales, static_cast<cudaStream_t>(stream)));
}

dpo_status dpo_checkpoint_unpack(int32_t dtype, int32_t rows, int32_t d,
                                 const dpo_checkpoint* from, void* y, int64_t y_stride,
                                 void* stream) {
  NvtxRange nvtx_range("dpo_checkpoint_unpack");
  dpo_status s;
  if ((s = dtype_ok(dtype)) != DPO_OK) return s;
  if ((s = shape_ok(rows, d)) != DPO_OK) return s;
  if (from == nullptr) return DPO_ERR_INVALID_ARG;
  if (rows == 0) return DPO_OK;
  Span ys;
  if ((s = rows_ok(y, dtype, rows, d, y_stride, &ys)) != DPO_OK) return s;
  if ((s = ckpt_ok(from)) != DPO_OK) return s;
  if (!ckpt_apart(from, rows, d, ys)) return DPO_ERR_INVALID_ARG;
  return cuda_status(launch_ckpt_unpack(dtype == DPO_BF16, rows, d, from->codes, from->scales, y,
                                        y_stride, static_cast<cudaStream_t>(stream)));
}

dpo_status dpo_norm_forward(const dpo_norm* norm, void* y, int64_t y_stride, float* mean,
                            float* rstd, const dpo_checkpoint* save, void* stream) {
  NvtxRange nvtx_range("dpo_norm_forward");
  if (norm != nullptr && norm->rows == 0) {      // nothing to read or write
    dpo_status s = dtype_ok(norm->dtype);
    return s != DPO_OK ? s : shape_ok(0, norm->d);
  }
  NormIn in;
  Span x, ys;
  dpo_status s = norm_ok(norm, &in, &x);
  if (s != DPO_OK) return s;
  const int32_t rows = norm->rows, d = norm->d;
  if (!(norm->eps >= 0.f) || !std::isfinite(norm->eps)) return DPO_ERR_INVALID_ARG;
  if (mean != nullptr && norm->kind == DPO_NORM_RMS) return DPO_ERR_INVALID_ARG;
  if (!aligned4(mean) || !aligned4(rstd)) return DPO_ERR_INVALID_ARG;
  if ((s = rows_ok(y, norm->dtype, rows, d, y_stride, &ys)) != DPO_OK) return s;
  const int64_t row_bytes = d * size_of(norm->dtype);
  if (norm->from != nullptr) {
    if (save != nullptr || !ckpt_apart(norm->from, rows, d, ys)) return DPO_ERR_INVALID_ARG;
  } else if (!same_rows(x, ys) && !rows_apart(x, ys, row_bytes, row_bytes)) {
    return DPO_ERR_INVALID_ARG;
  }
  if (save != nullptr) {
    if ((s = ckpt_ok(save)) != DPO_OK) return s;
    if (!ckpt_apart(save, rows, d, x) || !ckpt_apart(save, rows, d, ys) ||
        !apart(codes_span(save, rows, d), scales_span(save, rows, d)))
      return DPO_ERR_INVALID_ARG;
  }
  const int sms = device_sms();
  if (sms < 1) return DPO_ERR_CUDA;
  return cuda_status(launch_norm_fwd(in, y, y_stride, mean, rstd,
                                     save != nullptr ? save->codes : nullptr,
                                     save != nullptr ? save->scales : nullptr, sms,
                                     static_cast<cudaStream_t>(stream)));
}

dpo_status dpo_norm_workspace_size(int32_t rows, int32_t d, size_t* bytes) {
  const dpo_status s = shape_ok(rows, d);
  if (s != DPO_OK) return s;
  if (bytes != nullptr) *bytes = norm_ws_bytes(d);
  return DPO_OK;
}

dpo_status dpo_norm_backward(const dpo_norm* norm, const dpo_norm_grads* g, void* ws,
                             size_t ws_bytes, void* stream) {
  NvtxRange nvtx_range("dpo_norm_backward");
  if (norm == nullptr || g == nullptr) return DPO_ERR_INVALID_ARG;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  dpo_status s;
  if (!aligned4(g->dweight) || !aligned4(g->dbias)) return DPO_ERR_INVALID_ARG;
  if (g->accumulate != 0 && g->accumulate != 1) return DPO_ERR_INVALID_ARG;
  if (norm->rows == 0) {
    if ((s = dtype_ok(norm->dtype)) != DPO_OK) return s;
    if ((s = shape_ok(0, norm->d)) != DPO_OK) return s;
    for (float* out : {g->dweight, g->dbias})
      if (out != nullptr && !g->accumulate &&
          cudaMemsetAsync(out, 0, sizeof(float) * norm->d, st) != cudaSuccess)
        return DPO_ERR_CUDA;
    return DPO_OK;
  }
  NormIn in;
  Span x, dys, dxs;
  if ((s = norm_ok(norm, &in, &x)) != DPO_OK) return s;
  const int32_t rows = norm->rows, d = norm->d;
  if ((s = dtype_ok(g->dy_dtype)) != DPO_OK) return s;
  if (g->rstd == nullptr || !aligned4(g->rstd) || !aligned4(g->mean) ||
      (g->mean == nullptr) != (norm->kind == DPO_NORM_RMS))
    return DPO_ERR_INVALID_ARG;
  if ((s = rows_ok(g->dy, g->dy_dtype, rows, d, g->dy_stride, &dys)) != DPO_OK) return s;
  if (g->dx != nullptr) {
    if ((s = rows_ok(g->dx, norm->dtype, rows, d, g->dx_stride, &dxs)) != DPO_OK) return s;
    const int64_t dx_row = d * size_of(norm->dtype), dy_row = d * size_of(g->dy_dtype);
    if (!same_rows(dxs, dys) && !rows_apart(dys, dxs, dy_row, dx_row)) return DPO_ERR_INVALID_ARG;
    if (norm->from != nullptr ? !ckpt_apart(norm->from, rows, d, dxs)
                              : !rows_apart(x, dxs, dx_row, dx_row))
      return DPO_ERR_INVALID_ARG;
  }
  if (g->dweight != nullptr && g->dweight == g->dbias) return DPO_ERR_INVALID_ARG;
  if (ws == nullptr || ws_bytes < norm_ws_bytes(d) || reinterpret_cast<uintptr_t>(ws) % 256 != 0)
    return DPO_ERR_WORKSPACE;
  const int sms = device_sms();
  if (sms < 1) return DPO_ERR_CUDA;
  const NormGradBuf buf{g->mean, g->rstd, g->dy, g->dy_dtype == DPO_BF16, g->dy_stride, g->dx,
                        g->dx_stride, g->dweight, g->dbias, g->accumulate,
                        static_cast<float*>(ws)};
  return cuda_status(launch_norm_bwd(in, buf, sms, st));
}

}  // extern "C"
