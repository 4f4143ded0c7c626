// fk_q8_api.cu -- argument checks and dispatch of the 8-bit linear layer
// (declared in include/fk_q8.h).  Every check runs on the host before
// anything is enqueued, as in fk_api.cu.
#include <cuda_runtime.h>

#include <cfloat>
#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "fk_q8_internal.h"

namespace fk {
namespace {

bool float_dtype(int d) { return d == FK_F32 || d == FK_BF16; }
bool q8_dtype(int d) { return d == FK_I8 || d == FK_E4M3; }
size_t size_of(int d) { return d == FK_F32 ? 4 : d == FK_BF16 ? 2 : 1; }
bool known_epilogue(int e) {
  return e == FK_EPILOGUE_NONE || e == FK_EPILOGUE_GELU_TANH || e == FK_EPILOGUE_GELU_ERF;
}

// A span of caller memory: where it is, and what may share its bytes.
struct Span {
  const void* p;
  size_t bytes, align;
};

bool overlap(const Span& a, const Span& b) {
  if (a.p == nullptr || b.p == nullptr) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return x < y + b.bytes && y < x + a.bytes;
}

// The exact same bytes (in-place operation).
bool same(const Span& a, const Span& b) { return a.p == b.p && a.bytes == b.bytes; }

// Spans present (not NULL) must be aligned, must not wrap, and must lie in
// memory of the current device.  The first loop runs without a device.
fk_status check_spans(const Span* s, int count) {
  for (int i = 0; i < count; ++i) {
    if (s[i].p == nullptr) continue;
    const uintptr_t a = reinterpret_cast<uintptr_t>(s[i].p);
    if (a % s[i].align != 0 || a > UINTPTR_MAX - s[i].bytes) return FK_ERR_INVALID_ARG;
  }
  return FK_OK;
}
fk_status check_memory(const Span* s, int count) {
  for (int i = 0; i < count; ++i) {
    if (s[i].p == nullptr) continue;
    const fk_status st = validate_span(s[i].p, s[i].bytes, s[i].align);
    if (st != FK_OK) return st;
  }
  return FK_OK;
}

// rows * cols elements of at most 4 bytes (and one 4-byte word per row and
// per column) must be addressable.
bool shape_ok(size_t rows, size_t cols) { return rows <= SIZE_MAX / 8 / cols; }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The mode of rows of `pitch` bytes in the given buffers (NULL ones aside);
// parameters (and, for aligned rows, codes) sit on 16-byte boundaries.
RowMode row_mode(size_t pitch, std::initializer_list<const void*> rows, const void* params, const void* codes) {
  if (!aligned16(params)) return kRowsAny;
  uintptr_t at = 0;
  bool first = true;
  for (const void* p : rows) {
    if (p == nullptr) continue;
    const uintptr_t off = reinterpret_cast<uintptr_t>(p) % 16;
    if (!first && off != at) return kRowsAny;
    at = off;
    first = false;
  }
  return at == 0 && pitch % 16 == 0 && aligned16(codes) ? kRowsAligned : kRowsShifted;
}

// Run `launch(ws)` with the caller's workspace, or with one taken
// stream-ordered from the library's pool when `own` is set.
template <typename F>
fk_status with_workspace(size_t need, void* ws, size_t ws_bytes, bool own, const Span* spans, int count,
                         cudaStream_t s, F launch) {
  if (need == 0) return report_cuda(launch(nullptr));
  if (own) {
    cudaError_t e = workspace_alloc(&ws, need, s);
    if (e != cudaSuccess) return report_cuda(e);
    e = launch(ws);
    const cudaError_t f = cudaFreeAsync(ws, s);
    return report_cuda(e != cudaSuccess ? e : f);
  }
  if (ws == nullptr || ws_bytes < need) return FK_ERR_INVALID_ARG;
  const Span w = {ws, need, 16};
  fk_status st = check_spans(&w, 1);
  if (st != FK_OK) return st;
  for (int i = 0; i < count; ++i)
    if (overlap(w, spans[i])) return FK_ERR_INVALID_ARG;
  st = check_memory(&w, 1);
  if (st != FK_OK) return st;
  return report_cuda(launch(ws));
}

fk_status rmsnorm_bwd_call(const void* dy, const void* h, const float* gamma, const void* dres, void* dx,
                           float* dgamma, size_t rows, size_t cols, int dtype, float eps, void* ws,
                           size_t ws_bytes, bool own, void* stream) {
  if (!float_dtype(dtype)) return FK_ERR_UNSUPPORTED_DTYPE;
  if (!(eps >= 0.0f) || !(eps <= FLT_MAX)) return FK_ERR_INVALID_ARG;
  if (cols == 0) return FK_OK;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    if (dgamma == nullptr) return FK_OK;
    if (cols > SIZE_MAX / 8) return FK_ERR_INVALID_ARG;
    const Span g = {dgamma, cols * 4, 4};
    fk_status st = check_spans(&g, 1);
    if (st == FK_OK) st = check_memory(&g, 1);
    return st != FK_OK ? st : report_cuda(cudaMemsetAsync(dgamma, 0, cols * 4, s));
  }
  if (!shape_ok(rows, cols)) return FK_ERR_INVALID_ARG;
  if (dy == nullptr || h == nullptr || dx == nullptr) return FK_ERR_INVALID_ARG;
  const size_t es = size_of(dtype), bytes = rows * cols * es;
  const Span sp[6] = {{dy, bytes, es},  {h, bytes, es},  {gamma, cols * 4, 4},
                      {dres, bytes, es}, {dx, bytes, es}, {dgamma, cols * 4, 4}};
  fk_status st = check_spans(sp, 6);
  if (st != FK_OK) return st;
  for (int i : {0, 1, 3})
    if (overlap(sp[4], sp[i]) && !same(sp[4], sp[i])) return FK_ERR_INVALID_ARG;
  if (overlap(sp[4], sp[2])) return FK_ERR_INVALID_ARG;
  for (int i = 0; i < 5; ++i)
    if (overlap(sp[5], sp[i])) return FK_ERR_INVALID_ARG;
  st = check_memory(sp, 6);
  if (st != FK_OK) return st;
  const RmsnormBwdArgs a = {dy, h, gamma, dres, dx, dgamma, rows, cols, dtype, eps,
                            row_mode(cols * es, {dy, h, dres, dx}, gamma, nullptr)};
  // the library takes what this call uses; a caller's is as large as any call of the shape may need
  const size_t need = own ? rmsnorm_bwd_workspace(rows, cols, dtype, dgamma != nullptr, a.mode)
                          : rmsnorm_bwd_workspace(rows, cols, dtype, dgamma != nullptr);
  return with_workspace(need, ws, ws_bytes, own, sp, 6, s,
                        [&](void* w) { return launch_rmsnorm_bwd(a, w, s); });
}

fk_status matmul_call(const void* a, const void* b, const float* a_scales, const float* b_scales, const float* bias,
                      void* c, size_t m, size_t n, size_t k, int dtype, int out_dtype, int epilogue, void* ws,
                      size_t ws_bytes, bool own, void* stream, bool give_up = false) {
  if (!q8_dtype(dtype) || !float_dtype(out_dtype)) return FK_ERR_UNSUPPORTED_DTYPE;
  if (!known_epilogue(epilogue)) return FK_ERR_INVALID_ARG;
  if (m == 0 || n == 0) return FK_OK;
  constexpr size_t kLimit = (size_t{1} << 31) - 256;  // tile indexes stay in 32 bits
  if (k == 0 || m > kLimit || n > kLimit || k > kLimit || (dtype == FK_I8 && k > 131071)) return FK_ERR_INVALID_ARG;
  if (a == nullptr || b == nullptr || a_scales == nullptr || b_scales == nullptr || c == nullptr)
    return FK_ERR_INVALID_ARG;
  const size_t os = size_of(out_dtype);
  const Span sp[6] = {{a, m * k, 1},      {b, n * k, 1},    {a_scales, m * 4, 4},
                      {b_scales, n * 4, 4}, {bias, n * 4, 4}, {c, m * n * os, os}};
  fk_status st = check_spans(sp, 6);
  if (st != FK_OK) return st;
  for (int i = 0; i < 5; ++i)
    if (overlap(sp[5], sp[i])) return FK_ERR_INVALID_ARG;
  st = check_memory(sp, 6);
  if (st != FK_OK) return st;
  const DeviceInfo* dev = current_device_info(nullptr);
  if (dev == nullptr) return FK_ERR_UNSUPPORTED_DEVICE;
  const MatmulQ8Args args = {a, b, a_scales, b_scales, bias, c, m, n, k, dtype, out_dtype, epilogue, give_up};
  const size_t need = matmul_q8_workspace(m, n, k, aligned16(a) && aligned16(b));
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  return with_workspace(need, ws, ws_bytes, own, sp, 6, s,
                        [&](void* w) { return launch_matmul_q8(args, w, dev->sm_count, s); });
}

}  // namespace
}  // namespace fk

extern "C" {

fk_status fk_rmsnorm_rows(const void* x, const void* residual, const float* gamma, void* y, float* scales, void* h,
                          size_t rows, size_t cols, int dtype, int out_dtype, float eps, void* stream) {
  using namespace fk;
  if (!float_dtype(dtype) || (out_dtype != dtype && !q8_dtype(out_dtype))) return FK_ERR_UNSUPPORTED_DTYPE;
  if (!(eps >= 0.0f) || !(eps <= FLT_MAX)) return FK_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return FK_OK;
  if (!shape_ok(rows, cols)) return FK_ERR_INVALID_ARG;
  const bool q8 = q8_dtype(out_dtype);
  if (x == nullptr || y == nullptr || q8 != (scales != nullptr) || (h != nullptr && residual == nullptr))
    return FK_ERR_INVALID_ARG;
  const size_t es = size_of(dtype), n = rows * cols;
  const Span sx = {x, n * es, es}, sr = {residual, n * es, es}, sg = {gamma, cols * 4, 4},
             sy = {y, n * size_of(out_dtype), size_of(out_dtype)}, ss = {scales, rows * 4, 4}, sh = {h, n * es, es};
  const Span sp[6] = {sx, sr, sg, sy, ss, sh};
  fk_status st = check_spans(sp, 6);
  if (st != FK_OK) return st;
  for (const Span* in : {&sx, &sr}) {
    if (overlap(sh, *in) && !same(sh, *in)) return FK_ERR_INVALID_ARG;
    if (overlap(sy, *in) && (q8 || !same(sy, *in))) return FK_ERR_INVALID_ARG;
    if (overlap(ss, *in)) return FK_ERR_INVALID_ARG;
  }
  if (overlap(sy, sg) || overlap(ss, sg) || overlap(sh, sg)) return FK_ERR_INVALID_ARG;
  if (overlap(sy, ss) || overlap(sy, sh) || overlap(ss, sh)) return FK_ERR_INVALID_ARG;
  st = check_memory(sp, 6);
  if (st != FK_OK) return st;
  const RowMode mode = row_mode(cols * es, {x, residual, h, q8 ? nullptr : y}, gamma, q8 ? y : nullptr);
  const RmsnormArgs a = {x, residual, gamma, y, scales, h, rows, cols, dtype, out_dtype, eps, mode};
  return report_cuda(launch_rmsnorm(a, static_cast<cudaStream_t>(stream)));
}

fk_status fk_rmsnorm_rows_bwd(const void* dy, const void* h, const float* gamma, const void* dres, void* dx,
                              float* dgamma, size_t rows, size_t cols, int dtype, float eps, void* stream) {
  return fk::rmsnorm_bwd_call(dy, h, gamma, dres, dx, dgamma, rows, cols, dtype, eps, nullptr, 0, true, stream);
}

fk_status fk_rmsnorm_rows_bwd_ws(const void* dy, const void* h, const float* gamma, const void* dres, void* dx,
                                 float* dgamma, size_t rows, size_t cols, int dtype, float eps, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  return fk::rmsnorm_bwd_call(dy, h, gamma, dres, dx, dgamma, rows, cols, dtype, eps, workspace, workspace_bytes,
                              false, stream);
}

fk_status fk_rmsnorm_rows_bwd_workspace(size_t rows, size_t cols, int dtype, int want_dgamma, size_t* bytes) {
  if (bytes == nullptr) return FK_ERR_INVALID_ARG;
  if (!fk::float_dtype(dtype)) return FK_ERR_UNSUPPORTED_DTYPE;
  *bytes = 0;
  if (rows == 0 || cols == 0) return FK_OK;
  if (!fk::shape_ok(rows, cols)) return FK_ERR_INVALID_ARG;
  *bytes = fk::rmsnorm_bwd_workspace(rows, cols, dtype, want_dgamma != 0);
  return FK_OK;
}

fk_status fk_quantize_rows(const void* x, void* q, float* scales, size_t rows, size_t cols, int dtype,
                           int out_dtype, int epilogue, void* stream) {
  using namespace fk;
  if (!float_dtype(dtype) || !q8_dtype(out_dtype)) return FK_ERR_UNSUPPORTED_DTYPE;
  if (!known_epilogue(epilogue)) return FK_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return FK_OK;
  if (!shape_ok(rows, cols)) return FK_ERR_INVALID_ARG;
  if (x == nullptr || q == nullptr || scales == nullptr) return FK_ERR_INVALID_ARG;
  const size_t es = size_of(dtype), n = rows * cols;
  const Span sp[3] = {{x, n * es, es}, {q, n, 1}, {scales, rows * 4, 4}};
  fk_status st = check_spans(sp, 3);
  if (st != FK_OK) return st;
  if (overlap(sp[0], sp[1]) || overlap(sp[0], sp[2]) || overlap(sp[1], sp[2])) return FK_ERR_INVALID_ARG;
  st = check_memory(sp, 3);
  if (st != FK_OK) return st;
  const QuantizeArgs a = {x, q, scales, rows, cols, dtype, out_dtype, epilogue, row_mode(cols * es, {x}, nullptr, q)};
  return report_cuda(launch_quantize(a, static_cast<cudaStream_t>(stream)));
}

fk_status fk_matmul_q8(const void* a, const void* b, const float* a_scales, const float* b_scales, const float* bias,
                       void* c, size_t m, size_t n, size_t k, int dtype, int out_dtype, int epilogue, void* stream) {
  return fk::matmul_call(a, b, a_scales, b_scales, bias, c, m, n, k, dtype, out_dtype, epilogue, nullptr, 0, true,
                         stream);
}

fk_status fk_matmul_q8_ws(const void* a, const void* b, const float* a_scales, const float* b_scales,
                          const float* bias, void* c, size_t m, size_t n, size_t k, int dtype, int out_dtype,
                          int epilogue, void* workspace, size_t workspace_bytes, void* stream) {
  return fk::matmul_call(a, b, a_scales, b_scales, bias, c, m, n, k, dtype, out_dtype, epilogue, workspace,
                         workspace_bytes, false, stream);
}

fk_status fk_matmul_q8_wait_selftest(const void* a, const void* b, const float* a_scales, const float* b_scales,
                                     float* c, size_t m, size_t n, size_t k, int dtype, void* stream) {
  return fk::matmul_call(a, b, a_scales, b_scales, nullptr, c, m, n, k, dtype, FK_F32, FK_EPILOGUE_NONE, nullptr, 0,
                         true, stream, true);
}

fk_status fk_matmul_q8_workspace(size_t m, size_t n, size_t k, int aligned, size_t* bytes) {
  if (bytes == nullptr) return FK_ERR_INVALID_ARG;
  constexpr size_t kLimit = (size_t{1} << 31) - 256;  // tile indexes stay in 32 bits
  *bytes = 0;
  if (m == 0 || n == 0) return FK_OK;
  if (k == 0 || m > kLimit || n > kLimit || k > kLimit) return FK_ERR_INVALID_ARG;
  *bytes = fk::matmul_q8_workspace(m, n, k, aligned != 0);
  return FK_OK;
}

}  // extern "C"
