// C ABI of the microscaled operators (declared in include/hsl.h): argument checks,
// workspace layout and the choice of kernel.  Nothing is kept between calls: all
// data, the workspace included, is the caller's.
#include <algorithm>
#include <atomic>
#include <cstdio>
#include <initializer_list>

#include "common.cuh"
#include "internal.h"
#include "mx.cuh"
#include "mx_ops.h"

namespace hsl {
namespace {

hsl_status bad_arg(const char* why) {
  set_message(why);
  return HSL_ERR_INVALID_ARG;
}
hsl_status bad_arg(const char* what, const char* why) {
  char text[96];
  std::snprintf(text, sizeof(text), "%s%s", what, why);
  return bad_arg(text);
}
hsl_status not_supported(const char* why) {
  set_message(why);
  return HSL_ERR_UNSUPPORTED;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }
bool dtype_ok(hsl_dtype d) { return d == HSL_F32 || d == HSL_BF16; }
constexpr int64_t kMaxSize = int64_t(1) << 30;  // rows, columns, tokens: indices stay in 32 bits
bool size_ok(int64_t v) { return v >= 1 && v <= kMaxSize; }

// The checks that every operator makes of a matrix in blocks.
hsl_status check_mx(const hsl_mx* q, int elem, const char* what) {
  if (!q) return bad_arg(what, " is NULL");
  if (q->elem != HSL_MX_E2M1 && q->elem != HSL_MX_INT8) return bad_arg(what, ": unknown element type");
  if (elem >= 0 && int(q->elem) != elem)
    return not_supported(elem == HSL_MX_E2M1 ? "the weights must hold e2m1 blocks"
                                             : "the checkpoint must hold int8 blocks");
  if (q->rows < 0 || q->rows > kMaxSize || !size_ok(q->cols)) return bad_arg(what, ": rows or cols out of range");
  if (q->rows > 0 && (!q->codes || !q->scales)) return bad_arg(what, ": codes/scales is NULL");
  if (!aligned16(q->codes) || !aligned16(q->scales))
    return bad_arg(what, ": codes and scales must be 16-byte aligned");
  return HSL_OK;
}

// A call's outputs and scratch may not share memory with each other or with its inputs.
struct Span {
  const void* p;
  int64_t bytes;
};
bool meet(const Span& a, const Span& b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  return a.p && b.p && x < y + uintptr_t(b.bytes) && y < x + uintptr_t(a.bytes);
}
hsl_status check_apart(std::initializer_list<Span> out, std::initializer_list<Span> in) {
  for (const Span* o = out.begin(); o != out.end(); ++o) {
    for (const Span* p = out.begin(); p != o; ++p)
      if (meet(*o, *p)) return bad_arg("two outputs, or an output and the workspace, overlap");
    for (const Span& i : in)
      if (meet(*o, i)) return bad_arg("an output or the workspace overlaps an input");
  }
  return HSL_OK;
}
Span codes_of(const hsl_mx* q) {
  return {q->codes, q->rows * mx::code_pitch(q->cols, q->elem == HSL_MX_INT8)};
}
Span scales_of(const hsl_mx* q) { return {q->scales, q->rows * mx::scale_pitch(q->cols)}; }
int64_t size_of(hsl_dtype d) { return d == HSL_F32 ? 4 : 2; }
// Matrices start on a whole element (the kernels load elements at least).
hsl_status check_whole(std::initializer_list<const void*> ps, hsl_dtype d) {
  for (const void* p : ps)
    if (reinterpret_cast<uintptr_t>(p) % size_of(d)) return bad_arg("a matrix does not start on a whole element");
  return HSL_OK;
}
// add may be the output itself
Span add_of(const void* add, const void* out, int64_t bytes) { return {add == out ? nullptr : add, bytes}; }

MxOperand operand(const hsl_mx* q, bool trans) {
  MxOperand o;
  o.p = q->codes;
  o.scales = static_cast<const uint8_t*>(q->scales);
  o.pitch = mx::code_pitch(q->cols, q->elem == HSL_MX_INT8);
  o.spitch = mx::scale_pitch(q->cols);
  o.kind = q->elem == HSL_MX_INT8 ? MxOperand::kInt8 : MxOperand::kE2M1;
  o.trans = trans ? 1 : 0;
  o.vec = 0;
  return o;
}
MxOperand operand(const void* p, hsl_dtype dt, int64_t pitch, bool trans) {
  MxOperand o;
  o.p = p;
  o.scales = nullptr;
  o.pitch = pitch;
  o.spitch = 0;
  o.kind = dt == HSL_F32 ? MxOperand::kF32 : MxOperand::kBF16;
  o.trans = trans ? 1 : 0;
  o.vec = dt == HSL_F32 && pitch % 4 == 0 && aligned16(p) ? 1 : 0;
  return o;
}

// Scratch of the fp32 kernels: Z and G of the factor gradients, then a product's K ranges.
size_t zg_bytes(int64_t T, int64_t r) { return size_t(round_up(2 * T * r * 4, 256)); }
size_t simt_bytes(hsl_mx_op op, int64_t T, int64_t m, int64_t n, int64_t r) {
  switch (op) {
    case HSL_MX_OP_APPLY: return mx_simt_workspace(T, m, n);
    case HSL_MX_OP_APPLY_T: return mx_simt_workspace(T, n, m);
    case HSL_MX_OP_MATMUL: return mx_simt_workspace(T, m, n);
    default: break;
  }
  if (r == 0) return 0;
  const size_t parts[] = {mx_simt_workspace(T, r, n), mx_simt_workspace(T, r, m), mx_simt_workspace(m, r, T),
                          mx_simt_workspace(n, r, T), mx_simt_workspace(T, n, r)};
  return zg_bytes(T, r) + *std::max_element(parts, parts + 5);
}
// Whether a call takes the tensor-core kernels is decided by its sizes here and by the alignment of its
// pointers at the call, so the scratch holds either.
size_t workspace_bytes(hsl_mx_op op, int64_t T, int64_t m, int64_t n, int64_t r, hsl_dtype dt) {
  if (T == 0 || m == 0) return simt_bytes(op, T, m, n, r);
  if (op == HSL_MX_OP_MATMUL) return mx_matmul_supported() ? 0 : simt_bytes(op, T, m, n, r);
  if (dt == HSL_F32) {
    if (op == HSL_MX_OP_APPLY && T <= kMxDecodeF32Max) return mx_decode_f32_workspace(T, m, n);
    return simt_bytes(op, T, m, n, r);
  }
  if (op == HSL_MX_OP_APPLY && mx_decode_fits(T, m, n)) return mx_decode_workspace(T, n);
  const size_t tc = op == HSL_MX_OP_FACTOR_GRAD ? (r > 0 ? mx_gemm_grad_workspace(T, m, n, r) : 0)
                                                : mx_gemm_apply_workspace(op == HSL_MX_OP_APPLY_T, T, m, n);
  return std::max(tc, simt_bytes(op, T, m, n, r));
}

hsl_status check_workspace(const void* ws, size_t have, size_t need) {
  if (need == 0) return HSL_OK;
  if (!ws || have < need) {
    char text[64];
    std::snprintf(text, sizeof(text), "workspace too small: %zu bytes needed", need);
    return bad_arg(text);
  }
  if (!aligned16(ws)) return bad_arg("workspace must be 16-byte aligned");
  return HSL_OK;
}

// The error words of the kernels' files, read and cleared in one step each, so that no report falls between the two.
struct ErrorWords {
  uint32_t* p[4];
};
constexpr unsigned kTakeSlots = 64;  // checks under way at a time
__device__ uint32_t g_mx_taken[kTakeSlots];
__global__ void k_mx_take(const ErrorWords w, uint32_t* out, bool inject) {
  if (inject) set_error(w.p[0], kErrTimeout);
  uint32_t all = 0;
  for (uint32_t* p : w.p) all |= atomicExch(p, 0u);
  *out = all;
}

}  // namespace
}  // namespace hsl

using namespace hsl;

extern "C" {

hsl_status hsl_mx_pitch(int64_t cols, hsl_mx_elem elem, int64_t* code_pitch, int64_t* scale_pitch) {
  set_message("");
  if (!code_pitch || !scale_pitch) return bad_arg("NULL argument");
  if (elem != HSL_MX_E2M1 && elem != HSL_MX_INT8) return bad_arg("unknown element type");
  if (!size_ok(cols)) return bad_arg("cols out of range");
  *code_pitch = mx::code_pitch(cols, elem == HSL_MX_INT8);
  *scale_pitch = mx::scale_pitch(cols);
  return HSL_OK;
}

hsl_status hsl_mx_quantize(const void* X, hsl_dtype dtype, int64_t rows, int64_t cols,
                           hsl_mx_elem elem, void* codes, void* scales, hsl_stream s) {
  set_message("");
  if (!dtype_ok(dtype)) return bad_arg("unknown dtype");
  const hsl_mx q = {codes, scales, rows, cols, elem};
  if (hsl_status e = check_mx(&q, -1, "the result")) return e;
  if (rows == 0) return HSL_OK;
  if (!X) return bad_arg("X is NULL");
  if (hsl_status e = check_whole({X}, dtype)) return e;
  if (hsl_status e = check_apart({codes_of(&q), scales_of(&q)}, {{X, rows * cols * size_of(dtype)}})) return e;
  return mx_quantize_run(X, dtype, rows, cols, elem == HSL_MX_INT8, codes, scales,
                         static_cast<cudaStream_t>(s));
}

hsl_status hsl_mx_dequantize(const hsl_mx* q, void* X, hsl_dtype dtype, hsl_stream s) {
  set_message("");
  if (!dtype_ok(dtype)) return bad_arg("unknown dtype");
  if (hsl_status e = check_mx(q, -1, "the matrix")) return e;
  if (q->rows == 0) return HSL_OK;
  if (!X) return bad_arg("X is NULL");
  if (hsl_status e = check_whole({X}, dtype)) return e;
  if (hsl_status e = check_apart({{X, q->rows * q->cols * size_of(dtype)}}, {codes_of(q), scales_of(q)})) return e;
  return mx_dequantize_run(q->codes, q->scales, q->rows, q->cols, q->elem == HSL_MX_INT8, X, dtype,
                           static_cast<cudaStream_t>(s));
}

hsl_status hsl_mx_workspace(hsl_mx_op op, int64_t batch, int64_t m, int64_t n, int64_t r,
                            hsl_dtype dtype, size_t* bytes) {
  set_message("");
  if (!bytes) return bad_arg("bytes is NULL");
  if (op < HSL_MX_OP_APPLY || op > HSL_MX_OP_FACTOR_GRAD) return bad_arg("unknown operator");
  if (!dtype_ok(dtype)) return bad_arg("unknown dtype");
  if (batch < 0 || batch > kMaxSize || m < 0 || m > kMaxSize || !size_ok(n) || r < 0 || r > 256)
    return bad_arg("a size is out of range");
  *bytes = workspace_bytes(op, batch, m, n, r, dtype);
  return HSL_OK;
}

hsl_status hsl_mx4_apply(const hsl_mx* D, const void* X, const void* add, void* Y, int64_t batch,
                         hsl_dtype dtype, void* ws, size_t ws_bytes, hsl_stream stream) {
  set_message("");
  if (!dtype_ok(dtype)) return bad_arg("unknown dtype");
  if (hsl_status e = check_mx(D, HSL_MX_E2M1, "D")) return e;
  if (batch < 0 || batch > kMaxSize) return bad_arg("batch out of range");
  if (batch == 0 || D->rows == 0) return HSL_OK;
  if (!X || !Y) return bad_arg("X/Y is NULL");
  if (hsl_status e = check_whole({X, add, Y}, dtype)) return e;
  const size_t need = workspace_bytes(HSL_MX_OP_APPLY, batch, D->rows, D->cols, 0, dtype);
  if (hsl_status e = check_workspace(ws, ws_bytes, need)) return e;
  const int64_t xb = batch * D->cols * size_of(dtype), yb = batch * D->rows * size_of(dtype);
  if (hsl_status e = check_apart({{Y, yb}, {ws, int64_t(need)}},
                                 {{X, xb}, add_of(add, Y, yb), codes_of(D), scales_of(D)}))
    return e;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == HSL_BF16 && mx_decode_fits(batch, D->rows, D->cols))
    return mx_decode_run(operand(D, false), D->rows, D->cols, X, add, Y, batch, ws, s);
  if (dtype == HSL_BF16 && mx_gemm_supported(X))
    return mx_gemm_apply_run(false, operand(D, false), D->rows, D->cols, X, add, Y, batch, ws, s);
  if (dtype == HSL_F32 && batch <= kMxDecodeF32Max)
    return mx_decode_f32_run(operand(D, false), D->rows, D->cols, X, add, Y, batch, ws, s);
  return mx_simt_run(operand(X, dtype, D->cols, false), operand(D, false), batch, D->rows, D->cols,
                     add, Y, dtype, ws, false, s);
}

hsl_status hsl_mx4_apply_t(const hsl_mx* D, const void* dY, const void* add, void* dX, int64_t batch,
                           hsl_dtype dtype, void* ws, size_t ws_bytes, hsl_stream stream) {
  set_message("");
  if (!dtype_ok(dtype)) return bad_arg("unknown dtype");
  if (hsl_status e = check_mx(D, HSL_MX_E2M1, "D")) return e;
  if (batch < 0 || batch > kMaxSize) return bad_arg("batch out of range");
  if (batch == 0) return HSL_OK;
  if (!dX || (D->rows > 0 && !dY)) return bad_arg("dY/dX is NULL");
  if (hsl_status e = check_whole({dY, add, dX}, dtype)) return e;
  const size_t need = workspace_bytes(HSL_MX_OP_APPLY_T, batch, D->rows, D->cols, 0, dtype);
  if (hsl_status e = check_workspace(ws, ws_bytes, need)) return e;
  const int64_t xb = batch * D->cols * size_of(dtype), yb = batch * D->rows * size_of(dtype);
  if (hsl_status e = check_apart({{dX, xb}, {ws, int64_t(need)}},
                                 {{dY, yb}, add_of(add, dX, xb), codes_of(D), scales_of(D)}))
    return e;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == HSL_BF16 && D->rows > 0 && mx_gemm_supported(dY))
    return mx_gemm_apply_run(true, operand(D, true), D->rows, D->cols, dY, add, dX, batch, ws, s);
  return mx_simt_run(operand(dY, dtype, D->rows, false), operand(D, true), batch, D->cols, D->rows,
                     add, dX, dtype, ws, false, s);
}

hsl_status hsl_mx4_matmul(const hsl_mx* A, const hsl_mx* B, const void* add, void* Y, hsl_dtype dtype,
                          void* ws, size_t ws_bytes, hsl_stream stream) {
  set_message("");
  if (!dtype_ok(dtype)) return bad_arg("unknown dtype");
  if (hsl_status e = check_mx(A, HSL_MX_E2M1, "A")) return e;
  if (hsl_status e = check_mx(B, HSL_MX_E2M1, "B")) return e;
  if (A->cols != B->cols) return bad_arg("A and B must have the same number of columns");
  if (A->rows == 0 || B->rows == 0) return HSL_OK;
  if (!Y) return bad_arg("Y is NULL");
  if (hsl_status e = check_whole({add, Y}, dtype)) return e;
  const size_t need = workspace_bytes(HSL_MX_OP_MATMUL, A->rows, B->rows, A->cols, 0, dtype);
  if (hsl_status e = check_workspace(ws, ws_bytes, need)) return e;
  const int64_t yb = A->rows * B->rows * size_of(dtype);
  if (hsl_status e = check_apart({{Y, yb}, {ws, int64_t(need)}},
                                 {add_of(add, Y, yb), codes_of(A), scales_of(A), codes_of(B), scales_of(B)}))
    return e;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (mx_matmul_supported())
    return mx_matmul_run(operand(A, false), A->rows, operand(B, false), B->rows, A->cols, add, Y, dtype, s);
  return mx_simt_run(operand(A, false), operand(B, false), A->rows, B->rows, A->cols, add, Y, dtype, ws, false, s);
}

hsl_status hsl_mx8_factor_grad(const hsl_mx* X, const void* dY, int64_t m, const void* U,
                               const void* V, int32_t r, const void* add, void* dU, void* dV, void* dX,
                               hsl_dtype dtype, void* ws, size_t ws_bytes, hsl_stream stream) {
  set_message("");
  if (!dtype_ok(dtype)) return bad_arg("unknown dtype");
  if (hsl_status e = check_mx(X, HSL_MX_INT8, "X")) return e;
  if (!size_ok(m)) return bad_arg("m out of range");
  if (r < 1 || r > 256) return not_supported("need 1 <= r <= 256");
  if (!U || !V || !dU || !dV) return bad_arg("U/V/dU/dV is NULL");
  if (add && !dX) return bad_arg("add without dX");
  const int64_t T = X->rows, n = X->cols;
  if (T > 0 && !dY) return bad_arg("dY is NULL");
  if (hsl_status e = check_whole({dY, U, V, add, dU, dV, dX}, dtype)) return e;
  const size_t need = workspace_bytes(HSL_MX_OP_FACTOR_GRAD, T, m, n, r, dtype);
  if (hsl_status e = check_workspace(ws, ws_bytes, need)) return e;
  const int64_t eb = size_of(dtype), ub = m * r * eb, vb = n * r * eb, xb = T * n * eb;
  if (hsl_status e = check_apart(
          {{dU, ub}, {dV, vb}, {dX, xb}, {ws, int64_t(need)}},
          {{dY, T * m * eb}, {U, ub}, {V, vb}, add_of(add, dX, xb), codes_of(X), scales_of(X)}))
    return e;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == HSL_BF16 && T > 0 && mx_gemm_supported(dY) && mx_gemm_supported(U) && mx_gemm_supported(V))
    return mx_gemm_grad_run(operand(X, false), T, n, dY, m, U, V, r, add, dU, dV, dX, ws, s);
  float* Z = static_cast<float*>(ws);
  float* G = Z ? Z + T * r : nullptr;
  void* part = Z ? static_cast<char*>(ws) + zg_bytes(T, r) : nullptr;
  const MxOperand x = operand(X, false), xt = operand(X, true);
  if (hsl_status e = mx_simt_run(x, operand(V, dtype, r, true), T, r, n, nullptr, Z, HSL_F32, part, false, s)) return e;
  if (hsl_status e = mx_simt_run(operand(dY, dtype, m, false), operand(U, dtype, r, true), T, r, m,
                                 nullptr, G, HSL_F32, part, T > 0, s))
    return e;
  if (hsl_status e = mx_simt_run(operand(dY, dtype, m, true), operand(Z, HSL_F32, r, true), m, r, T,
                                 nullptr, dU, dtype, part, T > 0, s))
    return e;
  if (hsl_status e = mx_simt_run(xt, operand(G, HSL_F32, r, true), n, r, T, nullptr, dV, dtype, part, true, s))
    return e;
  if (!dX) return HSL_OK;
  return mx_simt_run(operand(G, HSL_F32, r, false), operand(V, dtype, r, false), T, n, r, add, dX, dtype,
                     part, true, s);
}

hsl_status hsl_mx_check(hsl_stream stream) {
  set_message("");
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  ErrorWords w = {};
  uint32_t* taken = nullptr;
  if (cudaError_t e = mx_gemm_error_word(&w.p[0])) return cuda_fail(e, "error word address");
  if (cudaError_t e = mx_matmul_error_word(&w.p[1])) return cuda_fail(e, "error word address");
  if (cudaError_t e = mx_decode_error_word(&w.p[2])) return cuda_fail(e, "error word address");
  if (cudaError_t e = mx_grad_error_word(&w.p[3])) return cuda_fail(e, "error word address");
  if (cudaError_t e = cudaGetSymbolAddress(reinterpret_cast<void**>(&taken), g_mx_taken))
    return cuda_fail(e, "error word address");
  static std::atomic<unsigned> next{0};
  taken += next++ % kTakeSlots;
  // HSL_FAULT_INJECT=mxwait: as if a wait had given up (host-side failure testing)
  note_launch();
  k_mx_take<<<1, 1, 0, s>>>(w, taken, fault_injected("mxwait"));
  if (cudaError_t e = cudaGetLastError()) return cuda_fail(e, "error check launch");
  uint32_t all = 0;
  if (cudaError_t e = cudaMemcpyAsync(&all, taken, 4, cudaMemcpyDeviceToHost, s)) return cuda_fail(e, "error word read");
  if (cudaError_t e = cudaStreamSynchronize(s)) return cuda_fail(e, "stream synchronize");
  if (all == 0) return HSL_OK;
  set_message("a bounded device wait gave up");
  return HSL_ERR_TIMEOUT;
}

}  // extern "C"
