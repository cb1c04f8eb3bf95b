// C ABI of the 8-bit linear layer: validate on the host, then enqueue the
// kernels of int8.hip on the caller's stream.
#include <hip/hip_runtime_api.h>

#include "abi_internal.h"
#include "int8_kernels.h"
#include "qlora_int8.h"

namespace qlora {

bool int8_row_dims_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows <= kInt8MaxDim && cols >= 16 && cols <= kInt8MaxCols && cols % 16 == 0;
}

bool int8_dims_ok(int64_t T, int64_t rows, int64_t cols) {
  return int8_row_dims_ok(T, cols) && int8_row_dims_ok(rows, cols) && rows >= 1 &&
         (T == 0 || rows < (int64_t(1) << 40) / T);
}

Int8Plan int8_plan(int64_t T, int64_t rows, int64_t cols, bool with_codes) {
  Int8Plan p;
  p.splits = 1;
  if (T <= kInt8SkinnyTokens) {
    p.path = kInt8Skinny;
  } else {
    const int64_t tiles256 = ((T + 255) / 256) * ((rows + 255) / 256);
    p.path = tiles256 >= kGemmCUs ? kInt8Tile256 : kInt8Tile128;
  }
  size_t off = 0;
  p.codes_off = off;
  if (with_codes) off += align_up((size_t)T * (size_t)cols, kWsAlign);
  p.scale_off = off;
  if (with_codes) off += align_up(sizeof(float) * (size_t)T, kWsAlign);
  p.part_off = off;
  if (p.splits > 1)
    off += align_up(sizeof(int32_t) * (size_t)p.splits * (size_t)T * (size_t)rows, kWsAlign);
  p.total = off;
  return p;
}

namespace {

qlora_status hip_status(hipError_t e) {
  if (e == hipSuccess) return QLORA_OK;
  set_last_hip_error((int)e);
  return QLORA_ERR_HIP;
}

bool compute_dtype_ok(int d) { return d == QLORA_COMPUTE_BF16 || d == QLORA_COMPUTE_FP16; }

// The product of given codes (X16 NULL) or of 16-bit tokens.
qlora_status product(const int8_t* W, const float* w_scale, int64_t rows, int64_t cols,
                     const int8_t* X, const float* x_scale, const uint16_t* X16, bool given,
                     int64_t T, int compute_dtype, uint16_t* Y, void* ws, size_t ws_bytes,
                     void* stream) {
  if (!compute_dtype_ok(compute_dtype)) return QLORA_ERR_FORMAT;
  if (!int8_dims_ok(T, rows, cols)) return QLORA_ERR_SHAPE;
  if (!W || !w_scale) return QLORA_ERR_NULL;
  if (!aligned16(W) || !aligned16(w_scale)) return QLORA_ERR_ALIGN;
  if (T == 0) return check_device();
  if (!Y || (given ? !X || !x_scale : !X16)) return QLORA_ERR_NULL;
  if (!aligned16(Y) || !aligned16(X) || !aligned16(x_scale) || !aligned16(X16))
    return QLORA_ERR_ALIGN;
  const Int8Plan p = int8_plan(T, rows, cols, !given);
  if (p.total > 0) {
    if (!ws) return QLORA_ERR_NULL;
    if (!aligned16(ws)) return QLORA_ERR_ALIGN;
    if (ws_bytes < p.total) return QLORA_ERR_WORKSPACE;
  }
  const qlora_status s = check_device();
  if (s != QLORA_OK) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* base = static_cast<char*>(ws);
  Int8Args a;
  a.X = X;
  a.x_scale = x_scale;
  a.W = W;
  a.w_scale = w_scale;
  a.T = T;
  a.rows = rows;
  a.cols = cols;
  a.Y = Y;
  a.splits = p.splits;
  a.part = p.splits > 1 ? reinterpret_cast<int32_t*>(base + p.part_off) : nullptr;
  hipError_t e = hipSuccess;
  if (!given) {
    Int8QuantArgs q;
    q.X = X16;
    q.rows = T;
    q.cols = cols;
    q.codes = reinterpret_cast<int8_t*>(base + p.codes_off);
    q.scale = reinterpret_cast<float*>(base + p.scale_off);
    a.X = q.codes;
    a.x_scale = q.scale;
    e = launch_int8_quantize(q, compute_dtype, st);
  }
  if (e == hipSuccess) e = launch_int8_product(a, p, compute_dtype == QLORA_COMPUTE_FP16, st);
  return hip_status(e);
}

}  // namespace

}  // namespace qlora

extern "C" {

qlora_status qlora_int8_quantize(const void* X, int x_type, int64_t rows, int64_t cols,
                                 int8_t* codes, float* scale, void* stream) {
  using namespace qlora;
  if (x_type != QLORA_TYPE_BF16 && x_type != QLORA_TYPE_FP16 && x_type != QLORA_TYPE_FP32)
    return QLORA_ERR_FORMAT;
  if (!int8_row_dims_ok(rows, cols)) return QLORA_ERR_SHAPE;
  if (rows == 0) return check_device();
  if (!X || !codes || !scale) return QLORA_ERR_NULL;
  if (!aligned16(X) || !aligned16(codes) || !aligned16(scale)) return QLORA_ERR_ALIGN;
  const qlora_status s = check_device();
  if (s != QLORA_OK) return s;
  Int8QuantArgs a;
  a.X = X;
  a.rows = rows;
  a.cols = cols;
  a.codes = codes;
  a.scale = scale;
  return hip_status(launch_int8_quantize(a, x_type, static_cast<hipStream_t>(stream)));
}

size_t qlora_int8_workspace(int64_t T, int64_t rows, int64_t cols, int x_given) {
  if (!qlora::int8_dims_ok(T, rows, cols) || T == 0) return 0;
  return qlora::int8_plan(T, rows, cols, x_given == 0).total;
}

qlora_status qlora_int8_matmul(const int8_t* W, const float* w_scale, int64_t rows, int64_t cols,
                               const int8_t* X, const float* x_scale, int64_t T,
                               int compute_dtype, uint16_t* Y, void* ws, size_t ws_bytes,
                               void* stream) {
  return qlora::product(W, w_scale, rows, cols, X, x_scale, nullptr, true, T, compute_dtype, Y, ws,
                        ws_bytes, stream);
}

qlora_status qlora_int8_linear_fwd(const int8_t* W, const float* w_scale, int64_t rows,
                                   int64_t cols, const uint16_t* X, int64_t T, int compute_dtype,
                                   uint16_t* Y, void* ws, size_t ws_bytes, void* stream) {
  return qlora::product(W, w_scale, rows, cols, nullptr, nullptr, X, false, T, compute_dtype, Y,
                        ws, ws_bytes, stream);
}

}  // extern "C"
