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
         (T == 0 || rows < kInt8MaxOut / T);
}

// The kernel and the split of the reduction with the least estimated time.
// The estimates (microseconds) are fits to a sweep of every kernel and split
// over 16 weights from 512 x 16384 to 16384 x 16384 and 4 .. 4096 tokens, three
// of each shape in turn (up to about 85 MB each they stay in the last-level
// cache); they rank the choices (on average 1% behind the best of the sweep, at
// worst 21%) and are no prediction of the time.
//   tiles: rounds of 256 workgroups, each (its 128-wide steps + 4 for the
//   pipeline's ends) times the tile's step; a split adds the write and read of
//   its int32 partials at 2.2 TB/s and a second launch.  (A CU holds two 64 x
//   128 workgroups.  Rounds of 512 for them, with a step of their own, ranked
//   the sweep worse, 4.7% behind the best.)  An unsplit reduction of 100 steps
//   and more over a weight of 10^8 and more takes 1.15 to 1.25 times its steps;
//   without the factor the sweep's picks are 1.3 instead of 1.1% behind;
//   streaming: the wave's chain over K, and T bytes read for every 16 weights.
// Both sides of the choices: 211 x 4096 x 11008 takes 22.4 to 23.2 us with 64 x
// 128 tiles in 2 splits, 22.7 to 23.0 with 128 x 128 ones in 3, 32.1 with 256 x
// 256 ones in 8; 640 x 4096 x 11008 38.4 us with 128 x 128 tiles unsplit, 50 us
// with 128 x 256 ones in 3; 640 x 8192 x 22016 128 us with 256 x 256 tiles in 2
// splits, 153 us with 128 x 256 ones unsplit; but 400 x 8192 x 22016 91 us as
// picked, 128 x 256 tiles in 2, and 83 us with 128 x 128 ones unsplit; 8192 x
// 11008 x 4096 329 us with 256 x 256 tiles, 388 us with 128 x 128; 16 x 4096 x
// 4096 6.7 us streamed, 9.3 us in tiles; 64 x 22016 x 8192 43 us in tiles, 114 us
// streamed.
Int8Plan int8_plan(int64_t T, int64_t rows, int64_t cols, bool with_codes) {
  struct Tile {
    Int8Path path;
    int64_t tm, tn;
    double step;
  };
  static const Tile tiles[4] = {{kInt8Tile64x128, 64, 128, 0.35},
                                {kInt8Tile128x128, 128, 128, 0.47},
                                {kInt8Tile128x256, 128, 256, 0.69},
                                {kInt8Tile256x256, 256, 256, 1.05}};
  static const uint32_t split_counts[8] = {1, 2, 3, 4, 6, 8, 12, 16};
  Int8Plan p;
  p.path = kInt8Tile256x256;
  p.splits = 1;
  double best = -1.0;
  if (T <= kInt8SkinnyTokens) {
    const double t16 = (double)T / 16.0;
    p.path = kInt8Skinny;
    best = 2.3 + 3.3e-4 * (double)cols * (1.0 + 0.66 * t16) +
           (double)rows * (double)cols * (1.0 / 58e6 + t16 / 9.9e6);
  }
  const uint32_t steps = (uint32_t)((cols + 127) / 128);
  const bool long_stream = steps >= 100 && (double)rows * (double)cols >= 1e8;
  constexpr double kLongStream = 1.18;
  const double partials = 8.0 * (double)T * (double)rows / 2.2e6;
  for (const Tile& t : tiles) {
    const int64_t n = ((T + t.tm - 1) / t.tm) * ((rows + t.tn - 1) / t.tn);
    for (uint32_t s : split_counts) {
      if (s > 1 && steps < 2 * s) break;
      const int64_t rounds = (n * s + kGemmCUs - 1) / kGemmCUs;
      const double step = s == 1 && long_stream ? kLongStream * t.step : t.step;
      double c = 1.5 + (double)rounds * step * (double)((steps + s - 1) / s + 4);
      if (s > 1) c += 2.0 + partials * (double)s;
      if (best < 0.0 || c < best) {
        best = c;
        p.path = t.path;
        p.splits = (int)s;
      }
    }
  }
  if (with_codes && p.path == kInt8Skinny && T <= 16 && T * cols <= kInt8FusedBytes) {
    p.path = kInt8Fused;
    with_codes = false;
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
  if (!given && p.path != kInt8Fused) {
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
  if (e == hipSuccess) e = launch_int8_product(a, X16, p, compute_dtype == QLORA_COMPUTE_FP16, st);
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
