// C ABI of the linear layer and the gated block in 8-bit floating point:
// validate on the host, then enqueue the kernels of fp8.hip on the caller's
// stream.
#include <hip/hip_runtime_api.h>

#include "abi_internal.h"
#include "fp8_kernels.h"
#include "qlora_fp8.h"

namespace qlora {

bool fp8_row_dims_ok(int64_t rows, int64_t cols) {
  return rows >= 0 && rows <= kFp8MaxDim && cols >= 16 && cols <= kFp8MaxCols && cols % 16 == 0;
}

bool fp8_dims_ok(int64_t T, int64_t rows, int64_t cols, int64_t outs) {
  return fp8_row_dims_ok(T, cols) && fp8_row_dims_ok(rows, cols) && rows >= 1 &&
         (T == 0 || outs < kFp8MaxOut / T);
}

// The kernel and the split of the reduction with the least estimated time.
// The estimates (microseconds) are fits to a sweep of every kernel and split
// over 21 weights from 1024 x 1024 to 28672 x 8192 and 1 .. 4096 tokens, each call
// with another copy of the weight, so that it comes from memory as in a model's pass
// (640 MB of copies in turn), and to a lesser part to one over 10 weights of which the
// last-level cache held all calls'.  They rank the choices (on average 1.1% behind the
// best of the first sweep, at worst 17%: 1 x 22016 x 4096; of the second 0.9%, at
// worst 14%) and are no prediction of the time.  They are smooth in the weight's bytes:
// with a step at 10^8 of them, fitted to weights in the cache, 7 x 14336 x 8192 ran
// unsplit, 40 us, where 4 parts take 27.
//   tiles: what one CU has to do, its steps of 128 columns + the pipeline's ends
//   times the tile's step; of the two smaller tiles a CU runs two workgroups at a
//   time, which take `two` a step.  No less than the weights at a rate between the
//   memory's and the cache's (the lesser of the two counts an eighth: many choices
//   end at the same bytes).  A split adds the write and read of its float32 partials
//   and a second launch.
//   streaming: the wave's chain over the columns, and the tokens' codes read for
//   every 16 weights.
Fp8Plan fp8_plan(int64_t T, int64_t outs, int64_t cols, bool x16) {
  struct Tile {
    Fp8Path path;
    int64_t tm, tn;
    double start, one, two, ends;
  };
  static const Tile tiles[4] = {{kFp8Tile64x128, 64, 128, 1.46, 0.399, 0.609, 4.61},
                                {kFp8Tile128x128, 128, 128, 1.97, 0.419, 0.616, 6.71},
                                {kFp8Tile128x256, 128, 256, 0.525, 0.547, 1.094, 11.2},
                                {kFp8Tile256x256, 256, 256, 0.277, 0.888, 1.776, 8.68}};
  static const uint32_t split_counts[8] = {1, 2, 3, 4, 6, 8, 12, 16};
  Fp8Plan p;
  p.path = kFp8Tile256x256;
  p.splits = 1;
  double best = -1.0;
  const double weights = (double)outs * (double)cols;
  if (T <= kFp8SkinnyTokens) {
    const double t16 = (double)T / 16.0;
    p.path = kFp8Skinny;
    best = 2.47 + 3.91e-4 * (double)cols * (1.0 + 0.019 * t16) +
           weights * 1e-6 * (0.263 + 0.0542 * t16);
  }
  const uint32_t steps = (uint32_t)fp8_blocks(cols);
  const double least = 4.81 + weights / 11.5e6;
  for (const Tile& t : tiles) {
    const int64_t n = ((T + t.tm - 1) / t.tm) * ((outs + t.tn - 1) / t.tn);
    for (uint32_t s : split_counts) {
      if (s > 1 && steps < 2 * s) break;
      const int64_t a_cu = (n * s + kGemmCUs - 1) / kGemmCUs;
      double c = t.start + ((double)(a_cu / 2) * t.two + (double)(a_cu % 2) * t.one) *
                               ((double)((steps + s - 1) / s) + t.ends);
      c = c < least ? least + 0.134 * c : c + 0.134 * least;
      if (s > 1) c += 3.82 + 8.0 * (double)T * (double)outs * (double)s / 8.12e6;
      if (best < 0.0 || c < best) {
        best = c;
        p.path = t.path;
        p.splits = (int)s;
      }
    }
  }
  bool with_codes = x16;
  // Tokens quantised inside the streaming kernel, by every workgroup of 16 outputs,
  // and so in the best choice with a launch of their own, us: 1 x 4096 x 4096 7.5 :
  // 9.1, 1 x 28672 x 8192 45.6 : 53.7, 2 x 32000 x 4096 29.9 : 32.8, 8 x 22016 x 1024 9.8 :
  // 10.5; with more than 2^24 codes in all 4 x 65536 x 2048 32.0 : 29.0, 8 x 100000 x
  // 1024 31.1 : 26.1.
  if (x16 && T <= kFp8FusedTokens && T * 128 * (int64_t)steps <= kFp8FusedBytes &&
      T * 8 * (int64_t)steps * outs <= kFp8FusedAll) {
    p.path = kFp8Fused;
    p.splits = 1;
    with_codes = false;
  }
  size_t off = 0;
  p.codes_off = off;
  if (with_codes) off += align_up((size_t)T * (size_t)cols, kWsAlign);
  p.scale_off = off;
  if (with_codes) off += align_up(sizeof(float) * (size_t)T * (size_t)fp8_blocks(cols), kWsAlign);
  p.part_off = off;
  if (p.splits > 1)
    off += align_up(sizeof(float) * (size_t)p.splits * (size_t)T * (size_t)outs, kWsAlign);
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

struct Fp8Mat {
  const uint8_t* codes;
  const float* scale;
};

// The product of given codes (x) or of 16-bit tokens (X16) with one weight, or
// the gated block of two.
qlora_status product(const Fp8Mat (&w)[2], bool gated, int64_t rows, int64_t cols, const Fp8Mat& x,
                     const uint16_t* X16, bool given, int64_t T, int act, int compute_dtype,
                     uint16_t* Y, void* ws, size_t ws_bytes, void* stream) {
  const int64_t outs = gated ? 2 * rows : rows;
  if (!compute_dtype_ok(compute_dtype)) return QLORA_ERR_FORMAT;
  if (gated && act != QLORA_ACT_SILU && act != QLORA_ACT_GELU_TANH) return QLORA_ERR_FORMAT;
  if (!fp8_dims_ok(T, rows, cols, outs)) return QLORA_ERR_SHAPE;
  for (int i = 0; i < (gated ? 2 : 1); ++i) {
    if (!w[i].codes || !w[i].scale) return QLORA_ERR_NULL;
    if (!aligned16(w[i].codes) || !aligned16(w[i].scale)) return QLORA_ERR_ALIGN;
  }
  if (T == 0) return check_device();
  if (!Y || (given ? !x.codes || !x.scale : !X16)) return QLORA_ERR_NULL;
  if (!aligned16(Y) || !aligned16(x.codes) || !aligned16(x.scale) || !aligned16(X16))
    return QLORA_ERR_ALIGN;
  const Fp8Plan p = fp8_plan(T, outs, cols, !given);
  if (p.total > 0) {
    if (!ws) return QLORA_ERR_NULL;
    if (!aligned16(ws)) return QLORA_ERR_ALIGN;
    if (ws_bytes < p.total) return QLORA_ERR_WORKSPACE;
  }
  const qlora_status s = check_device();
  if (s != QLORA_OK) return s;
  hipStream_t st = static_cast<hipStream_t>(stream);
  char* base = static_cast<char*>(ws);
  Fp8Args a;
  a.X = x.codes;
  a.x_scale = x.scale;
  a.X16 = X16;
  for (int i = 0; i < 2; ++i) {
    a.W[i] = w[i].codes;
    a.w_scale[i] = w[i].scale;
  }
  a.T = T;
  a.rows = rows;
  a.cols = cols;
  a.Y = Y;
  a.splits = p.splits;
  a.part = p.splits > 1 ? reinterpret_cast<float*>(base + p.part_off) : nullptr;
  a.act = act;
  hipError_t e = hipSuccess;
  if (!given && p.path != kFp8Fused) {
    Fp8QuantArgs q;
    q.X = X16;
    q.rows = T;
    q.cols = cols;
    q.codes = reinterpret_cast<uint8_t*>(base + p.codes_off);
    q.scale = reinterpret_cast<float*>(base + p.scale_off);
    a.X = q.codes;
    a.x_scale = q.scale;
    e = launch_fp8_quantize(q, compute_dtype, st);
  }
  if (e == hipSuccess)
    e = launch_fp8_product(a, p, gated, compute_dtype == QLORA_COMPUTE_FP16, st);
  return hip_status(e);
}

qlora_status quantize(const void* X, int x_type, int64_t rows, int64_t cols, uint8_t* codes,
                      float* scale, void* stream, bool weight) {
  if (x_type != QLORA_TYPE_BF16 && x_type != QLORA_TYPE_FP16 && x_type != QLORA_TYPE_FP32)
    return QLORA_ERR_FORMAT;
  if (!fp8_row_dims_ok(rows, cols) || (weight && rows < 1)) return QLORA_ERR_SHAPE;
  if (rows == 0) return check_device();
  if (!X || !codes || !scale) return QLORA_ERR_NULL;
  if (!aligned16(X) || !aligned16(codes) || !aligned16(scale)) return QLORA_ERR_ALIGN;
  const qlora_status s = check_device();
  if (s != QLORA_OK) return s;
  Fp8QuantArgs a;
  a.X = X;
  a.rows = rows;
  a.cols = cols;
  a.codes = codes;
  a.scale = scale;
  hipStream_t st = static_cast<hipStream_t>(stream);
  return hip_status(weight ? launch_fp8_quantize_weight(a, x_type, st)
                           : launch_fp8_quantize(a, x_type, st));
}

}  // namespace

}  // namespace qlora

extern "C" {

qlora_status qlora_fp8_quantize(const void* X, int x_type, int64_t rows, int64_t cols,
                                uint8_t* codes, float* scale, void* stream) {
  return qlora::quantize(X, x_type, rows, cols, codes, scale, stream, false);
}

qlora_status qlora_fp8_quantize_weight(const void* W, int w_type, int64_t rows, int64_t cols,
                                       uint8_t* codes, float* scale, void* stream) {
  return qlora::quantize(W, w_type, rows, cols, codes, scale, stream, true);
}

size_t qlora_fp8_workspace(int64_t T, int64_t rows, int64_t cols, int x_given) {
  if (!qlora::fp8_dims_ok(T, rows, cols, rows) || T == 0) return 0;
  return qlora::fp8_plan(T, rows, cols, x_given == 0).total;
}

size_t qlora_fp8_gated_workspace(int64_t T, int64_t rows, int64_t cols) {
  if (!qlora::fp8_dims_ok(T, rows, cols, 2 * rows) || T == 0) return 0;
  return qlora::fp8_plan(T, 2 * rows, cols, true).total;
}

qlora_status qlora_fp8_matmul(const uint8_t* W, const float* w_scale, int64_t rows, int64_t cols,
                              const uint8_t* X, const float* x_scale, int64_t T,
                              int compute_dtype, uint16_t* Y, void* ws, size_t ws_bytes,
                              void* stream) {
  return qlora::product({{W, w_scale}, {nullptr, nullptr}}, false, rows, cols, {X, x_scale},
                        nullptr, true, T, 0, compute_dtype, Y, ws, ws_bytes, stream);
}

qlora_status qlora_fp8_linear_fwd(const uint8_t* W, const float* w_scale, int64_t rows,
                                  int64_t cols, const uint16_t* X, int64_t T, int compute_dtype,
                                  uint16_t* Y, void* ws, size_t ws_bytes, void* stream) {
  return qlora::product({{W, w_scale}, {nullptr, nullptr}}, false, rows, cols, {nullptr, nullptr},
                        X, false, T, 0, compute_dtype, Y, ws, ws_bytes, stream);
}

qlora_status qlora_fp8_gated_fwd(const uint8_t* W_gate, const float* gate_scale,
                                 const uint8_t* W_up, const float* up_scale, int64_t rows,
                                 int64_t cols, const uint16_t* X, int64_t T, int act,
                                 int compute_dtype, uint16_t* H, void* ws, size_t ws_bytes,
                                 void* stream) {
  return qlora::product({{W_gate, gate_scale}, {W_up, up_scale}}, true, rows, cols,
                        {nullptr, nullptr}, X, false, T, act, compute_dtype, H, ws, ws_bytes,
                        stream);
}

}  // extern "C"
