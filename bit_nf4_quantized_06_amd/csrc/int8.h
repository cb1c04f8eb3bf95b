// Host-side shapes, plan and workspace of the 8-bit linear layer, and the
// launchers of its kernels (int8.hip).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "qlora_int8.h"

namespace qlora {

// Which kernel computes Y = Xq W^T.
enum Int8Path {
  kInt8Fused,        // few 16-bit tokens: quantised inside the streaming kernel
  kInt8Skinny,       // at most kInt8SkinnyTokens: the weight streamed once, no LDS
  kInt8Tile64x128,   // tiles of tokens x outputs through LDS
  kInt8Tile128x128,
  kInt8Tile128x256,
  kInt8Tile256x256,
};
constexpr int64_t kInt8SkinnyTokens = 64;
// Codes of all tokens that every workgroup of the streaming kernel quantises
// itself.  More than these cost more than a launch of their own: 1 x 8192 x 8192
// 16.0 us against 19.1 with two launches, 2 x 4096 x 4096 8.2 against 9.0, but
// 3 x 4096 x 4096 9.5 against 9.0 and 8 x 4096 x 4096 17.0 against 9.3.
constexpr int64_t kInt8FusedBytes = 8192;
// 128^2 (2^17 - 16) < 2^31: the int32 sums are exact for any codes
constexpr int64_t kInt8MaxCols = (int64_t(1) << 17) - 16;
// grids stay below 2^32 threads: 1024 a row of the quantiser, 256 a tile of at
// least 2^13 outputs of the product
constexpr int64_t kInt8MaxDim = (int64_t(1) << 22) - 1;
constexpr int64_t kInt8MaxOut = int64_t(1) << 36;

struct Int8Plan {
  Int8Path path;
  int splits;              // parts of the reduction (tile paths), 1: no partials
  size_t codes_off, scale_off, part_off, total;
};

bool int8_row_dims_ok(int64_t rows, int64_t cols);
bool int8_dims_ok(int64_t T, int64_t rows, int64_t cols);
// with_codes: the call quantises its tokens, so their codes and scales live
// in the workspace.
Int8Plan int8_plan(int64_t T, int64_t rows, int64_t cols, bool with_codes);

struct Int8QuantArgs {
  const void* X;           // [rows, cols] of type x_type
  int64_t rows, cols;
  int8_t* codes;           // [rows, cols]
  float* scale;            // [rows]
};

struct Int8Args {
  const int8_t* X;         // [T, cols] codes
  const float* x_scale;    // [T]
  const int8_t* W;         // [rows, cols] codes
  const float* w_scale;    // [rows]
  int64_t T, rows, cols;
  uint16_t* Y;             // [T, rows]
  int32_t* part;           // [splits][T][rows] with splits > 1
  int splits;
};

}  // namespace qlora
