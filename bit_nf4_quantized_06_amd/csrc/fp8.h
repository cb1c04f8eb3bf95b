// Host-side shapes, plan and workspace of the linear layer in 8-bit floating
// point, and what its kernels (fp8.hip) are given.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "qlora_fp8.h"

namespace qlora {

// Which kernel computes Y = Xq W^T.
enum Fp8Path {
  kFp8Fused,        // few 16-bit tokens: quantised inside the streaming kernel
  kFp8Skinny,       // at most kFp8SkinnyTokens: the weight streamed once, no LDS
  kFp8Tile64x128,   // tiles of tokens x outputs through LDS
  kFp8Tile128x128,
  kFp8Tile128x256,
  kFp8Tile256x256,
};
constexpr int64_t kFp8SkinnyTokens = 32;
// Codes (of whole blocks) of all tokens that every workgroup of the streaming
// kernel quantises itself, at most 16 tokens.
constexpr int64_t kFp8FusedBytes = 8192;
constexpr int64_t kFp8FusedTokens = 16;
constexpr int64_t kFp8FusedAll = int64_t(1) << 24;   // codes over all workgroups
constexpr int64_t kFp8MaxCols = (int64_t(1) << 17) - 16;
// grids stay below 2^32 threads: 256 a tile of at least 2^13 outputs of the product
constexpr int64_t kFp8MaxDim = (int64_t(1) << 22) - 1;
constexpr int64_t kFp8MaxOut = int64_t(1) << 36;

struct Fp8Plan {
  Fp8Path path;
  int splits;              // parts of the reduction (tile paths), 1: no partials
  size_t codes_off, scale_off, part_off, total;
};

constexpr int64_t fp8_blocks(int64_t cols) { return (cols + QLORA_FP8_BLOCK - 1) / QLORA_FP8_BLOCK; }
bool fp8_row_dims_ok(int64_t rows, int64_t cols);
// outs: outputs a token (2 rows in the gated block)
bool fp8_dims_ok(int64_t T, int64_t rows, int64_t cols, int64_t outs);
// x16: the call quantises its tokens, so unless the streaming kernel does,
// their codes and scales live in the workspace.
Fp8Plan fp8_plan(int64_t T, int64_t outs, int64_t cols, bool x16);

struct Fp8QuantArgs {
  const void* X;           // [rows, cols] of type x_type
  int64_t rows, cols;
  uint8_t* codes;          // [rows, cols]
  float* scale;            // [KB, rows], or of a weight [ceil(rows / 128), KB]
};

struct Fp8Args {
  const uint8_t* X;        // [T, cols] codes
  const float* x_scale;    // [KB, T]
  const uint16_t* X16;     // kFp8Fused: the 16-bit tokens [T, cols]
  const uint8_t* W[2];     // [rows, cols] codes; [1]: the up projection of a gated block
  const float* w_scale[2]; // [ceil(rows / 128), KB]
  int64_t T, rows, cols;
  uint16_t* Y;             // [T, rows]
  float* part;             // [splits][T][outs] with splits > 1
  int splits;
  int act;                 // gated
};

}  // namespace qlora
