// The linear layer in 8-bit integers (gfx950, int8 MFMA).
//
//   quantise:  s_i = RN32(max_k |x_ik| / 127),  c_ik = nearest integer to
//              x_ik / s_i (ties to even; 0 where s_i = 0)
//   product:   Y_tn = RN16(sx_t * sw_n * sum_k cx_tk cw_nk)
// with one scale a row: a row is an output channel of the weight, a token of
// the activations.  The sums are exact in 32-bit integers (at most 2^17
// terms of at most 127^2), so no order of summation and no split changes a
// result; the only roundings are the codes themselves, the sum's conversion
// and two products in float32, and the one rounding to 16 bits.
#include <hip/hip_runtime.h>

#include "gemm_common.h"
#include "int8.h"
#include "int8_kernels.h"

namespace qlora {

namespace {

typedef int32_t i32x4_t __attribute__((ext_vector_type(4)));
typedef int32_t i32x16_t __attribute__((ext_vector_type(16)));

// ---------------------------------------------------------------------------
// Quantisation of rows.
// ---------------------------------------------------------------------------

// Nearest integer to x / s, ties to even, from the product with the rounded
// reciprocal: that candidate r is off by at most one, and only next to a
// border.  The remainder x - r s is exact in one FMA (it is a multiple of
// half an ulp of s below s in size), so comparing it with s / 2 settles the
// border and the tie exactly.  Both x and s are pre-scaled by the caller so
// that s is far from the subnormals.
__device__ __forceinline__ int nearest_code(float x, float s, float inv) {
  const float r = __builtin_rintf(x * inv);
  const float e = __builtin_fmaf(-r, s, x);
  const float h = 0.5f * s;
  const float ae = fabsf(e);
  const int ri = (int)r;
  const bool off = ae > h || (ae == h && (ri & 1));
  int c = off ? ri + (e < 0.0f ? -1 : 1) : ri;
  c = c > 127 ? 127 : (c < -127 ? -127 : c);
  return c;
}

// 16 bytes of a row: 8 elements of 16 bits or 4 of 32.
template <int kType>
struct RowVec {
  static constexpr int N = kType == QLORA_TYPE_FP32 ? 4 : 8;
  u32x4_t v;
  __device__ __forceinline__ float at(int i) const {
    if (kType == QLORA_TYPE_FP32) return __uint_as_float(v[i]);
    const uint32_t w = v[i >> 1];
    if (kType == QLORA_TYPE_BF16) return (i & 1) ? bf16_hi_to_f32(w) : bf16_lo_to_f32(w);
    return lo16_to_f32<true>((i & 1) ? w >> 16 : w);
  }
};

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return (uint32_t)(a & 255) | ((uint32_t)(b & 255) << 8) | ((uint32_t)(c & 255) << 16) |
         ((uint32_t)d << 24);
}

template <int kType>
__device__ __forceinline__ void store_codes(int8_t* dst, const RowVec<kType>& x, float s,
                                            float inv, float up) {
  int c[RowVec<kType>::N];
#pragma unroll
  for (int i = 0; i < RowVec<kType>::N; ++i)
    c[i] = inv == 0.0f ? 0 : nearest_code(x.at(i) * up, s, inv);
  if constexpr (kType == QLORA_TYPE_FP32)
    *reinterpret_cast<uint32_t*>(dst) = pack4(c[0], c[1], c[2], c[3]);
  else
    *reinterpret_cast<uint2*>(dst) =
        uint2{pack4(c[0], c[1], c[2], c[3]), pack4(c[4], c[5], c[6], c[7])};
}

// One workgroup a row.  kNV > 0: the row's vectors stay in registers (kNV a
// thread) between the maximum and the codes, one read of the row; kNV = 0:
// rows too long for that are read twice (the second time from the cache).
template <int kType, int kNV>
__global__ __launch_bounds__(256) void int8_quantize_kernel(Int8QuantArgs a) {
  constexpr int N = RowVec<kType>::N;
  __shared__ float red[4];
  const int64_t row = blockIdx.x;
  const int tid = threadIdx.x;
  const int nvec = (int)(a.cols / N);
  const u32x4_t* src = reinterpret_cast<const u32x4_t*>(a.X) + row * (int64_t)nvec;
  RowVec<kType> x[kNV > 0 ? kNV : 1];
  float m = 0.0f;
  if constexpr (kNV > 0) {
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const int i = tid + 256 * j;
      x[j].v = i < nvec ? src[i] : u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < kNV; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) m = fmaxf(m, fabsf(x[j].at(e)));
  } else {
    for (int i = tid; i < nvec; i += 256) {
      x[0].v = src[i];
#pragma unroll
      for (int e = 0; e < N; ++e) m = fmaxf(m, fabsf(x[0].at(e)));
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  if ((tid & 63) == 0) red[tid >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
  const float scale = __fdiv_rn(m, 127.0f);
  // scales below 2^-100 would take the reciprocal out of range: the row and
  // the scale are multiplied by 2^96 first (exact; quotients do not change)
  const float up = scale < 0x1p-100f ? 0x1p96f : 1.0f;
  const float s = scale * up;
  const float inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
  if (tid == 0) a.scale[row] = scale;
  int8_t* dst = a.codes + row * a.cols;
  if constexpr (kNV > 0) {
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const int i = tid + 256 * j;
      if (i < nvec) store_codes<kType>(dst + (int64_t)i * N, x[j], s, inv, up);
    }
  } else {
    for (int i = tid; i < nvec; i += 256) {
      x[0].v = src[i];
      store_codes<kType>(dst + (int64_t)i * N, x[0], s, inv, up);
    }
  }
}

template <int kType>
hipError_t quantize_type(const Int8QuantArgs& a, hipStream_t stream) {
  const int64_t nvec = a.cols / RowVec<kType>::N;
  const dim3 grid((unsigned)a.rows), block(256);
  if (nvec <= 256)
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 1>), grid, block, 0, stream, a);
  else if (nvec <= 512)
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 2>), grid, block, 0, stream, a);
  else if (nvec <= 1024)
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 4>), grid, block, 0, stream, a);
  else if (nvec <= 2048)
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 8>), grid, block, 0, stream, a);
  else if (nvec <= 4096)
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 16>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 0>), grid, block, 0, stream, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Products of many tokens: tiles through LDS.
// ---------------------------------------------------------------------------

// A workgroup of WM x WN waves computes a TM-token x TN-output tile, each
// wave MI x NJ MFMA blocks of 32 x 32; the reduction advances 128 a step (128
// bytes a row of either operand).  Both operands come by DMA into LDS rings
// (weights three stages, activations two), in rows of 8 chunks of 16 bytes,
// chunk' = chunk ^ swz_g(row): the reads of 16 rows at one chunk then touch
// all banks evenly.  The weights are the MFMA's row operand, so a lane's
// accumulators are 4 consecutive outputs of one token.
template <int MI, int NJ, int WM, int WN>
struct I8Tile {
  static constexpr int TM = 32 * MI * WM, TN = 32 * NJ * WN, kWaves = WM * WN;
  static constexpr int LX = TM / 8 / kWaves, LW = TN / 8 / kWaves;   // DMAs a wave and step
  static constexpr int kXBytes = TM * 128, kWBytes = TN * 128;
  static_assert(LX % 2 == 0 && LW % 2 == 0, "the lane offsets alternate with the row block");
};

template <class Tile>
struct I8Ctx {
  uint8_t* W[3];
  uint8_t* X[2];
  int lane, wave;
  int step0, nsteps, last;   // this split's first step and step count; the step with K's tail
  uint32_t K;
  const int8_t *x_base, *w_base;
  uint32_t x_bytes, w_bytes;
  uint32_t voff[2], voff_tail[2];
  int x_frag[4], w_frag[4];  // per 32-byte slice
};

template <class Tile>
__device__ __forceinline__ void i8_issue_x(const I8Ctx<Tile>& c, uint8_t* stage, int step) {
  const int ks = c.step0 + step;
  const bool tail = ks == c.last;
#pragma unroll
  for (int i = 0; i < Tile::LX; ++i) {
    const int blk8 = c.wave * Tile::LX + i;
    const uint32_t soff =
        step < c.nsteps ? (uint32_t)ks * 128u + (uint32_t)(blk8 * 8) * c.K : kOOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(c.x_base, c.x_bytes),
                                             (lds_void_t*)(stage + blk8 * 1024), 16,
                                             tail ? c.voff_tail[i & 1] : c.voff[i & 1], soff, 0,
                                             0);
  }
}

// Columns past K of the last step read the next row (or 0 past the range);
// the activations there are 0.
template <class Tile>
__device__ __forceinline__ void i8_issue_w(const I8Ctx<Tile>& c, uint8_t* stage, int step) {
  const int ks = c.step0 + step;
#pragma unroll
  for (int i = 0; i < Tile::LW; ++i) {
    const int blk8 = c.wave * Tile::LW + i;
    const uint32_t soff =
        step < c.nsteps ? (uint32_t)ks * 128u + (uint32_t)(blk8 * 8) * c.K : kOOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(c.w_base, c.w_bytes),
                                             (lds_void_t*)(stage + blk8 * 1024), 16,
                                             c.voff[i & 1], soff, 0, 0);
  }
}

template <int MI, int NJ, class Tile>
__device__ __forceinline__ void i8_frags(const I8Ctx<Tile>& c, const uint8_t* xs,
                                         const uint8_t* ws, int s, i32x4_t (&fx)[MI],
                                         i32x4_t (&fw)[NJ]) {
#pragma unroll
  for (int j = 0; j < NJ; ++j)
    fw[j] = *reinterpret_cast<const i32x4_t*>(ws + c.w_frag[s] + 32 * j * 128);
#pragma unroll
  for (int i = 0; i < MI; ++i)
    fx[i] = *reinterpret_cast<const i32x4_t*>(xs + c.x_frag[s] + 32 * i * 128);
}

// One step on weight stage SW and activation stage SX.  Slice 0 issues the
// activations of step+1, slice 1 the weights of step+2; the barrier before
// the step's last MFMAs waits for all but those weights, and the first
// fragments of the next step are read under the MFMAs behind it.
template <int MI, int NJ, class Tile, int SW, int SX>
__device__ __forceinline__ void i8_step(const I8Ctx<Tile>& c, int step, i32x16_t (&acc)[MI][NJ],
                                        i32x4_t (&fx)[2][MI], i32x4_t (&fw)[2][NJ]) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kM = MI * NJ;
  constexpr int kR = MI + NJ;
  const uint8_t* ws = c.W[SW];
  const uint8_t* xs = c.X[SX];
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const int f = s & 1;
    if (s == 0) i8_issue_x(c, c.X[(SX + 1) & 1], step + 1);
    if (s == 1) i8_issue_w(c, c.W[(SW + 2) % 3], step + 2);
    i8_frags<MI, NJ>(c, xs, ws, s + 1, fx[f ^ 1], fw[f ^ 1]);
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[f][j], fx[f][i], acc[i][j], 0, 0, 0);
    const int loads = s == 0 ? Tile::LX : (s == 1 ? Tile::LW : 0);
#pragma unroll
    for (int q = 0; q < kM; ++q) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, (kR + kM - 1) / kM, 0);
      if (q < loads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
#pragma unroll
  for (int i = 0; i < MI / 2; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[1][j], fx[1][i], acc[i][j], 0, 0, 0);
  __builtin_amdgcn_sched_barrier(0);
  __builtin_amdgcn_s_setprio(0);
  barrier_keep_vmem<Tile::LW>();   // the stages of step+1 are complete and visible
  i32x4_t gx[MI], gw[NJ];
  i8_frags<MI, NJ>(c, c.X[(SX + 1) & 1], c.W[(SW + 1) % 3], 0, gx, gw);
#pragma unroll
  for (int i = MI / 2; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
      acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[1][j], fx[1][i], acc[i][j], 0, 0, 0);
#pragma unroll
  for (int i = 0; i < MI; ++i) fx[0][i] = gx[i];
#pragma unroll
  for (int j = 0; j < NJ; ++j) fw[0][j] = gw[j];
#endif
}

// kPart: store the int32 sums of one part of the reduction (blockIdx.y);
// otherwise scale, round and write Y.
template <int MI, int NJ, int WM, int WN, bool kF16, bool kPart>
__global__ __launch_bounds__(64 * WM * WN, 2) void int8_gemm_kernel(Int8Args g) {
#if defined(__HIP_DEVICE_COMPILE__)
  using Tile = I8Tile<MI, NJ, WM, WN>;
  __shared__ __attribute__((aligned(1024))) uint8_t sw0[Tile::kWBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sw1[Tile::kWBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sw2[Tile::kWBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sx0[Tile::kXBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sx1[Tile::kXBytes];
  I8Ctx<Tile> c{{sw0, sw1, sw2}, {sx0, sx1}};
  c.lane = threadIdx.x & 63;
  c.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = c.wave / WN, wn = c.wave % WN;
  const int l32 = c.lane & 31, lhi = c.lane >> 5;
  const int mt = (int)((g.T + Tile::TM - 1) / Tile::TM);
  const int nt = (int)((g.rows + Tile::TN - 1) / Tile::TN);
  int tm, tn;
  tile_coords(blockIdx.x, mt, nt, tm, tn);
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
  const int64_t m0 = (int64_t)tm * Tile::TM, n0 = (int64_t)tn * Tile::TN;
  const int rows_here = (int)(g.T - m0 < Tile::TM ? g.T - m0 : Tile::TM);
  const int outs_here = (int)(g.rows - n0 < Tile::TN ? g.rows - n0 : Tile::TN);
  c.K = (uint32_t)g.cols;
  {
    const int all = (int)((g.cols + 127) / 128);
    const int per = (all + g.splits - 1) / g.splits;
    c.step0 = kPart ? (int)blockIdx.y * per : 0;
    const int end = c.step0 + per < all ? c.step0 + per : all;
    c.nsteps = kPart ? (end > c.step0 ? end - c.step0 : 0) : all;
    c.last = all - 1;
  }
  c.x_base = g.X + m0 * g.cols;
  c.x_bytes = (uint32_t)rows_here * c.K;
  c.w_base = g.W + n0 * g.cols;
  c.w_bytes = (uint32_t)outs_here * c.K;
  {
    const int rl = c.lane >> 3;
#pragma unroll
    for (int par = 0; par < 2; ++par) {
      const int ch = (c.lane & 7) ^ swz_g(8 * par + rl);
      c.voff[par] = (uint32_t)rl * c.K + 16u * (uint32_t)ch;
      c.voff_tail[par] = (uint32_t)c.last * 128u + 16u * (uint32_t)ch < c.K ? c.voff[par] : kOOB;
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int xr = 32 * MI * wm + l32, wr = 32 * NJ * wn + l32;
      c.x_frag[s] = xr * 128 + (((2 * s + lhi) ^ swz_g(xr)) << 4);
      c.w_frag[s] = wr * 128 + (((2 * s + lhi) ^ swz_g(wr)) << 4);
    }
  }
  i32x16_t acc[MI][NJ];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;

  i8_issue_w(c, sw0, 0);
  i8_issue_x(c, sx0, 0);
  i8_issue_w(c, sw1, 1);
  barrier_keep_vmem<Tile::LW>();
  i32x4_t fx[2][MI], fw[2][NJ];
  i8_frags<MI, NJ>(c, sx0, sw0, 0, fx[0], fw[0]);
  int step = 0;
  for (; step + 6 <= c.nsteps; step += 6) {
    i8_step<MI, NJ, Tile, 0, 0>(c, step, acc, fx, fw);
    i8_step<MI, NJ, Tile, 1, 1>(c, step + 1, acc, fx, fw);
    i8_step<MI, NJ, Tile, 2, 0>(c, step + 2, acc, fx, fw);
    i8_step<MI, NJ, Tile, 0, 1>(c, step + 3, acc, fx, fw);
    i8_step<MI, NJ, Tile, 1, 0>(c, step + 4, acc, fx, fw);
    i8_step<MI, NJ, Tile, 2, 1>(c, step + 5, acc, fx, fw);
  }
  if (step < c.nsteps) i8_step<MI, NJ, Tile, 0, 0>(c, step, acc, fx, fw);
  if (step + 1 < c.nsteps) i8_step<MI, NJ, Tile, 1, 1>(c, step + 1, acc, fx, fw);
  if (step + 2 < c.nsteps) i8_step<MI, NJ, Tile, 2, 0>(c, step + 2, acc, fx, fw);
  if (step + 3 < c.nsteps) i8_step<MI, NJ, Tile, 0, 1>(c, step + 3, acc, fx, fw);
  if (step + 4 < c.nsteps) i8_step<MI, NJ, Tile, 1, 0>(c, step + 4, acc, fx, fw);

  if constexpr (kPart) {
    // the stages must not be freed to another workgroup while DMAs land
    __builtin_amdgcn_s_waitcnt(0);
    int32_t* part = g.part + (int64_t)blockIdx.y * g.T * g.rows;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int64_t t = m0 + 32 * (MI * wm + i) + l32;
      if (t < g.T) {
#pragma unroll
        for (int j = 0; j < NJ; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int64_t n = n0 + 32 * (NJ * wn + j) + 8 * q + 4 * lhi;
            int32_t* d = part + t * g.rows + n;
            if (n + 4 <= g.rows && (g.rows & 3) == 0) {
              *reinterpret_cast<i32x4_t*>(d) =
                  i32x4_t{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2],
                          acc[i][j][4 * q + 3]};
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (n + e < g.rows) d[e] = acc[i][j][4 * q + e];
            }
          }
      }
    }
  } else {
    // Each wave scales and rounds its 32 MI x 32 NJ tile into LDS, token
    // rows of 64 NJ bytes with their 16-byte chunks swizzled by the row, and
    // writes whole rows with 16-byte stores.
    static_assert(NJ == 2, "token rows of 128 bytes");
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    constexpr int kOut = 32 * MI * 128;   // bytes a wave
    static_assert(2 * kOut <= Tile::kWBytes && 2 * kOut <= Tile::kXBytes,
                  "two waves' tiles a stage");
    uint8_t* stg = (c.wave >> 1) == 0 ? sw0 : (c.wave >> 1) == 1 ? sw1
                 : (c.wave >> 1) == 2 ? sw2 : sx0;
    stg += (c.wave & 1) * kOut;
    const __amdgpu_buffer_rsrc_t sr = make_rsrc(g.w_scale + n0, (uint32_t)outs_here * 4u);
    f32x4_t sw[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t n = (uint32_t)(32 * (NJ * wn + j) + 8 * q + 4 * lhi);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sw[j][q][e] = __builtin_bit_cast(
              float, __builtin_amdgcn_raw_buffer_load_b32(sr, (n + (uint32_t)e) * 4u, 0, 0));
      }
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int lr = 32 * i + l32;
      const int64_t t = m0 + 32 * MI * wm + lr;
      const float sx = t < g.T ? g.x_scale[t] : 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float v[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = (float)acc[i][j][4 * q + e] * sw[j][q][e] * sx;
          *reinterpret_cast<uint2*>(stg + lr * 128 + (((4 * j + q) ^ (lr & 7)) << 4) + 8 * lhi) =
              uint2{pack16x2<kF16>(v[0], v[1]), pack16x2<kF16>(v[2], v[3])};
        }
    }
    const int ch = c.lane & 7;
    const int64_t n = n0 + 32 * NJ * wn + 8 * ch;
#pragma unroll
    for (int it = 0; it < 4 * MI; ++it) {
      const int row = 8 * it + (c.lane >> 3);
      const u32x4_t v =
          *reinterpret_cast<const u32x4_t*>(stg + row * 128 + ((ch ^ (row & 7)) << 4));
      const int64_t t = m0 + 32 * MI * wm + row;
      if (t < g.T && n < g.rows) {
        uint16_t* d = g.Y + t * g.rows + n;
        if ((g.rows & 7) == 0) {
          *reinterpret_cast<u32x4_t*>(d) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (n + e < g.rows) d[e] = (uint16_t)(v[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }
#endif
}

// Y = RN16(sx sw sum of the parts), one output a thread and step.
template <bool kF16>
__global__ __launch_bounds__(256) void int8_finish_kernel(Int8Args g) {
  const int64_t n_all = g.T * g.rows;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n_all;
       i += (int64_t)gridDim.x * 256) {
    int32_t v = 0;
    for (int s = 0; s < g.splits; ++s) v += g.part[(int64_t)s * n_all + i];
    const int64_t t = i / g.rows;
    const float y = (float)v * g.w_scale[i - t * g.rows] * g.x_scale[t];
    g.Y[i] = (uint16_t)(pack16x2<kF16>(y, 0.0f) & 0xFFFFu);
  }
}

// ---------------------------------------------------------------------------
// Products of few tokens: the weight streamed once, no LDS on its way.
// ---------------------------------------------------------------------------

// A workgroup of kWaves waves owns 16 RG outputs and all (up to 16 TG)
// tokens; the waves take the 128-byte pieces of the rows in turn.  Lane l
// loads bytes 32 g .. 32 g + 31 of row l % 16 (g = l / 16) of both operands,
// the two 16-byte halves feeding one 16x16x64 MFMA each: which reduction
// index meets which MFMA slot is free as long as both operands agree.  The
// waves' int32 sums are added in LDS.
template <int RG, int TG, int kWaves, bool kF16>
__global__ __launch_bounds__(64 * kWaves) void int8_skinny_kernel(Int8Args g) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(16))) int32_t red[kWaves][RG * TG * 256];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, gq = lane >> 4;
  const uint32_t K = (uint32_t)g.cols;
  const int64_t n0 = (int64_t)blockIdx.x * (16 * RG);
  const int outs_here = (int)(g.rows - n0 < 16 * RG ? g.rows - n0 : 16 * RG);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(g.W + n0 * g.cols, (uint32_t)outs_here * K);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.X, (uint32_t)g.T * K);
  i32x4_t acc[RG][TG];
#pragma unroll
  for (int a = 0; a < RG; ++a)
#pragma unroll
    for (int b = 0; b < TG; ++b) acc[a][b] = i32x4_t{0, 0, 0, 0};
  const int pieces = (int)((K + 127) / 128);
  for (int p = wave; p < pieces; p += kWaves) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = (uint32_t)p * 128u + 32u * (uint32_t)gq + 16u * (uint32_t)h;
      i32x4_t w[RG], x[TG];
#pragma unroll
      for (int a = 0; a < RG; ++a)
        w[a] = __builtin_bit_cast(
            i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                         wr, k < K ? (uint32_t)(16 * a + r16) * K + k : kOOB, 0, 0));
#pragma unroll
      for (int b = 0; b < TG; ++b)
        x[b] = __builtin_bit_cast(
            i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
                         xr, k < K ? (uint32_t)(16 * b + r16) * K + k : kOOB, 0, 0));
#pragma unroll
      for (int a = 0; a < RG; ++a)
#pragma unroll
        for (int b = 0; b < TG; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[a], x[b], acc[a][b], 0, 0, 0);
    }
  }
  // acc[a][b][e]: output 16 a + 4 gq + e, token 16 b + r16
#pragma unroll
  for (int a = 0; a < RG; ++a)
#pragma unroll
    for (int b = 0; b < TG; ++b)
#pragma unroll
      for (int e = 0; e < 4; ++e)
        red[wave][(16 * b + r16) * (16 * RG) + 16 * a + 4 * gq + e] = acc[a][b][e];
  __syncthreads();
  for (int i = threadIdx.x; i < RG * TG * 256; i += 64 * kWaves) {
    const int64_t t = i / (16 * RG);
    const int64_t n = n0 + i % (16 * RG);
    if (t < g.T && n < g.rows) {
      int32_t v = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += red[w][i];
      const float y = (float)v * g.w_scale[n] * g.x_scale[t];
      g.Y[t * g.rows + n] = (uint16_t)(pack16x2<kF16>(y, 0.0f) & 0xFFFFu);
    }
  }
#endif
}

template <bool kF16>
hipError_t int8_launch(const Int8Args& a, const Int8Plan& p, hipStream_t stream) {
  if (p.path == kInt8Skinny) {
    const dim3 grid((unsigned)((a.rows + 15) / 16));
    if (a.T <= 16)
      hipLaunchKernelGGL((int8_skinny_kernel<1, 1, 8, kF16>), grid, dim3(512), 0, stream, a);
    else if (a.T <= 32)
      hipLaunchKernelGGL((int8_skinny_kernel<1, 2, 8, kF16>), grid, dim3(512), 0, stream, a);
    else
      hipLaunchKernelGGL((int8_skinny_kernel<1, 4, 8, kF16>), grid, dim3(512), 0, stream, a);
    return hipGetLastError();
  }
  const int64_t side = p.path == kInt8Tile256 ? 256 : 128;
  const dim3 grid((unsigned)(((a.T + side - 1) / side) * ((a.rows + side - 1) / side)),
                  (unsigned)a.splits);
  if (p.path == kInt8Tile256) {
    if (a.splits == 1)
      hipLaunchKernelGGL((int8_gemm_kernel<4, 2, 2, 4, kF16, false>), grid, dim3(512), 0, stream,
                         a);
    else
      hipLaunchKernelGGL((int8_gemm_kernel<4, 2, 2, 4, kF16, true>), grid, dim3(512), 0, stream,
                         a);
  } else {
    if (a.splits == 1)
      hipLaunchKernelGGL((int8_gemm_kernel<2, 2, 2, 2, kF16, false>), grid, dim3(256), 0, stream,
                         a);
    else
      hipLaunchKernelGGL((int8_gemm_kernel<2, 2, 2, 2, kF16, true>), grid, dim3(256), 0, stream,
                         a);
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.splits > 1) {
    int64_t blocks = (a.T * a.rows + 255) / 256;
    if (blocks > 8192) blocks = 8192;
    hipLaunchKernelGGL((int8_finish_kernel<kF16>), dim3((unsigned)blocks), dim3(256), 0, stream,
                       a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

hipError_t launch_int8_quantize(const Int8QuantArgs& a, int x_type, hipStream_t stream) {
  switch (x_type) {
    case QLORA_TYPE_BF16: return quantize_type<QLORA_TYPE_BF16>(a, stream);
    case QLORA_TYPE_FP16: return quantize_type<QLORA_TYPE_FP16>(a, stream);
    case QLORA_TYPE_FP32: return quantize_type<QLORA_TYPE_FP32>(a, stream);
  }
  return hipErrorInvalidValue;
}

hipError_t launch_int8_product(const Int8Args& a, const Int8Plan& p, bool f16,
                               hipStream_t stream) {
  return f16 ? int8_launch<true>(a, p, stream) : int8_launch<false>(a, p, stream);
}

}  // namespace qlora
