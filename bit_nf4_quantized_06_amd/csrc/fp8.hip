// The linear layer and the gated feed-forward block in 8-bit floating point
// (gfx950, E4M3 MFMA).
//
//   quantise:  s = RN32(max |x| / 448) of a block, c = E4M3 nearest to
//              RN32(x / s), ties to even (0 where s = 0)
//   product:   P_tn = sum_b sx_bt sw_nb sum_{k in b} cx_tk cw_nk
//   linear:    Y = RN16(P);  gated: H = RN16(act(P_gate) P_up)
// with one scale for 128 columns of a token and for 128 x 128 weights.  A
// block of 128 columns is exactly one 16x16x128 MFMA, whose four float32 sums a
// lane are multiplied by the two scales and added to the accumulators by the
// vector unit (four FMAs for 32 cycles of the matrix core).  The MFMA itself is
// a little less than float32: it adds the products of 8 consecutive codes as
// fixed-point numbers cut at 2^-13 of the largest's power of two (measured; the
// older 16x16x32 form gives the same bits).  Over normal values that is 1.5e-5 of
// the result in norm, 5e-5 where magnitudes spread over 2^11.
#include <hip/hip_runtime.h>

#include "act.h"
#include "fp8.h"
#include "fp8_kernels.h"
#include "gemm_common.h"

namespace qlora {

namespace {

typedef int32_t i32x8_t __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Quantisation.
// ---------------------------------------------------------------------------

__device__ __forceinline__ float fp8_maximum(float a, float b) {   // NaN if either is
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_elementwise_maximum(a, b);
#else
  return a > b ? a : b;
#endif
}

// A block's scale from its largest magnitude, and what its codes are formed
// with.  A magnitude that is infinite or NaN leaves inv 0: codes 0.  Below
// 2^-80 the remainders of the division would leave the range: block and scale
// are multiplied by 2^96 first (exact; the quotients do not change).
struct BlockScale {
  float scale, s, inv, up;
  __device__ __forceinline__ explicit BlockScale(float largest) {
    scale = __fdiv_rn(largest, 448.0f);
    up = scale < 0x1p-80f ? 0x1p96f : 1.0f;
    s = scale * up;
    inv = s > 0.0f && s < __builtin_inff() ? __fdiv_rn(1.0f, s) : 0.0f;
  }
  // RN32(x / s).  q is within 1.5 ulp of the quotient, the
  // first remainder brings it within one, and from there the remainder times a
  // correctly rounded 1 / s gives the correctly rounded quotient (Markstein's
  // theorem).
  __device__ __forceinline__ float quotient(float v) const {
    float q = v * inv;
    q = __builtin_fmaf(__builtin_fmaf(-q, s, v), inv, q);
    return __builtin_fmaf(__builtin_fmaf(-q, s, v), inv, q);
  }
};

// four codes of one 32-bit word: v_cvt_pk_fp8_f32 rounds to nearest even
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int w = 0;
#if defined(__HIP_DEVICE_COMPILE__)
  w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, w, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
#endif
  return (uint32_t)w;
}

// 8 consecutive values of a row: 16 bytes, or 32 in float32.
template <int kType>
struct Vec8 {
  static constexpr int kLoads = kType == QLORA_TYPE_FP32 ? 2 : 1;
  u32x4_t v[kLoads];
  __device__ __forceinline__ void load(const void* base, int64_t element) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(
        static_cast<const char*>(base) + element * (kType == QLORA_TYPE_FP32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < kLoads; ++i) v[i] = p[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) v[i] = u32x4_t{0u, 0u, 0u, 0u};
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (kType == QLORA_TYPE_FP32) return __uint_as_float(v[i >> 2][i & 3]);
    const uint32_t w = v[0][i >> 1];
    if (kType == QLORA_TYPE_BF16) return (i & 1) ? bf16_hi_to_f32(w) : bf16_lo_to_f32(w);
    return lo16_to_f32<true>((i & 1) ? w >> 16 : w);
  }
  __device__ __forceinline__ float largest() const {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fp8_maximum(m, fabsf(at(i)));
    return m;
  }
  __device__ __forceinline__ uint2 codes(const BlockScale& b) const {
    if (b.inv == 0.0f) return uint2{0u, 0u};
    float q[8];
    if (b.up == 1.0f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = b.quotient(at(i));
    } else {
      // (only a scale that is itself subnormal, rounded coarsely, leaves
      // quotients past 448)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[i] = __builtin_amdgcn_fmed3f(b.quotient(at(i) * b.up), -448.0f, 448.0f);
    }
    return uint2{e4m3x4(q[0], q[1], q[2], q[3]), e4m3x4(q[4], q[5], q[6], q[7])};
  }
};

// A block's 128 columns in 16 lanes, 8 each: consecutive ones of 16 bits, 4 of
// each half of the block in float32, so that every load and store of the lanes is
// contiguous.  left: the columns that the block has (a multiple of 16).
template <int kType>
__device__ __forceinline__ void load_block(Vec8<kType>& x, const void* base, int64_t element, int l,
                                           int64_t left) {
  x.zero();
  if constexpr (kType == QLORA_TYPE_FP32) {
    const u32x4_t* p = reinterpret_cast<const u32x4_t*>(static_cast<const float*>(base) + element);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (64 * h + 4 * l < left) x.v[h] = p[16 * h + l];
  } else {
    if (8 * l < left) x.load(base, element + 8 * l);
  }
}

template <int kType>
__device__ __forceinline__ void store_block(const Vec8<kType>& x, const BlockScale& b,
                                            uint8_t* dst, int l, int64_t left) {
  const uint2 c = x.codes(b);
  if constexpr (kType == QLORA_TYPE_FP32) {
    if (4 * l < left) *reinterpret_cast<uint32_t*>(dst + 4 * l) = c.x;
    if (64 + 4 * l < left) *reinterpret_cast<uint32_t*>(dst + 64 + 4 * l) = c.y;
  } else {
    if (8 * l < left) *reinterpret_cast<uint2*>(dst + 8 * l) = c;
  }
}

// Tokens: a workgroup takes 16 kRows rows of one block of columns, a thread rows
// r, r + 16, ...; the scales of a block of columns lie together.  Bound by memory:
// 4001 x 4096 bf16 (49 MB) 9.7 us a call among others, 5.1 TB/s (10.4 the kernel alone
// under a trace).
template <int kType, int kRows>
__global__ __launch_bounds__(256) void fp8_quantize_kernel(Fp8QuantArgs a) {
  const int l = threadIdx.x & 15;
  const int64_t r0 = (int64_t)blockIdx.y * (16 * kRows) + (threadIdx.x >> 4);
  const int64_t k0 = (int64_t)blockIdx.x * 128, left = a.cols - k0;
  Vec8<kType> x[kRows];
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    x[j].zero();
    if (r0 + 16 * j < a.rows)
      load_block<kType>(x[j], a.X, (r0 + 16 * j) * a.cols + k0, l, left);
  }
#pragma unroll
  for (int j = 0; j < kRows; ++j) {
    float m = x[j].largest();
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) m = fp8_maximum(m, __shfl_xor(m, d));
    const int64_t row = r0 + 16 * j;
    if (row < a.rows) {
      const BlockScale b(m);
      store_block<kType>(x[j], b, a.codes + row * a.cols + k0, l, left);
      if (l == 0) a.scale[(int64_t)blockIdx.x * a.rows + row] = b.scale;
    }
  }
}

// Weights: a workgroup holds one 128 x 128 block in registers, 64 weights a
// thread.  11008 x 4096 bf16 (135 MB): 25 us, 5.4 TB/s.
template <int kType>
__global__ __launch_bounds__(256) void fp8_quantize_weight_kernel(Fp8QuantArgs a) {
  __shared__ float red[4];
  const int l = threadIdx.x & 15;
  const int64_t r0 = (int64_t)blockIdx.y * 128 + (threadIdx.x >> 4);
  const int64_t k0 = (int64_t)blockIdx.x * 128, left = a.cols - k0;
  Vec8<kType> x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j].zero();
    if (r0 + 16 * j < a.rows)
      load_block<kType>(x[j], a.X, (r0 + 16 * j) * a.cols + k0, l, left);
  }
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) m = fp8_maximum(m, x[j].largest());
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fp8_maximum(m, __shfl_xor(m, d));
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
  __syncthreads();
  const BlockScale b(fp8_maximum(fp8_maximum(red[0], red[1]), fp8_maximum(red[2], red[3])));
  if (threadIdx.x == 0) a.scale[(int64_t)blockIdx.y * gridDim.x + blockIdx.x] = b.scale;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (r0 + 16 * j < a.rows)
      store_block<kType>(x[j], b, a.codes + (r0 + 16 * j) * a.cols + k0, l, left);
}

// ---------------------------------------------------------------------------
// Products of many tokens: tiles through LDS.
// ---------------------------------------------------------------------------

__device__ __forceinline__ f32x4_t mfma_e4m3(const u32x4_t (&a)[2], const u32x4_t (&b)[2]) {
#if defined(__HIP_DEVICE_COMPILE__)
  const i32x8_t x = {(int)a[0][0], (int)a[0][1], (int)a[0][2], (int)a[0][3],
                     (int)a[1][0], (int)a[1][1], (int)a[1][2], (int)a[1][3]};
  const i32x8_t y = {(int)b[0][0], (int)b[0][1], (int)b[0][2], (int)b[0][3],
                     (int)b[1][0], (int)b[1][1], (int)b[1][2], (int)b[1][3]};
  // formats 0, 0: E4M3; scales 0: the form without block scales
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, f32x4_t{0.f, 0.f, 0.f, 0.f}, 0, 0,
                                                          0, 0, 0, 0);
#else
  return f32x4_t{0.f, 0.f, 0.f, 0.f};
#endif
}

// A workgroup of WM x WN waves computes a TM-token x TN-output tile, each wave
// MI x 4 MFMA blocks of 16 x 16; the reduction advances one block of 128
// columns a step (128 bytes a row of either operand).  Both operands come by
// DMA into LDS rings of SW weight and SX activation stages, in rows of 8 chunks
// of 16 bytes, chunk' = chunk ^ swz_g(row): the reads of 16 rows at one chunk
// then touch all banks evenly.  Lane l holds chunks l / 16 and l / 16 + 4 of
// row l % 16 of both operands: which 32 of the 128 columns a lane has does not
// matter, as long as both operands agree.  The weights are the MFMA's row
// operand, so a lane's sums are 4 consecutive outputs of one token.
//
// Gated: the tile's 32-row groups of weights come from the gate and the up
// projection in turn, so a wave holds both of the same 32 outputs.
//
// Which tile: fp8_plan.  256 x 256: 8192 x 11008 x 4096 330 to 375 us with the card's
// clock (2.0 to 2.2 PFLOP/s; a library product with one scale a tensor reaches 3.0),
// matrix cores busy 54%, vector unit 35%, LDS reads 23% of its cycles, waves waiting
// for loads and barriers 28%, and a last of 6 rounds with 0.4 of its tiles; gated
// 4000 x 11008 x 4096 the same.  128 x 256 in 4 parts: 317 x 4096 x 11008 29 us
// and 5 for the sum, matrix cores busy 20%: latency, 22 steps a CU.  64 x 128 in 4
// parts: 24 x 8192 x 22016 38 us, 4.8 TB/s of weights; gated 7 x 11008 x 4096 16.7 us,
// 5.4 TB/s.
template <int MI_, int WM_, int WN_, int SW_, int SX_>
struct F8Tile {
  static constexpr int MI = MI_, NJ = 4, WM = WM_, WN = WN_, SW = SW_, SX = SX_;
  static constexpr int TM = 16 * MI * WM, TN = 16 * NJ * WN, kWaves = WM * WN;
  static constexpr int LX = TM / 8 / kWaves, LW = TN / 8 / kWaves;   // DMAs a wave and step
  static constexpr int kXBytes = TM * 128, kWBytes = TN * 128;
  static_assert(SW == SX || SW == SX + 1, "the wait count below");
  // waves a SIMD: two workgroups of four waves share a CU where the LDS holds both
  static constexpr int kWavesSimd =
      kWaves / 4 * (2 * (SW * kWBytes + SX * kXBytes) <= 160 * 1024 ? 2 : 1);
  static constexpr int kUnroll = SW == SX ? SW : SW * SX;
};

template <class Tile, bool kGated>
struct F8Ctx {
  static constexpr int kScales = (Tile::MI + 3) / 4 + (kGated ? 2 : 1);   // scale loads a step
  // loads issued after those of step+1 when step ends: scales and activations
  // of step+SX-1 go out before the weights of step+SW-1
  static constexpr int kKeep = (Tile::SX - 2) * (Tile::LX + Tile::LW + kScales) +
                               (Tile::SW == Tile::SX ? 0 : Tile::LW);
  static_assert(kKeep < 64, "vmcnt");
  uint8_t* W[Tile::SW];
  uint8_t* X[Tile::SX];
  int lane, wave;
  int step0, nsteps, last;   // this split's first step and step count; the step with K's tail
  int tail;                  // that step of this split, or -1
  uint32_t K;
  const uint8_t *x_base, *w_base[2];
  uint32_t x_bytes, w_bytes;
  uint32_t voff[2], voff_tail[2];
  int x_frag, w_frag;        // lane's first chunk of row block 0; the second is ^ 64 bytes
  // scales: of the tile's tokens at block 0, tokens there are, tokens a block
  const float *sx_base, *sw_base[2];
  uint32_t sx_bytes;
  int64_t T;
  uint32_t sx_voff;
};

// Scales of one block of columns: lane l of x[q] holds token 64 q + l of the
// wave's (f8_spread hands them to the MFMA's lanes).
template <class Tile, bool kGated>
struct F8Scales {
  float x[(Tile::MI + 3) / 4];
  float w[kGated ? 2 : 1];
};

// v of 64 lanes -> the four rows of 16, each in every row
__device__ __forceinline__ void f8_spread(float v, float (&o)[4]) {
#if defined(__HIP_DEVICE_COMPILE__)
  const uint32_t u = __float_as_uint(v);
  const auto a = __builtin_amdgcn_permlane32_swap(u, u, false, false);   // rows 0 1 0 1, 2 3 2 3
  const auto b = __builtin_amdgcn_permlane16_swap(a[0], a[0], false, false);
  const auto c = __builtin_amdgcn_permlane16_swap(a[1], a[1], false, false);
  o[0] = __uint_as_float(b[0]);
  o[1] = __uint_as_float(b[1]);
  o[2] = __uint_as_float(c[0]);
  o[3] = __uint_as_float(c[1]);
#endif
}

template <class Tile, bool kGated>
__device__ __forceinline__ void f8_issue_scales(const F8Ctx<Tile, kGated>& c, int step,
                                                F8Scales<Tile, kGated>& s) {
  const int ks = c.step0 + step;
  const bool in = step < c.nsteps;
  const __amdgpu_buffer_rsrc_t xr =
      make_rsrc(c.sx_base + (in ? ks : c.step0) * c.T, in ? c.sx_bytes : 0u);
#pragma unroll
  for (int q = 0; q < (Tile::MI + 3) / 4; ++q)
    s.x[q] = __builtin_bit_cast(
        float, __builtin_amdgcn_raw_buffer_load_b32(xr, c.sx_voff + 256u * q, 0, 0));
#pragma unroll
  for (int p = 0; p < (kGated ? 2 : 1); ++p)
    s.w[p] = __builtin_bit_cast(
        float, __builtin_amdgcn_raw_buffer_load_b32(
                   make_rsrc(c.sw_base[p], (uint32_t)(c.last + 1) * 4u),
                   in ? (uint32_t)ks * 4u : kOOB, 0, 0));
}

template <class Tile, bool kGated>
__device__ __forceinline__ void f8_issue_x(const F8Ctx<Tile, kGated>& c, uint8_t* stage, int step) {
  const int ks = c.step0 + step;
  const bool tail = step == c.tail;
#pragma unroll
  for (int i = 0; i < Tile::LX; ++i) {
    const int blk8 = c.wave * Tile::LX + i;
    const uint32_t soff =
        step_soff(step, c.nsteps, (uint32_t)ks * 128u + (uint32_t)(blk8 * 8) * c.K);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(c.x_base, c.x_bytes),
                                             (lds_void_t*)(stage + blk8 * 1024), 16,
                                             tail ? c.voff_tail[blk8 & 1] : c.voff[blk8 & 1],
                                             soff, 0, 0);
  }
}

template <class Tile, bool kGated>
__device__ __forceinline__ void f8_issue_w(const F8Ctx<Tile, kGated>& c, uint8_t* stage, int step) {
  const int ks = c.step0 + step;
  const bool tail = step == c.tail;
#pragma unroll
  for (int i = 0; i < Tile::LW; ++i) {
    const int blk8 = c.wave * Tile::LW + i;
    const int up = kGated ? (blk8 >> 2) & 1 : 0;
    const int row = kGated ? 32 * (blk8 >> 3) + 8 * (blk8 & 3) : 8 * blk8;
    const uint32_t soff = step_soff(step, c.nsteps, (uint32_t)ks * 128u + (uint32_t)row * c.K);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(up ? c.w_base[1] : c.w_base[0], c.w_bytes),
                                             (lds_void_t*)(stage + blk8 * 1024), 16,
                                             tail ? c.voff_tail[blk8 & 1] : c.voff[blk8 & 1],
                                             soff, 0, 0);
  }
}

__device__ __forceinline__ void f8_frag(const uint8_t* p, int off, u32x4_t (&f)[2]) {
  f[0] = *reinterpret_cast<const u32x4_t*>(p + off);
  f[1] = *reinterpret_cast<const u32x4_t*>(p + (off ^ 64));
}

// What a wave carries from MFMA to MFMA: the fragments of the four weight row
// blocks, of two token blocks, the products of two token blocks that the
// accumulators are still to take, and the scales of the older of them.
template <bool kGated>
struct F8Regs {
  u32x4_t fw[4][2], fx[2][2];
  f32x4_t part[2][4];
  float s[kGated ? 2 : 1];
};

template <bool kGated>
__device__ __forceinline__ void f8_add(f32x4_t (&acc)[4], const f32x4_t (&part)[4],
                                       const float (&s)[kGated ? 2 : 1]) {
#pragma unroll
  for (int j = 0; j < 4; ++j)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      acc[j][e] = __builtin_fmaf(part[j][e], s[kGated ? j >> 1 : 0], acc[j][e]);
}

// One step on weight stage W and activation stage X (compile-time, so the
// compiler sees that a DMA into one stage does not touch another).  Token block
// i's four MFMAs go out while the vector unit adds block i - 1's products and
// the LDS hands over block i + 1's fragment.  The loads for the steps ahead go
// out with the first blocks, into the stages that the step before read; the
// barrier before the last block waits for the stages of the next step, whose
// first fragments are read under the last block's MFMAs: those of the weights
// into the registers that each MFMA has just read.
template <class Tile, bool kGated, int W, int X>
__device__ __forceinline__ void f8_step(const F8Ctx<Tile, kGated>& c, int step,
                                        f32x4_t (&acc)[Tile::MI][4], F8Regs<kGated>& r,
                                        F8Scales<Tile, kGated> (&sc)[Tile::SX]) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int MI = Tile::MI, SW = Tile::SW, SX = Tile::SX;
  constexpr int kP = kGated ? 2 : 1;
  static_assert(MI % 2 == 0, "");
  const uint8_t* xs = c.X[X];
  const uint8_t* ws_next = c.W[(W + 1) % SW];
  const uint8_t* xs_next = c.X[(X + 1) % SX];
  float sx[(MI + 3) / 4][4];
#pragma unroll
  for (int q = 0; q < (MI + 3) / 4; ++q) f8_spread(sc[X].x[q], sx[q]);
  float sw[kP];
#pragma unroll
  for (int p = 0; p < kP; ++p) sw[p] = sc[X].w[p];
  f8_issue_scales(c, step + SX - 1, sc[(X + SX - 1) % SX]);
#pragma unroll
  for (int i = 0; i < MI; ++i) {
    const bool last = i == MI - 1;
    if (i == 0) f8_issue_x(c, c.X[(X + SX - 1) % SX], step + SX - 1);
    if (i == (MI > 2 ? 1 : 0)) f8_issue_w(c, c.W[(W + SW - 1) % SW], step + SW - 1);
    if (last) {
      __builtin_amdgcn_sched_barrier(0);
      // everybody has this step's fragments; the stages of step+1 are complete
      barrier_keep_vmem<F8Ctx<Tile, kGated>::kKeep>();
    } else {
      f8_frag(xs, c.x_frag + 16 * (i + 1) * 128, r.fx[(i + 1) & 1]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r.part[i & 1][j] = mfma_e4m3(r.fw[j], r.fx[i & 1]);
      if (last) f8_frag(ws_next, c.w_frag + 16 * j * 128, r.fw[j]);
    }
    if (last) f8_frag(xs_next, c.x_frag, r.fx[0]);
    f8_add<kGated>(acc[(i + MI - 1) % MI], r.part[(i + 1) & 1], r.s);
#pragma unroll
    for (int p = 0; p < kP; ++p) r.s[p] = sx[i >> 2][i & 3] * sw[p];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if (last)
        __builtin_amdgcn_sched_group_barrier(0x100, 2, 0);
      else
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x020, 4, 0);
      __builtin_amdgcn_sched_group_barrier(0x002, 6, 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
#endif
}

// steps I, I + 1, ... kUnroll - 1 of a group (kAll: whole groups, no exits)
template <class Tile, bool kGated, int I, bool kAll>
__device__ __forceinline__ void f8_steps(const F8Ctx<Tile, kGated>& c, int step,
                                         f32x4_t (&acc)[Tile::MI][4], F8Regs<kGated>& r,
                                         F8Scales<Tile, kGated> (&sc)[Tile::SX]) {
  if constexpr (I < (kAll ? Tile::kUnroll : Tile::kUnroll - 1)) {
    if (!kAll && step >= c.nsteps) return;
    f8_step<Tile, kGated, I % Tile::SW, I % Tile::SX>(c, step, acc, r, sc);
    f8_steps<Tile, kGated, I + 1, kAll>(c, step + 1, acc, r, sc);
  }
}

template <class Tile, bool kGated, int I>
__device__ __forceinline__ void f8_first_loads(const F8Ctx<Tile, kGated>& c,
                                               F8Scales<Tile, kGated> (&sc)[Tile::SX]) {
  // in the order of the steps: scales and X(i), W(i); with one more weight
  // stage W(0) first, then scales and X(i), W(i + 1)
  if constexpr (I < Tile::SX - 1) {
    if (I == 0 && Tile::SW > Tile::SX) f8_issue_w(c, c.W[0], 0);
    f8_issue_scales(c, I, sc[I]);
    f8_issue_x(c, c.X[I], I);
    f8_issue_w(c, c.W[Tile::SW > Tile::SX ? I + 1 : I], Tile::SW > Tile::SX ? I + 1 : I);
    f8_first_loads<Tile, kGated, I + 1>(c, sc);
  }
}

// kPart: store the float32 sums of one part of the reduction (blockIdx.y);
// otherwise round and write Y (gated: the activation and the product first).
template <class Tile, bool kF16, bool kPart, bool kGated>
__global__ __launch_bounds__(64 * Tile::kWaves, Tile::kWavesSimd) void fp8_gemm_kernel(Fp8Args g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int MI = Tile::MI, WN = Tile::WN, SW = Tile::SW, SX = Tile::SX;
  // one object a stage (16 unused bytes where the ring has two activation stages)
  __shared__ __attribute__((aligned(1024))) uint8_t sw0[Tile::kWBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sw1[Tile::kWBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sw2[Tile::kWBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sx0[Tile::kXBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sx1[Tile::kXBytes];
  __shared__ __attribute__((aligned(1024))) uint8_t sx2[2 < SX ? Tile::kXBytes : 16];
  static_assert(SW == 3 && (SX == 2 || SX == 3), "stages");
  uint8_t* const all_w[3] = {sw0, sw1, sw2};
  uint8_t* const all_x[3] = {sx0, sx1, sx2};
  constexpr int kOuts = kGated ? Tile::TN / 2 : Tile::TN;   // outputs (of each projection) a tile
  F8Ctx<Tile, kGated> c;
#pragma unroll
  for (int i = 0; i < SW; ++i) c.W[i] = all_w[i];
#pragma unroll
  for (int i = 0; i < SX; ++i) c.X[i] = all_x[i];
  c.lane = threadIdx.x & 63;
  c.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = c.wave / WN, wn = c.wave % WN;
  const int l16 = c.lane & 15, lq = c.lane >> 4;
  const int mt = (int)((g.T + Tile::TM - 1) / Tile::TM);
  const int nt = (int)((g.rows + kOuts - 1) / kOuts);
  int tm, tn;
  tile_coords(blockIdx.x, mt, nt, tm, tn);
  tm = __builtin_amdgcn_readfirstlane(tm);
  tn = __builtin_amdgcn_readfirstlane(tn);
  const int64_t m0 = (int64_t)tm * Tile::TM, n0 = (int64_t)tn * kOuts;
  const int rows_here = (int)(g.T - m0 < Tile::TM ? g.T - m0 : Tile::TM);
  const int outs_here = (int)(g.rows - n0 < kOuts ? g.rows - n0 : kOuts);
  c.K = (uint32_t)g.cols;
  const int all = (int)((g.cols + 127) / 128);
  {
    const int per = (all + g.splits - 1) / g.splits;
    c.step0 = kPart ? (int)blockIdx.y * per : 0;
    const int end = c.step0 + per < all ? c.step0 + per : all;
    c.nsteps = kPart ? (end > c.step0 ? end - c.step0 : 0) : all;
    if (c.nsteps == 0) c.step0 = 0;
    c.last = all - 1;
    c.tail = tail_step(c.last, c.step0, c.nsteps);
  }
  c.x_base = g.X + m0 * g.cols;
  c.x_bytes = (uint32_t)rows_here * c.K;
  c.w_base[0] = g.W[0] + n0 * g.cols;
  c.w_base[1] = kGated ? g.W[1] + n0 * g.cols : nullptr;
  c.w_bytes = (uint32_t)outs_here * c.K;
  c.T = g.T;
  c.sx_base = g.x_scale + m0;
  c.sx_bytes = (uint32_t)rows_here * 4u;
  c.sx_voff = (uint32_t)(16 * MI * wm + c.lane) * 4u;
  {
    // the wave's outputs lie in one block of 128 (a tile's first output is a
    // multiple of 64, and of 128 where the tile is wider)
    const int64_t first = n0 + (kGated ? 32 * wn : 64 * wn);
    const int64_t row = (first < g.rows ? first : n0) / 128;
    c.sw_base[0] = g.w_scale[0] + row * all;
    c.sw_base[1] = kGated ? g.w_scale[1] + row * all : nullptr;
  }
  {
    const int rl = c.lane >> 3;
#pragma unroll
    for (int par = 0; par < 2; ++par) {
      const int ch = (c.lane & 7) ^ swz_g(8 * par + rl);
      c.voff[par] = (uint32_t)rl * c.K + 16u * (uint32_t)ch;
      c.voff_tail[par] = (uint32_t)c.last * 128u + 16u * (uint32_t)ch < c.K ? c.voff[par] : kOOB;
    }
    const int xr = 16 * MI * wm + l16, wr = 64 * wn + l16;
    c.x_frag = xr * 128 + ((lq ^ swz_g(xr)) << 4);
    c.w_frag = wr * 128 + ((lq ^ swz_g(wr)) << 4);
  }
  f32x4_t acc[MI][4];
#pragma unroll
  for (int i = 0; i < MI; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  F8Scales<Tile, kGated> sc[SX];
  f8_first_loads<Tile, kGated, 0>(c, sc);
  barrier_keep_vmem<F8Ctx<Tile, kGated>::kKeep>();
  F8Regs<kGated> r;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f8_frag(sw0, c.w_frag + 16 * j * 128, r.fw[j]);
    r.part[1][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  f8_frag(sx0, c.x_frag, r.fx[0]);
  r.s[0] = 0.0f;
  if constexpr (kGated) r.s[1] = 0.0f;
  int step = 0;
  for (; step + Tile::kUnroll <= c.nsteps; step += Tile::kUnroll)
    f8_steps<Tile, kGated, 0, true>(c, step, acc, r, sc);
  f8_steps<Tile, kGated, 0, false>(c, step, acc, r, sc);
  f8_add<kGated>(acc[MI - 1], r.part[1], r.s);
  // the scales loaded past the last step are used too, for all the compiler
  // knows: it may not drop their loads, which the wait counts include
#pragma unroll
  for (int i = 0; i < SX; ++i) {
#pragma unroll
    for (int q = 0; q < (MI + 3) / 4; ++q) asm volatile("" ::"v"(sc[i].x[q]));
#pragma unroll
    for (int p = 0; p < (kGated ? 2 : 1); ++p) asm volatile("" ::"v"(sc[i].w[p]));
  }

  // acc[i][j][e]: token 16 i + l16, output 16 j + 4 lq + e of the wave (gated: j
  // < 2 of the gate, j >= 2 of the up projection, outputs 16 (j & 1) + ...)
  if constexpr (kPart) {
    // the stages must not be freed to another workgroup while DMAs land
    __builtin_amdgcn_s_waitcnt(0);
    const int64_t outs = kGated ? 2 * g.rows : g.rows;
    float* part = g.part + (int64_t)blockIdx.y * g.T * outs;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int64_t t = m0 + 16 * (MI * wm + i) + l16;
      if (t < g.T) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int64_t n = kGated ? n0 + 32 * wn + 16 * (j & 1) + 4 * lq
                                   : n0 + 64 * wn + 16 * j + 4 * lq;
          float* d = part + t * outs + (kGated && j >= 2 ? g.rows : 0) + n;
          if (n + 4 <= g.rows && (g.rows & 3) == 0) {
            *reinterpret_cast<f32x4_t*>(d) = acc[i][j];
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (n + e < g.rows) d[e] = acc[i][j][e];
          }
        }
      }
    }
  } else {
    // Each wave rounds its 16 MI x 64 tile (gated: x 32) into LDS, token rows of
    // 128 (64) bytes with their 16-byte chunks swizzled by the row, and writes
    // whole rows with 16-byte stores.
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();
    constexpr int kRow = kGated ? 64 : 128;       // bytes a token
    constexpr int kOut = 16 * MI * 128;           // bytes a wave
    static_assert(2 * kOut <= Tile::kWBytes && (Tile::kWaves <= 6 || 2 * kOut <= Tile::kXBytes),
                  "two waves' tiles a stage");
    static_assert(Tile::kWaves <= 8, "stages for every wave");
    uint8_t* stg = (c.wave >> 1) == 0 ? sw0 : (c.wave >> 1) == 1 ? sw1
                 : (c.wave >> 1) == 2 ? sw2 : sx0;
    stg += (c.wave & 1) * kOut;
    constexpr int kJ = kGated ? 2 : 4;
    constexpr int kMask = kGated ? 3 : 7;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int lr = 16 * i + l16;
      const int sw = kGated ? (lr >> 1) & kMask : lr & kMask;
#pragma unroll
      for (int j = 0; j < kJ; ++j) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = kGated ? act_value(acc[i][j][e], g.act) * acc[i][j + (kGated ? 2 : 0)][e]
                        : acc[i][j][e];
        *reinterpret_cast<uint2*>(stg + lr * kRow + (((2 * j + (lq >> 1)) ^ sw) << 4) +
                                  8 * (lq & 1)) =
            uint2{pack16x2<kF16>(v[0], v[1]), pack16x2<kF16>(v[2], v[3])};
      }
    }
    constexpr int kLanes = kRow / 16;              // a row
    const int ch = c.lane % kLanes;
    const int64_t n = n0 + (kGated ? 32 : 64) * wn + 8 * ch;
#pragma unroll
    for (int it = 0; it < 16 * MI * kLanes / 64; ++it) {
      const int row = (64 / kLanes) * it + c.lane / kLanes;
      const int sw = kGated ? (row >> 1) & kMask : row & kMask;
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(stg + row * kRow + ((ch ^ sw) << 4));
      const int64_t t = m0 + 16 * MI * wm + row;
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

// Y = RN16(sum of the parts in their order) (gated: act(P_gate) P_up of the
// sums), V consecutive outputs a thread and step (one where rows % 4 leaves
// them unaligned).
template <bool kF16, int V, bool kGated>
__global__ __launch_bounds__(256) void fp8_finish_kernel(Fp8Args g) {
  const int64_t n_all = g.T * g.rows;
  const int64_t outs = kGated ? 2 * g.rows : g.rows;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; i < n_all;
       i += (int64_t)gridDim.x * 256 * V) {
    float v[kGated ? 2 : 1][V];
    const int64_t t = i / g.rows;
    const int64_t n = i - t * g.rows;
#pragma unroll
    for (int p = 0; p < (kGated ? 2 : 1); ++p) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[p][e] = 0.0f;
      const float* src = g.part + t * outs + p * g.rows + n;
#pragma unroll 4
      for (int s = 0; s < g.splits; ++s) {
        const float* q = src + (int64_t)s * g.T * outs;
        if constexpr (V == 4) {
          const f32x4_t x = __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(q));
#pragma unroll
          for (int e = 0; e < 4; ++e) v[p][e] += x[e];
        } else {
          v[p][0] += q[0];
        }
      }
    }
    if constexpr (kGated) {
#pragma unroll
      for (int e = 0; e < V; ++e) v[0][e] = act_value(v[0][e], g.act) * v[kGated ? 1 : 0][e];
    }
    if constexpr (V == 4)
      *reinterpret_cast<uint2*>(g.Y + i) =
          uint2{pack16x2<kF16>(v[0][0], v[0][1]), pack16x2<kF16>(v[0][2], v[0][3])};
    else
      g.Y[i] = (uint16_t)(pack16x2<kF16>(v[0][0], 0.0f) & 0xFFFFu);
  }
}

// ---------------------------------------------------------------------------
// Products of few tokens: the weight streamed once, no LDS on its way.
// ---------------------------------------------------------------------------

// A workgroup of 8 waves owns 16 outputs (gated: of both projections) and all
// (up to 16 TG) tokens; the waves take pieces of kU blocks of 128 columns in
// turn.  Lane l loads the 16 bytes at 16 (l / 16) and at 64 + 16 (l / 16) of
// row l % 16's block of both operands.  All loads of a piece go out before its
// MFMAs.  The waves' float32 sums are added in LDS in a fixed order.  1 x 4096 x
// 4096: 5.7 us for 17 MB, the launch's start and end and four loads one after the
// other; 1 x 22016 x 8192 from memory 35 us, 5.2 TB/s.
//
// kFused: the tokens come in 16 bits and every workgroup quantises all of them
// itself into LDS, which for at most kFp8FusedBytes codes costs less than the
// launch and the round trip of a kernel of their own; the weights of the first
// pieces are in flight meanwhile.  (Each wave quantising in registers what it is
// about to multiply, without LDS or a barrier, leaves most lanes idle and did 1 x
// 8192 x 8192 in 31.8 us, 1 x 4096 x 4096 in 9.7.)
constexpr int kF8SkinnyWaves = 8;
constexpr int kFp8FusedVecs = (int)(kFp8FusedBytes / 8 / (64 * kF8SkinnyWaves));   // a thread

template <int kU>
__device__ __forceinline__ void f8_skinny_load(__amdgpu_buffer_rsrc_t r, uint32_t row, uint32_t K,
                                               int piece, int gq, u32x4_t (&v)[kU][2]) {
#pragma unroll
  for (int u = 0; u < kU; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = (uint32_t)(piece + u) * 128u + 64u * (uint32_t)h + 16u * (uint32_t)gq;
      v[u][h] = __builtin_bit_cast(
          u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, k < K ? row * K + k : kOOB, 0, 0));
    }
}

template <int TG, bool kF16, bool kFused, bool kGated>
__global__ __launch_bounds__(64 * kF8SkinnyWaves) void fp8_skinny_kernel(Fp8Args g) {
#if defined(__HIP_DEVICE_COMPILE__)
  static_assert(!kFused || TG == 1, "");
  constexpr int kP = kGated ? 2 : 1;
  constexpr int kU = 2;
  constexpr int kThreads = 64 * kF8SkinnyWaves;
  constexpr int kType = kF16 ? QLORA_TYPE_FP16 : QLORA_TYPE_BF16;
  __shared__ __attribute__((aligned(16))) float red[kF8SkinnyWaves][kP][TG * 256];
  // fused: the codes, rows of whole blocks and 16 bytes (so the rows of one read
  // start in different banks), and the scales
  __shared__ __attribute__((aligned(16))) uint8_t xc[kFused ? kFp8FusedBytes + 16 * 16 : 16];
  __shared__ float xs[kFused ? kFp8FusedBytes / 128 : 1];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, gq = lane >> 4;
  const uint32_t K = (uint32_t)g.cols;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int outs_here = (int)(g.rows - n0 < 16 ? g.rows - n0 : 16);
  const int pieces = (int)((K + 127) / 128);
  __amdgpu_buffer_rsrc_t wr[kP], swr[kP];
#pragma unroll
  for (int p = 0; p < kP; ++p) {
    wr[p] = make_rsrc(g.W[p] + n0 * g.cols, (uint32_t)outs_here * K);
    swr[p] = make_rsrc(g.w_scale[p] + n0 / 128 * pieces, (uint32_t)pieces * 4u);
  }
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.X, (uint32_t)g.T * K);
  const __amdgpu_buffer_rsrc_t sxr = make_rsrc(g.x_scale, (uint32_t)(g.T * pieces) * 4u);
  f32x4_t acc[kP][TG];
#pragma unroll
  for (int p = 0; p < kP; ++p)
#pragma unroll
    for (int b = 0; b < TG; ++b) acc[p][b] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  // the next piece's loads are in flight while this one is worked on
  struct Piece {
    u32x4_t w[kP][kU][2];
    float sw[kP][kU];
    u32x4_t x[kFused ? 1 : TG][kU][2];
    float sx[TG][kU];
  };
  auto load = [&](int at, Piece& q) {
#pragma unroll
    for (int p = 0; p < kP; ++p) {
      f8_skinny_load<kU>(wr[p], (uint32_t)r16, K, at, gq, q.w[p]);
#pragma unroll
      for (int u = 0; u < kU; ++u)
        q.sw[p][u] = __builtin_bit_cast(
            float, __builtin_amdgcn_raw_buffer_load_b32(swr[p], (uint32_t)(at + u) * 4u, 0, 0));
    }
    if constexpr (!kFused) {
#pragma unroll
      for (int b = 0; b < TG; ++b) {
        f8_skinny_load<kU>(xr, (uint32_t)(16 * b + r16), K, at, gq, q.x[b]);
#pragma unroll
        for (int u = 0; u < kU; ++u)
          q.sx[b][u] = __builtin_bit_cast(
              float, __builtin_amdgcn_raw_buffer_load_b32(
                         sxr, 16 * b + r16 < (int)g.T && at + u < pieces
                                  ? (uint32_t)((at + u) * (int)g.T + 16 * b + r16) * 4u : kOOB,
                         0, 0));
      }
    }
  };
  Piece cur, nxt;
  int at = wave * kU;
  if (at < pieces) load(at, cur);
  const uint32_t xrow = (uint32_t)pieces * 128u + 16u;
  if constexpr (kFused) {
    // 16 threads a block, as in the quantiser
    const int all = (int)g.T * pieces * 16;
    Vec8<kType> x[kFp8FusedVecs];
#pragma unroll
    for (int j = 0; j < kFp8FusedVecs; ++j) {
      const int i = tid + kThreads * j;
      const int block = i >> 4, row = block / pieces;
      const int k = (block - row * pieces) * 128 + 8 * (i & 15);
      x[j].zero();
      if (i < all && k < (int)K) x[j].load(g.X16, (int64_t)row * K + k);
    }
#pragma unroll
    for (int j = 0; j < kFp8FusedVecs; ++j) {
      const int i = tid + kThreads * j;
      const int block = i >> 4, row = block / pieces;
      float m = x[j].largest();
#pragma unroll
      for (int d = 8; d > 0; d >>= 1) m = fp8_maximum(m, __shfl_xor(m, d));
      if (i < all) {
        const BlockScale b(m);
        *reinterpret_cast<uint2*>(xc + (uint32_t)row * xrow +
                                  (uint32_t)(block - row * pieces) * 128u + 8u * (i & 15)) =
            x[j].codes(b);
        if ((i & 15) == 0) xs[block] = b.scale;
      }
    }
    __syncthreads();
  }
  for (; at < pieces; at += kF8SkinnyWaves * kU) {
    load(at + kF8SkinnyWaves * kU, nxt);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      u32x4_t x[TG][2];
      float sx[TG];
      if constexpr (kFused) {
        const bool in = r16 < (int)g.T && at + u < pieces;
        sx[0] = in ? xs[r16 * pieces + at + u] : 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          x[0][h] = u32x4_t{0u, 0u, 0u, 0u};
          if (in)
            x[0][h] = *reinterpret_cast<const u32x4_t*>(
                xc + (uint32_t)r16 * xrow + (uint32_t)(at + u) * 128u + 64u * h + 16u * gq);
        }
      } else {
#pragma unroll
        for (int b = 0; b < TG; ++b) {
#pragma unroll
          for (int h = 0; h < 2; ++h) x[b][h] = cur.x[kFused ? 0 : b][u][h];
          sx[b] = cur.sx[b][u];
        }
      }
#pragma unroll
      for (int p = 0; p < kP; ++p)
#pragma unroll
        for (int b = 0; b < TG; ++b) {
          const f32x4_t part = mfma_e4m3(cur.w[p][u], x[b]);
          const float s = sx[b] * cur.sw[p][u];
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[p][b][e] = __builtin_fmaf(part[e], s, acc[p][b][e]);
        }
    }
    cur = nxt;
  }
  // acc[p][b][e]: output 4 gq + e, token 16 b + r16
#pragma unroll
  for (int p = 0; p < kP; ++p)
#pragma unroll
    for (int b = 0; b < TG; ++b)
      *reinterpret_cast<f32x4_t*>(&red[wave][p][(16 * b + r16) * 16 + 4 * gq]) = acc[p][b];
  __syncthreads();
  for (int i = tid; i < TG * 256; i += kThreads) {
    const int64_t t = i / 16;
    const int64_t n = n0 + i % 16;
    if (t < g.T && n < g.rows) {
      float v[kP];
#pragma unroll
      for (int p = 0; p < kP; ++p) {
        v[p] = 0.0f;
#pragma unroll
        for (int q = 0; q < kF8SkinnyWaves; ++q) v[p] += red[q][p][i];
      }
      const float y = kGated ? act_value(v[0], g.act) * v[kP - 1] : v[0];
      g.Y[t * g.rows + n] = (uint16_t)(pack16x2<kF16>(y, 0.0f) & 0xFFFFu);
    }
  }
#endif
}

template <class Tile, bool kF16, bool kGated>
void fp8_tiles(const Fp8Args& a, hipStream_t stream) {
  constexpr int kOuts = kGated ? Tile::TN / 2 : Tile::TN;
  const dim3 grid((unsigned)(((a.T + Tile::TM - 1) / Tile::TM) * ((a.rows + kOuts - 1) / kOuts)),
                  (unsigned)a.splits);
  const dim3 block(64 * Tile::kWaves);
  if (a.splits == 1)
    hipLaunchKernelGGL((fp8_gemm_kernel<Tile, kF16, false, kGated>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((fp8_gemm_kernel<Tile, kF16, true, kGated>), grid, block, 0, stream, a);
}

template <bool kF16, bool kGated>
hipError_t fp8_launch(const Fp8Args& a, const Fp8Plan& p, hipStream_t stream) {
  switch (p.path) {
    case kFp8Fused:
    case kFp8Skinny: {
      const dim3 grid((unsigned)((a.rows + 15) / 16)), block(64 * kF8SkinnyWaves);
      if (p.path == kFp8Fused)
        hipLaunchKernelGGL((fp8_skinny_kernel<1, kF16, true, kGated>), grid, block, 0, stream, a);
      else if (a.T <= 16)
        hipLaunchKernelGGL((fp8_skinny_kernel<1, kF16, false, kGated>), grid, block, 0, stream, a);
      else
        hipLaunchKernelGGL((fp8_skinny_kernel<2, kF16, false, kGated>), grid, block, 0, stream, a);
      return hipGetLastError();
    }
    case kFp8Tile64x128: fp8_tiles<F8Tile<2, 2, 2, 3, 3>, kF16, kGated>(a, stream); break;
    case kFp8Tile128x128: fp8_tiles<F8Tile<4, 2, 2, 3, 2>, kF16, kGated>(a, stream); break;
    case kFp8Tile128x256: fp8_tiles<F8Tile<4, 2, 4, 3, 3>, kF16, kGated>(a, stream); break;
    case kFp8Tile256x256: fp8_tiles<F8Tile<8, 2, 4, 3, 2>, kF16, kGated>(a, stream); break;
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.splits > 1) {
    const bool quads = a.rows % 4 == 0;
    int64_t blocks = (a.T * a.rows / (quads ? 4 : 1) + 255) / 256;
    if (blocks > 8192) blocks = 8192;
    if (quads)
      hipLaunchKernelGGL((fp8_finish_kernel<kF16, 4, kGated>), dim3((unsigned)blocks), dim3(256), 0,
                         stream, a);
    else
      hipLaunchKernelGGL((fp8_finish_kernel<kF16, 1, kGated>), dim3((unsigned)blocks), dim3(256), 0,
                         stream, a);
    e = hipGetLastError();
  }
  return e;
}

// Rows a thread: 8 where that still makes four workgroups a CU, else 2 or 1.
template <int kType>
void quantize_tokens(const Fp8QuantArgs& a, hipStream_t stream) {
  const int64_t kb = fp8_blocks(a.cols);
  auto grid = [&](int rows) { return dim3((unsigned)kb, (unsigned)((a.rows + rows - 1) / rows)); };
  if (a.rows * kb >= 1024 * 128)
    hipLaunchKernelGGL((fp8_quantize_kernel<kType, 8>), grid(128), dim3(256), 0, stream, a);
  else if (a.rows * kb >= 1024 * 32)
    hipLaunchKernelGGL((fp8_quantize_kernel<kType, 2>), grid(32), dim3(256), 0, stream, a);
  else
    hipLaunchKernelGGL((fp8_quantize_kernel<kType, 1>), grid(16), dim3(256), 0, stream, a);
}

template <int kType>
void quantize_weight(const Fp8QuantArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)fp8_blocks(a.cols), (unsigned)((a.rows + 127) / 128));
  hipLaunchKernelGGL((fp8_quantize_weight_kernel<kType>), grid, dim3(256), 0, stream, a);
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8QuantArgs& a, int x_type, hipStream_t stream) {
  switch (x_type) {
    case QLORA_TYPE_BF16: quantize_tokens<QLORA_TYPE_BF16>(a, stream); break;
    case QLORA_TYPE_FP16: quantize_tokens<QLORA_TYPE_FP16>(a, stream); break;
    case QLORA_TYPE_FP32: quantize_tokens<QLORA_TYPE_FP32>(a, stream); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_fp8_quantize_weight(const Fp8QuantArgs& a, int w_type, hipStream_t stream) {
  switch (w_type) {
    case QLORA_TYPE_BF16: quantize_weight<QLORA_TYPE_BF16>(a, stream); break;
    case QLORA_TYPE_FP16: quantize_weight<QLORA_TYPE_FP16>(a, stream); break;
    case QLORA_TYPE_FP32: quantize_weight<QLORA_TYPE_FP32>(a, stream); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

hipError_t launch_fp8_product(const Fp8Args& a, const Fp8Plan& p, bool gated, bool f16,
                              hipStream_t stream) {
  if (gated) return f16 ? fp8_launch<true, true>(a, p, stream) : fp8_launch<false, true>(a, p, stream);
  return f16 ? fp8_launch<true, false>(a, p, stream) : fp8_launch<false, false>(a, p, stream);
}

}  // namespace qlora
