// The linear layer in 8-bit integers (gfx950, int8 MFMA).
//
//   quantise:  s_i = RN32(max_k |x_ik| / 127),  c_ik = nearest integer to
//              x_ik / s_i (ties to even; 0 where s_i = 0)
//   product:   Y_tn = RN16(sx_t * sw_n * sum_k cx_tk cw_nk)
// with one scale a row: a row is an output channel of the weight, a token of
// the activations.  The sums are exact in 32-bit integers (at most 2^17 - 16
// terms of at most 128^2: given codes of -128 are taken as they are), so no order of summation and no split changes a
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
// border and the tie exactly.
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

// The larger of two magnitudes, NaN if either is: a row that holds a NaN has
// it as its scale.
__device__ __forceinline__ float maximum(float a, float b) {
#if defined(__HIP_DEVICE_COMPILE__)
  return __builtin_elementwise_maximum(a, b);
#else
  return a > b ? a : b;
#endif
}

// A row's scale from its largest magnitude, and what its codes are formed
// with.  A largest magnitude that is infinite or NaN leaves inv 0: codes 0.  A
// scale below 2^-100 would take the reciprocal out of range: the row and the
// scale are multiplied by 2^96 first (exact; the quotients do not change).
struct RowScale {
  float scale, s, inv, up;
  __device__ __forceinline__ explicit RowScale(float largest) {
    scale = __fdiv_rn(largest, 127.0f);
    up = scale < 0x1p-100f ? 0x1p96f : 1.0f;
    s = scale * up;
    inv = s > 0.0f ? __fdiv_rn(1.0f, s) : 0.0f;
  }
};

// Codes of one vector.  x * inv + 1.5 * 2^23 in one FMA rounds x * inv to an
// integer r (its low bits) with one rounding; where the remainder
// x * inv - r stays clear of one half (inv is off by 2^-24 relative, so the
// quotient by under 2^-16), r is the nearest integer to the real quotient.
// Otherwise, about one vector in a thousand, nearest_code decides.  Six
// operations an element instead of sixteen: without this the conversion, not
// the memory, bounds the kernel (13.9 against 10.1 us for 4001 x 4096 bf16).
template <int kType>
__device__ __forceinline__ void store_codes(int8_t* dst, const RowVec<kType>& x,
                                            const RowScale& r) {
  constexpr int N = RowVec<kType>::N;
  uint32_t w[N / 4];
  float far = 0.0f;
#pragma unroll
  for (int q = 0; q < N / 4; ++q) {
    uint32_t t[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float v = x.at(4 * q + e);
      const float m = __builtin_fmaf(v, r.inv, 12582912.0f);
      const float d = __builtin_fmaf(v, r.inv, -(m - 12582912.0f));
      far = fmaxf(far, fabsf(d));
      t[e] = __float_as_uint(m);
    }
    // the low byte of each
    w[q] = perm(perm(t[3], t[2], 0x0C0C0400u), perm(t[1], t[0], 0x0C0C0400u), 0x05040100u);
  }
  if (far > 0.49996f || r.up != 1.0f || r.inv == 0.0f) {
#pragma unroll
    for (int q = 0; q < N / 4; ++q) {
      int c[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        c[e] = r.inv == 0.0f ? 0 : nearest_code(x.at(4 * q + e) * r.up, r.s, r.inv);
      w[q] = pack4(c[0], c[1], c[2], c[3]);
    }
  }
  if constexpr (kType == QLORA_TYPE_FP32)
    *reinterpret_cast<uint32_t*>(dst) = w[0];
  else
    *reinterpret_cast<uint2*>(dst) = uint2{w[0], w[N / 4 - 1]};
}

// kW waves a row (kW = 1: four rows a workgroup, no exchange in LDS).  kNV >
// 0: the row's vectors stay in registers (kNV a lane) between the maximum and
// the codes, one read of the row; kNV = 0: rows too long for that are read
// twice (the second time from the cache).
// Bound by memory: 4001 x 4096 bf16 (49 MB) takes 9.7 us, the rate of a large
// copy (5.0 TB/s); 11008 x 4096 fp32 (225 MB) 37.4 us, 6.0 TB/s, part of it from
// the last-level cache.  Below about 1000 rows the launch and one round trip
// are what it takes: 211 x 11008 5.5 us.
template <int kType, int kNV, int kW>
__global__ __launch_bounds__(kW == 1 ? 256 : 64 * kW) void int8_quantize_kernel(Int8QuantArgs a) {
  constexpr int N = RowVec<kType>::N;
  constexpr int kT = 64 * kW;   // threads a row
  __shared__ float red[kW];
  const int64_t row = kW == 1 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (kW == 1 && row >= a.rows) return;
  const int tid = kW == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int nvec = (int)(a.cols / N);
  const u32x4_t* src = reinterpret_cast<const u32x4_t*>(a.X) + row * (int64_t)nvec;
  RowVec<kType> x[kNV > 0 ? kNV : 1];
  float m = 0.0f;
  if constexpr (kNV > 0) {
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const int i = tid + kT * j;
      x[j].v = i < nvec ? src[i] : u32x4_t{0u, 0u, 0u, 0u};
    }
#pragma unroll
    for (int j = 0; j < kNV; ++j)
#pragma unroll
      for (int e = 0; e < N; ++e) m = maximum(m, fabsf(x[j].at(e)));
  } else {
    for (int i = tid; i < nvec; i += kT) {
      x[0].v = src[i];
#pragma unroll
      for (int e = 0; e < N; ++e) m = maximum(m, fabsf(x[0].at(e)));
    }
  }
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = maximum(m, __shfl_xor(m, d));
  if constexpr (kW > 1) {
    if ((tid & 63) == 0) red[tid >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kW; ++q) m = maximum(m, red[q]);
  }
  const RowScale r(m);
  if (tid == 0) a.scale[row] = r.scale;
  int8_t* dst = a.codes + row * a.cols;
  if constexpr (kNV > 0) {
#pragma unroll
    for (int j = 0; j < kNV; ++j) {
      const int i = tid + kT * j;
      if (i < nvec) store_codes<kType>(dst + (int64_t)i * N, x[j], r);
    }
  } else {
    for (int i = tid; i < nvec; i += kT) {
      x[0].v = src[i];
      store_codes<kType>(dst + (int64_t)i * N, x[0], r);
    }
  }
}

// Waves a row.  Few rows: 16, for latency (211 x 11008 bf16: 5.4 us against 8.1
// with 4).  Many rows: 4 (8192 x 4096 bf16: 21.7 us against 25.3 with one and
// 40.3 with 16), or one for short rows (16384 x 1024 bf16: 14.1 us against 19.4
// with 4).  nvec: 16-byte vectors a row.
int int8_quantize_waves(int64_t rows, int64_t nvec) {
  if (rows < 640) return nvec <= 64 ? 1 : (nvec <= 128 ? 4 : 16);
  return nvec <= 128 ? 1 : 4;
}

template <int kType, int kW>
bool quantize_rows(const Int8QuantArgs& a, hipStream_t stream) {
  const int64_t nvec = a.cols / RowVec<kType>::N;
  const dim3 grid((unsigned)(kW == 1 ? (a.rows + 3) / 4 : a.rows)), block(kW == 1 ? 256 : 64 * kW);
  if (nvec <= 64 * kW * 1)
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 1, kW>), grid, block, 0, stream, a);
  else if (nvec <= 64 * kW * 2)
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 2, kW>), grid, block, 0, stream, a);
  else if (nvec <= 64 * kW * 4)
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 4, kW>), grid, block, 0, stream, a);
  else if (nvec <= 64 * kW * 8)
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 8, kW>), grid, block, 0, stream, a);
  else
    return false;
  return true;
}

template <int kType>
hipError_t quantize_type(const Int8QuantArgs& a, hipStream_t stream) {
  const int w = int8_quantize_waves(a.rows, a.cols / RowVec<kType>::N);
  bool done = false;
  if (w <= 1) done = quantize_rows<kType, 1>(a, stream);
  if (!done && w <= 4) done = quantize_rows<kType, 4>(a, stream);
  if (!done) done = quantize_rows<kType, 16>(a, stream);
  if (!done)
    hipLaunchKernelGGL((int8_quantize_kernel<kType, 0, 16>), dim3((unsigned)a.rows), dim3(1024), 0,
                       stream, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Products of many tokens: tiles through LDS.
// ---------------------------------------------------------------------------

// A workgroup of WM x WN waves computes a TM-token x TN-output tile, each
// wave MI x NJ MFMA blocks of 32 x 32; the reduction advances 128 a step (128
// bytes a row of either operand).  Both operands come by DMA into LDS rings
// of SW weight and SX activation stages, in rows of 8 chunks of 16 bytes,
// chunk' = chunk ^ swz_g(row): the reads of 16 rows at one chunk then touch
// all banks evenly.  The weights are the MFMA's row operand, so a lane's
// accumulators are 4 consecutive outputs of one token.
// What bounds it: with many tokens the matrix cores at the clock the power
// allows (8192 x 11008 x 4096 on 256 x 256 tiles: 327 us, 2.26 POP/s, the pipe busy
// 60% of the cycles at 1.79 GHz); with few the stream of weights (16 x 22016 x
// 8192 on 64 x 128 tiles: 39.4 us, 4.6 TB/s); between them the latency of the
// loads into LDS (211 x 4096 x 11008 on 64 x 128 tiles in 2 splits: 19.6 us, 13
// TB/s out of the L2s, the pipe busy 16%, waves waiting for memory or the barrier
// 55% of their time; on 128 x 128 tiles in 4 splits 18.3 to 23.8 us between cards).
// 128 bytes a row and step: whole cache lines of either operand.
template <int MI_, int NJ_, int WM_, int WN_, int SW_, int SX_>
struct I8Tile {
  static constexpr int MI = MI_, NJ = NJ_, WM = WM_, WN = WN_, SW = SW_, SX = SX_;
  static constexpr int TM = 32 * MI * WM, TN = 32 * NJ * WN, kWaves = WM * WN;
  static constexpr int LX = TM / 8 / kWaves, LW = TN / 8 / kWaves;   // DMAs a wave and step
  static constexpr int kXBytes = TM * 128, kWBytes = TN * 128;
  static_assert(SW == SX || SW == SX + 1, "the wait count below");
  // loads issued after those of step+1 when step ends: the activations of
  // step+SX-1 go out before the weights of step+SW-1
  static constexpr int kKeep =
      SW == SX ? (SX - 2) * (LX + LW) : (SX - 2) * (LX + LW) + LW;
  static constexpr int kUnroll = SW == SX ? SW : SW * SX;
  static_assert(kKeep < 64, "vmcnt");
};

template <class Tile>
struct I8Ctx {
  uint8_t* W[Tile::SW];
  uint8_t* X[Tile::SX];
  int lane, wave;
  int step0, nsteps, last;   // this split's first step and step count; the step with K's tail
  int tail;                  // that step of this split, or -1
  uint32_t K;
  const int8_t *x_base, *w_base;
  uint32_t x_bytes, w_bytes;
  uint32_t voff[2], voff_tail[2];
  int x_frag[4], w_frag[4];  // per 32-byte slice
};

template <class Tile>
__device__ __forceinline__ void i8_issue_x(const I8Ctx<Tile>& c, uint8_t* stage, int step) {
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

// Columns past K of the last step read the next row (or 0 past the range);
// the activations there are 0.
template <class Tile>
__device__ __forceinline__ void i8_issue_w(const I8Ctx<Tile>& c, uint8_t* stage, int step) {
  const int ks = c.step0 + step;
#pragma unroll
  for (int i = 0; i < Tile::LW; ++i) {
    const int blk8 = c.wave * Tile::LW + i;
    const uint32_t soff =
        step_soff(step, c.nsteps, (uint32_t)ks * 128u + (uint32_t)(blk8 * 8) * c.K);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(make_rsrc(c.w_base, c.w_bytes),
                                             (lds_void_t*)(stage + blk8 * 1024), 16,
                                             c.voff[blk8 & 1], soff, 0, 0);
  }
}

template <class Tile>
__device__ __forceinline__ void i8_frags(const I8Ctx<Tile>& c, const uint8_t* xs,
                                         const uint8_t* ws, int s, i32x4_t (&fx)[Tile::MI],
                                         i32x4_t (&fw)[Tile::NJ]) {
#pragma unroll
  for (int j = 0; j < Tile::NJ; ++j)
    fw[j] = *reinterpret_cast<const i32x4_t*>(ws + c.w_frag[s] + 32 * j * 128);
#pragma unroll
  for (int i = 0; i < Tile::MI; ++i)
    fx[i] = *reinterpret_cast<const i32x4_t*>(xs + c.x_frag[s] + 32 * i * 128);
}

// One step on weight stage W and activation stage X (compile-time, so the
// compiler sees that a DMA into one stage does not touch another).  Slice 0
// issues the activations of step+SX-1 and slice 1 the weights of step+SW-1,
// into the stages the previous step read; the barrier before the step's last
// MFMAs waits for the stages of step+1, and the first fragments of the next
// step are read under the MFMAs behind it.
template <class Tile, int W, int X>
__device__ __forceinline__ void i8_step(const I8Ctx<Tile>& c, int step,
                                        i32x16_t (&acc)[Tile::MI][Tile::NJ],
                                        i32x4_t (&fx)[2][Tile::MI], i32x4_t (&fw)[2][Tile::NJ]) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int MI = Tile::MI, NJ = Tile::NJ, SW = Tile::SW, SX = Tile::SX;
  constexpr int kM = MI * NJ;
  constexpr int kR = MI + NJ;
  constexpr int kL = ((Tile::LX > Tile::LW ? Tile::LX : Tile::LW) + kM - 1) / kM;
  const uint8_t* ws = c.W[W];
  const uint8_t* xs = c.X[X];
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int s = 0; s < 3; ++s) {
    const int f = s & 1;
    if (s == 0) i8_issue_x(c, c.X[(X + SX - 1) % SX], step + SX - 1);
    if (s == 1) i8_issue_w(c, c.W[(W + SW - 1) % SW], step + SW - 1);
    i8_frags(c, xs, ws, s + 1, fx[f ^ 1], fw[f ^ 1]);
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
      if (q * kL < loads) __builtin_amdgcn_sched_group_barrier(0x020, kL, 0);
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
  barrier_keep_vmem<Tile::kKeep>();   // the stages of step+1 are complete and visible
  i32x4_t gx[MI], gw[NJ];
  i8_frags(c, c.X[(X + 1) % SX], c.W[(W + 1) % SW], 0, gx, gw);
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

// steps I, I + 1, ... kUnroll - 1 of a group (kAll: whole groups, no exits)
template <class Tile, int I, bool kAll>
__device__ __forceinline__ void i8_steps(const I8Ctx<Tile>& c, int step,
                                         i32x16_t (&acc)[Tile::MI][Tile::NJ],
                                         i32x4_t (&fx)[2][Tile::MI],
                                         i32x4_t (&fw)[2][Tile::NJ]) {
  if constexpr (I < (kAll ? Tile::kUnroll : Tile::kUnroll - 1)) {
    if (!kAll && step >= c.nsteps) return;
    i8_step<Tile, I % Tile::SW, I % Tile::SX>(c, step, acc, fx, fw);
    i8_steps<Tile, I + 1, kAll>(c, step + 1, acc, fx, fw);
  }
}

template <class Tile, int I>
__device__ __forceinline__ void i8_first_loads(const I8Ctx<Tile>& c) {
  // in the order of the steps: X(i), W(i); with one more weight stage W(0)
  // first, then X(i), W(i + 1)
  if constexpr (I < Tile::SX - 1) {
    if (I == 0 && Tile::SW > Tile::SX) i8_issue_w(c, c.W[0], 0);
    i8_issue_x(c, c.X[I], I);
    i8_issue_w(c, c.W[Tile::SW > Tile::SX ? I + 1 : I], Tile::SW > Tile::SX ? I + 1 : I);
    i8_first_loads<Tile, I + 1>(c);
  }
}

// kPart: store the int32 sums of one part of the reduction (blockIdx.y);
// otherwise scale, round and write Y.
template <class Tile, bool kF16, bool kPart>
__global__ __launch_bounds__(64 * Tile::kWaves, Tile::kWaves / 4) void int8_gemm_kernel(
    Int8Args g) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int MI = Tile::MI, NJ = Tile::NJ, WN = Tile::WN, SW = Tile::SW, SX = Tile::SX;
  // one object a stage (16 bytes where the ring has no such stage: unused)
  __shared__ __attribute__((aligned(1024))) uint8_t sw0[0 < SW ? Tile::kWBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sw1[1 < SW ? Tile::kWBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sw2[2 < SW ? Tile::kWBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sw3[3 < SW ? Tile::kWBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sx0[0 < SX ? Tile::kXBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sx1[1 < SX ? Tile::kXBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sx2[2 < SX ? Tile::kXBytes : 16];
  __shared__ __attribute__((aligned(1024))) uint8_t sx3[3 < SX ? Tile::kXBytes : 16];
  static_assert(SW >= 3 && SW <= 4 && SX >= 2 && SX <= 4, "stages");
  uint8_t* const all_w[4] = {sw0, sw1, sw2, sw3};
  uint8_t* const all_x[4] = {sx0, sx1, sx2, sx3};
  I8Ctx<Tile> c;
#pragma unroll
  for (int i = 0; i < SW; ++i) c.W[i] = all_w[i];
#pragma unroll
  for (int i = 0; i < SX; ++i) c.X[i] = all_x[i];
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
    c.tail = tail_step(c.last, c.step0, c.nsteps);
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

  i8_first_loads<Tile, 0>(c);
  barrier_keep_vmem<Tile::kKeep>();
  i32x4_t fx[2][MI], fw[2][NJ];
  i8_frags(c, sx0, sw0, 0, fx[0], fw[0]);
  int step = 0;
  for (; step + Tile::kUnroll <= c.nsteps; step += Tile::kUnroll)
    i8_steps<Tile, 0, true>(c, step, acc, fx, fw);
  i8_steps<Tile, 0, false>(c, step, acc, fx, fw);

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
    static_assert(2 * kOut <= Tile::kWBytes && (Tile::kWaves <= 6 || 2 * kOut <= Tile::kXBytes),
                  "two waves' tiles a stage");
    static_assert(2 * SW >= Tile::kWaves || (SW == 3 && Tile::kWaves == 8), "stages for every wave");
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

// Y = RN16(sx sw sum of the parts), four consecutive outputs a thread and
// step (one where rows % 4 leaves them unaligned).  Integer parts: their order
// does not matter.  2 parts of 211 x 4096: 4.1 us, mostly the launch and one round
// trip.  (The last part to arrive adding all of them instead of a launch of its
// own: 180 x 4096 x 11008 29.0 against 22.8 us, 64 x 4096 x 11008 19.8 against
// 16.7, about 3 of either in a launch that zeroed the counters, which the
// quantiser's launch could do: 26 against 22.8, and equal.)
template <bool kF16, int V>
__global__ __launch_bounds__(256) void int8_finish_kernel(Int8Args g) {
  const int64_t n_all = g.T * g.rows;
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; i < n_all;
       i += (int64_t)gridDim.x * 256 * V) {
    int32_t v[V];
#pragma unroll
    for (int e = 0; e < V; ++e) v[e] = 0;
#pragma unroll 4
    for (int s = 0; s < g.splits; ++s) {
      const int32_t* p = g.part + (int64_t)s * n_all + i;
      if constexpr (V == 4) {
        const i32x4_t x = __builtin_nontemporal_load(reinterpret_cast<const i32x4_t*>(p));
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += x[e];
      } else {
        v[0] += p[0];
      }
    }
    const int64_t t = i / g.rows;
    const int64_t n = i - t * g.rows;
    const float sx = g.x_scale[t];
    if constexpr (V == 4) {
      const f32x4_t sw = *reinterpret_cast<const f32x4_t*>(g.w_scale + n);
      float y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) y[e] = (float)v[e] * sw[e] * sx;
      *reinterpret_cast<uint2*>(g.Y + i) =
          uint2{pack16x2<kF16>(y[0], y[1]), pack16x2<kF16>(y[2], y[3])};
    } else {
      g.Y[i] = (uint16_t)(pack16x2<kF16>((float)v[0] * g.w_scale[n] * sx, 0.0f) & 0xFFFFu);
    }
  }
}

// ---------------------------------------------------------------------------
// Products of few tokens: the weight streamed once, no LDS on its way.
// ---------------------------------------------------------------------------

// A workgroup of 8 waves owns 16 outputs and all (up to 16 TG) tokens; the
// waves take pieces of 128 kU bytes of the rows in turn.  Lane l loads 16
// bytes at 16 (l / 16) of row l % 16 of both operands, twice for the two
// halves of 128 bytes, and each load feeds one 16x16x64 MFMA.  (The two
// halves as 64 contiguous bytes a row and load: 46.8 against 54.6 us for
// 16 x 22016 x 8192 with each lane's 32 bytes contiguous.)  All loads of a
// piece go out before its MFMAs.  The waves' int32 sums are added in LDS.
// Bound by latency: 1 x 4096 x 4096 takes 7.0 us, of which the launch, the
// quantisation, one round trip to memory and the sums are all but 3.4 us.
//
// kFused: the tokens come in 16 bits and every workgroup quantises all of
// them itself into LDS, which for at most kInt8FusedBytes codes costs less
// than the launch and the round trip of a kernel of their own; the loads of
// the first pieces are in flight meanwhile.
constexpr int kSkinnyWaves = 8;
constexpr int kFusedVecs = (int)(kInt8FusedBytes / 8 / (64 * kSkinnyWaves));   // a thread

template <int kU>
__device__ __forceinline__ void skinny_load(__amdgpu_buffer_rsrc_t r, uint32_t row, uint32_t K,
                                            int piece, int gq, i32x4_t (&v)[kU][2]) {
#pragma unroll
  for (int u = 0; u < kU; ++u)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t k = (uint32_t)(piece + u) * 128u + 64u * (uint32_t)h + 16u * (uint32_t)gq;
      v[u][h] = __builtin_bit_cast(
          i32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, k < K ? row * K + k : kOOB, 0, 0));
    }
}

template <int TG, bool kF16, bool kFused>
__global__ __launch_bounds__(64 * kSkinnyWaves) void int8_skinny_kernel(Int8Args g,
                                                                        const uint16_t* X16) {
#if defined(__HIP_DEVICE_COMPILE__)
  static_assert(!kFused || TG == 1, "");
  constexpr int kU = kFused ? 4 : 2;
  constexpr int kThreads = 64 * kSkinnyWaves;
  __shared__ __attribute__((aligned(16))) int32_t red[kSkinnyWaves][TG * 256];
  // fused: the codes, rows of K + 16 bytes (so the rows of one read start in
  // different banks), each row's largest magnitude, and its scale
  __shared__ __attribute__((aligned(16))) uint8_t xc[kFused ? kInt8FusedBytes + 16 * 16 : 16];
  __shared__ uint32_t xmax[16];
  const int tid = threadIdx.x;
  const int lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int r16 = lane & 15, gq = lane >> 4;
  const uint32_t K = (uint32_t)g.cols;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int outs_here = (int)(g.rows - n0 < 16 ? g.rows - n0 : 16);
  const __amdgpu_buffer_rsrc_t wr = make_rsrc(g.W + n0 * g.cols, (uint32_t)outs_here * K);
  const __amdgpu_buffer_rsrc_t xr = make_rsrc(g.X, (uint32_t)g.T * K);
  const int pieces = (int)((K + 127) / 128);
  i32x4_t acc[TG];
#pragma unroll
  for (int b = 0; b < TG; ++b) acc[b] = i32x4_t{0, 0, 0, 0};
  int p = wave * kU;
  i32x4_t w[kU][2];
  skinny_load<kU>(wr, (uint32_t)r16, K, p, gq, w);
  if constexpr (kFused) {
    using Vec = RowVec<kF16 ? QLORA_TYPE_FP16 : QLORA_TYPE_BF16>;
    constexpr int kType = kF16 ? QLORA_TYPE_FP16 : QLORA_TYPE_BF16;
    const int nvec = (int)(K / 8);                  // vectors of 8 a row
    const int all = (int)g.T * nvec;
    const u32x4_t* src = reinterpret_cast<const u32x4_t*>(X16);
    Vec x[kFusedVecs];
#pragma unroll
    for (int j = 0; j < kFusedVecs; ++j) {
      const int i = tid + kThreads * j;
      x[j].v = i < all ? src[i] : u32x4_t{0u, 0u, 0u, 0u};
    }
    if (tid < 16) xmax[tid] = 0u;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kFusedVecs; ++j) {
      if (wave * 64 + kThreads * j < all) {         // uniform: the wave's first vector
        float m = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = maximum(m, fabsf(x[j].at(e)));
        const int i = tid + kThreads * j;
        const int row = i < all ? i / nvec : (int)g.T - 1;
        // one row: reduce in registers first; a border inside the wave: lane
        // by lane (magnitudes order as their bits, NaN above infinity)
        if (__builtin_amdgcn_readfirstlane(row) == __builtin_amdgcn_readlane(row, 63)) {
#pragma unroll
          for (int d = 32; d > 0; d >>= 1) m = maximum(m, __shfl_xor(m, d));
          if (lane == 0) atomicMax(&xmax[row], __float_as_uint(m) & 0x7FFFFFFFu);
        } else {
          atomicMax(&xmax[row], __float_as_uint(m) & 0x7FFFFFFFu);
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kFusedVecs; ++j) {
      const int i = tid + kThreads * j;
      if (i < all) {
        const int row = i / nvec;
        const RowScale s(__uint_as_float(xmax[row]));
        int8_t* const dst = reinterpret_cast<int8_t*>(xc) + row * (int)(K + 16);
        store_codes<kType>(dst + (i - row * nvec) * 8, x[j], s);
      }
    }
    __syncthreads();
  }
  for (; p < pieces; p += kSkinnyWaves * kU) {
    i32x4_t x[TG][kU][2];
    if constexpr (kFused) {
#pragma unroll
      for (int u = 0; u < kU; ++u)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t k = (uint32_t)(p + u) * 128u + 64u * (uint32_t)h + 16u * (uint32_t)gq;
          x[0][u][h] = i32x4_t{0, 0, 0, 0};
          if (k < K && r16 < (int)g.T)
            x[0][u][h] = *reinterpret_cast<const i32x4_t*>(xc + (uint32_t)r16 * (K + 16) + k);
        }
    } else {
#pragma unroll
      for (int b = 0; b < TG; ++b)
        skinny_load<kU>(xr, (uint32_t)(16 * b + r16), K, p, gq, x[b]);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int b = 0; b < TG; ++b)
          acc[b] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[u][h], x[b][u][h], acc[b], 0, 0, 0);
    if (p + kSkinnyWaves * kU < pieces)
      skinny_load<kU>(wr, (uint32_t)r16, K, p + kSkinnyWaves * kU, gq, w);
  }
  // acc[b][e]: output 4 gq + e, token 16 b + r16
#pragma unroll
  for (int b = 0; b < TG; ++b)
    *reinterpret_cast<i32x4_t*>(&red[wave][(16 * b + r16) * 16 + 4 * gq]) = acc[b];
  __syncthreads();
  for (int i = tid; i < TG * 256; i += kThreads) {
    const int64_t t = i / 16;
    const int64_t n = n0 + i % 16;
    if (t < g.T && n < g.rows) {
      int32_t v = 0;
#pragma unroll
      for (int q = 0; q < kSkinnyWaves; ++q) v += red[q][i];
      const float sx = kFused ? RowScale(__uint_as_float(xmax[t])).scale : g.x_scale[t];
      const float y = (float)v * g.w_scale[n] * sx;
      g.Y[t * g.rows + n] = (uint16_t)(pack16x2<kF16>(y, 0.0f) & 0xFFFFu);
    }
  }
#endif
}

template <class Tile, bool kF16>
void int8_tiles(const Int8Args& a, hipStream_t stream) {
  const dim3 grid((unsigned)(((a.T + Tile::TM - 1) / Tile::TM) *
                             ((a.rows + Tile::TN - 1) / Tile::TN)),
                  (unsigned)a.splits);
  const dim3 block(64 * Tile::kWaves);
  if (a.splits == 1)
    hipLaunchKernelGGL((int8_gemm_kernel<Tile, kF16, false>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((int8_gemm_kernel<Tile, kF16, true>), grid, block, 0, stream, a);
}

template <bool kF16>
hipError_t int8_launch(const Int8Args& a, const uint16_t* X16, const Int8Plan& p,
                       hipStream_t stream) {
  switch (p.path) {
    case kInt8Fused:
    case kInt8Skinny: {
      const dim3 grid((unsigned)((a.rows + 15) / 16)), block(64 * kSkinnyWaves);
      if (p.path == kInt8Fused)
        hipLaunchKernelGGL((int8_skinny_kernel<1, kF16, true>), grid, block, 0, stream, a, X16);
      else if (a.T <= 16)
        hipLaunchKernelGGL((int8_skinny_kernel<1, kF16, false>), grid, block, 0, stream, a, X16);
      else if (a.T <= 32)
        hipLaunchKernelGGL((int8_skinny_kernel<2, kF16, false>), grid, block, 0, stream, a, X16);
      else
        hipLaunchKernelGGL((int8_skinny_kernel<4, kF16, false>), grid, block, 0, stream, a, X16);
      return hipGetLastError();
    }
    case kInt8Tile64x128: int8_tiles<I8Tile<1, 2, 2, 2, 3, 3>, kF16>(a, stream); break;
    case kInt8Tile128x128: int8_tiles<I8Tile<2, 2, 2, 2, 4, 4>, kF16>(a, stream); break;
    case kInt8Tile128x256: int8_tiles<I8Tile<4, 2, 1, 4, 3, 3>, kF16>(a, stream); break;
    case kInt8Tile256x256: int8_tiles<I8Tile<4, 2, 2, 4, 3, 2>, kF16>(a, stream); break;
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.splits > 1) {
    const bool quads = a.rows % 4 == 0;
    int64_t blocks = (a.T * a.rows / (quads ? 4 : 1) + 255) / 256;
    if (blocks > 8192) blocks = 8192;
    if (quads)
      hipLaunchKernelGGL((int8_finish_kernel<kF16, 4>), dim3((unsigned)blocks), dim3(256), 0,
                         stream, a);
    else
      hipLaunchKernelGGL((int8_finish_kernel<kF16, 1>), dim3((unsigned)blocks), dim3(256), 0,
                         stream, a);
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

hipError_t launch_int8_product(const Int8Args& a, const uint16_t* X16, const Int8Plan& p, bool f16,
                               hipStream_t stream) {
  return f16 ? int8_launch<true>(a, X16, p, stream) : int8_launch<false>(a, X16, p, stream);
}

}  // namespace qlora
