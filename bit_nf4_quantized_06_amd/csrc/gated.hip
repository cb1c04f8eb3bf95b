// The gated feed-forward block's own kernels (gfx950); its matrix products are
// the dense layer's (gemm.hip, gemv.hip, lora.hip).
//
//   P_i = X dequant(W_i)^T + s (X A_i^T) B_i^T,   H = act(P_gate) P_up
//   dG = dH P_up act'(P_gate),   dU = dH act(P_gate)
//   dX = sum_i d_i dequant(W_i) + s (d_i B_i) A_i
//   dA_i = s (d_i B_i)^T X,   dB_i = s d_i^T U_i,   U_i = X A_i^T
//
// U on its way to P and d B on its way to dX are two 16-bit terms each, s enters
// the float32 products (gated_reduce_kernel says why).
//
// Roundings of the backward.  dG and dU meet the weights in 16 bits, like every
// gradient between two layers; dX is a 16-bit tensor itself.  The adapters'
// gradients are float32, so there d and d B are split into 16-bit terms, each the
// rest of the ones before it, whose products add up in float32: three in bf16 (24
// bits; with two, 2^-17 of d, dB was off by 3.1e-6 in norm, twice what float32
// sums are) and two in fp16 (22 bits).  The kernel that forms dG and dU multiplies
// the terms by B from registers, and dB's forms d again from dH and the
// projections, since reading the terms of two gradients would be more bytes than
// reading the three inputs.  In fp16 the rest of d is multiplied by 2^11 first and
// summed apart, so it is no smaller than the value and leaves the range of normal
// numbers no sooner (22 bits from 2^-14 on, none closer than 2^-36); d B's terms
// are those of d B times a power of two for 128 rows.
#include "act.h"
#include "device_common.h"
#include "gated_kernels.h"
#include "group.h"
#include "step_offsets.h"

namespace qlora {

namespace {

template <bool kF16>
__device__ __forceinline__ float elem16(const u32x4_t& v, int i) {
  const uint32_t w = v[i >> 1];
  if (!kF16) return (i & 1) ? bf16_hi_to_f32(w) : bf16_lo_to_f32(w);
  return lo16_to_f32<true>((i & 1) ? w >> 16 : w);
}

constexpr int kTerms(bool f16) { return grad_terms(f16); }

// What the rest of d is multiplied by before it is rounded to the next term.
constexpr float term_up(bool f16) { return f16 ? 2048.0f : 1.0f; }

// Two values in 16-bit terms.  (A value past the type's range is an infinite first
// term and a NaN in the next: what it meets is not finite either way.)
template <bool kF16>
__device__ __forceinline__ void split_pair(float a, float b, uint32_t (&t)[kTerms(kF16)]) {
#pragma unroll
  for (int k = 0; k < kTerms(kF16); ++k) {
    t[k] = pack16x2<kF16>(a, b);
#if defined(__HIP_DEVICE_COMPILE__)
    if (!kF16) asm("" : "+v"(t[k]));   // one conversion of the pair, not one more for each half
#endif
    if (k + 1 < kTerms(kF16)) {
      a = (a - lo16_to_f32<kF16>(t[k])) * term_up(kF16);
      b = (b - (kF16 ? lo16_to_f32<true>(t[k] >> 16) : bf16_hi_to_f32(t[k]))) * term_up(kF16);
    }
  }
}

// dG (t[0]) and dU (t[1]) of 8 elements in terms.
template <bool kF16, int kAct>
__device__ __forceinline__ void gate_grads(const u32x4_t (&x)[3],
                                           u32x4_t (&t)[2][kTerms(kF16)]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float g[2], u[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float value, slope;
      act_both<kAct>(elem16<kF16>(x[1], 2 * q + e), value, slope);
      const float d = elem16<kF16>(x[0], 2 * q + e);
      g[e] = d * elem16<kF16>(x[2], 2 * q + e) * slope;
      u[e] = d * value;
    }
    uint32_t w[kTerms(kF16)];
    split_pair<kF16>(g[0], g[1], w);
#pragma unroll
    for (int k = 0; k < kTerms(kF16); ++k) t[0][k][q] = w[k];
    split_pair<kF16>(u[0], u[1], w);
#pragma unroll
    for (int k = 0; k < kTerms(kF16); ++k) t[1][k][q] = w[k];
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// dG, dU and the partials of dG B_gate and dU B_up.
//
// Workgroup = 4 waves over 128 tokens, wave w tokens 32 w .. + 31 (two MFMA
// 16x16x32 row groups); it walks one split of the rows of W (the columns of dH)
// 64 at a time.  A lane holds 8 consecutive columns of one token, which is the
// MFMA's operand, so dH and the projections go to registers, dG and dU are
// formed there, stored, and multiplied from there.  B_gate and B_up (64 rows of
// r, as in memory) go by DMA into one of two LDS stages, read transposed.
//
// 8192 tokens of 11008 x 4096, r 64, bf16: 218 to 227 us with the card's clock for
// 0.57 GB read and 0.39 written (4.2 to 4.4 TB/s; a copy would take 180 to 190);
// fp16 230, at rank 48 203, at rank 128 312.  Waves wait for the vector and matrix
// units 57% of their time and for memory or a barrier 14%: 24 vector operations an
// element, two of them at a quarter of the rate.  fp16's second term has accumulators of its own, so from rank 64 on it
// runs one wave a SIMD, at 112 and 128 with spills (23 and up to 103 registers).
// ---------------------------------------------------------------------------
template <int NJ>
struct GbCtx {
  __amdgpu_buffer_rsrc_t in[3], out[2], br[2];
  uint32_t off[2];          // row group: the lane's byte offset at column 0, or OOB
  int64_t kb, ke;
  int wave, lane;
};

// At rank 64, rows of 128 bytes, the 32-byte pieces of a row of B lie at piece ^
// gb_swz(row) in LDS, so the four rows of a transposed read touch different banks
// (8192 tokens of 11008 x 4096 235 -> 226 us with the shorter slope and splitting).
// Other ranks' rows do so anyway, but for 128, where the addresses that the swizzle
// takes make fp16 spill (312 -> 354 us).
template <int NJ>
__device__ __forceinline__ int gb_swz(int row) {
  return NJ == 4 ? (row >> 1) & 1 : 0;
}

template <int NJ>
__device__ __forceinline__ void gb_load_b(const GbCtx<NJ>& c, int it, uint16_t* stage) {
  const int64_t k0 = c.kb + (int64_t)it * 64;
#pragma unroll
  for (int i = 0; i < NJ; ++i) {
    const int q = c.wave * NJ + i;      // 1 KB piece of the 4 NJ KB of both
    const int part = q >= 2 * NJ;
    const uint32_t byte = (uint32_t)(1024 * (q - part * 2 * NJ) + 16 * c.lane);
    const int row = (int)(byte / (32 * NJ));
    const uint32_t off = k0 + row < c.ke
                             ? (uint32_t)(k0 * 32 * NJ) + (byte ^ (uint32_t)(32 * gb_swz<NJ>(row)))
                             : kOOB;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(part ? c.br[1] : c.br[0],
                                             (lds_void_t*)(stage + q * 512), 16, off, 0, 0, 0);
  }
}

template <int NJ>
__device__ __forceinline__ uint32_t gb_off(const GbCtx<NJ>& c, int it, int u, int g) {
  const int64_t k = c.kb + (int64_t)it * 64 + 8 * (c.lane >> 4) + 32 * u;
  return k < c.ke && c.off[g] != kOOB ? c.off[g] + (uint32_t)(k * 2) : kOOB;
}

template <int NJ>
__device__ __forceinline__ void gb_load_x(const GbCtx<NJ>& c, int it, int g,
                                          u32x4_t (&x)[2][2][3]) {
#pragma unroll
  for (int q = 0; q < 3; ++q)
#pragma unroll
    for (int u = 0; u < 2; ++u) x[u][g][q] = bload16(c.in[q], gb_off(c, it, u, g));
}

// One iteration on stage SI: B of the next goes out first, then for each row
// group this one's gradients, their stores and the next one's inputs, and the
// products.  Both halves of a token's 128 bytes are loaded (stored) one after the
// other: half an iteration apart, the second found the line gone from the caches.  What is newer than B's loads at the next wait: 8
// stores and 12 loads.
template <int NJ, bool kF16, int kAct, int SI>
__device__ __forceinline__ void gb_iter(const GbCtx<NJ>& c, int it, uint16_t* const (&st)[2],
                                        u32x4_t (&x)[2][2][3], f32x4_t (&acc)[2][2][NJ],
                                        f32x4_t (&low)[2][2][kF16 ? NJ : 1]) {
#if defined(__HIP_DEVICE_COMPILE__)
  // B(it) has landed, everybody has it, and everybody is done with the other stage
  __builtin_amdgcn_s_waitcnt((20 & 0xF) | ((20 >> 4) << 14) | (7 << 4) | (0xF << 8));
  asm volatile("s_barrier" ::: "memory");
  gb_load_b(c, it + 1, st[SI ^ 1]);
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    u32x4_t t[2][2][kTerms(kF16)];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      gate_grads<kF16, kAct>(x[u][g], t[u]);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int u = 0; u < 2; ++u)
        __builtin_amdgcn_raw_buffer_store_b128(t[u][p][0], c.out[p], gb_off(c, it, u, g), 0, 0);
    gb_load_x(c, it + 1, g, x);
    __builtin_amdgcn_sched_barrier(0);
    // (a term of every accumulator before the next term: no MFMA waits for the
    // one before it)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int row = 32 * u + 8 * (c.lane >> 4) + ((c.lane & 15) >> 2);
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        u32x4_t rf[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) {
          const uint16_t* b = st[SI] + p * (64 * 16 * NJ) + row * (16 * NJ) +
                              16 * (j ^ gb_swz<NJ>(row)) + 4 * (c.lane & 3);
          rf[j] = ld_tr_pair(b, b + 4 * (16 * NJ));
        }
#pragma unroll
        for (int k = 0; k < kTerms(kF16); ++k)
#pragma unroll
          for (int j = 0; j < NJ; ++j) {
            if (kF16 && k > 0)
              low[p][g][kF16 ? j : 0] = mfma16<kF16>(t[u][p][k], rf[j], low[p][g][kF16 ? j : 0]);
            else
              acc[p][g][j] = mfma16<kF16>(t[u][p][k], rf[j], acc[p][g][j]);
          }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
  }
#endif
}

template <int NJ, bool kF16, int kAct>
__global__ __launch_bounds__(256, NJ <= (kF16 ? 3 : 4) ? 2 : 1) void gated_bwd_kernel(GatedBwd a, int64_t chunk) {
#if defined(__HIP_DEVICE_COMPILE__)
  __shared__ __attribute__((aligned(1024))) uint16_t s0[2 * 64 * 16 * NJ];
  __shared__ __attribute__((aligned(1024))) uint16_t s1[2 * 64 * 16 * NJ];
  uint16_t* const st[2] = {s0, s1};
  GbCtx<NJ> c;
  c.lane = threadIdx.x & 63;
  c.wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t m0 = (int64_t)blockIdx.x * 128 + 32 * c.wave;
  c.kb = (int64_t)blockIdx.y * chunk;
  c.ke = c.kb + chunk < a.rows ? c.kb + chunk : a.rows;
  const int nit = c.ke > c.kb ? (int)((c.ke - c.kb + 63) / 64) : 0;
  const uint64_t bytes = (uint64_t)a.T * a.rows * 2;
  c.in[0] = rsrc(a.dH, bytes);
  c.in[1] = rsrc(a.Pg, bytes);
  c.in[2] = rsrc(a.Pu, bytes);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    c.out[p] = rsrc(a.d[p], bytes);
    c.br[p] = rsrc(a.B[p], (uint64_t)a.rows * (16 * NJ) * 2);
  }
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    const int64_t t = m0 + 16 * g + (c.lane & 15);
    c.off[g] = t < a.T ? (uint32_t)(t * a.rows * 2) : kOOB;
  }
  f32x4_t acc[2][2][NJ];
  f32x4_t low[2][2][kF16 ? NJ : 1];
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int g = 0; g < 2; ++g) {
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[p][g][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < (kF16 ? NJ : 1); ++j) low[p][g][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  if (nit > 0) {
    u32x4_t x[2][2][3];
    gb_load_b(c, 0, s0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int g = 0; g < 2; ++g) gb_load_x(c, 0, g, x);
    // only 12 loads are newer than B's before the first iteration
    __builtin_amdgcn_s_waitcnt(12 | (7 << 4) | (0xF << 8));
    int it = 0;
    for (; it + 2 <= nit; it += 2) {
      gb_iter<NJ, kF16, kAct, 0>(c, it, st, x, acc, low);
      gb_iter<NJ, kF16, kAct, 1>(c, it + 1, st, x, acc, low);
    }
    if (it < nit) gb_iter<NJ, kF16, kAct, 0>(c, it, st, x, acc, low);
    // the inputs loaded past the end are used too, for all the compiler knows:
    // it may not drop their loads, which the wait counts include
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int g = 0; g < 2; ++g)
#pragma unroll
        for (int q = 0; q < 3; ++q) asm volatile("" ::"v"(x[u][g][q]));
    // the loads issued past the end read nothing; let them land before exit
    __builtin_amdgcn_s_waitcnt((7 << 4) | (0xF << 8));
  }
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float* out = a.P[p] + (int64_t)blockIdx.y * a.T * (16 * NJ);
    float m = 0.0f;
#pragma unroll
    for (int g = 0; g < 2; ++g)
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t t = m0 + 16 * g + 4 * (c.lane >> 4) + e;
          float v = acc[p][g][j][e];
          if constexpr (kF16) v += low[p][g][j][e] * (1.0f / term_up(true));
          m = larger_finite(m, v);   // rows past T are 0
          if (t < a.T) out[t * (16 * NJ) + 16 * j + (c.lane & 15)] = v;
        }
    if constexpr (kF16) {
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
      if (c.lane == 0)
        a.ts[p].largest[((int64_t)blockIdx.y * a.ts[p].slots + blockIdx.x) * 4 + c.wave] = m;
    }
  }
#endif
}

int gated_bwd_splits(int64_t T, int64_t rows) {
  const int64_t tiles = (T + 127) / 128;
  int64_t s = (512 + tiles - 1) / tiles;
  const int64_t most = (rows + 127) / 128;
  if (s > most) s = most;
  if (s > 32) s = 32;
  return (int)(s < 1 ? 1 : s);
}

static int64_t chunk_of(int64_t n, int splits, int64_t unit) {
  const int64_t c = (n + splits - 1) / splits;
  return (c + unit - 1) / unit * unit;
}

hipError_t launch_gated_bwd(const GatedBwd& a, hipStream_t stream) {
  const int64_t chunk = chunk_of(a.rows, a.splits, 64);
  const dim3 grid((unsigned)((a.T + 127) / 128), (unsigned)a.splits);
  switch (a.r >> 4) {
#define QLORA_GATED_LAUNCH(NJ, F16, ACT)                                                         \
  hipLaunchKernelGGL((gated_bwd_kernel<NJ, F16, ACT>), grid, dim3(256), 0, stream, a, chunk)
#define QLORA_GATED_CASE(NJ)                                                                     \
  case NJ:                                                                                       \
    if (a.act_fn == QLORA_ACT_SILU) {                                                            \
      if (a.f16) QLORA_GATED_LAUNCH(NJ, true, QLORA_ACT_SILU);                                   \
      else QLORA_GATED_LAUNCH(NJ, false, QLORA_ACT_SILU);                                        \
    } else {                                                                                     \
      if (a.f16) QLORA_GATED_LAUNCH(NJ, true, QLORA_ACT_GELU_TANH);                              \
      else QLORA_GATED_LAUNCH(NJ, false, QLORA_ACT_GELU_TANH);                                   \
    }                                                                                            \
    break;
    QLORA_GATED_CASE(1) QLORA_GATED_CASE(2) QLORA_GATED_CASE(3) QLORA_GATED_CASE(4)
    QLORA_GATED_CASE(5) QLORA_GATED_CASE(6) QLORA_GATED_CASE(7) QLORA_GATED_CASE(8)
#undef QLORA_GATED_CASE
#undef QLORA_GATED_LAUNCH
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// dB_i = d_i^T U_i and dA_i = (d_i B_i)^T X: split partials over the tokens.
//
// A workgroup of 4 waves takes 128 columns q of the wide operand (dB: of the
// gradients d, both; dA: of X), wave w columns 32 w .. + 31, and 16 NP of the r
// columns p of the narrow one (U, or the terms of d B) from p0 on, 32 tokens at a
// time.  The reduction runs over tokens, so both operands need 8 consecutive
// tokens of one column: they go to registers (the next 32 tokens' while these are
// worked on), to LDS -- dB's wide operand as d's terms, formed there from dH and
// both projections -- and ds_read_b64_tr_b16 hands each lane 4 consecutive tokens
// of one column.  Planes of the wide operand: 32 rows x 16 chunks of 8, chunk' =
// chunk ^ f(row), as in the dense layer's gradients.  dU's terms take the place of
// dG's in LDS (32 KB instead of 56), so three workgroups fit a CU.
//
// 8192 tokens of 11008 x 4096, r 64, bf16: 194 us for 0.71 GB read (3.7 TB/s); 210
// without the narrow planes' swizzle (as B's in the kernel above; bank conflicts
// 16% of the cycles, now 5%).  Steps before that, on cards with a lower clock: 283
// with the activation chosen at run time, 250 with both gradients' terms in LDS at
// once, 228.  Waves wait for the vector and matrix units 49% of their time (busy 37%
// and 23%: d is formed again, 24 vector operations an element) and for memory or a
// barrier 14%.  509 tokens of 2736 x 1024, r 16, fp16: 9.5 us, mostly the latency of
// four iterations.
// ---------------------------------------------------------------------------
template <int NP, bool kF16, int kAct, bool kA>
__device__ __forceinline__ void grads_run(const GatedGrads& a, int64_t chunk, int qb,
                                          uint16_t* lds) {
#if defined(__HIP_DEVICE_COMPILE__)
  constexpr int kT = kTerms(kF16);
  constexpr int kWide = kA ? 1 : kT, kNarrow = kA ? 2 * kT : 2;   // planes
  uint16_t* const wide = lds;
  uint16_t* const narrow = lds + kWide * 32 * 128;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t Q = kA ? a.cols : a.rows;
  const int64_t q0 = (int64_t)qb * 128;
  const int p0 = (int)blockIdx.z * 16 * NP;
  const int64_t tb = (int64_t)blockIdx.y * chunk;
  const int64_t te = tb + chunk < a.T ? tb + chunk : a.T;
  const int nit = te > tb ? (int)((te - tb + 31) / 32) : 0;
  const uint64_t bytes = (uint64_t)a.T * Q * 2;
  const __amdgpu_buffer_rsrc_t in[3] = {rsrc(kA ? a.X : a.dH, bytes), rsrc(a.Pg, bytes),
                                        rsrc(a.Pu, bytes)};
  // thread: rows tid / 16 and + 16 of the 32, chunk tid % 16 (8 columns); of a
  // narrow plane 16 bytes, 2 NP threads a row
  const int row = tid >> 4, ch = tid & 15;
  const int64_t col = q0 + 8 * ch;
  const int nrow = tid / (2 * NP), ncol = p0 + 8 * (tid % (2 * NP));
  const bool has = tid < 64 * NP && ncol < a.r;
  u32x4_t x[2][kA ? 1 : 3], nv[kNarrow];
  auto load = [&](int it) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t t = tb + (int64_t)it * 32 + row + 16 * h;
      const uint32_t off = t < te && col < Q ? (uint32_t)((t * Q + col) * 2) : kOOB;
#pragma unroll
      for (int q = 0; q < (kA ? 1 : 3); ++q) x[h][q] = bload16(in[q], off);
    }
    const int64_t t = tb + (int64_t)it * 32 + nrow;
    const uint32_t off = has && t < te ? (uint32_t)((t * a.r + ncol) * 2) : kOOB;
#pragma unroll
    for (int k = 0; k < kNarrow; ++k) {
      const uint16_t* base = kA ? a.terms[k / kT] + (int64_t)(k % kT) * a.T * a.r : a.U[kA ? 0 : k];
      nv[k] = bload16(rsrc(base, (uint64_t)a.T * a.r * 2), off);
    }
  };
  f32x4_t acc[2][NP][2];
  f32x4_t low[2][kF16 ? NP : 1][2];
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int g = 0; g < 2; ++g) {
#pragma unroll
      for (int j = 0; j < NP; ++j) acc[p][j][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int j = 0; j < (kF16 ? NP : 1); ++j) low[p][j][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    }
  auto fold = [&](int it) {
    const int64_t tile = (tb + 32 * (int64_t)it) / 128;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const float down = a.down[p][tile];
#pragma unroll
      for (int j = 0; j < NP; ++j)
#pragma unroll
        for (int g = 0; g < 2; ++g) {
          low[p][kF16 ? j : 0][g] += acc[p][j][g] * down;
          acc[p][j][g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        }
    }
  };
  if (nit > 0) load(0);
  for (int it = 0; it < nit; ++it) {
    if constexpr (kA && kF16) {
      // the tile before is done (a part starts at a multiple of 32 rows): its
      // products join `low`, here the sum of the tiles, in their own scale
      if (it > 0 && ((tb >> 5) + it) % 4 == 0) fold(it - 1);
    }
    __syncthreads();                           // everybody done with the previous planes
    u32x4_t t[2][kA ? 1 : 2][kT];              // row, gradient, term
    if constexpr (!kA) {
#pragma unroll
      for (int h = 0; h < 2; ++h) gate_grads<kF16, kAct>(x[h], t[h]);
    }
    auto store_wide = [&](int p) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = row + 16 * h;
        const int f = 4 * (r & 3) + 2 * ((r >> 3) & 1);
        uint16_t* const dst = wide + r * 128 + ((ch ^ f) << 3);
        if constexpr (kA) {
          *reinterpret_cast<u32x4_t*>(dst) = x[h][0];
        } else {
#pragma unroll
          for (int k = 0; k < kT; ++k)
            *reinterpret_cast<u32x4_t*>(dst + k * 32 * 128) = t[h][p][k];
        }
      }
    };
    store_wide(0);
    if (tid < 64 * NP) {
#pragma unroll
      for (int k = 0; k < kNarrow; ++k)
        *reinterpret_cast<u32x4_t*>(narrow + k * 32 * 16 * NP +
                                    (tid * 8 ^ 16 * gb_swz<NP>(nrow))) = nv[k];
    }
    if (it + 1 < nit) load(it + 1);
    __syncthreads();
    const int b = lane & 3;
    const int r0 = 8 * (lane >> 4) + ((lane & 15) >> 2);
    const int f = 4 * (r0 & 3) + 2 * ((r0 >> 3) & 1);   // the same 4 rows on
    auto wide_frag = [&](int plane, int g) {
      const int cc = 32 * wave + 16 * g + 4 * b;
      const uint16_t* s = wide + plane * 32 * 128 + r0 * 128 + (((cc >> 3) ^ f) << 3) + (cc & 7);
      return ld_tr_pair(s, s + 4 * 128);
    };
    auto narrow_frag = [&](int plane, int j) {
      const uint16_t* s = narrow + plane * 32 * 16 * NP + r0 * (16 * NP) +
                          16 * (j ^ gb_swz<NP>(r0)) + 4 * b;
      return ld_tr_pair(s, s + 4 * (16 * NP));
    };
    u32x4_t wf[2];
    if constexpr (kA) {
#pragma unroll
      for (int g = 0; g < 2; ++g) wf[g] = wide_frag(0, g);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      if constexpr (!kA) {
        if (p == 1) {                          // dU's terms in the place of dG's
          __syncthreads();
          store_wide(1);
          __syncthreads();
        }
      }
      u32x4_t nf[NP];
#pragma unroll
      for (int k = 0; k < kT; ++k) {
        if (kA || k == 0) {
#pragma unroll
          for (int j = 0; j < NP; ++j) nf[j] = narrow_frag(kA ? p * kT + k : p, j);
        }
        if constexpr (!kA) {
#pragma unroll
          for (int g = 0; g < 2; ++g) wf[g] = wide_frag(k, g);
        }
#pragma unroll
        for (int j = 0; j < NP; ++j)
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            if (kF16 && !kA && k > 0)
              low[p][kF16 ? j : 0][g] = mfma16<kF16>(nf[j], wf[g],
                                                     low[p][kF16 ? j : 0][g]);
            else
              acc[p][j][g] = mfma16<kF16>(nf[j], wf[g], acc[p][j][g]);
          }
      }
    }
  }
  if constexpr (kA && kF16) {
    if (nit > 0) fold(nit - 1);
  }
  // acc[p][j][g][e]: column q0 + 32 w + 16 g + lane % 16, p0 + 16 j + 4 (lane / 16) + e
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float* out = (kA ? a.part_a[p] : a.part_b[p]) + (int64_t)blockIdx.y * Q * a.r;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int64_t q = q0 + 32 * wave + 16 * g + (lane & 15);
      if (q >= Q) continue;
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const int pc = p0 + 16 * j + 4 * (lane >> 4);
        if (pc >= a.r) continue;
        f32x4_t v = acc[p][j][g];
        if constexpr (kF16 && !kA) v += low[p][j][g] * (1.0f / term_up(true));
        if constexpr (kF16 && kA) v = low[p][j][g];
        if constexpr (kA) {
#pragma unroll
          for (int e = 0; e < 4; ++e) out[(int64_t)(pc + e) * Q + q] = v[e];
        } else {
          *reinterpret_cast<f32x4_t*>(out + q * a.r + pc) = v;
        }
      }
    }
  }
#endif
}

// The first workgroups dB's columns, the others dA's.
template <int NP, bool kF16, int kAct>
__global__ __launch_bounds__(256, kF16 ? 2 : 3) void gated_grads_kernel(GatedGrads a, int64_t chunk) {
  constexpr int kT = kTerms(kF16);
  constexpr int kB = kT * 32 * 128 + 2 * 32 * 16 * NP, kA = 32 * 128 + 2 * kT * 32 * 16 * NP;
  __shared__ __attribute__((aligned(1024))) uint16_t lds[kA > kB ? kA : kB];
  const int nb = (int)((a.rows + 127) / 128);
  if ((int)blockIdx.x < nb)
    grads_run<NP, kF16, kAct, false>(a, chunk, (int)blockIdx.x, lds);
  else
    grads_run<NP, kF16, kAct, true>(a, chunk, (int)blockIdx.x - nb, lds);
}

// columns of U a workgroup takes: all up to 64, else in two halves
static int grad_np(int32_t r) { return r <= 64 ? r >> 4 : ((r >> 4) + 1) / 2; }

int gated_grad_splits(int64_t T, int64_t rows, int64_t cols, int32_t r) {
  const int64_t wg = ((rows + 127) / 128 + (cols + 127) / 128) * (r > 64 ? 2 : 1);
  int64_t s = (768 + wg - 1) / wg;
  const int64_t most = (T + 127) / 128;
  if (s > most) s = most;
  if (s > 16) s = 16;
  return (int)(s < 1 ? 1 : s);
}

hipError_t launch_gated_grads(const GatedGrads& a, hipStream_t stream) {
  const int64_t chunk = chunk_of(a.T, a.splits, 32);
  const int np = grad_np(a.r);
  const dim3 grid((unsigned)((a.rows + 127) / 128 + (a.cols + 127) / 128), (unsigned)a.splits,
                  (unsigned)((a.r / 16 + np - 1) / np));
  switch (np) {
#define QLORA_GATED_LAUNCH(NP, F16, ACT)                                                          \
  hipLaunchKernelGGL((gated_grads_kernel<NP, F16, ACT>), grid, dim3(256), 0, stream, a, chunk)
#define QLORA_GATED_CASE(NP)                                                                      \
  case NP:                                                                                        \
    if (a.act_fn == QLORA_ACT_SILU) {                                                             \
      if (a.f16) QLORA_GATED_LAUNCH(NP, true, QLORA_ACT_SILU);                                    \
      else QLORA_GATED_LAUNCH(NP, false, QLORA_ACT_SILU);                                         \
    } else {                                                                                      \
      if (a.f16) QLORA_GATED_LAUNCH(NP, true, QLORA_ACT_GELU_TANH);                               \
      else QLORA_GATED_LAUNCH(NP, false, QLORA_ACT_GELU_TANH);                                    \
    }                                                                                             \
    break;
    QLORA_GATED_CASE(1) QLORA_GATED_CASE(2) QLORA_GATED_CASE(3) QLORA_GATED_CASE(4)
#undef QLORA_GATED_CASE
#undef QLORA_GATED_LAUNCH
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

// out = scale times the sum of the parts in their order, four values a thread;
// blockIdx.y: which gradient.
__global__ __launch_bounds__(256) void gated_sum_kernel(GatedSum a) {
  const int k = blockIdx.y;
  const int64_t n = a.n[k];
  const float* part = a.part[k];
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < n;
       i += (int64_t)gridDim.x * 1024) {
    f32x4_t v = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int s = 0; s < a.splits; ++s) v += *reinterpret_cast<const f32x4_t*>(part + s * n + i);
    *reinterpret_cast<f32x4_t*>(a.out[k] + i) = v * a.scale;
  }
}

hipError_t launch_gated_sum(const GatedSum& a, hipStream_t stream) {
  int64_t most = 0;
  for (int k = 0; k < 4; ++k) most = a.n[k] > most ? a.n[k] : most;
  int64_t blocks = (most / 4 + 255) / 256;
  if (blocks > 2048) blocks = 2048;
  hipLaunchKernelGGL(gated_sum_kernel, dim3((unsigned)blocks, 4), dim3(256), 0, stream, a);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Few tokens: the sums of the streaming kernel's partials, the LoRA products
// and the activation.  A workgroup takes 64 outputs of 4 TW tokens (from t0 on),
// wave w tokens w, w + 4, ..., a lane one output.  s U stays in float32 here: the
// products with B are the vector unit's.
// ---------------------------------------------------------------------------
template <int TW, bool kF16>
__global__ __launch_bounds__(256) void gated_finish_kernel(GatedFinish a) {
  __shared__ __attribute__((aligned(16))) float us[2][4 * TW * 128];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int r = a.r;
  const int t0 = (int)blockIdx.y * 4 * TW;
  const int here = (int)a.T - t0 < 4 * TW ? (int)a.T - t0 : 4 * TW;
  const int TR = here * r;
  const int64_t n = (int64_t)blockIdx.x * 64 + lane;
  const int64_t nc = n < a.rows ? n : a.rows - 1;
  // the first partials of P are on their way before U's are waited for
  constexpr int kBatch = TW == 1 ? 8 : 4;
  auto load = [&](int s0, float (&x)[2][kBatch][TW]) {
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
#pragma unroll
        for (int k = 0; k < TW; ++k) {
          const int64_t t = t0 + (wave + 4 * k < here ? wave + 4 * k : here - 1);
          const int s = s0 + i < a.splits ? s0 + i : a.splits - 1;
          x[p][i][k] = a.P[p][(s * a.T + t) * a.rows + nc];
        }
  };
  float v[2][TW], x0[2][kBatch][TW];
  load(0, x0);
  for (int i = tid; i < 2 * TR; i += 256) {
    const int p = i >= TR;
    const int e = i - p * TR;
    const float* src = a.PU[p] + (int64_t)t0 * r + e;
    const int64_t plane = a.T * r;
    float u = 0.0f;
    for (int s0 = 0; s0 < a.splits; s0 += 4) {
      float x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        x[j] = src[(s0 + j < a.splits ? s0 + j : a.splits - 1) * plane];
#pragma unroll
      for (int j = 0; j < 4; ++j) u += s0 + j < a.splits ? x[j] : 0.0f;
    }
    us[p][e] = u * a.scale;
    if (blockIdx.x == 0 && a.U_save[p])
      a.U_save[p][(int64_t)t0 * r + e] = (uint16_t)(pack16x2<kF16>(u, 0.0f) & 0xFFFFu);
  }
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int k = 0; k < TW; ++k) v[p][k] = 0.0f;
  for (int s0 = 0; s0 < a.splits; s0 += kBatch) {
    if (s0 > 0) load(s0, x0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i)
#pragma unroll
      for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int k = 0; k < TW; ++k) v[p][k] += s0 + i < a.splits ? x0[p][i][k] : 0.0f;
  }
  __syncthreads();
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float l[TW];
#pragma unroll
    for (int k = 0; k < TW; ++k) l[k] = 0.0f;
    for (int c = 0; c < r; c += 8) {
      const u32x4_t b = *reinterpret_cast<const u32x4_t*>(a.B[p] + nc * r + c);
#pragma unroll
      for (int k = 0; k < TW; ++k) {
        const float* u = &us[p][(wave + 4 * k) * r + c];   // stale past `here`, never stored
#pragma unroll
        for (int e = 0; e < 8; ++e) l[k] += u[e] * elem16<kF16>(b, e);
      }
    }
#pragma unroll
    for (int k = 0; k < TW; ++k) v[p][k] += l[k];
  }
  if (n >= a.rows) return;
#pragma unroll
  for (int k = 0; k < TW; ++k) {
    if (wave + 4 * k < here) {
      const int64_t o = (int64_t)(t0 + wave + 4 * k) * a.rows + n;
      const uint32_t gu = pack16x2<kF16>(v[0][k], v[1][k]);
      if (a.P_save[0]) {
        a.P_save[0][o] = (uint16_t)(gu & 0xFFFFu);
        a.P_save[1][o] = (uint16_t)(gu >> 16);
      }
      a.H[o] = (uint16_t)(pack16x2<kF16>(act_value(v[0][k], a.act_fn) * v[1][k], 0.0f) & 0xFFFFu);
    }
  }
}

hipError_t launch_gated_finish(const GatedFinish& a, hipStream_t stream) {
  const int64_t tokens = a.T <= 4 ? 4 : 16;
  const dim3 grid((unsigned)((a.rows + 63) / 64), (unsigned)((a.T + tokens - 1) / tokens));
#define QLORA_GATED_CASE(TW)                                                                \
  if (a.f16)                                                                                \
    hipLaunchKernelGGL((gated_finish_kernel<TW, true>), grid, dim3(256), 0, stream, a);     \
  else                                                                                      \
    hipLaunchKernelGGL((gated_finish_kernel<TW, false>), grid, dim3(256), 0, stream, a);
  if (a.T <= 4) {
    QLORA_GATED_CASE(1)
  } else {
    QLORA_GATED_CASE(4)
  }
#undef QLORA_GATED_CASE
  return hipGetLastError();
}

}  // namespace qlora
