// C ABI of the expert-grouped NF4 linear layer: validate on the host, then
// enqueue the grouped kernels (gemm.hip, gemv.hip, lora.hip) on the caller's
// stream.
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <string.h>

#include "abi_internal.h"
#include "grouped_kernels.h"
#include "qlora_experts.h"

namespace qlora {

GroupedWs grouped_ws_layout(int64_t T, int32_t experts, const WeightDims& d, int32_t r, bool bwd) {
  GroupedWs L;
  memset(&L, 0, sizeof(L));
  // Few rows an expert on average: stream the weights of the experts that have
  // any, in tiles of 16 or 32 rows; more: the tiled GEMM.  Few experts or small
  // weights leave the GEMM with too few tiles for the chip, so there the border
  // lies higher.  Streamed against tiled, us, ragged counts:
  //   17 rows   64 x 1024 x 2048 45 : 44   16 x 4096^2 66 : 89   1 x 4096^2 17 : 43
  //   24 rows   64 x 1024 x 2048 50 : 44   16 x 4096^2 75 : 87   8 x 4096 x 11008 120 : 118
  //   32 rows   64 x 1024 x 2048 61 : 45   16 x 4096^2 94 : 86   8 x 11008 x 4096 114 : 129
  //   48 rows   8 x 4096^2 74 : 65   4 x 4096^2 48 : 54   8 x 1024 x 2048 22 : 41
  //   64 rows   4 x 11008 x 4096 110 : 80   4 x 4096^2 53 : 53   32 x 1024^2 37 : 33
  // Tiles of 16 against 32 rows: 10 rows 64 x 1024 x 2048 41 : 43, 8 x 4096 x 11008
  // 86 : 98, 16 x 4096^2 59 : 62; 16 rows 50 : 45, 93 : 103, 81 : 66.
  const int64_t mean = (T + experts - 1) / experts;
  const bool small = d.rows * d.cols <= kGroupSmallWeights / experts;
  if (!bwd && mean <= (small ? 64 : (experts <= 8 ? 32 : 24))) L.skinny = mean <= 10 ? 16 : 32;
  // Few rows an expert, or few tiles in all: 128 x 128 tiles, two workgroups a CU;
  // less of a tile is empty, more workgroups share the chip, and one's start and
  // end (about 10 us of a tile) pass under the other's steps.  Otherwise 256 x 256,
  // which decode each weight half as often.  The best border depends on how
  // uneven the counts are, which the host does not know: this one is on average
  // 3, 2 and 1% behind the better of the two for even, uneven (deviation of the
  // log 0.5) and very uneven (1.0) counts over 13 shapes of 2 .. 64 experts and 72
  // .. 320 rows each.  128-row against 256-row tiles, us, forward and backward:
  //   72 rows, even   16 x 4096 x 2048 51 : 53, 70 : 76   64 x 512 x 2048 45 : 52, 53 : 59
  //   160 rows, uneven   32 x 2048 x 2048 71% and 75%   even   121% and 119%
  //   192 rows, even   4 x 4096^2 62 : 79, 68 : 87   8 x 11008 x 4096 236 : 193, 234 : 204
  //   320 rows   2 x 4096^2 83% and 84%   16 x 4096^2 112% and 110%
  const int64_t out = bwd ? d.cols : d.rows;
  const bool few_tiles = experts * ((mean + 255) / 256) * ((out + 255) / 256) <= 96;
  L.mi = mean <= 160 || few_tiles ? 2 : 4;
  const int64_t tiles = group_tile_bound(T, experts, 128);
  // twice the dense split count: with ragged tiles about two workgroups a CU
  // (8192 rows of 11008 columns, r = 64: 63 against 77 us; four times: 59, but
  // 3 us more in the sum of the partials)
  L.s_proj = 2 * lora_proj_splits(tiles * 128, bwd ? d.rows : d.cols, r);
  size_t off = 0;
  if (L.skinny) {
    const int64_t slots = group_tile_bound(T, experts, L.skinny);
    // 64 weight rows a workgroup; split the reduction by 2, 4 or 8 while that
    // makes at most 1200 workgroups and leaves each one round of its four
    // waves (8 blocks; 2 rows of 8 experts of 11008 x 4096: 25.5 us with 2
    // splits, 29.4 with one, 27.0 with 8)
    const int64_t wg = slots * ((d.rows + 63) / 64);
    L.s_gemv = 1;
    while (L.s_gemv < 8 && 2 * L.s_gemv * wg <= 1200 && 16 * L.s_gemv <= d.cols / 64) L.s_gemv *= 2;
    L.gemv_off = off;
    off += align_up(sizeof(float) * (size_t)L.s_gemv * (size_t)T * (size_t)d.rows, kWsAlign);
    L.gemv_u_off = off;
    off += align_up(sizeof(float) * (size_t)L.s_gemv * (size_t)T * (size_t)r, kWsAlign);
  } else {
    L.proj_off = off;
    off += align_up(sizeof(float) * (size_t)L.s_proj * (size_t)T * (size_t)r, kWsAlign);
    L.terms_off = off;
    off += align_up(2 * (size_t)(bwd ? grad_terms(d.f16) : kSeedTerms) * (size_t)T * (size_t)r,
                    kWsAlign);
    L.part_off = off;
    off += kGroupPartBytes;
    L.cnt_off = off;
    off += align_up(sizeof(uint32_t) * kGroupCounters, kWsAlign);
  }
  if (bwd) {
    if (d.f16) {
      const size_t slots = sizeof(float) * (size_t)term_slots(T, experts);
      L.largest_off = off;
      off += align_up((size_t)L.s_proj * slots, kWsAlign);
      L.down_off = off;
      off += align_up(slots, kWsAlign);
    }
    const int64_t wg = ((d.cols + 127) / 128 + (d.rows + 127) / 128) * experts * ((r + 63) / 64);
    int64_t s = (512 + wg - 1) / wg;
    if (s > (mean + 255) / 256) s = (mean + 255) / 256;
    L.s_grad = (int)(s > 16 ? 16 : (s < 1 ? 1 : s));
    if (L.s_grad > 1) {
      const size_t one = sizeof(float) * (size_t)L.s_grad * (size_t)experts * (size_t)r;
      L.grad_a_off = off;
      off += align_up(one * (size_t)d.cols, kWsAlign);
      L.grad_b_off = off;
      off += align_up(one * (size_t)d.rows, kWsAlign);
    }
  }
  L.total = off;
  return L;
}

namespace {

qlora_status hip_status(hipError_t e) {
  if (e == hipSuccess) return QLORA_OK;
  set_last_hip_error((int)e);
  return QLORA_ERR_HIP;
}

template <typename P>
P* at(void* ws, size_t off) {
  return reinterpret_cast<P*>(static_cast<char*>(ws) + off);
}

// Rows of one expert; false unless the stack's rows divide evenly into
// experts of a shape the linear kernels take.
bool expert_dims(int64_t rows_all, int32_t experts, int64_t* rows) {
  if (experts < 1 || experts > kMaxExperts || rows_all % experts != 0) return false;
  *rows = rows_all / experts;
  return *rows % 16 == 0;
}

bool rank_ok(int32_t r) { return r >= 16 && r <= QLORA_MAX_RANK && r % 16 == 0; }

// dA's operand, up to 3 planes of [T, r] 16-bit numbers, is addressed with
// 32-bit byte offsets; and every expert may take a partial tile of each 128
// outputs, 1024 x 2^20 / 128 workgroups of 256 threads: grids below 2^32
bool grouped_dims_ok(int64_t T, int64_t rows, int64_t cols, int32_t r) {
  return linear_dims_ok(T, rows, cols) && rank_ok(r) && T * r < (int64_t(1) << 28) &&
         rows <= (int64_t(1) << 20) && cols <= (int64_t(1) << 20);
}

qlora_status check_grouped(const qlora_nf4_weight* w, int32_t experts, int64_t T, int32_t r,
                           float alpha, WeightDims* d) {
  const qlora_status s = check_descriptor(w, d);
  if (s != QLORA_OK) return s;
  if (d->qt != QLORA_QUANT_NF4) return QLORA_ERR_FORMAT;
  int64_t rows;
  if (!expert_dims(d->rows, experts, &rows)) return QLORA_ERR_SHAPE;
  d->rows = rows;
  if (!grouped_dims_ok(T, rows, d->cols, r) || !isfinite(alpha)) return QLORA_ERR_SHAPE;
  return QLORA_OK;
}

void set_weight(GemmArgs& g, const qlora_nf4_weight* w, const WeightDims& d, void* ws,
                const GroupedWs& L) {
  g.codes = w->codes;
  g.code8 = w->absmax_code;
  g.s2 = w->absmax_scale;
  g.mu = w->absmax_offset;
  g.rows = d.rows;
  g.cols = d.cols;
  g.keep = nullptr;
  g.dq = d.dq;
  g.f16 = d.f16;
  g.wdq = nullptr;
  g.split_from = 0;
  g.part = at<float>(ws, L.part_off);
  g.cnt = at<uint32_t>(ws, L.cnt_off);
}

hipError_t enqueue_fwd(const qlora_nf4_weight* w, const WeightDims& d, const GroupArgs& ga,
                       const uint16_t* X, const uint16_t* A, const uint16_t* B, int32_t r,
                       float scale, uint16_t* Y, uint16_t* U_save, void* ws, const GroupedWs& L,
                       hipStream_t st) {
  if (L.skinny) {
    GemvArgs g;
    g.X = X;
    g.codes = w->codes;
    g.code8 = w->absmax_code;
    g.s2 = w->absmax_scale;
    g.mu = w->absmax_offset;
    g.rows = d.rows;
    g.cols = d.cols;
    g.T = ga.T;
    g.A = A;
    g.B = B;
    g.r = r;
    g.scale = scale;
    g.Y = Y;
    g.U_save = U_save;
    g.P = at<float>(ws, L.gemv_off);
    g.PU = at<float>(ws, L.gemv_u_off);
    g.splits = L.s_gemv;
    g.dq = d.dq;
    g.f16 = d.f16;
    return launch_grouped_gemv(g, ga, L.skinny, st);
  }
  float* P = at<float>(ws, L.proj_off);
  uint16_t* Ut = at<uint16_t>(ws, L.terms_off);
  hipError_t e = launch_grouped_proj(X, A, false, ga, d.cols, r, L.s_proj, P, TermScale{}, d.f16, st);
  if (e == hipSuccess)
    e = launch_grouped_reduce(GroupedReduce{P, r, L.s_proj, scale, U_save, Ut, kSeedTerms, d.f16,
                                            at<uint32_t>(ws, L.cnt_off), TermScale{}},
                              ga, st);
  if (e == hipSuccess) {
    GemmArgs g;
    set_weight(g, w, d, ws, L);
    g.act = X;
    g.lora_l = Ut;
    g.lora_r = B;
    g.r = r;
    g.out = Y;
    g.T = ga.T;
    e = launch_grouped_gemm(g, ga, GroupSeed{}, false, L.mi, st);
  }
  return e;
}

hipError_t enqueue_bwd(const qlora_nf4_weight* w, const WeightDims& d, const GroupArgs& ga,
                       const uint16_t* X, const uint16_t* dY, const uint16_t* A,
                       const uint16_t* B, int32_t r, float scale, const uint16_t* U, uint16_t* dX,
                       float* dA, float* dB, void* ws, const GroupedWs& L, hipStream_t st) {
  float* P = at<float>(ws, L.proj_off);
  uint16_t* Gt = at<uint16_t>(ws, L.terms_off);
  const int terms = grad_terms(d.f16);
  TermScale ts{};
  if (d.f16)
    ts = TermScale{at<float>(ws, L.largest_off), at<float>(ws, L.down_off),
                   term_slots(ga.T, ga.experts)};
  hipError_t e = launch_grouped_proj(dY, B, true, ga, d.rows, r, L.s_proj, P, ts, d.f16, st);
  if (e == hipSuccess)
    e = launch_grouped_reduce(GroupedReduce{P, r, L.s_proj, 1.0f, nullptr, Gt, terms, d.f16,
                                            at<uint32_t>(ws, L.cnt_off), ts},
                              ga, st);
  if (e == hipSuccess) {
    GemmArgs g;
    set_weight(g, w, d, ws, L);
    g.act = dY;
    g.lora_l = Gt;
    g.lora_r = A;
    g.r = r;
    g.out = dX;
    g.T = ga.T;
    e = launch_grouped_gemm(g, ga, GroupSeed{scale, ts.down}, true, L.mi, st);
  }
  if (e == hipSuccess) {
    GroupedGrads gg;
    gg.G = Gt;
    gg.n_terms = terms;
    gg.X = X;
    gg.U = U;
    gg.dY = dY;
    gg.rows = d.rows;
    gg.cols = d.cols;
    gg.r = r;
    gg.scale = scale;
    gg.dA = dA;
    gg.dB = dB;
    gg.Pa = L.s_grad > 1 ? at<float>(ws, L.grad_a_off) : nullptr;
    gg.Pb = L.s_grad > 1 ? at<float>(ws, L.grad_b_off) : nullptr;
    gg.splits = L.s_grad;
    gg.down = ts.down;
    gg.f16 = d.f16;
    e = launch_grouped_grads(gg, ga, st);
  }
  return e;
}

}  // namespace

}  // namespace qlora

extern "C" {

size_t qlora_grouped_linear_workspace(int64_t T, int32_t experts, int64_t rows, int64_t cols,
                                      int32_t r, int compute_dtype, int is_bwd) {
  using namespace qlora;
  WeightDims d;
  if (experts < 1 || experts > kMaxExperts || check_weight_shape(rows, cols, &d) != QLORA_OK)
    return 0;
  if (compute_dtype != QLORA_COMPUTE_BF16 && compute_dtype != QLORA_COMPUTE_FP16) return 0;
  if (!grouped_dims_ok(T, rows, cols, r) || T == 0) return 0;
  d.f16 = compute_dtype == QLORA_COMPUTE_FP16;
  return grouped_ws_layout(T, experts, d, r, is_bwd != 0).total;
}

qlora_status qlora_grouped_linear_fwd(const qlora_nf4_weight* w, int32_t experts,
                                      const uint16_t* X, int64_t T, const int32_t* offsets,
                                      const uint16_t* A, const uint16_t* B, int32_t r,
                                      float alpha, uint16_t* Y, uint16_t* U_save, void* ws,
                                      size_t ws_bytes, void* stream) {
  using namespace qlora;
  WeightDims d;
  qlora_status s = check_grouped(w, experts, T, r, alpha, &d);
  if (s != QLORA_OK) return s;
  if (!A || !B || !offsets) return QLORA_ERR_NULL;
  if (!aligned16(A) || !aligned16(B) || !aligned16(offsets)) return QLORA_ERR_ALIGN;
  if (T == 0) return check_device();
  if (!X || !Y || !ws) return QLORA_ERR_NULL;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(ws) || !aligned16(U_save))
    return QLORA_ERR_ALIGN;
  const GroupedWs L = grouped_ws_layout(T, experts, d, r, false);
  if (ws_bytes < L.total) return QLORA_ERR_WORKSPACE;
  s = check_device();
  if (s != QLORA_OK) return s;
  const GroupArgs ga{offsets, experts, T};
  return hip_status(enqueue_fwd(w, d, ga, X, A, B, r, alpha / (float)r, Y, U_save, ws, L,
                                static_cast<hipStream_t>(stream)));
}

qlora_status qlora_grouped_linear_bwd(const qlora_nf4_weight* w, int32_t experts,
                                      const uint16_t* X, const uint16_t* dY, int64_t T,
                                      const int32_t* offsets, const uint16_t* A,
                                      const uint16_t* B, int32_t r, float alpha,
                                      const uint16_t* U_saved, uint16_t* dX, float* dA, float* dB,
                                      void* ws, size_t ws_bytes, void* stream) {
  using namespace qlora;
  WeightDims d;
  qlora_status s = check_grouped(w, experts, T, r, alpha, &d);
  if (s != QLORA_OK) return s;
  if (!A || !B || !offsets || !dA || !dB) return QLORA_ERR_NULL;
  if (!aligned16(A) || !aligned16(B) || !aligned16(offsets) || !aligned16(dA) || !aligned16(dB))
    return QLORA_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (T == 0) {   // sums over no rows
    s = check_device();
    if (s != QLORA_OK) return s;
    hipError_t e = launch_zero_f32(dA, (int64_t)experts * r * d.cols, st);
    if (e == hipSuccess) e = launch_zero_f32(dB, (int64_t)experts * d.rows * r, st);
    return hip_status(e);
  }
  if (!X || !dY || !U_saved || !dX || !ws) return QLORA_ERR_NULL;
  if (!aligned16(X) || !aligned16(dY) || !aligned16(U_saved) || !aligned16(dX) || !aligned16(ws))
    return QLORA_ERR_ALIGN;
  const GroupedWs L = grouped_ws_layout(T, experts, d, r, true);
  if (ws_bytes < L.total) return QLORA_ERR_WORKSPACE;
  s = check_device();
  if (s != QLORA_OK) return s;
  const GroupArgs ga{offsets, experts, T};
  return hip_status(enqueue_bwd(w, d, ga, X, dY, A, B, r, alpha / (float)r, U_saved, dX, dA, dB,
                                ws, L, st));
}

}  // extern "C"
