// C ABI of the gated feed-forward block over NF4 weights: validate on the
// host, then enqueue the kernels (gated.hip, gemm.hip, gemv.hip, lora.hip) on
// the caller's stream.
#include <hip/hip_runtime_api.h>
#include <string.h>

#include "abi_internal.h"
#include "gated_kernels.h"
#include "qlora_gated.h"

namespace qlora {
namespace {

// Estimated time (microseconds) of the GEMM that decodes its weights in LDS, in
// tiles of 64 mi: rounds of its steps and its start and end, and the sums of split
// tiles.  Fitted to both directions of 44 sizes from 65 x 1024 x 2048 to 4096 x
// 11008 x 4096 (tokens, rows, columns), it picks on average 0.2% behind the better
// of the two, at worst 7.7%.  256-row against 128-row tiles, us: 65 tokens of 11008
// x 4096 forward 80 : 56, 512 116 : 143, 768 backward 219 : 282; 1024 tokens of
// 2736 x 1024 forward 51 : 36.
double decode_time(int64_t T, const WeightDims& d, bool bwd, int mi) {
  const GroupSplit sp = gated_split(T, d.rows, d.cols, bwd, mi);
  const int64_t steps = bwd ? 2 * ((d.rows + 63) / 64) : d.cols / 64;
  const double step = mi == 2 ? 0.959 : 1.204, ends = mi == 2 ? 35.7 : 60.6;
  double c = (double)(sp.full / group_slots(mi)) * ((double)steps * step + ends);
  if (sp.units > sp.full) {
    c += (double)((steps + sp.parts - 1) / sp.parts) * step + ends;
    if (sp.parts > 1) c += (mi == 2 ? 2.51 : 2.03) * sp.parts;
  }
  return c;
}

// Most tokens of the streaming forward.  Streaming against tiles, us: 64 tokens of
// 22016 x 8192 168 : 145, 4096 x 4096 46 : 41, 2736 x 1024 20 : 23; 48 tokens 144 :
// 145, 42 : 41, 11008 x 4096 48 : 54.
int64_t gated_gemv_tokens(const WeightDims& d) {
  return d.n <= (int64_t(1) << 23) ? kGemvMaxTokens : 48;
}

}  // namespace

GatedWs gated_ws_layout(int64_t T, const WeightDims& d, int32_t r, bool bwd) {
  GatedWs L;
  memset(&L, 0, sizeof(L));
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align_up(bytes, kWsAlign);
    return at;
  };
  const size_t t = (size_t)T, rows = (size_t)d.rows, cols = (size_t)d.cols, rr = (size_t)r;
  if (!bwd && T <= gated_gemv_tokens(d)) {
    // 64 weight rows a workgroup; split the reduction by 2, 4 or 8 while that
    // makes at most 1200 workgroups, leaves each one round of its four waves (8
    // blocks) and the partials few (11008 x 4096, one token: 23.2 us with 2
    // splits, 24.6 with 3, 26.9 with one; 4096 x 4096: 15.4 with 8, 26.1 with
    // one; 16 tokens 24.1 with 4, 26.8 with 8)
    const int64_t wg = 2 * ((d.rows + 63) / 64);
    L.s_gemv = 1;
    while (L.s_gemv < 8 && 2 * L.s_gemv * wg <= 1200 && 16 * L.s_gemv <= d.cols / 64 &&
           2 * L.s_gemv * T <= 64)
      L.s_gemv *= 2;
    for (int i = 0; i < 2; ++i) {
      L.gemv_off[i] = take(sizeof(float) * (size_t)L.s_gemv * t * rows);
      L.gemv_u_off[i] = take(sizeof(float) * (size_t)L.s_gemv * t * rr);
    }
    L.total = off;
    return L;
  }
  L.s_proj = bwd ? gated_bwd_splits(T, d.rows) : lora_proj_splits(T, d.cols, r);
  // forward: tiles of 128 outputs of both projections; backward: one
  // reduction over the rows of both
  const int64_t out_len = bwd ? d.cols : 2 * d.rows;
  const int64_t red_len = bwd ? 2 * ((d.rows + 63) / 64 * 64) : d.cols;
  const int64_t tiles = ((T + kGemmTileTokens - 1) / kGemmTileTokens) *
                        ((out_len + kGemmTileOut - 1) / kGemmTileOut);
  // (with few tiles the once-dequantised kernel, whose tiles are 256 x 256 and
  // split at most in two, leaves most CUs idle: 2560 tokens of 2736 x 1024, 40
  // tiles, backward 155 us against 101; 4096 x 4096, 160 tiles, 264 against 279)
  L.pre_dq = T >= pre_dq_min_tokens() && pre_dq_fits(d) && tiles >= 160;
  for (int i = 0; i < 2; ++i) {
    L.proj_off[i] = take(sizeof(float) * (size_t)L.s_proj * t * rr);
    // in the backward bf16's three (fp16: two)
    L.terms_off[i] = take(2 * (size_t)(bwd ? grad_terms(false) : kSeedTerms) * t * rr);
    L.largest_off[i] = take(sizeof(float) * 4 * (size_t)L.s_proj * (size_t)gated_slots(T));
    L.down_off[i] = take(sizeof(float) * (size_t)gated_slots(T));
    if (L.pre_dq) L.wdq_off[i] = take(2 * (size_t)d.n);
  }
  if (bwd) {
    L.s_grad = gated_grad_splits(T, d.rows, d.cols, r);
    for (int i = 0; i < 2; ++i) {
      L.at_off[i] = take(2 * cols * rr);
      L.d_off[i] = take(2 * t * rows);
      L.grad_a_off[i] = take(sizeof(float) * (size_t)L.s_grad * rr * cols);
      L.grad_b_off[i] = take(sizeof(float) * (size_t)L.s_grad * rr * rows);
    }
  }
  size_t tile_floats = 65536;
  int parts = 2;
  if (L.pre_dq) {
    L.mi = 4;
    L.gemm_split = gemm_split_from(T, out_len, red_len);
    L.n_split = (int)tiles - L.gemm_split;
  } else {
    L.mi = decode_time(T, d, bwd, 2) <= decode_time(T, d, bwd, 4) ? 2 : 4;
    const GroupSplit sp = gated_split(T, d.rows, d.cols, bwd, L.mi);
    parts = sp.parts;
    L.n_split = parts > 1 ? (sp.units - sp.full) / parts : 0;
    tile_floats = (size_t)(64 * L.mi) * (size_t)(64 * L.mi);
  }
  if (L.n_split > 0) {
    L.split_part_off = take(sizeof(float) * (size_t)L.n_split * (size_t)parts * tile_floats);
    L.split_cnt_off = take(sizeof(uint32_t) * (size_t)L.n_split);
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

// [T, r] 16-bit planes are addressed with 32-bit byte offsets
bool gated_rank_ok(int64_t T, int32_t r) { return T * r < (int64_t(1) << 28); }

struct Gated {
  const qlora_nf4_weight* w[2];
  const uint16_t* A[2];
  const uint16_t* B[2];
  WeightDims d;
  int64_t T;
  int32_t r;
  float scale;
  int act;
};

qlora_status check_gated(const Gated& in, float alpha, WeightDims* d) {
  WeightDims up;
  qlora_status s = check_linear_args(in.w[0], in.T, in.r, alpha, d);
  if (s != QLORA_OK) return s;
  s = check_linear_args(in.w[1], in.T, in.r, alpha, &up);
  if (s != QLORA_OK) return s;
  if (up.rows != d->rows || up.cols != d->cols) return QLORA_ERR_SHAPE;
  if (!gated_rank_ok(in.T, in.r)) return QLORA_ERR_SHAPE;
  if (up.dq != d->dq || up.f16 != d->f16) return QLORA_ERR_FORMAT;
  if (in.act != QLORA_ACT_SILU && in.act != QLORA_ACT_GELU_TANH) return QLORA_ERR_FORMAT;
  for (int i = 0; i < 2; ++i) {
    if (!in.A[i] || !in.B[i]) return QLORA_ERR_NULL;
    if (!aligned16(in.A[i]) || !aligned16(in.B[i])) return QLORA_ERR_ALIGN;
  }
  return QLORA_OK;
}

TermScale term_scale_at(const Gated& c, int i, void* ws, const GatedWs& L) {
  return c.d.f16 ? TermScale{at<float>(ws, L.largest_off[i]), at<float>(ws, L.down_off[i]),
                             gated_slots(c.T)}
                 : TermScale{};
}

void set_reduce(GatedReduce& a, const Gated& c, int i, void* ws, const GatedWs& L) {
  a.terms[i] = at<uint16_t>(ws, L.terms_off[i]);
  a.ts[i] = term_scale_at(c, i, ws, L);
  ProjReduce& p = a.part[i];
  p.P = at<float>(ws, L.proj_off[i]);
  p.T = c.T;
  p.r = c.r;
  p.splits = L.s_proj;
  p.f16 = c.d.f16;
  if (i == 0 && L.n_split > 0) {
    p.zero_cnt = at<uint32_t>(ws, L.split_cnt_off);
    p.n_zero = L.n_split;
  }
  if (L.pre_dq) {
    p.dq_codes = c.w[i]->codes;
    p.dq_code8 = c.w[i]->absmax_code;
    p.dq_s2 = c.w[i]->absmax_scale;
    p.dq_mu = c.w[i]->absmax_offset;
    p.dq_words = c.d.n / 8;
    p.dq_dq = c.d.dq;
    p.dq_out = at<uint16_t>(ws, L.wdq_off[i]);
  }
}

void set_gemm(GemmArgs& g, GateArgs& u, const Gated& c, void* ws, const GatedWs& L) {
  g.codes = c.w[0]->codes;
  g.code8 = c.w[0]->absmax_code;
  g.s2 = c.w[0]->absmax_scale;
  g.mu = c.w[0]->absmax_offset;
  g.rows = c.d.rows;
  g.cols = c.d.cols;
  g.lora_l = at<uint16_t>(ws, L.terms_off[0]);
  g.r = c.r;
  g.T = c.T;
  g.keep = nullptr;
  g.dq = c.d.dq;
  g.f16 = c.d.f16;
  g.wdq = L.pre_dq ? at<uint16_t>(ws, L.wdq_off[0]) : nullptr;
  g.split_from = L.gemm_split;
  const bool split = L.n_split > 0;
  g.part = split ? at<float>(ws, L.split_part_off) : nullptr;
  g.cnt = split ? at<uint32_t>(ws, L.split_cnt_off) : nullptr;
  u.codes = c.w[1]->codes;
  u.code8 = c.w[1]->absmax_code;
  u.s2 = c.w[1]->absmax_scale;
  u.mu = c.w[1]->absmax_offset;
  u.wdq = L.pre_dq ? at<uint16_t>(ws, L.wdq_off[1]) : nullptr;
  u.act = nullptr;
  u.lora_l = at<uint16_t>(ws, L.terms_off[1]);
  u.p_gate = u.p_up = nullptr;
  u.act_fn = c.act;
  u.scale = c.scale;
  for (int i = 0; i < 2; ++i) u.down[i] = term_scale_at(c, i, ws, L).down;
}

hipError_t enqueue_fwd(const Gated& c, const uint16_t* X, uint16_t* H, uint16_t* const (&P)[2],
                       uint16_t* const (&U)[2], void* ws, const GatedWs& L, hipStream_t st) {
  if (L.s_gemv > 0) {
    GemvArgs g[2];
    GatedFinish f;
    for (int i = 0; i < 2; ++i) {
      g[i].X = X;
      g[i].codes = c.w[i]->codes;
      g[i].code8 = c.w[i]->absmax_code;
      g[i].s2 = c.w[i]->absmax_scale;
      g[i].mu = c.w[i]->absmax_offset;
      g[i].rows = c.d.rows;
      g[i].cols = c.d.cols;
      g[i].T = c.T;
      g[i].A = c.A[i];
      g[i].B = c.B[i];
      g[i].r = c.r;
      g[i].scale = c.scale;
      g[i].Y = nullptr;
      g[i].U_save = nullptr;
      g[i].P = at<float>(ws, L.gemv_off[i]);
      g[i].PU = at<float>(ws, L.gemv_u_off[i]);
      g[i].splits = L.s_gemv;
      g[i].dq = c.d.dq;
      g[i].f16 = c.d.f16;
      f.P[i] = g[i].P;
      f.PU[i] = g[i].PU;
      f.B[i] = c.B[i];
      f.U_save[i] = U[i];
      f.P_save[i] = P[i];
    }
    f.H = H;
    f.T = c.T;
    f.rows = c.d.rows;
    f.r = c.r;
    f.splits = L.s_gemv;
    f.scale = c.scale;
    f.act_fn = c.act;
    f.f16 = c.d.f16;
    const hipError_t e = launch_gated_gemv_partial(g[0], g[1], st);
    return e == hipSuccess ? launch_gated_finish(f, st) : e;
  }
  float* const part[2] = {at<float>(ws, L.proj_off[0]), at<float>(ws, L.proj_off[1])};
  const TermScale ts[2] = {term_scale_at(c, 0, ws, L), term_scale_at(c, 1, ws, L)};
  hipError_t e = launch_gated_proj(X, c.A, c.T, c.d.cols, c.r, L.s_proj, part, ts, c.d.f16, st);
  if (e == hipSuccess) {
    GatedReduce a{};
    a.n_terms = kSeedTerms;
    for (int i = 0; i < 2; ++i) {
      set_reduce(a, c, i, ws, L);
      a.part[i].out_rm = U[i];
    }
    e = launch_gated_reduce(a, st);
  }
  if (e == hipSuccess) {
    GemmArgs g;
    GateArgs u;
    set_gemm(g, u, c, ws, L);
    g.act = X;
    g.lora_r = c.B[0];
    u.lora_r = c.B[1];
    g.out = H;
    u.p_gate = P[0];
    u.p_up = P[1];
    e = launch_gated_fwd_gemm(g, u, L.mi, st);
  }
  return e;
}

hipError_t enqueue_bwd(const Gated& c, const uint16_t* X, const uint16_t* dH,
                       const uint16_t* const (&P)[2], const uint16_t* const (&U)[2], uint16_t* dX,
                       float* const (&dA)[2], float* const (&dB)[2], void* ws, const GatedWs& L,
                       hipStream_t st) {
  GatedBwd b;
  b.dH = dH;
  b.Pg = P[0];
  b.Pu = P[1];
  for (int i = 0; i < 2; ++i) {
    b.B[i] = c.B[i];
    b.d[i] = at<uint16_t>(ws, L.d_off[i]);
    b.P[i] = at<float>(ws, L.proj_off[i]);
    b.ts[i] = term_scale_at(c, i, ws, L);
  }
  b.T = c.T;
  b.rows = c.d.rows;
  b.r = c.r;
  b.splits = L.s_proj;
  b.act_fn = c.act;
  b.f16 = c.d.f16;
  hipError_t e = launch_gated_bwd(b, st);
  if (e == hipSuccess) {
    GatedReduce a{};
    a.n_terms = grad_terms(c.d.f16);
    a.common = true;
    for (int i = 0; i < 2; ++i) {
      set_reduce(a, c, i, ws, L);
      a.tj[i].n = 1;
      a.tj[i].job[0] = TransposeJob{c.A[i], c.r, c.d.cols, at<uint16_t>(ws, L.at_off[i]), c.r};
    }
    e = launch_gated_reduce(a, st);
  }
  if (e == hipSuccess) {
    GemmArgs g;
    GateArgs u;
    set_gemm(g, u, c, ws, L);
    g.act = b.d[0];
    u.act = b.d[1];
    g.lora_r = at<uint16_t>(ws, L.at_off[0]);
    u.lora_r = at<uint16_t>(ws, L.at_off[1]);
    g.out = dX;
    e = launch_gated_dx_gemm(g, u, L.mi, st);
  }
  GatedSum s{};
  if (e == hipSuccess) {
    GatedGrads gg;
    gg.dH = dH;
    gg.Pg = P[0];
    gg.Pu = P[1];
    gg.X = X;
    for (int i = 0; i < 2; ++i) {
      gg.U[i] = U[i];
      gg.terms[i] = at<uint16_t>(ws, L.terms_off[i]);
      gg.down[i] = term_scale_at(c, i, ws, L).down;
      gg.part_a[i] = at<float>(ws, L.grad_a_off[i]);
      gg.part_b[i] = at<float>(ws, L.grad_b_off[i]);
      s.part[i] = gg.part_a[i];
      s.out[i] = dA[i];
      s.n[i] = c.d.cols * c.r;
      s.part[2 + i] = gg.part_b[i];
      s.out[2 + i] = dB[i];
      s.n[2 + i] = c.d.rows * c.r;
    }
    gg.T = c.T;
    gg.rows = c.d.rows;
    gg.cols = c.d.cols;
    gg.r = c.r;
    gg.splits = L.s_grad;
    gg.act_fn = c.act;
    gg.f16 = c.d.f16;
    e = launch_gated_grads(gg, st);
  }
  s.splits = L.s_grad;
  s.scale = c.scale;
  return e == hipSuccess ? launch_gated_sum(s, st) : e;
}

}  // namespace
}  // namespace qlora

extern "C" {

size_t qlora_gated_linear_workspace(int64_t T, int64_t rows, int64_t cols, int32_t r, int is_bwd) {
  using namespace qlora;
  WeightDims d;
  if (check_weight_shape(rows, cols, &d) != QLORA_OK || !linear_dims_ok(T, rows, cols)) return 0;
  if (r < 16 || r > QLORA_MAX_RANK || (r % 16) != 0 || T == 0 || !gated_rank_ok(T, r)) return 0;
  return gated_ws_layout(T, d, r, is_bwd != 0).total;
}

qlora_status qlora_gated_linear_fwd(const qlora_nf4_weight* gate, const qlora_nf4_weight* up,
                                    const uint16_t* X, int64_t T, const uint16_t* A_gate,
                                    const uint16_t* B_gate, const uint16_t* A_up,
                                    const uint16_t* B_up, int32_t r, float alpha, int act,
                                    uint16_t* H, uint16_t* P_gate, uint16_t* P_up,
                                    uint16_t* U_gate, uint16_t* U_up, void* ws, size_t ws_bytes,
                                    void* stream) {
  using namespace qlora;
  Gated c{{gate, up}, {A_gate, A_up}, {B_gate, B_up}, {}, T, r, alpha / (float)r, act};
  qlora_status s = check_gated(c, alpha, &c.d);
  if (s != QLORA_OK) return s;
  if (T == 0) return check_device();
  const bool save = P_gate || P_up || U_gate || U_up;
  if (!X || !H || !ws || (save && (!P_gate || !P_up || !U_gate || !U_up))) return QLORA_ERR_NULL;
  if (!aligned16(X) || !aligned16(H) || !aligned16(ws) || !aligned16(P_gate) ||
      !aligned16(P_up) || !aligned16(U_gate) || !aligned16(U_up))
    return QLORA_ERR_ALIGN;
  const GatedWs L = gated_ws_layout(T, c.d, r, false);
  if (ws_bytes < L.total) return QLORA_ERR_WORKSPACE;
  s = check_device();
  if (s != QLORA_OK) return s;
  return hip_status(enqueue_fwd(c, X, H, {P_gate, P_up}, {U_gate, U_up}, ws, L,
                                static_cast<hipStream_t>(stream)));
}

qlora_status qlora_gated_linear_bwd(const qlora_nf4_weight* gate, const qlora_nf4_weight* up,
                                    const uint16_t* X, const uint16_t* dH, int64_t T,
                                    const uint16_t* A_gate, const uint16_t* B_gate,
                                    const uint16_t* A_up, const uint16_t* B_up, int32_t r,
                                    float alpha, int act, const uint16_t* P_gate,
                                    const uint16_t* P_up, const uint16_t* U_gate,
                                    const uint16_t* U_up, uint16_t* dX, float* dA_gate,
                                    float* dB_gate, float* dA_up, float* dB_up, void* ws,
                                    size_t ws_bytes, void* stream) {
  using namespace qlora;
  Gated c{{gate, up}, {A_gate, A_up}, {B_gate, B_up}, {}, T, r, alpha / (float)r, act};
  qlora_status s = check_gated(c, alpha, &c.d);
  if (s != QLORA_OK) return s;
  float* const grads[4] = {dA_gate, dA_up, dB_gate, dB_up};
  for (float* p : grads) {
    if (!p) return QLORA_ERR_NULL;
    if (!aligned16(p)) return QLORA_ERR_ALIGN;
  }
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (T == 0) {   // sums over no tokens
    s = check_device();
    if (s != QLORA_OK) return s;
    hipError_t e = hipSuccess;
    for (int i = 0; i < 4 && e == hipSuccess; ++i)
      e = launch_zero_f32(grads[i], (int64_t)r * (i < 2 ? c.d.cols : c.d.rows), st);
    return hip_status(e);
  }
  const void* const need[8] = {X, dH, P_gate, P_up, U_gate, U_up, dX, ws};
  for (const void* p : need)
    if (!p) return QLORA_ERR_NULL;
  for (const void* p : need)
    if (!aligned16(p)) return QLORA_ERR_ALIGN;
  const GatedWs L = gated_ws_layout(T, c.d, r, true);
  if (ws_bytes < L.total) return QLORA_ERR_WORKSPACE;
  s = check_device();
  if (s != QLORA_OK) return s;
  return hip_status(enqueue_bwd(c, X, dH, {P_gate, P_up}, {U_gate, U_up}, dX, {dA_gate, dA_up},
                                {dB_gate, dB_up}, ws, L, st));
}

}  // extern "C"
