// C ABI of the layers of experts and of the 8-bit products (forge.h): host-side validation and the sequence
// of launches. Nothing here allocates or synchronises.
#include "forge_check.h"
#include "forge_ops.h"

using namespace forge;

namespace {

// routes of a plan, tokens of a call: below these (places are 32-bit; a grid holds fewer than 2^32 threads)
constexpr int64_t kMaxRoutes = (int64_t)1 << 30, kMaxTokens = (int64_t)1 << 26;
// k of an 8-bit product: sums of 2^17 - 16 products of at most 2^14 stay below 2^31
constexpr int64_t kMaxQ8 = (int64_t)1 << 17;

int check_experts(int experts, const int64_t* offsets) {
  if (experts < 1 || experts > FORGE_MAX_EXPERTS) return FORGE_ERR_SHAPE;
  if (!offsets) return FORGE_ERR_NULL;
  return ((uintptr_t)offsets & 7u) ? FORGE_ERR_ALIGN : FORGE_OK;
}

// A stack's rows per expert span less than 2^31 bytes; the whole may span more.
int check_part(const forge_tensor* t, int experts) {
  if (t->rows % experts) return FORGE_ERR_SHAPE;
  return !t->data || t->rows / experts * t->ld * (int64_t)elem_size(t->dtype) < ((int64_t)1 << 31) ? FORGE_OK
                                                                                                  : FORGE_ERR_UNSUPPORTED;
}
// A stack of matrices [experts * rows, cols].
int check_stack(const forge_tensor* t, int dtype, int experts, int64_t rows, int64_t cols) {
  int r = check_io(t, dtype);
  if (r) return r;
  if (t->rows != rows * experts || t->cols != cols) return FORGE_ERR_SHAPE;
  return check_part(t, experts);
}

// 8-bit rows with a factor each. `wide`: the factors are read four at a time.
int check_q8(const forge_tensor* t, int64_t rows, int64_t cols, bool wide) {
  if (!t) return FORGE_ERR_NULL;
  if (t->dtype != FORGE_I8) return FORGE_ERR_DTYPE;
  if (!t->data && t->rows != 0 && t->cols != 0) return FORGE_ERR_NULL;
  int r = check_shape(t);
  if (r) return r;
  if (t->rows != rows || t->cols != cols) return FORGE_ERR_SHAPE;
  if (!t->scale && rows > 0) return FORGE_ERR_NULL;
  if (!aligned16(t->data) || t->cols % 16 || t->ld % 16 || ((uintptr_t)t->scale & (wide ? 15u : 3u))) return FORGE_ERR_ALIGN;
  return FORGE_OK;
}
// without the factors, whose extent as 8-bit rows is another than that of moments
forge_tensor codes_of(const forge_tensor* t) {
  forge_tensor c = *t;
  c.scale = nullptr;
  return c;
}

void set_group(LinArgs& g, int experts, const int64_t* offsets) {
  g.experts = experts;
  g.offsets = offsets;
}

// The product's sums, in float32, as the result.
void set_sums(LinArgs& g, const forge_tensor* Y) {
  g.splits = 1;
  g.e.acc = (float*)Y->data;
  g.e.ldacc = Y->ld;
  g.e.acc_write = 1;
}

// (pairs of 8-bit integers stand where the kernels count bfloat16 elements)
void set_pair_q8(LinArgs& g, int s, const forge_tensor* A, const forge_tensor* B) {
  set_pair(g, s, A->data, A->ld / 2, B->data, B->ld / 2, B->cols / 2);
}

// The forward products of 8-bit rows; Wu: the gated one's second stack or NULL; experts = 0: not grouped.
int linear_q8(const forge_tensor* X, const forge_tensor* W, const forge_tensor* Wu, int experts, const int64_t* offsets,
              const forge_tensor* bias, int act, const forge_tensor* R, forge_tensor* Y, hipStream_t st) {
  int r;
  if (!X || !W || !Y) return FORGE_ERR_NULL;
  if (!act_ok(act)) return FORGE_ERR_UNSUPPORTED;
  if (offsets && (r = check_experts(experts, offsets))) return r;
  const int64_t parts = offsets ? experts : 1, T = X->rows, in = W->cols;
  if ((r = check_q8(W, W->rows, in, true)) || (r = check_q8(X, T, in, false)) || (Wu && (r = check_q8(Wu, W->rows, in, true))))
    return r;
  if (W->rows % parts) return FORGE_ERR_SHAPE;
  const int64_t out = W->rows / parts;
  const bool wide = offsets && !Wu && Y->dtype == FORGE_F32;  // the sums as they are
  if ((r = wide ? check_wide(Y, T, out) : check_mat(Y, FORGE_BF16, T, out))) return r;
  if (wide && (act != FORGE_ACT_NONE || out % 8)) return FORGE_ERR_UNSUPPORTED;
  if (bias && (r = check_mat(bias, bias->dtype == FORGE_F32 ? FORGE_F32 : FORGE_BF16, 1, out))) return r;
  if (R && (r = check_mat(R, FORGE_BF16, T, out))) return r;
  if (in >= kMaxQ8 || !fits_31(X)) return FORGE_ERR_UNSUPPORTED;
  if ((r = check_part(W, (int)parts)) || (Wu && (r = check_part(Wu, (int)parts)))) return r;
  const forge_tensor x = codes_of(X), w = codes_of(W), wu = Wu ? codes_of(Wu) : forge_tensor{};
  const forge_tensor sx = flat(X->scale, T * 4), sw = flat(W->scale, W->rows * 4), su = flat(Wu ? Wu->scale : nullptr, W->rows * 4),
                     off = flat(offsets, (parts + 1) * 8);
  const forge_tensor* outs[1] = {Y};
  const forge_tensor* ins[9] = {&x, &w, Wu ? &wu : nullptr, &sx, &sw, &su, &off, bias, R};
  if ((r = check_alias(outs, 1, ins, 9))) return r;
  if (T == 0 || out == 0) return FORGE_OK;
  LinArgs g{};
  set_pair_q8(g, 0, W, X);
  if (Wu) set_pair_q8(g, 1, Wu, X);
  g.nsrc = 1;
  g.M = (int32_t)out;
  g.N = (int32_t)T;
  if (offsets) set_group(g, experts, offsets);
  g.e.sx = X->scale;
  g.e.sw = W->scale;
  if (wide) {
    set_sums(g, Y);
    return hip_status(launch_lin_q8(L_ACC, g, st));
  }
  g.e.act = act;
  g.e.out = Y->data;
  g.e.ldo = Y->ld;
  if (Wu) g.e.sw2 = Wu->scale;
  if (R) {
    g.e.in1 = R->data;
    g.e.ld1 = R->ld;
  }
  if (bias) {
    g.e.bias = bias->data;
    g.e.bias_f32 = bias->dtype == FORGE_F32;
  }
  return hip_status(launch_lin_q8(Wu ? L_GATED : L_LINEAR, g, st));
}

}  // namespace

extern "C" {

int64_t forge_expert_plan_workspace(int64_t T, int64_t k, int32_t experts) {
  if (T <= 0 || k <= 0 || T >= kMaxRoutes || k >= kMaxRoutes || T * k >= kMaxRoutes || experts < 1 || experts > FORGE_MAX_EXPERTS)
    return 0;
  int64_t per;
  const int64_t blocks = expert_plan_blocks(T * k, &per);
  return blocks > 1 ? up(blocks * experts * 4, 16) : 0;
}

int forge_expert_plan(const int64_t* idx, int64_t T, int64_t k, int32_t experts, int64_t* offsets, int32_t* pos,
                      void* workspace, int64_t workspace_bytes, forge_stream_t stream) {
  int r = check_experts(experts, offsets);
  if (r) return r;
  if (T < 0 || k < 1) return FORGE_ERR_SHAPE;
  if (T >= kMaxRoutes || k >= kMaxRoutes || T * k >= kMaxRoutes) return FORGE_ERR_UNSUPPORTED;
  const int64_t n = T * k;
  if (n > 0 && (!idx || !pos)) return FORGE_ERR_NULL;
  if (((uintptr_t)idx & 7u) || ((uintptr_t)pos & 3u)) return FORGE_ERR_ALIGN;
  const int64_t need = forge_expert_plan_workspace(T, k, experts);
  if ((r = check_workspace(workspace, workspace_bytes, need))) return r;
  const forge_tensor ti = flat(idx, n * 8), to = flat(offsets, (experts + 1) * 8), tp = flat(pos, n * 4), tw = flat(workspace, need);
  const forge_tensor* outs[3] = {&to, &tp, &tw};
  const forge_tensor* ins[1] = {&ti};
  if ((r = check_alias(outs, 3, ins, 1))) return r;
  return hip_status(launch_expert_plan(idx, n, experts, offsets, pos, (int*)workspace, (hipStream_t)stream));
}

int forge_expert_dispatch(const forge_tensor* X, const int32_t* pos, int64_t k, forge_tensor* Xp, forge_stream_t stream) {
  int r;
  if (!X || !Xp) return FORGE_ERR_NULL;
  if (is_fp8(X->dtype)) return FORGE_ERR_UNSUPPORTED;
  const bool q8 = X->dtype == FORGE_I8;
  if (q8) {
    if ((r = check_q8(X, X->rows, X->cols, false)) || (r = check_q8(Xp, Xp->rows, X->cols, false))) return r;
    if (!fits_31(X) || !fits_31(Xp)) return FORGE_ERR_UNSUPPORTED;
  } else {
    if ((r = op_dtype(X))) return r;
    if ((r = check_mat(X, X->dtype, X->rows, X->cols)) || (r = check_mat(Xp, X->dtype, Xp->rows, X->cols))) return r;
  }
  if (k < 1) return FORGE_ERR_SHAPE;
  if (X->rows >= kMaxTokens || k >= kMaxRoutes || X->rows * k >= kMaxRoutes) return FORGE_ERR_UNSUPPORTED;
  if (X->rows > 0 && !pos) return FORGE_ERR_NULL;
  if ((uintptr_t)pos & 3u) return FORGE_ERR_ALIGN;
  const forge_tensor x = codes_of(X), y = codes_of(Xp), tp = flat(pos, X->rows * k * 4),
                     sx = flat(q8 ? X->scale : nullptr, X->rows * 4), sy = flat(q8 ? Xp->scale : nullptr, Xp->rows * 4);
  const forge_tensor* outs[2] = {&y, &sy};
  const forge_tensor* ins[3] = {&x, &tp, &sx};
  if ((r = check_alias(outs, 2, ins, 3))) return r;
  if (X->rows == 0 || Xp->rows == 0 || (X->cols == 0 && !q8)) return FORGE_OK;
  const int es = elem_size(X->dtype);
  return hip_status(launch_expert_dispatch(X->data, X->ld * es, pos, (int)k, X->rows, Xp->rows, Xp->data, Xp->ld * es,
                                           (int)(X->cols * es / 16), q8 ? X->scale : nullptr, q8 ? Xp->scale : nullptr,
                                           (hipStream_t)stream));
}

// What both directions of the combination check and share. Y: the result, or its gradient.
static int check_combine(const forge_tensor* Yp, const int32_t* pos, int64_t k, const float* weights, const forge_tensor* Y,
                         CombineArgs& a) {
  int r;
  if ((r = op_dtype(Y)) || (r = check_mat(Y, Y->dtype, Y->rows, Y->cols))) return r;
  if (Yp) {
    if ((r = op_dtype(Yp))) return r;
    const bool wide = Yp->dtype == FORGE_F32 && Y->dtype == FORGE_BF16;
    if ((r = wide ? check_wide(Yp, Yp->rows, Y->cols) : check_mat(Yp, Y->dtype, Yp->rows, Y->cols))) return r;
  }
  if (k < 1) return FORGE_ERR_SHAPE;
  if (Y->rows >= kMaxTokens || k >= kMaxRoutes || Y->rows * k >= kMaxRoutes) return FORGE_ERR_UNSUPPORTED;
  if (Y->rows > 0 && !pos) return FORGE_ERR_NULL;
  if (((uintptr_t)pos & 3u) || ((uintptr_t)weights & 3u)) return FORGE_ERR_ALIGN;
  a.Yp = Yp ? Yp->data : nullptr;
  a.ldp = Yp ? Yp->ld : 0;
  a.places = Yp ? Yp->rows : 0;
  a.pos = pos;
  a.w = weights;
  a.k = (int)k;
  a.Y = Y->data;
  a.ldy = Y->ld;
  a.tokens = Y->rows;
  a.cols = (int)Y->cols;
  return FORGE_OK;
}

int forge_expert_combine(const forge_tensor* Yp, const int32_t* pos, int64_t k, const float* weights,
                         const forge_tensor* R, forge_tensor* Y, forge_stream_t stream) {
  if (!Yp || !Y) return FORGE_ERR_NULL;
  CombineArgs a{};
  int r = check_combine(Yp, pos, k, weights, Y, a);
  if (r) return r;
  if (R && (r = check_mat(R, Y->dtype, Y->rows, Y->cols))) return r;
  const forge_tensor tp = flat(pos, Y->rows * k * 4), tw = flat(weights, Y->rows * k * 4);
  const forge_tensor* outs[1] = {Y};
  const forge_tensor* ins[4] = {Yp, R, &tp, &tw};
  if ((r = check_alias(outs, 1, ins, 4))) return r;
  if (Y->rows == 0 || Y->cols == 0) return FORGE_OK;
  if (R) {
    a.R = R->data;
    a.ldr = R->ld;
  }
  return hip_status(launch_expert_combine(Y->dtype == FORGE_BF16, Yp->dtype == FORGE_F32, a, (hipStream_t)stream));
}

int forge_expert_combine_backward(const forge_tensor* dY, const forge_tensor* Yp, const int32_t* pos, int64_t k,
                                  const float* weights, forge_tensor* dYp, float* dweights, forge_stream_t stream) {
  if (!dY || (dweights && !Yp)) return FORGE_ERR_NULL;
  CombineArgs a{};
  int r = check_combine(Yp, pos, k, weights, dY, a);
  if (r) return r;
  if (dYp && (r = check_mat(dYp, dY->dtype, dYp->rows, dY->cols))) return r;
  if (dYp && Yp && dYp->rows != Yp->rows) return FORGE_ERR_SHAPE;
  if ((uintptr_t)dweights & 3u) return FORGE_ERR_ALIGN;
  const forge_tensor tp = flat(pos, dY->rows * k * 4), tw = flat(weights, dY->rows * k * 4), td = flat(dweights, dY->rows * k * 4);
  const forge_tensor* outs[2] = {dYp, &td};
  const forge_tensor* ins[4] = {dY, Yp, &tp, &tw};
  if ((r = check_alias(outs, 2, ins, 4))) return r;
  if (dY->rows == 0 || (!dYp && !dweights)) return FORGE_OK;
  if (dYp) {
    a.dYp = dYp->data;
    a.lddp = dYp->ld;
    a.places = dYp->rows;
  }
  a.dw = dweights;
  return hip_status(launch_expert_combine_backward(dY->dtype == FORGE_BF16, Yp && Yp->dtype == FORGE_F32, a, (hipStream_t)stream));
}

int forge_expert_linear(const forge_tensor* X, const forge_tensor* W, int32_t experts, const int64_t* offsets,
                        int32_t act, forge_tensor* Y, forge_tensor* Z, forge_stream_t stream) {
  int r;
  if (!X || !W || !Y) return FORGE_ERR_NULL;
  if ((r = op_dtype(W)) || (r = op_dtype(X)) || (r = check_experts(experts, offsets))) return r;
  if (!act_ok(act)) return FORGE_ERR_UNSUPPORTED;
  const int dt = W->dtype;
  const int64_t T = X->rows, out = W->rows / experts, in = W->cols;
  const bool wide = dt == FORGE_BF16 && Y->dtype == FORGE_F32;  // the sums as they are
  if ((r = check_mat(X, dt, T, in)) || (r = check_stack(W, dt, experts, out, in)) ||
      (r = wide ? check_wide(Y, T, out) : check_mat(Y, dt, T, out)))
    return r;
  if (wide && (act != FORGE_ACT_NONE || Z || out % 8)) return FORGE_ERR_UNSUPPORTED;
  if (Z && (r = check_mat(Z, dt, T, out))) return r;
  const forge_tensor off = flat(offsets, (experts + 1) * 8);
  const forge_tensor* outs[2] = {Y, Z};
  const forge_tensor* ins[3] = {X, W, &off};
  if ((r = check_alias(outs, 2, ins, 3))) return r;
  if (T == 0 || out == 0) return FORGE_OK;
  LinArgs g{};
  set_pair(g, 0, W->data, W->ld, X->data, X->ld, in);
  g.nsrc = 1;
  g.M = (int32_t)out;
  g.N = (int32_t)T;
  set_group(g, experts, offsets);
  if (wide) {
    set_sums(g, Y);
    return hip_status(launch_lin_expert(1, L_ACC, false, g, (hipStream_t)stream));
  }
  g.e.act = act;
  g.e.out = Y->data;
  g.e.ldo = Y->ld;
  if (Z) {
    g.e.out2 = Z->data;
    g.e.ldo2 = Z->ld;
  }
  return hip_status(launch_lin_expert(dt == FORGE_BF16, L_LINEAR, false, g, (hipStream_t)stream));
}

int forge_expert_gated(const forge_tensor* X, const forge_tensor* Wg, const forge_tensor* Wu, int32_t experts,
                       const int64_t* offsets, int32_t act, forge_tensor* H, forge_tensor* G, forge_tensor* U,
                       forge_stream_t stream) {
  int r;
  if (!X || !Wg || !Wu || !H || (!G) != (!U)) return FORGE_ERR_NULL;
  if ((r = op_dtype(Wg)) || (r = op_dtype(X)) || (r = check_experts(experts, offsets))) return r;
  if (!act_ok(act)) return FORGE_ERR_UNSUPPORTED;
  const int dt = Wg->dtype;
  const int64_t T = X->rows, hid = Wg->rows / experts, in = Wg->cols;
  if ((r = check_mat(X, dt, T, in)) || (r = check_stack(Wg, dt, experts, hid, in)) ||
      (r = check_stack(Wu, dt, experts, hid, in)) || (r = check_mat(H, dt, T, hid)))
    return r;
  if (G && ((r = check_mat(G, dt, T, hid)) || (r = check_mat(U, dt, T, hid)))) return r;
  const forge_tensor off = flat(offsets, (experts + 1) * 8);
  const forge_tensor* outs[3] = {H, G, U};
  const forge_tensor* ins[4] = {X, Wg, Wu, &off};
  if ((r = check_alias(outs, 3, ins, 4))) return r;
  if (T == 0 || hid == 0) return FORGE_OK;
  LinArgs g{};
  set_pair(g, 0, Wg->data, Wg->ld, X->data, X->ld, in);
  set_pair(g, 1, Wu->data, Wu->ld, X->data, X->ld, in);
  g.nsrc = 1;
  g.M = (int32_t)hid;
  g.N = (int32_t)T;
  set_group(g, experts, offsets);
  g.e.act = act;
  g.e.out = H->data;
  g.e.ldo = H->ld;
  if (G) {
    g.e.out2 = G->data;
    g.e.ldo2 = G->ld;
    g.e.out3 = U->data;
    g.e.ldo3 = U->ld;
  }
  return hip_status(launch_lin_expert(dt == FORGE_BF16, L_GATED, false, g, (hipStream_t)stream));
}

int forge_expert_gated_dgrad(const forge_tensor* dY, const forge_tensor* Wd, const forge_tensor* G,
                             const forge_tensor* U, int32_t experts, const int64_t* offsets, int32_t act,
                             forge_tensor* dG, forge_tensor* dU, forge_tensor* H, forge_stream_t stream) {
  int r;
  if (!dY || !Wd || !G || !U || !dG || !dU) return FORGE_ERR_NULL;
  if ((r = op_dtype(Wd)) || (r = op_dtype(dY)) || (r = check_experts(experts, offsets))) return r;
  if (!act_ok(act)) return FORGE_ERR_UNSUPPORTED;
  const int dt = Wd->dtype;
  const int64_t T = dY->rows, out = Wd->rows / experts, hid = Wd->cols;
  if ((r = check_mat(dY, dt, T, out)) || (r = check_stack(Wd, dt, experts, out, hid)) || (r = check_mat(G, dt, T, hid)) ||
      (r = check_mat(U, dt, T, hid)) || (r = check_mat(dG, dt, T, hid)) || (r = check_mat(dU, dt, T, hid)))
    return r;
  if (H && (r = check_mat(H, dt, T, hid))) return r;
  const forge_tensor off = flat(offsets, (experts + 1) * 8);
  const forge_tensor* outs[3] = {dG, dU, H};
  const forge_tensor* ins[5] = {G, U, dY, Wd, &off};
  if ((r = check_alias(outs, 3, ins, 5))) return r;
  if (T == 0 || hid == 0) return FORGE_OK;
  LinArgs g{};
  set_pair(g, 0, Wd->data, Wd->ld, dY->data, dY->ld, out);
  g.nsrc = 1;
  g.M = (int32_t)hid;
  g.N = (int32_t)T;
  set_group(g, experts, offsets);
  g.e.act = act;
  g.e.in1 = G->data;
  g.e.ld1 = G->ld;
  g.e.in2 = U->data;
  g.e.ld2 = U->ld;
  g.e.out = dG->data;
  g.e.ldo = dG->ld;
  g.e.out2 = dU->data;
  g.e.ldo2 = dU->ld;
  if (H) {
    g.e.out3 = H->data;
    g.e.ldo3 = H->ld;
  }
  return hip_status(launch_lin_expert(dt == FORGE_BF16, L_DGATE, true, g, (hipStream_t)stream));
}

int64_t forge_expert_dgrad_group_workspace(int64_t rows, int64_t in, int64_t sum_out, int32_t experts, int32_t dtype) {
  if (rows <= 0 || in <= 0 || sum_out <= 0 || rows >= kMaxDim || in >= kMaxDim || sum_out >= FORGE_MAX_GROUP * kMaxDim ||
      experts < 1 || experts > FORGE_MAX_EXPERTS)
    return 0;
  const int64_t s = lin_expert_splits(dtype == FORGE_BF16, in, rows, experts, sum_out);
  return s > 1 ? s * rows * in * 4 : 0;
}

static int expert_dgrad_group(int32_t n_layers, const forge_tensor* dY, const forge_tensor* W, int32_t experts,
                              const int64_t* offsets, forge_tensor* dX, bool split, void* workspace,
                              int64_t workspace_bytes, forge_stream_t stream) {
  int r;
  if (!dY || !W || !dX) return FORGE_ERR_NULL;
  if (n_layers < 1 || n_layers > FORGE_MAX_GROUP) return FORGE_ERR_SHAPE;
  if ((r = op_dtype(dX)) || (r = check_experts(experts, offsets))) return r;
  const int dt = dX->dtype;
  const int64_t T = dX->rows, in = dX->cols;
  int64_t rows = 0;
  LinArgs g{};
  const forge_tensor off = flat(offsets, (experts + 1) * 8);
  const forge_tensor* ins[2 * FORGE_MAX_GROUP + 1];
  for (int l = 0; l < n_layers; ++l) {
    if ((r = op_dtype(&dY[l])) || (r = op_dtype(&W[l]))) return r;
    const int64_t out = W[l].rows / experts;
    if ((r = check_mat(&dY[l], dt, T, out)) || (r = check_stack(&W[l], dt, experts, out, in))) return r;
    ins[2 * l] = &dY[l];
    ins[2 * l + 1] = &W[l];
    rows += out;
    if (out == 0) continue;  // a layer without rows adds nothing
    set_pair(g, g.nsrc++, W[l].data, W[l].ld, dY[l].data, dY[l].ld, out);
  }
  ins[2 * n_layers] = &off;
  if ((r = check_mat(dX, dt, T, in))) return r;
  const int64_t need = split ? forge_expert_dgrad_group_workspace(T, in, rows, experts, dt) : 0;
  if ((r = check_workspace(workspace, workspace_bytes, need))) return r;
  const forge_tensor ws = flat(workspace, need);
  const forge_tensor* outs[2] = {dX, &ws};
  if ((r = check_alias(outs, 2, ins, 2 * n_layers + 1))) return r;
  if (T == 0 || in == 0) return FORGE_OK;
  g.M = (int32_t)in;
  g.N = (int32_t)T;
  g.splits = need ? lin_expert_splits(dt == FORGE_BF16, in, T, experts, rows) : 1;
  set_group(g, experts, offsets);
  g.e.out = dX->data;
  g.e.ldo = dX->ld;
  if (g.splits > 1) {
    g.e.acc = (float*)workspace;
    g.e.ldacc = in;
    g.e.acc_write = 1;
  }
  r = hip_status(launch_lin_expert(dt == FORGE_BF16, L_ACC, true, g, (hipStream_t)stream));
  return r || g.splits <= 1 ? r : hip_status(launch_acc_join(g, (hipStream_t)stream));
}

int forge_expert_dgrad_group(int32_t n_layers, const forge_tensor* dY, const forge_tensor* W, int32_t experts,
                             const int64_t* offsets, forge_tensor* dX, forge_stream_t stream) {
  return expert_dgrad_group(n_layers, dY, W, experts, offsets, dX, false, nullptr, 0, stream);
}

int forge_expert_dgrad_group_split(int32_t n_layers, const forge_tensor* dY, const forge_tensor* W, int32_t experts,
                                   const int64_t* offsets, forge_tensor* dX, void* workspace, int64_t workspace_bytes,
                                   forge_stream_t stream) {
  return expert_dgrad_group(n_layers, dY, W, experts, offsets, dX, true, workspace, workspace_bytes, stream);
}

// Operands of the stack's weight gradient, for W [experts * out, in] of type dt.
static int check_wgrad(const forge_tensor* X, const forge_tensor* dY, int experts, const int64_t* offsets, int dt) {
  int r;
  if (!X || !dY) return FORGE_ERR_NULL;
  if (is_fp8(X->dtype) || is_fp8(dY->dtype)) return FORGE_ERR_UNSUPPORTED;
  if ((r = check_experts(experts, offsets))) return r;
  if ((r = check_mat(X, dt, X->rows, X->cols)) || (r = check_mat(dY, dt, X->rows, dY->cols))) return r;
  return FORGE_OK;
}

int forge_expert_wgrad(const forge_tensor* X, const forge_tensor* dY, int32_t experts, const int64_t* offsets,
                       float* dW, int64_t ld_dw, forge_stream_t stream) {
  int r = op_dtype(X);
  if (r) return r;
  if ((r = check_wgrad(X, dY, experts, offsets, X->dtype))) return r;
  const forge_tensor dWt{dW, FORGE_F32, 0, dY->cols * experts, X->cols, ld_dw, nullptr};
  if ((r = check_io(&dWt, FORGE_F32)) || (r = check_part(&dWt, experts))) return r;
  const forge_tensor off = flat(offsets, (experts + 1) * 8);
  const forge_tensor* outs[1] = {&dWt};
  const forge_tensor* ins[3] = {X, dY, &off};
  if ((r = check_alias(outs, 1, ins, 3))) return r;
  if (dY->cols == 0 || X->cols == 0) return FORGE_OK;
  const GemmDims d{(int32_t)X->rows, (int32_t)dY->cols, (int32_t)X->cols, X->ld, dY->ld};
  return hip_status(launch_wgrad_store_expert(X->dtype == FORGE_BF16, X->data, dY->data, d, offsets, experts, dW, ld_dw,
                                              (hipStream_t)stream));
}

int forge_expert_wgrad_step(const forge_tensor* X, const forge_tensor* dY, forge_tensor* W, forge_tensor* m,
                            forge_tensor* v, int32_t experts, const int64_t* offsets, int32_t opt,
                            const forge_hyper* hyper, int64_t step, uint64_t seed, forge_stream_t stream) {
  int r = op_dtype(W);
  if (r) return r;
  if ((r = check_hyper(opt, hyper, step))) return r;
  const int io = W->dtype;
  if ((r = check_wgrad(X, dY, experts, offsets, io)) || (r = check_stack(W, io, experts, dY->cols, X->cols))) return r;
  const int fmt = check_states(opt, io, W, m, v);
  if (fmt < 0) return fmt;
  const int sl = opt_slots(opt);
  if (W->rows * W->cols >= ((int64_t)1 << 32)) return FORGE_ERR_UNSUPPORTED;
  if (((sl & 1) && (r = check_part(m, experts))) || ((sl & 2) && (r = check_part(v, experts)))) return r;
  const forge_tensor off = flat(offsets, (experts + 1) * 8);
  const forge_tensor* outs[3] = {W, (sl & 1) ? m : nullptr, (sl & 2) ? v : nullptr};
  const forge_tensor* ins[3] = {X, dY, &off};
  if ((r = check_alias(outs, 3, ins, 3))) return r;
  forge_scalars sc;
  if ((r = forge_step_scalars(opt, hyper, step, &sc))) return r;
  if (W->rows == 0 || W->cols == 0) return FORGE_OK;
  const OptArgs a = make_args(W, m, v, opt, sc, seed, step);
  const GemmDims d{(int32_t)X->rows, (int32_t)dY->cols, (int32_t)X->cols, X->ld, dY->ld};
  const int sr = io == FORGE_BF16 && hyper->stochastic_round ? 1 : 0;
  return hip_status(launch_wgrad_fused_expert(io == FORGE_BF16, fmt, opt, sr, X->data, dY->data, d, offsets, experts, a,
                                              (hipStream_t)stream));
}

int forge_quantize_rows(const forge_tensor* X, forge_tensor* Q, forge_stream_t stream) {
  int r;
  if (!X || !Q) return FORGE_ERR_NULL;
  if ((r = op_dtype(X)) || (r = check_mat(X, X->dtype, X->rows, X->cols)) || (r = check_q8(Q, X->rows, X->cols, false))) return r;
  if (X->rows >= kMaxTokens) return FORGE_ERR_UNSUPPORTED;
  const forge_tensor q = codes_of(Q), s = flat(Q->scale, X->rows * 4);
  const forge_tensor* outs[2] = {&q, &s};
  const forge_tensor* ins[1] = {X};
  if ((r = check_alias(outs, 2, ins, 1))) return r;
  if (X->rows == 0) return FORGE_OK;
  return hip_status(launch_quantize_rows(X->dtype == FORGE_BF16, X->data, X->ld, (int8_t*)Q->data, Q->ld, Q->scale, X->rows,
                                         (int)X->cols, (hipStream_t)stream));
}

int forge_linear_q8(const forge_tensor* X, const forge_tensor* W, const forge_tensor* bias, int32_t act,
                    const forge_tensor* R, forge_tensor* Y, forge_stream_t stream) {
  return linear_q8(X, W, nullptr, 0, nullptr, bias, act, R, Y, (hipStream_t)stream);
}

int forge_gated_q8(const forge_tensor* X, const forge_tensor* Wg, const forge_tensor* Wu, int32_t act, forge_tensor* H,
                   forge_stream_t stream) {
  if (!Wu) return FORGE_ERR_NULL;
  return linear_q8(X, Wg, Wu, 0, nullptr, nullptr, act, nullptr, H, (hipStream_t)stream);
}

int forge_expert_linear_q8(const forge_tensor* X, const forge_tensor* W, int32_t experts, const int64_t* offsets,
                           int32_t act, forge_tensor* Y, forge_stream_t stream) {
  if (!offsets) return FORGE_ERR_NULL;
  return linear_q8(X, W, nullptr, experts, offsets, nullptr, act, nullptr, Y, (hipStream_t)stream);
}

int forge_expert_gated_q8(const forge_tensor* X, const forge_tensor* Wg, const forge_tensor* Wu, int32_t experts,
                          const int64_t* offsets, int32_t act, forge_tensor* H, forge_stream_t stream) {
  if (!Wu || !offsets) return FORGE_ERR_NULL;
  return linear_q8(X, Wg, Wu, experts, offsets, nullptr, act, nullptr, H, (hipStream_t)stream);
}

int32_t forge_expert_tile(int32_t product, int64_t rows, int64_t cols, int64_t k, int32_t experts, int32_t dtype) {
  if (rows < 1 || cols < 1 || k < 0 || rows >= kMaxDim || cols >= kMaxDim || k >= kMaxDim || experts < 1 || experts > FORGE_MAX_EXPERTS)
    return FORGE_ERR_SHAPE;
  if (dtype != FORGE_BF16 && dtype != FORGE_I8) return FORGE_ERR_DTYPE;
  const bool q8 = dtype == FORGE_I8;
  switch (product) {
    case FORGE_EXPERT_LINEAR:
      return q8 ? lin_q8_expert_edge(L_LINEAR, cols, rows, k, experts) : lin_expert_edge(L_LINEAR, false, cols, rows, k, experts);
    case FORGE_EXPERT_SUMS:
      return q8 ? lin_q8_expert_edge(L_ACC, cols, rows, k, experts) : lin_expert_edge(L_ACC, false, cols, rows, k, experts);
    case FORGE_EXPERT_GATED:
      return q8 ? lin_q8_expert_edge(L_GATED, cols, rows, k, experts) : lin_expert_edge(L_GATED, false, cols, rows, k, experts);
    case FORGE_EXPERT_GATED_DGRAD: return q8 ? FORGE_ERR_DTYPE : lin_expert_edge(L_DGATE, true, cols, rows, k, experts);
    case FORGE_EXPERT_DGRAD: return q8 ? FORGE_ERR_DTYPE : lin_expert_edge(L_ACC, true, cols, rows, k, experts);
    case FORGE_EXPERT_WGRAD:
      if (q8) return FORGE_ERR_DTYPE;
      return k * cols * 4 < ((int64_t)1 << 31) ? wgrad_expert_edge(k, cols, experts) : FORGE_ERR_UNSUPPORTED;
    default: return FORGE_ERR_UNSUPPORTED;
  }
}

}  // extern "C"
