// C ABI of the operators around the fused step (the second half of forge.h): host-side
// validation and the sequence of launches. Nothing here allocates or synchronises.
#include "forge_check.h"
#include "forge_ops.h"

using namespace forge;

namespace {

// Operand type of a call: every tensor given must have it.
int op_dtype(const forge_tensor* t) {
  if (!t) return FORGE_ERR_NULL;
  if (is_fp8(t->dtype)) return FORGE_ERR_UNSUPPORTED;
  return t->dtype == FORGE_F32 || t->dtype == FORGE_BF16 ? FORGE_OK : FORGE_ERR_DTYPE;
}

// A dense operand or result of the given size.
int check_mat(const forge_tensor* t, int dtype, int64_t rows, int64_t cols) {
  int r = check_io(t, dtype);
  if (r) return r;
  if (t->rows != rows || t->cols != cols) return FORGE_ERR_SHAPE;
  return fits_31(t) ? FORGE_OK : FORGE_ERR_UNSUPPORTED;
}

bool act_ok(int act) { return act >= FORGE_ACT_NONE && act <= FORGE_ACT_GELU_TANH; }

int hip_status(hipError_t e) { return e == hipSuccess ? FORGE_OK : FORGE_ERR_HIP; }

// Plain memory as a tensor, for the overlap checks.
forge_tensor flat(const void* p, int64_t bytes) {
  return forge_tensor{const_cast<void*>(p), FORGE_I8, 0, p && bytes > 0 ? 1 : 0, bytes, bytes, nullptr};
}

int check_workspace(const void* ws, int64_t have, int64_t need) {
  if (need == 0) return FORGE_OK;
  if (have < need) return FORGE_ERR_SCRATCH;
  if (!ws) return FORGE_ERR_NULL;
  return ((uintptr_t)ws & 15u) ? FORGE_ERR_ALIGN : FORGE_OK;
}

int64_t up(int64_t x, int64_t a) { return (x + a - 1) / a * a; }

// One pair of operands of a product.
void set_pair(LinArgs& g, int s, const void* A, int64_t lda, const void* B, int64_t ldb, int64_t K) {
  g.A[s] = A;
  g.lda[s] = lda;
  g.B[s] = B;
  g.ldb[s] = ldb;
  g.K[s] = (int32_t)K;
}

// ---- cross entropy: sizes ----
constexpr int64_t kPieceBytes = (int64_t)1 << 30;  // of dz, where the caller gives no size

// bytes between the rows of W or dW, below this (256 of its rows are addressed by 32-bit offsets)
constexpr int64_t kHeadPitch = (int64_t)1 << 23;

// Logits of a call, below this: the pairs of the vocabulary's blocks would fill the memory (2^42
// logits: 256 GB), and the kernels count their tiles in 32 bits.
constexpr int64_t kMaxLogits = (int64_t)1 << 42;

// W of the head: as check_io, but any number of bytes (tiles and pieces address it by 64-bit
// offsets) and any number of rows.
int check_head(const forge_tensor* X, const forge_tensor* W, const int64_t* target) {
  int r = op_dtype(W);
  if (r) return r;
  if (!X) return FORGE_ERR_NULL;
  if (is_fp8(X->dtype)) return FORGE_ERR_UNSUPPORTED;
  if ((r = check_io(W, W->dtype)) || (r = check_io(X, W->dtype))) return r;
  if (X->cols != W->cols || W->rows < 1) return FORGE_ERR_SHAPE;
  if (!fits_31(X) || W->ld * (int64_t)elem_size(W->dtype) >= kHeadPitch) return FORGE_ERR_UNSUPPORTED;
  if (X->rows * W->rows >= kMaxLogits) return FORGE_ERR_UNSUPPORTED;
  if (!target && X->rows > 0) return FORGE_ERR_NULL;
  return ((uintptr_t)target & 7u) ? FORGE_ERR_ALIGN : FORGE_OK;
}

// Vocabulary entries of a piece: at least 8, dz and the piece's rows of W below 2^31 bytes.
int64_t piece_of(int64_t T, int64_t ldw, int64_t vocab, int es, int64_t piece) {
  const int64_t most_rows = T > 0 ? (((int64_t)1 << 31) - 1) / (T * es) / 8 * 8 : vocab;
  const int64_t most_w = ldw > 0 ? (((int64_t)1 << 31) - 1) / (ldw * es) / 8 * 8 : vocab;
  int64_t p = piece;
  if (p <= 0) {
    // about kPieceBytes of dz each, pieces of even size, whole large tiles
    const int64_t want = T > 0 ? kPieceBytes / (T * es) : vocab;
    const int64_t n = want > 0 ? (vocab + want - 1) / want : vocab;
    p = up((vocab + n - 1) / n, 256);
  }
  if (p > most_rows) p = most_rows;
  if (p > most_w) p = most_w;
  const int64_t all = up(vocab, 8);
  if (p > all) p = all;
  return p < 8 ? 8 : p;
}

// Workspaces. Forward: the partial results, the targets' logits, the losses' partial sums.
struct FwdWs {
  int64_t part, tlogit, tsum, bytes;
};
FwdWs fwd_ws(int64_t T, int64_t vocab, int64_t block) {
  FwdWs w;
  w.part = 0;
  w.tlogit = up((vocab + block - 1) / block * T * 8, 16);
  w.tsum = w.tlogit + up(T * 4, 16);
  w.bytes = w.tsum + (int64_t)lse_join_groups(T) * 16;
  return w;
}
// Backward: a piece's dz (rows of up(piece, 8) entries), the sums of dX over the pieces, one set
// per part of the k range.
struct BwdWs {
  int64_t dz, acc, bytes;
  int splits;
};
BwdWs bwd_ws(int64_t T, int64_t in, int64_t piece, int es) {
  BwdWs w;
  w.dz = 0;
  w.acc = up(T * up(piece, 8) * es, 16);
  w.splits = T > 0 && in > 0 ? lin_splits(es == 2, in, T, piece) : 1;
  // room for them in any case: a W of wide pitch may take more, smaller pieces
  w.bytes = w.acc + w.splits * T * in * 4;
  return w;
}

// What the backward calls share. Wp: the piece's rows of W.
struct XentCall {
  const forge_tensor* X;
  const forge_tensor* W;
  const int64_t* target;
  int64_t ignore;
  const float* lse;
  const float* dloss;
  int per_token;
  const float* total;
  forge_tensor* dX;
  int64_t piece;
  char* ws;
  BwdWs w;
};

int check_xent_grad(const XentCall& c, int64_t piece, int64_t ws_bytes) {
  if (c.X->rows > 0 && (!c.lse || !c.dloss)) return FORGE_ERR_NULL;
  if (((uintptr_t)c.lse & 3u) || ((uintptr_t)c.dloss & 3u) || ((uintptr_t)c.total & 3u)) return FORGE_ERR_ALIGN;
  if (piece < 0 || piece % 8) return FORGE_ERR_SHAPE;
  if (c.dX) {
    int r = check_mat(c.dX, c.W->dtype, c.X->rows, c.X->cols);
    if (r) return r;
  }
  // the documented size (a W of wide pitch may take smaller pieces, which need less)
  const int64_t need = forge_linear_xent_workspace(c.X->rows, c.X->cols, c.W->rows, c.W->dtype, 1, piece);
  return check_workspace(c.ws, ws_bytes, need > c.w.bytes ? need : c.w.bytes);
}

// dz of vocabulary entries v0 .. v0 + n - 1 into the workspace. folded: the common factor
// too goes into dz before its rounding.
int enqueue_dz(const XentCall& c, int64_t v0, int64_t n, bool folded, hipStream_t st) {
  const int bf16 = c.W->dtype == FORGE_BF16, es = bf16 ? 2 : 4;
  LinArgs g{};
  set_pair(g, 0, (const char*)c.W->data + v0 * c.W->ld * es, c.W->ld, c.X->data, c.X->ld, c.X->cols);
  g.nsrc = 1;
  g.M = (int32_t)n;
  g.N = (int32_t)c.X->rows;
  g.e.out = c.ws + c.w.dz;
  g.e.ldo = up(c.piece, 8);
  g.e.target = c.target;
  g.e.ignore = c.ignore;
  g.e.v0 = v0;
  g.e.vocab = c.W->rows;
  g.e.lse = c.lse;
  if (c.per_token) g.e.weight = c.dloss;
  if (folded) {
    g.e.scale = c.per_token ? nullptr : c.dloss;
    g.e.count = c.total ? c.total + 1 : nullptr;
  }
  return hip_status(launch_lin(bf16, L_DLOGIT, false, false, g, st));
}

// dX (+)= dz W over the piece; scaled and rounded with the last piece
int enqueue_dx(const XentCall& c, int64_t v0, int64_t n, bool folded, hipStream_t st) {
  const int bf16 = c.W->dtype == FORGE_BF16, es = bf16 ? 2 : 4;
  LinArgs g{};
  set_pair(g, 0, (const char*)c.W->data + v0 * c.W->ld * es, c.W->ld, c.ws + c.w.dz, up(c.piece, 8), n);
  g.nsrc = 1;
  g.M = (int32_t)c.X->cols;
  g.N = (int32_t)c.X->rows;
  g.e.out = c.dX->data;
  g.e.ldo = c.dX->ld;
  g.e.acc = (float*)(c.ws + c.w.acc);
  g.e.ldacc = c.X->cols;
  const bool last = v0 + n >= c.W->rows;
  g.splits = c.w.splits;
  g.e.acc_read = v0 > 0;
  g.e.acc_write = g.splits > 1 || !last;
  if (!folded) {
    g.e.scale = c.per_token ? nullptr : c.dloss;
    g.e.count = c.total ? c.total + 1 : nullptr;
  }
  const int r = hip_status(launch_lin(bf16, L_ACC, true, false, g, st));
  return r || g.splits <= 1 || !last ? r : hip_status(launch_acc_join(g, st));
}

}  // namespace

extern "C" {

int forge_linear_forward(const forge_tensor* X, const forge_tensor* W, const forge_tensor* bias, int32_t act,
                         const forge_tensor* R, forge_tensor* Y, forge_tensor* Z, forge_stream_t stream) {
  int r;
  if (!X || !W || !Y) return FORGE_ERR_NULL;
  if ((r = op_dtype(W)) || (r = op_dtype(X))) return r;
  if (!act_ok(act)) return FORGE_ERR_UNSUPPORTED;
  const int dt = W->dtype;
  const int64_t T = X->rows, out = W->rows, in = W->cols;
  if ((r = check_mat(X, dt, T, in)) || (r = check_mat(W, dt, out, in)) || (r = check_mat(Y, dt, T, out))) return r;
  if (bias && (r = check_mat(bias, bias->dtype == FORGE_F32 ? FORGE_F32 : dt, 1, out))) return r;
  if (R && (r = check_mat(R, dt, T, out))) return r;
  if (Z && (r = check_mat(Z, dt, T, out))) return r;
  const forge_tensor* outs[2] = {Y, Z};
  const forge_tensor* ins[4] = {X, W, bias, R};
  if ((r = check_alias(outs, 2, ins, 4))) return r;
  if (T == 0 || out == 0) return FORGE_OK;
  LinArgs g{};
  set_pair(g, 0, W->data, W->ld, X->data, X->ld, in);
  g.nsrc = 1;
  g.M = (int32_t)out;
  g.N = (int32_t)T;
  g.e.act = act;
  g.e.out = Y->data;
  g.e.ldo = Y->ld;
  if (Z) {
    g.e.out2 = Z->data;
    g.e.ldo2 = Z->ld;
  }
  if (R) {
    g.e.in1 = R->data;
    g.e.ld1 = R->ld;
  }
  if (bias) {
    g.e.bias = bias->data;
    g.e.bias_f32 = bias->dtype == FORGE_F32;
  }
  return hip_status(launch_lin(dt == FORGE_BF16, L_LINEAR, false, false, g, (hipStream_t)stream));
}

int64_t forge_linear_act_backward_workspace(int64_t T, int64_t out) {
  if (T <= 0 || out <= 0 || T >= kMaxDim || out >= kMaxDim) return 0;
  const int64_t b = act_backward_blocks(T, out);
  return b > 1 ? up(b * out * 4, 16) : 0;
}

int forge_linear_act_backward(const forge_tensor* dY, const forge_tensor* Z, int32_t act, forge_tensor* dZ,
                              float* dbias, void* workspace, int64_t workspace_bytes, forge_stream_t stream) {
  int r = op_dtype(dY);
  if (r) return r;
  if (!act_ok(act)) return FORGE_ERR_UNSUPPORTED;
  const int dt = dY->dtype;
  const int64_t T = dY->rows, out = dY->cols;
  if ((r = check_mat(dY, dt, T, out))) return r;
  if (act != FORGE_ACT_NONE && (!Z || !dZ)) return FORGE_ERR_NULL;
  if (Z && (r = check_mat(Z, dt, T, out))) return r;
  if (dZ && (r = check_mat(dZ, dt, T, out))) return r;
  if ((uintptr_t)dbias & 15u) return FORGE_ERR_ALIGN;
  const int64_t need = dbias ? forge_linear_act_backward_workspace(T, out) : 0;
  if ((r = check_workspace(workspace, workspace_bytes, need))) return r;
  const forge_tensor db = flat(dbias, out * 4), ws = flat(workspace, need);
  const forge_tensor* outs[3] = {dZ, &db, &ws};
  const forge_tensor* ins[2] = {dY, Z};
  if ((r = check_alias(outs, 3, ins, 2))) return r;
  if (out == 0 || (!dZ && !dbias) || (T == 0 && !dbias)) return FORGE_OK;
  return hip_status(launch_act_backward(dt == FORGE_BF16, act, dY->data, dY->ld, Z ? Z->data : nullptr, Z ? Z->ld : 0,
                                        dZ ? dZ->data : nullptr, dZ ? dZ->ld : 0, dbias, (float*)workspace, (int)T,
                                        (int)out, (hipStream_t)stream));
}

int forge_gated_forward(const forge_tensor* X, const forge_tensor* Wg, const forge_tensor* Wu, int32_t act,
                        forge_tensor* H, forge_tensor* G, forge_tensor* U, forge_stream_t stream) {
  int r;
  if (!X || !Wg || !Wu || !H || (!G) != (!U)) return FORGE_ERR_NULL;
  if ((r = op_dtype(Wg)) || (r = op_dtype(X))) return r;
  if (!act_ok(act)) return FORGE_ERR_UNSUPPORTED;
  const int dt = Wg->dtype;
  const int64_t T = X->rows, hid = Wg->rows, in = Wg->cols;
  if ((r = check_mat(X, dt, T, in)) || (r = check_mat(Wg, dt, hid, in)) || (r = check_mat(Wu, dt, hid, in)) ||
      (r = check_mat(H, dt, T, hid)))
    return r;
  if (G && ((r = check_mat(G, dt, T, hid)) || (r = check_mat(U, dt, T, hid)))) return r;
  const forge_tensor* outs[3] = {H, G, U};
  const forge_tensor* ins[3] = {X, Wg, Wu};
  if ((r = check_alias(outs, 3, ins, 3))) return r;
  if (T == 0 || hid == 0) return FORGE_OK;
  LinArgs g{};
  set_pair(g, 0, Wg->data, Wg->ld, X->data, X->ld, in);
  set_pair(g, 1, Wu->data, Wu->ld, X->data, X->ld, in);
  g.nsrc = 1;
  g.M = (int32_t)hid;
  g.N = (int32_t)T;
  g.e.act = act;
  g.e.out = H->data;
  g.e.ldo = H->ld;
  if (G) {
    g.e.out2 = G->data;
    g.e.ldo2 = G->ld;
    g.e.out3 = U->data;
    g.e.ldo3 = U->ld;
  }
  return hip_status(launch_lin(dt == FORGE_BF16, L_GATED, false, false, g, (hipStream_t)stream));
}

// The gated backward's tensors (dG, dU, H, G, U) checked and set in e. extra: one more input.
static int gated_epi(const forge_tensor* G, const forge_tensor* U, int32_t act, forge_tensor* dG, forge_tensor* dU,
                     forge_tensor* H, int dt, int64_t T, int64_t hid, const forge_tensor* in_a,
                     const forge_tensor* in_b, LinEpiArgs& e) {
  int r;
  if (!G || !U || !dG || !dU) return FORGE_ERR_NULL;
  if (!act_ok(act)) return FORGE_ERR_UNSUPPORTED;
  if ((r = check_mat(G, dt, T, hid)) || (r = check_mat(U, dt, T, hid)) || (r = check_mat(dG, dt, T, hid)) ||
      (r = check_mat(dU, dt, T, hid)))
    return r;
  if (H && (r = check_mat(H, dt, T, hid))) return r;
  const forge_tensor* outs[3] = {dG, dU, H};
  const forge_tensor* ins[4] = {G, U, in_a, in_b};
  if ((r = check_alias(outs, 3, ins, 4))) return r;
  e.act = act;
  e.in1 = G->data;
  e.ld1 = G->ld;
  e.in2 = U->data;
  e.ld2 = U->ld;
  e.out = dG->data;
  e.ldo = dG->ld;
  e.out2 = dU->data;
  e.ldo2 = dU->ld;
  if (H) {
    e.out3 = H->data;
    e.ldo3 = H->ld;
  }
  return FORGE_OK;
}

int forge_gated_backward(const forge_tensor* dH, const forge_tensor* G, const forge_tensor* U, int32_t act,
                         forge_tensor* dG, forge_tensor* dU, forge_tensor* H, forge_stream_t stream) {
  int r = op_dtype(dH);
  if (r) return r;
  const int dt = dH->dtype;
  const int64_t T = dH->rows, hid = dH->cols;
  if ((r = check_mat(dH, dt, T, hid))) return r;
  LinEpiArgs e{};
  if ((r = gated_epi(G, U, act, dG, dU, H, dt, T, hid, dH, nullptr, e))) return r;
  if (T == 0 || hid == 0) return FORGE_OK;
  return hip_status(launch_gated_backward(dt == FORGE_BF16, dH->data, dH->ld, e, (int)T, (int)hid, (hipStream_t)stream));
}

int forge_gated_dgrad(const forge_tensor* dY, const forge_tensor* Wd, const forge_tensor* G, const forge_tensor* U,
                      int32_t act, forge_tensor* dG, forge_tensor* dU, forge_tensor* H, forge_stream_t stream) {
  int r;
  if (!dY || !Wd) return FORGE_ERR_NULL;
  if ((r = op_dtype(Wd)) || (r = op_dtype(dY))) return r;
  const int dt = Wd->dtype;
  const int64_t T = dY->rows, out = Wd->rows, hid = Wd->cols;
  if ((r = check_mat(dY, dt, T, out)) || (r = check_mat(Wd, dt, out, hid))) return r;
  LinArgs g{};
  if ((r = gated_epi(G, U, act, dG, dU, H, dt, T, hid, dY, Wd, g.e))) return r;
  if (T == 0 || hid == 0) return FORGE_OK;
  set_pair(g, 0, Wd->data, Wd->ld, dY->data, dY->ld, out);
  g.nsrc = 1;
  g.M = (int32_t)hid;
  g.N = (int32_t)T;
  return hip_status(launch_lin(dt == FORGE_BF16, L_DGATE, true, false, g, (hipStream_t)stream));
}

// The group's product; split: with the documented workspace.
static int dgrad_group(int32_t n_layers, const forge_tensor* dY, const forge_tensor* W, forge_tensor* dX, bool split,
                       void* workspace, int64_t workspace_bytes, hipStream_t st) {
  int r;
  if (!dY || !W || !dX) return FORGE_ERR_NULL;
  if (n_layers < 1 || n_layers > FORGE_MAX_GROUP) return FORGE_ERR_SHAPE;
  if ((r = op_dtype(dX))) return r;
  const int dt = dX->dtype;
  const int64_t T = dX->rows, in = dX->cols;
  LinArgs g{};
  const forge_tensor* ins[2 * FORGE_MAX_GROUP];
  int64_t rows = 0;
  for (int l = 0; l < n_layers; ++l) {
    if ((r = op_dtype(&dY[l])) || (r = op_dtype(&W[l]))) return r;
    if ((r = check_mat(&dY[l], dt, T, W[l].rows)) || (r = check_mat(&W[l], dt, W[l].rows, in))) return r;
    ins[2 * l] = &dY[l];
    ins[2 * l + 1] = &W[l];
    rows += W[l].rows;
    if (W[l].rows == 0) continue;  // a layer without rows adds nothing
    set_pair(g, g.nsrc++, W[l].data, W[l].ld, dY[l].data, dY[l].ld, W[l].rows);
  }
  if ((r = check_mat(dX, dt, T, in))) return r;
  const int64_t need = split ? forge_linear_dgrad_group_workspace(T, in, rows, dt) : 0;
  if ((r = check_workspace(workspace, workspace_bytes, need))) return r;
  const forge_tensor ws = flat(workspace, need);
  const forge_tensor* outs[2] = {dX, &ws};
  if ((r = check_alias(outs, 2, ins, 2 * n_layers))) return r;
  if (T == 0 || in == 0) return FORGE_OK;
  g.M = (int32_t)in;
  g.N = (int32_t)T;
  g.e.out = dX->data;
  g.e.ldo = dX->ld;
  g.splits = need ? lin_splits(dt == FORGE_BF16, in, T, rows) : 1;
  if (g.splits > 1) {
    g.e.acc = (float*)workspace;
    g.e.ldacc = in;
    g.e.acc_write = true;
  }
  r = hip_status(launch_lin(dt == FORGE_BF16, L_ACC, true, false, g, st));
  return r || g.splits <= 1 ? r : hip_status(launch_acc_join(g, st));
}

int forge_linear_dgrad_group(int32_t n_layers, const forge_tensor* dY, const forge_tensor* W, forge_tensor* dX,
                             forge_stream_t stream) {
  return dgrad_group(n_layers, dY, W, dX, false, nullptr, 0, (hipStream_t)stream);
}

int64_t forge_linear_dgrad_group_workspace(int64_t T, int64_t in, int64_t rows, int32_t dtype) {
  if (T <= 0 || in <= 0 || rows <= 0 || T >= kMaxDim || in >= kMaxDim || rows >= FORGE_MAX_GROUP * kMaxDim) return 0;
  const int64_t s = lin_splits(dtype == FORGE_BF16, in, T, rows);
  return s > 1 ? s * T * in * 4 : 0;
}

int forge_linear_dgrad_group_split(int32_t n_layers, const forge_tensor* dY, const forge_tensor* W, forge_tensor* dX,
                                   void* workspace, int64_t workspace_bytes, forge_stream_t stream) {
  return dgrad_group(n_layers, dY, W, dX, true, workspace, workspace_bytes, (hipStream_t)stream);
}

int64_t forge_linear_xent_workspace(int64_t T, int64_t in, int64_t vocab, int32_t dtype, int32_t backward,
                                    int64_t piece) {
  if (T < 0 || in < 0 || vocab < 1 || T >= kMaxDim || in >= kMaxDim || vocab >= kMaxDim || piece < 0) return 0;
  if (T * vocab >= kMaxLogits) return 0;
  const int es = dtype == FORGE_BF16 ? 2 : 4;
  if (!backward) return fwd_ws(T, vocab, lin_lse_block(dtype == FORGE_BF16, (int)vocab, (int)T)).bytes;
  const int64_t p = piece_of(T, in, vocab, es, piece);
  return bwd_ws(T, in, p, es).bytes;
}

int forge_linear_xent_forward(const forge_tensor* X, const forge_tensor* W, const int64_t* target, int64_t ignore,
                              float* loss, float* lse, float* total, void* workspace, int64_t workspace_bytes,
                              forge_stream_t stream) {
  int r = check_head(X, W, target);
  if (r) return r;
  const int bf16 = W->dtype == FORGE_BF16;
  const int64_t T = X->rows, V = W->rows;
  if (!total || (T > 0 && !lse)) return FORGE_ERR_NULL;
  if (((uintptr_t)loss & 3u) || ((uintptr_t)lse & 3u) || ((uintptr_t)total & 3u)) return FORGE_ERR_ALIGN;
  const int64_t block = lin_lse_block(bf16, (int)V, (int)T);
  const FwdWs w = fwd_ws(T, V, block);
  if ((r = check_workspace(workspace, workspace_bytes, w.bytes))) return r;
  const forge_tensor tt = flat(target, T * 8), lo = flat(loss, T * 4), ls = flat(lse, T * 4), to = flat(total, 12),
                     ws = flat(workspace, w.bytes);
  const forge_tensor* outs[4] = {&lo, &ls, &to, &ws};
  const forge_tensor* ins[3] = {X, W, &tt};
  if ((r = check_alias(outs, 4, ins, 3))) return r;
  char* base = (char*)workspace;
  float* part = (float*)(base + w.part);
  float* tl = (float*)(base + w.tlogit);
  if (T > 0) {
    LinArgs g{};
    set_pair(g, 0, W->data, W->ld, X->data, X->ld, X->cols);
    g.nsrc = 1;
    g.M = (int32_t)V;
    g.N = (int32_t)T;
    g.e.target = target;
    g.e.part = part;
    g.e.part_ld = T;
    g.e.tlogit = tl;
    if ((r = hip_status(launch_lin(bf16, L_LSE, false, false, g, (hipStream_t)stream)))) return r;
  }
  return hip_status(launch_lse_join(part, (V + block - 1) / block, tl, target, ignore, V, loss, lse, total,
                                    (double*)(base + w.tsum), (int)T, (hipStream_t)stream));
}

int forge_linear_xent_backward(const forge_tensor* X, const forge_tensor* W, const int64_t* target, int64_t ignore,
                               const float* lse, const float* dloss, int32_t per_token, const float* total,
                               forge_tensor* dX, forge_tensor* dW, int64_t piece, void* workspace,
                               int64_t workspace_bytes, forge_stream_t stream) {
  int r = check_head(X, W, target);
  if (r) return r;
  const int bf16 = W->dtype == FORGE_BF16, es = bf16 ? 2 : 4;
  const int64_t T = X->rows, V = W->rows, in = W->cols;
  XentCall c{X, W, target, ignore, lse, dloss, per_token != 0, total, dX, piece_of(T, W->ld, V, es, piece),
             (char*)workspace, BwdWs{}};
  c.w = bwd_ws(T, in, c.piece, es);
  if ((r = check_xent_grad(c, piece, workspace_bytes))) return r;
  if (dW) {
    if ((r = check_io(dW, W->dtype))) return r;
    if (dW->rows != V || dW->cols != in) return FORGE_ERR_SHAPE;
    if (dW->ld * es >= kHeadPitch) return FORGE_ERR_UNSUPPORTED;
  }
  const forge_tensor ws = flat(workspace, c.w.bytes), tt = flat(target, T * 8), ls = flat(lse, T * 4),
                     dl = flat(dloss, per_token ? T * 4 : 4), to = flat(total, 12);
  const forge_tensor* outs[3] = {dX, dW, &ws};
  const forge_tensor* ins[6] = {X, W, &tt, &ls, &dl, &to};
  if ((r = check_alias(outs, 3, ins, 6))) return r;
  if (in == 0 || (!dX && !dW)) return FORGE_OK;
  hipStream_t st = (hipStream_t)stream;
  for (int64_t v0 = 0; v0 < V; v0 += c.piece) {
    const int64_t n = V - v0 < c.piece ? V - v0 : c.piece;
    if (T > 0 && (r = enqueue_dz(c, v0, n, false, st))) return r;
    if (dX && T > 0 && (r = enqueue_dx(c, v0, n, false, st))) return r;
    if (!dW) continue;
    LinArgs g{};
    set_pair(g, 0, X->data, X->ld, c.ws + c.w.dz, up(c.piece, 8), T);
    g.nsrc = 1;
    g.M = (int32_t)in;
    g.N = (int32_t)n;
    g.e.out = (char*)dW->data + v0 * dW->ld * es;
    g.e.ldo = dW->ld;
    g.e.scale = per_token ? nullptr : dloss;
    g.e.count = total ? total + 1 : nullptr;
    if ((r = hip_status(launch_lin(bf16, L_ACC, true, true, g, st)))) return r;
  }
  return FORGE_OK;
}

int forge_linear_xent_step(const forge_tensor* X, forge_tensor* W, forge_tensor* m, forge_tensor* v, int32_t opt,
                           const forge_hyper* hyper, int64_t step, uint64_t seed, const int64_t* target,
                           int64_t ignore, const float* lse, const float* dloss, int32_t per_token,
                           const float* total, forge_tensor* dX, int64_t piece, void* workspace,
                           int64_t workspace_bytes, forge_stream_t stream) {
  int r = check_head(X, W, target);
  if (r) return r;
  if ((r = check_hyper(opt, hyper, step))) return r;
  const int io = W->dtype, bf16 = io == FORGE_BF16, es = bf16 ? 2 : 4;
  const int64_t T = X->rows, V = W->rows, in = W->cols;
  const int fmt = check_states(opt, io, W, m, v);
  if (fmt < 0) return fmt;
  const int sl = opt_slots(opt);
  if (V * in >= ((int64_t)1 << 32) || !fits_31(W) || ((sl & 1) && !fits_31(m)) || ((sl & 2) && !fits_31(v)))
    return FORGE_ERR_UNSUPPORTED;
  XentCall c{X, W, target, ignore, lse, dloss, per_token != 0, total, dX, piece_of(T, W->ld, V, es, piece),
             (char*)workspace, BwdWs{}};
  c.w = bwd_ws(T, in, c.piece, es);
  if ((r = check_xent_grad(c, piece, workspace_bytes))) return r;
  const forge_tensor ws = flat(workspace, c.w.bytes), tt = flat(target, T * 8), ls = flat(lse, T * 4),
                     dl = flat(dloss, per_token ? T * 4 : 4), to = flat(total, 12);
  const forge_tensor* outs[5] = {W, (sl & 1) ? m : nullptr, (sl & 2) ? v : nullptr, dX, &ws};
  const forge_tensor* ins[5] = {X, &tt, &ls, &dl, &to};
  if ((r = check_alias(outs, 5, ins, 5))) return r;
  forge_scalars sc;
  if ((r = forge_step_scalars(opt, hyper, step, &sc))) return r;
  if (in == 0) return FORGE_OK;
  hipStream_t st = (hipStream_t)stream;
  const int sr = bf16 && hyper->stochastic_round ? 1 : 0;
  const OptArgs whole = make_args(W, m, v, opt, sc, seed, step);
  const int ms = fmt == ST_F32 ? 4 : fmt == ST_BF16 ? 2 : 1;
  for (int64_t v0 = 0; v0 < V; v0 += c.piece) {
    const int64_t n = V - v0 < c.piece ? V - v0 : c.piece;
    if (T > 0 && (r = enqueue_dz(c, v0, n, true, st))) return r;
    if (dX && T > 0 && (r = enqueue_dx(c, v0, n, true, st))) return r;
    // the piece's rows as a layer of its own; its elements keep their places in the random
    // stream of the whole W (counter v0 in + index, and the stream is linear in the counter)
    OptArgs a = whole;
    a.out = (int32_t)n;
    a.W = (char*)whole.W + v0 * whole.ldw * es;
    if (whole.m) a.m = (char*)whole.m + v0 * whole.ldm * ms;
    if (whole.v) a.v = (char*)whole.v + v0 * whole.ldv * ms;
    if (whole.m_scale) a.m_scale = whole.m_scale + v0 * (in / 64);
    if (whole.v_scale) a.v_scale = whole.v_scale + v0 * (in / 64);
    a.rng_base = whole.rng_base + 0x9E3779B97F4A7C15ull * ((uint64_t)v0 * (uint64_t)in);
    const GemmDims d{(int32_t)T, (int32_t)n, (int32_t)in, X->ld, up(c.piece, 8)};
    if ((r = hip_status(launch_wgrad_fused(bf16, fmt, opt, sr, X->data, c.ws + c.w.dz, d, a, st)))) return r;
  }
  return FORGE_OK;
}

}  // extern "C"
