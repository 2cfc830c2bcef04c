// Host side of the activation-checkpoint, RMSNorm and embedding entry points:
// argument validation and dispatch.  Implements include/forge.h.

#include "forge_checks.h"

namespace {

constexpr int64_t kMax31 = 1ll << 31;

Act8 act8_args(const forge_act8& q) {
  return {static_cast<uint8_t*>(q.q.data), q.q.ld, q.scale, (int32_t)act8_nb(q), q.block == 32 ? 5 : q.block == 64 ? 6 : 7};
}

bool is_float(int dtype) { return dtype == FORGE_F32 || dtype == FORGE_BF16; }

// A matrix of F32 or BF16, or absent.
forge_status check_float_mat(const forge_mat* m, int64_t rows, int64_t cols) {
  if (!m) return FORGE_OK;
  const forge_status st = check_mat(*m, rows, cols);
  if (st != FORGE_OK) return st;
  return is_float(m->dtype) ? FORGE_OK : FORGE_E_DTYPE;
}

// The buffers of a call: nothing written overlaps anything else.
struct Uses {
  Range r[12];
  bool out[12];
  int n = 0;
  void add(const Range& range, bool written) {
    r[n] = range;
    out[n++] = written;
  }
  forge_status check() const {
    for (int i = 0; i < n; ++i)
      for (int j = 0; j < n; ++j)
        if (i != j && out[i] && overlap(r[i], r[j])) return FORGE_E_ALIAS;
    return FORGE_OK;
  }
};
Range opt_range(const forge_mat* m) { return m ? mat_range(*m) : Range(); }

// Exactly the same matrix: each element is read and then written by one thread.
bool same_mat(const forge_mat* a, const forge_mat* b) {
  return a && b && a->data == b->data && a->dtype == b->dtype && (a->ld == b->ld || a->rows <= 1);
}

// A caller's scratch of `need` bytes.
forge_status check_workspace(const void* ws, int64_t bytes, int64_t need) {
  if (bytes < 0) return FORGE_E_SHAPE;
  if (need == 0) return FORGE_OK;
  if (!ws) return FORGE_E_NULL;
  if (bytes < need) return FORGE_E_SHAPE;
  return aligned(ws, 16) ? FORGE_OK : FORGE_E_ALIGN;
}

forge_status check_act_copy(const forge_act8* Q, const forge_mat* X) {
  if (!Q || !X) return FORGE_E_NULL;
  const int64_t rows = X->rows, cols = X->cols;
  forge_status st = check_float_mat(X, rows, cols);
  if (st != FORGE_OK) return st;
  if ((st = check_act8(*Q, rows, cols)) != FORGE_OK) return st;
  Uses u;
  u.add(mat_range(*X), true);
  u.add(mat_range(Q->q), true);
  u.add(act8_scale_range(*Q), true);
  return u.check();
}

void act8_input(const forge_act8* X, KArgs8& a) {
  a.x8 = act8_args(*X);
  a.x_fmt = X->q.dtype == FORGE_S8 ? FMT_S8 : FMT_E4M3;
  // the asynchronous mainloop: 16-byte aligned rows of dY and 4-byte aligned rows of
  // codes (a buffer load's alignment), both in whole 16-byte segments, byte offsets
  // that fit the 32-bit buffer addressing
  a.x_dma = (vec_ok(a.dY, a.lddy, 8, 2) && a.N % 8 == 0 && vec_ok(X->q.data, X->q.ld, 4, 1) && a.K % 16 == 0 &&
             (uint64_t)a.BT * (uint64_t)a.lddy * 2 < (1ull << 31) && (uint64_t)a.BT * (uint64_t)X->q.ld < (1ull << 31))
                ? 1 : 0;
}

// Token ids: T values of 4 or 8 bytes.
forge_status check_ids(const void* ids, int32_t id_bytes, int64_t T) {
  if (id_bytes != 4 && id_bytes != 8) return FORGE_E_SHAPE;
  if (T < 0 || T >= kMax31) return FORGE_E_SHAPE;
  if (T > 0 && !ids) return FORGE_E_NULL;
  return aligned(ids, id_bytes) ? FORGE_OK : FORGE_E_ALIGN;
}

constexpr int64_t round16(int64_t n) { return (n + 15) & ~15ll; }

// ids, dY, scale and workspace of an embedding gradient of V x K; fills the launch arguments.
forge_status check_embed_grad(const void* ids, int32_t id_bytes, int64_t T, const forge_mat* dY, double scale, int64_t V,
                              int64_t K, void* ws, int64_t ws_bytes, Uses& u, EmbedArgs& e) {
  if (!dY) return FORGE_E_NULL;
  forge_status st = check_ids(ids, id_bytes, T);
  if (st != FORGE_OK) return st;
  if (V < 0 || K < 0 || V >= kMax31 || K >= kMax31 || T >= EMBED_MAX_TOKENS) return FORGE_E_SHAPE;
  if ((st = check_float_mat(dY, T, K)) != FORGE_OK) return st;
  if (!std::isfinite((float)scale)) return FORGE_E_HYPER;
  const int64_t need = V > 0 && K > 0 ? forge_embed_workspace_bytes(T, V) : 0;
  if ((st = check_workspace(ws, ws_bytes, need)) != FORGE_OK) return st;
  u.add(raw_range(ids, (uint64_t)T * (uint64_t)id_bytes), false);
  u.add(mat_range(*dY), false);
  u.add(raw_range(ws, (uint64_t)need), true);
  std::memset(&e, 0, sizeof(e));
  e.ids = ids; e.id_bytes = id_bytes;
  e.T = T; e.V = V; e.K = K;
  e.dY = dY->data; e.lddy = dY->ld; e.dy_fmt = dY->dtype;
  e.scale = (float)scale;
  char* p = static_cast<char*>(ws);
  e.key = reinterpret_cast<int32_t*>(p);    p += round16(4 * T);
  e.perm = reinterpret_cast<int32_t*>(p);   p += round16(4 * T);
  e.tile = reinterpret_cast<int32_t*>(p);   p += round16(4 * (V / EMBED_ROWS + 2));
  e.part = reinterpret_cast<uint64_t*>(p);
  return FORGE_OK;
}

}  // namespace

extern "C" {

forge_status forge_act_quantize(const forge_mat* X, forge_act8* Q, void* stream) {
  const forge_status st = check_act_copy(Q, X);
  if (st != FORGE_OK) return st;
  return hip_status(launch_act_quantize(X->data, X->ld, X->dtype, act8_args(*Q), Q->q.dtype, X->rows, X->cols,
                                        (hipStream_t)stream));
}

forge_status forge_act_dequantize(const forge_act8* Q, forge_mat* X, void* stream) {
  const forge_status st = check_act_copy(Q, X);
  if (st != FORGE_OK) return st;
  return hip_status(launch_act_dequantize(act8_args(*Q), Q->q.dtype, X->data, X->ld, X->dtype, X->rows, X->cols,
                                          (hipStream_t)stream));
}

forge_status forge_wgrad_check_act8(const forge_act8* X, const forge_mat* dY, const forge_mat* W, const forge_state* m,
                                    const forge_state* v, const forge_hyper* h, int64_t step) {
  if (!X) return FORGE_E_NULL;
  Plan pl;
  return validate(&X->q, dY, W, m, v, h, step, pl, nullptr, X);
}

forge_status forge_wgrad_step_act8(const forge_act8* X, const forge_mat* dY, forge_mat* W, forge_state* m,
                                   forge_state* v, const forge_hyper* h, int64_t step, uint64_t seed, void* stream) {
  if (!X) return FORGE_E_NULL;
  Plan pl;
  const forge_status st = validate(&X->q, dY, W, m, v, h, step, pl, nullptr, X);
  if (st != FORGE_OK || pl.empty) return st;
  KArgs8 a;
  static_cast<KArgs&>(a) = make_args(&X->q, dY, W, m, v, h, step, seed, pl);
  act8_input(X, a);
  return hip_status(launch_fused_act8(a, pl.w_fmt, h->opt, pl.m_fmt, pl.v_fmt, (hipStream_t)stream));
}

forge_status forge_wgrad_accumulate_act8(const forge_act8* X, const forge_mat* dY, forge_mat* acc, int32_t first,
                                         void* stream) {
  if (!X) return FORGE_E_NULL;
  Plan pl;
  forge_status st = validate_inputs(&X->q, dY, pl, X);
  if (st != FORGE_OK) return st;
  if ((st = check_acc(acc, pl.N, pl.K)) != FORGE_OK) return st;
  const Range ra = mat_range(*acc);
  if (overlap(ra, mat_range(X->q)) || overlap(ra, act8_scale_range(*X)) || overlap(ra, mat_range(*dY)))
    return FORGE_E_ALIAS;
  if (pl.empty) return FORGE_OK;
  KArgs8 a;
  std::memset(&a, 0, sizeof(a));
  input_args(&X->q, dY, pl, a);
  acc_args(acc, a);
  a.dw_add = first ? 0 : 1;
  act8_input(X, a);
  return hip_status(launch_gemm_act8(a, (hipStream_t)stream));
}

forge_status forge_rmsnorm(const forge_mat* X, const forge_mat* R, const forge_mat* gamma, double eps, forge_mat* H,
                           forge_mat* Y, forge_act8* Q, float* rstd, void* stream) {
  if (!X || !gamma) return FORGE_E_NULL;
  if (!R != !H) return FORGE_E_NULL;
  if (!H && !Y && !Q && !rstd) return FORGE_E_NULL;
  const int64_t rows = X->rows, cols = X->cols;
  forge_status st;
  if ((st = check_float_mat(X, rows, cols)) != FORGE_OK) return st;
  if ((st = check_float_mat(R, rows, cols)) != FORGE_OK) return st;
  if ((st = check_float_mat(H, rows, cols)) != FORGE_OK) return st;
  if ((st = check_float_mat(Y, rows, cols)) != FORGE_OK) return st;
  if ((st = check_float_mat(gamma, 1, cols)) != FORGE_OK) return st;
  if (Q && (st = check_act8(*Q, rows, cols)) != FORGE_OK) return st;
  if (R && R->dtype != H->dtype) return FORGE_E_DTYPE;
  if (rows >= kMax31 || cols >= kMax31) return FORGE_E_SHAPE;
  // the kernels add eps in fp32: a positive one must stay positive and finite there
  const float eps32 = (float)eps;
  if (!std::isfinite(eps32) || eps < 0 || (eps32 == 0.f && eps != 0)) return FORGE_E_HYPER;
  if (!aligned(rstd, 4)) return FORGE_E_ALIGN;
  Uses u;
  if (!same_mat(H, X)) u.add(mat_range(*X), false);
  if (!same_mat(H, R)) u.add(opt_range(R), false);
  u.add(mat_range(*gamma), false);
  u.add(opt_range(H), true);
  u.add(opt_range(Y), true);
  u.add(raw_range(rstd, (uint64_t)rows * 4), true);
  if (Q) {
    u.add(mat_range(Q->q), true);
    u.add(act8_scale_range(*Q), true);
  }
  if ((st = u.check()) != FORGE_OK) return st;
  NormArgs a;
  std::memset(&a, 0, sizeof(a));
  a.X = X->data; a.ldx = X->ld; a.x_fmt = X->dtype;
  if (R) {
    a.R = R->data; a.ldr = R->ld; a.r_fmt = R->dtype;
    a.H = H->data; a.ldh = H->ld;
  }
  a.gamma = gamma->data; a.g_fmt = gamma->dtype;
  if (Y) { a.Y = Y->data; a.ldy = Y->ld; a.y_fmt = Y->dtype; }
  if (Q) { a.q = act8_args(*Q); a.q_fmt = Q->q.dtype; }
  a.rstd = rstd;
  a.rows = rows; a.K = (int32_t)cols;
  a.eps = eps32;
  return hip_status(launch_rmsnorm(a, (hipStream_t)stream));
}

int64_t forge_rmsnorm_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || cols <= 0 || rows >= kMax31 || cols >= kMax31) return 0;
  return (int64_t)norm_parts(rows, cols) * ((cols + 3) & ~3ll) * 4;
}

forge_status forge_rmsnorm_backward(const forge_mat* dY, const forge_mat* H, const forge_mat* gamma, const float* rstd,
                                    const forge_mat* dR, forge_mat* dX, float* dgamma, int32_t first, void* workspace,
                                    int64_t workspace_bytes, void* stream) {
  if (!dY || !H || !gamma) return FORGE_E_NULL;
  if (!dX && !dgamma) return FORGE_E_NULL;
  const int64_t rows = H->rows, cols = H->cols;
  forge_status st;
  if ((st = check_float_mat(H, rows, cols)) != FORGE_OK) return st;
  if ((st = check_float_mat(dY, rows, cols)) != FORGE_OK) return st;
  if ((st = check_float_mat(dR, rows, cols)) != FORGE_OK) return st;
  if ((st = check_float_mat(dX, rows, cols)) != FORGE_OK) return st;
  if ((st = check_float_mat(gamma, 1, cols)) != FORGE_OK) return st;
  if (rows >= kMax31 || cols >= kMax31) return FORGE_E_SHAPE;
  if (rows > 0 && cols > 0 && !rstd) return FORGE_E_NULL;
  if (dR && !dX) return FORGE_E_NULL;
  if (dR && dR->dtype != dX->dtype) return FORGE_E_DTYPE;
  if (!aligned(rstd, 4) || !aligned(dgamma, 4)) return FORGE_E_ALIGN;
  const int64_t need = dgamma ? forge_rmsnorm_workspace_bytes(rows, cols) : 0;
  if ((st = check_workspace(workspace, workspace_bytes, need)) != FORGE_OK) return st;
  Uses u;
  if (!same_mat(dX, dY)) u.add(mat_range(*dY), false);
  if (!same_mat(dX, dR)) u.add(opt_range(dR), false);
  u.add(mat_range(*H), false);
  u.add(mat_range(*gamma), false);
  u.add(raw_range(rstd, (uint64_t)rows * 4), false);
  u.add(opt_range(dX), true);
  u.add(raw_range(dgamma, (uint64_t)cols * 4), true);
  u.add(raw_range(workspace, (uint64_t)need), true);
  if ((st = u.check()) != FORGE_OK) return st;
  NormBwdArgs a;
  std::memset(&a, 0, sizeof(a));
  a.dY = dY->data; a.lddy = dY->ld; a.dy_fmt = dY->dtype;
  a.H = H->data; a.ldh = H->ld; a.h_fmt = H->dtype;
  a.gamma = gamma->data; a.g_fmt = gamma->dtype;
  a.rstd = rstd;
  if (dR) { a.dR = dR->data; a.lddr = dR->ld; }
  if (dX) { a.dX = dX->data; a.lddx = dX->ld; a.dx_fmt = dX->dtype; }
  a.dgamma = dgamma;
  a.ws = static_cast<float*>(workspace);
  a.first = first ? 1 : 0;
  a.rows = rows; a.K = (int32_t)cols;
  return hip_status(launch_rmsnorm_backward(a, (hipStream_t)stream));
}

forge_status forge_embed(const void* ids, int32_t id_bytes, int64_t T, const forge_mat* W, double scale, forge_mat* Y,
                         void* stream) {
  if (!W || !Y) return FORGE_E_NULL;
  const int64_t V = W->rows, K = W->cols;
  forge_status st = check_ids(ids, id_bytes, T);
  if (st != FORGE_OK) return st;
  if ((st = check_float_mat(W, V, K)) != FORGE_OK) return st;
  if ((st = check_float_mat(Y, T, K)) != FORGE_OK) return st;
  if (V >= kMax31 || K >= kMax31) return FORGE_E_SHAPE;
  if (!std::isfinite((float)scale)) return FORGE_E_HYPER;
  Uses u;
  u.add(raw_range(ids, (uint64_t)T * (uint64_t)id_bytes), false);
  u.add(mat_range(*W), false);
  u.add(mat_range(*Y), true);
  if ((st = u.check()) != FORGE_OK) return st;
  return hip_status(launch_embed(ids, id_bytes, T, W->data, W->ld, W->dtype, V, K, (float)scale, Y->data, Y->ld, Y->dtype,
                                 (hipStream_t)stream));
}

int64_t forge_embed_workspace_bytes(int64_t T, int64_t V) {
  if (T < 0 || V <= 0 || T >= EMBED_MAX_TOKENS || V >= kMax31) return 0;
  return 2 * round16(4 * T) + round16(4 * (V / EMBED_ROWS + 2)) + (T > EMBED_PART ? 8 * T : 0);
}

forge_status forge_embed_accumulate(const void* ids, int32_t id_bytes, int64_t T, const forge_mat* dY, double scale,
                                    forge_mat* acc, int32_t first, void* workspace, int64_t workspace_bytes,
                                    void* stream) {
  if (!acc) return FORGE_E_NULL;
  forge_status st = check_acc(acc, acc->rows, acc->cols);
  if (st != FORGE_OK) return st;
  Uses u;
  EmbedArgs e;
  st = check_embed_grad(ids, id_bytes, T, dY, scale, acc->rows, acc->cols, workspace, workspace_bytes, u, e);
  if (st != FORGE_OK) return st;
  u.add(mat_range(*acc), true);
  if ((st = u.check()) != FORGE_OK) return st;
  return hip_status(launch_embed_accumulate(e, static_cast<float*>(acc->data), acc->ld, first != 0, (hipStream_t)stream));
}

forge_status forge_embed_step(const void* ids, int32_t id_bytes, int64_t T, const forge_mat* dY, double scale,
                              forge_mat* W, forge_state* m, forge_state* v, const forge_hyper* h, int64_t step,
                              uint64_t seed, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!W) return FORGE_E_NULL;
  // the weight, state and hyper-parameter checks of forge_wgrad_step, with no tokens
  const int64_t V = W->rows, K = W->cols;
  const forge_mat none_x = {nullptr, FORGE_BF16, 0, K, K > 0 ? K : 1}, none_y = {nullptr, FORGE_BF16, 0, V, V > 0 ? V : 1};
  Plan pl;
  forge_status st = validate(&none_x, &none_y, W, m, v, h, step, pl);
  if (st != FORGE_OK) return st;
  Uses u;
  EmbedArgs e;
  st = check_embed_grad(ids, id_bytes, T, dY, scale, V, K, workspace, workspace_bytes, u, e);
  if (st != FORGE_OK) return st;
  Range outs[5], ins[2];
  layer_ranges(&none_x, &none_y, W, m, v, pl, outs, ins);
  for (const Range& r : outs) u.add(r, true);
  if ((st = u.check()) != FORGE_OK) return st;
  if ((V + EMBED_ROWS - 1) / EMBED_ROWS * ((K + 127) / 128) >= EMBED_MAX_TILES) return FORGE_E_SHAPE;
  if (pl.empty) return FORGE_OK;
  const KArgs a = make_args(&none_x, &none_y, W, m, v, h, step, seed, pl);
  return hip_status(launch_embed_step(a, e, pl.w_fmt, h->opt, pl.m_fmt, pl.v_fmt, (hipStream_t)stream));
}

}  // extern "C"
