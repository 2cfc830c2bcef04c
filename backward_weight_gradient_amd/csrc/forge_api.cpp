// Host side of libforge: argument validation, per-call scalars, dispatch.
// Implements include/forge.h.

#include "forge_checks.h"

static_assert(FORGE_GROUP_MAX == forge::GROUP_MAX, "group size of the ABI and the kernels");
static_assert(FORGE_DGRAD_SCRATCH_BYTES == forge::DGRAD_SCRATCH_BYTES, "scratch size of the ABI and the kernels");
static_assert(FORGE_QUOTIENT_COUNTS == forge::QUOTIENT_CHECK_BLOCKS * 8, "quotient check counters of the ABI and the kernel");

namespace {
thread_local hipError_t g_last_hip = hipSuccess;
}  // namespace

namespace forge {
forge_status hip_status(hipError_t e) {
  if (e == hipSuccess) return FORGE_OK;
  g_last_hip = e;
  return FORGE_E_HIP;
}
}  // namespace forge

extern "C" {

forge_status forge_wgrad_check(const forge_mat* X, const forge_mat* dY, const forge_mat* W, const forge_state* m,
                               const forge_state* v, const forge_hyper* h, int64_t step) {
  Plan pl;
  return validate(X, dY, W, m, v, h, step, pl);
}

forge_status forge_wgrad_step(const forge_mat* X, const forge_mat* dY, forge_mat* W, forge_state* m, forge_state* v,
                              const forge_hyper* h, int64_t step, uint64_t seed, void* stream) {
  Plan pl;
  forge_status st = validate(X, dY, W, m, v, h, step, pl);
  if (st != FORGE_OK || pl.empty) return st;
  const KArgs a = make_args(X, dY, W, m, v, h, step, seed, pl);
  return hip_status(launch_fused(a, pl.in_fmt, pl.w_fmt, h->opt, pl.m_fmt, pl.v_fmt, (hipStream_t)stream));
}

forge_status forge_wgrad_step_fp8w(const forge_mat* X, const forge_mat* dY, forge_state* W, forge_state* m,
                                   forge_state* v, const forge_hyper* h, int64_t step, uint64_t seed, void* stream) {
  if (!W) return FORGE_E_NULL;
  Plan pl;
  forge_status st = validate(X, dY, &W->q, m, v, h, step, pl, W);
  if (st != FORGE_OK || pl.empty) return st;
  KArgs a = make_args(X, dY, &W->q, m, v, h, step, seed, pl);
  a.wsc = W->scale;
  return hip_status(launch_fused_fp8w(a, h->opt, pl.m_fmt, pl.v_fmt, (hipStream_t)stream));
}

forge_status forge_wgrad_check_fp8w(const forge_mat* X, const forge_mat* dY, const forge_state* W,
                                    const forge_state* m, const forge_state* v, const forge_hyper* h, int64_t step) {
  if (!W) return FORGE_E_NULL;
  Plan pl;
  return validate(X, dY, &W->q, m, v, h, step, pl, W);
}

forge_status forge_dgrad_fp8w(const forge_mat* dY, const forge_state* W, forge_mat* dX, void* stream) {
  if (!W) return FORGE_E_NULL;
  DgArgs g;
  bool fast = false;
  const forge_status st = check_dgrad(dY, &W->q, dX, g, fast, W);
  if (st != FORGE_OK) return st;
  // the bf16 matrix-core kernel: 16-byte rows of dY (8 bf16) and W (16
  // codes), whole 16-byte segments, buffer offsets within 32 bits
  const int64_t N = dY->cols, K = W->q.cols;
  const bool fast8 = dY->dtype == FORGE_BF16 && N % 8 == 0 && K % 16 == 0 && vec_ok(dY->data, dY->ld, 8, 2) &&
                     vec_ok(W->q.data, W->q.ld, 16, 1) && (uint64_t)dY->rows * (uint64_t)dY->ld * 2 < (1ull << 31) &&
                     (uint64_t)N * (uint64_t)W->q.ld < (1ull << 31) &&
                     (uint64_t)N * (uint64_t)(K / W->block) * 4 < (1ull << 31);
  return hip_status(launch_dgrad_fp8w(g, fast8, (hipStream_t)stream));
}

forge_status forge_wgrad_step_group(const forge_layer* layers, int32_t n, const forge_hyper* h, int64_t step,
                                    void* stream) {
  if (n < 1 || n > FORGE_GROUP_MAX) return FORGE_E_SHAPE;
  if (!layers || !h) return FORGE_E_NULL;
  Plan pl[FORGE_GROUP_MAX];
  for (int i = 0; i < n; ++i) {
    const forge_layer& L = layers[i];
    const forge_status st = validate(L.X, L.dY, L.W, L.m, L.v, h, step, pl[i]);
    if (st != FORGE_OK) return st;
  }
  // one kernel instantiation serves the group: identical formats
  int ref = -1;
  for (int i = 0; i < n; ++i) {
    if (pl[i].empty) continue;
    if (ref < 0) { ref = i; continue; }
    const Plan& a = pl[ref];
    const Plan& b = pl[i];
    if (a.in_fmt != b.in_fmt || a.w_fmt != b.w_fmt || a.m_fmt != b.m_fmt || a.v_fmt != b.v_fmt ||
        a.block != b.block)
      return FORGE_E_UNSUPPORTED;
  }
  if (ref < 0) return FORGE_OK;
  // layers are independent: nothing one layer writes may overlap any buffer of another
  Range outs[FORGE_GROUP_MAX][5], ins[FORGE_GROUP_MAX][2];
  for (int i = 0; i < n; ++i) {
    const forge_layer& L = layers[i];
    layer_ranges(L.X, L.dY, L.W, L.m, L.v, pl[i], outs[i], ins[i]);
  }
  for (int i = 0; i < n; ++i)
    for (int j = 0; j < n; ++j) {
      if (i == j) continue;
      for (int p = 0; p < 5; ++p) {
        for (int q = 0; q < 5; ++q)
          if (overlap(outs[i][p], outs[j][q])) return FORGE_E_ALIAS;
        for (int q = 0; q < 2; ++q)
          if (overlap(outs[i][p], ins[j][q])) return FORGE_E_ALIAS;
      }
    }
  // eligible layers share one launch; the others get their own
  GroupArgs g;
  std::memset(&g, 0, sizeof(g));
  int64_t tiles = 0;
  for (int i = 0; i < n; ++i) {
    if (pl[i].empty) continue;
    const forge_layer& L = layers[i];
    const KArgs a = make_args(L.X, L.dY, L.W, L.m, L.v, h, step, L.seed, pl[i]);
    if (group_eligible(a, pl[i].in_fmt)) {
      g.layer[g.n] = a;
      g.first_tile[g.n] = (int32_t)tiles;
      tiles += (int64_t)a.tiles_n * a.tiles_k;
      ++g.n;
    } else {
      const forge_status st =
          hip_status(launch_fused(a, pl[i].in_fmt, pl[i].w_fmt, h->opt, pl[i].m_fmt, pl[i].v_fmt, (hipStream_t)stream));
      if (st != FORGE_OK) return st;
    }
  }
  if (g.n == 0) return FORGE_OK;
  g.first_tile[g.n] = (int32_t)tiles;
  return hip_status(launch_fused_group(g, pl[ref].w_fmt, h->opt, pl[ref].m_fmt, pl[ref].v_fmt, (hipStream_t)stream));
}

forge_status forge_wgrad_unfused(const forge_mat* X, const forge_mat* dY, forge_mat* W, forge_state* m,
                                 forge_state* v, const forge_hyper* h, int64_t step, uint64_t seed, void* dW,
                                 int32_t dW_dtype, void* stream) {
  Plan pl;
  forge_status st = validate(X, dY, W, m, v, h, step, pl);
  if (st != FORGE_OK) return st;
  if (dW_dtype != FORGE_F32 && dW_dtype != FORGE_BF16) return FORGE_E_DTYPE;
  if (pl.empty) return FORGE_OK;
  if (dW == nullptr) return FORGE_E_NULL;
  if (!aligned(dW, 16)) return FORGE_E_ALIGN;
  const Range ws = raw_range(dW, (uint64_t)pl.N * (uint64_t)pl.K * (uint64_t)elem_size(dW_dtype));
  Range outs[5], ins[2];
  layer_ranges(X, dY, W, m, v, pl, outs, ins);
  for (const Range& r : outs)
    if (overlap(ws, r)) return FORGE_E_ALIAS;
  for (const Range& r : ins)
    if (overlap(ws, r)) return FORGE_E_ALIAS;
  KArgs a = make_args(X, dY, W, m, v, h, step, seed, pl);
  a.dW = dW;
  a.dw_fmt = dW_dtype == FORGE_F32 ? FMT_F32 : FMT_BF16;
  a.vec_dw = ((pl.K % 4) == 0 && pitch_ok(pl.K, 4)) ? 1 : 0;   // the workspace is 16-byte aligned with ld = K
  hipError_t e = launch_gemm(a, pl.in_fmt, (hipStream_t)stream);
  if (e == hipSuccess) e = launch_step(a, pl.w_fmt, h->opt, pl.m_fmt, pl.v_fmt, (hipStream_t)stream);
  return hip_status(e);
}

forge_status forge_wgrad_accumulate(const forge_mat* X, const forge_mat* dY, forge_mat* acc, int32_t first,
                                    void* stream) {
  Plan pl;
  forge_status st = validate_inputs(X, dY, pl);
  if (st != FORGE_OK) return st;
  if ((st = check_acc(acc, pl.N, pl.K)) != FORGE_OK) return st;
  const Range ra = mat_range(*acc);
  if (overlap(ra, mat_range(*X)) || overlap(ra, mat_range(*dY))) return FORGE_E_ALIAS;
  if (pl.empty) return FORGE_OK;
  KArgs a;
  std::memset(&a, 0, sizeof(a));
  input_args(X, dY, pl, a);
  acc_args(acc, a);
  a.dw_add = first ? 0 : 1;
  return hip_status(launch_gemm(a, pl.in_fmt, (hipStream_t)stream));
}

forge_status forge_wgrad_step_accumulated(const forge_mat* X, const forge_mat* dY, forge_mat* acc, forge_mat* W,
                                          forge_state* m, forge_state* v, const forge_hyper* h, int64_t step,
                                          uint64_t seed, void* stream) {
  Plan pl;
  forge_status st = validate(X, dY, W, m, v, h, step, pl);
  if (st != FORGE_OK) return st;
  if ((st = check_acc(acc, pl.N, pl.K)) != FORGE_OK) return st;
  Range outs[5], ins[2];
  layer_ranges(X, dY, W, m, v, pl, outs, ins);
  const Range ra = mat_range(*acc);
  for (const Range& r : outs)
    if (overlap(ra, r)) return FORGE_E_ALIAS;
  for (const Range& r : ins)
    if (overlap(ra, r)) return FORGE_E_ALIAS;
  if (pl.empty) return FORGE_OK;
  KArgs a = make_args(X, dY, W, m, v, h, step, seed, pl);
  acc_args(acc, a);
  // aligned bf16: one fused kernel adds the accumulator to the tile in the
  // epilogue; otherwise this micro-batch is added into the accumulator and
  // the step reads it back (the same fp32 addition, so the same result)
  if (pl.in_fmt == FORGE_BF16 && a.dma_ok && a.vec_state && a.vec_dw && pl.K % 4 == 0)
    return hip_status(launch_fused_acc(a, pl.w_fmt, h->opt, pl.m_fmt, pl.v_fmt, (hipStream_t)stream));
  a.dw_add = 1;
  hipError_t e = launch_gemm(a, pl.in_fmt, (hipStream_t)stream);
  if (e == hipSuccess) e = launch_step(a, pl.w_fmt, h->opt, pl.m_fmt, pl.v_fmt, (hipStream_t)stream);
  return hip_status(e);
}

forge_status forge_dgrad(const forge_mat* dY, const forge_mat* W, forge_mat* dX, void* stream) {
  DgArgs g;
  bool fast = false;
  const forge_status st = check_dgrad(dY, W, dX, g, fast);
  if (st != FORGE_OK) return st;
  return hip_status(launch_dgrad(g, fast, (hipStream_t)stream));
}

int64_t forge_dgrad_workspace_bytes(int64_t BT, int64_t N, int64_t K) {
  if (BT <= 0 || N <= 0 || K <= 0 || BT >= (1ll << 31) || N >= (1ll << 31) || K >= (1ll << 31)) return 0;
  const int s = dgrad_splits(BT, N, K);
  return s > 1 ? (int64_t)s * BT * K * 4 : 0;
}

// The workspace of the split dX kernel, checked against every buffer of the
// call (`others`), and the split recorded in g; no-op where no split applies.
static forge_status attach_dgrad_workspace(DgArgs& g, bool fast, void* workspace, int64_t workspace_bytes,
                                           const Range* others, int n_others) {
  if (workspace_bytes < 0) return FORGE_E_SHAPE;
  const int64_t need = forge_dgrad_workspace_bytes(g.BT, g.N, g.K);
  if (!fast || need == 0) return FORGE_OK;
  if (!workspace) return FORGE_E_NULL;
  if (workspace_bytes < need) return FORGE_E_SHAPE;
  if (!aligned(workspace, 16)) return FORGE_E_ALIGN;
  const Range rw = raw_range(workspace, (uint64_t)need);
  for (int i = 0; i < n_others; ++i)
    if (overlap(rw, others[i])) return FORGE_E_ALIAS;
  g.splits = dgrad_splits(g.BT, g.N, g.K);
  g.ws = static_cast<float*>(workspace);
  return FORGE_OK;
}

forge_status forge_dgrad_split(const forge_mat* dY, const forge_mat* W, forge_mat* dX, void* workspace,
                               int64_t workspace_bytes, void* stream) {
  DgArgs g;
  bool fast = false;
  forge_status st = check_dgrad(dY, W, dX, g, fast);
  if (st != FORGE_OK) return st;
  const Range others[3] = {mat_range(*dY), mat_range(*W), mat_range(*dX)};
  if ((st = attach_dgrad_workspace(g, fast, workspace, workspace_bytes, others, 3)) != FORGE_OK) return st;
  return hip_status(launch_dgrad(g, fast, (hipStream_t)stream));
}

forge_status forge_dgrad_split_noalloc(const forge_mat* dY, const forge_mat* W, forge_mat* dX, void* stream) {
  DgArgs g;
  bool fast = false;
  const forge_status st = check_dgrad(dY, W, dX, g, fast);
  if (st != FORGE_OK) return st;
  const int64_t need = fast ? forge_dgrad_workspace_bytes(g.BT, g.N, g.K) : 0;
  if (need > FORGE_DGRAD_SCRATCH_BYTES) return FORGE_E_SCRATCH;
  if (need > 0) g.splits = dgrad_splits(g.BT, g.N, g.K);
  return hip_status(launch_dgrad_scratch(g, fast, (hipStream_t)stream));
}

static forge_status backward_step(const forge_mat* X, const forge_mat* dY, forge_mat* W, forge_state* m,
                                  forge_state* v, const forge_hyper* h, int64_t step, uint64_t seed, forge_mat* dX,
                                  bool split, void* workspace, int64_t workspace_bytes, void* stream) {
  Plan pl;
  forge_status st = validate(X, dY, W, m, v, h, step, pl);
  if (st != FORGE_OK) return st;
  DgArgs g;
  bool fast = false;
  if ((st = check_dgrad(dY, W, dX, g, fast)) != FORGE_OK) return st;
  Range outs[5], ins[2];
  layer_ranges(X, dY, W, m, v, pl, outs, ins);
  const Range rx = mat_range(*dX);
  for (const Range& r : outs)
    if (overlap(rx, r)) return FORGE_E_ALIAS;
  for (const Range& r : ins)
    if (overlap(rx, r)) return FORGE_E_ALIAS;
  if (split) {
    const Range others[8] = {outs[0], outs[1], outs[2], outs[3], outs[4], ins[0], ins[1], rx};
    if ((st = attach_dgrad_workspace(g, fast, workspace, workspace_bytes, others, 8)) != FORGE_OK) return st;
  }
  // stream order is the contract: dX reads W before the fused step rewrites it
  hipError_t e = launch_dgrad(g, fast, (hipStream_t)stream);
  if (e != hipSuccess) return hip_status(e);
  if (pl.empty) return FORGE_OK;
  const KArgs a = make_args(X, dY, W, m, v, h, step, seed, pl);
  return hip_status(launch_fused(a, pl.in_fmt, pl.w_fmt, h->opt, pl.m_fmt, pl.v_fmt, (hipStream_t)stream));
}

forge_status forge_backward_step(const forge_mat* X, const forge_mat* dY, forge_mat* W, forge_state* m, forge_state* v,
                                 const forge_hyper* h, int64_t step, uint64_t seed, forge_mat* dX, void* stream) {
  return backward_step(X, dY, W, m, v, h, step, seed, dX, false, nullptr, 0, stream);
}

forge_status forge_backward_step_split(const forge_mat* X, const forge_mat* dY, forge_mat* W, forge_state* m,
                                       forge_state* v, const forge_hyper* h, int64_t step, uint64_t seed,
                                       forge_mat* dX, void* workspace, int64_t workspace_bytes, void* stream) {
  return backward_step(X, dY, W, m, v, h, step, seed, dX, true, workspace, workspace_bytes, stream);
}

forge_status forge_debug_sr_bf16(const float* in, uint16_t* out, int64_t n, uint64_t seed, int64_t step,
                                 uint32_t tensor_id, void* stream) {
  if (n < 0 || (uint64_t)n >= (1ull << 32)) return FORGE_E_SHAPE;
  if (step < 1) return FORGE_E_STEP;
  if (n == 0) return FORGE_OK;
  if (!in || !out) return FORGE_E_NULL;
  if (!aligned(in, 4) || !aligned(out, 2)) return FORGE_E_ALIGN;
  if (overlap(raw_range(in, (uint64_t)n * 4), raw_range(out, (uint64_t)n * 2))) return FORGE_E_ALIAS;
  const uint32_t key = sr_key(seed, (uint64_t)step, tensor_id);
  return hip_status(launch_debug_sr(in, out, (uint32_t)n, key, (hipStream_t)stream));
}

forge_status forge_debug_e4m3(const float* in, uint8_t* out, int64_t n, void* stream) {
  if (n < 0 || (uint64_t)n >= (1ull << 32)) return FORGE_E_SHAPE;
  if (n == 0) return FORGE_OK;
  if (!in || !out) return FORGE_E_NULL;
  if (!aligned(in, 4)) return FORGE_E_ALIGN;
  if (overlap(raw_range(in, (uint64_t)n * 4), raw_range(out, (uint64_t)n))) return FORGE_E_ALIAS;
  return hip_status(launch_debug_e4m3(in, out, (uint32_t)n, (hipStream_t)stream));
}

forge_status forge_debug_e4m3_sr(const float* in, uint8_t* out, int64_t n, uint64_t seed, int64_t step,
                                 void* stream) {
  if (n < 0 || (uint64_t)n >= (1ull << 32)) return FORGE_E_SHAPE;
  if (step < 1) return FORGE_E_STEP;
  if (n == 0) return FORGE_OK;
  if (!in || !out) return FORGE_E_NULL;
  if (!aligned(in, 4)) return FORGE_E_ALIGN;
  if (overlap(raw_range(in, (uint64_t)n * 4), raw_range(out, (uint64_t)n))) return FORGE_E_ALIAS;
  return hip_status(launch_debug_e4m3_sr(in, out, (uint32_t)n, sr_key(seed, (uint64_t)step, 0), (hipStream_t)stream));
}

forge_status forge_debug_quotients(uint64_t* counts, void* stream) {
  if (!counts) return FORGE_E_NULL;
  if (!aligned(counts, 8)) return FORGE_E_ALIGN;
  return hip_status(launch_debug_quotients(reinterpret_cast<unsigned long long*>(counts), (hipStream_t)stream));
}

forge_status forge_debug_quant(const float* in, uint8_t* codes, float* scales, int64_t rows, int64_t cols,
                               int32_t dtype, int32_t second_moment, int32_t block, void* stream) {
  if (dtype != FORGE_S8 && dtype != FORGE_U8 && dtype != FORGE_E4M3) return FORGE_E_DTYPE;
  if (second_moment != 0 && second_moment != 1) return FORGE_E_DTYPE;
  if ((dtype == FORGE_S8 && second_moment) || (dtype == FORGE_U8 && !second_moment)) return FORGE_E_DTYPE;
  if (!(block == 32 || block == 64 || block == 128)) return FORGE_E_SHAPE;
  if (rows < 0 || cols < 0 || cols % block != 0) return FORGE_E_SHAPE;
  if ((uint64_t)rows * (uint64_t)cols >= (1ull << 32) || rows >= (1ll << 31) || cols >= (1ll << 31))
    return FORGE_E_SHAPE;
  if (rows == 0 || cols == 0) return FORGE_OK;
  if (!in || !codes || !scales) return FORGE_E_NULL;
  if (!aligned(in, 4) || !aligned(codes, 4) || !aligned(scales, 4)) return FORGE_E_ALIGN;
  const uint64_t n = (uint64_t)rows * (uint64_t)cols;
  const Range ri = raw_range(in, n * 4), rc = raw_range(codes, n), rs = raw_range(scales, n / (uint64_t)block * 4);
  if (overlap(ri, rc) || overlap(ri, rs) || overlap(rc, rs)) return FORGE_E_ALIAS;
  return hip_status(launch_debug_quant(in, codes, scales, (int)rows, (int)cols, dtype, second_moment != 0, block,
                                       (hipStream_t)stream));
}

forge_status forge_debug_copy(const void* src, void* dst, int64_t bytes, void* stream) {
  if (bytes < 0 || bytes % 16 != 0) return FORGE_E_SHAPE;
  if (bytes == 0) return FORGE_OK;
  if (!src || !dst) return FORGE_E_NULL;
  if (!aligned(src, 16) || !aligned(dst, 16)) return FORGE_E_ALIGN;
  if (overlap(raw_range(src, (uint64_t)bytes), raw_range(dst, (uint64_t)bytes))) return FORGE_E_ALIAS;
  return hip_status(launch_debug_copy(src, dst, (uint64_t)bytes, (hipStream_t)stream));
}

forge_status forge_debug_state_stream(uint16_t* W, float* m, float* v, int64_t N, int64_t K, void* stream) {
  if (N < 0 || K < 0 || N % 128 != 0 || K % 128 != 0) return FORGE_E_SHAPE;
  if ((uint64_t)N * (uint64_t)K >= (1ull << 32) || N >= (1ll << 31) || K >= (1ll << 31)) return FORGE_E_SHAPE;
  if (N == 0 || K == 0) return FORGE_OK;
  if (!W || !m || !v) return FORGE_E_NULL;
  if (!aligned(W, 8) || !aligned(m, 16) || !aligned(v, 16)) return FORGE_E_ALIGN;
  const uint64_t n = (uint64_t)N * (uint64_t)K;
  const Range rw = raw_range(W, 2 * n), rm = raw_range(m, 4 * n), rv = raw_range(v, 4 * n);
  if (overlap(rw, rm) || overlap(rw, rv) || overlap(rm, rv)) return FORGE_E_ALIAS;
  return hip_status(launch_debug_state_stream(W, m, v, (int)N, (int)K, (hipStream_t)stream));
}

forge_status forge_debug_mfma_peak(float* out, int32_t blocks, int32_t iters, void* stream) {
  if (blocks < 1 || blocks > (1 << 20) || iters < 1 || iters > (1 << 20)) return FORGE_E_SHAPE;
  if (!out) return FORGE_E_NULL;
  if (!aligned(out, 4)) return FORGE_E_ALIGN;
  return hip_status(launch_debug_mfma(out, blocks, iters, (hipStream_t)stream));
}

const char* forge_last_error(void) { return hipGetErrorString(g_last_hip); }

const char* forge_status_str(forge_status s) {
  switch (s) {
    case FORGE_OK: return "FORGE_OK";
    case FORGE_E_NULL: return "FORGE_E_NULL: a required pointer is NULL";
    case FORGE_E_SHAPE: return "FORGE_E_SHAPE: shapes disagree or exceed a limit";
    case FORGE_E_DTYPE: return "FORGE_E_DTYPE: dtype not allowed here";
    case FORGE_E_ALIGN: return "FORGE_E_ALIGN: misaligned pointer";
    case FORGE_E_STEP: return "FORGE_E_STEP: step must be >= 1";
    case FORGE_E_HYPER: return "FORGE_E_HYPER: invalid optimizer or hyper-parameter";
    case FORGE_E_ALIAS: return "FORGE_E_ALIAS: an output overlaps another buffer";
    case FORGE_E_UNSUPPORTED: return "FORGE_E_UNSUPPORTED: combination not implemented";
    case FORGE_E_HIP: return "FORGE_E_HIP: HIP launch error";
    case FORGE_E_SCRATCH: return "FORGE_E_SCRATCH: the call needs more than the static scratch array holds";
  }
  return "unknown forge_status";
}

const char* forge_version(void) { return "forge-mi355x 0.1.0 (gfx950)"; }

}  // extern "C"
