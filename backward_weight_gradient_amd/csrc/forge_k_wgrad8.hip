// Kernels of the fused step and of gradient accumulation with X in 8 bits.
#include "forge_wgrad8.h"

namespace forge {

FORGE_ACT8_LIST(FORGE_INSTANTIATE_ACT8)

// Gradient accumulation: a.dW (fp32) = G, or += G with a.dw_add.
template <int MODE>
__global__ void __launch_bounds__(NT, 2) k_gemm_act8(const KArgs8 a) {
  __shared__ __attribute__((aligned(16))) char lds[LDS_BYTES];
  int ti, tj;
  tile_coords(blockIdx.x, a.tiles_n, a.tiles_k, ti, tj);
  const int row0 = ti * TILE, col0 = tj * TILE;
  tile_gradient_by<MainAct8<MODE>>(a, lds, row0, col0);
  const float* sG = reinterpret_cast<const float*>(lds);
  const int cl = 8 * (threadIdx.x & 15);
  const int64_t c = col0 + cl;
#pragma unroll 4
  for (int r = threadIdx.x >> 4; r < TILE; r += NT / 16) {
    if (row0 + r >= a.N) return;
    float* out = static_cast<float*>(a.dW) + (int64_t)(row0 + r) * a.lddw;
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = sG[r * GP + cl + i];
    if (a.dw_add) {
      float o[8];
      row_load8<FMT_F32>(out, c, a.K, o);
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = o[i] + g[i];
    }
    row_store8<FMT_F32>(out, c, a.K, g);
  }
}

hipError_t launch_gemm_act8(const KArgs8& a, hipStream_t st) {
  if (a.N >= 8 && a.K >= 8) hipLaunchKernelGGL((k_gemm_act8<ROW_BIG>), tile_grid(a), dim3(NT), 0, st, a);
  else hipLaunchKernelGGL((k_gemm_act8<ROW_ANY>), tile_grid(a), dim3(NT), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_fused_act8(const KArgs8& a, int w_fmt, int opt, int m_fmt, int v_fmt, hipStream_t st) {
#define X(O, M, V) \
  if (opt == O && m_fmt == M && v_fmt == V) return combo_fused_act8<O, M, V>(a, w_fmt, st);
  FORGE_ACT8_LIST(X)
#undef X
  return hipErrorInvalidValue;
}

}  // namespace forge
