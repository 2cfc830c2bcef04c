// Kernels of the fused step and of gradient accumulation with X in 8 bits.
#include "forge_wgrad8.h"

namespace forge {

FORGE_ACT8_LIST(FORGE_INSTANTIATE_ACT8)

// Gradient accumulation: a.dW (fp32) = G, or += G with a.dw_add, from a G tile in LDS.
template <int ROWS, int THREADS>
__device__ __forceinline__ void store_g(const KArgs8& a, const float* sG, int row0, int col0) {
  const int cl = 8 * (threadIdx.x & 15);
  const int64_t c = col0 + cl;
#pragma unroll 4
  for (int r = threadIdx.x >> 4; r < ROWS; r += THREADS / 16) {
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

template <int XF>
__global__ void __launch_bounds__(NT, 2) k_gemm_act8_dma(const KArgs8 a) {
  __shared__ __attribute__((aligned(16))) char lds[LDS_BYTES];
  int ti, tj;
  tile_coords(blockIdx.x, a.tiles_n, a.tiles_k, ti, tj);
  f32x16 acc[2][2];
  Act8Loop<XF, 4, 2> loop;
  loop.run(a, lds, ti * TILE, tj * TILE, acc);
  bar();   // every wave is done with the stages before G overwrites them
  float* sG = reinterpret_cast<float*>(lds);
  store_acc(sG, acc, threadIdx.x);
  __syncthreads();
  store_g<TILE, NT>(a, sG, ti * TILE, tj * TILE);
}

template <int ROWS, int WAVES>
__global__ void __launch_bounds__(64 * WAVES, 1) k_gemm_act8_split(const KArgs8 a) {
  using M = Act8Split<ROWS, WAVES>;
  __shared__ __attribute__((aligned(16))) char lds[M::LDS];
  int ti, tj;
  tile_by_xcd((int)gridDim.x / a.tiles_k, a.tiles_k, ti, tj);
  f32x16 acc[M::BI][4];
  if (a.x_fmt == FMT_S8) M::template run<FMT_S8>(a, lds, ti * ROWS, tj * TILE, acc);
  else M::template run<FMT_E4M3>(a, lds, ti * ROWS, tj * TILE, acc);
  float* sG = reinterpret_cast<float*>(lds);
  M::join(sG, acc);
  store_g<ROWS, 64 * WAVES>(a, sG, ti * ROWS, tj * TILE);
}

__global__ void __launch_bounds__(NT, 2) k_gemm_act8_tiny(const KArgs8 a) {
  __shared__ __attribute__((aligned(16))) char lds[LDS_BYTES];
  int ti, tj;
  tile_coords(blockIdx.x, a.tiles_n, a.tiles_k, ti, tj);
  tile_gradient_by<MainAct8>(a, lds, ti * TILE, tj * TILE);
  store_g<TILE, NT>(a, reinterpret_cast<const float*>(lds), ti * TILE, tj * TILE);
}

// As for the step, but without the 256 x 256 tiles, which no accumulation has: 4096 x 4096,
// BT 8192 takes 314 us on the ring from S8 X and 265 from bf16 X, gate_proj at BT 512 105 and
// 91 (the step itself 266 and 248, 222 and 216).  The accumulator's rows may be of any
// alignment.
hipError_t launch_gemm_act8(const KArgs8& a, hipStream_t st) {
  if (act8_split(a, a.x_dma) && act8_few(a))
    hipLaunchKernelGGL((k_gemm_act8_split<32, 16>), split_grid<32>(a), dim3(1024), 0, st, a);
  else if (act8_split(a, a.x_dma)) hipLaunchKernelGGL((k_gemm_act8_split<64, 8>), split_grid<64>(a), dim3(512), 0, st, a);
  else if (a.x_dma && a.x_fmt == FMT_S8) hipLaunchKernelGGL((k_gemm_act8_dma<FMT_S8>), tile_grid(a), dim3(NT), 0, st, a);
  else if (a.x_dma) hipLaunchKernelGGL((k_gemm_act8_dma<FMT_E4M3>), tile_grid(a), dim3(NT), 0, st, a);
  else hipLaunchKernelGGL(k_gemm_act8_tiny, tile_grid(a), dim3(NT), 0, st, a);
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
