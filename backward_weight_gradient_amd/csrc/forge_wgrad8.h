// The fused weight gradient with X in 8 bits.
//
// G = dY^T X with X = code * 2^e.  The exponent differs from token to token, so
// it cannot leave the sum; each 8 bits are decoded to the bf16 they stand for
// (exactly) between global memory and LDS, after which the matrix-core loop is
// that of bf16 inputs: every element of G sees the same MFMA sequence as with
// the decoded X, and the results are the same bit for bit.
#pragma once

#include "forge_act8.h"

namespace forge {

// 8 codes as 8 bf16 values.
template <int XF>
__device__ __forceinline__ u32x4 act8_bf16x8(u32x2 w, float f) {
  float x[8];
  act8_decode4<XF>(w[0], f, x);
  act8_decode4<XF>(w[1], f, x + 4);
  return u32x4{bf16x2_rne(x[0], x[1]), bf16x2_rne(x[2], x[3]), bf16x2_rne(x[4], x[5]), bf16x2_rne(x[6], x[7])};
}

// Any shape and alignment: MainBF16 with its register staging, X decoded on the
// way into LDS.
struct MainAct8 {
  static constexpr int TK = MainBF16::TK;
  static constexpr int OPB = MainBF16::OPB;
  static constexpr int STAGE = MainBF16::STAGE;
  u32x4 ra[4];
  u32x2 rc[4];
  uint32_t rs[4];
  bool e4m3;

  __device__ __forceinline__ void load(const KArgs8& a, int kc, int row0, int col0) {
    const int tid = threadIdx.x;
    const int f = (tid & 15) * 8;
    const int64_t cy = row0 + f, cx = col0 + f;
    e4m3 = a.x_fmt == FMT_E4M3;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int tok = kc * TK + (tid >> 4) + 16 * r;
      const bool in = tok < a.BT;
      const uint16_t* y = static_cast<const uint16_t*>(a.dY) + (int64_t)tok * a.lddy;
      u32x4 w = {0u, 0u, 0u, 0u};
      if (in && cy + 8 <= a.N) {
        w = *reinterpret_cast<const u32x4_u*>(y + cy);
      } else if (in) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (cy + i < a.N) w[i >> 1] |= (uint32_t)y[cy + i] << (16 * (i & 1));
      }
      ra[r] = w;
      rc[r] = in ? codes_load8(a.x8.codes + (int64_t)tok * a.x8.ld, cx, a.K) : u32x2{0u, 0u};
      rs[r] = in && cx < a.K ? (uint32_t)a.x8.scale[(int64_t)tok * a.x8.nb + (cx >> a.x8.sh)] : 0u;
    }
  }

  __device__ __forceinline__ void store(char* stage) const {
    const int tid = threadIdx.x;
    const int f = (tid & 15) * 8;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = (tid >> 4) + 16 * r;
      const float s = act8_mul(rs[r]);
      *reinterpret_cast<u32x4*>(stage + MainBF16::off(t, f)) = ra[r];
      *reinterpret_cast<u32x4*>(stage + OPB + MainBF16::off(t, f)) =
          e4m3 ? act8_bf16x8<FMT_E4M3>(rc[r], s) : act8_bf16x8<FMT_S8>(rc[r], s);
    }
  }

  __device__ __forceinline__ static void compute(f32x16 (&acc)[2][2], char* stage, int wr, int wc, int lane) {
    MainBF16::compute(acc, stage, wr, wc, lane);
  }
};

template <int OPT, int WF, int MF, int VF>
__global__ void __launch_bounds__(NT, 2) k_fused_act8(const KArgs8 a) {
  __shared__ __attribute__((aligned(16))) char lds[LDS_BYTES];
  int ti, tj;
  tile_coords(blockIdx.x, a.tiles_n, a.tiles_k, ti, tj);
  const int row0 = ti * TILE, col0 = tj * TILE;
  Epilogue<Step<OPT, WF, MF, VF, false>, FMT_NONE, false, 4> epi;
  epi.tid = threadIdx.x;
  tile_gradient_by<MainAct8>(a, lds, row0, col0);
  epi.prefetch(a, row0, col0);
  epi.run_prefetched(a, reinterpret_cast<const float*>(lds), row0, col0);
}

template <int O, int M, int V>
hipError_t combo_fused_act8(const KArgs8& a, int w_fmt, hipStream_t st) {
  if (w_fmt == FMT_BF16) hipLaunchKernelGGL((k_fused_act8<O, FMT_BF16, M, V>), tile_grid(a), dim3(NT), 0, st, a);
  else if (w_fmt == FMT_F32) hipLaunchKernelGGL((k_fused_act8<O, FMT_F32, M, V>), tile_grid(a), dim3(NT), 0, st, a);
  else return hipErrorInvalidValue;
  return hipGetLastError();
}
#define FORGE_INSTANTIATE_ACT8(O, M, V) \
  template hipError_t combo_fused_act8<O, M, V>(const KArgs8&, int, hipStream_t);

}  // namespace forge
