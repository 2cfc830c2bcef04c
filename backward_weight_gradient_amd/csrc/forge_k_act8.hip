// Activations to and from 8 bits.  Both directions stream: s bytes read and
// 1 + 1/block written per element (or the reverse), no arithmetic to speak of,
// so they are bound by HBM: 8192 x 14336 bf16 and S8 take 62 us to 8 bits and 60 back
// (354 MB, 5.8 TB/s).  X is read past the caches, which leaves them to the codes: both
// ways in turn take 121 us so, 136 with X through them (8192 x 4096, where all of it
// fits, 37.5 and 36.2; codes past the caches too: 123 and 40).
//
// Thread mapping: a lane owns 8 consecutive columns, so a block of 32, 64 or 128
// columns is 4, 8 or 16 adjacent lanes of one DPP row, which reduce its absmax
// without LDS.  A workgroup's 256 threads cover 256 / tpr rows of tpr * 8
// columns, tpr a power of two from 16 to 256 chosen so that a row is covered
// by as few idle lanes as possible; each thread holds UNR such rows, all
// requested before the first is used.
#include "forge_act8.h"

#include <algorithm>

namespace forge {

constexpr int ACT_UNR = 4;

struct ActArgs {
  const void* X; void* Xo; int64_t ldx;
  Act8 q;
  int64_t rows, K;
  int32_t tsh;      // log2(threads per row)
  int32_t segs;     // column segments of tpr * 8
  int64_t units;    // (rows / (rows per workgroup), segment) pairs
};

template <int MODE, int XF, int QF>
__device__ __forceinline__ void quantize_unit(const ActArgs& a, int64_t unit) {
  const int64_t rb = unit / a.segs;
  const int seg = (int)(unit - rb * a.segs);
  const int tpr = 1 << a.tsh, rpb = NT >> a.tsh;
  const int64_t c = ((int64_t)seg * tpr + (threadIdx.x & (tpr - 1))) * 8;
  const int64_t r0 = rb * (rpb * ACT_UNR) + (threadIdx.x >> a.tsh);
  constexpr int es = XF == FMT_F32 ? 4 : 2;
  Raw8<XF> w[ACT_UNR];
#pragma unroll
  for (int u = 0; u < ACT_UNR; ++u) {
    const int64_t r = min(r0 + (int64_t)u * rpb, a.rows - 1);   // a row past the end: read again, not stored
    w[u] = row_raw8<XF, MODE, true>(static_cast<const char*>(a.X) + r * a.ldx * es, c, a.K);
  }
#pragma unroll
  for (int u = 0; u < ACT_UNR; ++u) {
    const int64_t r = r0 + (int64_t)u * rpb;
    float x[8];
    row_val8<XF, MODE>(w[u], c, a.K, x);
    act8_store8<QF>(a.q, r, r < a.rows ? c : a.K, a.K, x);
  }
}

template <int MODE, int XF, int QF>
__device__ __forceinline__ void dequantize_unit(const ActArgs& a, int64_t unit) {
  const int64_t rb = unit / a.segs;
  const int seg = (int)(unit - rb * a.segs);
  const int tpr = 1 << a.tsh, rpb = NT >> a.tsh;
  const int64_t c = ((int64_t)seg * tpr + (threadIdx.x & (tpr - 1))) * 8;
  const int64_t r0 = rb * (rpb * ACT_UNR) + (threadIdx.x >> a.tsh);
  if (c >= a.K) return;
  constexpr int es = XF == FMT_F32 ? 4 : 2;
  u32x2 w[ACT_UNR];
  uint32_t s[ACT_UNR];
#pragma unroll
  for (int u = 0; u < ACT_UNR; ++u) {
    const int64_t r = min(r0 + (int64_t)u * rpb, a.rows - 1);
    w[u] = codes_raw8<MODE>(a.q.codes + r * a.q.ld, c, a.K);
    s[u] = a.q.scale[r * a.q.nb + (c >> a.q.sh)];
  }
#pragma unroll
  for (int u = 0; u < ACT_UNR; ++u) {
    const int64_t r = r0 + (int64_t)u * rpb;
    if (r >= a.rows) return;
    float x[8];
    const float f = act8_mul(s[u]);
    const u32x2 v = codes_val8<MODE>(w[u], c, a.K);
    act8_decode4<QF>(v[0], f, x);
    act8_decode4<QF>(v[1], f, x + 4);
    row_store8<XF>(static_cast<char*>(a.Xo) + r * a.ldx * es, c, a.K, x);
  }
}

template <bool QUANT, int MODE, int XF, int QF>
__global__ void __launch_bounds__(NT) k_act(const ActArgs a) {
  for (int64_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    if constexpr (QUANT) quantize_unit<MODE, XF, QF>(a, unit);
    else dequantize_unit<MODE, XF, QF>(a, unit);
  }
}

// Threads per row: the power of two (16 .. 256) that covers ceil(K / 8) lanes in
// the fewest lanes, the larger one on a tie (idle lanes cost: 65536 x 128 to 8 bits
// 6.7 us with 16, 31 with 256; 16384 x 1003 11.4 with 128, 14.8 with 16).
static int act_tsh(int64_t K) {
  const int64_t lanes = (K + 7) / 8;
  int best = 8;
  int64_t cost = -1;
  for (int s = 8; s >= 4; --s) {
    const int64_t c = ((lanes + (1 << s) - 1) >> s) << s;
    if (cost < 0 || c < cost) { cost = c; best = s; }
  }
  return best;
}

template <bool QUANT>
static hipError_t launch_act(ActArgs a, int x_fmt, int q_fmt, hipStream_t st) {
  if (a.rows == 0 || a.K == 0) return hipSuccess;
  a.tsh = act_tsh(a.K);
  a.segs = (int32_t)(((a.K + 7) / 8 + (1 << a.tsh) - 1) >> a.tsh);
  const int64_t rpb = (int64_t)(NT >> a.tsh) * ACT_UNR;
  a.units = ((a.rows + rpb - 1) / rpb) * a.segs;
  const unsigned grid = (unsigned)std::min<int64_t>(a.units, 1 << 22);
#define FORGE_ACT(XF, QF)                                                                                     \
  if (x_fmt == XF && q_fmt == QF) {                                                      \
    if (a.K >= 8) hipLaunchKernelGGL((k_act<QUANT, ROW_BIG, XF, QF>), dim3(grid), dim3(NT), 0, st, a); \
    else hipLaunchKernelGGL((k_act<QUANT, ROW_ANY, XF, QF>), dim3(grid), dim3(NT), 0, st, a);          \
    return hipGetLastError();                                                            \
  }
  FORGE_ACT(FMT_BF16, FMT_S8)
  FORGE_ACT(FMT_BF16, FMT_E4M3)
  FORGE_ACT(FMT_F32, FMT_S8)
  FORGE_ACT(FMT_F32, FMT_E4M3)
#undef FORGE_ACT
  return hipErrorInvalidValue;
}

hipError_t launch_act_quantize(const void* X, int64_t ldx, int x_fmt, const Act8& q, int q_fmt, int64_t rows, int64_t K,
                               hipStream_t st) {
  return launch_act<true>({X, nullptr, ldx, q, rows, K, 0, 0, 0}, x_fmt, q_fmt, st);
}
hipError_t launch_act_dequantize(const Act8& q, int q_fmt, void* X, int64_t ldx, int x_fmt, int64_t rows, int64_t K,
                                 hipStream_t st) {
  return launch_act<false>({nullptr, X, ldx, q, rows, K, 0, 0, 0}, x_fmt, q_fmt, st);
}

}  // namespace forge
