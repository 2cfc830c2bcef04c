// Root-mean-square norm with the residual's addition and 8-bit output, and its
// backward pass.
//
// Forward, per row: h = rn(x + r), s = 1 / sqrt(sum h^2 / K + eps), y = h s gamma.
// Backward, per row, with g = gamma dy and n = h s:
//   dx = s (g - n sum(g n) / K) + dr;   dgamma = sum over rows of dy n.
// One pass over the data each way: a row is held in registers by LPR lanes, VEC
// vectors of 8 columns each (lane i of the row, vector j: columns 8 (j LPR + i)
// on), so its sum is a reduction over lanes and nothing is read twice.  All sums
// are fp32: a row's over a lane's values and then a tree over the lanes, dgamma's
// over a workgroup's rows in order, then over its row groups, then over the
// workgroups' partial sums in a fixed order (k_norm_dgamma).
// Both kernels move 6 to 12 bytes per element for about 10 flops: bound by HBM.
#include "forge_act8.h"

#include <algorithm>

namespace forge {

// Sum over the LPR lanes of a row (LPR 16, 64: inside a wave; 256, 1024: over
// the 4 or 16 waves of the row through LDS).  Every lane gets the sum.  part:
// one float per wave of the workgroup; two buffers used in turn let one barrier
// a row do (a wave writes a buffer again only after the next barrier, which all
// waves reach after they read it).
template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __uint_as_float((uint32_t)__builtin_amdgcn_mov_dpp((int)__float_as_uint(x), CTRL, 0xF, 0xF, true));
}
template <int LPR>
__device__ __forceinline__ float row_sum(float x, float* part) {
  x = dpp_add<0x140>(dpp_add<0x141>(dpp_add<0x4E>(dpp_add<0xB1>(x))));
  if constexpr (LPR >= 64) {
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
  }
  if constexpr (LPR > 64) {
    constexpr int W = LPR / 64;
    const int wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) part[wave] = x;
    __syncthreads();
    x = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) x += part[(wave & ~(W - 1)) + i];
  }
  return x;
}

template <int MODE>
__device__ __forceinline__ void load8_as(int fmt, const void* base, int64_t elem, int64_t c, int64_t K, float (&x)[8]) {
  if (fmt == FMT_F32) row_load8<FMT_F32, MODE>(static_cast<const float*>(base) + elem, c, K, x);
  else row_load8<FMT_BF16, MODE>(static_cast<const uint16_t*>(base) + elem, c, K, x);
}
template <int MODE>
__device__ __forceinline__ void store8_as(int fmt, void* base, int64_t elem, int64_t c, int64_t K, const float (&x)[8]) {
  if (fmt == FMT_F32) row_store8<FMT_F32, MODE>(static_cast<float*>(base) + elem, c, K, x);
  else row_store8<FMT_BF16, MODE>(static_cast<uint16_t*>(base) + elem, c, K, x);
}

constexpr int norm_threads(int lpr) { return lpr > 256 ? lpr : 256; }

// 8 columns of a row: Y and the 8-bit copy.
template <int MODE>
__device__ __forceinline__ void norm_out8(const NormArgs& a, int64_t row, int64_t c, int64_t lim, const float (&y)[8]) {
  if (a.Y) store8_as<MODE>(a.y_fmt, a.Y, row * a.ldy, c, lim, y);
  if (a.q.codes) {
    float z[8];       // columns from K on do not count in a block's absmax (0 * s may be NaN)
#pragma unroll
    for (int e = 0; e < 8; ++e) z[e] = c + e < lim ? y[e] : 0.f;
    if (a.q_fmt == FMT_S8) act8_store8<FMT_S8, MODE>(a.q, row, c, lim, z);
    else act8_store8<FMT_E4M3, MODE>(a.q, row, c, lim, z);
  }
}

// h = x + r, rounded to r's type and stored as H.
template <int RF, int MODE>
__device__ __forceinline__ void add_residual8(const NormArgs& a, int64_t row, int64_t c, int64_t lim, const float (&r)[8],
                                              float (&h)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) h[e] += r[e];
  if constexpr (RF == FMT_BF16) {   // the norm is of H as stored
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const uint32_t w = bf16x2_rne(h[e], h[e + 1]);
      h[e] = __uint_as_float(w << 16);
      h[e + 1] = __uint_as_float(w & 0xFFFF0000u);
    }
  }
  row_store8<RF, MODE>(static_cast<char*>(a.H) + row * a.ldh * (RF == FMT_F32 ? 4 : 2), c, lim, h);
}

// A row that needs VEC vectors ends in the last of them; the others are whole.
template <int MODE, int VEC, class F>
__device__ __forceinline__ void each_vector(F&& f) {
#pragma unroll
  for (int j = 0; j + 1 < VEC; ++j) f(std::integral_constant<int, ROW_WHOLE>{}, j);
  f(std::integral_constant<int, MODE>{}, VEC - 1);
}

// RF: the residual's format, FMT_NONE without one.
template <int XF, int RF, int LPR, int VEC, int MODE>
__global__ void __launch_bounds__(norm_threads(LPR)) k_rmsnorm(const NormArgs a) {
  constexpr int THREADS = norm_threads(LPR), RPB = THREADS / LPR;
  constexpr int xs = XF == FMT_F32 ? 4 : 2, rs = RF == FMT_F32 ? 4 : 2;
  __shared__ float part[2][16];
  const int i = threadIdx.x & (LPR - 1);
  const int64_t K = a.K;
  float gam[VEC][8];
  each_vector<MODE, VEC>([&](auto w, int j) {
    load8_as<w()>(a.g_fmt, a.gamma, 0, (int64_t)(j * LPR + i) * 8, K, gam[j]);
  });
  int buf = 0;
  for (int64_t base = (int64_t)blockIdx.x * RPB; base < a.rows; base += (int64_t)gridDim.x * RPB, buf ^= 1) {
    const int64_t row = base + threadIdx.x / LPR, rd = min(row, a.rows - 1);
    const bool live = row < a.rows;
    const int64_t lim = live ? K : 0;     // a row past the end reads the last one and stores nothing
    Raw8<XF> xr[VEC];
    Raw8<RF == FMT_NONE ? FMT_BF16 : RF> rr[VEC];
    each_vector<MODE, VEC>([&](auto w, int j) {
      const int64_t c = (int64_t)(j * LPR + i) * 8;
      xr[j] = row_raw8<XF, w()>(static_cast<const char*>(a.X) + rd * a.ldx * xs, c, K);
      if constexpr (RF != FMT_NONE) rr[j] = row_raw8<RF, w()>(static_cast<const char*>(a.R) + rd * a.ldr * rs, c, K);
    });
    float h[VEC][8];
    each_vector<MODE, VEC>([&](auto w, int j) {
      const int64_t c = (int64_t)(j * LPR + i) * 8;
      row_val8<XF, w()>(xr[j], c, K, h[j]);
      if constexpr (RF != FMT_NONE) {
        float r[8];
        row_val8<RF, w()>(rr[j], c, K, r);
        add_residual8<RF, w()>(a, row, c, lim, r, h[j]);
      }
    });
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(h[j][e], h[j][e], ss);
    ss = row_sum<LPR>(ss, part[buf]);
    const float s = 1.f / sqrtf(ss / (float)a.K + a.eps);
    if (a.rstd && live && i == 0) a.rstd[row] = s;
    if (!a.Y && !a.q.codes) continue;
    each_vector<MODE, VEC>([&](auto w, int j) {
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = (h[j][e] * s) * gam[j][e];
      norm_out8<w()>(a, row, (int64_t)(j * LPR + i) * 8, lim, y);
    });
  }
}

// Rows of any length: one per 1024-thread workgroup, read a second time (H,
// or X without a residual) for the output.
template <int XF, int RF>
__global__ void __launch_bounds__(1024) k_rmsnorm_long(const NormArgs a) {
  constexpr int xs = XF == FMT_F32 ? 4 : 2, rs = RF == FMT_F32 ? 4 : 2;
  __shared__ float part[2][16];
  const int64_t K = a.K;
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
    float ss = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < K; c += 8192) {
      float h[8];
      row_load8<XF>(static_cast<const char*>(a.X) + row * a.ldx * xs, c, K, h);
      if constexpr (RF != FMT_NONE) {
        float r[8];
        row_load8<RF>(static_cast<const char*>(a.R) + row * a.ldr * rs, c, K, r);
        add_residual8<RF, ROW_ANY>(a, row, c, K, r, h);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(h[e], h[e], ss);
    }
    ss = row_sum<1024>(ss, part[buf]);
    const float s = 1.f / sqrtf(ss / (float)a.K + a.eps);
    if (a.rstd && threadIdx.x == 0) a.rstd[row] = s;
    if (!a.Y && !a.q.codes) continue;
    // every lane of a block's group stays in the loop together: K rounded up to 128
    for (int64_t c = (int64_t)threadIdx.x * 8; c < ((K + 127) & ~127ll); c += 8192) {
      float h[8], g[8], y[8];
      // (what this thread itself stored as H above)
      if constexpr (RF != FMT_NONE) row_load8<RF>(static_cast<const char*>(a.H) + row * a.ldh * rs, c, K, h);
      else row_load8<XF>(static_cast<const char*>(a.X) + row * a.ldx * xs, c, K, h);
      load8_as<ROW_ANY>(a.g_fmt, a.gamma, 0, c, K, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = (h[e] * s) * g[e];
      norm_out8<ROW_ANY>(a, row, c, K, y);
    }
  }
}

// ------------------------------------------------------------------------
// Backward
// ------------------------------------------------------------------------
constexpr int NB_T = 1024;                // threads of the backward kernel
// Workgroups of the backward kernels, each with a part of dgamma's sums: one per CU
// (calls in a captured graph, dgamma's second kernel in them, no residual gradient: 8192 x
// 4096 bf16 36.0 us; 128: 41.2, 512: 38.9, 1024: 45.6; 1021 x 5001 bf16 15.4, 17.9, 18.5, 26.2).
constexpr int NB_PARTS = 256;

// dx of 8 columns: s (g - n mean) + dr.
template <int MODE>
__device__ __forceinline__ void norm_dx8(const NormBwdArgs& a, int64_t row, int64_t c, int64_t lim, float s, float mean,
                                         const float (&n)[8], const float (&d)[8], const float (&g)[8]) {
  float dx[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) dx[e] = s * fmaf(-n[e], mean, d[e] * g[e]);
  if (a.dR) {
    float r[8];
    load8_as<MODE>(a.dx_fmt, a.dR, min(row, a.rows - 1) * a.lddr, c, a.K, r);
#pragma unroll
    for (int e = 0; e < 8; ++e) dx[e] += r[e];
  }
  store8_as<MODE>(a.dx_fmt, a.dX, row * a.lddx, c, lim, dx);
}

template <int HF, int DF, int LPR, int VEC, int MODE>
__global__ void __launch_bounds__(NB_T) k_rmsnorm_backward(const NormBwdArgs a) {
  constexpr int RPB = NB_T / LPR;
  constexpr int hs = HF == FMT_F32 ? 4 : 2, ds = DF == FMT_F32 ? 4 : 2;
  __shared__ float part[2][16];
  __shared__ float comb[RPB > 1 ? LPR * VEC * 8 : 1];
  const int i = threadIdx.x & (LPR - 1);
  const int64_t K = a.K;
  const float fk = (float)a.K;
  float gam[VEC][8], dg[VEC][8];
  each_vector<MODE, VEC>([&](auto w, int j) {
    load8_as<w()>(a.g_fmt, a.gamma, 0, (int64_t)(j * LPR + i) * 8, K, gam[j]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dg[j][e] = 0.f;
  });
  // With one vector a lane the next row is requested (as stored) before the current
  // one is reduced, so that its latency passes behind the reduction's barrier; with
  // two there are no registers for that at 1024 threads.
  constexpr bool AHEAD = VEC == 1;
  Raw8<HF> hn[VEC];
  Raw8<DF> dn[VEC];
  float sn = 0.f;
  const auto request = [&](int64_t row) {
    const int64_t rd = min(row, a.rows - 1);       // past the end: the last row again, cleared below
    sn = a.rstd[rd];
    each_vector<MODE, VEC>([&](auto w, int j) {
      const int64_t c = (int64_t)(j * LPR + i) * 8;
      hn[j] = row_raw8<HF, w()>(static_cast<const char*>(a.H) + rd * a.ldh * hs, c, K);
      dn[j] = row_raw8<DF, w()>(static_cast<const char*>(a.dY) + rd * a.lddy * ds, c, K);
    });
  };
  int buf = 0;
  int64_t base = (int64_t)blockIdx.x * RPB;
  if (AHEAD) request(base + threadIdx.x / LPR);
  for (; base < a.rows; base += (int64_t)gridDim.x * RPB, buf ^= 1) {
    const int64_t row = base + threadIdx.x / LPR;
    if (!AHEAD) request(row);
    const bool live = row < a.rows;
    const float s = sn;
    float n[VEC][8], d[VEC][8];
    each_vector<MODE, VEC>([&](auto w, int j) {
      const int64_t c = (int64_t)(j * LPR + i) * 8;
      row_val8<HF, w()>(hn[j], c, K, n[j]);
      row_val8<DF, w()>(dn[j], c, K, d[j]);
    });
    if (AHEAD) request(row + (int64_t)gridDim.x * RPB);
    float dot = 0.f;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[j][e] *= s;
        const float dn = d[j][e] * n[j][e];
        dot = fmaf(dn, gam[j][e], dot);
        dg[j][e] += live ? dn : 0.f;
      }
    if (!a.dX) continue;
    const float mean = row_sum<LPR>(dot, part[buf]) / fk;
    each_vector<MODE, VEC>([&](auto w, int j) {
      norm_dx8<w()>(a, row, (int64_t)(j * LPR + i) * 8, live ? K : 0, s, mean, n[j], d[j], gam[j]);
    });
  }
  if (!a.dgamma) return;
  // The workgroup's row groups in order: those of one wave by lane exchange,
  // then one group after another through LDS.
  if constexpr (LPR < 64) {
#pragma unroll
    for (int j = 0; j < VEC; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dg[j][e] += __shfl_xor(dg[j][e], 16);
        dg[j][e] += __shfl_xor(dg[j][e], 32);
      }
  }
  if constexpr (RPB > 1) {
    constexpr int GL = LPR < 64 ? 64 : LPR;          // lanes of one group of the second step
    const int grp = threadIdx.x / GL;
    for (int g = 0; g < NB_T / GL; ++g) {
      if (grp == g && (threadIdx.x & (GL - 1)) < LPR) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float* p = comb + (j * LPR + i) * 8 + e;
            *p = g == 0 ? dg[j][e] : *p + dg[j][e];
          }
      }
      __syncthreads();
    }
    if (threadIdx.x >= LPR) return;
#pragma unroll
    for (int j = 0; j < VEC; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) dg[j][e] = comb[(j * LPR + i) * 8 + e];
  }
  const int64_t pitch = (K + 3) & ~3ll;
  each_vector<MODE, VEC>([&](auto w, int j) {
    row_store8<FMT_F32, w()>(a.ws + blockIdx.x * pitch, (int64_t)(j * LPR + i) * 8, K, dg[j]);
  });
}

// Rows of any length: one per workgroup, read twice; a workgroup's sums for
// dgamma live in its part of the workspace (each thread reads and writes its own
// columns only).
template <int HF, int DF>
__global__ void __launch_bounds__(NB_T) k_rmsnorm_backward_long(const NormBwdArgs a) {
  constexpr int hs = HF == FMT_F32 ? 4 : 2, ds = DF == FMT_F32 ? 4 : 2;
  __shared__ float part[2][16];
  const int64_t K = a.K;
  float* ws = a.ws + blockIdx.x * ((K + 3) & ~3ll);
  int buf = 0;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, buf ^= 1) {
    const char* hp = static_cast<const char*>(a.H) + row * a.ldh * hs;
    const char* dp = static_cast<const char*>(a.dY) + row * a.lddy * ds;
    const float s = a.rstd[row];
    float dot = 0.f;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < K; c += 8192) {
      float n[8], d[8], g[8];
      row_load8<HF>(hp, c, K, n);
      row_load8<DF>(dp, c, K, d);
      load8_as<ROW_ANY>(a.g_fmt, a.gamma, 0, c, K, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) dot = fmaf(d[e] * g[e], n[e] * s, dot);
    }
    const float mean = row_sum<1024>(dot, part[buf]) / (float)a.K;
    for (int64_t c = (int64_t)threadIdx.x * 8; c < K; c += 8192) {
      float n[8], d[8], g[8];
      row_load8<HF>(hp, c, K, n);
      row_load8<DF>(dp, c, K, d);
      load8_as<ROW_ANY>(a.g_fmt, a.gamma, 0, c, K, g);
#pragma unroll
      for (int e = 0; e < 8; ++e) n[e] *= s;
      if (a.dgamma) {
        float t[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
        if (row != (int64_t)blockIdx.x) row_load8<FMT_F32>(ws, c, K, t);
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = fmaf(d[e], n[e], t[e]);
        row_store8<FMT_F32>(ws, c, K, t);
      }
      if (a.dX) norm_dx8<ROW_ANY>(a, row, c, K, s, mean, n, d, g);
    }
  }
}

// dgamma (+)= the sum of the parts: 16 lanes of 4 columns by 16 groups of parts.
// (8192 x 4096: 4 us for 4 MB.)
__global__ void __launch_bounds__(NT) k_norm_dgamma(const NormBwdArgs a) {
  __shared__ float sum[16][64 + 4];
  const int64_t pitch = ((int64_t)a.K + 3) & ~3ll;
  const int cl = 4 * (threadIdx.x & 15), grp = threadIdx.x >> 4;
  for (int64_t c0 = (int64_t)blockIdx.x * 64; c0 < a.K; c0 += (int64_t)gridDim.x * 64) {
    const int64_t c = c0 + cl;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    if (c < pitch) {
#pragma unroll 4
      for (int p = grp; p < a.parts; p += 16) s += *reinterpret_cast<const f32x4*>(a.ws + p * pitch + c);
    }
    __syncthreads();                       // the columns before are summed
#pragma unroll
    for (int e = 0; e < 4; ++e) sum[grp][cl + e] = s[e];
    __syncthreads();
    const int64_t col = c0 + threadIdx.x;
    if (threadIdx.x < 64 && col < a.K) {
      float t = 0.f;
#pragma unroll
      for (int g = 0; g < 16; ++g) t += sum[g][threadIdx.x];
      a.dgamma[col] = a.first ? t : a.dgamma[col] + t;
    }
  }
}

// ------------------------------------------------------------------------
// Launchers.  Rows of 8 to 16384 columns are held in registers, in the smallest
// (LPR, VEC) whose LPR * VEC * 8 columns hold one, in kernels of their own where all
// vectors are whole (8192 x 4096 forward 41.0 us, 42.6 in the general one; 65536 x 128
// 12.2, 12.8): more lanes than a row needs idle
// (65536 x 128 forward 12.4 us with 16, 21.6 with 64; 16384 x 1024 21.6 with 64, 27.5
// with 256, 66 with 1024).  Others are read twice (2048 x 16384: 44 us in registers, 63
// read twice; backward 43 and 95).  8192 x 4096 bf16 in a captured graph: forward with a
// residual 42 us (268 MB, 6.4 TB/s), without 22; backward with dgamma 36.5 us (201 MB,
// 5.5 TB/s), with the residual's gradient as well 46 (268 MB, 5.8 TB/s).
// ------------------------------------------------------------------------
constexpr int64_t NORM_REG_COLS = 16384;
#define FORGE_NORM_SHAPES(X) X(16, 1) X(64, 1) X(64, 2) X(256, 1) X(256, 2) X(1024, 1) X(1024, 2)

template <int XF, int RF>
static hipError_t launch_fwd(const NormArgs& a, hipStream_t st) {
  // enough workgroups to fill the chip once; each takes several rows, gamma in registers
  const auto grid = [&](int threads, int rpb) {
    return dim3((unsigned)std::min<int64_t>((a.rows + rpb - 1) / rpb, 256 * (2048 / threads)));
  };
#define FORGE_NORM(LPR, VEC)                                                                           \
  if (a.K >= 8 && a.K <= LPR * VEC * 8) {                                                                          \
    constexpr int T = norm_threads(LPR);                                                               \
    if (a.K % 8 == 0) hipLaunchKernelGGL((k_rmsnorm<XF, RF, LPR, VEC, ROW_WHOLE>), grid(T, T / LPR), dim3(T), 0, st, a); \
    else hipLaunchKernelGGL((k_rmsnorm<XF, RF, LPR, VEC, ROW_BIG>), grid(T, T / LPR), dim3(T), 0, st, a); \
    return hipGetLastError();                                                                          \
  }
  FORGE_NORM_SHAPES(FORGE_NORM)
#undef FORGE_NORM
  hipLaunchKernelGGL((k_rmsnorm_long<XF, RF>), grid(1024, 1), dim3(1024), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t st) {
  if (a.rows == 0 || a.K == 0) return hipSuccess;
  const bool xf = a.x_fmt == FMT_F32;
  if (!a.R) return xf ? launch_fwd<FMT_F32, FMT_NONE>(a, st) : launch_fwd<FMT_BF16, FMT_NONE>(a, st);
  if (a.r_fmt == FMT_F32) return xf ? launch_fwd<FMT_F32, FMT_F32>(a, st) : launch_fwd<FMT_BF16, FMT_F32>(a, st);
  return xf ? launch_fwd<FMT_F32, FMT_BF16>(a, st) : launch_fwd<FMT_BF16, FMT_BF16>(a, st);
}

// Lanes per row of the backward kernel for K columns.
static int norm_bwd_lpr(int64_t K) { return K <= 128 ? 16 : K <= 1024 ? 64 : K <= 4096 ? 256 : 1024; }

int norm_parts(int64_t rows, int64_t K) {
  const int64_t rpb = K < 8 || K > NORM_REG_COLS ? 1 : NB_T / norm_bwd_lpr(K);
  return (int)std::min<int64_t>((rows + rpb - 1) / rpb, NB_PARTS);
}

template <int HF, int DF>
static hipError_t launch_bwd(const NormBwdArgs& a, hipStream_t st) {
  const dim3 grid((unsigned)a.parts), b(NB_T);
#define FORGE_NORM_BWD(LPR, VEC)                                                                         \
  if (a.K >= 8 && a.K <= LPR * VEC * 8) {                                                                            \
    if (a.K % 8 == 0) hipLaunchKernelGGL((k_rmsnorm_backward<HF, DF, LPR, VEC, ROW_WHOLE>), grid, b, 0, st, a); \
    else hipLaunchKernelGGL((k_rmsnorm_backward<HF, DF, LPR, VEC, ROW_BIG>), grid, b, 0, st, a);           \
    return hipGetLastError();                                                                            \
  }
  FORGE_NORM_SHAPES(FORGE_NORM_BWD)
#undef FORGE_NORM_BWD
  hipLaunchKernelGGL((k_rmsnorm_backward_long<HF, DF>), grid, b, 0, st, a);
  return hipGetLastError();
}

hipError_t launch_rmsnorm_backward(const NormBwdArgs& args, hipStream_t st) {
  NormBwdArgs a = args;
  if (a.K == 0) return hipSuccess;
  a.parts = norm_parts(a.rows, a.K);
  if (a.rows > 0) {
    const bool hf = a.h_fmt == FMT_F32, df = a.dy_fmt == FMT_F32;
    const hipError_t e = hf ? (df ? launch_bwd<FMT_F32, FMT_F32>(a, st) : launch_bwd<FMT_F32, FMT_BF16>(a, st))
                            : (df ? launch_bwd<FMT_BF16, FMT_F32>(a, st) : launch_bwd<FMT_BF16, FMT_BF16>(a, st));
    if (e != hipSuccess) return e;
  }
  if (!a.dgamma) return hipSuccess;
  hipLaunchKernelGGL(k_norm_dgamma, dim3((unsigned)std::min<int64_t>(((int64_t)a.K + 63) / 64, 1 << 20)), dim3(NT), 0, st, a);
  return hipGetLastError();
}

}  // namespace forge
