// Embedding lookup, tokens sorted by id, and the gradient of the rows that occur.
#include "forge_act8.h"

#include <algorithm>

namespace forge {

// Token i's row of W: its id, or V (a padding token) where that is outside 0 .. V - 1.
__device__ __forceinline__ int64_t token_row(const void* ids, int id_bytes, int64_t i, int64_t V) {
  const int64_t id = id_bytes == 8 ? static_cast<const int64_t*>(ids)[i] : static_cast<const int32_t*>(ids)[i];
  return (uint64_t)id < (uint64_t)V ? id : V;
}

// ------------------------------------------------------------------------
// Lookup: Y[t] = scale W[ids[t]].  A gather of whole rows: s bytes read and
// written per element, bound by HBM.  Threads map to (token, 8 columns) as in
// the 8-bit copy's kernels; each thread takes EMB_UNR tokens, whose ids and then
// rows are requested together.
// ------------------------------------------------------------------------
constexpr int EMB_UNR = 4;

struct LookupArgs {
  const void* ids; int32_t id_bytes;
  int64_t T, V, K;
  const void* W; int64_t ldw;
  void* Y; int64_t ldy;
  float scale;
  int32_t tsh, segs;
  int64_t units;
};

template <int WF, int YF>
__global__ void __launch_bounds__(NT) k_embed(const LookupArgs a) {
  const int tpr = 1 << a.tsh, rpb = NT >> a.tsh;
  constexpr int ws = WF == FMT_F32 ? 4 : 2, ys = YF == FMT_F32 ? 4 : 2;
  for (int64_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const int64_t rb = unit / a.segs;
    const int seg = (int)(unit - rb * a.segs);
    const int64_t c = ((int64_t)seg * tpr + (threadIdx.x & (tpr - 1))) * 8;
    const int64_t t0 = rb * (rpb * EMB_UNR) + (threadIdx.x >> a.tsh);
    if (c >= a.K) continue;
    int64_t row[EMB_UNR];
#pragma unroll
    for (int u = 0; u < EMB_UNR; ++u) {
      const int64_t t = t0 + (int64_t)u * rpb;
      row[u] = t < a.T ? token_row(a.ids, a.id_bytes, t, a.V) : a.V;
    }
    float x[EMB_UNR][8];
#pragma unroll
    for (int u = 0; u < EMB_UNR; ++u)
      row_load8<WF>(static_cast<const char*>(a.W) + row[u] * a.ldw * ws, c, row[u] < a.V ? a.K : 0, x[u]);
#pragma unroll
    for (int u = 0; u < EMB_UNR; ++u) {
      const int64_t t = t0 + (int64_t)u * rpb;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[u][e] = row[u] < a.V ? x[u][e] * a.scale : 0.f;
      if (t < a.T) row_store8<YF>(static_cast<char*>(a.Y) + t * a.ldy * ys, c, a.K, x[u]);
    }
  }
}

hipError_t launch_embed(const void* ids, int id_bytes, int64_t T, const void* W, int64_t ldw, int w_fmt, int64_t V,
                        int64_t K, float scale, void* Y, int64_t ldy, int y_fmt, hipStream_t st) {
  if (T == 0 || K == 0) return hipSuccess;
  LookupArgs a{ids, id_bytes, T, V, K, W, ldw, Y, ldy, scale, 0, 0, 0};
  const int64_t lanes = (K + 7) / 8;
  a.tsh = 0;
  while (a.tsh < 8 && (1 << a.tsh) < lanes) ++a.tsh;
  a.segs = (int32_t)((lanes + (1 << a.tsh) - 1) >> a.tsh);
  const int64_t rpb = (int64_t)(NT >> a.tsh) * EMB_UNR;
  a.units = ((T + rpb - 1) / rpb) * a.segs;
  const dim3 grid((unsigned)std::min<int64_t>(a.units, 1 << 22)), b(NT);
  const bool wf = w_fmt == FMT_F32, yf = y_fmt == FMT_F32;
  if (wf && yf) hipLaunchKernelGGL((k_embed<FMT_F32, FMT_F32>), grid, b, 0, st, a);
  else if (wf) hipLaunchKernelGGL((k_embed<FMT_F32, FMT_BF16>), grid, b, 0, st, a);
  else if (yf) hipLaunchKernelGGL((k_embed<FMT_BF16, FMT_F32>), grid, b, 0, st, a);
  else hipLaunchKernelGGL((k_embed<FMT_BF16, FMT_BF16>), grid, b, 0, st, a);
  return hipGetLastError();
}

// ------------------------------------------------------------------------
// Tokens sorted by id, stable, in two launches and without atomics:
//  k_embed_parts sorts each part of PART tokens in LDS (bitonic, on the pairs
//    (row, index), which are all different, so the order is that of a stable
//    sort), and zeroes start / end;
//  k_embed_ranks gives every token its place: its place in its own part, plus
//    for every earlier part the number of tokens with a row <= its own, for every
//    later part of those with a smaller row (binary searches), and marks where
//    each row begins and ends.
// Work: T log^2 PART in LDS, then T (T / PART) log PART reads of L2; larger parts
// where there are many tokens keep the second term short.
// ------------------------------------------------------------------------
template <int PART>
__global__ void __launch_bounds__(1024) k_embed_parts(const EmbedArgs e) {
  __shared__ uint64_t s[PART];
  const int64_t n0 = (int64_t)blockIdx.x * PART;
  if (n0 < e.T) {
    for (int i = threadIdx.x; i < PART; i += 1024) {
      const int64_t t = n0 + i;
      s[i] = t < e.T ? ((uint64_t)token_row(e.ids, e.id_bytes, t, e.V) << 32) | (uint64_t)t : ~0ull;
    }
    __syncthreads();
    for (int k = 2; k <= PART; k <<= 1)
      for (int j = k >> 1; j > 0; j >>= 1) {
        for (int i = threadIdx.x; i < PART / 2; i += 1024) {
          const int lo = 2 * i - (i & (j - 1)), hi = lo + j;   // i's bits with a 0 put in at j
          const uint64_t x = s[lo], y = s[hi];
          const bool up = (lo & k) == 0;
          if ((x > y) == up) { s[lo] = y; s[hi] = x; }
        }
        __syncthreads();
      }
    for (int i = threadIdx.x; i < PART; i += 1024)
      if (n0 + i < e.T) e.part[n0 + i] = s[i];
  }
  for (int64_t v = (int64_t)blockIdx.x * 1024 + threadIdx.x; v <= e.V; v += (int64_t)gridDim.x * 1024) {
    e.start[v] = 0;
    e.end[v] = 0;
  }
}

// First place in the sorted a[0 .. n) whose row is >= r.
__device__ __forceinline__ int part_lower(const uint64_t* a, int n, uint64_t r) {
  int lo = 0;
  while (n > 0) {
    const int h = n >> 1;
    const bool less = (a[lo + h] >> 32) < r;
    lo = less ? lo + h + 1 : lo;
    n = less ? n - h - 1 : h;
  }
  return lo;
}

__global__ void __launch_bounds__(NT) k_embed_ranks(const EmbedArgs e, int part) {
  const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (i >= e.T) return;
  const uint64_t x = e.part[i], row = x >> 32;
  const int64_t own = i / part;
  int64_t rank = i - own * part;
  bool first = rank == 0 || (e.part[i - 1] >> 32) != row;
  bool last = i + 1 >= min(e.T, (own + 1) * part) || (e.part[i + 1] >> 32) != row;
  for (int64_t b = 0, n0 = 0; n0 < e.T; ++b, n0 += part) {
    if (b == own) continue;
    const int n = (int)min((int64_t)part, e.T - n0);
    const uint64_t* p = e.part + n0;
    if (b < own) {
      const int u = part_lower(p, n, row + 1);
      rank += u;
      first = first && !(u > 0 && (p[u - 1] >> 32) == row);
    } else {
      const int l = part_lower(p, n, row);
      rank += l;
      last = last && !(l < n && (p[l] >> 32) == row);
    }
  }
  e.key[rank] = (int32_t)row;
  e.perm[rank] = (int32_t)(x & 0xFFFFFFFFu);
  if (first) e.start[row] = (int32_t)rank;
  if (last) e.end[row] = (int32_t)rank + 1;
}

hipError_t launch_embed_sort(const EmbedArgs& e, hipStream_t st) {
  const int64_t part = embed_part(e.T);
  const int64_t parts = (e.T + part - 1) / part;
  // at least one workgroup per 64 Ki entries of start / end
  const unsigned grid = (unsigned)std::max<int64_t>(parts, std::min<int64_t>(256, e.V / 65536 + 1));
  if (part == 2048) hipLaunchKernelGGL((k_embed_parts<2048>), dim3(grid), dim3(1024), 0, st, e);
  else hipLaunchKernelGGL((k_embed_parts<8192>), dim3(grid), dim3(1024), 0, st, e);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess || e.T == 0) return err;
  hipLaunchKernelGGL(k_embed_ranks, dim3((unsigned)((e.T + NT - 1) / NT)), dim3(NT), 0, st, e, (int)part);
  return hipGetLastError();
}

// ------------------------------------------------------------------------
// acc[v] (+)= scale sum of dY over the tokens of v, for the rows that occur: a
// workgroup per (sorted place, 128 columns) that works where its place begins a
// row.  16 lanes of 8 columns by 16 tokens at a time; the 16 sums are added in a
// fixed order.
// ------------------------------------------------------------------------
template <int DF>
__global__ void __launch_bounds__(NT) k_embed_rows(const EmbedArgs e, float* acc, int64_t ldacc, int add) {
  __shared__ float sum[16][TILE + 4];
  const int64_t segs = (e.K + TILE - 1) / TILE;
  constexpr int ds = DF == FMT_F32 ? 4 : 2;
  const int cl = 8 * (threadIdx.x & 15), slot = threadIdx.x >> 4;
  for (int64_t unit = blockIdx.x; unit < e.T * segs; unit += gridDim.x) {
    const int64_t p = unit / segs, c0 = (unit - p * segs) * TILE, c = c0 + cl;
    const int v = e.key[p];
    if (v >= e.V || e.start[v] != p) continue;
    const int n = e.end[v];
    float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int64_t i = p + slot; i < n; i += 16) {
      float x[8];
      row_load8<DF>(static_cast<const char*>(e.dY) + (int64_t)e.perm[i] * e.lddy * ds, c, e.K, x);
#pragma unroll
      for (int k = 0; k < 8; ++k) s[k] += x[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[slot][cl + k] = s[k];
    __syncthreads();
    const int64_t q = c0 + threadIdx.x;
    if (threadIdx.x < TILE && q < e.K) {
      float g = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) g += sum[k][threadIdx.x];
      float* o = acc + (int64_t)v * ldacc + q;
      g *= e.scale;
      *o = add ? *o + g : g;
    }
  }
}

// Zero rows of an fp32 matrix.
__global__ void __launch_bounds__(NT) k_embed_zero(float* acc, int64_t ld, int64_t V, int64_t K) {
  const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t v = blockIdx.x; v < V; v += gridDim.x)
    for (int64_t c = (int64_t)threadIdx.x * 8; c < K; c += NT * 8) row_store8<FMT_F32>(acc + v * ld, c, K, z);
}

hipError_t launch_embed_accumulate(const EmbedArgs& e, float* acc, int64_t ldacc, bool first, hipStream_t st) {
  if (e.V == 0 || e.K == 0) return hipSuccess;
  if (first) {
    hipLaunchKernelGGL(k_embed_zero, dim3((unsigned)std::min<int64_t>(e.V, 1 << 20)), dim3(NT), 0, st, acc, ldacc, e.V,
                       e.K);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (e.T == 0) return hipSuccess;
  hipError_t err = launch_embed_sort(e, st);
  if (err != hipSuccess) return err;
  const int64_t units = e.T * ((e.K + TILE - 1) / TILE);
  const dim3 grid((unsigned)std::min<int64_t>(units, 1 << 22));
  if (e.dy_fmt == FMT_F32) hipLaunchKernelGGL((k_embed_rows<FMT_F32>), grid, dim3(NT), 0, st, e, acc, ldacc, first ? 0 : 1);
  else hipLaunchKernelGGL((k_embed_rows<FMT_BF16>), grid, dim3(NT), 0, st, e, acc, ldacc, first ? 0 : 1);
  return hipGetLastError();
}

hipError_t launch_embed_step(const KArgs& a, const EmbedArgs& e, int w_fmt, int opt, int m_fmt, int v_fmt,
                             hipStream_t st) {
  const hipError_t err = launch_embed_sort(e, st);
  if (err != hipSuccess) return err;
#define X(O, M, V) \
  if (opt == O && m_fmt == M && v_fmt == V) return combo_embed<O, M, V>(a, e, w_fmt, st);
  FORGE_STATE_LIST(X)
#undef X
  return hipErrorInvalidValue;
}

}  // namespace forge
