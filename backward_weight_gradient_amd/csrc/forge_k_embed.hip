// Embedding lookup, tokens sorted by id, and the gradient of the rows that occur.
#include "forge_act8.h"

#include <algorithm>

namespace forge {

// An id as a row of W: V (a padding token) where it is outside 0 .. V - 1.
__device__ __forceinline__ int64_t id_row(int64_t id, int64_t V) { return (uint64_t)id < (uint64_t)V ? id : V; }

// N ids at places at(u) (all in range), requested together: one branch for all of them.
template <int N, class F>
__device__ __forceinline__ void load_ids(const void* ids, int id_bytes, F&& at, int64_t (&id)[N]) {
  if (id_bytes == 8) {
#pragma unroll
    for (int u = 0; u < N; ++u) id[u] = static_cast<const int64_t*>(ids)[at(u)];
  } else {
#pragma unroll
    for (int u = 0; u < N; ++u) id[u] = static_cast<const int32_t*>(ids)[at(u)];
  }
}

// Zero a matrix of format fmt.
__global__ void __launch_bounds__(NT) k_zero_rows(void* p, int64_t ld, int fmt, int64_t rows, int64_t K) {
  const float z[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
    for (int64_t c = (int64_t)threadIdx.x * 8; c < K; c += NT * 8) {
      if (fmt == FMT_F32) row_store8<FMT_F32>(static_cast<float*>(p) + r * ld, c, K, z);
      else row_store8<FMT_BF16>(static_cast<uint16_t*>(p) + r * ld, c, K, z);
    }
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

template <int MODE, int WF, int YF>
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
    load_ids(a.ids, a.id_bytes, [&](int u) { return min(t0 + (int64_t)u * rpb, a.T - 1); }, row);
    Raw8<WF> w[EMB_UNR];
#pragma unroll
    for (int u = 0; u < EMB_UNR; ++u) {
      row[u] = id_row(row[u], a.V);
      // (padding reads row 0 and is cleared)
      w[u] = row_raw8<WF, MODE>(static_cast<const char*>(a.W) + (row[u] < a.V ? row[u] : 0) * a.ldw * ws, c, a.K);
    }
#pragma unroll
    for (int u = 0; u < EMB_UNR; ++u) {
      const int64_t t = t0 + (int64_t)u * rpb;
      float x[8];
      row_val8<WF, MODE>(w[u], c, a.K, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = row[u] < a.V ? x[e] * a.scale : 0.f;
      if (t < a.T) row_store8<YF>(static_cast<char*>(a.Y) + t * a.ldy * ys, c, a.K, x);
    }
  }
}

hipError_t launch_embed(const void* ids, int id_bytes, int64_t T, const void* W, int64_t ldw, int w_fmt, int64_t V,
                        int64_t K, float scale, void* Y, int64_t ldy, int y_fmt, hipStream_t st) {
  if (T == 0 || K == 0) return hipSuccess;
  if (V == 0) {   // nothing but padding
    hipLaunchKernelGGL(k_zero_rows, dim3((unsigned)std::min<int64_t>(T, 1 << 20)), dim3(NT), 0, st, Y, ldy, y_fmt, T, K);
    return hipGetLastError();
  }
  LookupArgs a{ids, id_bytes, T, V, K, W, ldw, Y, ldy, scale, 0, 0, 0};
  const int64_t lanes = (K + 7) / 8;
  a.tsh = 0;
  while (a.tsh < 8 && (1 << a.tsh) < lanes) ++a.tsh;
  a.segs = (int32_t)((lanes + (1 << a.tsh) - 1) >> a.tsh);
  const int64_t rpb = (int64_t)(NT >> a.tsh) * EMB_UNR;
  a.units = ((T + rpb - 1) / rpb) * a.segs;
  const dim3 grid((unsigned)std::min<int64_t>(a.units, 1 << 22)), b(NT);
  const bool wf = w_fmt == FMT_F32, yf = y_fmt == FMT_F32;
#define FORGE_LOOKUP(MODE)                                                                        \
  if (wf && yf) hipLaunchKernelGGL((k_embed<MODE, FMT_F32, FMT_F32>), grid, b, 0, st, a);         \
  else if (wf) hipLaunchKernelGGL((k_embed<MODE, FMT_F32, FMT_BF16>), grid, b, 0, st, a);         \
  else if (yf) hipLaunchKernelGGL((k_embed<MODE, FMT_BF16, FMT_F32>), grid, b, 0, st, a);         \
  else hipLaunchKernelGGL((k_embed<MODE, FMT_BF16, FMT_BF16>), grid, b, 0, st, a);                \
  return hipGetLastError();
  if (K >= 8) { FORGE_LOOKUP(ROW_BIG) }
  FORGE_LOOKUP(ROW_ANY)
#undef FORGE_LOOKUP
}

// ------------------------------------------------------------------------
// Tokens sorted by id, stable, without atomics.
//  k_embed_place: each token's place within its part of EMBED_PART tokens, by
//    counting: place(i) = #{j: row_j < row_i} + #{j < i: row_j = row_i}.  A workgroup
//    places 16 tokens against the whole part in LDS, 16 threads a token; two
//    instructions a pair.  Quadratic, but spread over the whole chip: 8192 tokens
//    are 67 M pairs.
//  k_embed_ranks (more than one part): a token's place in its own part, plus for
//    every earlier part the number of tokens with a row <= its own, for every later
//    part of those with a smaller row (binary searches).
// ------------------------------------------------------------------------
constexpr int PLACE_TOKENS = 16;

__global__ void __launch_bounds__(NT) k_embed_place(const EmbedArgs e, int one_part) {
  __shared__ __attribute__((aligned(16))) uint32_t row[EMBED_PART];
  __shared__ int sums[4][PLACE_TOKENS];
  constexpr int per_part = EMBED_PART / PLACE_TOKENS;
  const int64_t n0 = (int64_t)(blockIdx.x / per_part) * EMBED_PART;
  const int i0 = (int)(blockIdx.x % per_part) * PLACE_TOKENS;       // first token, within the part
  const int n = (int)min((int64_t)EMBED_PART, e.T - n0);
  if (i0 >= n) return;
  const int n64 = (n + 63) & ~63;
  for (int b = threadIdx.x; b < n64; b += 8 * NT) {
    int64_t id[8];
    load_ids(e.ids, e.id_bytes, [&](int u) { return n0 + min(b + u * NT, n - 1); }, id);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = b + u * NT;
      if (i < n64) row[i] = i < n ? (uint32_t)id_row(id[u], e.V) : 0xFFFFFFFFu;   // past the end: never smaller
    }
  }
  __syncthreads();
  const int sub = threadIdx.x >> 4, i = i0 + (threadIdx.x & 15);    // 16 subsets of the part by 16 tokens
  const uint32_t own = i < n ? row[i] : 0u;
  int count = 0;
#pragma unroll 4
  for (int j0 = 0; j0 < n64; j0 += 64) {
    const int j = j0 + 4 * sub;
    const u32x4 r = *reinterpret_cast<const u32x4*>(row + j);
    if (j0 + 64 <= i0 || j0 >= i0 + PLACE_TOKENS) {
      // all of these come before every token of the workgroup, or all after
      const uint32_t lim = own + (j0 < i0 ? 1u : 0u);
#pragma unroll
      for (int k = 0; k < 4; ++k) count += r[k] < lim ? 1 : 0;
    } else {
#pragma unroll
      for (int k = 0; k < 4; ++k) count += r[k] < own + (j + k < i ? 1u : 0u) ? 1 : 0;
    }
  }
  count += __shfl_xor(count, 16);
  count += __shfl_xor(count, 32);
  if ((threadIdx.x & 63) < PLACE_TOKENS) sums[threadIdx.x >> 6][threadIdx.x & 15] = count;
  __syncthreads();
  if (threadIdx.x < PLACE_TOKENS && i < n) {
    const int64_t at = n0 + sums[0][threadIdx.x] + sums[1][threadIdx.x] + sums[2][threadIdx.x] + sums[3][threadIdx.x];
    if (one_part) {
      e.key[at] = (int32_t)own;
      e.perm[at] = i;
    } else {
      e.part[at] = ((uint64_t)own << 32) | (uint64_t)(n0 + i);
    }
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

__global__ void __launch_bounds__(NT) k_embed_ranks(const EmbedArgs e) {
  const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (i >= e.T) return;
  const uint64_t x = e.part[i], row = x >> 32;
  const int64_t own = i / EMBED_PART;
  int64_t rank = i - own * EMBED_PART;
  for (int64_t b = 0, n0 = 0; n0 < e.T; ++b, n0 += EMBED_PART) {
    if (b == own) continue;
    rank += part_lower(e.part + n0, (int)min((int64_t)EMBED_PART, e.T - n0), b < own ? row + 1 : row);
  }
  e.key[rank] = (int32_t)row;
  e.perm[rank] = (int32_t)(x & 0xFFFFFFFFu);
}

hipError_t launch_embed_sort(const EmbedArgs& e, hipStream_t st) {
  if (e.T == 0) return hipSuccess;
  const int64_t parts = (e.T + EMBED_PART - 1) / EMBED_PART;
  const int64_t last = e.T - (parts - 1) * EMBED_PART;
  const unsigned grid =
      (unsigned)((parts - 1) * (EMBED_PART / PLACE_TOKENS) + (last + PLACE_TOKENS - 1) / PLACE_TOKENS);
  hipLaunchKernelGGL(k_embed_place, dim3(grid), dim3(NT), 0, st, e, parts == 1 ? 1 : 0);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || parts == 1) return err;
  hipLaunchKernelGGL(k_embed_ranks, dim3((unsigned)((e.T + NT - 1) / NT)), dim3(NT), 0, st, e);
  return hipGetLastError();
}

// ------------------------------------------------------------------------
// acc[v] (+)= scale sum of dY over the tokens of v, for the rows that occur.  The
// first `longs` workgroups take the rows of more than ROW_LONG tokens: such a run
// of the sorted tokens holds a place that is a multiple of ROW_LONG, and the first
// of those (with each 64 columns of the row) is its unit of work: 32 tokens at a
// time, 8 lanes of 8 columns each.  The other workgroups take the short rows: a
// wave per (place that begins a row, ROW_COLS columns), the tokens in order.
// Every sum has a fixed order.
// ------------------------------------------------------------------------
constexpr int ROW_LONG = 32, ROW_COLS = 512, ROW_SEG = 64;

// End of the run of row v that place p belongs to (keys past the end differ); all
// lanes of the wave.  64 places in steps of `step`, then 64 in steps of one: two
// reads find the end of a run of up to 64 step.
__device__ __forceinline__ int64_t run_end(const EmbedArgs& e, int64_t p, int v, int step) {
  const int lane = threadIdx.x & 63;
  const auto first_other = [&](int64_t at, int64_t by) {   // the first lane whose place is not in the run (64: none)
    const int64_t i = at + lane * by;
    const uint64_t m = __ballot(i >= e.T || e.key[i] != v);
    return m ? __builtin_ctzll(m) : 64;
  };
  while (step > 1) {
    const int k = first_other(p, step);
    p += (int64_t)(k - 1) * step;       // the last place seen inside the run (k > 0: p itself is)
    if (k < 64) break;
  }
  for (;;) {
    const int k = first_other(p, 1);
    p += k;
    if (k < 64) return p;
  }
}

constexpr int ROW_PERM = 1024;          // tokens of a long row staged in LDS at a time

template <int MODE, int DF>
__device__ __forceinline__ void rows_long(const EmbedArgs& e, float* acc, int64_t ldacc, int add, int64_t unit, int64_t segs,
                                          float (&sum)[4][ROW_SEG], int32_t (&tok)[ROW_PERM]) {
  constexpr int ds = DF == FMT_F32 ? 4 : 2;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t p = unit / segs * ROW_LONG, c = unit % segs * ROW_SEG + 8 * (lane & 7);
  const int v = e.key[p];
  if (v >= e.V || (p > 0 && e.key[p - ROW_LONG] == v)) return;      // padding, or an earlier multiple owns the run
  const int64_t q = p - (lane & (ROW_LONG - 1));                    // p, p - 1, .. p - 31
  const uint64_t before = __ballot(q < 0 || e.key[q < 0 ? 0 : q] != v) & 0xFFFFFFFFull;
  const int64_t first = p - (before ? __builtin_ctzll(before) : ROW_LONG) + 1;
  const int64_t end = run_end(e, p, v, 64);
  if (end - first <= ROW_LONG) return;
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const int slot = wave * 8 + (lane >> 3);
  for (int64_t b = first; b < end; b += ROW_PERM) {
    const int n = (int)min((int64_t)ROW_PERM, end - b);
    __syncthreads();                                                // the tokens staged before are read
    for (int i = threadIdx.x; i < n; i += NT) tok[i] = e.perm[b + i];
    __syncthreads();
    const auto at = [&](int i) {
      return static_cast<const char*>(e.dY) + (int64_t)tok[min(slot + 32 * i, n - 1)] * e.lddy * ds;
    };
    sum_rows<MODE, DF>(at, (n + 31) / 32, (n - slot + 31) / 32, c, e.K, s);
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s[k] += __shfl_xor(s[k], 8);
    s[k] += __shfl_xor(s[k], 16);
    s[k] += __shfl_xor(s[k], 32);
  }
  if (lane < 8) {                                                   // (the last unit's sums were read before the barriers above)
#pragma unroll
    for (int k = 0; k < 8; ++k) sum[wave][8 * lane + k] = s[k];
  }
  __syncthreads();
  const int64_t col = unit % segs * ROW_SEG + threadIdx.x;
  if (threadIdx.x < ROW_SEG && col < e.K) {
    const float g = (((sum[0][threadIdx.x] + sum[1][threadIdx.x]) + sum[2][threadIdx.x]) + sum[3][threadIdx.x]) * e.scale;
    float* o = acc + (int64_t)v * ldacc + col;
    *o = add ? *o + g : g;
  }
}

template <int MODE, int DF>
__device__ __forceinline__ void rows_short(const EmbedArgs& e, float* acc, int64_t ldacc, int add, int64_t p, int64_t c0) {
  constexpr int ds = DF == FMT_F32 ? 4 : 2;
  const int lane = threadIdx.x & 63;
  const int v = e.key[p];
  if (v >= e.V || (p > 0 && e.key[p - 1] == v)) return;
  const int n = (int)min((int64_t)(ROW_LONG + 1), run_end(e, p, v, 1) - p);
  if (n > ROW_LONG) return;
  const int tok = lane < n ? e.perm[p + lane] : 0;
  static_assert(ROW_COLS == 64 * 8, "a wave's columns");
  const int64_t c = c0 + 8 * lane;
  float* o = acc + (int64_t)v * ldacc;
  Raw8<FMT_F32> old;
  if (add) old = row_raw8<FMT_F32, MODE>(o, c, e.K);
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  const auto at = [&](int i) {
    return static_cast<const char*>(e.dY) + (int64_t)__builtin_amdgcn_readlane(tok, min(i, n - 1)) * e.lddy * ds;
  };
  sum_rows<MODE, DF>(at, n, n, c, e.K, s);
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] *= e.scale;
  if (add) {
    float x[8];
    row_val8<FMT_F32, MODE>(old, c, e.K, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = x[k] + s[k];
  }
  row_store8<FMT_F32>(o, c, e.K, s);
}

template <int MODE, int DF>
__global__ void __launch_bounds__(NT) k_embed_rows(const EmbedArgs e, float* acc, int64_t ldacc, int add, int longs) {
  __shared__ float sum[4][ROW_SEG];
  __shared__ int32_t tok[ROW_PERM];
  if ((int)blockIdx.x < longs) {
    const int64_t segs = (e.K + ROW_SEG - 1) / ROW_SEG, units = (e.T + ROW_LONG - 1) / ROW_LONG * segs;
    for (int64_t u = blockIdx.x; u < units; u += longs) rows_long<MODE, DF>(e, acc, ldacc, add, u, segs, sum, tok);
  } else {
    const int64_t groups = (e.K + ROW_COLS - 1) / ROW_COLS;
    const int64_t stride = (int64_t)(gridDim.x - longs) * 4;
    for (int64_t u = ((int64_t)blockIdx.x - longs) * 4 + (threadIdx.x >> 6); u < e.T * groups; u += stride)
      rows_short<MODE, DF>(e, acc, ldacc, add, u / groups, u % groups * ROW_COLS);
  }
}

hipError_t launch_embed_accumulate(const EmbedArgs& e, float* acc, int64_t ldacc, bool first, hipStream_t st) {
  if (e.V == 0 || e.K == 0) return hipSuccess;
  if (first) {
    hipLaunchKernelGGL(k_zero_rows, dim3((unsigned)std::min<int64_t>(e.V, 1 << 20)), dim3(NT), 0, st, acc, ldacc,
                       (int)FMT_F32, e.V, e.K);
    const hipError_t err = hipGetLastError();
    if (err != hipSuccess) return err;
  }
  if (e.T == 0) return hipSuccess;
  const hipError_t err = launch_embed_sort(e, st);
  if (err != hipSuccess) return err;
  const int64_t long_units = e.T > ROW_LONG ? (e.T + ROW_LONG - 1) / ROW_LONG * ((e.K + ROW_SEG - 1) / ROW_SEG) : 0;
  const int64_t shorts = (e.T * ((e.K + ROW_COLS - 1) / ROW_COLS) + 3) / 4;
  const int longs = (int)std::min<int64_t>(long_units, 2048);
  const dim3 grid((unsigned)(longs + std::min<int64_t>(shorts, 1 << 20)));
#define FORGE_ROWS(MODE)                                                                                                        \
  if (e.dy_fmt == FMT_F32)                                                                                                      \
    hipLaunchKernelGGL((k_embed_rows<MODE, FMT_F32>), grid, dim3(NT), 0, st, e, acc, ldacc, first ? 0 : 1, longs);              \
  else hipLaunchKernelGGL((k_embed_rows<MODE, FMT_BF16>), grid, dim3(NT), 0, st, e, acc, ldacc, first ? 0 : 1, longs);          \
  return hipGetLastError();
  if (e.K >= 8) { FORGE_ROWS(ROW_BIG) }
  FORGE_ROWS(ROW_ANY)
#undef FORGE_ROWS
}

// tile[i] = the first place whose row is >= i * rows, for i = 0 .. tiles (the step's
// row tiles and the end of the last).
__global__ void __launch_bounds__(NT) k_embed_tiles(const EmbedArgs e, int64_t rows, int64_t tiles) {
  const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (i > tiles) return;
  const int64_t r = min(i * rows, e.V);
  int64_t lo = 0, n = e.T;
  while (n > 0) {
    const int64_t h = n >> 1;
    const bool less = e.key[lo + h] < r;
    lo = less ? lo + h + 1 : lo;
    n = less ? n - h - 1 : h;
  }
  e.tile[i] = (int32_t)lo;
}

hipError_t launch_embed_tiles(const EmbedArgs& e, int64_t rows, int64_t tiles, hipStream_t st) {
  hipLaunchKernelGGL(k_embed_tiles, dim3((unsigned)(tiles / NT + 1)), dim3(NT), 0, st, e, rows, tiles);
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
