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

// Lanes of `each` columns that a row is spread over, as a power of two, at most 2^most.
inline int lane_shift(int64_t K, int each, int most) {
  int sh = 0;
  while (sh < most && ((int64_t)each << sh) < K) ++sh;
  return sh;
}

// Zero rows x K of format FMT: workgroup wg of wgs, each of nt threads, a row to 1 << sh
// of them.  Bound by HBM; past the caches 128256 x 4096 fp32 are cleared at 6 TB/s
// (through them at 5).
struct ZeroArgs {
  void* p; int64_t ld, rows, K;
  int32_t sh;
};
template <int FMT>
__device__ __forceinline__ void zero_rows(const ZeroArgs& z, int64_t wg, int64_t wgs, int nt) {
  using E = std::conditional_t<FMT == FMT_F32, float, uint16_t>;
  using E4 = std::conditional_t<FMT == FMT_F32, f32x4_e, u32x2_e>;
  const int per = nt >> z.sh;
  for (int64_t r = wg * per + (threadIdx.x >> z.sh); r < z.rows; r += wgs * per) {
    E* p = static_cast<E*>(z.p) + r * z.ld;
    for (int64_t c = (int64_t)(threadIdx.x & ((1 << z.sh) - 1)) * 4; c < z.K; c += (int64_t)4 << z.sh) {
      if (c + 4 <= z.K) __builtin_nontemporal_store(E4{}, reinterpret_cast<E4*>(p + c));
      else for (int64_t k = c; k < z.K; ++k) p[k] = E(0);
    }
  }
}
template <int FMT>
__global__ void __launch_bounds__(NT) k_zero_rows(const ZeroArgs z) {
  zero_rows<FMT>(z, blockIdx.x, gridDim.x, NT);
}

// ------------------------------------------------------------------------
// Lookup: Y[t] = scale W[ids[t]].  A gather of whole rows: s bytes read and
// written per element, bound by HBM.  Threads map to (token, 8 columns) as in
// the 8-bit copy's kernels; each thread takes EMB_UNR tokens, whose ids and then
// rows are requested together.  8192 tokens of 128256 x 4096 bf16: 19 us (134 MB,
// 7 TB/s).
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
  const int sh = lane_shift(K, 8, 8), rows = NT >> sh;      // rows of a workgroup
  if (V == 0) {   // nothing but padding
    const ZeroArgs z{Y, ldy, T, K, sh};
    const dim3 g((unsigned)std::min<int64_t>((T + rows - 1) / rows, 1 << 20));
    if (y_fmt == FMT_F32) hipLaunchKernelGGL(k_zero_rows<FMT_F32>, g, dim3(NT), 0, st, z);
    else hipLaunchKernelGGL(k_zero_rows<FMT_BF16>, g, dim3(NT), 0, st, z);
    return hipGetLastError();
  }
  const int64_t segs = (K + ((int64_t)8 << sh) - 1) >> (sh + 3), per = (int64_t)rows * EMB_UNR;
  const LookupArgs a{ids, id_bytes, T, V, K, W, ldw, Y, ldy, scale, sh, (int32_t)segs, (T + per - 1) / per * segs};
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
//    places 32 tokens against the whole part in LDS, 64 threads of a column of 16
//    for each two; two instructions a pair.  Quadratic, but spread over the whole
//    chip: the 67 M pairs of 8192 tokens take 10 us, 5000 tokens 7 us (4 waves a
//    workgroup instead of 16: 15 and 13 us, one wave a SIMD hides nothing).  Where
//    the step's row tiles begin is counted in the same way (bound workgroups), and
//    the accumulator is cleared meanwhile (zero workgroups).
//  k_embed_ranks (more than one part): a token's place in its own part, plus for
//    every earlier part the number of tokens with a row <= its own, for every later
//    part of those with a smaller row (binary searches); the bounds likewise.
// ------------------------------------------------------------------------
constexpr int PLACE_TOKENS = 32;     // 2 per thread: an LDS read serves two counts
constexpr int PLACE_NT = 1024, PLACE_WAVES = PLACE_NT / 64, PLACE_STEP = 4 * PLACE_NT / 16;
constexpr int64_t PLACE_ZERO_WGS = 1 << 20;   // most workgroups that clear
static_assert((EMBED_MAX_TOKENS / PLACE_TOKENS + EMBED_MAX_TILES / PLACE_TOKENS + 1 + PLACE_ZERO_WGS) * PLACE_NT < (1ll << 32),
              "fewer than 2^32 threads");

// bounds: tile[i] = the first place whose row is >= i * EMBED_ROWS, for i = 0 .. bounds - 1.
struct SortArgs {
  EmbedArgs e;
  int64_t bounds;
  ZeroArgs zero;
  int32_t place_wgs, bound_wgs, parts;
};

__global__ void __launch_bounds__(PLACE_NT) k_embed_place(const SortArgs a) {
  __shared__ __attribute__((aligned(16))) uint32_t row[EMBED_PART];
  __shared__ int sums[PLACE_WAVES][PLACE_TOKENS];
  const EmbedArgs& e = a.e;
  const int wg = (int)blockIdx.x - a.place_wgs;                     // < 0: places tokens
  if (wg >= a.bound_wgs) {
    zero_rows<FMT_F32>(a.zero, wg - a.bound_wgs, (int64_t)gridDim.x - a.place_wgs - a.bound_wgs, PLACE_NT);
    return;
  }
  constexpr int per_part = EMBED_PART / PLACE_TOKENS;
  const int64_t n0 = wg < 0 ? (int64_t)(blockIdx.x / per_part) * EMBED_PART : 0;
  const int i0 = wg < 0 ? (int)(blockIdx.x % per_part) * PLACE_TOKENS : EMBED_PART;   // first token, within the part
  const int n = (int)min((int64_t)EMBED_PART, e.T - n0);
  const int all = (n + PLACE_STEP - 1) & ~(PLACE_STEP - 1);
  for (int b = threadIdx.x; b < all; b += 8 * PLACE_NT) {
    int64_t id[8];
    load_ids(e.ids, e.id_bytes, [&](int u) { return n0 + min(b + u * PLACE_NT, n - 1); }, id);
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = b + u * PLACE_NT;
      if (i < all) row[i] = i < n ? (uint32_t)id_row(id[u], e.V) : 0xFFFFFFFFu;   // past the end: never smaller
    }
  }
  __syncthreads();
  const int sub = threadIdx.x >> 4;                                 // 64 subsets of the part by 16 pairs of tokens
  int i[2], count[2] = {0, 0};
  uint32_t own[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = 16 * h + (threadIdx.x & 15);
    i[h] = i0 + k;
    own[h] = wg < 0 ? row[min(i[h], n - 1)] : (uint32_t)min(((int64_t)wg * PLACE_TOKENS + k) * EMBED_ROWS, e.V);
  }
#pragma unroll 4
  for (int j0 = 0; j0 < all; j0 += PLACE_STEP) {
    const int j = j0 + 4 * sub;
    const u32x4 r = *reinterpret_cast<const u32x4*>(row + j);
    if (wg >= 0 || j0 + PLACE_STEP <= i0 || j0 >= i0 + PLACE_TOKENS) {
      // all of these come before every token of the workgroup, or all after
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t lim = own[h] + (wg < 0 && j0 < i0 ? 1u : 0u);
#pragma unroll
        for (int k = 0; k < 4; ++k) count[h] += r[k] < lim ? 1 : 0;
      }
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int k = 0; k < 4; ++k) count[h] += r[k] < own[h] + (j + k < i[h] ? 1u : 0u) ? 1 : 0;
    }
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    count[h] += __shfl_xor(count[h], 16);
    count[h] += __shfl_xor(count[h], 32);
    if ((threadIdx.x & 63) < 16) sums[threadIdx.x >> 6][16 * h + (threadIdx.x & 15)] = count[h];
  }
  __syncthreads();
  if (threadIdx.x >= PLACE_TOKENS) return;
  int at = 0;
#pragma unroll
  for (int w = 0; w < PLACE_WAVES; ++w) at += sums[w][threadIdx.x];
  if (wg >= 0) {
    const int64_t k = (int64_t)wg * PLACE_TOKENS + threadIdx.x;
    if (k < a.bounds) e.tile[k] = at;
    return;
  }
  const int t = i0 + threadIdx.x;
  if (t >= n) return;
  const uint32_t v = row[t];
  if (a.parts == 1) {
    e.key[at] = (int32_t)v;
    e.perm[at] = t;
  } else {
    e.part[n0 + at] = ((uint64_t)v << 32) | (uint64_t)(n0 + t);
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

__global__ void __launch_bounds__(NT) k_embed_ranks(const SortArgs a) {
  const EmbedArgs& e = a.e;
  const int64_t i = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (i >= e.T + a.bounds) return;
  const bool token = i < e.T;
  const uint64_t x = token ? e.part[i] : 0;
  const uint64_t row = token ? x >> 32 : (uint64_t)min((i - e.T) * EMBED_ROWS, e.V);
  const int64_t own = token ? i / EMBED_PART : -1;
  int64_t rank = token ? i - own * EMBED_PART : 0;
  for (int64_t b = 0, n0 = 0; n0 < e.T; ++b, n0 += EMBED_PART) {
    if (b == own) continue;
    rank += part_lower(e.part + n0, (int)min((int64_t)EMBED_PART, e.T - n0), b < own ? row + 1 : row);
  }
  if (token) {
    e.key[rank] = (int32_t)row;
    e.perm[rank] = (int32_t)(x & 0xFFFFFFFFu);
  } else {
    e.tile[i - e.T] = (int32_t)rank;
  }
}

// Sort the tokens; bounds > 0: where the step's tiles begin too; zero.rows > 0: clear those.
static hipError_t sort_tokens(const EmbedArgs& e, int64_t bounds, const ZeroArgs& zero, hipStream_t st) {
  SortArgs a{e, bounds, zero, 0, 0, (int32_t)((e.T + EMBED_PART - 1) / EMBED_PART)};
  if (e.T > 0) {
    const int64_t last = e.T - (int64_t)(a.parts - 1) * EMBED_PART;
    a.place_wgs = (int32_t)((a.parts - 1) * (EMBED_PART / PLACE_TOKENS) + (last + PLACE_TOKENS - 1) / PLACE_TOKENS);
    if (a.parts == 1) a.bound_wgs = (int32_t)((bounds + PLACE_TOKENS - 1) / PLACE_TOKENS);
  }
  const int64_t per = PLACE_NT >> zero.sh, zero_wgs = std::min<int64_t>((zero.rows + per - 1) / per, PLACE_ZERO_WGS);
  const unsigned grid = (unsigned)(a.place_wgs + a.bound_wgs + zero_wgs);
  if (grid == 0) return hipSuccess;
  hipLaunchKernelGGL(k_embed_place, dim3(grid), dim3(PLACE_NT), 0, st, a);
  const hipError_t err = hipGetLastError();
  if (err != hipSuccess || a.parts <= 1) return err;
  hipLaunchKernelGGL(k_embed_ranks, dim3((unsigned)((e.T + bounds + NT - 1) / NT)), dim3(NT), 0, st, a);
  return hipGetLastError();
}

hipError_t launch_embed_sort(const EmbedArgs& e, int64_t tiles, hipStream_t st) {
  return sort_tokens(e, e.T > 0 ? tiles + 1 : 0, ZeroArgs{nullptr, 0, 0, 0, 0}, st);
}

// ------------------------------------------------------------------------
// acc[v] (+)= scale sum of dY over the tokens of v, for the rows that occur.  The
// first `longs` workgroups take the rows of more than ROW_LONG tokens: such a run
// of the sorted tokens holds a place that is a multiple of ROW_LONG, and the first
// of those (with each 64 columns of the row) is its unit of work: 32 tokens at a
// time, 8 lanes of 8 columns each.  The other workgroups take the short rows: a
// wave per (place that begins a row, ROW_COLS columns), the tokens in order.
// Every sum has a fixed order.  Bound by HBM for many rows (8192 tokens of 128256 x
// 4096 added to fp32: 71 us with the sort, 335 MB, 4.7 TB/s), by the latency of the
// sort and of a row's loads for few (5000 of 1000 x 1001 bf16: 18 us with the sort;
// half of 8192 tokens on one of 1000 rows of 1024: 41).  Rows are read 8 at a time:
// one at a time the last takes 74 us.
// ------------------------------------------------------------------------
constexpr int ROW_LONG = 32, ROW_COLS = 512, ROW_SEG = 64;

// End of the run of row v that place p belongs to (keys past the end differ); all
// lanes of the wave.  64 places in steps of 64, then 64 in steps of one: two reads find
// the end of a run of up to 4096.
__device__ __forceinline__ int64_t run_end(const EmbedArgs& e, int64_t p, int v) {
  const int lane = threadIdx.x & 63;
  const auto first_other = [&](int64_t at, int64_t by) {   // the first lane whose place is not in the run (64: none)
    const int64_t i = at + lane * by;
    const uint64_t m = __ballot(i >= e.T || e.key[i] != v);
    return m ? __builtin_ctzll(m) : 64;
  };
  for (;;) {
    const int k = first_other(p, 64);
    p += (int64_t)(k - 1) * 64;         // the last place seen inside the run (k > 0: p itself is)
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
  const int64_t end = run_end(e, p, v);
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
    // (half as many fp32 rows at a time: the kernel keeps to 128 registers)
    sum_rows<MODE, DF, DF == FMT_F32 ? 4 : 8>(at, (n + 31) / 32, (n - slot + 31) / 32, c, e.K, s);
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
  // the 64 places from p on and the one before, requested together
  const int64_t i = min(p + lane, e.T - 1);
  const int key = e.key[i], tok = e.perm[i], before = e.key[p > 0 ? p - 1 : 0];
  const int v = __builtin_amdgcn_readfirstlane(key);
  if (v >= e.V || (p > 0 && before == v)) return;
  const uint64_t others = __ballot(p + lane >= e.T || key != v);
  const int n = others ? __builtin_ctzll(others) : 64;
  if (n > ROW_LONG) return;
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
__global__ void __launch_bounds__(NT, 4) k_embed_rows(const EmbedArgs e, float* acc, int64_t ldacc, int add, int longs) {
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
  const hipError_t err = sort_tokens(e, 0, ZeroArgs{acc, ldacc, first ? e.V : 0, e.K, lane_shift(e.K, 4, 10)}, st);
  if (err != hipSuccess || e.T == 0) return err;
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

hipError_t launch_embed_step(const KArgs& a, const EmbedArgs& e, int w_fmt, int opt, int m_fmt, int v_fmt,
                             hipStream_t st) {
#define X(O, M, V) \
  if (opt == O && m_fmt == M && v_fmt == V) return combo_embed<O, M, V>(a, e, w_fmt, st);
  FORGE_STATE_LIST(X)
#undef X
  return hipErrorInvalidValue;
}

}  // namespace forge
