// The optimizer step on an embedding's gradient: the fused step's epilogue on
// tiles whose gradient is gathered from the sorted tokens.
#pragma once

#include "forge_act8.h"

namespace forge {

// G tile (EMBED_ROWS rows of W from row0, 128 columns from col0) into LDS:
//   sG[r * GP + c] = scale * sum over the tokens of row row0 + r of dY[token][col0 + c].
// first, last: the tile's places among the sorted tokens.  16 lanes of 8 columns per
// token.  A row of up to LONG_ROW tokens belongs to one wave, 4 tokens at a time; a
// longer one to the whole workgroup, 16 at a time.  Sums over a slot's tokens in
// order, then over the slots in a fixed order.  rng: 2 EMBED_ROWS ints, red: 3 x 128 floats.
constexpr int LONG_ROW = 32;

// Tokens slot, slot + step, .. of first .. last - 1 of the sorted ones, and then the sum
// over the wave's 4 slots.  (A slot with no token of its own has mine <= 0.)
template <int MODE, int DF>
__device__ __forceinline__ void gather_tokens(const EmbedArgs& e, int first, int last, int slot, int step, int64_t c,
                                              float (&s)[8]) {
  constexpr int ds = DF == FMT_F32 ? 4 : 2;
#pragma unroll
  for (int k = 0; k < 8; ++k) s[k] = 0.f;
  const auto at = [&](int i) {
    return static_cast<const char*>(e.dY) + (int64_t)e.perm[min(first + slot + i * step, last - 1)] * e.lddy * ds;
  };
  // (half as many fp32 rows at a time: the kernel keeps to 128 registers)
  sum_rows<MODE, DF, DF == FMT_F32 ? 4 : 8>(at, (last - first + step - 1) / step, (last - first - slot + step - 1) / step, c, e.K, s);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    s[k] += __shfl_xor(s[k], 16);
    s[k] += __shfl_xor(s[k], 32);
  }
}

template <int MODE, int DF>
__device__ __forceinline__ void embed_tile(const EmbedArgs& e, float* sG, int* rng, float* red, int row0, int col0, int first,
                                           int last) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int cl = 8 * (lane & 15);
  const int64_t c = (int64_t)col0 + cl;
  for (int i = tid; i < EMBED_ROWS * GP / 4; i += NT) reinterpret_cast<f32x4*>(sG)[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  if (first >= last) {     // (the same for the whole workgroup)
    __syncthreads();
    return;
  }
  for (int i = tid; i < 2 * EMBED_ROWS; i += NT) rng[i] = 0;
  __syncthreads();
  for (int p = first + tid; p < last; p += NT) {
    const int k = e.key[p];
    if (p == first || e.key[p - 1] != k) rng[2 * (k - row0)] = p;
    if (p + 1 == last || e.key[p + 1] != k) rng[2 * (k - row0) + 1] = p + 1;
  }
  __syncthreads();
  const int r = lane;
  const int n = r < EMBED_ROWS ? rng[2 * r + 1] - rng[2 * r] : 0;
  // rows of this wave (r % 4 == wave) with few tokens, then the long rows with all waves
  uint64_t mine = __ballot(n > 0 && n <= LONG_ROW && (r & 3) == wave), all = __ballot(n > LONG_ROW);
  while (mine) {
    const int k = __builtin_ctzll(mine);
    mine &= mine - 1;
    float s[8];
    gather_tokens<MODE, DF>(e, rng[2 * k], rng[2 * k + 1], lane >> 4, 4, c, s);
    if (lane < 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sG[k * GP + cl + i] = s[i] * e.scale;
    }
  }
  while (all) {   // the same rows in every wave
    const int k = __builtin_ctzll(all);
    all &= all - 1;
    float s[8];
    gather_tokens<MODE, DF>(e, rng[2 * k], rng[2 * k + 1], tid >> 4, 16, c, s);
    if (wave > 0 && lane < 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) red[(wave - 1) * TILE + cl + i] = s[i];
    }
    __syncthreads();
    if (wave == 0 && lane < 16) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        sG[k * GP + cl + i] =
            (((s[i] + red[cl + i]) + red[TILE + cl + i]) + red[2 * TILE + cl + i]) * e.scale;
    }
    __syncthreads();
  }
  __syncthreads();
}

// FAST, ANY: rows of at least 8 elements, ANY of any alignment.
template <bool FAST, bool ANY, int OPT, int WF, int MF, int VF>
__global__ void __launch_bounds__(NT, 4) k_embed_step(const KArgs a, const EmbedArgs e) {
  __shared__ __attribute__((aligned(16))) float sG[EMBED_ROWS * GP];
  __shared__ int rng[2 * EMBED_ROWS];
  __shared__ float red[3 * TILE];
  constexpr int MODE = FAST || ANY ? ROW_BIG : ROW_ANY;
  int ti = (int)blockIdx.x / a.tiles_k, tj = (int)blockIdx.x - ti * a.tiles_k;
  if (ANY) tile_by_xcd((int)gridDim.x / a.tiles_k, a.tiles_k, ti, tj);
  const int row0 = ti * EMBED_ROWS, col0 = tj * TILE;
  Epilogue<Step<OPT, WF, MF, VF, FAST, 0, ANY>, FMT_NONE, FAST, 4, NT, false, false, EMBED_ROWS> epi;
  epi.tid = threadIdx.x;
  epi.prefetch(a, row0, col0);
  const int first = e.T ? e.tile[ti] : 0, last = e.T ? e.tile[ti + 1] : 0;
  if (e.dy_fmt == FMT_F32) embed_tile<MODE, FMT_F32>(e, sG, rng, red, row0, col0, first, last);
  else embed_tile<MODE, FMT_BF16>(e, sG, rng, red, row0, col0, first, last);
  epi.run_prefetched(a, sG, row0, col0);
}

// FAST: rows of whole 128-byte lines, whose accesses bypass the caches and whose
// tiles go out row of tiles by row.  Other rows share lines at the tiles' seams, and
// streaming parts of lines through different XCDs costs far more than the lines
// themselves: with tiles of 128 rows 37929 x 2984 (bf16 moments, 161 tokens) took 629 us so,
// 337 with cached accesses and neighbouring tiles on one XCD (46421 x 1459, fp32 moments, 124
// tokens: 530 and 316).
//
// Tiles of 16 rows, four workgroups to a CU: small ones hide each other's gathering.
// With AdamW, bf16 W and fp32 moments 8192 tokens of 128256 x 4096 take 1773 us (10.6 GB,
// 6.0 TB/s: bound by HBM), 1837 with tiles of 128 rows; 8192 of 32000 x 4096 458 and 502
// (two workgroups to a CU: 500); 4096 of 1000 x 1024, bound by latency, 17 and 44; the
// unaligned 46421 x 1459 with 124 tokens 280 and 313, 37929 x 2985 with bf16 moments and 161
// tokens 316 and 352.  Tokens cost more where the state is small: the last takes 284 us with
// 100 tokens, 338 with 1000, 470 with 8192 (spread over the vocabulary).
template <int O, int M, int V>
hipError_t combo_embed(const KArgs& a, const EmbedArgs& e, int w_fmt, hipStream_t st) {
  const bool fast = a.vec_state && a.K % 64 == 0 && a.ldw % 64 == 0 && a.ldm % 64 == 0 && a.ldv % 64 == 0;
  if (w_fmt != FMT_BF16 && w_fmt != FMT_F32) return hipErrorInvalidValue;
  const int64_t tiles = (a.N + EMBED_ROWS - 1) / EMBED_ROWS;
  const hipError_t err = launch_embed_sort(e, tiles, st);
  if (err != hipSuccess) return err;
  const dim3 grid((unsigned)(tiles * a.tiles_k));
#define FORGE_EMBED(FA, ANY)                                                                                          \
  if (w_fmt == FMT_BF16) hipLaunchKernelGGL((k_embed_step<FA, ANY, O, FMT_BF16, M, V>), grid, dim3(NT), 0, st, a, e); \
  else hipLaunchKernelGGL((k_embed_step<FA, ANY, O, FMT_F32, M, V>), grid, dim3(NT), 0, st, a, e);                    \
  return hipGetLastError();
  if (fast) { FORGE_EMBED(true, false) }
  if (a.K >= 8) { FORGE_EMBED(false, true) }
  FORGE_EMBED(false, false)
#undef FORGE_EMBED
}
#define FORGE_INSTANTIATE_EMBED(O, M, V) \
  template hipError_t combo_embed<O, M, V>(const KArgs&, const EmbedArgs&, int, hipStream_t);

}  // namespace forge
