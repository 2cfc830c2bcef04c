// The fused weight gradient with X in 8 bits.
//
// G = dY^T X with X = code * 2^e.  The exponent differs from token to token, so
// it cannot leave the sum; each 8 bits are decoded to the bf16 they stand for
// (exactly) between global memory and LDS, after which the matrix-core loop is
// that of bf16 inputs.  In the kernels of aligned layers every element of G sees the
// same MFMA sequence as with the decoded X, so the results are the same bit for bit.
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

// Layers with fewer than 8 outputs or 16 inputs: MainBF16 with its register staging,
// X decoded on the way into LDS.
struct MainAct8 {
  static constexpr int MODE = ROW_ANY;
  static constexpr int TK = MainBF16::TK;
  static constexpr int OPB = MainBF16::OPB;
  static constexpr int STAGE = MainBF16::STAGE;
  Raw8<FMT_BF16> ra[4];
  u32x2 rc[4];
  uint32_t rs[4];
  int64_t cy, cx, N, K;
  int tok0, BT;
  bool e4m3;

  __device__ __forceinline__ void load(const KArgs8& a, int kc, int row0, int col0) {
    const int tid = threadIdx.x;
    const int f = (tid & 15) * 8;
    cy = row0 + f;
    cx = col0 + f;
    N = a.N;
    K = a.K;
    BT = a.BT;
    tok0 = kc * TK + (tid >> 4);
    e4m3 = a.x_fmt == FMT_E4M3;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int64_t tok = min(tok0 + 16 * r, a.BT - 1);   // past the end: read again, cleared in store()
      ra[r] = row_raw8<FMT_BF16, MODE>(static_cast<const uint16_t*>(a.dY) + tok * a.lddy, cy, a.N);
      rc[r] = codes_raw8<MODE>(a.x8.codes + tok * a.x8.ld, cx, a.K);
      rs[r] = (uint32_t)a.x8.scale[tok * a.x8.nb + (min(cx, (int64_t)a.K - 1) >> a.x8.sh)];
    }
  }

  __device__ __forceinline__ void store(char* stage) const {
    const int tid = threadIdx.x;
    const int f = (tid & 15) * 8;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const int t = (tid >> 4) + 16 * r;
      const bool in = tok0 + 16 * r < BT;
      const u32x4 w = row_place8<FMT_BF16, MODE>(ra[r], in ? cy : N, N).a;
      const u32x2 c = codes_val8<MODE>(rc[r], in ? cx : K, K);
      const float s = act8_mul(in ? rs[r] : 0u);   // (a cleared code times a NaN scale would be a NaN)
      *reinterpret_cast<u32x4*>(stage + MainBF16::off(t, f)) = w;
      *reinterpret_cast<u32x4*>(stage + OPB + MainBF16::off(t, f)) =
          e4m3 ? act8_bf16x8<FMT_E4M3>(c, s) : act8_bf16x8<FMT_S8>(c, s);
    }
  }

  __device__ __forceinline__ static void compute(f32x16 (&acc)[2][2], char* stage, int wr, int wc, int lane) {
    MainBF16::compute(acc, stage, wr, wc, lane);
  }
};

// ------------------------------------------------------------------------
// Aligned shapes.  dY goes to LDS by the asynchronous loads of the bf16 kernels;
// X cannot (its bytes have to be decoded), so each thread loads 16 codes and
// their scale byte of one token into registers D chunks ahead, and writes the 16
// decoded bf16 into the same swizzled LDS rows two chunks before they are used:
//   iteration kc:  [wait dY(kc); barrier]  issue dY(kc + S - 1)
//                  read and multiply chunk kc
//                  decode X(kc + 2) into stage (kc + 2) % S;  request X(kc + 2 + D)
// Stage (kc + 2) % S held chunk kc + 2 - S, which every wave is done with at
// iteration kc's barrier (S >= 3).  X(kc + 2)'s LDS writes are waited for by
// iteration kc + 1's last fragment wait (lgkmcnt(0)) and seen by all waves after
// the barrier of iteration kc + 2.  Tokens past the end and loads past the last
// chunk read as zero (buffer bounds), so every iteration issues the same loads
// and the waits are constants.
// ------------------------------------------------------------------------

// 16 codes and the scale byte of one token in flight: one value of five words, so
// that the byte stays a whole register from its load to its use (as a loop-carried
// byte of its own the compiler masks it at the top of the loop and waits there).
typedef uint32_t u32x5 __attribute__((ext_vector_type(5)));

// X's way into LDS.  W: the LDS row's width in features (128 or 256), W / 16
// threads per token.
template <int XF, int W>
struct XStage {
  __amdgpu_buffer_rsrc_t rC, rS;
  uint32_t oobC, oobS, offC, offS;   // byte offsets of this thread's codes / scale in token row 0
  uint32_t ldc, nb;
  int trow;                          // token within the chunk
  uint32_t lds;                      // byte offset of the 16 bf16 within an operand region
  bool fok;                          // the 16 columns are inside the matrix (K % 16 == 0)

  // gtid: thread among the 2 W that fill a 32-token chunk
  __device__ __forceinline__ void init(const KArgs8& a, int col0, int gtid) {
    trow = gtid / (W / 16);
    const int f = 16 * (gtid & (W / 16 - 1));
    oobC = (uint32_t)((uint64_t)a.BT * a.x8.ld);
    oobS = (uint32_t)((uint64_t)a.BT * a.x8.nb);
    rC = make_rsrc(a.x8.codes, oobC);
    rS = make_rsrc(a.x8.scale, oobS);
    ldc = (uint32_t)a.x8.ld;
    nb = (uint32_t)a.x8.nb;
    fok = col0 + f < a.K;
    offC = (uint32_t)(col0 + f);
    offS = (uint32_t)((col0 + f) >> a.x8.sh);
    lds = (uint32_t)(trow * (W * 2) + ((f * 2) ^ ((trow & 3) << 6)));
  }
  __device__ __forceinline__ u32x5 request(const KArgs8& a, int kc) const {
    const int tok = kc * 32 + trow;
    const bool in = tok < a.BT && fok;
    const u32x4 c = __builtin_bit_cast(
        u32x4, __builtin_amdgcn_raw_buffer_load_b128(rC, in ? (uint32_t)tok * ldc + offC : oobC, 0, 0));
    const uint32_t s =
        (uint32_t)__builtin_amdgcn_raw_buffer_load_b8(rS, in ? (uint32_t)tok * nb + offS : oobS, 0, 0);
    return u32x5{c[0], c[1], c[2], c[3], s};
  }
  // Codes 4 i .. 4 i + 3 as two words of bf16.
  __device__ __forceinline__ static u32x2 word(const u32x5& v, int i, float f) {
    float x[4];
    act8_decode4<XF>(v[i], f, x);
    return u32x2{bf16x2_rne(x[0], x[1]), bf16x2_rne(x[2], x[3])};
  }
  // A 16-byte half of the thread's 32 bytes into the region at `region` (an LDS
  // byte address).  Inline assembly: the compiler would otherwise wait for the
  // asynchronous loads to LDS, of which it cannot tell the stage.
  template <int H>
  __device__ __forceinline__ void put(uint32_t region, u32x2 lo, u32x2 hi) const {
    const u32x4 v = {lo[0], lo[1], hi[0], hi[1]};
    asm volatile("ds_write_b128 %0, %1 offset:%2" ::"v"(region + lds), "v"(v), "i"(16 * H));
  }
  // Nothing that uses the loaded words moves above this point (it would wait for
  // them there).
  __device__ __forceinline__ static void pin(u32x5& v) { asm volatile("" : "+v"(v)); }
  __device__ __forceinline__ void store(uint32_t region, const u32x5& v) const {
    const float f = act8_mul(v[4]);
    put<0>(region, word(v, 0, f), word(v, 1, f));
    put<1>(region, word(v, 2, f), word(v, 3, f));
  }
};

// dY's half of MainBF16DmaT.
template <int STAGES>
struct MainDy {
  static constexpr int TK = 32, S = STAGES;
  static constexpr int OPB = TK * TILE * 2, STAGE = 2 * OPB;
  __amdgpu_buffer_rsrc_t rA;
  uint32_t oob, base[2];
  int trow[2], wave;
  bool fok[2];

  __device__ __forceinline__ void init(const KArgs8& a, int row0) {
    const int lane = threadIdx.x & 63;
    wave = threadIdx.x >> 6;
    oob = (uint32_t)((uint64_t)a.BT * a.lddy * 2);
    rA = make_rsrc(a.dY, oob);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = 4 * (2 * wave + r) + (lane >> 4);
      const int c = (lane & 15) ^ ((t & 3) << 2);
      trow[r] = t;
      fok[r] = row0 + c * 8 < a.N;
      base[r] = (uint32_t)(row0 + c * 8) * 2;
    }
  }
  __device__ __forceinline__ void issue(const KArgs8& a, int kc, char* stage) const {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int tok = kc * TK + trow[r];
      const uint32_t o = (tok < a.BT && fok[r]) ? (uint32_t)tok * (uint32_t)(a.lddy * 2) + base[r] : oob;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_void*)(stage + (2 * wave + r) * 1024), 16, o, 0, 0, 0);
    }
  }
};

// Phase 1 for a 256-thread workgroup; acc as dma_accumulate leaves it.  On
// return no load or LDS access of this wave is outstanding.
template <int XF, int S, int D>
struct Act8Loop {
  using M = MainDy<S>;
  static_assert(S >= 3 && D == S - 2, "the vmcnt waits count loads for this pair");
  M ml;
  XStage<XF, TILE> xs;
  u32x5 x[D];                        // X(kc + 2 + j) in x[(kc + j) % D] at iteration kc
  uint32_t lds0, fofsA[2], fofsB[2];

  __device__ __forceinline__ uint32_t region(int k) const { return lds0 + (uint32_t)((k % S) * M::STAGE) + M::OPB; }

  template <int J>
  __device__ __forceinline__ void iteration(const KArgs8& a, char* ring, int kc, f32x16 (&acc)[2][2]) {
    bar();
    ml.issue(a, kc + S - 1, ring + ((kc + S - 1) % S) * M::STAGE);
    __builtin_amdgcn_sched_barrier(0);
    const uint32_t cur = lds0 + (uint32_t)((kc % S) * M::STAGE);
    u32x2 f0[8], f1[8];
    uint32_t pa[2], pb[2];
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      pa[b] = cur + fofsA[b];
      pb[b] = cur + fofsB[b];
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f0[2 * b] = tr_read_at<0>(pa[b]);
      f0[2 * b + 1] = tr_read_at<1024>(pa[b]);
      f0[4 + 2 * b] = tr_read_at<0>(pb[b]);
      f0[4 + 2 * b + 1] = tr_read_at<1024>(pb[b]);
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      f1[2 * b] = tr_read_at<4096>(pa[b]);
      f1[2 * b + 1] = tr_read_at<5120>(pa[b]);
      f1[4 + 2 * b] = tr_read_at<4096>(pb[b]);
      f1[4 + 2 * b + 1] = tr_read_at<5120>(pb[b]);
    }
    lds_wait<8>(f0);
#pragma unroll
    for (int bi = 0; bi < 2; ++bi)
#pragma unroll
      for (int bj = 0; bj < 2; ++bj)
        acc[bi][bj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag_join(f0[2 * bi], f0[2 * bi + 1]),
                                                              frag_join(f0[4 + 2 * bj], f0[4 + 2 * bj + 1]),
                                                              acc[bi][bj], 0, 0, 0);
    __builtin_amdgcn_sched_barrier(0);
    lds_wait<0>(f1);
#pragma unroll
    for (int bi = 0; bi < 2; ++bi)
#pragma unroll
      for (int bj = 0; bj < 2; ++bj)
        acc[bi][bj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag_join(f1[2 * bi], f1[2 * bi + 1]),
                                                              frag_join(f1[4 + 2 * bj], f1[4 + 2 * bj + 1]),
                                                              acc[bi][bj], 0, 0, 0);
    xs.pin(x[J]);
    xs.store(region(kc + 2), x[J]);
    __builtin_amdgcn_sched_barrier(0);
    x[J] = xs.request(a, kc + 2 + D);
    __builtin_amdgcn_sched_barrier(0);
    // dY(kc + 1), which iteration kc + 2 - S = kc - D issued, landed: since then
    // X(kc + 2) and four loads in each of D iterations (the prologue's dY chunks
    // have at least as many behind them)
    wait_vmcnt<4 * D + 2>();
  }

  template <int... J>
  __device__ __forceinline__ void sweep(const KArgs8& a, char* ring, int kc, f32x16 (&acc)[2][2],
                                        std::integer_sequence<int, J...>) {
    (iteration<J>(a, ring, kc + J, acc), ...);
  }

  __device__ __forceinline__ void run(const KArgs8& a, char* ring, int row0, int col0, f32x16 (&acc)[2][2]) {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int wr = wave >> 1, wc = wave & 1;
    lds0 = (uint32_t)(uintptr_t)(lds_void*)ring;
#pragma unroll
    for (int bi = 0; bi < 2; ++bi)
#pragma unroll
      for (int bj = 0; bj < 2; ++bj)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[bi][bj][e] = 0.f;
    const int nk = (a.BT + M::TK - 1) / M::TK;
    if (nk == 0) return;
    const int t = 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int f = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      fofsA[b] = (uint32_t)MainBF16::off(t, wr * 64 + b * 32 + f);
      fofsB[b] = (uint32_t)(M::OPB + MainBF16::off(t, wc * 64 + b * 32 + f));
    }
    ml.init(a, row0);
    xs.init(a, col0, tid);
    u32x5 x0 = xs.request(a, 0), x1 = xs.request(a, 1);
#pragma unroll
    for (int k = 0; k < S - 1; ++k) ml.issue(a, k, ring + k * M::STAGE);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < D; ++j) x[j] = xs.request(a, 2 + j);
    __builtin_amdgcn_sched_barrier(0);
    xs.store(region(0), x0);
    xs.store(region(1), x1);
    // dY(0) landed: the S - 2 later chunks and X(2 .. D + 1) may be in flight
    wait_vmcnt<2 * (S - 2) + 2 * D>();
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    // (a last sweep past nk multiplies chunks of zeros)
    for (int kc = 0; kc < nk; kc += D) sweep(a, ring, kc, acc, std::make_integer_sequence<int, D>{});
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  }
};

// The occupancy, ring depth and passes in flight of k_fused.
template <int XF, int OPT, int WF, int MF, int VF, int BLK = 0, bool FULL = false>
__global__ void __launch_bounds__(NT, (three_per_cu<OPT, WF, MF, VF, true, false, false>() ? 3 : 2))
    k_fused_act8_dma(const KArgs8 a) {
  constexpr bool OCC3 = three_per_cu<OPT, WF, MF, VF, true, false, false>();
  __shared__ __attribute__((aligned(16))) char lds[OCC3 ? LDS_HALF : LDS_BYTES];
  int ti, tj;
  tile_coords(blockIdx.x, a.tiles_n, a.tiles_k, ti, tj);
  const int row0 = ti * TILE, col0 = tj * TILE;
  Epilogue<Step<OPT, WF, MF, VF, true, BLK>, FMT_NONE, true, epi_depth<OPT, WF, MF, VF, true, false, false>(), NT, false,
           FULL> epi;
  epi.tid = threadIdx.x;
  constexpr int PRE = epi_pre<OPT, WF, MF, VF, true, false, false>();
  epi.template prefetch<PRE>(a, row0, col0);
  f32x16 acc[2][2];
  Act8Loop<XF, OCC3 ? 3 : 4, OCC3 ? 1 : 2> loop;
  loop.run(a, lds, row0, col0, acc);
  bar();   // every wave is done with the stages before G overwrites them
  if constexpr (OCC3) {
    epi.template prefetch_rest<PRE>(a, row0, col0);
    epi.run_halves_rm(a, reinterpret_cast<float*>(lds), acc, row0, col0);
  } else {
    store_acc(reinterpret_cast<float*>(lds), acc, threadIdx.x);
    __syncthreads();
    epi.run_prefetched_rm(a, reinterpret_cast<const float*>(lds), row0, col0);
  }
}

// ------------------------------------------------------------------------
// Long token axes: wide_accumulate (256 x 256 per workgroup of 8 waves) with X
// decoded on the way.  Iteration kc decodes X(kc + 1) between the MFMAs of its
// first k-step into stage (kc + 1) % 4, which held chunk kc - 3; the fragment
// wait and the barrier between the k-steps make it visible to the second, which
// reads it.  Two chunks of X are in flight, so the loop is unrolled by two.
// ------------------------------------------------------------------------
struct MainWideDy {
  static constexpr int TK = MainWide::TK, S = MainWide::S, ROWB = MainWide::ROWB;
  static constexpr int OPB = MainWide::OPB, STAGE = MainWide::STAGE;
  __amdgpu_buffer_rsrc_t rA;
  uint32_t oob, base[2];
  int trow[2], wave;
  bool fok[2];

  __device__ __forceinline__ void init(const KArgs8& a, int row0) {
    const int lane = threadIdx.x & 63;
    wave = threadIdx.x >> 6;
    oob = (uint32_t)((uint64_t)a.BT * a.lddy * 2);
    rA = make_rsrc(a.dY, oob);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int t = 2 * (8 * r + wave) + (lane >> 5);
      const int c = (lane & 31) ^ ((t & 3) << 2);
      trow[r] = t;
      fok[r] = row0 + c * 8 < a.N;
      base[r] = (uint32_t)(row0 + c * 8) * 2;
    }
  }
  template <int R>
  __device__ __forceinline__ void issue_one(const KArgs8& a, int kc, char* stage) const {
    const int tok = kc * TK + trow[R];
    const uint32_t o = (tok < a.BT && fok[R]) ? (uint32_t)tok * (uint32_t)(a.lddy * 2) + base[R] : oob;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(rA, (lds_void*)(stage + (8 * R + wave) * 1024), 16, o, 0, 0, 0);
  }
};

template <int XF>
struct Act8Wide {
  using M = MainWideDy;
  static constexpr int D = 2;
  M ml;
  XStage<XF, MainWide::W> xs;
  u32x5 x[D];                        // X(kc + 1 + j) in x[(kc + j) % D] at iteration kc
  uint32_t lds0, off[6], adr[6];
  u32x2 f0[12], f1[12];

  // MFMA slot I of a k-step: fragment reads as wide_one; FIRST: X's decoding (words
  // at even slots, their 16-byte writes at slots 3 and 7), else dY's loads.
  template <bool FIRST, int J, int I>
  __device__ __forceinline__ void slot(const KArgs8& a, int kc, char* ring, f32x16 (&acc)[4][2], u32x2 (&w)[4], float f) {
    u32x2 (&cur)[12] = FIRST ? f0 : f1;
    u32x2 (&nxt)[12] = FIRST ? f1 : f0;
    constexpr int bi = I >> 1, bj = I & 1, T0 = FIRST ? 16 : 0;
    acc[bi][bj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag_join(cur[2 * bi], cur[2 * bi + 1]),
                                                          frag_join(cur[8 + 2 * bj], cur[8 + 2 * bj + 1]),
                                                          acc[bi][bj], 0, 0, 0);
    nxt[I] = tr_read_at<(T0 + 4 * (I & 1)) * M::ROWB>(adr[I >> 1]);
    if constexpr ((I & 1) == 0) {
      constexpr int R = 8 + I / 2;
      nxt[R] = tr_read_at<(T0 + 4 * (R & 1)) * M::ROWB>(adr[4 + ((R - 8) >> 1)]);
    }
    if constexpr (FIRST) {
      if constexpr ((I & 1) == 0) w[I / 2] = xs.word(x[J], I / 2, f);
      const uint32_t region = lds0 + (uint32_t)(((kc + 1) % M::S) * M::STAGE) + M::OPB;
      if constexpr (I == 3) xs.template put<0>(region, w[0], w[1]);
      if constexpr (I == 7) xs.template put<1>(region, w[2], w[3]);
    } else {
      if constexpr (I == 0) ml.template issue_one<0>(a, kc + M::S, ring + (kc % M::S) * M::STAGE);
      if constexpr (I == 4) ml.template issue_one<1>(a, kc + M::S, ring + (kc % M::S) * M::STAGE);
    }
    __builtin_amdgcn_sched_barrier(0);
  }
  template <bool FIRST, int J, int... I>
  __device__ __forceinline__ void kstep(const KArgs8& a, int kc, char* ring, f32x16 (&acc)[4][2],
                                        std::integer_sequence<int, I...>) {
    u32x2 w[4];
    float f = 0.f;
    if constexpr (FIRST) {
      xs.pin(x[J]);
      f = act8_mul(x[J][4]);
    }
    (slot<FIRST, J, I>(a, kc, ring, acc, w, f), ...);
  }

  template <int J>
  __device__ __forceinline__ void iteration(const KArgs8& a, char* ring, int kc, f32x16 (&acc)[4][2]) {
    kstep<true, J>(a, kc, ring, acc, std::make_integer_sequence<int, 8>{});
    x[J] = xs.request(a, kc + 1 + D);
    __builtin_amdgcn_sched_barrier(0);
    lds_wait12(f1);
    // dY(kc + 1), issued by iteration kc - 3, landed: since then X in three iterations
    // and dY in two (the prologue's loads have at least as many behind them)
    wait_vmcnt<10>();
    bar();
    const uint32_t st = lds0 + (uint32_t)(((kc + 1) % M::S) * M::STAGE);
#pragma unroll
    for (int r = 0; r < 6; ++r) adr[r] = st + off[r];
    kstep<false, J>(a, kc, ring, acc, std::make_integer_sequence<int, 8>{});
    lds_wait12(f0);
  }

  __device__ __forceinline__ void run(const KArgs8& a, char* ring, int row0, int col0, f32x16 (&acc)[4][2]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int wr = wave >> 2, wc = wave & 3;
    lds0 = (uint32_t)(uintptr_t)(lds_void*)ring;
#pragma unroll
    for (int bi = 0; bi < 4; ++bi)
#pragma unroll
      for (int bj = 0; bj < 2; ++bj)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[bi][bj][e] = 0.f;
    const int nk = (a.BT + M::TK - 1) / M::TK;
    if (nk == 0) return;
    const int tl = 8 * (lane >> 5) + ((lane & 15) >> 2);
    const int fl = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
#pragma unroll
    for (int b = 0; b < 4; ++b) off[b] = (uint32_t)MainWide::off(tl, wr * 128 + b * 32 + fl);
#pragma unroll
    for (int b = 0; b < 2; ++b) off[4 + b] = (uint32_t)(M::OPB + MainWide::off(tl, wc * 64 + b * 32 + fl));
    ml.init(a, row0);
    xs.init(a, col0, threadIdx.x);
    static_assert(M::S == 4 && D == 2, "the vmcnt waits count loads for this pair");
    u32x5 x0 = xs.request(a, 0);
#pragma unroll
    for (int k = 0; k < M::S; ++k) {
      ml.template issue_one<0>(a, k, ring + k * M::STAGE);
      ml.template issue_one<1>(a, k, ring + k * M::STAGE);
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < D; ++j) x[j] = xs.request(a, 1 + j);
    __builtin_amdgcn_sched_barrier(0);
    xs.store(lds0 + M::OPB, x0);
    wait_vmcnt<10>();   // dY(0) landed: three chunks of dY and two of X behind it
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    bar();
#pragma unroll
    for (int r = 0; r < 6; ++r) adr[r] = lds0 + off[r];
#pragma unroll
    for (int r = 0; r < 12; ++r)
      f0[r] = tr_read(adr[r < 8 ? (r >> 1) : 4 + ((r - 8) >> 1)] + (uint32_t)(4 * (r & 1) * M::ROWB));
    lds_wait12(f0);
    for (int kc = 0; kc < nk; kc += 2) {   // (a last iteration past nk multiplies zeros)
      iteration<0>(a, ring, kc, acc);
      iteration<1>(a, ring, kc + 1, acc);
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  }
};

// As k_fused_wide.
template <int XF, int OPT, int WF, int MF, int VF, bool FULL>
__global__ void __launch_bounds__(2 * NT, 1) k_fused_act8_wide(const KArgs8 a) {
  __shared__ __attribute__((aligned(16))) char lds[LDS_WIDE];
  const int tw = (a.K + MainWide::W - 1) / MainWide::W;
  const int mi = (int)blockIdx.x / tw;
  const int row0 = mi * MainWide::W, col0 = ((int)blockIdx.x - mi * tw) * MainWide::W;
  f32x16 acc[4][2];
  Act8Wide<XF> loop;
  loop.run(a, lds, row0, col0, acc);
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int wr = wave >> 2, wc = wave & 3;
  float* sG = reinterpret_cast<float*>(lds);
  Epilogue<Step<OPT, WF, MF, VF, true>, FMT_NONE, true, 2, 2 * NT, false, FULL> epi;
  epi.tid = threadIdx.x;
  for (int sub = 0; sub < 4; ++sub) {
    const int srow0 = row0 + (sub >> 1) * TILE, scol0 = col0 + (sub & 1) * TILE;
    bar();                                   // the ring / the previous sub-tile is no longer read
    if (wr == (sub >> 1) && (wc >> 1) == (sub & 1)) {
#pragma unroll
      for (int bi = 0; bi < 4; ++bi)
#pragma unroll
        for (int bj = 0; bj < 2; ++bj)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int r = bi * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3);
            const int c = (wc & 1) * 64 + bj * 32 + (lane & 31);
            sG[r * GP + c] = acc[bi][bj][e];
          }
    }
    __syncthreads();
    if (srow0 < a.N && scol0 < a.K) epi.run_tile_rm(a, sG, srow0, scol0);
  }
}

// ------------------------------------------------------------------------
// Few tiles, or rows the ring does not take (N >= 8, K >= 16): the token axis split
// over the WAVES waves of a workgroup.  A tile is ROWS rows x 128 columns; wave w takes
// the 32-token chunks w, w + WAVES, .. alone, with a slab of LDS of its own (so its loop
// has no barrier), and the sums are added in a fixed order at the end.  Any alignment:
// rows are loaded into registers a chunk ahead, the vector that a row ends in shifted
// into place.  Bound by the latency of a wave's chunk: 0.6 us with 64 rows and 8 waves.
// LDS: WAVES slabs of 12 or 10 KiB (dY 32 x ROWS, X 32 x 128, bf16), then WAVES / 2 G
// tiles over them.
// ------------------------------------------------------------------------
// 16 codes at column c of a row of K >= 16: the load of those at min(c, K - 16), and
// what moves them into place.
__device__ __forceinline__ u32x4 codes_raw16(const uint8_t* p, int64_t c, int64_t K) {
  typedef uint32_t u32x4_c __attribute__((ext_vector_type(4), aligned(1)));
  return *reinterpret_cast<const u32x4_c*>(p + min(c, K - 16));
}
__device__ __forceinline__ u32x4 codes_shift16(u32x4 w, int s) {   // down by s places (0 .. 15)
  w = s & 8 ? u32x4{w[2], w[3], 0u, 0u} : w;
  w = s & 4 ? u32x4{w[1], w[2], w[3], 0u} : w;
  return u32x4{__builtin_amdgcn_alignbyte(w[1], w[0], s & 3), __builtin_amdgcn_alignbyte(w[2], w[1], s & 3),
               __builtin_amdgcn_alignbyte(w[3], w[2], s & 3), w[3] >> (8 * (s & 3))};
}

template <int ROWS, int WAVES>
struct Act8Split {
  static constexpr int BI = ROWS / 32;                      // 32-row blocks of the tile
  static constexpr int DY = 32 * ROWS * 2, SLAB = DY + 32 * TILE * 2;
  static constexpr int G = ROWS * GP;                       // floats of one G tile
  static constexpr int LDS = WAVES * SLAB > WAVES / 2 * G * 4 ? WAVES * SLAB : WAVES / 2 * G * 4;
  static_assert(LDS <= 160 * 1024, "LDS budget");
  static constexpr int YL = ROWS / 8, NY = YL / 2;          // lanes per token of dY, and its loads per chunk

  // byte offset of (token, feature) in the dY half of a slab: where rows take 128 bytes,
  // every other pair of them shifted by 64, so that the 4 rows of a transposing read
  // lie in different banks (X's rows: MainBF16::off)
  __device__ __forceinline__ static int off_dy(int t, int f) {
    return t * (ROWS * 2) + ((f * 2) ^ (ROWS == 64 ? (t & 2) << 5 : 0));
  }

  __device__ __forceinline__ static bf16x8 frag(const char* lo, int hi) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)lo);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(lo + hi));
    const s16x4 both[2] = {a, b};
    return __builtin_bit_cast(bf16x8, both);
  }

  template <int XF>
  __device__ __forceinline__ static void run(const KArgs8& a, char* lds, int row0, int col0, f32x16 (&acc)[BI][4]) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    char* slab = lds + wave * SLAB;
#pragma unroll
    for (int bi = 0; bi < BI; ++bi)
#pragma unroll
      for (int bj = 0; bj < 4; ++bj)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[bi][bj][e] = 0.f;
    const int nk = token_chunks(a.BT, 32);
    const int t0 = lane >> 3, ty = lane / YL;      // X: tokens t0 + 8 r of a chunk; dY: ty + 64 / YL r
    const int64_t cy = row0 + 8 * (lane & (YL - 1)), cx = col0 + 16 * (lane & 7);
    const int64_t sx = min(cx, (int64_t)a.K - 1) >> a.x8.sh;
    Raw8<FMT_BF16> ry[NY];
    u32x4 rx[4];
    uint32_t rs[4];
    const auto request = [&](int kc) {
#pragma unroll
      for (int r = 0; r < NY; ++r) {
        const int64_t tok = min((int64_t)kc * 32 + ty + 64 / YL * r, (int64_t)a.BT - 1);   // past the end: read again, cleared below
        ry[r] = row_raw8<FMT_BF16, ROW_BIG>(static_cast<const uint16_t*>(a.dY) + tok * a.lddy, cy, a.N);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int64_t tok = min((int64_t)kc * 32 + t0 + 8 * r, (int64_t)a.BT - 1);
        rx[r] = codes_raw16(a.x8.codes + tok * a.x8.ld, cx, a.K);
        rs[r] = (uint32_t)a.x8.scale[tok * a.x8.nb + sx];
      }
    };
    const int tl = 8 * (lane >> 5) + ((lane & 15) >> 2), fl = 16 * ((lane >> 4) & 1) + 4 * (lane & 3);
    if (wave < nk) request(wave);
    // Only the vectors that a row ends in need moving; one wholly past the end holds
    // other columns' values, which reach nothing but elements of G that are not stored.
    const bool move = (row0 + ROWS > a.N && (a.N & 7)) || (col0 + TILE > a.K && (a.K & 15));
    const int ey = (int)min((int64_t)7, cy - min(cy, (int64_t)a.N - 8)), ex = (int)min((int64_t)15, cx - min(cx, (int64_t)a.K - 16));
    for (int kc = wave; kc < nk; kc += WAVES) {
      if (move) {
#pragma unroll
        for (int r = 0; r < NY; ++r) ry[r] = raw_shift8<FMT_BF16>(ry[r], ey);
#pragma unroll
        for (int r = 0; r < 4; ++r) rx[r] = codes_shift16(rx[r], ex);
      }
      if (a.BT - kc * 32 < 32) {   // tokens past the end
#pragma unroll
        for (int r = 0; r < NY; ++r)
          if (kc * 32 + ty + 64 / YL * r >= a.BT) ry[r].a = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (kc * 32 + t0 + 8 * r >= a.BT) {
            rx[r] = u32x4{0u, 0u, 0u, 0u};
            rs[r] = 0u;
          }
      }
#pragma unroll
      for (int r = 0; r < NY; ++r)
        *reinterpret_cast<u32x4*>(slab + off_dy(ty + 64 / YL * r, 8 * (lane & (YL - 1)))) = ry[r].a;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int t = t0 + 8 * r;
        const float f = act8_mul(rs[r]);
        char* x = slab + DY + MainBF16::off(t, 16 * (lane & 7));
        *reinterpret_cast<u32x4*>(x) = act8_bf16x8<XF>(u32x2{rx[r][0], rx[r][1]}, f);
        *reinterpret_cast<u32x4*>(x + 16) = act8_bf16x8<XF>(u32x2{rx[r][2], rx[r][3]}, f);
      }
      if (kc + WAVES < nk) request(kc + WAVES);
      // the wave's own LDS writes before its lanes' reads (the hardware runs a wave's
      // LDS accesses in order)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        bf16x8 fa[BI], fb[4];
#pragma unroll
        for (int b = 0; b < BI; ++b) fa[b] = frag(slab + off_dy(tl, b * 32 + fl) + ks * 16 * ROWS * 2, 4 * ROWS * 2);
#pragma unroll
        for (int b = 0; b < 4; ++b)
          fb[b] = frag(slab + DY + MainBF16::off(tl, b * 32 + fl) + ks * 16 * TILE * 2, 4 * TILE * 2);
#pragma unroll
        for (int bi = 0; bi < BI; ++bi)
#pragma unroll
          for (int bj = 0; bj < 4; ++bj)
            acc[bi][bj] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa[bi], fb[bj], acc[bi][bj], 0, 0, 0);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }

  // The sum of the waves' tiles into the first G tile of LDS: the first half of the waves
  // write theirs, the others add theirs to those, and the threads add what results.
  __device__ __forceinline__ static void join(float* sG, const f32x16 (&acc)[BI][4]) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    float* mine = sG + (wave & (WAVES / 2 - 1)) * G;
    __syncthreads();                             // the slabs are no longer read
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (wave / (WAVES / 2) == h) {
#pragma unroll
        for (int bi = 0; bi < BI; ++bi)
#pragma unroll
          for (int bj = 0; bj < 4; ++bj)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              float* p = mine + (bi * 32 + 8 * (e >> 2) + 4 * (lane >> 5) + (e & 3)) * GP + bj * 32 + (lane & 31);
              *p = h == 0 ? acc[bi][bj][e] : *p + acc[bi][bj][e];
            }
      }
      __syncthreads();
    }
#pragma unroll
    for (int i = threadIdx.x; i < ROWS * TILE / 4; i += 64 * WAVES) {
      float* p = sG + (i >> 5) * GP + 4 * (i & 31);
      f32x4 g = *reinterpret_cast<f32x4*>(p);
#pragma unroll
      for (int k = 1; k < WAVES / 2; ++k) g += *reinterpret_cast<f32x4*>(p + k * G);
      *reinterpret_cast<f32x4*>(p) = g;
    }
    __syncthreads();
  }
};

template <int ROWS, int WAVES, int OPT, int WF, int MF, int VF>
__global__ void __launch_bounds__(64 * WAVES, 1) k_fused_act8_split(const KArgs8 a) {
  using M = Act8Split<ROWS, WAVES>;
  constexpr int ET = 2 * NT;                         // threads of the epilogue
  constexpr bool EARLY = WAVES == 8;                 // (16 waves have no registers for it)
  __shared__ __attribute__((aligned(16))) char lds[M::LDS];
  int ti, tj;
  tile_by_xcd((int)gridDim.x / a.tiles_k, a.tiles_k, ti, tj);
  const int row0 = ti * ROWS, col0 = tj * TILE;
  f32x16 acc[M::BI][4];
  if (a.x_fmt == FMT_S8) M::template run<FMT_S8>(a, lds, row0, col0, acc);
  else M::template run<FMT_E4M3>(a, lds, row0, col0, acc);
  Epilogue<Step<OPT, WF, MF, VF, false, 0, true>, FMT_NONE, false, 2, ET, false, false, ROWS> epi;
  epi.tid = threadIdx.x;
  const bool steps = threadIdx.x < ET;               // (whole waves)
  if (EARLY && steps) epi.prefetch(a, row0, col0);
  float* sG = reinterpret_cast<float*>(lds);
  M::join(sG, acc);
  if (!EARLY && steps) epi.prefetch(a, row0, col0);
  if (steps) epi.run_prefetched(a, sG, row0, col0);
}

template <int OPT, int WF, int MF, int VF>
__global__ void __launch_bounds__(NT, 2) k_fused_act8_tiny(const KArgs8 a) {
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

// Which kernel takes a layer (measured with AdamW, fp32 moments):
//  - the ring of 128 x 128 tiles (k_fused_act8_dma) needs dY's aligned rows in whole 16-byte
//    segments, K in whole 16-column segments of codes, and enough tiles: with 128 of them
//    (1024 x 2048) it takes 16.0 / 26.8 / 59.9 us at BT 256 / 1024 / 4096, the split kernel
//    12.4 / 17.9 / 34.9; with 256 (2048 x 2048) 21.1 / 31.7 / 65.4 against 23.3 / 32.7 /
//    65.9; below BT 128 the split kernel's joining costs more than it saves (64 x 64: 8.5
//    against 5.8 us);
//  - the 256 x 256 tiles (k_fused_act8_wide) pay for long token axes once they fill the
//    chip: at BT 8192 239 against 302 us for 256 of them (4096 x 4096), but 212
//    against 109 for 64 (2048 x 2048);
//  - of the split kernel's two shapes 32 rows and 16 waves win while every tile has a CU
//    to itself (1024 x 1024: 13.7 against 17.2 us at BT 1024, 46 against 57 at 8192; 336 x
//    128 33 against 45 at BT 6427), 64 rows and 8 waves beyond (1001 x 1503, 384 tiles of
//    32 rows: 20.2 against 16.1 us at BT 512, 100 against 72 at 8192);
//  - everything else of at least 8 x 16 is the split kernel's (3000 x 3000, where K is no
//    multiple of 16: 300 us at BT 8192, 527 through registers).
inline bool act8_ring(const KArgs8& a) { return a.x_dma && a.vec_state && a.K % 4 == 0; }
inline bool act8_split(const KArgs8& a, bool ring) {
  return a.N >= 8 && a.K >= 16 && (!ring || ((int64_t)a.tiles_n * a.tiles_k < 256 && a.BT >= 128));
}
inline bool act8_few(const KArgs8& a) { return ((int64_t)a.N + 31) / 32 * a.tiles_k <= 256; }
inline bool act8_wide(const KArgs8& a) {
  return a.BT >= WIDE_MIN_BT && (int64_t)((a.N + 255) / 256) * ((a.K + 255) / 256) >= 192;
}
template <int ROWS>
inline dim3 split_grid(const KArgs8& a) {
  return dim3((unsigned)((a.N + ROWS - 1) / ROWS * a.tiles_k));
}

template <int XF, int O, int M, int V>
hipError_t fused_act8_dma(const KArgs8& a, int w_fmt, hipStream_t st) {
#define FORGE_ACT8_DMA(WF, BLK, FULL)                                                                                 \
  hipLaunchKernelGGL((k_fused_act8_dma<XF, O, WF, M, V, BLK, FULL>), tile_grid(a), dim3(NT), 0, st, a);               \
  return hipGetLastError();
  if (act8_wide(a)) {   // (combo_fused's variants)
    const dim3 g((unsigned)(((a.N + 255) / 256) * ((a.K + 255) / 256)));
    if constexpr (full_pays(M, V)) {
      if (whole_tiles(a) && w_fmt == FMT_BF16) {
        hipLaunchKernelGGL((k_fused_act8_wide<XF, O, FMT_BF16, M, V, true>), g, dim3(2 * NT), 0, st, a);
        return hipGetLastError();
      }
    }
    if (w_fmt == FMT_BF16) hipLaunchKernelGGL((k_fused_act8_wide<XF, O, FMT_BF16, M, V, false>), g, dim3(2 * NT), 0, st, a);
    else hipLaunchKernelGGL((k_fused_act8_wide<XF, O, FMT_F32, M, V, false>), g, dim3(2 * NT), 0, st, a);
    return hipGetLastError();
  }
  if (w_fmt == FMT_BF16) {
    // the variants of k_fused that pay with a bf16 weight (combo_fused)
    if constexpr (fmt_blocked(M)) {
      if (a.block == 128 && whole_tiles(a)) { FORGE_ACT8_DMA(FMT_BF16, 128, true) }
    } else if constexpr (full_pays(M, V) && !(M == FMT_F32 && V == FMT_F32)) {
      if (whole_tiles(a)) { FORGE_ACT8_DMA(FMT_BF16, 0, true) }
    }
    FORGE_ACT8_DMA(FMT_BF16, 0, false)
  }
  FORGE_ACT8_DMA(FMT_F32, 0, false)
#undef FORGE_ACT8_DMA
}

template <int O, int M, int V>
hipError_t combo_fused_act8(const KArgs8& a, int w_fmt, hipStream_t st) {
  if (w_fmt != FMT_BF16 && w_fmt != FMT_F32) return hipErrorInvalidValue;
  const bool wbf = w_fmt == FMT_BF16, ring = act8_ring(a);
  if (act8_split(a, ring)) {
    if (act8_few(a)) {
      if (wbf) hipLaunchKernelGGL((k_fused_act8_split<32, 16, O, FMT_BF16, M, V>), split_grid<32>(a), dim3(1024), 0, st, a);
      else hipLaunchKernelGGL((k_fused_act8_split<32, 16, O, FMT_F32, M, V>), split_grid<32>(a), dim3(1024), 0, st, a);
    } else {
      if (wbf) hipLaunchKernelGGL((k_fused_act8_split<64, 8, O, FMT_BF16, M, V>), split_grid<64>(a), dim3(512), 0, st, a);
      else hipLaunchKernelGGL((k_fused_act8_split<64, 8, O, FMT_F32, M, V>), split_grid<64>(a), dim3(512), 0, st, a);
    }
  } else if (ring) {
    return a.x_fmt == FMT_S8 ? fused_act8_dma<FMT_S8, O, M, V>(a, w_fmt, st)
                             : fused_act8_dma<FMT_E4M3, O, M, V>(a, w_fmt, st);
  } else if (wbf) {
    hipLaunchKernelGGL((k_fused_act8_tiny<O, FMT_BF16, M, V>), tile_grid(a), dim3(NT), 0, st, a);
  } else {
    hipLaunchKernelGGL((k_fused_act8_tiny<O, FMT_F32, M, V>), tile_grid(a), dim3(NT), 0, st, a);
  }
  return hipGetLastError();
}
#define FORGE_INSTANTIATE_ACT8(O, M, V) \
  template hipError_t combo_fused_act8<O, M, V>(const KArgs8&, int, hipStream_t);

}  // namespace forge
