// 8-bit activations (forge_act8): codes with one power-of-two scale byte per
// block of a row, on the device.  x is held as code * 2^e.
#pragma once

#include "forge_device.h"

namespace forge {

// 16- and 8-byte accesses at element alignment: gfx950 takes vector loads and
// stores of global memory at any byte address.
typedef uint32_t u32x4_u __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t u32x2_u __attribute__((ext_vector_type(2), aligned(1)));
typedef float f32x4_u __attribute__((ext_vector_type(4), aligned(4)));

// Row and column of a workgroup's tile, 8 rows of tiles at a time, each row on one XCD
// (workgroups go to the 8 XCDs in turn): neighbours in a row share the lines at their
// seam in that XCD's cache.  The rows left over follow in plain order.
__device__ __forceinline__ void tile_by_xcd(int rows, int cols, int& ti, int& tj) {
  const int b = (int)blockIdx.x, g = b / (8 * cols);
  const bool whole = 8 * g + 8 <= rows;
  ti = whole ? 8 * g + (b & 7) : b / cols;
  tj = whole ? (b - 8 * g * cols) >> 3 : b - ti * cols;
}

constexpr int ACT8_EMIN = -120;           // smallest exponent: the smallest E4M3 step, 2^-9, stays exact in bf16 (2^-133)
constexpr uint32_t ACT8_NAN = 255;        // scale byte of a block that held an infinity or a NaN

__device__ __forceinline__ uint32_t lanes4_max(uint32_t x) {   // over aligned groups of 4 lanes
  return dpp_umax<0x4E>(dpp_umax<0xB1>(x));
}

// Scale byte of a block from the bit pattern of its absmax a: the exponent e of
// the smallest power of two with a <= Q 2^e.  Q = 127 is 1.984375 * 2^6 and 448
// is 1.75 * 2^8, so e is a's exponent minus 6 (8), plus one where a's fraction
// exceeds Q's: the addition carries into the exponent field exactly then.
// Infinities and NaNs have the patterns from 0x7F800000 on.
template <int FMT>
__device__ __forceinline__ uint32_t act8_scale_byte(uint32_t abits) {
  constexpr uint32_t FRAC = FMT == FMT_S8 ? 0x7E0000u : 0x600000u;
  constexpr int SH = FMT == FMT_S8 ? 6 : 8;
  const int e = (int)((abits + (0x7FFFFFu - FRAC)) >> 23) - SH;   // biased by 127
  return abits >= 0x7F800000u ? ACT8_NAN : (uint32_t)max(e, ACT8_EMIN + 127);
}

// 2^e of a scale byte (NaN for ACT8_NAN) and 2^-e (0 for ACT8_NAN).
__device__ __forceinline__ float act8_mul(uint32_t byte) {
  return __uint_as_float((byte << 23) | (byte == ACT8_NAN ? 0x400000u : 0u));
}
__device__ __forceinline__ float act8_inv(uint32_t byte) {
  return byte == ACT8_NAN ? 0.f : __uint_as_float((254u - byte) << 23);
}

// Codes of 8 values: x 2^-e rounded to nearest even.  x 2^-e is exact (or below
// half the smallest code's step); |x 2^-e| <= Q, so nothing saturates.  poison:
// the block's scale byte is ACT8_NAN.
template <int FMT>
__device__ __forceinline__ u32x2 act8_encode(const float (&x)[8], float inv, bool poison) {
  u32x2 w;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float y0 = x[4 * h] * inv, y1 = x[4 * h + 1] * inv, y2 = x[4 * h + 2] * inv, y3 = x[4 * h + 3] * inv;
    if constexpr (FMT == FMT_S8) {
      // the low byte of y + 1.5 * 2^23 is rint(y) in two's complement (|y| <= 127)
      const uint32_t b0 = __float_as_uint(y0 + 0x1.8p23f), b1 = __float_as_uint(y1 + 0x1.8p23f);
      const uint32_t b2 = __float_as_uint(y2 + 0x1.8p23f), b3 = __float_as_uint(y3 + 0x1.8p23f);
      w[h] = __builtin_amdgcn_perm(b1, b0, 0x0C0C0400u) | __builtin_amdgcn_perm(b3, b2, 0x04000C0Cu);
    } else {
      int c = __builtin_amdgcn_cvt_pk_fp8_f32(y0, y1, 0, false);
      w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(y2, y3, c, true);
    }
    w[h] = poison ? 0u : w[h];
  }
  return w;
}

// 4 codes as fp32 stored values, f = act8_mul(scale byte).
template <int FMT>
__device__ __forceinline__ void act8_decode4(uint32_t w, float f, float* x) {
  if constexpr (FMT == FMT_S8) {
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = (float)(int8_t)((w >> (8 * i)) & 0xFFu) * f;
  } else {
    e4m3_unpack4(w, x);
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] *= f;
  }
}

// 8 elements of a row of K at column c, of type FMT (F32 / BF16), as stored.  p: the
// row's element 0 (a row that exists: callers clamp the row).
// Loads and their decoding are apart, and neither has a branch that depends on the
// lane (but the skipped load of WHOLE): a load whose value is used inside such a
// branch is waited for there, one after another, where several should be in flight.
//  ROW_WHOLE: K % 8 == 0, so 8 columns are inside or outside together; outside is 0.
//  ROW_BIG: K >= 8; the load is of the 8 elements at min(c, K - 8), row_val8 shifts
//    those of the vector that K ends in into place and clears columns from K on.
//  ROW_ANY: ROW_BIG, and rows shorter than 8 element by element (decided at run time,
//    so each load stands in a branch of its own: for code off the hot path).
enum RowMode : int { ROW_ANY, ROW_BIG, ROW_WHOLE };

template <int FMT> struct Raw8;
template <> struct Raw8<FMT_F32> { f32x4 a, b; };
template <> struct Raw8<FMT_BF16> { u32x4 a; };

// STREAM: past the caches, for data that nothing reads again soon.
template <bool STREAM, class T>
__device__ __forceinline__ T load_as(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const T*>(p));
  else return *static_cast<const T*>(p);
}
template <int FMT, int MODE = ROW_ANY, bool STREAM = false>
__device__ __forceinline__ Raw8<FMT> row_raw8(const void* p, int64_t c, int64_t K) {
  Raw8<FMT> r;
  if constexpr (FMT == FMT_F32) r.a = r.b = f32x4{0.f, 0.f, 0.f, 0.f};
  else r.a = u32x4{0u, 0u, 0u, 0u};
  if constexpr (MODE == ROW_WHOLE) {
    if (c < K) {
      if constexpr (FMT == FMT_F32) {
        const float* q = static_cast<const float*>(p) + c;
        r.a = load_as<STREAM, f32x4_u>(q);
        r.b = load_as<STREAM, f32x4_u>(q + 4);
      } else {
        r.a = load_as<STREAM, u32x4_u>(static_cast<const uint16_t*>(p) + c);
      }
    }
  } else if (MODE == ROW_BIG || K >= 8) {
    const int64_t at = min(c, K - 8);
    if constexpr (FMT == FMT_F32) {
      const float* q = static_cast<const float*>(p) + at;
      r.a = load_as<STREAM, f32x4_u>(q);
      r.b = load_as<STREAM, f32x4_u>(q + 4);
    } else {
      r.a = load_as<STREAM, u32x4_u>(static_cast<const uint16_t*>(p) + at);
    }
  } else {
    for (int64_t i = K - 1; i >= 0; --i) {   // last element first, each pushing the others up
      if constexpr (FMT == FMT_F32) {
        r.b = f32x4{r.a[3], r.b[0], r.b[1], r.b[2]};
        r.a = f32x4{static_cast<const float*>(p)[i], r.a[0], r.a[1], r.a[2]};
      } else {
        r.a = u32x4{(r.a[0] << 16) | static_cast<const uint16_t*>(p)[i], (r.a[1] << 16) | (r.a[0] >> 16),
                    (r.a[2] << 16) | (r.a[1] >> 16), (r.a[3] << 16) | (r.a[2] >> 16)};
      }
    }
  }
  return r;
}

// 8 elements moved down by s places (0 .. 7; 8: all cleared), zeros above.
template <int FMT>
__device__ __forceinline__ Raw8<FMT> raw_shift8(Raw8<FMT> r, int s) {
  if constexpr (FMT == FMT_F32) {
    const f32x4 z = {0.f, 0.f, 0.f, 0.f};
    r.a = s & 4 ? r.b : r.a;
    r.b = s & 4 ? z : r.b;
    r.a = s & 2 ? f32x4{r.a[2], r.a[3], r.b[0], r.b[1]} : r.a;
    r.b = s & 2 ? f32x4{r.b[2], r.b[3], 0.f, 0.f} : r.b;
    r.a = s & 1 ? f32x4{r.a[1], r.a[2], r.a[3], r.b[0]} : r.a;
    r.b = s & 1 ? f32x4{r.b[1], r.b[2], r.b[3], 0.f} : r.b;
    r.a = s & 8 ? z : r.a;
    r.b = s & 8 ? z : r.b;
  } else {
    const u32x4 z = {0u, 0u, 0u, 0u};
    r.a = s & 4 ? u32x4{r.a[2], r.a[3], 0u, 0u} : r.a;
    r.a = s & 2 ? u32x4{r.a[1], r.a[2], r.a[3], 0u} : r.a;
    r.a = s & 1 ? u32x4{(r.a[0] >> 16) | (r.a[1] << 16), (r.a[1] >> 16) | (r.a[2] << 16),
                        (r.a[2] >> 16) | (r.a[3] << 16), r.a[3] >> 16}
                : r.a;
    r.a = s & 8 ? z : r.a;
  }
  return r;
}
// Elements that the load of row_raw8 began too early, 8 from K on (rows shorter than 8
// begin at 0: nothing to shift for c = 0).
template <int MODE = ROW_ANY>
__device__ __forceinline__ int row_early8(int64_t c, int64_t K) {
  return MODE == ROW_BIG || K >= 8 ? (int)min((int64_t)8, c - min(c, K - 8)) : c > 0 ? 8 : 0;
}
// The loaded elements in their places, as stored.
template <int FMT, int MODE = ROW_ANY>
__device__ __forceinline__ Raw8<FMT> row_place8(const Raw8<FMT>& r, int64_t c, int64_t K) {
  if constexpr (MODE == ROW_WHOLE) return r;
  else return raw_shift8<FMT>(r, row_early8<MODE>(c, K));
}
template <int FMT, int MODE = ROW_ANY>
__device__ __forceinline__ void row_val8(const Raw8<FMT>& raw, int64_t c, int64_t K, float (&x)[8]) {
  const Raw8<FMT> r = row_place8<FMT, MODE>(raw, c, K);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (FMT == FMT_F32) {
      x[i] = r.a[i];
      x[4 + i] = r.b[i];
    } else {
      x[2 * i] = __uint_as_float(r.a[i] << 16);
      x[2 * i + 1] = __uint_as_float(r.a[i] & 0xFFFF0000u);
    }
  }
}

template <int FMT, int MODE = ROW_ANY>
__device__ __forceinline__ void row_load8(const void* p, int64_t c, int64_t K, float (&x)[8]) {
  row_val8<FMT, MODE>(row_raw8<FMT, MODE>(p, c, K), c, K, x);
}

// The reverse: 8 values rounded to FMT (nearest even); columns from K on are not
// written (the vector that K ends in: 4, 2 and 1 elements as its length asks).
template <int FMT, int MODE = ROW_ANY>
__device__ __forceinline__ void row_store8(void* p, int64_t c, int64_t K, const float (&x)[8]) {
  if constexpr (FMT == FMT_F32) {
    float* q = static_cast<float*>(p) + c;
    if (c + 8 <= K) {
      *reinterpret_cast<f32x4_u*>(q) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4_u*>(q + 4) = f32x4{x[4], x[5], x[6], x[7]};
    } else if (MODE != ROW_WHOLE && c < K) {
      const int n = (int)(K - c);
      float y[4] = {x[0], x[1], x[2], x[3]};
      if (n & 4) {
        *reinterpret_cast<f32x4_u*>(q) = f32x4{y[0], y[1], y[2], y[3]};
        y[0] = x[4]; y[1] = x[5]; y[2] = x[6];
        q += 4;
      }
      if (n & 2) {
        q[0] = y[0];
        q[1] = y[1];
        y[0] = y[2];
        q += 2;
      }
      if (n & 1) q[0] = y[0];
    }
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + c;
    const u32x4 w = {bf16x2_rne(x[0], x[1]), bf16x2_rne(x[2], x[3]), bf16x2_rne(x[4], x[5]), bf16x2_rne(x[6], x[7])};
    if (c + 8 <= K) {
      *reinterpret_cast<u32x4_u*>(q) = w;
    } else if (MODE != ROW_WHOLE && c < K) {
      const int n = (int)(K - c);
      uint32_t y0 = w[0], y1 = w[1];
      if (n & 4) {
        *reinterpret_cast<u32x2_e*>(q) = u32x2_e{y0, y1};
        y0 = w[2];
        y1 = w[3];
        q += 4;
      }
      if (n & 2) {
        *reinterpret_cast<u32_e*>(q) = y0;
        y0 = y1;
        q += 2;
      }
      if (n & 1) q[0] = (uint16_t)y0;
    }
  }
}

// Store 8 codes of a row; columns from K on are not written.
template <int MODE = ROW_ANY>
__device__ __forceinline__ void codes_store8(uint8_t* p, int64_t c, int64_t K, u32x2 w) {
  uint8_t* q = p + c;
  if (c + 8 <= K) {
    *reinterpret_cast<u32x2_u*>(q) = w;
  } else if (MODE != ROW_WHOLE && c < K) {
    const int n = (int)(K - c);
    uint32_t y = w[0];
    if (n & 4) {
      *reinterpret_cast<u32_e*>(q) = y;
      y = w[1];
      q += 4;
    }
    if (n & 2) {
      q[0] = (uint8_t)y;
      q[1] = (uint8_t)(y >> 8);
      y >>= 16;
      q += 2;
    }
    if (n & 1) q[0] = (uint8_t)y;
  }
}
// 8 codes at column c, the same way: the load, then codes_val8.
template <int MODE = ROW_ANY>
__device__ __forceinline__ u32x2 codes_raw8(const uint8_t* p, int64_t c, int64_t K) {
  if (MODE == ROW_BIG || K >= 8) return *reinterpret_cast<const u32x2_u*>(p + min(c, K - 8));
  u32x2 w = {0u, 0u};
  for (int64_t i = K - 1; i >= 0; --i) w = u32x2{(w[0] << 8) | p[i], (w[1] << 8) | (w[0] >> 24)};
  return w;
}
template <int MODE = ROW_ANY>
__device__ __forceinline__ u32x2 codes_val8(u32x2 w, int64_t c, int64_t K) {
  const int s = MODE == ROW_BIG || K >= 8 ? (int)min((int64_t)8, c - min(c, K - 8)) : c > 0 ? 8 : 0;
  const uint32_t lo = s & 4 ? w[1] : w[0], hi = s & 4 ? 0u : w[1];
  const u32x2 v = {__builtin_amdgcn_alignbyte(hi, lo, s & 3), hi >> (8 * (s & 3))};
  return s & 8 ? u32x2{0u, 0u} : v;
}

// Quantise and store the 8 values at column c of row r, the lane's share of a
// block that spans 2^sh / 8 adjacent lanes (values from K on are 0).  Every lane
// of a block's group must call this together.
template <int FMT, int MODE = ROW_ANY>
__device__ __forceinline__ void act8_store8(const Act8& q, int64_t r, int64_t c, int64_t K, const float (&x)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  a = q.sh == 7 ? lanes16_max(a) : q.sh == 6 ? lanes8_max(a) : lanes4_max(a);
  const uint32_t byte = act8_scale_byte<FMT>(a);
  const u32x2 w = act8_encode<FMT>(x, act8_inv(byte), byte == ACT8_NAN);
  if (c >= K) return;
  codes_store8<MODE>(q.codes + r * q.ld, c, K, w);
  if ((c & ((1 << q.sh) - 1)) == 0) q.scale[r * q.nb + (c >> q.sh)] = (uint8_t)byte;
}

// s += the rows at(0) .. at(mine - 1) of an array of type FMT at column c, in order.
// at(i) is the address of a row's element 0, valid for every i (callers clamp it);
// count: the largest `mine` of the wave.  B or B / 2 rows are in flight at a time, those
// past the lane's own count read and left out, so no load waits for another.
template <int MODE, int FMT, int B, class AT>
__device__ __forceinline__ void sum_rows_batch(AT&& at, int m, int mine, int64_t c, int64_t K, float (&s)[8]) {
  Raw8<FMT> r[B];
#pragma unroll
  for (int u = 0; u < B; ++u) r[u] = row_raw8<FMT, MODE>(at(m + u), c, K);
#pragma unroll
  for (int u = 0; u < B; ++u) {
    float x[8];
    row_val8<FMT, MODE>(r[u], c, K, x);
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] = m + u < mine ? s[k] + x[k] : s[k];
  }
}
template <int MODE, int FMT, int B = 8, class AT>
__device__ __forceinline__ void sum_rows(AT&& at, int count, int mine, int64_t c, int64_t K, float (&s)[8]) {
  int m = 0;
  for (; count - m > B / 2; m += B) sum_rows_batch<MODE, FMT, B>(at, m, mine, c, K, s);
  if (count - m > 1) sum_rows_batch<MODE, FMT, B / 2>(at, m, mine, c, K, s);
  else if (count - m == 1) sum_rows_batch<MODE, FMT, 1>(at, m, mine, c, K, s);
}

}  // namespace forge
