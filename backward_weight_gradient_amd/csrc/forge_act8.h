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

// 8 elements of a row at column c of type FMT (F32 / BF16) as fp32; columns from
// K on are 0.  p: the row's element 0.  WHOLE: K % 8 == 0 (or K = 0), so 8 columns
// are inside or outside together and no element-wise tail is compiled.
template <int FMT, bool WHOLE = false>
__device__ __forceinline__ void row_load8(const void* p, int64_t c, int64_t K, float (&x)[8]) {
  if constexpr (FMT == FMT_F32) {
    const float* q = static_cast<const float*>(p) + c;
    f32x4 a = {0.f, 0.f, 0.f, 0.f}, b = a;
    if (c + 8 <= K) {
      a = *reinterpret_cast<const f32x4_u*>(q);
      b = *reinterpret_cast<const f32x4_u*>(q + 4);
    } else if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (c + i < K) a[i] = q[i];
        if (c + 4 + i < K) b[i] = q[4 + i];
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) { x[i] = a[i]; x[4 + i] = b[i]; }
  } else {
    const uint16_t* q = static_cast<const uint16_t*>(p) + c;
    u32x4 a = {0u, 0u, 0u, 0u};
    if (c + 8 <= K) {
      a = *reinterpret_cast<const u32x4_u*>(q);
    } else if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < K) a[i >> 1] |= (uint32_t)q[i] << (16 * (i & 1));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(a[i] << 16);
      x[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

// The reverse: 8 values rounded to FMT (nearest even); columns from K on are not written.
template <int FMT, bool WHOLE = false>
__device__ __forceinline__ void row_store8(void* p, int64_t c, int64_t K, const float (&x)[8]) {
  if constexpr (FMT == FMT_F32) {
    float* q = static_cast<float*>(p) + c;
    if (c + 8 <= K) {
      *reinterpret_cast<f32x4_u*>(q) = f32x4{x[0], x[1], x[2], x[3]};
      *reinterpret_cast<f32x4_u*>(q + 4) = f32x4{x[4], x[5], x[6], x[7]};
    } else if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < K) q[i] = x[i];
    }
  } else {
    uint16_t* q = static_cast<uint16_t*>(p) + c;
    const u32x4 w = {bf16x2_rne(x[0], x[1]), bf16x2_rne(x[2], x[3]), bf16x2_rne(x[4], x[5]), bf16x2_rne(x[6], x[7])};
    if (c + 8 <= K) {
      *reinterpret_cast<u32x4_u*>(q) = w;
    } else if constexpr (!WHOLE) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < K) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
  }
}

// Store 8 codes of a row; columns from K on are not written.
template <bool WHOLE = false>
__device__ __forceinline__ void codes_store8(uint8_t* p, int64_t c, int64_t K, u32x2 w) {
  if (c + 8 <= K) {
    *reinterpret_cast<u32x2_u*>(p + c) = w;
  } else if constexpr (!WHOLE) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (c + i < K) p[c + i] = (uint8_t)(w[i >> 2] >> (8 * (i & 3)));
  }
}
__device__ __forceinline__ u32x2 codes_load8(const uint8_t* p, int64_t c, int64_t K) {
  if (c + 8 <= K) return *reinterpret_cast<const u32x2_u*>(p + c);
  u32x2 w = {0u, 0u};
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (c + i < K) w[i >> 2] |= (uint32_t)p[c + i] << (8 * (i & 3));
  return w;
}

// Quantise and store the 8 values at column c of row r, the lane's share of a
// block that spans 2^sh / 8 adjacent lanes (values from K on are 0).  Every lane
// of a block's group must call this together.
template <int FMT, bool WHOLE = false>
__device__ __forceinline__ void act8_store8(const Act8& q, int64_t r, int64_t c, int64_t K, const float (&x)[8]) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) a = max(a, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  a = q.sh == 7 ? lanes16_max(a) : q.sh == 6 ? lanes8_max(a) : lanes4_max(a);
  const uint32_t byte = act8_scale_byte<FMT>(a);
  const u32x2 w = act8_encode<FMT>(x, act8_inv(byte), byte == ACT8_NAN);
  if (c >= K) return;
  codes_store8<WHOLE>(q.codes + r * q.ld, c, K, w);
  if ((c & ((1 << q.sh) - 1)) == 0) q.scale[r * q.nb + (c >> q.sh)] = (uint8_t)byte;
}

}  // namespace forge
