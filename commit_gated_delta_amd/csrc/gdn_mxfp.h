// gdn_mxfp.h -- rows of a cache held in 4 bits: blocks of 32 channels, each
// with a scale 2^(b - 127) from a byte b and 32 codes of 4 bits (sign, two
// bits of exponent, one of fraction: 0, 0.5, 1, 1.5, 2, 3, 4, 6), two codes a
// byte, the even channel in the lower half.  These are the elements and
// scales that gfx950 converts itself.
#pragma once
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "gdn.h"

namespace gdnk {

struct Fp4Rows {
  uint8_t* codes;   // [rows][d / 2]
  uint8_t* scales;  // [rows][d / 32]
};

constexpr uint32_t kScaleNan = 255;  // every value of the block is a NaN
constexpr uint32_t kScaleMost = 251, kScaleLeast = 1;  // of what is written
// Blocks whose scale byte is at least this read as NaN (their largest values
// are past f32).
constexpr uint32_t kScaleOdd = 253;

// Cache rows are counted in 32 bits (2^32 of them fill the memory).
static bool rows_fit(const gdn_kv_dims& d) {
  return (double)d.n_pages * d.page_size * d.h_kv < 4294967296.0;
}

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t codes_u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  const bf16x2 r = {(__bf16)lo, (__bf16)hi};  // to nearest, ties to even
  return __builtin_bit_cast(uint32_t, r);
}

// What a block's values are multiplied by (byte 0: 2^-127, below the normal
// numbers; the conversions read the exponent field alone).
__device__ __forceinline__ float fp4_scale(uint32_t byte) {
  return __uint_as_float(byte << 23);
}

// Values of a dword of codes as four dwords of bf16 (exact: two significant
// bits).  The conversion gives NaN for byte 255.
__device__ __forceinline__ codes_u32x4 fp4_values(uint32_t codes,
                                                  uint32_t byte) {
  const float s = fp4_scale(byte);
  codes_u32x4 r;
  r[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 0));
  r[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 1));
  r[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 2));
  r[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, s, 3));
  return r;
}

// f64 to f32 with an odd last bit wherever something is cut off: rounded once
// more, to fewer bits, it comes out as the f64 number itself would (borders
// between codes and scales have even last bits).  Past f32 the largest number,
// not an infinity.
__device__ __forceinline__ float to_odd(double x) {
  const float f = (float)x;
  uint32_t u = __float_as_uint(f);
  if ((double)f != x) u = (u - (fabs((double)f) > fabs(x) ? 1 : 0)) | 1;
  return __uint_as_float(u);
}

// Codes of eight channels of a block whose other 24 are in the neighbouring
// lanes (four aligned lanes hold a block).  The scale is the smallest power
// of two that keeps the block's largest magnitude a <= 6 s; nothing is cut
// off then (below 6 2^124), and the nearest code is off by at most s / 4 of a
// magnitude up to 2 s, s / 2 up to 4 s and s up to 6 s.
struct Coded {
  uint32_t codes, scale;
};
template <int CTRL>
__device__ __forceinline__ uint32_t quad_max(uint32_t x) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, 0xf, 0xf, true);
  return o > x ? o : x;
}
__device__ __forceinline__ Coded fp4_code(const float (&x)[8]) {
  uint32_t a = 0;  // (magnitudes compare as their bits do, infinities and NaN above all)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t u = __float_as_uint(x[i]) & 0x7fffffffu;
    a = u > a ? u : a;
  }
  a = quad_max<0xB1>(a);  // quad_perm [1,0,3,2]
  a = quad_max<0x4E>(a);  // quad_perm [2,3,0,1]
  // a = f 2^k with 1 <= f < 2: 2^(k - 2) when f <= 1.5, else 2^(k - 1)
  int b = (int)(a >> 23) - 2 + ((a & 0x7fffffu) > 0x400000u);
  b = b < (int)kScaleLeast ? kScaleLeast : b > (int)kScaleMost ? kScaleMost : b;
  const bool finite = a < 0x7f800000u;
  const float s = fp4_scale((uint32_t)b);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], s, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], s, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], s, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], s, 3);
  return {finite ? w : 0u, finite ? (uint32_t)b : kScaleNan};
}

}  // namespace gdnk
