// gdn_mfma_op.h -- operands of the 16 x 16 matrix instructions as the serving
// operators use them: fragments of eight k-slots from rows staged in LDS, and
// f32 values as operands of bf16 products.
//
// Lane 16 g + n of a wave holds A[n][8 g + e] and B[8 g + e][n] (e = 0..7)
// and of a result D[4 g + e][n] (e = 0..3).  A product sums over its slots in
// any order, so a slot may stand for any k as long as A and B agree.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

namespace gdn {
namespace op {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Staged rows in LDS.  bf16: W entries a row, its 16-byte pieces permuted by
// an XOR with the row against bank conflicts (256 bytes a cycle): of a piece
// of 16 rows (fragments along the row), or, in a tile of kColumns that is
// only read transposed, of 32 bytes of eight rows.  (Transposed reads of the
// first kind, 64 bytes of eight rows in halves of pieces, take two cycles.)
// A row of fewer than 16 pieces shares its 256 bytes with the next ones.
// Permutations repeat every 16 rows, so a lane computes its offsets once.
// f32: rows one piece apart from a multiple of the banks.
template <typename TIn, int W, bool kColumns = false>
struct Tile {
  static constexpr int kPer = 16 / sizeof(TIn);  // entries per piece
  static constexpr int kPieces = W / kPer;
  static constexpr bool kSwizzled = sizeof(TIn) == 2;
  static constexpr int kPitch = kSwizzled ? W : W + kPer;
  // Entry offset of piece p of row r.
  static __device__ __forceinline__ int at(int r, int p) {
    if constexpr (kSwizzled && kColumns) {
      if constexpr (kPieces >= 16) p ^= (r & 7) << 1;
      else if constexpr (kPieces == 8) p ^= (r >> 1 & 3) << 1;
    } else if constexpr (kSwizzled) {
      if constexpr (kPieces >= 16) p ^= (r & 3) << 2 | (r >> 2 & 3);
      else if constexpr (kPieces == 8) p ^= (r >> 1 & 1) << 2 | (r >> 2 & 3);
      else p ^= r >> 2 & 3;
    }
    return r * kPitch + p * kPer;
  }
};

// Infinities and NaN among inputs.  A product of the matrix cores takes its
// masked entries as zeros, and 0 times an infinity or a NaN is a NaN: rows
// that hold such values are found here and treated apart.
template <typename TIn>
struct Special {  // bits that a dword sets when one of its values is special
  static constexpr uint32_t kExp = sizeof(TIn) == 2 ? 0x7f807f80u : 0x7f800000u;
  static constexpr uint32_t kOne = sizeof(TIn) == 2 ? 0x00800080u : 0x00800000u;
  static constexpr uint32_t kHit = sizeof(TIn) == 2 ? 0x80008000u : 0x80000000u;
  uint32_t seen = 0;
  __device__ __forceinline__ void look(u32x4 w) {
#pragma unroll
    for (int e = 0; e < 4; ++e) seen |= (w[e] & kExp) + kOne;
  }
  __device__ __forceinline__ bool any() const { return seen & kHit; }
  // w with special values as zeros.
  static __device__ __forceinline__ u32x4 cleared(u32x4 w) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if constexpr (sizeof(TIn) == 2) {
        if ((w[e] & 0x7f80u) == 0x7f80u) w[e] &= 0xffff0000u;
        if ((w[e] & 0x7f800000u) == 0x7f800000u) w[e] &= 0xffffu;
      } else {
        if ((w[e] & kExp) == kExp) w[e] = 0;
      }
    }
    return w;
  }
};

__device__ __forceinline__ float value_of(uint16_t x) {
  return __uint_as_float((uint32_t)x << 16);
}
__device__ __forceinline__ float value_of(float x) { return x; }

// Operand fragments of eight k-slots.  Raw: inputs as they are; Wide: f32
// values.
template <typename TIn>
struct Op;

template <>
struct Op<uint16_t> {
  typedef u32x4 Raw;
  static constexpr int kParts = 3;
  struct Wide {
    u32x4 part[kParts];
  };
  static __device__ __forceinline__ f32x4 mul(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(
        __builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0,
        0);
  }
  // A product with a wide operand takes kSteps instructions, smallest part
  // first; run a step over several accumulators before the next one, and no
  // instruction waits for the one before it.
  static constexpr int kSteps = kParts;
  static __device__ __forceinline__ f32x4 step(int i, const Wide& a, u32x4 b,
                                               f32x4 c) {
    return mul(a.part[kParts - 1 - i], b, c);
  }
  static __device__ __forceinline__ f32x4 step(int i, u32x4 a, const Wide& b,
                                               f32x4 c) {
    return mul(a, b.part[kParts - 1 - i], c);
  }
  static __device__ __forceinline__ f32x4 mul(const Wide& a, u32x4 b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) c = step(i, a, b, c);
    return c;
  }
  static __device__ __forceinline__ f32x4 mul(u32x4 a, const Wide& b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < kSteps; ++i) c = step(i, a, b, c);
    return c;
  }
  // x as the sum of its upper 8 bits, the next 8 and the last 8: the high
  // halves of x, of x minus the first part, and of what is left then.
  static __device__ __forceinline__ Wide wide(f32x4 x, f32x4 y) {
    Wide w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = i < 2 ? x[2 * i] : y[2 * i - 4];
      float b = i < 2 ? x[2 * i + 1] : y[2 * i - 3];
#pragma unroll
      for (int part = 0; part < kParts; ++part) {
        const uint32_t ua = __float_as_uint(a), ub = __float_as_uint(b);
        w.part[part][i] = __builtin_amdgcn_perm(ub, ua, 0x07060302u);
        a -= __uint_as_float(ua & 0xffff0000u);
        b -= __uint_as_float(ub & 0xffff0000u);
      }
    }
    return w;
  }
  // Slot i of the value whose parts are given.
  static __device__ __forceinline__ float slot(const u32x4 (&part)[kParts],
                                               int i) {
    float x = 0.f;
#pragma unroll
    for (int y = kParts - 1; y >= 0; --y) {
      uint32_t w = part[y][0];
#pragma unroll
      for (int k = 1; k < 4; ++k) w = i >> 1 == k ? part[y][k] : w;
      x += __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
    }
    return x;
  }
  // Slots e = 0..7 of a raw fragment as f32, times s.
  static __device__ __forceinline__ Wide scaled(u32x4 a, f32x4 s0, f32x4 s1) {
    f32x4 x, y;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      x[2 * i] = __uint_as_float(a[i] << 16) * s0[2 * i];
      x[2 * i + 1] = __uint_as_float(a[i] & 0xffff0000u) * s0[2 * i + 1];
      y[2 * i] = __uint_as_float(a[2 + i] << 16) * s1[2 * i];
      y[2 * i + 1] = __uint_as_float(a[2 + i] & 0xffff0000u) * s1[2 * i + 1];
    }
    return wide(x, y);
  }
  // Entries 8 p .. 8 p + 7 of row r0 + r (r0 a multiple of 16).
  template <typename TL>
  static __device__ __forceinline__ u32x4 row(const uint16_t* tile, int r0,
                                              int r, int p) {
    return *reinterpret_cast<const u32x4*>(tile + TL::at(r, p) +
                                           r0 * TL::kPitch);
  }
  // Column reads.  Lane 16 g + i receives rows 4 g .. 4 g + 3 (first half of
  // the slots) and 16 + 4 g .. 16 + 4 g + 3 (second), counted from row r0 (a
  // multiple of 32), of column col0 + step * (i / 4) + i % 4.  The
  // transposing LDS read hands lane i of 16 entry i % 4 of the 8 bytes
  // addressed by lane 4 e + i / 4 of them as its entry e, so lane i addresses
  // row 4 g + i / 4, entries col0 + step * (i % 4) and the three after it.
  template <typename TL>
  static __device__ __forceinline__ u32x4 column(const uint16_t* tile, int r0,
                                                 int col0, int step, int lane) {
    const int r = 4 * (lane >> 4) + ((lane & 15) >> 2);
    const int c = col0 + step * (lane & 3);
    const uint16_t* p = tile + TL::at(r, c >> 3) + (c & 7) + r0 * TL::kPitch;
    const uint2 a = tr(p), b = tr(p + 16 * TL::kPitch);
    return u32x4{a.x, a.y, b.x, b.y};
  }
  static __device__ __forceinline__ uint2 tr(const uint16_t* p) {
    return __builtin_bit_cast(
        uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                   (__attribute__((address_space(3))) s16x4*)p));
  }
};

template <>
struct Op<float> {
  static constexpr int kParts = 2;  // slots 0..3 and 4..7
  struct Raw {
    u32x4 part[kParts];
    __device__ __forceinline__ float at(int e) const {
      return __uint_as_float(part[e / 4][e % 4]);
    }
  };
  typedef Raw Wide;
  static constexpr int kSteps = 8;
  static __device__ __forceinline__ f32x4 step(int e, const Raw& a,
                                               const Raw& b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x4f32(a.at(e), b.at(e), c, 0, 0, 0);
  }
  static __device__ __forceinline__ f32x4 mul(const Raw& a, const Raw& b,
                                              f32x4 c) {
#pragma unroll
    for (int e = 0; e < kSteps; ++e) c = step(e, a, b, c);
    return c;
  }
  static __device__ __forceinline__ Raw wide(f32x4 x, f32x4 y) {
    return {__builtin_bit_cast(u32x4, x), __builtin_bit_cast(u32x4, y)};
  }
  static __device__ __forceinline__ float slot(const u32x4 (&part)[kParts],
                                               int i) {
    uint32_t w = part[0][0];
#pragma unroll
    for (int k = 1; k < 8; ++k) w = i == k ? part[k / 4][k % 4] : w;
    return __uint_as_float(w);
  }
  static __device__ __forceinline__ Raw scaled(const Raw& a, f32x4 s0,
                                               f32x4 s1) {
    return wide(__builtin_bit_cast(f32x4, a.part[0]) * s0,
                __builtin_bit_cast(f32x4, a.part[1]) * s1);
  }
  template <typename TL>
  static __device__ __forceinline__ Raw row(const float* tile, int r0, int r,
                                            int p) {
    const u32x4* at = reinterpret_cast<const u32x4*>(
        tile + (r0 + r) * TL::kPitch + 8 * p);
    return {at[0], at[1]};
  }
  template <typename TL>
  static __device__ __forceinline__ Raw column(const float* tile, int r0,
                                               int col0, int step, int lane) {
    const int i = lane & 15;
    const float* p = tile + (r0 + 4 * (lane >> 4)) * TL::kPitch + col0 +
                     step * (i >> 2) + (i & 3);
    Raw r;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      r.part[0][e] = __float_as_uint(p[e * TL::kPitch]);
      r.part[1][e] = __float_as_uint(p[(16 + e) * TL::kPitch]);
    }
    return r;
  }
};

}  // namespace op
}  // namespace gdn
