// row_quant.cuh — quantisation of a row held in registers, shared by the norm
// and the cache write.  The scales and codes are those of quant_math.cuh,
// except for a row with a NaN or an infinity: its scale is NaN and its codes
// are 0, so that it reads back as NaN and its codes stay finite (a cached row
// that a mask hides must not reach a sum: 0 * code is 0, 0 * NaN is not).
#pragma once
#include "f32x2.cuh"
#include "loads.cuh"
#include "ptx.cuh"
#include "quant_math.cuh"

namespace qg {

// Eight fp32 values as four packed pairs (the two-wide arithmetic of sm_100).
using Chunk = uint64_t[4];
__device__ __forceinline__ void unpack_chunk(const uint4& v, Chunk& x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("mov.b64 %0, {%1, %2};" : "=l"(x[i]) : "r"(w[i] << 16), "r"(w[i] & 0xffff0000u));
}
__device__ __forceinline__ uint4 pack_chunk(const Chunk& x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack_f32x2(x[i], a, b);
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The larger magnitude, NaN if either is NaN (fmaxf would drop it); the sign
// is of no meaning.
__device__ __forceinline__ float absmax_nan(float m, float x) {
  float r;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(m), "f"(x));
  return r;
}
__device__ __forceinline__ float absmax_chunk(const Chunk& x) {
  float m[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    unpack_f32x2(x[i], a, b);
    m[i] = absmax_nan(a, b);
  }
  return absmax_nan(absmax_nan(m[0], m[1]), absmax_nan(m[2], m[3]));
}

// Scale of a row, and its reciprocal: correctly rounded, or 0 for a scale below
// kSmallScale, whose codes are divided.  An operand's scale is the
// quantisers' divided one.  A cached row's (CACHED) is the product with the
// rounded 1 / 448 or 1 / 127, which is how a division by a constant is
// computed for tensors: the two differ by a unit in the last place at most,
// but bf16 values lie on the ties of the codes often (1 in 16 where amax is
// 1.75 times a power of two), and a tie goes the way its scale leans.
constexpr float kSmallScale = 8.077935669463161e-28f;  // 2^-90
template <bool INT8, bool CACHED>
__device__ __forceinline__ void row_scale(float amax, float& s, float& inv) {
  amax = fabsf(amax);
  if (!(amax <= 3.402823466e38f)) {
    s = __uint_as_float(0x7fc00000u);
    inv = 0.f;
  } else {
    if constexpr (CACHED) s = amax > 0.f ? __fmul_rn(amax, 1.f / (INT8 ? 127.f : 448.f)) : 1.f;
    else s = scale_of_amax<INT8>(amax);
    inv = s >= kSmallScale ? __fdiv_rn(1.f, s) : 0.f;
  }
}

// Codes of 8 values, low byte first: round(x / s), as quant8 gives them; all
// zero for a row whose scale is NaN.
// The quotient is q = x inv, improved by its own remainder (P. Markstein's
// division, IBM J. Res. Dev. 34, 1990): with inv the correctly rounded 1 / s,
// q within a unit of x / s and r = x - q s exact (fma), q + r inv rounds as
// the division does.  (The plain product does not: it leaves the tie on one
// side or the other, and bf16 values over amax / 127 are ties often.)  Three
// two-wide instructions for two values.
// r is exact while its last bit, 2^-46 of q s, is one that fp32 has: the
// smallest quotient that is not far below every tie is 2^-10 (e4m3), so
// s >= 2^-149 + 46 + 10 = 2^-93 is enough.  Rows below 2^-90 are divided.
template <bool INT8>
__device__ __forceinline__ uint2 chunk_codes(const Chunk& x, float s, float inv) {
  if (s != s) return make_uint2(0u, 0u);
  float v[8];
  if (inv != 0.f) {
    const uint64_t k = pack_f32x2(inv, inv), ns = pack_f32x2(-s, -s);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t q = mul_f32x2(x[j], k);
      unpack_f32x2(fma_f32x2(fma_f32x2(q, ns, x[j]), k, q), v[2 * j], v[2 * j + 1]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      unpack_f32x2(x[j], v[2 * j], v[2 * j + 1]);
      v[2 * j] = __fdiv_rn(v[2 * j], s);
      v[2 * j + 1] = __fdiv_rn(v[2 * j + 1], s);
    }
  }
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (INT8) {
      // |x / s| <= 127 and a rounding: nothing to clamp but the pack's own range
      const int q[4] = {__float2int_rn(v[4 * h]), __float2int_rn(v[4 * h + 1]), __float2int_rn(v[4 * h + 2]),
                        __float2int_rn(v[4 * h + 3])};
      uint32_t r;
      asm("{\n\t.reg .b32 t;\n\tcvt.pack.sat.s8.s32.b32 t, %4, %3, 0;\n\tcvt.pack.sat.s8.s32.b32 %0, %2, %1, t;\n\t}"
          : "=r"(r)
          : "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3]));
      w[h] = r;
    } else {
      w[h] = cvt_e4m3x2(v[4 * h], v[4 * h + 1]) | (cvt_e4m3x2(v[4 * h + 2], v[4 * h + 3]) << 16);
    }
  }
  return make_uint2(w[0], w[1]);
}

// Byte offset of scale (r, c) in the 128x4 tiled NVFP4 layout of C columns.
__device__ __forceinline__ size_t sf_offset(int r, int c, int C) {
  const size_t atom = (size_t)(r / 128) * (C / 4) + (c / 4);
  return atom * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4 + (c % 4);
}

}  // namespace qg
