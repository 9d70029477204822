// row_quant.cuh — quantisation of a row held in registers, shared by the norm
// and the cache write.  The scales and codes are those of quant_math.cuh,
// except for a row with a NaN or an infinity: its scale is NaN and its codes
// are 0, so that it reads back as NaN and its codes stay finite (a cached row
// that a mask hides must not reach a sum: 0 * code is 0, 0 * NaN is not).
#pragma once
#include "quant_math.cuh"

namespace qg {

// Maximum of the magnitudes' bit patterns: ordered like the magnitudes, with
// infinity and NaN above every finite value.
__device__ __forceinline__ uint32_t absmax_bits8(const float (&x)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7fffffffu);
  return m;
}

template <bool INT8>
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
  if (amax_bits >= 0x7f800000u) return __uint_as_float(0x7fc00000u);
  return scale_of_amax<INT8>(__uint_as_float(amax_bits));
}

template <bool INT8>
__device__ __forceinline__ uint2 row_codes(const float (&x)[8], float s) {
  if (s != s) return make_uint2(0u, 0u);
  return quant8<INT8>(x, s);
}

// Byte offset of scale (r, c) in the 128x4 tiled NVFP4 layout of C columns.
__device__ __forceinline__ size_t sf_offset(int r, int c, int C) {
  const size_t atom = (size_t)(r / 128) * (C / 4) + (c / 4);
  return atom * 512 + (r % 32) * 16 + ((r % 128) / 32) * 4 + (c % 4);
}

}  // namespace qg
