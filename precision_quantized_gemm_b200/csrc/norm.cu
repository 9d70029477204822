// norm.cu — the norms before and after a block, fused with the block's gate
// and scales, the residual sum and the quantisation of the next product's
// operand:
//   b = P(x) * g                 P: none, or a norm with the post weight
//   h = residual_scale * r + block_scale * b
//   y = N(h)                     N: RMS or LayerNorm with the pre weight
// h leaves as bf16, y as bf16 and / or as an operand of one of the four
// formats.  Every sum, h and y are fp32: h and y are each rounded once, y
// straight to the codes (no bf16 in between).
//
// Bound: HBM for many rows (each input read once, each output written once),
// latency for few.  One CTA owns a row, which stays in registers (chunks of 8
// elements per thread) between its up to five reductions.  16384 x 5120 with a
// post norm, to e4m3: 107 us, 5.5 TB/s (84 % of a copy's rate; as bf16 without
// the post norm 103 us, all of it); the issue slots are 66 % full (29
// instructions an element), so instructions are what else there is to save.
// 1 x 5120: 4.1 us in a graph, launch included.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"
#include "row_quant.cuh"

namespace qg {
namespace {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum / maximum over the CTA, the same in every thread.  Each call of a row
// takes its own 36 words of `red`, so one barrier is enough; the warps'
// partials are read four at a time (the last warp zeroes the fours' rest),
// which is a shorter chain than a second round of shuffles.
__device__ __forceinline__ void partial(float v, float* red) {
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (l == 0) red[w] = v;
  else if (w == warps - 1 && l < 4) red[w + l] = 0.f;
  __syncthreads();
}
__device__ __forceinline__ float cta_sum(float v, float* red) {
  partial(warp_sum(v), red);
  float s = 0.f;
  for (int i = 0; i < (int)(blockDim.x >> 5); i += 4) {
    const float4 p = *reinterpret_cast<const float4*>(red + i);
    s += (p.x + p.y) + (p.z + p.w);
  }
  return s;
}
// Of magnitudes, NaN kept: their bit patterns are ordered like them, NaN last.
__device__ __forceinline__ float cta_absmax(float v, float* red) {
  partial(__uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu)), red);
  float m = 0.f;
  for (int i = 0; i < (int)(blockDim.x >> 5); i += 4) {
    const float4 p = *reinterpret_cast<const float4*>(red + i);
    m = absmax_nan(absmax_nan(m, absmax_nan(p.x, p.y)), absmax_nan(p.z, p.w));
  }
  return m;
}

// x <- norm(x) * (w + offset) + b over the row's `nch` chunks.
// FULL: every thread has all CH chunks.
template <int CH, bool FULL>
__device__ __forceinline__ void norm_row(Chunk (&x)[CH], int nch, float inv_n, bool layer, float eps,
                                         const uint4* w, const uint4* b, float offset,
                                         float* red) {
  if (layer) {
    uint64_t s = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) s = add_f32x2(s, x[i][j]);
    float a, c;
    unpack_f32x2(s, a, c);
    const float mean = cta_sum(a + c, red) * inv_n;
    const uint64_t m = pack_f32x2(-mean, -mean);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const bool in = FULL || threadIdx.x + i * blockDim.x < nch;
#pragma unroll
      for (int j = 0; j < 4; ++j) x[i][j] = in ? add_f32x2(x[i][j], m) : 0ull;
    }
  }
  uint64_t q = 0;
#pragma unroll
  for (int i = 0; i < CH; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) q = fma_f32x2(x[i][j], x[i][j], q);
  float a, c;
  unpack_f32x2(q, a, c);
  const float r = rsqrtf(cta_sum(a + c, red + 36) * inv_n + eps);
  const uint64_t r2 = pack_f32x2(r, r), o2 = pack_f32x2(offset, offset);
  // what a call may leave out is asked for once, around the chunks: asked for
  // in each, it is issued all the same, with its lanes off
  auto scaled = [&](bool with_offset) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      if (FULL || at < nch) {
        Chunk v;
        unpack_chunk(fresh(w + at), v);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = mul_f32x2(mul_f32x2(x[i][j], r2), with_offset ? add_f32x2(v[j], o2) : v[j]);
      }
    }
  };
  if (offset != 0.f) scaled(true);
  else scaled(false);
  if (b != nullptr) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int at = threadIdx.x + i * blockDim.x;
      if (FULL || at < nch) {
        Chunk v;
        unpack_chunk(fresh(b + at), v);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[i][j] = add_f32x2(x[i][j], v[j]);
      }
    }
  }
}

template <int CH, bool FULL>
__global__ void __launch_bounds__(512, CH == 4 ? 2 : 1) norm_kernel(const NormParams p) {
  __shared__ __align__(16) float red[5 * 36];
  griddep_launch_dependents();
  griddep_wait();
  const int m = blockIdx.x;
  const int nch = p.N / 8;
  const bool nvf4 = p.format == QG_NVFP4;
  float g = 1.f;
  if (nvf4) {
    const float a = fresh(p.static_amax);
    g = a > 0.f ? __fdiv_rn(a, 2688.f) : 1.f;
    if (m == 0 && threadIdx.x == 0) *p.global_scale = g;
  }
  if (m >= p.M) {  // the scale rows that pad the last 128-row atom
    for (int c = threadIdx.x; c < p.sf_cols; c += blockDim.x)
      static_cast<uint8_t*>(p.scale)[sf_offset(m, c, p.sf_cols)] = 0;
    return;
  }
  const uint4* rr = p.residual ? reinterpret_cast<const uint4*>(p.residual + (size_t)m * p.ldr) : nullptr;
  const uint4* xr = p.x ? reinterpret_cast<const uint4*>(p.x + (size_t)m * p.ldx) : nullptr;
  const uint4* gr = p.gate ? reinterpret_cast<const uint4*>(p.gate + (size_t)m * p.ldg) : nullptr;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  uint4 rv[CH], xv[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int c = threadIdx.x + i * blockDim.x;
    rv[i] = rr && (FULL || c < nch) ? rr[c] : zero;
    xv[i] = xr && (FULL || c < nch) ? xr[c] : zero;
  }
  Chunk v[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) unpack_chunk(xv[i], v[i]);
  if (p.post_norm)
    norm_row<CH, FULL>(v, nch, p.inv_n, p.post_norm == QG_NORM_LAYER, p.eps, p.post_weight, p.post_bias, p.weight_offset,
                 red);
  const uint64_t bs = pack_f32x2(p.block_scale, p.block_scale), rs = pack_f32x2(p.residual_scale, p.residual_scale);
  if (gr != nullptr) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (FULL || c < nch) {
        Chunk gv;
        unpack_chunk(gr[c], gv);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][j] = mul_f32x2(v[i][j], gv[j]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    Chunk r;
    unpack_chunk(rv[i], r);
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i][j] = fma_f32x2(rs, r[j], mul_f32x2(bs, v[i][j]));
  }
  if (p.h != nullptr) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if (FULL || c < nch) reinterpret_cast<uint4*>(p.h + (size_t)m * p.ldh)[c] = pack_chunk(v[i]);
    }
  }
  if (!p.pre_norm) return;
  norm_row<CH, FULL>(v, nch, p.inv_n, p.pre_norm == QG_NORM_LAYER, p.eps, p.pre_weight, p.pre_bias, p.weight_offset,
               red + 72);
  if (p.y != nullptr) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if ((FULL || c < nch)) reinterpret_cast<uint4*>(p.y + (size_t)m * p.ldy)[c] = pack_chunk(v[i]);
    }
  }
  if (p.q == nullptr) return;
  if (p.format == QG_FP8_DYNAMIC || p.format == QG_W8A8_INT8) {
    float a = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) a = absmax_nan(a, absmax_chunk(v[i]));
    a = cta_absmax(a, red + 144);
    const bool int8 = p.format == QG_W8A8_INT8;
    float s, inv;
    if (int8) row_scale<true, false>(a, s, inv);
    else row_scale<false, false>(a, s, inv);
    if (threadIdx.x == 0) static_cast<float*>(p.scale)[m] = s;
    uint2* q = reinterpret_cast<uint2*>(p.q + (size_t)m * p.N);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      if ((FULL || c < nch)) q[c] = int8 ? chunk_codes<true>(v[i], s, inv) : chunk_codes<false>(v[i], s, inv);
    }
  } else if (p.format == QG_BLOCK_FP8) {
    // a 128-element group is 16 chunks, held by 16 neighbouring threads
    // (blockDim.x is a multiple of 32, N of 128)
    uint2* q = reinterpret_cast<uint2*>(p.q + (size_t)m * p.N);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      float a = absmax_chunk(v[i]);
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) a = absmax_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
      if ((FULL || c < nch)) {
        float s, inv;
        row_scale<false, false>(a, s, inv);
        if ((c & 15) == 0) static_cast<float*>(p.scale)[(size_t)m * (p.N / 128) + c / 16] = s;
        q[c] = chunk_codes<false>(v[i], s, inv);
      }
    }
  } else {
    // NVFP4: a 16-element block is two neighbouring threads' chunks
    uint32_t* q = reinterpret_cast<uint32_t*>(p.q + (size_t)m * (p.N / 2));
    uint8_t* sf = static_cast<uint8_t*>(p.scale);
#pragma unroll 1
    for (int i = 0; i < CH; ++i) {
      const int c = threadIdx.x + i * blockDim.x;
      float t[8];
#pragma unroll
      for (int e = 0; e < CH; ++e)
        if (e == i) {
#pragma unroll
          for (int j = 0; j < 4; ++j) unpack_f32x2(v[e][j], t[2 * j], t[2 * j + 1]);
        }
      const float own = absmax8(t);
      const float a = fmaxf(own, __shfl_xor_sync(0xffffffffu, own, 1));
      if ((FULL || c < nch)) {
        const uint32_t code = cvt_e4m3x2(__fdiv_rn(__fdiv_rn(a, 6.f), g), 0.f) & 0xFF;
        const float d = __fmul_rn(dec_e4m3(code), g);
        uint32_t packed = 0;
        if (d != 0.f) {
#pragma unroll
          for (int j = 0; j < 8; ++j) t[j] = __fdiv_rn(t[j], d);
          packed = cvt_e2m1x8(t);
        }
        q[c] = packed;
        if ((c & 1) == 0) sf[sf_offset(m, c / 2, p.sf_cols)] = (uint8_t)code;
      }
    }
    for (int c = p.N / 16 + threadIdx.x; c < p.sf_cols; c += blockDim.x) sf[sf_offset(m, c, p.sf_cols)] = 0;
  }
}

template <int CH>
cudaError_t launch_ch(const NormParams& p, int rows, int threads, cudaStream_t st, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(rows);
  cfg.blockDim = dim3(threads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, p.N == threads * CH * 8 ? norm_kernel<CH, true> : norm_kernel<CH, false>, p);
}

}  // namespace

cudaError_t launch_norm(const NormParams& p, cudaStream_t st, bool pdl) {
  const int nch = p.N / 8;
  // NVFP4 also writes the scale rows that pad the last 128-row atom
  const int rows = p.q != nullptr && p.format == QG_NVFP4 ? (p.M + 127) / 128 * 128 : p.M;
  auto threads = [&](int ch) { return ((nch + ch - 1) / ch + 31) / 32 * 32; };
  // Few rows, or narrow ones: two chunks a thread, the shorter chain (1 x 5120:
  // 4.3 us, 6.2 with four; 296 x 8192: 6.5, 8.3; 2048 x 1024: 6.2, 8.3; one
  // chunk is no shorter).  Many: four, which spread the reductions and scales
  // over more elements (16384 x 5120: 107 us, 139 with two; 2048: 45, 52; at
  // 16384 x 1024 both take 28 to 29).  Eight only where four would need more
  // than 512 threads (16384 x 8192: 170 us with eight, 167 with four).
  if (threads(2) <= (p.M <= 2 * 148 ? 512 : 64)) return launch_ch<2>(p, rows, threads(2), st, pdl);
  if (threads(4) <= 512) return launch_ch<4>(p, rows, threads(4), st, pdl);
  return launch_ch<8>(p, rows, threads(8), st, pdl);
}

}  // namespace qg
