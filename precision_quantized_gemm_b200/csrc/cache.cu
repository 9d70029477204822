// cache.cu — the quantised key / value cache: keys and values quantised per
// (token, head) as they are written, with the rotation of queries and keys in
// the same pass, and rows read back as bf16.
//
// Rotation of channel pair j by theta = position * frequency[j]:
//   (a, b) -> magnitude * (a cos - b sin, b cos + a sin),
// the pair being (j, j + R/2) or (2j, 2j + 1) of the head's first R channels.
// theta is formed and reduced to half a turn in 64 bits (a far position times
// a frequency near 1 has no fraction left in 32), then cos and sin are fp32.
// The rotated key is quantised from fp32: its only rounding is the code's.
//
// Bound: HBM for many tokens, latency for few.  A row of head_dim elements is
// head_dim / 8 neighbouring lanes of 8 elements, so amax is a shuffle; cos and
// sin of a token are computed once per CTA and shared.
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

constexpr int kThreads = 256;

template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheWriteParams p) {
  constexpr int L = D / 8;            // lanes per row
  constexpr int ROWS = kThreads / L;  // rows per pass of the CTA
  __shared__ float2 turn[D / 2];      // (cos, sin) * magnitude
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.x;
  const int half = p.rope_dim / 2;
  if ((int)threadIdx.x < half) {
    // whole turns drop out exactly: r = rint(x) and x - r are exact in 64 bits
    const double x = (double)__ldg(p.positions + t) * (__ldg(p.frequency + threadIdx.x) * 0.15915494309189535);
    float s, c;
    sincospif(2.f * (float)(x - rint(x)), &s, &c);
    turn[threadIdx.x] = make_float2(c * p.magnitude, s * p.magnitude);
  }
  __syncthreads();
  const int lane = threadIdx.x % L;
  const int slot = __ldg(p.slots + t);
  const bool store = slot >= 0 && slot < p.slots_total;
  const int rows = p.q_heads + 2 * p.kv_heads;
  for (int r0 = blockIdx.y * ROWS; r0 < rows; r0 += gridDim.y * ROWS) {
    const int r = r0 + threadIdx.x / L;
    const bool live = r < rows;
    const bool is_q = r < p.q_heads, is_k = !is_q && r < p.q_heads + p.kv_heads;
    const int h = is_q ? r : (is_k ? r - p.q_heads : r - p.q_heads - p.kv_heads);
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (live) {
      const __nv_bfloat16* src = is_q   ? p.q + (size_t)t * p.ldq
                                 : is_k ? p.k + (size_t)t * p.ldk
                                        : p.v + (size_t)t * p.ldv;
      unpack8(reinterpret_cast<const uint4*>(src + h * D)[lane], x);
    }
    if (half > 0) {
      const bool rot = (is_q || is_k) && lane * 8 < p.rope_dim;
      if (p.interleaved) {
        if (rot) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float2 cs = turn[lane * 4 + j];
            const float a = x[2 * j], b = x[2 * j + 1];
            x[2 * j] = a * cs.x - b * cs.y;
            x[2 * j + 1] = b * cs.x + a * cs.y;
          }
        }
      } else {
        // the partner of channel j is R/2 channels away: R/16 lanes (R % 16 == 0)
        const int step = p.rope_dim / 16;
        const bool low = lane < step;
        const int partner = rot ? (low ? lane + step : lane - step) : lane;
        const int from = (threadIdx.x & 31) - lane + partner;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float other = __shfl_sync(0xffffffffu, x[j], from);
          if (rot) {
            const float2 cs = turn[(low ? lane : lane - step) * 8 + j];
            x[j] = low ? x[j] * cs.x - other * cs.y : x[j] * cs.x + other * cs.y;
          }
        }
      }
    }
    Chunk y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = pack_f32x2(x[2 * j], x[2 * j + 1]);
    float a = absmax_chunk(y);
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) a = absmax_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
    if (!live) continue;
    if (is_q) {
      reinterpret_cast<uint4*>(p.q_out + (size_t)t * p.ldqo + h * D)[lane] = pack_chunk(y);
    } else if (store) {
      const size_t row = ((size_t)(slot >> p.page_shift) * p.kv_heads + h << p.page_shift) +
                         (slot & ((1 << p.page_shift) - 1));
      float s, inv;
      row_scale<INT8>(a, s, inv);
      if (lane == 0) (is_k ? p.k_scale : p.v_scale)[row] = s;
      reinterpret_cast<uint2*>((is_k ? p.k_codes : p.v_codes) + row * D)[lane] = chunk_codes<INT8>(y, s, inv);
    }
  }
}

// 16 codes -> 16 bf16 values, each the fp32 product code * scale rounded once.
template <bool INT8>
__device__ __forceinline__ void dequant16(const uint4& c, float s, uint4 (&out)[2]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  __nv_bfloat162* o = reinterpret_cast<__nv_bfloat162*>(out);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[4];
    if constexpr (INT8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) f[j] = (float)(int8_t)(w[i] >> (8 * j));
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t h2;
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"((uint16_t)(w[i] >> (16 * j))));
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h2));
        f[2 * j] = v.x;
        f[2 * j + 1] = v.y;
      }
    }
    o[2 * i] = __floats2bfloat162_rn(f[0] * s, f[1] * s);
    o[2 * i + 1] = __floats2bfloat162_rn(f[2] * s, f[3] * s);
  }
}

// One row (token, head, key or value) per D / 16 neighbouring lanes.
template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const CacheReadParams p) {
  constexpr int L = D / 16;
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x % L;
  const long long rows = (long long)p.tokens * p.kv_heads;
  for (long long r = (long long)blockIdx.x * (kThreads / L) + threadIdx.x / L; r < rows;
       r += (long long)gridDim.x * (kThreads / L)) {
    const int t = (int)(r / p.kv_heads), h = (int)(r % p.kv_heads);
    const int slot = __ldg(p.slots + t);
    uint4 k[2], v[2];
    if (slot >= 0 && slot < p.slots_total) {
      const size_t row = ((size_t)(slot >> p.page_shift) * p.kv_heads + h << p.page_shift) +
                         (slot & ((1 << p.page_shift) - 1));
      const uint4 kc = reinterpret_cast<const uint4*>(p.k_codes + row * D)[lane];
      const uint4 vc = reinterpret_cast<const uint4*>(p.v_codes + row * D)[lane];
      dequant16<INT8>(kc, p.k_scale[row], k);
      dequant16<INT8>(vc, p.v_scale[row], v);
    } else {
      k[0] = k[1] = v[0] = v[1] = make_uint4(0u, 0u, 0u, 0u);
    }
    uint4* ko = reinterpret_cast<uint4*>(p.k + (size_t)t * p.ldk + h * D) + lane * 2;
    uint4* vo = reinterpret_cast<uint4*>(p.v + (size_t)t * p.ldv + h * D) + lane * 2;
    ko[0] = k[0];
    ko[1] = k[1];
    vo[0] = v[0];
    vo[1] = v[1];
  }
}

template <class P>
cudaError_t launch(void (*fn)(P), const P& p, dim3 grid, cudaStream_t st, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, fn, p);
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteParams& p, int tokens, int head_dim, bool int8, cudaStream_t st,
                               bool pdl) {
  const int rows = p.q_heads + 2 * p.kv_heads;
  const int per = kThreads / (head_dim / 8);
  // few tokens: a CTA per pass of its rows, so that no pass waits for another
  const int parts = tokens <= 2 * 148 ? (rows + per - 1) / per : 1;
  const dim3 grid(tokens, parts);
  auto fn = head_dim == 128 ? (int8 ? cache_write_kernel<128, true> : cache_write_kernel<128, false>)
                            : (int8 ? cache_write_kernel<64, true> : cache_write_kernel<64, false>);
  return launch(fn, p, grid, st, pdl);
}

cudaError_t launch_cache_read(const CacheReadParams& p, int head_dim, bool int8, cudaStream_t st, bool pdl) {
  const int per = kThreads / (head_dim / 16);
  const long long ctas = ((long long)p.tokens * p.kv_heads + per - 1) / per;
  const dim3 grid((unsigned)(ctas < (1 << 30) ? ctas : (1 << 30)));
  auto fn = head_dim == 128 ? (int8 ? cache_read_kernel<128, true> : cache_read_kernel<128, false>)
                            : (int8 ? cache_read_kernel<64, true> : cache_read_kernel<64, false>);
  return launch(fn, p, grid, st, pdl);
}

}  // namespace qg
