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
// sin of a token are computed once per CTA and shared.  8191 tokens of 32 + 2 x
// 8 heads of 128: written in 40 us (4.6 TB/s, 71 % of a copy's rate; the warps
// wait for loads half of the time, and the issue slots are 64 % full).  100,000
// tokens of 8 heads read in 107 us (5.8 TB/s, 89 %).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"
#include "quant_math.cuh"
#include "row_quant.cuh"

namespace qg {
namespace {

constexpr int kThreads = 128;

// A lane's part in the rotation of its 8 channels: for halves the cosines and
// signed sines of the 8, with the partner's values a shuffle away; for pairs
// those of its 4 pairs.
struct Turn {
  uint64_t c[4], s[4];
  int from;    // lane of the partner (halves)
  bool on;
};
__device__ __forceinline__ void rotate(Chunk& x, const uint4& raw, const Turn& r, bool interleaved) {
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  if (interleaved) {
    if (r.on) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // (a, b) (c, c) + (b, a) (-s, s)
        const uint64_t swapped = pack_f32x2(__uint_as_float(w[j] & 0xffff0000u), __uint_as_float(w[j] << 16));
        x[j] = fma_f32x2(swapped, r.s[j], mul_f32x2(x[j], r.c[j]));
      }
    }
  } else {
    uint4 o;
    o.x = __shfl_sync(0xffffffffu, w[0], r.from);
    o.y = __shfl_sync(0xffffffffu, w[1], r.from);
    o.z = __shfl_sync(0xffffffffu, w[2], r.from);
    o.w = __shfl_sync(0xffffffffu, w[3], r.from);
    if (r.on) {
      Chunk y;
      unpack_chunk(o, y);
#pragma unroll
      for (int j = 0; j < 4; ++j) x[j] = fma_f32x2(y[j], r.s[j], mul_f32x2(x[j], r.c[j]));
    }
  }
}

// One token per blockIdx.x; its query, key and value rows are dealt to the
// CTA's groups of L lanes, AHEAD passes of loads at a time: the first are in
// flight while the turns are formed (8191 tokens of 32 + 2 x 8 heads: 40 us;
// a pass at a time 43 us, two 42, six 43; several tokens per CTA 48 to 61 us).
template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const CacheWriteParams p) {
  constexpr int L = D / 8;            // lanes per row
  constexpr int ROWS = kThreads / L;  // rows per pass of the CTA
  constexpr int AHEAD = 4;
  __shared__ __align__(16) float turn_c[D / 2], turn_s[D / 2];
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.x;
  const int half = p.rope_dim / 2;
  const int lane = threadIdx.x % L, g = threadIdx.x / L;
  const int rows = p.q_heads + 2 * p.kv_heads, step = gridDim.y * ROWS;
  const uint4* qs = reinterpret_cast<const uint4*>(p.q + (size_t)t * p.ldq) + lane;
  const uint4* ks = reinterpret_cast<const uint4*>(p.k + (size_t)t * p.ldk) + lane;
  const uint4* vs = reinterpret_cast<const uint4*>(p.v + (size_t)t * p.ldv) + lane;
  auto load = [&](int r) {
    if (r < p.q_heads) return qs[r * L];
    if (r < p.q_heads + p.kv_heads) return ks[(r - p.q_heads) * L];
    if (r < rows) return vs[(r - p.q_heads - p.kv_heads) * L];
    return make_uint4(0u, 0u, 0u, 0u);
  };
  uint4 raw[AHEAD];
#pragma unroll
  for (int i = 0; i < AHEAD; ++i) raw[i] = load(blockIdx.y * ROWS + i * step + g);
  const int slot = fresh(p.slots + t);
  Turn turn = {};
  turn.on = lane * 8 < p.rope_dim;
  turn.from = threadIdx.x & 31;
  if (half > 0) {
    if ((int)threadIdx.x < half) {
      // whole turns drop out exactly: r = rint(x) and x - r are exact in 64 bits
      const double x = (double)fresh(p.positions + t) * (fresh(p.frequency + threadIdx.x) * 0.15915494309189535);
      float s, c;
      sincospif(2.f * (float)(x - rint(x)), &s, &c);
      turn_c[threadIdx.x] = c * p.magnitude;
      turn_s[threadIdx.x] = s * p.magnitude;
    }
    __syncthreads();
    // a lane's channels are the same in every row: its turn stays in registers
    if (turn.on && p.interleaved) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float c = turn_c[lane * 4 + j], s = turn_s[lane * 4 + j];
        turn.c[j] = pack_f32x2(c, c);
        turn.s[j] = pack_f32x2(-s, s);
      }
    } else if (turn.on) {
      // the partner of channel j is R/2 channels away: R/16 lanes (R % 16 == 0)
      const int apart = p.rope_dim / 16;
      const bool low = lane < apart;
      const int at = (low ? lane : lane - apart) * 8;
      turn.from += low ? apart : -apart;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 c = *reinterpret_cast<const float2*>(turn_c + at + 2 * j);
        const float2 s = *reinterpret_cast<const float2*>(turn_s + at + 2 * j);
        turn.c[j] = pack_f32x2(c.x, c.y);
        turn.s[j] = low ? pack_f32x2(-s.x, -s.y) : pack_f32x2(s.x, s.y);
      }
    }
  }
  const bool store = slot >= 0 && slot < p.slots_total;
  const size_t row0 = store ? ((size_t)(slot >> p.page_shift) * p.kv_heads << p.page_shift) +
                                  (slot & ((1 << p.page_shift) - 1))
                            : 0;
  uint4* dst = reinterpret_cast<uint4*>(p.q_out + (size_t)t * p.ldqo) + lane;
  for (int r0 = blockIdx.y * ROWS; r0 < rows; r0 += AHEAD * step) {
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) {
      const int first = r0 + i * step;  // of the CTA's rows in this pass
      const int r = first + g;
      if (first >= rows) break;
      const bool is_q = r < p.q_heads, is_k = !is_q && r < p.q_heads + p.kv_heads;
      Chunk x;
      unpack_chunk(raw[i], x);
      if (half > 0 && first < p.q_heads + p.kv_heads) {
        Turn own = turn;
        own.on = turn.on && (is_q || is_k);
        rotate(x, raw[i], own, p.interleaved);
      }
      if (first + ROWS <= p.q_heads) {  // queries only: rotated, rounded once
        dst[r * L] = pack_chunk(x);
        continue;
      }
      float a = absmax_chunk(x);
#pragma unroll
      for (int o = L / 2; o > 0; o >>= 1) a = absmax_nan(a, __shfl_xor_sync(0xffffffffu, a, o));
      if (is_q) {
        dst[r * L] = pack_chunk(x);
      } else if (r < rows && store) {
        const int h = r - p.q_heads - (is_k ? 0 : p.kv_heads);
        const size_t row = row0 + ((size_t)h << p.page_shift);
        float s, inv;
        row_scale<INT8, true>(a, s, inv);
        if (lane == 0) (is_k ? p.k_scale : p.v_scale)[row] = s;
        reinterpret_cast<uint2*>((is_k ? p.k_codes : p.v_codes) + row * D)[lane] = chunk_codes<INT8>(x, s, inv);
      }
    }
    if (r0 + AHEAD * step < rows) {
#pragma unroll
      for (int i = 0; i < AHEAD; ++i) raw[i] = load(r0 + (AHEAD + i) * step + g);
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
    const int slot = fresh(p.slots + t);
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

cudaError_t launch_cache_write(const CacheWriteParams& p, int head_dim, bool int8, cudaStream_t st,
                               bool pdl) {
  const int rows = p.q_heads + 2 * p.kv_heads;
  const int per = kThreads / (head_dim / 8);
  // few tokens: a CTA per pass of its rows, so that no pass waits for another
  // (up to the grid's limit; further passes are a CTA's next).  32 tokens of 40
  // + 2 x 8 heads: 4.2 us, 6.2 with a CTA per token; 600 tokens: 10.4 us, 6.2.
  const int parts = p.tokens <= 2 * 148 ? std::min((rows + per - 1) / per, 65535) : 1;
  auto fn = head_dim == 128 ? (int8 ? cache_write_kernel<128, true> : cache_write_kernel<128, false>)
                            : (int8 ? cache_write_kernel<64, true> : cache_write_kernel<64, false>);
  return launch(fn, p, dim3(p.tokens, parts), st, pdl);
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
