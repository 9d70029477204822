// attend.cu — attention over the quantised cache for few rows per key head
// (single tokens and small trees): qg_attend_rows_kernel, the merge of items
// that span CTAs, and the choice between the kernels.
//
// Bound: HBM.  16 rows (the query heads of one key head, times the drafted
// tokens) read 2 D code bytes and 8 scale bytes per position, 4 x 16 x D
// flops: 31 flops per byte at most, far below the warp-level MMA's rate.  So
// the kernel is built to keep loads in flight: every warp streams its own
// blocks of 32 positions through its own ring (TMA boxes of whole rows with
// the row-wide swizzle, bulk copies for the scales), with no barrier between
// warps until the end of an item.  Codes become f16 in registers on their way
// into mma.sync fragments; the swizzle makes both fragment reads free of bank
// conflicts (D = 128), and the head's channels are permuted the same way in
// queries and keys so that a lane reads 16 neighbouring codes at once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "attend_common.cuh"
#include "attend_tile.cuh"
#include "attr_cache.h"
#include "internal.h"
#include "ptx.cuh"

namespace qg {
namespace {

constexpr int kRows = 16;     // rows per item
constexpr int kUnit = 64;     // positions per unit of work
constexpr int kBlock = 32;    // positions per ring stage of a warp
constexpr int kWarps = 8;
constexpr int kStages = 2;

template <int D>
struct RowsSmem {
  static constexpr int kCodes = kBlock * D;                  // K or V codes of a stage
  static constexpr int kStage = 2 * kCodes + 2 * kBlock * 4;  // + K and V scales
  static constexpr int kStageAlloc = (kStage + 1023) / 1024 * 1024;
  static constexpr int kRing = kWarps * kStages * kStageAlloc;
  static constexpr int kMergeRow = D + 4;                    // floats; spreads rows over banks
  static constexpr int kMerge = 4 * kRows * kMergeRow * 4;
  static constexpr int kTotal = 1024 + kRing + kMerge;
};

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int row) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(smem_u32(bar)), "r"(0), "r"(row)
      : "memory");
}
__device__ __forceinline__ uint4 lds16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t f16x2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// Byte offset of 16-byte chunk c of row r under the TMA swizzle of D-byte rows.
template <int D>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (D == 128) return r * 128 + ((c ^ (r & 7)) << 4);
  else return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

template <int D, bool INT8>
__global__ void __launch_bounds__(kWarps * 32, 1)
    qg_attend_rows_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                          const AttendParams p) {
  using S = RowsSmem<D>;
  constexpr int KS = D / 16;   // MMA steps over the head's channels
  constexpr int NT = D / 8;    // 8-channel output tiles
  extern __shared__ uint8_t smem_raw[];
  __shared__ Sched sched;
  __shared__ __align__(8) uint64_t bars[kWarps * kStages];
  __shared__ float2 vsc[kWarps][kBlock];       // (log2 vs, 1 / vs) of the block in hand
  __shared__ float part_m[kWarps][kRows], part_l[kWarps][kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t ring = base + warp * kStages * S::kStageAlloc;
  float* merge = reinterpret_cast<float*>(smem_raw + (base - smem_u32(smem_raw)) + S::kRing);
  uint64_t* bar = bars + warp * kStages;
  if (lane == 0)
    for (int i = 0; i < kStages; ++i) mbar_init(bar + i, 1);
  if (threadIdx.x == 0) {
    prefetch_tmap(&tmap_k);
    prefetch_tmap(&tmap_v);
  }
  fence_barrier_init();
  griddep_launch_dependents();
  griddep_wait();
  const Share share = plan_units(p, kRows, kUnit, sched);
  if (threadIdx.x == 0) p.records[blockIdx.x] = merge_record(p, sched, share, kRows);
  if (blockIdx.x >= share.ctas || share.total == 0) return;
  const int share_begin = share.begin(blockIdx.x), share_end = share.begin(blockIdx.x + 1);
  uint32_t phase = 0;  // bit i: parity of the ring stage's next wait
  bool ok = true, drained = false;

#pragma unroll 1
  for (int u = share_begin; u < share_end;) {
    const Piece x = find_piece(p, sched, kRows, u, share_end);
    const int tok0 = sched.tok0[x.seq], len = sched.len[x.seq];
    const int rows = min(sched.n[x.seq], p.max_q) * p.group;
    const int begin = x.unit0 * kUnit, end = min(x.unit1 * kUnit, len);
    const int past = len - sched.n[x.seq];      // position of drafted token 0
    const int nblk = begin < end ? (end - begin + kBlock - 1) / kBlock : 0;
    const int* table = p.table + (size_t)x.seq * p.ldp;

    // lanes below `runs` each load the codes and scales of one run of
    // box_rows positions (within a page) of the block
    const int runs = kBlock / p.box_rows;
    const int run_off = lane * p.box_rows;
    auto page_of = [&](int blk) {
      const int pos = begin + blk * kBlock + run_off;
      if (lane >= runs || blk >= nblk || pos >= end) return 0;
      return min(max(__ldg(table + (pos >> p.page_shift)), 0), p.pages - 1);
    };
    auto issue = [&](int blk, int page) {
      const int st = (blk / kWarps) % kStages;
      const int pos0 = begin + blk * kBlock;
      const int live = min((end - pos0 + p.box_rows - 1) / p.box_rows, runs);
      const uint32_t dst = ring + st * S::kStageAlloc;
      if (lane == 0) mbar_arrive_expect_tx(bar + st, live * p.box_rows * (2 * D + 8));
      __syncwarp();
      if (lane < live) {
        const int pos = pos0 + run_off;
        const int row = (page * p.kv_heads + x.head << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        tma_rows(dst + run_off * D, &tmap_k, bar + st, row);
        tma_rows(dst + S::kCodes + run_off * D, &tmap_v, bar + st, row);
        const uint32_t sc = dst + 2 * S::kCodes + run_off * 4;
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(sc),
            "l"(p.k_scale + row), "r"(p.box_rows * 4), "r"(smem_u32(bar + st))
            : "memory");
        asm volatile(
            "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                sc + kBlock * 4),
            "l"(p.v_scale + row), "r"(p.box_rows * 4), "r"(smem_u32(bar + st))
            : "memory");
      }
    };
    // the ring is empty between items (a stage's parity carries on); reads and
    // writes of the last item's blocks come before the copies that refill it
    fence_proxy_async_smem();
    __syncwarp();
    int ahead = warp;
    int next_page = page_of(ahead);
    if (ok) {
#pragma unroll 1
      for (int i = 0; i < kStages; ++i) {
        if (ahead < nblk) issue(ahead, next_page);
        ahead += kWarps;
        next_page = page_of(ahead);
      }
    }

    // queries of rows g and g + 8, f16, channels in the order of the key reads
    uint32_t qa[KS][4];
    float row_scale[2];
    int tok[2];       // drafted token of the row, -1 past the last row
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = x.row0 + g + 8 * i;
      const bool live = row < rows;
      tok[i] = live ? row / p.group : -1;
      const __nv_bfloat16* src =
          p.q + (size_t)(tok0 + (live ? tok[i] : 0)) * p.ldq + (x.head * p.group + (live ? row % p.group : 0)) * D;
      float amax = 0.f;
      uint4 raw[D / 32];  // 8 channels each
#pragma unroll
      for (int c = 0; c < D / 64; ++c)  // 16-channel chunks t (and t + 4)
#pragma unroll
        for (int hlf = 0; hlf < 2; ++hlf) {
          const uint4 v = live ? reinterpret_cast<const uint4*>(src)[(t + 4 * c) * 2 + hlf] : make_uint4(0, 0, 0, 0);
          raw[c * 2 + hlf] = v;
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u))));
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float up, down;
      row_power(amax, up, down);
      row_scale[i] = down * p.scale_log2;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint32_t w[4] = {raw[c].x, raw[c].y, raw[c].z, raw[c].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t h = f16x2(__uint_as_float(w[j] << 16) * up, __uint_as_float(w[j] & 0xffff0000u) * up);
          // pair e of the lane's 2 KS pairs: step e / 2, the step's low or high channels
          const int e = c * 4 + j;
          qa[e >> 1][i + 2 * (e & 1)] = h;
        }
      }
    }

    float o[NT][4];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[j][i] = 0.f;
    float m[2] = {kNegInf, kNegInf}, l[2] = {0.f, 0.f};

    for (int blk = warp; blk < nblk; blk += kWarps) {
      const int st = (blk / kWarps) % kStages;
      const uint32_t kb = ring + st * S::kStageAlloc, vb = kb + S::kCodes, sb = vb + S::kCodes;
      const int pos0 = begin + blk * kBlock;
      if (ok) ok = mbar_wait(bar + st, (phase >> st) & 1, p.err, p.wait_ns);
      phase ^= 1u << st;
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) break;
      const bool tail = pos0 + kBlock > end || pos0 + kBlock > past;
      {
        float vs;
        asm volatile("ld.shared.f32 %0, [%1];" : "=f"(vs) : "r"(sb + kBlock * 4 + lane * 4));
        float a, b;
        value_scale(vs, a, b);
        vsc[warp][lane] = make_float2(a, b);
      }
      if (pos0 + kBlock > end) {
        // rows past the last position hold whatever the page held: an e4m3
        // NaN code there would reach the sums through 0 * NaN
        for (int r = end - pos0 + (lane >> 3); r < kBlock; r += 4)
          for (int c = (lane & 7); c < D / 16; c += 8)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + r * D + c * 16), "r"(0) : "memory");
      }
      __syncwarp();
      // scores: 4 tiles of 8 positions
      float s[4][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) s[nt][i] = 0.f;
        uint32_t w[D / 16];
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 v = lds16(kb + chunk_at<D>(nt * 8 + g, t + 4 * c));
          w[4 * c] = v.x;
          w[4 * c + 1] = v.y;
          w[4 * c + 2] = v.z;
          w[4 * c + 3] = v.w;
        }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t b0, b1;
          decode4<INT8>(w[k], b0, b1);
          mma16816(s[nt], qa[k], b0, b1);
        }
      }
      float top[2] = {m[0], m[1]};
      float2 sc[4][2];
      uint32_t see[2] = {0, 0};  // bits of the block's positions from this lane's first on
      if (tail) {
#pragma unroll
        for (int r = 0; r < 2; ++r) see[r] = (uint32_t)(seen_bits(p, tok0, tok[r], end - pos0, past - pos0) >> (2 * t));
      }
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        float2 ks;
        asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(ks.x), "=f"(ks.y) : "r"(sb + (nt * 8 + 2 * t) * 4));
        sc[nt][0] = vsc[warp][nt * 8 + 2 * t];
        sc[nt][1] = vsc[warp][nt * 8 + 2 * t + 1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = i & 1, r = i >> 1;
          s[nt][i] = fmaf(s[nt][i] * row_scale[r], e ? ks.y : ks.x, sc[nt][e].x);
          if (tail && !((see[r] >> (nt * 8 + e)) & 1)) s[nt][i] = kNegInf;
          top[r] = fmaxf(top[r], s[nt][i]);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
        top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
        float f[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          f[r] = top[r] > m[r] ? ex2(m[r] - top[r]) : 1.f;  // m = -inf: 0
          m[r] = top[r];
          l[r] *= f[r];
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[j][i] *= f[i >> 1];
      }
      const float mm[2] = {m[0] == kNegInf ? 0.f : m[0], m[1] == kNegInf ? 0.f : m[1]};
      uint32_t pa[2][4];
#pragma unroll
      for (int nt = 0; nt < 4; ++nt) {
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          w[i] = ex2(s[nt][i] - mm[i >> 1]);
          l[i >> 1] = fmaf(w[i], sc[nt][i & 1].y, l[i >> 1]);
        }
        pa[nt >> 1][(nt & 1) * 2] = f16x2(w[0], w[1]);
        pa[nt >> 1][(nt & 1) * 2 + 1] = f16x2(w[2], w[3]);
      }
      // o += w . codes: 2 steps of 16 positions; a lane reads its 4 positions'
      // codes of channels [16 g, 16 g + 16) ([8 g, 8 g + 8) for D = 64)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t v[4][NT / 4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = k * 16 + (i >> 1) * 8 + 2 * t + (i & 1);
          if constexpr (D == 128) {
            const uint4 q = lds16(vb + chunk_at<D>(r, g));
            v[i][0] = q.x;
            v[i][1] = q.y;
            v[i][2] = q.z;
            v[i][3] = q.w;
          } else {
            const uint2 q = lds8(vb + chunk_at<D>(r, g >> 1) + (g & 1) * 8);
            v[i][0] = q.x;
            v[i][1] = q.y;
          }
        }
#pragma unroll
        for (int w = 0; w < NT / 4; ++w) {
          // bytes of two positions side by side: channels 0, 1 then 2, 3
          uint32_t b0[4], b1[4];
          decode4<INT8>(__byte_perm(v[0][w], v[1][w], 0x5140), b0[0], b0[1]);
          decode4<INT8>(__byte_perm(v[0][w], v[1][w], 0x7362), b0[2], b0[3]);
          decode4<INT8>(__byte_perm(v[2][w], v[3][w], 0x5140), b1[0], b1[1]);
          decode4<INT8>(__byte_perm(v[2][w], v[3][w], 0x7362), b1[2], b1[3]);
#pragma unroll
          for (int j = 0; j < 4; ++j) mma16816(o[4 * w + j], pa[k], b0[j], b1[j]);
        }
      }
      __syncwarp();
      if (ahead < nblk) {
        // this lane's reads (and, in a tail block, writes) of the stage come
        // before the copies that refill it
        fence_proxy_async_smem();
        issue(ahead, next_page);
        ahead += kWarps;
        next_page = page_of(ahead);
      }
    }
    if (!ok && !drained) {
      drained = true;
      // a wait ran out: the copies still in flight land before shared memory
      // is given up (bounded as well)
      for (int i = 0; i < kStages; ++i) (void)mbar_wait(bar + i, (phase >> i) & 1, p.err, p.wait_ns);
    }

    // the warps' partials meet: maxima, then the scaled sums 4 warps at a time
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
      l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
      if (l[r] != l[r]) m[r] = 0.f;  // a NaN row keeps its place in the merges
      if (t == 0) {
        part_m[warp][g + 8 * r] = m[r];
        part_l[warp][g + 8 * r] = l[r];
      }
    }
    __syncthreads();
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float top = kNegInf;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w][g + 8 * r]);
      f[r] = m[r] == kNegInf ? 0.f : ex2(m[r] - top);
    }
#pragma unroll
    for (int half = 1; half >= 0; --half) {
      if (warp / 4 == half) {
        float* dst = merge + (warp % 4) * kRows * S::kMergeRow;
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int e = 0; e < 2; ++e)
#pragma unroll
            for (int j = 0; j < NT; j += 4) {
              // o[j][2 r + e]: row g + 8 r, channel NT (2 t + e) + j
              float4* d4 = reinterpret_cast<float4*>(dst + (g + 8 * r) * S::kMergeRow + NT * (2 * t + e) + j);
              float4 v = make_float4(o[j][2 * r + e] * f[r], o[j + 1][2 * r + e] * f[r], o[j + 2][2 * r + e] * f[r],
                                     o[j + 3][2 * r + e] * f[r]);
              if (half == 0) {
                const float4 a = *d4;
                v = make_float4(v.x + a.x, v.y + a.y, v.z + a.z, v.w + a.w);
              }
              *d4 = v;
            }
      }
      __syncthreads();
    }
    const bool whole = x.unit0 == 0 && x.unit1 == x.units;
    const int slot = 2 * blockIdx.x + (u == share_begin ? 0 : 1);
    float* part = p.partial + (size_t)slot * kRows * (D + 2);
    constexpr int TPR = kWarps * 32 / kRows;  // threads per row
    constexpr int CPT = D / TPR;              // channels per thread
    const int row = threadIdx.x / TPR, c0 = (threadIdx.x % TPR) * CPT;
    float top = kNegInf, sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, part_m[w][row]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += part_m[w][row] == kNegInf ? 0.f : part_l[w][row] * ex2(part_m[w][row] - top);
    float acc[CPT];
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      acc[j] = 0.f;
#pragma unroll
      for (int w = 0; w < 4; ++w) acc[j] += merge[w * kRows * S::kMergeRow + row * S::kMergeRow + c0 + j];
    }
    if (whole) {
      const int r = x.row0 + row;
      if (r < rows) {
        const size_t tk = tok0 + r / p.group;
        const int h = x.head * p.group + r % p.group;
        // a row that saw nothing: zeros, and a log-sum of -inf
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        __nv_bfloat162 v[CPT / 2];
#pragma unroll
        for (int j = 0; j < CPT / 2; ++j) v[j] = __floats2bfloat162_rn(acc[2 * j] * inv, acc[2 * j + 1] * inv);
        __nv_bfloat16* dst = p.out + tk * p.ldo + h * D + c0;
        if constexpr (CPT == 8) *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(v);
        else *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(v);
        if (p.lse != nullptr && c0 == 0)
          p.lse[tk * p.q_heads + h] = sum == 0.f ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < CPT; j += 4)
        *reinterpret_cast<float4*>(part + row * D + c0 + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
      if (c0 == 0) {
        part[kRows * D + row] = top;
        part[kRows * D + kRows + row] = sum;
      }
    }
    __syncthreads();
    u += x.unit1 - x.unit0;
  }
}

// Merge of the items that span CTAs: CTA c takes the one of its record, ROWS
// rows per blockIdx.y.  WPR warps share a row: each takes every WPR-th part,
// D / 32 channels a lane; they meet in shared memory.
template <int D, int ROWS, int WPR>
__global__ void __launch_bounds__(ROWS * WPR * 32) qg_attend_merge_kernel(const AttendParams p, int tile_rows) {
  constexpr int CPL = D / 32;
  __shared__ float acc_s[ROWS][WPR][D], sum_s[ROWS][WPR];
  griddep_launch_dependents();
  griddep_wait();
  const MergeRecord rec = p.records[blockIdx.x];
  if (rec.last < 0 || rec.row0 + (int)blockIdx.y * ROWS >= rec.rows) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int mr = warp / WPR, g = warp % WPR;
  const int row = blockIdx.y * ROWS + mr, r = rec.row0 + row;
  const size_t stride = (size_t)tile_rows * (D + 2);
  auto part_of = [&](int c) { return p.partial + (c == (int)blockIdx.x ? rec.slot : 2 * c) * stride; };
  float top = kNegInf, sum = 0.f, acc[CPL];
#pragma unroll
  for (int j = 0; j < CPL; ++j) acc[j] = 0.f;
  for (int c = blockIdx.x + lane; c <= rec.last; c += 32) top = fmaxf(top, part_of(c)[tile_rows * D + row]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll 4
  for (int c = blockIdx.x + g; c <= rec.last; c += WPR) {
    const float* part = part_of(c);
    const float m = part[tile_rows * D + row], l = part[tile_rows * D + tile_rows + row];
    float v[CPL];
    if constexpr (CPL == 4) *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(part + row * D + lane * 4);
    else *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(part + row * D + lane * 2);
    const float f = m == kNegInf ? 0.f : ex2(m - top);
    sum = fmaf(l, f, sum);
#pragma unroll
    for (int j = 0; j < CPL; ++j) acc[j] = fmaf(v[j], f, acc[j]);
  }
  if constexpr (WPR > 1) {
#pragma unroll
    for (int j = 0; j < CPL; ++j) acc_s[mr][g][lane * CPL + j] = acc[j];
    if (lane == 0) sum_s[mr][g] = sum;
    __syncthreads();
    if (g != 0) return;
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      sum += sum_s[mr][w];
#pragma unroll
      for (int j = 0; j < CPL; ++j) acc[j] += acc_s[mr][w][lane * CPL + j];
    }
  }
  if (r >= rec.rows) return;
  const int tok = r / p.group;
  const size_t tk = rec.tok0 + tok;
  const int h = rec.head * p.group + r - tok * p.group;
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  __nv_bfloat162 v[CPL / 2];
#pragma unroll
  for (int j = 0; j < CPL / 2; ++j) v[j] = __floats2bfloat162_rn(acc[2 * j] * inv, acc[2 * j + 1] * inv);
  __nv_bfloat16* dst = p.out + tk * p.ldo + h * D + lane * CPL;
  if constexpr (CPL == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<const uint2*>(v);
  else *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<const uint32_t*>(v);
  if (p.lse != nullptr && lane == 0)
    p.lse[tk * p.q_heads + h] = sum == 0.f ? kNegInf : (top + log2f(sum)) * 0.6931471805599453f;
}

cudaError_t launch_pdl(const void* fn, dim3 grid, int threads, size_t smem, void** args, cudaStream_t st, bool pdl) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

template <int D, bool INT8>
cudaError_t launch_rows(const AttendParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int ctas,
                        cudaStream_t st, bool pdl) {
  static GrowOnlyAttr opened;
  const void* fn = (const void*)qg_attend_rows_kernel<D, INT8>;
  constexpr int smem = RowsSmem<D>::kTotal;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const int e = opened.ensure(
      dev, smem, [&](int v) { return (int)cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v); });
  if (e != 0) return (cudaError_t)e;
  void* args[] = {(void*)&tk, (void*)&tv, (void*)&p};
  return launch_pdl(fn, dim3(ctas), kWarps * 32, smem, args, st, pdl);
}

template <int D, bool INT8>
cudaError_t launch_tile(const AttendParams& p, const uint8_t* k, const uint8_t* v, int ctas, cudaStream_t st,
                        bool pdl) {
  static GrowOnlyAttr opened;
  const void* fn = (const void*)qg_attend_tile_kernel<D, INT8>;
  constexpr int smem = TileSmem<D>::kTotal;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const int e = opened.ensure(
      dev, smem, [&](int v) { return (int)cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v); });
  if (e != 0) return (cudaError_t)e;
  void* args[] = {(void*)&k, (void*)&v, (void*)&p};
  return launch_pdl(fn, dim3(ctas), kTileThreads, smem, args, st, pdl);
}

// The rows kernel may leave an item in a part per SM, of few rows: four warps
// a row.  The tile kernel's items have up to 128 rows: one warp each.
template <int D>
cudaError_t launch_merge(const AttendParams& p, bool tiles, int ctas, cudaStream_t st, bool pdl) {
  int tile_rows = tiles ? kTileRows : kRows;
  void* args[] = {(void*)&p, (void*)&tile_rows};
  if (tiles)
    return launch_pdl((const void*)qg_attend_merge_kernel<D, 16, 1>, dim3(ctas, kTileRows / 16), 512, 0, args, st, pdl);
  return launch_pdl((const void*)qg_attend_merge_kernel<D, 2, 4>, dim3(ctas, kRows / 2), 256, 0, args, st, pdl);
}

}  // namespace

// More rows than one 16-row tile read the codes once per 16 rows in the rows
// kernel; the tile kernel reads them once per 128.
bool attend_tiles(int rows_max) { return rows_max > kRows; }

size_t attend_workspace(int head_dim, int rows_max, int sms) {
  return sizeof(MergeRecord) * sms + (size_t)2 * sms * (attend_tiles(rows_max) ? kTileRows : kRows) * (head_dim + 2) * 4;
}

cudaError_t launch_attend(AttendParams p, void* workspace, const uint8_t* k, const uint8_t* v, const CUtensorMap* tk,
                          const CUtensorMap* tv, int head_dim, bool int8, int sms, cudaStream_t st, bool pdl) {
  const bool tiles = attend_tiles(p.max_q * p.group);
  p.records = static_cast<MergeRecord*>(workspace);
  p.partial = reinterpret_cast<float*>(p.records + sms);
  cudaError_t e;
  if (tiles) {
    if (head_dim == 128)
      e = int8 ? launch_tile<128, true>(p, k, v, sms, st, pdl) : launch_tile<128, false>(p, k, v, sms, st, pdl);
    else
      e = int8 ? launch_tile<64, true>(p, k, v, sms, st, pdl) : launch_tile<64, false>(p, k, v, sms, st, pdl);
  } else if (head_dim == 128) {
    e = int8 ? launch_rows<128, true>(p, *tk, *tv, sms, st, pdl) : launch_rows<128, false>(p, *tk, *tv, sms, st, pdl);
  } else {
    e = int8 ? launch_rows<64, true>(p, *tk, *tv, sms, st, pdl) : launch_rows<64, false>(p, *tk, *tv, sms, st, pdl);
  }
  if (e != cudaSuccess) return e;
  return head_dim == 128 ? launch_merge<128>(p, tiles, sms, st, pdl) : launch_merge<64>(p, tiles, sms, st, pdl);
}

}  // namespace qg
