// attend.cu — attention over the quantised cache for few rows per key head
// (single tokens and small trees): qg_attend_rows_kernel, the merge of items
// that span CTAs, and the choice between the kernels.
//
// Bound: HBM.  8 NR rows (the query heads of one key head, times the drafted
// tokens) read 2 D code bytes and 8 scale bytes per position: 16 flops per
// byte and row tile, far below the warp-level MMA's rate.  What is scarce is
// issue: decoding to f16 takes an instruction per two codes.  So positions are
// the MMA's 16-row operand and the query rows its 8 columns,
//   S^T = K Q^T,  O^T = V^T W^T,
// which for the usual 4 to 8 query heads of a key head halves the MMAs, the
// exponentials and the registers of the other orientation (64 x 16384
// positions, 64 query and 8 key heads: 311 us there, 235 us here).
// That case moves its bytes at 6.0 TB/s (92 % of a copy's rate); 1 x 131072
// positions take 58 us, of which 42 are the bytes.  Short pieces (64 sequences
// of up to 1000 positions, 4 tokens each: 51 us) are bound by a piece's chain:
// pages, blocks, some 2000 cycles a block and warp, the join.
// Every warp streams its own blocks of 32 positions through its own ring (TMA
// boxes of whole rows with the row-wide swizzle, bulk copies for the scales),
// with no barrier between warps until the end of an item.  The swizzle makes
// both fragment reads free of bank conflicts (D = 128), and the head's
// channels are permuted the same way in queries and keys so that a lane reads
// 16 neighbouring codes at once.
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

constexpr int kUnit = 64;     // positions per unit of work
constexpr int kBlock = 32;    // positions per ring stage of a warp
constexpr int kStages = 2;

// Warps per CTA: as many as the registers of NR row tiles leave room for (a
// warp issues an instruction every four to five cycles).
template <int NR>
constexpr int kRowsWarps = NR == 1 ? 12 : 8;

template <int D, int NR>
struct RowsSmem {
  static constexpr int kCodes = kBlock * D;                  // K or V codes of a stage
  static constexpr int kStage = 2 * kCodes;
  // a warp's results of a piece lie in its own ring, empty by then
  static constexpr int kMergeRow = D + 4;                    // floats; spreads rows over banks
  static constexpr int kResult = 8 * NR * kMergeRow * 4;
  static constexpr int kWarpRing = kStages * kStage > kResult ? kStages * kStage : (kResult + 1023) / 1024 * 1024;
  static constexpr int kRing = kRowsWarps<NR> * kWarpRing;
  static constexpr int kScale = 2 * kBlock * 4;              // K and V scales of a stage
  static constexpr int kScales = kRowsWarps<NR> * kStages * kScale;
  static constexpr int kTotal = 1024 + kRing + kScales;
};

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int row) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(
          dst),
      "l"(map), "r"(smem_u32(bar)), "r"(0), "r"(row)
      : "memory");
}
__device__ __forceinline__ void bulk_floats(uint32_t dst, const float* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(smem_u32(bar))
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
__device__ __forceinline__ float lds4(uint32_t a) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Transpose of an 8 x 8 b16 matrix held as fragments.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
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

template <int D, bool INT8, int NR>
__global__ void __launch_bounds__(kRowsWarps<NR> * 32, 1)
    qg_attend_rows_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                          const AttendParams p) {
  using S = RowsSmem<D, NR>;
  constexpr int WARPS = kRowsWarps<NR>;
  constexpr int ROWS = 8 * NR;
  constexpr int KS = D / 16;   // MMA steps over the head's channels
  constexpr int MT = D / 16;   // 16-channel output tiles
  extern __shared__ uint8_t smem_raw[];
  __shared__ Sched sched;
  __shared__ __align__(8) uint64_t bars[WARPS * kStages];
  __shared__ float4 pos_scale[WARPS][kBlock];  // (key scale, log2 vs, 1 / vs) of the block in hand
  __shared__ float part_m[WARPS][ROWS], part_l[WARPS][ROWS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t ring = base + warp * S::kWarpRing;
  const uint32_t scale_ring = base + S::kRing + warp * kStages * S::kScale;
  const float* results = reinterpret_cast<const float*>(smem_raw + (base - smem_u32(smem_raw)));
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
  const Share share = plan_units(p, ROWS, kUnit, sched);
  if (threadIdx.x == 0) p.records[blockIdx.x] = merge_record(p, sched, share, ROWS);
  if (blockIdx.x >= share.ctas || share.total == 0) return;
  const int share_begin = share.begin(blockIdx.x), share_end = share.begin(blockIdx.x + 1);
  uint32_t phase = 0;  // bit i: parity of the ring stage's next wait
  bool ok = true;

  Piece x = find_piece(p, sched, ROWS, share_begin, share_end);
#pragma unroll 1
  for (int u = share_begin; u < share_end;) {
    if (u > share_begin) next_piece(p, sched, ROWS, kUnit, u, share_end, x);
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
      return min(max(fresh(table + (pos >> p.page_shift)), 0), p.pages - 1);
    };
    auto issue = [&](int blk, int page) {
      const int st = (blk / WARPS) % kStages;
      const int pos0 = begin + blk * kBlock;
      const int live = min((end - pos0 + p.box_rows - 1) / p.box_rows, runs);
      const uint32_t dst = ring + st * S::kStage;
      if (lane == 0) mbar_arrive_expect_tx(bar + st, live * p.box_rows * (2 * D + 8));
      __syncwarp();
      if (lane < live) {
        const int pos = pos0 + run_off;
        const int row = (page * p.kv_heads + x.head << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        tma_rows(dst + run_off * D, &tmap_k, bar + st, row);
        tma_rows(dst + S::kCodes + run_off * D, &tmap_v, bar + st, row);
        const uint32_t sc = scale_ring + st * S::kScale + run_off * 4;
        bulk_floats(sc, p.k_scale + row, p.box_rows * 4, bar + st);
        bulk_floats(sc + kBlock * 4, p.v_scale + row, p.box_rows * 4, bar + st);
      }
    };
    // What the piece needs from memory is asked for at once: its queries, the
    // pages of the first blocks, then the blocks.
    // query row g of each row tile
    uint4 qv[NR][D / 64][2];
    int mine[NR];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int row = x.row0 + 8 * i + g;
      mine[i] = row < rows ? row / p.group : -1;
      const uint4* src = reinterpret_cast<const uint4*>(
          p.q + (size_t)(tok0 + max(mine[i], 0)) * p.ldq +
          (x.head * p.group + (mine[i] < 0 ? 0 : row - mine[i] * p.group)) * D);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)  // 16-channel chunks t (and t + 4)
#pragma unroll
        for (int hlf = 0; hlf < 2; ++hlf)
          qv[i][c][hlf] = mine[i] >= 0 ? fresh(src + (t + 4 * c) * 2 + hlf) : make_uint4(0, 0, 0, 0);
    }
    int first_page[kStages];
#pragma unroll
    for (int i = 0; i < kStages; ++i) first_page[i] = page_of(warp + i * WARPS);
    int ahead = warp + kStages * WARPS;
    int next_page = page_of(ahead);
    // the ring is empty between pieces (a stage's parity carries on); reads and
    // writes of the last piece's results come before the copies that refill it
    fence_proxy_async_smem();
    __syncwarp();
    if (ok) {
#pragma unroll
      for (int i = 0; i < kStages; ++i)
        if (warp + i * WARPS < nblk) issue(warp + i * WARPS, first_page[i]);
    }

    // f16, channels in the order of the key reads; scale and drafted token of
    // rows 2 t and 2 t + 1, the lane's score columns (-1: past the last row)
    uint32_t qb[NR][KS][2];
    float power[NR][2];
    int tok[NR][2];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      float amax = 0.f;
      uint32_t raw[KS][2];
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
#pragma unroll
        for (int hlf = 0; hlf < 2; ++hlf) {
          const uint4 v = qv[i][c][hlf];
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // pair e of the lane's 2 KS pairs: step e / 2, the step's low or high channels
            const int e = c * 8 + hlf * 4 + j;
            raw[e >> 1][e & 1] = w[j];
            amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[j] << 16)), fabsf(__uint_as_float(w[j] & 0xffff0000u))));
          }
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      float up, down;
      row_power(amax, up, down);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e)
          qb[i][k][e] =
              f16x2(__uint_as_float(raw[k][e] << 16) * up, __uint_as_float(raw[k][e] & 0xffff0000u) * up);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        power[i][e] = __shfl_sync(0xffffffffu, down, (2 * t + e) * 4) * p.scale_log2;
        tok[i][e] = __shfl_sync(0xffffffffu, mine[i], (2 * t + e) * 4);
      }
    }

    // o[i][j]: channels NC g + 2 j (first pair) and the next (second) of row
    // tile i's rows 2 t, 2 t + 1; NC = D / 8 channels a lane
    float o[NR][MT][4], m[NR][2], l[NR][2];
#pragma unroll
    for (int i = 0; i < NR; ++i) {
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][j][e] = 0.f;
      m[i][0] = m[i][1] = kNegInf;
      l[i][0] = l[i][1] = 0.f;
    }

#pragma unroll 1
    for (int blk = ok ? warp : nblk; blk < nblk; blk += WARPS) {
      const int st = (blk / WARPS) % kStages;
      const uint32_t kb = ring + st * S::kStage, vb = kb + S::kCodes, sb = scale_ring + st * S::kScale;
      const int pos0 = begin + blk * kBlock;
      const bool tail = pos0 + kBlock > end || pos0 + kBlock > past;
      uint32_t seen[NR][2];  // of the block's positions, from this lane's first on
      if (tail) {
        // while the block is on its way
        unsigned long long drafted[NR][2];
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) drafted[i][e] = drafted_bits(p, tok0, tok[i][e], past - pos0);
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            seen[i][e] = (uint32_t)(seen_bits(p, tok[i][e], end - pos0, past - pos0, drafted[i][e]) >> g);
      }
      ok = __all_sync(0xffffffffu, mbar_wait(bar + st, (phase >> st) & 1, p.err, p.wait_ns));
      if (!ok) {
        // a wait ran out: the copies still in flight, this block's and the
        // next ones', land before shared memory is given up (bounded as well);
        // a stage's phase is the one that has not been passed
        for (int i = 0; i < kStages; ++i) {
          const int s = (blk / WARPS + i) % kStages;
          if (blk + i * WARPS < nblk) (void)mbar_wait(bar + s, (phase >> s) & 1, p.err, p.wait_ns);
        }
        break;
      }
      phase ^= 1u << st;
      {
        float a, b;
        value_scale(lds4(sb + kBlock * 4 + lane * 4), a, b);
        pos_scale[warp][lane] = make_float4(lds4(sb + lane * 4), a, b, 0.f);
      }
      if (pos0 + kBlock > end) {
        // rows past the last position hold whatever the page held: an e4m3
        // NaN code there would reach the sums through 0 * NaN
        for (int r = end - pos0 + (lane >> 3); r < kBlock; r += 4)
          for (int c = (lane & 7); c < D / 16; c += 8)
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(vb + r * D + c * 16), "r"(0) : "memory");
      }
      __syncwarp();
      // scores: 2 tiles of 16 positions; a lane has positions 16 mt + g and + 8
      float s[2][NR][4];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[mt][i][e] = 0.f;
        uint32_t w[2][KS];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            const uint4 v = lds16(kb + chunk_at<D>(mt * 16 + h * 8 + g, t + 4 * c));
            w[h][4 * c] = v.x;
            w[h][4 * c + 1] = v.y;
            w[h][4 * c + 2] = v.z;
            w[h][4 * c + 3] = v.w;
          }
#pragma unroll
        for (int k = 0; k < KS; ++k) {
          uint32_t a0, a1, a2, a3;
          decode4<INT8>(w[0][k], a0, a2);
          decode4<INT8>(w[1][k], a1, a3);
#pragma unroll
          for (int i = 0; i < NR; ++i) mma16816(s[mt][i], a0, a1, a2, a3, qb[i][k][0], qb[i][k][1]);
        }
      }
      float4 sc[2][2];
#pragma unroll
      for (int mt = 0; mt < 2; ++mt)
#pragma unroll
        for (int h = 0; h < 2; ++h) sc[mt][h] = pos_scale[warp][mt * 16 + h * 8 + g];
      bool grown = false;
#pragma unroll
      for (int i = 0; i < NR; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
#pragma unroll
          for (int mt = 0; mt < 2; ++mt)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              float& v = s[mt][i][2 * h + e];
              v = fmaf(v * power[i][e], sc[mt][h].x, sc[mt][h].y);
              if (tail && !((seen[i][e] >> (mt * 16 + h * 8)) & 1)) v = kNegInf;
              grown |= v > m[i][e] + kRescaleAt;  // m = -inf: anything seen
            }
        }
      if (__any_sync(0xffffffffu, grown)) {
        // a new reference where a row's maximum has passed the old one by more
        // than 2^8 (weights stay below 2^15); sums and accumulator follow
#pragma unroll
        for (int i = 0; i < NR; ++i)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float top = fmaxf(fmaxf(s[0][i][e], s[0][i][2 + e]), fmaxf(s[1][i][e], s[1][i][2 + e]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
            const bool up = top > m[i][e] + kRescaleAt;
            const float f = up ? ex2(m[i][e] - top) : 1.f;  // m = -inf: 0
            if (up) m[i][e] = top;
            l[i][e] *= f;
#pragma unroll
            for (int j = 0; j < MT; ++j) {
              o[i][j][e] *= f;
              o[i][j][2 + e] *= f;
            }
          }
      }
      uint32_t wb[2][NR][2];  // weights as the second operand of each 16 positions
#pragma unroll
      for (int i = 0; i < NR; ++i) {
        const float ref[2] = {m[i][0] == kNegInf ? 0.f : m[i][0] - kWeightUp, m[i][1] == kNegInf ? 0.f : m[i][1] - kWeightUp};
#pragma unroll
        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float w[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              w[e] = ex2(s[mt][i][2 * h + e] - ref[e]);
              l[i][e] = fmaf(w[e], sc[mt][h].z, l[i][e]);
            }
            wb[mt][i][h] = transpose8x8(f16x2(w[0], w[1]));
          }
      }
      // o^T += codes^T . w^T: a lane reads its 4 positions' codes of channels
      // [16 g, 16 g + 16) ([8 g, 8 g + 8) for D = 64)
#pragma unroll
      for (int mt = 0; mt < 2; ++mt) {
        uint32_t v[4][D / 32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = mt * 16 + (i >> 1) * 8 + 2 * t + (i & 1);
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
        for (int w = 0; w < D / 32; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            // bytes of two positions side by side: channels 4 w + 2 h and the next
            const uint32_t sel = h ? 0x7362 : 0x5140;
            uint32_t a0, a1, a2, a3;
            decode4<INT8>(__byte_perm(v[0][w], v[1][w], sel), a0, a1);
            decode4<INT8>(__byte_perm(v[2][w], v[3][w], sel), a2, a3);
#pragma unroll
            for (int i = 0; i < NR; ++i) mma16816(o[i][2 * w + h], a0, a1, a2, a3, wb[mt][i][0], wb[mt][i][1]);
          }
      }
      __syncwarp();
      if (ahead < nblk) {
        // this lane's reads (and, in a tail block, writes) of the stage come
        // before the copies that refill it
        fence_proxy_async_smem();
        issue(ahead, next_page);
        ahead += WARPS;
        next_page = page_of(ahead);
      }
    }
    // the warps' results meet, each in its own ring with its own reference
#pragma unroll
    for (int i = 0; i < NR; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[i][e] += __shfl_xor_sync(0xffffffffu, l[i][e], d);
        if (l[i][e] != l[i][e]) m[i][e] = 0.f;  // a NaN row keeps its place in the merges
        if (g == 0) {
          part_m[warp][8 * i + 2 * t + e] = m[i][e];
          part_l[warp][8 * i + 2 * t + e] = l[i][e];
        }
        const uint32_t dst = ring + ((8 * i + 2 * t + e) * S::kMergeRow + (D / 8) * g) * 4;
#pragma unroll
        for (int j = 0; j < MT; j += 2)
          asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 8 * j), "f"(o[i][j][e]), "f"(o[i][j][2 + e]),
                       "f"(o[i][j + 1][e]), "f"(o[i][j + 1][2 + e])
                       : "memory");
      }
    __syncthreads();
    const bool whole = x.unit0 == 0 && x.unit1 == x.units;
    const int slot = 2 * blockIdx.x + (u == share_begin ? 0 : 1);
    float* part = p.partial + (size_t)slot * ROWS * (D + 2);
    // 4 channels a thread
    for (int at = threadIdx.x; at < ROWS * (D / 4); at += WARPS * 32) {
      const int row = at / (D / 4), c0 = at % (D / 4) * 4;
      float top = kNegInf, sum = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) top = fmaxf(top, part_m[w][row]);
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < WARPS; ++w) {
        const float f = part_m[w][row] == kNegInf ? 0.f : ex2(part_m[w][row] - top);
        const float4 v =
            *reinterpret_cast<const float4*>(results + w * (S::kWarpRing / 4) + row * S::kMergeRow + c0);
        sum = fmaf(part_l[w][row], f, sum);
        acc = make_float4(fmaf(v.x, f, acc.x), fmaf(v.y, f, acc.y), fmaf(v.z, f, acc.z), fmaf(v.w, f, acc.w));
      }
      if (whole) {
        const int r = x.row0 + row;
        if (r < rows) {
          const int tk = r / p.group, h = x.head * p.group + r - tk * p.group;
          // a row that saw nothing: zeros, and a log-sum of -inf
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          __nv_bfloat162 v[2] = {__floats2bfloat162_rn(acc.x * inv, acc.y * inv),
                                 __floats2bfloat162_rn(acc.z * inv, acc.w * inv)};
          *reinterpret_cast<uint2*>(p.out + (size_t)(tok0 + tk) * p.ldo + h * D + c0) = *reinterpret_cast<uint2*>(v);
          if (p.lse != nullptr && c0 == 0)
            p.lse[(size_t)(tok0 + tk) * p.q_heads + h] =
                sum == 0.f ? kNegInf : (top - kWeightUp + log2f(sum)) * 0.6931471805599453f;
        }
      } else {
        *reinterpret_cast<float4*>(part + row * D + c0) = acc;
        if (c0 == 0) {
          part[ROWS * D + row] = top;
          part[ROWS * D + ROWS + row] = sum;
        }
      }
    }
    fence_proxy_async_smem();  // the results' places become the ring again
    __syncthreads();
    u += x.unit1 - x.unit0;
  }
}

// Merge of the items that span CTAs: CTA c takes the one of its record, ROWS
// rows per blockIdx.y.  WPR warps share a row: each takes every WPR-th part,
// D / 32 channels a lane; they meet in shared memory.  TILE: parts as the tile
// kernel's fragments lie.
template <int D, int ROWS, int WPR, bool TILE>
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
    if constexpr (TILE) {
      // fragments of 16 rows x 8 channels: lane 4 g + t of its warp left
      // channels 2 t, 2 t + 1 of rows g and g + 8
      const int c = lane * CPL;
      const float* at = part + (((row >> 4) * (D / 8) + (c >> 3)) * 32 + (row & 7) * 4 + ((c & 7) >> 1)) * 4 +
                        ((row >> 3) & 1) * 2;
#pragma unroll
      for (int j = 0; j < CPL; j += 2)
        *reinterpret_cast<float2*>(v + j) = *reinterpret_cast<const float2*>(at + j * 2);
    } else if constexpr (CPL == 4) {
      *reinterpret_cast<float4*>(v) = *reinterpret_cast<const float4*>(part + row * D + lane * 4);
    } else {
      *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(part + row * D + lane * 2);
    }
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
    p.lse[tk * p.q_heads + h] = sum == 0.f ? kNegInf : (top - kWeightUp + log2f(sum)) * 0.6931471805599453f;
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

template <int D, bool INT8, int NR>
cudaError_t launch_rows_nr(const AttendParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int ctas,
                           cudaStream_t st, bool pdl) {
  static GrowOnlyAttr opened;
  const void* fn = (const void*)qg_attend_rows_kernel<D, INT8, NR>;
  constexpr int smem = RowsSmem<D, NR>::kTotal;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return cudaErrorInvalidDevice;
  const int e = opened.ensure(
      dev, smem, [&](int v) { return (int)cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, v); });
  if (e != 0) return (cudaError_t)e;
  void* args[] = {(void*)&tk, (void*)&tv, (void*)&p};
  return launch_pdl(fn, dim3(ctas), kRowsWarps<NR> * 32, smem, args, st, pdl);
}
template <int D, bool INT8>
cudaError_t launch_rows(const AttendParams& p, const CUtensorMap& tk, const CUtensorMap& tv, int tile_rows, int ctas,
                        cudaStream_t st, bool pdl) {
  switch (tile_rows) {
    case 8: return launch_rows_nr<D, INT8, 1>(p, tk, tv, ctas, st, pdl);
    case 16: return launch_rows_nr<D, INT8, 2>(p, tk, tv, ctas, st, pdl);
    case 24: return launch_rows_nr<D, INT8, 3>(p, tk, tv, ctas, st, pdl);
  }
  if constexpr (D == 64) {
    if (tile_rows == 32) return launch_rows_nr<D, INT8, 4>(p, tk, tv, ctas, st, pdl);
  }
  return cudaErrorInvalidValue;
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
cudaError_t launch_merge(const AttendParams& p, int tile_rows, int ctas, cudaStream_t st, bool pdl) {
  void* args[] = {(void*)&p, (void*)&tile_rows};
  if (tile_rows == kTileRows)
    return launch_pdl((const void*)qg_attend_merge_kernel<D, 16, 1, true>, dim3(ctas, kTileRows / 16), 512, 0, args, st, pdl);
  return launch_pdl((const void*)qg_attend_merge_kernel<D, 2, 4, false>, dim3(ctas, tile_rows / 2), 256, 0, args, st, pdl);
}

// Rows of an item.  The rows kernel takes 8 to 24 (32 where a head of 64
// leaves the registers) and its time per position grows with them; the tile
// kernel's is that of 128 for any number.  16 sequences of up to 8000
// positions, 8 key heads of 128: 24 rows 72 us against 88, 32 rows 95 (two
// items of 16, or one that spills) against 90.
int tile_rows_of(int wanted, int head_dim) {
  const int rows = wanted <= 8 ? 8 : (wanted + 7) / 8 * 8;
  return rows <= (head_dim == 64 ? 32 : 24) ? rows : kTileRows;
}

}  // namespace

AttendSplit attend_split(int rows, int head_dim) {
  const int tile_rows = tile_rows_of(rows, head_dim);
  return {tile_rows, tile_rows == kTileRows ? kTilePos : kUnit};
}

bool attend_tiles(int rows, int head_dim) { return tile_rows_of(rows, head_dim) == kTileRows; }

size_t attend_workspace(int head_dim, int rows_max, int sms) {
  return sizeof(MergeRecord) * sms + (size_t)2 * sms * tile_rows_of(rows_max, head_dim) * (head_dim + 2) * 4;
}

cudaError_t launch_attend(AttendParams p, void* workspace, const uint8_t* k, const uint8_t* v, const CUtensorMap* tk,
                          const CUtensorMap* tv, int rows, int head_dim, bool int8, int sms, cudaStream_t st, bool pdl) {
  rows = tile_rows_of(rows, head_dim);
  p.records = static_cast<MergeRecord*>(workspace);
  p.partial = reinterpret_cast<float*>(p.records + sms);
  cudaError_t e;
  if (rows == kTileRows) {
    if (head_dim == 128)
      e = int8 ? launch_tile<128, true>(p, k, v, sms, st, pdl) : launch_tile<128, false>(p, k, v, sms, st, pdl);
    else
      e = int8 ? launch_tile<64, true>(p, k, v, sms, st, pdl) : launch_tile<64, false>(p, k, v, sms, st, pdl);
  } else if (head_dim == 128) {
    e = int8 ? launch_rows<128, true>(p, *tk, *tv, rows, sms, st, pdl)
             : launch_rows<128, false>(p, *tk, *tv, rows, sms, st, pdl);
  } else {
    e = int8 ? launch_rows<64, true>(p, *tk, *tv, rows, sms, st, pdl)
             : launch_rows<64, false>(p, *tk, *tv, rows, sms, st, pdl);
  }
  if (e != cudaSuccess) return e;
  return head_dim == 128 ? launch_merge<128>(p, rows, sms, st, pdl) : launch_merge<64>(p, rows, sms, st, pdl);
}

}  // namespace qg
