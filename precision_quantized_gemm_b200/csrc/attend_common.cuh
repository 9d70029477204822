// attend_common.cuh — what the attention kernels over the quantised cache
// share: the split of the work over the CTAs, the softmax in the codes' units
// and the decode of codes to f16.
//
// One row of an item is one query head of one drafted token; the rows of the
// query heads that share a key head are stacked (row = token * group + head).
// With key codes kc and scale ks, value codes vc and scale vs:
//   s_j = scale * log2(e) * (q . kc_j) ks_j            (base-2 scores)
//   t_j = s_j + log2(vs_j),  m: max_j t_j, or less by up to kRescaleAt (tiles:
//                            also more, by up to 1)
//   w_j = 2^(t_j - m + 7)  in [0, 2^15],  l = sum_j w_j / vs_j
//   o   = sum_j w_j vc_j / l,       lse = ln 2 (m - 7 + log2 l)
// so the value scale rides in the exponent and the weights are f16 (11 bits;
// bf16 would give them 8).  l has them in fp32; the products round them to
// f16, whose step below 2^-14 is 2^-24: each is off by 2^-31 of the largest at
// most where it is that small (the 7 brings the largest near f16's top), n of
// them by n 2^-31 of a value, half of bf16's half step for 2^22 positions.
// Codes are exact in f16.  Queries are f16 after a
// power of two per row brings their largest magnitude to [2^14, 2^15).
// Sums, maxima and accumulators are fp32.
//
// Value scales are held to [2^-80, 2^125].  A smaller row counts as that small
// (below 4e-22 in magnitude), which keeps l finite: w_j / vs_j is at most
// 2^95, and 2^31 positions of it stay below fp32's 2^128.  The upper bound
// keeps 1 / vs normal; no row of bf16 values reaches it.  A NaN
// scale (a row with a NaN or an infinity) makes the rows that see it NaN.
// Where the scales a row sees are more than 2^100 apart, the weight of the
// smaller ones may underflow, and their share of l with it.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "internal.h"
#include "loads.cuh"
#include "ptx.cuh"

namespace qg {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kVsMin = 8.271806125530277e-25f;  // 2^-80
constexpr float kVsMax = 4.253529586511731e37f;   // 2^125
constexpr float kRescaleAt = 8.f;                 // log2: how far a score may pass its row's reference
constexpr float kWeightUp = 7.f;                  // log2 of the weight at the reference

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two e4m3 codes (the low or the high half of w) -> two f16.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(w));
  return r;
}
__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Four codes of one word -> f16 pairs (0, 1) and (2, 3).  int8: the byte with
// its top bit flipped is code + 128, which under the f16 exponent of 1024 is
// the f16 number 1152 + code.
template <bool INT8>
__device__ __forceinline__ void decode4(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (INT8) {
    const uint32_t u = w ^ 0x80808080u;
    lo = hsub2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
    hi = hsub2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
  } else {
    lo = e4m3x2_to_f16x2((uint16_t)w);
    hi = e4m3x2_to_f16x2((uint16_t)(w >> 16));
  }
}

// ------------------------------------------------------- split of the work --
// The positions of every (sequence, key head, row tile) are cut into units of
// `unit` positions; the units of all items in order are dealt to the CTAs in
// equal contiguous shares, so ragged lengths balance without a host copy.  An
// item that spans CTAs leaves one partial (o, m, l) per CTA, which a second
// kernel merges in CTA order: the same inputs give the same bits.
// All counts are 32-bit (the host bounds the units).
struct Sched {
  int pre[kAttendMaxBatch + 1];   // units of the sequences before b; [batch]: all
  int tok0[kAttendMaxBatch];      // first token in q
  int n[kAttendMaxBatch];         // tokens
  int len[kAttendMaxBatch];       // cached positions
  int warp_tot[32];
};
struct Share {
  int total, quota, extra, ctas;  // units; the first `extra` CTAs take quota + 1
  __device__ __forceinline__ int begin(int c) const { return c * quota + min(c, extra); }
  // The CTA whose share holds unit u.
  __device__ __forceinline__ int of(int u) const {
    const int wide = extra * (quota + 1);
    return u < wide ? (int)((unsigned)u / (unsigned)(quota + 1)) : extra + (int)((unsigned)(u - wide) / (unsigned)quota);
  }
};

// Every thread of the CTA calls it (blockDim.x a multiple of 32, up to 1024);
// ends with a barrier.
__device__ __forceinline__ Share plan_units(const AttendParams& p, int tile_rows, int unit, Sched& s) {
  const int per = (p.batch + blockDim.x - 1) / blockDim.x;
  const int b0 = threadIdx.x * per, b1 = min(b0 + per, p.batch);
  int sum = 0;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int a = min(max(fresh(p.q_offsets + b), 0), p.tokens);
    const int n = max(min(max(fresh(p.q_offsets + b + 1), 0), p.tokens) - a, 0);
    // the table's row covers ldp pages
    const int len = min(max(fresh(p.kv_len + b), 0), p.ldp << p.page_shift);
    s.tok0[b] = a;
    s.n[b] = n;
    s.len[b] = len;
    const int tiles = (min(n, p.max_q) * p.group + tile_rows - 1) / tile_rows;
    // a sequence without cached positions still has rows to write (zeros)
    const int u = tiles * p.kv_heads * max((len + unit - 1) / unit, 1);
    s.pre[b + 1] = u;
    sum += u;
  }
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  int inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (l >= d) inc += o;
  }
  if (l == 31) s.warp_tot[w] = inc;
  __syncthreads();
  int run = l < w ? s.warp_tot[l] : 0;  // of the warps before
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) run += __shfl_xor_sync(0xffffffffu, run, d);
  run += inc - sum;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    run += s.pre[b + 1];
    s.pre[b + 1] = run;
  }
  if (threadIdx.x == 0) s.pre[0] = 0;
  __syncthreads();
  Share x;
  x.total = s.pre[p.batch];
  x.ctas = max(min((int)gridDim.x, x.total), 1);
  x.quota = (unsigned)x.total / (unsigned)x.ctas;
  x.extra = x.total - x.quota * x.ctas;
  return x;
}

// One CTA's part of one item: units [unit0, unit1) of its `units`.
struct Piece {
  int seq, head, row0, unit0, unit1, units;
};
__device__ __forceinline__ Piece find_piece(const AttendParams& p, const Sched& s, int tile_rows, int u, int end) {
  int lo = 0, hi = p.batch - 1;  // the last sequence with pre[b] <= u
#pragma unroll 1
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.pre[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  Piece x;
  x.seq = lo;
  const int tiles = (min(s.n[lo], p.max_q) * p.group + tile_rows - 1) / tile_rows;
  x.units = (unsigned)(s.pre[lo + 1] - s.pre[lo]) / (unsigned)(tiles * p.kv_heads);
  const int r = u - s.pre[lo];
  const int item = (unsigned)r / (unsigned)x.units;
  x.unit0 = r - item * x.units;
  x.unit1 = min(x.units, x.unit0 + (end - u));
  x.head = (unsigned)item / (unsigned)tiles;
  x.row0 = (item - x.head * tiles) * tile_rows;
  return x;
}

// The piece after x in a share: the next item from its first unit (u) on,
// without a search or a division.  Call with u < end.
__device__ __forceinline__ void next_piece(const AttendParams& p, const Sched& s, int tile_rows, int unit, int u, int end,
                                           Piece& x) {
  x.row0 += tile_rows;
  if (x.row0 >= min(s.n[x.seq], p.max_q) * p.group) {
    x.row0 = 0;
    if (++x.head == p.kv_heads) {
      x.head = 0;
      // past sequences without tokens; u < end: there is one with units
      do ++x.seq;
      while (s.pre[x.seq + 1] <= u);
      x.units = max((s.len[x.seq] + unit - 1) / unit, 1);
    }
  }
  x.unit0 = 0;
  x.unit1 = min(x.units, end - u);
}

// What the merge has to know of an item that starts in a CTA's share and goes
// on past it (there is at most one): every CTA of the grid leaves one record
// in the workspace, `last` < 0 for none.  The parts are this CTA's slot and
// the first slot of each CTA up to `last`.
struct MergeRecord {
  int last, slot, row0, rows, tok0, head;
  int pad[2];
};
__device__ __forceinline__ MergeRecord merge_record(const AttendParams& p, const Sched& s, const Share& share,
                                                    int tile_rows) {
  MergeRecord r = {};
  r.last = -1;
  const int c = blockIdx.x;
  if (c + 1 >= share.ctas) return r;  // nothing goes on past the last share
  const int begin = share.begin(c), end = share.begin(c + 1);
  const Piece x = find_piece(p, s, tile_rows, end - 1, share.total);
  const int first = end - 1 - x.unit0;  // the item's first unit
  if (first < begin || x.unit0 + 1 >= x.units) return r;
  r.last = share.of(first + x.units - 1);
  r.slot = 2 * c + (first > begin ? 1 : 0);
  r.row0 = x.row0;
  r.rows = min(s.n[x.seq], p.max_q) * p.group;
  r.tok0 = s.tok0[x.seq];
  r.head = x.head;
  return r;
}

// Which of 64 positions token i of a sequence sees, as bits: of the first
// `count`, the `before` that precede the drafted tokens (negative: the first
// is drafted token -before), and the drafted ones of its mask row.  (i < 0: a
// row past the last, nothing.)  In two steps, so that the loads for several
// rows are in flight together: the mask row's bits from the window on, and
// what the window makes of them.
__device__ __forceinline__ unsigned long long drafted_bits(const AttendParams& p, int tok0, int i, int before) {
  if (p.mask == nullptr) return 0ull;  // causal: nothing to load
  const int word = before < 0 ? -before >> 6 : 0, shift = before < 0 ? -before & 63 : 0;
  const unsigned long long* row = p.mask + (size_t)(tok0 + max(i, 0)) * p.mask_words;
  unsigned long long bits = 0, next = 0;
  if (i >= 0 && word < p.mask_words) bits = fresh(row + word);
  if (i >= 0 && shift > 0 && word + 1 < p.mask_words) next = fresh(row + word + 1);
  return shift > 0 ? bits >> shift | next << (64 - shift) : bits;
}
__device__ __forceinline__ unsigned long long seen_bits(const AttendParams& p, int i, int count, int before,
                                                        unsigned long long drafted) {
  if (i < 0 || count <= 0) return 0ull;
  const unsigned long long all = count >= 64 ? ~0ull : (1ull << count) - 1;
  if (before >= 64) return all;
  if (p.mask == nullptr) {
    const int n = i + 1 + before;  // drafted tokens up to i
    drafted = n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
  } else if (before > 0) {
    drafted <<= before;
  }
  const unsigned long long prefix = before > 0 ? (1ull << before) - 1 : 0ull;
  return all & (prefix | drafted);
}

// Scale's log2 and reciprocal with the bounds of the header comment.  log2 is
// the exponent plus the approximate log2 of the mantissa in [1, 2), whose
// absolute error is 2^-22 (that of the whole would grow with the exponent).
__device__ __forceinline__ void value_scale(float vs, float& log2_vs, float& inv_vs) {
  const float c = fminf(fmaxf(vs, kVsMin), kVsMax);  // NaN -> kVsMin; normal
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv_vs) : "f"(c));
  const uint32_t bits = __float_as_uint(c);
  float lg;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(lg) : "f"(__uint_as_float((bits & 0x7fffffu) | 0x3f800000u)));
  lg += (float)((int)(bits >> 23) - 127);
  log2_vs = vs - vs == 0.f ? lg : __uint_as_float(0x7fc00000u);
}

// Power of two that brings a row's largest magnitude to [2^14, 2^15) (below
// 2^-112: as near as 2^126 brings it), and its inverse; 1 for a zero row or
// one with an infinity.  Both are normal.
__device__ __forceinline__ void row_power(float amax, float& up, float& down) {
  const int e = (int)(__float_as_uint(amax) >> 23) & 0xff;
  const int shift = amax > 0.f && e < 255 ? min(14 + 127 - e, 126) : 0;
  up = __uint_as_float((uint32_t)(127 + shift) << 23);
  down = __uint_as_float((uint32_t)(127 - shift) << 23);
}

}  // namespace qg
