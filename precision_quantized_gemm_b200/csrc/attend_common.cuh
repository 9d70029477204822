// attend_common.cuh — what the attention kernels over the quantised cache
// share: the split of the work over the CTAs, the softmax in the codes' units
// and the decode of codes to f16.
//
// One row of an item is one query head of one drafted token; the rows of the
// query heads that share a key head are stacked (row = token * group + head).
// With key codes kc and scale ks, value codes vc and scale vs:
//   s_j = scale * log2(e) * (q . kc_j) ks_j            (base-2 scores)
//   t_j = s_j + log2(vs_j),  m = max_j t_j
//   w_j = 2^(t_j - m)  in [0, 1],   l = sum_j w_j / vs_j
//   o   = sum_j w_j vc_j / l,       lse = ln 2 (m + log2 l)
// so the value scale rides in the exponent and the weights are f16 (11 bits;
// bf16 would give them 8): a weight below 2^-24 of the largest adds nothing
// that bf16 outputs keep.  Codes are exact in f16.  Queries are f16 after a
// power of two per row brings their largest magnitude to [2^14, 2^15).
// Sums, maxima and accumulators are fp32.
//
// Value scales are held to [2^-110, 2^95] (a smaller row counts as that
// small: below 4e-31 in magnitude), which keeps 1 / vs and l finite.  A NaN
// scale (a row with a NaN or an infinity) makes the rows that see it NaN.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace qg {

constexpr float kNegInf = -__builtin_huge_valf();
constexpr float kVsMin = 7.703719777548943e-34f;  // 2^-110
constexpr float kVsMax = 3.961408125713217e28f;   // 2^95

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
struct Share {
  long long total, begin, end;  // units
  int ctas;                     // CTAs with work
};

__device__ __forceinline__ int seq_tokens(const AttendParams& p, int b) {
  const int a = min(max(__ldg(p.q_offsets + b), 0), p.tokens);
  const int e = min(max(__ldg(p.q_offsets + b + 1), 0), p.tokens);
  return max(e - a, 0);
}
__device__ __forceinline__ int seq_len(const AttendParams& p, int b) {
  // the table's row covers ldp pages
  const long long cap = (long long)p.ldp << p.page_shift;
  return (int)min((long long)max(__ldg(p.kv_len + b), 0), cap);
}
__device__ __forceinline__ int seq_row_tiles(const AttendParams& p, int n, int tile_rows) {
  return (min(n, p.max_q) * p.group + tile_rows - 1) / tile_rows;
}
// a sequence without cached positions still has rows to write (zeros)
__device__ __forceinline__ int seq_units(int len, int unit) { return max((len + unit - 1) / unit, 1); }

// pre[b] = units of the sequences before b, pre[batch] = all units.  Every
// thread of the CTA calls it (blockDim.x a multiple of 32, up to 1024).
__device__ __forceinline__ void scan_units(const AttendParams& p, int tile_rows, int unit, long long* pre,
                                           long long* warp_tot) {
  const int per = (p.batch + blockDim.x - 1) / blockDim.x;
  const int b0 = threadIdx.x * per;
  long long sum = 0;
  for (int b = b0; b < min(b0 + per, p.batch); ++b) {
    const int rt = seq_row_tiles(p, seq_tokens(p, b), tile_rows);
    const long long u = rt ? (long long)rt * p.kv_heads * seq_units(seq_len(p, b), unit) : 0;
    pre[b + 1] = u;
    sum += u;
  }
  const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
  long long inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, d);
    if (l >= d) inc += o;
  }
  if (l == 31) warp_tot[w] = inc;
  __syncthreads();
  long long run = inc - sum;
  for (int j = 0; j < w; ++j) run += warp_tot[j];
  for (int b = b0; b < min(b0 + per, p.batch); ++b) {
    run += pre[b + 1];
    pre[b + 1] = run;
  }
  if (threadIdx.x == 0) pre[0] = 0;
  __syncthreads();
}
__device__ __forceinline__ long long share_begin(long long total, int ctas, int c) { return total * c / ctas; }
// The CTA whose share holds unit u.
__device__ __forceinline__ int share_of(long long total, int ctas, long long u) {
  return (int)(((u + 1) * ctas - 1) / total);
}
__device__ __forceinline__ Share my_share(const AttendParams& p, const long long* pre, int ctas_max, int c) {
  Share s;
  s.total = pre[p.batch];
  s.ctas = (int)min((long long)ctas_max, s.total);
  s.begin = c < s.ctas ? share_begin(s.total, s.ctas, c) : 0;
  s.end = c < s.ctas ? share_begin(s.total, s.ctas, c + 1) : 0;
  return s;
}

// One CTA's part of one item.
struct Piece {
  int seq, head, row0;       // sequence, key head, first row
  int tok0, n, len;          // first token in q, tokens, cached positions
  int rows;                  // rows of the sequence (tokens within max_q x group)
  int unit0, unit1, units;   // units [unit0, unit1) of the item's `units`
};
__device__ __forceinline__ Piece find_piece(const AttendParams& p, const long long* pre, int tile_rows, int unit,
                                            long long u, long long end) {
  int lo = 0, hi = p.batch - 1;  // the last sequence with pre[b] <= u
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (pre[mid] <= u) lo = mid;
    else hi = mid - 1;
  }
  Piece x;
  x.seq = lo;
  x.n = seq_tokens(p, lo);
  x.len = seq_len(p, lo);
  x.tok0 = min(max(__ldg(p.q_offsets + lo), 0), p.tokens);
  x.rows = min(x.n, p.max_q) * p.group;
  const int rt = seq_row_tiles(p, x.n, tile_rows);
  x.units = seq_units(x.len, unit);
  const long long r = u - pre[lo];
  const int item = (int)(r / x.units);
  x.unit0 = (int)(r % x.units);
  x.unit1 = (int)min((long long)x.units, x.unit0 + (end - u));
  x.head = item / rt;
  x.row0 = (item % rt) * tile_rows;
  return x;
}

// Which of the 64 positions from `pos0` on token i of a sequence sees, as bits:
// the positions before the drafted ones, and the drafted tokens of its mask
// row, up to `end`.  (i < 0: a row past the last, nothing.)
__device__ __forceinline__ unsigned long long seen_bits(const AttendParams& p, int tok0, int i, int pos0, int past,
                                                        int end) {
  const int count = end - pos0, before = past - pos0;  // positions in range; those before the drafted ones
  if (i < 0 || count <= 0) return 0ull;
  const unsigned long long all = count >= 64 ? ~0ull : (1ull << count) - 1;
  if (before >= 64) return all;
  unsigned long long drafted;  // bit e: drafted token e - before (a negative one is not cached)
  if (p.mask == nullptr) {
    const int n = i + 1 + before;  // drafted tokens up to i
    drafted = n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1;
  } else {
    const unsigned long long* row = p.mask + (size_t)(tok0 + i) * p.mask_words;
    if (before >= 0) {
      drafted = __ldg(row) << before;
    } else {
      const int word = -before >> 6, shift = -before & 63;
      drafted = word < p.mask_words ? __ldg(row + word) >> shift : 0ull;
      if (shift && word + 1 < p.mask_words) drafted |= __ldg(row + word + 1) << (64 - shift);
    }
  }
  const unsigned long long prefix = before > 0 ? (1ull << before) - 1 : 0ull;
  return all & (prefix | drafted);
}

// Scale's log2 and reciprocal with the bounds of the header comment.
__device__ __forceinline__ void value_scale(float vs, float& log2_vs, float& inv_vs) {
  const float c = fminf(fmaxf(vs, kVsMin), kVsMax);  // NaN -> kVsMin
  inv_vs = __fdividef(1.f, c);
  log2_vs = vs - vs == 0.f ? log2f(c) : __uint_as_float(0x7fc00000u);
}

// Power of two that brings a row's largest magnitude to [2^14, 2^15), and its
// inverse; 1 for a zero row or one with an infinity.
__device__ __forceinline__ void row_power(float amax, float& up, float& down) {
  const int e = (int)(__float_as_uint(amax) >> 23) & 0xff;
  const int shift = amax > 0.f && e < 255 ? min(max(14 + 127 - e, -100), 100) : 0;
  up = __uint_as_float((uint32_t)(127 + shift) << 23);
  down = __uint_as_float((uint32_t)(127 - shift) << 23);
}

}  // namespace qg
