// attend_tile.cuh — attention over the quantised cache for many rows per key
// head (trees of drafted tokens): tiles of 128 rows x 128 positions on
// tcgen05, one CTA per SM.
//
//   S = Q K^T      A = Q (TMEM, f16), B = K (shared, f16, K-major)  -> TMEM fp32
//   O += W V       A = W (TMEM, f16), B = V (shared, f16, MN-major) -> TMEM fp32
//
// 16 warps in four roles, joined by mbarriers:
//   0-7   softmax: warp w owns rows 32 (w % 4) .. + 31 (its TMEM lanes), the
//         first or the second 64 positions of a tile: a thread holds 64 scores
//         of one row in registers, agrees on the row's maximum with its
//         partner in warp w ^ 4, and writes the f16 weights to TMEM
//   8-11  decode: codes from global memory to f16 in the swizzled operand
//         tiles, the next tile's codes in registers meanwhile
//   12    MMA: one thread issues S of tile j + 1 before O of tile j
//   13    the tiles ahead: where their positions lie, what of them counts,
//         their scales (log2 and reciprocal once per position), and the
//         prefetch of their codes into L2
// Only warp 13 walks sequences, heads and pages; the others read its tile
// descriptors.  That is for the instruction cache: five roles' loops share
// it, and with a walk inlined into each the warps waited for instructions
// five times as long as they issued (350 us against TIMING for 8 trees of
// 32-64 tokens, 64 query and 8 key heads, 2048-8192 positions).
//
// What bounds it: per tile the two MMAs are 1024 tensor cycles, the 16384
// exponentials 1024 cycles of the 16-wide unit, and shared memory carries the
// decoded tiles twice (64 KB written, 64 KB read by the MMAs: 1024 cycles).
// That is why Q and W sit in TMEM (from shared memory they would add 64 KB a
// tile) and codes do not pass through shared memory on their way to f16.
// The accumulator is rescaled only when a row's maximum has grown by more
// than 2^8 since its reference was taken: weights stay below 256, and sums
// and accumulator keep the same reference, so the result is unchanged.
#pragma once
#include "attend_common.cuh"

namespace qg {

constexpr int kTileRows = 128;
constexpr int kTilePos = 128;       // positions per tile = unit of work
constexpr int kTileThreads = 512;
constexpr int kTileStages = 6;     // descriptors and scales ahead
constexpr float kRescaleAt = 8.f;   // log2

template <int D>
struct TileSmem {
  static constexpr int kOperand = kTilePos * D * 2;    // f16 tile of K or V
  static constexpr int kScales = 3 * kTilePos * 4;     // key scale, log2 vs, 1 / vs
  static constexpr int kTotal = 1024 + 4 * kOperand + kTileStages * kScales;
};
// What a tile is; written by warp 13.
struct TileDesc {
  int run[kTilePos / 16];  // cache row of the 1st of each 16 positions
  int count;               // positions of the sequence from the tile's first on (may pass 128)
  int before;              // those before the drafted tokens (may be negative)
  int first, last;         // of its piece
  int whole;               // the piece is the whole item
  int row0, rows;          // first row, rows of the sequence
  int tok0, head, slot;    // slot: partial result, when not whole
};
// TMEM columns
constexpr int kTmemS = 0;        // two score tiles of 128
constexpr int kTmemO = 256;      // D
constexpr int kTmemW = 384;      // 64: 128 f16 weights
constexpr int kTmemQ = 448;      // D / 2
constexpr int kTmemCols = 512;

__host__ __device__ constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
  return (1u << 4)                            // D = f32; A, B = f16
         | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// D[tmem] (+)= A[tmem, f16] . B[smem]
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// MN-major operand, 128-byte swizzle: rows (K) of 64 f16, 8-row atoms of 1024
// bytes; `mn_step` bytes from one block of 64 to the next.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t mn_step) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFF) >> 4);
  d |= (uint64_t)(mn_step >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,"
      "%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(
          r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ void unpack_f32x2(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t lds_u64(uint32_t a) {
  uint64_t v;
  asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void lds_2u64(uint32_t a, uint64_t& x, uint64_t& y) {
  asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(x), "=l"(y) : "r"(a));
}
// Barrier of the 64 threads of warps w and w ^ 4 (ids 1 .. 4).
__device__ __forceinline__ void pair_sync(int id) { asm volatile("bar.sync %0, 64;" ::"r"(id + 1) : "memory"); }

template <int D, bool INT8>
__global__ void __launch_bounds__(kTileThreads, 1) qg_attend_tile_kernel(const uint8_t* __restrict__ k_codes,
                                                                          const uint8_t* __restrict__ v_codes,
                                                                          const AttendParams p) {
  using S = TileSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Sched sched;
  __shared__ TileDesc descs[kTileStages];
  // full: the operand tile is decoded / the scores, weights, queries are in
  // TMEM; free: its reader is done (s_full also frees K's buffer, o_done the
  // weights').  No barrier can complete two phases past one of its waiters:
  // each next phase needs what that waiter does after the wait.
  __shared__ __align__(8) uint64_t k_full[2], v_full[2], v_free[2], s_full[2], s_free[2], w_full, o_done, q_full, idle,
      d_full[kTileStages], d_free[kTileStages];
  __shared__ uint32_t tmem_ptr;
  __shared__ float swap_a[2][kTileRows], swap_m[2][kTileRows], swap_l[2][kTileRows];  // between partners
  __shared__ bool pair_ok[2][4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t k_tile = base, v_tile = base + 2 * S::kOperand, scales = base + 4 * S::kOperand;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 4);
      mbar_init(&v_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&v_free[i], 1);
      mbar_init(&s_free[i], 8);
    }
    mbar_init(&w_full, 8);
    mbar_init(&o_done, 1);
    mbar_init(&q_full, 8);
    mbar_init(&idle, 1);
    for (int i = 0; i < kTileStages; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_free[i], 13);  // softmax, decode and MMA warps
    }
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(&tmem_ptr, kTmemCols);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  griddep_wait();
  const Share share = plan_units(p, kTileRows, kTilePos, sched);  // also orders the barriers' set-up
  tc_fence_after();
  const uint32_t tmem = tmem_ptr;
  const bool works = (int)blockIdx.x < share.ctas && share.total > 0;
  const int u0 = works ? share.begin(blockIdx.x) : 0, u1 = works ? share.begin(blockIdx.x + 1) : 0;
  const int tiles = u1 - u0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait(bar, parity, p.err, p.wait_ns);
    return ok;
  };

  if (warp < 8) {
    // ------------------------------------------------------------- softmax --
    const int half = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    constexpr int OC = D / 2;     // accumulator columns of this thread
    float m = kNegInf, power = 0.f;
    uint64_t l2 = 0;
    int tok = -1;
    bool live_warp = false;
    int st = 0;
    uint32_t ring = 0;  // parity of the descriptors' turn
    // Partners agree on whether the next descriptor is there: what it says
    // decides which of the pair's barriers they meet at.  (The barrier also
    // ends the turn's use of swap_m.)
    auto open = [&]() {
      wait(&d_full[st], ring);
      __syncwarp();
      if (lane == 0) pair_ok[half][warp & 3] = ok;
      pair_sync(warp & 3);
      return pair_ok[0][warp & 3] && pair_ok[1][warp & 3];
    };
    bool have = tiles > 0 && open();
#pragma unroll 1
    for (int j = 0; j < tiles && have; ++j) {
      const TileDesc& x = descs[st];
      const bool first = x.first, last = x.last;
      if (first) {
        // queries: f16, the row's largest magnitude brought to [2^14, 2^15);
        // this thread's half of the channels
        const int r = x.row0 + row;
        live_warp = x.row0 + (warp & 3) * 32 < x.rows;
        tok = r < x.rows ? r / p.group : -1;
        const __nv_bfloat16* src =
            tok < 0 ? nullptr
                    : p.q + (size_t)(x.tok0 + tok) * p.ldq + (x.head * p.group + r - tok * p.group) * D + half * (D / 2);
        uint32_t q[D / 4];
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) {
          const uint4 v = src ? reinterpret_cast<const uint4*>(src)[c] : make_uint4(0, 0, 0, 0);
          q[4 * c] = v.x;
          q[4 * c + 1] = v.y;
          q[4 * c + 2] = v.z;
          q[4 * c + 3] = v.w;
        }
#pragma unroll
        for (int c = 0; c < D / 4; ++c)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(q[c] << 16)), fabsf(__uint_as_float(q[c] & 0xffff0000u))));
        swap_a[half][row] = amax;
        pair_sync(warp & 3);
        amax = fmaxf(amax, swap_a[half ^ 1][row]);
        float up, down;
        row_power(amax, up, down);
        power = down * p.scale_log2;
#pragma unroll
        for (int c = 0; c < D / 4; ++c) {
          const __half2 h =
              __floats2half2_rn(__uint_as_float(q[c] << 16) * up, __uint_as_float(q[c] & 0xffff0000u) * up);
          q[c] = *reinterpret_cast<const uint32_t*>(&h);
        }
        tmem_st(lanes + kTmemQ + half * (D / 4), q);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full);
        m = kNegInf;
        l2 = 0;
      }
      const uint32_t sc = scales + st * S::kScales + half * 64 * 4;
      wait(&s_full[j & 1], (j >> 1) & 1);
      float t[64];
      float top = kNegInf;
      if (live_warp && __all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        uint32_t lo[32], hi[32];
        tmem_ld32(lanes + kTmemS + (j & 1) * 128 + half * 64, lo);
        tmem_ld32(lanes + kTmemS + (j & 1) * 128 + half * 64 + 32, hi);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < 32; ++i) {
          t[i] = __uint_as_float(lo[i]);
          t[i + 32] = __uint_as_float(hi[i]);
        }
        const uint64_t pw = pack_f32x2(power, power);
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          uint64_t ka, kb, va, vb;
          lds_2u64(sc + i * 4, ka, kb);
          lds_2u64(sc + kTilePos * 4 + i * 4, va, vb);
          unpack_f32x2(fma_f32x2(mul_f32x2(pack_f32x2(t[i], t[i + 1]), pw), ka, va), t[i], t[i + 1]);
          unpack_f32x2(fma_f32x2(mul_f32x2(pack_f32x2(t[i + 2], t[i + 3]), pw), kb, vb), t[i + 2], t[i + 3]);
        }
        if (x.before < kTilePos || x.count < kTilePos) {
          const unsigned long long see = seen_bits(p, x.tok0, tok, x.count - half * 64, x.before - half * 64);
          const uint32_t see_lo = (uint32_t)see, see_hi = (uint32_t)(see >> 32);
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (!((i < 32 ? see_lo >> i : see_hi >> (i - 32)) & 1)) t[i] = kNegInf;
        }
#pragma unroll
        for (int i = 0; i < 64; ++i) top = fmaxf(top, t[i]);
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&s_free[j & 1]);
      swap_m[half][row] = top;
      pair_sync(warp & 3);
      top = fmaxf(top, swap_m[half ^ 1][row]);
      const bool grown = top > m + kRescaleAt || (m == kNegInf && top > kNegInf);
      // the accumulator, the weights' columns and (below) the sums follow the
      // previous tile's product
      if (j > 0) wait(&o_done, (j - 1) & 1);
      if (live_warp && __all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        if (__any_sync(0xffffffffu, grown)) {
          const float f = grown ? ex2(m - top) : 1.f;
          if (grown) m = top;
          l2 = mul_f32x2(l2, pack_f32x2(f, f));
          if (!first) {
#pragma unroll
            for (int c = 0; c < OC; c += 32) {
              uint32_t o[32];
              tmem_ld32(lanes + kTmemO + half * OC + c, o);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
              tmem_st(lanes + kTmemO + half * OC + c, o);
            }
          }
        }
        const float ref = m == kNegInf ? 0.f : -m;
        uint32_t wt[32];
#pragma unroll
        for (int i = 0; i < 64; i += 4) {
          uint64_t ia, ib;
          lds_2u64(sc + 2 * kTilePos * 4 + i * 4, ia, ib);
          const float a = ex2(t[i] + ref), b = ex2(t[i + 1] + ref), c = ex2(t[i + 2] + ref), d = ex2(t[i + 3] + ref);
          l2 = fma_f32x2(pack_f32x2(a, b), ia, l2);
          l2 = fma_f32x2(pack_f32x2(c, d), ib, l2);
          const __half2 h0 = __floats2half2_rn(a, b), h1 = __floats2half2_rn(c, d);
          wt[i / 2] = *reinterpret_cast<const uint32_t*>(&h0);
          wt[i / 2 + 1] = *reinterpret_cast<const uint32_t*>(&h1);
        }
        tmem_st(lanes + kTmemW + half * 32, wt);
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&w_full);

      if (last) {
        // the item's (or this part's) result
        float la, lb;
        unpack_f32x2(l2, la, lb);
        float l = la + lb;
        swap_l[half][row] = l;
        pair_sync(warp & 3);
        l += swap_l[half ^ 1][row];
        if (l != l) m = 0.f;  // a NaN row keeps its place in the merge
        wait(&o_done, j & 1);
        if (live_warp && __all_sync(0xffffffffu, ok)) {
          tc_fence_after();
          const bool whole = x.whole, write = tok >= 0;
          const int r = x.row0 + row;
          float* part = p.partial + (size_t)x.slot * kTileRows * (D + 2);
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const size_t tk = write ? x.tok0 + tok : 0;
          const int h = write ? x.head * p.group + r - tok * p.group : 0;
#pragma unroll
          for (int c = 0; c < OC; c += 32) {
            uint32_t o[32];
            tmem_ld32(lanes + kTmemO + half * OC + c, o);
            tmem_ld_wait();
            if (write && whole) {
              __nv_bfloat16* dst = p.out + tk * p.ldo + h * D + half * OC + c;
#pragma unroll
              for (int i = 0; i < 32; i += 8) {
                // a row that saw nothing: zeros (its weights were all zero)
                __nv_bfloat162 v[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  v[e] = __floats2bfloat162_rn(__uint_as_float(o[i + 2 * e]) * inv, __uint_as_float(o[i + 2 * e + 1]) * inv);
                reinterpret_cast<uint4*>(dst + i)[0] = *reinterpret_cast<const uint4*>(v);
              }
            } else if (write) {
              float* dst = part + row * D + half * OC + c;
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<uint4*>(dst + i) = make_uint4(o[i], o[i + 1], o[i + 2], o[i + 3]);
            }
          }
          if (write && half == 0) {
            if (whole) {
              if (p.lse != nullptr)
                p.lse[tk * p.q_heads + h] = l == 0.f ? kNegInf : (m + log2f(l)) * 0.6931471805599453f;
            } else {
              part[kTileRows * D + row] = m;
              part[kTileRows * D + kTileRows + row] = l;
            }
          }
          tc_fence_before();
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_free[st]);
      if (++st == kTileStages) st = 0, ring ^= 1;
      if (j + 1 < tiles) have = open();
    }
  } else if (warp < 12) {
    // -------------------------------------------------------------- decode --
    // K of tile j + 1 before V of tile j.  A lane holds 16 codes of a row: the
    // 8 lanes of a store phase are 2 rows x 4 of the 16-byte chunks of one
    // 64-channel block, which the swizzle spreads over all banks.
    constexpr int RPI = D == 128 ? 4 : 8;     // rows per warp instruction
    constexpr int N = 32 / RPI;               // instructions per warp and tile
    const int c = D == 128 ? (lane & 3) + ((lane >> 4) << 2) : lane & 3;
    const int r0 = (warp - 8) * 32 + (D == 128 ? (lane >> 2) & 3 : lane >> 2);
    auto load = [&](int j, const uint8_t* codes, uint4 (&buf)[N], bool done) {
      const int st = j % kTileStages;
      wait(&d_full[st], (j / kTileStages) & 1);
      if (!__all_sync(0xffffffffu, ok)) return;
      const TileDesc& x = descs[st];
      const int run[2] = {x.run[(warp - 8) * 2], x.run[(warp - 8) * 2 + 1]};
      const int count = x.count - r0;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        buf[i] = make_uint4(0u, 0u, 0u, 0u);
        if (i * RPI < count)
          buf[i] = __ldg(reinterpret_cast<const uint4*>(
                             codes + (size_t)(run[i / (N / 2)] + (r0 & 15) + i % (N / 2) * RPI) * D) + c);
      }
      if (done) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_free[st]);
      }
    };
    auto store = [&](uint32_t tile, const uint4 (&buf)[N]) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int r = r0 + i * RPI;
        const uint32_t line = tile + (D == 128 ? (uint32_t)(c >> 2) * (kTilePos * 128) : 0u) + r * 128;
        const uint32_t w[4] = {buf[i].x, buf[i].y, buf[i].z, buf[i].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t f[4];
          decode4<INT8>(w[2 * e], f[0], f[1]);
          decode4<INT8>(w[2 * e + 1], f[2], f[3]);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(line + ((((c & 3) * 2 + e) ^ (r & 7)) << 4)),
                       "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3])
                       : "memory");
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
    };
    uint4 kb[N] = {}, vb[N] = {};
    if (tiles > 0) load(0, k_codes, kb, false);
    // turn j: K of tile j + 1, then V of tile j (turn -1: only K)
#pragma unroll 1
    for (int j = -1; j < tiles; ++j) {
      const int i = j + 1;
      if (i < tiles) {
        if (i >= 2) wait(&s_full[i & 1], ((i - 2) >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        store(k_tile + (i & 1) * S::kOperand, kb);
        if (lane == 0) mbar_arrive(&k_full[i & 1]);
        if (i + 1 < tiles) load(i + 1, k_codes, kb, false);
      }
      if (j >= 0) {
        if (j >= 2) wait(&v_free[j & 1], ((j - 2) >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        store(v_tile + (j & 1) * S::kOperand, vb);
        if (lane == 0) mbar_arrive(&v_full[j & 1]);
      }
      if (i < tiles) load(i, v_codes, vb, true);
    }
  } else if (warp == 12) {
    // ----------------------------------------------------------------- MMA --
    if (lane == 0) {
      const uint64_t kd = sdesc_sw128(k_tile), vd = sdesc_mn_sw128(v_tile, kTilePos * 128);
      int queries = 0;
      bool first = false;  // tile j + 1 is the first of its piece
      auto look = [&](int j) {
        const int st = j % kTileStages;
        if (!wait(&d_full[st], (j / kTileStages) & 1)) return;
        first = descs[st].first;
        mbar_arrive(&d_free[st]);
      };
      auto scores = [&](int j) {
        if (first && !wait(&q_full, queries++ & 1)) return;
        if (!wait(&k_full[j & 1], (j >> 1) & 1)) return;
        if (j >= 2 && !wait(&s_free[j & 1], ((j - 2) >> 1) & 1)) return;
        tc_fence_after();
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          mma_f16_ts(tmem + kTmemS + (j & 1) * 128, tmem + kTmemQ + 8 * k,
                     kd + (((j & 1) * S::kOperand + (k >> 2) * (kTilePos * 128) + (k & 3) * 32) >> 4),
                     idesc_f16(kTilePos, false), k > 0);
        mma_commit(&s_full[j & 1]);
      };
      // turn j: scores of tile j + 1, then the product of tile j; the other
      // way round where a piece starts: its first scores need its queries,
      // which wait for the last piece's last product
#pragma unroll 1
      for (int j = -1; j < tiles && ok; ++j) {
        const bool start = j >= 0 && first;  // tile j opens its piece
        if (j + 1 < tiles) look(j + 1);
        else first = false;
#pragma unroll 1
        for (int part = 0; part < 2 && ok; ++part) {
          if ((part == 1) == first) {
            if (j + 1 < tiles) scores(j + 1);
          } else if (j >= 0) {
            if (!wait(&w_full, j & 1) || !wait(&v_full[j & 1], (j >> 1) & 1)) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < kTilePos / 16; ++k)
              mma_f16_ts(tmem + kTmemO, tmem + kTmemW + 8 * k, vd + (((j & 1) * S::kOperand + k * 2048) >> 4),
                         idesc_f16(D, true), !start || k > 0);
            mma_commit(&o_done);
            mma_commit(&v_free[j & 1]);
          }
        }
      }
      // MMAs still in flight (a wait ran out) end before TMEM is given up
      mma_commit(&idle);
      (void)mbar_wait(&idle, 0, p.err, p.wait_ns);
    }
    __syncwarp();
  } else if (warp == 13) {
    // ------------------------------------------------- scales and prefetch --
    // A turn loads what tile j + 1 needs before it hands over tile j.  Lane i
    // has positions 4 i .. 4 i + 3: within one run of 16, whose row its first
    // lane hands on.
    Piece x = {};
    int tile = 0, len = 0;
    auto step = [&](int j) {
      if (j == 0 || tile + 1 == x.unit1) {
        x = find_piece(p, sched, kTileRows, u0 + j, u1);
        tile = x.unit0;
        len = sched.len[x.seq];
      } else {
        ++tile;
      }
    };
    int row = 0, count = 0;
    float4 ks = {}, vs = {};
    auto fetch = [&]() {
      count = len - tile * kTilePos;
      row = 0;
      ks = vs = make_float4(1.f, 1.f, 1.f, 1.f);
      if (lane * 4 < count) {
        const int pos = tile * kTilePos + lane * 4;
        const int page = min(max(__ldg(p.table + (size_t)x.seq * p.ldp + (pos >> p.page_shift)), 0), p.pages - 1);
        row = (page * p.kv_heads + x.head << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        ks = __ldg(reinterpret_cast<const float4*>(p.k_scale + row));
        vs = __ldg(reinterpret_cast<const float4*>(p.v_scale + row));
        if ((lane & 3) == 0) {
          bulk_prefetch_l2(k_codes + (size_t)row * D, 16 * D);
          bulk_prefetch_l2(v_codes + (size_t)row * D, 16 * D);
        }
      }
    };
    if (tiles > 0) {
      step(0);
      fetch();
    }
    int st = 0;
    uint32_t ring = 1;
#pragma unroll 1
    for (int j = 0; j < tiles; ++j) {
      if (j >= kTileStages) wait(&d_free[st], ring);
      if (!__all_sync(0xffffffffu, ok)) break;
      TileDesc& d = descs[st];
      if ((lane & 3) == 0) d.run[lane >> 2] = row;
      if (lane == 0) {
        d.count = count;
        d.before = count - sched.n[x.seq];
        d.first = j == 0 || tile == x.unit0;
        d.last = tile + 1 == x.unit1;
        d.whole = x.unit0 == 0 && x.unit1 == x.units;
        d.row0 = x.row0;
        d.rows = min(sched.n[x.seq], p.max_q) * p.group;
        d.tok0 = sched.tok0[x.seq];
        d.head = x.head;
        d.slot = 2 * blockIdx.x + (j == tile - x.unit0 ? 0 : 1);  // the share's first piece or a later one
      }
      const uint32_t at = scales + st * S::kScales + lane * 16;
      const float k4[4] = {ks.x, ks.y, ks.z, ks.w}, v4[4] = {vs.x, vs.y, vs.z, vs.w};
      float a[4], b[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) value_scale(v4[i], a[i], b[i]);
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(k4[0]), "f"(k4[1]), "f"(k4[2]),
                   "f"(k4[3])
                   : "memory");
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + kTilePos * 4), "f"(a[0]), "f"(a[1]),
                   "f"(a[2]), "f"(a[3])
                   : "memory");
      asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + 2 * kTilePos * 4), "f"(b[0]), "f"(b[1]),
                   "f"(b[2]), "f"(b[3])
                   : "memory");
      if (j + 1 < tiles) {
        step(j + 1);
        fetch();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_full[st]);
      if (++st == kTileStages) st = 0, ring ^= 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace qg
