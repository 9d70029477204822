// attend_tile.cuh — attention over the quantised cache for many rows per key
// head (trees of drafted tokens): tiles of 128 rows x 128 positions on
// tcgen05, one CTA per SM.
//
//   S = Q K^T      A = Q (TMEM, f16), B = K (shared, f16, K-major)  -> TMEM fp32
//   O += W V       A = W (TMEM, f16), B = V (shared, f16, MN-major) -> TMEM fp32
//
// 28 warps in four roles, joined by mbarriers:
//   0-15  softmax: warps 0-7 take the even tiles, 8-15 the odd ones; each
//         group has its own scores, accumulator, maxima and sums, which meet
//         when a piece ends.  A warp has 16 rows (half of the 32 TMEM lanes it
//         may touch), a thread 2 rows x 32 positions (the 16x256b fragments:
//         one position's scales serve 8 rows of a load), and writes the f16
//         weights over the scores in TMEM.
//   16-23 decode: codes from global memory to f16 in the swizzled operand
//         tiles, the next tile's codes in registers meanwhile
//   24    MMA: one thread issues scores and products as they can go
//   25-27 the tiles ahead, in turn: where their positions lie, what of them
//         counts, and their scales (log2 and reciprocal once per position)
//
// What bounds it: per tile the two MMAs are 1024 tensor cycles, the 16384
// exponentials 1024 cycles of the 16-wide unit, and shared memory carries 160
// KB (the decoded tiles written and read, Q read): 1280 cycles.  A softmax
// warp issues an instruction every 6 to 8 cycles (dependent arithmetic,
// MUFU and shared loads), so it takes 16 of them, and two tiles at once, to
// fill the issue slots: with 8 warps, whether two to a tile or on alternate
// tiles, a tile took over 6500 cycles.
// Trees of 64 tokens over up to 8192 positions, 64 query and 8 key heads of
// 128 (8 sequences): 161 us, 460 TFLOP/s (28 % of the dense rate).  Of that 118
// us go with the tiles (softmax alone 77, MMAs and barriers alone 65, decode
// hidden), 43 with start, changes of piece, partial results and their merge.
// W sits in TMEM over S, and codes do not pass through shared memory on their
// way to f16, because shared memory has no room for either in time.
// Only warps 25-27 walk sequences, heads and pages; the others read tile
// descriptors.  That is for the instruction cache, which the roles' loops
// share: with a walk inlined into each role the warps waited for instructions
// five times as long as they issued.
// The accumulator is rescaled only when a row's maximum has grown by more
// than 2^8 since its reference was taken: weights stay below 2^15, and sums
// and accumulator keep the same reference, so the result is unchanged.
// References are whole numbers: the factors are powers of two, and the f16
// weights that a tile already has take them without a second rounding (but
// for those that leave f16's normal range: 2^-32 of the largest, as above).
#pragma once
#include "attend_common.cuh"
#include "f32x2.cuh"

namespace qg {

constexpr int kTileRows = 128;
constexpr int kTilePos = 128;       // positions per tile = unit of work
constexpr int kTileThreads = 896;
constexpr int kTileStages = 6;     // descriptors and scales ahead

template <int D>
struct TileSmem {
  static constexpr int kOperand = kTilePos * D * 2;    // f16 tile of K or V
  static constexpr int kScales = 3 * kTilePos * 4;     // key scale, log2 vs, 1 / vs
  static constexpr int kTotal = 1024 + 5 * kOperand + kTileStages * kScales;  // K, V twice, Q
};
// The spin of a wait, out of line: the instruction cache holds one copy.
__device__ __noinline__ bool tile_spin(uint64_t* bar, uint32_t parity, unsigned int* err, unsigned long long limit) {
  return mbar_wait(bar, parity, err, limit);
}

// What a tile is; written by warps 25-27.
struct TileDesc {
  int run[kTilePos / 16];  // cache row of the 1st of each 16 positions
  int count;               // positions of the sequence from the tile's first on (may pass 128)
  int before;              // those before the drafted tokens (may be negative)
  int item;                // its item's first unit
  int index;               // of its piece
  int last, next_last;     // it ends the piece; the next tile does
  int whole;               // the piece is the whole item
  int row0, rows;          // first row, rows of the sequence
  int tok0, head, slot;    // slot: partial result, when not whole
};
// TMEM columns
constexpr int kTmemS = 0;        // a score tile of 128 per group; its weights over the first 64
constexpr int kTmemO = 256;      // 128 (D used) per group
constexpr int kTmemCols = 512;
__host__ __device__ constexpr uint32_t idesc_f16(int n, bool b_mn_major) {
  return (1u << 4)                            // D = f32; A, B = f16
         | (b_mn_major ? 1u << 16 : 0u) | ((uint32_t)(n >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}
// D[tmem] (+)= A[smem] . B[smem]
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
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
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ uint64_t lds_u64(uint32_t a) {
  uint64_t v;
  asm volatile("ld.shared.u64 %0, [%1];" : "=l"(v) : "r"(a));
  return v;
}
// Fragments of 16 lanes: of each 8 columns (256 bits) a thread has two of row
// lane / 4 and two of row lane / 4 + 8; of each 128 bits one word of either.
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]) : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_16x256b(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_16x256b(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_ld_16x128b(uint32_t taddr, uint32_t (&r)[2]) {
  asm volatile("tcgen05.ld.sync.aligned.16x128b.x1.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(taddr));
}
__device__ __forceinline__ void tmem_st_16x128b(uint32_t taddr, const uint32_t (&r)[2]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x1.b32 [%2], {%0,%1};" ::"r"(r[0]), "r"(r[1]), "r"(taddr) : "memory");
}
__device__ __forceinline__ void tmem_st_16x128b(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.16x128b.x4.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(taddr) : "memory");
}

template <int D, bool INT8>
__global__ void __launch_bounds__(kTileThreads, 1) qg_attend_tile_kernel(const uint8_t* k_codes, const uint8_t* v_codes,
                                                                          const AttendParams p) {
  using S = TileSmem<D>;
  extern __shared__ uint8_t smem_raw[];
  __shared__ Sched sched;
  __shared__ TileDesc descs[kTileStages];
  // full: the operand tile is decoded / the scores, weights, queries are
  // there.  s_full also frees K's buffer, o_done V's and the weights'.  A wait
  // names a phase by its parity, so its waiter must be sure of the phase
  // before (it has waited for it, or for something that followed it), and the
  // phase after must need what it does after the wait.
  __shared__ __align__(8) uint64_t k_full[2], v_full[2], s_full[2], w_full[2], o_done[2], o_free, q_full, idle,
      d_full[kTileStages], d_free[kTileStages];
  // a group's maxima and sums when the other ends the piece, per warp of 16
  // rows (two turns each)
  __shared__ __align__(8) uint64_t l_full[2][2][8];
  __shared__ float l_turn[2][2][kTileRows], m_turn[2][2][kTileRows];
  __shared__ uint32_t seen[16][16][4];  // a softmax warp's rows: which of a tile's positions they see
  __shared__ float q_down[16][16];      // and the inverse of their queries' power
  __shared__ uint32_t tmem_ptr;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t base = (smem_u32(smem_raw) + 1023) & ~1023u;
  const uint32_t k_tile = base, v_tile = base + 2 * S::kOperand, q_tile = base + 4 * S::kOperand,
                 scales = base + 5 * S::kOperand;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&k_full[i], 8);
      mbar_init(&v_full[i], 8);
      mbar_init(&s_full[i], 1);
      mbar_init(&w_full[i], 8);
      mbar_init(&o_done[i], 1);
      for (int r = 0; r < 8; ++r) {
        mbar_init(&l_full[i][0][r], 1);
        mbar_init(&l_full[i][1][r], 1);
      }
    }
    mbar_init(&o_free, 8);
    mbar_init(&q_full, 8);
    mbar_init(&idle, 1);
    for (int i = 0; i < kTileStages; ++i) {
      mbar_init(&d_full[i], 1);
      mbar_init(&d_free[i], 17);  // 8 softmax and 8 decode warps, the MMA warp
    }
    fence_barrier_init();
  }
  if (warp == 24) {
    tmem_alloc(&tmem_ptr, kTmemCols);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  griddep_wait();
  tc_fence_before();
  const Share share = plan_units(p, kTileRows, kTilePos, sched);  // also orders the barriers' set-up
  tc_fence_after();
  const uint32_t tmem = tmem_ptr;
  const bool works = (int)blockIdx.x < share.ctas && share.total > 0;
  const int u0 = works ? share.begin(blockIdx.x) : 0, u1 = works ? share.begin(blockIdx.x + 1) : 0;
  const int tiles = u1 - u0;
  bool ok = true;
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (ok && !mbar_test_wait(bar, parity)) ok = tile_spin(bar, parity, p.err, p.wait_ns);
    return ok;
  };

  if (warp < 16) {
    // ------------------------------------------------------------- softmax --
    // Row i of a thread (i < 2) is row rw + 8 i + lane / 4; its positions are
    // 8 k + 2 (lane % 4) and the next, k < 16.
    const int group = warp >> 3, part16 = warp & 7, rw = (warp & 3) * 32 + ((warp >> 2) & 1) * 16;
    const int g = lane >> 2, t = lane & 3;
    const uint32_t s_at = tmem + ((uint32_t)rw << 16) + kTmemS + group * 128;
    const uint32_t o_at = tmem + ((uint32_t)rw << 16) + kTmemO + group * 128;
    float m[2], power[2];
    uint64_t l2[2];
    int tok[2];
    int item = -1, made = 0, taken = 0;
    bool live = false;
#pragma unroll 1
    for (int j = group; j < tiles; j += 2) {
      const int st = j % kTileStages;
      wait(&d_full[st], (j / kTileStages) & 1);
      if (!__all_sync(0xffffffffu, ok)) break;
      const TileDesc& x = descs[st];
      const bool opens = x.item != item;  // this group's first tile of the piece
      if (opens) {
        // its queries, f16, each row's largest magnitude brought to
        // [2^14, 2^15).  The group of the piece's first tile stores them; the
        // other needs the powers alone.  Lane l knows row rw + l % 16's place;
        // the lanes of a load share rows of D / 8 chunks.
        item = x.item;
        live = x.row0 + rw < x.rows;
        const int r = x.row0 + rw + (lane & 15);
        const int mine = r < x.rows ? r / p.group : -1;
        const long long place =
            (long long)(x.tok0 + max(mine, 0)) * p.ldq + (x.head * p.group + (mine < 0 ? 0 : r - mine * p.group)) * D;
        // the last piece's scores are done with its queries
        if (x.index == 0 && j > 0) wait(&s_full[(j - 1) & 1], ((j - 1) >> 1) & 1);
        const bool store = x.index == 0 && __all_sync(0xffffffffu, ok);
        constexpr int LR = D / 8, RPL = 32 / LR;
        const int chunk = lane % LR;
#pragma unroll 1
        for (int b = lane / LR; b < 16; b += 4 * RPL) {
          uint4 v[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const long long at = __shfl_sync(0xffffffffu, place, b + i * RPL);
            v[i] = make_uint4(0u, 0u, 0u, 0u);
            if (__shfl_sync(0xffffffffu, mine, b + i * RPL) >= 0)
              v[i] = fresh(reinterpret_cast<const uint4*>(p.q + at) + chunk);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
            // bf16 magnitudes are ordered like their bits, two to a word
            uint32_t top = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
#pragma unroll
            for (int d = LR / 2; d > 0; d >>= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, d));
            float up, down;
            row_power(__uint_as_float(max(top << 16, top & 0xffff0000u)), up, down);
            if (chunk == 0) q_down[warp][b + i * RPL] = down;
            if (store) {
              uint32_t f[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __half2 y =
                    __floats2half2_rn(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xffff0000u) * up);
                f[e] = *reinterpret_cast<const uint32_t*>(&y);
              }
              const int row = rw + b + i * RPL;
              asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                               q_tile + (chunk >> 3) * (kTileRows * 128) + row * 128 + (((chunk ^ row) & 7) << 4)),
                           "r"(f[0]), "r"(f[1]), "r"(f[2]), "r"(f[3])
                           : "memory");
            }
          }
        }
        if (x.index == 0) fence_proxy_async_smem();
        __syncwarp();
        if (x.index == 0 && lane == 0) mbar_arrive(&q_full);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          power[i] = q_down[warp][8 * i + g] * p.scale_log2;
          tok[i] = __shfl_sync(0xffffffffu, mine, 8 * i + g);
          m[i] = kNegInf;
          l2[i] = 0;
        }
      }
      const uint32_t sc = scales + st * S::kScales + t * 8;
      const bool part_seen = x.before < kTilePos || x.count < kTilePos;
      if (part_seen && live) {
        // while the scores are on their way
        unsigned long long drafted[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) drafted[i] = drafted_bits(p, x.tok0, tok[i], x.before - t * 32);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          seen[warp][8 * i + g][t] = (uint32_t)seen_bits(p, tok[i], x.count - t * 32, x.before - t * 32, drafted[i]);
        __syncwarp();
      }
      // the scores of this tile followed this group's last product (the MMA
      // thread waits for it): the accumulator may be read and scaled
      wait(&s_full[group], (j >> 1) & 1);
      if (live && __all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        // 32 positions at a time
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          const uint32_t at = sc + c * 128;
          uint32_t sv[16];
          tmem_ld_16x256b(s_at + 32 * c, sv);
          tmem_ld_wait();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t ks = lds_u64(at + k * 32), vs = lds_u64(at + kTilePos * 4 + k * 32);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              uint32_t& a = sv[4 * k + 2 * i];
              uint32_t& b = sv[4 * k + 2 * i + 1];
              const uint64_t raw = pack_f32x2(__uint_as_float(a), __uint_as_float(b));
              unpack_u32x2(fma_f32x2(mul_f32x2(raw, pack_f32x2(power[i], power[i])), ks, vs), a, b);
            }
          }
          if (part_seen) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t bits = seen[warp][8 * i + g][c] >> (2 * t);
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                  if (!((bits >> (k * 8 + e)) & 1)) sv[4 * k + 2 * i + e] = __float_as_uint(kNegInf);
            }
            __syncwarp();
          }
          // whether a score passes its row's reference by more than it may:
          // each lane asks for its own, the row's maximum is formed only then
          float top[2][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int e = 0; e < 2; ++e)
              top[i][e] = fmaxf(__uint_as_float(sv[2 * i + e]), __uint_as_float(sv[4 + 2 * i + e]));
#pragma unroll
            for (int k = 2; k < 4; ++k)
#pragma unroll
              for (int e = 0; e < 2; ++e) top[i][e] = fmaxf(top[i][e], __uint_as_float(sv[4 * k + 2 * i + e]));
            top[i][0] = fmaxf(top[i][0], top[i][1]);
          }
          // m = -inf (nothing seen yet): anything seen passes it
          const bool grown = top[0][0] > m[0] + kRescaleAt || top[1][0] > m[1] + kRescaleAt;
          if (__any_sync(0xffffffffu, grown)) {
            // sums, accumulator and the tile's first weights follow the new reference
            float f[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float now = top[i][0];
              now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 1));
              now = fmaxf(now, __shfl_xor_sync(0xffffffffu, now, 2));
              const bool up = now > m[i] + kRescaleAt;
              now = ceilf(now);  // references are whole, factors powers of two
              f[i] = up ? ex2(m[i] - now) : 1.f;  // m = -inf: 0
              if (up) m[i] = now;
              l2[i] = mul_f32x2(l2[i], pack_f32x2(f[i], f[i]));
            }
            // what this warp stored before (the tile's earlier weights, and the
            // accumulator if the reference moved in them) is read back now
            tmem_st_wait();
            if (!opens) {
#pragma unroll 1
              for (int d = 0; d < D; d += 16) {
                uint32_t o[8];
                tmem_ld_16x256b(o_at + d, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * ((e & 2) ? f[1] : f[0]));
                tmem_st_16x256b(o_at + d, o);
              }
            }
            if (c > 0) {
#pragma unroll 1
              for (int d = 0; d < 16 * c; d += 4) {
                uint32_t w[2];
                tmem_ld_16x128b(s_at + d, w);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
                  const __half2 y = __floats2half2_rn(v.x * f[i], v.y * f[i]);
                  w[i] = *reinterpret_cast<const uint32_t*>(&y);
                }
                tmem_st_16x128b(s_at + d, w);
              }
            }
          }
          // the weights go over the scores, 16 columns for 32: what they cover is read
          const float ref[2] = {m[0] == kNegInf ? 0.f : kWeightUp - m[0], m[1] == kNegInf ? 0.f : kWeightUp - m[1]};
          uint32_t w[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint64_t iv = lds_u64(at + 2 * kTilePos * 4 + k * 32);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              float u, v;
              unpack_f32x2(add_f32x2(pack_f32x2(__uint_as_float(sv[4 * k + 2 * i]), __uint_as_float(sv[4 * k + 2 * i + 1])),
                                     pack_f32x2(ref[i], ref[i])),
                           u, v);
              u = ex2(u);
              v = ex2(v);
              l2[i] = fma_f32x2(pack_f32x2(u, v), iv, l2[i]);
              const __half2 y = __floats2half2_rn(u, v);
              w[2 * k + i] = *reinterpret_cast<const uint32_t*>(&y);
            }
          }
          tmem_st_16x128b(s_at + 16 * c, w);
        }
        tmem_st_wait();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&w_full[group]);

      if (x.last || x.next_last) {
        float l[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          float a, b;
          unpack_f32x2(l2[i], a, b);
          a += b;
          a += __shfl_xor_sync(0xffffffffu, a, 1);
          a += __shfl_xor_sync(0xffffffffu, a, 2);
          l[i] = a;
          if (a != a) m[i] = 0.f;  // a NaN row keeps its place in the merges
        }
        if (x.next_last) {
          // the other group ends the piece
          const int turn = made & 1;
          if (t == 0) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              l_turn[group][turn][rw + 8 * i + g] = l[i];
              m_turn[group][turn][rw + 8 * i + g] = m[i];
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&l_full[group][turn][part16]);
          ++made;
        } else {
          // o = (own + other's) / l, each brought to the larger reference
          const bool both = x.index > 0;
          float f[2] = {1.f, 1.f}, of[2] = {0.f, 0.f};
          if (both) {
            const int turn = taken & 1;
            wait(&l_full[group ^ 1][turn][part16], (taken >> 1) & 1);
            ++taken;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const float om = m_turn[group ^ 1][turn][rw + 8 * i + g], ol = l_turn[group ^ 1][turn][rw + 8 * i + g];
              const float now = fmaxf(m[i], om);
              f[i] = m[i] == kNegInf ? 0.f : ex2(m[i] - now);
              of[i] = om == kNegInf ? 0.f : ex2(om - now);
              m[i] = now;
              l[i] = l[i] * f[i] + ol * of[i];
            }
            // the group's product is the last before o_free: this wait's phase
            // follows the one its scores followed
            wait(&o_done[group ^ 1], ((j - 1) >> 1) & 1);
          }
          wait(&o_done[group], (j >> 1) & 1);
          if (live && __all_sync(0xffffffffu, ok)) {
            tc_fence_after();
            const bool whole = x.whole;
            float* part = p.partial + (size_t)x.slot * kTileRows * (D + 2);
            size_t at[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int row = rw + 8 * i + g, r = x.row0 + row;
              const size_t tk = x.tok0 + max(tok[i], 0);
              const int h = tok[i] < 0 ? 0 : x.head * p.group + r - tok[i] * p.group;
              at[i] = tk * p.ldo + h * D + 2 * t;
              if (t == 0 && tok[i] >= 0) {
                if (!whole) {
                  part[kTileRows * D + row] = m[i];
                  part[kTileRows * D + kTileRows + row] = l[i];
                } else if (p.lse != nullptr) {
                  p.lse[tk * p.q_heads + h] = l[i] == 0.f ? kNegInf : (m[i] - kWeightUp + log2f(l[i])) * 0.6931471805599453f;
                }
              }
              if (whole) {
                // a row that saw nothing: zeros (its weights were all zero)
                const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
                f[i] *= inv;
                of[i] *= inv;
              }
            }
            // (alone, its own again with a factor of 0)
            const uint32_t other = both ? tmem + ((uint32_t)rw << 16) + kTmemO + (group ^ 1) * 128 : o_at;
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t o[8], q[8];
              tmem_ld_16x256b(o_at + c, o);
              tmem_ld_16x256b(other + c, q);
              tmem_ld_wait();
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float y[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                  y[e] = fmaf(__uint_as_float(q[4 * k + e]), of[e >> 1], __uint_as_float(o[4 * k + e]) * f[e >> 1]);
                if (!whole) {
                  // as the fragments lie: whole lines (the merge knows)
                  reinterpret_cast<float4*>(part)[((rw >> 4) * (D / 8) + c / 8 + k) * 32 + lane] =
                      make_float4(y[0], y[1], y[2], y[3]);
                } else {
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    if (tok[i] >= 0)
                      *reinterpret_cast<__nv_bfloat162*>(p.out + at[i] + c + 8 * k) =
                          __floats2bfloat162_rn(y[2 * i], y[2 * i + 1]);
                }
              }
              __syncwarp();
            }
            tc_fence_before();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&o_free);
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&d_free[st]);
    }
  } else if (warp < 24) {
    // -------------------------------------------------------------- decode --
    // K of tile j + 1 before V of tile j; a warp has 16 positions.  A lane
    // holds 16 codes of a row: the 8 lanes of a store phase are 2 rows x 4 of
    // the 16-byte chunks of one 64-channel block, which the swizzle spreads
    // over all banks.
    constexpr int RPI = D == 128 ? 4 : 8;     // rows per warp instruction
    constexpr int N = 16 / RPI;               // instructions per warp and tile
    const int c = D == 128 ? (lane & 3) + ((lane >> 4) << 2) : lane & 3;
    const int r0 = D == 128 ? (lane >> 2) & 3 : lane >> 2;   // of the warp's positions
    const int w0 = (warp - 16) * 16;
    auto load = [&](int j, const uint8_t* codes, uint4 (&buf)[N], bool done) {
      const int st = j % kTileStages;
      wait(&d_full[st], (j / kTileStages) & 1);
      if (!__all_sync(0xffffffffu, ok)) return;
      const int count = descs[st].count - w0 - r0;
      const uint4* src = reinterpret_cast<const uint4*>(codes + (size_t)(descs[st].run[warp - 16] + r0) * D) + c;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        buf[i] = make_uint4(0u, 0u, 0u, 0u);
        if (i * RPI < count) buf[i] = fresh(src + i * RPI * (D / 16));
      }
      if (done) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_free[st]);
      }
    };
    // chunk (c % 4) * 2 + e of row r sits at that ^ (r % 8); rows RPI apart
    // differ by RPI * 128 bytes and, for RPI = 4, in bit 2 of r % 8
    const uint32_t line = (D == 128 ? (uint32_t)(c >> 2) * (kTilePos * 128) : 0u) + (w0 + r0) * 128;
    const uint32_t chunk0 = (((c & 3) * 2) ^ (r0 & 7)) << 4, chunk1 = (((c & 3) * 2 + 1) ^ (r0 & 7)) << 4;
    auto store = [&](uint32_t tile, const uint4 (&buf)[N]) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint32_t flip = D == 128 && (i & 1) ? 64u : 0u;
        const uint32_t w[4] = {buf[i].x, buf[i].y, buf[i].z, buf[i].w};
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          uint32_t f[4];
          decode4<INT8>(w[2 * e], f[0], f[1]);
          decode4<INT8>(w[2 * e + 1], f[2], f[3]);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(tile + line + ((e ? chunk1 : chunk0) ^ flip) +
                                                                        i * RPI * 128),
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
        if (j >= 2) wait(&o_done[j & 1], ((j - 2) >> 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        store(v_tile + (j & 1) * S::kOperand, vb);
        if (lane == 0) mbar_arrive(&v_full[j & 1]);
      }
      if (i < tiles) load(i, v_codes, vb, true);
    }
  } else {
    if (warp == 24) {
      // --------------------------------------------------------------- MMA --
      if (lane == 0) {
        const uint64_t qd = sdesc_sw128(q_tile), kd = sdesc_sw128(k_tile), vd = sdesc_mn_sw128(v_tile, kTilePos * 128);
        // Scores and products each in tile order, whichever can go first: the
        // scores of tile n wait for the product of n - 2 (its weights are in
        // their columns), which other work can cover.
        int pieces = 0, opened = 0;  // whose scores, whose products have begun
        int n = 0, j = 0;            // next tile for scores, for the product
        int n_index = -1;            // of tile n in its piece, -1: not looked up
        uint32_t index = 0;          // bits 2 s, 2 s + 1: min(index, 2) of the tile in score columns s
        unsigned long long since = 0;
        int idle_turns = 0;
        while (j < tiles) {
          bool moved = false;
          if (j < n) {
            const int s = j & 1, at = (index >> (2 * s)) & 3;
            if (mbar_test_wait(&w_full[s], (j >> 1) & 1) && mbar_test_wait(&v_full[s], (j >> 1) & 1) &&
                // a piece's first product: the last piece is out
                (at != 0 || opened == 0 || mbar_test_wait(&o_free, (opened - 1) & 1))) {
              if (at == 0) ++opened;
              tc_fence_after();
              const uint64_t vt = vd + ((s * S::kOperand) >> 4);
#pragma unroll
              for (int k = 0; k < kTilePos / 16; ++k)
                mma_f16_ts(tmem + kTmemO + s * 128, tmem + kTmemS + s * 128 + 8 * k, vt + ((k * 2048) >> 4),
                           idesc_f16(D, true), at > 1 || k > 0);
              mma_commit(&o_done[s]);
              ++j;
              moved = true;
            }
          }
          if (n < tiles && n < j + 2) {
            const int s = n & 1, st = n % kTileStages;
            if (n_index < 0 && mbar_test_wait(&d_full[st], (n / kTileStages) & 1)) {
              n_index = descs[st].index;
              mbar_arrive(&d_free[st]);
            }
            if (n_index >= 0 && mbar_test_wait(&k_full[s], (n >> 1) & 1) &&
                (n < 2 || mbar_test_wait(&o_done[s], ((n - 2) >> 1) & 1)) &&
                (n_index > 0 || mbar_test_wait(&q_full, pieces & 1))) {
              if (n_index == 0) ++pieces;
              tc_fence_after();
              const uint64_t kt = kd + ((s * S::kOperand) >> 4);
#pragma unroll
              for (int k = 0; k < D / 16; ++k) {
                const uint32_t at = ((k >> 2) * (kTilePos * 128) + (k & 3) * 32) >> 4;
                mma_f16_ss(tmem + kTmemS + s * 128, qd + at, kt + at, idesc_f16(kTilePos, false), k > 0);
              }
              mma_commit(&s_full[s]);
              index = (index & ~(3u << (2 * s))) | ((uint32_t)min(n_index, 2) << (2 * s));
              n_index = -1;
              ++n;
              moved = true;
            }
          }
          if (moved) {
            idle_turns = 0;
          } else if ((++idle_turns & 63) == 0) {
            // bounded, like every wait
            const unsigned long long now = globaltimer();
            if (idle_turns == 64) since = now;
            else if (now - since > p.wait_ns) {
              atomicOr(p.err, kErrWaitTimeout);
              break;
            }
          }
        }
        // MMAs still in flight (a wait ran out) end before TMEM is given up
        mma_commit(&idle);
        (void)mbar_wait(&idle, 0, p.err, p.wait_ns);
      }
      __syncwarp();
    } else {
      // --------------------------------------------------- the tiles ahead --
      // Warp 25 + i takes tiles i, i + 3, ...: the chain from page table to
      // scales is longer than a tile's turn.  Lane i has positions 4 i .. 4 i
      // + 3: within one run of 16, whose row its first lane hands on.
      Piece x = {};
      int item = 0, done = 0;  // units of the item at hand: [item, done)
#pragma unroll 1
      for (int j = warp - 25; j < tiles; j += 3) {
        const int u = u0 + j;
        if (u >= done) {
          x = find_piece(p, sched, kTileRows, u, u1);
          item = u - x.unit0;
          done = item + x.units;
        }
        const int tile = u - item, count = sched.len[x.seq] - tile * kTilePos;
        int row = 0;
        float4 ks = make_float4(1.f, 1.f, 1.f, 1.f), vs = ks;
        if (lane * 4 < count) {
          const int pos = tile * kTilePos + lane * 4;
          const int page = min(max(fresh(p.table + (size_t)x.seq * p.ldp + (pos >> p.page_shift)), 0), p.pages - 1);
          row = (page * p.kv_heads + x.head << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
          ks = fresh(reinterpret_cast<const float4*>(p.k_scale + row));
          vs = fresh(reinterpret_cast<const float4*>(p.v_scale + row));
        }
        const int st = j % kTileStages;
        if (j >= kTileStages) wait(&d_free[st], (j / kTileStages - 1) & 1);
        if (!__all_sync(0xffffffffu, ok)) break;
        TileDesc& d = descs[st];
        if ((lane & 3) == 0) d.run[lane >> 2] = row;
        if (lane == 0) {
          d.count = count;
          d.before = count - sched.n[x.seq];
          d.item = item;
          d.index = u - max(item, u0);
          d.last = u + 1 == u1 || u + 1 == done;
          d.next_last = !d.last && (u + 2 == u1 || u + 2 == done);
          d.whole = item >= u0 && done <= u1;
          d.row0 = x.row0;
          d.rows = min(sched.n[x.seq], p.max_q) * p.group;
          d.tok0 = sched.tok0[x.seq];
          d.head = x.head;
          d.slot = 2 * blockIdx.x + (item <= u0 ? 0 : 1);  // the share's first piece or a later one
        }
        const uint32_t at = scales + st * S::kScales + lane * 16;
        const float v4[4] = {vs.x, vs.y, vs.z, vs.w};
        float a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) value_scale(v4[i], a[i], b[i]);
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(ks.x), "f"(ks.y), "f"(ks.z), "f"(ks.w)
                     : "memory");
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + kTilePos * 4), "f"(a[0]), "f"(a[1]),
                     "f"(a[2]), "f"(a[3])
                     : "memory");
        asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + 2 * kTilePos * 4), "f"(b[0]), "f"(b[1]),
                     "f"(b[2]), "f"(b[3])
                     : "memory");
        __syncwarp();
        if (lane == 0) mbar_arrive(&d_full[st]);
      }
      if (warp == 25 && lane == 0) p.records[blockIdx.x] = merge_record(p, sched, share, kTileRows);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 24) tmem_dealloc(tmem, kTmemCols);
}

}  // namespace qg
