// internal.h — declarations shared by the library's translation units.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace qg {

struct GemmParams;

}  // namespace qg
#include "../../include/qgemm.h"
namespace qg {

qg_status check_run_args(qg_format f, const qg_operand* A, const qg_operand* W, int M, int N, int K,
                         const qg_config* cfg, void* workspace, size_t ws_bytes, void* Y, int ldy,
                         int out_kind);

constexpr int kNvfp4AmaxMaxCtas = 296;   // partial-amax slots in the NVFP4 quant workspace

// Configuration feasibility (the checks of qgemm_run), the shared memory a
// launch takes, the SM count of the current device (148 without one), the
// fixed-rule default configuration (api.cu).
qg_status config_check(qg_format f, int M, int N, int K, const qg_config* c);
size_t config_smem(qg_format f, int M, int K, const qg_config* c);
int device_sm_count();
qg_status rule_default_config(qg_format f, int M, int N, int K, qg_config* out);
// The candidate grid the scorer ranks and the tuner times (scorer.cu), before
// feasibility checks.
void candidate_grid(qg_format f, int M, int N, int K, qg_config* out, int max_out, int* n_out);

cudaError_t launch_quant_rows(bool int8, const void* X, int R, int K, int ldx, void* q,
                              float* scale, cudaStream_t st, bool pdl);
cudaError_t launch_quant_act_groups(const void* X, int M, int K, int ldx, void* q, float* scale,
                                    cudaStream_t st, bool pdl);
cudaError_t launch_quant_weight_blocks(const void* W, int N, int K, void* q, float* scale,
                                       cudaStream_t st, bool pdl);
int nvfp4_amax_ctas(int R, int K);
cudaError_t launch_quant_nvfp4(const void* X, int R, int K, int ldx, const float* static_amax,
                               void* q, void* sf, float* gscale, float* partial,
                               cudaStream_t st, bool pdl, const int* offsets = nullptr,
                               int experts = 0);

// The launch state of the current device (api.cu): SM count, device error
// word, programmatic dependent launch and the limit of in-kernel waits.
struct LaunchState {
  int sms;
  unsigned int* err;
  bool pdl;
  unsigned long long wait_ns;
};
qg_status launch_state(LaunchState* out);
// The operand of a rows x K activation has every buffer it needs (api.cu).
qg_status check_operand_out(qg_format f, int rows, int K, const qg_operand* out);
// A 2D byte tensor [rows, row_bytes], boxes of box_rows whole rows (64 or 128
// bytes) with the swizzle of that width (api.cu).
bool make_row_tmap(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows, uint32_t box_rows);

// Kernel parameters of the norm (norm.cu).
struct NormParams {
  const __nv_bfloat16 *residual, *x, *gate;
  const uint4 *post_weight, *post_bias, *pre_weight, *pre_bias;
  __nv_bfloat16 *h, *y;
  uint8_t* q;                // operand codes, NULL: none
  void* scale;
  float* global_scale;       // NVFP4
  const float* static_amax;  // NVFP4
  int M, N, ldr, ldx, ldg, ldh, ldy, sf_cols;
  int format, post_norm, pre_norm;
  float residual_scale, block_scale, eps, weight_offset, inv_n;
};
cudaError_t launch_norm(const NormParams& p, cudaStream_t st, bool pdl);

// Kernel parameters of the cache write and read (cache.cu).
struct CacheWriteParams {
  const __nv_bfloat16 *q, *k, *v;
  __nv_bfloat16* q_out;
  uint8_t *k_codes, *v_codes;
  float *k_scale, *v_scale;
  const int *slots, *positions;
  const double* frequency;
  int tokens, ldq, ldk, ldv, ldqo, q_heads, kv_heads, rope_dim, interleaved, page_shift, slots_total;
  float magnitude;
};
cudaError_t launch_cache_write(const CacheWriteParams& p, int head_dim, bool int8, cudaStream_t st, bool pdl);
struct CacheReadParams {
  const uint8_t *k_codes, *v_codes;
  const float *k_scale, *v_scale;
  __nv_bfloat16 *k, *v;
  const int* slots;
  int tokens, ldk, ldv, kv_heads, page_shift, slots_total;
};
cudaError_t launch_cache_read(const CacheReadParams& p, int head_dim, bool int8, cudaStream_t st, bool pdl);

// Kernel parameters of the attention over the cache (attend.cu).
struct MergeRecord;
struct AttendParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* out;
  float* lse;                 // NULL: not wanted
  const int *q_offsets, *kv_len, *table;
  const unsigned long long* mask;  // NULL: causal
  const float *k_scale, *v_scale;
  MergeRecord* records; // workspace: one per CTA, then the partial results
  float* partial;
  int ldq, ldo, ldp, mask_words, q_heads, kv_heads, group, batch, tokens, max_q;
  int pages, page_shift, box_rows;
  float scale_log2;           // softmax scale * log2(e)
  unsigned int* err;
  unsigned long long wait_ns;
};
constexpr int kAttendMaxBatch = 1024;
size_t attend_workspace(int head_dim, int rows_max, int sms);
// How a call's work is cut: rows of an item, positions of a unit.
struct AttendSplit {
  int tile_rows, unit;
};
AttendSplit attend_split(int rows, int head_dim);
bool attend_tiles(int rows, int head_dim);  // whether the tile kernel takes so many rows per key head
cudaError_t launch_attend(AttendParams p, void* workspace, const uint8_t* k, const uint8_t* v, const CUtensorMap* tk,
                          const CUtensorMap* tv, int rows, int head_dim, bool int8, int sms, cudaStream_t st, bool pdl);

// GEMM launchers, one per format (each in its own translation unit).
// Returns cudaErrorInvalidValue for a (swap, tile_n) pair not instantiated.
#define QG_DECLARE_GEMM_LAUNCH(NAME)                                                      \
  cudaError_t NAME(bool swap, int tile_n, const CUtensorMap& tp, const CUtensorMap& tq,    \
                   const CUtensorMap& ty,                                                  \
                   const GemmParams& prm, dim3 grid, cudaStream_t st, bool pdl);           \
  size_t NAME##_smem(int tile_n, bool swap, int stages, int nkt_max, int recv_cols,        \
                     int act_tiles);                                                       \
  bool NAME##_cluster_fits(int tile_n, bool swap, int stages, int act_tiles);              \
  cudaError_t NAME##_reduce(const GemmParams& prm, cudaStream_t st, bool pdl);             \
  cudaError_t NAME##_grouped(int tile_n, const CUtensorMap& tp, const CUtensorMap& tq,     \
                             const CUtensorMap& ty,                                        \
                             const GemmParams& prm, dim3 grid, cudaStream_t st, bool pdl); \
  cudaError_t NAME##_skinny(int tile_n, int rows, const CUtensorMap& tw, const CUtensorMap& ta, \
                            const GemmParams& prm, dim3 grid, cudaStream_t st, bool pdl);     \
  size_t NAME##_skinny_smem(int tile_n, int rows, int stages);                              \
  cudaError_t NAME##_persist(int tile_n, const CUtensorMap& tp, const CUtensorMap& tq,     \
                             const CUtensorMap& ty, const GemmParams& prm, dim3 grid,      \
                             cudaStream_t st, bool pdl);                                   \
  size_t NAME##_persist_smem(int tile_n, int stages, int nkt);                              \
  cudaError_t NAME##_pair(int tile_n, const CUtensorMap& tp, const CUtensorMap& tq,        \
                          const CUtensorMap& ty, const GemmParams& prm, dim3 grid,         \
                          cudaStream_t st, bool pdl);                                      \
  size_t NAME##_pair_smem(int tile_n, int stages, int nkt);
QG_DECLARE_GEMM_LAUNCH(launch_gemm_fp8)
QG_DECLARE_GEMM_LAUNCH(launch_gemm_int8)
QG_DECLARE_GEMM_LAUNCH(launch_gemm_block)
QG_DECLARE_GEMM_LAUNCH(launch_gemm_nvf4)
#undef QG_DECLARE_GEMM_LAUNCH

}  // namespace qg
