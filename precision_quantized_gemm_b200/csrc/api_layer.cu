// api_layer.cu — C ABI of the operators between a decoder layer's quantised
// products: the norm with a quantised output, the rotary cache write, the
// cache read and the attention over the cache.  Argument checks and launches.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "../../include/qgemm.h"
#include "internal.h"

namespace {

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
// A bf16 matrix with rows of `width` elements, `ld` apart, read 16 bytes at a time.
bool good_rows(const void* p, int ld, int width) { return p && aligned(p, 16) && ld >= width && ld % 8 == 0; }
bool good_vector(const void* p) { return aligned(p, 16); }  // NULL is one

qg_status check_cache(const qg_cache* c) {
  if (!c) return QG_ERR_INVALID_ARG;
  size_t codes, scales;
  const qg_status s = qgemm_cache_bytes(c->format, c->pages, c->page_size, c->kv_heads, c->head_dim, &codes, &scales);
  if (s != QG_OK) return s;
  if (!c->k || !c->v || !c->k_scale || !c->v_scale) return QG_ERR_INVALID_ARG;
  if (!aligned(c->k, 16) || !aligned(c->v, 16) || !aligned(c->k_scale, 16) || !aligned(c->v_scale, 16))
    return QG_ERR_INVALID_ARG;
  // a token's row of heads is counted in 32 bits, like the strides
  if ((long long)c->kv_heads * c->head_dim > 0x7fffffffLL) return QG_ERR_UNSUPPORTED;
  return QG_OK;
}
int shift_of(int pow2) {
  int s = 0;
  while ((1 << s) < pow2) ++s;
  return s;
}

// Rows per key head of a sequence of max_q tokens: what the workspace goes by.
long long rows_per_key_head(const qg_cache* c, const qg_attend* a) {
  return (long long)a->max_q * (a->q_heads / c->kv_heads);
}

// Units of work that the sizes of a call allow, cut for so many rows per key
// head; counted in 32 bits by the kernels.
bool units_fit(const qg_cache* c, const qg_attend* a, int rows) {
  const qg::AttendSplit split = qg::attend_split(rows, c->head_dim);
  const long long most = (long long)std::min(a->max_q, a->tokens) * (a->q_heads / c->kv_heads);
  const double tiles = (double)((most + split.tile_rows - 1) / split.tile_rows);
  const double units = (double)a->max_pages * c->page_size / split.unit + 1;
  return units * tiles * c->kv_heads * a->batch <= 0x7fffff00;
}

// Rows per key head that a call's kernel goes by: those of its mean sequence.
// Either kernel takes sequences of any number of tokens, and max_q may be far
// above most of them.  8192 positions, 64 query and 8 key heads of 128, by
// the mean and by max_q: 64 single tokens (max_q 64) 182 and 344 us, 63 and
// one of 32 240 and 404 us, 63 and one of 129 408 and 459 us.  Where the
// smaller items would be too many to count, those of max_q.
int kernel_rows(const qg_cache* c, const qg_attend* a) {
  const int mean = (int)(((long long)a->tokens + a->batch - 1) / a->batch);
  const int rows = std::min(a->max_q, mean) * (a->q_heads / c->kv_heads);
  return units_fit(c, a, rows) ? rows : (int)rows_per_key_head(c, a);
}

qg_status check_attend(const qg_cache* c, const qg_attend* a) {
  if (!a) return QG_ERR_INVALID_ARG;
  const qg_status s = check_cache(c);
  if (s != QG_OK) return s;
  if (a->batch <= 0 || a->tokens <= 0 || a->max_q <= 0 || a->q_heads <= 0 || a->max_pages <= 0)
    return QG_ERR_INVALID_ARG;
  if (a->q_heads % c->kv_heads != 0) return QG_ERR_INVALID_ARG;
  if ((long long)a->q_heads * c->head_dim > 0x7fffffffLL) return QG_ERR_INVALID_ARG;
  const int width = a->q_heads * c->head_dim;
  if (!good_rows(a->q, a->ldq, width) || !good_rows(a->out, a->ldo, width)) return QG_ERR_INVALID_ARG;
  if (!a->q_offsets || !a->kv_len || !a->page_table || !aligned(a->q_offsets, 4) || !aligned(a->kv_len, 4) ||
      !aligned(a->page_table, 4) || !aligned(a->lse, 4))
    return QG_ERR_INVALID_ARG;
  if (a->tree_mask && (!aligned(a->tree_mask, 8) || a->mask_words <= 0)) return QG_ERR_INVALID_ARG;
  if (!(a->scale > -3.0e38f && a->scale < 3.0e38f)) return QG_ERR_INVALID_ARG;
  if (a->batch > qg::kAttendMaxBatch || a->max_q > QGEMM_ATTEND_MAX_Q) return QG_ERR_UNSUPPORTED;
  // positions of a sequence are 32-bit, like the units of work
  const double positions = (double)a->max_pages * c->page_size;
  if (rows_per_key_head(c, a) > 0x7fff0000 || positions > 0x7fffff00 || !units_fit(c, a, kernel_rows(c, a)))
    return QG_ERR_UNSUPPORTED;
  return QG_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------- norm --
qg_status qgemm_norm(const qg_norm* n, int M, int N, qg_format f, qg_operand* out, const float* static_amax,
                     void* stream) {
  if (!n || M <= 0 || N <= 0 || N % 8 != 0) return QG_ERR_INVALID_ARG;
  if (n->pre_norm < QG_NORM_NONE || n->pre_norm > QG_NORM_LAYER || n->post_norm < QG_NORM_NONE ||
      n->post_norm > QG_NORM_LAYER)
    return QG_ERR_INVALID_ARG;
  if (!n->residual && !n->x) return QG_ERR_INVALID_ARG;
  if (n->residual && !good_rows(n->residual, n->ldr, N)) return QG_ERR_INVALID_ARG;
  if (n->x && !good_rows(n->x, n->ldx, N)) return QG_ERR_INVALID_ARG;
  // a gate row for every row of x (ldg >= N), or one for all (ldg = 0)
  if (n->gate && (!n->x || !aligned(n->gate, 16) || (n->ldg != 0 && (n->ldg < N || n->ldg % 8 != 0))))
    return QG_ERR_INVALID_ARG;
  if (n->post_norm && (!n->x || !n->post_weight)) return QG_ERR_INVALID_ARG;
  if (!n->post_norm && (n->post_weight || n->post_bias)) return QG_ERR_INVALID_ARG;
  if (n->pre_norm ? !n->pre_weight : (n->pre_weight || n->pre_bias)) return QG_ERR_INVALID_ARG;
  if (!good_vector(n->post_weight) || !good_vector(n->post_bias) || !good_vector(n->pre_weight) ||
      !good_vector(n->pre_bias))
    return QG_ERR_INVALID_ARG;
  if (n->h && !good_rows(n->h, n->ldh, N)) return QG_ERR_INVALID_ARG;
  if (n->y && !good_rows(n->y, n->ldy, N)) return QG_ERR_INVALID_ARG;
  if ((n->y || out) && !n->pre_norm) return QG_ERR_INVALID_ARG;
  if (!n->h && !n->y && !out) return QG_ERR_INVALID_ARG;
  if (!(n->eps >= 0.f)) return QG_ERR_INVALID_ARG;
  if (N > QGEMM_NORM_MAX_WIDTH) return QG_ERR_UNSUPPORTED;
  size_t qb = 0, sb = 0;
  qg_status s;
  if (out) {
    if ((s = qgemm_operand_bytes(f, 0, M, N, &qb, &sb)) != QG_OK) return s;
    if ((s = qg::check_operand_out(f, M, N, out)) != QG_OK) return s;
    // a row's CTA cannot know the amax of the whole tensor
    if (f == QG_NVFP4 && !static_amax) return QG_ERR_UNSUPPORTED;
    if (f == QG_NVFP4 && !aligned(static_amax, 4)) return QG_ERR_INVALID_ARG;
  }
  qg::LaunchState st;
  if ((s = qg::launch_state(&st)) != QG_OK) return s;
  qg::NormParams p = {};
  p.residual = static_cast<const __nv_bfloat16*>(n->residual);
  p.x = static_cast<const __nv_bfloat16*>(n->x);
  p.gate = static_cast<const __nv_bfloat16*>(n->gate);
  p.post_weight = static_cast<const uint4*>(n->post_weight);
  p.post_bias = static_cast<const uint4*>(n->post_bias);
  p.pre_weight = static_cast<const uint4*>(n->pre_weight);
  p.pre_bias = static_cast<const uint4*>(n->pre_bias);
  p.h = static_cast<__nv_bfloat16*>(n->h);
  p.y = static_cast<__nv_bfloat16*>(n->y);
  p.ldr = n->ldr;
  p.ldx = n->ldx;
  p.ldg = n->ldg;
  p.ldh = n->ldh;
  p.ldy = n->ldy;
  p.M = M;
  p.N = N;
  p.format = -1;
  if (out) {
    p.q = static_cast<uint8_t*>(out->q);
    p.scale = out->scale;
    p.global_scale = out->global_scale;
    p.static_amax = static_amax;
    p.format = f;
    p.sf_cols = ((N + 255) / 256) * 16;
  }
  p.post_norm = n->post_norm;
  p.pre_norm = n->pre_norm;
  p.residual_scale = n->residual_scale;
  p.block_scale = n->block_scale;
  p.eps = n->eps;
  p.weight_offset = n->weight_offset;
  p.inv_n = 1.f / (float)N;
  return qg::launch_norm(p, (cudaStream_t)stream, st.pdl) == cudaSuccess ? QG_OK : QG_ERR_CUDA;
}

// ------------------------------------------------------------------ cache --
qg_status qgemm_cache_bytes(qg_format f, int pages, int page_size, int kv_heads, int head_dim, size_t* code_bytes,
                            size_t* scale_bytes) {
  if (pages <= 0 || page_size <= 0 || kv_heads <= 0 || head_dim <= 0 || !code_bytes || !scale_bytes)
    return QG_ERR_INVALID_ARG;
  if (f < QG_FP8_DYNAMIC || f > QG_NVFP4) return QG_ERR_INVALID_ARG;
  if (f != QG_FP8_DYNAMIC && f != QG_W8A8_INT8) return QG_ERR_UNSUPPORTED;
  if (head_dim != 64 && head_dim != 128) return QG_ERR_UNSUPPORTED;
  if (page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0) return QG_ERR_UNSUPPORTED;
  // rows (page, head, place) and slots (page, place) are 32-bit
  const long long rows = (long long)pages * page_size;
  if (rows > 0x7fffffffLL / kv_heads) return QG_ERR_UNSUPPORTED;
  *code_bytes = (size_t)rows * kv_heads * head_dim;
  *scale_bytes = (size_t)rows * kv_heads * 4;
  return QG_OK;
}

qg_status qgemm_cache_write(const qg_cache* c, const qg_cache_write* w, int tokens, void* stream) {
  qg_status s = check_cache(c);
  if (s != QG_OK) return s;
  if (!w || tokens <= 0 || !w->slots || !aligned(w->slots, 4)) return QG_ERR_INVALID_ARG;
  const int width = c->kv_heads * c->head_dim;
  if (!good_rows(w->k, w->ldk, width) || !good_rows(w->v, w->ldv, width)) return QG_ERR_INVALID_ARG;
  if (w->q_heads < 0 || (w->q_heads > 0) != (w->q != nullptr) || (w->q != nullptr) != (w->q_out != nullptr))
    return QG_ERR_INVALID_ARG;
  if ((long long)w->q_heads * c->head_dim > 0x7fffffffLL) return QG_ERR_INVALID_ARG;
  if (w->q && (!good_rows(w->q, w->ldq, w->q_heads * c->head_dim) ||
               !good_rows(w->q_out, w->ldqo, w->q_heads * c->head_dim)))
    return QG_ERR_INVALID_ARG;
  if (w->rope_dim < 0 || w->rope_dim > c->head_dim || w->rope_dim % 16 != 0) return QG_ERR_INVALID_ARG;
  if (w->rope_dim && (!w->positions || !w->frequency || !aligned(w->positions, 4) || !aligned(w->frequency, 8)))
    return QG_ERR_INVALID_ARG;
  qg::LaunchState st;
  if ((s = qg::launch_state(&st)) != QG_OK) return s;
  qg::CacheWriteParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(w->q);
  p.k = static_cast<const __nv_bfloat16*>(w->k);
  p.v = static_cast<const __nv_bfloat16*>(w->v);
  p.q_out = static_cast<__nv_bfloat16*>(w->q_out);
  p.k_codes = static_cast<uint8_t*>(c->k);
  p.v_codes = static_cast<uint8_t*>(c->v);
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.slots = w->slots;
  p.positions = w->positions;
  p.frequency = w->frequency;
  p.tokens = tokens;
  p.ldq = w->ldq;
  p.ldk = w->ldk;
  p.ldv = w->ldv;
  p.ldqo = w->ldqo;
  p.q_heads = w->q_heads;
  p.kv_heads = c->kv_heads;
  p.rope_dim = w->rope_dim;
  p.interleaved = w->interleaved != 0;
  p.page_shift = shift_of(c->page_size);
  p.slots_total = c->pages << p.page_shift;
  p.magnitude = w->magnitude;
  return qg::launch_cache_write(p, c->head_dim, c->format == QG_W8A8_INT8, (cudaStream_t)stream, st.pdl) ==
                 cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

qg_status qgemm_cache_read(const qg_cache* c, const int32_t* slots, int tokens, void* k, int ldk, void* v, int ldv,
                           void* stream) {
  qg_status s = check_cache(c);
  if (s != QG_OK) return s;
  const int width = c->kv_heads * c->head_dim;
  if (tokens <= 0 || !slots || !aligned(slots, 4) || !good_rows(k, ldk, width) || !good_rows(v, ldv, width))
    return QG_ERR_INVALID_ARG;
  qg::LaunchState st;
  if ((s = qg::launch_state(&st)) != QG_OK) return s;
  qg::CacheReadParams p = {};
  p.k_codes = static_cast<const uint8_t*>(c->k);
  p.v_codes = static_cast<const uint8_t*>(c->v);
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.k = static_cast<__nv_bfloat16*>(k);
  p.v = static_cast<__nv_bfloat16*>(v);
  p.slots = slots;
  p.tokens = tokens;
  p.ldk = ldk;
  p.ldv = ldv;
  p.kv_heads = c->kv_heads;
  p.page_shift = shift_of(c->page_size);
  p.slots_total = c->pages << p.page_shift;
  return qg::launch_cache_read(p, c->head_dim, c->format == QG_W8A8_INT8, (cudaStream_t)stream, st.pdl) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

// -------------------------------------------------------------- attention --
size_t qgemm_attend_workspace_size(const qg_cache* c, const qg_attend* a) {
  if (!c || !a || c->head_dim <= 0 || c->kv_heads <= 0 || a->q_heads <= 0 || a->max_q <= 0) return 0;
  const long long rows = rows_per_key_head(c, a);
  return rows > 0x7fff0000 ? 0 : qg::attend_workspace(c->head_dim, (int)rows, qg::device_sm_count());
}

qg_status qgemm_attend(const qg_cache* c, const qg_attend* a, void* workspace, size_t ws_bytes, void* stream) {
  qg_status s = check_attend(c, a);
  if (s != QG_OK) return s;
  qg::LaunchState st;
  if ((s = qg::launch_state(&st)) != QG_OK) return s;
  const int group = a->q_heads / c->kv_heads;
  if (!workspace || !aligned(workspace, 16) || ws_bytes < qg::attend_workspace(c->head_dim, a->max_q * group, st.sms))
    return QG_ERR_WORKSPACE;
  qg::AttendParams p = {};
  p.q = static_cast<const __nv_bfloat16*>(a->q);
  p.out = static_cast<__nv_bfloat16*>(a->out);
  p.lse = a->lse;
  p.q_offsets = a->q_offsets;
  p.kv_len = a->kv_len;
  p.table = a->page_table;
  p.mask = reinterpret_cast<const unsigned long long*>(a->tree_mask);
  p.k_scale = c->k_scale;
  p.v_scale = c->v_scale;
  p.ldq = a->ldq;
  p.ldo = a->ldo;
  p.ldp = a->max_pages;
  p.mask_words = a->mask_words;
  p.q_heads = a->q_heads;
  p.kv_heads = c->kv_heads;
  p.group = group;
  p.batch = a->batch;
  p.tokens = a->tokens;
  p.max_q = a->max_q;
  p.pages = c->pages;
  p.page_shift = shift_of(c->page_size);
  p.box_rows = std::min(c->page_size, 32);
  p.scale_log2 = a->scale * 1.4426950408889634f;
  p.err = st.err;
  p.wait_ns = st.wait_ns;
  CUtensorMap tk, tv;
  const int rows = kernel_rows(c, a);
  if (!qg::attend_tiles(rows, c->head_dim)) {
    const uint64_t all = (uint64_t)c->pages * c->kv_heads * c->page_size;
    if (!qg::make_row_tmap(&tk, c->k, c->head_dim, all, p.box_rows)) return QG_ERR_CUDA;
    if (!qg::make_row_tmap(&tv, c->v, c->head_dim, all, p.box_rows)) return QG_ERR_CUDA;
  }
  return qg::launch_attend(p, workspace, static_cast<const uint8_t*>(c->k), static_cast<const uint8_t*>(c->v), &tk, &tv,
                           rows, c->head_dim, c->format == QG_W8A8_INT8, st.sms, (cudaStream_t)stream,
                           st.pdl) == cudaSuccess
             ? QG_OK
             : QG_ERR_CUDA;
}

}  // extern "C"
