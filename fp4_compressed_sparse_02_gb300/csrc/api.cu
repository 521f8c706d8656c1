// Host-side C ABI: argument validation, workspace sizing and dispatch.  No kernel
// launches happen before every host-visible argument has been checked.
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "csa2.h"
#include <cstdint>
#include "internal.h"

namespace {

thread_local char g_msg[512] = "";

csa2_status fail(csa2_status st, const char* fmt, ...) {
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(g_msg, sizeof(g_msg), fmt, ap);
  va_end(ap);
  return st;
}

csa2_status ok() {
  g_msg[0] = 0;
  return CSA2_OK;
}

csa2_status cuda_status(cudaError_t e, const char* where) {
  if (e != cudaSuccess) return fail(CSA2_ERR_CUDA, "%s: %s", where, cudaGetErrorString(e));
  return ok();
}

#define REQUIRE(cond, st, ...) \
  do {                         \
    if (!(cond)) return fail(st, __VA_ARGS__); \
  } while (0)

csa2_status check_cache(const csa2_cache& c, bool need_codes, bool need_idx) {
  REQUIRE(c.page_table, CSA2_ERR_INVALID_ARG, "cache.page_table is NULL");
  REQUIRE(c.page_size == CSA2_PAGE_SIZE, CSA2_ERR_UNSUPPORTED_SHAPE, "cache.page_size must be 64 (got %d)",
          c.page_size);
  REQUIRE(c.num_pages > 0 && c.num_seqs > 0 && c.max_pages > 0, CSA2_ERR_INVALID_ARG,
          "cache.num_pages/num_seqs/max_pages must be positive");
  REQUIRE(c.num_pages <= (1 << 25), CSA2_ERR_UNSUPPORTED_SHAPE,
          "cache.num_pages must be <= 2^25 (row indices are 31-bit)");
  REQUIRE(c.d == 128 || c.d == 512, CSA2_ERR_UNSUPPORTED_SHAPE, "cache.d must be 128 or 512 (got %d)", c.d);
  if (need_codes) {
    REQUIRE(c.codes && c.scales, CSA2_ERR_INVALID_ARG, "cache.codes/scales is NULL");
    REQUIRE(((uintptr_t)c.codes & 15) == 0 && ((uintptr_t)c.scales & 15) == 0, CSA2_ERR_INVALID_ARG,
            "cache.codes/scales must be 16-byte aligned");
  }
  REQUIRE(c.idx_k_dtype == CSA2_BF16 || c.idx_k_dtype == CSA2_FP8E4M3, CSA2_ERR_INVALID_ARG,
          "cache.idx_k_dtype must be CSA2_BF16 or CSA2_FP8E4M3");
  if (need_idx) {
    if (c.idx_k_dtype == CSA2_BF16) {
      REQUIRE(c.idx_k, CSA2_ERR_INVALID_ARG, "cache.idx_k is NULL");
      REQUIRE(((uintptr_t)c.idx_k & 15) == 0, CSA2_ERR_INVALID_ARG, "cache.idx_k must be 16-byte aligned");
    } else {
      REQUIRE(c.idx_k8 && c.idx_k8_scale, CSA2_ERR_INVALID_ARG, "cache.idx_k8 / idx_k8_scale is NULL");
      REQUIRE(((uintptr_t)c.idx_k8 & 15) == 0 && ((uintptr_t)c.idx_k8_scale & 15) == 0, CSA2_ERR_INVALID_ARG,
              "cache.idx_k8 and idx_k8_scale must be 16-byte aligned");
    }
    REQUIRE(c.d_ik == 64 || c.d_ik == 128, CSA2_ERR_UNSUPPORTED_SHAPE, "cache.d_ik must be 64 or 128 (got %d)",
            c.d_ik);
  }
  return CSA2_OK;
}

csa2_status check_compress(const csa2_compress_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_compress_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  REQUIRE(a->T >= 0, CSA2_ERR_INVALID_ARG, "T < 0");
  REQUIRE(a->m >= 1 && a->m <= 8, CSA2_ERR_UNSUPPORTED_SHAPE, "m must be in 1..8 (got %d)", a->m);
  REQUIRE(a->T % a->m == 0, CSA2_ERR_INVALID_ARG, "T (%d) is not a multiple of m (%d)", a->T, a->m);
  csa2_status s = check_cache(a->cache, true, a->W_ik != nullptr);
  if (s != CSA2_OK) return s;
  const int d = a->cache.d;
  if (a->W_kv) {
    REQUIRE(a->H, CSA2_ERR_INVALID_ARG, "H is NULL");
    REQUIRE(a->h_dtype == CSA2_BF16 || a->h_dtype == CSA2_F32, CSA2_ERR_INVALID_ARG, "bad h_dtype");
    REQUIRE(a->d_model > 0 && a->d_model % 32 == 0, CSA2_ERR_UNSUPPORTED_SHAPE,
            "d_model must be a positive multiple of 32 (got %d)", a->d_model);
    REQUIRE(a->m == 1 || a->W_z, CSA2_ERR_INVALID_ARG, "W_z is NULL with m > 1");
  } else {
    REQUIRE(a->C, CSA2_ERR_INVALID_ARG, "given mode: C is NULL");
    REQUIRE(a->m == 1 || a->Z, CSA2_ERR_INVALID_ARG, "given mode: Z is NULL with m > 1");
  }
  REQUIRE(a->d_rope == 0 || a->d_rope == 32 || a->d_rope == 64, CSA2_ERR_UNSUPPORTED_SHAPE,
          "d_rope must be 0, 32 or 64 (got %d)", a->d_rope);
  REQUIRE(a->d_rope <= d, CSA2_ERR_UNSUPPORTED_SHAPE, "d_rope > d");
  if (a->d_rope) {
    REQUIRE(a->rope_cos && a->rope_sin && a->pos, CSA2_ERR_INVALID_ARG, "RoPE tables or pos is NULL");
    REQUIRE(a->rope_max_pos > 0, CSA2_ERR_INVALID_ARG, "rope_max_pos must be positive");
  }
  if (a->T > 0) REQUIRE(a->seq && a->entry, CSA2_ERR_INVALID_ARG, "seq/entry is NULL");
  return CSA2_OK;
}

csa2_status check_append(const csa2_append_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_append_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  REQUIRE(a->B >= 0, CSA2_ERR_INVALID_ARG, "B < 0");
  REQUIRE(a->m >= 1 && a->m <= 8, CSA2_ERR_UNSUPPORTED_SHAPE, "m must be in 1..8 (got %d)", a->m);
  csa2_status s = check_cache(a->cache, true, a->W_ik != nullptr);
  if (s != CSA2_OK) return s;
  REQUIRE(a->h_dtype == CSA2_BF16 || a->h_dtype == CSA2_F32, CSA2_ERR_INVALID_ARG, "bad h_dtype");
  REQUIRE(a->d_model > 0 && a->d_model % 32 == 0, CSA2_ERR_UNSUPPORTED_SHAPE,
          "d_model must be a positive multiple of 32 (got %d)", a->d_model);
  REQUIRE(a->d_rope == 0 || a->d_rope == 32 || a->d_rope == 64, CSA2_ERR_UNSUPPORTED_SHAPE,
          "d_rope must be 0, 32 or 64 (got %d)", a->d_rope);
  REQUIRE(a->d_rope <= a->cache.d, CSA2_ERR_UNSUPPORTED_SHAPE, "d_rope > d");
  if (a->B > 0) {
    REQUIRE(a->H && a->W_kv && a->seq && a->tok_pos, CSA2_ERR_INVALID_ARG, "H/W_kv/seq/tok_pos is NULL");
    REQUIRE(a->m == 1 || (a->W_z && a->pend), CSA2_ERR_INVALID_ARG, "W_z and pend are required when m > 1");
    if (a->d_rope)
      REQUIRE(a->rope_cos && a->rope_sin && a->rope_max_pos > 0, CSA2_ERR_INVALID_ARG,
              "RoPE tables are NULL or rope_max_pos <= 0");
    REQUIRE(((uintptr_t)a->H & 15) == 0 && ((uintptr_t)a->W_kv & 15) == 0 && ((uintptr_t)a->W_z & 15) == 0,
            CSA2_ERR_INVALID_ARG, "H, W_kv and W_z must be 16-byte aligned");
  }
  return CSA2_OK;
}

csa2_status check_index_common(int B, int H_i, const uint16_t* q, const float* w, const csa2_cache& c,
                               const int32_t* seq_of, int k, int* topk, int* topk_len) {
  REQUIRE(B >= 0, CSA2_ERR_INVALID_ARG, "B < 0");
  REQUIRE(H_i >= 1 && H_i <= 32, CSA2_ERR_UNSUPPORTED_SHAPE, "H_i must be in 1..32 (got %d)", H_i);
  REQUIRE(k >= 1 && k <= 2048, CSA2_ERR_UNSUPPORTED_SHAPE, "k must be in 1..2048 (got %d)", k);
  csa2_status s = check_cache(c, false, true);
  if (s != CSA2_OK) return s;
  if (B > 0) REQUIRE(q && w && seq_of && topk && topk_len, CSA2_ERR_INVALID_ARG, "a required pointer is NULL");
  return CSA2_OK;
}

csa2_status check_full(const csa2_index_full_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_index_full_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  csa2_status s = check_index_common(a->B, a->H_i, a->q_idx, a->w, a->cache, a->seq_of, a->k, a->topk, a->topk_len);
  if (s != CSA2_OK) return s;
  REQUIRE(a->num_blocks >= 1 && a->per_block >= 1 && a->per_block <= 32, CSA2_ERR_UNSUPPORTED_SHAPE,
          "need num_blocks >= 1 and per_block in 1..32");
  REQUIRE((long long)a->num_blocks * a->per_block <= 16384, CSA2_ERR_UNSUPPORTED_SHAPE,
          "num_blocks * per_block must be <= 16384");
  REQUIRE(a->max_n >= 0 && (long long)a->max_n <= (long long)a->cache.max_pages * CSA2_PAGE_SIZE,
          CSA2_ERR_INVALID_ARG, "max_n must be in [0, max_pages*64]");
  if (a->B > 0) REQUIRE(a->n_vis && a->pool && a->pool_len, CSA2_ERR_INVALID_ARG, "a required pointer is NULL");
  REQUIRE(a->group >= 0, CSA2_ERR_INVALID_ARG, "group must be >= 0 (got %d)", a->group);
  if (a->group > 1) {
    REQUIRE(a->B % a->group == 0, CSA2_ERR_INVALID_ARG, "B (%d) must be a multiple of group (%d)", a->B, a->group);
  }
  return CSA2_OK;
}

csa2_status check_reindex(const csa2_index_reindex_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_index_reindex_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  csa2_status s = check_index_common(a->B, a->H_i, a->q_idx, a->w, a->cache, a->seq_of, a->k, a->topk, a->topk_len);
  if (s != CSA2_OK) return s;
  REQUIRE(a->pool_stride >= 1 && a->pool_stride <= 16384, CSA2_ERR_UNSUPPORTED_SHAPE,
          "pool_stride must be in 1..16384");
  if (a->B > 0) REQUIRE(a->pool && a->pool_len, CSA2_ERR_INVALID_ARG, "pool/pool_len is NULL");
  return CSA2_OK;
}

csa2_status check_attn(const csa2_attn_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_attn_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  REQUIRE(a->B >= 0, CSA2_ERR_INVALID_ARG, "B < 0");
  REQUIRE(a->Hq == 8 || a->Hq == 16 || a->Hq == 32 || a->Hq == 64, CSA2_ERR_UNSUPPORTED_SHAPE,
          "Hq must be 8, 16, 32 or 64 (got %d)", a->Hq);
  csa2_status s = check_cache(a->cache, true, false);
  if (s != CSA2_OK) return s;
  REQUIRE(a->k >= 0 && a->swa_max >= 0 && a->k + a->swa_max <= 4096, CSA2_ERR_UNSUPPORTED_SHAPE,
          "need k >= 0, swa_max >= 0, k + swa_max <= 4096");
  REQUIRE(a->out_dtype == CSA2_BF16 || a->out_dtype == CSA2_F32, CSA2_ERR_INVALID_ARG, "bad out_dtype");
  if (a->B > 0) {
    REQUIRE(a->q && a->seq_of && a->out, CSA2_ERR_INVALID_ARG, "q/seq_of/out is NULL");
    REQUIRE(((uintptr_t)a->q & 15) == 0, CSA2_ERR_INVALID_ARG, "q must be 16-byte aligned");
    if (a->k > 0) REQUIRE(a->topk, CSA2_ERR_INVALID_ARG, "topk is NULL");
    if (a->swa_max > 0)
      REQUIRE(a->swa && a->swa_scale && a->swa_start && a->swa_len && a->swa_rows > 0, CSA2_ERR_INVALID_ARG,
              "SWA pointers are NULL or swa_rows <= 0");
  }
  return CSA2_OK;
}

csa2_status check_swa_quant(const csa2_swa_quant_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_swa_quant_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  REQUIRE(a->R >= 0, CSA2_ERR_INVALID_ARG, "R < 0");
  REQUIRE(a->d == 128 || a->d == 512, CSA2_ERR_UNSUPPORTED_SHAPE, "d must be 128 or 512 (got %d)", a->d);
  REQUIRE(a->x_dtype == CSA2_BF16 || a->x_dtype == CSA2_F32, CSA2_ERR_INVALID_ARG, "bad x_dtype");
  if (a->R > 0) {
    REQUIRE(a->x && a->swa && a->swa_scale, CSA2_ERR_INVALID_ARG, "x/swa/swa_scale is NULL");
    REQUIRE(a->swa_rows > 0, CSA2_ERR_INVALID_ARG, "swa_rows must be positive");
    REQUIRE(a->row_idx || a->R <= a->swa_rows, CSA2_ERR_INVALID_ARG, "R > swa_rows without row_idx");
    REQUIRE(((uintptr_t)a->x & 15) == 0, CSA2_ERR_INVALID_ARG, "x must be 16-byte aligned");
    REQUIRE(((uintptr_t)a->swa & (a->d == 512 ? 15 : 3)) == 0, CSA2_ERR_INVALID_ARG,
            "swa must be 16-byte (d = 512) or 4-byte (d = 128) aligned");
  }
  return CSA2_OK;
}

bool is_float(csa2_dtype t) { return t == CSA2_BF16 || t == CSA2_F32; }
bool on(const void* p, csa2_dtype t) { return ((uintptr_t)p & (t == CSA2_F32 ? 3 : 1)) == 0; }

// most: what the kernels' 32-bit offsets reach, with the whole steps they round cols up to, or less
csa2_status check_fp4_rows(const csa2_fp4_rows& m, const char* name, int multiple, int most) {
  REQUIRE(m.rows >= 0 && m.rows <= (1 << 23), CSA2_ERR_UNSUPPORTED_SHAPE, "%s.rows must be in 0..2^23 (got %d)", name,
          m.rows);
  REQUIRE(m.cols > 0 && m.cols % multiple == 0, CSA2_ERR_UNSUPPORTED_SHAPE,
          "%s.cols must be a positive multiple of %d (got %d)", name, multiple, m.cols);
  REQUIRE(m.cols <= most, CSA2_ERR_UNSUPPORTED_SHAPE, "%s.cols must be at most %d (got %d)", name, most, m.cols);
  if (m.rows > 0) {
    REQUIRE(m.codes && m.scales, CSA2_ERR_INVALID_ARG, "%s.codes/scales is NULL", name);
    REQUIRE(((uintptr_t)m.codes & 15) == 0 && ((uintptr_t)m.scales & 15) == 0, CSA2_ERR_INVALID_ARG,
            "%s.codes/scales must be 16-byte aligned", name);
    REQUIRE(((uintptr_t)m.gscale & 3) == 0, CSA2_ERR_INVALID_ARG, "%s.gscale must be 4-byte aligned", name);
  }
  return CSA2_OK;
}

csa2_status check_rms_norm(const csa2_rms_norm_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_rms_norm_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  REQUIRE(a->T >= 0, CSA2_ERR_INVALID_ARG, "T < 0");
  REQUIRE(a->D >= 1 && a->D <= 32768, CSA2_ERR_UNSUPPORTED_SHAPE, "D must be in 1..32768 (got %d)", a->D);
  REQUIRE(is_float(a->x_dtype), CSA2_ERR_INVALID_ARG, "bad x_dtype");
  REQUIRE(a->eps >= 0.f, CSA2_ERR_INVALID_ARG, "eps must be >= 0");
  REQUIRE(!a->weight || is_float(a->weight_dtype), CSA2_ERR_INVALID_ARG, "bad weight_dtype");
  REQUIRE(!a->weight || on(a->weight, a->weight_dtype), CSA2_ERR_INVALID_ARG, "weight is not aligned to its type");
  REQUIRE(a->out_form >= CSA2_BF16 && a->out_form <= CSA2_FP4E2M1X2, CSA2_ERR_INVALID_ARG, "bad out_form");
  if (a->out_form == CSA2_FP8E4M3)
    REQUIRE(a->scale_group == 0 || a->scale_group == 128, CSA2_ERR_UNSUPPORTED_SHAPE,
            "scale_group must be 0 or 128 (got %d)", a->scale_group);
  if (a->out_form == CSA2_FP4E2M1X2) {
    REQUIRE(a->out4.rows == a->T && a->out4.cols == a->D, CSA2_ERR_INVALID_ARG, "out4 must be [T][D]");
    csa2_status s = check_fp4_rows(a->out4, "out4", 16, 1 << 30);
    if (s != CSA2_OK) return s;
  }
  if (a->T > 0) {
    REQUIRE(a->x && on(a->x, a->x_dtype), CSA2_ERR_INVALID_ARG, "x is NULL or not aligned to its type");
    if (a->residual) {
      REQUIRE(is_float(a->res_dtype), CSA2_ERR_INVALID_ARG, "bad res_dtype");
      REQUIRE(a->residual_out, CSA2_ERR_INVALID_ARG, "residual_out is NULL with a residual");
      REQUIRE(on(a->residual, a->res_dtype) && on(a->residual_out, a->res_dtype), CSA2_ERR_INVALID_ARG,
              "residual or residual_out is not aligned to its type");
      REQUIRE(a->T == 1 || a->residual_out_stride >= a->D, CSA2_ERR_INVALID_ARG, "residual_out rows overlap");
    } else {
      REQUIRE(!a->residual_out, CSA2_ERR_INVALID_ARG, "residual_out without a residual");
    }
    if (a->out_form != CSA2_FP4E2M1X2) {
      REQUIRE(a->out, CSA2_ERR_INVALID_ARG, "out is NULL");
      REQUIRE(a->out_form == CSA2_FP8E4M3 || on(a->out, a->out_form), CSA2_ERR_INVALID_ARG,
              "out is not aligned to its type");
      REQUIRE(a->T == 1 || a->out_stride >= a->D, CSA2_ERR_INVALID_ARG, "out rows overlap");
    }
    if (a->out_form == CSA2_FP8E4M3)
      REQUIRE(a->out_scale && on(a->out_scale, CSA2_F32), CSA2_ERR_INVALID_ARG, "out_scale is NULL or not aligned");
  }
  return CSA2_OK;
}

csa2_status check_rope(const csa2_rope_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_rope_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  REQUIRE(a->T >= 0 && a->H >= 0, CSA2_ERR_INVALID_ARG, "T or H < 0");
  REQUIRE(a->D >= 1 && a->D <= 4096, CSA2_ERR_UNSUPPORTED_SHAPE, "D must be in 1..4096 (got %d)", a->D);
  REQUIRE(a->d_rope >= 2 && a->d_rope % 2 == 0, CSA2_ERR_UNSUPPORTED_SHAPE, "d_rope must be even and >= 2 (got %d)",
          a->d_rope);
  REQUIRE(a->rot_first >= 0 && a->rot_first <= a->D - a->d_rope, CSA2_ERR_INVALID_ARG,
          "rot_first + d_rope must lie in 0..D");
  REQUIRE(is_float(a->dtype), CSA2_ERR_INVALID_ARG, "bad dtype");
  if (a->T > 0 && a->H > 0) {
    REQUIRE(a->x && a->out && a->pos && a->rope_cos && a->rope_sin, CSA2_ERR_INVALID_ARG, "a required pointer is NULL");
    REQUIRE(a->rope_max_pos > 0, CSA2_ERR_INVALID_ARG, "rope_max_pos must be positive");
    REQUIRE(on(a->x, a->dtype) && on(a->out, a->dtype), CSA2_ERR_INVALID_ARG, "x or out is not aligned to its type");
    REQUIRE(on(a->pos, CSA2_F32) && on(a->rope_cos, CSA2_F32) && on(a->rope_sin, CSA2_F32), CSA2_ERR_INVALID_ARG,
            "pos or a table is not aligned to its type");
    REQUIRE(a->out != a->x || (a->out_stride_t == a->x_stride_t && a->out_stride_h == a->x_stride_h),
            CSA2_ERR_INVALID_ARG, "in place x and out must have the same strides");
    // the heads of a token, or the tokens of a head, are the inner rows of the output
    const int64_t st = a->T > 1 ? a->out_stride_t : INT64_MAX, sh = a->H > 1 ? a->out_stride_h : INT64_MAX;
    const int64_t inner = sh <= st ? sh : st, outer = sh <= st ? st : sh, n = sh <= st ? a->H : a->T;
    REQUIRE(inner >= a->D && (outer == INT64_MAX || outer >= (n - 1) * inner + a->D), CSA2_ERR_INVALID_ARG,
            "out rows overlap");
  }
  return CSA2_OK;
}

csa2_status check_rope_table(const csa2_rope_table_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_rope_table_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  REQUIRE(a->positions >= 0 && a->positions <= (1 << 24), CSA2_ERR_UNSUPPORTED_SHAPE,
          "positions must be in 0..2^24 (got %d)", a->positions);
  REQUIRE(a->d_rope >= 2 && a->d_rope % 2 == 0 && a->d_rope <= 256, CSA2_ERR_UNSUPPORTED_SHAPE,
          "d_rope must be even and in 2..256 (got %d)", a->d_rope);
  REQUIRE(a->scaling >= CSA2_ROPE_PLAIN && a->scaling <= CSA2_ROPE_YARN, CSA2_ERR_INVALID_ARG, "bad scaling");
  REQUIRE(a->theta > 1.0 && a->theta <= 1e30, CSA2_ERR_INVALID_ARG, "theta must be in (1, 1e30]");
  REQUIRE(a->magnitude > 0.0 && a->magnitude <= 1e30, CSA2_ERR_INVALID_ARG, "magnitude must be in (0, 1e30]");
  if (a->scaling != CSA2_ROPE_PLAIN)
    REQUIRE(a->factor >= 1.0 && a->factor <= 1e30, CSA2_ERR_INVALID_ARG, "factor must be in [1, 1e30]");
  if (a->scaling == CSA2_ROPE_YARN) {
    REQUIRE(a->orig_positions > 0, CSA2_ERR_INVALID_ARG, "orig_positions must be positive");
    REQUIRE(a->beta_slow > 0.0 && a->beta_slow < a->beta_fast && a->beta_fast <= 1e30, CSA2_ERR_INVALID_ARG,
            "need 0 < beta_slow < beta_fast");
  }
  if (a->positions > 0)
    REQUIRE(a->rope_cos && a->rope_sin && on(a->rope_cos, CSA2_F32) && on(a->rope_sin, CSA2_F32), CSA2_ERR_INVALID_ARG,
            "rope_cos/rope_sin is NULL or not aligned");
  return CSA2_OK;
}

csa2_status check_fp4_quant(const csa2_fp4_quant_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_fp4_quant_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  REQUIRE(is_float(a->x_dtype), CSA2_ERR_INVALID_ARG, "bad x_dtype");
  csa2_status s = check_fp4_rows(a->out, "out", 16, 1 << 30);
  if (s != CSA2_OK) return s;
  if (a->out.rows > 0)
    REQUIRE(a->x && on(a->x, a->x_dtype), CSA2_ERR_INVALID_ARG, "x is NULL or not aligned to its type");
  return CSA2_OK;
}

constexpr int kMaxSum = 1 << 26;   // a sum this long ends in a small part of the time that the product's waits allow

csa2_status check_fp4_linear(const csa2_fp4_linear_args* a) {
  REQUIRE(a, CSA2_ERR_INVALID_ARG, "args is NULL");
  REQUIRE(a->struct_size == sizeof(csa2_fp4_linear_args), CSA2_ERR_INVALID_ARG, "struct_size mismatch");
  csa2_status s = check_fp4_rows(a->x, "x", 32, kMaxSum);
  if (s != CSA2_OK) return s;
  s = check_fp4_rows(a->w, "w", 32, kMaxSum);
  if (s != CSA2_OK) return s;
  REQUIRE(a->x.cols == a->w.cols, CSA2_ERR_INVALID_ARG, "x.cols (%d) != w.cols (%d)", a->x.cols, a->w.cols);
  REQUIRE(is_float(a->out_dtype), CSA2_ERR_INVALID_ARG, "bad out_dtype");
  if (a->x.rows > 0 && a->w.rows > 0)
    REQUIRE(a->out && on(a->out, a->out_dtype), CSA2_ERR_INVALID_ARG, "out is NULL or not aligned to its type");
  return CSA2_OK;
}

csa2_status check_ws(size_t need, void* ws, size_t have) {
  REQUIRE(have >= need, CSA2_ERR_WORKSPACE_TOO_SMALL, "workspace needs %zu bytes, got %zu", need, have);
  REQUIRE(need == 0 || ws, CSA2_ERR_INVALID_ARG, "workspace is NULL");
  REQUIRE(need == 0 || ((uintptr_t)ws & 255) == 0, CSA2_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  return CSA2_OK;
}

}  // namespace

extern "C" {

csa2_status csa2_compress_quant_workspace(const csa2_compress_args* a, size_t* bytes) {
  csa2_status s = check_compress(a);
  if (s != CSA2_OK) return s;
  REQUIRE(bytes, CSA2_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = csa2::compress_workspace_bytes(*a);
  return ok();
}

csa2_status csa2_compress_quant(const csa2_compress_args* a, void* ws, size_t ws_bytes, void* stream) {
  csa2_status s = check_compress(a);
  if (s != CSA2_OK) return s;
  s = check_ws(csa2::compress_workspace_bytes(*a), ws, ws_bytes);
  if (s != CSA2_OK) return s;
  if (a->T == 0) return ok();
  return cuda_status(csa2::launch_compress(*a, ws, static_cast<cudaStream_t>(stream)), "csa2_compress_quant");
}

csa2_status csa2_compress_append_workspace(const csa2_append_args* a, size_t* bytes) {
  csa2_status s = check_append(a);
  if (s != CSA2_OK) return s;
  REQUIRE(bytes, CSA2_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = csa2::append_workspace_bytes(*a);
  return ok();
}

csa2_status csa2_compress_append(const csa2_append_args* a, void* ws, size_t ws_bytes, void* stream) {
  csa2_status s = check_append(a);
  if (s != CSA2_OK) return s;
  s = check_ws(csa2::append_workspace_bytes(*a), ws, ws_bytes);
  if (s != CSA2_OK) return s;
  return cuda_status(csa2::launch_append(*a, ws, static_cast<cudaStream_t>(stream)), "csa2_compress_append");
}

csa2_status csa2_index_full_workspace(const csa2_index_full_args* a, size_t* bytes) {
  csa2_status s = check_full(a);
  if (s != CSA2_OK) return s;
  REQUIRE(bytes, CSA2_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = csa2::index_full_workspace_bytes(*a);
  return ok();
}

csa2_status csa2_index_full(const csa2_index_full_args* a, void* ws, size_t ws_bytes, void* stream) {
  csa2_status s = check_full(a);
  if (s != CSA2_OK) return s;
  s = check_ws(csa2::index_full_workspace_bytes(*a), ws, ws_bytes);
  if (s != CSA2_OK) return s;
  return cuda_status(csa2::launch_index_full(*a, ws, static_cast<cudaStream_t>(stream)), "csa2_index_full");
}

csa2_status csa2_index_full_noalloc(const csa2_index_full_args* a, void* stream) {
  csa2_status s = check_full(a);
  if (s != CSA2_OK) return s;
  REQUIRE(a->cache.idx_k_dtype == CSA2_BF16, CSA2_ERR_UNSUPPORTED_SHAPE,
          "csa2_index_full_noalloc: the FP8 indexer-K form needs workspace for the quantised indexer Q; "
          "use csa2_index_full");
  const long long need = (long long)a->B * a->num_blocks * a->per_block;
  REQUIRE(need <= CSA2_NOALLOC_MAX_SCORES, CSA2_ERR_UNSUPPORTED_SHAPE,
          "csa2_index_full_noalloc: B*num_blocks*per_block = %lld exceeds the fixed scratch of %d scores",
          need, CSA2_NOALLOC_MAX_SCORES);
  void* scratch = nullptr;
  size_t have = 0;
  cudaError_t e = csa2::index_noalloc_scratch(&scratch, &have);
  if (e != cudaSuccess) return cuda_status(e, "csa2_index_full_noalloc: scratch address lookup");
  // the fixed scratch holds the pool scores only: no tensor-core score matrix
  return cuda_status(csa2::launch_index_full(*a, scratch, static_cast<cudaStream_t>(stream), false),
                     "csa2_index_full_noalloc");
}

csa2_status csa2_index_reindex_workspace(const csa2_index_reindex_args* a, size_t* bytes) {
  csa2_status s = check_reindex(a);
  if (s != CSA2_OK) return s;
  REQUIRE(bytes, CSA2_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = csa2::index_reindex_workspace_bytes(*a);
  return ok();
}

csa2_status csa2_index_reindex(const csa2_index_reindex_args* a, void* ws, size_t ws_bytes, void* stream) {
  csa2_status s = check_reindex(a);
  if (s != CSA2_OK) return s;
  s = check_ws(csa2::index_reindex_workspace_bytes(*a), ws, ws_bytes);
  if (s != CSA2_OK) return s;
  return cuda_status(csa2::launch_index_reindex(*a, ws, static_cast<cudaStream_t>(stream)), "csa2_index_reindex");
}

csa2_status csa2_sparse_attn_workspace(const csa2_attn_args* a, size_t* bytes) {
  csa2_status s = check_attn(a);
  if (s != CSA2_OK) return s;
  REQUIRE(bytes, CSA2_ERR_INVALID_ARG, "bytes is NULL");
  *bytes = csa2::attn_workspace_bytes(*a);
  return ok();
}

csa2_status csa2_sparse_attn(const csa2_attn_args* a, void* ws, size_t ws_bytes, void* stream) {
  csa2_status s = check_attn(a);
  if (s != CSA2_OK) return s;
  s = check_ws(csa2::attn_workspace_bytes(*a), ws, ws_bytes);
  if (s != CSA2_OK) return s;
  return cuda_status(csa2::launch_attn(*a, ws, static_cast<cudaStream_t>(stream)), "csa2_sparse_attn");
}

csa2_status csa2_swa_quant(const csa2_swa_quant_args* a, void* stream) {
  csa2_status s = check_swa_quant(a);
  if (s != CSA2_OK) return s;
  return cuda_status(csa2::launch_swa_quant(*a, static_cast<cudaStream_t>(stream)), "csa2_swa_quant");
}

csa2_status csa2_rms_norm(const csa2_rms_norm_args* a, void* stream) {
  csa2_status s = check_rms_norm(a);
  if (s != CSA2_OK) return s;
  return cuda_status(csa2::launch_rms_norm(*a, static_cast<cudaStream_t>(stream)), "csa2_rms_norm");
}

csa2_status csa2_rope(const csa2_rope_args* a, void* stream) {
  csa2_status s = check_rope(a);
  if (s != CSA2_OK) return s;
  return cuda_status(csa2::launch_rope(*a, static_cast<cudaStream_t>(stream)), "csa2_rope");
}

csa2_status csa2_rope_table(const csa2_rope_table_args* a, void* stream) {
  csa2_status s = check_rope_table(a);
  if (s != CSA2_OK) return s;
  return cuda_status(csa2::launch_rope_table(*a, static_cast<cudaStream_t>(stream)), "csa2_rope_table");
}

csa2_status csa2_fp4_quant(const csa2_fp4_quant_args* a, void* stream) {
  csa2_status s = check_fp4_quant(a);
  if (s != CSA2_OK) return s;
  return cuda_status(csa2::launch_fp4_quant(*a, static_cast<cudaStream_t>(stream)), "csa2_fp4_quant");
}

csa2_status csa2_fp4_linear(const csa2_fp4_linear_args* a, void* stream) {
  csa2_status s = check_fp4_linear(a);
  if (s != CSA2_OK) return s;
  return cuda_status(csa2::launch_fp4_linear(*a, static_cast<cudaStream_t>(stream)), "csa2_fp4_linear");
}

const char* csa2_last_error_message(void) { return g_msg; }

csa2_status csa2_get_device_error(uint32_t* word) {
  REQUIRE(word, CSA2_ERR_INVALID_ARG, "word is NULL");
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return cuda_status(e, "csa2_get_device_error");
  *word = csa2::read_clear_error_compress() | csa2::read_clear_error_proj() | csa2::read_clear_error_index() |
          csa2::read_clear_error_score() | csa2::read_clear_error_attn() | csa2::read_clear_error_rope() |
          csa2::read_clear_error_fp4();
  csa2_status s = cuda_status(cudaGetLastError(), "csa2_get_device_error");
  if (s != CSA2_OK) return s;
  if (*word & CSA2_DEVERR_TIMEOUT) return fail(CSA2_ERR_TIMEOUT, "a bounded wait gave up (device word 0x%x)", *word);
  if (*word) return fail(CSA2_ERR_DEVICE_CHECK, "a device-side check failed (device word 0x%x)", *word);
  return CSA2_OK;
}

int32_t csa2_version(void) { return 100; }

csa2_status csa2_selftest_wait_timeout(int32_t polls, void* stream) {
  REQUIRE(polls >= 1 && polls <= (1 << 20), CSA2_ERR_INVALID_ARG, "polls must be in 1..2^20 (got %d)", polls);
  return cuda_status(csa2::launch_selftest_wait(polls, static_cast<cudaStream_t>(stream)),
                     "csa2_selftest_wait_timeout");
}

}  // extern "C"
