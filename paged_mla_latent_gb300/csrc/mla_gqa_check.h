// Host-side argument checks shared by the entry points for layers whose heads keep their own
// keys and values (mla_gqa_rope_and_cache, mla_gqa_decode, mla_prompt_attention, mla_gqa_block_*).
#pragma once

#include <stdint.h>

#include "../../include/paged_mla.h"

namespace pmla {

inline bool gqa_aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// (n, heads, width) BF16: last dim contiguous, the other strides non-negative multiples of
// `unit` elements, the base aligned to as many.  An empty tensor may have a null pointer.
inline bool gqa_check_bf16(const mla_tensor_t* t, int64_t n, int64_t heads, int64_t width, int unit) {
  if (!t || t->dtype != MLA_DTYPE_BF16 || t->ndim != 3) return false;
  if (t->shape[0] != n || t->shape[1] != heads || t->shape[2] != width) return false;
  if (!t->ptr && n != 0) return false;
  for (int i = 0; i < 2; ++i)
    if (t->stride[i] < 0 || t->stride[i] % unit != 0) return false;
  return t->stride[2] == 1 && gqa_aligned(t->ptr, 2 * static_cast<uintptr_t>(unit));
}

// No two rows of a (n, heads, width) output share an element: the inner of its two outer dims
// steps at least a row, the other at least the inner one's extent.  (Rows in one place would be
// written by several threads at once, the last of which differs from call to call.)
inline bool gqa_rows_apart(const mla_tensor_t* t) {
  const bool heads_inner = t->stride[1] <= t->stride[0];
  int64_t extent = t->shape[2];
  for (int i = 0; i < 2; ++i) {
    const int dim = (i == 0) == heads_inner ? 1 : 0;
    if (t->shape[dim] <= 1) continue;        // never stepped
    if (t->stride[dim] < extent) return false;
    extent += (t->shape[dim] - 1) * t->stride[dim];
  }
  return true;
}

inline bool gqa_check_i32(const mla_tensor_t* t, int64_t n) {
  return t && (t->ptr || n == 0) && t->dtype == MLA_DTYPE_INT32 && t->ndim == 1 &&
         t->shape[0] == n && (n <= 1 || t->stride[0] == 1) && gqa_aligned(t->ptr, 4);
}

inline bool gqa_check_scalar(const mla_tensor_t* t) {
  if (!t || !t->ptr || t->dtype != MLA_DTYPE_FP32 || t->ndim < 0 || t->ndim > 4) return false;
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] != 1) return false;
  return gqa_aligned(t->ptr, 4);
}

inline bool gqa_check_scalar_i32(const mla_tensor_t* t) {
  if (!t || !t->ptr || t->dtype != MLA_DTYPE_INT32 || t->ndim < 0 || t->ndim > 4) return false;
  for (int i = 0; i < t->ndim; ++i)
    if (t->shape[i] != 1) return false;
  return gqa_aligned(t->ptr, 4);
}

// A checked pair of per-head caches: the entry of head h in slot s of page p starts
// p * page_pitch + s * slot_pitch + h * head_pitch bytes into either.
struct GqaCache {
  uint8_t *k, *v;
  int64_t page_pitch, slot_pitch, head_pitch;   // bytes
  int64_t n_pages;
  int log2_page;
  bool fp8;
  const float *k_scale, *v_scale;               // null for BF16
};

// k_cache, v_cache: (N_pages, PS, Hk, D) of one type and one set of strides, PS a power of
// two <= 1024, last dim contiguous, the strides of the other dims multiples of 16 bytes, no
// two entries overlapping, N_pages * PS < 2^31.  The order of slots and heads inside a page
// is the strides' (either may be the outer one).
inline int gqa_check_cache_layout(const mla_tensor_t* k, const mla_tensor_t* v, int64_t Hk, int64_t D,
                                  GqaCache* out) {
  if (!k || !v || !k->ptr || !v->ptr || k->ndim != 4 || v->ndim != 4) return MLA_ERR_INVALID_ARG;
  if (k->dtype != MLA_DTYPE_BF16 && k->dtype != MLA_DTYPE_FP8_E4M3FN) return MLA_ERR_INVALID_ARG;
  if (v->dtype != k->dtype) return MLA_ERR_INVALID_ARG;
  const int64_t size = k->dtype == MLA_DTYPE_BF16 ? 2 : 1;
  const int64_t N = k->shape[0], PS = k->shape[1];
  if (N < 1 || PS < 1 || k->shape[2] != Hk || k->shape[3] != D) return MLA_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    if (v->shape[i] != k->shape[i] || (k->shape[i] > 1 && v->stride[i] != k->stride[i]))
      return MLA_ERR_INVALID_ARG;
  if (k->stride[3] != 1 || !gqa_aligned(k->ptr, 16) || !gqa_aligned(v->ptr, 16))
    return MLA_ERR_INVALID_ARG;
  if (PS > 1024 || (PS & (PS - 1)) != 0) return MLA_ERR_UNSUPPORTED;
  if (N > 0x7FFFFFFF / PS) return MLA_ERR_INVALID_ARG;
  // the pitch of a size-1 dim is never stepped
  int64_t sp = PS > 1 ? k->stride[1] * size : 0, hp = Hk > 1 ? k->stride[2] * size : 0;
  int64_t pp = N > 1 ? k->stride[0] * size : 0;
  if (sp % 16 || hp % 16 || pp % 16 || sp < 0 || hp < 0 || pp < 0) return MLA_ERR_INVALID_ARG;
  const int64_t row = D * size;
  // entries nest: the inner of (slot, head) steps at least a row, the outer at least the
  // inner's extent, the page at least the outer's
  const bool heads_inner = PS == 1 || (Hk > 1 && hp <= sp);
  int64_t extent = row;
  for (int i = 0; i < 2; ++i) {
    const bool head = (i == 0) == heads_inner;
    const int64_t n = head ? Hk : PS, pitch = head ? hp : sp;
    if (n > 1) {
      if (pitch < extent) return MLA_ERR_INVALID_ARG;
      extent += (n - 1) * pitch;
    }
  }
  if (N > 1 && pp < extent) {
    // pages may also interleave inside a larger stride (heads outermost): every page's
    // entries then lie in the gap between two heads
    if (!(Hk > 1 && pp >= (PS > 1 ? (PS - 1) * sp + row : row) && hp >= (N - 1) * pp + (PS - 1) * sp + row))
      return MLA_ERR_INVALID_ARG;
  }
  out->k = static_cast<uint8_t*>(k->ptr);
  out->v = static_cast<uint8_t*>(v->ptr);
  out->page_pitch = pp;
  out->slot_pitch = sp;
  out->head_pitch = hp;
  out->n_pages = N;
  out->log2_page = 0;
  while ((int64_t{1} << out->log2_page) < PS) ++out->log2_page;
  out->fp8 = size == 1;
  out->k_scale = out->v_scale = nullptr;
  return MLA_OK;
}

// The same with the caches' scales: one FP32 each with E4M3FN, NULL with BF16.
inline int gqa_check_cache(const mla_tensor_t* k, const mla_tensor_t* v, const mla_tensor_t* ks,
                           const mla_tensor_t* vs, int64_t Hk, int64_t D, GqaCache* out) {
  const int st = gqa_check_cache_layout(k, v, Hk, D, out);
  if (st != MLA_OK) return st;
  if (out->fp8 ? (!gqa_check_scalar(ks) || !gqa_check_scalar(vs)) : (ks || vs)) return MLA_ERR_INVALID_ARG;
  if (out->fp8) {
    out->k_scale = static_cast<const float*>(ks->ptr);
    out->v_scale = static_cast<const float*>(vs->ptr);
  }
  return MLA_OK;
}

// E4M3FN caches with a scale for each block of slots and head.
struct GqaBlockCache : GqaCache {
  float *ks, *vs;
  int64_t sc_page, sc_block, sc_head;           // strides of both in elements
  int log2_block;                               // slots of a block
};

// Caches as above, E4M3FN; k_scale, v_scale: (N_pages, NB, Hk) FP32 of one set of strides, no
// two elements in one place, NB a power of two <= PS with at most 128 slots a block.
inline int gqa_check_block_cache(const mla_tensor_t* k, const mla_tensor_t* v, const mla_tensor_t* ks,
                                 const mla_tensor_t* vs, int64_t Hk, int64_t D, GqaBlockCache* out) {
  const int st = gqa_check_cache_layout(k, v, Hk, D, out);
  if (st != MLA_OK) return st;
  if (!out->fp8 || !ks || !vs || !ks->ptr || !vs->ptr) return MLA_ERR_INVALID_ARG;
  if (ks->dtype != MLA_DTYPE_FP32 || vs->dtype != MLA_DTYPE_FP32 || ks->ndim != 3 || vs->ndim != 3)
    return MLA_ERR_INVALID_ARG;
  if (!gqa_aligned(ks->ptr, 4) || !gqa_aligned(vs->ptr, 4)) return MLA_ERR_INVALID_ARG;
  const int64_t NB = ks->shape[1], PS = int64_t{1} << out->log2_page;
  if (ks->shape[0] != k->shape[0] || NB < 1 || NB > PS || ks->shape[2] != Hk) return MLA_ERR_INVALID_ARG;
  int64_t stride[3], extent = 1;
  for (int i = 0; i < 3; ++i) {
    if (vs->shape[i] != ks->shape[i] || (ks->shape[i] > 1 && vs->stride[i] != ks->stride[i]))
      return MLA_ERR_INVALID_ARG;
    stride[i] = ks->shape[i] > 1 ? ks->stride[i] : 0;      // never stepped otherwise
  }
  bool taken[3] = {};
  for (int n = 0; n < 3; ++n) {                            // from the innermost dim outwards
    int at = -1;
    for (int i = 0; i < 3; ++i)
      if (!taken[i] && (at < 0 || stride[i] < stride[at])) at = i;
    taken[at] = true;
    if (ks->shape[at] <= 1) continue;
    if (stride[at] < extent) return MLA_ERR_INVALID_ARG;
    extent += (ks->shape[at] - 1) * stride[at];
  }
  if ((NB & (NB - 1)) != 0 || PS / NB > 128) return MLA_ERR_UNSUPPORTED;
  out->ks = static_cast<float*>(ks->ptr);
  out->vs = static_cast<float*>(vs->ptr);
  out->sc_page = stride[0];
  out->sc_block = stride[1];
  out->sc_head = stride[2];
  out->log2_block = 0;
  while ((int64_t{1} << out->log2_block) < PS / NB) ++out->log2_block;
  return MLA_OK;
}

// A page table: kv_indptr (B+1), kv_indices, kv_last_page_lens (B; NULL where pages hold one
// token).
inline bool gqa_check_pages(const mla_tensor_t* indptr, const mla_tensor_t* indices,
                            const mla_tensor_t* last, int64_t B, int log2_page) {
  if (!gqa_check_i32(indptr, B + 1) || !indices || indices->ndim != 1 ||
      !gqa_check_i32(indices, indices->shape[0]))
    return false;
  return last ? gqa_check_i32(last, B) : log2_page == 0;
}

}  // namespace pmla
