// mla_gqa_block_decode: attention of a request's newest tokens over a paged e4m3 cache with a
// scale for each block of positions and head (the kernel's header has the mathematics, the
// split and the figures).
#include "mla_gqa_check.h"
#include "mla_gqa_decode_kernel.cuh"

namespace {
constexpr int64_t kMaxQ = 64;        // as mla_decode
}

extern "C" int mla_get_gqa_block_decode_workspace_size(int32_t num_heads, int32_t num_kv_heads,
                                                       int32_t head_dim, int32_t max_seqlen_q,
                                                       int32_t num_sms, size_t* bytes_out) {
  if (!bytes_out || num_heads < 1 || num_kv_heads < 1 || num_heads > 1024 ||
      num_heads % num_kv_heads != 0 || head_dim < 1 || max_seqlen_q < 1 || max_seqlen_q > kMaxQ ||
      num_sms > 65536)
    return MLA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MLA_ERR_UNSUPPORTED;
  int sms = num_sms;
  if (num_sms <= 0) {
    const int st = sms_for(&sms);
    if (st != MLA_OK) return st;
  }
  *bytes_out = workspace_for(sms, static_cast<int64_t>(num_heads / num_kv_heads) * max_seqlen_q, head_dim);
  return MLA_OK;
}

extern "C" int mla_gqa_block_decode(const mla_tensor_t* q, const mla_tensor_t* k_cache,
                                    const mla_tensor_t* v_cache, const mla_tensor_t* k_scale,
                                    const mla_tensor_t* v_scale, const mla_tensor_t* o,
                                    const mla_tensor_t* qo_indptr, const mla_tensor_t* kv_indptr,
                                    const mla_tensor_t* kv_indices,
                                    const mla_tensor_t* kv_last_page_lens, int32_t max_seqlen_q,
                                    float sm_scale, const mla_tensor_t* lse_out, void* workspace,
                                    size_t workspace_bytes, mla_stream_t stream_) {
  if (!q || !k_cache || !qo_indptr || q->ndim != 3 || k_cache->ndim != 4 || qo_indptr->ndim != 1)
    return MLA_ERR_INVALID_ARG;
  const int64_t T = q->shape[0], Hq = q->shape[1], D = q->shape[2], Hk = k_cache->shape[2];
  const int64_t B = qo_indptr->shape[0] - 1;
  if (T < 0 || T > 0x7FFFFFFF || B < 0 || B > 0xFFFFFF || Hq < 1 || Hq > 1024 || Hk < 1 || Hq % Hk != 0)
    return MLA_ERR_INVALID_ARG;
  if (max_seqlen_q < 1 || max_seqlen_q > kMaxQ) return MLA_ERR_INVALID_ARG;
  if (!gqa_check_bf16(q, T, Hq, D, 8)) return MLA_ERR_INVALID_ARG;
  GqaBlockCache c;
  const int st = gqa_check_block_cache(k_cache, v_cache, k_scale, v_scale, Hk, D, &c);
  if (st != MLA_OK) return st;
  if (!o || (!o->ptr && T > 0) || o->ndim != 3 || (o->dtype != MLA_DTYPE_BF16 && o->dtype != MLA_DTYPE_FP32) ||
      o->shape[0] != T || o->shape[1] != Hq || o->shape[2] != D || o->stride[2] != 1 ||
      o->stride[0] < 0 || o->stride[1] < 0 || !gqa_rows_apart(o) ||
      !gqa_aligned(o->ptr, o->dtype == MLA_DTYPE_FP32 ? 4 : 2))
    return MLA_ERR_INVALID_ARG;
  if (!gqa_check_i32(qo_indptr, B + 1) ||
      !gqa_check_pages(kv_indptr, kv_indices, kv_last_page_lens, B, c.log2_page))
    return MLA_ERR_INVALID_ARG;
  if (lse_out && ((!lse_out->ptr && T > 0) || lse_out->dtype != MLA_DTYPE_FP32 || lse_out->ndim != 2 ||
                  lse_out->shape[0] != T || lse_out->shape[1] != Hq || (Hq > 1 && lse_out->stride[1] != 1) ||
                  (T > 1 && lse_out->stride[0] != Hq) || !gqa_aligned(lse_out->ptr, 4)))
    return MLA_ERR_INVALID_ARG;
  if (!(sm_scale == sm_scale)) return MLA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return MLA_ERR_UNSUPPORTED;
  if (!workspace || !gqa_aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  const int64_t G = Hq / Hk, rows = G * max_seqlen_q;
  if (workspace_bytes < workspace_for(1, rows, D)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  const int cs = sms_for(&sms);
  if (cs != MLA_OK) return cs;
  if (workspace_bytes < workspace_for(sms, rows, D)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (B == 0 || T == 0) return MLA_OK;

  GqaDecodeParams p = {};
  p.q = static_cast<const uint16_t*>(q->ptr);
  p.q_tok = q->stride[0];
  p.q_head = q->stride[1];
  p.k = c.k;
  p.v = c.v;
  p.page_pitch = c.page_pitch;
  p.slot_pitch = c.slot_pitch;
  p.head_pitch = c.head_pitch;
  p.log2_page = c.log2_page;
  p.n_pages = c.n_pages;
  p.kv_indptr = static_cast<const int32_t*>(kv_indptr->ptr);
  p.kv_indices = static_cast<const int32_t*>(kv_indices->ptr);
  p.last = kv_last_page_lens ? static_cast<const int32_t*>(kv_last_page_lens->ptr) : nullptr;
  p.n_idx = kv_indices->shape[0];
  p.sm_scale = sm_scale;
  p.o = o->ptr;
  p.o_f32 = o->dtype == MLA_DTYPE_FP32;
  p.o_tok = o->stride[0];
  p.o_head = o->stride[1];
  p.lse = lse_out ? static_cast<float*>(lse_out->ptr) : nullptr;
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hk = static_cast<int>(Hk);
  p.G = static_cast<int>(G);
  const int heads = 8 * head_tiles(rows, narrow_units(D, true));
  p.chunks = static_cast<int>((rows + heads - 1) / heads);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.err = reinterpret_cast<int*>(ws);
  p.counters = reinterpret_cast<int*>(ws + kHeaderBytes);
  p.slots = reinterpret_cast<float*>(ws + kHeaderBytes + counters_for(sms));
  p.qo_indptr = static_cast<const int32_t*>(qo_indptr->ptr);
  p.n_tok = T;
  p.max_q = max_seqlen_q;
  p.ks = c.ks;
  p.vs = c.vs;
  p.sc_page = c.sc_page;
  p.sc_block = c.sc_block;
  p.sc_head = c.sc_head;
  p.log2_block = c.log2_block;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  const cudaError_t e = D == 64 ? launch_nt<64, true, true>(p, sms, s) : launch_nt<128, true, true>(p, sms, s);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
