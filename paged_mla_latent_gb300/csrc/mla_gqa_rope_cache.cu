// mla_gqa_rope_and_cache: the step before mla_prompt_attention and mla_gqa_decode.
//
// A layer whose heads keep their own keys and values appends them to a paged cache: the
// first R columns of every query and key head are rotated by the token's position, the
// rotated q (and, where the prompt's own attention reads them, the rotated keys) go out in
// bf16, and each token's keys and values land at its cache slot as bf16 or as e4m3 codes.
//
//   pair i of a row: (x, y) -> (x cos_i - y sin_i, y cos_i + x sin_i), i < R/2, the pairs
//   (2i, 2i+1) or (i, i + R/2); columns from R on pass through.
//
// Bytes bound (3 flops an element).  One item is 16 columns of one row: two 16-byte loads
// whose results two 16-byte bf16 stores (or 16 bytes of codes) take, so that every access is
// a whole 16-byte word; 8 pairs share the item's 8 cosines and sines, which come from L1 or
// L2 for all but a token's first head.  Arithmetic is the definition's in fp32, every
// product, sum and quotient rounded on its own, and one rounding to the stored type (a bf16
// value is off by at most 2^-8 of itself, an e4m3 code by 2^-4), so the bytes are exact.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/paged_mla.h"
#include "mla_gqa_check.h"
#include "ptx.cuh"

namespace {

using namespace pmla;

constexpr int kThreads = 256;

struct RopeAppendParams {
  const uint16_t *q, *k, *v;        // bf16 bits
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;   // strides in elements
  uint16_t *q_out, *k_out;          // k_out may be null
  int64_t qo_tok, qo_head, ko_tok, ko_head;
  const int32_t* positions;
  const int32_t* slot_mapping;
  const float* cos_sin;
  int64_t cs_row, max_pos;
  const float *k_scale, *v_scale;   // e4m3 caches only
  uint8_t *k_cache, *v_cache;
  int64_t page_pitch, slot_pitch, head_pitch;   // bytes, both caches
  int log2_page;
  int64_t n_slots;
  int64_t n_tok;
  int Hq, Hk;
  int half_rot;                     // R / 2
  int neox;
  int* err;
};

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Eight fp32 values divided by s, to eight e4m3 codes.
__device__ __forceinline__ uint2 quantise8(const float* x, float s) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    c[i] = f32x2_to_e4m3x2(__fdiv_rn(x[2 * i + 1], s), __fdiv_rn(x[2 * i], s));
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
__device__ __forceinline__ uint4 round8(const float* x) {
  return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

template <int D, bool kFp8>
__global__ void __launch_bounds__(kThreads) gqa_rope_append_kernel(const RopeAppendParams p) {
  constexpr int kPieces = D / 16;
  const int rows = p.Hq + 2 * p.Hk;
  const uint32_t per_tok = static_cast<uint32_t>(rows) * kPieces;
  // the block's first item by one 64-bit division, the thread's by a 32-bit one
  const int64_t base = static_cast<int64_t>(blockIdx.x) * kThreads;
  const int64_t t0 = base / per_tok;
  const uint32_t local = static_cast<uint32_t>(base - t0 * per_tok) + threadIdx.x;
  const int64_t t = t0 + local / per_tok;
  if (t >= p.n_tok) return;
  const uint32_t item = local % per_tok;
  const int row = static_cast<int>(item / kPieces);
  const int piece = static_cast<int>(item % kPieces);
  const bool is_q = row < p.Hq;
  const bool is_k = !is_q && row < p.Hq + p.Hk;
  const int h = is_q ? row : (is_k ? row - p.Hq : row - p.Hq - p.Hk);

  // columns of the item's two 16-byte words
  const bool rot = (is_q || is_k) && piece * 8 < p.half_rot;
  const bool halves = rot && p.neox;
  const int c0 = halves ? 8 * piece : 16 * piece;
  const int c1 = halves ? p.half_rot + 8 * piece : 16 * piece + 8;
  const uint16_t* src = is_q ? p.q + t * p.q_tok + h * p.q_head
                             : (is_k ? p.k + t * p.k_tok + h * p.k_head
                                     : p.v + t * p.v_tok + h * p.v_head);
  // loads that depend on no other first
  const uint4 a = *reinterpret_cast<const uint4*>(src + c0);
  const uint4 b = *reinterpret_cast<const uint4*>(src + c1);
  const int32_t slot = is_q ? -1 : __ldg(p.slot_mapping + t);
  float scale = 1.f;
  if (kFp8 && !is_q) scale = __ldg(is_k ? p.k_scale : p.v_scale);

  float x[8], y[8];   // the results for c0 .. c0+7 and c1 .. c1+7
  {
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = lo_f32(wa[i]);
      x[2 * i + 1] = hi_f32(wa[i]);
      y[2 * i] = lo_f32(wb[i]);
      y[2 * i + 1] = hi_f32(wb[i]);
    }
  }
  if (rot) {
    const int32_t pos = __ldg(p.positions + t);
    if (pos < 0 || pos >= p.max_pos) {
      if (row == 0 && piece == 0) atomicOr(p.err, kErrBadIndex);
      return;                       // the token's rotated columns stay unwritten
    }
    const float* cs = p.cos_sin + pos * p.cs_row + 8 * piece;
    float c[8], s[8];
    *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(cs));
    *reinterpret_cast<float4*>(c + 4) = __ldg(reinterpret_cast<const float4*>(cs + 4));
    *reinterpret_cast<float4*>(s) = __ldg(reinterpret_cast<const float4*>(cs + p.half_rot));
    *reinterpret_cast<float4*>(s + 4) = __ldg(reinterpret_cast<const float4*>(cs + p.half_rot + 4));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      // halves: the pair is (x[i], y[i]); interleaved: neighbours of one word
      float& u = halves ? x[i] : (i < 4 ? x[2 * (i & 3)] : y[2 * (i & 3)]);
      float& w = halves ? y[i] : (i < 4 ? x[2 * (i & 3) + 1] : y[2 * (i & 3) + 1]);
      const float u0 = u, w0 = w;
      u = __fsub_rn(__fmul_rn(u0, c[i]), __fmul_rn(w0, s[i]));
      w = __fadd_rn(__fmul_rn(w0, c[i]), __fmul_rn(u0, s[i]));
    }
  }
  // columns that pass through keep their bits in bf16
  const uint4 out0 = rot ? round8(x) : a, out1 = rot ? round8(y) : b;
  uint16_t* dst = nullptr;
  if (is_q) dst = p.q_out + t * p.qo_tok + h * p.qo_head;
  if (is_k && p.k_out) dst = p.k_out + t * p.ko_tok + h * p.ko_head;
  if (dst) {
    *reinterpret_cast<uint4*>(dst + c0) = out0;
    *reinterpret_cast<uint4*>(dst + c1) = out1;
  }
  if (is_q || slot < 0) return;
  if (slot >= p.n_slots) {
    if (is_k && h == 0 && piece == 0) atomicOr(p.err, kErrBadRowId);
    return;
  }
  uint8_t* entry = (is_k ? p.k_cache : p.v_cache) + (slot >> p.log2_page) * p.page_pitch +
                   (slot & ((1 << p.log2_page) - 1)) * p.slot_pitch + h * p.head_pitch;
  if (!kFp8) {
    *reinterpret_cast<uint4*>(entry + 2 * c0) = out0;
    *reinterpret_cast<uint4*>(entry + 2 * c1) = out1;
  } else {
    const uint2 e0 = quantise8(x, scale), e1 = quantise8(y, scale);
    if (halves) {
      *reinterpret_cast<uint2*>(entry + c0) = e0;
      *reinterpret_cast<uint2*>(entry + c1) = e1;
    } else {
      *reinterpret_cast<uint4*>(entry + c0) = make_uint4(e0.x, e0.y, e1.x, e1.y);
    }
  }
}

}  // namespace

extern "C" int mla_gqa_rope_and_cache(
    const mla_tensor_t* q, const mla_tensor_t* k, const mla_tensor_t* v,
    const mla_tensor_t* positions, const mla_tensor_t* cos_sin, int32_t is_neox,
    const mla_tensor_t* slot_mapping, const mla_tensor_t* k_scale, const mla_tensor_t* v_scale,
    const mla_tensor_t* q_out, const mla_tensor_t* k_out, const mla_tensor_t* k_cache,
    const mla_tensor_t* v_cache, int32_t* error_word, mla_stream_t stream_) {
  if (!q || !k || q->ndim != 3 || k->ndim != 3) return MLA_ERR_INVALID_ARG;
  const int64_t T = q->shape[0], Hq = q->shape[1], Hk = k->shape[1], D = q->shape[2];
  if (T < 0 || Hq < 1 || Hk < 1 || Hq > 1024 || Hq % Hk != 0) return MLA_ERR_INVALID_ARG;
  if (!gqa_check_bf16(q, T, Hq, D, 8) || !gqa_check_bf16(k, T, Hk, D, 8) ||
      !gqa_check_bf16(v, T, Hk, D, 8) || !gqa_check_bf16(q_out, T, Hq, D, 8) ||
      (k_out && !gqa_check_bf16(k_out, T, Hk, D, 8)))
    return MLA_ERR_INVALID_ARG;
  if (!gqa_check_i32(positions, T) || !gqa_check_i32(slot_mapping, T)) return MLA_ERR_INVALID_ARG;
  if (is_neox != 0 && is_neox != 1) return MLA_ERR_INVALID_ARG;
  if (!cos_sin || !cos_sin->ptr || cos_sin->dtype != MLA_DTYPE_FP32 || cos_sin->ndim != 2 ||
      cos_sin->shape[0] < 1 || cos_sin->stride[1] != 1 || !gqa_aligned(cos_sin->ptr, 16))
    return MLA_ERR_INVALID_ARG;
  const int64_t R = cos_sin->shape[1];
  if (R < 16 || R % 16 != 0 || R > D) return MLA_ERR_INVALID_ARG;
  if (cos_sin->shape[0] > 1 && (cos_sin->stride[0] < R || cos_sin->stride[0] % 4 != 0))
    return MLA_ERR_INVALID_ARG;
  GqaCache c;
  const int st = gqa_check_cache(k_cache, v_cache, k_scale, v_scale, Hk, D, &c);
  if (st != MLA_OK) return st;
  if (!error_word) return MLA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return MLA_ERR_UNSUPPORTED;
  if (T == 0) return MLA_OK;

  RopeAppendParams p;
  p.q = static_cast<const uint16_t*>(q->ptr);
  p.k = static_cast<const uint16_t*>(k->ptr);
  p.v = static_cast<const uint16_t*>(v->ptr);
  p.q_tok = q->stride[0];
  p.q_head = q->stride[1];
  p.k_tok = k->stride[0];
  p.k_head = k->stride[1];
  p.v_tok = v->stride[0];
  p.v_head = v->stride[1];
  p.q_out = static_cast<uint16_t*>(q_out->ptr);
  p.qo_tok = q_out->stride[0];
  p.qo_head = q_out->stride[1];
  p.k_out = k_out ? static_cast<uint16_t*>(k_out->ptr) : nullptr;
  p.ko_tok = k_out ? k_out->stride[0] : 0;
  p.ko_head = k_out ? k_out->stride[1] : 0;
  p.positions = static_cast<const int32_t*>(positions->ptr);
  p.slot_mapping = static_cast<const int32_t*>(slot_mapping->ptr);
  p.cos_sin = static_cast<const float*>(cos_sin->ptr);
  p.cs_row = cos_sin->shape[0] > 1 ? cos_sin->stride[0] : R;
  p.max_pos = cos_sin->shape[0];
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
  p.k_cache = c.k;
  p.v_cache = c.v;
  p.page_pitch = c.page_pitch;
  p.slot_pitch = c.slot_pitch;
  p.head_pitch = c.head_pitch;
  p.log2_page = c.log2_page;
  p.n_slots = c.n_pages << c.log2_page;
  p.n_tok = T;
  p.Hq = static_cast<int>(Hq);
  p.Hk = static_cast<int>(Hk);
  p.half_rot = static_cast<int>(R / 2);
  p.neox = is_neox;
  p.err = error_word;

  const int64_t items = T * (Hq + 2 * Hk) * (D / 16);
  const int64_t blocks = (items + kThreads - 1) / kThreads;
  if (blocks > 0x7FFFFFFF) return MLA_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(blocks);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  if (D == 64) {
    if (c.fp8) gqa_rope_append_kernel<64, true><<<grid, kThreads, 0, s>>>(p);
    else gqa_rope_append_kernel<64, false><<<grid, kThreads, 0, s>>>(p);
  } else {
    if (c.fp8) gqa_rope_append_kernel<128, true><<<grid, kThreads, 0, s>>>(p);
    else gqa_rope_append_kernel<128, false><<<grid, kThreads, 0, s>>>(p);
  }
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
