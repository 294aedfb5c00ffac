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
// Bytes bound (3 flops an element).  An item is two 8-column words of a row, half a region's
// width apart (the region of rotated columns or the rest), so that eight lanes read and write
// whole 128-byte lines; with the pairs (i, i + R/2) the two words are each other's partners,
// with (2i, 2i+1) each holds its own pairs.  In large calls a thread takes the item of kStrip
// heads: the item's 8 cosines and sines are read once for them and their loads are in flight
// together.  Arithmetic is the definition's in fp32, every product, sum and quotient rounded
// on its own, and one rounding to the stored type (a bf16 value is off by at most 2^-8 of
// itself, an e4m3 code by 2^-4), so the bytes are exact.  Blocks go from token to token, the
// next token's position and slot read a token ahead, its words sent for from DRAM.
//
// Measured (one GB300): 16,384 tokens, 32/8 heads of 128, e4m3 cache and rotated keys kept,
// 411 MB: 70 us, 5.9 TB/s (0.86 of the copy rate; latency: 96 registers leave 18 warps a SM;
// four heads a thread 80); 64 tokens, 16/2 heads: 2 us in a CUDA graph (a call's host side is 10).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/paged_mla.h"
#include "mla_gqa_check.h"
#include "ptx.cuh"

namespace {

using namespace pmla;

constexpr int kStripHeads = 2;

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
  int* err;
};

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// Two fp32 values in a register pair and the packed operations on them.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(x));
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Quotients by one scale.  Markstein's theorem (1990): with r = 1/s correctly rounded, q = x r
// and e = x - q s (exact in one fused operation), q + e r rounds to the correctly rounded
// quotient, where nothing over- or underflows.  Scales between 2^-40 and 2^40 keep e normal
// for every x whose code is not zero; beyond +-1024 the code is saturated whatever the
// quotient, so q stops there.  Other scales divide.
struct Divisor {
  float s, r;
  bool plain;
  __device__ __forceinline__ void divide(float& x, float& y) const {
    if (plain) {
      x = __fdiv_rn(x, s);
      y = __fdiv_rn(y, s);
      return;
    }
    const uint64_t v = pair(x, y), rr = pair(r, r);
    float a, b;
    unpair(mul2(v, rr), &a, &b);
    a = fminf(fmaxf(a, -1024.f), 1024.f);
    b = fminf(fmaxf(b, -1024.f), 1024.f);
    const uint64_t q = pair(a, b);
    unpair(fma2(fma2(q, pair(-s, -s), v), rr, q), &x, &y);
  }
};
__device__ __forceinline__ Divisor make_divisor(float scale) {
  Divisor d;
  d.s = scale;
  d.r = __fdiv_rn(1.f, scale);
  d.plain = !(fabsf(scale) >= 0x1p-40f && fabsf(scale) <= 0x1p40f);
  return d;
}
// Eight fp32 values divided by the scale, to eight e4m3 codes.
__device__ __forceinline__ uint2 quantise8(const float* x, const Divisor& d) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a = x[2 * i], b = x[2 * i + 1];
    d.divide(a, b);
    c[i] = f32x2_to_e4m3x2(b, a);
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}
__device__ __forceinline__ uint4 round8(const float* x) {
  return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}

// Threads of a block, of which three fit a SM at least: 80 registers a thread, but 96 for e4m3
// strips (16,384 tokens, pairs (i, i + R/2): 72 us with 96, 77 with 80, 87 with the 106 that the
// compiler would take, which leave four warps a quarter of the SM instead of five).
constexpr int block_threads(bool fp8, int strip) { return fp8 && strip > 1 ? 192 : 256; }
template <int D, bool kFp8, bool kNeox, int kStrip>
__global__ void __launch_bounds__(block_threads(kFp8, kStrip), 3) gqa_rope_append_kernel(const RopeAppendParams p) {
  constexpr int kPieces = D / 16;
  // strips of heads a token: q, then k, then v; a thread keeps its item from token to token
  const int q_strips = (p.Hq + kStrip - 1) / kStrip, k_strips = (p.Hk + kStrip - 1) / kStrip;
  const int item = blockIdx.y * blockDim.x + threadIdx.x;
  const int strip = item / kPieces;
  const int piece = item % kPieces;
  if (strip >= q_strips + 2 * k_strips) return;
  const bool is_q = strip < q_strips;
  const bool is_k = !is_q && strip < q_strips + k_strips;
  const int h0 = (is_q ? strip : (is_k ? strip - q_strips : strip - q_strips - k_strips)) * kStrip;
  const int heads = is_q ? p.Hq : p.Hk;

  // columns of the item's words
  const bool rot = (is_q || is_k) && piece * 8 < p.half_rot;
  const int first = rot || !(is_q || is_k) ? 0 : 2 * p.half_rot;     // the region's first column
  const int half = rot ? p.half_rot : (D - first) / 2;
  const int c0 = first + 8 * (piece - first / 16);                   // the other: half further on
  const int64_t head = is_q ? p.q_head : (is_k ? p.k_head : p.v_head);
  const int64_t tok = is_q ? p.q_tok : (is_k ? p.k_tok : p.v_tok);
  const uint16_t* src0 = (is_q ? p.q : (is_k ? p.k : p.v)) + h0 * head + c0;
  const int64_t dst_head = is_q ? p.qo_head : p.ko_head, dst_tok = is_q ? p.qo_tok : p.ko_tok;
  uint16_t* dst0 = is_q ? p.q_out : (is_k ? p.k_out : nullptr);
  if (dst0) dst0 += h0 * dst_head + c0;
  uint8_t* cache = (is_k ? p.k_cache : p.v_cache) + h0 * p.head_pitch + c0 * (kFp8 ? 1 : 2);
  Divisor div = {};
  if (kFp8 && !is_q) div = make_divisor(__ldg(is_k ? p.k_scale : p.v_scale));

  int64_t t = blockIdx.x;
  int32_t pos = rot ? __ldg(p.positions + t) : 0, slot = is_q ? -1 : __ldg(p.slot_mapping + t);
  while (true) {
    // loads that depend on no other first: the item's words, its angles, and the next token's
    // position and slot
    uint4 a[kStrip], b[kStrip];
    const uint16_t* src = src0 + t * tok;
#pragma unroll
    for (int i = 0; i < kStrip; ++i)
      if (h0 + i < heads) {
        a[i] = *reinterpret_cast<const uint4*>(src + i * head);
        b[i] = *reinterpret_cast<const uint4*>(src + i * head + half);
      }
    float c[8], s[8];
    const bool known = pos >= 0 && pos < p.max_pos;
    if (rot && known) {
      // the angles of the first word's pairs and of the second's (halves: one set of eight)
      const float* cs = p.cos_sin + pos * p.cs_row;
      const int i0 = kNeox ? 8 * piece : 4 * piece, i1 = kNeox ? i0 + 4 : i0 + p.half_rot / 2;
      *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(cs + i0));
      *reinterpret_cast<float4*>(c + 4) = __ldg(reinterpret_cast<const float4*>(cs + i1));
      *reinterpret_cast<float4*>(s) = __ldg(reinterpret_cast<const float4*>(cs + p.half_rot + i0));
      *reinterpret_cast<float4*>(s + 4) = __ldg(reinterpret_cast<const float4*>(cs + p.half_rot + i1));
    }
    const int64_t t_next = t + gridDim.x;
    int32_t pos_next = 0, slot_next = -1;
    if (t_next < p.n_tok) {
      if (rot) pos_next = __ldg(p.positions + t_next);
      if (!is_q) slot_next = __ldg(p.slot_mapping + t_next);
    }
    // the next token's words into L2 meanwhile: they cost no registers there (16,384 tokens,
    // e4m3: 76 us with, 87 without; two tokens ahead 78, ahead of this token's loads 98)
    if (t_next < p.n_tok) {
      const uint16_t* next = src0 + t_next * tok;
#pragma unroll
      for (int i = 0; i < kStrip; ++i)
        if (h0 + i < heads) {
          asm volatile("prefetch.global.L2 [%0];" ::"l"(next + i * head));
          asm volatile("prefetch.global.L2 [%0];" ::"l"(next + i * head + half));
        }
    }
    const bool bad_slot = slot >= p.n_slots;
    if (bad_slot && is_k && h0 == 0 && piece == 0) atomicOr(p.err, kErrBadRowId);
    if (!known && strip == 0 && piece == 0) atomicOr(p.err, kErrBadIndex);
    uint8_t* entry = nullptr;
    if (slot >= 0 && !bad_slot)
      entry = cache + (slot >> p.log2_page) * p.page_pitch + (slot & ((1 << p.log2_page) - 1)) * p.slot_pitch;
    uint16_t* dst = dst0 ? dst0 + t * dst_tok : nullptr;

    if (known)                                     // else the token's rotated columns stay unwritten
#pragma unroll
    for (int i = 0; i < kStrip; ++i) {
      if (h0 + i >= heads) break;
      float x[8], y[8];   // the results for c0 .. c0+7 and c1 .. c1+7
      {
        const uint32_t wa[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, wb[4] = {b[i].x, b[i].y, b[i].z, b[i].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[2 * k] = lo_f32(wa[k]);
          x[2 * k + 1] = hi_f32(wa[k]);
          y[2 * k] = lo_f32(wb[k]);
          y[2 * k + 1] = hi_f32(wb[k]);
        }
      }
      if (rot) {
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          // two pairs (u, w) at once; halves: u in x, w in y; interleaved: neighbours
          float& u0 = kNeox ? x[k] : (k < 4 ? x[2 * k] : y[2 * k - 8]);
          float& w0 = kNeox ? y[k] : (k < 4 ? x[2 * k + 1] : y[2 * k - 7]);
          float& u1 = kNeox ? x[k + 1] : (k < 4 ? x[2 * k + 2] : y[2 * k - 6]);
          float& w1 = kNeox ? y[k + 1] : (k < 4 ? x[2 * k + 3] : y[2 * k - 5]);
          const uint64_t u = pair(u0, u1), w = pair(w0, w1);
          const uint64_t cc = pair(c[k], c[k + 1]), ss = pair(s[k], s[k + 1]), ms = pair(-s[k], -s[k + 1]);
          // (the sums are scalar: a packed sum of packed products comes out fused, its products
          // unrounded)
          float a0, a1, b0, b1;
          unpair(mul2(u, cc), &a0, &a1);
          unpair(mul2(w, ms), &b0, &b1);
          u0 = __fadd_rn(a0, b0);
          u1 = __fadd_rn(a1, b1);
          unpair(mul2(w, cc), &a0, &a1);
          unpair(mul2(u, ss), &b0, &b1);
          w0 = __fadd_rn(a0, b0);
          w1 = __fadd_rn(a1, b1);
        }
      }
      // columns that pass through keep their bits in bf16
      const uint4 out0 = rot ? round8(x) : a[i], out1 = rot ? round8(y) : b[i];
      if (dst) {
        *reinterpret_cast<uint4*>(dst + i * dst_head) = out0;
        *reinterpret_cast<uint4*>(dst + i * dst_head + half) = out1;
      }
      if (!entry) continue;
      uint8_t* at = entry + i * p.head_pitch;
      if (!kFp8) {
        *reinterpret_cast<uint4*>(at) = out0;
        *reinterpret_cast<uint4*>(at + 2 * half) = out1;
      } else {
        *reinterpret_cast<uint2*>(at) = quantise8(x, div);
        *reinterpret_cast<uint2*>(at + half) = quantise8(y, div);
      }
    }
    if (t_next >= p.n_tok) break;
    t = t_next;
    pos = pos_next;
    slot = slot_next;
  }
}

template <int D, bool kFp8, bool kNeox>
int launch(const RopeAppendParams& p, int sms, cudaStream_t s) {
  const int64_t rows = p.n_tok * (p.Hq + 2 * p.Hk);
  // strips pay once there are items for several full waves of threads
  const bool strips = rows * (D / 16) >= static_cast<int64_t>(sms) * 2048 * 4;
  const int n = strips ? kStripHeads : 1;
  const int items = ((p.Hq + n - 1) / n + 2 * ((p.Hk + n - 1) / n)) * (D / 16);
  const int most = block_threads(kFp8, n);
  const int threads = items < most ? (items + 31) / 32 * 32 : most;
  const unsigned parts = (items + threads - 1) / threads;
  // whole waves of the blocks that are resident at a time, each going from token to token: one in
  // small calls (4,089 tokens, 25/5 heads of 64, e4m3: 11 us, two 12, broken waves 14); three of
  // strips, whose ends come at different times (16,384 tokens, 64/8 heads, e4m3: 121 us, two 126,
  // one 145; bf16 117, two 117, one 130)
  const int resident = (kFp8 && strips ? 20 : 24) / (threads / 32);      // warps a SM by registers
  int64_t blocks = static_cast<int64_t>(sms) * resident * (strips ? 3 : 1) / parts;
  if (blocks > p.n_tok || blocks < 1) blocks = blocks < 1 ? 1 : p.n_tok;
  const dim3 grid(static_cast<unsigned>(blocks), parts);
  if (strips) gqa_rope_append_kernel<D, kFp8, kNeox, kStripHeads><<<grid, threads, 0, s>>>(p);
  else gqa_rope_append_kernel<D, kFp8, kNeox, 1><<<grid, threads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

template <int D>
int launch(const RopeAppendParams& p, bool fp8, bool neox, int sms, cudaStream_t s) {
  if (fp8) return neox ? launch<D, true, true>(p, sms, s) : launch<D, true, false>(p, sms, s);
  return neox ? launch<D, false, true>(p, sms, s) : launch<D, false, false>(p, sms, s);
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
  if (!gqa_rows_apart(q_out) || (k_out && !gqa_rows_apart(k_out))) return MLA_ERR_INVALID_ARG;
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
  p.err = error_word;

  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  return D == 64 ? launch<64>(p, c.fp8, is_neox, sms, s) : launch<128>(p, c.fp8, is_neox, sms, s);
}
