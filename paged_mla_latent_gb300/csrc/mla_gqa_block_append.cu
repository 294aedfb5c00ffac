// mla_gqa_block_append: a step's new keys and values into a paged e4m3 cache with a scale for
// each block of positions and head, its queries and keys rotated on the way.
//
//   rot as in mla_gqa_rope_and_cache.  For a block (BS positions, one head) with new values x:
//   a = max |x| (finite ones), s(a) = the smallest power of two with a <= 448 s, 2^-60 at least;
//   scale' = s(a) where the block starts in this call, max(scale, s(a)) where earlier calls left
//   values in it; codes e(x / scale'), and e(code scale / scale') of the earlier ones where the
//   scale grew.  Powers of two cost no precision (e4m3 has three bits whatever the scale) and
//   make quotients and the earlier codes' growth exact but for e4m3's subnormals.
//
// Bytes bound.  A unit is a block (32 positions of smaller ones; 16,384 tokens of 32/8 heads in
// blocks of 16: 76 us, 90 before with 16, chunks as below 15, 17 and with 64 19) of up to 256 columns' threads of
// heads' keys or values: eight (or four) threads a row of a head, each with two 8-column words half
// a region apart (the rotated columns or the rest), which with pairs (i, i + R/2) are each other's
// partners.  The rows are read twice, for the maxima and, from L2, for the codes: kept in registers
// or shared memory between, they cost more occupancy than the second reading costs (16,384
// tokens, 8 heads of 128, keys and values alone: 61 us with a warp's 16 rows in registers, 55
// so).  Units are found without a scan: request b's start at qo_indptr[b] / unit + 2 b (each
// has at most T_b / unit + 2), and the slots between stay idle.  Queries are turned by blocks of
// the same launch, a warp four (or eight) tokens and up to four heads.
//
// Measured (one GB300, in a CUDA graph): 16,384 tokens, 32/8 heads of 128, blocks of 64, rotated
// keys kept, 411 MB: 74 us, 5.5 TB/s (0.83 of the copy rate; with keys and values before the
// queries 77, so with units of 8 heads 82, of 2 83, without the L2 prefetch 78); 37 requests of 1 to
// 700 tokens, 25/5 heads of 64, 49 MB: 15 us; one token of 64 requests, 16/2 heads: 5 us, a chain of
// request, lists, page, scale and words.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/paged_mla.h"
#include "mla_gqa_check.h"
#include "mla_gqa_pages.cuh"
#include "ptx.cuh"

namespace {

using namespace pmla;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kLog2Unit = 5, kUnit = 1 << kLog2Unit;         // positions of a unit, where blocks have fewer

struct BlockAppendParams {
  const uint16_t *q, *k, *v;                // bf16 bits
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;   // strides in elements
  uint16_t *q_out, *k_out;                  // k_out may be null
  int64_t qo_tok, qo_head, ko_tok, ko_head;
  const int32_t* positions;
  const float* cos_sin;
  int64_t cs_row, max_pos;
  const int32_t* qo_indptr;
  PageList pages;
  int64_t n_pages;
  uint8_t *k_cache, *v_cache;
  int64_t page_pitch, slot_pitch, head_pitch;   // bytes, both caches
  float *ks, *vs;
  int64_t sc_page, sc_block, sc_head;       // elements, both
  int log2_block;
  int64_t n_tok;
  int B, Hq, Hk;
  int half_rot;                             // R / 2
  int part_heads, parts;                    // heads a unit takes; units of a block's keys and values
  unsigned kv_ctas, q_ctas;                 // then some blocks that look the lists over
  unsigned every;                           // of them one of so many is for keys and values, until those are out
  int strip;                                // query heads a warp takes
  int* err;
};

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ uint4 round8(const float* x) {
  return make_uint4(bf16x2(x[0], x[1]), bf16x2(x[2], x[3]), bf16x2(x[4], x[5]), bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void widen8(const uint4& w, float* x) {
  const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = lo_f32(v[i]);
    x[2 * i + 1] = hi_f32(v[i]);
  }
}

// Two fp32 values in a register pair, and their products.
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

// A lane's columns of a row: two words of eight.
struct Columns {
  bool rot;
  int c0, half, piece;
};
template <int D>
__device__ __forceinline__ Columns columns_of(int piece, bool turned, int half_rot) {
  Columns c;
  c.piece = piece;
  c.rot = turned && piece * 8 < half_rot;
  const int first = c.rot || !turned ? 0 : 2 * half_rot;       // the region's first column
  c.half = c.rot ? half_rot : (D - first) / 2;
  c.c0 = first + 8 * (piece - first / 16);
  return c;
}

struct Angles {
  float c[8], s[8];
};
template <bool kNeox>
__device__ __forceinline__ void load_angles(const BlockAppendParams& p, int64_t pos, int piece, Angles* a) {
  // the angles of the first word's pairs and of the second's (halves: one set of eight)
  const float* cs = p.cos_sin + pos * p.cs_row;
  const int i0 = kNeox ? 8 * piece : 4 * piece, i1 = kNeox ? i0 + 4 : i0 + p.half_rot / 2;
  *reinterpret_cast<float4*>(a->c) = __ldg(reinterpret_cast<const float4*>(cs + i0));
  *reinterpret_cast<float4*>(a->c + 4) = __ldg(reinterpret_cast<const float4*>(cs + i1));
  *reinterpret_cast<float4*>(a->s) = __ldg(reinterpret_cast<const float4*>(cs + p.half_rot + i0));
  *reinterpret_cast<float4*>(a->s + 4) = __ldg(reinterpret_cast<const float4*>(cs + p.half_rot + i1));
}
// Sixteen values with their pairs turned, every operation rounded on its own.
template <bool kNeox>
__device__ __forceinline__ void turn(float* x, const Angles& a) {
  float* y = x + 8;
#pragma unroll
  for (int k = 0; k < 8; k += 2) {          // two pairs at once; the sums are scalar: packed ones
    float& u0 = kNeox ? x[k] : (k < 4 ? x[2 * k] : y[2 * k - 8]);        // come out fused with the products
    float& w0 = kNeox ? y[k] : (k < 4 ? x[2 * k + 1] : y[2 * k - 7]);
    float& u1 = kNeox ? x[k + 1] : (k < 4 ? x[2 * k + 2] : y[2 * k - 6]);
    float& w1 = kNeox ? y[k + 1] : (k < 4 ? x[2 * k + 3] : y[2 * k - 5]);
    const uint64_t u = pair(u0, u1), w = pair(w0, w1);
    const uint64_t cc = pair(a.c[k], a.c[k + 1]), ss = pair(a.s[k], a.s[k + 1]);
    float a0, a1, b0, b1;
    unpair(mul2(u, cc), &a0, &a1);
    unpair(mul2(w, ss), &b0, &b1);
    u0 = __fsub_rn(a0, b0);
    u1 = __fsub_rn(a1, b1);
    unpair(mul2(w, cc), &a0, &a1);
    unpair(mul2(u, ss), &b0, &b1);
    w0 = __fadd_rn(a0, b0);
    w1 = __fadd_rn(a1, b1);
  }
}

// The smallest power of two s with a <= 448 s = 1.75 2^8 s, between 2^-60 and 2^120.
__device__ __forceinline__ float power_for(float a) {
  const uint32_t bits = __float_as_uint(a);
  int k = static_cast<int>(bits >> 23) - (127 + 8) + ((bits & 0x7FFFFFu) > 0x600000u);
  k = k < -60 ? -60 : (k > 120 ? 120 : k);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

__device__ __noinline__ float quotient(float x, float scale) { return __fdiv_rn(x, scale); }
// Eight values over a scale as codes: the scale is nearly always a power of two with a normal
// reciprocal (r, else 0), which is exact; others divide, out of the way.
__device__ __forceinline__ float exact_reciprocal(float scale) {
  const uint32_t bits = __float_as_uint(scale);
  const bool exact = (bits & 0x7FFFFFu) == 0 && bits >= (64u << 23) && bits <= (252u << 23);
  return exact ? __uint_as_float((254u << 23) - bits) : 0.f;
}
__device__ __forceinline__ uint2 quantise8(const float* x, float scale, float r) {
  uint32_t c[4];
  if (r != 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b;
      unpair(mul2(pair(x[2 * i], x[2 * i + 1]), pair(r, r)), &a, &b);
      c[i] = f32x2_to_e4m3x2(b, a);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = f32x2_to_e4m3x2(quotient(x[2 * i + 1], scale), quotient(x[2 * i], scale));
  }
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

struct Request {
  int64_t t0;                               // its first new token
  int tokens, held;
  bool sound;
};
__device__ __forceinline__ Request request_of(const BlockAppendParams& p, int b) {
  const int64_t t0 = __ldg(p.qo_indptr + b), t1 = __ldg(p.qo_indptr + b + 1);
  const int held = p.pages.positions(b);
  return {t0, static_cast<int>(t1 - t0), held, t0 >= 0 && t1 >= t0 && t1 <= p.n_tok && held >= t1 - t0};
}

// The first of a request's slots, where its units are.
__device__ __forceinline__ int64_t first_slot(const BlockAppendParams& p, int b, int log2_unit) {
  return static_cast<int64_t>(__ldg(p.qo_indptr + b) >> log2_unit) + 2 * static_cast<int64_t>(b);
}
// The unit of request b that a slot stands for, the g0-th of the request's positions; no tokens where it is none.
struct Unit {
  Request r;
  int64_t g0;
  int b;
  bool sure;                                // that it is no other request's
};
__device__ __forceinline__ Unit unit_of(const BlockAppendParams& p, int b, int64_t slot, int log2_unit) {
  Unit u = {request_of(p, b), 0, b, false};
  const int64_t nth = slot - first_slot(p, b, log2_unit), t1 = u.r.t0 + u.r.tokens;
  u.g0 = ((u.r.held - u.r.tokens) >> log2_unit) + nth;
  u.sure = nth >= 0 && u.r.t0 >= 0 && u.r.tokens >= 0 && t1 <= p.n_tok &&
           (b + 1 == p.B || slot < (t1 >> log2_unit) + 2 * static_cast<int64_t>(b + 1));
  if (!u.r.sound || nth < 0 || u.g0 << log2_unit >= u.r.held) u.r.tokens = 0;
  return u;
}
// Entries of the token list that lie outside the call lead a search astray: past them, then.
__device__ __noinline__ int owner_beside_bad_lists(const BlockAppendParams& p, int lane, int64_t slot, int log2_unit) {
  return warp_owner<true>(p.B, lane, slot, [&](int b) -> int64_t {
    const int t = __ldg(p.qo_indptr + b);
    return t < 0 || t > p.n_tok ? -1 : first_slot(p, b, log2_unit);
  });
}

// Queries: a warp takes 32 / (D/16) tokens and a strip of up to 4 heads, whose words are all in
// flight before the angles, which wait for the positions.
constexpr int kMostStrip = 4;
template <int D, bool kNeox>
__device__ __forceinline__ void turn_queries(const BlockAppendParams& p, int64_t item, int lane) {
  constexpr int kPieces = D / 16, kRows = 32 / kPieces;
  const int strips = (p.Hq + p.strip - 1) / p.strip;
  const int64_t group = item / strips;
  const int h0 = static_cast<int>(item - group * strips) * p.strip;
  const int64_t t = group * kRows + lane / kPieces;
  if (t >= p.n_tok) return;
  int64_t live = __ldg(p.qo_indptr + p.B);
  if (live < 0) live = p.n_tok;             // an end that makes no sense
  const int64_t pos = __ldg(p.positions + t);
  const Columns c = columns_of<D>(lane % kPieces, true, p.half_rot);
  const int h1 = h0 + p.strip < p.Hq ? h0 + p.strip : p.Hq;
  const uint16_t* src = p.q + t * p.q_tok + h0 * p.q_head + c.c0;
  uint4 w[kMostStrip][2];
#pragma unroll
  for (int i = 0; i < kMostStrip; ++i)
    if (h0 + i < h1) {
      w[i][0] = *reinterpret_cast<const uint4*>(src + i * p.q_head);
      w[i][1] = *reinterpret_cast<const uint4*>(src + i * p.q_head + c.half);
    }
  if (t >= live) return;
  Angles a;
  const bool known = pos >= 0 && pos < p.max_pos;
  if (!known && h0 == 0 && c.piece == 0) atomicOr(p.err, kErrBadIndex);
  if (c.rot && !known) return;              // the token's rotated columns stay unwritten
  if (c.rot) load_angles<kNeox>(p, pos, c.piece, &a);
  uint16_t* dst = p.q_out + t * p.qo_tok + h0 * p.qo_head + c.c0;
#pragma unroll
  for (int i = 0; i < kMostStrip; ++i)
    if (h0 + i < h1) {
      if (c.rot) {
        float x[16];
        widen8(w[i][0], x);
        widen8(w[i][1], x + 8);
        turn<kNeox>(x, a);
        w[i][0] = round8(x);
        w[i][1] = round8(x + 8);
      }
      *reinterpret_cast<uint4*>(dst + i * p.qo_head) = w[i][0];
      *reinterpret_cast<uint4*>(dst + i * p.qo_head + c.half) = w[i][1];
    }
}

template <int D, bool kNeox>
__global__ void __launch_bounds__(kThreads, 3) gqa_block_append_kernel(const BlockAppendParams p) {
  constexpr int kPieces = D / 16;           // threads a row of a head
  constexpr int kMostHeads = kThreads / kPieces;
  __shared__ uint32_t s_top[kUnit][kMostHeads];          // largest |x| of each block and head, bits
  __shared__ float s_scale[kUnit][kMostHeads];
  __shared__ float s_ratio[kMostHeads];     // of the continued block's old scale to its new one
  __shared__ bool s_grew[kMostHeads];
  const int tid = threadIdx.x, lane = tid & 31;
  if (blockIdx.x >= p.kv_ctas + p.q_ctas) {
    const int64_t i = static_cast<int64_t>(blockIdx.x - p.kv_ctas - p.q_ctas) * kThreads + tid;
    if (i < p.B && !request_of(p, static_cast<int>(i)).sound) atomicOr(p.err, kErrBadIndptr);
    return;
  }
  const unsigned nth = blockIdx.x / p.every;
  if (nth >= p.kv_ctas || blockIdx.x != nth * p.every) {
    const unsigned before = nth + 1 < p.kv_ctas ? nth + 1 : p.kv_ctas;     // blocks for keys and values
    turn_queries<D, kNeox>(p, static_cast<int64_t>(blockIdx.x - before) * kWarps + (tid >> 5), lane);
    return;
  }
  // ---- the unit: a request, a block of positions (or 32 of smaller blocks), keys or values
  const int slot = nth / p.parts, part = nth - slot * p.parts;
  const bool is_k = (part & 1) == 0;
  const int first_head = (part >> 1) * p.part_heads;
  const int heads = p.Hk - first_head < p.part_heads ? p.Hk - first_head : p.part_heads;
  const int bs = 1 << p.log2_block;
  const int log2_unit = p.log2_block > kLog2Unit ? p.log2_block : kLog2Unit;
  Unit found = unit_of(p, warp_owner<false>(p.B, lane, slot, [&](int b) { return first_slot(p, b, log2_unit); }), slot, log2_unit);
  if (!found.r.tokens) {                    // an idle slot, or hidden by a bad list
    if (found.sure) return;
    found = unit_of(p, owner_beside_bad_lists(p, lane, slot, log2_unit), slot, log2_unit);
    if (!found.r.tokens) return;
  }
  const int b = found.b;
  const Request r = found.r;
  const int64_t t0 = r.t0, g0 = found.g0;
  const int held = r.held, begin = held - r.tokens;          // the first new position
  const int base = static_cast<int>(g0) << log2_unit, end = base + (1 << log2_unit);
  const int lo = begin > base ? begin : base, hi = held < end ? held : end;      // its new positions

  const int64_t idx0 = __ldg(p.pages.indptr + b);
  const int ps_mask = (1 << p.pages.log2_page) - 1;
  uint8_t* cache = is_k ? p.k_cache : p.v_cache;
  float* scales = is_k ? p.ks : p.vs;
  auto page_at = [&](int pos) -> int {      // -1: outside the cache
    const int page = __ldg(p.pages.indices + idx0 + (pos >> p.pages.log2_page));
    return page >= 0 && page < p.n_pages ? page : -1;
  };
  // a block and head a thread: where its scale is, and the scale where earlier positions have one
  const int n_scales = ((hi - 1 - base) / bs + 1) * heads;
  auto scale_of = [&](int i, bool* continued) -> float* {
    const int at = base + i / heads * bs;
    const int pos = at > lo ? at : lo;      // the block's first new position
    *continued = at < begin;
    if (pos >= hi || at + bs <= lo) return nullptr;
    const int page = page_at(pos);
    if (page < 0) return nullptr;
    return scales + page * p.sc_page + ((pos & ps_mask) >> p.log2_block) * p.sc_block + (first_head + i % heads) * p.sc_head;
  };
  for (int i = tid; i < n_scales; i += kThreads) s_top[i / heads][i % heads] = 0;
  if (tid < heads) s_grew[tid] = false;
  __syncthreads();

  // ---- the largest value of each block and head.  A thread has two words of eight columns of a
  // head; the block goes over the rows `at_once` at a time, a thread `kBatch` rows in flight.
  const int row_threads = heads * kPieces, at_once = kThreads / row_threads;
  const int tg = tid / row_threads, hl = tid / kPieces - tg * heads, piece = tid % kPieces;
  const int h = first_head + hl;
  const bool active = tg < at_once;
  const Columns col = columns_of<D>(piece, is_k, p.half_rot);
  const int64_t src_tok = is_k ? p.k_tok : p.v_tok;
  const uint16_t* src = (is_k ? p.k + h * p.k_head : p.v + h * p.v_head) + col.c0 + (t0 - begin) * src_tok;
  constexpr int kBatch = 2;
  const bool once = lo + at_once * kBatch >= hi;         // one batch: its words stay
  uint4 w[kBatch][2];
  int angle[kBatch];
  auto fetch = [&](int row0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = row0 + i * at_once;
      if (active && row < hi) {
        w[i][0] = *reinterpret_cast<const uint4*>(src + row * src_tok);
        w[i][1] = *reinterpret_cast<const uint4*>(src + row * src_tok + col.half);
        angle[i] = col.rot ? __ldg(p.positions + t0 + row - begin) : -1;
      } else {
        w[i][0] = w[i][1] = make_uint4(0, 0, 0, 0);
        angle[i] = -1;
      }
    }
  };
  // a rotary position outside the table: the row's rotated columns stay unwritten
  auto known = [&](int i) { return !col.rot || (angle[i] >= 0 && angle[i] < p.max_pos); };
  auto values = [&](int i, float* x) {
    widen8(w[i][0], x);
    widen8(w[i][1], x + 8);
    if (col.rot && known(i)) {
      Angles a;
      load_angles<kNeox>(p, angle[i], piece, &a);
      turn<kNeox>(x, a);
    }
  };
  float top = 0.f;
#pragma unroll 1
  for (int row0 = lo + tg; row0 - tg < hi; row0 += at_once * kBatch) {
    fetch(row0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = row0 + (kBatch + i) * at_once;
      if (active && row < hi) {             // the next batch's words into L2 meanwhile
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + row * src_tok));
        asm volatile("prefetch.global.L2 [%0];" ::"l"(src + row * src_tok + col.half));
      }
    }
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      float x[16], most = 0.f;
      values(i, x);
#pragma unroll
      for (int k = 0; k < 16; ++k) most = fmaxf(most, fabsf(x[k]));     // (passes a NaN over)
      if (most == INFINITY) {               // the largest that is finite
        most = 0.f;
#pragma unroll
        for (int k = 0; k < 16; ++k) most = fmaxf(most, fabsf(x[k]) < INFINITY ? fabsf(x[k]) : 0.f);
      }
      if (!known(i)) most = 0.f;
      if (bs >= kUnit) {
        top = fmaxf(top, most);
      } else if (most > 0.f) {
        atomicMax(&s_top[(row0 + i * at_once - base) >> p.log2_block][hl], __float_as_uint(most));
      }
    }
  }
  if (bs >= kUnit) {
#pragma unroll
    for (int d = 1; d < kPieces; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
    if (active && piece == 0 && top > 0.f) atomicMax(&s_top[0][hl], __float_as_uint(top));
  }
  __syncthreads();

  // ---- the scales
  for (int i = tid; i < n_scales; i += kThreads) {
    bool continued;
    float* at = scale_of(i, &continued);
    const float fit = power_for(__uint_as_float(s_top[i / heads][i % heads]));
    float scale = fit;
    if (at) {
      const float old = continued ? *at : 0.f;
      if (continued && old >= fit) {
        scale = old;
      } else if (continued && fit > old) {
        s_grew[i % heads] = true;
        s_ratio[i % heads] = __fdiv_rn(old, fit);
      }
      *at = scale;
    }
    s_scale[i / heads][i % heads] = scale;
  }
  __syncthreads();

  // ---- codes, and the rotated keys in bf16: the words once more (from L2), or still there
#pragma unroll 1
  for (int row0 = lo + tg; row0 - tg < hi; row0 += at_once * kBatch) {
    if (!once) fetch(row0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int row = row0 + i * at_once;
      if (!active || row >= hi) continue;
      const bool put = known(i);
      float x[16];
      values(i, x);
      if (is_k && p.k_out && put) {
        uint16_t* dst = p.k_out + (t0 + row - begin) * p.ko_tok + h * p.ko_head + col.c0;
        *reinterpret_cast<uint4*>(dst) = round8(x);
        *reinterpret_cast<uint4*>(dst + col.half) = round8(x + 8);
      }
      const int page = page_at(row);
      if (page < 0) {
        if (piece == 0) atomicOr(p.err, kErrBadRowId);
      } else if (!put) {
        if (piece == 0 && h == 0) atomicOr(p.err, kErrBadIndex);
      } else {
        uint8_t* dst = cache + page * p.page_pitch + (row & ps_mask) * p.slot_pitch + h * p.head_pitch + col.c0;
        const float scale = s_scale[bs >= kUnit ? 0 : (row - base) >> p.log2_block][hl], inv = exact_reciprocal(scale);
        *reinterpret_cast<uint2*>(dst) = quantise8(x, scale, inv);
        *reinterpret_cast<uint2*>(dst + col.half) = quantise8(x + 8, scale, inv);
      }
    }
  }

  // ---- earlier codes of the continued block, where its scale grew
  const int joined = begin & ~(bs - 1);      // its first position
  if (joined >= begin || joined < base || joined >= end || !active || !s_grew[hl]) return;
  const float ratio = s_ratio[hl];
  for (int row = joined + tg; row < begin; row += at_once) {
    const int page = page_at(row);
    if (page < 0) continue;
    uint4* at = reinterpret_cast<uint4*>(cache + page * p.page_pitch + (row & ps_mask) * p.slot_pitch + h * p.head_pitch + 16 * piece);
    uint4 codes = *at;
    uint32_t* c = reinterpret_cast<uint32_t*>(&codes);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo2 = e4m3x2_to_f16x2(c[i]), hi2 = e4m3x2_to_f16x2(c[i] >> 16);
      const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo2));
      const float2 e = __half22float2(*reinterpret_cast<const __half2*>(&hi2));
      const uint32_t low = f32x2_to_e4m3x2(a.y * ratio, a.x * ratio), high = f32x2_to_e4m3x2(e.y * ratio, e.x * ratio);
      c[i] = low | (high << 16);
    }
    *at = codes;
  }
}

template <int D, bool kNeox>
int launch(BlockAppendParams& p, int sms, cudaStream_t s) {
  constexpr int kRows = 32 / (D / 16);
  const int unit = p.log2_block > kLog2Unit ? p.log2_block : kLog2Unit;
  p.part_heads = 32 / (D / 16);            // a warp a row: 1 KB of neighbours in a token
  if (p.part_heads > p.Hk) p.part_heads = p.Hk;
  p.parts = 2 * ((p.Hk + p.part_heads - 1) / p.part_heads);
  const int64_t kv_ctas = ((p.n_tok >> unit) + 2 * static_cast<int64_t>(p.B)) * p.parts;
  // query heads a warp: the warps of one wave (24 a SM) take all of them where that is up to 4 each
  const int64_t groups = (p.n_tok + kRows - 1) / kRows;
  p.strip = 1;
  while (p.strip < kMostStrip && p.strip < p.Hq && groups * ((p.Hq + p.strip - 1) / p.strip) > static_cast<int64_t>(sms) * 24) p.strip *= 2;
  const int64_t q_items = groups * ((p.Hq + p.strip - 1) / p.strip);
  const int64_t q_ctas = (q_items + kWarps - 1) / kWarps;
  const int64_t look_ctas = (p.B + kThreads - 1) / kThreads;
  const int64_t ctas = kv_ctas + q_ctas + look_ctas;
  if (ctas > 0x7FFFFFFF) return MLA_ERR_UNSUPPORTED;
  p.kv_ctas = static_cast<unsigned>(kv_ctas);
  p.q_ctas = static_cast<unsigned>(q_ctas);
  // Keys and values, the longer chains, come first; where their units, without the slots between
  // requests, are more than two waves (three blocks a SM) every other block turns queries, which stream
  // while the others wait.  Units, us with keys and values first and in turns: prompts of one length
  // 512 41.3 and 41.0, 768 58.8 and 55.6, 1,024 77.2 and 73.7, 2,048 150 and 144; ragged chunks 334 15.2
  // and 17.6, 612 28.0 and 29.1, 852 33.5 and 34.2, 1,704 73.2 and 67.2.
  p.every = (p.n_tok >> unit) * p.parts > 6 * static_cast<int64_t>(sms) && q_ctas >= kv_ctas ? 2 : 1;
  gqa_block_append_kernel<D, kNeox><<<static_cast<unsigned>(ctas), kThreads, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}

}  // namespace

extern "C" int mla_gqa_block_append(
    const mla_tensor_t* q, const mla_tensor_t* k, const mla_tensor_t* v,
    const mla_tensor_t* positions, const mla_tensor_t* cos_sin, int32_t is_neox,
    const mla_tensor_t* qo_indptr, const mla_tensor_t* kv_indptr, const mla_tensor_t* kv_indices,
    const mla_tensor_t* kv_last_page_lens, const mla_tensor_t* q_out, const mla_tensor_t* k_out,
    const mla_tensor_t* k_cache, const mla_tensor_t* v_cache, const mla_tensor_t* k_scale,
    const mla_tensor_t* v_scale, int32_t* error_word, mla_stream_t stream_) {
  if (!q || !k || !qo_indptr || q->ndim != 3 || k->ndim != 3 || qo_indptr->ndim != 1) return MLA_ERR_INVALID_ARG;
  const int64_t T = q->shape[0], Hq = q->shape[1], Hk = k->shape[1], D = q->shape[2];
  const int64_t B = qo_indptr->shape[0] - 1;
  if (T < 0 || T > 0x7FFFFFFF || B < 0 || B > 0xFFFFFF || Hq < 1 || Hk < 1 || Hq > 1024 || Hq % Hk != 0)
    return MLA_ERR_INVALID_ARG;
  if (!gqa_check_bf16(q, T, Hq, D, 8) || !gqa_check_bf16(k, T, Hk, D, 8) ||
      !gqa_check_bf16(v, T, Hk, D, 8) || !gqa_check_bf16(q_out, T, Hq, D, 8) ||
      (k_out && !gqa_check_bf16(k_out, T, Hk, D, 8)))
    return MLA_ERR_INVALID_ARG;
  if (!gqa_rows_apart(q_out) || (k_out && !gqa_rows_apart(k_out))) return MLA_ERR_INVALID_ARG;
  if (!gqa_check_i32(positions, T) || !gqa_check_i32(qo_indptr, B + 1)) return MLA_ERR_INVALID_ARG;
  if (is_neox != 0 && is_neox != 1) return MLA_ERR_INVALID_ARG;
  if (!cos_sin || !cos_sin->ptr || cos_sin->dtype != MLA_DTYPE_FP32 || cos_sin->ndim != 2 ||
      cos_sin->shape[0] < 1 || cos_sin->stride[1] != 1 || !gqa_aligned(cos_sin->ptr, 16))
    return MLA_ERR_INVALID_ARG;
  const int64_t R = cos_sin->shape[1];
  if (R < 16 || R % 16 != 0 || R > D) return MLA_ERR_INVALID_ARG;
  if (cos_sin->shape[0] > 1 && (cos_sin->stride[0] < R || cos_sin->stride[0] % 4 != 0))
    return MLA_ERR_INVALID_ARG;
  GqaBlockCache c;
  const int st = gqa_check_block_cache(k_cache, v_cache, k_scale, v_scale, Hk, D, &c);
  if (st != MLA_OK) return st;
  if (!gqa_check_pages(kv_indptr, kv_indices, kv_last_page_lens, B, c.log2_page)) return MLA_ERR_INVALID_ARG;
  if (!error_word || !gqa_aligned(error_word, 4)) return MLA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return MLA_ERR_UNSUPPORTED;
  if (T == 0 || B == 0) return MLA_OK;

  BlockAppendParams p = {};
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
  p.cos_sin = static_cast<const float*>(cos_sin->ptr);
  p.cs_row = cos_sin->shape[0] > 1 ? cos_sin->stride[0] : R;
  p.max_pos = cos_sin->shape[0];
  p.qo_indptr = static_cast<const int32_t*>(qo_indptr->ptr);
  p.pages.indptr = static_cast<const int32_t*>(kv_indptr->ptr);
  p.pages.indices = static_cast<const int32_t*>(kv_indices->ptr);
  p.pages.last = kv_last_page_lens ? static_cast<const int32_t*>(kv_last_page_lens->ptr) : nullptr;
  p.pages.n_idx = kv_indices->shape[0];
  p.pages.log2_page = c.log2_page;
  p.n_pages = c.n_pages;
  p.k_cache = c.k;
  p.v_cache = c.v;
  p.page_pitch = c.page_pitch;
  p.slot_pitch = c.slot_pitch;
  p.head_pitch = c.head_pitch;
  p.ks = c.ks;
  p.vs = c.vs;
  p.sc_page = c.sc_page;
  p.sc_block = c.sc_block;
  p.sc_head = c.sc_head;
  p.log2_block = c.log2_block;
  p.n_tok = T;
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hk = static_cast<int>(Hk);
  p.half_rot = static_cast<int>(R / 2);
  p.err = error_word;

  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  if (D == 64) return is_neox ? launch<64, true>(p, sms, s) : launch<64, false>(p, sms, s);
  return is_neox ? launch<128, true>(p, sms, s) : launch<128, false>(p, sms, s);
}
