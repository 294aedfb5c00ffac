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
// Bytes bound.  A warp takes tiles of 16 positions of one head: eight (or four) lanes a row, a
// lane two 8-column words half a region apart (the rotated columns or the rest), which with
// pairs (i, i + R/2) are each other's partners.  A unit is a block (16 positions where blocks are
// smaller) of one head's keys or values; its rows stay in registers from the maximum to the
// codes.  Blocks of more than 16 positions have a warp a tile and meet in shared memory where
// requests bring many tokens; where they bring few, one warp walks the block's tiles with new
// rows.  Units are found without a scan: request b's start at qo_indptr[b] / 16m + 2 b (each has
// at most T_b / 16m + 2), and the slots between stay idle.
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
constexpr int kTile = 16;                   // positions a warp takes at a time

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
  int unit_warps;                           // warps of a unit: 1, or a block's tiles
  int kv_slots;                             // units of one head's keys
  unsigned kv_ctas, q_ctas;                 // then some that look the lists over
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
  for (int k = 0; k < 8; ++k) {
    float& u = kNeox ? x[k] : (k < 4 ? x[2 * k] : y[2 * k - 8]);
    float& w = kNeox ? y[k] : (k < 4 ? x[2 * k + 1] : y[2 * k - 7]);
    const float uc = __fmul_rn(u, a.c[k]), ws = __fmul_rn(w, a.s[k]);
    const float wc = __fmul_rn(w, a.c[k]), us = __fmul_rn(u, a.s[k]);
    u = __fsub_rn(uc, ws);
    w = __fadd_rn(wc, us);
  }
}

// The smallest power of two s with a <= 448 s = 1.75 2^8 s, between 2^-60 and 2^120.
__device__ __forceinline__ float power_for(float a) {
  const uint32_t bits = __float_as_uint(a);
  int k = static_cast<int>(bits >> 23) - (127 + 8) + ((bits & 0x7FFFFFu) > 0x600000u);
  k = k < -60 ? -60 : (k > 120 ? 120 : k);
  return __uint_as_float(static_cast<uint32_t>(k + 127) << 23);
}

// x / s; s is nearly always a power of two with a normal reciprocal.
struct Quotient {
  float s, r;
  bool exact;
  __device__ explicit Quotient(float scale) : s(scale) {
    const uint32_t bits = __float_as_uint(scale);
    exact = (bits & 0x7FFFFFu) == 0 && bits >= (64u << 23) && bits <= (252u << 23);
    r = __uint_as_float((254u << 23) - (exact ? bits : 127u << 23));
  }
  __device__ float operator()(float x) const { return exact ? x * r : __fdiv_rn(x, s); }
};
__device__ __forceinline__ uint2 quantise8(const float* x, const Quotient& d) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = f32x2_to_e4m3x2(d(x[2 * i + 1]), d(x[2 * i]));
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

// Queries: a warp takes 32 / (D/16) tokens and a strip of heads, whose angles it reads once.
template <int D, bool kNeox>
__device__ __forceinline__ void turn_queries(const BlockAppendParams& p, int64_t item, int lane) {
  constexpr int kPieces = D / 16, kRows = 32 / kPieces;
  const int strips = (p.Hq + p.strip - 1) / p.strip;
  const int64_t group = item / strips;
  const int h0 = static_cast<int>(item - group * strips) * p.strip;
  const int64_t t = group * kRows + lane / kPieces;
  const int64_t live = __ldg(p.qo_indptr + p.B);
  if (t >= p.n_tok || t >= live) return;
  const Columns c = columns_of<D>(lane % kPieces, true, p.half_rot);
  Angles a;
  const int64_t pos = __ldg(p.positions + t);
  const bool known = pos >= 0 && pos < p.max_pos;
  if (!known && h0 == 0 && c.piece == 0) atomicOr(p.err, kErrBadIndex);
  if (c.rot && !known) return;              // the token's rotated columns stay unwritten
  if (c.rot) load_angles<kNeox>(p, pos, c.piece, &a);
  const uint16_t* src = p.q + t * p.q_tok + c.c0;
  uint16_t* dst = p.q_out + t * p.qo_tok + c.c0;
  const int h1 = h0 + p.strip < p.Hq ? h0 + p.strip : p.Hq;
  constexpr int kAtOnce = 4;
  for (int h = h0; h < h1; h += kAtOnce) {
    uint4 w[kAtOnce][2];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (h + i < h1) {
        w[i][0] = *reinterpret_cast<const uint4*>(src + (h + i) * p.q_head);
        w[i][1] = *reinterpret_cast<const uint4*>(src + (h + i) * p.q_head + c.half);
      }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (h + i < h1) {
        if (c.rot) {
          float x[16];
          widen8(w[i][0], x);
          widen8(w[i][1], x + 8);
          turn<kNeox>(x, a);
          w[i][0] = round8(x);
          w[i][1] = round8(x + 8);
        }
        *reinterpret_cast<uint4*>(dst + (h + i) * p.qo_head) = w[i][0];
        *reinterpret_cast<uint4*>(dst + (h + i) * p.qo_head + c.half) = w[i][1];
      }
  }
}

template <int D, bool kNeox>
__global__ void __launch_bounds__(kThreads, 2) gqa_block_append_kernel(const BlockAppendParams p) {
  constexpr int kPieces = D / 16;           // lanes a row
  constexpr int kRows = 32 / kPieces;       // rows a warp reads at once
  constexpr int kSteps = kTile / kRows;
  __shared__ float s_top[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (blockIdx.x >= p.kv_ctas + p.q_ctas) {
    const int64_t i = static_cast<int64_t>(blockIdx.x - p.kv_ctas - p.q_ctas) * kThreads + threadIdx.x;
    if (i < p.B && !request_of(p, static_cast<int>(i)).sound) atomicOr(p.err, kErrBadIndptr);
    return;
  }
  if (blockIdx.x >= p.kv_ctas) {
    turn_queries<D, kNeox>(p, static_cast<int64_t>(blockIdx.x - p.kv_ctas) * kWarps + warp, lane);
    return;
  }
  // ---- the warp's unit: a request, a block of positions, a head's keys or values
  const int uw = p.unit_warps, wi = warp & (uw - 1);
  const int unit = blockIdx.x * (kWarps / uw) + warp / uw;
  const int slot = unit / (2 * p.Hk);
  if (slot >= p.kv_slots) return;
  const int part = unit - slot * (2 * p.Hk);
  const bool is_k = part < p.Hk;
  const int h = is_k ? part : part - p.Hk;
  const int bs = 1 << p.log2_block;
  const int log2_group = p.log2_block > 4 ? p.log2_block : 4;
  auto start = [&](int b) { return static_cast<int64_t>(__ldg(p.qo_indptr + b) >> log2_group) + 2 * static_cast<int64_t>(b); };
  const int b = warp_owner(p.B, lane, slot, start);
  const Request r = request_of(p, b);
  const int64_t t0 = r.t0;
  const int held = r.held, begin = held - r.tokens;          // the first new position
  const int64_t g0 = (begin >> log2_group) + (slot - start(b));
  if (!r.sound || r.tokens == 0 || slot < start(b) || g0 << log2_group >= held) return;   // an idle slot
  const int base = static_cast<int>(g0) << log2_group;

  const Columns col = columns_of<D>(lane % kPieces, is_k, p.half_rot);
  const int rr = lane / kPieces;
  const int64_t idx0 = __ldg(p.pages.indptr + b);
  const int ps_mask = (1 << p.pages.log2_page) - 1;
  const uint16_t* src = is_k ? p.k + h * p.k_head + col.c0 : p.v + h * p.v_head + col.c0;
  const int64_t src_tok = is_k ? p.k_tok : p.v_tok;
  uint8_t* cache = (is_k ? p.k_cache : p.v_cache) + h * p.head_pitch;
  float* scales = (is_k ? p.ks : p.vs) + h * p.sc_head;
  auto page_at = [&](int pos) -> int64_t {   // -1: outside the cache
    const int64_t page = __ldg(p.pages.indices + idx0 + (pos >> p.pages.log2_page));
    return page >= 0 && page < p.n_pages ? page : -1;
  };
  auto scale_at = [&](int64_t page, int pos) { return scales + page * p.sc_page + ((pos & ps_mask) >> p.log2_block) * p.sc_block; };
  // the block that the new positions continue, if it is in this unit: its scale
  const int joined = begin & ~(bs - 1);      // its first position
  const bool continues = joined < begin && joined >= base && joined < base + (1 << log2_group);
  float before = 0.f;
  if (continues) {
    const int64_t page = page_at(joined);
    if (page >= 0) before = *scale_at(page, joined);
  }

  // ---- a tile's rows, rotated: x, and which of them are there
  float x[kSteps][16];
  uint32_t there = 0;
  auto load = [&](int row0) {
    uint4 w[kSteps][2];
    there = 0;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int row = row0 + s * kRows + rr;
      const int64_t t = t0 + row - begin;
      if (row >= begin && row < held) {
        there |= 1u << s;
        w[s][0] = *reinterpret_cast<const uint4*>(src + t * src_tok);
        w[s][1] = *reinterpret_cast<const uint4*>(src + t * src_tok + col.half);
      } else {
        w[s][0] = w[s][1] = make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      widen8(w[s][0], x[s]);
      widen8(w[s][1], x[s] + 8);
      if (col.rot && there >> s & 1) {
        const int64_t pos = __ldg(p.positions + t0 + row0 + s * kRows + rr - begin);
        if (pos >= 0 && pos < p.max_pos) {
          Angles a;
          load_angles<kNeox>(p, pos, col.piece, &a);
          turn<kNeox>(x[s], a);
        } else {
          there &= ~(1u << s);               // these columns stay unwritten
        }
      }
    }
  };
  const int tiles = 1 << (log2_group - 4);
  auto has_new = [&](int tile) { return base + tile * kTile < held && base + (tile + 1) * kTile > begin; };
  float top[kSteps];                         // of the lane's row's block, in each step
#pragma unroll
  for (int s = 0; s < kSteps; ++s) top[s] = 0.f;
  int loaded = -1, last_tile = -1;
  for (int tile = wi; tile < tiles; tile += uw) {
    if (!has_new(tile)) continue;
    load(base + tile * kTile);
    loaded = last_tile = tile;
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
      if (there >> s & 1)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float a = fabsf(x[s][i]);
          top[s] = fmaxf(top[s], a < INFINITY ? a : 0.f);     // (a NaN is not either)
        }
  }
  const int lanes = bs >= kRows ? 32 : bs * kPieces;          // lanes whose rows share a block
#pragma unroll
  for (int s = 0; s < kSteps; ++s)
    for (int d = 1; d < lanes; d <<= 1) top[s] = fmaxf(top[s], __shfl_xor_sync(0xffffffffu, top[s], d));
#pragma unroll
  for (int d = 1; d < kSteps; d <<= 1)
    if (bs >= 2 * d * kRows) {
#pragma unroll
      for (int s = 0; s < kSteps; ++s)
        if ((s & d) == 0) top[s] = top[s + d] = fmaxf(top[s], top[s + d]);
    }
  if (uw > 1) {
    if (lane == 0) s_top[warp] = top[0];
    asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / uw), "r"(32 * uw) : "memory");
    float all = 0.f;
    for (int w = 0; w < uw; ++w) all = fmaxf(all, s_top[(warp & ~(uw - 1)) + w]);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) top[s] = all;
  }
  __syncwarp();                              // every lane has read the old scale

  // ---- codes, scales, and the rotated keys in bf16
  float grown = 0.f;                         // the continued block's scale
  for (int tile = last_tile; tile >= 0; tile -= uw) {
    if (!has_new(tile)) break;
    if (tile != loaded) load(base + tile * kTile);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int row = base + tile * kTile + s * kRows + rr;
      const int block = row & ~(bs - 1);
      const bool continued = continues && block == joined;
      const float fit = power_for(top[s]);
      const float scale = continued && before >= fit ? before : fit;
      if (row < begin || row >= held) continue;
      const int64_t t = t0 + row - begin;
      if (is_k && p.k_out && there >> s & 1) {
        uint16_t* dst = p.k_out + t * p.ko_tok + h * p.ko_head + col.c0;
        *reinterpret_cast<uint4*>(dst) = round8(x[s]);
        *reinterpret_cast<uint4*>(dst + col.half) = round8(x[s] + 8);
      }
      const int64_t page = page_at(row);
      if (page < 0) {
        if (lane % kPieces == 0) atomicOr(p.err, kErrBadRowId);
        continue;
      }
      if (is_k && h == 0 && col.rot && col.piece == 0 && !(there >> s & 1)) atomicOr(p.err, kErrBadIndex);
      if (there >> s & 1) {
        uint8_t* dst = cache + page * p.page_pitch + (row & ps_mask) * p.slot_pitch + col.c0;
        const Quotient d(scale);
        *reinterpret_cast<uint2*>(dst) = quantise8(x[s], d);
        *reinterpret_cast<uint2*>(dst + col.half) = quantise8(x[s] + 8, d);
      }
      // the block's first new row writes its scale
      if (lane % kPieces == 0 && (row == block || row == begin)) *scale_at(page, row) = scale;
    }
  }
  // ---- earlier codes of the continued block, where its scale grew
  if (!continues) return;
  {
    // the block's rows share a tile or the whole unit: the lane's own step has its maximum
    float mine = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
      const int row = (bs > kTile ? base : joined & ~(kTile - 1)) + s * kRows + rr;
      if (bs > kTile || (row & ~(bs - 1)) == joined) mine = fmaxf(mine, top[s]);
    }
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) mine = fmaxf(mine, __shfl_xor_sync(0xffffffffu, mine, d));
    grown = power_for(mine);
  }
  if (!(grown > before)) return;
  const float ratio = __fdiv_rn(before, grown);
  for (int row = (joined & ~(kTile - 1)) + wi * kTile + rr; row < begin; row += kRows) {
    // (a warp's rows: its tiles, kRows at a time)
    if (uw > 1 && ((row - base) / kTile) % uw != wi) continue;
    if (row < joined) continue;
    const int64_t page = page_at(row);
    if (page < 0) continue;
    uint4* at = reinterpret_cast<uint4*>(cache + page * p.page_pitch + (row & ps_mask) * p.slot_pitch + 16 * (lane % kPieces));
    uint4 w = *at;
    uint32_t* c = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = e4m3x2_to_f16x2(c[i]), hi = e4m3x2_to_f16x2(c[i] >> 16);
      const __half2 l2 = *reinterpret_cast<const __half2*>(&lo), h2 = *reinterpret_cast<const __half2*>(&hi);
      const float2 a = __half22float2(l2), e = __half22float2(h2);
      const uint32_t low = f32x2_to_e4m3x2(a.y * ratio, a.x * ratio), high = f32x2_to_e4m3x2(e.y * ratio, e.x * ratio);
      c[i] = low | (high << 16);
    }
    *at = w;
  }
}

template <int D, bool kNeox>
int launch(BlockAppendParams& p, int sms, cudaStream_t s) {
  constexpr int kRows = 32 / (D / 16);
  // a warp a tile of a block where requests bring that many tokens, else one that walks them
  const int tiles = p.log2_block > 4 ? 1 << (p.log2_block - 4) : 1;
  p.unit_warps = p.n_tok >= 16 * static_cast<int64_t>(p.B) ? tiles : 1;
  const int group = p.log2_block > 4 ? p.log2_block : 4;
  const int64_t slots = (p.n_tok >> group) + 2 * static_cast<int64_t>(p.B);
  const int64_t units = slots * 2 * p.Hk;
  const int64_t kv_ctas = (units * p.unit_warps + kWarps - 1) / kWarps;
  // query heads a warp: as many as leave every SM some warps
  const int64_t groups = (p.n_tok + kRows - 1) / kRows;
  p.strip = 1;
  while (p.strip < 8 && groups * (p.Hq / (2 * p.strip)) >= static_cast<int64_t>(sms) * 16) p.strip *= 2;
  const int64_t q_items = groups * ((p.Hq + p.strip - 1) / p.strip);
  const int64_t q_ctas = (q_items + kWarps - 1) / kWarps;
  const int64_t look_ctas = (p.B + kThreads - 1) / kThreads;
  const int64_t ctas = kv_ctas + q_ctas + look_ctas;
  if (units > 0x7FFFFFF0 || ctas > 0x7FFFFFFF) return MLA_ERR_UNSUPPORTED;
  p.kv_slots = static_cast<int>(slots);
  p.kv_ctas = static_cast<unsigned>(kv_ctas);
  p.q_ctas = static_cast<unsigned>(q_ctas);
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
