// What the two kernels of mla_gqa_block_decode share: the line of work, its spans and units, and the
// join of a unit's pieces.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "mla_gqa_decode_common.cuh"
#include "mla_gqa_pages.cuh"
#include "ptx.cuh"

namespace pmla {

constexpr float kLeastScale = 0x1p-60f;   // smaller scales of values count as this

struct BlockDecodeParams {
  const uint16_t* q;
  int64_t q_tok, q_head;
  const uint8_t *k, *v;
  int64_t page_pitch, slot_pitch, head_pitch;
  const float *ks, *vs;
  int64_t sc_page, sc_block, sc_head;   // strides in elements, both
  int log2_block;
  int64_t n_pages;
  PageList pages;
  const int32_t* qo_indptr;
  int64_t n_tok;
  int max_q;
  float sm_scale;
  void* o;
  int o_f32;
  int64_t o_tok, o_head;
  float* lse;
  int B, Hq, Hk, G;
  int* err;
  int* counters;                     // one a CTA: the unit that leaves its span's end
  float* slots;                      // two a CTA: m[R], l[R], o[R][D], R the rows of a unit
};

// The kernel for more than 16 query rows of a KV head, and whether it takes a call (mla_gqa_block_wide.cu).
bool block_wide_takes(const BlockDecodeParams& p, int64_t D);
cudaError_t launch_block_wide(const BlockDecodeParams& p, int64_t D, int sms, cudaStream_t stream);

}  // namespace pmla

namespace {

using namespace pmla;

__device__ __forceinline__ float lg2_approx(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float rcp_approx(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// Positions that some rows of a unit see and some do not are the new tokens' but the first.  A NaN
// among their values would reach all rows, zero times NaN being NaN.  So values that are NaN give
// way (codes to zero, scales to one), and the first such position is kept for the rows that see it:
// of each column, and of each head's scales.
constexpr int kNoPosition = 0x7FFFFFFF;
struct NanMarks {
  int first[128], scale[2];
  int any;
  __device__ __forceinline__ void clear(int i, int step) {
    for (int c = i; c < 128; c += step) first[c] = kNoPosition;
    if (i < 2) scale[i] = kNoPosition;
    if (i == 2) any = 0;
  }
  // Whether the column, of the unit's head hp, is NaN in a row that sees `seen` positions.
  __device__ __forceinline__ bool reach(int column, int hp, int seen) const {
    return first[column] < seen || scale[hp] < seen;
  }
  __device__ __noinline__ void drop(uint4* chunk, int at, int column) {
    any = 1;
    uint8_t* const code = reinterpret_cast<uint8_t*>(chunk);
    for (int b = 0; b < 16; ++b)
      if ((code[b] & 0x7F) == 0x7F) {
        atomicMin(first + column + b, at);
        code[b] = 0;
      }
  }
  // 16 codes of position `at` from a column on.
  __device__ __forceinline__ void look(uint4* chunk, int at, int column) {
    const uint4 w = *chunk;
    auto sevens = [](uint32_t x) { return (x & 0x7F7F7F7Fu) + 0x01010101u; };      // 0x80 where a byte is 0x7F or 0xFF
    if ((sevens(w.x) | sevens(w.y) | sevens(w.z) | sevens(w.w)) & 0x80808080u) drop(chunk, at, column);
  }
  __device__ __forceinline__ void look(float* v_scale, int at, int hp) {
    if (!isnan(*v_scale)) return;
    any = 1;
    atomicMin(scale + hp, at);
    *v_scale = 1.f;
  }
};

// The line of work, of all requests or of those before one: tiles of all units, and units.
struct Line {
  int64_t tiles, units;
  __device__ Line operator+(const Line& o) const { return {tiles + o.tiles, units + o.units}; }
  __device__ Line operator-(const Line& o) const { return {tiles - o.tiles, units - o.units}; }
  __device__ int64_t length(int cost) const { return tiles + cost * units; }
};
__device__ __forceinline__ Line shfl_up(const Line& x, int d) {
  return {__shfl_up_sync(0xffffffffu, x.tiles, d), __shfl_up_sync(0xffffffffu, x.units, d)};
}

// Where a span's border, x tiles into a unit of n, cuts it: pieces of fewer than kLeastPiece
// tiles go to the neighbouring span, so units of fewer than twice as many stay whole.
template <class S>
__device__ __forceinline__ int snap(int64_t x, int n) {
  if (x >= n) return n;
  if (x < S::kLeastPiece) return 0;
  return n - x < S::kLeastPiece ? n : static_cast<int>(x);
}

// A request's positions and new tokens; none where its lists make no sense.
struct Request {
  int len, tokens;
};
__device__ __forceinline__ Request request_of(const BlockDecodeParams& p, int b, bool flag) {
  const int64_t s = __ldg(p.qo_indptr + b), e = __ldg(p.qo_indptr + b + 1);
  int len = p.pages.positions(b);
  bool sound = len >= 0;
  if (!sound) len = 0;
  int tokens = 0;
  if (s >= 0 && e >= s && e <= p.n_tok && e - s <= p.max_q) tokens = static_cast<int>(e - s);
  else sound = false;
  if (!sound && flag) atomicOr(p.err, kErrBadIndptr);
  return {len, tokens};
}
template <class S>
__device__ __forceinline__ int chunks_of(const BlockDecodeParams& p, int tokens) {
  return (tokens * p.G + S::kHeads - 1) / S::kHeads;
}
// The request's part of the line.
template <class S>
__device__ __forceinline__ Line request_line(const BlockDecodeParams& p, const Request& r) {
  const int64_t units = r.len > 0 ? chunks_of<S>(p, r.tokens) * ((p.Hk + S::HP - 1) / S::HP) : 0;
  return {(r.len + S::kTile - 1) / S::kTile * units, units};
}

__device__ __forceinline__ void store_o(const BlockDecodeParams& p, int64_t tok, int h, int d, float x) {
  const int64_t at = tok * p.o_tok + h * p.o_head + d;
  if (p.o_f32) static_cast<float*>(p.o)[at] = x;
  else static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(x);
}

// One piece of a unit.
struct Piece {
  Request r;
  int64_t tok0, idx0;                // the request's first token and first page
  int hk0, h0, nh;                   // first KV head; first row of the chunk, rows of a head
  int live_rows;                     // rows of the unit from there on are nobody's (no such head)
  int t0, t1, n_tiles;               // its tiles, of the unit's
  int64_t u0;                        // the unit's first tile on the line
};

// A CTA's span of the line, and the request that it starts in.
struct Span {
  int64_t begin, end, length;        // on the line; of every span
  int cost;                          // of a unit, besides its tiles
  int b;
  Request r;
  int64_t base;                      // the line position of request b
};
template <int kWarps>
struct SpanShared {
  Line scan[kWarps];
  int64_t base;
  int b, empty, last;
  Request r;
};

// Finds it; empty requests get their rows on the way.  False where there is nothing to do (for
// all threads alike).
template <class S>
__device__ __forceinline__ bool find_span(const BlockDecodeParams& p, SpanShared<S::kWarps>* sh, Span* out) {
  constexpr int D = S::D, kWarps = S::kWarps, kThreads = S::kThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  // ---- the line: its length, this CTA's span, and the request its span starts in.  The
  // first kThreads requests stay in registers, so that a batch of up to kThreads pays one round
  // trip to memory here.
  if (tid == 0) sh->empty = 0;
  __syncthreads();
  Line mine = {0, 0};
  Request r0 = {0, 0};
#pragma unroll 4
  for (int b = tid; b < p.B; b += kThreads) {
    const Request r = request_of(p, b, cta == 0);
    if (b < kThreads) r0 = r;
    mine = mine + request_line<S>(p, r);
    if (r.len == 0 && b % gridDim.x == cta) sh->empty = 1;
  }
  const Line mine0 = request_line<S>(p, r0);
  Line inc = mine0;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const Line o = shfl_up(inc, i);
    if (lane >= i) inc = inc + o;
  }
  if (p.B > kThreads) {
#pragma unroll
    for (int i = 16; i; i >>= 1) {
      mine.tiles += __shfl_xor_sync(0xffffffffu, mine.tiles, i);
      mine.units += __shfl_xor_sync(0xffffffffu, mine.units, i);
    }
  } else if (lane == 31) {
    mine = inc;
  }
  if (lane == 31) sh->scan[warp] = mine;
  __syncthreads();
  Line all = {0, 0}, before = {0, 0};
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before = before + sh->scan[w];
    all = all + sh->scan[w];
  }
  // a unit's cost, less where CTAs have little to do: then cuts pay earlier
  const int64_t share = quotient(all.tiles, 10 * static_cast<int64_t>(gridDim.x));
  const int cost = static_cast<int>(share > S::kUnitCost ? S::kUnitCost : (share < S::kLeastCost ? S::kLeastCost : share));
  const int64_t total = all.length(cost);
  const int64_t span = quotient(total + gridDim.x - 1, gridDim.x);
  const int64_t x_begin = cta * span;
  const int64_t x_end = x_begin + span < total ? x_begin + span : total;
  if (sh->empty)                                    // empty requests: o = 0, lse = -inf
    for (int b = cta; b < p.B; b += gridDim.x) {
      const Request r = request_of(p, b, false);
      if (r.len != 0) continue;
      const int64_t tok = __ldg(p.qo_indptr + b);
      for (int e = tid; e < r.tokens * p.Hq * D; e += kThreads) {
        const int h = e / D % p.Hq;
        const int64_t at = tok + e / D / p.Hq;
        store_o(p, at, h, e % D, 0.f);
        if (e % D == 0 && p.lse) p.lse[at * p.Hq + h] = -INFINITY;
      }
    }
  if (x_begin >= x_end) return false;
  if (p.B <= kThreads) {
    const int64_t start = (before + inc - mine0).length(cost), n = mine0.length(cost);
    if (n > 0 && x_begin >= start && x_begin < start + n) {
      sh->b = tid;
      sh->r = r0;
      sh->base = start;
    }
    __syncthreads();
  } else {
    Line done = {0, 0};    // the line before this block of kThreads requests
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int b = b0 + tid;
      const Request r = b < p.B ? request_of(p, b, false) : Request{0, 0};
      const Line part = request_line<S>(p, r);
      Line run = part;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const Line o = shfl_up(run, i);
        if (lane >= i) run = run + o;
      }
      __syncthreads();
      if (lane == 31) sh->scan[warp] = run;
      __syncthreads();
      Line start = done + run - part;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) start = start + sh->scan[w];
        done = done + sh->scan[w];
      }
      const int64_t at = start.length(cost), n = part.length(cost);
      if (n > 0 && x_begin >= at && x_begin < at + n) {
        sh->b = b;
        sh->r = r;
        sh->base = at;
      }
      if (done.length(cost) > x_begin) break;
    }
    __syncthreads();
  }
  *out = {x_begin, x_end, span, cost, sh->b, sh->r, sh->base};
  return true;
}

// The piece at line position *x of the span, and *x behind its unit; false where the neighbours'
// spans have all of the unit.
template <class S>
__device__ __forceinline__ bool next_piece(const BlockDecodeParams& p, Span& s, int64_t* x, Piece* u) {
  int64_t whole;
  while (*x >= s.base + (whole = request_line<S>(p, s.r).length(s.cost))) {        // the next request with work
    s.base += whole;
    ++s.b;
    s.r = request_of(p, s.b, false);
  }
  u->n_tiles = (s.r.len + S::kTile - 1) / S::kTile;
  const int64_t weight = u->n_tiles + s.cost;
  const int ui = static_cast<int>(quotient(*x - s.base, weight));
  u->u0 = s.base + ui * weight + s.cost;
  u->t0 = snap<S>(s.begin - u->u0, u->n_tiles);
  u->t1 = snap<S>(s.end - u->u0, u->n_tiles);
  *x = u->u0 + u->n_tiles;
  if (u->t0 >= u->t1) return false;
  const int rows = s.r.tokens * p.G, chunks = chunks_of<S>(p, s.r.tokens);
  u->r = s.r;
  u->hk0 = ui / chunks;
  u->h0 = (ui - u->hk0 * chunks) * S::kHeads;
  u->hk0 *= S::HP;
  u->nh = rows - u->h0 < S::kHeads ? rows - u->h0 : S::kHeads;
  u->live_rows = u->hk0 + S::HP <= p.Hk ? S::kRows : (p.Hk - u->hk0) * S::kHeads;
  u->tok0 = __ldg(p.qo_indptr + s.b);
  u->idx0 = __ldg(p.pages.indptr + s.b);
  return true;
}

// Whether a row of the unit is somebody's.
template <class S>
__device__ __forceinline__ bool row_there(const Piece& u, int row) {
  return row < u.live_rows && row % S::kHeads < u.nh;
}

// A row's results from its columns d .. d + n - 1, its reference in units of log2 and its sum.
template <class S, int n>
__device__ __forceinline__ void finish_row(const BlockDecodeParams& p, const Piece& u, int row, int d, const float* oo,
                                           float mm, float ll) {
  const int h = u.h0 + row % S::kHeads, of = h / p.G;
  const int hq = (u.hk0 + row / S::kHeads) * p.G + h - of * p.G;
  const int64_t tok = u.tok0 + of;
  const bool none = ll == 0.f;
  const float f = none ? 0.f : 1.f / ll;
#pragma unroll
  for (int i = 0; i < n; ++i) store_o(p, tok, hq, d + i, none ? 0.f : oo[i] * f);
  if (d == 0 && p.lse) p.lse[tok * p.Hq + hq] = none ? -INFINITY : (mm == -INFINITY ? 0.f : mm) * kLn2 + logf(ll);
}

// Where a CTA leaves its part of a unit that others have parts of: m[R], l[R], o[R][D].
template <class S>
__device__ __forceinline__ float* part_slot(const BlockDecodeParams& p, const Piece& u) {
  return p.slots + (2 * static_cast<int64_t>(blockIdx.x) + (u.t0 == 0 ? 1 : 0)) * S::kSlotFloats;
}

// After a CTA's part: the last span to arrive joins the unit's pieces, in the spans' order.  s_m, s_l:
// R floats each; over: room for m and l of all pieces in shared memory.  By S::kJoinThreads threads.
template <class S>
__device__ __forceinline__ void join_parts(const BlockDecodeParams& p, const Span& s, const Piece& u,
                                           SpanShared<S::kWarps>* sh, float* s_m, float* s_l, float* over) {
  constexpr int D = S::D, kRows = S::kRows, kWarps = S::kJoinWarps, kThreads = S::kJoinThreads;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t first = quotient(u.u0 + S::kLeastPiece - 1, s.length);
  const int64_t last = quotient(u.u0 + u.n_tiles - S::kLeastPiece, s.length);
  const int used = S::HP == 1 ? u.nh : u.live_rows;          // rows to look at
  S::join_sync();
  if (tid == 0) {
    int* c = p.counters + first;
    __threadfence();                   // the CTA's part before its arrival
    const int seen = atomicAdd(c, 1);
    sh->last = seen == last - first;
    if (sh->last) *c = 0;               // as it was found, for the next call
    __threadfence();                   // the others' parts after theirs
  }
  S::join_sync();
  if (sh->last) {
    const int np = static_cast<int>(last - first) + 1;
    float* s_f = over;         // [piece][row], over the rings
    float* s_s = s_f + np * kRows;
    // parts lie two slots apart, the first one a slot further on
    const float* parts = p.slots + 2 * first * S::kSlotFloats;
    for (int e = tid; e < np * kRows; e += kThreads) {
      const int i = e / kRows, h = e - i * kRows;
      const float* sl = parts + (2 * i + (i == 0 ? 1 : 0)) * S::kSlotFloats;
      s_f[e] = row_there<S>(u, h) ? __ldcg(sl + h) : 0.f;
      s_s[e] = row_there<S>(u, h) ? __ldcg(sl + kRows + h) : 0.f;
    }
    S::join_sync();
    // a warp a row, lanes over pieces
    for (int h = warp; h < used; h += kWarps) {
      if (!row_there<S>(u, h)) continue;
      float mm = -INFINITY, ll = 0.f;
      for (int i = lane; i < np; i += 32) mm = fmaxf(mm, s_f[i * kRows + h]);
#pragma unroll
      for (int d = 16; d; d >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, d));
      for (int i = lane; i < np; i += 32) {
        const float mw = s_f[i * kRows + h];
        const float f = mw == -INFINITY ? 1.f : ex2_approx(mw - mm);
        s_f[i * kRows + h] = f;
        ll += f * s_s[i * kRows + h];
      }
#pragma unroll
      for (int d = 16; d; d >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, d);
      if (lane == 0) {
        s_m[h] = mm;
        s_l[h] = ll;
      }
    }
    S::join_sync();
    constexpr int kEach = 4 * kThreads;  // columns the threads take at once
    for (int e0 = 4 * tid; e0 < used * D; e0 += 2 * kEach) {
      const bool two = S::kTwo && e0 + kEach < used * D;
      const int h = e0 / D, h2 = (e0 + kEach) / D;
      float oo[8] = {};
      for (int i0 = 0; i0 < np; i0 += S::kAhead) {       // all their loads in flight at once
        float4 y[2 * S::kAhead];       // (the odd ones unused without a second word)
#pragma unroll
        for (int i = 0; i < S::kAhead; ++i)
          if (i0 + i < np) {
            const float* at = parts + (2 * (i0 + i) + (i0 + i == 0 ? 1 : 0)) * S::kSlotFloats + 2 * kRows + e0;
            y[2 * i] = __ldcg(reinterpret_cast<const float4*>(at));
            if (two) y[2 * i + 1] = __ldcg(reinterpret_cast<const float4*>(at + kEach));
          }
#pragma unroll
        for (int i = 0; i < S::kAhead; ++i) {
          if (i0 + i >= np) break;
          const float f = s_f[(i0 + i) * kRows + h];
          oo[0] += f * y[2 * i].x;
          oo[1] += f * y[2 * i].y;
          oo[2] += f * y[2 * i].z;
          oo[3] += f * y[2 * i].w;
          if (!two) continue;
          const float f2 = s_f[(i0 + i) * kRows + h2];
          oo[4] += f2 * y[2 * i + 1].x;
          oo[5] += f2 * y[2 * i + 1].y;
          oo[6] += f2 * y[2 * i + 1].z;
          oo[7] += f2 * y[2 * i + 1].w;
        }
      }
      if (row_there<S>(u, h)) finish_row<S, 4>(p, u, h, e0 % D, oo, s_m[h], s_l[h]);
      if (two && row_there<S>(u, h2)) finish_row<S, 4>(p, u, h2, (e0 + kEach) % D, oo + 4, s_m[h2], s_l[h2]);
    }
  }
}

}  // namespace
