// mla_gqa_decode: attention of one new token a request over a paged cache of per-head keys
// and values, split over the cache's length and joined in the same launch.
//
//   s_j = sm_scale * k_scale * q . k_j,   o = v_scale * sum_j e^{s_j - lse} v_j,
//   lse = ln sum_j e^{s_j}, over the request's L positions, for each of the G = Hq / Hk query
//   heads of a KV head.
//
// Bound by the cache's bytes: 2 D elements a position and KV head, each used by G heads.
// Measured (GB300, pages of 128 or 16, calls in a CUDA graph; on its own a call takes at least the
// 10 us of its host side): 64 requests of 2,048 to 65,536 positions, two KV
// heads, bf16, 1.51 GB: 223 us, 6.77 TB/s (the copy rate); one of 142,000 positions,
// eight KV heads, e4m3, 291 MB: 57 us, of which 40 stream the cache, the rest are the plan, the
// first tiles and the join of 19 pieces a unit; 37 ragged requests, 10.6 MB: 11.5 us; one of 137
// positions: 5.4 us.  64 requests of 8,192 positions, two KV heads of 64, eight query heads each:
// 48 us in bf16 (5.5 TB/s), 37 in e4m3 (3.6).
//
// Work split.  A unit is (request, KV head, chunk of 8 NT query heads); its positions are cut
// into tiles of 16 or 32.  All units' tiles form one line and every CTA takes an equal span of it,
// so ragged lengths, few long requests and many short ones all fill the GPU.  A unit that
// crosses a span's end leaves partials (m, l, o in fp32) in workspace slots; the CTA that
// arrives last at the unit's counter joins them in the order of the spans, so the result does
// not depend on the order of arrival.
//
// Inside a CTA four or eight warps take tiles in turn, each with its own ring of cp.async stages, its
// own running maximum, sum and output, and no barrier until the span's piece ends.
//   S^T (16 positions x 8 heads) = K (16 x D) . q^T by mma.sync m16n8k16 with K as the A
//   operand, so that 8 heads fill the MMA's N exactly (a step has at most a few heads a KV
//   head; tcgen05's smallest M of 64 rows would be mostly padding, and the MMAs hide under
//   the loads); softmax over positions; O^T (D x 8) += V^T . P^T, where P^T's fragments come
//   from S^T's by one 8x8 transpose (movmatrix).
// A bf16 cache multiplies in bf16, P rounded to bf16 (2^-8 of each weight at most, the sum l
// kept in fp32 from the unrounded weights).  An e4m3 cache multiplies in f16, into which its
// codes convert exactly: each q row is scaled by a power of two to a maximum in [2^13, 2^14)
// (q's 8 bits fit f16's 11; what falls below f16's range is under 2^-38 of the row's
// maximum), P carries a factor 2^14 that cancels against l (rounded by at most 2^-11).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/paged_mla.h"
#include "mla_gqa_check.h"
#include "ptx.cuh"

namespace {

using namespace pmla;

constexpr int kHeaderBytes = 256;    // error word
constexpr int kSmWarps = 8;          // warps a SM, in two CTAs or in one
constexpr int kMaxSms = 160;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

struct GqaDecodeParams {
  const uint16_t* q;
  int64_t q_tok, q_head;
  const uint8_t *k, *v;
  int64_t page_pitch, slot_pitch, head_pitch;
  int log2_page;
  int64_t n_pages;
  const int32_t *kv_indptr, *kv_indices, *last;
  int64_t n_idx;
  const float *k_scale, *v_scale;
  float sm_scale;
  void* o;
  int o_f32;
  int64_t o_tok, o_head;
  float* lse;
  int B, Hq, Hk, G, chunks;
  int* err;
  int* counters;                     // one a CTA: the unit that leaves its span's end
  float* slots;                      // two a CTA: m[R], l[R], o[R][D] with R = 8 NT
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t* r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool kF16>
__device__ __forceinline__ void mma16816(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  if constexpr (kF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}

// D columns, cache type, n-tiles of 8 query heads, warps a CTA; kStages tiles in flight a warp.
template <int D_, bool kFp8_, int NT_, int W_>
struct DecodeShape {
  static constexpr int D = D_, NT = NT_;
  static constexpr int kWarps = W_, kThreads = 32 * W_;
  static constexpr int kCtasPerSm = kSmWarps / W_;
  static constexpr int kMaxCtas = kMaxSms * kCtasPerSm;    // a unit has at most one piece a CTA
  static constexpr bool kFp8 = kFp8_;
  static constexpr int kRow = D * (kFp8 ? 1 : 2);          // bytes of a K or V row
  // positions a warp takes at a time, in groups of 16 (the MMA's M): rows of 128 bytes or less
  // two groups, so that the softmax's shuffles and the loop are paid half as often (64 requests
  // of 8,192 positions, e4m3, 64-wide rows: 42 us with one, 36 with two; 128-wide: 56 and 54)
  static constexpr int MT = kRow <= 128 && NT <= 2 ? 2 : 1;
  static constexpr int kTile = 16 * MT;
  static constexpr int kTileBytes = 2 * kTile * kRow;      // K then V
  static constexpr int kHeads = 8 * NT;
  // about 24 KB in flight a warp (eight warps a SM: 192 KB)
  static constexpr int kStages = 24576 / kTileBytes < 8 ? 24576 / kTileBytes : 8;
  static constexpr int kWarpBytes = kStages * kTileBytes;
  static constexpr int kJoinBytes = kWarps * kHeads * D * 4;   // per-warp outputs, over the rings
  static constexpr int kPieceBytes = 2 * kMaxCtas * kHeads * 4;   // m and l of a unit's pieces, over them too
  static constexpr int kOverBytes = kJoinBytes > kPieceBytes ? kJoinBytes : kPieceBytes;
  static constexpr int kBuf = kWarps * kWarpBytes > kOverBytes ? kWarps * kWarpBytes : kOverBytes;
  static constexpr int kSmem = kBuf + 2 * kWarps * kHeads * 4;
  static_assert(kCtasPerSm * (kSmem + 1024 + 64) <= 233472, "shared memory of a SM");
  static constexpr int kSlotFloats = kHeads * (D + 2);
  static constexpr bool kTwo = kHeads * D > 4 * kThreads;  // a join's thread has two words of o
  static constexpr int kAhead = NT == 4 ? 2 : (kTwo ? 10 : 20);   // pieces whose words are in flight
  // what a unit costs besides its tiles (page ids, the first tile's way from DRAM, the joins:
  // about 2.5 us), in tiles at the bandwidth of four warps (22 bytes a ns); CTAs of eight take
  // the same (one of 142,000 positions: 59 us; with 0.7 of it 63, with 1.5 times it 61)
  static constexpr int kUnitCost = 55000 / kTileBytes;
};

// Weight of one unit of a request on the line of work.
template <class S>
__device__ __forceinline__ int64_t line_weight(int len) {
  return len > 0 ? (len + S::kTile - 1) / S::kTile + S::kUnitCost : 0;
}

// Where a span's border, x tiles into a unit of n, cuts it: pieces shorter than their fixed
// cost go to the neighbouring span, so units of fewer than 2 kUnitCost tiles stay whole.
template <class S>
__device__ __forceinline__ int snap(int64_t x, int n) {
  if (x >= n) return n;
  if (x < S::kUnitCost) return 0;
  return n - x < S::kUnitCost ? n : static_cast<int>(x);
}

// a / b for a >= 0, b > 0, by the 32-bit divide where both fit.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// Byte offset of 16-byte chunk c of row r: chunks are permuted within 128 bytes so that
// eight rows' equal chunks fall into different banks.
template <int kRow>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
  if constexpr (kRow >= 128) return r * kRow + ((c ^ (r & 7)) << 4);
  else return r * kRow + ((c ^ ((r >> 1) & 3)) << 4);      // 64-byte rows: two a line
}

// Positions of request b, 0 where its page list makes no sense.
__device__ __forceinline__ int request_len(const GqaDecodeParams& p, int b, bool flag) {
  const int64_t s = __ldg(p.kv_indptr + b), e = __ldg(p.kv_indptr + b + 1);
  const int last_len = p.last ? __ldg(p.last + b) : 1 << p.log2_page;
  if (s < 0 || e < s || e > p.n_idx) {
    if (flag) atomicOr(p.err, kErrBadIndptr);
    return 0;
  }
  if (e == s) return 0;
  const int ps = 1 << p.log2_page;
  const int last = last_len < 1 ? 1 : (last_len > ps ? ps : last_len);
  const int64_t len = ((e - s - 1) << p.log2_page) + last;
  if (len > 0x7FFFFF00) {
    if (flag) atomicOr(p.err, kErrBadIndptr);
    return 0;
  }
  return static_cast<int>(len);
}

__device__ __forceinline__ void store_o(const GqaDecodeParams& p, int b, int h, int d, float x) {
  const int64_t at = b * p.o_tok + h * p.o_head + d;
  if (p.o_f32) static_cast<float*>(p.o)[at] = x;
  else static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(x);
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, S::kCtasPerSm) gqa_decode_kernel(const GqaDecodeParams p) {
  constexpr int D = S::D, NT = S::NT, MT = S::MT, kRow = S::kRow, kTile = S::kTile, kHeads = S::kHeads;
  constexpr int kWarps = S::kWarps, kThreads = S::kThreads;
  constexpr bool kFp8 = S::kFp8;
  extern __shared__ __align__(128) uint8_t smem[];
  float* s_m = reinterpret_cast<float*>(smem + S::kBuf);       // [warp][head]
  float* s_l = s_m + kWarps * kHeads;
  __shared__ int64_t sh_scan[kWarps];
  __shared__ int64_t sh_base;
  __shared__ int sh_b, sh_len, sh_last, sh_empty;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int units = p.Hk * p.chunks;
  const int cta = blockIdx.x;

  // ---- the line: its length, this CTA's span, and the request its span starts in.  The
  // first kThreads requests' lengths stay in registers, so that a batch of up to kThreads
  // pays one round trip to memory here.
  if (tid == 0) sh_empty = 0;
  __syncthreads();
  int64_t mine = 0, inc = 0;
  int len0 = 0;
#pragma unroll 4
  for (int b = tid; b < p.B; b += kThreads) {
    const int len = request_len(p, b, cta == 0);
    if (b < kThreads) len0 = len;
    mine += line_weight<S>(len);
    if (len == 0 && b % gridDim.x == cta) sh_empty = 1;
  }
  const int64_t mine0 = line_weight<S>(len0);
  inc = mine0;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, inc, i);
    if (lane >= i) inc += o;
  }
  if (p.B > kThreads) {
#pragma unroll
    for (int i = 16; i; i >>= 1) mine += __shfl_xor_sync(0xffffffffu, mine, i);
  } else {
    mine = __shfl_sync(0xffffffffu, inc, 31);
  }
  if (lane == 0) sh_scan[warp] = mine;
  __syncthreads();
  int64_t total = 0, before = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh_scan[w];
    total += sh_scan[w];
  }
  total *= units;
  const int64_t span = quotient(total + gridDim.x - 1, gridDim.x);
  const int64_t x_begin = cta * span;
  const int64_t x_end = x_begin + span < total ? x_begin + span : total;
  if (sh_empty)                                    // empty requests: o = 0, lse = -inf
    for (int b = cta; b < p.B; b += gridDim.x) {
      if (request_len(p, b, false) != 0) continue;
      for (int e = tid; e < p.Hq * D; e += kThreads) {
        store_o(p, b, e / D, e % D, 0.f);
        if (e % D == 0 && p.lse) p.lse[static_cast<int64_t>(b) * p.Hq + e / D] = -INFINITY;
      }
    }
  if (x_begin >= x_end) return;
  if (p.B <= kThreads) {
    const int64_t start = (before + inc - mine0) * units;
    if (mine0 > 0 && x_begin >= start && x_begin < start + mine0 * units) {
      sh_b = tid;
      sh_len = len0;
      sh_base = start;
    }
    __syncthreads();
  } else {
    int64_t done = 0;      // the line before this block of kThreads requests
    for (int b0 = 0; b0 < p.B; b0 += kThreads) {
      const int b = b0 + tid;
      const int len = b < p.B ? request_len(p, b, false) : 0;
      const int64_t n = line_weight<S>(len) * units;
      int64_t run = n;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, run, i);
        if (lane >= i) run += o;
      }
      __syncthreads();
      if (lane == 31) sh_scan[warp] = run;
      __syncthreads();
      int64_t start = done + run - n, all = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        if (w < warp) start += sh_scan[w];
        all += sh_scan[w];
      }
      if (n > 0 && x_begin >= start && x_begin < start + n) {
        sh_b = b;
        sh_len = len;
        sh_base = start;
      }
      done += all;
      if (done > x_begin) break;
    }
    __syncthreads();
  }
  int b = sh_b, len = sh_len;
  int64_t base = sh_base;              // the line position of request b
  int n_tiles = (len + kTile - 1) / kTile;
  int64_t weight = line_weight<S>(len);

  const uint32_t ring = smem_u32(smem) + warp * S::kWarpBytes;
  const float kscale = kFp8 ? __ldg(p.k_scale) : 1.f;
  const float vscale = kFp8 ? __ldg(p.v_scale) : 1.f;
  const int g = lane >> 2, cq = lane & 3;

  for (int64_t x = x_begin; x < x_end;) {
    while (x >= base + weight * units) {           // the next request with work
      base += weight * units;
      ++b;
      len = request_len(p, b, false);
      n_tiles = (len + kTile - 1) / kTile;
      weight = line_weight<S>(len);
    }
    const int u = static_cast<int>(quotient(x - base, weight));
    const int64_t u0 = base + u * weight + S::kUnitCost;           // the unit's first tile
    const int t0 = snap<S>(x_begin - u0, n_tiles), t1 = snap<S>(x_end - u0, n_tiles);
    x = u0 + n_tiles;
    if (t0 >= t1) continue;                        // the neighbours' spans have all of it
    const int hk = u / p.chunks;
    const int h0 = (u - hk * p.chunks) * kHeads;                   // first head of the chunk
    const int nh = p.G - h0 < kHeads ? p.G - h0 : kHeads;
    const int64_t idx0 = p.kv_indptr[b];

    // ---- loads of one tile: its page ids one tile ahead, then 16-byte cp.asyncs
    const uint8_t* kh = p.k + hk * p.head_pitch;
    const uint8_t* vh = p.v + hk * p.head_pitch;
    const int ps_mask = (1 << p.log2_page) - 1;
    const bool one_page = (1 << p.log2_page) >= kTile;    // a tile never crosses a page
    auto page_of = [&](int t) -> int {       // lane's page id for tile t (-1: no position)
      const int j = t * kTile + (one_page ? 0 : lane & (kTile - 1));
      return t < t1 && j < len ? __ldg(p.kv_indices + idx0 + (j >> p.log2_page)) : -1;
    };
    constexpr int kChunks = kRow / 16, kRowsAt = 32 / kChunks;
    const int lc = lane % kChunks, lr = lane / kChunks;
    auto issue = [&](int t, int stage, int page) {
      if (t < t1) {
        const uint32_t dst = ring + stage * S::kTileBytes;
        const bool ok = page >= 0 && page < p.n_pages;
        if (one_page) {
          if (!ok && lane == 0) atomicOr(p.err, kErrBadRowId);     // reads as zeros
          const int64_t off = ok ? page * p.page_pitch + ((t * kTile) & ps_mask) * p.slot_pitch : 0;
          int64_t at = off + lr * p.slot_pitch + 16 * lc;
          const int rows = ok ? len - t * kTile : 0;
#pragma unroll
          for (int i = 0; i < kTile / kRowsAt; ++i) {
            const int r = i * kRowsAt + lr;
            const uint32_t n = r < rows ? 16u : 0u;
            const uint32_t d = dst + chunk_at<kRow>(r, lc);
            cp_async_16(d, kh + (n ? at : 0), n);
            cp_async_16(d + kTile * kRow, vh + (n ? at : 0), n);
            at += kRowsAt * p.slot_pitch;
          }
        } else {
          const int j = t * kTile + (lane & (kTile - 1));
          int64_t off = -1;
          if (j < len) {
            if (ok) off = page * p.page_pitch + (j & ps_mask) * p.slot_pitch;
            else atomicOr(p.err, kErrBadRowId);
          }
#pragma unroll
          for (int i = 0; i < kTile / kRowsAt; ++i) {
            const int r = i * kRowsAt + lr;
            const int64_t ro = __shfl_sync(0xffffffffu, off, r);
            const uint32_t n = ro >= 0 ? 16u : 0u;
            const int64_t at = (ro >= 0 ? ro : 0) + 16 * lc;
            const uint32_t d = dst + chunk_at<kRow>(r, lc);
            cp_async_16(d, kh + at, n);
            cp_async_16(d + kTile * kRow, vh + at, n);
          }
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    int t_load = t0 + warp;
    int page;
    {
      int ahead[S::kStages];               // the first tiles' page ids, read together
#pragma unroll
      for (int i = 0; i < S::kStages; ++i) ahead[i] = page_of(t_load + i * kWarps);
#pragma unroll
      for (int i = 0; i < S::kStages - 1; ++i) issue(t_load + i * kWarps, i, ahead[i]);
      t_load += (S::kStages - 1) * kWarps;
      page = ahead[S::kStages - 1];
    }

    // ---- q fragments: head 8 nt + g, columns as the K fragments hold them
    uint32_t qf[NT][D / 16][2];
    float sc[NT][2];                   // softmax scale in log2 units of heads 2 cq, 2 cq + 1
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int h = 8 * nt + g;
      const bool live = h < nh;
      const uint16_t* row = p.q + b * p.q_tok + (static_cast<int64_t>(hk) * p.G + h0 + (live ? h : 0)) * p.q_head;
      if constexpr (!kFp8) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          qf[nt][kk][0] = live ? __ldg(reinterpret_cast<const uint32_t*>(row + 16 * kk + 2 * cq)) : 0u;
          qf[nt][kk][1] = live ? __ldg(reinterpret_cast<const uint32_t*>(row + 16 * kk + 8 + 2 * cq)) : 0u;
        }
        sc[nt][0] = sc[nt][1] = p.sm_scale * kLog2e;
      } else {
        // the fragment's k columns 2cq, 2cq+1, 8+2cq, 9+2cq are the row's 4cq .. 4cq+3
        float mx = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint2 w = live ? __ldg(reinterpret_cast<const uint2*>(row + 16 * kk + 4 * cq)) : make_uint2(0, 0);
          qf[nt][kk][0] = w.x;
          qf[nt][kk][1] = w.y;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            mx = fmaxf(mx, fabsf(__uint_as_float(qf[nt][kk][i] << 16)));
            mx = fmaxf(mx, fabsf(__uint_as_float(qf[nt][kk][i] & 0xFFFF0000u)));
          }
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        int e = 267 - static_cast<int>(__float_as_uint(mx) >> 23);   // 2^(13 - exponent), biased
        e = e > 253 ? 253 : e;
        const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
        const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qf[nt][kk][i];
            qf[nt][kk][i] = f32x2_to_f16x2(__uint_as_float(w & 0xFFFF0000u) * up, __uint_as_float(w << 16) * up);
          }
        // heads 2cq and 2cq+1 of this n-tile: their q rows sit at lanes 8cq and 8cq+4
        const float d0 = __shfl_sync(0xffffffffu, down, 8 * cq);
        const float d1 = __shfl_sync(0xffffffffu, down, 8 * cq + 4);
        const float f = p.sm_scale * kscale * kLog2e;
        sc[nt][0] = f * d0;
        sc[nt][1] = f * d1;
      }
    }

    float acc[NT][D / 16][4];
    float m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[nt][i][j] = 0.f;
      m[nt][0] = m[nt][1] = -INFINITY;
      l[nt][0] = l[nt][1] = 0.f;
    }

    int stage = 0;
#pragma unroll 1
    for (int t = t0 + warp; t < t1; t += kWarps) {
      asm volatile("cp.async.wait_group %0;" ::"n"(S::kStages - 2) : "memory");
      __syncwarp();                        // every lane's part of the tile; the freed stage too
      {
        const int next = page_of(t_load + kWarps);
        int s = stage + S::kStages - 1;
        if (s >= S::kStages) s -= S::kStages;
        issue(t_load, s, page);
        page = next;
        t_load += kWarps;
      }
      const uint32_t kt = ring + stage * S::kTileBytes, vt = kt + kTile * kRow;

      float sT[NT][MT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < MT; ++u) sT[nt][u][0] = sT[nt][u][1] = sT[nt][u][2] = sT[nt][u][3] = 0.f;
      if constexpr (!kFp8) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            uint32_t a[4];
            ldsm4(kt + chunk_at<kRow>(16 * u + (lane & 15), 2 * kk + (lane >> 4)), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(sT[nt][u], a, qf[nt][kk][0], qf[nt][kk][1]);
          }
      } else {
#pragma unroll
        for (int kk = 0; kk < D / 32; ++kk)
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            uint32_t r[4];                 // rows g / g+8, bytes 4cq..4cq+3 of two 16-column steps
            ldsm4(kt + chunk_at<kRow>(16 * u + (lane & 15), 2 * kk + (lane >> 4)), r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t a[4] = {e4m3x2_to_f16x2(r[2 * i]), e4m3x2_to_f16x2(r[2 * i + 1]),
                                     e4m3x2_to_f16x2(r[2 * i] >> 16), e4m3x2_to_f16x2(r[2 * i + 1] >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma16816<true>(sT[nt][u], a, qf[nt][2 * kk + i][0], qf[nt][2 * kk + i][1]);
            }
          }
      }
      // ---- softmax over the tile's positions (rows g, g + 8 of each group), per head (columns)
      const int j0 = t * kTile + g;
      uint32_t pf[NT][MT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mt[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            sT[nt][u][i] = j0 + 16 * u + 8 * (i >> 1) < len ? sT[nt][u][i] * sc[nt][i & 1] : -INFINITY;
            mt[i & 1] = fmaxf(mt[i & 1], sT[nt][u][i]);
          }
#pragma unroll
        for (int x16 = 4; x16 < 32; x16 <<= 1) {
          mt[0] = fmaxf(mt[0], __shfl_xor_sync(0xffffffffu, mt[0], x16));
          mt[1] = fmaxf(mt[1], __shfl_xor_sync(0xffffffffu, mt[1], x16));
        }
        const bool grew = mt[0] > m[nt][0] || mt[1] > m[nt][1];
        if (__any_sync(0xffffffffu, grew)) {
          float f[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mn = fmaxf(m[nt][i], mt[i]);
            // nothing finite yet: the old sum is zero and stays so
            f[i] = m[nt][i] == -INFINITY ? 0.f : ex2_approx(m[nt][i] - mn);
            m[nt][i] = mn;
            l[nt][i] *= f[i];
          }
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            acc[nt][i][0] *= f[0];
            acc[nt][i][1] *= f[1];
            acc[nt][i][2] *= f[0];
            acc[nt][i][3] *= f[1];
          }
        }
        // weights; with e4m3 they carry 2^14, in l too
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          float w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float mm = m[nt][i & 1] == -INFINITY ? 0.f : m[nt][i & 1];
            w[i] = ex2_approx(sT[nt][u][i] - mm + (kFp8 ? 14.f : 0.f));
            l[nt][i & 1] += w[i];
          }
          pf[nt][u][0] = transpose8x8(kFp8 ? f32x2_to_f16x2(w[1], w[0]) : pack_bf16(w[0], w[1]));
          pf[nt][u][1] = transpose8x8(kFp8 ? f32x2_to_f16x2(w[3], w[2]) : pack_bf16(w[2], w[3]));
        }
      }
      // ---- O^T += V^T . P^T
      const int vr = (lane & 7) + ((lane >> 4) << 3);      // position row of the transposed load
      const int vc = (lane >> 3) & 1;
      if constexpr (!kFp8) {
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            uint32_t a[4];                 // columns 16 i + g / + 8, positions 2cq.. / + 8
            ldsm4_t(vt + chunk_at<kRow>(16 * u + vr, 2 * i + vc), a);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(acc[nt][i], a, pf[nt][u][0], pf[nt][u][1]);
          }
      } else {
#pragma unroll
        for (int u = 0; u < MT; ++u)
#pragma unroll
          for (int i = 0; i < D / 32; ++i) {
            // each register: column pair (2g, 2g+1) of a 16-column group at positions 2cq, 2cq+1
            uint32_t r[4];
            ldsm4_t(vt + chunk_at<kRow>(16 * u + vr, 2 * i + vc), r);
#pragma unroll
            for (int k2 = 0; k2 < 2; ++k2) {
              const uint32_t lo = __byte_perm(r[k2], 0, 0x3120), hi = __byte_perm(r[k2 + 2], 0, 0x3120);
              const uint32_t a[4] = {e4m3x2_to_f16x2(lo), e4m3x2_to_f16x2(lo >> 16),
                                     e4m3x2_to_f16x2(hi), e4m3x2_to_f16x2(hi >> 16)};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<true>(acc[nt][2 * i + k2], a, pf[nt][u][0], pf[nt][u][1]);
            }
          }
      }
      stage = stage + 1 == S::kStages ? 0 : stage + 1;
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");

    // ---- the warps' partial results meet in shared memory (over the idle rings)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int x16 = 4; x16 < 32; x16 <<= 1) l[nt][i] += __shfl_xor_sync(0xffffffffu, l[nt][i], x16);
        if (g == 0) {
          s_m[warp * kHeads + 8 * nt + 2 * cq + i] = m[nt][i];
          s_l[warp * kHeads + 8 * nt + 2 * cq + i] = l[nt][i];
        }
      }
    __syncthreads();                       // rings idle in every warp, m and l written
    float* s_o = reinterpret_cast<float*>(smem);            // [warp][head][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int h = 8 * nt + 2 * cq + (j & 1);
          const int d = kFp8 ? 16 * i + 2 * g + (j >> 1) : 16 * i + g + 8 * (j >> 1);
          s_o[(warp * kHeads + h) * D + d] = acc[nt][i][j];
        }
    __syncthreads();
    const bool whole = t0 == 0 && t1 == n_tiles;
    // columns d .. d+3 of the chunk's head h, and its lse
    auto finish = [&](int h, int d, const float* oo, float mm, float ll) {
      const int hq = hk * p.G + h0 + h;
      const bool none = ll == 0.f;
      const float f = none ? 0.f : vscale / ll;
#pragma unroll
      for (int i = 0; i < 4; ++i) store_o(p, b, hq, d + i, none ? 0.f : oo[i] * f);
      if (d == 0 && p.lse)
        p.lse[static_cast<int64_t>(b) * p.Hq + hq] =
            none ? -INFINITY : (mm == -INFINITY ? 0.f : mm) * kLn2 + logf(ll) - (kFp8 ? 14.f * kLn2 : 0.f);
    };
    float* slot = p.slots + (2 * static_cast<int64_t>(cta) + (t0 == 0 ? 1 : 0)) * S::kSlotFloats;
    for (int e = 4 * tid; e < nh * D; e += 4 * kThreads) {
      const int h = e / D, d = e - h * D;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * kHeads + h]);
      float ll = 0.f, oo[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = s_m[w * kHeads + h];
        // a warp with no position keeps m = -inf, l = 0, o = 0; one whose scores are all -inf
        // or NaN keeps its l and o
        const float f = mw == -INFINITY ? 1.f : ex2_approx(mw - mm);
        const float4 x = *reinterpret_cast<const float4*>(s_o + (w * kHeads + h) * D + d);
        ll += f * s_l[w * kHeads + h];
        oo[0] += f * x.x;
        oo[1] += f * x.y;
        oo[2] += f * x.z;
        oo[3] += f * x.w;
      }
      if (whole) {
        finish(h, d, oo, mm, ll);
      } else {
        *reinterpret_cast<float4*>(slot + 2 * kHeads + e) = make_float4(oo[0], oo[1], oo[2], oo[3]);
        if (d == 0) {
          slot[h] = mm;
          slot[kHeads + h] = ll;
        }
      }
    }
    if (!whole) {
      // ---- the last span to arrive joins the unit's pieces, in the spans' order
      const int64_t first = quotient(u0 + S::kUnitCost - 1, span);
      const int64_t last = quotient(u0 + n_tiles - S::kUnitCost, span);
      __syncthreads();
      if (tid == 0) {
        int* c = p.counters + first;
        __threadfence();                   // the CTA's part before its arrival
        const int seen = atomicAdd(c, 1);
        sh_last = seen == last - first;
        if (sh_last) *c = 0;               // as it was found, for the next call
        __threadfence();                   // the others' parts after theirs
      }
      __syncthreads();
      if (sh_last) {
        const int np = static_cast<int>(last - first) + 1;
        float* s_f = reinterpret_cast<float*>(smem);         // [piece][head], over the rings
        float* s_s = s_f + np * kHeads;
        // parts lie two slots apart, the first one a slot further on
        const float* parts = p.slots + 2 * first * S::kSlotFloats;
        for (int e = tid; e < np * kHeads; e += kThreads) {
          const int i = e / kHeads, h = e - i * kHeads;
          const float* sl = parts + (2 * i + (i == 0 ? 1 : 0)) * S::kSlotFloats;
          s_f[e] = h < nh ? __ldcg(sl + h) : 0.f;
          s_s[e] = h < nh ? __ldcg(sl + kHeads + h) : 0.f;
        }
        __syncthreads();
        // a warp a head, lanes over pieces
        for (int h = warp; h < nh; h += kWarps) {
          float mm = -INFINITY, ll = 0.f;
          for (int i = lane; i < np; i += 32) mm = fmaxf(mm, s_f[i * kHeads + h]);
#pragma unroll
          for (int x16 = 16; x16; x16 >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xffffffffu, mm, x16));
          for (int i = lane; i < np; i += 32) {
            const float mw = s_f[i * kHeads + h];
            const float f = mw == -INFINITY ? 1.f : ex2_approx(mw - mm);
            s_f[i * kHeads + h] = f;
            ll += f * s_s[i * kHeads + h];
          }
#pragma unroll
          for (int x16 = 16; x16; x16 >>= 1) ll += __shfl_xor_sync(0xffffffffu, ll, x16);
          if (lane == 0) {
            s_m[h] = mm;
            s_l[h] = ll;
          }
        }
        __syncthreads();
        constexpr int kEach = 4 * kThreads;  // columns the threads take at once
        for (int e0 = 4 * tid; e0 < nh * D; e0 += 2 * kEach) {
          const bool two = S::kTwo && e0 + kEach < nh * D;
          const int h = e0 / D, h2 = (e0 + kEach) / D;
          float oo[8] = {};
          for (int i0 = 0; i0 < np; i0 += S::kAhead) {       // all their loads in flight at once
            float4 x[2 * S::kAhead];       // (the odd ones unused without a second word)
#pragma unroll
            for (int i = 0; i < S::kAhead; ++i)
              if (i0 + i < np) {
                const float* at = parts + (2 * (i0 + i) + (i0 + i == 0 ? 1 : 0)) * S::kSlotFloats + 2 * kHeads + e0;
                x[2 * i] = __ldcg(reinterpret_cast<const float4*>(at));
                if (two) x[2 * i + 1] = __ldcg(reinterpret_cast<const float4*>(at + kEach));
              }
#pragma unroll
            for (int i = 0; i < S::kAhead; ++i) {
              if (i0 + i >= np) break;
              const float f = s_f[(i0 + i) * kHeads + h];
              oo[0] += f * x[2 * i].x;
              oo[1] += f * x[2 * i].y;
              oo[2] += f * x[2 * i].z;
              oo[3] += f * x[2 * i].w;
              if (!two) continue;
              const float f2 = s_f[(i0 + i) * kHeads + h2];
              oo[4] += f2 * x[2 * i + 1].x;
              oo[5] += f2 * x[2 * i + 1].y;
              oo[6] += f2 * x[2 * i + 1].z;
              oo[7] += f2 * x[2 * i + 1].w;
            }
          }
          finish(h, e0 % D, oo, s_m[h], s_l[h]);
          if (two) finish(h2, (e0 + kEach) % D, oo + 4, s_m[h2], s_l[h2]);
        }
      }
    }
    __syncthreads();                       // the rings are free for the next piece
  }
}

// SMs that calls use: all of a GB300's 152.
int sms_for(int* out) {
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  *out = sms < kMaxSms ? sms : kMaxSms;
  return MLA_OK;
}

// n-tiles of 8 query heads a unit takes: the whole group up to 32 heads, so that the cache is
// read once.  With 128-wide e4m3 rows at most 16: 32 heads' outputs and queries do not fit the
// registers next to the conversions (64 requests of 8,192 positions, 32 heads a KV head: 159 us
// in one unit, 99 in two; bf16 rows: 122 and 173).
int head_tiles(int64_t G, bool narrow) { return G <= 8 ? 1 : (G <= 16 || narrow ? 2 : 4); }
bool narrow_units(int64_t D, bool fp8) { return D == 128 && fp8; }

// Counters and slots for two CTAs a SM, which all calls of a shape fit.
size_t counters_for(int sms) { return (static_cast<size_t>(sms) * 2 * 4 + 255) / 256 * 256; }
size_t workspace_for(int sms, int64_t G, int64_t D) {
  return kHeaderBytes + counters_for(sms) +
         2 * 2 * static_cast<size_t>(sms) * 8 * head_tiles(G, false) * static_cast<size_t>(D + 2) * 4;
}

template <int D, bool kFp8, int NT, int W>
cudaError_t launch_as(const GqaDecodeParams& p, int sms, cudaStream_t stream) {
  using S = DecodeShape<D, kFp8, NT, W>;
  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!attr_set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(gqa_decode_kernel<S>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) return e;
      attr_set[dev] = true;
    }
  }
  gqa_decode_kernel<S><<<sms * S::kCtasPerSm, S::kThreads, S::kSmem, stream>>>(p);
  return cudaGetLastError();
}

// Where the units are no more than the SMs, one CTA of eight warps a SM: half the pieces to
// join, and a unit that one CTA has to itself gets a whole SM.  Otherwise two of four, one of
// which streams while the other ends a piece.  With eight and with four, us: e4m3, eight heads a
// KV head of 128, pages of 16: 2 units of 8,000 positions 12 and 19, 152 of 2,000 18 and 23, 304
// of 500 16 and 12; bf16, 8,192 units of 16 positions 156 and 90.
template <int D, bool kFp8, int NT>
cudaError_t launch(const GqaDecodeParams& p, int sms, cudaStream_t stream) {
  if (static_cast<int64_t>(p.B) * p.Hk * p.chunks <= sms) return launch_as<D, kFp8, NT, 8>(p, sms, stream);
  return launch_as<D, kFp8, NT, 4>(p, sms, stream);
}

template <int D, bool kFp8>
cudaError_t launch_nt(const GqaDecodeParams& p, int sms, cudaStream_t s) {
  constexpr bool kNarrow = D == 128 && kFp8;
  const int nt = head_tiles(p.G, kNarrow);
  if (nt == 1) return launch<D, kFp8, 1>(p, sms, s);
  if constexpr (!kNarrow)
    if (nt == 4) return launch<D, kFp8, 4>(p, sms, s);
  return launch<D, kFp8, 2>(p, sms, s);
}

}  // namespace

extern "C" int mla_get_gqa_decode_workspace_size(int32_t batch_size, int32_t num_heads,
                                                 int32_t num_kv_heads, int32_t head_dim,
                                                 int32_t num_sms, size_t* bytes_out) {
  if (!bytes_out || batch_size < 0 || num_heads < 1 || num_kv_heads < 1 || num_heads > 1024 ||
      num_heads % num_kv_heads != 0 || head_dim < 1 || num_sms > 65536)
    return MLA_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return MLA_ERR_UNSUPPORTED;
  int sms = num_sms;
  if (num_sms <= 0) {
    const int st = sms_for(&sms);
    if (st != MLA_OK) return st;
  }
  *bytes_out = workspace_for(sms, num_heads / num_kv_heads, head_dim);
  return MLA_OK;
}

extern "C" int mla_gqa_decode(const mla_tensor_t* q, const mla_tensor_t* k_cache,
                              const mla_tensor_t* v_cache, const mla_tensor_t* o,
                              const mla_tensor_t* kv_indptr, const mla_tensor_t* kv_indices,
                              const mla_tensor_t* kv_last_page_lens, float sm_scale,
                              const mla_tensor_t* k_scale, const mla_tensor_t* v_scale,
                              const mla_tensor_t* lse_out, void* workspace, size_t workspace_bytes,
                              mla_stream_t stream_) {
  if (!q || !k_cache || q->ndim != 3 || k_cache->ndim != 4) return MLA_ERR_INVALID_ARG;
  const int64_t B = q->shape[0], Hq = q->shape[1], D = q->shape[2], Hk = k_cache->shape[2];
  if (B < 0 || B > 0xFFFFFF || Hq < 1 || Hq > 1024 || Hk < 1 || Hq % Hk != 0) return MLA_ERR_INVALID_ARG;
  if (!gqa_check_bf16(q, B, Hq, D, 8)) return MLA_ERR_INVALID_ARG;
  GqaCache c;
  const int st = gqa_check_cache(k_cache, v_cache, k_scale, v_scale, Hk, D, &c);
  if (st != MLA_OK) return st;
  if (!o || (!o->ptr && B > 0) || o->ndim != 3 || (o->dtype != MLA_DTYPE_BF16 && o->dtype != MLA_DTYPE_FP32) ||
      o->shape[0] != B || o->shape[1] != Hq || o->shape[2] != D || o->stride[2] != 1 ||
      o->stride[0] < 0 || o->stride[1] < 0 || !gqa_rows_apart(o) ||
      !gqa_aligned(o->ptr, o->dtype == MLA_DTYPE_FP32 ? 4 : 2))
    return MLA_ERR_INVALID_ARG;
  if (!gqa_check_i32(kv_indptr, B + 1)) return MLA_ERR_INVALID_ARG;
  if (!kv_indices || kv_indices->ndim != 1 || !gqa_check_i32(kv_indices, kv_indices->shape[0]))
    return MLA_ERR_INVALID_ARG;
  if (c.log2_page > 0 && !kv_last_page_lens) return MLA_ERR_INVALID_ARG;
  if (kv_last_page_lens && !gqa_check_i32(kv_last_page_lens, B)) return MLA_ERR_INVALID_ARG;
  if (lse_out && ((!lse_out->ptr && B > 0) || lse_out->dtype != MLA_DTYPE_FP32 || lse_out->ndim != 2 ||
                  lse_out->shape[0] != B || lse_out->shape[1] != Hq || (Hq > 1 && lse_out->stride[1] != 1) ||
                  (B > 1 && lse_out->stride[0] != Hq) || !gqa_aligned(lse_out->ptr, 4)))
    return MLA_ERR_INVALID_ARG;
  if (!(sm_scale == sm_scale)) return MLA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return MLA_ERR_UNSUPPORTED;
  if (!workspace || !gqa_aligned(workspace, 256)) return MLA_ERR_INVALID_ARG;
  const int64_t G = Hq / Hk;
  if (workspace_bytes < workspace_for(1, G, D)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  const int cs = sms_for(&sms);
  if (cs != MLA_OK) return cs;
  if (workspace_bytes < workspace_for(sms, G, D)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (B == 0) return MLA_OK;

  GqaDecodeParams p;
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
  p.k_scale = c.k_scale;
  p.v_scale = c.v_scale;
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
  const int heads = 8 * head_tiles(G, narrow_units(D, c.fp8));
  p.chunks = static_cast<int>((G + heads - 1) / heads);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.err = reinterpret_cast<int*>(ws);
  p.counters = reinterpret_cast<int*>(ws + kHeaderBytes);
  p.slots = reinterpret_cast<float*>(ws + kHeaderBytes + counters_for(sms));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e;
  if (D == 64) e = c.fp8 ? launch_nt<64, true>(p, sms, s) : launch_nt<64, false>(p, sms, s);
  else e = c.fp8 ? launch_nt<128, true>(p, sms, s) : launch_nt<128, false>(p, sms, s);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
