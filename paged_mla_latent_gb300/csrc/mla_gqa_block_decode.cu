// mla_gqa_block_decode: attention of a request's newest tokens over a paged e4m3 cache with a
// scale for each block of positions and head, split over the cache's length and joined in the
// same launch.
//
//   s_j = sm_scale * kscale(j) * q . kcode_j,   o = sum_j e^{s_j - lse} vscale(j) vcode_j,
//   lse = ln sum_j e^{s_j}, over the positions that the row sees, for the T G query rows of a KV
//   head (T new tokens, G = Hq / Hk query heads).
//
// Work split as in mla_gqa_decode: a unit is (request, KV heads, chunk of 8 NT rows of each), its
// positions are cut into tiles, all units lie on one line, each as long as its tiles and a fixed
// cost, and every CTA takes an equal span.  A unit that crosses a span's end leaves partials (m, l,
// o in fp32) in workspace slots, joined in the order of the spans by the CTA that arrives last.
//
// Inside a CTA the warps take tiles in turn, each with its own rings of cp.async stages for keys and
// for values, its own reference m, sum and output, and no barrier until the span's piece ends.
//   S^T (16 positions x 8 rows) = K (16 x D) . q^T by mma.sync m16n8k16 in f16, into which e4m3
//   converts exactly: positions are the MMA's M, so that eight query rows fill its N (tcgen05's
//   smallest M of 64 rows would be mostly padding).  q's rows are scaled by a power of two to a
//   maximum in [2^13, 2^14) (bf16's 8 bits fit f16's 11; what falls below f16's range is under
//   2^-38 of the row's maximum).  O^T (D x 8) += V^T . P^T, whose fragments come from S^T's by one
//   8x8 transpose (movmatrix).
// The scale of a position's values goes into its weight's exponent: a_j = log2(e) s_j + log2 vscale(j)
// and P_j = 2^(a_j - max + 14), rounded to f16 (2^-11), while the sum takes P_j / vscale(j) in fp32;
// what falls under f16's range is below 2^-38 of the largest.
// 64-wide heads are taken in pairs, 128 bytes of a slot at a time: alone they use half of every
// line that DRAM delivers (64 requests of 32,768 positions, two heads: 170 us alone, 103 paired).
// A unit has at most 16 rows of each head.  More go to the kernel of mla_gqa_block_wide.cu, which feeds
// the codes to tcgen05 (64 requests of 2,048 to 65,536 positions, four tokens of eight heads: 116
// us), or, where the cache's layout is none for it, run here in units of 16 that read the cache again
// (187; 32 rows in one unit fit the registers with nothing beside them: 209).
//
// With several new tokens a NaN among their values must not reach rows that do not see it (zero times
// NaN): edge tiles are looked over, and rows marked at a piece's end (64 requests of 8,192, two tokens of
// eight heads: 65.5 us, 63 without).
//
// Measured (one GB300, in a CUDA graph): 64 requests of 2,048 to 65,536 positions, 16/2 heads of 128, 507
// MB: 86 us, 5.9 TB/s (0.88 of the copy rate); one of 142,000, 64/8 heads: 56 us, of which 44 stream the
// cache and the rest are the plan, the first tiles and the join; 37 of up to 4,089, 20/4 heads of 64: 12
// us; one of 137, 32/8 heads: 6.2 us.
//
// Also tried: e4m3 MMAs (m16n8k32) with q and P as two codes each, whose operands the compiler
// converts to f16 all the same (102 us for 64 requests of 16,384 positions, two KV heads; 91 as
// it is); sixteen warps of half the registers (100); the next tile's scores ahead of this one's
// weights (101); a reference that moves only where a score passes it by 6 (100).
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/paged_mla.h"
#include "mla_gqa_check.h"
#include "mla_gqa_block_decode.cuh"
#include "mla_gqa_decode_common.cuh"
#include "ptx.cuh"

namespace {

using namespace pmla;

constexpr int64_t kMaxQ = 64;        // as mla_decode
constexpr int kSmWarps = 8;          // warps a SM, in two CTAs or in one
constexpr float kShift = 14.f;       // weights carry 2^14, in the sum too

__device__ __forceinline__ void cp_async_4(uint32_t dst, const float* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Two pairs of e4m3 codes as two of f16 values.
__device__ __forceinline__ void e4m3x4_to_f16(uint32_t codes, uint32_t& lo, uint32_t& hi) {
  asm("{\n.reg .b16 a, b;\nmov.b32 {a, b}, %2;\ncvt.rn.f16x2.e4m3x2 %0, a;\ncvt.rn.f16x2.e4m3x2 %1, b;\n}"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

// D columns, n-tiles of 8 query rows of a head, KV heads a unit, warps a CTA, whether a request may
// have several new tokens.
template <int D_, int NT_, int HP_, int W_, bool kMany_>
struct BlockShape {
  static constexpr int D = D_, NT = NT_, HP = HP_;
  static constexpr bool kMany = kMany_;
  static constexpr int CT = NT * HP;                       // column tiles of 8 rows
  static constexpr int kWarps = W_, kThreads = 32 * W_;
  static constexpr int kJoinWarps = kWarps, kJoinThreads = kThreads;
  __device__ static __forceinline__ void join_sync() { __syncthreads(); }
  static constexpr int kCtasPerSm = kSmWarps / W_;
  static constexpr int kMaxCtas = kMaxSms * kCtasPerSm;    // a unit has at most one piece a CTA
  static constexpr int kRow = D * HP;                      // bytes of a K or V row
  static_assert(CT <= 4 && (kRow == 64 || kRow == 128), "registers, and the swizzles");
  // positions a warp takes at a time, in groups of 16 (the MMA's M)
  static constexpr int MT = 2, kTile = 16 * MT;
  static constexpr int kTileBytes = 2 * kTile * kRow;      // K then V
  static constexpr int kStageBytes = kTileBytes + 8 * kTile * HP;  // and their scales
  // tiles that a warp has room for, about 24 KB (eight warps a SM: 192 KB)
  static constexpr int kStages = 24576 / kTileBytes < 8 ? 24576 / kTileBytes : 8;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kHeads = 8 * NT, kRows = 8 * CT;    // rows of a head, of a unit
  static constexpr int kJoinBytes = kWarps * kRows * D * 4;        // per-warp outputs, over the rings
  static constexpr int kPieceBytes = 2 * kMaxCtas * kRows * 4;     // m and l of a unit's pieces, over them too
  static constexpr int kOverBytes = kJoinBytes > kPieceBytes ? kJoinBytes : kPieceBytes;
  static constexpr int kBuf = kWarps * kWarpBytes > kOverBytes ? kWarps * kWarpBytes : kOverBytes;
  static constexpr int kSmem = kBuf + 2 * kWarps * kRows * 4 + kRows * D * 2 + kRows * 4 + (kMany ? sizeof(NanMarks) : 0);
  static_assert(kCtasPerSm * (kSmem + 1024 + 64) <= 233472, "shared memory of a SM");
  static constexpr int kSlotFloats = kRows * (D + 2);
  static constexpr bool kTwo = kRows * D > 4 * kThreads;   // a join's thread has two words of o
  static constexpr int kAhead = CT == 4 ? 4 : (kTwo ? 10 : 20);    // pieces whose words are in flight
  // what a unit costs besides its tiles (page ids, the first tile's way from DRAM, the joins), in
  // tiles: 7 us at a SM's share of the bandwidth where CTAs have many tiles, a tenth of what they
  // have but at least 1.2 us where they have few.  64 requests of 2,048 to 65,536 positions, two KV
  // heads of 128: 95 us with 1.2 us, 88 with 5, 86.5 with 7, 86.5 with 10; one of 142,000, eight KV
  // heads: 57, 63, 57; 37 of up to 4,089: 12.9, 14.7, 15.4 (13.0 with the tenth).  CTAs of four warps,
  // 256 requests of 500 to 4,000: 170 us with 55 KB's time, 164 with 100, 159 with 150, 167 with 250.
  static constexpr int kUnitCost = (W_ == 8 ? 350000 : 150000) / kTileBytes, kLeastCost = 55000 / kTileBytes;
  static constexpr int kLeastPiece = 55000 / kTileBytes;   // of a cut unit
};

// q's rows in f16, scaled, into shared memory, their columns in the order in which K's
// fragments hold theirs: of 16 columns lane cq has 4 cq .. 4 cq + 3.  sc: each row's factor
// from a product to a score in units of log2.
template <class S>
__device__ __forceinline__ void stage_queries(const BlockDecodeParams& p, const Piece& u, uint8_t* s_q, float* s_sc,
                                              int warp, int lane) {
  constexpr int kLanes = S::D / 4;
  for (int ur = warp; ur < S::kRows; ur += S::kWarps) {
    const int hk = u.hk0 + ur / S::kHeads, h = ur % S::kHeads;
    const bool live = h < u.nh && hk < p.Hk;
    const int r = u.h0 + (live ? h : 0), of = r / p.G;     // the row's token
    const uint16_t* row = p.q + (u.tok0 + of) * p.q_tok +
                          (static_cast<int64_t>(live ? hk : u.hk0) * p.G + r - of * p.G) * p.q_head;
    uint2 w = make_uint2(0, 0);
    if (live && lane < kLanes) w = __ldg(reinterpret_cast<const uint2*>(row) + lane);
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t x = i ? w.y : w.x;
      mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(x << 16)), fabsf(__uint_as_float(x & 0xFFFF0000u))));
    }
    mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
    int e = 267 - static_cast<int>(__float_as_uint(mx) >> 23);     // 2^(13 - exponent), biased
    e = e > 253 ? 253 : e;
    const float up = __uint_as_float(static_cast<uint32_t>(e) << 23);
    const float down = __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
    if (lane < kLanes) {
      uint8_t* at = s_q + ur * S::D * 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x = i ? w.y : w.x;
        const int chunk = 2 * (lane >> 2) + i;
        *reinterpret_cast<uint32_t*>(at + ((chunk ^ (ur & 7)) << 4) + 4 * (lane & 3)) =
            f32x2_to_f16x2(__uint_as_float(x & 0xFFFF0000u) * up, __uint_as_float(x << 16) * up);
      }
    }
    if (lane == 0) s_sc[ur] = p.sm_scale * kLog2e * down;
  }
}

// New tokens' values that are NaN, of a tile's rows that not all query rows see: marked.
template <class S>
__device__ __noinline__ void clean_values(uint8_t* v, float* scales, NanMarks* marks, int at0, int from, int end, int lane) {
  constexpr int kChunks = S::kRow / 16, kTile = S::kTile;
  if (from < 0) from = 0;
  if (end > kTile) end = kTile;
#pragma unroll 1
  for (int e = kChunks * from + lane; e < kChunks * end; e += 32)
    marks->look(reinterpret_cast<uint4*>(v + chunk_at<S::kRow>(e / kChunks, e % kChunks)), at0 + e / kChunks, 16 * (e % kChunks));
  if (lane >= from && lane < end)
    for (int hp = 0; hp < S::HP; ++hp) marks->look(scales + hp * kTile + lane, at0 + lane, hp);
}

// The warp's tiles of a piece: output, maximum and sum of its rows (o's columns 16 i + 2 g and
// the next of rows 2 cq, 2 cq + 1 of each column tile; m and l of those rows, l per lane).
template <class S>
__device__ __forceinline__ void walk_tiles(const BlockDecodeParams& p, const Piece& u, uint8_t* smem, uint8_t* s_q,
                                           float* s_sc, NanMarks* marks, int warp, int lane, float (&acc)[S::CT][S::D / 16][4],
                                           float (&m)[S::CT][2], float (&l)[S::CT][2]) {
  constexpr int D = S::D, NT = S::NT, HP = S::HP, CT = S::CT, MT = S::MT, kTile = S::kTile, kRow = S::kRow;
  constexpr int kStages = S::kStages;
  const int g = lane >> 2, cq = lane & 3;
  uint8_t* const ring_ptr = smem + warp * S::kWarpBytes;
  const uint32_t ring = smem_u32(ring_ptr);
  const int first = u.t0 + warp;
  const int len = u.r.len;

  // ---- loads of a tile: its page ids a tile ahead, then 16-byte cp.asyncs
  const int ps_mask = (1 << p.pages.log2_page) - 1;
  const bool one_page = (1 << p.pages.log2_page) >= kTile;      // a tile never crosses a page
  constexpr int kChunks = kRow / 16, kRowsAt = 32 / kChunks;
  const int lc = lane % kChunks, lr = lane / kChunks;
  const int lane_head = u.hk0 + lc / (D / 16);             // KV head of the lane's 16 bytes
  const int64_t lane_off = lane_head * p.head_pitch + 16 * (lc % (D / 16));
  const bool lane_live = HP == 1 || lane_head < p.Hk;
  auto page_of = [&](int t) -> int {       // lane's page id for tile t (-1: no position)
    const int j = t * kTile + (one_page ? 0 : lane);
    return t < u.t1 && j < len ? __ldg(p.pages.indices + u.idx0 + (j >> p.pages.log2_page)) : -1;
  };
  auto load = [&](int t, int stage, int page) {
    if (t < u.t1) {
      const uint32_t dst = ring + stage * S::kStageBytes;
      const int at0 = t * kTile;
      const bool ok = page >= 0 && page < p.n_pages;
      if (one_page) {
        if (!ok && lane == 0) atomicOr(p.err, kErrBadRowId);     // reads as zeros
        const int rows = ok && lane_live ? len - at0 : 0;
        int64_t at = rows > 0 ? page * p.page_pitch + ((at0 & ps_mask) + lr) * p.slot_pitch + lane_off : 0;
#pragma unroll
        for (int k = 0; k < kTile / kRowsAt; ++k) {
          const int r = k * kRowsAt + lr;
          const uint32_t n = r < rows ? 16u : 0u;
          const uint32_t d = dst + chunk_at<kRow>(r, lc);
          cp_async_16(d, p.k + (n ? at : 0), n);
          cp_async_16(d + kTile * kRow, p.v + (n ? at : 0), n);
          at += kRowsAt * p.slot_pitch;
        }
      } else {
        const int j = at0 + (lane);
        int64_t off = -1;
        if (j < len) {
          if (ok) off = page * p.page_pitch + (j & ps_mask) * p.slot_pitch;
          else atomicOr(p.err, kErrBadRowId);
        }
#pragma unroll
        for (int k = 0; k < kTile / kRowsAt; ++k) {
          const int r = k * kRowsAt + lr;
          const int64_t ro = __shfl_sync(0xffffffffu, off, r);
          const uint32_t n = ro >= 0 && lane_live ? 16u : 0u;
          const int64_t at = n ? ro + lane_off : 0;
          const uint32_t d = dst + chunk_at<kRow>(r, lc);
          cp_async_16(d, p.k + at, n);
          cp_async_16(d + kTile * kRow, p.v + at, n);
        }
      }
      // the scales of the tile's positions, head by head K's, then V's
#pragma unroll
      for (int e0 = 0; e0 < 2 * HP * kTile; e0 += 32) {
        const int e = e0 + lane, hp = e / kTile % HP, j = at0 + (lane);
        const bool there = ok && j < len && u.hk0 + hp < p.Hk;
        const int64_t at = there ? page * p.sc_page + ((j & ps_mask) >> p.log2_block) * p.sc_block +
                                       static_cast<int64_t>(u.hk0 + hp) * p.sc_head : 0;
        cp_async_4(dst + S::kTileBytes + 4 * e, (e < HP * kTile ? p.ks : p.vs) + at, there ? 4u : 0u);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  int t_load = first, page;
  {
    int ahead[kStages];                    // the first tiles' page ids, read together
#pragma unroll
    for (int i = 0; i < kStages; ++i) ahead[i] = page_of(t_load + i * S::kWarps);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load(t_load + i * S::kWarps, i, ahead[i]);
    t_load += (kStages - 1) * S::kWarps;
    page = ahead[kStages - 1];
  }
  stage_queries<S>(p, u, s_q, s_sc, warp, lane);
  if constexpr (S::kMany) marks->clear(32 * warp + lane, S::kThreads);
  __syncthreads();
  uint32_t qf[CT][D / 32][4];              // of two 16-column steps
  float sc[CT][2];                         // of rows 2 cq, 2 cq + 1
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk)
      ldsm4(smem_u32(s_q) + (8 * ct + (lane & 7)) * D * 2 + (((4 * kk + (lane >> 3)) ^ (lane & 7)) << 4), qf[ct][kk]);
    sc[ct][0] = s_sc[8 * ct + 2 * cq];
    sc[ct][1] = s_sc[8 * ct + 2 * cq + 1];
  }
  const int least = len - u.r.tokens + 1;  // positions that the first token sees

  int stage = 0;
#pragma unroll 1
  for (int t = first; t < u.t1; t += S::kWarps) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
    __syncwarp();                          // every lane's part of the tile; the freed stage too
    {
      const int next = page_of(t_load + S::kWarps);
      load(t_load, stage == 0 ? kStages - 1 : stage - 1, page);
      page = next;
      t_load += S::kWarps;
    }
    const uint32_t kt = ring + stage * S::kStageBytes, vt = kt + kTile * kRow;
    float* scales = reinterpret_cast<float*>(ring_ptr + stage * S::kStageBytes + S::kTileBytes);
    if constexpr (S::kMany)
      if ((t + 1) * kTile > least) {
        const int at0 = t * kTile;
        clean_values<S>(ring_ptr + (stage * S::kStageBytes + kTile * kRow), scales + HP * kTile, marks, at0, least - at0, len - at0, lane);
        __syncwarp();
      }
    stage = stage + 1 == kStages ? 0 : stage + 1;

    float s[CT][MT][4];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) s[ct][mt][0] = s[ct][mt][1] = s[ct][mt][2] = s[ct][mt][3] = 0.f;
#pragma unroll
    for (int hp = 0; hp < HP; ++hp)
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          uint32_t r[4];                   // rows g / g+8, bytes 4cq..4cq+3 of two 16-column steps
          ldsm4(kt + chunk_at<kRow>(16 * mt + (lane & 15), hp * (D / 16) + 2 * kk + (lane >> 4)), r);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t a[4];
            e4m3x4_to_f16(r[2 * i], a[0], a[2]);
            e4m3x4_to_f16(r[2 * i + 1], a[1], a[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<true>(s[hp * NT + nt][mt], a, qf[hp * NT + nt][kk][2 * i], qf[hp * NT + nt][kk][2 * i + 1]);
          }
        }
      }
    // ---- softmax over the tile's positions (rows g, g + 8 of each group), per row of q (columns).
    // The scale of v goes into the weights' exponents, so that their maximum bounds weight times
    // scale; the sum takes the weights without it.
    float ksc[HP][MT][2], lvs[HP][MT][2], rvs[HP][MT][2];
#pragma unroll
    for (int hp = 0; hp < HP; ++hp)
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ksc[hp][mt][k] = scales[hp * kTile + 16 * mt + 8 * k + g];
          const float x = scales[(HP + hp) * kTile + 16 * mt + 8 * k + g];
          const float y = x < kLeastScale ? kLeastScale : x;
          lvs[hp][mt][k] = lg2_approx(y);
          rvs[hp][mt][k] = rcp_approx(y);
        }
    const int j0 = t * kTile;
    uint32_t pf[CT][MT][2];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          s[ct][mt][k] = fmaf(s[ct][mt][k] * ksc[ct / NT][mt][k >> 1], sc[ct][k & 1], lvs[ct / NT][mt][k >> 1]);
      if (j0 + kTile > least) {            // causal among the new tokens, and the list's end
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int lim = least + (u.h0 + 8 * (ct % NT) + 2 * cq + k) / p.G;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if (j0 + 16 * mt + g >= lim) s[ct][mt][k] = -INFINITY;
            if (j0 + 16 * mt + 8 + g >= lim) s[ct][mt][k + 2] = -INFINITY;
          }
        }
      }
      float top[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        top[k] = fmaxf(fmaxf(s[ct][0][k], s[ct][0][k + 2]), fmaxf(s[ct][1][k], s[ct][1][k + 2]));
      }
#pragma unroll
      for (int d = 4; d < 32; d <<= 1) {
        top[0] = fmaxf(top[0], __shfl_xor_sync(0xffffffffu, top[0], d));
        top[1] = fmaxf(top[1], __shfl_xor_sync(0xffffffffu, top[1], d));
      }
      if (__any_sync(0xffffffffu, top[0] > m[ct][0] || top[1] > m[ct][1])) {
        float f[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float to = fmaxf(m[ct][k], top[k]);
          // nothing finite yet: the old sum is zero and stays so
          f[k] = m[ct][k] == -INFINITY ? 0.f : ex2_approx(m[ct][k] - to);
          m[ct][k] = to;
          l[ct][k] *= f[k];
        }
#pragma unroll
        for (int d = 0; d < D / 16; ++d)
#pragma unroll
          for (int k = 0; k < 4; ++k) acc[ct][d][k] *= f[k & 1];
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        float w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float mm = m[ct][k & 1] == -INFINITY ? 0.f : m[ct][k & 1];
          w[k] = ex2_approx(s[ct][mt][k] - mm + kShift);
          l[ct][k & 1] = fmaf(w[k], rvs[ct / NT][mt][k >> 1], l[ct][k & 1]);
        }
        pf[ct][mt][0] = transpose8x8(f32x2_to_f16x2(w[1], w[0]));
        pf[ct][mt][1] = transpose8x8(f32x2_to_f16x2(w[3], w[2]));
      }
    }
    // ---- O^T += V^T . P^T
    const int vr = (lane & 7) + ((lane >> 4) << 3);        // position row of the transposed load
    const int vc = (lane >> 3) & 1;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int hp = 0; hp < HP; ++hp)
#pragma unroll
        for (int d = 0; d < D / 32; ++d) {
          // each register: column pair (2g, 2g+1) of a 16-column group at positions 2cq, 2cq+1
          uint32_t r[4];
          ldsm4_t(vt + chunk_at<kRow>(16 * mt + vr, hp * (D / 16) + 2 * d + vc), r);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            uint32_t a[4];
            e4m3x4_to_f16(__byte_perm(r[k], 0, 0x3120), a[0], a[1]);
            e4m3x4_to_f16(__byte_perm(r[k + 2], 0, 0x3120), a[2], a[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              mma16816<true>(acc[hp * NT + nt][2 * d + k], a, pf[hp * NT + nt][mt][0], pf[hp * NT + nt][mt][1]);
          }
        }
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, S::kCtasPerSm) gqa_block_decode_kernel(const BlockDecodeParams p) {
  constexpr int D = S::D, HP = S::HP, CT = S::CT, kRows = S::kRows, kWarps = S::kWarps, kThreads = S::kThreads;
  extern __shared__ __align__(128) uint8_t smem[];
  float* s_m = reinterpret_cast<float*>(smem + S::kBuf);       // [warp][row]
  float* s_l = s_m + kWarps * kRows;
  float* s_sc = s_l + kWarps * kRows;                          // [row]
  uint8_t* s_q = reinterpret_cast<uint8_t*>(s_sc + kRows);     // [row][D], f16
  NanMarks* marks = reinterpret_cast<NanMarks*>(s_q + kRows * D * 2);      // of the piece
  __shared__ SpanShared<kWarps> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, cq = lane & 3;
  Span span;
  if (!find_span<S>(p, &sh, &span)) return;

  for (int64_t x = span.begin; x < span.end;) {
    Piece u;
    if (!next_piece<S>(p, span, &x, &u)) continue;
    float acc[CT][D / 16][4], m[CT][2], l[CT][2];
#pragma unroll
    for (int ct = 0; ct < CT; ++ct) {
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[ct][i][j] = 0.f;
      m[ct][0] = m[ct][1] = -INFINITY;
      l[ct][0] = l[ct][1] = 0.f;
    }
    walk_tiles<S>(p, u, smem, s_q, s_sc, marks, warp, lane, acc, m, l);

    // ---- the warps' partial results meet in shared memory (over the idle rings)
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[ct][i] += __shfl_xor_sync(0xffffffffu, l[ct][i], d);
        if (g == 0) {
          s_m[warp * kRows + 8 * ct + 2 * cq + i] = m[ct][i] - kShift;
          s_l[warp * kRows + 8 * ct + 2 * cq + i] = l[ct][i];
        }
      }
    __syncthreads();                       // rings idle in every warp, m and l written
    float* s_o = reinterpret_cast<float*>(smem);            // [warp][row][D]
#pragma unroll
    for (int ct = 0; ct < CT; ++ct)
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)        // columns 16 i + 2 g and the next
          *reinterpret_cast<float2*>(s_o + (warp * kRows + 8 * ct + 2 * cq + j) * D + 16 * i + 2 * g) =
              make_float2(acc[ct][i][j], acc[ct][i][j + 2]);
    __syncthreads();
    const bool whole = u.t0 == 0 && u.t1 == u.n_tiles;
    const int used = HP == 1 ? u.nh : u.live_rows;           // rows to look at
    float* slot = part_slot<S>(p, u);
    for (int e = 4 * tid; e < used * D; e += 4 * kThreads) {
      const int h = e / D, d = e - h * D;
      if (!row_there<S>(u, h)) continue;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w * kRows + h]);
      float ll = 0.f, oo[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float mw = s_m[w * kRows + h];
        // a warp with no position keeps m = -inf, l = 0, o = 0; one whose scores are all -inf
        // or NaN keeps its l and o
        const float f = mw == -INFINITY ? 1.f : ex2_approx(mw - mm);
        const float4 y = *reinterpret_cast<const float4*>(s_o + (w * kRows + h) * D + d);
        ll += f * s_l[w * kRows + h];
        oo[0] += f * y.x;
        oo[1] += f * y.y;
        oo[2] += f * y.z;
        oo[3] += f * y.w;
      }
      if constexpr (S::kMany)
        if (marks->any) {
          const int hp = h / S::kHeads, seen = u.r.len - u.r.tokens + 1 + (u.h0 + h % S::kHeads) / p.G;
          for (int i = 0; i < 4; ++i)
            if (marks->reach(hp * D + d + i, hp, seen)) oo[i] = NAN;
          if (marks->scale[hp] < seen) ll = NAN;
        }
      if (whole) {
        finish_row<S, 4>(p, u, h, d, oo, mm, ll);
      } else {
        *reinterpret_cast<float4*>(slot + 2 * kRows + e) = make_float4(oo[0], oo[1], oo[2], oo[3]);
        if (d == 0) {
          slot[h] = mm;
          slot[kRows + h] = ll;
        }
      }
    }
    if (!whole) join_parts<S>(p, span, u, &sh, s_m, s_l, s_o);
    __syncthreads();                       // the rings are free for the next piece
  }
}

// n-tiles of 8 query rows that a unit takes of each of its KV heads.
int row_tiles(int64_t rows) { return rows <= 8 ? 1 : 2; }
// KV heads a unit: 64-wide ones in pairs.
int unit_heads(int64_t D, int64_t Hk) { return D == 64 && Hk > 1 ? 2 : 1; }

// Counters and slots for two CTAs a SM, which all calls of a shape fit.
size_t counters_for(int sms) { return (static_cast<size_t>(sms) * 2 * 4 + 255) / 256 * 256; }
size_t workspace_for(int sms, int64_t rows, int64_t D, int64_t Hk) {
  return kHeaderBytes + counters_for(sms) +
         2 * 2 * static_cast<size_t>(sms) * 8 * row_tiles(rows) * unit_heads(D, Hk) * static_cast<size_t>(D + 2) * 4;
}

template <int D, int NT, int HP, int W, bool kMany>
cudaError_t launch_as(const BlockDecodeParams& p, int sms, cudaStream_t stream) {
  using S = BlockShape<D, NT, HP, W, kMany>;
  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!attr_set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(gqa_block_decode_kernel<S>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) return e;
      attr_set[dev] = true;
    }
  }
  gqa_block_decode_kernel<S><<<sms * S::kCtasPerSm, S::kThreads, S::kSmem, stream>>>(p);
  return cudaGetLastError();
}

// Where the units are no more than the SMs, one CTA of eight warps a SM: half the pieces to
// join, and a unit that one CTA has to itself gets a whole SM.  Otherwise two of four, one of
// which streams while the other ends a piece.
template <int D, int NT, int HP>
cudaError_t launch(const BlockDecodeParams& p, int sms, cudaStream_t stream) {
  const int64_t rows = static_cast<int64_t>(p.G) * p.max_q;
  const int64_t units = static_cast<int64_t>(p.B) * ((p.Hk + HP - 1) / HP) * ((rows + 8 * NT - 1) / (8 * NT));
  // (One new token sees all positions: without the marks of those that others do not.)
  if (units <= sms) return p.max_q == 1 ? launch_as<D, NT, HP, 8, false>(p, sms, stream) : launch_as<D, NT, HP, 8, true>(p, sms, stream);
  return p.max_q == 1 ? launch_as<D, NT, HP, 4, false>(p, sms, stream) : launch_as<D, NT, HP, 4, true>(p, sms, stream);
}

template <int D, int HP>
cudaError_t launch(const BlockDecodeParams& p, int sms, cudaStream_t s) {
  const int nt = row_tiles(static_cast<int64_t>(p.G) * p.max_q);
  return nt == 1 ? launch<D, 1, HP>(p, sms, s) : launch<D, 2, HP>(p, sms, s);
}
cudaError_t launch(const BlockDecodeParams& p, int64_t D, int sms, cudaStream_t s) {
  if (block_wide_takes(p, D)) return launch_block_wide(p, D, sms, s);
  if (D == 128) return launch<128, 1>(p, sms, s);
  // Pairs halve the units, which costs where caches lie in L2: one head each where the page list has
  // room for no more than 32 MB (37 requests of up to 4,089 positions, four heads: 11.5 us alone,
  // 13.0 in pairs; 64 of 16,384, two heads: 77 and 62).  The lengths themselves are the device's, so
  // that a list with room to spare counts as long, and gets pairs.
  const bool small = (p.pages.n_idx << p.pages.log2_page) * p.Hk * 2 * D <= 32 << 20;
  return unit_heads(D, p.Hk) == 2 && !small ? launch<64, 2>(p, sms, s) : launch<64, 1>(p, sms, s);
}

}  // namespace

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
  *bytes_out = workspace_for(sms, static_cast<int64_t>(num_heads / num_kv_heads) * max_seqlen_q, head_dim, num_kv_heads);
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
  if (workspace_bytes < workspace_for(1, rows, D, Hk)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  int sms = 0;
  const int cs = sms_for(&sms);
  if (cs != MLA_OK) return cs;
  if (workspace_bytes < workspace_for(sms, rows, D, Hk)) return MLA_ERR_WORKSPACE_TOO_SMALL;
  if (B == 0 || T == 0) return MLA_OK;

  BlockDecodeParams p = {};
  p.q = static_cast<const uint16_t*>(q->ptr);
  p.q_tok = q->stride[0];
  p.q_head = q->stride[1];
  p.k = c.k;
  p.v = c.v;
  p.page_pitch = c.page_pitch;
  p.slot_pitch = c.slot_pitch;
  p.head_pitch = c.head_pitch;
  p.ks = c.ks;
  p.vs = c.vs;
  p.sc_page = c.sc_page;
  p.sc_block = c.sc_block;
  p.sc_head = c.sc_head;
  p.log2_block = c.log2_block;
  p.n_pages = c.n_pages;
  p.pages.indptr = static_cast<const int32_t*>(kv_indptr->ptr);
  p.pages.indices = static_cast<const int32_t*>(kv_indices->ptr);
  p.pages.last = kv_last_page_lens ? static_cast<const int32_t*>(kv_last_page_lens->ptr) : nullptr;
  p.pages.n_idx = kv_indices->shape[0];
  p.pages.log2_page = c.log2_page;
  p.qo_indptr = static_cast<const int32_t*>(qo_indptr->ptr);
  p.n_tok = T;
  p.max_q = max_seqlen_q;
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
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.err = reinterpret_cast<int*>(ws);
  p.counters = reinterpret_cast<int*>(ws + kHeaderBytes);
  p.slots = reinterpret_cast<float*>(ws + kHeaderBytes + counters_for(sms));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  return launch(p, D, sms, s) == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
