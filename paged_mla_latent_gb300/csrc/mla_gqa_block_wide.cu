// mla_gqa_block_decode for many query rows a KV head (several new tokens, large groups): the products
// on tcgen05 straight from the cache's e4m3 codes.  The work's split, the units on their line and the
// join of pieces are the narrow kernel's (mla_gqa_block_decode.cu); a unit has up to 32 rows of one
// 128-wide head, or 16 of each of a pair of 64-wide ones, whose 128 bytes of a slot are one row of a
// tile: more rows of a head are more units, each of which reads the cache again.
//
// A tile is 128 positions: the MMA's M (tensor memory's lanes).
//   S^T (128 x 64) = K (128 x 128 bytes) . q^T, a head's rows as two e4m3 planes side by side in N:
//     q up = high + 2^-5 low, its largest in [2^7, 2^8): bf16's eight bits are four and four, and what
//     is lost is below 2^-22 of the row's largest.  A head of a pair takes its 64 bytes of K only: a
//     NaN there is no other head's.
//   a_j = log2(e) s_j + log2 vscale(j), p_j = 2^(a_j - m + 5) for a reference m that moves only where an
//     a_j passes it by more than 3: p stays below 2^8, e4m3 ends at 448.  (Moving costs some 800
//     cycles: with room for 4, 3, 2 and 1 the first case below took 112, 114, 117 and 120 us.)
//   O^T (128 columns x 96) += V^T . P^T, V^T read MN-major from the same layout, P as three e4m3
//     planes: p (rounded to f16) = h + 2^-5 l + 2^-10 l', 11 bits down to 2^-13 of the largest
//     weight times scale, below that multiples of 2^-24 of it.  A position loses half of one at
//     most, n of them n 2^-25 of what the largest has: 2^-8, bf16's half step, at 131,072, and 2^-5 at
//     1,048,576, where weights that small are all that there is.
// Eight MMAs a tile, 64 (32 for a pair) and 96 columns wide: about 400 cycles of the tensor pipe for 32 KB, which take
// 1,420 from memory.
//
// Warps: two groups of four take a TMEM lane a thread (a position: its scales, its weights of 16
// rows), one issues the MMAs, one copies tiles (TMA, a box a page, five stages), two fetch scales.
// The last three go from piece to piece without the others, so that a piece's first tiles are there
// when its queries are; scores of the next tile are formed while this one's weights are.  Every wait
// is bounded.  The scale warps also look over the new tokens' values, which some rows see and some do
// not: NaN among them give way, and the rows that see them are marked behind the piece.
//
// Measured, us in a graph: 64 requests of 2,048 to 65,536 positions, 4 new tokens, 16/2 heads of 128
// (544 MB): 116, the narrow kernel 187; 64 of 8,192, 4 tokens, 16/2 heads of 64: 72 and 84 (134 MB, read
// twice: two units a pair).  A tile
// takes 1,500 to 1,700 cycles: the softmax warps are busy 1,100 of them (the vote on the reference
// 120, the fence before the MMAs 160, two waits 300).  Copies by 16-byte cp.async kept seven warps busy
// and the first case at 176; scales loaded by the softmax warps held each tile for a trip to memory
// (2,700 cycles); four groups, even and odd tiles apart, had 96 registers a thread and took 133 where
// two took 127; one warp group with 32 rows a thread 279.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <mutex>

#include "../../include/paged_mla.h"
#include "mla_api_internal.h"
#include "mla_gqa_block_decode.cuh"
#include "ptx.cuh"

namespace {

using namespace pmla;

constexpr float kTop = 5.f;            // log2 of a weight at the reference
constexpr float kRoom = 3.f;           // how far a score may pass it
constexpr float kNone = -3.402823466e38f;      // the reference of a row that has seen no position: the lowest finite one
constexpr int kSoftmaxWarps = 8, kMmaWarp = kSoftmaxWarps, kLoadWarp = kMmaWarp + 1, kScaleWarps = 2;

// D columns, KV heads a unit.
template <int D_, int HP_>
struct WideShape {
  static constexpr int D = D_, HP = HP_;
  static_assert(D * HP == 128, "a tile's rows are 128 bytes");
  static constexpr int kWarps = kLoadWarp + 1 + kScaleWarps, kThreads = 32 * kWarps;
  static constexpr int kRows = 32, kHeads = kRows / HP;    // rows of a unit, of a head
  static constexpr int kTile = 128;
  static constexpr int kHalf = kTile * 128, kStageBytes = 2 * kHalf;       // K, then V
  static constexpr int kStages = 5;
  static constexpr int kQOff = kStages * kStageBytes, kQBytes = 2 * kRows * 128;
  static constexpr int kPOff = kQOff + kQBytes, kPGroup = 16 * kTile, kPBytes = 3 * kRows * kTile;
  // a join's weights, over q and P and what they lack: copies of the next piece go on meanwhile
  static constexpr int kMaxCtas = kMaxSms, kJoinBytes = 2 * kMaxCtas * kRows * 4;
  static constexpr int kScaleOff = kQOff + (kJoinBytes > kQBytes + 2 * kPBytes ? kJoinBytes : kQBytes + 2 * kPBytes),
                       kStageScales = 2 * HP * kTile;   // floats: K's, V's
  static constexpr int kMisc = kScaleOff + kStages * kStageScales * 4;
  // NaN among new tokens' values, by piece: the scale warps are at most kStages tiles ahead of the
  // weights, each of another piece, and what a piece has is read while its weights' last product is awaited
  static constexpr int kMarks = kMisc + 2048, kMarkPieces = 8;
  static_assert(kMarkPieces >= kStages + 2, "");
  static constexpr int kSmem = kMarks + kMarkPieces * sizeof(NanMarks);
  static_assert(kMisc % 16 == 0 && kQOff % 1024 == 0 && kPOff % 1024 == 0 && kScaleOff % 16 == 0, "");
  static_assert(kSmem + 1024 <= 227 * 1024, "shared memory");
  static constexpr int kJoinWarps = kMmaWarp + 1, kJoinThreads = 32 * kJoinWarps;
  __device__ static __forceinline__ void join_sync() { asm volatile("bar.sync 3, %0;" ::"n"(kJoinThreads) : "memory"); }
  static constexpr int kSlotFloats = kRows * (D + 2);
  static constexpr bool kTwo = kRows * D > 4 * kJoinThreads;
  static constexpr int kAhead = 8;
  static constexpr int kUnitCost = 350000 / kStageBytes, kLeastCost = 55000 / kStageBytes + 1;
  static constexpr int kLeastPiece = 55000 / kStageBytes + 1;
  // tensor memory: two tiles' scores, the output
  static constexpr int kScores = 2 * kRows, kOut = 2 * kScores, kTmemCols = 256;
  static_assert(kOut + 3 * kRows <= kTmemCols, "tensor memory");
};

struct WideMisc {                              // m, sc, l and part are read 16 bytes at a time
  uint64_t full[5], scales[5], empty[5], s_full[2], p_full[2], pv[2], drain;
  alignas(16) float m[32], sc[32], l[32];      // of the rows
  alignas(16) float part[32][4];               // of the four warps of a group
  int64_t out[32];                             // where a row's output goes, -1: nowhere
  uint32_t tmem;
  int abort_flag;
  uint32_t pieces;                             // of the softmax warps, the one at hand the last
};
static_assert(sizeof(WideMisc) <= 2048 && offsetof(WideMisc, m) % 16 == 0 && offsetof(WideMisc, sc) % 16 == 0 &&
                  offsetof(WideMisc, l) % 16 == 0 && offsetof(WideMisc, part) % 16 == 0 && offsetof(WideMisc, out) % 8 == 0,
              "");

// Barriers: of the scale warps, of a group of 128 threads.
__device__ __forceinline__ void bar_scales() { asm volatile("bar.sync 4, %0;" ::"n"(32 * kScaleWarps) : "memory"); }
__device__ __forceinline__ void bar_group(int g) { asm volatile("bar.sync %0, 128;" ::"r"(1 + g) : "memory"); }
__device__ __forceinline__ bool any_group(int g, bool x) {
  uint32_t r;
  asm volatile("{\n.reg .pred p, q;\nsetp.ne.u32 p, %2, 0;\nbar.red.or.pred q, %1, 128, p;\nselp.u32 %0, 1, 0, q;\n}"
               : "=r"(r)
               : "r"(1 + g), "r"(static_cast<uint32_t>(x))
               : "memory");
  return r != 0;
}
// 16 values over the warp's lanes, halving the values at each step: lane's result is value
// row16(lane)'s.
template <bool kMax>
__device__ __forceinline__ float over_lanes(float* v, int lane) {
#pragma unroll
  for (int n = 8, d = 16; n; n >>= 1, d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int k = 0; k < n; ++k) {
      const float got = __shfl_xor_sync(0xffffffffu, up ? v[k] : v[k + n], d), keep = up ? v[k + n] : v[k];
      v[k] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 1);
  return kMax ? fmaxf(v[0], got) : v[0] + got;
}
__device__ __forceinline__ int row16(int lane) { return lane >> 1; }

// What two f16 values lack as e4m3 codes, times 32.
__device__ __forceinline__ uint32_t rest_f16x2(uint32_t x, uint32_t codes) {
  return f16x2_mul(f16x2_sub(x, e4m3x2_to_f16x2(codes)), 0x50005000u);
}

__device__ __forceinline__ void tma_4d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// After tmem_wait_ld: code that reads these registers stays behind the wait.
template <int N>
__device__ __forceinline__ void landed(float (&v)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) asm volatile("" : "+f"(v[k]));
}

// Byte offset of 16-byte chunk c of row r: rows of 128 bytes, eight of them a swizzle atom.
__device__ __forceinline__ uint32_t atom_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// q's rows: a head's high planes, then its low ones; sc: each row's factor from a product of
// high to a score in units of log2.  By the softmax warps, four rows each.
template <class S>
__device__ __forceinline__ void stage_queries(const BlockDecodeParams& p, const Piece& u, uint8_t* s_q, float* s_sc,
                                              int warp, int lane) {
  constexpr int kLanes = S::D / 4;          // four columns each
  constexpr int kMine = S::kRows / kSoftmaxWarps;
  uint2 w[kMine];
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int ur = warp + kSoftmaxWarps * k, hp = ur / S::kHeads, hk = u.hk0 + hp, h = ur % S::kHeads;
    // a lane's place in the 128 columns: those of the row's head
    const int col = lane - hp * kLanes;
    w[k] = make_uint2(0, 0);
    if (h < u.nh && hk < p.Hk && col >= 0 && col < kLanes) {
      const int r = u.h0 + h, of = r / p.G;              // the row's token
      const uint16_t* row = p.q + (u.tok0 + of) * p.q_tok + (static_cast<int64_t>(hk) * p.G + r - of * p.G) * p.q_head;
      w[k] = __ldg(reinterpret_cast<const uint2*>(row) + col);
    }
  }
#pragma unroll
  for (int k = 0; k < kMine; ++k) {
    const int ur = warp + kSoftmaxWarps * k;
    const float x[4] = {__uint_as_float(w[k].x << 16), __uint_as_float(w[k].x & 0xFFFF0000u),
                        __uint_as_float(w[k].y << 16), __uint_as_float(w[k].y & 0xFFFF0000u)};
    float mx = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
    mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
    int e = 261 - static_cast<int>(__float_as_uint(mx) >> 23);     // 2^(7 - exponent), biased
    e = e > 253 ? 253 : (e < 7 ? 7 : e);
    // (an infinite q: all of its row NaN)
    const float up = mx < INFINITY ? __uint_as_float(static_cast<uint32_t>(e) << 23) : NAN;
    uint32_t high = 0, low = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float a = x[2 * i] * up, b = x[2 * i + 1] * up;
      const uint32_t c = f32x2_to_e4m3x2(b, a), f = e4m3x2_to_f16x2(c);
      const float2 back = __half22float2(*reinterpret_cast<const __half2*>(&f));
      high |= c << (16 * i);
      low |= static_cast<uint32_t>(f32x2_to_e4m3x2((b - back.y) * 32.f, (a - back.x) * 32.f)) << (16 * i);
    }
    const int at = ur / S::kHeads * S::kHeads + ur;      // behind the planes of the heads before
    *reinterpret_cast<uint32_t*>(s_q + atom_at(at, lane >> 2) + 4 * (lane & 3)) = high;
    *reinterpret_cast<uint32_t*>(s_q + atom_at(at + S::kHeads, lane >> 2) + 4 * (lane & 3)) = low;
    if (lane == 0) s_sc[ur] = p.sm_scale * kLog2e * __uint_as_float(static_cast<uint32_t>(254 - e) << 23);
  }
}

// A tile's values, by the scale warps.  What lies behind the list may be NaN: zeros instead.  So may
// new tokens' values, in rows that not all query rows see, from `from` to `end`: marked.
template <class S>
__device__ __forceinline__ void clean_values(uint8_t* v, float* scales, NanMarks* marks, int tile0, int from, int end, int thread) {
  constexpr int kTile = S::kTile, kStep = 32 * kScaleWarps;
#pragma unroll 1
  for (int row = thread; row < kTile; row += kStep) {
    if (row >= end) {
#pragma unroll
      for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(v + row * 128 + 16 * c) = make_uint4(0, 0, 0, 0);
    } else if (row >= from) {
      for (int h = 0; h < S::HP; ++h) marks->look(scales + h * kTile + row, tile0 + row, h);
    }
  }
#pragma unroll 1
  for (int e = 8 * (from > 0 ? from : 0) + thread; e < 8 * (end < kTile ? end : kTile); e += kStep)     // (16-byte chunks)
    marks->look(reinterpret_cast<uint4*>(v + atom_at(e >> 3, e & 7)), tile0 + (e >> 3), 16 * (e & 7));
}

template <class S>
__device__ __noinline__ void clean_values_call(uint8_t* v, float* scales, NanMarks* marks, int tile0, int from, int end, int thread) {
  clean_values<S>(v, scales, marks, tile0, from, end, thread);
}

// NaN in the rows of a piece that see one among the new tokens' values: a thread a column, in rows'
// outputs; and a thread a row, in their lse (or in a part's sums).  The head's rows start at r0.
template <class S>
__device__ __noinline__ void mark_rows(const NanMarks& marks, const int64_t* out, void* o, bool bf16, int r0, int G, int least,
                                       int thread, float* sums, int64_t lse0, int Hq) {
  const int column = thread & 127;
  for (int row = thread >> 7; row < S::kRows && thread < 256; row += 2) {
    const int hp = row / S::kHeads;
    if (out[row] < 0 || (S::HP > 1 && column / S::D != hp) || !marks.reach(column, hp, least + (r0 + row % S::kHeads) / G)) continue;
    if (bf16) static_cast<__nv_bfloat16*>(o)[out[row] + column % S::D] = __float2bfloat16_rn(NAN);
    else static_cast<float*>(o)[out[row] + column % S::D] = NAN;
  }
  if (thread < S::kRows && out[thread] >= 0 && sums) {
    const int hp = thread / S::kHeads, r = r0 + thread % S::kHeads, of = r / G;
    if (marks.scale[hp] < least + of)
      sums[lse0 < 0 ? thread : lse0 + static_cast<int64_t>(of) * Hq + hp * G + r - of * G] = NAN;
  }
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, 1) gqa_block_wide_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, const BlockDecodeParams p) {
  constexpr int D = S::D, HP = S::HP, kRows = S::kRows, kHeads = S::kHeads, kTile = S::kTile, kStages = S::kStages;
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ SpanShared<S::kWarps> sh;
  WideMisc* misc = reinterpret_cast<WideMisc*>(smem + S::kMisc);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sbase = smem_u32(smem);
  if ((sbase & 1023u) != 0) {                // the swizzled layouts need it
    if (tid == 0) atomicOr(p.err, kErrMisaligned);
    return;
  }
  Span span;
  if (!find_span<S>(p, &sh, &span)) return;
  auto bar = [&](const uint64_t* b) { return smem_u32(b); };
  volatile int* abort_flag = &misc->abort_flag;
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(bar(misc->full + i), 1);
      mbar_init(bar(misc->scales + i), 32 * kScaleWarps);
      mbar_init(bar(misc->empty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(misc->s_full + i), 1);
      mbar_init(bar(misc->p_full + i), kSoftmaxWarps);
      mbar_init(bar(misc->pv + i), 1);
    }
    mbar_init(bar(&misc->drain), 1);
    *abort_flag = 0;
    misc->pieces = ~0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(smem_u32(&misc->tmem), S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc->tmem;

  uint32_t done = 0;                         // the CTA's tiles before this piece
  NanMarks* const all_marks = reinterpret_cast<NanMarks*>(smem + S::kMarks);
  bool ok = true;                            // MMA and copying warps: no wait has given up
  uint32_t issued = 0;                       // tiles that the copying warp has asked for, pieces of the scale warps
  auto wait = [&](const uint64_t* b, uint32_t parity) {
    if (ok) ok = warp_bcast(mbar_wait(bar(b), parity, abort_flag, p.err));
    return ok;
  };
  // Copying warps go through the pieces by themselves, up to five tiles ahead of the others.
  for (int64_t x = span.begin; x < span.end;) {
    Piece u;
    if (!next_piece<S>(p, span, &x, &u)) continue;
    const int n = u.t1 - u.t0;
    const int len = u.r.len;
    if (warp == kLoadWarp) {
      // ---- copies: a box of the tile's rows in one page a lane.  Pages that are not there lie
      // outside the tensor: zeros.
      const int log2_rows = p.pages.log2_page < 7 ? p.pages.log2_page : 7;      // of a box
      const int ps_mask = (1 << p.pages.log2_page) - 1;
      const int first = lane << log2_rows;               // the lane's box's first row
      const int x0 = D == 128 ? 0 : 64 * u.hk0, y0 = D == 128 ? u.hk0 : 0;
      auto page_of = [&](int i) -> int {
        const int j = (u.t0 + i) * kTile + first;
        return i < n && first < kTile && j < len ? __ldg(p.pages.indices + u.idx0 + (j >> p.pages.log2_page)) : -1;
      };
      int page = page_of(0), next = page_of(1);
#pragma unroll 2
      for (int i = 0; i < n; ++i) {
        const uint32_t it = done + i, stage = it % kStages, use = it / kStages;
        if (use > 0 && !wait(misc->empty + stage, (use - 1) & 1)) break;
        const uint32_t dst = sbase + stage * S::kStageBytes + first * 128;
        if (lane == 0) mbar_arrive_expect_tx(bar(misc->full + stage), S::kStageBytes);
        __syncwarp();
        if (first < kTile) {
          const int z = ((u.t0 + i) * kTile + first) & ps_mask;
          const int at = page >= 0 && page < p.n_pages ? page : static_cast<int>(p.n_pages);
          tma_4d(dst, &tm_k, x0, y0, z, at, bar(misc->full + stage));
          tma_4d(dst + S::kHalf, &tm_v, x0, y0, z, at, bar(misc->full + stage));
        }
        issued = it + 1;
        page = next;
        next = page_of(i + 2);
      }
      done += n;
      continue;
    }
    if (warp > kLoadWarp) {
      // ---- scales: two positions a lane, the loads of four tiles in flight
      NanMarks* const marks = all_marks + issued++ % S::kMarkPieces;
      const int least = len - u.r.tokens + 1;            // positions that every row sees
      marks->clear(tid - 32 * (kLoadWarp + 1), 32 * kScaleWarps);
      __syncwarp();
      bar_scales();
      constexpr int kMine = 4 / kScaleWarps, kBatch = 4;
      const int row0 = 32 * (warp - kLoadWarp - 1) + lane;
      const int ps_mask = (1 << p.pages.log2_page) - 1;
      auto page_of = [&](int i, int k) -> int {
        const int j = (u.t0 + i) * kTile + row0 + 32 * kScaleWarps * k;
        return i < n && j < len ? __ldg(p.pages.indices + u.idx0 + (j >> p.pages.log2_page)) : -1;
      };
      int page[kBatch][kMine];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int k = 0; k < kMine; ++k) page[b][k] = page_of(b, k);
#pragma unroll 1
      for (int i0 = 0; i0 < n; i0 += kBatch) {
        float sc[kBatch][kMine][2 * HP];
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
          for (int k = 0; k < kMine; ++k) {
            const int j = (u.t0 + i0 + b) * kTile + row0 + 32 * kScaleWarps * k;
            const bool there = page[b][k] >= 0 && page[b][k] < p.n_pages;
            if (!there && i0 + b < n && j < len) atomicOr(p.err, kErrBadRowId);        // reads as zeros
            const int64_t at = page[b][k] * p.sc_page + ((j & ps_mask) >> p.log2_block) * p.sc_block + u.hk0 * p.sc_head;
#pragma unroll
            for (int h = 0; h < HP; ++h) {
              const bool mine = there && u.hk0 + h < p.Hk;
              sc[b][k][h] = mine ? __ldg(p.ks + at + h * p.sc_head) : 0.f;
              sc[b][k][HP + h] = mine ? __ldg(p.vs + at + h * p.sc_head) : 0.f;
            }
            page[b][k] = page_of(i0 + kBatch + b, k);
          }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          const int i = i0 + b;
          if (i >= n) break;
          const uint32_t it = done + i, stage = it % kStages, use = it / kStages;
          if (use > 0) mbar_wait(bar(misc->empty + stage), (use - 1) & 1, abort_flag, p.err);
          float* const s_scale = reinterpret_cast<float*>(smem + S::kScaleOff) + stage * S::kStageScales;
#pragma unroll
          for (int k = 0; k < kMine; ++k)
#pragma unroll
            for (int h = 0; h < 2 * HP; ++h) s_scale[h * kTile + row0 + 32 * kScaleWarps * k] = sc[b][k][h];
          // Weights, which come after the scales, keep the product waiting.
          if (const int tile0 = (u.t0 + i) * kTile; tile0 + kTile > least) {
            mbar_wait(bar(misc->full + stage), (it / kStages) & 1, abort_flag, p.err);
            // (As a call where units have one head, in place where they have two: 115 and 71 us for four
            // tokens of eight heads, 128 and 64 wide; a call for both 115 and 76, in place 118 and 71.)
            uint8_t* const v = smem + stage * S::kStageBytes + S::kHalf;
            float* const v_scale = s_scale + HP * kTile;
            if constexpr (HP == 1) clean_values_call<S>(v, v_scale, marks, tile0, least - tile0, len - tile0, row0);
            else clean_values<S>(v, v_scale, marks, tile0, least - tile0, len - tile0, row0);
            fence_proxy_async_smem();
          }
          mbar_arrive(bar(misc->scales + stage));
        }
      }
      done += n;
      continue;
    }
    if (warp < kSoftmaxWarps) stage_queries<S>(p, u, smem + S::kQOff, misc->sc, warp, lane);
    if (tid < kRows) misc->m[tid] = kNone;
    fence_proxy_async_smem();
    S::join_sync();
    if (warp == kMmaWarp) {
      // ---- the MMAs: the whole warp runs the loop, an elected lane issues
      constexpr uint32_t idesc_qk = idesc_f8(128, 2 * kHeads, false, false);
      constexpr uint32_t idesc_pv = idesc_f8(128, 3 * kRows, true, true);
      const uint64_t k0 = smem_desc(sbase, 16, 1024, kSw128);
      const uint64_t v0 = smem_desc(sbase + S::kHalf, S::kHalf, 1024, kSw128);
      const uint64_t q0 = smem_desc(sbase + S::kQOff, 16, 1024, kSw128);
      // P: eight positions a core matrix of 128 bytes (16 columns each), those 128 bytes apart,
      // groups of 16 columns kPGroup apart
      const uint64_t p0 = smem_desc(sbase + S::kPOff, 128, S::kPGroup, kSwNone);
      auto weigh = [&](int i) {                // O += V^T . P^T of tile i
        const uint32_t it = done + i, stage = it % kStages;
        if (!wait(misc->p_full + (it & 1), (it >> 1) & 1)) return;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kTile / 32; ++kk)
          mma_f8_warp(tmem + S::kOut, desc_at(v0, stage * S::kStageBytes + kk * 32 * 128),
                      desc_at(p0, (it & 1) * S::kPBytes + kk * 4 * 128), idesc_pv, i == 0 && kk == 0 ? 0u : 1u);
        mma_commit_warp(bar(misc->empty + stage));
        mma_commit_warp(bar(misc->pv + (it & 1)));
      };
      for (int i = 0; i < n; ++i) {
        const uint32_t it = done + i, stage = it % kStages;
        if (!wait(misc->full + stage, (it / kStages) & 1)) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          const int hp = kk / (D / 32);
          mma_f8_warp(tmem + (it & 1) * S::kScores + hp * 2 * kHeads, desc_at(k0, stage * S::kStageBytes + 32 * kk),
                      desc_at(q0, hp * 2 * kHeads * 128 + 32 * kk), idesc_qk, kk % (D / 32) > 0 ? 1u : 0u);
        }
        mma_commit_warp(bar(misc->s_full + (it & 1)));
        if (i > 0) weigh(i - 1);
      }
      if (ok) weigh(n - 1);
      __syncwarp();
    } else {
      // ---- weights: a thread a position and 16 rows, of one head
      const int grp = warp >> 2, c0 = 16 * grp, hp = c0 / kHeads;
      const uint32_t tl = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
      const uint32_t s_at = tl + hp * kHeads + c0;       // the scores of its rows' high planes
      const int prow = 32 * (warp & 3) + lane;
      const int least = len - u.r.tokens + 1;            // positions that the first token sees
      const float* const s_scale = reinterpret_cast<const float*>(smem + S::kScaleOff) + hp * kTile + prow;
      uint8_t* const p_at = smem + S::kPOff + (prow >> 3) * 128 + (prow & 7) * 16;
      float* const s_m = misc->m + c0;
      float* const s_l = misc->l + c0;
      float l[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) l[k] = 0.f;
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const uint32_t it = done + i, stage = it % kStages;
        mbar_wait(bar(misc->scales + stage), (it / kStages) & 1, abort_flag, p.err);
        const float ks = s_scale[stage * S::kStageScales], vs = s_scale[stage * S::kStageScales + HP * kTile];
        const float least_vs = vs < kLeastScale ? kLeastScale : vs;
        const float lv = lg2_approx(least_vs), rv = rcp_approx(least_vs);
        const int j = (u.t0 + i) * kTile + prow;
        mbar_wait(bar(misc->s_full + (it & 1)), (it >> 1) & 1, abort_flag, p.err);
        tc_fence_after();
        float a[16], lo[16];
        tmem_ld16(s_at + (it & 1) * S::kScores, a);
        tmem_ld16(s_at + (it & 1) * S::kScores + kHeads, lo);
        tmem_wait_ld();
        landed(a);
        landed(lo);
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 sc = *reinterpret_cast<const float4*>(misc->sc + c0 + k);
          const float f[4] = {sc.x, sc.y, sc.z, sc.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) a[k + e] = fmaf(fmaf(lo[k + e], 0.03125f, a[k + e]), f[e] * ks, lv);
        }
        if ((u.t0 + i + 1) * kTile > least) {  // causal among the new tokens, and the list's end
#pragma unroll 1
          for (int t = j < least ? 0 : (j - least + 1) * p.G - u.h0 - c0 % kHeads, k = 0; k < t && k < 16; ++k) {
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (e == k) a[e] = -INFINITY;      // rows of tokens before the position's
          }
        }
        float most = -INFINITY;
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 m = *reinterpret_cast<const float4*>(s_m + k);
          most = fmaxf(most, fmaxf(fmaxf(a[k] - m.x, a[k + 1] - m.y), fmaxf(a[k + 2] - m.z, a[k + 3] - m.w)));
        }
        if (any_group(grp, most > kRoom)) {
          // ---- the references move up to the tile's maxima, sums and output with them
          float v[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) v[k] = a[k];
          const float t = over_lanes<true>(v, lane);
          if ((lane & 1) == 0) misc->part[c0 + row16(lane)][warp & 3] = t;
          bar_group(grp);
          if (prow < 16) {
            const float4 x4 = *reinterpret_cast<const float4*>(misc->part[c0 + prow]);
            const float to = fmaxf(s_m[prow], fmaxf(fmaxf(x4.x, x4.y), fmaxf(x4.z, x4.w)));
            s_l[prow] = ex2_approx(s_m[prow] - to);
            s_m[prow] = to;
          }
          bar_group(grp);
          if (i > 0) {                         // the output of the tiles before
            mbar_wait(bar(misc->pv + ((it - 1) & 1)), ((it - 1) >> 1) & 1, abort_flag, p.err);
            tc_fence_after();
          }
#pragma unroll
          for (int k = 0; k < 16; ++k) l[k] *= s_l[k];
          if (i > 0) {
#pragma unroll 1
            for (int c = c0; c < 3 * kRows; c += kRows) {
              float o[16];
              tmem_ld16(tl + S::kOut + c, o);
              tmem_wait_ld();
              landed(o);
#pragma unroll
              for (int k = 0; k < 16; ++k) o[k] *= s_l[k];
              tmem_st16(tl + S::kOut + c, o);
            }
            tmem_wait_st();
          }
        }
        // ---- weights in three planes, this position's 16 bytes of each
        uint32_t h[4], lo1[4], lo2[4];
#pragma unroll
        for (int k = 0; k < 16; k += 4) {
          const float4 m4 = *reinterpret_cast<const float4*>(s_m + k);
          const float m[4] = {m4.x, m4.y, m4.z, m4.w};
          uint32_t c[2][3];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float w0 = ex2_approx(a[k + 2 * e] + (kTop - m[2 * e])),
                        w1 = ex2_approx(a[k + 2 * e + 1] + (kTop - m[2 * e + 1]));
            l[k + 2 * e] = fmaf(w0, rv, l[k + 2 * e]);
            l[k + 2 * e + 1] = fmaf(w1, rv, l[k + 2 * e + 1]);
            const uint32_t y = f32x2_to_f16x2(w1, w0);
            c[e][0] = f16x2_to_e4m3x2(y);
            const uint32_t y1 = rest_f16x2(y, c[e][0]);
            c[e][1] = f16x2_to_e4m3x2(y1);
            c[e][2] = f16x2_to_e4m3x2(rest_f16x2(y1, c[e][1]));
          }
          h[k / 4] = c[0][0] | c[1][0] << 16;
          lo1[k / 4] = c[0][1] | c[1][1] << 16;
          lo2[k / 4] = c[0][2] | c[1][2] << 16;
        }
        uint8_t* at = p_at + (it & 1) * S::kPBytes + grp * S::kPGroup;
        *reinterpret_cast<uint4*>(at) = make_uint4(h[0], h[1], h[2], h[3]);
        *reinterpret_cast<uint4*>(at + kRows / 16 * S::kPGroup) = make_uint4(lo1[0], lo1[1], lo1[2], lo1[3]);
        *reinterpret_cast<uint4*>(at + 2 * kRows / 16 * S::kPGroup) = make_uint4(lo2[0], lo2[1], lo2[2], lo2[3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(misc->p_full + (it & 1)));
      }
      // ---- the rows' sums over the positions; where their outputs go
      const float sum = over_lanes<false>(l, lane);
      if ((lane & 1) == 0) misc->part[c0 + row16(lane)][warp & 3] = sum;
      bar_group(grp);
      if (tid == 0) ++misc->pieces;            // (read between this piece's last barrier and the next one's first)
      const bool whole = u.t0 == 0 && u.t1 == u.n_tiles;
      float* slot = part_slot<S>(p, u);
      if (prow < 16) {
        const int row = c0 + prow;
        const float4 x4 = *reinterpret_cast<const float4*>(misc->part[row]);
        const float ll = (x4.x + x4.y) + (x4.z + x4.w), mm = s_m[prow] - kTop;
        int64_t to = -1;
        if (row_there<S>(u, row)) {
          const int hr = u.h0 + row % kHeads, of = hr / p.G, hq = (u.hk0 + hp) * p.G + hr - of * p.G;
          to = (u.tok0 + of) * p.o_tok + hq * p.o_head;
          if (whole && p.lse) p.lse[(u.tok0 + of) * p.Hq + hq] = ll == 0.f ? -INFINITY : mm * kLn2 + logf(ll);
          if (!whole) {
            to = 2 * kRows + row * D;
            slot[row] = mm;
            slot[kRows + row] = ll;
          }
        }
        misc->out[row] = to;
        s_l[prow] = whole ? (ll == 0.f ? 0.f : 1.f / ll) : 1.f;
      }
      bar_group(grp);
      // ---- the output: a thread a column
      const uint32_t it = done + n - 1;
      mbar_wait(bar(misc->pv + (it & 1)), (it >> 1) & 1, abort_flag, p.err);
      tc_fence_after();
      const int d = prow % D;
      float o[16], o1[16], o2[16];
      tmem_ld16(tl + S::kOut + c0, o);
      tmem_ld16(tl + S::kOut + kRows + c0, o1);
      tmem_ld16(tl + S::kOut + 2 * kRows + c0, o2);
      tmem_wait_ld();
      landed(o);
      landed(o1);
      landed(o2);
      if (HP == 1 || hp == prow / D) {         // (a pair's other columns are the other head's)
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int64_t to = misc->out[c0 + k];
          const float f = s_l[k], y = f == 0.f ? 0.f : fmaf(fmaf(o2[k], 0.03125f, o1[k]), 0.03125f, o[k]) * f;
          if (to < 0) continue;
          if (!whole) slot[to + d] = y;
          else if (p.o_f32) static_cast<float*>(p.o)[to + d] = y;
          else static_cast<__nv_bfloat16*>(p.o)[to + d] = __float2bfloat16_rn(y);
        }
      }
      tc_fence_before();
    }
    done += n;
    S::join_sync();                          // the piece's MMAs are done, its rows written
    tc_fence_after();
    if (const NanMarks* marks = all_marks + misc->pieces % S::kMarkPieces; marks->any) {
      const bool whole = u.t0 == 0 && u.t1 == u.n_tiles;
      mark_rows<S>(*marks, misc->out, whole ? p.o : part_slot<S>(p, u), whole && !p.o_f32, u.h0, p.G, len - u.r.tokens + 1, tid,
                   whole ? p.lse : part_slot<S>(p, u) + kRows, whole ? u.tok0 * p.Hq + u.hk0 * p.G : -1, p.Hq);
    }
    if (!(u.t0 == 0 && u.t1 == u.n_tiles)) {
      join_parts<S>(p, span, u, &sh, misc->m, misc->l, reinterpret_cast<float*>(smem + S::kQOff));
      S::join_sync();
    }
  }
  __syncthreads();
  // After a wait that gave up, copies and MMAs may still be in flight.
  if (*abort_flag && warp == kLoadWarp)
    for (uint32_t it = issued > kStages ? issued - kStages : 0; it < issued; ++it)
      mbar_wait_drain(bar(misc->full + it % kStages), (it / kStages) & 1);
  if (*abort_flag && warp == kMmaWarp) {
    mma_commit_warp(bar(&misc->drain));
    mbar_wait_drain(bar(&misc->drain), 0);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// A cache as (bytes of a row, KV heads, slots, pages); pairs of 64-wide heads lie side by side in
// a slot's row, whose bytes are the first dimension then.  A box: 128 bytes of a page's slots.
bool encode(EncodeTiledFn enc, CUtensorMap* m, const BlockDecodeParams& p, const uint8_t* base, int64_t D) {
  const cuuint64_t ps = cuuint64_t{1} << p.pages.log2_page, heads = D == 128 ? p.Hk : 1;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D == 128 ? 128 : D * p.Hk), heads, ps,
                              static_cast<cuuint64_t>(p.n_pages)};
  auto stride = [](cuuint64_t n, int64_t pitch) { return static_cast<cuuint64_t>(n > 1 ? pitch : 128); };
  const cuuint64_t strides[3] = {stride(heads, p.head_pitch), stride(ps, p.slot_pitch), stride(dims[3], p.page_pitch)};
  const cuuint32_t box[4] = {128, 1, static_cast<cuuint32_t>(ps < 128 ? ps : 128), 1}, step[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, box, step,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class S>
cudaError_t launch(const BlockDecodeParams& p, int sms, cudaStream_t stream) {
  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!attr_set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(gqa_block_wide_kernel<S>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) return e;
      attr_set[dev] = true;
    }
  }
  EncodeTiledFn enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  CUtensorMap tm_k, tm_v;
  if (!enc || !encode(enc, &tm_k, p, p.k, S::D) || !encode(enc, &tm_v, p, p.v, S::D)) return cudaErrorInvalidValue;
  gqa_block_wide_kernel<S><<<sms, S::kThreads, S::kSmem, stream>>>(tm_k, tm_v, p);
  return cudaGetLastError();
}

}  // namespace

// More than 16 query rows a KV head, the narrow kernel's unit: up to there a unit of it reads a cache
// once as well, and is faster or equal (us here and there: 32/2 heads of 128, 64 requests of 8,192:
// 65 and 63; 16/2 heads, 16,384: 105 and 92).  Above, the narrow one reads it once for every 16
// rows, and this one once for every 32 of a 128-wide head (32 rows: 116 and 187); of 64-wide heads it
// reads it once for every 16, too, and is faster all the same (32 rows: 72 and 84).  Boxes want pages of at
// least a swizzle atom's eight slots, strides that a tensor map can hold, and pairs of 64-wide heads
// side by side.
bool pmla::block_wide_takes(const BlockDecodeParams& p, int64_t D) {
  const auto fits = [](int64_t n, int64_t pitch) { return n <= 1 || (pitch > 0 && pitch % 16 == 0 && pitch < int64_t{1} << 40); };
  const int64_t ps = int64_t{1} << p.pages.log2_page;
  if (static_cast<int64_t>(p.G) * p.max_q <= 16 || ps < 8 || p.n_pages < 1 || p.n_pages > 0x7FFFFFFF) return false;
  if (!fits(ps, p.slot_pitch) || !fits(p.n_pages, p.page_pitch)) return false;
  return D == 128 ? fits(p.Hk, p.head_pitch) : p.Hk > 1 && p.head_pitch == 64;
}

cudaError_t pmla::launch_block_wide(const BlockDecodeParams& p, int64_t D, int sms, cudaStream_t stream) {
  return D == 128 ? launch<WideShape<128, 1>>(p, sms, stream) : launch<WideShape<64, 2>>(p, sms, stream);
}
