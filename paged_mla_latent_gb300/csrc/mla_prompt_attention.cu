// mla_prompt_attention: causal attention of whole prompts, packed one after another, with
// grouped heads.
//
//   request b: T query tokens, L key positions (L > T: a prefix that was cached before); query
//   t sees j <= L - T + t:  s_j = sm_scale q . k_j,  lse = ln sum e^{s_j},
//   o = sum e^{s_j - lse} v_j.  A query that sees nothing gives o = 0, lse = -inf.
//
// 2 (D + Dv) operations a visible (query, key) pair and head on the tensor cores, one
// exponential each: bound by the MMAs (M = N = 128, K = 16 at 8192 operations a cycle and SM)
// while the exponentials of one tile hide under the MMAs of another.
//
// Work.  A unit is 256 query rows of one KV head, two tiles of 128.  A row is one (token,
// query head) pair: a tile holds 128 / G tokens with all G heads of the group, so short
// prompts fill the MMA's M, a K/V tile is read once for the whole group, and the causal edge
// wastes G times fewer columns than a tile of one head's tokens.  All units form one line,
// each as long as the positions it reads plus a fixed cost, and each of one CTA a SM takes an
// equal span of it.  A long unit is cut where a span ends: the parts leave (m, l, O) in fp32
// in the workspace and a second kernel joins them (12 heads of 4,089 queries behind 63,911
// positions are 192 units for 152 SMs: whole units would leave a third of the SMs idle).
// Spans are worked off from their ends: neighbouring spans of one head, whose units are
// equally long, then read the same K/V tiles at the same time, from L2.
//
//   warps 0-3, 4-7 : softmax of tile 0 / 1, a thread a row: S from tensor memory, maximum,
//                    exponentials, P as bf16 back over S's columns.
//   warp 8         : walks the span, queues its pieces for the others and loads them by TMA: K
//                    and V tiles of 128 positions in 16 KB chunks of 64 columns (128-byte
//                    swizzle) through one ring.
//   warp 9         : tcgen05.mma issuer.  S = Q K^T from shared memory; O += P V with P (the A
//                    operand) in tensor memory.  Order: PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1),
//                    so that one tile's MMAs run while the other's softmax does.  (An issuer
//                    for each tile: their MMAs interleave, both tiles' results come later,
//                    16,384 tokens 1856 us instead of 1568.)
//   warps 10-11    : for the tiles on the causal edge and at a request's end, zeroes the V rows
//                    past the request (another request's, or stale memory) and takes
//                    non-finite values out of V (0 * inf would reach rows that do not see
//                    them); rows that do see one get it back at the end, times its weight.
// Tensor memory: S_0 S_1 O_0 O_1, 128 columns each (all 512; 64-wide values leave half of an O's
// unused); P_s lies over S_s, rounded to V's bf16 (by 2^-8 of a weight at most).
//
// The running maximum is only raised when it would grow by more than 8 (in log2): then the
// thread rescales its row of O itself (the MMA that wrote S(j) was issued after PV(j-1), so
// O is idle).  Weights stay below 2^8, sums in fp32.  P is rounded to bf16 (2^-8 of each
// weight at most); l is summed from the unrounded weights.
//
// Measured (GB300, one call after another, inputs in turn): 16,384 tokens, 32/8 heads of 128:
// 1.40 to 1.42 ms, 1555 to 1575 TFLOP/s (0.82 of cuBLAS's burst bf16 rate, 0.91 of its sustained
// one), of which 1.28 ms in the kernel alone, the tensor pipe 75 % busy; 4,089 queries behind
// 63,911 positions, 12 heads of 192/128: 1.30 to 1.31 ms, 1575 to 1590 TFLOP/s; 24 packed prompts
// of 17 to 4,089: 277 us, 1030 TFLOP/s.  64-wide heads (in a graph): 16,384 tokens 1.20 ms, 915
// TFLOP/s; the packed prompts 245 us.  What bounds it: a tile's loop is its softmax (about 1500
// cycles) and then its PV and QK (1024; 512 with 64-wide heads), of which two tiles' overlap; in
// short units the ends (Q behind the last S, the last PV, the result: 7400 cycles).
//
// Every wait is bounded (2 s): one that runs out sets the error word and ends the CTA.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/paged_mla.h"
#include "mla_api_internal.h"
#include "mla_gqa_check.h"
#include "ptx.cuh"

namespace pmla {
namespace {

constexpr int kRows = 128;                 // query rows of a tile (the MMA's M)
constexpr int kKeys = 128;                 // positions of a K/V tile
constexpr int kChunk = 128 * 128;          // 128 rows of 64 bf16 columns
constexpr int kThreads = 384;
constexpr int kEdges = 8;                  // barriers of edge tiles; the ring holds at most 6 V tiles
constexpr int kLoads = 16;                 // barriers of K and V tiles; the ring holds at most 12
constexpr int kQueue = 4;                  // pieces queued
constexpr int kConsumers = 11;             // warps that read a queued piece
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.f;              // log2 growth of the maximum that forces a rescale

// Fixed cost of a unit on the line (its Q, the first tile's way, its result: 7,400 cycles against
// 2,700 a tile, fitted over the CTAs of packed prompts of 128-wide heads, and taken for the other
// widths without a fit of their own) in positions; with 512 those prompts take 278 us instead of
// 266.  The fewest K/V tiles a part of a cut unit may have: writing and
// joining a part moves 266 KB, about four tiles' time of an SM.
constexpr int kUnitCost = 352;
constexpr int kMinCut = 8;                 // a power of two
constexpr int kMaxParts = 512;             // parts of one unit: at most one a span

template <int D_, int DV_>
struct PromptShape {
  static constexpr int D = D_, DV = DV_;
  static constexpr int KC = D / 64, VC = DV / 64;          // chunks of a K / V tile
  static constexpr int kQBytes = 2 * KC * kChunk;
  static constexpr int NC = 14 - 2 * KC;                   // ring chunks: 224 KB with Q
  static constexpr int kBarOff = kQBytes + NC * kChunk;
  static constexpr int kSmem = kBarOff + 1024 + 1024;      // barriers and queue, alignment
  static constexpr int kPartFloats = 2 * kRows * (DV + 2); // a cut part: m, l, O
  static_assert(kSmem <= 232448, "shared memory");
};

struct Cut;

struct PromptParams {
  const int32_t *qo_indptr, *kv_indptr;
  int B, Hq, Hk, G;
  int tok_tile;                            // tokens of a 128-row tile: 128 / G
  int64_t n_tok, n_keys;
  float scale_log2;                        // sm_scale log2(e)
  uint16_t* o;
  int64_t o_tok, o_head;
  float* lse;
  const uint16_t *q, *k, *v;               // for the rows that see a non-finite value
  int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;
  float* parts;                            // two a CTA; null: units are not cut
  Cut* cuts;                               // one a CTA
  int* err;
};

// Part of a unit: K/V tiles [j0, j1).
struct Piece {
  int row0;         // first query token's row of q and o
  int toks;         // query tokens from there to the request's end
  int pos0;         // position of the first of them among the keys (negative: sees nothing)
  int kv0;          // the request's first key row
  int hk;
  int j0, j1;
  int part;         // where a cut piece leaves its result; -1: the unit is whole
};

// What the join needs of the unit whose first part a CTA leaves (tiles = 0: none), and whether
// a wait of the CTA ran out, so that parts of its may be missing (written as it ends).
struct Cut {
  Piece unit;
  int tiles;
  int gave_up;
  int64_t u0, weight, span;                // on the line
};

// K/V tiles that tile s of a unit needs (its last token's).
__device__ __forceinline__ int tiles_of(const Piece& w, int s, int tok_tile) {
  const int a = s * tok_tile;
  if (a >= w.toks) return 0;
  const int seen = w.pos0 + (a + tok_tile < w.toks ? a + tok_tile : w.toks);
  return seen > 0 ? (seen + kKeys - 1) / kKeys : 0;
}
// The first K/V tile of a piece that holds positions some row of the unit does not see.
__device__ __forceinline__ int first_edge(const Piece& w) {
  const int clear = w.pos0 + 1 > 0 ? (w.pos0 + 1) / kKeys : 0;
  return clear > w.j0 ? clear : w.j0;
}

// ---- the line of work
struct Request {
  int q0, T, kv0, L;
  int units;                               // units of one KV head
  // line length of the first i units of a head
  __device__ int64_t cum(int i, int cta_tok) const {
    if (units == 0) return 0;
    const int64_t fixed = kUnitCost + (L > T ? L - T : 0);
    const int64_t full = i < units ? i : units - 1;
    int64_t x = full * fixed + cta_tok * (full * (full + 1) / 2);
    if (i >= units) x += fixed + T;
    return x;
  }
};
__device__ __forceinline__ Request load_request(const PromptParams& p, int b, int cta_tok, bool flag) {
  Request r = {0, 0, 0, 0, 0};
  const int64_t s = __ldg(p.qo_indptr + b), e = __ldg(p.qo_indptr + b + 1);
  const int64_t ks = __ldg(p.kv_indptr + b), ke = __ldg(p.kv_indptr + b + 1);
  if (s < 0 || e < s || e > p.n_tok) {     // the request is left out
    if (flag) atomicOr(p.err, kErrBadIndptr);
    return r;
  }
  r.q0 = static_cast<int>(s);
  r.T = static_cast<int>(e - s);
  r.units = (r.T + cta_tok - 1) / cta_tok;
  if (ks < 0 || ke < ks || ke > p.n_keys) {   // no keys
    if (flag) atomicOr(p.err, kErrBadIndptr);
    return r;
  }
  r.kv0 = static_cast<int>(ks);
  r.L = static_cast<int>(ke - ks);
  return r;
}
__device__ __forceinline__ int64_t warp_scan(int64_t x, int lane) {
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int64_t o = __shfl_up_sync(0xffffffffu, x, i);
    if (lane >= i) x += o;
  }
  return x;
}
// A unit and where it starts on the line.
struct Unit {
  Request r;
  int b, hk, i;
  int64_t u0;
};
// A CTA's span [x0, x1) of the line and the unit that holds x1 - 1 (a warp together).  The
// first 32 requests stay in the lanes' registers, so that a batch of as many pays one round
// trip to memory.
struct Span {
  int64_t x0, x1, length;
  Unit last;
};
__device__ __forceinline__ Span find_span(const PromptParams& p, int cta_tok, int lane) {
  Span sp;
  Request mine = {0, 0, 0, 0, 0};
  int64_t total = 0;
#pragma unroll 4
  for (int b = lane; b < p.B; b += 32) {
    const Request r = load_request(p, b, cta_tok, blockIdx.x == 0);
    if (b < 32) mine = r;
    total += r.cum(r.units, cta_tok);
  }
#pragma unroll
  for (int i = 16; i; i >>= 1) total += __shfl_xor_sync(0xffffffffu, total, i);
  total *= p.Hk;
  sp.length = (total + gridDim.x - 1) / gridDim.x;
  sp.x0 = blockIdx.x * sp.length;
  sp.x1 = sp.x0 + sp.length < total ? sp.x0 + sp.length : total;
  Unit& u = sp.last;
  u = {};
  if (sp.x0 >= sp.x1) return sp;
  const int64_t x = sp.x1 - 1;
  int64_t done = 0;
  for (int b0 = 0; b0 < p.B; b0 += 32) {
    Request r = mine;
    if (b0 > 0) {
      r = {0, 0, 0, 0, 0};
      if (b0 + lane < p.B) r = load_request(p, b0 + lane, cta_tok, false);
    }
    const int64_t n = r.cum(r.units, cta_tok) * p.Hk;
    const int64_t end = done + warp_scan(n, lane);
    const uint32_t who = __ballot_sync(0xffffffffu, x < end && x >= end - n);
    if (who) {
      const int src = __ffs(who) - 1;
      u.b = b0 + src;
      done = __shfl_sync(0xffffffffu, end - n, src);
      u.r.q0 = __shfl_sync(0xffffffffu, r.q0, src);
      u.r.T = __shfl_sync(0xffffffffu, r.T, src);
      u.r.kv0 = __shfl_sync(0xffffffffu, r.kv0, src);
      u.r.L = __shfl_sync(0xffffffffu, r.L, src);
      u.r.units = __shfl_sync(0xffffffffu, r.units, src);
      break;
    }
    done = __shfl_sync(0xffffffffu, end, 31);
  }
  const int64_t head = u.r.cum(u.r.units, cta_tok);
  while (x - done >= head) {               // (at most Hk times)
    done += head;
    ++u.hk;
  }
  int lo = 0, hi = u.r.units - 1;
  while (lo < hi) {                        // the last unit that starts at or before x
    const int mid = (lo + hi + 1) >> 1;
    if (u.r.cum(mid, cta_tok) <= x - done) lo = mid;
    else hi = mid - 1;
  }
  u.i = lo;
  u.u0 = done + u.r.cum(lo, cta_tok);
  return sp;
}
__device__ __forceinline__ Piece unit_piece(const Unit& u, int cta_tok, int tok_tile) {
  Piece w;
  const int tok0 = u.i * cta_tok;
  w.row0 = u.r.q0 + tok0;
  w.toks = u.r.T - tok0;
  w.pos0 = u.r.L - u.r.T + tok0;
  w.kv0 = u.r.kv0;
  w.hk = u.hk;
  const int n0 = tiles_of(w, 0, tok_tile), n1 = tiles_of(w, 1, tok_tile);
  w.j0 = 0;
  w.j1 = n0 > n1 ? n0 : n1;
  w.part = -1;
  return w;
}
// The K/V tile at which a border at point x of the line cuts a unit of n tiles that starts at
// u0 and is `weight` long.  Short units stay whole, with the span that holds their middle;
// long ones are cut at multiples of kMinCut tiles.
__host__ __device__ __forceinline__ int cut_at(int64_t u0, int64_t weight, int n, int64_t x, bool cuts) {
  if (x <= u0) return 0;
  if (x >= u0 + weight) return n;
  if (!cuts || n < 2 * kMinCut) return x > u0 + weight / 2 ? n : 0;
  const int64_t t = (x - u0 - kUnitCost) >> 7;
  if (t >= n) return n;
  if (t < kMinCut) return 0;
  return n - t < kMinCut ? n : static_cast<int>(t) & ~(kMinCut - 1);
}

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z,
                                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// Runs of MMAs by a converged warp, one elected lane issuing: bf16 operands, fp32 accumulator.
// One election and one set of descriptors a run; a branch or an election between the MMAs
// costs more than the MMA takes (issued one by one with a branch each, 16,384 tokens took 2280
// us instead of 1770).
//
// D[tmem] (+)= A[smem] . B[smem] over 64 columns of K (four MMAs, 32 bytes apart in both).
__device__ __forceinline__ void mma_ss4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b64 a, b;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 a, %1, 2;\n\tadd.s64 b, %2, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 4;\n\tadd.s64 b, %2, 4;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "add.s64 a, %1, 6;\n\tadd.s64 b, %2, 6;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, t;\n\t"
      "}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// The same with A in tensor memory (lane = row, each 32-bit column two bf16 of consecutive k)
// over 64 of K: four MMAs, 8 columns of A and 16 rows (2048 bytes) of B apart.
__device__ __forceinline__ void mma_ts4(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, t, e;\n\t.reg .b64 b;\n\t.reg .b32 a;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.eq.b32 t, 0, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t"
      "add.s32 a, %1, 8;\n\tadd.s64 b, %2, 128;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 16;\n\tadd.s64 b, %2, 256;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "add.s32 a, %1, 24;\n\tadd.s64 b, %2, 384;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a], b, %3, t;\n\t"
      "}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// Two fp32 values in one 64-bit register pair, and the packed operations on them.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float* lo, float* hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(x));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// kind::f16, D f32, A and B bf16 (fields as in the other kernels); B MN-major or K-major.
__host__ __device__ constexpr uint32_t idesc_bf16(int N, bool b_mn_major) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) |
         ((static_cast<uint32_t>(N) >> 3) << 17) | ((128u >> 4) << 24);
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
// Four lanes hold four 16-byte words each, v[4 w + k].  Afterwards v[4 i + k] is word lane & 3
// of lane ^ i.  A thread has a row of O: stored as it lies, an instruction would write 16 bytes
// into each of 32 rows; so it writes 64 bytes into each of eight.
__device__ __forceinline__ void transpose4(uint32_t* v, int lane) {
  const bool b = lane & 1, c = lane & 2;
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = v[8 * k + i], y = v[8 * k + 4 + i];
      v[8 * k + i] = b ? y : x;
      v[8 * k + 4 + i] = __shfl_xor_sync(0xffffffffu, b ? x : y, 1);
    }
#pragma unroll
  for (int r = 0; r < 2; ++r)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = v[4 * r + i], y = v[8 + 4 * r + i];
      v[4 * r + i] = c ? y : x;
      v[8 + 4 * r + i] = __shfl_xor_sync(0xffffffffu, c ? x : y, 2);
    }
}
__device__ __forceinline__ bool half_nonfinite(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }
// The word with zeros in place of its non-finite halves.
__device__ __noinline__ uint32_t finite_halves(uint32_t w) {
  return (half_nonfinite(w) ? 0u : w & 0xFFFFu) | (half_nonfinite(w >> 16) ? 0u : w & 0xFFFF0000u);
}

// The weight 2^(scale2 q . k + off) of one key in a row of n columns.
__device__ __forceinline__ float key_weight(const uint16_t* q, const uint16_t* k, int n, float scale2, float off) {
  float dot = 0.f;
#pragma unroll 1
  for (int i = 0; i < n; i += 2) {
    const uint32_t a = *reinterpret_cast<const uint32_t*>(q + i), b = *reinterpret_cast<const uint32_t*>(k + i);
    dot = fmaf(__uint_as_float(a << 16), __uint_as_float(b << 16), dot);
    dot = fmaf(__uint_as_float(a & 0xFFFF0000u), __uint_as_float(b & 0xFFFF0000u), dot);
  }
  return ex2_approx(fmaf(dot, scale2, off));
}

template <class S>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const PromptParams p) {
  constexpr int KC = S::KC, VC = S::VC, NC = S::NC, DV = S::DV;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const uint32_t ring = sbase + S::kQBytes;
  // barriers: full[kLoads] and empty[kLoads] (K and V tiles in turn), q_full, q_empty, s_full[2],
  // p_full[2][2] (the halves of a tile), o_full[2], clean[kEdges], edge[kEdges] (a V tile on the edge lands there, so that
  // the warps that clean it need not follow the ring), item_full[kQueue], item_empty[kQueue],
  // drain
  const uint32_t bars = sbase + S::kBarOff;
  const uint32_t full0 = bars, empty0 = full0 + 8 * kLoads, q_full = empty0 + 8 * kLoads;
  const uint32_t q_empty = q_full + 8;
  const uint32_t s_full = q_empty + 8, p_full = s_full + 16, o_full = p_full + 32;
  const uint32_t clean0 = o_full + 16, edge0 = clean0 + 8 * kEdges;
  const uint32_t item_full = edge0 + 8 * kEdges, item_empty = item_full + 8 * kQueue;
  const uint32_t drain = item_empty + 8 * kQueue;
  uint8_t* words = smem + S::kBarOff + 16 * kLoads + 16 + 64 + 16 * kEdges + 16 * kQueue + 16;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(words);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(words + 4);
  volatile int* bad_v = reinterpret_cast<volatile int*>(words + 8);           // [kQueue]
  volatile uint32_t* landing = reinterpret_cast<volatile uint32_t*>(words + 8 + 4 * kQueue);  // [kLoads]
  Piece* queue = reinterpret_cast<Piece*>(words + 8 + 4 * kQueue + 4 * kLoads);   // [kQueue]

  // (the broadcasts make the compiler's analysis see what is uniform in a warp: an MMA whose
  // descriptors it keeps in uniform registers issues in its own time, otherwise in about 80
  // cycles)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int cta_tok = 2 * p.tok_tile;

  if (warp == 8 && lane == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    for (int i = 0; i < kLoads; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full + 8 * s, 1);
      mbar_init(p_full + 16 * s, 4);
      mbar_init(p_full + 16 * s + 8, 4);
      mbar_init(o_full + 8 * s, 1);
    }
    for (int i = 0; i < kEdges; ++i) mbar_init(clean0 + 8 * i, 64);
    for (int i = 0; i < kEdges; ++i) mbar_init(edge0 + 8 * i, 1);
    for (int i = 0; i < kQueue; ++i) {
      mbar_init(item_full + 8 * i, 1);
      mbar_init(item_empty + 8 * i, kConsumers);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
  asm volatile("griddepcontrol.launch_dependents;");     // the join may be launched

  // The it-th piece for a consumer warp: false at the span's end (or on abort).
  auto next_piece = [&](int it, Piece* w) -> bool {
    if (!warp_bcast(mbar_wait(item_full + 8 * (it % kQueue), (it / kQueue) & 1, abort_flag, p.err))) return false;
    *w = queue[it % kQueue];
    return w->j0 >= 0;
  };
  auto piece_read = [&](int it) {
    __syncwarp();
    if (lane == 0) mbar_arrive(item_empty + 8 * (it % kQueue));
  };

  if (warp >= 8) {
    if (warp == 8) {
      // ---------------------------------------------------------- the span's pieces, TMA
      const Span sp = find_span(p, cta_tok, lane);
      const int64_t x0 = sp.x0, x1 = sp.x1;
      Unit u = sp.last;
      const bool cuts = p.parts != nullptr;
      if (cuts && lane == 0) p.cuts[blockIdx.x].tiles = 0;
      if (lane == 0) {
        const uint32_t box = static_cast<uint32_t>(p.tok_tile) * p.G * 128;
        int i = 0, n = 0, edges = 0, nq = 0;   // chunks, loads, edge tiles, Qs so far
        int it = 0;
        bool ok = true;
        auto push = [&](const Piece& w) {
          const int q = it % kQueue;
          if (it >= kQueue && !mbar_wait(item_empty + 8 * q, ((it / kQueue) - 1) & 1, abort_flag, p.err)) {
            ok = false;
            return;
          }
          queue[q] = w;
          bad_v[q] = 0;
          mbar_arrive(item_full + 8 * q);
          ++it;
        };
        auto load = [&](const Piece& w) {
          const int e0 = first_edge(w);
          for (int j = w.j0; j < w.j1; ++j) {
            for (int v = 0; v < 2; ++v) {
              const int chunks = v ? VC : KC;
              if (j == w.j0 && v) {            // Q behind the first K tile
                if (nq > 0 && !mbar_wait(q_empty, (nq - 1) & 1, abort_flag, p.err)) {
                  ok = false;
                  return;
                }
                const int tiles = w.toks > p.tok_tile ? 2 : 1;
                mbar_arrive_expect_tx(q_full, tiles * KC * box);
                for (int s = 0; s < tiles; ++s)
                  for (int k = 0; k < KC; ++k)
                    tma_3d(sbase + (s * KC + k) * kChunk, &tm_q, 64 * k, w.hk * p.G,
                           w.row0 + s * p.tok_tile, q_full);
                ++nq;
              }
              const int reused = i + chunks - 1 - NC;   // the last chunk this load overwrites
              if (reused >= 0) {
                const int l = 2 * (reused / (KC + VC)) + (reused % (KC + VC) >= KC ? 1 : 0);
                if (!mbar_wait(empty0 + 8 * (l % kLoads), (l / kLoads) & 1, abort_flag, p.err)) {
                  ok = false;
                  return;
                }
              }
              uint32_t bar = full0 + 8 * (n % kLoads), parity = (n / kLoads) & 1;
              if (v && j >= e0) {
                mbar_arrive(bar);              // keeps its phases in step
                bar = edge0 + 8 * (edges % kEdges);
                parity = (edges / kEdges) & 1;
                ++edges;
              }
              landing[n % kLoads] = bar | (parity << 31);
              mbar_arrive_expect_tx(bar, chunks * kChunk);
              for (int c = 0; c < chunks; ++c, ++i)
                tma_3d(ring + (i % NC) * kChunk, v ? &tm_v : &tm_k, 64 * c, w.hk, w.kv0 + j * kKeys, bar);
              ++n;
            }
          }
        };
        while (ok && x0 < x1) {
          const int64_t weight = u.r.cum(u.i + 1, cta_tok) - u.r.cum(u.i, cta_tok);
          Piece w = unit_piece(u, cta_tok, p.tok_tile);
          const int tiles = w.j1;
          bool mine = x0 <= u.u0 && u.u0 < x1;   // rows that see nothing: the span of their start
          if (tiles > 0) {
            w.j0 = cut_at(u.u0, weight, tiles, x0, cuts);
            w.j1 = cut_at(u.u0, weight, tiles, x1, cuts);
            mine = w.j0 < w.j1;
            if (mine && (w.j0 > 0 || w.j1 < tiles)) {
              w.part = 2 * blockIdx.x + (w.j0 == 0 ? 1 : 0);
              if (w.j0 == 0) p.cuts[blockIdx.x] = {w, tiles, 0, u.u0, weight, sp.length};
            }
          }
          if (mine) {
            push(w);
            if (ok) load(w);
          }
          if (u.u0 <= x0) break;
          if (--u.i < 0) {                     // the unit before
            if (--u.hk < 0) {
              do u.r = load_request(p, --u.b, cta_tok, false);
              while (u.r.units == 0);
              u.hk = p.Hk - 1;
            }
            u.i = u.r.units - 1;
          }
          u.u0 -= u.r.cum(u.i + 1, cta_tok) - u.r.cum(u.i, cta_tok);
        }
        if (ok) {
          Piece end = {};
          end.j0 = -1;
          push(end);
        }
        // no copy may be in flight when the CTA ends
        if (nq > 0) mbar_wait_drain(q_full, (nq - 1) & 1);
        for (int l = 0; l < (n < kLoads ? n : kLoads); ++l)
          mbar_wait_drain(landing[l] & 0x7FFFFFFFu, landing[l] >> 31);
      }
      __syncwarp();
    } else if (warp == 9) {
      // ---------------------------------------------------------- MMA issuer
      constexpr uint32_t id_qk = idesc_bf16(kKeys, false);
      constexpr uint32_t id_pv = idesc_bf16(DV, true), id_pv64 = idesc_bf16(64, true);
      bool ok = true;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        ok = ok && warp_bcast(mbar_wait(bar, parity, abort_flag, p.err));
        tc_fence_after();
      };
      // the barriers of tile t's K (v = 0) and V (v = 1), t counted over the whole span
      auto wait_tile = [&](int t, int v) {
        const int l = 2 * t + v;
        wait(full0 + 8 * (l % kLoads), (l / kLoads) & 1);
      };
      auto free_tile = [&](int t, int v) { mma_commit_warp(empty0 + 8 * ((2 * t + v) % kLoads)); };
      // S_s = Q_s K(t)^T
      auto qk = [&](int s, int t) {
        const int i = t * (KC + VC);
#pragma unroll
        for (int c = 0; c < KC; ++c)
          mma_ss4(tmem + 128 * s, smem_desc(sbase + (s * KC + c) * kChunk, 16, 1024, kSw128),
                  smem_desc(ring + ((i + c) % NC) * kChunk, 16, 1024, kSw128), id_qk, c > 0 ? 1u : 0u);
        mma_commit_warp(s_full + 8 * s);
      };
      // O_s += P_s V(t) over half of the tile's positions
      auto pv = [&](int s, int t, int half, bool first) {
        const int slot = (t * (KC + VC) + KC) % NC;
        const uint64_t v0 = desc_at(smem_desc(ring + slot * kChunk, kChunk, 1024, kSw128), 8192 * half);
        const uint32_t o = tmem + 256 + 128 * s, pt = tmem + 128 * s + 32 * half;
        const uint32_t acc = first ? 0u : 1u;
        // V's two chunks lie at the ring's two ends (with an even KC a V tile starts in an even
        // slot of the even ring: never)
        if (VC == 2 && KC % 2 == 1 && slot == NC - 1) {
          mma_ts4(o, pt, v0, id_pv64, acc);
          mma_ts4(o + 64, pt, desc_at(smem_desc(ring, kChunk, 1024, kSw128), 8192 * half), id_pv64, acc);
        } else {
          mma_ts4(o, pt, v0, id_pv, acc);
        }
      };
      int base = 0, edges = 0, nq = 0;         // K/V tiles, edge tiles, Qs so far
      uint32_t done = 0;                       // parities of either row tile's tiles so far
      Piece w;
      for (int it = 0; ok && next_piece(it, &w); ++it) {
        piece_read(it);
        const int n = __shfl_sync(0xffffffffu, w.j1 - w.j0, 0);
        if (n <= 0) continue;
        int c0 = tiles_of(w, 0, p.tok_tile), c1 = tiles_of(w, 1, p.tok_tile);
        // K/V tiles of either row tile (may be negative), the first one on the edge
        c0 = __shfl_sync(0xffffffffu, (c0 < w.j1 ? c0 : w.j1) - w.j0, 0);
        c1 = __shfl_sync(0xffffffffu, (c1 < w.j1 ? c1 : w.j1) - w.j0, 0);
        const int e0 = __shfl_sync(0xffffffffu, first_edge(w) - w.j0, 0);
        wait(q_full, nq & 1);
        ++nq;
        wait_tile(base, 0);
        if (!ok) break;
        if (c0 > 0) qk(0, base);
        if (c1 > 0) qk(1, base);
        free_tile(base, 0);
        if (n == 1) mma_commit_warp(q_empty);
        for (int t = 0; t < n; ++t) {
          if (t >= e0) {
            wait(clean0 + 8 * (edges % kEdges), (edges / kEdges) & 1);
            ++edges;
          } else {
            wait_tile(base + t, 1);
          }
          bool k_here = false;
#pragma unroll
          for (int s = 0; s < 2; ++s) {
            const int c = s ? c1 : c0;
            if (t < c) {
              wait(p_full + 16 * s, (done >> s) & 1);
              if (!ok) break;
              pv(s, base + t, 0, t == 0);
              wait(p_full + 16 * s + 8, (done >> s) & 1);
              done ^= 1u << s;
              if (!ok) break;
              pv(s, base + t, 1, false);
              if (t + 1 == c) mma_commit_warp(o_full + 8 * s);
            }
            if (s) free_tile(base + t, 1);
            if (t + 1 < c) {
              if (!k_here) wait_tile(base + t + 1, 0);   // behind PV, which hides the wait
              k_here = true;
              if (!ok) break;
              qk(s, base + t + 1);
            }
          }
          if (!ok) break;
          if (t + 1 < n) {
            free_tile(base + t + 1, 0);
            if (t + 2 == n) mma_commit_warp(q_empty);
          }
        }
        base += n;
      }
      mma_commit_warp(drain);
      __syncwarp();
    } else {
      // ---------------------------------------------------------- V on the edge
      int base = 0, edges = 0;                 // tiles, edge tiles so far
      bool ok = true;
      Piece w;
      for (int it = 0; ok && next_piece(it, &w); ++it) {
        const int len = w.pos0 + w.toks;       // the request's keys
        for (int j = first_edge(w); j < w.j1 && ok; ++j, ++edges) {
          const int iv = (base + j - w.j0) * (KC + VC) + KC;
          const bool tail = (j + 1) * kKeys > len;
          bool bad = false;
          ok = mbar_wait(edge0 + 8 * (edges % kEdges), (edges / kEdges) & 1, abort_flag, p.err);
          for (int c = 0; c < VC && ok; ++c) {
            uint4* chunk = reinterpret_cast<uint4*>(smem + S::kQBytes + ((iv + c) % NC) * kChunk);
            // (the swizzle moves 16-byte words inside a 128-byte row only)
#pragma unroll 4
            for (int e = threadIdx.x - 320; e < 128 * 8; e += 64) {
              if (tail && j * kKeys + (e >> 3) >= len) {
                chunk[e] = make_uint4(0, 0, 0, 0);
                continue;
              }
              uint4 x = chunk[e];
              // a half whose exponent is all ones carries into its top bit
              const uint32_t m = 0x7F807F80u, one = 0x00800080u;
              const uint32_t top = ((x.x & m) + one) | ((x.y & m) + one) | ((x.z & m) + one) | ((x.w & m) + one);
              if (__builtin_expect(top & 0x80008000u, 0)) {
                x.x = finite_halves(x.x);
                x.y = finite_halves(x.y);
                x.z = finite_halves(x.z);
                x.w = finite_halves(x.w);
                chunk[e] = x;
                bad = true;
              }
            }
          }
          if (bad) bad_v[it % kQueue] = 1;
          fence_proxy_async_smem();
          if (ok) mbar_arrive(clean0 + 8 * (edges % kEdges));
        }
        base += w.j1 - w.j0;
        piece_read(it);
      }
    }
  } else {
    // ------------------------------------------------------------ softmax, one row a thread
    const int s = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + 128 * s + lane_base, t_o = tmem + 256 + 128 * s + lane_base;
    const int tt = r / p.G, hg = r - tt * p.G;
    const int tok = s * p.tok_tile + tt;       // in the unit
    int done = 0, outs = 0, edges = 0;
    bool ok = true;
    Piece w;
    for (int it = 0; ok && next_piece(it, &w); ++it) {
      const bool live = tt < p.tok_tile && tok < w.toks;
      // the last position the row sees
      const int lim = w.pos0 + tok;
      const int nt = tiles_of(w, s, p.tok_tile);
      const int j1 = nt < w.j1 ? nt : w.j1;
      const int e0 = first_edge(w);
      float m = -INFINITY, l = 0.f;
      for (int j = w.j0; j < j1; ++j, ++done) {
        ok = warp_bcast(mbar_wait(s_full + 8 * s, done & 1, abort_flag, p.err));
        if (!ok) break;
        tc_fence_after();
        // two passes over S, 64 columns at a time, in loops: the roles share the SM's instruction
        // caches, which a row of 128 registers and its unrolled code overran
        float mt = -INFINITY;
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          float x[64];
          tmem_ld32(t_s + 64 * half, x);
          tmem_ld32(t_s + 64 * half + 32, x + 32);
          tmem_wait_ld_regs(x, x + 16);
          tmem_wait_ld_regs(x + 32, x + 48);
          const int last = lim - j * kKeys - 64 * half;
          if (j >= e0 && !__all_sync(0xffffffffu, last >= 63)) {
#pragma unroll
            for (int c = 0; c < 64; c += 32) {
              const int n = last - c + 1;          // columns of this group that the row sees
              const uint32_t seen = n >= 32 ? 0xFFFFFFFFu : (n <= 0 ? 0u : (1u << n) - 1u);
#pragma unroll
              for (int i = 0; i < 32; ++i) x[c + i] = seen & (1u << i) ? x[c + i] : -INFINITY;
            }
            tmem_st32(t_s + 64 * half, x);
            tmem_st32(t_s + 64 * half + 32, x + 32);
          }
          float mx[2] = {x[0], x[1]};
#pragma unroll
          for (int i = 2; i < 62; i += 4) {
            mx[0] = max3(mx[0], x[i], x[i + 2]);
            mx[1] = max3(mx[1], x[i + 1], x[i + 3]);
          }
          mt = fmaxf(mt, max3(fmaxf(mx[0], mx[1]), x[62], x[63]));
        }
        if (j >= e0) tmem_wait_st();
        // raise the maximum where it grew by more than kRaise (always from -inf); each row by
        // itself, so that no row's result depends on its neighbours (or on idle rows)
        const bool raise = live && mt > m && !((mt - m) * p.scale_log2 <= kRaise);
        if (__any_sync(0xffffffffu, raise)) {
          const float mn = raise ? mt : m;
          const float f = m == mn ? 1.f : ex2_approx((m - mn) * p.scale_log2);   // 0 from -inf
          m = mn;
          l *= f;
          if (j > w.j0) {
#pragma unroll 1
            for (int c = 0; c < DV; c += 16) {
              float o[16];
              tmem_ld16(t_o + c, o);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] *= f;
              tmem_st16(t_o + c, o);
            }
          }
        }
        const float off = m == -INFINITY ? 0.f : -m * p.scale_log2;
        const uint64_t scale2 = pair(p.scale_log2, p.scale_log2), off2 = pair(off, off);
        uint64_t sum[2] = {0, 0};
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
          float x[64];
          tmem_ld32(t_s + 64 * half, x);
          tmem_ld32(t_s + 64 * half + 32, x + 32);
          tmem_wait_ld_regs(x, x + 16);
          tmem_wait_ld_regs(x + 32, x + 48);
          uint32_t pk[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const uint64_t y = fma2(pair(x[2 * i], x[2 * i + 1]), scale2, off2);
            float a, b;
            unpair(y, &a, &b);
            a = ex2_approx(a);
            b = ex2_approx(b);
            sum[i & 1] = add2(sum[i & 1], pair(a, b));
            pk[i] = pack_bf16(a, b);
          }
          tmem_st32(t_s + 32 * half, reinterpret_cast<float*>(pk));
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_full + 16 * s + 8 * half);
        }
        float s0, s1, s2, s3;
        unpair(sum[0], &s0, &s1);
        unpair(sum[1], &s2, &s3);
        l += (s0 + s1) + (s2 + s3);
      }
      // ---- the row's result
      const bool any = j1 > w.j0;
      if (any && ok) ok = warp_bcast(mbar_wait(o_full + 8 * s, outs & 1, abort_flag, p.err));
      outs += any ? 1 : 0;
      const int n_edge = w.j1 > e0 ? w.j1 - e0 : 0;
      if (n_edge > 0 && ok) {
        const int e = edges + n_edge - 1;
        ok = warp_bcast(mbar_wait(clean0 + 8 * (e % kEdges), (e / kEdges) & 1, abort_flag, p.err));
      }
      edges += n_edge;
      if (!ok) break;
      const bool fix = any && n_edge > 0 && bad_v[it % kQueue] != 0;
      piece_read(it);
      if (s * p.tok_tile >= w.toks) continue;
      tc_fence_after();
      const bool whole = w.part < 0;
      const float inv = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      const bool none = whole && l == 0.f;
      const bool any_none = __any_sync(0xffffffffu, none);
      const int h = w.hk * p.G + hg;
      const int64_t row = static_cast<int64_t>(w.row0) + tok;
      // this lane's words go to the rows of its group of four lanes
      const int64_t mine = live ? row * p.o_tok + h * p.o_head : -1;
      const int64_t dst[4] = {mine, __shfl_xor_sync(0xffffffffu, mine, 1), __shfl_xor_sync(0xffffffffu, mine, 2),
                              __shfl_xor_sync(0xffffffffu, mine, 3)};
      float* stats = whole ? nullptr : p.parts + w.part * static_cast<int64_t>(S::kPartFloats) + s * kRows + r;
      float* part = whole ? nullptr : p.parts + w.part * static_cast<int64_t>(S::kPartFloats) + 4 * kRows + (s * kRows + r) * DV;
      const float m2 = m == -INFINITY ? m : m * p.scale_log2;
#pragma unroll 1
      for (int c = 0; c < DV; c += 32) {
        float o[32];
        if (any) {
          tmem_ld32(t_o + c, o);
          tmem_wait_ld_regs(o, o + 16);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
        const uint64_t inv2 = pair(inv, inv);
#pragma unroll
        for (int i = 0; i < 16; ++i) unpair(mul2(pair(o[2 * i], o[2 * i + 1]), inv2), &o[2 * i], &o[2 * i + 1]);
        if (__builtin_expect(fix && live, 0))
          for (int j = e0 * kKeys; j <= lim && j < w.j1 * kKeys; ++j) {
            const int64_t key = static_cast<int64_t>(w.kv0) + j;
            const uint32_t* vr = reinterpret_cast<const uint32_t*>(p.v + key * p.v_tok + w.hk * p.v_head + c);
            bool bad = false;
#pragma unroll 1
            for (int i = 0; i < 16; ++i) bad |= half_nonfinite(vr[i]) || half_nonfinite(vr[i] >> 16);
            if (!bad) continue;
            // a weight of zero makes inf NaN, as where PV has the value itself
            const float weight = key_weight(p.q + row * p.q_tok + h * p.q_head, p.k + key * p.k_tok + w.hk * p.k_head,
                                            S::D, p.scale_log2, m == -INFINITY ? 0.f : -m2);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t x = vr[i];
              if (half_nonfinite(x)) o[2 * i] += weight * __uint_as_float(x << 16);
              if (half_nonfinite(x >> 16)) o[2 * i + 1] += weight * __uint_as_float(x & 0xFFFF0000u);
            }
          }
        __syncwarp();
        if (any_none) {                          // a row without any weight is zero
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = none ? 0.f : o[i];
        }
        uint32_t y[16];
        if (whole) {
#pragma unroll
          for (int i = 0; i < 16; ++i) y[i] = pack_bf16(o[2 * i], o[2 * i + 1]);
          transpose4(y, lane);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (dst[i] >= 0)
              *reinterpret_cast<uint4*>(p.o + dst[i] + c + 8 * (lane & 3)) =
                  make_uint4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]);
        } else if (live) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<float4*>(part + c + 4 * i) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
      }
      if (live && whole && p.lse)
        p.lse[row * p.Hq + h] = l == 0.f ? -INFINITY : (m == -INFINITY ? 0.f : m2) * kLn2 + logf(l);
      if (live && !whole) {
        stats[0] = m2;
        stats[2 * kRows] = l;
      }
      tc_fence_before();                       // O is read before the next piece's P arrives
    }
  }
  tc_fence_before();
  __syncthreads();
  if (p.parts && threadIdx.x == 0) p.cuts[blockIdx.x].gave_up = *abort_flag;
  if (warp == 9) {
    if (lane == 0) mbar_wait_drain(drain, 0);   // all issued MMAs complete (bounded)
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of the unit that span blockIdx.x cuts and has the first part of; blockIdx.y
// takes 32 of its 256 rows, eight threads a row.  Bytes bound: the parts, from L2.  Where a CTA
// gave up, cut units stay unwritten: a missing part's place holds whatever was there.
template <int DV>
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptParams p) {
  constexpr int kPart = 2 * kRows * (DV + 2);
  __shared__ int sh_n, sh_parts[kMaxParts];
  const int first = blockIdx.x;
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the attention's results
  const Cut& cut = p.cuts[first];
  const int tiles = cut.tiles;
  if (tiles == 0) return;
  const Piece w = cut.unit;
  if (threadIdx.x == 0) {
    int parts = 0;
    sh_parts[parts++] = 2 * first + 1;
    int t = w.j1;
    for (int i = first + 1; t < tiles; ++i) {            // spans between two cuts, some empty
      const int e = cut_at(cut.u0, cut.weight, tiles, (i + 1) * cut.span, true);
      if (e > t) sh_parts[parts++] = 2 * i;
      t = e;
    }
    sh_n = parts;
  }
  int gave_up = 0;
  for (int i = threadIdx.x; i <= gridDim.x; i += blockDim.x) gave_up |= p.cuts[i].gave_up;
  if (__syncthreads_or(gave_up)) return;
  const int n_parts = sh_n;
  const int row = 32 * blockIdx.y + (threadIdx.x >> 3), q = threadIdx.x & 7;
  const int s = row / kRows, r = row - s * kRows;
  const int tt = r / p.G, tok = s * p.tok_tile + tt;
  if (tt >= p.tok_tile || tok >= w.toks) return;
  auto part = [&](int i) { return p.parts + static_cast<int64_t>(sh_parts[i]) * kPart; };
  float mm = -INFINITY;
  for (int i = 0; i < n_parts; ++i) mm = fmaxf(mm, part(i)[row]);
  float ll = 0.f, o[DV / 8];
#pragma unroll
  for (int k = 0; k < DV / 8; ++k) o[k] = 0.f;
  for (int i = 0; i < n_parts; ++i) {
    const float m = part(i)[row], l = part(i)[2 * kRows + row];
    // a part that no key has weight in: m = -inf, l = 0 (NaN scores keep their l)
    const float f = m == -INFINITY ? 1.f : ex2_approx(m - mm);
    ll += f * l;
    const float* at = part(i) + 4 * kRows + row * DV;
#pragma unroll
    for (int k = 0; k < DV / 32; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(at + 32 * k + 4 * q);
      o[4 * k] += f * x.x;
      o[4 * k + 1] += f * x.y;
      o[4 * k + 2] += f * x.z;
      o[4 * k + 3] += f * x.w;
    }
  }
  const bool none = ll == 0.f;
  const float inv = none ? 0.f : 1.f / ll;
  const int h = w.hk * p.G + r - tt * p.G;
  const int64_t at = static_cast<int64_t>(w.row0) + tok;
#pragma unroll
  for (int k = 0; k < DV / 32; ++k) {
    uint2 y;
    y.x = pack_bf16(none ? 0.f : o[4 * k] * inv, none ? 0.f : o[4 * k + 1] * inv);
    y.y = pack_bf16(none ? 0.f : o[4 * k + 2] * inv, none ? 0.f : o[4 * k + 3] * inv);
    *reinterpret_cast<uint2*>(p.o + at * p.o_tok + h * p.o_head + 32 * k + 4 * q) = y;
  }
  if (q == 0 && p.lse)
    p.lse[at * p.Hq + h] = none ? -INFINITY : (mm == -INFINITY ? 0.f : mm) * kLn2 + logf(ll);
}

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// (tokens, heads, width) bf16 as (width, heads, tokens), box 64 columns x box_heads x box_toks.
int encode(EncodeTiledFn enc, CUtensorMap* m, const mla_tensor_t* t, int box_heads, int box_toks) {
  const int64_t n = t->shape[0], heads = t->shape[1], width = t->shape[2];
  // the stride of a size-1 dim is never stepped: any valid one will do
  const int64_t sh = heads > 1 ? t->stride[1] : width;
  const int64_t st = n > 1 ? t->stride[0] : heads * sh;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(width), static_cast<cuuint64_t>(heads),
                        static_cast<cuuint64_t>(n)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(sh * 2), static_cast<cuuint64_t>(st * 2)};
  cuuint32_t box[3] = {64, static_cast<cuuint32_t>(box_heads), static_cast<cuuint32_t>(box_toks)};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, t->ptr, dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? MLA_OK : MLA_ERR_INVALID_ARG;
}

template <int D, int DV>
cudaError_t launch(const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                   const PromptParams& p, int sms, cudaStream_t stream) {
  using S = PromptShape<D, DV>;
  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lk(mu);
    if (!attr_set[dev]) {
      const cudaError_t e = cudaFuncSetAttribute(prompt_attention_kernel<S>,
                                                 cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
      if (e != cudaSuccess) return e;
      attr_set[dev] = true;
    }
  }
  prompt_attention_kernel<S><<<sms, kThreads, S::kSmem, stream>>>(tq, tk, tv, p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !p.parts) return e;
  // launched while this one runs (its blocks wait for the grid's end): the launch is hidden
  cudaLaunchConfig_t join = {};
  join.gridDim = dim3(sms - 1, 8);
  join.blockDim = dim3(256);
  join.stream = stream;
  cudaLaunchAttribute early = {};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  join.attrs = &early;
  join.numAttrs = 1;
  return cudaLaunchKernelEx(&join, prompt_join_kernel<DV>, p);
}

int sms_of_device(int* out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(out, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  return MLA_OK;
}

// Bytes of the parts and cuts a call may leave: none where no request can be long enough to be
// cut.
size_t cuts_for(int sms) { return (static_cast<size_t>(sms) * sizeof(Cut) + 255) / 256 * 256; }
size_t parts_for(int sms, int64_t n_keys, int64_t DV) {
  if (n_keys <= (2 * kMinCut - 1) * kKeys || sms < 2 || sms > kMaxParts) return 0;
  return cuts_for(sms) + 2 * static_cast<size_t>(sms) * 2 * kRows * static_cast<size_t>(DV + 2) * 4;
}

// Strides TMA can step: positive where the dim has more than one entry.
bool steppable(const mla_tensor_t* t) {
  return (t->shape[0] <= 1 || t->stride[0] > 0) && (t->shape[1] <= 1 || t->stride[1] > 0);
}

}  // namespace
}  // namespace pmla

extern "C" int mla_get_prompt_workspace_size(int64_t n_keys, int32_t v_head_dim, int32_t num_sms,
                                             size_t* bytes_out) {
  using namespace pmla;
  if (!bytes_out || n_keys < 0 || num_sms > 65536) return MLA_ERR_INVALID_ARG;
  if (v_head_dim != 64 && v_head_dim != 128) return MLA_ERR_UNSUPPORTED;
  int sms = num_sms;
  if (num_sms <= 0) {
    const int st = sms_of_device(&sms);
    if (st != MLA_OK) return st;
  }
  *bytes_out = parts_for(sms, n_keys, v_head_dim);
  return MLA_OK;
}

extern "C" int mla_prompt_attention(const mla_tensor_t* q, const mla_tensor_t* k,
                                    const mla_tensor_t* v, const mla_tensor_t* o,
                                    const mla_tensor_t* qo_indptr, const mla_tensor_t* kv_indptr,
                                    float sm_scale, const mla_tensor_t* lse_out,
                                    int32_t* error_word, void* workspace, size_t workspace_bytes,
                                    mla_stream_t stream_) {
  using namespace pmla;
  if (!q || !k || !v || q->ndim != 3 || k->ndim != 3 || v->ndim != 3) return MLA_ERR_INVALID_ARG;
  const int64_t n_tok = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t n_keys = k->shape[0], Hk = k->shape[1], DV = v->shape[2];
  if (n_tok < 0 || n_keys < 0 || n_tok >= 0x7FFFFF00 || n_keys >= 0x7FFFFF00) return MLA_ERR_INVALID_ARG;
  if (Hq < 1 || Hk < 1 || Hq > 1024 || Hq % Hk != 0) return MLA_ERR_INVALID_ARG;
  if (!gqa_check_bf16(q, n_tok, Hq, D, 8) || !gqa_check_bf16(k, n_keys, Hk, D, 8) ||
      !gqa_check_bf16(v, n_keys, Hk, DV, 8) || !gqa_check_bf16(o, n_tok, Hq, DV, 8) ||
      !gqa_rows_apart(o))
    return MLA_ERR_INVALID_ARG;
  if (!steppable(q) || !steppable(k) || !steppable(v)) return MLA_ERR_INVALID_ARG;
  if (!qo_indptr || qo_indptr->ndim != 1 || qo_indptr->shape[0] < 1) return MLA_ERR_INVALID_ARG;
  const int64_t B = qo_indptr->shape[0] - 1;
  if (B > 0xFFFFFF || !gqa_check_i32(qo_indptr, B + 1) || !gqa_check_i32(kv_indptr, B + 1))
    return MLA_ERR_INVALID_ARG;
  if (lse_out && ((!lse_out->ptr && n_tok > 0) || lse_out->dtype != MLA_DTYPE_FP32 || lse_out->ndim != 2 ||
                  lse_out->shape[0] != n_tok || lse_out->shape[1] != Hq || (Hq > 1 && lse_out->stride[1] != 1) ||
                  (n_tok > 1 && lse_out->stride[0] != Hq) || !gqa_aligned(lse_out->ptr, 4)))
    return MLA_ERR_INVALID_ARG;
  if (!(sm_scale > 0.f) || sm_scale > 3.0e38f || !error_word) return MLA_ERR_INVALID_ARG;
  const int64_t G = Hq / Hk;
  const bool s64 = D == 64 && DV == 64, s128 = D == 128 && DV == 128, s192 = D == 192 && DV == 128;
  if (!(s64 || s128 || s192) || G > kRows) return MLA_ERR_UNSUPPORTED;
  if (workspace && !gqa_aligned(workspace, 16)) return MLA_ERR_INVALID_ARG;
  if (n_tok == 0 || B == 0) return MLA_OK;
  int sms = 0;
  const int cs = sms_of_device(&sms);
  if (cs != MLA_OK) return cs;
  const size_t need = parts_for(sms, n_keys, DV);
  if (workspace && workspace_bytes < need) return MLA_ERR_WORKSPACE_TOO_SMALL;

  PromptParams p;
  p.qo_indptr = static_cast<const int32_t*>(qo_indptr->ptr);
  p.kv_indptr = static_cast<const int32_t*>(kv_indptr->ptr);
  p.B = static_cast<int>(B);
  p.Hq = static_cast<int>(Hq);
  p.Hk = static_cast<int>(Hk);
  p.G = static_cast<int>(G);
  p.tok_tile = static_cast<int>(kRows / G);
  p.n_tok = n_tok;
  p.n_keys = n_keys;
  p.scale_log2 = sm_scale * kLog2e;
  p.o = static_cast<uint16_t*>(o->ptr);
  p.o_tok = o->stride[0];
  p.o_head = o->stride[1];
  p.lse = lse_out ? static_cast<float*>(lse_out->ptr) : nullptr;
  p.q = static_cast<const uint16_t*>(q->ptr);
  p.q_tok = q->stride[0];
  p.q_head = q->stride[1];
  p.k = static_cast<const uint16_t*>(k->ptr);
  p.k_tok = k->stride[0];
  p.k_head = k->stride[1];
  p.v = static_cast<const uint16_t*>(v->ptr);
  p.v_tok = v->stride[0];
  p.v_head = v->stride[1];
  p.err = error_word;
  p.cuts = static_cast<Cut*>(workspace);
  p.parts = workspace && need > 0 ? reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + cuts_for(sms)) : nullptr;

  EncodeTiledFn enc = reinterpret_cast<EncodeTiledFn>(tensor_map_encoder());
  if (!enc) return MLA_ERR_CUDA;
  CUtensorMap tq, tk, tv;
  int st = encode(enc, &tq, q, p.G, p.tok_tile);
  if (st != MLA_OK) return st;
  // without keys nothing is loaded: the maps then describe q
  const bool keys = n_keys > 0;
  st = encode(enc, &tk, keys ? k : q, 1, keys ? kKeys : 1);
  if (st != MLA_OK) return st;
  st = encode(enc, &tv, keys ? v : q, 1, keys ? kKeys : 1);
  if (st != MLA_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream_);
  cudaError_t e;
  if (s64) e = launch<64, 64>(tq, tk, tv, p, sms, s);
  else if (s128) e = launch<128, 128>(tq, tk, tv, p, sms, s);
  else e = launch<192, 128>(tq, tk, tv, p, sms, s);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
