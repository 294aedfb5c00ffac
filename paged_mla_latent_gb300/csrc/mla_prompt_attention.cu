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
// One CTA per (256 query rows, KV head), two tiles of 128 rows.  A row is one (token, query
// head) pair: a tile holds 128 / G tokens with all G heads of the group, so short prompts fill
// the MMA's M, a K/V tile is read once for the whole group, and the causal edge wastes G times
// fewer columns than a tile of one head's tokens.
//   warps 0-3, 4-7 : softmax of tile 0 / 1, a thread a row: S from tensor memory, maximum,
//                    exponentials, P as bf16 back over S's columns.
//   warp 8         : TMA.  K and V tiles of 128 positions come in 16 KB chunks of 64 columns
//                    (128-byte swizzle) through one ring; each has its own barriers.
//   warp 9         : tcgen05.mma issuer.  S = Q K^T from shared memory; O += P V with P (the A
//                    operand) in tensor memory.  Order: PV_0(j) QK_0(j+1) PV_1(j) QK_1(j+1),
//                    so that one tile's MMAs run while the other's softmax does.
//   warps 10-11    : for the tiles on the causal edge and at a request's end, zero the V rows
//                    past the request (another request's, or stale memory) and take non-finite
//                    values out of V (0 * inf would reach rows that do not see them); rows that
//                    do see one get it back at the end.
// Tensor memory: S_0 S_1 O_0 O_1, 128 columns each (all 512); P_s lies over S_s.
//
// The running maximum is only raised when it would grow by more than 8 (in log2): then the
// thread rescales its row of O itself (the MMA that wrote S(j) was issued after PV(j-1), so
// O is idle).  Weights stay below 2^8, sums in fp32.  P is rounded to bf16 (2^-8 of each
// weight at most); l is summed from the unrounded weights.
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
constexpr int kMaxEdge = 4;                // K/V tiles on the causal edge of a CTA (at most 3)
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRaise = 8.f;              // log2 growth of the maximum that forces a rescale

template <int D_, int DV_>
struct PromptShape {
  static constexpr int D = D_, DV = DV_;
  static constexpr int KC = D / 64, VC = DV / 64;          // chunks of a K / V tile
  static constexpr int kQBytes = 2 * KC * kChunk;
  static constexpr int NC = 14 - 2 * KC;                   // ring chunks: 224 KB with Q
  static constexpr int kBarOff = kQBytes + NC * kChunk;
  static constexpr int kSmem = kBarOff + 512 + 1024;       // barriers, alignment
  static_assert(kSmem <= 232448, "shared memory");
};

struct PromptParams {
  const int32_t *qo_indptr, *kv_indptr;
  int B, Hq, Hk, G;
  int tok_tile;                            // tokens of a 128-row tile: 128 / G
  int64_t n_tok, n_keys;
  float scale_log2;                        // sm_scale log2(e)
  uint16_t* o;
  int64_t o_tok, o_head;
  float* lse;
  const uint16_t* v;                       // for the rows that see a non-finite value
  int64_t v_tok, v_head;
  int* err;
};

__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z,
                                       uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(z), "r"(bar)
      : "memory");
}
// D[tmem] (+)= A[smem] . B[smem], bf16, fp32 accumulator; a converged warp, one lane issuing.
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.and.b32 p, %4, 0, e;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// The same with A in tensor memory: lane = row, each 32-bit column two bf16 of consecutive k.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.and.b32 p, %4, 0, e;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
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
__device__ __forceinline__ bool half_nonfinite(uint32_t h) { return (h & 0x7F80u) == 0x7F80u; }

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
  // barriers: full[NC], empty[NC], q_full, s_full[2], p_full[2], o_full[2], clean[4], drain,
  // edge[4][2] (the chunks of a V tile on the edge arrive there, each once, so that the warps
  // that clean them need not follow the ring)
  const uint32_t bars = sbase + S::kBarOff;
  const uint32_t full0 = bars, empty0 = full0 + 8 * NC, q_full = empty0 + 8 * NC;
  const uint32_t s_full = q_full + 8, p_full = s_full + 16, o_full = p_full + 16;
  const uint32_t clean0 = o_full + 16, drain = clean0 + 8 * kMaxEdge;
  const uint32_t edge0 = drain + 8;
  uint8_t* words = smem + S::kBarOff + 16 * NC + 8 + 48 + 8 * kMaxEdge + 8 + 16 * kMaxEdge;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(words);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(words + 4);
  volatile int* bad_v = reinterpret_cast<volatile int*>(words + 8);
  volatile int* work = reinterpret_cast<volatile int*>(words + 16);   // b, tile of b

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int hk = blockIdx.x % p.Hk;
  const int tile_id = blockIdx.x / p.Hk;
  const int cta_tok = 2 * p.tok_tile;

  if (warp == 8 && lane == 0) {
    prefetch_tensormap(&tm_q);
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    for (int i = 0; i < NC; ++i) {
      mbar_init(full0 + 8 * i, 1);
      mbar_init(empty0 + 8 * i, 1);
    }
    mbar_init(q_full, 1);
    for (int s = 0; s < 2; ++s) {
      mbar_init(s_full + 8 * s, 1);
      mbar_init(p_full + 8 * s, 128);
      mbar_init(o_full + 8 * s, 1);
    }
    for (int i = 0; i < kMaxEdge; ++i) mbar_init(clean0 + 8 * i, 64);
    for (int i = 0; i < 2 * kMaxEdge; ++i) mbar_init(edge0 + 8 * i, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *bad_v = 0;
    fence_mbar_init();
  }
  // ---- which request and which of its tiles: a scan over the requests' tile counts
  if (warp == 0) {
    int64_t done = 0;
    int fb = -1, ft = 0;
    for (int b0 = 0; b0 < p.B; b0 += 32) {
      const int b = b0 + lane;
      int64_t n = 0;
      if (b < p.B) {
        const int64_t s = p.qo_indptr[b], e = p.qo_indptr[b + 1];
        if (s < 0 || e < s || e > p.n_tok) {
          if (blockIdx.x == 0) atomicOr(p.err, kErrBadIndptr);    // the request is left out
        } else {
          n = (e - s + cta_tok - 1) / cta_tok;
        }
      }
      int64_t inc = n;
#pragma unroll
      for (int i = 1; i < 32; i <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, inc, i);
        if (lane >= i) inc += o;
      }
      const int64_t start = done + inc - n;
      const bool hit = tile_id >= start && tile_id < start + n;
      const uint32_t who = __ballot_sync(0xffffffffu, hit);
      if (who) {
        const int src = __ffs(who) - 1;
        fb = b0 + src;
        // the longest tiles (the last tokens) first
        ft = __shfl_sync(0xffffffffu, static_cast<int>(start + n - 1 - tile_id), src);
        break;
      }
      done += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) {
      work[0] = fb;
      work[1] = ft;
    }
  }
  __syncthreads();
  const int b = work[0];
  if (b < 0) return;                       // past the last tile
  const int tok0 = work[1] * cta_tok;      // the CTA's first token in the request
  const int64_t q0 = p.qo_indptr[b];
  const int T = static_cast<int>(p.qo_indptr[b + 1] - q0);
  int64_t kv0 = p.kv_indptr[b];
  int64_t L = p.kv_indptr[b + 1] - kv0;
  if (kv0 < 0 || L < 0 || kv0 + L > p.n_keys) {
    if (threadIdx.x == 0) atomicOr(p.err, kErrBadIndptr);
    kv0 = L = 0;
  }
  // position of the tiles' first token; tiles of keys each tile needs (its last token's)
  const int64_t pos0 = L - T + tok0;
  int n_kv[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    const int a = tok0 + s * p.tok_tile;
    const int e = a + p.tok_tile < T ? a + p.tok_tile : T;
    const int64_t seen = a < T ? L - T + e : 0;
    n_kv[s] = seen > 0 ? static_cast<int>((seen + kKeys - 1) / kKeys) : 0;
  }
  const int n_all = n_kv[0] > n_kv[1] ? n_kv[0] : n_kv[1];
  // K/V tiles from here on hold positions that some row does not see
  const int n_clear = pos0 + 1 > 0 ? static_cast<int>((pos0 + 1) / kKeys) : 0;

  if (warp == 9) {
    tmem_alloc(smem_u32(const_cast<uint32_t*>(tmem_slot)), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 8) {
    // ------------------------------------------------------------ TMA
    if (lane == 0 && n_all > 0) {
      const uint32_t box = static_cast<uint32_t>(p.tok_tile) * p.G * 128;
      const int nq = n_kv[1] > 0 ? 2 : 1;
      mbar_arrive_expect_tx(q_full, nq * KC * box);
      for (int s = 0; s < nq; ++s)
        for (int c = 0; c < KC; ++c)
          tma_3d(sbase + (s * KC + c) * kChunk, &tm_q, 64 * c, hk * p.G,
                 static_cast<int>(q0) + tok0 + s * p.tok_tile, q_full);
      // the barrier (and its phase) that chunk i, the c-th of tile j, completes on
      auto landing = [&](int i, int j, int c, uint32_t* parity) {
        const bool edge = c >= KC && j >= n_clear;
        *parity = edge ? 0 : (i / NC) & 1;
        return edge ? edge0 + 8 * (2 * (j - n_clear) + c - KC) : full0 + 8 * (i % NC);
      };
      int issued = 0;
      for (int j = 0, i = 0; j < n_all; ++j) {
        bool ok = true;
        for (int c = 0; c < KC + VC; ++c, ++i) {
          const int slot = i % NC;
          if (i >= NC && !mbar_wait(empty0 + 8 * slot, ((i / NC) - 1) & 1, abort_flag, p.err)) {
            ok = false;
            break;
          }
          uint32_t parity;
          const uint32_t bar = landing(i, j, c, &parity);
          if (bar != full0 + 8 * slot) mbar_arrive(full0 + 8 * slot);   // keeps its phases in step
          mbar_arrive_expect_tx(bar, kChunk);
          const bool is_k = c < KC;
          tma_3d(ring + slot * kChunk, is_k ? &tm_k : &tm_v, 64 * (is_k ? c : c - KC), hk,
                 static_cast<int>(kv0) + j * kKeys, bar);
          issued = i + 1;
        }
        if (!ok) break;
      }
      // no copy may be in flight when the CTA ends
      mbar_wait_drain(q_full, 0);
      for (int i = issued > NC ? issued - NC : 0; i < issued; ++i) {
        uint32_t parity;
        const uint32_t bar = landing(i, i / (KC + VC), i % (KC + VC), &parity);
        mbar_wait_drain(bar, parity);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    constexpr uint32_t id_qk = idesc_bf16(kKeys, false);
    constexpr uint32_t id_pv = idesc_bf16(DV, true), id_pv64 = idesc_bf16(64, true);
    bool ok = n_all > 0;
    auto wait = [&](uint32_t bar, uint32_t parity) {
      ok = ok && warp_bcast(mbar_wait(bar, parity, abort_flag, p.err));
      tc_fence_after();
    };
    auto wait_chunk = [&](int i) { wait(full0 + 8 * (i % NC), (i / NC) & 1); };
    auto free_chunks = [&](int i, int n) {
      for (int c = 0; c < n; ++c) mma_commit_warp(empty0 + 8 * ((i + c) % NC));
    };
    // S_s = Q_s K(j)^T, the chunks of K(j) from ring index i on
    auto qk = [&](int s, int i, bool wait_k) {
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        if (wait_k) wait_chunk(i + c);
        if (!ok) return;
        const uint64_t a = smem_desc(sbase + (s * KC + c) * kChunk, 16, 1024, kSw128);
        const uint64_t bd = smem_desc(ring + ((i + c) % NC) * kChunk, 16, 1024, kSw128);
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mma_ss(tmem + 128 * s, desc_at(a, 32 * k), desc_at(bd, 32 * k), id_qk, (c > 0 || k > 0) ? 1u : 0u);
      }
      mma_commit_warp(s_full + 8 * s);
    };
    // O_s += P_s V(j): 16 positions (8 columns of P, 16 rows of V) an MMA
    auto pv = [&](int s, int i, bool first) {
      const int slot = i % NC;
      const bool split = VC == 2 && slot == NC - 1;      // V's chunks lie at the ring's two ends
      const uint64_t v0 = smem_desc(ring + slot * kChunk, kChunk, 1024, kSw128);
      const uint64_t v1 = smem_desc(ring, kChunk, 1024, kSw128);
      const uint32_t o = tmem + 256 + 128 * s, pt = tmem + 128 * s;
#pragma unroll
      for (int k = 0; k < kKeys / 16; ++k) {
        const uint32_t acc = (!first || k > 0) ? 1u : 0u;
        if (!split) {
          mma_ts(o, pt + 8 * k, desc_at(v0, 2048 * k), id_pv, acc);
        } else {
          mma_ts(o, pt + 8 * k, desc_at(v0, 2048 * k), id_pv64, acc);
          mma_ts(o + 64, pt + 8 * k, desc_at(v1, 2048 * k), id_pv64, acc);
        }
      }
    };
    if (ok) {
      wait(q_full, 0);
      if (ok) qk(0, 0, true);
      if (ok && n_kv[1] > 0) qk(1, 0, n_kv[0] == 0);
      if (ok) free_chunks(0, KC);
    }
    for (int j = 0; j < n_all && ok; ++j) {
      const int iv = j * (KC + VC) + KC, ik = (j + 1) * (KC + VC);
      const int s_first = j < n_kv[0] ? 0 : 1;
      const int s_last = j < n_kv[1] ? 1 : 0;
      const int k_first = j + 1 < n_kv[0] ? 0 : 1, k_last = j + 1 < n_kv[1] ? 1 : 0;
      for (int s = s_first; s <= s_last && ok; ++s) {
        wait(p_full + 8 * s, j & 1);
        if (s == s_first) {
          if (j >= n_clear) {
            wait(clean0 + 8 * (j - n_clear), 0);
          } else {
            for (int c = 0; c < VC; ++c) wait_chunk(iv + c);
          }
        }
        if (!ok) break;
        pv(s, iv, j == 0);
        if (s == s_last) free_chunks(iv, VC);
        if (j + 1 < n_kv[s]) {
          qk(s, ik, s == k_first);
          if (!ok) break;
          if (s == k_last) free_chunks(ik, KC);
        } else {
          mma_commit_warp(o_full + 8 * s);
        }
      }
    }
    mma_commit_warp(drain);
    __syncwarp();
  } else if (warp >= 10) {
    // ------------------------------------------------------------ V on the edge
    const int ct = threadIdx.x - 320;
    bool ok = true;
    for (int j = n_clear; j < n_all && ok; ++j) {
      const int iv = j * (KC + VC) + KC;
      bool bad = false;
      for (int c = 0; c < VC && ok; ++c) {
        const int slot = (iv + c) % NC;
        ok = mbar_wait(edge0 + 8 * (2 * (j - n_clear) + c), 0, abort_flag, p.err);
        if (!ok) break;
        uint8_t* chunk = smem + S::kQBytes + slot * kChunk;
        // (the swizzle moves 16-byte words inside a 128-byte row only)
#pragma unroll 4
        for (int e = ct; e < 128 * 8; e += 64) {
          uint4* at = reinterpret_cast<uint4*>(chunk) + e;
          if (static_cast<int64_t>(j) * kKeys + (e >> 3) >= L) {
            *at = make_uint4(0, 0, 0, 0);
            continue;
          }
          uint4 x = *at;
          uint32_t w[4] = {x.x, x.y, x.z, x.w};
          bool any = false;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (half_nonfinite(w[i])) {
              w[i] &= 0xFFFF0000u;
              any = true;
            }
            if (half_nonfinite(w[i] >> 16)) {
              w[i] &= 0xFFFFu;
              any = true;
            }
          }
          if (any) {
            *at = make_uint4(w[0], w[1], w[2], w[3]);
            bad = true;
          }
        }
      }
      if (bad) *bad_v = 1;
      fence_proxy_async_smem();
      if (ok) mbar_arrive(clean0 + 8 * (j - n_clear));
    }
  } else {
    // ------------------------------------------------------------ softmax, one row a thread
    const int s = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = static_cast<uint32_t>(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + 128 * s + lane_base, t_o = tmem + 256 + 128 * s + lane_base;
    const int tt = r / p.G;
    const int tok = tok0 + s * p.tok_tile + tt;
    const bool live = tt < p.tok_tile && tok < T;
    // the last position the row sees (rows of no token: as the tile's last)
    const int64_t lim = L - T + (tok < T ? tok : T - 1);
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    for (int j = 0; j < n_kv[s]; ++j) {
      ok = warp_bcast(mbar_wait(s_full + 8 * s, j & 1, abort_flag, p.err));
      if (!ok) break;
      tc_fence_after();
      float x[128];
      tmem_ld32(t_s, x);
      tmem_ld32(t_s + 32, x + 32);
      tmem_ld32(t_s + 64, x + 64);
      tmem_ld32(t_s + 96, x + 96);
      tmem_wait_ld_regs(x, x + 16);
      tmem_wait_ld_regs(x + 32, x + 48);
      tmem_wait_ld_regs(x + 64, x + 80);
      tmem_wait_ld_regs(x + 96, x + 112);
      if (j >= n_clear) {
        const int64_t rel = lim - static_cast<int64_t>(j) * kKeys;
        const int last = rel < -1 ? -1 : (rel > kKeys ? kKeys : static_cast<int>(rel));
#pragma unroll
        for (int i = 0; i < 128; ++i) x[i] = i <= last ? x[i] : -INFINITY;
      }
      float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int i = 4; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], x[i]);
      const float mt = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      // raise the maximum where it grew by more than kRaise (always from -inf); each row by
      // itself, so that no row's result depends on its neighbours (or on idle rows)
      const bool raise = live && mt > m && !((mt - m) * p.scale_log2 <= kRaise);
      if (__any_sync(0xffffffffu, raise)) {
        const float mn = raise ? mt : m;
        const float f = m == mn ? 1.f : ex2_approx((m - mn) * p.scale_log2);   // 0 from -inf
        m = mn;
        l *= f;
        if (j > 0) {
#pragma unroll 1
          for (int c = 0; c < DV; c += 32) {
            float o[32];
            tmem_ld32(t_o + c, o);
            tmem_wait_ld_regs(o, o + 16);
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] *= f;
            tmem_st32(t_o + c, o);
          }
        }
      }
      const float off = m == -INFINITY ? 0.f : -m * p.scale_log2;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
      float pk[64];
#pragma unroll
      for (int i = 0; i < 64; ++i) {
        const float a = ex2_approx(fmaf(x[2 * i], p.scale_log2, off));
        const float c = ex2_approx(fmaf(x[2 * i + 1], p.scale_log2, off));
        sum[i & 1] += a;
        sum[2 + (i & 1)] += c;
        pk[i] = __uint_as_float(pack_bf16(a, c));
      }
      tmem_st32(t_s, pk);
      tmem_st32(t_s + 32, pk + 32);
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(p_full + 8 * s);
    }
    // ---- the row's result
    if (n_kv[s] > 0 && ok) ok = warp_bcast(mbar_wait(o_full + 8 * s, 0, abort_flag, p.err));
    if (ok && tok0 + s * p.tok_tile < T) {
      bool fix = false;
      for (int j = n_clear; j < n_kv[s] && ok; ++j)
        ok = warp_bcast(mbar_wait(clean0 + 8 * (j - n_clear), 0, abort_flag, p.err));
      if (n_kv[s] > n_clear) fix = *bad_v != 0;
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;
      const int h = hk * p.G + r - tt * p.G;
      uint16_t* orow = p.o + (q0 + tok) * p.o_tok + h * p.o_head;
#pragma unroll 1
      for (int c = 0; c < DV; c += 32) {
        float o[32];
        if (n_kv[s] > 0) {
          tmem_ld32(t_o + c, o);
          tmem_wait_ld_regs(o, o + 16);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] = l == 0.f ? 0.f : o[i] * inv;
        if (fix && live)
          for (int64_t j = static_cast<int64_t>(n_clear) * kKeys; j <= lim; ++j) {
            const uint16_t* vr = p.v + (kv0 + j) * p.v_tok + hk * p.v_head + c;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (half_nonfinite(vr[i])) o[i] += __uint_as_float(static_cast<uint32_t>(vr[i]) << 16);
          }
        if (live) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(orow + c + 8 * i) =
                make_uint4(pack_bf16(o[8 * i], o[8 * i + 1]), pack_bf16(o[8 * i + 2], o[8 * i + 3]),
                           pack_bf16(o[8 * i + 4], o[8 * i + 5]), pack_bf16(o[8 * i + 6], o[8 * i + 7]));
        }
      }
      if (live && p.lse)
        p.lse[(q0 + tok) * p.Hq + h] =
            l == 0.f ? -INFINITY : ((m == -INFINITY ? 0.f : m) * p.scale_log2) * kLn2 + logf(l);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    if (lane == 0) mbar_wait_drain(drain, 0);   // all issued MMAs complete (bounded)
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
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
                   const PromptParams& p, unsigned grid, cudaStream_t stream) {
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
  prompt_attention_kernel<S><<<grid, kThreads, S::kSmem, stream>>>(tq, tk, tv, p);
  return cudaGetLastError();
}

// Strides TMA can step: positive where the dim has more than one entry.
bool steppable(const mla_tensor_t* t) {
  return (t->shape[0] <= 1 || t->stride[0] > 0) && (t->shape[1] <= 1 || t->stride[1] > 0);
}

}  // namespace
}  // namespace pmla

extern "C" int mla_prompt_attention(const mla_tensor_t* q, const mla_tensor_t* k,
                                    const mla_tensor_t* v, const mla_tensor_t* o,
                                    const mla_tensor_t* qo_indptr, const mla_tensor_t* kv_indptr,
                                    float sm_scale, const mla_tensor_t* lse_out,
                                    int32_t* error_word, mla_stream_t stream_) {
  using namespace pmla;
  if (!q || !k || !v || q->ndim != 3 || k->ndim != 3 || v->ndim != 3) return MLA_ERR_INVALID_ARG;
  const int64_t n_tok = q->shape[0], Hq = q->shape[1], D = q->shape[2];
  const int64_t n_keys = k->shape[0], Hk = k->shape[1], DV = v->shape[2];
  if (n_tok < 0 || n_keys < 0 || n_tok >= 0x7FFFFF00 || n_keys >= 0x7FFFFF00) return MLA_ERR_INVALID_ARG;
  if (Hq < 1 || Hk < 1 || Hq > 1024 || Hq % Hk != 0) return MLA_ERR_INVALID_ARG;
  if (!gqa_check_bf16(q, n_tok, Hq, D, 8) || !gqa_check_bf16(k, n_keys, Hk, D, 8) ||
      !gqa_check_bf16(v, n_keys, Hk, DV, 8) || !gqa_check_bf16(o, n_tok, Hq, DV, 8))
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
  if (n_tok == 0 || B == 0) return MLA_OK;

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
  p.v = static_cast<const uint16_t*>(v->ptr);
  p.v_tok = v->stride[0];
  p.v_head = v->stride[1];
  p.err = error_word;
  // every request has at most one tile that is not full
  const int64_t tiles = n_tok / (2 * p.tok_tile) + (B < n_tok ? B : n_tok);
  if (tiles * Hk > 0x7FFFFFFF) return MLA_ERR_UNSUPPORTED;
  const unsigned grid = static_cast<unsigned>(tiles * Hk);

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
  if (s64) e = launch<64, 64>(tq, tk, tv, p, grid, s);
  else if (s128) e = launch<128, 128>(tq, tk, tv, p, grid, s);
  else e = launch<192, 128>(tq, tk, tv, p, grid, s);
  return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
