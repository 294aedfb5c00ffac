// mla_gqa_block_gather: requests' keys and values as packed bf16 rows for mla_prompt_attention,
// the cached positions from a paged e4m3 cache with a scale for each block and head, the newest
// ones from the step's own keys and values.
//
//   k_rows[row_indptr[b] + j] = bf16(code * scale)            (j < L_b - T_b, or T_b = 0)
//                             = k_new[qo_indptr[b] + j - (L_b - T_b)]
//
// Bytes bound: a byte read and two written an element, no arithmetic to speak of.  Blocks go from
// tile to tile of rows.  One warp looks a tile ahead for where its rows come from (the request by
// bisection over the starts in shared memory, its lists, its page: three round trips to memory),
// the others copy, eight columns of a row at a time, K and V together.
//
// Measured (one GB300, in a CUDA graph): 63,911 cached and 4,089 new positions, 8 heads of 128, 426
// MB: 72 us, 5.9 TB/s, which a plain copy of as many bytes takes, too (75 us; 85 us without the
// warp ahead, a block a tile); 53 prompts of 1 to 700 tokens behind 0 to 300, two heads of 64: 5 us.
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

constexpr int kCopy = 256, kThreads = kCopy + 32;        // copying threads, and a warp ahead of them
constexpr int kMostRows = 32;               // rows of a tile, a lane each of that warp
constexpr int kMostStarts = 1024;           // requests whose starts fit shared memory

struct BlockGatherParams {
  const uint8_t *k, *v;
  int64_t page_pitch, slot_pitch, head_pitch;
  int64_t n_pages;
  const float *ks, *vs;
  int64_t sc_page, sc_block, sc_head;
  int log2_block;
  PageList pages;
  const int32_t *row_indptr, *qo_indptr;    // qo_indptr null: every position from the cache
  const uint16_t *k_new, *v_new;
  int64_t kn_tok, kn_head, vn_tok, vn_head;
  int64_t n_new;
  uint16_t *k_rows, *v_rows;
  int64_t ko_tok, ko_head, vo_tok, vo_head;
  int64_t n_rows;
  int B, Hk, pieces;                        // 8-column pieces of a head's row
  int tile;                                 // rows a block of threads takes
  int* err;
};

// Where a row comes from.
struct Source {
  int64_t at;                               // bytes into the caches, or the new token; -1: nowhere
  int64_t scale;                            // elements into the scales; -1: a new token, or nowhere
};
constexpr int64_t kZeros = -2;              // a scale: the page is outside the cache

__device__ __forceinline__ uint4 widen(const uint2& codes, float scale) {
  uint32_t r[4];
  const uint32_t c[2] = {codes.x, codes.y};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t h = e4m3x2_to_f16x2(c[i >> 1] >> (16 * (i & 1)));
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
    const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * scale, f.y * scale);
    r[i] = *reinterpret_cast<const uint32_t*>(&b);
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

// The last request that starts at or before a row.  Starts rise; with kBad, but for those outside the
// output: the next one that is not speaks for them.
template <bool kBad, class Start>
__device__ __forceinline__ int request_at(const BlockGatherParams& p, int64_t row, Start start) {
  int lo = 0, hi = p.B;                     // the answer lies in [lo, hi)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    int at = mid;
    int64_t s = start(at);
    if constexpr (kBad)
      while ((s < 0 || s > p.n_rows) && ++at < hi) s = start(at);
    if (s <= row && (!kBad || at < hi)) lo = at;
    else hi = mid;
  }
  return lo;
}

// Where a row of the output comes from, by its request's lists.
template <class Start>
__device__ __forceinline__ Source source_of(const BlockGatherParams& p, int64_t row, Start start) {
  Source from = {-1, -1};
  if (row >= p.n_rows) return from;
  int lo = request_at<false>(p, row, start);
  int64_t s = start(lo), e = start(lo + 1);
  if (row < s || row >= e || s < 0 || e > p.n_rows) {          // a row of none, or hidden by a bad list
    lo = request_at<true>(p, row, start);
    s = start(lo);
    e = start(lo + 1);
    if (row < s || row >= e) return from;
  }
  const int held = p.pages.positions(lo);
  const int64_t idx0 = __ldg(p.pages.indptr + lo);
  int64_t t0 = 0, t1 = 0;
  if (p.qo_indptr) {
    t0 = __ldg(p.qo_indptr + lo);
    t1 = __ldg(p.qo_indptr + lo + 1);
  }
  if (held < 0 || s < 0 || e - s != held || e > p.n_rows || t0 < 0 || t1 < t0 || t1 > p.n_new || t1 - t0 > held) return from;
  const int j = static_cast<int>(row - s), cached = held - static_cast<int>(t1 - t0);
  if (j >= cached) {
    from.at = t0 + j - cached;
    return from;
  }
  const int64_t page = __ldg(p.pages.indices + idx0 + (j >> p.pages.log2_page));
  if (page >= 0 && page < p.n_pages) {
    const int slot = j & ((1 << p.pages.log2_page) - 1);
    from.at = page * p.page_pitch + slot * p.slot_pitch;
    from.scale = page * p.sc_page + (slot >> p.log2_block) * p.sc_block;
  } else {
    from.scale = kZeros;
    atomicOr(p.err, kErrBadRowId);
  }
  return from;
}

__global__ void __launch_bounds__(kThreads, 4) gqa_block_gather_kernel(const BlockGatherParams p) {
  __shared__ int32_t s_start[kMostStarts + 1];
  __shared__ Source s_from[2][kMostRows];
  const int tid = threadIdx.x;
  const bool fits = p.B <= kMostStarts;
  if (fits) {
    for (int i = tid; i <= p.B; i += kThreads) s_start[i] = __ldg(p.row_indptr + i);
    __syncthreads();
  }
  auto start = [&](int b) -> int64_t { return fits ? s_start[b] : __ldg(p.row_indptr + b); };
  const int64_t end = start(p.B), rows = end < 0 || end > p.n_rows ? p.n_rows : end;
  const bool ahead = tid >= kCopy;
  int64_t row0 = static_cast<int64_t>(blockIdx.x) * p.tile;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * p.tile;
  if (ahead) {
    if (tid - kCopy < p.tile) s_from[0][tid - kCopy] = source_of(p, row0 + tid - kCopy, start);
  } else {
    // requests whose lists make no sense: the copying threads look them over first
    for (int64_t b = static_cast<int64_t>(blockIdx.x) * kCopy + tid; b < p.B; b += static_cast<int64_t>(gridDim.x) * kCopy) {
      const int held = p.pages.positions(static_cast<int>(b));
      const int64_t s = start(b), e = start(b + 1);
      bool sound = held >= 0 && s >= 0 && e - s == held && e <= p.n_rows;
      if (p.qo_indptr) {
        const int64_t t0 = __ldg(p.qo_indptr + b), t1 = __ldg(p.qo_indptr + b + 1);
        sound = sound && t0 >= 0 && t1 >= t0 && t1 <= p.n_new && t1 - t0 <= held;
      }
      if (!sound) atomicOr(p.err, kErrBadIndptr);
    }
  }
  const int columns = p.Hk * p.pieces;      // 8-column pieces of a row
  const int at_once = columns < kCopy ? kCopy / columns : 1;      // rows
  const int first = tid / (columns < kCopy ? columns : kCopy);
  const int c0 = columns < kCopy ? tid - first * columns : tid;
  int buf = 0;
  __syncthreads();
#pragma unroll 1
  for (; row0 < rows; row0 += stride, buf ^= 1) {
    if (ahead) {
      if (row0 + stride < rows && tid - kCopy < p.tile)
        s_from[buf ^ 1][tid - kCopy] = source_of(p, row0 + stride + tid - kCopy, start);
    } else if (first < at_once) {
#pragma unroll 1
      for (int c = c0; c < columns; c += kCopy) {
        const int h = c / p.pieces, col = 8 * (c - h * p.pieces);
        const int64_t in = h * p.head_pitch + col, sc = h * p.sc_head;
        constexpr int kAtOnce = 2;
#pragma unroll 1
        for (int r0 = first; r0 < p.tile; r0 += kAtOnce * at_once) {
          uint2 kc[kAtOnce], vc[kAtOnce];
          float ks[kAtOnce], vs[kAtOnce];
          Source from[kAtOnce];
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            const int r = r0 + i * at_once;
            from[i] = r < p.tile ? s_from[buf][r] : Source{-1, -1};
            kc[i] = vc[i] = make_uint2(0, 0);
            if (from[i].scale >= 0) {
              kc[i] = __ldg(reinterpret_cast<const uint2*>(p.k + from[i].at + in));
              vc[i] = __ldg(reinterpret_cast<const uint2*>(p.v + from[i].at + in));
              ks[i] = __ldg(p.ks + from[i].scale + sc);
              vs[i] = __ldg(p.vs + from[i].scale + sc);
            }
          }
#pragma unroll
          for (int i = 0; i < kAtOnce; ++i) {
            if (from[i].at < 0 && from[i].scale != kZeros) continue;
            uint4 k = make_uint4(0, 0, 0, 0), v = k;
            if (from[i].scale >= 0) {
              k = widen(kc[i], ks[i]);
              v = widen(vc[i], vs[i]);
            } else if (from[i].at >= 0) {
              k = __ldg(reinterpret_cast<const uint4*>(p.k_new + from[i].at * p.kn_tok + h * p.kn_head + col));
              v = __ldg(reinterpret_cast<const uint4*>(p.v_new + from[i].at * p.vn_tok + h * p.vn_head + col));
            }
            const int64_t row = row0 + r0 + i * at_once;
            *reinterpret_cast<uint4*>(p.k_rows + row * p.ko_tok + h * p.ko_head + col) = k;
            *reinterpret_cast<uint4*>(p.v_rows + row * p.vo_tok + h * p.vo_head + col) = v;
          }
        }
      }
    }
    __syncthreads();
  }
}

}  // namespace

extern "C" int mla_gqa_block_gather(const mla_tensor_t* k_cache, const mla_tensor_t* v_cache,
                                    const mla_tensor_t* k_scale, const mla_tensor_t* v_scale,
                                    const mla_tensor_t* kv_indptr, const mla_tensor_t* kv_indices,
                                    const mla_tensor_t* kv_last_page_lens,
                                    const mla_tensor_t* row_indptr, const mla_tensor_t* qo_indptr,
                                    const mla_tensor_t* k_new, const mla_tensor_t* v_new,
                                    const mla_tensor_t* k_rows, const mla_tensor_t* v_rows,
                                    int32_t* error_word, mla_stream_t stream_) {
  if (!k_cache || !row_indptr || !k_rows || k_cache->ndim != 4 || row_indptr->ndim != 1 || k_rows->ndim != 3)
    return MLA_ERR_INVALID_ARG;
  const int64_t Hk = k_cache->shape[2], D = k_cache->shape[3], B = row_indptr->shape[0] - 1, n = k_rows->shape[0];
  if (Hk < 1 || Hk > 1024 || B < 0 || B > 0xFFFFFF || n < 0 || n > 0x7FFFFFFF) return MLA_ERR_INVALID_ARG;
  GqaBlockCache c;
  const int st = gqa_check_block_cache(k_cache, v_cache, k_scale, v_scale, Hk, D, &c);
  if (st != MLA_OK) return st;
  if (!gqa_check_i32(row_indptr, B + 1) ||
      !gqa_check_pages(kv_indptr, kv_indices, kv_last_page_lens, B, c.log2_page))
    return MLA_ERR_INVALID_ARG;
  if (!qo_indptr != !k_new || !qo_indptr != !v_new) return MLA_ERR_INVALID_ARG;
  int64_t n_new = 0;
  if (qo_indptr) {
    if (k_new->ndim != 3) return MLA_ERR_INVALID_ARG;
    n_new = k_new->shape[0];
    if (n_new < 0 || !gqa_check_i32(qo_indptr, B + 1) || !gqa_check_bf16(k_new, n_new, Hk, D, 8) ||
        !gqa_check_bf16(v_new, n_new, Hk, D, 8))
      return MLA_ERR_INVALID_ARG;
  }
  if (!gqa_check_bf16(k_rows, n, Hk, D, 8) || !gqa_check_bf16(v_rows, n, Hk, D, 8) ||
      !gqa_rows_apart(k_rows) || !gqa_rows_apart(v_rows))
    return MLA_ERR_INVALID_ARG;
  if (!error_word || !gqa_aligned(error_word, 4)) return MLA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return MLA_ERR_UNSUPPORTED;
  if (B == 0 || n == 0) return MLA_OK;

  BlockGatherParams p = {};
  p.k = c.k;
  p.v = c.v;
  p.page_pitch = c.page_pitch;
  p.slot_pitch = c.slot_pitch;
  p.head_pitch = c.head_pitch;
  p.n_pages = c.n_pages;
  p.ks = c.ks;
  p.vs = c.vs;
  p.sc_page = c.sc_page;
  p.sc_block = c.sc_block;
  p.sc_head = c.sc_head;
  p.log2_block = c.log2_block;
  p.pages.indptr = static_cast<const int32_t*>(kv_indptr->ptr);
  p.pages.indices = static_cast<const int32_t*>(kv_indices->ptr);
  p.pages.last = kv_last_page_lens ? static_cast<const int32_t*>(kv_last_page_lens->ptr) : nullptr;
  p.pages.n_idx = kv_indices->shape[0];
  p.pages.log2_page = c.log2_page;
  p.row_indptr = static_cast<const int32_t*>(row_indptr->ptr);
  if (qo_indptr) {
    p.qo_indptr = static_cast<const int32_t*>(qo_indptr->ptr);
    p.k_new = static_cast<const uint16_t*>(k_new->ptr);
    p.v_new = static_cast<const uint16_t*>(v_new->ptr);
    p.kn_tok = k_new->stride[0];
    p.kn_head = k_new->stride[1];
    p.vn_tok = v_new->stride[0];
    p.vn_head = v_new->stride[1];
  }
  p.n_new = n_new;
  p.k_rows = static_cast<uint16_t*>(k_rows->ptr);
  p.v_rows = static_cast<uint16_t*>(v_rows->ptr);
  p.ko_tok = k_rows->stride[0];
  p.ko_head = k_rows->stride[1];
  p.vo_tok = v_rows->stride[0];
  p.vo_head = v_rows->stride[1];
  p.n_rows = n;
  p.B = static_cast<int>(B);
  p.Hk = static_cast<int>(Hk);
  p.pieces = static_cast<int>(D / 8);
  // about 16 K columns of K and as many of V a tile, whole waves of resident blocks
  p.tile = kMostRows;
  while (p.tile > 8 && p.tile * Hk * D > 16384) p.tile /= 2;
  p.err = error_word;
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  int64_t blocks = (n + p.tile - 1) / p.tile;
  if (blocks > 4 * static_cast<int64_t>(sms)) blocks = 4 * sms;
  gqa_block_gather_kernel<<<static_cast<unsigned>(blocks), kThreads, 0, reinterpret_cast<cudaStream_t>(stream_)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
