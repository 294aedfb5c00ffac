// mla_build_page_table: the page table of a step built on the device from the requests' lengths,
// pages for the new tokens taken from a stack of free ones, and the positions and cache slots
// of the new tokens.
//
// With L_b positions after the step, T_b of them new, and pages of PS: P_b = ceil(L_b / PS)
// pages, of which O_b = ceil((L_b - T_b) / PS) were there; the others take the stack's topmost
// ids in the requests' order, so the result does not depend on which block runs first.  Whole
// numbers only: running sums of P, T, L and P - O over the requests, then one entry after
// another.
//
// Bound by latency in a step (launch, the lengths, the sums, a table entry: three dependent
// round trips), by the bytes of the lists where pages are small.  Every block forms the sums of
// all requests for itself (a few microseconds less than a second launch that waits for them)
// and then takes groups of four entries of the lists, found by bisection in shared memory.
//
// Measured (one GB300, in a CUDA graph): 64 requests of up to 65,536 positions, one new token each, pages
// of 128: 5.1 us; 24 of 68,000 positions, 4,089 new, one-token pages, 7.4 MB of lists: 7.2 us (8.0 with two
// blocks a SM and the stack's count claimed at the end; 6.4 and 7.2 with it read and claimed by a thread that
// writes entries, too).
#include <cuda_runtime.h>
#include <stdint.h>

#include <mutex>

#include "../../include/paged_mla.h"
#include "mla_gqa_check.h"
#include "ptx.cuh"

namespace {

using namespace pmla;

constexpr int kThreads = 256, kWarps = kThreads / 32;        // a block's, and a warp for the pool's count
constexpr int kBlock = kThreads + 32;
constexpr int kEach = 4;               // consecutive entries a thread takes
constexpr int64_t kMaxRequests = 16384;      // three sums of each in shared memory
constexpr int64_t kIntMax = 0x7FFFFFFF;

struct PageTableParams {
  const int32_t *seq_lens, *new_lens;
  int32_t* table;
  int64_t table_row;
  int max_pages;
  int log2_page;
  int B;
  const int32_t *free_pages, *free_count;    // null: no pool
  int64_t n_pool;
  int32_t* free_count_out;
  int32_t *qo_indptr, *key_indptr, *kv_indptr, *kv_indices, *last;
  int64_t n_idx;
  int32_t *positions, *slots;
  int64_t n_tok;                             // -1: neither is wanted
  int* err;                                  // error bits, arrivals
};

struct Sums {
  int64_t pages, tokens, keys, taken;
  __device__ Sums operator+(const Sums& o) const {
    return {pages + o.pages, tokens + o.tokens, keys + o.keys, taken + o.taken};
  }
};

__device__ __forceinline__ Sums shfl_up(const Sums& s, int d) {
  return {__shfl_up_sync(0xffffffffu, s.pages, d), __shfl_up_sync(0xffffffffu, s.tokens, d),
          __shfl_up_sync(0xffffffffu, s.keys, d), __shfl_up_sync(0xffffffffu, s.taken, d)};
}

__device__ __forceinline__ int32_t saturated(int64_t x) { return static_cast<int32_t>(x < kIntMax ? x : kIntMax); }

// The last request that starts at or before entry i (pre[0 .. B], i < pre[B]).
__device__ __forceinline__ int owner(const int32_t* pre, int B, int64_t i) {
  int lo = 0, hi = B;                        // pre[lo] <= i < pre[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid] <= i) lo = mid;
    else hi = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(kBlock) page_table_kernel(const PageTableParams p) {
  extern __shared__ int32_t s_pre[];         // running sums: pages, tokens, pages taken
  int32_t* s_kv = s_pre;
  int32_t* s_qo = s_kv + p.B + 1;
  int32_t* s_taken = s_qo + p.B + 1;
  __shared__ Sums s_warp[kWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int ps_mask = (1 << p.log2_page) - 1;
  __shared__ int32_t s_held;                 // the pool's count, read once for all of the block
  const bool counts = tid == kThreads;
  if (counts) s_held = p.free_count ? __ldcg(p.free_count) : 0;

  Sums run = {};
  for (int b0 = 0; b0 < p.B || b0 == 0; b0 += kThreads) {
    const int b = tid < kThreads ? b0 + tid : p.B;
    Sums x = {};
    int last = ps_mask + 1;                  // of no page: the formula all the same
    if (b < p.B) {
      const int64_t len = __ldg(p.seq_lens + b), fresh = __ldg(p.new_lens + b);
      const int64_t pages = (len + ps_mask) >> p.log2_page;
      if (len >= 0 && fresh >= 0 && fresh <= len && pages <= p.max_pages) {
        const int64_t had = (len - fresh + ps_mask) >> p.log2_page;
        x = {pages, fresh, len, p.free_count ? pages - had : 0};
        if (len > 0) last = static_cast<int>(len - ((pages - 1) << p.log2_page));
      } else if (blockIdx.x == 0) {
        atomicOr(p.err, kErrBadIndptr);
      }
    }
    Sums inc = x;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const Sums o = shfl_up(inc, d);
      if (lane >= d) inc = inc + o;
    }
    __syncthreads();
    if (lane == 31 && warp < kWarps) s_warp[warp] = inc;
    __syncthreads();
    Sums all = run;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w == warp) inc = inc + all;
      all = all + s_warp[w];
    }
    run = all;
    if (b < p.B) {
      s_kv[b + 1] = saturated(inc.pages);
      s_qo[b + 1] = saturated(inc.tokens);
      s_taken[b + 1] = saturated(inc.taken);
      if (blockIdx.x == 0) {
        p.kv_indptr[b + 1] = saturated(inc.pages);
        p.qo_indptr[b + 1] = saturated(inc.tokens);
        p.key_indptr[b + 1] = saturated(inc.keys);
        p.last[b] = last;
      }
    }
  }
  if (tid == 0) s_kv[0] = s_qo[0] = s_taken[0] = 0;
  const bool cut = run.pages > p.n_idx || run.keys > kIntMax || (p.n_tok >= 0 && run.tokens > p.n_tok);
  if (run.pages > kIntMax) run = {};         // no lists of pages that their sums cannot tell apart
  __syncthreads();
  const int32_t held = s_held;
  const int64_t n_free = held >= 0 && held <= p.n_pool ? held : 0;
  if (warp == kWarps) {
    // The count may be written in place, so a block arrives when it has read it, and the one that
    // arrives last writes it.  (By a warp that writes nothing else: fences wait for a warp's
    // stores, 1.5 us on a warp with entries of the lists.)
    if (counts && p.free_count_out) {
      bool last = true;
      if (gridDim.x > 1) {
        __threadfence();                     // the read before the arrival
        last = atomicAdd(p.err + 1, 1) == static_cast<int>(gridDim.x) - 1;
        __threadfence();                     // the others' arrivals before the write
        if (last) p.err[1] = 0;              // as it was found, for the next call
      }
      if (last) *p.free_count_out = held - static_cast<int32_t>(run.taken < n_free ? run.taken : n_free);
    }
    return;
  }
  if (tid == 0 && blockIdx.x == 0) {
    p.kv_indptr[0] = p.qo_indptr[0] = p.key_indptr[0] = 0;
    if (cut) atomicOr(p.err, kErrBadOutput);
    if (run.taken > n_free) atomicOr(p.err, kErrBadIndex);
  }

  // page j of request b: one that it had, or a new one by its place in the stack
  auto page_of = [&](int b, int j, int fresh_from) -> int32_t {
    if (j < fresh_from) return __ldg(p.table + b * p.table_row + j);
    const int64_t nth = n_free - 1 - (static_cast<int64_t>(s_taken[b]) + j - fresh_from);
    return nth >= 0 ? __ldg(p.free_pages + nth) : -1;
  };
  auto fresh_from = [&](int b) -> int {      // the first page of request b that is taken now
    return s_kv[b + 1] - s_kv[b] - (s_taken[b + 1] - s_taken[b]);
  };

  const int64_t n_list = run.pages;
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kThreads * kEach;
  const int64_t first = (static_cast<int64_t>(blockIdx.x) * kThreads + tid) * kEach;
  for (int64_t i0 = first; i0 < n_list; i0 += stride) {
    int b = owner(s_kv, p.B, i0);
    int from = fresh_from(b);
    int32_t page[kEach];
#pragma unroll
    for (int k = 0; k < kEach; ++k) {
      if (i0 + k >= n_list) break;
      while (i0 + k >= s_kv[b + 1]) from = fresh_from(++b);
      const int j = static_cast<int>(i0 + k - s_kv[b]);
      page[k] = page_of(b, j, from);
      if (j >= from) p.table[b * p.table_row + j] = page[k];
    }
#pragma unroll
    for (int k = 0; k < kEach; ++k)
      if (i0 + k < n_list && i0 + k < p.n_idx) p.kv_indices[i0 + k] = page[k];
  }
  if (p.n_tok > 0) {
    const int64_t total = run.tokens < kIntMax ? run.tokens : kIntMax;
    for (int64_t i0 = first; i0 < p.n_tok; i0 += stride) {
      int b = i0 < total ? owner(s_qo, p.B, i0) : 0;
#pragma unroll
      for (int k = 0; k < kEach; ++k) {
        const int64_t i = i0 + k;
        if (i >= p.n_tok) break;
        int32_t position = 0, slot = -1;     // behind the last request: no token
        if (i < total) {
          while (i >= s_qo[b + 1]) ++b;
          position = __ldg(p.seq_lens + b) - __ldg(p.new_lens + b) + static_cast<int32_t>(i - s_qo[b]);
          const int32_t page = page_of(b, position >> p.log2_page, fresh_from(b));
          const int64_t at = (static_cast<int64_t>(page) << p.log2_page) + (position & ps_mask);
          if (page >= 0 && at <= kIntMax) slot = static_cast<int32_t>(at);
          else atomicOr(p.err, kErrBadIndex);
        }
        p.positions[i] = position;
        p.slots[i] = slot;
      }
    }
  }
}

bool out_i32(const mla_tensor_t* t, int64_t n) { return gqa_check_i32(t, n) && (t->ptr || n == 0); }

}  // namespace

extern "C" int mla_build_page_table(const mla_tensor_t* seq_lens, const mla_tensor_t* new_lens,
                                    const mla_tensor_t* block_table, int32_t page_size,
                                    const mla_tensor_t* free_pages, const mla_tensor_t* free_count,
                                    const mla_tensor_t* free_count_out,
                                    const mla_tensor_t* qo_indptr, const mla_tensor_t* key_indptr,
                                    const mla_tensor_t* kv_indptr, const mla_tensor_t* kv_indices,
                                    const mla_tensor_t* kv_last_page_lens,
                                    const mla_tensor_t* positions, const mla_tensor_t* slot_mapping,
                                    int32_t* error_word, mla_stream_t stream_) {
  if (!seq_lens || seq_lens->ndim != 1) return MLA_ERR_INVALID_ARG;
  const int64_t B = seq_lens->shape[0];
  if (B < 0 || !gqa_check_i32(seq_lens, B) || !gqa_check_i32(new_lens, B)) return MLA_ERR_INVALID_ARG;
  if (!block_table || block_table->dtype != MLA_DTYPE_INT32 || block_table->ndim != 2 ||
      block_table->shape[0] != B || block_table->shape[1] < 0 || !gqa_aligned(block_table->ptr, 4))
    return MLA_ERR_INVALID_ARG;
  const int64_t width = block_table->shape[1];
  if (!block_table->ptr && B * width != 0) return MLA_ERR_INVALID_ARG;
  if ((width > 1 && block_table->stride[1] != 1) || (B > 1 && block_table->stride[0] < width))
    return MLA_ERR_INVALID_ARG;
  if (page_size < 1) return MLA_ERR_INVALID_ARG;
  if (page_size > 1024 || (page_size & (page_size - 1)) != 0) return MLA_ERR_UNSUPPORTED;
  if (width > kIntMax / page_size) return MLA_ERR_INVALID_ARG;
  const bool pool = free_pages || free_count || free_count_out;
  if (pool && (!free_pages || free_pages->ndim != 1 || !gqa_check_i32(free_pages, free_pages->shape[0]) ||
               !gqa_check_scalar_i32(free_count) || !gqa_check_scalar_i32(free_count_out)))
    return MLA_ERR_INVALID_ARG;
  if (!out_i32(qo_indptr, B + 1) || !out_i32(key_indptr, B + 1) || !out_i32(kv_indptr, B + 1) ||
      !out_i32(kv_last_page_lens, B))
    return MLA_ERR_INVALID_ARG;
  if (!kv_indices || kv_indices->ndim != 1 || !out_i32(kv_indices, kv_indices->shape[0]))
    return MLA_ERR_INVALID_ARG;
  if (!positions != !slot_mapping) return MLA_ERR_INVALID_ARG;
  if (positions && (positions->ndim != 1 || !out_i32(positions, positions->shape[0]) ||
                    !out_i32(slot_mapping, positions->shape[0])))
    return MLA_ERR_INVALID_ARG;
  if (!error_word || !gqa_aligned(error_word, 4)) return MLA_ERR_INVALID_ARG;
  if (B > kMaxRequests) return MLA_ERR_UNSUPPORTED;

  PageTableParams p = {};
  p.seq_lens = static_cast<const int32_t*>(seq_lens->ptr);
  p.new_lens = static_cast<const int32_t*>(new_lens->ptr);
  p.table = static_cast<int32_t*>(block_table->ptr);
  p.table_row = B > 1 ? block_table->stride[0] : 0;
  p.max_pages = static_cast<int>(width);
  while ((1 << p.log2_page) < page_size) ++p.log2_page;
  p.B = static_cast<int>(B);
  if (pool) {
    p.free_pages = static_cast<const int32_t*>(free_pages->ptr);
    p.n_pool = free_pages->shape[0];
    p.free_count = static_cast<const int32_t*>(free_count->ptr);
    p.free_count_out = static_cast<int32_t*>(free_count_out->ptr);
  }
  p.qo_indptr = static_cast<int32_t*>(qo_indptr->ptr);
  p.key_indptr = static_cast<int32_t*>(key_indptr->ptr);
  p.kv_indptr = static_cast<int32_t*>(kv_indptr->ptr);
  p.kv_indices = static_cast<int32_t*>(kv_indices->ptr);
  p.n_idx = kv_indices->shape[0];
  p.last = static_cast<int32_t*>(kv_last_page_lens->ptr);
  p.n_tok = -1;
  if (positions) {
    p.positions = static_cast<int32_t*>(positions->ptr);
    p.slots = static_cast<int32_t*>(slot_mapping->ptr);
    p.n_tok = positions->shape[0];
  }
  p.err = error_word;

  static std::mutex mu;
  static bool attr_set[64] = {};
  int dev = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MLA_ERR_CUDA;
  const size_t smem = 3 * (static_cast<size_t>(B) + 1) * sizeof(int32_t);
  if (smem > 40 * 1024) {
    std::lock_guard<std::mutex> lk(mu);
    if (!attr_set[dev]) {
      if (cudaFuncSetAttribute(page_table_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               static_cast<int>(3 * (kMaxRequests + 1) * sizeof(int32_t))) != cudaSuccess)
        return MLA_ERR_CUDA;
      attr_set[dev] = true;
    }
  }
  const int64_t longest = p.n_idx > p.n_tok ? p.n_idx : p.n_tok;
  int64_t blocks = (longest + kThreads * kEach - 1) / (kThreads * kEach);
  if (blocks > 4 * sms) blocks = 4 * sms;
  if (blocks < 1) blocks = 1;
  page_table_kernel<<<static_cast<unsigned>(blocks), kBlock, smem, reinterpret_cast<cudaStream_t>(stream_)>>>(p);
  return cudaGetLastError() == cudaSuccess ? MLA_OK : MLA_ERR_CUDA;
}
