// Host simulation of the page table's kernel (test-suite only): the kernel's own source, which the
// test writes to page_table_kernel.inc, over a call's arrays.
#include "cuda_host.h"

#include "../../include/paged_mla.h"
#include "../../paged_mla_latent_gb300/csrc/mla_gqa_check.h"

#include "page_table_kernel.inc"

// n: B, width, log2 of the page size, F, entries of kv_indices and of positions, blocks.
// a: seq_lens, new_lens, block_table, free_pages, free_count, free_count_out, qo, key, kv, indices, last,
// positions, slots, error word (null as in the call).
extern "C" int page_table(const int64_t* n, int32_t* const* a, const int* order) {
  PageTableParams p = {};
  p.B = static_cast<int>(n[0]);
  p.table_row = n[1];
  p.max_pages = static_cast<int>(n[1]);
  p.log2_page = static_cast<int>(n[2]);
  p.n_pool = n[3];
  p.n_idx = n[4];
  p.n_tok = n[5];
  p.seq_lens = a[0];
  p.new_lens = a[1];
  p.table = a[2];
  p.free_pages = a[3];
  p.free_count = a[4];
  p.free_count_out = a[5];
  p.qo_indptr = a[6];
  p.key_indptr = a[7];
  p.kv_indptr = a[8];
  p.kv_indices = a[9];
  p.last = a[10];
  p.positions = a[11];
  p.slots = a[12];
  p.err = a[13];
  sim::grid.x = static_cast<unsigned>(n[6]);
  return sim::run(static_cast<int>(n[6]), kBlock, order, [&] { page_table_kernel(p); }) ? 0 : -1;
}
