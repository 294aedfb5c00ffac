// Page lists on the device, for kernels that walk requests' positions.
#pragma once

#include <stdint.h>

namespace pmla {

struct PageList {
  const int32_t *indptr, *indices, *last;   // last: null for one-token pages
  int64_t n_idx;
  int log2_page;

  // Positions of request b; -1 where its list makes no sense.
  __device__ __forceinline__ int positions(int b) const {
    const int64_t s = __ldg(indptr + b), e = __ldg(indptr + b + 1);
    const int ps = 1 << log2_page;
    const int fill = last ? __ldg(last + b) : ps;
    if (s < 0 || e < s || e > n_idx) return -1;
    if (e == s) return 0;
    const int64_t n = ((e - s - 1) << log2_page) + (fill < 1 ? 1 : (fill > ps ? ps : fill));
    return n > 0x7FFFFF00 ? -1 : static_cast<int>(n);
  }
};

// The last b in [0, n) with start(b) <= x, by a whole warp (starts rise): 31 probes at a time, so
// that lists of up to 32 take one round trip to memory, of 1,024 two.  With kBad, starts may be
// negative, where a list's entry makes no sense: the next one that does speaks for a probe's stretch.
template <bool kBad, class Start>
__device__ __forceinline__ int warp_owner(int n, int lane, int64_t x, Start start) {
  int lo = 0, width = n;                    // the answer lies in [lo, lo + width)
  while (width > 1) {
    const int step = (width + 31) / 32;
    int at = (lane + 1) * step;             // lane 31's probe is never inside
    bool before;
    if constexpr (kBad) {
      const int end = at + step < width ? at + step : width;
      int64_t s = at < width ? start(lo + at) : -1;
      while (s < 0 && ++at < end) s = start(lo + at);
      before = s >= 0 && s <= x;
    } else {
      before = at < width && start(lo + at) <= x;
    }
    const int passed = 32 - __clz(__ballot_sync(0xffffffffu, before));     // up to the last one
    lo += passed * step;
    width = width - passed * step < step ? width - passed * step : step;
  }
  return lo;
}

}  // namespace pmla
