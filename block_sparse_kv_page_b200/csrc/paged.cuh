// Device helpers of the paged cache: lengths, row ranges and e4m3 rows.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"
#include "paged.h"

namespace sa {

// Tokens of sequence b; 0 (flagged) for a length that the table cannot hold.
SA_DEV int paged_tokens(const PagedView& kv, int b, int* status) {
  const int N = __ldg(kv.seq_len + b);
  if (N < 0 || (long long)N > (long long)kv.max_pages * kv.page_size) {
    flag_status(status, SA_ERR_DEVICE_CHECK);
    return 0;
  }
  return N;
}

// New rows [r0, r0 + return value) of sequence b; none (flagged) for a range
// outside the row arrays.
SA_DEV int paged_rows(const int32_t* row_off, int n_rows, int b, int& r0, int* status) {
  r0 = __ldg(row_off + b);
  const int r1 = __ldg(row_off + b + 1);
  if (r0 < 0 || r1 < r0 || r1 > n_rows) {
    flag_status(status, SA_ERR_DEVICE_CHECK);
    return 0;
  }
  return r1 - r0;
}

// Pool page of table entry p of sequence b; -1 (flagged) if it is out of range.
SA_DEV int paged_page(const PagedView& kv, int b, int p, int* status) {
  const int page = __ldg(kv.table + (size_t)b * kv.max_pages + p);
  if (page < 0 || page >= kv.n_pages) {
    flag_status(status, SA_ERR_DEVICE_CHECK);
    return -1;
  }
  return page;
}

SA_DEV long long paged_offset(const PagedView& kv, int page, int head, int slot) {
  return (long long)page * kv.page_stride + (long long)head * kv.head_stride + (long long)slot * kv.token_stride;
}
SA_DEV size_t scale_index(const PagedView& kv, int page, int head, int slot) {
  return ((size_t)page * kv.Hkv + head) * kv.page_size + slot;
}

// The exponent of a row's scale: the smallest k with amax <= 448 * 2^k,
// 448 = 1.75 * 2^8, from amax's own exponent and mantissa (so no rounding can
// put it one off); clipped so that 2^k, 2^-k and every code * 2^k stay normal
// or exact in fp32 and bf16.
SA_DEV int e4m3_exponent(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127;
  const int k = e - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(-124, min(119, k));
}

}  // namespace sa
