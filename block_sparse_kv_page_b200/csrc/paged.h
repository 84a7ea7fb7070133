// Internal interface of the paged-cache calls (api_paged.cu and the kernel
// files cache_io.cu, paged_decode.cu, chunk_attn.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "sparse_attn.h"

namespace sa {

// Plain copy of the paged cache's description, passed to kernels by value.
struct PagedView {
  int B, Hkv, page_size, max_pages;
  long long n_pages;
  int e4m3;
  unsigned char* k;            // bf16 or e4m3 elements
  unsigned char* v;
  long long page_stride, head_stride, token_stride;  // bytes
  uint8_t* k_scale;            // [n_pages][Hkv][page_size], e4m3 only
  uint8_t* v_scale;
  const int32_t* table;        // [B][max_pages]
  const int32_t* seq_len;
};

struct CacheWriteArgs {
  PagedView kv;
  const __nv_bfloat16* k_new;
  const __nv_bfloat16* v_new;
  long long row_stride;        // elements
  const int32_t* row_off;
  int n_rows;
  int* status;                 // nullable
};
cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t st);

struct CacheReadArgs {
  PagedView kv;
  int first_token;
  __nv_bfloat16* k_out;        // [B][Hkv][cap][128]
  __nv_bfloat16* v_out;
  long long cap;
  int* status;                 // nullable
};
cudaError_t launch_cache_read(const CacheReadArgs& a, cudaStream_t st);

struct PagedAttnArgs {
  PagedView kv;
  const __nv_bfloat16* q;
  long long q_row_stride;      // elements
  int Hq, G;
  const int32_t* row_off;      // null: row b is the one new row of sequence b
  int n_rows;
  int window, sinks;           // window 0 = everything up to the row
  float scale;
  float* out;                  // one of the two is set
  __nv_bfloat16* out_bf16;
  float* lse;                  // nullable
  int* status;
};
cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t st);

}  // namespace sa
