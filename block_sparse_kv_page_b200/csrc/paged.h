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
  unsigned items;              // (sequence, head, 16 tokens) triples
  int* status;                 // nullable
};
cudaError_t launch_cache_read(CacheReadArgs a, cudaStream_t st);

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

// Chunk attention (chunk_attn.cu).
// A partial result of 128 vectors: [32 groups of 4 dims][128 vectors][4], then
// [128][reference maximum, sum].
constexpr int kChunkMl = 128 * 128, kChunkPart = kChunkMl + 2 * 128;
struct ChunkRec {                    // a pair cut between CTAs, kept by the CTA that holds its first block
  int row0, rows, g, last, single;   // rows 0: none; last: the CTA that holds its last block
};
struct ChunkOdd {                    // sequences from .. to of which a CTA met results that are no numbers
  int from, to;                      // from > to: none
};
struct ChunkArgs {
  CUtensorMap tmap_q;                // [n_rows][Hq][128], box R x G x 64, 128B swizzle
  CUtensorMap tmap_k, tmap_v;        // [n_pages][Hkv][page_size][128], box 1 x 1 x hb x 64 (bf16, 128B
                                     // swizzle) or x 128 (codes)
  PagedAttnArgs p;
  float scale_log2;                  // scale * log2(e)
  int R;                             // rows of a tile, floor(128 / G)
  int hb;                            // rows of a K or V box: divides page_size and the block
  float* parts;                      // [grid][head, tail segment][slot][kChunkPart]
  float* xbuf;                       // [grid][kChunkPart]
  ChunkRec* recs;                    // [grid]
  ChunkOdd* odd;                     // [grid]
};
cudaError_t launch_chunk(const ChunkArgs& a, int grid, cudaStream_t st);
int chunk_block_tokens();
// Single-token attention (paged_decode.cu).
struct PagedDecodeArgs {
  CUtensorMap tmap_k, tmap_v;        // [n_pages][Hkv][page_size][128], box 1 x 1 x 16 x 128 bytes, 128B swizzle
  PagedAttnArgs p;                   // row b of sequence b
  float scale_log2;                  // scale * log2(e) = scale_frac * 2^scale_exp, |scale_frac| < 1
  float scale_frac;
  int scale_exp;
  int by_unit;                       // recs by unit (b * Hkv + g) instead of by CTA
  float* parts;                      // [grid][head, tail segment][8 heads][132]
  int4* recs;                        // cut units: first CTA (-1: none), last CTA, b, g
};
int paged_decode_grid(int sms);
size_t paged_decode_part_floats();   // per CTA
// recs: entries of a.recs, the smaller of units and grid
cudaError_t launch_paged_decode(const PagedDecodeArgs& a, int grid, int recs, cudaStream_t st);

}  // namespace sa
