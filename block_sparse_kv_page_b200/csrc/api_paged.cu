// C-ABI entry points of the paged cache: host-side argument validation and
// kernel launches (cache_io.cu, chunk_attn.cu, paged_decode.cu).
//
// Workspace: the layout of the other calls (api.cu): the status word at 0, the
// unit counters (not used here, left as they are), per-call scratch from
// kScratch on.
#include <cmath>
#include <cstdint>
#include <numeric>

#include "common.cuh"
#include "internal.h"
#include "paged.h"

namespace sa {

namespace {

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

// Scratch of the attention calls, from kScratch on.
struct PagedScratch {
  size_t parts, xbuf, recs, odd, total;
};
PagedScratch paged_scratch() {
  const size_t sms = (size_t)device_sm_count();
  PagedScratch s;
  s.parts = kScratch;
  s.xbuf = s.parts + align256(sms * 2 * 2 * kChunkPart * sizeof(float));
  s.recs = s.xbuf + align256(sms * kChunkPart * sizeof(float));
  s.odd = s.recs + align256(sms * sizeof(ChunkRec));
  s.total = s.odd + align256(sms * sizeof(ChunkOdd));
  // (the decode's parts and records, smaller, lie in the same place)
  return s;
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

sa_status launched(cudaError_t e) {
  if (e != cudaSuccess) {
    cudaGetLastError();
    return SA_ERR_CUDA;
  }
  return SA_OK;
}

sa_status check_paged(const sa_paged_desc* kv) {
  if (!kv) return SA_ERR_INVALID;
  if (kv->batch < 1 || kv->n_kv_heads < 1 || kv->max_pages < 1 || kv->n_pages < 1) return SA_ERR_INVALID;
  if (kv->dtype != SA_KV_BF16 && kv->dtype != SA_KV_E4M3) return SA_ERR_INVALID;
  if (kv->head_dim != kHeadDim) return SA_ERR_UNSUPPORTED;
  if (kv->page_size % 16 != 0 || kv->page_size < 16 || kv->page_size > 256) return SA_ERR_UNSUPPORTED;
  // (blocks of up to 64 tokens are counted, and ended, in 32 bits)
  if (kv->n_pages > 0x7fffffffLL || (long long)kv->max_pages * kv->page_size > 0x7fffff00LL)
    return SA_ERR_UNSUPPORTED;
  if (!kv->k || !kv->v || !aligned(kv->k, 16) || !aligned(kv->v, 16)) return SA_ERR_INVALID;
  const int64_t step = kv->dtype == SA_KV_E4M3 ? 16 : 8;  // elements of 16 bytes
  if (kv->token_stride < kHeadDim || kv->token_stride % step || kv->head_stride < kHeadDim ||
      kv->head_stride % step || kv->page_stride < kHeadDim || kv->page_stride % step)
    return SA_ERR_INVALID;
  // the tensor maps of the attention kernels take strides below 2^40 bytes
  const int64_t most = ((int64_t)1 << 40) / (kv->dtype == SA_KV_E4M3 ? 1 : 2);
  if (kv->token_stride >= most || kv->head_stride >= most || kv->page_stride >= most) return SA_ERR_UNSUPPORTED;
  if (kv->dtype == SA_KV_E4M3) {
    if (!kv->k_scale || !kv->v_scale || !aligned(kv->k_scale, 16) || !aligned(kv->v_scale, 16))
      return SA_ERR_INVALID;
  } else if (kv->k_scale || kv->v_scale) {
    return SA_ERR_INVALID;
  }
  if (!kv->page_table || !kv->seq_len || !aligned(kv->page_table, 4) || !aligned(kv->seq_len, 4))
    return SA_ERR_INVALID;
  return SA_OK;
}

PagedView paged_view(const sa_paged_desc* kv) {
  PagedView v{};
  const int bytes = kv->dtype == SA_KV_E4M3 ? 1 : 2;
  v.B = kv->batch;
  v.Hkv = kv->n_kv_heads;
  v.page_size = kv->page_size;
  v.max_pages = kv->max_pages;
  v.n_pages = kv->n_pages;
  v.e4m3 = kv->dtype == SA_KV_E4M3 ? 1 : 0;
  v.k = (unsigned char*)kv->k;
  v.v = (unsigned char*)kv->v;
  v.page_stride = kv->page_stride * bytes;
  v.head_stride = kv->head_stride * bytes;
  v.token_stride = kv->token_stride * bytes;
  v.k_scale = kv->k_scale;
  v.v_scale = kv->v_scale;
  v.table = kv->page_table;
  v.seq_len = kv->seq_len;
  return v;
}

// The status word of an optional workspace.
sa_status status_word(void* ws, size_t ws_bytes, int** status) {
  *status = nullptr;
  if (!ws) return SA_OK;
  if (!aligned(ws, 256) || ws_bytes < 256) return SA_ERR_WORKSPACE;
  *status = (int*)ws;
  return SA_OK;
}

sa_status check_heads(const sa_paged_desc* kv, int n_q_heads, int* G) {
  if (n_q_heads < 1 || n_q_heads % kv->n_kv_heads != 0) return SA_ERR_INVALID;
  *G = n_q_heads / kv->n_kv_heads;
  if (*G > kMaxGroup) return SA_ERR_UNSUPPORTED;
  return SA_OK;
}

// Tensor maps of the pool, [n_pages][Hkv][page_size][128], boxes of `rows` rows
// of 128 bytes (64 bf16 or 128 codes).
bool cache_maps(const PagedView& kv, CUtensorMap* k, CUtensorMap* v, int rows) {
  const unsigned long long d[4] = {kHeadDim, (unsigned long long)kv.page_size, (unsigned long long)kv.Hkv,
                                   (unsigned long long)kv.n_pages};
  const unsigned long long s[3] = {(unsigned long long)kv.token_stride, (unsigned long long)kv.head_stride,
                                   (unsigned long long)kv.page_stride};
  const unsigned b[4] = {kv.e4m3 ? 128u : 64u, (unsigned)rows, 1, 1};
  const CUtensorMapDataType dt = kv.e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
  // (rows of 128 codes, token by token: with 256-byte fetches L2 brought the
  // neighbouring head's row along, 1.5 times the bytes)
  return encode_tmap_nd(k, kv.k, dt, 4, d, s, b, true, !kv.e4m3) &&
         encode_tmap_nd(v, kv.v, dt, 4, d, s, b, true, !kv.e4m3);
}

sa_status decode(const PagedAttnArgs& p, unsigned char* ws, cudaStream_t st) {
  PagedDecodeArgs a{};
  const PagedView& kv = p.kv;
  a.p = p;
  a.scale_log2 = p.scale * kLog2e;
  a.scale_frac = std::frexp(a.scale_log2, &a.scale_exp);
  if (!cache_maps(kv, &a.tmap_k, &a.tmap_v, 16)) return SA_ERR_CUDA;
  const int grid = paged_decode_grid(device_sm_count());
  const long long units = (long long)kv.B * kv.Hkv;
  a.by_unit = units <= grid ? 1 : 0;
  const size_t part_bytes = align256((size_t)grid * paged_decode_part_floats() * sizeof(float));
  a.parts = (float*)(ws + kScratch);
  a.recs = (int4*)(ws + kScratch + part_bytes);
  if (kScratch + part_bytes + (size_t)grid * sizeof(int4) > paged_scratch().total) return SA_ERR_WORKSPACE;
  return launched(launch_paged_decode(a, grid, a.by_unit ? (int)units : grid, st));
}

sa_status chunk(const PagedAttnArgs& p, unsigned char* ws, cudaStream_t st) {
  ChunkArgs a{};
  const PagedView& kv = p.kv;
  const int blk = chunk_block_tokens();
  a.p = p;
  a.scale_log2 = p.scale * kLog2e;
  a.R = 128 / p.G;
  a.hb = std::gcd(kv.page_size, blk);
  const unsigned long long qd[3] = {kHeadDim, (unsigned long long)p.Hq, (unsigned long long)p.n_rows};
  const unsigned long long qs[2] = {kHeadDim * 2, (unsigned long long)p.q_row_stride * 2};
  const unsigned qb[3] = {64, (unsigned)p.G, (unsigned)a.R};
  if (!encode_tmap_nd(&a.tmap_q, p.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, qd, qs, qb, true, true)) return SA_ERR_CUDA;
  // bf16: halves of 64 dims, swizzled for the MMA; e4m3: whole rows of codes
  if (!cache_maps(kv, &a.tmap_k, &a.tmap_v, a.hb)) return SA_ERR_CUDA;
  const PagedScratch sc = paged_scratch();
  a.parts = (float*)(ws + sc.parts);
  a.xbuf = (float*)(ws + sc.xbuf);
  a.recs = (ChunkRec*)(ws + sc.recs);
  a.odd = (ChunkOdd*)(ws + sc.odd);
  return launched(launch_chunk(a, device_sm_count(), st));
}

sa_status paged_attention(const sa_paged_desc* kv, const void* q, int64_t q_row_stride, int n_q_heads,
                          const int32_t* row_off, int n_rows, int window, int sinks, float scale, void* out,
                          int out_dtype, float* lse, void* ws, size_t ws_bytes, void* stream) {
  PagedAttnArgs a{};
  sa_status s = check_paged(kv);
  if (s != SA_OK) return s;
  if ((s = check_heads(kv, n_q_heads, &a.G)) != SA_OK) return s;
  if (!q || !aligned(q, 16) || q_row_stride < (int64_t)n_q_heads * kHeadDim || q_row_stride % 8)
    return SA_ERR_INVALID;
  if (n_rows < 0 || window < 0 || sinks < 0 || !std::isfinite(scale * kLog2e)) return SA_ERR_INVALID;
  if (!out || !aligned(out, 16) || (lse && !aligned(lse, 4))) return SA_ERR_INVALID;
  if (out_dtype != SA_OUT_F32 && out_dtype != SA_OUT_BF16) return SA_ERR_INVALID;
  const size_t need = sparse_attn_paged_workspace_size(kv, n_q_heads);
  if (!ws || !aligned(ws, 256) || ws_bytes < need) return SA_ERR_WORKSPACE;
  if (n_rows == 0) return SA_OK;
  a.kv = paged_view(kv);
  a.q = (const __nv_bfloat16*)q;
  a.q_row_stride = q_row_stride;
  a.Hq = n_q_heads;
  a.row_off = row_off;
  a.n_rows = n_rows;
  a.window = window;
  a.sinks = sinks;
  a.scale = scale;
  if (out_dtype == SA_OUT_BF16) a.out_bf16 = (__nv_bfloat16*)out;
  else a.out = (float*)out;
  a.lse = lse;
  a.status = (int*)ws;
  // a window that no position passes is none (and keeps p - window in range)
  if ((long long)window > (long long)kv->max_pages * kv->page_size) a.window = 0;
  if (!row_off) return decode(a, (unsigned char*)ws, (cudaStream_t)stream);
  return chunk(a, (unsigned char*)ws, (cudaStream_t)stream);
}

}  // namespace
}  // namespace sa

using namespace sa;

extern "C" {

size_t sparse_attn_paged_workspace_size(const sa_paged_desc* kv, int32_t n_q_heads) {
  int G;
  if (check_paged(kv) != SA_OK || check_heads(kv, n_q_heads, &G) != SA_OK) return 0;
  return paged_scratch().total;
}

sa_status sparse_attn_cache_write(const sa_paged_desc* kv, const void* k_new, const void* v_new,
                                  int64_t row_stride, const int32_t* row_off, int32_t n_rows, void* ws,
                                  size_t ws_bytes, void* stream) {
  sa_status s = check_paged(kv);
  if (s != SA_OK) return s;
  CacheWriteArgs a{};
  if (!k_new || !v_new || !aligned(k_new, 16) || !aligned(v_new, 16)) return SA_ERR_INVALID;
  if (row_stride < (int64_t)kv->n_kv_heads * kHeadDim || row_stride % 8) return SA_ERR_INVALID;
  if (!row_off || !aligned(row_off, 4) || n_rows < 0) return SA_ERR_INVALID;
  if ((s = status_word(ws, ws_bytes, &a.status)) != SA_OK) return s;
  if (n_rows == 0) return SA_OK;
  if ((long long)n_rows * kv->n_kv_heads > 0x7fffffffLL) return SA_ERR_UNSUPPORTED;
  a.kv = paged_view(kv);
  a.k_new = (const __nv_bfloat16*)k_new;
  a.v_new = (const __nv_bfloat16*)v_new;
  a.row_stride = row_stride;
  a.row_off = row_off;
  a.n_rows = n_rows;
  return launched(launch_cache_write(a, (cudaStream_t)stream));
}

sa_status sparse_attn_cache_read(const sa_paged_desc* kv, int32_t first_token, void* k_out, void* v_out,
                                 int64_t cap_tokens, void* ws, size_t ws_bytes, void* stream) {
  sa_status s = check_paged(kv);
  if (s != SA_OK) return s;
  CacheReadArgs a{};
  if (!k_out || !v_out || !aligned(k_out, 16) || !aligned(v_out, 16) || cap_tokens < 1) return SA_ERR_INVALID;
  if ((s = status_word(ws, ws_bytes, &a.status)) != SA_OK) return s;
  // one item per (sequence, head, 16 tokens)
  if ((double)kv->batch * kv->n_kv_heads * kv->max_pages * (kv->page_size / 16) > 1073741823.0)
    return SA_ERR_UNSUPPORTED;
  a.kv = paged_view(kv);
  a.first_token = first_token;
  a.k_out = (__nv_bfloat16*)k_out;
  a.v_out = (__nv_bfloat16*)v_out;
  a.cap = cap_tokens;
  return launched(launch_cache_read(a, (cudaStream_t)stream));
}

sa_status sparse_attn_chunk(const sa_paged_desc* kv, const void* q, int64_t q_row_stride, int32_t n_q_heads,
                            const int32_t* row_off, int32_t n_rows, int32_t window, int32_t sinks, float scale,
                            void* out, int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (!row_off || !aligned(row_off, 4)) return SA_ERR_INVALID;
  return paged_attention(kv, q, q_row_stride, n_q_heads, row_off, n_rows, window, sinks, scale, out, out_dtype,
                         lse, ws, ws_bytes, stream);
}

sa_status sparse_attn_paged_decode(const sa_paged_desc* kv, const void* q, int64_t q_row_stride,
                                   int32_t n_q_heads, int32_t window, int32_t sinks, float scale, void* out,
                                   int32_t out_dtype, float* lse, void* ws, size_t ws_bytes, void* stream) {
  if (!kv) return SA_ERR_INVALID;
  return paged_attention(kv, q, q_row_stride, n_q_heads, nullptr, kv->batch, window, sinks, scale, out, out_dtype,
                         lse, ws, ws_bytes, stream);
}

}  // extern "C"
