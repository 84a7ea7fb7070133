// Writing new tokens into the paged cache (quantising them) and reading it
// back into one contiguous bf16 cache.
//
// Both only move rows of 128 values: a (token, head) pair is 512 bytes of
// bf16 K and V outside and 258 bytes inside an e4m3 cache (128 codes and one
// scale byte each), so HBM bounds them.  Measured: eight prompts of up to 32k
// tokens, 8 heads, written in 170 us (5.6 TB/s), read back in 183 us (5.5); a
// copy reaches 6.5.
#include "paged.cuh"
#include "internal.h"

namespace sa {
namespace {

constexpr int kWriteThreads = 256;

// Write: 16 lanes share a row and HG of its heads, 8 values of each K and V row
// per lane: every load of the heads is issued first, the maximum goes through
// four shuffles inside the half warp, the stores are 8 bytes (e4m3) or 16 a
// lane.  The row's place (its sequence, its page) is found once for the HG
// heads; with a head at a time, and 64-bit divisions, those instructions bound
// the kernel (219 us for eight prompts, 947 MB).
template <bool E4M3>
SA_DEV void write_row(const uint4 x, unsigned char* dst, uint8_t* scale, int l, bool ok) {
  if (!E4M3) {
    if (ok) *reinterpret_cast<uint4*>(dst + 16 * l) = x;
    return;
  }
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  // |bf16| compare as their bits do
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7fffu, (w[i] >> 16) & 0x7fffu));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int k = e4m3_exponent(__uint_as_float(m << 16));
  const float inv = __uint_as_float((uint32_t)(127 - k) << 23);  // 2^-k: the product is exact
  uint32_t c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(w[2 * i]) * inv, bf16_hi(w[2 * i]) * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(bf16_lo(w[2 * i + 1]) * inv, bf16_hi(w[2 * i + 1]) * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    c[i] = lo | (hi << 16);
  }
  if (ok) {
    *reinterpret_cast<uint2*>(dst + 8 * l) = make_uint2(c[0], c[1]);
    if (l == 0) *scale = (uint8_t)(k + 127);
  }
}

template <bool E4M3, int HG>
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const __grid_constant__ CacheWriteArgs a) {
  const int l = threadIdx.x & 15;
  const unsigned groups = (unsigned)a.kv.Hkv / HG;
  const unsigned x = blockIdx.x * (kWriteThreads / 16) + (threadIdx.x >> 4);  // (row, group of heads)
  const int row = (int)(x / groups), h0 = (int)(x - (unsigned)row * groups) * HG;
  const bool in = row < a.n_rows;
  uint4 kx[HG], vx[HG];
  const size_t src = (size_t)row * a.row_stride + (size_t)h0 * kHeadDim + 8 * l;
#pragma unroll
  for (int h = 0; h < HG; ++h) {
    kx[h] = in ? ldg_nc128(a.k_new + src + h * kHeadDim) : make_uint4(0u, 0u, 0u, 0u);
    vx[h] = in ? ldg_nc128(a.v_new + src + h * kHeadDim) : make_uint4(0u, 0u, 0u, 0u);
  }
  int page = -1, slot = 0;
  if (in) {
    // the row's sequence: the last b with row_off[b] <= row (empty ones skipped)
    int lo = 0, hi = a.kv.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.row_off + mid) <= row) lo = mid;
      else hi = mid;
    }
    int r0;
    const int m = paged_rows(a.row_off, a.n_rows, lo, r0, a.status);
    if (row >= r0 && row < r0 + m) {
      const int N = paged_tokens(a.kv, lo, a.status);
      const int t = N - m + (row - r0);
      if (t < 0) {
        flag_status(a.status, SA_ERR_DEVICE_CHECK);
      } else {
        const int p = t / a.kv.page_size;
        slot = t - p * a.kv.page_size;
        page = paged_page(a.kv, lo, p, a.status);
      }
    }
  }
  const bool ok = page >= 0;
  const long long off = paged_offset(a.kv, ok ? page : 0, h0, slot);
  const size_t at = scale_index(a.kv, ok ? page : 0, h0, slot);
#pragma unroll
  for (int h = 0; h < HG; ++h) {
    const long long o = off + h * a.kv.head_stride;
    const size_t s = at + (size_t)h * a.kv.page_size;
    write_row<E4M3>(kx[h], a.kv.k + o, a.kv.k_scale + s, l, ok);
    write_row<E4M3>(vx[h], a.kv.v + o, a.kv.v_scale + s, l, ok);
  }
}

constexpr int kReadThreads = 256;

SA_DEV uint32_t bf16_pair_of_codes(uint32_t two, float scale) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x * scale, f.y * scale);  // exact
}

// Read: a warp takes the K or the V of 16 tokens of one (sequence, head), 16
// lanes a row, so that every store instruction writes whole rows; its loads come
// first, all at once.
template <bool E4M3>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ CacheReadArgs a, unsigned tiles) {
  const int lane = threadIdx.x & 31, rl = lane >> 4, l = lane & 15;
  const unsigned warps = gridDim.x * (kReadThreads / 32);
  const unsigned heads = (unsigned)a.kv.Hkv;
  for (unsigned x = blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5); x < 2 * a.items; x += warps) {
    const unsigned it = x >> 1;
    const unsigned u = it / tiles, tile = it - u * tiles;
    const int b = (int)(u / heads), h = (int)(u - (unsigned)b * heads), t0 = (int)tile * 16;
    const int N = paged_tokens(a.kv, b, a.status);
    const int first = a.first_token >= 0 ? a.first_token : max(0, N + a.first_token);
    int e = min(N, t0 + 16);
    const int s = max(first, t0);
    if (s >= e) continue;
    if (e > a.cap) {
      flag_status(a.status, SA_ERR_DEVICE_CHECK);
      e = (int)a.cap;
      if (s >= e) continue;
    }
    const int p = t0 / a.kv.page_size;
    const int page = paged_page(a.kv, b, p, a.status);
    if (page < 0) continue;
    const int slot0 = t0 - p * a.kv.page_size;
    const unsigned char* src = ((x & 1) ? a.kv.v : a.kv.k) + paged_offset(a.kv, page, h, slot0) +
                               rl * a.kv.token_stride + (E4M3 ? 8 : 16) * l;
    const uint8_t* scale = E4M3 ? ((x & 1) ? a.kv.v_scale : a.kv.k_scale) + scale_index(a.kv, page, h, slot0) + rl : nullptr;
    __nv_bfloat16* dst = ((x & 1) ? a.v_out : a.k_out) + ((size_t)u * a.cap + (size_t)(t0 + rl)) * kHeadDim + 8 * l;
    uint4 v[8];
    uint32_t sc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {  // rows 2 i + rl
      const int t = t0 + 2 * i + rl;
      const bool in = t >= s && t < e;
      v[i] = make_uint4(0u, 0u, 0u, 0u);
      sc[i] = 0u;
      if (E4M3) {
        if (in) {
          const uint2 c = __ldg(reinterpret_cast<const uint2*>(src + 2 * i * a.kv.token_stride));
          v[i].x = c.x;
          v[i].y = c.y;
          sc[i] = __ldg(scale + 2 * i);
        }
      } else if (in) {
        v[i] = ldg_nc128(src + 2 * i * a.kv.token_stride);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int t = t0 + 2 * i + rl;
      if (t < s || t >= e) continue;
      if (E4M3) {
        const float f = __uint_as_float(sc[i] << 23);
        v[i] = make_uint4(bf16_pair_of_codes(v[i].x & 0xffffu, f), bf16_pair_of_codes(v[i].x >> 16, f),
                          bf16_pair_of_codes(v[i].y & 0xffffu, f), bf16_pair_of_codes(v[i].y >> 16, f));
      }
      *reinterpret_cast<uint4*>(dst + 2 * i * kHeadDim) = v[i];
    }
  }
}

template <bool E4M3>
cudaError_t launch_write(const CacheWriteArgs& a, cudaStream_t st) {
  const int hg = a.kv.Hkv % 4 == 0 ? 4 : (a.kv.Hkv % 2 == 0 ? 2 : 1);
  const long long threads = (long long)a.n_rows * (a.kv.Hkv / hg) * 16;
  const unsigned blocks = (unsigned)((threads + kWriteThreads - 1) / kWriteThreads);
  if (hg == 4) cache_write_kernel<E4M3, 4><<<blocks, kWriteThreads, 0, st>>>(a);
  else if (hg == 2) cache_write_kernel<E4M3, 2><<<blocks, kWriteThreads, 0, st>>>(a);
  else cache_write_kernel<E4M3, 1><<<blocks, kWriteThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t st) {
  return a.kv.e4m3 ? launch_write<true>(a, st) : launch_write<false>(a, st);
}

cudaError_t launch_cache_read(CacheReadArgs a, cudaStream_t st) {
  const long long tiles = (long long)a.kv.max_pages * a.kv.page_size / 16;
  const long long items = (long long)a.kv.B * a.kv.Hkv * tiles;
  if (items > 0x3fffffffLL) return cudaErrorInvalidValue;
  a.items = (unsigned)items;
  const long long per = kReadThreads / 32;
  long long blocks = (2 * items + per - 1) / per;
  const long long most = 16LL * device_sm_count();
  if (blocks > most) blocks = most;
  if (a.kv.e4m3) cache_read_kernel<true><<<(unsigned)blocks, kReadThreads, 0, st>>>(a, (unsigned)tiles);
  else cache_read_kernel<false><<<(unsigned)blocks, kReadThreads, 0, st>>>(a, (unsigned)tiles);
  return cudaGetLastError();
}

}  // namespace sa
