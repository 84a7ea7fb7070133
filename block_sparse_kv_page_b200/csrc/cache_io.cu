// Writing new tokens into the paged cache (quantising them) and reading it
// back into one contiguous bf16 cache.
//
// Both only move rows of 128 values: a (token, head) pair is 512 bytes of
// bf16 K and V outside and 258 bytes inside an e4m3 cache (128 codes and one
// scale byte each), so HBM bounds them.
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kWriteThreads = 256;

// Write: 16 lanes share one (row, head), 8 values of its K and of its V each:
// one 16-byte load per lane and row, the maximum by four shuffles inside the
// half warp, one 8-byte (e4m3) or 16-byte (bf16) store.
template <bool E4M3>
SA_DEV void write_row(const CacheWriteArgs& a, const uint4 x, unsigned char* pool, uint8_t* scale, long long off,
                      size_t at, int l) {
  if (!E4M3) {
    *reinterpret_cast<uint4*>(pool + off + 16 * l) = x;
    return;
  }
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float f[8], m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
    m = fmaxf(m, fmaxf(fabsf(f[2 * i]), fabsf(f[2 * i + 1])));
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const int k = e4m3_exponent(m);
  const float inv = __uint_as_float((uint32_t)(127 - k) << 23);  // 2^-k: the product is exact
  uint32_t c[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i] * inv, f[4 * i + 1] * inv), __NV_SATFINITE,
                                                 __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[4 * i + 2] * inv, f[4 * i + 3] * inv),
                                                 __NV_SATFINITE, __NV_E4M3);
    c[i] = lo | (hi << 16);
  }
  if (off >= 0) {
    *reinterpret_cast<uint2*>(pool + off + 8 * l) = make_uint2(c[0], c[1]);
    if (l == 0) scale[at] = (uint8_t)(k + 127);
  }
}

template <bool E4M3>
__global__ void __launch_bounds__(kWriteThreads) cache_write_kernel(const __grid_constant__ CacheWriteArgs a) {
  const int l = threadIdx.x & 15;
  const long long x = ((long long)blockIdx.x * kWriteThreads + threadIdx.x) >> 4;  // (row, head)
  const long long all = (long long)a.n_rows * a.kv.Hkv;
  const int Hkv = a.kv.Hkv;
  const int row = (int)(x / Hkv), h = (int)(x % Hkv);
  // the row's sequence: the last b with row_off[b] <= row (empty ones skipped)
  long long off = -1;
  size_t at = 0;
  uint4 kx = make_uint4(0u, 0u, 0u, 0u), vx = kx;
  if (x < all) {
    const size_t src = (size_t)row * a.row_stride + (size_t)h * kHeadDim + 8 * l;
    kx = ldg_nc128(a.k_new + src);
    vx = ldg_nc128(a.v_new + src);
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
        const int p = t / a.kv.page_size, slot = t - p * a.kv.page_size;
        const int page = paged_page(a.kv, lo, p, a.status);
        if (page >= 0) {
          off = paged_offset(a.kv, page, h, slot);
          at = scale_index(a.kv, page, h, slot);
        }
      }
    }
  }
  if (E4M3 || off >= 0) {
    write_row<E4M3>(a, kx, a.kv.k, a.kv.k_scale, off, at, l);
    write_row<E4M3>(a, vx, a.kv.v, a.kv.v_scale, off, at, l);
  }
}

constexpr int kReadThreads = 256;

SA_DEV uint32_t bf16_pair_of_codes(uint32_t two, float scale) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16(f.x * scale, f.y * scale);  // exact
}

// Read: a warp takes 16 tokens of one (sequence, head), 4 rows at a time.
template <bool E4M3>
__global__ void __launch_bounds__(kReadThreads) cache_read_kernel(const __grid_constant__ CacheReadArgs a, int tiles) {
  const int lane = threadIdx.x & 31;
  const long long warp = ((long long)blockIdx.x * kReadThreads + threadIdx.x) >> 5;
  const long long warps = (long long)gridDim.x * (kReadThreads / 32);
  const long long items = (long long)a.kv.B * a.kv.Hkv * tiles;
  for (long long it = warp; it < items; it += warps) {
    const int tile = (int)(it % tiles);
    const int u = (int)(it / tiles);
    const int b = u / a.kv.Hkv, h = u % a.kv.Hkv;
    const int N = paged_tokens(a.kv, b, a.status);
    const int t0 = a.first_token >= 0 ? a.first_token : max(0, N + a.first_token);
    int e = min(N, tile * 16 + 16);
    const int s = max(t0, tile * 16);
    if (s >= e) continue;
    if (e > a.cap) {
      flag_status(a.status, SA_ERR_DEVICE_CHECK);
      e = (int)a.cap;
      if (s >= e) continue;
    }
    const int p = tile * 16 / a.kv.page_size;
    const int page = paged_page(a.kv, b, p, a.status);
    if (page < 0) continue;
    const int slot0 = tile * 16 - p * a.kv.page_size;
    const long long off = paged_offset(a.kv, page, h, slot0);
    const size_t at = scale_index(a.kv, page, h, slot0);
    const size_t dst = ((size_t)u * a.cap + (size_t)tile * 16) * kHeadDim;
    const int r4 = lane >> 3, l = lane & 7;
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      const unsigned char* src = (kv ? a.kv.v : a.kv.k) + off;
      __nv_bfloat16* out = (kv ? a.v_out : a.k_out) + dst;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + r4;
        const int t = tile * 16 + r;
        if (t < s || t >= e) continue;
        uint4* o = reinterpret_cast<uint4*>(out + r * kHeadDim + 16 * l);
        if (E4M3) {
          const uint4 c = ldg_nc128(src + r * a.kv.token_stride + 16 * l);
          const float sc = __uint_as_float((uint32_t)__ldg((kv ? a.kv.v_scale : a.kv.k_scale) + at + r) << 23);
          o[0] = make_uint4(bf16_pair_of_codes(c.x & 0xffffu, sc), bf16_pair_of_codes(c.x >> 16, sc),
                            bf16_pair_of_codes(c.y & 0xffffu, sc), bf16_pair_of_codes(c.y >> 16, sc));
          o[1] = make_uint4(bf16_pair_of_codes(c.z & 0xffffu, sc), bf16_pair_of_codes(c.z >> 16, sc),
                            bf16_pair_of_codes(c.w & 0xffffu, sc), bf16_pair_of_codes(c.w >> 16, sc));
        } else {
          const unsigned char* r_src = src + r * a.kv.token_stride + 32 * l;
          o[0] = ldg_nc128(r_src);
          o[1] = ldg_nc128(r_src + 16);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteArgs& a, cudaStream_t st) {
  const long long threads = (long long)a.n_rows * a.kv.Hkv * 16;
  const long long blocks = (threads + kWriteThreads - 1) / kWriteThreads;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  if (a.kv.e4m3) cache_write_kernel<true><<<(unsigned)blocks, kWriteThreads, 0, st>>>(a);
  else cache_write_kernel<false><<<(unsigned)blocks, kWriteThreads, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_cache_read(const CacheReadArgs& a, cudaStream_t st) {
  const int tiles = (int)((long long)a.kv.max_pages * a.kv.page_size / 16);
  const long long items = (long long)a.kv.B * a.kv.Hkv * tiles;
  const long long per = kReadThreads / 32;
  long long blocks = (items + per - 1) / per;
  if (blocks > 148 * 16) blocks = 148 * 16;
  if (a.kv.e4m3) cache_read_kernel<true><<<(unsigned)blocks, kReadThreads, 0, st>>>(a, tiles);
  else cache_read_kernel<false><<<(unsigned)blocks, kReadThreads, 0, st>>>(a, tiles);
  return cudaGetLastError();
}

}  // namespace sa
