// Attention over the paged cache, the plain kernel: one warp per (row, query
// head), lane l holding dims 4 l .. 4 l + 3, an online softmax over the tokens
// the row sees.
#include "paged.cuh"

namespace sa {
namespace {

constexpr int kWarpsPA = 8;

SA_DEV float4 load_row4(const PagedView& kv, const unsigned char* pool, const uint8_t* scale, int page, int head,
                        int slot, int lane) {
  const unsigned char* p = pool + paged_offset(kv, page, head, slot);
  if (kv.e4m3) {
    const uint32_t c = *reinterpret_cast<const uint32_t*>(p + 4 * lane);
    const float s = __uint_as_float((uint32_t)scale[scale_index(kv, page, head, slot)] << 23);
    const __half2_raw h0 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c & 0xffffu), __NV_E4M3);
    const __half2_raw h1 = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(c >> 16), __NV_E4M3);
    const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&h0));
    const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&h1));
    return make_float4(a.x * s, a.y * s, b.x * s, b.y * s);
  }
  const uint2 x = *reinterpret_cast<const uint2*>(p + 8 * lane);
  return make_float4(bf16_lo(x.x), bf16_hi(x.x), bf16_lo(x.y), bf16_hi(x.y));
}

__global__ void __launch_bounds__(32 * kWarpsPA) paged_attn_kernel(const __grid_constant__ PagedAttnArgs a) {
  const int lane = threadIdx.x & 31;
  const long long x = (long long)blockIdx.x * kWarpsPA + (threadIdx.x >> 5);
  if (x >= (long long)a.n_rows * a.Hq) return;
  const int row = (int)(x / a.Hq), h = (int)(x % a.Hq), g = h / a.G;
  const float ninf = -__int_as_float(0x7f800000);
  int b = row, r0 = row, m = 1;
  if (a.row_off) {
    int lo = 0, hi = a.kv.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(a.row_off + mid) <= row) lo = mid;
      else hi = mid;
    }
    b = lo;
    m = paged_rows(a.row_off, a.n_rows, b, r0, a.status);
    if (row < r0 || row >= r0 + m) return;
  }
  const int N = paged_tokens(a.kv, b, a.status);
  const int p = N - m + (row - r0);
  if (p < 0 && a.row_off) flag_status(a.status, SA_ERR_DEVICE_CHECK);
  const uint2 qx = *reinterpret_cast<const uint2*>(a.q + (size_t)row * a.q_row_stride + (size_t)h * kHeadDim + 4 * lane);
  const float4 q = make_float4(bf16_lo(qx.x), bf16_hi(qx.x), bf16_lo(qx.y), bf16_hi(qx.y));
  float mx = ninf, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  const int w0 = a.window ? max(0, p - a.window + 1) : 0;
  for (int t = 0; t <= p; ++t) {
    if (t < w0 && t >= a.sinks) t = w0;
    const int pg = t / a.kv.page_size;
    const int page = paged_page(a.kv, b, pg, a.status);
    if (page < 0) continue;
    const int slot = t - pg * a.kv.page_size;
    const float4 k = load_row4(a.kv, a.kv.k, a.kv.k_scale, page, g, slot, lane);
    float z = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) z += __shfl_xor_sync(0xffffffffu, z, s);
    z *= a.scale;
    const float nm = fmaxf(mx, z);
    const float f = expf(mx - nm), e = expf(z - nm);
    const float4 v = load_row4(a.kv, a.kv.v, a.kv.v_scale, page, g, slot, lane);
    l = l * f + e;
    o.x = o.x * f + e * v.x;
    o.y = o.y * f + e * v.y;
    o.z = o.z * f + e * v.z;
    o.w = o.w * f + e * v.w;
    mx = nm;
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  const size_t dst = ((size_t)row * a.Hq + h) * kHeadDim + 4 * lane;
  if (a.out_bf16)
    *reinterpret_cast<uint2*>(a.out_bf16 + dst) = make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  else
    *reinterpret_cast<float4*>(a.out + dst) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  if (a.lse && lane == 0) a.lse[(size_t)row * a.Hq + h] = l > 0.f ? mx + logf(l) : ninf;
}

}  // namespace

cudaError_t launch_paged_attn(const PagedAttnArgs& a, cudaStream_t st) {
  const long long blocks = ((long long)a.n_rows * a.Hq + kWarpsPA - 1) / kWarpsPA;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  paged_attn_kernel<<<(unsigned)blocks, 32 * kWarpsPA, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace sa
