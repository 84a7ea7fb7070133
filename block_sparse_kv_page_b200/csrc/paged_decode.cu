// Single-token attention over the paged cache: one row per sequence.
//
// Mathematics: the newest row of sequence b, position N - 1, query head h of KV
// head g: out = sum exp(z_t - lse) v_t over the visible tokens, z_t = scale
// q . k_t, in one pass with a running maximum and sum.  Every visible token's K
// and V are read once for the G <= 8 heads that share them; that read bounds it.
// Measured: 32 sequences of up to 32k tokens, 8 KV heads, e4m3: 228 us, 5.0
// TB/s; one of 29.5k tokens, 4 KV heads, bf16: 21 us, where the read itself
// takes 9.4 and the rest is latency (lengths, table, first tiles, merge).
//
// Units are (sequence, KV head) pairs, cut into tiles of 16 tokens (those of
// the first tokens and of the window; a page is whole tiles).  The work is the
// list of all units' tiles; the grid takes equal runs of it (each unit counting
// kC0 tiles more, the cost of starting one), cut anywhere, so that one long
// sequence fills every SM and ragged batches stay balanced.  The prefix is
// computed from the lengths on the device by every CTA.  A unit cut between
// CTAs leaves unnormalised parts in the workspace, merged by
// decode_combine_kernel in CTA order: results do not depend on scheduling.
//
// Inside a CTA the four warps take tiles in turn, each with a ring of its own:
// TMA boxes of 16 rows, 128B-swizzled, three CTAs and 192 KiB of rings per SM.
// Per tile (tensor cores, fp32 accumulation):
//   S^T [16 tokens x 8 heads] = K Q^T;
//   P: exp2 of the scaled scores in fp32, as two bf16 terms (three for fp32
//      outputs: 2^-16 and 2^-24 of a weight), moved to the B layout;
//   O^T [128 dims x 8 heads] += V^T P^T.
// e4m3: codes become fragments in registers.  The order of the reduction
// axis is free as long as both operands share it, so a lane takes whole 16-byte
// pieces of a row: 32 dims of two tokens for K, 16 dims of four tokens for V,
// free of bank conflicts under the swizzle.  Codes become f16, one conversion per
// pair: q is scaled per head to fit, and weights times V's scales are taken
// relative to the largest scale seen, which is followed like the maximum; tiles
// with a weight below what f16 holds take the same products in bf16 (whose
// conversion, by shifts and masks, costs three times as much: 16 sequences of
// 32k tokens 187 us, 223 where every tile takes it).  The rows' scales (powers of two)
// multiply the scores and the weights, 4 values a lane instead of 256.
#include <cuda_fp16.h>

#include <type_traits>

#include "paged.cuh"
#include "internal.h"

namespace sa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kC0 = 6;          // cost of starting a unit, in tiles
// Least work of a CTA: small calls are a chain of latencies, so they are spread
// as far as a start's cost allows (1 sequence of 2k tokens, 4 KV heads, in a
// graph: 7.7 us; shares of 10, 14, 18 and 24: 9.0, 9.9, 11.1, 12.3).
constexpr int kMinShare = kC0;
constexpr int kPart = kHeadDim + 4;          // floats of a head's part: acc, maximum, sum, 2 unused
constexpr int kMergeBytes = kWarps * kMaxGroup * (kHeadDim + 2) * 4;

template <bool E4M3>
struct Ring {
  static constexpr int kBox = 2048;                  // 16 rows x 128 B
  static constexpr int kSub = E4M3 ? 2 : 1;           // tiles of 16 tokens per ring stage
  static constexpr int kTile = kSub * (E4M3 ? 2 : 4) * kBox;
  static constexpr int kStages = 2;
  static constexpr int kRing = kWarps * kStages * kTile;
  static constexpr int kOffScale = kRing;            // [warp][stage][tile][K 16 | V 16]
  static constexpr int kOffBars = kOffScale + (E4M3 ? kWarps * kStages * kSub * 32 : 0);
  static constexpr int kSmem = 1024 + kOffBars + kWarps * kStages * 8;
  static_assert(kMergeBytes <= kRing, "the warps' results are merged in the ring");
};

SA_DEV float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}
SA_DEV uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// The codes in the high / low bytes of both halves of x as a bf16 pair: a
// code's 7 low bits are the exponent and mantissa of a bf16 2^120 times
// smaller, subnormals included.
constexpr uint32_t kTwo120 = 0x7b807b80u;  // (2^120, 2^120)
SA_DEV uint32_t bf16_high_codes(uint32_t x) {
  return mul_bf16x2((x & 0x80008000u) | ((x >> 4) & 0x07f007f0u), kTwo120);
}
// Two codes (the low or the high half of x) as an f16 pair: exact.
SA_DEV uint32_t f16_of_codes(uint32_t x, bool high) {
  uint32_t r;
  if (high)
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, hi;\n}\n" : "=r"(r) : "r"(x));
  else
    asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %1;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n}\n" : "=r"(r) : "r"(x));
  return r;
}
SA_DEV void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
SA_DEV uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
SA_DEV uint32_t bf16_low_codes(uint32_t x) {
  return mul_bf16x2(((x << 8) & 0x80008000u) | ((x << 4) & 0x07f007f0u), kTwo120);
}

// Tiles of a unit: tokens [0, S) and [lo, N).
struct Unit {
  int N, lo, S, st, wt0, nt;
};
SA_DEV Unit unit_of(const PagedDecodeArgs& a, int tokens) {
  Unit u;
  u.N = tokens;
  u.lo = a.p.window && u.N > a.p.window ? u.N - a.p.window : 0;
  u.S = a.p.window ? min(a.p.sinks, u.N) : 0;
  u.wt0 = u.lo >> 4;
  u.st = min((u.S + 15) >> 4, u.wt0);
  u.nt = u.st + ((u.N + 15) >> 4) - u.wt0;
  return u;
}

template <bool E4M3, int TERMS>
__global__ void __launch_bounds__(kThreads, 3) paged_decode_kernel(const __grid_constant__ PagedDecodeArgs a) {
  using R = Ring<E4M3>;
  extern __shared__ unsigned char smem_raw[];
  __shared__ long long s_scan[kWarps];
  __shared__ long long s_plan[3];  // work in the first sequence before this CTA's, its index, its tokens
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = lane >> 2, c = lane & 3;
  const PagedView& kv = a.p.kv;
  const int Hkv = kv.Hkv, G = a.p.G, B = kv.B;
  const float ninf = -__int_as_float(0x7f800000);
  int* status = a.p.status;
  uint64_t* bars = reinterpret_cast<uint64_t*>(base + R::kOffBars) + warp * R::kStages;
  unsigned char* ring = base + warp * (R::kStages * R::kTile);
  unsigned char* scales = base + R::kOffScale + warp * (R::kStages * R::kSub * 32);
  constexpr int SUB = R::kSub;
  // Weights, at most 1 in the units of the largest V scale, are multiplied by
  // 2^kUp, so that f16 holds 2^-14 .. 2^15 of them as normal numbers.  A tile with a weight that is
  // not zero but under kLeast takes the bf16 products, whose range is fp32's:
  // 2^-14 leaves one f16 term its 2^-11 of a weight (bf16 outputs), 2^-6 two
  // terms 2^-19 (the second is rounded to 2^-25).
  constexpr int kUp = 15;
  constexpr float kLeast = TERMS == 3 ? 0x1p-6f : 0x1p-14f;
  if (lane == 0) {
    for (int s = 0; s < R::kStages; ++s) mbar_init(bars + s, 1);
    fence_barrier_init();
  }
  if (tid == 0) {
    prefetch_tmap(&a.tmap_k);
    prefetch_tmap(&a.tmap_v);
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_trigger();  // decode_combine_kernel may be scheduled; it waits for this grid's end

  // ---- this CTA's run of the work
  auto prefix = [&](long long v, long long& total) -> long long {
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += s_scan[w];
      all += s_scan[w];
    }
    __syncthreads();
    total = all;
    return before + x - v;
  };
  int tokens = 0;  // of the sequence last asked for
  auto seq_work = [&](int b) -> long long {
    if (b >= B) return 0;
    tokens = paged_tokens(kv, b, status);
    return (long long)Hkv * (unit_of(a, tokens).nt + kC0);
  };
  long long total = 0, w = 0, ex = 0;
  for (int b0 = 0; b0 < B; b0 += kThreads) {
    long long t;
    w = seq_work(b0 + tid);
    ex = prefix(w, t) + total;
    total += t;
  }
  // as many CTAs as have kMinShare each; the first `more` of them take one tile more than `each`
  const int nc = total >= (long long)gridDim.x * kMinShare ? (int)gridDim.x : max(1, (int)total / kMinShare);
  const long long each = total >> 31 ? total / nc : (int)total / nc;
  const int more = (int)(total - each * nc);
  if ((int)blockIdx.x >= nc) {
    if (!a.by_unit && tid == 0) a.recs[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  const long long w0 = each * blockIdx.x + min((int)blockIdx.x, more);
  const long long w1 = w0 + each + ((int)blockIdx.x < more ? 1 : 0);
  {
    long long run = 0;
    for (int b0 = 0; b0 < B; b0 += kThreads) {
      if (B > kThreads) {
        long long t;
        w = seq_work(b0 + tid);
        ex = prefix(w, t) + run;
        run += t;
      }
      if (w && ex <= w0 && w0 < ex + w) {
        s_plan[0] = w0 - ex;
        s_plan[1] = b0 + tid;
        s_plan[2] = tokens;
      }
    }
  }
  __syncthreads();
  int b = (int)s_plan[1];
  Unit u = unit_of(a, (int)s_plan[2]);
  const long long in = s_plan[0];  // into the sequence's work
  int g = in >> 31 ? (int)(in / (u.nt + kC0)) : (int)in / (u.nt + kC0);
  int off = (int)(in - (long long)g * (u.nt + kC0));
  long long rem = w1 - w0, at = w0 - off;  // at: where the unit's work begins
  if (!a.by_unit && tid == 0) a.recs[blockIdx.x] = make_int4(-1, 0, 0, 0);

  uint32_t gi = 0;  // ring position of this warp
  bool alive = true;
  while (rem > 0) {
    const int cost = u.nt + kC0;
    const int take = (int)min(rem, (long long)(cost - off));
    const int i0 = min(max(off - kC0, 0), u.nt), i1 = min(max(off + take - kC0, 0), u.nt);
    const bool begins = i0 == 0 && (i1 > 0 || (u.nt == 0 && off == 0));
    if (i1 > i0 || begins) {
      // ---- this warp's tiles, SUB at a time: i0 + SUB (warp + 4 it) + u of
      // iteration it; lane k keeps the pages of its tiles 32 j + k (in that
      // order), the next 32 looked up while these are used;
      // asked for ahead of Q, so that the two latencies overlap
      const int nt = i1 - i0;
      const int n_it = max(0, ((nt + SUB - 1) / SUB - warp + kWarps - 1) / kWarps);
      auto tile_of = [&](int x) { return SUB * (warp + kWarps * (x / SUB)) + x % SUB; };  // in [i0, i1): < nt
      auto start_of = [&](int i) { return 16 * (i0 + i < u.st ? i0 + i : u.wt0 + i0 + i - u.st); };
      const int n_pages = (int)kv.n_pages;
      auto look = [&](int x, int& page, int& slot) {
        page = -2;  // no such tile
        slot = 0;
        const int i = tile_of(x);
        if (i < nt) {
          const int t = start_of(i), e = t / kv.page_size;
          slot = t - e * kv.page_size;
          page = __ldg(kv.table + (size_t)b * kv.max_pages + e);
          if (page == -2) page = -1;
        }
      };
      int pages, pages1, slots, slots1;
      look(lane, pages, slots);
      look(32 + lane, pages1, slots1);

      // ---- Q fragments (B operand) in the order of the reduction axis that the K fragments have
      const bool head_ok = gq < G;
      const __nv_bfloat16* qrow =
          a.p.q + (size_t)b * a.p.q_row_stride + (size_t)(g * G + (head_ok ? gq : 0)) * kHeadDim;
      uint32_t bq[16];
      int q_exp = 0;      // of head gq: its values are q * 2^-q_exp here
      bool wide = false;  // f16 does not hold some head's values
      if (E4M3) {
        // f16, as the codes become: each head's values times the power of two
        // that brings the largest below 2^14.  Step s: dims 32 c + 4 s + {0, 1}
        // and {2, 3}.  f16 holds all but those under 2^-31 of the largest; where
        // it does not hold one exactly, keys and queries go to bf16, the largest
        // brought below 2^111 (sums stay below 2^127), in the order {0, 2}, {1, 3}.
        uint4 x[4];
        uint32_t top = 0u, low = 0xffffffffu;  // of two values each: the largest |q|, the smallest but 0, as bits
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          x[s] = head_ok ? ldg_nc128(qrow + 32 * c + 8 * s) : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t y[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            top = __vmaxu2(top, y[i] & 0x7fff7fffu);
            low = __vminu2(low, __vsub2(y[i] & 0x7fff7fffu, 0x00010001u));  // (less one: 0 becomes the largest)
          }
        }
        int mq = max(top & 0xffffu, top >> 16);
        mq = max(mq, __shfl_xor_sync(0xffffffffu, mq, 1));
        mq = max(mq, __shfl_xor_sync(0xffffffffu, mq, 2));
        const int e = min(253, max(1, 127 + 13 - ((mq >> 7) - 127)));
        const float up = __uint_as_float((uint32_t)e << 23);
        q_exp = 127 - e;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const uint32_t y[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) bq[4 * s + i] = pack_f16(bf16_lo(y[i]) * up, bf16_hi(y[i]) * up);
        }
        // 8 bits of a value from 2^-17 on reach f16's last place, 2^-24
        const bool exact = (int)min(low & 0xffffu, low >> 16) >= ((127 - 17 + 127 - e) << 7) - 1;
        wide = __any_sync(0xffffffffu, !exact);
        if (wide) {
          const int ew = min(253, max(1, 127 + 110 - ((mq >> 7) - 127)));
          const float upw = __uint_as_float((uint32_t)ew << 23);
          q_exp = 127 - ew;
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const uint32_t y[4] = {x[s].x, x[s].y, x[s].z, x[s].w};
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              bq[4 * s + i] = pack_bf16(bf16_lo(y[i]) * upw, bf16_lo(y[i + 1]) * upw);
              bq[4 * s + i + 1] = pack_bf16(bf16_hi(y[i]) * upw, bf16_hi(y[i + 1]) * upw);
            }
          }
        }
      }
      // Sums of heads 2 c, 2 c + 1 times zs, times the row's scale (e4m3), times
      // zu are scores.  A sum is below 2^30 in e4m3 (2^127 if wide), so with zs
      // within 2^-60 .. 2^90 (2^-120 .. 1) no product on the way overflows, or loses bits, where the score
      // does not; what scale and 2^q_exp leave for zu is 1 but for queries or
      // scales near the ends of fp32.  (Above 2^127, both past 2^100, it is
      // capped: only lse shows it, scores are 2^60 apart there.)
      float zs0 = a.scale_log2, zs1 = a.scale_log2, zu0 = 1.f, zu1 = 1.f;
      if (E4M3) {
        auto split = [&](int q, float& zs, float& zu) {
          const int e = a.scale_exp + q, in = min(max(e, wide ? -120 : -60), wide ? 0 : 90);
          zs = a.scale_frac * __uint_as_float((uint32_t)(127 + in) << 23);
          zu = __uint_as_float((uint32_t)(127 + min(max(e - in, -126), 127)) << 23);
        };
        split(__shfl_sync(0xffffffffu, q_exp, 8 * c), zs0, zu0);
        split(__shfl_sync(0xffffffffu, q_exp, 8 * c + 4), zs1, zu1);
      }
      if (!E4M3) {  // step s: dims 16 s + 2 c (+ 1), 16 s + 8 + 2 c (+ 1)
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          bq[2 * s] = head_ok ? __ldg(reinterpret_cast<const uint32_t*>(qrow + 16 * s + 2 * c)) : 0u;
          bq[2 * s + 1] = head_ok ? __ldg(reinterpret_cast<const uint32_t*>(qrow + 16 * s + 8 + 2 * c)) : 0u;
        }
      }
      float m0 = ninf, m1 = ninf, l0 = 0.f, l1 = 0.f;
      float acc[8][4];
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
      // e4m3: acc is held in units of 2^(e_acc - 127 - kUp), e_acc the largest V
      // scale byte of a visible token so far: weight * scale is at most 2^kUp
      int e_acc = -1000;

      auto page_of = [&](int x, int j) { return __shfl_sync(0xffffffffu, (x >> 5) == j ? pages : pages1, x & 31); };
      auto issue = [&](int it, int j) {  // every lane; a few of them copy
        const uint32_t s = (gi + (uint32_t)it) % R::kStages;
        unsigned char* st = ring + s * R::kTile;
        const int x0 = it * SUB;
        int page[SUB], slot[SUB], good = 0;
#pragma unroll
        for (int y = 0; y < SUB; ++y) {
          page[y] = page_of(x0 + y, j);
          slot[y] = __shfl_sync(0xffffffffu, ((x0 + y) >> 5) == j ? slots : slots1, (x0 + y) & 31);
          if ((unsigned)page[y] < (unsigned)n_pages) ++good;
          else if (page[y] != -2 && lane == 0) flag_status(status, SA_ERR_DEVICE_CHECK);
        }
        if (lane == 0) {
          if (good) mbar_arrive_expect_tx(bars + s, good * (R::kTile / SUB + (E4M3 ? 32 : 0)));
          else mbar_arrive(bars + s);  // nothing to load: complete the phase
        }
        __syncwarp();
        const int y = SUB == 1 ? 0 : lane >> 2, l = lane & 3;
        if (lane < 4 * SUB) {
          const int pg = y ? page[SUB - 1] : page[0], sl = y ? slot[SUB - 1] : slot[0];
          if ((unsigned)pg < (unsigned)n_pages) {
            unsigned char* dst = st + y * (R::kTile / SUB);
            if (E4M3) {
              if (l < 2)
                tma_load_4d(dst + l * R::kBox, l ? &a.tmap_v : &a.tmap_k, 0, sl, g, pg, bars + s);
              else
                bulk_load(scales + (s * SUB + y) * 32 + 16 * (l & 1),
                          ((l & 1) ? kv.v_scale : kv.k_scale) + scale_index(kv, pg, g, sl), 16, bars + s);
            } else {
              tma_load_4d(dst + l * R::kBox, l < 2 ? &a.tmap_k : &a.tmap_v, 64 * (l & 1), sl, g, pg, bars + s);
            }
          }
        }
      };
      int issued = 0;
      if (alive)
        for (; issued < min(n_it, R::kStages - 1); ++issued) issue(issued, 0);
      // ldmatrix lane addressing (bf16): matrix = lane / 8, row in matrix = lane % 8
      const int lrow_a = (lane & 7) + 8 * ((lane >> 3) & 1), lchk_a = lane >> 4;
      const int lrow_v = (lane & 7) + 8 * (lane >> 4), lchk_v = (lane >> 3) & 1;
      for (int it = 0; it < n_it && alive; ++it) {
        const int j = (it * SUB) >> 5;
        __syncwarp();  // every lane is done with the stage about to be refilled
        if (issued < n_it) {
          issue(issued, j);
          ++issued;
        }
        const uint32_t s_it = (gi + (uint32_t)it) % R::kStages;
        if (!__all_sync(0xffffffffu, mbar_wait(bars + s_it, ((gi + (uint32_t)it) / R::kStages) & 1u, status))) {
          alive = false;
          break;
        }
        bool good[SUB], edge[SUB], v0[SUB], v1[SUB];
        float z[SUB][4];
        int ea[SUB], eb[SUB];  // V scale bytes of this lane's tokens
        float mx0 = ninf, mx1 = ninf;
#pragma unroll
        for (int y = 0; y < SUB; ++y) {
          good[y] = (unsigned)page_of(it * SUB + y, j) < (unsigned)n_pages;
          unsigned char* st = ring + s_it * R::kTile + y * (R::kTile / SUB);
          // visible tokens of the tile: all of them but in the first and last tiles
          const int t0 = start_of(SUB * (warp + kWarps * it) + y);
          v0[y] = v1[y] = good[y];
          edge[y] = good[y] && (t0 + 16 > u.N || (t0 < u.lo && t0 + 16 > u.S));
          if (edge[y]) {
            const int ta = t0 + gq, tb = ta + 8;
            v0[y] = ta < u.N && (ta < u.S || ta >= u.lo);
            v1[y] = tb < u.N && (tb < u.S || tb >= u.lo);
            if (!E4M3) {  // V rows of other tokens may hold anything: zeros before they meet a weight of 0
              for (int x = lane; x < 256; x += 32) {
                const int row = x >> 4, ch = x & 15, t = t0 + row;
                if (!(t < u.N && (t < u.S || t >= u.lo)))
                  *reinterpret_cast<uint4*>(st + (2 + (ch >> 3)) * R::kBox + swz128(row, ch & 7)) =
                      make_uint4(0u, 0u, 0u, 0u);
              }
              fence_proxy_async();
              __syncwarp();
            }
          }
        }
        // ---- S^T = K Q^T, two chains a tile (a tile that was not loaded gives junk, which nothing sees)
        float s[SUB][4], s2[SUB][4];
#pragma unroll
        for (int y = 0; y < SUB; ++y)
#pragma unroll
          for (int x = 0; x < 4; ++x) s[y][x] = s2[y][x] = 0.f;
        if (E4M3) {
          auto products = [&](auto f16) {
#pragma unroll
            for (int y = 0; y < SUB; ++y) {
              const unsigned char* st = ring + s_it * R::kTile + y * (R::kTile / SUB);
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const uint4 xk = lds128(st + swz128(gq, 2 * c + h)), yk = lds128(st + swz128(gq + 8, 2 * c + h));
                const uint32_t xs[4] = {xk.x, xk.y, xk.z, xk.w}, ys[4] = {yk.x, yk.y, yk.z, yk.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const int k = 4 * h + i;
                  if (f16)
                    mma_f16(i & 1 ? s2[y] : s[y], f16_of_codes(xs[i], false), f16_of_codes(ys[i], false),
                            f16_of_codes(xs[i], true), f16_of_codes(ys[i], true), bq[2 * k], bq[2 * k + 1]);
                  else
                    mma_bf16(i & 1 ? s2[y] : s[y], bf16_low_codes(xs[i]), bf16_low_codes(ys[i]),
                             bf16_high_codes(xs[i]), bf16_high_codes(ys[i]), bq[2 * k], bq[2 * k + 1]);
                }
              }
            }
          };
          products(std::true_type{});
          if (wide) {  // (again: a choice between the two, ahead of them, cost the usual path 2%)
#pragma unroll
            for (int y = 0; y < SUB; ++y)
#pragma unroll
              for (int x = 0; x < 4; ++x) s[y][x] = s2[y][x] = 0.f;
            products(std::false_type{});
          }
        } else {
#pragma unroll
          for (int y = 0; y < SUB; ++y) {
            const unsigned char* st = ring + s_it * R::kTile + y * (R::kTile / SUB);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t a0, a1, a2, a3;
              ldsm_x4(a0, a1, a2, a3, st + (k >> 2) * R::kBox + swz128(lrow_a, 2 * (k & 3) + lchk_a));
              mma_bf16(k & 1 ? s2[y] : s[y], a0, a1, a2, a3, bq[2 * k], bq[2 * k + 1]);
            }
          }
        }
#pragma unroll
        for (int y = 0; y < SUB; ++y) {
          float ka = 1.f, kb = 1.f;  // the tokens' scales
          if (E4M3) {
            const unsigned char* sc = scales + (s_it * SUB + y) * 32;
            ka = __uint_as_float((uint32_t)sc[gq] << 23);
            kb = __uint_as_float((uint32_t)sc[gq + 8] << 23);
            ea[y] = sc[16 + gq];
            eb[y] = sc[16 + gq + 8];
          }
          // tokens gq / gq + 8, heads 2 c / 2 c + 1
          z[y][0] = v0[y] ? (s[y][0] + s2[y][0]) * zs0 * ka : ninf;
          z[y][1] = v0[y] ? (s[y][1] + s2[y][1]) * zs1 * ka : ninf;
          z[y][2] = v1[y] ? (s[y][2] + s2[y][2]) * zs0 * kb : ninf;
          z[y][3] = v1[y] ? (s[y][3] + s2[y][3]) * zs1 * kb : ninf;
          mx0 = fmaxf(mx0, fmaxf(z[y][0], z[y][2]));
          mx1 = fmaxf(mx1, fmaxf(z[y][1], z[y][3]));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, o));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, o));
        }
        if (E4M3) {
          mx0 *= zu0;
          mx1 *= zu1;
        }
        const float mn0 = fmaxf(m0, mx0), mn1 = fmaxf(m1, mx1);
        if (__any_sync(0xffffffffu, mn0 > m0 || mn1 > m1)) {
          const float al0 = mn0 == ninf ? 1.f : fast_exp2(m0 - mn0), al1 = mn1 == ninf ? 1.f : fast_exp2(m1 - mn1);
          m0 = mn0;
          m1 = mn1;
          l0 *= al0;
          l1 *= al1;
#pragma unroll
          for (int mt = 0; mt < 8; ++mt) {
            acc[mt][0] *= al0;
            acc[mt][1] *= al1;
            acc[mt][2] *= al0;
            acc[mt][3] *= al1;
          }
        }
        const float r0 = m0 == ninf ? 0.f : -m0, r1 = m1 == ninf ? 0.f : -m1;  // nothing seen: exp2(-inf) = 0
        if (E4M3) {
          int hi = -1000;
#pragma unroll
          for (int y = 0; y < SUB; ++y) hi = max(hi, max(v0[y] ? ea[y] : -1000, v1[y] ? eb[y] : -1000));
          hi = __reduce_max_sync(0xffffffffu, hi);
          if (hi > e_acc) {
            const float f = e_acc < hi - 126 ? 0.f : __uint_as_float((uint32_t)(127 + e_acc - hi) << 23);
            e_acc = hi;
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              acc[mt][0] *= f;
              acc[mt][1] *= f;
              acc[mt][2] *= f;
              acc[mt][3] *= f;
            }
          }
        }
#pragma unroll
        for (int y = 0; y < SUB; ++y) {
          if (!good[y]) continue;
          unsigned char* st = ring + s_it * R::kTile + y * (R::kTile / SUB);
          float p0 = fast_exp2(fmaf(z[y][0], zu0, r0)), p1 = fast_exp2(fmaf(z[y][1], zu1, r1));
          float p2 = fast_exp2(fmaf(z[y][2], zu0, r0)), p3 = fast_exp2(fmaf(z[y][3], zu1, r1));
          l0 += p0 + p2;
          l1 += p1 + p3;
          bool f16_holds = false;  // f16 holds every weight of the tile
          if (E4M3) {  // times 2^(scale - e_acc + kUp); a scale byte of a hidden token may be anything
            const float fa = v0[y] ? __uint_as_float((uint32_t)max(0, 127 + kUp + ea[y] - e_acc) << 23) : 0.f;
            const float fb = v1[y] ? __uint_as_float((uint32_t)max(0, 127 + kUp + eb[y] - e_acc) << 23) : 0.f;
            p0 *= fa;
            p1 *= fa;
            p2 *= fb;
            p3 *= fb;
            // (less one: a zero becomes the largest word; weights compare as their bits do)
            const uint32_t least = min(min(__float_as_uint(p0) - 1u, __float_as_uint(p1) - 1u),
                                       min(__float_as_uint(p2) - 1u, __float_as_uint(p3) - 1u));
            f16_holds = !__any_sync(0xffffffffu, least < __float_as_uint(kLeast) - 1u);
          }
          if (E4M3 && f16_holds && !edge[y]) {
            // Weights and codes in f16.  fp32 outputs: two terms, 2^-19 of a
            // weight and less; bf16 outputs: one, 2^-11 (the output's own
            // rounding is 2^-8).
            constexpr int FT = TERMS == 3 ? 2 : 1;
            uint32_t bt0[FT], bt1[FT];
#pragma unroll
            for (int x = 0; x < FT; ++x) {
              const __half2 lo = __floats2half2_rn(p0, p1), hi = __floats2half2_rn(p2, p3);
              if (x + 1 < FT) {
                p0 -= __low2float(lo);
                p1 -= __high2float(lo);
                p2 -= __low2float(hi);
                p3 -= __high2float(hi);
              }
              bt0[x] = movmatrix_t(*reinterpret_cast<const uint32_t*>(&lo));
              bt1[x] = movmatrix_t(*reinterpret_cast<const uint32_t*>(&hi));
            }
            // m-tile mt: dims 16 gq + mt and 16 gq + 8 + mt; tokens 2 c, 2 c + 1, 2 c + 8, 2 c + 9
            const unsigned char* vt = st + R::kBox;
            const uint4 x0 = lds128(vt + swz128(2 * c, gq)), x1 = lds128(vt + swz128(2 * c + 1, gq));
            const uint4 x2 = lds128(vt + swz128(2 * c + 8, gq)), x3 = lds128(vt + swz128(2 * c + 9, gq));
            const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
            const uint32_t w2[4] = {x2.x, x2.y, x2.z, x2.w}, w3[4] = {x3.x, x3.y, x3.z, x3.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // bytes 2 i and 2 i + 1 of both tokens, side by side
              const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
              const uint32_t ta = prmt(w0[i >> 1], w1[i >> 1], sel), tb = prmt(w0[2 + (i >> 1)], w1[2 + (i >> 1)], sel);
              const uint32_t tc = prmt(w2[i >> 1], w3[i >> 1], sel), td = prmt(w2[2 + (i >> 1)], w3[2 + (i >> 1)], sel);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t a0 = f16_of_codes(ta, k), a1 = f16_of_codes(tb, k);
                const uint32_t a2 = f16_of_codes(tc, k), a3 = f16_of_codes(td, k);
#pragma unroll
                for (int x = 0; x < FT; ++x) mma_f16(acc[2 * i + k], a0, a1, a2, a3, bt0[x], bt1[x]);
              }
            }
            continue;
          }
          // P (C layout: [token][head]) -> bf16 terms -> B layout ([head][token])
          uint32_t bt0[TERMS], bt1[TERMS];
#pragma unroll
          for (int x = 0; x < TERMS; ++x) {
            const uint32_t lo = pack_bf16(p0, p1), hi = pack_bf16(p2, p3);
            p0 -= bf16_lo(lo);
            p1 -= bf16_hi(lo);
            p2 -= bf16_lo(hi);
            p3 -= bf16_hi(hi);
            bt0[x] = movmatrix_t(lo);
            bt1[x] = movmatrix_t(hi);
          }
          // ---- O^T += V^T P^T
          if (E4M3) {  // as above, in bf16: for weights far below the largest, which need its range, and
                       // where tokens are hidden, whose codes may be NaN (here they become numbers)
            const unsigned char* vt = st + R::kBox;
            const uint4 x0 = lds128(vt + swz128(2 * c, gq)), x1 = lds128(vt + swz128(2 * c + 1, gq));
            const uint4 x2 = lds128(vt + swz128(2 * c + 8, gq)), x3 = lds128(vt + swz128(2 * c + 9, gq));
            const uint32_t w0[4] = {x0.x, x0.y, x0.z, x0.w}, w1[4] = {x1.x, x1.y, x1.z, x1.w};
            const uint32_t w2[4] = {x2.x, x2.y, x2.z, x2.w}, w3[4] = {x3.x, x3.y, x3.z, x3.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // byte pairs (2 i, 2 i + 1) of the 8 dims, and of the 8 after them
              const uint32_t sel = i & 1 ? 0x7632 : 0x5410;
              const uint32_t ta = prmt(w0[i >> 1], w1[i >> 1], sel), tb = prmt(w0[2 + (i >> 1)], w1[2 + (i >> 1)], sel);
              const uint32_t tc = prmt(w2[i >> 1], w3[i >> 1], sel), td = prmt(w2[2 + (i >> 1)], w3[2 + (i >> 1)], sel);
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t a0 = k ? bf16_high_codes(ta) : bf16_low_codes(ta);
                const uint32_t a1 = k ? bf16_high_codes(tb) : bf16_low_codes(tb);
                const uint32_t a2 = k ? bf16_high_codes(tc) : bf16_low_codes(tc);
                const uint32_t a3 = k ? bf16_high_codes(td) : bf16_low_codes(td);
#pragma unroll
                for (int x = 0; x < TERMS; ++x) mma_bf16(acc[2 * i + k], a0, a1, a2, a3, bt0[x], bt1[x]);
              }
            }
          } else {  // m-tile mt: dims 16 mt + gq and 16 mt + 8 + gq
#pragma unroll
            for (int mt = 0; mt < 8; ++mt) {
              uint32_t a0, a1, a2, a3;
              ldsm_x4_t(a0, a1, a2, a3, st + (2 + (mt >> 2)) * R::kBox + swz128(lrow_v, 2 * (mt & 3) + lchk_v));
#pragma unroll
              for (int x = 0; x < TERMS; ++x) mma_bf16(acc[mt], a0, a1, a2, a3, bt0[x], bt1[x]);
            }
          }
        }
        if (((it * SUB) & 31) == 32 - SUB) {
          pages = pages1;
          slots = slots1;
          look(it * SUB + SUB + 32 + lane, pages1, slots1);
        }
      }
      if (!alive) {  // the copies issued have landed before the ring goes (bounded)
        for (int it = max(0, issued - R::kStages); it < issued; ++it)
          mbar_wait(bars + (gi + (uint32_t)it) % R::kStages, ((gi + (uint32_t)it) / R::kStages) & 1u, nullptr);
      }
      gi += (uint32_t)n_it;

      if (E4M3) {  // acc in its own units again
        const float f = e_acc < 0 ? 0.f : __uint_as_float((uint32_t)e_acc << 23);
        const float down = 1.f / (float)(1 << kUp);
#pragma unroll
        for (int mt = 0; mt < 8; ++mt) {
          // (in two steps: f alone spans the normal numbers)
          acc[mt][0] = acc[mt][0] * down * f;
          acc[mt][1] = acc[mt][1] * down * f;
          acc[mt][2] = acc[mt][2] * down * f;
          acc[mt][3] = acc[mt][3] * down * f;
        }
      }

      // ---- merge the warps in shared memory
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) {
        l0 += __shfl_xor_sync(0xffffffffu, l0, o);
        l1 += __shfl_xor_sync(0xffffffffu, l1, o);
      }
      // (the maximum passes over NaN scores: where there was nothing else, the
      // merges would take the part for one that saw no token)
      if (l0 != l0) m0 = fmaxf(m0, 0.f);
      if (l1 != l1) m1 = fmaxf(m1, 0.f);
      __syncthreads();  // the rings are no longer read
      float* w_acc = reinterpret_cast<float*>(base);               // [warp][8][128]
      float* w_ml = w_acc + kWarps * kMaxGroup * kHeadDim;         // [warp][8][2]
      if (gq == 0) {
        *reinterpret_cast<float4*>(w_ml + (warp * kMaxGroup + 2 * c) * 2) = make_float4(m0, l0, m1, l1);
      }
#pragma unroll
      for (int mt = 0; mt < 8; ++mt) {
        const int d = E4M3 ? 16 * gq + mt : 16 * mt + gq;
        float* h0 = w_acc + (warp * kMaxGroup + 2 * c) * kHeadDim + d;
        h0[0] = acc[mt][0];
        h0[kHeadDim] = acc[mt][1];
        h0[8] = acc[mt][2];
        h0[kHeadDim + 8] = acc[mt][3];
      }
      __syncthreads();
      const int h = tid >> 4, d0 = (tid & 15) * 8;  // head and dims of this thread
      float M = ninf, L = 0.f, A[8];
#pragma unroll
      for (int x = 0; x < 8; ++x) A[x] = 0.f;
#pragma unroll
      for (int y = 0; y < kWarps; ++y) M = fmaxf(M, w_ml[(y * kMaxGroup + h) * 2]);
      if (M != ninf) {
#pragma unroll
        for (int y = 0; y < kWarps; ++y) {
          const float f = fast_exp2(w_ml[(y * kMaxGroup + h) * 2] - M);
          L += w_ml[(y * kMaxGroup + h) * 2 + 1] * f;
          const float* src = w_acc + (y * kMaxGroup + h) * kHeadDim + d0;
#pragma unroll
          for (int x = 0; x < 8; ++x) A[x] += src[x] * f;
        }
      }
      const bool whole = i0 == 0 && i1 == u.nt;
      if (h < G) {
        const size_t row = (size_t)b * a.p.Hq + (size_t)g * G + h;
        if (!whole) {
          float* dst = a.parts + (((size_t)blockIdx.x * 2 + (i0 == 0 ? 1 : 0)) * kMaxGroup + h) * kPart;
          *reinterpret_cast<float4*>(dst + d0) = make_float4(A[0], A[1], A[2], A[3]);
          *reinterpret_cast<float4*>(dst + d0 + 4) = make_float4(A[4], A[5], A[6], A[7]);
          if (d0 == 0) *reinterpret_cast<float2*>(dst + kHeadDim) = make_float2(M, L);
        } else {
          const float inv = L != 0.f ? 1.f / L : 0.f;
          if (a.p.out) {
            float* o = a.p.out + row * kHeadDim + d0;
            *reinterpret_cast<float4*>(o) = make_float4(A[0] * inv, A[1] * inv, A[2] * inv, A[3] * inv);
            *reinterpret_cast<float4*>(o + 4) = make_float4(A[4] * inv, A[5] * inv, A[6] * inv, A[7] * inv);
          } else {
            *reinterpret_cast<uint4*>(a.p.out_bf16 + row * kHeadDim + d0) =
                make_uint4(pack_bf16(A[0] * inv, A[1] * inv), pack_bf16(A[2] * inv, A[3] * inv),
                           pack_bf16(A[4] * inv, A[5] * inv), pack_bf16(A[6] * inv, A[7] * inv));
          }
          if (a.p.lse && d0 == 0) a.p.lse[row] = L != 0.f ? M * kLn2 + logf(L) : ninf;
        }
      }
      if (tid == 0 && i0 == 0) {  // whether, and up to which CTA, the unit goes on
        int last = -1;
        if (!whole) {
          const long long x = at + cost - 1, longer = (each + 1) * more;
          last = x < longer ? (int)(x / (each + 1)) : (int)(more + (x - longer) / each);
        }
        if (a.by_unit) a.recs[b * Hkv + g] = make_int4(last < 0 ? -1 : (int)blockIdx.x, last, b, g);
        else if (last >= 0) a.recs[blockIdx.x] = make_int4((int)blockIdx.x, last, b, g);
      }
      fence_proxy_async();  // generic accesses to the ring before the next copies into it
      __syncthreads();
    }
    rem -= take;
    if (off + take == cost) {
      at += cost;
      off = 0;
      if (++g == Hkv) {
        g = 0;
        if (++b < B) u = unit_of(a, paged_tokens(kv, b, nullptr));
      }
    } else {
      off += take;
    }
  }
}

// Merge of the parts of a unit that was cut: a block per (cut unit, head); warp
// w takes parts w, w + 8, ..., lane l dims 4 l .. 4 l + 3; the warps' results
// are then merged in warp order.
__global__ void __launch_bounds__(256) decode_combine_kernel(const __grid_constant__ PagedDecodeArgs a) {
  grid_dep_wait();
  __shared__ float s_o[8][kHeadDim];
  __shared__ float2 s_ml[8];
  const int G = a.p.G;
  const int4 rec = a.recs[blockIdx.x / G];
  if (rec.x < 0) return;
  const int h = blockIdx.x % G, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float ninf = -__int_as_float(0x7f800000);
  const int np = rec.y - rec.x + 1;
  float M = ninf, L = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int kBatch = 8;
  for (int p0 = warp; p0 < np; p0 += 8 * kBatch) {
    float2 ml[kBatch];
    float4 v[kBatch];
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int p = p0 + 8 * i;
      const bool ok = p < np;
      const float* src =
          a.parts + (((size_t)(rec.x + (ok ? p : 0)) * 2 + (!ok || p == 0 ? 1 : 0)) * kMaxGroup + h) * kPart;
      ml[i] = ok ? __ldcg(reinterpret_cast<const float2*>(src + kHeadDim)) : make_float2(ninf, 0.f);
      v[i] = ok ? __ldcg(reinterpret_cast<const float4*>(src) + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float nm = M;
#pragma unroll
    for (int i = 0; i < kBatch; ++i) nm = fmaxf(nm, ml[i].x);
    if (nm == ninf) continue;
    const float f = fast_exp2(M - nm);
    L *= f;
    o = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const float e = fast_exp2(ml[i].x - nm);
      L += ml[i].y * e;
      o.x += v[i].x * e;
      o.y += v[i].y * e;
      o.z += v[i].z * e;
      o.w += v[i].w * e;
    }
    M = nm;
  }
  *reinterpret_cast<float4*>(&s_o[warp][4 * lane]) = o;
  if (lane == 0) s_ml[warp] = make_float2(M, L);
  __syncthreads();
  if (warp) return;
  M = ninf;
#pragma unroll
  for (int y = 0; y < 8; ++y) M = fmaxf(M, s_ml[y].x);
  L = 0.f;
  o = make_float4(0.f, 0.f, 0.f, 0.f);
  if (M != ninf) {
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      const float e = fast_exp2(s_ml[y].x - M);
      const float4 v = *reinterpret_cast<const float4*>(&s_o[y][4 * lane]);
      L += s_ml[y].y * e;
      o.x += v.x * e;
      o.y += v.y * e;
      o.z += v.z * e;
      o.w += v.w * e;
    }
  }
  const float inv = L != 0.f ? 1.f / L : 0.f;
  const size_t row = (size_t)rec.z * a.p.Hq + (size_t)rec.w * G + h;
  if (a.p.out)
    *reinterpret_cast<float4*>(a.p.out + row * kHeadDim + 4 * lane) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
  else
    *reinterpret_cast<uint2*>(a.p.out_bf16 + row * kHeadDim + 4 * lane) =
        make_uint2(pack_bf16(o.x * inv, o.y * inv), pack_bf16(o.z * inv, o.w * inv));
  if (a.p.lse && lane == 0) a.p.lse[row] = L != 0.f ? M * kLn2 + logf(L) : ninf;
}

template <bool E4M3, int TERMS>
cudaError_t launch(const PagedDecodeArgs& a, int grid, cudaStream_t st) {
  auto* k = paged_decode_kernel<E4M3, TERMS>;
  const cudaError_t e = set_smem_attr((const void*)k, Ring<E4M3>::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, (unsigned)grid, kThreads, Ring<E4M3>::kSmem, st, a);
}

}  // namespace

int paged_decode_grid(int sms) { return 3 * sms; }

size_t paged_decode_part_floats() { return 2 * (size_t)kMaxGroup * kPart; }

cudaError_t launch_paged_decode(const PagedDecodeArgs& a, int grid, int recs, cudaStream_t st) {
  const bool f32 = a.p.out != nullptr;
  const cudaError_t e = a.p.kv.e4m3 ? (f32 ? launch<true, 3>(a, grid, st) : launch<true, 2>(a, grid, st))
                                    : (f32 ? launch<false, 3>(a, grid, st) : launch<false, 2>(a, grid, st));
  if (e != cudaSuccess) return e;
  return launch_pdl(decode_combine_kernel, (unsigned)recs * a.p.G, 256, 0, st, a);
}

}  // namespace sa
