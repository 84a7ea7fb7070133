// Attention of a chunk of new rows of every sequence over its paged cache, on
// tcgen05.
//
// Mathematics: row i of sequence b at position p = N_b - m_b + i, query head h
// of KV head g: z_t = scale q . k_t over the visible tokens t (t <= p, inside
// the window or among the first tokens), out = sum exp(z_t - lse) v_t, by one
// pass over the tokens with a running reference maximum and sum.  Measured: 2048
// rows over 32k tokens, 28 heads, bf16: 1.07 ms (870 TFLOP/s; the tensor pipe is
// 45% busy: QK, softmax and PV wait for one another, and for shared memory); four
// prompts of up to 2048 tokens, 32 heads, e4m3: 234 us.
//
// Units.  A query vector is a (row, query head) pair.  The G heads of a KV head
// and R = floor(128 / G) consecutive rows make a tile of up to 128 vectors (M of
// the MMA); two tiles (2 R rows) make a pair that shares every K/V block of BLK
// tokens.  Where a pair has rows for one tile only, both tile slots take that
// tile and every other block each, and merge at the end.
//
// Split.  The work is the list of (sequence, KV head, pair) with nb blocks
// each; the grid is one CTA per SM and takes equal runs of nb + kC0 over that
// list, cut anywhere, so that neither the number of pairs nor the causal
// triangle leaves SMs idle and a few rows over a long cache spread over every
// SM.  Every CTA computes the list's prefix from the lengths on the device
// (no host copy: a captured launch replays with other lengths).  A pair cut
// between CTAs leaves unnormalised partial results in the workspace, which
// combine_kernel merges in CTA order: results do not depend on scheduling.
//
// CTA, warp-specialised, every wait bounded:
//   warps 0-7, 8-15  softmax of tile slot 0, 1: two threads per query vector
//                    (TMEM lane), each half of the block's scores in registers.
//                    Weights are taken against a reference that both threads
//                    hold; it is raised to the row's maximum only when a half
//                    block's sum of weights passes 2^20 (fp32 and bf16 hold them
//                    as exactly there), and the block's weights are taken again;
//                    whether any row needs that is one barrier reduction over
//                    the pair of warps, and no maximum is taken otherwise.  (With a
//                    thread per row, two warps per scheduler, the chain of
//                    loads, maxima and exponentials was bound by its latency:
//                    2600 cycles per 64 tokens, 1024 of them exponentials.)
//   warp 16          TMA of the queries and of the K and V tiles (boxes of up to
//                    BLK rows inside a page; boxes that no row of the pair
//                    needs, or whose page is bad, are fetched from past the
//                    pool's end and so read as zeros);
//   warps 17, 18     issue S = Q K^T of slot 0 / 1 (one thread each) into one of
//                    the slot's two S buffers;
//   warp 19          issues O += P V of both slots once the softmax has written
//                    P over S.  The softmax always finds the next scores ready,
//                    and the products of one block run under the softmax of the
//                    next.  (With one buffer of 128 tokens a slot's softmax and
//                    products alternate and their latencies add up: 5080 cycles
//                    per 128 tokens and pair against 2240 of MMA time.  The
//                    products' operands fill shared memory's bandwidth, so a
//                    wait on a barrier costs 200 cycles even when it is over;
//                    one thread per slot for both products took 2490 cycles per
//                    64 tokens, the three take about 1600.);
//   warps 20-23, 24-27 (e4m3 cache) turn the codes of K, of V, fetched into a
//                    ring of their own, into bf16 tiles: code * 2^k is exactly
//                    a bf16, so the products are those of a bf16 cache of the
//                    rounded values.
// Roles run ahead of each other over block and segment boundaries; only the
// mbarriers order them.
//
// A weight of 0 keeps no NaN or infinity of a V row out of the products.  Rows
// that no row of the pair sees are zeros by the time of PV.  In rows that some
// see and others do not such a value makes its dim NaN in every vector of the
// tile; so a look at the first vector's result shows it.  combine_kernel then
// looks through those V rows, and takes the dims that have such a value again,
// token by token.  (A bf16 cache only: what the converters write are numbers.
// Four bf16 prompts 127 -> 130 us, 16 rows over 29.5k tokens 43.8 -> 46.9;
// looking through the V rows ahead of PV cost the prompts 1 to 38 us and the
// short calls 2 to 6, by whichever warps.)
//
// P is rounded to bf16 where the output is bf16 (its error, 2^-8 per weight, is
// that of the output's own rounding); for fp32 outputs it is split into three
// bf16 terms (24 bits), which leaves room for one S buffer per slot.
#include "paged.cuh"
#include "tcgen05.cuh"
#include "internal.h"

namespace sa {
namespace {

constexpr int kC0 = 2;              // cost of starting a pair, in blocks
// Least work of a CTA: small calls are a chain of latencies and so spread widely
// (16 rows over 2k tokens, 4 KV heads, bf16, fp32 outputs, in a graph: 22.4 us;
// shares of 4 and 6: 23.2 and 27.6).
constexpr int kMinShare = kC0 + 1;
constexpr int kInfo = 16;
constexpr int BLK = 64;             // tokens of a block
constexpr int NR = 4;               // tiles of codes in flight (K, V alternating)
constexpr int kQTileBytes = 2 * 128 * 128;
constexpr int kRingBytes = 128 * 1024;
constexpr uint32_t kColS = 0, kColO = 256;  // slot t: S / P at 128 t, O at 256 + 128 t

template <int TERMS>
struct Shape {
  static constexpr int NB = TERMS == 1 ? 2 : 1;       // S buffers of a slot
  static constexpr int kHalf = BLK * 128;             // 64 dims of a tile
  static constexpr int kSlot = 2 * kHalf;             // a K or V tile
  static constexpr int NS = kRingBytes / kSlot;       // ring slots (K, V alternating)
  static constexpr int kOffRing = 2 * kQTileBytes;
  static constexpr int kRaw = BLK * 128;              // codes of a K or V tile
  static constexpr int kOffRaw = kOffRing + kRingBytes;   // e4m3 only: NR tiles of codes
  static constexpr int kNumBars = 2 * NS + 2 + 2 * 6 + 2 + 1 + 2 * NR;
  static constexpr int off_bars(bool e4m3) { return kOffRaw + (e4m3 ? NR * kRaw : 0); }
  static constexpr int off_info(bool e4m3) { return off_bars(e4m3) + 8 * kNumBars; }
  static constexpr int off_scale(bool e4m3) { return (off_info(e4m3) + 4 * (kInfo + 1) + 15) & ~15; }
  static constexpr int off_x(bool e4m3) { return off_scale(e4m3) + (e4m3 ? NR * BLK : 0); }
  static constexpr int smem(bool e4m3) { return 1024 + off_x(e4m3) + 2 * 128 * 4; }
};

// Registers per thread of the softmax, of the issuing and copying warps and of
// the converters, once the warpgroups have split what the launch gave them.
template <bool E4M3>
struct Regs {
  static constexpr int kSoftmax = E4M3 ? 88 : 104, kIssue = E4M3 ? 56 : 64, kConvert = 48;
  static constexpr int kThreads = E4M3 ? 896 : 640;
  static constexpr int kTotal = 512 * kSoftmax + 128 * kIssue + (E4M3 ? 256 * kConvert : 0);
};

template <int R>
SA_DEV void reg_alloc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(R));
}
template <int R>
SA_DEV void reg_dealloc() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(R));
}

// Whether `v` holds in any thread of the 2 warps that meet at barrier `id`.
SA_DEV bool pair_any(int id, bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n bar.red.or.pred q, %2, 64, p;\n selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "r"(id)
      : "memory");
  return r != 0;
}
// The lowest n bits, n clipped to [0, 32].
SA_DEV uint32_t first_bits(int n) { return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u); }

SA_DEV void pair_sync(int id) { asm volatile("bar.sync %0, 64;\n" ::"r"(id) : "memory"); }

SA_DEV float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// MN-major view of V: 8-token atoms 1 KiB apart, the two 64-dim halves apart
// by HALF bytes.
template <int HALF>
SA_DEV uint64_t v_desc(const unsigned char* v) {
  return (tc::smem_desc_sw128(v) & ~(0x3FFFull << 16)) | ((uint64_t)(HALF >> 4) << 16);
}

// Blocks of pair j of a sequence: tokens [0, S) (first tokens) and [lo, p1].
struct Geom {
  int rows, p0, p1, lo, S, sb, wb0, nb;
};
SA_DEV Geom pair_geom(const ChunkArgs& a, int N, int m, int j) {
  Geom q;
  q.rows = min(2 * a.R, m - 2 * a.R * j);
  q.p0 = N - m + 2 * a.R * j;
  q.p1 = q.p0 + q.rows - 1;
  q.lo = a.p.window && q.p0 >= a.p.window ? q.p0 - a.p.window + 1 : 0;
  q.S = a.p.window ? min(a.p.sinks, q.p1 + 1) : 0;
  if (q.p1 < 0) {
    q.sb = q.wb0 = q.nb = 0;
    return q;
  }
  q.wb0 = q.lo / BLK;
  q.sb = min((q.S + BLK - 1) / BLK, q.wb0);
  q.nb = q.sb + q.p1 / BLK - q.wb0 + 1;
  return q;
}

// A run [i0, i1) of the blocks of one pair, on this CTA.
struct Seg : Geom {
  int b, g, N, row0;          // row0: first row of the pair in the row arrays
  int i0, i1, cost;
  bool single;                // rows for one tile only
  unsigned long long w;       // where the pair's work begins
};

struct Plan {
  int b, g, j, off;
  unsigned more;
  unsigned long long w0, w1, each;
  // The CTA that has unit x of the work.
  SA_DEV int cta_of(unsigned long long x) const {
    const unsigned long long longer = (each + 1) * more;
    if (x < longer) return (int)(x / (each + 1));
    return (int)(more + (x - longer) / each);
  }
};

// Walks the segments of a CTA; every role has its own.
struct Cursor {
  int b, g, j, off, N, m, r0, pairs;
  unsigned long long w, rem;
  SA_DEV Cursor(const ChunkArgs& a, const Plan& p)
      : b(p.b), g(p.g), j(p.j), off(p.off), N(0), m(0), r0(0), pairs(0), w(p.w0 - p.off), rem(p.w1 - p.w0) {
    if (rem) load(a);
  }
  SA_DEV void load(const ChunkArgs& a) {
    for (; b < a.p.kv.B; ++b) {
      m = paged_rows(a.p.row_off, a.p.n_rows, b, r0, a.p.status);
      if (m > 0) break;
    }
    if (b < a.p.kv.B) {
      N = paged_tokens(a.p.kv, b, a.p.status);
      pairs = (m + 2 * a.R - 1) / (2 * a.R);
    }
  }
  SA_DEV bool next(const ChunkArgs& a, Seg& s) {
    while (rem && b < a.p.kv.B) {
      static_cast<Geom&>(s) = pair_geom(a, N, m, j);
      s.cost = s.nb + kC0;
      const int take = (int)min(rem, (unsigned long long)(s.cost - off));
      const int from = off, to = off + take;
      rem -= take;
      s.b = b;
      s.g = g;
      s.N = N;
      s.row0 = r0 + 2 * a.R * j;
      s.i0 = min(max(from - kC0, 0), s.nb);
      s.i1 = min(max(to - kC0, 0), s.nb);
      s.single = s.rows <= a.R;
      s.w = w;
      if (to == s.cost) {
        w += s.cost;
        off = 0;
        if (++j == pairs) {
          j = 0;
          if (++g == a.p.kv.Hkv) {
            g = 0;
            ++b;
            load(a);
          }
        }
      }
      if (s.i1 > s.i0 || (s.nb == 0 && from == 0)) return true;
    }
    return false;
  }
};

// Work of the sequences b (one per thread of a converged warp), one KV head;
// their tokens and new rows.
SA_DEV unsigned long long seq_work(const ChunkArgs& a, int b, int& N, int& m) {
  int r0;
  N = m = 0;
  if (b < a.p.kv.B) {
    m = paged_rows(a.p.row_off, a.p.n_rows, b, r0, a.p.status);
    N = paged_tokens(a.p.kv, b, a.p.status);
  }
  const int pairs = (m + 2 * a.R - 1) / (2 * a.R);
  unsigned long long w = 0;
  if (pairs <= 8)
    for (int j = 0; j < pairs; ++j) w += pair_geom(a, N, m, j).nb + kC0;
  unsigned many = __ballot_sync(0xffffffffu, pairs > 8);  // long ones: the whole warp
  const int lane = threadIdx.x & 31;
  while (many) {
    const int src = __ffs(many) - 1;
    many &= many - 1;
    const int sn = __shfl_sync(0xffffffffu, N, src), sm = __shfl_sync(0xffffffffu, m, src);
    const int sp = __shfl_sync(0xffffffffu, pairs, src);
    unsigned long long x = 0;
    for (int j = lane; j < sp; j += 32) x += pair_geom(a, sn, sm, j).nb + kC0;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    if (lane == src) w = x;
  }
  return w;
}

// Exclusive prefix over the block and its total (every thread calls it).
SA_DEV unsigned long long scan64(unsigned long long v, unsigned long long* scratch, unsigned long long& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  unsigned long long x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) scratch[warp] = x;
  __syncthreads();
  unsigned long long base = 0, tot = 0;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) base += scratch[w];
    tot += scratch[w];
  }
  __syncthreads();
  total = tot;
  return base + x - v;
}

// The pair of sequence (N, m) that holds unit `off` of one head's work (a warp).
SA_DEV void find_pair(const ChunkArgs& a, int N, int m, unsigned long long off, Plan* plan) {
  const int lane = threadIdx.x & 31, pairs = (m + 2 * a.R - 1) / (2 * a.R);
  unsigned long long before = 0;
  for (int j0 = 0; j0 < pairs; j0 += 32) {
    const int j = j0 + lane;
    const unsigned long long cst = j < pairs ? pair_geom(a, N, m, j).nb + kC0 : 0;
    unsigned long long x = cst;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    x += before;
    if (cst && x - cst <= off && off < x) {
      plan->j = j;
      plan->off = (int)(off - (x - cst));
    }
    before = __shfl_sync(0xffffffffu, x, 31);
  }
}

// This CTA's run of a list of `total` work.
SA_DEV void share(unsigned long long total, Plan* plan) {
  // as many CTAs as have kMinShare each; the first `more` of them take one unit more than `each`
  const unsigned n = total >= (unsigned long long)gridDim.x * kMinShare ? gridDim.x : max(1u, (unsigned)total / kMinShare);
  const unsigned c = blockIdx.x;
  const unsigned long long each = total >> 32 ? total / n : (unsigned)total / n;
  const unsigned more = (unsigned)(total - each * n);
  plan->each = each;
  plan->more = more;
  plan->w0 = c < n ? each * c + min(c, more) : 0;
  plan->w1 = c < n ? plan->w0 + each + (c < more ? 1u : 0u) : 0;
}

// This CTA's share of the work (every thread calls it; scratch: 30 words; the
// caller synchronises before the plan is read).
SA_DEV void make_plan(const ChunkArgs& a, Plan* plan, unsigned long long* scratch) {
  const int T = blockDim.x, tid = threadIdx.x, lane = tid & 31, B = a.p.kv.B;
  const unsigned long long H = a.p.kv.Hkv;
  if (B <= 32) {  // one warp, without block barriers: 3200 cycles instead of 5000
    if (tid >= 32) return;
    int N = 0, m = 0;
    const unsigned long long per = seq_work(a, lane, N, m), w = per * H;
    unsigned long long x = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned long long y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    Plan p;
    share(__shfl_sync(0xffffffffu, x, 31), &p);
    p.b = B;
    p.g = p.j = p.off = 0;
    const unsigned here = __ballot_sync(0xffffffffu, w && x - w <= p.w0 && p.w0 < x);
    if (p.w1 != p.w0 && here) {
      p.b = __ffs(here) - 1;
      const unsigned long long in = p.w0 - __shfl_sync(0xffffffffu, x - w, p.b), one = __shfl_sync(0xffffffffu, per, p.b);
      p.g = (in >> 32) || (one >> 32) ? (int)(in / one) : (int)((unsigned)in / (unsigned)one);
      if (lane == 0) *plan = p;
      __syncwarp();
      find_pair(a, __shfl_sync(0xffffffffu, N, p.b), __shfl_sync(0xffffffffu, m, p.b), in - (unsigned long long)p.g * one,
                plan);
    } else if (lane == 0) {
      *plan = p;
    }
    return;
  }
  unsigned long long total = 0, w = 0, w1 = 0, t, ex = 0;
  int N, m;
  for (int base = 0; base < B; base += T) {
    w1 = seq_work(a, base + tid, N, m);
    w = w1 * H;
    ex = scan64(w, scratch, t) + total;
    total += t;
  }
  if (tid == 0) {
    share(total, plan);
    plan->b = B;
    plan->g = plan->j = plan->off = 0;
  }
  __syncthreads();
  const unsigned long long w0 = plan->w0;
  if (plan->w1 == w0) return;
  unsigned long long run = 0;
  for (int base = 0; base < B; base += T) {
    if (B > T) {
      w1 = seq_work(a, base + tid, N, m);
      w = w1 * H;
      ex = scan64(w, scratch, t) + run;
      run += t;
    }
    if (w && ex <= w0 && w0 < ex + w) {
      plan->b = base + tid;
      scratch[28] = w0 - ex;
      scratch[29] = w1;
    }
  }
  __syncthreads();
  if (tid < 32) {
    const unsigned long long in = scratch[28], per = scratch[29];
    const int b = plan->b, g = (in >> 32) || (per >> 32) ? (int)(in / per) : (int)((unsigned)in / (unsigned)per);
    int r0;
    m = paged_rows(a.p.row_off, a.p.n_rows, b, r0, nullptr);
    N = paged_tokens(a.p.kv, b, nullptr);
    if (tid == 0) plan->g = g;
    find_pair(a, N, m, in - (unsigned long long)g * per, plan);
  }
}

// 4 codes -> two bf16 pairs: a code's 7 low bits are the exponent and mantissa
// of a bf16 2^120 times smaller, subnormals included; m2 holds 2^(120 + k) (and
// then `more`, another power of two, for rows past 2^127) in both halves.
SA_DEV uint32_t mul_bf16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.bf16x2 %0, %1, %2;\n" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
SA_DEV uint2 bf16_of_codes(uint32_t w, uint32_t m2) {
  const uint32_t odd = mul_bf16x2((w & 0x80008000u) | ((w >> 4) & 0x07f007f0u), m2);
  const uint32_t even = mul_bf16x2(((w << 8) & 0x80008000u) | ((w << 4) & 0x07f007f0u), m2);
  return make_uint2(prmt(even, odd, 0x5410), prmt(even, odd, 0x7632));
}

// Two fp32 values in one 64-bit register pair, for the packed instructions.
SA_DEV unsigned long long pack_f2(float x, float y) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
SA_DEV void unpack_f2(unsigned long long v, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(v));
}
SA_DEV unsigned long long fma_f2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
SA_DEV unsigned long long add_f2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
template <bool E4M3, int TERMS>
__global__ void __launch_bounds__(Regs<E4M3>::kThreads, 1) chunk_kernel(const __grid_constant__ ChunkArgs a) {
  using Sh = Shape<TERMS>;
  constexpr int NS = Sh::NS, NB = Sh::NB;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint32_t s_tmem;
  __shared__ Plan s_plan;
  __shared__ unsigned long long s_scan[30];
  unsigned char* base = reinterpret_cast<unsigned char*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  unsigned char* qs = base;
  unsigned char* ring = base + Sh::kOffRing;
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(base + Sh::off_bars(E4M3));
  uint64_t* kv_empty = kv_full + NS;
  uint64_t* q_full = kv_empty + NS;
  uint64_t* q_empty = q_full + 1;
  uint64_t* s_full = q_empty + 1;   // [slot][buffer]
  uint64_t* p_full = s_full + 4;    // [slot][buffer]
  uint64_t* o_done = p_full + 4;    // [slot][parity of the PV]
  uint64_t* x_full = o_done + 4;
  uint64_t* x_empty = x_full + 1;
  uint64_t* drain = x_empty + 1;
  uint64_t* raw_full = drain + 1;   // [NR]
  uint64_t* raw_empty = raw_full + NR;
  // [block % kInfo]: its 16-token pieces on bad pages; [kInfo]: whether any piece ever was
  volatile uint32_t* info = reinterpret_cast<uint32_t*>(base + Sh::off_info(E4M3));
  unsigned char* raw = base + Sh::kOffRaw;
  unsigned char* raw_scale = base + Sh::off_scale(E4M3);  // [NR][BLK]
  volatile float* xchg = reinterpret_cast<float*>(base + Sh::off_x(E4M3));  // [slot][128]

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float ninf = -__int_as_float(0x7f800000);
  int* status = a.p.status;

  if (tid == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(kv_full + s, E4M3 ? 4 : 1);
      mbar_init(kv_empty + s, s & 1 ? 1 : 2);  // K: both slots' issuers, V: one
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 2);
    for (int i = 0; i < 4; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 8);
      mbar_init(o_done + i, 1);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(raw_full + i, 1);
      mbar_init(raw_empty + i, 4);
    }
    mbar_init(x_full, 8);
    mbar_init(x_empty, 8);
    mbar_init(drain, 3);
    info[kInfo] = 0u;
    fence_barrier_init();
    prefetch_tmap(&a.tmap_q);
    prefetch_tmap(&a.tmap_k);
    prefetch_tmap(&a.tmap_v);
  }
  if (warp == 0) {
    tc::tmem_alloc(&s_tmem, 512);
    tc::tmem_relinquish();
  }
  grid_dep_wait();
  make_plan(a, &s_plan, s_scan);
  if (tid == 0) {
    a.recs[blockIdx.x] = ChunkRec{0, 0, 0, 0, 0};
    if (!E4M3) a.odd[blockIdx.x] = ChunkOdd{0x7fffffff, -1};
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  const uint32_t tmem = s_tmem;
  const PagedView& kv = a.p.kv;
  Cursor cur(a, s_plan);
  Seg sg;

  if (warp >= 16 && warp < 20) {
    reg_dealloc<Regs<E4M3>::kIssue>();
    if (warp == 16) {
      // ---- producer
      int n = 0, segs = 0, issued = 0;  // issued: K and V tiles
      bool ok = true;
      const int hb = a.hb, nbox = BLK / hb, sub = lane >> 1;  // this lane's box: rows sub * hb .., half lane & 1
      while (ok && cur.next(a, sg)) {
        if (sg.i0 == sg.i1) continue;
        if (segs > 0) ok = mbar_wait(q_empty, (segs - 1) & 1u, status);
        if (!__all_sync(0xffffffffu, ok)) {
          ok = false;
          break;
        }
        const int tiles = sg.single ? 1 : 2;
        if (lane == 0) mbar_arrive_expect_tx(q_full, (uint32_t)(tiles * 2 * 128 * a.p.G * a.R));
        __syncwarp();
        if (lane < 2 * tiles)
          tma_load_3d(qs + (lane >> 1) * kQTileBytes + (lane & 1) * (128 * 128), &a.tmap_q, 64 * (lane & 1),
                      sg.g * a.p.G, sg.row0 + (lane >> 1) * a.R, q_full);
        ++segs;
        // Table entry and slot of this lane's box of block i; entry -1 where no
        // row of the pair needs it.  Looked up a block ahead: the lookup's
        // latency would otherwise stand between a freed tile and its copy.
        auto lookup = [&](int i, int& entry, int& slot) {
          const int t0 = (i < sg.sb ? i : sg.wb0 + i - sg.sb) * BLK + sub * hb;
          entry = -1;
          slot = 0;
          if (sub < nbox && i < sg.i1 && (t0 < sg.S || (t0 <= sg.p1 && t0 + hb > sg.lo))) {
            const int p = t0 / kv.page_size;
            slot = t0 - p * kv.page_size;
            entry = __ldg(kv.table + (size_t)sg.b * kv.max_pages + p);
            if (entry == -1) entry = -2;
          }
        };
        int entry, slot;
        lookup(sg.i0, entry, slot);
        for (int i = sg.i0; ok && i < sg.i1; ++i, ++n) {
          int entry1, slot1;
          lookup(i + 1, entry1, slot1);
          const bool good = entry >= 0 && entry < kv.n_pages;
          const int at = good ? entry : (int)kv.n_pages;  // past the pool: zeros
          const uint32_t mine = !good && entry != -1 ? ((1u << (hb / 16)) - 1u) << (sub * (hb / 16)) : 0u;
          const uint32_t bad = __reduce_or_sync(0xffffffffu, mine);
          if (mine) flag_status(status, SA_ERR_DEVICE_CHECK);
          const uint32_t boxes = __popc(__ballot_sync(0xffffffffu, good && !(lane & 1)));
#pragma unroll 1
          for (int w = 0; w < 2; ++w) {
            const CUtensorMap* tmap = w ? &a.tmap_v : &a.tmap_k;
            const int x = 2 * n + w;
            const int rs = E4M3 ? x % NR : x % NS;
            const uint32_t use = (uint32_t)(E4M3 ? x / NR : x / NS);
            if (use > 0) ok = mbar_wait((E4M3 ? raw_empty : kv_empty) + rs, (use - 1) & 1u, status);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            // the softmax reads it once the block's scores are there, which
            // takes this K tile (ordered by the barriers on that way)
            if (w == 0 && lane == 0) {
              info[n % kInfo] = bad;
              if (bad) info[kInfo] = 1u;
            }
            if (E4M3) {  // codes with their rows' scale bytes
              if (lane == 0) mbar_arrive_expect_tx(raw_full + rs, (uint32_t)Sh::kRaw + boxes * hb);
              __syncwarp();
              if (sub < nbox && !(lane & 1)) {
                tma_load_4d(raw + rs * Sh::kRaw + sub * hb * 128, tmap, 0, slot, sg.g, at, raw_full + rs);
                if (good)
                  bulk_load(raw_scale + rs * BLK + sub * hb,
                            (w ? kv.v_scale : kv.k_scale) + scale_index(kv, at, sg.g, slot), hb, raw_full + rs);
              }
            } else {
              if (lane == 0) mbar_arrive_expect_tx(kv_full + rs, Sh::kSlot);
              __syncwarp();
              if (sub < nbox)
                tma_load_4d(ring + rs * Sh::kSlot + (lane & 1) * Sh::kHalf + sub * hb * 128, tmap, 64 * (lane & 1),
                            slot, sg.g, at, kv_full + rs);
            }
            issued = x + 1;
          }
          entry = entry1;
          slot = slot1;
        }
      }
      // every copy issued has landed before the CTA ends (bounded)
      if (segs > 0) mbar_wait(q_full, (segs - 1) & 1u, nullptr);
      if (E4M3) {
        for (int x = max(0, issued - NR); x < issued; ++x) mbar_wait(raw_full + x % NR, (uint32_t)(x / NR) & 1u, nullptr);
      } else {
        for (int x = max(0, issued - NS); x < issued; ++x) mbar_wait(kv_full + x % NS, (uint32_t)(x / NS) & 1u, nullptr);
      }
    } else if (warp < 19 && lane == 0) {
      // ---- QK of slot t: of two tiles, its tile and every block; of one tile,
      // the blocks of its parity
      const int t = warp - 17;
      const uint32_t idesc_s = tc::idesc_f32acc(tc::kFmtBF16, 128, BLK);
      const uint32_t ts = tmem + kColS + 128u * t;
      const uint64_t k_desc = tc::smem_desc_sw128(ring);
      int n = 0, segs = 0;
      uint32_t c = 0;  // QKs issued
      bool ok = true;
      while (ok && cur.next(a, sg)) {
        const int n0 = n;
        if (sg.i1 == sg.i0) continue;
        n += sg.i1 - sg.i0;
        if (!(ok = mbar_wait(q_full, segs & 1u, status))) break;
        ++segs;
        const bool single = sg.single;
        const int step = single ? 2 : 1;
        int m = single ? n0 + ((n0 ^ t) & 1) : n0;
        const uint64_t q_desc = tc::smem_desc_sw128(qs + (single ? 0 : t * kQTileBytes));
        if (m >= n) mbar_arrive(q_empty);
#pragma unroll 1
        for (; m < n; m += step) {
          const int ks = (2 * m) % NS;
          const uint32_t b = c % NB;
          if (!(ok = mbar_wait(kv_full + ks, (uint32_t)((2 * m) / NS) & 1u, status))) break;
          // the buffer is free once the PV of the slot's block c - NB is done
          if (c >= (uint32_t)NB && !(ok = mbar_wait(o_done + 2 * t + ((c - NB) & 1u), ((c - NB) >> 1) & 1u, status))) break;
          tc::fence_after_sync();
          const uint64_t kd = k_desc + (uint64_t)(ks * (Sh::kSlot >> 4));
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              tc::mma_bf16_ss(ts + 64u * b, q_desc + (uint64_t)(h * (128 * 128 / 16) + 2 * x),
                              kd + (uint64_t)(h * (Sh::kHalf / 16) + 2 * x), idesc_s, (h | x) != 0);
          tc::commit(s_full + 2 * t + b);
          tc::commit(kv_empty + ks);
          if (single) tc::commit(kv_empty + ks);
          if (m + step >= n) tc::commit(q_empty);
          ++c;
        }
      }
      // every MMA issued has completed before TMEM is freed (bounded)
      tc::commit(drain);
      mbar_wait(drain, 0, nullptr);
    } else if (warp == 19 && lane == 0) {
      // ---- PV of both slots
      const uint32_t idesc_o = tc::idesc_f32acc(tc::kFmtBF16, 128, kHeadDim) | (1u << 16);  // V MN-major
      const uint64_t vt_desc = v_desc<Sh::kHalf>(ring);
      int n = 0;
      uint32_t c0 = 0, c1 = 0;  // PVs issued per slot
      bool ok = true;
      while (ok && cur.next(a, sg)) {
        const int n0 = n, n_end = n + sg.i1 - sg.i0;
        const bool single = sg.single;
#pragma unroll 1
        for (; ok && n < n_end; ++n) {
          const int vs = (2 * n) % NS + 1;
          if (!(ok = mbar_wait(kv_full + vs, (uint32_t)((2 * n) / NS) & 1u, status))) break;
          const uint64_t vd = vt_desc + (uint64_t)(vs * (Sh::kSlot >> 4));
#pragma unroll 1
          for (int t = single ? (n & 1) : 0; t < (single ? (n & 1) + 1 : 2); ++t) {
            const uint32_t c = t ? c1 : c0, b = c % NB;
            if (!(ok = mbar_wait(p_full + 2 * t + b, (c / NB) & 1u, status))) break;
            tc::fence_after_sync();
            const bool acc = single ? n >= n0 + 2 : n > n0;
#pragma unroll
            for (int x = 0; x < TERMS; ++x)
#pragma unroll
              for (int j = 0; j < BLK / 16; ++j)
                tc::mma_bf16_ts(tmem + kColO + 128u * t, tmem + kColS + 128u * t + 64u * b + (uint32_t)(x * (BLK / 2) + 8 * j),
                                vd + (uint64_t)(128 * j), idesc_o, acc || (x | j) != 0);
            tc::commit(o_done + 2 * t + (c & 1u));
            if (t) ++c1;
            else ++c0;
          }
          tc::commit(kv_empty + vs);
        }
      }
      tc::commit(drain);
      mbar_wait(drain, 0, nullptr);
    }
  } else if (warp >= 20) {
    // ---- e4m3 -> bf16: 8 threads per row, 16 rows at a time.  Eight lanes in a
    // row take half of rows r and r ^ 5: under both swizzles their 16-byte pieces
    // then fall into different banks, of the codes (rows that differ in bit 2)
    // and of the bf16 tile, where a lane has two (rows that differ in bit 0).
    if constexpr (E4M3) {
      reg_dealloc<Regs<E4M3>::kConvert>();
      const int w = (warp - 20) >> 2;  // K or V
      const int c = (lane & 3) | ((lane >> 1) & 4), j = 2 * (warp & 3) + (lane >> 4);
      const int r16 = ((j & 3) | ((j & 4) << 1)) ^ (lane & 4 ? 5 : 0);
      int n = 0;
      bool ok = true;
      while (ok && cur.next(a, sg)) {
        for (int i = sg.i0; ok && i < sg.i1; ++i, ++n) {
          const int kb0 = (i < sg.sb ? i : sg.wb0 + i - sg.sb) * BLK;
          // rows that no row of the pair sees become zeros, whatever they hold
          const bool edge = kb0 + BLK > sg.p1 + 1 || (kb0 < sg.lo && kb0 + BLK > sg.S);
          const int ks = (2 * n) % NS;
          const uint32_t use = (uint32_t)((2 * n) / NS);
          {
            const int rs = (2 * n + w) % NR;
            ok = mbar_wait(raw_full + rs, (uint32_t)((2 * n + w) / NR) & 1u, status);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            uint4 code[BLK / 16];
            uint32_t sc[BLK / 16];
#pragma unroll
            for (int s = 0; s < BLK / 16; ++s) {
              code[s] = lds128(raw + rs * Sh::kRaw + swz128(16 * s + r16, c));
              sc[s] = raw_scale[rs * BLK + 16 * s + r16];
            }
            if (edge) {
#pragma unroll
              for (int s = 0; s < BLK / 16; ++s) {
                const int tok = kb0 + 16 * s + r16;
                if (!(tok < sg.S || (tok >= sg.lo && tok <= sg.p1))) code[s] = make_uint4(0u, 0u, 0u, 0u);
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(raw_empty + rs);
            if (use > 0) ok = mbar_wait(kv_empty + ks + w, (use - 1) & 1u, status);
            if (!__all_sync(0xffffffffu, ok)) {
              ok = false;
              break;
            }
            unsigned char* dst = ring + (ks + w) * Sh::kSlot + (c >> 2) * Sh::kHalf;
#pragma unroll
            for (int s = 0; s < BLK / 16; ++s) {
              const int k = (int)sc[s] - 127;  // the row's scale is 2^k
              const uint32_t m1 = (uint32_t)(min(max(120 + k, -126), 127) + 127) << 7;
              const uint32_t m2 = m1 | (m1 << 16);
              uint2 o[4] = {bf16_of_codes(code[s].x, m2), bf16_of_codes(code[s].y, m2), bf16_of_codes(code[s].z, m2),
                            bf16_of_codes(code[s].w, m2)};
              if (120 + k > 127) {  // past bf16's largest power of two: in two steps
                const uint32_t e1 = (uint32_t)(k - 7 + 127) << 7, e2 = e1 | (e1 << 16);
#pragma unroll
                for (int y = 0; y < 4; ++y) o[y] = make_uint2(mul_bf16x2(o[y].x, e2), mul_bf16x2(o[y].y, e2));
              }
              const int r = 16 * s + r16;
              *reinterpret_cast<uint4*>(dst + swz128(r, 2 * (c & 3))) = make_uint4(o[0].x, o[0].y, o[1].x, o[1].y);
              *reinterpret_cast<uint4*>(dst + swz128(r, 2 * (c & 3) + 1)) = make_uint4(o[2].x, o[2].y, o[3].x, o[3].y);
            }
            fence_proxy_async();  // the tile before the tensor cores read it
            __syncwarp();
            if (lane == 0) mbar_arrive(kv_full + ks + w);
          }
        }
      }
    }
  } else {
    // ---- softmax of slot t, columns 32 half .. 32 half + 31 of a block
    reg_alloc<Regs<E4M3>::kSoftmax>();
    const int t = warp >> 3, half = (warp >> 2) & 1, quarter = warp & 3;
    const int id = 1 + 4 * t + quarter;  // barrier of the two warps that share rows
    const int r = 32 * quarter + lane;
    const int G = a.p.G, R = a.R;
    const int rr = r / G, hh = r - rr * G;
    const uint32_t lane_off = (uint32_t)(32 * quarter) << 16;
    const uint32_t ts = tmem + lane_off + kColS + 128u * t;
    const uint32_t to = tmem + lane_off + kColO + 128u * t + 64u * half;  // this thread's half of the dims
    const int window = a.p.window, sinks = a.p.sinks;
    const float sl2 = a.scale_log2;
    volatile float* xr = xchg + 128 * t + r;
    int n = 0, nx = 0;
    uint32_t cnt = 0;  // blocks this slot has done
    // After a wait has run out the warp goes through the same steps without
    // waiting, so that its partner never stands at their barrier alone.
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      if (!dead) dead = !__all_sync(0xffffffffu, mbar_wait(bar, parity, status));
    };
    while (cur.next(a, sg)) {
      const int row = (sg.single ? 0 : t * R) + rr;  // in the pair
      const bool vok = r < G * R && row < sg.rows;
      const int qpos = vok ? sg.p0 + row : -1;
      float mref = ninf, lh = 0.f;  // reference maximum (log2 units); this half's sum against it
      bool used = false;
      // Blocks that begin in [plain0, plain0 + plain_n) are seen whole by every
      // row of the pair.  With a scale that is not positive none counts as such.
      const int plain0 = window && sg.p1 >= window ? sg.p1 - window + 1 : 0;
      const unsigned plain_n = sl2 > 0.f ? (unsigned)max(0, sg.p0 + 2 - BLK - plain0) : 0u;
      for (int i = sg.i0; i < sg.i1; ++i, ++n) {
        if (sg.single && (n & 1) != t) continue;
        const int kb0 = (i < sg.sb ? i : sg.wb0 + i - sg.sb) * BLK;
        const uint32_t b = cnt % NB, tb = ts + 64u * b;
        wait(s_full + 2 * t + b, (cnt / NB) & 1u);
        tc::fence_after_sync();
        const bool plain = (unsigned)(kb0 - plain0) < plain_n && info[kInfo] == 0u;
        float sv[32], sum, mul;
        uint32_t p1[16];
        auto scores = [&] {
          {
            uint32_t q[32];
            tc::ld_32x32b_x32(tb + 32 * half, q);
            tc::wait_ld();
            tc::reg_fence(q);
#pragma unroll
            for (int x = 0; x < 32; ++x) sv[x] = __uint_as_float(q[x]);
          }
          mul = sl2;
          if (!plain) {
            const uint32_t bad = info[n % kInfo];
            // bit x: token kh0 + x is seen
            const int kh0 = kb0 + 32 * half;  // this thread's first token
            uint32_t see = first_bits(qpos - kh0 + 1);
            if (window) see &= ~first_bits(qpos - window - kh0 + 1) | first_bits(sinks - kh0);
            const uint32_t b2 = bad >> (2 * half);
            see &= ~((b2 & 1u ? 0x0000ffffu : 0u) | (b2 & 2u ? 0xffff0000u : 0u));
            mul = 1.f;
#pragma unroll
            for (int x = 0; x < 32; ++x) sv[x] = (see >> x) & 1u ? sv[x] * sl2 : ninf;
          }
        };
        auto weights = [&] {
          const float nmn = mref == ninf ? 0.f : -mref;  // nothing seen so far: every p is exp2(-inf) = 0
          unsigned long long rq[2] = {0ull, 0ull};       // partial sums, two values each
          const unsigned long long mul2 = pack_f2(mul, mul), nmn2 = pack_f2(nmn, nmn);
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            float e0, e1;
            unpack_f2(fma_f2(pack_f2(sv[2 * j], sv[2 * j + 1]), mul2, nmn2), e0, e1);
            e0 = fast_exp2(e0);
            e1 = fast_exp2(e1);
            rq[j & 1] = add_f2(rq[j & 1], pack_f2(e0, e1));
            p1[j] = pack_bf16(e0, e1);
            if (TERMS == 3) {  // what the first term leaves
              sv[2 * j] = e0 - bf16_lo(p1[j]);
              sv[2 * j + 1] = e1 - bf16_hi(p1[j]);
            }
          }
          float s0, s1, s2, s3;
          unpack_f2(rq[0], s0, s1);
          unpack_f2(rq[1], s2, s3);
          sum = (s0 + s1) + (s2 + s3);
        };
        if (used) {
          scores();
          weights();
        }
        // (a sum that is NaN because scores are does not ask for it, nor do lanes without a vector)
        if (!used || pair_any(id, vok && (sum > 0x1p20f || mref == ninf))) {
          // S is still in place: the scores need not be kept for this
          scores();
          // rare: the row's maximum over both halves, and what follows from it
          float mx = ninf;
#pragma unroll
          for (int x = 0; x < 32; ++x) mx = fmaxf(mx, sv[x]);
          if (mx != ninf) mx *= mul;
          if (half == 0) *xr = mx;
          pair_sync(id);
          if (half == 1) {
            mx = fmaxf(mx, *xr);
            *xr = mx;
          }
          pair_sync(id);
          if (half == 0) mx = *xr;
          const bool upd = mx > mref;
          const float alpha = !upd ? 1.f : (mref == ninf ? 0.f : fast_exp2(mref - mx));
          if (upd) mref = mx;
          lh *= alpha;
          if (used && __any_sync(0xffffffffu, upd)) {
            // O is at rest once the slot's last PV is done (the next waits for
            // P).  Of one parity the PV barrier is never two phases past this
            // wait: PV cnt + 1 needs the P that comes after it.
            wait(o_done + 2 * t + ((cnt - 1) & 1u), ((cnt - 1) >> 1) & 1u);
            tc::fence_after_sync();
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              uint32_t o[16];
              tc::ld_32x32b_x16(to + 16 * c, o);
              tc::wait_ld();
              tc::reg_fence(o);
#pragma unroll
              for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * alpha);
              tc::st_32x32b_x16(to + 16 * c, o);
            }
          }
          weights();
        }
        lh += sum;
        // P lies over S: the other half's scores have been read (pair_any, pair_sync)
        tc::st_32x32b_x16(tb + 16 * half, p1);
        if constexpr (TERMS == 3) {
#pragma unroll
          for (int x = 1; x < 3; ++x) {
#pragma unroll
            for (int j = 0; j < 16; ++j) {
              p1[j] = pack_bf16(sv[2 * j], sv[2 * j + 1]);
              sv[2 * j] -= bf16_lo(p1[j]);
              sv[2 * j + 1] -= bf16_hi(p1[j]);
            }
            tc::st_32x32b_x16(tb + 32 * x + 16 * half, p1);
          }
        }
        // bf16 tiles hold whatever the cache has at tokens that no row of the
        // pair sees: their V rows are zeroed before PV reads them
        if (!E4M3 && !plain && (kb0 + BLK > sg.p1 + 1 || (kb0 < sg.lo && kb0 + BLK > sg.S))) {
          const int vs = (2 * n) % NS + 1;
          wait(kv_full + vs, (uint32_t)((2 * n) / NS) & 1u);
          unsigned char* vt = ring + vs * Sh::kSlot;
          for (int x = 128 * half + r; x < BLK * 16; x += 256) {
            const int y = x >> 4, ch = x & 15, tok = kb0 + y;
            if (!(tok < sg.S || (tok >= sg.lo && tok <= sg.p1)))
              *reinterpret_cast<uint4*>(vt + (ch >> 3) * Sh::kHalf + swz128(y, ch & 7)) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async();
        }
        tc::wait_st();
        tc::fence_before_sync();  // P and the rescaled O before PV reads them
        __syncwarp();
        if (lane == 0) mbar_arrive(p_full + 2 * t + b);
        ++cnt;
        used = true;
      }
      // ---- the row's result: this thread's half of the dims; first the sum of
      // both halves of the tokens
      if (sg.nb > 0) {
        if (half == 0) *xr = lh;
        pair_sync(id);
        if (half == 1) {
          lh = *xr + lh;
          *xr = lh;
        }
        pair_sync(id);
        if (half == 0) lh = *xr;
        // (the maximum passes over NaN scores: where there was nothing else, the
        // merges would take the part for one that saw no token)
        if (lh != lh) mref = fmaxf(mref, 0.f);
      }
      if (used) {
        wait(o_done + 2 * t + ((cnt - 1) & 1u), ((cnt - 1) >> 1) & 1u);
        tc::fence_after_sync();
      }
      const bool whole = sg.i0 == 0 && sg.i1 == sg.nb;
      const bool merge = sg.single && sg.nb > 0;  // both slots have a part of the rows
      float f0 = 1.f, f1 = 0.f;                   // weights of this slot's and the other slot's result
      const float* other = nullptr;
      float* xpart = a.xbuf + (size_t)blockIdx.x * kChunkPart;
      if (merge && t == 1 && nx > 0) wait(x_empty, (nx - 1) & 1u);
      if (merge && t == 0) {
        wait(x_full, nx & 1u);
        const float2 ml = __ldcg(reinterpret_cast<const float2*>(xpart + kChunkMl + 2 * r));
        const float M = fmaxf(mref, ml.x);
        if (M != ninf) {
          f0 = fast_exp2(mref - M);
          f1 = fast_exp2(ml.x - M);
        }
        lh = lh * f0 + ml.y * f1;
        mref = M;
        other = xpart;
      }
      float* part = nullptr;  // where an unnormalised result goes
      if (merge && t == 1) {
        part = xpart;
      } else if (!whole) {
        part = a.parts + (((size_t)blockIdx.x * 2 + (sg.i0 == 0 ? 1 : 0)) * 2 + t) * kChunkPart;
      }
      const float inv = part ? 1.f : (lh != 0.f ? 1.f / lh : 0.f);
      const size_t orow = vok ? (size_t)(sg.row0 + row) * a.p.Hq + (size_t)sg.g * G + hh : 0;
      const bool mine = vok && !dead && !(sg.single && t == 1 && sg.nb == 0);  // (then slot 0 writes the zeros)
      f0 *= inv;
      f1 *= inv;
      float odd = 0.f;  // lanes that have some of vector 0: NaN if it has a result that is no number
      if (!part && !other) {
        // The usual end: straight to the output.  With a thread per row each
        // store instruction touches 32 lines; here lanes take 16 rows x 8 columns
        // each time, 4 lanes a row (four prompts: 224 -> 218 us).
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {  // rows 16 (c & 1) .., columns 32 (c >> 1) ..
          uint32_t q[16];
          if (used) {
            tc::ld_16x256b_x4(to + ((uint32_t)(16 * (c & 1)) << 16) + 32u * (c >> 1), q);
            tc::wait_ld();
            tc::reg_fence(q);
          } else {
#pragma unroll
            for (int x = 0; x < 16; ++x) q[x] = 0u;
          }
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // row lane / 4 + 8 y of the 16
            const int from = 16 * (c & 1) + 8 * y + (lane >> 2);
            const float f = __shfl_sync(0xffffffffu, f0, from);
            const bool on = __shfl_sync(0xffffffffu, (int)mine, from) != 0;
            const size_t ro = ((size_t)(uint32_t)__shfl_sync(0xffffffffu, (int)(orow >> 32), from) << 32) |
                              (uint32_t)__shfl_sync(0xffffffffu, (int)(uint32_t)orow, from);
            float o[8];  // columns 8 n + 2 (lane % 4), + 1
#pragma unroll
            for (int n = 0; n < 4; ++n) {
              o[2 * n] = __uint_as_float(q[4 * n + 2 * y]) * f;
              o[2 * n + 1] = __uint_as_float(q[4 * n + 2 * y + 1]) * f;
            }
            if (!E4M3 && y == 0 && !(c & 1) && quarter == 0 && lane < 4)
#pragma unroll
              for (int n = 0; n < 8; ++n) odd = fmaf(o[n], 0.f, odd);
            const int d0 = 64 * half + 32 * (c >> 1);
            if (a.p.out) {
              float* d = a.p.out + ro * kHeadDim + d0 + 2 * (lane & 3);
#pragma unroll
              for (int n = 0; n < 4; ++n)
                if (on) *reinterpret_cast<float2*>(d + 8 * n) = make_float2(o[2 * n], o[2 * n + 1]);
            } else {
              // 4 x 4 words across 4 lanes: lane l ends with the 8 columns of group n = l % 4
              uint32_t w[4];
#pragma unroll
              for (int n = 0; n < 4; ++n) w[n] = pack_bf16(o[2 * n], o[2 * n + 1]);
#pragma unroll
              for (int s = 1; s < 4; s <<= 1) {
                const bool up = lane & s;
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                  if (n & s) continue;
                  const uint32_t give = up ? w[n] : w[n | s];
                  const uint32_t got = __shfl_xor_sync(0xffffffffu, give, s);
                  if (up) w[n] = got;
                  else w[n | s] = got;
                }
              }
              if (on)
                *reinterpret_cast<uint4*>(a.p.out_bf16 + ro * kHeadDim + d0 + 8 * (lane & 3)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
          }
        }
      } else {
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t q[16];
        if (used) {
          tc::ld_32x32b_x16(to + 16 * c, q);
          tc::wait_ld();
          tc::reg_fence(q);
        } else {
#pragma unroll
          for (int x = 0; x < 16; ++x) q[x] = 0u;
        }
        float o[16];
#pragma unroll
        for (int x = 0; x < 16; ++x) o[x] = __uint_as_float(q[x]) * f0;
        const int d0 = 64 * half + 16 * c;
        // (parts lie by groups of 4 dims, rows within: a warp's accesses are whole lines)
        if (other) {
          float4 y[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) y[x] = __ldcg(reinterpret_cast<const float4*>(other) + (d0 / 4 + x) * 128 + r);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            o[4 * x] += y[x].x * f1;
            o[4 * x + 1] += y[x].y * f1;
            o[4 * x + 2] += y[x].z * f1;
            o[4 * x + 3] += y[x].w * f1;
          }
        }
        if (!E4M3 && r == 0)
#pragma unroll
          for (int x = 0; x < 16; ++x) odd = fmaf(o[x], 0.f, odd);
        if (mine) {
          if (part) {
#pragma unroll
            for (int x = 0; x < 4; ++x)
              reinterpret_cast<float4*>(part)[(d0 / 4 + x) * 128 + r] =
                  make_float4(o[4 * x], o[4 * x + 1], o[4 * x + 2], o[4 * x + 3]);
          } else if (a.p.out) {
            float* d = a.p.out + orow * kHeadDim + d0;
#pragma unroll
            for (int x = 0; x < 16; x += 4)
              *reinterpret_cast<float4*>(d + x) = make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
          } else {
            uint4* d = reinterpret_cast<uint4*>(a.p.out_bf16 + orow * kHeadDim + d0);
            d[0] = make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
            d[1] = make_uint4(pack_bf16(o[8], o[9]), pack_bf16(o[10], o[11]), pack_bf16(o[12], o[13]),
                              pack_bf16(o[14], o[15]));
          }
        }
      }
      }
      if (mine && half == 0) {
        if (part) *reinterpret_cast<float2*>(part + kChunkMl + 2 * r) = make_float2(mref, lh);
        else if (a.p.lse) a.p.lse[orow] = lh != 0.f ? mref * kLn2 + logf(lh) : ninf;
        if (sg.i0 == 0 && qpos < 0) flag_status(status, SA_ERR_DEVICE_CHECK);
      }
      if (!E4M3 && odd != 0.f) {
        atomicMin(&a.odd[blockIdx.x].from, sg.b);
        atomicMax(&a.odd[blockIdx.x].to, sg.b);
      }
      if (merge) {
        __threadfence_block();
        __syncwarp();
        if (lane == 0) mbar_arrive(t == 1 ? x_full : x_empty);
        ++nx;
      }
      tc::fence_before_sync();
      if (tid == 0 && !whole && sg.i0 == 0) {
        const int c = s_plan.cta_of(sg.w + sg.cost - 1);  // it holds the pair's last block
        a.recs[blockIdx.x] = ChunkRec{sg.row0, sg.rows, sg.g, c, sg.single ? 1 : 0};
      }
    }
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::fence_after_sync();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// What follows is for a bf16 cache with values that are no numbers in V rows that
// some rows of a pair see and others do not.

// Dims of this lane (a bit each; a warp, 4 dims a lane) in which the row at position
// p has lost its result to a value that it does not see, and would not have lost
// it to one that it sees.
SA_DEV uint32_t dims_to_take(const ChunkArgs& a, int b, int g, const Geom& q, int p) {
  const PagedView& kv = a.p.kv;
  const int window = a.p.window, sinks = a.p.sinks;
  // (and the first row's own token, which all see: with it a whole call of NaN needs nothing)
  const int before = window ? max(q.p1 - window + 1 - q.lo, 0) : 0, all = before + q.rows;
  uint32_t seen = 0u, others = 0u;
#pragma unroll 4
  for (int x = 0; x < all; ++x) {
    const int t = x < before ? q.lo + x : q.p0 + x - before;
    if (t < 0) continue;
    const int e = t / kv.page_size, page = __ldg(kv.table + (size_t)b * kv.max_pages + e);
    if (page < 0 || page >= kv.n_pages) continue;
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(kv.v + paged_offset(kv, page, g, t - e * kv.page_size)) +
                          (threadIdx.x & 31));
    // the top bits of halves with an exponent of 255
    const uint32_t x0 = ((w.x & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    const uint32_t x1 = ((w.y & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    const uint32_t dims = ((x0 >> 15) & 1u) | ((x0 >> 30) & 2u) | ((x1 >> 13) & 4u) | ((x1 >> 28) & 8u);
    if (t <= p && (!window || t > p - window || t < sinks)) seen |= dims;
    else others |= dims;
  }
  return others & ~seen;
}

// One more token of a softmax: score z (log2 units; -inf: not seen), D dims of its value.
template <int D>
SA_DEV void next_token(float z, const uint32_t (&v)[D / 2], float& m, float& l, float (&o)[D]) {
  const float ninf = -__int_as_float(0x7f800000);
  const float mn = fmaxf(m, z), f = mn == ninf ? 1.f : fast_exp2(m - mn);
  const float w = z == ninf ? 0.f : fast_exp2(z - mn);
  m = mn;
  l = l * f + w;
#pragma unroll
  for (int d = 0; d < D; d += 2) {
    o[d] = o[d] * f + (z == ninf ? 0.f : w * bf16_lo(v[d / 2]));
    o[d + 1] = o[d + 1] * f + (z == ninf ? 0.f : w * bf16_hi(v[d / 2]));
  }
}

// Row `row` of sequence b at position p, query head h: a warp, 4 dims a lane.
SA_DEV float4 again_vector(const ChunkArgs& a, int b, int row, int p, int h) {
  const PagedView& kv = a.p.kv;
  const int lane = threadIdx.x & 31, g = h / a.p.G;
  const float ninf = -__int_as_float(0x7f800000);
  const uint2 qw = *reinterpret_cast<const uint2*>(a.p.q + (size_t)row * a.p.q_row_stride + (size_t)h * kHeadDim + 4 * lane);
  const int lo = a.p.window && p >= a.p.window ? p - a.p.window + 1 : 0, first = min(a.p.window ? a.p.sinks : 0, lo);
  const int all = first + p + 1 - lo;
  float m = ninf, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int x0 = 0; x0 < all; x0 += 32) {  // 32 tokens: a lane looks up the place of one, then 4 at a time
    const int t = x0 + lane < first ? x0 + lane : lo + x0 + lane - first, e = t / kv.page_size;
    const int page = x0 + lane < all ? __ldg(kv.table + (size_t)b * kv.max_pages + e) : -1;
    const int slot = t - e * kv.page_size;
#pragma unroll 1
    for (int y = 0; y < min(32, all - x0); y += 4) {
      uint2 k[4], v[4];
      bool in[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int pg = __shfl_sync(0xffffffffu, page, y + u), sl = __shfl_sync(0xffffffffu, slot, y + u);
        in[u] = pg >= 0 && pg < kv.n_pages;
        const long long at = paged_offset(kv, in[u] ? pg : 0, g, in[u] ? sl : 0) + 8 * lane;
        k[u] = __ldg(reinterpret_cast<const uint2*>(kv.k + at));
        v[u] = __ldg(reinterpret_cast<const uint2*>(kv.v + at));
      }
      float z[4];
#pragma unroll
      for (int u = 0; u < 4; ++u)
        z[u] = bf16_lo(qw.x) * bf16_lo(k[u].x) + bf16_hi(qw.x) * bf16_hi(k[u].x) + bf16_lo(qw.y) * bf16_lo(k[u].y) +
               bf16_hi(qw.y) * bf16_hi(k[u].y);
#pragma unroll
      for (int s = 16; s > 0; s >>= 1)
#pragma unroll
        for (int u = 0; u < 4; ++u) z[u] += __shfl_xor_sync(0xffffffffu, z[u], s);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint32_t vu[2] = {v[u].x, v[u].y};
        next_token<4>(in[u] ? z[u] * a.scale_log2 : ninf, vu, m, l, o);
      }
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
  return make_float4(o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv);
}

// The 8 dims from 4 d4 of a lane's vector - row `row` of the cut pair that begins in
// row0, query head h of KV head g - where the merge of its parts gave some that are
// no numbers (a warp).
struct Dims8 {
  float4 o[2];
};
__device__ __noinline__ Dims8 again_parts(const ChunkArgs& a, int row0, int g, int row, int h, bool ok, int d4,
                                          Dims8 was) {
  const PagedView& kv = a.p.kv;
  const float ninf = -__int_as_float(0x7f800000);
  int b = 0, r0 = 0, m = 0;
  for (; b < kv.B; ++b) {  // the sequence that has the row
    m = paged_rows(a.p.row_off, a.p.n_rows, b, r0, nullptr);
    if (row0 >= r0 && row0 - r0 < m) break;
  }
  if (b == kv.B) return was;
  const int N = paged_tokens(kv, b, nullptr), lane = threadIdx.x & 31;
  const Geom q = pair_geom(a, N, m, (row0 - r0) / (2 * a.R));
  const int p = q.p0 + row;
  if (!(__ballot_sync(0xffffffffu, dims_to_take(a, b, g, q, -1) != 0u) & (3u << d4))) return was;  // (no value at all)
  uint32_t take = 0u;  // this lane's groups of 4 dims
  for (unsigned todo = __ballot_sync(0xffffffffu, ok); todo; todo &= todo - 1) {
    const int from = __ffs(todo) - 1;
    const unsigned dims =
        __ballot_sync(0xffffffffu, dims_to_take(a, b, g, q, __shfl_sync(0xffffffffu, p, from)) != 0u);
    if (lane == from) take = (dims >> d4) & 3u;
  }
  if (!__any_sync(0xffffffffu, take != 0u)) return was;
  // a lane has a vector: its query comes 8 dims at a time, keys and values are the same for all
  const uint4* qr = reinterpret_cast<const uint4*>(a.p.q + (size_t)(row0 + (ok ? row : 0)) * a.p.q_row_stride +
                                                   (size_t)(ok ? h : g * a.p.G) * kHeadDim);
  const int first = min(q.S, q.lo), all = first + q.p1 + 1 - q.lo;
  float mx = ninf, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int x0 = 0; x0 < all; x0 += 4) {
    long long at[4];
    bool see[4];
    float z[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int x = x0 + u, t = x < first ? x : q.lo + x - first, e = t / kv.page_size;
      const int page = x < all ? __ldg(kv.table + (size_t)b * kv.max_pages + e) : -1;
      see[u] = page >= 0 && page < kv.n_pages;
      at[u] = paged_offset(kv, see[u] ? page : 0, g, see[u] ? t - e * kv.page_size : 0);
      see[u] = see[u] && t <= p && (!a.p.window || t > p - a.p.window || t < a.p.sinks);
    }
#pragma unroll 1
    for (int c = 0; c < 16; ++c) {
      const uint4 qw = __ldg(qr + c);
      const uint32_t qv[4] = {qw.x, qw.y, qw.z, qw.w};
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const uint4 kw = __ldg(reinterpret_cast<const uint4*>(kv.k + at[u]) + c);
        const uint32_t kx[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
        for (int d = 0; d < 4; ++d) z[u] += bf16_lo(qv[d]) * bf16_lo(kx[d]) + bf16_hi(qv[d]) * bf16_hi(kx[d]);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4 vw = __ldg(reinterpret_cast<const uint4*>(kv.v + at[u] + 8 * d4));
      const uint32_t vv[4] = {vw.x, vw.y, vw.z, vw.w};
      next_token<8>(see[u] ? z[u] * a.scale_log2 : ninf, vv, mx, l, o);
    }
  }
  const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
  for (int x = 0; x < 2; ++x)
    if (take >> x & 1u) was.o[x] = make_float4(o[4 * x] * inv, o[4 * x + 1] * inv, o[4 * x + 2] * inv, o[4 * x + 3] * inv);
  return was;
}

// Rows of the pairs that were not cut, of the sequences that CTAs met results in
// that are no numbers (the whole grid, a warp at a time).
__device__ __noinline__ void again_rows(const ChunkArgs& a, int ctas) {
  const int lane = threadIdx.x & 31, warps = gridDim.x * (blockDim.x / 32);
  const int first = (threadIdx.x >> 5) * gridDim.x + blockIdx.x;
  for (int b = 0; b < a.p.kv.B; ++b) {
    int r0;
    const int m = paged_rows(a.p.row_off, a.p.n_rows, b, r0, nullptr), N = paged_tokens(a.p.kv, b, nullptr);
    bool met = false;
    for (int c = lane; c < ctas; c += 32) met |= a.odd[c].from <= b && b <= a.odd[c].to;
    if (m <= 0 || !__any_sync(0xffffffffu, met)) continue;
    for (long long x = first; x < (long long)m * a.p.Hq; x += warps) {
      const int i = (int)(x / a.p.Hq), h = (int)(x - (long long)i * a.p.Hq), g = h / a.p.G, j = i / (2 * a.R);
      const size_t at = ((size_t)(r0 + i) * a.p.Hq + h) * kHeadDim + 4 * lane;
      float4 o;
      if (a.p.out) {
        o = *reinterpret_cast<const float4*>(a.p.out + at);
      } else {
        const uint2 w = *reinterpret_cast<const uint2*>(a.p.out_bf16 + at);
        o = make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
      }
      if (!__any_sync(0xffffffffu, o.x * 0.f + o.y * 0.f + o.z * 0.f + o.w * 0.f != 0.f)) continue;
      bool cut = false;
      for (int c = lane; c < ctas; c += 32) cut |= a.recs[c].rows > 0 && a.recs[c].row0 == r0 + 2 * a.R * j && a.recs[c].g == g;
      if (__any_sync(0xffffffffu, cut)) continue;  // again_parts
      const uint32_t dims = dims_to_take(a, b, g, pair_geom(a, N, m, j), N - m + i);
      if (!__any_sync(0xffffffffu, dims != 0u)) continue;
      o = again_vector(a, b, r0 + i, N - m + i, h);
      if (!dims) continue;  // (the other dims stay as they are)
      if (a.p.out)
        *reinterpret_cast<float4*>(a.p.out + at) = o;
      else
        *reinterpret_cast<uint2*>(a.p.out_bf16 + at) = make_uint2(pack_bf16(o.x, o.y), pack_bf16(o.z, o.w));
    }
  }
}

// Merge of the partial results of the pairs that were cut: a warp's task is 32
// vectors (one per lane) and 8 dims of the pair that one CTA began, its parts in
// CTA order.  Tasks go round the grid, so that the few pairs of a short chunk
// over a long cache, in many parts each, use every SM.
constexpr int kCombineThreads = 256;
template <bool E4M3>
__global__ void __launch_bounds__(kCombineThreads) combine_kernel(const __grid_constant__ ChunkArgs a, int ctas) {
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float ninf = -__int_as_float(0x7f800000);
  const int G = a.p.G, R = a.R;
  bool met = false;  // rare: results that are no numbers
  if (!E4M3)
    for (int c = threadIdx.x; c < ctas; c += kCombineThreads) met |= a.odd[c].from <= a.odd[c].to;
  const int stride = gridDim.x * (kCombineThreads / 32);
  for (int task = warp * gridDim.x + blockIdx.x; task < ctas * 128; task += stride) {
    const int c0 = task >> 7;
    const ChunkRec rec = a.recs[c0];
    if (rec.rows <= 0) continue;
    const int v = ((task >> 4) & 7) * 32 + lane, d4 = (task & 15) * 2;  // vector; group of 4 dims
    const int t = v >> 7, r = v & 127;
    const int rr = r / G, row = t * R + rr;
    if (rec.single && t) continue;
    const bool ok = r < G * R && row < rec.rows;
    if (!__any_sync(0xffffffffu, ok)) continue;
    float M = ninf, L = 0.f;
    float4 o[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
    const int np = rec.last - c0 + 1;
    constexpr int kBatch = 8;
    for (int p0 = 0; p0 < np; p0 += kBatch) {
      float2 ml[kBatch];
      float4 y[kBatch][2];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int p = p0 + i;
        const bool in = p < np && ok;
        const float* src = a.parts + (((size_t)(c0 + (in ? p : 0)) * 2 + (!in || p == 0 ? 1 : 0)) * 2 + t) * kChunkPart;
        ml[i] = in ? __ldcg(reinterpret_cast<const float2*>(src + kChunkMl + 2 * r)) : make_float2(ninf, 0.f);
#pragma unroll
        for (int x = 0; x < 2; ++x)
          y[i][x] = in ? __ldcg(reinterpret_cast<const float4*>(src) + (d4 + x) * 128 + r) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float nm = M;
#pragma unroll
      for (int i = 0; i < kBatch; ++i) nm = fmaxf(nm, ml[i].x);
      if (nm == ninf) continue;
      const float f = fast_exp2(M - nm);
      L *= f;
#pragma unroll
      for (int x = 0; x < 2; ++x) o[x] = make_float4(o[x].x * f, o[x].y * f, o[x].z * f, o[x].w * f);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float w = fast_exp2(ml[i].x - nm);
        L += ml[i].y * w;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          o[x].x += y[i][x].x * w;
          o[x].y += y[i][x].y * w;
          o[x].z += y[i][x].z * w;
          o[x].w += y[i][x].w * w;
        }
      }
      M = nm;
    }
    const float inv = L != 0.f ? 1.f / L : 0.f;
    float odd = 0.f;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      o[x] = make_float4(o[x].x * inv, o[x].y * inv, o[x].z * inv, o[x].w * inv);
      odd += o[x].x * 0.f + o[x].y * 0.f + o[x].z * 0.f + o[x].w * 0.f;
    }
    if (!E4M3 && __any_sync(0xffffffffu, odd != 0.f)) {
      const Dims8 y = again_parts(a, rec.row0, rec.g, row, rec.g * G + r - rr * G, ok, d4, Dims8{{o[0], o[1]}});
      o[0] = y.o[0];
      o[1] = y.o[1];
    }
    if (!ok) continue;
    const size_t orow = (size_t)(rec.row0 + row) * a.p.Hq + (size_t)rec.g * G + (r - rr * G);
    if (a.p.out) {
      float4* d = reinterpret_cast<float4*>(a.p.out + orow * kHeadDim) + d4;
      d[0] = o[0];
      d[1] = o[1];
    } else {
      *reinterpret_cast<uint4*>(a.p.out_bf16 + orow * kHeadDim + 4 * d4) =
          make_uint4(pack_bf16(o[0].x, o[0].y), pack_bf16(o[0].z, o[0].w), pack_bf16(o[1].x, o[1].y), pack_bf16(o[1].z, o[1].w));
    }
    if (a.p.lse && d4 == 0) a.p.lse[orow] = L != 0.f ? M * kLn2 + logf(L) : ninf;
  }
  if (!E4M3 && __syncthreads_or(met)) again_rows(a, ctas);
}

template <bool E4M3, int TERMS>
cudaError_t launch(const ChunkArgs& a, int grid, cudaStream_t st) {
  auto* k = chunk_kernel<E4M3, TERMS>;
  constexpr int smem = Shape<TERMS>::smem(E4M3);
  static_assert(smem <= 227 * 1024, "shared memory of one CTA");
  const cudaError_t e = set_smem_attr((const void*)k, smem);
  if (e != cudaSuccess) return e;
  // The split waits for ever if it asks for more than the block was given.
  static const bool fits = [&] {
    cudaFuncAttributes at;
    return cudaFuncGetAttributes(&at, (const void*)k) == cudaSuccess && at.numRegs * Regs<E4M3>::kThreads >= Regs<E4M3>::kTotal;
  }();
  if (!fits) return cudaErrorInvalidConfiguration;
  return launch_pdl(k, (unsigned)grid, Regs<E4M3>::kThreads, smem, st, a);
}

}  // namespace

int chunk_block_tokens() { return BLK; }

cudaError_t launch_chunk(const ChunkArgs& a, int grid, cudaStream_t st) {
  const bool f32 = a.p.out != nullptr;
  const cudaError_t e = a.p.kv.e4m3 ? (f32 ? launch<true, 3>(a, grid, st) : launch<true, 1>(a, grid, st))
                                    : (f32 ? launch<false, 3>(a, grid, st) : launch<false, 1>(a, grid, st));
  if (e != cudaSuccess) return e;
  return launch_pdl(a.p.kv.e4m3 ? combine_kernel<true> : combine_kernel<false>, (unsigned)grid * 4, kCombineThreads, 0, st, a,
                    grid);
}

}  // namespace sa
