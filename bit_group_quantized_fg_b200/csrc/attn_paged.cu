// Attention of one query token per sequence over the paged 4-bit cache (include/fg.h,
// fg_paged_attention): out = sum_t softmax_t(q K_t / sqrt(hd)) V_t over the visible positions,
// K_t = mn + c s per group of G dims, several query heads per key/value head.
//
// HBM bounds it: a position costs hd + 8 hd/G bytes per key/value head and 4 hd flops per query
// head, so the cache is read once, and the work per byte that the issue slots can afford is what
// the layout below is made for.  A unit of work is a tile of 64 positions of one (sequence, key/value
// head); the units of the whole batch, in order, are divided evenly over the warps of the GPU
// (each warp a run of consecutive tiles, whatever the lengths), every warp streaming its run
// through a shared-memory ring of its own with bulk copies (one each for the codes and the
// parameters of K and V, per page the tile lies in) and merging nothing with other warps.  A
// context that several warps share leaves partial (max, sum, acc) results that a second kernel
// joins.
//
// Both products run on mma.sync m16n8k16 (a key/value head has few query rows, so a tcgen05 tile
// would be nearly empty): scores D = K_codes q with 16 positions as rows, values E = V_codes^T w
// with 16 dims as rows.  A 4-bit code is a valid fp16 operand as it is: the bits 0..15 of the
// mantissa of a subnormal number are c 2^-24, exactly, so a pair of codes is one AND of the packed
// word (codes in bits 4-7 of a half are 16 c 2^-24; the factor goes into q or the epilogue).  No
// offset has to be taken off again.  The parameters are applied in fp32:
//   score_t = sum_n s_tn D_tn + mn_tn (sum_{d in n} q_d),
//   out_d = sum_t (p_t s_tn) c_td + sum_t p_t mn_tn,   n the group of d,
// with q scaled by a power of two so that its largest value is near 2^12, and the weights p_t s_tn
// rounded to fp16 relative to a power of two near the largest s of the group that the warp has seen (2^-11 of
// each weight down to 2^-14 of that reference, 2^-25 of the reference below; both scalings are exact).  What a
// weight's rounding took off is added back in fp32 with the mean code 7.5
// (a part of the sum over mn), so that the rounding counts against c - 7.5, not against c: on the larger cases
// the error drops from 2.7 to 1.5 times that of the output's own rounding.  The softmax is fp32 with exp2; the running maximum of a row is raised only
// when a score passes it by more than 2^8, so the usual tile needs one vote.
//
// The 8 columns of an MMA hold the RW query rows 8 / RW times over.  Every column of a row then has
// the same scores, and the lanes of copy i keep those of the 16-position block i: one pass of the
// softmax serves 8 / RW blocks (4 for a single row, whose lanes hold two positions), and the value
// product of block i takes the weights in the columns of copy i and zeros elsewhere.  The copies
// are added up at the end of a context.
//
// Measured: 256 sequences of 543 positions, 56 heads of 128 (784 MB): 165 to 176 us on different GPUs, 4.5 TB/s, 69 % of a
// copy's rate; 8 sequences of 32k, 32 query heads on 8 (194 MB): 53 us; 48 sequences that see 4096
// positions, 32 on 4 (117 MB): 50 us; 1 sequence of 700, 12 heads of 64: 10 us, two launches.  No unit
// is saturated.  In the first case (930 instructions per tile of 64 positions) DRAM is 72 % busy, the integer
// pipe, which takes the codes apart, 58 %, the issue slots 52 %, with 10 warps per SM to hide the rest; in the
// third (1790 instructions per tile: a softmax pass per 16 positions, four groups per head) the issue slots 48 %, the
// integer pipe 33 %, with 7 warps per SM.
#include <algorithm>

#include "paged_common.cuh"
#include "sm100.cuh"

namespace fg {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTP = 64;  // positions per tile: 4 blocks of 16
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kUnset = 536870912.f;  // 2^29, before any value scale was seen: the smallest one in fp16, 2^-24, passes 16 with it
constexpr float kMid = 7.5f;  // the mean code, which what the rounding of a weight takes off is given back with

// CTAs per SM, a matter of room alone: registers allow 2 with 16 query rows, 3 below; shared memory 3 up to tiles of 9216 bytes
constexpr int ctas_of(int rows, int slot) { return rows == 16 || slot > 9216 ? 2 : 3; }

template <int HD, int G, int RW, int NT>
struct Cfg {
  static constexpr int NG = HD / G;           // groups of a head
  static constexpr int ROWS = RW * NT;        // query rows of an item: NT tiles of 8 columns
  static constexpr int NB = RW == 1 ? 4 : 8 / RW;  // blocks that share a pass of the softmax
  static constexpr int WPG = G / 32;          // K words a lane holds of a row's group
  static constexpr int MPG = G / 16;          // 16-dim tiles of a group
  static constexpr int RC = HD / 2, RP = NG * 4;                  // row bytes
  static constexpr int oV = kTP * RC, oKP = 2 * kTP * RC, oVP = oKP + kTP * RP;
  static constexpr int SLOT = oVP + kTP * RP;                     // bytes of a tile
  static constexpr int DEPTH = 2;                                 // tiles in a warp's ring
  static constexpr int kSmem = kWarps * DEPTH * SLOT + 128;       // + alignment
  static constexpr int CTAS = ctas_of(ROWS, SLOT);                // resident CTAs per SM
};

// What a sequence's query sees: positions [lo, n) and [0, sk); its tiles, `st` of them sinks.
struct Seq {
  int n, lo, sk, st, lot, T;
};
__device__ __forceinline__ Seq seq_of(const PagedView& c, const int32_t* lens, int b, int window, int n_sink) {
  Seq s;
  s.n = max(0, min(__ldg(lens + b), int(c.max_pages) << c.page_shift));
  s.lo = window > 0 ? max(0, s.n - window) : 0;
  s.sk = min(n_sink, s.lo);
  s.lot = s.lo / kTP;
  s.st = min((s.sk + kTP - 1) / kTP, s.lot);
  s.T = s.st + (s.n + kTP - 1) / kTP - s.lot;
  return s;
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   sm100::smem_u32(dst)),
               "l"(src), "r"(bytes), "r"(sm100::smem_u32(bar))
               : "memory");
}
template <int N>
__device__ __forceinline__ void lds_words(const uint8_t* p, uint32_t (&w)[N]) {
  if constexpr (N == 1) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    w[0] = v.x;
    w[1] = v.y;
  } else {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    w[0] = v.x;
    w[1] = v.y;
    w[2] = v.z;
    w[3] = v.w;
  }
}

// A tile's entry in the ring, written by the warp that copies it.
struct __align__(16) Meta {
  int pos, flags, rem, h;  // rem: tiles of the same context that follow; h: (key/value head, row tile)
  int b, n, lo, sk;
};
// flags: bits 0-3 below, 4-6 blocks of 16 positions in the ring, from 16 on which lanes' pages are there
enum : int { kFirst = 1, kLast = 2, kBegun = 4, kFull = 8 };

struct Rec {
  int b, h, further, pad;  // a context that starts in this warp's run and goes on in `further` more
};

template <int HD, int G, int RW, int NT>
__global__ void __launch_bounds__(kThreads, (Cfg<HD, G, RW, NT>::CTAS))
    paged_attn_kernel(PagedView c, const __half* __restrict__ q, int64_t q_stride, const int32_t* __restrict__ lens, int rep,
                      int window, int n_sink, __half* __restrict__ out, float* __restrict__ part_acc,
                      float* __restrict__ part_ml, Rec* __restrict__ recs, int* __restrict__ err) {
  using C = Cfg<HD, G, RW, NT>;
  using namespace sm100;
  constexpr int NG = C::NG, NB = C::NB, ROWS = C::ROWS, WPG = C::WPG, MPG = C::MPG, DEPTH = C::DEPTH;
  constexpr int RE = RW == 1 ? 1 : 2;  // query rows of a lane in a column tile
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_raw + ((128 - (smem_u32(smem_raw) & 127)) & 127);
  __shared__ __align__(8) uint64_t bars[kWarps][DEPTH];
  __shared__ Meta metas[kWarps][DEPTH];
  __shared__ int64_t pre[kThreads + 1];
  __shared__ int64_t wsum[kWarps];
  __shared__ int wmax[kWarps];
  __shared__ int abort_flag;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q4 = lane & 3;
  const int n_rt = (rep + ROWS - 1) / ROWS, H = c.nkv * n_rt;
  const int64_t h_all = int64_t(c.nkv) * rep * HD;
  if (lane < DEPTH) mbar_init(&bars[warp][lane], 1);
  if (tid == 0) abort_flag = 0;
  fence_barrier_init();
  pdl_wait();  // the previous kernel in the stream has finished (see fg_launch)

  // ---- units before every thread's share of the sequences; the longest context
  const int per = (c.B + kThreads - 1) / kThreads;
  int64_t mine = 0;
  int tmax = 0;
  for (int i = 0; i < per; ++i) {
    const int b = tid * per + i;
    if (b >= c.B) break;
    const int T = seq_of(c, lens, b, window, n_sink).T;
    mine += int64_t(T) * H;
    tmax = max(tmax, T);
  }
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t t = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += t;
    tmax = max(tmax, __shfl_xor_sync(0xffffffffu, tmax, o));
  }
  if (lane == 31) wsum[warp] = incl;
  if (lane == 0) wmax[warp] = tmax;
  __syncthreads();
  int64_t base = 0;
  for (int w = 0; w < warp; ++w) base += wsum[w];
  pre[tid] = base + incl - mine;
  if (tid == kThreads - 1) pre[kThreads] = base + incl;
  __syncthreads();
  const int64_t N = pre[kThreads];
  tmax = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
  // sequences that see nothing
  for (int b = blockIdx.x; b < c.B; b += gridDim.x) {
    if (seq_of(c, lens, b, window, n_sink).T == 0)
      for (int64_t i = tid; i < h_all / 8; i += kThreads)
        reinterpret_cast<uint4*>(out + int64_t(b) * h_all)[i] = make_uint4(0, 0, 0, 0);
  }

  // ---- this warp's run of units; neighbouring runs on different SMs
  const int worker = warp * gridDim.x + blockIdx.x, workers = kWarps * gridDim.x;
  // A long context alone: every warp more that shares it is a partial more for the joining kernel (ROWS hd floats), so
  // a run gets longer with the square root of the context.  One context of 64k, 8 heads of 4 rows: 48 us with 256
  // warps each, 52 us with 64; 4 heads of 8 rows: 49 us with 128, 57 us with 64, but at 8k 35 us with 128, 28 us with 64.
  const int q_min = int(ceilf(sqrtf(float(tmax) * (ROWS >= 8 ? 1.f / 16 : 1.f / 64))));
  const int64_t Q = max((N + workers - 1) / workers, int64_t(q_min));
  const int64_t u0 = int64_t(worker) * Q;
  if (lane == 0) recs[worker].further = 0;
  if (u0 >= N) return;
  const int cnt = int(min(Q, N - u0));

  // ---- the copying side: the tile to copy next
  int i_b, i_h, i_t;
  Seq i_s;
  {
    int below = 0;  // threads whose share starts at or before u0
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) below += __popc(__ballot_sync(0xffffffffu, pre[lane + 32 * i] <= u0));
    int64_t left = u0 - pre[below - 1];
    i_b = (below - 1) * per;
    for (;;) {  // 32 sequences at a time
      const int b = i_b + lane;
      const int64_t un = b < c.B ? int64_t(seq_of(c, lens, b, window, n_sink).T) * H : 0;
      int64_t s = un;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, s > left);
      if (hit) {
        const int l = __ffs(hit) - 1;
        left -= __shfl_sync(0xffffffffu, s - un, l);
        i_b += l;
        break;
      }
      left -= __shfl_sync(0xffffffffu, s, 31);
      i_b += 32;
      if (i_b >= c.B) return;  // lengths that changed meanwhile: nothing to do
    }
    i_s = seq_of(c, lens, i_b, window, n_sink);
    i_h = int(left / i_s.T);
    i_t = int(left - int64_t(i_h) * i_s.T);
  }
  int issued = 0;
  // lane 4 * piece + kind copies the K codes, V codes, K or V parameters of one page's part of the tile
  const int kind = lane & 3, piece = lane >> 2, psize = min(1 << c.page_shift, kTP);
  const bool copies = piece < kTP / psize;
  const int rb = kind < 2 ? C::RC : C::RP;
  const uint8_t* src0 = kind == 0   ? c.kc
                        : kind == 1 ? c.vc
                        : kind == 2 ? reinterpret_cast<const uint8_t*>(c.kp)
                                    : reinterpret_cast<const uint8_t*>(c.vp);
  const uint32_t head_bytes = uint32_t(rb) << c.page_shift;
  const int64_t page_bytes = int64_t(head_bytes) * c.nkv;
  uint8_t* const dst0 = ring + warp * DEPTH * C::SLOT + (kind == 0 ? 0 : kind == 1 ? C::oV : kind == 2 ? C::oKP : C::oVP) +
                        piece * psize * rb;
  auto tile_pos = [&]() { return (i_t < i_s.st ? i_t : i_s.lot + i_t - i_s.st) * kTP; };
  auto page_of = [&](int pos) {  // the page of this lane's part of the tile; -1: not there
    const int pi = (pos + piece * psize) >> c.page_shift;
    int p = -1;
    if (copies && pi < c.max_pages) p = __ldg(c.table + int64_t(i_b) * c.max_pages + pi);
    return p < c.n_pages ? p : -1;
  };
  int i_pos = tile_pos();
  int i_page = page_of(i_pos);
  auto issue = [&](int sl) {
    const int blocks = min(kTP / 16, (i_s.n - i_pos + 15) >> 4);  // only those that hold a cached position
    const int rows = min(psize, blocks * 16 - piece * psize);
    const bool ok = copies && i_page >= 0 && rows > 0;
    const uint32_t bytes = ok ? uint32_t(rows * rb) : 0u;
    const uint32_t total = __reduce_add_sync(0xffffffffu, bytes);
    const unsigned there = __ballot_sync(0xffffffffu, i_page >= 0) & 0x1111u;  // bits 0, 4, 8, 12
    if (lane == 0) {
      const int rem = i_s.T - 1 - i_t;
      const bool full = i_pos + kTP <= i_s.n && (i_pos >= i_s.lo || i_pos + kTP <= i_s.sk) && total == uint32_t(C::SLOT);
      const int flags = (issued == 0 || i_t == 0 ? kFirst : 0) | (issued == cnt - 1 || rem == 0 ? kLast : 0) |
                        (i_t <= issued ? kBegun : 0) | (full ? kFull : 0) | (blocks << 4) | int(there << 16);
      int4* md = reinterpret_cast<int4*>(&metas[warp][sl]);
      md[0] = make_int4(i_pos, flags, rem, i_h);
      md[1] = make_int4(i_b, i_s.n, i_s.lo, i_s.sk);
      mbar_expect_tx(&bars[warp][sl], total);
    }
    __syncwarp();  // the barrier expects its bytes before the first of them can land
    if (ok) {
      const int in_page = (i_pos + piece * psize) & ((1 << c.page_shift) - 1);
      const uint8_t* src = src0 + i_page * page_bytes + (uint64_t(uint32_t(NT == 1 ? i_h : i_h / n_rt)) * head_bytes + uint32_t(in_page * rb));
      bulk_load(dst0 + sl * C::SLOT, src, bytes, &bars[warp][sl]);
    }
    // on to the next tile, whose page is looked up here, an iteration before its copy
    if (++issued < cnt) {
      if (++i_t == i_s.T) {
        i_t = 0;
        if (++i_h == H) {
          i_h = 0;
          do {
            ++i_b;
            i_s = seq_of(c, lens, min(i_b, c.B - 1), window, n_sink);
          } while (i_s.T == 0 && i_b < c.B - 1);
          i_b = min(i_b, c.B - 1);
        }
      }
      i_pos = tile_pos();
      i_page = page_of(i_pos);
    }
  };
  for (int i = 0; i < DEPTH && i < cnt; ++i) issue(i);

  // ---- the computing side
  uint32_t qb[NT][HD / 16][2];        // q as B fragments: column g holds query row g % RW (of column tile nt)
  float kap[NT][RE], Qn[NT][RE][NG];  // per query row of this lane: factor of D, sums of q per group
  float m[NT][RE], mz[NT][RE], l[NT][RE], amn[NT][RE][NG], inv[NG], mid[NG];  // mz: m, or 0 where m is -inf
  float acc[NT][HD / 16][4];
  const int pA = (g >> 1) + 4 * (g & 1), pB = pA + 8;  // positions of D's rows g and g + 8 (see the V loads)
  const int copy = RW == 1 ? q4 : 2 * q4 / RW;         // the copy that this lane's columns belong to
  auto row_of = [&](int e) { return RW == 1 ? 0 : (2 * q4 + e) & (RW - 1); };

  int sl = 0;
  uint32_t ph = 0;
  for (int u = 0; u < cnt; ++u) {
    if (!__all_sync(0xffffffffu, mbar_wait(&bars[warp][sl], ph, &abort_flag, err, 0x10000))) {
      // give up: the copies still under way land (or their waits run out) before the warp leaves
      for (int v = u; v < issued; ++v) {
        mbar_wait_drain(&bars[warp][sl], ph);
        if (++sl == DEPTH) sl = 0, ph ^= 1;
      }
      return;
    }
    const uint8_t* st = ring + (warp * DEPTH + sl) * C::SLOT;
    const int4 m0 = *reinterpret_cast<const int4*>(&metas[warp][sl]);  // pos, flags, rem, h
    const int flags = m0.y, blocks = (flags >> 4) & 7;
    const int4 m1 = *(reinterpret_cast<const int4*>(&metas[warp][sl]) + 1);  // b, n, lo, sk
    if (flags & kFirst) {
      const int kvh = m0.w / n_rt, r0 = (m0.w - kvh * n_rt) * ROWS;
      const __half* qrow = q + int64_t(m1.x) * q_stride + (int64_t(kvh) * rep + r0) * HD;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int row = nt * RW + (g & (RW - 1));
        const bool ok = r0 + row < rep;
        uint4 w[HD / 32];
        float mx = 0.f, sum[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          sum[n] = 0.f;
#pragma unroll
          for (int i = 0; i < WPG; ++i) {
            uint4& x = w[n * WPG + i];
            x = ok ? __ldg(reinterpret_cast<const uint4*>(qrow + int64_t(row) * HD) + n * (G / 8) + q4 * WPG + i)
                   : make_uint4(0, 0, 0, 0);
            const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 f = __half22float2(u32_as_h2(xs[e]));
              mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
              sum[n] += f.x + f.y;
            }
          }
        }
#pragma unroll
        for (int o = 1; o < 4; o <<= 1) {
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
#pragma unroll
          for (int n = 0; n < NG; ++n) sum[n] += __shfl_xor_sync(0xffffffffu, sum[n], o);
        }
        // the power of two that brings the row's largest value to [2^12, 2^13)
        int ex = int((__float_as_uint(mx) >> 23) & 255) - 127;
        if (mx == 0.f || !(mx < INFINITY)) ex = 12;
        const float f = __uint_as_float(uint32_t(12 - ex + 127) << 23), finv = __uint_as_float(uint32_t(ex - 12 + 127) << 23);
        const float sc = kLog2e * rsqrtf(float(HD));
#pragma unroll
        for (int i = 0; i < HD / 32; ++i) {
          const uint32_t xs[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
          uint32_t ys[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // even dims at f, odd ones (codes 16 times as large) at f / 16
            const float2 v = __half22float2(u32_as_h2(xs[e]));
            ys[e] = h2_as_u32(__floats2half2_rn(v.x * f, v.y * (f * 0.0625f)));
          }
          qb[nt][2 * i][0] = __byte_perm(ys[0], ys[2], 0x5410);
          qb[nt][2 * i][1] = __byte_perm(ys[0], ys[2], 0x7632);
          qb[nt][2 * i + 1][0] = __byte_perm(ys[1], ys[3], 0x5410);
          qb[nt][2 * i + 1][1] = __byte_perm(ys[1], ys[3], 0x7632);
        }
#pragma unroll
        for (int e = 0; e < RE; ++e) {
          const int src = row_of(e) * 4;
          kap[nt][e] = __shfl_sync(0xffffffffu, finv, src) * (16777216.f * sc);
#pragma unroll
          for (int n = 0; n < NG; ++n) Qn[nt][e][n] = __shfl_sync(0xffffffffu, sum[n], src) * sc;
          m[nt][e] = -INFINITY;
          mz[nt][e] = 0.f;
          l[nt][e] = 0.f;
#pragma unroll
          for (int n = 0; n < NG; ++n) amn[nt][e][n] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < HD / 16; ++i) acc[nt][i][0] = acc[nt][i][1] = acc[nt][i][2] = acc[nt][i][3] = 0.f;
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) inv[n] = kUnset, mid[n] = kMid / kUnset;
    }

#pragma unroll
    for (int b0 = 0; b0 < kTP / 16; b0 += NB) {
      // ---- scores of NB blocks: this lane keeps those of block b0 + copy, sc[nt][e + 2 (position 8 further)]
      float sc[NT][4], sv[2][NG], mv[2][NG];
      {
        float d[NT][NG][4];
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const uint8_t* kr = st + (b0 + i) * 16 * C::RC;
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            uint32_t wA[WPG], wB[WPG];
            lds_words(kr + pA * C::RC + 4 * (n * (G / 8) + q4 * WPG), wA);
            lds_words(kr + pB * C::RC + 4 * (n * (G / 8) + q4 * WPG), wB);
            float x[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
#pragma unroll
            for (int j = 0; j < WPG; ++j) {
              const uint32_t a = wA[j], b = wB[j], a8 = a >> 8, b8 = b >> 8;
              constexpr uint32_t kLo = 0x000F000Fu, kHi = 0x00F000F0u;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const int ks = 2 * (n * WPG + j);
                mma16816(x[nt], a & kLo, b & kLo, a & kHi, b & kHi, qb[nt][ks][0], qb[nt][ks][1]);
                mma16816(x[nt], a8 & kLo, b8 & kLo, a8 & kHi, b8 & kHi, qb[nt][ks + 1][0], qb[nt][ks + 1][1]);
              }
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (e % 2 < RE && (i == 0 || copy == i)) d[nt][n][e] = x[nt][e];
          }
        }
        uint32_t kp[2][NG], vp[2][NG];
        const int mine = (b0 + (NB > 1 ? copy : 0)) * 16;
        lds_words(st + C::oKP + (mine + pA) * C::RP, kp[0]);
        lds_words(st + C::oKP + (mine + pB) * C::RP, kp[1]);
        lds_words(st + C::oVP + (mine + pA) * C::RP, vp[0]);
        lds_words(st + C::oVP + (mine + pB) * C::RP, vp[1]);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          float km[NG], ks[NG];
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            const float2 k = __half22float2(u32_as_h2(kp[x][n])), v = __half22float2(u32_as_h2(vp[x][n]));
            km[n] = k.x;
            ks[n] = k.y;
            mv[x][n] = v.x;
            sv[x][n] = v.y;
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int e = 0; e < RE; ++e) {
              float t = ks[0] * d[nt][0][2 * x + e], w = km[0] * Qn[nt][e][0];
#pragma unroll
              for (int n = 1; n < NG; ++n) {
                t = fmaf(ks[n], d[nt][n][2 * x + e], t);
                w = fmaf(km[n], Qn[nt][e][n], w);
              }
              sc[nt][2 * x + e] = fmaf(t, kap[nt][e], w);
            }
          }
        }
        if (!(flags & kFull)) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const int in_tile = mine + (x ? pB : pA), pos = m0.x + in_tile;
            const bool ok = pos < m1.y && (pos >= m1.z || pos < m1.w) && ((flags >> (16 + 4 * (in_tile >> min(c.page_shift, 6)))) & 1);
            if (!ok) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < RE; ++e) sc[nt][2 * x + e] = -INFINITY;
#pragma unroll
              for (int n = 0; n < NG; ++n) sv[x][n] = mv[x][n] = 0.f;
            }
          }
        }
      }

      // ---- raise the maximum of a row, or the reference of a group's value scales, where they fell behind
      float top[NT][RE], smax[NG];
      bool raise = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < RE; ++e) {
          top[nt][e] = fmaxf(sc[nt][e], sc[nt][2 + e]);
          raise |= top[nt][e] > m[nt][e] + 8.f;
        }
      }
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        smax[n] = fmaxf(fabsf(sv[0][n]), fabsf(sv[1][n]));
        raise |= smax[n] * inv[n] > 16.f;
      }
      if (__any_sync(0xffffffffu, raise)) {
#pragma unroll
        for (int n = 0; n < NG; ++n) {
#pragma unroll
          for (int o = 1; o < 32; o <<= 1) smax[n] = fmaxf(smax[n], __shfl_xor_sync(0xffffffffu, smax[n], o));
          if (smax[n] * inv[n] > 16.f && smax[n] < INFINITY) {  // the first scale above 0 always
            const float to = __uint_as_float((253u << 23) - (__float_as_uint(smax[n]) & 0x7f800000u));  // smax to [0.5, 1)
            const float r = to / inv[n];  // a power of two
            inv[n] = to;
            mid[n] = kMid / to;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < MPG; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[nt][n * MPG + i][e] *= r;
          }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int e = 0; e < RE; ++e) {
            float x = top[nt][e];
#pragma unroll
            for (int o = RW == 8 ? 4 : RW == 4 ? 2 : 1; o < 32; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
            if (x > m[nt][e] + 8.f) {
              const float r = ex2(m[nt][e] - x);  // 0 from -inf
              m[nt][e] = mz[nt][e] = x;
              l[nt][e] *= r;
#pragma unroll
              for (int n = 0; n < NG; ++n) amn[nt][e][n] *= r;
#pragma unroll
              for (int i = 0; i < HD / 16; ++i) {
                acc[nt][i][e] *= r;
                acc[nt][i][2 + e] *= r;
                if (RW == 1) {
                  acc[nt][i][1] *= r;
                  acc[nt][i][3] *= r;
                }
              }
            }
          }
        }
      }

      // ---- weights: row k of column g's fragment is w of position k (+ 8) of block g's copy
      uint32_t bw[NT][NG][2];
      {
        float si[2][NG];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int n = 0; n < NG; ++n) si[x][n] = sv[x][n] * inv[n];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float p[2][RE];
#pragma unroll
          for (int x = 0; x < 2; ++x) {
#pragma unroll
            for (int e = 0; e < RE; ++e) {
              p[x][e] = ex2(sc[nt][2 * x + e] - mz[nt][e]);
              l[nt][e] += p[x][e];
#pragma unroll
              for (int n = 0; n < NG; ++n) amn[nt][e][n] = fmaf(p[x][e], mv[x][n], amn[nt][e][n]);
            }
          }
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            if constexpr (RW == 1) {  // even columns: positions 0-7 of the block, odd ones: 8-15
              const float w0 = p[0][0] * si[0][n], w1 = p[1][0] * si[1][n];
              const __half2 h = __floats2half2_rn(w0, w1);
              const float2 f = __half22float2(h);
              amn[nt][0][n] = fmaf((w0 - f.x) + (w1 - f.y), mid[n], amn[nt][0][n]);
              bw[nt][n][0] = bw[nt][n][1] = transpose8x8(h2_as_u32(h));
            } else {
#pragma unroll
              for (int x = 0; x < 2; ++x) {
                const float w0 = p[x][0] * si[x][n], w1 = p[x][RE - 1] * si[x][n];
                const __half2 h = __floats2half2_rn(w0, w1);
                const float2 f = __half22float2(h);
                amn[nt][0][n] = fmaf(w0 - f.x, mid[n], amn[nt][0][n]);
                amn[nt][RE - 1][n] = fmaf(w1 - f.y, mid[n], amn[nt][RE - 1][n]);
                bw[nt][n][x] = transpose8x8(h2_as_u32(h));
              }
            }
          }
        }
      }
      // ---- values.  V: rows q4, q4 + 4, q4 + 8, q4 + 12 of the block are the positions 2q4, 2q4 + 1,
      // 2q4 + 8, 2q4 + 9 of the MMA (neighbouring lanes on neighbouring rows: two-way bank conflicts at most)
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        const uint8_t* vr = st + C::oV + ((b0 + i) * 16 + q4) * C::RC;
        const bool in0 = RW == 1 ? g == 2 * i : g / RW == i, in1 = RW == 1 ? g == 2 * i + 1 : g / RW == i;
#pragma unroll
        for (int n = 0; n < NG; ++n) {
          uint32_t w0[NT], w1[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            w0[nt] = NB == 1 || in0 ? bw[nt][n][0] : 0u;
            w1[nt] = NB == 1 || in1 ? bw[nt][n][1] : 0u;
          }
          constexpr int VW = G == 128 ? 2 : 1;  // words of a lane's G/8 dims; half a word for G = 32
          uint32_t v[4][VW];
#pragma unroll
          for (int r = 0; r < 4; ++r)
            lds_words(vr + 4 * r * C::RC + (n * G + (G == 32 ? (g >> 1) * 8 : g * (G / 8))) / 2, v[r]);
#pragma unroll
          for (int hw = 0; hw < (G == 32 ? 1 : 2 * VW); ++hw) {  // 16 bits (4 dims) of the four rows at a time
            const uint32_t sel = G == 32 ? ((g & 1) ? 0x7632u : 0x5410u) : ((hw & 1) ? 0x7632u : 0x5410u);
            const uint32_t x01 = __byte_perm(v[0][hw / 2], v[1][hw / 2], sel), x23 = __byte_perm(v[2][hw / 2], v[3][hw / 2], sel);
            const uint32_t y01 = x01 >> 8, y23 = x23 >> 8;
            constexpr uint32_t kLo = 0x000F000Fu, kHi = 0x00F000F0u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              mma16816(acc[nt][n * MPG + 2 * hw], x01 & kLo, x01 & kHi, x23 & kLo, x23 & kHi, w0[nt], w1[nt]);
              mma16816(acc[nt][n * MPG + 2 * hw + 1], y01 & kLo, y01 & kHi, y23 & kLo, y23 & kHi, w0[nt], w1[nt]);
            }
          }
        }
      }
      if (b0 + NB >= blocks) break;
    }
    __syncwarp();  // every lane has read the slot before it is refilled
    if (issued < cnt) issue(sl);
    if (++sl == DEPTH) sl = 0, ph ^= 1;

    if (flags & kLast) {
      // add up the copies and the lanes; lane: dims n*G + g*(G/8) .. + G/8 - 1 of every group n
      const bool begun = flags & kBegun, whole = begun && m0.z == 0;
      const int kvh = m0.w / n_rt, r0 = (m0.w - kvh * n_rt) * ROWS;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int e = 0; e < RE; ++e) {
#pragma unroll
          for (int o = RW == 8 ? 4 : RW == 4 ? 2 : 1; o < 32; o <<= 1) {
            l[nt][e] += __shfl_xor_sync(0xffffffffu, l[nt][e], o);
#pragma unroll
            for (int n = 0; n < NG; ++n) amn[nt][e][n] += __shfl_xor_sync(0xffffffffu, amn[nt][e][n], o);
          }
#pragma unroll
          for (int i = 0; i < HD / 16; ++i) {
            if (RW == 1) {
              acc[nt][i][0] += acc[nt][i][1];
              acc[nt][i][2] += acc[nt][i][3];
            }
#pragma unroll
            for (int o = RW == 4 ? 2 : 1; o < (RW == 8 ? 1 : 4); o <<= 1) {
              acc[nt][i][e] += __shfl_xor_sync(0xffffffffu, acc[nt][i][e], o);
              acc[nt][i][2 + e] += __shfl_xor_sync(0xffffffffu, acc[nt][i][2 + e], o);
            }
          }
          const int row = nt * RW + row_of(e);
          if (copy != 0 || r0 + row >= rep) continue;
          const float li = whole ? (l[nt][e] == 0.f ? 0.f : 1.f / l[nt][e]) : 1.f;  // 0: nothing was visible
          const int64_t ps = (int64_t(worker) * 2 + (begun ? 1 : 0)) * ROWS + row;
#pragma unroll
          for (int n = 0; n < NG; ++n) {
            const float ke = 16777216.f / inv[n], ko = 1048576.f / inv[n];  // 2^24, and 2^20 for codes 16 times as large
            float o[2 * MPG];
#pragma unroll
            for (int j = 0; j < MPG; ++j) {
              o[2 * j] = fmaf(acc[nt][n * MPG + j][e], ke, amn[nt][e][n]) * li;
              o[2 * j + 1] = fmaf(acc[nt][n * MPG + j][2 + e], ko, amn[nt][e][n]) * li;
            }
            const int d0 = n * G + g * (G / 8);
            if (whole) {
              uint2* dst = reinterpret_cast<uint2*>(out + int64_t(m1.x) * h_all + (int64_t(kvh) * rep + r0 + row) * HD + d0);
#pragma unroll
              for (int j = 0; j < MPG / 2; ++j)
                dst[j] = make_uint2(h2_as_u32(__floats2half2_rn(o[4 * j], o[4 * j + 1])),
                                    h2_as_u32(__floats2half2_rn(o[4 * j + 2], o[4 * j + 3])));
            } else {
              float4* dst = reinterpret_cast<float4*>(part_acc + ps * HD + d0);
#pragma unroll
              for (int j = 0; j < MPG / 2; ++j) dst[j] = make_float4(o[4 * j], o[4 * j + 1], o[4 * j + 2], o[4 * j + 3]);
            }
          }
          if (!whole && g == 0) {
            part_ml[ps * 2] = m[nt][e];
            part_ml[ps * 2 + 1] = l[nt][e];
          }
        }
      }
      if (begun && !whole && lane == 0) {
        Rec r;
        r.b = m1.x;
        r.h = m0.w;
        r.further = int((m0.z + Q - 1) / Q);
        r.pad = 0;
        recs[worker] = r;
      }
    }
  }
}

// Joins the partial results of the contexts that several warps shared, one CTA per context: the
// warp whose run it starts in (slot 1 of that warp) and the `further` ones after it (their slot 0).
// A few warps per query row, each with every WPR-th partial.
__host__ __device__ constexpr int join_warps(int rows) { return rows >= 8 ? 2 : rows == 4 ? 4 : 8; }  // per row
template <int HD, int ROWS>
__global__ void __launch_bounds__(32 * ROWS * join_warps(ROWS)) paged_join_kernel(int nkv, int rep,
                                                                                const float* __restrict__ part_acc,
                                                                                const float* __restrict__ part_ml,
                                                                                const Rec* __restrict__ recs,
                                                                                __half* __restrict__ out) {
  pdl_wait();  // the previous kernel in the stream has finished (see fg_launch)
  constexpr int WPR = join_warps(ROWS);
  constexpr int V = HD / 32;              // values per lane
  __shared__ float sh[ROWS * WPR][HD + 1];
  const Rec r = recs[blockIdx.x];
  if (r.further == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = warp / WPR, sub = warp % WPR;
  const int n_rt = (rep + ROWS - 1) / ROWS, kvh = r.h / n_rt, r0 = (r.h - kvh * n_rt) * ROWS;
  const int parts = r.further + 1;
  auto slot = [&](int i) { return (int64_t(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * ROWS + row; };
  float L = 0.f, acc[V];
#pragma unroll
  for (int j = 0; j < V; ++j) acc[j] = 0.f;
  if (r0 + row < rep) {
    float M = -INFINITY;
    for (int i = lane; i < parts; i += 32) M = fmaxf(M, part_ml[slot(i) * 2]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    if (M == -INFINITY) M = 0.f;  // nothing visible anywhere: every weight is 0
#pragma unroll 4
    for (int i = sub; i < parts; i += WPR) {
      const int64_t s = slot(i);
      const float w = ex2(part_ml[s * 2] - M);
      L = fmaf(part_ml[s * 2 + 1], w, L);
      if constexpr (V == 4) {
        const float4 a = *reinterpret_cast<const float4*>(part_acc + s * HD + lane * 4);
        acc[0] = fmaf(a.x, w, acc[0]);
        acc[1] = fmaf(a.y, w, acc[1]);
        acc[2] = fmaf(a.z, w, acc[2]);
        acc[3] = fmaf(a.w, w, acc[3]);
      } else {
        const float2 a = *reinterpret_cast<const float2*>(part_acc + s * HD + lane * 2);
        acc[0] = fmaf(a.x, w, acc[0]);
        acc[1] = fmaf(a.y, w, acc[1]);
      }
    }
#pragma unroll
    for (int j = 0; j < V; ++j) sh[warp][lane * V + j] = acc[j];
    if (lane == 0) sh[warp][HD] = L;
  }
  __syncthreads();
  if (sub != 0 || r0 + row >= rep) return;
#pragma unroll
  for (int w = 1; w < WPR; ++w) {
    L += sh[warp + w][HD];
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] += sh[warp + w][lane * V + j];
  }
  const float li = L == 0.f ? 0.f : 1.f / L;
  __half2* dst = reinterpret_cast<__half2*>(out + ((int64_t(r.b) * nkv + kvh) * rep + r0 + row) * HD + lane * V);
#pragma unroll
  for (int j = 0; j < V / 2; ++j) dst[j] = __floats2half2_rn(acc[2 * j] * li, acc[2 * j + 1] * li);
}

int rows_of(int rep) { return rep <= 2 ? rep : rep <= 4 ? 4 : rep <= 8 ? 8 : 16; }
int max_workers(int rows) { return num_sms() * (rows == 16 ? 2 : 3) * kWarps; }

}  // namespace

// Workspace: {acc [workers][2][rows][hd], (max, sum) [workers][2][rows], Rec [workers]}.
size_t paged_attention_ws_bytes(int nh, int nkv, int hd) {
  if (nh <= 0 || nkv <= 0 || nh % nkv || (hd != 64 && hd != 128)) return 0;
  const int rows = rows_of(nh / nkv);
  return size_t(max_workers(rows)) * (size_t(2 * rows) * (hd + 2) * sizeof(float) + sizeof(Rec));
}

namespace {

template <int HD, int G, int RW, int NT>
int launch(const PagedView& view, const __half* q, int64_t q_stride, const int32_t* lens, int rep, int window, int n_sink,
           __half* out, void* ws, cudaStream_t s) {
  using C = Cfg<HD, G, RW, NT>;
  constexpr int ROWS = C::ROWS;
  static_assert(C::CTAS <= (ROWS == 16 ? 2 : 3), "max_workers counts at least as many");
  static std::atomic<uint64_t> attr_done{0};
  FG_TRY(ensure_smem_attr(paged_attn_kernel<HD, G, RW, NT>, C::kSmem, attr_done));
  int* err = device_error_ptr();
  if (!err) return fail(FG_ERR_CUDA, "device error flag unavailable");
  // no more CTAs than the fullest cache has tiles (the lengths themselves are on the device)
  const int n_rt = (rep + ROWS - 1) / ROWS;
  const int64_t tiles = int64_t(view.B) * view.nkv * n_rt * (((int64_t(view.max_pages) << view.page_shift) + kTP - 1) / kTP);
  const int grid = int(std::min<int64_t>(num_sms() * C::CTAS, tiles));
  const int workers = grid * kWarps;
  float* acc = reinterpret_cast<float*>(ws);
  float* ml = acc + size_t(workers) * 2 * ROWS * HD;
  Rec* recs = reinterpret_cast<Rec*>(ml + size_t(workers) * 2 * ROWS * 2);
  FG_LAUNCH("paged attention kernel", (paged_attn_kernel<HD, G, RW, NT>), dim3(grid), dim3(kThreads), size_t(C::kSmem), s, view,
            q, q_stride, lens, rep, window, n_sink, out, acc, ml, recs, err);
  FG_LAUNCH("paged attention join kernel", (paged_join_kernel<HD, ROWS>), dim3(workers),
            dim3(32 * ROWS * join_warps(ROWS)), size_t(0), s, view.nkv, rep, acc, ml, recs, out);
  return FG_OK;
}

template <int HD, int G>
int launch_rows(const PagedView& view, const __half* q, int64_t q_stride, const int32_t* lens, int rep, int window,
                int n_sink, __half* out, void* ws, cudaStream_t s) {
  switch (rows_of(rep)) {
    case 1: return launch<HD, G, 1, 1>(view, q, q_stride, lens, rep, window, n_sink, out, ws, s);
    case 2: return launch<HD, G, 2, 1>(view, q, q_stride, lens, rep, window, n_sink, out, ws, s);
    case 4: return launch<HD, G, 4, 1>(view, q, q_stride, lens, rep, window, n_sink, out, ws, s);
    case 8: return launch<HD, G, 8, 1>(view, q, q_stride, lens, rep, window, n_sink, out, ws, s);
    default: return launch<HD, G, 8, 2>(view, q, q_stride, lens, rep, window, n_sink, out, ws, s);
  }
}

}  // namespace

int paged_attention_impl(const void* q, int64_t q_stride, const fg_paged_cache* c, const int32_t* lens, int nh,
                         int window, int n_sink, void* out, void* ws, size_t ws_bytes, cudaStream_t s) {
  FG_TRY(check_paged(c));
  if (!q || !lens || !out) return fail(FG_ERR_INVALID_ARG, "null pointer");
  if (nh <= 0 || nh % c->n_kv_heads) return fail(FG_ERR_SHAPE, "n_heads must be a multiple of n_kv_heads");
  if (n_sink < 0) return fail(FG_ERR_INVALID_ARG, "n_sink must not be negative");
  const int hd = c->head_dim, G = c->group;
  if (int64_t(nh) * hd > (1 << 24)) return fail(FG_ERR_SHAPE, "more than 2^24 query values a row");
  if (q_stride < int64_t(nh) * hd || q_stride % 8)
    return fail(FG_ERR_ALIGN, "q_stride must be >= n_heads * head_dim and a multiple of 8");
  if (!aligned16(q) || !aligned16(out)) return fail(FG_ERR_ALIGN, "q and out must be 16-byte aligned");
  if (!aligned4(lens) || !aligned4(c->page_table)) return fail(FG_ERR_ALIGN, "index arrays must be 4-byte aligned");
  const size_t need = paged_attention_ws_bytes(nh, c->n_kv_heads, hd);
  if (!ws || ws_bytes < need) return fail(FG_ERR_WORKSPACE, "paged attention needs %zu workspace bytes", need);
  if (!aligned16(ws)) return fail(FG_ERR_ALIGN, "workspace must be 16-byte aligned");
  ProfScope ps(PROF_DECODE_ATTN, s, 0.0, 4.0 * c->B * nh * hd);  // q and out; the lengths are on the device
  const PagedView view = paged_view(c);
  const int rep = nh / c->n_kv_heads;
  auto* Q = reinterpret_cast<const __half*>(q);
  auto* O = reinterpret_cast<__half*>(out);
  if (hd == 128 && G == 128) return launch_rows<128, 128>(view, Q, q_stride, lens, rep, window, n_sink, O, ws, s);
  if (hd == 128 && G == 64) return launch_rows<128, 64>(view, Q, q_stride, lens, rep, window, n_sink, O, ws, s);
  if (hd == 128) return launch_rows<128, 32>(view, Q, q_stride, lens, rep, window, n_sink, O, ws, s);
  if (G == 64) return launch_rows<64, 64>(view, Q, q_stride, lens, rep, window, n_sink, O, ws, s);
  return launch_rows<64, 32>(view, Q, q_stride, lens, rep, window, n_sink, O, ws, s);
}

}  // namespace fg
