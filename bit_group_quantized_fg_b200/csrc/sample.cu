// Sampling with temperature, top-k, top-p and min-p (include/fg.h, fg_sample).
//
// For a row of logits x, T > 0: w_i = exp((x_i - max x) / T), held as the integer
// rint(w_i * 2^44).  Sums of at most 2^18 of them fit 64 bits, so every sum is exact and the
// drawn token does not depend on the order of summation.  In the order of falling logit (ties
// by lowest id) top-k, top-p and min-p each keep a prefix; the kept set is the shortest one.
//
// Every token has a rank value of its own, its logit's order-preserving bits above its reversed
// id, so a prefix is "rank value >= cut".  A cut is found by a histogram of 2048 bins that are linear in
// the logit (of counts for top-k, of approximate fp32 weights for top-p), the exact weights above the bin it names,
// and the order of that bin's few tokens, which are counted out.  Should the exact sums say that the prefix
// ends in another bin, the search goes on with the approximate ones corrected by the difference.  A bin with
// more than 512 tokens becomes the range of the next histogram; logits that are all equal are binned by their
// ids.  So do the tokens behind the last bin whose weights the approximation still tells apart (2^-14 of the range's
// largest: one likely token and a top-p just above its probability): their histogram is relative to the largest of
// them, so a row takes four histograms and ten passes at most over the distributions tried (two passes usually), however far
// down the cut lies.
// The token is drawn by two levels of running sums in the order of the ids.
//
// What bounds it is instructions, not the 4 bytes of a logit: a row is read from HBM once and from L2 in
// the later passes (maximum; total weight, for top-p alone; histogram, with a shared-memory atomic per token; kept
// weights).  So the row is narrowed down early to a list of at most 4096 tokens per CTA, all those from some logit
// on, which the rest then works on:
//   top-k up to 512 (per CTA)  at least k tokens are as large as the smallest of the m-th largest maxima of each
//              warp's lanes, m warps' worth of k, which the first pass has at hand; no histogram of the row
//   others     what lies above the bin that the row's first histogram names, where that is few enough.
// Weights in 64 bits (~30 instructions) are computed for the tokens above a cut, gathered so that a warp computes 32 at a
// time, and for a whole row only where its sum is asked for (top-p without top-k, and no filter at all).
// Few rows are shared by a cluster of up to 8 CTAs, each with a range of the ids and a share of the bins, which
// exchange maxima, bins, sums and lists through distributed shared memory and all come to the same results.
//
// Logits of N(0, 1), calls back to back over 300 MB of them.  256 rows of 50272 (51 MB; copying them takes 8 us): 32 us
// with top-k 40, 39 us with top-k 40 and top-p 0.9, 39 us without a filter, 117 / 139 / 167 us with top-p 0.5 / 0.9 / 0.999,
// 14 us for the largest logit.  3 rows of 128001 on clusters of 8 CTAs: 25, 37, 14, 52 / 55 / 55 and 9 us.  With settings
// mixed by row a batch takes as long as its slowest kind of row (all 256 CTAs are resident at once, a row each): 105 to
// 132 us and 31 to 37 us, by which settings were drawn and by their logits.
#include <cooperative_groups.h>

#include <algorithm>

#include "fg_common.cuh"

namespace fg {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxVocab = 1 << 18;
constexpr int kBins = 2048;
constexpr int kList = 512;      // tokens of a bin that are ordered by counting
constexpr int kFirst = 16;      // loads in flight per thread in the first pass, which comes from HBM
constexpr int kCand = 4096;     // tokens of the list that a row is narrowed down to
constexpr int kTable = 256;     // steps of the exponential's table
constexpr int kUnroll = 8;
using u64 = unsigned long long;

// Order-preserving key of a logit; 0 for those that are never drawn (-inf, NaN).
__device__ __forceinline__ uint32_t key_of(float x) {
  if (!(x > -INFINITY)) return 0u;
  const uint32_t u = __float_as_uint(x == 0.f ? 0.f : x);  // -0 ties with +0
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}
__device__ __forceinline__ float logit_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xffffffffu));
}
// Rank value of a token: larger comes first.  0: never drawn.
__device__ __forceinline__ u64 rank_of(float x, int id) {
  const uint32_t k = key_of(x);
  return k ? (u64(k) << 18) | u64(kMaxVocab - 1 - id) : 0;
}

struct Shared {
  double table[kTable];       // 2^(i / 256)
  uint32_t hist[kBins];       // counts of the bins, or approximate weights in steps of 2^-20 of the largest considered (a
                              // bin of 4096 tokens near it wraps: the exact sums then correct the search)
  u64 list[kList];            // rank values of this CTA's tokens in a cut's bin
  u64 merged[kList];          // those of the whole row (their weights then take the place of `list`)
  u64 cand[kCand];            // rank values of the tokens of this CTA that may be kept
  float queue[kWarps][64];    // logits that wait for their weights
  u64 red[2][kWarps];
  u64 pair[2];                // two values of this CTA, for the others
  u64 out[2];
  uint32_t n_list, n_cand;
  int bin;
};

// Weights of a row's tokens as integers.
struct Weights {
  const double* table;
  float m;                  // the largest logit
  double md, c;             // m, log2(e) / T
  // 2^y for y = (x - m) log2(e) / T <= 0: 2^(k / 256) from the table times 2^r, |r| <= 2^-9, by the first terms of its
  // series (the first one left out is below 1.4e-13).  Rounded to a multiple of 2^-44 by adding 1.5 * 2^8 (whose last
  // mantissa bit is 2^-44).
  __device__ __forceinline__ u64 operator()(float x) const {
    if (m == INFINITY) return x == INFINITY ? u64(1) << 44 : 0;
    const double y = (double(x) - md) * c;
    if (!(y > -46.0)) return 0;  // below half a step, -inf and NaN
    const double t = y + 26388279066624.0;           // 1.5 * 2^44: a multiple of 2^-8
    const double r = y - (t - 26388279066624.0);
    const int k = int(uint32_t(__double2loint(t)));  // 256 y rounded, in two's complement
    double p = fma(r, 0.055504108664821580, 0.24022650695910071);  // (ln 2)^3 / 6, (ln 2)^2 / 2
    p = fma(p, r, 0.69314718055994531);                            // ln 2
    p = fma(p, r, 1.0);
    p *= table[k & (kTable - 1)];
    const double w = __hiloint2double(__double2hiint(p) + ((k >> 8) << 20), __double2loint(p));  // times 2^(k / 256)
    return u64(__double_as_longlong(w + 384.0)) - u64(0x4078000000000000ull);
  }
};

template <class T>
__device__ __forceinline__ T warp_sum(T v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
// Exclusive sums over the threads of the block (in thread order) and the total.
__device__ __forceinline__ u64 block_scan(u64 v, u64* red, u64& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  u64 s = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 t = __shfl_up_sync(0xffffffffu, s, o);
    if (lane >= o) s += t;
  }
  __syncthreads();
  if (lane == 31) red[warp] = s;
  __syncthreads();
  u64 before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w == warp) before = total;
    total += red[w];
  }
  return before + s - v;
}

// f(x, id) for the ids i0 .. i1 - 1 of the row, `step` ids apart from `first` on, kUnroll loads at a time.  Every lane of
// a warp makes the same calls (`on`: whether there is such an id).
template <int step, class F>
__device__ __forceinline__ void for_ids(const float* x, int i0, int i1, int first, F&& f) {
  for (int i = i0; i < i1; i += kUnroll * step) {
    float v[kUnroll];
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) {
      const int id = i + first + j * step;
      v[j] = id < i1 ? __ldg(x + id) : -INFINITY;
    }
#pragma unroll
    for (int j = 0; j < kUnroll; ++j) f(v[j], i + first + j * step);
  }
}

// Sum of the weights of gathered logits: 32 at a time.
struct Gather {
  float* queue;   // [64] of the warp
  int n = 0;
  u64 sum = 0;
  __device__ __forceinline__ void operator()(const Weights& weight, float v, bool take) {
    const unsigned mask = __ballot_sync(0xffffffffu, take);
    if (mask == 0) return;
    const int lane = threadIdx.x & 31;
    if (take) queue[n + __popc(mask & ((1u << lane) - 1u))] = v;
    n += __popc(mask);
    if (n >= 32) {
      __syncwarp();
      n -= 32;
      sum += weight(queue[n + lane]);
      __syncwarp();
    }
  }
  __device__ __forceinline__ u64 finish(const Weights& weight) {
    __syncwarp();
    if (int(threadIdx.x & 31) < n) sum += weight(queue[threadIdx.x & 31]);
    __syncwarp();
    n = 0;
    return sum;
  }
};

// A cluster of `ctas` CTAs per row.
template <int ctas>
__global__ void __launch_bounds__(kThreads, (ctas == 1 ? 2 : 1))
    sample_kernel(const float* __restrict__ logits, int64_t ld, int V, const float* __restrict__ temperature,
                  const int32_t* __restrict__ top_k, const float* __restrict__ top_p, const float* __restrict__ min_p,
                  const float* __restrict__ u, int32_t* __restrict__ tokens, float* __restrict__ logprob) {
  extern __shared__ __align__(16) uint8_t smem_raw[];
  Shared& sh = *reinterpret_cast<Shared*>(smem_raw);
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = ctas > 1 ? int(cluster.block_rank()) : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / ctas;
  const float* x = logits + int64_t(b) * ld;
  const int seg = (V + ctas - 1) / ctas, i0 = min(V, rank * seg), i1 = min(V, i0 + seg);
  if (tid < kTable) sh.table[tid] = exp2(double(tid) / kTable);
  pdl_wait();  // the previous kernel in the stream has finished (see fg_launch)
  auto sync = [&]() {
    if (ctas > 1) cluster.sync();
    else __syncthreads();
  };
  // f(value of `p` in CTA r) for every CTA r of the cluster
  auto of_all = [&](auto* p, auto&& f) {
#pragma unroll
    for (int r = 0; r < ctas; ++r) f(r, ctas > 1 ? *cluster.map_shared_rank(p, r) : *p);
  };
  // Combines two values over the row, in every thread of the cluster (fa and fb: sum, min or max).
  auto combine = [&](u64& va, u64& vb, auto&& fa, auto&& fb) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      va = fa(va, __shfl_xor_sync(0xffffffffu, va, o));
      vb = fb(vb, __shfl_xor_sync(0xffffffffu, vb, o));
    }
    __syncthreads();
    if (lane == 0) sh.red[0][warp] = va, sh.red[1][warp] = vb;
    __syncthreads();
    if (warp == 0) {
      va = sh.red[0][lane % kWarps];
      vb = sh.red[1][lane % kWarps];
#pragma unroll
      for (int o = kWarps / 2; o > 0; o >>= 1) {
        va = fa(va, __shfl_xor_sync(0xffffffffu, va, o));
        vb = fb(vb, __shfl_xor_sync(0xffffffffu, vb, o));
      }
      if (lane == 0) sh.pair[0] = va, sh.pair[1] = vb;
    }
    sync();
    of_all(&sh.pair[0], [&](int r, u64 v) { va = r ? fa(va, v) : v; });
    of_all(&sh.pair[1], [&](int r, u64 v) { vb = r ? fb(vb, v) : v; });
    sync();  // they have been read
  };
  auto larger = [](u64 p, u64 q) { return max(p, q); };
  auto smaller = [](u64 p, u64 q) { return min(p, q); };
  auto plus = [](u64 p, u64 q) { return p + q; };

  // ---- the first token of the row and its smallest drawable logit
  u64 best, lowest;
  float top = -INFINITY;  // of this thread's tokens
  {
    float low = INFINITY;
    int top_id = -1;
    for (int i = i0; i < i1; i += kFirst * kThreads) {
      float v[kFirst], m = -INFINITY;
#pragma unroll
      for (int j = 0; j < kFirst; ++j) {
        const int id = i + tid + j * kThreads;
        v[j] = id < i1 ? __ldg(x + id) : -INFINITY;
      }
#pragma unroll
      for (int j = 0; j < kFirst; ++j) {
        m = fmaxf(m, v[j]);
        low = fminf(low, v[j] > -INFINITY ? v[j] : INFINITY);
      }
      if (m > top) {  // the ids of a thread grow: of equal logits the first is kept
#pragma unroll
        for (int j = 0; j < kFirst; ++j)
          if (v[j] > top) top = v[j], top_id = i + tid + j * kThreads;
      }
    }
    best = top_id >= 0 ? rank_of(top, top_id) : 0;
    lowest = top_id >= 0 ? rank_of(low, 0) : ~u64(0);  // (its id does not matter)
  }
  combine(best, lowest, larger, smaller);

  const float T = temperature ? temperature[b] : 1.f;
  const int k = top_k ? top_k[b] : 0;
  const float p = top_p ? top_p[b] : 1.f;
  if (best == 0 || !(T > 0.f) || k == 1 || p <= 0.f) {  // nothing to draw, or the arg max
    if (rank == 0 && tid == 0) {
      tokens[b] = best == 0 ? 0 : kMaxVocab - 1 - int(best & (kMaxVocab - 1));
      if (logprob) logprob[b] = best == 0 ? -INFINITY : 0.f;
    }
    return;
  }
  Weights weight;
  weight.table = sh.table;
  weight.m = logit_of(uint32_t(best >> 18));
  weight.c = 1.4426950408889634 / double(T);
  weight.md = double(weight.m);
  Gather gather;
  gather.queue = sh.queue[warp];

  const bool do_k = k > 0 && k < V, do_p = p < 1.f;

  // ---- the tokens under consideration and their bins: logits x_hi .. x_lo, in steps of 1 / scale (kLinear) or of 2^shift
  // keys (kKeys: a range of few keys, or too narrow for a scale), or those equal to x_hi, in steps of 2^shift ids
  enum { kLinear, kKeys, kIds } by = kLinear;
  float x_hi = 0.f, x_lo = 0.f, scale = 0.f;
  int shift = 0;
  auto consider = [&](float high, float low) {
    x_hi = high;
    x_lo = low;
    const double range = double(high) - double(low);
    const uint32_t keys = key_of(high) - key_of(low);
    by = keys == 0 ? kIds : keys < kBins || range < 1e-30 ? kKeys : kLinear;
    scale = by == kLinear ? float((kBins - 1) / range) : 0.f;
    shift = 0;
    while (((by == kIds ? uint32_t(V - 1) : keys) >> shift) >= kBins) ++shift;
  };
  auto bin_at = [&](float v, int id) -> int {  // falling with v (for equal ones rising with the id); -1: not considered
    if (!(v <= x_hi && v >= x_lo)) return -1;
    if (by == kLinear) return int(fminf((x_hi - v) * scale, float(kBins - 1)));
    return by == kKeys ? int((key_of(x_hi) - key_of(v)) >> shift) : id >> shift;
  };
  // the weight in fp32, in steps of 2^-20 of that of x_hi: near enough to name a bin
  const float c32 = fminf(float(weight.c), 3.402823466e38f);  // finite: x_hi itself has 2^20 at any temperature
  auto rough = [&](float v) {
    float w;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(w) : "f"(fmaf(v - x_hi, c32, 20.f)));
    return weight.m == INFINITY ? uint32_t(v == INFINITY) << 20 : __float2uint_rn(w);
  };
  // f(logit, id) for the tokens of this CTA's list or ids.  Every lane of a warp makes the same calls.
  bool listed = false;
  int n_cand = 0;
  auto each = [&](auto&& f) {
    if (listed) {
      for (int i = 0; i < n_cand; i += kThreads) {
        const u64 c = i + tid < n_cand ? sh.cand[i + tid] : 0;
        f(c ? logit_of(uint32_t(c >> 18)) : -INFINITY, kMaxVocab - 1 - int(c & (kMaxVocab - 1)));
      }
    } else {
      for_ids<kThreads>(x, i0, i1, tid, f);
    }
  };
  // Lists the row's tokens from the logit `from` on, if they fit.
  auto list_from = [&](float from) {
    if (tid == 0) sh.n_cand = 0;
    __syncthreads();
    for_ids<kThreads>(x, i0, i1, tid, [&](float v, int id) {
      const bool take = v >= from && v > -INFINITY;
      const unsigned mask = __ballot_sync(0xffffffffu, take);
      if (mask == 0) return;
      uint32_t at = 0;
      if (lane == 0) at = atomicAdd(&sh.n_cand, uint32_t(__popc(mask)));
      at = __shfl_sync(0xffffffffu, at, 0) + __popc(mask & ((1u << lane) - 1u));
      if (take && at < kCand) sh.cand[at] = rank_of(v, id);
    });
    __syncthreads();
    if (tid == 0) sh.pair[0] = sh.n_cand;
    sync();
    listed = true;
    of_all(&sh.pair[0], [&](int, u64 n) { listed = listed && n <= kCand; });
    sync();  // they have been read
    n_cand = int(sh.n_cand);
  };
  // Every CTA adds up a share of the row's bins and keeps it in place: J bins per thread from b0 on.
  constexpr int kShare = kBins / ctas, J = kShare >= kThreads ? kShare / kThreads : 1;
  const int b0 = rank * kShare + tid * J;
  const bool has_bins = tid * J < kShare;
  auto fill = [&](bool by_n) {
    for (int i = tid; i < kBins; i += kThreads) sh.hist[i] = 0;
    sync();
    each([&](float v, int id) {
      if (!__any_sync(0xffffffffu, v >= x_lo)) return;
      const int bin = bin_at(v, id);
      if (bin >= 0) atomicAdd(&sh.hist[bin], by_n ? 1u : rough(v));
    });
    sync();
    if (ctas > 1) {
      uint32_t n[J] = {};
      if (has_bins) {
#pragma unroll
        for (int j = 0; j < J; ++j) of_all(&sh.hist[b0 + j], [&](int, uint32_t v) { n[j] += v; });
      }
      sync();  // every histogram has been read
      if (has_bins) {
#pragma unroll
        for (int j = 0; j < J; ++j) sh.hist[b0 + j] = n[j];
      }
      __syncthreads();
    }
  };

  // Counts or approximate weights before this thread's bins.
  auto before_bins = [&]() {
    u64 t = 0, total;
    if (has_bins) {
#pragma unroll
      for (int j = 0; j < J; ++j) t += sh.hist[b0 + j];
    }
    u64 pre = block_scan(t, sh.red[0], total);
    if (ctas > 1) {
      if (tid == 0) sh.pair[0] = total;
      sync();
      of_all(&sh.pair[0], [&](int r, u64 v) { pre += r < rank ? v : 0; });
      sync();  // they have been read
    }
    return pre;
  };
  // The first bin of first .. last with anything in it that satisfies enough(what comes before its end), or kBins.
  auto first_bin = [&](u64 pre, int first, int last, auto&& enough) {
    if (tid == 0) sh.bin = kBins;
    __syncthreads();
    if (has_bins) {
      u64 e = pre;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        e += sh.hist[b0 + j];
        if (sh.hist[b0 + j] && b0 + j >= first && b0 + j <= last && enough(e)) {
          atomicMin(&sh.bin, b0 + j);
          break;
        }
      }
    }
    sync();
    int bin = kBins;
    of_all(&sh.bin, [&](int, int v) { bin = min(bin, v); });
    sync();  // they have been read
    return bin;
  };
  // No logit below this lies in the bin or before it (a hundredth of a bin for the roundings).
  auto reach_of = [&](int bin) {
    return by == kLinear ? float(fmax(double(x_hi) - (bin + 1.01) / double(scale), double(x_lo))) : x_lo;
  };
  const float all = logit_of(uint32_t(lowest >> 18));

  // The rank value that the shortest prefix with need_n tokens (by_n) or a weight of need_w ends at, when it does not end
  // below the logit `low`; `reached`: the weight of that prefix (for top-p).  0 when the row has fewer tokens.
  auto cut_at = [&](bool by_n, u64 need_n, double need_w, float low, u64& reached) -> u64 {
    const uint32_t* hist = sh.hist;
    u64 above_n = 0, above_w = 0;                             // of the tokens that come before those considered
    consider(weight.m, weight.m == INFINITY ? weight.m : low);  // where there are +inf logits, only those
    fill(by_n);
    int list_bin = -1;  // the last bin whose tokens the list holds, where it was made here
    bool may_list = !listed && by == kLinear;
    for (;;) {
      // before this thread's bins: tokens of the row, or weights of those considered in the histogram's steps
      const u64 pre = before_bins() + (by_n ? above_n : 0);
      const double step = by_n ? 1.0 : double(weight(x_hi)) * 9.5367431640625e-07;  // 2^-20
      int first = 0, last = kBins - 1;                                            // the bin lies between these
      u64 done = above_w;                                                         // weight of what comes before `first`
      double fix = 0.0;                                                           // of the approximate weights
      u64 n_before = 0, a = 0, in = 0, n_in = 0;
      int bin = -1;
      bool behind = false;  // the cut lies behind the bins whose approximate weights say anything
      for (;;) {
        // the first bin that reaches what is needed, else the last with anything in it
        const double left = by_n ? 0.0 : (need_w - double(above_w) - fix) / step;
        bin = first_bin(pre, first, last, [&](u64 e) { return by_n ? e >= need_n : double(e) >= left; });
        if (bin == kBins) {
          if (by_n) return 0;
          if (tid == 0) sh.bin = -1;
          __syncthreads();
          if (has_bins) {
#pragma unroll
            for (int j = 0; j < J; ++j)
              if (hist[b0 + j] && b0 + j >= first && b0 + j <= last) atomicMax(&sh.bin, b0 + j);
          }
          sync();
          bin = -1;
          of_all(&sh.bin, [&](int, int v) { bin = max(bin, v); });
          if (bin < 0) {
            behind = first > 0;  // (the bin of x_hi is among those done: the next range is a smaller one)
            if (behind) break;
            bin = first;  // all sums wrapped to 0: the exact ones of the first bin say how to go on
          }
        }
        if (may_list) {
          // the tokens up to the bin (and the next one, for what is approximate), from their weights
          may_list = false;
          list_bin = bin + !by_n;
          u64 n = 0, none = 0;
          if (has_bins) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
              const uint32_t w = by_n ? 1u : rough(x_hi - float(b0 + j + 1) / scale);
              if (b0 + j <= list_bin) n += by_n ? hist[b0 + j] : w < 4 ? kMaxVocab : hist[b0 + j] / w;
            }
          }
          combine(n, none, plus, plus);
          if (n <= kCand * ctas) list_from(reach_of(list_bin));
          if (!listed) list_bin = -1;
        }
        if (list_bin >= 0 && bin > list_bin) listed = false, list_bin = -1;
        // what the histogram says comes before it
        if (has_bins && bin >= b0 && bin < b0 + J) {
          u64 e = pre;
          for (int j = 0; b0 + j < bin; ++j) e += hist[b0 + j];
          sh.out[0] = e;
        }
        if (tid == 0) sh.n_list = 0;
        sync();
        u64 e = 0;
        {
          const int owner = bin / kShare;
          of_all(&sh.out[0], [&](int r, u64 v) { e = r == owner ? v : e; });
        }
        if (by_n) n_before = e;
        // the exact weights before it and in it, and its rank values as far as the list takes them
        u64 mine = 0;
        gather.sum = 0;
        const float reach = reach_of(bin);
        each([&](float v, int id) {
          if (!__any_sync(0xffffffffu, v >= reach)) return;
          const int at = bin_at(v, id);
          if (at == bin) {
            const uint32_t i = atomicAdd(&sh.n_list, 1u);
            if (i < kList) sh.list[i] = rank_of(v, id);
            if (do_p) mine += weight(v);
          }
          if (do_p) gather(weight, v, at >= 0 && at < bin);
        });
        a = do_p ? gather.finish(weight) : 0;
        in = mine;
        __syncthreads();
        n_in = 0;
        if (do_p) combine(a, in, plus, plus);
        else sync();
        of_all(&sh.n_list, [&](int, uint32_t v) { n_in += v; });
        a += above_w;
        if (by_n) break;
        const bool back = double(a) >= need_w && bin_at(weight.m, 0) != bin && first < bin;
        const bool on = double(a + in) < need_w && bin < last;
        if (!back && !on) break;
        if (back) {
          last = bin - 1;
        } else {
          first = bin + 1;
          done = a + in;
          behind = double(in) < 64.0 * step * double(n_in);  // what follows weighs less than 64 steps a token
          if (behind) break;
        }
        fix = double(a - above_w) - double(e) * step;
        sync();  // the lists' lengths have been read
      }
      if (!behind) first = last = bin;
      if (list_bin >= 0 && last > list_bin) listed = false;
      above_w = behind ? done : a;
      above_n = n_before;
      list_bin = -1;
      if (!behind && n_in <= kList) break;
      // too many for the list, or too far down: the bin, or those that are left, become the range of the next histogram
      u64 mx = 0, mn = ~u64(0);
      each([&](float v, int id) {
        const int at = bin_at(v, id);
        if (at >= first && at <= last) {
          const u64 r = rank_of(v, id);
          mx = max(mx, r);
          mn = min(mn, r);
        }
      });
      combine(mx, mn, larger, smaller);
      consider(logit_of(uint32_t(mx >> 18)), logit_of(uint32_t(mn >> 18)));
      fill(by_n);
    }
    // the lists of the cluster, ordered by counting
    int n = 0;
    of_all(&sh.n_list, [&](int r, uint32_t n_r) {
      if (tid < int(n_r)) sh.merged[n + tid] = ctas > 1 ? *cluster.map_shared_rank(&sh.list[tid], r) : sh.list[tid];
      n += int(n_r);
    });
    sync();  // the lists have been read
    static_assert(kList <= kThreads, "one token per thread");
    u64 mine = 0, w = 0, before_w = above_w, before = above_n;
    if (tid < n) {
      mine = sh.merged[tid];
      w = do_p ? weight(logit_of(uint32_t(mine >> 18))) : 0;
      sh.list[tid] = w;
    }
    __syncthreads();
    if (tid < n) {
#pragma unroll 4
      for (int i = 0; i < n; ++i) {
        const bool ahead = sh.merged[i] > mine;
        before += ahead;
        before_w += ahead ? sh.list[i] : 0;
      }
      // the prefix ends at the first token with which it reaches what is needed; it has one token at least
      if (by_n ? before + 1 == need_n
               : double(before_w + w) >= need_w && (mine == best || double(before_w) < need_w)) {
        sh.out[0] = mine;
        sh.out[1] = before_w + w;
      }
    }
    __syncthreads();
    const u64 cut = sh.out[0];
    reached = sh.out[1];
    __syncthreads();
    return cut;
  };
  u64 cut = 1;  // every token that may be drawn
  u64 mass = 0;
  auto sum_weights = [&]() {
    u64 t = 0, none = 0;
    for_ids<kThreads>(x, i0, i1, tid, [&](float v, int) { t += weight(v); });
    combine(t, none, plus, plus);
    return t;
  };
  if (do_k) {
    const int m = (k + kWarps * ctas - 1) / (kWarps * ctas);
    if (m <= 32) {
      // the m-th largest of the lanes' maxima, by a sort of the warp (falling with the lane)
      float t = top;
#pragma unroll
      for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
        for (int o = size / 2; o > 0; o /= 2) {
          const float other = __shfl_xor_sync(0xffffffffu, t, o);
          const bool high = ((lane & size) == 0) == ((lane & o) == 0);
          t = high ? fmaxf(t, other) : fminf(t, other);
        }
      }
      u64 mth = key_of(__shfl_sync(0xffffffffu, t, m - 1)), none = 0;
      combine(mth, none, smaller, larger);
      if (mth != 0) list_from(logit_of(uint32_t(mth)));
    }
    cut = max(cut, cut_at(true, u64(k), 0.0, all, mass));
  }
  if (do_p && cut != best) {
    const double share = double(p);
    if (cut == 1) {  // no top-k, or fewer tokens than that: the weight of the whole row
      listed = false;
      mass = sum_weights();
    }
    u64 ignored;
    const float low = cut == 1 ? all : logit_of(uint32_t(cut >> 18));  // top-p of the top-k set ends inside it
    cut = max(cut, cut_at(false, 0, share * double(mass), low, ignored));
  }
  const float mp = min_p ? min_p[b] : 0.f;
  const u64 min_w = mp > 0.f ? u64(ceil(fmin(double(mp), 1.0) * 17592186044416.0)) : 0;  // 2^44: the least integer that passes
  // a logit below this has a weight below min_w (with room for the rounding of both): its weight is not computed
  const float min_logit =
      mp > 0.f && weight.m < INFINITY ? float(double(weight.m) + (log2(fmin(double(mp), 1.0)) - 1e-3) / weight.c) : -INFINITY;
  const float cut_logit = cut == 1 ? -3.402823466e38f : logit_of(uint32_t(cut >> 18));
  const int cut_id = cut == 1 ? V : kMaxVocab - 1 - int(cut & (kMaxVocab - 1));
  auto passes = [&](float v, int id) { return v >= cut_logit && (v > cut_logit || id <= cut_id) && v >= min_logit; };
  auto kept = [&](float v, int id) -> u64 {
    const u64 w = passes(v, id) ? weight(v) : 0;
    return w >= min_w ? w : 0;
  };

  // ---- weights of the kept tokens: a bucket of ids per thread (listed), or a range of ids per warp
  const int bucket_shift = max(0, 32 - __clz(max(1, i1 - i0 - 1)) - 9);  // ids of this CTA in at most 512 buckets
  static_assert(kThreads == 512, "a bucket per thread");
  const int sub = (i1 - i0 + kWarps - 1) / kWarps;
  const int s0 = min(i1, i0 + warp * sub), s1 = min(i1, s0 + sub);
  u64 mine = 0;
  if (cut == best) listed = false;  // one token: found by its id below
  if (listed) {
    sh.merged[tid] = 0;
    __syncthreads();
    each([&](float v, int id) {
      const u64 w = v > -INFINITY ? kept(v, id) : 0;
      if (w) atomicAdd(&sh.merged[(id - i0) >> bucket_shift], w);
    });
    __syncthreads();
    mine = sh.merged[tid];
  } else if (cut == 1 && !(mp > 0.f)) {
    for_ids<32>(x, s0, s1, lane, [&](float v, int) { mine += weight(v); });
  } else if (cut == 1 || mp > 0.f) {
    for_ids<32>(x, s0, s1, lane, [&](float v, int id) { mine += kept(v, id); });
  } else {
    gather.sum = 0;
    for_ids<32>(x, s0, s1, lane, [&](float v, int id) { gather(weight, v, passes(v, id)); });
    mine = gather.finish(weight);
  }
  const u64 bucket = mine;
  mine = warp_sum(mine);
  __syncthreads();
  if (lane == 0) sh.red[0][warp] = mine;
  __syncthreads();
  if (tid == 0) {
    u64 t = 0;
    for (int w = 0; w < kWarps; ++w) t += sh.red[0][w];
    sh.pair[0] = t;
  }
  sync();
  u64 total = 0, before = 0, own = 0;
  of_all(&sh.pair[0], [&](int r, u64 v) {
    if (r == rank) before = total, own = v;
    total += v;
  });
  // ---- the token: the lowest id whose running sum exceeds u * total
  const float uu = u[b];
  const double ud = uu > 0.f ? fmin(double(uu), 1.0 - 5.9604644775390625e-08) : 0.0;
  const u64 target = u64(ud * double(total));
  if (listed) {
    if (before <= target && target < before + own) {
      // the bucket, then the tokens in it in the order of their ids
      u64 all_buckets;
      const u64 pre = before + block_scan(bucket, sh.red[1], all_buckets);
      if (pre <= target && target < pre + bucket) sh.bin = tid, sh.out[0] = pre;
      if (tid == 0) sh.n_list = 0;
      __syncthreads();
      const int at = sh.bin;
      const u64 start = sh.out[0];
      each([&](float v, int id) {
        if (v > -INFINITY && (id - i0) >> bucket_shift == at && kept(v, id)) sh.list[atomicAdd(&sh.n_list, 1u)] = rank_of(v, id);
      });
      __syncthreads();
      const int n = int(sh.n_list);  // at most 512: the ids of a bucket
      if (tid < n) {
        const u64 me = sh.list[tid];
        u64 run = start;
        for (int i = 0; i < n; ++i)  // lower ids have larger low bits
          if ((sh.list[i] & (kMaxVocab - 1)) > (me & (kMaxVocab - 1))) run += weight(logit_of(uint32_t(sh.list[i] >> 18)));
        const u64 wi = weight(logit_of(uint32_t(me >> 18)));
        if (run <= target && target < run + wi) {
          tokens[b] = kMaxVocab - 1 - int(me & (kMaxVocab - 1));
          if (logprob) logprob[b] = float(log(double(wi) / double(total)));
        }
      }
    }
  } else if (before <= target && target < before + own) {
    int w = 0;
    while (target >= before + sh.red[0][w]) before += sh.red[0][w++];
    const int a0 = min(i1, i0 + w * sub), a1 = min(i1, a0 + sub), per = (a1 - a0 + kThreads - 1) / kThreads;
    const int c0 = min(a1, a0 + tid * per), c1 = min(a1, c0 + per);
    u64 t = 0, all;
    for (int i = c0; i < c1; i += kUnroll) {
      float v[kUnroll];
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) v[j] = i + j < c1 ? __ldg(x + i + j) : -INFINITY;
#pragma unroll
      for (int j = 0; j < kUnroll; ++j) t += v[j] > -INFINITY ? kept(v[j], i + j) : 0;
    }
    u64 run = before + block_scan(t, sh.red[1], all);
    if (run <= target && target < run + t) {
      for (int i = c0; i < c1; ++i) {
        const u64 wi = kept(__ldg(x + i), i);
        if (target < run + wi) {
          tokens[b] = i;
          if (logprob) logprob[b] = float(log(double(wi) / double(total)));
          break;
        }
        run += wi;
      }
    }
  }
  sync();  // the others have read this CTA's values
}

}  // namespace

int check_sample(const float* logits, int64_t ld, int B, int V, const float* temperature, const int32_t* top_k,
                 const float* top_p, const float* min_p, const float* u, const int32_t* tokens, const float* logprob) {
  if (B != 0 && (!logits || !u || !tokens)) return fail(FG_ERR_INVALID_ARG, "null pointer");
  if (B < 0 || V <= 0 || ld < V) return fail(FG_ERR_SHAPE, "bad logits shape");
  if (V > kMaxVocab) return fail(FG_ERR_UNSUPPORTED, "vocab above 2^18");
  const void* ptrs[] = {logits, temperature, top_k, top_p, min_p, u, tokens, logprob};
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 3u) return fail(FG_ERR_ALIGN, "pointers must be 4-byte aligned");
  return FG_OK;
}

int sample_impl(const float* logits, int64_t ld, int B, int V, const float* temperature, const int32_t* top_k,
                const float* top_p, const float* min_p, const float* u, int32_t* tokens, float* logprob,
                cudaStream_t s) {
  FG_TRY(check_sample(logits, ld, B, V, temperature, top_k, top_p, min_p, u, tokens, logprob));
  if (B == 0) return FG_OK;
  ProfScope ps(PROF_OTHER, s, 0.0, double(B) * V * 4.0);
  // CTAs per row: as many as find an SM each, with at least 7168 ids.  Top-p 0.9 (top-k 40 and top-p 0.9 behind the comma),
  // N(0, 1): 24 rows of 50272 45, 31 us on 4 CTAs, 92, 71 on 8, which take two rounds, 65, 33 on 2, 100, 29 on 1; one row 44, 29
  // on 4, 46, 35 on 8.  3 rows of 128001: 55, 37 us on 8, 75, 33 on 4, 225, 38 on 1.  256 rows of 50272: 139, 39 us on 1 (two
  // CTAs share an SM), 248, 127 on 2.
  int ctas = 1;
  while (ctas < 8 && int64_t(B) * ctas * 2 <= num_sms() && V >= ctas * 14336) ctas *= 2;
  if (int64_t(B) * ctas > 0x7fffffff) return fail(FG_ERR_SHAPE, "too many rows");
  auto kernel = ctas == 8 ? sample_kernel<8> : ctas == 4 ? sample_kernel<4> : ctas == 2 ? sample_kernel<2> : sample_kernel<1>;
  static std::atomic<uint64_t> attr_done[9] = {};
  FG_TRY(ensure_smem_attr(kernel, int(sizeof(Shared)), attr_done[ctas]));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(unsigned(B * ctas));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(Shared);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  at[1].id = cudaLaunchAttributeClusterDimension;
  at[1].val.clusterDim.x = unsigned(ctas);
  at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 2;
  count_launch();
  const cudaError_t e =
      cudaLaunchKernelEx(&cfg, kernel, logits, ld, V, temperature, top_k, top_p, min_p, u, tokens, logprob);
  if (e != cudaSuccess) return cuda_fail(e, "sample kernel");
  return FG_OK;
}

}  // namespace fg
