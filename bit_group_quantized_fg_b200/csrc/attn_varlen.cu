// Causal attention over packed ragged fp16 rows with a cached prefix, grouped heads, a sliding
// window and sinks (include/fg.h, fg_varlen_attention).
//
// out_i = sum_t softmax_t(q_i . k_t / sqrt(hd)) v_t over the visible t, flash style: fp32 online
// softmax, P rounded to fp16 (2^-11 of each weight) for the second product, nothing of size L x L
// in memory.
//
// Persistent, one CTA per SM that takes item after item, on the 5th-generation tensor cores.  A work item is two query tiles
// of 128 rows that read the same keys: two heads of a key/value group when the group has an even
// number of them, else two neighbouring tiles of one head; heavy (late) tiles first.  (Where there is
// one query tile per head: two heads, whose key tiles alternate.)  Twelve warps:
//   warps 0-3 and 4-7  softmax of query tile 0 and 1, a thread per row
//   warp 8 (one thread) every MMA, warp 9 (one thread) every copy, warp 10 (one thread) fetches the numbers of the
//   items to come (11 only makes up the warpgroup)
// Tensor memory: S0, S1 (128 columns each, P over the first 64 as fp16 pairs), O0, O1.
//   copies   Q of the item, then key and value tiles of 128 rows, two of each in flight (TMA, 128-byte
//            swizzle), ahead of the MMAs over the item's end into the next one
//   MMAs     ... P0 V, Q0 K' , P1 V, Q1 K' ... : while tile 0's softmax runs, the tensor cores work on
//            tile 1.  MMAs of one thread execute in order, so "S complete" also says that the P V before
//            it has landed: a softmax that has its S may rescale O without another wait.
//   softmax  the row of S in registers; P = 2^(s - m) against the maximum m of the first tile that the row sees
//            any key of, which is raised (and O rescaled) only when the weights of a tile add up to more than 2^13: until then
//            every P fits fp16 and the fp32 sums with the same relative precision as against the true
//            maximum, and no maximum has to be taken.
// What bounds it: the tensor cores and the exponentials in turn (each 53 % busy; with the exponentials left out 2 x 8191
// rows still took 480 us of 560), where keys are many; HBM and the start of items where they are few.
// Measured: 2 sequences of 8191, window 2048, 32 heads on 8 (498 GFLOP): 525 us cold, 608 us repeated
// under the power limit; 64 x up to 512, 32 heads of 128 (802 MB): 238 us, 275 us repeated; 4 x 32, 12 heads
// of 64: 11 us.  Two heads that share their keys as one item against two neighbouring tiles of a head,
// where both are possible: 560 and 582 us, so an even group is paired.
// Only tiles that some row sees are visited.  In tiles at the edge of what is visible, P is 0 for
// keys a row does not see; there the value tile is also scanned for NaN and infinities (0 * NaN is
// NaN): where there are any they are taken out of shared memory, and the rows that do see them get
// them back in the epilogue.
#include <cudaTypedefs.h>

#include <algorithm>

#include "paged_common.cuh"
#include "sm100.cuh"

namespace fg {

int make_map_2d(CUtensorMap* m, const void* base, CUtensorMapDataType dt, int elem_bytes, uint64_t inner,
                uint64_t outer, uint64_t row_bytes, uint32_t box_inner, uint32_t box_outer, CUtensorMapSwizzle swz);

namespace {

constexpr int kT = 128;           // query rows and keys of a tile
constexpr int kBox = kT * 128;    // a [128 rows x 64 fp16] swizzled box (16 KB)
constexpr int kThreads = 384;
// Registers: 168 a thread at launch (384 of them); the softmax warpgroups hold a row of 128 scores and take what the
// third one gives up: 2 * 128 * 216 + 128 * 72 = 384 * 168.
constexpr int kRegsSoftmax = 216, kRegsIssue = 72;

template <int HD>
struct VCfg {
  static constexpr int NB = HD / 64;            // 64-column boxes across the head
  static constexpr int kTile = NB * kBox;       // bytes of a Q, K or V tile
  static constexpr int kOffK = 2 * kTile;       // two query tiles, then two key and two value tiles
  static constexpr int kOffV = 4 * kTile;
  static constexpr int kOffStage = 6 * kTile;   // 4 KB per softmax warp for its output
  static constexpr int kSmem = kOffStage + 8 * 4096 + 1024;  // + alignment
  static constexpr uint32_t kTmemCols = 512;    // S0, S1 at 0 and 128; O0, O1 at 256 and 384
};

struct VArgs {
  const int32_t *q_start, *k_start;
  __half* out;
  int n_q, n_k, B, max_q, nh, rep, window, n_sink;
  int paired;       // 1: an item is two heads of 128 rows; 0: one head of 256 rows
  int n_units;      // heads or head pairs
  int n_qt;         // query tiles (pairs of them when not paired) of the longest sequence
  uint32_t per, items;  // items of one query tile, of all
  int dynamic;      // 1: a CTA per item was asked for, and the running ones take over those not yet started
};

// The starts of an item's sequence, fetched an item ahead: their latency is not waited for.
struct Starts {
  int qs, qe, ks, ke;
};
__device__ __forceinline__ Starts fetch_starts(const VArgs& a, uint32_t idx) {
  if (idx >= a.items) return Starts{0, 0, 0, 0};
  const int b = int(idx % a.per / uint32_t(a.n_units));
  return Starts{__ldg(a.q_start + b), __ldg(a.q_start + b + 1), __ldg(a.k_start + b), __ldg(a.k_start + b + 1)};
}

// One work item: two query tiles over the keys of a sequence.  split: they are two heads that do not share their keys.
template <int split>
struct Item {
  int qs, nq, ks;          // first query row, query count, first key row
  int q0, dq, head, dh;    // tile 1: first query q0 + dq, head + dh
  int p0, p1[2];           // positions of the first query (tile 1: + dq) and of each tile's last (-1: sees nothing)
  int st, w0[2];           // a tile needs the key tiles below st and those from w0 on, up to its last position
  int window, n_sink;
  // Steps: key tiles, or (split) 2 * key tile + query tile.

  __device__ __forceinline__ bool load(const VArgs& a, uint32_t idx, const Starts& r) {
    const int rows = a.paired ? kT : 2 * kT;
    const int qt = a.n_qt - 1 - int(idx / a.per), unit = int(idx % a.per % uint32_t(a.n_units));
    qs = min(max(r.qs, 0), a.n_q);
    const int all = min(max(r.qe, 0), a.n_q) - qs;
    nq = min(all, a.max_q);
    ks = min(max(r.ks, 0), a.n_k);
    const int nk = max(0, min(max(r.ke, 0), a.n_k) - ks);
    window = a.window;
    n_sink = a.n_sink;
    q0 = qt * rows;
    if (q0 >= nq) return false;
    dq = a.paired ? 0 : kT;
    dh = a.paired ? 1 : 0;
    head = a.paired ? 2 * unit : unit;
    p0 = nk - all + q0;
    p1[0] = p0 + min(kT, nq - q0) - 1;
    p1[1] = q0 + dq < nq ? p0 + dq + min(kT, nq - q0 - dq) - 1 : -1;
    st = window > 0 ? (n_sink + kT - 1) / kT : 0;
    w0[0] = window > 0 ? max(0, p0 - window + 1) / kT : 0;
    w0[1] = window > 0 ? max(0, p0 + dq - window + 1) / kT : 0;
    return true;
  }
  __device__ __forceinline__ int tile(int step) const { return step >> split; }
  __device__ __forceinline__ bool need(int i, int last, int w, int step) const {
    const int kt = tile(step);
    return kt * kT <= last && (kt < st || kt >= w) && !(split && (step & 1) != i);
  }
  __device__ __forceinline__ bool need(int i, int step) const { return need(i, p1[i], w0[i], step); }
  // every row at positions lo .. hi sees all of key tile kt
  __device__ __forceinline__ bool full(int lo, int hi, int kt) const {
    const int t0 = kt * kT, t1 = t0 + kT - 1;
    return t1 <= lo && (window <= 0 || t0 > hi - window || t1 < n_sink);
  }
  // the step after this one (-1: the first one) that a query tile needs, or -1
  __device__ __forceinline__ int next(int step) const {
    if (split && !(step & 1)) return step + 1;  // the two heads have the same positions
    int kt = tile(step) + 1;
    if (kt >= st) kt = max(kt, p1[0] >= 0 ? w0[0] : w0[1]);
    return kt * kT <= max(p1[0], p1[1]) ? kt << split : -1;
  }
};

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two fp32 operations in one instruction (each rounded as the single one).
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// The items of a CTA after its first one.  Statically every gridDim.x-th; dynamically those of CTAs that have not started
// yet, which the scheduling thread cancels one by one (clusterlaunchcontrol), up to kAhead in advance of the slowest
// reader.  Every reader gets the same sequence; the answers stand in a ring.
constexpr int kAhead = 3, kReaders = 10;
struct Answers {
  __align__(16) uint4 answer[kAhead];
  __align__(8) uint64_t full[kAhead], empty[kAhead];
};
// The CTA that was cancelled, or ~0 when there was none left.
__device__ __forceinline__ uint32_t cancelled(const uint4* answer) {
  uint32_t x, got;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.u32 %1, 1, 0, p;\n\t"
      "mov.u32 %0, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, y, z, w}, h;\n\t}"
      : "=r"(x), "=r"(got)
      : "r"(sm100::smem_u32(answer))
      : "memory");
  return got ? x : 0xffffffffu;
}
struct Reader {
  uint32_t n = 0;
  // Called by a single thread, or by a whole warp (`one`: the lane that says that it has read).
  __device__ __forceinline__ uint32_t next(const VArgs& a, uint32_t idx, Answers& q, volatile int* abort_p, int* err, bool warp_wide,
                                           bool one) {
    if (!a.dynamic) return idx + gridDim.x;
    const uint32_t s = n % kAhead, ph = (n / kAhead) & 1;
    ++n;
    bool ok = sm100::mbar_wait(&q.full[s], ph, abort_p, err, 0x100000);
    if (warp_wide) ok = __all_sync(0xffffffffu, ok);
    const uint32_t x = ok ? cancelled(&q.answer[s]) : 0xffffffffu;
    if (warp_wide) __syncwarp();
    if (one) sm100::mbar_arrive(&q.empty[s]);
    return x;
  }
};

template <int HD, int SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    varlen_attn_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv, const VArgs a, const __half* __restrict__ v, int64_t kv_stride,
                       int* __restrict__ err) {
  using namespace sm100;
  using C = VCfg<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  __shared__ __align__(8) uint64_t bars[17];
  uint64_t* kfull = bars + 0;    // [2] key tile landed
  uint64_t* kempty = bars + 2;   // [2] its products are complete
  uint64_t* vfull = bars + 4;    // [2]
  uint64_t* vempty = bars + 6;   // [2]
  uint64_t* qfull = bars + 8;    // the item's query tiles landed
  uint64_t* qempty = bars + 9;   // the item's Q K products are complete
  uint64_t* sfull = bars + 10;   // [2] S of query tile i complete (and the P V before it)
  uint64_t* pfull = bars + 12;   // [2] P of query tile i written (one arrival per warp)
  uint64_t* ofin = bars + 14;    // [2] the item's last P V of query tile i is complete
  uint64_t* bar_d = bars + 16;   // drain on abort
  __shared__ Answers answers;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  // By the parity of an item's number: 1 + the last item whose values were cleaned of NaN and infinities.  A later
  // item's mark may cover an earlier one's: the epilogue then looks for values to give back and finds none.
  __shared__ uint32_t dirty[2];
  volatile int* abort_p = &abort_flag;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int i = 0; i < 17; ++i) mbar_init(&bars[i], (i == 12 || i == 13) ? 4 : 1);
    for (int i = 0; i < kAhead; ++i) {
      mbar_init(&answers.full[i], 1);
      mbar_init(&answers.empty[i], kReaders);
    }
    abort_flag = 0;
    dirty[0] = dirty[1] = 0;
    fence_barrier_init();
  }
  if (warp == 8) tmem_alloc(&tmem_slot, C::kTmemCols);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  pdl_wait();  // the previous kernel in the stream has finished (see fg_launch)
  Item<SPLIT> it;

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
    if (warp == 9) {
    // ------------------------------------------------------------ copies
    if (lane == 0) {
      prefetch_tmap(&tq);
      prefetch_tmap(&tk);
      prefetch_tmap(&tv);
      bool ok = true;
      uint32_t nk = 0, n = 0, items = 0;  // key tiles, value tiles and items so far
      Starts nx = fetch_starts(a, blockIdx.x);
      Reader reader;
      for (uint32_t idx = blockIdx.x, following; idx < a.items && ok; idx = following) {
        const bool any = it.load(a, idx, nx);
        following = reader.next(a, idx, answers, abort_p, err, false, true);
        nx = fetch_starts(a, following);
        if (!any) continue;
        int kt = it.next(-1);
        if (kt < 0) continue;  // no query of the item sees anything
        auto col = [&]() { return (it.head + (SPLIT ? kt & 1 : 0)) / a.rep * HD; };
        auto load_k = [&]() {
          const int s = n & 1;
          if (n >= 2 && !mbar_wait(&kempty[s], ((n >> 1) & 1) ^ 1, abort_p, err, 0x20000)) return false;
          mbar_expect_tx(&kfull[s], C::kTile);
          for (int x = 0; x < C::NB; ++x)
            tma_load_2d(smem + C::kOffK + s * C::kTile + x * kBox, &tk, col() + 64 * x, it.ks + it.tile(kt) * kT, &kfull[s]);
          ++nk;
          return true;
        };
        // the first key tile does not wait for the last item's queries to be read
        if (!(ok = load_k())) break;
        if (items > 0 && !(ok = mbar_wait(qempty, (items - 1) & 1, abort_p, err, 0x20000))) break;
        ++items;
        const bool two = it.p1[1] >= 0 || it.q0 + it.dq < it.nq;
        mbar_expect_tx(qfull, (two ? 2 : 1) * C::kTile);
        for (int i = 0; i < (two ? 2 : 1); ++i)
          for (int x = 0; x < C::NB; ++x)
            tma_load_2d(smem + i * C::kTile + x * kBox, &tq, (it.head + i * it.dh) * HD + 64 * x, it.qs + it.q0 + i * it.dq, qfull);
        for (;;) {
          const int s = n & 1;
          if (n >= 2 && !(ok = mbar_wait(&vempty[s], ((n >> 1) & 1) ^ 1, abort_p, err, 0x20000))) break;
          mbar_expect_tx(&vfull[s], C::kTile);
          for (int x = 0; x < C::NB; ++x)
            tma_load_2d(smem + C::kOffV + s * C::kTile + x * kBox, &tv, col() + 64 * x, it.ks + it.tile(kt) * kT, &vfull[s]);
          ++n;
          if ((kt = it.next(kt)) < 0) break;
          if (!(ok = load_k())) break;
        }
      }
      if (!ok) {
        // the copies still under way land before the CTA leaves
        if (items > 0) mbar_wait_drain(qfull, (items - 1) & 1);
        for (uint32_t i = nk > 2 ? nk - 2 : 0; i < nk; ++i) mbar_wait_drain(&kfull[i & 1], (i >> 1) & 1);
        for (uint32_t i = n > 2 ? n - 2 : 0; i < n; ++i) mbar_wait_drain(&vfull[i & 1], (i >> 1) & 1);
      }
    }
    __syncwarp();
    } else if (warp == 10) {
    // ------------------------------------------------------------ the items to come
    if (lane == 0 && a.dynamic) {
      for (uint32_t n = 0;; ++n) {
        const uint32_t s = n % kAhead, ph = (n / kAhead) & 1;
        if (n >= kAhead && !mbar_wait(&answers.empty[s], ph ^ 1, abort_p, err, 0x200000)) break;
        fence_proxy_async_smem();  // the last answer has been read
        mbar_expect_tx(&answers.full[s], 16);
        asm volatile(
            "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                smem_u32(&answers.answer[s])),
            "r"(smem_u32(&answers.full[s]))
            : "memory");
        mbar_wait_drain(&answers.full[s], ph);  // (every answer has landed when the CTA leaves)
        if (cancelled(&answers.answer[s]) == 0xffffffffu) break;  // no more may be asked for after that
      }
    }
    __syncwarp();
    } else if (warp == 8) {
    // ------------------------------------------------------------ MMAs
    if (elect_one()) {
      constexpr uint32_t idesc_qk = idesc_f16_f32(kT, kT, false);
      constexpr uint32_t idesc_pv = idesc_f16_f32(kT, HD, true);
      // descriptors of the first 16 columns (rows of V); the others are steps of their 16-byte address field
      const uint64_t dq0 = smem_desc_sw128(smem_u32(smem), 16, 1024);
      const uint64_t dk0 = smem_desc_sw128(smem_u32(smem + C::kOffK), 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(smem_u32(smem + C::kOffV), kBox, 1024);
      constexpr uint64_t kTileStep = C::kTile >> 4;
      bool ok = true;
      uint32_t n = 0, items = 0, cnt[2] = {0, 0};  // key tiles, items, P of each query tile so far
      auto qk = [&](int i, uint32_t n_) {          // S_i = Q_i K' of the n_-th key tile
        const uint64_t dq = dq0 + i * kTileStep, dk = dk0 + (n_ & 1) * kTileStep;
#pragma unroll
        for (int kk = 0; kk < HD / 16; ++kk) {
          constexpr uint64_t kBoxStep = kBox >> 4;
          const uint64_t step = (kk >> 2) * kBoxStep + (kk & 3) * 2;
          mma_f16_ss(tmem + 128 * i, dq + step, dk + step, idesc_qk, kk > 0);
        }
        mma_commit(&sfull[i]);
      };
      Starts nx = fetch_starts(a, blockIdx.x);
      Reader reader;
      for (uint32_t idx = blockIdx.x, following; idx < a.items && ok; idx = following) {
        const bool any = it.load(a, idx, nx);
        following = reader.next(a, idx, answers, abort_p, err, false, true);
        nx = fetch_starts(a, following);
        if (!any) continue;
        int kt = it.next(-1);
        if (kt < 0) continue;
        bool need0 = it.need(0, kt), need1 = it.need(1, kt);
        uint32_t acc0 = 0, acc1 = 0;  // O of each query tile holds something of this item
        if (!(ok = mbar_wait(&kfull[n & 1], (n >> 1) & 1, abort_p, err, 0x40000))) break;
        if (!(ok = mbar_wait(qfull, items & 1, abort_p, err, 0x40000))) break;
        ++items;
        tc_fence_after();
        if (need0) qk(0, n);
        if (need1) qk(1, n);
        mma_commit(&kempty[n & 1]);
        // split: the other head's scores are under way before this one's weights are waited for
        while (SPLIT) {
          const int kn = it.next(kt), i = kt & 1;
          if (kn >= 0) {
            if (!(ok = mbar_wait(&kfull[(n + 1) & 1], ((n + 1) >> 1) & 1, abort_p, err, 0x40000))) break;
            tc_fence_after();
            if (i) qk(0, n + 1);
            else qk(1, n + 1);
            mma_commit(&kempty[(n + 1) & 1]);
          } else {
            mma_commit(qempty);
          }
          if (!(ok = mbar_wait(&vfull[n & 1], (n >> 1) & 1, abort_p, err, 0x40000))) break;
          if (!(ok = mbar_wait(&pfull[i], (i ? cnt[1]++ : cnt[0]++) & 1, abort_p, err, 0x40000))) break;
          tc_fence_after();
          const uint64_t dv = dv0 + (n & 1) * kTileStep;
          const uint32_t acc = i ? acc1 : acc0;
#pragma unroll
          for (int kk = 0; kk < kT / 16; ++kk)
            mma_f16_ts(tmem + 256 + 128 * i, tmem + 128 * i + 8 * kk, dv + 128 * kk, idesc_pv, kk > 0 ? 1u : acc);
          (i ? acc1 : acc0) = 1;
          mma_commit(&vempty[n & 1]);
          ++n;
          if (kn < 0 || it.next(kn) < 0) mma_commit(&ofin[i]);  // the head's last key tile
          if (kn < 0) break;
          kt = kn;
        }
        while (!SPLIT) {
          const int kn = it.next(kt);
          const bool next0 = kn >= 0 && it.need(0, kn), next1 = kn >= 0 && it.need(1, kn);
          if (kn < 0) mma_commit(qempty);  // the last Q K of the item has been issued
          const uint64_t dv = dv0 + (n & 1) * kTileStep;
          if (!(ok = mbar_wait(&vfull[n & 1], (n >> 1) & 1, abort_p, err, 0x40000))) break;
          if (kn >= 0 && !(ok = mbar_wait(&kfull[(n + 1) & 1], ((n + 1) >> 1) & 1, abort_p, err, 0x40000))) break;
          if (need0) {
            if (!(ok = mbar_wait(&pfull[0], cnt[0] & 1, abort_p, err, 0x40000))) break;
            ++cnt[0];
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kT / 16; ++kk)
              mma_f16_ts(tmem + 256, tmem + 8 * kk, dv + 128 * kk, idesc_pv, kk > 0 ? 1u : acc0);
            acc0 = 1;
          }
          if (kn < 0 && acc0) mma_commit(&ofin[0]);  // O_0 is final
          if (next0) qk(0, n + 1);
          if (need1) {
            if (!(ok = mbar_wait(&pfull[1], cnt[1] & 1, abort_p, err, 0x40000))) break;
            ++cnt[1];
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < kT / 16; ++kk)
              mma_f16_ts(tmem + 384, tmem + 128 + 8 * kk, dv + 128 * kk, idesc_pv, kk > 0 ? 1u : acc1);
            acc1 = 1;
          }
          mma_commit(&vempty[n & 1]);
          ++n;
          if (kn < 0) {
            if (acc1) mma_commit(&ofin[1]);
            break;
          }
          if (next1) qk(1, n);
          mma_commit(&kempty[n & 1]);
          kt = kn;
          need0 = next0;
          need1 = next1;
        }
      }
      if (!ok) {
        mma_commit(bar_d);
        mbar_wait_drain(bar_d, 0);
      }
    }
    __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------ softmax and epilogue
    const int i = warp >> 2, r = threadIdx.x & 127;
    const uint32_t lane_off = uint32_t((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + 128 * i + lane_off, tO = tmem + 256 + 128 * i + lane_off;
    const float sl2 = 1.4426950408889634f * rsqrtf(float(HD));  // log2(e) / sqrt(hd)
    const int64_t h_all = int64_t(a.nh) * HD;
    bool ok = true;
    uint32_t n = 0, items = 0, cnt = 0, fin = 0;  // key tiles, items, S and O of this query tile so far
    Starts nx = fetch_starts(a, blockIdx.x);
    Reader reader;
    for (uint32_t idx = blockIdx.x, following; idx < a.items && ok; idx = following) {
      const bool any = it.load(a, idx, nx);
      following = reader.next(a, idx, answers, abort_p, err, true, lane == 0);
      nx = fetch_starts(a, following);
      if (!any) continue;
      // (selected, not indexed: the arrays stay in registers)
      const int q0 = it.q0 + i * it.dq, head = it.head + i * it.dh;
      const int p_lo = it.p0 + i * it.dq, p_hi = i ? it.p1[1] : it.p1[0], w0 = i ? it.w0[1] : it.w0[0];
      const bool valid = q0 + r < it.nq;
      const int p = p_lo + r;
      __half* out_head = a.out + (int64_t(it.qs) + q0) * h_all + head * HD;
      int kt = it.next(-1);
      if (kt < 0) {
        if (valid)
          for (int c = 0; c < HD / 8; ++c) reinterpret_cast<uint4*>(out_head + r * h_all)[c] = make_uint4(0, 0, 0, 0);
        continue;
      }
      float m_run = -INFINITY, mz = 0.f, l_run = 0.f;
      bool started = false, has_o = false;  // every row of the warp has a maximum; O holds something of this item
      for (; kt >= 0; kt = it.next(kt), ++n) {
        if (!it.need(i, p_hi, w0, kt)) continue;
        const int t0 = it.tile(kt) * kT;
        const bool masked = !it.full(p_lo, p_hi, it.tile(kt));
        ok = mbar_wait(&sfull[i], cnt & 1, abort_p, err, 0x80000);
        if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
        ++cnt;
        tc_fence_after();
        if (masked) {
          // values of keys that some row does not see: none may be NaN or infinite in the product
          ok = mbar_wait(&vfull[n & 1], (n >> 1) & 1, abort_p, err, 0x80000);
          if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
          uint4* vt = reinterpret_cast<uint4*>(smem + C::kOffV + (n & 1) * C::kTile) + r;
          const __half2 zero = __floats2half2_rn(0.f, 0.f);
          __half2 z[4] = {zero, zero, zero, zero};
#pragma unroll
          for (int c = 0; c < C::kTile / 16; c += 128) {
            const uint4 w = vt[c];
            z[0] = __hfma2(u32_as_h2(w.x), zero, z[0]);
            z[1] = __hfma2(u32_as_h2(w.y), zero, z[1]);
            z[2] = __hfma2(u32_as_h2(w.z), zero, z[2]);
            z[3] = __hfma2(u32_as_h2(w.w), zero, z[3]);
          }
          z[0] = __hadd2(__hadd2(z[0], z[1]), __hadd2(z[2], z[3]));
          if (__hisnan(__low2half(z[0])) || __hisnan(__high2half(z[0]))) {
            atomicMax(&dirty[items & 1], items + 1);
            __threadfence_block();
            for (int c = 0; c < C::kTile / 16; c += 128) {
              uint32_t* w = reinterpret_cast<uint32_t*>(vt + c);
              for (int e = 0; e < 4; ++e) {
                uint32_t x = w[e];
                if ((x & 0x7c00u) == 0x7c00u) x &= 0xffff0000u;
                if ((x & 0x7c000000u) == 0x7c000000u) x &= 0xffffu;
                w[e] = x;
              }
            }
            fence_proxy_async_smem();
          }
        }
        // the row's scores; those of keys it does not see are -inf
        uint32_t s[kT];
        auto load_scores = [&]() {
#pragma unroll
          for (int c = 0; c < kT; c += 32) tmem_ld_32x32b_x32(tS + c, *reinterpret_cast<uint32_t(*)[32]>(&s[c]));
          tmem_ld_wait();
#pragma unroll
          for (int c = 0; c < kT; ++c) asm volatile("" : "+r"(s[c]));  // nothing reads them before the wait
          if (masked) {
            const int last = p - t0;                                             // key c is seen when c <= last and
            const int first = it.window > 0 ? last - it.window : -kT;            // (c > first or c < sinks)
            const int sinks = it.window > 0 ? it.n_sink - t0 : 0;
#pragma unroll
            for (int c0 = 0; c0 < kT; c0 += 32) {
              auto below = [&](int x) {  // the bits of columns c0 .. c0 + 31 that are below x
                const int y = x - c0;
                return y <= 0 ? 0u : y >= 32 ? 0xffffffffu : (1u << y) - 1u;
              };
              const uint32_t seen = below(last + 1) & (~below(first + 1) | below(sinks));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(seen & (1u << c))) s[c0 + c] = 0xff800000u;
            }
          }
        };
        load_scores();
        float l_new;
        for (;;) {
          if (!started) {
            // the row's maximum of this tile becomes the reference, O and l are scaled to it (nothing yet: 0)
            float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < kT; c += 8)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[e] = max3(x[e], __uint_as_float(s[c + 2 * e]), __uint_as_float(s[c + 2 * e + 1]));
            const float mx = fmaxf(max3(x[0], x[1], x[2]), x[3]) * sl2;
            if (has_o && __any_sync(0xffffffffu, mx > m_run)) {
              const float alpha = mx > m_run ? ex2(m_run - mx) : 1.f;
#pragma unroll 1
              for (int c = 0; c < HD; c += 8) {
                uint32_t o[8];
                tmem_ld_32x32b_x8(tO + c, o);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st_32x32b_x8(tO + c, o);
              }
            }
            if (mx > m_run) {
              l_run *= ex2(m_run - mx);  // 0 from -inf
              m_run = mz = mx;
            }
          }
          // P = 2^(s - m) in place of the first half of the scores
          const uint64_t sl22 = pack2(sl2, sl2), mz2 = pack2(-mz, -mz);
          uint64_t ls[2] = {0, 0};
#pragma unroll
          for (int c = 0; c < kT; c += 2) {
            float e0, e1;
            unpack2(fma2(pack2(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), sl22, mz2), e0, e1);
            e0 = ex2(e0);
            e1 = ex2(e1);
            ls[(c >> 1) & 1] = add2(ls[(c >> 1) & 1], pack2(e0, e1));
            s[c / 2] = h2_as_u32(__floats2half2_rn(e0, e1));
          }
          float l0, l1;
          unpack2(add2(ls[0], ls[1]), l0, l1);
          l_new = l0 + l1;
          // The maximum of a later tile is not looked for: as long as the row's weights of this tile add up to at most
          // 2^13 each of them is exact enough in fp16 and fp32 against the old one.  A row that passes it sends its
          // warp back for a new maximum.
          if (!started || !__any_sync(0xffffffffu, l_new > 8192.f)) break;
          started = false;
          load_scores();
        }
        started = __all_sync(0xffffffffu, !valid || m_run > -INFINITY);  // a row may see nothing of the first tiles
        has_o = true;
        l_run += l_new;
        tmem_st_32x32b_x32(tS, *reinterpret_cast<uint32_t(*)[32]>(&s[0]));
        tmem_st_32x32b_x32(tS + 32, *reinterpret_cast<uint32_t(*)[32]>(&s[32]));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[i]);
      }
      if (!ok) break;
      const uint32_t item = items++;
      if (!has_o) {  // no query of this tile sees anything
        if (valid)
          for (int c = 0; c < HD / 8; ++c) reinterpret_cast<uint4*>(out_head + r * h_all)[c] = make_uint4(0, 0, 0, 0);
        continue;
      }
      // epilogue: O / l to fp16, once the item's last P V has landed
      ok = mbar_wait(&ofin[i], fin & 1, abort_p, err, 0x80000);
      if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
      ++fin;
      tc_fence_after();
      const bool give_back = *reinterpret_cast<volatile uint32_t*>(&dirty[item & 1]) > item;
      const float inv = 1.f / l_run;
      // 64 columns of the warp's 32 rows at a time through shared memory, so that 8 lanes store a row's 128 bytes
      uint8_t* stage = smem + C::kOffStage + warp * 4096;
      const int rows_left = it.nq - q0 - (warp & 3) * 32;  // of this warp's 32 rows
#pragma unroll 1
      for (int c0 = 0; c0 < HD; c0 += 64) {
        __syncwarp();  // the stage has been read
#pragma unroll 1
        for (int c = c0; c < c0 + 64; c += 32) {
          uint32_t o[32];
          tmem_ld_32x32b_x32(tO + c, o);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) asm volatile("" : "+r"(o[e]));
          if (give_back && valid) {  // NaN and infinities that were taken out of the values, for the rows that see them
            const __half* vc = v + int64_t(head / a.rep) * HD + c;
            for (int k2 = it.next(-1); k2 >= 0; k2 = it.next(k2)) {
              const int k3 = it.tile(k2);
              if (SPLIT && (k2 & 1) != i) continue;  // the other head's values
              if ((!it.need(0, k2) || it.full(it.p0, it.p1[0], k3)) && (!it.need(1, k2) || it.full(it.p0 + it.dq, it.p1[1], k3)))
                continue;
              for (int t = k3 * kT; t < (k3 + 1) * kT && t <= p; ++t) {
                if (it.window > 0 && t <= p - it.window && t >= it.n_sink) continue;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                  const float y = __half2float(vc[(int64_t(it.ks) + t) * kv_stride + e]);
                  if (!(fabsf(y) < INFINITY)) o[e] = __float_as_uint(__uint_as_float(o[e]) + y);
                }
              }
            }
          }
#pragma unroll
          for (int e = 0; e < 32; e += 2)  // l = 0: this row saw nothing
            o[e / 2] = l_run == 0.f ? 0u : h2_as_u32(__floats2half2_rn(__uint_as_float(o[e]) * inv, __uint_as_float(o[e + 1]) * inv));
#pragma unroll
          for (int e = 0; e < 4; ++e) {  // 16-byte pieces in the order piece ^ row, so that neither side has bank conflicts
            const int piece = (c - c0) / 8 + e;
            *reinterpret_cast<uint4*>(stage + lane * 128 + ((piece ^ (lane & 7)) << 4)) =
                make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        __syncwarp();
        __half* dst = out_head + int64_t((warp & 3) * 32 + (lane >> 3)) * h_all + c0 + (lane & 7) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int row = 4 * e + (lane >> 3);
          const uint4 w = *reinterpret_cast<const uint4*>(stage + row * 128 + (((lane & 7) ^ (row & 7)) << 4));
          if (row < rows_left) *reinterpret_cast<uint4*>(dst + int64_t(4 * e) * h_all) = w;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

}  // namespace

int varlen_attention_impl(const void* q, int64_t q_stride, int64_t n_q, const void* k, const void* v, int64_t kv_stride,
                          int64_t n_k, const int32_t* q_start, const int32_t* k_start, int B, int max_q, int nh, int nkv,
                          int hd, int window, int n_sink, void* out, cudaStream_t s) {
  // no rows: there may be no buffer
  if (!q_start || !k_start || (n_q != 0 && (!q || !out)) || (n_k != 0 && (!k || !v)))
    return fail(FG_ERR_INVALID_ARG, "null pointer");
  if (B <= 0 || B > 65535 || max_q < 0 || n_q < 0 || n_k < 0 || n_q > (1 << 30) || n_k > (1 << 30))
    return fail(FG_ERR_SHAPE, "bad batch (1..65535 sequences, at most 2^30 rows)");
  if (hd != 64 && hd != 128) return fail(FG_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
  if (nh <= 0 || nkv <= 0 || nh % nkv || nh > 65535) return fail(FG_ERR_SHAPE, "n_heads must be a multiple of n_kv_heads");
  if (int64_t(nh) * hd > (1 << 24)) return fail(FG_ERR_SHAPE, "more than 2^24 query values a row");
  if (n_sink < 0) return fail(FG_ERR_INVALID_ARG, "n_sink must not be negative");
  if (q_stride < int64_t(nh) * hd || q_stride % 8 || kv_stride < int64_t(nkv) * hd || kv_stride % 8)
    return fail(FG_ERR_ALIGN, "strides must hold a row and be multiples of 8");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(out))
    return fail(FG_ERR_ALIGN, "pointers must be 16-byte aligned");
  if (!aligned4(q_start) || !aligned4(k_start)) return fail(FG_ERR_ALIGN, "index arrays must be 4-byte aligned");
  if (max_q == 0 || n_q == 0) return FG_OK;
  CUtensorMap tq, tk, tv;
  const auto f16 = CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const auto sw = CU_TENSOR_MAP_SWIZZLE_128B;
  if (n_k == 0) k = v = q, kv_stride = q_stride;  // no key tile is ever copied then
  const uint64_t rows_k = uint64_t(n_k ? n_k : n_q);
  FG_TRY(make_map_2d(&tq, q, f16, 2, uint64_t(nh) * hd, uint64_t(n_q), uint64_t(q_stride) * 2, 64, kT, sw));
  FG_TRY(make_map_2d(&tk, k, f16, 2, uint64_t(nkv) * hd, rows_k, uint64_t(kv_stride) * 2, 64, kT, sw));
  FG_TRY(make_map_2d(&tv, v, f16, 2, uint64_t(nkv) * hd, rows_k, uint64_t(kv_stride) * 2, 64, kT, sw));
  int* err = device_error_ptr();
  if (!err) return fail(FG_ERR_CUDA, "device error flag unavailable");
  VArgs a;
  a.q_start = q_start;
  a.k_start = k_start;
  a.out = reinterpret_cast<__half*>(out);
  a.n_q = int(n_q);
  a.n_k = int(n_k);
  a.B = B;
  a.max_q = int(std::min<int64_t>(max_q, n_q));
  a.nh = nh;
  a.rep = nh / nkv;
  a.window = std::min(window, 1 << 30);  // positions stay below 2^30
  a.n_sink = std::min(n_sink, 1 << 30);
  // Two heads that share their keys are an item.  So are two that do not where no sequence has a second query tile,
  // unless there are SMs for every head.  64 x 128 rows, 32 heads: 60 us against 89; 4 x 32, 12 heads: 12 against 11.
  const bool split = a.rep % 2 && nh % 2 == 0 && a.max_q <= kT && int64_t(nh) * B > num_sms();
  a.paired = a.rep % 2 == 0 || split;
  a.n_units = a.paired ? nh / 2 : nh;
  const int rows = a.paired ? kT : 2 * kT;
  a.n_qt = (a.max_q + rows - 1) / rows;
  if (int64_t(a.n_units) * B * a.n_qt > 0x7fffffff) return fail(FG_ERR_SHAPE, "more than 2^31 - 1 query tiles in the batch");
  a.per = uint32_t(a.n_units) * uint32_t(B);
  a.items = a.per * uint32_t(a.n_qt);
  // the lengths are on the device: the profile counts the rows' bytes, no products
  ProfScope ps(PROF_PREFILL_ATTN, s, 0.0, double(n_q) * nh * hd * 4.0 + double(n_k) * nkv * hd * 4.0);
  // Items differ in length and SMs in speed: a CTA that is done takes the next item that has not been started (64 x up
  // to 512 rows, 32 heads: 238 us against 250 with fixed shares; 2 x 8191, window 2048: 525 against 565).  With very many items, most of which may be queries that a shorter sequence does not have,
  // fixed shares are even enough and skipping is cheaper.
  // (The scheduling thread waits for whole items: their length is bounded so that its wait's limit is far away.)
  a.dynamic = a.items > uint32_t(num_sms()) && a.items <= uint32_t(num_sms()) * 64u && n_k <= (1 << 22);
  const dim3 grid(a.dynamic ? a.items : unsigned(std::min<int64_t>(a.items, num_sms())));
  auto* V = reinterpret_cast<const __half*>(v);
#define FG_VARLEN(HD_, SPLIT_)                                                                                      \
  do {                                                                                                              \
    static std::atomic<uint64_t> attr_done{0};                                                                      \
    FG_TRY(ensure_smem_attr(varlen_attn_kernel<HD_, SPLIT_>, VCfg<HD_>::kSmem, attr_done));                         \
    FG_LAUNCH("varlen attention kernel", (varlen_attn_kernel<HD_, SPLIT_>), grid, dim3(kThreads),                   \
              size_t(VCfg<HD_>::kSmem), s, tq, tk, tv, a, V, kv_stride, err);                                       \
  } while (0)
  if (hd == 128) {
    if (split) FG_VARLEN(128, 1);
    else FG_VARLEN(128, 0);
  } else {
    if (split) FG_VARLEN(64, 1);
    else FG_VARLEN(64, 0);
  }
#undef FG_VARLEN
  return FG_OK;
}

}  // namespace fg
