// Append to and read back from the paged 4-bit cache (include/fg.h: fg_paged_append,
// fg_paged_read).
//
// Both move rows between a packed ragged batch and the pages: row r belongs to the sequence b
// with row_start[b] <= r < row_start[b + 1] and to its position pos0[b] + r - row_start[b].  The
// arithmetic is the group quantizer of fg_quantize_pack (quant_common.cuh) and one fused
// multiply-add per value the other way, so both are bound by HBM: 2 B of fp16 per value against
// 0.5 B of code and 4/G B of parameters.  20000 rows of 32 heads of 128 (64 prompts of up to
// 512; 419 MB each way): 107 us to append, 3.9 TB/s, and 69 us to read back, 6.1 TB/s; a decode step's 256 rows
// of 56 heads appended and read: 15 us.  The append's busiest unit are the issue slots (69 %; 257 instructions a thread
// for 16 values, DRAM 44 %); the dense quantizer runs the same arithmetic at 5.2 TB/s in CTAs that stay and loop, while
// every CTA here starts with dependent lookups and a barrier, and stores 8 bytes of codes a thread.
#include <algorithm>

#include "paged_common.cuh"
#include "quant_common.cuh"

namespace fg {
namespace {

constexpr int kThreads = 256;

// The slots of rows r0 .. r0 + ROWS - 1, one warp each: -1 not in the cache, -2 row of no sequence.
template <int ROWS>
__device__ __forceinline__ void find_rows(const PagedView& c, const int32_t* row_start, const int32_t* pos0, int64_t r0,
                                          int64_t n_rows, int64_t (&slot)[ROWS]) {
  static_assert(ROWS <= kThreads / 32, "a warp per row");
  const int warp = threadIdx.x >> 5;
  if (warp >= ROWS) return;
  const int64_t r = r0 + warp;
  int64_t s = -2;
  if (r < n_rows) {
    const int b = row_start ? row_sequence(row_start, c.B, r) : (r < c.B ? int(r) : -1);
    if (b >= 0) {
      const int64_t first = pos0 ? __ldg(pos0 + b) : 0;
      s = page_slot(c, b, first + (row_start ? r - __ldg(row_start + b) : 0));
    }
  }
  if ((threadIdx.x & 31) == 0) slot[warp] = s;
}

// One thread per 16 values of each of ROWS rows, all of whose loads are under way before the first is used;
// blockIdx.y chooses K or V.
template <int HD, int G, int ROWS>
__global__ void __launch_bounds__(kThreads) paged_append_kernel(PagedView c, const __half* __restrict__ k,
                                                                const __half* __restrict__ v, int64_t row_stride,
                                                                int64_t n_rows, const int32_t* __restrict__ row_start,
                                                                const int32_t* __restrict__ pos0) {
  pdl_wait();  // the previous kernel in the stream has finished (see fg_launch)
  __shared__ int64_t slot[ROWS];
  constexpr int TPG = G / 16;
  uint2* codes = reinterpret_cast<uint2*>(blockIdx.y == 0 ? c.kc : c.vc);
  __half2* params = blockIdx.y == 0 ? c.kp : c.vp;
  const int cpr = c.nkv * (HD / 16);  // chunks per row
  const int64_t r0 = int64_t(blockIdx.x) * ROWS;
  const __half* src = (blockIdx.y == 0 ? k : v) + r0 * row_stride;
  const int rows = int(min(int64_t(ROWS), n_rows - r0));
  for (int c0 = 0; c0 < cpr; c0 += kThreads) {
    const int cc = c0 + threadIdx.x;
    uint4 a[ROWS], b[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      a[i] = b[i] = make_uint4(0, 0, 0, 0);
      if (cc < cpr && i < rows) {
        const uint4* p = reinterpret_cast<const uint4*>(src + i * row_stride) + 2 * cc;
        a[i] = __ldg(p);
        b[i] = __ldg(p + 1);
      }
    }
    if (c0 == 0) {  // the rows' places are looked up behind the first loads
      find_rows<ROWS>(c, row_start, pos0, r0, n_rows, slot);
      __syncthreads();
    }
    const int head = cc / (HD / 16), x = cc % (HD / 16);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const GroupQ q = quantize_chunk16<TPG>(a[i], b[i]);  // every lane takes part in the shuffles
      const int64_t s = slot[i];
      if (cc < cpr && s >= 0) {
        const int64_t at = s + (int64_t(head) << c.page_shift);
        codes[at * (HD / 16) + x] = q.words;
        if (x % TPG == 0) params[at * (HD / G) + x / TPG] = q.params;
      }
    }
  }
}

// One thread per 8 values (one code word, one 16-byte store) of each of ROWS rows; blockIdx.y chooses K or V.
template <int HD, int G, int ROWS>
__global__ void __launch_bounds__(kThreads) paged_read_kernel(PagedView c, __half* __restrict__ k, __half* __restrict__ v,
                                                              int64_t row_stride, int64_t n_rows,
                                                              const int32_t* __restrict__ row_start,
                                                              const int32_t* __restrict__ pos0) {
  pdl_wait();  // the previous kernel in the stream has finished (see fg_launch)
  __shared__ int64_t slot[ROWS];
  const uint32_t* codes = reinterpret_cast<const uint32_t*>(blockIdx.y == 0 ? c.kc : c.vc);
  const __half2* params = blockIdx.y == 0 ? c.kp : c.vp;
  const int wpr = c.nkv * (HD / 8);  // code words per row
  const int64_t r0 = int64_t(blockIdx.x) * ROWS;
  __half* dst = (blockIdx.y == 0 ? k : v) + r0 * row_stride;
  find_rows<ROWS>(c, row_start, pos0, r0, n_rows, slot);
  __syncthreads();
  for (int w = threadIdx.x; w < wpr; w += kThreads) {
    const int head = w / (HD / 8), x = w % (HD / 8);
    uint32_t word[ROWS];
    __half2 par[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      word[i] = 0;
      par[i] = __floats2half2_rn(0.f, 0.f);
      if (slot[i] >= 0) {
        const int64_t at = slot[i] + (int64_t(head) << c.page_shift);
        word[i] = codes[at * (HD / 8) + x];
        par[i] = params[at * (HD / G) + x / (G / 8)];
      }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      if (slot[i] == -2) continue;
      uint32_t o[4];
      dequant8(word[i], __high2half2(par[i]), __low2half2(par[i]), o);  // not in the cache: code 0, min 0
      reinterpret_cast<uint4*>(dst + i * row_stride)[w] = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

// Rows per CTA: four where that still leaves several CTAs for every SM (their loads overlap, the lookups are shared),
// else one, so that a decode step's rows are spread over all SMs.  The 20000 rows appended and read: 181 us with four,
// 195 us with two, 263 us with one; 132 rows: 13 us with four, 11 us with one.
bool many_rows(int64_t n_rows) { return n_rows >= int64_t(num_sms()) * 8; }

int check_rows(const fg_paged_cache* c, const void* k, const void* v, int64_t row_stride, int64_t n_rows,
               const int32_t* row_start, const int32_t* pos0) {
  FG_TRY(check_paged(c));
  if (n_rows != 0 && (!k || !v)) return fail(FG_ERR_INVALID_ARG, "null pointer");  // no rows: there may be no buffer
  if (n_rows < 0 || n_rows > 0x7fffffff) return fail(FG_ERR_SHAPE, "bad row count");
  if (row_stride < int64_t(c->n_kv_heads) * c->head_dim || row_stride % 8)
    return fail(FG_ERR_ALIGN, "row_stride must be >= n_kv_heads * head_dim and a multiple of 8");
  if (!aligned16(k) || !aligned16(v)) return fail(FG_ERR_ALIGN, "k and v must be 16-byte aligned");
  if (!aligned4(row_start) || !aligned4(pos0) || !aligned4(c->page_table))
    return fail(FG_ERR_ALIGN, "index arrays must be 4-byte aligned");
  return FG_OK;
}

}  // namespace

int paged_append_impl(const fg_paged_cache* c, const void* k, const void* v, int64_t row_stride, int64_t n_rows,
                      const int32_t* row_start, const int32_t* pos0, cudaStream_t s) {
  FG_TRY(check_rows(c, k, v, row_stride, n_rows, row_start, pos0));
  if (!pos0) return fail(FG_ERR_INVALID_ARG, "null pos0");
  if (!row_start && n_rows > c->B) return fail(FG_ERR_SHAPE, "without row_start there is one row per sequence");
  if (n_rows == 0) return FG_OK;
  const int hd = c->head_dim, G = c->group;
  ProfScope ps(PROF_QUANT, s, 0.0, double(n_rows) * c->n_kv_heads * hd * 2.0 * (2.0 + 0.5 + 4.0 / G));
  const bool many = many_rows(n_rows);
  const dim3 grid(unsigned(many ? (n_rows + 3) / 4 : n_rows), 2);
  const PagedView view = paged_view(c);
  auto* K = reinterpret_cast<const __half*>(k);
  auto* V = reinterpret_cast<const __half*>(v);
#define FG_APPEND(HD_, G_)                                                                                             \
  FG_LAUNCH("paged append kernel", (many ? paged_append_kernel<HD_, G_, 4> : paged_append_kernel<HD_, G_, 1>), grid, \
            dim3(kThreads), size_t(0), s, view, K, V, row_stride, n_rows, row_start, pos0)
  if (hd == 128 && G == 128) FG_APPEND(128, 128);
  else if (hd == 128 && G == 64) FG_APPEND(128, 64);
  else if (hd == 128) FG_APPEND(128, 32);
  else if (G == 64) FG_APPEND(64, 64);
  else FG_APPEND(64, 32);
#undef FG_APPEND
  return FG_OK;
}

int paged_read_impl(const fg_paged_cache* c, int64_t n_rows, const int32_t* row_start, const int32_t* pos0, void* k,
                    void* v, int64_t row_stride, cudaStream_t s) {
  FG_TRY(check_rows(c, k, v, row_stride, n_rows, row_start, pos0));
  if (!row_start) return fail(FG_ERR_INVALID_ARG, "null row_start");
  if (n_rows == 0) return FG_OK;
  const int hd = c->head_dim, G = c->group;
  ProfScope ps(PROF_QUANT, s, 0.0, double(n_rows) * c->n_kv_heads * hd * 2.0 * (2.0 + 0.5 + 4.0 / G));
  const bool many = many_rows(n_rows);
  const dim3 grid(unsigned(many ? (n_rows + 3) / 4 : n_rows), 2);
  const PagedView view = paged_view(c);
  auto* K = reinterpret_cast<__half*>(k);
  auto* V = reinterpret_cast<__half*>(v);
#define FG_READ(HD_, G_)                                                                                         \
  FG_LAUNCH("paged read kernel", (many ? paged_read_kernel<HD_, G_, 4> : paged_read_kernel<HD_, G_, 1>), grid, \
            dim3(kThreads), size_t(0), s, view, K, V, row_stride, n_rows, row_start, pos0)
  if (hd == 128 && G == 128) FG_READ(128, 128);
  else if (hd == 128 && G == 64) FG_READ(128, 64);
  else if (hd == 128) FG_READ(128, 32);
  else if (G == 64) FG_READ(64, 64);
  else FG_READ(64, 32);
#undef FG_READ
  return FG_OK;
}

}  // namespace fg
