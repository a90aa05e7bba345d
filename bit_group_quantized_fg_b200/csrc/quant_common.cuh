// The group quantizer of a 16-value chunk, shared by the quantize/append kernels and by the
// decode attention kernel that appends a step's new token (include/fg.h, fg_quantize_pack:
// mn = min, mx = max with zero extremes as +0, s = fp16(fp32(mx - mn) / 15),
// code = clamp(rint(fp32(x - mn) / s), 0, 15), every code 0 when s == 0).  Both callers get
// the same codes bit for bit.
#pragma once

#include "fg_common.cuh"

namespace fg {
namespace {

struct GroupQ {
  uint2 words;     // 16 packed codes (element i in bits 4i..4i+3 of words.x, then words.y)
  __half2 params;  // {mn, s}
};

// Packed fp32 pairs (sm_100 f32x2 arithmetic: two IEEE fp32 operations, each rounded to
// nearest even, in one instruction).
__device__ __forceinline__ uint64_t f2_pack(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_sub(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// Codes of 16 values by the definition itself: rint(RN(fp32(x - mn) / s)) with the IEEE
// quotient, clamped to 15 (kept out of line: only reached when the fast path is unsure).  A value
// whose quotient is a NaN gets code 15.
__device__ __noinline__ uint2 exact_codes16(uint4 a, uint4 b, float mn, float sf) {
  const __half2* ha = reinterpret_cast<const __half2*>(&a);
  const __half2* hb = reinterpret_cast<const __half2*>(&b);
  uint32_t w[2] = {0u, 0u};
  for (int i = 0; i < 16; ++i) {
    const __half2 pr = (i < 8) ? ha[i / 2] : hb[(i - 8) / 2];
    const float x = (i & 1) ? __high2float(pr) : __low2float(pr);
    const float d = __fsub_rn(x, mn), y = sf == 0.0f ? __fmul_rn(d, 0.0f) : __fdiv_rn(d, sf);
    const int q = y < 15.0f ? __float2int_rn(y) : 15;
    w[i / 8] |= uint32_t(q) << (4 * (i % 8));
  }
  return make_uint2(w[0], w[1]);
}

// The same codes where s is subnormal, s = j 2^-24 with j < 2^10, without a division: fp32(x - mn) < 2^-10 is exact and a
// multiple i 2^-24 too, so i / j is a half-integer or at least 1 / (2 j) > 2^-11 away from every one, and rounding its
// product with 1/s to a multiple of 2^-14 (the last bit of 768 + y) gives the half-integer itself or leaves it on its
// side.  Small values fall on half-integers often: 1 GiB of N(0, 1e-4) takes 280 us (all by division 861), of N(0, 1e-6)
// 378 us (875), of N(0, 1) 286 us.
__device__ __noinline__ uint2 small_codes16(uint4 a, uint4 b, float mn, float sf) {
  const __half2* ha = reinterpret_cast<const __half2*>(&a);
  const __half2* hb = reinterpret_cast<const __half2*>(&b);
  uint32_t w[2] = {0u, 0u};
  const float rcp = __frcp_rn(sf);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const __half2 pr = (i < 8) ? ha[i / 2] : hb[(i - 8) / 2];
    const float x = (i & 1) ? __high2float(pr) : __low2float(pr);
    const float y = __fsub_rn(__fmaf_rn(__fsub_rn(x, mn), rcp, 768.0f), 768.0f);
    const int q = y < 15.0f ? __float2int_rn(y) : 15;
    w[i / 8] |= uint32_t(q) << (4 * (i % 8));
  }
  return make_uint2(w[0], w[1]);
}

// Quantize 16 consecutive values (two 16-byte vectors) that are part of a group spread over
// TPG = G/16 adjacent lanes.  Every lane of the warp must call this (full-mask shuffles).
// min/max run on packed fp16 (comparisons are exact); the scale and the reciprocal are
// computed once per 16 values, the per-value steps on packed fp32 pairs.
template <int TPG>
__device__ __forceinline__ GroupQ quantize_chunk16(uint4 a, uint4 b) {
  const __half2* ha = reinterpret_cast<const __half2*>(&a);
  const __half2* hb = reinterpret_cast<const __half2*>(&b);
  __half2 lo = __hmin2(__hmin2(ha[0], ha[1]), __hmin2(ha[2], ha[3]));
  __half2 hi = __hmax2(__hmax2(ha[0], ha[1]), __hmax2(ha[2], ha[3]));
  lo = __hmin2(lo, __hmin2(__hmin2(hb[0], hb[1]), __hmin2(hb[2], hb[3])));
  hi = __hmax2(hi, __hmax2(__hmax2(hb[0], hb[1]), __hmax2(hb[2], hb[3])));
  float mn = fminf(__low2float(lo), __high2float(lo));
  float mx = fmaxf(__low2float(hi), __high2float(hi));
#pragma unroll
  for (int o = 1; o < TPG; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  mn = __fadd_rn(mn, 0.0f);  // -0 -> +0
  mx = __fadd_rn(mx, 0.0f);
  const __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.0f));
  const float sf = __half2float(s16);
  // The code is rint of r = RN(d / s).  r1 = RN(d * RN(1/s)) differs from r by less than
  // 1.5 * 2^-23 * |r| < 2^-18 (r < 16), so rint(r1) == rint(r) unless r1 lies within 2^-18 of
  // a half-integer; inside the wider 2^-17 window the exact IEEE quotient is used instead.
  // rint is taken by adding 1.5 * 2^23 (for 0 <= r1 < 2^22 the sum's ulp is 1, so the add
  // rounds half to even and the low mantissa bits hold the integer).  A zero scale gets a
  // zero reciprocal, which makes every code 0.
  const float rcp = sf == 0.0f ? 0.0f : __frcp_rn(sf);
  const float kMagic = 12582912.0f;  // 1.5 * 2^23
  const uint64_t MN2 = f2_pack(mn, mn), RCP2 = f2_pack(rcp, rcp), MAG2 = f2_pack(kMagic, kMagic);
  const uint64_t C256 = f2_pack(256.f, 256.f);
  // The integers q stand in T - magic; four of them are put together by exact fp32 sums, magic + q0 + 256 q2 + 16 (q1
  // + 256 q3) < 2^24, whose low half then holds the four codes (1 GiB, group 64: 273 -> 262 us against a minimum, shifts
  // and ORs per code).  That no q passes 15 needs a scale that is not too small: s is (mx - mn) / 15 to
  // 2^-25 at most where it is subnormal, so r <= 15 (1 + 2^-5) < 15.5 from s = 2^-20 on; smaller and infinite scales and
  // NaNs take the paths out of line.
  float worst = 0.f;
  uint32_t four[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    uint64_t T[2], Q[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float2 xf = __half22float2(j < 2 ? ha[2 * j + e] : hb[2 * j + e - 4]);
      const uint64_t R = f2_mul(f2_sub(f2_pack(xf.x, xf.y), MN2), RCP2);
      T[e] = f2_add(R, MAG2);
      Q[e] = f2_sub(T[e], MAG2);
      float f0, f1;
      f2_unpack(f2_sub(R, Q[e]), f0, f1);
      asm("{.reg .f32 x, y;\n\tabs.f32 x, %1;\n\tabs.f32 y, %2;\n\tmax.NaN.f32 %0, %0, x, y;}" : "+f"(worst) : "f"(f0), "f"(f1));
    }
    float t0, t1, q0, q1, lo4, hi4;
    f2_unpack(T[0], t0, t1);
    f2_unpack(Q[0], q0, q1);
    f2_unpack(f2_fma(Q[1], C256, f2_pack(t0, q1)), lo4, hi4);
    four[j] = __float_as_uint(fmaf(hi4, 16.f, lo4));
  }
  GroupQ r;
  r.words = make_uint2(__byte_perm(four[0], four[1], 0x5410), __byte_perm(four[2], four[3], 0x5410));
  const bool usual = sf == 0.0f || (sf >= 9.5367431640625e-07f && sf < INFINITY);  // 2^-20
  if (!(usual && worst <= 0.5f - 7.62939453125e-06f))
    r.words = sf > 0.0f && sf < 6.103515625e-05f ? small_codes16(a, b, mn, sf) : exact_codes16(a, b, mn, sf);  // 2^-14
  r.params = __halves2half2(__float2half_rn(mn), s16);
  return r;
}

}  // namespace
}  // namespace fg
