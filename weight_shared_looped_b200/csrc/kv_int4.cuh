// The 4-bit KV cache format: one K or V row of a (token, head) in groups of 32
// values, each group asymmetric with an fp16 scale and an fp16 zero point.
//
//   lo, hi = least and largest value of the group (fp16 values, widened to fp32)
//   scale  = fp16, rounded towards zero, of fl32((hi - lo) / 15);   zero = lo
//   code   = clamp(rint(fl32(fl32(x - lo) * fl32(1 / scale))), 0, 15)   (0 when scale == 0)
//   value  = zero + code * scale
//
// Every step is an IEEE fp32 operation, so codes and parameters are a pure
// function of the row: the standalone writer, the prefill append and the
// decode append give the same bits.  The scale is rounded towards zero so that
// no value leaves [lo, hi] (with a scale rounded up, a group that spans the
// fp16 range would read back as infinity).  What that costs at the group's upper
// end, beyond half a step: at most 15 * 2^-10 of a step; for ranges below 15 * 2^-14,
// whose scale is subnormal in fp16, less than 15 * 2^-24 in all (many steps of such a
// group: a range below 15 * 2^-24 has scale 0 and reads back as lo).  A zero point of -0 is stored as +0, which
// keeps the bits independent of the order of the minimum.  A group holding a
// NaN or an infinity gets NaN parameters and codes 0: whoever attends it sees
// NaN, nobody a plausible number.
//
// Layout: code words as the packed INT4 weights have them (word j of a row
// holds elements 8j .. 8j + 7, element 8j + i in bits 4i .. 4i + 3), unsigned;
// parameters one 32-bit pair per group, scale in the low half.
#pragma once

#include <cuda_fp16.h>
#include <math_constants.h>
#include <stdint.h>

namespace tl {

constexpr int kInt4Group = 32;

struct Int4Group {
  float lo, inv;      // code = rint((x - lo) * inv)
  uint32_t param;     // scale | zero << 16
};

// lo, hi: the group's extremes as fp32 (NaN if any value is NaN)
__device__ __forceinline__ Int4Group kv_int4_group(float lo, float hi) {
  Int4Group g;
  const float range = __fsub_rn(hi, lo);
  if (!(range < CUDART_INF_F)) {   // NaN, infinities of either sign
    g.lo = 0.f;
    g.inv = 0.f;
    g.param = 0x7fff7fffu;
    return g;
  }
  const __half s = __float2half_rz(__fdiv_rn(range, 15.0f));
  const float sf = __half2float(s);
  g.lo = lo;
  g.inv = sf > 0.f ? __frcp_rn(sf) : 0.f;
  const __half z = __float2half_rn(__fadd_rn(lo, 0.f));
  g.param = (uint32_t)__half_as_ushort(s) | ((uint32_t)__half_as_ushort(z) << 16);
  return g;
}

// The code of x as the low bits of an integer: adding 1.5 * 2^23 rounds a value of
// [0, 15] to the nearest integer, ties to even, in the low mantissa bits (no
// conversion instruction, of which the GPU has few).  The difference is never
// negative.  Codes of a group with NaN parameters are set to 0 by the caller
// (kv_int4_marked).
constexpr uint32_t kInt4CodeBias = 0x4B400000u;   // the bits of 1.5 * 2^23
__device__ __forceinline__ uint32_t kv_int4_biased(float x, const Int4Group& g) {
  return __float_as_uint(__fadd_rn(fminf(__fmul_rn(__fsub_rn(x, g.lo), g.inv), 15.f), 12582912.f));
}
__device__ __forceinline__ bool kv_int4_marked(const Int4Group& g) { return g.param == 0x7fff7fffu; }

__device__ __forceinline__ uint32_t kv_int4_code(float x, const Int4Group& g) {
  return kv_int4_marked(g) ? 0u : kv_int4_biased(x, g) - kInt4CodeBias;
}

__device__ __forceinline__ uint32_t kv_h2_bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
__device__ __forceinline__ __half2 kv_bits_h2(uint32_t u) { return *reinterpret_cast<__half2*>(&u); }

// The codes in bits 0-3 (LOW) or 4-7 of both halves of x, as an exact fp16
// pair: the nibble becomes the low mantissa bits of 1024 (1024 + c, or
// 1024 + 16 c), and one exact half2 operation takes the rest away.
template <bool LOW>
__device__ __forceinline__ __half2 kv_int4_pair(uint32_t x) {
  uint32_t v;
  if (LOW) {
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(x), "r"(0x000F000Fu), "r"(0x64006400u));
    return __hadd2(kv_bits_h2(v), __float2half2_rn(-1024.f));
  }
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(v) : "r"(x), "r"(0x00F000F0u), "r"(0x64006400u));
  return __hfma2(kv_bits_h2(v), __float2half2_rn(0.0625f), __float2half2_rn(-64.f));
}

// Rotate-half RoPE of the pair (x0, x1) by (cos, sin), with the roundings written out:
// whoever makes a 4-bit entry must make the same one, and left to the compiler two
// kernels fused different products of the second sum.
__device__ __forceinline__ float2 kv_rope(float x0, float x1, float2 cs) {
  return make_float2(__fmaf_rn(x0, cs.x, -__fmul_rn(x1, cs.y)), __fmaf_rn(x0, cs.y, __fmul_rn(x1, cs.x)));
}

// A warp appends one group of a K row and of a V row, lane l holding element l of
// each: eight code words (kc, vc: the group's four) and a parameter pair each.
__device__ __forceinline__ void kv_int4_append_group(__half k, __half v, uint32_t* kc, uint32_t* vc, uint32_t* kp,
                                                     uint32_t* vp) {
  const int lane = threadIdx.x & 31;
  const __half2 kv = __halves2half2(k, v);   // K and V reduced together
  __half2 mn = kv, mx = kv;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    mn = __hmin2_nan(mn, kv_bits_h2(__shfl_xor_sync(0xffffffffu, kv_h2_bits(mn), o)));
    mx = __hmax2_nan(mx, kv_bits_h2(__shfl_xor_sync(0xffffffffu, kv_h2_bits(mx), o)));
  }
  const Int4Group gk = kv_int4_group(__low2float(mn), __low2float(mx));
  const Int4Group gv = kv_int4_group(__high2float(mn), __high2float(mx));
  uint32_t wk = kv_int4_code(__low2float(kv), gk) << (4 * (lane & 7));
  uint32_t wv = kv_int4_code(__high2float(kv), gv) << (4 * (lane & 7));
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) {
    wk |= __shfl_xor_sync(0xffffffffu, wk, o);
    wv |= __shfl_xor_sync(0xffffffffu, wv, o);
  }
  if ((lane & 7) == 0) {
    kc[lane >> 3] = wk;
    vc[lane >> 3] = wv;
  }
  if (lane == 0) {
    *kp = gk.param;
    *vp = gv.param;
  }
}

}  // namespace tl
