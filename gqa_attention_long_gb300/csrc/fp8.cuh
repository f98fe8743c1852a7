// fp8.cuh — the 8-bit cache format on the device: e4m3 codes with one fp32 scale for each kv head and block of 128 rows
// (column b of [8][Smax/128 + 1]), how a block's scale follows the rows that are appended to it, and a warp's form of the
// norm and rotation of a k row that is about to be encoded.
//
// A block that a call begins gets the power of two s = 2^e, the least with amax <= 448 s (not under 2^-100). Rows that are
// appended to a block keep its scale s if they fit, amax <= 448 s; else it becomes s 2^k for the least k that fits, and the
// rows before them are rounded again, code 2^-k: only the exponent changes, so that a value stays what it was unless it
// falls among e4m3's subnormals (there it moves by at most half of 2^-9 s 2^k). A scale is thus never more than twice what its rows need when
// they came through here, and how often they were moved does not add up in any value's error above those subnormals.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "internal.cuh"
#include "mxfp4.cuh"  // Pair arithmetic
#include "ptx.cuh"

namespace ea {

constexpr float kF8Max = 448.0f;
constexpr int kF8FirstExp = -100;  // of a block's scale before its first row
constexpr int kF8TopExp = 118;     // no scale grows past this exponent (448 times it is still finite): larger values saturate

__device__ __forceinline__ float f8_pow2(int e) {  // |e| <= 126
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}
// How many times scale s (positive, finite) has to be doubled to hold amax.
__device__ __forceinline__ int f8_growth(float amax, float s) {
  const float t = kF8Max * s;
  if (!(amax > t)) return 0;
  const uint32_t a = __float_as_uint(amax), b = __float_as_uint(t);
  const int k = static_cast<int>(a >> 23) - static_cast<int>(b >> 23) + ((a & 0x7FFFFFu) > (b & 0x7FFFFFu) ? 1 : 0);
  return max(0, min(k, kF8TopExp + 127 - static_cast<int>(__float_as_uint(s) >> 23)));
}
__device__ __forceinline__ float f8_grown(float s, int k) {  // s 2^k, k in [0, 218]
  return s * f8_pow2(k >> 1) * f8_pow2(k - (k >> 1));
}
// What the codes of the rows before are multiplied by when their scale is doubled k times (at 2^-60 nothing is left).
__device__ __forceinline__ float f8_shrink(int k) { return f8_pow2(-min(k, 60)); }

// Four values as e4m3 codes, the first in the low byte: nearest, ties to the even code, saturating at 448; NaN is NaN.
__device__ __forceinline__ uint32_t f8_pack4(float a, float b, float c, float d) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// Four codes as numbers (exact).
__device__ __forceinline__ void f8_unpack4(uint32_t w, float (&x)[4]) {
  const float2 a = unpack_f16x2(cvt_f16x2_e4m3x2(static_cast<uint16_t>(w & 0xFFFFu)));
  const float2 b = unpack_f16x2(cvt_f16x2_e4m3x2(static_cast<uint16_t>(w >> 16)));
  x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}
// Four codes times f, rounded to codes again.
__device__ __forceinline__ uint32_t f8_rescale4(uint32_t w, float f) {
  float x[4];
  f8_unpack4(w, x);
  return f8_pack4(x[0] * f, x[1] * f, x[2] * f, x[3] * f);
}
__device__ __forceinline__ uint4 f8_rescale16(uint4 w, float f) {
  return make_uint4(f8_rescale4(w.x, f), f8_rescale4(w.y, f), f8_rescale4(w.z, f), f8_rescale4(w.w, f));
}
// x / s, rounded to nearest: a scale that is a power of two (every one that this library's writers begin) needs no division.
struct F8Quotient {
  float s, inv;
  bool pow2;
  __device__ __forceinline__ explicit F8Quotient(float scale) : s(scale) {
    const uint32_t b = __float_as_uint(scale);
    pow2 = (b & 0x7FFFFFu) == 0u && b >= 0x00800000u && b <= 0x7E000000u;  // 2^-126 .. 2^125, whose inverse is normal
    inv = pow2 ? __uint_as_float(0x7F000000u - b) : 0.f;
  }
  __device__ __forceinline__ float operator()(float x) const { return pow2 ? x * inv : __fdiv_rn(x, s); }
};

// A row's channels in one warp: lane i holds channels 2i, 2i + 1 (x[0], x[1]) and their RoPE partners 64 + 2i, 65 + 2i
// (x[2], x[3]), so that the rotation stays within a lane.
__device__ __forceinline__ void f8_load_row(const __nv_bfloat16* row, int lane, float (&x)[4]) {
  const uint32_t a = *reinterpret_cast<const uint32_t*>(row + 2 * lane), b = *reinterpret_cast<const uint32_t*>(row + 64 + 2 * lane);
  x[0] = __uint_as_float(a << 16);
  x[1] = __uint_as_float(a & 0xFFFF0000u);
  x[2] = __uint_as_float(b << 16);
  x[3] = __uint_as_float(b & 0xFFFF0000u);
}
__device__ __forceinline__ float f8_row_max(const float (&x)[4]) {
  float a = fmaxf(fmaxf(fabsf(x[0]), fabsf(x[1])), fmaxf(fabsf(x[2]), fabsf(x[3])));
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, m));
  return a;
}
// RMS norm and rotation in fp32 (rot: the position's rotations by frequency, cosine x + y, sine z + w).
__device__ __forceinline__ void f8_norm_rope(const float (&x)[4], const float (&g)[4], const float4* rot, int lane, float (&y)[4]) {
  float ss = fmaf(x[0], x[0], x[1] * x[1]) + fmaf(x[2], x[2], x[3] * x[3]);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  const float rs = rsqrtf(ss * (1.0f / kD) + 1e-6f);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float4 a = rot[2 * lane + e];
    const float nl = x[e] * rs * g[e], nh = x[2 + e] * rs * g[2 + e];
    y[e] = fmaf(nl, a.x, -nh * a.z);
    y[2 + e] = fmaf(nh, a.x, nl * a.z);
  }
}
// The same correctly rounded to fp32 but for one in 2^20 (pairs of fp32 numbers, see mxfp4.cuh): a k row is encoded, and one that is off in
// its last bits can land on another code than the formula's.
__device__ __forceinline__ void f8_norm_rope_pair(const float (&x)[4], const float (&g)[4], const float4* rot, int lane, float (&y)[4]) {
  Pair ss = pair_sum(__fmul_rn(x[0], x[0]), __fmul_rn(x[1], x[1])) + pair_sum(__fmul_rn(x[2], x[2]), __fmul_rn(x[3], x[3]));
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1)
    ss = ss + Pair{__shfl_xor_sync(0xffffffffu, ss.h, m), __shfl_xor_sync(0xffffffffu, ss.l, m)};
  const Pair rs = pair_rsqrt_mean(ss);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float4 a = rot[2 * lane + e];
    const Pair cs = {a.x, a.y}, sn = {a.z, a.w};
    const float nl = __fmul_rn(x[e], g[e]), nh = __fmul_rn(x[2 + e], g[2 + e]);
    y[e] = ((cs * nl + -(sn * nh)) * rs).h;
    y[2 + e] = ((cs * nh + sn * nl) * rs).h;
  }
}

// Sums of weights (at most one each, of up to 2^22 rows) times V, codes of at most 448 under scales of up to 2^94, stay under 2^125. V under a larger
// scale is counted times a power of two, `down`, which brings it there; sums that were formed under another one are multiplied by what it
// changed by. At the end the weights' sum is multiplied by it, too, and their reference raised by as much: the sums then stand to each other as they should.
constexpr float kF8TopSum = 0x1p94f;
__device__ __forceinline__ float f8_lower(float scale) {  // scale > kF8TopSum: 2^93 over its power of two
  return f8_pow2(93 + 127 - static_cast<int>(__float_as_uint(scale) >> 23));
}
__device__ __forceinline__ float2 f8_lowered(float2 ml, float down) {
  return make_float2(ml.x + static_cast<float>(127 - static_cast<int>(__float_as_uint(down) >> 23)), ml.y * down);
}

// The sum of a key's eight softmax weights, from its scores and the log2-sum-exps.
__device__ __forceinline__ float f8_weight(const float4& a, const float4& b, const float4& la, const float4& lb) {
  return ((ex2_approx(a.x - la.x) + ex2_approx(a.y - la.y)) + (ex2_approx(a.z - la.z) + ex2_approx(a.w - la.w))) +
         ((ex2_approx(b.x - lb.x) + ex2_approx(b.y - lb.y)) + (ex2_approx(b.z - lb.z) + ex2_approx(b.w - lb.w)));
}
}  // namespace ea
