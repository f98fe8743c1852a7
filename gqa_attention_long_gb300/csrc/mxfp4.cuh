// mxfp4.cuh — the 4-bit cache format on the device: E2M1 codes (two to a byte, the lower channel in
// the low nibble) with one power-of-two scale byte e + 127 per 32 channels of a row, its encoder
// and decoder, and the norm and rotation of a k row that is about to be encoded.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "internal.cuh"
#include "ptx.cuh"
#include "rope.cuh"

namespace ea {

constexpr int kMxRowBytes = kD / 2;    // codes of one row
constexpr int kMxRowScales = kD / 32;  // scale bytes of one row: one 32-bit word

// ------------------------------------------------------------------------------- encoder
// e = floor(log2(amax)) - 2, clamped to [-127, 127]; 0 for amax = 0, 127 for an infinite amax.
__device__ __forceinline__ int mx_exponent(float amax) {
  const int f = static_cast<int>(__float_as_uint(amax) >> 23);
  return amax == 0.f ? 0 : f == 255 ? 127 : max(f - 129, -127);
}
// 2^e for e in [-127, 127] (2^-127 is a subnormal).
__device__ __forceinline__ float mx_pow2(int e) {
  return __uint_as_float(e == -127 ? 0x00400000u : static_cast<uint32_t>(e + 127) << 23);
}
// A NaN is encoded as a zero of its sign, and a block's maximum is of its numbers. Two forms of this, by kLook:
// the maximum tells that there is one (it is NaN then), and only so are the values replaced; or every value is
// tested as it is encoded: more instructions (a third of the writer's), but less code, for a row that comes alone
// (one token's attention over 64 layers: 72.8 us, and 73.7 with a look).
template <bool kLook>
__device__ __forceinline__ float mx_max(float a, float b) {
  if (!kLook) return fmaxf(a, b);
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}
template <bool kLook>
__device__ __forceinline__ float mx_amax8(const float (&x)[8]) {
  float d = 0.f;
  if (kLook) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) asm("max.NaN.f32 %0, %0, %1, %2;" : "+f"(d) : "f"(fabsf(x[i])), "f"(fabsf(x[i + 1])));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) d = fmaxf(d, fabsf(x[i]));
  }
  return d;
}
__device__ __forceinline__ void mx_clean8(float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] == x[i] ? x[i] : copysignf(0.f, x[i]);
}
// Eight values times inv = 2^-e, as E2M1 codes: nearest, ties to the even code, saturating at 6; the product is
// exact. With kLook, none is NaN.
template <bool kLook>
__device__ __forceinline__ uint32_t mx_pack8(const float (&x)[8], float inv) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = kLook || x[i] == x[i] ? x[i] * inv : copysignf(0.f, x[i]);
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
  return r;
}

// ------------------------------------------------------------------------------- decoder
// What a scale byte stands for: 2^(b - 127), NaN for 255 (which no encoder here writes).
__device__ __forceinline__ float mx_scale(uint32_t b) {
  return __uint_as_float(b == 0 ? 0x00400000u : b == 255 ? 0x7FC00000u : b << 23);
}
// Eight codes -> four f16 pairs (exact), channels in order.
__device__ __forceinline__ void mx_unpack8(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
__device__ __forceinline__ void mx_values8(uint32_t w, float scale, float (&x)[8]) {
  uint32_t h[4];
  mx_unpack8(w, h);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack_f16x2(h[i]);
    x[2 * i] = f.x * scale;
    x[2 * i + 1] = f.y * scale;
  }
}

// ------------------------------------------------------------------- a k row's norm, rotation and codes
// A k row is normed, rotated, rounded to fp32 and encoded. The encoder has borders (2.5 -> 2, just
// above -> 3), and a row that is off in its last fp32 bits can land on another code than the
// formula's. So the row is formed in fp32 with a bound on its error, and where the bound leaves a code or an
// exponent open (about one row in two hundred), once more as unevaluated sums h + l of two fp32 numbers
// (about 2^-45 relative; Dekker's and Knuth's error-free sums). FP64 arithmetic, 1/60 of the fp32 rate here, would bound the kernels; pairs
// throughout took three times the instructions.
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair pair_fast_sum(float a, float b) {  // |a| >= |b| or a = 0
  const float s = __fadd_rn(a, b);
  return {s, __fadd_rn(b, -__fadd_rn(s, -a))};
}
__device__ __forceinline__ Pair pair_sum(float a, float b) {
  const float s = __fadd_rn(a, b), bb = __fadd_rn(s, -a);
  return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -bb)), __fadd_rn(b, -bb))};
}
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const Pair s = pair_sum(a.h, b.h);
  return pair_fast_sum(s.h, __fadd_rn(s.l, __fadd_rn(a.l, b.l)));
}
__device__ __forceinline__ Pair operator-(Pair a) { return {-a.h, -a.l}; }
__device__ __forceinline__ Pair operator*(Pair a, float b) {
  const float p = __fmul_rn(a.h, b);
  return pair_fast_sum(p, __fmaf_rn(a.l, b, __fmaf_rn(a.h, b, -p)));
}
__device__ __forceinline__ Pair operator*(Pair a, Pair b) {
  const float p = __fmul_rn(a.h, b.h);
  return pair_fast_sum(p, __fmaf_rn(a.h, b.l, __fmaf_rn(a.l, b.h, __fmaf_rn(a.h, b.h, -p))));
}

// 1 / sqrt(ss / 128 + 1e-6)
__device__ __forceinline__ Pair pair_rsqrt_mean(Pair ss) {
  constexpr double kEps = 1e-6;
  constexpr float kEpsHi = static_cast<float>(kEps), kEpsLo = static_cast<float>(kEps - kEpsHi);
  const Pair m = Pair{ss.h * (1.0f / kD), ss.l * (1.0f / kD)} + Pair{kEpsHi, kEpsLo};
  // one Newton step from the hardware estimate r: r (1 + e/2 + 3 e^2 / 8), e = 1 - m r^2
  const float r = rsqrtf(m.h);
  const Pair u = m * (Pair{r, 0.f} * r);
  const float e = __fadd_rn(__fadd_rn(1.0f, -u.h), -u.l);
  return pair_fast_sum(r, r * fmaf(0.375f * e, e, 0.5f * e));
}
// The power of two below a row's largest magnitude.
__device__ __forceinline__ int f16_exponent(float amax) {
  return amax == 0.f ? 0 : min(max(static_cast<int>(__float_as_uint(amax) >> 23) - 127, -126), 126);
}
// A q row held by an octet, times the power of two that puts its largest magnitude in [1, 2), so that f16 holds any gain's
// rows, to 11 bits down to 2^-14 of their largest channel (tensor cores take 16-bit operands beside codes, and a
// rounding of 2^-12 in a score's terms stays under the bf16 output's); factor = scale over that power.
__device__ __forceinline__ void f16_row(float (&yl)[8], float (&yh)[8], float scale, float& factor) {
  float amax = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) amax = fmaxf(amax, fmaxf(fabsf(yl[e]), fabsf(yh[e])));
#pragma unroll
  for (int m = 4; m >= 1; m >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, m));
  const int e = f16_exponent(amax);
  const float inv = mx_pow2(-e);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    yl[k] *= inv;
    yh[k] *= inv;
  }
  factor = scale * mx_pow2(e);
}

// The normed, rotated row rounded to fp32, held by an octet as in norm_rope (lane i: channels [8i, 8i+8) and their
// partners [64+8i, 64+8i+8)); angle(e, cs, sn) gives frequency 8i + e's cosine and sine. A square of a bf16 number,
// and the product of two, is exact in fp32.
template <class Angle>
__device__ __forceinline__ void pair_norm_rope(const float (&xl)[8], const float (&xh)[8], const float (&gl)[8],
                                               const float (&gh)[8], Angle angle, float (&yl)[8], float (&yh)[8]) {
  Pair ss = {0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    ss = ss + Pair{__fmul_rn(xl[e], xl[e]), 0.f};
    ss = ss + Pair{__fmul_rn(xh[e], xh[e]), 0.f};
  }
#pragma unroll
  for (int m = 4; m >= 1; m >>= 1)
    ss = ss + Pair{__shfl_xor_sync(0xffffffffu, ss.h, m), __shfl_xor_sync(0xffffffffu, ss.l, m)};
  const Pair rs = pair_rsqrt_mean(ss);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    Pair cs, sn;
    angle(e, cs, sn);
    const float nl = __fmul_rn(xl[e], gl[e]), nh = __fmul_rn(xh[e], gh[e]);
    yl[e] = ((cs * nl + -(sn * nh)) * rs).h;
    yh[e] = ((cs * nh + sn * nl) * rs).h;
  }
}

// Encodes a row held by an octet: each lane's two words of codes, its blocks' exponents (block i / 4 and 2 + i / 4).
template <bool kLook>
__device__ __forceinline__ void mx_encode_octet(float (&xl)[8], float (&xh)[8], uint32_t& cl, uint32_t& ch, int& el,
                                                int& eh) {
  float al, ah;
  auto blocks_max = [&] {
    al = mx_amax8<kLook>(xl);
    ah = mx_amax8<kLook>(xh);
#pragma unroll
    for (int m = 2; m >= 1; m >>= 1) {
      al = mx_max<kLook>(al, __shfl_xor_sync(0xffffffffu, al, m));
      ah = mx_max<kLook>(ah, __shfl_xor_sync(0xffffffffu, ah, m));
    }
  };
  blocks_max();
  if (kLook && __any_sync(0xffffffffu, al != al || ah != ah)) {
    mx_clean8(xl);
    mx_clean8(xh);
    blocks_max();
  }
  el = mx_exponent(al);
  eh = mx_exponent(ah);
  cl = mx_pack8<kLook>(xl, mx_pow2(-el));
  ch = mx_pack8<kLook>(xh, mx_pow2(-eh));
}

// Norms, rotates and encodes a k row held by an octet (all four octets of the warp do so together): cs, sn in fp32 as in
// norm_rope, angle as in pair_norm_rope.
template <bool kLook, class Angle>
__device__ __forceinline__ void mx_encode_k_octet(const float (&xl)[8], const float (&xh)[8], const float (&gl)[8],
                                                  const float (&gh)[8], const float (&cs)[8], const float (&sn)[8],
                                                  Angle angle, uint32_t& cl, uint32_t& ch, int& el, int& eh) {
  float yl[8], yh[8];
  norm_rope(xl, xh, gl, gh, cs, sn, yl, yh);
  // |n cos| + |n' sin| <= |n| + |n'| = sl: an output is off by less than 2^-18 of it. (The sum of squares: 19
  // additions, 2^-19.7, half of which reaches the root; 2^-22 each for the root, the two products by it and the
  // gain, and the angle's cosine and sine; the rotation's own 2^-24. Under 2^-19 together.) The norm of the
  // rotated pair bounds both terms: |n| + |n'| <= sqrt(2) |(y, y')| <= 1.5 (|y| + |y'|).
  float dl = 0.f, dh, al = mx_amax8<kLook>(yl), ah = mx_amax8<kLook>(yh), d[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    d[e] = (fabsf(yl[e]) + fabsf(yh[e])) * (1.5f * 0x1p-18f);
    dl = fmaxf(dl, d[e]);
  }
#pragma unroll
  for (int m = 2; m >= 1; m >>= 1) {
    al = mx_max<kLook>(al, __shfl_xor_sync(0xffffffffu, al, m));
    ah = mx_max<kLook>(ah, __shfl_xor_sync(0xffffffffu, ah, m));
    dl = fmaxf(dl, __shfl_xor_sync(0xffffffffu, dl, m));
  }
  dh = dl;
  el = mx_exponent(al);
  eh = mx_exponent(ah);
  float a[8], b[8];
  const float il = mx_pow2(-el), ih = mx_pow2(-eh);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a[e] = yl[e] - d[e];
    b[e] = yl[e] + d[e];
  }
  cl = mx_pack8<kLook>(a, il);
  bool open = mx_pack8<kLook>(b, il) != cl;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a[e] = yh[e] - d[e];
    b[e] = yh[e] + d[e];
  }
  ch = mx_pack8<kLook>(a, ih);
  open |= mx_pack8<kLook>(b, ih) != ch;
  open |= mx_exponent(al - dl) != mx_exponent(al + dl) || mx_exponent(ah - dh) != mx_exponent(ah + dh);
  open |= !(al + ah < 1e30f) || !(al > 1e-30f) || !(ah > 1e-30f);  // infinities, NaN and all but zero rows: the long way
  if (__any_sync(0xffffffffu, open)) {
    pair_norm_rope(xl, xh, gl, gh, angle, yl, yh);
    mx_encode_octet<kLook>(yl, yh, cl, ch, el, eh);
  }
}

// Stores such a row as row `row` of a cache, and its values to val (if not null); i: the lane of the octet.
__device__ __forceinline__ void mx_store_octet(uint32_t cl, uint32_t ch, int el, int eh, uint8_t* codes, uint8_t* scales,
                                               size_t row, int i, __nv_bfloat16* val) {
  codes += row * kMxRowBytes;
  *reinterpret_cast<uint32_t*>(codes + 4 * i) = cl;
  *reinterpret_cast<uint32_t*>(codes + 32 + 4 * i) = ch;
  if ((i & 3) == 0) {
    scales += row * kMxRowScales + (i >> 2);
    scales[0] = static_cast<uint8_t>(el + 127);
    scales[2] = static_cast<uint8_t>(eh + 127);
  }
  if (val != nullptr) {
    float x[8];
    mx_values8(cl, mx_pow2(el), x);
    *reinterpret_cast<uint4*>(val + 8 * i) = pack8(x, false);
    mx_values8(ch, mx_pow2(eh), x);
    *reinterpret_cast<uint4*>(val + 64 + 8 * i) = pack8(x, false);
  }
}

}  // namespace ea
