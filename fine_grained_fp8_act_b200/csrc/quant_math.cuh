// quant_math.cuh -- the per-element arithmetic of the fine-grained FP8
// quantization, shared by the stand-alone quantization kernels and the GEMM
// epilogue that quantizes a layer's output for the next layer (both must give
// the same bits).
//
// scale = max(amax / 448, 2^-126) in correctly rounded float32; UE8M0 keeps
// the smallest power of two >= scale ("Transformers 中的细粒度 FP8 量化 ...",
// §七 补充: float scales round *up* to UE8M0); element = e4m3(RN_f32(x /
// scale')) with a round-to-nearest-even, saturating cast.
#pragma once

#include <cuda_fp8.h>

#include <cstdint>

namespace fg8 {
namespace qm {

constexpr float kMinScale = 1.17549435082228750797e-38f;  // 2^-126

__device__ __forceinline__ float group_scale(float amax) {
  return fmaxf(__fdiv_rn(amax, 448.0f), kMinScale);
}

// Smallest power of two >= s (s a positive normal float) as a UE8M0 byte.
__device__ __forceinline__ uint32_t e8m0_ceil_byte(float s) {
  const uint32_t b = __float_as_uint(s);
  return (b >> 23) + ((b & 0x7FFFFFu) != 0u);
}

// 2^(127 - byte): the exact reciprocal of the UE8M0 scale (byte <= 253).
__device__ __forceinline__ float e8m0_reciprocal(uint32_t byte) { return __uint_as_float((254u - byte) << 23); }

// Correctly rounded float32 a / b from y = RN(1/b): one refinement brings
// q within one ulp of a/b, and a second FMA-based correction step is then
// exact by Markstein's theorem (remainder r = a - q*b computed exactly by the
// FMA; q' = RN(q + r*y)).  The sign of a zero quotient is taken from a.
__device__ __forceinline__ float div_rn_from_rcp(float a, float b, float y) {
  float q = __fmul_rn(a, y);
  float r = __fmaf_rn(-q, b, a);
  q = __fmaf_rn(r, y, q);
  r = __fmaf_rn(-q, b, a);
  q = __fmaf_rn(r, y, q);
  return copysignf(q, a);
}

// The same correctly rounded quotient for two values at once with packed
// f32x2 arithmetic (each lane of FMUL2/FFMA2 rounds exactly like the scalar op).
__device__ __forceinline__ float2 div2_rn_from_rcp(float2 a, float b, float y) {
  const float2 Y = make_float2(y, y), nB = make_float2(-b, -b);
  float2 q = __fmul2_rn(a, Y);
  float2 r = __ffma2_rn(q, nB, a);
  q = __ffma2_rn(r, Y, q);
  r = __ffma2_rn(q, nB, a);
  q = __ffma2_rn(r, Y, q);
  return make_float2(copysignf(q.x, a.x), copysignf(q.y, a.y));
}

__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ void unpack_bf16x8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ float ex2_approx(float x) {  // 2^x, relative error 2^-22; below 2^-126: 0
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp_approx(float x) {  // 1 / x within one ulp, x and 1 / x normal
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// silu(g) * u for two values, in float32: g / (1 + e) * u with e = exp(-g) =
// 2^t.  t = -g log2(e) is carried as a float and its remainder, t = hn - 2 r,
// and 2^t = 2^hn (1 - 2 r ln 2): the remainder would cost |g| 2^-25 of e
// otherwise.  At most some 10 2^-24 relative in all: e 4 (2^-22) and 1/2 for
// its factor, then the sum, the reciprocal (an ulp), two products.  On 16.8M
// normal gates the mean is 0.82 2^-24 and the largest 4.3, where expf and a
// rounded division (torch's float32 form) have 0.71 and 3.5; of 127M codes made
// of either, 189 and 191 differ from the 64-bit ones.  So all kernels take
// the cheap form, and a row's codes do not depend on how many rows there are.
// No finite gate needs a clamp.  Below -88 e overflows to inf, times a
// factor of either sign, and 1 / d is a zero; from -87.336 on, where 1 / d is
// no normal float32, it is 0 already (all of silu's 88 2^-126 there).  Above
// 88 e is 0 and its factor finite: r comes from g log2(e) / 2, which bf16's
// largest values do not overflow.
// NEG: the negated value, by the signs of the constants.
template <bool NEG = false>
__device__ __forceinline__ float2 silu_mul2(float2 g, float2 u) {
  constexpr float kHalfL = 0.721347510814666748046875f;    // log2(e) / 2, rounded to float32
  constexpr float kHalfLLo = 9.62981495558310593435e-9f;   // log2(e) / 2 - kHalfL
  constexpr float k2Ln2 = NEG ? 1.386294361119890618834f : -1.386294361119890618834f;
  constexpr float kOne = NEG ? -1.0f : 1.0f;
  const float2 one = make_float2(kOne, kOne);
  const float2 h = __fmul2_rn(g, make_float2(-kHalfL, -kHalfL));
  const float2 hn = __fadd2_rn(h, h);
  const float2 r = __ffma2_rn(g, make_float2(kHalfLLo, kHalfLLo), __ffma2_rn(g, make_float2(kHalfL, kHalfL), h));
  const float2 e = make_float2(ex2_approx(hn.x), ex2_approx(hn.y));
  const float2 d = __ffma2_rn(e, __ffma2_rn(r, make_float2(k2Ln2, k2Ln2), one), one);
  return __fmul2_rn(__fmul2_rn(g, make_float2(rcp_approx(d.x), rcp_approx(d.y))), u);
}

// group_scale without the division: amax / 448 correctly rounded wherever
// that is a normal float32, since the remainder amax - q 448 is then a multiple
// of 2^-149 below 2^24 of them, exact down to q = 2^-126 (amax = 2^-117.2);
// smaller quotients end at the floor.  An infinite amax (a product past
// float32) stays infinite: its remainder would be NaN, and the floor in its
// place would turn the group into next to nothing.
__device__ __forceinline__ float group_scale_fast(float amax) {
  constexpr float kInv = 1.0f / 448.0f;  // RN(1 / 448)
  const float s = fmaxf(div_rn_from_rcp(amax, 448.0f, kInv), kMinScale);
  return amax < __int_as_float(0x7f800000) ? s : amax;
}

// Codes of values v that float32 arithmetic made (not of given bf16 values),
// which come NEGATED, n = -v.  (Behind the RMS norm 766 and 780 of 105M codes
// differ from the 64-bit ones in float32 torch and here.)  The quotient takes one FMA correction of
// q0 = v y, y the approximate 1/s: q1 = q0 - (q0 s - v) y.  q0 is within 3 ulp
// of v / s, so the correction is right to 2^-21 ulp before q1's rounding: q1
// is v / s where that is a float32 (ties between two codes are kept) and next
// to correctly rounded otherwise.  With n in place of v both steps are plain
// FMAs, and a zero keeps its sign without being given it: for v = -0 the
// correction is (+0)(-y) + (-0) = -0.
template <int FMT, int N>
__device__ __forceinline__ void quantize_negated(const float2 (&n)[N], float s, uint32_t sbyte,
                                                 uint32_t (&codes)[N / 2]) {
  float2 q[N];
  if (FMT == 0) {
    const float y = -rcp_approx(s);
    const float2 Y = make_float2(y, y), S = make_float2(s, s);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 q0 = __fmul2_rn(n[i], Y);
      q[i] = __ffma2_rn(__ffma2_rn(q0, S, n[i]), Y, q0);
    }
  } else {
    const float inv = -e8m0_reciprocal(sbyte);
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = __fmul2_rn(n[i], make_float2(inv, inv));
  }
#pragma unroll
  for (int i = 0; i < N / 2; ++i) codes[i] = pack_e4m3x4(q[2 * i].x, q[2 * i].y, q[2 * i + 1].x, q[2 * i + 1].y);
}

// Quantize 16 values (two 16-byte bf16 loads) with the group's scale;
// returns 16 packed e4m3 bytes.
template <int FMT>
__device__ __forceinline__ uint4 quantize16(const float (&f)[16], float s, uint32_t sbyte) {
  float q[16];
  if (FMT == 0) {
    const float y = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 r = div2_rn_from_rcp(make_float2(f[i], f[i + 1]), s, y);
      q[i] = r.x;
      q[i + 1] = r.y;
    }
  } else {
    const float inv = e8m0_reciprocal(sbyte);  // x * 2^-e is the correctly rounded x / 2^e
    const float2 I = make_float2(inv, inv);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float2 r = __fmul2_rn(make_float2(f[i], f[i + 1]), I);
      q[i] = r.x;
      q[i + 1] = r.y;
    }
  }
  return make_uint4(pack_e4m3x4(q[0], q[1], q[2], q[3]), pack_e4m3x4(q[4], q[5], q[6], q[7]),
                    pack_e4m3x4(q[8], q[9], q[10], q[11]), pack_e4m3x4(q[12], q[13], q[14], q[15]));
}

}  // namespace qm
}  // namespace fg8
