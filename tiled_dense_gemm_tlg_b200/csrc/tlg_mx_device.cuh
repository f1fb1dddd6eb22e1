// Device-side pieces of the microscaled (MX) operators: element types, the scale of a
// 32-element block, conversion to and from E2M1 (4 bits) and E4M3 (8 bits), the scale
// layout, and the derivatives of the activations.
//
// An MX block is 32 elements along a row and one E8M0 byte b, which stands for 2^(b - 127);
// 0xFF stands for NaN.  Scales sit in tiles of 128 rows x 4 blocks, 512 bytes: byte
// (row, block) of a tile at (row % 32) * 16 + (row / 32) * 4 + block, the order in which the
// tensor core takes them from shared memory, tiles of one 128-row group side by side.
#pragma once

#include <cuda_bf16.h>

#include "tlg_gemm_kernel.cuh"

namespace tlg {

constexpr int kMxBlock = 32;

// Element type codes (the values of tlg_type) and format codes (tlg_mx_format).
constexpr int kTypeF32 = 0, kTypeF16 = 1, kTypeBF16 = 2;
constexpr int kE2M1 = 0, kE4M3 = 1;

template <int T>
constexpr int kTypeBytes = T == kTypeF32 ? 4 : 2;

// Bytes one block of 32 elements takes in a row of Q.
template <int FMT>
constexpr int kBlockBytes = FMT == kE2M1 ? 16 : 32;

__host__ __device__ __forceinline__ int64_t mx_blocks(int64_t cols) {
  return (cols + kMxBlock - 1) / kMxBlock;
}

// Offset of the scale of (row, block) in S; tiles_x = ceil(blocks / 4).
__device__ __forceinline__ int64_t scale_offset(int64_t row, int block, int64_t tiles_x) {
  return ((row >> 7) * tiles_x + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (block & 3);
}

// ------------------------------------------------------------------ element types

// Word j of a lane's elements: one fp32, or two 16-bit elements (the even one low).
template <int T>
__device__ __forceinline__ void unpack2(uint32_t w, float &lo, float &hi) {
  if constexpr (T == kTypeF16) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
    lo = f.x;
    hi = f.y;
  } else {
    lo = __uint_as_float(w << 16);
    hi = __uint_as_float(w & 0xffff0000u);
  }
}

template <int T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  if constexpr (T == kTypeF16) {
    return pack_half2(lo, hi);
  } else {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
  }
}

// A lane's 16 bytes as fp32 values, and back (one rounding).
template <int T, int E>
__device__ __forceinline__ void to_floats(const uint32_t (&w)[4], float (&v)[E]) {
  if constexpr (T == kTypeF32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(w[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) unpack2<T>(w[j], v[2 * j], v[2 * j + 1]);
  }
}

template <int T, int E>
__device__ __forceinline__ void from_floats(const float (&v)[E], uint32_t (&w)[4]) {
  if constexpr (T == kTypeF32) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = pack2<T>(v[2 * j], v[2 * j + 1]);
  }
}

// The larger of m and the magnitudes of w's two elements, each half by itself; a NaN stays.
template <int T>
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t w) {
  uint32_t r;
  if constexpr (T == kTypeF16)
    asm("{\n\t.reg .b32 t;\n\tabs.f16x2 t, %2;\n\tmax.NaN.f16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(m), "r"(w));
  else
    asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %2;\n\tmax.NaN.bf16x2 %0, %1, t;\n\t}" : "=r"(r) : "r"(m), "r"(w));
  return r;
}

// Bits of a 16-bit magnitude as fp32: NaN and infinity stay the largest.
template <int T>
__device__ __forceinline__ uint32_t magnitude_bits(uint32_t half) {
  if constexpr (T == kTypeF16)
    return __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(half))));
  else
    return half << 16;
}

// Bits of the largest magnitude, as fp32, among the elements in w.  As integers they order like
// the values, with infinity and then NaN above every finite one, so a non-finite element shows
// in the result.
template <int T, int N>
__device__ __forceinline__ uint32_t amax_bits(const uint32_t (&w)[N]) {
  uint32_t m = 0;
  if constexpr (T == kTypeF32) {
#pragma unroll
    for (int j = 0; j < N; ++j) m = max(m, w[j] & 0x7fffffffu);
    return m;
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) m = max_abs2<T>(m, w[j]);
    return magnitude_bits<T>(max(m & 0xffffu, m >> 16));
  }
}

// ------------------------------------------------------------------ scale of a block

// The block's scale byte from the bits of its largest magnitude:
//  - E2M1: 2^(floor(log2 amax) - 2), so the largest element lands in [4, 8) and a value above
//    6 saturates.  Choosing the next power where it would saturate costs the other 31
//    elements half of their eight levels to spare one element at most one step.
//  - E4M3: the smallest power of two with amax <= 448 * 2^e.  Its elements have an exponent of
//    their own, so the larger scale costs no precision, and no element saturates.
// Exponents clamp to -127 (an all-zero block too).  A block with a NaN or an infinity gets
// the NaN scale: every element of it reads back as NaN.
template <int FMT>
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax >= 0x7f800000u) return 255u;
  const int f = static_cast<int>(amax >> 23);
  if constexpr (FMT == kE2M1)
    return static_cast<uint32_t>(max(f - 2, 0));
  else
    return static_cast<uint32_t>(max(f - 8 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0), 0));
}

// 2^-e for a finite block's scale byte (e + 127 <= 252, so the result is a normal number).
// For the NaN scale 0: a finite element of such a block is stored as 0.
__device__ __forceinline__ float inverse_scale(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^e, NaN for 0xFF.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  if (byte == 0u) return __uint_as_float(0x00400000u);
  return byte == 255u ? __uint_as_float(0x7fffffffu) : __uint_as_float(byte << 23);
}

// ------------------------------------------------------------------ conversions

// Four values to E2M1 (16 bits), round to nearest even, saturating: element 2i in the low half of byte i.
__device__ __forceinline__ uint32_t to_e2m1x4(const float *v) {
  uint16_t r;
  asm("{\n\t.reg .b8 a, b;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "mov.b16 %0, {a, b};\n\t}"
      : "=h"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
  return r;
}

__device__ __forceinline__ uint32_t to_e2m1x8(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// Four values to E4M3, round to nearest even, saturating.
__device__ __forceinline__ uint32_t to_e4m3x4(const float *v) {
  uint32_t r;
  asm("{\n\t.reg .b16 a, b;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 b, %4, %3;\n\t"
      "mov.b32 %0, {a, b};\n\t}"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]));
  return r;
}

// Four E4M3 elements to fp32 (by way of fp16, which holds every one exactly).
__device__ __forceinline__ void from_e4m3x4(uint32_t w, float *v) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
  unpack2<kTypeF16>(lo, v[0], v[1]);
  unpack2<kTypeF16>(hi, v[2], v[3]);
}

// Four E2M1 elements (the low 16 bits of w) to fp32.
__device__ __forceinline__ void from_e2m1x4(uint32_t w, float *v) {
  uint32_t lo, hi;
  asm("{\n\t.reg .b8 a, b;\n\tmov.b16 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "h"(static_cast<uint16_t>(w)));
  unpack2<kTypeF16>(lo, v[0], v[1]);
  unpack2<kTypeF16>(hi, v[2], v[3]);
}

__device__ __forceinline__ void from_e2m1x8(uint32_t w, float *v) {
  uint32_t p[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(p[0]), "=r"(p[1]), "=r"(p[2]), "=r"(p[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) unpack2<kTypeF16>(p[i], v[2 * i], v[2 * i + 1]);
}

// Bytes a lane's E elements take in Q, and the words that hold them (4 E2M1 elements: half a word).
template <int FMT, int E>
constexpr int kQBytes = FMT == kE2M1 ? E / 2 : E;
template <int FMT, int E>
constexpr int kQWords = (kQBytes<FMT, E> + 3) / 4;

// v times 2^-e, rounded to the format.  The product is exact, or so small that it rounds to 0.
template <int FMT, int E>
__device__ __forceinline__ void encode(const float (&v)[E], float inv, uint32_t (&q)[kQWords<FMT, E>]) {
  float t[E];
#pragma unroll
  for (int j = 0; j < E; j += 2)
    f2_unpack(f2_mul(f2_pack(v[j], v[j + 1]), f2_splat(inv)), t[j], t[j + 1]);
#pragma unroll
  for (int j = 0; j < kQWords<FMT, E>; ++j) {
    if constexpr (FMT == kE4M3)
      q[j] = to_e4m3x4(t + 4 * j);
    else if constexpr (E == 4)
      q[j] = to_e2m1x4(t);
    else
      q[j] = to_e2m1x8(t + 8 * j);
  }
}

template <int FMT, int E>
__device__ __forceinline__ void decode(const uint32_t (&q)[kQWords<FMT, E>], float scale, float (&v)[E]) {
#pragma unroll
  for (int j = 0; j < kQWords<FMT, E>; ++j) {
    if constexpr (FMT == kE4M3)
      from_e4m3x4(q[j], v + 4 * j);
    else if constexpr (E == 4)
      from_e2m1x4(q[j], v);
    else
      from_e2m1x8(q[j], v + 8 * j);
  }
#pragma unroll
  for (int j = 0; j < E; j += 2)
    f2_unpack(f2_mul(f2_pack(v[j], v[j + 1]), f2_splat(scale)), v[j], v[j + 1]);
}

// ------------------------------------------------------------------ activations

// The activation of a lane's values; T is the type the result is stored in (the 16-bit
// types take GELU's shorter fit).
template <int T, int E>
__device__ __forceinline__ void activate_lane(int act, float (&v)[E]) {
  if (act == kActRelu) {
#pragma unroll
    for (int j = 0; j < E; ++j) v[j] = fmaxf(v[j], 0.0f);
  } else if (act == kActGelu) {
#pragma unroll
    for (int j = 0; j < E; j += 2) gelu_erf_2<T != kTypeF32>(v[j], v[j + 1]);
  } else if (act == kActSilu || act == kActGeluTanh) {
    const SigmoidForm f = sigmoid_form(act);
#pragma unroll
    for (int j = 0; j < E; j += 2) sigmoid_form_apply_2(f, v[j], v[j + 1]);
  }
}

// The larger of the two; a NaN stays.
__device__ __forceinline__ float max_nan(float x, float y) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(x), "f"(y));
  return r;
}

// x held to [-limit, limit]; a NaN stays.
__device__ __forceinline__ float clamp_nan(float x, float limit) {
  float r;
  asm("{\n\t.reg .f32 t;\n\tmin.NaN.f32 t, %1, %2;\n\tmax.NaN.f32 %0, t, %3;\n\t}"
      : "=f"(r)
      : "f"(x), "f"(limit), "f"(-limit));
  return r;
}

// GELU'(x) = Phi(x) + x phi(x): with a = |x| and T(a) = Phi(-a) - a phi(a) it is T(a) below 0 and
// 1 - T(a) above.  T(a) = exp(-a^2 / 2) (E(t) - a / sqrt(2 pi)), E a degree-6 polynomial in
// t = 1 / (1 + 0.38 a) (fit_gelu_slope.py beside this file prints it).  Its error is below 2e-7, and
// below 0, where T is taken as it is, at most 1e-5 of T from -2 on: a gradient that is scaled up, or
// a difference 1/2 - (1/2 - T), would show more.  a is held to 14, where the exponential is 0 (an
// infinite a would give 0 times infinity); a NaN stays.
__device__ __forceinline__ constexpr float gelu_slope_coef(int k) {  // lowest degree first
  constexpr float c[7] = {0.000803342089f, 0.139656156f, 0.221370354f, -0.081764549f,
                          0.440671146f, -0.27447772f, 0.0537412576f};
  return c[k];
}

__device__ __forceinline__ void gelu_slope_2(float x0, float x1, float &s0, float &s1) {
  auto mag = [](float x) {
    float r;
    asm("{\n\t.reg .f32 t;\n\tabs.f32 t, %1;\n\tmin.NaN.f32 %0, t, %2;\n\t}" : "=f"(r) : "f"(x), "f"(14.0f));
    return r;
  };
  const uint64_t a = f2_pack(mag(x0), mag(x1));
  float u0, u1, d0, d1;
  f2_unpack(f2_mul(f2_mul(a, f2_splat(-0.72134752044448170f)), a), u0, u1);  // -a^2/2 log2(e)
  f2_unpack(f2_fma(a, f2_splat(0.38f), f2_splat(1.0f)), d0, d1);
  const uint64_t t = f2_pack(rcp_approx(d0), rcp_approx(d1));
  uint64_t p = f2_splat(gelu_slope_coef(6));
#pragma unroll
  for (int k = 5; k >= 0; --k) p = f2_fma(p, t, f2_splat(gelu_slope_coef(k)));
  p = f2_fma(a, f2_splat(-0.39894228040143268f), p);  // -1 / sqrt(2 pi)
  const uint64_t s = f2_mul(p, f2_pack(ex2_approx(u0), ex2_approx(u1)));
  float t0, t1, r0, r1;
  f2_unpack(s, t0, t1);
  f2_unpack(f2_fma(s, f2_splat(-1.0f), f2_splat(1.0f)), r0, r1);
  s0 = x0 < 0.0f ? t0 : r0;
  s1 = x1 < 0.0f ? t1 : r1;
}

// The derivative of x sigmoid(u): s + x s (1 - s) u'(x), with s = 1 / (1 + t), 1 - s = t s,
// t = 2^(-u log2 e).  x is held to where the derivative is 0 or 1 to fp32's last place and t
// still finite, so no product is 0 times infinity (a saved value may read back as infinity: the
// largest fp32 and bf16 values round up to 2^128 in 8 bits); a NaN stays.
//   SiLU: u = x; |x| held to 80.
__device__ __forceinline__ void silu_slope_2(float x0, float x1, float &s0, float &s1) {
  const uint64_t x = f2_pack(clamp_nan(x0, 80.0f), clamp_nan(x1, 80.0f));
  float z0, z1;
  f2_unpack(f2_mul(x, f2_splat(-1.4426950408889634f)), z0, z1);
  const uint64_t t = f2_pack(ex2_approx(z0), ex2_approx(z1));
  float d0, d1;
  f2_unpack(f2_add(t, f2_splat(1.0f)), d0, d1);
  const uint64_t s = f2_pack(rcp_approx(d0), rcp_approx(d1));
  f2_unpack(f2_fma(f2_mul(x, s), f2_mul(t, s), s), s0, s1);
}

//   tanh GELU: u = c (x + 0.044715 x^3), c = 2 sqrt(2/pi); |x| held to 9.5 (u < 77).
__device__ __forceinline__ void gelu_tanh_slope_2(float x0, float x1, float &s0, float &s1) {
  constexpr float kC1 = 1.5957691216057308f, kC3 = 0.044715f * kC1, kNegLog2e = -1.4426950408889634f;
  const uint64_t x = f2_pack(clamp_nan(x0, 9.5f), clamp_nan(x1, 9.5f));
  const uint64_t xx = f2_mul(x, x);
  float z0, z1;
  f2_unpack(f2_mul(x, f2_fma(f2_splat(kC3 * kNegLog2e), xx, f2_splat(kC1 * kNegLog2e))), z0, z1);
  const uint64_t t = f2_pack(ex2_approx(z0), ex2_approx(z1));
  float d0, d1;
  f2_unpack(f2_add(t, f2_splat(1.0f)), d0, d1);
  const uint64_t s = f2_pack(rcp_approx(d0), rcp_approx(d1));
  const uint64_t du = f2_mul(x, f2_fma(f2_splat(3.0f * kC3), xx, f2_splat(kC1)));
  f2_unpack(f2_fma(f2_mul(du, s), f2_mul(t, s), s), s0, s1);
}

// d[j] *= act'(z[j]).  ReLU's derivative at 0 is 0, and d is dropped there whatever it is (an
// infinite d included); a NaN z makes d NaN for every activation but the identity, which leaves d.
template <int E>
__device__ __forceinline__ void slope_lane(int act, const float (&z)[E], float (&d)[E]) {
  if (act == kActRelu) {
#pragma unroll
    for (int j = 0; j < E; ++j) d[j] = z[j] > 0.0f ? d[j] : max_nan(z[j], 0.0f);
  } else if (act == kActGelu) {
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      float s0, s1;
      gelu_slope_2(z[j], z[j + 1], s0, s1);
      f2_unpack(f2_mul(f2_pack(d[j], d[j + 1]), f2_pack(s0, s1)), d[j], d[j + 1]);
    }
  } else if (act == kActSilu) {
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      float s0, s1;
      silu_slope_2(z[j], z[j + 1], s0, s1);
      f2_unpack(f2_mul(f2_pack(d[j], d[j + 1]), f2_pack(s0, s1)), d[j], d[j + 1]);
    }
  } else if (act == kActGeluTanh) {
#pragma unroll
    for (int j = 0; j < E; j += 2) {
      float s0, s1;
      gelu_tanh_slope_2(z[j], z[j + 1], s0, s1);
      f2_unpack(f2_mul(f2_pack(d[j], d[j + 1]), f2_pack(s0, s1)), d[j], d[j + 1]);
    }
  }
}

}  // namespace tlg
