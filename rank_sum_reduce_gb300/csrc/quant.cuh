// quant.cuh -- 8-bit (e4m3) output of a normalised row, with its scales.
//
// With t = h * w and y = t * rms (fp32), a group of columns that shares a
// scale s has amax = max |y| = max |t| * rms: rounding to nearest is
// monotonic, so the product of the largest |t| is the largest product.  max
// |t| needs no rms, so it is found before the row statistic's barriers (for a
// row-wide scale it travels with the sum of squares) and the scales cost no
// exchange of their own.
//
// Rounding: s is rounded once to its stored type, q = e4m3(y * (1 / s)) with
// 1 / s rounded once, both in fp32 (two roundings of 2^-24 before the one of
// 2^-4 to e4m3).  The largest |y| of a group lands on 448, or below it for a
// power-of-two s; the conversion saturates.
#pragma once

#include <cuda_fp8.h>

#include <type_traits>

#include "car_device.cuh"

namespace car {

// == car_scale_kind
enum ScaleKind : int { kScaleRow = 0, kScaleGroup128 = 1, kScaleMx32 = 2, kScaleStatic = 3 };

struct QuantOut {
  uint8_t* q;       // [rows, N] e4m3
  void* scales;     // fp32 [rows], fp32 [rows, groups], e8m0 [rows, groups], or fp32 [1] (read)
  int kind;         // ScaleKind
  int groups;       // groups per row (kScaleGroup128, kScaleMx32)
};

constexpr float kE4m3Max = 448.f;

// |t| as bits: unsigned order is the order of magnitudes, infinity and then
// NaN on top, so one integer maximum also carries "not finite".
__device__ __forceinline__ uint32_t abs_bits(float t) { return __float_as_uint(t) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t warp_max(uint32_t m) { return __reduce_max_sync(0xFFFFFFFFu, m); }

// Lanes (each with one 16-byte vector of E elements) that share a scale.
template <int E>
__device__ __forceinline__ int group_lanes(int kind) {
  return (kind == kScaleGroup128 ? 128 : 32) / E;
}

// Maximum over the `lanes` (a power of two) neighbouring lanes of a group.
__device__ __forceinline__ uint32_t group_max(uint32_t m, int lanes) {
  for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  return m;
}

// fp32 scale of a group: amax / 448, at least 2^-126 so that 1 / s is finite;
// NaN when amax is not finite.
__device__ __forceinline__ float scale_f32(float amax) {
  if (!(amax <= 3.402823466e38f)) return __int_as_float(0x7fc00000);
  return fmaxf(__fdiv_rn(amax, kE4m3Max), 1.17549435e-38f);
}

// e8m0 scale: the smallest 2^(k - 127) that is not below amax / 448, 1 <= k;
// 255 (NaN) when amax is not finite.  448 = 1.75 * 2^8, so with amax =
// m * 2^e the exponent is e - 8 for m <= 1.75 and e - 7 above.
__device__ __forceinline__ uint32_t scale_e8m0(float amax) {
  const uint32_t b = __float_as_uint(amax);
  if (b >= 0x7F800000u) return 255u;  // amax >= 0: infinity or NaN (a negative NaN too)
  const int k = (int)(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return k < 1 ? 1u : (uint32_t)k;
}
__device__ __forceinline__ float inverse_e8m0(uint32_t k) {
  return k == 255u ? __int_as_float(0x7fc00000) : __uint_as_float((254u - k) << 23);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Vector `v` (E elements from column v * E) of a row of e4m3 codes.
__device__ __forceinline__ void store_e4m3(uint8_t* row, int v, const float (&y)[8], float inv) {
  uint2 o;
  o.x = e4m3x4(__fmul_rn(y[0], inv), __fmul_rn(y[1], inv), __fmul_rn(y[2], inv), __fmul_rn(y[3], inv));
  o.y = e4m3x4(__fmul_rn(y[4], inv), __fmul_rn(y[5], inv), __fmul_rn(y[6], inv), __fmul_rn(y[7], inv));
  *reinterpret_cast<uint2*>(row + (int64_t)v * 8) = o;
}
__device__ __forceinline__ void store_e4m3(uint8_t* row, int v, const float (&y)[4], float inv) {
  *reinterpret_cast<uint32_t*>(row + (int64_t)v * 4) =
      e4m3x4(__fmul_rn(y[0], inv), __fmul_rn(y[1], inv), __fmul_rn(y[2], inv), __fmul_rn(y[3], inv));
}

// 1 / s for the whole row: its scale from the row's max |t| (stored by the
// one thread that has `first`), or the caller's.  Unused by the group kinds.
__device__ __forceinline__ float row_inverse(const QuantOut& o, int64_t row, float rms, uint32_t tmax, bool first) {
  if (o.kind == kScaleStatic) return __frcp_rn(__ldg(static_cast<const float*>(o.scales)));
  if (o.kind != kScaleRow) return 0.f;
  const float s = scale_f32(__fmul_rn(rms, __uint_as_float(tmax)));
  if (first) static_cast<float*>(o.scales)[row] = s;
  return __frcp_rn(s);
}

// 1 / s of the group that holds vector v, given max |t| of the group; the
// group's first lane stores the scale.
template <int E>
__device__ __forceinline__ float group_inverse(const QuantOut& o, int64_t row, int v, float rms, uint32_t gmax, bool ok) {
  const float amax = __fmul_rn(rms, __uint_as_float(gmax));
  const int lanes = group_lanes<E>(o.kind);
  const bool first = ok && (v & (lanes - 1)) == 0;
  const int64_t at = row * (int64_t)o.groups + v / lanes;
  if (o.kind == kScaleMx32) {
    const uint32_t k = scale_e8m0(amax);
    if (first) static_cast<uint8_t*>(o.scales)[at] = (uint8_t)k;
    return inverse_e8m0(k);
  }
  const float s = scale_f32(amax);
  if (first) static_cast<float*>(o.scales)[at] = s;
  return __frcp_rn(s);
}

}  // namespace car
