// quant.cuh -- 8-bit (e4m3) output of a normalised row, with its scales.
//
// With t = h * w and y = t * rms (fp32), a group of columns that shares a
// scale s has amax = max |y| = max |t| * rms: rounding to nearest is
// monotonic, so the product of the largest |t| is the largest product.  max
// |t| needs no rms, so it is found before the row statistic's barriers (for a
// row-wide scale it travels with the sum of squares) and the scales cost no
// exchange of their own.
//
// Rounding: s is stored in fp32 or as a power of two; t * (rms * (1 / s)) is
// formed in fp32 (a few roundings of 2^-24 before the one of 2^-4 to e4m3).
// The largest |y| of a group lands on 448, or below it for a power-of-two s;
// the conversion saturates.
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

// Largest magnitude so far, over two more values; NaN once one is NaN (the
// three-operand form halves the instructions).
__device__ __forceinline__ float max_abs(float m, float a, float b) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
  return r;
}
// As bits, magnitudes order as unsigned integers, with infinity and then NaN
// on top: one integer maximum across lanes also carries "not finite".
__device__ __forceinline__ uint32_t abs_bits(float t) { return __float_as_uint(t) & 0x7FFFFFFFu; }

__device__ __forceinline__ uint32_t warp_max(uint32_t m) { return __reduce_max_sync(0xFFFFFFFFu, m); }

// Lanes, each with one 16-byte vector of E elements, that share a scale.
template <int E, int KIND>
constexpr int kGroupLanes = (KIND == kScaleGroup128 ? 128 : 32) / E;

// Maximum of each m[k] over the neighbouring lanes of its group.
template <int E, int KIND, int VPT>
__device__ __forceinline__ void group_max(uint32_t (&m)[VPT]) {
#pragma unroll
  for (int o = 1; o < kGroupLanes<E, KIND>; o <<= 1) {
#pragma unroll
    for (int k = 0; k < VPT; k++) m[k] = max(m[k], __shfl_xor_sync(0xFFFFFFFFu, m[k], o));
  }
}

// From each vector's own max |t| to its group's (group kinds), or to the
// warp's over all its vectors, which is returned (row scale).
template <int E, int VPT>
__device__ __forceinline__ uint32_t spread_max(int kind, uint32_t (&m)[VPT]) {
  if (kind == kScaleGroup128) {
    group_max<E, kScaleGroup128>(m);
  } else if (kind == kScaleMx32) {
    group_max<E, kScaleMx32>(m);
  } else if (kind == kScaleRow) {
    uint32_t all = 0u;
#pragma unroll
    for (int k = 0; k < VPT; k++) all = max(all, m[k]);
    return warp_max(all);
  }
  return 0u;
}

// fp32 scale of a group: amax / 448 (as a product with 1 / 448: within 2^-23
// of the quotient), at least 2^-126 so that 1 / s is finite; NaN when amax is
// not finite.
__device__ __forceinline__ float scale_f32(float amax) {
  const float s = fmaxf(__fmul_rn(amax, 1.f / kE4m3Max), 1.17549435e-38f);
  return amax <= 3.402823466e38f ? s : __int_as_float(0x7fc00000);
}
// 1 / s of a normal s within one unit of 2^-23, in one instruction.
__device__ __forceinline__ float reciprocal(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return r;
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

// Vector `v` (E elements from column v * E) of a row of e4m3 codes of
// t * rms / s.  The two factors are multiplied first; where that product
// leaves the finite range (a huge rms over a tiny scale) or is NaN, they are
// applied one after the other.
template <int E>
__device__ __forceinline__ void store_e4m3(uint8_t* row, int v, const float (&t)[E], float rms, float inv) {
  const float f = __fmul_rn(rms, inv);
  float y[E];
  if (f <= 3.402823466e38f) {
#pragma unroll
    for (int e = 0; e < E; e++) y[e] = __fmul_rn(t[e], f);
  } else {
#pragma unroll
    for (int e = 0; e < E; e++) y[e] = __fmul_rn(__fmul_rn(t[e], rms), inv);
  }
  if constexpr (E == 8) {
    *reinterpret_cast<uint2*>(row + (int64_t)v * 8) =
        make_uint2(e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7]));
  } else {
    *reinterpret_cast<uint32_t*>(row + (int64_t)v * 4) = e4m3x4(y[0], y[1], y[2], y[3]);
  }
}

// 1 / s for the whole row: its scale from the row's max |t| (stored by the
// one thread that has `first`), or the caller's.  Unused by the group kinds.
__device__ __forceinline__ float row_inverse(const QuantOut& o, int64_t row, float rms, uint32_t tmax, bool first) {
  if (o.kind == kScaleStatic) return __frcp_rn(__ldg(static_cast<const float*>(o.scales)));  // any finite s > 0
  if (o.kind != kScaleRow) return 0.f;
  const float s = scale_f32(__fmul_rn(rms, __uint_as_float(tmax)));
  if (first) static_cast<float*>(o.scales)[row] = s;
  return reciprocal(s);
}

// 1 / s of the group that holds vector v, given max |t| of the group; the
// group's first lane stores the scale.
template <int E>
__device__ __forceinline__ float group_inverse(const QuantOut& o, int64_t row, int v, float rms, uint32_t gmax, bool ok) {
  const float amax = __fmul_rn(rms, __uint_as_float(gmax));
  const int64_t at = row * (int64_t)o.groups;
  if (o.kind == kScaleMx32) {
    constexpr int L = kGroupLanes<E, kScaleMx32>;
    const uint32_t k = scale_e8m0(amax);
    if (ok && v % L == 0) static_cast<uint8_t*>(o.scales)[at + v / L] = (uint8_t)k;
    return inverse_e8m0(k);
  }
  constexpr int L = kGroupLanes<E, kScaleGroup128>;
  const float s = scale_f32(amax);
  if (ok && v % L == 0) static_cast<float*>(o.scales)[at + v / L] = s;
  return reciprocal(s);
}

}  // namespace car
