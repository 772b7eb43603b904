// The codes of a cache row from its values (kv_cache.hip, rotary.hip).
#pragma once

#include "common.h"

namespace qaff {
namespace {

template <bool F16_>
__device__ __forceinline__ float act_to_f32(uint32_t bits) {
  return F16_ ? f16_bits_to_f32(bits & 0xffffu) : bf16_bits_to_f32(bits & 0xffffu);
}

// minimum or maximum over the G/8 lanes of a group: exchanges inside quads,
// then half-rows and rows mirrored
template <int G, bool MIN>
__device__ __forceinline__ float group_reduce(float v) {
  auto f = [](float a, float b) { return MIN ? fminf(a, b) : fmaxf(a, b); };
  v = f(v, dpp_mov<0xB1>(v));   // quad_perm 1,0,3,2
  v = f(v, dpp_mov<0x4E>(v));   // quad_perm 2,3,0,1
  if (G >= 64) v = f(v, dpp_mov<0x141>(v));  // row_half_mirror
  if (G >= 128) v = f(v, dpp_mov<0x140>(v));  // row_mirror
  return v;
}

// Codes of 8 values of a group from its stored scale and bias, packed:
//   q = clamp(rint((x - b) / s), 0, QMAX), 0 when s == 0.
// The division is d r with r = 1/s, then one correction by the residual,
// q0 + (d - s q0) r.  That is the IEEE quotient of d and s, bit for bit, for
// a scale of at most 11 significant bits whose reciprocal is a normal number:
// the corrected sum is within 3 * 2^-24 units of the last place of d/s before
// its rounding, while d/s, if not a rounding boundary m (25 bits) itself,
// lies at least 2^-12 units from one (|d - s m| is a multiple of the product
// of their last places), and it is never one (s m has 25 bits or more, d
// 24).  Other scales take the IEEE division.
template <int BITS, bool F16_>
__device__ __forceinline__ void codes_of(const float (&x)[8], float s, float b, uint32_t* w) {
  constexpr float QMAX = (float)((1 << BITS) - 1);
  float q[8];
  const float r = __fdiv_rn(1.f, s);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float d = __fsub_rn(x[j], b), q0 = __fmul_rn(d, r);
    q[j] = __fmaf_rn(__fmaf_rn(-s, q0, d), r, q0);
  }
  if (!(s >= 0x1p-90f && s <= 0x1p90f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = s != 0.f ? __fdiv_rn(__fsub_rn(x[j], b), s) : 0.f;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = fminf(fmaxf(rintf(q[j]), 0.f), QMAX);  // (0 for a NaN)
  if constexpr (BITS == 8) {
#pragma unroll
    for (int k = 0; k < 2; ++k)
      w[k] = (uint32_t)q[4 * k] | (uint32_t)q[4 * k + 1] << 8 | (uint32_t)q[4 * k + 2] << 16 | (uint32_t)q[4 * k + 3] << 24;
  } else {
    // four codes at a time as one number, exact in fp32
    constexpr float B = (float)(1 << BITS);
    const auto four = [&](int j) {
      return (uint32_t)__fmaf_rn(__fmaf_rn(__fmaf_rn(q[j + 3], B, q[j + 2]), B, q[j + 1]), B, q[j]);
    };
    w[0] = four(0) | four(4) << (4 * BITS);
  }
}

// Where a thread's 8 columns of a row lie, in units of the cache's arrays.
struct KvRowAt {
  size_t row;         // the cache's row
  uint32_t ch;        // which 8 columns
  uint32_t per_row;   // D/8
};

// Writes 8 columns of a row: the G/8 lanes of a group, neighbours, share its
// minimum and maximum.  x: the values, quiet where they are NaN.
template <int BITS, int G, bool F16_>
__device__ __forceinline__ void write_codes(const float (&x)[8], const KvRowAt& at, uint32_t* packed, uint16_t* scales,
                                            uint16_t* biases) {
  float lo = __builtin_inff(), hi = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = fminf(lo, x[j]);
    hi = fmaxf(hi, x[j]);
  }
  lo = group_reduce<G, true>(lo);
  hi = group_reduce<G, false>(hi);
  const uint16_t sb = f32_to_act_bits(__fdiv_rn(__fsub_rn(hi, lo), (float)((1 << BITS) - 1)), F16_);
  const uint16_t bb = f32_to_act_bits(lo, F16_);
  uint32_t w[2];
  codes_of<BITS, F16_>(x, act_to_f32<F16_>(sb), act_to_f32<F16_>(bb), w);
  uint8_t* codes = (uint8_t*)packed + (at.row * at.per_row + at.ch) * BITS;
  if constexpr (BITS == 8)
    *reinterpret_cast<u32x2_t*>(codes) = u32x2_t{w[0], w[1]};
  else if constexpr (BITS == 4)
    *reinterpret_cast<uint32_t*>(codes) = w[0];
  else
    *reinterpret_cast<uint16_t*>(codes) = (uint16_t)w[0];
  if (at.ch % (G / 8) == 0) {
    const size_t g = at.row * (at.per_row / (G / 8)) + at.ch / (G / 8);
    scales[g] = sb;
    biases[g] = bb;
  }
}

}  // namespace
}  // namespace qaff

// FN<bits, group, is f16>(...) of the cache c
#define QAFF_KV_CASES(FN, ...)                        \
  switch (c.bits * 1000 + c.G) {                      \
    case 2032: c.dt == F16 ? FN<2, 32, true>(__VA_ARGS__) : FN<2, 32, false>(__VA_ARGS__); break; \
    case 2064: c.dt == F16 ? FN<2, 64, true>(__VA_ARGS__) : FN<2, 64, false>(__VA_ARGS__); break; \
    case 2128: c.dt == F16 ? FN<2, 128, true>(__VA_ARGS__) : FN<2, 128, false>(__VA_ARGS__); break; \
    case 4032: c.dt == F16 ? FN<4, 32, true>(__VA_ARGS__) : FN<4, 32, false>(__VA_ARGS__); break; \
    case 4064: c.dt == F16 ? FN<4, 64, true>(__VA_ARGS__) : FN<4, 64, false>(__VA_ARGS__); break; \
    case 4128: c.dt == F16 ? FN<4, 128, true>(__VA_ARGS__) : FN<4, 128, false>(__VA_ARGS__); break; \
    case 8032: c.dt == F16 ? FN<8, 32, true>(__VA_ARGS__) : FN<8, 32, false>(__VA_ARGS__); break; \
    case 8064: c.dt == F16 ? FN<8, 64, true>(__VA_ARGS__) : FN<8, 64, false>(__VA_ARGS__); break; \
    case 8128: c.dt == F16 ? FN<8, 128, true>(__VA_ARGS__) : FN<8, 128, false>(__VA_ARGS__); break; \
    default: return hipErrorNotSupported;             \
  }
