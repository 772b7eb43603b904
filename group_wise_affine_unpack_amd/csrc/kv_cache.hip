// The paged key-value cache in the affine layout: rows quantized as they are
// written, and read back.  A row is one token's key or value of one head
// (D columns): D*bits/32 code words, D/G scales, D/G biases, at
// [page, head, offset] of the cache's arrays, slot = page*page_size + offset.
//   write: per group of G columns the min/max rule of quantize_pack_affine
//          (IEEE fp32, scale and bias stored in the activation type, codes
//          against the stored values), so a cache row holds the bits that
//          quantize_pack_affine gives that row
//   read:  code*scale + bias in fp32 (the product is exact, the sum rounded),
//          then rounded to the activation type
// A slot outside the cache is not written, and reads as zeros.
// One thread per 8 columns (one 16-byte load or store of the dense row); the
// G/8 threads of a group are neighbouring lanes.
#include "common.h"

namespace qaff {
namespace {

template <bool F16_>
__device__ __forceinline__ float act_to_f32(uint32_t bits) {
  return F16_ ? f16_bits_to_f32(bits & 0xffffu) : bf16_bits_to_f32(bits & 0xffffu);
}

template <int BITS, int G, bool F16_>
__global__ __launch_bounds__(256) void kv_append_kernel(KvCache c, const uint16_t* __restrict__ k,
                                                        const uint16_t* __restrict__ v, long kts, long khs, long vts,
                                                        long vhs, const int64_t* __restrict__ slots, uint32_t items,
                                                        FastDiv per_row, FastDiv heads, FastDiv page) {
  // item = ((token * 2 + key or value) * heads + head) * (D/8) + chunk
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= items) return;  // items is a multiple of G/8: groups leave whole
  const uint32_t row = per_row.div(i), ch = i - row * per_row.d;
  const uint32_t tv = heads.div(row), h = row - tv * heads.d;
  const uint32_t tok = tv >> 1;
  const bool is_v = tv & 1;
  const int64_t slot = slots[tok];
  if (slot < 0 || slot >= c.num_slots) return;
  const uint16_t* src = is_v ? v + (long)tok * vts + (long)h * vhs : k + (long)tok * kts + (long)h * khs;
  const u32x4_t raw = *reinterpret_cast<const u32x4_t*>(src + 8 * ch);
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = act_to_f32<F16_>(raw[j / 2] >> (16 * (j & 1)));
  float lo = __builtin_inff(), hi = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    lo = fminf(lo, x[j]);
    hi = fmaxf(hi, x[j]);
  }
#pragma unroll
  for (int o = 1; o < G / 8; o <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, o));
    hi = fmaxf(hi, __shfl_xor(hi, o));
  }
  constexpr float QMAX = (float)((1 << BITS) - 1);
  const uint16_t sb = f32_to_act_bits(__fdiv_rn(__fsub_rn(hi, lo), QMAX), F16_);
  const uint16_t bb = f32_to_act_bits(lo, F16_);
  const float s = act_to_f32<F16_>(sb), b = act_to_f32<F16_>(bb);
  uint32_t q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j)
    q[j] = s != 0.f ? (uint32_t)fminf(fmaxf(rintf(__fdiv_rn(__fsub_rn(x[j], b), s)), 0.f), QMAX) : 0u;
  const uint32_t pg = page.div((uint32_t)slot), off = (uint32_t)slot - pg * page.d;
  const size_t crow = ((size_t)pg * heads.d + h) * page.d + off;  // the cache's row
  uint8_t* codes = (uint8_t*)(is_v ? c.v_packed : c.k_packed) + (crow * per_row.d + ch) * BITS;
  if constexpr (BITS == 8) {
    u32x2_t w;
    w[0] = q[0] | q[1] << 8 | q[2] << 16 | q[3] << 24;
    w[1] = q[4] | q[5] << 8 | q[6] << 16 | q[7] << 24;
    *reinterpret_cast<u32x2_t*>(codes) = w;
  } else {
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) w |= q[j] << (BITS * j);
    if constexpr (BITS == 4)
      *reinterpret_cast<uint32_t*>(codes) = w;
    else
      *reinterpret_cast<uint16_t*>(codes) = (uint16_t)w;
  }
  if (ch % (G / 8) == 0) {
    const size_t g = crow * (per_row.d / (G / 8)) + ch / (G / 8);
    (is_v ? c.v_scales : c.k_scales)[g] = sb;
    (is_v ? c.v_biases : c.k_biases)[g] = bb;
  }
}

template <int BITS, int G, bool F16_>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                      const int64_t* __restrict__ slots, uint32_t items,
                                                      FastDiv per_row, FastDiv heads, FastDiv page) {
  // item = (token * heads + head) * (D/8) + chunk; blockIdx.y = key or value
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= items) return;
  const bool is_v = blockIdx.y;
  const uint32_t row = per_row.div(i), ch = i - row * per_row.d;
  const uint32_t tok = heads.div(row), h = row - tok * heads.d;
  const int64_t slot = slots[tok];
  u32x4_t o = {0u, 0u, 0u, 0u};
  if (slot >= 0 && slot < c.num_slots) {
    const uint32_t pg = page.div((uint32_t)slot), off = (uint32_t)slot - pg * page.d;
    const size_t crow = ((size_t)pg * heads.d + h) * page.d + off;
    const uint8_t* codes = (const uint8_t*)(is_v ? c.v_packed : c.k_packed) + (crow * per_row.d + ch) * BITS;
    const size_t g = crow * (per_row.d / (G / 8)) + ch / (G / 8);
    const float s = act_to_f32<F16_>((is_v ? c.v_scales : c.k_scales)[g]);
    const float b = act_to_f32<F16_>((is_v ? c.v_biases : c.k_biases)[g]);
    uint32_t w[2] = {0u, 0u};
    if constexpr (BITS == 8) {
      const u32x2_t t = *reinterpret_cast<const u32x2_t*>(codes);
      w[0] = t[0];
      w[1] = t[1];
    } else if constexpr (BITS == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(codes);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(codes);
    }
    uint16_t e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint32_t q = BITS == 8 ? (w[j / 4] >> (8 * (j & 3))) & 255u : (w[0] >> (BITS * j)) & ((1u << BITS) - 1u);
      e[j] = f32_to_act_bits(__fmaf_rn((float)q, s, b), F16_);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = (uint32_t)e[2 * j] | (uint32_t)e[2 * j + 1] << 16;
  }
  *reinterpret_cast<u32x4_t*>((is_v ? v : k) + (size_t)i * 8) = o;
}

template <int BITS, int G>
void launch_append_dt(const KvCache& c, const KvRows& r, const int64_t* slots, uint32_t items, hipStream_t s) {
  const dim3 grid((items + 255u) / 256u), block(256);
  const FastDiv row((uint32_t)c.head_dim / 8), heads((uint32_t)c.kv_heads), page((uint32_t)c.page_size);
  if (c.dt == F16)
    hipLaunchKernelGGL((kv_append_kernel<BITS, G, true>), grid, block, 0, s, c, (const uint16_t*)r.k,
                       (const uint16_t*)r.v, r.kts, r.khs, r.vts, r.vhs, slots, items, row, heads, page);
  else
    hipLaunchKernelGGL((kv_append_kernel<BITS, G, false>), grid, block, 0, s, c, (const uint16_t*)r.k,
                       (const uint16_t*)r.v, r.kts, r.khs, r.vts, r.vhs, slots, items, row, heads, page);
}

template <int BITS, int G>
void launch_read_dt(const KvCache& c, const int64_t* slots, void* k, void* v, uint32_t items, hipStream_t s) {
  const dim3 grid((items + 255u) / 256u, 2), block(256);
  const FastDiv row((uint32_t)c.head_dim / 8), heads((uint32_t)c.kv_heads), page((uint32_t)c.page_size);
  if (c.dt == F16)
    hipLaunchKernelGGL((kv_read_kernel<BITS, G, true>), grid, block, 0, s, c, (uint16_t*)k, (uint16_t*)v, slots, items,
                       row, heads, page);
  else
    hipLaunchKernelGGL((kv_read_kernel<BITS, G, false>), grid, block, 0, s, c, (uint16_t*)k, (uint16_t*)v, slots, items,
                       row, heads, page);
}

#define QAFF_KV_CASES(FN, ...)                        \
  switch (c.bits * 1000 + c.G) {                      \
    case 2032: FN<2, 32>(__VA_ARGS__); break;         \
    case 2064: FN<2, 64>(__VA_ARGS__); break;         \
    case 2128: FN<2, 128>(__VA_ARGS__); break;        \
    case 4032: FN<4, 32>(__VA_ARGS__); break;         \
    case 4064: FN<4, 64>(__VA_ARGS__); break;         \
    case 4128: FN<4, 128>(__VA_ARGS__); break;        \
    case 8032: FN<8, 32>(__VA_ARGS__); break;         \
    case 8064: FN<8, 64>(__VA_ARGS__); break;         \
    case 8128: FN<8, 128>(__VA_ARGS__); break;        \
    default: return hipErrorNotSupported;             \
  }

}  // namespace

hipError_t launch_kv_append(const KvCache& c, const KvRows& r, const int64_t* slots, int64_t T, hipStream_t s) {
  const int64_t items = T * 2 * c.kv_heads * (c.head_dim / 8);
  if (items >= (int64_t(1) << 31)) return hipErrorNotSupported;
  QAFF_KV_CASES(launch_append_dt, c, r, slots, (uint32_t)items, s)
  return hipGetLastError();
}

hipError_t launch_kv_read(const KvCache& c, const int64_t* slots, void* k, void* v, int64_t T, hipStream_t s) {
  const int64_t items = T * c.kv_heads * (c.head_dim / 8);
  if (items >= (int64_t(1) << 31)) return hipErrorNotSupported;
  QAFF_KV_CASES(launch_read_dt, c, slots, k, v, (uint32_t)items, s)
  return hipGetLastError();
}

}  // namespace qaff
