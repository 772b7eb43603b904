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
// A NaN takes no part in its group's minimum and maximum and gets code 0.
// A slot outside the cache is not written, and reads as zeros.
// One thread per 8 columns (one 16-byte load or store of the dense row); the
// G/8 threads of a group are neighbouring lanes.
#include "common.h"
#include "kv_codes.h"

namespace qaff {
namespace {

struct KvGrid {
  uint32_t items;  // threads' worth of work (a multiple of G/8)
  FastDiv per_row, heads, page;
};

template <int BITS, int G, bool F16_>
__global__ __launch_bounds__(256) void kv_append_kernel(KvCache c, KvRows r, const int64_t* __restrict__ slots,
                                                        KvGrid n) {
  // item = ((token * 2 + key or value) * heads + head) * (D/8) + chunk
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n.items) return;  // (a multiple of G/8: groups leave whole)
  const uint32_t row = n.per_row.div(i), ch = i - row * n.per_row.d;
  const uint32_t tv = n.heads.div(row), h = row - tv * n.heads.d, tok = tv >> 1;
  const bool is_v = tv & 1;
  const int64_t slot = slots[tok];
  const uint16_t* src = is_v ? (const uint16_t*)r.v + (long)tok * r.vts + (long)h * r.vhs
                             : (const uint16_t*)r.k + (long)tok * r.kts + (long)h * r.khs;
  const u32x4_t raw = *reinterpret_cast<const u32x4_t*>(src + 8 * ch);
  if (slot < 0 || slot >= c.num_slots) return;  // (a group's lanes together: they share the token)
  float x[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    x[j] = act_to_f32<F16_>(raw[j / 2] >> (16 * (j & 1)));
    // a signaling NaN would make the minimum so far a NaN, and the next value then the minimum: only quiet ones take no part
    if constexpr (!F16_) x[j] = __builtin_canonicalizef(x[j]);  // (f16's conversion has made them quiet)
  }
  const uint32_t pg = n.page.div((uint32_t)slot), off = (uint32_t)slot - pg * n.page.d;
  const KvRowAt at{((size_t)pg * n.heads.d + h) * n.page.d + off, ch, n.per_row.d};
  write_codes<BITS, G, F16_>(x, at, is_v ? c.v_packed : c.k_packed, is_v ? c.v_scales : c.k_scales,
                             is_v ? c.v_biases : c.k_biases);
}

// U items a thread, a workgroup's width apart, their loads in flight together.
template <int BITS, int G, bool F16_, int U>
__global__ __launch_bounds__(256) void kv_read_kernel(KvCache c, uint16_t* __restrict__ k, uint16_t* __restrict__ v,
                                                      const int64_t* __restrict__ slots, KvGrid n) {
  // item = (token * heads + head) * (D/8) + chunk; blockIdx.y = key or value
  const bool is_v = blockIdx.y;
  const uint8_t* packed = (const uint8_t*)(is_v ? c.v_packed : c.k_packed);
  const uint16_t* scales = is_v ? c.v_scales : c.k_scales;
  const uint16_t* biases = is_v ? c.v_biases : c.k_biases;
  uint32_t ch[U], h[U], w[U][2], sb[U], bb[U];
  int64_t slot[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = min((blockIdx.x * U + u) * 256u + threadIdx.x, n.items - 1);
    const uint32_t row = n.per_row.div(i), tok = n.heads.div(row);
    ch[u] = i - row * n.per_row.d;
    h[u] = row - tok * n.heads.d;
    slot[u] = slots[tok];
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const bool there = slot[u] >= 0 && slot[u] < c.num_slots;
    const uint32_t at = there ? (uint32_t)slot[u] : 0u;  // (slot 0 is read in the place of one outside)
    const uint32_t pg = n.page.div(at), off = at - pg * n.page.d;
    const size_t crow = ((size_t)pg * n.heads.d + h[u]) * n.page.d + off;
    const uint8_t* codes = packed + (crow * n.per_row.d + ch[u]) * BITS;
    const size_t g = crow * (n.per_row.d / (G / 8)) + ch[u] / (G / 8);
    sb[u] = scales[g];
    bb[u] = biases[g];
    if constexpr (BITS == 8) {
      const u32x2_t t = *reinterpret_cast<const u32x2_t*>(codes);
      w[u][0] = t[0];
      w[u][1] = t[1];
    } else if constexpr (BITS == 4) {
      w[u][0] = *reinterpret_cast<const uint32_t*>(codes);
    } else {
      w[u][0] = *reinterpret_cast<const uint16_t*>(codes);
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t i = (blockIdx.x * U + u) * 256u + threadIdx.x;
    if (i >= n.items) break;
    const float s = act_to_f32<F16_>(sb[u]), b = act_to_f32<F16_>(bb[u]);
    u32x4_t o;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t e[2];
#pragma unroll
      for (int k2 = 0; k2 < 2; ++k2) {
        const int m = 2 * j + k2;
        const uint32_t q = BITS == 8 ? (w[u][m / 4] >> (8 * (m & 3))) & 255u : (w[u][0] >> (BITS * m)) & ((1u << BITS) - 1u);
        float value = __fmaf_rn((float)q, s, b);
        // (the compiler would fold it into the rounding to f16 and leave its own out: 8-bit codes, one value in 10^6)
        if constexpr (F16_) asm("" : "+v"(value));
        e[k2] = f32_to_act_bits(value, F16_);
      }
      o[j] = e[0] | e[1] << 16;
    }
    if (slot[u] < 0 || slot[u] >= c.num_slots) o = u32x4_t{0u, 0u, 0u, 0u};
    __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t*>((is_v ? v : k) + (size_t)i * 8));
  }
}

KvGrid grid_of(const KvCache& c, uint32_t items) {
  return KvGrid{items, FastDiv((uint32_t)c.head_dim / 8), FastDiv((uint32_t)c.kv_heads), FastDiv((uint32_t)c.page_size)};
}

template <int BITS, int G, bool F16_>
void launch_append_dt(const KvCache& c, const KvRows& r, const int64_t* slots, uint32_t items, hipStream_t s) {
  hipLaunchKernelGGL((kv_append_kernel<BITS, G, F16_>), dim3((items + 255u) / 256u), dim3(256), 0, s, c, r, slots,
                     grid_of(c, items));
}

template <int BITS, int G, bool F16_>
void launch_read_dt(const KvCache& c, const int64_t* slots, void* k, void* v, uint32_t items, hipStream_t s) {
  const KvGrid n = grid_of(c, items);
  const uint32_t wgs = (items + 255u) / 256u;
  // four items a thread once that leaves every CU eight workgroups of keys or values
  // (65536 tokens, D = 128, 4-bit: 106 us with one, 61 with two, 57 with four, 58 with eight)
  if (wgs <= 1024)
    hipLaunchKernelGGL((kv_read_kernel<BITS, G, F16_, 1>), dim3(wgs, 2), dim3(256), 0, s, c, (uint16_t*)k, (uint16_t*)v,
                       slots, n);
  else
    hipLaunchKernelGGL((kv_read_kernel<BITS, G, F16_, 4>), dim3((wgs + 3) / 4, 2), dim3(256), 0, s, c, (uint16_t*)k,
                       (uint16_t*)v, slots, n);
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
