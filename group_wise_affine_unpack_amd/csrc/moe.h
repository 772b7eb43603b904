// A mixture-of-experts block on affine experts for a few tokens: from the
// router's logits to the block's output,
//     y = resid + scale * sum_e p_e  D_e (silu(G_e x) * (U_e x)),
// the sum over a token's top_k experts, every matrix codes * scale + bias in
// groups of G columns.
//
// Kernels: up (routing, G and U, silu: one f32 row h of each chosen pair of
// token and expert), down (D on those rows: one f32 partial row a pair), join
// (a token's pairs added in the order of their logits, the residual, the one
// rounding).  No atomics: the same call gives the same bits.
//
// Routing is done by each workgroup for itself: an expert is a token's r-th
// choice when r others have a larger logit (or the same and a lower index),
// which a wave counts with ballots.  Workgroups run over all experts, or,
// where there are fewer pairs than experts, over the pairs, of which the first
// token's takes the expert.
//
// The products run on the matrix cores for every number of tokens, 16 weight
// rows a tile and 16 rows of x (M = 1 uses one of them: the matrix cores are
// idle anyway, and the codes need no arithmetic of their own).  Codes are
// masked where they lie into f16 pairs, subnormal numbers code * 2^-24 * 2^s;
// the 2^s is taken out of the x entry that meets it.  x is scaled per row by
// a power of two so that its largest entry is near 2^15 and held in f16,
// exact for entries down to 2^-25 of the largest; h, which is f32, as two f16
// rows, high and low part, 22 bits.  Per group of columns the scale
// multiplies the sum of codes * x, the bias the sum of x, both in fp32.
//
// Bound by memory: every chosen expert's weights once.  Wide loads of whole
// 64-byte pieces of 16 rows, four a wave in flight; the parameters of a tile
// and the rows of x lie in LDS.  The four lanes of a row hold 16 bytes each,
// and a matrix instruction takes codes of one group only, so pieces are
// exchanged between lanes (two or four swaps per four words) where a piece
// pair is longer than a group.
#pragma once

#include <algorithm>

#include "common.h"

namespace qaff {
namespace {

constexpr uint32_t MOE_OOB = 0x80000000u;  // past the end of any tile's rows
constexpr int MOE_MAX_M = 256;

__device__ __forceinline__ u32x4_t moe_ld128(__amdgpu_buffer_rsrc_t r, uint32_t off) {
  return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)off, 0, 2));  // streamed once
}

__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}
__device__ __forceinline__ void swap16(uint32_t& a, uint32_t& b) {
  const auto r = __builtin_amdgcn_permlane16_swap(a, b, false, false);
  a = r[0];
  b = r[1];
}

// A span: 64 bytes of a weight row, 16 for each of its four lanes h; NJ
// matrix instructions of 32 codes, lane h holding 8 of them.
template <int BITS, int G>
struct Span {
  static constexpr int CODES = 512 / BITS, NJ = CODES / 32;
  static constexpr int GROUPS = CODES > G ? CODES / G : 1, JPG = NJ / GROUPS;
  static constexpr int PIECE = 128 / BITS;  // codes of 16 bytes
  // 0: a span is within a group; 1: pieces of two lanes; 2: a piece; 3: half a piece (2-bit, G = 32)
  static constexpr int MIX = CODES <= G ? 0 : CODES == 2 * G ? 1 : CODES == 4 * G ? 2 : 3;

  // Columns of instruction j's 8 codes of lane h: four from `lo`, four from `hi`; fragment entry 2i is lo + i, 2i + 1 hi + i.
  __device__ static __forceinline__ void columns(int j, int h, int& lo, int& hi) {
    if constexpr (BITS == 4) {
      lo = MIX == 0 ? h * 32 + j * 8
         : MIX == 1 ? ((h & 1) + 2 * (j >> 1)) * 32 + ((j & 1) + 2 * (h >> 1)) * 8
                    : j * 32 + h * 8;
      hi = lo + 4;
    } else if constexpr (BITS == 8) {
      lo = MIX == 0 ? h * 16 + j * 8 : ((h & 1) + 2 * j) * 16 + (h >> 1) * 8;
      hi = lo + 4;
    } else if constexpr (MIX == 3) {
      lo = (j >> 1) * 64 + (2 * (j & 1) + (h & 1)) * 16 + (h >> 1) * 8;
      hi = lo + 4;
    } else {
      const int w = j >> 1;  // the word, two instructions each
      const int word = MIX == 1 ? ((h & 1) + 2 * (w >> 1)) * 64 + ((w & 1) + 2 * (h >> 1)) * 16 : w * 64 + h * 16;
      lo = word + 4 * (j & 1);
      hi = lo + 8;
    }
  }
  // what entry i of lo and hi is divided by: its code's place in the f16
  __device__ static __forceinline__ float unit(int i) {
    return BITS == 8 ? 1.f : BITS == 4 ? ((i & 1) ? 0x1p-4f : 1.f) : (i == 0 ? 1.f : i == 1 ? 0x1p-2f : i == 2 ? 0x1p-4f : 0x1p-6f);
  }
  // f16 bits of 1 / unit: what a sum of x takes in the place of codes
  __device__ static __forceinline__ uint32_t ones(int i) {
    const uint32_t e = BITS == 8 ? 0 : BITS == 4 ? 4 * (i & 1) : 2 * i;
    return (0x3C00u + (e << 10)) * 0x10001u;
  }

  // the four words of a lane exchanged so that word j (words 2j, 2j + 1 for 8 bits) holds codes of one group in every lane
  __device__ static __forceinline__ void exchange(u32x4_t& w) {
    if constexpr (MIX >= 1) {
      uint32_t a = w[0], b = w[1], c = w[2], d = w[3];
      swap32(a, c);
      swap32(b, d);
      if constexpr (MIX >= 2) {
        swap16(a, b);
        swap16(c, d);
      }
      w = u32x4_t{a, b, c, d};
    }
  }
  // fragment of instruction j; `half` selects the bytes of a half word (MIX 3)
  __device__ static __forceinline__ f16x8_t codes(const u32x4_t& w, int j, uint32_t half) {
    u32x4_t r;
    if constexpr (BITS == 4) {
      const uint32_t t = w[j], u = t >> 8;
      r = u32x4_t{t & 0x000F000Fu, t & 0x00F000F0u, u & 0x000F000Fu, u & 0x00F000F0u};
    } else if constexpr (BITS == 8) {
      const uint32_t a = w[2 * j], b = w[2 * j + 1];  // bytes of a: 0..3, of b: 4..7; 0x0c is a zero
      r = u32x4_t{__builtin_amdgcn_perm(b, a, 0x0c040c00u), __builtin_amdgcn_perm(b, a, 0x0c050c01u),
                  __builtin_amdgcn_perm(b, a, 0x0c060c02u), __builtin_amdgcn_perm(b, a, 0x0c070c03u)};
    } else {
      uint32_t t;
      if constexpr (MIX == 3) {
        uint32_t a = w[j >> 1], b = a;
        swap32(a, b);
        t = __builtin_amdgcn_perm(0u, (j & 1) ? b : a, half);
      } else {
        t = (j & 1) ? w[j >> 1] >> 8 : w[j >> 1];
      }
      r = u32x4_t{t & 0x00030003u, t & 0x000C000Cu, t & 0x00300030u, t & 0x00C000C0u};
    }
    return __builtin_bit_cast(f16x8_t, r);
  }
};

// ---- routing -----------------------------------------------------------

__device__ __forceinline__ float moe_logit(const MoeArgs& a, int m, int e) {
  return load_as_f32(a.logits, (long)m * a.E + e, a.logit_dt);
}

__device__ __forceinline__ float moe_wave_max(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

// Rank of expert e among token m's logits (a NaN counts as minus infinity),
// and its weight before the division by their sum, exp(z - largest).  All of
// a wave's lanes get them.  Rank E: never chosen (minus infinity).
__device__ __forceinline__ int moe_rank(const MoeArgs& a, int m, int e, int lane, float* weight) {
  const float z0 = fmaxf(moe_logit(a, m, e), -__builtin_inff());
  int rank = 0;
  float top = -__builtin_inff();
  for (int i = 0; i < a.E; i += 64) {
    const int o = i + lane;
    const float z = o < a.E ? fmaxf(moe_logit(a, m, o), -__builtin_inff()) : -__builtin_inff();
    rank += __builtin_popcountll(__ballot(o < a.E && (z > z0 || (z == z0 && o < e))));
    top = fmaxf(top, z);
  }
  *weight = expf(z0 - moe_wave_max(top));
  return z0 == -__builtin_inff() ? a.E : rank;
}

// The tokens whose choice is expert e: their pairs (token * top_k + rank) in
// list[0 .. count) in the order of the tokens; all threads get the count.
struct MoeList {
  int list[MOE_MAX_M];
  float weight[MOE_MAX_M];
  int rank[MOE_MAX_M];
  int part[4];
};
__device__ __forceinline__ int moe_tokens(const MoeArgs& a, int e, MoeList& l) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int m = wave; m < a.M; m += 4) {
    float w;
    const int r = moe_rank(a, m, e, lane, &w);
    if (lane == 0) {
      l.rank[m] = r;
      l.weight[m] = w;
    }
  }
  __syncthreads();
  const int m = threadIdx.x;
  const int r = m < a.M ? l.rank[m] : a.E;
  const float w = m < a.M ? l.weight[m] : 0.f;
  const bool mine = r < a.top_k;
  const uint64_t all = __ballot(mine);
  if (lane == 0) l.part[wave] = __builtin_popcountll(all);
  __syncthreads();
  int at = __builtin_popcountll(all & ((1ull << lane) - 1)), count = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (i < wave) at += l.part[i];
    count += l.part[i];
  }
  if (mine) {
    l.list[at] = m * a.top_k + r;
    l.weight[at] = w;
  }
  __syncthreads();
  return count;
}

// the expert that token m chooses r-th, or -1 (every thread gets it); `z` holds E words
__device__ __forceinline__ int moe_choice(const MoeArgs& a, int m, int r, float* z, int* found) {
  if (threadIdx.x == 0) *found = -1;
  for (int e = threadIdx.x; e < a.E; e += 256) z[e] = fmaxf(moe_logit(a, m, e), -__builtin_inff());
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 256) {
    const float z0 = z[e];
    int rank = 0;
    for (int o = 0; o < a.E; ++o) rank += z[o] > z0 || (z[o] == z0 && o < e);
    if (rank == r && z0 > -__builtin_inff()) *found = e;
  }
  __syncthreads();
  return *found;
}

// ---- the product ---------------------------------------------------------

// power of two that brings a row's largest entry into [2^14, 2^15): 1 for a row of zeros, NaN for one that is not finite
__device__ __forceinline__ float moe_row_scale(float amax) {
  if (!(amax <= 0x1.fffffep127f)) return __builtin_nanf("");
  if (amax == 0.f) return 1.f;
  const int e = __builtin_amdgcn_frexp_expf(amax);  // amax in [2^(e-1), 2^e)
  return __builtin_ldexpf(1.f, min(15 - e, 126));
}

// 4 columns of row `src` from column k as floats; zeros from `end` on
template <bool DOWN, bool F16_>
__device__ __forceinline__ void moe_load4(const void* src, int k, int end, float (&v)[4]) {
  if (k >= end) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = 0.f;
  } else if constexpr (DOWN) {
    const f32x4_t t = *reinterpret_cast<const f32x4_t*>((const float*)src + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = t[i];
  } else {
    const u32x2_t t = *reinterpret_cast<const u32x2_t*>((const uint16_t*)src + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t b = (t[i / 2] >> (16 * (i & 1))) & 0xffffu;
      v[i] = F16_ ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
    }
  }
}

// Up (DOWN = false): x rows of the activation type; a tile is 16 rows of G
// and the same 16 of U.  Down: h rows of f32 as two f16 rows each; a tile is
// 32 rows of D.  NI: registers of an output tile in use, 1 for up to four
// rows of x, else 4.  Row v of x (v = 2 token + part in down) is row (v % 4)
// * 4 + v / 4 of the matrix instruction, so that the first four rows' results
// lie in one register.
template <int BITS, int G, bool F16_, int NI, bool DOWN>
__global__ __launch_bounds__(256) void moe_kernel(MoeArgs a, MoeShape s) {
  using S = Span<BITS, G>;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ MoeList l;
  __shared__ float row_scale[16];
  __shared__ int found;
  unsigned char* xs = lds;                                             // [unit][rows][16 bytes]
  uint16_t* prm = reinterpret_cast<uint16_t*>(lds + s.x_bytes);        // [tile][scale, bias][16][groups of a chunk]
  float* red = reinterpret_cast<float*>(lds);                          // [wave][tile][NI][64], after the last chunk

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int slot = blockIdx.y, tile = blockIdx.x;

  // the expert and its tokens
  int e, count;
  if constexpr (DOWN) {
    count = a.counts[2 * slot];
    e = a.counts[2 * slot + 1];
    if (count == 0) return;
    for (int i = threadIdx.x; i < count; i += 256) l.list[i] = a.lists[(long)slot * a.M + i];
    __syncthreads();
  } else {
    e = slot;
    bool take = true;
    int m = 0;
    if (s.pairs) {
      m = slot / a.top_k;
      e = moe_choice(a, m, slot - m * a.top_k, reinterpret_cast<float*>(lds), &found);
      take = e >= 0;
    }
    count = take ? moe_tokens(a, e, l) : 0;
    if (s.pairs && count && l.list[0] / a.top_k != m) count = 0;  // an earlier token's slot takes the expert
    if (tile == 0) {
      if (threadIdx.x == 0) {
        a.counts[2 * slot] = count;
        a.counts[2 * slot + 1] = e;
      }
      for (int i = threadIdx.x; i < count; i += 256) {
        a.lists[(long)slot * a.M + i] = l.list[i];
        a.weights[l.list[i]] = l.weight[i];
      }
    }
    if (count == 0) return;
  }

  const int K = s.K, ng = K / G, row_bytes = K * BITS / 8;
  const int spans = (row_bytes + 63) / 64;
  const int steps = (spans + 3) / 4;   // of four spans, one a wave
  const int rows = DOWN ? a.N : 2 * a.I;  // of an expert's matrix
  const long row0 = (long)e * rows + (DOWN ? 32 * tile : 16 * tile), row1 = row0 + (DOWN ? 16 : a.I);
  const uint32_t* packed = DOWN ? a.down_packed : a.gate_up_packed;
  const uint16_t* scales = DOWN ? a.down_scales : a.gate_up_scales;
  const uint16_t* biases = DOWN ? a.down_biases : a.gate_up_biases;
  const __amdgpu_buffer_rsrc_t rw0 = make_rsrc((const char*)packed + row0 * row_bytes, 16u * (uint32_t)row_bytes);
  const __amdgpu_buffer_rsrc_t rw1 = make_rsrc((const char*)packed + row1 * row_bytes, 16u * (uint32_t)row_bytes);
  const uint32_t woff = (uint32_t)(c * row_bytes + h * 16);
  const uint32_t half = (h >> 1) ? 0x0c030c02u : 0x0c010c00u;
  const f16x8_t ones = __builtin_bit_cast(f16x8_t, u32x4_t{S::ones(0), S::ones(1), S::ones(2), S::ones(3)});
  const int per_pass = DOWN ? s.rows / 2 : s.rows;  // tokens at a time

  auto issue = [&](int step, u32x4_t (&w)[2]) __attribute__((always_inline)) {
    const int at = (4 * step + wave) * 64;
    const uint32_t off = at + h * 16 < row_bytes ? woff + (uint32_t)at : MOE_OOB;
    w[0] = moe_ld128(rw0, off);
    w[1] = moe_ld128(rw1, off);
  };

  for (int first = 0; first < count; first += per_pass) {
    const int tokens = min(per_pass, count - first), vrows = DOWN ? 2 * tokens : tokens;
    u32x4_t w[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) issue(i, w[i]);

    auto source = [&](int t) -> const void* {
      const int pair = l.list[first + t];
      return DOWN ? (const void*)(a.h + (long)pair * a.I) : (const void*)((const uint16_t*)a.x + (long)(pair / a.top_k) * K);
    };
    // the rows' powers of two
    for (int t = wave; t < tokens; t += 4) {
      const void* src = source(t);
      float most = 0.f;
      for (int k = 4 * lane; k < K; k += 256) {
        float v[4];
        moe_load4<DOWN, F16_>(src, k, K, v);
#pragma unroll
        for (int i = 0; i < 4; ++i) most = nan_max(most, fabsf(v[i]));
      }
      most = wave_max_f32(most);
      if (lane == 0) row_scale[t] = moe_row_scale(most);
    }

    const int vrow = min((c >> 2) + 4 * (c & 3), vrows - 1);  // the x row that this lane feeds
    f32x4_t acc[2];
    acc[0] = acc[1] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const unsigned char* xa = xs + (h * s.rows + vrow) * 16;

    auto compute = [&](int at, u32x4_t (&wq)[2]) __attribute__((always_inline)) {
      // `at`: the span's place in the chunk
      S::exchange(wq[0]);
      S::exchange(wq[1]);
#pragma unroll
      for (int g = 0; g < S::GROUPS; ++g) {
        f32x4_t sum = {0.f, 0.f, 0.f, 0.f}, d0 = sum, d1 = sum;
#pragma unroll
        for (int jj = 0; jj < S::JPG; ++jj) {
          const int j = g * S::JPG + jj;
          const f16x8_t x = *reinterpret_cast<const f16x8_t*>(xa + (size_t)(at * S::NJ + j) * 4 * s.rows * 16);
          sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, ones, sum, 0, 0, 0);
          d0 = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, S::codes(wq[0], j, half), d0, 0, 0, 0);
          d1 = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, S::codes(wq[1], j, half), d1, 0, 0, 0);
        }
        const int group = min(at * S::CODES / G + g, s.chunk_groups - 1);
        const uint16_t* p = prm + c * s.chunk_groups + group;
        const int plane = 16 * s.chunk_groups;
        const auto value = [&](int i) {
          const uint32_t b = p[i * plane];
          return F16_ ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
        };
        const float s0 = value(0) * 0x1p24f, b0 = value(1), s1 = value(2) * 0x1p24f, b1 = value(3);
#pragma unroll
        for (int i = 0; i < NI; ++i) {
          acc[0][i] = fmaf(s0, d0[i], fmaf(b0, sum[i], acc[0][i]));
          acc[1][i] = fmaf(s1, d1[i], fmaf(b1, sum[i], acc[1][i]));
        }
      }
    };

    for (int k0 = 0; k0 < steps; k0 += 4) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int k = k0 + u;
        if (k < steps) {
          if (k % s.chunk_steps == 0) {
            // the next chunk of columns: x rows as f16 fragments, and the parameters of both tiles
            const int chunk = k / s.chunk_steps, col0 = chunk * s.chunk_steps * 4 * S::CODES;
            const int units = s.chunk_steps * 4 * S::NJ * 4;
            __syncthreads();
            for (int t = 0; t < tokens; ++t) {
              const void* src = source(t);
              const float sc = row_scale[t];
              for (int un = threadIdx.x; un < units; un += 256) {
                const int hh = un & 3, sj = un >> 2, span = sj / S::NJ, j = sj % S::NJ;
                int lo, hi;
                S::columns(j, hh, lo, hi);
                const int base = col0 + span * S::CODES;
                float va[4], vb[4];
                moe_load4<DOWN, F16_>(src, base + lo, K, va);
                moe_load4<DOWN, F16_>(src, base + hi, K, vb);
                u32x4_t top, low;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float x = va[i] * sc, y = vb[i] * sc;
                  const _Float16 xh = (_Float16)x, yh = (_Float16)y;
                  top[i] = f32_to_f16_bits((float)xh * S::unit(i)) | (uint32_t)f32_to_f16_bits((float)yh * S::unit(i)) << 16;
                  if constexpr (DOWN)
                    low[i] = f32_to_f16_bits((x - (float)xh) * S::unit(i)) |
                             (uint32_t)f32_to_f16_bits((y - (float)yh) * S::unit(i)) << 16;
                }
                unsigned char* dst = xs + ((size_t)un * s.rows + (DOWN ? 2 * t : t)) * 16;
                *reinterpret_cast<u32x4_t*>(dst) = top;
                if constexpr (DOWN) *reinterpret_cast<u32x4_t*>(dst + 16) = low;
              }
            }
            const int gc = s.chunk_groups, g0 = col0 / G;
            if (gc == ng) {  // a tile's rows lie one after the other: whole 16-byte pieces
              for (int i = threadIdx.x; i < 8 * ng; i += 256) {
                const int which = i / (2 * ng), piece = i - which * 2 * ng;
                const uint16_t* src = ((which & 1) ? biases : scales) + ((which >> 1) ? row1 : row0) * ng;
                reinterpret_cast<u32x4_t*>(prm + which * 16 * ng)[piece] = reinterpret_cast<const u32x4_t*>(src)[piece];
              }
            } else {
              for (int i = threadIdx.x; i < 64 * gc; i += 256) {
                const int r = i / gc, gi = i - r * gc, which = r >> 4;
                const uint16_t* src = ((which & 1) ? biases : scales) + (((which >> 1) ? row1 : row0) + (r & 15)) * ng;
                prm[i] = src[min(g0 + gi, ng - 1)];
              }
            }
            __syncthreads();
          }
          compute(4 * (k % s.chunk_steps) + wave, w[u]);
          issue(k + 4, w[u]);
        }
      }
    }

    // the waves' sums
    __syncthreads();
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < NI; ++i) red[((wave * 2 + t) * NI + i) * 64 + lane] = acc[t][i];
    __syncthreads();
    const auto total = [&](int t, int v, int col) {
      float sum = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) sum += red[((q * 2 + t) * NI + (v >> 2)) * 64 + (v & 3) * 16 + col];
      return sum;
    };
    if constexpr (DOWN) {
      for (int i = threadIdx.x; i < 32 * tokens; i += 256) {
        const int t = i >> 5, n = i & 31;
        const float sum = total(n >> 4, 2 * t, n & 15) + total(n >> 4, 2 * t + 1, n & 15);
        a.part[(long)l.list[first + t] * a.N + 32 * tile + n] = sum / row_scale[t];
      }
    } else {
      const int t = threadIdx.x >> 4, n = threadIdx.x & 15;
      if (t < tokens) {
        const float back = 1.f / row_scale[t], g = total(0, t, n) * back, up = total(1, t, n) * back;
        a.h[(long)l.list[first + t] * a.I + 16 * tile + n] = g / (1.f + expf(-g)) * up;
      }
    }
    __syncthreads();
  }
}

template <int BITS, int G, bool F16_>
hipError_t launch_moe_dt(const MoeArgs& a, bool down, hipStream_t st) {
  using S = Span<BITS, G>;
  MoeShape s;
  s.K = down ? a.I : a.N;
  s.pairs = (int64_t)a.M * a.top_k < a.E;
  s.rows = down ? 2 * std::min(a.M, 8) : std::min(a.M, 16);
  const int steps = (s.K * BITS / 8 + 255) / 256;
  // columns a chunk: x and the parameters in at most 48 KiB of LDS
  const int step_bytes = 4 * S::CODES * 2 * s.rows + 64 * 2 * std::max(1, 4 * S::CODES / G);
  const int most = std::max(1, 49152 / step_bytes), chunks = (steps + most - 1) / most;
  s.chunk_steps = (steps + chunks - 1) / chunks;
  s.chunk_groups = chunks == 1 ? s.K / G : s.chunk_steps * 4 * S::CODES / G;
  s.x_bytes = s.chunk_steps * 4 * S::CODES * 2 * s.rows;
  const int ni = s.rows <= 4 ? 1 : 4;
  const int lds = std::max({s.x_bytes + 64 * 2 * s.chunk_groups, 8 * ni * 256, a.E * 4});
  const dim3 grid((unsigned)(down ? a.N / 32 : a.I / 16), (unsigned)(s.pairs ? a.M * a.top_k : a.E));
#define QAFF_MOE(NI, DOWN) hipLaunchKernelGGL((moe_kernel<BITS, G, F16_, NI, DOWN>), grid, dim3(256), lds, st, a, s)
  if (down) {
    if (ni == 1) QAFF_MOE(1, true);
    else QAFF_MOE(4, true);
  } else {
    if (ni == 1) QAFF_MOE(1, false);
    else QAFF_MOE(4, false);
  }
#undef QAFF_MOE
  return hipGetLastError();
}

}  // namespace

template <int BITS>
hipError_t launch_moe_bits(const MoeArgs& a, bool down, hipStream_t st) {
  switch (a.G * 2 + (a.act_dt == F16)) {
    case 64: return launch_moe_dt<BITS, 32, false>(a, down, st);
    case 65: return launch_moe_dt<BITS, 32, true>(a, down, st);
    case 128: return launch_moe_dt<BITS, 64, false>(a, down, st);
    case 129: return launch_moe_dt<BITS, 64, true>(a, down, st);
    case 256: return launch_moe_dt<BITS, 128, false>(a, down, st);
    case 257: return launch_moe_dt<BITS, 128, true>(a, down, st);
    default: return hipErrorNotSupported;
  }
}

}  // namespace qaff
