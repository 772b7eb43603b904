// A mixture-of-experts block on affine experts for a few tokens: from the
// router's logits to the block's output,
//     y = resid + scale * sum_e p_e  D_e (silu(G_e x) * (U_e x)),
// the sum over a token's top_k experts, every matrix codes * scale + bias in
// groups of G columns.
//
// Kernels, for a batch: route (one workgroup: every token's choices, and the
// tokens of every chosen expert), up (G, U and silu: one f32 row h of each pair
// of token and choice), down (D on those rows: one f32 partial row a pair),
// join (a token's pairs added in the order of their logits, the residual, the
// one rounding).  For up to four tokens two: up, each workgroup of which finds
// its expert itself, and down, whose workgroups go through all chosen experts
// and finish y.  No atomics: the same call gives the same bits.
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
// Bound by memory: every chosen expert's weights once.  A wave streams 16 or
// 32 rows of weights in quads of four spans, a span being 64 bytes of every
// row: the loads of a quad are issued while the one before is computed.  The
// parameters of a row's groups come with them, one load a lane: its four lanes
// take the scales and biases of both tiles and hand them round.  A matrix
// instruction takes codes of one group only, so the 16-byte pieces that the
// four lanes of a row hold are exchanged (two or four swaps per four words)
// where a span is longer than a group.  With many rows a wave takes whole rows
// (KS = 1) and x, shared by the workgroup, fills LDS once; with few, or long
// ones, the four waves take a part of the columns each (KS = 4), with their own
// part of x.
#pragma once

#include <algorithm>

#include "common.h"

namespace qaff {
namespace {

constexpr uint32_t MOE_OOB = 0x80000000u;  // past the end of any tile's rows

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
  // f16 bits of 2^-24 / unit, what a sum of x takes in the place of codes (subnormal, as they are)
  __device__ static __forceinline__ uint32_t ones(int i) {
    return (BITS == 8 ? 1u : BITS == 4 ? ((i & 1) ? 16u : 1u) : 1u << (2 * i)) * 0x10001u;
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

// ---- x into LDS -----------------------------------------------------------

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

template <bool DOWN, bool F16_>
__device__ __forceinline__ float moe_amax(const void* src, int k, int end, int step) {
  float most = 0.f;
  for (; k < end; k += step) {
    float v[4];
    moe_load4<DOWN, F16_>(src, k, end, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) most = nan_max(most, fabsf(v[i]));
  }
  return most;
}

// Fragments `from`, from + step, ... below `count` of a row from column col0
// on, times sc: fragment un = (span * NJ + instruction) * 4 + lane quarter lies
// at (un * rows + v) * 16 bytes.  In down a row is two, high and low part.
template <int BITS, int G, bool F16_, bool DOWN>
__device__ __forceinline__ void moe_stage(const void* src, float sc, int col0, int K, int from, int step, int count,
                                          unsigned char* xs, int rows, int v) {
  using S = Span<BITS, G>;
  for (int un = from; un < count; un += step) {
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
    unsigned char* dst = xs + ((size_t)un * rows + v) * 16;
    *reinterpret_cast<u32x4_t*>(dst) = top;
    if constexpr (DOWN) *reinterpret_cast<u32x4_t*>(dst + 16) = low;
  }
}

// ---- the stream of weights ------------------------------------------------

typedef __attribute__((ext_vector_type(2), aligned(4))) uint32_t u32x2_a4;
typedef __attribute__((ext_vector_type(4), aligned(4))) uint32_t u32x4_a4;

// A wave's view of NT tiles of 16 rows of one expert's matrix.
template <int BITS, int G, bool F16_, int NT>
struct Stream {
  using S = Span<BITS, G>;
  static constexpr int QG = 4 * S::CODES / G;  // groups of a quad: 2 to 32
  static constexpr int MPG = G / 32;           // matrix instructions of a group
  static constexpr int COLS = 4 * S::CODES;    // columns of a quad
  struct Quad {
    u32x4_t w[4][NT];
    uint32_t p[QG / 2];  // two groups of this lane's plane: scales, biases of tile 0, of tile 1 by h (of one tile, by h % 2)
  };
  __amdgpu_buffer_rsrc_t rw[NT];
  const uint16_t* plane;
  uint32_t woff;
  int row_bytes, ng, h;

  __device__ __forceinline__ void open(const uint32_t* packed, const uint16_t* scales, const uint16_t* biases, long row0,
                                       long row1, int K, int lane) {
    const int c = lane & 15;
    h = lane >> 4;
    row_bytes = K * BITS / 8;
    ng = K / G;
    rw[0] = make_rsrc((const char*)packed + row0 * row_bytes, 16u * (uint32_t)row_bytes);
    if constexpr (NT == 2) rw[1] = make_rsrc((const char*)packed + row1 * row_bytes, 16u * (uint32_t)row_bytes);
    woff = (uint32_t)(c * row_bytes + h * 16);
    plane = ((h & 1) ? biases : scales) + ((NT == 2 && (h >> 1) ? row1 : row0) + c) * ng;
  }

  __device__ __forceinline__ void load(int q, Quad& d) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = (4 * q + i) * 64;
      const uint32_t off = at + h * 16 < row_bytes ? woff + (uint32_t)at : MOE_OOB;  // (past a row's end: zeros)
#pragma unroll
      for (int t = 0; t < NT; ++t) d.w[i][t] = moe_ld128(rw[t], off);
    }
    const int g0 = q * QG;
    if (g0 + QG <= ng && !(ng & 1)) {  // (rows of an odd number of groups start between words)
      const uint16_t* p = plane + g0;
      if constexpr (QG == 2) {
        d.p[0] = *reinterpret_cast<const uint32_t*>(p);
      } else if constexpr (QG == 4) {
        const u32x2_a4 v = *reinterpret_cast<const u32x2_a4*>(p);
        d.p[0] = v[0];
        d.p[1] = v[1];
      } else {
#pragma unroll
        for (int i = 0; i < QG / 8; ++i) {
          const u32x4_a4 v = reinterpret_cast<const u32x4_a4*>(p)[i];
#pragma unroll
          for (int k = 0; k < 4; ++k) d.p[4 * i + k] = v[k];
        }
      }
    } else {  // a row's last group in the place of those behind it, which meet codes and x of zero
#pragma unroll
      for (int i = 0; i < QG / 2; ++i)
        d.p[i] = plane[min(g0 + 2 * i, ng - 1)] | (uint32_t)plane[min(g0 + 2 * i + 1, ng - 1)] << 16;
    }
  }

  // acc += quad times x; xa: this lane's x of the quad's first fragment, `stride` bytes from one instruction to the next
  template <int NI>
  __device__ __forceinline__ void compute(Quad& d, const unsigned char* xa, int stride, float (&acc)[NT][NI]) const {
    const uint32_t half = (h >> 1) ? 0x0c030c02u : 0x0c010c00u;
    const f16x8_t ones = __builtin_bit_cast(f16x8_t, u32x4_t{S::ones(0), S::ones(1), S::ones(2), S::ones(3)});
    uint32_t pl[2 * NT];
#pragma unroll
    for (int gi = 0; gi < QG; ++gi) {
      if ((gi & 1) == 0) {
        uint32_t a = d.p[gi / 2];
        if constexpr (NT == 2) {
          uint32_t b = a;
          swap32(a, b);
          pl[2] = pl[3] = b;
          swap16(pl[2], pl[3]);
        }
        pl[0] = pl[1] = a;
        swap16(pl[0], pl[1]);
      }
      f32x4_t sum = {0.f, 0.f, 0.f, 0.f}, dot[NT];
#pragma unroll
      for (int t = 0; t < NT; ++t) dot[t] = sum;
#pragma unroll
      for (int jj = 0; jj < MPG; ++jj) {
        const int mm = gi * MPG + jj, sp = mm / S::NJ, j = mm % S::NJ;
        if (j == 0) {
#pragma unroll
          for (int t = 0; t < NT; ++t) S::exchange(d.w[sp][t]);
        }
        const f16x8_t x = *reinterpret_cast<const f16x8_t*>(xa + mm * stride);
        sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, ones, sum, 0, 0, 0);
#pragma unroll
        for (int t = 0; t < NT; ++t)
          dot[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(x, S::codes(d.w[sp][t], j, half), dot[t], 0, 0, 0);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const auto value = [&](uint32_t v) {
          const uint32_t b = (gi & 1) ? v >> 16 : v & 0xffffu;
          return F16_ ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
        };
        const float s = value(pl[2 * t]), b = value(pl[2 * t + 1]);
#pragma unroll
        for (int i = 0; i < NI; ++i) acc[t][i] = fmaf(s, dot[t][i], fmaf(b, sum[i], acc[t][i]));
      }
    }
  }
};

// acc += quads [q0, q1) of the stream, x from LDS (xa as in compute, for quad q0)
template <int NI, class St, int NT>
__device__ __forceinline__ void moe_quads(const St& st, int q0, int q1, typename St::Quad& a, const unsigned char* xa, int stride,
                                          float (&acc)[NT][NI]) {
  // `a` holds quad q0 already
  typename St::Quad b;
  const int quad = St::QG * St::MPG * stride;
  for (int q = q0; q < q1; q += 2, xa += 2 * quad) {
    if (q + 1 < q1) st.load(q + 1, b);
    st.template compute<NI>(a, xa, stride, acc);
    if (q + 1 < q1) {
      if (q + 2 < q1) st.load(q + 2, a);
      st.template compute<NI>(b, xa + quad, stride, acc);
    }
  }
}

// ---- routing of a few tokens ----------------------------------------------

constexpr int MOE_FEW = 4;  // tokens whose experts each workgroup finds for itself

// The r-th choice of token m, found by every workgroup of its slot: the expert
// and the pairs of the tokens that chose it too, when m is the first of them.
// z: [M, E] logits in LDS.  The slot's first workgroup leaves what down needs.
struct MoeFew {
  int found, count;
  int list[MOE_FEW], rank[MOE_FEW];
  float weight[MOE_FEW];
  float part[4];
  int cpart[4];
};
__device__ __forceinline__ int moe_find(const MoeArgs& a, int slot, bool leave, float* z, MoeFew& l) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int m = slot / a.top_k, r = slot - m * a.top_k;
  bool nan = false;
  if (threadIdx.x == 0) l.found = -1;
  for (int i = threadIdx.x; i < a.M * a.E; i += 256) {
    const float v = load_as_f32(a.logits, i, a.logit_dt);
    z[i] = v == v ? v : -__builtin_inff();
    nan |= v != v && i / a.E == m;
  }
  __syncthreads();
  // every expert's place among token m's
  const float* zm = z + m * a.E;
  float sum = 0.f, top = -__builtin_inff();
  int chosen = 0;
  const bool meta = leave && r == 0;
  if (meta) {
    for (int o = 0; o < a.E; ++o) top = fmaxf(top, zm[o]);
  }
  for (int e = threadIdx.x; e < a.E; e += 256) {
    const float z0 = zm[e];
    int rank = 0;
    for (int o = 0; o < a.E; ++o) rank += zm[o] > z0 || (zm[o] == z0 && o < e);
    const bool there = z0 > -__builtin_inff();
    if (rank == r && there) l.found = e;
    if (there && (rank < a.top_k || !a.renormalize)) sum += expf(z0 - top);
    chosen += there && rank < a.top_k;
  }
  if (meta) {  // token m's number of choices, and what its weights are divided by
    sum = wave_sum(sum);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) chosen += __shfl_xor(chosen, d);
    nan = __ballot(nan) != 0;
    if (lane == 0) {
      l.part[wave] = nan ? __builtin_nanf("") : sum;
      l.cpart[wave] = chosen;
    }
  }
  __syncthreads();
  if (meta && threadIdx.x == 0) {
    a.sums[m] = l.part[0] + l.part[1] + l.part[2] + l.part[3];
    a.choices[m] = l.cpart[0] + l.cpart[1] + l.cpart[2] + l.cpart[3];
  }
  const int e = l.found;
  if (wave < a.M && e >= 0) {  // where token `wave` has the expert
    const float* zt = z + wave * a.E;
    const float z0 = zt[e];
    int rank = 0;
    float most = -__builtin_inff();
    for (int i = 0; i < a.E; i += 64) {
      const int o = i + lane;
      const float v = o < a.E ? zt[o] : -__builtin_inff();
      rank += __builtin_popcountll(__ballot(o < a.E && (v > z0 || (v == z0 && o < e))));
      most = fmaxf(most, v);
    }
    most = wave_max_f32(most);
    if (lane == 0) {
      l.rank[wave] = z0 > -__builtin_inff() ? rank : a.E;
      l.weight[wave] = expf(z0 - most);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    int count = 0, first = -1;
    for (int t = 0; t < a.M && e >= 0; ++t)
      if (l.rank[t] < a.top_k) {
        if (first < 0) first = t;
        l.list[count] = t * a.top_k + l.rank[t];
        if (leave) a.weights[t * a.top_k + l.rank[t]] = l.weight[t];
        ++count;
      }
    l.count = first == m ? count : 0;  // (else an earlier token's slot takes the expert)
    if (leave) {
      a.counts[2 * slot] = l.count;
      a.counts[2 * slot + 1] = e;
      for (int i = 0; i < l.count; ++i) a.lists[slot * a.M + i] = l.list[i];
    }
  }
  __syncthreads();
  return e;
}

// ---- kernels ---------------------------------------------------------------

// Up (DOWN = false): x rows of the activation type; a tile is 16 rows of G and
// the same 16 of U.  Down: h rows of f32 as two f16 rows each; a tile is 32
// rows of D.  Row v of x (v = 2 token + part in down) is row (v % 4) * 4 + v /
// 4 of the matrix instruction, so that the first four rows' results lie in one
// register.
template <int BITS, int G, bool F16_, bool DOWN>
__device__ __forceinline__ void moe_open(const MoeArgs& a, int e, int tile, int K, int lane, Stream<BITS, G, F16_, 2>& st) {
  const long row0 = (long)e * (DOWN ? a.N : 2 * a.I) + (DOWN ? 32 * tile : 16 * tile);
  st.open(DOWN ? a.down_packed : a.gate_up_packed, DOWN ? a.down_scales : a.gate_up_scales,
          DOWN ? a.down_biases : a.gate_up_biases, row0, row0 + (DOWN ? 16 : a.I), K, lane);
}

template <bool DOWN>
__device__ __forceinline__ const void* moe_source(const MoeArgs& a, int pair) {
  return DOWN ? (const void*)(a.h + (long)pair * a.I) : (const void*)((const uint16_t*)a.x + (long)(pair / a.top_k) * a.N);
}

// whole rows a wave (KS = 1): the workgroup's x in LDS, then every wave its tiles
template <int BITS, int G, bool F16_, bool DOWN, int NI>
__device__ __forceinline__ void moe_rows(const MoeArgs& a, const MoeShape& s, int e, const int* list, int tokens,
                                         const float* row_scale, const unsigned char* xs, int tile0, int tile1) {
  using St = Stream<BITS, G, F16_, 2>;
  const int lane = threadIdx.x & 63;
  const int c = lane & 15, h = lane >> 4, vrows = DOWN ? 2 * tokens : tokens;
  const int quads = (s.K + St::COLS - 1) / St::COLS;
  const unsigned char* xa = xs + (h * s.rows + min((c >> 2) + 4 * (c & 3), vrows - 1)) * 16;
  float back[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) back[i] = 0x1p24f / row_scale[DOWN ? (4 * i + h) / 2 : 4 * i + h];
  St st;
  typename St::Quad w;
  if (tile0 >= tile1) return;
  moe_open<BITS, G, F16_, DOWN>(a, e, tile0, s.K, lane, st);
  st.load(0, w);
  for (int tile = tile0; tile < tile1; ++tile) {
    float acc[2][NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[0][i] = acc[1][i] = 0.f;
    moe_quads<NI>(st, 0, quads, w, xa, 4 * s.rows * 16, acc);
    if (tile + 1 < tile1) {
      moe_open<BITS, G, F16_, DOWN>(a, e, tile + 1, s.K, lane, st);
      st.load(0, w);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int v = 4 * i + h;
      if constexpr (DOWN) {
        // the high and the low part's sums are neighbours: lanes of even h take tile 0's total, of odd h tile 1's
        uint32_t p = __float_as_uint(acc[0][i]), q = __float_as_uint(acc[1][i]);
        swap16(p, q);
        const float sum = __uint_as_float(p) + __uint_as_float(q);
        if (v / 2 < tokens) a.part[(long)list[v / 2] * a.N + 32 * tile + 16 * (h & 1) + c] = sum * back[i];
      } else {
        const float g = acc[0][i] * back[i], u = acc[1][i] * back[i];
        if (v < tokens) a.h[(long)list[v] * a.I + 16 * tile + c] = g / (1.f + expf(-g)) * u;
      }
    }
  }
}

// a part of the columns a wave (KS = 4), each with its own x
template <int BITS, int G, bool F16_, bool DOWN, int NI>
__device__ __forceinline__ void moe_parts(const MoeArgs& a, const MoeShape& s, int e, const int* list, int tokens,
                                          unsigned char* xs, float* row_scale, float* red, int tile) {
  using St = Stream<BITS, G, F16_, 2>;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4, vrows = DOWN ? 2 * tokens : tokens;
  const int quads = (s.K + St::COLS - 1) / St::COLS, each = (quads + 3) / 4;
  const int q0 = min(wave * each, quads), q1 = min(q0 + each, quads);
  St st;
  typename St::Quad w;
  moe_open<BITS, G, F16_, DOWN>(a, e, tile, s.K, lane, st);
  if (q0 < q1) st.load(q0, w);
  unsigned char* mine = xs + wave * s.x_bytes;
  float* scale = row_scale + 16 * wave;
  for (int t = 0; t < tokens; ++t) {
    const float most = moe_amax<DOWN, F16_>(moe_source<DOWN>(a, list[t]), q0 * St::COLS + 4 * lane, min(q1 * St::COLS, s.K), 256);
    const float sc = moe_row_scale(wave_max_f32(most));
    if (lane == 0) scale[t] = sc;
  }
  float acc[2][NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) acc[0][i] = acc[1][i] = 0.f;
  const unsigned char* xa = mine + (h * s.rows + min((c >> 2) + 4 * (c & 3), vrows - 1)) * 16;
  for (int q = q0; q < q1; q += s.chunk) {
    const int end = min(q + s.chunk, q1), units = (end - q) * 4 * St::S::NJ * 4;
    __builtin_amdgcn_wave_barrier();  // (LDS of this wave alone, whose operations stay in order)
    for (int t = 0; t < tokens; ++t)
      moe_stage<BITS, G, F16_, DOWN>(moe_source<DOWN>(a, list[t]), scale[t], q * St::COLS, s.K, lane, 64, units, mine, s.rows,
                                     DOWN ? 2 * t : t);
    __builtin_amdgcn_wave_barrier();
    if (q > q0) st.load(q, w);
    moe_quads<NI>(st, q, end, w, xa, 4 * s.rows * 16, acc);
  }
  // the waves' sums, each over its own power of two
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int v = 4 * i + h, t = DOWN ? v / 2 : v;
    const float back = q0 < q1 && t < tokens ? 0x1p24f / scale[t] : 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) red[((wave * 2 + k) * NI + i) * 64 + lane] = t < tokens ? acc[k][i] * back : 0.f;
  }
  __syncthreads();
  const auto total = [&](int k, int v, int col) {
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) sum += red[((q * 2 + k) * NI + (v >> 2)) * 64 + (v & 3) * 16 + col];
    return sum;
  };
  if constexpr (DOWN) {
    for (int i = threadIdx.x; i < 32 * tokens; i += 256) {
      const int t = i >> 5, n = i & 31;
      a.part[(long)list[t] * a.N + 32 * tile + n] = total(n >> 4, 2 * t, n & 15) + total(n >> 4, 2 * t + 1, n & 15);
    }
  } else {
    const int t = threadIdx.x >> 4, n = threadIdx.x & 15;
    if (t < tokens) {
      const float g = total(0, t, n), u = total(1, t, n);
      a.h[(long)list[t] * a.I + 16 * tile + n] = g / (1.f + expf(-g)) * u;
    }
  }
  __syncthreads();
}

template <int BITS, int G, bool F16_, bool DOWN, int KS>
__global__ __launch_bounds__(256) void moe_kernel(MoeArgs a, MoeShape s) {
  using St = Stream<BITS, G, F16_, 2>;
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ int list[16];
  __shared__ float row_scale[KS == 4 ? 64 : 16];
  __shared__ float red[KS == 4 ? 2048 : 64];
  const int slot = blockIdx.y, lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int count = a.counts[2 * slot], e = a.counts[2 * slot + 1];
  const int per_pass = DOWN ? s.rows / 2 : s.rows;
  for (int first = 0; first < count; first += per_pass) {
    const int tokens = min(per_pass, count - first);
    if (threadIdx.x < 16) list[threadIdx.x] = a.lists[(long)slot * a.M + min(first + (int)threadIdx.x, count - 1)];
    __syncthreads();
    if constexpr (KS == 4) {
      if ((DOWN ? 2 * tokens : tokens) <= 4) moe_parts<BITS, G, F16_, DOWN, 1>(a, s, e, list, tokens, lds, row_scale, red, blockIdx.x);
      else moe_parts<BITS, G, F16_, DOWN, 4>(a, s, e, list, tokens, lds, row_scale, red, blockIdx.x);
    } else {
      const int quads = (s.K + St::COLS - 1) / St::COLS, units = quads * 4 * St::S::NJ * 4;
      for (int t = 0; t < tokens; ++t) {
        const float most = wave_max_f32(moe_amax<DOWN, F16_>(moe_source<DOWN>(a, list[t]), 4 * (int)threadIdx.x, s.K, 1024));
        if (lane == 0) red[4 * t + wave] = most;
      }
      __syncthreads();
      if (threadIdx.x < 16) {
        const int t = min((int)threadIdx.x, tokens - 1);
        row_scale[threadIdx.x] = moe_row_scale(nan_max(nan_max(red[4 * t], red[4 * t + 1]), nan_max(red[4 * t + 2], red[4 * t + 3])));
      }
      __syncthreads();
      for (int t = 0; t < tokens; ++t)
        moe_stage<BITS, G, F16_, DOWN>(moe_source<DOWN>(a, list[t]), row_scale[t], 0, s.K, threadIdx.x, 256, units, lds, s.rows,
                                       DOWN ? 2 * t : t);
      __syncthreads();
      const int tile0 = (blockIdx.x * 4 + wave) * s.tiles, tile1 = min(tile0 + s.tiles, DOWN ? a.N / 32 : a.I / 16);
      if ((DOWN ? 2 * tokens : tokens) <= 4) moe_rows<BITS, G, F16_, DOWN, 1>(a, s, e, list, tokens, row_scale, lds, tile0, tile1);
      else moe_rows<BITS, G, F16_, DOWN, 4>(a, s, e, list, tokens, row_scale, lds, tile0, tile1);
      __syncthreads();
    }
  }
}

// up for a few tokens: a slot is a pair of token and choice
template <int BITS, int G, bool F16_>
__global__ __launch_bounds__(256) void moe_few_up_kernel(MoeArgs a, MoeShape s) {
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ float row_scale[64];
  __shared__ float red[512];
  __shared__ MoeFew l;
  const int e = moe_find(a, blockIdx.y, blockIdx.x == 0, reinterpret_cast<float*>(lds), l);
  if (l.count == 0) return;
  moe_parts<BITS, G, F16_, false, 1>(a, s, e, l.list, l.count, lds, row_scale, red, blockIdx.x);
}

// down for a few tokens: 16 rows of D for all slots, and y
constexpr int MOE_FEW_WAVES = 8;
template <int BITS, int G, bool F16_>
__global__ __launch_bounds__(64 * MOE_FEW_WAVES) void moe_few_down_kernel(MoeArgs a, MoeShape s) {
  using St = Stream<BITS, G, F16_, 1>;
  constexpr int NI = 2;  // eight x rows: four tokens' two parts
  extern __shared__ __attribute__((aligned(16))) unsigned char lds[];
  __shared__ float red[MOE_FEW_WAVES * NI * 64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int c = lane & 15, h = lane >> 4;
  const int slots = a.M * a.top_k, quads = (a.I + St::COLS - 1) / St::COLS;
  unsigned char* mine = lds + wave * s.x_bytes;
  float total[NI] = {0.f, 0.f};
  // this wave's share of all slots' quads
  const int all = slots * quads, from = wave * all / MOE_FEW_WAVES, to = (wave + 1) * all / MOE_FEW_WAVES;
  for (int at = from; at < to;) {
    const int slot = at / quads, q0 = at - slot * quads, q1 = min(quads, q0 + to - at);
    at += q1 - q0;
    const int count = a.counts[2 * slot], e = a.counts[2 * slot + 1];
    if (count == 0) continue;
    St st;
    typename St::Quad w;
    const long row0 = (long)e * a.N + 16 * blockIdx.x;
    st.open(a.down_packed, a.down_scales, a.down_biases, row0, row0, a.I, lane);
    st.load(q0, w);
    float acc[1][NI] = {{0.f, 0.f}};
    const int* list = a.lists + slot * a.M;
    const unsigned char* xa = mine + (h * s.rows + min((c >> 2) + 4 * (c & 3), 2 * count - 1)) * 16;
    float scale[MOE_FEW];
#pragma unroll
    for (int t = 0; t < MOE_FEW; ++t) {
      scale[t] = 1.f;
      if (t < count) {
        const int pair = list[t];
        const float most = moe_amax<true, F16_>(moe_source<true>(a, pair), q0 * St::COLS + 4 * lane, min(q1 * St::COLS, a.I), 256);
        scale[t] = moe_row_scale(wave_max_f32(most));
      }
    }
    for (int q = q0; q < q1; q += s.chunk) {
      const int end = min(q + s.chunk, q1), units = (end - q) * 4 * St::S::NJ * 4;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int t = 0; t < MOE_FEW; ++t)
        if (t < count)
          moe_stage<BITS, G, F16_, true>(moe_source<true>(a, list[t]), scale[t], q * St::COLS, a.I, lane, 64, units, mine, s.rows,
                                         2 * t);
      __builtin_amdgcn_wave_barrier();
      if (q > q0) st.load(q, w);
      moe_quads<NI>(st, q, end, w, xa, 4 * s.rows * 16, acc);
    }
    // x row v = 4 i + h holds part h % 2 of the list's token 2 i + h / 2; that token's sums go to row 2 token + part
#pragma unroll
    for (int t = 0; t < MOE_FEW; ++t) {
      if (t >= count) break;
      const int pair = list[t], m = pair / a.top_k;
      const float f = a.weights[pair] * (0x1p24f / scale[t]);
      // lane row h of register i is 4 i + h: take row 2 t + part to 2 m + part
      const float v = __shfl(acc[0][t >> 1], 16 * ((2 * t + (h & 1)) & 3) + c);
#pragma unroll
      for (int i = 0; i < NI; ++i)
        if (4 * i + h == 2 * m + (h & 1)) total[i] = fmaf(f, v, total[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < NI; ++i) red[(wave * NI + i) * 64 + lane] = total[i];
  __syncthreads();
  const int m = threadIdx.x >> 4, n = threadIdx.x & 15;
  if (m >= a.M) return;
  float v = 0.f;
#pragma unroll
  for (int q = 0; q < MOE_FEW_WAVES; ++q) {
    const float* p = red + (q * NI + (m >> 1)) * 64 + 32 * (m & 1) + n;  // rows 2 m and 2 m + 1
    v += p[0] + p[16];
  }
  const long at = (long)m * a.N + 16 * blockIdx.x + n;
  const float sum = a.sums[m];
  float y = a.resid ? load_as_f32(a.resid, at, a.act_dt) : 0.f;
  if (a.choices[m]) y = fmaf(a.scale / sum, v, y);
  if (sum != sum) y = __builtin_nanf("");
  ((uint16_t*)a.y)[at] = f32_to_act_bits(y, F16_);
}

template <int BITS, int G, bool F16_>
hipError_t launch_moe_dt(const MoeArgs& a, MoeStep step, hipStream_t st) {
  using St = Stream<BITS, G, F16_, 2>;
  MoeShape s{};
  const bool down = step == MOE_DOWN || step == MOE_FEW_DOWN;
  s.K = down ? a.I : a.N;
  const int quads = (s.K + St::COLS - 1) / St::COLS;
  if (step == MOE_FEW_DOWN) {
    s.rows = 2 * a.M;
    s.chunk = a.M <= 2 ? 2 : 1;
    s.x_bytes = s.chunk * St::COLS * 2 * s.rows;
    hipLaunchKernelGGL((moe_few_down_kernel<BITS, G, F16_>), dim3((unsigned)(a.N / 16)), dim3(64 * MOE_FEW_WAVES),
                       MOE_FEW_WAVES * s.x_bytes, st, a, s);
    return hipGetLastError();
  }
  const int slots = (int)std::min<int64_t>((int64_t)a.M * a.top_k, a.E), tiles = down ? a.N / 32 : a.I / 16;
  // x rows a pass: eight where an expert has four tokens or fewer on average (a second pass reads the weights again, from the caches)
  const int most = (int64_t)a.M * a.top_k <= 4 * (int64_t)a.E ? 8 : 16;
  s.rows = down ? std::min(2 * a.M, 16) : std::min(a.M, most);
  if (step == MOE_FEW_UP) s.rows = a.M;
  const int row_bytes = quads * St::COLS * 2;  // of x in LDS
  const bool whole = step != MOE_FEW_UP && s.rows * row_bytes <= 65536 && (int64_t)tiles * slots >= 2048;
  if (whole) {
    // 512 workgroups or more
    s.tiles = (int)std::max<int64_t>(1, std::min<int64_t>(8, (int64_t)tiles * slots / 2048));
    const dim3 grid((unsigned)((tiles + 4 * s.tiles - 1) / (4 * s.tiles)), (unsigned)slots);
    if (down) hipLaunchKernelGGL((moe_kernel<BITS, G, F16_, true, 1>), grid, dim3(256), s.rows * row_bytes, st, a, s);
    else hipLaunchKernelGGL((moe_kernel<BITS, G, F16_, false, 1>), grid, dim3(256), s.rows * row_bytes, st, a, s);
    return hipGetLastError();
  }
  // a wave's part of x: as many quads as fit 12 KiB, one at least
  const int quad_bytes = St::COLS * 2 * s.rows;
  s.chunk = std::max(1, std::min((quads + 3) / 4, 12288 / quad_bytes));
  s.x_bytes = s.chunk * quad_bytes;
  const dim3 grid((unsigned)tiles, (unsigned)(step == MOE_FEW_UP ? a.M * a.top_k : slots));
  const int lds = std::max(4 * s.x_bytes, step == MOE_FEW_UP ? a.M * a.E * 4 : 0);
  if (step == MOE_FEW_UP) hipLaunchKernelGGL((moe_few_up_kernel<BITS, G, F16_>), grid, dim3(256), lds, st, a, s);
  else if (down) hipLaunchKernelGGL((moe_kernel<BITS, G, F16_, true, 4>), grid, dim3(256), lds, st, a, s);
  else hipLaunchKernelGGL((moe_kernel<BITS, G, F16_, false, 4>), grid, dim3(256), lds, st, a, s);
  return hipGetLastError();
}

}  // namespace

template <int BITS>
hipError_t launch_moe_bits(const MoeArgs& a, MoeStep step, hipStream_t st) {
  switch (a.G * 2 + (a.act_dt == F16)) {
    case 64: return launch_moe_dt<BITS, 32, false>(a, step, st);
    case 65: return launch_moe_dt<BITS, 32, true>(a, step, st);
    case 128: return launch_moe_dt<BITS, 64, false>(a, step, st);
    case 129: return launch_moe_dt<BITS, 64, true>(a, step, st);
    case 256: return launch_moe_dt<BITS, 128, false>(a, step, st);
    case 257: return launch_moe_dt<BITS, 128, true>(a, step, st);
    default: return hipErrorNotSupported;
  }
}

}  // namespace qaff
