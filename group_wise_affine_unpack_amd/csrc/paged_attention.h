// Attention of one new token a sequence over the paged affine cache.
//     z[t] = scale * sum_d q[d] k[t,d],  t in [max(0, len - window), len)
//     p = softmax(z),  o[d] = sum_t p[t] v[t,d]
// with k and v = code*scale + bias as kv_cache_append_affine stored them; the
// g = heads/kv_heads query heads of a key head are the columns of one matrix
// product, up to 16 at a time.  A row that sees no token gives zeros.
//
// One wave takes 32 tokens of a key head a step, on the matrix cores
// (16x16x32, f16 in, fp32 out), codes as integers and the affine parameters
// in fp32 around the products:
//     logits   C_g[t,h] = sum_{d in group g} code[t,d] q[d,h]
//              z[t,h]   = c (sum_g ks[t,g] C_g[t,h] + kb[t,g] Q_g[h])
//              with Q_g[h] = sum_{d in group g} q[d,h]
//     values   o[d,h] = sum_t code[t,d] A_g[t,h] + sum_t vb[t,g] p[t,h]
//              with A_g[t,h] = p[t,h] vs[t,g], times a power of two, rounded to f16
// Codes: an f16 whose exponent bits are zero is its low ten bits times 2^-24,
// and the matrix cores keep such numbers, so masking a code where it lies in
// bits 0-9 of each 16-bit half (4-bit: bits 0-3 and, times 16, bits 4-7) is
// the whole conversion: one AND for two codes.  The factors 2^24 and 16 go to
// q (exact powers of two, per column) and to the outputs.
// The key biases' part of z is one product more, kb[t,g] by Q_g[h] cut into
// three 16-bit pieces, in the parameters' own type: 24 bits in bf16; in f16,
// whose steps end at 2^-24, to 2^-32 of the head's largest query entry, Q_g
// being taken 2^17 times larger (below 2^15) for that.
// Registers: C_g has the tokens of a lane's quarter (lane / 16) as rows and
// the head (lane % 16) as column, which is where the value product takes its
// second operand from, so p never leaves the lane.  Where a key head has few
// query heads, each takes FOLD of the 16 columns: column (sub, head) keeps the
// softmax of the tokens TOK sub + i of each quarter's four only, its other
// weights are zero, and the columns of a head are added at the end.  That
// takes the softmax's and the parameters' work of unused columns away.
// Value codes arrive as rows of tokens and are wanted as pairs of tokens: two
// tokens' codes of the same columns are put into the halves of one register
// first.
// q is scaled by a power of two per head so that its largest entry lies in
// [2^14, 2^15): entries are exact down to 2^-22 of the largest (2^-28 for 8-bit
// codes, whose factors are 1) and off by at most 2^-33 of it below.
// The softmax's reference mu is the largest logit seen when it was set (p of
// that token is a power of two, and its weights A exact), and
// p = 2^(z - mu - 30): sums of p vb and of p vs code then stay finite for any
// number of tokens.  A_g's power of two is each head's and group's own, from
// the products p vs of that group seen: it brings a wave's largest to 2^3 or
// more, so a weight keeps its 11 bits down to 2^-17 of the largest and is off
// by at most 2^-28 of it below.  (A power of two from the largest logit and
// the largest scale by themselves loses the weights' bits where a token with a
// scale far above the others has no weight, and where one group's scales lie
// far below another's.)  Most steps need neither a
// maximum over the lanes nor a rescaling: a wave's first one takes the value
// scales of its largest logit's token, and only one in which a logit passes
// mu by 4 or an A reaches 2^15 (wave-uniform branches) sets mu or the powers
// of two anew.  (With 2^7 for 2^3 the second kind is so frequent that 16
// sequences up to 4096 tokens take 18.5 us for 17.7; without the first step's
// own, 17.9.  A power of two of each group costs one product a weight over one
// of all groups: 64 sequences of 4096 tokens 61.2 -> 62.0 us at 4 bits and four
// heads a key head, 84.7 -> 90.4 at twenty, whose columns hold no spare tokens.)
//
// Memory: each wave copies the 32 tokens after the ones at work straight
// into LDS (16 bytes a lane, no register between, non-temporal: with the
// streaming hint 131072 tokens took 39.5 us where they took 44.5), and reads
// its operands from there in whatever layout they want.  What a lane reads
// of memory is thereby one code row's 16-byte piece instead of 28 loads of 2
// to 16 bytes a step.
// What bounds it: at 8 bits memory (64 sequences of 4096 tokens, D = 128:
// 571 MB in 95 us, 6.0 TB/s), at 4 bits the waits of 12 waves a CU on their
// copies and on each other's vector instructions, 250 a step of 4.6 KB with
// four heads a key head (302 MB in 60 to 62 us, 4.9 TB/s; vector pipes busy
// 62% of the time), for few tokens the chain lengths -> page table -> rows ->
// join.
// Measured and not kept: operands loaded from memory into registers with one
// step of look-ahead (70 us for those 302 MB where the copies took 64), three
// or four stages of look-ahead (64), four workgroups a CU (71), chunks of
// equal size instead of equal shares (a ragged 8-bit batch 119 against 101).
//
// Work: equal shares of all tiles of 128 tokens (paged_attn_kernel), four
// waves to a tile, joined through LDS; sequences cut by a share's end leave
// fp32 partial sums with their mu for a second kernel.  Short tables take a
// workgroup per sequence and unit instead (paged_attn_short_kernel).
// Instantiated per code width in paged_attention_b{2,4,8}.hip.
#pragma once

#include <algorithm>
#include <type_traits>

#include "common.h"

namespace qaff {
namespace {

constexpr float PBIAS = -30.f;     // log2 of p at the reference
constexpr float MROOM = 4.f;       // how far a logit may pass the reference (log2)
constexpr int ATOP = 4;            // log2 of the largest A of a group at a new power of two
constexpr uint32_t ALIM = 0x7800;  // f16 of 2^15, which no A may pass
constexpr int VEMIN = -100, VEMAX = 120;  // exponents of A's power of two (sums times 2^24 / it stay finite)

struct AttnMeta {
  int64_t start;  // a sequence's start on the line of one unit
  int tiles;      // its tiles
};

struct AttnWork {
  PagedAttnArgs a;
  FastDiv page;         // tokens a page
  int share, htiles;    // query heads a key head; tiles of 16 of them
  float* part_o;        // [2 workgroups][gm][D]
  float* part_ml;       // [2 workgroups][gm][2]
  AttnMeta* meta;       // [B + 1]; the last one: a workgroup's share of the line, a unit's start on it
};

template <int D_, int G_, int BITS_, bool F16_, int FOLD_, int WAVES_>
struct Cfg {
  static constexpr int D = D_, G = G_, BITS = BITS_, NG = D / G, WAVES = WAVES_;
  static constexpr bool ACT16 = F16_;
  static constexpr float QSUM = F16_ ? 0x1p17f : 1.f;  // Q_g's factor over the products of codes
  static constexpr int FOLD = FOLD_, HEADS = 16 / FOLD, TOK = 4 / FOLD;  // columns a head, heads, tokens a lane of a quarter's four
  static constexpr int KS = G / 32;                      // product steps a group (keys)
  static constexpr int KB = G / 4 * BITS / 8;            // key code bytes a lane and group
  static constexpr int KW = KB < 4 ? 1 : KB / 4;
  static constexpr int VC = G / 16;                      // value columns a lane and group
  static constexpr int VBITS = VC * BITS;                // value code bits a lane, token and group
  static constexpr int VW = VBITS <= 32 ? 1 : 2;
  static constexpr int SW = (TOK * NG + 1) / 2;          // words of the scales of a lane's tokens of 16
  static constexpr int BW = (NG + 1) / 2;                // words of one token's
  static constexpr int ROWB = D * BITS / 8;
  // A stage in LDS: 32 tokens' key codes, value codes, then per half the
  // key scales, key biases, value scales and value biases, each as in memory
  static constexpr int CODES = 16 * ROWB, PARAMS = 32 * NG;  // bytes of 16 tokens' codes, of one kind of parameter
  static constexpr int STAGE = 4 * CODES + 8 * PARAMS;
  // Two stages a wave, one ahead of the one at work.  (Three stages and two
  // workgroups a CU instead of three: 131072 tokens the same, a ragged 4-bit
  // batch of 64 sequences up to 8192 tokens 75 against 67 us.)
  static constexpr int STAGES = 2, LDS = WAVES * STAGES * STAGE;
  // Registers of a step: accumulators, q, what it reads of a stage, and about
  // 64 more (the compiler takes up to 25 on top).  Past 240, values are read
  // after the softmax (LATE), and where that makes room for a third workgroup
  // a CU (D = 96, G = 32, 4-bit, 20 heads a key head: 124 us for 136).
  static constexpr int KEYS = 2 * NG * KW + 2 * BW + 2 * SW, VALS = 4 * SW + 8 * NG * VW;
  static constexpr int ALL = D / 4 + D / 8 + 64 + KEYS + VALS;
  static constexpr bool LATE = ALL > 240 || (ALL > 168 && ALL <= 176 && LDS * 3 <= 155 * 1024);
  static constexpr int REGS =
      LATE ? D / 4 + D / 8 + 64 + (KEYS > 4 * SW + 8 * VW ? KEYS : 4 * SW + 8 * VW) : ALL;
  // workgroups of four waves a CU, by LDS and registers (one more than the registers hold spills: D = 128, G = 32,
  // 4-bit, 16 heads, 3 instead of 2: five times the time; D = 256, G = 32, 2-bit, 2 instead of 1: 288 against 191 us,
  // with eight heads 99 against 93.
  // Four where D = 64 leaves room, G = 64, 4-bit, 20 heads: 100 us, with three 108)
  static constexpr int PER_CU = LDS * 4 <= 155 * 1024 && REGS <= 118   ? 4
                                : LDS * 3 <= 155 * 1024 && REGS <= 165 ? 3
                                : LDS * 2 <= 155 * 1024 && REGS <= 228 && !(LATE && REGS + NG > 206) ? 2
                                                                       : 1;
  static constexpr int COPIES = (CODES + 1023) / 1024, PCOPIES = (8 * PARAMS + 1023) / 1024;
  // rows of 2^n 16-byte pieces keep piece c of row r at c ^ swizzle(r), so that a piece of many rows is spread over the banks
  static constexpr int PIECES = ROWB % 16 == 0 && ((ROWB / 16) & (ROWB / 16 - 1)) == 0 ? ROWB / 16 : 0;
  __device__ static constexpr int swizzle(int row) { return PIECES ? (row >> 2) & (PIECES - 1) & 3 : 0; }
  // where byte `b` of row `row` of 16 lies
  __device__ static constexpr int at(int row, int b) { return row * ROWB + ((b >> 4 ^ swizzle(row)) << 4) + (b & 15); }
};

template <int BYTES>
__device__ __forceinline__ void load_bytes(const uint8_t* p, uint32_t* out) {
  if constexpr (BYTES == 1)
    out[0] = *p;
  else if constexpr (BYTES == 2)
    out[0] = *reinterpret_cast<const uint16_t*>(p);
  else if constexpr (BYTES % 16 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 16; ++i) {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p + 16 * i);
#pragma unroll
      for (int j = 0; j < 4; ++j) out[4 * i + j] = v[j];
    }
  } else if constexpr (BYTES == 6) {
    out[0] = *reinterpret_cast<const uint16_t*>(p) | (uint32_t)*reinterpret_cast<const uint16_t*>(p + 2) << 16;
    out[1] = *reinterpret_cast<const uint16_t*>(p + 4);
  } else if constexpr (BYTES == 12) {
#pragma unroll
    for (int i = 0; i < 3; ++i) out[i] = *reinterpret_cast<const uint32_t*>(p + 4 * i);
  } else if constexpr (BYTES % 8 == 0) {
#pragma unroll
    for (int i = 0; i < BYTES / 8; ++i) {
      const u32x2_t v = *reinterpret_cast<const u32x2_t*>(p + 8 * i);
      out[2 * i] = v[0];
      out[2 * i + 1] = v[1];
    }
  } else {
    static_assert(BYTES == 4, "load size");
    out[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// element i of packed 16-bit values, as float
template <bool F16_>
__device__ __forceinline__ float half_at(const uint32_t* w, int i) {
  const uint32_t v = w[i / 2];
  if constexpr (F16_) return f16_bits_to_f32((i & 1) ? v >> 16 : v & 0xffffu);
  else return __uint_as_float((i & 1) ? v & 0xffff0000u : v << 16);
}

// sum and maximum over the four lanes of a head
__device__ __forceinline__ float quads_sum(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float quads_max(float v) {
  auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
  r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// Which column of a lane's G/4 the half `h` of register `r` of key step `s`
// holds, and the power of two its code is multiplied by there.
template <class C>
constexpr int key_dim(int s, int r, int h) {
  if (C::BITS == 8) return 8 * s + 4 * (r >> 1) + (r & 1) + 2 * h;
  if (C::BITS == 4) return 8 * s + r + 4 * h;
  if (C::G == 32) return r + 4 * h;
  return 16 * (s >> 1) + 4 * (s & 1) + r + 8 * h;
}
template <class C>
constexpr int key_shift(int r) {
  return C::BITS == 8 ? 0 : C::BITS == 4 ? 4 * (r & 1) : 2 * r;
}

__device__ __forceinline__ f16x8_t as_f16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  const u32x4_t v = {a, b, c, d};
  return __builtin_bit_cast(f16x8_t, v);
}

// key codes of step s of a group: 16 tokens by 32 columns over the wave
template <class C>
__device__ __forceinline__ f16x8_t key_codes(const uint32_t* w, int s) {
  if constexpr (C::BITS == 8) {
    const uint32_t a = w[2 * s], b = w[2 * s + 1], m = 0x00ff00ffu;
    return as_f16x8(a & m, (a >> 8) & m, b & m, (b >> 8) & m);
  } else if constexpr (C::BITS == 4) {
    const uint32_t a = w[s], b = a >> 8;
    return as_f16x8(a & 0x000f000fu, a & 0x00f000f0u, b & 0x000f000fu, b & 0x00f000f0u);
  } else {
    uint32_t a;
    if constexpr (C::G == 32)
      a = (w[0] & 0xffu) | (w[0] & 0xff00u) << 8;
    else
      a = (s & 1) ? w[s >> 1] >> 8 : w[s >> 1];
    return as_f16x8(a & 0x00030003u, a & 0x000c000cu, a & 0x00300030u, a & 0x00c000c0u);
  }
}

// value codes of column c of a group, of two tokens (the halves of `w`, whose
// half-words hold each token's 16-bit piece c / (16/BITS))
template <class C>
__device__ __forceinline__ uint32_t value_pair(uint32_t w, int c) {
  constexpr int PER = 16 / C::BITS, PERB = 8 / C::BITS;  // codes a piece, a byte
  const int in = c % PER;
  const uint32_t b = in >= PERB ? w >> 8 : w;
  return b & ((0x00010001u * ((1u << C::BITS) - 1u)) << (C::BITS * (in % PERB)));
}
template <class C>
constexpr int value_shift(int c) {
  return C::BITS * (c % (8 / C::BITS));
}

template <class C>
struct Wave {
  // constant over the loop
  f16x8_t q[C::NG][C::KS];
  u32x4_t qsum;           // the key biases' operand: Q_g of this lane's head (times QSUM), a 16-bit piece of it by the lane's quarter
  float zscale;           // logits to base 2, with q's power of two and the codes' taken back; > 0
  // running
  f32x4_t o[C::NG][C::VC];
  float l, bias[C::NG];   // sums over this lane's tokens
  float ve[C::NG];        // A's power of two
  float mref, mu, mlim;
};

// 16 bytes a lane from memory into LDS, without a register between: lane l's
// land at `lds` + 16 l.  The compiler does not see these loads: the wait for
// them is wait_copies below, and every LDS read of theirs comes after it.
// The first LANES lanes copy.  (Their mask is set here and not by a branch: one
// divergent branch in the loop makes the compiler treat its uniform ones as
// such, and copy every accumulator around them.)
template <int LANES>
__device__ __forceinline__ void copy_to_lds(const uint8_t* base, uint32_t off, uint32_t lds) {
  if constexpr (LANES >= 64) {
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" ::"v"(off), "s"(base), "s"(lds) : "memory");
  } else {
    uint64_t all;
    asm volatile(
        "s_mov_b64 %0, exec\n\ts_mov_b32 m0, %3\n\ts_mov_b64 exec, %4\n\t"
        "global_load_lds_dwordx4 %1, %2 nt\n\ts_mov_b64 exec, %0"
        : "=&s"(all)
        : "v"(off), "s"(base), "s"(lds), "s"((uint64_t(1) << LANES) - 1)
        : "memory");
  }
}
template <int LANES>
__device__ __forceinline__ void copy_to_lds(const uint8_t* p, uint32_t lds) {
  uint64_t all;
  asm volatile(
      "s_mov_b64 %0, exec\n\ts_mov_b32 m0, %2\n\ts_mov_b64 exec, %3\n\t"
      "global_load_lds_dwordx4 %1, off nt\n\ts_mov_b64 exec, %0"
      : "=&s"(all)
      : "v"(p), "s"(lds), "s"(LANES >= 64 ? ~uint64_t(0) : (uint64_t(1) << (LANES & 63)) - 1)
      : "memory");
}
// f(which of the copies, its lanes) for each of the copies of N 16-byte pieces
template <int N, int M = 0, class F>
__device__ __forceinline__ void copies(F&& f) {
  f(std::integral_constant<int, M>{}, std::integral_constant<int, (N - 64 * M < 64 ? N - 64 * M : 64)>{});
  if constexpr (N > 64 * (M + 1)) copies<N, M + 1>(f);
}
// until this wave's copies are in LDS
__device__ __forceinline__ void wait_copies() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// 16x16x32 product of 16-bit parameters and pieces of Q_g, in their own type
template <bool F16_>
__device__ __forceinline__ f32x4_t mfma_act(u32x4_t a, u32x4_t b, f32x4_t c) {
  if constexpr (F16_)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a), __builtin_bit_cast(bf16x8_t, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t pk_max_u16(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// q as the products take it, from this lane's columns of each group: raw
// [NG][G/4] 16-bit values of its head, zeros for a column that has none.
template <class C>
__device__ __forceinline__ void set_q(Wave<C>& w, const uint32_t (&raw)[C::NG][C::G / 8], bool have, int kq, float scale) {
  float qv[C::NG][C::G / 4], mx = 0.f;
#pragma unroll
  for (int g = 0; g < C::NG; ++g)
#pragma unroll
    for (int k = 0; k < C::G / 4; ++k) {
      qv[g][k] = have ? half_at<C::ACT16>(raw[g], k) : 0.f;
      mx = fmaxf(mx, fabsf(qv[g][k]));
    }
  mx = quads_max(mx);
  // the largest entry to [2^14, 2^15) (one below 2^-113 to less), with the sign of the scale; to less also
  // where zscale would pass below 2^-126, since z = -inf of a hidden token times a zscale of 0 is not hidden
  const float base2 = fabsf(scale) * 1.4426950408889634f;
  int e = 0;
  if (mx > 0.f && mx < __builtin_inff())
    e = min(min(14 - __builtin_amdgcn_frexp_expf(mx) + 1, 127), 149 + __builtin_amdgcn_frexp_expf(base2));
  const float to = scale == 0.f ? 0.f : __builtin_amdgcn_ldexpf(scale < 0.f ? -1.f : 1.f, e);
  const f16x2_t ones = {(_Float16)1.f, (_Float16)1.f};
  w.qsum = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
  for (int g = 0; g < C::NG; ++g) {
    float sum = 0.f;
#pragma unroll
    for (int s = 0; s < C::KS; ++s) {
      uint32_t reg[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const f16x2_t h = {(_Float16)(qv[g][key_dim<C>(s, r, 0)] * to), (_Float16)(qv[g][key_dim<C>(s, r, 1)] * to)};
        sum = __builtin_amdgcn_fdot2(h, ones, sum, false);
        const _Float16 f = (_Float16)(1.f / (float)(1 << key_shift<C>(r)));
        reg[r] = __builtin_bit_cast(uint32_t, h * f16x2_t{f, f});
      }
      w.q[g][s] = as_f16x8(reg[0], reg[1], reg[2], reg[3]);
    }
    // Q_g in QSUM'ths of the products of codes, cut into 16-bit pieces: quarter 0 holds the leading one
    float left = quads_sum(sum) * (0x1p-24f * C::QSUM);
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint16_t piece = f32_to_act_bits(left, C::ACT16);
      if (kq == k) w.qsum[g / 2] |= (uint32_t)piece << (16 * (g & 1));
      left -= C::ACT16 ? f16_bits_to_f32(piece) : bf16_bits_to_f32(piece);
    }
  }
  w.zscale = scale == 0.f ? 1.f : __builtin_amdgcn_ldexpf(base2, 24 - e);
}

// which of a head's FOLD columns a lane has, and with them the tokens TOK sub + i of its quarter
template <class C>
__device__ __forceinline__ int sub_of(int lane) {
  return C::FOLD == 1 ? 0 : (lane & 15) / C::HEADS;
}
template <class C>
__device__ __forceinline__ float own(const f32x4_t& v, int i, int sub) {
  if constexpr (C::FOLD == 1) return v[i];
  else if constexpr (C::FOLD == 2) return sub ? v[2 + i] : v[i];
  else {
    const float lo = (sub & 1) ? v[1] : v[0], hi = (sub & 1) ? v[3] : v[2];
    return (sub & 2) ? hi : lo;
  }
}
// sum and maximum over the columns of a head
template <class C>
__device__ __forceinline__ float fold_sum(float v) {
  if constexpr (C::FOLD >= 2) v += dpp_mov<0x128>(v);  // row_ror:8
  if constexpr (C::FOLD >= 4) v += dpp_mov<0x124>(v);  // row_ror:4
  return v;
}
template <class C>
__device__ __forceinline__ float fold_max(float v) {
  if constexpr (C::FOLD >= 2) v = fmaxf(v, dpp_mov<0x128>(v));
  if constexpr (C::FOLD >= 4) v = fmaxf(v, dpp_mov<0x124>(v));
  return v;
}

// whether `x` holds in some lane, as one scalar
__device__ __forceinline__ bool any_lane(bool x) {
  const uint64_t b = __builtin_amdgcn_ballot_w64(x);
  uint32_t any = (uint32_t)b | (uint32_t)(b >> 32);
  asm volatile("" : "+s"(any));
  return any != 0;
}

__device__ __forceinline__ int exponent(float v) { return (int)(__float_as_uint(v) >> 23) - 127; }

// maximum of pairs of 16-bit numbers over the lanes of a head
template <class C>
__device__ __forceinline__ uint32_t head_max_u16(uint32_t v) {
  auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = pk_max_u16(r[0], r[1]);
  r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = pk_max_u16(r[0], r[1]);
  if constexpr (C::FOLD >= 2) v = pk_max_u16(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xf, 0xf, false));
  if constexpr (C::FOLD >= 4) v = pk_max_u16(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xf, 0xf, false));
  return v;
}

// A new reference for the logits of the heads of this wave, and everything
// summed so far brought to it.
template <class C>
__device__ __forceinline__ void raise(Wave<C>& w, const float (&z)[2][C::TOK], const uint32_t (&vs)[2][C::SW], float zmax) {
  const float top = fold_max<C>(quads_max(zmax));
  const float m = fmaxf(w.mref, top), mu = m == -__builtin_inff() ? 0.f : m;
  const bool fresh = w.mref == -__builtin_inff();  // nothing is summed yet
  const float fall = w.mu - mu, f = fresh ? 0.f : __builtin_amdgcn_exp2f(fall);  // (an infinite logit makes its row NaN)
  const int rise = (int)fminf(floorf(mu) - floorf(w.mu), 300.f);  // in whole powers of two, without a drift
  // the value scales of the largest logit's token
  uint32_t s[C::BW];
#pragma unroll
  for (int k = 0; k < C::BW; ++k) {
    s[k] = 0;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < C::TOK; ++i) {
        uint32_t x;  // groups 2 k and 2 k + 1 of the token
        if constexpr (C::NG % 2 == 0)
          x = vs[u][i * (C::NG / 2) + k];
        else {
          const int e = i * C::NG + 2 * k;
          const uint32_t lo = (e & 1) ? vs[u][e / 2] >> 16 : vs[u][e / 2] & 0xffffu;
          x = 2 * k + 1 < C::NG ? lo | ((e & 1) ? vs[u][(e + 1) / 2] << 16 : vs[u][e / 2] & 0xffff0000u) : lo;
        }
        s[k] = pk_max_u16(s[k], z[u][i] * w.zscale == top ? x & 0x7fff7fffu : 0u);
      }
    s[k] = head_max_u16<C>(s[k]);
  }
  w.mref = m;
  w.mu = mu;
  w.mlim = m + MROOM;
  float fo[C::NG];
#pragma unroll
  for (int g = 0; g < C::NG; ++g) {
    w.bias[g] *= f;
    // A's power of two grows by as much; the first one is that of the largest logit's token, whose p is 2^PBIAS
    const int e = fresh ? ATOP - (int)PBIAS - exponent(half_at<C::ACT16>(s, g)) : exponent(w.ve[g]) + rise;
    const float ve = __builtin_amdgcn_ldexpf(1.f, max(min(e, VEMAX), VEMIN));
    fo[g] = fresh ? 1.f : __builtin_amdgcn_exp2f(fall + (float)(exponent(ve) - exponent(w.ve[g])));
    w.ve[g] = ve;
  }
  w.l *= f;
  if (any_lane(!fresh)) {
#pragma unroll
    for (int g = 0; g < C::NG; ++g)
#pragma unroll
      for (int c = 0; c < C::VC; ++c) w.o[g][c] *= fo[g];
  }
}

// A of this lane's tokens of a step: pairs of tokens of each 16, a token twice where the lane has one.
template <class C>
struct Weights {
  static constexpr int W = C::TOK == 4 ? 2 : 1;
  uint32_t a[C::NG][2 * W];
};
template <class C>
__device__ __forceinline__ void weights(const float (&p)[2][C::TOK], const uint32_t (&vs)[2][C::SW], int g, float ve,
                                        uint32_t (&out)[2 * Weights<C>::W]) {
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    _Float16 a[C::TOK];
#pragma unroll
    for (int i = 0; i < C::TOK; ++i) a[i] = (_Float16)(p[u][i] * ve * half_at<C::ACT16>(vs[u], i * C::NG + g));
#pragma unroll
    for (int k = 0; k < Weights<C>::W; ++k)
      out[Weights<C>::W * u + k] = __builtin_bit_cast(uint32_t, f16x2_t{a[2 * k % C::TOK], a[(2 * k + 1) % C::TOK]});
  }
}

// A's powers of two anew where its limit is passed, and the sums of A brought to them.
template <class C>
__device__ __forceinline__ void retarget(Wave<C>& w, const float (&p)[2][C::TOK], const uint32_t (&vs)[2][C::SW],
                                         Weights<C>& x) {
#pragma unroll
  for (int g = 0; g < C::NG; ++g) {
    // (opaque, and a group after the other: shared with the weights before the branch these would put a second side
    // to it, and all groups' at once take the registers of a workgroup a CU)
    uint32_t s[2][C::SW];
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < C::SW; ++i) {
        s[u][i] = vs[u][i];
        asm volatile("" : "+v"(s[u][i]));
      }
    float most = 0.f;
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < C::TOK; ++i) {
        const float v = fabsf(p[u][i] * half_at<C::ACT16>(s[u], i * C::NG + g));
        most = fmaxf(most, v < __builtin_inff() ? v : 0.f);  // (one that is not finite makes its own columns so)
      }
    most = fold_max<C>(quads_max(most));
    const int from = exponent(w.ve[g]), e = exponent(most), to = from + e < 15 ? from : max(ATOP - e, VEMIN);
    const float f = __builtin_amdgcn_ldexpf(1.f, to - from);
    w.ve[g] = __builtin_amdgcn_ldexpf(1.f, to);
#pragma unroll
    for (int c = 0; c < C::VC; ++c) w.o[g][c] *= f;
    weights<C>(p, s, g, w.ve[g], x.a[g]);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Lane offsets into a stage: codes by group, parameters.
template <class C>
struct Lanes {
  uint32_t k[C::NG][C::KB > 16 ? 2 : 1], v[C::NG], par, kb;
  uint32_t keep[2];  // of the pairs of a quarter's tokens, the halves that are this lane's
};

// 32 tokens from a stage in LDS.  tok: each half's first token; -1: no such
// tile, or its page lies outside the cache.  edge (uniform): some of the 32
// do not count.
template <class C>
__device__ __forceinline__ void step(Wave<C>& w, const uint8_t* st, const Lanes<C>& ln, const int (&tok)[2], bool edge,
                                     int first, int end, int lane) {
  // every read of the stage first (LATE: of the keys)
  uint32_t kc[2][C::NG][C::KW], kbw[2][C::BW], ks[2][C::SW], vs[2][C::SW], vb[2][C::SW], vc[2][4][C::NG][C::VW];
  auto read_values = [&](int u, int g) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_bytes<(C::VBITS < 8 ? 1 : C::VBITS / 8)>(st + (2 + u) * C::CODES + i * C::ROWB + ln.v[g], vc[u][i][g]);
  };
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* par = st + 4 * C::CODES + u * 4 * C::PARAMS;
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
      load_bytes<(C::KB > 16 ? 16 : C::KB)>(st + u * C::CODES + ln.k[g][0], kc[u][g]);
      if constexpr (C::KB > 16) load_bytes<16>(st + u * C::CODES + ln.k[g][1], kc[u][g] + 4);
    }
    load_bytes<2 * C::NG>(par + C::PARAMS + ln.kb, kbw[u]);
    load_bytes<2 * C::TOK * C::NG>(par + ln.par, ks[u]);
  }
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    const uint8_t* par = st + 4 * C::CODES + (u * 4 + 2) * C::PARAMS + ln.par;
    load_bytes<2 * C::TOK * C::NG>(par, vs[u]);
    if constexpr (!C::LATE) {
      load_bytes<2 * C::TOK * C::NG>(par + C::PARAMS, vb[u]);
#pragma unroll
      for (int g = 0; g < C::NG; ++g) read_values(u, g);
    }
  }
  float z[2][C::TOK], p[2][C::TOK];
  const int sub = sub_of<C>(lane);
#pragma unroll
  for (int u = 0; u < 2; ++u) {
    u32x4_t kb = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < C::BW; ++i) kb[i] = kbw[u][i];
    const f32x4_t zb = mfma_act<C::ACT16>(kb, w.qsum, f32x4_t{0.f, 0.f, 0.f, 0.f});
    f32x4_t acc[C::NG];
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
      acc[g] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < C::KS; ++s)
        acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_f16(key_codes<C>(kc[u][g], s), w.q[g][s], acc[g], 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < C::TOK; ++i) {
      z[u][i] = own<C>(zb, i, sub) * (1.f / C::QSUM);
#pragma unroll
      for (int g = 0; g < C::NG; ++g) z[u][i] = fmaf(half_at<C::ACT16>(ks[u], i * C::NG + g), own<C>(acc[g], i, sub), z[u][i]);
    }
  }
  // tokens that do not count get p = 0 and finite parameters
  auto counts = [&](int u, int i, int at) {
    const int t = tok[u] + at + i;
    return tok[u] >= 0 && t >= first && t < end;
  };
  auto hide = [&](uint32_t* x, int i) {
#pragma unroll
    for (int k = i * C::NG; k < (i + 1) * C::NG; ++k) x[k / 2] &= (k & 1) ? 0xffffu : 0xffff0000u;
  };
  if (edge) {
    int at = 4 * (lane >> 4) + C::TOK * sub;
    asm volatile("" : "+v"(at));  // (keeps the comparisons below inside the branch)
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < C::TOK; ++i)
        if (!counts(u, i, at)) {
          z[u][i] = -__builtin_inff();
          hide(vs[u], i);
          if constexpr (!C::LATE) hide(vb[u], i);
        }
  }
  float zmax = fmaxf(z[0][0], z[1][0]);
#pragma unroll
  for (int i = 1; i < C::TOK; ++i) zmax = fmaxf(zmax, fmaxf(z[0][i], z[1][i]));
  zmax *= w.zscale;
  if (any_lane(zmax > w.mlim)) raise<C>(w, z, vs, zmax);
  const float off = PBIAS - w.mu;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < C::TOK; ++i) p[u][i] = __builtin_amdgcn_exp2f(fmaf(z[u][i], w.zscale, off));
  Weights<C> x;
#pragma unroll
  for (int g = 0; g < C::NG; ++g) weights<C>(p, vs, g, w.ve[g], x.a[g]);
  uint32_t amax = x.a[0][0];
#pragma unroll
  for (int i = 1; i < 2 * Weights<C>::W * C::NG; ++i)
    amax = pk_max_u16(amax, x.a[i / (2 * Weights<C>::W)][i % (2 * Weights<C>::W)]);
  // (a scale below zero sets the top bit and passes the limit every time)
  if (any_lane(max(amax >> 16, amax & 0xffffu) > ALIM)) retarget<C>(w, p, vs, x);
  if constexpr (C::LATE) {
#pragma unroll
    for (int u = 0; u < 2; ++u) load_bytes<2 * C::TOK * C::NG>(st + 4 * C::CODES + (u * 4 + 3) * C::PARAMS + ln.par, vb[u]);
    if (edge) {
      int at = 4 * (lane >> 4) + C::TOK * sub;
      asm volatile("" : "+v"(at));
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int i = 0; i < C::TOK; ++i)
          if (!counts(u, i, at)) hide(vb[u], i);
    }
  }
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < C::TOK; ++i) {
      w.l += p[u][i];
#pragma unroll
      for (int g = 0; g < C::NG; ++g)
        w.bias[g] = fmaf(p[u][i], half_at<C::ACT16>(vb[u], i * C::NG + g), w.bias[g]);
    }
#pragma unroll
  for (int g = 0; g < C::NG; ++g) {
    uint32_t aw[4];  // pairs of the quarter's tokens; zeros for those that are not this lane's
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int k = 0; k < 2; ++k) aw[2 * u + k] = C::FOLD == 1 ? x.a[g][2 * u + k] : x.a[g][u] & ln.keep[k];
    const f16x8_t A = as_f16x8(aw[0], aw[1], aw[2], aw[3]);
    constexpr int PIECES = C::VBITS <= 16 ? 1 : C::VBITS / 16;
    if constexpr (C::LATE) {
      read_values(0, g);
      read_values(1, g);
    }
    uint32_t pr[PIECES][4];  // [piece][pair of tokens]
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = k >> 1, i = 2 * (k & 1);
      const uint32_t* x = vc[u][i][g];
      const uint32_t* y = vc[u][i + 1][g];
#pragma unroll
      for (int b = 0; b < PIECES; ++b)
        pr[b][k] = __builtin_amdgcn_perm(y[b / 2], x[b / 2], (b & 1) ? 0x07060302u : 0x05040100u);
      // two lanes share a byte of 2-bit codes where a group gives a lane two columns
      if constexpr (C::VBITS == 4) pr[0][k] >>= 4 * (lane & 1);
    }
#pragma unroll
    for (int c = 0; c < C::VC; ++c) {
      const int b = c / (16 / C::BITS) % PIECES;
      w.o[g][c] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
          as_f16x8(value_pair<C>(pr[b][0], c), value_pair<C>(pr[b][1], c), value_pair<C>(pr[b][2], c),
                   value_pair<C>(pr[b][3], c)),
          A, w.o[g][c], 0, 0, 0);
    }
  }
}

// What starting a unit costs a workgroup, in tiles; nothing where each takes
// one tile.  (Without it, a workgroup that a ragged batch gives many short
// units is the last: 64 sequences up to 8192 tokens, 4-bit, 90 us at 0, 67 at
// 2 and at 3; equal lengths the same.)
__device__ __forceinline__ int start_cost(int64_t tiles, int64_t workgroups) { return tiles <= workgroups ? 0 : 2; }

// Tokens [first, len) of sequence b; returns its tiles of 128 tokens from the
// 16-token tile of `first` on, at least one.
__device__ __forceinline__ int tiles_of(const PagedAttnArgs& a, int b, int& first, int& len) {
  len = (int)max(0l, min((long)a.seq_lens[b], (long)a.max_pages * a.c.page_size));
  first = a.window > 0 ? (int)max(0l, (long)len - a.window) : 0;
  return max(1, (int)(((long)len - (first & ~15) + 127) >> 7));
}

__device__ __forceinline__ uint32_t quotient(uint64_t n, uint64_t d) {
  return ((n | d) >> 32) == 0 ? (uint32_t)n / (uint32_t)d : (uint32_t)(n / d);
}

// inclusive sum over the 64 lanes
template <int CTRL, int ROWS>
__device__ __forceinline__ int scan_step(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int wave_scan(int v) {
  v = scan_step<0x111, 0xf>(v);  // row_shr:1, 2, 4, 8
  v = scan_step<0x112, 0xf>(v);
  v = scan_step<0x114, 0xf>(v);
  v = scan_step<0x118, 0xf>(v);
  v = scan_step<0x142, 0xa>(v);     // row_bcast:15 into rows 1 and 3
  return scan_step<0x143, 0xc>(v);  // row_bcast:31 into rows 2 and 3
}

// The work of all (sequence, unit of heads), in that order, on one line: each
// unit's start (start_cost) and then its tiles.  Where point x of it lies.
struct Place {
  int b, unit, at;
  int tiles, first, len;  // of the sequence
  int64_t start;          // its start on the line of one unit
};

// The batch as every wave sees it, a lane a sequence of the 64 at hand.
struct Batch {
  int b0, tiles, first, len;  // tiles with the start, 0 past the batch
  int lead;                   // a unit's start
  int64_t start;              // of sequence b0 on the line of one unit
};

__device__ __forceinline__ void batch_at(const AttnWork& w, int b0, Batch& s) {
  const int b = b0 + (int)(threadIdx.x & 63);
  s.b0 = b0;
  s.tiles = s.first = s.len = 0;
  if (b < w.a.B) s.tiles = s.lead + tiles_of(w.a, b, s.first, s.len);
}

// The line's length for one unit, with the first 64 sequences left at hand:
// no barrier, and at 64 sequences or fewer, one load.
__device__ __forceinline__ int64_t line_of(const AttnWork& w, int units, Batch& s) {
  double total = 0.0;
  s.lead = 0;
  for (int b0 = 64; b0 < w.a.B; b0 += 64) {
    batch_at(w, b0, s);
    total += s.tiles;
  }
  batch_at(w, 0, s);
  s.start = 0;
  const uint64_t n = (uint64_t)wave_sum_f64(total + s.tiles);  // (the same in every lane)
  const int64_t tiles = (int64_t)((uint64_t)__builtin_amdgcn_readfirstlane((uint32_t)(n >> 32)) << 32 |
                                  __builtin_amdgcn_readfirstlane((uint32_t)n));
  s.lead = start_cost(tiles * units, gridDim.x);
  if (s.tiles > 0) s.tiles += s.lead;
  return tiles + (int64_t)s.lead * w.a.B;
}

// Finds point x, at or past the sequences at hand.
__device__ __forceinline__ Place find_tile(const AttnWork& w, Batch& s, int64_t x, int units) {
  Place p;
  for (;;) {
    const int upto = wave_scan(s.tiles);
    const int64_t rel = x - s.start * units;  // (the first lane whose sequences up to it pass it)
    const uint64_t hit = __builtin_amdgcn_ballot_w64((int64_t)upto * units > rel);
    if (hit != 0 || s.b0 + 64 >= w.a.B) {
      const int l = __builtin_ctzll(hit | (uint64_t(1) << 63));
      p.b = s.b0 + l;
      const int line = __builtin_amdgcn_readlane(s.tiles, l);
      p.tiles = line - s.lead;
      p.first = __builtin_amdgcn_readlane(s.first, l);
      p.len = __builtin_amdgcn_readlane(s.len, l);
      p.start = s.start + __builtin_amdgcn_readlane(upto, l) - line;
      const uint64_t in = (uint64_t)(x - p.start * units);
      p.unit = (int)quotient(in, (uint32_t)line);
      p.at = (int)(in - (uint64_t)p.unit * (uint32_t)line);
      return p;
    }
    s.start += __builtin_amdgcn_readlane(upto, 63);
    batch_at(w, s.b0 + 64, s);
  }
}

// Attention of one unit of heads (key head, tile of 16 query heads) of
// sequence b to its tokens [begin, end) from `first` on, by all waves of the
// workgroup: written out if that is `whole`, else left as a part in `slot`.
template <class C>
__device__ __forceinline__ void attend(const AttnWork& wk, uint8_t* smem, float (&msh)[C::WAVES][16],
                                       float (&lsh)[C::WAVES][16], int b, int unit, int first, int begin, int end,
                                       bool whole, size_t slot) {
  constexpr int WAVES = C::WAVES, TILE = 32 * WAVES;
  const PagedAttnArgs& a = wk.a;
  const KvCache& c = a.c;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int n16 = lane & 15, kq = lane >> 4, sub = sub_of<C>(lane), head = n16 % C::HEADS;
  float* lds = reinterpret_cast<float*>(smem);
  const int j = unit / wk.htiles, ht = unit - j * wk.htiles;
  const int h0 = j * wk.share + C::HEADS * ht, gm = min(C::HEADS, wk.share - C::HEADS * ht);  // this unit's heads

  // q: lane (head n16, quarter kq) holds columns [kq G/4, (kq+1) G/4) of each group
  uint32_t qraw[C::NG][C::G / 8];
  {
    const uint16_t* q = (const uint16_t*)a.q + (long)b * a.qts + (long)(h0 + min(head, gm - 1)) * a.qhs;
#pragma unroll
    for (int g = 0; g < C::NG; ++g) load_bytes<C::G / 2>((const uint8_t*)(q + g * C::G + kq * (C::G / 4)), qraw[g]);
  }
  Wave<C> w;
#pragma unroll
  for (int g = 0; g < C::NG; ++g) {
    w.bias[g] = 0.f;
    w.ve[g] = __builtin_amdgcn_ldexpf(1.f, VEMAX);
#pragma unroll
    for (int v = 0; v < C::VC; ++v) w.o[g][v] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  w.l = 0.f;
  w.mref = w.mlim = -__builtin_inff();
  w.mu = 0.f;

  // this wave's steps: tokens begin + 32 (wave + WAVES i)
  const int t0 = begin + 32 * wave;
  const int steps = t0 < end ? (end - t0 + TILE - 1) / TILE : 0;
  if (steps > 0) {
    const int32_t* table = a.table + (long)b * a.table_stride;
    // lane k: where 16-token tile k of 32 steps lies, in tiles of the cache's rows; -1: no such tile, or its page is outside
    int at = -1, at_from = -32;
    Lanes<C> ln;
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
      const int col = g * (C::G * C::BITS / 8);
      ln.k[g][0] = (uint32_t)C::at(n16, col + kq * C::KB);
      if constexpr (C::KB > 16) ln.k[g][1] = (uint32_t)C::at(n16, col + kq * C::KB + 16);
      ln.v[g] = (uint32_t)C::at(4 * kq, col + n16 * C::VBITS / 8);
    }
    ln.par = (uint32_t)((4 * kq + C::TOK * sub) * 2 * C::NG);
#pragma unroll
    for (int k = 0; k < 2; ++k)
      ln.keep[k] = (C::TOK * sub / 2 != k) ? 0u : C::FOLD == 4 ? 0xffffu << (16 * (sub & 1)) : ~0u;
    ln.kb = (uint32_t)(n16 * 2 * C::NG);
    // what this lane copies: 16-byte piece 64 m + lane of 16 tokens' codes, and of a stage's parameters
    uint32_t src[C::COPIES];
#pragma unroll
    for (int m = 0; m < C::COPIES; ++m) {
      const int q = 64 * m + lane;
      if constexpr (C::PIECES > 0) {
        const int row = q / C::PIECES;
        src[m] = (uint32_t)(row * C::ROWB + ((q % C::PIECES ^ C::swizzle(row)) << 4));
      } else {
        src[m] = (uint32_t)(16 * q);
      }
    }
    const uint8_t* psrc[C::PCOPIES];
    bool phalf[C::PCOPIES];
#pragma unroll
    for (int m = 0; m < C::PCOPIES; ++m) {
      const int q = 64 * m + lane, part = q / (2 * C::NG);  // part = 4 half + kind
      const void* const kind[4] = {c.k_scales, c.k_biases, c.v_scales, c.v_biases};
      psrc[m] = (const uint8_t*)((part & 2) ? ((part & 1) ? kind[3] : kind[2]) : ((part & 1) ? kind[1] : kind[0])) +
                16 * (q % (2 * C::NG));
      phalf[m] = part >= 4;
    }
    const uint32_t ring = __builtin_amdgcn_readfirstlane(
        (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)smem + wave * C::STAGES * C::STAGE);
    auto copy = [&](int i, uint32_t dst) {  // stage i of this wave (page 0 in the place of one outside the cache)
      if (i >= at_from + 32) {  // uniform
        at_from = i;
        const int tok = t0 + TILE * (i + (lane >> 1)) + 16 * (lane & 1);
        const uint32_t tk = (uint32_t)min(tok, end - 1) & ~15u, pg = wk.page.div(tk);
        const int id = table[pg];
        const uint32_t tiles = (uint32_t)c.page_size >> 4;  // (fewer than 2^31 in any memory)
        at = tok < end && (uint32_t)id < (uint32_t)c.num_pages
                 ? (int)(((uint32_t)id * (uint32_t)c.kv_heads + (uint32_t)j) * tiles + ((tk - pg * wk.page.d) >> 4))
                 : -1;
      }
      uint32_t row[2];  // in tiles
#pragma unroll
      for (int u = 0; u < 2; ++u) row[u] = (uint32_t)max(__builtin_amdgcn_readlane(at, 2 * (i - at_from) + u), 0);
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const uint8_t* base = (const uint8_t*)(p < 2 ? c.k_packed : c.v_packed) + (size_t)row[p & 1] * C::CODES;
        copies<C::CODES / 16>([&](auto m, auto lanes) {
          copy_to_lds<decltype(lanes)::value>(base, src[decltype(m)::value], dst + p * C::CODES + 1024 * decltype(m)::value);
        });
      }
      copies<8 * C::PARAMS / 16>([&](auto m, auto lanes) {
        constexpr int M = decltype(m)::value;
        copy_to_lds<decltype(lanes)::value>(psrc[M] + (size_t)(phalf[M] ? row[1] : row[0]) * C::PARAMS,
                                            dst + 4 * C::CODES + 1024 * M);
      });
    };
    copy(0, ring);
    // (q's conversion stays behind the last of these copies: it waits for q, and with it for them)
#pragma unroll
    for (int g = 0; g < C::NG; ++g)
#pragma unroll
      for (int k = 0; k < C::G / 8; ++k) asm volatile("" : "+v"(qraw[g][k]));
    set_q<C>(w, qraw, head < gm, kq, a.scale);
    // the tiles of the stage being computed: the copies run ahead and may have gone on to the next 32 steps'
    int at_now = at, at_now_from = 0;
    uint32_t buf = 0;
    for (int i = 0; i < steps; ++i) {
      wait_copies();  // stage i is in LDS
      if (i == at_now_from + 32) {
        at_now = at;
        at_now_from = at_from;
      }
      // the reads of stage i - 1, whose place the next copies take, are done
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (i + 1 < steps) copy(i + 1, ring + (buf ^ C::STAGE));
      int tok[2];
      bool edge = false;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int t = t0 + TILE * i + 16 * u;
        const bool there = __builtin_amdgcn_readlane(at_now, 2 * (i - at_now_from) + u) >= 0;
        tok[u] = there ? t : -1;
        edge |= !there || t < first || t + 16 > end;
      }
      step<C>(w, smem + wave * C::STAGES * C::STAGE + buf, ln, tok, edge, first, end, lane);
      buf ^= C::STAGE;
    }
  }
  __syncthreads();
  // join the waves
  w.l = fold_sum<C>(quads_sum(w.l));
  const float m_own = (w.mref == -__builtin_inff() && w.l == w.l) ? -__builtin_inff() : w.mu;
  if (kq == 0 && sub == 0) {
    msh[wave][head] = m_own;
    lsh[wave][head] = w.l;
  }
  const int stride = C::D + 4;
#pragma unroll
  for (int g = 0; g < C::NG; ++g) {
    const float bs = fold_sum<C>(quads_sum(w.bias[g])), back = 0x1p24f / w.ve[g];
#pragma unroll
    for (int v = 0; v < C::VC; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i) w.o[g][v][i] = fold_sum<C>(w.o[g][v][i]);
    if (sub == 0 && head < gm) {
      float* dst = lds + (wave * gm + head) * stride + g * C::G + 4 * kq * C::VC;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < C::VC; ++v)
          dst[i * C::VC + v] = fmaf(w.o[g][v][i], back / (float)(1 << value_shift<C>(v)), bs);
    }
  }
  __syncthreads();
  const int gstore = min(16, wk.share);
  for (int i = t; i < gm * (C::D / 4); i += 64 * WAVES) {
    const int h = i / (C::D / 4), d4 = i - h * (C::D / 4);
    float m = msh[0][h];
#pragma unroll
    for (int k = 1; k < WAVES; ++k) m = fmaxf(m, msh[k][h]);
    f32x4_t o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
#pragma unroll
    for (int k = 0; k < WAVES; ++k) {
      const float f = msh[k][h] == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(msh[k][h] - m);
      const f32x4_t ok = *reinterpret_cast<const f32x4_t*>(lds + (k * gm + h) * stride + 4 * d4);
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = fmaf(f, ok[e], o[e]);
      l = fmaf(f, lsh[k][h], l);
    }
    if (whole) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      u32x2_t pk;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        pk[e] = (uint32_t)f32_to_act_bits(o[2 * e] * inv, C::ACT16) |
                (uint32_t)f32_to_act_bits(o[2 * e + 1] * inv, C::ACT16) << 16;
      *reinterpret_cast<u32x2_t*>((uint16_t*)a.out + ((size_t)b * a.heads + h0 + h) * C::D + 4 * d4) = pk;
    } else {
      *reinterpret_cast<f32x4_t*>(wk.part_o + (slot * gstore + h) * C::D + 4 * d4) = o;
      if (d4 == 0) {
        wk.part_ml[(slot * gstore + h) * 2] = m;
        wk.part_ml[(slot * gstore + h) * 2 + 1] = l;
      }
    }
  }
}

// Every workgroup takes an equal stretch of the line of all units' work: whole
// units, and at its ends parts of units that it shares with its neighbours.
// The lengths are on the device, so each finds its own from them.
template <class C>
__global__ __launch_bounds__(256, C::PER_CU) void paged_attn_kernel(AttnWork wk) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float msh[C::WAVES][16], lsh[C::WAVES][16];
  const PagedAttnArgs& a = wk.a;
  const int units = a.c.kv_heads * wk.htiles;
  Batch batch;
  const int64_t all = line_of(wk, units, batch) * units;
  const int64_t share = (all + gridDim.x - 1) / gridDim.x;
  const int64_t xend = min(share * (blockIdx.x + 1), all);
  if (blockIdx.x == 0 && threadIdx.x == 0) wk.meta[a.B] = AttnMeta{share, batch.lead};
  for (int64_t x = share * blockIdx.x; x < xend;) {
    const Place p = find_tile(wk, batch, x, units);
    const int take = (int)min((int64_t)(batch.lead + p.tiles - p.at), xend - x);
    if (p.unit == 0 && p.at == 0 && threadIdx.x == 0) wk.meta[p.b] = AttnMeta{p.start, p.tiles};
    const int tile = max(p.at - batch.lead, 0), tend = p.at + take - batch.lead;
    if (tend > tile) {  // uniform
      const int begin = (p.first & ~15) + 128 * tile;
      // a part that is not its unit's first is its workgroup's first
      attend<C>(wk, smem, msh, lsh, p.b, p.unit, p.first, begin, min((p.first & ~15) + 128 * tend, p.len),
                tend - tile == p.tiles, 2 * (size_t)blockIdx.x + (tile == 0));
    }
    x += take;
    if (x < xend) __syncthreads();
  }
}

// One workgroup per sequence and unit: short tables, no parts, one launch.
template <class C>
__global__ __launch_bounds__(64 * C::WAVES, C::WAVES == 4 ? C::PER_CU : 1) void paged_attn_short_kernel(AttnWork wk) {
  extern __shared__ __align__(1024) uint8_t smem[];
  __shared__ float msh[C::WAVES][16], lsh[C::WAVES][16];
  const int units = wk.a.c.kv_heads * wk.htiles;
  const int b = (int)blockIdx.x / units;
  int first, len;
  tiles_of(wk.a, b, first, len);
  first = __builtin_amdgcn_readfirstlane(first);
  len = __builtin_amdgcn_readfirstlane(len);
  attend<C>(wk, smem, msh, lsh, b, (int)blockIdx.x - b * units, first, first & ~15, len, true, 0);
}

// Joins the parts of one sequence and head: 32 lanes by GROUPS groups of parts.
template <bool F16_, int GROUPS>
__global__ __launch_bounds__(32 * GROUPS) void paged_attn_join_kernel(AttnWork wk) {
  const PagedAttnArgs& a = wk.a;
  const int b = blockIdx.y, head = blockIdx.x, t = threadIdx.x, D = a.c.head_dim;
  const AttnMeta mt = wk.meta[b];
  const uint64_t share = (uint64_t)wk.meta[a.B].start;
  const uint32_t lead = (uint32_t)wk.meta[a.B].tiles;
  const int j = head / wk.share, ht = (head - j * wk.share) / 16, h = head - j * wk.share - 16 * ht;
  const int gstore = min(16, wk.share);
  __shared__ float msh[GROUPS], osh[GROUPS][256 + 4], lsh[GROUPS];
  // the workgroups of this unit's first and last tile
  const uint64_t x0 = (uint64_t)mt.start * (a.c.kv_heads * wk.htiles) +
                      (uint64_t)(j * wk.htiles + ht) * (lead + mt.tiles) + lead;
  const uint32_t w0 = quotient(x0, share), w1 = quotient(x0 + mt.tiles - 1, share);
  if (w0 == w1) return;
  const int n = (int)(w1 - w0) + 1;
  auto at = [&](int k) { return (2 * (size_t)(w0 + k) + (k == 0)) * gstore + h; };
  const int grp = t >> 5, ln = t & 31;
  f32x4_t o[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  float m = -__builtin_inff(), l = 0.f;
  for (int k0 = grp; k0 < n; k0 += GROUPS * 4) {  // four parts' loads in flight
    f32x2_t ml[4];
    f32x4_t v[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const size_t s = at(min(k0 + GROUPS * i, n - 1));
      ml[i] = *reinterpret_cast<const f32x2_t*>(wk.part_ml + 2 * s);
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (4 * ln + 128 * e < D) v[i][e] = *reinterpret_cast<const f32x4_t*>(wk.part_o + s * D + 4 * ln + 128 * e);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (k0 + GROUPS * i >= n || ml[i][0] == -__builtin_inff()) continue;  // (a part that saw nothing)
      const float mn = fmaxf(m, ml[i][0]);
      const float fo = __builtin_amdgcn_exp2f(m - mn), fn = __builtin_amdgcn_exp2f(ml[i][0] - mn);
      m = mn;
      l = l * fo + ml[i][1] * fn;
#pragma unroll
      for (int e = 0; e < 2; ++e)
        if (4 * ln + 128 * e < D)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[e][c] = o[e][c] * fo + v[i][e][c] * fn;
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) *reinterpret_cast<f32x4_t*>(&osh[grp][4 * ln + 128 * e]) = o[e];
  if (ln == 0) {
    msh[grp] = m;
    lsh[grp] = l;
  }
  __syncthreads();
  if (t < D) {
    m = msh[0];
#pragma unroll
    for (int k = 1; k < GROUPS; ++k) m = fmaxf(m, msh[k]);
    float s = 0.f, ls = 0.f;
#pragma unroll
    for (int k = 0; k < GROUPS; ++k) {
      const float f = msh[k] == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(msh[k] - m);
      s = fmaf(f, osh[k][t], s);
      ls = fmaf(f, lsh[k], ls);
    }
    ((uint16_t*)a.out)[((size_t)b * a.heads + head) * D + t] = f32_to_act_bits(ls == 0.f ? 0.f : s / ls, F16_);
  }
}

// LDS of a launch: the ring, and after the loop [WAVES][heads][D + 4] floats
template <class C>
size_t attn_lds(int heads) {
  return std::max<size_t>(C::LDS, (size_t)C::WAVES * heads * (C::D + 4) * 4);
}

template <int D, int G, int BITS, bool F16_, int FOLD>
hipError_t launch_cfg(AttnWork& w, hipStream_t s) {
  using C = Cfg<D, G, BITS, F16_, FOLD, 4>;
  // eight waves where their stages fit
  using S = Cfg<D, G, BITS, F16_, FOLD, (Cfg<D, G, BITS, F16_, FOLD, 8>::LDS <= 155 * 1024 ? 8 : 4)>;
  const PagedAttnArgs& a = w.a;
  const int gm = w.share < 16 ? w.share : 16;
  const int64_t units = (int64_t)a.c.kv_heads * w.htiles;
  // the most tokens a sequence can see, and with them the rest of the window's first 16-token tile
  const int64_t table = (int64_t)a.max_pages * a.c.page_size;
  const int64_t seen = a.window > 0 ? std::min(table, a.window) : table;
  const int64_t tokens = a.window > 0 && a.window < table ? std::min(table, a.window + 15) : table;
  w.part_o = w.part_ml = nullptr;
  w.meta = nullptr;
  // Short sequences: a workgroup each, no parts, no second kernel.  A step
  // costs in proportion to D, and the more workgroups, the less the other
  // kernel gains by cutting sequences: up to 80K columns and tokens a unit, or
  // 2304 a workgroup (D = 128, 4-bit, 8 units: 576 tokens 8.1 against 8.8 us,
  // 1024 10.2 against 8.9; 64 units: 1024 10.7 against 11.5, 2048 15.2 against
  // 14.4; D = 256, 8 units: 320 9.7 against 10.3, 1024 14.1 against 10.5; 256
  // units: 2048 29 against 33).  Always up to 160 tokens, which callers who
  // capture a first call rely on.  Eight waves share a unit, four when there are
  // more than the CUs (128 sequences of 512 tokens: 24.5 against 32 us).
  const int64_t wgs = units * a.B;
  const int64_t cost = tokens * D * (8 / S::WAVES);
  if (tokens <= 2048 && (seen <= 160 || cost <= std::max<int64_t>(80 * 1024, 2304 * wgs)) &&
      wgs < (1 << 24)) {  // (2^32 threads at most in a launch)
    if (wgs > 256)
      hipLaunchKernelGGL(paged_attn_short_kernel<C>, dim3((unsigned)wgs), dim3(256), attn_lds<C>(gm), s, w);
    else
      hipLaunchKernelGGL(paged_attn_short_kernel<S>, dim3((unsigned)wgs), dim3(64 * S::WAVES), attn_lds<S>(gm), s, w);
    return hipGetLastError();
  }
  const size_t lds = attn_lds<C>(gm);
  int64_t resident = 0;
  hipError_t e = resident_workgroups(reinterpret_cast<const void*>(&paged_attn_kernel<C>), 256, lds, 8, &resident);
  if (e != hipSuccess) return e;
  const int64_t grid = std::min(resident, units * a.B * ((tokens + 127) / 128));  // (a workgroup a tile at most)
  const size_t slots = 2 * (size_t)grid;
  const size_t meta = ((a.B + 1) * sizeof(AttnMeta) + 255) & ~size_t(255);
  const size_t ml = (slots * gm * 2 * sizeof(float) + 255) & ~size_t(255);
  void* p = nullptr;
  e = stream_workspace(s, meta + ml + slots * gm * D * sizeof(float), &p);
  if (e != hipSuccess) return e;
  w.meta = static_cast<AttnMeta*>(p);
  w.part_ml = reinterpret_cast<float*>(static_cast<char*>(p) + meta);
  w.part_o = reinterpret_cast<float*>(static_cast<char*>(p) + meta + ml);
  hipLaunchKernelGGL(paged_attn_kernel<C>, dim3((unsigned)grid), dim3(256), lds, s, w);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const dim3 rows((unsigned)a.heads, (unsigned)a.B);
  // more than 32 parts a unit: one round of loads instead of three or four (131072 tokens: 34.6 against 35.1 us)
  if (grid > 32 * units * a.B)
    hipLaunchKernelGGL((paged_attn_join_kernel<F16_, 32>), rows, dim3(1024), 0, s, w);
  else
    hipLaunchKernelGGL((paged_attn_join_kernel<F16_, 8>), rows, dim3(256), 0, s, w);
  return hipGetLastError();
}

template <int D, int G, int BITS, bool F16_>
hipError_t launch_heads(AttnWork& w, hipStream_t s) {
  // a head takes as many columns as there are (64 sequences of 4096 tokens, D = 128, G = 64, 4-bit, four heads a key
  // head: 60.8 us, with one column each 69.3; eight heads: 67.4 and 73.4, with G = 32 86 and 95)
  return w.share <= 4   ? launch_cfg<D, G, BITS, F16_, 4>(w, s)
         : w.share <= 8 ? launch_cfg<D, G, BITS, F16_, 2>(w, s)
                        : launch_cfg<D, G, BITS, F16_, 1>(w, s);
}

}  // namespace

template <int BITS>
hipError_t launch_paged_attention_bits(const PagedAttnArgs& a, hipStream_t s) {
  AttnWork w{a, FastDiv((uint32_t)a.c.page_size)};
  w.share = a.heads / a.c.kv_heads;
  w.htiles = (w.share + 15) / 16;
#define QAFF_ATTN(D, G)                                                            \
  case D * 1000 + G:                                                               \
    return a.c.dt == F16 ? launch_heads<D, G, BITS, true>(w, s) : launch_heads<D, G, BITS, false>(w, s);
  switch (a.c.head_dim * 1000 + a.c.G) {
    QAFF_ATTN(64, 32)
    QAFF_ATTN(64, 64)
    QAFF_ATTN(96, 32)
    QAFF_ATTN(128, 32)
    QAFF_ATTN(128, 64)
    QAFF_ATTN(128, 128)
    QAFF_ATTN(192, 32)
    QAFF_ATTN(192, 64)
    QAFF_ATTN(256, 32)
    QAFF_ATTN(256, 64)
    QAFF_ATTN(256, 128)
    default: return hipErrorNotSupported;
  }
#undef QAFF_ATTN
}

}  // namespace qaff
