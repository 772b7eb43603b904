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
//              with A_g[t,h] = p[t,h] vs[t,g] rounded to f16
// Codes: an f16 whose exponent bits are zero is its low ten bits times 2^-24,
// and the matrix cores keep such numbers, so masking a code where it lies in
// bits 0-9 of each 16-bit half (4-bit: bits 0-3 and, times 16, bits 4-7) is
// the whole conversion: one AND for two codes.  The factors 2^24 and 16 go to
// q (exact powers of two, per column) and to the outputs.
// Registers: C_g has the tokens of a lane's quarter (lane / 16) as rows and
// the head (lane % 16) as column, which is where the value product takes its
// second operand from, so p never leaves the lane.  Value codes arrive as
// rows of tokens and are wanted as pairs of tokens: two tokens' codes of the
// same columns are put into the halves of one register first.
// q is scaled by a power of two per head so that its largest entry lies in
// [2^14, 2^15): exact for f16 queries and, below 2^-29 of the largest, off by
// at most 2^-39 of it for bf16 ones.
// The softmax's reference mu is the largest logit seen plus the exponent of
// the largest value scale seen, p = 2^(z - mu + 5): A stays below 2^15 while
// z grows by no more than 4 and vs by no more than 2^6, so most steps need
// neither a maximum over the lanes nor a rescaling; a step that passes the
// limits (a wave-uniform branch) sets a new mu.  A's smallest step is 2^-24,
// 2^-30 of the largest term.
//
// Work: the tokens of all sequences are cut into chunks of about equal size
// (the lengths are on the device, so each workgroup finds its chunk from
// them: a sum and a scan over the batch); four waves share a chunk, joined
// through LDS.  A sequence of one chunk is written out at once; the others
// leave fp32 partial sums with their mu, joined by a second kernel.
// Instantiated per code width in paged_attention_b{2,4,8}.hip.
#pragma once

#include "common.h"

namespace qaff {
namespace {

constexpr int WAVES = 4;
constexpr float PBIAS = 5.f;    // log2 of p at the reference
constexpr float MROOM = 4.f;    // how far a logit may pass the reference (log2)
constexpr float VROOM = 64.f;   // how far a value scale may pass it

struct AttnWork {
  PagedAttnArgs a;
  FastDiv page;         // tokens a page
  int share, htiles;    // query heads a key head; tiles of 16 of them
  int target, min_chunk;
  float* part_o;        // [slot][gm][D]
  float* part_ml;       // [slot][gm][2]
  int2* meta;           // [B]: chunks, first slot
};

template <int D_, int G_, int BITS_, bool F16_>
struct Cfg {
  static constexpr int D = D_, G = G_, BITS = BITS_, NG = D / G;
  static constexpr bool ACT16 = F16_;
  static constexpr int KS = G / 32;                      // product steps a group (keys)
  static constexpr int KB = G / 4 * BITS / 8;            // key code bytes a lane and group
  static constexpr int KW = KB < 4 ? 1 : KB / 4;
  static constexpr int VC = G / 16;                      // value columns a lane and group
  static constexpr int VBITS = VC * BITS;                // value code bits a lane, token and group
  static constexpr int VW = VBITS <= 32 ? 1 : 2;
  static constexpr int SW = 2 * NG;                      // words of four tokens' scales
  static constexpr int ROWB = D * BITS / 8;
};

template <class C>
struct Raw {  // what a step reads, as it lies in memory
  uint32_t kc[2][C::NG][C::KW], ks[2][C::SW], kb[2][C::SW];
  uint32_t vc[2][4][C::NG][C::VW], vs[2][C::SW], vb[2][C::SW];
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
  float qsum[C::NG];
  float zscale;           // logits to base 2, with q's power of two and the codes' taken back
  // running
  f32x4_t o[C::NG][C::VC];
  float l, bias[C::NG];   // sums over this lane's tokens
  float mref, mu, mlim, vexp, vlim;
};

template <class C>
__device__ __forceinline__ void load_raw(Raw<C>& r, int u, const KvCache& c, size_t row, uint32_t kvo, uint32_t vvo,
                                         uint32_t svo) {
  const uint8_t* kc = (const uint8_t*)c.k_packed + row * C::ROWB;
  const uint8_t* vc = (const uint8_t*)c.v_packed + row * C::ROWB;
  const size_t so = row * (2 * C::NG);
#pragma unroll
  for (int g = 0; g < C::NG; ++g) load_bytes<C::KB>(kc + kvo + g * (C::G * C::BITS / 8), r.kc[u][g]);
  load_bytes<8 * C::NG>((const uint8_t*)c.k_scales + so + svo, r.ks[u]);
  load_bytes<8 * C::NG>((const uint8_t*)c.k_biases + so + svo, r.kb[u]);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int g = 0; g < C::NG; ++g)
      load_bytes<(C::VBITS < 8 ? 1 : C::VBITS / 8)>(vc + vvo + i * C::ROWB + g * (C::G * C::BITS / 8), r.vc[u][i][g]);
  load_bytes<8 * C::NG>((const uint8_t*)c.v_scales + so + svo, r.vs[u]);
  load_bytes<8 * C::NG>((const uint8_t*)c.v_biases + so + svo, r.vb[u]);
}

// 32 tokens; bit 4 u + i of `live`: token 16 u + 4 (lane / 16) + i counts
// (all of the wave's do unless `edge`)
template <class C>
__device__ __forceinline__ void step(Wave<C>& w, const Raw<C>& r, bool edge, uint32_t live, int lane) {
  float z[2][4], p[2][4];
#pragma unroll
  for (int u = 0; u < 2; ++u) {
#pragma unroll
    for (int i = 0; i < 4; ++i) z[u][i] = 0.f;
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
      f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int s = 0; s < C::KS; ++s)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(key_codes<C>(r.kc[u][g], s), w.q[g][s], acc, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        z[u][i] = fmaf(half_at<C::ACT16>(r.ks[u], i * C::NG + g), acc[i], z[u][i]);
        z[u][i] = fmaf(half_at<C::ACT16>(r.kb[u], i * C::NG + g), w.qsum[g], z[u][i]);
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) z[u][i] *= w.zscale;
  }
  if (edge) {  // uniform
#pragma unroll
    for (int u = 0; u < 2; ++u)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!(live >> (4 * u + i) & 1u)) z[u][i] = -__builtin_inff();
  }
  float vs[2][4][C::NG], vmax = 0.f;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int g = 0; g < C::NG; ++g) {
        float v = half_at<C::ACT16>(r.vs[u], i * C::NG + g);
        if (edge && !(live >> (4 * u + i) & 1u)) v = 0.f;
        vs[u][i][g] = v;
        vmax = fmaxf(vmax, fabsf(v));
      }
  float zmax = fmaxf(fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[0][2], z[0][3])),
                     fmaxf(fmaxf(z[1][0], z[1][1]), fmaxf(z[1][2], z[1][3])));
  if (__builtin_amdgcn_ballot_w64(zmax > w.mlim || vmax > w.vlim)) {  // uniform: new references
    const float m = fmaxf(w.mref, quads_max(zmax));
    // the exponent of the largest scale, kept where 2^(5 - mu) and its sums stay finite
    const float vm = quads_max(vmax);
    const float e = fmaxf(w.vexp, fminf(fmaxf((float)((int)(__float_as_uint(vm) >> 23) - 127), -90.f), 110.f));
    const float mu = (m == -__builtin_inff() ? 0.f : m) + e;
    const float alpha = w.mref == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(w.mu - mu);
    w.mref = m;
    w.mu = mu;
    w.mlim = m + MROOM;
    w.vexp = e;
    w.vlim = __builtin_amdgcn_ldexpf(VROOM, (int)e);
    w.l *= alpha;
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
      w.bias[g] *= alpha;
#pragma unroll
      for (int c = 0; c < C::VC; ++c) w.o[g][c] *= alpha;
    }
  }
  const float off = PBIAS - w.mu;
#pragma unroll
  for (int u = 0; u < 2; ++u)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[u][i] = __builtin_amdgcn_exp2f(z[u][i] + off);
      w.l += p[u][i];
#pragma unroll
      for (int g = 0; g < C::NG; ++g) {
        float b = half_at<C::ACT16>(r.vb[u], i * C::NG + g);
        if (edge && !(live >> (4 * u + i) & 1u)) b = 0.f;
        w.bias[g] = fmaf(p[u][i], b, w.bias[g]);
      }
    }
#pragma unroll
  for (int g = 0; g < C::NG; ++g) {
    uint32_t aw[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = k >> 1, i = 2 * (k & 1);
      typedef _Float16 h2 __attribute__((ext_vector_type(2)));
      const h2 h = {(_Float16)(p[u][i] * vs[u][i][g]), (_Float16)(p[u][i + 1] * vs[u][i + 1][g])};
      aw[k] = __builtin_bit_cast(uint32_t, h);
    }
    const f16x8_t A = as_f16x8(aw[0], aw[1], aw[2], aw[3]);
    constexpr int PIECES = C::VBITS <= 16 ? 1 : C::VBITS / 16;
    uint32_t pr[PIECES][4];  // [piece][pair of tokens]
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int u = k >> 1, i = 2 * (k & 1);
      const uint32_t* x = r.vc[u][i][g];
      const uint32_t* y = r.vc[u][i + 1][g];
#pragma unroll
      for (int b = 0; b < PIECES; ++b) {
        if constexpr (C::VBITS <= 16)
          pr[b][k] = x[0] | y[0] << 16;
        else
          pr[b][k] = (b & 1) ? __builtin_amdgcn_perm(y[b / 2], x[b / 2], 0x07060302u)
                             : __builtin_amdgcn_perm(y[b / 2], x[b / 2], 0x05040100u);
      }
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

__device__ __forceinline__ int span_of(const PagedAttnArgs& a, int b, int& first, int& len) {
  len = (int)max(0l, min((long)a.seq_lens[b], (long)a.max_pages * a.c.page_size));
  first = a.window > 0 ? (int)max(0l, (long)len - a.window) : 0;
  return len - (first & ~15);
}

// inclusive sum over the 64 lanes
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int t = __shfl_up(v, o);
    if (lane >= o) v += t;
  }
  return v;
}

struct Place {  // a workgroup's chunk
  int b, c, n, slot0;
};

// Finds chunk `x` of the batch: sequence b is cut into n_b chunks of
// max(1, ceil(span / chunk)), chunk sized so that about `target` units cover
// everything.  False when there is no such chunk.
__device__ __forceinline__ bool find_chunk(const AttnWork& w, int x, int units_per_chunk, Place* out, int* sh) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, B = (int)w.a.B;
  int first, len, span0 = 0;
  long total = 0;
  for (int b0 = 0; b0 < B; b0 += 256) {
    const int s = b0 + t < B ? span_of(w.a, b0 + t, first, len) : 0;
    if (b0 == 0) span0 = s;
    total += s;
  }
  long* lsh = reinterpret_cast<long*>(sh);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) total += __shfl_xor(total, o);
  if (lane == 0) lsh[wave] = total;
  __syncthreads();
  total = (lsh[0] + lsh[1]) + (lsh[2] + lsh[3]);
  __syncthreads();
  const long want = (total * units_per_chunk + w.target - 1) / w.target;
  const int chunk = (int)min(max((want + 127) & ~127l, (long)w.min_chunk), (long)(1 << 30));
  int base = 0, sbase = 0;
  if (t == 0) sh[12] = 0;
  for (int b0 = 0; b0 < B; b0 += 256) {
    const bool in = b0 + t < B;
    const int s = b0 == 0 ? span0 : (in ? span_of(w.a, b0 + t, first, len) : 0);
    const int n = in ? max(1, (int)(((long)s + chunk - 1) / chunk)) : 0, m = n > 1 ? n : 0;
    const int in_n = wave_scan(n, lane), in_m = wave_scan(m, lane);
    __syncthreads();
    if (lane == 63) {
      sh[wave] = in_n;
      sh[4 + wave] = in_m;
    }
    __syncthreads();
    int pn = base, pm = sbase;
    for (int k = 0; k < wave; ++k) {
      pn += sh[k];
      pm += sh[4 + k];
    }
    base += (sh[0] + sh[1]) + (sh[2] + sh[3]);
    sbase += (sh[4] + sh[5]) + (sh[6] + sh[7]);
    const int at = x - (pn + in_n - n);
    if (in && at >= 0 && at < n) {
      sh[8] = b0 + t;
      sh[9] = at;
      sh[10] = n;
      sh[11] = pm + in_m - m;
      sh[12] = 1;
    }
    if (base > x) break;
  }
  __syncthreads();
  out->b = sh[8];
  out->c = sh[9];
  out->n = sh[10];
  out->slot0 = sh[11];
  return sh[12] != 0;
}

template <class C>
__global__ __launch_bounds__(256) void paged_attn_kernel(AttnWork wk) {
  const PagedAttnArgs& a = wk.a;
  const KvCache& c = a.c;
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int n16 = lane & 15, kq = lane >> 4;
  extern __shared__ float lds[];  // [WAVES][gm][D + 4]
  __shared__ __align__(8) int sh[16];
  __shared__ float msh[WAVES][16], lsh[WAVES][16];
  const int units_per_chunk = c.kv_heads * wk.htiles;
  const int x = (int)blockIdx.x / units_per_chunk, rest = (int)blockIdx.x - x * units_per_chunk;
  const int j = rest / wk.htiles, ht = rest - j * wk.htiles;
  Place pl;
  if (!find_chunk(wk, x, units_per_chunk, &pl, sh)) return;
  const int b = __builtin_amdgcn_readfirstlane(pl.b), ci = __builtin_amdgcn_readfirstlane(pl.c),
            nchunks = __builtin_amdgcn_readfirstlane(pl.n);
  if (wk.meta && ci == 0 && rest == 0 && t == 0) wk.meta[b] = make_int2(nchunks, pl.slot0);
  int first, len;
  const int span = span_of(a, b, first, len);
  first = __builtin_amdgcn_readfirstlane(first);
  len = __builtin_amdgcn_readfirstlane(len);
  const int csize = (((span + nchunks - 1) / nchunks) + 127) & ~127;
  const int begin = __builtin_amdgcn_readfirstlane((first & ~15) + ci * csize);
  const int end = __builtin_amdgcn_readfirstlane(min(begin + csize, len));
  const int h0 = j * wk.share + 16 * ht, gm = min(16, wk.share - 16 * ht);  // this tile's heads

  Wave<C> w;
  // q: lane (head n16, quarter kq) holds columns [kq G/4, (kq+1) G/4) of each group
  {
    float qv[C::NG][C::G / 4], mx = 0.f;
    const uint16_t* q = (const uint16_t*)a.q + (long)b * a.qts + (long)(h0 + n16) * a.qhs;
    const bool have = n16 < gm;
#pragma unroll
    for (int g = 0; g < C::NG; ++g)
#pragma unroll
      for (int e = 0; e < C::G / 32; ++e) {
        uint32_t raw[4] = {0u, 0u, 0u, 0u};
        if (have) load_bytes<16>((const uint8_t*)(q + g * C::G + kq * (C::G / 4) + 8 * e), raw);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float v = half_at<C::ACT16>(raw, k);
          qv[g][8 * e + k] = v;
          mx = fmaxf(mx, fabsf(v));
        }
      }
    mx = quads_max(mx);
    // the largest entry to [2^14, 2^15)
    int e = 0;
    if (mx > 0.f && mx < __builtin_inff()) e = 14 - __builtin_amdgcn_frexp_expf(mx) + 1;
#pragma unroll
    for (int g = 0; g < C::NG; ++g) {
      float sum = 0.f;
#pragma unroll
      for (int s = 0; s < C::KS; ++s) {
        uint32_t reg[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float lo = __builtin_amdgcn_ldexpf(qv[g][key_dim<C>(s, r, 0)], e);
          const float hi = __builtin_amdgcn_ldexpf(qv[g][key_dim<C>(s, r, 1)], e);
          const float f = 1.f / (float)(1 << key_shift<C>(r));
          reg[r] = (uint32_t)f32_to_f16_bits(lo * f) | (uint32_t)f32_to_f16_bits(hi * f) << 16;
          sum += lo + hi;
        }
        w.q[g][s] = as_f16x8(reg[0], reg[1], reg[2], reg[3]);
      }
      w.qsum[g] = quads_sum(sum) * 0x1p-24f;
    }
    w.zscale = __builtin_amdgcn_ldexpf(a.scale * 1.4426950408889634f, 24 - e);
  }
#pragma unroll
  for (int g = 0; g < C::NG; ++g) {
    w.bias[g] = 0.f;
#pragma unroll
    for (int v = 0; v < C::VC; ++v) w.o[g][v] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  }
  w.l = 0.f;
  w.mref = w.mlim = -__builtin_inff();
  w.mu = 0.f;
  w.vexp = -90.f;
  w.vlim = 0.f;

  // this wave's steps: tokens begin + 32 (wave + 4 i)
  const int t0 = begin + 32 * wave;
  const int steps = t0 < end ? (end - t0 + 127) >> 7 : 0;
  if (steps > 0) {
    const uint32_t kvo = (uint32_t)(n16 * C::ROWB + kq * C::KB);
    const uint32_t vvo = (uint32_t)(4 * kq * C::ROWB + n16 * C::VBITS / 8);
    const uint32_t svo = (uint32_t)(4 * kq * 2 * C::NG);
    const int32_t* table = a.table + (long)b * a.table_stride;
    int ids = -1, ids_from = -32;  // lane k: the page of 16-token tile k of 32 steps; -1: none
    auto load = [&](Raw<C>& r, int i, uint32_t& live) {
      if (i >= ids_from + 32) {  // uniform
        ids_from = i;
        const int tok = t0 + 128 * (i + (lane >> 1)) + 16 * (lane & 1);
        ids = -1;
        if (tok < end) {
          ids = table[wk.page.div((uint32_t)tok)];
          if ((uint32_t)ids >= (uint32_t)c.num_pages) ids = -1;
        }
      }
      live = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int tok = t0 + 128 * i + 16 * u;
        const int id = __builtin_amdgcn_readlane(ids, 2 * (i - ids_from) + u);
        const uint32_t off = id < 0 ? 0u : (uint32_t)tok - wk.page.div((uint32_t)tok) * wk.page.d;
        const size_t row = ((size_t)(id < 0 ? 0 : id) * c.kv_heads + j) * c.page_size + off;
        load_raw<C>(r, u, c, row, kvo, vvo, svo);
        if (id >= 0) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int tk = tok + 4 * kq + k;
            if (tk >= first && tk < end) live |= 1u << (4 * u + k);
          }
        }
      }
    };
    Raw<C> r0, r1;
    uint32_t live0, live1;
    load(r0, 0, live0);
    for (int i = 0;;) {
      load(r1, i + 1, live1);
      step<C>(w, r0, __builtin_amdgcn_ballot_w64(live0 != 0xffu) != 0, live0, lane);
      if (++i == steps) break;
      load(r0, i + 1, live0);
      step<C>(w, r1, __builtin_amdgcn_ballot_w64(live1 != 0xffu) != 0, live1, lane);
      if (++i == steps) break;
    }
  }
  // join the waves
  w.l = quads_sum(w.l);
  const float m_own = (w.mref == -__builtin_inff() && w.l == w.l) ? -__builtin_inff() : w.mu;
  if (kq == 0) {
    msh[wave][n16] = m_own;
    lsh[wave][n16] = w.l;
  }
  const int stride = C::D + 4;
#pragma unroll
  for (int g = 0; g < C::NG; ++g) {
    const float bs = quads_sum(w.bias[g]);
    if (n16 < gm) {
      float* dst = lds + (wave * gm + n16) * stride + g * C::G + 4 * kq * C::VC;
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int v = 0; v < C::VC; ++v)
          dst[i * C::VC + v] = fmaf(w.o[g][v][i], 0x1p24f / (float)(1 << value_shift<C>(v)), bs);
    }
  }
  __syncthreads();
  const bool whole = nchunks == 1;
  const size_t slot = ((size_t)(pl.slot0 + ci) * c.kv_heads + j) * wk.htiles + ht;
  const int gstore = min(16, wk.share);
  for (int i = t; i < gm * (C::D / 4); i += 256) {
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

// Joins the chunks of one sequence and head: 32 lanes by eight groups of chunks.
template <bool F16_>
__global__ __launch_bounds__(256) void paged_attn_join_kernel(AttnWork wk) {
  const PagedAttnArgs& a = wk.a;
  const int b = blockIdx.y, head = blockIdx.x, t = threadIdx.x, D = a.c.head_dim;
  const int2 mt = wk.meta[b];
  if (mt.x <= 1) return;
  const int j = head / wk.share, ht = (head - j * wk.share) / 16, h = head - j * wk.share - 16 * ht;
  const int gstore = min(16, wk.share);
  __shared__ float msh[4], osh[8][256 + 4], lsh[8];
  auto at = [&](int k) { return ((((size_t)(mt.y + k) * a.c.kv_heads + j) * wk.htiles + ht) * gstore + h); };
  float m = -__builtin_inff();
  for (int k = t; k < mt.x; k += 256) m = fmaxf(m, wk.part_ml[2 * at(k)]);
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor(m, o));
  if ((t & 63) == 0) msh[t >> 6] = m;
  __syncthreads();
  m = fmaxf(fmaxf(msh[0], msh[1]), fmaxf(msh[2], msh[3]));
  const int grp = t >> 5, ln = t & 31;
  f32x4_t o[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
  float l = 0.f;
  for (int k = grp; k < mt.x; k += 8) {
    const size_t s = at(k);
    const float mk = wk.part_ml[2 * s];
    const float f = mk == -__builtin_inff() ? 0.f : __builtin_amdgcn_exp2f(mk - m);
    l = fmaf(f, wk.part_ml[2 * s + 1], l);
#pragma unroll
    for (int e = 0; e < 2; ++e)
      if (4 * ln + 128 * e < D) {
        const f32x4_t v = *reinterpret_cast<const f32x4_t*>(wk.part_o + s * D + 4 * ln + 128 * e);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[e][i] = fmaf(f, v[i], o[e][i]);
      }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) *reinterpret_cast<f32x4_t*>(&osh[grp][4 * ln + 128 * e]) = o[e];
  if (ln == 0) lsh[grp] = l;
  __syncthreads();
  if (t < D) {
    float s = 0.f, ls = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      s += osh[k][t];
      ls += lsh[k];
    }
    ((uint16_t*)a.out)[((size_t)b * a.heads + head) * D + t] = f32_to_act_bits(ls == 0.f ? 0.f : s / ls, F16_);
  }
}

template <class C>
hipError_t launch_cfg(AttnWork& w, hipStream_t s) {
  const PagedAttnArgs& a = w.a;
  const void* fn = reinterpret_cast<const void*>(&paged_attn_kernel<C>);
  const int gm = w.share < 16 ? w.share : 16;
  const size_t lds = (size_t)WAVES * gm * (C::D + 4) * 4;
  int64_t resident = 0;
  hipError_t e = resident_workgroups(fn, 256, lds, 8, &resident);
  if (e != hipSuccess) return e;
  const int64_t units = (int64_t)a.c.kv_heads * w.htiles;
  w.target = (int)resident;
  w.min_chunk = 128;
  const int64_t grid = w.target + units * a.B;
  if (grid >= (int64_t(1) << 31)) return hipErrorNotSupported;
  const bool split = (int64_t)a.max_pages * a.c.page_size > w.min_chunk;
  w.part_o = w.part_ml = nullptr;
  w.meta = nullptr;
  if (split) {
    // a sequence of more than one chunk has at most 2 span / chunk of them
    const size_t slots = 2 * (size_t)w.target + 2 * units;
    const size_t meta = ((size_t)a.B * sizeof(int2) + 255) & ~size_t(255);
    const size_t ml = (slots * gm * 2 * sizeof(float) + 255) & ~size_t(255);
    void* p = nullptr;
    e = stream_workspace(s, meta + ml + slots * gm * C::D * sizeof(float), &p);
    if (e != hipSuccess) return e;
    w.meta = static_cast<int2*>(p);
    w.part_ml = reinterpret_cast<float*>(static_cast<char*>(p) + meta);
    w.part_o = reinterpret_cast<float*>(static_cast<char*>(p) + meta + ml);
  }
  hipLaunchKernelGGL(paged_attn_kernel<C>, dim3((unsigned)grid), dim3(256), lds, s, w);
  e = hipGetLastError();
  if (e == hipSuccess && split) {
    hipLaunchKernelGGL(paged_attn_join_kernel<C::ACT16>, dim3((unsigned)a.heads, (unsigned)a.B), dim3(256), 0, s, w);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

template <int BITS>
hipError_t launch_paged_attention_bits(const PagedAttnArgs& a, hipStream_t s) {
  AttnWork w{a, FastDiv((uint32_t)a.c.page_size)};
  w.share = a.heads / a.c.kv_heads;
  w.htiles = (w.share + 15) / 16;
#define QAFF_ATTN(D, G)                                                            \
  case D * 1000 + G:                                                               \
    return a.c.dt == F16 ? launch_cfg<Cfg<D, G, BITS, true>>(w, s) : launch_cfg<Cfg<D, G, BITS, false>>(w, s);
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
