// Root-mean-square norm over rows, with the residual's addition ahead of it,
// into the activation type or into the int8 codes of W4A8.
//     h[m,k] = x[m,k] + r[m,k], rounded once to the activation type (or x)
//     n[m,k] = (h[m,k] * rstd[m]) * w[k],  rstd = 1 / sqrt(mean_k h^2 + eps)
//     dense:  y = n rounded once
//     codes:  s_x = max_k |n| / 127 (IEEE division),
//             x_q = clamp(rint(n / s_x), -127, 127), zeros when s_x == 0
//             (a NaN among the n makes s_x NaN, so that products with it are)
// The norm reads h as stored, so the residual stream and the norm agree.
// The squares are taken and summed in fp64 (each is exact there, and none
// overflows) and rstd is rounded once to fp32.  The sum's order moves it by
// K 2^-53 of itself at most, so two orders round to the same rstd, and so to
// the same outputs, but for a rstd within 2^-15 of a step (K = 16384) from a
// rounding boundary, one row in 16384 at worst and far fewer in practice.
// Every other step is one IEEE fp32 operation.
#include <algorithm>

#include "common.h"

namespace qaff {
namespace {

template <bool F16_>
__device__ __forceinline__ float half_of(uint32_t w, int h) {
  if constexpr (F16_) return f16_bits_to_f32(h ? w >> 16 : w & 0xffffu);
  else return __uint_as_float(h ? w & 0xffff0000u : w << 16);
}

// (mean square + eps)^-1/2 in fp64, rounded once; with codes 0 for a row of zeros, whose n are zeros then without an eps too
template <bool CODES>
__device__ __forceinline__ float rstd_of(double sum, const NormArgs& a) {
  return CODES && sum == 0.0 ? 0.f : (float)(1.0 / sqrt(sum / (double)a.K + a.eps));
}

// h rstd w, each product rounded to fp32.  (The barrier keeps the second one
// from being folded into a rounding to f16, one v_fma_mix: dense outputs would
// then depend on the compiler.)
__device__ __forceinline__ float n_value(float h, float rstd, float w) {
  float n = __fmul_rn(__fmul_rn(h, rstd), w);
  asm("" : "+v"(n));
  return n;
}

// x_q = clamp(rint(n / s), -127, 127), 0 when s == 0, the division IEEE
__device__ __forceinline__ float code_of(float n, float s) {
  return s != 0.f ? fminf(fmaxf(rintf(__fdiv_rn(n, s)), -127.f), 127.f) : 0.f;
}
// The same for eight values, r = 1/s: n r corrected by its residual is within
// a few units of the last place (2^-17) of the quotient, so its whole number
// is the quotient's unless it lies next to a half, and then all eight take
// the division (2048 x 4096: 17.5 -> 16.2 us).
__device__ __forceinline__ void codes_of(const float (&n)[8], float s, float r, float (&q)[8]) {
  float next = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float q0 = __fmul_rn(n[j], r), q1 = __fmaf_rn(__fmaf_rn(-s, q0, n[j]), r, q0);
    q[j] = rintf(q1);
    next = fmaxf(next, fabsf(q1 - q[j]));
  }
  if (!(next < 0.4999f && s >= 0x1p-90f && s <= 0x1p90f)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = code_of(n[j], s);
  }
}

// A row per WPR waves (WAVES / WPR rows a workgroup), held in registers:
// thread i of the row takes the 8-value chunks i, i + 64 WPR, ... (CPT of
// them, K <= 512 WPR CPT).  16-byte aligned rows, K % 8 == 0.  Every load of
// the row, residual and weight is in flight before the first sum.
template <bool F16_, bool CODES, bool W32, int WAVES, int WPR, int CPT>
__global__ __launch_bounds__(64 * WAVES) void rmsnorm_rows_kernel(NormArgs a) {
  const int t = threadIdx.x, wave = t >> 6, sub = wave % WPR;
  const long m = (long)blockIdx.x * (WAVES / WPR) + wave / WPR;
  const int K8 = (int)(a.K >> 3), c0 = sub * 64 + (t & 63);
  __shared__ double sums[WAVES];
  __shared__ float maxs[WAVES];
  const bool in_row = WPR == WAVES || m < a.M;  // (a wave past the last row runs along for the barriers)
  const u32x4_t* x = (const u32x4_t*)((const uint16_t*)a.x + m * a.ldx);
  const u32x4_t* r = (const u32x4_t*)((const uint16_t*)a.resid + m * a.ldr);
  u32x4_t h[CPT], rr[CPT], w[CPT][W32 ? 2 : 1];
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = c0 + 64 * WPR * i;
    h[i] = u32x4_t{0u, 0u, 0u, 0u};
    if (in_row && c < K8) {
      h[i] = x[c];
      if (a.resid) rr[i] = r[c];
    }
  }
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = c0 + 64 * WPR * i;
    if (in_row && c < K8) {
      if constexpr (W32) {
        w[i][0] = ((const u32x4_t*)a.w)[2 * c];
        w[i][1] = ((const u32x4_t*)a.w)[2 * c + 1];
      } else {
        w[i][0] = ((const u32x4_t*)a.w)[c];
      }
    }
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = c0 + 64 * WPR * i;
    if (in_row && c < K8 && a.resid) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float lo = __fadd_rn(half_of<F16_>(h[i][j], 0), half_of<F16_>(rr[i][j], 0));
        const float hi = __fadd_rn(half_of<F16_>(h[i][j], 1), half_of<F16_>(rr[i][j], 1));
        h[i][j] = (uint32_t)f32_to_act_bits(lo, F16_) | (uint32_t)f32_to_act_bits(hi, F16_) << 16;
      }
      ((u32x4_t*)((uint16_t*)a.h_out + m * a.ldh))[c] = h[i];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double v = (double)half_of<F16_>(h[i][j / 2], j & 1);
      sum = fma(v, v, sum);
    }
  }
  sum = wave_sum_f64(sum);
  if constexpr (WPR > 1) {
    if ((t & 63) == 0) sums[wave] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int k = 0; k < WPR; ++k) sum += sums[wave - sub + k];
  }
  const float rstd = rstd_of<CODES>(sum, a);
  auto n_of = [&](int i, int j) {
    float wv;
    if constexpr (W32)
      wv = __uint_as_float(w[i][j / 4][j & 3]);
    else
      wv = a.w_dt == F16 ? half_of<true>(w[i][0][j / 2], j & 1) : half_of<false>(w[i][0][j / 2], j & 1);
    return n_value(half_of<F16_>(h[i][j / 2], j & 1), rstd, wv);
  };
  if constexpr (!CODES) {
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = c0 + 64 * WPR * i;
      if (in_row && c < K8) {
        u32x4_t o;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = (uint32_t)f32_to_act_bits(n_of(i, 2 * j), F16_) | (uint32_t)f32_to_act_bits(n_of(i, 2 * j + 1), F16_) << 16;
        ((u32x4_t*)((uint16_t*)a.y + m * a.K))[c] = o;
      }
    }
  } else {
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < CPT; ++i)
      if (in_row && c0 + 64 * WPR * i < K8)
#pragma unroll
        for (int j = 0; j < 8; ++j) mx = nan_max(mx, fabsf(n_of(i, j)));
    mx = wave_max_f32(mx);
    if constexpr (WPR > 1) {
      if ((t & 63) == 0) maxs[wave] = mx;
      __syncthreads();
      mx = 0.f;
#pragma unroll
      for (int k = 0; k < WPR; ++k) mx = nan_max(mx, maxs[wave - sub + k]);
    }
    const float s = __fdiv_rn(mx, 127.f);
    if (in_row && c0 == 0) a.s_x[m] = s;
    const float r = __fdiv_rn(1.f, s);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
      const int c = c0 + 64 * WPR * i;
      if (in_row && c < K8) {
        float n[8], q[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = n_of(i, j);
        codes_of(n, s, r, q);
        u32x2_t o;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t word = 0;  // (each byte holds the code plus 128: no clamp is needed, |n| <= 127 s up to rounding)
#pragma unroll
          for (int e = 0; e < 4; ++e) word = __builtin_amdgcn_cvt_pk_u8_f32(q[4 * j + e] + 128.f, e, word);
          o[j] = word ^ 0x80808080u;
        }
        ((u32x2_t*)(a.x_q + m * a.K))[c] = o;
      }
    }
  }
}

// One workgroup of 256 threads per row, any K and any row start.
template <bool F16_, bool CODES>
__global__ __launch_bounds__(256) void rmsnorm_any_kernel(NormArgs a) {
  const long m = blockIdx.x;
  const int t = threadIdx.x, K = (int)a.K;
  constexpr int DT = F16_ ? F16 : BF16;
  __shared__ double sums[4];
  __shared__ float maxs[4];
  const uint16_t* x = (const uint16_t*)a.x + m * a.ldx;
  const uint16_t* r = a.resid ? (const uint16_t*)a.resid + m * a.ldr : nullptr;
  uint16_t* ho = a.resid ? (uint16_t*)a.h_out + m * a.ldh : nullptr;
  double sum = 0.0;
  for (int k = t; k < K; k += 256) {
    float h = load_as_f32(x, k, DT);
    if (r) {
      const uint16_t b = f32_to_act_bits(__fadd_rn(h, load_as_f32(r, k, DT)), F16_);
      ho[k] = b;
      h = F16_ ? f16_bits_to_f32(b) : bf16_bits_to_f32(b);
    }
    sum = fma((double)h, (double)h, sum);
  }
  sum = wave_sum_f64(sum);
  if ((t & 63) == 0) sums[t >> 6] = sum;
  __syncthreads();
  sum = (sums[0] + sums[1]) + (sums[2] + sums[3]);
  const float rstd = rstd_of<CODES>(sum, a);
  const uint16_t* hs = r ? ho : x;  // each thread reads back what it wrote
  auto n_of = [&](int k) { return n_value(load_as_f32(hs, k, DT), rstd, load_as_f32(a.w, k, a.w_dt)); };
  if constexpr (!CODES) {
    uint16_t* y = (uint16_t*)a.y + m * K;
    for (int k = t; k < K; k += 256) y[k] = f32_to_act_bits(n_of(k), F16_);
  } else {
    float mx = 0.f;
    for (int k = t; k < K; k += 256) mx = nan_max(mx, fabsf(n_of(k)));
    mx = wave_max_f32(mx);
    if ((t & 63) == 0) maxs[t >> 6] = mx;
    __syncthreads();
    mx = nan_max(nan_max(maxs[0], maxs[1]), nan_max(maxs[2], maxs[3]));
    const float s = __fdiv_rn(mx, 127.f);
    if (t == 0) a.s_x[m] = s;
    for (int k = t; k < K; k += 256) a.x_q[m * K + k] = (int8_t)code_of(n_of(k), s);
  }
}

}  // namespace

namespace {

template <bool F16_, bool CODES, bool W32>
void launch_rows(const NormArgs& a, hipStream_t s) {
  const int64_t C = a.K / 8;  // 8-value chunks
  auto go = [&](auto kernel, int waves, int wpr) {
    hipLaunchKernelGGL(kernel, dim3((unsigned)((a.M + waves / wpr - 1) / (waves / wpr))), dim3(64 * waves), 0, s, a);
  };
  if (C <= 64)
    go(rmsnorm_rows_kernel<F16_, CODES, W32, 4, 1, 1>, 4, 1);
  else if (C <= 128)
    go(rmsnorm_rows_kernel<F16_, CODES, W32, 4, 2, 1>, 4, 2);
  else if (C <= 256)
    go(rmsnorm_rows_kernel<F16_, CODES, W32, 4, 4, 1>, 4, 4);
  else if (C <= 512)
    go(rmsnorm_rows_kernel<F16_, CODES, W32, 8, 8, 1>, 8, 8);
  else if (C <= 1024)
    go(rmsnorm_rows_kernel<F16_, CODES, W32, 8, 8, 2>, 8, 8);
  else
    go(rmsnorm_rows_kernel<F16_, CODES, W32, 16, 16, 2>, 16, 16);
}

template <bool F16_, bool CODES>
void launch_dt(const NormArgs& a, hipStream_t s) {
  auto at16 = [](const void* p, int64_t ld) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && ld % 8 == 0; };
  const bool rows = a.K % 8 == 0 && a.K <= 16384 && at16(a.x, a.ldx) && at16(a.w, 0) &&
                    (!a.resid || (at16(a.resid, a.ldr) && at16(a.h_out, a.ldh))) &&
                    (CODES ? (reinterpret_cast<uintptr_t>(a.x_q) & 7) == 0 : at16(a.y, 0));
  if (!rows)
    hipLaunchKernelGGL((rmsnorm_any_kernel<F16_, CODES>), dim3((unsigned)a.M), dim3(256), 0, s, a);
  else if (a.w_dt == F32)
    launch_rows<F16_, CODES, true>(a, s);
  else
    launch_rows<F16_, CODES, false>(a, s);
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& all, hipStream_t s) {
  // 2^21 rows a launch: one has fewer than 2^32 threads, and a row up to 1024 of them
  constexpr int64_t ROWS = int64_t(1) << 21;
  const bool f16 = all.act_dt == F16, codes = all.x_q != nullptr;
  for (int64_t m = 0; m < all.M; m += ROWS) {
    NormArgs a = all;
    a.M = std::min(all.M - m, ROWS);
    a.x = (const uint16_t*)all.x + m * all.ldx;
    if (all.resid) {
      a.resid = (const uint16_t*)all.resid + m * all.ldr;
      a.h_out = (uint16_t*)all.h_out + m * all.ldh;
    }
    if (codes) {
      a.x_q = all.x_q + m * all.K;
      a.s_x = all.s_x + m;
    } else {
      a.y = (uint16_t*)all.y + m * all.K;
    }
    if (f16 && codes)
      launch_dt<true, true>(a, s);
    else if (f16)
      launch_dt<true, false>(a, s);
    else if (codes)
      launch_dt<false, true>(a, s);
    else
      launch_dt<false, false>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace qaff
