// Root-mean-square norm over rows, with the residual's addition ahead of it,
// into the activation type or into the int8 codes of W4A8.
//     h[m,k] = x[m,k] + r[m,k], rounded once to the activation type (or x)
//     n[m,k] = (h[m,k] * rstd[m]) * w[k],  rstd = 1 / sqrt(mean_k h^2 + eps)
//     dense:  y = n rounded once
//     codes:  s_x = max_k |n| / 127 (IEEE division),
//             x_q = clamp(rint(n / s_x), -127, 127), zeros when s_x == 0
// The norm reads h as stored, so the residual stream and the norm agree.
// The squares are taken and summed in fp64 (each is exact there, and none
// overflows) and rstd is rounded once to fp32: the sum's order then leaves rstd's
// bits, and so the codes, unchanged.  Every other step is one IEEE fp32
// operation.
#include "common.h"

namespace qaff {
namespace {

// sum (fp64) or maximum (fp32) over the WPR waves of a row; every lane gets it
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ float wave_max_f32(float v) {
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

__device__ __forceinline__ float q8(float n, float s) {
  return s != 0.f ? fminf(fmaxf(rintf(__fdiv_rn(n, s)), -127.f), 127.f) : 0.f;
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
  const float rstd = (float)(1.0 / sqrt(sum / (double)K + a.eps));
  const uint16_t* hs = r ? ho : x;  // each thread reads back what it wrote
  auto n_of = [&](int k) { return __fmul_rn(__fmul_rn(load_as_f32(hs, k, DT), rstd), load_as_f32(a.w, k, a.w_dt)); };
  if constexpr (!CODES) {
    uint16_t* y = (uint16_t*)a.y + m * K;
    for (int k = t; k < K; k += 256) y[k] = f32_to_act_bits(n_of(k), F16_);
  } else {
    float mx = 0.f;
    for (int k = t; k < K; k += 256) mx = fmaxf(mx, fabsf(n_of(k)));
    mx = wave_max_f32(mx);
    if ((t & 63) == 0) maxs[t >> 6] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(maxs[0], maxs[1]), fmaxf(maxs[2], maxs[3]));
    const float s = __fdiv_rn(mx, 127.f);
    if (t == 0) a.s_x[m] = s;
    for (int k = t; k < K; k += 256) a.x_q[m * K + k] = (int8_t)q8(n_of(k), s);
  }
}

}  // namespace

hipError_t launch_rmsnorm(const NormArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.M), block(256);
  const bool f16 = a.act_dt == F16, codes = a.x_q != nullptr;
  if (f16 && codes)
    hipLaunchKernelGGL((rmsnorm_any_kernel<true, true>), grid, block, 0, s, a);
  else if (f16)
    hipLaunchKernelGGL((rmsnorm_any_kernel<true, false>), grid, block, 0, s, a);
  else if (codes)
    hipLaunchKernelGGL((rmsnorm_any_kernel<false, true>), grid, block, 0, s, a);
  else
    hipLaunchKernelGGL((rmsnorm_any_kernel<false, false>), grid, block, 0, s, a);
  return hipGetLastError();
}

}  // namespace qaff
