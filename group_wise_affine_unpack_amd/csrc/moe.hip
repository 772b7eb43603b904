// Mixture-of-experts block: the launches, and the kernel that adds a token's
// experts up (moe.h has the products).
#include "common.h"

namespace qaff {

hipError_t launch_moe_b2(const MoeArgs& a, bool down, hipStream_t s);
hipError_t launch_moe_b4(const MoeArgs& a, bool down, hipStream_t s);
hipError_t launch_moe_b8(const MoeArgs& a, bool down, hipStream_t s);

namespace {

hipError_t launch_moe_product(const MoeArgs& a, bool down, hipStream_t s) {
  return a.bits == 2 ? launch_moe_b2(a, down, s) : a.bits == 4 ? launch_moe_b4(a, down, s) : launch_moe_b8(a, down, s);
}

// y = resid + scale / sum * (sum over a token's choices, in their order, of
// weight * part), four columns a thread.  The sum of the weights: over the
// choices, or over all experts (softmax before the choice).  A NaN among the
// logits makes the row NaN.
__global__ __launch_bounds__(256) void moe_join_kernel(MoeArgs a) {
  const int m = blockIdx.y, lane = threadIdx.x & 63;
  float top = -__builtin_inff();
  int finite = 0;
  bool nan = false;
  for (int i = 0; i < a.E; i += 64) {
    const float z = i + lane < a.E ? load_as_f32(a.logits, (long)m * a.E + i + lane, a.logit_dt) : -__builtin_inff();
    nan |= z != z;
    finite += __builtin_popcountll(__ballot(z > -__builtin_inff()));
    top = fmaxf(top, z);
  }
  nan = __ballot(nan) != 0;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) top = fmaxf(top, __shfl_xor(top, d));
  const int choices = min(finite, a.top_k);
  float sum = 0.f;
  if (a.renormalize) {
    for (int r = 0; r < choices; ++r) sum += a.weights[m * a.top_k + r];
  } else {
    for (int i = 0; i < a.E; i += 64)
      if (i + lane < a.E) {
        const float z = load_as_f32(a.logits, (long)m * a.E + i + lane, a.logit_dt);
        sum += z > -__builtin_inff() ? expf(z - top) : 0.f;
      }
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) sum += __shfl_xor(sum, d);
  }
  const int n = (blockIdx.x * 256 + threadIdx.x) * 4;
  if (n >= a.N) return;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
  for (int r = 0; r < choices; ++r) {
    const int pair = m * a.top_k + r;
    const float w = a.weights[pair];
    const f32x4_t p = *reinterpret_cast<const f32x4_t*>(a.part + (long)pair * a.N + n);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fmaf(w, p[i], v[i]);
  }
  const float f = choices ? a.scale / sum : 0.f;
  const bool f16 = a.act_dt == F16;
  u32x2_t o;
  uint32_t e[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float r = a.resid ? load_as_f32(a.resid, (long)m * a.N + n + i, a.act_dt) : 0.f;
    float y = choices ? fmaf(f, v[i], r) : r;
    if (nan) y = __builtin_nanf("");
    e[i] = f32_to_act_bits(y, f16);
  }
  o[0] = e[0] | e[1] << 16;
  o[1] = e[2] | e[3] << 16;
  *reinterpret_cast<u32x2_t*>((uint16_t*)a.y + (long)m * a.N + n) = o;
}

}  // namespace

hipError_t launch_moe(MoeArgs& a, hipStream_t s) {
  // scratch: the slots' counts and lists, the pairs' weights, rows h and partial rows
  const size_t pairs = (size_t)a.M * a.top_k, slots = pairs < (size_t)a.E ? pairs : (size_t)a.E;
  const auto up = [](size_t n) { return (n + 255) & ~size_t(255); };
  const size_t counts = up(8 * slots), lists = up(4 * slots * a.M), weights = up(4 * pairs), h = up(4 * pairs * a.I);
  void* p = nullptr;
  hipError_t e = stream_workspace(s, counts + lists + weights + h + 4 * pairs * a.N, &p);
  if (e != hipSuccess) return e;
  char* q = static_cast<char*>(p);
  a.counts = reinterpret_cast<int*>(q);
  a.lists = reinterpret_cast<int*>(q + counts);
  a.weights = reinterpret_cast<float*>(q + counts + lists);
  a.h = reinterpret_cast<float*>(q + counts + lists + weights);
  a.part = reinterpret_cast<float*>(q + counts + lists + weights + h);
  e = launch_moe_product(a, false, s);
  if (e != hipSuccess) return e;
  e = launch_moe_product(a, true, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(moe_join_kernel, dim3((unsigned)((a.N + 1023) / 1024), (unsigned)a.M), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qaff
