// Attention of one new token a sequence over the paged affine cache.
//     z[t] = scale * sum_d q[d] k[t,d],  t in [max(0, len - window), len)
//     p = softmax(z),  o[d] = sum_t p[t] v[t,d]
// with k and v = code*scale + bias as kv_cache_append_affine stored them; the
// heads of a group of heads/kv_heads share one key head.  A row that sees no
// token gives zeros.
//
// One workgroup per sequence and query head: 256 tokens a step, a thread per
// token for the logits, a thread per column for the values.
#include "common.h"

namespace qaff {
namespace {

__global__ __launch_bounds__(256) void paged_attn_kernel(PagedAttnArgs a) {
  const KvCache& c = a.c;
  const int b = blockIdx.y, head = blockIdx.x, t = threadIdx.x, D = c.head_dim;
  const int kvh = head / (a.heads / c.kv_heads), W = D * c.bits / 32, NG = D / c.G;
  const bool f16 = c.dt == F16;
  __shared__ float qs[256], ps[256], red[4];
  __shared__ long rows[256];
  if (t < D) qs[t] = load_as_f32((const uint16_t*)a.q + (long)b * a.qts + (long)head * a.qhs, t, c.dt);
  const int len = (int)min((long)a.seq_lens[b], (long)a.max_pages * c.page_size);
  const int first = a.window > 0 ? (int)max(0l, (long)len - a.window) : 0;
  const uint32_t mask = (1u << c.bits) - 1u;
  auto value = [&](const uint32_t* w, const uint16_t* s, const uint16_t* bi, long row, int d) {
    const int per = 32 / c.bits;
    const uint32_t code = (w[row * W + d / per] >> (c.bits * (d % per))) & mask;
    return __fmaf_rn((float)code, load_as_f32(s, row * NG + d / c.G, c.dt), load_as_f32(bi, row * NG + d / c.G, c.dt));
  };
  float m = -__builtin_inff(), l = 0.f, o = 0.f;
  for (int t0 = first; t0 < len; t0 += 256) {
    __syncthreads();
    const int tok = t0 + t;
    float z = -__builtin_inff();
    rows[t] = -1;
    if (tok < len) {
      const int page = a.table[(long)b * a.table_stride + tok / c.page_size];
      if (page >= 0 && page < c.num_pages) {
        const long row = ((long)page * c.kv_heads + kvh) * c.page_size + tok % c.page_size;
        rows[t] = row;
        float acc = 0.f;
        for (int d = 0; d < D; ++d) acc = fmaf(qs[d], value(c.k_packed, c.k_scales, c.k_biases, row, d), acc);
        z = acc * a.scale;
      }
    }
    float mx = z;
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) mx = fmaxf(mx, __shfl_xor(mx, k));
    if ((t & 63) == 0) red[t >> 6] = mx;
    __syncthreads();
    mx = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float p = rows[t] >= 0 ? expf(z - mx) : 0.f;
    ps[t] = p;
    float sum = p;
#pragma unroll
    for (int k = 32; k >= 1; k >>= 1) sum += __shfl_xor(sum, k);
    __syncthreads();
    if ((t & 63) == 0) red[t >> 6] = sum;
    __syncthreads();
    const float alpha = m == mx ? 1.f : expf(m - mx);
    l = l * alpha + ((red[0] + red[1]) + (red[2] + red[3]));
    m = mx;
    o *= alpha;
    if (t < D)
      for (int i = 0; i < min(256, len - t0); ++i)
        if (rows[i] >= 0) o = fmaf(ps[i], value(c.v_packed, c.v_scales, c.v_biases, rows[i], t), o);
  }
  if (t < D) ((uint16_t*)a.out)[((long)b * a.heads + head) * D + t] = f32_to_act_bits(l > 0.f ? o / l : (l == 0.f ? 0.f : l), f16);
}

}  // namespace

hipError_t launch_paged_attention(const PagedAttnArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(paged_attn_kernel, dim3((unsigned)a.heads, (unsigned)a.B), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace qaff
