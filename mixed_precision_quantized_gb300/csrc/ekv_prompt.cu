// ekv_prompt.cu — causal attention over whole prompts, packed end to end.
//
// For token i of a sequence and query head h with KV head g = h / (Hq / Hkv):
//   o_ih = sum_{j <= i} softmax_j(sigma q_ih . k_jg) v_jg
// One warp per (token, query head): lanes hold 1/32 of the head's channels, keys
// are taken one at a time with a running maximum and sum.
#include <math_constants.h>

#include "ekv_internal.h"

namespace ekv {
namespace {

template <int D>
__global__ void __launch_bounds__(128)
prompt_kernel(int Hq, int Hkv, float scale_log2, int total, int n_seqs,
              const int32_t* __restrict__ cu, const __half* __restrict__ q, int64_t qs,
              const __half* __restrict__ k, int64_t ks, const __half* __restrict__ v, int64_t vs,
              __half* __restrict__ o, int64_t os) {
  constexpr int C = D / 32;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int i = (int)(row / Hq), h = (int)(row % Hq), g = h / (Hq / Hkv);
  if (i >= total) return;
  int start = -1;
  for (int z = 0; z < n_seqs; ++z) {
    const int a = cu[z], b = cu[z + 1];
    if (a >= 0 && b <= total && i >= a && i < b) start = a;
  }
  if (start < 0) return;  // behind the last sequence
  float qf[C], acc[C], m = -CUDART_INF_F, l = 0.f;
  for (int c = 0; c < C; ++c) {
    qf[c] = __half2float(q[i * qs + h * D + lane * C + c]) * scale_log2;
    acc[c] = 0.f;
  }
  for (int j = start; j <= i; ++j) {
    float x = 0.f;
    for (int c = 0; c < C; ++c) x = fmaf(qf[c], __half2float(k[j * ks + g * D + lane * C + c]), x);
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    const float mn = fmaxf(m, x), al = exp2f(m - mn), p = exp2f(x - mn);
    l = l * al + p;
    for (int c = 0; c < C; ++c)
      acc[c] = fmaf(p, __half2float(v[j * vs + g * D + lane * C + c]), acc[c] * al);
    m = mn;
  }
  for (int c = 0; c < C; ++c) o[i * os + h * D + lane * C + c] = __float2half_rn(acc[c] / l);
}

}  // namespace
}  // namespace ekv

extern "C" EKV_API int ekv_prompt_attn(int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                       float softmax_scale, int32_t total_tokens, int32_t n_seqs,
                                       const int32_t* cu_seqlens, const void* q, int64_t q_stride,
                                       const void* k, int64_t k_stride, const void* v,
                                       int64_t v_stride, void* o, int64_t o_stride, void* stream) {
  using namespace ekv;
  if (n_q_heads <= 0 || n_kv_heads <= 0 || n_q_heads % n_kv_heads || n_q_heads > 4096 ||
      total_tokens < 0 || n_seqs < 0 || !(softmax_scale >= 0.f) || softmax_scale > 3.0e38f)
    return EKV_EINVAL;
  if (head_dim != 64 && head_dim != 128) return EKV_EUNSUPPORTED;
  if (total_tokens == 0 || n_seqs == 0) return EKV_OK;
  if (!cu_seqlens || !q || !k || !v || !o) return EKV_EINVAL;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)o) & 15) return EKV_EINVAL;
  if ((uintptr_t)cu_seqlens & 3) return EKV_EINVAL;
  const int64_t rq = (int64_t)n_q_heads * head_dim, rk = (int64_t)n_kv_heads * head_dim;
  if (q_stride < rq || o_stride < rq || k_stride < rk || v_stride < rk ||
      ((q_stride | o_stride | k_stride | v_stride) & 7))
    return EKV_EINVAL;
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)head_dim);
  const float sl = scale * 1.4426950408889634f;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const unsigned grid = (unsigned)(((int64_t)total_tokens * n_q_heads + 3) / 4);
  auto fn = head_dim == 64 ? prompt_kernel<64> : prompt_kernel<128>;
  fn<<<grid, 128, 0, s>>>(n_q_heads, n_kv_heads, sl, total_tokens, n_seqs, cu_seqlens,
                          static_cast<const __half*>(q), q_stride, static_cast<const __half*>(k),
                          k_stride, static_cast<const __half*>(v), v_stride,
                          static_cast<__half*>(o), o_stride);
  return cudaGetLastError() == cudaSuccess ? EKV_OK : EKV_ECUDA;
}
