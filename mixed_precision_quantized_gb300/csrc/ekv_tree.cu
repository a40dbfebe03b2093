// ekv_tree.cu — attention of a tree of drafted tokens over the quantized paged cache.
//
// Every node i of a sequence's drafted tree (fp16 q, k, v of its own; parent
// parents[i] < i, -1 = none) attends over every cached token of the sequence, read
// from the mixed-format pages and the open block's staging rows as decode attention
// reads them, and over itself and its ancestors among the drafted nodes:
//   o_ih = sum_{t cached} p_t vhat_t + sum_{a in anc(i)} p_a v_a,
//   p = softmax over both of sigma q_ih . khat_t and sigma q_ih . k_a.
// One warp per (node, query head): lanes hold 1/32 of the head's channels, keys are
// taken one at a time with a running maximum and sum.
#include <math_constants.h>

#include "ekv_internal.h"

namespace ekv {
namespace {

// Value of channel c, row r of a quantized part of b bits (raw fp16 at 16).
__device__ float code_at(const uint8_t* part, int d, int b, int r, int c, bool asym) {
  if (b == 16) return __half2float(reinterpret_cast<const __half*>(part)[r * d + c]);
  const int u = (part[r * (d * b / 8) + c * b / 8] >> ((c * b) % 8)) & ((1 << b) - 1);
  return (float)(asym ? u : u - (1 << (b - 1)));
}
// Position of channel c's K scale (pair order of 2- and 4-bit pages).
__device__ int k_scale_pos(int b, int c) {
  if (b >= 8) return c;
  const int n = 32 / b, i = c % n;
  return c - i + (i < n / 2 ? 2 * i : 2 * (i - n / 2) + 1);
}

template <int D>
__global__ void __launch_bounds__(128)
tree_kernel(DevState st, int layer, int vb, int m, const int32_t* __restrict__ slots,
            const int32_t* __restrict__ n_nodes, const int32_t* __restrict__ parents,
            const __half* __restrict__ q, const __half* __restrict__ k,
            const __half* __restrict__ v, __half* __restrict__ o, int n_seqs) {
  constexpr int C = D / 32;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= (int64_t)n_seqs * m * st.Hq) return;
  const int h = (int)(row % st.Hq), i = (int)(row / st.Hq % m), z = (int)(row / st.Hq / m);
  const int g = h / st.G, cnt = n_nodes ? min(m, n_nodes[z]) : m;
  if (i >= cnt) return;
  const int slot = slots[z];
  const bool slot_ok = slot >= 0 && slot < st.S;
  if (!slot_ok && lane == 0) set_error(st, EKV_EINVAL);
  const int T = slot_ok ? st.len[ls_index(st, layer, slot)] : 0;
  float qf[C], acc[C], mx = -CUDART_INF_F, l = 0.f;
  for (int c = 0; c < C; ++c) {
    qf[c] = __half2float(q[(((size_t)z * m + i) * st.Hq + h) * D + lane * C + c]) * st.scale_log2;
    acc[c] = 0.f;
  }
  auto add = [&](const float* kf, const float* vf) {
    float x = 0.f;
    for (int c = 0; c < C; ++c) x = fmaf(qf[c], kf[c], x);
    for (int off = 16; off; off >>= 1) x += __shfl_xor_sync(0xffffffffu, x, off);
    const float mn = fmaxf(mx, x), al = exp2f(mx - mn), p = exp2f(x - mn);
    l = l * al + p;
    for (int c = 0; c < C; ++c) acc[c] = fmaf(p, vf[c], acc[c] * al);
    mx = mn;
  };
  const size_t lsh = lsh_index(st, layer, slot_ok ? slot : 0, g);
  for (int t = 0; t < T; ++t) {
    const int32_t e = st.bt[lsh * st.maxblk + t / BLOCK];
    if (e == -1) {
      if (lane == 0) set_error(st, EKV_ESTATE);
      continue;
    }
    const int fmt = entry_fmt(e), kb = bits_of_code(fmt >> 2), r = t % BLOCK;
    const bool asym = st.asym != 0, open = t / BLOCK * BLOCK + BLOCK > T;
    const uint8_t* kp = st.pool_base[fmt] + (size_t)entry_idx(e) * st.pool_page_bytes[fmt];
    const uint8_t* vp = kp + k_part_bytes(kb, D, asym);
    const __half* ks = reinterpret_cast<const __half*>(kp + BLOCK * D * kb / 8);
    const __half* vs = reinterpret_cast<const __half*>(vp + BLOCK * D * vb / 8);
    float kf[C], vf[C];
    for (int c = 0; c < C; ++c) {
      const int ch = lane * C + c;
      if (open) {
        kf[c] = __half2float(st.staging[lsh * (BLOCK * D) + r * D + ch]);
      } else {
        kf[c] = code_at(kp, D, kb, r, ch, asym);
        if (kb < 16) {
          const int sp = k_scale_pos(kb, ch);
          kf[c] = kf[c] * __half2float(ks[sp]) + (asym ? __half2float(ks[D + sp]) : 0.f);
        }
      }
      vf[c] = code_at(vp, D, vb, r, ch, asym);
      if (vb < 16)
        vf[c] = vf[c] * __half2float(vs[r]) + (asym ? __half2float(vs[BLOCK + r]) : 0.f);
    }
    add(kf, vf);
  }
  for (int a = i, steps = 0; a >= 0 && steps < m; ++steps) {
    float kf[C], vf[C];
    for (int c = 0; c < C; ++c) {
      const size_t at = (((size_t)z * m + a) * st.Hkv + g) * D + lane * C + c;
      kf[c] = __half2float(k[at]);
      vf[c] = __half2float(v[at]);
    }
    add(kf, vf);
    const int up = parents[(size_t)z * m + a];
    a = up < a ? up : -1;
  }
  for (int c = 0; c < C; ++c)
    o[(((size_t)z * m + i) * st.Hq + h) * D + lane * C + c] = __float2half_rn(acc[c] / l);
}

}  // namespace
}  // namespace ekv

extern "C" EKV_API int ekv_tree_attn_scratch_bytes(ekv_cache* cache, int32_t n_seqs,
                                                   int32_t max_nodes, int64_t* out) {
  using namespace ekv;
  DevState st;
  int splits, vb, pack;
  if (!out || max_nodes < 1 || max_nodes > EKV_TREE_MAX_NODES) return EKV_EINVAL;
  const int rc = attn_plan(cache, 0, n_seqs, &st, &splits, &vb, &pack);
  if (rc == EKV_OK) *out = 0;
  return rc;
}

extern "C" EKV_API int ekv_tree_attn(ekv_cache* cache, int32_t layer, int32_t n_seqs,
                                     const int32_t* seq_slots, int32_t max_nodes,
                                     const int32_t* n_nodes, const int32_t* parents, const void* q,
                                     const void* k, const void* v, void* o, void* scratch,
                                     int64_t scratch_bytes, void* stream) {
  using namespace ekv;
  DevState st;
  int splits, vb, pack;
  if (max_nodes < 1 || max_nodes > EKV_TREE_MAX_NODES) return EKV_EINVAL;
  const int rc = attn_plan(cache, layer, n_seqs, &st, &splits, &vb, &pack);
  if (rc != EKV_OK) return rc;
  if (n_seqs == 0) return EKV_OK;
  if (!seq_slots || !parents || !q || !k || !v || !o) return EKV_EINVAL;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)o) & 15) return EKV_EINVAL;
  if (((uintptr_t)seq_slots | (uintptr_t)n_nodes | (uintptr_t)parents) & 3) return EKV_EINVAL;
  int64_t need = 0;
  ekv_tree_attn_scratch_bytes(cache, n_seqs, max_nodes, &need);
  if (scratch_bytes < need || (need > 0 && (!scratch || ((uintptr_t)scratch & 15))))
    return EKV_EINVAL;
  const unsigned grid = (unsigned)(((int64_t)n_seqs * max_nodes * st.Hq + 3) / 4);
  auto fn = st.D == 64 ? tree_kernel<64> : tree_kernel<128>;
  fn<<<grid, 128, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      st, layer, vb, max_nodes, seq_slots, n_nodes, parents, static_cast<const __half*>(q),
      static_cast<const __half*>(k), static_cast<const __half*>(v), static_cast<__half*>(o), n_seqs);
  return cudaGetLastError() == cudaSuccess ? EKV_OK : EKV_ECUDA;
}
