// ekv_verify.cu — verification of drafted trees against the target's probabilities.
//
// A sequence's tree has nodes 0 .. cnt-1, node 0 the root (the last committed
// token), parents[i] < i; p_u is the target's distribution after node u, and q_u
// (optional) the draft distribution that u's children were sampled from.  From
// the root, the children c of the current node are tried in index order with
// r = p_u, Z = 1:
//   accept c iff  u_c q(x_c) Z < r(x_c)            (without q: q(x_c) = 1)
//   else          r <- max(r - Z q, 0), Z <- sum r (without q: Z <- Z - r(x_c), r(x_c) <- 0)
// An accepted child becomes the current node.  At a node with no accepted child the
// walk ends and the next token is the lowest index i with cum_i(r) > u_s sum r; if
// sum r = 0 it is drawn from p_u.  Every token is then distributed as the target's.
//
// Sums over the vocabulary are exact: probabilities go to unsigned 64-bit fixed
// point in units of 2^-60 (an fp32 value above 2^-36 converts without loss), whose
// sums do not depend on their order, so the sampled index is the same on every
// launch.  Decisions compare one product in fp64.
//
// Only the gathered p(x_c), q(x_c) of the drafted nodes are read for the walk, all
// at once; whole rows are read only where the residual is needed: the last node's p
// (and q), and with q each node at which a child was rejected.  Bound by latency:
// one launch, one round of gathers, one pass over the last row.  A cluster of CL
// CTAs shares a sequence's row passes, exchanging partial sums through distributed
// shared memory (no CTA writes another's before a cluster barrier has shown that it runs,
// and none leaves while another may write its own).  Measured: 32 trees of 64 nodes over
// 131,072 tokens 22 us a call (the host's share is as long), 16 sampled trees of 16 over
// 100,003 with draft probabilities 26 to 34 (two to three passes at the nodes with
// rejections, ~3 us each).
#include <cooperative_groups.h>

#include "ekv_internal.h"

namespace cg = cooperative_groups;

namespace ekv {
namespace {

constexpr int VT = 512;          // threads per CTA
constexpr int VWARPS = VT / 32;
constexpr int VMAX = EKV_TREE_MAX_NODES;

struct VerifyArgs {
  const float* p;
  const float* q;
  int64_t p_seq, p_row, q_seq, q_row;
  const int32_t *tokens, *parents, *n_nodes;
  const float *u, *us;
  int32_t *path, *n_accept, *next;
  int m, vocab;
};

// An entry of a row as it counts: clamped to [0, 1], NaN as 0.
__device__ __forceinline__ float entry(float x) { return x > 0.f ? fminf(x, 1.f) : 0.f; }
// 2^60 of an entry, truncated: the 24-bit mantissa shifted to its place (the conversion
// instruction to 64 bits runs at a fraction of the rate of the shifts).
__device__ __forceinline__ uint64_t fix60(float x) {
  x = entry(x);
  const uint32_t bits = __float_as_uint(x);
  const int up = (int)(bits >> 23) - 90;  // x = m 2^(e - 150)
  const uint64_t m = (bits & 0x7FFFFFu) | 0x800000u;
  return up >= 0 ? m << up : up > -24 ? m >> -up : 0;
}
// a * z in units of 2^-60, a < 2^62 and z < 2^62 (saturated by the caller).
__device__ __forceinline__ uint64_t mul60(uint64_t a, uint64_t z) {
  return __umul64hi(a << 2, z << 2);
}
// The residual after k rejections with draft probabilities: z[j] is Z before
// rejection j (z[0] = 1, taken exactly).
__device__ __forceinline__ uint64_t residual(uint64_t r, uint64_t q, const uint64_t* z, int k) {
  for (int j = 0; j < k; ++j) {
    const uint64_t cut = j == 0 ? q : mul60(q, z[j]);
    r = r > cut ? r - cut : 0;
  }
  return r;
}

// The same for four entries side by side (a loop of branches for each entry took four times
// as long: every step waits for the one before).
__device__ __forceinline__ void residual4(uint64_t* r, const uint64_t* q, const uint64_t* z,
                                          int k) {
  if (k == 0) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) r[j] = r[j] > q[j] ? r[j] - q[j] : 0;
#pragma unroll 1
  for (int i = 1; i < k; ++i) {
    const uint64_t zi = z[i];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint64_t cut = mul60(q[j], zi);
      r[j] = r[j] > cut ? r[j] - cut : 0;
    }
  }
}

// Entries i .. i + 3 of a row of n (zero outside it), as one load where they lie inside
// and on a 16-byte boundary.
__device__ __forceinline__ void load4(const float* row, int i, int n, float* f) {
  if (i >= 0 && i + 4 <= n && !(reinterpret_cast<uintptr_t>(row + i) & 15)) {
    const float4 t = *reinterpret_cast<const float4*>(row + i);
    f[0] = t.x; f[1] = t.y; f[2] = t.z; f[3] = t.w;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = i + j >= 0 && i + j < n ? row[i + j] : 0.f;
  }
}
// Entries by which a row starts behind a 16-byte boundary: its units begin that much
// before it, so that any row (an odd vocabulary) is read in aligned vectors.
__device__ __forceinline__ int lead(const float* row) {
  return (int)(reinterpret_cast<uintptr_t>(row) >> 2 & 3);
}

template <int CL>
__global__ void __launch_bounds__(VT, 2) verify_kernel(VerifyArgs A) {
  __shared__ int s_par[VMAX], s_tok[VMAX], s_path[VMAX], s_gone[VMAX], s_first[VMAX], s_ngone;
  __shared__ float s_u[VMAX], s_p[VMAX], s_q[VMAX];
  __shared__ bool s_twin[VMAX], s_ok[VMAX];
  __shared__ unsigned long long s_kids[VMAX];
  __shared__ uint64_t s_wsum[VWARPS], s_part[2][CL], s_z[VMAX];
  const int z = blockIdx.x / CL, rank = blockIdx.x % CL;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Waited for before the walk: the gathers lie between.
  if constexpr (CL > 1) cg::this_cluster().barrier_arrive();
  const int V = A.vocab;
  const int cnt = A.n_nodes ? min(A.m, A.n_nodes[z]) : A.m;
  const float* P = A.p + z * A.p_seq;
  const float* Q = A.q ? A.q + z * A.q_seq : nullptr;
  if (tid < VMAX) {
    s_par[tid] = -1;
    s_first[tid] = VMAX;
    s_kids[tid] = 0;
    if (tid == 0) s_ngone = 0;
    if (tid < cnt) {
      const int par = tid ? A.parents[(size_t)z * A.m + tid] : -1;
      const int tok = A.tokens[(size_t)z * A.m + tid];
      // a bad parent or a token outside the vocabulary: no one's child
      const bool ok = tid > 0 && par >= 0 && par < tid && tok >= 0 && tok < V;
      s_par[tid] = ok ? par : -1;
      s_tok[tid] = tok;
      s_u[tid] = A.u[(size_t)z * A.m + tid];
      s_p[tid] = ok ? entry(P[par * A.p_row + tok]) : 0.f;
      s_q[tid] = ok && Q ? entry(Q[par * A.q_row + tok]) : 1.f;
    }
  }
  __syncthreads();
  const int par = tid < cnt ? s_par[tid] : -1;
  if (par >= 0) atomicOr(&s_kids[par], 1ull << tid);
  __syncthreads();
  const unsigned long long before = par >= 0 ? s_kids[par] & ((1ull << tid) - 1) : 0;
  if (par >= 0) {
    bool twin = false;  // an earlier sibling has the same token
    for (unsigned long long x = before; x; x &= x - 1) twin |= s_tok[__ffsll(x) - 1] == s_tok[tid];
    s_twin[tid] = twin;
  }
  __syncthreads();
  if (par >= 0 && Q) s_ok[tid] = (double)s_u[tid] * (double)s_q[tid] < (double)s_p[tid];
  if (par >= 0 && !Q && !s_twin[tid]) {
    // Without draft probabilities every node's test is known at once: Z is 1 less the
    // mass of its earlier siblings (each token once).
    double left = 1.0;
    for (unsigned long long x = before; x; x &= x - 1) {
      const int j = __ffsll(x) - 1;
      if (!s_twin[j]) left -= (double)s_p[j];
    }
    if ((double)s_u[tid] * left < (double)s_p[tid]) atomicMin(&s_first[par], tid);
  }
  __syncthreads();

  // The slice of a row that this CTA sums, and each warp's chunk of it, in units
  // of 128 elements (one 16-byte load per lane): contiguous, in order.
  const int units = (V + 3 + 127) / 128;  // with the lead of a row
  const int per_warp = (units + CL * VWARPS - 1) / (CL * VWARPS);
  const int u0 = min(units, (rank * VWARPS + warp) * per_warp);
  const int u1 = min(units, u0 + per_warp);
  int flip = 0;
  // Sum of the residual over the whole row: node's p (and q) after k rejections
  // (with q), or with the tokens s_gone[0 .. ngone) taken out (without).  Every
  // thread of the cluster returns the total; s_wsum holds this CTA's chunk sums,
  // s_part[flip ^ 1] all CTAs' sums.
  auto row_sum = [&](int node, int k, int ngone) -> uint64_t {
    const float* pr = P + node * A.p_row;
    const float* qr = Q ? Q + node * A.q_row : nullptr;
    uint64_t sum = 0;
    // Short loops on purpose: each row is passed once or twice a launch, and code that is
    // run so seldom costs its instruction fetches (unrolled over 4 units a pass took 7 us).
    float a[4], b[4];
    const int at = lane * 4 - lead(pr);
    load4(pr, u0 * 128 + at, u0 < u1 ? V : 0, a);
    if (k == 0) {
#pragma unroll 1
      for (int t = u0; t < u1; ++t) {
        float c[4];
        load4(pr, (t + 1) * 128 + at, t + 1 < u1 ? V : 0, c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sum += fix60(a[j]);
          a[j] = c[j];
        }
      }
    } else {
      load4(qr, u0 * 128 + at, u0 < u1 ? V : 0, b);
#pragma unroll 1
      for (int t = u0; t < u1; ++t) {
        float c[4], d[4];
        load4(pr, (t + 1) * 128 + at, t + 1 < u1 ? V : 0, c);
        load4(qr, (t + 1) * 128 + at, t + 1 < u1 ? V : 0, d);
        uint64_t x[4], y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          x[j] = fix60(a[j]);
          y[j] = fix60(b[j]);
          a[j] = c[j];
          b[j] = d[j];
        }
        residual4(x, y, s_z, k);
        sum += x[0] + x[1] + x[2] + x[3];
      }
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) s_wsum[warp] = sum;
    __syncthreads();
    if (tid < ngone) {  // distinct tokens, each in one warp's chunk
      const int x = s_gone[tid], w = (x + lead(pr)) / 128 / per_warp - rank * VWARPS;
      if (w >= 0 && w < VWARPS)
        atomicAdd(reinterpret_cast<unsigned long long*>(&s_wsum[w]),
                  (unsigned long long)(0 - fix60(pr[x])));
    }
    __syncthreads();
    if (tid < CL) {
      uint64_t mine = 0;
      for (int w = 0; w < VWARPS; ++w) mine += s_wsum[w];
      if (CL == 1) s_part[flip][0] = mine;
      else *cg::this_cluster().map_shared_rank(&s_part[flip][rank], tid) = mine;
    }
    if (CL == 1) __syncthreads();
    else cg::this_cluster().sync();
    uint64_t total = 0;
    for (int r = 0; r < CL; ++r) total += s_part[flip][r];
    flip ^= 1;
    return total;
  };

  if constexpr (CL > 1) cg::this_cluster().barrier_wait();
  // The walk, the same in every thread of the cluster.
  int node = 0, nacc = 0, k = 0, ngone = 0;
  uint64_t total = 0;
  bool have = false;  // `total` is the residual's sum at the current node
  if (cnt > 0 && !Q) {
    for (int c; (c = s_first[node]) < VMAX; node = c) {
      if (tid == 0) s_path[nacc] = c;
      ++nacc;
    }
    // the tokens that the last node's rejected children took out
    if (par == node && !s_twin[tid]) s_gone[atomicAdd(&s_ngone, 1)] = s_tok[tid];
    __syncthreads();
    ngone = s_ngone;
  } else if (cnt > 0) {
    double left = 1.0;
    unsigned long long kids = s_kids[0];
    while (kids) {
      const int c = __ffsll(kids) - 1;
      kids &= kids - 1;
      // (a first child's test, r = p and Z = 1, was made for all nodes at once)
      const bool take =
          k == 0 ? s_ok[c]
                 : (double)s_u[c] * (double)s_q[c] * left <
                       (double)residual(fix60(s_p[c]), fix60(s_q[c]), s_z, k) * 0x1p-60;
      if (take) {
        if (tid == 0) s_path[nacc] = c;
        ++nacc;
        node = c;
        kids = s_kids[c];
        k = 0;
        left = 1.0;
        have = false;
        continue;
      }
      __syncthreads();
      if (tid == 0) s_z[k] = k == 0 ? 1ull << 60 : min(total, (uint64_t)((1ull << 62) - 1));
      ++k;
      __syncthreads();
      total = row_sum(node, k, 0);
      have = true;
      left = (double)total * 0x1p-60;
    }
  }

  if (cnt > 0) {
    if (!have) total = row_sum(node, k, ngone);
    if (total == 0 && (k > 0 || ngone > 0)) {
      k = ngone = 0;
      total = row_sum(node, 0, 0);
    }
    if (total > 0) {
      const float us = A.us[z];
      const uint64_t frac = us >= 1.f ? ~0ull : us > 0.f ? __float2ull_rz(us * 0x1p64f) : 0ull;
      const uint64_t target = __umul64hi(frac, total);  // floor(u_s * sum r) < sum r
      uint64_t base = 0;
      for (int r = 0; r < rank; ++r) base += s_part[flip ^ 1][r];
      for (int w = 0; w < warp; ++w) base += s_wsum[w];
      if (target >= base && target - base < s_wsum[warp]) {  // this warp's chunk holds it
        const float* pr = P + node * A.p_row;
        const float* qr = Q ? Q + node * A.q_row : nullptr;
#pragma unroll 1
        for (int t = u0; t < u1; ++t) {
          float a[4], b[4] = {0.f, 0.f, 0.f, 0.f};
          const int i0 = t * 128 + lane * 4 - lead(pr);
          load4(pr, i0, V, a);
          if (k) load4(qr, i0, V, b);
          uint64_t e[4], y[4], s = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            e[j] = fix60(a[j]);
            y[j] = fix60(b[j]);
          }
          residual4(e, y, s_z, k);
#pragma unroll 1
          for (int g = 0; g < ngone; ++g) {
            const int at = s_gone[g] - i0;
#pragma unroll
            for (int j = 0; j < 4; ++j)
              if (at == j) e[j] = 0;
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) s += e[j];
          uint64_t inc = s;
#pragma unroll 1
          for (int off = 1; off < 32; off <<= 1) {
            const uint64_t o = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += o;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, base + inc > target);
          if (hit) {
            if (lane == __ffs(hit) - 1) {
              uint64_t cum = base + inc - s;
              int at = i0;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                cum += e[j];
                at += cum <= target;
              }
              A.next[z] = at;
            }
            break;
          }
          base += __shfl_sync(0xffffffffu, inc, 31);
        }
      }
    }
  }
  __syncthreads();
  if (rank == 0) {
    if (tid < A.m) A.path[(size_t)z * A.m + tid] = tid < nacc ? s_path[tid] : -1;
    if (tid == 0) {
      A.n_accept[z] = nacc;
      if (cnt <= 0) A.next[z] = -1;
      else if (total == 0) A.next[z] = V - 1;  // an all-zero row
    }
  }
  if (CL > 1) cg::this_cluster().sync();  // no CTA leaves while another may write its sums
}

template <int CL>
cudaError_t launch_verify(const VerifyArgs& A, int n_seqs, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n_seqs * CL);
  cfg.blockDim = dim3(VT);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = CL;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, verify_kernel<CL>, A);
}

}  // namespace
}  // namespace ekv

extern "C" EKV_API int ekv_verify_tree(int32_t n_seqs, int32_t max_nodes, int32_t vocab,
                                       const float* target_probs, int64_t target_seq_stride,
                                       int64_t target_row_stride, const float* draft_probs,
                                       int64_t draft_seq_stride, int64_t draft_row_stride,
                                       const int32_t* tokens, const int32_t* parents,
                                       const int32_t* n_nodes, const float* u_accept,
                                       const float* u_sample, int32_t* path, int32_t* n_accept,
                                       int32_t* next_token, void* stream) {
  using namespace ekv;
  if (n_seqs < 0 || n_seqs > (1 << 20) || max_nodes < 1 || max_nodes > EKV_TREE_MAX_NODES ||
      vocab < 1 || vocab > (1 << 30))  // (entries are counted in int, a few units past the end)
    return EKV_EINVAL;
  if (n_seqs == 0) return EKV_OK;
  if (!target_probs || !tokens || !parents || !u_accept || !u_sample || !path || !n_accept ||
      !next_token)
    return EKV_EINVAL;
  if (((uintptr_t)target_probs | (uintptr_t)draft_probs | (uintptr_t)tokens | (uintptr_t)parents |
       (uintptr_t)n_nodes | (uintptr_t)u_accept | (uintptr_t)u_sample | (uintptr_t)path |
       (uintptr_t)n_accept | (uintptr_t)next_token) & 3)
    return EKV_EINVAL;
  if ((max_nodes > 1 && target_row_stride < vocab) || (n_seqs > 1 && target_seq_stride < 0))
    return EKV_EINVAL;
  if (draft_probs && ((max_nodes > 1 && draft_row_stride < vocab) ||
                      (n_seqs > 1 && draft_seq_stride < 0)))
    return EKV_EINVAL;
  VerifyArgs A = {};
  A.p = target_probs;
  A.q = draft_probs;
  A.p_seq = target_seq_stride;
  A.p_row = target_row_stride;
  A.q_seq = draft_seq_stride;
  A.q_row = draft_row_stride;
  A.tokens = tokens;
  A.parents = parents;
  A.n_nodes = n_nodes;
  A.u = u_accept;
  A.us = u_sample;
  A.path = path;
  A.n_accept = n_accept;
  A.next = next_token;
  A.m = max_nodes;
  A.vocab = vocab;
  // A cluster of 8 CTAs a sequence once a row has more than a few units a warp.  Kernel time of
  // 32 sequences of 8 nodes with eight CTAs and with one, us: 131,072 entries 14.9 and 54.0
  // (with draft probabilities 45 and 166), 16,384 7.9 and 10.7 (21 and 31), 8,192 6.7 and 7.8
  // (14.2 and 16.4), 4,096 6.7 and 6.2 (14.8 both), 1,024 6.6 and 4.9 (11.8 and 7.9): the
  // cluster's barriers against the row; one sequence crosses at the same sizes.
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e =
      vocab > 8192 ? launch_verify<8>(A, n_seqs, s) : launch_verify<1>(A, n_seqs, s);
  return e == cudaSuccess ? EKV_OK : EKV_ECUDA;
}
