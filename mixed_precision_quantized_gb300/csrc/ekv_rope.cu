// ekv_rope.cu — rotary positions of q and k before the append and the attention.
//
// Pair i of a head's first r channels, (x_a, x_b) = (i, i + r/2) (half layout) or
// (2i, 2i+1) (interleaved), turns by the angle t = pos * f_i:
//   y_a = g (x_a cos t - x_b sin t),  y_b = g (x_b cos t + x_a sin t)
// and the other d - r channels pass through.  f_i = base^(-2i/r), changed for
// long contexts by the configured scaling; g is the scaling's magnitude.
//
// The angle is kept in turns as a 64-bit fixed-point fraction: the table holds
// F_i = f_i / 2pi * 2^64 of a double f_i, and pos * F_i mod 2^64 is the fraction
// of a turn, exact in the product for every int32 position.  f_i <= 1 is within
// 2^-53 turns a position of its formula (the roundings of the exponent, pow and the
// division; 2^-55 measured), at position 131,072 within 2^-36 and at the last 2^-22.
// The top 32 bits go to fp32 (2^-26 turns) and through sincospif, so a far position
// loses nothing to range reduction and no fp64 arithmetic is spent.  The rotation is
// done in fp32 and rounded to fp16 once.
//
// Bound by memory: each q and k element is read and written once.  A CTA takes a
// few tokens; its threads first fill a shared table of cos and sin, one entry
// per (token, pair), which all q and k heads of the token share, then rotate
// 8 pairs (half layout) or 4 pairs (interleaved) per step in 16-byte accesses.
// Measured: 32,768 tokens of 48 heads of 128, interleaved, 133 us (805 MB: 6.05 TB/s, 0.89
// of a plain copy), one pair at a time (a rotated part that the vectors do not fit) 569; a thread that found its (token, head, unit) by division for every 16
// bytes took 164.  4,099 tokens of 72 heads read from a fused projection: 33 us; with 2
// tokens a CTA instead of 4 it takes 35.
#include <float.h>
#include <math.h>

#include "ekv_internal.h"

namespace ekv {
namespace {

constexpr int ROPE_THREADS = 256;
constexpr int ROPE_MAX_TOKENS = 4;   // tokens of one CTA at most
constexpr int ROPE_MAX_PAIRS = 64;   // head_dim / 2

struct RopeArgs {
  const uint64_t* turns;
  const int32_t* pos;
  const __half* x[2];   // q, k
  __half* y[2];
  int64_t xs[2], ys[2];  // token strides (elements)
  int heads[2];
  int64_t n;
  int d, rot, tokens;    // tokens per CTA
  float mag;
};

__device__ __forceinline__ void rotate2(uint32_t& a, uint32_t& b, float2 w0, float2 w1) {
  // a = (x_a0, x_a1), b = (x_b0, x_b1) of two pairs
  const float2 fa = __half22float2(*reinterpret_cast<__half2*>(&a));
  const float2 fb = __half22float2(*reinterpret_cast<__half2*>(&b));
  const __half2 ra = __floats2half2_rn(fa.x * w0.x - fb.x * w0.y, fa.y * w1.x - fb.y * w1.y);
  const __half2 rb = __floats2half2_rn(fb.x * w0.x + fa.x * w0.y, fb.y * w1.x + fa.y * w1.y);
  a = *reinterpret_cast<const uint32_t*>(&ra);
  b = *reinterpret_cast<const uint32_t*>(&rb);
}
__device__ __forceinline__ uint32_t rotate1(uint32_t ab, float2 w) {  // (x_a, x_b) of one pair
  const float2 f = __half22float2(*reinterpret_cast<__half2*>(&ab));
  const __half2 r = __floats2half2_rn(f.x * w.x - f.y * w.y, f.y * w.x + f.x * w.y);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// MODE 0: half layout, r a multiple of 16 (16-byte accesses); 1: interleaved, r a
// multiple of 8 (16-byte accesses); 2 / 3: half / interleaved for any even r, one
// pair at a time.
template <int MODE>
__global__ void __launch_bounds__(ROPE_THREADS) rope_kernel(RopeArgs A) {
  __shared__ float2 s_w[ROPE_MAX_TOKENS * ROPE_MAX_PAIRS];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * A.tokens;
  const int nt = (int)min((int64_t)A.tokens, A.n - t0);
  const int half = A.rot / 2;
  for (int i = tid; i < nt * half; i += ROPE_THREADS) {
    const int t = i / half, p = i - t * half;
    const uint64_t frac = (uint64_t)(int64_t)A.pos[t0 + t] * A.turns[p];
    float s, c;
    sincospif((float)(int32_t)(frac >> 32) * 0x1p-31f, &s, &c);  // 2 pi frac = pi (2 frac)
    s_w[t * ROPE_MAX_PAIRS + p] = make_float2(c * A.mag, s * A.mag);
  }
  __syncthreads();
  constexpr bool VEC = MODE < 2;
  // Units of one head: rotated ones, then (16-byte or single-channel) copies.  A thread
  // keeps its unit and goes through the (token, head) items, q's heads before k's.
  const int ru = MODE == 0 ? A.rot / 16 : MODE == 1 ? A.rot / 8 : half;
  const int units = ru + (VEC ? (A.d - A.rot) / 8 : A.d - A.rot);
  const int H = A.heads[0] + A.heads[1], groups = ROPE_THREADS / units;
  const int hg = tid / units, u = tid - hg * units;
  if (hg >= groups) return;
  const int ia = MODE < 2 ? 8 * u : MODE == 2 ? u : 2 * u;  // first channel
  const int ib = MODE == 0 ? half + 8 * u : MODE == 2 ? u + half : ia + 1;
  const int ic = A.rot + (u - ru) * (VEC ? 8 : 1);
  constexpr int N = 2;  // items in flight
  int t[N], h[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int it = hg + i * groups;
    t[i] = it / H;
    h[i] = it - t[i] * H;
  }
  while (t[0] < nt) {
    const __half* src[N];
    __half* dst[N];
    uint4 a[N], b[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const bool k = h[i] >= A.heads[0];
      const size_t head = (size_t)(k ? h[i] - A.heads[0] : h[i]) * A.d;
      src[i] = (k ? A.x[1] : A.x[0]) + (t0 + t[i]) * (k ? A.xs[1] : A.xs[0]) + head;
      dst[i] = (k ? A.y[1] : A.y[0]) + (t0 + t[i]) * (k ? A.ys[1] : A.ys[0]) + head;
      if (t[i] >= nt) continue;
      if (u < ru) {
        if (VEC) a[i] = *reinterpret_cast<const uint4*>(src[i] + ia);
        if (MODE == 0) b[i] = *reinterpret_cast<const uint4*>(src[i] + ib);
      } else if (VEC) {
        a[i] = *reinterpret_cast<const uint4*>(src[i] + ic);
      }
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (t[i] < nt) {
        const float2* w = s_w + t[i] * ROPE_MAX_PAIRS + (MODE == 0 ? 8 * u : MODE == 1 ? 4 * u : u);
        if (u >= ru) {
          if (src[i] != dst[i]) {
            if (VEC) *reinterpret_cast<uint4*>(dst[i] + ic) = a[i];
            else dst[i][ic] = src[i][ic];
          }
        } else if (MODE == 0) {
          rotate2(a[i].x, b[i].x, w[0], w[1]);
          rotate2(a[i].y, b[i].y, w[2], w[3]);
          rotate2(a[i].z, b[i].z, w[4], w[5]);
          rotate2(a[i].w, b[i].w, w[6], w[7]);
          *reinterpret_cast<uint4*>(dst[i] + ia) = a[i];
          *reinterpret_cast<uint4*>(dst[i] + ib) = b[i];
        } else if (MODE == 1) {
          a[i].x = rotate1(a[i].x, w[0]);
          a[i].y = rotate1(a[i].y, w[1]);
          a[i].z = rotate1(a[i].z, w[2]);
          a[i].w = rotate1(a[i].w, w[3]);
          *reinterpret_cast<uint4*>(dst[i] + ia) = a[i];
        } else {
          const float fa = __half2float(src[i][ia]), fb = __half2float(src[i][ib]);
          dst[i][ia] = __float2half_rn(fa * w->x - fb * w->y);
          dst[i][ib] = __float2half_rn(fb * w->x + fa * w->y);
        }
      }
      h[i] += N * groups;
      while (h[i] >= H) {
        h[i] -= H;
        ++t[i];
      }
    }
  }
}

bool valid_config(const ekv_rope_config* c) {
  if (!c || (c->head_dim != 64 && c->head_dim != 128)) return false;
  if (c->rot_dim < 2 || c->rot_dim > c->head_dim || (c->rot_dim & 1)) return false;
  if (c->layout != EKV_ROPE_HALF && c->layout != EKV_ROPE_INTERLEAVED) return false;
  if (c->scaling < EKV_ROPE_SCALE_NONE || c->scaling > EKV_ROPE_SCALE_YARN) return false;
  if (!(c->base > 1.0) || !isfinite(c->base)) return false;
  if (!(c->magnitude >= 0.0 && c->magnitude <= FLT_MAX)) return false;
  // (below DBL_MIN a frequency over it may be infinite)
  if (c->scaling != EKV_ROPE_SCALE_NONE && (!(c->factor >= DBL_MIN) || !isfinite(c->factor)))
    return false;
  if (c->scaling == EKV_ROPE_SCALE_BANDED || c->scaling == EKV_ROPE_SCALE_YARN) {
    if (!(c->original_len > 0.0) || !isfinite(c->original_len)) return false;
  }
  if (c->scaling == EKV_ROPE_SCALE_BANDED &&
      !(c->low_freq_factor > 0.0 && c->high_freq_factor > c->low_freq_factor &&
        isfinite(c->high_freq_factor)))
    return false;
  if (c->scaling == EKV_ROPE_SCALE_YARN &&
      !(c->beta_slow > 0.0 && c->beta_fast > c->beta_slow && isfinite(c->beta_fast)))
    return false;
  return true;
}

constexpr double kTwoPi = 6.283185307179586476925286766559;

float magnitude_of(const ekv_rope_config& c) {
  if (c.magnitude > 0.0) return (float)c.magnitude;
  return c.scaling == EKV_ROPE_SCALE_YARN && c.factor > 1.0 ? (float)(0.1 * log(c.factor) + 1.0)
                                                            : 1.f;
}

double freq_of(const ekv_rope_config& c, int i) {
  const int r = c.rot_dim;
  const double f = pow(c.base, -2.0 * i / r);
  switch (c.scaling) {
    case EKV_ROPE_SCALE_LINEAR: return f / c.factor;
    case EKV_ROPE_SCALE_BANDED: {
      const double turns = c.original_len * f / kTwoPi;  // over the original context
      double w = (turns - c.low_freq_factor) / (c.high_freq_factor - c.low_freq_factor);
      w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
      return f * (w + (1.0 - w) / c.factor);
    }
    case EKV_ROPE_SCALE_YARN: {
      // the pair index at which the original context holds `turns` turns
      auto edge = [&](double turns) {
        return r * log(c.original_len / (turns * kTwoPi)) / (2.0 * log(c.base));
      };
      const double lo = fmax(floor(edge(c.beta_fast)), 0.0);
      const double hi = fmin(ceil(edge(c.beta_slow)), r - 1.0);
      double w = (i - lo) / fmax(hi - lo, 1e-3);
      w = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
      return f * (1.0 - w + w / c.factor);
    }
    default: return f;
  }
}

}  // namespace
}  // namespace ekv

extern "C" EKV_API int ekv_rope_table(const ekv_rope_config* cfg, uint64_t* turns,
                                      float* magnitude) {
  using namespace ekv;
  if (!valid_config(cfg) || !turns) return EKV_EINVAL;
  for (int i = 0; i < cfg->rot_dim / 2; ++i) {
    double t = freq_of(*cfg, i) / kTwoPi;
    t -= floor(t);  // whole turns do not matter
    // t < 1 in doubles, so t * 2^64 < 2^64; split so that only bits below 2^-64 are cut
    const uint64_t hi = (uint64_t)(t * 0x1p32);
    turns[i] = (hi << 32) + (uint64_t)((t * 0x1p32 - (double)hi) * 0x1p32);
  }
  if (magnitude) *magnitude = magnitude_of(*cfg);
  return EKV_OK;
}

extern "C" EKV_API int ekv_rope(const ekv_rope_config* cfg, const uint64_t* turns, int64_t n_tokens,
                                const int32_t* positions, int32_t n_q_heads, const void* q,
                                int64_t q_stride, void* q_out, int64_t q_out_stride,
                                int32_t n_kv_heads, const void* k, int64_t k_stride, void* k_out,
                                int64_t k_out_stride, void* stream) {
  using namespace ekv;
  if (!valid_config(cfg) || n_tokens < 0 || n_tokens > 0x7FFFFFFF || n_q_heads < 0 ||
      n_kv_heads < 0 || n_q_heads > 4096 || n_kv_heads > 4096)
    return EKV_EINVAL;
  if (n_tokens == 0 || n_q_heads + n_kv_heads == 0) return EKV_OK;
  if (!turns || !positions || ((uintptr_t)turns & 7) || ((uintptr_t)positions & 3))
    return EKV_EINVAL;
  RopeArgs A = {};
  const int heads[2] = {n_q_heads, n_kv_heads};
  const void* xs[2] = {q, k};
  void* ys[2] = {q_out, k_out};
  const int64_t xst[2] = {q_stride, k_stride}, yst[2] = {q_out_stride, k_out_stride};
  for (int w = 0; w < 2; ++w) {
    A.heads[w] = heads[w];
    if (heads[w] == 0) continue;
    const int64_t row = (int64_t)heads[w] * cfg->head_dim;
    if (!xs[w] || !ys[w] || (((uintptr_t)xs[w] | (uintptr_t)ys[w]) & 15)) return EKV_EINVAL;
    if (xst[w] < row || yst[w] < row || ((xst[w] | yst[w]) & 7)) return EKV_EINVAL;
    if (xs[w] == ys[w] && xst[w] != yst[w]) return EKV_EINVAL;  // in place: the same rows
    A.x[w] = static_cast<const __half*>(xs[w]);
    A.y[w] = static_cast<__half*>(ys[w]);
    A.xs[w] = xst[w];
    A.ys[w] = yst[w];
  }
  A.turns = turns;
  A.pos = positions;
  A.n = n_tokens;
  A.d = cfg->head_dim;
  A.rot = cfg->rot_dim;
  A.mag = magnitude_of(*cfg);
  // Four tokens a CTA once there are enough of them for all SMs.  Kernel time with four and with
  // one, us: 40 heads of 128 at 256 tokens 4.3 and 3.1, 512 4.4 and 4.0, 1,024 5.8 and 6.3,
  // 2,048 9.4 and 10.1, 32,768 114 and 149; 6 heads at 256 2.7 both, 2,048 3.9 and 7.7.
  A.tokens = n_tokens >= 2048 ? ROPE_MAX_TOKENS : 1;
  const int64_t grid = (n_tokens + A.tokens - 1) / A.tokens;
  const bool inter = cfg->layout == EKV_ROPE_INTERLEAVED;
  const bool vec = A.rot % (inter ? 8 : 16) == 0;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (vec && !inter) rope_kernel<0><<<(unsigned)grid, ROPE_THREADS, 0, s>>>(A);
  else if (vec) rope_kernel<1><<<(unsigned)grid, ROPE_THREADS, 0, s>>>(A);
  else if (!inter) rope_kernel<2><<<(unsigned)grid, ROPE_THREADS, 0, s>>>(A);
  else rope_kernel<3><<<(unsigned)grid, ROPE_THREADS, 0, s>>>(A);
  return cudaGetLastError() == cudaSuccess ? EKV_OK : EKV_ECUDA;
}
