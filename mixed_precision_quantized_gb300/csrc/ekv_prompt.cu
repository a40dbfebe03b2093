// ekv_prompt.cu — causal attention over whole prompts, packed end to end.
//
// For token i of a sequence and query head h with KV head g = h / (Hq / Hkv):
//   o_ih = sum_{j <= i} softmax_j(sigma q_ih . k_jg) v_jg
// in one pass over the keys with a running maximum and sum.
//
// Bound by the tensor cores: 4 d flops for each (row, key) pair.  A work item is one or
// two query tiles of 128 rows (one head each, of one KV head's group, so both read the
// same K and V tiles); a CTA per SM walks its items.  Roles:
//   warp 9     TMA: Q tiles, then K and V tiles of 128 keys through a ring of slots
//   warp 8     tcgen05.mma: S_t = Q_t K^T (128 x 128 fp32 in tensor memory), then
//              O_t += P_t V with P_t read from tensor memory; the two tiles alternate,
//              so one tile's products run while the other's softmax does
//   warps 0-3 (tile 0), 4-7 (tile 1)  softmax, one row a thread: S from tensor memory,
//              running maximum, P = 2^(sigma log2(e) s - m) as fp16 over S's columns, row
//              sums in fp32, the final O / l
// The reference m of a row moves only when a score passes it by more than 2^8, so O is
// rescaled seldom; P carries a factor 2^7 (at most 2^15 in all), which keeps terms down
// to 2^-21 of the largest in fp16's normal range.  P's rounding to fp16 (2^-11 of each
// term, as the output's own) is what the tensor cores' fp16 operands ask for; sums and
// maxima are fp32 and are taken before it.
//
// Only a sequence's last key tile can hold rows behind it.  Their scores are masked by
// the diagonal (they are keys after every row), and their V rows are overwritten with
// zeros in shared memory before the product, so that nothing outside a sequence (NaN,
// infinities) reaches its rows.
//
// Measured: one sequence of 16,384 tokens, 32 query and 8 KV heads of 128: 1,457 us warm,
// 1,525 with inputs that change from call to call (1.44e15 flops a second), heads of 64 1,095
// (1.0e15: the exponentials, as many for half the products); 24 ragged sequences of up to
// 2,047: 298 us.  The tensor cores are busy three quarters of the time at
// 16K tokens and half of it at 4K; what is left is the chain from scores to probabilities to
// products at each item's ends.  Tried and slower: one loop of mixed steps for the two tiles'
// products (1,800: the operands' addresses are worked out between wait and issue), scores
// read twice, 32 columns at a time, instead of kept in registers (1,455 against 1,426).
//
// Items go heaviest first (by their row tile, over all sequences in order of length) and
// are dealt to the CTAs in alternating direction, which needs no counter in memory.
#include <cuda.h>
#include <math_constants.h>

#include "ekv_internal.h"
#include "ekv_tc.cuh"

namespace ekv {
namespace {

using namespace tc;

constexpr int BM = 128;            // rows of a query tile and keys of a KV tile
constexpr int PT = 384;            // threads: 8 softmax warps, MMA warp, TMA warp, 2 idle
// Registers a thread: 168 at launch (65,536 / 384, in eights).  The softmax warps hold a
// score row of 128 and its packed probabilities and take 208, the others keep 80:
// 256 x 208 + 128 x 80 = 63,488 of the launch's 64,512.
constexpr int REGS_SOFTMAX = 208, REGS_OTHER = 80;
constexpr int MAX_SEQS = 512;      // sequences of one launch
constexpr int SUB = BM * 128;      // bytes of a 64-channel sub-tile: 128 rows of 128 bytes

template <int D>
struct PCfg {
  static constexpr int TILE = BM * D * 2;
  static constexpr int SLOTS = D == 128 ? 4 : 8;
  static constexpr int Q_OFF = 0, KV_OFF = 2 * TILE, TAB_OFF = KV_OFF + SLOTS * TILE;
  static constexpr int SMEM = TAB_OFF + MAX_SEQS * 4 * 2 + MAX_SEQS * 2 + 256 + 1024;
};

struct PromptArgs {
  const int32_t* cu;
  int n_seqs, total;
  int Hq, Hkv, G;
  int unit;    // row tiles of one level (2 if G is odd: pairs may join two of them)
  int per;     // query tiles of an item (1 or 2)
  float sl;    // sigma log2(e)
  __half* o;
  int64_t os;
};

// Sequence table of a launch in shared memory: bounds, and the sequences by
// descending level count.
struct Table {
  int32_t* start;
  int32_t* len;
  uint16_t* order;
  int n;
};

__device__ __forceinline__ int levels_of(const PromptArgs& A, int len) {
  return (len + BM * A.unit - 1) / (BM * A.unit);
}

// Walks the items of this CTA, the same in every role.
struct Cursor {
  int level, cnt, base, round;
  int z, head, tile0;  // the item: sequence, KV head, first query tile of its level
  __device__ void init(const PromptArgs& A, const Table& t) {
    base = round = cnt = 0;
    level = t.n ? levels_of(A, t.len[t.order[0]]) - 1 : -1;
    grow(A, t);
  }
  __device__ void grow(const PromptArgs& A, const Table& t) {
    while (cnt < t.n && levels_of(A, t.len[t.order[cnt]]) > level) ++cnt;
  }
  __device__ bool next(const PromptArgs& A, const Table& t) {
    const int pairs = (A.unit * A.G + A.per - 1) / A.per;
    const int id = round * (int)gridDim.x +
                   ((round & 1) ? (int)gridDim.x - 1 - (int)blockIdx.x : (int)blockIdx.x);
    ++round;
    const int each = A.Hkv * pairs;
    while (level >= 0 && id >= base + cnt * each) {
      base += cnt * each;
      --level;
      grow(A, t);
    }
    if (level < 0) return false;
    const int r = id - base;
    z = t.order[r / each];
    head = r % each / pairs;
    tile0 = r % pairs * A.per;
    return true;
  }
  // Tile t of the item: its row tile and query head; false if there is none.
  __device__ bool tile(const PromptArgs& A, const Table& tb, int t, int& mt, int& h) const {
    const int i = tile0 + t;
    mt = level * A.unit + i / A.G;
    h = head * A.G + i % A.G;
    return t < A.per && i < A.unit * A.G && mt * BM < tb.len[z];
  }
};

template <int D>
__global__ void __launch_bounds__(PT, 1)
prompt_kernel(PromptArgs A, const __grid_constant__ CUtensorMap mq,
              const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv) {
  using Cfg = PCfg<D>;
  constexpr int SLOTS = Cfg::SLOTS, TILE = Cfg::TILE, NSUB = D / 64;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  const uint32_t sb = smem_u32(smem);
  Table tb;
  tb.start = reinterpret_cast<int32_t*>(smem + Cfg::TAB_OFF);
  tb.len = tb.start + MAX_SEQS;
  tb.order = reinterpret_cast<uint16_t*>(tb.len + MAX_SEQS);
  tb.n = A.n_seqs;
  uint64_t* bars = reinterpret_cast<uint64_t*>(tb.order + MAX_SEQS);
  const uint32_t b0 = smem_u32(bars);
  const uint32_t q_full = b0, q_empty = b0 + 16, s_full = b0 + 32, p_full = b0 + 48,
                 o_done = b0 + 64, tail = b0 + 80, kv_full = b0 + 96,
                 kv_empty = kv_full + 8 * SLOTS;
  volatile int* stop = reinterpret_cast<volatile int*>(bars + 12 + 2 * SLOTS);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(bars + 12 + 2 * SLOTS) + 1;
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;

  for (int z = tid; z < A.n_seqs; z += PT) {
    const int a = A.cu[z], b = A.cu[z + 1];
    const bool ok = a >= 0 && b <= A.total && a <= b;
    tb.start[z] = a;
    tb.len[z] = ok ? b - a : 0;
  }
  if (tid == 0) {
    for (int t = 0; t < 2; ++t) {
      bar_init(q_full + 8 * t, 1);
      bar_init(q_empty + 8 * t, 1);
      bar_init(s_full + 8 * t, 1);
      bar_init(p_full + 8 * t, 4);
      bar_init(o_done + 8 * t, 1);
    }
    bar_init(tail, 1);
    for (int i = 0; i < SLOTS; ++i) {
      bar_init(kv_full + 8 * i, 1);
      bar_init(kv_empty + 8 * i, 1);
    }
    *stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 8) tmem_alloc(smem_u32(s_tmem), 512);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tm = uniform(*s_tmem);  // columns: S0/P0 0.., S1/P1 128.., O0 256.., O1 256 + D..
  for (int z = tid; z < A.n_seqs; z += PT) {  // rank by length, longest first
    const int mine = levels_of(A, tb.len[z]);
    int rank = 0;
    for (int y = 0; y < A.n_seqs; ++y) {
      const int other = levels_of(A, tb.len[y]);
      rank += other > mine || (other == mine && y < z);
    }
    tb.order[rank] = (uint16_t)z;
  }
  __syncthreads();

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_OTHER));
    Cursor cur;
    cur.init(A, tb);
    if (warp == 9) {
      // ---- loads ---------------------------------------------------------------------
      int slot = 0;
      uint32_t ph = 1, qph = 3, tph = 0;  // parities; an empty barrier's first wait passes at once
      while (cur.next(A, tb)) {
        int nk = 0;
        const int start = tb.start[cur.z], len = tb.len[cur.z];
        for (int t = 0; t < 2; ++t) {
          int mt, h;
          if (!cur.tile(A, tb, t, mt, h)) continue;
          nk = max(nk, mt + 1);
          if (!warp_wait(q_empty + 8 * t, (qph >> t) & 1, stop)) break;
          qph ^= 1u << t;
          if (lane == 0) {
            bar_expect(q_full + 8 * t, TILE);
            for (int s = 0; s < NSUB; ++s)
              tma_3d(sb + Cfg::Q_OFF + t * TILE + s * SUB, &mq, s * 64, h, start + mt * BM,
                     q_full + 8 * t);
          }
        }
        for (int i = 0; i < 2 * nk && !*stop; ++i) {  // K0, V0, K1, V1, ...
          const int j = i >> 1;
          const bool is_v = i & 1;
          if (!warp_wait(kv_empty + 8 * slot, ph, stop)) break;
          const uint32_t dst = sb + Cfg::KV_OFF + slot * TILE;
          const int left = len - j * BM;  // rows of the sequence from this tile's first
          const bool cut = is_v && left < BM;
          const uint32_t bar = cut ? tail : kv_full + 8 * slot;
          if (lane == 0) {
            bar_expect(bar, TILE);
            for (int s = 0; s < NSUB; ++s)
              tma_3d(dst + s * SUB, is_v ? &mv : &mk, s * 64, cur.head, start + j * BM, bar);
          }
          if (cut) {  // zero the rows behind the sequence, then hand the tile over
            if (!warp_wait(tail, tph, stop)) break;
            tph ^= 1;
            uint8_t* v = smem + Cfg::KV_OFF + slot * TILE;
            for (int s = 0; s < NSUB; ++s)
              for (int x = left * 8 + lane; x < BM * 8; x += 32)
                reinterpret_cast<uint4*>(v + s * SUB)[x] = make_uint4(0, 0, 0, 0);
            fence_async_smem();
            __syncwarp();
            if (lane == 0) bar_arrive(kv_full + 8 * slot);
          }
          if (++slot == SLOTS) {
            slot = 0;
            ph ^= 1;
          }
        }
        if (*stop) break;
      }
    } else if (warp == 8) {
      // ---- products ------------------------------------------------------------------
      constexpr uint32_t ID_S = idesc_f16(BM, BM, false), ID_O = idesc_f16(BM, D, true);
      int slot = 0;
      uint32_t ph = 0, qph = 0, pph = 0;
      bool ok = true;
      auto scores = [&](int t, int ks) {
        const uint32_t a = sb + Cfg::Q_OFF + t * TILE;
        const uint32_t b = uniform(sb + Cfg::KV_OFF + ks * TILE);
        if (elect()) {
#pragma unroll
          for (int k = 0; k < D / 16; ++k) {
            const uint32_t off = (k / 4) * SUB + (k % 4) * 32;
            mma_ss(tm + t * BM, desc_sw128(a + off, 16, 1024), desc_sw128(b + off, 16, 1024), ID_S,
                   k > 0);
          }
          mma_commit(s_full + 8 * t);
        }
        __syncwarp();
      };
      auto values = [&](int t, int vs, bool first) {
        const uint32_t b = uniform(sb + Cfg::KV_OFF + vs * TILE);
        const bool acc = uniform(!first);
        if (elect()) {
#pragma unroll
          for (int k = 0; k < BM / 16; ++k)
            mma_ts(tm + 256 + t * D, tm + t * BM + k * 8, desc_sw128(b + k * 2048, SUB, 1024), ID_O,
                   acc || k > 0);
          mma_commit(o_done + 8 * t);
        }
        __syncwarp();
      };
      auto release = [&](uint32_t bar) {
        if (elect()) mma_commit(bar);
        __syncwarp();
      };
      auto wait_tile = [&]() {  // the ring's next tile; returns its slot
        ok = ok && warp_wait(kv_full + 8 * slot, ph, stop);
        const int at = slot;
        if (++slot == SLOTS) {
          slot = 0;
          ph ^= 1;
        }
        return at;
      };
      while (ok && cur.next(A, tb)) {
        int nk[2] = {0, 0};
        for (int t = 0; t < 2; ++t) {
          int mt, h;
          if (cur.tile(A, tb, t, mt, h)) nk[t] = mt + 1;
        }
        const int n = max(nk[0], nk[1]);
        if (n == 0) continue;
        int ks = wait_tile();
        for (int t = 0; t < 2 && ok; ++t) {
          if (!nk[t]) continue;
          ok = warp_wait(q_full + 8 * t, (qph >> t) & 1, stop);
          qph ^= 1u << t;
          fence_after();
          if (!ok) break;
          scores(t, ks);
          if (nk[t] == 1) release(q_empty + 8 * t);
        }
        if (!ok) break;
        release(kv_empty + 8 * ks);
        for (int j = 0; j < n && ok; ++j) {
          const int vs = wait_tile();
          if (j + 1 < n) ks = wait_tile();
          for (int t = 0; t < 2 && ok; ++t) {
            if (j >= nk[t]) continue;
            ok = warp_wait(p_full + 8 * t, (pph >> t) & 1, stop);
            if (!ok) break;
            pph ^= 1u << t;
            fence_after();
            values(t, vs, j == 0);
            if (j + 1 < nk[t]) {
              scores(t, ks);
              if (j + 2 == nk[t]) release(q_empty + 8 * t);
            }
          }
          if (!ok) break;
          release(kv_empty + 8 * vs);
          if (j + 1 < n) release(kv_empty + 8 * ks);
        }
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
    Cursor cur;
    cur.init(A, tb);
    // ---- softmax: thread = row -------------------------------------------------------
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t ts = tm + lanes + t * BM, to = tm + lanes + 256 + t * D;
    uint32_t sph = 0, oph = 0;
    constexpr float SLACK = 8.f, BOOST = 7.f;
    while (cur.next(A, tb)) {
      int mt, h;
      if (!cur.tile(A, tb, t, mt, h)) continue;
      const int nk = mt + 1;
      float xref = 0.f;  // the score that the reference m = sigma log2(e) xref goes by
      uint64_t l2 = pack2(0.f, 0.f);
      bool ok = !*stop;
      for (int j = 0; j < nk && ok; ++j) {
        ok = warp_wait(s_full + 8 * t, sph, stop);
        if (!ok) break;
        sph ^= 1;
        fence_after();
        uint32_t s[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(ts + 32 * c, s + 32 * c);
        tmem_wait_ld();
        float* x = reinterpret_cast<float*>(s);
        if (j == nk - 1) {  // the diagonal tile
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c > row) x[c] = -CUDART_INF_F;
        }
        float mx[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8)
#pragma unroll
          for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], fmaxf(x[c + 2 * u], x[c + 2 * u + 1]));
#pragma unroll
        for (int u = 0; u < 4; ++u) mx[u] = fmaxf(mx[u], x[124 + u]);
        const float xnew = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool move = (xnew - xref) * A.sl > SLACK;
        if (j == 0) {
          xref = xnew;
        } else if (__any_sync(0xffffffffu, move)) {
          // O holds the products up to tile j - 1: wait for them, rescale this row
          const float f = move ? ex2((xref - xnew) * A.sl) : 1.f;
          if (move) xref = xnew;
          ok = warp_wait(o_done + 8 * t, oph ^ 1, stop);
          if (!ok) break;
          fence_after();
          l2 = fma2(l2, pack2(f, f), pack2(0.f, 0.f));
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t r[32];
            tmem_ld32(to + 32 * c, r);
            tmem_wait_ld();
#pragma unroll
            for (int u = 0; u < 32; ++u) r[u] = __float_as_uint(__uint_as_float(r[u]) * f);
            tmem_st32(to + 32 * c, r);
          }
        }
        // Past 2^22 the rounding of m would show in the exponent (at 2^27 as infinite
        // probabilities): the differences are taken before the scale then.
        float off = BOOST - xref * A.sl;
        if (__any_sync(0xffffffffu, fabsf(xref * A.sl) >= 0x1p22f)) {
#pragma unroll
          for (int c = 0; c < 128; ++c) x[c] -= xref;
          off = BOOST;
        }
        const uint64_t sl2 = pack2(A.sl, A.sl), mm = pack2(off, off);
        uint32_t p[64];
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          float a, b;
          unpack2(fma2(pack2(x[2 * c], x[2 * c + 1]), sl2, mm), a, b);
          a = ex2(a);
          b = ex2(b);
          l2 = add2(l2, pack2(a, b));
          const __half2 hh = __floats2half2_rn(a, b);
          p[c] = *reinterpret_cast<const uint32_t*>(&hh);
        }
        tmem_st32(ts, p);
        tmem_st32(ts + 32, p + 32);
        tmem_wait_st();
        fence_before();
        __syncwarp();
        if (lane == 0) bar_arrive(p_full + 8 * t);
        oph ^= 1;  // the phase that this tile's product completes, inverted
      }
      // O / l; NaN if a wait gave up
      if (ok) ok = warp_wait(o_done + 8 * t, oph ^ 1, stop);
      fence_after();
      const int i = mt * BM + row;
      float la, lb;
      unpack2(l2, la, lb);
      const float inv = ok ? 1.f / (la + lb) : CUDART_NAN_F;
      const bool mine = i < tb.len[cur.z];
      __half* dst = A.o + (int64_t)(tb.start[cur.z] + (mine ? i : 0)) * A.os + (size_t)h * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t r[32];
        tmem_ld32(to + 32 * c, r);
        tmem_wait_ld();
        if (mine) {
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const __half2 hh = __floats2half2_rn(__uint_as_float(r[8 * u + 2 * k]) * inv,
                                                   __uint_as_float(r[8 * u + 2 * k + 1]) * inv);
              w[k] = *reinterpret_cast<const uint32_t*>(&hh);
            }
            *reinterpret_cast<uint4*>(dst + 32 * c + 8 * u) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      fence_before();
    }
  }
  __syncthreads();
  if (warp == 8) {
    fence_after();
    if (*stop)  // let copies and products still in flight land
      for (int i = 0; i < 2000; ++i) __nanosleep(1000);
    tmem_free(tm, 512);
  }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &r) != cudaSuccess ||
        r != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      p = nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// [tokens][heads][d] fp16 in boxes of 64 channels x 128 tokens of one head.
bool make_map(CUtensorMap* m, const void* p, int d, int heads, int64_t tokens, int64_t stride) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, BM}, el[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(p), dims, strides, box, el,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch_prompt(PromptArgs A, int n_seqs, int num_sm, const CUtensorMap& mq,
                          const CUtensorMap& mk, const CUtensorMap& mv, cudaStream_t s) {
  cudaError_t e = smem_once<prompt_kernel<D>, PCfg<D>::SMEM>();
  const int32_t* cu = A.cu;
  for (int z = 0; z < n_seqs && e == cudaSuccess; z += MAX_SEQS) {
    A.cu = cu + z;
    A.n_seqs = n_seqs - z < MAX_SEQS ? n_seqs - z : MAX_SEQS;
    // Most row tiles that the sequences can have (their lengths are on the device).
    const int64_t tiles = ((int64_t)A.total / BM + A.n_seqs) * A.Hq;
    A.per = tiles <= num_sm ? 1 : 2;
    const int64_t items = (tiles + A.per - 1) / A.per;
    const int grid = items < num_sm ? (int)items : num_sm;
    prompt_kernel<D><<<grid, PT, PCfg<D>::SMEM, s>>>(A, mq, mk, mv);
    e = cudaGetLastError();
  }
  return e;
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
      total_tokens < 0 || n_seqs < 0 || !(softmax_scale >= 0.f) || softmax_scale > 0x1p127f)
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
  const int64_t far = (int64_t)1 << 38;  // a tensor map's stride is below 2^40 bytes
  if (q_stride > far || k_stride > far || v_stride > far) return EKV_EINVAL;
  PromptArgs A = {};
  A.cu = cu_seqlens;
  A.total = total_tokens;
  A.Hq = n_q_heads;
  A.Hkv = n_kv_heads;
  A.G = n_q_heads / n_kv_heads;
  A.unit = A.G & 1 ? 2 : 1;
  const float scale = softmax_scale > 0.f ? softmax_scale : 1.0f / sqrtf((float)head_dim);
  A.sl = scale * 1.4426950408889634f;
  A.o = static_cast<__half*>(o);
  A.os = o_stride;
  const int num_sm = sm_count();
  if (num_sm <= 0) {
    cudaGetLastError();
    return EKV_ECUDA;
  }
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, q, head_dim, n_q_heads, total_tokens, q_stride) ||
      !make_map(&mk, k, head_dim, n_kv_heads, total_tokens, k_stride) ||
      !make_map(&mv, v, head_dim, n_kv_heads, total_tokens, v_stride))
    return EKV_ECUDA;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = head_dim == 64 ? launch_prompt<64>(A, n_seqs, num_sm, mq, mk, mv, s)
                                       : launch_prompt<128>(A, n_seqs, num_sm, mq, mk, mv, s);
  return e == cudaSuccess ? EKV_OK : EKV_ECUDA;
}
