// ekv_tree.cu — attention of a tree of drafted tokens over the quantized paged cache.
//
// Every node i of a sequence's drafted tree (fp16 q, k, v of its own; parent
// parents[i] < i, -1 = none) attends over every cached token of the sequence, read
// from the mixed-format pages and the open block's staging rows as decode attention
// reads them, and over itself and its ancestors among the drafted nodes:
//   o_ih = sum_{t cached} p_t vhat_t + sum_{a in anc(i)} p_a v_a,
//   p = softmax over both of sigma q_ih . khat_t and sigma q_ih . k_a.
//
// The rows of one (sequence, KV head) are its nodes times the G query heads of the group
// (1 to 512), so each page is worth 16 keys to all of them: it is read from memory and
// unpacked once, and the products go to tcgen05 with 128 rows as M.  Tokens are taken in
// tiles of 64 (4 pages); the drafted nodes are one more tile of raw fp16 rows.  Roles:
//   warp 17      page copies (cp.async.bulk) into a ring of raw tiles
//   warps 8-15   unpack a raw tile into swizzled fp16 operand tiles, a page's K or V a warp
//                (K on schedulers 0 and 1, V on 2 and 3: less code for each): K as hi + lo
//                (khat = code * scale = hi + lo exactly, two products; 2- and 16-bit K need
//                hi alone; asymmetric: hi + lo = code * scale + zero point to 22 bits), V as
//                the bare codes (exact in fp16)
//   warp 18      the V scales of a tile, for softmax
//   warps 16, 19 tcgen05.mma: S = Q K^T with Q in tensor memory, and O += P V (a warp each:
//                their waits in one loop took longer than the products)
//   warps 0-3, 4-7  softmax, one row a thread; the two groups take the even and the odd
//                token tiles of a pair, for the same rows.  Scores run up to two pairs ahead
//                (four score buffers in tensor memory), with one accumulator and one running
//                reference for both groups: before the exponentials of a pair a barrier with
//                an OR over the 256 threads tells whether any row's reference has to move,
//                which is seldom.
//
// What bounds it is instruction issue: a 64-token tile takes about 4,400 warp instructions
// (K 1,000, V 500, softmax 1,200 at 128 rows, the rest waits and bookkeeping of the roles)
// at 0.58 a cycle and scheduler, while the tensor cores are busy 40% of the time and DRAM
// 18%.  Measured at 131,072 tokens, 8 KV heads, 128 rows, 4-bit K and V: 121 us with the
// merging kernel (154 MB: 1.27 TB/s); asymmetric 164, 16-bit K and V 130 (537 MB: 4.1 TB/s),
// head size 64 105.  Tried and slower (against 119): 16 unpacking warps (128 us: more
// waits to issue), half a page a warp (136), unrolled unpacking or softmax loops (121, 124:
// the code of 20 warps in different roles outgrows the instruction caches; the stall for
// instructions was the largest of all until the loops were short), V scales read by each
// softmax thread from shared memory (140), polling waits without a suspend hint (203).
//
// A token's V scale s multiplies its probability: P' = 2^(x + log2 s - m) in fp16, where
// the reference m follows the largest x + log2 s, so the fp16 range goes to what the cached
// tokens add to the output, whatever their scales; the row sum adds P' / s in fp32.  The
// drafts' raw rows have s = 1, which may be far above the others': their tile, the last, is
// alone in its pair, so a reference that they raise rescales the accumulator in fp32 and
// takes no bits from any cached token's P'.  The log2 s come with the scores: 16 more
// channels of K hold log2 s / (sigma log2 e) as three fp16 parts, against a constant in Q
// (each softmax thread loading 64 of them twice from shared memory took longer than the
// exponentials).  As in prompt attention m moves only for a gain above 2^8, P' carries
// 2^7, and P' is the one value rounded to fp16.
//
// Work split: the token tiles of all (sequence, KV head, row tile) units laid end to end,
// cut into equal runs, one per CTA (one CTA an SM); a run may hold parts of several
// units.  A unit cut by run ends leaves fp32 partials (numerator, max, sum) in
// the scratch, and a second small kernel merges them by log-sum-exp.  The cut depends on
// the lengths only, so equal calls give equal bits.
#include <math_constants.h>

#include "ekv_internal.h"
#include "ekv_tc.cuh"

namespace ekv {
namespace {

using namespace tc;

constexpr int TM_ROWS = 128;      // rows of a row tile
constexpr int TN = 64;            // tokens of a token tile
constexpr int TPAGES = TN / BLOCK;
constexpr int TT = 640;           // threads (96 registers each)
constexpr int W_SCORES = 16, W_PAGES = 17, W_SCALES = 18, W_VALUES = 19;  // single-warp roles
constexpr int TSEQS = 256;        // sequences of one launch
constexpr int KST = 2;            // K operand tiles in flight (each free once its scores are)
constexpr int VST = 4;            // V operand tiles in flight (until their products are done)
constexpr int RAW_BYTES = 64 * 1024;
constexpr int RAW_MAX = 8;        // raw tiles in flight at most

template <int D>
struct TCfg {
  static constexpr int SUBT = TN * 128;              // 64 channels of a tile
  static constexpr int OPND = D / 64 * SUBT;         // one operand tile
  static constexpr int KSTAGE = 2 * OPND + SUBT;     // hi, lo, 16 more channels
  static constexpr int V_OFF = KST * KSTAGE;
  static constexpr int RAW_OFF = V_OFF + VST * OPND;
  static constexpr int MISC_OFF = RAW_OFF + RAW_BYTES;
};

// Runs of equal length: run c starts at total * c / grid = quot * c + rest * c / grid.
struct Runs {
  int64_t quot;
  int rest, grid;
  __device__ void init(int64_t total, int g) {
    grid = g;
    quot = total / g;
    rest = (int)(total - quot * g);
  }
  __device__ int64_t start(int c) const { return quot * c + rest * c / grid; }
};
// Raw tiles in flight for pages of `room` bytes.  (The drafts' tile takes a slot too,
// without copies.)
__device__ __forceinline__ int raw_tiles(int room) {
  return min(RAW_MAX, RAW_BYTES / (TPAGES * room));
}

// A segment: the token tiles s .. e-1 of one unit.
struct TMisc;
struct Seg {
  int z, h, row0, s, e, nt, len, cnt;
  int slot;  // of its partial
  __device__ bool whole() const { return s == 0 && e == nt; }
  // Tiles left out at the start of the first pair (0 or 1), so that the drafts' tile is alone in
  // its pair.
  __device__ int skip() const { return e == nt && !((e - s) & 1); }
  // Tokens of page pg of tile i (its raw tile in slot rs).
  __device__ int tokens(int i, const TMisc& M, int rs, int pg) const;
};

// Walks a CTA's segments in order.  Every warp has a walk of its own in shared memory, so
// that the (long) step is one out-of-line function and takes no registers of the roles.
struct Walk {
  int64_t lo, hi, a;  // run, offset of the next unit
  int z, unit, nunits, nt, len, cnt;
  Seg seg;
};

struct TMisc {
  int64_t pre[TSEQS + 1];       // tiles of the sequences before
  int32_t len[TSEQS];           // cached tokens
  int32_t slot[TSEQS];
  uint8_t cnt[TSEQS];           // nodes
  unsigned long long anc[2][64];  // ancestors-or-self of each node, by segment parity
  // of each token's V scale s: 1 / s and (asymmetric) the zero point over s
  alignas(16) float rsv[VST][TN];
  alignas(16) float zsv[VST][TN];
  alignas(8) uint16_t valid[VST][TPAGES];  // tokens that are there
  int32_t has_lo[KST];
  alignas(16) int32_t ent[RAW_MAX][TPAGES];  // page-table entries of a raw tile
  int32_t raw_lo[RAW_MAX];                   // whether its K needs the lo products
  float mx[2][TM_ROWS];         // row maxima of the two groups
  float lz[2][2][TM_ROWS];      // their row sums and zero-point sums
  alignas(8) uint64_t bars[2 * KST + 3 * VST + 2 * RAW_MAX + 1 + 4 + 4 + 2];
  Runs runs;
  Walk walk[TT / 32];
  int stop;
  uint32_t tmem;
};

struct TreeArgs {
  int layer, vb, m, n_seqs;
  const int32_t *slots, *n_nodes, *parents;
  const __half *q, *k, *v;
  __half* o;
  float* acc;       // [2 grid][D / 4][128] float4
  float2* ml;       // [2 grid][128] (reference score, sum)
  int64_t* pre;     // for the merging kernel: [n_seqs + 1], then the runs' starts [grid + 1]
  int grid;
  float q_ext, k_ext;  // Q's constant c for the log2 s channels, and 1 / (sl c)
};

__host__ __device__ inline int rows_of(int cnt, int G) { return cnt * G; }
__host__ __device__ inline int row_tiles(int rows) { return (rows + TM_ROWS - 1) / TM_ROWS; }
__host__ __device__ inline int tiles_of(int len) { return (len + TN - 1) / TN + 1; }  // + drafts
__host__ __device__ inline int64_t seq_tiles(int len, int cnt, int G, int Hkv) {
  const int r = rows_of(cnt, G);
  return cnt > 0 ? (int64_t)Hkv * row_tiles(r) * tiles_of(len) : 0;
}
// Tiles of a unit of nt tiles at offset a that lie in the run [lo, hi).
__host__ __device__ inline void unit_part(int64_t a, int nt, int64_t lo, int64_t hi, int& s,
                                          int& e) {
  const int64_t x = lo > a ? lo - a : 0, y = hi > a ? hi - a : 0;
  s = (int)(x < nt ? x : nt);
  e = (int)(y < nt ? y : nt);
}

__device__ __forceinline__ int Seg::tokens(int i, const TMisc& M, int rs, int pg) const {
  if (i == nt - 1) return min(BLOCK, max(0, cnt - BLOCK * pg));
  return M.ent[rs][pg] == -1 ? 0 : max(0, min(BLOCK, len - (i * TPAGES + pg) * BLOCK));
}

// First step: the sequence that holds the run's start.
__device__ __noinline__ void walk_init(Walk* w, const TMisc& M, int n_seqs) {
  w->lo = M.runs.start(blockIdx.x);
  w->hi = M.runs.start(blockIdx.x + 1);
  int p = 0, q = n_seqs;  // the last sequence that starts at or before the run
  while (q - p > 1) {
    const int mid = (p + q) / 2;
    if (M.pre[mid] <= w->lo) p = mid;
    else q = mid;
  }
  w->z = p - 1;
  w->unit = w->nunits = 0;
}
// Step to the next segment (false: none).
__device__ __noinline__ bool walk_step(Walk* at, const TMisc& M, int n_seqs, int G, int Hkv) {
  Walk v = *at;
  Walk* const w = &v;
  while (true) {
    if (w->unit >= w->nunits) {
      const int z = ++w->z;
      if (z >= n_seqs || M.pre[z] >= w->hi) break;
      w->len = M.len[z];
      w->cnt = M.cnt[z];
      const int r = rows_of(w->cnt, G);
      w->nunits = w->cnt > 0 ? Hkv * row_tiles(r) : 0;
      w->nt = tiles_of(w->len);
      w->a = M.pre[z];
      w->unit = 0;
      if (w->nunits && w->lo > w->a) {  // skip the units before the run
        const int64_t d = w->lo - w->a;
        const int64_t skip = d >> 31 ? d / w->nt : (uint32_t)d / (uint32_t)w->nt;
        w->unit = (int)(skip < w->nunits ? skip : w->nunits);
        w->a += (int64_t)w->unit * w->nt;
      }
      continue;
    }
    const int64_t a = w->a;
    if (a >= w->hi) break;
    Seg& g = w->seg;
    unit_part(a, w->nt, w->lo, w->hi, g.s, g.e);
    const int nr = row_tiles(rows_of(w->cnt, G));
    g.z = w->z;
    g.h = w->unit / nr;
    g.row0 = w->unit % nr * TM_ROWS;
    g.nt = w->nt;
    g.len = w->len;
    g.cnt = w->cnt;
    g.slot = 2 * blockIdx.x + (w->lo > a ? 0 : 1);
    w->a = a + w->nt;
    ++w->unit;
    if (g.s < g.e) {
      *at = v;
      return true;
    }
  }
  return false;
}
// By a whole warp: its next segment.
__device__ __forceinline__ bool next_seg(Walk* wk, const TMisc& M, const TreeArgs& A,
                                         const DevState& st, int lane, Seg& w) {
  int more = 0;
  if (lane == 0) more = walk_step(wk, M, A.n_seqs, st.G, st.Hkv);
  more = __shfl_sync(0xffffffffu, more, 0);
  __syncwarp();
  w = wk->seg;
  __syncwarp();
  return more != 0;
}

// ---- unpacking: 8 channels (group g) of one row as 4 words, in the order
// (0,4) (1,5) (2,6) (3,7), which 4-bit words unpack to with one AND-OR a pair.  Q is
// permuted the same way when it is loaded and O back when it is written. --------------
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hsub(uint32_t a, uint32_t b) {
  const __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hfma(uint32_t a, uint32_t b, uint32_t c) {
  const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b),
                            *reinterpret_cast<__half2*>(&c));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmul(uint32_t a, uint32_t b) {
  const __half2 r = __hmul2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hfms(uint32_t a, uint32_t b, uint32_t c) {  // a b - c
  const __half2 r = __hfma2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b),
                            __hneg2(*reinterpret_cast<__half2*>(&c)));
  return *reinterpret_cast<const uint32_t*>(&r);
}
__device__ __forceinline__ uint32_t hmin(uint32_t a, uint32_t b) {
  const __half2 r = __hmin2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// (a, b) as fp16, the largest finite value instead of infinity.
__device__ __forceinline__ uint32_t pack_finite(float a, float b) {
  uint32_t d;
  asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
  return d;
}
__device__ __forceinline__ void perm8(const uint4& u, uint32_t* w) {
  w[0] = __byte_perm(u.x, u.z, 0x5410);
  w[1] = __byte_perm(u.x, u.z, 0x7632);
  w[2] = __byte_perm(u.y, u.w, 0x5410);
  w[3] = __byte_perm(u.y, u.w, 0x7632);
}

constexpr uint32_t MAGIC = 0x64006400u;   // fp16 1024, 1024
// fp16 constants (both halves): 1024 + offset of the code width, and the same over the
// power of two that a code's position in the word multiplies it by.
__device__ __forceinline__ constexpr uint32_t both(uint32_t h) { return h | h << 16; }

// A row's 8 codes of group g as stored (raw fp16 for B = 16), and what they unpack to:
// signed codes q for the symmetric quantizer, unsigned u for the other.
template <int B>
struct Raw8 {
  uint32_t x[B == 16 ? 4 : B == 8 ? 2 : 1];
  __device__ __forceinline__ void load(const uint8_t* row, int g) {
    if constexpr (B == 16) {
      const uint4 u = *reinterpret_cast<const uint4*>(row + 16 * g);
      x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w;
    } else if constexpr (B == 8) {
      const uint2 u = *reinterpret_cast<const uint2*>(row + 8 * g);
      x[0] = u.x; x[1] = u.y;
    } else if constexpr (B == 4) {
      x[0] = *reinterpret_cast<const uint32_t*>(row + 4 * g);
    } else {
      x[0] = *reinterpret_cast<const uint16_t*>(row + 2 * g);
    }
  }
};
template <int B, bool ASYM>
__device__ __forceinline__ void unpack8w(const Raw8<B>& c, uint32_t* w) {
  if constexpr (B == 16) {
    perm8(make_uint4(c.x[0], c.x[1], c.x[2], c.x[3]), w);
  } else if constexpr (B == 8) {
    const uint32_t y0 = __byte_perm(c.x[0], c.x[1], 0x5140);
    const uint32_t y1 = __byte_perm(c.x[0], c.x[1], 0x7362);
    const uint32_t sub = both(ASYM ? 0x6400 : 0x6480);  // 1024 or 1152
    w[0] = hsub(__byte_perm(y0, 0x64646464u, 0x4140), sub);
    w[1] = hsub(__byte_perm(y0, 0x64646464u, 0x4342), sub);
    w[2] = hsub(__byte_perm(y1, 0x64646464u, 0x4140), sub);
    w[3] = hsub(__byte_perm(y1, 0x64646464u, 0x4342), sub);
  } else if constexpr (B == 4) {
    const uint32_t r = c.x[0], r8 = r >> 8;
    const uint32_t lo = both(ASYM ? 0x6400 : 0x6408);   // 1024 or 1032
    const uint32_t hi = both(ASYM ? 0xD400 : 0xD480);   // -64 or -72
    const uint32_t q16 = both(0x2C00);                  // 1/16
    w[0] = hsub(and_or(r, 0x000F000Fu, MAGIC), lo);
    w[1] = hfma(and_or(r, 0x00F000F0u, MAGIC), q16, hi);
    w[2] = hsub(and_or(r8, 0x000F000Fu, MAGIC), lo);
    w[3] = hfma(and_or(r8, 0x00F000F0u, MAGIC), q16, hi);
  } else {
    const uint32_t x = __byte_perm(c.x[0], 0, 0x4140);
    w[0] = hsub(and_or(x, 0x00030003u, MAGIC), both(ASYM ? 0x6400 : 0x6402));
    w[1] = hfma(and_or(x, 0x000C000Cu, MAGIC), both(0x3400), both(ASYM ? 0xDC00 : 0xDC08));
    w[2] = hfma(and_or(x, 0x00300030u, MAGIC), both(0x2C00), both(ASYM ? 0xD400 : 0xD420));
    w[3] = hfma(and_or(x, 0x00C000C0u, MAGIC), both(0x2400), both(ASYM ? 0xCC00 : 0xCC80));
  }
}
// Per-channel fp16 values (scales or zero points) of group g in the same order.
template <int B>
__device__ __forceinline__ void channel8(const uint8_t* arr, int g, uint32_t* w) {
  if constexpr (B == 8) {
    perm8(*reinterpret_cast<const uint4*>(arr + 16 * g), w);
  } else if constexpr (B == 4) {
    const uint4 u = *reinterpret_cast<const uint4*>(arr + 16 * g);
    w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
  } else {  // word j of 16 channels holds channels j and j + 8
    const uint4 a = *reinterpret_cast<const uint4*>(arr + 32 * (g >> 1));
    const uint4 b = *reinterpret_cast<const uint4*>(arr + 32 * (g >> 1) + 16);
    const uint32_t sel = g & 1 ? 0x7632u : 0x5410u;
    w[0] = __byte_perm(a.x, b.x, sel);
    w[1] = __byte_perm(a.y, b.y, sel);
    w[2] = __byte_perm(a.z, b.z, sel);
    w[3] = __byte_perm(a.w, b.w, sel);
  }
}

// A warp unpacks one page: lane (g, t0) takes group g of rows t0, t0 + STEP, ...; OFF[i] is
// where its i-th 16-byte chunk goes in the operand tile (swizzled: chunk g of row r sits at
// (g mod 8) xor (r mod 8); every 8 rows the pattern repeats 1024 bytes on).
template <int D>
struct Lane {
  static constexpr int GR = D / 8, STEP = 32 / GR;
  int g, t0;
  uint32_t off[4];
  __device__ Lane(int lane) : g(lane % GR), t0(lane / GR) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = t0 + i * STEP;
      off[i] = (g >> 3) * TCfg<D>::SUBT + row * 128 + (((g & 7) ^ (row & 7)) << 4);
    }
  }
};

// K rows at kp into dst (hi) and dst + OPND (lo).  FULL: all 16 rows hold tokens; else rows
// from n on are left as they are.  `lo`: the tile's lo part is used (zero it where this
// page needs none).
template <int D, int KB, bool ASYM, bool FULL>
__device__ __forceinline__ void unpack_k(const uint8_t* kp, int64_t stride, int n, uint8_t* dst,
                                         bool lo, const Lane<D>& ln) {
  constexpr int STEP = Lane<D>::STEP;
  constexpr int R = KB < 8 && !ASYM ? 4 : 2;  // rows at once
  constexpr bool HAS_LO = KB < 16 && (ASYM || KB > 2);
  // A scale rounds up in fp16, so the largest code times it may pass fp16's range (127 * 516,
  // 7 * 9360 for entries of 65504).  hi is formed with the scale cut to where it cannot
  // (515.5, 9352); lo = code * scale - hi stays exact: a small multiple of the scale's step.
  constexpr uint32_t TOP = both(KB == 8 ? 0x6007 : 0x7091);
  uint32_t sc[4], top[4], zp[4];
  if constexpr (KB < 16) {
    channel8<KB>(kp + BLOCK * D * KB / 8, ln.g, sc);
#pragma unroll
    for (int x = 0; x < 4; ++x) top[x] = KB > 2 && !ASYM ? hmin(sc[x], TOP) : sc[x];
    if constexpr (ASYM) channel8<KB>(kp + BLOCK * D * KB / 8 + 2 * D, ln.g, zp);
  }
#pragma unroll 1
  for (int c = 0; c < BLOCK; c += 4 * STEP) {
    const uint8_t* row = kp + (c + ln.t0) * stride;
    uint8_t* out = dst + c * 128;
#pragma unroll
    for (int j = 0; j < 4; j += R) {
      Raw8<KB> raw[R];
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (FULL || c + ln.t0 + (j + i) * STEP < n)
          raw[i].load(row + (j + i) * STEP * stride, ln.g);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        if (!FULL && c + ln.t0 + (j + i) * STEP >= n) continue;
        uint32_t w[4], l[4] = {0, 0, 0, 0};
        unpack8w<KB, ASYM>(raw[i], w);
        if constexpr (KB < 16 && !ASYM) {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t p = hmul(w[x], top[x]);
            if constexpr (KB > 2) l[x] = hfms(w[x], sc[x], p);  // the exact residual
            w[x] = p;
          }
        } else if constexpr (KB < 16) {  // u s + z in fp32, then hi + lo
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const float2 u = __half22float2(*reinterpret_cast<__half2*>(&w[x]));
            const float2 s = __half22float2(*reinterpret_cast<__half2*>(&sc[x]));
            const float2 z = __half22float2(*reinterpret_cast<__half2*>(&zp[x]));
            const float a = fmaf(u.x, s.x, z.x), b = fmaf(u.y, s.y, z.y);
            w[x] = pack_finite(a, b);  // (u s + z may pass fp16's range as well)
            const float2 pf = __half22float2(*reinterpret_cast<__half2*>(&w[x]));
            const __half2 r = __floats2half2_rn(a - pf.x, b - pf.y);
            l[x] = *reinterpret_cast<const uint32_t*>(&r);
          }
        }
        uint8_t* at = out + ln.off[j + i];
        *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
        if (HAS_LO || lo)
          *reinterpret_cast<uint4*>(at + TCfg<D>::OPND) = make_uint4(l[0], l[1], l[2], l[3]);
      }
    }
  }
}
// V rows at vp into dst; rows from n on become zero.  Codes are signed for both
// quantizers: u s + z = (u - 2^(b-1)) s + (z + 2^(b-1) s), so that the products P' q stay
// as small as the values.
template <int D, int VB, bool FULL>
__device__ __forceinline__ void unpack_v(const uint8_t* vp, int64_t stride, int n, uint8_t* dst,
                                         const Lane<D>& ln) {
  constexpr int STEP = Lane<D>::STEP;
  constexpr int R = VB < 8 ? 4 : 2;
#pragma unroll 1
  for (int c = 0; c < BLOCK; c += 4 * STEP) {
    const uint8_t* row = vp + (c + ln.t0) * stride;
    uint8_t* out = dst + c * 128;
#pragma unroll
    for (int j = 0; j < 4; j += R) {
      Raw8<VB> raw[R];
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (FULL || c + ln.t0 + (j + i) * STEP < n)
          raw[i].load(row + (j + i) * STEP * stride, ln.g);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        uint32_t w[4] = {0, 0, 0, 0};
        if (FULL || c + ln.t0 + (j + i) * STEP < n) unpack8w<VB, false>(raw[i], w);
        *reinterpret_cast<uint4*>(out + ln.off[j + i]) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

// The loop of an unpacking warp: one page of every tile, its K or its V part.
template <int D, bool ASYM, bool IS_K>
__device__ __forceinline__ void unpack_role(const DevState& st, const TreeArgs& A, uint8_t* smem,
                                            TMisc& M, uint32_t out_full, uint32_t out_empty,
                                            uint32_t raw_full, int warp, int lane) {
  using Cfg = TCfg<D>;
  const uint32_t raw_empty = raw_full + 8 * RAW_MAX;
  volatile int* stop = &M.stop;
  Seg w;
  const int kmax = max(2, st.kmax[A.layer]);
  const int page_room = (page_bytes(kmax, A.vb, D, ASYM) + 127) & ~127;
  const int nraw = raw_tiles(page_room);
  const int pg = (warp & 1) + (warp >> 1 & 2);  // page of the tile
  const Lane<D> hf(lane);
  int rs = 0, sg = 0;
  uint32_t rph = 0, eph = 1;
  bool ok = true;
  while (ok && next_seg(&M.walk[warp], M, A, st, lane, w)) {
    for (int i = w.s; i < w.e; ++i) {
      const bool drafts = i == w.nt - 1;
      const int at = sg, raw = rs;
      ok = ok && warp_wait(out_empty + 8 * sg, eph, stop);
      ok = ok && warp_wait(raw_full + 8 * rs, rph, stop);
      if (!ok) break;
      if (++sg == (IS_K ? KST : VST)) {
        sg = 0;
        eph ^= 1;
      }
      if (++rs == nraw) {
        rs = 0;
        rph ^= 1;
      }
      uint8_t* dst = smem + pg * BLOCK * 128 +
                     (IS_K ? at * Cfg::KSTAGE : Cfg::V_OFF + at * Cfg::OPND);
      // Where the part's rows are and how many hold tokens: in the raw tile; the open
      // block's K in the staging rows and V in its page, in memory; the drafts as given.
      const int n = w.tokens(i, M, raw, pg);
      const int32_t e = drafts ? -1 : M.ent[raw][pg];
      const int kb = bits_of_code(entry_fmt(e) >> 2);
      if constexpr (IS_K) {
        const bool lo = !drafts && M.raw_lo[raw] != 0;
        if (pg == 0 && lane == 0) M.has_lo[at] = lo;
        if (n == BLOCK && !drafts) {
          const uint8_t* page = smem + Cfg::RAW_OFF + (raw * TPAGES + pg) * page_room;
          switch (kb) {
            case 2: unpack_k<D, 2, ASYM, true>(page, D / 4, n, dst, lo, hf); break;
            case 4: unpack_k<D, 4, ASYM, true>(page, D / 2, n, dst, lo, hf); break;
            case 8: unpack_k<D, 8, ASYM, true>(page, D, n, dst, lo, hf); break;
            default: unpack_k<D, 16, ASYM, true>(page, 2 * D, n, dst, lo, hf); break;
          }
        } else if (n > 0) {
          const __half* kp =
              drafts ? A.k + (((size_t)w.z * A.m + BLOCK * pg) * st.Hkv + w.h) * D
                     : st.staging + lsh_index(st, A.layer, M.slot[w.z], w.h) * (BLOCK * D);
          unpack_k<D, 16, ASYM, false>(reinterpret_cast<const uint8_t*>(kp),
                                       2 * D * (drafts ? (int64_t)st.Hkv : 1), n, dst, lo, hf);
        }
      } else {
        const int fmt = entry_fmt(e), v_off = k_part_bytes(kb, D, ASYM);
        if (n == BLOCK && !drafts) {
          const uint8_t* vp = smem + Cfg::RAW_OFF + (raw * TPAGES + pg) * page_room + v_off;
          switch (A.vb) {
            case 2: unpack_v<D, 2, true>(vp, D / 4, n, dst, hf); break;
            case 4: unpack_v<D, 4, true>(vp, D / 2, n, dst, hf); break;
            case 8: unpack_v<D, 8, true>(vp, D, n, dst, hf); break;
            default: unpack_v<D, 16, true>(vp, 2 * D, n, dst, hf); break;
          }
        } else if (drafts) {
          const __half* vp = A.v + (((size_t)w.z * A.m + BLOCK * pg) * st.Hkv + w.h) * D;
          unpack_v<D, 16, false>(reinterpret_cast<const uint8_t*>(vp), 2 * D * (int64_t)st.Hkv, n,
                                 dst, hf);
        } else {  // the open block, or no tokens (zeros)
          const uint8_t* vp =
              n > 0 ? st.pool_base[fmt] + v_off + (size_t)entry_idx(e) * st.pool_page_bytes[fmt]
                    : nullptr;
          switch (A.vb) {
            case 2: unpack_v<D, 2, false>(vp, D / 4, n, dst, hf); break;
            case 4: unpack_v<D, 4, false>(vp, D / 2, n, dst, hf); break;
            case 8: unpack_v<D, 8, false>(vp, D, n, dst, hf); break;
            default: unpack_v<D, 16, false>(vp, 2 * D, n, dst, hf); break;
          }
        }
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) {
        bar_arrive(out_full + 8 * at);
        bar_arrive(raw_empty + 8 * raw);
      }
    }
  }
}

// A warp's scores at ts become their differences from each row's xref (out of line: in the
// loop of the softmax, where it hardly ever runs, it costs 1.3 us a call at tree_chain).
__device__ __noinline__ void far_scores(uint32_t ts, float xref) {
#pragma unroll 1
  for (int c = 0; c < TN; c += 16) {
    uint32_t v[16];
    tmem_ld16(ts + c, v);
    tmem_wait_ld();
#pragma unroll
    for (int u = 0; u < 16; ++u) v[u] = __float_as_uint(__uint_as_float(v[u]) - xref);
    tmem_st16(ts + c, v);
  }
  tmem_wait_st();
}

template <int D, bool ASYM>
__global__ void __launch_bounds__(TT, 1) tree_kernel(DevState st, TreeArgs A) {
  using Cfg = TCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  TMisc& M = *reinterpret_cast<TMisc*>(smem + Cfg::MISC_OFF);
  const uint32_t sb = smem_u32(smem);
  const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
  const uint32_t b0 = smem_u32(M.bars);
  const uint32_t k_full = b0, k_empty = k_full + 8 * KST, v_full = k_empty + 8 * KST,
                 v_empty = v_full + 8 * VST, sc_full = v_empty + 8 * VST,
                 raw_full = sc_full + 8 * VST, raw_empty = raw_full + 8 * RAW_MAX,
                 q_full = raw_empty + 8 * RAW_MAX,
                 s_full = q_full + 8, p_full = s_full + 32, o_done = p_full + 32;
  volatile int* stop = &M.stop;

  for (int z = tid; z < A.n_seqs; z += TT) {
    const int slot = A.slots[z];
    const bool ok = slot >= 0 && slot < st.S;
    if (!ok && blockIdx.x == 0) set_error(st, EKV_EINVAL);
    const int cnt = A.n_nodes ? min(A.m, max(0, A.n_nodes[z])) : A.m;
    M.slot[z] = ok ? slot : 0;
    M.len[z] = ok ? st.len[ls_index(st, A.layer, slot)] : 0;
    M.cnt[z] = (uint8_t)cnt;
  }
  if (tid == 0) {
    for (int i = 0; i < KST; ++i) {
      bar_init(k_full + 8 * i, TPAGES + 1);
      bar_init(k_empty + 8 * i, 1);
    }
    for (int i = 0; i < VST; ++i) {
      bar_init(v_full + 8 * i, TPAGES);
      bar_init(v_empty + 8 * i, 1);
      bar_init(sc_full + 8 * i, 1);
    }
    for (int i = 0; i < RAW_MAX; ++i) {
      bar_init(raw_full + 8 * i, 1);
      bar_init(raw_empty + 8 * i, 2 * TPAGES + 1);
    }
    bar_init(q_full, 8);
    for (int i = 0; i < 4; ++i) {  // [buffer][group]
      bar_init(s_full + 8 * i, 1);
      bar_init(p_full + 8 * i, 4);
    }
    for (int i = 0; i < 2; ++i) bar_init(o_done + 8 * i, 1);
    M.stop = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  for (int i = tid; i < KST * Cfg::SUBT / 16; i += TT) {  // the 16 channels start as zeros
    const int x = i * 16 % Cfg::SUBT;
    *reinterpret_cast<uint4*>(smem + i * 16 / Cfg::SUBT * Cfg::KSTAGE + 2 * Cfg::OPND + x) =
        make_uint4(0, 0, 0, 0);
  }
  fence_async_smem();
  if (warp == W_SCORES) tmem_alloc(smem_u32(&M.tmem), 512);
  fence_before();
  __syncthreads();
  fence_after();
  // Columns: Q at 0 (D / 2) and 192 (8), O at 64 (D), score buffer b of group t at
  // 256 + 128 b + 64 t.
  const uint32_t tm = uniform(M.tmem);
  if (warp == 0) {             // prefix of the sequences' tiles
    int64_t run = 0;
    for (int z0 = 0; z0 < A.n_seqs; z0 += 32) {
      const int z = z0 + lane;
      const int64_t c = z < A.n_seqs ? seq_tiles(M.len[z], M.cnt[z], st.G, st.Hkv) : 0;
      int64_t x = c;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, off);
        if (lane >= off) x += y;
      }
      if (z < A.n_seqs) M.pre[z] = run + x - c;
      run += __shfl_sync(0xffffffffu, x, 31);
    }
    if (lane == 0) {
      M.pre[A.n_seqs] = run;
      M.runs.init(run, A.grid);
    }
    __syncwarp();
    __syncwarp();
    if (blockIdx.x == 0) {
      for (int z = lane; z <= A.n_seqs; z += 32) A.pre[z] = M.pre[z];
      for (int c = lane; c <= A.grid; c += 32) A.pre[A.n_seqs + 1 + c] = M.runs.start(c);
    }
  }
  __syncthreads();
  if (lane == 0) walk_init(&M.walk[warp], M, A.n_seqs);
  __syncwarp();

  if (warp >= W_SCORES) {
    Seg w;
    // Raw tile: 4 pages, each sized for the widest page the layer has admitted.
    const int kmax = max(2, st.kmax[A.layer]);
    const int page_room = (page_bytes(kmax, A.vb, D, ASYM) + 127) & ~127;
    const int nraw = raw_tiles(page_room);
    if (warp == W_PAGES) {
      // ---- page copies ---------------------------------------------------------------
      int rs = 0;
      uint32_t ph = 1;
      bool ok = true;
      while (ok && next_seg(&M.walk[warp], M, A, st, lane, w)) {
        const int32_t* bt = st.bt + lsh_index(st, A.layer, M.slot[w.z], w.h) * st.maxblk;
        const int nblk = (w.len + BLOCK - 1) / BLOCK, sealed = w.len / BLOCK;
        // (the drafts' tile, the last, has no pages: its blocks lie behind the table's use)
        int32_t ahead = -1;
        for (int i = w.s; i < w.e && ok; ++i) {
          const int k = (i - w.s) & 7;
          if (k == 0) {  // table entries of the next 8 tiles
            const int b = i * TPAGES + lane;
            ahead = b < nblk ? bt[b] : -1;
          }
          ok = warp_wait(raw_empty + 8 * rs, ph, stop);
          if (!ok) break;
          const int32_t e = __shfl_sync(0xffffffffu, ahead, k * TPAGES + (lane & 3));
          const int b = i * TPAGES + (lane & 3);
          uint32_t bytes = 0;
          if (lane < TPAGES && b < nblk) {
            if (e == -1) set_error(st, EKV_ESTATE);
            else if (b < sealed) bytes = (uint32_t)st.pool_page_bytes[entry_fmt(e)];
          }
          if (lane < TPAGES) M.ent[rs][lane] = b < nblk ? e : -1;
          const bool sealed_lo = lane < TPAGES && e != -1 && b < sealed &&
                                 (entry_fmt(e) >> 2) < 3 && (ASYM || (entry_fmt(e) >> 2) > 0);
          const bool lo = __any_sync(0xffffffffu, sealed_lo);
          if (lane == 0) M.raw_lo[rs] = lo;
          uint32_t all = bytes;
          all += __shfl_xor_sync(0xffffffffu, all, 1);
          all += __shfl_xor_sync(0xffffffffu, all, 2);
          __syncwarp();
          if (lane == 0) bar_expect(raw_full + 8 * rs, all);
          __syncwarp();
          if (bytes) {
            const int fmt = entry_fmt(e);
            const uint8_t* src = st.pool_base[fmt] + (size_t)entry_idx(e) * bytes;
            asm volatile(
                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], "
                "%2, [%3];" ::"r"(sb + Cfg::RAW_OFF + (rs * TPAGES + lane) * page_room),
                "l"(src), "r"(bytes), "r"(raw_full + 8 * rs)
                : "memory");
          }
          if (++rs == nraw) {
            rs = 0;
            ph ^= 1;
          }
        }
      }
    } else if (warp == W_SCORES) {
      // ---- scores of token tile x into buffer (x / 2) mod 2 of group x mod 2 -----------
      constexpr uint32_t ID_S = idesc_f16(TM_ROWS, TN, false);
      int sg = 0, buf = 0;
      uint32_t kph = 0, qph = 0, oph = 3;  // a buffer's first scores wait for no product
      bool ok = true;
      while (ok && next_seg(&M.walk[warp], M, A, st, lane, w)) {
        const int x0 = w.skip(), n = x0 + w.e - w.s;
        ok = warp_wait(q_full, qph, stop);
        qph ^= 1;
#pragma unroll 1
        for (int x = x0; x < n && ok; ++x) {
          const int t = x & 1;
          ok = warp_wait(k_full + 8 * sg, kph, stop);
          if (t == 0 || x == x0) {  // the buffer's last probabilities have been used
            ok = ok && warp_wait(o_done + 8 * buf, (oph >> buf) & 1, stop);
            oph ^= 1u << buf;
          }
          if (!ok) break;
          fence_after();
          const uint32_t base = uniform(sb + sg * Cfg::KSTAGE);
          const uint32_t d = uniform(tm + 256 + 128 * buf + 64 * t);
          // sub-tiles of 64 channels: those of hi, then those of lo
          const int subs = uniform((M.has_lo[sg] ? 2 : 1) * (D / 64));
          if (elect()) {
#pragma unroll 1
            for (int y = 0; y < subs; ++y)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ts(d, tm + (y & (D / 64 - 1)) * 32 + 8 * k,
                       desc_sw128(base + y * Cfg::SUBT + k * 32, 16, 1024), ID_S, y > 0 || k > 0);
            mma_ts(d, tm + 192, desc_sw128(base + 2 * Cfg::OPND, 16, 1024), ID_S, true);
            mma_commit(s_full + 16 * buf + 8 * t);
            mma_commit(k_empty + 8 * sg);
          }
          __syncwarp();
          if (++sg == KST) {
            sg = 0;
            kph ^= 1;
          }
          if (t == 1 || x == n - 1) buf ^= 1;
        }
      }
    } else if (warp == W_VALUES) {
      // ---- products of the probabilities with V ----------------------------------------
      constexpr uint32_t ID_O = idesc_f16(TM_ROWS, D, true);
      int sg = 0, buf = 0;
      uint32_t vph = 0, pph = 0;
      bool ok = true;
      while (ok && next_seg(&M.walk[warp], M, A, st, lane, w)) {
        const int x0 = w.skip(), n = x0 + w.e - w.s;
#pragma unroll 1
        for (int x = x0; x < n && ok; ++x) {
          const int t = x & 1, i = 2 * buf + t;
          ok = warp_wait(v_full + 8 * sg, vph, stop) &&
               warp_wait(p_full + 8 * i, (pph >> i) & 1, stop);
          pph ^= 1u << i;
          if (!ok) break;
          fence_after();
          const uint32_t base = uniform(sb + Cfg::V_OFF + sg * Cfg::OPND);
          const uint32_t p = uniform(tm + 256 + 128 * buf + 64 * t);
          const bool acc = uniform(x > x0), last = uniform(t == 1 || x == n - 1);
          if (elect()) {
#pragma unroll
            for (int k = 0; k < TN / 16; ++k)
              mma_ts(tm + 64, p + 8 * k, desc_sw128(base + k * 2048, Cfg::SUBT, 1024), ID_O,
                     acc || k > 0);
            mma_commit(v_empty + 8 * sg);
            if (last) mma_commit(o_done + 8 * buf);
          }
          __syncwarp();
          if (++sg == VST) {
            sg = 0;
            vph ^= 1;
          }
          if (last) buf ^= 1;
        }
      }
    } else if (warp == W_SCALES) {
      // ---- V scales and which tokens there are, two tokens a lane -------------------
      int rs = 0, vs = 0, ks = 0;
      uint32_t rph = 0, eph = 1, kph = 1;
      bool ok = true;
      while (ok && next_seg(&M.walk[warp], M, A, st, lane, w)) {
        for (int i = w.s; i < w.e; ++i) {
          const bool drafts = i == w.nt - 1;
          ok = ok && warp_wait(raw_full + 8 * rs, rph, stop);
          ok = ok && warp_wait(k_empty + 8 * ks, kph, stop);
          ok = ok && warp_wait(v_empty + 8 * vs, eph, stop);
          if (!ok) break;
          const int n = drafts ? min(TN, w.cnt) : min(TN, w.len - i * TN);  // tokens of the tile
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const int tok = lane + 32 * u, pg = tok / BLOCK, r = tok % BLOCK;
            float s = 1.f, zv = 0.f;
            bool there = tok < n;
            if (!drafts) {
              const int32_t e = M.ent[rs][pg];
              there = there && e != -1;
              if (there && A.vb < 16) {
                const int fmt = entry_fmt(e);
                const int off =
                    k_part_bytes(bits_of_code(fmt >> 2), D, ASYM) + BLOCK * D * A.vb / 8;
                const __half* sp;
                if ((pg + 1) * BLOCK <= n)
                  sp = reinterpret_cast<const __half*>(smem + Cfg::RAW_OFF + off +
                                                       (rs * TPAGES + pg) * page_room);
                else  // the open block
                  sp = reinterpret_cast<const __half*>(
                      st.pool_base[fmt] + off + (size_t)entry_idx(e) * st.pool_page_bytes[fmt]);
                // A row of scale 0 holds zero codes (symmetric: signed 0, so any scale does;
                // asymmetric: unsigned 0, -2^(b-1) once centred, which the zero point below
                // cancels at any scale).  The smallest fp16 leaves the least of a rounded
                // probability times that code, and does not raise the reference above the
                // other rows' scaled values.
                s = __half2float(sp[r]);
                if (s == 0.f) s = 0x1p-24f;
                if (ASYM)
                  zv = fmaf(s, (float)(1 << (A.vb - 1)), __half2float(sp[BLOCK + r]));
              }
            }
            const float inv = __fdividef(1.f, s), y = __log2f(s) * A.k_ext;
            M.rsv[vs][tok] = inv;
            if (ASYM) M.zsv[vs][tok] = zv * inv;
            // y in three fp16 parts: the first channels of the token's row (swizzled)
            const __half h0 = __float2half_rn(y);
            const float y1 = y - __half2float(h0);
            const __half h1 = __float2half_rn(y1);
            const __half h2 = __float2half_rn(y1 - __half2float(h1));
            uint2 part;
            part.x = __half_as_ushort(h0) | (uint32_t)__half_as_ushort(h1) << 16;
            part.y = __half_as_ushort(h2);
            *reinterpret_cast<uint2*>(smem + ks * Cfg::KSTAGE + 2 * Cfg::OPND + tok * 128 +
                                      ((tok & 7) << 4)) = part;
            const uint32_t bits = __ballot_sync(0xffffffffu, there);
            if (lane == 0) reinterpret_cast<uint32_t*>(M.valid[vs])[u] = bits;
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            bar_arrive(sc_full + 8 * vs);
            bar_arrive(k_full + 8 * ks);
            bar_arrive(raw_empty + 8 * rs);
          }
          if (++vs == VST) {
            vs = 0;
            eph ^= 1;
          }
          if (++ks == KST) {
            ks = 0;
            kph ^= 1;
          }
          if (++rs == nraw) {
            rs = 0;
            rph ^= 1;
          }
        }
      }
    }
  } else if (warp >= 8) {
    // ---- unpacking -------------------------------------------------------------------
    if (!(warp & 2))
      unpack_role<D, ASYM, true>(st, A, smem, M, k_full, k_empty, raw_full, warp, lane);
    else
      unpack_role<D, ASYM, false>(st, A, smem, M, v_full, v_empty, raw_full, warp, lane);
  } else {
    // ---- softmax: thread = row, group t the token tiles s + t, s + t + 2, ... ----------
    Seg w;
    const int t = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t base = tm + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t to = base + 64 + t * (D / 2);  // this group's half of O's columns
    uint32_t sph = 0, oph = 0;                    // next phases of the buffers' barriers
    int buf = 0, par = 0, tiles = 0;  // buffer; segment parity; tiles of the segments before
    bool ok = true;
    constexpr float SLACK = 8.f, BOOST = 7.f, NONE = -1e30f;
    if (t == 0) {  // channels 0 to 2 of the 16: the constant
      const __half2 c2 = __floats2half2_rn(A.q_ext, A.q_ext);
      const uint32_t c = *reinterpret_cast<const uint32_t*>(&c2);
      const uint32_t x[16] = {c, c & 0xFFFFu};
      tmem_st16(base + 192, x);
      tmem_wait_st();
      fence_before();
    }
    while (next_seg(&M.walk[warp], M, A, st, lane, w)) {
      // This thread's row: node and query head of the group.
      const int r = w.row0 + row;
      const bool mine = r < rows_of(w.cnt, st.G);
      const int node = mine ? r / st.G : 0, gh = mine ? r - node * st.G : 0;
      const size_t qrow = (((size_t)w.z * A.m + node) * st.Hq + w.h * st.G + gh) * D;
      const bool idle = !__any_sync(0xffffffffu, mine);  // a warp without rows
#pragma unroll
      for (int c = t * (D / 64); c < (t + 1) * (D / 64); ++c) {  // half of Q's columns
        uint32_t x[16];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const uint4 v = mine ? __ldg(reinterpret_cast<const uint4*>(A.q + qrow) + 4 * c + u)
                               : make_uint4(0, 0, 0, 0);
          perm8(v, x + 4 * u);
        }
        tmem_st16(base + 16 * c, x);
      }
      tmem_wait_st();
      fence_before();
      // Each node's ancestors, by one warp, for the segment that holds the drafts.
      if (w.e == w.nt && warp == 0) {
        for (int i = lane; i < 64; i += 32) {
          unsigned long long a = 0;
          if (i < w.cnt) {
            int x = i;
            while (x >= 0) {
              a |= 1ull << x;
              const int up = A.parents[(size_t)w.z * A.m + x];
              x = up < x ? up : -1;
            }
          }
          M.anc[par][i] = a;
        }
      }
      __syncwarp();
      if (lane == 0) bar_arrive(q_full);
      asm volatile("bar.sync 1, 256;" ::: "memory");  // anc is there

      float xref = NONE;  // the score that the reference m = sigma log2(e) xref goes by
      float boost = BOOST;  // 7 - m
      bool far = false;
      uint64_t l2 = pack2(0.f, 0.f), z2 = pack2(0.f, 0.f);
      const int n = w.e - w.s;
#pragma unroll 1
      for (int x0 = -w.skip(); x0 < n; x0 += 2) {
        const bool there = x0 + t >= 0 && x0 + t < n, have = there && !idle;
        const int at = tiles + x0 + t, sg = at % VST;  // V stages go round over all tiles
        const uint32_t ts = base + 256 + 128 * buf + 64 * t;
        const int bi = 2 * buf + t;
        if (there) {
          ok = ok && warp_wait(sc_full + 8 * sg, (at / VST) & 1, stop);
          ok = ok && warp_wait(s_full + 8 * bi, (sph >> bi) & 1, stop);
          sph ^= 1u << bi;
          fence_after();
        }
        const uint64_t sl2 = pack2(st.scale_log2, st.scale_log2);
        unsigned long long seen = ~0ull;
        bool part = false;
        float xnew = -CUDART_INF_F;
        // Scores are read from tensor memory twice, 32 columns at a time (short loops
        // keep the roles' code within the instruction caches).
        if (have && ok) {
          seen = *reinterpret_cast<const unsigned long long*>(M.valid[sg]) &
                 (w.s + x0 + t == w.nt - 1 ? M.anc[par][node] : ~0ull);
          part = __any_sync(0xffffffffu, seen != ~0ull);
          float mx[4] = {-CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F, -CUDART_INF_F};
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
            float x[32];
            tmem_ld32(ts + 32 * hf, reinterpret_cast<uint32_t*>(x));
            tmem_wait_ld();
            if (part) {
              const uint32_t bits = (uint32_t)(seen >> (32 * hf));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(bits >> c & 1)) x[c] = -CUDART_INF_F;
            }
#pragma unroll
            for (int c = 0; c < 32; c += 2)
              mx[c >> 1 & 3] = fmaxf(mx[c >> 1 & 3], fmaxf(x[c], x[c + 1]));
          }
          xnew = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        }
        int moves;
        asm volatile(
            "{ .reg .pred p, q; setp.ne.s32 p, %1, 0; "
            "barrier.cta.red.or.pred.aligned q, 2, 256, p; selp.s32 %0, 1, 0, q; }"
            : "=r"(moves)
            : "r"((int)((xnew - xref) * st.scale_log2 > SLACK))
            : "memory");
        if (moves) {  // some row's reference moves
          M.mx[t][row] = xnew;
          asm volatile("bar.sync 1, 256;" ::: "memory");
          xnew = fmaxf(xnew, M.mx[t ^ 1][row]);
          const bool move = (xnew - xref) * st.scale_log2 > SLACK;
          const float f = move ? ex2((xref - xnew) * st.scale_log2) : 1.f;
          if (move) xref = xnew;
          // Past 2^22 the rounding of m would show in the exponent (at 2^24 as infinite
          // probabilities): the differences are taken before the scale then.
          const float m = xref * st.scale_log2;
          far = __any_sync(0xffffffffu, fabsf(m) >= 0x1p22f);
          boost = far ? BOOST : BOOST - m;
          l2 = fma2(l2, pack2(f, f), pack2(0.f, 0.f));
          if (ASYM) z2 = fma2(z2, pack2(f, f), pack2(0.f, 0.f));
          if (x0 > 0 && ok) {  // O holds the products up to the pair before: rescale it
            const int ob = buf ^ 1;
            ok = warp_wait(o_done + 8 * ob, (oph >> ob & 1) ^ 1, stop);
            fence_after();
            if (ok && !idle) {
#pragma unroll 1
              for (int c = 0; c < D / 2; c += 16) {
                uint32_t v[16];
                tmem_ld16(to + c, v);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 16; ++u) v[u] = __float_as_uint(__uint_as_float(v[u]) * f);
                tmem_st16(to + c, v);
              }
              tmem_wait_st();
            }
          }
          fence_before();
          asm volatile("bar.sync 1, 256;" ::: "memory");  // before any product of this pair
          fence_after();
        }
        if (have && ok) {
          if (far) far_scores(ts, xref);
          const uint64_t off = pack2(boost, boost);
#pragma unroll 1
          for (int hf = 0; hf < 2; ++hf) {
            float x[32];
            tmem_ld32(ts + 32 * hf, reinterpret_cast<uint32_t*>(x));
            const ulonglong2* rv = reinterpret_cast<const ulonglong2*>(M.rsv[sg]) + 8 * hf;
            const ulonglong2* zv = reinterpret_cast<const ulonglong2*>(M.zsv[sg]) + 8 * hf;
            tmem_wait_ld();
            if (part) {
              const uint32_t bits = (uint32_t)(seen >> (32 * hf));
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (!(bits >> c & 1)) x[c] = -CUDART_INF_F;
            }
            uint32_t p[16];
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              const ulonglong2 ra = rv[c];
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                float a, b;
                unpack2(fma2(pack2(x[4 * c + 2 * u], x[4 * c + 2 * u + 1]), sl2, off), a, b);
                a = ex2(a);
                b = ex2(b);
                const uint64_t ab = pack2(a, b);
                l2 = fma2(ab, u ? ra.y : ra.x, l2);
                if (ASYM) {
                  const ulonglong2 za = zv[c];
                  z2 = fma2(ab, u ? za.y : za.x, z2);
                }
                const __half2 hh = __floats2half2_rn(a, b);
                p[2 * c + u] = *reinterpret_cast<const uint32_t*>(&hh);
              }
            }
            tmem_st16(ts + 16 * hf, p);  // over scores already read
          }
          tmem_wait_st();
        }
        if (there) {
          fence_before();
          __syncwarp();
          if (lane == 0) bar_arrive(p_full + 8 * bi);
        }
        oph ^= 1u << buf;
        buf ^= 1;
      }
      const int ob = buf ^ 1;  // the last pair's products
      ok = ok && warp_wait(o_done + 8 * ob, (oph >> ob & 1) ^ 1, stop);
      fence_after();
      {
        float la, lb, za, zb;
        unpack2(l2, la, lb);
        unpack2(z2, za, zb);
        M.lz[t][0][row] = la + lb;
        M.lz[t][1][row] = za + zb;
      }
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const float l = M.lz[0][0][row] + M.lz[1][0][row], add = M.lz[0][1][row] + M.lz[1][1][row];
      const bool direct = w.whole();
      const float inv = l > 0.f ? 1.f / l : 0.f;
      float4* part4 = reinterpret_cast<float4*>(A.acc) + (size_t)w.slot * (D / 4) * TM_ROWS;
      if (!direct && mine && t == 0) A.ml[(size_t)w.slot * TM_ROWS + row] = make_float2(xref, l);
#pragma unroll 1
      for (int c = 0; c < D / 2; c += 16) {
        uint32_t x[16];
        tmem_ld16(to + c, x);
        tmem_wait_ld();
        if (!mine) continue;
        float v[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          // natural channel u of the 16: position in the unpacked order
          const int at = (u & 8) + ((u & 4) ? 2 * (u & 3) + 1 : 2 * (u & 3));
          v[u] = __uint_as_float(x[at]) + add;
        }
        const int ch = t * (D / 2) + c;
        if (direct) {
          uint32_t hw[8];
#pragma unroll
          for (int u = 0; u < 8; ++u) {
            const __half2 hh = l > 0.f ? __floats2half2_rn(v[2 * u] * inv, v[2 * u + 1] * inv)
                                       : __floats2half2_rn(0.f, 0.f);
            hw[u] = *reinterpret_cast<const uint32_t*>(&hh);
          }
          uint4* dst = reinterpret_cast<uint4*>(A.o + qrow + ch);
          dst[0] = make_uint4(hw[0], hw[1], hw[2], hw[3]);
          dst[1] = make_uint4(hw[4], hw[5], hw[6], hw[7]);
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            part4[(size_t)(ch / 4 + u) * TM_ROWS + row] =
                make_float4(v[4 * u], v[4 * u + 1], v[4 * u + 2], v[4 * u + 3]);
        }
      }
      fence_before();
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the accumulator and lz are read
      tiles += n;
      par ^= 1;
    }
    if (!ok && lane == 0) set_error(st, EKV_ETIMEOUT);
  }
  __syncthreads();
  if (warp == W_SCORES) {
    fence_after();
    if (*stop) {
      if (lane == 0) set_error(st, EKV_ETIMEOUT);
      for (int i = 0; i < 2000; ++i) __nanosleep(1000);  // copies and products in flight land
    }
    tmem_free(tm, 512);
  }
}

// Merge the partials of the units that run ends cut: a thread per (row, 4 channels).
constexpr int MAX_GRID = 256;
template <int D>
__global__ void __launch_bounds__(TM_ROWS) tree_merge_kernel(DevState st, TreeArgs A, int rt_max,
                                                             int groups) {
  __shared__ int64_t s_start[MAX_GRID + 1];
  __shared__ int s_slot[MAX_GRID];
  // Every CTA, also one without rows: the scratch that tree_kernel wrote is free for other work
  // once this launch is over.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int rt = blockIdx.x % rt_max, h = blockIdx.x / rt_max % st.Hkv;
  const int z = blockIdx.x / rt_max / st.Hkv, row = threadIdx.x;
  const int cnt = A.n_nodes ? min(A.m, max(0, A.n_nodes[z])) : A.m;
  const int rows = rows_of(cnt, st.G);
  if (rt * TM_ROWS >= rows) return;
  for (int i = row; i <= A.grid; i += TM_ROWS) s_start[i] = A.pre[A.n_seqs + 1 + i];
  // The runs that hold parts of this unit, [a, a + nt): c0 .. c1 - 1.
  const int64_t first = A.pre[z], units = (int64_t)st.Hkv * row_tiles(rows);
  const int nt = (int)((uint32_t)(A.pre[z + 1] - first) / (uint32_t)units);
  const int64_t a = first + (int64_t)(h * row_tiles(rows) + rt) * nt;
  __syncthreads();
  int c0 = 0, c1 = 0;
  for (int i0 = 0; i0 < A.grid; i0 += TM_ROWS) {
    const int i = i0 + row;
    c0 += __syncthreads_count(i < A.grid && s_start[i + 1] <= a);
    c1 += __syncthreads_count(i < A.grid && s_start[i] < a + nt);
  }
  if (c1 - c0 == 1) return;  // one CTA had the whole unit and wrote o
  for (int i = row; c0 + i < c1; i += TM_ROWS) {
    const int c = c0 + i;
    s_slot[i] = s_start[c] == s_start[c + 1] ? -1 : 2 * c + (s_start[c] > a ? 0 : 1);
  }
  __syncthreads();
  const int r = rt * TM_ROWS + row, n = c1 - c0;
  if (r >= rows) return;
  constexpr int U = 8;  // partials in flight
  float m = -1e30f;
  for (int i = 0; i < n; i += U) {
    float x[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = i + u < n ? s_slot[i + u] : -1;
      x[u] = k >= 0 ? __ldcg(&A.ml[(size_t)k * TM_ROWS + row].x) : -1e30f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) m = fmaxf(m, x[u]);
  }
  const int node = r / st.G, gh = r - node * st.G;
  __half* dst = A.o + (((size_t)z * A.m + node) * st.Hq + h * st.G + gh) * D;
  for (int g = blockIdx.y * groups; g < (int)(blockIdx.y + 1) * groups; ++g) {
    float l = 0.f;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < n; i += U) {
      float2 ml[U];
      float4 x[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = i + u < n ? s_slot[i + u] : -1;
        ml[u] = make_float2(-1e30f, 0.f);
        x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k >= 0) {
          ml[u] = __ldcg(&A.ml[(size_t)k * TM_ROWS + row]);
          x[u] = __ldcg(reinterpret_cast<const float4*>(A.acc) +
                        ((size_t)k * (D / 4) + g) * TM_ROWS + row);
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = ml[u].y > 0.f ? ex2((ml[u].x - m) * st.scale_log2) : 0.f;
        l = fmaf(f, ml[u].y, l);
        v.x = fmaf(f, x[u].x, v.x);
        v.y = fmaf(f, x[u].y, v.y);
        v.z = fmaf(f, x[u].z, v.z);
        v.w = fmaf(f, x[u].w, v.w);
      }
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    __align__(8) __half2 hh[2] = {__floats2half2_rn(v.x * inv, v.y * inv),
                                  __floats2half2_rn(v.z * inv, v.w * inv)};
    *reinterpret_cast<uint2*>(dst + 4 * g) = *reinterpret_cast<const uint2*>(hh);
  }
}

template <int D>
constexpr int tree_smem() {
  constexpr int bytes = TCfg<D>::MISC_OFF + (int)sizeof(TMisc) + 1024;
  static_assert(bytes <= 227 * 1024, "shared memory of a CTA");
  return bytes;
}

template <int D, bool ASYM>
cudaError_t launch_tree(const DevState& st, TreeArgs A, int n_seqs, cudaStream_t s) {
  cudaError_t e = smem_once<tree_kernel<D, ASYM>, tree_smem<D>()>();
  const TreeArgs B = A;
  for (int z = 0; z < n_seqs && e == cudaSuccess; z += TSEQS) {
    A.n_seqs = n_seqs - z < TSEQS ? n_seqs - z : TSEQS;
    A.slots = B.slots + z;
    A.n_nodes = B.n_nodes ? B.n_nodes + z : nullptr;
    A.parents = B.parents + (size_t)z * B.m;
    A.q = B.q + (size_t)z * B.m * st.Hq * D;
    A.o = B.o + (size_t)z * B.m * st.Hq * D;
    A.k = B.k + (size_t)z * B.m * st.Hkv * D;
    A.v = B.v + (size_t)z * B.m * st.Hkv * D;
    tree_kernel<D, ASYM><<<A.grid, TT, tree_smem<D>(), s>>>(st, A);
    e = cudaGetLastError();
    if (e != cudaSuccess) break;
    // One thread a row and 4 channels; with many row tiles each thread takes 4 of them.  Whole
    // call with four and with one, us: 32 tiles 34.9 and 29.4, 64 27.1 and 23.3 (52.6 and 50.6
    // with every row used), 128 36.3 and 36.0 (77.2 and 79.1), 256 54.1 and 56.9 (68.2, 70.6).
    const int rt_max = (rows_of(B.m, st.G) + TM_ROWS - 1) / TM_ROWS;
    const int tiles = A.n_seqs * st.Hkv * rt_max, groups = tiles >= 128 ? 4 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(tiles, D / 4 / groups);
    cfg.blockDim = dim3(TM_ROWS);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_merge_kernel<D>, st, A, rt_max, groups);
  }
  return e;
}

struct TreeScratch {
  int grid = 0;
  size_t acc = 0, ml = 0, pre = 0, bytes = 0;
};
// One CTA an SM; two partials a CTA (its first and its last segment).
int tree_scratch(const DevState& st, int n_seqs, TreeScratch* t) {
  t->grid = sm_count();
  if (t->grid <= 0) {
    cudaGetLastError();
    return EKV_ECUDA;
  }
  if (t->grid > MAX_GRID) t->grid = MAX_GRID;  // the merging kernel's table of parts
  const size_t parts = (size_t)t->grid * 2 * TM_ROWS;
  const int n = n_seqs < TSEQS ? n_seqs : TSEQS;
  t->acc = 0;
  t->ml = parts * st.D * sizeof(float);
  t->pre = t->ml + parts * sizeof(float2);
  t->bytes = t->pre + (size_t)(n + 1 + t->grid + 1) * sizeof(int64_t);
  return EKV_OK;
}

}  // namespace
}  // namespace ekv

extern "C" EKV_API int ekv_tree_attn_scratch_bytes(ekv_cache* cache, int32_t n_seqs,
                                                   int32_t max_nodes, int64_t* out) {
  using namespace ekv;
  DevState st;
  int splits, vb, pack;
  if (!out || max_nodes < 1 || max_nodes > EKV_TREE_MAX_NODES) return EKV_EINVAL;
  int rc = attn_plan(cache, 0, n_seqs, &st, &splits, &vb, &pack);
  if (rc != EKV_OK) return rc;
  TreeScratch t;
  rc = tree_scratch(st, n_seqs, &t);
  if (rc == EKV_OK) *out = (int64_t)t.bytes;
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
  int rc = attn_plan(cache, layer, n_seqs, &st, &splits, &vb, &pack);
  if (rc != EKV_OK) return rc;
  if (n_seqs == 0) return EKV_OK;
  if (!seq_slots || !parents || !q || !k || !v || !o) return EKV_EINVAL;
  if (((uintptr_t)q | (uintptr_t)k | (uintptr_t)v | (uintptr_t)o) & 15) return EKV_EINVAL;
  if (((uintptr_t)seq_slots | (uintptr_t)n_nodes | (uintptr_t)parents) & 3) return EKV_EINVAL;
  TreeScratch t;
  rc = tree_scratch(st, n_seqs, &t);
  if (rc != EKV_OK) return rc;
  if (!scratch || ((uintptr_t)scratch & 15) || scratch_bytes < (int64_t)t.bytes) return EKV_EINVAL;
  TreeArgs A = {};
  A.layer = layer;
  A.vb = vb;
  A.m = max_nodes;
  A.slots = seq_slots;
  A.n_nodes = n_nodes;
  A.parents = parents;
  A.q = static_cast<const __half*>(q);
  A.k = static_cast<const __half*>(k);
  A.v = static_cast<const __half*>(v);
  A.o = static_cast<__half*>(o);
  uint8_t* base = static_cast<uint8_t*>(scratch);
  A.acc = reinterpret_cast<float*>(base + t.acc);
  A.ml = reinterpret_cast<float2*>(base + t.ml);
  A.pre = reinterpret_cast<int64_t*>(base + t.pre);
  A.grid = t.grid;
  // c = 2^k near 1 / sl, so that log2 s / (sl c) is of the size of log2 s
  const int ex = -ilogbf(st.scale_log2);
  if (ex > 25 || ex < -14) return EKV_EUNSUPPORTED;
  A.q_ext = ldexpf(1.f, ex > 15 ? 15 : ex);
  A.k_ext = 1.f / (st.scale_log2 * A.q_ext);
  using Fn = cudaError_t (*)(const DevState&, TreeArgs, int, cudaStream_t);
  const Fn fn = st.D == 64 ? (st.asym ? launch_tree<64, true> : launch_tree<64, false>)
                           : (st.asym ? launch_tree<128, true> : launch_tree<128, false>);
  const cudaError_t e = fn(st, A, n_seqs, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? EKV_OK : EKV_ECUDA;
}
