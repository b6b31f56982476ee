// fa_q8_attn.cu -- attention of new queries over the 8-bit paged key/value cache, sm_103a: the
// kernel for up to 32 query rows a kv head (at head_dim 256 for any number), the joining kernel and
// the launches; fa_q8_chunk.cuh has the kernel for more rows.
//
// Key j of sequence b is slot j % page_size of page table[b][j / page_size]; its key is
// k_scale * k codes, its value v_scale * v codes, and query i of the q_len new positions sees key
// j iff j < len (and, with the causal rule, j <= len - q_len + i). O = softmax(scale q k^T) v and
// L = log sum exp; a query that sees no key gives O = 0 and L = -inf.
//
// Decoding reads every code once, so HBM bounds it; 152 SMs at the measured copy rate take in
// 23 codes a clock each, too many to widen them on the CUDA cores first. The tensor cores read
// the codes as they are (tcgen05 kind::f8f6f4), and the bf16 and f32 operands that meet them are
// split into 8-bit pieces, which cost only columns of an otherwise empty tile:
//  * q (8 significant bits) = hi + lo / 16, both e4m3 (4 bits each, hi the nearest), after a power
//    of two for each row that puts its largest element into [128, 256). Exact, except that
//    elements 2^-14 below the row's largest lose what is under 2^-22 of it.
//  * a softmax weight, rounded to 9 bits in f16, = p1 + p2 / 8 + p3 / 64, all e5m2: e5m2 is the
//    upper byte of an f16 (3 bits of the 9), so a piece is that byte of what the pieces before it
//    leave, times 8. In steps of 2^-33 of the row's largest weight at least, so that thousands of
//    small weights beside a key that takes nearly all still count (with the pieces unscaled the
//    steps are 2^-27, and a case like that was off by 1.3 times its tolerance).
// S^T = K q^T has the keys as the M = 128 rows of a tile and R query rows as 2 R columns: a thread
// owns a key, whose two scales are then the thread's constants, and holds its scores.
// O^T = V^T w^T has the head dim as M (V is read transposed, MN-major) and 3 R columns; the value
// scale is part of the weight: w = exp2(score + log2(v_scale) - m), m the running maximum of that
// sum less 11, so that a value counts down to 2^-33 of the row's largest weight times scale; the
// softmax's sum takes w / v_scale, or, in a tile with a scale 2^-96 of one that came before, an
// exponential of its own (there w may be 0 where w / v_scale is not). All sums are f32.
//
// Work: the (sequence, kv head, block of R rows) units, each ceil(len / 128) key tiles, form one
// list of tiles, cut evenly over persistent CTAs (the lengths are on the device; each CTA finds its
// part from them). A unit counts kUnitCost tiles more than it has, what its start and end cost. A
// CTA writes the units it has whole; of the others it leaves its share's O, m and sum, which a
// second kernel joins in the order of the keys.
//
// Warps of a CTA: one or two softmax warpgroups of 8 rows (thread = key of the tile, and head-dim
// row of O^T), then one warp each for the TMA copies of K and V pages (boxes of min(page_size, 128)
// rows), for issuing S^T, for O^T (it also clears what must not meet a weight: rows behind the
// sequence's end, NaN behind a query row), and for the list: it walks it, splits q and fetches the
// scales. All waits on barriers are bounded.
//
// Measured (device time of a call with both kernels): 64 sequences of 1k to 16k keys, head_dim 128,
// 32:8 heads, 963 MB: 150 us, 94 % of the measured copy rate (6787 GB/s); 16 sequences of 2k to 16k
// keys, 351 MB: 63 us (82 %), the start, the joining kernel and the last CTAs being the rest; with
// 16 rows a kv head 70 us for 322 MB, bound by the softmax's latency and issue; 128 sequences of up
// to 2047 keys at head_dim 64, 132 MB: 37 us, bound by latency and instruction fetch (issue active
// 38 %; a unit has 8 tiles, and its start and end take as long as four).
#include <float.h>

#include <algorithm>

#include "fa_common.cuh"
#include "fa_launch.h"
#include "fa_q8.cuh"

namespace fa {

namespace {
constexpr int kKT = 128;          // keys of a tile (the MMA M of S^T)
// Tiles' worth of a unit's start and end (128 sequences of up to 2k keys, head_dim 64: 51 us with
// 0, 40 with 2, 37 with 4; long sequences do not tell).
constexpr int kUnitCost = 4;
constexpr int kPageChunk = 128;   // block-table entries staged at a time
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// The weight of the score that m was taken from is 2^kTop; m stays until a weight passes
// 2^kMost (where f16 would not hold 8 times what the first piece leaves).
constexpr float kTop = 11.0f, kMost = 15.0f;
// The softmax's sums are held in units of 2^16: with value scales from 2^-100 to 2^100 neither
// w / v_scale nor 2^22 of them leave f32, and a row's sum is 2^-105 at least (its m less its
// largest score is at most 100 - 11). A factor between two m's may be any, so sums are scaled by
// its root twice (scale_sum).
constexpr float kSumExp = 16.0f, kSumUnit = 65536.0f;
// Value scales of a unit's keys (log2) may be this far below the largest up to their tile for
// w / v_scale to serve: a w below f32 (2^-126) is then that of a score 2^-41 of the largest one's.
constexpr float kApart = 96.0f;

// R query rows of a unit at a time. KST, VST: stages of the K and V rings; V has more, as a V tile
// stays until the weights of its keys are there (3 and 3 of 16 KB: 167 us, 2 and 4: 162 us for 64
// sequences of up to 16k keys).
template <int HD, int R_, int RL>
struct Q8Layout {
  static constexpr int R = R_;
  static constexpr int CTAS = HD > 128 ? 1 : HD == 64 && RL <= 4 ? 3 : 2;  // resident on an SM
  static constexpr int KST = HD == 64 && R == 16 ? 4 : 2;
  static constexpr int VST = HD == 64 || R == 8 ? 4 : HD == 128 ? 2 : 3;
  static constexpr int CH = HD <= 128 ? HD : 128;   // columns (bytes) of a swizzled row
  static constexpr int KCH = HD / CH;               // row chunks: 1, or 2 at head_dim 256
  static constexpr int NS = 2 * R;                  // columns of S^T: hi rows, lo rows
  static constexpr int NP = 4 * R;                  // columns of O^T: three pieces, one unused
  static constexpr int KV_BYTES = kKT * HD;
  static constexpr int Q_BYTES = NS * HD;
  static constexpr int P_BYTES = kKT * NP;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_V = OFF_K + KST * KV_BYTES;
  static constexpr int OFF_Q = OFF_V + VST * KV_BYTES;
  static constexpr int OFF_P = OFF_Q + 2 * Q_BYTES;
  static constexpr int SMEM_BYTES = OFF_P + 2 * P_BYTES + 1024;
  static constexpr int COL_S = 0;                   // two S^T buffers, then O^T
  static constexpr int COL_O = 2 * NS;
  static constexpr int TMEM_USED = COL_O + KCH * NP;
  static constexpr int TMEM_COLS = TMEM_USED <= 64 ? 64 : TMEM_USED <= 128 ? 128
                                   : TMEM_USED <= 256 ? 256 : 512;
  static constexpr int NWG = R / 8;                 // softmax warpgroups, 8 rows each
  static constexpr int THREADS = 128 * NWG + 128;
  static constexpr int TMA_WARP = 4 * NWG, S_WARP = TMA_WARP + 1, O_WARP = TMA_WARP + 2,
                       QS_WARP = TMA_WARP + 3;
  static_assert(TMEM_USED <= 512 && TMEM_COLS * CTAS <= 512, "TMEM budget");
  // dynamic, static (pages, scales, barriers, rows: below) and the driver's 1 KB
  static constexpr int STATIC_BYTES = 4 * kPageChunk + 16 * kKT + 72 * R + 512;
  static_assert((SMEM_BYTES + STATIC_BYTES + 1024) * CTAS <= 228 * 1024, "shared memory budget");
};

// Swizzle of a row of W bytes (W = 32, 64 or 128): the 16-byte chunk c of row r lies at chunk
// swz(c, r). (The swizzle XORs address bits 4.. with bits 7.., and tiles start on its period.)
template <int W>
__device__ __forceinline__ int swz(int c, int r) {
  return c ^ (W == 128 ? (r & 7) : W == 64 ? ((r >> 1) & 3) : ((r >> 2) & 1));
}
// Descriptor of an operand of rows of W bytes, swizzled by W: the next 8 rows are 8 W away, the
// next W-byte chunk (where there is one) `lbo`.
template <int W>
__device__ __forceinline__ Desc q8_desc(uint32_t saddr, uint32_t lbo) {
  const uint64_t mode = W == 128 ? 2 : W == 64 ? 4 : 6;
  uint64_t d = (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)((lbo >> 4) & 0x3FFFu) << 16;
  d |= (uint64_t)((8 * W) >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= mode << 61;
  return Desc{static_cast<uint32_t>(d), static_cast<uint32_t>(d >> 32)};
}
// Instruction descriptor, kind::f8f6f4, f32 accumulator; formats: 0 e4m3, 1 e5m2.
constexpr uint32_t idesc_f8(int a_fmt, int b_fmt, int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_fmt << 7) | ((uint32_t)b_fmt << 10) | ((uint32_t)a_mn << 15) |
         ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint32_t a_lo, uint32_t a_hi,
                                       uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 ad, bd;\n setp.ne.b32 p, %6, 0;\n"
      " mov.b64 ad, {%1, %2};\n mov.b64 bd, {%3, %4};\n"
      " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], ad, bd, %5, p;\n}\n" ::"r"(d_tmem),
      "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float (&r)[8]) {
  uint32_t v[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]),
                 "=r"(v[6]), "=r"(v[7])
               : "r"(taddr));
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = __uint_as_float(v[e]);
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 2^x, subnormal results included.
__device__ __forceinline__ float ex2_full(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// A sum times 2^-up, also where 2^-up is below f32 and the product is not.
__device__ __forceinline__ float scale_sum(float sum, float up) {
  const float root = ex2(-0.5f * up);
  return sum * root * root;
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                   taddr),
               "r"(__float_as_uint(r[0])), "r"(__float_as_uint(r[1])), "r"(__float_as_uint(r[2])),
               "r"(__float_as_uint(r[3])), "r"(__float_as_uint(r[4])), "r"(__float_as_uint(r[5])),
               "r"(__float_as_uint(r[6])), "r"(__float_as_uint(r[7]))
               : "memory");
}
// Scores of 8 rows: their hi columns, and the lo columns R further on.
template <int R>
__device__ __forceinline__ void load_scores(uint32_t taddr, uint32_t (&s)[16]) {
  if constexpr (R == 8) {
    tmem_ld16(taddr, s);
  } else {
    float a[8], b[8];
    tmem_ld8(taddr, a);
    tmem_ld8(taddr + R, b);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      s[e] = __float_as_uint(a[e]);
      s[8 + e] = __float_as_uint(b[e]);
    }
  }
}
// Two weights (>= 0, at most 2^15) -> two f16 rounded to 9 bits: cut to f16's 11, then the nearest
// of 9 (half up), which together is the nearest of the f32 value. (With f16's own rounding first,
// one weight in four was a tie and went up: O was 3.4e-4 too large, the sum being of the weights
// as they are.)
__device__ __forceinline__ uint32_t weight_f16x2(float lo, float hi) {
  uint32_t h;
  asm("cvt.rz.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return (h + 0x00020002u) & 0xfffcfffcu;
}
// 8 times what their upper bytes (the e5m2 pieces) leave; exact, and below 2^16.
__device__ __forceinline__ uint32_t f16x2_rest(uint32_t h) {
  const uint32_t top = h & 0xff00ff00u;
  const __half2 r = __hmul2(__hsub2(*reinterpret_cast<const __half2*>(&h),
                                    *reinterpret_cast<const __half2*>(&top)),
                            __float2half2_rn(8.0f));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// The barrier of the 128 threads of softmax warpgroup `wg`; true where any of them came with `v`.
__device__ __forceinline__ bool softmax_any(int wg, bool v) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 128, p;\n"
      " selp.s32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)v), "r"(wg + 1)
      : "memory");
  return r != 0;
}
// Bounded waits of this kernel. A first poll in line (suspended for as long as the hardware likes);
// what follows is out of line, with polls suspended for up to 20 us. (Most warps wait most of the
// time; short polls in line cost issue and the SM's instruction cache, which the softmax needs.)
// Under a limit below 100 us, which exists to make waits run out, those polls are not suspended,
// and S^T's wait for a unit's q, which always lasts a while at the start, begins with one that is
// not (elsewhere that costs 2 %).
__device__ __noinline__ bool wait_more(uint64_t* bar, uint32_t parity, WaitCtl* w) {
  const uint64_t t0 = globaltimer();
  const bool brief = w->limit_ns < 100000ull;
  for (;;) {
    uint32_t ok = 0;
    if (brief)
      ok = mbar_test_wait(bar, parity);
    else
      asm volatile(
          "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 20000;\n"
          " selp.u32 %0, 1, 0, p;\n}\n"
          : "=r"(ok)
          : "r"(smem_u32(bar)), "r"(parity)
          : "memory");
    if (ok) return true;
    if (*reinterpret_cast<volatile int*>(&w->abort)) return false;
    if (globaltimer() - t0 > w->limit_ns) {
      *reinterpret_cast<volatile int*>(&w->abort) = 1;
      return false;
    }
  }
}
__device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, WaitCtl* w) {
  return mbar_try_wait(bar, parity) || wait_more(bar, parity, w);
}
// The wait of a whole warp, that does not part its lanes: true for all or none.
template <bool SUSPEND = true>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, WaitCtl* w) {
  if (__all_sync(0xffffffffu,
                 SUSPEND ? mbar_try_wait(bar, parity) : mbar_test_wait(bar, parity)))
    return true;
  return __all_sync(0xffffffffu, wait_more(bar, parity, w));
}
// Largest value of the warp (NaN is passed over).
__device__ __forceinline__ float warp_max(float x) {
  float r;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

// The bytes of a word that are e4m3 NaN (0x7F, 0xFF): bit 7 of each.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t x) {
  return ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
}
// Rows r0 .. r1 - 1 of a V tile (kKT rows of CH bytes a chunk) become 0. Warp-wide; out of line, as
// the tiles at the end of a sequence are few.
template <int HD, int CH>
__device__ __noinline__ void clear_rows(uint8_t* vt, int r0, int r1, int lane) {
#pragma unroll 1
  for (int e = lane; e < (r1 - r0) * (HD / 16); e += 32) {
    const int r = r0 + e / (HD / 16), x = e % (HD / 16) * 16;
    *reinterpret_cast<uint4*>(vt + x / CH * (kKT * CH) + r * CH + x % CH) =
        make_uint4(0u, 0u, 0u, 0u);
  }
}
// NaN codes in the rows r0 .. r1 - 1 of a V tile, keys that some query rows of the block do not see
// (a weight of 0 would not keep a NaN out of O): the codes become 0, and the key's weight NaN for
// the query rows q that see it (n0 + r < lim[q]): byte q of the key's row of NP bytes in `pt`.
template <int HD, int CH, int RL, int NP>
__device__ __noinline__ void clear_nan(uint8_t* vt, uint8_t* pt, int r0, int r1, int n0,
                                       const int* lim, int lane) {
#pragma unroll 1
  for (int e = lane; e < (r1 - r0) * (HD / 16); e += 32) {
    const int r = r0 + e / (HD / 16), x = e % (HD / 16) * 16;
    uint4* at = reinterpret_cast<uint4*>(vt + x / CH * (kKT * CH) + r * CH + x % CH);
    uint4 v = *at;
    const uint4 z = make_uint4(nan_bytes(v.x), nan_bytes(v.y), nan_bytes(v.z), nan_bytes(v.w));
    if (z.x | z.y | z.z | z.w) {
      v.x &= ~((z.x >> 7) * 0xffu);
      v.y &= ~((z.y >> 7) * 0xffu);
      v.z &= ~((z.z >> 7) * 0xffu);
      v.w &= ~((z.w >> 7) * 0xffu);
      *at = v;
#pragma unroll 1
      for (int q = 0; q < RL; ++q)
        if (n0 + r < lim[q]) pt[r * NP + swz<NP>(0, r) * 16 + q] = 0x7f;
    }
  }
}

struct Q8K {
  const __nv_bfloat16* q;  // [B, H, lq, HD]
  const uint8_t* codes[2];  // K, V (where no tensor map is used)
  const float* k_scale;
  const float* v_scale;
  const int32_t* table;
  const int32_t* lens;
  __nv_bfloat16* o;
  float* lse;
  float* o_part;   // [2 * grid, R, HD]: O of a share, in units of 2^m
  float* ml_part;  // [2 * grid, 2, R]: m and the sum
  int* status;
  int B, Hk, lq, rows, rb, max_pages, num_pages, ps_shift, sb_shift;
  float scale_log2;
  unsigned long long wait_limit_ns;
};

__device__ __forceinline__ int q8_len(const Q8K& p, int b) {
  const long long cap = (long long)p.max_pages << p.ps_shift;
  const int raw = p.lens[b];
  return raw < 0 ? 0 : raw > cap ? (int)cap : raw;
}

// What a unit of sequence b counts in the list: kUnitCost and its tiles; 0 without keys.
__device__ __forceinline__ int q8_cost(const Q8K& p, int b) {
  const int len = q8_len(p, b);
  return len > 0 ? (len + kKT - 1) / kKT + kUnitCost : 0;
}
// The sum over all sequences (of one unit each), by one warp that has that of sequence `lane`.
// The host has checked that the whole list, Hk * rb times as long, fits 31 bits.
__device__ __forceinline__ int q8_all_costs(const Q8K& p, int mine, int lane) {
#pragma unroll 1
  for (int b = lane + 32; b < p.B; b += 32) mine += q8_cost(p, b);
  return (int)__reduce_add_sync(0xffffffffu, (unsigned)mine);
}
// A CTA's share: the list cut evenly over the grid.
__device__ __forceinline__ unsigned q8_share(unsigned all, unsigned grid) {
  return (all + grid - 1) / grid;
}

// The units of a CTA's share [t, t1) of the list, in order: the last warp walks it and publishes
// the units in shared memory, where the other roles take them from.
struct Walk {
  unsigned t, t1;    // next place in the list, end of the share
  unsigned pre;      // the list before sequence b
  int b, cost, len;  // sequence, what each of its units counts, its length
  // the unit found by next()
  int kh, rb, ja, jb;  // kv head, row block, tiles [ja, jb) of it (tiles that no row sees left out)
  int whole;           // the share has all of the unit's tiles
  int first;           // the share has its first tile

  // The share of CTA `cta` (warp-wide).
  __device__ __forceinline__ void init(const Q8K& p, unsigned cta, unsigned grid, int lane) {
    const unsigned U = (unsigned)(p.Hk * p.rb);
    const int mine = lane < p.B ? q8_cost(p, lane) : 0;
    const unsigned all = (unsigned)q8_all_costs(p, mine, lane) * U;
    const unsigned per = q8_share(all, grid);
    t = per * cta;  // (below all + grid)
    t1 = min(t + per, all);
    pre = 0;
    b = cost = len = 0;
    if (t >= t1) return;
#pragma unroll 1
    for (int base = 0;; base += 32) {  // ends: t lies below the sum over all sequences
      const unsigned n =
          (base == 0 ? mine : base + lane < p.B ? q8_cost(p, base + lane) : 0) * U;
      unsigned upto = n;
#pragma unroll 1
      for (int o = 1; o < 32; o *= 2) {
        const unsigned x = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += x;
      }
      const unsigned beyond = __ballot_sync(0xffffffffu, pre + upto > t);
      if (beyond || base + 32 >= p.B) {
        const int at = beyond ? __ffs(beyond) - 1 : 31;
        b = min(base + at, p.B - 1);
        pre += __shfl_sync(0xffffffffu, upto - n, at);
        break;
      }
      pre += __shfl_sync(0xffffffffu, upto, 31);
    }
    len = q8_len(p, b);
    cost = q8_cost(p, b);
  }

  template <bool MULTI>
  __device__ __forceinline__ bool next(const Q8K& p, int R) {
    const unsigned U = (unsigned)(p.Hk * p.rb);
    int je;
    do {  // (a share may end within what a unit counts before its tiles)
      if (t >= t1) return false;
#pragma unroll 1
      while (t >= pre + U * cost) {  // the next sequence with keys
        pre += U * cost;
        if (++b >= p.B) return false;
        len = q8_len(p, b);
        cost = q8_cost(p, b);
      }
      const unsigned in = t - pre, u = in / (unsigned)cost;
      kh = (int)u;
      const int from = (int)(in - u * cost), to = min(cost, from + (int)(t1 - t));
      t += to - from;
      ja = max(0, from - kUnitCost);
      je = max(0, to - kUnitCost);
    } while (je == 0);
    rb = 0;
    if (p.rb > 1) {
      const int u = kh;
      kh = (int)((unsigned)u / (unsigned)p.rb);
      rb = u - kh * p.rb;
    }
    first = ja == 0;
    whole = first && je == cost - kUnitCost;
    // keys that any row of the block sees
    jb = je;
    if (MULTI) {
      const int r0 = rb * R, r1 = min(p.rows, r0 + R) - 1;
      const int imax = r0 / p.lq == r1 / p.lq ? r1 % p.lq : p.lq - 1;
      const int seen = max(0, len - p.lq + imax + 1);
      jb = max(ja, min(je, (seen + kKT - 1) / kKT));
    }
    return true;
  }
};

struct Unit {
  int b, kh, rb, ja, jb, len, whole, first;
};
// Units in shared memory: the last warp publishes, the others read and free.
constexpr int kUnits = 4;
struct UnitRing {
  int4 at[kUnits][2];
  uint64_t full[kUnits], free[kUnits];
};
// The next unit, for a whole warp: false where a wait ran out. end: there is none.
__device__ __forceinline__ bool take_unit(UnitRing* ring, int un, Unit& u, bool& end, int lane,
                                          WaitCtl* wctl) {
  const int slot = un % kUnits;
  if (!wait_warp(&ring->full[slot], (un / kUnits) & 1, wctl)) return false;
  const int4 a = ring->at[slot][0], c = ring->at[slot][1];
  __syncwarp();
  if (lane == 0) mbar_arrive(&ring->free[slot]);
  u = Unit{a.x, a.y, a.z, a.w, c.x, c.y, c.z & 1, c.z & 2};
  end = c.z < 0;
  return true;
}

// RL: the rows of a unit that there can be (of the R that a tile has columns for): the softmax's
// arithmetic runs on these alone.
// MULTI: several new positions under the causal rule: the rows of a block see different keys.
template <int HD, int R, int RL, bool MULTI>
__global__ void __launch_bounds__(Q8Layout<HD, R, RL>::THREADS, Q8Layout<HD, R, RL>::CTAS)
    q8_attn_kernel(const __grid_constant__ CUtensorMap mK, const __grid_constant__ CUtensorMap mV,
                   const Q8K p) {
  using LY = Q8Layout<HD, R, RL>;
  constexpr int KST = LY::KST, VST = LY::VST;
  constexpr int KCH = LY::KCH, CH = LY::CH, NS = LY::NS, NP = LY::NP;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint64_t k_full[KST], v_full[VST], k_empty[KST], v_empty[VST];
  __shared__ uint64_t s_full[2], s_free[2], p_full[2], p_done[2], q_full[2], q_free[2];
  __shared__ uint64_t drain_s, drain_o;
  __shared__ __align__(16) UnitRing units;
  __shared__ uint32_t tmem_base_s;
  __shared__ WaitCtl wctl;
  __shared__ int bad_input;
  __shared__ int page_s[kPageChunk];
  __shared__ __align__(16) float sc_s[2][2][kKT];  // key scale, log2 of the value scale
  // One of a tile's value scales is kApart below another. Read after s_free, so four tiles deep:
  // when the scores of two tiles before are read, the weights of three before are done.
  __shared__ int apart_s[4];
  __shared__ __align__(16) float qs_s[2][R];       // rows: score factor
  __shared__ __align__(16) int lim_s[2][R];        // and the keys they see: those below it
  __shared__ __align__(16) float nm_s[2][R], red_s[4][R];  // -m; maxima or sums of the warps
  __shared__ __align__(16) float up_s[R], f_s[R];  // how far m moves, and O's factors then

  const int warp = warp_id(), lane = lane_id();
  Walk w;
  if (warp == LY::QS_WARP) w.init(p, blockIdx.x, gridDim.x, lane);
  if (threadIdx.x == 0) {
    wait_ctl_init(&wctl, p.wait_limit_ns);
    bad_input = 0;
#pragma unroll 1
    for (int s = 0; s < KST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
#pragma unroll 1
    for (int s = 0; s < VST; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
    }
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      mbar_init(&s_full[s], 2);  // the MMA, and the scales of its keys
      mbar_init(&s_free[s], 4 * LY::NWG);
      mbar_init(&p_full[s], 4 * LY::NWG);
      mbar_init(&p_done[s], 1);
      mbar_init(&q_full[s], 1);
      mbar_init(&q_free[s], 1 + LY::NWG);
    }
#pragma unroll 1
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(&units.full[s], 1);
      mbar_init(&units.free[s], 3 + 4 * LY::NWG);
    }
    mbar_init(&drain_s, 1);
    mbar_init(&drain_o, 1);
    fence_barrier_init();
  }
  if (warp == LY::S_WARP) {
    tmem_alloc(&tmem_base_s, LY::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base_s;
  grid_dep_trigger();

  if (warp == 0 && blockIdx.x == 0) {  // lengths out of range are clamped, and reported here
    bool bad = false;
#pragma unroll 1
    for (int b = lane; b < p.B; b += 32) bad |= p.lens[b] != q8_len(p, b);
    if (bad) bad_input = 1;
  }

  if (warp == LY::TMA_WARP) {
    // ------------------------------------------------------------------ K and V copies
    const bool leader = lane == 0;
    if (leader) {
      tma_prefetch_desc(&mK);
      tma_prefetch_desc(&mV);
    }
    const int box = min(1 << p.ps_shift, kKT);  // rows of a box
    const int nsub = kKT / box;                 // boxes of a tile and chunk (<= 16)
    const int z_oob = p.num_pages * p.Hk;       // a page past the cache: zero fill
    const int sub = lane / KCH, c = lane % KCH; // this lane's box
    int g = 0, gk = 0, gv = 0;                  // tiles, and copies of K and V, so far
    int page_b = -1, page_lo = 0;               // page_s: entries page_lo .. of sequence page_b
    Unit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit(&units, un, w, end, lane, &wctl)) && !end; ++un) {
      const int used = (w.len + (1 << p.ps_shift) - 1) >> p.ps_shift;
      const int32_t* row = p.table + (size_t)w.b * p.max_pages;
#pragma unroll 1
      for (int j = w.ja; j < w.jb && ok; ++j, ++g) {
        const int n0 = j * kKT;
        const int p_lo = n0 >> p.ps_shift, p_hi = min(used - 1, (n0 + kKT - 1) >> p.ps_shift);
        if (page_b != w.b || p_lo < page_lo || p_hi >= page_lo + kPageChunk) {
          page_b = w.b;
          page_lo = p_lo;
          __syncwarp();
          const int n = min(kPageChunk, used - page_lo);
#pragma unroll 1
          for (int e = lane; e < n; e += 32) {
            int pg = row[page_lo + e];
            if (pg < 0 || pg >= p.num_pages) {
              pg = -1;
              bad_input = 1;
            }
            page_s[e] = pg;
          }
          __syncwarp();
        }
        const int key = n0 + sub * box;
        int z = z_oob, y = 0;
        if (sub < nsub && key < w.len) {
          const int pg = page_s[(key >> p.ps_shift) - page_lo];
          if (pg >= 0) {
            z = pg * p.Hk + w.kh;
            y = key & ((1 << p.ps_shift) - 1);
          }
        }
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          const int st = g % (which ? VST : KST);
          const uint32_t use = g / (which ? VST : KST);
          uint64_t* full = which ? &v_full[st] : &k_full[st];
          if (leader) {
            if (use > 0) ok = wait(which ? &v_empty[st] : &k_empty[st], (use - 1) & 1, &wctl);
            if (ok) mbar_arrive_expect_tx(full, LY::KV_BYTES);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          uint8_t* dst = smem + (which ? LY::OFF_V : LY::OFF_K) + st * LY::KV_BYTES +
                         c * (kKT * CH) + sub * box * CH;
          if (sub < nsub) tma_load_3d(dst, which ? &mV : &mK, full, c * CH, y, z);
          ++(which ? gv : gk);
        }
        if (!ok) break;
      }
    }
    if (leader) {  // no copy may be in flight when the CTA ends
#pragma unroll 1
      for (int s = 0; s < KST; ++s) {
        const int n = (gk - s + KST - 1) / KST;  // copies into stage s
        if (n > 0) mbar_wait_drain(&k_full[s], (n - 1) & 1);
      }
#pragma unroll 1
      for (int s = 0; s < VST; ++s) {
        const int n = (gv - s + VST - 1) / VST;
        if (n > 0) mbar_wait_drain(&v_full[s], (n - 1) & 1);
      }
    }
  } else if (warp == LY::S_WARP) {
    // ------------------------------------------------------------------ S^T = K q^T
    const uint32_t id = idesc_f8(0, 0, kKT, NS, 0, 0);
    int g = 0;
    Unit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit(&units, un, w, end, lane, &wctl)) && !end; ++un) {
      ok = wait_warp<false>(&q_full[un & 1], (un >> 1) & 1, &wctl);
      const Desc qb = q8_desc<CH>(smem_u32(smem + LY::OFF_Q + (un & 1) * LY::Q_BYTES), 0);
#pragma unroll 1
      for (int j = w.ja; j < w.jb && ok; ++j, ++g) {
        const int st = g % KST, buf = g & 1;
        ok = wait_warp(&k_full[st], (g / KST) & 1, &wctl) &&
             (g < 2 || wait_warp(&s_free[buf], ((g >> 1) - 1) & 1, &wctl));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const Desc ka = q8_desc<CH>(smem_u32(smem + LY::OFF_K + st * LY::KV_BYTES), 0);
          const uint32_t tS = tbase + LY::COL_S + buf * NS;
#pragma unroll
          for (int ks = 0; ks < HD / 32; ++ks) {
            const int ch = ks * 32 / CH, in = ks * 32 % CH;
            mma_f8(tS, ka.at(ch * (kKT * CH) + in), ka.hi, qb.at(ch * (NS * CH) + in), qb.hi, id,
                   ks > 0 ? 1u : 0u);
          }
          mma_commit(&s_full[buf]);
          mma_commit(&k_empty[st]);
        }
        __syncwarp();
      }
      // (arrives at once where the unit had no tile)
      if (ok && lane == 0) mma_commit(&q_free[un & 1]);
    }
    if (lane == 0) {
      mma_commit(&drain_s);
      mbar_wait_drain(&drain_s, 0);
    }
    __syncwarp();
  } else if (warp == LY::O_WARP) {
    // ------------------------------------------------------------------ O^T += V^T w^T
    constexpr int MV = HD < 128 ? HD : 128;  // head-dim rows of an MMA
    const uint32_t id = idesc_f8(0, 1, MV, NP, 1, 1);
    int g = 0;
    Unit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit(&units, un, w, end, lane, &wctl)) && !end; ++un) {
#pragma unroll 1
      for (int j = w.ja; j < w.jb; ++j, ++g) {
        const int st = g % VST, buf = g & 1, n0 = j * kKT;
        ok = wait_warp(&v_full[st], (g / VST) & 1, &wctl) &&
             wait_warp(&p_full[buf], (g >> 1) & 1, &wctl);
        if (!ok) break;
        uint8_t* vt = smem + LY::OFF_V + st * LY::KV_BYTES;
        if (n0 + kKT > w.len - (MULTI ? p.lq - 1 : 0)) {
          const int tail = min(w.len - n0, kKT), hidden = max(w.len - p.lq + 1 - n0, 0);
          if (MULTI && hidden < tail)
            clear_nan<HD, CH, RL, NP>(vt, smem + LY::OFF_P + buf * LY::P_BYTES, hidden, tail, n0,
                                      lim_s[un & 1], lane);
          if (tail < kKT) clear_rows<HD, CH>(vt, tail, kKT, lane);  // behind the sequence's end
          fence_proxy_async();
          __syncwarp();
        }
        tc_fence_after();
        if (lane == 0) {
          const Desc va = q8_desc<CH>(smem_u32(vt), kKT * CH);
          const Desc pb = q8_desc<NP>(smem_u32(smem + LY::OFF_P + buf * LY::P_BYTES), 0);
#pragma unroll
          for (int h = 0; h < KCH; ++h)
#pragma unroll
            for (int ks = 0; ks < kKT / 32; ++ks)
              mma_f8(tbase + LY::COL_O + h * NP, va.at(h * (kKT * CH) + ks * 32 * CH), va.hi,
                     pb.at(ks * 32 * NP), pb.hi, id, (j > w.ja || ks > 0) ? 1u : 0u);
          mma_commit(&p_done[buf]);
          mma_commit(&v_empty[st]);
        }
        __syncwarp();
      }
    }
    if (lane == 0) {
      mma_commit(&drain_o);
      mbar_wait_drain(&drain_o, 0);
    }
    __syncwarp();
  } else if (warp == LY::QS_WARP) {
    // ------------------------------------------------------------------ the units, their q in
    // two pieces and their keys' scales
    constexpr int LPR = HD / 8, RPS = 32 / LPR;  // lanes of a row (8 columns each), rows of a step
    constexpr int QSTEPS = RL <= RPS ? 1 : RL / RPS;
    const int nb_shift = p.ps_shift - p.sb_shift, ps_mask = (1 << p.ps_shift) - 1;
    const unsigned page_scales = (unsigned)p.Hk << nb_shift;  // of a page's heads
    int g = 0, published = 0;
    uint32_t largest = 0;  // bits of the scales read
    bool ok = true, ended = false;
#pragma unroll 1
    for (int un = -1; ok; ++un) {  // (-1: nothing but the first unit's publication)
      int4 ua = make_int4(0, 0, 0, 0), uc = ua;
      if (un >= 0) {
        ua = units.at[un % kUnits][0];
        uc = units.at[un % kUnits][1];
        if (uc.z < 0) break;  // the end
      }
      const int kh = ua.y, ja = ua.w, jb = uc.x, len = uc.y;
      if (un >= 0) {
        // ---- q: row r of the block in pieces hi (row r of the operand) and lo (row R + r)
        const int qb = un & 1;
        if (un >= 2 && !wait_warp(&q_free[qb], ((un >> 1) - 1) & 1, &wctl)) break;
        uint8_t* dst = smem + LY::OFF_Q + qb * LY::Q_BYTES;
        const int r0 = ua.z * R, live = min(RL, p.rows - r0);
        const int col = lane % LPR * 8, ch = col / CH, in = col % CH;
        const __nv_bfloat16* src = p.q + (((size_t)ua.x * p.Hk + kh) * p.rows + r0) * HD + col;
        auto row_of = [&](int step) { return step * RPS + lane / LPR; };
        auto load = [&](int step) {
          return row_of(step) < live
                     ? __ldg(reinterpret_cast<const uint4*>(src + (size_t)row_of(step) * HD))
                     : make_uint4(0u, 0u, 0u, 0u);
        };
        if (lane < R) {
          const int i = MULTI ? (r0 + lane) % p.lq : 0;
          lim_s[qb][lane] = min(MULTI ? max(0, len - p.lq + i + 1) : len, jb * kKT);
        }
        uint4 x = load(0), x1 = QSTEPS > 1 ? load(1) : x;
#pragma unroll 1
        for (int step = 0; step < QSTEPS; ++step) {
          const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
          x = x1;
          if (QSTEPS > 2) x1 = load(step + 2);
          uint32_t m = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) m = __vmaxu2(m, xs[e] & 0x7fff7fffu);
          m = max(m & 0xffffu, m >> 16);
#pragma unroll
          for (int o = LPR / 2; o > 0; o /= 2) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
          // 2^sh puts the row's largest element into [128, 256); a row with an element that is not
          // finite becomes NaN
          const int sh = 134 - (int)max(m >> 7, 1u), r = row_of(step);
          const float f0 = __int_as_float((sh / 2 + 127) << 23);
          const float f1 = __int_as_float((sh - sh / 2 + 127) << 23);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float u = __uint_as_float(xs[e] << 16) * f0 * f1;
            const float v = __uint_as_float(xs[e] & 0xffff0000u) * f0 * f1;
            hi[e] = m >= 0x7f80u ? 0x7f7fu : e4m3x2_from_f32(u, v);
            const float2 h = f32_from_e4m3x2(hi[e]);
            lo[e] = e4m3x2_from_f32((u - h.x) * 16.0f, (v - h.y) * 16.0f);
          }
          if (r < RL) {
            uint8_t* at = dst + ch * (NS * CH) + in % 16;
            *reinterpret_cast<uint2*>(at + r * CH + swz<CH>(in / 16, r) * 16) =
                make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
            *reinterpret_cast<uint2*>(at + (R + r) * CH + swz<CH>(in / 16, R + r) * 16) =
                make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
            if (lane % LPR == 0)
              qs_s[qb][r] = p.scale_log2 * __int_as_float((127 - sh / 2) << 23) *
                            __int_as_float((127 - (sh - sh / 2)) << 23);
          }
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[qb]);
      }
      // ---- two units ahead, so that the copies of the next units' keys can start
#pragma unroll 1
      while (!ended && published < un + (un < 0 ? 2 : 3)) {
        const int slot = published % kUnits;
        if (published >= kUnits)
          ok = wait_warp(&units.free[slot], (published / kUnits - 1) & 1, &wctl);
        if (!ok) break;
        ended = !w.template next<MULTI>(p, R);
        if (lane == 0) {
          units.at[slot][0] = make_int4(w.b, w.kh, w.rb, w.ja);
          units.at[slot][1] = make_int4(w.jb, w.len, ended ? -1 : w.whole | w.first << 1, 0);
          mbar_arrive(&units.full[slot]);
        }
        ++published;
      }
      __syncwarp();
      if (un < 0) continue;
      // ---- scales: a lane has four keys in a row. Those of two tiles are on their way in
      // registers (used where they were loaded to: a copy would wait for the load), and the table
      // entries of the two after them
      const int32_t* table = p.table + (size_t)ua.x * p.max_pages;
      const unsigned head_scales = (unsigned)kh << nb_shift;
      const int end_key = min(len, jb * kKT);
      const bool wide = p.sb_shift >= 2;  // the four keys have one scale
      float ks[2][4], vs[2][4];
      float most = -INFINITY;  // log2 of the unit's largest value scale so far
      int page[2] = {-1, -1};
#pragma unroll 1
      for (int j = ja - 4; j < jb && ok; j += 2) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (j + h >= ja && j + h < jb) {
            const int buf = g & 1;
            const float least = __int_as_float((kQ8MinExp + 127) << 23);
            float4 k4 = make_float4(ks[h][0], ks[h][0], ks[h][0], ks[h][0]);
            const float l0 = lg2(fmaxf(vs[h][0], least));
            float4 l4 = make_float4(l0, l0, l0, l0);
            float lo = l0, hi = l0;
            largest = max(largest, max(__float_as_uint(ks[h][0]), __float_as_uint(vs[h][0])));
            if (!wide) {
#pragma unroll
              for (int e = 1; e < 4; ++e)
                largest =
                    max(largest, max(__float_as_uint(ks[h][e]), __float_as_uint(vs[h][e])));
              k4 = make_float4(ks[h][0], ks[h][1], ks[h][2], ks[h][3]);
              l4 = make_float4(l0, lg2(fmaxf(vs[h][1], least)), lg2(fmaxf(vs[h][2], least)),
                               lg2(fmaxf(vs[h][3], least)));
              lo = fminf(fminf(l4.x, l4.y), fminf(l4.z, l4.w));
              hi = fmaxf(fmaxf(l4.x, l4.y), fmaxf(l4.z, l4.w));
            }
            most = fmaxf(most, warp_max(hi));
            const float below = warp_max(-lo) + most;
            if (g >= 2) ok = ok && wait_warp(&s_free[buf], ((g >> 1) - 1) & 1, &wctl);
            if (lane == 0) apart_s[g & 3] = below > kApart;
            ++g;
            *reinterpret_cast<float4*>(&sc_s[buf][0][lane * 4]) = k4;
            *reinterpret_cast<float4*>(&sc_s[buf][1][lane * 4]) = l4;
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_full[buf]);
          }
          const int key = (j + h + 2) * kKT + lane * 4;
          const bool have = page[h] >= 0 && page[h] < p.num_pages;  // (else zeros, or no key)
          const size_t at = (size_t)(unsigned)page[h] * page_scales +
                            (head_scales + ((key & ps_mask) >> p.sb_shift));
          ks[h][0] = have ? __ldg(p.k_scale + at) : 0.0f;
          vs[h][0] = have ? __ldg(p.v_scale + at) : 1.0f;
          if (!wide) {
#pragma unroll
            for (int e = 1; e < 4; ++e) {
              const bool here = have && key + e < end_key;
              ks[h][e] = here ? __ldg(p.k_scale + at + (e >> p.sb_shift)) : 0.0f;
              vs[h][e] = here ? __ldg(p.v_scale + at + (e >> p.sb_shift)) : 1.0f;
            }
          }
          page[h] = key + 2 * kKT < end_key && j + h + 4 >= ja
                        ? table[(key + 2 * kKT) >> p.ps_shift] : -1;
        }
      }
    }
    if (largest > kQ8MaxScale) bad_input = 1;
  } else {
    // ------------------------------------------------------------------ softmax, and O out.
    // A warpgroup has the rows row0 .. row0 + 7 of the block (RW of them at most; with 16 rows two
    // groups share the latency of a tile: 46 us for a chunk of 32 positions, 49 with one group of
    // 16 rows). Rows that are not there (live of the RW are) have columns of q, S, w and O that
    // hold anything (NaN too) and are never used. A wait that runs out shows at the next
    // softmax_any, where all threads leave together.
    constexpr int RW = RL < 8 ? RL : 8;
    const int wg = LY::NWG == 1 ? 0 : warp >> 2, wl = warp & 3, row0 = wg * 8;
    const int key = threadIdx.x & 127;  // key of the tile
    const uint32_t lanes = tbase + ((uint32_t)(wl * 32) << 16);
    const uint64_t sixteenth = f2_pack(0.0625f, 0.0625f);
    int g = 0;
    Unit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0;; ++un) {
      const int qb = un & 1;
      ok = take_unit(&units, un, w, end, lane, &wctl);
      if (ok && !end) ok = wait_warp(&q_full[qb], (un >> 1) & 1, &wctl);
      if (softmax_any(wg, !ok) || end) break;
      const int r0 = w.rb * R + row0, live = min(RW, p.rows - r0);
      // tiles below lim_min need no test of the keys
      const int lim_min = min(MULTI ? max(0, w.len - p.lq + 1) : w.len, w.jb * kKT);
      float l[RW];
#pragma unroll
      for (int r = 0; r < RW; ++r) l[r] = 0.0f;
#pragma unroll 1
      for (int j = w.ja; j < w.jb; ++j, ++g) {
        const int buf = g & 1;
        const uint32_t ph = (g >> 1) & 1;
        ok = ok && wait_warp(&s_full[buf], ph, &wctl);
        tc_fence_after();
        uint32_t sr[16];  // hi of the 8 rows, lo
        load_scores<R>(lanes + LY::COL_S + buf * NS + row0, sr);
        const float kc = sc_s[buf][0][key], lsv = sc_s[buf][1][key];
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[buf]);
        const bool first = j == w.ja;
        float t[RW];
        const uint64_t kc2 = f2_pack(kc, kc), lsv2 = f2_pack(lsv, lsv);
#pragma unroll
        for (int r = 0; r < RW; r += 2) {
          const uint64_t qs = *reinterpret_cast<const uint64_t*>(&qs_s[qb][row0 + r]);
          const uint64_t nm =
              first ? 0ull : *reinterpret_cast<const uint64_t*>(&nm_s[qb][row0 + r]);
          const uint64_t hi = f2_pack(__uint_as_float(sr[r]), __uint_as_float(sr[r + 1]));
          const uint64_t lo = f2_pack(__uint_as_float(sr[8 + r]), __uint_as_float(sr[9 + r]));
          const uint64_t s = f2_mul(f2_fma(lo, sixteenth, hi), kc2);
          f2_unpack(f2_fma(s, qs, f2_add(lsv2, nm)), t[r], t[r + 1]);
        }
        if (j * kKT + kKT > lim_min) {
#pragma unroll
          for (int r = 0; r < RW; ++r)
            if (j * kKT + key >= (MULTI ? lim_s[qb][row0 + r] : lim_min)) t[r] = -INFINITY;
        }
        float top = t[0];
#pragma unroll
        for (int r = 1; r < RW; r += 2)
          top = r + 1 < RW ? fmax3(top, t[r], t[r + 1]) : fmaxf(top, t[r]);
        if (softmax_any(wg, top > kMost || first || !ok)) {
          // m moves: to the largest score so far, at a unit's first tile to the tile's own
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            const float mx = warp_max(t[r]);
            if (lane == 0) red_s[wl][row0 + r] = mx;
          }
          if (softmax_any(wg, !ok)) {
            ok = false;
            break;
          }
          if (key < RW) {
            const int r = row0 + key;
            const float mx =
                fmaxf(fmaxf(red_s[0][r], red_s[1][r]), fmaxf(red_s[2][r], red_s[3][r]));
            float up = mx - kTop;
            if (first ? mx == -INFINITY : !(up > 0.0f)) up = 0.0f;
            nm_s[qb][r] = first ? -up : nm_s[qb][r] - up;
            up_s[r] = up;
            f_s[r] = ex2(-up);
          }
          if (!first) {  // O is scaled too, once the last O^T MMA is done
            ok = wait_warp(&p_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &wctl);
            tc_fence_after();
          }
          softmax_any(wg, false);
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            t[r] -= up_s[row0 + r];
            if (!first) l[r] = scale_sum(l[r], up_s[row0 + r]);
          }
          if (!first) {
#pragma unroll 1
            for (int h = 0; h < 3 * KCH; ++h) {  // (f_s beyond RW: any)
              const uint32_t at = lanes + LY::COL_O + h / 3 * NP + h % 3 * R + row0;
              float x[8];
              tmem_ld8(at, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] *= f_s[row0 + e];
              tmem_st8(at, x);
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        // weights, their sum, and their pieces into shared memory, a key's row of NP bytes
        float inv = ex2(-lsv - kSumExp);  // 1 / value scale, in the sum's unit
        if (apart_s[g & 3]) {
          inv = 0.0f;
#pragma unroll
          for (int r = 0; r < RW; ++r) l[r] += ex2_full(t[r] - lsv - kSumExp);
        }
        if (g >= 2) ok = ok && wait_warp(&p_done[buf], ph ^ 1, &wctl);
        uint32_t pc[3][2];
#pragma unroll
        for (int r = 0; r < RW; r += 4) {
          uint32_t x[2];
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            if (r + e >= RW) {
              x[e / 2] = 0u;
              continue;
            }
            const float a = ex2(t[r + e]), b = ex2(t[r + e + 1]);
            l[r + e] = fmaf(a, inv, l[r + e]);
            l[r + e + 1] = fmaf(b, inv, l[r + e + 1]);
            x[e / 2] = weight_f16x2(a, b);
          }
#pragma unroll
          for (int i = 0; i < 3; ++i) {
            pc[i][r / 4] = __byte_perm(x[0], x[1], 0x7531);
            x[0] = f16x2_rest(x[0]);
            x[1] = f16x2_rest(x[1]);
          }
        }
        uint8_t* prow = smem + LY::OFF_P + buf * LY::P_BYTES + key * NP;
        if constexpr (RW <= 4) pc[0][1] = pc[1][1] = pc[2][1] = 0u;
        if constexpr (R == 8) {
          *reinterpret_cast<uint4*>(prow + swz<NP>(0, key) * 16) =
              make_uint4(pc[0][0], pc[0][1], pc[1][0], pc[1][1]);
          *reinterpret_cast<uint2*>(prow + swz<NP>(1, key) * 16) = make_uint2(pc[2][0], pc[2][1]);
        } else {
#pragma unroll
          for (int i = 0; i < 3; ++i)
            *reinterpret_cast<uint2*>(prow + swz<NP>(i, key) * 16 + row0) =
                make_uint2(pc[i][0], pc[i][1]);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      // the sums of the 128 threads
      const bool any = w.jb > w.ja;
#pragma unroll
      for (int r = 0; r < RW; ++r) {
        float x = l[r];
#pragma unroll
        for (int o = 16; o > 0; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (lane == 0) red_s[wl][row0 + r] = x;
      }
      if (any && ok) ok = wait_warp(&p_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &wctl);
      if (softmax_any(wg, !ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      // a row without keys: sum 0, and O (whose columns may hold anything then) 0
      const size_t unit_row = ((size_t)w.b * p.Hk + w.kh) * p.rows + r0;
      const size_t part = 2 * (size_t)blockIdx.x + (w.first ? 1 : 0);
      // this thread's head-dim row: a 64-row accumulator lies in lanes 0-15 of each warp
      const int col = HD == 64 ? wl * 16 + lane : key;
      const bool mine = HD > 64 || lane < 16;
      const size_t out_row = w.whole ? unit_row : part * R + row0;
#pragma unroll 1
      for (int h = 0; h < KCH; ++h) {
        float x[8], y[8], z[8];
        if (any) {
          const uint32_t at = lanes + LY::COL_O + h * NP + row0;
          tmem_ld8(at, x);
          tmem_ld8(at + R, y);
          tmem_ld8(at + 2 * R, z);
          tmem_wait_ld();
        }
        size_t at = out_row * HD + h * 128 + col;
#pragma unroll
        for (int e = 0; e < RW; ++e, at += HD) {
          const int r = row0 + e;
          const float sum = (red_s[0][r] + red_s[1][r]) + (red_s[2][r] + red_s[3][r]);
          float o = fmaf(fmaf(z[e], 0.125f, y[e]), 0.125f, x[e]);
          if (w.whole) o = __fdividef(o, sum) / kSumUnit;  // (2 ulp; o is rounded to bf16)
          if (sum == 0.0f) o = 0.0f;
          if (e < live && mine) {
            if (w.whole)
              p.o[at] = __float2bfloat16(o);
            else
              p.o_part[at] = o;
          }
        }
      }
      if (key < live) {
        const int r = row0 + key;
        const float sum = (red_s[0][r] + red_s[1][r]) + (red_s[2][r] + red_s[3][r]);
        const float m = any ? -nm_s[qb][r] : 0.0f;
        if (!w.whole) {
          p.ml_part[part * 2 * R + r] = m;
          p.ml_part[part * 2 * R + R + r] = sum;
        } else if (p.lse) {
          p.lse[unit_row + key] = sum == 0.0f ? -INFINITY : fmaf(m + kSumExp, kLn2, logf(sum));
        }
      }
      // (the next unit has the other half of nm_s, and writes red_s behind its first vote)
      tc_fence_before();
      if (key == 0) mbar_arrive(&q_free[qb]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == LY::S_WARP) tmem_dealloc(tbase, LY::TMEM_COLS);
  if (threadIdx.x == 0) {
    report_abort(&wctl, p.status);
    if (bad_input && p.status) atomicCAS(p.status, kStatusOk, kStatusBadInput);
  }
}

}  // namespace
}  // namespace fa

#include "fa_q8_chunk.cuh"

namespace fa {
namespace {

// Joins the shares of the units that were cut, and writes those of sequences without keys: a warp
// for each row, a CTA for (up to) 8 rows of a unit. Launched early: what it needs to know of the
// lengths it works out while the attention still runs. Then only latency counts (a few KB): a lane
// reads one share's m and sum, and the first shares' O is on its way before their weights are
// known.
template <int HD, int R>
__global__ void __launch_bounds__(256) q8_combine_kernel(const Q8K p, int grid) {
  const int warp = warp_id(), lane = lane_id();
  const unsigned U = (unsigned)(p.Hk * p.rb);  // blockIdx.x: (b * Hk + kh) * rb + row block
  const int b = (int)(blockIdx.x / U), in = (int)(blockIdx.x % U);
  const int kh = p.rb == 1 ? in : in / p.rb, rb = in - kh * p.rb;
  const int r0 = rb * R, live = min(R, p.rows - r0);
  const size_t unit_row = ((size_t)b * p.Hk + kh) * p.rows + r0;
  // every warp finds the unit's place in the list for itself
  unsigned before = 0;
  int mine = lane < p.B ? q8_cost(p, lane) : 0;
  const int cost = q8_cost(p, b);
  before = lane < b ? mine : 0;
#pragma unroll 1
  for (int i = lane + 32; i < b; i += 32) before += q8_cost(p, i);
  before = __reduce_add_sync(0xffffffffu, before);
  const unsigned per = q8_share((unsigned)q8_all_costs(p, mine, lane) * U, grid);
  if (cost == 0 && blockIdx.y == 0) {
    for (int e = threadIdx.x; e < live * HD; e += blockDim.x)
      p.o[unit_row * HD + e] = __float2bfloat16(0.f);
    if (p.lse)
      for (int e = threadIdx.x; e < live; e += blockDim.x) p.lse[unit_row + e] = -INFINITY;
  }
  // (by every CTA: what follows this kernel must find the attention done)
  grid_dep_wait();
  if (cost == 0) return;
  const unsigned a = before * U + (unsigned)in * cost;  // of its first tile and of its last:
  const int c0 = (int)((a + kUnitCost) / per), c1 = (int)((a + cost - 1) / per);
  if (c0 == c1) return;  // written whole
  // share i: slot 2 c0 + 1 (it begins there), then 2 c of each further CTA
  auto slot = [&](int c) { return (size_t)2 * c + (c == c0 ? 1 : 0); };
  const int r = (int)blockIdx.y * 8 + warp;
  if (r >= live) return;
  constexpr int CPL = HD / 32, AHEAD = 4;  // columns of a lane
  struct Part {
    float x[CPL];
  };
  auto load = [&](int c) {
    Part v;
    const float* src = p.o_part + (slot(min(c, c1)) * R + r) * HD + lane * CPL;
    if constexpr (CPL == 2) {
      const float2 f = *reinterpret_cast<const float2*>(src);
      v.x[0] = f.x, v.x[1] = f.y;
    } else {
#pragma unroll
      for (int e = 0; e < CPL; e += 4) {
        const float4 f = *reinterpret_cast<const float4*>(src + e);
        v.x[e] = f.x, v.x[e + 1] = f.y, v.x[e + 2] = f.z, v.x[e + 3] = f.w;
      }
    }
    return v;
  };
  float m = -FLT_MAX, sum = 0.0f, acc[CPL] = {};
#pragma unroll 1
  for (int base = c0; base <= c1; base += 32) {
    const int n = min(32, c1 - base + 1);
    float mi = -FLT_MAX, li = 0.0f;
    if (lane < n) {
      const float* ml = p.ml_part + slot(base + lane) * 2 * R + r;
      li = ml[R];
      if (li != 0.0f) mi = ml[0];
    }
    Part v[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) v[k] = load(base + k);
    float top = fmaxf(m, mi);
#pragma unroll
    for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float f = li == 0.0f ? 0.0f : ex2(mi - top), old = ex2(m - top);
    float part = scale_sum(li, top - mi);  // (0 stays 0)
    sum = scale_sum(sum, top - m);
    m = top;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) part += __shfl_xor_sync(0xffffffffu, part, o);
    sum += part;
#pragma unroll
    for (int e = 0; e < CPL; ++e) acc[e] *= old;
#pragma unroll 1
    for (int k0 = 0; k0 < n; k0 += AHEAD) {
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const float fk = __shfl_sync(0xffffffffu, f, k0 + k);  // (0 behind the last share)
        if (fk != 0.0f) {
#pragma unroll
          for (int e = 0; e < CPL; ++e) acc[e] = fmaf(v[k].x[e], fk, acc[e]);
        }
        v[k] = load(base + k0 + AHEAD + k);
      }
    }
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum / kSumUnit;
  uint32_t out[CPL / 2];
#pragma unroll
  for (int e = 0; e < CPL / 2; ++e) out[e] = pack_bf16(acc[2 * e] * inv, acc[2 * e + 1] * inv);
  __nv_bfloat16* dst = p.o + (unit_row + r) * HD + lane * CPL;
  if constexpr (CPL == 2)
    *reinterpret_cast<uint32_t*>(dst) = out[0];
  else if constexpr (CPL == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(out[0], out[1]);
  else
    *reinterpret_cast<uint4*>(dst) = make_uint4(out[0], out[1], out[2], out[3]);
  if (p.lse && lane == 0)
    p.lse[unit_row + r] = sum == 0.0f ? -INFINITY : fmaf(m + kSumExp, kLn2, logf(sum));
}

// Rows a kv head from which blocks of 128 rows are taken (head_dim 64 and 128 alone: at 256 that
// kernel's layout, with weights beside the scores and tiles of 128 keys, has neither the tensor
// memory nor the shared memory, and none with weights over their scores and tiles of 64 keys is
// written; more rows there read the keys again for every 16: 128 rows 814 us, 512 rows 3172). A tile
// of 128 keys takes the same time for any number of its rows, a block of 16 not half of that. 16
// sequences of 4k to 16k keys, 8 kv heads, head_dim 128, blocks of 16 against those of 128: 32 rows
// 115 / 128 us, 40 rows 156 / 128, 128 rows 399 / 139, 512 rows 1461 / 500; head_dim 64: 100 / 107,
// 141 / 108, 355 / 112, 1369 / 411.
constexpr int kChunkRows = 33;

struct Plan {
  int R, RL, rb, grid;
};

// Rows of a unit: the smallest block of 8, 16 or 128 that holds the G * q_len rows of a kv head,
// but 16 up to 32 rows; more rows take further passes over the keys, from L2. Grid: every CTA slot
// of the GPU, or one CTA for each tile there can be.
Plan make_plan(const Q8AttnArgs& a) {
  Plan pl;
  const int rows = a.G * a.lq;
  pl.R = rows <= 8 ? 8 : rows < kChunkRows || a.d > 128 ? 16 : 128;
  pl.RL = rows <= 2 ? 2 : rows <= 4 ? 4 : pl.R;
  pl.rb = (rows + pl.R - 1) / pl.R;
  const int ctas = 152 * (a.d > 128 || pl.R > 16 ? 1 : a.d == 64 && pl.RL <= 4 ? 3 : 2);
  const long long cap = (long long)a.max_pages << a.ps_shift;
  const long long tiles = ((cap + kKT - 1) / kKT + kUnitCost) * a.B * a.Hk * pl.rb;
  pl.grid = (int)std::min<long long>(ctas, tiles);
  return pl;
}

template <int HD, int R, int RL, bool MULTI>
cudaError_t attn_m(const Q8AttnArgs& a, const Q8AttnMaps& m, const Plan& pl, void* ws,
                   cudaStream_t s) {
  static OncePerKey<> smem_attr;
  cudaError_t e;
  Q8K p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.codes[0] = a.k;
  p.codes[1] = a.v;
  p.k_scale = a.k_scale;
  p.v_scale = a.v_scale;
  p.table = a.table;
  p.lens = a.lens;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.ml_part = static_cast<float*>(ws);
  p.o_part = p.ml_part + (size_t)2 * pl.grid * 2 * R;
  p.status = a.status;
  p.B = a.B;
  p.Hk = a.Hk;
  p.lq = a.lq;
  p.rows = a.G * a.lq;
  p.rb = pl.rb;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.ps_shift = a.ps_shift;
  p.sb_shift = a.sb_shift;
  p.scale_log2 = a.scale * kLog2e;
  p.wait_limit_ns = a.wait_limit_ns;
  if constexpr (R == 128) {
    using LY = Q8Chunk<HD>;
    auto kern = q8_chunk_kernel<HD, MULTI>;
    if ((e = set_smem_once(smem_attr, kern, LY::SMEM_BYTES)) != cudaSuccess) return e;
    profile_mark(kKernQ8Attn, 0, s);
    kern<<<pl.grid, LY::THREADS, LY::SMEM_BYTES, s>>>(p);
  } else {
    using LY = Q8Layout<HD, R, RL>;
    auto kern = q8_attn_kernel<HD, R, RL, MULTI>;
    if ((e = set_smem_once(smem_attr, kern, LY::SMEM_BYTES)) != cudaSuccess) return e;
    profile_mark(kKernQ8Attn, 0, s);
    kern<<<pl.grid, LY::THREADS, LY::SMEM_BYTES, s>>>(m.k, m.v, p);
  }
  e = cudaGetLastError();
  profile_mark(kKernQ8Attn, 1, s);
  if (e != cudaSuccess) return e;
  profile_mark(kKernQ8Combine, 0, s);
  const int rows = p.rows < R ? p.rows : R;
  e = launch_pdl(q8_combine_kernel<HD, R>,
                 dim3((unsigned)(a.B * a.Hk * pl.rb), (unsigned)((rows + 7) / 8)),
                 dim3((unsigned)(32 * (rows < 8 ? rows : 8))), 0, s, p, pl.grid);
  profile_mark(kKernQ8Combine, 1, s);
  return e;
}

template <int HD, int R, int RL>
cudaError_t attn_t(const Q8AttnArgs& a, const Q8AttnMaps& m, const Plan& pl, void* ws,
                   cudaStream_t s) {
  return a.causal && a.lq > 1 ? attn_m<HD, R, RL, true>(a, m, pl, ws, s)
                              : attn_m<HD, R, RL, false>(a, m, pl, ws, s);
}

template <int HD>
cudaError_t attn_d(const Q8AttnArgs& a, const Q8AttnMaps& m, const Plan& pl, void* ws,
                   cudaStream_t s) {
  switch (pl.RL) {
    case 2: return attn_t<HD, 8, 2>(a, m, pl, ws, s);
    case 4: return attn_t<HD, 8, 4>(a, m, pl, ws, s);
    case 8: return attn_t<HD, 8, 8>(a, m, pl, ws, s);
    case 16: return attn_t<HD, 16, 16>(a, m, pl, ws, s);
    default: break;
  }
  if constexpr (HD <= 128) return attn_t<HD, 128, 128>(a, m, pl, ws, s);
  return cudaErrorInvalidValue;
}
}  // namespace

int q8_box_rows(int page_size) { return page_size < kKT ? page_size : kKT; }
int q8_box_cols(int head_dim) { return head_dim < 128 ? head_dim : 128; }

long long q8_attn_tiles(const Q8AttnArgs& a) {
  const long long cap = (long long)a.max_pages << a.ps_shift;
  const int blocks = (a.G * a.lq + 15) / 16;  // (fewer with larger blocks)
  return (long long)a.B * a.Hk * blocks * ((cap + kKT - 1) / kKT + kUnitCost);
}

size_t q8_attn_workspace_bytes(const Q8AttnArgs& a) {
  const Plan pl = make_plan(a);
  return (size_t)2 * pl.grid * pl.R * (a.d + 2) * 4;
}

cudaError_t launch_q8_attn(const Q8AttnArgs& a, const Q8AttnMaps& m, void* ws, cudaStream_t s) {
  const Plan pl = make_plan(a);
  switch (a.d) {
    case 64: return attn_d<64>(a, m, pl, ws, s);
    case 128: return attn_d<128>(a, m, pl, ws, s);
    case 256: return attn_d<256>(a, m, pl, ws, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
