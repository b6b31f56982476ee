// fa_tree.cu -- attention of a tree of drafted tokens over the paged bf16 key/value cache, sm_103a.
//
// The T nodes of a sequence's tree are its last T keys, and its T query rows. A node sees every key
// before them, and of them those that its row of the mask names (its ancestors and itself):
//   visible(i, j) = j < len - T  or  mask[i][j - (len - T)] != 0      (0 <= j < len)
//   O_i = sum_j exp(s_ij - L_i) v_j,  s_ij = scale <q_i, k_j>,  L_i = log sum_j exp(s_ij)
// A node that sees no key gives O = 0 and L = -inf.
//
// The G query heads of a kv head and the T nodes are rows of one product, so that a key is read once
// for all of them; with 4 d bytes and 4 d flops a row for each key, HBM bounds it up to some 280 rows
// a kv head. S = Q K^T (M = 128 rows, N = 64 keys) and O += P V, with P over S in tensor memory (two
// buffers); a thread of the softmax has a row; the lazy rescale of the training forward. Scores, maxima,
// sums and O are f32. P is rounded to bf16, the type that the product takes beside V's; its sum is of
// what was not rounded. (As in the training forward. O is off by 0.0021 to 0.0023, root mean square
// relative to its formula in 64 bits; by 0.0017, its own rounding, were P exact, which would take a
// second product for what the rounding leaves.) What has to fit beside the bytes of a tile is a chain of
// latencies (scores, softmax, weights), so:
//  * up to 128 rows, head_dim 64 and 128: two CTAs an SM with 128 rows each, which fill each other's
//    waits and the starts and ends of each other's units. (One CTA with two softmax warpgroups on the
//    halves of 128-key tiles, an O each, joined at a unit's end, and rings 1.4 times as deep: 132 us
//    for 125 for 16 sequences of up to 16k keys with 128 rows, 350 for 342 for 64 with 48, 61 for 43
//    at head_dim 64.)
//  * at head_dim 64 with up to 64 (32) rows these are there twice (four times): a copy has a half (a
//    quarter) of a tile's keys, with a maximum, a sum and an O of its own; four warps share a tile's
//    exponentials then instead of two or one. They are joined at a unit's end, through shared memory.
//  * more rows: one CTA, whose two warpgroups have 128 of a block's 256 rows each, on the same keys
//    (two CTAs of 128 rows, which read keys again: 101 us for 90 for 16 sequences of up to 8k keys).
//    At head_dim 256 tensor memory holds one O: one warpgroup, blocks of 128 rows, one CTA.
//
// Work: the (sequence, kv head, row block) units, each ceil(len / 64) key tiles, form one list of
// tiles, cut evenly over persistent CTAs (the lengths are on the device; each CTA finds
// its part from them). A unit counts kUnitCost tiles more than it has, what its start and end cost. A
// CTA writes the units it has whole; of the others it leaves its share's O, m and sum, which a second
// kernel joins in the order of the keys. Where the table has room for a few tiles only (kWholeKeys) a
// unit is its first tile's CTA's, whole: cutting it would cost more than it evens out, and the second
// kernel and the scratch are saved.
//
// Warps: 0-3 (0-7) softmax, then one each for the copies of K pages, of V pages, for S, for O, and for
// the list: it walks the list ahead of the others (two units where two Q are held, else one), loads Q
// and packs the tree's mask into words. A page's part of a tile is one TMA box, min(page_size, 64) rows
// of all columns: what limits small copies is the number of them a warp can issue (copies alone, 131072
// keys of 8 heads, head_dim 128, pages of 16: 4.6 TB/s with a box for each 64 columns, 5.7 with one
// box, 6.3 with a warp each for K and V; pages of 8: 3.0, 4.2, 5.7). The mask is tested in the tiles of
// the last T keys alone.
// There a value that is not finite must meet no weight of a row that does not see it, not even 0: a
// last warp looks those tiles over as they land and clears it, and rows that see it get it added at the
// end (tree_odd). What every row sees, the values before the tree, is put right when all is done
// (tree_mend).
#include <float.h>

#include <algorithm>

#include "fa_common.cuh"
#include "fa_launch.h"
#include "fa_wait.cuh"

namespace fa {

namespace {
constexpr int kKT = 64;          // keys of a tile
// Tiles' worth of a unit's start and end (16 sequences of up to 8k keys, 256 rows, head_dim 128: 92 us
// with 3, 85 with 5, 82 with 8; 100 of up to 2k, 17 rows, head_dim 64: 51.0, 51.6, 53.2).
constexpr int kUnitCost = 5;
constexpr int kWholeKeys = 512;  // room of a table up to which units are not cut (see tree_plan)
constexpr int kPageChunk = 128;  // block-table entries staged at a time
constexpr int kUnits = 3;        // units published
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;

// C copies of a unit's rows, CT CTAs on an SM.
template <int HD, int C, int CT>
struct TreeLayout {
  static constexpr int NWG = HD <= 128 && CT == 1 ? 2 : 1;  // softmax warpgroups
  static constexpr int RC = 128 / C;                 // query rows of a copy
  static constexpr int ROWS = RC * NWG;              // of a unit
  static constexpr int NC = kKT / C;                 // keys of a tile that a thread has
  // Stages of the rings; V has more where there is room, as a V stage stays until the weights of its
  // keys are there.
  static constexpr int KST = HD == 64 ? (C > 1 ? 3 : CT == 2 ? 4 : 8) : HD == 128 && CT == 1 ? 4 : 2;
  static constexpr int VST = HD == 64 ? (CT == 2 ? 4 : 12) : KST;
  // Units whose Q is held: a second one costs stages. (Its load runs beside a unit's last softmax.)
  static constexpr int QB = HD == 64 && CT == 2 ? 2 : 1;
  static constexpr int KCH = HD / 64;
  static constexpr int Q_BYTES = 128 * HD * 2;       // of 128 rows
  static constexpr int ST_BYTES = kKT * HD * 2;
  static constexpr int OFF_K = (NWG == 1 ? QB : NWG) * Q_BYTES;
  static constexpr int OFF_V = OFF_K + KST * ST_BYTES;
  static constexpr int OFF_JOIN = OFF_V + VST * ST_BYTES;  // 32 columns of the copies' O
  static constexpr int OFF_BITS = OFF_JOIN + (C > 1 ? 128 * 128 : 0);  // the masks' words
  static constexpr int COL_S = NWG * HD;             // O of each warpgroup, then its two S (and P)
  static constexpr int TMEM_COLS = 512 / CT;
  static constexpr int SOFT = 4 * NWG;
  static constexpr int K_WARP = SOFT, V_WARP = SOFT + 1, S_WARP = SOFT + 2, O_WARP = SOFT + 3,
                       LIST_WARP = SOFT + 4, FIX_WARP = SOFT + 5;
  static constexpr int THREADS = 32 * (SOFT + 6);
  static __device__ __forceinline__ uint32_t col_s(int w, int b) { return COL_S + (w * 2 + b) * kKT; }
  static_assert(C == 1 || (CT == 2 && HD == 64), "not a variant");
  static_assert(COL_S + NWG * 2 * kKT <= TMEM_COLS, "TMEM budget");
  static constexpr int T_MAX = CT == 2 ? RC : kTreeMax;
  static constexpr int smem_bytes(int T) {
    return OFF_BITS + kUnits * T * ((T + 31) / 32) * 4 + 1024;
  }
  // (and what is static, and the driver's 1 KB)
  static_assert((smem_bytes(T_MAX) + 4096 + 1024) * CT <= 228 * 1024, "shared memory budget");
};

struct TreeK {
  const __nv_bfloat16* v;  // the cache, for values that are not finite
  const int32_t* table;
  const int32_t* lens;
  const uint8_t* mask;
  long long mask_stride;
  __nv_bfloat16* o;
  float* lse;      // [B, H, T]
  float* o_part;   // [2 * grid, HD / 4, ROWS, 4]: O of a share, in units of 2^m
  float* ml_part;  // [2 * grid, 2, ROWS]: m and the sum
  int* status;
  int B, Hk, T, words, rows, rb, max_pages, num_pages, ps_shift;
  int cut;  // units may be shared by CTAs
  float scale_log2;
  unsigned long long wait_limit_ns;
};

__device__ __forceinline__ int tree_len(const TreeK& p, int b) {
  const long long cap = (long long)p.max_pages << p.ps_shift;
  const int raw = p.lens[b];
  return raw < 0 ? 0 : raw > cap ? (int)cap : raw;
}
// What a unit of sequence b counts in the list; 0 without keys.
__device__ __forceinline__ int tree_cost(const TreeK& p, int b) {
  const int len = tree_len(p, b);
  return len > 0 ? (len + kKT - 1) / kKT + kUnitCost : 0;
}
// The sum over all sequences (of one unit each), by one warp that has that of sequence `lane`. The
// host has checked that the whole list, Hk * rb times as long, fits 31 bits.
__device__ __forceinline__ unsigned tree_all(const TreeK& p, int mine, int lane) {
#pragma unroll 1
  for (int b = lane + 32; b < p.B; b += 32) mine += tree_cost(p, b);
  return __reduce_add_sync(0xffffffffu, (unsigned)mine);
}
__device__ __forceinline__ unsigned tree_share(unsigned all, unsigned grid) {
  return (all + grid - 1) / grid;
}

// The units of a CTA's share [t, t1) of the list, in order (warp-wide).
struct TreeWalk {
  unsigned t, t1;      // next place in the list, end of the share
  unsigned pre;        // the list before sequence b
  int b, cost, len;    // sequence, what each of its units counts, its length
  int kh, rb, ja, jb;  // the unit found: kv head, row block, tiles [ja, jb)
  int whole, first;    // the share has all of the unit's tiles, its first one

  __device__ __forceinline__ void init(const TreeK& p, unsigned cta, unsigned grid, int lane) {
    const unsigned U = (unsigned)(p.Hk * p.rb);
    const int mine = lane < p.B ? tree_cost(p, lane) : 0;
    const unsigned all = tree_all(p, mine, lane) * U;
    const unsigned per = tree_share(all, grid);
    t = per * cta;  // (below all + grid)
    t1 = min(t + per, all);
    pre = 0;
    b = cost = len = 0;
    if (t >= t1) return;
#pragma unroll 1
    for (int base = 0;; base += 32) {  // ends: t lies below the sum over all sequences
      const unsigned n =
          (base == 0 ? mine : base + lane < p.B ? tree_cost(p, base + lane) : 0) * U;
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
    len = tree_len(p, b);
    cost = tree_cost(p, b);
  }

  // The next unit that has tiles in the share; false where there is none.
  __device__ __forceinline__ bool next(const TreeK& p) {
    const unsigned U = (unsigned)(p.Hk * p.rb);
    do {  // (a share may end within what a unit counts before its tiles)
      if (t >= t1) return false;
#pragma unroll 1
      while (t >= pre + U * cost) {  // the next sequence with keys
        pre += U * cost;
        if (++b >= p.B) return false;
        len = tree_len(p, b);
        cost = tree_cost(p, b);
      }
      const unsigned in = t - pre, u = in / (unsigned)cost;
      kh = (int)u;
      const int from = (int)(in - u * cost);
      const int to = p.cut ? min(cost, from + (int)(t1 - t)) : cost;
      t += to - from;
      if (!p.cut && from > 0) {  // the CTA's before
        jb = 0;
        continue;
      }
      ja = max(0, from - kUnitCost);
      jb = max(0, to - kUnitCost);
    } while (jb == 0);
    rb = 0;
    if (p.rb > 1) {
      const int u = kh;
      kh = (int)((unsigned)u / (unsigned)p.rb);
      rb = u - kh * p.rb;
    }
    first = ja == 0;
    whole = first && jb == cost - kUnitCost;
    return true;
  }
};

// Units in shared memory: the last warp publishes, the others read; the softmax's warps free a slot
// when they are done with the unit (its mask words are in the slot), the others at once.
struct TreeUnit {
  int b, kh, rb, ja, jb, len, whole, first;
};
struct TreeRing {
  int4 at[kUnits][2];
  uint64_t full[kUnits], free[kUnits];
  uint64_t bits_full[kUnits];       // the mask's words are there
  uint64_t odd_full[kUnits];        // the unit's tree has been looked over
  unsigned odd[kUnits][kTreeMax / 32];  // nodes whose values are not all finite
};
template <bool FREE>
__device__ __forceinline__ bool take_unit(TreeRing* ring, int un, TreeUnit& u, bool& end, int lane,
                                          WaitCtl* wctl) {
  const int slot = un % kUnits;
  if (!wait_warp(&ring->full[slot], (un / kUnits) & 1, wctl)) return false;
  const int4 a = ring->at[slot][0], c = ring->at[slot][1];
  if (FREE) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&ring->free[slot]);
  }
  u = TreeUnit{a.x, a.y, a.z, a.w, c.x, c.y, c.z & 1, c.z & 2};
  end = c.z < 0;
  return true;
}
// The tiles of the next unit, for a single thread: 0 at the end, -1 where a wait ran out.
__device__ __forceinline__ int take_tiles(TreeRing* ring, int un, WaitCtl* wctl) {
  const int slot = un % kUnits;
  if (!wait(&ring->full[slot], (un / kUnits) & 1, wctl)) return -1;
  const int ja = ring->at[slot][0].w, jb = ring->at[slot][1].x, c = ring->at[slot][1].z;
  mbar_arrive(&ring->free[slot]);
  return c < 0 ? 0 : jb - ja;
}

// Bits [s, s + 32) of a node's row of mask words: ones before it, zeros behind it.
__device__ __forceinline__ uint32_t mask_bits(const unsigned* row, int words, int s) {
  const int k = s >> 5;
  const uint32_t lo = k < 0 ? ~0u : k < words ? row[k] : 0u;
  const uint32_t hi = k + 1 < 0 ? ~0u : k + 1 < words ? row[k + 1] : 0u;
  return __funnelshift_r(lo, hi, s & 31);
}

// Packs a tree's mask [T, T] into words, a lane a word (warp-wide).
__device__ __forceinline__ void pack_mask(const uint8_t* mask, unsigned* out, int T, int words,
                                          int lane) {
  const bool wide = (T & 3) == 0 && (reinterpret_cast<uintptr_t>(mask) & 3) == 0;
#pragma unroll 1
  for (int f = lane; f < T * words; f += 32) {
    const int i = f / words, c0 = (f - i * words) * 32;
    const uint8_t* x = mask + (size_t)i * T + c0;
    const int n = min(32, T - c0);
    unsigned m = 0;
    if (wide) {  // 4 bytes at once (n is a multiple of 4 then)
      uint32_t y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        y[e] = 4 * e < n ? *reinterpret_cast<const uint32_t*>(x + 4 * e) : 0u;
#pragma unroll
      for (int e = 0; e < 8; ++e)  // bytes that are not 0, as 1, gathered into the top four bits
        m |= ((__vcmpne4(y[e], 0u) & 0x01010101u) * 0x10204080u >> 28) << (4 * e);
    } else {
      uint8_t y[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) y[e] = e < n ? x[e] : (uint8_t)0;
#pragma unroll
      for (int e = 0; e < 32; ++e) m |= (unsigned)(y[e] != 0) << e;
    }
    out[f] = m;
  }
}

// bf16 pairs of a word that are not finite: all ones in their halves.
__device__ __forceinline__ uint32_t odd_halves(uint32_t x) {
  return __vcmpgeu2(x & 0x7fff7fffu, 0x7f807f80u);
}

// Tiles of K and V lie in shared memory as [8 rows][64 columns] blocks of 1024 bytes, swizzled, those
// of 8 rows one after another.
// A V tile that has keys of the tree or rows behind the sequence's end: clears those rows, and values
// of the tree's keys that are not finite, whose nodes go into `odd`. Warp-wide; out of line, as such
// tiles are few.
template <int HD>
__device__ __noinline__ void tree_tile(uint8_t* vt, int n0, int tree0, int len, unsigned* odd,
                                       int lane) {
  constexpr int G8 = HD / 8;  // 16-byte groups of a row
  auto at = [&](int r, int g) {
    return reinterpret_cast<uint4*>(vt + (r / 8 * (HD / 64) + g / 8) * 1024 + (r & 7) * 128 +
                                    ((g % 8) ^ (r & 7)) * 16);
  };
  const int begin = max(0, tree0 - n0), end = min(kKT, len - n0);
  // A value times 0 is 0 or, of one that is not finite, NaN.
  const __nv_bfloat162 zero = __float2bfloat162_rn(0.0f);
  __nv_bfloat162 test[2] = {zero, zero};
#pragma unroll 4
  for (int e = lane + begin * G8; e < end * G8; e += 32) {
    const uint4 x = *at(e / G8, e % G8);
    test[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.x), zero, test[0]);
    test[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.y), zero, test[1]);
    test[0] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.z), zero, test[0]);
    test[1] = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x.w), zero, test[1]);
  }
  const float2 t = __bfloat1622float2(__hadd2(test[0], test[1]));
  if (__any_sync(0xffffffffu, t.x != t.x || t.y != t.y)) {
#pragma unroll 1
    for (int e = lane + begin * G8; e < end * G8; e += 32) {
      uint4* x = at(e / G8, e % G8);
      const uint4 v = *x;
      const uint4 z = make_uint4(odd_halves(v.x), odd_halves(v.y), odd_halves(v.z), odd_halves(v.w));
      if (z.x | z.y | z.z | z.w) {
        *x = make_uint4(v.x & ~z.x, v.y & ~z.y, v.z & ~z.z, v.w & ~z.w);
        const int node = n0 + e / G8 - tree0;
        atomicOr(&odd[node >> 5], 1u << (node & 31));
      }
    }
  }
#pragma unroll 4
  for (int e = lane + end * G8; e < kKT * G8; e += 32) *at(e / G8, e % G8) = make_uint4(0, 0, 0, 0);
}

// Values that tree_tile has cleared, of the nodes that a row sees, added to N of its columns.
template <int HD, int N>
__device__ __forceinline__ void tree_odd(const TreeK& p, float (&x)[N], const unsigned* odd,
                                         const unsigned* sees, const TreeUnit& u, int c) {
#pragma unroll 1
  for (int n = 0; n < p.T; ++n) {
    if (!(odd[n >> 5] >> (n & 31) & sees[n >> 5] >> (n & 31) & 1)) continue;
    const int key = u.len - p.T + n, slot = key & ((1 << p.ps_shift) - 1);
    const int page = p.table[(size_t)u.b * p.max_pages + (key >> p.ps_shift)];  // (it has been read)
    const __nv_bfloat16* v = p.v + ((((size_t)page * p.Hk + u.kh) << p.ps_shift) + slot) * HD + c;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const float f = __bfloat162float(v[e]);
      if (!isfinite(f)) x[e] += f;
    }
  }
}

// A value before the tree that is not finite has met weights of 0 (those that a copy has of the others'
// keys, and those that are 0 in 32 bits), which made NaN of it. In what a CTA has written such elements
// become what the values that are not finite come to: those of the share's keys before the tree, and of
// its nodes that the row sees. Rows whose sum is NaN (their scores were) stay as they are. Done by all
// warps, which have 8 columns each (a lane: one, of every fourth key and row), once everything else
// is. It hardly ever runs, but its place and its size count: 300 sequences of up to 1000 keys, 17 rows,
// head_dim 64 take 85 us without it and with this; 97 with a call in the softmax's warps or the list's
// (registers), 89 with a call here, 90 with 8 columns a lane (the kernel's instructions lie farther
// apart). At head_dim 128 looking for what is not finite costs 1 to 2 %.
template <int HD, int ROWS, int WARPS>
__device__ __forceinline__ void tree_mend(const TreeK& p) {
  const int lane = lane_id();
  TreeWalk u;
  u.init(p, blockIdx.x, gridDim.x, lane);
#pragma unroll 1
  while (u.next(p)) {
    const int tree0 = u.len - p.T, k0 = u.ja * kKT, k1 = min(u.jb * kKT, u.len);
    const size_t part = 2 * (size_t)blockIdx.x + (u.first ? 1 : 0);
    const size_t row0 = ((size_t)u.b * p.Hk + u.kh) * p.rows + u.rb * ROWS;
#pragma unroll 1
    for (int c = warp_id() * 8 + lane % 8; c < HD; c += WARPS * 8) {
      // a key's value where it is not finite, else 0 (pages outside are zeros)
      auto value = [&](int key) {
        const int page = p.table[(size_t)u.b * p.max_pages + (key >> p.ps_shift)];
        if (page < 0 || page >= p.num_pages) return 0.0f;
        const int slot = key & ((1 << p.ps_shift) - 1);
        const float x =
            __bfloat162float(p.v[((((size_t)page * p.Hk + u.kh) << p.ps_shift) + slot) * HD + c]);
        return isfinite(x) ? 0.0f : x;
      };
      float before = 0.0f;
      bool known = false;
#pragma unroll 1
      for (int r = lane / 8; r - lane / 8 < min(ROWS, p.rows - u.rb * ROWS); r += 4) {
        const bool mine = u.rb * ROWS + r < p.rows;
        __nv_bfloat16* const whole = p.o + (row0 + r) * HD + c;
        float* const share = p.o_part + ((part * (HD / 4) + c / 4) * ROWS + r) * 4 + c % 4;
        const float o = !mine ? 0.0f : u.whole ? __bfloat162float(*whole) : *share;
        bool nan = o != o;
        if (nan) {
          const float l = u.whole ? p.lse[row0 + r] : p.ml_part[(part * 2 + 1) * ROWS + r];
          nan = l == l;
        }
        if (!__any_sync(0xffffffffu, nan)) continue;
        if (!known) {  // what the keys before the tree come to, for all rows
          known = true;
#pragma unroll 1
          for (int k = k0 + lane / 8; k < min(k1, tree0); k += 4) before += value(k);
          before += __shfl_xor_sync(0xffffffffu, before, 8);
          before += __shfl_xor_sync(0xffffffffu, before, 16);
        }
        if (!nan || before == 0.0f) continue;  // (NaN of something else)
        const uint8_t* sees = p.mask + u.b * p.mask_stride + (size_t)((u.rb * ROWS + r) % p.T) * p.T;
        float x = before;
#pragma unroll 1
        for (int k = max(k0, tree0); k < k1; ++k)
          if (sees[k - tree0]) x += value(k);
        if (u.whole) *whole = __float2bfloat16(x);
        else *share = x;
      }
    }
  }
}

// The weights of a copy's keys, zeros for the others.
template <int C>
__device__ __forceinline__ void store_weights(uint32_t at, const uint32_t (&pk)[32 / C], int copy) {
#pragma unroll
  for (int k = 0; k < C; ++k) {
    uint32_t x[32 / C];
#pragma unroll
    for (int e = 0; e < 32 / C; ++e) x[e] = k == copy ? pk[e] : 0u;
    if constexpr (C == 2)
      tmem_st16(at + k * 16, x);
    else
      asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(
                       at + k * 8),
                   "r"(x[0]), "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]),
                   "r"(x[7])
                   : "memory");
  }
}
// The barrier of a warpgroup's threads.
__device__ __forceinline__ void soft_sync() {
  asm volatile("barrier.cta.sync 2, 128;" ::: "memory");
}

// The same; true where any of them came with `v`.
__device__ __forceinline__ bool soft_any(bool v) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 128, p;\n"
      " selp.s32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)v)
      : "memory");
  return r != 0;
}

template <int HD, int C, int CT>
__global__ void __launch_bounds__(TreeLayout<HD, C, CT>::THREADS, CT)
    tree_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                const __grid_constant__ CUtensorMap mV, const TreeK p) {
  using LY = TreeLayout<HD, C, CT>;
  constexpr int KCH = LY::KCH, NWG = LY::NWG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  // Tile g's S and P are in buffer g & 1 of each warpgroup. s_full: S is there; p_full: P is; p_done: O has
  // it. (The rings' empty barriers are their own: a stage may be filled again
  // when the phase of p_done or s_full that freed it is two phases old.)
  __shared__ uint64_t k_full[LY::KST], v_full[LY::VST], k_empty[LY::KST], v_empty[LY::VST];
  // of stages with V of the tree's keys: asked for (only then is v_full's phase the one of that copy),
  // and looked over
  __shared__ uint64_t v_tail[LY::VST], v_fixed[LY::VST];
  __shared__ uint64_t s_full[NWG][2], p_full[NWG][2], p_done[NWG][2], q_full[2], q_free[2];
  __shared__ uint64_t drain_s, drain_o;
  __shared__ __align__(16) TreeRing units;
  __shared__ uint32_t tmem_base_s;
  __shared__ WaitCtl wctl;
  __shared__ int bad_input;
  __shared__ int mend_s;  // something that is not finite has been written
  __shared__ int page_s[2][kPageChunk];
  __shared__ float2 ml_s[2][C > 1 ? 128 : 1];  // of a unit (even, odd): m and the sum of each copy's rows
  unsigned* bits = reinterpret_cast<unsigned*>(smem + LY::OFF_BITS);

  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    wait_ctl_init(&wctl, p.wait_limit_ns);
    bad_input = mend_s = 0;
#pragma unroll 1
    for (int s = 0; s < LY::KST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], 1);
    }
#pragma unroll 1
    for (int s = 0; s < LY::VST; ++s) {
      mbar_init(&v_full[s], 1);
      mbar_init(&v_empty[s], 1);
      mbar_init(&v_tail[s], 1);
      mbar_init(&v_fixed[s], 1);
    }
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      for (int w = 0; w < NWG; ++w) {
        mbar_init(&s_full[w][s], 1);
        mbar_init(&p_full[w][s], 4);
        mbar_init(&p_done[w][s], 1);
      }
      mbar_init(&q_full[s], 1);
      mbar_init(&q_free[s], 1);
    }
#pragma unroll 1
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(&units.full[s], 1);
      mbar_init(&units.free[s], 5 + LY::SOFT);
      mbar_init(&units.bits_full[s], 1);
      mbar_init(&units.odd_full[s], 1);
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

  if (warp == LY::K_WARP || warp == LY::V_WARP) {
    // ------------------------------------------------------------------ K or V copies
    const bool leader = lane == 0, is_v = warp == LY::V_WARP;
    const CUtensorMap* map = is_v ? &mV : &mK;
    uint64_t* full = is_v ? v_full : k_full;
    uint64_t* empty = is_v ? v_empty : k_empty;
    uint8_t* ring = smem + (is_v ? LY::OFF_V : LY::OFF_K);
    const int ST = is_v ? LY::VST : LY::KST;
    int* pages = page_s[is_v];
    if (leader) tma_prefetch_desc(map);
    const int box = min(1 << p.ps_shift, kKT);  // rows of a box
    const int boxes = kKT / box;                // of a tile (at most 8)
    const int z_oob = p.num_pages * p.Hk;       // a page past the cache: zero fill
    int g = 0, st = 0;                          // copies so far, the next one's stage
    int page_b = -1, page_lo = 0;               // pages: entries page_lo .. of sequence page_b
    TreeUnit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit<true>(&units, un, w, end, lane, &wctl)) && !end; ++un) {
      const int used = (w.len + (1 << p.ps_shift) - 1) >> p.ps_shift;
      const int32_t* row = p.table + (size_t)w.b * p.max_pages;
#pragma unroll 1
      for (int j = w.ja; j < w.jb; ++j, ++g) {
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
            pages[e] = pg;
          }
          __syncwarp();
        }
        const int key = n0 + lane * box;  // of this lane's box
        int z = z_oob, y = 0;
        if (lane < boxes && key < w.len) {
          const int pg = pages[(key >> p.ps_shift) - page_lo];
          if (pg >= 0) {
            z = pg * p.Hk + w.kh;
            y = (key & ((1 << p.ps_shift) - 1)) >> 3;
          }
        }
        if (leader) {
          if (g >= ST) ok = wait(&empty[st], (g / ST - 1) & 1, &wctl);
          if (ok) mbar_arrive_expect_tx(&full[st], LY::ST_BYTES);
          if (ok && is_v && n0 + kKT > w.len - p.T) mbar_arrive(&v_tail[st]);
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
        if (lane < boxes)
          tma_load_5d(ring + st * LY::ST_BYTES + lane * box * (HD * 2), map, &full[st], 0, 0, 0, y,
                      z);
        if (++st == ST) st = 0;
      }
    }
    if (leader) {  // no copy may be in flight when the CTA ends
#pragma unroll 1
      for (int s = 0; s < ST; ++s) {
        const int n = (g - s + ST - 1) / ST;  // copies into stage s
        if (n > 0) mbar_wait_drain(&full[s], (n - 1) & 1);
      }
    }
  } else if (warp == LY::S_WARP) {
    // ------------------------------------------------------------------ S = Q K^T
    // (Inside elect_one the compiler keeps descriptors in uniform registers; behind a test of the lane
    // an MMA takes 67 cycles to issue whatever its shape, so 45 for N = 64, 59 for 128, which is its
    // arithmetic, and with A in tensor memory 29 for N = 64.)
    if (elect_one()) {
      const uint32_t id = idesc_bf16(128, kKT, 0, 0);
      const Desc k0 = make_desc(smem_u32(smem + LY::OFF_K), 16, KCH * 1024);
      int g = 0, st = 0;
      bool ok = true;
#pragma unroll 1
      for (int un = 0; ok; ++un) {
        const int tiles = take_tiles(&units, un, &wctl);
        if (tiles <= 0) break;
        const int qs = un % LY::QB;
        const uint32_t qp = un / LY::QB & 1;
        // (a poll that is not suspended first: where a short limit runs out)
        ok = mbar_test_wait(&q_full[qs], qp) || wait_more(&q_full[qs], qp, &wctl);
#pragma unroll 1
        for (int e = g + tiles; ok && g < e; ++g) {
          const int buf = g & 1;
          const uint32_t before = ((g >> 1) - 1) & 1;  // the buffer's last P is done with
          for (int w = 0; w < NWG; ++w)
            if (ok && g >= 2) ok = wait(&p_done[w][buf], before, &wctl);
          ok = ok && wait(&k_full[st], (g / LY::KST) & 1, &wctl);
          if (!ok) break;
          tc_fence_after();
          const Desc kb{k0.at(st * LY::ST_BYTES), k0.hi};
#pragma unroll
          for (int w = 0; w < NWG; ++w) {
            const Desc qa = make_desc(smem_u32(smem + (NWG == 1 ? qs : w) * LY::Q_BYTES), 16, 1024);
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks)
              mma_ss2(tbase + LY::col_s(w, buf), qa.at((ks / 4) * (128 * 128) + (ks % 4) * 32), qa.hi,
                      kb.at((ks / 4) * 1024 + (ks % 4) * 32), kb.hi, id, ks > 0 ? 1u : 0u);
            mma_commit(&s_full[w][buf]);
          }
          mma_commit(&k_empty[st]);
          if (++st == LY::KST) st = 0;
        }
        if (ok) mma_commit(&q_free[qs]);
      }
      mma_commit(&drain_s);
      mbar_wait_drain(&drain_s, 0);
    }
    __syncwarp();
  } else if (warp == LY::O_WARP) {
    // ------------------------------------------------------------------ O += P V
    const uint32_t id = idesc_bf16(128, HD, 0, 1);
    int g = 0, st = 0;
    uint32_t vp = 0, fixed = 0;  // stage of V, and its phase; phases of v_fixed
    TreeUnit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit<true>(&units, un, w, end, lane, &wctl)) && !end; ++un) {
      const int tree0 = w.len - p.T;
#pragma unroll 1
      for (int j = w.ja; j < w.jb && ok; ++j, ++g) {
        const int buf = g & 1;
        ok = wait_warp(&v_full[st], vp, &wctl);
        if (ok && j * kKT + kKT > tree0) {
          ok = wait_warp(&v_fixed[st], fixed >> st & 1, &wctl);
          fixed ^= 1u << st;
        }
#pragma unroll
        for (int i = 0; i < NWG; ++i) {
          ok = ok && wait_warp(&p_full[i][buf], (g >> 1) & 1, &wctl);
          if (!ok) break;
          tc_fence_after();
          if (elect_one()) {
            // V, MN-major
            const Desc vb =
                make_desc(smem_u32(smem + LY::OFF_V + st * LY::ST_BYTES), 1024, KCH * 1024);
#pragma unroll
            for (int ks = 0; ks < kKT / 16; ++ks)
              mma_ts2(tbase + i * HD, tbase + LY::col_s(i, buf) + ks * 8,
                      vb.at(ks * (2 * KCH * 1024)), vb.hi, id, j > w.ja || ks > 0 ? 1u : 0u);
            mma_commit(&p_done[i][buf]);
            if (i == NWG - 1) mma_commit(&v_empty[st]);
          }
          __syncwarp();
        }
        if (++st == LY::VST) {
          st = 0;
          vp ^= 1;
        }
      }
    }
    if (elect_one()) {  // (the same thread)
      mma_commit(&drain_o);
      mbar_wait_drain(&drain_o, 0);
    }
    __syncwarp();
  } else if (warp == LY::FIX_WARP) {
    // ------------------------------------------------------------------ V of the tree's keys, as soon
    // as it has landed: what is not finite, and what lies behind the sequence's end
    if (!p.cut) {  // (else the joining kernel does it) rows of sequences without keys
#pragma unroll 1
      for (int b = blockIdx.x; b < p.B; b += gridDim.x) {
        if (tree_len(p, b) > 0) continue;
        const size_t r0 = (size_t)b * p.Hk * p.rows, n = (size_t)p.Hk * p.rows;
        for (size_t e = lane; e < n * (HD / 8); e += 32)
          reinterpret_cast<uint4*>(p.o + r0 * HD)[e] = make_uint4(0u, 0u, 0u, 0u);
        for (size_t e = lane; e < n; e += 32) p.lse[r0 + e] = -INFINITY;
      }
    }
    int g = 0;
    uint32_t asked = 0;  // phases of v_tail
    TreeUnit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit<true>(&units, un, w, end, lane, &wctl)) && !end; ++un) {
      const int slot = un % kUnits, tree0 = w.len - p.T;
#pragma unroll 1
      for (int j = max(w.ja, max(tree0, 0) / kKT); j < w.jb; ++j) {
        const int n = g + j - w.ja, st = n % LY::VST;
        ok = wait_warp(&v_tail[st], asked >> st & 1, &wctl) &&
             wait_warp(&v_full[st], n / LY::VST & 1, &wctl);
        if (!ok) break;
        asked ^= 1u << st;
        tree_tile<HD>(smem + LY::OFF_V + st * LY::ST_BYTES, j * kKT, tree0, w.len, units.odd[slot],
                      lane);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_fixed[st]);
      }
      g += w.jb - w.ja;
      if (lane == 0) mbar_arrive(&units.odd_full[slot]);
    }
  } else if (warp == LY::LIST_WARP) {
    // ------------------------------------------------------------------ units, masks and Q
    if (blockIdx.x == 0) {  // lengths out of range are clamped, and reported here
      bool bad = false;
#pragma unroll 1
      for (int b = lane; b < p.B; b += 32) bad |= p.lens[b] != tree_len(p, b);
      if (bad) bad_input = 1;
    }
    TreeWalk list;
    list.init(p, blockIdx.x, gridDim.x, lane);
    if (lane == 0) tma_prefetch_desc(&mQ);
    int packed[kUnits], loads = 0;  // whose mask a slot has; units whose Q is asked for
#pragma unroll
    for (int s = 0; s < kUnits; ++s) packed[s] = -1;
    bool ok = true, ended = false;
#pragma unroll 1
    for (int un = 0; ok && !ended; ++un) {
      const int slot = un % kUnits;
      if (un >= kUnits) ok = wait_warp(&units.free[slot], (un / kUnits - 1) & 1, &wctl);
      if (!ok) break;
      ended = !list.next(p);
      if (lane < kTreeMax / 32) units.odd[slot][lane] = 0;
      __syncwarp();
      if (lane == 0) {
        units.at[slot][0] = make_int4(list.b, list.kh, list.rb, list.ja);
        units.at[slot][1] =
            make_int4(list.jb, list.len, ended ? -1 : list.whole | list.first << 1, 0);
        mbar_arrive(&units.full[slot]);
      }
      __syncwarp();
      if (ended) break;
      const int qs = un % LY::QB, turn = un / LY::QB;
      if (turn > 0) ok = wait_warp(&q_free[qs], (turn - 1) & 1, &wctl);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&q_full[qs], NWG * LY::Q_BYTES);
        for (int i = 0; i < NWG * C; ++i)  // row blocks, or copies of one
          for (int c = 0; c < KCH; ++c)
            tma_load_3d(smem + (NWG == 1 ? qs * LY::Q_BYTES + i * LY::RC * 128 : i * LY::Q_BYTES) +
                            c * (128 * 128),
                        &mQ, &q_full[qs], c * 64, list.rb * LY::ROWS + (C > 1 ? 0 : i * 128),
                        list.b * p.Hk + list.kh);
      }
      ++loads;
      const int whose = p.mask_stride == 0 ? 0 : list.b;
      bool have = false;
#pragma unroll
      for (int s = 0; s < kUnits; ++s) {
        if (s == slot) {
          have = packed[s] == whose;
          packed[s] = whose;
        }
      }
      if (!have)
        pack_mask(p.mask + list.b * p.mask_stride, bits + slot * p.T * p.words, p.T, p.words, lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&units.bits_full[slot]);
      __syncwarp();
    }
    if (lane == 0) {  // no copy may be in flight when the CTA ends
      for (int i = 0; i < LY::QB; ++i) {
        const int n = (loads - i + LY::QB - 1) / LY::QB;  // of this buffer
        if (n > 0) mbar_wait_drain(&q_full[i], (n - 1) & 1);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax, and O out
    // Rows that are not there have q = 0 and columns that hold anything; warps without any row keep
    // the barriers going and do nothing else. A wait that runs out ends the warp's tiles; where copies
    // are joined all warps leave together.
    const int wg = warp >> 2, wl = warp & 3, row = threadIdx.x & 127;
    const uint32_t lanes = tbase + ((uint32_t)(wl * 32) << 16);
    const uint32_t tO = lanes + wg * HD;
    // copy `copy` of row r, with NC of a tile's keys
    constexpr int NC = LY::NC;
    // Where registers are few (two CTAs an SM) scores are taken twice, 32 at a time.
    constexpr bool LEAN = CT == 2 && NC == 64;
    const int copy = C == 1 ? 0 : row / LY::RC, r = row % LY::RC;
    const uint64_t c2 = f2_pack(p.scale_log2, p.scale_log2);
    int g = 0;
    TreeUnit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0;; ++un) {
      // (those that join meet once for each unit, whatever a warp has come upon: here, or at its end)
      ok = take_unit<false>(&units, un, w, end, lane, &wctl);
      if (!ok || end) {
        if (C > 1) soft_any(true);
        break;
      }
      const int slot = un % kUnits;
      const int r0 = w.rb * LY::ROWS + wg * 128;
      const bool live = r0 + wl * 32 % LY::RC < p.rows, mine = r0 + r < p.rows;
      const int node = mine ? (r0 + r) % p.T : 0;
      const unsigned* sees = bits + (slot * p.T + node) * p.words;
      // the first key of the tree, counted from this thread's first of tile 0
      const int tree0 = w.len - p.T - copy * NC;
      float m = -FLT_MAX / 2.0f, l = 0.0f;
#pragma unroll 1
      for (int j = w.ja; j < w.jb; ++j, ++g) {
        const int buf = g & 1, first = j * kKT - tree0;  // node of this thread's first key
        const uint32_t ph = (g >> 1) & 1, at = lanes + LY::col_s(wg, buf);
        ok = wait_warp(&s_full[wg][buf], ph, &wctl);
        // (every warp that is asked for has seen the words that it looks at)
        if (ok && first + NC > 0) ok = wait_warp(&units.bits_full[slot], (un / kUnits) & 1, &wctl);
        if (!ok) break;
        if (live) {
          tc_fence_after();
          uint32_t s[LEAN ? 32 : NC];
          auto scores = [&](int h) {  // 32 of them
            tmem_ld32(at + copy * NC + h, *reinterpret_cast<uint32_t(*)[32]>(&s[LEAN ? 0 : h]));
          };
          auto hide = [&](int h) {
            if (first + NC <= 0) return;
            const uint32_t vis = mask_bits(sees, p.words, first + h);
#pragma unroll
            for (int e = 0; e < 32 && e < NC; ++e)
              if (!(vis >> e & 1)) s[(LEAN ? 0 : h) + e] = 0xff800000u;  // -inf
          };
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          if constexpr (NC == 16) {
            tmem_ld16(at + copy * NC, s);
            tmem_wait_ld();
            hide(0);
#pragma unroll
            for (int e = 0; e < 16; e += 2)
              mx[e / 2 & 3] =
                  fmax3(mx[e / 2 & 3], __uint_as_float(s[e]), __uint_as_float(s[e + 1]));
          } else {
            if (!LEAN) {
#pragma unroll
              for (int h = 0; h < NC; h += 32) scores(h);
              tmem_wait_ld();
            }
#pragma unroll
            for (int h = 0; h < NC; h += 32) {
              if (LEAN) {
                scores(h);
                tmem_wait_ld();
              }
              hide(h);
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const uint32_t* x = &s[(LEAN ? 0 : h) + e];
                mx[e / 2 & 3] = fmax3(mx[e / 2 & 3], __uint_as_float(x[0]), __uint_as_float(x[1]));
              }
            }
          }
          const float m_new =
              fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2);
          if (j == w.ja) {
            m = m_new;
          } else if (__any_sync(0xffffffffu, m_new > m + kRescale)) {
            // O holds P V of this warpgroup's tiles before; only the last can be outstanding
            const float f = ex2(m - m_new);
            l *= f;
            ok = wait_warp(&p_done[wg][(g - 1) & 1], ((g - 1) >> 1) & 1, &wctl);
            if (!ok) break;
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < HD; c += 32) {
              uint32_t x[32];
              tmem_ld32(tO + c, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f);
              tmem_st32(tO + c, x);
            }
            tmem_wait_st();
            m = m_new;
          }
          const uint64_t nm = f2_pack(-m, -m);
          uint64_t sum[2] = {0ull, 0ull};
          constexpr int PN = NC < 32 ? NC : 32;  // keys whose weights are stored at once
#pragma unroll
          for (int h = 0; h < NC / PN; ++h) {
            if (LEAN) {  // (P of a half lies over scores that have been taken)
              scores(h * PN);
              tmem_wait_ld();
              hide(h * PN);
            }
            uint32_t pk[PN / 2];
#pragma unroll
            for (int e = 0; e < PN; e += 2) {
              const uint32_t* x = &s[(LEAN ? 0 : h * PN) + e];
              float a, b;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(x[0]), __uint_as_float(x[1])), c2, nm), a, b);
              a = ex2(a);
              b = ex2(b);
              sum[e / 2 & 1] = f2_add(sum[e / 2 & 1], f2_pack(a, b));
              pk[e / 2] = pack_bf16(a, b);
            }
            if constexpr (C == 1)
              tmem_st16(at + h * 16, pk);
            else
              store_weights<C>(at, pk, copy);
          }
          float a, b;
          f2_unpack(f2_add(sum[0], sum[1]), a, b);
          l += a + b;
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[wg][buf]);
      }
      // ---- the unit's end
      if (C > 1) {
        ml_s[un & 1][row] = make_float2(m, l);
        if (soft_any(!ok)) break;
      }
      // (with copies a wait that runs out here leaves O undefined, as the status says)
      ok = ok && wait_warp(&p_done[wg][(g - 1) & 1], ((g - 1) >> 1) & 1, &wctl) &&
           wait_warp(&units.odd_full[slot], (un / kUnits) & 1, &wctl);
      if (C == 1 && !ok) break;
      const bool none = l == 0.0f;
      float f = none ? 0.0f : 1.0f;  // O's factor
      if (C > 1) {
        const float2* ml = &ml_s[un & 1][r];
        const float mine_m = m;
#pragma unroll
        for (int k = 0; k < C; ++k) m = fmaxf(m, ml[k * LY::RC].x);
        f = none ? 0.0f : ex2(mine_m - m);
        l = 0.0f;
#pragma unroll
        for (int k = 0; k < C; ++k) {
          const float2 x = ml[k * LY::RC];
          if (x.y != 0.0f) l = fmaf(x.y, ex2(x.x - m), l);
        }
      }
      tc_fence_after();
      bool odd = false;
#pragma unroll
      for (int k = 0; k < kTreeMax / 32; ++k) odd |= units.odd[slot][k] != 0;
      const size_t unit_row = ((size_t)w.b * p.Hk + w.kh) * p.rows + r0 + r;
      const size_t part = 2 * (size_t)blockIdx.x + (w.first ? 1 : 0);
      const int prow = wg * 128 + r;  // of the unit's rows
      float4* o_part = reinterpret_cast<float4*>(p.o_part) + part * (HD / 4) * LY::ROWS + prow;
      if (w.whole && l != 0.0f) f *= 1.0f / l;
      // N columns from c on of this thread's row, where they go
      auto out = [&](auto& o, int c) {
        constexpr int N = sizeof(o) / 4;
        if (!mine) return;
        uint64_t test = 0ull;  // (a sum that is NaN is the scores' doing)
#pragma unroll
        for (int e = 0; e < N; e += 2) test = f2_fma(f2_pack(o[e], o[e + 1]), 0ull, test);
        float t0, t1;
        f2_unpack(test, t0, t1);
        if (t0 + t1 != 0.0f && l == l) mend_s = 1;
        if (odd) tree_odd<HD>(p, o, units.odd[slot], sees, w, c);
        if (w.whole) {
          __nv_bfloat16* dst = p.o + unit_row * HD + c;
#pragma unroll
          for (int k = 0; k < N; k += 8)
            *reinterpret_cast<uint4*>(dst + k) =
                make_uint4(pack_bf16(o[k], o[k + 1]), pack_bf16(o[k + 2], o[k + 3]),
                           pack_bf16(o[k + 4], o[k + 5]), pack_bf16(o[k + 6], o[k + 7]));
        } else {
#pragma unroll
          for (int k = 0; k < N; k += 4)
            o_part[(size_t)((c + k) / 4) * LY::ROWS] =
                make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
        }
      };
      if (live) {
#pragma unroll 1
        for (int c = 0; c < HD; c += 32) {
          uint32_t x[32];
          tmem_ld32(tO + c, x);
          tmem_wait_ld();
          float o[32];
#pragma unroll
          for (int e = 0; e < 32; ++e)  // (O of no weight holds anything)
            o[e] = none ? 0.0f : __uint_as_float(x[e]) * f;
          if constexpr (C == 1) {
            out(o, c);
            __syncwarp();
          } else {
            // the copies' sums, through shared memory: a thread has 32 / C of the 32 columns
            float4* join = reinterpret_cast<float4*>(smem + LY::OFF_JOIN);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              join[row * 8 + (k ^ (row & 7))] =
                  make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            soft_sync();
            constexpr int N = 32 / C;
            float z[N] = {};
#pragma unroll
            for (int i = 0; i < C; ++i) {
              const int from = r + i * LY::RC;
#pragma unroll
              for (int k = 0; k < N; k += 4) {
                const float4 v = join[from * 8 + ((copy * (N / 4) + k / 4) ^ (from & 7))];
                z[k] += v.x, z[k + 1] += v.y, z[k + 2] += v.z, z[k + 3] += v.w;
              }
            }
            soft_sync();
            out(z, c + copy * N);
          }
        }
        if (mine && copy == 0) {
          if (!w.whole) {
            p.ml_part[part * 2 * LY::ROWS + prow] = m;
            p.ml_part[(part * 2 + 1) * LY::ROWS + prow] = l;
          } else {
            p.lse[unit_row] = l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&units.free[slot]);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == LY::S_WARP) tmem_dealloc(tbase, LY::TMEM_COLS);
  if (threadIdx.x == 0) {
    report_abort(&wctl, p.status);
    if (bad_input && p.status) atomicCAS(p.status, kStatusOk, kStatusBadInput);
  }
  if (mend_s && !wctl.abort) tree_mend<HD, LY::ROWS, LY::THREADS / 32>(p);
}

// Joins the shares of the units that were cut, and writes those of sequences without keys: a thread
// has 8 columns of a row, a warp 32 rows. Launched early: what it needs to know of the lengths it
// works out while the attention still runs.
template <int HD, int ROWS>
__global__ void __launch_bounds__(32 * HD / 8) tree_combine_kernel(const TreeK p, int grid) {
  const int warp = warp_id(), lane = lane_id();
  const unsigned U = (unsigned)(p.Hk * p.rb);  // blockIdx.x: (b * Hk + kh) * rb + row block
  const int b = (int)(blockIdx.x / U), in = (int)(blockIdx.x % U);
  const int kh = p.rb == 1 ? in : in / p.rb, rb = in - kh * p.rb;
  const int row = (int)blockIdx.y * 32 + lane, R = rb * ROWS + row;  // of the unit, of the kv head
  const bool mine = row < ROWS && R < p.rows;
  const size_t out = ((size_t)b * p.Hk + kh) * p.rows + R;
  // every warp finds the unit's place in the list for itself
  int mine_cost = lane < p.B ? tree_cost(p, lane) : 0;
  const int cost = tree_cost(p, b);
  unsigned before = lane < b ? mine_cost : 0;
#pragma unroll 1
  for (int i = lane + 32; i < b; i += 32) before += tree_cost(p, i);
  before = __reduce_add_sync(0xffffffffu, before);
  const unsigned per = tree_share(tree_all(p, mine_cost, lane) * U, grid);
  uint4* dst = reinterpret_cast<uint4*>(p.o + out * HD + warp * 8);
  if (cost == 0 && mine) {
    *dst = make_uint4(0u, 0u, 0u, 0u);
    if (warp == 0) p.lse[out] = -INFINITY;
  }
  // (by every CTA: what follows this kernel must find the attention done)
  grid_dep_wait();
  if (cost == 0) return;
  const unsigned a = before * U + (unsigned)in * cost;  // of its first tile and of its last:
  const int c0 = (int)((a + kUnitCost) / per), c1 = (int)((a + cost - 1) / per);
  if (c0 == c1 || !mine) return;  // written whole
  // share i: slot 2 c0 + 1 (it begins there), then 2 c of each further CTA
  constexpr int AHEAD = 4;
  float m = -FLT_MAX / 2.0f, l = 0.0f, acc[8] = {};
#pragma unroll 1
  for (int c = c0; c <= c1; c += AHEAD) {
    float mi[AHEAD], li[AHEAD];
    float4 x[AHEAD][2];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int cc = min(c + k, c1);
      const size_t s = (size_t)2 * cc + (cc == c0 ? 1 : 0);
      mi[k] = p.ml_part[s * 2 * ROWS + row];
      li[k] = c + k <= c1 ? p.ml_part[(s * 2 + 1) * ROWS + row] : 0.0f;
      const float4* src = reinterpret_cast<const float4*>(p.o_part) +
                          (s * (HD / 4) + warp * 2) * ROWS + row;
      x[k][0] = src[0];
      x[k][1] = src[ROWS];
    }
    float top = m;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (li[k] != 0.0f) top = fmaxf(top, mi[k]);
    const float old = ex2(m - top);
    m = top;
    l *= old;
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[e] *= old;
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (li[k] == 0.0f) continue;
      const float f = ex2(mi[k] - top);
      l = fmaf(li[k], f, l);
      const float* y = &x[k][0].x;
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[e] = fmaf(y[e], f, acc[e]);
    }
  }
  // (what is not finite and met a factor of 0, as in tree_mend)
  bool nan = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) nan |= acc[e] != acc[e];
  if (nan && l == l) {
    float x[8] = {};
#pragma unroll 1
    for (int c = c0; c <= c1; ++c) {
      const size_t s = (size_t)2 * c + (c == c0 ? 1 : 0);
      if (p.ml_part[(s * 2 + 1) * ROWS + row] == 0.0f) continue;
      const float* src = p.o_part + ((s * (HD / 4) + warp * 2) * ROWS + row) * 4;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = src[e / 4 * ROWS * 4 + e % 4];
        if (!isfinite(y)) x[e] += y;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (acc[e] != acc[e] && x[e] != 0.0f) acc[e] = x[e];
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *dst = make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv),
                    pack_bf16(acc[4] * inv, acc[5] * inv), pack_bf16(acc[6] * inv, acc[7] * inv));
  if (warp == 0) p.lse[out] = l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l));
}

struct TreePlan {
  int C, CT, ROWS, rb, grid, cut;
};
TreePlan tree_plan(const TreeArgs& a) {
  TreePlan pl;
  const int rows = a.G * a.T;
  pl.C = a.d > 64 || rows > 64 ? 1 : rows > 32 ? 2 : 4;
  pl.CT = rows <= 128 && a.d <= 128 ? 2 : 1;
  pl.ROWS = pl.CT == 2 ? 128 / pl.C : a.d <= 128 ? 256 : 128;
  pl.rb = (rows + pl.ROWS - 1) / pl.ROWS;
  const long long cap = (long long)a.max_pages << a.ps_shift;
  // 100 sequences of up to 1000 keys, 48 rows, head_dim 128, 800 units: cut 64 us, whole 60; 20 of them: 21
  // and 23 us; 100 of up to 2k, 17 rows, head_dim 64: 52 and 54; 100 of up to 500 keys, 100 rows: 67 and 48.
  const long long units = (long long)a.B * a.Hk * pl.rb;
  pl.cut = cap > (units >= 152 * pl.CT ? 2 * kWholeKeys : kWholeKeys);
  const long long tiles = ((cap + kKT - 1) / kKT + kUnitCost) * a.B * a.Hk * pl.rb;
  pl.grid = (int)std::min<long long>(152 * pl.CT, tiles);
  return pl;
}

// Scratch for the shares' O, m and sums; L of the rows lies behind it where the caller wants none.
size_t parts_floats(const TreePlan& pl, int d) {
  return pl.cut ? (size_t)2 * pl.grid * pl.ROWS * (d + 2) : 0;
}

template <int HD, int C, int CT>
cudaError_t launch_tree_t(const TreeArgs& a, const TreeMaps& m, const TreePlan& pl, void* ws,
                          cudaStream_t s) {
  using LY = TreeLayout<HD, C, CT>;
  static OncePerKey<> smem_attr;
  auto kern = tree_kernel<HD, C, CT>;
  cudaError_t e = set_smem_once(smem_attr, kern, LY::smem_bytes(LY::T_MAX));
  if (e != cudaSuccess) return e;
  TreeK p;
  p.v = static_cast<const __nv_bfloat16*>(a.v_cache);
  p.table = a.table;
  p.lens = a.lens;
  p.mask = a.mask;
  p.mask_stride = a.mask_stride;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.o_part = static_cast<float*>(ws);
  p.ml_part = p.o_part + (size_t)2 * pl.grid * LY::ROWS * HD;
  p.lse = a.lse ? a.lse : p.o_part + parts_floats(pl, HD);
  p.status = a.status;
  p.B = a.B;
  p.Hk = a.Hk;
  p.T = a.T;
  p.words = (a.T + 31) / 32;
  p.rows = a.G * a.T;
  p.rb = pl.rb;
  p.cut = pl.cut;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.ps_shift = a.ps_shift;
  p.scale_log2 = a.scale * kLog2e;
  p.wait_limit_ns = a.wait_limit_ns;
  profile_mark(kKernTreeAttn, 0, s);
  kern<<<pl.grid, LY::THREADS, LY::smem_bytes(a.T), s>>>(m.q, m.k, m.v, p);
  e = cudaGetLastError();
  profile_mark(kKernTreeAttn, 1, s);
  if (e != cudaSuccess || !pl.cut) return e;
  const int live = std::min(p.rows, LY::ROWS);
  profile_mark(kKernTreeCombine, 0, s);
  e = launch_pdl(tree_combine_kernel<HD, LY::ROWS>,
                 dim3((unsigned)(a.B * a.Hk * pl.rb), (unsigned)((live + 31) / 32)), dim3(32 * HD / 8),
                 0, s, p, pl.grid);
  profile_mark(kKernTreeCombine, 1, s);
  return e;
}
}  // namespace

int tree_box_rows(int page_size) { return page_size < kKT ? page_size : kKT; }

long long tree_tiles(const TreeArgs& a) {
  const long long cap = (long long)a.max_pages << a.ps_shift;
  return ((cap + kKT - 1) / kKT + kUnitCost) * a.B * a.Hk * tree_plan(a).rb;
}

size_t tree_workspace_bytes(const TreeArgs& a) {
  const TreePlan pl = tree_plan(a);
  const size_t lse = a.lse ? 0 : (size_t)a.B * a.Hk * a.G * a.T;
  return (parts_floats(pl, a.d) + lse) * 4;
}

int tree_q_rows(const TreeArgs& a) { return 128 / tree_plan(a).C; }

cudaError_t launch_tree(const TreeArgs& a, const TreeMaps& m, void* ws, cudaStream_t s) {
  const TreePlan pl = tree_plan(a);
  switch (a.d) {
    case 64:
      return pl.CT == 1  ? launch_tree_t<64, 1, 1>(a, m, pl, ws, s)
             : pl.C == 1 ? launch_tree_t<64, 1, 2>(a, m, pl, ws, s)
             : pl.C == 2 ? launch_tree_t<64, 2, 2>(a, m, pl, ws, s)
                         : launch_tree_t<64, 4, 2>(a, m, pl, ws, s);
    case 128:
      return pl.CT == 1 ? launch_tree_t<128, 1, 1>(a, m, pl, ws, s)
                        : launch_tree_t<128, 1, 2>(a, m, pl, ws, s);
    case 256: return launch_tree_t<256, 1, 1>(a, m, pl, ws, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
