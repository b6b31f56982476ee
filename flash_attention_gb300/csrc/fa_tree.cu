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
// a kv head. Up to that the work beside the bytes has to fit in the time of the bytes, 700 cycles for a
// tile of 64 keys at head_dim 64, 1400 at 128: two softmax warpgroups (thread = row), which alternate.
//  * up to 128 rows (PAIR): each has every other key tile, with an O, a maximum and a sum of its own;
//    they are joined at a unit's end, in tensor memory, where a thread of either can read both O's;
//  * more rows: each has 128 of a block's 256, on the same key tiles. (At head_dim 256 tensor memory
//    holds one O: one warpgroup, blocks of 128 rows.)
// S = Q K^T (M = 128 rows, N = 64 keys) and O += P V, with P in bf16 over S in tensor memory (two S
// buffers for each warpgroup); the lazy rescale of the training forward. Sums are f32.
//
// Work: the (sequence, kv head, row block) units, each ceil(len / 64) key tiles, form one list of
// tiles, cut evenly over persistent CTAs, one on an SM (the lengths are on the device; each CTA finds
// its part from them). A unit counts kUnitCost tiles more than it has, what its start and end cost. A
// CTA writes the units it has whole; of the others it leaves its share's O, m and sum, which a second
// kernel joins in the order of the keys.
//
// Warps: 0-3 (0-7) softmax, then one each for the copies of K and V pages (TMA boxes of
// min(page_size, 64) rows), for S, for O, and for the list: it walks the list two units ahead, packs
// the tree's mask into words and loads Q. The mask is tested in the tiles of the last T keys alone.
// There a value that is not finite must meet no weight of a row that does not see it, not even 0: the
// O warp clears it, and rows that see it get it added at the end (tree_odd).
#include <float.h>

#include <algorithm>

#include "fa_common.cuh"
#include "fa_launch.h"
#include "fa_wait.cuh"

namespace fa {

namespace {
constexpr int kKT = 64;          // keys of a tile
constexpr int kUnitCost = 4;     // tiles' worth of a unit's start and end
constexpr int kPageChunk = 128;  // block-table entries staged at a time
constexpr int kUnits = 3;        // units published
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;

template <int HD, bool PAIR>
struct TreeLayout {
  static constexpr int NWG = HD <= 128 ? 2 : 1;      // softmax warpgroups
  static constexpr int ROWS = PAIR ? 128 : 128 * NWG;  // query rows of a unit
  static constexpr int ST = HD == 64 ? 8 : HD == 128 ? 4 : 2;  // stages of the K ring and the V ring
  static constexpr int KCH = HD / 64;
  static constexpr int Q_BYTES = 128 * HD * 2;       // of 128 rows; PAIR: two units' Q, else a unit's
  static constexpr int KV_BYTES = kKT * HD * 2;
  static constexpr int OFF_K = NWG * Q_BYTES;
  static constexpr int OFF_V = OFF_K + ST * KV_BYTES;
  static constexpr int OFF_BITS = OFF_V + ST * KV_BYTES;  // mask words, kUnits * T * ceil(T / 32)
  static constexpr int COL_S = NWG * HD;             // O of each warpgroup, then its two S
  static constexpr int TMEM_COLS = 512;
  static constexpr int SOFT = 4 * NWG;
  static constexpr int TMA_WARP = SOFT, S_WARP = SOFT + 1, O_WARP = SOFT + 2, LIST_WARP = SOFT + 3;
  static constexpr int THREADS = 32 * (SOFT + 4);
  static_assert(!PAIR || NWG == 2, "pairs need two warpgroups");
  static_assert(COL_S + NWG * 2 * kKT <= TMEM_COLS, "TMEM budget");
  static int smem_bytes(int T) { return OFF_BITS + kUnits * T * ((T + 31) / 32) * 4 + 1024; }
  static_assert(OFF_BITS + kUnits * kTreeMax * (kTreeMax / 32) * 4 + 1024 + 8192 <= 227 * 1024,
                "shared memory budget");
};

struct TreeK {
  const __nv_bfloat16* v;  // the cache, for values that are not finite
  const int32_t* table;
  const int32_t* lens;
  const uint8_t* mask;
  long long mask_stride;
  __nv_bfloat16* o;
  float* lse;
  float* o_part;   // [2 * grid, HD / 4, ROWS, 4]: O of a share, in units of 2^m
  float* ml_part;  // [2 * grid, 2, ROWS]: m and the sum
  int* status;
  int B, Hk, T, words, rows, rb, max_pages, num_pages, ps_shift;
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
      const int from = (int)(in - u * cost), to = min(cost, from + (int)(t1 - t));
      t += to - from;
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
  uint64_t odd_full[kUnits];        // the O warp has looked at all the unit's tiles
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

// Bits [s, s + 32) of a node's row of mask words: ones before it, zeros behind it.
__device__ __forceinline__ uint32_t mask_bits(const unsigned* row, int words, int s) {
  const int k = s >> 5;
  const uint32_t lo = k < 0 ? ~0u : k < words ? row[k] : 0u;
  const uint32_t hi = k + 1 < 0 ? ~0u : k + 1 < words ? row[k + 1] : 0u;
  return __funnelshift_r(lo, hi, s & 31);
}

// Packs a tree's mask [T, T] into words, 32 of them in flight (warp-wide).
__device__ __forceinline__ void pack_mask(const uint8_t* mask, unsigned* out, int T, int words,
                                          int lane) {
  const int n = T * words;
#pragma unroll 1
  for (int f0 = 0; f0 < n; f0 += 32) {
    uint8_t x[32];
    int i = f0 / words, w = f0 - i * words;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int c = 32 * w + lane;
      x[e] = f0 + e < n && c < T ? mask[(size_t)i * T + c] : (uint8_t)0;
      if (++w == words) {
        w = 0;
        ++i;
      }
    }
    unsigned mine = 0;
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const unsigned m = __ballot_sync(0xffffffffu, x[e] != 0);
      if (lane == e) mine = m;
    }
    if (f0 + lane < n) out[f0 + lane] = mine;
  }
}

// bf16 pairs of a word that are not finite: all ones in their halves.
__device__ __forceinline__ uint32_t odd_halves(uint32_t x) {
  return __vcmpgeu2(x & 0x7fff7fffu, 0x7f807f80u);
}

// A V tile that has keys of the tree or rows behind the sequence's end: clears those rows, and values
// of the tree's keys that are not finite, whose nodes go into `odd`. Warp-wide; out of line, as such
// tiles are few.
template <int HD>
__device__ __noinline__ void tree_tile(uint8_t* vt, int n0, int tree0, int len, unsigned* odd,
                                       int lane) {
  constexpr int G8 = HD / 8;  // 16-byte groups of a row
  auto at = [&](int r, int g) {
    return reinterpret_cast<uint4*>(vt + g / 8 * (kKT * 128) + r * 128 + ((g % 8) ^ (r & 7)) * 16);
  };
  const int end = min(kKT, len - n0);
#pragma unroll 1
  for (int e = lane + max(0, tree0 - n0) * G8; e < end * G8; e += 32) {
    const int r = e / G8;
    uint4* x = at(r, e % G8);
    uint4 v = *x;
    const uint4 z = make_uint4(odd_halves(v.x), odd_halves(v.y), odd_halves(v.z), odd_halves(v.w));
    if (z.x | z.y | z.z | z.w) {
      *x = make_uint4(v.x & ~z.x, v.y & ~z.y, v.z & ~z.z, v.w & ~z.w);
      const int node = n0 + r - tree0;
      atomicOr(&odd[node >> 5], 1u << (node & 31));
    }
  }
#pragma unroll 1
  for (int e = lane + end * G8; e < kKT * G8; e += 32) *at(e / G8, e % G8) = make_uint4(0, 0, 0, 0);
}

// Values that tree_tile has cleared, of the nodes that a row sees, added to 8 of its columns.
__device__ __noinline__ void tree_odd(const TreeK& p, float* x, const unsigned* odd,
                                      const unsigned* sees, const TreeUnit& u, int HD, int c) {
  const int tree0 = u.len - p.T;
  for (int n = 0; n < p.T; ++n) {
    if (!(odd[n >> 5] >> (n & 31) & sees[n >> 5] >> (n & 31) & 1)) continue;
    const int key = tree0 + n, slot = key & ((1 << p.ps_shift) - 1);
    const int page = p.table[(size_t)u.b * p.max_pages + (key >> p.ps_shift)];  // (it has been read)
    const __nv_bfloat16* v = p.v + ((((size_t)page * p.Hk + u.kh) << p.ps_shift) + slot) * HD + c;
    for (int e = 0; e < 8; ++e) {
      const float f = __bfloat162float(v[e]);
      if (!isfinite(f)) x[e] += f;
    }
  }
}

// The barrier of the softmax's threads; true where any of them came with `v`.
template <int N>
__device__ __forceinline__ bool soft_any(bool v) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, %2, p;\n"
      " selp.s32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)v), "n"(N)
      : "memory");
  return r != 0;
}

template <int HD, bool PAIR>
__global__ void __launch_bounds__(TreeLayout<HD, PAIR>::THREADS, 1)
    tree_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                const __grid_constant__ CUtensorMap mV, const TreeK p) {
  using LY = TreeLayout<HD, PAIR>;
  constexpr int ST = LY::ST, KCH = LY::KCH, NWG = LY::NWG;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  // Item n of a warpgroup: its n-th tile. S and P of it are in its buffer n & 1.
  __shared__ uint64_t k_full[ST], v_full[ST], k_empty[ST], v_empty[ST];
  __shared__ uint64_t s_full[NWG][2], p_full[NWG][2], p_done[NWG][2], q_full[2], q_free[2];
  __shared__ uint64_t o_free, drain_s, drain_o;
  __shared__ __align__(16) TreeRing units;
  __shared__ uint32_t tmem_base_s;
  __shared__ WaitCtl wctl;
  __shared__ int bad_input;
  __shared__ int page_s[kPageChunk];
  __shared__ float2 ml_s[2][2][128];  // of a unit (even, odd): m and the sum of each warpgroup's rows
  unsigned* bits = reinterpret_cast<unsigned*>(smem + LY::OFF_BITS);

  const int warp = warp_id(), lane = lane_id();
  if (threadIdx.x == 0) {
    wait_ctl_init(&wctl, p.wait_limit_ns);
    bad_input = 0;
#pragma unroll 1
    for (int s = 0; s < ST; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&v_full[s], 1);
      mbar_init(&k_empty[s], 1);
      mbar_init(&v_empty[s], 1);
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
      mbar_init(&units.free[s], 3 + LY::SOFT);
      mbar_init(&units.odd_full[s], 1);
    }
    mbar_init(&o_free, LY::SOFT);
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

  if (warp == LY::TMA_WARP) {
    // ------------------------------------------------------------------ K and V copies
    const bool leader = lane == 0;
    if (leader) {
      tma_prefetch_desc(&mK);
      tma_prefetch_desc(&mV);
    }
    const int box = min(1 << p.ps_shift, kKT);  // rows of a box
    const int boxes = kKT / box * KCH;          // of a tile (at most 32)
    const int z_oob = p.num_pages * p.Hk;       // a page past the cache: zero fill
    const int sub = lane / KCH, c = lane % KCH; // this lane's box
    int g = 0, gk = 0, gv = 0;                  // tiles, and copies of K and V, so far
    int page_b = -1, page_lo = 0;               // page_s: entries page_lo .. of sequence page_b
    TreeUnit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit<true>(&units, un, w, end, lane, &wctl)) && !end; ++un) {
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
        if (lane < boxes && key < w.len) {
          const int pg = page_s[(key >> p.ps_shift) - page_lo];
          if (pg >= 0) {
            z = pg * p.Hk + w.kh;
            y = key & ((1 << p.ps_shift) - 1);
          }
        }
        const int st = g % ST;
        const uint32_t use = g / ST;
#pragma unroll
        for (int which = 0; which < 2; ++which) {
          uint64_t* full = which ? &v_full[st] : &k_full[st];
          if (leader) {
            if (use > 0) ok = wait(which ? &v_empty[st] : &k_empty[st], (use - 1) & 1, &wctl);
            if (ok) mbar_arrive_expect_tx(full, LY::KV_BYTES);
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
          uint8_t* dst = smem + (which ? LY::OFF_V : LY::OFF_K) + st * LY::KV_BYTES +
                         c * (kKT * 128) + sub * box * 128;
          if (lane < boxes) tma_load_3d(dst, which ? &mV : &mK, full, c * 64, y, z);
          ++(which ? gv : gk);
        }
      }
    }
    if (leader) {  // no copy may be in flight when the CTA ends
#pragma unroll 1
      for (int s = 0; s < ST; ++s) {
        const int nk = (gk - s + ST - 1) / ST, nv = (gv - s + ST - 1) / ST;  // copies into stage s
        if (nk > 0) mbar_wait_drain(&k_full[s], (nk - 1) & 1);
        if (nv > 0) mbar_wait_drain(&v_full[s], (nv - 1) & 1);
      }
    }
  } else if (warp == LY::S_WARP) {
    // ------------------------------------------------------------------ S = Q K^T
    const uint32_t id = idesc_bf16(128, kKT, 0, 0);
    int g = 0;
    TreeUnit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit<true>(&units, un, w, end, lane, &wctl)) && !end; ++un) {
      const int qs = PAIR ? un & 1 : 0;
      ok = wait_warp<false>(&q_full[qs], (PAIR ? un >> 1 : un) & 1, &wctl);
#pragma unroll 1
      for (int j = w.ja; j < w.jb && ok; ++j, ++g) {
        const int st = g % ST;
        ok = wait_warp(&k_full[st], (g / ST) & 1, &wctl);
#pragma unroll
        for (int i = 0; i < (PAIR ? 1 : NWG); ++i) {
          const int wg = PAIR ? g & 1 : i, n = PAIR ? g >> 1 : g, buf = n & 1;
          // the buffer's last P is done with
          if (ok && n >= 2) ok = wait_warp(&p_done[wg][buf], ((n >> 1) - 1) & 1, &wctl);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const Desc qa = make_desc(smem_u32(smem + (PAIR ? qs : i) * LY::Q_BYTES), 16, 1024);
            const Desc kb = make_desc(smem_u32(smem + LY::OFF_K + st * LY::KV_BYTES), 16, 1024);
            const uint32_t tS = tbase + LY::COL_S + (wg * 2 + buf) * kKT;
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks)
              mma_ss2(tS, qa.at((ks / 4) * (128 * 128) + (ks % 4) * 32), qa.hi,
                      kb.at((ks / 4) * (kKT * 128) + (ks % 4) * 32), kb.hi, id, ks > 0 ? 1u : 0u);
            mma_commit(&s_full[wg][buf]);
          }
          __syncwarp();
        }
        if (ok && lane == 0) mma_commit(&k_empty[st]);
      }
      if (ok && lane == 0) mma_commit(&q_free[qs]);
      __syncwarp();
    }
    if (lane == 0) {
      mma_commit(&drain_s);
      mbar_wait_drain(&drain_s, 0);
    }
    __syncwarp();
  } else if (warp == LY::O_WARP) {
    // ------------------------------------------------------------------ O += P V
    const uint32_t id = idesc_bf16(128, HD, 0, 1);
    int g = 0;
    TreeUnit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit<true>(&units, un, w, end, lane, &wctl)) && !end; ++un) {
      const int slot = un % kUnits, tree0 = w.len - p.T;
#pragma unroll 1
      for (int j = w.ja; j < w.jb && ok; ++j, ++g) {
        const int st = g % ST, n0 = j * kKT;
        uint8_t* vt = smem + LY::OFF_V + st * LY::KV_BYTES;
        ok = wait_warp(&v_full[st], (g / ST) & 1, &wctl);
        if (!ok) break;
        if (n0 + kKT > tree0) {
          tree_tile<HD>(vt, n0, tree0, w.len, units.odd[slot], lane);
          fence_proxy_async();
          __syncwarp();
        }
        if (j == w.jb - 1 && lane == 0) mbar_arrive(&units.odd_full[slot]);
        // a unit's first O is written over the last one's when both warpgroups have read that
        if (PAIR && j == w.ja && un > 0) ok = wait_warp(&o_free, (un - 1) & 1, &wctl);
#pragma unroll
        for (int i = 0; i < (PAIR ? 1 : NWG); ++i) {
          const int wg = PAIR ? g & 1 : i, n = PAIR ? g >> 1 : g, buf = n & 1;
          ok = ok && wait_warp(&p_full[wg][buf], (n >> 1) & 1, &wctl);
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t tP = tbase + LY::COL_S + (wg * 2 + buf) * kKT;
            const Desc vb = make_desc(smem_u32(vt), kKT * 128, 1024);  // V, MN-major
            const bool more = j - w.ja >= (PAIR ? 2 : 1);
#pragma unroll
            for (int ks = 0; ks < kKT / 16; ++ks)
              mma_ts2(tbase + wg * HD, tP + ks * 8, vb.at(ks * 2048), vb.hi, id,
                      more || ks > 0 ? 1u : 0u);
            mma_commit(&p_done[wg][buf]);
          }
          __syncwarp();
        }
        if (ok && lane == 0) mma_commit(&v_empty[st]);
        __syncwarp();
      }
    }
    if (lane == 0) {
      mma_commit(&drain_o);
      mbar_wait_drain(&drain_o, 0);
    }
    __syncwarp();
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
      if (!ended) {
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
          pack_mask(p.mask + list.b * p.mask_stride, bits + slot * p.T * p.words, p.T, p.words,
                    lane);
        if (lane < kTreeMax / 32) units.odd[slot][lane] = 0;
        __syncwarp();
      }
      if (lane == 0) {
        units.at[slot][0] = make_int4(list.b, list.kh, list.rb, list.ja);
        units.at[slot][1] =
            make_int4(list.jb, list.len, ended ? -1 : list.whole | list.first << 1, 0);
        mbar_arrive(&units.full[slot]);
      }
      __syncwarp();
      if (ended) break;
      const int qs = PAIR ? un & 1 : 0, turn = PAIR ? un >> 1 : un;
      if (turn > 0) ok = wait_warp(&q_free[qs], (turn - 1) & 1, &wctl);
      if (!ok) break;
      if (lane == 0) {
        constexpr int tiles = PAIR ? 1 : NWG;
        mbar_arrive_expect_tx(&q_full[qs], tiles * LY::Q_BYTES);
        for (int i = 0; i < tiles; ++i)
          for (int c = 0; c < KCH; ++c)
            tma_load_3d(smem + (PAIR ? qs : i) * LY::Q_BYTES + c * (128 * 128), &mQ, &q_full[qs],
                        c * 64, list.rb * LY::ROWS + i * 128, list.b * p.Hk + list.kh);
      }
      ++loads;
      __syncwarp();
    }
    if (lane == 0) {  // no copy may be in flight when the CTA ends
      if (PAIR) {
        if (loads > 0) mbar_wait_drain(&q_full[0], ((loads - 1) >> 1) & 1);
        if (loads > 1) mbar_wait_drain(&q_full[1], ((loads - 2) >> 1) & 1);
      } else if (loads > 0) {
        mbar_wait_drain(&q_full[0], (loads - 1) & 1);
      }
    }
  } else {
    // ------------------------------------------------------------------ softmax, and O out
    // Rows that are not there have q = 0 and columns that hold anything; warps without any row keep
    // the barriers going and do nothing else. A wait that runs out ends the warp's tiles; where the
    // warpgroups meet (PAIR) both leave together.
    const int wg = warp >> 2, wl = warp & 3, row = threadIdx.x & 127;
    const uint32_t lanes = tbase + ((uint32_t)(wl * 32) << 16);
    const uint32_t tO = lanes + wg * HD, tS = lanes + LY::COL_S + wg * 2 * kKT;
    const float c2 = p.scale_log2;
    int g = 0;  // PAIR: tiles of the CTA so far, this warpgroup's are those of its parity
    TreeUnit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0;; ++un) {
      ok = take_unit<false>(&units, un, w, end, lane, &wctl);
      if (PAIR ? soft_any<32 * LY::SOFT>(!ok) || end : !ok || end) break;
      const int slot = un % kUnits;
      const int r0 = w.rb * LY::ROWS + (PAIR ? 0 : wg * 128);
      const bool live = r0 + wl * 32 < p.rows, mine = r0 + row < p.rows;
      const int node = mine ? (r0 + row) % p.T : 0;
      const unsigned* sees = bits + (slot * p.T + node) * p.words;
      const int tree0 = w.len - p.T;
      float m = -FLT_MAX / 2.0f, l = 0.0f;
      bool any = false;  // a tile of the unit was this warpgroup's
#pragma unroll 1
      for (int j = w.ja + (PAIR ? (g ^ wg) & 1 : 0); j < w.jb; j += PAIR ? 2 : 1) {
        const int n = PAIR ? (g + j - w.ja) >> 1 : g + j - w.ja, buf = n & 1;
        const uint32_t at = tS + buf * kKT;
        ok = wait_warp(&s_full[wg][buf], (n >> 1) & 1, &wctl);
        if (!ok) break;
        if (live) {
          tc_fence_after();
          uint32_t s[2][32];
          tmem_ld32(at, s[0]);
          tmem_ld32(at + 32, s[1]);
          tmem_wait_ld();
          const int first = j * kKT - tree0;  // node of the tile's first key
          if (first + kKT > 0) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t vis = mask_bits(sees, p.words, first + h * 32);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(vis >> e & 1)) s[h][e] = 0xff800000u;  // -inf
            }
          }
          float mx = -INFINITY;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              mx = fmax3(mx, __uint_as_float(s[h][e]), __uint_as_float(s[h][e + 1]));
          const float m_new = fmaxf(m, mx * c2);
          if (!any) {
            m = m_new;
          } else if (__any_sync(0xffffffffu, m_new > m + kRescale)) {
            // O holds P V of this warpgroup's tiles before; only the last can be outstanding
            const float f = ex2(m - m_new);
            l *= f;
            ok = wait_warp(&p_done[wg][(n - 1) & 1], ((n - 1) >> 1) & 1, &wctl);
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
          float sum = 0.0f;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float a = ex2(fmaf(__uint_as_float(s[h][2 * e]), c2, -m));
              const float b = ex2(fmaf(__uint_as_float(s[h][2 * e + 1]), c2, -m));
              sum += a + b;
              pk[e] = pack_bf16(a, b);
            }
            tmem_st16(at + h * 16, pk);
          }
          l += sum;
          tmem_wait_st();
          tc_fence_before();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[wg][buf]);
        any = true;
      }
      // ---- the unit's end: O of all its tiles, of both warpgroups where they share the rows
      const int tiles = w.jb - w.ja;
      const int mine_last = PAIR ? g + tiles - 1 - ((g + tiles - 1 - wg) & 1) : g + tiles - 1;
      g += tiles;
      if (ok && any) {
        const int n = PAIR ? mine_last >> 1 : mine_last;  // this warpgroup's last item
        ok = wait_warp(&p_done[wg][n & 1], (n >> 1) & 1, &wctl);
      }
      if (ok) ok = wait_warp(&units.odd_full[slot], (un / kUnits) & 1, &wctl);
      float f0 = 1.0f, f1 = 0.0f;  // factors of O (this warpgroup's, or the first's) and the second's
      if (PAIR) {
        ml_s[un & 1][wg][row] = make_float2(m, l);
        tc_fence_before();  // (the other warpgroup reads this one's O too)
        if (soft_any<32 * LY::SOFT>(!ok)) break;
        const float2 a = ml_s[un & 1][0][row], b = ml_s[un & 1][1][row];
        m = fmaxf(a.x, b.x);
        f0 = a.y == 0.0f ? 0.0f : ex2(a.x - m);
        f1 = b.y == 0.0f ? 0.0f : ex2(b.x - m);
        l = a.y * f0 + b.y * f1;
      } else if (!ok) {
        break;
      } else if (l == 0.0f) {
        f0 = 0.0f;
      }
      tc_fence_after();
      bool odd = false;
#pragma unroll
      for (int k = 0; k < kTreeMax / 32; ++k) odd |= units.odd[slot][k] != 0;
      const size_t unit_row = ((size_t)w.b * p.Hk + w.kh) * p.rows + r0 + row;
      const size_t part = 2 * (size_t)blockIdx.x + (w.first ? 1 : 0);
      const int prow = PAIR ? row : wg * 128 + row;  // of the unit's rows
      float4* o_part = reinterpret_cast<float4*>(p.o_part) + part * (HD / 4) * LY::ROWS + prow;
      const float inv = l == 0.0f ? 0.0f : 1.0f / l;
      if (w.whole) {
        f0 *= inv;
        f1 *= inv;
      }
      if (live) {
        constexpr int COLS = PAIR ? HD / 2 : HD;
#pragma unroll 1
        for (int c = PAIR ? wg * COLS : 0, ce = c + COLS; c < ce; c += 16) {
          uint32_t x[16], y[16];
          tmem_ld16((PAIR ? lanes : tO) + c, x);
          if (PAIR) tmem_ld16(lanes + HD + c, y);
          tmem_wait_ld();
          float o[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            o[e] = f0 == 0.0f ? 0.0f : __uint_as_float(x[e]) * f0;  // (O of no weight holds anything)
            if (PAIR) o[e] += f1 == 0.0f ? 0.0f : __uint_as_float(y[e]) * f1;
          }
          if (odd && mine) {
            tree_odd(p, o, units.odd[slot], sees, w, HD, c);
            tree_odd(p, o + 8, units.odd[slot], sees, w, HD, c + 8);
          }
          if (!mine) {
          } else if (w.whole) {
            uint4* dst = reinterpret_cast<uint4*>(p.o + unit_row * HD + c);
#pragma unroll
            for (int k = 0; k < 2; ++k)
              dst[k] = make_uint4(pack_bf16(o[8 * k], o[8 * k + 1]), pack_bf16(o[8 * k + 2], o[8 * k + 3]),
                                  pack_bf16(o[8 * k + 4], o[8 * k + 5]),
                                  pack_bf16(o[8 * k + 6], o[8 * k + 7]));
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              o_part[(size_t)(c / 4 + k) * LY::ROWS] =
                  make_float4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
          }
          __syncwarp();
        }
        if (mine && (!PAIR || wg == 0)) {
          if (!w.whole) {
            p.ml_part[part * 2 * LY::ROWS + prow] = m;
            p.ml_part[(part * 2 + 1) * LY::ROWS + prow] = l;
          } else if (p.lse) {
            p.lse[unit_row] = l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l));
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (PAIR) mbar_arrive(&o_free);
        mbar_arrive(&units.free[slot]);
      }
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
    if (p.lse && warp == 0) p.lse[out] = -INFINITY;
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
      if (f != 0.0f) {
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] = fmaf(y[e], f, acc[e]);
      }
    }
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  *dst = make_uint4(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv),
                    pack_bf16(acc[4] * inv, acc[5] * inv), pack_bf16(acc[6] * inv, acc[7] * inv));
  if (p.lse && warp == 0) p.lse[out] = l == 0.0f ? -INFINITY : fmaf(m, kLn2, logf(l));
}

struct TreePlan {
  int ROWS, rb, grid;
};
TreePlan tree_plan(const TreeArgs& a) {
  TreePlan pl;
  const int rows = a.G * a.T;
  pl.ROWS = rows <= 128 || a.d > 128 ? 128 : 256;
  pl.rb = (rows + pl.ROWS - 1) / pl.ROWS;
  const long long cap = (long long)a.max_pages << a.ps_shift;
  const long long tiles = ((cap + kKT - 1) / kKT + kUnitCost) * a.B * a.Hk * pl.rb;
  pl.grid = (int)std::min<long long>(152, tiles);
  return pl;
}

template <int HD, bool PAIR>
cudaError_t launch_tree_t(const TreeArgs& a, const TreeMaps& m, void* ws, cudaStream_t s) {
  using LY = TreeLayout<HD, PAIR>;
  static OncePerKey<> smem_attr;
  const TreePlan pl = tree_plan(a);
  auto kern = tree_kernel<HD, PAIR>;
  cudaError_t e = set_smem_once(smem_attr, kern, LY::smem_bytes(kTreeMax));
  if (e != cudaSuccess) return e;
  TreeK p;
  p.v = static_cast<const __nv_bfloat16*>(a.v_cache);
  p.table = a.table;
  p.lens = a.lens;
  p.mask = a.mask;
  p.mask_stride = a.mask_stride;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.o_part = static_cast<float*>(ws);
  p.ml_part = p.o_part + (size_t)2 * pl.grid * LY::ROWS * HD;
  p.status = a.status;
  p.B = a.B;
  p.Hk = a.Hk;
  p.T = a.T;
  p.words = (a.T + 31) / 32;
  p.rows = a.G * a.T;
  p.rb = pl.rb;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.ps_shift = a.ps_shift;
  p.scale_log2 = a.scale * kLog2e;
  p.wait_limit_ns = a.wait_limit_ns;
  profile_mark(kKernTreeAttn, 0, s);
  kern<<<pl.grid, LY::THREADS, LY::smem_bytes(a.T), s>>>(m.q, m.k, m.v, p);
  e = cudaGetLastError();
  profile_mark(kKernTreeAttn, 1, s);
  if (e != cudaSuccess) return e;
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
  return (size_t)2 * pl.grid * pl.ROWS * (a.d + 2) * 4;
}

cudaError_t launch_tree(const TreeArgs& a, const TreeMaps& m, void* ws, cudaStream_t s) {
  const bool pair = a.G * a.T <= 128;
  switch (a.d) {
    case 64: return pair ? launch_tree_t<64, true>(a, m, ws, s) : launch_tree_t<64, false>(a, m, ws, s);
    case 128:
      return pair ? launch_tree_t<128, true>(a, m, ws, s) : launch_tree_t<128, false>(a, m, ws, s);
    case 256: return launch_tree_t<256, false>(a, m, ws, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
