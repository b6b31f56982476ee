// fa_q8_chunk.cuh -- the 8-bit cache's attention for many query rows a kv head (a chunk of a
// prompt), included by fa_q8_attn.cu: the same units, shares and joining kernel, in blocks of 128
// rows.
//
// With 128 rows on a tile of 128 keys the codes are read once for all of them, and what counts is
// the work for each score. So the query rows are the M of both products (a thread has a row and
// half the keys of a tile; its row's maximum and sum are its own), and the operands are f16:
//  * codes widened to f16 (exact) as they are stored to shared memory, in the 128-byte swizzled
//    rows that the tensor cores read, by four warps of their own, each thread from the bytes that
//    it has asked for itself (cp.async into shared memory, one tile ahead at head_dim 128, two at
//    64: without a barrier, and without the registers that loads would hold);
//  * q times a power of two for each row (its largest element into [128, 256)): exact down to
//    2^-32 of that element;
//  * weights in f16: 11 bits, in steps of 2^-35 of the row's largest at least; they go to tensor
//    memory, from where O += w V takes them.
// The scales are those of the tile's columns here, from shared memory; m, the sums and their
// units are those of the smaller blocks.
//
// What bounds it: the softmax's warps, which wait for little (at head_dim 64 7 % of their time for
// scores, 3 % at their votes, 5 % for a free half of w): two of them on a scheduler, with their
// exponentials and the chain from scores to weights; at head_dim 128 the widening's shared-memory
// traffic too. A tile takes about 3000 cycles at head_dim 64 and 3600 at 128, for any number of
// its 128 rows: 16 sequences of 4k to 16k keys, 8 kv heads of 128 rows, 168 M scores: 112 us and
// 139 us. (From about 640 rows a kv head on, reading the keys back as bf16 and the variable-length
// attention are faster.) Tried: codes through registers instead of cp.async (they spilled: 410 us
// for 48 rows at head_dim 128 where cp.async took 185), scores 32 columns and scales 8 keys at a
// time (no faster).
//
// Warps: 0-7 softmax (two warpgroups, half the keys of a tile each, and half the columns of O),
// 8-11 keys and values, 12 the MMAs, 13 the list of units. One CTA an SM.
#pragma once

namespace fa {
namespace {

template <int HD>
struct Q8Chunk {
  static constexpr int R = 128;
  static constexpr int KV_BYTES = kKT * HD * 2;
  static constexpr int OFF_K = R * HD * 2;  // after Q: two K tiles, two V tiles
  static constexpr int OFF_V = OFF_K + 2 * KV_BYTES;
  // Codes on their way: tiles ahead of the one that is being widened, slots of a K or V tile.
  static constexpr int AHEAD = HD == 64 ? 2 : 1, SLOTS = 2 * AHEAD + 1;
  static constexpr int OFF_C = OFF_V + 2 * KV_BYTES;
  static constexpr int SMEM_BYTES = OFF_C + SLOTS * kKT * HD + 1024;
  static constexpr int COL_S = 0, COL_O = 2 * kKT, COL_P = 3 * kKT;  // two S, O, two w (f16)
  static constexpr int TMEM_COLS = 512;
  static constexpr int SOFT = 8, CONV = 4, MMA_WARP = 12, LIST_WARP = 13;
  static constexpr int THREADS = 32 * 14;
  static_assert(HD <= 128, "O has 128 columns");
  static_assert(SMEM_BYTES + 9216 + 1024 <= 228 * 1024, "shared memory budget");  // (and static)
};

// kind::f16 with f16 operands, f32 accumulator.
constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) |
         ((uint32_t)(M >> 4) << 24);
}
// Where the 8 elements from column `col` (a multiple of 8) of row r of a tile of 128 rows lie:
// chunks of 64 columns, rows of 128 bytes, swizzled.
__device__ __forceinline__ int f16_at(int r, int col) {
  return col / 64 * (128 * 128) + r * 128 + ((col % 64 / 8) ^ (r & 7)) * 16;
}
// Four codes -> four f16.
__device__ __forceinline__ uint2 f16x4_from_e4m3(uint32_t c) {
  uint2 h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h.x) : "h"((uint16_t)c));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h.y) : "h"((uint16_t)(c >> 16)));
  return h;
}
__device__ __forceinline__ uint32_t f16x2_from_f32(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}
// 16 bytes, or zeros, to shared memory; the groups of a thread, in order.
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, bool have) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(have ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// The barrier of the softmax's 256 threads; true where any of them came with `v`.
__device__ __forceinline__ bool chunk_any(bool v) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.pred q, 1, 256, p;\n"
      " selp.s32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)v)
      : "memory");
  return r != 0;
}

// The same for the 64 threads that have rows 32 `pair` .. + 31: a warp of each half.
__device__ __forceinline__ bool pair_any(int pair, bool v) {
  int r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.s32 p, %1, 0;\n barrier.cta.red.or.pred q, %2, 64, p;\n"
      " selp.s32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((int)v), "r"(pair + 2)
      : "memory");
  return r != 0;
}

template <int HD, bool MULTI>
__global__ void __launch_bounds__(Q8Chunk<HD>::THREADS, 1) q8_chunk_kernel(const Q8K p) {
  using LY = Q8Chunk<HD>;
  constexpr int R = LY::R;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  __shared__ uint64_t k_full[2], v_full[2], s_full[2], s_free[2], p_full[2], p_done[2], q_full;
  __shared__ uint64_t drain;
  __shared__ __align__(16) UnitRing units;
  __shared__ uint32_t tmem_base_s;
  __shared__ WaitCtl wctl;
  __shared__ int bad_input;
  // Of a tile's keys: key scale, log2 of the value scale, its inverse in the sums' unit. Written
  // when the scores of two tiles before are read, so that the weights of three before are done.
  __shared__ __align__(16) float ks_s[4][kKT];
  __shared__ __align__(16) float lv_s[4][kKT];
  __shared__ __align__(16) float iv_s[5][kKT];  // (the last: zeros)
  // Largest and least of the value scales' log2 that each of the warps has: of the unit's tiles so
  // far, of this one.
  __shared__ __align__(16) float most_s[2][LY::CONV], least_s[2][LY::CONV];
  __shared__ int iv_at[4];  // where in iv_s the sum of a tile takes its factors
  __shared__ unsigned vn_s[2][kKT / 32];  // keys whose value has a NaN, where some rows see it
  __shared__ float qs_s[R], red_s[2][R];  // rows: score factor; maxima or sums of the two halves

  const int warp = warp_id(), lane = lane_id();
  Walk list;
  if (warp == LY::LIST_WARP) list.init(p, blockIdx.x, gridDim.x, lane);
  if (threadIdx.x < kKT) iv_s[4][threadIdx.x] = 0.0f;
  if (threadIdx.x == 0) {
    wait_ctl_init(&wctl, p.wait_limit_ns);
    bad_input = 0;
#pragma unroll 1
    for (int s = 0; s < 2; ++s) {
      mbar_init(&k_full[s], 4);
      mbar_init(&v_full[s], 4);
      mbar_init(&s_full[s], 2);  // the MMA, and (through the MMA's warp) the keys' scales
      mbar_init(&s_free[s], LY::SOFT);  // S is read; its MMA has read K before
      mbar_init(&p_full[s], LY::SOFT);
      mbar_init(&p_done[s], 1);         // O has the tile; w and V are free
    }
#pragma unroll 1
    for (int s = 0; s < kUnits; ++s) {
      mbar_init(&units.full[s], 1);
      mbar_init(&units.free[s], LY::SOFT + LY::CONV + 1);
    }
    mbar_init(&q_full, LY::SOFT);
    mbar_init(&drain, 1);
    fence_barrier_init();
  }
  if (warp == LY::MMA_WARP) {
    tmem_alloc(&tmem_base_s, LY::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = tmem_base_s;
  grid_dep_trigger();

  if (warp == LY::LIST_WARP) {
    if (blockIdx.x == 0) {  // lengths out of range are clamped, and reported here
      bool bad = false;
#pragma unroll 1
      for (int b = lane; b < p.B; b += 32) bad |= p.lens[b] != q8_len(p, b);
      if (bad) bad_input = 1;
    }
    bool ended = false;
#pragma unroll 1
    for (int un = 0; !ended; ++un) {
      const int slot = un % kUnits;
      if (un >= kUnits && !wait_warp(&units.free[slot], (un / kUnits - 1) & 1, &wctl)) break;
      ended = !list.next<MULTI>(p, R);
      if (lane == 0) {
        units.at[slot][0] = make_int4(list.b, list.kh, list.rb, list.ja);
        units.at[slot][1] =
            make_int4(list.jb, list.len, ended ? -1 : list.whole | list.first << 1, 0);
        mbar_arrive(&units.full[slot]);
      }
      __syncwarp();
    }
  } else if (warp == LY::MMA_WARP) {
    const uint32_t id_s = idesc_f16(R, kKT, 0, 0), id_o = idesc_f16(R, HD, 0, 1);
    const Desc qa = make_desc(smem_u32(smem), 16, 1024);
    int g = 0, nq = 0;  // tiles whose O is issued; units with tiles (the others have no q)
    Unit w;
    bool ok = true, end = false;
    auto issue_s = [&](int g) {
      const int buf = g & 1;
      ok = wait_warp(&k_full[buf], (g >> 1) & 1, &wctl) &&
           (g < 2 || wait_warp(&s_free[buf], ((g >> 1) - 1) & 1, &wctl));
      if (!ok) return;
      tc_fence_after();
      if (lane == 0) {
        const Desc kb = make_desc(smem_u32(smem + LY::OFF_K + buf * LY::KV_BYTES), 16, 1024);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const int at = ks / 4 * (128 * 128) + ks % 4 * 32;
          mma_ss2(tbase + LY::COL_S + buf * kKT, qa.at(at), qa.hi, kb.at(at), kb.hi, id_s,
                  ks > 0 ? 1u : 0u);
        }
        mma_commit(&s_full[buf]);
        // value scales too far apart for w / v_scale: the sum takes exponentials of its own
        const float4 hi = *reinterpret_cast<const float4*>(most_s[buf]);
        const float4 lo = *reinterpret_cast<const float4*>(least_s[buf]);
        const float most = fmaxf(fmaxf(hi.x, hi.y), fmaxf(hi.z, hi.w));
        const float least = fminf(fminf(lo.x, lo.y), fminf(lo.z, lo.w));
        iv_at[g & 3] = most - least > kApart ? 4 : g & 3;
        mbar_arrive(&s_full[buf]);
      }
      __syncwarp();
    };
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit(&units, un, w, end, lane, &wctl)) && !end; ++un) {
      if (w.ja == w.jb) continue;
      ok = wait_warp<false>(&q_full, nq++ & 1, &wctl);
#pragma unroll 1
      for (int j = w.ja - 1; j < w.jb && ok; ++j) {  // S runs one tile ahead of O
        if (j + 1 < w.jb) issue_s(g + (j >= w.ja ? 1 : 0));
        if (j < w.ja || !ok) continue;
        const int buf = g & 1;
        ok = wait_warp(&v_full[buf], (g >> 1) & 1, &wctl) &&
             wait_warp(&p_full[buf], (g >> 1) & 1, &wctl);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const Desc vb =
              make_desc(smem_u32(smem + LY::OFF_V + buf * LY::KV_BYTES), 128 * 128, 1024);
#pragma unroll
          for (int ks = 0; ks < kKT / 16; ++ks)
            mma_ts2(tbase + LY::COL_O, tbase + LY::COL_P + buf * (kKT / 2) + ks * 8,
                    vb.at(ks * 2048), vb.hi, id_o, (j > w.ja || ks > 0) ? 1u : 0u);
          mma_commit(&p_done[buf]);
        }
        __syncwarp();
        ++g;
      }
    }
    if (lane == 0) {
      mma_commit(&drain);
      mbar_wait_drain(&drain, 0);
    }
    __syncwarp();
  } else if (warp >= LY::SOFT) {
    // ------------------------------------------------------------------ codes to f16 tiles
    // A warp has 32 keys of the tile: lane l the page and the scale of key l; of the codes LPR
    // lanes have a row (16 codes each), RPS rows at a time.
    constexpr int LPR = HD / 16, RPS = 32 / LPR, STEPS = 32 / RPS;
    // (at head_dim 128 the lanes of a row's two halves change places with those of the next row:
    // what 8 lanes store together then lies in different banks)
    const int row0 = (warp - LY::SOFT) * 32, rr = lane / LPR ^ (HD == 128 ? lane >> 2 & 1 : 0);
    const int col = lane % LPR * 16;
    const int nb_shift = p.ps_shift - p.sb_shift, ps_mask = (1 << p.ps_shift) - 1;
    const size_t page_bytes = (size_t)p.Hk * HD << p.ps_shift;
    const size_t page_scales = (size_t)p.Hk << nb_shift;
    const uint32_t raw = smem_u32(smem + LY::OFF_C) + (warp - LY::SOFT) * (32 * HD) + lane * 16;
    int g = 0;
    uint32_t largest = 0;  // bits of the scales read
    Unit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0; ok && (ok = take_unit(&units, un, w, end, lane, &wctl)) && !end; ++un) {
      const int32_t* table = p.table + (size_t)w.b * p.max_pages;
      const int end_key = min(w.len, w.jb * kKT);
      const unsigned in_page = ((unsigned)w.kh * HD << p.ps_shift) + col;
      const unsigned head_scales = (unsigned)w.kh << nb_shift;
      // The page of this lane's key of tile j (-1: there is no key), not looked at before it is
      // used: a test here would wait for the load.
      auto page_of = [&](int j) {
        const int key = j * kKT + row0 + lane;
        return key < end_key ? table[key >> p.ps_shift] : -1;
      };
      auto is_page = [&](int pg) { return (unsigned)pg < (unsigned)p.num_pages; };
      // K and V of the g-th tile, j of the unit, whose pages are pg, into slots 2 g and 2 g + 1
      auto fetch = [&](int g, int j, int pg) {
        const uint32_t dk = raw + 2 * g % LY::SLOTS * (kKT * HD);
        const uint32_t dv = raw + (2 * g + 1) % LY::SLOTS * (kKT * HD);
        if (j < w.jb) {
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const int r = s * RPS + rr, page = __shfl_sync(0xffffffffu, pg, r);
            const unsigned in = (unsigned)(j * kKT + row0 + r) & ps_mask;
            const bool have = is_page(page);  // (else zeros)
            const size_t at = (have ? (unsigned)page : 0u) * page_bytes + (in * HD + in_page);
            copy16_async(dk + s * 512, p.codes[0] + at, have);
            copy16_async(dv + s * 512, p.codes[1] + at, have);
          }
        }
        copies_commit();
      };
      auto scale_of = [&](const float* scales, int j, int pg) {  // (keys that are not there have
        const int key = j * kKT + row0 + lane, in = key & ps_mask;  // codes of 0 and no weight)
        if (is_page(pg))
          return __ldg(scales + pg * page_scales + (head_scales + (in >> p.sb_shift)));
        if (key < end_key) bad_input = 1;
        return 1.0f;
      };
      float most = -INFINITY;
      int pg[LY::AHEAD + 2];  // of tiles j, j + 1, ..
#pragma unroll
      for (int i = 0; i < LY::AHEAD + 1; ++i) pg[i] = page_of(w.ja + i);
      float ks = scale_of(p.k_scale, w.ja, pg[0]), vs = scale_of(p.v_scale, w.ja, pg[0]);
#pragma unroll
      for (int i = 0; i < LY::AHEAD; ++i) fetch(g + i, w.ja + i, pg[i]);
#pragma unroll 1
      for (int j = w.ja; j < w.jb; ++j, ++g) {
        const int buf = g & 1;
        pg[LY::AHEAD + 1] = page_of(j + LY::AHEAD + 1);
        auto codes_of = [&](int item, int s) {
          uint4 x;
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                       : "r"(raw + item % LY::SLOTS * (kKT * HD) + s * 512)
                       : "memory");
          return x;
        };
        auto store = [&](uint8_t* tile, int s, const uint4& x) {
          const int r = row0 + s * RPS + rr;
          const uint2 a = f16x4_from_e4m3(x.x), b = f16x4_from_e4m3(x.y);
          const uint2 c = f16x4_from_e4m3(x.z), d = f16x4_from_e4m3(x.w);
          *reinterpret_cast<uint4*>(tile + f16_at(r, col)) = make_uint4(a.x, a.y, b.x, b.y);
          *reinterpret_cast<uint4*>(tile + f16_at(r, col + 8)) = make_uint4(c.x, c.y, d.x, d.y);
        };
        if (g >= 2) ok = wait_warp(&s_free[buf], ((g >> 1) - 1) & 1, &wctl);
        if (!ok) break;
        const float l = lg2(fmaxf(vs, __int_as_float((kQ8MinExp + 127) << 23)));
        largest = max(largest, max(__float_as_uint(ks), __float_as_uint(vs)));
        ks_s[g & 3][row0 + lane] = ks;
        lv_s[g & 3][row0 + lane] = l;
        iv_s[g & 3][row0 + lane] = ex2(-l - kSumExp);
        most = fmaxf(most, warp_max(l));
        const float least = -warp_max(-l);
        if (lane == 0) {
          most_s[buf][warp - LY::SOFT] = most;
          least_s[buf][warp - LY::SOFT] = least;
        }
        ks = scale_of(p.k_scale, j + 1, pg[1]);
        vs = scale_of(p.v_scale, j + 1, pg[1]);
        copies_wait<LY::AHEAD - 1>();
        uint4 x[STEPS];
#pragma unroll
        for (int s = 0; s < STEPS; ++s) x[s] = codes_of(2 * g, s);
#pragma unroll
        for (int s = 0; s < STEPS; ++s) store(smem + LY::OFF_K + buf * LY::KV_BYTES, s, x[s]);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&k_full[buf]);

        // (into the slots of this tile's K and of the last one's V)
        fetch(g + LY::AHEAD, j + LY::AHEAD, pg[LY::AHEAD]);
        if (g >= 2) ok = wait_warp(&p_done[buf], ((g >> 1) - 1) & 1, &wctl);
        if (!ok) break;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) x[s] = codes_of(2 * g + 1, s);
        unsigned nans = 0;
        if (MULTI && (j + 1) * kKT > w.len - p.lq + 1) {
          // Keys that not every row sees: NaN in a value must meet no weight there, not even 0.
          // Its code becomes 0, and the key's weight NaN where it is seen.
          const int hidden = w.len - p.lq + 1 - j * kKT - row0;
#pragma unroll
          for (int s = 0; s < STEPS; ++s) {
            const int r = s * RPS + rr;
            const uint4 z = make_uint4(nan_bytes(x[s].x), nan_bytes(x[s].y),
                                       nan_bytes(x[s].z), nan_bytes(x[s].w));
            if (r >= hidden && (z.x | z.y | z.z | z.w)) {
              x[s].x &= ~((z.x >> 7) * 0xffu);
              x[s].y &= ~((z.y >> 7) * 0xffu);
              x[s].z &= ~((z.z >> 7) * 0xffu);
              x[s].w &= ~((z.w >> 7) * 0xffu);
              nans |= 1u << r;
            }
          }
          nans = __reduce_or_sync(0xffffffffu, nans);
        }
        if (lane == 0) vn_s[buf][warp - LY::SOFT] = nans;
#pragma unroll
        for (int s = 0; s < STEPS; ++s) store(smem + LY::OFF_V + buf * LY::KV_BYTES, s, x[s]);
#pragma unroll
        for (int i = 0; i < LY::AHEAD + 1; ++i) pg[i] = pg[i + 1];
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&v_full[buf]);
      }
    }
    copies_wait<0>();
    if (largest > kQ8MaxScale) bad_input = 1;
  } else {
    // ------------------------------------------------------------------ q, softmax, and O out
    // Rows that are not there have q = 0. A row is two threads', and its 32 rows two warps': these
    // vote on a tile alone (all 256 threads together, with two more waits a tile: 32.7 us for 5
    // sequences of up to 4k keys and 128 rows, so 28.8). A wait that runs out shows at the next
    // vote, where both leave the tiles; the vote at a unit's end takes all out of the loop.
    const int wg = warp >> 2, row = threadIdx.x & 127, col0 = wg * 64;
    const uint32_t lanes = tbase + ((uint32_t)((warp & 3) * 32) << 16);
    int g = 0;
    Unit w;
    bool ok = true, end = false;
#pragma unroll 1
    for (int un = 0;; ++un) {
      ok = take_unit(&units, un, w, end, lane, &wctl);
      if (chunk_any(!ok) || end) break;
      const int r0 = w.rb * R, live = min(R, p.rows - r0);
      const size_t unit_row = ((size_t)w.b * p.Hk + w.kh) * p.rows + r0;
      const bool any = w.jb > w.ja;
      if (any) {  // q: two threads a row (every warp has seen the last unit's scores: Q is free)
        constexpr int N = HD / 16;  // 16-byte loads of a thread
        const int qr = threadIdx.x >> 1, c0 = (threadIdx.x & 1) * (HD / 2);
        const uint4* src = reinterpret_cast<const uint4*>(p.q + (unit_row + qr) * HD + c0);
        uint4 x[N];
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) {
          x[e] = qr < live ? __ldg(src + e) : make_uint4(0u, 0u, 0u, 0u);
          m = __vmaxu2(__vmaxu2(m, x[e].x & 0x7fff7fffu), x[e].y & 0x7fff7fffu);
          m = __vmaxu2(__vmaxu2(m, x[e].z & 0x7fff7fffu), x[e].w & 0x7fff7fffu);
        }
        m = max(m & 0xffffu, m >> 16);
        m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
        // 2^sh puts the row's largest element into [128, 256); a row with an element that is not
        // finite becomes NaN
        const int sh = 134 - (int)max(m >> 7, 1u);
        const float f0 = __int_as_float((sh / 2 + 127) << 23);
        const float f1 = __int_as_float((sh - sh / 2 + 127) << 23);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const uint32_t xs[4] = {x[e].x, x[e].y, x[e].z, x[e].w};
          uint32_t h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            h[i] = m >= 0x7f80u ? 0x7fff7fffu
                                : f16x2_from_f32(__uint_as_float(xs[i] << 16) * f0 * f1,
                                                 __uint_as_float(xs[i] & 0xffff0000u) * f0 * f1);
          *reinterpret_cast<uint4*>(smem + f16_at(qr, c0 + 8 * e)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
        if (c0 == 0)
          qs_s[qr] = p.scale_log2 * __int_as_float((127 - sh / 2) << 23) *
                     __int_as_float((127 - (sh - sh / 2)) << 23);
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full);
      }
      chunk_any(false);
      const float qs = qs_s[row];
      const uint64_t qs2 = f2_pack(qs, qs);
      const int lim = MULTI ? max(0, w.len - p.lq + (r0 + row) % p.lq + 1) : w.len;
      // tiles below lim_min need no test of the keys
      const int lim_min = MULTI ? max(0, w.len - p.lq + 1) : w.len;
      float nm = 0.0f;  // -m
      uint64_t l2 = 0;  // the sum, in two parts
#pragma unroll 1
      for (int j = w.ja; j < w.jb; ++j, ++g) {
        const int buf = g & 1;
        const uint32_t ph = (g >> 1) & 1;
        ok = ok && wait_warp(&s_full[buf], ph, &wctl);
        tc_fence_after();
        const bool first = j == w.ja;
        const int at = iv_at[g & 3];
        const uint64_t nm2 = f2_pack(nm, nm);
        float t[64];
        uint32_t sr[2][16];  // scores of 16 keys, and of the next 16 on their way
        tmem_ld16(lanes + LY::COL_S + buf * kKT + col0, sr[0]);
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 16) {
          ulonglong2 k4[4], l4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            k4[c] = *reinterpret_cast<const ulonglong2*>(&ks_s[g & 3][col0 + c0 + 4 * c]);
            l4[c] = *reinterpret_cast<const ulonglong2*>(&lv_s[g & 3][col0 + c0 + 4 * c]);
          }
          tmem_wait_ld();
          if (c0 < 48)
            tmem_ld16(lanes + LY::COL_S + buf * kKT + col0 + c0 + 16, sr[(c0 / 16 + 1) & 1]);
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            const uint32_t* s = &sr[c0 / 16 & 1][c];
            const uint64_t k2 = c & 2 ? k4[c / 4].y : k4[c / 4].x;
            const uint64_t l2v = c & 2 ? l4[c / 4].y : l4[c / 4].x;
            const uint64_t s2 = f2_pack(__uint_as_float(s[0]), __uint_as_float(s[1]));
            f2_unpack(f2_fma(f2_mul(s2, k2), qs2, f2_add(l2v, nm2)), t[c0 + c], t[c0 + c + 1]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_free[buf]);
        if (j * kKT + kKT > lim_min) {
          const int left = lim - j * kKT - col0;
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c >= left) t[c] = -INFINITY;
        }
        float top = t[0], top1 = t[1];
#pragma unroll
        for (int c = 2; c < 62; c += 4) {
          top = fmax3(top, t[c], t[c + 1]);
          top1 = fmax3(top1, t[c + 2], t[c + 3]);
        }
        top = fmaxf(fmax3(top, t[62], t[63]), top1);
        if (pair_any(warp & 3, top > kMost || first || !ok)) {
          // m moves: to the largest score so far, at a unit's first tile to the tile's own
          red_s[wg][row] = top;
          if (pair_any(warp & 3, !ok)) {
            ok = false;
            break;
          }
          const float mx = fmaxf(red_s[0][row], red_s[1][row]);
          float up = mx - kTop;
          if (first ? mx == -INFINITY : !(up > 0.0f)) up = 0.0f;
          nm -= up;
          const float f = ex2(-up);
#pragma unroll
          for (int c = 0; c < 64; ++c) t[c] -= up;
          if (!first) {  // O is scaled too, once the last O MMA is done
            const float root = ex2(-0.5f * up);  // (scale_sum)
            l2 = f2_mul(f2_mul(l2, f2_pack(root, root)), f2_pack(root, root));
            ok = wait_warp(&p_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &wctl);
            tc_fence_after();
#pragma unroll 1
            for (int c = 0; c < HD / 2; c += 8) {
              const uint32_t at = lanes + LY::COL_O + wg * (HD / 2) + c;
              float x[8];
              tmem_ld8(at, x);
              tmem_wait_ld();
#pragma unroll
              for (int e = 0; e < 8; ++e) x[e] *= f;
              tmem_st8(at, x);
            }
            tmem_wait_st();
          }
        }
        if (at == 4) {
          // (rare, and a loop through local memory: unrolled it made every tile slower)
          float4 y[16];
#pragma unroll
          for (int c = 0; c < 16; ++c)
            y[c] = make_float4(t[4 * c], t[4 * c + 1], t[4 * c + 2], t[4 * c + 3]);
          float x = 0.0f;
#pragma unroll 1
          for (int c = 0; c < 64; ++c)
            x += ex2_full(reinterpret_cast<const float*>(y)[c] - lv_s[g & 3][col0 + c] - kSumExp);
          l2 = f2_add(l2, f2_pack(x, 0.0f));
        }
        // weights and their sum; to the tensor cores as f16
        if (g >= 2) ok = ok && wait_warp(&p_done[buf], ph ^ 1, &wctl);
        uint32_t pw[32];
#pragma unroll
        for (int c0 = 0; c0 < 64; c0 += 16) {
          ulonglong2 i4[4];
#pragma unroll
          for (int c = 0; c < 4; ++c)
            i4[c] = *reinterpret_cast<const ulonglong2*>(&iv_s[at][col0 + c0 + 4 * c]);
#pragma unroll
          for (int c = c0; c < c0 + 16; c += 4) {
            const float a = ex2(t[c]), b = ex2(t[c + 1]), d = ex2(t[c + 2]), e = ex2(t[c + 3]);
            l2 = f2_fma(f2_pack(a, b), i4[(c - c0) / 4].x, l2);
            l2 = f2_fma(f2_pack(d, e), i4[(c - c0) / 4].y, l2);
            pw[c / 2] = f16x2_from_f32(a, b);
            pw[c / 2 + 1] = f16x2_from_f32(d, e);
          }
        }
        if (MULTI && j * kKT + kKT > lim_min) {
          ok = ok && wait_warp(&v_full[buf], ph, &wctl);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned nans = vn_s[buf][wg * 2 + h];
            if (nans == 0) continue;
            const int left = lim - j * kKT - col0 - h * 32;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if ((nans >> c & 1) && c < left) pw[h * 16 + c / 2] |= 0x7fffu << (c % 2 * 16);
          }
        }
        tc_fence_after();
        tmem_st32(lanes + LY::COL_P + buf * (kKT / 2) + wg * 32, pw);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[buf]);
      }
      float la, lb;
      f2_unpack(l2, la, lb);
      if (any && ok) ok = wait_warp(&p_done[(g - 1) & 1], ((g - 1) >> 1) & 1, &wctl);
      red_s[wg][row] = la + lb;
      if (chunk_any(!ok)) break;
      tc_fence_after();
      // a row without keys: sum 0, and O 0
      const float sum = red_s[0][row] + red_s[1][row];
      const size_t part = 2 * (size_t)blockIdx.x + (w.first ? 1 : 0);
      const size_t out_row = w.whole ? unit_row + row : part * R + row;
#pragma unroll 1
      for (int c = wg * (HD / 2); c < (wg + 1) * (HD / 2); c += 8) {
        float x[8] = {};
        if (any) {
          tmem_ld8(lanes + LY::COL_O + c, x);
          tmem_wait_ld();
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (w.whole) x[e] = __fdividef(x[e], sum) / kSumUnit;  // (2 ulp; rounded to bf16)
          if (sum == 0.0f) x[e] = 0.0f;
        }
        if (row >= live) {
        } else if (w.whole) {
          *reinterpret_cast<uint4*>(p.o + out_row * HD + c) =
              make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                         pack_bf16(x[6], x[7]));
        } else {
          float4* dst = reinterpret_cast<float4*>(p.o_part + out_row * HD + c);
          dst[0] = make_float4(x[0], x[1], x[2], x[3]);
          dst[1] = make_float4(x[4], x[5], x[6], x[7]);
        }
        __syncwarp();
      }
      if (wg == 0 && row < live) {
        const float m = any ? -nm : 0.0f;
        if (!w.whole) {
          p.ml_part[part * 2 * R + row] = m;
          p.ml_part[part * 2 * R + R + row] = sum;
        } else if (p.lse) {
          p.lse[unit_row + row] = sum == 0.0f ? -INFINITY : fmaf(m + kSumExp, kLn2, logf(sum));
        }
      }
      // (red_s is written again behind the next unit's votes)
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == LY::MMA_WARP) tmem_dealloc(tbase, LY::TMEM_COLS);
  if (threadIdx.x == 0) {
    report_abort(&wctl, p.status);
    if (bad_input && p.status) atomicCAS(p.status, kStatusOk, kStatusBadInput);
  }
}

}  // namespace
}  // namespace fa
