// fa_q8_cache.cu -- the 8-bit key/value cache's writer (quantise new rows into the pages) and
// reader (a batch's rows back as bf16), sm_103a.
//
// Writer. The n new rows of sequence b become its positions first .. len - 1, first = len - n.
// Positions fall into scale blocks of sb slots (sb divides the page size, so a block lies in one
// page). For each block that gets a new row, with a the largest finite |x| of its new rows:
//   s = 2^k, k = max(ceil(log2(a / 448)), -100)       (448: the largest e4m3 value)
//   s = max(s, the block's scale) if the block holds earlier tokens of the sequence
//   new codes e4m3(x / s); where s grew, earlier codes c become e4m3(c * (old scale / s))
// A power of two costs an e4m3 code nothing (its precision is relative), makes x / s exact (one
// rounding a value) and lets a block's earlier codes survive a growing scale unchanged unless
// they leave the normal range. In bf16 bits k is the exponent field - 135, + 1 above 1.75 times
// the binade (448 = 1.75 * 2^8), so the rule runs on integers.
//
// Both kernels move bytes (2 in and 1 out for an element, or 1 in and 2 out) and are bound by
// HBM as long as they spend few instructions on an element: at 164 and 138 for 8 elements they
// were bound by issue (85 and 66 us for 16 prompts of up to 8k tokens). So a lane holds 8 columns
// of a row, a warp takes 8 steps of 32 / (d / 8) rows, all loaded before the first is used (4 KB
// of bf16), and the way to them (sequence, length, table) is gone once for four heads. Where the
// rows of a warp lie in one page (page_size >= 2048 / d) they are one run of bytes; smaller pages
// are looked up row by row. A scale block up to a warp's rows is reduced inside the warp, a larger
// one over the warps of its CTA.
#include <math.h>

#include "fa_common.cuh"
#include "fa_launch.h"
#include "fa_q8.cuh"

namespace fa {

namespace {
constexpr int kSteps = 8;  // row steps of a warp

template <int HD>
struct RowLanes {
  static constexpr int LPR = HD / 8;           // lanes of a row
  static constexpr int RPS = 32 / LPR;         // rows of a step
  static constexpr int TR = RPS * kSteps;      // rows of a warp
};

struct Q8RowsK {
  uint8_t* codes[2];   // k, v
  float* scales[2];
  __nv_bfloat16* rows[2];
  long long st_b[2], st_h[2], st_r[2];  // strides of `rows` in elements
  const int32_t* cu;     // packed batch: [B + 1]; nullptr: new_len rows for each sequence
  const int32_t* table;  // [B, max_pages]
  const int32_t* lens;   // [B] (writer)
  int* status;
  int B, Hk, total, new_len, max_pages, num_pages, ps_shift, sb_shift;
  unsigned page_bytes, page_scales;  // of the codes and scales of a page's heads
};

__device__ __forceinline__ void flag_bad(int* status) {
  if (status) atomicCAS(status, kStatusOk, kStatusBadInput);
}

// Rows of sequence b: where they start in the packed batch, and how many there are.
__device__ __forceinline__ void seq_rows(const Q8RowsK& p, int b, int& start, int& n) {
  start = 0;
  n = p.new_len;
  if (p.cu) varlen_seq(p.cu, b, p.total, p.total, start, n);
}

// The offsets of sequence `item` are out of range (item i looks at sequence i's; there are at least
// four items a sequence). What finds a slot's owner takes offsets that do not decrease, and may
// pass over a sequence where they do: no owner would report it.
__device__ __forceinline__ bool bad_offsets(const Q8RowsK& p, long long item) {
  int start, n;
  return p.cu && item < p.B && varlen_seq(p.cu, (int)item, p.total, p.total, start, n);
}

// Pages of a warp's `rows` rows from position p0 on: lane i holds that of entry
// (p0 >> ps_shift) + i, -1 where the table names none of the cache. Entries whose positions all
// lie outside [from, end) are not read.
__device__ __forceinline__ int lane_page(const Q8RowsK& p, int b, int p0, int rows, int from,
                                         int end, int lane, bool& bad) {
  const int entry = (p0 >> p.ps_shift) + lane;
  if (lane > (rows - 1) >> p.ps_shift || (long long)entry << p.ps_shift >= end ||
      (long long)(entry + 1) << p.ps_shift <= from)
    return -1;
  const int pg = p.table[(size_t)b * p.max_pages + entry];
  if (pg >= 0 && pg < p.num_pages) return pg;
  bad = true;
  return -1;
}

// Scale exponent of a block whose largest finite |x| has the bf16 bits `amax`.
__device__ __forceinline__ int scale_exp(uint32_t amax) {
  return max((int)(amax >> 7) - 135 + ((amax & 0x7fu) > 0x60u ? 1 : 0), kQ8MinExp);
}
__device__ __forceinline__ float exp2i(int k) { return __int_as_float((k + 127) << 23); }

__device__ __forceinline__ float2 bf16x2_f32(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// x / s for 8 values of a row as codes, where s = 1 / inv is a power of two (x * inv is exact).
__device__ __forceinline__ uint2 quantise8(const uint4& x, float inv) {
  const uint64_t inv2 = f2_pack(inv, inv);
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t c[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float lo, hi;
    f2_unpack(f2_mul(f2_pack(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u)),
                     inv2), lo, hi);
    c[e] = e4m3x2_from_f32(lo, hi);
  }
  return make_uint2(__byte_perm(c[0], c[1], 0x5410), __byte_perm(c[2], c[3], 0x5410));
}
// The same for any s and any values (the cases that are rare: a scale that another writer chose
// stays, or a value is not finite): NaN where the conversion would saturate an infinity.
__device__ __noinline__ uint2 quantise8_any(uint4 x, float s) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float y[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = bf16x2_f32(w[e]);
    y[2 * e] = isfinite(f.x) ? f.x / s : NAN;
    y[2 * e + 1] = isfinite(f.y) ? f.y / s : NAN;
  }
  return make_uint2(e4m3x4_from_f32(y[0], y[1], y[2], y[3]),
                    e4m3x4_from_f32(y[4], y[5], y[6], y[7]));
}
// Codes times a ratio below 1, rounded again.
__device__ __noinline__ uint2 requantise8(uint2 c, float ratio) {
  const float2 f0 = f32_from_e4m3x2(c.x), f1 = f32_from_e4m3x2(c.x >> 16);
  const float2 f2 = f32_from_e4m3x2(c.y), f3 = f32_from_e4m3x2(c.y >> 16);
  return make_uint2(e4m3x4_from_f32(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio),
                    e4m3x4_from_f32(f2.x * ratio, f2.y * ratio, f3.x * ratio, f3.y * ratio));
}
// |x| of 8 values, the largest in each half (the order of bf16 bits is that of their absolute
// values; infinities and NaN lie at and above 0x7f80).
__device__ __forceinline__ uint32_t absmax8(const uint4& x, uint32_t m) {
  m = __vmaxu2(m, x.x & 0x7fff7fffu);
  m = __vmaxu2(m, x.y & 0x7fff7fffu);
  m = __vmaxu2(m, x.z & 0x7fff7fffu);
  return __vmaxu2(m, x.w & 0x7fff7fffu);
}
__device__ __noinline__ uint4 finite8(uint4 x) {  // 0 for what is not finite
  x.x &= ~__vcmpgeu2(x.x & 0x7fff7fffu, 0x7f807f80u);
  x.y &= ~__vcmpgeu2(x.y & 0x7fff7fffu, 0x7f807f80u);
  x.z &= ~__vcmpgeu2(x.z & 0x7fff7fffu, 0x7f807f80u);
  x.w &= ~__vcmpgeu2(x.w & 0x7fff7fffu, 0x7f807f80u);
  return x;
}

// SPB: steps of a scale block inside a warp (1: a block of at most one step). `wpb` warps of
// the CTA share a unit of max(rows of a warp, scale block) positions. An item is a unit of K or V
// of `heads` heads in turn. ONE: the rows of a warp lie in one page. THREADS: 256, or up to 1024
// where a scale block takes more than 8 warps.
template <int HD, int SPB, bool ONE, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 3 : 1)
    q8_write_kernel(const Q8RowsK p, long long items, int wpb, int heads) {
  using RL = RowLanes<HD>;
  constexpr int GROUPS = kSteps / SPB;
  __shared__ uint32_t warp_max[32];
  const int warp = warp_id(), lane = lane_id();
  const int sb = 1 << p.sb_shift, ps_mask = (1 << p.ps_shift) - 1;
  const int unit = RL::TR * wpb;
  const long long item = (long long)blockIdx.x * (blockDim.x / 32 / wpb) + warp / wpb;
  const int which = (int)(item & 1);
  const int hgroups = (p.Hk + heads - 1) / heads;
  const int h0 = (int)((item >> 1) % hgroups) * heads;
  const long long slot = (item >> 1) / hgroups;
  bool live = item < items, bad = bad_offsets(p, item);
  int b = 0, start = 0, n = 0, len = 0, first = 0, p0 = 0;
  if (live) {
    auto offset = [&](int i) { return p.cu ? (long long)p.cu[i] : (long long)i * p.new_len; };
    b = q8_slot_owner(slot, p.B, unit, lane, offset);
    len = p.lens[b];
    seq_rows(p, b, start, n);
    if (len < 0 || len > (long long)p.max_pages << p.ps_shift) {  // no place is the right one
      bad = true;
      live = false;
    }
    first = len - n;
    const long long u = slot - (offset(b) / unit + 2ll * b);
    const long long at = (max(first, 0) / unit + u) * unit;  // first position of this unit
    live = live && u >= 0 && at < len && n > 0;
    p0 = live ? (int)at + (warp % wpb) * RL::TR : 0;
  }
  const int lo = max(first, 0);  // new rows are the positions lo .. len - 1
  const int r = lane / RL::LPR, col = lane % RL::LPR * 8;
  // what the rows p0 + t * RPS + r are, bit t: new, or written or looked at (earlier rows of a
  // block that gets a new one are); `page`: theirs, ONE: that of them all
  const int lane_pg = live ? lane_page(p, b, p0, RL::TR, lo & ~(sb - 1), len, lane, bad) : -1;
  uint32_t isnew = 0, look = 0;
  int page[ONE ? 1 : kSteps];
#pragma unroll
  for (int t = 0; t < kSteps; ++t) {
    const int pos = p0 + t * RL::RPS + r;
    const int pg =
        __shfl_sync(0xffffffffu, lane_pg, ONE ? 0 : (pos >> p.ps_shift) - (p0 >> p.ps_shift));
    page[ONE ? 0 : t] = pg;
    isnew |= (uint32_t)(live && pos >= lo && pos < len) << t;
    look |= (uint32_t)(live && pos < len && (pos | (sb - 1)) >= lo && pg >= 0) << t;
  }
  // earlier tokens of a block: only the block that `first` lies in has some
  const bool has_old = live && (p0 & ~(sb - 1)) < first && sb > 1;
  const int lanes = min(32, RL::LPR << p.sb_shift);  // lanes of a block
  // most warps: nothing but new rows
  const bool full = ONE && !has_old && __all_sync(0xffffffffu, isnew == 0xffu && look == 0xffu);
  const long long row_step = RL::RPS * p.st_r[which];
  const __nv_bfloat16* src =
      p.rows[which] + h0 * p.st_h[which] + col +
      (p.cu ? (long long)start * p.st_r[which] : b * p.st_b[which]) +
      (long long)(p0 - first + r) * p.st_r[which];
  for (int h = 0; h < heads; ++h, src += p.st_h[which]) {
    const int head = h0 + h;
    const bool on = live && head < p.Hk;
    uint4 x[kSteps];
    uint32_t m[GROUPS];
    if (full && on) {
#pragma unroll
      for (int t = 0; t < kSteps; ++t)
        x[t] = __ldg(reinterpret_cast<const uint4*>(src + t * row_step));
    } else {
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        x[t] = make_uint4(0u, 0u, 0u, 0u);
        if (on && (isnew >> t & 1))
          x[t] = __ldg(reinterpret_cast<const uint4*>(src + t * row_step));
      }
    }
    uint32_t odd = 0;
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      m[g] = 0;
#pragma unroll
      for (int t = g * SPB; t < (g + 1) * SPB; ++t) m[g] = absmax8(x[t], m[g]);
      odd = __vmaxu2(odd, m[g]);
    }
    odd = max(odd & 0xffffu, odd >> 16);
    const bool any = __any_sync(0xffffffffu, odd >= 0x7f80u);  // a value is not finite
    if (any) {
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        m[g] = 0;
#pragma unroll
        for (int t = g * SPB; t < (g + 1) * SPB; ++t) m[g] = absmax8(finite8(x[t]), m[g]);
      }
    }
    // of a row's lanes: the page's codes of this head, and its scales
    auto codes = [&](int t) {
      const int in = (p0 & ps_mask) + t * RL::RPS + r;  // (ONE: no wrap)
      return p.codes[which] + (size_t)(unsigned)page[ONE ? 0 : t] * p.page_bytes +
             ((unsigned)((head << p.ps_shift) + (ONE ? in : in & ps_mask)) * HD + col);
    };
    auto scale = [&](int t) {
      const int in = ((p0 & ps_mask) + t * RL::RPS + r) & ps_mask;
      return p.scales[which] + (size_t)(unsigned)page[ONE ? 0 : t] * p.page_scales +
             (unsigned)((head << (p.ps_shift - p.sb_shift)) + (in >> p.sb_shift));
    };
    float was[GROUPS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      m[g] = max(m[g] & 0xffffu, m[g] >> 16);
      if (lanes == 32) {
        m[g] = __reduce_max_sync(0xffffffffu, m[g]);
      } else {
        for (int o = lanes / 2; o > 0; o /= 2)
          m[g] = max(m[g], __shfl_xor_sync(0xffffffffu, m[g], o));
      }
      // the block's scale where it holds earlier tokens, read before any warp writes it
      was[g] = 0.0f;
      if (has_old) {
#pragma unroll
        for (int t = g * SPB; t < (g + 1) * SPB; ++t)
          if (on && (look >> t & 1) && ((p0 + t * RL::RPS + r) & ~(sb - 1)) < first)
            was[g] = *scale(t);
        for (int o = lanes / 2; o > 0; o /= 2)
          was[g] = fmaxf(was[g], __shfl_xor_sync(0xffffffffu, was[g], o));
      }
    }
    if (wpb > 1) {  // (then GROUPS = 1: one block for each unit)
      if (lane == 0) warp_max[warp] = m[0];
      __syncthreads();
      for (int i = warp / wpb * wpb; i < (warp / wpb + 1) * wpb; ++i) m[0] = max(m[0], warp_max[i]);
      __syncthreads();
    }
    if (!on) continue;
    if (full && !any) {
      uint8_t* dst = codes(0);
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const float s = exp2i(scale_exp(m[g]));
        const float inv = __uint_as_float(0x7f000000u - __float_as_uint(s));
#pragma unroll
        for (int t = g * SPB; t < (g + 1) * SPB; ++t)
          *reinterpret_cast<uint2*>(dst + t * (RL::RPS * HD)) = quantise8(x[t], inv);
        // (a block of several steps begins with the first one's first row)
        if (col == 0 && (SPB > 1 ? r == 0 : (r & (sb - 1)) == 0) &&
            ((p0 & (sb - 1)) == 0 || SPB < 8))
          *scale(g * SPB) = s;
      }
      continue;
    }
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const float s = fmaxf(exp2i(scale_exp(m[g])), was[g]);
      const bool plain = !any && (__float_as_uint(s) & 0x7fffffu) == 0;
      const float inv = __uint_as_float(0x7f000000u - __float_as_uint(s));  // (a power of two's)
#pragma unroll
      for (int t = g * SPB; t < (g + 1) * SPB; ++t) {
        if (!(look >> t & 1)) continue;
        uint2* dst = reinterpret_cast<uint2*>(codes(t));
        if (isnew >> t & 1) {
          *dst = plain ? quantise8(x[t], inv) : quantise8_any(x[t], s);
          // the block's scale, by its first new row
          const int pos = p0 + t * RL::RPS + r;
          if (col == 0 && ((pos & (sb - 1)) == 0 || pos == lo)) *scale(t) = s;
        } else if (was[g] > 0.0f && s > was[g]) {
          *dst = requantise8(*dst, was[g] / s);
        }
      }
    }
  }
  if (bad) flag_bad(p.status);
}

// Row i of sequence b is its key i: bf16(code * scale). ONE, `heads`: as for the writer.
template <int HD, bool ONE>
__global__ void __launch_bounds__(256, 4)
    q8_read_kernel(const Q8RowsK p, long long items, int heads) {
  using RL = RowLanes<HD>;
  const int warp = warp_id(), lane = lane_id();
  const int ps_mask = (1 << p.ps_shift) - 1;
  const long long item = (long long)blockIdx.x * 8 + warp;
  if (item >= items) return;
  const int which = (int)(item & 1);
  const int hgroups = (p.Hk + heads - 1) / heads;
  const int h0 = (int)((item >> 1) % hgroups) * heads;
  const long long slot = (item >> 1) / hgroups;
  auto offset = [&](int i) { return (long long)p.cu[i]; };
  const int b = q8_slot_owner(slot, p.B, RL::TR, lane, offset);
  int start, n;
  varlen_seq(p.cu, b, p.total, p.total, start, n);
  bool bad = bad_offsets(p, item);
  const long long cap = (long long)p.max_pages << p.ps_shift;
  bad |= n > cap;
  const long long u = slot - (offset(b) / RL::TR + 2ll * b);
  if (u >= 0 && u * RL::TR < n) {
    const int p0 = (int)(u * RL::TR), end = (int)(n < cap ? n : cap);
    const int r = lane / RL::LPR, col = lane % RL::LPR * 8;
    const int lane_pg = lane_page(p, b, p0, RL::TR, 0, end, lane, bad);
    // bit t: row p0 + t * RPS + r is there (else zeros: past the table's end, or of no page)
    uint32_t have = 0;
    int page[ONE ? 1 : kSteps];
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const int pos = p0 + t * RL::RPS + r;
      const int pg =
          __shfl_sync(0xffffffffu, lane_pg, ONE ? 0 : (pos >> p.ps_shift) - (p0 >> p.ps_shift));
      page[ONE ? 0 : t] = pg;
      have |= (uint32_t)(pos < end && pg >= 0) << t;
    }
    const long long row_step = RL::RPS * p.st_r[which];
    __nv_bfloat16* dst = p.rows[which] + h0 * p.st_h[which] + col +
                         (long long)(start + p0 + r) * p.st_r[which];
    const int stop = min(p.Hk, h0 + heads);
    const bool one_scale = ONE && (1 << p.sb_shift) >= RL::TR;  // of all the warp's rows
    for (int head = h0; head < stop; ++head, dst += p.st_h[which]) {
      uint2 c[kSteps];
      float s[kSteps];
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        const int in = (p0 & ps_mask) + t * RL::RPS + r;
        c[t] = make_uint2(0u, 0u);
        if (have >> t & 1)
          c[t] = __ldg(reinterpret_cast<const uint2*>(
              p.codes[which] + (size_t)(unsigned)page[ONE ? 0 : t] * p.page_bytes +
              ((unsigned)((head << p.ps_shift) + (ONE ? in : in & ps_mask)) * HD + col)));
      }
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        const int in = ((p0 & ps_mask) + t * RL::RPS + r) & ps_mask;
        s[t] = t > 0 && one_scale ? s[0] : 0.0f;
        if ((t == 0 || !one_scale) && (have >> t & 1))
          s[t] = __ldg(p.scales[which] + (size_t)(unsigned)page[ONE ? 0 : t] * p.page_scales +
                       (unsigned)((head << (p.ps_shift - p.sb_shift)) + (in >> p.sb_shift)));
      }
#pragma unroll
      for (int t = 0; t < kSteps; ++t) {
        if (p0 + t * RL::RPS + r >= n) continue;
        const uint64_t s2 = f2_pack(s[t], s[t]);
        const uint32_t w[4] = {c[t].x, c[t].x >> 16, c[t].y, c[t].y >> 16};
        uint32_t o[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 f = f32_from_e4m3x2(w[e]);
          float x, y;
          f2_unpack(f2_mul(f2_pack(f.x, f.y), s2), x, y);
          o[e] = pack_bf16(x, y);
        }
        __stcs(reinterpret_cast<uint4*>(dst + t * row_step), make_uint4(o[0], o[1], o[2], o[3]));
      }
    }
  }
  if (bad) flag_bad(p.status);
}

Q8RowsK rows_params(const Q8RowsArgs& a) {
  Q8RowsK p;
  for (int w = 0; w < 2; ++w) {
    p.codes[w] = static_cast<uint8_t*>(a.codes[w]);
    p.scales[w] = a.scales[w];
    p.rows[w] = static_cast<__nv_bfloat16*>(a.rows[w]);
    p.st_b[w] = a.st_b[w];
    p.st_h[w] = a.st_h[w];
    p.st_r[w] = a.st_r[w];
  }
  p.cu = a.cu;
  p.table = a.table;
  p.lens = a.lens;
  p.status = a.status;
  p.B = a.B;
  p.Hk = a.Hk;
  p.total = a.total;
  p.new_len = a.new_len;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.ps_shift = a.ps_shift;
  p.sb_shift = a.sb_shift;
  p.page_bytes = (unsigned)a.Hk * a.d << a.ps_shift;  // (checked to fit)
  p.page_scales = (unsigned)a.Hk << (a.ps_shift - a.sb_shift);
  return p;
}

// Heads of an item: four, where that still leaves 16 warps for each SM.
int heads_of(long long warps_per_head, int Hk) {
  return Hk >= 4 && warps_per_head * Hk / 4 >= 152 * 16 ? 4 : 1;
}

template <int HD, int SPB, bool ONE>
cudaError_t write_t(const Q8RowsArgs& a, cudaStream_t s) {
  using RL = RowLanes<HD>;
  const int sb = 1 << a.sb_shift;
  const int wpb = sb > RL::TR ? sb / RL::TR : 1;
  const int warps = wpb > 8 ? wpb : 8;
  const long long total = a.cu ? a.total : (long long)a.B * a.new_len;
  const long long slots = q8_unit_slots(total, a.B, RL::TR * wpb);
  const int heads = heads_of(slots * wpb * 2, a.Hk);
  const long long items = slots * ((a.Hk + heads - 1) / heads) * 2;
  const long long per = warps / wpb;
  const unsigned grid = (unsigned)((items + per - 1) / per);
  profile_mark(kKernQ8Write, 0, s);
  if constexpr (SPB == 8 && ONE && HD >= 128) {
    if (warps > 8)
      q8_write_kernel<HD, SPB, ONE, 1024><<<grid, warps * 32, 0, s>>>(rows_params(a), items, wpb,
                                                                      heads);
  }
  if (warps == 8)
    q8_write_kernel<HD, SPB, ONE, 256><<<grid, 256, 0, s>>>(rows_params(a), items, wpb, heads);
  const cudaError_t e = cudaGetLastError();
  profile_mark(kKernQ8Write, 1, s);
  return e;
}

template <int HD, int SPB>
cudaError_t write_s(const Q8RowsArgs& a, cudaStream_t s) {
  // (a block of 8 steps is all of a warp's rows, and a page holds whole blocks; at head_dim 256 a
  // warp has 8 rows, the smallest page)
  if constexpr (SPB < 8 && RowLanes<HD>::TR > 8)
    if ((1 << a.ps_shift) < RowLanes<HD>::TR) return write_t<HD, SPB, false>(a, s);
  return write_t<HD, SPB, true>(a, s);
}

template <int HD>
cudaError_t write_d(const Q8RowsArgs& a, cudaStream_t s) {
  const int spb = (1 << a.sb_shift) / RowLanes<HD>::RPS;  // steps of a block (0: less than one)
  if (spb >= 8) return write_s<HD, 8>(a, s);
  if (spb == 4) return write_s<HD, 4>(a, s);
  if (spb == 2) return write_s<HD, 2>(a, s);
  return write_s<HD, 1>(a, s);
}

template <int HD>
cudaError_t read_d(const Q8RowsArgs& a, cudaStream_t s) {
  const long long slots = q8_unit_slots(a.total, a.B, RowLanes<HD>::TR);
  const int heads = heads_of(slots * 2, a.Hk);
  const long long items = slots * ((a.Hk + heads - 1) / heads) * 2;
  const unsigned grid = (unsigned)((items + 7) / 8);
  profile_mark(kKernQ8Read, 0, s);
  bool one = true;
  if constexpr (RowLanes<HD>::TR > 8) {
    one = (1 << a.ps_shift) >= RowLanes<HD>::TR;
    if (!one) q8_read_kernel<HD, false><<<grid, 256, 0, s>>>(rows_params(a), items, heads);
  }
  if (one) q8_read_kernel<HD, true><<<grid, 256, 0, s>>>(rows_params(a), items, heads);
  const cudaError_t e = cudaGetLastError();
  profile_mark(kKernQ8Read, 1, s);
  return e;
}
}  // namespace

long long q8_rows_items(const Q8RowsArgs& a) {
  const int tr = 2048 / a.d;  // rows of a warp; larger units make fewer items
  const long long total = a.cu ? a.total : (long long)a.B * a.new_len;
  return q8_unit_slots(total, a.B, tr) * a.Hk * 2;
}

cudaError_t launch_q8_write(const Q8RowsArgs& a, cudaStream_t s) {
  switch (a.d) {
    case 64: return write_d<64>(a, s);
    case 128: return write_d<128>(a, s);
    case 256: return write_d<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_q8_read(const Q8RowsArgs& a, cudaStream_t s) {
  switch (a.d) {
    case 64: return read_d<64>(a, s);
    case 128: return read_d<128>(a, s);
    case 256: return read_d<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
