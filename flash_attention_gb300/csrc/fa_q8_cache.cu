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
// HBM. A lane holds 8 columns of a row; a warp takes 8 steps of 32 / (d / 8) rows, all of them
// loaded before the first is used, so that 4 KB of bf16 are in flight for each warp. A scale
// block up to that size is reduced inside its warp, a larger one over the warps of its CTA.
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
};

__device__ __forceinline__ void flag_bad(int* status) {
  if (status) atomicCAS(status, kStatusOk, kStatusBadInput);
}

// Rows of sequence b: where they start in the packed batch, and how many there are.
__device__ __forceinline__ bool seq_rows(const Q8RowsK& p, int b, int& start, int& n) {
  if (!p.cu) {
    start = 0;
    n = p.new_len;
    return false;
  }
  return varlen_seq(p.cu, b, p.total, p.total, start, n);
}

// Page of a position, or -1 (and a flag) where the table names none.
__device__ __forceinline__ int page_of(const Q8RowsK& p, int b, int pos, bool& bad) {
  const int pg = p.table[(size_t)b * p.max_pages + (pos >> p.ps_shift)];
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
  const float2 a = bf16x2_f32(x.x), b = bf16x2_f32(x.y), c = bf16x2_f32(x.z), d = bf16x2_f32(x.w);
  return make_uint2(e4m3x4_from_f32(a.x * inv, a.y * inv, b.x * inv, b.y * inv),
                    e4m3x4_from_f32(c.x * inv, c.y * inv, d.x * inv, d.y * inv));
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
__device__ __forceinline__ uint4 finite8(uint4 x) {  // 0 for what is not finite
  x.x &= ~__vcmpgeu2(x.x & 0x7fff7fffu, 0x7f807f80u);
  x.y &= ~__vcmpgeu2(x.y & 0x7fff7fffu, 0x7f807f80u);
  x.z &= ~__vcmpgeu2(x.z & 0x7fff7fffu, 0x7f807f80u);
  x.w &= ~__vcmpgeu2(x.w & 0x7fff7fffu, 0x7f807f80u);
  return x;
}

// SPB: steps of a scale block inside a warp (1: a block of at most one step). `wpb` warps of
// the CTA share a unit of max(rows of a warp, scale block) positions. An item is a unit of K or V
// of `heads` heads in turn, which share the way to the unit (offsets, length, table).
// THREADS: 256, or up to 1024 where a scale block takes more than 8 warps.
template <int HD, int SPB, int THREADS>
__global__ void __launch_bounds__(THREADS, THREADS == 256 ? 3 : 1)
    q8_write_kernel(const Q8RowsK p, long long items, int wpb, int heads) {
  using RL = RowLanes<HD>;
  constexpr int GROUPS = kSteps / SPB;
  __shared__ uint32_t warp_max[32];
  const int warp = warp_id(), lane = lane_id();
  const int sb = 1 << p.sb_shift, ps_mask = (1 << p.ps_shift) - 1;
  const int nb_shift = p.ps_shift - p.sb_shift;
  const int unit = RL::TR * wpb;
  const long long item = (long long)blockIdx.x * (blockDim.x / 32 / wpb) + warp / wpb;
  const int which = (int)(item & 1);
  const int hgroups = (p.Hk + heads - 1) / heads;
  const int h0 = (int)((item >> 1) % hgroups) * heads;
  const long long slot = (item >> 1) / hgroups;
  bool live = item < items, bad = false;
  int b = 0, start = 0, n = 0, len = 0, first = 0, p0 = 0;
  if (live) {
    auto offset = [&](int i) { return p.cu ? (long long)p.cu[i] : (long long)i * p.new_len; };
    b = q8_slot_owner(slot, p.B, unit, lane, offset);
    len = p.lens[b];
    bad |= seq_rows(p, b, start, n);
    if (len < 0 || len > (long long)p.max_pages << p.ps_shift) {  // no place is the right one
      bad = true;
      live = false;
    }
    first = len - n;
    const long long u = slot - (offset(b) / unit + 2ll * b);
    const long long at = (max(first, 0) / unit + u) * unit;  // first position of this unit
    live = live && u >= 0 && at < len && n > 0;
    p0 = (int)at + (warp % wpb) * RL::TR;
  }
  const int lo = max(first, 0);  // new rows are the positions lo .. len - 1
  const int r = lane / RL::LPR, col = lane % RL::LPR * 8;
  // pages of the warp's rows: lane i holds that of entry (p0 >> ps_shift) + i
  int page = -1;
  if (live && lane <= (RL::TR - 1) >> p.ps_shift && ((p0 >> p.ps_shift) + lane) << p.ps_shift < len)
    page = p.table[(size_t)b * p.max_pages + (p0 >> p.ps_shift) + lane];
  int at[kSteps];  // page of the row; -1: left out
  bool isnew[kSteps];
#pragma unroll
  for (int t = 0; t < kSteps; ++t) {
    const int pos = p0 + t * RL::RPS + r;
    at[t] = __shfl_sync(0xffffffffu, page, (pos >> p.ps_shift) - (p0 >> p.ps_shift));
    isnew[t] = live && pos >= lo && pos < len;
    // earlier rows of a block that gets a new one are looked at too
    const bool look = live && pos < len && (pos | (sb - 1)) >= lo;
    if (look && (at[t] < 0 || at[t] >= p.num_pages)) bad = true;
    if (!look || at[t] < 0 || at[t] >= p.num_pages) at[t] = -1;
  }
  // earlier tokens of a block: only the block that `first` lies in has some
  const bool has_old = live && p0 < first;
  const int lanes = min(32, RL::LPR << p.sb_shift);  // lanes of a block
  for (int h = 0; h < heads; ++h) {
    const int head = h0 + h;
    const bool on = live && head < p.Hk;
    const __nv_bfloat16* src = p.rows[which] + head * p.st_h[which] + col +
                               (p.cu ? (long long)start * p.st_r[which] : b * p.st_b[which]);
    uint4 x[kSteps];
    uint32_t m[GROUPS];
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      x[t] = make_uint4(0u, 0u, 0u, 0u);
      if (on && isnew[t])
        x[t] = __ldg(reinterpret_cast<const uint4*>(
            src + (long long)(p0 - first + t * RL::RPS + r) * p.st_r[which]));
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
        for (int t = g * SPB; t < (g + 1) * SPB; ++t) {
          const int pos = p0 + t * RL::RPS + r;
          if (on && at[t] >= 0 && (pos & ~(sb - 1)) < first)
            was[g] = p.scales[which][(((size_t)at[t] * p.Hk + head) << nb_shift) +
                                     ((pos & ps_mask) >> p.sb_shift)];
        }
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
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) {
      const float s = fmaxf(exp2i(scale_exp(m[g])), was[g]);
      const bool plain = !any && (__float_as_uint(s) & 0x7fffffu) == 0;
      const float inv = __uint_as_float(0x7f000000u - __float_as_uint(s));  // (a power of two's)
#pragma unroll
      for (int t = g * SPB; t < (g + 1) * SPB; ++t) {
        if (at[t] < 0) continue;
        const int pos = p0 + t * RL::RPS + r, in = pos & ps_mask;
        const size_t row = (size_t)at[t] * p.Hk + head;
        uint2* dst = reinterpret_cast<uint2*>(p.codes[which] + ((row << p.ps_shift) + in) * HD + col);
        if (isnew[t]) {
          *dst = plain ? quantise8(x[t], inv) : quantise8_any(x[t], s);
          // the block's scale, by its first new row
          if (col == 0 && ((in & (sb - 1)) == 0 || pos == lo))
            p.scales[which][(row << nb_shift) + (in >> p.sb_shift)] = s;
        } else if (was[g] > 0.0f && s > was[g]) {
          *dst = requantise8(*dst, was[g] / s);
        }
      }
    }
  }
  if (bad) flag_bad(p.status);
}

// Row i of sequence b is its key i: bf16(code * scale).
template <int HD>
__global__ void __launch_bounds__(256) q8_read_kernel(const Q8RowsK p, long long items) {
  using RL = RowLanes<HD>;
  const int warp = warp_id(), lane = lane_id();
  const long long item = (long long)blockIdx.x * 8 + warp;
  if (item >= items) return;
  const int which = (int)(item & 1);
  const int head = (int)((item >> 1) % p.Hk);
  const long long slot = (item >> 1) / p.Hk;
  auto offset = [&](int i) { return (long long)p.cu[i]; };
  const int b = q8_slot_owner(slot, p.B, RL::TR, lane, offset);
  int start, n;
  bool bad = varlen_seq(p.cu, b, p.total, p.total, start, n);
  const long long cap = (long long)p.max_pages << p.ps_shift;
  bad |= n > cap;
  const long long u = slot - (offset(b) / RL::TR + 2ll * b);
  const long long p0 = u * RL::TR;
  const int r = lane / RL::LPR, col = lane % RL::LPR * 8;
  if (u >= 0 && p0 < n) {
    __nv_bfloat16* dst = p.rows[which] + head * p.st_h[which] + start * p.st_r[which] + col;
    uint2 c[kSteps];
    float s[kSteps];
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const long long pos = p0 + t * RL::RPS + r;
      c[t] = make_uint2(0u, 0u);
      s[t] = 0.0f;
      if (pos >= n || pos >= cap) continue;  // (rows past the table's end: zeros, flagged)
      const int pg = page_of(p, b, (int)pos, bad);
      if (pg < 0) continue;
      const int slot_in = (int)pos & ((1 << p.ps_shift) - 1);
      const size_t at = (size_t)pg * p.Hk + head;
      c[t] = __ldg(reinterpret_cast<const uint2*>(p.codes[which] +
                                                  ((at << p.ps_shift) + slot_in) * HD + col));
      s[t] = __ldg(p.scales[which] + (at << (p.ps_shift - p.sb_shift)) + (slot_in >> p.sb_shift));
    }
#pragma unroll
    for (int t = 0; t < kSteps; ++t) {
      const long long pos = p0 + t * RL::RPS + r;
      if (pos >= n) continue;
      const float2 f0 = f32_from_e4m3x2(c[t].x), f1 = f32_from_e4m3x2(c[t].x >> 16);
      const float2 f2 = f32_from_e4m3x2(c[t].y), f3 = f32_from_e4m3x2(c[t].y >> 16);
      uint4 out;
      out.x = pack_bf16(f0.x * s[t], f0.y * s[t]);
      out.y = pack_bf16(f1.x * s[t], f1.y * s[t]);
      out.z = pack_bf16(f2.x * s[t], f2.y * s[t]);
      out.w = pack_bf16(f3.x * s[t], f3.y * s[t]);
      *reinterpret_cast<uint4*>(dst + pos * p.st_r[which]) = out;
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
  return p;
}

template <int HD, int SPB>
cudaError_t write_t(const Q8RowsArgs& a, cudaStream_t s) {
  using RL = RowLanes<HD>;
  const int sb = 1 << a.sb_shift;
  const int wpb = sb > RL::TR ? sb / RL::TR : 1;
  const int warps = wpb > 8 ? wpb : 8;
  const long long total = a.cu ? a.total : (long long)a.B * a.new_len;
  const long long slots = q8_unit_slots(total, a.B, RL::TR * wpb);
  // heads of an item: four, where that still leaves 16 warps for each SM
  const int heads = a.Hk >= 4 && slots * wpb * a.Hk / 4 * 2 >= 152 * 16 ? 4 : 1;
  const long long items = slots * ((a.Hk + heads - 1) / heads) * 2;
  const long long per = warps / wpb;
  profile_mark(kKernQ8Write, 0, s);
  const unsigned grid = (unsigned)((items + per - 1) / per);
  if constexpr (SPB == 8 && HD >= 128) {
    if (warps > 8)
      q8_write_kernel<HD, SPB, 1024><<<grid, warps * 32, 0, s>>>(rows_params(a), items, wpb, heads);
  }
  if (warps == 8)
    q8_write_kernel<HD, SPB, 256><<<grid, 256, 0, s>>>(rows_params(a), items, wpb, heads);
  const cudaError_t e = cudaGetLastError();
  profile_mark(kKernQ8Write, 1, s);
  return e;
}

template <int HD>
cudaError_t write_d(const Q8RowsArgs& a, cudaStream_t s) {
  const int spb = (1 << a.sb_shift) / RowLanes<HD>::RPS;  // steps of a block (0: less than one)
  if (spb >= 8) return write_t<HD, 8>(a, s);
  if (spb == 4) return write_t<HD, 4>(a, s);
  if (spb == 2) return write_t<HD, 2>(a, s);
  return write_t<HD, 1>(a, s);
}

template <int HD>
cudaError_t read_d(const Q8RowsArgs& a, cudaStream_t s) {
  const long long items = q8_unit_slots(a.total, a.B, RowLanes<HD>::TR) * a.Hk * 2;
  profile_mark(kKernQ8Read, 0, s);
  q8_read_kernel<HD><<<(unsigned)((items + 7) / 8), 256, 0, s>>>(rows_params(a), items);
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
