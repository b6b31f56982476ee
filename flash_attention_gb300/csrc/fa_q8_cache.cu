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

// x / s for 8 values of a row as codes. inv: 1 / s where s is a power of two (then exact), else 0.
__device__ __forceinline__ uint2 quantise8(const uint4& x, float s, float inv, bool odd) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  float y[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = bf16x2_f32(w[e]);
    y[2 * e] = inv != 0.0f ? f.x * inv : f.x / s;
    y[2 * e + 1] = inv != 0.0f ? f.y * inv : f.y / s;
  }
  if (odd) {  // a value that is not finite: NaN, where the conversion would saturate infinities
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (!isfinite(y[e])) y[e] = NAN;
  }
  return make_uint2(e4m3x4_from_f32(y[0], y[1], y[2], y[3]),
                    e4m3x4_from_f32(y[4], y[5], y[6], y[7]));
}

// SPB: steps of a scale block inside a warp (1: a block of at most one step). `wpb` warps of
// the CTA share a unit of max(rows of a warp, scale block) positions.
template <int HD, int SPB>
__global__ void __launch_bounds__(1024)
    q8_write_kernel(const Q8RowsK p, long long items, int wpb) {
  using RL = RowLanes<HD>;
  __shared__ uint32_t warp_max[32];
  const int warp = warp_id(), lane = lane_id();
  const int sb = 1 << p.sb_shift;
  const int unit = RL::TR * wpb;
  // the items of a CTA: K and V of a head, then the next head, then the next unit
  const long long item = (long long)blockIdx.x * (blockDim.x / 32 / wpb) + warp / wpb;
  const int which = (int)(item & 1);
  const int head = (int)((item >> 1) % p.Hk);
  const long long slot = (item >> 1) / p.Hk;
  bool live = item < items, bad = false;
  int b = 0, start = 0, n = 0, len = 0, first = 0;
  long long p0 = 0;
  if (live) {
    auto offset = [&](int i) { return p.cu ? (long long)p.cu[i] : (long long)i * p.new_len; };
    b = q8_slot_owner(slot, p.B, unit, lane, offset);
    bad |= seq_rows(p, b, start, n);
    len = p.lens[b];
    if (len < 0 || len > (long long)p.max_pages << p.ps_shift) {  // no place is the right one
      bad = true;
      live = false;
    }
    first = len - n;
    const long long u = slot - (offset(b) / unit + 2ll * b);
    p0 = (long long)(max(first, 0) / unit + u) * unit;  // first position of this unit
    live = live && u >= 0 && p0 < len && n > 0;
  }
  p0 += (warp % wpb) * RL::TR;
  const int lo = max(first, 0);  // new rows are the positions lo .. len - 1
  const int r = lane / RL::LPR, col = lane % RL::LPR * 8;
  const __nv_bfloat16* src = p.rows[which] + head * p.st_h[which] + col +
                             (p.cu ? (long long)start * p.st_r[which] : b * p.st_b[which]);
  uint4 x[kSteps];
  int pg[kSteps];
  uint32_t amax[kSteps / SPB];
  float old[kSteps / SPB];
  bool odd = false;
#pragma unroll
  for (int t = 0; t < kSteps; ++t) {
    const long long pos = p0 + t * RL::RPS + r;
    x[t] = make_uint4(0u, 0u, 0u, 0u);
    pg[t] = -1;
    if (live && pos >= lo && pos < len)
      x[t] = __ldg(reinterpret_cast<const uint4*>(src + (pos - first) * p.st_r[which]));
    // earlier rows of a block that gets a new one are looked at too
    if (live && pos < len && (pos | (sb - 1)) >= lo) pg[t] = page_of(p, b, (int)pos, bad);
  }
#pragma unroll
  for (int g = 0; g < kSteps / SPB; ++g) {
    uint32_t m2 = 0;
    old[g] = 0.0f;
#pragma unroll
    for (int t = g * SPB; t < (g + 1) * SPB; ++t) {
      const uint32_t w[4] = {x[t].x, x[t].y, x[t].z, x[t].w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t a = w[e] & 0x7fff7fffu;
        const uint32_t inf = __vcmpgeu2(a, 0x7f807f80u);
        odd |= inf != 0;
        m2 = __vmaxu2(m2, a & ~inf);
      }
      // the block's scale, where it holds earlier tokens: those of the one block with `first`
      // inside, read before any warp writes it
      const long long pos = p0 + t * RL::RPS + r;
      if (pg[t] >= 0 && (pos & ~(long long)(sb - 1)) < first)
        old[g] = p.scales[which][(((size_t)pg[t] * p.Hk + head) << (p.ps_shift - p.sb_shift)) +
                                 ((pos & ((1 << p.ps_shift) - 1)) >> p.sb_shift)];
    }
    amax[g] = max(m2 & 0xffffu, m2 >> 16);
    const int lanes = min(32, RL::LPR << p.sb_shift);  // lanes of a block
    for (int o = lanes / 2; o > 0; o /= 2)
      amax[g] = max(amax[g], __shfl_xor_sync(0xffffffffu, amax[g], o));
  }
  if (wpb > 1) {  // (then SPB = kSteps: one block for each unit)
    if (lane == 0) warp_max[warp] = amax[0];
    __syncthreads();
    for (int w = warp / wpb * wpb; w < (warp / wpb + 1) * wpb; ++w)
      amax[0] = max(amax[0], warp_max[w]);
  }
  odd = __any_sync(0xffffffffu, odd);
#pragma unroll
  for (int g = 0; g < kSteps / SPB; ++g) {
    // lanes of rows past the end hold no old scale; the block's first rows do
    float was = old[g];
    const int lanes = min(32, RL::LPR << p.sb_shift);
    for (int o = lanes / 2; o > 0; o /= 2)
      was = fmaxf(was, __shfl_xor_sync(0xffffffffu, was, o));
    const float s = fmaxf(exp2i(scale_exp(amax[g])), was);
    const bool pow2 = (__float_as_uint(s) & 0x7fffffu) == 0;
    const float inv = pow2 ? 1.0f / s : 0.0f;
    const bool grew = was > 0.0f && s > was;
    const float ratio = grew ? was / s : 1.0f;
#pragma unroll
    for (int t = g * SPB; t < (g + 1) * SPB; ++t) {
      if (pg[t] < 0) continue;
      const long long pos = p0 + t * RL::RPS + r;
      const int slot_in = (int)pos & ((1 << p.ps_shift) - 1);
      const size_t at = (size_t)pg[t] * p.Hk + head;
      uint2* dst = reinterpret_cast<uint2*>(p.codes[which] +
                                            ((at << p.ps_shift) + slot_in) * HD + col);
      if (pos >= lo) {
        *dst = quantise8(x[t], s, inv, odd);
        // the block's scale, by its first new row
        if (col == 0 && ((slot_in & (sb - 1)) == 0 || pos == lo))
          p.scales[which][(at << (p.ps_shift - p.sb_shift)) + (slot_in >> p.sb_shift)] = s;
      } else if (grew) {
        const uint2 c = *dst;
        const float2 f0 = f32_from_e4m3x2(c.x), f1 = f32_from_e4m3x2(c.x >> 16);
        const float2 f2 = f32_from_e4m3x2(c.y), f3 = f32_from_e4m3x2(c.y >> 16);
        *dst = make_uint2(e4m3x4_from_f32(f0.x * ratio, f0.y * ratio, f1.x * ratio, f1.y * ratio),
                          e4m3x4_from_f32(f2.x * ratio, f2.y * ratio, f3.x * ratio, f3.y * ratio));
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
  const long long items = q8_unit_slots(total, a.B, RL::TR * wpb) * a.Hk * 2;
  const long long per = warps / wpb;
  profile_mark(kKernQ8Write, 0, s);
  q8_write_kernel<HD, SPB><<<(unsigned)((items + per - 1) / per), warps * 32, 0, s>>>(
      rows_params(a), items, wpb);
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
