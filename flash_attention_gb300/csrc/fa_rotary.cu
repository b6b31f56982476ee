// fa_rotary.cu -- rows of queries and keys turned by their positions, and new rows appended to a
// paged bf16 cache with that rotation on the way, sm_103a.
//
// Both kernels are one: up to three segments of heads (queries and keys, or keys, values and
// queries), each with its source rows and its destination, rows of a tensor or slots of pages. They
// move 4 bytes an element and are bound by HBM as long as what surrounds the bytes is cheap. What
// is not cheap is a row's sines and cosines, about 30 instructions for each pair, and what leads
// to its place (sequence, length, table). Neither depends on the head: a thread has 16 elements of
// a row, two runs of 8 whose pairs lie inside them (the first and second half's, or 4 + 4
// neighbours), finds 8 sines and cosines and its place once, and walks over the heads of a group.
#include "fa_common.cuh"
#include "fa_launch.h"
#include "fa_rotary.cuh"

namespace fa {

namespace {
// (128: two sequences of 4096 rows, 40 heads of 128, 28.1 us; 256: 28.4, and 4.7 for 3.7 in small calls)
constexpr int kThreads = 128, kKeepThreads = 256;
constexpr int kAhead = 4;  // heads whose elements are on their way at once

struct RowsK {
  RowSeg seg[3];
  Rope rope;
  const int32_t* cu;     // packed batch: [B + 1]; nullptr: n rows for each sequence
  const int32_t* table;  // paged destinations: [B, max_pages] and [B]
  const int32_t* lens;
  int* status;
  int B, n, rows;        // rows: B * n, or of the packed batch
  int Hk, max_pages, num_pages, ps_shift;
  int group;             // heads of a CTA
};

// The sequence that row `row` of a packed batch belongs to: the last b with cu[b] <= row (-1 where
// there is none).
__device__ __forceinline__ int row_owner(const int32_t* cu, int B, int row) {
  int lo = -1, hi = B;  // cu[lo] <= row (lo = -1: none known), the answer is below hi
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= row) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t turned(float x1, float x2, float y1, float y2, float c0,
                                           float s0, float c1, float s1, uint32_t& second) {
  second = pack_bf16(fmaf(x1, s0, x2 * c0), fmaf(y1, s1, y2 * c1));
  return pack_bf16(fmaf(x1, c0, -(x2 * s0)), fmaf(y1, c1, -(y2 * s1)));
}

// Two runs of 8 elements, turned: pairs (a[e], b[e]).
__device__ __forceinline__ void turn_halves(uint4& a, uint4& b, const float (&c)[8],
                                            const float (&s)[8]) {
  uint32_t* pa = &a.x;
  uint32_t* pb = &b.x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t second;
    const uint32_t first = turned(bf16_lo(pa[e]), bf16_lo(pb[e]), bf16_hi(pa[e]), bf16_hi(pb[e]),
                                  c[2 * e], s[2 * e], c[2 * e + 1], s[2 * e + 1], second);
    pa[e] = first;
    pb[e] = second;
  }
}
// A run of 8 elements, its neighbours turned.
__device__ __forceinline__ void turn_pairs(uint4& a, const float* c, const float* s) {
  uint32_t* pa = &a.x;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float x1 = bf16_lo(pa[e]), x2 = bf16_hi(pa[e]);
    pa[e] = pack_bf16(fmaf(x1, c[e], -(x2 * s[e])), fmaf(x1, s[e], x2 * c[e]));
  }
}

template <int HD, bool PAGED>
__global__ void __launch_bounds__(kThreads) rows_kernel(const __grid_constant__ RowsK p) {
  constexpr int TPR = HD / 16;  // threads of a row
  const int t = threadIdx.x % TPR;
  const long long at = (long long)blockIdx.x * (kThreads / TPR) + threadIdx.x / TPR;
  // the segment and its heads
  int g = blockIdx.y, which = 0;
  while (g >= p.seg[which].groups) g -= p.seg[which++].groups;
  const RowSeg& seg = p.seg[which];
  const int h0 = g * p.group, h1 = min(h0 + p.group, seg.heads);

  if (p.cu && blockIdx.y == 0 && blockIdx.x == 0) {  // offsets out of range are reported here
    bool bad = threadIdx.x == 0 && (p.cu[0] != 0 || p.cu[p.B] > p.rows);
    for (int b = threadIdx.x; b < p.B; b += kThreads) bad |= p.cu[b + 1] < p.cu[b];
    if (bad && p.status) atomicCAS(p.status, kStatusOk, kStatusBadInput);
  }
  if (PAGED && blockIdx.y == 0 && blockIdx.x == 0) {
    bool bad = false;
    for (int b = threadIdx.x; b < p.B; b += kThreads)
      bad |= p.lens[b] < 0 || p.lens[b] > (long long)p.max_pages << p.ps_shift;
    if (bad && p.status) atomicCAS(p.status, kStatusOk, kStatusBadInput);
  }
  if (at >= p.rows) return;
  const int row = (int)at;
  // row i of the n rows of sequence b
  int b, i, n = p.n;
  if (p.cu) {
    b = row_owner(p.cu, p.B, row);
    if (b < 0 || row >= p.cu[b + 1]) return;  // behind the last sequence
    i = row - p.cu[b];
    n = p.cu[b + 1] - p.cu[b];
  } else {
    b = row / p.n;
    i = row - b * p.n;
  }
  int place = i + p.rope.offset;  // its position (the host has checked that it fits)
  bool store = true;
  size_t slot = 0;                // its page's first row, and the slot in the page
  if constexpr (PAGED) {
    const int len = p.lens[b];
    place = (int)((unsigned)len - (unsigned)n + (unsigned)i);
    if (seg.paged) {
      store = len >= 0 && len <= (long long)p.max_pages << p.ps_shift && place >= 0;
      if (store) {
        const int page = p.table[(size_t)b * p.max_pages + (place >> p.ps_shift)];
        store = page >= 0 && page < p.num_pages;
        if (!store && p.status) atomicCAS(p.status, kStatusOk, kStatusBadInput);
        slot = ((size_t)(unsigned)page * p.Hk << p.ps_shift) + (place & ((1 << p.ps_shift) - 1));
      }
      if (!store) return;
    }
  }
  // this thread's elements: 8 from c0 and 8 from c1 on
  const Rope& rope = p.rope;
  const bool turn = seg.turn;
  const int half = turn ? rope.half : 0;
  int c0, c1;
  bool turn0, turn1;
  if (turn && !rope.inter) {
    turn0 = turn1 = t < half / 8;
    const int u = t - half / 8, rest = HD / 2 - half;
    c0 = turn0 ? t * 8 : 2 * half + u * 8;
    c1 = turn0 ? half + t * 8 : 2 * half + rest + u * 8;
  } else {
    c0 = t * 8;
    c1 = HD / 2 + t * 8;
    turn0 = c0 < 2 * half;
    turn1 = c1 < 2 * half;
  }
  const __nv_bfloat16* src =
      seg.src + (p.cu ? (long long)row * seg.ss[2] : b * seg.ss[0] + i * seg.ss[2]);
  __nv_bfloat16* dst;
  long long head_step = seg.ds[1];
  if (PAGED && seg.paged) {
    dst = seg.dst + slot * HD;
    head_step = (long long)HD << p.ps_shift;
  } else {
    dst = seg.dst + (p.cu ? (long long)row * seg.ds[2] : b * seg.ds[0] + i * seg.ds[2]);
  }
  uint4 x[kAhead], y[kAhead];
  auto load = [&](int h) {
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (h + e < h1) {
        const __nv_bfloat16* s = src + (h + e) * seg.ss[1];
        x[e] = *reinterpret_cast<const uint4*>(s + c0);
        y[e] = *reinterpret_cast<const uint4*>(s + c1);
      }
    }
  };
  load(h0);
  float c[8], s[8];
  if (turn0) {
    if (rope.pos) place = rope.pos[p.cu ? (long long)row : b * rope.pos_stride + i];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      // (pairs of the second run of neighbours that does not turn: any frequency)
      const int f = rope.inter ? (e < 4 ? c0 / 2 + e : turn1 ? c1 / 2 + e - 4 : 0) : t * 8 + e;
      bool fine;
      const uint64_t turns = turns_of(rope.inv_freq[f], fine);
      turn_at(place, turns, c[e], s[e]);
      c[e] = fine ? c[e] * rope.scale : __int_as_float(0x7fc00000);
      s[e] = fine ? s[e] * rope.scale * rope.sign : __int_as_float(0x7fc00000);
    }
  }
  for (int h = h0; h < h1; h += kAhead) {
#pragma unroll
    for (int e = 0; e < kAhead; ++e) {
      if (h + e >= h1) break;
      if (turn0) {
        if (rope.inter) {
          turn_pairs(x[e], c, s);
          if (turn1) turn_pairs(y[e], c + 4, s + 4);
        } else {
          turn_halves(x[e], y[e], c, s);
        }
      }
      __nv_bfloat16* d = dst + (h + e) * head_step;
      *reinterpret_cast<uint4*>(d + c0) = x[e];
      *reinterpret_cast<uint4*>(d + c1) = y[e];
    }
    load(h + kAhead);
  }
}

template <int HD>
cudaError_t launch_rows_d(const RowsArgs& a, cudaStream_t s) {
  RowsK p;
  int groups = 0;
  // Heads of a CTA: 8, as sines, cosines and places serve them all (two sequences of 4096 rows, 40 heads
  // of 128: 28.4 us, 30.8 with 4, with 16 and 32 as with 8; prompts of 8192 rows 205 and 226 us), few
  // where the rows alone do not fill the GPU.
  const long long row_ctas = (a.rows + kThreads / (HD / 16) - 1) / (kThreads / (HD / 16));
  int heads = 0;
  for (int i = 0; i < 3; ++i) heads += a.seg[i].heads;
  p.group = 8;
  while (p.group > 1 && row_ctas * ((heads + p.group - 1) / p.group) < 2 * 152) p.group /= 2;
  for (int i = 0; i < 3; ++i) {
    p.seg[i] = a.seg[i];
    p.seg[i].groups = (a.seg[i].heads + p.group - 1) / p.group;
    groups += p.seg[i].groups;
  }
  p.rope = a.rope;
  p.cu = a.cu;
  p.table = a.table;
  p.lens = a.lens;
  p.status = a.status;
  p.B = a.B;
  p.n = a.n;
  p.rows = a.rows;
  p.Hk = a.Hk;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.ps_shift = a.ps_shift;
  const dim3 grid((unsigned)row_ctas, (unsigned)groups);
  const int kernel = a.table ? kKernPagedAppend : kKernRotary;
  profile_mark(kernel, 0, s);
  if (a.table)
    rows_kernel<HD, true><<<grid, kThreads, 0, s>>>(p);
  else
    rows_kernel<HD, false><<<grid, kThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  profile_mark(kernel, 1, s);
  return e;
}

// The rows that `keep` names of a sequence's last T, moved to the front of the T. The row that goes
// to place i comes from place keep[i] >= i (keep ascends), so rows may be moved in order: a thread
// has 8 columns of K or V of one head and moves them for all rows, 8 rows at a time; no thread reads
// what another writes. The next 8 rows are asked for before the last 8 are written: they lie behind all
// places that these go to, and may lie where later ones go. (A few KB for a sequence: latency is all
// that counts.)
struct KeepK {
  __nv_bfloat16* cache[2];
  const int32_t* table;
  const int32_t* lens;
  const int32_t* keep;    // [B, M]
  const int32_t* counts;  // [B]
  int32_t* new_lens;      // [B]
  int* status;
  int Hk, d8, max_pages, num_pages, ps_shift, T, M;
};

__global__ void __launch_bounds__(kKeepThreads) keep_kernel(const KeepK p) {
  __shared__ long long src_s[kTreeMax], dst_s[kTreeMax];  // slots (-1: the row stays)
  const int b = blockIdx.x;
  const long long cap = (long long)p.max_pages << p.ps_shift;
  const int len = p.lens[b], count = p.counts[b];
  bool good = len >= 0 && len <= cap && count >= 0 && count <= p.M;
  bool bad = !good;
  const int base = good ? len - p.T : 0;
  for (int i = threadIdx.x; good && i < count; i += kKeepThreads) {
    const int k = p.keep[(size_t)b * p.M + i];
    const int before = i > 0 ? p.keep[(size_t)b * p.M + i - 1] : -1;
    long long src = -1, dst = -1;
    if (k <= before || k >= p.T || (k != i && base + i < 0)) {
      good = false;
    } else if (k != i) {
      auto slot = [&](int pos) -> long long {
        const int page = p.table[(size_t)b * p.max_pages + (pos >> p.ps_shift)];
        if (page < 0 || page >= p.num_pages) return -1;
        return ((long long)page * p.Hk << p.ps_shift) + (pos & ((1 << p.ps_shift) - 1));
      };
      src = slot(base + k);
      dst = slot(base + i);
      if (src < 0 || dst < 0) {
        bad = true;
        src = -1;
      }
    }
    src_s[i] = src;
    dst_s[i] = dst;
  }
  bad |= !good;
  good = __syncthreads_and(good);
  if (bad && p.status) atomicCAS(p.status, kStatusOk, kStatusBadInput);
  if (blockIdx.y == 0 && threadIdx.x == 0)
    p.new_lens[b] = good ? max(0, base + count) : len;
  const int col = blockIdx.y * kKeepThreads + threadIdx.x;
  if (!good || col >= 2 * p.Hk * p.d8) return;
  const int which = col / (p.Hk * p.d8), h = col / p.d8 % p.Hk, c = col % p.d8;
  uint4* cache = reinterpret_cast<uint4*>(p.cache[which]);
  auto place = [&](long long slot) { return (slot + ((long long)h << p.ps_shift)) * p.d8 + c; };
  auto load = [&](uint4 (&x)[8], int i0) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i0 + e < count && src_s[i0 + e] >= 0) x[e] = cache[place(src_s[i0 + e])];
  };
  auto store = [&](const uint4 (&x)[8], int i0) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (i0 + e < count && src_s[i0 + e] >= 0) cache[place(dst_s[i0 + e])] = x[e];
  };
  uint4 x[8], y[8];
  load(x, 0);
#pragma unroll 1
  for (int i0 = 0; i0 < count; i0 += 16) {
    load(y, i0 + 8);
    store(x, i0);
    load(x, i0 + 16);
    store(y, i0 + 8);
  }
}
}  // namespace

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t s) {
  switch (a.d) {
    case 64: return launch_rows_d<64>(a, s);
    case 128: return launch_rows_d<128>(a, s);
    case 256: return launch_rows_d<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_keep(const KeepArgs& a, cudaStream_t s) {
  KeepK p;
  p.cache[0] = static_cast<__nv_bfloat16*>(a.k_cache);
  p.cache[1] = static_cast<__nv_bfloat16*>(a.v_cache);
  p.table = a.table;
  p.lens = a.lens;
  p.keep = a.keep;
  p.counts = a.counts;
  p.new_lens = a.new_lens;
  p.status = a.status;
  p.Hk = a.Hk;
  p.d8 = a.d / 8;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.ps_shift = a.ps_shift;
  p.T = a.T;
  p.M = a.M;
  const int cols = 2 * p.Hk * p.d8;
  profile_mark(kKernPagedKeep, 0, s);
  const dim3 grid((unsigned)a.B, (unsigned)((cols + kKeepThreads - 1) / kKeepThreads));
  keep_kernel<<<grid, kKeepThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  profile_mark(kKernPagedKeep, 1, s);
  return e;
}

}  // namespace fa
