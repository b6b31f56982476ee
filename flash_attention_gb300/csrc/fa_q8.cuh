// fa_q8.cuh -- what the kernels of the 8-bit key/value cache share: e4m3 conversions and the
// lookup of a packed batch's sequences.
//
// The cache holds e4m3 codes [num_pages, Hk, page_size, d] and one f32 scale for each block of
// scale_block slots of a page and each head, [num_pages, Hk, page_size / scale_block]; a code c
// with the scale s stands for c * s.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace fa {

// Exponent of the smallest scale that the writer uses (an all-zero block has it). The attention
// reads smaller value scales as this one, so that log2 of a scale is always finite.
constexpr int kQ8MinExp = -100;
// The largest scale that the attention admits, 2^100, as its f32 bits: those of negative values and
// of NaN are larger.
constexpr uint32_t kQ8MaxScale = 0x71800000u;

// Two floats -> two e4m3 codes (round to nearest even, saturating; NaN -> 0x7F): `lo` in bits 0-7.
__device__ __forceinline__ uint32_t e4m3x2_from_f32(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Four floats -> four codes in one word.
__device__ __forceinline__ uint32_t e4m3x4_from_f32(float a, float b, float c, float d) {
  return e4m3x2_from_f32(a, b) | (e4m3x2_from_f32(c, d) << 16);
}
// Two codes -> two floats (exact: every e4m3 value is an f16 value).
__device__ __forceinline__ float2 f32_from_e4m3x2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

// A batch's rows cut into units of `unit` positions, aligned in each sequence, without a pass
// over the lengths: sequence b owns the unit slots cu[b] / unit + 2 b and on, and n rows touch
// at most n / unit + 2 units (the first one may begin, and the last one end, inside a unit).
__host__ __device__ inline long long q8_unit_slots(long long total, int batch, int unit) {
  return total / unit + 2ll * batch;
}

// The sequence that owns `slot` (warp-wide): the last b in [0, batch) with
// start(b) / unit + 2 b <= slot, found 32 candidates at a time. `start` reads the offset of a
// sequence's first row; whatever it returns, the answer lies in [0, batch).
template <class F>
__device__ __forceinline__ int q8_slot_owner(long long slot, int batch, int unit, int lane,
                                             F start) {
  int lo = 0, n = batch;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int b = lo + lane * step;
    const bool below = lane * step < n && (lane == 0 || start(b) / unit + 2ll * b <= slot);
    const int last = __popc(__ballot_sync(0xffffffffu, below)) - 1;  // lane 0 always counts
    n = min(step, n - last * step);
    lo += last * step;
    if (n < 1) n = 1;
  }
  return min(lo, batch - 1);
}

}  // namespace fa
