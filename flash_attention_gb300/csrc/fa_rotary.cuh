// fa_rotary.cuh -- rotary positions: the angle of a position, and the turn of a row's elements.
//
// Pair i of the first rotary_dim elements of a row, (x1, x2), at position p turns by the angle
// a = p * inv_freq[i]:  s (x1 cos a - x2 sin a, x1 sin a + x2 cos a). Pairs are the elements i and
// i + rotary_dim / 2, or 2 i and 2 i + 1 (interleaved).
//
// The angle is a number of turns of which only the fraction counts, so it is kept as one: inv_freq
// becomes turns per position in units of 2^-64, and p times that, in 64-bit integers that wrap, is
// the fraction of a turn, at most p + 1 units off for |inv_freq| <= 1: 2^-32 of a turn at the last
// 32-bit position. (An angle held in 32 bits is 2^-5 of a radian off at position 10^6.) Its upper 32
// bits become radians in f32, whatever the position: below 2^-24.3 of a turn off by their rounding, the
// constant's and the product's, 2^-21.6 of a radian. The hardware's sine and cosine of them are good to
// 2^-21 within pi. Together that is 2^-12 of what a bf16 is rounded by.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fa_launch.h"  // Rope

namespace fa {

// Turns per position, in units of 2^-64, of a frequency in radians per position; `fine` becomes
// false for one that is not finite. (In integers: the units for 64-bit floats are two a clock on
// an SM.) f = m * 2^(e - 1075), and m * 2^66 / (2 pi) * 2^(e - 1077) are its turns.
__device__ __forceinline__ uint64_t turns_of(double f, bool& fine) {
  constexpr uint64_t kTurn = 0xa2f9836e4e441529ull;  // 2^66 / (2 pi), rounded down
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)(bits >> 52) & 0x7ff, down = 1024 - e;
  const uint64_t m = (bits << 11) | (1ull << 63);  // 53 bits at the top
  const uint64_t p = __umul64hi(m, kTurn);
  uint64_t t = down >= 64 ? 0ull : down >= 0 ? p >> down : down > -64 ? p << -down : 0ull;
  fine = e != 0x7ff;
  return (bits >> 63) ? 0ull - t : t;
}

// Cosine and sine of `pos` times the frequency `turns`.
__device__ __forceinline__ void turn_at(int pos, uint64_t turns, float& c, float& s) {
  const uint32_t part = (uint32_t)(((uint64_t)(int64_t)pos * turns) >> 32);
  const float a = (float)(int32_t)part * 1.4629180792671596e-9f;  // 2 pi / 2^32
  c = __cosf(a);
  s = __sinf(a);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

}  // namespace fa
