// fa_wait.cuh -- bounded waits on mbarriers for kernels whose warps wait most of the time: suspended
// polls, out of line.
#pragma once

#include "fa_common.cuh"

namespace fa {
namespace {

// A first poll in line (suspended for as long as the hardware likes);
// what follows is out of line, with polls suspended for up to 20 us. (Most warps wait most of the
// time; short polls in line cost issue and the SM's instruction cache, which the softmax needs.)
// Under a limit below 100 us, which exists to make waits run out, those polls are not suspended,
// and a wait that always lasts a while (SUSPEND false) begins with one that is not, so that it runs
// out there (elsewhere that costs 2 %).
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

}  // namespace
}  // namespace fa
