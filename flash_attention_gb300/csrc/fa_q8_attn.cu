// fa_q8_attn.cu -- attention of a few new queries per sequence over the 8-bit paged key/value
// cache, sm_103a.
//
// Key j of sequence b is slot j % page_size of page table[b][j / page_size]; its key is
// k_scale * k codes, its value v_scale * v codes, and query i of the q_len new positions sees key
// j iff j < len (and, with the causal rule, j <= len - q_len + i). O = softmax(scale q k^T) v and
// L = log sum exp; a query that sees no key gives O = 0 and L = -inf.
//
// The plainest form: one CTA for each query row, a warp for each key in turn (a lane holds
// d / 32 columns), an online softmax in each warp, the warps joined in shared memory.
#include <float.h>

#include "fa_common.cuh"
#include "fa_launch.h"
#include "fa_q8.cuh"

namespace fa {

namespace {
constexpr int kWarps = 8;

template <int HD>
__global__ void __launch_bounds__(kWarps * 32) q8_attn_kernel(const Q8AttnArgs p) {
  constexpr int CPL = HD / 32;  // columns of a lane
  __shared__ float acc_s[kWarps][HD], m_s[kWarps], l_s[kWarps];
  const int warp = warp_id(), lane = lane_id();
  const long long row = blockIdx.x;  // (b * H + h) * lq + i
  const int i = (int)(row % p.lq), h = (int)(row / p.lq % p.H), b = (int)(row / p.lq / p.H);
  const int kh = h / p.G;
  const int ps = 1 << p.ps_shift;
  const long long cap = (long long)p.max_pages * ps;
  const int raw = p.lens[b];
  const int len = raw < 0 ? 0 : raw > cap ? (int)cap : raw;
  bool bad = raw != len;
  const int seen = p.causal ? len - p.lq + i + 1 : len;  // keys 0 .. seen - 1
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(p.q) + row * HD + lane * CPL;
  float qr[CPL], acc[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    qr[c] = __bfloat162float(q[c]) * p.scale;
    acc[c] = 0.0f;
  }
  float m = -FLT_MAX / 2, l = 0.0f;
  for (int j = warp; j < seen; j += kWarps) {
    const int pg = p.table[(size_t)b * p.max_pages + (j >> p.ps_shift)];
    if (pg < 0 || pg >= p.num_pages) bad = true;
    float s = 0.0f, vs = 0.0f, vv[CPL] = {};
    if (pg >= 0 && pg < p.num_pages) {
      const size_t at = (size_t)pg * p.Hk + kh;
      const size_t blk = (at << (p.ps_shift - p.sb_shift)) + ((j & (ps - 1)) >> p.sb_shift);
      const size_t off = ((at << p.ps_shift) + (j & (ps - 1))) * HD + lane * CPL;
#pragma unroll
      for (int c = 0; c < CPL; c += 2) {
        const float2 kc = f32_from_e4m3x2(*reinterpret_cast<const uint16_t*>(p.k + off + c));
        const float2 vc = f32_from_e4m3x2(*reinterpret_cast<const uint16_t*>(p.v + off + c));
        s += qr[c] * kc.x + qr[c + 1] * kc.y;
        vv[c] = vc.x;
        vv[c + 1] = vc.y;
      }
      for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
      s *= p.k_scale[blk];
      vs = p.v_scale[blk];
    }
    const float mn = fmaxf(m, s);
    const float f = expf(m - mn), w = expf(s - mn);
    l = l * f + w;
#pragma unroll
    for (int c = 0; c < CPL; ++c) acc[c] = acc[c] * f + w * vs * vv[c];
    m = mn;
  }
#pragma unroll
  for (int c = 0; c < CPL; ++c) acc_s[warp][lane * CPL + c] = acc[c];
  if (lane == 0) {
    m_s[warp] = m;
    l_s[warp] = l;
  }
  __syncthreads();
  float mt = -FLT_MAX / 2, lt = 0.0f;
  for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, m_s[w]);
  for (int w = 0; w < kWarps; ++w) lt += l_s[w] * expf(m_s[w] - mt);
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + row * HD;
  if (threadIdx.x < HD) {
    float a = 0.0f;
    for (int w = 0; w < kWarps; ++w) a += acc_s[w][threadIdx.x] * expf(m_s[w] - mt);
    o[threadIdx.x] = __float2bfloat16(seen > 0 ? a / lt : 0.0f);
  }
  if (threadIdx.x == 0 && p.lse) p.lse[row] = seen > 0 ? mt + logf(lt) : -INFINITY;
  if (bad && lane == 0 && p.status) atomicCAS(p.status, kStatusOk, kStatusBadInput);
}

template <int HD>
cudaError_t attn_t(const Q8AttnArgs& a, cudaStream_t s) {
  profile_mark(kKernQ8Attn, 0, s);
  q8_attn_kernel<HD><<<(unsigned)((long long)a.B * a.H * a.lq), kWarps * 32, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  profile_mark(kKernQ8Attn, 1, s);
  return e;
}
}  // namespace

cudaError_t launch_q8_attn(const Q8AttnArgs& a, cudaStream_t s) {
  switch (a.d) {
    case 64: return attn_t<64>(a, s);
    case 128: return attn_t<128>(a, s);
    case 256: return attn_t<256>(a, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fa
