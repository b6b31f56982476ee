// fa_tree.cu -- attention of a tree of drafted tokens over the paged bf16 key/value cache, sm_103a.
//
// The T nodes of a sequence's tree are its last T keys, and its T query rows. A node sees every key
// before them, and of them those that its row of the mask names (its ancestors and itself):
//   visible(i, j) = j < len - T  or  mask[i][j - (len - T)] != 0      (0 <= j < len)
//   O_i = sum_j exp(s_ij - L_i) v_j,  s_ij = scale <q_i, k_j>,  L_i = log sum_j exp(s_ij)
// A node that sees no key gives O = 0 and L = -inf.
//
// A warp has a query row, its lanes a piece of the head dim each; one pass over the keys with the
// running maximum and sum.
#include <float.h>

#include "fa_common.cuh"
#include "fa_launch.h"

namespace fa {

namespace {
struct TreeK {
  const __nv_bfloat16* q;
  const __nv_bfloat16* k;
  const __nv_bfloat16* v;
  const int32_t* table;
  const int32_t* lens;
  const uint8_t* mask;
  long long mask_stride;
  __nv_bfloat16* o;
  float* lse;
  int* status;
  int B, Hk, G, T, max_pages, num_pages, ps_shift;
  float scale;
};

template <int HD>
__global__ void __launch_bounds__(256) tree_kernel(const TreeK p) {
  constexpr int E = HD / 32;
  const long long row = (long long)blockIdx.x * 8 + warp_id();  // (b * H + h) * T + i
  const int lane = lane_id();
  const int H = p.Hk * p.G;
  if (row >= (long long)p.B * H * p.T) return;
  const int i = (int)(row % p.T), h = (int)(row / p.T % H), b = (int)(row / p.T / H);
  const long long cap = (long long)p.max_pages << p.ps_shift;
  const int raw = p.lens[b], len = raw < 0 ? 0 : raw > cap ? (int)cap : raw;
  bool bad = raw != len;
  float q[E], acc[E], m = -FLT_MAX / 2, l = 0.0f;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    q[e] = __bfloat162float(p.q[row * HD + lane * E + e]) * p.scale;
    acc[e] = 0.0f;
  }
  const uint8_t* mask = p.mask + b * p.mask_stride + (long long)i * p.T;
  for (int j = 0; j < len; ++j) {
    const int node = j - (len - p.T);
    if (node >= 0 && !mask[node]) continue;
    const int page = p.table[(size_t)b * p.max_pages + (j >> p.ps_shift)];
    const bool have = page >= 0 && page < p.num_pages;
    bad |= !have;
    float k[E], v[E], s = 0.0f;
    const size_t at = ((((size_t)(have ? page : 0) * p.Hk + h / p.G) << p.ps_shift) +
                       (j & ((1 << p.ps_shift) - 1))) * HD + lane * E;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      k[e] = have ? __bfloat162float(p.k[at + e]) : 0.0f;
      v[e] = have ? __bfloat162float(p.v[at + e]) : 0.0f;
      s = fmaf(q[e], k[e], s);
    }
#pragma unroll
    for (int o = 16; o > 0; o /= 2) s += __shfl_xor_sync(0xffffffffu, s, o);
    const float top = fmaxf(m, s), f = expf(m - top), w = expf(s - top);
    m = top;
    l = fmaf(l, f, w);
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = fmaf(acc[e], f, w * v[e]);
  }
#pragma unroll
  for (int e = 0; e < E; ++e)
    p.o[row * HD + lane * E + e] = __float2bfloat16(l > 0.0f ? acc[e] / l : l == 0.0f ? 0.0f : l);
  if (p.lse && lane == 0) p.lse[row] = l == 0.0f ? -INFINITY : m + logf(l);
  if (bad && p.status) atomicCAS(p.status, kStatusOk, kStatusBadInput);
}
}  // namespace

cudaError_t launch_tree(const TreeArgs& a, cudaStream_t s) {
  TreeK p;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.k = static_cast<const __nv_bfloat16*>(a.k_cache);
  p.v = static_cast<const __nv_bfloat16*>(a.v_cache);
  p.table = a.table;
  p.lens = a.lens;
  p.mask = a.mask;
  p.mask_stride = a.mask_stride;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.status = a.status;
  p.B = a.B;
  p.Hk = a.Hk;
  p.G = a.G;
  p.T = a.T;
  p.max_pages = a.max_pages;
  p.num_pages = a.num_pages;
  p.ps_shift = a.ps_shift;
  p.scale = a.scale;
  const unsigned grid = (unsigned)(((long long)a.B * a.Hk * a.G * a.T + 7) / 8);
  profile_mark(kKernTreeAttn, 0, s);
  switch (a.d) {
    case 64: tree_kernel<64><<<grid, 256, 0, s>>>(p); break;
    case 128: tree_kernel<128><<<grid, 256, 0, s>>>(p); break;
    case 256: tree_kernel<256><<<grid, 256, 0, s>>>(p); break;
    default: return cudaErrorInvalidValue;
  }
  const cudaError_t e = cudaGetLastError();
  profile_mark(kKernTreeAttn, 1, s);
  return e;
}

}  // namespace fa
