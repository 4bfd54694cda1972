// Attention of a few new tokens per sequence over the 4-bit key/value cache.
//
// Per query row: S_j = scale * sum_e s_K(j,e) sum_{i in group e} q_i n_K(j,i),
// P = softmax over the keys j that the row may see, O = sum_j P_j s_V n_V.
// The codes are used as they stand, never rounded to 16 bits.
//
// One CTA per query row, its warps taking the keys in turn with a running
// maximum and sum each, joined at the end.
#include <cuda_runtime.h>

#include "fa.h"
#include "fa_kernels.h"
#include "fa_kv4.cuh"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 128;

template <bool BF16, int D, bool O32>
__global__ void __launch_bounds__(kThreads) fa_kv4_fwd_kernel(const Kv4FwdParams p) {
  constexpr int W = D / 32, NW = kThreads / 32;
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32;
  const long long row = blockIdx.x;
  const int t = (int)(row % p.T), head = (int)(row / p.T % p.H), b = (int)(row / p.T / p.H);
  const int h = head / (p.H / p.c.Hkv);
  const int n = kv4_count(p.c, b, p.T);
  const long long start = p.c.start[b];
  long long keys = t >= n ? 0 : p.causal ? start + t + 1 : start + n;
  // lane owns elements lane*W .. lane*W + W - 1, all in one group
  float q[W], o[W], m = -INFINITY, l = 0.f;
  const uint16_t* qr = static_cast<const uint16_t*>(p.q) + row * D + lane * W;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    q[i] = kv4_scale<BF16>(qr[i]) * p.scale_log2;
    o[i] = 0.f;
  }
  for (long long j = warp; j < keys; j += NW) {
    const uint8_t* blk = kv4_block_of(p.c, b, h, j, kv4_block_bytes(D));
    if (blk == nullptr) continue;
    const int key = (int)j & 15, half = key >> 3, e0 = lane * W, grp = e0 / 32;
    const uint16_t* sc = reinterpret_cast<const uint16_t*>(blk + 16 * D) + key * 2 * W + grp;
    const uint32_t kw = reinterpret_cast<const uint32_t*>(blk)[((half * 8 + (key & 7)) * 4 + e0 % 32 / 8) * W + grp];
    const int r = e0 / (D / 8), w = e0 % (D / 8) / 4;
    const uint32_t vw =
        reinterpret_cast<const uint32_t*>(blk + 8 * D)[((half * 8 + r) * 4 + ((key & 7) >> 1)) * W + w];
    const uint32_t kh = (kw >> (e0 % 8 / 4 * 16)) & 0xffffu, vh = (vw >> ((key & 1) * 16)) & 0xffffu;
    const uint32_t kn = ((kh >> 2) | (kh << 14)) & 0xffffu, vn = ((vh >> 2) | (vh << 14)) & 0xffffu;
    const float sk = kv4_scale<BF16>(sc[0]), sv = kv4_scale<BF16>(sc[W]);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) s = fmaf(q[i], (float)((int)((kn >> (4 * (e0 % 4 + i))) & 15u) - 8), s);
    s *= sk;
#pragma unroll
    for (int d = 16; d; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    const float mn = fmaxf(m, s), f = m == -INFINITY ? 0.f : exp2f(m - mn), pj = exp2f(s - mn);
    l = l * f + pj;
    m = mn;
#pragma unroll
    for (int i = 0; i < W; ++i)
      o[i] = o[i] * f + pj * (sv * (float)((int)((vn >> (4 * (e0 % 4 + i))) & 15u) - 8));
  }
  __shared__ float sm[NW], sl[NW], so[NW][D];
  if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
  for (int i = 0; i < W; ++i) so[warp][lane * W + i] = o[i];
  __syncthreads();
  if (threadIdx.x < D) {
    float mm = -INFINITY, ll = 0.f, oo = 0.f;
    for (int k = 0; k < NW; ++k) mm = fmaxf(mm, sm[k]);
    for (int k = 0; k < NW; ++k) {
      const float f = sm[k] == -INFINITY ? 0.f : exp2f(sm[k] - mm);
      ll += f * sl[k];
      oo += f * so[k][threadIdx.x];
    }
    oo = ll == 0.f ? 0.f : oo / ll;
    const long long at = row * D + threadIdx.x;
    if constexpr (O32)
      static_cast<float*>(p.o)[at] = oo;
    else if constexpr (BF16)
      static_cast<__nv_bfloat16*>(p.o)[at] = __float2bfloat16_rn(oo);
    else
      static_cast<__half*>(p.o)[at] = __float2half_rn(oo);
    if (threadIdx.x == 0) p.lse[row] = (mm + log2f(ll)) * 0.69314718055994531f;
  }
}

}  // namespace

cudaError_t launch_kv4_fwd(bool bf16, bool o32, int d, const Kv4FwdParams& p, cudaStream_t st) {
  const dim3 grid((unsigned)((long long)p.B * p.H * p.T));
#define FA_KV4(BB, DD) \
  (o32 ? launch_chained(fa_kv4_fwd_kernel<BB, DD, true>, grid, dim3(kThreads), 0, st, p) \
       : launch_chained(fa_kv4_fwd_kernel<BB, DD, false>, grid, dim3(kThreads), 0, st, p))
  if (bf16) return d == 64 ? FA_KV4(true, 64) : FA_KV4(true, 128);
  return d == 64 ? FA_KV4(false, 64) : FA_KV4(false, 128);
#undef FA_KV4
}

}  // namespace fa
