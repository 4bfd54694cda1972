// Writing keys and values into the 4-bit cache and reading them back.
//
// Of every 32 elements x of a row, ext is the largest if it exceeds the
// negative of the smallest, else the smallest; s = -ext/8 rounded to the row's
// 16-bit type (exact unless it falls below that type's normal range), and x
// is held as n = clamp(floor(x/s + 1/2), -8, 7).  The element of largest
// magnitude is n = -8 and comes back exactly; every other one is off by at
// most s/2, except an element of the opposite sign above 7.5/8 of that
// magnitude, which is clipped to 7s.
//
// Both calls stream: a row costs 2D bytes on the 16-bit side and 9D/16 in the
// cache, and nothing is kept between rows.
#include <cuda_runtime.h>

#include "fa.h"
#include "fa_kernels.h"
#include "fa_kv4.cuh"
#include "sm100_ptx.cuh"

namespace fa {
namespace {

constexpr int kThreads = 256;

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t u) {
  if constexpr (BF16)
    return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
  else
    return __half22float2(*reinterpret_cast<__half2*>(&u));
}

template <bool BF16>
__device__ __forceinline__ uint32_t max2_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16)
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <bool BF16>
__device__ __forceinline__ uint32_t min2_nan(uint32_t a, uint32_t b) {
  return max2_nan<BF16>(a ^ 0x80008000u, b ^ 0x80008000u) ^ 0x80008000u;
}

// Largest element (low half) and negative of the smallest (high half) of the
// 32 elements that four neighbouring lanes hold.
template <bool BF16>
__device__ __forceinline__ uint32_t extremes(const uint4& x) {
  uint32_t hi = max2_nan<BF16>(max2_nan<BF16>(x.x, x.y), max2_nan<BF16>(x.z, x.w));
  uint32_t lo = min2_nan<BF16>(min2_nan<BF16>(x.x, x.y), min2_nan<BF16>(x.z, x.w)) ^ 0x80008000u;
  uint32_t v = max2_nan<BF16>(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
  v = max2_nan<BF16>(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return max2_nan<BF16>(v, __shfl_xor_sync(0xffffffffu, v, 2));
}

// NaN -> 0, +-inf -> +-largest finite, in both half-words.
template <bool BF16>
__device__ __forceinline__ uint32_t finite2(uint32_t u) {
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h = (u >> (16 * i)) & 0xffffu;
    const uint32_t mag = h & 0x7fffu;
    if (mag > kInf) h = 0;
    if (mag == kInf) h = (h & 0x8000u) | (kInf - 1);
    r |= h << (16 * i);
  }
  return r;
}

// Quantises eight elements of a group whose other 24 are in the neighbouring
// lanes.  Returns the eight codes as a word of two half-words; *s16 gets the
// group's scale.
//
// x/s is a ratio of two numbers of at most 11 bits, so it lies on k + 1/2
// exactly or at least 2^-13 away from it; x * (1/s) is within 2^-20 of it (at
// most 8 in magnitude, two roundings of 2^-24 relative), and adding 2^-16
// puts ties, and only ties, above the border.
template <bool BF16>
__device__ __forceinline__ uint32_t quantise8(uint4 x, uint16_t* s16) {
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  uint32_t v = extremes<BF16>(x);
  const bool odd = (v & 0x7fffu) >= kInf || ((v >> 16) & 0x7fffu) >= kInf;
  if (__any_sync(0xffffffffu, odd)) {
    x = make_uint4(finite2<BF16>(x.x), finite2<BF16>(x.y), finite2<BF16>(x.z), finite2<BF16>(x.w));
    v = extremes<BF16>(x);
  }
  const float2 m = unpack2<BF16>(v);
  const float ext = m.x > m.y ? m.x : -m.y;
  uint16_t h;
  if constexpr (BF16)
    h = __bfloat16_as_ushort(__float2bfloat16_rn(ext * -0.125f));
  else
    h = __half_as_ushort(__float2half_rn(ext * -0.125f));
  float s = kv4_scale<BF16>(h);
  const bool none = fabsf(s) < 1.17549435e-38f;
  if (none) h = 0;
  *s16 = h;
  const float rs = none ? 0.f : __frcp_rn(s);
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t half[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack2<BF16>(in[2 * j + i / 2]);
      float t = fmaf(i & 1 ? f.y : f.x, rs, 8.5f + 1.f / 65536.f);
      t = fminf(fmaxf(t, 0.f), 15.5f);
      c[i] = __float_as_uint(__fadd_rz(t, 8388608.f));   // floor in the low bits
    }
    // sum of c_i 16^i; what the 0x4b of each float leaves is above bit 23
    half[j] = c[0] + (c[1] << 4) + (c[2] << 8) + (c[3] << 12);
  }
  return __byte_perm(half[0], half[1], 0x5410);
}

struct WriteParams {
  Kv4Cache c;
  const uint4* k;
  const uint4* v;
  int B, T;
  unsigned pairs;       // pairs of neighbouring positions per (sequence, head)
  long long units;      // B * Hkv * pairs
};

// D/8 lanes hold a row, eight elements each, K and V alike; 2 * D/8 lanes the
// two tokens of an even position and its successor, whose V codes share words.
template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) fa_kv4_write_kernel(const WriteParams p) {
  constexpr int L = D / 8, W = D / 32, UPW = 32 / (2 * L);
  grid_dependency_wait();
  grid_dependents_launch();
  const int lane = threadIdx.x % 32, l = lane % L, par = (lane / L) & 1;
  const long long u = ((long long)blockIdx.x * kThreads + threadIdx.x) / 32 * UPW + lane / (2 * L);
  uint8_t* blk = nullptr;
  long long pos = 0;
  uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
  if (u < p.units) {
    const long long bh = u / p.pairs;
    const int b = (int)(bh / p.c.Hkv), h = (int)(bh - (long long)b * p.c.Hkv);
    const int start = p.c.start[b];
    pos = (start & ~1) + 2ll * (u - bh * p.pairs) + par;
    const long long t = pos - start;
    if (t >= 0 && t < kv4_count(p.c, b, p.T)) {
      blk = kv4_block_of(p.c, b, h, pos, kv4_block_bytes(D));
      if (blk != nullptr) {
        const size_t at = ((size_t)bh * p.T + (size_t)t) * L + l;
        xk = p.k[at];
        xv = p.v[at];
      }
    }
  }
  uint16_t sk, sv;
  const uint32_t wk = quantise8<BF16>(xk, &sk);
  const uint32_t wv = quantise8<BF16>(xv, &sv);
  // the even token's lane completes the word of its first four elements of V, the odd one's that of the others
  const uint32_t other = __shfl_xor_sync(0xffffffffu, par ? wv & 0xffffu : wv >> 16, L);
  const bool both = __shfl_xor_sync(0xffffffffu, (int)(blk != nullptr), L) != 0 && blk != nullptr;
  if (blk == nullptr) return;
  const int key = (int)pos & 15, half = key >> 3;
  reinterpret_cast<uint32_t*>(blk)[((half * 8 + (key & 7)) * 4 + l % 4) * W + l / 4] = wk;
  uint32_t* vw = reinterpret_cast<uint32_t*>(blk + 8 * D) + ((half * 8 + l % 4 * 2) * 4 + ((key & 7) >> 1)) * W + l / 4;
  if (both) {
    vw[4 * W * par] = par ? __byte_perm(other, wv, 0x7610) : __byte_perm(wv, other, 0x5410);
  } else {
    reinterpret_cast<uint16_t*>(vw)[par] = (uint16_t)wv;
    reinterpret_cast<uint16_t*>(vw + 4 * W)[par] = (uint16_t)(wv >> 16);
  }
  if (l % 4 == 0) {
    uint16_t* s = reinterpret_cast<uint16_t*>(blk + 16 * D) + key * 2 * W + l / 4;
    s[0] = sk;
    s[W] = sv;
  }
}

// Eight codes (a word of two half-words) times s, in the 16-bit type.
template <bool BF16>
__device__ __forceinline__ uint4 values8(uint32_t w, float s) {
  uint32_t r[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int sh = 16 * (j / 2) + 8 * (j % 2);
    const float a = (float)((int)((w >> sh) & 15u) - 8) * s, b = (float)((int)((w >> (sh + 4)) & 15u) - 8) * s;
    if constexpr (BF16) {
      __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
      r[j] = *reinterpret_cast<uint32_t*>(&h);
    } else {
      __half2 h = __floats2half2_rn(a, b);
      r[j] = *reinterpret_cast<uint32_t*>(&h);
    }
  }
  return make_uint4(r[0], r[1], r[2], r[3]);
}

struct ReadParams {
  Kv4Cache c;
  uint4* k;
  uint4* v;
  int N;
  long long rows;       // B * Hkv * N
};

// D/8 lanes a row, eight elements each of K and of V.
template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) fa_kv4_read_kernel(const ReadParams p) {
  constexpr int L = D / 8, W = D / 32;
  grid_dependency_wait();
  grid_dependents_launch();
  const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
  const long long row = i / L;
  const int l = (int)(i % L);
  if (row >= p.rows) return;
  const long long bh = row / p.N;
  const int b = (int)(bh / p.c.Hkv), h = (int)(bh - (long long)b * p.c.Hkv), t = (int)(row - bh * p.N);
  uint4 xk = make_uint4(0, 0, 0, 0), xv = xk;
  if (t < kv4_count(p.c, b, p.N)) {
    const long long pos = (long long)p.c.start[b] + t;
    const uint8_t* blk = kv4_block_of(p.c, b, h, pos, kv4_block_bytes(D));
    if (blk != nullptr) {
      const int key = (int)pos & 15, half = key >> 3;
      const uint16_t* s = reinterpret_cast<const uint16_t*>(blk + 16 * D) + key * 2 * W + l / 4;
      const uint32_t wk = reinterpret_cast<const uint32_t*>(blk)[((half * 8 + (key & 7)) * 4 + l % 4) * W + l / 4];
      const uint32_t* vw =
          reinterpret_cast<const uint32_t*>(blk + 8 * D) + ((half * 8 + l % 4 * 2) * 4 + ((key & 7) >> 1)) * W + l / 4;
      const uint2 v = make_uint2(vw[0], vw[4 * W]);
      xk = values8<BF16>(wk, kv4_scale<BF16>(s[0]));
      xv = values8<BF16>(__byte_perm(v.x, v.y, key & 1 ? 0x7632 : 0x5410), kv4_scale<BF16>(s[W]));
    }
  }
  p.k[(size_t)i] = xk;
  p.v[(size_t)i] = xv;
}

}  // namespace

cudaError_t launch_kv4_write(bool bf16, int d, const Kv4Cache& c, const void* k, const void* v, int B, int T,
                             cudaStream_t st) {
  WriteParams p{c, static_cast<const uint4*>(k), static_cast<const uint4*>(v), B, T, (unsigned)(T / 2 + 1), 0};
  p.units = (long long)B * c.Hkv * p.pairs;
  const long long per_cta = kThreads / 32 * (32 / (2 * (d / 8)));
  const long long grid = (p.units + per_cta - 1) / per_cta;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  auto kern = bf16 ? (d == 64 ? fa_kv4_write_kernel<true, 64> : fa_kv4_write_kernel<true, 128>)
                   : (d == 64 ? fa_kv4_write_kernel<false, 64> : fa_kv4_write_kernel<false, 128>);
  return launch_chained(kern, dim3((unsigned)grid), dim3(kThreads), 0, st, p);
}

cudaError_t launch_kv4_read(bool bf16, int d, const Kv4Cache& c, void* k, void* v, int B, int N, cudaStream_t st) {
  ReadParams p{c, static_cast<uint4*>(k), static_cast<uint4*>(v), N, (long long)B * c.Hkv * N};
  const long long grid = (p.rows * (d / 8) + kThreads - 1) / kThreads;
  if (grid > 0x7fffffffll) return cudaErrorInvalidConfiguration;
  auto kern = bf16 ? (d == 64 ? fa_kv4_read_kernel<true, 64> : fa_kv4_read_kernel<true, 128>)
                   : (d == 64 ? fa_kv4_read_kernel<false, 64> : fa_kv4_read_kernel<false, 128>);
  return launch_chained(kern, dim3((unsigned)grid), dim3(kThreads), 0, st, p);
}

}  // namespace fa
