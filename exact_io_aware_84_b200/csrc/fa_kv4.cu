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
// cache, and nothing is kept between rows.  A warp takes a block of 16
// positions of a head, lane 4g + t the elements 32e + 8t .. + 7 of the keys g
// and 8 + g, so that a block's codes are whole 16-byte vectors of its lanes: K
// as they come out, V after a transposition of half-words (movmatrix).
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
  uint32_t r;
  if constexpr (BF16)
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// All lanes of a warp together: volatile, so that it stays where the source
// has the warp whole.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// Largest of a lane's eight elements of a group (low half) and negative of
// the smallest (high half).
template <bool BF16>
__device__ __forceinline__ uint32_t extremes(const uint4& x) {
  const uint32_t hi = max2_nan<BF16>(max2_nan<BF16>(x.x, x.y), max2_nan<BF16>(x.z, x.w));
  const uint32_t lo = min2_nan<BF16>(min2_nan<BF16>(x.x, x.y), min2_nan<BF16>(x.z, x.w)) ^ 0x80008000u;
  return max2_nan<BF16>(__byte_perm(hi, lo, 0x5410), __byte_perm(hi, lo, 0x7632));
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

// The extremes of four groups that four neighbouring lanes hold together; lane
// t gets those of group t.
template <bool BF16>
__device__ __forceinline__ uint32_t extremes_of_mine(const uint4 (&x)[4], int t) {
  uint32_t m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = extremes<BF16>(x[j]);
  const bool up = (t & 2) != 0, odd = (t & 1) != 0;
  const uint32_t a = max2_nan<BF16>(up ? m[2] : m[0], __shfl_xor_sync(0xffffffffu, up ? m[0] : m[2], 2));
  const uint32_t b = max2_nan<BF16>(up ? m[3] : m[1], __shfl_xor_sync(0xffffffffu, up ? m[1] : m[3], 2));
  return max2_nan<BF16>(odd ? b : a, __shfl_xor_sync(0xffffffffu, odd ? a : b, 1));
}

// Quantises four groups, of each of which four neighbouring lanes hold eight
// elements: the codes as words of two half-words.  Returns the scale of group
// t in lane t.
//
// x/s is a ratio of two numbers of at most 11 bits, so it lies on k + 1/2
// exactly or at least 2^-13 away from it; the product with an approximate 1/s
// is within 2^-19 of it (at most 8 in magnitude).  Adding 2^-16 puts ties, and
// only ties, above the border.  In sixteenths the sum saturates to [0, 1];
// times 16 (1 - 2^-22), at most 2^-18 less, and added to 2^23 with truncation,
// it leaves its floor, 0 to 15, in the low bits.
template <bool BF16>
__device__ __forceinline__ uint16_t quantise4(uint4 (&x)[4], uint32_t (&word)[4], int lane) {
  constexpr uint32_t kInf = BF16 ? 0x7f80u : 0x7c00u;
  const int t = lane % 4;
  uint32_t v = extremes_of_mine<BF16>(x, t);
  const bool strange = (v & 0x7fffu) >= kInf || ((v >> 16) & 0x7fffu) >= kInf;
  if (__any_sync(0xffffffffu, strange)) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[j] = make_uint4(finite2<BF16>(x[j].x), finite2<BF16>(x[j].y), finite2<BF16>(x[j].z), finite2<BF16>(x[j].w));
    v = extremes_of_mine<BF16>(x, t);
  }
  const float2 m = unpack2<BF16>(v);
  const float ext = m.x > m.y ? m.x : -m.y;
  uint16_t h;
  if constexpr (BF16)
    h = __bfloat16_as_ushort(__float2bfloat16_rn(ext * -0.125f));
  else
    h = __half_as_ushort(__float2half_rn(ext * -0.125f));
  const float s = kv4_scale<BF16>(h);
  float rs;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rs) : "f"(s));
  if (fabsf(s) < 1.17549435e-38f) rs = 0.f, h = 0;
  rs *= 0.0625f;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float r = __shfl_sync(0xffffffffu, rs, (lane & 28) + j);
    const uint32_t in[4] = {x[j].x, x[j].y, x[j].z, x[j].w};
    uint32_t half[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t c[4];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 f = unpack2<BF16>(in[2 * i + k]);
        c[2 * k] = __float_as_uint(__fmaf_rz(__saturatef(fmaf(f.x, r, (8.5f + 1.f / 65536.f) / 16.f)),
                                             16.f - 1.f / 262144.f, 8388608.f));
        c[2 * k + 1] = __float_as_uint(__fmaf_rz(__saturatef(fmaf(f.y, r, (8.5f + 1.f / 65536.f) / 16.f)),
                                                 16.f - 1.f / 262144.f, 8388608.f));
      }
      // sum of c_i 16^i; what the 0x4b of each float leaves is above bit 23
      half[i] = c[0] + c[1] * 16u + c[2] * 256u + c[3] * 4096u;
    }
    word[j] = __byte_perm(half[0], half[1], 0x5410);
  }
  return h;
}

// A warp's block of positions: sequence, head, and position of its first key.
struct Unit {
  int b, h, n;       // n: tokens of the sequence
  long long bh, pos, start;
};

__device__ __forceinline__ Unit unit_of(const Kv4Cache& c, unsigned u, unsigned blocks, int T) {
  Unit r;
  r.bh = u / blocks;
  r.b = (int)r.bh / c.Hkv;
  r.h = (int)r.bh - r.b * c.Hkv;
  r.start = c.start[r.b];
  r.n = kv4_count(c, r.b, T);
  r.pos = (r.start & ~15ll) + 16ll * (u - (unsigned)r.bh * blocks);
  return r;
}

struct WriteParams {
  Kv4Cache c;
  const uint4* k;
  const uint4* v;
  int T;
  unsigned blocks, units;   // of a head of a sequence, in all
};

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) fa_kv4_write_kernel(const WriteParams p) {
  constexpr int W = D / 32;
  const unsigned u = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  grid_dependency_wait();
  grid_dependents_launch();
  if (u >= p.units) return;
  const Unit r = unit_of(p.c, u, p.blocks, p.T);
  const long long first = r.pos - r.start;         // the block's first token, of this call's
  if (first >= r.n || first <= -16 || r.n == 0) return;
  uint8_t* const blk = kv4_block_of(p.c, r.b, r.h, r.pos, kv4_block_bytes(D));
  if (blk == nullptr) return;
  auto there = [&](int key) { return first + key >= 0 && first + key < r.n; };

  // One half at a time: with both in flight fewer warps are, and 2 x 16 heads x
  // 8192 x 128 took 33 us instead of 28.
#pragma unroll 1
  for (int half = 0; half < 2; ++half) {
    if (first + half * 8 >= r.n || first + half * 8 + 8 <= 0) continue;
    const bool mine = there(half * 8 + g);
    uint4 x[2 * W];
#pragma unroll
    for (int j = 0; j < 2 * W; ++j) {
      x[j] = make_uint4(0, 0, 0, 0);
      const size_t row = (size_t)r.bh * p.T + (size_t)(first + half * 8 + g);
      if (mine) x[j] = (j < W ? p.k : p.v)[row * (D / 8) + 4 * (j % W) + t];
    }

    uint32_t word[2 * W];
#pragma unroll
    for (int q = 0; q < W / 2; ++q) {   // four groups at a time
      uint4 (&x4)[4] = *reinterpret_cast<uint4(*)[4]>(&x[4 * q]);
      uint32_t (&w4)[4] = *reinterpret_cast<uint32_t(*)[4]>(&word[4 * q]);
      const uint16_t s = quantise4<BF16>(x4, w4, lane);
      if (mine) reinterpret_cast<uint16_t*>(blk + 16 * D)[(half * 8 + g) * 2 * W + 4 * q + t] = s;
    }
    __syncwarp();
#pragma unroll
    for (int e = 0; e < W; ++e) word[W + e] = transpose8x8(word[W + e]);   // lane: r = g, keys 2t and 2t + 1
    uint32_t* const kw = reinterpret_cast<uint32_t*>(blk) + (half * 32 + lane) * W;
    uint32_t* const vw = reinterpret_cast<uint32_t*>(blk + 8 * D) + (half * 32 + lane) * W;
    const bool low = there(half * 8 + 2 * t), high = there(half * 8 + 2 * t + 1);
    if constexpr (W == 4) {
      if (mine) *reinterpret_cast<uint4*>(kw) = make_uint4(word[0], word[1], word[2], word[3]);
      if (low && high) *reinterpret_cast<uint4*>(vw) = make_uint4(word[4], word[5], word[6], word[7]);
    } else {
      if (mine) *reinterpret_cast<uint2*>(kw) = make_uint2(word[0], word[1]);
      if (low && high) *reinterpret_cast<uint2*>(vw) = make_uint2(word[2], word[3]);
    }
    if (low != high) {   // the other half-words are another call's
#pragma unroll
      for (int e = 0; e < W; ++e)
        reinterpret_cast<uint16_t*>(vw + e)[high] = (uint16_t)(high ? word[W + e] >> 16 : word[W + e]);
    }
  }
}

// Eight codes (a word of two half-words) times s, rounded once to the 16-bit
// type: n is exact in it, from 128 + c (bf16) or 1024 + c (fp16).
template <bool BF16>
__device__ __forceinline__ uint4 values8(uint32_t w, uint16_t s) {
  uint32_t v[4];   // elements i and i + 4
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t c = (w >> (4 * i) & 0x000f000fu) | (BF16 ? 0x43004300u : 0x64006400u);
    if constexpr (BF16) {
      const __nv_bfloat162 n = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&c), __float2bfloat162_rn(136.f));
      const __nv_bfloat162 y = __hmul2(n, __bfloat162bfloat162(__ushort_as_bfloat16(s)));
      v[i] = *reinterpret_cast<const uint32_t*>(&y);
    } else {
      const __half2 n = __hsub2(*reinterpret_cast<const __half2*>(&c), __float2half2_rn(1032.f));
      const __half2 y = __hmul2(n, __half2half2(__ushort_as_half(s)));
      v[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
  }
  return make_uint4(__byte_perm(v[0], v[1], 0x5410), __byte_perm(v[2], v[3], 0x5410), __byte_perm(v[0], v[1], 0x7632),
                    __byte_perm(v[2], v[3], 0x7632));
}

struct ReadParams {
  Kv4Cache c;
  uint4* k;
  uint4* v;
  int N;
  unsigned blocks, units;
};

template <bool BF16, int D>
__global__ void __launch_bounds__(kThreads) fa_kv4_read_kernel(const ReadParams p) {
  constexpr int W = D / 32;
  const unsigned u = blockIdx.x * (kThreads / 32) + threadIdx.x / 32;
  const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
  grid_dependency_wait();
  grid_dependents_launch();
  if (u >= p.units) return;
  const Unit r = unit_of(p.c, u, p.blocks, p.N);
  const long long first = r.pos - r.start;
  if (first >= p.N || first <= -16) return;
  const uint8_t* blk = nullptr;
  if (first < r.n && r.n > 0) blk = kv4_block_of(p.c, r.b, r.h, r.pos, kv4_block_bytes(D));

  uint32_t kw[2][W], vw[2][W], sw[2][W];   // sw: the scales of a key, two to a word
#pragma unroll
  for (int half = 0; half < 2; ++half) {
#pragma unroll
    for (int e = 0; e < W; ++e) kw[half][e] = vw[half][e] = sw[half][e] = 0;
    if (blk != nullptr) {
      if constexpr (W == 4) {
        const uint4 a = reinterpret_cast<const uint4*>(blk)[half * 32 + lane];
        const uint4 b = reinterpret_cast<const uint4*>(blk + 8 * D)[half * 32 + lane];
        const uint4 c = reinterpret_cast<const uint4*>(blk + 16 * D)[half * 8 + g];
        kw[half][0] = a.x, kw[half][1] = a.y, kw[half][2] = a.z, kw[half][3] = a.w;
        vw[half][0] = b.x, vw[half][1] = b.y, vw[half][2] = b.z, vw[half][3] = b.w;
        sw[half][0] = c.x, sw[half][1] = c.y, sw[half][2] = c.z, sw[half][3] = c.w;
      } else {
        const uint2 a = reinterpret_cast<const uint2*>(blk)[half * 32 + lane];
        const uint2 b = reinterpret_cast<const uint2*>(blk + 8 * D)[half * 32 + lane];
        const uint2 c = reinterpret_cast<const uint2*>(blk + 16 * D)[half * 8 + g];
        kw[half][0] = a.x, kw[half][1] = a.y;
        vw[half][0] = b.x, vw[half][1] = b.y;
        sw[half][0] = c.x, sw[half][1] = c.y;
      }
    }
  }
  __syncwarp();
#pragma unroll
  for (int half = 0; half < 2; ++half)
#pragma unroll
    for (int e = 0; e < W; ++e) vw[half][e] = transpose8x8(vw[half][e]);
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const long long row = first + half * 8 + g;
    const bool live = blk != nullptr && row < r.n;
    if (row < 0 || row >= p.N) continue;
#pragma unroll
    for (int e = 0; e < W; ++e) {
      const size_t at = ((size_t)r.bh * p.N + (size_t)row) * (D / 8) + 4 * e + t;
      const uint4 none = make_uint4(0, 0, 0, 0);
      p.k[at] = live ? values8<BF16>(kw[half][e], (uint16_t)(sw[half][e / 2] >> (16 * (e & 1)))) : none;
      p.v[at] = live ? values8<BF16>(vw[half][e], (uint16_t)(sw[half][(W + e) / 2] >> (16 * (e & 1)))) : none;
    }
  }
}

}  // namespace

// Blocks that T tokens lie in at most, wherever the first one is, and warps.
static bool units_of(int B, int Hkv, int T, unsigned* blocks, unsigned* units, unsigned* grid) {
  const long long a = ((long long)T + 14) / 16 + 1, all = a * B * Hkv;
  *blocks = (unsigned)a;
  *units = (unsigned)all;
  *grid = (unsigned)((all + kThreads / 32 - 1) / (kThreads / 32));
  return all < (1ll << 32) - kThreads;
}

cudaError_t launch_kv4_write(bool bf16, int d, const Kv4Cache& c, const void* k, const void* v, int B, int T,
                             cudaStream_t st) {
  WriteParams p{c, static_cast<const uint4*>(k), static_cast<const uint4*>(v), T, 0, 0};
  unsigned grid;
  if (!units_of(B, c.Hkv, T, &p.blocks, &p.units, &grid)) return cudaErrorInvalidConfiguration;
  auto kern = bf16 ? (d == 64 ? fa_kv4_write_kernel<true, 64> : fa_kv4_write_kernel<true, 128>)
                   : (d == 64 ? fa_kv4_write_kernel<false, 64> : fa_kv4_write_kernel<false, 128>);
  return launch_chained(kern, dim3(grid), dim3(kThreads), 0, st, p);
}

cudaError_t launch_kv4_read(bool bf16, int d, const Kv4Cache& c, void* k, void* v, int B, int N, cudaStream_t st) {
  ReadParams p{c, static_cast<uint4*>(k), static_cast<uint4*>(v), N, 0, 0};
  unsigned grid;
  if (!units_of(B, c.Hkv, N, &p.blocks, &p.units, &grid)) return cudaErrorInvalidConfiguration;
  auto kern = bf16 ? (d == 64 ? fa_kv4_read_kernel<true, 64> : fa_kv4_read_kernel<true, 128>)
                   : (d == 64 ? fa_kv4_read_kernel<false, 64> : fa_kv4_read_kernel<false, 128>);
  return launch_chained(kern, dim3(grid), dim3(kThreads), 0, st, p);
}

}  // namespace fa
