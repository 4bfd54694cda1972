// Attention of a few new tokens per sequence over the 4-bit key/value cache.
//
// Per query row: S_j = scale * sum_e s_K(j,e) sum_{i in group e} q_i n_K(j,i),
// P = softmax over the keys j that the row may see, O = sum_j P_j s_V n_V.
// The codes are used as they stand, never rounded to 16 bits.
//
// Work.  A unit is one key head's tile of up to NT * 8 query rows; its keys
// are cut into steps of 64 (NT = 1) or 32.  Lengths are known on the device
// only.  Two divisions:
//   near: a cluster of up to 8 CTAs to a unit, whose warps take equal shares
//     of its steps and which joins them through distributed shared memory.
//     For few and short units: one kernel, no plan, no trip through memory.
//   far: the steps of all units, laid end to end, are divided evenly over the
//     warps of a grid that fills the GPU once (each CTA sums the lengths up
//     first).  A warp that holds a unit from its first to its last step writes
//     the result; the pieces of a unit that lies across warps go to the
//     workspace, and a second kernel joins them.
// Sums are in a fixed order: the same call gives the same bits.
//
// A step.  Its blocks of 16 keys come by asynchronous bulk copy into a ring
// that belongs to the warp, so no warp waits for another.
//   S^T = K Q^T by mma.m16n8k16, keys as rows and 8 query rows as columns:
//     nothing is wasted when four or eight query heads share a key head.  A
//     code c = n + 8 enters as the fp16 subnormal that its nibble is; each
//     group's sum of 32 starts at -8 times the sum of q and is then scaled in
//     float32.  q goes in as fp16, its row's largest element brought to
//     2^14 .. 2^15 by a power of two that the scale takes back: elements below
//     2^-24 of the row's largest round, at 2^-35 of it.  Where four or two rows
//     are all there are, each takes C = 2 or 4 columns.
//   O^T = V^T P^T: the head's elements as rows.  V's codes become n by one
//     fp16 subtraction, exactly: a sum over many keys must not carry an offset
//     (taking it back by a product with -8 measured 6% slower).  P s_V is
//     rounded to fp16 after a factor v_up of its row, which O's end takes back,
//     and changes from accumulator to operand order by movmatrix.  A product's
//     rows belong to one group of 32 elements, as s_V does; with C > 1 they
//     belong to two, and a row's columns hold P s_V for one group each, so that
//     C times fewer are made.
// P is taken relative to 2^m, m 48 below the running maximum where it was last
// moved (in log2); it moves only when a score passes that maximum by 8.  Weights
// down to 2^-174 so stay in float32's range, for bf16 values reach 2^128.  v_up
// follows the row's largest P |s_V| so far in the same way: it falls, bringing
// that to 2^6, when a bound on the step's passes 2^15, and it rises as m
// does, so that what O's sums are relative to does not change with m.  (Where
// P |s_V| passes 2^120, m rises by 56 instead.)  A row thus rounds relative to
// the products of the keys that it sees: keys of other rows, and keys of no
// weight whatever their values, have no say.  The bound is the largest P of a
// lane's keys times the largest |s_V| of any key of theirs; the products
// themselves are looked at, as logarithms, where it passes.  (A factor
// common to a tile's rows and taken from V's scales alone was 2 to 5% faster and
// lost rows beside a key of large V that they did not see.)  P s_V in fp16 adds
// 2^-11 a term to an error that O's own rounding to fp16 bounds by 2^-11 (2.1e-4
// to 2.9e-4 over 24 x 4 tokens of 128); two halves of P s_V would double the
// products, of which a step has as many for V as for K.
//
// What bounds it.  Reading the cache once: 9D/8 bytes a key and key head, 104 SM
// cycles for 16 keys at d = 128.  The steps of 64 sequences of up to 8192 keys
// and 4 rows take 117, start and ends among them: 257 instructions and 16
// products, which fill 56% of the issue slots and 45% of the integer pipe, the
// busiest one.  No pipe is full, nor memory (58%): a warp's own chain of
// dependent instructions, with three warps a scheduler, is what takes the time.
// Measured on B200 (graph of calls): 8 sequences of 65536 keys and 8 rows 115 us,
// 5.3 TB/s; 64 sequences of up to 8192 keys and 4 rows 69 us, 4.8 TB/s, about
// 14 us of both being the start, the ends of units and the joining kernel; one
// sequence of 1000 keys 8.4 us.  A product costs its pipe 8.5 cycles a SM
// quarter and delays the integer instructions beside it (4 of them and 4
// half-precision ones: 12.8), so 24 products in place of 32 subtractions lost.
#include <cuda_runtime.h>

#include <atomic>

#include "fa.h"
#include "fa_kernels.h"
#include "fa_kv4.cuh"
#include "sm100_ptx.cuh"

namespace fa {

// What the joining kernel needs to know of a unit that ends behind the range
// of the worker in which it begins (parts = 0 for others).
struct Kv4Join {
  long long row;   // first row of the unit in O and LSE
  int rows;
  int worker, parts;   // the worker, and how many pieces follow in those behind it
};

namespace {

constexpr int kWarps = 4;               // of a CTA
constexpr int kThreads = 32 * kWarps;
constexpr int kSeen = kThreads;         // sequences whose lengths a CTA keeps at hand
constexpr float kUnit = 16777216.f;     // scores and O are summed in units of 2^-24, the subnormals' step
constexpr float kLeast = -3.402823466e38f;   // a maximum before the first key
constexpr float kBelow = 48.f;          // log2 by which m lies below the running maximum when it moves,
constexpr float kLazy = 56.f;           // and by which a score may pass m
constexpr float kMostUp = 0x1p70f;      // P v_up stays finite
constexpr float kVPass = 15.f;          // log2: P |s_V| v_up stays in fp16's range
constexpr float kMostV = 120.f;         // log2 of a P |s_V| for which v_up would get too small

template <int D, int NT, int C>
struct Shape {
  static constexpr int W = D / 32, Rows = 8 * NT / C, Block = kv4_block_bytes(D);
  // Blocks of a step, CTAs a SM (as registers allow) and steps on their way to
  // a warp (as shared memory allows).
  static constexpr int Blocks = NT == 1 ? 4 : 2, Step = kKv4Block * Blocks;
  static constexpr int CtasPerSm = W * NT <= 2 ? 4 : W * NT <= 4 ? 3 : 2;
  static constexpr int Stages = CtasPerSm == 3 && D == 128 ? 2 : CtasPerSm == 4 ? 3 : 4;
  static constexpr int Slot = Rows * (D + 2);   // floats of a partial result: O, then m and l by row
  static constexpr int RowBytes = 4 * NT * W * 16;   // per warp: what is taken off the scores of each column pair
  static constexpr int Stage = Blocks * Block;
  static constexpr size_t Smem = (size_t)kWarps * (Stages * Stage + RowBytes);
};

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                         const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ uint32_t hsub2(uint32_t a, uint32_t b) {
  __half2 r = __hsub2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
  return *reinterpret_cast<uint32_t*>(&r);
}

// The codes of places 0 and 2 (in units of 2^-24) and of places 1 and 3 (of
// 2^-20) of a half-word, or of one shifted by 8, less their offset.
__device__ __forceinline__ uint32_t code_even(uint32_t x) { return hsub2(x & 0x000f000fu, 0x00080008u); }
__device__ __forceinline__ uint32_t code_odd(uint32_t x) { return hsub2(x & 0x00f000f0u, 0x00800080u); }

// Of both half-words, the one of larger magnitude (its sign is of no use).
template <bool BF16>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (BF16)
    asm("max.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The scale in the low or high half of a word; a mixed-precision addition, as
// the integer pipe is the busier one.
template <bool BF16>
__device__ __forceinline__ float scale_half(uint32_t w, int high) {
  if constexpr (BF16) {
    float r;
    if (high)
      asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; add.f32.bf16 %0, h, %2;}" : "=f"(r) : "r"(w), "f"(-0.f));
    else
      asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; add.f32.bf16 %0, l, %2;}" : "=f"(r) : "r"(w), "f"(-0.f));
    return r;
  } else {
    return kv4_scale<false>((uint16_t)(w >> (16 * high)));
  }
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ float quad_max(float x) {
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
  x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
  return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}

__device__ __forceinline__ float quad_sum(float x) {
  x += __shfl_xor_sync(0xffffffffu, x, 4);
  x += __shfl_xor_sync(0xffffffffu, x, 8);
  return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

__device__ __forceinline__ float lg2_approx(float x) {
  float r;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }   // -126 <= e <= 127

// l is about 2^kBelow: as near to 0 as its logarithm gets, for its bits' sake.
__device__ __forceinline__ float lse_of(float m, float l) {
  return (m + kBelow + log2f(l * 0x1p-48f)) * 0.69314718055994531f;
}

// How far a sequence reaches in this call.
struct Reach {
  int n, keys, steps;   // tokens, keys that the last of them sees, steps of a unit (at least one)
  long long start;

  __device__ __forceinline__ Reach(const Kv4FwdParams& p, int first, int count, int step) : n(count), start(first) {
    const long long end = n > 0 ? start + n : 0, cap = (long long)p.c.max_pages << p.c.page_shift;
    keys = (int)(end < 0 ? 0 : end > cap ? cap : end);
    steps = keys > 0 ? (int)(((long long)keys + step - 1) / step) : 1;
  }
};

// Two elements of O in 16 bits.  O is an average of finite values, but P s_V's
// rounding can put it half a step past fp16's largest (bf16's is further off).
template <bool BF16>
__device__ __forceinline__ uint32_t pack_o(float a, float b) {
  if constexpr (!BF16) {
    a = fabsf(a) > 65504.f ? copysignf(65504.f, a) : a;
    b = fabsf(b) > 65504.f ? copysignf(65504.f, b) : b;
  }
  return pack2<BF16>(a, b);
}

__device__ __forceinline__ float* slot_of(const Kv4FwdParams& p, long long worker, int which, int slot_floats) {
  return p.partials + (size_t)(2 * worker + which) * slot_floats;
}

// Part of a row's result: O, the maximum m (in log2) and sum l.  l = 0: no key.
struct Piece {
  float4 o;
  float m, l;

  // With N more, each O[i] with its m and l.  O stays an average, under weights
  // of at most 1: no sum overflows that O itself does not.  Where a weight is
  // small, 2^64 of it goes to O[i], so that it does not underflow.
  template <int N>
  __device__ __forceinline__ void add(const float4 (&x)[N], const float2 (&ml)[N]) {
    float top = m;
#pragma unroll
    for (int i = 0; i < N; ++i) top = fmaxf(top, ml[i].x);
    float w[N + 1], down[N + 1], sum = 0.f;   // the last one is this piece's
#pragma unroll
    for (int i = 0; i <= N; ++i) {
      const float at = (i < N ? ml[i].x : m) - top;
      const bool small = at < -64.f;
      w[i] = (i < N ? ml[i].y : l) * ex2_approx(small ? at + 64.f : at);
      down[i] = small ? 0x1p-64f : 1.f;
      sum = fmaf(w[i], down[i], sum);
    }
    const float inv = sum > 0.f ? __fdividef(1.f, sum) : 0.f;
    const float keep = w[N] * inv;
    o.x = o.x * down[N] * keep, o.y = o.y * down[N] * keep, o.z = o.z * down[N] * keep, o.w = o.w * down[N] * keep;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float y = w[i] * inv;
      o.x = fmaf(x[i].x * down[i], y, o.x), o.y = fmaf(x[i].y * down[i], y, o.y);
      o.z = fmaf(x[i].z * down[i], y, o.z), o.w = fmaf(x[i].w * down[i], y, o.w);
    }
    m = top;
    l = sum;
  }
};

template <bool BF16>
__device__ __forceinline__ void store_result(const Kv4FwdParams& p, const Piece& x, long long row, int D, int col) {
  const float4 o = x.o;
  if (p.o32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.o) + row * D + col) = o;
  else
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + row * D + col) =
        make_uint2(pack_o<BF16>(o.x, o.y), pack_o<BF16>(o.z, o.w));
  if (col == 0) p.lse[row] = lse_of(x.m, x.l);
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Joins the pieces that the warps of a cluster have left at the start of their
// rings: the CTAs divide the unit's rows and columns.
template <bool BF16, int D, int NT, int C>
__device__ __forceinline__ void join_in_cluster(const Kv4FwdParams& p, const uint8_t* ring_all) {
  using Sh = Shape<D, NT, C>;
  __syncwarp();
  cluster_sync();
  const unsigned unit = blockIdx.x / (unsigned)p.cluster, rank = blockIdx.x % (unsigned)p.cluster;
  const unsigned u = unit % (unsigned)p.units_per_seq, tile = u % (unsigned)p.row_tiles;
  const long long group_rows = (long long)(p.H / p.c.Hkv) * p.T;
  const long long row0 = (unit / (unsigned)p.units_per_seq * (long long)p.c.Hkv + u / p.row_tiles) * group_rows + (long long)tile * Sh::Rows;
  const long long left = group_rows - (long long)tile * Sh::Rows;
  const int rows = left < Sh::Rows ? (int)left : Sh::Rows;
  const uint32_t base = smem_u32(ring_all);
  for (int i = rank * kThreads + threadIdx.x; i < rows * (D / 4); i += p.cluster * kThreads) {
    const int row = i / (D / 4), col = 4 * (i % (D / 4));
    Piece sum{make_float4(0.f, 0.f, 0.f, 0.f), kLeast, 0.f};
#pragma unroll 2
    for (int r = 0; r < p.cluster; ++r) {
      uint32_t there;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(there) : "r"(base), "r"(r));
      float4 x[kWarps];
      float2 ml[kWarps];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const uint32_t at = there + w * Sh::Stages * Sh::Stage;
        asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                     : "=f"(x[w].x), "=f"(x[w].y), "=f"(x[w].z), "=f"(x[w].w)
                     : "r"(at + (row * D + col) * 4));
        asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                     : "=f"(ml[w].x), "=f"(ml[w].y)
                     : "r"(at + (Sh::Rows * D + 2 * row) * 4));
      }
      sum.add(x, ml);
    }
    store_result<BF16>(p, sum, row0 + row, D, col);
  }
  __syncwarp();
  cluster_sync();   // no CTA ends while another reads its shared memory
}

// Near: a cluster of CTAs to a unit, whose warps divide its steps and whose
// shared memory joins them.  Else all warps divide all steps.
template <bool BF16, int D, int NT, int C, bool Near>
__global__ void __launch_bounds__(kThreads, (Shape<D, NT, C>::CtasPerSm)) fa_kv4_fwd_kernel(const Kv4FwdParams p) {
  using Sh = Shape<D, NT, C>;
  constexpr int W = Sh::W, ST = Sh::Stages, KB = Sh::Blocks, Block = Sh::Block;
  constexpr int kBatch = 32 / KB;   // steps whose pages a warp looks up at once
  extern __shared__ __align__(128) uint8_t ring_all[];
  __shared__ __align__(8) uint64_t bars[kWarps][ST];
  __shared__ long long warp_sum[kWarps], split[2];
  __shared__ int abort_flag;
  __shared__ int2 seen[kSeen];   // start and count
  long long* const chunk_sum = reinterpret_cast<long long*>(ring_all);   // until the first copies

  const int lane = threadIdx.x % 32, warp = threadIdx.x / 32, g = lane / 4, t = lane % 4;
  const int column_class = t * C / 4;   // which of a row's C columns this lane's are
  uint8_t* const ring = ring_all + (size_t)warp * ST * Sh::Stage;
  float4* const less = reinterpret_cast<float4*>(ring_all + (size_t)kWarps * ST * Sh::Stage + warp * Sh::RowBytes) + t;
  const uint32_t bar0 = smem_u32(&bars[warp][0]), ring0 = smem_u32(ring);
  if (threadIdx.x == 0) abort_flag = 0;
  if (lane < ST) mbar_init(bar0 + 8 * lane, KB);
  fence_mbar_init();
  __syncthreads();
  grid_dependency_wait();
  grid_dependents_launch();

  // A unit: sequence, key head, tile of query rows.
  struct Place {
    int b, h, tile;
  };
  int b_seen = 0;
  auto reach = [&](int b) {
    const int i = b - b_seen;
    const int2 x = !Near && i < kSeen ? seen[i] : make_int2(p.c.start[b], kv4_count(p.c, b, p.T));
    return Reach(p, x.x, x.y, Sh::Step);
  };
  // To the unit that follows (the last one's successor is the last one).
  auto move_on = [&](Place& x, Reach& r) {
    if (++x.tile < p.row_tiles) return;
    x.tile = 0;
    if (++x.h < p.c.Hkv) return;
    x.h = 0;
    if (x.b < p.B - 1) r = reach(++x.b);
  };
  auto past_table = [&](const Reach& r) {
    if (r.n > 0 && r.start + r.n > r.keys && r.start + r.n > 0) kv4_no_page(p.c);
  };

  // ---- which steps are this warp's
  const long long worker = (long long)blockIdx.x * kWarps + warp;
  int left = 0;   // steps (2^31 of them would be hours)
  Place at{0, 0, 0};   // the unit at hand
  int at_step = 0;     // and the step in it that comes next
  if constexpr (Near) {
    const unsigned unit = blockIdx.x / (unsigned)p.cluster, tiles = (unsigned)p.row_tiles, heads = (unsigned)p.c.Hkv;
    at = Place{(int)(unit / tiles / heads), (int)(unit / tiles % heads), (int)(unit % tiles)};
    const Reach r = reach(at.b);
    if (at.h == 0 && at.tile == 0 && threadIdx.x == 0) past_table(r);
    const long long part = worker - (long long)unit * p.cluster * kWarps, parts = p.cluster * kWarps;
    at_step = (int)(part * r.steps / parts);
    left = (int)((part + 1) * r.steps / parts) - at_step;
  } else {
    const int per = (p.B + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int i = 0, b = threadIdx.x * per; i < per && b < p.B; ++i, ++b) {
      const int2 x = make_int2(p.c.start[b], kv4_count(p.c, b, p.T));
      const Reach r(p, x.x, x.y, Sh::Step);
      if (per == 1) seen[threadIdx.x] = x;
      mine += r.steps;
      if (blockIdx.x == 0) past_table(r);
    }
    mine *= p.units_per_seq;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) before += warp_sum[i];
      total += warp_sum[i];
    }
    chunk_sum[threadIdx.x] = before + incl - mine;
    __syncthreads();

    const long long workers = total < p.workers ? total : p.workers;
    const long long each = total / workers, more = total - each * workers;   // the first `more` have one step more
    auto begin_of = [&](long long w) { return w < workers ? w * each + (w < more ? w : more) : total; };
    const long long here = begin_of(worker);
    if (threadIdx.x == 0) split[0] = each, split[1] = more;
    // the last chunk of sequences that does not begin behind a step
    auto chunk_of = [&](long long step) {
      int n = 0;
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) n += __popc(__ballot_sync(0xffffffffu, chunk_sum[32 * i + lane] <= step));
      return n - 1;
    };
    const int first = chunk_of(here);
    const long long first_sum = chunk_sum[first];
    if (per > 1) {   // not all of them fit: from the CTA's first one on
      b_seen = chunk_of(begin_of(worker - warp)) * per;
      for (int i = threadIdx.x; i < kSeen && b_seen + i < p.B; i += kThreads)
        seen[i] = make_int2(p.c.start[b_seen + i], kv4_count(p.c, b_seen + i, p.T));
    }
    fence_async_smem();   // the first copies go where chunk_sum was
    __syncthreads();
    if (lane == 0 && !p.join_units) p.joins[worker].parts = 0;   // unless a unit goes on behind the range
    left = (int)(begin_of(worker + 1) - here);
    if (left == 0) return;
    long long rem = here - first_sum;   // steps behind the first one of sequence at.b
    at.b = first * per;
    Reach r = reach(at.b);
    while (rem >= r.steps * p.units_per_seq && at.b < p.B - 1) {
      rem -= r.steps * p.units_per_seq;
      r = reach(++at.b);
    }
    rem = min(rem, r.steps * p.units_per_seq - 1);   // nothing, unless lengths change under the call
    const unsigned u = (unsigned)((unsigned long long)rem / (unsigned)r.steps);
    at_step = (int)(rem - (long long)u * r.steps);
    at.h = (int)(u / (unsigned)p.row_tiles);
    at.tile = (int)(u % (unsigned)p.row_tiles);
  }

  // ---- the producer: lane i looks up block i % KB of step kBatch k + i / KB
  const int my_step = lane / KB;
  const uint32_t my_dst = ring0 + lane % KB * Block;
  Place next = at;
  Reach next_reach = reach(at.b);
  int next_block = KB * at_step + lane;   // of the unit `next`, or as many behind it
  int page_next = -1, in_page_next = 0;
  const int per_page_shift = p.c.page_shift - 4;
  auto look_up = [&](bool there) {   // there: the step is this warp's
    page_next = -2;                  // no such block: nothing to copy
    while (next_block >= KB * next_reach.steps) {
      next_block -= KB * next_reach.steps;
      move_on(next, next_reach);
    }
    if (there && (long long)next_block * kKv4Block < next_reach.keys) {
      page_next = p.c.table[(size_t)next.b * p.c.max_pages + (size_t)(next_block >> per_page_shift)];
      if (page_next < 0) page_next = -1;
      in_page_next = (next.h << per_page_shift) + (next_block & ((1 << per_page_shift) - 1));
    }
    next_block += 32;
  };
  const uint8_t* src = nullptr;
  uint32_t bytes = 0;             // to copy: a block, or none
  uint32_t have = 0;              // which blocks of this batch exist
  // The step `ahead` steps in front of the one at hand, at place `make` of its
  // batch, goes to stage `to`.
  auto produce = [&](int make, int ahead, int to) {
    if (make == 0) {
      const bool ok = page_next >= 0 && page_next < p.c.n_pages;
      if (!ok && page_next != -2) kv4_no_page(p.c);
      bytes = ok ? Block : 0;
      src = p.c.pool + (((size_t)(ok ? page_next : 0) * p.c.Hkv << per_page_shift) + in_page_next) * (size_t)Block;
      have = __ballot_sync(0xffffffffu, ok);
      look_up(ahead + kBatch + my_step < left);
    }
    if (my_step == make) {
      mbar_arrive_expect_tx(bar0 + 8 * to, bytes);
      if (bytes != 0) bulk_load(my_dst + to * Sh::Stage, src, Block, bar0 + 8 * to);
    }
  };
  look_up(my_step < left);
#pragma unroll
  for (int i = 0; i < ST; ++i)
    if (i < left && !(i == 0 && worker == 0 && (p.debug_flags & 4) != 0)) produce(i, i, i);

  const bool no_steps = left == 0;
  const WaitCtx wc{p.wait_limit_ns, &abort_flag, p.c.status};
  const int group = p.H / p.c.Hkv;
  const long long unit_rows = (long long)group * p.T;
  uint32_t exist = 0;                          // as `have`, from the step to come on
  int take = 0, slot = 0;                      // the step's place in its batch, its stage's in the ring
  uint32_t phase = 0;
  bool alive = true;
  int flying = 0;                              // stages on their way when a wait ran out

  Reach r = reach(at.b);
  while (left > 0) {
    // ---- one unit's share
    const int s0 = at_step, s1 = r.steps - s0 < left ? r.steps : s0 + left;
    const long long row_in = (long long)at.tile * Sh::Rows;
    const long long row0 = ((long long)at.b * p.H + (long long)at.h * group) * p.T + row_in;
    const int rows = unit_rows - row_in < Sh::Rows ? (int)(unit_rows - row_in) : Sh::Rows;
    const bool begins = s0 == 0, ends = s1 == r.steps;
    const int left_then = left - (s1 - s0);
    const long long unit = ((long long)at.b * p.c.Hkv + at.h) * p.row_tiles + at.tile;
    if (!alive) {   // a wait ran out before: nothing to join
      if (!Near && begins && p.join_units && lane == 0) p.joins[unit].parts = 0;
      left = left_then;
      at_step = 0;
      move_on(at, r);
      continue;
    }

    uint32_t qb[NT][W][4];
    float f[NT][2];   // of the rows of this lane's columns
    int lim[NT][2];
    unsigned full_end = 0x7fffffffu, last_key = 0;
    const long long cap = (long long)p.c.max_pages << p.c.page_shift;
    auto limit_of = [&](int row) -> int {
      if (row >= rows) return 0;
      const int tok = (int)(((unsigned)row_in + row) % (unsigned)p.T);
      if (tok >= r.n) return 0;
      const long long e = p.causal ? r.start + tok + 1 : r.start + r.n;
      return (int)(e < 0 ? 0 : e > cap ? cap : e);
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int my_row = 8 * nt + g % (8 / C);   // a row in each of its C columns
      const int my_lim = limit_of(my_row);
      const uint4* qr = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.q) + (row0 + my_row) * D) + t;
      uint4 raw[W];
#pragma unroll
      for (int e = 0; e < W; ++e) raw[e] = my_lim > 0 ? qr[4 * e] : make_uint4(0, 0, 0, 0);
      uint32_t most = 0;
#pragma unroll
      for (int e = 0; e < W; ++e)
        most = max_abs2<BF16>(most, max_abs2<BF16>(max_abs2<BF16>(raw[e].x, raw[e].y), max_abs2<BF16>(raw[e].z, raw[e].w)));
      float top = fmaxf(fabsf(kv4_scale<BF16>((uint16_t)most)), fabsf(kv4_scale<BF16>((uint16_t)(most >> 16))));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      int ex = 14 + 127 - (int)(__float_as_uint(top) >> 23);   // top * 2^ex in [2^14, 2^15)
      ex = ex > 126 ? 126 : ex;                             // for the rest all of bf16 is exact
      // never 0: a masked score is -infinity, and stays that
      const float up = pow2(ex), back = fminf(fmaxf(p.scale_log2 * kUnit * pow2(-ex), 0x1p-149f), 3e38f);
      f[nt][0] = __shfl_sync(0xffffffffu, back, 8 * t);
      f[nt][1] = __shfl_sync(0xffffffffu, back, 8 * t + 4);
#pragma unroll
      for (int e = 0; e < W; ++e) {
        float v[8];
        const uint32_t xs[4] = {raw[e].x, raw[e].y, raw[e].z, raw[e].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = scale_half<BF16>(xs[i], 0);
          v[2 * i + 1] = scale_half<BF16>(xs[i], 1);
        }
        float even = 0.f, odd = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x_up = i & 1 ? up * 0.0625f : up;   // the codes of odd places weigh 16 times those of even ones
          qb[nt][e][i] = pack2<false>(v[i] * x_up, v[i + 4] * x_up);
          const float2 y = __half22float2(*reinterpret_cast<__half2*>(&qb[nt][e][i]));
          (i & 1 ? odd : even) += y.x + y.y;
        }
        float c = -8.f / kUnit * (even + 16.f * odd);
        c += __shfl_xor_sync(0xffffffffu, c, 1);
        c += __shfl_xor_sync(0xffffffffu, c, 2);
        const float c0 = __shfl_sync(0xffffffffu, c, 8 * t), c1 = __shfl_sync(0xffffffffu, c, 8 * t + 4);
        __syncwarp();
        less[4 * (nt * W + e)] = make_float4(c0, c1, c0, c1);   // all lanes of a column pair write the same
      }
      if (my_lim > 0) full_end = min(full_end, (unsigned)my_lim);
      last_key = max(last_key, (unsigned)my_lim);
      lim[nt][0] = __shfl_sync(0xffffffffu, my_lim, 8 * t);
      lim[nt][1] = __shfl_sync(0xffffffffu, my_lim, 8 * t + 4);
    }
    __syncwarp();
    full_end = __reduce_min_sync(0xffffffffu, full_end);
    last_key = __reduce_max_sync(0xffffffffu, last_key);

    float o[NT][W][2][4], m[NT][2], l[NT][2];
    float v_up[NT][2];   // P s_V goes in times v_up, up to kVPass
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int e = 0; e < W; ++e)
#pragma unroll
        for (int i = 0; i < 8; ++i) o[nt][e][i / 4][i % 4] = 0.f;
#pragma unroll
      for (int c = 0; c < 2; ++c) m[nt][c] = kLeast, l[nt][c] = 0.f, v_up[nt][c] = kMostUp;
    }

    for (int s = s0; s < s1; ++s, --left) {
      const uint32_t bar = bar0 + 8 * slot;
      if (!warp_all(mbar_try_wait(bar, phase))) {
        alive = warp_all(mbar_wait(bar, phase, wc));
        if (!alive) {
          flying = min(ST, left);
          break;
        }
      }
      if (take == 0) exist = have;   // the producer is at most ST steps ahead: in the same batch
      const uint32_t which = exist & ((1u << KB) - 1);
      exist >>= KB;
      const unsigned key0 = (unsigned)s * Sh::Step;
      if (which != 0 && key0 < last_key) {
        uint8_t* const base = ring + slot * Sh::Stage;
        float sc[NT][KB][4];
        uint32_t top2 = 0;   // V's scales: the largest magnitudes in even and odd groups
#pragma unroll
        for (int bk = 0; bk < KB; ++bk) {
          const uint8_t* blk = base + bk * Block;
          float sk[2][W];
          uint32_t kw[2][W];
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t raw[W];
            if constexpr (W == 4) {
              const uint4 x = reinterpret_cast<const uint4*>(blk)[half * 32 + lane];
              kw[half][0] = x.x, kw[half][1] = x.y, kw[half][2] = x.z, kw[half][3] = x.w;
              const uint4 y = reinterpret_cast<const uint4*>(blk + 16 * D)[half * 8 + g];
              raw[0] = y.x, raw[1] = y.y, raw[2] = y.z, raw[3] = y.w;
            } else {
              const uint2 x = reinterpret_cast<const uint2*>(blk)[half * 32 + lane];
              kw[half][0] = x.x, kw[half][1] = x.y;
              const uint2 y = reinterpret_cast<const uint2*>(blk + 16 * D)[half * 8 + g];
              raw[0] = y.x, raw[1] = y.y;
            }
#pragma unroll
            for (int e = 0; e < W; ++e) sk[half][e] = scale_half<BF16>(raw[e / 2], e & 1);
#pragma unroll
            for (int e = 0; e < W / 2; ++e) top2 = max_abs2<BF16>(top2, raw[W / 2 + e]);
          }
#pragma unroll
          for (int e = 0; e < W; ++e) {
            float d[NT][4];
            const uint32_t x0 = kw[0][e], x1 = kw[1][e];
            const uint32_t a0[4] = {x0 & 0x000f000fu, x1 & 0x000f000fu, x0 & 0x00f000f0u, x1 & 0x00f000f0u};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float4 c = less[4 * (nt * W + e)];
              const float c4[4] = {c.x, c.y, c.z, c.w};
              mma16816(d[nt], a0, qb[nt][e][0], qb[nt][e][1], c4);
            }
            const uint32_t y0 = __byte_perm(x0, 0, 0x4341), y1 = __byte_perm(x1, 0, 0x4341);
            const uint32_t z0 = y0 & 0x00f000f0u, z1 = y1 & 0x00f000f0u;
            const uint32_t a1[4] = {hsub2(y0, z0), hsub2(y1, z1), z0, z1};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816(d[nt], a1, qb[nt][e][2], qb[nt][e][3], d[nt]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                sc[nt][bk][i] = e == 0 ? d[nt][i] * sk[i / 2][0] : fmaf(d[nt][i], sk[i / 2][e], sc[nt][bk][i]);
          }
        }
        if (which != (1u << KB) - 1 || key0 + Sh::Step > full_end) {
          // keys that a row does not see; V's scales behind the last key may be
          // anything, and become 0
          top2 = 0;
#pragma unroll
          for (int bk = 0; bk < KB; ++bk)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              const unsigned key = key0 + 16 * bk + 8 * half + g;
              const bool there = (which >> bk & 1u) != 0;
              uint32_t* const vs = reinterpret_cast<uint32_t*>(base + bk * Block + 16 * D) + (half * 8 + g) * W + W / 2;
#pragma unroll
              for (int e = 0; e < W / 2; ++e) {
                if (there && key < last_key)
                  top2 = max_abs2<BF16>(top2, vs[e]);
                else if (t == 0)
                  vs[e] = 0;
              }
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  if (!there || key >= (unsigned)lim[nt][c]) sc[nt][bk][2 * half + c] = -INFINITY;
            }
          fence_async_smem();   // before the next copy to this stage
          __syncwarp();
        }
        const float v_top = fmaxf(fabsf(kv4_scale<BF16>((uint16_t)top2)), fabsf(kv4_scale<BF16>((uint16_t)(top2 >> 16))));
        bool pass = false;
        float top[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            top[nt][c] = fmaxf(sc[nt][0][c], sc[nt][0][2 + c]);
#pragma unroll
            for (int bk = 1; bk < KB; ++bk) top[nt][c] = fmax3(top[nt][c], sc[nt][bk][c], sc[nt][bk][2 + c]);
            const float room = fminf(kLazy, kVPass - lg2_approx(v_top * v_up[nt][c]));
            pass = pass || fmaf(top[nt][c], f[nt][c], -m[nt][c]) > room;
          }
        if (__any_sync(0xffffffffu, pass)) {
          float most[NT][2];   // log2 of the row's largest P |s_V| in this step, P relative to a score of 0
          float fo[NT][2];     // what O's sums are multiplied by
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              const float best = quad_max(top[nt][c]);
              most[nt][c] = -INFINITY;
              fo[nt][c] = 1.f;
              if (fmaf(best, f[nt][c], -m[nt][c]) > kLazy) {   // of this row alone
                const float to = fmaf(best, f[nt][c], -kBelow), fm = ex2_approx(m[nt][c] - to);
                const float up = fminf(v_up[nt][c] * ex2_approx(to - m[nt][c]), kMostUp);
                fo[nt][c] = __fdividef(fm * up, v_up[nt][c]);   // 1, or less where v_up is at its end
                v_up[nt][c] = up;
                m[nt][c] = to;
                l[nt][c] *= fm;
              }
            }
#pragma unroll
          for (int i = 0; i < 2 * KB; ++i) {
            const uint32_t* const vs = reinterpret_cast<const uint32_t*>(base + i / 2 * Block + 16 * D) + (i % 2 * 8 + g) * W + W / 2;
            uint32_t x = vs[0];
#pragma unroll
            for (int e = 1; e < W / 2; ++e) x = max_abs2<BF16>(x, vs[e]);
            const float sv = lg2_approx(fmaxf(fabsf(kv4_scale<BF16>((uint16_t)x)), fabsf(kv4_scale<BF16>((uint16_t)(x >> 16)))));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c = 0; c < 2; ++c) most[nt][c] = fmaxf(most[nt][c], fmaf(sc[nt][i / 2][2 * (i % 2) + c], f[nt][c], sv));
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float z = quad_max(most[nt][c]) - m[nt][c];
              if (z + lg2_approx(v_up[nt][c]) > kVPass) {
                if (z > kMostV) {   // V near bf16's largest: m goes up instead
                  m[nt][c] += kLazy;
                  z -= kLazy;
                  l[nt][c] *= 0x1p-56f;
                  fo[nt][c] *= 0x1p-56f;
                }
                const float up = ex2_approx(6.f - z);
                fo[nt][c] *= __fdividef(up, v_up[nt][c]);
                v_up[nt][c] = up;
              }
#pragma unroll
              for (int i = 0; i < 2 * W; ++i) {
                o[nt][i / 2][i % 2][c] *= fo[nt][c];
                o[nt][i / 2][i % 2][2 + c] *= fo[nt][c];
              }
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          uint64_t sum = f2_pack(l[nt][0], l[nt][1]);
          const uint64_t neg = f2_pack(-m[nt][0], -m[nt][1]);
#pragma unroll
          for (int i = 0; i < 2 * KB; ++i) {
            float(&x)[4] = sc[nt][i / 2];
            float x0, x1;
            f2_unpack(f2_fma(f2_pack(x[2 * (i % 2)], x[2 * (i % 2) + 1]), f2_pack(f[nt][0], f[nt][1]), neg), x0, x1);
            const uint64_t pp = f2_pack(ex2_approx(x0), ex2_approx(x1));
            sum = f2_add(sum, pp);
            f2_unpack(f2_mul(pp, f2_pack(v_up[nt][0], v_up[nt][1])), x[2 * (i % 2)], x[2 * (i % 2) + 1]);
          }
          f2_unpack(sum, l[nt][0], l[nt][1]);
        }
        // ---- O^T += V^T P^T
#pragma unroll
        for (int bk = 0; bk < KB; ++bk) {
          const uint8_t* blk = base + bk * Block + 8 * D;
          uint32_t vw[2][W], b[NT][W / C][2];
          float sv[2][W / C];   // the scales of this lane's groups
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t* const scales = reinterpret_cast<const uint32_t*>(blk + 8 * D) + (half * 8 + g) * W + W / 2;
            if constexpr (W == 4) {
              const uint4 x = reinterpret_cast<const uint4*>(blk)[half * 32 + lane];
              vw[half][0] = x.x, vw[half][1] = x.y, vw[half][2] = x.z, vw[half][3] = x.w;
            } else {
              const uint2 x = reinterpret_cast<const uint2*>(blk)[half * 32 + lane];
              vw[half][0] = x.x, vw[half][1] = x.y;
            }
            if constexpr (W / C == 1) {
              sv[half][0] = scale_half<BF16>(scales[column_class / 2] >> (16 * (column_class & 1)), 0);
            } else if constexpr (W / C == 2) {
              const uint32_t x = scales[C == 1 ? 0 : column_class];
              sv[half][0] = scale_half<BF16>(x, 0), sv[half][1] = scale_half<BF16>(x, 1);
            } else {
              const uint2 x = *reinterpret_cast<const uint2*>(scales);
              sv[half][0] = scale_half<BF16>(x.x, 0), sv[half][1] = scale_half<BF16>(x.x, 1);
              sv[half][2] = scale_half<BF16>(x.y, 0), sv[half][3] = scale_half<BF16>(x.y, 1);
            }
          }
#pragma unroll
          for (int e = 0; e < W / C; ++e)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const float(&pr)[4] = sc[nt][bk];
              b[nt][e][0] = transpose8x8(pack2<false>(pr[0] * sv[0][e], pr[1] * sv[0][e]));
              b[nt][e][1] = transpose8x8(pack2<false>(pr[2] * sv[1][e], pr[3] * sv[1][e]));
            }
#pragma unroll
          for (int e = 0; e < W; ++e) {
            uint32_t a0[4], a1[4];
            if constexpr (C == 1) {
              // group e: elements 4g and 4g + 1, 4g + 2 and 4g + 3
              const uint32_t x0 = vw[0][e], x1 = vw[1][e], y0 = x0 >> 8, y1 = x1 >> 8;
              a0[0] = code_even(x0), a0[1] = code_odd(x0), a0[2] = code_even(x1), a0[3] = code_odd(x1);
              a1[0] = code_even(y0), a1[1] = code_odd(y0), a1[2] = code_even(y1), a1[3] = code_odd(y1);
            } else {
              // groups e / 2 and e / 2 + W / 2: element 4g + 2 (e % 2), and the one behind it
              const int sh = 8 * (e % 2);
              const uint32_t x0 = vw[0][e / 2] >> sh, x1 = vw[1][e / 2] >> sh;
              const uint32_t y0 = vw[0][(e + W) / 2] >> sh, y1 = vw[1][(e + W) / 2] >> sh;
              a0[0] = code_even(x0), a0[1] = code_even(y0), a0[2] = code_even(x1), a0[3] = code_even(y1);
              a1[0] = code_odd(x0), a1[1] = code_odd(y0), a1[2] = code_odd(x1), a1[3] = code_odd(y1);
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint32_t(&bb)[2] = b[nt][C == 1 ? e : C == 2 ? e / 2 : 0];
              mma16816(o[nt][e][0], a0, bb[0], bb[1], o[nt][e][0]);
              mma16816(o[nt][e][1], a1, bb[0], bb[1], o[nt][e][1]);
            }
          }
        }
      }
      __syncwarp();
      if (left > ST) produce((take + ST) % kBatch, ST, slot);
      phase ^= slot == ST - 1;
      slot = slot == ST - 1 ? 0 : slot + 1;
      take = (take + 1) % kBatch;
    }
    if (!alive) {
      if (!Near && begins && p.join_units && lane == 0) p.joins[unit].parts = 0;
      left = left_then;
      at_step = 0;
      move_on(at, r);
      continue;
    }

    // ---- the unit's result, or this warp's piece of it
    float* part = begins && ends ? nullptr : slot_of(p, worker, begins ? 1 : 0, Sh::Slot);
    if constexpr (Near) part = reinterpret_cast<float*>(ring);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int row = 8 * nt + (2 * t + c) % (8 / C);
        float ll = quad_sum(l[nt][c]);
        if (row >= rows) continue;
        if (lim[nt][c] == 0) ll = 0.f;   // steps that all other rows see whole do not mask this one
        const float even = ll == 0.f ? 0.f : kUnit / ll, odd = even * 0.0625f, v_down = __fdividef(1.f, v_up[nt][c]);
#pragma unroll
        for (int e = 0; e < W; e += C == 1 ? 1 : 2) {
          float4 x;
          int group = e;
          if constexpr (C == 1) {
            x = make_float4(o[nt][e][0][c], o[nt][e][0][2 + c], o[nt][e][1][c], o[nt][e][1][2 + c]);
          } else {
            // of this tile's two groups the one that this lane's columns are for
            const bool second = column_class >= C / 2;
            group = e / 2 + (second ? W / 2 : 0);
            if (C == 4 && group != column_class) continue;
            x = second ? make_float4(o[nt][e][0][2 + c], o[nt][e][1][2 + c], o[nt][e + 1][0][2 + c], o[nt][e + 1][1][2 + c])
                       : make_float4(o[nt][e][0][c], o[nt][e][1][c], o[nt][e + 1][0][c], o[nt][e + 1][1][c]);
          }
          x.x *= even, x.y *= odd, x.z *= even, x.w *= odd;
          x.x *= v_down, x.y *= v_down, x.z *= v_down, x.w *= v_down;
          const int col = 32 * group + 4 * g;
          if (part != nullptr)
            *reinterpret_cast<float4*>(part + row * D + col) = x;
          else if (p.o32)
            *reinterpret_cast<float4*>(static_cast<float*>(p.o) + (row0 + row) * D + col) = x;
          else
            *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.o) + (row0 + row) * D + col) =
                make_uint2(pack_o<BF16>(x.x, x.y), pack_o<BF16>(x.z, x.w));
        }
        if (g == 0 && column_class == 0) {
          if (part != nullptr)
            *reinterpret_cast<float2*>(part + Sh::Rows * D + 2 * row) = make_float2(m[nt][c], ll);
          else
            p.lse[row0 + row] = lse_of(m[nt][c], ll);
        }
      }
    if (!Near && begins && lane == 0 && (p.join_units || !ends)) {
      int parts = 0;
      if (!ends) {   // then this worker's range ends here, and the unit's last step lies behind it
        const long long each = split[0], more = split[1];
        const long long last = (worker + 1) * each + (worker + 1 < more ? worker + 1 : more) + (r.steps - s1) - 1;
        const long long more_end = more * (each + 1);
        parts = (int)((last < more_end ? last / (each + 1) : more + (last - more_end) / each) - worker);
      }
      p.joins[p.join_units ? unit : worker] = Kv4Join{row0, rows, (int)worker, parts};
    }
    at_step = 0;
    move_on(at, r);
  }
  if (!alive) {
    // copies in flight land before the CTA's shared memory goes
    for (; flying > 0; --flying) {
      mbar_wait_drain(bar0 + 8 * slot, phase, p.wait_limit_ns);
      phase ^= slot == ST - 1;
      slot = slot == ST - 1 ? 0 : slot + 1;
    }
  }
  if constexpr (Near) {
    if (no_steps || !alive) {   // an empty piece
      float* const part = reinterpret_cast<float*>(ring);
      for (int i = lane; i < Sh::Rows * D; i += 32) part[i] = 0.f;
      for (int i = lane; i < Sh::Rows; i += 32)
        *reinterpret_cast<float2*>(part + Sh::Rows * D + 2 * i) = make_float2(kLeast, 0.f);
    }
    join_in_cluster<BF16, D, NT, C>(p, ring_all);
  }
}

// O and LSE of the units that lie across workers.  Pieces are normalised, with
// their maximum m (in log2) and sum l beside them; a piece that saw no key has
// l = 0.  Where a unit has many pieces, records are kept by unit and a CTA of
// 256 threads joins a row of one; else they are kept for the unit that begins
// in a worker and goes on behind it, and one of 128 threads joins 128 fours of
// its elements.  Threads to spare take the pieces in turn, eight at a time in
// flight.
constexpr int kJoinThreads = 256;   // at most

// It does not let the next kernel start early: an attention kernel's CTAs that
// settle between this one's CTAs measured slower than ones that wait.
template <bool BF16, int D, int NT, int C>
__global__ void __launch_bounds__(kJoinThreads) fa_kv4_join_kernel(const Kv4FwdParams p) {
  using Sh = Shape<D, NT, C>;
  __shared__ Piece shared[kJoinThreads];
  grid_dependency_wait();
  const Kv4Join j = p.joins[blockIdx.x];
  const int first = blockIdx.y * p.join_items;
  if (j.parts == 0 || j.rows * (D / 4) <= first) return;
  // a record of this call is in range; lengths that change under the call, or a
  // workspace that another one uses at the same time, can leave others
  if (j.parts < 0 || j.parts >= p.workers || j.worker < 0 || j.worker >= p.workers - j.parts || j.rows > Sh::Rows || j.row < 0 ||
      j.row > (long long)p.B * p.H * p.T - j.rows)
    return;
  const int worker = j.worker;
  const int items = min(j.rows * (D / 4) - first, p.join_items), turns = min((int)blockDim.x / items, j.parts + 1);
  const int item = threadIdx.x % items, turn = threadIdx.x / items;
  const int row = (first + item) / (D / 4), col = 4 * ((first + item) % (D / 4));
  Piece sum{make_float4(0.f, 0.f, 0.f, 0.f), kLeast, 0.f};
  if (turn < turns) {
    constexpr int kFly = 8;
    for (int k0 = turn; k0 <= j.parts; k0 += kFly * turns) {
      float4 x[kFly];
      float2 ml[kFly];
#pragma unroll
      for (int i = 0; i < kFly; ++i) {
        const int k = k0 + i * turns;
        ml[i] = make_float2(kLeast, 0.f);
        x[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (k <= j.parts) {
          const float* part = slot_of(p, worker + k, k == 0 ? 1 : 0, Sh::Slot);
          ml[i] = *reinterpret_cast<const float2*>(part + Sh::Rows * D + 2 * row);
          x[i] = *reinterpret_cast<const float4*>(part + row * D + col);
        }
      }
      sum.add(x, ml);
    }
    shared[threadIdx.x] = sum;
  }
  __syncthreads();
  if (turn != 0) return;
  for (int k = 1; k < turns; ++k) {
    const Piece& other = shared[k * items + item];
    const float4 x[1] = {other.o};
    const float2 ml[1] = {make_float2(other.m, other.l)};
    sum.add(x, ml);
  }
  store_result<BF16>(p, sum, j.row + row, D, col);
}

constexpr int kMaxSms = 160;
// Most keys a warp for which a unit gets a cluster.  Clusters are faster where
// units are many or short, the other division where a few long ones leave it
// the whole GPU; no bound on this number alone is right for all (us in clusters,
// in the other division; keys a warp):
//   d = 128, 4 rows, 8 key heads: 1 sequence of 1000 (31) 8.4, 9.9; of 4096 (128)
//     10.4, 11.2; of 8192 (256) 13.1, 12.4; of 16384 (512) 18.4, 16.0; 4 of 12000
//     (375) 23.8, 21.0; 16 of up to 2000 14.4, 18.2; of 4096 (341) 22.5, 25.6; of
//     5500 (458) 28.8, 32.3; of up to 9000 (750) 33.9, 28.7
//   d = 64, 12 heads of one row: 8 of 1024 8.7, 11.3; of 6000 (300) 16.8, 18.5; of
//     9500 (475) 22.4, 22.8
//   d = 64, 384 rows a key head, 1 of 6000 (375) 24.0, 28.2; of 7800 (487) 28.4, 32.3
constexpr int kNear = 512;

// Lets a kernel have its dynamic shared memory, once per device.
template <typename Kernel>
cudaError_t prepare(Kernel* kern, size_t smem, std::atomic<unsigned long long>* done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if ((done->load(std::memory_order_relaxed) & bit) != 0) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e == cudaSuccess) done->fetch_or(bit, std::memory_order_relaxed);
  return e;
}

template <bool BF16, int D, int NT, int C>
cudaError_t launch(Kv4FwdParams p, void* workspace, int sms, cudaStream_t st) {
  using Sh = Shape<D, NT, C>;
  static std::atomic<unsigned long long> near_done{0}, far_done{0};
  cudaError_t e;
  const long long rows = (long long)(p.H / p.c.Hkv) * p.T;
  p.row_tiles = (int)((rows + Sh::Rows - 1) / Sh::Rows);
  p.units_per_seq = (long long)p.c.Hkv * p.row_tiles;
  const long long units = p.B * p.units_per_seq;

  // Few and short units: a cluster each.  The largest cluster that has a step
  // for each warp and leaves an eighth of the GPU's places free (a cluster's
  // CTAs lie in one of its parts, so the last places do not fill: 144 units of
  // 1000 keys, d = 64, take 10.3 us in clusters of 3 and 14.4 in clusters of 4),
  // while no warp gets more than kNear keys.  Lengths are on the device, so all
  // this goes by the table's room for them: under a table for 131072 positions
  // one sequence of 1000 keys takes 10.0 us instead of 8.4.
  const long long most = (((long long)p.c.max_pages << p.c.page_shift) + Sh::Step - 1) / Sh::Step;   // steps of a unit
  const long long places = (long long)sms * Sh::CtasPerSm * 7 / 8;
  int cluster = 8;
  while (cluster > 1 && (units * cluster > places || (cluster - 1) * kWarps >= most)) --cluster;
  if (units * cluster <= places && most <= (long long)cluster * kWarps * (kNear / Sh::Step)) {
    p.cluster = cluster;
    auto kern = fa_kv4_fwd_kernel<BF16, D, NT, C, true>;
    if ((e = prepare(kern, Sh::Smem, &near_done)) != cudaSuccess) return e;
    return launch_chained_clusters(kern, dim3((unsigned)(units * cluster)), dim3(kThreads), Sh::Smem, st, cluster, p);
  }

  const int grid = (sms < kMaxSms ? sms : kMaxSms) * Sh::CtasPerSm;
  p.workers = grid * kWarps;
  // Few rows in all, and so many pieces to each: a row to a CTA of the joining
  // kernel.  Else a CTA to each worker's last unit.  us by row and by worker, of
  // rows in all: d = 128, 64 rows 54.5, 75.5; 256 90, 97; 512 114, 117; 768 108,
  // 108; 1024 109.8, 108.0; 1536 112.3, 108.0; 192 units of 16 rows 50.9, 41.7.  d = 64: 512 74.0, 76.0; 576 58.6, 59.5; 1024 72.8, 70.7; 1536 in units of
  // one row 76.4, 77.3.
  p.join_units = units * Sh::Rows <= 4ll * sms;
  p.join_items = p.join_units ? D / 4 : 128;
  p.joins = static_cast<Kv4Join*>(workspace);
  p.partials = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sizeof(Kv4Join) * kMaxSms * kWarps * 4);
  auto kern = fa_kv4_fwd_kernel<BF16, D, NT, C, false>;
  if ((e = prepare(kern, Sh::Smem, &far_done)) != cudaSuccess) return e;
  if ((e = launch_chained(kern, dim3(grid), dim3(kThreads), Sh::Smem, st, p)) != cudaSuccess) return e;
  const dim3 join_grid(p.join_units ? (unsigned)units : (unsigned)p.workers,
                       (unsigned)((Sh::Rows * D / 4 + p.join_items - 1) / p.join_items));
  return launch_chained(fa_kv4_join_kernel<BF16, D, NT, C>, join_grid, dim3(p.join_units ? kJoinThreads : 128),
                        0, st, p);
}

}  // namespace

// Query rows that share a key head go in tiles of 8 columns, two or four columns
// to a row where few do.  64 sequences of up to 8192 keys, us with four, two and
// one column a row: d = 128, 1 row 65.2, 66.7, 68.8; 2 rows 66.3, 68.3, 70.2; 4 rows
// 68.7 with two and 70.1 with one; d = 64, 2 rows 46.4 and 47.0, 4 rows 47.3 and 47.7.
// Two tiles a unit where more than 8 rows do.  24 sequences of up to 5000 keys,
// us with two tiles and with one: d = 128, 9 rows 38.9, 40.3; 16 rows 41.1, 41.7;
// d = 64, 9 rows 26.9, 27.3; 16 rows 28.3, 28.1; two sequences of 3000 keys and 384
// rows, d = 64, 15.4, 18.2.  One tile is the better one where 17 to 24 rows do not
// fill the second pair (24 rows: 60.9, 54.2; d = 64 39.8, 35.8) and for a short
// sequence alone (1000 keys, 16 rows 11.4, 9.0).  (Four, where registers allow
// them at d = 64, lost: 18.4 against 14.8 us for two sequences of 3000 keys and
// 384 rows a head.)
template <typename F>
static auto kv4_variant(int d, long long rows, F&& f) {
  if (d == 128) {
    if (rows <= 2) return f.template operator()<128, 1, 4>();
    if (rows <= 4) return f.template operator()<128, 1, 2>();
    if (rows <= 8) return f.template operator()<128, 1, 1>();
    return f.template operator()<128, 2, 1>();
  }
  if (rows <= 4) return f.template operator()<64, 1, 2>();
  if (rows <= 8) return f.template operator()<64, 1, 1>();
  return f.template operator()<64, 2, 1>();
}

namespace {

struct Workspace {
  template <int D, int NT, int C>
  size_t operator()() const {
    return sizeof(Kv4Join) * kMaxSms * kWarps * 4 +
           (size_t)kMaxSms * Shape<D, NT, C>::CtasPerSm * kWarps * 2 * Shape<D, NT, C>::Slot * 4;
  }
};

struct Launch {
  bool bf16;
  const Kv4FwdParams& p;
  void* workspace;
  int sms;
  cudaStream_t st;

  template <int D, int NT, int C>
  cudaError_t operator()() const {
    return bf16 ? launch<true, D, NT, C>(p, workspace, sms, st) : launch<false, D, NT, C>(p, workspace, sms, st);
  }
};

}  // namespace

size_t kv4_fwd_workspace(int d, long long rows) { return kv4_variant(d, rows, Workspace{}); }

cudaError_t launch_kv4_fwd(bool bf16, int d, const Kv4FwdParams& p, void* workspace, int sms, cudaStream_t st) {
  return kv4_variant(d, (long long)(p.H / p.c.Hkv) * p.T, Launch{bf16, p, workspace, sms, st});
}

}  // namespace fa
