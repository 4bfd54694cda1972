// Layout of the 4-bit key/value cache, shared by the kernels that write it,
// read it back and attend to it.
//
// The pool is [n_pages][Hkv][page/16] blocks of 16 tokens, 18 D bytes each, K
// and V together so that one contiguous copy fetches all that 16 keys need:
//
//   [0,    8D)  K codes.  32-bit word ((half*8 + g)*4 + t)*W + e of key
//               half*8 + g holds the elements 32e + 8t + 0..7 (W = D/32 words
//               of one lane lie together): low half-word elements 0..3, high
//               half-word 4..7.
//   [8D,  16D)  V codes.  Word ((half*8 + r)*4 + t)*W + e holds the elements
//               32e + 4r + 0..3 of the keys half*8 + 2t (low half-word) and
//               half*8 + 2t + 1 (high half-word).
//   [16D, 18D)  scales, 16-bit, key by key: W of K, then W of V, one per 32
//               elements.
//
// These are the orders in which a warp's lanes hold the A operand of
// mma.m16n8k16 with the keys (K) and the head's elements (V) as rows: lane
// 4g + t reads its share of 16 keys with one or two vector loads, and no
// code moves between lanes.  A half-word belongs to one key, so writing a
// token touches no byte of another one.
//
// A half-word's four codes c = n + 8 are its nibbles in order.  Under the
// masks 0x000f and 0x00f0 a code is an fp16 subnormal as it stands, c 2^-24 or
// c 2^-20, which the tensor cores multiply exactly; the word shifted right by
// 8 brings the other two codes to the same places: 5 integer instructions for
// 8 codes.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "fa.h"
#include "fa_kernels.h"

namespace fa {

constexpr int kKv4Group = 32;   // elements that share a scale
constexpr int kKv4Block = 16;   // tokens of a block

__host__ __device__ constexpr int kv4_block_bytes(int d) { return 18 * d; }

// What the calls share.
struct Kv4Cache {
  uint8_t* pool;       // [n_pages][Hkv][page/16] blocks
  const int* table;    // [B][max_pages]
  const int* start;    // [B]: position of the call's first token
  const int* count;    // [B] tokens of each sequence, or null (= T)
  int n_pages;
  int page_shift;      // page = 1 << page_shift tokens
  int max_pages;
  int Hkv;
  int* status;         // device status words: of waits, of pages
};

struct Kv4Join;

struct Kv4FwdParams {
  Kv4Cache c;
  const void* q;       // [B, H, T, D] 16-bit
  void* o;             // [B, H, T, D] 16-bit, or fp32 when o32
  float* lse;          // [B, H, T]
  int B, H, T;
  float scale_log2;    // scale * log2(e)
  int causal;
  int o32;
  uint64_t wait_limit_ns;
  int debug_flags;     // bit 2: withhold one arrival (timeout test)
  // set by the launch
  int row_tiles;             // tiles of query rows a key head
  long long units_per_seq;   // Hkv * row_tiles
  int cluster;               // CTAs that share a unit, where clusters do
  int workers;               // warps of the grid, where they do not
  int join_units;            // joins go by unit, else by worker
  int join_items;            // fours of elements a CTA of the joining kernel
  Kv4Join* joins;            // [units or workers]
  float* partials;           // [workers][2] pieces of results
};

cudaError_t launch_kv4_write(bool bf16, int d, const Kv4Cache& c, const void* k, const void* v, int B, int T,
                             cudaStream_t st);
cudaError_t launch_kv4_read(bool bf16, int d, const Kv4Cache& c, void* k, void* v, int B, int N, cudaStream_t st);
// Bytes of the attention's workspace; rows = query rows that share a key head.
size_t kv4_fwd_workspace(int d, long long rows);
cudaError_t launch_kv4_fwd(bool bf16, int d, const Kv4FwdParams& p, void* workspace, int sms, cudaStream_t st);

// launch_chained in clusters of `cluster` CTAs.
template <typename... Params, typename... Args>
inline cudaError_t launch_chained_clusters(void (*kern)(Params...), dim3 grid, dim3 block, size_t smem,
                                           cudaStream_t st, int cluster, Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kern, std::forward<Args>(args)...);
}

// Tokens of sequence b in this call: count clamped to [0, T].
__device__ __forceinline__ int kv4_count(const Kv4Cache& c, int b, int T) {
  if (c.count == nullptr) return T;
  const int n = c.count[b];
  return n < 0 ? 0 : (n > T ? T : n);
}

__device__ __forceinline__ void kv4_no_page(const Kv4Cache& c) { atomicCAS(c.status + 1, 0, FA_ERR_PAGE); }

// Byte address of the block that holds position pos of sequence b, head h, or
// null (and FA_ERR_PAGE recorded) where no such block exists.
__device__ __forceinline__ uint8_t* kv4_block_of(const Kv4Cache& c, int b, int h, long long pos, int block_bytes) {
  if (pos >= 0 && pos < ((long long)c.max_pages << c.page_shift)) {
    const int pg = c.table[(size_t)b * c.max_pages + (size_t)(pos >> c.page_shift)];
    if ((unsigned)pg < (unsigned)c.n_pages) {
      const int per_page = 1 << (c.page_shift - 4);
      const int sub = (int)(pos >> 4) & (per_page - 1);
      return c.pool + (((size_t)pg * c.Hkv + h) * per_page + sub) * (size_t)block_bytes;
    }
  }
  kv4_no_page(c);
  return nullptr;
}

template <bool BF16>
__device__ __forceinline__ float kv4_scale(uint16_t u) {
  if constexpr (BF16)
    return __uint_as_float((uint32_t)u << 16);
  else
    return __half2float(__ushort_as_half(u));
}

}  // namespace fa
