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
