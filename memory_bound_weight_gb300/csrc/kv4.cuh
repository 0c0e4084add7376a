// kv4.cuh -- layout of the 4-bit paged key/value cache and the conversions its
// kernels share.
//
// A page holds page_size tokens (a multiple of 16) of every KV head: per head
// page_size / 16 blocks, each of 16 tokens of that head, contiguous:
//   K codes  8 D bytes | V codes  8 D bytes | K meta 64 D/G | V meta 64 D/G
// with one (scale, minimum) fp16 pair per token and group of G dimensions,
// meta[t][group]. A value is scale * code + minimum, code 0 .. 15.
//
// The codes lie in the order in which lanes of m16n8k16 read them, so that a
// warp takes a block from shared memory with 16-byte reads that hit every bank
// once, and no code is moved between lanes. With lane = 4 g + c:
//   K (the token is the row of the A operand, tokens g and g + 8): dimension d
//     of plane p = d / 128 (one plane of 64 when D = 64), e = d % 128: the
//     32-bit word e / 32 of lane quarter c = e % 32 / 8, nibble e % 8. The words
//     j of the four quarters are 32 consecutive dimensions, two k-steps of one
//     group.
//   V (transposed: the dimension is the row, the token the k index): token
//     t = 8 h + 2 c + b; dimension d = 64 w + 8 slot + g: nibble `slot` of the
//     lane's word (h, b, w). The words of tokens 2c and 2c + 1, merged halfword
//     by halfword, are the operand's (k, k + 1) pairs.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "device.cuh"

namespace mbw {

__host__ __device__ constexpr int kv4_block_bytes(int D, int G) { return 16 * D + 128 * (D / G); }

// Byte of token t's K word that holds dimensions 8 l .. 8 l + 7 (the word's nibble i is dimension 8 l + i).
__host__ __device__ __forceinline__ int kv4_k_word(int D, int t, int l) {
    const int span = D < 128 ? D : 128;  // dimensions of a plane
    const int p = 8 * l / span, e = l % (span / 8);
    return p * 8 * span + t * (span / 2) + (e % 4) * (span / 8) + (e / 4) * 4;
}
// Byte of token t's V word for dimensions 64 w + 8 slot + g, slot = 0 .. 7.
__host__ __device__ __forceinline__ int kv4_v_word(int D, int t, int g, int w) {
    const int q = ((t >> 3) * 2 + (t & 1)) * (D / 64) + w;
    return 8 * D + (q >> 2) * 512 + (4 * g + ((t & 7) >> 1)) * 16 + (q & 3) * 4;
}
// Byte of token t's (scale, minimum) pair of group i; v: 0 for K, 1 for V.
__host__ __device__ __forceinline__ int kv4_meta(int D, int G, int t, int i, int v) {
    return 16 * D + v * 64 * (D / G) + (t * (D / G) + i) * 4;
}

// The first position that a query at pos sees under a window; pos may lie far before 0, and the window be any.
__device__ __forceinline__ int kv4_first_seen(int pos, int window) { return window && pos + 1 > window ? pos + 1 - window : 0; }

__device__ __forceinline__ float2 kv4_pair(uint32_t m) {
    return __half22float2(*reinterpret_cast<const __half2*>(&m));
}

}  // namespace mbw
