// The paged MXFP4 KV cache: where a token's codes and scales sit, and how they become values.
//
// The cache is a pool of pages of P tokens (P a power of two, 16 to 256). Per page and KV head it
// holds a K chunk and then a V chunk, each of P * 17 d / 32 bytes: P rows of d / 2 code bytes, then
// P rows of nb = d / 32 scale bytes (blocks of 32 run along d, so that a single token can be added
// without touching its neighbours). Inside a chunk the bytes are interleaved so that the fragments
// of mma.m16n8k16 come out of global memory with one wide load per lane and no shuffle:
//   * K row: word w (4 bytes: 8 codes) of block b at byte w * 4 nb + 4 b. Lane c of a quad holds
//     word c of every block, i.e. a quarter of each block of its key; which of a block's 32 channels
//     meet in one k-step does not matter as long as Q is read in the same order.
//   * V row: half-word h (2 bytes: 4 codes) of block b at byte h * 2 nb + 2 b. Lane g of the eight
//     lanes that share a key holds 4 channels of every block.
//   * scale rows: the 16 tokens i of a group are ordered so that the keys of one lane are neighbours:
//     keys g and g + 8 for K, keys 2c, 2c + 1, 2c + 8, 2c + 9 for V.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>

namespace mxattn {

__host__ __device__ constexpr uint32_t cache_row_bytes(uint32_t d) { return d / 2; }
__host__ __device__ constexpr uint32_t cache_chunk_bytes(uint32_t d, uint32_t page) { return page * (d / 32) * 17u; }

// Row of token i (mod 16) among the scale rows of its 16 tokens.
__device__ __forceinline__ uint32_t k_scale_row(uint32_t i) { return (i & 7u) * 2u + (i >> 3); }
__device__ __forceinline__ uint32_t v_scale_row(uint32_t i) { return ((i & 7u) >> 1) * 4u + (i >> 3) * 2u + (i & 1u); }

// Four bytes (eight codes) -> four half2: byte j gives elements 2j (low half) and 2j + 1.
__device__ __forceinline__ void e2m1x8_to_half2(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// The words of piece p of a V row (nb = 4: half-words 2p, 2p + 1 of each block; nb = 2: half-words
// 4p .. 4p + 3) from the words that hold them, and back: both directions pair low and high halves.
__device__ __forceinline__ uint32_t lo16x2(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x5410); }
__device__ __forceinline__ uint32_t hi16x2(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }

}  // namespace mxattn
