// nibble.cuh -- layout of a paged cache held in 4 bits.
//
// A page of one KV head is a row of blocks of 16 tokens, 18 D bytes each:
//   codes of K   [D / 32 groups][16 tokens][16 bytes]   channel 2 b of the group in the low, 2 b + 1 in the high
//                                                      four bits of byte b
//   scales of K  [8][D / 32][2] fp16                     of tokens r and r + 8, side by side
//   codes and scales of V, the same
// so a block is one contiguous copy, each group's codes are the rows of 8 x 8 matrices for
// ldmatrix as they lie (16 bytes apart: no bank is hit twice), and the scales of the two
// tokens that a lane of a 16-row product holds are one word.
#pragma once

#include "fathom_internal.cuh"

namespace fathom {

constexpr int kNibTokens = 16;   // of a block
__host__ __device__ constexpr int nib_block_bytes(int D) { return 18 * D; }
// Offsets in a block: V's part, a part's scales, the word of a group's codes and the
// scale of a token.
__host__ __device__ constexpr int nib_half(int D) { return 9 * D; }
__host__ __device__ constexpr int nib_scales(int D) { return 8 * D; }
__host__ __device__ constexpr int nib_code(int group, int token) { return group * 256 + token * 16; }
__host__ __device__ constexpr int nib_scale(int D, int group, int token) {
    return 4 * ((token & 7) * (D / 32) + group) + 2 * (token >> 3);
}
// Byte offset of the block that holds place `slot` of (page, head).
__device__ __forceinline__ int64_t nib_block(const fathom_nibble_pages &p, int page, int head, int slot) {
    return page * p.page_stride + head * p.head_stride + (int64_t)(slot / kNibTokens) * nib_block_bytes(p.D);
}

}  // namespace fathom
