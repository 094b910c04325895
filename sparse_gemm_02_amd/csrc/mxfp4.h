// Layouts of 4-bit floating point operands, shared by their packing and the product.
#pragma once
#include "common.h"

namespace slope {

constexpr uint32_t kMxBad = 255;                     // the scale of a block with an infinity or a NaN

// A row of K values: 64 bytes of codes for each 128 of them, 16 bytes of scales for each
// 512 (so that four stages' scales of a row are one aligned load).
__host__ __device__ constexpr int64_t mx_code_bytes(int64_t K) { return cdiv(K, 128) * 64; }
__host__ __device__ constexpr int64_t mx_scale_bytes(int64_t K) { return cdiv(K, 512) * 16; }

// Chunk (t, s) of a 2:4 weight: rows 64t .. 64t+63, dense columns 128s .. 128s+127,
// four blocks a row, at (t * stages + s) * kMxChunkBytes:
//   for block pairs h = 0 (blocks 0, 1) and 1 (blocks 2, 3), 16 bytes a row: of each
//   block the word of its groups' first kept codes and that of the second ones;
//   from kMxMaskAt on for h = 0 and 1, 8 bytes a row: of each block the word of kept
//   positions (nibble g, bit p: value 4g + p is kept);
//   from kMxScaleAt on 4 bytes a row: the blocks' scales.
constexpr int kMxRows = 64, kMxCols = 128;
constexpr int kMxMaskAt = kMxRows * 32, kMxScaleAt = kMxMaskAt + kMxRows * 16, kMxChunkBytes = kMxScaleAt + kMxRows * 4;

// Bit 0 of each nibble to all four: times 15, in 16-bit halves.
__device__ __forceinline__ uint32_t wide_nibbles(uint32_t bits) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, (u16x2)(__builtin_bit_cast(u16x2, bits) * u16x2{15, 15}));
}
// The four words of a dense block from its kept codes and masks k of the four positions.  Of
// two kept positions the lower one has the first code: position 0 is the first, 3 the
// second; 1 is the second if 0 is kept, 2 the first if 3 is.
__device__ __forceinline__ u32x4 expanded(uint32_t first, uint32_t second, u32x4 k) {
  return u32x4{first & k[0], k[1] & ((second & k[0]) | (first & ~k[0])), k[2] & ((first & k[3]) | (second & ~k[3])), second & k[3]};
}
// ... and from its kept positions (17 operations).
__device__ __forceinline__ u32x4 expand24(uint32_t first, uint32_t second, uint32_t kept) {
  return expanded(first, second, u32x4{wide_nibbles(kept & 0x11111111u), wide_nibbles((kept >> 1) & 0x11111111u),
                                       wide_nibbles((kept >> 2) & 0x11111111u), wide_nibbles((kept >> 3) & 0x11111111u)});
}

}  // namespace slope
