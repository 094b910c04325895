// Layouts of 4-bit floating point operands, shared by their packing and the product.
#pragma once
#include "common.h"

namespace slope {

constexpr uint32_t kMxBad = 255;                     // the scale of a block with an infinity or a NaN

// Chunk (t, s) of a 2:4 weight: rows 64t .. 64t+63, dense columns 128s .. 128s+127,
// four blocks a row, at (t * stages + s) * kMxChunkBytes:
//   for block pairs h = 0 (blocks 0, 1) and 1 (blocks 2, 3), 16 bytes a row: of each
//   block the word of its groups' first kept codes and that of the second ones;
//   from kMxMaskAt on for h = 0 and 1, 8 bytes a row: of each block the word of kept
//   positions (nibble g, bit p: value 4g + p is kept);
//   from kMxScaleAt on 4 bytes a row: the blocks' scales.
constexpr int kMxRows = 64, kMxCols = 128;
constexpr int kMxMaskAt = kMxRows * 32, kMxScaleAt = kMxMaskAt + kMxRows * 16, kMxChunkBytes = kMxScaleAt + kMxRows * 4;

// The four words of a dense block from its kept codes and positions (21 operations).
// Of two kept positions the lower one has the first code: position 0 is the first,
// 3 the second; 1 is the second if 0 is kept, 2 the first if 3 is.
__device__ __forceinline__ u32x4 expand24(uint32_t first, uint32_t second, uint32_t kept) {
  auto wide = [](uint32_t bits) { return (bits << 4) - bits; };      // bit 0 of each nibble to all four
  const uint32_t k0 = wide(kept & 0x11111111u), k1 = wide((kept >> 1) & 0x11111111u);
  const uint32_t k2 = wide((kept >> 2) & 0x11111111u), k3 = wide((kept >> 3) & 0x11111111u);
  return u32x4{first & k0, k1 & ((second & k0) | (first & ~k0)), k2 & ((first & k3) | (second & ~k3)), second & k3};
}

}  // namespace slope
