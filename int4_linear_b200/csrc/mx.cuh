// Sizes of the microscaled 4-bit formats (see fq_mx_format in fq.h).
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/fq.h"

namespace fq {

constexpr int kMxTileRows = 128;   // rows of one scale tile
constexpr int kMxTileBlocks = 4;   // blocks along K of one scale tile
constexpr int kMxTileBytes = kMxTileRows * kMxTileBlocks;

__host__ __device__ constexpr int mx_block(int fmt) { return fmt == FQ_NVFP4 ? 16 : 32; }

// Byte of scale (row r, block b) among B blocks per row.
__host__ __device__ constexpr size_t mx_scale_offset(int r, int b, int B) {
  return (size_t(r / kMxTileRows) * (B / kMxTileBlocks) + b / kMxTileBlocks) * kMxTileBytes + (r % 32) * 16 +
         (r % kMxTileRows / 32) * 4 + b % kMxTileBlocks;
}

}  // namespace fq
