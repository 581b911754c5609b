// Sums of columns, for a bias gradient (gfx950).  Internal header.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "mbok_device.h"

namespace mbok {

// dst[c] (+)= sum over rows of src[row][c]: bf16 rows of a gradient, or the fp32
// sums of its slices.  Small enough to run beside another kernel's last blocks.
struct ColumnSums {
  const void* src;
  int64_t ld;
  int bf16, rows, cols, accumulate;
  float* dst;
};

constexpr int kSumColumns = 32;  // columns of a block of 256 threads
inline int sum_blocks(const ColumnSums& c) { return (c.cols + kSumColumns - 1) / kSumColumns; }

// Block `block` of 256 threads: 8 rows of threads take every eighth row each, in a
// fixed order.
__device__ __forceinline__ void column_sums(const ColumnSums& c, int block) {
  __shared__ float part[8][kSumColumns];
  const int x = threadIdx.x % kSumColumns, y = threadIdx.x / kSumColumns;
  const int col = block * kSumColumns + x;
  float total = 0.f;
  if (col < c.cols) {
    if (c.bf16) {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(c.src) + col;
#pragma unroll 8
      for (int r = y; r < c.rows; r += 8) total += bf16_bits_to_f32(p[r * c.ld]);
    } else {
      const float* p = reinterpret_cast<const float*>(c.src) + col;
#pragma unroll 8
      for (int r = y; r < c.rows; r += 8) total += p[r * c.ld];
    }
  }
  part[y][x] = total;
  __syncthreads();
  if (y || col >= c.cols) return;
#pragma unroll
  for (int i = 1; i < 8; ++i) total += part[i][x];
  c.dst[col] = c.accumulate ? c.dst[col] + total : total;
}

}  // namespace mbok
