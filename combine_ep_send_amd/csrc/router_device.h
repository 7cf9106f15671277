// What the kernels before the dispatch share (gfx950, wave64).
#pragma once

#include "epdc_device.h"

namespace epdc {

// out[c] = sum over r of part[r][c], rows of `columns` floats: a wave takes 64
// columns, one a lane, and rows r, r + along, ... of them, `along` waves of a
// workgroup side by side; their sums then add up in order.  The order depends on
// the sizes alone.
__global__ __launch_bounds__(1024) static void sum_rows_kernel(const float* part, int rows,
                                                               int64_t columns, float* out,
                                                               int along, int64_t block0) {
  __shared__ float acc[16][kWave];
  const int waves = int(blockDim.x) / kWave, w = wave_id();
  const int across = waves / along, r0 = w % along;
  const int64_t c = ((block0 + blockIdx.x) * across + w / along) * kWave + lane_id();
  float s = 0.0f;
  if (c < columns) {
    const float* p = part + c;
    int r = r0;
    for (; r + 7 * along < rows; r += 8 * along) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[int64_t(r + i * along) * columns];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; r < rows; r += along) s += p[int64_t(r) * columns];
  }
  if (along > 1) {
    acc[w][lane_id()] = s;
    __syncthreads();
    if (r0 != 0) return;
    for (int i = 1; i < along; ++i) s += acc[w + i][lane_id()];
  }
  if (c < columns) out[c] = s;
}

// As many waves as leave each eight rows, up to 16.
inline void launch_sum_rows(const float* part, int rows, int64_t columns, float* out,
                            hipStream_t s) {
  int along = 1;
  while (along < 16 && rows > 8 * along) along *= 2;
  const int waves = along < 4 ? 4 : along;
  const int64_t each = int64_t(waves / along) * kWave;      // columns of a workgroup
  for_each_launch((columns + each - 1) / each, waves * kWave, [&](int64_t b0, unsigned g) {
    sum_rows_kernel<<<g, waves * kWave, 0, s>>>(part, rows, columns, out, along, b0);
  });
}

}  // namespace epdc
