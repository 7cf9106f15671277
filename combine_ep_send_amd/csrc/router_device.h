// What the kernels before the dispatch share (gfx950, wave64).
#pragma once

#include "epdc_device.h"

namespace epdc {

// out[c] = sum over r of part[r][c], rows of `columns` floats: a workgroup takes
// 64 columns, one a lane, and its waves rows r, r + waves, ...; the waves' sums
// then add up in order.  The order depends on the sizes alone.
__global__ __launch_bounds__(1024) static void sum_rows_kernel(const float* part, int rows,
                                                               int64_t columns, float* out,
                                                               int64_t block0) {
  __shared__ float acc[16][kWave];
  const int waves = int(blockDim.x) / kWave, w = wave_id();
  const int64_t c = (block0 + blockIdx.x) * kWave + lane_id();
  float s = 0.0f;
  if (c < columns) {
    const float* p = part + c;
    int r = w;
    for (; r + 7 * waves < rows; r += 8 * waves) {
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = p[int64_t(r + i * waves) * columns];
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[i];
    }
    for (; r < rows; r += waves) s += p[int64_t(r) * columns];
  }
  acc[w][lane_id()] = s;
  __syncthreads();
  if (w != 0 || c >= columns) return;
  for (int i = 1; i < waves; ++i) s += acc[i][lane_id()];
  out[c] = s;
}

// As many waves as leave each eight rows, up to 16.
inline void launch_sum_rows(const float* part, int rows, int64_t columns, float* out,
                            hipStream_t s) {
  int waves = 1;
  while (waves < 16 && rows > 8 * waves) waves *= 2;
  for_each_launch((columns + kWave - 1) / kWave, waves * kWave, [&](int64_t b0, unsigned g) {
    sum_rows_kernel<<<g, waves * kWave, 0, s>>>(part, rows, columns, out, b0);
  });
}

}  // namespace epdc
