// What the kernels before the dispatch share (gfx950, wave64).
#pragma once

#include "epdc_device.h"

namespace epdc {

// The value of the partner lane at each step of a join over 2, 4, 8, 16, 32, 64
// lanes: after a step all lanes of the block hold the same, so any pairing of
// the two halves does.  Within 16 lanes by data-parallel moves.
template <int STEP>
__device__ __forceinline__ int partner(int v) {
  if constexpr (STEP == 0) return __builtin_amdgcn_update_dpp(v, v, 0xB1, 0xF, 0xF, false);
  if constexpr (STEP == 1) return __builtin_amdgcn_update_dpp(v, v, 0x4E, 0xF, 0xF, false);
  if constexpr (STEP == 2) return __builtin_amdgcn_update_dpp(v, v, 0x141, 0xF, 0xF, false);
  if constexpr (STEP == 3) return __builtin_amdgcn_update_dpp(v, v, 0x140, 0xF, 0xF, false);
  return __shfl_xor(v, 1 << STEP);
}
template <int STEP>
__device__ __forceinline__ double partner(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = uint32_t(partner<STEP>(int(uint32_t(b))));
  const uint32_t hi = uint32_t(partner<STEP>(int(uint32_t(b >> 32))));
  return __builtin_bit_cast(double, (uint64_t(hi) << 32) | lo);
}

template <int STEP>
__device__ __forceinline__ float partner(float v) {
  return __int_as_float(partner<STEP>(__float_as_int(v)));
}

// 1 / y, both in the normal range: the hardware's estimate and two of Newton's steps.
__device__ __forceinline__ double inverse(double y) {
  double r = __builtin_amdgcn_rcp(y);
  r = __builtin_fma(r, __builtin_fma(-y, r, 1.0), r);
  return __builtin_fma(r, __builtin_fma(-y, r, 1.0), r);
}

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
