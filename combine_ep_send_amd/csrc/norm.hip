// RMS norm with the residual's addition and an 8-bit output, and its gradient
// (gfx950, wave64).  A few operations a byte: HBM bounds both.
#include "router_device.h"
#include "router_launch.h"

namespace epdc {

namespace {

constexpr int kNormMaxWaves = kNormMaxThreads / kWave;
constexpr int64_t kNormMaxGrid = 1 << 20;       // rows past it come round again

template <typename F>
__device__ __forceinline__ F wave_sum(F v) {
  v += partner<0>(v);
  v += partner<1>(v);
  v += partner<2>(v);
  v += partner<3>(v);
  v += partner<4>(v);
  return v + partner<5>(v);
}

// Sum over the workgroup, the same in every thread: lanes first, then waves in
// order.  `part` alternates between two rows from one call to the next, so that
// one barrier a call is enough.
template <typename F>
__device__ __forceinline__ F block_sum(F v, F* part) {
  v = wave_sum(v);
  const int waves = int(blockDim.x) / kWave;
  if (waves == 1) return v;
  if (lane_id() == 0) part[wave_id()] = v;
  __syncthreads();
  F s = 0;
  for (int w = 0; w < waves; ++w) s += part[w];
  return s;
}

// 1 / sqrt(x), x >= 0: the hardware's estimate and two of Newton's steps, which 0 and
// infinity would turn into NaN.
__device__ __forceinline__ double inverse_root(double x) {
  const double r = __builtin_amdgcn_rsq(x);
  if (!(x > 0.0 && x < INFINITY)) return r;
  const double h = 0.5 * x;
  const double s = __builtin_fma(r, __builtin_fma(-h * r, r, 0.5), r);
  return __builtin_fma(s, __builtin_fma(-h * s, s, 0.5), s);
}

// Rows are written with non-temporal stores (16384 rows of 4096 channels with a
// residual: forward 95 -> 79 us, backward 106 -> 102) and, where a call's inputs are
// too large for the cache to hold any of, read with non-temporal loads (NT: 16384
// rows of 7168, backward 173 -> 161 us, forward with codes 200 -> 194; inputs that
// the 256 MB of the Infinity Cache can hold are read slower so: 16384 rows of 4096,
// forward 79 -> 89).
template <bool NT>
__device__ __forceinline__ u32x4 fetch(const u32x4* p) {
  if constexpr (NT) return ld_stream(p);
  return *p;
}

// Eight weights of piece j.
template <bool W32>
__device__ __forceinline__ void load_weight(const void* weight, int j, float (&w)[8]) {
  if constexpr (W32) {
    const u32x4 lo = static_cast<const u32x4*>(weight)[2 * j];
    const u32x4 hi = static_cast<const u32x4*>(weight)[2 * j + 1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      w[i] = __uint_as_float(lo[i]);
      w[4 + i] = __uint_as_float(hi[i]);
    }
  } else {
    unpack8(static_cast<const u32x4*>(weight)[j], w);
  }
}

// e4m3 codes and scale of 128 values held by 16 lanes, 8 each, in 64 bits (v; y: the
// same as fp32): the rules of the dispatch's fp8 rows, scale and quotient rounded once.
// Scaled values lie on the border of two codes about once in 10^4, where the scale's
// rounding decides: with the largest value rounded to fp32 before its division, 26 % of
// the scales and one code in 20000 came out as the neighbour.  v / scale is v times
// 1 / scale in 64 bits, one division for the lane.  NaN is left out of amax; only a lane
// with one, or a group with an infinity, needs the encoder that knows NaN.  A quotient
// passes 448 by 2^-24 of it, or by more where the scale is subnormal; past 464 the
// conversion instruction gives NaN, so the quotients are clamped first, which is the
// saturation the codes call for.
__device__ __forceinline__ u32x2 quantize_group(const double (&v)[8], const float (&y)[8],
                                                bool pow2, float& scale) {
  double m = 0.0;
  float sum = 0.0f;                        // NaN where a value is (or infinities cancel)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    m = fmax(m, fabs(v[i]));
    sum += y[i];
  }
  m = fmax(m, partner<0>(m));
  m = fmax(m, partner<1>(m));
  m = fmax(m, partner<2>(m));
  m = fmax(m, partner<3>(m));
  // m / 448: the product with the inverse, and what is left of m
  const double part = m * (1.0 / 448.0);
  scale = m < INFINITY
              ? float(__builtin_fma(__builtin_fma(-448.0, part, m), 1.0 / 448.0, part))
              : INFINITY;
  if (pow2) scale = pow2_ceil(scale);
  if (sum == sum && m < INFINITY) {
    if (scale == 0.0f) return u32x2{0u, 0u};
    const double by = inverse(double(scale));
    float t[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      t[i] = __builtin_amdgcn_fmed3f(float(v[i] * by), -448.0f, 448.0f);
    u32x2 c;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int w = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * j], t[4 * j + 1], 0, false);
      c[j] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(t[4 * j + 2], t[4 * j + 3], w, true));
    }
    return c;
  }
  const double by = 1.0 / double(scale);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = scale > 0.0f ? e4m3_encode(float(v[i] * by)) : (v[i] != v[i] ? 0x7Fu : 0u);
  return u32x2{c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24),
               c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24)};
}

// ---------------------------------------------------------------------------
// Forward: one workgroup a row, the row in registers between the sum of squares
// and the output, so that every byte moves once.  The squares of two neighbours add up
// in fp32, the rest of the row's sum in 64 bits, as are the values that become codes
// (Q): of 117 million codes about 35 then are not those of 64 bits throughout (eight
// neighbours: 590, at 169 instead of 170 us; all squares in 64 bits: none, at 177).  A
// value that goes to bf16 alone is in fp32.  16384 rows of 7168 channels with residual and
// codes: 170 to 195 us (1061 MB, 5.4 to 6.2 TB/s).  A thread's pieces lie a workgroup
// apart: consecutive threads move consecutive 16-byte pieces, and 16 neighbours hold a
// 128-channel group.
// ---------------------------------------------------------------------------
template <int PT, bool W32, bool NT, bool Q>
__global__ __launch_bounds__(kNormMaxThreads) void rms_norm_kernel(NormArgs a) {
  __shared__ double part[2][kNormMaxWaves];
  const int H8 = a.H >> 3, n = int(blockDim.x);
  const double by_h = 1.0 / double(a.H);
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const u32x4* x = static_cast<const u32x4*>(a.x) + t * H8;
    u32x4 v[PT], r[PT];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const int j = i * n + int(threadIdx.x);
      v[i] = u32x4{0u, 0u, 0u, 0u};
      if (j < H8) v[i] = fetch<NT>(x + j);
    }
    if (a.residual) {
      const u32x4* res = static_cast<const u32x4*>(a.residual) + t * H8;
#pragma unroll
      for (int i = 0; i < PT; ++i) {
        const int j = i * n + int(threadIdx.x);
        r[i] = u32x4{0u, 0u, 0u, 0u};
        if (j < H8) r[i] = fetch<NT>(res + j);
      }
      u32x4* ro = static_cast<u32x4*>(a.residual_out) + t * H8;
#pragma unroll
      for (int i = 0; i < PT; ++i) {
        const int j = i * n + int(threadIdx.x);
        float f[8], g[8];
        unpack8(v[i], f);
        unpack8(r[i], g);
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] += g[k];
        v[i] = pack8(f);                    // the norm is of the row as it is kept
        if (j < H8) st_stream(ro + j, v[i]);
      }
    }
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      float f[8];
      unpack8(v[i], f);
#pragma unroll
      for (int k = 0; k < 8; k += 2)
        sum += double(__builtin_fmaf(f[k + 1], f[k + 1], f[k] * f[k]));
    }
    sum = block_sum(sum, part[turn]);
    // Squares that fp32 does not hold are taken once more in 64 bits: below 2^-100 for the
    // row (its additions are off by up to 2^-150 each, by 2^-135 in all) or infinite.  The
    // same in the whole workgroup.
    const double all_eps = double(a.H) * double(a.eps);
    if (!(sum + all_eps >= 0x1p-100 && sum < INFINITY)) {
      turn ^= 1;
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < PT; ++i) {
        // unpacked anew, or the floats would take registers up to here in every row
        asm volatile("" : "+v"(v[i]));
        float f[8];
        unpack8(v[i], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) sum = __builtin_fma(double(f[k]), double(f[k]), sum);
      }
      sum = block_sum(sum, part[turn]);
    }
    const double rstd = inverse_root((sum + all_eps) * by_h);
    if (a.rstd && threadIdx.x == 0) a.rstd[t] = float(rstd);
    // without codes y is in fp32; the least rows' rstd, up to 2^141, is past it
    const float lift = rstd > 0x1p120 ? 0x1p21f : 1.0f;
    const float rstd32 = float(rstd > 0x1p120 ? rstd * 0x1p-21 : rstd);
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const int j = i * n + int(threadIdx.x);
      if (j >= H8) continue;                // whole groups of 16 lanes where there are codes
      float f[8], w[8];
      unpack8(v[i], f);
      load_weight<W32>(a.weight, j, w);
      double y[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if constexpr (Q) {
          y[k] = double(f[k]) * rstd * double(w[k]);
          f[k] = float(y[k]);
        } else {
          f[k] = f[k] * lift * rstd32 * w[k];
        }
      }
      if (a.out) st_stream(static_cast<u32x4*>(a.out) + t * H8 + j, pack8(f));
      if constexpr (Q) {
        float scale;
        static_cast<u32x2*>(a.q)[t * H8 + j] = quantize_group(y, f, a.pow2, scale);
        if ((j & 15) == 0) a.scale[t * (H8 >> 4) + (j >> 4)] = scale;
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Backward: a workgroup takes rows in turn and keeps its sums of the weight's
// gradient in registers; they go out as one row of partial sums a workgroup,
// which a second launch adds up in order.  16384 rows of 4096 channels with the
// residual's gradient: 98 us (537 MB, 5.5 TB/s) and 7 us to add up.
// ---------------------------------------------------------------------------
template <int PT, bool W32, bool NT>
__global__ __launch_bounds__(kNormMaxThreads) void rms_norm_backward_kernel(NormArgs a) {
  __shared__ float part[2][kNormMaxWaves];
  const int H8 = a.H >> 3, n = int(blockDim.x);
  // eight pieces leave the registers no room for the weights
  constexpr bool kHold = PT < 8;
  float w[kHold ? PT : 1][8], dw[PT][8];
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    const int j = i * n + int(threadIdx.x);
#pragma unroll
    for (int k = 0; k < 8; ++k) dw[i][k] = 0.0f;
    if (!kHold) continue;
#pragma unroll
    for (int k = 0; k < 8; ++k) w[i][k] = 0.0f;
    if (j < H8) load_weight<W32>(a.weight, j, w[i]);
  }
  auto weights = [&](int i) -> float (&)[8] {
    if constexpr (!kHold) {
      const int j = i * n + int(threadIdx.x);
      load_weight<W32>(a.weight, j < H8 ? j : 0, w[0]);
      return w[0];
    } else {
      return w[i];
    }
  };
  int turn = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x, turn ^= 1) {
    const u32x4* s = static_cast<const u32x4*>(a.x) + t * H8;
    const u32x4* dy = static_cast<const u32x4*>(a.dy) + t * H8;
    const u32x4* dr = static_cast<const u32x4*>(a.residual) + t * H8;
    u32x4 sv[PT], dv[PT], rv[kHold ? PT : 1];
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const int j = i * n + int(threadIdx.x);
      sv[i] = dv[i] = rv[kHold ? i : 0] = u32x4{0u, 0u, 0u, 0u};
      if (j < H8) {
        sv[i] = fetch<NT>(s + j);
        dv[i] = fetch<NT>(dy + j);
        if (kHold && a.residual) rv[i] = fetch<NT>(dr + j);
      }
    }
    const float rstd = a.rstd[t];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      float f[8], d[8];
      const float(&wi)[8] = weights(i);
      unpack8(sv[i], f);
      unpack8(dv[i], d);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float m = f[k] * rstd;
        dw[i][k] = __builtin_fmaf(d[k], m, dw[i][k]);
        sum = __builtin_fmaf(d[k] * wi[k], m, sum);
      }
    }
    const float mean = block_sum(sum, part[turn]) / float(a.H);
    u32x4* dx = static_cast<u32x4*>(a.out) + t * H8;
#pragma unroll
    for (int i = 0; i < PT; ++i) {
      const int j = i * n + int(threadIdx.x);
      if (j >= H8) continue;
      float f[8], d[8], r[8];
      const float(&wi)[8] = weights(i);
      if (!kHold && a.residual) rv[0] = fetch<NT>(dr + j);
      unpack8(sv[i], f);
      unpack8(dv[i], d);
      unpack8(rv[kHold ? i : 0], r);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float v = rstd * (d[k] * wi[k] - f[k] * rstd * mean);
        d[k] = a.residual ? v + r[k] : v;
      }
      st_stream(dx + j, pack8(d));
    }
  }
  if (!a.dweight) return;
  u32x4* p = reinterpret_cast<u32x4*>(a.part) + int64_t(blockIdx.x) * (2 * H8);
#pragma unroll
  for (int i = 0; i < PT; ++i) {
    const int j = i * n + int(threadIdx.x);
    if (j >= H8) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      p[2 * j + h] = u32x4{__float_as_uint(dw[i][4 * h]), __float_as_uint(dw[i][4 * h + 1]),
                           __float_as_uint(dw[i][4 * h + 2]), __float_as_uint(dw[i][4 * h + 3])};
  }
}

template <int PT, bool W32>
void launch_norm_pt(const NormArgs& a, bool backward, unsigned g, int threads, hipStream_t s) {
  const bool nt = norm_streams(a.T, a.H, (backward ? 2 : 1) + (a.residual ? 1 : 0));
  if (backward && nt)
    rms_norm_backward_kernel<PT, W32, true><<<g, threads, 0, s>>>(a);
  else if (backward)
    rms_norm_backward_kernel<PT, W32, false><<<g, threads, 0, s>>>(a);
  else if (a.q && nt)
    rms_norm_kernel<PT, W32, true, true><<<g, threads, 0, s>>>(a);
  else if (a.q)
    rms_norm_kernel<PT, W32, false, true><<<g, threads, 0, s>>>(a);
  else if (nt)
    rms_norm_kernel<PT, W32, true, false><<<g, threads, 0, s>>>(a);
  else
    rms_norm_kernel<PT, W32, false, false><<<g, threads, 0, s>>>(a);
}

template <bool W32>
void launch_norm_w(const NormArgs& a, bool backward, unsigned g, hipStream_t s) {
  const NormShape n = norm_shape(a.H);
  if (n.pieces == 1)
    launch_norm_pt<1, W32>(a, backward, g, n.threads, s);
  else if (n.pieces == 2)
    launch_norm_pt<2, W32>(a, backward, g, n.threads, s);
  else if (n.pieces == 4)
    launch_norm_pt<4, W32>(a, backward, g, n.threads, s);
  else
    launch_norm_pt<8, W32>(a, backward, g, n.threads, s);
}

void launch_norm(const NormArgs& a, bool backward, unsigned g, hipStream_t s) {
  if (a.w32)
    launch_norm_w<true>(a, backward, g, s);
  else
    launch_norm_w<false>(a, backward, g, s);
}

}  // namespace

hipError_t launch_rms_norm(const NormArgs& a, hipStream_t s) {
  launch_norm(a, false, unsigned(a.T < kNormMaxGrid ? a.T : kNormMaxGrid), s);
  return hipGetLastError();
}

hipError_t launch_rms_norm_backward(const NormArgs& a, hipStream_t s) {
  const int g = norm_groups(a.T, a.H);
  if (g > 0) launch_norm(a, true, unsigned(g), s);
  if (a.dweight) launch_sum_rows(a.part, g, a.H, a.dweight, s);    // zeros for no rows
  return hipGetLastError();
}

}  // namespace epdc
