// Training side of the expert path: the gated activation with its 8-bit
// checkpoint, its backward pass, and the gradient of the combine (gfx950,
// wave64).  A few operations per byte each: HBM bounds all three.
#include "epdc_device.h"
#include "expert_launch.h"

namespace epdc {

namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int64_t max_blocks(int threads) { return int64_t(UINT32_MAX) / threads; }

// One workgroup of `threads` per item; grids beyond the limit of 2^32 - 1
// work-items go out as several launches, each told its first item.
template <typename Launch>
void for_each_launch(int64_t items, int threads, Launch launch) {
  const int64_t most = max_blocks(threads);
  for (int64_t i0 = 0; i0 < items; i0 += most)
    launch(i0, unsigned(items - i0 < most ? items - i0 : most));
}

__device__ __forceinline__ void unpack8(u32x4 v, float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
}

__device__ __forceinline__ u32x4 pack8(const float (&f)[8]) {
  return u32x4{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
               pack_bf16x2(f[6], f[7])};
}

// 1 / (1 + exp(-g)): exp on the hardware's base-2 exponential, relative error
// about |g| * 2^-23, and a reciprocal within one unit in the last place.  The
// reciprocal instruction flushes results below 2^-126, so it takes a quarter of
// the sum; the product with 1/4 keeps subnormals.  Past |g| = 88.7 the
// exponential is 0 or infinite and the result 1 or 0.
__device__ __forceinline__ float sigmoid(float g) {
  return 0.25f * __builtin_amdgcn_rcpf(__builtin_fmaf(__expf(-g), 0.25f, 0.25f));
}

// e4m3 codes and scale of 128 channels held by 16 lanes, 8 each: scale =
// fl32(amax * fl32(1/448)) with NaN left out of amax, codes of fl32(x /
// scale); a group of zeros has scale 0 and codes 0.  Only a lane with a NaN,
// or a group with an infinity, needs the encoder that knows NaN.  Every other
// quotient is finite and below 464, where the hardware conversion gives the
// same codes: the scale is off amax/448 by at most 2^-23 relative when normal
// and by less than 0.4 % when subnormal (amax >= 2^-133).
__device__ __forceinline__ u32x2 quantize8(u32x4 v, const float (&f)[8], float& scale) {
  u16x2 m2 = {0, 0};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    m2 = __builtin_elementwise_max(m2, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
  uint32_t mh = max(uint32_t(m2.x), uint32_t(m2.y));
  const bool lane_nan = mh > 0x7F80u;
  if (lane_nan) {
    mh = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = v[i] & 0x7FFFu, hi = (v[i] >> 16) & 0x7FFFu;
      if (lo <= 0x7F80u) mh = max(mh, lo);
      if (hi <= 0x7F80u) mh = max(mh, hi);
    }
  }
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) mh = max(mh, uint32_t(__shfl_xor(int(mh), o)));
  const float amax = __uint_as_float(mh << 16);
  scale = amax * (1.0f / 448.0f);
  if (!lane_nan && mh != 0x7F80u) {
    if (mh == 0u) return u32x2{0u, 0u};
    float q[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = f[i] / scale;
    u32x2 c;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      int w = __builtin_amdgcn_cvt_pk_fp8_f32(q[4 * j], q[4 * j + 1], 0, false);
      c[j] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(q[4 * j + 2], q[4 * j + 3], w, true));
    }
    return c;
  }
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = amax > 0.0f ? e4m3_encode(f[i] / scale) : (f[i] != f[i] ? 0x7Fu : 0u);
  return u32x2{c[0] | (c[1] << 8) | (c[2] << 16) | (c[3] << 24),
               c[4] | (c[5] << 8) | (c[6] << 16) | (c[7] << 24)};
}

__device__ __forceinline__ void dequantize8(u32x2 c, float scale, float (&f)[8]) {
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8(int(c[j]), false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8(int(c[j]), true);
    f[4 * j] = lo[0] * scale;
    f[4 * j + 1] = lo[1] * scale;
    f[4 * j + 2] = hi[0] * scale;
    f[4 * j + 3] = hi[1] * scale;
  }
}

// Rows of the call: the device's count where there is one.
__device__ __forceinline__ int64_t rows_in_use(const SwigluArgs& a) {
  if (!a.row_count) return a.rows;
  const int64_t n = a.row_count[0];
  return n < 0 ? 0 : n < a.rows ? n : a.rows;
}

// ---------------------------------------------------------------------------
// A thread takes 8 gate channels and the 8 up channels that go with them; 16
// neighbours make a 128-channel group on either side.  Consecutive threads
// read and write consecutive 16-byte pieces (8-byte ones of the codes), so
// that every wave's access is one run of memory.  Each byte moves once and no
// sum crosses a group, so nothing is staged.  HBM bounds both: 8192 rows of
// I = 2048 take 28 us (4.8 TB/s) forward and 27 us (6.2 TB/s) backward with h,
// 65536 rows 236 us (5.7 TB/s) backward.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kBlock) void swiglu_fp8_kernel(SwigluArgs a, int64_t block0) {
  const int P = a.inner >> 3;                       // pieces per half row, a multiple of 16
  const int64_t p = (block0 + blockIdx.x) * kBlock + threadIdx.x;
  const int64_t r = p / P;
  const int j = int(p - r * P);
  if (r >= rows_in_use(a)) return;                  // whole groups of 16 lanes
  const u32x4* in = static_cast<const u32x4*>(a.gate_up) + r * (2 * P);
  const u32x4 gv = in[j], uv = in[P + j];
  float g[8], u[8], h[8], gs, us;
  unpack8(gv, g);
  unpack8(uv, u);
#pragma unroll
  for (int i = 0; i < 8; ++i) h[i] = g[i] * sigmoid(g[i]) * u[i];
  const u32x2 gq = quantize8(gv, g, gs), uq = quantize8(uv, u, us);
  static_cast<u32x4*>(a.h)[r * P + j] = pack8(h);
  u32x2* q = static_cast<u32x2*>(a.q) + r * (2 * P);
  q[j] = gq;
  q[P + j] = uq;
  if ((j & 15) == 0) {
    float* s = a.scale + r * (P >> 3);
    s[j >> 4] = gs;
    s[(P + j) >> 4] = us;
  }
}

__global__ __launch_bounds__(kBlock) void swiglu_fp8_backward_kernel(SwigluArgs a, int64_t block0) {
  const int P = a.inner >> 3;
  const int64_t p = (block0 + blockIdx.x) * kBlock + threadIdx.x;
  const int64_t r = p / P;
  const int j = int(p - r * P);
  if (r >= rows_in_use(a)) return;
  const u32x2* q = static_cast<const u32x2*>(a.q) + r * (2 * P);
  const float* sc = a.scale + r * (P >> 3);
  const u32x2 gq = q[j], uq = q[P + j];
  const float gs = sc[j >> 4], us = sc[(P + j) >> 4];
  const u32x4 dv = static_cast<const u32x4*>(a.dh)[r * P + j];
  float g[8], u[8], d[8], dg[8], du[8], h[8];
  dequantize8(gq, gs, g);
  dequantize8(uq, us, u);
  unpack8(dv, d);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float s = sigmoid(g[i]);
    const float gl = g[i] * s;
    dg[i] = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
    du[i] = d[i] * gl;
    h[i] = gl * u[i];
  }
  u32x4* o = static_cast<u32x4*>(a.d_gate_up) + r * (2 * P);
  o[j] = pack8(dg);
  o[P + j] = pack8(du);
  if (a.h) static_cast<u32x4*>(a.h)[r * P + j] = pack8(h);
}

// ---------------------------------------------------------------------------
// Gradient of the combine: one workgroup per token, one 16-byte piece of the
// row per thread (rows of more than 4096 channels in several passes).  A
// thread holds its piece of dout, loads the piece of every distinct row y the
// token reads, keeps the products' sums and stores the scaled piece; the
// workgroup then adds the sums up, lanes first, waves in order.  HBM bounds
// it: 4096 tokens, K = 6, H = 4096 take 60 us (5.5 TB/s); 16384 tokens, K = 8,
// H = 7168 663 us (5.2 TB/s), with workgroups of up to 1024 threads 691.  Non-temporal reads and writes of
// rows that nothing reads again soon; plain ones took 680 to 714.
// ---------------------------------------------------------------------------
constexpr int kGradMaxBlock = 512;

template <int KMAX, bool WEIGHTED, bool DOT>
__global__ __launch_bounds__(kGradMaxBlock) void combine_backward_kernel(CombineBackwardArgs a,
                                                                         int64_t token0) {
  __shared__ float part[kGradMaxBlock / kWave][KMAX];
  const int H8 = a.H >> 3;
  const int64_t t = token0 + blockIdx.x;
  int32_t rows[KMAX];
  float c[KMAX];           // weight of the distinct row that slot k names first
  int from[KMAX];          // slot whose row slot k shares, itself if first, -1: no row
#pragma unroll
  for (int k = 0; k < KMAX; ++k) {
    rows[k] = k < a.K ? a.token_row[t * a.K + k] : -1;
    c[k] = WEIGHTED && k < a.K ? a.w[t * a.K + k] : 1.0f;
  }
#pragma unroll
  for (int k = 0; k < KMAX; ++k) {
    from[k] = rows[k] >= 0 && int64_t(rows[k]) < a.R ? k : -1;
#pragma unroll
    for (int q = k - 1; q >= 0; --q)
      if (from[k] >= 0 && from[q] == q && rows[q] == rows[k]) from[k] = q;
  }
  if (WEIGHTED) {
#pragma unroll
    for (int k = 1; k < KMAX; ++k)
#pragma unroll
      for (int q = 0; q < k; ++q)
        if (from[k] == q) c[q] += c[k];
  }
  float dot[KMAX];
#pragma unroll
  for (int k = 0; k < KMAX; ++k) dot[k] = 0.0f;
  const u32x4* y = static_cast<const u32x4*>(a.y);
  u32x4* dy = static_cast<u32x4*>(a.dy);
  for (int j = threadIdx.x; j < H8; j += int(blockDim.x)) {
    const u32x4 dv = static_cast<const u32x4*>(a.dout)[t * H8 + j];
    u32x4 v[KMAX];
    if (DOT) {
#pragma unroll
      for (int k = 0; k < KMAX; ++k)
        if (from[k] == k) v[k] = ld_stream(y + int64_t(rows[k]) * H8 + j);
    }
    float d[8];
    unpack8(dv, d);
#pragma unroll
    for (int k = 0; k < KMAX; ++k) {
      if (from[k] != k) continue;
      u32x4 o = dv;
      if (WEIGHTED) {
        float s[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) s[i] = c[k] * d[i];
        o = pack8(s);
      }
      st_stream(dy + int64_t(rows[k]) * H8 + j, o);
      if (DOT) {
        float f[8];
        unpack8(v[k], f);
#pragma unroll
        for (int i = 0; i < 8; ++i) dot[k] = __builtin_fmaf(f[i], d[i], dot[k]);
      }
    }
  }
  if (!DOT) return;
#pragma unroll
  for (int k = 0; k < KMAX; ++k) {
    if (from[k] != k) continue;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) dot[k] += __shfl_xor(dot[k], o);
    if (lane_id() == 0) part[wave_id()][k] = dot[k];
  }
  __syncthreads();
  const int waves = int(blockDim.x) / kWave;
#pragma unroll
  for (int k = 0; k < KMAX; ++k) {
    if (int(threadIdx.x) != k || k >= a.K) continue;
    float s = 0.0f;
    if (from[k] >= 0)
      for (int w = 0; w < waves; ++w) s += part[w][from[k]];
    a.dw[t * a.K + k] = s;
  }
}

template <int KMAX>
void launch_combine_backward_k(const CombineBackwardArgs& a, hipStream_t s) {
  const int64_t H8 = a.H >> 3;
  const int64_t passes = (H8 + kGradMaxBlock - 1) / kGradMaxBlock;
  const int threads = int(((H8 + passes - 1) / passes + kWave - 1) / kWave) * kWave;
  for_each_launch(a.T, threads, [&](int64_t t0, unsigned g) {
    if (a.dw)
      combine_backward_kernel<KMAX, true, true><<<g, threads, 0, s>>>(a, t0);
    else if (a.w)
      combine_backward_kernel<KMAX, true, false><<<g, threads, 0, s>>>(a, t0);
    else
      combine_backward_kernel<KMAX, false, false><<<g, threads, 0, s>>>(a, t0);
  });
}

}  // namespace

hipError_t launch_swiglu_fp8(const SwigluArgs& a, hipStream_t s) {
  const int64_t blocks = (a.rows * (a.inner >> 3) + kBlock - 1) / kBlock;
  for_each_launch(blocks, kBlock, [&](int64_t b0, unsigned g) {
    swiglu_fp8_kernel<<<g, kBlock, 0, s>>>(a, b0);
  });
  return hipGetLastError();
}

hipError_t launch_swiglu_fp8_backward(const SwigluArgs& a, hipStream_t s) {
  const int64_t blocks = (a.rows * (a.inner >> 3) + kBlock - 1) / kBlock;
  for_each_launch(blocks, kBlock, [&](int64_t b0, unsigned g) {
    swiglu_fp8_backward_kernel<<<g, kBlock, 0, s>>>(a, b0);
  });
  return hipGetLastError();
}

hipError_t launch_combine_backward(const CombineBackwardArgs& a, hipStream_t s) {
  if (a.K <= 2)
    launch_combine_backward_k<2>(a, s);
  else if (a.K <= 4)
    launch_combine_backward_k<4>(a, s);
  else if (a.K <= 8)
    launch_combine_backward_k<8>(a, s);
  else
    launch_combine_backward_k<16>(a, s);
  return hipGetLastError();
}

}  // namespace epdc
