// The router's logits and their gradients (gfx950, wave64): three products of
// which one side is small.  The matrix cores take bf16 and sum in fp32
// (v_mfma_f32_16x16x32_bf16); what is fp32 (the logits' gradient) takes part as
// the sum of two or three bf16 numbers.
#include "epdc_device.h"
#include "router_launch.h"

namespace epdc {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr uint32_t kOob = 0x80000000u;      // past every descriptor's range (< 2^31 bytes)

__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int64_t bytes) {
  // stride 0, 32-bit data format: offsets are bytes, checked against `bytes`
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, int(bytes), 0x00027000);
}
__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// Barrier that orders LDS alone: loads from memory stay in flight.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

struct GemmArgs {
  const void* a;                 // [parts][M][lda] bf16
  const void* b;                 // [N][ldb] bf16
  int64_t M;
  int N, K;
  int lda, ldb;                  // elements, multiples of 8
  int64_t plane;                 // elements from part to part of a
  int each;                      // stages a workgroup takes
  void* out;                     // [M][N] bf16, or fp32 [splits][M][N]
};

// ---------------------------------------------------------------------------
// out[m, n] = sum over k of A[m, k] B[n, k], A the sum of PARTS bf16 arrays.
// The rows of A go through LDS, which the waves side by side along n share; a
// wave's rows of B come straight into its registers, in a ring of D stages with
// the rows of A.  Loads go through descriptors whose range check gives zeros for
// rows and channels past the end, so nothing branches.
// LDS holds a row of a stage as 16-byte pieces, piece p at p ^ (row & 7): the
// eight rows that a read takes at once then lie in different banks.
// ---------------------------------------------------------------------------
template <int MT, int WN, int PARTS, bool BF16OUT>
__global__ __launch_bounds__(kBlock) void gemm_kernel(GemmArgs g, int64_t mb0) {
  constexpr int WK = 4 / WN, BM = 16 * MT, D = 2;
  constexpr int P = 8 * WK;                              // pieces of a row and stage
  constexpr int LOADS = (BM * P + kBlock - 1) / kBlock;  // pieces of A a thread loads, a part
  constexpr int kBuffers = 2 * PARTS * BM * P;
  constexpr int kReduce = WK > 1 ? WK * BM * WN * 64 / 4 : 0;
  __shared__ u32x4 lds[kBuffers > kReduce ? kBuffers : kReduce];
  const int lane = lane_id(), n = lane & 15, q = lane >> 4;
  const int wn = wave_id() % WN, wk = wave_id() / WN;
  const int64_t m0 = (mb0 + blockIdx.x) * BM;
  const int n0 = int(blockIdx.y) * (64 * WN);
  const int rows = int(g.M - m0 < BM ? g.M - m0 : BM);
  const int cols = g.N - n0 < 64 * WN ? g.N - n0 : 64 * WN;
  rsrc_t ar[PARTS];
#pragma unroll
  for (int p = 0; p < PARTS; ++p)
    ar[p] = make_rsrc(static_cast<const uint16_t*>(g.a) + p * g.plane + m0 * g.lda,
                      int64_t(rows) * g.lda * 2);
  const rsrc_t br = make_rsrc(static_cast<const uint16_t*>(g.b) + int64_t(n0) * g.ldb,
                              int64_t(cols) * g.ldb * 2);
  const int st0 = int(blockIdx.z) * g.each, st1 = st0 + g.each;
  u32x4 av[D][PARTS][LOADS], bv[D][4][2];
  auto load = [&](int d, int st) {
    const int left = st < st1 ? g.K - st * (64 * WK) : 0;          // channels from the stage on
    const int so = st < st1 ? st * (128 * WK) : 0;
#pragma unroll
    for (int i = 0; i < LOADS; ++i) {
      const int at = i * kBlock + int(threadIdx.x), row = at / P, piece = at % P;
      const uint32_t off = row < BM && piece * 8 < left
                               ? uint32_t(row) * uint32_t(2 * g.lda) + uint32_t(piece * 16)
                               : kOob;
#pragma unroll
      for (int p = 0; p < PARTS; ++p)
        av[d][p][i] = __builtin_amdgcn_raw_buffer_load_b128(ar[p], off, so, 0);
    }
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int piece = wk * 8 + s * 4 + q;
        const uint32_t off = piece * 8 < left
                                 ? uint32_t(wn * 64 + t * 16 + n) * uint32_t(2 * g.ldb) +
                                       uint32_t(piece * 16)
                                 : kOob;
        bv[d][t][s] = __builtin_amdgcn_raw_buffer_load_b128(br, off, so, 0);
      }
  };
  f32x4 acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int d = 0; d < D; ++d) load(d, st0 + d);
  for (int st = st0; st < st1; st += D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      u32x4* buf = lds + (d & 1) * (PARTS * BM * P);
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int at = i * kBlock + int(threadIdx.x), row = at / P, piece = at % P;
        if (row < BM) {
#pragma unroll
          for (int p = 0; p < PARTS; ++p)
            buf[(p * BM + row) * P + (piece ^ (row & 7))] = av[d][p][i];
        }
      }
      u32x4 b[4][2];
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int s = 0; s < 2; ++s) b[t][s] = bv[d][t][s];
      lds_barrier();
      load(d, st + d + D);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int p = 0; p < PARTS; ++p)
#pragma unroll
          for (int m = 0; m < MT; ++m) {
            const int row = m * 16 + n;
            const u32x4 a = buf[(p * BM + row) * P + ((wk * 8 + s * 4 + q) ^ (row & 7))];
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[m][t] = mfma(a, b[t][s], acc[m][t]);
          }
    }
  }
  const int64_t plane = int64_t(blockIdx.z) * g.M * g.N;
  auto store = [&](int row, int col, float v) {
    if (row >= rows || col >= cols) return;
    const int64_t at = (m0 + row) * g.N + n0 + col;
    if constexpr (BF16OUT)
      static_cast<uint16_t*>(g.out)[at] = uint16_t(pack_bf16x2(v, 0.0f));
    else
      static_cast<float*>(g.out)[plane + at] = v;
  };
  if constexpr (WK == 1) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          store(m * 16 + q * 4 + i, wn * 64 + t * 16 + n, acc[m][t][i]);
  } else {
    // the waves along k add up in order
    float* sum = reinterpret_cast<float*>(lds);
    lds_barrier();
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          sum[(wk * BM + m * 16 + q * 4 + i) * (64 * WN) + wn * 64 + t * 16 + n] = acc[m][t][i];
    lds_barrier();
    for (int at = int(threadIdx.x); at < BM * 64 * WN; at += kBlock) {
      float v = 0.0f;
#pragma unroll
      for (int k = 0; k < WK; ++k) v += sum[k * (BM * 64 * WN) + at];
      store(at / (64 * WN), at % (64 * WN), v);
    }
  }
}

// out[i] = sum over s of part[s][i], in order.
__global__ __launch_bounds__(kBlock) void sum_planes_kernel(const float* part, int planes,
                                                            int64_t count, float* out) {
  const int64_t step = int64_t(gridDim.x) * kBlock;
  for (int64_t i = int64_t(blockIdx.x) * kBlock + threadIdx.x; i < count; i += step) {
    float v = 0.0f;
    for (int s = 0; s < planes; ++s) v += part[s * count + i];
    out[i] = v;
  }
}

// A float as the sum of three bf16 numbers, exact where the last is no smaller
// than bf16 goes; what rounds to an infinity or is none has no further parts.
__device__ __forceinline__ void split3(float v, uint32_t (&p)[3]) {
  p[0] = pack_bf16x2(v, 0.0f) & 0xFFFFu;
  const bool fin = (p[0] & 0x7F80u) != 0x7F80u;
  const float r = fin ? v - bf16_lo(p[0]) : 0.0f;
  p[1] = pack_bf16x2(r, 0.0f) & 0xFFFFu;
  p[2] = pack_bf16x2(r - bf16_lo(p[1]), 0.0f) & 0xFFFFu;
}

constexpr int kTileSide = 64;

// A 64 x 64 tile of dlogits in parts: rows [2][T][Ep] and, transposed, columns
// [3][Ep][Tp], zeros past its end.
__global__ __launch_bounds__(kBlock) void split_kernel(const float* dl, int64_t T, int E,
                                                       uint16_t* rows, uint16_t* columns) {
  __shared__ float tile[kTileSide][kTileSide + 1];
  const int64_t t0 = int64_t(blockIdx.x) * kTileSide;
  const int e0 = int(blockIdx.y) * kTileSide;
  const int64_t Ep = int64_t(gridDim.y) * kTileSide, Tp = int64_t(gridDim.x) * kTileSide;
  const int c = int(threadIdx.x) & 63;
  for (int r = int(threadIdx.x) >> 6; r < kTileSide; r += kBlock / 64)
    tile[r][c] = t0 + r < T && e0 + c < E ? dl[(t0 + r) * E + e0 + c] : 0.0f;
  __syncthreads();
  for (int r = int(threadIdx.x) >> 6; r < kTileSide; r += kBlock / 64) {
    uint32_t p[3];
    if (rows && t0 + r < T) {
      split3(tile[r][c], p);
#pragma unroll
      for (int i = 0; i < 2; ++i) rows[(i * T + t0 + r) * Ep + e0 + c] = uint16_t(p[i]);
    }
    if (columns) {
      split3(tile[c][r], p);
#pragma unroll
      for (int i = 0; i < 3; ++i) columns[(i * Ep + e0 + r) * Tp + t0 + c] = uint16_t(p[i]);
    }
  }
}

// w [E][H] to [H][Ep], zeros past E.
__global__ __launch_bounds__(kBlock) void transpose_kernel(const uint16_t* w, int E, int H,
                                                           uint16_t* wt) {
  __shared__ uint16_t tile[kTileSide][kTileSide + 2];
  const int h0 = int(blockIdx.x) * kTileSide, e0 = int(blockIdx.y) * kTileSide;
  const int64_t Ep = int64_t(gridDim.y) * kTileSide;
  const int c = int(threadIdx.x) & 63;
  for (int r = int(threadIdx.x) >> 6; r < kTileSide; r += kBlock / 64)
    tile[r][c] = e0 + r < E && h0 + c < H ? w[int64_t(e0 + r) * H + h0 + c] : uint16_t(0);
  __syncthreads();
  for (int r = int(threadIdx.x) >> 6; r < kTileSide; r += kBlock / 64)
    if (h0 + r < H) wt[int64_t(h0 + r) * Ep + e0 + c] = tile[c][r];
}

struct OuterArgs {
  const void* d;                 // [3][Ep][Tp] bf16
  const void* x;                 // [T][H] bf16
  int64_t T, Tp;
  int E, Ep, H;
  int64_t each;                  // steps of 32 tokens a workgroup takes
  float* out;                    // [splits][E][H]
};

// ---------------------------------------------------------------------------
// dw[e, h] = sum over t of D[e, t] x[t, h], D the sum of three bf16 arrays.  A
// wave takes 64 experts and 64 channels.  The sum runs along the rows of x, so
// a fragment needs eight tokens of one channel in a lane: lane n loads four
// neighbouring channels 4n.. of eight rows, 128 bytes of a row at a time, and
// swaps halves of words; fragment c then holds the channels 4n + c.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kBlock) void outer_kernel(OuterArgs g) {
  const int lane = lane_id(), n = lane & 15, q = lane >> 4;
  const int h0 = int(blockIdx.x) * 256 + wave_id() * 64 + n * 4;
  const int e0 = int(blockIdx.y) * 64;
  const int64_t s0 = int64_t(blockIdx.z) * g.each;
  const int64_t steps = (g.T + 31) / 32;
  const int64_t s1 = s0 + g.each < steps ? s0 + g.each : steps;
  f32x4 acc[4][4];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int c = 0; c < 4; ++c) acc[m][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  const uint16_t* d = static_cast<const uint16_t*>(g.d) + int64_t(e0 + n) * g.Tp + q * 8;
  const uint16_t* x = static_cast<const uint16_t*>(g.x) + h0;
  for (int64_t s = s0; s < s1; ++s) {
    const int64_t t0 = s * 32 + q * 8;
    u32x2 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = u32x2{0u, 0u};
      if (h0 < g.H && t0 + i < g.T) v[i] = *reinterpret_cast<const u32x2*>(x + (t0 + i) * g.H);
    }
    u32x4 b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        b[2 * w][i] = __builtin_amdgcn_perm(v[2 * i + 1][w], v[2 * i][w], 0x05040100u);
        b[2 * w + 1][i] = __builtin_amdgcn_perm(v[2 * i + 1][w], v[2 * i][w], 0x07060302u);
      }
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const u32x4 a = *reinterpret_cast<const u32x4*>(
            d + (int64_t(p) * g.Ep + m * 16) * g.Tp + s * 32);
#pragma unroll
        for (int c = 0; c < 4; ++c) acc[m][c] = mfma(a, b[c], acc[m][c]);
      }
  }
  float* out = g.out + int64_t(blockIdx.z) * g.E * g.H;
  if (h0 >= g.H) return;
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int e = e0 + m * 16 + q * 4 + i;
      if (e < g.E)
        *reinterpret_cast<f32x4*>(out + int64_t(e) * g.H + h0) =
            f32x4{acc[m][0][i], acc[m][1][i], acc[m][2][i], acc[m][3][i]};
    }
}

template <int MT, int WN, int PARTS, bool BF16OUT>
void launch_gemm_shape(const GemmArgs& g, const GemmShape& s, hipStream_t stream) {
  const int64_t most = max_blocks(kBlock) / (int64_t(s.nb) * s.splits);
  for (int64_t b0 = 0; b0 < s.mb; b0 += most) {
    const dim3 grid{unsigned(s.mb - b0 < most ? s.mb - b0 : most), unsigned(s.nb),
                    unsigned(s.splits)};
    gemm_kernel<MT, WN, PARTS, BF16OUT><<<grid, kBlock, 0, stream>>>(g, b0);
  }
}

template <int PARTS, bool BF16OUT>
void launch_gemm(const GemmArgs& g, const GemmShape& s, hipStream_t stream) {
  if (s.mt == 1) {
    if (s.wn == 1)
      launch_gemm_shape<1, 1, PARTS, BF16OUT>(g, s, stream);
    else if (s.wn == 2)
      launch_gemm_shape<1, 2, PARTS, BF16OUT>(g, s, stream);
    else
      launch_gemm_shape<1, 4, PARTS, BF16OUT>(g, s, stream);
  } else if (s.mt == 2) {
    if (s.wn == 1)
      launch_gemm_shape<2, 1, PARTS, BF16OUT>(g, s, stream);
    else if (s.wn == 2)
      launch_gemm_shape<2, 2, PARTS, BF16OUT>(g, s, stream);
    else
      launch_gemm_shape<2, 4, PARTS, BF16OUT>(g, s, stream);
  } else {
    if (s.wn == 1)
      launch_gemm_shape<4, 1, PARTS, BF16OUT>(g, s, stream);
    else if (s.wn == 2)
      launch_gemm_shape<4, 2, PARTS, BF16OUT>(g, s, stream);
    else
      launch_gemm_shape<4, 4, PARTS, BF16OUT>(g, s, stream);
  }
}

void launch_sum_planes(const float* part, int planes, int64_t count, float* out, hipStream_t s) {
  const int64_t blocks = (count + kBlock - 1) / kBlock;
  sum_planes_kernel<<<unsigned(blocks < (1 << 20) ? blocks : (1 << 20)), kBlock, 0, s>>>(
      part, planes, count, out);
}

}  // namespace

hipError_t launch_router_logits(const LogitsArgs& a, hipStream_t s) {
  const GemmShape shape = gemm_shape(a.T, a.E, a.H, true);
  GemmArgs g{};
  g.a = a.x;
  g.b = a.w;
  g.M = a.T;
  g.N = a.E;
  g.K = a.H;
  g.lda = g.ldb = a.H;
  g.each = shape.each;
  g.out = shape.splits > 1 ? a.ws : static_cast<void*>(a.logits);
  launch_gemm<1, false>(g, shape, s);
  if (shape.splits > 1)
    launch_sum_planes(static_cast<const float*>(a.ws), shape.splits, a.T * a.E, a.logits, s);
  return hipGetLastError();
}

hipError_t launch_router_logits_backward(const LogitsArgs& a, hipStream_t s) {
  const LogitsBackwardSpace at = logits_backward_space(a.T, a.E, a.H);
  char* ws = static_cast<char*>(a.ws);
  uint16_t* rows = reinterpret_cast<uint16_t*>(ws + at.rows);
  uint16_t* columns = reinterpret_cast<uint16_t*>(ws + at.columns);
  uint16_t* wt = reinterpret_cast<uint16_t*>(ws + at.wt);
  const int Ep = int(pad64(a.E));
  const int64_t Tp = pad64(a.T);
  if (a.T > 0) {
    const dim3 grid{unsigned(Tp / kTileSide), unsigned(Ep / kTileSide), 1u};
    split_kernel<<<grid, kBlock, 0, s>>>(a.dlogits, a.T, a.E, a.dx ? rows : nullptr,
                                         a.dw ? columns : nullptr);
  }
  if (a.dx) {
    const dim3 grid{unsigned((a.H + kTileSide - 1) / kTileSide), unsigned(Ep / kTileSide), 1u};
    transpose_kernel<<<grid, kBlock, 0, s>>>(static_cast<const uint16_t*>(a.w), a.E, a.H, wt);
    const GemmShape shape = gemm_shape(a.T, a.H, Ep, false);
    GemmArgs g{};
    g.a = rows;
    g.b = wt;
    g.M = a.T;
    g.N = a.H;
    g.K = Ep;
    g.lda = g.ldb = Ep;
    g.plane = a.T * Ep;
    g.each = shape.each;
    g.out = a.dx;
    launch_gemm<2, true>(g, shape, s);
  }
  if (a.dw) {
    const OuterShape o = outer_shape(a.T, a.E, a.H);
    OuterArgs g{};
    g.d = columns;
    g.x = a.x;
    g.T = a.T;
    g.Tp = Tp;
    g.E = a.E;
    g.Ep = Ep;
    g.H = a.H;
    g.each = o.each;
    g.out = o.splits > 1 ? reinterpret_cast<float*>(ws + at.part) : a.dw;
    const dim3 grid{unsigned(o.hb), unsigned(o.eb), unsigned(o.splits)};
    outer_kernel<<<grid, kBlock, 0, s>>>(g);
    if (o.splits > 1)
      launch_sum_planes(g.out, o.splits, int64_t(a.E) * a.H, a.dw, s);
  }
  return hipGetLastError();
}

}  // namespace epdc
