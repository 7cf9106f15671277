// The router's logits and their gradients (gfx950, wave64): three products of
// which one side is small.  The matrix cores take bf16 and sum in fp32
// (v_mfma_f32_16x16x32_bf16); what is fp32 (the logits' gradient) takes part as
// the sum of two or three bf16 numbers.
#include "router_device.h"
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

// The order of a stage's instructions: its 2 M products with, between them, READS
// LDS reads, the WRITES writes, READS further reads and WRITES loads.
template <int M, int READS, int WRITES>
__device__ __forceinline__ void interleave() {
  constexpr int kProduct = 0x008, kLoad = 0x020, kRead = 0x100, kWrite = 0x200;
#pragma unroll
  for (int i = 0; i < READS; ++i) {
    __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
  }
#pragma unroll
  for (int i = 0; i < M - READS; ++i) {
    __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kWrite, (WRITES + M - READS - 1) / (M - READS), 0);
  }
#pragma unroll
  for (int i = 0; i < READS; ++i) {
    __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
  }
#pragma unroll
  for (int i = 0; i < M - READS; ++i) {
    __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
    __builtin_amdgcn_sched_group_barrier(kLoad, (WRITES + M - READS - 1) / (M - READS), 0);
  }
}

// That of the wide form, 2 M products a half: M LDS reads and M / 2 loads of weights in
// the first, then LA writes; M reads in the second, then LA loads of rows.
template <int M, int LA>
__device__ __forceinline__ void interleave_wide() {
  constexpr int kProduct = 0x008, kLoad = 0x020, kRead = 0x100, kWrite = 0x200;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < M; ++i) {
      __builtin_amdgcn_sched_group_barrier(kProduct, 1, 0);
      __builtin_amdgcn_sched_group_barrier(kRead, 1, 0);
      if (h == 0 && i % 2 == 0) __builtin_amdgcn_sched_group_barrier(kLoad, 1, 0);
    }
#pragma unroll
    for (int i = 0; i < LA; ++i) {
      __builtin_amdgcn_sched_group_barrier(kProduct, M / LA, 0);
      if (h == 0) __builtin_amdgcn_sched_group_barrier(kWrite, 1, 0);
      if (h == 1) __builtin_amdgcn_sched_group_barrier(kLoad, 1, 0);
    }
  }
}

struct LogitsGemm {
  const void* x;                 // [T][H] bf16
  const void* w;                 // [E][H] bf16
  int64_t T;
  int E, H;
  int each;                      // stages a workgroup takes
  float* out;                    // [splits][T][E]
};

// A lane's logits of N tiles, four neighbours every 16; `left` experts lie before the
// row's end.
template <int N>
__device__ __forceinline__ void store_tiles(float* to, const f32x4 (&v)[N], int left, int E) {
  if ((E & 3) == 0) {
#pragma unroll
    for (int t = 0; t < N; ++t)
      if (16 * t < left) __builtin_memcpy(to + 16 * t, &v[t], 16);
  } else {
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (16 * t + i < left) to[16 * t + i] = v[t][i];
  }
}

// ---------------------------------------------------------------------------
// out[t, e] = sum over h of x[t, h] w[e, h].  A workgroup takes 16 MT WM tokens
// and 64 WN experts, a wave 16 MT of the former and 64 of the latter; a stage is
// 64 channels of both.  Eight lanes load 128 bytes of a row into a ring of R
// stages in registers; from there a stage goes to one of three buffers in LDS,
// two stages before it is used, so that behind the one barrier of a stage the
// fragments of its first products are in registers already, and loads, LDS
// writes and reads all run between the products.  (Fragments loaded straight
// from memory have neighbouring lanes in different rows, and a load of 1 KB then
// takes 70 cycles: 129 us for 16384 tokens, 256 experts, 7168 channels.)
// Loads go through descriptors whose range check gives zeros for rows and
// channels past the end.  HBM bounds it up to 64 experts (16384 tokens of 7168
// channels 47 us, 5.0 TB/s); with 256 the L2 caches do, which give every 64 tokens
// all the weights (99 us).
// LDS holds a row of a stage as eight 16-byte pieces, permuted by three bits of
// the row, so that the eight rows that a read takes at once lie in different
// banks.  w is the instruction's first operand, so that a lane's four results are
// neighbouring experts.
// ---------------------------------------------------------------------------
template <int MT, int WM, int WN>
__global__ __launch_bounds__(kBlock) void logits_kernel(LogitsGemm g, int64_t mb0) {
  static_assert(WM * WN == 4, "four waves");
  constexpr int BM = 16 * MT * WM, BN = 64 * WN, R = 3;
  constexpr int kA = BM * 8, kB = BN * 8;                // pieces of a stage
  constexpr int LA = (kA + kBlock - 1) / kBlock, LB = kB / kBlock;
  __shared__ u32x4 lds[3 * (kA + kB)];
  const int lane = lane_id(), n = lane & 15, q = lane >> 4;
  const int wn = wave_id() % WN, wm = wave_id() / WN;
  const int64_t m0 = (mb0 + blockIdx.x) * BM;
  const int n0 = int(blockIdx.y) * BN;
  const int rows = int(g.T - m0 < BM ? g.T - m0 : BM);
  const int cols = g.E - n0 < BN ? g.E - n0 : BN;
  const int pitch = 2 * g.H;                             // bytes of a row
  const rsrc_t ar = make_rsrc(static_cast<const uint16_t*>(g.x) + m0 * g.H, int64_t(rows) * pitch);
  const rsrc_t br = make_rsrc(static_cast<const uint16_t*>(g.w) + int64_t(n0) * g.H,
                              int64_t(cols) * pitch);
  const int stages = (g.H + 63) / 64;
  const int st0 = int(blockIdx.z) * g.each;
  const int count = stages - st0 < g.each ? stages - st0 : g.each;
  const int row0 = int(threadIdx.x) >> 3, piece = int(threadIdx.x) & 7;
  const uint32_t off0 = uint32_t(row0) * uint32_t(pitch) + uint32_t(piece * 16);
  const uint32_t step = 32u * uint32_t(pitch);
  const int awrite = row0 * 8 + (piece ^ (row0 & 7)), bwrite = kA + awrite;
  u32x4 av[R][LA], bv[R][LB];
  auto load = [&](int d, int i0) {
    const int st = st0 + i0;
    const bool in = i0 < count && st * 64 + piece * 8 < g.H;
    const int so = i0 < count ? st * 128 : 0;
    const uint32_t off = in ? off0 : kOob;
#pragma unroll
    for (int i = 0; i < LA; ++i)
      av[d][i] = __builtin_amdgcn_raw_buffer_load_b128(ar, off + uint32_t(i) * step, so, 0);
#pragma unroll
    for (int i = 0; i < LB; ++i)
      bv[d][i] = __builtin_amdgcn_raw_buffer_load_b128(br, off + uint32_t(i) * step, so, 0);
  };
  auto write = [&](int d, int buf) {
    u32x4* to = lds + buf * (kA + kB);
#pragma unroll
    for (int i = 0; i < LA; ++i)
      if (kA % kBlock == 0 || int(threadIdx.x) + i * kBlock < kA) to[awrite + i * 256] = av[d][i];
#pragma unroll
    for (int i = 0; i < LB; ++i) to[bwrite + i * 256] = bv[d][i];
  };
  const int aread = (wm * 16 * MT + n) * 8, bread = kA + (wn * 64 + n) * 8;
  auto read = [&](int buf, int s, u32x4 (&a)[MT], u32x4 (&b)[4]) {
    const u32x4* from = lds + buf * (kA + kB);
    const int at = (s * 4 + q) ^ (n & 7);
#pragma unroll
    for (int t = 0; t < 4; ++t) b[t] = from[bread + t * 128 + at];
#pragma unroll
    for (int m = 0; m < MT; ++m) a[m] = from[aread + m * 128 + at];
  };
  f32x4 acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 a0[MT], b0[4], a1[MT], b1[4];
  auto products = [&](const u32x4 (&a)[MT], const u32x4 (&b)[4]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < 4; ++t) acc[m][t] = mfma(b[t], a[m], acc[m][t]);
  };
  // stages 0 and 1 into LDS, 2 and on into the ring: stage i's place is i % R
  load(0, 0);
  load(1, 1);
  load(2, 2);
  write(0, 0);
  load(0, 3);
  write(1, 1);
  load(1, 4);
  lds_barrier();
  read(0, 0, a0, b0);
  for (int st = 0; st < count; st += 3) {
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      // stage st + d in buffer d; the next in (d + 1) % 3; d + 2 is written
      read(d, 1, a1, b1);
      products(a0, b0);
      write((d + 2) % R, (d + 2) % 3);
      load((d + 2) % R, st + d + 2 + R);
      read((d + 1) % 3, 0, a0, b0);
      products(a1, b1);
      // a product, then one of the others, while there are any
      interleave<MT * 4, MT + 4, LA + LB>();
      lds_barrier();
    }
  }
  float* out = g.out + (int64_t(blockIdx.z) * g.T + m0) * g.E + n0;
  const int col = wn * 64 + q * 4;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = (wm * MT + m) * 16 + n;
    if (row < rows) store_tiles<4>(out + int64_t(row) * g.E + col, acc[m], cols - col, g.E);
  }
}

// ---------------------------------------------------------------------------
// The same for many tokens: a workgroup takes 128 of them and 128 experts, a wave all
// the tokens and 32 experts.  The weights come in the order of the matrix cores
// (wf_kernel), straight into registers, 1 KB a load, so that LDS moves the tokens'
// rows alone and a weight is loaded once for 128 tokens.  16384 tokens, 256 experts,
// 7168 channels take 80 us with the rows from HBM (264 MB, 3.3 TB/s), 57 with most of
// them in the Infinity Cache, and 64 tokens a workgroup 99.  The rows' wait bounds
// it: loads return in order, so a wait for weights is one for rows too.  256 experts a
// workgroup (71 us, but then in two splits, whose sum takes 17 more) and a last
// workgroup that adds the splits up (112: its fences write L2 back) were slower.
// ---------------------------------------------------------------------------
__global__ __launch_bounds__(kBlock, 2) void logits_wide_kernel(LogitsGemm g, const u32x4* wf,
                                                                int nb, int64_t b0) {
  constexpr int MT = kWideTokens / 16, kA = kWideTokens * 8, LA = kA / kBlock;
  __shared__ u32x4 lds[3 * kA];
  const int lane = lane_id(), n = lane & 15, q = lane >> 4;
  // Workgroups go to the eight XCDs in turn: those of the same tokens are eight
  // apart, so that the second finds the rows in its XCD's L2.
  const int64_t b = b0 + blockIdx.x, turn = b / (8 * nb);
  const int r = int(b - turn * (8 * nb));
  const int64_t m0 = (turn * 8 + (r & 7)) * kWideTokens;
  const int n0 = (r >> 3) * kWideExperts + wave_id() * 32;
  if (m0 >= g.T) return;
  const int rows = int(g.T - m0 < kWideTokens ? g.T - m0 : kWideTokens);
  const int pitch = 2 * g.H;                             // bytes of a row
  const rsrc_t ar = make_rsrc(static_cast<const uint16_t*>(g.x) + m0 * g.H, int64_t(rows) * pitch);
  const int stages = (g.H + 63) / 64;
  const int st0 = int(blockIdx.z) * g.each;
  const int count = stages - st0 < g.each ? stages - st0 : g.each;
  const int row0 = int(threadIdx.x) >> 3, piece = int(threadIdx.x) & 7;
  const uint32_t off0 = uint32_t(row0) * uint32_t(pitch) + uint32_t(piece * 16);
  const uint32_t step = 32u * uint32_t(pitch);
  const bool own = n0 < g.E;                             // else the wave has no experts
  // 4 KB a stage, zeros past the last: also where a weight is infinite, a stage past the
  // end adds nothing
  const rsrc_t wr = make_rsrc(wf + int64_t(own ? n0 >> 5 : 0) * stages * (4 * kWave),
                              int64_t(stages) * 4096);
  u32x4 av[3][LA], wv[3][2][2];
  auto load_x = [&](int d, int i0) {
    const int st = st0 + i0;
    const bool in = i0 < count && st * 64 + piece * 8 < g.H;
#pragma unroll
    for (int i = 0; i < LA; ++i)
      av[d][i] = __builtin_amdgcn_raw_buffer_load_b128(
          ar, (in ? off0 : kOob) + uint32_t(i) * step, i0 < count ? st * 128 : 0, 0);
  };
  auto load_w = [&](int d, int i0) {
    const uint32_t off = i0 < count ? uint32_t(lane * 16) : kOob;
    const int so = i0 < count ? (st0 + i0) * 4096 : 0;
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int t = 0; t < 2; ++t)
        wv[d][s][t] = __builtin_amdgcn_raw_buffer_load_b128(
            wr, off + uint32_t((s * 2 + t) * 1024), so, 0);
  };
  auto write = [&](int d, int buf) {
#pragma unroll
    for (int i = 0; i < LA; ++i)
      lds[buf * kA + (row0 + i * 32) * 8 + (piece ^ (row0 & 7))] = av[d][i];
  };
  auto read = [&](int buf, int s, u32x4 (&a)[MT]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
      a[m] = lds[buf * kA + (m * 16 + n) * 8 + ((s * 4 + q) ^ (n & 7))];
  };
  f32x4 acc[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < 2; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
  u32x4 a0[MT], a1[MT];
  auto products = [&](const u32x4 (&a)[MT], const u32x4 (&b)[2]) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int t = 0; t < 2; ++t) acc[m][t] = mfma(b[t], a[m], acc[m][t]);
  };
  // issued in the loop's order, for the waits at its top count the loads after
  // the one they wait for on both ways there
  load_x(0, 0);
  load_x(1, 1);
  load_x(2, 2);
  __builtin_amdgcn_sched_barrier(0);
  load_w(0, 0);
  __builtin_amdgcn_sched_barrier(0);
  write(0, 0);
  load_x(0, 3);
  __builtin_amdgcn_sched_barrier(0);
  load_w(1, 1);
  __builtin_amdgcn_sched_barrier(0);
  write(1, 1);
  load_x(1, 4);
  __builtin_amdgcn_sched_barrier(0);
  lds_barrier();
  read(0, 0, a0);
  for (int st = 0; st < count; st += 3) {
#pragma unroll
    for (int d = 0; d < 3; ++d) {
      // as in logits_kernel; the weights are two stages ahead: loads return in
      // order, so that a wait for them is one for the rows loaded before them
      load_w((d + 2) % 3, st + d + 2);
      read(d, 1, a1);
      products(a0, wv[d][0]);
      write((d + 2) % 3, (d + 2) % 3);
      load_x((d + 2) % 3, st + d + 5);
      read((d + 1) % 3, 0, a0);
      products(a1, wv[d][1]);
      interleave_wide<MT, LA>();
      lds_barrier();
    }
  }
  if (!own) return;
  float* out = g.out + (int64_t(blockIdx.z) * g.T + m0) * g.E + n0;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int row = m * 16 + n;
    if (row < rows)
      store_tiles<2>(out + int64_t(row) * g.E + q * 4, acc[m], g.E - n0 - q * 4, g.E);
  }
}

// wf: the weights in the matrix cores' order, [experts / 32][channels / 32][2 tiles]
// blocks of 1 KB, 16 bytes a lane: lane (n, q) holds channels 8 q and on of the
// block's 32 of expert n of the tile; zeros past the ends.
__global__ __launch_bounds__(kBlock) void wf_kernel(const u32x4* w, int E, int H, int Ep,
                                                    int64_t Hp, u32x4* out) {
  const int64_t at = int64_t(blockIdx.x) * kBlock + threadIdx.x;
  const int H8 = int(Hp >> 3);
  const int e = int(at / H8), h8 = int(at - int64_t(e) * H8);
  if (e >= Ep) return;
  const u32x4 v = e < E && h8 * 8 < H ? w[int64_t(e) * (H >> 3) + h8] : u32x4{0u, 0u, 0u, 0u};
  out[((int64_t(e >> 5) * (H8 >> 2) + (h8 >> 2)) * 2 + ((e >> 4) & 1)) * kWave +
      (h8 & 3) * 16 + (e & 15)] = v;
}

// A float as the sum of three bf16 numbers, exact where the last is no smaller
// than bf16 goes.  A finite number that rounds to an infinity starts from the
// largest finite one, 2^-8 of it away at most; infinities and NaN have no further
// parts.
__device__ __forceinline__ void split3(float v, uint32_t (&p)[3]) {
  const bool fin = (__float_as_uint(v) & 0x7F800000u) != 0x7F800000u;
  p[0] = pack_bf16x2(v, 0.0f) & 0xFFFFu;
  if (fin && (p[0] & 0x7FFFu) == 0x7F80u) p[0] -= 1u;
  const float r = fin ? v - bf16_lo(p[0]) : 0.0f;
  p[1] = pack_bf16x2(r, 0.0f) & 0xFFFFu;
  p[2] = pack_bf16x2(r - bf16_lo(p[1]), 0.0f) & 0xFFFFu;
}

__device__ __forceinline__ uint32_t half(uint32_t lo, uint32_t hi) { return lo | (hi << 16); }

// ---------------------------------------------------------------------------
// Operands of the gradients' products in the order in which the matrix cores
// take them: blocks of 1 KB, 16 bytes a lane, lane (n, q) = (lane & 15, lane >> 4)
// holding eight k of row n, k = 8 q and on of the block's 32.  A wave then loads
// a block as one run of memory.
// ---------------------------------------------------------------------------

// columns: dlogits transposed, [Ep / 64][Tp / 32][4 tiles][3 parts] blocks: rows
// are experts, k tokens; zeros past their ends.  A thread makes the pieces of
// eight tokens of an expert.
__device__ __forceinline__ void columns_piece(const float* dl, int64_t T, int E, int Ep,
                                              u32x4* out, int64_t at) {
  const int64_t t8 = at / Ep, T32 = (T + 31) / 32;
  const int e = int(at - t8 * Ep);
  if (t8 >= T32 * 4) return;
  uint32_t p[8][3];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    split3(e < E && t8 * 8 + i < T ? dl[(t8 * 8 + i) * E + e] : 0.0f, p[i]);
  const int64_t block = ((int64_t(e >> 6) * T32 + (t8 >> 2)) * 4 + ((e >> 4) & 3)) * 3;
  const int lane = int(t8 & 3) * 16 + (e & 15);
#pragma unroll
  for (int j = 0; j < 3; ++j)
    out[(block + j) * kWave + lane] = u32x4{half(p[0][j], p[1][j]), half(p[2][j], p[3][j]),
                                            half(p[4][j], p[5][j]), half(p[6][j], p[7][j])};
}

// wt: the weights transposed, [Hp / 64][Ep / 32][4 tiles] blocks: rows are
// channels, k experts; zeros past their ends.  Row r of tile i is channel
// (i / 2) * 32 + (r / 4) * 8 + (i % 2) * 4 + r % 4 of 64, so that a lane of the product
// gets eight neighbours from two tiles.
__device__ __forceinline__ void wt_piece(const uint16_t* w, int E, int H, int Ep, int64_t Hp,
                                         u32x4* out, int64_t at) {
  const int e8 = int(at / Hp);
  const int64_t h = at - e8 * Hp;
  if (e8 * 8 >= Ep) return;
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = h < H && e8 * 8 + i < E ? w[int64_t(e8 * 8 + i) * H + h] : 0u;
  const int r = int(h & 3) | int((h >> 3) & 3) << 2;
  const int tile = int((h >> 5) & 1) * 2 + int((h >> 2) & 1);
  out[(((h >> 6) * (Ep >> 5) + (e8 >> 2)) * 4 + tile) * kWave + (e8 & 3) * 16 + r] =
      u32x4{half(v[0], v[1]), half(v[2], v[3]), half(v[4], v[5]), half(v[6], v[7])};
}

// Both: the first `wt_blocks` workgroups make wt, the others columns.
__global__ __launch_bounds__(kBlock) void operands_kernel(LogitsArgs a, int Ep, int64_t Hp,
                                                          u32x4* wt, int64_t wt_blocks,
                                                          u32x4* columns, int64_t block0) {
  const int64_t b = block0 + blockIdx.x;
  if (b < wt_blocks)
    wt_piece(static_cast<const uint16_t*>(a.w), a.E, a.H, Ep, Hp, wt, b * kBlock + threadIdx.x);
  else
    columns_piece(a.dlogits, a.T, a.E, Ep, columns, (b - wt_blocks) * kBlock + threadIdx.x);
}

// ---------------------------------------------------------------------------
// dx[t, h] = sum over e of dlogits[t, e] w[e, h].  A workgroup keeps its 16 MT
// tokens' rows of dlogits in LDS, as two bf16 parts in the order above, and
// walks along the channels: each wave streams its share of wt, 64 channels at a
// time, and stores 64 bytes of a token's row by four lanes.  8195 tokens, 64 experts,
// 4096 channels take 20 us (3.4 TB/s written), 16384, 256 and 7168 100 to 122 us: 120 GFLOP
// in two parts, 1.0 to 1.2 PFLOP/s of the 1.9 that products alone reach here.  Within 256
// registers two workgroups share a compute unit (264 registers: 164 us).
// ---------------------------------------------------------------------------
struct DxArgs {
  const float* dl;
  const u32x4* wt;
  int64_t T;
  int E, Ep, H;
  int each;                      // blocks of 64 channels a workgroup takes
  void* dx;
};

template <int MT>
__global__ __launch_bounds__(kBlock, 2) void dx_kernel(DxArgs g, int64_t mb0) {
  extern __shared__ u32x4 rows[];            // [2 parts][Ep / 32][MT] blocks
  const int lane = lane_id(), n = lane & 15, q = lane >> 4;
  const int64_t m0 = (mb0 + blockIdx.x) * (16 * MT);
  const int K32 = g.Ep >> 5, E8 = g.Ep >> 3;
  const int part = K32 * MT * kWave;
  for (int at = int(threadIdx.x); at < 16 * MT * E8; at += kBlock) {
    const int r = at / E8, e = (at - r * E8) * 8;
    float v[8];
    const float* from = g.dl + (m0 + r) * g.E + e;
    const int left = m0 + r < g.T ? g.E - e : 0;
    if ((g.E & 3) == 0 && left >= 8) {
      __builtin_memcpy(v, __builtin_assume_aligned(from, 4), 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < left ? from[i] : 0.0f;
    }
    uint32_t p[8][3];
#pragma unroll
    for (int i = 0; i < 8; ++i) split3(v[i], p[i]);
    const int to = ((e >> 5) * MT + (r >> 4)) * kWave + ((e >> 3) & 3) * 16 + (r & 15);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      rows[j * part + to] = u32x4{half(p[0][j], p[1][j]), half(p[2][j], p[3][j]),
                                  half(p[4][j], p[5][j]), half(p[6][j], p[7][j])};
  }
  __syncthreads();
  // this wave's blocks of 64 channels
  const int all = (g.H + 63) >> 6;
  const int first = int(blockIdx.y) * g.each;
  const int end = first + g.each < all ? first + g.each : all;
  const int share = (end - first + 3) / 4;
  const int hb0 = first + wave_id() * share;
  const int hb1 = hb0 + share < end ? hb0 + share : end;
  if (hb0 >= hb1) return;
  const int pairs = K32 >> 1;                // steps of 64 experts a block
  const int64_t total = int64_t(hb1 - hb0) * pairs;
  const u32x4* w = g.wt + int64_t(hb0) * K32 * (4 * kWave) + lane;
  u32x4 b[2][2][4], a[2][2][MT];
  auto load = [&](int d, int s, int64_t p) {
    if (p >= total) return;                  // the same for the whole wave
#pragma unroll
    for (int t = 0; t < 4; ++t) b[d][s][t] = w[((p * 2 + s) * 4 + t) * kWave];
  };
  auto read = [&](int d, int k32) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int m = 0; m < MT; ++m) a[d][j][m] = rows[j * part + (k32 * MT + m) * kWave + lane];
  };
  f32x4 acc[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int t = 0; t < 4; ++t) acc[m][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int d = 0; d < 2; ++d)
#pragma unroll
    for (int s = 0; s < 2; ++s) load(d, s, d);
  read(0, 0);
  int k = 0, hb = hb0;
  for (int64_t p0 = 0; p0 < total; p0 += 2) {
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      if (p0 + d >= total) break;
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        // the next step's rows, which start over with every block of channels
        read(s ^ 1, s == 0 ? 2 * k + 1 : k + 1 < pairs ? 2 * k + 2 : 0);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int t = 0; t < 4; ++t) acc[m][t] = mfma(b[d][s][t], a[s][j][m], acc[m][t]);
        load(d, s, p0 + d + 2);
#pragma unroll
        for (int i = 0; i < 2 * MT; ++i) {
          __builtin_amdgcn_sched_group_barrier(0x008, 4, 0);     // four products,
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);     // an LDS read
        }
      }
      if (++k < pairs) continue;
      const int h = hb * 64 + q * 8;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int64_t t = m0 + m * 16 + n;
        u32x4* to = reinterpret_cast<u32x4*>(static_cast<uint16_t*>(g.dx) + t * g.H + h);
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (t < g.T && h + 32 * i < g.H)
            to[4 * i] = u32x4{pack_bf16x2(acc[m][2 * i][0], acc[m][2 * i][1]),
                          pack_bf16x2(acc[m][2 * i][2], acc[m][2 * i][3]),
                          pack_bf16x2(acc[m][2 * i + 1][0], acc[m][2 * i + 1][1]),
                          pack_bf16x2(acc[m][2 * i + 1][2], acc[m][2 * i + 1][3])};
#pragma unroll
        for (int t4 = 0; t4 < 4; ++t4) acc[m][t4] = f32x4{0.f, 0.f, 0.f, 0.f};
      }
      k = 0;
      ++hb;
    }
  }
}

// ---------------------------------------------------------------------------
// dw[e, h] = sum over t of dlogits[t, e] x[t, h].  A workgroup takes 64 experts
// and 128 channels, its waves every fourth step of 32 tokens; they add up at the
// end, in order.  The sum runs along the rows of x, so a fragment needs eight
// tokens of one channel in a lane: lane n loads eight neighbouring channels 8n..
// of eight rows, 256 bytes of a row at a time, and swaps halves of words;
// fragment c then holds the channels 8n + c, and a lane's results are neighbours.
// The matrix cores bound it: 16384 tokens, 256 experts, 7168 channels take 174 to 206
// us, 180 GFLOP in three parts, 0.9 to 1.0 PFLOP/s (with fragments of dlogits from rows
// a token apart 540 us); 8195, 64 and 4096, with eight steps a wave, 20 us (with loads
// two steps ahead 31).
// ---------------------------------------------------------------------------
struct DwArgs {
  const u32x4* columns;
  const void* x;                 // [T][H] bf16
  int64_t T;
  int E, H;
  int64_t each;                  // steps of 32 tokens a workgroup takes
  float* out;                    // [splits][E][H]
};

__global__ __launch_bounds__(kBlock, 1) void dw_kernel(DwArgs g) {
  constexpr int kPitch = 132;                // floats a row of sums
  __shared__ float sum[4][64][kPitch];
  const int lane = lane_id(), n = lane & 15, q = lane >> 4, wave = wave_id();
  const int h0 = int(blockIdx.x) * 128;
  const int e0 = int(blockIdx.y) * 64;
  const int64_t T32 = (g.T + 31) / 32;
  const int64_t s0 = int64_t(blockIdx.z) * g.each;
  const int64_t s1 = s0 + g.each < T32 ? s0 + g.each : T32;
  const u32x4* columns = g.columns + int64_t(blockIdx.y) * T32 * (12 * kWave) + lane;
  const uint32_t pitch = uint32_t(2 * g.H);
  const uint32_t off = h0 + n * 8 < g.H ? uint32_t(q * 8) * pitch + uint32_t(2 * (h0 + n * 8))
                                        : kOob;
  u32x4 a[12], v[8];
  auto load = [&](int64_t s) {
    if (s >= s1) return;                     // the same for the whole wave
#pragma unroll
    for (int i = 0; i < 12; ++i) a[i] = columns[(s * 12 + i) * kWave];
    const int64_t left = g.T - s * 32;
    const rsrc_t xr = make_rsrc(static_cast<const uint16_t*>(g.x) + s * 32 * g.H,
                                (left < 32 ? left : 32) * pitch);
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = __builtin_amdgcn_raw_buffer_load_b128(xr, off + uint32_t(i) * pitch, 0, 0);
  };
  f32x4 acc[4][8];
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[m][c] = f32x4{0.f, 0.f, 0.f, 0.f};
  load(s0 + wave);
  for (int64_t s = s0 + wave; s < s1; s += 4) {
    u32x4 b[8], d[12];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        b[2 * w][i] = __builtin_amdgcn_perm(v[2 * i + 1][w], v[2 * i][w], 0x05040100u);
        b[2 * w + 1][i] = __builtin_amdgcn_perm(v[2 * i + 1][w], v[2 * i][w], 0x07060302u);
      }
#pragma unroll
    for (int i = 0; i < 12; ++i) d[i] = a[i];
    load(s + 4);
#pragma unroll
    for (int p = 0; p < 3; ++p)
#pragma unroll
      for (int m = 0; m < 4; ++m)
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[m][c] = mfma(d[m * 3 + p], b[c], acc[m][c]);
  }
#pragma unroll
  for (int m = 0; m < 4; ++m)
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<f32x4*>(&sum[wave][m * 16 + q * 4 + i][n * 8 + 4 * j]) =
            f32x4{acc[m][4 * j][i], acc[m][4 * j + 1][i], acc[m][4 * j + 2][i],
                  acc[m][4 * j + 3][i]};
  __syncthreads();
  float* out = g.out + int64_t(blockIdx.z) * g.E * g.H;
  for (int at = int(threadIdx.x); at < 64 * 32; at += kBlock) {
    const int r = at >> 5, c = (at & 31) * 4;
    if (e0 + r >= g.E || h0 + c >= g.H) continue;
    f32x4 t = *reinterpret_cast<const f32x4*>(&sum[0][r][c]);
#pragma unroll
    for (int w = 1; w < 4; ++w) t += *reinterpret_cast<const f32x4*>(&sum[w][r][c]);
    *reinterpret_cast<f32x4*>(out + int64_t(e0 + r) * g.H + h0 + c) = t;
  }
}

template <int MT, int WM, int WN>
void launch_logits_shape(const LogitsGemm& g, const LogitsShape& s, hipStream_t stream) {
  const int64_t most = max_blocks(kBlock) / (int64_t(s.nb) * s.splits);
  for (int64_t b0 = 0; b0 < s.mb; b0 += most) {
    const dim3 grid{unsigned(s.mb - b0 < most ? s.mb - b0 : most), unsigned(s.nb),
                    unsigned(s.splits)};
    logits_kernel<MT, WM, WN><<<grid, kBlock, 0, stream>>>(g, b0);
  }
}

template <int MT>
void launch_dx(const DxArgs& g, const DxShape& s, hipStream_t stream) {
  const unsigned lds = unsigned(2 * 16 * MT * g.Ep * 2);
  const int64_t most = max_blocks(kBlock) / s.splits;
  for (int64_t b0 = 0; b0 < s.mb; b0 += most) {
    const dim3 grid{unsigned(s.mb - b0 < most ? s.mb - b0 : most), unsigned(s.splits), 1u};
    dx_kernel<MT><<<grid, kBlock, lds, stream>>>(g, b0);
  }
}

}  // namespace

hipError_t launch_router_logits(const LogitsArgs& a, hipStream_t s) {
  const LogitsShape shape = logits_shape(a.T, a.E, a.H);
  LogitsGemm g{};
  g.x = a.x;
  g.w = a.w;
  g.T = a.T;
  g.E = a.E;
  g.H = a.H;
  g.each = shape.each;
  g.out = shape.splits > 1 ? static_cast<float*>(a.ws) : a.logits;
  if (shape.wide) {
    const WideSpace at = wide_space(shape, a.T, a.E, a.H);
    char* ws = static_cast<char*>(a.ws);
    u32x4* wf = reinterpret_cast<u32x4*>(ws + at.wf);
    if (shape.splits > 1) g.out = reinterpret_cast<float*>(ws + at.part);
    const int64_t pieces = at.experts * (at.channels >> 3);
    wf_kernel<<<unsigned((pieces + kBlock - 1) / kBlock), kBlock, 0, s>>>(
        static_cast<const u32x4*>(a.w), a.E, a.H, int(at.experts), at.channels, wf);
    const int64_t blocks = (shape.mb + 7) / 8 * 8 * shape.nb;
    for_each_launch(blocks, kBlock * shape.splits, [&](int64_t b0, unsigned n) {
      const dim3 grid{n, 1u, unsigned(shape.splits)};
      logits_wide_kernel<<<grid, kBlock, 0, s>>>(g, wf, shape.nb, b0);
    });
  } else if (shape.bm == 16)
    launch_logits_shape<1, 1, 4>(g, shape, s);
  else if (shape.bm == 32)
    launch_logits_shape<2, 1, 4>(g, shape, s);
  else if (shape.wn == 1)
    launch_logits_shape<1, 4, 1>(g, shape, s);
  else if (shape.wn == 2)
    launch_logits_shape<2, 2, 2>(g, shape, s);
  else
    launch_logits_shape<4, 1, 4>(g, shape, s);
  if (shape.splits > 1)
    launch_sum_rows(g.out, shape.splits, a.T * a.E, a.logits, s);
  return hipGetLastError();
}

hipError_t launch_router_logits_backward(const LogitsArgs& a, hipStream_t s) {
  const LogitsBackwardSpace at = logits_backward_space(a.T, a.E, a.H);
  char* ws = static_cast<char*>(a.ws);
  u32x4* columns = reinterpret_cast<u32x4*>(ws + at.columns);
  u32x4* wt = reinterpret_cast<u32x4*>(ws + at.wt);
  const int Ep = int(pad64(a.E));
  const int64_t Hp = pad64(a.H), per = kBlock;
  const int64_t wt_blocks = a.dx ? (Hp * (Ep / 8) + per - 1) / per : 0;
  const int64_t column_blocks = a.dw ? ((a.T + 31) / 32 * 4 * Ep + per - 1) / per : 0;
  for_each_launch(wt_blocks + column_blocks, kBlock, [&](int64_t b0, unsigned grid) {
    operands_kernel<<<grid, kBlock, 0, s>>>(a, Ep, Hp, wt, wt_blocks, columns, b0);
  });
  if (a.dx) {
    const DxShape shape = dx_shape(a.T, a.H, Ep);
    DxArgs g{};
    g.dl = a.dlogits;
    g.wt = wt;
    g.T = a.T;
    g.E = a.E;
    g.Ep = Ep;
    g.H = a.H;
    g.each = shape.each;
    g.dx = a.dx;
    if (shape.mt == 1)
      launch_dx<1>(g, shape, s);
    else if (shape.mt == 2)
      launch_dx<2>(g, shape, s);
    else
      launch_dx<4>(g, shape, s);
  }
  if (a.dw) {
    const DwShape shape = dw_shape(a.T, a.E, a.H);
    DwArgs g{};
    g.columns = columns;
    g.x = a.x;
    g.T = a.T;
    g.E = a.E;
    g.H = a.H;
    g.each = shape.each;
    g.out = shape.splits > 1 ? reinterpret_cast<float*>(ws + at.part) : a.dw;
    const dim3 grid{unsigned(shape.hb), unsigned(shape.eb), unsigned(shape.splits)};
    dw_kernel<<<grid, kBlock, 0, s>>>(g);
    if (shape.splits > 1)
      launch_sum_rows(g.out, shape.splits, int64_t(a.E) * a.H, a.dw, s);
  }
  return hipGetLastError();
}

}  // namespace epdc
