// Products of a few rows with their experts' matrices, a whole expert layer
// for a few tokens, and the 4-bit weight quantizer (gfx950, wave64).
//
// With a few rows an expert's matrix is read once and used a handful of
// times, so the weights' bytes bound every kernel here.  The matrix cores do
// the arithmetic all the same: D[row][n] += X[row][k] W[n][k] with
// v_mfma_f32_16x16x32_bf16 takes up to 16 rows at the cost of one, sums
// over the lanes by itself and leaves the vector unit to the 4-bit decoding.
//
// A wave owns 16*NT weight rows n and walks blocks of 128 channels.  Lane l
// holds row l % 16 of each tile and the lane group g = l / 16 a quarter of the
// block's channels.  Loads are 16 bytes a lane through buffer descriptors
// whose range check returns zeros for the rows past N, the token rows past
// the expert's count and the channels past K, so nothing branches.  Loads
// return in order, hence the rows x are fetched as far ahead as the weights:
// both sit in a ring of D blocks of registers.
#include "epdc_device.h"
#include "expert_launch.h"

namespace epdc {

namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr uint32_t kOob = 0x80000000u;      // past every descriptor's range (< 2^31 bytes)
constexpr int kBlockK = 128;                // channels per block

__device__ __forceinline__ rsrc_t make_rsrc(const void* p, int64_t bytes) {
  // stride 0, 32-bit data format: offsets are bytes, checked against `bytes`
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, int(bytes), 0x00027000);
}

__device__ __forceinline__ u32x4 load16(rsrc_t r, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(r, off, 0, 0);
}

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                 __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Bytes of one weight row and of its scales.
template <int KIND>
__device__ __forceinline__ int row_bytes(int K) { return KIND == kWBf16 ? 2 * K : K / 2; }
template <int KIND>
__device__ __forceinline__ int scale_bytes(int K) {
  return KIND == kWFp4 ? K / 32
                       : KIND == kWInt4G32 ? K / 16
                                           : KIND == kWInt4G64 ? K / 32 : K / 64;
}

// Which channels a lane group holds.  A lane's 16 bytes are 8 channels of a
// bf16 row but 32 of a 4-bit row.  One matrix instruction sums over all four
// lane groups, so a scale that differs between them has to be applied before
// it (fp4: a power of two, exact in bf16) or the lanes have to share it:
// int4 with one scale per 128 channels does; with 32 or 64 the four dwords
// are transposed between the lane groups first, which leaves instruction j
// with the channels 32j..32j+31.  kSplit: group g holds channels 32g..32g+31
// and instruction j their j-th eight; otherwise group g holds the g-th eight
// of instruction j's 32 channels.
template <int KIND>
constexpr bool kSplit = KIND == kWFp4 || KIND == kWInt4G128;

template <int KIND>
struct RawW {
  u32x4 v[KIND == kWBf16 ? 4 : 1];
  uint32_t s0, s1;
};

// The 4x4 transposition of dwords between lane groups: dword j of group g
// becomes dword g of group j (row swaps of the two bits of g against j's).
__device__ __forceinline__ u32x4 transpose_groups(u32x4 v) {
  auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

// Eight e2m1 codes times a power of two, as bf16 (exact: two significant
// bits; the conversion reads only the scale's exponent, 0 standing for 2^-127
// and 255 for NaN).
__device__ __forceinline__ u32x4 decode_fp4(uint32_t d, float scale) {
  typedef __bf16 b2 __attribute__((ext_vector_type(2)));
  const b2 p0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 0);
  const b2 p1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 1);
  const b2 p2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 2);
  const b2 p3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(d, scale, 3);
  return u32x4{__builtin_bit_cast(uint32_t, p0), __builtin_bit_cast(uint32_t, p1),
               __builtin_bit_cast(uint32_t, p2), __builtin_bit_cast(uint32_t, p3)};
}

// Eight int4 codes c as the bf16 numbers 16 + c (exact: c in the top four
// mantissa bits of 16), in the order 0 4 1 5 2 6 3 7.  c - 8 = (16 + c) - 24,
// so the product with the row is this one's minus 24 times the row's sum,
// which another matrix instruction gives for all the tiles of a block.
__device__ __forceinline__ u32x4 decode_int4(uint32_t d) {
  constexpr uint32_t m = 0x00780078u, b = 0x41804180u;
  return u32x4{((d << 3) & m) | b, ((d >> 1) & m) | b, ((d >> 5) & m) | b, ((d >> 9) & m) | b};
}
constexpr uint32_t kMinus24 = 0xC1C0C1C0u;

// A row's eight channels in that order.
__device__ __forceinline__ u32x4 order_int4(u32x4 x) {
  return u32x4{__builtin_amdgcn_perm(x.z, x.x, 0x05040100u),
               __builtin_amdgcn_perm(x.z, x.x, 0x07060302u),
               __builtin_amdgcn_perm(x.w, x.y, 0x05040100u),
               __builtin_amdgcn_perm(x.w, x.y, 0x07060302u)};
}

// Sums of the blocks kb0, kb0 + step, ... below kb1 into acc: MT tiles of 16
// rows x against NT tiles of 16 weight rows.  xoff, woff and soff are the
// lane's byte offsets of its row (kOob: none), without the lane group's part.
// A row x is the sum of XP bf16 rows, `plane` bytes apart.
template <int KIND, int NT, int MT, int XP, int D>
__device__ __forceinline__ void few_tile(rsrc_t xr, rsrc_t wr, rsrc_t sr,
                                         const uint32_t (&xoff)[MT], const uint32_t (&woff)[NT],
                                         const uint32_t (&soff)[NT], uint32_t plane, int K,
                                         int kb0, int kb1, int step, f32x4 (&acc)[MT][NT]) {
  constexpr int WV = KIND == kWBf16 ? 4 : 1;
  const int g = lane_id() >> 4;
  RawW<KIND> wb[D][NT];
  u32x4 xb[D][MT][XP * 4];

  auto load = [&](int d, int kb) {
    const bool in = kb < kb1;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int j = 0; j < WV; ++j) {
        const bool ok = in && (KIND != kWBf16 || kb * kBlockK + j * 32 + g * 8 < K);
        const uint32_t off = KIND == kWBf16 ? woff[nt] + uint32_t(kb * 256 + j * 64 + g * 16)
                                            : woff[nt] + uint32_t(kb * 64 + g * 16);
        wb[d][nt].v[j] = load16(wr, ok ? off : kOob);
      }
      if constexpr (KIND == kWFp4) {
        wb[d][nt].s0 = uint32_t(uint8_t(__builtin_amdgcn_raw_buffer_load_b8(
            sr, in ? soff[nt] + uint32_t(kb * 4 + g) : kOob, 0, 0)));
      } else if constexpr (KIND == kWInt4G128) {
        wb[d][nt].s0 = uint32_t(uint16_t(__builtin_amdgcn_raw_buffer_load_b16(
            sr, in ? soff[nt] + uint32_t(kb * 2) : kOob, 0, 0)));
      } else if constexpr (KIND == kWInt4G64) {
        wb[d][nt].s0 =
            __builtin_amdgcn_raw_buffer_load_b32(sr, in ? soff[nt] + uint32_t(kb * 4) : kOob, 0, 0);
      } else if constexpr (KIND == kWInt4G32) {
        const auto s =
            __builtin_amdgcn_raw_buffer_load_b64(sr, in ? soff[nt] + uint32_t(kb * 8) : kOob, 0, 0);
        wb[d][nt].s0 = s[0];
        wb[d][nt].s1 = s[1];
      }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = kSplit<KIND> ? g * 32 + j * 8 : j * 32 + g * 8;
        const bool ok = in && (KIND != kWBf16 || kb * kBlockK + c < K);
        const uint32_t off = xoff[mt] + uint32_t((kb * kBlockK + c) * 2);
#pragma unroll
        for (int p = 0; p < XP; ++p)
          xb[d][mt][p * 4 + j] = load16(xr, ok ? off + p * plane : kOob);
      }
  };

  auto compute = [&](int d) {
    if constexpr (KIND == kWBf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int p = 0; p < XP; ++p)
              acc[mt][nt] = mfma(xb[d][mt][p * 4 + j], wb[d][nt].v[j], acc[mt][nt]);
    } else if constexpr (KIND == kWFp4) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const float sc = __uint_as_float(wb[d][nt].s0 << 23);
        const u32x4 v = wb[d][nt].v[0];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const u32x4 b = decode_fp4(v[j], sc);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int p = 0; p < XP; ++p)
              acc[mt][nt] = mfma(xb[d][mt][p * 4 + j], b, acc[mt][nt]);
        }
      }
    } else {
      constexpr int Q = KIND == kWInt4G128 ? 1 : KIND == kWInt4G64 ? 2 : 4;   // groups a block
      constexpr int J = 4 / Q;                                                // products a group
      const u32x4 minus = {kMinus24, kMinus24, kMinus24, kMinus24};
      u32x4 x[MT][XP * 4];
      f32x4 base[MT][Q];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          base[mt][q] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = q * J; j < q * J + J; ++j)
#pragma unroll
            for (int p = 0; p < XP; ++p) {
              x[mt][p * 4 + j] = order_int4(xb[d][mt][p * 4 + j]);
              base[mt][q] = mfma(x[mt][p * 4 + j], minus, base[mt][q]);
            }
        }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const u32x4 v =
            KIND == kWInt4G128 ? wb[d][nt].v[0] : transpose_groups(wb[d][nt].v[0]);
        u32x4 b[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) b[j] = decode_int4(v[j]);
#pragma unroll
        for (int q = 0; q < Q; ++q) {
          const uint32_t sw = q < 2 ? wb[d][nt].s0 : wb[d][nt].s1;
          const float sc = Q > 1 && (q & 1) ? bf16_hi(sw) : bf16_lo(sw);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            f32x4 part = base[mt][q];
#pragma unroll
            for (int j = q * J; j < q * J + J; ++j)
#pragma unroll
              for (int p = 0; p < XP; ++p) part = mfma(x[mt][p * 4 + j], b[j], part);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              acc[mt][nt][i] = __builtin_fmaf(sc, part[i], acc[mt][nt][i]);
          }
        }
      }
    }
  };

#pragma unroll
  for (int d = 0; d < D; ++d) load(d, kb0 + d * step);
  for (int kb = kb0; kb < kb1; kb += D * step) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      compute(d);
      load(d, kb + (d + D) * step);
    }
  }
}

// ---------------------------------------------------------------------------
// Which experts the slots name.  Every workgroup works out for itself the
// y-th expert in use (ascending) and that expert's slots: at most 1024 ids
// out of the L2, three barriers.  A launch of its own would cost more than
// these few microseconds, most of which pass while other workgroups stream.
// ---------------------------------------------------------------------------
__device__ __forceinline__ int slot_expert(const int64_t* ids64, const int32_t* ids32,
                                           int64_t first, int experts, int s) {
  if (ids64) {
    const int64_t e = ids64[s] - first;
    return ids64[s] >= 0 && e >= 0 && e < experts ? int(e) : -1;
  }
  if (ids32) {
    const int e = ids32[s];
    return e >= 0 && e < experts ? e : -1;
  }
  return 0;
}

struct SharedPlan {
  uint32_t bits[kFewExperts / 32];
  int16_t id[kFewSlots];
  uint16_t list[kFewSlots];
};

// Returns the number of slots of the y-th expert in use, 0 if there is none;
// `first`: the slots of lower experts; `active`: experts in use.
__device__ __forceinline__ int find_expert(SharedPlan& sp, const FewArgs& a, int y, int& expert,
                                           int& first, int& active) {
  const int tid = threadIdx.x;
  const int lane = lane_id();
  if (tid < kFewExperts / 32) sp.bits[tid] = 0u;
  __syncthreads();
  for (int s = tid; s < a.slots; s += kBlock) {
    const int e = slot_expert(a.ids64, a.ids32, a.first_expert, a.experts, s);
    sp.id[s] = int16_t(e);
    if (e >= 0) atomicOr(&sp.bits[e >> 5], 1u << (e & 31));
  }
  __syncthreads();
  // every wave by itself: a prefix sum of the bit counts finds the word
  const uint32_t word = lane < kFewExperts / 32 ? sp.bits[lane] : 0u;
  const int n = __popc(word);
  int incl = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up(incl, o);
    if (lane >= o) incl += v;
  }
  active = __builtin_amdgcn_readlane(incl, 31);
  if (y >= active) return 0;
  const uint64_t hit = ballot(lane < 32 && incl - n <= y && y < incl);
  const int src = __ffsll((unsigned long long)hit) - 1;
  uint32_t w = __builtin_amdgcn_readlane(word, src);
  for (int r = y - __builtin_amdgcn_readlane(incl - n, src); r > 0; --r) w &= w - 1;
  expert = src * 32 + __ffs(w) - 1;
  int m = 0;
  first = 0;
  for (int s0 = 0; s0 < a.slots; s0 += kWave) {
    const int s = s0 + lane;
    const int e = s < a.slots ? int(sp.id[s]) : -1;
    const uint64_t mine = ballot(e == expert);
    if (wave_id() == 0 && e == expert) sp.list[m + __popcll(mine & lanemask_lt())] = uint16_t(s);
    m += __popcll(mine);
    first += __popcll(ballot(e >= 0 && e < expert));
  }
  __syncthreads();
  return m;
}

// ---------------------------------------------------------------------------
// Few rows against their experts' matrices: grid (tiles of weight rows,
// experts in use at most).  The four waves of a workgroup take every fourth
// block of channels each and add up through LDS in a fixed order.  GATED: a
// tile is half gate and half up rows and y = silu(g) * u.
// ---------------------------------------------------------------------------
template <int KIND, int NT, int MT, bool GATED, int D>
__global__ __launch_bounds__(kBlock) void few_rows_kernel(FewArgs a) {
  constexpr int C = GATED ? NT / 2 : NT;             // tiles of output channels
  constexpr int kRow = NT * 16 + 4;                  // + 4: the lane groups' rows in other banks
  __shared__ SharedPlan sp;
  __shared__ float red[kWavesPerBlock][MT * 16][kRow];
  const int lane = lane_id(), wave = wave_id();
  int e = 0, first = 0, active = 0;
  int m = find_expert(sp, a, blockIdx.y, e, first, active);
  e = __builtin_amdgcn_readfirstlane(e);
  m = __builtin_amdgcn_readfirstlane(m);
  if (GATED && blockIdx.x == 0) {
    if (blockIdx.y == 0 && threadIdx.x == 0) a.plan->active = active;
    if (m > 0 && threadIdx.x == 0) {
      a.plan->expert[blockIdx.y] = e;
      a.plan->first[blockIdx.y] = first;
      a.plan->count[blockIdx.y] = m;
    }
    for (int i = threadIdx.x; i < m; i += kBlock) a.plan->order[first + i] = sp.list[i];
  }
  if (m == 0) return;

  const int rows = GATED ? 2 * a.N : a.N;
  const int wrow = row_bytes<KIND>(a.K), srow = scale_bytes<KIND>(a.K);
  const int64_t wbytes = int64_t(rows) * wrow, sbytes = int64_t(rows) * srow;
  const rsrc_t wr = make_rsrc(static_cast<const char*>(a.w.q) + e * wbytes, wbytes);
  const rsrc_t sr = KIND == kWBf16
                        ? wr
                        : make_rsrc(static_cast<const char*>(a.w.scale) + e * sbytes, sbytes);
  const rsrc_t xr = make_rsrc(a.x, int64_t(a.rows) * a.K * 2);
  const int n0 = blockIdx.x * (C * 16);
  uint32_t woff[NT], soff[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int c = n0 + (nt % C) * 16 + (lane & 15);
    const int r = GATED && nt >= C ? a.N + c : c;
    woff[nt] = c < a.N ? uint32_t(r) * uint32_t(wrow) : kOob;
    soff[nt] = c < a.N ? uint32_t(r) * uint32_t(srow) : kOob;
  }
  const int nkb = (a.K + kBlockK - 1) / kBlockK;
  for (int c0 = 0; c0 < m; c0 += 16 * MT) {
    uint32_t xoff[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int i = c0 + mt * 16 + (lane & 15);
      xoff[mt] = i < m ? uint32_t(sp.list[i] / a.top) * uint32_t(a.K * 2) : kOob;
    }
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    few_tile<KIND, NT, MT, 1, D>(xr, wr, sr, xoff, woff, soff, 0u, a.K, wave, nkb,
                                 kWavesPerBlock, acc);
    if (c0 > 0) __syncthreads();                     // the last chunk's sums have been read
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          red[wave][mt * 16 + (lane >> 4) * 4 + i][nt * 16 + (lane & 15)] = acc[mt][nt][i];
    __syncthreads();
    const int mc = m - c0 < 16 * MT ? m - c0 : 16 * MT;
    __bf16* y = static_cast<__bf16*>(a.y);
    for (int i = threadIdx.x; i < mc * (C * 16); i += kBlock) {
      const int r = i / (C * 16), c = i % (C * 16);
      if (n0 + c >= a.N) continue;
      float v = 0.f, u = 0.f;
#pragma unroll
      for (int w = 0; w < kWavesPerBlock; ++w) {
        v += red[w][r][c];
        if (GATED) u += red[w][r][C * 16 + c];
      }
      const int slot = sp.list[c0 + r];
      if (GATED) {
        // h in two bf16 parts, 16 significant bits together: bf16 alone would
        // double the squared error of the layer's output.  The first part is
        // cut, not rounded, so that it stays finite where h is.
        v = v / (1.0f + __expf(-v)) * u;
        const bool finite = __builtin_fabsf(v) < __builtin_inff();
        const __bf16 hi = finite ? __bf16(__uint_as_float(__float_as_uint(v) & 0xFFFF0000u))
                                 : __bf16(v);
        __bf16* h = y + int64_t(slot) * (2 * a.N) + n0 + c;
        h[0] = hi;
        h[a.N] = __bf16(finite ? v - float(hi) : 0.0f);
      } else {
        y[int64_t(slot) * a.N + n0 + c] = __bf16(v);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Second launch of a layer: the down products and the weighted sum.  A
// workgroup owns 16 output channels of every token, so the sum over a token's
// experts needs no atomics: its eight waves share out (expert, part of the
// channels) and leave each slot's products in LDS, then one thread per
// (token, channel) adds them up in the order of the slots.
// ---------------------------------------------------------------------------
constexpr int kDownWaves = 8;
constexpr int kDownBlock = kDownWaves * kWave;
constexpr int kDownMaxSplit = 8;

struct DownShared {
  int16_t expert[kFewExperts];
  uint16_t first[kFewExperts];
  uint16_t count[kFewExperts];
  uint16_t order[kFewSlots];
  float w[kFewSlots];
  uint8_t local[kFewSlots];
};

template <int KIND, int MT, int D>
__global__ __launch_bounds__(kDownBlock) void few_down_kernel(DownArgs a, int max_split) {
  __shared__ DownShared ds;
  extern __shared__ float prod[];                    // [split][slots][16]
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
  const int slots = a.T * a.K;
  const int most = slots < a.experts ? slots : a.experts;
  const int active = a.plan->active;
  for (int i = tid; i < most; i += kDownBlock) {     // entries past `active` are not used
    ds.expert[i] = int16_t(a.plan->expert[i]);
    ds.first[i] = uint16_t(a.plan->first[i]);
    ds.count[i] = uint16_t(a.plan->count[i]);
  }
  for (int i = tid; i < slots; i += kDownBlock) {
    ds.order[i] = uint16_t(a.plan->order[i]);
    ds.w[i] = a.topk_weights[i];
    ds.local[i] = slot_expert(a.ids64, nullptr, a.first_expert, a.experts, i) >= 0;
  }
  __syncthreads();

  const int nkb = (a.I + kBlockK - 1) / kBlockK;
  // parts per expert: the smallest of 1, 2, 4, 8 that leaves the busiest wave
  // the least to do
  int split = 1;
  {
    int best = (active + kDownWaves - 1) / kDownWaves * kDownMaxSplit;
    for (int s = 2; s <= max_split && s <= nkb; s *= 2) {
      const int cost = (active * s + kDownWaves - 1) / kDownWaves * (kDownMaxSplit / s);
      if (cost < best) best = cost, split = s;
    }
  }
  const int n0 = blockIdx.x * 16;
  const int c = n0 + (lane & 15);
  const int wrow = row_bytes<KIND>(a.I), srow = scale_bytes<KIND>(a.I);
  const int64_t wbytes = int64_t(a.H) * wrow, sbytes = int64_t(a.H) * srow;
  const uint32_t woff[1] = {c < a.H ? uint32_t(c) * uint32_t(wrow) : kOob};
  const uint32_t soff[1] = {c < a.H ? uint32_t(c) * uint32_t(srow) : kOob};
  const rsrc_t xr = make_rsrc(a.h, int64_t(slots) * a.I * 4);
  for (int u = wave; u < active * split; u += kDownWaves) {
    const int i = u / split, part = u % split;
    const int e = __builtin_amdgcn_readfirstlane(int(ds.expert[i]));
    const int m = __builtin_amdgcn_readfirstlane(int(ds.count[i]));
    const int first = __builtin_amdgcn_readfirstlane(int(ds.first[i]));
    const rsrc_t wr = make_rsrc(static_cast<const char*>(a.w.q) + e * wbytes, wbytes);
    const rsrc_t sr = KIND == kWBf16
                          ? wr
                          : make_rsrc(static_cast<const char*>(a.w.scale) + e * sbytes, sbytes);
    for (int c0 = 0; c0 < m; c0 += 16 * MT) {
      uint32_t xoff[MT];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int r = c0 + mt * 16 + (lane & 15);
        xoff[mt] = r < m ? uint32_t(ds.order[first + r]) * uint32_t(a.I * 4) : kOob;
      }
      f32x4 acc[MT][1];
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) acc[mt][0] = f32x4{0.f, 0.f, 0.f, 0.f};
      few_tile<KIND, 1, MT, 2, D>(xr, wr, sr, xoff, woff, soff, uint32_t(a.I * 2), a.I,
                                  part * nkb / split, (part + 1) * nkb / split, 1, acc);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = c0 + mt * 16 + (lane >> 4) * 4 + j;
          if (r < m)
            prod[(part * slots + ds.order[first + r]) * 16 + (lane & 15)] = acc[mt][0][j];
        }
    }
  }
  __syncthreads();
  for (int i = tid; i < a.T * 16; i += kDownBlock) {
    const int t = i >> 4, ch = n0 + (i & 15);
    if (ch >= a.H) continue;
    float sum = 0.f;
    for (int k = 0; k < a.K; ++k) {
      const int s = t * a.K + k;
      if (!ds.local[s]) continue;
      float y = 0.f;
      for (int p = 0; p < split; ++p) y += prod[(p * slots + s) * 16 + (i & 15)];
      sum += ds.w[s] * y;
    }
    const int64_t o = int64_t(t) * a.H + ch;
    if (a.bias0) sum += float(static_cast<const __bf16*>(a.bias0)[o]);
    if (a.bias1) sum += float(static_cast<const __bf16*>(a.bias1)[o]);
    static_cast<__bf16*>(a.out)[o] = __bf16(sum);
  }
}

// ---------------------------------------------------------------------------
// bf16 rows to 4-bit codes and scales.  A lane takes 8 channels (16 bytes in,
// 4 out); the group/8 lanes of a group share its largest magnitude.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t e2m1_code(float v) {
  // nearest of 0 .5 1 1.5 2 3 4 6, ties to the even code
  const float a = __builtin_fabsf(v);
  const uint32_t c = a <= 0.25f ? 0u
                     : a < 0.75f ? 1u
                     : a <= 1.25f ? 2u
                     : a < 1.75f ? 3u
                     : a <= 2.5f ? 4u
                     : a < 3.5f ? 5u
                     : a <= 5.0f ? 6u : 7u;
  return c | ((__float_as_uint(v) >> 28) & 8u);
}

template <bool FP4>
__global__ __launch_bounds__(kBlock) void quantize_w4_kernel(QuantArgs a, int64_t pieces) {
  const int64_t p = int64_t(blockIdx.x) * kBlock + threadIdx.x;
  const bool in = p < pieces;                // a group's lanes are all in or all out
  u32x4 v = {0u, 0u, 0u, 0u};
  if (in) v = static_cast<const u32x4*>(a.w)[p];
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(v[i]);
    f[2 * i + 1] = bf16_hi(v[i]);
  }
  uint32_t mx = 0u;                          // on the bits: NaN above infinity above the rest
#pragma unroll
  for (int i = 0; i < 8; ++i) mx = max(mx, __float_as_uint(f[i]) & 0x7FFFFFFFu);
  const int lanes = a.group / 8;
  for (int o = 1; o < lanes; o <<= 1) mx = max(mx, uint32_t(__shfl_xor(int(mx), o)));
  if (!in) return;
  const float amax = __uint_as_float(mx);
  const bool bad = mx >= 0x7F800000u;
  uint32_t code = 0u;
  const int64_t gi = p / lanes;
  const bool lead = p % lanes == 0;
  if (FP4) {
    uint32_t byte = 0u;
    if (bad) {
      byte = 255u;
    } else if (mx != 0u) {
      const uint32_t u = __float_as_uint(amax / 6.0f);
      // exponent of the next power of two at or above; subnormals give 0 or 1
      byte = (u >> 23) + ((u & 0x7FFFFFu) > (u >> 23 ? 0u : 0x400000u) ? 1u : 0u);
      const float inv = __uint_as_float((254u - byte) << 23);      // 2^(127 - byte), exact
#pragma unroll
      for (int i = 0; i < 8; ++i) code |= e2m1_code(f[i] * inv) << (4 * i);
    }
    if (lead) static_cast<uint8_t*>(a.scale)[gi] = uint8_t(byte);
  } else {
    const float sc = bf16_lo(pack_bf16x2(amax / 7.0f, 0.f));
    code = 0x88888888u;
    if (!bad && sc > 0.f) {
      code = 0u;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float q = fminf(fmaxf(__builtin_rintf(f[i] / sc), -8.f), 7.f);
        code |= uint32_t(int(q) + 8) << (4 * i);
      }
    }
    if (lead) {
      static_cast<uint16_t*>(a.scale)[gi] =
          bad ? uint16_t(0x7FC0) : uint16_t(__float_as_uint(sc) >> 16);
    }
  }
  static_cast<uint32_t*>(a.q)[p] = code;
}

template <int KIND, bool GATED>
hipError_t rows_variant(const FewArgs& a, hipStream_t s) {
  // A first cut: two tiles a wave (a gate and an up tile), 16 rows at a time.
  constexpr int NT = 2;
  constexpr int C = GATED ? NT / 2 : NT;
  const unsigned most = unsigned(a.slots < a.experts ? a.slots : a.experts);
  const dim3 grid(unsigned((a.N + C * 16 - 1) / (C * 16)), most);
  few_rows_kernel<KIND, NT, 1, GATED, 2><<<grid, kBlock, 0, s>>>(a);
  return hipGetLastError();
}

template <bool GATED>
hipError_t rows_kind(const FewArgs& a, hipStream_t s) {
  switch (a.w.kind) {
    case kWBf16: return rows_variant<kWBf16, GATED>(a, s);
    case kWFp4: return rows_variant<kWFp4, GATED>(a, s);
    case kWInt4G32: return rows_variant<kWInt4G32, GATED>(a, s);
    case kWInt4G64: return rows_variant<kWInt4G64, GATED>(a, s);
    default: return rows_variant<kWInt4G128, GATED>(a, s);
  }
}

template <int KIND>
hipError_t down_variant(const DownArgs& a, hipStream_t s) {
  // LDS of the products: 64 bytes a slot and part, at most 64 KiB
  const int slots = a.T * a.K;
  int split = kDownMaxSplit;
  while (split > 1 && split * slots > 1024) split >>= 1;
  few_down_kernel<KIND, 1, 2><<<dim3(unsigned((a.H + 15) / 16)), kDownBlock,
                                size_t(split) * size_t(slots) * 64, s>>>(a, split);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_few_rows(const FewArgs& a, bool gated, hipStream_t s) {
  return gated ? rows_kind<true>(a, s) : rows_kind<false>(a, s);
}

hipError_t launch_few_down(const DownArgs& a, hipStream_t s) {
  switch (a.w.kind) {
    case kWBf16: return down_variant<kWBf16>(a, s);
    case kWFp4: return down_variant<kWFp4>(a, s);
    case kWInt4G32: return down_variant<kWInt4G32>(a, s);
    case kWInt4G64: return down_variant<kWInt4G64>(a, s);
    default: return down_variant<kWInt4G128>(a, s);
  }
}

hipError_t launch_quantize_w4(const QuantArgs& a, hipStream_t s) {
  const int64_t pieces = a.rows * (a.channels / 8);
  // at most 2^31 - 1 workgroups a launch; the caller's size limit keeps below
  const dim3 grid(unsigned((pieces + kBlock - 1) / kBlock));
  if (a.fp4)
    quantize_w4_kernel<true><<<grid, kBlock, 0, s>>>(a, pieces);
  else
    quantize_w4_kernel<false><<<grid, kBlock, 0, s>>>(a, pieces);
  return hipGetLastError();
}

}  // namespace epdc
