// Products of a few rows with their experts' matrices, a whole expert layer
// for a few tokens, and the 4-bit weight quantizer (gfx950, wave64).
//
// With a few rows an expert's matrix is read once and used a handful of
// times, so the weights' bytes bound every kernel here.  The matrix cores do
// the arithmetic all the same: D[row][n] += X[row][k] W[n][k] with
// v_mfma_f32_16x16x32_bf16 takes up to 16 rows at the cost of one, sums
// over the lanes by itself and leaves the vector unit to the 4-bit decoding.
//
// A wave owns 16*NT weight rows n and walks along the channels in stages of
// NV*64 bytes of each row.  Loads are 16 bytes a lane through buffer
// descriptors whose range check returns zeros for the rows past N, the token
// rows past the expert's count and the channels past K, so nothing branches.
// Loads return in order, hence the rows x are fetched as far ahead as the
// weights: both sit in a ring of D stages of registers, and x goes through LDS
// on its way to the matrix cores.
#include "epdc_device.h"
#include "expert_launch.h"

#include <type_traits>

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

template <int KIND>
constexpr bool kIsBf16 = KIND == kWBf16 || KIND == kWBf16Stream;
template <int KIND>
constexpr bool kIsInt4 = KIND == kWInt4G32 || KIND == kWInt4G64 || KIND == kWInt4G128;

// Channels of a 16-byte vector's 64-byte share of a row: 32 bf16 or 128 4-bit.
template <int KIND>
constexpr int kVecK = kIsBf16<KIND> ? 32 : 128;

// Bytes of one weight row and of its scales, and scale bytes per 128 channels.
template <int KIND>
__device__ __forceinline__ int row_bytes(int K) { return kIsBf16<KIND> ? 2 * K : K / 2; }
template <int KIND>
constexpr int kScaleBytes =
    KIND == kWFp4 ? 4 : KIND == kWInt4G32 ? 8 : KIND == kWInt4G64 ? 4 : 2;
template <int KIND>
__device__ __forceinline__ int scale_bytes(int K) { return K / 128 * kScaleBytes<KIND>; }

// Which channels a lane group (the lanes 16g..16g+15) holds.  A lane's 16
// bytes are 8 channels of a bf16 row but 32 of a 4-bit row.  One matrix
// instruction sums over all four lane groups, so a scale that differs between
// them has to be applied before it (fp4: a power of two, exact in bf16) or the
// lanes have to share it: int4 with one scale per 128 channels does; with 32
// or 64 the four dwords are transposed between the lane groups first, which
// leaves instruction j with the channels 32j..32j+31.  kSplit: group g holds
// channels 32g..32g+31 and instruction j their j-th eight; otherwise group g
// holds the g-th eight of instruction j's 32 channels.
template <int KIND>
constexpr bool kSplit = KIND == kWFp4 || KIND == kWInt4G128;

// The 4x4 transposition of dwords between lane groups: dword j of group g
// becomes dword g of group j (row swaps of the two bits of g against j's).
__device__ __forceinline__ u32x4 transpose_groups(u32x4 v) {
  auto a = __builtin_amdgcn_permlane32_swap(v.x, v.z, false, false);
  auto b = __builtin_amdgcn_permlane32_swap(v.y, v.w, false, false);
  auto c = __builtin_amdgcn_permlane16_swap(a[0], b[0], false, false);
  auto d = __builtin_amdgcn_permlane16_swap(a[1], b[1], false, false);
  return u32x4{c[0], c[1], d[0], d[1]};
}

// out[b]: the word that lane group b (of the first NV) holds, in every group.
template <int NV>
__device__ __forceinline__ void spread_groups(uint32_t w, uint32_t (&out)[NV]) {
  if constexpr (NV == 4) {
    auto h = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
    auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
    out[0] = lo[0];
    out[1] = lo[1];
    out[2] = hi[0];
    out[3] = hi[1];
  } else {                       // two groups hold each word already
    auto p = __builtin_amdgcn_permlane16_swap(w, w, false, false);
    out[0] = p[0];
    out[1] = p[1];
  }
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

// Eight int4 codes c as the bf16 numbers (c - 8) / 16, exact.  c ^ 8 is c - 8 in
// two's complement, which a conversion instruction reads from the low four bits
// of a byte; its fp32 result has the bf16 one in the upper half.  A zero weight
// is a zero, so its channel drops out of the sum whatever its size, and a group
// of 128 channels below 2^122 sums to less than 2^128.  (16 + c takes eight
// operations instead of fourteen, but 24 times the row's sum has to come off
// again, in products of its own: beside a large channel the others lose their
// low bits, and sums leave fp32 earlier.  128 tokens, 32 experts of 7168 x 2048
// in groups of 128, a layer, take 305 us this way and 323 that way; one matrix of
// 7168 x 7168 in groups of 32 and 16 rows 26 and 24.)
__device__ __forceinline__ u32x4 decode_int4(uint32_t d) {
  uint32_t lo = d ^ 0x88888888u;
  uint32_t hi = lo >> 4;
  asm("" : "+v"(lo), "+v"(hi));          // kept apart: the conversions then pick their bytes
  u32x4 out;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = i ? (lo >> (8 * i)) & 0xFFu : lo, b = i ? (hi >> (8 * i)) & 0xFFu : hi;
    out[i] = __builtin_amdgcn_perm(__float_as_uint(__builtin_amdgcn_cvt_off_f32_i4(int(b))),
                                   __float_as_uint(__builtin_amdgcn_cvt_off_f32_i4(int(a))),
                                   0x07060302u);
  }
  return out;
}
// What a 1 of the accumulated sums stands for.
template <int KIND>
constexpr float kUnit = kIsInt4<KIND> ? 16.0f : 1.0f;

// ---------------------------------------------------------------------------
// A stage of weights: NV 16-byte vectors a lane of each tile of 16 rows.
// Vector q of lane group g is bytes 64q + 16g.. of the stage.  Loads that take
// whole 128-byte lines may carry the non-temporal hint, which moves memory
// faster (a read of 125 MB: 6.1 against 5.0 TB/s); with 64 bytes of 16 rows the
// hint makes it slowest of all (4.1).  So a pair of vectors is loaded as rows
// 0-7 and rows 8-15, the lanes n >= 8 of a tile taking the second vector's
// share, and the halves change places afterwards.
// One scale load covers the stage, lane group g taking vector g's: loaded
// vector by vector, the few bytes of each row cost more requests than the
// weights (fp4 at 7168 channels: 38 against 26 us).
// ---------------------------------------------------------------------------
template <int KIND, int NT, int NV>
struct Stage {
  u32x4 v[NT][NV];
  uint32_t s[NT][2];
};

// A lane's byte offsets into a matrix (kOob: no such row), its share of the
// stage included: its two weight rows and its scale row of each tile.
template <int NT>
struct Rows {
  uint32_t w[NT][2];
  uint32_t s[NT];
};

// Tiles of output channels c0.. below `limit`, `tiles` of them before the next
// set (the up rows); tile t starts at matrix row tile_row(t).
template <int KIND, int NT, int NV, typename TileRow>
__device__ __forceinline__ void set_rows(Rows<NT>& r, int K, TileRow tile_row, int c0, int limit,
                                         int tiles) {
  const int n = lane_id() & 15, g = lane_id() >> 4;
  const int wrow = row_bytes<KIND>(K), srow = scale_bytes<KIND>(K);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int c = c0 + (nt % tiles) * 16;              // output channel of the tile's row 0
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = (n & 7) + 8 * h;
      r.w[nt][h] = c + k < limit ? uint32_t(tile_row(nt) + k) * uint32_t(wrow) +
                                       uint32_t((n >> 3) * 64 + g * 16)
                                 : kOob;
    }
    r.s[nt] = c + n < limit ? uint32_t(tile_row(nt) + n) * uint32_t(srow) +
                                  uint32_t((g & (NV - 1)) * kScaleBytes<KIND>)
                            : kOob;
  }
}

// Stage `st` of the rows, or zeros if it is not `in`.  The stage's offset is
// the same for every lane and goes into the scalar offset; what remains a
// lane's business is whether its channels lie below K.
template <int KIND, int NT, int NV>
__device__ __forceinline__ void load_stage(Stage<KIND, NT, NV>& stage, rsrc_t wr, rsrc_t sr,
                                           const Rows<NT>& rows, int K, int st, bool in) {
  const int g = lane_id() >> 4, up = (lane_id() >> 3) & 1;
  const int left = in ? K - st * (NV * kVecK<KIND>) : 0;         // channels from the stage on
  const int so = in ? st * (NV * 64) : 0;
  const int ss = in ? st * (NV * kScaleBytes<KIND>) : 0;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int i = 0; i < NV; i += 2) {
      const bool ok = (i + up) * kVecK<KIND> + (kIsBf16<KIND> ? g * 8 : 0) < left;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        stage.v[nt][i + h] = __builtin_amdgcn_raw_buffer_load_b128(
            wr, (ok ? rows.w[nt][h] : kOob) + i * 64, so, KIND == kWBf16Stream ? 2 : 0);
    }
    if constexpr (!kIsBf16<KIND>) {
      const uint32_t off = (g & (NV - 1)) * 128 < left ? rows.s[nt] : kOob;
      if constexpr (KIND == kWInt4G128) {
        stage.s[nt][0] = uint32_t(uint16_t(__builtin_amdgcn_raw_buffer_load_b16(sr, off, ss, 0)));
      } else if constexpr (KIND == kWInt4G32) {
        const auto sc = __builtin_amdgcn_raw_buffer_load_b64(sr, off, ss, 0);
        stage.s[nt][0] = sc[0];
        stage.s[nt][1] = sc[1];
      } else {
        stage.s[nt][0] = __builtin_amdgcn_raw_buffer_load_b32(sr, off, ss, 0);
      }
    }
  }
}

// The halves of a pair of loads change places: lanes n < 8 give their part of
// row n + 8 to lane n + 8 and get the second vector of their own row.
__device__ __forceinline__ void exchange_halves(u32x4& a, u32x4& b) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr int kRor8 = 0x128;                       // rotate by 8 within 16 lanes
    const int x = int(a[i]), y = int(b[i]);
    a[i] = uint32_t(__builtin_amdgcn_update_dpp(x, y, kRor8, 0xF, 0xC, false));
    b[i] = uint32_t(__builtin_amdgcn_update_dpp(y, x, kRor8, 0xF, 0x3, false));
  }
}

// The scale words of a stage's vectors, one set for every lane.
template <int KIND, int NT, int NV>
struct Scales {
  uint32_t s0[NT][NV], s1[NT][NV];
};

// A stage as loaded, put in order.
template <int KIND, int NT, int NV>
__device__ __forceinline__ void open_stage(Stage<KIND, NT, NV>& st, Scales<KIND, NT, NV>& sc) {
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int q = 0; q < NV; q += 2) exchange_halves(st.v[nt][q], st.v[nt][q + 1]);
    if constexpr (!kIsBf16<KIND>) spread_groups<NV>(st.s[nt][0], sc.s0[nt]);
    if constexpr (KIND == kWInt4G32) spread_groups<NV>(st.s[nt][1], sc.s1[nt]);
  }
}

// Vector q's products into acc: MT tiles of 16 rows x against NT tiles of 16
// weight rows.  A row x is the sum of XP bf16 rows.  x(mt, p, j): the fragment
// of row tile mt, part p, for product j of the vector (bf16: the only one), as
// it lies in memory; use(mt): whether the tile has rows at all.
template <int KIND, int NT, int NV, int MT, int XP, typename X, typename Use>
__device__ __forceinline__ void vector_products(const Stage<KIND, NT, NV>& st,
                                                const Scales<KIND, NT, NV>& scales, int q, X x,
                                                Use use, f32x4 (&acc)[MT][NT]) {
  if constexpr (kIsBf16<KIND>) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (!use(mt)) continue;
#pragma unroll
      for (int p = 0; p < XP; ++p) {
        const u32x4 a = x(mt, p, 0);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = mfma(a, st.v[nt][q], acc[mt][nt]);
      }
    }
  } else if constexpr (KIND == kWFp4) {
    u32x4 b[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint32_t byte = scales.s0[nt][q] >> ((lane_id() >> 4) * 8);   // lane group g: byte g
      const float sc = __uint_as_float((byte << 23) & 0x7F800000u);
#pragma unroll
      for (int j = 0; j < 4; ++j) b[nt][j] = decode_fp4(st.v[nt][q][j], sc);
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      if (!use(mt)) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int p = 0; p < XP; ++p) {
          const u32x4 a = x(mt, p, j);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = mfma(a, b[nt][j], acc[mt][nt]);
        }
    }
  } else {
    constexpr int Q = KIND == kWInt4G128 ? 1 : KIND == kWInt4G64 ? 2 : 4;   // groups a vector
    constexpr int J = 4 / Q;                                                // products a group
    u32x4 v[NT], b[NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      v[nt] = kSplit<KIND> ? st.v[nt][q] : transpose_groups(st.v[nt][q]);
    auto decode = [&](int j) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) b[nt][j] = decode_int4(v[nt][j]);
    };
    auto products = [&](int mt, int i) {
      u32x4 a[J][XP];
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int p = 0; p < XP; ++p) a[j][p] = x(mt, p, i * J + j);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        f32x4 part = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int p = 0; p < XP; ++p) part = mfma(a[j][p], b[nt][i * J + j], part);
        const uint32_t sw = i < 2 ? scales.s0[nt][q] : scales.s1[nt][q];
        const float sc = Q > 1 && (i & 1) ? bf16_hi(sw) : bf16_lo(sw);
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[mt][nt][k] = __builtin_fmaf(sc, part[k], acc[mt][nt][k]);
      }
    };
    // Decoded all at once, one group's products cover the wait for another's (42
    // rows, 2 matrices of 4608 x 3328 in groups of 32, one weight tile a wave: 19
    // us against 24 group by group; 16 rows of one of 7168 x 7168: 26.5 against
    // 31.5).  The registers do not hold that for two weight tiles and eight or
    // more fragments of x a vector (64 tokens, 32 experts of 7168 x 2048 in groups
    // of 32, a layer: 323 us group by group, 575 all at once).
    if constexpr (NT == 1 || Q * MT * XP < 8) {
#pragma unroll
      for (int j = 0; j < 4; ++j) decode(j);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        if (!use(mt)) continue;
#pragma unroll
        for (int i = 0; i < Q; ++i) products(mt, i);
      }
    } else {
#pragma unroll
      for (int i = 0; i < Q; ++i) {
#pragma unroll
        for (int j = 0; j < J; ++j) decode(i * J + j);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          if (use(mt)) products(mt, i);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Up to four rows x for one wave alone: the stage's channels of the rows go
// through an LDS corner of the wave's own, 128 channels of all four a load.
// Rows past the fourth of a fragment repeat the four, and their products are
// not used.  A wave's LDS accesses stay in order, so no barrier is needed.
// ---------------------------------------------------------------------------
// Blocks of 128 channels of x a stage needs.
template <int KIND, int NV>
constexpr int kXBlocks = kIsBf16<KIND> ? NV / 4 : NV;
// 16-byte pieces from row to row: the four rows and four lane groups that a
// fragment reads at once then lie in different banks.
template <int KIND>
constexpr int kXPitch = kSplit<KIND> ? 17 : 20;
template <int KIND, int NV, int XP>
constexpr int kXPieces = kXBlocks<KIND, NV> * XP * kFewRows * kXPitch<KIND>;

template <int KIND, int NT, int NV, int XP, int D>
__device__ __forceinline__ void own_tile(rsrc_t xr, uint32_t xoff, int plane, u32x4* xs,
                                         rsrc_t wr, rsrc_t sr, const Rows<NT>& rows, int K, int st0,
                                         int st1, int step, f32x4 (&acc)[1][NT]) {
  constexpr int XB = kXBlocks<KIND, NV>;
  static_assert(!kIsBf16<KIND> || NV % 4 == 0, "a stage holds whole blocks of x");
  const int lane = lane_id();
  Stage<KIND, NT, NV> w[D];
  u32x4 xb[D][XB][XP];
  auto load = [&](int d, int st) {
    const bool in = st < st1;
    const int left = in ? K - st * (NV * kVecK<KIND>) : 0;
    const int so = in ? st * (NV * kVecK<KIND> * 2) : 0;
    // xoff: the lane's piece (lane % 16) of 128 channels of row lane / 16
#pragma unroll
    for (int b = 0; b < XB; ++b) {
      const uint32_t off = (b * 128 + (lane & 15) * 8 < left ? xoff : kOob) + b * 256;
#pragma unroll
      for (int p = 0; p < XP; ++p)
        xb[d][b][p] = __builtin_amdgcn_raw_buffer_load_b128(xr, off, so + p * plane, 0);
    }
    load_stage<KIND, NT, NV>(w[d], wr, sr, rows, K, st, in);
  };
#pragma unroll
  for (int d = 0; d < D; ++d) {
    load(d, st0 + d * step);
    __builtin_amdgcn_sched_barrier(0);
  }
  for (int st = st0; st < st1; st += D * step) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
#pragma unroll
      for (int b = 0; b < XB; ++b)
#pragma unroll
        for (int p = 0; p < XP; ++p)
          xs[((b * XP + p) * kFewRows + (lane >> 4)) * kXPitch<KIND> + (lane & 15)] =
              xb[d][b][p];
      __builtin_amdgcn_wave_barrier();
      Scales<KIND, NT, NV> sc;
      open_stage<KIND, NT, NV>(w[d], sc);
#pragma unroll
      for (int q = 0; q < NV; ++q)
        vector_products<KIND, NT, NV, 1, XP>(
            w[d], sc, q,
            [&](int, int p, int j) {
              const int g = lane >> 4;
              const int b = kIsBf16<KIND> ? q / 4 : q, i = kIsBf16<KIND> ? q % 4 : j;
              const int piece = kSplit<KIND> ? g * 4 + i : i * 4 + g;
              return xs[((b * XP + p) * kFewRows + (lane & 3)) * kXPitch<KIND> + piece];
            },
            [](int) { return true; }, acc);
      __builtin_amdgcn_wave_barrier();
      // kept in this order, so that a stage's wait leaves the later stages'
      // loads in flight
      __builtin_amdgcn_sched_barrier(0);
      load(d, st + (d + D) * step);
      __builtin_amdgcn_sched_barrier(0);
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
template <int BLOCK>
__device__ __forceinline__ int find_expert(SharedPlan& sp, const FewArgs& a, int y, int& expert,
                                           int& first, int& active) {
  const int tid = threadIdx.x;
  const int lane = lane_id();
  if (tid < kFewExperts / 32) sp.bits[tid] = 0u;
  __syncthreads();
  for (int s = tid; s < a.slots; s += BLOCK) {
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

// Zeros for the rows that name no expert, C channels from n0 on.
template <int C, int BLOCK>
__device__ __forceinline__ void zero_unnamed(const SharedPlan& sp, const FewArgs& a, int n0) {
  for (int i = threadIdx.x; i < a.slots * C; i += BLOCK) {
    const int s = i / C, c = n0 + i % C;
    if (sp.id[s] < 0 && c < a.N) static_cast<__bf16*>(a.y)[int64_t(s) * a.N + c] = __bf16(0.0f);
  }
}

// A layer's first launch leaves the plan for the second.
template <int BLOCK>
__device__ __forceinline__ void write_plan(const SharedPlan& sp, const FewArgs& a, int e, int first,
                                           int m, int active) {
  if (threadIdx.x == 0) {
    if (blockIdx.y == 0) a.plan->active = active;
    if (m > 0) {
      a.plan->expert[blockIdx.y] = e;
      a.plan->first[blockIdx.y] = first;
      a.plan->count[blockIdx.y] = m;
    }
  }
  for (int i = threadIdx.x; i < m; i += BLOCK) a.plan->order[first + i] = sp.list[i];
}

// h = silu(g) * u in two bf16 parts, off by at most 2^-17 of it: bf16 alone would
// double the squared error of the layer's output, a third part would take half
// as many products again.  The first part is rounded (cut, it would leave 2^-16),
// but cut where rounding would make it infinite.
__device__ __forceinline__ void store_h(__bf16* row, int64_t N, float g, float u) {
  const float v = g / (1.0f + __expf(-g)) * u;
  const bool finite = __builtin_fabsf(v) < __builtin_inff();
  __bf16 hi = __bf16(v);
  if (finite && __builtin_fabsf(float(hi)) == __builtin_inff())
    hi = __bf16(__uint_as_float(__float_as_uint(v) & 0xFFFF0000u));
  row[0] = hi;
  row[N] = __bf16(finite ? v - float(hi) : 0.0f);
}

// Descriptors of expert e's matrix and its scales.
template <int KIND>
__device__ __forceinline__ rsrc_t matrix_rsrc(const Weights& w, int e, int rows, int K) {
  const int64_t bytes = int64_t(rows) * row_bytes<KIND>(K);
  return make_rsrc(static_cast<const char*>(w.q) + e * bytes, bytes);
}
template <int KIND>
__device__ __forceinline__ rsrc_t scale_rsrc(const Weights& w, int e, int rows, int K) {
  if (kIsBf16<KIND>) return make_rsrc(w.q, 0);        // not read
  const int64_t bytes = int64_t(rows) * scale_bytes<KIND>(K);
  return make_rsrc(static_cast<const char*>(w.scale) + e * bytes, bytes);
}

// ---------------------------------------------------------------------------
// Up to four rows an expert at a time: grid (tiles of weight rows, experts in
// use at most).  The W waves of a workgroup take every W-th stage of the
// channels each, which spreads a small matrix over more of the chip, and add
// up through LDS in a fixed order.  kOutGated: a tile is half gate and half up
// rows.  Bound by the weights and, under 10 us, by the launch and the first
// loads: the gate and up rows of 8 fp4 experts of 7168 x 2048 for one token, 125
// MB, 30 us (4.2 TB/s); one row, int4 4096 x 7168, 15 MB, 8.2 us, of which the
// waves wait for 56 %: each has three or four stages, two rounds of loads one
// after the other, and the first starts after find_expert.
// ---------------------------------------------------------------------------
template <int KIND, int NT, int NV, int W, int OUT, int D>
__global__ __launch_bounds__(W * kWave) void few_thin_kernel(FewArgs a) {
  constexpr bool GATED = OUT == kOutGated;
  constexpr int C = GATED ? NT / 2 : NT;               // tiles of output channels
  constexpr int XP = OUT == kOutF32 ? 2 : 1;           // h has two parts
  __shared__ SharedPlan sp;
  __shared__ u32x4 xs[W][kXPieces<KIND, NV, XP>];
  __shared__ float red[W][kFewRows][NT * 16];
  const int lane = lane_id(), wave = wave_id();
  int e = 0, first = 0, active = 0;
  int m = find_expert<W * kWave>(sp, a, blockIdx.y, e, first, active);
  e = __builtin_amdgcn_readfirstlane(e);
  m = __builtin_amdgcn_readfirstlane(m);
  if (GATED && blockIdx.x == 0) write_plan<W * kWave>(sp, a, e, first, m, active);
  const int n0 = blockIdx.x * (C * 16);
  if (OUT == kOutBf16 && blockIdx.y == 0) zero_unnamed<C * 16, W * kWave>(sp, a, n0);
  if (m == 0) return;

  const int all = GATED ? 2 * a.N : a.N;
  const rsrc_t wr = matrix_rsrc<KIND>(a.w, e, all, a.K);
  const rsrc_t sr = scale_rsrc<KIND>(a.w, e, all, a.K);
  const rsrc_t xr = make_rsrc(a.x, int64_t(a.rows) * a.K * (2 * XP));
  Rows<NT> rows;
  set_rows<KIND, NT, NV>(
      rows, a.K, [&](int nt) { return n0 + (nt % C) * 16 + (nt >= C ? a.N : 0); }, n0, a.N, C);
  const int stages = (a.K + NV * kVecK<KIND> - 1) / (NV * kVecK<KIND>);
  for (int c0 = 0; c0 < m; c0 += kFewRows) {
    const int i = c0 + (lane >> 4);
    const uint32_t xoff = i < m ? uint32_t(sp.list[i] / a.top) * uint32_t(a.K * 2 * XP) +
                                      uint32_t(lane & 15) * 16u
                                : kOob;
    f32x4 acc[1][NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) acc[0][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    own_tile<KIND, NT, NV, XP, D>(xr, xoff, a.K * 2, xs[wave], wr, sr, rows, a.K, wave, stages, W,
                                  acc);
    if (c0 > 0) __syncthreads();                       // the last rows' sums have been read
    if (lane < 16) {                                   // lane l: channel l of rows 0..3
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int k = 0; k < kFewRows; ++k)
          red[wave][k][nt * 16 + lane] = kUnit<KIND> * acc[0][nt][k];
    }
    __syncthreads();
    const int mc = m - c0 < kFewRows ? m - c0 : kFewRows;
    for (int k = threadIdx.x; k < mc * (C * 16); k += W * kWave) {
      const int r = k / (C * 16), c = k % (C * 16);
      if (n0 + c >= a.N) continue;
      float v = 0.f, u = 0.f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        v += red[w][r][c];
        if (GATED) u += red[w][r][C * 16 + c];
      }
      const int64_t slot = sp.list[c0 + r];
      if constexpr (GATED)
        store_h(static_cast<__bf16*>(a.y) + slot * (2 * a.N) + n0 + c, a.N, v, u);
      else if constexpr (OUT == kOutBf16)
        static_cast<__bf16*>(a.y)[slot * a.N + n0 + c] = __bf16(v);
      else
        static_cast<float*>(a.y)[slot * a.N + n0 + c] = v;
    }
  }
}

__device__ __forceinline__ void lds_barrier() {
  // LDS accesses done, then the barrier; loads from memory stay in flight
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// ---------------------------------------------------------------------------
// The same for more rows: the four waves of a workgroup own different weight
// rows and share the rows x, which each fetches its part of and passes on
// through LDS, stage by stage.  A row x then comes out of the L2 once for
// 64*NT weight rows.  bf16 is bound by the weights: 48 rows, 8 matrices of 7168
// x 2048, 235 MB, 45 us (5.2 TB/s) a call.  32 rows for each of 32 int4 experts of
// 7168 x 2048 take 192 us (gate and up) and 165 us (down): at a vector instruction
// per four cycles and a matrix instruction per sixteen, the former would take 71
// and 43 us alone, the latter 29 and 29.  The waves wait for memory, LDS and
// barriers 28 and 39 % of their time: the registers allow two waves a SIMD, which
// do not cover it.  Eight instances spill registers to scratch memory (int4 in
// groups of 32 with two weight tiles and two or three row tiles, 9 to 32, in the
// down product 29 and 65; in groups of 64 and 128 the down product with three
// row tiles, 6 and 8: 15 of the 44 MB that the down product above writes).
// ---------------------------------------------------------------------------
template <int KIND, int NT, int NV, int MT, int XP, int OUT, int D>
__global__ __launch_bounds__(kBlock, 2) void few_wide_kernel(FewArgs a) {
  constexpr bool GATED = OUT == kOutGated;
  constexpr int C = GATED ? NT / 2 : NT;               // tiles of output channels a wave
  constexpr int XB = kXBlocks<KIND, NV>;
  static_assert(D * XB % 2 == 0, "the two buffers of x take turns");
  __shared__ SharedPlan sp;
  __shared__ u32x4 xs[2][MT][XP][4][kWave];
  const int lane = lane_id(), wave = wave_id();
  int e = 0, first = 0, active = 0;
  int m = find_expert<kBlock>(sp, a, blockIdx.y, e, first, active);
  e = __builtin_amdgcn_readfirstlane(e);
  m = __builtin_amdgcn_readfirstlane(m);
  if (GATED && blockIdx.x == 0) write_plan<kBlock>(sp, a, e, first, m, active);
  if (OUT == kOutBf16 && blockIdx.y == 0)
    zero_unnamed<C * 16 * kWavesPerBlock, kBlock>(sp, a, blockIdx.x * (C * 16 * kWavesPerBlock));
  if (m == 0) return;

  const int all = GATED ? 2 * a.N : a.N;
  const rsrc_t wr = matrix_rsrc<KIND>(a.w, e, all, a.K);
  const rsrc_t sr = scale_rsrc<KIND>(a.w, e, all, a.K);
  const rsrc_t xr = make_rsrc(a.x, int64_t(a.rows) * a.K * (2 * XP));
  const int n0 = (blockIdx.x * kWavesPerBlock + wave) * (C * 16);
  Rows<NT> rows;
  set_rows<KIND, NT, NV>(
      rows, a.K, [&](int nt) { return n0 + (nt % C) * 16 + (nt >= C ? a.N : 0); }, n0, a.N, C);
  const int stages = (a.K + NV * kVecK<KIND> - 1) / (NV * kVecK<KIND>);
  for (int c0 = 0; c0 < m; c0 += 16 * MT) {
    const int left = m - c0;
    // This wave fetches rows 4*wave.. of every tile, 256 bytes of four rows a
    // load.  A fragment is 64 pieces of 16 bytes, g*16 + row for lane group g;
    // piece c goes into fragment and group (c % 4, c / 4) or the other way
    // round, and its place among the group's 16 turns by c: writes (one row,
    // 16 pieces) and reads (one piece, 16 rows) both reach all the banks.
    const int row = wave * 4 + (lane >> 4), piece = lane & 15;
    const int frag = kSplit<KIND> ? piece & 3 : piece >> 2;
    const int group = kSplit<KIND> ? piece >> 2 : piece & 3;
    const int to = group * 16 + ((row + piece) & 15);
    uint32_t xoff[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
      const int i = c0 + mt * 16 + row;
      xoff[mt] = i < m ? uint32_t(sp.list[i] / a.top) * uint32_t(a.K * 2 * XP) +
                             uint32_t(piece * 16)
                       : kOob;
    }
    f32x4 acc[MT][NT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
    Stage<KIND, NT, NV> w[D];
    u32x4 xb[D][MT][XP][XB];
    auto load = [&](int d, int st) {
      const bool in = st < stages;
      const int left = in ? a.K - st * (NV * kVecK<KIND>) : 0;
      const int so = in ? st * (NV * kVecK<KIND> * 2) : 0;
      const int mine = piece * 8;                      // the lane's channel of every 128
#pragma unroll
      for (int b = 0; b < XB; ++b) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          const uint32_t off = (b * 128 + mine < left ? xoff[mt] : kOob) + b * 256;
#pragma unroll
          for (int p = 0; p < XP; ++p)
            xb[d][mt][p][b] =
                __builtin_amdgcn_raw_buffer_load_b128(xr, off, so + p * (2 * a.K), 0);
        }
      }
      load_stage<KIND, NT, NV>(w[d], wr, sr, rows, a.K, st, in);
    };
#pragma unroll
    for (int d = 0; d < D; ++d) {
      load(d, d);
      __builtin_amdgcn_sched_barrier(0);
    }
    for (int st = 0; st < stages; st += D) {
#pragma unroll
      for (int d = 0; d < D; ++d) {
        Scales<KIND, NT, NV> sc;
        open_stage<KIND, NT, NV>(w[d], sc);
#pragma unroll
        for (int b = 0; b < XB; ++b) {
          // the buffers alternate over the whole loop (D * XB is even): one is
          // written again only after the barrier that follows its last reads
          const int buf = (d * XB + b) & 1;
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int p = 0; p < XP; ++p) xs[buf][mt][p][frag][to] = xb[d][mt][p][b];
          lds_barrier();
#pragma unroll
          for (int q = b * (NV / XB); q < (b + 1) * (NV / XB); ++q)
            vector_products<KIND, NT, NV, MT, XP>(
                w[d], sc, q,
                [&](int mt, int p, int j) {
                  const int f = kIsBf16<KIND> ? q % 4 : j, g = lane >> 4;
                  const int c = kSplit<KIND> ? g * 4 + f : f * 4 + g;
                  return xs[buf][mt][p][f][g * 16 + ((lane + c) & 15)];
                },
                [&](int mt) { return mt == 0 || mt * 16 < left; }, acc);
        }
        __builtin_amdgcn_sched_barrier(0);             // as in own_tile
        load(d, st + d + D);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    lds_barrier();                                     // the next rows write the first buffer
    // lane l holds channel l % 16 of rows 4 * (l / 16) + 0..3 of each tile
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = mt * 16 + (lane >> 4) * 4 + i;
        if (r >= left) continue;
        const int64_t slot = sp.list[c0 + r];
#pragma unroll
        for (int t = 0; t < C; ++t) {
          const int c = n0 + t * 16 + (lane & 15);
          if (c >= a.N) continue;
          if constexpr (OUT == kOutGated)
            store_h(static_cast<__bf16*>(a.y) + slot * (2 * a.N) + c, a.N,
                    kUnit<KIND> * acc[mt][t][i], kUnit<KIND> * acc[mt][C + t][i]);
          else if constexpr (OUT == kOutBf16)
            static_cast<__bf16*>(a.y)[slot * a.N + c] = __bf16(kUnit<KIND> * acc[mt][t][i]);
          else
            static_cast<float*>(a.y)[slot * a.N + c] = kUnit<KIND> * acc[mt][t][i];
        }
      }
  }
}

// ---------------------------------------------------------------------------
// Second launch of a layer of a few slots: the down products and the weighted
// sum.  A workgroup owns 16*NT output channels of every token, so the sum over
// a token's experts needs no atomics: its eight waves share out (expert, part of
// the channels) and leave each slot's products in LDS, then one thread per
// (token, channel) adds them up in the order of the slots.  One token, 8 fp4
// experts of 7168 x 2048: 62 MB in 20 us (3.1 TB/s), some 5 us of it the launch
// and the first loads.
// ---------------------------------------------------------------------------
constexpr int kDownWaves = 8;
constexpr int kDownBlock = kDownWaves * kWave;
constexpr int kDownMaxSplit = 8;

template <int KIND, int NT, int NV, int D>
__global__ __launch_bounds__(kDownBlock) void few_down_kernel(DownArgs a) {
  extern __shared__ float prod[];                      // [split][slots][C]
  __shared__ u32x4 xs[kDownWaves][kXPieces<KIND, NV, 2>];
  __shared__ int16_t expert[kDownSlots], order[kDownSlots], first[kDownSlots], count[kDownSlots];
  __shared__ float weight[kDownSlots];
  __shared__ uint8_t local[kDownSlots];
  constexpr int C = NT * 16;
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
  const int slots = a.T * a.K;
  const int active = a.plan->active;
  if (tid < slots) {                                   // entries past `active` are not used
    expert[tid] = int16_t(a.plan->expert[tid]);
    first[tid] = int16_t(a.plan->first[tid]);
    count[tid] = int16_t(a.plan->count[tid]);
    order[tid] = int16_t(a.plan->order[tid]);
    weight[tid] = a.topk_weights[tid];
    local[tid] = slot_expert(a.ids64, nullptr, a.first_expert, a.experts, tid) >= 0;
  }
  __syncthreads();

  const int stages = (a.I + NV * kVecK<KIND> - 1) / (NV * kVecK<KIND>);
  // parts per expert: the smallest of 1, 2, 4, 8 that leaves the busiest wave
  // the least to do
  int split = 1;
  {
    int best = (active + kDownWaves - 1) / kDownWaves * kDownMaxSplit;
    for (int s = 2; s <= kDownMaxSplit && s <= stages; s *= 2) {
      const int cost = (active * s + kDownWaves - 1) / kDownWaves * (kDownMaxSplit / s);
      if (cost < best) best = cost, split = s;
    }
  }
  const int n0 = blockIdx.x * C;
  Rows<NT> rows;
  set_rows<KIND, NT, NV>(rows, a.I, [&](int nt) { return n0 + nt * 16; }, n0, a.H, NT);
  const rsrc_t xr = make_rsrc(a.h, int64_t(slots) * a.I * 4);
  for (int u = wave; u < active * split; u += kDownWaves) {
    const int i = u / split, part = u % split;
    const int e = __builtin_amdgcn_readfirstlane(int(expert[i]));
    const int m = __builtin_amdgcn_readfirstlane(int(count[i]));
    const int f = __builtin_amdgcn_readfirstlane(int(first[i]));
    const rsrc_t wr = matrix_rsrc<KIND>(a.w, e, a.H, a.I);
    const rsrc_t sr = scale_rsrc<KIND>(a.w, e, a.H, a.I);
    for (int c0 = 0; c0 < m; c0 += kFewRows) {
      const int r = c0 + (lane >> 4);
      const uint32_t xoff =
          r < m ? uint32_t(order[f + r]) * uint32_t(a.I * 4) + uint32_t(lane & 15) * 16u : kOob;
      f32x4 acc[1][NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[0][nt] = f32x4{0.f, 0.f, 0.f, 0.f};
      own_tile<KIND, NT, NV, 2, D>(xr, xoff, a.I * 2, xs[wave], wr, sr, rows, a.I,
                                  part * stages / split, (part + 1) * stages / split, 1, acc);
      if (lane < 16) {
#pragma unroll
        for (int k = 0; k < kFewRows; ++k)
          if (c0 + k < m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              prod[(part * slots + order[f + c0 + k]) * C + nt * 16 + lane] =
                  kUnit<KIND> * acc[0][nt][k];
      }
    }
  }
  __syncthreads();
  for (int i = tid; i < a.T * C; i += kDownBlock) {
    const int t = i / C, ch = n0 + i % C;
    if (ch >= a.H) continue;
    float sum = 0.f;
    for (int k = 0; k < a.K; ++k) {
      const int s = t * a.K + k;
      if (!local[s]) continue;
      float y = 0.f;
      for (int p = 0; p < split; ++p) y += prod[(p * slots + s) * C + i % C];
      sum += weight[s] * y;
    }
    const int64_t o = int64_t(t) * a.H + ch;
    if (a.bias0) sum += float(static_cast<const __bf16*>(a.bias0)[o]);
    if (a.bias1) sum += float(static_cast<const __bf16*>(a.bias1)[o]);
    static_cast<__bf16*>(a.out)[o] = __bf16(sum);
  }
}

// The weighted sum of the slots' products y [slots, H], where the down products
// are a launch of their own: one thread per token and four channels.
__global__ __launch_bounds__(kBlock) void few_sum_kernel(DownArgs a) {
  const int t = blockIdx.y;
  const int c = (blockIdx.x * kBlock + threadIdx.x) * 4;
  if (c >= a.H) return;
  f32x4 sum = {0.f, 0.f, 0.f, 0.f};
  for (int k = 0; k < a.K; ++k) {
    const int s = t * a.K + k;
    if (slot_expert(a.ids64, nullptr, a.first_expert, a.experts, s) < 0) continue;
    const float w = a.topk_weights[s];
    const f32x4 y = *reinterpret_cast<const f32x4*>(a.y + int64_t(s) * a.H + c);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum[i] += w * y[i];
  }
  const int64_t o = int64_t(t) * a.H + c;
  for (const void* b : {a.bias0, a.bias1}) {
    if (!b) continue;
    const u32x2 v = *reinterpret_cast<const u32x2*>(static_cast<const __bf16*>(b) + o);
    sum[0] += bf16_lo(v.x);
    sum[1] += bf16_hi(v.x);
    sum[2] += bf16_lo(v.y);
    sum[3] += bf16_hi(v.y);
  }
  *reinterpret_cast<u32x2*>(static_cast<__bf16*>(a.out) + o) =
      u32x2{pack_bf16x2(sum[0], sum[1]), pack_bf16x2(sum[2], sum[3])};
}

// ---------------------------------------------------------------------------
// bf16 rows to 4-bit codes and scales.  A lane takes 8 channels (16 bytes in,
// 4 out); the group/8 lanes of a group share its largest magnitude.  Vector
// instructions bound it, not memory: 237 a wave for int4 (nine exact divisions),
// 245 for fp4 (the choice of the code, with as many scalar ones for its
// branches), in both a 64-bit division for the group's index.  65536 x 7168 take
// 376 us as int4 in groups of 128 (3.1 TB/s), 379 us as fp4; at one instruction
// per four cycles those alone take 350 and 370.  Weights pass here once, so it
// stays simple.
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
__global__ __launch_bounds__(kBlock) void quantize_w4_kernel(QuantArgs a, int64_t block0,
                                                             int64_t pieces) {
  const int64_t p = (block0 + blockIdx.x) * kBlock + threadIdx.x;
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

FewSizes sizes_of(const FewArgs& a) {
  return FewSizes{a.slots, a.rows, a.per_token, a.experts, a.N, a.K};
}

template <int KIND, int NT, int MT, int OUT>
hipError_t launch_wide(const FewArgs& a, hipStream_t s) {
  constexpr int C = (OUT == kOutGated ? NT / 2 : NT) * 16 * kWavesPerBlock;
  constexpr int NV = kIsBf16<KIND> ? 4 : 2;           // 256 bytes of a bf16 row, 128 of a 4-bit one
  constexpr int XP = OUT == kOutF32 ? 2 : 1;
  const dim3 grid(unsigned((a.N + C - 1) / C), unsigned(most_experts(sizes_of(a))));
  few_wide_kernel<KIND, NT, NV, MT, XP, OUT, 2><<<grid, kBlock, 0, s>>>(a);
  return hipGetLastError();
}

template <int KIND, int OUT, int W>
hipError_t launch_thin(const FewArgs& a, hipStream_t s) {
  constexpr int NT = OUT == kOutGated ? 2 : 1;
  constexpr int NV = kIsBf16<KIND> ? 4 : 2;
  const dim3 grid(unsigned((a.N + 15) / 16), unsigned(most_experts(sizes_of(a))));
  few_thin_kernel<KIND, NT, NV, W, OUT, 2><<<grid, W * kWave, 0, s>>>(a);
  return hipGetLastError();
}

template <int KIND, int OUT>
hipError_t rows_variant(const FewArgs& a, hipStream_t s) {
  const FewForm f = few_form(sizes_of(a), FewOut(OUT), kIsBf16<KIND>);
  if (f.waves == 8) return launch_thin<KIND, OUT, 8>(a, s);
  if (f.waves != 0) return launch_thin<KIND, OUT, 4>(a, s);
  if constexpr (OUT != kOutGated) {
    if (f.weight_tiles == 1)
      return f.row_tiles == 1 ? launch_wide<KIND, 1, 1, OUT>(a, s)
                              : launch_wide<KIND, 1, 2, OUT>(a, s);
  }
  if (f.row_tiles == 1) return launch_wide<KIND, 2, 1, OUT>(a, s);
  if (f.row_tiles == 2) return launch_wide<KIND, 2, 2, OUT>(a, s);
  return launch_wide<KIND, 2, 3, OUT>(a, s);
}

template <int KIND, int NT>
hipError_t launch_down(const DownArgs& a, hipStream_t s) {
  constexpr int C = NT * 16;
  constexpr int NV = kIsBf16<KIND> ? 4 : 2;
  few_down_kernel<KIND, NT, NV, 2>
      <<<dim3(unsigned((a.H + C - 1) / C)), kDownBlock,
         size_t(kDownMaxSplit) * size_t(a.T * a.K) * C * 4, s>>>(a);
  return hipGetLastError();
}

template <int KIND>
hipError_t down_variant(const DownArgs& a, hipStream_t s) {
  if constexpr (!kIsBf16<KIND>)
    if (down_tiles(a.H, false) == 2) return launch_down<KIND, 2>(a, s);
  return launch_down<KIND, 1>(a, s);
}

// Calls fn with the weight kind as a compile-time constant.
template <typename Fn>
hipError_t with_kind(WeightKind kind, Fn fn) {
  switch (kind) {
    case kWBf16: return fn(std::integral_constant<int, kWBf16>());
    case kWBf16Stream: return fn(std::integral_constant<int, kWBf16Stream>());
    case kWFp4: return fn(std::integral_constant<int, kWFp4>());
    case kWInt4G32: return fn(std::integral_constant<int, kWInt4G32>());
    case kWInt4G64: return fn(std::integral_constant<int, kWInt4G64>());
    default: return fn(std::integral_constant<int, kWInt4G128>());
  }
}

WeightKind stream_kind(const Weights& w, int experts, int rows, int K) {
  return w.kind == kWBf16 && streams_bf16(w.q, experts, rows, K) ? kWBf16Stream : w.kind;
}

}  // namespace

hipError_t launch_few_rows(const FewArgs& a, bool gated, hipStream_t s) {
  return with_kind(stream_kind(a.w, a.experts, gated ? 2 * a.N : a.N, a.K), [&](auto kind) {
    constexpr int KIND = decltype(kind)::value;
    return gated ? rows_variant<KIND, kOutGated>(a, s) : rows_variant<KIND, kOutBf16>(a, s);
  });
}

hipError_t launch_few_down(const DownArgs& a, hipStream_t s) {
  const WeightKind kind_now = stream_kind(a.w, a.experts, a.H, a.I);
  if (few_down_joined(a.T * a.K, a.H, a.I))
    return with_kind(kind_now, [&](auto kind) {
      return down_variant<decltype(kind)::value>(a, s);
    });
  FewArgs f{};
  f.x = a.h;
  f.ids64 = a.ids64;
  f.first_expert = a.first_expert;
  f.slots = a.T * a.K;
  f.top = 1;
  f.rows = f.slots;
  f.per_token = a.K;
  f.experts = a.experts;
  f.N = a.H;
  f.K = a.I;
  f.w = a.w;
  f.y = a.y;
  const hipError_t e = with_kind(kind_now, [&](auto kind) {
    return rows_variant<decltype(kind)::value, kOutF32>(f, s);
  });
  if (e != hipSuccess) return e;
  const dim3 grid(unsigned((a.H / 4 + kBlock - 1) / kBlock), unsigned(a.T));
  few_sum_kernel<<<grid, kBlock, 0, s>>>(a);
  return hipGetLastError();
}

hipError_t launch_quantize_w4(const QuantArgs& a, hipStream_t s) {
  const int64_t pieces = a.rows * (a.channels / 8);
  const int64_t blocks = (pieces + kBlock - 1) / kBlock;
  constexpr int64_t kMost = int64_t(UINT32_MAX) / kBlock;      // work-items a launch, 2^32 - 1
  for (int64_t b0 = 0; b0 < blocks; b0 += kMost) {
    const dim3 grid(unsigned(blocks - b0 < kMost ? blocks - b0 : kMost));
    if (a.fp4)
      quantize_w4_kernel<true><<<grid, kBlock, 0, s>>>(a, b0, pieces);
    else
      quantize_w4_kernel<false><<<grid, kBlock, 0, s>>>(a, b0, pieces);
  }
  return hipGetLastError();
}

}  // namespace epdc
