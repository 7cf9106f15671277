// Which kernel of expert.hip a few-row product or a layer of a few tokens takes:
// host arithmetic on sizes, types and alignment alone, without HIP, so that a
// host program can ask for the kernel of any call.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace epdc {

// What the first launch of a layer, a row call and the second launch of a layer
// (where the sum is a launch of its own) write.
enum FewOut : int { kOutGated = 0, kOutBf16 = 1, kOutF32 = 2 };

constexpr int kCus = 256;
constexpr int kFewRows = 4;        // rows of x a pass of the thin form takes
constexpr int kDownSlots = 64;     // most slots whose sum is joined to the down products

// Sizes of a launch, as in FewArgs.
struct FewSizes {
  int slots, rows, per_token, experts;
  int N, K;
};

inline int most_experts(const FewSizes& a) { return a.slots < a.experts ? a.slots : a.experts; }

// Workgroups of a launch whose workgroups cover `channels` output channels.
inline int64_t groups_of(const FewSizes& a, int channels) {
  return int64_t((a.N + channels - 1) / channels) * most_experts(a);
}

// An expert's rows are not known on the host, so the average over the experts
// stands for them.  It counts the slots of other GPUs' experts too, and is then
// too large (few_form gives the price).
inline int average_rows(const FewSizes& a) { return (a.slots + a.experts - 1) / a.experts; }

// Thin where an expert's rows come to one pass of four anyway, or where the
// wide form would leave most of the chip idle; not where the channels are too
// few for its four waves.  Thin against wide, whole calls in a graph: a layer of
// 7 tokens, 27 bf16 experts of 3928 x 1408, 92 against 118 us; of 10 tokens, 26
// of 5392 x 144, 26 against 51; 8 rows, 9 int4 matrices of 96 x 5760, 7.5
// against 22.  The other way round: 76 rows, 9 bf16 matrices of 2040 x 3368, 54
// against 42; a layer of 32 tokens, 29 int4 experts of 640 x 896, 48 against 28;
// 8 rows, 10 bf16 matrices of 5632 x 232, 9.6 against 7.5.  The price: 128 rows
// spread over 64 int4 matrices of 7168 x 2048, 147 against 98 (bf16: 268 on
// either side); all 128 rows on one of them, 91 against 80 (bf16: 159 and 136).
inline bool takes_thin(const FewSizes& a, FewOut out, bool bf16) {
  if (a.rows <= kFewRows * a.per_token) return true;
  if (a.K < (bf16 ? 512 : 1024)) return false;
  const int average = average_rows(a);
  const int64_t groups = groups_of(a, out == kOutGated ? 64 : 128);
  return average <= 2 || (groups < 192 && average <= 6) || (groups < 48 && average <= 16);
}

// waves > 0: the thin form with so many waves a workgroup.  Otherwise the wide
// form: a wave's tiles of 16 weight rows and the tiles of 16 rows of x a pass.
struct FewForm {
  int waves, weight_tiles, row_tiles;
};

// The thin form: four waves a workgroup, or eight where few workgroups have
// long rows (eight against four: one row, int4 4096 x 7168, 256 workgroups, 8.2
// against 9.5 us, in groups of 32 9.0 against 11.0, fp4 level at 7.5, bf16 12.8
// against 12.1; one row, int4 16384 x 7168, 20.4 against 17.6, 2048 x 2048, 5.6
// against 5.0; one token through 8 experts of 7168 x 2048, 1024 workgroups, the
// layer: fp4 54 against 50, int4 60 against 52).
//
// The wide form: 48 rows at a time from an average of 28 on, 16 where no more can
// come or are likely.  48 against 32, layers of 128 tokens, 32 experts of 7168 x
// 2048, which 32 rows at a time read twice for half the experts: int4 in groups
// of 128 301 against 364 us, of 64 316 against 388, fp4 273 against 362; in
// groups of 32, whose 48-row kernels spill registers, 591 against 501.  Slots of
// other GPUs' experts make the average too large: 7 of 8 of them, four rows an
// expert in truth, 48 against 16 at a time, int4 in groups of 128 251 against 196,
// of 32 506 against 210, fp4 220 against 187 (8 bf16 experts of 4096 x 1408, 48
// against 32: 78 against 71).  Weight rows: two tiles a wave, or one where two
// would leave half the units idle (one against two: 42 rows, 2 matrices of 4648 x
// 3328, int4 19 against 25, in groups of 32 19 against 34, fp4 15 against 20, bf16
// 20 against 30; 9 rows, 4 fp4 matrices of 1000 x 640, 5.6 against 6.7).  Four for
// bf16 win on some sizes (48 rows, 8 matrices of 7168 x 2048: 42 us against 47)
// and lose on more (24 rows, 4 of 14336 x 4096: 98 against 89; 100 rows, 16 of
// 4096 x 2048: 62 against 53; a layer of 97 tokens, 22 experts of 6680 x 2040: 485
// against 449), with no rule on sizes to tell them apart.
inline FewForm few_form(const FewSizes& a, FewOut out, bool bf16) {
  if (takes_thin(a, out, bf16))
    return FewForm{groups_of(a, 16) <= 2 * kCus && a.K >= 4096 ? 8 : 4, 0, 0};
  const int average = average_rows(a);
  const int row_tiles = a.rows <= 16 * a.per_token || average <= 12 ? 1 : average < 28 ? 2 : 3;
  // gate and up rows need a tile each
  const bool one = out != kOutGated && row_tiles < 3 && groups_of(a, 128) < kCus / 2;
  return FewForm{0, one ? 1 : 2, row_tiles};
}

// Whether bf16 matrices are read with the non-temporal hint: rows of whole
// 128-byte lines, and 64 MB of them or more, of which little would stay in the
// last-level cache (256 MB) beside anything else.  With both, 48 rows of 8
// matrices of 7168 x 2048 take 47 against 53 us, of 3584 x 2048 (117 MB) 27.6
// against 29.6; rows that start inside a line fetch it twice under the
// hint (8 matrices of 7160 x 7160: 183 against 159 us), and 42 MB of matrices
// read again and again stay in the cache without it (20.5 against 19.7 in a
// graph).  4-bit weights are read plainly.
inline bool streams_bf16(const void* w, int experts, int rows, int K) {
  const int64_t bytes = int64_t(experts) * rows * K * 2;
  return K % 64 == 0 && reinterpret_cast<uintptr_t>(w) % 128 == 0 && bytes >= (64 << 20);
}

// Products and sum in one launch for a few slots (it saves a launch and y),
// unless few output channels would make few workgroups, each of which reads its
// rows of every expert: 5 tokens, 30 slots of 384 x 1664 int4 experts take 39 us
// joined and 20 apart.  With more than 32 slots the wide form shares weights that
// this one reads per pass, unless the products are too small for that to show: 48
// slots of 13 fp4 experts of 3456 x 1664, 59 us joined and 52 apart; 64 of 64
// experts of 7168 x 2048, 299 and 268; but 32 slots of 32 int4 experts of 4096 x
// 1024, 52 and 74; 18 slots of 15 bf16 experts of 4888 x 136, 17 and 20.  The
// price: 64 slots of 32 int4 experts of 4096 x 1024, 77 joined and 92 apart; with
// most experts elsewhere, 42 slots of 5888 x 768, 25 joined and 27 apart.
inline bool few_down_joined(int slots, int hidden, int inner) {
  return (slots <= kDownSlots / 2 && hidden >= 2048) ||
         (slots <= kDownSlots && slots * int64_t(inner) <= 8192);
}

// The joined down products: 32 channels a workgroup for 4-bit weights if that
// leaves enough workgroups, else 16 (32 against 16, layers: one token, 8 experts
// of 7168 x 2048, fp4 51 against 53 us, int4 57 against 58, in groups of 32 62.6
// against 63.3; 4 tokens, 32 such experts, fp4 149 against 167, int4 166 against
// 171; one token, 8 experts of 4096 x 2048, fp4 37 against 33, int4 43 against
// 36; 3 tokens, 512 x 256, fp4 10.6 against 9.6.  bf16 rows of 16 channels fill a
// wave's loads as two tiles of 4-bit ones do.)
inline int down_tiles(int hidden, bool bf16) {
  return !bf16 && hidden >= 32 * kCus * 3 / 4 ? 2 : 1;
}

}  // namespace epdc
