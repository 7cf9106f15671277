// Sizes and variants of the launches before the dispatch: host arithmetic on
// sizes and types alone, without HIP.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace epdc {

constexpr int kRouterChannels = 65536;

// ---- norm -------------------------------------------------------------------
// A workgroup takes a row at a time; a thread holds PT 16-byte pieces of it.
constexpr int kNormChannels = 32768;
constexpr int kNormMaxThreads = 512;

struct NormShape {
  int pieces;      // PT: 1, 2, 4 or 8
  int threads;
};

inline NormShape norm_shape(int H) {
  const int n = H / 8;
  int pt = 1;
  while (pt < 8 && n > pt * kNormMaxThreads) pt *= 2;
  const int t = (n + pt - 1) / pt;
  return NormShape{pt, (t + 63) / 64 * 64};
}

// Workgroups of the backward pass, each with one row of partial sums of the
// weight's gradient: as many as the chip holds at once, by the waves that the
// kernel's registers allow a compute unit, and four a compute unit at most.  In us,
// the sums' launch included, with two, four and eight: 16384 rows of 512 channels 33,
// 25 and 27, of 2048 62, 60 and 66; of 4096, where three fit, 94 with two and 104; 2500
// of 5120 26 and 29.
inline int norm_groups(int64_t T, int H) {
  const NormShape n = norm_shape(H);
  const int waves = n.pieces == 1 ? 24 : n.pieces == 2 ? 16 : 8;
  int per_cu = waves / (n.threads / 64);
  if (per_cu < 1) per_cu = 1;
  if (per_cu > 4) per_cu = 4;
  const int most = 256 * per_cu;
  // two rows or more each: a row of sums costs as much to move as a row.  With one,
  // two and eight rows: 64 rows of 4096 channels 7.0, 7.5 and 14 us, 300 11.2, 9.6 and
  // 15.8, 1237 of 2056 18, 16 and 17
  const int64_t want = (T + 1) / 2;
  return int(want < most ? want : most);
}

// Whether rows are read with non-temporal loads: `inputs` arrays of rows that come
// to one and a half times the Infinity Cache.
inline bool norm_streams(int64_t T, int H, int inputs) {
  return T * H * 2 * inputs >= int64_t(384) << 20;
}

// ---- choice of the experts ----------------------------------------------------
// A token is chosen for by `lanes` lanes (16 or 64), each holding up to `per`
// experts of one group.
struct RouteShape {
  int lanes;
  int per;
};

inline int ceil_pow2(int v) {
  int p = 1;
  while (p < v) p *= 2;
  return p;
}

inline RouteShape route_shape(int E, int groups) {
  const int size = E / groups, slots = ceil_pow2(groups);      // groups <= 16
  for (int lanes = 16;; lanes = 64) {
    const int width = lanes / slots;                           // lanes of a group
    const int per = ceil_pow2((size + width - 1) / width);
    if (per <= 16 || lanes == 64) return RouteShape{lanes, per};
  }
}

// Tokens that take part, by the padding's `count`; and the token whose logits are read
// in t's place: no logits of a padding token are, nor any where there are none else.
constexpr int64_t route_live(int64_t T, int64_t count) {
  return count < 0 ? 0 : count < T ? count : T;
}
constexpr int64_t route_row(int64_t t, int64_t live) { return t < live ? t : live - 1; }

// ---- the router's products -----------------------------------------------------
constexpr int kGemmGroups = 256;      // workgroups that fill the chip

// Logits: a workgroup takes bm tokens and 64 * wn experts over `each` stages of
// 64 channels; the channels are split over workgroups, whose sums a second launch adds
// up, as long as these do not outnumber the compute units (where they may, by less
// than one split: 8195 tokens, 64 experts, 4096 channels 23 us instead of 21, 12000 33
// instead of 27).
//
// The wide form from 129 experts and 2048 tokens on.  Wide and not, in us: 256 experts
// of 7168 channels 1024 tokens 24 and 22, 2048 26 and 26, 4096 33 and 37, 16384 87 and
// 105; 1024 experts of 4096 channels 1024 tokens 33 and 29, 2048 40 and 42, 8192 73 and
// 115.  160 experts of 4096 channels take 22 and 19 at 2048 tokens, 32 and 37 at 8192,
// 256 of 1024 channels 25 and 24 at 8192; 128 experts 66 and 64 (16384 tokens of 7168
// channels), 27 and 31 (8195 of 4096), 23 and 18 (2048 of 7168).
struct LogitsShape {
  int bm, wn;
  int64_t mb;
  int nb, splits, each;
  bool wide;                     // the form with the weights in the matrix cores' order
};

constexpr int kWideTokens = 128, kWideExperts = 128;

inline LogitsShape logits_shape(int64_t T, int E, int H) {
  LogitsShape g{};
  g.wn = E <= 64 ? 1 : E <= 128 ? 2 : 4;
  g.wide = E > 128 && T >= 2048;
  g.bm = g.wide ? kWideTokens : T <= 16 ? 16 : T <= 32 ? 32 : 64;
  if (g.bm < 64) g.wn = 4;
  const int experts = g.wide ? kWideExperts : 64 * g.wn;
  g.mb = T > 0 ? (T + g.bm - 1) / g.bm : 1;
  g.nb = (E + experts - 1) / experts;
  const int stages = (H + 63) / 64;
  const int64_t tiles = g.mb * g.nb;
  int64_t want = kGemmGroups / tiles;
  if (want < 1) want = 1;
  if (want > stages) want = stages;
  g.each = int((stages + want - 1) / want);
  g.splits = (stages + g.each - 1) / g.each;
  return g;
}

// The rows' gradient: a workgroup keeps 16 * mt tokens' rows of dlogits in LDS,
// 64 KB of them, and takes `each` blocks of 64 channels: four, one a wave, or more, and
// so many that two workgroups a compute unit are not passed.  Both gradients in us, with
// one, four and eight blocks at least: 64 tokens, 64 experts, 4096 channels 13.0, 13.4
// and 14.8, 300 x 160 x 5120 30, 30 and 33, many tokens alike; with one, two and four
// workgroups a compute unit: 8195 x 64 x 4096 57, 51 and 51, 4096 x 256 x 7168 97, 94 and
// 102.
struct DxShape {
  int mt;
  int64_t mb;
  int splits, each;
};

inline DxShape dx_shape(int64_t T, int H, int Ep) {
  DxShape d{};
  const int most = Ep <= 256 ? 4 : Ep <= 512 ? 2 : 1;
  const int fit = T <= 16 ? 1 : T <= 32 ? 2 : 4;
  d.mt = most < fit ? most : fit;
  d.mb = (T + 16 * d.mt - 1) / (16 * d.mt);
  const int blocks = (H + 63) / 64;
  int64_t want = 2 * kGemmGroups / (d.mb > 0 ? d.mb : 1);
  if (want > (blocks + 3) / 4) want = (blocks + 3) / 4;
  if (want < 1) want = 1;
  d.each = int((blocks + want - 1) / want);
  d.splits = (blocks + d.each - 1) / d.each;
  return d;
}

// The weights' gradient: a workgroup takes 64 experts and 128 channels over
// `each` steps of 32 tokens: four, one a wave, or more.  Both gradients in us, with two,
// four and eight at least: 512 tokens, 64 experts, 4096 channels 22, 20 and 20, 300 x 160 x
// 5120 30, 30 and 25, from 1024 tokens on alike.
struct DwShape {
  int eb, hb, splits;
  int64_t each;
};

inline DwShape dw_shape(int64_t T, int E, int H) {
  DwShape d{};
  d.eb = (E + 63) / 64;
  d.hb = (H + 127) / 128;
  const int64_t steps = (T + 31) / 32;
  int64_t want = kGemmGroups / (int64_t(d.eb) * d.hb);
  if (want > steps / 4) want = steps / 4;
  if (want < 1) want = 1;
  d.each = steps ? (steps + want - 1) / want : 1;
  d.splits = steps ? int((steps + d.each - 1) / d.each) : 1;
  return d;
}

// Workspaces.
constexpr int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }

struct WideSpace {
  int64_t experts;   // of the copy of the weights: whole waves
  int64_t channels;  // whole stages
  size_t wf;         // the weights in the matrix cores' order
  size_t part;       // [splits][T][E] fp32
  size_t total;
};
inline WideSpace wide_space(const LogitsShape& g, int64_t T, int E, int H) {
  WideSpace s{};
  s.experts = (E + 31) / 32 * 32;
  s.channels = pad64(H);
  s.wf = 0;
  s.part = (size_t(s.experts) * size_t(s.channels) * 2 + 255) / 256 * 256;
  s.total = s.part + (g.splits > 1 ? size_t(g.splits) * size_t(T) * size_t(E) * 4 : 0);
  return s;
}
inline size_t logits_ws_bytes(int64_t T, int E, int H) {
  const LogitsShape g = logits_shape(T, E, H);
  if (g.wide) return wide_space(g, T, E, H).total;
  return 256 + (g.splits > 1 ? size_t(g.splits) * size_t(T) * size_t(E) * 4 : 0);
}

struct LogitsBackwardSpace {
  size_t columns;    // dlogits transposed, in three bf16 parts
  size_t wt;         // the weights transposed
  size_t part;       // partial sums of dw [splits][E][H] fp32
  size_t total;
};

inline LogitsBackwardSpace logits_backward_space(int64_t T, int E, int H) {
  const size_t Ep = size_t(pad64(E));
  const DwShape d = dw_shape(T, E, H);
  LogitsBackwardSpace s{};
  s.columns = 0;
  s.wt = s.columns + 6 * Ep * ((size_t(T) + 31) / 32 * 32);
  s.part = s.wt + 2 * Ep * size_t(pad64(H));
  s.total = s.part + (d.splits > 1 ? size_t(d.splits) * size_t(E) * size_t(H) * 4 : 0) + 256;
  return s;
}

}  // namespace epdc
