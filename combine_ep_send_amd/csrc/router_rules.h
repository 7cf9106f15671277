// Sizes and variants of the launches before the dispatch: host arithmetic on
// sizes and types alone, without HIP.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace epdc {

constexpr int kRouterChannels = 65536;

// ---- norm -------------------------------------------------------------------
// A workgroup takes a row at a time; a thread holds PT 16-byte pieces of it.
struct NormShape {
  int pieces;      // PT: 1, 2, 4 or 8
  int threads;
};

inline NormShape norm_shape(int H) {
  const int n = H / 8;
  int pt = 1;
  while (pt < 8 && n > pt * 512) pt *= 2;
  const int t = (n + pt - 1) / pt;
  return NormShape{pt, (t + 63) / 64 * 64};
}

// Workgroups of the backward pass, each with one row of partial sums of the
// weight's gradient.
inline int norm_groups(int64_t T) { return int(T < 1024 ? T : 1024); }

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

// ---- the router's products -----------------------------------------------------
// out[m, n] = sum over k of A[m, k] B[n, k]: a workgroup takes 16 * mt rows of A
// and 64 * wn rows of B; its four waves are wn side by side along n times
// 4 / wn along k, and a stage is 64 channels k for each of the latter.  The
// stages are split over `splits` workgroups, `each` a workgroup.
struct GemmShape {
  int mt, wn;
  int64_t mb;
  int nb, splits, each;
};

constexpr int kGemmGroups = 256;      // workgroups that fill the chip

inline GemmShape gemm_shape(int64_t M, int N, int K, bool splittable) {
  GemmShape g{};
  g.mt = M <= 16 ? 1 : M <= 32 ? 2 : 4;
  g.mb = M > 0 ? (M + 16 * g.mt - 1) / (16 * g.mt) : 1;
  g.wn = N <= 64 || g.mb * ((N + 63) / 64) < kGemmGroups ? 1 : N <= 128 ? 2 : 4;
  g.nb = (N + 64 * g.wn - 1) / (64 * g.wn);
  const int depth = 64 * (4 / g.wn);
  const int stages = (K + depth - 1) / depth;
  int64_t want = splittable ? kGemmGroups / (g.mb * g.nb) : 1;
  if (want < 1) want = 1;
  if (want > stages) want = stages;
  g.each = int((stages + want - 1) / want);
  g.splits = (stages + g.each - 1) / g.each;
  return g;
}

// The weights' gradient: a workgroup takes 64 experts and 256 channels (64 a
// wave) over `each` steps of 32 tokens.
struct OuterShape {
  int eb, hb, splits;
  int64_t each;
};

inline OuterShape outer_shape(int64_t T, int E, int H) {
  OuterShape o{};
  o.eb = (E + 63) / 64;
  o.hb = (H + 255) / 256;
  const int64_t steps = (T + 31) / 32;
  int64_t want = 512 / (int64_t(o.eb) * o.hb);
  if (want > 64) want = 64;
  if (want > steps / 4) want = steps / 4;
  if (want < 1) want = 1;
  o.each = (steps + want - 1) / want;
  if (o.each < 1) o.each = 1;
  o.splits = steps ? int((steps + o.each - 1) / o.each) : 1;
  return o;
}

// Workspaces.  Padded sizes: experts and tokens to 64.
inline int64_t pad64(int64_t v) { return (v + 63) / 64 * 64; }

inline size_t logits_ws_bytes(int64_t T, int E, int H) {
  const GemmShape g = gemm_shape(T, E, H, true);
  return 256 + (g.splits > 1 ? size_t(g.splits) * size_t(T) * size_t(E) * 4 : 0);
}

struct LogitsBackwardSpace {
  size_t rows;       // dlogits in two bf16 parts [2][T][Ep]
  size_t columns;    // in three, transposed [3][Ep][Tp]
  size_t wt;         // the weights transposed [H][Ep]
  size_t part;       // partial sums of dw [splits][E][H] fp32
  size_t total;
};

inline LogitsBackwardSpace logits_backward_space(int64_t T, int E, int H) {
  const size_t Ep = size_t(pad64(E)), Tp = size_t(pad64(T));
  const OuterShape o = outer_shape(T, E, H);
  auto up = [](size_t b) { return (b + 255) / 256 * 256; };
  LogitsBackwardSpace s{};
  s.rows = 0;
  s.columns = s.rows + up(4 * size_t(T) * Ep);
  s.wt = s.columns + up(6 * Tp * Ep);
  s.part = s.wt + up(2 * size_t(H) * Ep);
  s.total = s.part + (o.splits > 1 ? size_t(o.splits) * size_t(E) * size_t(H) * 4 : 0) + 256;
  return s;
}

}  // namespace epdc
