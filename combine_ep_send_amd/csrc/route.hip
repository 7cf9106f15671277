// Choice of a token's experts from the router's logits, and the gradient of
// its weights (gfx950, wave64).
//
// 16 or 64 lanes choose for a token.  Everything that decides is in 64 bits:
// where scores lie so close that 32 bits would order them by their rounding,
// the choice still is the formula's, and an fp64 operation takes no longer
// here than an fp32 one.  A key's last ten bits give way to its expert's
// number, so that one comparison orders by key, then by the lower number; a
// key that is a logit has 29 spare bits and loses nothing.
//
// Each lane sorts what it holds and the lanes join their lists pairwise, the
// largest K of both: the larger of a[i] and b[N-1-i] are the largest N, in an
// order that log2(N) rounds of compare-exchange sort.
//
// The vector unit bounds it: 16384 tokens, 256 experts in 8 groups, sigmoid and bias
// take 16 us, 1640 instructions a wave of four tokens (18 MB: 3 us of memory); by
// logits alone 9 us, 64 experts 7.
#include "router_device.h"
#include "router_launch.h"

namespace epdc {

namespace {

// kNone: no key.  Every key lies above kLowest, since keys come from fp32 sums and
// infinite ones are cut to kLargest; kNone lies below it with any number in its
// last bits.
constexpr double kNone = -1.7e308;
constexpr double kLowest = -1.6e308;
constexpr double kLargest = 1.0e300;
constexpr uint32_t kIndexBits = 1023;
static_assert(kIndexBits >= 1024 - 1, "an expert's number fits");

__device__ __forceinline__ double key_of(double v, int e) {
  // +0.0 turns -0 into +0, which are equal
  const uint64_t b = __builtin_bit_cast(uint64_t, fmin(v, kLargest) + 0.0);
  const uint32_t hi = uint32_t(b >> 32);
  // the larger code for the lower number; a negative key's the other way round
  const uint32_t code = uint32_t(kIndexBits - e) ^ (uint32_t(int32_t(hi) >> 31) & kIndexBits);
  const uint32_t lo = (uint32_t(b) & ~kIndexBits) | code;
  return __builtin_bit_cast(double, (uint64_t(hi) << 32) | lo);
}
__device__ __forceinline__ int expert_of(double key) {
  const uint64_t b = __builtin_bit_cast(uint64_t, key);
  const int c = int(uint32_t(b) & kIndexBits);
  return (b >> 63) ? c : int(kIndexBits) - c;
}

__device__ __forceinline__ double from_lane(double v, int lane) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = uint32_t(__shfl(int(uint32_t(b)), lane));
  const uint32_t hi = uint32_t(__shfl(int(uint32_t(b >> 32)), lane));
  return __builtin_bit_cast(double, (uint64_t(hi) << 32) | lo);
}

// Reduction over the LANES lanes of a token, the same in all of them.
template <int LANES, int STEP = 0, typename Op>
__device__ __forceinline__ double over_lanes(double v, Op op) {
  if constexpr ((1 << STEP) < LANES)
    return over_lanes<LANES, STEP + 1>(op(v, partner<STEP>(v)), op);
  else
    return v;
}
__device__ __forceinline__ double add(double a, double b) { return a + b; }
__device__ __forceinline__ double larger(double a, double b) { return fmax(a, b); }

__device__ __forceinline__ void exchange(double& a, double& b) {
  const double hi = fmax(a, b);
  b = fmin(a, b);
  a = hi;
}
// A bitonic sequence into descending order.
template <int N>
__device__ __forceinline__ void merge(double (&v)[N]) {
#pragma unroll
  for (int j = N / 2; j > 0; j /= 2)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if ((i & j) == 0) exchange(v[i], v[i + j]);
}
template <int N>
__device__ __forceinline__ void sort(double (&v)[N]) {
#pragma unroll
  for (int k = 2; k <= N; k *= 2)
#pragma unroll
    for (int j = k / 2; j > 0; j /= 2)
#pragma unroll
      for (int i = 0; i < N; ++i)
        if ((i & j) == 0) {
          if ((i & k) == 0)
            exchange(v[i], v[i + j]);
          else
            exchange(v[i + j], v[i]);
        }
}

// The lanes' descending lists of N into one of the largest KP.
template <int LANES, int KP, int N, int STEP = 0>
__device__ __forceinline__ void join(const double (&v)[N], double (&out)[KP]) {
  if constexpr ((1 << STEP) >= LANES) {
#pragma unroll
    for (int i = 0; i < KP; ++i) out[i] = i < N ? v[i] : kNone;
  } else if constexpr (N < KP) {
    double w[2 * N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      w[i] = v[i];
      w[2 * N - 1 - i] = partner<STEP>(v[i]);
    }
    merge(w);
    join<LANES, KP, 2 * N, STEP + 1>(w, out);
  } else {
    double w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) w[i] = fmax(v[i], partner<STEP>(v[N - 1 - i]));
    merge(w);
    join<LANES, KP, N, STEP + 1>(w, out);
  }
}

// The two largest of the lists (b0, b1) of a group's `width` lanes.
template <int LANES, int STEP = 0>
__device__ __forceinline__ void best_two(double& b0, double& b1, int width) {
  if constexpr ((1 << STEP) < LANES) {
    if ((1 << STEP) >= width) return;
    const double c0 = partner<STEP>(b0), c1 = partner<STEP>(b1);
    b1 = fmax(fmin(b0, c0), fmax(b1, c1));
    b0 = fmax(b0, c0);
    best_two<LANES, STEP + 1>(b0, b1, width);
  }
}

// How many of the token's lanes hold more than v.
template <int TURN>
__device__ __forceinline__ int turned_lanes(double v) {
  if constexpr (TURN < 16) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = uint32_t(__builtin_amdgcn_update_dpp(
        int(uint32_t(b)), int(uint32_t(b)), 0x120 + TURN, 0xF, 0xF, false));
    const uint32_t hi = uint32_t(__builtin_amdgcn_update_dpp(
        int(uint32_t(b >> 32)), int(uint32_t(b >> 32)), 0x120 + TURN, 0xF, 0xF, false));
    return (__builtin_bit_cast(double, (uint64_t(hi) << 32) | lo) > v ? 1 : 0) +
           turned_lanes<TURN + 1>(v);
  }
  return 0;
}
template <int LANES>
__device__ __forceinline__ int better_lanes(double v) {
  if constexpr (LANES == 16) return turned_lanes<1>(v);
  int n = 0;
  for (int i = 1; i < LANES; ++i)
    n += from_lane(v, (lane_id() & ~(LANES - 1)) | ((lane_id() + i) & (LANES - 1))) > v ? 1 : 0;
  return n;
}

// The largest KP (or all PER) of a lane's keys, descending.
template <int KP, int PER>
struct Local {
  static constexpr int N = PER < KP ? PER : KP;
  double v[N];
  __device__ __forceinline__ explicit Local(const double (&k)[PER]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = k[i];
    sort(v);
#pragma unroll
    for (int b = N; b < PER; b += N) {
      double w[N];
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = k[b + i];
      sort(w);
#pragma unroll
      for (int i = 0; i < N; ++i) v[i] = fmax(v[i], w[N - 1 - i]);
      merge(v);
    }
  }
};

// exp(x) for -800 <= x <= 0 (64 bits hold no less than exp(-745)), NaN for NaN:
// Cody and Waite's reduction x = n ln 2 + r with |r| <= ln 2 / 2, ln 2 in two parts
// of which n times the first is exact, and the Taylor polynomial of degree 12 of
// exp(r), whose remainder is below 2^-52.
__device__ __forceinline__ double exp_within(double x) {
  const double n = __builtin_rint(x * 1.4426950408889634);
  double r = __builtin_fma(n, -0x1.62e42feep-1, x);
  r = __builtin_fma(n, -0x1.a39ef35793c76p-33, r);
  constexpr double kInverse[13] = {1.0,         1.0,          1.0 / 2,       1.0 / 6,
                                   1.0 / 24,    1.0 / 120,    1.0 / 720,     1.0 / 5040,
                                   1.0 / 40320, 1.0 / 362880, 1.0 / 3628800, 1.0 / 39916800,
                                   1.0 / 479001600};
  double p = kInverse[12];
#pragma unroll
  for (int i = 11; i >= 0; --i) p = __builtin_fma(p, r, kInverse[i]);
  return __builtin_amdgcn_ldexp(p, int(n));
}
// The same for any x <= 0.
__device__ __forceinline__ double exp_down(double x) {
  return exp_within(x < -800.0 ? -800.0 : x);
}

// From exp(-|l|), without cancellation on either side.  The first is for logits
// that are no NaN.
__device__ __forceinline__ double sigmoid_key(float l) {
  const double x = exp_within(double(fmaxf(-fabsf(l), -800.0f)));
  return (l >= 0.0f ? 1.0 : x) * inverse(1.0 + x);
}
__device__ __forceinline__ double sigmoid(double l) {
  const double x = exp_down(-fabs(l));
  return (l >= 0.0 ? 1.0 : x) * inverse(1.0 + x);
}
__device__ __forceinline__ double sigmoid_slope(double l) {
  const double x = exp_down(-fabs(l)), r = inverse(1.0 + x);
  return x * r * r;
}

// ---------------------------------------------------------------------------
// Lane r of a group's `width` lanes (one group: all lanes) holds the group's
// experts r, r + width, ..., or, where the group's size is a multiple of four and
// the logits and the bias are 16-byte aligned, r-th fours of neighbours: 16 loads
// of two neighbouring floats a group became 4 loads (16384 tokens, 256 experts in
// 8 groups: 22 -> 16 us).
// ---------------------------------------------------------------------------
template <int LANES, int PER, int KP>
__global__ __launch_bounds__(kBlock) void route_kernel(RouteArgs a, int width, bool fours,
                                                         int64_t block0) {
  constexpr int kTokens = kBlock / LANES;
  const int li = int(threadIdx.x) & (LANES - 1);
  const int64_t t0 = (block0 + blockIdx.x) * kTokens;
  const int64_t t = t0 + int(threadIdx.x) / LANES;
  const int64_t all = a.token_count ? route_live(a.T, a.token_count[0]) : a.T;
  if (t0 >= all) {                     // padding throughout, for the whole workgroup
    if (t < a.T && li < a.K) {
      a.topk_idx[t * a.K + li] = -1;
      a.topk_weights[t * a.K + li] = 0.0f;
    }
    return;
  }
  // every lane takes part in the moves; only the loads and stores are masked
  const bool live = t < all;
  const int size = a.E / a.groups;
  const int g = li / width, first = li & (width - 1);
  // every place is loaded, so that the loads go out together; what is none of
  // the token's (one past the last loads the last one's) becomes -infinity
  const float* row = a.logits + route_row(t, all) * a.E;
  // place of the lane's j-th expert in its group: fours have steps of 1 inside
  const int base = g * size + (fours ? 4 * first : first), inside = fours ? 1 : width;
  auto expert = [&](int j) { return base + (j & 3) * inside + (j >> 2) * 4 * width; };
  // experts from here on are none of the lane's
  const int limit = g < a.groups ? (g + 1) * size : 0;
  auto load = [&](const float* from, float (&v)[PER]) {
    if (fours) {
#pragma unroll
      for (int j = 0; j < PER; j += 4) {
        const int e = expert(j);
        const float4 f = *reinterpret_cast<const float4*>(from + (e < a.E ? e : 0));
        v[j] = f.x;
        if (j + 1 < PER) v[j + 1] = f.y;
        if (j + 2 < PER) v[j + 2] = f.z;
        if (j + 3 < PER) v[j + 3] = f.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < PER; ++j) v[j] = from[expert(j) < a.E ? expert(j) : 0];
    }
  };
  float l[PER];
  load(row, l);
  const int own = live ? limit : 0;
#pragma unroll
  for (int j = 0; j < PER; ++j) l[j] = expert(j) < own ? l[j] : -INFINITY;
  const bool by_score = a.bias || (a.groups > 1 && a.group_top == 2);
  const bool whole = !a.sigmoid && (by_score || !a.renorm);
  double most = 0.0, total = 1.0;
  if (whole) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) m = fmaxf(m, l[j]);
    most = over_lanes<LANES>(double(m), larger);
    total = 0.0;
  }
  double k[PER];
#pragma unroll
  for (int j = 0; j < PER; ++j) k[j] = double(l[j]);
  if (whole) {
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const double p = exp_down(k[j] - most);
      total += expert(j) < limit ? p : 0.0;
      if (by_score) k[j] = p;
    }
    total = over_lanes<LANES>(total, add);
    if (by_score) {
      const double each = 1.0 / total;
#pragma unroll
      for (int j = 0; j < PER; ++j) k[j] *= each;
    }
  } else if (by_score) {
#pragma unroll
    for (int j = 0; j < PER; ++j) k[j] = sigmoid_key(l[j]);
  }
  if (a.bias) {
    float b[PER];
    load(a.bias, b);
#pragma unroll
    for (int j = 0; j < PER; ++j) k[j] += double(b[j]);
  }
#pragma unroll
  for (int j = 0; j < PER; ++j)
    // a NaN on either side and -infinity: none
    k[j] = fmax(l[j] > -INFINITY ? k[j] : kNone, kNone);
  if (a.groups > 1) {
    double b0 = kNone, b1 = kNone;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      b1 = fmax(b1, fmin(b0, k[j]));
      b0 = fmax(b0, k[j]);
    }
    best_two<LANES>(b0, b1, width);
    double worth = b0;
    if (a.group_top == 2 && b1 > kLowest) worth = b0 + b1;
    if (b0 > kLowest) worth = key_of(worth, g);
    if (better_lanes<LANES>(worth) >= a.kept * width) {
#pragma unroll
      for (int j = 0; j < PER; ++j) k[j] = kNone;
    }
  }
#pragma unroll
  for (int j = 0; j < PER; ++j) k[j] = key_of(k[j], expert(j));
  double top[KP];
  {
    const Local<KP, PER> mine(k);
    join<LANES, KP>(mine.v, top);
  }
  // lane i writes slot i
  double mine = kNone;
#pragma unroll
  for (int i = 0; i < KP; ++i)
    if (li == i) mine = top[i];
  const bool chosen = li < a.K && mine > kLowest;
  const int e = chosen ? expert_of(mine) : -1;
  double s = 0.0;
  if (a.sigmoid) {
    if (chosen) s = sigmoid(double(row[e]));
  } else {
    const float le = chosen ? row[e] : -INFINITY;
    if (a.renorm) most = over_lanes<16>(double(le), larger);
    if (chosen) s = exp_down(double(le) - most);
  }
  if (a.renorm) total = over_lanes<16>(s, add);
  if (t >= a.T || li >= a.K) return;
  a.topk_idx[t * a.K + li] = e;
  // no sum: no weights.  The quotient first: least scores times a small scale would be 0
  a.topk_weights[t * a.K + li] =
      chosen && total != 0.0 ? float(double(a.scale) * (s / total)) : 0.0f;
}

// ---------------------------------------------------------------------------
// Gradient.  Lane k has slot k's share of the gradient, which goes to its
// expert's place in a row in LDS; the lanes then write the row out, with what
// a softmax's denominator adds for every expert.  16384 tokens of 256 experts take 13 us
// where that is so (2.7 TB/s), else 8, since the logits are then read at the chosen
// places alone.
// ---------------------------------------------------------------------------
template <int LANES, int PER>
__global__ __launch_bounds__(kBlock) void route_backward_kernel(RouteArgs a, int64_t block0) {
  constexpr int kTokens = kBlock / LANES;
  __shared__ double grad[kTokens][LANES * PER];
  const int li = int(threadIdx.x) & (LANES - 1);
  const int64_t t = (block0 + blockIdx.x) * kTokens + int(threadIdx.x) / LANES;
  const bool live = t < a.T;
  double* g = grad[int(threadIdx.x) / LANES];
#pragma unroll
  for (int j = 0; j < PER; ++j) g[j * LANES + li] = 0.0;
  const float* row = a.logits + (live ? t : a.T - 1) * a.E;
  int e = -1;
  double d = 0.0;
  if (live && li < a.K) {
    const int64_t id = a.topk_idx[t * a.K + li];
    if (id >= 0 && id < a.E) {
      e = int(id);
      d = double(a.scale) * double(a.dweights[t * a.K + li]);
    }
  }
  const float le = e >= 0 ? row[e] : -INFINITY;
  const bool any = over_lanes<LANES>(e >= 0 ? 1.0 : 0.0, add) > 0.0;
  const bool whole = !a.sigmoid && !a.renorm;
  double p[PER];                       // whole: exp(l - most) of the lane's experts
  double most = 0.0, total = 1.0, s = 0.0, mean = 0.0;
  if (whole) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      const int i = j * LANES + li;
      p[j] = double(row[i < a.E ? i : 0]);
    }
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      if (j * LANES + li >= a.E) p[j] = -INFINITY;
      m = fmaxf(m, float(p[j]));
    }
    most = over_lanes<LANES>(double(m), larger);
    total = 0.0;
#pragma unroll
    for (int j = 0; j < PER; ++j) {
      p[j] = exp_down(p[j] - most);
      if (j * LANES + li < a.E) total += p[j];
    }
    total = over_lanes<LANES>(total, add);
  } else if (!a.sigmoid) {
    most = over_lanes<16>(double(le), larger);
  }
  if (e >= 0)
    s = a.sigmoid ? sigmoid(double(le)) : le == -INFINITY ? 0.0 : exp_down(double(le) - most);
  if (a.renorm) total = over_lanes<16>(s, add);
  // no sum: no gradient, every s and slope being 0.  Quotients, since the reciprocal
  // of a sum of sigmoids below 2^-1024 (logits below -709) is infinite; a softmax's sum
  // is 1 or more
  const double below = total != 0.0 ? total : 1.0;
  if (a.renorm || whole) {
    // the weight among the chosen (renorm), or among all
    const double share = s / below;
    mean = over_lanes<LANES>(d * share, add);          // every lane needs it
    if (a.sigmoid)
      d -= mean;
    else
      d = (whole ? d : d - mean) * share;
  }
  if (a.sigmoid) d = e >= 0 ? d * (sigmoid_slope(double(le)) / below) : 0.0;
  // an expert that several slots name: its first slot adds them up
  bool first = e >= 0;
  double sum = 0.0;
  for (int k = 0; k < a.K; ++k) {
    const int lane = (lane_id() & ~(LANES - 1)) + k;
    const int ek = __shfl(e, lane);
    const double dk = from_lane(d, lane);
    if (ek == e) {
      if (k < li) first = false;
      sum += dk;
    }
  }
  __syncthreads();                     // after the zeros
  if (first) g[e] = sum;
  __syncthreads();
  if (!live) return;
  const double each = 1.0 / below;
#pragma unroll
  for (int j = 0; j < PER; ++j) {
    const int i = j * LANES + li;
    if (i >= a.E) continue;
    double v = g[i];
    if (whole && any) v -= p[j] * each * mean;
    a.dlogits[t * a.E + i] = float(v);
  }
}

template <int LANES, int PER, int KP>
void launch_route_k(const RouteArgs& a, hipStream_t s) {
  const int64_t blocks = (a.T + kBlock / LANES - 1) / (kBlock / LANES);
  const int width = LANES / ceil_pow2(a.groups);
  const bool fours = PER >= 4 && a.E / a.groups % 4 == 0 &&
                     (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0 &&
                     (reinterpret_cast<uintptr_t>(a.bias) & 15) == 0;
  for_each_launch(blocks, kBlock, [&](int64_t b0, unsigned g) {
    route_kernel<LANES, PER, KP><<<g, kBlock, 0, s>>>(a, width, fours, b0);
  });
}

template <int LANES, int PER>
void launch_route_per(const RouteArgs& a, hipStream_t s) {
  if (a.K <= 2)
    launch_route_k<LANES, PER, 2>(a, s);
  else if (a.K <= 4)
    launch_route_k<LANES, PER, 4>(a, s);
  else if (a.K <= 8)
    launch_route_k<LANES, PER, 8>(a, s);
  else
    launch_route_k<LANES, PER, 16>(a, s);
}

template <int LANES, int PER>
void launch_route_backward_per(const RouteArgs& a, hipStream_t s) {
  const int64_t blocks = (a.T + kBlock / LANES - 1) / (kBlock / LANES);
  for_each_launch(blocks, kBlock, [&](int64_t b0, unsigned g) {
    route_backward_kernel<LANES, PER><<<g, kBlock, 0, s>>>(a, b0);
  });
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t s) {
  const RouteShape r = route_shape(a.E, a.groups);
  if (r.lanes == 16) {
    if (r.per == 1)
      launch_route_per<16, 1>(a, s);
    else if (r.per == 2)
      launch_route_per<16, 2>(a, s);
    else if (r.per == 4)
      launch_route_per<16, 4>(a, s);
    else if (r.per == 8)
      launch_route_per<16, 8>(a, s);
    else
      launch_route_per<16, 16>(a, s);
  } else if (r.per <= 8) {
    launch_route_per<64, 8>(a, s);
  } else if (r.per == 16) {
    launch_route_per<64, 16>(a, s);
  } else {
    launch_route_per<64, 32>(a, s);
  }
  return hipGetLastError();
}

hipError_t launch_route_backward(const RouteArgs& a, hipStream_t s) {
  const RouteShape r = route_shape(a.E, 1);
  if (r.lanes == 16) {
    if (r.per == 1)
      launch_route_backward_per<16, 1>(a, s);
    else if (r.per == 2)
      launch_route_backward_per<16, 2>(a, s);
    else if (r.per == 4)
      launch_route_backward_per<16, 4>(a, s);
    else if (r.per == 8)
      launch_route_backward_per<16, 8>(a, s);
    else
      launch_route_backward_per<16, 16>(a, s);
  } else if (r.per <= 8) {
    launch_route_backward_per<64, 8>(a, s);
  } else {
    launch_route_backward_per<64, 16>(a, s);
  }
  return hipGetLastError();
}

}  // namespace epdc
