// Host-side validation sweep of the calls before the dispatch (epdc_router.h): a
// seeded random mix of extreme sizes, types and pointers against a library
// whose host code is built with the address and undefined-behaviour
// sanitizers.  As expert_sweep, only for a machine without a GPU.
//
//   router_sweep SEED ITERS
#include <climits>
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "epdc_router.h"

namespace {

std::mt19937_64 rng;

template <typename T, size_t N>
T pick(const T (&v)[N]) {
  return v[rng() % N];
}

const int64_t kI64[] = {-1, 0, 1, 16, 17, 33, 2047, 2048, 16384, (1LL << 30) - 1, 1LL << 30,
                        1LL << 31, INT64_MAX, INT64_MIN};
const int kI32[] = {-1, 0, 1, 2, 3, 4, 8, 12, 16, 17, 64, 128, 129, 256, 1000, 1024, 1025, 7168,
                    32768, 32776, 65536, 65544, INT_MAX, INT_MIN};
const size_t kSizes[] = {0, 1, 255, size_t(1) << 20, SIZE_MAX};
const int kFlag[] = {0, 1, 2, -1};
const float kFloat[] = {0.0f, 1.0f, -1.0f, 1e-6f, INFINITY, -INFINITY, NAN, 3e38f};

void* ptr() {
  static void* const p[] = {nullptr, (void*)0x10000, (void*)0x10002, (void*)0x10004,
                            (void*)0x10008, (void*)0x10100, (void*)0x10200};
  return pick(p);
}
template <typename T>
T* p() {
  return static_cast<T*>(ptr());
}

}  // namespace

int main(int argc, char** argv) {
  if (argc != 3) {
    std::fprintf(stderr, "usage: %s SEED ITERS\n", argv[0]);
    return 1;
  }
  int devices = 0;
  if (hipGetDeviceCount(&devices) == hipSuccess && devices > 0) {
    std::fprintf(stderr, "router_sweep: %d GPU(s) visible; this sweep runs only without a GPU\n",
                 devices);
    return 2;
  }
  rng.seed(std::strtoull(argv[1], nullptr, 10));
  const long iters = std::strtol(argv[2], nullptr, 10);
  long rejected = 0, passed = 0;
  for (long it = 0; it < iters; ++it) {
    int st = EP_OK;
    const int64_t T = pick(kI64);
    const int a = pick(kI32), b = pick(kI32), c = pick(kI32);
    switch (it % 8) {
      case 0:
        st = ep_rms_norm(ptr(), ptr(), ptr(), pick(kFlag), T, a, pick(kFloat), ptr(), ptr(), ptr(),
                         p<float>(), pick(kFlag), p<float>(), nullptr);
        break;
      case 1:
        st = ep_rms_norm_backward(ptr(), ptr(), ptr(), pick(kFlag), p<float>(), ptr(), T, a, ptr(),
                                  p<float>(), ptr(), pick(kSizes), nullptr);
        break;
      case 2:
        st = ep_router_logits(ptr(), ptr(), T, a, b, p<float>(), ptr(), pick(kSizes), nullptr);
        break;
      case 3:
        st = ep_router_logits_backward(p<float>(), ptr(), ptr(), T, a, b, ptr(), p<float>(), ptr(),
                                       pick(kSizes), nullptr);
        break;
      case 4:
        st = ep_route(p<float>(), T, a, b, pick(kFlag), p<float>(), c, pick(kI32), pick(kFlag),
                      pick(kFlag), pick(kFloat), p<int32_t>(), p<int64_t>(), p<float>(), nullptr);
        break;
      case 5:
        st = ep_route_backward(p<float>(), p<float>(), p<int64_t>(), T, a, b, pick(kFlag),
                               pick(kFlag), pick(kFloat), p<float>(), nullptr);
        break;
      case 6:
        st = ep_dispatch_permute_quantized(ptr(), ptr(), a, T, b, p<int32_t>(), c, pick(kI64),
                                           ptr(), ptr(), nullptr);
        break;
      default:
        // a size for what the call would take, 0 for what it refuses
        if ((ep_rms_norm_backward_workspace_bytes(T, a) == 0) !=
            (T < 0 || T >= (1LL << 30) || a <= 0 || a % 8 != 0 || a > EPDC_NORM_CHANNELS))
          return 3;
        const bool bad = T < 0 || T >= (1LL << 30) || a < 1 || a > EPDC_MAX_BINS || b <= 0 ||
                         b % 8 != 0 || b > EPDC_ROUTER_CHANNELS;
        if ((ep_router_logits_workspace_bytes(T, a, b) == 0) != bad ||
            (ep_router_logits_backward_workspace_bytes(T, a, b) == 0) != bad)
          return 4;
    }
    if (st == EP_ERR_INVALID_ARG || st == EP_ERR_UNSUPPORTED || st == EP_ERR_WORKSPACE)
      ++rejected;
    else
      ++passed;
  }
  std::printf("done: %ld rejected, %ld passed validation\n", rejected, passed);
  return rejected > 0 && passed > 0 ? 0 : 5;
}
