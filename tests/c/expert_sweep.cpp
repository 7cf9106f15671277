// Host-side validation sweep of the expert-side calls (epdc_expert.h): a
// seeded random mix of extreme sizes, formats and pointers against a library
// whose host code is built with the address and undefined-behaviour
// sanitizers.  As abi_sweep.cpp, only for a machine without a GPU.
//
//   expert_sweep SEED ITERS
#include <climits>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "epdc_expert.h"

namespace {

std::mt19937_64 rng;

template <typename T, size_t N>
T pick(const T (&v)[N]) {
  return v[rng() % N];
}

const int64_t kI64[] = {-1, 0, 1, 4, 128, 129, 1024, 1025, (1LL << 30) - 1, 1LL << 30,
                        1LL << 31, INT64_MAX, INT64_MIN};
const int kI32[] = {-1, 0, 1, 2, 8, 12, 16, 17, 32, 64, 128, 1024, 1025, 7168, 65536, 131072,
                    INT_MAX, INT_MIN};
const size_t kSizes[] = {0, 1, 255, size_t(1) << 20, SIZE_MAX};
const int kFmt[] = {0, 1, 2, 3, -1};

void* ptr() {
  static void* const p[] = {nullptr, (void*)0x10000, (void*)0x10002, (void*)0x10008,
                            (void*)0x10100, (void*)0x10200};
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
    std::fprintf(stderr, "expert_sweep: %d GPU(s) visible; this sweep runs only without a GPU\n",
                 devices);
    return 2;
  }
  rng.seed(std::strtoull(argv[1], nullptr, 10));
  const long iters = std::strtol(argv[2], nullptr, 10);
  long rejected = 0, passed = 0;
  for (long it = 0; it < iters; ++it) {
    int st = EP_OK;
    switch (it % 7) {
      case 0:
        st = ep_quantize_w4(ptr(), pick(kI64), pick(kI32), pick(kFmt), pick(kI32), ptr(), ptr(),
                            nullptr);
        break;
      case 1:
        st = ep_expert_matvec(ptr(), p<const int32_t>(), pick(kI64), pick(kI32), pick(kI32),
                              pick(kI32), pick(kFmt), pick(kI32), ptr(), ptr(), ptr(), nullptr);
        break;
      case 2:
        st = ep_moe_tokens(ptr(), p<const int64_t>(), p<const float>(), pick(kI64), pick(kI32),
                           pick(kI32), pick(kI32), pick(kI32), pick(kI32), pick(kFmt), pick(kI32),
                           ptr(), ptr(), pick(kFmt), pick(kI32), ptr(), ptr(), ptr(), ptr(), ptr(),
                           ptr(), pick(kSizes), nullptr);
        break;
      case 3:
        st = ep_swiglu_fp8(ptr(), pick(kI64), pick(kI32), p<const int32_t>(), ptr(), ptr(),
                           p<float>(), nullptr);
        break;
      case 4:
        st = ep_swiglu_fp8_backward(ptr(), ptr(), p<const float>(), pick(kI64), pick(kI32),
                                    p<const int32_t>(), ptr(), ptr(), nullptr);
        break;
      case 5:
        st = ep_combine_backward(ptr(), ptr(), pick(kI64), p<const int32_t>(), p<const float>(),
                                 pick(kI64), pick(kI32), pick(kI32), ptr(), p<float>(), nullptr);
        break;
      default: {
        volatile size_t s = ep_moe_tokens_workspace_bytes(pick(kI64), pick(kI32), pick(kI32),
                                                          pick(kI32));
        (void)s;
        continue;
      }
    }
    if (st == EP_OK || st == EP_ERR_LAUNCH)
      ++passed;
    else if (st == EP_ERR_INVALID_ARG || st == EP_ERR_UNSUPPORTED || st == EP_ERR_WORKSPACE)
      ++rejected;
    else
      return 2;  // not a status the ABI defines
  }
  std::printf("done: %ld rejected, %ld passed validation\n", rejected, passed);
  return 0;
}
