// sandwich.cu with waits that run out, for test_gpu_sandwich_waits: a row's copies
// are waited for as they are (2 s at most, so every copy has landed), and then
// reported as not there from the second use of a stage on.  The limit after which
// a kernel gives a row up is 0.2 ms here.
#include "tc_ops.h"

namespace dwdp {
__device__ __forceinline__ bool late_try_wait(uint32_t bar, uint32_t parity) {
    const uint64_t since = global_timer();
    bool there = mbar_try_wait(bar, parity);
    while (!there && global_timer() - since <= kWaitLimitNs) there = mbar_try_wait(bar, parity);
    return there && parity == 0;
}
constexpr uint64_t kShortLimitNs = 200000;
}  // namespace dwdp

#define mbar_try_wait late_try_wait
#define kWaitLimitNs kShortLimitNs
#include "sandwich.cu"
