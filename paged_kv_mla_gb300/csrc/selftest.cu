// selftest.cu -- exercises the bounded mbarrier waits every pipeline kernel relies on: warps
// wait, each in one of the forms, on an mbarrier phase that nothing will complete.  The one that
// keeps time must give up after its limit, record PKM_ERR_TIMEOUT and end the others' waits; the
// caller's status word says so only if all did, none early and none much later.  The context
// stays usable: failure detection is tested this way, without any fault, trap or hang.
#include "pkm_device.cuh"
#include "pkm_internal.h"

namespace pkm {
namespace {

constexpr int kForms = 3;  // mbar_wait, which keeps time; mbar_wait_flag; that at cluster scope

__global__ void wait_timeout_kernel(int32_t* status, uint64_t timeout_ns) {
    __shared__ uint64_t bar;
    __shared__ int abort_flag, found, good;
    __shared__ uint64_t t0;  // before every warp's wait
    const int form = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort_flag = found = good = 0;
        fence_mbar_init();
        t0 = globaltimer_ns();
    }
    __syncthreads();
    // no thread ever arrives on `bar`: phase 0 never completes
    const WaitCtl wc{&abort_flag, &found, timeout_ns};
    const uint32_t tries = static_cast<uint32_t>(min(timeout_ns / 8, uint64_t{UINT32_MAX}));
    bool ok = false;
    if (form == 0) {
        if (lane == 0) ok = mbar_wait(&bar, 0, wc);
    } else {
        ok = form == 1 ? mbar_wait_flag(&bar, 0, wc.abort_flag, tries)
                       : mbar_wait_flag<true>(&bar, 0, wc.abort_flag, tries);
    }
    const uint64_t took = globaltimer_ns() - t0;
    const bool in_time = took >= timeout_ns && took <= timeout_ns + timeout_ns / 2 + 5000000;
    const bool all = __all_sync(0xffffffffu, !ok && (in_time || (form == 0 && lane > 0)));
    if (lane == 0 && all) atomicAdd(&good, 1);
    __syncthreads();
    if (threadIdx.x == 0 && good == kForms && found == PKM_ERR_TIMEOUT && abort_flag != 0)
        report(status, PKM_ERR_TIMEOUT);
}

}  // namespace

cudaError_t launch_wait_timeout_check(int32_t* status, uint64_t timeout_ns, cudaStream_t stream) {
    wait_timeout_kernel<<<1, 32 * kForms, 0, stream>>>(status, timeout_ns);
    return cudaGetLastError();
}

}  // namespace pkm
