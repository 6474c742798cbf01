// selftest.cu -- kda_selftest_device_timeout: exercises the bounded-wait failure path.
//
// Every mbarrier wait in the library's kernels gives up after a time limit, records
// KDA_ERR_DEVICE_TIMEOUT in the per-device status word and lets the kernel return, so a
// broken pipeline ends with an error the host can read instead of a hung GPU.  This entry
// point makes that path observable without breaking anything: one thread initialises an
// mbarrier that expects one arrival which never comes, and waits on it with a short limit.
// kda_selftest_role_timeout does the same for the waits of the latent-attention kernels' roles,
// which count tries.
#include "kda_common.cuh"
#include "kda_internal.h"
#include "mla_tc.cuh"

namespace kda {
namespace {

__global__ void timeout_kernel(unsigned long long limit_ns, unsigned int *status)
{
    __shared__ __align__(8) uint64_t bar;
    if (threadIdx.x != 0)
        return;
    mbar_init(&bar, 1);
    fence_mbar_init_cluster();
    mbar_wait_bounded(&bar, 0, status, limit_ns);  // nothing arrives: runs out after limit_ns
}

// A role as the latent-attention kernels have them: a loop that waits and lets one lane act.  The
// barriers never complete.  `acted` counts what must not happen once a wait has run out.
__global__ void role_timeout_kernel(uint32_t tries, unsigned int *status)
{
    __shared__ __align__(8) uint64_t bar[3];
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int i = 0; i < 3; ++i)
            mbar_init(&bar[i], 1);
        fence_mbar_init_cluster();
    }
    __syncwarp();
    int acted = 0;
    mla::Waits wait{false, tries};
    for (int i = 0; i < 3; ++i) {
        wait(&bar[0], 0);
        if (mla::elect() && !wait.dead)
            ++acted;
    }
    mla::Waits three{false, tries};
    three(&bar[0], 0, &bar[1], 0, &bar[2], 0);  // the first runs out, the others are not waited for
    mla::Waits mixed{lane == 3, tries};         // one lane's wait ran out
    for (int i = 0; i < 3; ++i) {
        mixed(&bar[0], 0);
        if (mla::elect() && !mixed.dead)
            ++acted;
    }
    if (acted > 0 || !wait.dead || !three.dead)
        report_device_error(status, KDA_ERR_DEVICE_BOUNDS);
    __syncwarp();
    wait.finish(status);
}

}  // namespace
}  // namespace kda

using namespace kda;

extern "C" kda_status kda_selftest_device_timeout(uint32_t limit_us, kda_stream_t stream)
{
    if (limit_us < 1 || limit_us > 2000000u)
        return KDA_ERR_INVALID_ARG;
    unsigned int *status = device_status_ptr();
    if (!status)
        return KDA_ERR_CUDA;
    timeout_kernel<<<1, 32, 0, (cudaStream_t)stream>>>((unsigned long long)limit_us * 1000ull, status);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}

extern "C" kda_status kda_selftest_role_timeout(uint32_t tries, kda_stream_t stream)
{
    if (tries < 1 || tries > mla::kWaitTries)
        return KDA_ERR_INVALID_ARG;
    unsigned int *status = device_status_ptr();
    if (!status)
        return KDA_ERR_CUDA;
    role_timeout_kernel<<<1, 32, 0, (cudaStream_t)stream>>>(tries, status);
    return cudaGetLastError() == cudaSuccess ? KDA_OK : KDA_ERR_CUDA;
}
