// gq_selftest.cu -- the failure path of the kernels' bounded waits, exercised without a fault.
//
// Every wait of the kernels for a bulk copy (mbar_wait_warp), and every wait between the roles of the weight
// gradient's kernel (mbar_wait_cycles_warp, mbar_wait_cycles), gives up after a limit instead of hanging.  This
// kernel waits with those same functions on mbarriers whose phase nothing ever completes (no thread arrives, no
// copy is issued), so the waits run out; where all did, the plan's timeout flag is raised, and the kernel returns
// normally.
#include "gq_device.cuh"

namespace gq {
namespace {

__global__ void __launch_bounds__(96) k_wait_selftest(unsigned int *status, unsigned long long limit_ns)
{
    __shared__ unsigned long long bar[3];
    __shared__ int gave_up[3];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) {
        mbar_init(&bar[warp], 1);  // one arrival expected, none will come
        fence_barrier_init();
    }
    __syncwarp();
    const long long cycles = 2 * (long long)limit_ns;  // no clock here passes 2 GHz
    bool done;
    if (warp == 0) done = mbar_wait_warp(&bar[0], 0u, limit_ns);
    else if (warp == 1) done = mbar_wait_cycles_warp(smem_u32(&bar[1]), 0u, cycles);
    else done = lane != 0 || mbar_wait_cycles(smem_u32(&bar[2]), 0u, cycles);
    if (lane == 0) gave_up[warp] = !done;
    __syncthreads();
    if (threadIdx.x == 0 && gave_up[0] && gave_up[1] && gave_up[2]) atomicOr(status, kStatusTimeout);
}

}  // namespace

cudaError_t launch_wait_selftest(unsigned int *status, unsigned long long limit_ns, cudaStream_t stream)
{
    k_wait_selftest<<<1, 96, 0, stream>>>(status, limit_ns);
    return cudaGetLastError();
}

}  // namespace gq
