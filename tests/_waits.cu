// Test kernels of the bounded waits (wf_device.cuh): one warp, barriers that are complete
// or that nothing completes, short limits.
#include "wf_internal.h"

using namespace wf;

// Lanes below `split` wait for a phase that is complete, the others for one that never
// will be; out[lane] is what the wait told the lane.
__global__ void part_ways_kernel(int split, int* out) {
    __shared__ uint64_t bars[2];
    const int lane = threadIdx.x;
    if (lane == 0) {
        mbar_init(&bars[0], 1);
        mbar_init(&bars[1], 1);
        fence_mbar_init();
        mbar_arrive(&bars[0]);
    }
    __syncwarp();
    out[lane] = mbar_wait_warp(&bars[lane < split ? 0 : 1], 0, 100) ? 1 : 0;
}

extern "C" int part_ways(int split, int* out) {
    part_ways_kernel<<<1, 32>>>(split, out);
    return (int)cudaGetLastError();
}
