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

// A ring of `slots` barriers given `uses` phases in turn, of which the last `missing` are never
// completed: what the drain says.
__global__ void drain_kernel(int slots, int uses, int missing, int* out) {
    __shared__ uint64_t bars[8];
    const int lane = threadIdx.x;
    if (lane == 0) {
        for (int s = 0; s < slots; ++s) mbar_init(&bars[s], 1);
        fence_mbar_init();
        for (int u = 0; u < uses - missing; ++u) mbar_arrive(&bars[u % slots]);
    }
    __syncwarp();
    out[lane] = mbar_drain_ring(bars, slots, uses, 100) ? 1 : 0;
}

extern "C" int drain(int slots, int uses, int missing, int* out) {
    if (slots < 1 || slots > 8 || uses < 0 || missing < 0 || missing > uses) return -1;
    drain_kernel<<<1, 32>>>(slots, uses, missing, out);
    return (int)cudaGetLastError();
}
