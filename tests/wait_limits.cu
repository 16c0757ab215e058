// What a wait of a pair of CTAs leaves behind when it runs out: the flag of both.
#include "matmul_common.cuh"
#include "tc_common.cuh"

using namespace edge;

// CTA `who` of the pair (2: neither) waits for a barrier that nothing arrives on, then arrives on
// the other one's barrier; the other waits for that.  out: the flag as each thread sees it.
__global__ void __cluster_dims__(2, 1, 1) pair_kernel(int who, uint64_t limit, uint32_t* out) {
    __shared__ uint64_t never, told;
    __shared__ uint32_t flag;
    const int rank = blockIdx.x & 1;
    if (threadIdx.x == 0) {
        bar_init(smem_addr(&never), 1);
        bar_init(smem_addr(&told), 1);
        flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    cluster_sync();
    volatile uint32_t* failed = &flag;
    const int first = who == 2 ? 0 : who;
    if (rank == first) {
        if (who != 2) bar_wait<true>(smem_addr(&never), 0, failed, limit);
        if (threadIdx.x == 0) {
            asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(smem_addr(&told), rank ^ 1)) : "memory");
        }
    } else {
        bar_wait<true>(smem_addr(&told), 0, failed);
    }
    out[blockIdx.x * blockDim.x + threadIdx.x] = *failed;
    cluster_sync();
}

// A CTA by itself: its own flag, and a second wait that ends at once.
__global__ void one_kernel(uint64_t limit, uint32_t* out) {
    __shared__ uint64_t never;
    __shared__ uint32_t flag;
    if (threadIdx.x == 0) {
        bar_init(smem_addr(&never), 1);
        flag = 0;
    }
    __syncthreads();
    volatile uint32_t* failed = &flag;
    bar_wait(smem_addr(&never), 0, failed, limit);
    const uint64_t t0 = now_ns();
    bar_wait(smem_addr(&never), 0, failed);
    out[threadIdx.x] = *failed;
    out[blockDim.x + threadIdx.x] = (uint32_t)((now_ns() - t0) / 1000000);
}

extern "C" int pair(int who, uint64_t limit, uint32_t* out) {
    pair_kernel<<<2, 32>>>(who, limit, out);
    const cudaError_t e = cudaGetLastError();
    return (int)(e != cudaSuccess ? e : cudaDeviceSynchronize());
}
extern "C" int one(uint64_t limit, uint32_t* out) {
    one_kernel<<<1, 32>>>(limit, out);
    const cudaError_t e = cudaGetLastError();
    return (int)(e != cudaSuccess ? e : cudaDeviceSynchronize());
}
