// wait_limit.cu -- the waits of the tensor-core kernels (leyline_tcgen05.cuh) when nobody arrives, in a kernel of one CTA
// without loads or products, with a limit of 0.2 ms; built by tests/test_gpu_wait_limit.py.
#include "leyline_pool_state.h"
#include "leyline_tcgen05.cuh"

namespace leyline {

constexpr int kWaitThreads = 64;
constexpr unsigned long long kLimit = 200000;

struct WaitResult {
    int complete[kWaitThreads];  // a wait that ends
    int local[kWaitThreads];     // waits that nobody ends: 1 if they claim that somebody did
    int cluster[kWaitThreads];
    int quit;
    int milliseconds;
};

__global__ void __launch_bounds__(kWaitThreads) wait_kernel(WaitResult* out, int32_t* status)
{
    __shared__ unsigned long long bars[2];
    __shared__ int quit;
    if (threadIdx.x == 0) {
        mbar_init(smem_addr(&bars[0]), 1);
        mbar_init(smem_addr(&bars[1]), 1);
        quit = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    if (threadIdx.x == 0) mbar_arrive(smem_addr(&bars[0]));
    const unsigned long long t0 = global_ns();
    out->complete[threadIdx.x] = mbar_wait(smem_addr(&bars[0]), 0, &quit, status, kLimit);
    __syncthreads();
    out->local[threadIdx.x] = mbar_wait(smem_addr(&bars[1]), 0, &quit, status, kLimit);
    __syncthreads();
    if (threadIdx.x == 0) {
        out->quit = quit;
        quit = 0;
    }
    __syncthreads();
    out->cluster[threadIdx.x] = mbar_wait_cluster(smem_addr(&bars[1]), 0, &quit, status, kLimit);
    __syncthreads();
    if (threadIdx.x == 0) {
        out->quit += quit;
        out->milliseconds = (int)((global_ns() - t0) / 1000000);
    }
}

}  // namespace leyline

using namespace leyline;

// Runs the kernel on the pool's device with its status word.  0, or a CUDA error code.
extern "C" int wait_limit(leyline_pool_t* pool, WaitResult* out)
{
    DeviceGuard guard(pool->device);
    WaitResult* dev = nullptr;
    cudaError_t e = cudaMalloc(&dev, sizeof(WaitResult));
    if (e != cudaSuccess) return (int)e;
    e = cudaMemset(dev, 0xff, sizeof(WaitResult));
    if (e == cudaSuccess) {
        wait_kernel<<<1, kWaitThreads>>>(dev, pool->d_status);
        e = cudaGetLastError();
    }
    if (e == cudaSuccess) e = cudaMemcpy(out, dev, sizeof(WaitResult), cudaMemcpyDeviceToHost);
    cudaFree(dev);
    return (int)e;
}
