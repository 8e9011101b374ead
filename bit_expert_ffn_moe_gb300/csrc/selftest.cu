// selftest.cu -- failure-detection self-test of the bounded device waits.
//
// Every barrier wait in this library's kernels gives up after a bounded time, records
// MOE_ERR_TIMEOUT in the workspace status word and lets its kernel finish, so a copy or a signal
// that never arrives surfaces as an error status that the host reads, not as a hung GPU.
// moe_selftest_wait_timeout exercises exactly that path without faulting anything: one thread
// waits on an mbarrier phase that no thread ever completes, with a short time limit; the wait
// runs out, the status is recorded and the kernel returns normally, leaving the context usable.
// Meanwhile another thread has issued all of its copies without having seen anybody give up, and
// lets them land (land, common.cuh) before the CTA looks at its shared memory and ends.
#include "common.cuh"

namespace moe {
namespace {

constexpr int kPlaces = 4, kSteps = 6, kBytes = 512;  // a ring, and copies of the control block's last bytes into it

__global__ void wait_timeout_kernel(Ctrl* ctrl, unsigned long long limit_ns) {
    __shared__ __align__(128) unsigned char ring[kPlaces][kBytes];
    __shared__ __align__(8) uint64_t bar, full[kPlaces];
    const unsigned char* from = reinterpret_cast<const unsigned char*>(ctrl + 1) - kSteps * kBytes;
    for (int i = threadIdx.x; i < kPlaces * kBytes; i += blockDim.x) ring[0][i] = ~from[i % kBytes];  // (something else)
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        for (int i = 0; i < kPlaces; ++i) mbar_init(&full[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    asm volatile("fence.proxy.async;" ::: "memory");
    __syncthreads();
    bool done = false;
    if (threadIdx.x == 0) {
        unsigned long long t0, t;
        asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t0));
        while (true) {
            if (mbar_try_wait(&bar, 0)) {  // phase 0 of a barrier expecting one arrival that never comes
                done = true;
                break;
            }
            asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
            if (t - t0 > limit_ns) break;
        }
    } else if (threadIdx.x == 32) {
        volatile int never = 0;
        for (int i = 0; i < kSteps; ++i) {
            // (a place is free for its second step once it is full: nobody reads it)
            if (i >= kPlaces) mbar_wait(&full[i % kPlaces], 0, &never, nullptr, 100000000LL);
            mbar_arrive_expect_tx(&full[i % kPlaces], kBytes);
            bulk_load(ring[i % kPlaces], from + i * kBytes, kBytes, &full[i % kPlaces]);
        }
        land(full, kSteps, kPlaces);
    }
    bool landed = true;
    __syncthreads();
    for (int i = kSteps - kPlaces; i < kSteps; ++i)
        for (int b = threadIdx.x; b < kBytes; b += blockDim.x) landed &= ring[i % kPlaces][b] == from[i * kBytes + b];
    landed = __syncthreads_and(landed);
    if (threadIdx.x == 0 && !done) set_status(&ctrl->status, landed ? MOE_ERR_TIMEOUT : MOE_ERR_CUDA);
}

}  // namespace
}  // namespace moe

using namespace moe;

extern "C" moe_status moe_selftest_wait_timeout(void* ws, size_t ws_bytes, int limit_us, moe_stream_t stream) {
    if (ws == nullptr || (reinterpret_cast<uintptr_t>(ws) % 256) != 0 || ws_bytes < sizeof(Ctrl))
        return MOE_ERR_WORKSPACE;
    if (limit_us < 1 || limit_us > 1000000) return MOE_ERR_INVALID_ARG;
    Ctrl* ctrl = static_cast<Ctrl*>(ws);
    wait_timeout_kernel<<<1, 64, 0, (cudaStream_t)stream>>>(ctrl, 1000ull * (unsigned long long)limit_us);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
