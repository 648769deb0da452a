// Test-only kernel that stands for a predecessor in a chain of dependent
// launches: it lets the next kernel start at once, holds the stream for a given
// time (a communication kernel that waits for a late rank), and only then writes
// what the next kernel reads.
#include <cstdint>

#include <cuda_runtime.h>

namespace {

__device__ __forceinline__ unsigned long long now_ns()
{
    unsigned long long t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// One block.  The hold ends by the timer, or by a count of SM cycles.
__global__ void hold_then_copy(unsigned long long ns, long long cycles, const uint8_t *from, uint8_t *to, int64_t bytes)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const unsigned long long t0 = now_ns();
    const long long c0 = clock64();
    while (now_ns() - t0 < ns && clock64() - c0 < cycles)
        __nanosleep(1000);
    __syncthreads();
    for (int64_t i = threadIdx.x; i < bytes; i += blockDim.x)
        to[i] = from[i];
}

}  // namespace

extern "C" __attribute__((visibility("default"))) int pdl_hold(uint64_t ns, const void *from, void *to, int64_t bytes,
                                                                void *stream)
{
    hold_then_copy<<<1, 256, 0, static_cast<cudaStream_t>(stream)>>>(ns, 4 * (long long)ns, static_cast<const uint8_t *>(from),
                                                                     static_cast<uint8_t *>(to), bytes);
    return (int)cudaGetLastError();
}
