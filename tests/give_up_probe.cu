// Test-only build of the product kernels whose waits run out at a chosen time
// after a block's start (and have a limit of about 1 ms instead of 2 s), with a
// kernel that takes over the shared memory that their blocks leave and looks for
// anything that still arrives there.
#define TSFN_RUN_OUT
#define TSFN_WAIT_CYCLES 2000000LL
#include "nvfp4_gemm.cu"

namespace {

constexpr int kWords = (232448 - 1024) / 4;

__device__ __forceinline__ uint32_t pattern(int i) { return 0x9E3779B9u * (uint32_t)(i + 1) ^ blockIdx.x; }

__global__ void __launch_bounds__(1024, 1) squat_kernel(uint32_t *bad)
{
    extern __shared__ uint32_t words[];
    for (int i = threadIdx.x; i < kWords; i += blockDim.x)
        words[i] = pattern(i);
    __syncthreads();
    const long long t0 = clock64();
    while (clock64() - t0 < 20000) {
    }
    __syncthreads();
    uint32_t n = 0;
    for (int i = threadIdx.x; i < kWords; i += blockDim.x)
        n += static_cast<volatile uint32_t *>(words)[i] != pattern(i);
    if (n != 0)
        atomicAdd(bad, n);
    tsfn::pdl_wait();  // (this kernel ends after the one before)
}

}  // namespace

#define TS_TEST extern "C" __attribute__((visibility("default")))

// Waits that begin `cycles` after their block's start run out.
TS_TEST int set_run_out(int64_t cycles)
{
    const long long v = cycles;
    return (int)cudaMemcpyToSymbol(tsfn::g_run_out, &v, sizeof(v));
}

TS_TEST int stalls(uint32_t *count) { return (int)tsfn::read_stalled_waits(count); }

// Over the SMs' shared memory, as it becomes free.
TS_TEST int squat(uint32_t *bad, void *stream)
{
    const int bytes = kWords * 4;
    const cudaError_t err = cudaFuncSetAttribute(squat_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err != cudaSuccess)
        return (int)err;
    return (int)tsfn::launch_kernel(squat_kernel, dim3((unsigned)tsfn::current_device_sms()), dim3(1024), (size_t)bytes,
                                    static_cast<cudaStream_t>(stream), true, bad);
}

// The arguments of ts_nvfp4_grouped_gemm, or of ts_nvfp4_gemm where E is 0.  Sizes are the caller's to check.
TS_TEST int product(const void *a, const void *a_scale, const void *b, const void *b_scale, const float *alpha,
                    const int32_t *start, const int32_t *count, int64_t E, int64_t rows, int64_t entries, int64_t N,
                    int64_t K, void *out, int64_t ldo, void *stream)
{
    tsfn::GemmArgs g{};
    g.tok = static_cast<const uint8_t *>(a);
    g.tok_sf = static_cast<const uint8_t *>(a_scale);
    g.tok_rows = rows;
    g.wgt = static_cast<const uint8_t *>(b);
    g.wgt_sf = static_cast<const uint8_t *>(b_scale);
    g.alpha = alpha;
    g.N = N;
    g.K = K;
    g.out = static_cast<uint16_t *>(out);
    g.ldo = ldo;
    g.start = start;
    g.count = count;
    g.experts = (int)E;
    g.entries = entries;
    return (int)tsfn::launch_nvfp4_gemm(g, false, static_cast<cudaStream_t>(stream));
}
