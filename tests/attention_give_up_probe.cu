// Test-only build of the prompt attention whose waits run out at a chosen time
// after a block's start (and have a limit of about 1 ms instead of 2 s), with a
// kernel that takes over the shared memory that its blocks leave and looks for
// anything that still arrives there.
#define TSFN_RUN_OUT
#define TSFN_WAIT_CYCLES 2000000LL
#include "attn_prompt.cu"

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

TS_TEST int stalls(uint32_t *count) { return (int)tsfn::read_attn_stalled_waits(count); }

TS_TEST int64_t workspace(int64_t D) { return tsfn::attn_prompt_workspace(D); }

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

// The first kernel of many rows (causal, contiguous q and out), or the one that joins its parts.  Sizes are the
// caller's to check.
template <int D>
static cudaError_t launch(const tsfn::AttnArgs &a, bool join, cudaStream_t stream)
{
    if (join)
        return tsfn::launch_kernel(tsfn::attn_join_rows_kernel<D>, dim3(tsfn::kBlocks, tsfn::kRows / 8), dim3(256), (size_t)0, stream, false, a,
                                   tsfn::kBlocks);
    const int bytes = tsfn::Smem<D>::kBytes;
    const cudaError_t err = cudaFuncSetAttribute(tsfn::attn_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    cudaFuncAttributes of;
    if (err != cudaSuccess || cudaFuncGetAttributes(&of, tsfn::attn_prompt_kernel<D>) != cudaSuccess || of.numRegs != 128)
        return cudaErrorInvalidConfiguration;
    return tsfn::launch_kernel(tsfn::attn_prompt_kernel<D>, dim3(tsfn::kBlocks), dim3(tsfn::kThreads), (size_t)bytes, stream, false, a);
}

TS_TEST int attend(const void *q, int64_t T, int64_t q_heads, const int32_t *cu, int64_t B, void *pages, int64_t num_pages,
                   int64_t page_size, int64_t heads, int64_t D, const float *k_scale, const float *v_scale, const int32_t *table,
                   int64_t max_pages, const int32_t *lens, float scale, void *out, float *lse, void *space, int join, void *stream)
{
    tsfn::AttnArgs a{};
    a.q = static_cast<const uint16_t *>(q);
    a.ldq = a.ldo = q_heads * D;
    a.T = T;
    a.hq = (int)q_heads;
    a.group = (int)(q_heads / heads);
    a.div_group = tsfn::div_magic((uint32_t)a.group);
    a.cu = cu;
    a.B = (int)B;
    a.cache.pages = static_cast<uint8_t *>(pages);
    a.cache.slots = num_pages * page_size;
    a.cache.num_pages = (int)num_pages;
    a.cache.page_size = (int)page_size;
    a.cache.div_page = tsfn::div_magic((uint32_t)page_size);
    a.cache.heads = (int)heads;
    a.cache.k_scale = k_scale;
    a.cache.v_scale = v_scale;
    a.D = (int)D;
    a.table = table;
    a.max_pages = max_pages;
    a.lens = lens;
    a.scale = scale;
    a.causal = true;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.partial = static_cast<float *>(space);
    const cudaStream_t on = static_cast<cudaStream_t>(stream);
    return (int)(D == 64 ? launch<64>(a, join != 0, on) : launch<128>(a, join != 0, on));
}
