// Internal interface between the checks of the NVFP4 and expert-routing entry
// points (api_nvfp4_moe.cu) and their launchers.  Sizes are validated; the
// contents of the index arrays are not, and the kernels check them.  Any input may
// be the output of the kernel before, which still runs when a dependent launch
// begins: the kernels read none of them through the non-coherent path (ld.global.nc),
// whose loads may also be moved ahead of the wait for that kernel.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "launch.h"

namespace tsfn {

// Rows of x to NVFP4 or copied, row t to itself (row_of == nullptr) or to the
// k rows row_of[t*k ..].
struct RowsArgs {
    const uint16_t *x;
    int64_t ldx;
    int64_t T;
    int64_t K;               // columns
    const int32_t *row_src;  // rows with a negative entry are left out (may be null)
    const int32_t *row_of;   // [T, k] destinations, or null
    int k;
    int64_t rows;            // rows of the output
    uint16_t *out;           // copy form
    const float *g;          // NVFP4 form: global scale
    uint8_t *codes;
    uint8_t *sf;
    int sf_layout;
    int64_t sf_rows;         // rows of the scale-factor buffer
    int64_t sf_cols;         // K/16, padded to a multiple of 4 when swizzled
    int tpr_log2;            // lanes per row, as a power of two
};

struct DequantArgs {
    const uint8_t *codes;
    const uint8_t *sf;
    int sf_layout;
    int64_t sf_cols;
    int64_t T;
    int64_t K;
    const float *g;
    const int32_t *row_src;
    uint16_t *out;
    int64_t ldo;
    int tpr_log2;
};

struct CombineArgs {
    const uint16_t *y;
    int64_t rows;
    int64_t ldy;
    int64_t H;
    const int32_t *row_of;
    const float *weights;  // may be null (combine): 1
    int64_t T;
    int k;
    uint16_t *out;  // combine: out; gradient: dy
    int64_t ldo;
    const uint16_t *dout;  // gradient only
    int64_t ldd;
    float *dweights;
};

struct SortArgs {
    const int32_t *ids;
    int64_t n;  // T * k entries
    int E;
    int align;
    int64_t rows;  // length of row_src
    int32_t *row_of;
    int32_t *row_src;
    int32_t *start;
    int32_t *count;
    int warps;         // warps of a block that have entries
    int64_t per_warp;  // entries of one warp, a multiple of 32
};

struct GemmArgs {
    const uint8_t *tok;  // codes of the tokens' matrix [tok_rows, K/2]
    const uint8_t *tok_sf;
    int64_t tok_rows;
    const uint8_t *wgt;  // codes of the weights [experts * N, K/2]
    const uint8_t *wgt_sf;
    const float *alpha;
    int64_t N;
    int64_t K;
    uint16_t *out;
    int64_t ldo;
    // grouped form (experts > 0)
    const int32_t *start;
    const int32_t *count;
    int experts;
    int64_t entries;
};

// As launch_kernel, in clusters of `cluster` blocks.
template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream, bool pdl,
                            unsigned cluster, Args &&...args)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cluster;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
}

cudaError_t launch_quantize(const RowsArgs &a, bool pdl, cudaStream_t stream);
cudaError_t launch_dequantize(const DequantArgs &a, bool pdl, cudaStream_t stream);
cudaError_t launch_dispatch(const RowsArgs &a, bool pdl, cudaStream_t stream);
cudaError_t launch_combine(const CombineArgs &a, bool pdl, cudaStream_t stream);
cudaError_t launch_combine_grad(const CombineArgs &a, bool pdl, cudaStream_t stream);
cudaError_t launch_sort(const SortArgs &a, bool pdl, cudaStream_t stream);
cudaError_t launch_nvfp4_gemm(const GemmArgs &a, bool pdl, cudaStream_t stream);
cudaError_t read_stalled_waits(uint32_t *count);

}  // namespace tsfn
