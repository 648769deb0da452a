// Expert routing: the stable order of (token, slot) entries by expert, the
// weighted sum of the experts' rows back into token order, and its gradient.
#include <cooperative_groups.h>

#include "device_util.cuh"
#include "launch_nvfp4.h"

namespace cg = cooperative_groups;

namespace tsfn {

namespace {

// ---------------------------------------------------------------------------
// sort
// ---------------------------------------------------------------------------
//
// A counting sort in one cluster, each warp taking consecutive entries so that
// the order is stable without atomics.  Pass 1 counts each warp's entries per
// expert (the lanes with the same expert find each other with match.any; the
// first adds their number).  A thread per expert then turns the counts into
// offsets: over the warps of the block, over the blocks of the cluster (their
// totals read through distributed shared memory) and, by a block scan of the
// counts rounded up to `align`, over the experts.  Pass 2 reads the ids again
// (from L2) and an entry's row is its warp's offset plus its rank among the
// lanes with the same expert.

constexpr int kSortThreads = 1024;
constexpr int kSortCluster = 8;

__global__ void __launch_bounds__(kSortThreads, 1) moe_sort_kernel(const __grid_constant__ SortArgs a)
{
    extern __shared__ int32_t smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nthr = blockDim.x, nw = nthr >> 5;
    const int E = a.E;
    int32_t *hist = smem;           // [nw][E] counts, then each warp's next row
    int32_t *total = hist + nw * E; // [E] this block's counts
    int32_t *used = total + E;      // [E] the row behind an expert's last entry
    int32_t *next = used + E;       // [E] the next expert's first row
    int32_t *carry = next + E;      // [32] the warps' sums

    for (int i = tid; i < nw * E; i += nthr)
        hist[i] = 0;
    __syncthreads();
    pdl_wait();

    const int rank = (int)cluster.block_rank();
    const int64_t begin = ((int64_t)rank * nw + warp) * a.per_warp;
    const int64_t end = begin + a.per_warp < a.n ? begin + a.per_warp : a.n;
    int32_t *mine = hist + warp * E;
    for (int64_t i0 = begin; i0 < end; i0 += 32) {
        const int64_t i = i0 + lane;
        const int id = i < end ? __ldg(a.ids + i) : -1;
        const bool held = id >= 0 && id < E;
        const unsigned same = __match_any_sync(0xffffffffu, held ? id : -1);
        if (held && lane == __ffs(same) - 1)
            mine[id] += __popc(same);
        __syncwarp();
    }
    __syncthreads();
    for (int e = tid; e < E; e += nthr) {  // counts -> offsets inside the block
        int32_t sum = 0;
        for (int w = 0; w < nw; ++w) {
            const int32_t c = hist[w * E + e];
            hist[w * E + e] = sum;
            sum += c;
        }
        total[e] = sum;
    }
    cluster.sync();

    // a thread per expert: its count in the whole call and in the blocks before
    // this one, and its first row by a scan of the rounded counts
    const int blocks = (int)cluster.num_blocks();
    int32_t before = 0, all = 0;
    if (tid < E) {
        for (int b = 0; b < blocks; ++b) {
            const int32_t c = *cluster.map_shared_rank(total + tid, b);
            before += b < rank ? c : 0;
            all += c;
        }
    }
    const int32_t padded = (all + a.align - 1) / a.align * a.align;
    int32_t scan = padded;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int32_t up = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o)
            scan += up;
    }
    if (lane == 31)
        carry[warp] = scan;
    __syncthreads();
    int32_t start = scan - padded;
    for (int w = 0; w < warp; ++w)
        start += carry[w];
    if (tid < E) {
        used[tid] = start + all;
        next[tid] = start + padded;
        for (int w = 0; w < nw; ++w)
            hist[w * E + tid] += start + before;
        if (rank == 0) {
            a.start[tid] = start;
            a.count[tid] = all;
            if (tid == E - 1)
                a.start[E] = start + padded;
        }
    }
    __syncthreads();
    // rows without an entry: behind each expert's last one, and behind the last expert
    const int threads = blocks * nthr;
    for (int e = rank * nw + warp; e < E; e += blocks * nw)
        for (int32_t r = used[e] + lane; r < next[e]; r += 32)
            a.row_src[r] = -1;
    for (int64_t r = next[E - 1] + (int64_t)rank * nthr + tid; r < a.rows; r += threads)
        a.row_src[r] = -1;
    pdl_launch_dependents();

    for (int64_t i0 = begin; i0 < end; i0 += 32) {
        const int64_t i = i0 + lane;
        const int id = i < end ? __ldg(a.ids + i) : -1;
        const bool held = id >= 0 && id < E;
        const unsigned same = __match_any_sync(0xffffffffu, held ? id : -1);
        int32_t row = -1;
        if (held)
            row = mine[id] + __popc(same & ((1u << lane) - 1));
        __syncwarp();
        if (held && lane == __ffs(same) - 1)
            mine[id] += __popc(same);
        __syncwarp();
        if (i < end) {
            a.row_of[i] = row;
            if (held)
                a.row_src[row] = (int32_t)i;
        }
    }
    cluster.sync();  // a block's counts stay readable until every block is done
}

// ---------------------------------------------------------------------------
// combine and its gradient
// ---------------------------------------------------------------------------

constexpr int kSlots = 8;  // slots whose rows are in flight together

__device__ __forceinline__ bool row_ok(int64_t r, int64_t rows) { return r >= 0 && r < rows; }

// One thread per chunk of 8 columns of an output row.
__global__ void __launch_bounds__(256) moe_combine_kernel(const __grid_constant__ CombineArgs a)
{
    const int64_t t = blockIdx.x;
    const int c = blockIdx.y * blockDim.x + threadIdx.x;
    pdl_wait();
    if (c >= (int)(a.H >> 3))
        return;
    float acc[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
        acc[e] = 0.0f;
    const int32_t *row_of = a.row_of + t * a.k;
    for (int j0 = 0; j0 < a.k; j0 += kSlots) {
        uint4 v[kSlots];
        float w[kSlots];
        bool on[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            const bool slot = j0 + j < a.k;
            const int64_t r = slot ? (int64_t)__ldg(row_of + j0 + j) : -1;
            on[j] = row_ok(r, a.rows);
            w[j] = 1.0f;
            if (on[j]) {
                v[j] = ld_stream(a.y + r * a.ldy + (int64_t)c * 8);
                if (a.weights != nullptr)
                    w[j] = __ldg(a.weights + t * a.k + j0 + j);
            }
        }
        if (j0 + kSlots >= a.k)
            pdl_launch_dependents();
#pragma unroll
        for (int j = 0; j < kSlots; ++j)
            if (on[j]) {
                float f[8];
                unpack8(v[j], f);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    acc[e] = fmaf(w[j], f[e], acc[e]);
            }
    }
    st_v4(a.out + t * a.ldo + (int64_t)c * 8, pack8(acc));
}

// One block per token: dout's chunk is read once for up to 8 slots, whose rows
// of y are read and whose rows of dy are written with it; the dot products are
// summed over the block in a fixed order.
constexpr int kGradThreads = 256;

__global__ void __launch_bounds__(kGradThreads) moe_combine_grad_kernel(const __grid_constant__ CombineArgs a)
{
    __shared__ float part[kGradThreads / 32][kSlots];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nc = (int)(a.H >> 3);
    pdl_wait();
    const uint16_t *drow = a.dout + t * a.ldd;
    for (int j0 = 0; j0 < a.k; j0 += kSlots) {
        int64_t r[kSlots];
        float w[kSlots], dot[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            r[j] = j0 + j < a.k ? (int64_t)__ldg(a.row_of + t * a.k + j0 + j) : -1;
            if (!row_ok(r[j], a.rows))
                r[j] = -1;
            w[j] = r[j] >= 0 ? __ldg(a.weights + t * a.k + j0 + j) : 0.0f;
            dot[j] = 0.0f;
        }
        for (int c = tid; c < nc; c += kGradThreads) {
            uint4 y[kSlots];
            const uint4 dv = ld_keep(drow + (int64_t)c * 8);
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (r[j] >= 0)
                    y[j] = ld_stream(a.y + r[j] * a.ldy + (int64_t)c * 8);
            float d[8];
            unpack8(dv, d);
#pragma unroll
            for (int j = 0; j < kSlots; ++j)
                if (r[j] >= 0) {
                    float f[8], o[8];
                    unpack8(y[j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        dot[j] = fmaf(d[e], f[e], dot[j]);
                        o[e] = __fmul_rn(w[j], d[e]);
                    }
                    st_v4(a.out + r[j] * a.ldo + (int64_t)c * 8, pack8(o));
                }
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            dot[j] = warp_sum(dot[j]);
            if (lane == 0)
                part[warp][j] = dot[j];
        }
        __syncthreads();
        if (tid < kSlots && j0 + tid < a.k) {
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < kGradThreads / 32; ++i)
                s += part[i][tid];
            a.dweights[t * a.k + j0 + tid] = s;
        }
        __syncthreads();
    }
    pdl_launch_dependents();
}

}  // namespace

cudaError_t launch_sort(const SortArgs &a, bool pdl, cudaStream_t stream)
{
    SortArgs b = a;
    // a block for up to 8192 entries (8 steps of a warp), else a cluster
    const int blocks = a.n > 8192 ? kSortCluster : 1;
    const int64_t want = (a.n + 31) / 32;
    int warps = blocks > 1 || want >= 32 ? 32 : (want < 1 ? 1 : (int)want);
    const int least = (a.E + 31) / 32;  // a thread per expert
    warps = warps < least ? least : warps;
    const int64_t all = (int64_t)blocks * warps;
    b.per_warp = ((a.n + all - 1) / all + 31) / 32 * 32;
    const size_t smem = (size_t)((warps + 3) * a.E + 32) * sizeof(int32_t);
    static std::atomic<bool> grown[kMaxCachedDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    if (dev >= kMaxCachedDevices || !grown[dev].load(std::memory_order_relaxed)) {
        err = cudaFuncSetAttribute(moe_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (35 * 1024 + 32) * (int)sizeof(int32_t));
        if (err != cudaSuccess)
            return err;
        if (dev < kMaxCachedDevices)
            grown[dev].store(true, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)blocks);
    cfg.blockDim = dim3((unsigned)(warps * 32));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)blocks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = pdl ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, moe_sort_kernel, b);
}

cudaError_t launch_combine(const CombineArgs &a, bool pdl, cudaStream_t stream)
{
    const int nc = (int)(a.H / 8);
    const int segs = (nc + 255) / 256;
    const int nthr = ((nc + segs - 1) / segs + 31) / 32 * 32;
    const dim3 grid((unsigned)a.T, (unsigned)((nc + nthr - 1) / nthr));
    return launch_kernel(moe_combine_kernel, grid, dim3((unsigned)nthr), 0, stream, pdl, a);
}

cudaError_t launch_combine_grad(const CombineArgs &a, bool pdl, cudaStream_t stream)
{
    return launch_kernel(moe_combine_grad_kernel, dim3((unsigned)a.T), dim3(kGradThreads), 0, stream, pdl, a);
}

}  // namespace tsfn
