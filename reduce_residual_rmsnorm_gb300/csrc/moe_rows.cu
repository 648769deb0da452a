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
// A counting sort in one cluster of 8 or 16 blocks, each warp taking consecutive
// entries so that the order is stable.  Pass 1 counts each warp's entries per
// expert in shared memory.  A thread per expert turns the counts into offsets:
// over the warps of the block, over the blocks of the cluster (their totals read
// through distributed shared memory) and, by a block scan of the counts rounded
// up to `align`, over the experts.  Pass 2: an entry's row is its warp's offset
// plus its rank among the lanes with the same expert, found by a vote on each bit
// of the id (match.any goes over the distinct ids one by one: 41.2 us against 28.6
// at 32768 x 8 entries over 256 experts).  What bounds it is latency, and with
// many entries the scattered stores of a few SMs: ids are loaded 8 steps ahead,
// and kept in registers between the passes where a warp has no more than 256.
// us over 8 and 16 blocks: 256 x 8 entries over 64 experts 3.3 3.35, 1024 x 8 5.2 4.0,
// 8192 x 8 8.9 6.8, 32768 x 8 26.6 16.5; 16 x 8 entries take 2.8 (3.2 with starts at
// multiples of 128, whose row_src has 8 K entries).  One block instead of the
// cluster measured 2.5 and 3.5 us on the last two, 64 at 8192 x 8.

constexpr int kSortThreads = 1024;
constexpr int kSortSteps = 8;  // steps of 32 entries whose ids are loaded together

template <int BLOCKS>
__global__ void __launch_bounds__(kSortThreads, 1) moe_sort_kernel(const __grid_constant__ SortArgs a)
{
    extern __shared__ int32_t smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nthr = blockDim.x;
    const int E = a.E, nw = a.warps;  // warps with entries
    int32_t *hist = smem;             // [nw][E] counts, then each warp's next row after the expert's base
    int32_t *total = hist + nw * E;   // [E] this block's counts
    int32_t *base = total + E;        // [E] the expert's first row of this block
    int32_t *used = base + E;         // [E] the row behind an expert's last entry
    int32_t *next = used + E;         // [E] the next expert's first row
    int32_t *carry = next + E;        // [32] the warps' sums

    for (int i = tid; i < nw * E; i += nthr)
        hist[i] = 0;
    __syncthreads();
    pdl_wait();

    const int rank = (int)blockIdx.x;  // the grid is one cluster
    const int64_t begin = ((int64_t)rank * nw + warp) * a.per_warp;
    const int64_t stop = begin + a.per_warp < a.n ? begin + a.per_warp : a.n;
    const int64_t end = warp < nw ? stop : begin;
    int32_t *mine = hist + warp * E;
    int id[kSortSteps];
    auto load = [&](int64_t i0) {
#pragma unroll
        for (int u = 0; u < kSortSteps; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            const int v = i < end ? a.ids[i] : -1;
            id[u] = v >= 0 && v < E ? v : -1;
        }
    };
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kSortSteps) {
        load(i0);
#pragma unroll
        for (int u = 0; u < kSortSteps; ++u)
            if (id[u] >= 0)
                atomicAdd(mine + id[u], 1);
    }
    __syncthreads();
    if (tid < E) {  // counts -> offsets inside the block
        int32_t sum = 0;
#pragma unroll 4
        for (int w = 0; w < nw; ++w) {
            const int32_t c = hist[w * E + tid];
            hist[w * E + tid] = sum;
            sum += c;
        }
        total[tid] = sum;
    }
    cluster.sync();

    // a thread per expert: its count in the whole call and in the blocks before
    // this one, and its first row by a scan of the rounded counts
    int32_t before = 0, all = 0;
    if (tid < E) {
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) {
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
        base[tid] = start + before;
        if (rank == 0) {
            a.start[tid] = start;
            a.count[tid] = all;
            if (tid == E - 1)
                a.start[E] = start + padded;
        }
    }
    __syncthreads();
    pdl_launch_dependents();

    const int bits = 32 - __clz(E - 1);
    for (int64_t i0 = begin; i0 < end; i0 += 32 * kSortSteps) {
        if (a.per_warp > 32 * kSortSteps)
            load(i0);
#pragma unroll
        for (int u = 0; u < kSortSteps; ++u) {
            const int64_t i = i0 + 32 * u + lane;
            if (i - lane >= end)
                break;
            const bool held = id[u] >= 0;
            unsigned same = __ballot_sync(0xffffffffu, held);  // and has the same bits
            for (int b = 0; b < bits; ++b) {
                const bool on = (id[u] >> b) & 1;
                const unsigned with = __ballot_sync(0xffffffffu, on);
                same &= on ? with : ~with;
            }
            int32_t row = -1;
            if (held)
                row = base[id[u]] + mine[id[u]] + __popc(same & ((1u << lane) - 1));
            __syncwarp();
            if (held && lane == __ffs(same) - 1)
                mine[id[u]] += __popc(same);
            __syncwarp();
            if (i < end) {
                a.row_of[i] = row;
                if (held)
                    a.row_src[row] = (int32_t)i;
            }
        }
    }
    // rows without an entry: behind each expert's last one, and behind the last expert
    const int threads = BLOCKS * nthr, warps = threads >> 5;
    for (int e = rank * (nthr >> 5) + warp; e < E; e += warps)
        for (int32_t r = used[e] + lane; r < next[e]; r += 32)
            a.row_src[r] = -1;
    for (int64_t r = next[E - 1] + (int64_t)rank * nthr + tid; r < a.rows; r += threads)
        a.row_src[r] = -1;
    cluster.sync();  // a block's counts stay readable until every block is done
}

// ---------------------------------------------------------------------------
// combine and its gradient
// ---------------------------------------------------------------------------

constexpr int kSlots = 8;  // slots whose rows are in flight together

// For data that is read again, once for each group of slots.
__device__ __forceinline__ uint4 ld_cached(const void *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ bool row_ok(int64_t r, int64_t rows) { return r >= 0 && r < rows; }

// One thread per chunk of 8 columns of an output row.  Bound by memory: 8192 x 8 rows
// of 7168 in 158.7 us, 98 % of the copy rate; with few tokens by latency, so a group's
// rows are looked up before the first of them is read (16 x 8 rows 1.9 us; 2.4 with
// each lookup beside its load).
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
        int32_t r[kSlots];
        uint4 v[kSlots];
        float w[kSlots];
        bool on[kSlots];
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            r[j] = j0 + j < a.k ? row_of[j0 + j] : -1;
            on[j] = row_ok(r[j], a.rows);
        }
#pragma unroll
        for (int j = 0; j < kSlots; ++j) {
            w[j] = 1.0f;
            if (on[j]) {
                v[j] = ld_stream(a.y + r[j] * a.ldy + (int64_t)c * 8);
                if (a.weights != nullptr)
                    w[j] = a.weights[t * a.k + j0 + j];
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

// One block per token: dout's chunk is read once for up to SLOTS slots, whose
// rows of y are read and whose rows of dy are written with it; the dot products
// are summed over the block in an order that H alone fixes.  Bound by memory:
// 4096 x 8 rows of 7168 in 156.5 us, 94 % of the copy rate.  Blocks of up to 512
// threads measured 173.7 us there, 4.8 against 4.7 at 16 tokens.
constexpr int kGradThreads = 256;

template <int SLOTS>
__global__ void __launch_bounds__(kGradThreads, SLOTS > 4 ? 2 : 3) moe_combine_grad_kernel(const __grid_constant__ CombineArgs a)
{
    __shared__ float part[kGradThreads / 32][SLOTS];
    const int64_t t = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int nc = (int)(a.H >> 3);
    pdl_wait();
    const uint16_t *drow = a.dout + t * a.ldd;
    for (int j0 = 0; j0 < a.k; j0 += SLOTS) {
        int64_t r[SLOTS];
        float w[SLOTS], dot[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            r[j] = j0 + j < a.k ? (int64_t)a.row_of[t * a.k + j0 + j] : -1;
            if (!row_ok(r[j], a.rows))
                r[j] = -1;
            w[j] = r[j] >= 0 ? a.weights[t * a.k + j0 + j] : 0.0f;
            dot[j] = 0.0f;
        }
        for (int c = tid; c < nc; c += blockDim.x) {
            uint4 y[SLOTS];
            const uint4 dv = ld_cached(drow + (int64_t)c * 8);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
                if (r[j] >= 0)
                    y[j] = ld_stream(a.y + r[j] * a.ldy + (int64_t)c * 8);
            float d[8];
            unpack8(dv, d);
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
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
        for (int j = 0; j < SLOTS; ++j) {
            dot[j] = warp_sum(dot[j]);
            if (lane == 0)
                part[warp][j] = dot[j];
        }
        __syncthreads();
        if (tid < SLOTS && j0 + tid < a.k) {
            float s = 0.0f;
            for (int i = 0; i < (int)(blockDim.x >> 5); ++i)
                s += part[i][tid];
            a.dweights[t * a.k + j0 + tid] = s;
        }
        __syncthreads();
    }
    pdl_launch_dependents();
}

}  // namespace

namespace {

template <int BLOCKS>
cudaError_t launch_sort_over(const SortArgs &a, bool pdl, cudaStream_t stream)
{
    SortArgs b = a;
    const int64_t steps = (a.n + 32 * BLOCKS - 1) / (32 * BLOCKS);  // of 32 entries, per block
    b.warps = steps < 1 ? 1 : (steps < 32 ? (int)steps : 32);
    const int64_t all = (int64_t)BLOCKS * b.warps;
    b.per_warp = ((a.n + all - 1) / all + 31) / 32 * 32;
    // a thread per expert, and enough to fill row_src with few stores each
    const int64_t fill = a.rows / (8 * BLOCKS) < 1024 ? (a.rows / (8 * BLOCKS) + 31) / 32 * 32 : 1024;
    int nthr = b.warps * 32;
    nthr = nthr < (a.E + 31) / 32 * 32 ? (a.E + 31) / 32 * 32 : nthr;
    nthr = nthr < fill ? (int)fill : nthr;
    const size_t smem = (size_t)((b.warps + 4) * a.E + 32) * sizeof(int32_t);
    static std::atomic<bool> grown[kMaxCachedDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    if (dev >= kMaxCachedDevices || !grown[dev].load(std::memory_order_relaxed)) {
        err = cudaFuncSetAttribute(moe_sort_kernel<BLOCKS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                   (36 * 1024 + 32) * (int)sizeof(int32_t));
        if (err == cudaSuccess && BLOCKS > 8)
            err = cudaFuncSetAttribute(moe_sort_kernel<BLOCKS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (err != cudaSuccess)
            return err;
        if (dev < kMaxCachedDevices)
            grown[dev].store(true, std::memory_order_relaxed);
    }
    return launch_clusters(moe_sort_kernel<BLOCKS>, dim3(BLOCKS), dim3((unsigned)nthr), smem, stream, pdl, BLOCKS, b);
}

}  // namespace

cudaError_t launch_sort(const SortArgs &a, bool pdl, cudaStream_t stream)
{
    return a.n <= 4096 ? launch_sort_over<8>(a, pdl, stream) : launch_sort_over<16>(a, pdl, stream);
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
    // no more threads than chunks and no more slots in registers than the call
    // has: 4096 x 2 rows of 1024 in 7.1 us, 20.5 with 256 threads and 8 slots
    const int nc = (int)(a.H / 8);
    const dim3 grid((unsigned)a.T), block((unsigned)(nc < kGradThreads ? (nc + 31) / 32 * 32 : kGradThreads));
    if (a.k <= 4)
        return launch_kernel(moe_combine_grad_kernel<4>, grid, block, 0, stream, pdl, a);
    return launch_kernel(moe_combine_grad_kernel<kSlots>, grid, block, 0, stream, pdl, a);
}

}  // namespace tsfn
