// NVFP4 matrix products on the fifth-generation tensor cores: out = alpha A B^T
// for one matrix of weights, or for each expert's with its own rows.
//
//   out[m, n] = bf16(alpha * sum_k (a sf_a)[m, k] (b sf_b)[n, k])       fp32 sums
//
// tcgen05.mma kind::mxf4nvf4 multiplies 64 packed E2M1 values of K per
// instruction with one E4M3 scale factor per 16, from shared memory into
// tensor memory.  Its operands are named P (128 rows a block, the accumulator's
// lanes) and Q (the accumulator's columns) here.  Which matrix is which:
//   - up to 64 tokens (128 with a long K): weights on P, tokens on Q, so that a
//     tile is no wider than the tokens need (nvfp4_few_kernel).  Bound by the
//     weights' bytes, and where those are few by latency.
//   - more tokens: pairs of blocks (nvfp4_pair_kernel) with tokens on P and weights
//     on Q.  Bound by the tensor cores: 7.5 PFLOP/s at 8192 x 7168 x 7168, 86 % of
//     a tile's cycles, and by the power limit in long runs.
//   - experts: pairs with weights on P and an expert's tokens on Q, whose number of
//     columns follows them.  Bound by the experts' bytes (within 3 to 11 % of them up
//     to 64 tokens an expert), then as above.
//
// One block per SM, persistent over the tiles.  One warp copies (two where tokens
// are few): codes by TMA under the 128-byte swizzle, 256 elements of K (128 bytes a
// row) per stage, scale factors in the 512-byte tiles of their 128x4 layout, which
// is the layout tensor memory wants.  Warp 1 multiplies: scale factors from shared
// to tensor memory, then the products.  The other warps write the finished
// accumulator, one of two, while the next tile's products run.  Every wait has a
// limit, after which the block records it and ends, once the copies, products and
// sums that its cluster has in flight have arrived.
#include <cuda.h>

#include "device_util.cuh"
#include "launch_nvfp4.h"
#include "tcgen05.cuh"

namespace tsfn {

namespace {

__device__ uint32_t g_stalled_waits;

constexpr int kThreads = 224;
constexpr int kP = 128;               // rows of P per tile
constexpr int kSfTile = 512;          // bytes of a 128-row, 64-element tile of scale factors
#ifndef TSFN_WAIT_CYCLES
#define TSFN_WAIT_CYCLES 4000000000LL
#endif
constexpr long long kWaitCycles = TSFN_WAIT_CYCLES;  // a wait's limit: about 2 s
constexpr int kSmemLimit = 232448;    // bytes of shared memory of a block

struct KernelArgs {
    const uint8_t *p_sf;
    const uint8_t *q_sf;
    const float *alpha;
    uint16_t *out;
    int64_t ldo;
    int64_t p_rows, q_rows;  // dense: rows of P and Q
    int kblocks;             // ceil(K / 64)
    int split_log2;          // dense, few tokens: 2^split_log2 blocks of a cluster share a tile's K
    int wgt_rows;            // grouped: N
    int wgt_bands;           // grouped: 128-row bands of an expert's scale factors
    int64_t tok_rows;        // grouped: rows of the sorted tokens
    const int32_t *start;
    const int32_t *count;
    int experts;
};

// One tile: the first rows of P and Q in their tensor maps, their scale-factor
// bands of 128 rows, and the part of the output it covers.
struct Tile {
    int32_t p_row, q_row;
    int32_t p_band, q_band;
    int q_bands;   // of the tile's rows of Q
    int64_t tok0;  // output rows tok0 .. tok0 + tok_n
    int tok_n;
    int64_t wgt0;  // output columns wgt0 .. wgt0 + wgt_n
    int wgt_n;
    int expert;
};

// Few tokens: weights on P, all tokens one tile of Q.
__device__ __forceinline__ Tile few_tile(const KernelArgs &a, int32_t id)
{
    Tile t;
    t.p_row = id * kP;
    t.q_row = 0;
    t.p_band = id;
    t.q_band = 0;
    t.q_bands = 1;
    t.tok0 = 0;
    t.tok_n = (int)a.q_rows;
    t.wgt0 = t.p_row;
    t.wgt_n = (int)(a.p_rows - t.p_row < kP ? a.p_rows - t.p_row : kP);
    t.expert = 0;
    return t;
}

// Pairs: tokens on P, weights on Q.  Groups of 6 P tiles pass over Q together, so
// that pairs running at the same time share rows of both (8192 x 7168 x 7168 112.5
// us, 16384 x 5120 x 5120 116.6; groups of 4 112.8 and 121.1, of 8 114.1 and 119.8,
// of 16 115.4 and 121.4).  (Tiles are fewer than 2^31, since the output fits the
// GPU: 32-bit divisions.)
template <int BN>
__device__ __forceinline__ Tile dense_tile(const KernelArgs &a, uint32_t id)
{
    constexpr uint32_t kGroup = 6;
    const uint32_t np = (uint32_t)((a.p_rows + 2 * kP - 1) / (2 * kP)), nq = (uint32_t)((a.q_rows + BN - 1) / BN);
    const uint32_t group = id / (kGroup * nq);
    const uint32_t gp = np - group * kGroup < kGroup ? np - group * kGroup : kGroup;
    const uint32_t in = id - group * kGroup * nq;
    const uint32_t q = in / gp, p = group * kGroup + in - q * gp;
    Tile t;
    t.p_row = (int32_t)(p * 2 * kP);
    t.q_row = (int32_t)(q * BN);
    t.p_band = t.p_row >> 7;
    t.q_band = t.q_row >> 7;
    t.q_bands = (BN + 127) / 128;
    t.tok0 = t.p_row;
    t.tok_n = (int)(a.p_rows - t.p_row < 2 * kP ? a.p_rows - t.p_row : 2 * kP);
    t.wgt0 = t.q_row;
    t.wgt_n = (int)(a.q_rows - t.q_row < BN ? a.q_rows - t.q_row : BN);
    t.expert = 0;
    return t;
}

// Pairs, grouped: weights on P, an expert's tokens on Q.  first[e]: tiles of tokens
// before expert e.  Groups of 8 tiles of an expert's tokens pass over its weights
// together, so that pairs running at the same time share rows of both (32768 tokens
// of one expert of 4096 x 7168: 326 us over all tokens first, 268 in groups; in
// groups of 4 as fast, of 16 271).
template <int BN>
__device__ __forceinline__ Tile grouped_tile(const KernelArgs &a, const int32_t *first, uint32_t id)
{
    const uint32_t nw = ((uint32_t)a.wgt_rows + 2 * kP - 1) / (2 * kP), before = id / nw;
    int lo = 0, hi = a.experts;  // the expert e with first[e] <= before < first[e + 1]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((uint32_t)first[mid] <= before)
            lo = mid;
        else
            hi = mid;
    }
    constexpr uint32_t kGroup = 8;
    const uint32_t nt = (uint32_t)(first[lo + 1] - first[lo]), from = id - (uint32_t)first[lo] * nw;
    const uint32_t group = from / (kGroup * nw);
    const uint32_t gt = nt - group * kGroup < kGroup ? nt - group * kGroup : kGroup;
    const uint32_t in = from - group * kGroup * nw;
    const uint32_t w = in / gt;
    const int t0 = (int)(group * kGroup + in - w * gt) * BN, w0 = (int)w * 2 * kP;
    const int count = a.count[lo], start = a.start[lo];
    Tile t;
    t.expert = lo;
    t.tok0 = start + t0;
    t.tok_n = count - t0 < BN ? count - t0 : BN;
    t.wgt0 = w0;
    t.wgt_n = a.wgt_rows - w0 < 2 * kP ? a.wgt_rows - w0 : 2 * kP;
    t.p_row = lo * a.wgt_rows + w0;
    t.q_row = start + t0;
    t.p_band = lo * a.wgt_bands + (w0 >> 7);
    t.q_band = t.q_row >> 7;
    t.q_bands = (t.tok_n + 127) >> 7;
    return t;
}

template <int BN, bool GROUPED>
__device__ __forceinline__ Tile pair_tile(const KernelArgs &a, const int32_t *first, int64_t id)
{
    if constexpr (GROUPED)
        return grouped_tile<BN>(a, first, (uint32_t)id);
    else
        return dense_tile<BN>(a, (uint32_t)id);
}

// Tiles of a grouped call; every thread of the block takes part and fills
// first[0 .. experts].  No more than experts with rows of their own can have: where
// they share rows the numbers stay in 32 bits, and the last experts' tiles fall away.
template <int BN>
__device__ __forceinline__ int64_t grouped_tiles(const KernelArgs &a, int32_t *first)
{
    const int lane = threadIdx.x & 31;
    for (int e = threadIdx.x; e < a.experts; e += blockDim.x) {
        const int start = a.start[e], count = a.count[e];
        const bool good = start >= 0 && (start & 127) == 0 && count > 0 && (int64_t)start + count <= a.tok_rows;
        first[e + 1] = good ? (count + BN - 1) / BN : 0;
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // inclusive scan
        const int32_t most = (int32_t)(a.tok_rows / BN) + a.experts;
        int32_t sum = 0;
        for (int e0 = 0; e0 < a.experts; e0 += 32) {
            int32_t v = e0 + lane < a.experts ? first[e0 + lane + 1] : 0;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int32_t up = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o)
                    v += up;
            }
            v = sum + v < most ? sum + v : most;
            if (e0 + lane < a.experts)
                first[e0 + lane + 1] = v;
            sum = __shfl_sync(0xffffffffu, v, 31);
        }
        if (lane == 0)
            first[0] = 0;
    }
    __syncthreads();
    return (int64_t)first[a.experts] * ((a.wgt_rows + 2 * kP - 1) / (2 * kP));
}

#ifdef TSFN_RUN_OUT
// For the tests of the give-up path, which are built with it: the waits that begin
// this many cycles after their block's start run out at once.
__device__ long long g_run_out = 1LL << 62;

__device__ __forceinline__ long long &block_start()
{
    __shared__ long long start;
    return start;
}

__device__ __forceinline__ bool run_out()
{
    return __shfl_sync(0xffffffffu, (int)(clock64() - block_start() >= g_run_out), 0) != 0;
}
#endif

// A wait ran into its limit: the block gives up, and the others of its pair or cluster
// of pairs (PEERS of them with it), whose copies and products reach its memory.
template <int PEERS>
__device__ __noinline__ void give_up(volatile int *dead)
{
    *dead = 1;
    for (uint32_t r = 0; PEERS > 1 && r < PEERS; ++r)
        st_cluster32(map_rank(smem_u32((const void *)dead), r), 1);
    atomicAdd(&g_stalled_waits, 1u);
}

// Wait with a limit, for what is in flight when a block gives up.
__device__ __noinline__ void wait_last(uint32_t bar, uint32_t parity)
{
    const long long t0 = clock64();
    while (!mbar_try_wait(bar, parity) && clock64() - t0 < kWaitCycles) {
    }
}

// The same for the copies of the last fills of the stages, with one limit for all
// (a fill that another warp or block left undone does not complete; what came of it
// has arrived by then).
__device__ __noinline__ void wait_fills(uint32_t full, uint32_t fills, uint32_t stages)
{
    const long long t0 = clock64();
    for (uint32_t i = 0; i < stages && i < fills; ++i) {
        const uint32_t fill = fills - 1 - i;
        while (!mbar_try_wait(full + 8 * (fill % stages), (fill / stages) & 1) && clock64() - t0 < kWaitCycles) {
        }
    }
}

template <bool CLUSTER>
__device__ __forceinline__ bool try_wait(uint32_t bar, uint32_t parity)
{
    return CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
}

template <bool CLUSTER, int PEERS>
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int *dead)
{
    const long long t0 = clock64();
    while (!*dead) {
        if (try_wait<CLUSTER>(bar, parity))
            return true;
        if (clock64() - t0 > kWaitCycles)
            give_up<PEERS>(dead);
    }
    return false;
}

// The whole warp waits; false in every lane when a wait ran into its limit,
// here or elsewhere in the block.  CLUSTER: for what another block sent.
template <int PEERS, bool CLUSTER = false>
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *dead)
{
#ifdef TSFN_RUN_OUT
    if (run_out()) {
        if ((threadIdx.x & 31) == 0)
            give_up<PEERS>(dead);
        __syncwarp();
        return false;
    }
#endif
    return __all_sync(0xffffffffu, try_wait<CLUSTER>(bar, parity) || wait_slow<CLUSTER, PEERS>(bar, parity, dead));
}

// ---------------------------------------------------------------------------
// few tokens
// ---------------------------------------------------------------------------
//
// A tile is 128 rows of the weights and all tokens, so that a row of weights is
// read once.  Where few tiles leave SMs idle, 2 or 4 blocks of a cluster share a
// tile's K and each sums up a share of the tokens from all of them, in their
// order.  Latency counts here: two warps copy, since an issue takes about 100
// cycles; the partial sums travel by stores that the receiving barrier counts,
// with no fence; the cluster's last arrival orders nothing (3.8 us below with one
// that waits for the outputs); and a tile is found before the dependency wait.
// 1 x 4096 x 4096 takes 3.5 us (1.4 of bytes): about 0.2 us from the wait to the
// first copy's issue, 0.9 to its arrival, 0.9 for the four steps, 0.2 to the
// accumulator, 0.3 to the exchanged sums.

template <int BN>
struct Shape {
    static constexpr int kCodes = kP * 128 + BN * 128;  // bytes of codes per stage
    static constexpr int kSf = 8 * kSfTile;             // bytes of scale factors per stage
    static constexpr int kPartials = BN * kP * 4;
    static constexpr int kFixed = 1024 + kPartials;     // and alignment
    static constexpr int kStages = (kSmemLimit - kFixed - 256) / (kCodes + kSf);
    static constexpr int kSmem = kFixed + kStages * (kCodes + kSf);
    static constexpr int kSfP = 2 * BN;       // tensor-memory column of P's scale factors
    static constexpr int kSfQ = kSfP + 16;    // and of Q's
    static constexpr int kColumns = 512;      // one block per SM: all of it
    static_assert(kSfQ + 16 <= kColumns, "accumulators and scale factors fit tensor memory");
};

// What a block that gave up has in flight ends: each copying warp's copies, and the
// products.  (Out of line here and below: the kernels' ends stay short.)
__device__ __noinline__ void few_drain(int warp, uint32_t full, uint32_t fills, uint32_t stages, uint32_t drained)
{
    if (warp == 0 || warp == 6) {
        wait_fills(full, fills, stages);
    } else if (warp == 1) {
        if (elect_one())
            mma_commit(drained);
        __syncwarp();
        wait_last(drained, 0);
    }
    __syncwarp();
}

template <int BN>
__global__ void __launch_bounds__(kThreads, 1)
    nvfp4_few_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ KernelArgs a)
{
    using S = Shape<BN>;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * S::kStages + 6];
    __shared__ uint32_t tmem_at;
    __shared__ uint32_t fills_made[2];  // by the two copying warps
    __shared__ int dead_flag;
    const uint32_t pad = (1024 - (smem_u32(raw) & 1023)) & 1023;
    const uint32_t codes = smem_u32(raw) + pad;
    const uint32_t sf = codes + S::kStages * S::kCodes;
    const uint32_t sums = sf + S::kStages * S::kSf;  // the cluster's partial sums of this block's share
    volatile int *dead = &dead_flag;

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages;
    const uint32_t acc_full = empty + 8 * S::kStages, acc_empty = acc_full + 16, drained = acc_empty + 16;
    const uint32_t partial = drained + 8;  // the cluster's partial sums are here
    const int lg = a.split_log2, split = 1 << lg, rank = (int)cluster_rank();

    // four-token groups of the partial sums that this block sums up
    const int fours = ((int)a.q_rows + 3) >> 2, my_fours = rank < fours ? (fours - rank + split - 1) >> lg : 0;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_empty + 8 * i, 4);
        }
        mbar_init(drained, 1);
        mbar_init(partial, 1);
        mbar_fence_init();
        if (split > 1)
            mbar_expect_tx(partial, (uint32_t)(split * my_fours * kP * 16));
        dead_flag = 0;
#ifdef TSFN_RUN_OUT
        block_start() = clock64();
#endif
        tma_prefetch_map(&p_map);
        tma_prefetch_map(&q_map);
    }
    if (warp == 1)
        tmem_alloc(smem_u32(&tmem_at), S::kColumns);
    tmem_fence_before();
    __syncthreads();
    if (split > 1)
        cluster_sync_relaxed();  // the barriers of every block are ready
    tmem_fence_after();
    const uint32_t tmem = tmem_at;
    // (each warp waits for the kernel before on its own, before its first wait with a limit)
    const int32_t tiles = (int32_t)((a.p_rows + kP - 1) / kP);
    // this block's steps of 256 elements of K, and its tiles
    const int all_steps = (a.kblocks + 3) >> 2;
    const int kt0 = (all_steps * rank) >> lg, kt1 = (all_steps * (rank + 1)) >> lg;
    const int32_t id0 = (int32_t)blockIdx.x >> lg, stride = (int32_t)gridDim.x >> lg;

    if (warp == 0 || warp == 6) {
        // ---- copies: warp 0 P, warp 6 Q; an issue takes about 100 cycles ----
        const bool of_p = warp == 0;
        const CUtensorMap *map = of_p ? &p_map : &q_map;
        int s = 0;
        uint32_t parity = 0;
        uint32_t fills = 0;
        bool good = true;
        for (int32_t id = id0; good && id < tiles; id += stride) {
            const Tile t = few_tile(a, id);
            const uint8_t *from = of_p ? a.p_sf + (int64_t)t.p_band * a.kblocks * kSfTile : a.q_sf;
            const int32_t row = of_p ? t.p_row : t.q_row;
            if (fills == 0)
                pdl_wait();
            for (int kt = kt0; kt < kt1; ++kt) {
                good = wait_warp<1>(empty + 8 * s, parity ^ 1, dead);
                if (!good)
                    break;
                const int nkb = a.kblocks - 4 * kt < 4 ? a.kblocks - 4 * kt : 4;
                const uint32_t bar = full + 8 * s;
                const uint32_t c = codes + s * S::kCodes + (of_p ? 0 : kP * 128);
                const uint32_t f = sf + s * S::kSf + (of_p ? 0 : 4 * kSfTile);
                if (elect_one()) {
                    if (of_p)  // (Q's bytes may be there before they are expected)
                        mbar_expect_tx(bar, (uint32_t)(S::kCodes + 2 * nkb * kSfTile));
                    tma_load_2d(c, map, kt * 128, row, bar);
                    bulk_load(f, from + (int64_t)kt * 4 * kSfTile, (uint32_t)(nkb * kSfTile), bar);
                }
                __syncwarp();
                ++fills;
                if (++s == S::kStages) {
                    s = 0;
                    parity ^= 1;
                }
            }
        }
        pdl_launch_dependents();
        if (lane == 0)
            fills_made[of_p ? 0 : 1] = fills;
    } else if (warp == 1) {
        // ---- products ----
        constexpr uint32_t idesc = idesc_nvfp4(kP, BN);
        int s = 0;
        uint32_t parity = 0;
        int64_t n = 0;
        bool good = true;
        pdl_wait();  // (the limit of a wait is for this kernel's work, not for the kernel before)
        for (int32_t id = id0; good && id < tiles; id += stride, ++n) {
            const uint32_t acc = (uint32_t)n & 1;
            good = wait_warp<1>(acc_empty + 8 * acc, ((uint32_t)(n >> 1) & 1) ^ 1, dead);
            if (!good)
                break;
            const uint32_t d = tmem + acc * BN;
            for (int kt = kt0; kt < kt1; ++kt) {
                good = wait_warp<1>(full + 8 * s, parity, dead);
                if (!good)
                    break;
                tmem_fence_after();
                const int nkb = a.kblocks - 4 * kt < 4 ? a.kblocks - 4 * kt : 4;
                if (elect_one()) {
                    const uint32_t c = codes + s * S::kCodes, f = sf + s * S::kSf;
                    const uint64_t fd = desc_sf_tile(f);
                    const uint64_t pd = desc_swizzled128(c), qd = desc_swizzled128(c + kP * 128);
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb)
                        if (kb < nkb) {
                            tmem_copy_sf(tmem + S::kSfP + 4 * kb, fd + kb * (kSfTile >> 4));
                            tmem_copy_sf(tmem + S::kSfQ + 4 * kb, fd + (4 + kb) * (kSfTile >> 4));
                        }
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb)
                        if (kb < nkb)
                            mma_nvfp4(d, pd + 2 * kb, qd + 2 * kb, idesc, tmem + S::kSfP + 4 * kb,
                                      tmem + S::kSfQ + 4 * kb, kt > kt0 || kb > 0);
                    mma_commit(empty + 8 * s);
                    if (kt + 1 == kt1)
                        mma_commit(acc_full + 8 * acc);
                }
                __syncwarp();
                if (++s == S::kStages) {
                    s = 0;
                    parity ^= 1;
                }
            }
        }
    } else {
        // ---- output ----
        const int quad = warp & 3;
        const int row = quad * 32 + lane;  // lane of the accumulator
        // byte offset of block r's partial sums of four tokens, the i-th of a block's share: [split][BN / 4 / split][128][4]
        auto sum_at = [&](int r, int i) { return 16 * ((((r * (BN / 4)) >> lg) + i) * kP + row); };
        int64_t n = 0;
        float alpha = 0.0f;
        for (int32_t id = id0; id < tiles; id += stride, ++n) {
            const Tile t = few_tile(a, id);
            if (n == 0) {
                pdl_wait();
                alpha = *a.alpha;
            }
            const uint32_t acc = (uint32_t)n & 1;
            if (!wait_warp<1>(acc_full + 8 * acc, (uint32_t)(n >> 1) & 1, dead))
                break;
            tmem_fence_after();
#pragma unroll 1
            for (int c0 = 0; c0 < BN; c0 += 32) {
                if (c0 >= t.tok_n)
                    break;
                uint32_t v[32];
                tmem_load32(tmem + acc * BN + ((uint32_t)quad << 21) + c0, v);
                tmem_wait_loads();
                // lane = output column, register = token
                if (split > 1) {
                    // four tokens' partial sums to the block that sums them up
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int four = (c0 >> 2) + j;
                        const uint32_t to = four & (split - 1);
                        if (4 * four < t.tok_n)
                            st_async_cluster(map_rank(sums + sum_at(rank, four >> lg), to),
                                             make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]),
                                             map_rank(partial, to));
                    }
                } else if (row < t.wgt_n) {
                    uint16_t *o = a.out + (t.tok0 + c0) * a.ldo + t.wgt0 + row;
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (c0 + i < t.tok_n)
                            o[i * a.ldo] = (uint16_t)pack_bf16x2(__uint_as_float(v[i]) * alpha, 0.0f);
                }
            }
            if (split > 1) {  // the only tile of the cluster
                if (my_fours == 0 || !wait_warp<1, true>(partial, 0, dead))
                    break;
                for (int four = rank; four < fours; four += split) {
                    float f[4] = {0.0f, 0.0f, 0.0f, 0.0f};
                    for (int r = 0; r < split; ++r) {  // in the blocks' order
                        const uint4 w = ld_shared(sums + sum_at(r, four >> lg));
                        f[0] += __uint_as_float(w.x);
                        f[1] += __uint_as_float(w.y);
                        f[2] += __uint_as_float(w.z);
                        f[3] += __uint_as_float(w.w);
                    }
                    // two neighbouring columns in one word: even lanes the first two tokens, odd lanes the others
                    const bool odd = lane & 1;
                    const float p0 = __shfl_xor_sync(0xffffffffu, odd ? f[0] : f[2], 1);
                    const float p1 = __shfl_xor_sync(0xffffffffu, odd ? f[1] : f[3], 1);
                    const int tok = 4 * four + (odd ? 2 : 0);
                    uint16_t *o = a.out + (t.tok0 + tok) * a.ldo + t.wgt0 + (row & ~1);
                    if (row < t.wgt_n && tok < t.tok_n)
                        *reinterpret_cast<uint32_t *>(o) =
                            odd ? pack_bf16x2(p0 * alpha, f[2] * alpha) : pack_bf16x2(f[0] * alpha, p0 * alpha);
                    if (row < t.wgt_n && tok + 1 < t.tok_n)
                        *reinterpret_cast<uint32_t *>(o + a.ldo) =
                            odd ? pack_bf16x2(p1 * alpha, f[3] * alpha) : pack_bf16x2(f[1] * alpha, p1 * alpha);
                }
                break;
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(acc_empty + 8 * acc);
        }
    }
    __syncwarp();
    if (split > 1)
        cluster_arrive_relaxed();
    tmem_fence_before();
    __syncthreads();
    const bool gave_up = *dead != 0;  // some warp of the block
    if (gave_up)  // the copies and products of every warp end before the block's memory goes
        few_drain(warp, full, fills_made[warp == 6], S::kStages, drained);
    if (warp == 1) {
        tmem_fence_after();
        tmem_dealloc(tmem, S::kColumns);
    }
    if (split > 1) {
        cluster_wait();  // no block ends while another may still send it sums
        if (gave_up)     // (it has not seen them arrive)
            wait_last(partial, 0);
    }
}

// ---------------------------------------------------------------------------
// pair form: two blocks on one tile of 256 rows of P by BN of Q
// ---------------------------------------------------------------------------
//
// Each block of a cluster of two holds 128 rows of P and half of Q's in its
// shared memory; the first block's products (cta_group::2) read both and write
// the accumulators of both, so that a block copies half of what a 128 x 256
// tile of its own would need (8192 x 7168 x 7168: 183 us with tiles of 128 x 128
// for each block, 123 so).  The scale factors of Q's rows are in both blocks.
// Both blocks' copies complete on the first block's barrier; its commits free
// the stages and publish the accumulators in both.
//
// A tile is as wide, BN = 128, 192 or 256, as its call's waves of tiles are cheapest.
//
// Two accumulators of 256 columns and 48 columns of scale factors do not fit
// the 512 columns: the accumulators share 64, which the output warps read
// first and then give back, so that the next tile's products run during the
// rest.  The output goes through shared memory, 32 rows of 64 bytes a warp and
// step, and out by TMA.
//
// SPLIT: two pairs of a cluster of four share the K of their one tile, since a
// block's copies alone, 28 KB a step, take 310 cycles of its 360; each gives the
// other half of its sums (256 x 2112 x 7168: 6.4 us, 8.05 in one pair).
//
// Of the 16.7 K cycles that a tile takes at K = 7168 (14.3 K of them products),
// the products wait 1.0 K for the shared columns, 0.4 K for the first stage and
// 180 a stage for the copies.  Tried without gain: a second staging buffer
// (K = 512 4 % faster, K = 7168 1 % slower), 128-byte rows of output (1 % slower),
// Q's scale factors multicast to the pair or both bands of them in one copy (none),
// the next tile found ahead (none; 7 % slower grouped), an expert's weights fetched
// to L2 ahead of the copies (1 to 18 % slower).

constexpr int kPairThreads = 320;

template <int BN, bool SPLIT = false>
struct PairShape {
    static constexpr bool kShared = BN == 256;                   // the accumulators share columns
    static constexpr int kBands = (BN + 127) / 128;
    static constexpr int kCodes = kP * 128 + (BN / 2) * 128;     // bytes per stage and block
    static constexpr int kSf = 4 * kSfTile * (1 + kBands);
    static constexpr int kOut = 8 * 32 * 64;                     // staging: warps x rows x bytes
    static constexpr int kSums = SPLIT ? 8 * 32 * 128 : 0;       // the other pair's sums: warps x rows x bytes
    static constexpr int kFixed = 1024 + kOut + kSums + 4 * 1032;  // and alignment, the experts' first tiles
    static constexpr int kStages = (kSmemLimit - kFixed - 256) / (kCodes + kSf);
    static constexpr int kSmem = kFixed + kStages * (kCodes + kSf);
    static constexpr int kAcc1 = kShared ? BN - 64 : BN;         // column of the second accumulator
    static constexpr int kSfP = kAcc1 + BN;                      // columns of the scale factors
    static constexpr int kSfQ = kSfP + 16;
    static constexpr int kChunks = BN / 32;                      // 32-column pieces of the output
    static_assert(kSfQ + 16 * kBands <= 512, "accumulators and scale factors fit tensor memory");
    static_assert(!SPLIT || BN == 128, "a warp has two pieces of the output and gives one away");
};

// What the blocks of a pair have in flight ends, when one of them gave up: the copies
// of both, which complete in the first, and the products.
__device__ __noinline__ void pair_drain(int warp, uint32_t in_cluster, uint32_t full, uint32_t fills_at, uint32_t stages,
                                        uint32_t drained)
{
    const uint32_t rank = in_cluster & 1, lead = in_cluster & 2;
    if (warp == 0 && rank == 0) {
        const uint32_t mine = ld_cluster32(map_rank(fills_at, lead)), other = ld_cluster32(map_rank(fills_at, lead | 1));
        wait_fills(full, mine > other ? mine : other, stages);
    } else if (warp == 1) {
        if (rank == 0 && elect_one())
            pair_commit(drained, 3u << lead);
        __syncwarp();
        wait_last(drained, 0);
    }
    __syncwarp();
}

template <int BN, bool GROUPED, bool SPLIT>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(SPLIT ? 4 : 2, 1, 1)
    nvfp4_pair_kernel(const __grid_constant__ CUtensorMap p_map, const __grid_constant__ CUtensorMap q_map,
                      const __grid_constant__ CUtensorMap psf_map, const __grid_constant__ CUtensorMap qsf_map,
                      const __grid_constant__ CUtensorMap out_map, const __grid_constant__ KernelArgs a)
{
    using S = PairShape<BN, SPLIT>;
    constexpr int kPeers = SPLIT ? 4 : 2;
    extern __shared__ uint8_t raw[];
    __shared__ uint64_t bars[2 * S::kStages + 6];
    __shared__ uint32_t tmem_at;
    __shared__ uint32_t fills_made;
    __shared__ int dead_flag;
    const uint32_t pad = (1024 - (smem_u32(raw) & 1023)) & 1023;
    const uint32_t codes = smem_u32(raw) + pad;
    const uint32_t stage_out = codes + S::kStages * S::kCodes;
    const uint32_t sf = stage_out + S::kOut;
    const uint32_t sums = sf + S::kStages * S::kSf;
    int32_t *first = reinterpret_cast<int32_t *>(raw + pad + S::kStages * (S::kCodes + S::kSf) + S::kOut + S::kSums);
    volatile int *dead = &dead_flag;

    const int warp = __shfl_sync(0xffffffffu, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t in_cluster = cluster_rank(), rank = in_cluster & 1, lead = in_cluster & 2;
    const uint32_t both = 3u << lead;  // the pair's blocks
    const uint32_t full = smem_u32(bars), empty = full + 8 * S::kStages;
    const uint32_t acc_full = empty + 8 * S::kStages, acc_free = acc_full + 16, drained = acc_free + 16,
                   partial = drained + 8;

    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full + 8 * s, 1);
            mbar_init(empty + 8 * s, 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(acc_full + 8 * i, 1);
            mbar_init(acc_free + 8 * i, 16);  // the output warps of both blocks
        }
        mbar_init(drained, 1);
        mbar_init(partial, 1);
        mbar_fence_init();
        if (SPLIT)
            mbar_expect_tx(partial, S::kSums);
        dead_flag = 0;
#ifdef TSFN_RUN_OUT
        block_start() = clock64();
#endif
        tma_prefetch_map(&p_map);
        tma_prefetch_map(&q_map);
        tma_prefetch_map(&psf_map);
        tma_prefetch_map(&qsf_map);
        tma_prefetch_map(&out_map);
    }
    if (warp == 1)
        pair_tmem_alloc(smem_u32(&tmem_at), 512);
    tmem_fence_before();
    __syncthreads();
    cluster_sync_relaxed();
    tmem_fence_after();
    const uint32_t tmem = tmem_at;
    int64_t tiles;
    if constexpr (GROUPED) {
        pdl_wait();
        tiles = grouped_tiles<BN>(a, first);
    } else {  // (each warp waits on its own, before its first wait with a limit)
        tiles = ((a.p_rows + 2 * kP - 1) / (2 * kP)) * ((a.q_rows + BN - 1) / BN);
    }
    auto tile_of = [&](int64_t id) { return pair_tile<BN, GROUPED>(a, first, id); };
    // columns of the products of a tile: all, or the expert's tokens rounded up
    auto columns = [](const Tile &t) { return GROUPED ? (t.tok_n + 31) & ~31 : BN; };
    // this pair's steps of 256 elements of K, and its tiles
    const int all_steps = (a.kblocks + 3) >> 2;
    const int kt0 = SPLIT && lead ? all_steps >> 1 : 0, kt1 = SPLIT && !lead ? all_steps >> 1 : all_steps;
    const int64_t id0 = blockIdx.x >> (SPLIT ? 2 : 1), stride = gridDim.x >> (SPLIT ? 2 : 1);

    if (warp == 0) {
        // ---- copies ----
        int s = 0;
        uint32_t parity = 0;
        uint32_t fills = 0;
        bool good = true;
        const uint32_t full0 = map_rank(full, lead);
        for (int64_t id = id0; good && id < tiles; id += stride) {
            const Tile t = tile_of(id);
            const int32_t p_row = t.p_row + (int32_t)rank * kP, q_row = t.q_row + (int32_t)rank * (columns(t) / 2);
            const int q_bands = GROUPED ? t.q_bands : S::kBands;
            const int32_t p_band = t.p_band + (int32_t)rank, q_band = t.q_band;
            if (!GROUPED && fills == 0)
                pdl_wait();
            for (int kt = kt0; kt < kt1; ++kt) {
                good = wait_warp<kPeers>(empty + 8 * s, parity ^ 1, dead);
                if (!good)
                    break;
                const uint32_t bar = full0 + 8 * s;
                const uint32_t c = codes + s * S::kCodes, f = sf + s * S::kSf;
                if (elect_one()) {
                    if (rank == 0)
                        mbar_expect_tx(full + 8 * s, 2u * (uint32_t)(S::kCodes + 4 * kSfTile * (1 + q_bands)));
                    pair_load_2d(c, &p_map, kt * 128, p_row, bar);
                    pair_load_2d(c + kP * 128, &q_map, kt * 128, q_row, bar);
                    pair_load_2d(f, &psf_map, kt * 256, p_band, bar);
#pragma unroll
                    for (int b = 0; b < S::kBands; ++b)
                        if (b < q_bands)
                            pair_load_2d(f + 4 * (1 + b) * kSfTile, &qsf_map, kt * 256, q_band + b, bar);
                }
                __syncwarp();
                ++fills;
                if (++s == S::kStages) {
                    s = 0;
                    parity ^= 1;
                }
            }
        }
        pdl_launch_dependents();
        if (lane == 0)
            fills_made = fills;
    } else if (warp == 1) {
        // ---- products, by the first block for both ----
        int s = 0;
        uint32_t parity = 0;
        int64_t n = 0;
        bool good = true;
        if (!GROUPED)
            pdl_wait();  // (the limit of a wait is for this kernel's work, not for the kernel before)
        for (int64_t id = id0; rank == 0 && good && id < tiles; id += stride, ++n) {
            const uint32_t idesc = idesc_nvfp4(2 * kP, (uint32_t)(GROUPED ? columns(tile_of(id)) : BN));
            // the tile before has given the shared columns back, or the one before
            // that its accumulator (without one: at once)
            good = S::kShared ? wait_warp<kPeers>(acc_free, ((uint32_t)n & 1) ^ 1, dead)
                              : wait_warp<kPeers>(acc_free + 8 * ((uint32_t)n & 1), ((uint32_t)(n >> 1) & 1) ^ 1, dead);
            if (!good)
                break;
            const uint32_t d = tmem + ((uint32_t)n & 1) * S::kAcc1;
            // (tiles of 192 rows of Q begin in the middle of every other band)
            const uint32_t sf_q = tmem + S::kSfQ + (BN == 192 ? (uint32_t)(tile_of(id).q_row & 127) >> 5 : 0);
            for (int kt = kt0; kt < kt1; ++kt) {
                good = wait_warp<kPeers>(full + 8 * s, parity, dead);
                if (!good)
                    break;
                tmem_fence_after();
                const int nkb = a.kblocks - 4 * kt < 4 ? a.kblocks - 4 * kt : 4;
                if (elect_one()) {
                    const uint32_t c = codes + s * S::kCodes;
                    const uint64_t fd = desc_sf_tile(sf + s * S::kSf);
                    const uint64_t pd = desc_swizzled128(c), qd = desc_swizzled128(c + kP * 128);
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb)
                        if (kb < nkb) {
                            pair_copy_sf(tmem + S::kSfP + 4 * kb, fd + kb * (kSfTile >> 4));
#pragma unroll
                            for (int b = 0; b < S::kBands; ++b)
                                pair_copy_sf(tmem + S::kSfQ + 4 * (S::kBands * kb + b),
                                             fd + (4 * (1 + b) + kb) * (kSfTile >> 4));
                        }
#pragma unroll
                    for (int kb = 0; kb < 4; ++kb)
                        if (kb < nkb)
                            pair_mma_nvfp4(d, pd + 2 * kb, qd + 2 * kb, idesc, tmem + S::kSfP + 4 * kb,
                                           sf_q + 4 * S::kBands * kb, kt > kt0 || kb > 0);
                    pair_commit(empty + 8 * s, both);
                    if (kt + 1 == kt1)
                        pair_commit(acc_full + 8 * ((uint32_t)n & 1), both);
                }
                __syncwarp();
                if (++s == S::kStages) {
                    s = 0;
                    parity ^= 1;
                }
            }
        }
    } else {
        // ---- output: two warps for each 32 lanes, every other 32 columns ----
        const int quad = warp & 3, half = (warp - 2) >> 2;
        const uint32_t stage = stage_out + (warp - 2) * (32 * 64);
        const uint32_t free0 = map_rank(acc_free, lead);
        int64_t n = 0;
        float alpha = 0.0f;
        for (int64_t id = id0; id < tiles; id += stride, ++n) {
            const Tile t = tile_of(id);
            if (!GROUPED && n == 0) {
                pdl_wait();
                alpha = *a.alpha;
            }
            if (GROUPED)
                alpha = a.alpha[t.expert];
            const uint32_t acc = (uint32_t)n & 1;
            if (!wait_warp<kPeers>(acc_full + 8 * acc, (uint32_t)(n >> 1) & 1, dead))
                break;
            tmem_fence_after();
            const int row0 = (int)rank * kP + quad * 32;  // of the warp's lanes in the tile
            const int lanes = (GROUPED ? t.wgt_n : t.tok_n) - row0, cols = GROUPED ? t.tok_n : t.wgt_n;
            const uint32_t src = tmem + acc * S::kAcc1 + ((uint32_t)quad << 21);
            // 32-column pieces, this warp's first one among the shared: the last two of
            // the first accumulator, the first two of the second
            const int first_piece = half + (S::kShared && acc == 0 ? S::kChunks - 2 : 0);
            auto column = [&](int i) { return (S::kShared ? (2 * i + first_piece) & (S::kChunks - 1) : 2 * i + first_piece) * 32; };
            uint32_t v[2][32];
            tmem_load32(src + column(0), v[0]);
            if (SPLIT)
                tmem_load32(src + column(1), v[1]);
            tmem_wait_loads();
            if (SPLIT) {
                // (the cluster's only tile) each pair gives one of a warp's two pieces to
                // the other and adds the other's sums to the one it keeps
                const uint32_t to = in_cluster ^ 2, at = sums + ((warp - 2) * 256 + lane) * 16;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    uint4 w;
                    w.x = lead ? v[0][4 * j] : v[1][4 * j];
                    w.y = lead ? v[0][4 * j + 1] : v[1][4 * j + 1];
                    w.z = lead ? v[0][4 * j + 2] : v[1][4 * j + 2];
                    w.w = lead ? v[0][4 * j + 3] : v[1][4 * j + 3];
                    st_async_cluster(map_rank(at + j * 512, to), w, map_rank(partial, to));
                }
                if (!wait_warp<kPeers, true>(partial, 0, dead))
                    break;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint4 w = ld_shared(at + j * 512);
                    const uint32_t got[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t kept = lead ? v[1][4 * j + e] : v[0][4 * j + e];
                        v[0][4 * j + e] = __float_as_uint(__uint_as_float(kept) + __uint_as_float(got[e]));
                    }
                }
            }
            if (S::kShared) {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster_relaxed(free0);
            }
#pragma unroll
            for (int i = 0; i < (SPLIT ? 1 : S::kChunks / 2); ++i) {
                const int c0 = column(SPLIT ? (int)(lead >> 1) : i);
                if (!SPLIT && i + 1 < S::kChunks / 2)
                    tmem_load32(src + column(i + 1), v[(i + 1) & 1]);
                if (lanes > 0 && c0 < cols) {
                    if (lane == 0)
                        bulk_wait_read<0>();
                    __syncwarp();
                    // 32 rows of 64 bytes under the 64-byte swizzle: 16-byte piece j of
                    // row r lies at j ^ (r / 2 % 4)
                    const int rows = GROUPED ? cols - c0 : lanes;  // that are the call's (the expert's)
                    if constexpr (GROUPED) {
                        // lane = output column, register = row: neighbouring lanes exchange, an
                        // even lane takes both columns of the first of two rows, an odd one of the second
                        const bool odd = lane & 1;
                        const int at = lane >> 1;
#pragma unroll
                        for (int r = 0; r < 32; r += 2) {
                            const uint32_t mine = v[i & 1][r], other = v[i & 1][r + 1];
                            const float got = __uint_as_float(__shfl_xor_sync(0xffffffffu, odd ? mine : other, 1)) * alpha;
                            const float kept = __uint_as_float(odd ? other : mine) * alpha;
                            st_shared32(stage + (r + odd) * 64 + (((at >> 2) ^ ((r >> 1) & 3)) << 4) + (at & 3) * 4,
                                        odd ? pack_bf16x2(got, kept) : pack_bf16x2(kept, got));
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            float f[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                f[e] = __uint_as_float(v[i & 1][8 * j + e]) * alpha;
                            st_shared(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4), pack8(f));
                        }
                    }
                    const int64_t row = t.tok0 + (GROUPED ? c0 : row0), col = t.wgt0 + (GROUPED ? row0 : c0);
                    if (!GROUPED || rows >= 32) {
                        fence_async_proxy();
                        __syncwarp();
                        if (lane == 0) {
                            tma_store_2d(&out_map, stage, (int32_t)col, (int32_t)row);
                            bulk_commit();
                        }
                    } else {
                        // rows of the next expert follow: 4 lanes per row, 16 bytes each
                        __syncwarp();
#pragma unroll
                        for (int r0 = 0; r0 < 32; r0 += 8) {
                            const int r = r0 + (lane >> 2), j = lane & 3;
                            const uint4 w = ld_shared(stage + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
                            if (r < rows && 8 * j < lanes)
                                *reinterpret_cast<uint4 *>(a.out + (row + r) * a.ldo + col + 8 * j) = w;
                        }
                    }
                }
                tmem_wait_loads();
            }
            if (!S::kShared) {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive_cluster_relaxed(free0 + 8 * acc);
            }
        }
        if (lane == 0)
            bulk_wait_read<0>();
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();  // no block ends while another's products, arrivals or sums may reach it
    if (*dead) {  // in every block of the cluster: what is in flight ends before any block's memory goes
        pair_drain(warp, in_cluster, full, smem_u32(&fills_made), S::kStages, drained);
        if (SPLIT)
            wait_last(partial, 0);
        __syncwarp();
        cluster_sync();
    }
    if (warp == 1) {
        tmem_fence_after();
        pair_tmem_dealloc(tmem, 512);
    }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                              const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                              CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's tensor-map encoder, found once.
EncodeFn encode_fn()
{
    static const EncodeFn fn = [] {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult found;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &found) !=
                cudaSuccess ||
            found != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<EncodeFn>(p);
    }();
    return fn;
}

// Codes [rows, K/2] in boxes of 128 bytes by `box_rows` rows, 128-byte swizzle,
// zeros outside.
bool codes_map(CUtensorMap *map, const uint8_t *codes, int64_t rows, int64_t K, int box_rows)
{
    const EncodeFn fn = encode_fn();
    if (fn == nullptr)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(K / 2), (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(K / 2)};
    const cuuint32_t box[2] = {128, (cuuint32_t)box_rows}, step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale factors in the 128x4 layout as [bands, kblocks * 512] bytes in boxes of
// four tiles (2048 bytes, as 256 words of 8), zeros outside.
bool sf_map(CUtensorMap *map, const uint8_t *sf, int64_t bands, int64_t kblocks)
{
    const EncodeFn fn = encode_fn();
    if (fn == nullptr)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)(kblocks * kSfTile / 8), (cuuint64_t)bands};
    const cuuint64_t strides[1] = {(cuuint64_t)(kblocks * kSfTile)};
    const cuuint32_t box[2] = {4 * kSfTile / 8, 1}, step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT64, 2, const_cast<uint8_t *>(sf), dims, strides, box, step,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The output [rows, N] in boxes of 32 rows by 32 columns, 64-byte swizzle.
bool out_tile_map(CUtensorMap *map, uint16_t *out, int64_t rows, int64_t N, int64_t ldo)
{
    const EncodeFn fn = encode_fn();
    if (fn == nullptr)
        return false;
    const cuuint64_t dims[2] = {(cuuint64_t)N, (cuuint64_t)rows};
    const cuuint64_t strides[1] = {(cuuint64_t)(ldo * 2)};
    const cuuint32_t box[2] = {32, 32}, step[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, out, dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

KernelArgs kernel_args(const GemmArgs &g, bool swap)
{
    KernelArgs a{};
    a.p_sf = swap ? g.wgt_sf : g.tok_sf;
    a.q_sf = swap ? g.tok_sf : g.wgt_sf;
    a.alpha = g.alpha;
    a.out = g.out;
    a.ldo = g.ldo;
    a.p_rows = swap ? g.N : g.tok_rows;
    a.q_rows = swap ? g.tok_rows : g.N;
    a.kblocks = (int)((g.K + 63) / 64);
    a.wgt_rows = (int)g.N;
    a.wgt_bands = (int)((g.N + 127) / 128);
    a.tok_rows = g.tok_rows;
    a.start = g.start;
    a.count = g.count;
    a.experts = g.experts;
    return a;
}

// Opt in to `bytes` of shared memory, once per kernel and device.
template <typename Kernel>
cudaError_t grow_smem(Kernel kernel, int bytes, std::atomic<bool> (&grown)[kMaxCachedDevices], int dev)
{
    if (dev < kMaxCachedDevices && grown[dev].load(std::memory_order_relaxed))
        return cudaSuccess;
    const cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess && dev < kMaxCachedDevices)
        grown[dev].store(true, std::memory_order_relaxed);
    return err;
}

// Blocks (as a power of two) that share the K of a tile of few tokens: 4 or 2
// where all tiles still run at once (of clusters of 4 a GB300 runs 36 at a time
// on its 152 SMs, of 8 only 15) and K is long enough to pay for the exchange,
// which takes about 0.5 us for a group of 4 tokens and grows with the groups.
// us alone, over 2, over 4:
//   M=1   N=4096 K=1024 2.8 2.7 2.9, K=4096 5.6 3.9 3.8;  N=7168 K=1024 2.8 3.0, K=2048 3.8 3.7
//   M=32  N=4096 K=1024 2.9 3.4 3.5, K=2048 3.9 4.0 3.7, K=4096 5.8 4.9 4.3;  N=7168 K=2048 3.9 4.4
//   M=64  N=2112 K=2048 5.0 5.2 4.0;  N=4096 K=4096 7.0 6.2 5.2
int split_log2_of(int64_t tiles, int steps, int64_t tokens, int sms)
{
    const bool one_group = tokens <= 4;
    if (4 * tiles <= sms - sms / 16 && steps >= (one_group ? 4 : 8))
        return 2;
    return 2 * tiles <= sms && steps >= (one_group ? 8 : 12) ? 1 : 0;
}

template <int BN>
cudaError_t launch_few(const GemmArgs &g, bool pdl, cudaStream_t stream)
{
    using S = Shape<BN>;
    static std::atomic<bool> grown[kMaxCachedDevices];
    int dev = 0;
    const int sms = current_device_sms(&dev);
    if (sms <= 0)
        return cudaErrorInvalidDevice;
    const cudaError_t err = grow_smem(nvfp4_few_kernel<BN>, S::kSmem, grown, dev);
    if (err != cudaSuccess)
        return err;
    CUtensorMap p_map, q_map;
    if (!codes_map(&p_map, g.wgt, g.N, g.K, kP) || !codes_map(&q_map, g.tok, g.tok_rows, g.K, BN))
        return cudaErrorInvalidValue;
    KernelArgs a = kernel_args(g, true);
    const int64_t tiles = (g.N + kP - 1) / kP, grid = tiles < sms ? tiles : sms;
    a.split_log2 = split_log2_of(tiles, (a.kblocks + 3) / 4, g.tok_rows, sms);
    return launch_clusters(nvfp4_few_kernel<BN>, dim3((unsigned)(grid << a.split_log2)), dim3(kThreads),
                           (size_t)S::kSmem, stream, pdl, 1u << a.split_log2, p_map, q_map, a);
}

template <int BN, bool GROUPED, bool SPLIT = false>
cudaError_t launch_pairs(const GemmArgs &g, bool pdl, cudaStream_t stream)
{
    static std::atomic<bool> grown[kMaxCachedDevices];
    int dev = 0;
    const int sms = current_device_sms(&dev);
    if (sms < 2)
        return cudaErrorInvalidDevice;
    const cudaError_t err = grow_smem(nvfp4_pair_kernel<BN, GROUPED, SPLIT>, PairShape<BN, SPLIT>::kSmem, grown, dev);
    if (err != cudaSuccess)
        return err;
    const KernelArgs a = kernel_args(g, GROUPED);
    const int64_t experts = GROUPED ? g.experts : 1;
    CUtensorMap tok_map, wgt_map, tok_sf_map, wgt_sf_map, out_map;
    if (!codes_map(&tok_map, g.tok, g.tok_rows, g.K, GROUPED ? BN / 2 : kP) ||
        !codes_map(&wgt_map, g.wgt, experts * g.N, g.K, GROUPED ? kP : BN / 2) ||
        !sf_map(&tok_sf_map, g.tok_sf, (g.tok_rows + 127) / 128, a.kblocks) ||
        !sf_map(&wgt_sf_map, g.wgt_sf, experts * a.wgt_bands, a.kblocks) ||
        !out_tile_map(&out_map, g.out, g.tok_rows, g.N, g.ldo))
        return cudaErrorInvalidValue;
    int64_t pairs = sms / 2;
    if (!GROUPED) {
        const int64_t tiles = ((a.p_rows + 2 * kP - 1) / (2 * kP)) * ((a.q_rows + BN - 1) / BN);
        pairs = tiles < pairs ? tiles : pairs;
    }
    return launch_kernel(nvfp4_pair_kernel<BN, GROUPED, SPLIT>, dim3((unsigned)((SPLIT ? 4 : 2) * pairs)), dim3(kPairThreads),
                         (size_t)PairShape<BN, SPLIT>::kSmem, stream, pdl, GROUPED ? wgt_map : tok_map, GROUPED ? tok_map : wgt_map,
                         GROUPED ? wgt_sf_map : tok_sf_map, GROUPED ? tok_sf_map : wgt_sf_map, out_map, a);
}

}  // namespace

cudaError_t launch_nvfp4_gemm(const GemmArgs &g, bool pdl, cudaStream_t stream)
{
    if (g.experts > 0) {
        // Tiles of 128 or 256 tokens, by an expert's share of the entries.  64 experts of
        // 4096 x 7168, us with tiles of 128 and of 256: 2 tokens an expert 126 and 132, 32
        // 162 and 172, 64 171 and 175, 96 182 and 182, 128 194 and 191, 256 280 and 231.
        // (Tiles of 64 tokens of one block each: 128 with 2 tokens, 210 with 64.)
        if (g.entries <= 96 * (int64_t)g.experts)
            return launch_pairs<128, true>(g, pdl, stream);
        return launch_pairs<256, true>(g, pdl, stream);
    }
    if (g.tok_rows <= 32)
        return launch_few<32>(g, pdl, stream);
    if (g.tok_rows <= 64)
        return launch_few<64>(g, pdl, stream);
    const int sms = current_device_sms();
    const int steps = (int)((g.K + 255) / 256);
    const int64_t np = (g.tok_rows + 2 * kP - 1) / (2 * kP), pairs = sms > 1 ? sms / 2 : 1;
    const int64_t t128 = np * ((g.N + 127) / 128);
    const bool two_calls = 8 * t128 <= sms;  // over two pairs each, the next call's blocks fit beside this one's
    // up to 128 tokens still as one tile's columns where few tiles walk a long K (us so and
    // in pairs: M=65 N=2112 K=2048 5.7 4.4, K=7168 5.5 6.2, M=104 6.4 6.3, M=128 6.9 6.4;
    // N=4096 K=7168 M=128 7.3 7.3; M=128 N=2112 K=16384 9.4 9.8)
    if (g.tok_rows <= (two_calls && steps < 40 ? 96 : 128) && steps >= 20 &&
        split_log2_of((g.N + kP - 1) / kP, steps, g.tok_rows, sms) == 2)
        return launch_few<128>(g, pdl, stream);
    // a tile's K over two pairs where it is long enough to pay for the exchange, of
    // which the next call hides a part (us in one pair and over two: 17 tiles, M=256
    // N=2112, K=2048 4.4 4.5, K=4096 5.8 5.25, K=7168 8.05 6.4; 32 tiles, N=4096, K=4096
    // 5.8 6.05, K=7168 8.1 7.2)
    if (4 * t128 <= sms - sms / 16 && steps >= (two_calls ? 12 : 20))
        return launch_pairs<128, false, true>(g, pdl, stream);
    // the width whose waves of pairs take least: a wave with tiles of 128 rows of weights
    // 0.65 and of 192 0.83 of the time with 256 (K=7168: 5.7, 7.3 and 8.8 us).  us with 128,
    // 192, 256: N=7168 K=7168 M=512 14.1 10.8 12.1, M=1024 20.3 17.7 20.3, M=2048 36.9 32.0
    // 29.6; N=5120 K=5120 M=768 11.6 13.2 9.8, M=1024 15.4 13.1 15.9; N=2112 K=7168 M=1024
    // 9.0 10.4 11.1
    auto waves = [&](int64_t width) { return (np * ((g.N + width - 1) / width) + pairs - 1) / pairs; };
    const int64_t c128 = 65 * waves(128), c192 = 83 * waves(192), c256 = 100 * waves(256);
    if (c128 < c192 && c128 < c256)
        return launch_pairs<128, false>(g, pdl, stream);
    if (c192 < c256)
        return launch_pairs<192, false>(g, pdl, stream);
    return launch_pairs<256, false>(g, pdl, stream);
}

cudaError_t read_stalled_waits(uint32_t *count)
{
    const cudaError_t err = cudaDeviceSynchronize();
    if (err != cudaSuccess)
        return err;
    return cudaMemcpyFromSymbol(count, g_stalled_waits, sizeof(*count));
}

}  // namespace tsfn
