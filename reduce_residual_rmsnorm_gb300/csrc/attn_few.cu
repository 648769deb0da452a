// Attention of few rows at a time over the paged NVFP4 cache: decoded tokens, and a
// few queries of a sequence.
//
//   out = sum_j p_j V[j] / sum_j p_j,   p_j = exp2(c q.K[j] - m)      c = scale log2(e) / k_scale
//
// Bound by the cache's bytes, 9/8 D a key and head.  The rows of a unit are up to 8 NT
// (NT 1, 2 or 4) of the (query, head) pairs that share a key head, so a key is read once
// for them.  E2M1 times E4M3 has at most 6 significant bits: K and V are exact in fp16, and
// a row of q is too after scaling by a power of two, so fp16 products with fp32 sums
// lose nothing; p is rounded to fp16, by an eighth of the output's own rounding to bf16 for
// weights above 2^-21 of the row's largest, by 2^-32 of that for smaller ones.  The keys are
// the 16 rows of mma.m16n8k16 (the rows of q its 8 columns):
//   S^T = K q^T     a lane's part of a row of K is 16 contiguous bytes of codes: which
//                   d a product's k stands for is free as long as q follows
//   O^T = V^T p^T   a lane holds D/8 contiguous d of 4 keys; two keys' nibbles are
//                   joined in one byte before the conversion, which then gives pairs
//                   along the keys, as the product wants them; p^T by movmatrix
// (mma.sync, not tcgen05: that takes its operands from shared or tensor memory, where K and V
// would have to be written as fp16 first, four times the bytes of their codes; mma.sync takes
// them from the registers in which they are made.  The tensor pipe is a quarter busy.)
//
// A warp takes a run of tiles of 16 keys, with copies of the next ones under way, and has
// a running maximum and sum of its own.  The maximum follows only when a score passes it
// by 2^8, so most tiles take one vote instead of a reduction and a rescaling.
//
// Work is split in one of two ways:
//   - units that are all resident at once: a cluster of up to 8 blocks for each, whose parts
//     are joined through the cluster's shared memory: one launch and no workspace;
//   - evenly: all units' tiles in one row, cut into equal shares, so that sequences of
//     any lengths keep every block busy.  A unit inside a share is written at once; of a
//     unit over several, each block leaves its part in the workspace and
//     attn_join_kernel joins them in order.
// 64 sequences of 0 to 16384 keys, 64 heads over 8 of 128: 98 us, 4.4 TB/s.  The tiles run at
// the memory's rate (435 MB in 64 us; 340 instructions a tile and warp, nine tenths of what
// four blocks can issue); beside them 8 us pass until the first tiles are there, 10 to 20
// between most blocks' end and the last one's, 5 for the join.  One sequence of 131072
// keys and 8 heads over one: 16 us; of 1024 keys 4.9, a chain of latencies.
#include "async_copy.cuh"
#include "attn_util.cuh"
#include "device_util.cuh"
#include "launch_attention.h"
#include "launch_nvfp4.h"
#include "tcgen05.cuh"

namespace tsfn {

namespace {

// Even shares: for 8 rows blocks of 4 warps, four to an SM (64 sequences up to 16384 keys:
// 107.7 us; blocks of 8 warps 113.7, five blocks of 4 with 96 registers 111.7, all three
// measured with a way of 12 tiles, see below); for more rows the registers of an SM go to one block of 8.
// Clusters: blocks of 8 warps, for the time of a single call.
constexpr int kSms = 152;
constexpr int kClusterWarps = 8;
constexpr int share_warps(int nt) { return nt == 1 ? 4 : 8; }
constexpr int blocks_per_sm(int nt) { return nt == 1 ? 4 : 1; }
constexpr int blocks_of(int nt) { return kSms * blocks_per_sm(nt); }
// Rows of a unit, in eights: 17 and more go 32 at a time, so that a key is turned into
// fp16 once for them.
int eights_of(int64_t rows) { return rows <= 8 ? 1 : (rows <= 16 ? 2 : 4); }
constexpr int kStages = 4;  // tiles of a warp whose copies are under way
constexpr int kShare = 8;     // tiles of a share, at least
// What going to a unit costs, in tiles of a block, when work is split (more makes short units
// longer, so that blocks with many of them do not end last).  us, 8 key heads of 128, by way:
//                               12     16     20     24     32
//   8 rows, 64 of 0-16384 keys  131.3  126.8  127.0  127.4  129.4
//           300 of 0-4096       169.7  164.1  160.3  161.1  164.0
//  16 rows, 64 of 0-16384       229.9  226.0  222.2  216.1  210.7
//  32 rows, 64 of 0-16384       328.7  324.1  314.7  308.6  301.6
//           300 of 0-4096       487.0  472.8  464.7  457.9  440.0
// Sequences of equal lengths do not depend on it (64 of 8192: 130 us, with 32 rows 280).  For
// 16 and more rows the best lies beyond 24.
constexpr int way_of(int nt) { return nt == 1 ? 20 : 24; }
// Clusters take calls whose units are all resident at once, with at most this many keys a
// block (16 tiles a warp: with more, sequences of different lengths leave SMs idle), or half
// as many where the clusters leave most of the SMs idle.  Clusters against even shares, us,
// 8 rows, D = 128:
//   1 unit        1024 keys 4.9 / 9.0    8192 keys 9.4 / 9.4     16384 keys 15.0 / 10.5
//   8 units       1024 keys 5.3 / 11.5   16384 keys 15.3 / 16.0  32768 keys 26.0 / 19.5
//   128 units     lengths up to 1024 8.8 / 14.8, to 4096 18.5 / 19.2, to 8192 31.1 / 24.0
constexpr int64_t kClusterKeys = 2048;
constexpr int kMostBlocks = 8;  // of a cluster
// Blocks of a cluster, a power of two; 0: even shares.
int cluster_of(int64_t B, int64_t heads, int64_t rows, int64_t keys, int64_t window)
{
    const int nt = eights_of(rows);
    const int64_t units = B * heads * ((rows + 8 * nt - 1) / (8 * nt)), resident = kSms * (nt == 1 ? 2 : 1);
    if (window > 0 && window + rows < keys)
        keys = window + rows;  // (no more queries than rows)
    for (int blocks = kMostBlocks; blocks >= 1; blocks /= 2)
        if (units * blocks <= resident)
            return keys <= (units * blocks < resident / 8 ? kClusterKeys / 2 : kClusterKeys) * blocks ? blocks : 0;
    return 0;
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum.
__device__ __forceinline__ void mma_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
                 : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}

// Four bytes of codes of two keys, the d of each nibble alike, times the keys' scales:
// fp16 pairs (key 0, key 1) of the even d (e) and of the odd ones (o).
__device__ __forceinline__ void join_keys(uint32_t w0, uint32_t w1, uint32_t scale, uint32_t (&e)[4], uint32_t (&o)[4])
{
    const uint32_t even = (w0 & 0x0F0F0F0Fu) | ((w1 << 4) & 0xF0F0F0F0u);
    const uint32_t odd = ((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u);
    e[0] = mul_f16x2(e2m1x2<0>(even), scale);
    e[1] = mul_f16x2(e2m1x2<1>(even), scale);
    e[2] = mul_f16x2(e2m1x2<2>(even), scale);
    e[3] = mul_f16x2(e2m1x2<3>(even), scale);
    o[0] = mul_f16x2(e2m1x2<0>(odd), scale);
    o[1] = mul_f16x2(e2m1x2<1>(odd), scale);
    o[2] = mul_f16x2(e2m1x2<2>(odd), scale);
    o[3] = mul_f16x2(e2m1x2<3>(odd), scale);
}

// A unit's run of tiles for one block.
struct Run {
    int b, head, rows, first, count;  // first tile (of 16 keys) of the sequence, and how many
    int row0;                         // first of the sequence's (query, head) pairs
    Seq s;
};

template <int D, int NT, int WARPS>
struct Shared {
    using L = Layout<D>;
    static constexpr int NR = 8 * NT;
    static constexpr int kRing = WARPS * (kStages * L::kTile > NR * D * 4 ? kStages * L::kTile : NR * D * 4);
    // the copies, [warps][stages][tile]; after them the warps' O [warps][NR][D]
    static constexpr int kMs = kRing, kLs = kMs + WARPS * NR * 4;  // the warps' maxima and sums
    static constexpr int kQ = kLs + WARPS * NR * 4;                // q's fragments of the products
    static constexpr int kFactor = kQ + NR * D * 2, kHi = kFactor + NR * 4, kLo = kHi + NR * 4;  // of each row
    static constexpr int kLimits = kLo + NR * 4, kBytes = kLimits + NT * 16;  // of each 8 rows
    // where 4 elements of a row of O are, in fours: lanes that write together have
    // different rows and d, and no bank in common
    static __device__ __forceinline__ int place(int row, int four)
    {
        const int r = (row >> 1) & 3;
        return row * (D / 4) + (four ^ (D == 128 ? r : (r & 1) | (r & 2) << 1));
    }
};

// The parts (m, l, O) of a run's rows by the block's warps, in shared memory.
template <int D, int NT, int WARPS>
__device__ __forceinline__ void attend(const AttnArgs &a, const Run &run, float k_scale, uint8_t *smem)
{
    using L = Layout<D>;
    using Sh = Shared<D, NT, WARPS>;
    constexpr int NR = 8 * NT;
    constexpr int KS = D / 16;  // products of S per tile and 8 rows, and of O
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const Seq &s = run.s;
    uint8_t *const ring = smem;
    const uint32_t my_ring = smem_addr(ring) + warp * kStages * L::kTile;

    // this warp's tiles and their copies: 18 D contiguous bytes each
    const int begin = (int)((int64_t)run.count * warp / WARPS), mine = (int)((int64_t)run.count * (warp + 1) / WARPS) - begin;
    const int key0 = (run.first + begin) * 16, tiles_of_page = a.cache.page_size >> 4;
    const int32_t *const table = a.table + (int64_t)run.b * a.max_pages;
    const int pages = (int)((s.len + a.cache.page_size - 1) / a.cache.page_size);  // that hold keys
    int page_at = (int)div_by((uint32_t)key0, a.cache.div_page);
    int in_page = (key0 - page_at * a.cache.page_size) >> 4;
    auto page_of = [&](int i) -> int32_t { return mine > 0 && i < pages ? table[i] : -1; };
    int32_t next_page = page_of(page_at);
    const uint8_t *src = nullptr;
    auto to_page = [&]() {
        const int32_t page = next_page;
        next_page = page_of(++page_at);
        src = nullptr;
        if (page >= 0 && page < a.cache.num_pages)
            src = a.cache.pages + (((int64_t)page * a.cache.heads + run.head) * tiles_of_page + in_page) * L::kTile + lane * 16;
    };
    to_page();
    uint32_t in_cache = 0;  // bit i: of the copy i before the last one
    uint32_t fill = my_ring + lane * 16;
    const uint32_t ring_end = fill + kStages * L::kTile;
    auto issue = [&](bool more) {
        in_cache <<= 1;
        if (more) {
            if (in_page == tiles_of_page) {
                in_page = 0;
                to_page();
            }
            if (src != nullptr) {
                in_cache |= 1;
#pragma unroll
                for (int i = 0; i < L::kChunks / 32; ++i)
                    copy16(fill + i * 512, src + i * 512);
                if (lane < L::kChunks % 32)
                    copy16(fill + L::kChunks / 32 * 512, src + L::kChunks / 32 * 512);
                src += L::kTile;
            }
            ++in_page;
        }
        fill += L::kTile;
        if (fill == ring_end)
            fill -= kStages * L::kTile;
        copies_commit();
    };
    for (int k = 0; k < kStages - 1; ++k)
        issue(k < mine);

    // the rows of q as fp16, each scaled by a power of two; their factors and limits; by a
    // warp for 8 of them
    if (warp < NT) {
        const int col = warp * 8 + g;
        const bool live = col < run.rows;
        const int r = run.row0 + col, i = live ? (int)div_by((uint32_t)r, a.div_group) : 0, qh = live ? r - i * a.group : 0;
        const uint16_t *q = a.q + (int64_t)(s.q0 + i) * a.ldq + ((int64_t)run.head * a.group + qh) * D + t * (D / 4);
        uint4 v[KS / 2];
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            if (live)
                asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(v[j].x), "=r"(v[j].y), "=r"(v[j].z), "=r"(v[j].w) : "l"(q + j * 8) : "memory");
        }
        float amax = 0.0f;
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
            float f[8];
            unpack8(v[j], f);
#pragma unroll
            for (int e = 0; e < 8; ++e)
                amax = fmaxf(amax, fabsf(f[e]));
        }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        float down;
        const float up = fp16_scale(amax, down);
#pragma unroll
        for (int j = 0; j < KS / 2; ++j) {
            float f[8];
            unpack8(v[j], f);
            *reinterpret_cast<uint4 *>(smem + Sh::kQ + ((warp * (KS / 2) + j) * 32 + lane) * 16) =
                make_uint4(pack_f16x2(f[0] * up, f[1] * up), pack_f16x2(f[2] * up, f[3] * up), pack_f16x2(f[4] * up, f[5] * up),
                           pack_f16x2(f[6] * up, f[7] * up));
        }
        // limits of this row's keys
        int h = a.causal ? s.len - s.n + i + 1 : s.len;  // (may be <= 0)
        int l = a.window > 0 ? h - a.window : 0;
        if (!live) {
            h = 0x7fffffff;
            l = 0;
        }
        l = l < 0 ? 0 : l;
        if (t == 0) {
            reinterpret_cast<float *>(smem + Sh::kFactor)[col] = score_factor(a, down, k_scale);
            reinterpret_cast<int *>(smem + Sh::kHi)[col] = min(h, s.len);
            reinterpret_cast<int *>(smem + Sh::kLo)[col] = l;
        }
        const int hi_min = __reduce_min_sync(0xffffffffu, h), lo_max = __reduce_max_sync(0xffffffffu, l);
        const int hi_max = __reduce_max_sync(0xffffffffu, live ? h : 0), lo_min = __reduce_min_sync(0xffffffffu, live ? l : 0x7fffffff);
        if (lane == 0)
            *reinterpret_cast<int4 *>(smem + Sh::kLimits + warp * 16) = make_int4(min(hi_min, s.len), lo_max, min(hi_max, s.len), lo_min);
    }
    __syncthreads();
    int hi_min = 0x7fffffff, lo_max = 0;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int2 limits = *reinterpret_cast<const int2 *>(smem + Sh::kLimits + nt * 16);
        hi_min = min(hi_min, limits.x);
        lo_max = max(lo_max, limits.y);
    }
    float2 kept[NT];  // the rows' factors (32 rows leave no registers for them)
#pragma unroll
    for (int nt = 0; nt < NT && NT < 4; ++nt)
        kept[nt] = *reinterpret_cast<const float2 *>(smem + Sh::kFactor + (nt * 8 + 2 * t) * 4);

    float o[NT][KS][4];
    // the maximum less kLift (0 while there is none), how far above that a score may be (-inf
    // while there is none), and the sum
    float off[NT][2], room[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[nt][i][j] = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            room[nt][j] = -INFINITY;
            off[nt][j] = l[nt][j] = 0.0f;
        }
    }
    // rows g and g + 8 of K are keys k0 and k0 + 8: t and t + 4 then follow each other in p^T
    const int k0 = (g >> 1) + 4 * (g & 1);
    const uint8_t *tile = ring + warp * kStages * L::kTile;
    const uint8_t *const tile_end = tile + kStages * L::kTile;
    // tiles that every row sees: plain of them from the first plain_at on
    const int plain_at = max((lo_max - key0 + 15) >> 4, 0), plain = max((hi_min - key0 + (hi_min < key0 ? -15 : 0)) / 16 - plain_at, 0);
    for (int k = 0; k < mine; ++k, tile = tile + L::kTile == tile_end ? tile_end - kStages * L::kTile : tile + L::kTile) {
        __syncwarp();  // the stage that is filled next has been read
        issue(k + kStages - 1 < mine);
        copies_wait<kStages - 1>();
        __syncwarp();
        if (!(in_cache >> (kStages - 1) & 1))
            continue;
        float sc[NT][4];
        {
            float s2[NT][4];
            uint32_t w[2][KS / 2], sf[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const uint8_t *p = tile + (k0 + 8 * r) * L::kRow + t * (L::kRow / 4);
                const uint8_t *ps = tile + L::kKsf + (k0 + 8 * r) * (D / 16);
                if constexpr (D == 128) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(p);
                    w[r][0] = v.x;
                    w[r][1] = v.y;
                    w[r][2] = v.z;
                    w[r][3] = v.w;
                    sf[r] = e4m3x2(*reinterpret_cast<const uint16_t *>(ps + 2 * t));
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(p);
                    w[r][0] = v.x;
                    w[r][1] = v.y;
                    sf[r] = e4m3x2(ps[t]);
                }
            }
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) {  // a word: 8 d, two products
                // the two words of a block of 16 share its scale
                const uint32_t s0 = __byte_perm(sf[0], 0, i < 2 ? 0x1010 : 0x3232);
                const uint32_t s1 = __byte_perm(sf[1], 0, i < 2 ? 0x1010 : 0x3232);
                const uint32_t a00 = mul_f16x2(e2m1x2<0>(w[0][i]), s0), a01 = mul_f16x2(e2m1x2<1>(w[0][i]), s0);
                const uint32_t a02 = mul_f16x2(e2m1x2<2>(w[0][i]), s0), a03 = mul_f16x2(e2m1x2<3>(w[0][i]), s0);
                const uint32_t a10 = mul_f16x2(e2m1x2<0>(w[1][i]), s1), a11 = mul_f16x2(e2m1x2<1>(w[1][i]), s1);
                const uint32_t a12 = mul_f16x2(e2m1x2<2>(w[1][i]), s1), a13 = mul_f16x2(e2m1x2<3>(w[1][i]), s1);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 q = *reinterpret_cast<const uint4 *>(smem + Sh::kQ + ((nt * (KS / 2) + i) * 32 + lane) * 16);
                    // (two sums side by side, where there are not four of them anyway: a
                    // product waits for the one before in its sum)
                    float(&second)[4] = NT < 4 ? s2[nt] : sc[nt];
                    if (i == 0)
                        mma_first(sc[nt], a00, a10, a01, a11, q.x, q.y);
                    else
                        mma(sc[nt], a00, a10, a01, a11, q.x, q.y);
                    if (i == 0 && NT < 4)
                        mma_first(second, a02, a12, a03, a13, q.z, q.w);
                    else
                        mma(second, a02, a12, a03, a13, q.z, q.w);
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT && NT < 4; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sc[nt][j] += s2[nt][j];
        }
        uint32_t vb[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            vb[j] = tile[L::kVsf + (t + 4 * j) * (D / 16) + (D == 128 ? g : g >> 1)];
        if ((unsigned)(k - plain_at) >= (unsigned)plain) {  // -inf where a row does not see the key
            const int key = key0 + k * 16;
            const int *hi = reinterpret_cast<const int *>(smem + Sh::kHi), *lo = reinterpret_cast<const int *>(smem + Sh::kLo);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int at = key + k0 + 8 * (j >> 1), col = nt * 8 + 2 * t + (j & 1);
                    if (!(at < hi[col] && at >= lo[col]))
                        sc[nt][j] = -INFINITY;
                }
            int hi_max = 0, lo_min = 0x7fffffff;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int2 limits = *reinterpret_cast<const int2 *>(smem + Sh::kLimits + nt * 16 + 8);
                hi_max = max(hi_max, limits.x);
                lo_min = min(lo_min, limits.y);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int at = key + t + 4 * j;
                if (!(at < hi_max && at >= lo_min))
                    vb[j] = 0;  // what a slot that nobody sees holds may be NaN
            }
        }
        // x: scores in units of log2, less the maximum
        float x[NT][4];
        auto factor = [&](int nt) { return NT < 4 ? kept[nt] : *reinterpret_cast<const float2 *>(smem + Sh::kFactor + (nt * 8 + 2 * t) * 4); };
        bool grow = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const float2 cf = factor(nt);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                x[nt][j] = fmaf(sc[nt][j], j & 1 ? cf.y : cf.x, -off[nt][j & 1]);
                grow = grow || x[nt][j] > room[nt][j & 1];
            }
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float f[2];
                const float2 cf = factor(nt);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float c = j ? cf.y : cf.x;
                    const float s0 = __fmul_rn(sc[nt][j], c), s1 = __fmul_rn(sc[nt][j + 2], c);
                    float top = fmaxf(s0, s1);
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                    const bool some = room[nt][j] != -INFINITY;
                    top -= kLift;
                    top = some ? fmaxf(top, off[nt][j]) : top;
                    f[j] = some ? exp2_approx(off[nt][j] - top) : 0.0f;
                    off[nt][j] = top == -INFINITY ? 0.0f : top;
                    const bool far = fabsf(off[nt][j]) >= kFar;  // (comes here for every tile)
                    room[nt][j] = top == -INFINITY ? -INFINITY : (far ? -0x1p127f : kLift + kSlack);
                    l[nt][j] *= f[j];
                    x[nt][j] = far ? s0 - off[nt][j] : fmaf(sc[nt][j], c, -off[nt][j]);
                    x[nt][j + 2] = far ? s1 - off[nt][j] : fmaf(sc[nt][j + 2], c, -off[nt][j]);
                }
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    o[nt][i][0] *= f[0];
                    o[nt][i][1] *= f[1];
                    o[nt][i][2] *= f[0];
                    o[nt][i][3] *= f[1];
                }
            }
        }
        uint32_t pt[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                p[j] = exp2_approx(x[nt][j]);
                l[nt][j & 1] += p[j];
            }
            pt[nt][0] = transpose8(pack_f16x2(p[0], p[1]));
            pt[nt][1] = transpose8(pack_f16x2(p[2], p[3]));
        }
        // O^T: a lane's keys are t, t + 4, t + 8, t + 12, its d those from g D/8 on
        const uint32_t vs[2] = {e4m3x2(__byte_perm(vb[0], vb[1], 0x0040)), e4m3x2(__byte_perm(vb[2], vb[3], 0x0040))};
        uint32_t w[4][D / 64];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint8_t *p = tile + L::kV + (t + 4 * j) * L::kRow + g * (D / 16);
            if constexpr (D == 128) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                w[j][0] = v.x;
                w[j][1] = v.y;
            } else {
                w[j][0] = *reinterpret_cast<const uint32_t *>(p);
            }
        }
#pragma unroll
        for (int h2 = 0; h2 < D / 64; ++h2) {  // words of a lane's codes
            uint32_t e0[4], o0[4], e1[4], o1[4];
            join_keys(w[0][h2], w[1][h2], vs[0], e0, o0);
            join_keys(w[2][h2], w[3][h2], vs[1], e1, o1);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma(o[nt][h2 * 4 + i], e0[i], o0[i], e1[i], o1[i], pt[nt][0], pt[nt][1]);
        }
    }
    copies_wait<0>();
    __syncthreads();  // the ring is free

    float4 *const parts = reinterpret_cast<float4 *>(ring) + warp * NR * (D / 4);
    float *const ms = reinterpret_cast<float *>(smem + Sh::kMs), *const ls = reinterpret_cast<float *>(smem + Sh::kLs);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float v = l[nt][j];
            v += __shfl_xor_sync(0xffffffffu, v, 4);
            v += __shfl_xor_sync(0xffffffffu, v, 8);
            v += __shfl_xor_sync(0xffffffffu, v, 16);
            const int col = nt * 8 + 2 * t + j;
            if (g == 0) {
                ms[warp * NR + col] = room[nt][j] == -INFINITY ? -INFINITY : off[nt][j];
                ls[warp * NR + col] = v;
            }
#pragma unroll
            for (int i = 0; i < KS; i += 2)
                parts[Sh::place(col, g * (D / 32) + i / 2)] = make_float4(o[nt][i][j], o[nt][i][j + 2], o[nt][i + 1][j], o[nt][i + 1][j + 2]);
        }
    }
    __syncthreads();
}

// Parts with maxima m_i and sums l_i are joined with factors exp2(m_i - max); a part
// without a maximum has nothing, or what is not a number.
__device__ __forceinline__ float join_factor(float m, float l, float top)
{
    return m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : exp2_approx(m - top);
}

// What lane i's part counts for, of N parts with maximum m and sum l each (lanes i, i + N, ..
// have the same one); the parts' maximum and sum.
template <int N>
__device__ __forceinline__ float part_factor(float m, float l, float &top, float &sum)
{
    top = m;
#pragma unroll
    for (int o = 1; o < N; o <<= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float f = join_factor(m, l, top);
    sum = f * l;
#pragma unroll
    for (int o = 1; o < N; o <<= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return f;
}

__device__ __forceinline__ void add_scaled(float4 &acc, float f, const float4 &v)
{
    acc.x = fmaf(f, v.x, acc.x);
    acc.y = fmaf(f, v.y, acc.y);
    acc.z = fmaf(f, v.z, acc.z);
    acc.w = fmaf(f, v.w, acc.w);
}

// 4 elements of a row, summed over the block's warps (by whole warps, of any rows).
template <int D, int NT, int WARPS>
__device__ __forceinline__ float4 join_warps(const uint8_t *smem, int row, int four, float &top, float &sum)
{
    using Sh = Shared<D, NT, WARPS>;
    constexpr int NR = 8 * NT;
    const int w0 = threadIdx.x % WARPS;
    const float f = part_factor<WARPS>(reinterpret_cast<const float *>(smem + Sh::kMs)[w0 * NR + row],
                                       reinterpret_cast<const float *>(smem + Sh::kLs)[w0 * NR + row], top, sum);
    const float4 *const parts = reinterpret_cast<const float4 *>(smem) + Sh::place(row, four);
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < WARPS; ++w)
        add_scaled(acc, __shfl_sync(0xffffffffu, f, w, WARPS), parts[w * NR * (D / 4)]);
    return acc;
}

// 4 elements of a row of the output, and its lse.
template <int D>
__device__ __forceinline__ void put_row(const AttnArgs &a, int q0, int head, int64_t row, int d, const float4 &acc, float top, float sum, float vg)
{
    const int i = (int)div_by((uint32_t)row, a.div_group);
    const int qh = head * a.group + ((int)row - i * a.group);
    const float by = sum == 0.0f ? 0.0f : 1.0f / sum, of = 1.0f / vg;  // (their product may be out of range)
    *reinterpret_cast<uint2 *>(a.out + (int64_t)(q0 + i) * a.ldo + (int64_t)qh * D + d) =
        make_uint2(pack_bf16x2(acc.x * by * of, acc.y * by * of), pack_bf16x2(acc.z * by * of, acc.w * by * of));
    if (a.lse != nullptr && d == 0)
        a.lse[(int64_t)(q0 + i) * a.hq + qh] = sum == 0.0f ? -INFINITY : (top == -INFINITY ? 0.0f : top) * kLn2 + logf(sum);
}

// Even shares.
template <int D, int NT>
__global__ void __launch_bounds__(share_warps(NT) * 32, blocks_per_sm(NT)) attn_few_kernel(const __grid_constant__ AttnArgs a)
{
    constexpr int NR = 8 * NT, kWarps = share_warps(NT), kThreads = kWarps * 32, kWarpRows = 128 / D;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ int64_t sums[kThreads];
    __shared__ int64_t warp_sums[kWarps];
    __shared__ int64_t state[6];
    __shared__ Run kept;
    __shared__ float k_scale;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float *const slots = a.partial + (int64_t)gridDim.x * (sizeof(Record) / 4);
    Record *const record = reinterpret_cast<Record *>(a.partial) + blockIdx.x;
    pdl_wait();

    // every block's share of the tiles: thread i sums the sequences i * per ..
    const int per = (a.B + kThreads - 1) / kThreads;
    int64_t sum = 0;
    for (int b = tid * per; b < a.B && b < (tid + 1) * per; ++b)
        sum += weight(a, sequence<NR>(a, b), way_of(NT));
    int64_t scan = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xffffffffu, scan, o);
        if (lane >= o)
            scan += v;
    }
    if (lane == 31)
        warp_sums[warp] = scan;
    __syncthreads();
    int64_t total = 0;
    for (int i = 0; i < kWarps; ++i) {
        if (i < warp)
            scan += warp_sums[i];
        total += warp_sums[i];
    }
    sums[tid] = scan;  // inclusive
    __syncthreads();
    const int64_t even = (total + gridDim.x - 1) / gridDim.x, share = even > kShare ? even : kShare;
    int64_t pos = blockIdx.x * share;
    int64_t end = pos + share < total ? pos + share : total;
    if (tid == 0)
        record->last = -1;
    if (pos >= end) {
        pdl_launch_dependents();
        return;
    }
    Run run;
    int64_t base;  // tiles before the sequence
    {
        int lo = 0, hi = kThreads - 1;  // the first thread whose sum passes pos
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (sums[mid] > pos)
                hi = mid;
            else
                lo = mid + 1;
        }
        run.b = lo * per;
        base = lo > 0 ? sums[lo - 1] : 0;
    }
    run.s = sequence<NR>(a, run.b);
    if (tid == 0)
        k_scale = *a.cache.k_scale;

    while (pos < end) {
        while (pos >= base + weight(a, run.s, way_of(NT))) {
            base += weight(a, run.s, way_of(NT));
            run.s = sequence<NR>(a, ++run.b);
        }
        const int64_t unit = (pos - base) / (run.s.tiles + way_of(NT));
        const int skip = (int)(pos - base - unit * (run.s.tiles + way_of(NT))), all = run.s.tiles + way_of(NT) - skip;
        const int length = (int)(all < end - pos ? all : end - pos);
        run.first = max(skip - way_of(NT), 0);
        run.count = max(skip + length - way_of(NT), 0) - run.first;
        if (run.count == 0) {  // the way alone
            pos += length;
            continue;
        }
        run.first += run.s.first;
        run.head = (int)(unit / run.s.parts);
        run.row0 = (int)(unit - (int64_t)run.head * run.s.parts) * NR;
        run.rows = run.s.n * a.group - run.row0 < NR ? run.s.n * a.group - run.row0 : NR;
        // (kept in shared memory over the tiles, for the registers' sake)
        if (tid == 0) {
            state[0] = pos;
            state[1] = end;
            state[2] = base;
            state[3] = share;
            state[4] = pos - skip + run.s.tiles + way_of(NT);  // the unit's end
            state[5] = length;
            kept = run;
        }
        __syncthreads();
        attend<D, NT, kWarps>(a, kept, k_scale, smem);
        run = kept;
        pos = state[0];
        end = state[1];
        base = state[2];
        const bool begins = run.first == run.s.first, ends = run.first + run.count == run.s.first + run.s.tiles;
        if (begins && !ends && tid == 0) {
            record->last = (int32_t)((state[4] - 1) / state[3]);
            record->q0 = run.s.q0;
            record->head = run.head;
            record->rows = run.rows;
            record->row0 = run.row0;
        }
        float *slot = slots + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * slot_floats(NR, D);
        for (int r0 = tid / 32 * kWarpRows; r0 < run.rows; r0 += kWarps * kWarpRows) {
            const int row = r0 + lane / (D / 4), d = (tid % (D / 4)) * 4;
            float top, sum_l;
            const float4 acc = join_warps<D, NT, kWarps>(smem, row, d / 4, top, sum_l);
            if (row >= run.rows)
                continue;
            if (begins && ends) {
                put_row<D>(a, run.s.q0, run.head, run.row0 + row, d, acc, top, sum_l, *a.cache.v_scale);
            } else {
                *reinterpret_cast<float4 *>(slot + row * D + d) = acc;
                if (d == 0) {
                    slot[NR * D + row] = top;
                    slot[NR * D + NR + row] = sum_l;
                }
            }
        }
        pos += state[5];
        __syncthreads();  // before the state and the ring are filled again
    }
    pdl_launch_dependents();
}

// A cluster for each sequence and key head, and (the grid's y) row tile: its blocks share
// the keys.  Each block joins the cluster's parts of NR / blocks rows, which the others
// write into its shared memory.
template <int D, int NT>
__global__ void __launch_bounds__(kClusterWarps * 32, NT == 1 ? 2 : 1) attn_cluster_kernel(const __grid_constant__ AttnArgs a, int blocks)
{
    constexpr int NR = 8 * NT, kWarps = kClusterWarps, kWarpRows = 128 / D;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float part[NR][D];  // [blocks][NR / blocks][D]
    __shared__ float part_m[NR], part_l[NR];
    const int tid = threadIdx.x, lane = tid & 31, rank = (int)cluster_rank();
    const int each = NR / blocks, unit = blockIdx.x / blocks;
    cluster_arrive_relaxed();  // (a block's shared memory is there once it has started)
    Run run;
    run.b = unit / a.cache.heads;
    run.head = unit - run.b * a.cache.heads;
    // the table is read where the copies begin: have it nearer by then
    for (int64_t i = (int64_t)tid * 32; i < a.max_pages; i += kWarps * 32 * 32)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(a.table + (int64_t)run.b * a.max_pages + i));
    pdl_wait();
    const float k_scale = *a.cache.k_scale;
    run.s = sequence<NR>(a, run.b);
    if ((int)blockIdx.y >= run.s.parts)
        cluster_wait();
    for (int rt = blockIdx.y; rt < run.s.parts; rt += gridDim.y) {
        run.row0 = rt * NR;
        run.rows = run.s.n * a.group - run.row0 < NR ? run.s.n * a.group - run.row0 : NR;
        const int begin = (int)((int64_t)run.s.tiles * rank / blocks);
        run.first = run.s.first + begin;
        run.count = (int)((int64_t)run.s.tiles * (rank + 1) / blocks) - begin;
        attend<D, NT, kWarps>(a, run, k_scale, smem);
        const float vg = *a.cache.v_scale;
        cluster_wait();  // every block has started, and has read what it was given before
        for (int r0 = tid / 32 * kWarpRows; r0 < run.rows; r0 += kWarps * kWarpRows) {
            const int row = r0 + lane / (D / 4), d = (tid % (D / 4)) * 4;
            float top, sum_l;
            const float4 acc = join_warps<D, NT, kWarps>(smem, row, d / 4, top, sum_l);
            if (row >= run.rows)
                continue;
            const int to = row / each, at = rank * each + row - to * each;
            st_cluster128(map_rank(smem_addr(&part[at][d]), to), acc);
            if (d == 0) {
                st_cluster32(map_rank(smem_addr(&part_m[at]), to), __float_as_uint(top));
                st_cluster32(map_rank(smem_addr(&part_l[at]), to), __float_as_uint(sum_l));
            }
        }
        cluster_sync();
        for (int r0 = tid / 32 * kWarpRows; r0 < each; r0 += kWarps * kWarpRows) {
            const int r = r0 + lane / (D / 4), d = (tid % (D / 4)) * 4, row = rank * each + r;
            const int at = (lane % kMostBlocks) * each + (r < each ? r : 0);
            const bool some = lane % kMostBlocks < blocks;
            float top, sum_l;
            const float f = part_factor<kMostBlocks>(some ? part_m[at] : -INFINITY, some ? part_l[at] : 0.0f, top, sum_l);
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int i = 0; i < blocks; ++i)
                add_scaled(acc, __shfl_sync(0xffffffffu, f, i, kMostBlocks), *reinterpret_cast<const float4 *>(&part[i * each + (r < each ? r : 0)][d]));
            if (r < each && row < run.rows)
                put_row<D>(a, run.s.q0, run.head, run.row0 + row, d, acc, top, sum_l, vg);
        }
        if (rt + (int)gridDim.y < run.s.parts)
            cluster_arrive();
    }
    pdl_launch_dependents();
}

// Units over several blocks: block (x, y, z) has row y of the x-th of them, and of that
// the z-th LANES times 4 elements; each set of LANES lanes takes a run of the parts in
// order, whose loads are all under way together.
template <int D, int LANES, int THREADS>
__global__ void __launch_bounds__(THREADS) attn_join_kernel(const __grid_constant__ AttnArgs a, int blocks, int NR)
{
    constexpr int kSets = THREADS / LANES, kWarps = THREADS / 32, kMost = blocks_of(1);
    __shared__ float4 acc_of[kWarps][LANES];
    __shared__ float factor[kMost], l_of[kWarps], top_of[kWarps];
    __shared__ int counts[kMost / 32 + 1], which;
    const int row = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    pdl_wait();
    pdl_launch_dependents();
    const Record *records = reinterpret_cast<const Record *>(a.partial);
    int first = blockIdx.x;
    if ((int)gridDim.x < blocks) {  // fewer units than blocks: look for the x-th that is over several
        if (tid == 0)
            which = -1;
        for (int i = tid; i < (blocks + 31) / 32 * 32; i += THREADS) {
            const unsigned some = __ballot_sync(0xffffffffu, i < blocks && records[i].last >= 0);
            if (lane == 0)
                counts[i >> 5] = (int)some;
        }
        __syncthreads();
        if (tid < 32) {
            const unsigned some = lane < (blocks + 31) / 32 ? (unsigned)counts[lane] : 0u;
            int before = __popc(some);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int up = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o)
                    before += up;
            }
            before -= __popc(some);
            for (unsigned left = some; left != 0; left &= left - 1, ++before)
                if (before == first)
                    which = lane * 32 + __ffs(left) - 1;
        }
        __syncthreads();
        first = which;
        if (first < 0)
            return;
    }
    const Record rec = records[first];
    if (rec.last < 0 || row >= rec.rows)
        return;
    const float *slots = a.partial + (int64_t)blocks * (sizeof(Record) / 4);
    auto slot_of = [&](int i) { return slots + ((int64_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * slot_floats(NR, D); };
    const int n = rec.last - first + 1;  // at most `blocks`
    // the parts' maxima, and what each part counts for
    float top = -INFINITY;
    for (int i = tid; i < n; i += THREADS) {
        factor[i] = slot_of(i)[NR * D + row];
        top = fmaxf(top, factor[i]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (lane == 0)
        top_of[tid >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < THREADS / 32; ++i)
        top = fmaxf(top, top_of[i]);
    const int set = tid / LANES, d = ((int)blockIdx.z * LANES + tid % LANES) * 4, per = (n + kSets - 1) / kSets;
    const int i0 = min(n, set * per), i1 = min(n, i0 + per);
    float l = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int i = i0; i < i1; ++i) {
        const float *slot = slot_of(i);
        const float li = slot[NR * D + NR + row];
        const float4 v = *reinterpret_cast<const float4 *>(slot + row * D + d);
        const float f = join_factor(factor[i], li, top);
        l = fmaf(f, li, l);
        add_scaled(acc, f, v);
    }
    // the sets of a warp, then the warps
    auto over_sets = [&]() {
#pragma unroll
        for (int o = LANES; o < 32; o <<= 1) {
            l += __shfl_xor_sync(0xffffffffu, l, o);
            acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
            acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
            acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
            acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
        }
    };
    over_sets();
    if (lane < LANES)
        acc_of[tid >> 5][lane] = acc;
    if (lane == 0)
        l_of[tid >> 5] = l;
    __syncthreads();
    if (tid >= 32)
        return;
    l = 0.0f;
    acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
    for (int i = lane / LANES; i < kWarps; i += 32 / LANES) {
        l += l_of[i];
        add_scaled(acc, 1.0f, acc_of[i][lane % LANES]);
    }
    over_sets();
    if (lane < LANES)
        put_row<D>(a, rec.q0, rec.head, rec.row0 + row, d, acc, top, l, *a.cache.v_scale);
}

// Dynamic shared memory above 48 KB, asked for once a device.
template <typename K>
cudaError_t allow_shared(K kernel, int bytes, std::atomic<bool> (&ready)[kMaxCachedDevices])
{
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    const bool cached = dev >= 0 && dev < kMaxCachedDevices;
    if (cached && ready[dev].load(std::memory_order_relaxed))
        return cudaSuccess;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess && cached)
        ready[dev].store(true, std::memory_order_relaxed);
    return err;
}

template <int D, int NT>
cudaError_t launch_few(const AttnArgs &a, int64_t rows, bool pdl, cudaStream_t stream)
{
    constexpr int kBlocks = blocks_of(NT);
    const int cluster = cluster_of(a.B, a.cache.heads, rows, a.max_pages * a.cache.page_size, a.window);
    if (cluster > 0) {
        constexpr int smem = Shared<D, NT, kClusterWarps>::kBytes;
        static std::atomic<bool> ready[kMaxCachedDevices];
        const cudaError_t err = allow_shared(attn_cluster_kernel<D, NT>, smem, ready);
        if (err != cudaSuccess)
            return err;
        return launch_clusters(attn_cluster_kernel<D, NT>, dim3((unsigned)(a.B * a.cache.heads * cluster), (unsigned)((rows + 8 * NT - 1) / (8 * NT))),
                               dim3(kClusterWarps * 32), smem, stream, pdl, (unsigned)cluster, a, cluster);
    }
    constexpr int smem = Shared<D, NT, share_warps(NT)>::kBytes;
    static std::atomic<bool> ready[kMaxCachedDevices];
    cudaError_t err = allow_shared(attn_few_kernel<D, NT>, smem, ready);
    if (err != cudaSuccess)
        return err;
    err = launch_kernel(attn_few_kernel<D, NT>, dim3(kBlocks), dim3(share_warps(NT) * 32), smem, stream, pdl, a);
    if (err != cudaSuccess)
        return err;
    // at most as many units as rows of 8 NT, and one more for each sequence and head
    const int64_t units = a.cache.heads * (a.T * a.group / (8 * NT) + a.B);
    if (units * 8 * NT * (D / 32) <= 2 * kSms)  // few units, of many parts each: all resident at once
        return launch_kernel(attn_join_kernel<D, 8, 1024>, dim3((unsigned)units, 8 * NT, D / 32), dim3(1024), 0, stream, true, a, kBlocks, 8 * NT);
    return launch_kernel(attn_join_kernel<D, D / 4, 256>, dim3((unsigned)(units < kBlocks ? units : kBlocks), 8 * NT), dim3(256), 0, stream, true, a,
                         kBlocks, 8 * NT);
}

}  // namespace

bool attn_few_clusters(int64_t B, int64_t heads, int64_t rows, int64_t keys, int64_t window)
{
    // (and no smaller call of as many keys takes shares)
    if (window > 0 && window + rows < keys)
        keys = window + rows;
    return cluster_of(B, heads, rows, keys, 0) > 0 && keys <= kClusterKeys / 2 * kMostBlocks;
}

cudaError_t launch_attn_few(const AttnArgs &a, int64_t rows, bool pdl, cudaStream_t stream)
{
    switch (eights_of(rows)) {
    case 1: return a.D == 64 ? launch_few<64, 1>(a, rows, pdl, stream) : launch_few<128, 1>(a, rows, pdl, stream);
    case 2: return a.D == 64 ? launch_few<64, 2>(a, rows, pdl, stream) : launch_few<128, 2>(a, rows, pdl, stream);
    default: return a.D == 64 ? launch_few<64, 4>(a, rows, pdl, stream) : launch_few<128, 4>(a, rows, pdl, stream);
    }
}

int64_t attn_few_workspace(int64_t D)
{
    int64_t most = 0;  // (the same for every form, so that it does not shrink where max_q grows)
    for (int nt = 1; nt <= 4; nt *= 2) {
        const int64_t n = blocks_of(nt) * ((int64_t)sizeof(Record) + 2 * 4 * slot_floats(8 * nt, (int)D));
        most = n > most ? n : most;
    }
    return most;
}

}  // namespace tsfn
