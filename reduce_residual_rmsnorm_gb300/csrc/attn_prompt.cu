// Attention of many rows over the paged NVFP4 cache, on the fifth-generation tensor
// cores: prompts, and pieces of them after what the cache holds.
//
//   S = q K^T,   p_j = exp2(c S_j - m),   O = p V,   out = O / (sum_j p_j v_scale)
//
// A block works on 256 rows, (query, head) pairs that share a key head, as two tiles of
// 128, and goes over the keys 128 at a time.  K and V are exact in fp16 (6 significant
// bits), as are rows of q scaled by a power of two; products are tcgen05.mma kind::f16
// with fp32 sums in tensor memory, where S, p (fp16, over S) and O of both tiles take
// all 512 columns (D = 128).  Roles of the block's 13 warps:
//   - 4 for each tile: a thread has a row: its maximum and sum, exp2, p back to tensor
//     memory, and the rescaling of O, only when a score passes the maximum by 2^8;
//   - 4 turn codes and scale factors into fp16 tiles in shared memory, two stages
//     deep, K and V alike with the codes of the next keys already in registers: K is
//     read along d, V across it, so neither is transposed;
//   - one issues the products: while one tile's p is made, the other's run.
//
// Work is split evenly as in attn_few.cu: all units' key tiles in one row, cut into
// equal shares; what a share leaves of a unit is joined by attn_join_rows_kernel.
// Every wait has a limit, after which the block records it and ends.
#include "attn_util.cuh"
#include "device_util.cuh"
#include "tcgen05.cuh"

namespace tsfn {

namespace {

__device__ uint32_t g_stalled_waits;

#ifndef TSFN_WAIT_CYCLES
#define TSFN_WAIT_CYCLES 4000000000LL
#endif
constexpr long long kWaitCycles = TSFN_WAIT_CYCLES;  // a wait's limit: about 2 s

constexpr int kRows = 256;          // rows of a unit
constexpr int kKeys = 128;          // keys of a step
constexpr int kBlocks = 152;        // one for each SM
constexpr int kShare = 4;           // steps of a share, at least
constexpr int kMakers = 128;        // threads that make K and V
constexpr int kThreads = kRows + kMakers + 32;
constexpr int kSeqs = 256;          // sequences whose weights are summed at a time

// Shared memory: q of both tiles, two stages of K and of V, each in blocks of 64 d
// (128 bytes) by 128 rows under the 128-byte swizzle.
template <int D>
struct Smem {
    static constexpr int kBlock = 128 * 128;
    static constexpr int kMatrix = D / 64 * kBlock;
    static constexpr int kQ = 0, kK = 2 * kMatrix, kV = 4 * kMatrix, kBytes = 6 * kMatrix + 1024;
};

struct Barriers {
    uint64_t q_full[2], s_full[2], p_full[2], o_full[2];  // of each tile
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];  // of each stage
    uint64_t last;
};

__device__ __forceinline__ void give_up(volatile int *dead)
{
    *dead = 1;
    atomicAdd(&g_stalled_waits, 1u);
}

// The whole warp waits for a phase; false where the block has given up.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *dead)
{
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
        return true;
    const long long t0 = clock64();
    for (;;) {
        if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
            return true;
        const bool late = clock64() - t0 > kWaitCycles;
        if (__any_sync(0xffffffffu, late || *dead != 0)) {
            if ((threadIdx.x & 31) == 0 && *dead == 0)
                give_up(dead);
            return false;
        }
    }
}

// The loads before it are done: the registers are used after it only.
__device__ __forceinline__ void loaded(uint32_t (&v)[32])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]), "+r"(v[8]),
                   "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]),
                   "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                   "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
}

// Rows rt * 256 .. of a sequence: the steps of keys that any of them sees.
struct Part {
    int row0, rows;
    int first, steps;     // at least one step
    int see_lo, see_hi;   // keys that some row sees
};

__device__ __forceinline__ Part part_of(const AttnArgs &a, const Seq &s, int rt)
{
    Part p;
    const int all = (int)(s.n * a.group);
    p.row0 = rt * kRows;
    p.rows = all - p.row0 < kRows ? all - p.row0 : kRows;
    const int i0 = p.row0 / a.group, i1 = (p.row0 + p.rows - 1) / a.group;
    int hi = a.causal ? (int)(s.len - s.n + i1 + 1) : s.len;
    int lo = a.window > 0 ? (int)(s.len - s.n + i0 + 1) - a.window : 0;
    p.see_hi = hi < 0 ? 0 : hi;
    p.see_lo = lo < 0 ? 0 : lo;
    p.first = p.see_lo / kKeys;
    const int steps = (p.see_hi + kKeys - 1) / kKeys - p.first;
    p.steps = steps > 1 ? steps : 1;
    return p;
}

// The steps of a sequence's row tiles for one key head, by a whole warp.
__device__ __forceinline__ int64_t steps_of(const AttnArgs &a, const Seq &s)
{
    int64_t sum = 0;
    for (int rt = threadIdx.x & 31; rt < s.parts; rt += 32)
        sum += part_of(a, s, rt).steps;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// Where a share stands: the unit (sequence, key head, row tile) and the step in it.
struct Place {
    int64_t pos, end;  // steps of all units
    int b, head, rt, step;
    Seq s;
    Part part;
};

__device__ __forceinline__ int left_of(const Place &p)
{
    const int64_t here = p.part.steps - p.step, left = p.end - p.pos;
    return (int)(here < left ? here : left);
}

__device__ __forceinline__ void next_unit(const AttnArgs &a, Place &p, int count)
{
    p.pos += count;
    if (p.pos >= p.end)
        return;
    p.step = 0;
    if (++p.rt == p.s.parts) {
        p.rt = 0;
        if (++p.head == a.cache.heads) {
            p.head = 0;
            do
                p.s = sequence<kRows>(a, ++p.b);
            while (p.s.parts == 0);
        }
    }
    p.part = part_of(a, p.s, p.rt);
}

// To the next unit, whose first step comes after `count` of this one's (by one lane, for
// its warp).
__device__ __forceinline__ void advance(const AttnArgs &a, Place &place, int count)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        Place p = place;
        next_unit(a, p, count);
        place = p;
    }
    __syncwarp();
}

// This block's share, found by all warps together (each thread gets it).
__device__ __forceinline__ Place my_share(const AttnArgs &a, int64_t *weights, int64_t &share)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // inclusive sums of the weights of sequences c0 .. c0 + 255
    auto sums = [&](int c0) {
        __syncthreads();
        for (int i = warp; i < kSeqs && c0 + i < a.B; i += kThreads / 32) {
            const int64_t w = steps_of(a, sequence<kRows>(a, c0 + i)) * a.cache.heads;
            if (lane == 0)
                weights[i] = w;
        }
        __syncthreads();
        if (warp == 0) {
            int64_t v[kSeqs / 32], run = 0;
#pragma unroll
            for (int i = 0; i < kSeqs / 32; ++i) {
                const int at = lane * (kSeqs / 32) + i;
                run += c0 + at < a.B ? weights[at] : 0;
                v[i] = run;
            }
            int64_t before = run;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, before, o);
                if (lane >= o)
                    before += up;
            }
            before -= run;
#pragma unroll
            for (int i = 0; i < kSeqs / 32; ++i)
                weights[lane * (kSeqs / 32) + i] = before + v[i];
        }
        __syncthreads();
    };
    int64_t total = 0;
    for (int c0 = 0; c0 < a.B; c0 += kSeqs) {
        sums(c0);
        total += weights[kSeqs - 1];
    }
    const int64_t even = (total + gridDim.x - 1) / gridDim.x;
    share = even > kShare ? even : kShare;
    Place p;
    p.pos = blockIdx.x * share;
    p.end = p.pos + share < total ? p.pos + share : total;
    p.b = p.head = p.rt = p.step = 0;
    if (p.pos >= p.end)
        return p;
    int64_t base = 0;
    int c0 = 0;
    for (;; c0 += kSeqs) {
        if (a.B > kSeqs)
            sums(c0);
        if (p.pos < base + weights[kSeqs - 1])
            break;
        base += weights[kSeqs - 1];
    }
    int lo = 0, hi = kSeqs - 1;  // the first sequence whose sum passes pos
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (base + weights[mid] > p.pos)
            hi = mid;
        else
            lo = mid + 1;
    }
    p.b = c0 + lo;
    int64_t r = p.pos - base - (lo > 0 ? weights[lo - 1] : 0);
    p.s = sequence<kRows>(a, p.b);
    const int64_t each = steps_of(a, p.s);
    p.head = (int)(r / each);
    r -= p.head * each;
    // the row tile, 32 at a time
    for (int rt0 = 0;; rt0 += 32) {
        const int steps = rt0 + lane < p.s.parts ? part_of(a, p.s, rt0 + lane).steps : 0;
        int64_t scan = steps;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o)
                scan += up;
        }
        const unsigned past = __ballot_sync(0xffffffffu, scan > r);
        if (past != 0) {
            const int at = __ffs(past) - 1;
            p.rt = rt0 + at;
            p.step = (int)(r - (__shfl_sync(0xffffffffu, scan, at) - __shfl_sync(0xffffffffu, steps, at)));
            break;
        }
        r -= __shfl_sync(0xffffffffu, scan, 31);
    }
    p.part = part_of(a, p.s, p.rt);
    return p;
}

// 16 bytes of codes (32 d of a key) as fp16 into a row's half of a block of a swizzled
// matrix.  `row`: the row's address, `half`: chunk 0 or 4 of it, `turn`: row % 8.  Lanes
// with the two blocks of a row (`swap`) write their words in opposite order, so that 8
// lanes' stores fill 128 bytes.
__device__ __forceinline__ void put_codes(uint32_t row, uint32_t half, uint32_t turn, bool swap, uint4 w, uint32_t sf2)
{
    const uint32_t sf = e4m3x2(sf2);
    const uint32_t s0 = __byte_perm(sf, 0, swap ? 0x3232 : 0x1010), s1 = __byte_perm(sf, 0, swap ? 0x1010 : 0x3232);
    const uint32_t word[4] = {swap ? w.z : w.x, swap ? w.w : w.y, swap ? w.x : w.z, swap ? w.y : w.w};
    const uint32_t first = (half + (swap ? 2 : 0)) ^ turn;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t s = i < 2 ? s0 : s1;
        st_shared(row + (first ^ i) * 16, make_uint4(mul_f16x2(e2m1x2<0>(word[i]), s), mul_f16x2(e2m1x2<1>(word[i]), s),
                                                     mul_f16x2(e2m1x2<2>(word[i]), s), mul_f16x2(e2m1x2<3>(word[i]), s)));
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) attn_prompt_kernel(const __grid_constant__ AttnArgs a)
{
    using S = Smem<D>;
    using L = Layout<D>;
    constexpr uint32_t kSCol = 0, kOCol = 256;  // tensor memory: S (and p) of both tiles, then O
    extern __shared__ uint8_t raw[];
    __shared__ Barriers bars;
    __shared__ int64_t weights[kSeqs];
    __shared__ uint32_t tmem_at;
    __shared__ volatile int dead;
    __shared__ uint8_t seen[4][8];  // whether a step's tiles of 16 keys lie in the cache
    const uint32_t smem = (smem_u32(raw) + 1023) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5;

    Record *const record = reinterpret_cast<Record *>(a.partial) + blockIdx.x;
    float *const slots = a.partial + (int64_t)gridDim.x * (sizeof(Record) / 4);

    if (warp == kThreads / 32 - 1)
        tmem_alloc(smem_u32(&tmem_at), 512);
    if (tid == 0) {
        dead = 0;
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.q_full[i]), 128);
            mbar_init(smem_u32(&bars.s_full[i]), 1);
            mbar_init(smem_u32(&bars.p_full[i]), 128);
            mbar_init(smem_u32(&bars.o_full[i]), 1);
            mbar_init(smem_u32(&bars.k_full[i]), kMakers);
            mbar_init(smem_u32(&bars.k_empty[i]), 1);
            mbar_init(smem_u32(&bars.v_full[i]), kMakers);
            mbar_init(smem_u32(&bars.v_empty[i]), 1);
        }
        mbar_init(smem_u32(&bars.last), 1);
        mbar_fence_init();
    }
    tmem_fence_before();
    pdl_wait();
    // (a copy for each warp, in shared memory for the registers' sake)
    __shared__ Place places[kThreads / 32];
    __shared__ int64_t share_of;
    Place &place = places[warp];
    {
        int64_t share;
        const Place first = my_share(a, weights, share);
        if ((tid & 31) == 0)
            place = first;
        if (tid == 0)
            share_of = share;
    }
    __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_at;
    if (tid == 0)
        record->last = -1;

    if (warp < 8) {
        // ---- softmax: thread (tile, r) has row r of its tile
        const int tile = warp >> 2, r = tid & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane 32 (warp % 4) of tensor memory
        const uint32_t s_at = tmem + kSCol + tile * 128 + lanes, o_at = tmem + kOCol + tile * D + lanes;
        const uint32_t q_smem = smem + S::kQ + tile * S::kMatrix;
        const uint32_t s_full = smem_u32(&bars.s_full[tile]), p_full = smem_u32(&bars.p_full[tile]);
        const float vg = *a.cache.v_scale;
        const float c0 = a.scale * kLog2e / *a.cache.k_scale;
        uint32_t step = 0, done = 0, units_done = 0;  // steps of the block and of this tile
        bool alive = true;
        while (alive && place.pos < place.end) {
            const int count = left_of(place);
            const int rows = place.part.rows - tile * 128;  // of this tile
            if (rows > 0) {
                // this row of q, scaled by a power of two, as fp16
                const int row = place.part.row0 + tile * 128 + r;
                const bool live = r < rows;
                const int i = live ? row / a.group : 0;
                const int qh = place.head * a.group + (live ? row - i * a.group : 0);
                const uint16_t *src = a.q + (int64_t)(place.s.q0 + i) * a.ldq + (int64_t)qh * D;
                float amax = 0.0f, down;
                auto chunk = [&](int c, float (&f)[8]) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (live)
                        asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(src + c * 8) : "memory");
                    unpack8(v, f);
                };
                // (read twice: 16 chunks would take 64 registers)
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    float f[8];
                    chunk(c, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        amax = fmaxf(amax, fabsf(f[e]));
                }
                const float up = fp16_scale(amax, down);
#pragma unroll 4
                for (int c = 0; c < D / 8; ++c) {
                    float f[8];
                    chunk(c, f);
                    st_shared(q_smem + (c >> 3) * S::kBlock + r * 128 + (((c & 7) ^ (r & 7)) * 16),
                              make_uint4(pack_f16x2(f[0] * up, f[1] * up), pack_f16x2(f[2] * up, f[3] * up),
                                         pack_f16x2(f[4] * up, f[5] * up), pack_f16x2(f[6] * up, f[7] * up)));
                }
                fence_async_proxy();
                mbar_arrive(smem_u32(&bars.q_full[tile]));
                const float cf = c0 * down;
                int hi = a.causal ? (int)(place.s.len - place.s.n + i + 1) : place.s.len;
                int lo = a.window > 0 ? hi - a.window : 0;
                if (!live) {  // (its scores are zeros)
                    hi = 0x7fffffff;
                    lo = 0;
                }
                const int hi_min = min(__reduce_min_sync(0xffffffffu, hi), place.s.len);
                const int lo_max = __reduce_max_sync(0xffffffffu, lo);

                float m = -INFINITY, l = 0.0f;
                for (int k = 0; k < count; ++k, ++done) {
                    const int key = (place.part.first + place.step + k) * kKeys;
                    alive = wait(s_full, done & 1, &dead);
                    if (!alive)
                        break;
                    tmem_fence_after();
                    const uint2 in = *reinterpret_cast<const uint2 *>(seen[(step + k) & 3]);
                    const bool whole = key >= lo_max && key + kKeys <= hi_min && in.x == 0x01010101u && in.y == 0x01010101u;
                    auto mask = [&](uint32_t (&v)[32], int c) {
                        // bit j: key 32 c + j of the step is seen
                        const int h = min(max(min(hi, place.s.len) - key - 32 * c, 0), 32), w = min(max(lo - key - 32 * c, 0), 32);
                        const uint32_t ok = (c < 2 ? in.x : in.y) >> (16 * (c & 1));
                        const uint32_t sees = (uint32_t)((1ull << h) - (1ull << min(w, h))) &
                                              ((ok & 1 ? 0xFFFFu : 0u) | (ok & 0x100 ? 0xFFFF0000u : 0u));
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(sees >> j & 1))
                                v[j] = 0xFF800000u;
                    };
                    float top = -INFINITY;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_load32(s_at + 32 * c, v);
                        loaded(v);
                        if (!whole)
                            mask(v, c);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            top = fmaxf(top, __uint_as_float(v[j]));
                    }
                    top *= cf;
                    const bool grow = top > m + kSlack;
                    if (__any_sync(0xffffffffu, grow)) {
                        const float to = fmaxf(m, top);
                        const float f = m == -INFINITY ? 0.0f : exp2_approx(m - to);
                        m = to;
                        l *= f;
                        if (k > 0) {
#pragma unroll 1
                            for (int c = 0; c < D / 32; ++c) {
                                uint32_t v[32];
                                tmem_load32(o_at + 32 * c, v);
                                loaded(v);
#pragma unroll
                                for (int j = 0; j < 32; ++j)
                                    v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
                                tmem_store32(o_at + 32 * c, v);
                            }
                        }
                    }
                    const float off = m == -INFINITY ? 0.0f : -m;
                    float sum[2] = {0.0f, 0.0f};
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32], p[16];
                        tmem_load32(s_at + 32 * c, v);
                        loaded(v);
                        if (!whole)
                            mask(v, c);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float e0 = exp2_approx(__fmaf_rn(__uint_as_float(v[2 * j]), cf, off));
                            const float e1 = exp2_approx(__fmaf_rn(__uint_as_float(v[2 * j + 1]), cf, off));
                            sum[0] += e0;
                            sum[1] += e1;
                            p[j] = pack_f16x2(e0, e1);
                        }
                        tmem_store16(s_at + 16 * c, p);
                    }
                    l += sum[0] + sum[1];
                    tmem_wait_stores();
                    tmem_fence_before();
                    mbar_arrive(p_full);
                }
                if (alive)
                    alive = wait(smem_u32(&bars.o_full[tile]), units_done & 1, &dead);
                ++units_done;
                if (alive) {
                    tmem_fence_after();
                    const bool begins = place.step == 0, ends = place.step + count == place.part.steps;
                    const bool whole_unit = begins && ends;
                    const float inv = l == 0.0f ? 0.0f : 1.0f / (l * vg);
                    float *slot = slots + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * slot_floats(kRows, D);
                    uint16_t *dst = a.out + (int64_t)(place.s.q0 + i) * a.ldo + (int64_t)qh * D;
                    float *part = slot + (tile * 128 + r) * D;
#pragma unroll 1
                    for (int c = 0; c < D / 32; ++c) {
                        uint32_t v[32];
                        tmem_load32(o_at + 32 * c, v);
                        loaded(v);
                        if (live && whole_unit) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float f[8];
#pragma unroll
                                for (int e = 0; e < 8; ++e)
                                    f[e] = __uint_as_float(v[8 * j + e]) * inv;
                                *reinterpret_cast<uint4 *>(dst + 32 * c + 8 * j) = pack8(f);
                            }
                        } else if (live) {
#pragma unroll
                            for (int j = 0; j < 8; ++j)
                                *reinterpret_cast<uint4 *>(part + 32 * c + 4 * j) = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
                        }
                        __syncwarp();
                    }
                    if (live && whole_unit && a.lse != nullptr)
                        a.lse[(int64_t)(place.s.q0 + i) * a.hq + qh] = l == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) * kLn2 + logf(l);
                    if (live && !whole_unit) {
                        slot[kRows * D + tile * 128 + r] = m;
                        slot[kRows * D + kRows + tile * 128 + r] = l;
                    }
                    if (tid == 0 && begins && !ends) {
                        record->last = (int32_t)((place.pos - place.step + place.part.steps - 1) / share_of);
                        record->q0 = (int32_t)place.s.q0;
                        record->head = place.head;
                        record->rows = place.part.rows;
                        record->row0 = place.part.row0;
                    }
                }
                tmem_fence_before();
            }
            step += count;
            advance(a, place, count);
        }
    } else if (warp < 8 + kMakers / 32) {
        // ---- K and V in fp16: a thread has 16 bytes of the codes of every 32nd (64th) key
        const int id = tid - kRows;
        constexpr int kRowChunks = D / 32;                   // 16-byte chunks of a key's codes
        constexpr int kStep = kMakers / kRowChunks;          // keys from one of a thread's chunks to the next
        constexpr int kPer = kKeys / kStep;
        const int key_at = id / kRowChunks, c = id % kRowChunks;
        const uint32_t codes_at = (key_at & 15) * L::kRow + c * 16, sf_at = L::kKsf + (key_at & 15) * (D / 16) + 2 * c;
        const uint32_t row_at = smem + (c >> 1) * S::kBlock + key_at * 128, half = (c & 1) * 4, turn = key_at & 7;
        const bool swap = (c & 2) != 0;
        uint32_t it = 0;
        uint4 kw[kPer], vw[kPer];
        uint32_t ksf[kPer], vsf[kPer];
        uint32_t in = 0;  // whether the chunks' keys lie in the cache
        int64_t n = place.end - place.pos;
        int ahead = 0;
        auto fetch = [&]() {  // the codes of the next step
            if (place.pos >= place.end)
                return;
            const int key0 = (place.part.first + place.step + ahead) * kKeys;
            const int32_t *table = a.table + (int64_t)place.b * a.max_pages;
            in = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const int key = key0 + i * kStep + key_at, tile_key = key & ~15;
                uint32_t at = 0;
                int32_t page = -1;
                if (tile_key < place.s.len) {
                    at = div_by((uint32_t)tile_key, a.cache.div_page);
                    page = table[at];
                }
                kw[i] = vw[i] = make_uint4(0, 0, 0, 0);
                ksf[i] = vsf[i] = 0;
                if (page >= 0 && page < a.cache.num_pages) {
                    in |= 1u << i;
                    const int tile = (tile_key - (int)at * a.cache.page_size) >> 4;
                    const uint8_t *src =
                        a.cache.pages + (((int64_t)page * a.cache.heads + place.head) * (a.cache.page_size >> 4) + tile) * L::kTile;
                    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(kw[i].x), "=r"(kw[i].y), "=r"(kw[i].z), "=r"(kw[i].w) : "l"(src + codes_at) : "memory");
                    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(vw[i].x), "=r"(vw[i].y), "=r"(vw[i].z), "=r"(vw[i].w) : "l"(src + L::kV + codes_at) : "memory");
                    asm volatile("ld.global.u16 %0, [%1];" : "=r"(ksf[i]) : "l"(src + sf_at) : "memory");
                    asm volatile("ld.global.u16 %0, [%1];" : "=r"(vsf[i]) : "l"(src + (L::kVsf - L::kKsf) + sf_at) : "memory");
                    if (key >= place.part.see_hi || key < place.part.see_lo || key >= place.s.len)
                        vsf[i] = 0;  // what a slot that nobody sees holds may be NaN
                }
            }
            if (++ahead == left_of(place)) {
                advance(a, place, ahead);
                ahead = 0;
            }
        };
        fetch();
        for (; n > 0; --n, ++it) {
            const int st = it & 1;
            const uint32_t phase = (it >> 1) & 1;
            if (it >= 2 && !wait(smem_u32(&bars.k_empty[st]), phase ^ 1, &dead))
                break;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (c == 0 && (key_at & 15) == 0)
                    seen[it & 3][(i * kStep + key_at) >> 4] = (uint8_t)(in >> i & 1);
                put_codes(row_at + S::kK + st * S::kMatrix + i * kStep * 128, half, turn, swap, kw[i], ksf[i]);
            }
            fence_async_proxy();
            mbar_arrive(smem_u32(&bars.k_full[st]));
            if (it >= 2 && !wait(smem_u32(&bars.v_empty[st]), phase ^ 1, &dead))
                break;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                put_codes(row_at + S::kV + st * S::kMatrix + i * kStep * 128, half, turn, swap, vw[i], vsf[i]);
            fence_async_proxy();
            mbar_arrive(smem_u32(&bars.v_full[st]));
            fetch();
        }
    } else {
        // ---- products
        constexpr uint32_t kIdS = idesc_f16(128, kKeys, false), kIdO = idesc_f16(128, D, true);
        const uint32_t s_full[2] = {smem_u32(&bars.s_full[0]), smem_u32(&bars.s_full[1])};
        // (the addresses go through an asm so that descriptors are not kept in registers
        // over the whole loop)
        auto scores = [&](int tile, int st) {  // S = q K^T
            uint32_t base = smem;
            asm volatile("" : "+r"(base));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k >> 2) * S::kBlock + (k & 3) * 32;
                    mma_f16(tmem + kSCol + tile * 128, desc_swizzled128(base + S::kQ + tile * S::kMatrix + off),
                            desc_swizzled128(base + S::kK + st * S::kMatrix + off), kIdS, k > 0);
                }
                mma_commit(s_full[tile]);
            }
            __syncwarp();
        };
        auto values = [&](int tile, int st, bool more) {  // O (+)= p V
            uint32_t base = smem;
            asm volatile("" : "+r"(base));
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kKeys / 16; ++k)
                    mma_f16_tmem(tmem + kOCol + tile * D, tmem + kSCol + tile * 128 + k * 8,
                                 desc_swizzled128_across(base + S::kV + st * S::kMatrix + k * 2048, S::kBlock), kIdO, more || k > 0);
            }
            __syncwarp();
        };
        auto commit = [&](uint64_t *bar) {
            if (elect_one())
                mma_commit(smem_u32(bar));
            __syncwarp();
        };
        uint32_t it = 0, units = 0, units1 = 0, p1 = 0;
        bool alive = true;
        while (alive && place.pos < place.end) {
            const int count = left_of(place);
            const bool two = place.part.rows > 128;
            const int st0 = it & 1;
            alive = wait(smem_u32(&bars.q_full[0]), units & 1, &dead) && wait(smem_u32(&bars.k_full[st0]), (it >> 1) & 1, &dead);
            if (!alive)
                break;
            tmem_fence_after();
            scores(0, st0);
            if (two) {
                if (!(alive = wait(smem_u32(&bars.q_full[1]), units1 & 1, &dead)))
                    break;
                tmem_fence_after();
                scores(1, st0);
            }
            commit(&bars.k_empty[st0]);
            for (int k = 0; k < count; ++k, ++it) {
                const int st = it & 1, next = st ^ 1;
                const bool last = k + 1 == count;
                if (!(alive = wait(smem_u32(&bars.v_full[st]), (it >> 1) & 1, &dead) && wait(smem_u32(&bars.p_full[0]), it & 1, &dead)))
                    break;
                tmem_fence_after();
                values(0, st, k > 0);
                if (last) {
                    commit(&bars.o_full[0]);
                } else {
                    if (!(alive = wait(smem_u32(&bars.k_full[next]), ((it + 1) >> 1) & 1, &dead)))
                        break;
                    tmem_fence_after();
                    scores(0, next);
                }
                if (two) {
                    if (!(alive = wait(smem_u32(&bars.p_full[1]), p1 & 1, &dead)))
                        break;
                    ++p1;
                    tmem_fence_after();
                    values(1, st, k > 0);
                }
                commit(&bars.v_empty[st]);
                if (two) {
                    if (last)
                        commit(&bars.o_full[1]);
                    else
                        scores(1, next);
                }
                if (!last)
                    commit(&bars.k_empty[next]);
            }
            ++units;
            units1 += two;
            if (alive)
                advance(a, place, count);
        }
        if (!alive) {  // what has been issued ends before its memory goes
            commit(&bars.last);
            const long long t0 = clock64();
            while (!mbar_try_wait(smem_u32(&bars.last), 0) && clock64() - t0 < kWaitCycles) {
            }
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    pdl_launch_dependents();
    if (warp == kThreads / 32 - 1) {
        tmem_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// Units over several blocks: a block has 8 rows of one, a warp each where the parts are
// few; else the warps share a row's parts.
template <int D>
__global__ void __launch_bounds__(256) attn_join_rows_kernel(const __grid_constant__ AttnArgs a, int blocks)
{
    constexpr int V = D / 32;  // floats of a lane
    __shared__ float acc_of[8][D];
    __shared__ float m_of[8], l_of[8];
    const int first = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_wait();
    pdl_launch_dependents();
    const Record rec = reinterpret_cast<const Record *>(a.partial)[first];
    const int row0 = blockIdx.y * 8;
    if (rec.last < 0 || row0 >= rec.rows)
        return;
    const float *slots = a.partial + (int64_t)blocks * (sizeof(Record) / 4);
    const int n = rec.last - first + 1;
    const float vg = *a.cache.v_scale;

    // parts i0 .. i1 of a row in order
    auto gather = [&](int row, int i0, int i1, float &m, float &l, float (&acc)[V]) {
        m = -INFINITY;
        l = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j)
            acc[j] = 0.0f;
#pragma unroll 4
        for (int i = i0; i < i1; ++i) {
            const float *slot = slots + ((int64_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * slot_floats(kRows, D);
            const float mi = slot[kRows * D + row], li = slot[kRows * D + kRows + row];
            float v[V];
#pragma unroll
            for (int j = 0; j < V; ++j)
                v[j] = slot[row * D + j * 32 + lane];
            const float top = fmaxf(m, mi);
            const float f0 = m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : exp2_approx(m - top);
            const float f1 = mi == -INFINITY ? (li == 0.0f ? 0.0f : 1.0f) : exp2_approx(mi - top);
            m = top;
            l = l * f0 + li * f1;
#pragma unroll
            for (int j = 0; j < V; ++j)
                acc[j] = acc[j] * f0 + v[j] * f1;
        }
    };
    auto write = [&](int row, float m, float l, const float (&acc)[V]) {
        const int64_t r = rec.row0 + row, i = r / a.group;
        const int64_t qh = (int64_t)rec.head * a.group + (r - i * a.group);
        const float inv = l == 0.0f ? 0.0f : 1.0f / (l * vg);
        uint16_t *dst = a.out + (rec.q0 + i) * a.ldo + qh * D;
#pragma unroll
        for (int j = 0; j < V; ++j)
            dst[j * 32 + lane] = (uint16_t)pack_bf16x2(acc[j] * inv, 0.0f);
        if (a.lse != nullptr && lane == 0)
            a.lse[(rec.q0 + i) * a.hq + qh] = l == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) * kLn2 + logf(l);
    };
    float m, l, acc[V];
    if (n <= 8) {
        if (row0 + warp < rec.rows) {
            gather(row0 + warp, 0, n, m, l, acc);
            write(row0 + warp, m, l, acc);
        }
        return;
    }
    const int per = (n + 7) / 8;
    for (int row = row0; row < row0 + 8 && row < rec.rows; ++row) {
        gather(row, min(n, warp * per), min(n, (warp + 1) * per), m, l, acc);
#pragma unroll
        for (int j = 0; j < V; ++j)
            acc_of[warp][j * 32 + lane] = acc[j];
        if (lane == 0) {
            m_of[warp] = m;
            l_of[warp] = l;
        }
        __syncthreads();
        if (warp == 0) {
            float top = -INFINITY, sum = 0.0f;
            for (int w = 0; w < 8; ++w)
                top = fmaxf(top, m_of[w]);
#pragma unroll
            for (int j = 0; j < V; ++j)
                acc[j] = 0.0f;
            for (int w = 0; w < 8; ++w) {
                const float f = m_of[w] == -INFINITY ? (l_of[w] == 0.0f ? 0.0f : 1.0f) : exp2_approx(m_of[w] - top);
                sum = fmaf(f, l_of[w], sum);
#pragma unroll
                for (int j = 0; j < V; ++j)
                    acc[j] = fmaf(f, acc_of[w][j * 32 + lane], acc[j]);
            }
            write(row, top, sum, acc);
        }
        __syncthreads();
    }
}

template <int D>
cudaError_t launch_prompt(const AttnArgs &a, bool pdl, cudaStream_t stream)
{
    static std::atomic<bool> ready[kMaxCachedDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    const bool cached = dev >= 0 && dev < kMaxCachedDevices;
    if (!cached || !ready[dev].load(std::memory_order_relaxed)) {
        err = cudaFuncSetAttribute(attn_prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Smem<D>::kBytes);
        if (err != cudaSuccess)
            return err;
        if (cached)
            ready[dev].store(true, std::memory_order_relaxed);
    }
    err = launch_kernel(attn_prompt_kernel<D>, dim3(kBlocks), dim3(kThreads), Smem<D>::kBytes, stream, pdl, a);
    if (err != cudaSuccess)
        return err;
    return launch_kernel(attn_join_rows_kernel<D>, dim3(kBlocks, kRows / 8), dim3(256), 0, stream, true, a, kBlocks);
}

}  // namespace

cudaError_t launch_attn_prompt(const AttnArgs &a, bool pdl, cudaStream_t stream)
{
    return a.D == 64 ? launch_prompt<64>(a, pdl, stream) : launch_prompt<128>(a, pdl, stream);
}

int64_t attn_prompt_workspace(int64_t D)
{
    return kBlocks * ((int64_t)sizeof(Record) + 2 * 4 * slot_floats(kRows, (int)D));
}

cudaError_t read_attn_stalled_waits(uint32_t *count)
{
    return cudaMemcpyFromSymbol(count, g_stalled_waits, sizeof(*count));
}

}  // namespace tsfn
