// Attention of many rows over the paged NVFP4 cache, on the fifth-generation tensor
// cores: prompts, and pieces of them after what the cache holds.
//
//   S = q K^T,   p_j = exp2(c S_j - m),   O = p V,   out = O / sum_j p_j / v_scale
//
// A block works on 256 rows, (query, head) pairs that share a key head, as two tiles of
// 128, and goes over the keys 128 at a time.  K and V are exact in fp16 (6 significant
// bits), as are rows of q scaled by a power of two; products are tcgen05.mma kind::f16
// with fp32 sums in tensor memory, where S, p (fp16, over S) and O of both tiles take
// all 512 columns (D = 128).  Roles of the block's warps:
//   - 4 for each tile: a thread has a row: its maximum and sum, exp2, p back to tensor
//     memory, and the rescaling of O, only when a score passes the maximum by 2^8;
//   - two copy the codes and scale factors of the next keys into shared memory, one K's and
//     one V's, which lie in one piece for each 16 of them (issuing the 16 copies of a step
//     takes a warp 1300 cycles);
//   - 4 turn them into fp16 tiles there, two stages deep, K and V alike: K is read along
//     d, V across it, so neither is transposed;
//   - one issues the products: while one tile's p is made, the other's run.
// Code that runs once a unit is kept in loops: straight through, its instructions come
// from memory for every unit anew, which took 13000 cycles of one.
//
// Work is split evenly as in attn_few.cu: all units' key tiles in one row, cut into
// equal shares; what a share leaves of a unit is joined by attn_join_rows_kernel.
// Every wait has a limit, after which the block records it, waits (with the limit again) for
// its copies and products in flight, and ends: what it has not written is not defined.
//
// A prompt of 8191 tokens, 64 heads over 8 of 128: 788 us, 1.39 PFLOP/s, 73 % of a large
// library product's rate, the tensor pipe 61 % busy; of 64 columns 675 us, where the products
// take 288 and the exponentials 226 (9.5 T/s measured).  A step of 128 keys takes 3000 cycles
// for 2048 of products.  Most of the rest is a tile's own chain: its scores' way to the
// registers and the maximum 450 cycles, p in two halves 1300, the second half's products and
// the next scores 850, and 400 until waits end and products are issued, with the other
// tile's products in between; then shared memory, which the products read 1500 cycles of a
// step, and makers and copies use 800.  Going to the next 256 rows takes 10000 cycles.
// Measured and not kept: p in one piece (the same) or in quarters (20 % slower, an arrival costs
// more than it hides), a warp for each tile's products (30 % slower, the tiles fall into
// step), polling waits (2 to 9 % slower), the code that goes to the next rows unrolled (2 %
// slower), a warp of its own that copies the next rows of q as soon as their place is free
// (25 % slower: its 64 passes a tile take longer than the rows' own warps do).
#include "attn_util.cuh"
#include "device_util.cuh"
#include "f32x2.cuh"
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
constexpr int kThreads = kRows + kMakers + 128;  // four warp groups; of the last three warps work
// Registers of a thread of each: the 128 that each is launched with, divided anew.
constexpr int kRowRegs = 192, kMakerRegs = 72, kOtherRegs = 56;
static_assert(kRows * kRowRegs + kMakers * kMakerRegs + 128 * kOtherRegs <= kThreads * 128, "");
// What going to a unit costs, in steps, when work is split.  us for 2, 3, 4, 5, 6:
//   D = 128, 8191 queries              868  808  773  782  792;  D = 64  700  666  675  681  691
//            5 x 1024 of 1024-6144     403  367  351  352  357           316  292  298  301  306
//            40 x 64 of 64-4096        181  161  150  151  150           129  119  122  126  127
constexpr int kSwitch = 4;
constexpr int kCopies = 13;          // the warps that copy codes: of K, of V
constexpr int kProducts = 12;        // the warp that issues them
constexpr int kRawSlots = 3;         // places for codes
constexpr int kSeqs = 256;          // sequences whose weights are summed at a time

// Shared memory: q of both tiles, two stages of K and of V, each in blocks of 64 d
// (128 bytes) by 128 rows under the 128-byte swizzle; three times the codes and scale
// factors of 128 keys, of K and of V in turn.  (A copy takes 2500 cycles to come: with one
// place each for K and V, the makers waited 1200 cycles of a step's 3700 for them.)
template <int D>
struct Smem {
    static constexpr int kBlock = 128 * 128;
    static constexpr int kMatrix = D / 64 * kBlock;
    static constexpr int kCodes = kKeys * (D / 2), kRaw = kCodes + kKeys * (D / 16);
    static constexpr int kQ = 0, kK = 2 * kMatrix, kV = 4 * kMatrix, kRaws = 6 * kMatrix, kBytes = kRaws + kRawSlots * kRaw + 1024;
};

struct Barriers {
    uint64_t q_full[2], s_full[2], o_full[2];  // of each tile
    uint64_t p_full[2][2];                     // of each half of a step's p, and tile
    uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];  // of each stage
    uint64_t raw_full[kRawSlots], raw_empty[kRawSlots];     // the codes
    uint64_t last;
};

#ifdef TSFN_RUN_OUT
// For the tests of the give-up path, which are built with it: the waits that begin
// this many cycles after their block's start run out at once.
__device__ long long g_run_out = 1LL << 62;

__device__ __forceinline__ long long &block_start()
{
    __shared__ long long start;
    return start;
}
#endif

__device__ __forceinline__ void give_up(volatile int *dead)
{
    *dead = 1;
    atomicAdd(&g_stalled_waits, 1u);
}

// A warp arrives, by one lane after all of them got here: 32 arrivals on one barrier take
// their turns.
__device__ __forceinline__ void warp_arrive(uint32_t bar)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0)
        mbar_arrive(bar);
}

// The whole warp waits for a phase; false where the block has given up.
__device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity, volatile int *dead)
{
#ifdef TSFN_RUN_OUT
    if (__shfl_sync(0xffffffffu, (int)(clock64() - block_start() >= g_run_out), 0) != 0) {
        if ((threadIdx.x & 31) == 0)
            give_up(dead);
        __syncwarp();
        return false;
    }
#endif
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

template <int N>
__device__ __forceinline__ void more_registers()
{
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers()
{
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
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
    const int i0 = (int)div_by((uint32_t)p.row0, a.div_group), i1 = (int)div_by((uint32_t)(p.row0 + p.rows - 1), a.div_group);
    int hi = a.causal ? (int)(s.len - s.n + i1 + 1) : s.len;
    int lo = a.window > 0 ? (int)(s.len - s.n + i0 + 1) - a.window : 0;
    p.see_hi = hi < 0 ? 0 : hi;
    p.see_lo = lo < 0 ? 0 : lo;
    p.first = p.see_lo / kKeys;
    const int steps = (p.see_hi + kKeys - 1) / kKeys - p.first;
    p.steps = steps > 1 ? steps : 1;
    return p;
}

// The steps of a sequence's row tiles for one key head and the ways to them, by a whole warp.
__device__ __forceinline__ int64_t steps_of(const AttnArgs &a, const Seq &s)
{
    int64_t sum = 0;
    for (int rt = threadIdx.x & 31; rt < s.parts; rt += 32)
        sum += part_of(a, s, rt).steps + kSwitch;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

// Where a share stands: the unit (sequence, key head, row tile) and how far into its
// kSwitch + steps.
struct Place {
    int64_t pos, end;  // of all units
    int b, head, rt, at;
    Seq s;
    Part part;
};

// What a share has of the unit that it stands at.
struct Segment {
    int step, count;  // steps; count may be 0
    int length;       // with the way there
};

__device__ __forceinline__ Segment segment_of(const Place &p)
{
    const int64_t here = p.part.steps + kSwitch - p.at, left = p.end - p.pos;
    Segment g;
    g.length = (int)(here < left ? here : left);
    g.step = max(p.at - kSwitch, 0);
    g.count = max(p.at + g.length - kSwitch, 0) - g.step;
    return g;
}

__device__ __forceinline__ void next_unit(const AttnArgs &a, Place &p, int length)
{
    p.pos += length;
    if (p.pos >= p.end)
        return;
    p.at = 0;
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

// To the next unit, `length` on (by one lane, for its warp).
__device__ __forceinline__ void advance(const AttnArgs &a, Place &place, int length)
{
    __syncwarp();
    if ((threadIdx.x & 31) == 0) {
        Place p = place;
        next_unit(a, p, length);
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
    p.b = p.head = p.rt = p.at = 0;
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
        const int steps = rt0 + lane < p.s.parts ? part_of(a, p.s, rt0 + lane).steps + kSwitch : 0;
        int scan = steps;  // (32 of at most 2^23)
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, scan, o);
            if (lane >= o)
                scan += up;
        }
        const unsigned past = __ballot_sync(0xffffffffu, scan > r);
        if (past != 0) {
            const int at = __ffs(past) - 1;
            p.rt = rt0 + at;
            p.at = (int)(r - (__shfl_sync(0xffffffffu, scan, at) - __shfl_sync(0xffffffffu, steps, at)));
            break;
        }
        r -= __shfl_sync(0xffffffffu, scan, 31);
    }
    p.part = part_of(a, p.s, p.rt);
    return p;
}

// The places for codes in turn: which one, and the parity of its use.
struct Turns {
    uint32_t slot = 0, phase = 0, uses = 0;
    __device__ __forceinline__ void next()
    {
        ++uses;
        if (++slot == kRawSlots) {
            slot = 0;
            phase ^= 1;
        }
    }
};

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// 16 bytes of codes (32 d of a key) as fp16 into half of a row of a swizzled block: `row`
// is the row's address, `first` the place of its first chunk.
__device__ __forceinline__ void put_codes(uint32_t row, uint32_t first, uint4 w, uint32_t sf2)
{
    const uint32_t sf = e4m3x2(sf2);
    const uint32_t s0 = __byte_perm(sf, 0, 0x1010), s1 = __byte_perm(sf, 0, 0x3232);
    const uint32_t word[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t s = i < 2 ? s0 : s1;
        st_shared(row + (first ^ (16 * i)), make_uint4(mul_f16x2(e2m1x2<0>(word[i]), s), mul_f16x2(e2m1x2<1>(word[i]), s),
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
    __shared__ uint32_t next_use[2];  // of the places for codes, that K's and V's copies did not get to
    __shared__ int64_t out_at[kRows];
    __shared__ int32_t lse_at[kRows];
    // of a step: whether its tiles of 16 keys lie in the cache; the keys that some row sees,
    // and whether there is no such step
    __shared__ uint8_t seen[4][8];
    __shared__ int32_t see_lo[4], see_hi[4], no_more[4];
    const uint32_t smem = (smem_u32(raw) + 1023) & ~1023u;
    const int tid = threadIdx.x, warp = tid >> 5;

    Record *const record = reinterpret_cast<Record *>(a.partial) + blockIdx.x;
    float *const slots = a.partial + (int64_t)gridDim.x * (sizeof(Record) / 4);

    if (warp == kProducts)
        tmem_alloc(smem_u32(&tmem_at), 512);
    if (tid == 0) {
        dead = 0;
#ifdef TSFN_RUN_OUT
        block_start() = clock64();
#endif
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&bars.q_full[i]), 4);
            mbar_init(smem_u32(&bars.s_full[i]), 1);
            mbar_init(smem_u32(&bars.p_full[0][i]), 4);
            mbar_init(smem_u32(&bars.p_full[1][i]), 4);
            mbar_init(smem_u32(&bars.o_full[i]), 1);
            mbar_init(smem_u32(&bars.k_full[i]), kMakers / 32);
            mbar_init(smem_u32(&bars.k_empty[i]), 1);
            mbar_init(smem_u32(&bars.v_full[i]), kMakers / 32);
            mbar_init(smem_u32(&bars.v_empty[i]), 1);
        }
        for (int i = 0; i < kRawSlots; ++i) {
            mbar_init(smem_u32(&bars.raw_full[i]), 1);
            mbar_init(smem_u32(&bars.raw_empty[i]), kMakers / 32);
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
        more_registers<kRowRegs>();
        const int tile = warp >> 2, r = tid & 127, lane = tid & 31;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // lane 32 (warp % 4) of tensor memory
        const uint32_t s_at = tmem + kSCol + tile * 128 + lanes, o_at = tmem + kOCol + tile * D + lanes;
        const uint32_t q_smem = smem + S::kQ + tile * S::kMatrix;
        const uint32_t s_full = smem_u32(&bars.s_full[tile]);
        const float vg = *a.cache.v_scale;
        const float k_scale = *a.cache.k_scale;
        uint32_t step = 0, done = 0, units_done = 0;  // steps of the block and of this tile
        bool alive = true;
        // the query and head of row `of` of the tile; whether there is one
        auto find = [&](int of, int &i, int &qh) -> bool {
            const int at = tile * 128 + of, row = place.part.row0 + at;
            const bool live = at < place.part.rows;
            i = live ? (int)div_by((uint32_t)row, a.div_group) : 0;
            qh = place.head * a.group + (live ? row - i * a.group : 0);
            return live;
        };
        // where the row is in q, in the unit that the place is at (in the weights' memory,
        // which is not used any more)
        static_assert(kRows <= kSeqs, "");
        int64_t *const q_from = weights;
        auto find_q = [&]() {
            int i, qh;
            const bool live = find(r, i, qh);
            q_from[tid] = live ? (int64_t)(place.s.q0 + i) * a.ldq + (int64_t)qh * D : -1;
            __syncwarp();
        };
        // 64 columns of the warp's rows of q, as they are: 8 neighbouring lanes a row
        auto copy_q = [&](int block) {
#pragma unroll 2
            for (int j = 0; j < 8; ++j) {
                const int row = (warp & 3) * 32 + j * 4 + lane / 8, c = lane & 7;
                const uint32_t dst = q_smem + block * S::kBlock + row * 128 + ((c ^ (row & 7)) * 16);
                const int64_t from = q_from[tile * 128 + row];
                if (from >= 0)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(a.q + from + block * 64 + c * 8) : "memory");
                else
                    st_shared(dst, make_uint4(0, 0, 0, 0));
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        // to the next unit in which this tile has rows and steps
        auto to_rows = [&]() {
            while (place.pos < place.end) {
                const Segment g = segment_of(place);
                if (g.count > 0 && place.part.rows > tile * 128)
                    break;
                step += g.count;
                advance(a, place, g.length);
            }
        };
        constexpr int kLast = D / 64 - 1;  // block of columns
        to_rows();
        if (place.pos < place.end) {
            find_q();
#pragma unroll 1
            for (int block = 0; block <= kLast; ++block)
                copy_q(block);
        }
        while (alive && place.pos < place.end) {
            const Segment segment = segment_of(place);
            const int count = segment.count;
            // this row of q, scaled by a power of two, as fp16
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            __syncwarp();
            float down;
            const uint32_t q_row = q_smem + r * 128;
            uint32_t top2[2] = {0, 0};  // pairs of bf16
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                const uint4 v = ld_shared(q_row + (c >> 3) * S::kBlock + (((c & 7) ^ (r & 7)) * 16));
                top2[0] = max_bf16x2(max_bf16x2(top2[0], v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
                top2[1] = max_bf16x2(max_bf16x2(top2[1], v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
            }
            top2[0] = max_bf16x2(top2[0], top2[1]);
            const float up = fp16_scale(fmaxf(__uint_as_float(top2[0] << 16), __uint_as_float(top2[0] & 0xFFFF0000u)), down);
#pragma unroll 4
            for (int c = 0; c < D / 8; ++c) {
                const uint32_t at = q_row + (c >> 3) * S::kBlock + (((c & 7) ^ (r & 7)) * 16);
                float f[8];
                unpack8(ld_shared(at), f);
                st_shared(at, make_uint4(pack_f16x2(f[0] * up, f[1] * up), pack_f16x2(f[2] * up, f[3] * up),
                                         pack_f16x2(f[4] * up, f[5] * up), pack_f16x2(f[6] * up, f[7] * up)));
            }
            fence_async_proxy();
            warp_arrive(smem_u32(&bars.q_full[tile]));
            // (a score is at most 2^8 times K's largest times D times its factor; where that may be
            // far, it is rounded on its own, in the pass that few steps have)
            const float all_of = score_factor(a, down, k_scale);
            const bool far = all_of >= kFar / (256.0f * 2688.0f * D), some_far = __any_sync(0xffffffffu, far);
            const float cf = far ? 1.0f : all_of, before = far ? all_of : 1.0f;
            int hi, lo;  // the keys that the row sees
            {
                int i, qh;
                const bool live = find(r, i, qh);
                hi = a.causal ? place.s.len - place.s.n + i + 1 : place.s.len;
                lo = a.window > 0 ? hi - a.window : 0;
                hi = live ? hi : place.s.len;  // (a row that there is not scores zeros)
                lo = live ? lo : 0;
            }
            const int hi_min = __reduce_min_sync(0xffffffffu, hi);
            const int lo_max = __reduce_max_sync(0xffffffffu, lo);
            const int key0 = (place.part.first + segment.step) * kKeys;

            float m = -INFINITY, l = 0.0f;  // the maximum less kLift, and the sum
            for (int k = 0; k < count; ++k, ++done) {
                const int key = key0 + k * kKeys;
                alive = wait(s_full, done & 1, &dead);
                if (!alive)
                    break;
                tmem_fence_after();
                const uint2 in = *reinterpret_cast<const uint2 *>(seen[(step + k) & 3]);
                if (some_far || !(key >= lo_max && key + kKeys <= hi_min && in.x == 0x01010101u && in.y == 0x01010101u)) {
                    // -inf for what the row does not see, a pass of its own: few steps have any
#pragma unroll 1
                    for (int c = 0; c < 4; ++c) {
                        uint32_t v[32];
                        tmem_load32(s_at + 32 * c, v);
                        // bit j: key 32 c + j of the step is seen
                        const int h = min(max(hi - key - 32 * c, 0), 32), w = min(max(lo - key - 32 * c, 0), 32);
                        const uint32_t ok = (c < 2 ? in.x : in.y) >> (16 * (c & 1));
                        const uint32_t sees = (uint32_t)((1ull << h) - (1ull << min(w, h))) &
                                              ((ok & 1 ? 0xFFFFu : 0u) | (ok & 0x100 ? 0xFFFF0000u : 0u));
                        loaded(v);
                        if (some_far) {
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                v[j] = __float_as_uint(__fmul_rn(__uint_as_float(v[j]), before));
                        }
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (!(sees >> j & 1))
                                v[j] = 0xFF800000u;
                        tmem_store32(s_at + 32 * c, v);
                    }
                    tmem_wait_stores();
                }
                // all of the row's scores at once: a load from tensor memory takes hundreds
                // of cycles while products run
                uint32_t v[4][32];
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    tmem_load32(s_at + 32 * c, v[c]);
                float top[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    loaded(v[c]);
                    top[c] = __uint_as_float(v[c][0]);
                }
#pragma unroll
                for (int j = 1; j < 31; j += 2)
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        top[c] = fmaxf(fmaxf(top[c], __uint_as_float(v[c][j])), __uint_as_float(v[c][j + 1]));
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    top[c] = fmaxf(top[c], __uint_as_float(v[c][31]));
                const float to = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * cf;
                if (__any_sync(0xffffffffu, k == 0 || to > m + (kLift + kSlack))) {  // the maximum follows
                    const float next = fmaxf(m, to - kLift), f = m == -INFINITY ? 0.0f : exp2_approx(m - next);
                    m = next;
                    l *= f;
#pragma unroll 1
                    for (int c = 0; c < (k > 0 ? D / 32 : 0); ++c) {
                        uint32_t o[32];
                        tmem_load32(o_at + 32 * c, o);
                        loaded(o);
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            o[j] = __float_as_uint(__uint_as_float(o[j]) * f);
                        tmem_store32(o_at + 32 * c, o);
                    }
                }
                // p, in two halves: the products with the first run beside the second
                const float off = m == -INFINITY ? 0.0f : -m;
                const uint64_t by = pair(cf, cf), plus = pair(off, off);
                uint64_t part[2] = {0, 0};
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    uint32_t p[32];
#pragma unroll
                    for (int j = 0; j < 32; ++j) {
                        const uint32_t *x = &v[2 * half + (j >> 4)][2 * (j & 15)];
                        float e0, e1;
                        unpair(fma2(pair(__uint_as_float(x[0]), __uint_as_float(x[1])), by, plus), e0, e1);
                        e0 = exp2_approx(e0);
                        e1 = exp2_approx(e1);
                        part[j & 1] = add2(part[j & 1], pair(e0, e1));
                        p[j] = pack_f16x2(e0, e1);
                    }
                    tmem_store32(s_at + 32 * half, p);
                    tmem_wait_stores();
                    tmem_fence_before();
                    warp_arrive(smem_u32(&bars.p_full[half][tile]));
                }
                float s0, s1;
                unpair(add2(part[0], part[1]), s0, s1);
                l += s0 + s1;
            }
            if (!alive)
                break;
            // where the rows go
            const bool begins = segment.step == 0, ends = segment.step + count == place.part.steps, whole_unit = begins && ends;
            float *const slot = slots + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * slot_floats(kRows, D);
            {
                int i, qh;
                const bool live = find(r, i, qh);
                out_at[tid] = live ? (int64_t)(place.s.q0 + i) * a.ldo + (int64_t)qh * D : -1;
                lse_at[tid] = (place.s.q0 + i) * a.hq + qh;
            }
            if (tid == 0 && begins && !ends) {
                record->last = (int32_t)((place.pos - place.at + place.part.steps + kSwitch - 1) / share_of);
                record->q0 = place.s.q0;
                record->head = place.head;
                record->rows = place.part.rows;
                record->row0 = place.part.row0;
            }
            step += count;
            advance(a, place, segment.length);
            to_rows();
            if (place.pos < place.end)
                find_q();
            alive = wait(smem_u32(&bars.o_full[tile]), units_done & 1, &dead);
            if (!alive)
                break;
            ++units_done;
            tmem_fence_after();
            // (no product reads q now: the next unit's takes its place, but for the last block,
            // which the rows go through on their way out)
            if (place.pos < place.end)
#pragma unroll 1
                for (int block = 0; block < kLast; ++block)
                    copy_q(block);
            // 128 bytes of a row at a time, written by 8 neighbouring lanes (lanes that write
            // their own rows took 4000 cycles)
            const float by = l == 0.0f ? 0.0f : 1.0f / l, of = 1.0f / vg;  // (their product may be out of range)
            const uint32_t way_out = q_smem + kLast * S::kBlock + (warp & 3) * 32 * 128;
#pragma unroll 1
            for (int at = 0; at < D; at += whole_unit ? 64 : 32) {
#pragma unroll 1
                for (int half = 0; half < (whole_unit ? 2 : 1); ++half) {
                    uint32_t v[32];
                    tmem_load32(o_at + at + 32 * half, v);
                    loaded(v);
                    if (whole_unit) {
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float f[8];
#pragma unroll
                            for (int e = 0; e < 8; e += 2)
                                unpair(mul2(mul2(pair(__uint_as_float(v[8 * k + e]), __uint_as_float(v[8 * k + e + 1])), twice(by)), twice(of)),
                                       f[e], f[e + 1]);
                            st_shared(way_out + lane * 128 + (((half * 4 + k) ^ (lane & 7)) * 16), pack8(f));
                        }
                    } else {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            st_shared(way_out + lane * 128 + ((k ^ (lane & 7)) * 16),
                                      make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]));
                    }
                }
                __syncwarp();
#pragma unroll 2
                for (int j = 0; j < 8; ++j) {
                    const int row = j * 4 + lane / 8, c = lane & 7, of = (warp * 32) + row;
                    const uint4 v = ld_shared(way_out + row * 128 + ((c ^ (row & 7)) * 16));
                    const int64_t to = out_at[of];
                    if (to >= 0) {
                        if (whole_unit)
                            *reinterpret_cast<uint4 *>(a.out + to + at + 8 * c) = v;
                        else
                            *reinterpret_cast<uint4 *>(slot + of * D + at + 4 * c) = v;
                    }
                }
                __syncwarp();
            }
            if (place.pos < place.end)
                copy_q(kLast);
            if (out_at[tid] >= 0) {
                if (!whole_unit) {
                    slot[kRows * D + tid] = m;
                    slot[kRows * D + kRows + tid] = l;
                } else if (a.lse != nullptr) {
                    a.lse[lse_at[tid]] = l == 0.0f ? -INFINITY : (m == -INFINITY ? 0.0f : m) * kLn2 + logf(l);
                }
            }
            tmem_fence_before();
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");  // (where the block gave up)
    } else if (warp < 8 + kMakers / 32) {
        // ---- K and V in fp16: a thread has 16 bytes of the codes of every 32nd (64th) key.
        // 8 neighbouring lanes read 128 bytes of codes and write 128 bytes without a conflict.
        fewer_registers<kMakerRegs>();
        const int lane = tid & 31, maker = warp - 8;
        constexpr int kStep = D == 128 ? 32 : 64;
        const int key_at = D == 128 ? maker * 8 + (lane & 7) : maker * 16 + (lane >> 1);
        const int c = D == 128 ? ((lane & 7) >> 1) ^ (lane >> 3) : lane & 1;
        const uint32_t codes_at = smem + S::kRaws + key_at * L::kRow + c * 16, sf_at = smem + S::kRaws + S::kCodes + key_at * (D / 16) + 2 * c;
        const uint32_t row_at = smem + (c >> 1) * S::kBlock + key_at * 128, first = ((c & 1) * 4 ^ (key_at & 7)) * 16;
        Turns raw;
        for (uint32_t it = 0;; ++it) {
            const int st = it & 1;
            const uint32_t phase = (it >> 1) & 1;
            if (!wait(smem_u32(&bars.raw_full[raw.slot]), raw.phase, &dead) || no_more[it & 3] != 0)
                break;
            if (it >= 2 && !wait(smem_u32(&bars.k_empty[st]), phase ^ 1, &dead))
                break;
#pragma unroll 2
            for (int key = 0; key < kKeys; key += kStep)
                put_codes(row_at + S::kK + st * S::kMatrix + key * 128, first, ld_shared(codes_at + raw.slot * S::kRaw + key * L::kRow),
                          ld_shared16(sf_at + raw.slot * S::kRaw + key * (D / 16)));
            fence_async_proxy();
            warp_arrive(smem_u32(&bars.raw_empty[raw.slot]));
            warp_arrive(smem_u32(&bars.k_full[st]));
            raw.next();
            if (!wait(smem_u32(&bars.raw_full[raw.slot]), raw.phase, &dead) ||
                (it >= 2 && !wait(smem_u32(&bars.v_empty[st]), phase ^ 1, &dead)))
                break;
            const int lo = see_lo[it & 3], hi = see_hi[it & 3];
#pragma unroll 2
            for (int key = 0; key < kKeys; key += kStep) {
                const int at = key + key_at;
                // (what a slot that nobody sees holds may be NaN)
                const bool use = at >= lo && at < hi && seen[it & 3][at >> 4] != 0;
                put_codes(row_at + S::kV + st * S::kMatrix + key * 128, first, ld_shared(codes_at + raw.slot * S::kRaw + key * L::kRow),
                          use ? ld_shared16(sf_at + raw.slot * S::kRaw + key * (D / 16)) : 0);
            }
            fence_async_proxy();
            warp_arrive(smem_u32(&bars.raw_empty[raw.slot]));
            warp_arrive(smem_u32(&bars.v_full[st]));
            raw.next();
        }
    } else if (warp == kCopies || warp == kCopies + 1) {
        // ---- codes and scale factors: lanes 0..7 have a step's tiles of 16 keys
        fewer_registers<kOtherRegs>();
        const int lane = tid & 31, which = warp - kCopies;  // K (0) or V (1)
        uint32_t it = 0;
        bool alive = true;
        Turns raw;
        if (which == 1)
            raw.next();
        auto room = [&]() -> bool { return raw.uses < kRawSlots || wait(smem_u32(&bars.raw_empty[raw.slot]), raw.phase ^ 1, &dead); };
        // a step's keys and tiles, looked up while the step before is copied
        int key0 = 0, see0 = 0, see1 = 0, ahead = 0;
        bool in = false;
        const uint8_t *src = nullptr;
        auto look_up = [&]() -> bool {
            Segment segment = segment_of(place);
            while (ahead == segment.count) {
                advance(a, place, segment.length);
                if (place.pos >= place.end)
                    return false;
                segment = segment_of(place);
                ahead = 0;
            }
            key0 = (place.part.first + segment.step + ahead++) * kKeys;
            see0 = place.part.see_lo - key0;
            see1 = min(place.part.see_hi, place.s.len) - key0;
            const int key = key0 + lane * 16;
            int32_t page = -1;
            uint32_t at = 0;
            if (lane < 8 && key < place.s.len) {
                at = div_by((uint32_t)key, a.cache.div_page);
                page = a.table[(int64_t)place.b * a.max_pages + at];
            }
            in = page >= 0 && page < a.cache.num_pages;
            src = a.cache.pages + (((int64_t)(in ? page : 0) * a.cache.heads + place.head) * (a.cache.page_size >> 4) +
                                   ((key - (int)at * a.cache.page_size) >> 4)) * L::kTile;
            return true;
        };
        for (bool more = place.pos < place.end && look_up(); more; ++it) {
            if (!(alive = room()))
                break;
            if (which == 0) {
                // (the products with the V four steps before have run, or V two before would not
                // have been made: nobody reads what is overwritten)
                if (lane < 8)
                    seen[it & 3][lane] = in;
                if (lane == 0) {
                    see_lo[it & 3] = see0;
                    see_hi[it & 3] = see1;
                    no_more[it & 3] = 0;
                }
            }
            const uint32_t bar = smem_u32(&bars.raw_full[raw.slot]), to = smem + S::kRaws + raw.slot * S::kRaw;
            const int tiles = __popc(__ballot_sync(0xffffffffu, in));
            __syncwarp();  // (the arrival hands on what the lanes wrote; a vote orders no memory)
            if (lane == 0)
                mbar_expect_tx(bar, tiles * S::kRaw / 8);
            __syncwarp();
            if (in) {
                bulk_load(to + lane * 16 * L::kRow, src + which * L::kV, 16 * L::kRow, bar);
                bulk_load(to + S::kCodes + lane * D, src + L::kKsf + which * D, D, bar);
            }
            __syncwarp();
            raw.next();
            raw.next();
            more = look_up();
        }
        if (which == 0 && alive && room()) {
            if (lane == 0)
                no_more[it & 3] = 1;
            warp_arrive(smem_u32(&bars.raw_full[raw.slot]));
            raw.uses += 2;
        }
        if (lane == 0)
            next_use[which] = raw.uses;
    } else {
        // ---- products, by one warp
        fewer_registers<kOtherRegs>();
        if (warp == kProducts) {
        const bool lead = elect_one();
        constexpr uint32_t kIdS = idesc_f16(128, kKeys, false), kIdO = idesc_f16(128, D, true);
        const uint32_t s_full[2] = {smem_u32(&bars.s_full[0]), smem_u32(&bars.s_full[1])};
        // (the addresses go through an asm so that descriptors are not kept in registers
        // over the whole loop; a product takes one lane chosen once and additions to low
        // words: choosing it and making descriptors anew for each took 886 us where this
        // takes 787)
        auto scores = [&](int tile, int st) {  // S = q K^T
            uint32_t base = smem;
            asm volatile("" : "+r"(base));
            const uint64_t q = desc_swizzled128(base + S::kQ + tile * S::kMatrix), k_at = desc_swizzled128(base + S::kK + st * S::kMatrix);
            if (lead) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = (k >> 2) * S::kBlock + (k & 3) * 32;
                    mma_f16(tmem + kSCol + tile * 128, desc_plus(q, off), desc_plus(k_at, off), kIdS, k > 0);
                }
                mma_commit(s_full[tile]);
            }
        };
        auto values = [&](int tile, int st, int half, bool more) {  // O (+)= p V, half of the keys
            uint32_t base = smem;
            asm volatile("" : "+r"(base));
            const uint64_t v = desc_swizzled128_across(base + S::kV + st * S::kMatrix + half * (kKeys / 32) * 2048, S::kBlock);
            const uint32_t p_at = tmem + kSCol + tile * 128 + half * (kKeys / 32) * 8;
            if (lead) {
#pragma unroll
                for (int k = 0; k < kKeys / 32; ++k)
                    mma_f16_tmem(tmem + kOCol + tile * D, p_at + k * 8, desc_plus(v, k * 2048), kIdO, k > 0 || more || half > 0);
            }
        };
        // both halves of a tile's step, as p comes
        auto both = [&](int tile, int st, uint32_t phase, bool more) -> bool {
            for (int half = 0; half < 2; ++half) {
                if (!wait(smem_u32(&bars.p_full[half][tile]), phase, &dead))
                    return false;
                tmem_fence_after();
                values(tile, st, half, more);
            }
            return true;
        };
        auto commit = [&](uint64_t *bar) {
            if (lead)
                mma_commit(smem_u32(bar));
        };
        uint32_t it = 0, units = 0, units1 = 0, p1 = 0;
        bool alive = true;
        while (alive && place.pos < place.end) {
            const Segment segment = segment_of(place);
            const int count = segment.count;
            if (count == 0) {
                advance(a, place, segment.length);
                continue;
            }
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
                if (!(alive = wait(smem_u32(&bars.v_full[st]), (it >> 1) & 1, &dead) && both(0, st, it & 1, k > 0)))
                    break;
                if (last) {
                    commit(&bars.o_full[0]);
                } else {
                    if (!(alive = wait(smem_u32(&bars.k_full[next]), ((it + 1) >> 1) & 1, &dead)))
                        break;
                    tmem_fence_after();
                    scores(0, next);
                }
                if (two) {
                    if (!(alive = both(1, st, p1 & 1, k > 0)))
                        break;
                    ++p1;
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
                advance(a, place, segment.length);
        }
        // what has been issued ends before its memory goes, whichever warp gave up
        commit(&bars.last);
        const long long t0 = clock64();
        while (!mbar_try_wait(smem_u32(&bars.last), 0) && clock64() - t0 < kWaitCycles) {
        }
        }
    }
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if (dead != 0) {  // the block gave up: copies in flight arrive before their memory goes
        const long long t0 = clock64();
        if (warp == kCopies) {  // the last use of each place
            for (int slot = 0; slot < kRawSlots; ++slot) {
                int last = -1;
                for (int back = 2; back <= 2 * kRawSlots; back += 2)
                    for (int which = 0; which < 2; ++which) {
                        const int use = (int)next_use[which] - back;
                        if (use > last && use % kRawSlots == slot)
                            last = use;
                    }
                while (last >= 0 && !mbar_try_wait(smem_u32(&bars.raw_full[slot]), last / kRawSlots & 1) && clock64() - t0 < kWaitCycles) {
                }
            }
        }
        __syncwarp();
    }
    pdl_launch_dependents();
    if (warp == kProducts) {
        tmem_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

// R neighbouring rows of a unit over n blocks, by a warp: their parts in order, UNROLL of
// them under way together.
template <int D, int R, int UNROLL>
__device__ __forceinline__ void join_rows(const AttnArgs &a, const Record &rec, const float *slots, int first, int n, int row0)
{
    constexpr int V = D / 32;  // floats of a lane
    const int lane = threadIdx.x & 31;
    float m[R], l[R], acc[R][V];
#pragma unroll
    for (int u = 0; u < R; ++u) {
        m[u] = -INFINITY;
        l[u] = 0.0f;
#pragma unroll
        for (int j = 0; j < V; ++j)
            acc[u][j] = 0.0f;
    }
#pragma unroll UNROLL
    for (int i = 0; i < n; ++i) {
        const float *slot = slots + ((int64_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * slot_floats(kRows, D);
#pragma unroll
        for (int u = 0; u < R; ++u) {
            const int row = min(row0 + u, rec.rows - 1);
            const float mi = slot[kRows * D + row], li = slot[kRows * D + kRows + row];
            float v[V];
            if constexpr (V == 4) {
                const float4 w = *reinterpret_cast<const float4 *>(slot + row * D + lane * V);
                v[0] = w.x;
                v[1] = w.y;
                v[2] = w.z;
                v[3] = w.w;
            } else {
                const float2 w = *reinterpret_cast<const float2 *>(slot + row * D + lane * V);
                v[0] = w.x;
                v[1] = w.y;
            }
            const float top = fmaxf(m[u], mi);
            const float f0 = m[u] == -INFINITY ? (l[u] == 0.0f ? 0.0f : 1.0f) : exp2_approx(m[u] - top);
            const float f1 = mi == -INFINITY ? (li == 0.0f ? 0.0f : 1.0f) : exp2_approx(mi - top);
            m[u] = top;
            l[u] = l[u] * f0 + li * f1;
#pragma unroll
            for (int j = 0; j < V; ++j)
                acc[u][j] = acc[u][j] * f0 + v[j] * f1;
        }
    }
    const float vg = *a.cache.v_scale;
#pragma unroll
    for (int u = 0; u < R; ++u) {
        if (row0 + u >= rec.rows)
            break;
        const uint32_t r = (uint32_t)rec.row0 + row0 + u, i = div_by(r, a.div_group);
        const int64_t qh = (int64_t)rec.head * a.group + (r - i * a.group), q = (int64_t)rec.q0 + i;
        const float by = l[u] == 0.0f ? 0.0f : 1.0f / l[u], of = 1.0f / vg;
        uint32_t *dst = reinterpret_cast<uint32_t *>(a.out + q * a.ldo + qh * D + lane * V);
#pragma unroll
        for (int j = 0; j < V / 2; ++j)
            dst[j] = pack_bf16x2(acc[u][2 * j] * by * of, acc[u][2 * j + 1] * by * of);
        if (a.lse != nullptr && lane == 0)
            a.lse[q * a.hq + qh] = l[u] == 0.0f ? -INFINITY : (m[u] == -INFINITY ? 0.0f : m[u]) * kLn2 + logf(l[u]);
    }
}

// Units over several blocks: where the parts are few, a warp has 4 rows of one (and the last
// blocks of a unit nothing); else a row.
template <int D>
__global__ void __launch_bounds__(256) attn_join_rows_kernel(const __grid_constant__ AttnArgs a, int blocks)
{
    const int first = blockIdx.x, warp = threadIdx.x >> 5;
    pdl_wait();
    pdl_launch_dependents();
    const Record rec = reinterpret_cast<const Record *>(a.partial)[first];
    const int n = rec.last - first + 1, each = n <= 8 ? 4 : 1, row0 = ((int)blockIdx.y * 8 + warp) * each;
    if (rec.last < 0 || row0 >= rec.rows)
        return;
    const float *slots = a.partial + (int64_t)blocks * (sizeof(Record) / 4);
    if (each == 4)
        join_rows<D, 4, 2>(a, rec, slots, first, n, row0);
    else
        join_rows<D, 1, 8>(a, rec, slots, first, n, row0);
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
        // (a division of more registers than a block is launched with would wait for ever)
        cudaFuncAttributes of;
        err = cudaFuncGetAttributes(&of, attn_prompt_kernel<D>);
        if (err == cudaSuccess && of.numRegs != 128)
            err = cudaErrorInvalidConfiguration;
        if (err != cudaSuccess)
            return err;
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
