// Per-head RMSNorm of queries and keys and rotation by position in one pass, with
// the keys and values written to the 4-bit cache; its gradient; the cache read back.
//
//   n = (x rsqrt(mean x^2 + eps)) w,   y = n turned by the position's angles
//
// Bound by memory.  A head's row of D elements lies on D/8 neighbouring lanes, 16
// bytes each (a power of two of lanes, those behind D/8 idle), so the sum of squares
// is a butterfly of a few steps and a lane's partner in the rotation is at a fixed
// distance.  Products and sums are rounded one by one, in the formula's order, and a key's
// squares are summed in an order that the header states: a key one step of bf16 away may be
// another code in the cache, or another scale factor of a block, so its bits are to be
// the same wherever it is computed.  (Weights multiplied into the cosines and sines, bf16
// partners exchanged and one fused addition took as long, with 3 in 100000 elements a step
// away.)  A group of lanes takes a run of heads of one token, the next ones' loads under way,
// and the position's cosines and sines and the weights are read once for them.
// 16383 tokens of 64 + 8 heads of 128, half of each turned: 100.7 us, 6.04 TB/s; with 8 heads of
// keys and values kept and read back, 16384 tokens: 141.7 us (the calls take 116 and 19).
// Equal shares of all heads to each warp with copies to shared memory, as the gradient has
// them, took 105 and 168: half as many instructions again a head.
#include "async_copy.cuh"
#include "device_util.cuh"
#include "f32x2.cuh"
#include "launch_attention.h"
#include "tcgen05.cuh"

namespace tsfn {

namespace {

// Blocks to an SM by their registers (16384 tokens, 64 + 8 heads of 128, with the cache
// written and read back: 142 us, and 150 with six blocks; without the cache, 64 columns
// turned: 100.7, and 101.8 with nine, which spill).
constexpr int kThreads = 128;
constexpr int rope_blocks_per_sm(bool pairs, bool cache) { return cache ? (pairs ? 6 : 7) : 8; }

// Coherent loads of what is used again (weights, tables, positions).
__device__ __forceinline__ uint4 ld_again(const void *p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p) : "memory");
    return v;
}

__device__ __forceinline__ void ld_angles(const float *p, int n4, float (&f)[8])
{
#pragma unroll
    for (int i = 0; i < 2; ++i)
        if (i < n4) {
            const uint4 v = ld_again(p + 4 * i);
            f[4 * i] = __uint_as_float(v.x);
            f[4 * i + 1] = __uint_as_float(v.y);
            f[4 * i + 2] = __uint_as_float(v.z);
            f[4 * i + 3] = __uint_as_float(v.w);
        }
}

// Sum over the lanes of a head's row, neighbours first, the same bits on each of them.
__device__ __forceinline__ float group_sum(float v, int lanes)
{
    for (int o = 1; o < lanes; o <<= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// A key's squares, from its row in shared memory, are summed in an order of their own: column j
// to sum j mod 32, then neighbouring sums together.  This lane's N of the 32 sums, from `row` on.
template <int N>
__device__ __forceinline__ float key_squares(uint32_t row, int columns)
{
    if constexpr (N > 2) {
        const float a = key_squares<N / 2>(row, columns);
        return a + key_squares<N / 2>(row + N, columns - N / 2);
    } else {
        float s0 = 0.0f, s1 = 0.0f;
#pragma unroll 1
        for (; columns > 0; columns -= 128, row += 256) {
            uint32_t v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                v[j] = 0;
                if (columns > 32 * j) {
                    if constexpr (N == 2)
                        asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v[j]) : "r"(row + 64 * j) : "memory");
                    else
                        v[j] = ld_shared16(row + 64 * j);
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float lo = __uint_as_float(v[j] << 16), hi = __uint_as_float(v[j] & 0xFFFF0000u);
                s0 = __fmaf_rn(lo, lo, s0);
                if constexpr (N == 2)
                    s1 = __fmaf_rn(hi, hi, s1);
            }
        }
        return s0 + s1;
    }
}

__device__ __forceinline__ float key_squares_of(uint32_t row, int c, int lanes, int D)
{
    const int at = c * (32 / lanes);
    row += 2 * at;
    switch (lanes) {
    case 2: return key_squares<16>(row, D - at);
    case 4: return key_squares<8>(row, D - at);
    case 8: return key_squares<4>(row, D - at);
    case 16: return key_squares<2>(row, D - at);
    default: return key_squares<1>(row, D - at);
    }
}

// What a lane does in the rotation: chunk c of 8 columns of a row.
struct Turn {
    bool in;        // the chunk is rotated
    bool first;     // halves: the pairs' first elements
    int partner;    // halves: lane with the pairs' other elements
    int angle;      // index of the chunk's first cosine
};

__device__ __forceinline__ Turn turn_of(int c, int lane, int rot, bool pairs)
{
    const int half = rot >> 4;  // chunks of half of the rotated columns
    Turn t;
    t.in = c < 2 * half;
    t.first = c < half;
    t.partner = !t.in || pairs ? lane : (t.first ? lane + half : lane - half);
    t.angle = pairs ? 4 * c : 8 * (t.first ? c : c - half);
    return t;
}

// What a lane's 8 columns are multiplied by, and their partners: the rotation is
//   y = x by + x' with,   x' the partner's columns (PAIRS: the neighbours exchanged),
// by = cos, with = -+ sin; 1 and -0 for columns that are not rotated, which with a partner of 0
// leave every x as it is; s = -1 turns back.
struct Factors {
    uint64_t by[4], with[4];
};

template <bool PAIRS>
__device__ __forceinline__ Factors factors_of(const float (&cs)[8], const float (&sn)[8], const Turn &t, float s)
{
    Factors f;
    const float k = t.first ? -s : s;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (PAIRS) {
            f.by[i] = t.in ? twice(cs[i]) : twice(1.0f);
            f.with[i] = t.in ? pair(-s * sn[i], s * sn[i]) : twice(-0.0f);
        } else {
            f.by[i] = t.in ? pair(cs[2 * i], cs[2 * i + 1]) : twice(1.0f);
            f.with[i] = t.in ? pair(k * sn[2 * i], k * sn[2 * i + 1]) : twice(-0.0f);
        }
    }
    return f;
}

// The partner's fp32 columns, where the rotation comes after the norm.
template <bool PAIRS>
__device__ __forceinline__ uint64_t partner2(uint64_t v, const Turn &t)
{
    float lo, hi;
    unpair(v, lo, hi);
    return PAIRS ? pair(hi, lo) : pair(__shfl_sync(0xffffffffu, lo, t.partner), __shfl_sync(0xffffffffu, hi, t.partner));
}

// The lane's partner columns in bf16: another lane's, or its own neighbours exchanged; zeros
// where nothing is rotated (0 times an infinity would not be 0).
template <bool PAIRS>
__device__ __forceinline__ void partners(const uint4 &x, const Turn &t, uint64_t (&o)[4])
{
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = PAIRS ? __funnelshift_l(w[i], w[i], 16) : __shfl_sync(0xffffffffu, w[i], t.partner);
        o[i] = widen2(t.in ? p : 0u);
    }
}

__device__ __forceinline__ uint4 pack2x4(const uint64_t (&v)[4])
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        unpair(v[i], lo, hi);
        w[i] = pack_bf16x2(lo, hi);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where the codes of K and V and the scale factors of a slot's head begin.
__device__ __forceinline__ uint8_t *cache_tile(const CacheArgs &c, int D, int64_t slot, int h, int *in_tile)
{
    const uint32_t page = div_by((uint32_t)slot, c.div_page);
    const int off = (int)((uint32_t)slot - page * (uint32_t)c.page_size);
    *in_tile = off & 15;
    const int64_t tile = ((int64_t)page * c.heads + h) * (c.page_size >> 4) + (off >> 4);
    return c.pages + tile * 18 * D;
}

// A row's chunk of 8 bf16 to NVFP4 (the arithmetic of ts_nvfp4_quantize), the two lanes
// of a block together: codes by each, the scale factor by the first.
__device__ __forceinline__ void put_chunk(const uint4 &v, float g, bool live, uint8_t *codes, uint8_t *sf, int c)
{
    float n[8];
    unpack8(v, n);
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        amax = fmaxf(amax, fabsf(n[e]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const uint32_t s = cvt_e4m3(__fmul_rn(g, div_const_rn(amax, 6.0f, kRcp6)));
    const float d = e4m3_value(s);
    uint32_t q = 0;
    if (d != 0.0f) {
        const float es = __fdiv_rn(g, d);
#pragma unroll
        for (int e = 0; e < 8; ++e)
            n[e] = __fmul_rn(n[e], es);
        q = cvt_e2m1x8(n);
    }
    if (live) {
        *reinterpret_cast<uint32_t *>(codes + 4 * c) = q;
        if ((c & 1) == 0)
            sf[c >> 1] = (uint8_t)s;
    }
}

// A group of lanes takes a run of heads of one token, two at a time with the next two's
// loads under way.  KEYS: of keys, and with a CACHE of values; else of queries.
template <bool PAIRS, bool KEYS, bool CACHE>
__device__ __forceinline__ void rope_run(const RopeArgs &a, uint32_t id, uint4 (&rows)[2][kThreads])
{
    const int lanes = 1 << a.lanes_log2;
    const int lane = threadIdx.x & 31, c = lane & (lanes - 1);
    const int64_t t = div_by(id, KEYS ? a.div_kv : a.div_q);
    const int run = (int)(id - t * (KEYS ? a.runs_kv : a.runs_q));
    const bool values = CACHE && run >= a.runs_k;
    const int h0 = (values ? run - a.runs_k : run) * a.run_heads;
    const int heads = KEYS ? a.hk : a.hq;
    const bool in_row = c < (a.D >> 3);

    bool live = t < a.T;
    const int32_t pos = live ? a.pos[t] : -1;
    const int n = live ? min(a.run_heads, heads - h0) : 0, most = __reduce_max_sync(0xffffffffu, n);
    const uint16_t *src = (values ? a.v + t * a.ldv : (KEYS ? a.k + t * a.ldk : a.q + t * a.ldq)) + (int64_t)h0 * a.D + c * 8;
    uint4 x[2], next[2];
    auto load = [&](int h, uint4 (&to)[2]) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            to[u] = make_uint4(0, 0, 0, 0);
            if (in_row && h + u < n)
                to[u] = ld_stream(src + (h + u) * a.D);
        }
    };
    load(0, next);
    live = live && pos >= 0 && pos < a.max_pos;
    uint8_t *codes = nullptr;  // of the head in the token's slot; how far on its scale factors are, 0: not kept
    int to_sf = 0;
    float g = 0.0f;
    if (CACHE && live) {
        const int64_t slot = a.slots[t];
        g = values ? *a.cache.v_scale : *a.cache.k_scale;
        if (slot >= 0 && slot < a.cache.slots) {
            int in_tile = 0;
            codes = cache_tile(a.cache, a.D, slot, h0, &in_tile) + (values ? 8 * a.D : 0) + in_tile * (a.D >> 1);
            to_sf = (values ? 9 : 16) * a.D - in_tile * (a.D >> 4) * 7;
        }
    }
    Turn turn = turn_of(c, lane, a.rot, PAIRS);
    turn.in = turn.in && !values;
    float cs[8] = {}, sn[8] = {};
    if (live && turn.in) {
        const float *p = a.table + (int64_t)pos * a.rot + turn.angle;
        ld_angles(p, PAIRS ? 1 : 2, cs);
        ld_angles(p + (a.rot >> 1), PAIRS ? 1 : 2, sn);
    }
    const uint16_t *w = KEYS ? a.kw : a.qw;
    const Factors f = factors_of<PAIRS>(cs, sn, turn, 1.0f);
    uint64_t wf[4] = {twice(1.0f), twice(1.0f), twice(1.0f), twice(1.0f)};
    if (w != nullptr && in_row && !values) {
        const uint4 v = ld_again(w + c * 8);
        const uint32_t ww[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            wf[i] = widen2(ww[i]);
    }
    pdl_launch_dependents();
    const float inv_d = 1.0f / (float)a.D;
    uint16_t *dst = (KEYS ? a.k_out + t * a.ldko : a.q_out + t * a.ldqo) + (int64_t)h0 * a.D + c * 8;
    const bool to_rows = live && in_row && !values && (!KEYS || a.k_out != nullptr);
    const uint32_t mine = smem_addr(&rows[0][threadIdx.x]);

    for (int h = 0; h < most; h += 2) {
        x[0] = next[0];
        x[1] = next[1];
        load(h + 2, next);
        float sq[2] = {};
        if (KEYS && w != nullptr) {
            st_shared(mine, x[0]);
            st_shared(mine + kThreads * 16, x[1]);
            __syncwarp();
#pragma unroll
            for (int u = 0; u < 2; ++u)
                sq[u] = key_squares_of(mine - c * 16 + u * kThreads * 16, c, lanes, a.D);
            __syncwarp();
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            if (u > 0 && h + u >= most)  // (few tokens: one head each)
                break;
            float r = 1.0f;
            if (w != nullptr)
                r = rsqrtf(__fadd_rn(__fmul_rn(group_sum(KEYS ? sq[u] : sumsq_bf16x8(x[u], 0.0f), lanes), inv_d), a.eps));
            uint64_t n2[4];
            const uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint64_t v = mul2(mul2(widen2(xw[i]), twice(r)), wf[i]);
                const uint64_t other = partner2<PAIRS>(v, turn), o = turn.in ? other : 0;  // (0 times an infinity would not be 0)
                n2[i] = add_products2(mul2(v, f.by[i]), mul2(o, f.with[i]), twice(a.one));
            }
            const uint4 y = values ? x[u] : pack2x4(n2);
            if (to_rows && h + u < n)
                st_v4(dst + (h + u) * a.D, y);
            if (CACHE) {
                put_chunk(y, g, in_row && h + u < n && to_sf != 0, codes, codes + to_sf, c);
                codes += (a.cache.page_size >> 4) * 18 * a.D;
            }
        }
    }
}

template <bool PAIRS, bool CACHE>
__global__ void __launch_bounds__(kThreads, rope_blocks_per_sm(PAIRS, CACHE)) rope_kernel(const __grid_constant__ RopeArgs a)
{
    __shared__ __align__(16) uint4 rows[2][kThreads];
    // every kv_every-th block has runs of keys (and values), up to kv_blocks of them, the others
    // runs of queries (100.7 and 141.7 us; every block with runs of both 116.8 and 149.5, keys and
    // values of all tokens first 102.6 and 156.9)
    const uint32_t turn = div_by(blockIdx.x, a.div_every);
    const bool keys = turn < (uint32_t)a.kv_blocks && turn * a.kv_every == blockIdx.x;
    const int64_t block = keys ? turn : blockIdx.x - min(turn + 1, (uint32_t)a.kv_blocks);
    const uint32_t id = (uint32_t)((block * kThreads + threadIdx.x) >> a.lanes_log2);  // (below 2^31: the calls' limit on T * heads)
    pdl_wait();
    if (keys)
        rope_run<PAIRS, true, CACHE>(a, id, rows);
    else
        rope_run<PAIRS, false, false>(a, id, rows);
}

// ---------------------------------------------------------------------------
// gradient
// ---------------------------------------------------------------------------

// dx = r (g - x r^2 mean(g x)), g = (dy turned back) w, dw = sum over rows of (dy turned
// back) x r.  The weights' gradient is summed by each lane over its share, then over the
// groups of a block in order, and over the blocks by grad_sum_kernel.
// Each group has an equal share of the heads of all tokens (whole runs of 16 left some with
// six where others had five: 92 us), one row of steps whose copies to shared memory are under
// way kGradAhead steps before; registers would not hold as many (106 us; two or five steps
// ahead are within 2 % of three).
// 8192 tokens of 64 + 8 heads of 128: 83.5 us with the sums, 5.46 TB/s.
constexpr int kGradThreads = 128, kGradAhead = 3, kGradStages = kGradAhead + 1;
constexpr int kGradRing = kGradStages * 2 * kGradThreads * 16;  // [stages][x, dy][threads]

template <bool PAIRS>
__global__ void __launch_bounds__(kGradThreads, 5) rope_grad_kernel(const __grid_constant__ RopeGradArgs a)
{
    extern __shared__ __align__(16) uint8_t smem[];
    float *const sums = reinterpret_cast<float *>(smem + kGradRing);  // [groups of lanes][lanes * 8]
    const int lanes = 1 << a.lanes_log2;
    const int lane = threadIdx.x & 31, c = lane & (lanes - 1);
    const int groups = kGradThreads >> a.lanes_log2, group = threadIdx.x >> a.lanes_log2;
    const bool in_row = c < (a.D >> 3);
    const Turn turn = turn_of(c, lane, a.rot, PAIRS);
    const float inv_d = 1.0f / (float)a.D;
    uint8_t *const ring = smem + threadIdx.x * 16;
    int put = 0, take = 0;  // stages, as offsets
    auto next = [](int at) { return at + 2 * kGradThreads * 16 == kGradRing ? 0 : at + 2 * kGradThreads * 16; };
    pdl_wait();
#pragma unroll 1
    for (int kind = 0; kind < 2; ++kind) {
        const uint16_t *w = a.w[kind];
        uint64_t wf[4] = {}, acc[4] = {};
        if (w != nullptr && in_row) {
            const uint4 v = ld_again(w + c * 8);
            const uint32_t ww[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                wf[i] = widen2(ww[i]);
        }
        // the group's steps: its share of all heads of all tokens, one after the other
        const int heads = a.heads[kind];
        const int64_t all = a.T * heads, sharers = (int64_t)gridDim.x * groups, sharer = (int64_t)blockIdx.x * groups + group;
        const int64_t begin = all * sharer / sharers;
        const int n = (int)(all * (sharer + 1) / sharers - begin), most = __reduce_max_sync(0xffffffffu, n);
        int64_t t = div_by((uint32_t)begin, a.div_heads[kind]);
        int h = (int)(begin - t * heads), in_h = h, in_step = 0;
        const uint16_t *xs = a.x[kind] + t * a.ldx[kind] + (int64_t)h * a.D + c * 8;
        const uint16_t *ds = a.dy[kind] + t * a.lddy[kind] + (int64_t)h * a.D + c * 8;
        uint16_t *to = a.dx[kind] + t * a.lddx[kind] + (int64_t)h * a.D + c * 8;
        auto issue = [&]() {
            if (in_row && in_step < n) {
                copy16(smem_addr(ring + put), xs);
                copy16(smem_addr(ring + put + kGradThreads * 16), ds);
            }
            copies_commit();
            put = next(put);
            xs += a.D;
            ds += a.D;
            ++in_step;
            if (++in_h == heads) {
                in_h = 0;
                xs += a.ldx[kind] - (int64_t)heads * a.D;
                ds += a.lddy[kind] - (int64_t)heads * a.D;
            }
        };
        put = take;  // (no copies are under way)
#pragma unroll 1
        for (int i = 0; i < kGradAhead; ++i)
            issue();
        auto pos_at = [&](int64_t token) { return n > 0 && token < a.T ? a.pos[token] : -1; };
        int32_t next_pos = pos_at(t);
        bool live = false;
        Factors f;
        for (int step = 0; step < most; ++step) {
            issue();
            if (step == 0 || h == heads) {  // a token's first
                if (step > 0) {
                    h = 0;
                    ++t;
                    to += a.lddx[kind] - (int64_t)heads * a.D;
                }
                const int32_t pos = next_pos;
                next_pos = pos_at(t + 1);
                live = pos >= 0 && pos < a.max_pos;
                float cs[8] = {}, sn[8] = {};
                if (live && turn.in) {
                    const float *p = a.table + (int64_t)pos * a.rot + turn.angle;
                    ld_angles(p, PAIRS ? 1 : 2, cs);
                    ld_angles(p + (a.rot >> 1), PAIRS ? 1 : 2, sn);
                }
                f = factors_of<PAIRS>(cs, sn, turn, -1.0f);
            }
            copies_wait<kGradAhead>();
            uint4 x = *reinterpret_cast<const uint4 *>(ring + take), d = *reinterpret_cast<const uint4 *>(ring + take + kGradThreads * 16);
            take = next(take);
            const bool on = live && in_row && step < n;
            if (!on)  // (what a row that is left out holds may be NaN)
                x = d = make_uint4(0, 0, 0, 0);
            const uint32_t dw[4] = {d.x, d.y, d.z, d.w}, xw[4] = {x.x, x.y, x.z, x.w};
            uint64_t o[4], v[4];
            partners<PAIRS>(d, turn, o);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                v[i] = fma2(widen2(dw[i]), f.by[i], mul2(o[i], f.with[i]));
            if (w != nullptr) {
                // both sums over the row side by side: x^2, and g x with g = d w
                uint64_t gx = 0;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    gx = fma2(mul2(v[i], wf[i]), widen2(xw[i]), gx);
                float s0, s1;
                unpair(gx, s0, s1);
                float sq = sumsq_bf16x8(x, 0.0f), dot = s0 + s1;
                for (int k = lanes >> 1; k > 0; k >>= 1) {
                    sq += __shfl_xor_sync(0xffffffffu, sq, k);
                    dot += __shfl_xor_sync(0xffffffffu, dot, k);
                }
                const float r = rsqrtf(__fmaf_rn(sq, inv_d, a.eps));
                const uint64_t by = twice(r), less = twice(-(dot * inv_d) * r * r);
                const uint64_t sum = twice(on ? r : 0.0f);  // (no 0 times the root of 1 / 0)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint64_t xf = widen2(xw[i]);
                    acc[i] = fma2(mul2(v[i], xf), sum, acc[i]);
                    v[i] = mul2(fma2(xf, less, mul2(v[i], wf[i])), by);
                }
            }
            if (on)
                st_v4(to, pack2x4(v));
            to += a.D;
            ++h;
        }
        if (w != nullptr) {
            if (kind == 1)
                __syncthreads();  // the queries' sums have been read
#pragma unroll
            for (int i = 0; i < 4; ++i)
                unpair(acc[i], sums[group * lanes * 8 + c * 8 + 2 * i], sums[group * lanes * 8 + c * 8 + 2 * i + 1]);
            __syncthreads();
            for (int j = threadIdx.x; j < a.D; j += kGradThreads) {
                float s = 0.0f;
                for (int i = 0; i < groups; ++i)
                    s += sums[i * lanes * 8 + j];
                a.partial[((int64_t)blockIdx.x * 2 + kind) * a.D + j] = s;
            }
        }
    }
    pdl_launch_dependents();
}

// dw[kind][j] = the blocks' sums in order: 128 lanes for each of 8 columns take every
// 128th block, so that all loads are under way together.
constexpr int kSumThreads = 1024, kSumColumns = 8;

__global__ void __launch_bounds__(kSumThreads) grad_sum_kernel(const float *partial, int blocks, int D, float *dqw, float *dkw)
{
    __shared__ float sums[kSumThreads / 32][kSumColumns];
    const int col = blockIdx.x * kSumColumns + threadIdx.x % kSumColumns, lane = threadIdx.x & 31;  // (D is a multiple of 16)
    pdl_wait();
    pdl_launch_dependents();
    float s = 0.0f;
#pragma unroll 6
    for (int i = threadIdx.x / kSumColumns; i < blocks; i += kSumThreads / kSumColumns)
        s += partial[(int64_t)i * 2 * D + col];
    auto over_lanes = [&]() {
#pragma unroll
        for (int o = kSumColumns; o < 32; o <<= 1)
            s += __shfl_xor_sync(0xffffffffu, s, o);
    };
    over_lanes();
    if (lane < kSumColumns)
        sums[threadIdx.x >> 5][lane] = s;
    __syncthreads();
    if (threadIdx.x >= 32)
        return;
    s = 0.0f;
    for (int i = lane / kSumColumns; i < kSumThreads / 32; i += 32 / kSumColumns)
        s += sums[i][lane % kSumColumns];
    over_lanes();
    if (lane < kSumColumns)
        (col < D ? dqw : dkw)[col < D ? col : col - D] = s;
}

// ---------------------------------------------------------------------------
// read back
// ---------------------------------------------------------------------------

// A group of lanes per token and head: K, then V.
__global__ void __launch_bounds__(kThreads) cache_read_kernel(const __grid_constant__ CacheReadArgs a, DivMagic div_heads)
{
    const int lanes = 1 << a.lanes_log2;
    const int c = threadIdx.x & (lanes - 1);
    const int64_t id = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> a.lanes_log2;
    const int64_t t = div_by((uint32_t)id, div_heads);
    const int h = (int)(id - t * a.cache.heads);
    pdl_wait();
    if (t < a.T && c < (a.D >> 3)) {
        const int64_t slot = a.slots[t];
        if (slot >= 0 && slot < a.cache.slots) {
            int in_tile;
            const uint8_t *tile = cache_tile(a.cache, a.D, slot, h, &in_tile);
            uint32_t codes[2], sf[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                codes[i] = *reinterpret_cast<const volatile uint32_t *>(tile + i * 8 * a.D + in_tile * (a.D >> 1) + 4 * c);
                sf[i] = *reinterpret_cast<const volatile uint8_t *>(tile + (16 + i) * a.D + in_tile * (a.D >> 4) + (c >> 1));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (a.out[i] == nullptr)
                    continue;
                const float s = __fdiv_rn(e4m3_value(sf[i]), i == 0 ? *a.cache.k_scale : *a.cache.v_scale);
                // (E2M1 is exact in fp16, and that in fp32)
                uint32_t two[4];
                asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t"
                    "cvt.rn.f16x2.e2m1x2 %1, b;\n\tcvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
                    : "=r"(two[0]), "=r"(two[1]), "=r"(two[2]), "=r"(two[3]) : "r"(codes[i]));
                float f[8];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
                        : "=f"(f[2 * e]), "=f"(f[2 * e + 1]) : "r"(two[e]));
                    f[2 * e] = __fmul_rn(f[2 * e], s);
                    f[2 * e + 1] = __fmul_rn(f[2 * e + 1], s);
                }
                st_v4(a.out[i] + t * a.ld[i] + (int64_t)h * a.D + c * 8, pack8(f));
            }
        }
    }
    pdl_launch_dependents();
}

// Heads of a run: as many as leave every SM 64 groups of lanes with one each, so that
// the factors are made once for several; at most 16.  (The bits do not depend on it.)
int run_heads(int64_t rows, int lanes_log2)
{
    const int64_t per = (rows << lanes_log2) / (152 * 1024);
    return per < 1 ? 1 : (per > 16 ? 16 : (int)per);
}

template <bool PAIRS>
cudaError_t launch_rope_as(const RopeArgs &a, bool pdl, cudaStream_t stream)
{
    const dim3 grid((unsigned)(a.kv_blocks + a.q_blocks)), block(kThreads);
    return a.keep ? launch_kernel(rope_kernel<PAIRS, true>, grid, block, 0, stream, pdl, a)
                  : launch_kernel(rope_kernel<PAIRS, false>, grid, block, 0, stream, pdl, a);
}

}  // namespace

cudaError_t launch_rope(const RopeArgs &args, bool pdl, cudaStream_t stream)
{
    RopeArgs a = args;
    a.run_heads = run_heads(a.T * (a.hq + 2 * a.hk), a.lanes_log2);
    a.runs_q = (a.hq + a.run_heads - 1) / a.run_heads;
    a.runs_k = (a.hk + a.run_heads - 1) / a.run_heads;
    a.runs_kv = (a.keep ? 2 : 1) * a.runs_k;
    const auto blocks = [&](int64_t runs) { return (int)(((a.T * runs << a.lanes_log2) + kThreads - 1) / kThreads); };
    a.kv_blocks = blocks(a.runs_kv);
    a.q_blocks = blocks(a.runs_q);
    a.kv_every = (a.kv_blocks + a.q_blocks) / a.kv_blocks;
    a.div_every = div_magic((uint32_t)a.kv_every);
    a.div_q = div_magic((uint32_t)a.runs_q);
    a.div_kv = div_magic((uint32_t)a.runs_kv);
    a.one = 1.0f;
    return a.pairs ? launch_rope_as<true>(a, pdl, stream) : launch_rope_as<false>(a, pdl, stream);
}

cudaError_t launch_rope_grad(const RopeGradArgs &args, bool pdl, cudaStream_t stream)
{
    RopeGradArgs a = args;
    for (int i = 0; i < 2; ++i)
        a.div_heads[i] = div_magic((uint32_t)a.heads[i]);
    const int64_t most = a.heads[0] > a.heads[1] ? a.heads[0] : a.heads[1];
    const int groups = kGradThreads >> a.lanes_log2;
    const int64_t want = (a.T * most + groups - 1) / groups;
    const int blocks = (int)(want < 1 ? 1 : (want > kGradBlocks ? kGradBlocks : want));
    const size_t smem = kGradRing + kGradThreads * 8 * sizeof(float);
    const cudaError_t err = a.pairs ? launch_kernel(rope_grad_kernel<true>, dim3((unsigned)blocks), dim3(kGradThreads), smem, stream, pdl, a)
                                    : launch_kernel(rope_grad_kernel<false>, dim3((unsigned)blocks), dim3(kGradThreads), smem, stream, pdl, a);
    if (err != cudaSuccess || a.w[0] == nullptr)
        return err;
    return launch_kernel(grad_sum_kernel, dim3((unsigned)(2 * a.D / kSumColumns)), dim3(kSumThreads), 0, stream, true,
                         (const float *)a.partial, blocks, a.D, a.dw[0], a.dw[1]);
}

cudaError_t launch_cache_read(const CacheReadArgs &a, bool pdl, cudaStream_t stream)
{
    const int64_t blocks = (((a.T * a.cache.heads) << a.lanes_log2) + kThreads - 1) / kThreads;
    return launch_kernel(cache_read_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, stream, pdl, a,
                         div_magic((uint32_t)a.cache.heads));
}

}  // namespace tsfn
