// Attention of few rows at a time over the paged NVFP4 cache: decoded tokens, and a
// few queries of a sequence.
//
//   out = sum_j p_j V[j] / sum_j p_j,   p_j = exp2(c q.K[j] - m)      c = scale log2(e) / k_scale
//
// Bound by the cache's bytes, 9/8 D a key and head.  The rows of a unit are up to
// 8 NT of the (query, head) pairs that share a key head, so a key is read once for
// them.  E2M1 times E4M3 has at most 6 significant bits: K and V are exact in fp16, and
// a row of q is too after scaling by a power of two, so fp16 products with fp32 sums
// lose nothing.  The keys are the 16 rows of mma.m16n8k16 (the rows of q its 8 columns):
//   S^T = K q^T     a lane's part of a row of K is 16 contiguous bytes of codes: which
//                   d a product's k stands for is free as long as q follows
//   O^T = V^T p^T   a lane holds D/8 contiguous d of 4 keys; two keys' nibbles are
//                   joined in one byte before the conversion, which then gives pairs
//                   along the keys, as the product wants them; p^T by movmatrix
// (mma.sync, not tcgen05: 8 rows would leave 15/16 of a tcgen05 tile empty, and the
// tensor pipe is a third busy here.)
//
// A warp takes every 8th tile of 16 keys of its block's share, with copies of the next tiles
// under way, with a running maximum and sum of its own.  The maximum follows only when a
// score passes it by 2^8, so most tiles take one vote instead of a reduction and a
// rescaling; p <= 256 is far from fp16's end.
//
// Work is split evenly: all units' tiles in one row, cut into equal shares, so that
// sequences of any lengths keep every block busy.  A unit inside a share is written
// at once; of a unit over several, each block leaves its part in the workspace and
// attn_join_kernel joins them in order.
#include "attn_util.cuh"
#include "device_util.cuh"
#include "launch_attention.h"

namespace tsfn {

namespace {

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// Blocks of an SM and copies of tiles in flight: 16 rows take the registers of a whole SM.
constexpr int blocks_per_sm(int nt) { return nt == 1 ? 2 : 1; }
constexpr int blocks_of(int nt) { return 152 * blocks_per_sm(nt); }
constexpr int stages_of(int nt) { return nt == 1 ? 4 : 6; }
constexpr int kShare = 8;     // tiles of a share, at least
__device__ __forceinline__ uint32_t smem_addr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }

__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
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

// Where 16-byte chunk i of a tile goes in shared memory.  Keys t and t + 4 of each 8
// become neighbours, so that 8 lanes' reads of K fill 128 bytes; V's chunks are
// exchanged between pairs of keys, so that half a warp's reads fill 128 bytes (D = 128).
template <int D>
__device__ __forceinline__ uint32_t chunk_place(int i)
{
    using L = Layout<D>;
    constexpr int per = L::kRow / 16;
    if (i < 16 * per) {
        const int key = i / per;
        return ((key & 8) + 2 * (key & 3) + ((key >> 2) & 1)) * L::kRow + (i % per) * 16;
    }
    if (i < 32 * per) {
        const int v = i - 16 * per, key = v / per;
        return L::kV + key * L::kRow + ((v % per) ^ (D == 128 ? key & 2 : 0)) * 16;
    }
    return i * 16;
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, blocks_per_sm(NT)) attn_few_kernel(const __grid_constant__ AttnArgs a)
{
    using L = Layout<D>;
    constexpr int NR = 8 * NT, kStages = stages_of(NT);
    constexpr int KS = D / 16;  // products of S per tile and 8 rows, and of O
    extern __shared__ __align__(16) uint8_t smem[];
    uint8_t *ring = smem;  // [warps][stages][tile], and after a segment the warps' O [warps][NR][D]
    float *ms = reinterpret_cast<float *>(smem + kWarps * kStages * L::kTile);  // [warps][NR]
    float *ls = ms + kWarps * NR;
    __shared__ int64_t sums[kThreads];
    __shared__ int64_t warp_sums[kWarps];
    static_assert(kWarps * NR * D * 4 <= kWarps * kStages * L::kTile, "");

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    float *const slots = a.partial + (int64_t)gridDim.x * (sizeof(Record) / 4);
    Record *const record = reinterpret_cast<Record *>(a.partial) + blockIdx.x;
    pdl_wait();

    // every block's share of the tiles: thread i sums the sequences i * per ..
    const int per = (a.B + kThreads - 1) / kThreads;
    int64_t sum = 0;
    for (int b = tid * per; b < a.B && b < (tid + 1) * per; ++b)
        sum += weight(a, sequence<NR>(a, b));
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
    const int64_t end = pos + share < total ? pos + share : total;
    if (tid == 0)
        record->last = -1;
    if (pos >= end) {
        pdl_launch_dependents();
        return;
    }
    int b;
    int64_t base;  // tiles before sequence b
    {
        int lo = 0, hi = kThreads - 1;  // the first thread whose sum passes pos
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (sums[mid] > pos)
                hi = mid;
            else
                lo = mid + 1;
        }
        b = lo * per;
        base = lo > 0 ? sums[lo - 1] : 0;
    }
    Seq s = sequence<NR>(a, b);
    const float kg = *a.cache.k_scale, vg = *a.cache.v_scale;
    const float c0 = a.scale * kLog2e / kg;

    const uint32_t my_ring = smem_addr(ring) + warp * kStages * L::kTile;

    while (pos < end) {
        while (pos >= base + weight(a, s)) {
            base += weight(a, s);
            s = sequence<NR>(a, ++b);
        }
        const int64_t unit = (pos - base) / s.tiles;
        const int tile0 = (int)(pos - base - unit * s.tiles);
        const int count = (int)(s.tiles - tile0 < end - pos ? s.tiles - tile0 : end - pos);
        const int head = (int)(unit / s.parts);
        const int64_t row0 = (unit - (int64_t)head * s.parts) * NR;
        const int rows = (int)(s.n * a.group - row0 < NR ? s.n * a.group - row0 : NR);

        // the rows of q as fp16, each scaled by a power of two; column factors and limits
        uint32_t qf[NT][KS][2];
        float cf[NT][2];
        int hi[NT][2], lo[NT][2];
        int hi_min = 0x7fffffff, hi_max = 0, lo_min = 0x7fffffff, lo_max = 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int col = nt * 8 + g;
            const bool live = col < rows;
            const int64_t r = row0 + col;
            const int64_t i = live ? r / a.group : 0;
            const int qh = live ? (int)(r - i * a.group) : 0;
            const uint16_t *src = a.q + (s.q0 + i) * a.ldq + ((int64_t)head * a.group + qh) * D + t * (D / 4);
            uint4 v[KS / 2];
#pragma unroll
            for (int j = 0; j < KS / 2; ++j) {
                v[j] = make_uint4(0, 0, 0, 0);
                if (live)
                    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
                                 : "=r"(v[j].x), "=r"(v[j].y), "=r"(v[j].z), "=r"(v[j].w) : "l"(src + j * 8) : "memory");
            }
            float f[KS / 2][8], amax = 0.0f;
#pragma unroll
            for (int j = 0; j < KS / 2; ++j) {
                unpack8(v[j], f[j]);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    amax = fmaxf(amax, fabsf(f[j][e]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            float down;
            const float up = fp16_scale(amax, down);
#pragma unroll
            for (int j = 0; j < KS / 2; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    qf[nt][2 * j + e / 2][e & 1] = pack_f16x2(f[j][2 * e] * up, f[j][2 * e + 1] * up);
            // limits of this column's keys
            int h = a.causal ? (int)(s.len - s.n + i + 1) : s.len;  // (may be <= 0)
            int l = a.window > 0 ? h - a.window : 0;
            if (!live) {
                h = 0x7fffffff;
                l = 0;
            }
            l = l < 0 ? 0 : l;
            const float c = c0 * down;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int from = (2 * t + j) * 4;
                cf[nt][j] = __shfl_sync(0xffffffffu, c, from);
                hi[nt][j] = __shfl_sync(0xffffffffu, h, from);
                lo[nt][j] = __shfl_sync(0xffffffffu, l, from);
            }
            hi_min = min(hi_min, h);
            lo_max = max(lo_max, l);
            if (live) {
                hi_max = max(hi_max, h);
                lo_min = min(lo_min, l);
            }
        }
        hi_min = __reduce_min_sync(0xffffffffu, hi_min);
        lo_max = __reduce_max_sync(0xffffffffu, lo_max);
        hi_max = __reduce_max_sync(0xffffffffu, hi_max);
        lo_min = __reduce_min_sync(0xffffffffu, lo_min);
        hi_min = min(hi_min, s.len);

        float o[NT][KS][4];
        float m[NT][2], l[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[nt][i][j] = 0.0f;
            m[nt][0] = m[nt][1] = -INFINITY;
            l[nt][0] = l[nt][1] = 0.0f;
        }

        const int mine = count > warp ? (count - warp + kWarps - 1) / kWarps : 0;  // tiles of this warp
        const int64_t table = (int64_t)b * a.max_pages;
        const int key0 = (s.first + tile0 + warp) * 16;
        uint32_t ok = 0;  // stages whose tile lies in the cache
        auto page_of = [&](int k) -> int32_t {
            const int key = key0 + k * kWarps * 16;
            return k < mine && key < s.len ? a.table[table + div_by((uint32_t)key, a.cache.div_page)] : -1;
        };
        int32_t next_page = page_of(0);
        auto issue = [&](int k) {
            const int32_t page = next_page;
            next_page = page_of(k + 1);
            const int stage = k % kStages;
            ok &= ~(1u << stage);
            if (k < mine && page >= 0 && page < a.cache.num_pages) {
                ok |= 1u << stage;
                const int key = key0 + k * kWarps * 16;
                const int in_page = key - (int)div_by((uint32_t)key, a.cache.div_page) * a.cache.page_size;
                const uint8_t *src =
                    a.cache.pages + (((int64_t)page * a.cache.heads + head) * (a.cache.page_size >> 4) + (in_page >> 4)) * L::kTile;
                const uint32_t dst = my_ring + stage * L::kTile;
#pragma unroll
                for (int i = 0; i < (L::kChunks + 31) / 32; ++i)
                    if (i * 32 + lane < L::kChunks)
                        copy16(dst + chunk_place<D>(i * 32 + lane), src + (i * 32 + lane) * 16);
            }
            copies_commit();
        };
        for (int k = 0; k < kStages - 1; ++k)
            issue(k);
        for (int k = 0; k < mine; ++k) {
            __syncwarp();  // the stage that is filled next has been read
            issue(k + kStages - 1);
            copies_wait<kStages - 1>();
            __syncwarp();
            const int stage = k % kStages;
            const int key = key0 + k * kWarps * 16;
            if (!(ok >> stage & 1))
                continue;
            const uint8_t *tile = ring + (warp * kStages + stage) * L::kTile;

            // S^T: rows g and g + 8 are keys k0 and k0 + 8
            const int k0 = (g >> 1) + 4 * (g & 1);
            float sc[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sc[nt][j] = 0.0f;
            {
                uint32_t w[2][KS / 2], sf[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const uint8_t *p = tile + (g + 8 * r) * L::kRow + t * (L::kRow / 4);
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
                        mma(sc[nt], a00, a10, a01, a11, qf[nt][2 * i][0], qf[nt][2 * i][1]);
                        mma(sc[nt], a02, a12, a03, a13, qf[nt][2 * i + 1][0], qf[nt][2 * i + 1][1]);
                    }
                }
            }
            // scores in units of log2; -inf where a row does not see the key
            const bool whole = key >= lo_max && key + 16 <= hi_min;
            bool grow = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float v = sc[nt][j] * cf[nt][j & 1];
                    if (!whole) {
                        const int at = key + k0 + 8 * (j >> 1);
                        v = at < hi[nt][j & 1] && at >= lo[nt][j & 1] && at < s.len ? v : -INFINITY;
                    }
                    sc[nt][j] = v;
                    grow = grow || v > m[nt][j & 1] + kSlack;
                }
            if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float f[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        float top = fmaxf(sc[nt][j], sc[nt][j + 2]);
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        top = fmaxf(top, m[nt][j]);
                        f[j] = m[nt][j] == -INFINITY ? 0.0f : exp2_approx(m[nt][j] - top);
                        m[nt][j] = top;
                        l[nt][j] *= f[j];
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
                    const float top = m[nt][j & 1];
                    p[j] = exp2_approx(sc[nt][j] - (top == -INFINITY ? 0.0f : top));
                    l[nt][j & 1] += p[j];
                }
                pt[nt][0] = transpose8(pack_f16x2(p[0], p[1]));
                pt[nt][1] = transpose8(pack_f16x2(p[2], p[3]));
            }
            // O^T: a lane's keys are t, t + 4, t + 8, t + 12, its d those from g D/8 on
            uint32_t vs[2];
            {
                const uint8_t *ps = tile + L::kVsf + t * (D / 16) + (D == 128 ? g : g >> 1);
                uint32_t b4[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    b4[j] = ps[4 * j * (D / 16)];
                    const int at = key + t + 4 * j;
                    if (!whole && !(at < hi_max && at >= lo_min && at < s.len))
                        b4[j] = 0;  // what a slot that nobody sees holds may be NaN
                }
                vs[0] = e4m3x2(b4[0] | b4[1] << 8);
                vs[1] = e4m3x2(b4[2] | b4[3] << 8);
            }
#pragma unroll
            for (int h2 = 0; h2 < D / 64; ++h2) {  // words of a lane's codes
                uint32_t w[4];
                if constexpr (D == 64) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        w[j] = *reinterpret_cast<const uint32_t *>(tile + L::kV + (t + 4 * j) * L::kRow + g * 4);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int kk = t + 4 * j;
                        w[j] = *reinterpret_cast<const uint32_t *>(tile + L::kV + kk * L::kRow + (((g >> 1) ^ (kk & 2)) * 16) + (g & 1) * 8 + h2 * 4);
                    }
                }
                uint32_t e0[4], o0[4], e1[4], o1[4];
                join_keys(w[0], w[1], vs[0], e0, o0);
                join_keys(w[2], w[3], vs[1], e1, o1);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
                        mma(o[nt][h2 * 4 + i], e0[i], o0[i], e1[i], o1[i], pt[nt][0], pt[nt][1]);
            }
        }
        copies_wait<0>();
        __syncthreads();  // the ring is free

        // the warps' parts: (m, l, O) of each row
        float *parts = reinterpret_cast<float *>(ring) + warp * NR * D;
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
                    ms[warp * NR + col] = m[nt][j];
                    ls[warp * NR + col] = v;
                }
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    *reinterpret_cast<float2 *>(parts + col * D + g * (D / 8) + 2 * i) = make_float2(o[nt][i][j], o[nt][i][j + 2]);
            }
        }
        __syncthreads();
        const bool begins = tile0 == 0, ends = tile0 + count == s.tiles;
        if (begins && !ends && tid == 0) {
            record->last = (int32_t)((pos - tile0 + s.tiles - 1) / share);
            record->q0 = (int32_t)s.q0;
            record->head = head;
            record->rows = rows;
            record->row0 = row0;
        }
        float *slot = slots + ((int64_t)blockIdx.x * 2 + (begins ? 1 : 0)) * slot_floats(NR, D);
        constexpr int kSets = kThreads / (D / 4);  // rows in one pass
        for (int row = tid / (D / 4); row < rows; row += kSets) {
            const int d = (tid % (D / 4)) * 4;
            float top = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w)
                top = fmaxf(top, ms[w * NR + row]);
            float sum_l = 0.0f;
            float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float mw = ms[w * NR + row];
                const float f = mw == -INFINITY ? (ls[w * NR + row] == 0.0f ? 0.0f : 1.0f) : exp2_approx(mw - top);
                sum_l = fmaf(f, ls[w * NR + row], sum_l);
                const float4 v = *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(ring) + (w * NR + row) * D + d);
                acc.x = fmaf(f, v.x, acc.x);
                acc.y = fmaf(f, v.y, acc.y);
                acc.z = fmaf(f, v.z, acc.z);
                acc.w = fmaf(f, v.w, acc.w);
            }
            if (begins && ends) {
                const int64_t r = row0 + row, i = r / a.group;
                const int64_t qh = (int64_t)head * a.group + (r - i * a.group);
                const float inv = sum_l == 0.0f ? 0.0f : 1.0f / (sum_l * vg);
                *reinterpret_cast<uint2 *>(a.out + (s.q0 + i) * a.ldo + qh * D + d) =
                    make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
                if (a.lse != nullptr && d == 0)
                    a.lse[(s.q0 + i) * a.hq + qh] = sum_l == 0.0f ? -INFINITY : (top == -INFINITY ? 0.0f : top) * kLn2 + logf(sum_l);
            } else {
                *reinterpret_cast<float4 *>(slot + row * D + d) = acc;
                if (d == 0) {
                    slot[NR * D + row] = top;
                    slot[NR * D + NR + row] = sum_l;
                }
            }
        }
        __syncthreads();  // before the ring is filled again
        pos += count;
    }
    pdl_launch_dependents();
}

// One block per (unit over several blocks, row): its parts in order.
template <int D>
__global__ void __launch_bounds__(256) attn_join_kernel(const __grid_constant__ AttnArgs a, int blocks, int NR)
{
    constexpr int kLanes = D / 4, kParts = 256 / kLanes;
    __shared__ float4 acc_of[kParts][kLanes];
    __shared__ float m_of[kParts], l_of[kParts];
    const int first = blockIdx.x, row = blockIdx.y;
    pdl_wait();
    pdl_launch_dependents();
    const Record rec = reinterpret_cast<const Record *>(a.partial)[first];
    if (rec.last < 0 || row >= rec.rows)
        return;
    const float *slots = a.partial + (int64_t)blocks * (sizeof(Record) / 4);
    const int part = threadIdx.x / kLanes, d = (threadIdx.x % kLanes) * 4;
    float m = -INFINITY, l = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // each set of lanes takes a run of the blocks, so that the order is the keys'
    const int n = rec.last - first + 1, per = (n + kParts - 1) / kParts;
    const int i1 = min(n, (part + 1) * per);
#pragma unroll 4
    for (int i = part * per; i < i1; ++i) {
        const float *slot = slots + ((int64_t)(first + i) * 2 + (i == 0 ? 1 : 0)) * slot_floats(NR, D);
        const float mi = slot[NR * D + row], li = slot[NR * D + NR + row];
        const float4 v = *reinterpret_cast<const float4 *>(slot + row * D + d);
        const float top = fmaxf(m, mi);
        const float f0 = m == -INFINITY ? (l == 0.0f ? 0.0f : 1.0f) : exp2_approx(m - top);
        const float f1 = mi == -INFINITY ? (li == 0.0f ? 0.0f : 1.0f) : exp2_approx(mi - top);
        m = top;
        l = l * f0 + li * f1;
        acc.x = acc.x * f0 + v.x * f1;
        acc.y = acc.y * f0 + v.y * f1;
        acc.z = acc.z * f0 + v.z * f1;
        acc.w = acc.w * f0 + v.w * f1;
    }
    acc_of[part][threadIdx.x % kLanes] = acc;
    if (d == 0) {
        m_of[part] = m;
        l_of[part] = l;
    }
    __syncthreads();
    if (part != 0)
        return;
    float top = -INFINITY, sum = 0.0f;
    for (int i = 0; i < kParts; ++i)
        top = fmaxf(top, m_of[i]);
    acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int i = 0; i < kParts; ++i) {
        const float f = m_of[i] == -INFINITY ? (l_of[i] == 0.0f ? 0.0f : 1.0f) : exp2_approx(m_of[i] - top);
        const float4 v = acc_of[i][threadIdx.x];
        sum = fmaf(f, l_of[i], sum);
        acc.x = fmaf(f, v.x, acc.x);
        acc.y = fmaf(f, v.y, acc.y);
        acc.z = fmaf(f, v.z, acc.z);
        acc.w = fmaf(f, v.w, acc.w);
    }
    const int64_t r = rec.row0 + row, i = r / a.group;
    const int64_t qh = (int64_t)rec.head * a.group + (r - i * a.group);
    const float inv = sum == 0.0f ? 0.0f : 1.0f / (sum * *a.cache.v_scale);
    *reinterpret_cast<uint2 *>(a.out + (rec.q0 + i) * a.ldo + qh * D + d) =
        make_uint2(pack_bf16x2(acc.x * inv, acc.y * inv), pack_bf16x2(acc.z * inv, acc.w * inv));
    if (a.lse != nullptr && d == 0)
        a.lse[(rec.q0 + i) * a.hq + qh] = sum == 0.0f ? -INFINITY : (top == -INFINITY ? 0.0f : top) * kLn2 + logf(sum);
}

template <int D, int NT>
cudaError_t launch_few(const AttnArgs &a, bool pdl, cudaStream_t stream)
{
    constexpr int kBlocks = blocks_of(NT), smem = kWarps * stages_of(NT) * Layout<D>::kTile + 2 * kWarps * 8 * NT * 4;
    static std::atomic<bool> ready[kMaxCachedDevices];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess)
        return err;
    const bool cached = dev >= 0 && dev < kMaxCachedDevices;
    if (!cached || !ready[dev].load(std::memory_order_relaxed)) {
        err = cudaFuncSetAttribute(attn_few_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (err != cudaSuccess)
            return err;
        if (cached)
            ready[dev].store(true, std::memory_order_relaxed);
    }
    err = launch_kernel(attn_few_kernel<D, NT>, dim3(kBlocks), dim3(kThreads), smem, stream, pdl, a);
    if (err != cudaSuccess)
        return err;
    return launch_kernel(attn_join_kernel<D>, dim3(kBlocks, 8 * NT), dim3(256), 0, stream, true, a, kBlocks, 8 * NT);
}

}  // namespace

cudaError_t launch_attn_few(const AttnArgs &a, int64_t rows, bool pdl, cudaStream_t stream)
{
    if (a.D == 64)
        return rows <= 8 ? launch_few<64, 1>(a, pdl, stream) : launch_few<64, 2>(a, pdl, stream);
    return rows <= 8 ? launch_few<128, 1>(a, pdl, stream) : launch_few<128, 2>(a, pdl, stream);
}

int64_t attn_few_workspace(int64_t D)
{
    int64_t most = 0;  // (the same for every form, so that it does not shrink where max_q grows)
    for (int nt = 1; nt <= 2; ++nt) {
        const int64_t n = blocks_of(nt) * ((int64_t)sizeof(Record) + 2 * 4 * slot_floats(8 * nt, (int)D));
        most = n > most ? n : most;
    }
    return most;
}

}  // namespace tsfn
