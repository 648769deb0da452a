// Row-wise NVFP4: bf16 rows to codes and scale factors, the values read back,
// and token rows put in expert order, as bf16 or as NVFP4.
//
// Quantiser, for each 16-column block (the arithmetic of the NVFP4 epilogue of
// fused_rows.cu, on x itself; every step one fp32 rounding):
//   sf = e4m3(g * (amax/6)),  code = e2m1(x * (g / value(sf))),  0 if value(sf) == 0
//
// All three are bound by memory.  Work unit of a warp: 1024 columns of one row,
// or several whole rows where a row is shorter, all loads issued before the
// first is used.  The quantiser gives a lane whole blocks (two, 32 lanes apart),
// so that a block's scale is computed once; four lanes gather their scale
// factors into one 32-bit store.  The others give a lane chunks of 8 columns.
#include "device_util.cuh"
#include "launch_nvfp4.h"

namespace tsfn {

namespace {

constexpr int kThreads = 256;  // at most
constexpr int kChunks = 4;  // chunks of 8 columns per lane
constexpr int kBlocks = 2;  // blocks of 16 columns per lane

// Where row m's scale factors begin and how far a group of 4 lies from the next,
// for rows of sf_cols of them in one of the three layouts (those of
// sf_layout.cuh, whose functions take the fused call's arguments).
__device__ __forceinline__ int64_t sf_row_base(int layout, int64_t sf_cols, int64_t m)
{
    const int64_t groups = sf_cols >> 2;
    if (layout == kSfSwizzled128x4)  // 512-byte tiles: row 32*i + j of a tile at byte 16*j + 4*i
        return (m >> 7) * groups * 512 + (m & 31) * 16 + ((m & 127) >> 5) * 4;
    if (layout == kSfSwizzled8x4)  // 32-byte tiles, row-major inside
        return (m >> 3) * groups * 32 + (m & 7) * 4;
    return m * sf_cols;
}

__device__ __forceinline__ int sf_group_stride(int layout)
{
    return layout == kSfSwizzled128x4 ? 512 : (layout == kSfSwizzled8x4 ? 32 : 4);
}

// The 16 E2M1 codes of a block, and its scale factor.
__device__ __forceinline__ uint2 quantize_block(const uint4 (&v)[2], float g, uint32_t &sf)
{
    float n[2][8];
    unpack8(v[0], n[0]);
    unpack8(v[1], n[1]);
    float amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e)
        amax = fmaxf(amax, fmaxf(fabsf(n[0][e]), fabsf(n[1][e])));
    sf = cvt_e4m3(__fmul_rn(g, div_const_rn(amax, 6.0f, kRcp6)));
    const float d = e4m3_value(sf);
    if (d == 0.0f)
        return make_uint2(0, 0);
    const float es = __fdiv_rn(g, d);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        n[0][e] = __fmul_rn(n[0][e], es);
        n[1][e] = __fmul_rn(n[1][e], es);
    }
    return make_uint2(cvt_e2m1x8(n[0]), cvt_e2m1x8(n[1]));
}

// The scale factors of four lanes' blocks in one word, on the first lane.
__device__ __forceinline__ uint32_t gather_sf(uint32_t sf)
{
    const uint32_t two = sf | (__shfl_down_sync(0xffffffffu, sf, 1) << 8);
    return two | (__shfl_down_sync(0xffffffffu, two, 2) << 16);
}

// Stores the scale factors of a row's blocks b0 + 2^lg * i: four at a time where
// a row's come in fours, else one by one, and zeros in the padding columns.
__device__ __forceinline__ void store_sf(const RowsArgs &a, int64_t row, int b0, int lg, const uint32_t (&sf)[kBlocks])
{
    const int nb = (int)(a.K >> 4);
    const int stride = sf_group_stride(a.sf_layout);
    uint8_t *p = a.sf + sf_row_base(a.sf_layout, a.sf_cols, row);
    if ((nb & 3) == 0) {
        if ((b0 & 3) == 0) {  // (2^lg >= 4 here)
            p += (int64_t)(b0 >> 2) * stride;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i)
                if (b0 + (i << lg) < nb)
                    *reinterpret_cast<uint32_t *>(p + (int64_t)(i << lg >> 2) * stride) = sf[i];
        }
    } else {
#pragma unroll
        for (int i = 0; i < kBlocks; ++i) {
            const int k = b0 + (i << lg);
            if (k < nb)
                p[(int64_t)(k >> 2) * stride + (k & 3)] = (uint8_t)sf[i];
            if (k + 1 == nb)
                for (int kk = nb; kk < (int)a.sf_cols; ++kk)
                    p[(int64_t)(kk >> 2) * stride + (kk & 3)] = 0;
        }
    }
}

// Row t -> NVFP4 row t, or its k rows (SCATTER).  WIDE: a warp per 1024 columns of
// a row.  As many blocks per SM as the registers allow, which the latency of a
// warp's one round of loads needs (16384 x 5120 in the 128x4 layout: 30.9 us with
// 5, 33.1 with 4; the copy floor is 31.7, some of the output stays in L2).
// A dispatch of 4096 x 8 rows of 7168 takes 38.7 us, 28.8 without the scale
// factors: a row's lie 512 bytes apart, so every 4 of them are a line of their
// own for the store unit.  Its codes go out with the streaming hint (43.6 us
// without): they are eight times the tokens and displace them.
template <bool SCATTER, bool WIDE>
__global__ void __launch_bounds__(kThreads, SCATTER ? 4 : 5) nvfp4_rows_kernel(const __grid_constant__ RowsArgs a)
{
    const int lg = WIDE ? 5 : a.tpr_log2;
    const int lane = threadIdx.x & 31;
    const int64_t t = (((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) << (5 - lg)) + (lane >> lg);
    const int nb = (int)(a.K >> 4);
    const int b0 = (int)blockIdx.y * (32 * kBlocks) + (lane & ((1 << lg) - 1));
    pdl_wait();
    bool live = t < a.T;
    if (!SCATTER && live && a.row_src != nullptr)
        live = a.row_src[t] >= 0;
    const uint16_t *row = a.x + t * a.ldx + (int64_t)b0 * 16;
    uint4 v[kBlocks][2];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
        if (live && b0 + (i << lg) < nb) {
            v[i][0] = ld_stream(row + (int64_t)(i << lg) * 16);
            v[i][1] = ld_stream(row + (int64_t)(i << lg) * 16 + 8);
        }
    }
    const float g = *a.g;
    pdl_launch_dependents();
    uint2 codes[kBlocks];
    uint32_t sf[kBlocks];
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
        codes[i] = quantize_block(v[i], g, sf[i]);
        const uint32_t four = gather_sf(sf[i]);
        if ((nb & 3) == 0)
            sf[i] = four;
    }
    if (live) {
        const int k = SCATTER ? a.k : 1;
        const int32_t *row_of = SCATTER ? a.row_of + t * a.k : nullptr;
        int64_t r = SCATTER ? (int64_t)*row_of : t;
        for (int j = 0; j < k; ++j) {
            const int64_t r_next = SCATTER && j + 1 < k ? (int64_t)row_of[j + 1] : 0;
            if (!SCATTER || (r >= 0 && r < a.rows)) {
                uint8_t *out = a.codes + r * (a.K >> 1) + (int64_t)b0 * 8;
#pragma unroll
                for (int i = 0; i < kBlocks; ++i)
                    if (b0 + (i << lg) < nb) {
                        if (SCATTER)
                            st_v2(out + (int64_t)(i << lg) * 8, codes[i]);
                        else
                            *reinterpret_cast<uint2 *>(out + (int64_t)(i << lg) * 8) = codes[i];
                    }
                store_sf(a, r, b0, lg, sf);
            }
            r = r_next;
        }
    } else if (!SCATTER && a.row_src == nullptr && t < a.sf_rows) {
        // a padding row of a swizzled layout: zeros only
        const uint32_t none[kBlocks] = {};
        store_sf(a, t, b0, lg, none);
    }
}

// Row t -> its k rows, copied.  Where a warp has one token, its lanes look up the rows
// of 32 slots in one load and pass them round (16 x 8 rows of 7168 1.9 us; one load
// after the other, which the stores hold up, 2.1).
__global__ void __launch_bounds__(kThreads) dispatch_rows_kernel(const __grid_constant__ RowsArgs a)
{
    const int lane = threadIdx.x & 31;
    const int l = lane & ((1 << a.tpr_log2) - 1);
    const int64_t t = (((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) << (5 - a.tpr_log2)) + (lane >> a.tpr_log2);
    const int nc = (int)(a.K >> 3);
    const int c0 = (int)blockIdx.y * (32 * kChunks) + l;
    pdl_wait();
    if (t >= a.T)
        return;
    const uint16_t *row = a.x + t * a.ldx;
    uint4 v[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = c0 + (i << a.tpr_log2);
        if (c < nc)
            v[i] = ld_stream(row + (int64_t)c * 8);
    }
    pdl_launch_dependents();
    const int32_t *row_of = a.row_of + t * a.k;
    const bool wide = a.tpr_log2 == 5;
    int32_t mine = 0;
#pragma unroll 8
    for (int j = 0; j < a.k; ++j) {
        int32_t r;
        if (wide) {
            if ((j & 31) == 0)
                mine = j + lane < a.k ? row_of[j + lane] : -1;
            r = __shfl_sync(0xffffffffu, mine, j & 31);
        } else
            r = row_of[j];
        if (r < 0 || r >= a.rows)
            continue;
        uint16_t *out = a.out + r * a.K;
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
            const int c = c0 + (i << a.tpr_log2);
            if (c < nc)
                st_v4(out + (int64_t)c * 8, v[i]);
        }
    }
}

// Two E2M1 codes -> two fp32 values (the hardware conversion to f16, exact).
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte)
{
    float2 f;
    asm("{\n\t.reg .b8 b;\n\t.reg .b32 h;\n\t.reg .b16 lo, hi;\n\t"
        "cvt.u8.u32 b, %2;\n\t"
        "cvt.rn.f16x2.e2m1x2 h, b;\n\t"
        "mov.b32 {lo, hi}, h;\n\t"
        "cvt.f32.f16 %0, lo;\n\t"
        "cvt.f32.f16 %1, hi;\n\t}"
        : "=f"(f.x), "=f"(f.y)
        : "r"(byte));
    return f;
}

__global__ void __launch_bounds__(kThreads) nvfp4_values_kernel(const __grid_constant__ DequantArgs a)
{
    const int lane = threadIdx.x & 31;
    const int l = lane & ((1 << a.tpr_log2) - 1);
    const int64_t t = (((int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5)) << (5 - a.tpr_log2)) + (lane >> a.tpr_log2);
    const int nc = (int)(a.K >> 3);
    const int c0 = (int)blockIdx.y * (32 * kChunks) + l;
    pdl_wait();
    if (t >= a.T || (a.row_src != nullptr && a.row_src[t] < 0))
        return;
    const uint8_t *codes = a.codes + t * (a.K >> 1);
    const uint8_t *sf = a.sf + sf_row_base(a.sf_layout, a.sf_cols, t);
    const int stride = sf_group_stride(a.sf_layout);
    uint32_t w[kChunks], s[kChunks];
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = c0 + (i << a.tpr_log2);
        if (c < nc) {
            const int k = c >> 1;
            w[i] = *reinterpret_cast<const uint32_t *>(codes + (int64_t)c * 4);
            s[i] = sf[(int64_t)(k >> 2) * stride + (k & 3)];
        }
    }
    const float g = *a.g;
    pdl_launch_dependents();
    uint16_t *out = a.out + t * a.ldo;
#pragma unroll
    for (int i = 0; i < kChunks; ++i) {
        const int c = c0 + (i << a.tpr_log2);
        if (c < nc) {
            const float d = __fdiv_rn(e4m3_value(s[i]), g);
            float f[8];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 p = e2m1x2_values((w[i] >> (8 * e)) & 0xFFu);
                f[2 * e] = __fmul_rn(p.x, d);
                f[2 * e + 1] = __fmul_rn(p.y, d);
            }
            st_v4(out + (int64_t)c * 8, pack8(f));
        }
    }
}

// Lanes per row of `units` chunks or blocks: 32 with up to `each` of them, fewer
// (but at least 4 where there are 4) where a row has less, so that a warp takes
// several rows.
int lanes_log2(int64_t units, int each)
{
    int l = 0;
    while (l < 5 && (1 << l) < units && ((each << l) < units || l < 2))
        ++l;
    return l;
}

// Rows along x, 1024 columns of a row along y; 8 warps a block, fewer where the
// warps would not reach every SM (a dispatch of 16 x 8 rows of 7168: 2.0 us, 3.6
// on 14 blocks of 8 warps).
struct Launch {
    dim3 grid, block;
};

Launch launch_of(int64_t rows, int64_t K, int tpr_log2)
{
    const int64_t per_warp = 1 << (5 - tpr_log2), segs = (K + 1023) / 1024;
    const int64_t warps = (rows + per_warp - 1) / per_warp;  // along the rows
    const int sms = current_device_sms();
    int64_t w = sms > 0 ? (warps * segs + sms - 1) / sms : kThreads / 32;
    w = w < kThreads / 32 ? w : kThreads / 32;
    return {dim3((unsigned)((warps + w - 1) / w), (unsigned)segs), dim3((unsigned)(32 * w))};
}

}  // namespace

cudaError_t launch_quantize(const RowsArgs &a, bool pdl, cudaStream_t stream)
{
    RowsArgs b = a;
    b.tpr_log2 = lanes_log2(a.K / 16, kBlocks);
    const int64_t rows = a.row_src == nullptr ? a.sf_rows : a.T;
    const Launch l = launch_of(rows, a.K, b.tpr_log2);
    if (b.tpr_log2 == 5)
        return launch_kernel(nvfp4_rows_kernel<false, true>, l.grid, l.block, 0, stream, pdl, b);
    return launch_kernel(nvfp4_rows_kernel<false, false>, l.grid, l.block, 0, stream, pdl, b);
}

cudaError_t launch_dispatch(const RowsArgs &a, bool pdl, cudaStream_t stream)
{
    RowsArgs b = a;
    b.tpr_log2 = a.out != nullptr ? lanes_log2(a.K / 8, kChunks) : lanes_log2(a.K / 16, kBlocks);
    const Launch l = launch_of(a.T, a.K, b.tpr_log2);
    if (a.out != nullptr)
        return launch_kernel(dispatch_rows_kernel, l.grid, l.block, 0, stream, pdl, b);
    if (b.tpr_log2 == 5)
        return launch_kernel(nvfp4_rows_kernel<true, true>, l.grid, l.block, 0, stream, pdl, b);
    return launch_kernel(nvfp4_rows_kernel<true, false>, l.grid, l.block, 0, stream, pdl, b);
}

cudaError_t launch_dequantize(const DequantArgs &a, bool pdl, cudaStream_t stream)
{
    DequantArgs b = a;
    b.tpr_log2 = lanes_log2(a.K / 8, kChunks);
    const Launch l = launch_of(a.T, a.K, b.tpr_log2);
    return launch_kernel(nvfp4_values_kernel, l.grid, l.block, 0, stream, pdl, b);
}

}  // namespace tsfn
