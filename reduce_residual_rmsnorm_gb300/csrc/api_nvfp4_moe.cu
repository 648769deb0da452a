// The C ABI declared in include/ts_nvfp4_moe.h: host-side argument checks, then
// one kernel launch on the caller's stream.
#include <cstdint>

#include <cuda_runtime.h>

#include "api_util.h"
#include "launch_nvfp4.h"
#include "ts_nvfp4_moe.h"

using namespace tsfn;

namespace {

constexpr int64_t kMaxCols = 65536;
constexpr int64_t kMaxSlots = 64;
constexpr int64_t kMaxExperts = 1024;
constexpr int64_t kMaxEntries = 1LL << 30;

struct Buffer {
    const void *p;
    int64_t bytes;
    int align;
    const char *name;
    bool output;
    bool optional;
};

// Every buffer present and aligned, no output over another buffer.  `empty`:
// a call without rows, whose buffers may be NULL.
template <int N>
int check_buffers(const Buffer (&b)[N], bool empty)
{
    for (const Buffer &x : b) {
        if (x.p == nullptr && !x.optional && !empty)
            return fail(TS_ERR_NULL, "%s is NULL", x.name);
        if (!aligned(x.p, (uintptr_t)x.align))
            return fail(TS_ERR_ALIGN, "%s is not %d-byte aligned", x.name, x.align);
    }
    for (int i = 0; i < N; ++i) {
        if (!b[i].output || b[i].p == nullptr)
            continue;
        for (int j = 0; j < N; ++j) {
            if (j == i || b[j].p == nullptr || (b[j].output && j < i))
                continue;
            if (overlap(span(b[i].p, b[i].bytes, ""), span(b[j].p, b[j].bytes, "")))
                return fail(TS_ERR_ALIAS, "%s overlaps %s", b[i].name, b[j].name);
        }
    }
    return TS_OK;
}

int check_flags(uint32_t flags)
{
    if (flags & ~(uint32_t)TS_FLAG_PDL)
        return fail(TS_ERR_UNSUPPORTED, "unknown flag bits 0x%x", flags & ~(uint32_t)TS_FLAG_PDL);
    return TS_OK;
}

int check_rows(const char *name, int64_t rows)
{
    if (rows < 0 || rows > kMaxRows)
        return fail(TS_ERR_SHAPE, "%s = %lld outside 0..%lld", name, (long long)rows, (long long)kMaxRows);
    return TS_OK;
}

int check_cols(const char *name, int64_t cols, int64_t multiple)
{
    if (cols < multiple || cols % multiple != 0)
        return fail(TS_ERR_SHAPE, "%s = %lld must be a positive multiple of %lld", name, (long long)cols,
                    (long long)multiple);
    if (cols > kMaxCols)
        return fail(TS_ERR_UNSUPPORTED, "%s = %lld above the supported maximum %lld", name, (long long)cols,
                    (long long)kMaxCols);
    return TS_OK;
}

int check_stride(const char *name, int64_t ld, int64_t cols)
{
    if (ld < cols || ld % 8 != 0 || ld > (1LL << 30))  // (rows of 2^31 stay within 64 bits of bytes)
        return fail(TS_ERR_SHAPE, "%s = %lld must be a multiple of 8 in %lld..2^30", name, (long long)ld,
                    (long long)cols);
    return TS_OK;
}

int check_slots(int64_t T, int64_t k)
{
    if (k < 1 || k > kMaxSlots)
        return fail(TS_ERR_SHAPE, "k = %lld outside 1..%lld", (long long)k, (long long)kMaxSlots);
    if (T * k >= kMaxEntries)
        return fail(TS_ERR_SHAPE, "T * k = %lld must be below 2^30", (long long)(T * k));
    return TS_OK;
}

int check_layout(int layout)
{
    if (layout != TS_SF_SWIZZLED_128x4 && layout != TS_SF_SWIZZLED_8x4 && layout != TS_SF_LINEAR)
        return fail(TS_ERR_BAD_PATTERN, "sf_layout %d is not a QuantizationSFLayout code", layout);
    return TS_OK;
}

// Rows and columns of the scale-factor buffer of [rows, cols] values.
void sf_sizes(int layout, int64_t rows, int64_t cols, int64_t *sf_rows, int64_t *sf_cols)
{
    const int64_t tile = layout == TS_SF_SWIZZLED_128x4 ? 128 : (layout == TS_SF_SWIZZLED_8x4 ? 8 : 1);
    *sf_rows = (rows + tile - 1) / tile * tile;
    *sf_cols = layout == TS_SF_LINEAR ? cols / 16 : (cols / 16 + 3) / 4 * 4;
}

// Bytes from the first to the last element of a strided bf16 matrix.
int64_t bf16_bytes(int64_t rows, int64_t cols, int64_t ld) { return rows > 0 ? ((rows - 1) * ld + cols) * 2 : 0; }

int launched(cudaError_t err)
{
    if (err != cudaSuccess)
        return fail(TS_ERR_LAUNCH, "kernel launch failed: %s (%s)", cudaGetErrorName(err), cudaGetErrorString(err));
    return ok();
}

const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }
const uint8_t *u8(const void *p) { return static_cast<const uint8_t *>(p); }

}  // namespace

#define TS_TRY(expr)              \
    do {                          \
        const int status_ = expr; \
        if (status_ != TS_OK)     \
            return status_;       \
    } while (0)

extern "C" int ts_nvfp4_quantize(const void *x, int64_t T, int64_t K, int64_t ldx, const float *scale_factor,
                                 const int32_t *row_src, void *quant_out, void *scale_out, int sf_layout,
                                 uint32_t flags, void *stream)
{
    TS_TRY(check_flags(flags));
    TS_TRY(check_rows("T", T));
    TS_TRY(check_cols("K", K, 16));
    TS_TRY(check_stride("ldx", ldx, K));
    TS_TRY(check_layout(sf_layout));
    RowsArgs a{};
    sf_sizes(sf_layout, T, K, &a.sf_rows, &a.sf_cols);
    const Buffer b[] = {{x, bf16_bytes(T, K, ldx), 16, "x", false, false},
                        {scale_factor, 4, 4, "scale_factor", false, false},
                        {row_src, T * 4, 4, "row_src", false, true},
                        {quant_out, T * (K / 2), 16, "quant_out", true, false},
                        {scale_out, a.sf_rows * a.sf_cols, 4, "scale_out", true, false}};
    TS_TRY(check_buffers(b, T == 0));
    if (T == 0)
        return ok();
    a.x = u16(x);
    a.ldx = ldx;
    a.T = T;
    a.K = K;
    a.row_src = row_src;
    a.rows = T;
    a.g = scale_factor;
    a.codes = static_cast<uint8_t *>(quant_out);
    a.sf = static_cast<uint8_t *>(scale_out);
    a.sf_layout = sf_layout;
    return launched(launch_quantize(a, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

extern "C" int ts_nvfp4_dequantize(const void *quant, const void *scale, int sf_layout, int64_t T, int64_t K,
                                   const float *scale_factor, const int32_t *row_src, void *out, int64_t ldo,
                                   uint32_t flags, void *stream)
{
    TS_TRY(check_flags(flags));
    TS_TRY(check_rows("T", T));
    TS_TRY(check_cols("K", K, 16));
    TS_TRY(check_stride("ldo", ldo, K));
    TS_TRY(check_layout(sf_layout));
    DequantArgs a{};
    int64_t sf_rows = 0;
    sf_sizes(sf_layout, T, K, &sf_rows, &a.sf_cols);
    const Buffer b[] = {{quant, T * (K / 2), 16, "quant", false, false},
                        {scale, sf_rows * a.sf_cols, 4, "scale", false, false},
                        {scale_factor, 4, 4, "scale_factor", false, false},
                        {row_src, T * 4, 4, "row_src", false, true},
                        {out, bf16_bytes(T, K, ldo), 16, "out", true, false}};
    TS_TRY(check_buffers(b, T == 0));
    if (T == 0)
        return ok();
    a.codes = u8(quant);
    a.sf = u8(scale);
    a.sf_layout = sf_layout;
    a.T = T;
    a.K = K;
    a.g = scale_factor;
    a.row_src = row_src;
    a.out = static_cast<uint16_t *>(out);
    a.ldo = ldo;
    return launched(launch_dequantize(a, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

namespace {

// The sizes of a product that both forms check alike.
int check_product(int64_t N, int64_t K, int64_t ldo)
{
    if (N < 8 || N % 8 != 0 || N > (1LL << 24))
        return fail(TS_ERR_SHAPE, "N = %lld must be a multiple of 8 in 8..2^24", (long long)N);
    TS_TRY(check_cols("K", K, 32));
    return check_stride("ldo", ldo, N);
}

}  // namespace

extern "C" int ts_nvfp4_gemm(const void *a, const void *a_scale, const void *b, const void *b_scale,
                             const float *alpha, int64_t M, int64_t N, int64_t K, void *out, int64_t ldo,
                             uint32_t flags, void *stream)
{
    TS_TRY(check_flags(flags));
    TS_TRY(check_rows("M", M));
    TS_TRY(check_product(N, K, ldo));
    int64_t a_rows = 0, b_rows = 0, cols = 0;
    sf_sizes(TS_SF_SWIZZLED_128x4, M, K, &a_rows, &cols);
    sf_sizes(TS_SF_SWIZZLED_128x4, N, K, &b_rows, &cols);
    const Buffer bufs[] = {{a, M * (K / 2), 16, "a", false, false},
                           {a_scale, a_rows * cols, 16, "a_scale", false, false},
                           {b, N * (K / 2), 16, "b", false, false},
                           {b_scale, b_rows * cols, 16, "b_scale", false, false},
                           {alpha, 4, 4, "alpha", false, false},
                           {out, bf16_bytes(M, N, ldo), 16, "out", true, false}};
    TS_TRY(check_buffers(bufs, M == 0));
    if (M == 0)
        return ok();
    GemmArgs g{};
    g.tok = u8(a);
    g.tok_sf = u8(a_scale);
    g.tok_rows = M;
    g.wgt = u8(b);
    g.wgt_sf = u8(b_scale);
    g.alpha = alpha;
    g.N = N;
    g.K = K;
    g.out = static_cast<uint16_t *>(out);
    g.ldo = ldo;
    return launched(launch_nvfp4_gemm(g, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

extern "C" int ts_nvfp4_grouped_gemm(const void *a, const void *a_scale, const void *b, const void *b_scale,
                                     const float *alpha, const int32_t *expert_start, const int32_t *expert_count,
                                     int64_t E, int64_t rows, int64_t entries, int64_t N, int64_t K, void *out,
                                     int64_t ldo, uint32_t flags, void *stream)
{
    TS_TRY(check_flags(flags));
    TS_TRY(check_rows("rows", rows));
    TS_TRY(check_product(N, K, ldo));
    if (E < 1 || E > kMaxExperts)
        return fail(TS_ERR_SHAPE, "E = %lld outside 1..%lld", (long long)E, (long long)kMaxExperts);
    if (E * N > kMaxRows - 511)  // (32-bit row coordinates, to the end of the last tile)
        return fail(TS_ERR_SHAPE, "E * N = %lld above %lld", (long long)(E * N), (long long)(kMaxRows - 511));
    if (rows % 128 != 0)
        return fail(TS_ERR_SHAPE, "rows = %lld must be a multiple of 128", (long long)rows);
    if (entries < 0)
        return fail(TS_ERR_SHAPE, "entries = %lld is negative", (long long)entries);
    int64_t a_rows = 0, b_rows = 0, cols = 0;
    sf_sizes(TS_SF_SWIZZLED_128x4, rows, K, &a_rows, &cols);
    sf_sizes(TS_SF_SWIZZLED_128x4, N, K, &b_rows, &cols);
    const Buffer bufs[] = {{a, rows * (K / 2), 16, "a", false, false},
                           {a_scale, a_rows * cols, 16, "a_scale", false, false},
                           {b, E * N * (K / 2), 16, "b", false, false},
                           {b_scale, E * b_rows * cols, 16, "b_scale", false, false},
                           {alpha, E * 4, 4, "alpha", false, false},
                           {expert_start, (E + 1) * 4, 4, "expert_start", false, false},
                           {expert_count, E * 4, 4, "expert_count", false, false},
                           {out, bf16_bytes(rows, N, ldo), 16, "out", true, false}};
    TS_TRY(check_buffers(bufs, rows == 0));
    if (rows == 0)
        return ok();
    GemmArgs g{};
    g.tok = u8(a);
    g.tok_sf = u8(a_scale);
    g.tok_rows = rows;
    g.wgt = u8(b);
    g.wgt_sf = u8(b_scale);
    g.alpha = alpha;
    g.N = N;
    g.K = K;
    g.out = static_cast<uint16_t *>(out);
    g.ldo = ldo;
    g.start = expert_start;
    g.count = expert_count;
    g.experts = (int)E;
    g.entries = entries;
    return launched(launch_nvfp4_gemm(g, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

extern "C" int64_t ts_moe_rows(int64_t T, int64_t k, int64_t E, int64_t row_align)
{
    if (T < 0 || T > kMaxRows || k < 1 || k > kMaxSlots || T * k >= kMaxEntries || E < 1 || E > kMaxExperts ||
        row_align < 1 || row_align > 256)
        return -1;
    const int64_t n = T * k, used = n < E ? n : E;
    return (n + used * (row_align - 1) + row_align - 1) / row_align * row_align;
}

extern "C" int ts_moe_sort(const int32_t *expert_ids, int64_t T, int64_t k, int64_t E, int64_t row_align,
                           int64_t rows, int32_t *row_of, int32_t *row_src, int32_t *expert_start,
                           int32_t *expert_count, uint32_t flags, void *stream)
{
    TS_TRY(check_flags(flags));
    TS_TRY(check_rows("T", T));
    TS_TRY(check_slots(T, k));
    if (E < 1 || E > kMaxExperts)
        return fail(TS_ERR_SHAPE, "E = %lld outside 1..%lld", (long long)E, (long long)kMaxExperts);
    if (row_align < 1 || row_align > 256)
        return fail(TS_ERR_SHAPE, "row_align = %lld outside 1..256", (long long)row_align);
    TS_TRY(check_rows("rows", rows));
    if (rows < ts_moe_rows(T, k, E, row_align))
        return fail(TS_ERR_SHAPE, "rows = %lld below ts_moe_rows = %lld", (long long)rows,
                    (long long)ts_moe_rows(T, k, E, row_align));
    // without tokens the experts' starts and counts are still written
    const Buffer b[] = {{expert_ids, T * k * 4, 4, "expert_ids", false, T == 0},
                        {row_of, T * k * 4, 4, "row_of", true, T == 0},
                        {row_src, rows * 4, 4, "row_src", true, rows == 0},
                        {expert_start, (E + 1) * 4, 4, "expert_start", true, false},
                        {expert_count, E * 4, 4, "expert_count", true, false}};
    TS_TRY(check_buffers(b, false));
    SortArgs a{};
    a.ids = expert_ids;
    a.n = T * k;
    a.E = (int)E;
    a.align = (int)row_align;
    a.rows = rows;
    a.row_of = row_of;
    a.row_src = row_src;
    a.start = expert_start;
    a.count = expert_count;
    return launched(launch_sort(a, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

extern "C" int ts_moe_dispatch(const void *x, int64_t T, int64_t H, int64_t ldx, const int32_t *row_of, int64_t k,
                               int64_t rows, void *out, const float *scale_factor, void *quant_out,
                               void *scale_out, int sf_layout, uint32_t flags, void *stream)
{
    const bool fp4 = out == nullptr && (quant_out != nullptr || scale_out != nullptr || scale_factor != nullptr);
    TS_TRY(check_flags(flags));
    TS_TRY(check_rows("T", T));
    TS_TRY(check_rows("rows", rows));
    TS_TRY(check_cols("H", H, fp4 ? 16 : 8));
    TS_TRY(check_stride("ldx", ldx, H));
    TS_TRY(check_slots(T, k));
    if (out != nullptr && (quant_out != nullptr || scale_out != nullptr || scale_factor != nullptr))
        return fail(TS_ERR_UNSUPPORTED, "out and the NVFP4 buffers exclude each other");
    RowsArgs a{};
    if (fp4) {
        TS_TRY(check_layout(sf_layout));
        sf_sizes(sf_layout, rows, H, &a.sf_rows, &a.sf_cols);
    }
    const bool empty = T == 0 || rows == 0;
    const Buffer b[] = {{x, bf16_bytes(T, H, ldx), 16, "x", false, false},
                        {row_of, T * k * 4, 4, "row_of", false, false},
                        {out, rows * H * 2, 16, "out", true, fp4},
                        {scale_factor, 4, 4, "scale_factor", false, !fp4},
                        {quant_out, rows * (H / 2), 16, "quant_out", true, !fp4},
                        {scale_out, a.sf_rows * a.sf_cols, 4, "scale_out", true, !fp4}};
    TS_TRY(check_buffers(b, empty));
    if (empty)
        return ok();
    a.x = u16(x);
    a.ldx = ldx;
    a.T = T;
    a.K = H;
    a.row_of = row_of;
    a.k = (int)k;
    a.rows = rows;
    a.out = static_cast<uint16_t *>(out);
    a.g = scale_factor;
    a.codes = static_cast<uint8_t *>(quant_out);
    a.sf = static_cast<uint8_t *>(scale_out);
    a.sf_layout = sf_layout;
    return launched(launch_dispatch(a, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

extern "C" int ts_moe_combine(const void *y, int64_t rows, int64_t H, int64_t ldy, const int32_t *row_of,
                              const float *weights, int64_t T, int64_t k, void *out, int64_t ldo, uint32_t flags,
                              void *stream)
{
    TS_TRY(check_flags(flags));
    TS_TRY(check_rows("T", T));
    TS_TRY(check_rows("rows", rows));
    TS_TRY(check_cols("H", H, 8));
    TS_TRY(check_stride("ldy", ldy, H));
    TS_TRY(check_stride("ldo", ldo, H));
    TS_TRY(check_slots(T, k));
    const Buffer b[] = {{y, bf16_bytes(rows, H, ldy), 16, "y", false, rows == 0},
                        {row_of, T * k * 4, 4, "row_of", false, false},
                        {weights, T * k * 4, 4, "weights", false, true},
                        {out, bf16_bytes(T, H, ldo), 16, "out", true, false}};
    TS_TRY(check_buffers(b, T == 0));
    if (T == 0)
        return ok();
    CombineArgs a{};
    a.y = u16(y);
    a.rows = rows;
    a.ldy = ldy;
    a.H = H;
    a.row_of = row_of;
    a.weights = weights;
    a.T = T;
    a.k = (int)k;
    a.out = static_cast<uint16_t *>(out);
    a.ldo = ldo;
    return launched(launch_combine(a, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

extern "C" int ts_moe_combine_grad(const void *dout, int64_t ldd, const void *y, int64_t ldy, int64_t rows,
                                   int64_t H, const int32_t *row_of, const float *weights, int64_t T, int64_t k,
                                   void *dy, int64_t lddy, float *dweights, uint32_t flags, void *stream)
{
    TS_TRY(check_flags(flags));
    TS_TRY(check_rows("T", T));
    TS_TRY(check_rows("rows", rows));
    TS_TRY(check_cols("H", H, 8));
    TS_TRY(check_stride("ldd", ldd, H));
    TS_TRY(check_stride("ldy", ldy, H));
    TS_TRY(check_stride("lddy", lddy, H));
    TS_TRY(check_slots(T, k));
    const Buffer b[] = {{dout, bf16_bytes(T, H, ldd), 16, "dout", false, false},
                        {y, bf16_bytes(rows, H, ldy), 16, "y", false, rows == 0},
                        {row_of, T * k * 4, 4, "row_of", false, false},
                        {weights, T * k * 4, 4, "weights", false, false},
                        {dy, bf16_bytes(rows, H, lddy), 16, "dy", true, rows == 0},
                        {dweights, T * k * 4, 4, "dweights", true, false}};
    TS_TRY(check_buffers(b, T == 0));
    if (T == 0)
        return ok();
    CombineArgs a{};
    a.y = u16(y);
    a.rows = rows;
    a.ldy = ldy;
    a.H = H;
    a.row_of = row_of;
    a.weights = weights;
    a.T = T;
    a.k = (int)k;
    a.out = static_cast<uint16_t *>(dy);
    a.ldo = lddy;
    a.dout = u16(dout);
    a.ldd = ldd;
    a.dweights = dweights;
    return launched(launch_combine_grad(a, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

extern "C" int ts_stalled_waits(uint32_t *count)
{
    if (count == nullptr)
        return fail(TS_ERR_NULL, "count is NULL");
    return launched(read_stalled_waits(count));
}
