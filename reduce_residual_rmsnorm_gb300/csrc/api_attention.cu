// The C ABI declared in include/ts_attention.h: host-side argument checks, then one
// or two kernel launches on the caller's stream.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "api_util.h"
#include "launch_attention.h"
#include "ts_attention.h"

using namespace tsfn;

namespace {

constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxHeadRows = 1LL << 30;  // tokens x heads: 32-bit indexes of rows
constexpr int64_t kMaxKeys = 1LL << 30;      // of a sequence

// Rows of `width` bytes, `ld` bytes apart; flat buffers are one row.
struct Rows {
    const void *p;
    int64_t rows;
    int64_t width;
    int64_t ld;
    int align;
    const char *name;
    bool output;
    bool optional;
    const void *twin;  // an output that may be this input (same address and stride)
    int64_t twin_ld;
};

Rows flat(const void *p, int64_t bytes, int align, const char *name, bool output = false, bool optional = false)
{
    return {p, bytes > 0 ? 1 : 0, bytes, bytes, align, name, output, optional, nullptr, 0};
}

Rows matrix(const void *p, int64_t rows, int64_t cols, int64_t ld, const char *name, bool output = false,
            bool optional = false, const void *twin = nullptr, int64_t twin_ld = 0)
{
    return {p, rows, cols * 2, ld * 2, 16, name, output, optional, twin, twin_ld * 2};
}

bool rows_overlap(const Rows &a, const Rows &b)
{
    if (a.p == nullptr || b.p == nullptr || a.rows == 0 || b.rows == 0)
        return false;
    const Span x = span(a.p, (a.rows - 1) * a.ld + a.width, ""), y = span(b.p, (b.rows - 1) * b.ld + b.width, "");
    if (!overlap(x, y))
        return false;
    if (a.rows > 1 && b.rows > 1 && a.ld == b.ld) {  // columns of one matrix
        const int64_t from_x = y.lo >= x.lo ? (int64_t)((y.lo - x.lo) % (uint64_t)a.ld)
                                            : (a.ld - (int64_t)((x.lo - y.lo) % (uint64_t)a.ld)) % a.ld;
        return !(from_x >= a.width && from_x + b.width <= a.ld);
    }
    return true;
}

template <int N>
int check_rows_of(const Rows (&b)[N], bool empty)
{
    for (const Rows &x : b) {
        if (x.p == nullptr && !x.optional && !empty)
            return fail(TS_ERR_NULL, "%s is NULL", x.name);
        if (!aligned(x.p, (uintptr_t)x.align))
            return fail(TS_ERR_ALIGN, "%s is not %d-byte aligned", x.name, x.align);
    }
    for (int i = 0; i < N; ++i) {
        if (!b[i].output)
            continue;
        for (int j = 0; j < N; ++j) {
            if (j == i || (b[j].output && j < i))
                continue;
            if (b[i].p != nullptr && b[i].twin == b[j].p && b[i].p == b[j].p && b[i].twin_ld == b[i].ld && b[j].ld == b[i].ld &&
                !b[j].output)
                continue;  // in place
            if (rows_overlap(b[i], b[j]))
                return fail(TS_ERR_ALIAS, "%s overlaps %s", b[i].name, b[j].name);
        }
    }
    return TS_OK;
}

int check_range(const char *name, int64_t v, int64_t lo, int64_t hi)
{
    if (v < lo || v > hi)
        return fail(TS_ERR_SHAPE, "%s = %lld outside %lld..%lld", name, (long long)v, (long long)lo, (long long)hi);
    return TS_OK;
}

int check_flag_bits(uint32_t flags)
{
    if (flags & ~(uint32_t)TS_FLAG_PDL)
        return fail(TS_ERR_UNSUPPORTED, "unknown flag bits 0x%x", flags & ~(uint32_t)TS_FLAG_PDL);
    return TS_OK;
}

int check_head_dim(int64_t D)
{
    if (D < 16 || D > 256 || D % 16 != 0)
        return fail(TS_ERR_SHAPE, "head_dim = %lld must be a multiple of 16 in 16..256", (long long)D);
    return TS_OK;
}

int check_ld(const char *name, int64_t ld, int64_t cols)
{
    if (ld < cols || ld % 8 != 0 || ld > (1LL << 30))
        return fail(TS_ERR_SHAPE, "%s = %lld must be a multiple of 8 in %lld..2^30", name, (long long)ld, (long long)cols);
    return TS_OK;
}

int lanes_log2(int64_t D)
{
    int lg = 1;
    while ((8 << lg) < D)
        ++lg;
    return lg;
}

int check_cache(const ts_kv_cache_t &c)
{
    if (const int st = check_head_dim(c.head_dim))
        return st;
    if (const int st = check_range("cache heads", c.heads, 1, kMaxHeads))
        return st;
    if (c.page_size < 16 || c.page_size > 65536 || c.page_size % 16 != 0)
        return fail(TS_ERR_SHAPE, "page_size = %lld must be a multiple of 16 in 16..65536", (long long)c.page_size);
    if (c.num_pages < 0 || c.num_pages > kMaxRows / c.page_size)
        return fail(TS_ERR_SHAPE, "num_pages = %lld outside 0..%lld", (long long)c.num_pages, (long long)(kMaxRows / c.page_size));
    return TS_OK;
}

CacheArgs cache_args(const ts_kv_cache_t &c)
{
    CacheArgs a{};
    a.pages = static_cast<uint8_t *>(c.pages);
    a.slots = c.num_pages * c.page_size;
    a.num_pages = (int)c.num_pages;
    a.page_size = (int)c.page_size;
    a.div_page = div_magic((uint32_t)c.page_size);
    a.heads = (int)c.heads;
    a.k_scale = c.k_scale;
    a.v_scale = c.v_scale;
    return a;
}

int64_t cache_bytes(const ts_kv_cache_t &c) { return c.num_pages * c.heads * (c.page_size / 16) * 18 * c.head_dim; }

int launched(cudaError_t err)
{
    if (err != cudaSuccess)
        return fail(TS_ERR_LAUNCH, "kernel launch failed: %s (%s)", cudaGetErrorName(err), cudaGetErrorString(err));
    return ok();
}

const uint16_t *u16(const void *p) { return static_cast<const uint16_t *>(p); }

}  // namespace

#define TS_TRY(expr)              \
    do {                          \
        const int status_ = expr; \
        if (status_ != TS_OK)     \
            return status_;       \
    } while (0)

namespace {

// What the rotary calls check alike.
int check_rope(int64_t T, int64_t q_heads, int64_t k_heads, int64_t D, int64_t max_pos, int64_t rot, int interleaved, float eps)
{
    TS_TRY(check_range("T", T, 0, kMaxRows));
    TS_TRY(check_range("q_heads", q_heads, 1, kMaxHeads));
    TS_TRY(check_range("k_heads", k_heads, 1, kMaxHeads));
    TS_TRY(check_head_dim(D));
    TS_TRY(check_range("T * (q_heads + 2 k_heads)", T * (q_heads + 2 * k_heads), 0, kMaxHeadRows));
    TS_TRY(check_range("max_pos", max_pos, 1, kMaxRows));
    if (rot < 16 || rot > D || rot % 16 != 0)
        return fail(TS_ERR_SHAPE, "rot = %lld must be a multiple of 16 in 16..%lld", (long long)rot, (long long)D);
    TS_TRY(check_range("interleaved", interleaved, 0, 1));
    if (!(eps >= 0.0f) || std::isinf(eps))
        return fail(TS_ERR_UNSUPPORTED, "eps = %g must be finite and not negative", (double)eps);
    return TS_OK;
}

}  // namespace

extern "C" int ts_qk_norm_rope(const void *q, int64_t ldq, const void *k, int64_t ldk, int64_t T, int64_t q_heads,
                               int64_t k_heads, int64_t head_dim, const void *q_weight, const void *k_weight, float eps,
                               const int32_t *positions, const float *cos_sin, int64_t max_pos, int64_t rot,
                               int interleaved, void *q_out, int64_t ldqo, void *k_out, int64_t ldko, const void *v,
                               int64_t ldv, const ts_kv_cache_t *cache, const int32_t *slots, uint32_t flags, void *stream)
{
    const int64_t D = head_dim;
    TS_TRY(check_flag_bits(flags));
    TS_TRY(check_rope(T, q_heads, k_heads, D, max_pos, rot, interleaved, eps));
    TS_TRY(check_ld("ldq", ldq, q_heads * D));
    TS_TRY(check_ld("ldk", ldk, k_heads * D));
    TS_TRY(check_ld("ldqo", ldqo, q_heads * D));
    if (k_out != nullptr)
        TS_TRY(check_ld("ldko", ldko, k_heads * D));
    if ((q_weight == nullptr) != (k_weight == nullptr))
        return fail(TS_ERR_UNSUPPORTED, "q_weight and k_weight are given together or not at all");
    ts_kv_cache_t c{};
    const bool kept = cache != nullptr;
    if (kept) {
        c = *cache;
        TS_TRY(check_cache(c));
        if (c.heads != k_heads || c.head_dim != D)
            return fail(TS_ERR_SHAPE, "a cache of %lld heads of %lld for keys of %lld heads of %lld", (long long)c.heads,
                        (long long)c.head_dim, (long long)k_heads, (long long)D);
        TS_TRY(check_ld("ldv", ldv, k_heads * D));
    } else if (v != nullptr || slots != nullptr) {
        return fail(TS_ERR_UNSUPPORTED, "v and slots need a cache");
    }
    const Rows b[] = {matrix(q, T, q_heads * D, ldq, "q"),
                      matrix(k, T, k_heads * D, ldk, "k"),
                      flat(q_weight, D * 2, 16, "q_weight", false, true),
                      flat(k_weight, D * 2, 16, "k_weight", false, true),
                      flat(positions, T * 4, 4, "positions"),
                      flat(cos_sin, max_pos * rot * 4, 16, "cos_sin"),
                      matrix(v, kept ? T : 0, k_heads * D, ldv, "v", false, !kept),
                      flat(slots, T * 4, 4, "slots", false, !kept),
                      flat(c.k_scale, 4, 4, "k_scale", false, !kept),
                      flat(c.v_scale, 4, 4, "v_scale", false, !kept),
                      flat(c.pages, cache_bytes(c), 16, "pages", true, !kept || c.num_pages == 0),
                      matrix(q_out, T, q_heads * D, ldqo, "q_out", true, false, q, ldq),
                      matrix(k_out, T, k_heads * D, ldko, "k_out", true, kept, k, ldk)};
    TS_TRY(check_rows_of(b, T == 0));
    if (T == 0)
        return ok();
    RopeArgs a{};
    a.q = u16(q);
    a.k = u16(k);
    a.v = u16(v);
    a.ldq = ldq;
    a.ldk = ldk;
    a.ldv = ldv;
    a.T = T;
    a.hq = (int)q_heads;
    a.hk = (int)k_heads;
    a.D = (int)D;
    a.lanes_log2 = lanes_log2(D);
    a.qw = u16(q_weight);
    a.kw = u16(k_weight);
    a.eps = eps;
    a.pos = positions;
    a.table = cos_sin;
    a.max_pos = (int)max_pos;
    a.rot = (int)rot;
    a.pairs = interleaved != 0;
    a.q_out = static_cast<uint16_t *>(q_out);
    a.k_out = static_cast<uint16_t *>(k_out);
    a.ldqo = ldqo;
    a.ldko = ldko;
    if (kept)
        a.cache = cache_args(c);
    a.slots = slots;
    a.keep = kept;
    return launched(launch_rope(a, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

extern "C" int64_t ts_qk_norm_rope_grad_workspace(int64_t head_dim)
{
    if (head_dim < 16 || head_dim > 256 || head_dim % 16 != 0)
        return -1;
    return (int64_t)kGradBlocks * 2 * head_dim * 4;
}

extern "C" int ts_qk_norm_rope_grad(const void *dq_out, int64_t lddqo, const void *dk_out, int64_t lddko, const void *q,
                                    int64_t ldq, const void *k, int64_t ldk, int64_t T, int64_t q_heads, int64_t k_heads,
                                    int64_t head_dim, const void *q_weight, const void *k_weight, float eps,
                                    const int32_t *positions, const float *cos_sin, int64_t max_pos, int64_t rot,
                                    int interleaved, void *dq, int64_t lddq, void *dk, int64_t lddk, float *dq_weight,
                                    float *dk_weight, void *workspace, uint32_t flags, void *stream)
{
    const int64_t D = head_dim;
    TS_TRY(check_flag_bits(flags));
    TS_TRY(check_rope(T, q_heads, k_heads, D, max_pos, rot, interleaved, eps));
    TS_TRY(check_ld("lddqo", lddqo, q_heads * D));
    TS_TRY(check_ld("lddko", lddko, k_heads * D));
    TS_TRY(check_ld("ldq", ldq, q_heads * D));
    TS_TRY(check_ld("ldk", ldk, k_heads * D));
    TS_TRY(check_ld("lddq", lddq, q_heads * D));
    TS_TRY(check_ld("lddk", lddk, k_heads * D));
    const bool norm = q_weight != nullptr;
    if (norm != (k_weight != nullptr))
        return fail(TS_ERR_UNSUPPORTED, "q_weight and k_weight are given together or not at all");
    if (!norm && (dq_weight != nullptr || dk_weight != nullptr))
        return fail(TS_ERR_UNSUPPORTED, "gradients of weights that are not given");
    const bool empty = T == 0;
    const Rows b[] = {matrix(dq_out, T, q_heads * D, lddqo, "dq_out", false, empty),
                      matrix(dk_out, T, k_heads * D, lddko, "dk_out", false, empty),
                      matrix(q, T, q_heads * D, ldq, "q", false, empty),
                      matrix(k, T, k_heads * D, ldk, "k", false, empty),
                      flat(q_weight, D * 2, 16, "q_weight", false, true),
                      flat(k_weight, D * 2, 16, "k_weight", false, true),
                      flat(positions, T * 4, 4, "positions", false, empty),
                      flat(cos_sin, max_pos * rot * 4, 16, "cos_sin", false, empty),
                      matrix(dq, T, q_heads * D, lddq, "dq", true, empty, dq_out, lddqo),
                      matrix(dk, T, k_heads * D, lddk, "dk", true, empty, dk_out, lddko),
                      flat(dq_weight, D * 4, 4, "dq_weight", true, !norm),
                      flat(dk_weight, D * 4, 4, "dk_weight", true, !norm),
                      flat(workspace, norm ? ts_qk_norm_rope_grad_workspace(D) : 0, 16, "workspace", true, !norm)};
    TS_TRY(check_rows_of(b, false));
    if (empty && !norm)
        return ok();
    RopeGradArgs a{};
    a.dy[0] = u16(dq_out);
    a.dy[1] = u16(dk_out);
    a.x[0] = u16(q);
    a.x[1] = u16(k);
    a.lddy[0] = lddqo;
    a.lddy[1] = lddko;
    a.ldx[0] = ldq;
    a.ldx[1] = ldk;
    a.T = T;
    a.heads[0] = (int)q_heads;
    a.heads[1] = (int)k_heads;
    a.D = (int)D;
    a.lanes_log2 = lanes_log2(D);
    a.w[0] = u16(q_weight);
    a.w[1] = u16(k_weight);
    a.eps = eps;
    a.pos = positions;
    a.table = cos_sin;
    a.max_pos = (int)max_pos;
    a.rot = (int)rot;
    a.pairs = interleaved != 0;
    a.dx[0] = static_cast<uint16_t *>(dq);
    a.dx[1] = static_cast<uint16_t *>(dk);
    a.lddx[0] = lddq;
    a.lddx[1] = lddk;
    a.dw[0] = dq_weight;
    a.dw[1] = dk_weight;
    a.partial = static_cast<float *>(workspace);
    return launched(launch_rope_grad(a, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

extern "C" int ts_kv_cache_read(const ts_kv_cache_t *cache, const int32_t *slots, int64_t T, void *k_out, int64_t ldk,
                                void *v_out, int64_t ldv, uint32_t flags, void *stream)
{
    TS_TRY(check_flag_bits(flags));
    TS_TRY(check_range("T", T, 0, kMaxRows));
    if (cache == nullptr)
        return fail(TS_ERR_NULL, "cache is NULL");
    const ts_kv_cache_t c = *cache;
    TS_TRY(check_cache(c));
    const int64_t cols = c.heads * c.head_dim;
    TS_TRY(check_range("T * heads", T * c.heads, 0, kMaxHeadRows));
    if (k_out != nullptr)
        TS_TRY(check_ld("ldk", ldk, cols));
    if (v_out != nullptr)
        TS_TRY(check_ld("ldv", ldv, cols));
    const Rows b[] = {flat(c.pages, cache_bytes(c), 16, "pages", false, c.num_pages == 0),
                      flat(c.k_scale, 4, 4, "k_scale"),
                      flat(c.v_scale, 4, 4, "v_scale"),
                      flat(slots, T * 4, 4, "slots"),
                      matrix(k_out, T, cols, ldk, "k_out", true, true),
                      matrix(v_out, T, cols, ldv, "v_out", true, true)};
    TS_TRY(check_rows_of(b, T == 0));
    if (T == 0 || (k_out == nullptr && v_out == nullptr))
        return ok();
    CacheReadArgs a{};
    a.cache = cache_args(c);
    a.D = (int)c.head_dim;
    a.lanes_log2 = lanes_log2(c.head_dim);
    a.slots = slots;
    a.T = T;
    a.out[0] = static_cast<uint16_t *>(k_out);
    a.out[1] = static_cast<uint16_t *>(v_out);
    a.ld[0] = ldk;
    a.ld[1] = ldv;
    return launched(launch_cache_read(a, (flags & TS_FLAG_PDL) != 0, static_cast<cudaStream_t>(stream)));
}

namespace {

int check_attention(int64_t q_heads, int64_t heads, int64_t D, int64_t max_q)
{
    TS_TRY(check_range("q_heads", q_heads, 1, kMaxHeads));
    TS_TRY(check_range("cache heads", heads, 1, kMaxHeads));
    if (q_heads % heads != 0)
        return fail(TS_ERR_SHAPE, "q_heads = %lld is not a multiple of the cache's %lld heads", (long long)q_heads,
                    (long long)heads);
    if (D != 64 && D != 128)
        return fail(TS_ERR_UNSUPPORTED, "head_dim = %lld: attention takes 64 or 128", (long long)D);
    return check_range("max_q", max_q, 1, kMaxRows);
}

// Which kernel: rows of a sequence that share a key head, for the kernel of few rows at most.
// Few against many rows, us, 1 sequence of 1024 keys, 8 up to 2048, 32 up to 8192, 8 key heads:
//   D = 128   32 rows 8.6 / 20.8, 17.2 / 24.5, 121.6 / 117.1    40 rows 13.8 / 20.8, 24.6 / 22.7, 127 / 117
//   D = 64    32 rows 7.0 / 18.0, 12.8 / 21.7,  87.7 /  99.8    48 rows 12.4 / 18.0, 16.9 / 20.1, 80.5 / 81.1
constexpr int64_t few_rows(int64_t D) { return D == 64 ? 48 : 32; }

int64_t attention_workspace(int64_t B, int64_t heads, int64_t rows, int64_t D, int64_t keys, int64_t window)
{
    if (rows <= few_rows(D) && attn_few_clusters(B, heads, rows, keys, window))
        return 0;
    const int64_t few = attn_few_workspace(D), prompt = rows <= few_rows(D) ? 0 : attn_prompt_workspace(D);
    return few > prompt ? few : prompt;  // (does not shrink where a bound grows)
}

}  // namespace

extern "C" int64_t ts_nvfp4_attention_workspace(int64_t B, int64_t q_heads, int64_t heads, int64_t head_dim, int64_t max_q,
                                                int64_t max_keys, int64_t window)
{
    if (check_attention(q_heads, heads, head_dim, max_q) != TS_OK || B < 0 || B > 65536 || max_keys < 0 || max_keys > kMaxKeys ||
        window < 0 || window > kMaxRows)
        return -1;
    return attention_workspace(B, heads, max_q * (q_heads / heads), head_dim, max_keys, window);
}

extern "C" int ts_nvfp4_attention(const void *q, int64_t ldq, int64_t T, int64_t q_heads, const int32_t *cu_q, int64_t B,
                                  int64_t max_q, const ts_kv_cache_t *cache, const int32_t *block_table, int64_t max_pages,
                                  const int32_t *kv_lens, float scale, int causal, int64_t window, void *out, int64_t ldo,
                                  float *lse, void *workspace, uint32_t flags, void *stream)
{
    TS_TRY(check_flag_bits(flags));
    if (cache == nullptr)
        return fail(TS_ERR_NULL, "cache is NULL");
    const ts_kv_cache_t c = *cache;
    TS_TRY(check_cache(c));
    const int64_t D = c.head_dim;
    TS_TRY(check_attention(q_heads, c.heads, D, max_q));
    TS_TRY(check_range("T", T, 0, kMaxRows));
    TS_TRY(check_range("T * q_heads", T * q_heads, 0, kMaxHeadRows));
    TS_TRY(check_range("B", B, 0, 65536));
    if (cu_q == nullptr && T != B)
        return fail(TS_ERR_SHAPE, "T = %lld queries of B = %lld sequences need cu_q", (long long)T, (long long)B);
    TS_TRY(check_range("max_pages", max_pages, 0, kMaxKeys / c.page_size));
    TS_TRY(check_ld("ldq", ldq, q_heads * D));
    TS_TRY(check_ld("ldo", ldo, q_heads * D));
    if (!(scale > 0.0f) || std::isinf(scale))
        return fail(TS_ERR_UNSUPPORTED, "scale = %g must be finite and positive", (double)scale);
    TS_TRY(check_range("causal", causal, 0, 1));
    TS_TRY(check_range("window", window, 0, kMaxRows));
    if (window > 0 && causal == 0)
        return fail(TS_ERR_UNSUPPORTED, "a window needs causal");
    const int64_t rows = max_q * (q_heads / c.heads);
    const int64_t space = attention_workspace(B, c.heads, rows, D, max_pages * c.page_size, window);
    const Rows b[] = {matrix(q, T, q_heads * D, ldq, "q"),
                      flat(cu_q, (B + 1) * 4, 4, "cu_q", false, true),
                      flat(c.pages, cache_bytes(c), 16, "pages", false, c.num_pages == 0),
                      flat(c.k_scale, 4, 4, "k_scale"),
                      flat(c.v_scale, 4, 4, "v_scale"),
                      flat(block_table, B * max_pages * 4, 4, "block_table", false, max_pages == 0),
                      flat(kv_lens, B * 4, 4, "kv_lens"),
                      matrix(out, T, q_heads * D, ldo, "out", true),
                      flat(lse, T * q_heads * 4, 4, "lse", true, true),
                      flat(workspace, space, 16, "workspace", true, space == 0)};
    const bool empty = T == 0 || B == 0;
    TS_TRY(check_rows_of(b, empty));
    if (empty)
        return ok();
    AttnArgs a{};
    a.q = u16(q);
    a.ldq = ldq;
    a.T = T;
    a.hq = (int)q_heads;
    a.group = (int)(q_heads / c.heads);
    a.div_group = div_magic((uint32_t)a.group);
    a.cu = cu_q;
    a.B = (int)B;
    a.cache = cache_args(c);
    a.D = (int)D;
    a.table = block_table;
    a.max_pages = max_pages;
    a.lens = kv_lens;
    a.scale = scale;
    a.causal = causal != 0;
    a.window = (int)(window < kMaxKeys ? window : kMaxKeys);  // (a row's position less it stays within 32 bits)
    a.out = static_cast<uint16_t *>(out);
    a.ldo = ldo;
    a.lse = lse;
    a.partial = static_cast<float *>(workspace);
    const bool pdl = (flags & TS_FLAG_PDL) != 0;
    const cudaStream_t on = static_cast<cudaStream_t>(stream);
    return launched(rows <= few_rows(D) ? launch_attn_few(a, rows, pdl, on) : launch_attn_prompt(a, pdl, on));
}
