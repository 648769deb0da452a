// Internal interface between the checks of the attention entry points
// (api_attention.cu) and their launchers.  Sizes are validated; positions, slots,
// lengths and tables are not, and the kernels check them.  As in launch_nvfp4.h, no
// input is read through the non-coherent path.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "launch.h"

namespace tsfn {

// The paged cache; offsets as documented for ts_kv_cache_t.
struct CacheArgs {
    uint8_t *pages;
    int64_t slots;     // num_pages * page_size
    int num_pages;
    int page_size;
    DivMagic div_page;  // division by page_size
    int heads;
    const float *k_scale;
    const float *v_scale;
};

struct RopeArgs {
    const uint16_t *q, *k, *v;  // v: with a cache only
    int64_t ldq, ldk, ldv;
    int64_t T;
    int hq, hk, D;
    int lanes_log2;  // lanes of a head's row: 8 columns each
    const uint16_t *qw, *kw;  // both or neither
    float eps;
    const int32_t *pos;
    const float *table;
    int max_pos, rot;
    bool pairs;
    uint16_t *q_out, *k_out;  // k_out may be null with a cache
    int64_t ldqo, ldko;
    bool keep;  // with a cache
    CacheArgs cache;
    const int32_t *slots;
    // a run: up to run_heads heads of one token; runs of a token's q, of its k, of k and v
    int run_heads, runs_q, runs_k, runs_kv;
    int q_blocks, kv_blocks, kv_every;  // blocks of runs of each; every kv_every-th is of the latter
    float one;  // 1, for add_products2
    DivMagic div_q, div_kv, div_every;  // division by runs_q, runs_kv, kv_every
};

struct RopeGradArgs {
    const uint16_t *dy[2], *x[2];  // q, k
    int64_t lddy[2], ldx[2];
    int64_t T;
    int heads[2];
    int D, lanes_log2;
    const uint16_t *w[2];
    float eps;
    const int32_t *pos;
    const float *table;
    int max_pos, rot;
    bool pairs;
    uint16_t *dx[2];
    int64_t lddx[2];
    float *dw[2];
    float *partial;  // [blocks, 2, D]
    DivMagic div_heads[2];
};

struct CacheReadArgs {
    CacheArgs cache;
    int D, lanes_log2;
    const int32_t *slots;
    int64_t T;
    uint16_t *out[2];
    int64_t ld[2];
};

struct AttnArgs {
    const uint16_t *q;
    int64_t ldq;
    int64_t T;
    int hq, group;  // query heads, and those of a key head
    DivMagic div_group;
    const int32_t *cu;  // may be null: one query a sequence
    int B;
    CacheArgs cache;
    int D;
    const int32_t *table;
    int64_t max_pages;
    const int32_t *lens;
    float scale;
    bool causal;
    int window;  // 0: none
    uint16_t *out;
    int64_t ldo;
    float *lse;
    float *partial;
};

// Blocks of the gradient: five for each of 152 SMs.
constexpr int kGradBlocks = 760;

cudaError_t launch_rope(const RopeArgs &a, bool pdl, cudaStream_t stream);
cudaError_t launch_rope_grad(const RopeGradArgs &a, bool pdl, cudaStream_t stream);
cudaError_t launch_cache_read(const CacheReadArgs &a, bool pdl, cudaStream_t stream);

// Attention of few rows (queries x heads of a key head) at a time, and of many.
cudaError_t launch_attn_few(const AttnArgs &a, int64_t rows, bool pdl, cudaStream_t stream);
int64_t attn_few_workspace(int64_t D);
// Whether the first needs no workspace: units by clusters.  keys: a bound of a sequence's.
bool attn_few_clusters(int64_t B, int64_t heads, int64_t rows, int64_t keys, int64_t window);
cudaError_t launch_attn_prompt(const AttnArgs &a, bool pdl, cudaStream_t stream);
int64_t attn_prompt_workspace(int64_t D);
cudaError_t read_attn_stalled_waits(uint32_t *count);

}  // namespace tsfn
