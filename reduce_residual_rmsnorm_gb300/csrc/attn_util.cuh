// What the two attention kernels share: the sequences of a call, the parts that blocks
// leave for one another, and NVFP4 to fp16.
#pragma once

#include <cstdint>

#include "launch_attention.h"

namespace tsfn {

// p is exp2(score - top) 2^kLift, so that fp16 keeps what is far below the largest: 11 bits
// down to 2^-21 of it, and something down to 2^-32.  The top follows a score only when that
// passes it by 2^kSlack; p stays below 2^(kLift + kSlack), fp16's end at 2^16.  What is kept
// of a row as its maximum is top - kLift: sums and outputs of parts go with that.
constexpr float kLift = 7.0f, kSlack = 8.0f;
// Scores from here on are rounded before the top is taken off them: their neighbouring fp32
// are 2 and more apart, and one operation for both would leave what the top's own rounding
// lost, up to any power of two.
constexpr float kFar = 0x1p24f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// What a block leaves for a unit that it began and others go on with.
struct Record {
    int32_t last;   // the last block of the unit, or -1: nothing to join
    int32_t q0;     // the sequence's first query
    int32_t head;   // key head
    int32_t rows;   // rows of the unit
    int64_t row0;   // the unit's first row among the sequence's (query, head) pairs
};

__host__ __device__ constexpr int64_t slot_floats(int rows, int D) { return (int64_t)rows * (D + 2); }

struct Seq {
    int q0;
    int n;      // queries (n * group < 2^30, as T * q_heads)
    int len;    // keys
    int first;  // first tile of 16 keys that a query sees
    int tiles;  // at least 1
    int parts;  // row tiles
};

template <int NR>
__device__ __forceinline__ Seq sequence(const AttnArgs &a, int b)
{
    Seq s;
    if (a.cu != nullptr) {
        const int T = (int)a.T;
        int lo = a.cu[b], hi = a.cu[b + 1];
        lo = lo < 0 ? 0 : (lo > T ? T : lo);
        hi = hi > T ? T : hi;
        s.q0 = lo;
        s.n = hi > lo ? hi - lo : 0;
    } else {
        s.q0 = b;
        s.n = 1;
    }
    const int64_t room = a.max_pages * a.cache.page_size;
    int64_t len = a.lens[b];
    len = len < 0 ? 0 : (len > room ? room : len);
    s.len = (int)len;
    int64_t lo = a.window > 0 ? len - s.n + 1 - a.window : 0;  // the first query's first key
    lo = lo < 0 ? 0 : lo;
    s.first = (int)(lo >> 4);
    const int last = (int)((len + 15) >> 4);
    s.tiles = last - s.first > 1 ? last - s.first : 1;
    s.parts = (s.n * a.group + NR - 1) / NR;
    return s;
}

__device__ __forceinline__ int64_t weight(const AttnArgs &a, const Seq &s, int way) { return (int64_t)s.parts * a.cache.heads * (s.tiles + way); }

// The power of two that takes a row of q with the largest magnitude amax into [2^7, 2^8),
// where fp16 loses only what is below 2^-33 of amax; and its inverse.
__device__ __forceinline__ float fp16_scale(float amax, float &down)
{
    int e = (int)(__float_as_uint(amax) >> 23) - 127;
    e = e < -119 ? -119 : (e > 126 ? 126 : e);
    down = __uint_as_float((uint32_t)(120 + e) << 23);
    return __uint_as_float((uint32_t)(134 - e) << 23);
}

// What the scores of a row, scaled by 1 / down, are multiplied by to be in units of log2.  Not
// below the smallest normal number (a row of zeros, or tiny scales: the scores are zeros
// then): -inf, where a key is not seen, times 0 would not be -inf.
__device__ __forceinline__ float score_factor(const AttnArgs &a, float down, float k_scale)
{
    const float f = a.scale * kLog2e * down / k_scale;
    return f < 0x1p-126f ? 0x1p-126f : f;
}

__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The codes of byte I of w as two fp16, the low nibble's in the low half.
template <int I>
__device__ __forceinline__ uint32_t e2m1x2(uint32_t w)
{
    uint32_t r;
    if constexpr (I == 0)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (I == 1)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b;\n\t}" : "=r"(r) : "r"(w));
    else if constexpr (I == 2)
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, c;\n\t}" : "=r"(r) : "r"(w));
    else
        asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, d;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

// Two E4M3 in the low 16 bits as two fp16.
__device__ __forceinline__ uint32_t e4m3x2(uint32_t w)
{
    uint32_t r;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int D>
struct Layout {
    static constexpr int kTile = 18 * D;            // bytes
    static constexpr int kRow = D / 2;              // bytes of a key's codes
    static constexpr int kV = 8 * D, kKsf = 16 * D, kVsf = 17 * D;
    static constexpr int kChunks = kTile / 16;
};

}  // namespace tsfn
