// summary.cuh -- the 8-bit summary of a block of 64 rows, and the order of scores.
//
// A block's rows are added in 32 bits, in halves (row i to row i + 32, then i + 16, ... i + 1; rows that
// are not there count as 0), and divided by their number.  The mean's codes are its multiples of the scale
// amax / 127, to the nearest (ties to even).  Every step is one correctly rounded operation in a fixed
// order, so that a block has one summary wherever it is taken; and a product of two summaries' codes is a
// whole number below 2^21, exact in any order of adding.  A choice by scores therefore does not depend
// on how the work is split.
// A mean with a channel that is not finite has codes 0 and the scale +infinity.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>
#include <cstdint>

#include "bsattn.h"

namespace bsattn {

constexpr int kBlockRows = 64;

template <bool BF16>
__device__ __forceinline__ float2 two_floats(uint32_t w) {
    if constexpr (BF16) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        return __half22float2(*reinterpret_cast<__half2*>(&w));
    }
}

// The scale of values whose largest magnitude is `top` (infinity or NaN: not finite).
__device__ __forceinline__ float scale8(float top, bool finite) { return finite ? __fdiv_rn(top, 127.f) : INFINITY; }

// A value's code, in [-127, 127].  (The clamp is for scales that are subnormal and so rounded coarsely.)
__device__ __forceinline__ int code8(float x, float scale, bool finite) {
    if (!finite || scale == 0.f) return 0;
    return max(min(__float2int_rn(__fdiv_rn(x, scale)), 127), -127);
}

// Whole numbers that order as scores do; 0 stands below all of them, and so for a place that may not be
// chosen.  -0 counts as 0.
constexpr uint32_t kForced = 0xffffffffu;        // above every score
__device__ __forceinline__ uint32_t key_of(float score) {
    const int u = __float_as_int(score + 0.f);
    return static_cast<uint32_t>(u ^ ((u >> 31) | static_cast<int>(0x80000000u)));
}
__device__ __forceinline__ float score_of(uint32_t key) {
    const int k = static_cast<int>(key);
    return __int_as_float(k < 0 ? k ^ static_cast<int>(0x80000000u) : ~k);
}

// A key between lo and hi (hi - lo > 1) at which the next count is taken: the mean of the two scores for
// the first steps, which halves what lies between them wherever the scores are spread evenly, then the
// middle of the keys, which ends after 32 steps whatever they are.
__device__ __forceinline__ uint32_t between(uint32_t lo, uint32_t hi, int step) {
    const float a = score_of(lo), b = score_of(hi);
    uint32_t mid = lo + (hi - lo) / 2;
    if (step < 16 && isfinite(a) && isfinite(b)) mid = key_of(0.5f * a + 0.5f * b);
    return max(min(mid, hi - 1), lo + 1);
}

// NT rising keys between lo and hi at which the next counts are taken, likewise: equal parts of the scores' range for
// the first eight steps, then of the keys'.  Where fewer lie between, some are given twice.
template <int NT>
__device__ __forceinline__ void thresholds(uint32_t lo, uint32_t hi, int step, uint32_t (&t)[NT]) {
    const float a = score_of(lo), b = score_of(hi), by = (b - a) * (1.f / (NT + 1));
    const bool even = step < 8 && isfinite(a) && isfinite(b) && isfinite(by);
    const uint32_t gap = hi - lo;
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const uint32_t mid = even ? key_of(fmaf(by, static_cast<float>(i + 1), a))
                                  : lo + gap / (NT + 1) * (i + 1) + gap % (NT + 1) * (i + 1) / (NT + 1);
        t[i] = max(min(mid, hi - 1), lo + 1);
        if (i > 0) t[i] = max(t[i], t[i - 1]);
    }
}

// A warp's sum of a block's rows: lane l holds channels 8 (l % (D / 8)) + 0 .. 7 of it, all lanes with the
// same channels the same.  `row(r)` gives the address of the lane's 16 bytes of row r < count.
template <int D, bool BF16, typename Row>
__device__ __forceinline__ void block_sum(Row row, int count, float (&sum)[8]) {
    constexpr int kAt = 256 / D;              // rows that a warp reads at once: 2 or 4
    constexpr int kEach = kBlockRows / kAt;   // rows of a lane: 32 or 16, row kAt j + sub
    const int sub = (threadIdx.x & 31) / (D / 8);
    // 16 rows in flight a lane: with row kAt j + sub the halves of 32, 16, 8 (and 4) rows are a lane's own
#pragma unroll
    for (int batch = 0; batch < kEach / 16; ++batch) {
        uint4 raw[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const int r = kAt * (i * (kEach / 16) + batch) + sub;
            raw[i] = r < count ? __ldg(row(r)) : make_uint4(0, 0, 0, 0);
        }
        float x[8];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
            float2 v[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
                v[i] = two_floats<BF16>(c == 0 ? raw[i].x : c == 1 ? raw[i].y : c == 2 ? raw[i].z : raw[i].w);
#pragma unroll
            for (int half = 8; half > 0; half >>= 1)
#pragma unroll
                for (int i = 0; i < half; ++i) {
                    v[i].x = __fadd_rn(v[i].x, v[i + half].x);
                    v[i].y = __fadd_rn(v[i].y, v[i + half].y);
                }
            x[2 * c] = v[0].x;
            x[2 * c + 1] = v[0].y;
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = batch == 0 ? x[e] : __fadd_rn(sum[e], x[e]);
    }
#pragma unroll
    for (int m = 16; m >= D / 8; m >>= 1)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = __fadd_rn(sum[e], __shfl_xor_sync(0xffffffffu, sum[e], m));
}

// The mean of `count` rows with that sum, and from it the lane's eight codes and the block's scale.
template <int D>
__device__ __forceinline__ float summarise(const float (&sum)[8], int count, int (&code)[8]) {
    const float n = static_cast<float>(count);
    float mean[8], top = 0.f;
    bool finite = true;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        mean[e] = __fdiv_rn(sum[e], n);
        const float a = fabsf(mean[e]);
        finite = finite && a <= FLT_MAX;
        top = fmaxf(top, a);
    }
    finite = __all_sync(0xffffffffu, finite);
#pragma unroll
    for (int m = 1; m < D / 8; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    const float scale = scale8(top, finite);
#pragma unroll
    for (int e = 0; e < 8; ++e) code[e] = code8(mean[e], scale, finite);
    return scale;
}

}  // namespace bsattn
