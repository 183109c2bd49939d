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
#include "mma16.cuh"

namespace bsattn {

constexpr int kBlockRows = 64;

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

// NT rising keys between lo and hi (hi - lo > 1) at which the next counts are taken: equal parts of the scores' range
// for the first eight steps, which is quick wherever the scores are spread evenly, then of the keys', which ends within
// log 2^32 to the base NT + 1 more whatever they are.  Where fewer lie between, some are given twice.
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

// A warp's blocks on their way to it: stages of 64 rows in shared memory, of which a lane copies and adds up the same
// 16-byte pieces, so that it waits for its own copies only and BYTES a warp are on their way whatever the registers
// hold.  Lane l has channels 8 (l % (D / 8)) + 0 .. 7 of rows kAt j + l / (D / 8).
template <int D, int BYTES = 32768>
struct BlockRing {
    static constexpr int kAt = 256 / D;              // rows that a warp copies at once: 2 or 4
    static constexpr int kEach = kBlockRows / kAt;   // rows of a lane: 32 or 16
    static constexpr int kStage = kBlockRows * D * 2;
    static constexpr int kBytes = BYTES;
    static constexpr int kDepth = kBytes / kStage;   // blocks of 16 or 8 KB: 2 or 4 in 32 KB, 3 or 6 in 48
    uint8_t* at;                                     // the stages from the lane's first piece on

    __device__ __forceinline__ explicit BlockRing(uint8_t* base) : at(base + (threadIdx.x & 31) * 16) {}

    // The block whose first row begins, for the lane's channels, at `first`, a row `step` bytes after another, of
    // which `count` are there; the others come as 0.
    __device__ __forceinline__ void fetch(int stage, const char* first, long long step, int count) const {
        const int sub = (threadIdx.x & 31) / (D / 8);
        const uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(at)) + stage * kStage;
        const char* from = first + sub * step;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const bool on = kAt * j + sub < count;
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + j * 512), "l"(on ? from : first),
                         "r"(on ? 16 : 0)
                         : "memory");
            from += kAt * step;
        }
    }
    __device__ __forceinline__ static void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
    // All but the last kDepth - 1 groups are there.
    __device__ __forceinline__ static void wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory"); }

    // The sums of the lane's channels, all lanes with the same channels the same.
    template <bool BF16>
    __device__ __forceinline__ void sum(int stage, float (&s)[8]) const {
        // with row kAt j + sub the halves of 32, 16, 8, 4 (and 2) rows are a lane's own: eight rows at a time
        constexpr int kParts = kEach / 8;
        const uint8_t* from = at + stage * kStage;
        float y[kParts][8];
#pragma unroll
        for (int part = 0; part < kParts; ++part) {
            uint4 raw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) raw[i] = *reinterpret_cast<const uint4*>(from + (i * kParts + part) * 512);
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                float2 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = mma16::unpack2<BF16>(c == 0 ? raw[i].x : c == 1 ? raw[i].y : c == 2 ? raw[i].z : raw[i].w);
#pragma unroll
                for (int half = 4; half > 0; half >>= 1)
#pragma unroll
                    for (int i = 0; i < half; ++i) {
                        v[i].x = __fadd_rn(v[i].x, v[i + half].x);
                        v[i].y = __fadd_rn(v[i].y, v[i + half].y);
                    }
                y[part][2 * c] = v[0].x;
                y[part][2 * c + 1] = v[0].y;
            }
        }
#pragma unroll
        for (int half = kParts / 2; half > 0; half >>= 1)
#pragma unroll
            for (int i = 0; i < half; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) y[i][e] = __fadd_rn(y[i][e], y[i + half][e]);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[e] = y[0][e];
#pragma unroll
        for (int m = 16; m >= D / 8; m >>= 1)
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = __fadd_rn(s[e], __shfl_xor_sync(0xffffffffu, s[e], m));
    }
};

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
