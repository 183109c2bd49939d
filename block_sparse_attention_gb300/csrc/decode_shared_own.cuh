// decode_shared_own.cuh -- a decode over shared prefixes: the sequences' own tokens (decode_shared.cu calls this).
//
// Each byte of a sequence's own K and V is used once, by the G <= 8 query heads of its kv head, so HBM bandwidth
// bounds this; sequences have few own tokens or many.  Every warp is by itself: an equal part of all units of 32
// keys, for one kv head, from one sequence to the next without a break (the next sequence's K, V and queries are
// on their way before the one before is done), and what it has of a sequence goes to the workspace as a piece.
// The products are those of decode_stream.cu, transposed, so that the G heads are the n = 8 side of mma.sync
// m16n8k16: S^T [16 keys x 8] = K Q^T and O^T [d x 8] += V^T P^T.
// An SM does 124 GB/s so (d = 128, its 12 warps, 192 KB on their way): each byte is written to shared memory and read
// from it once, and 128 bytes a cycle allow no more than 130.  The whole GPU is at 6.2 TB/s, a quarter of it at 4.7.
// Units of 64 keys by six warps: the same; of 16 keys: half of it.
#pragma once

#include <climits>
#include <cmath>
#include <type_traits>

#include "decode_shared.cuh"
#include "mma16.cuh"
#include "ptx.cuh"

namespace bsattn {

constexpr int kOwnWarps = kSharedThreads / 32;           // of a CTA, 16 KB of shared memory each
constexpr int kStretches = 512;                          // of sequences, a thread each; the last ones are empty
static_assert(kSharedThreads <= kStretches, "a thread a stretch");
constexpr int kTok = 32, kTiles = kTok / 16;             // keys of a unit
// exp2 is taken of x - max + 12: weights up to 4096, so that a weight 2^-24 of the largest is
// still a normal fp16 number and 2^-36 the smallest one
constexpr float kWeightLog2 = 12.f;
// What is taken off x.  In fp16 rounded up, so that no weight passes 2^12 where scores are so large that 32 bits have them
// to the nearest 8 or more; bf16 has room for that.
template <bool BF16>
__device__ __forceinline__ float weight_reference(float top) {
    return BF16 ? top - kWeightLog2 : __fadd_ru(top, -kWeightLog2);
}
template <bool BF16>
__device__ __forceinline__ float log_sum(float top, float sum) {
    if (sum == 0.f) return -INFINITY;
    return BF16 ? top + log2f(sum) - kWeightLog2 : weight_reference<BF16>(top) + log2f(sum);
}

template <int D>
struct OwnRing {
    static constexpr int kStages = 2 * (128 / D);        // K or V of a unit each
    static constexpr uint32_t kStage = kTok * D * 2;
    static constexpr uint32_t kRing = kStages * kStage;  // of one warp
    static constexpr uint32_t kBars = kOwnWarps * kRing; // full[warp][stage]
    static constexpr uint32_t kInfo = kBars + 8 * kOwnWarps * kStages;    // (sequence, keys) of a stage
    static constexpr uint32_t kUpto = kInfo + 8 * kOwnWarps * kStages;    // [kStretches] units up to a stretch's end
    static constexpr uint32_t kBytes = kUpto + 8 * kStretches;
    static_assert(kStage % 1024 == 0, "swizzled tiles start on 1024 bytes");
};

// One warp's part, for kv head g, of the units of all sequences.  `sm` is on 1024 bytes; the CTA has written upto_of
// there, set up the barriers, and met at a barrier since.  Parts from the last unit on are empty.
template <int D, bool BF16>
__device__ __forceinline__ void own_tokens(const CUtensorMap* tm_k, const CUtensorMap* tm_v, const SharedCall& p, uint8_t* sm,
                                           volatile int* abort_flag, int part, int g, long long chunk, long long total) {
    using namespace mma16;
    using R = OwnRing<D>;
    using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
    constexpr int kStages = R::kStages;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint8_t* ring = sm + warp * R::kRing;
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + R::kBars) + warp * kStages;
    volatile int2* info = reinterpret_cast<int2*>(sm + R::kInfo) + warp * kStages;
    const long long* upto_of = reinterpret_cast<const long long*>(sm + R::kUpto);
    const int G = p.Hq / p.Hkv;
    const int per = (p.B + kSharedThreads - 1) / kSharedThreads;        // sequences of a stretch
    const long long x0 = part * chunk;
    const int n = static_cast<int>(min(chunk, total - x0));     // units of this warp
    if (x0 >= total) return;

    // the next batch of units begins at unit `cu` of sequence `cb`
    int cb, cu;
    {
        int t = 0;
#pragma unroll
        for (int step = kStretches / 2; step > 0; step >>= 1)
            if (upto_of[t + step - 1] <= x0) t += step;
        long long before = t > 0 ? upto_of[t - 1] : 0;
        cb = t * per;
        for (;; ++cb) {
            const int u = own_units(own_len(p, cb));
            if (x0 < before + u) break;
            before += u;
        }
        cu = static_cast<int>(x0 - before);
    }

    // ---------------------------------------------------------------- feeding
    // Lane i knows sequence, cache row and keys of the warp's unit base + i, for `count` of them.
    int base = 0, count = 0;
    int look_b = 0, look_row = -1, look_keys = 0;
    bool bad = false;
    const auto look_up = [&] {
        base += count;
        for (;;) {
            // lane i: sequence cb + i; `ends`: units up to its end
            const int len = cb + lane < p.B ? own_len(p, cb + lane) : 0;
            int ends = own_units(len);
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, ends, o);
                if (lane >= o) ends += u;
            }
            const int have = __shfl_sync(0xffffffffu, ends, 31) - cu;
            if (have <= 0) {
                cb += 32;
                cu = 0;
                continue;
            }
            count = min(have, 32);
            // the sequence that unit cu + lane is of, and (for the next batch) unit cu + count
            const auto find = [&](int u) {
                int s = 0;
#pragma unroll
                for (int half = 16; half > 0; half >>= 1)
                    if (__shfl_sync(0xffffffffu, ends, s + half - 1) <= u) s += half;
                if (__shfl_sync(0xffffffffu, ends, s) <= u) ++s;
                return s;
            };
            const int s = find(cu + lane), next = find(cu + count);
            const int before = __shfl_sync(0xffffffffu, ends, (s - 1) & 31), len_s = __shfl_sync(0xffffffffu, len, s & 31);
            const int next_before = __shfl_sync(0xffffffffu, ends, (next - 1) & 31);
            look_b = cb + s;
            look_row = -1;
            look_keys = 0;
            if (lane < count) {
                const int key = (cu + lane - (s > 0 ? before : 0)) * kTok, lp = key / p.page_size;
                const int page = lp < p.own_pages ? p.own_table[static_cast<size_t>(look_b) * p.own_pages + lp] : -1;
                if (page < 0 || page >= p.num_pages) {
                    bad = true;
                } else {
                    look_row = page * p.page_size + key - lp * p.page_size;
                    look_keys = min(len_s - key, kTok);
                }
            }
            cu = cu + count - (next > 0 ? next_before : 0);
            cb += next;
            return;
        }
    };
    const uint64_t once = l2_evict_first();
    int issued = 0;
    // Half h is K of unit h / 2 if h is even, its V if it is odd.
    const auto issue = [&](int h) {
        ++issued;
        const int k = h >> 1;
        if (k >= base + count) look_up();
        const int row = __shfl_sync(0xffffffffu, look_row, k - base);
        const int keys = __shfl_sync(0xffffffffu, look_keys, k - base);
        const int b = __shfl_sync(0xffffffffu, look_b, k - base);
        const int st = h % kStages;
        if (lane == 0) {
            info[st].x = b;
            info[st].y = keys;
            if (row < 0) {
                mbar_arrive(&full[st]);                             // nothing to load: the unit is skipped
            } else {
                mbar_arrive_expect_tx(&full[st], R::kStage);
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    tma_load_3d(ring + st * R::kStage + c * (kTok * 128), h & 1 ? tm_v : tm_k, &full[st], c * 64, g, row, once);
            }
        }
        __syncwarp();
    };
    // the four channels of head lane / 4 that the lane's K registers hold in each k16 step
    const auto queries = [&](int b, uint32_t (&to)[D / 16][2]) {
        const T* qg = static_cast<const T*>(p.q) + (static_cast<size_t>(b) * p.Hq + g * G) * D;
        const int hq = lane >> 2, j = lane & 3;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
            const T* src = qg + hq * D + kk * 16 + 2 * j;
            to[kk][0] = hq < G ? __ldg(reinterpret_cast<const uint32_t*>(src)) : 0u;
            to[kk][1] = hq < G ? __ldg(reinterpret_cast<const uint32_t*>(src + 8)) : 0u;
        }
    };

    const int r8 = lane >> 2, j4 = lane & 3;
    for (int h = 0; h < kStages && h < 2 * n; ++h) issue(h);
    uint32_t qb[D / 16][2], qn[D / 16][2];
    float o[D / 16][4];
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;     // l of this lane's keys only
    int cur = info[0].x;
    queries(cur, qb);
    const auto begin = [&] {
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        m0 = m1 = -INFINITY;
        l0 = l1 = 0.f;
    };
    // The piece of sequence b to the workspace.
    const auto end = [&](int b) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, w);
            l1 += __shfl_xor_sync(0xffffffffu, l1, w);
        }
        const size_t row = ((static_cast<size_t>(part) + b) * p.Hkv + g) * G + 2 * j4;
        const float inv0 = l0 == 0.f ? 0.f : 1.f / l0, inv1 = l1 == 0.f ? 0.f : 1.f / l1;
        if (r8 == 0) {
            if (2 * j4 < G) p.own_lse[row] = log_sum<BF16>(m0, l0);
            if (2 * j4 + 1 < G) p.own_lse[row + 1] = log_sum<BF16>(m1, l1);
        }
        float* to = p.own_o + row * D + r8;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) {
            if (2 * j4 < G) {
                to[16 * mt] = o[mt][0] * inv0;
                to[16 * mt + 8] = o[mt][2] * inv0;
            }
            if (2 * j4 + 1 < G) {
                to[D + 16 * mt] = o[mt][1] * inv1;
                to[D + 16 * mt + 8] = o[mt][3] * inv1;
            }
        }
    };
    begin();
    int done = 0, begun = 0;                                     // units
    // Waits for half h; issues half h + kStages into its stage once it is read.
    const auto arrived = [&](int h) {
        const bool ok = warp_wait_within(&full[h % kStages], (h / kStages) & 1, p.budget_ns, abort_flag, p.status);
        __syncwarp();
        return ok;
    };
    const auto consumed = [&](int h) {
        __syncwarp();
        if (h + kStages < 2 * n) issue(h + kStages);
    };
    for (; done < n; ++done) {
        const int hk = 2 * done;
        if (!arrived(hk)) break;
        const uint8_t* stage = ring + (hk % kStages) * R::kStage;
        const int b = info[hk % kStages].x, keys = info[hk % kStages].y;
        begun = done + 1;
        if (b != cur) {
            end(cur);
            begin();
            cur = b;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                qb[kk][0] = qn[kk][0];
                qb[kk][1] = qn[kk][1];
            }
        }
        // the queries of the sequence that begins with the next unit
        const auto look_ahead = [&] {
            if (done + 1 >= n) return;
            const int next = info[(hk + 2) % kStages].x;
            if (next != cur) queries(next, qn);
        };
        if (keys == 0) {                                            // no page
            consumed(hk);
            look_ahead();
            if (!arrived(hk + 1)) break;
            consumed(hk + 1);
            continue;
        }
        float x[kTiles][4];
        const uint32_t kbase = smem_u32(stage);
        const int mat = lane >> 3;
#pragma unroll
        for (int mt = 0; mt < kTiles; ++mt) {
            float sc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int col = kk * 16 + (mat >> 1) * 8;
                uint32_t a[4];
                ldsm4(kbase + (col >> 6) * (kTok * 128) + sw128_offset(16 * mt + (mat & 1) * 8 + (lane & 7), col & 63), a);
                mma16816<BF16>(sc, a, qb[kk][0], qb[kk][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
                x[mt][e] = 16 * mt + r8 + 8 * (e >> 1) < keys ? sc[e] * p.scale_log2 : -INFINITY;
        }
        consumed(hk);
        look_ahead();
        float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
        for (int mt = 0; mt < kTiles; ++mt) {
            t0 = fmaxf(t0, fmaxf(x[mt][0], x[mt][2]));
            t1 = fmaxf(t1, fmaxf(x[mt][1], x[mt][3]));
        }
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
            t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, w));
            t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, w));
        }
        if (__any_sync(0xffffffffu, t0 > m0 || t1 > m1)) {
            const float n0 = fmaxf(m0, t0), n1 = fmaxf(m1, t1);
            const float a0 = ex2_approx(m0 - (n0 == -INFINITY ? 0.f : n0));
            const float a1 = ex2_approx(m1 - (n1 == -INFINITY ? 0.f : n1));
            m0 = n0;
            m1 = n1;
            l0 *= a0;
            l1 *= a1;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                o[mt][0] *= a0;
                o[mt][1] *= a1;
                o[mt][2] *= a0;
                o[mt][3] *= a1;
            }
        }
        const float z0 = m0 == -INFINITY ? 0.f : weight_reference<BF16>(m0);
        const float z1 = m1 == -INFINITY ? 0.f : weight_reference<BF16>(m1);
        uint32_t pb[kTiles][2];
#pragma unroll
        for (int mt = 0; mt < kTiles; ++mt) {
            const float p0 = ex2_approx(x[mt][0] - z0), p1 = ex2_approx(x[mt][1] - z1);
            const float p2 = ex2_approx(x[mt][2] - z0), p3 = ex2_approx(x[mt][3] - z1);
            l0 += p0 + p2;
            l1 += p1 + p3;
            pb[mt][0] = transpose8x8(pack2<BF16>(p0, p1));
            pb[mt][1] = transpose8x8(pack2<BF16>(p2, p3));
        }
        if (!arrived(hk + 1)) break;
        uint8_t* vs = ring + ((hk + 1) % kStages) * R::kStage;
        if (keys < kTok) {
            // rows past the end may hold anything: a weight of 0 must not meet a NaN
            for (int e = lane; e < (kTok - keys) * (D / 8); e += 32) {
                const int r = keys + e / (D / 8), c = e % (D / 8);
                *reinterpret_cast<uint4*>(vs + (c >> 3) * (kTok * 128) + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
        }
        const uint32_t vbase = smem_u32(vs);
#pragma unroll
        for (int mt = 0; mt < kTiles; ++mt)
#pragma unroll
            for (int dt = 0; dt < D / 16; ++dt) {
                const int col = dt * 16 + (mat & 1) * 8;
                uint32_t a[4];
                ldsm4_t(vbase + (col >> 6) * (kTok * 128) + sw128_offset(16 * mt + (mat >> 1) * 8 + (lane & 7), col & 63), a);
                mma16816<BF16>(o[dt], a, pb[mt][0], pb[mt][1]);
            }
        consumed(hk + 1);
    }
    if (done < n) {
        // After a wait that expired: copies in flight land, and every piece that lacks a unit is handed over as NaN.
        const uint64_t dl = global_timer_ns() + 200000000ull;
        for (int h = max(issued - kStages, 0); h < issued; ++h) wait_parity_drain(&full[h % kStages], (h / kStages) & 1, dl);
        l0 = l1 = __int_as_float(0x7fffffff);
        end(cur);
        for (int k = begun; k < n; ++k) {
            // units on their way are noted at their stages, the others come after them in the batch or in later ones
            if (2 * k >= issued && k >= base + count) look_up();
            const int b = 2 * k < issued ? info[2 * k % kStages].x : __shfl_sync(0xffffffffu, look_b, k - base);
            if (b != cur) {
                cur = b;
                end(cur);
            }
        }
    } else {
        end(cur);
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.status, BSATTN_ERR_BAD_INDEX);
}

}  // namespace bsattn
