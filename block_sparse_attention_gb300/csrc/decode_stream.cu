// decode_stream.cu -- one query token per sequence over a paged 4-bit cache, and sliding-window
// decode with sinks over a 16-bit cache, sm_103a.
//
// For query head h of sequence b, reading kv head g = h / (Hq / Hkv), with n = cache_seqlens[b]:
//     out = sum_j p_j v_j / sum_j p_j,   p_j = exp(q . k_j / sqrt(d)),   j over the visible tokens
// Visible is every j < n; or, with a window w and s sinks, j < s or j >= n - w; or the tokens of
// the chosen 64-token blocks (4-bit cache).  No visible token gives exactly 0.
//
// Each K/V byte is used once, by the G <= 8 query heads of its kv head, so HBM bandwidth bounds
// this, and everything is arranged around equal shares of bytes in flight:
//   * The visible tokens of a sequence are cut into units (64 tokens at 4 bits, 32 at 16 bits).  All
//     sequences' units, end to end, are cut into equal parts, one CTA for each (part, kv head), as many as
//     fit the GPU at once: ragged lengths leave no CTA longer than another.  A CTA finds its part with one
//     pass over the lengths.  The kv heads of a part run next to each other, so that neighbouring rows of a
//     16-bit cache are read at about the same time.
//   * Each of a CTA's four warps takes every fourth unit and feeds itself: lane 0 issues the copies of
//     its K and then its V into the warp's own ring of stages (TMA boxes with a 128-byte swizzle at 16
//     bits; plain bulk copies at 4 bits, where a unit of a head is contiguous), with an mbarrier for each
//     stage.  No producer warp, and warps wait for nothing but their own data.
//   * The products are transposed, so that the G <= 8 heads are the n = 8 side of mma.sync m16n8k16:
//     S^T [16 tokens x 8] = K Q^T and O^T [d x 8] += V^T P^T, P moving from the first product's
//     accumulators to the second's operand by an in-register 8x8 transpose.
//     Weights are rounded to the type of the product, the cache's or, at 4 bits, fp16; their sum and O are
//     32-bit.
//   * At 4 bits an operand register is one conversion of a code pair and one product with its scale,
//     exact in fp16.  Which channel (K) or token (V) a matrix index stands for is free as long as
//     both factors agree, so K gives each lane 32 consecutive channels of a token (16 bytes) and V 16
//     channels of four tokens (8 bytes each): wide shared-memory loads, one or two scales for each.
//   * A piece of a (sequence, kv head) that is not whole goes to the workspace as (O / l, log-sum-exp);
//     the last CTA to finish (atomic ticket) joins the pieces in a fixed order.
//
// What bounds it, 32 query heads over 8 kv heads, d = 128, bf16:
//   16 bits, 192 sequences with a 4096 window (2.94 GB): 410 us, 7.2 TB/s, all that HBM gives a reader.
//   4 bits, 16 sequences of 8k-64k tokens (715 MB): 138 us, 5.2 TB/s; 64 with a 4096 window and 64 sinks (286
//     MB) 69 us, 4.1 TB/s.  Bound by turning codes into fp16 operands (issue slots 57 %, ALU 48 %): 111 us without the arithmetic, 135 us without the copies.
//   Short calls are a chain of latencies: 8 sequences with a 1024 window (34 MB) 11.4 us, one sequence of
//     16385 tokens at 4 bits (19 MB) 15.4 us.  Of those, 1.1 us go to finding the part, 0.9 to the table,
//     0.8 to the first copy, 4 to two units a warp, 1.6 to the pieces and the ticket, 3 to joining 33 pieces,
//     and 2.5 to the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>
#include <cmath>
#include <type_traits>

#include "host_internal.h"
#include "kv4.cuh"
#include "mma16.cuh"
#include "ptx.cuh"

namespace bsattn {
namespace {

using namespace mma16;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr size_t kHeader = 256;           // status word + padding
// One ticket for each (first part of a divided item, kv head): a part begins at most one such item, so
// their number goes by the GPU and not by the batch, and a workspace zeroed once serves every shape.
constexpr int kMaxTickets = 1024;
// exp2 is taken of x - max + 12: weights up to 4096, so that a weight 2^-24 of the largest is
// still a normal fp16 number and 2^-36 the smallest one
constexpr float kWeightLog2 = 12.f;
constexpr int kBatch = 12;                // pieces joined in one trip to L2

struct StreamParams {
    const void* q;
    const uint8_t* kc;              // 4-bit cache
    const uint8_t* ks;
    const uint8_t* vc;
    const uint8_t* vs;
    const int32_t* seqlens;
    const int32_t* chosen;          // [B, Hkv, max_sel] 64-token blocks, or null
    const int32_t* table;           // [B, max_pages], or null: contiguous rows of Smax tokens
    void* out;
    int* status;
    int* tickets;                   // [parts * Hkv]
    float* lse_part;                // [parts][2][Hkv][8]
    float* o_part;                  // [parts][2][Hkv][G][d]
    int B, Hq, Hkv, max_sel, window, sinks;
    int page_size, max_pages, num_pages, Smax;
    int parts;
    float score_log2;               // log2(e) / sqrt(d), and the keys' unit
    float v_unit;
    unsigned long long budget_ns;
};

// Shared memory of one CTA: rings first (1024-byte aligned for the swizzle), then barriers.  The
// joining of the four warps' results reuses the rings once they are drained.
template <int D, bool KV4>
struct Ring {
    static constexpr int kTok = KV4 ? 64 : 32;                   // tokens of a unit
    // A stage holds K or V of a unit; two a warp.  With three, 196 KB an SM in flight at 16 bits instead of
    // 131, 192 sequences with a 4096 window took 430 us against 410: DRAM serves fewer streams better.  At
    // 4 bits the conversions bound the kernel and it made no difference (139 us against 138).
    static constexpr int kStages = 2 * (128 / D);
    static constexpr int kCtas = KV4 ? 3 : 2;                    // resident CTAs per SM
    static constexpr int kLeast = 64 / kTok * kWarps;            // units of a part: 64 tokens a warp
    static constexpr int kSpare = 128 / kTok * kWarps;           // 128 tokens a warp
    static constexpr uint32_t kCodes = kTok * D / 2;             // 4 bits: codes, then scales
    static constexpr uint32_t kScales = kTok * D / kGroup4;
    static constexpr uint32_t kStage = KV4 ? kCodes + kScales : kTok * D * 2;
    static constexpr uint32_t kRing = kStages * kStage;          // of one warp
    static constexpr int kRow = D + 4;                           // padded row of the joining scratch
    static constexpr uint32_t kJoinWarp = (16 + 8 * kRow) * 4;   // m[8], l[8], O[8][kRow]
    static constexpr uint32_t kMain = kWarps * (kRing > kJoinWarp ? kRing : kJoinWarp);
    static constexpr uint32_t kBars = (kMain + 15) & ~15u;       // full[warp][stage]
    static constexpr uint32_t kKey0 = kBars + 8 * kWarps * kStages;
    static constexpr uint32_t kMisc = (kKey0 + 4 * kWarps * kStages + 15) & ~15u;   // holds 8-byte values
    static constexpr uint32_t kSlack = KV4 ? 0 : 1024;           // room to align the base up for the swizzle
    static constexpr uint32_t kBytes = kSlack + kMisc + 64;
    static_assert(KV4 || kStage % 1024 == 0, "swizzled tiles start on 1024 bytes");
    static_assert(kStage % 16 == 0 && kJoinWarp % 16 == 0 && kBars % 8 == 0 && kMisc % 16 == 0, "alignment");
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_u32(dst)),
                 "l"(src), "r"(bytes), "r"(smem_u32(bar))
                 : "memory");
}

// The visible units of one sequence: `near` units from unit `from`, after `head` sink units.
struct Span {
    int len;          // tokens
    int head, from, n;
};

template <int TOK>
__device__ __forceinline__ Span span_of(const StreamParams& p, int b) {
    Span s;
    int len = p.seqlens[b];
    if (len < 0) len = 0;
    if (!p.table && len > p.Smax) len = p.Smax;
    s.len = len;
    s.head = 0;
    s.from = 0;
    if (p.chosen) {
        s.n = p.max_sel * (64 / TOK);
        return s;
    }
    const int all = len / TOK + (len % TOK != 0);
    if (p.window > 0) {
        const int first = len > p.window ? (len - p.window) / TOK : 0;
        const int sink = min(p.sinks, len);
        s.head = min(sink / TOK + (sink % TOK != 0), first);
        s.from = first - s.head;                    // unit of the i-th visible one past the sinks: i + from
    }
    s.n = all - s.from;
    return s;
}

template <int D, bool BF16, bool KV4>
__global__ void __launch_bounds__(kThreads, Ring<D, KV4>::kCtas)
    stream_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                  const StreamParams p) {
    using R = Ring<D, KV4>;
    using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
    // At 4 bits both products run in fp16 (the cache's values are exact there, bf16 queries are scaled)
    constexpr bool kBf = BF16 && !KV4;
    constexpr int kTok = R::kTok, kStages = R::kStages, kTiles = kTok / 16;
    extern __shared__ __align__(128) uint8_t smem_raw[];
    uint8_t* sm = KV4 ? smem_raw
                      : reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t* ring = sm + warp * R::kRing;
    uint64_t* full = reinterpret_cast<uint64_t*>(sm + R::kBars) + warp * kStages;
    int* key0_of = reinterpret_cast<int*>(sm + R::kKey0) + warp * kStages;
    int* misc = reinterpret_cast<int*>(sm + R::kMisc);      // [0] abort [1] last [2] b [3] b's first part
    long long* start = reinterpret_cast<long long*>(misc + 4);          // units [0] before b, [1] up to its end
    volatile int* abort_flag = &misc[0];
    __shared__ long long warp_sums[kWarps];
    __shared__ int warp_parts[kWarps];

    const int part = blockIdx.x / p.Hkv, g = blockIdx.x - part * p.Hkv;
    const int G = p.Hq / p.Hkv;

    if (lane == 0)
        for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
    if (tid == 0) misc[0] = 0;
    fence_barrier_init();

    // ------------------------------------------------------------ this CTA's part of all units
    // thread t sums the units of its stretch of sequences; sequences without a token get their zeros
    const int per = (p.B + kThreads - 1) / kThreads;
    long long sum = 0;
    for (int k = 0; k < per; ++k) {
        const int b = tid * per + k;
        if (b >= p.B) break;
        const Span s = span_of<kTok>(p, b);
        sum += s.n;
        if (g == 0 && part == b % p.parts) {
            const int len = p.seqlens[b];
            const long long room = p.table ? static_cast<long long>(p.max_pages) * p.page_size : p.Smax;
            if (len < 0 || len > room) atomicOr(p.status, BSATTN_ERR_BAD_INDEX);
            if (s.n == 0) {
                uint4* o = reinterpret_cast<uint4*>(static_cast<T*>(p.out) + static_cast<size_t>(b) * p.Hq * D);
                for (int e = 0; e < p.Hq * D / 8; ++e) o[e] = make_uint4(0, 0, 0, 0);
            }
        }
    }
    long long upto = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
    }
    if (lane == 31) warp_sums[warp] = upto;
    __syncthreads();
    long long total = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) upto += warp_sums[w];
        total += warp_sums[w];
    }
    // parts of a multiple of four units (one a warp), 64 tokens a warp at least: one round at 4 bits (two
    // would take 11.6 us for 1500 tokens, one takes 10.3), two at 16 bits (with one, 200 tokens took 8.5 us
    // instead of 8.0 and 700 8.8 instead of 9.6: joining costs what the shorter loop gains)
    const auto part_of = [&](long long n) {
        const long long c = (total + n - 1) / n;
        return max((c + kWarps - 1) / kWarps * kWarps, static_cast<long long>(R::kLeast));
    };
    long long chunk = part_of(p.parts);
    // A part that ends one sequence and begins another does both one after the other, with all their
    // latencies: 4 to 5 us.  Where it makes the parts no more than kSpare units longer, every sequence is
    // cut for itself: ceil(n_b / chunk) parts each, p.parts in all or fewer with this chunk.  (32 query
    // heads, 8 kv heads, d = 128: 2 sequences of 1500 tokens 17.4 -> 11.6 us at 4 bits, 14.3 -> 10.0 us at
    // 16; 8 of 9000 31.2 -> 26.1 us; done whatever the parts grow by, 32 of 9000 would take 118 us, not 73.)
    bool apart = false;
    if (p.B <= kThreads && p.B < p.parts) {
        const long long longer = part_of(p.parts - p.B);
        apart = longer - chunk <= R::kSpare;
        if (apart) chunk = longer;
    }
    long long x0 = part * chunk;
    if (apart) {
        // thread t has sequence t's units
        const int n = static_cast<int>((sum + chunk - 1) / chunk);
        int parts_upto = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int u = __shfl_up_sync(0xffffffffu, parts_upto, o);
            if (lane >= o) parts_upto += u;
        }
        if (lane == 31) warp_parts[warp] = parts_upto;
        __syncthreads();
        int parts = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) parts_upto += warp_parts[w];
            parts += warp_parts[w];
        }
        if (part >= parts) return;                 // the whole CTA
        if (parts_upto - n <= part && part < parts_upto) {
            misc[2] = tid;
            misc[3] = parts_upto - n;
            start[0] = upto - sum;
            start[1] = upto;
        }
    } else {
        if (x0 >= total) return;                   // the whole CTA: x0 and total are the same for all
        if (upto - sum <= x0 && x0 < upto) {
            int b = tid * per;
            long long before = upto - sum;
            for (;; ++b) {
                const int n = span_of<kTok>(p, b).n;
                if (x0 < before + n) break;
                before += n;
            }
            misc[2] = b;
            start[0] = before;
            start[1] = total;
        }
    }
    __syncthreads();
    int b = misc[2];
    long long before = start[0];
    const int first = misc[3];
    if (apart) x0 = before + (part - first) * chunk;
    const long long x1 = min(x0 + chunk, start[1]);

    int seq = 0;                                   // units this warp has issued, over all pieces
    bool ok = true;
    // After a wait that expired the CTA goes through the rest of its pieces without reading anything and
    // hands each over as NaN: every ticket is taken, so that the workspace is ready for the next call, and
    // no row comes out that lacks a piece and does not show it.
    bool lost = false;
    for (long long x = x0; x < x1;) {
        const Span s = span_of<kTok>(p, b);
        if (s.n == 0) {
            ++b;
            continue;
        }
        const int i0 = static_cast<int>(x - before);
        const int i1 = static_cast<int>(min(static_cast<long long>(s.n), x1 - before));
        const int mine = i1 - i0 > warp && !lost ? (i1 - i0 - warp + kWarps - 1) / kWarps : 0;
        // tokens [lo, hi) and those before `sinks` are visible
        const int lo = p.window > 0 && !p.chosen ? max(0, s.len - p.window) : 0;
        const int sinks = p.window > 0 && !p.chosen ? p.sinks : 0;

        // ---------------------------------------------------------------- feeding
        // Unit k of this warp in this piece.  Lane L looks unit (k & ~31) + L up, 32 at a time.
        int look_key = 0, look_row = -1, look_page = 0;
        bool bad = false;
        auto look_up = [&](int k) {
            const int i = i0 + warp + kWarps * (k + lane);
            look_row = -1;
            look_key = 0;
            if (k + lane >= mine) return;
            int key;
            if (p.chosen) {
                const int t = p.chosen[(static_cast<size_t>(b) * p.Hkv + g) * p.max_sel + i / (64 / kTok)];
                if (t < 0) return;                                  // an empty slot
                if (t >= s.len / 64 + (s.len % 64 != 0)) {
                    bad = true;
                    return;
                }
                key = t * 64 + (i % (64 / kTok)) * kTok;
                if (key >= s.len) return;                           // second half past the end
            } else {
                key = (i < s.head ? i : i + s.from) * kTok;
            }
            look_key = key;
            if (p.table) {
                const int lp = key / p.page_size;
                const int page = lp < p.max_pages ? p.table[static_cast<size_t>(b) * p.max_pages + lp] : -1;
                if (page < 0 || page >= p.num_pages) {
                    bad = true;
                    return;
                }
                look_page = page;
                look_row = key - lp * p.page_size;
            } else {
                look_page = b;
                look_row = key;
            }
        };
        // Half h is K of unit h / 2 if h is even, its V if it is odd.
        auto issue = [&](int h) {
            const int k = h >> 1;
            if ((h & 63) == 0) look_up(k);
            const int row = __shfl_sync(0xffffffffu, look_row, k & 31);
            const int page = __shfl_sync(0xffffffffu, look_page, k & 31);
            const int key = __shfl_sync(0xffffffffu, look_key, k & 31);
            const int st = seq % kStages;
            ++seq;
            if (lane == 0) {
                key0_of[st] = row < 0 ? -1 : key;
                if (row < 0) {
                    mbar_arrive(&full[st]);                         // nothing to load: the unit is skipped
                } else {
                    uint8_t* dst = ring + st * R::kStage;
                    mbar_arrive_expect_tx(&full[st], R::kStage);
                    if constexpr (KV4) {
                        const size_t at = (static_cast<size_t>(page) * p.Hkv + g) * p.page_size + row;
                        bulk_load(dst, (h & 1 ? p.vc : p.kc) + at * (D / 2), R::kCodes, &full[st]);
                        bulk_load(dst + R::kCodes, (h & 1 ? p.vs : p.ks) + at * (D / kGroup4), R::kScales, &full[st]);
                    } else {
                        const int r = (p.table ? page * p.page_size : page * p.Smax) + row;
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            tma_load_3d(dst + c * (kTok * 128), h & 1 ? &tm_v : &tm_k, &full[st], c * 64, g, r);
                    }
                }
            }
        };
        // the first copies are on their way before the queries are read: both take a trip to memory
        const int base_seq = seq;
        for (int h = 0; h < kStages && h < 2 * mine; ++h) issue(h);

        // ---------------------------------------------------------------- queries
        // lane holds the four channels of head lane/4 that its K registers hold in each k16 step
        uint32_t qb[D / 16][2];
        float c0 = p.score_log2, c1 = p.score_log2;       // of heads 2 (lane % 4) + {0, 1}
        {
            const T* qg = reinterpret_cast<const T*>(p.q) + (static_cast<size_t>(b) * p.Hq + g * G) * D;
            const int hq = lane >> 2, j = lane & 3;
            const bool on = hq < G;
            if constexpr (KV4) {
                float top = 0.f;
                uint4 raw[D / 32];
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    raw[w] = on ? *reinterpret_cast<const uint4*>(qg + hq * D + j * (D / 4) + 8 * w)
                                : make_uint4(0, 0, 0, 0);
                    const uint32_t r[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float2 f = unpack2<BF16>(r[e]);
                        top = fmaxf(top, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // a power of two brings the head's largest query value into [1, 2): fp16 then holds
                // bf16 values exactly, but for those 2^-17 of the largest and less (off by 2^-25 of it).  At
                // the ends of bf16's range it gets into [2, 4) or below 1, as the power and its inverse have to
                // be normal 32-bit numbers; an infinite factor would turn a score of 0 into NaN.
                const int e = max(min(static_cast<int>(__float_as_uint(top) >> 23) - 127, 126), -126);
                const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    const uint32_t r[4] = {raw[w].x, raw[w].y, raw[w].z, raw[w].w};
#pragma unroll
                    for (int e2 = 0; e2 < 4; ++e2) {
                        const float2 f = unpack2<BF16>(r[e2]);
                        qb[2 * w + (e2 >> 1)][e2 & 1] = pack2<false>(f.x * down, f.y * down);
                    }
                }
                c0 = fminf(c0 * __shfl_sync(0xffffffffu, up, 8 * j), FLT_MAX);
                c1 = fminf(c1 * __shfl_sync(0xffffffffu, up, 8 * j + 4), FLT_MAX);
            } else {
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const T* src = qg + hq * D + kk * 16 + 2 * j;
                    qb[kk][0] = on ? *reinterpret_cast<const uint32_t*>(src) : 0u;
                    qb[kk][1] = on ? *reinterpret_cast<const uint32_t*>(src + 8) : 0u;
                }
            }
        }

        // ---------------------------------------------------------------- the warp's units
        float o[D / 16][4];
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
        float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;     // l of this lane's tokens only
        const int r8 = lane >> 2, j4 = lane & 3;
        // K row r8 of a tile is token r8 with the pairs (2,3) and (6,7) swapped: the V loads of a lane
        // quad then fall on rows of both parities, halving their bank conflicts
        const int tok_r = r8 ^ ((r8 >> 1) & 1);
        // Waits for half h and returns its stage; issues half h + kStages into it once it is read.
        auto arrived = [&](int h) -> uint8_t* {
            const int at = base_seq + h, st = at % kStages;
            if (!warp_wait_within(&full[st], (at / kStages) & 1, p.budget_ns, abort_flag, p.status)) {
                ok = false;
                return nullptr;
            }
            __syncwarp();
            return ring + st * R::kStage;
        };
        auto consumed = [&](int h) {
            __syncwarp();
            if (h + kStages < 2 * mine) issue(h + kStages);
        };
        for (int k = 0; k < mine; ++k) {
            uint8_t* stage = arrived(2 * k);
            if (!stage) break;
            const int key0 = key0_of[(base_seq + 2 * k) % kStages];
            if (key0 < 0) {
                consumed(2 * k);
                if (!arrived(2 * k + 1)) break;
                consumed(2 * k + 1);
                continue;
            }
            {
                // tokens [key0, key0 + kTok): visible [max(lo, 0), len) and [0, sinks)
                const bool edge = key0 + kTok > s.len || (key0 < lo && key0 + kTok > sinks);
                auto seen = [&](int t) { return t < s.len && (t >= lo || t < sinks); };
                float x[kTiles][4];
#pragma unroll
                for (int mt = 0; mt < kTiles; ++mt) {
                    float sc[4] = {0.f, 0.f, 0.f, 0.f};
                    if constexpr (KV4) {
                        // two rows of D / 4 channels for this lane
                        const uint8_t* ra = stage + (16 * mt + tok_r) * (D / 2) + j4 * (D / 8);
                        const uint8_t* sa = stage + R::kCodes + (16 * mt + tok_r) * (D / 16) + j4 * (D / 64);
                        uint32_t wa[D / 32], wb[D / 32], s0, s1;
                        if constexpr (D == 128) {
                            *reinterpret_cast<uint4*>(wa) = *reinterpret_cast<const uint4*>(ra);
                            *reinterpret_cast<uint4*>(wb) = *reinterpret_cast<const uint4*>(ra + 8 * (D / 2));
                            s0 = *reinterpret_cast<const uint16_t*>(sa);
                            s1 = *reinterpret_cast<const uint16_t*>(sa + 8 * (D / 16));
                        } else {
                            *reinterpret_cast<uint2*>(wa) = *reinterpret_cast<const uint2*>(ra);
                            *reinterpret_cast<uint2*>(wb) = *reinterpret_cast<const uint2*>(ra + 8 * (D / 2));
                            s0 = *sa;
                            s1 = sa[8 * (D / 16)];
                        }
                        const uint32_t sa2 = e4m3x2_to_f16(s0), sb2 = e4m3x2_to_f16(s1);
#pragma unroll
                        for (int w = 0; w < D / 32; ++w) {
                            // words 0-1 are one group of 16 channels, words 2-3 the next
                            const uint32_t ka = __byte_perm(sa2, 0, w < 2 ? 0x1010 : 0x3232);
                            const uint32_t kb = __byte_perm(sb2, 0, w < 2 ? 0x1010 : 0x3232);
                            uint32_t f[4], h[4];
                            e2m1_word_to_f16(wa[w], f[0], f[1], f[2], f[3]);
                            e2m1_word_to_f16(wb[w], h[0], h[1], h[2], h[3]);
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const uint32_t a[4] = {hmul2_u32(f[2 * e], ka), hmul2_u32(h[2 * e], kb),
                                                       hmul2_u32(f[2 * e + 1], ka), hmul2_u32(h[2 * e + 1], kb)};
                                mma16816<false>(sc, a, qb[2 * w + e][0], qb[2 * w + e][1]);
                            }
                        }
                    } else {
                        const uint32_t kbase = smem_u32(stage);
                        const int mat = lane >> 3;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const int col = kk * 16 + (mat >> 1) * 8;
                            uint32_t a[4];
                            ldsm4(kbase + (col >> 6) * (kTok * 128) + sw128_offset(16 * mt + (mat & 1) * 8 + (lane & 7), col & 63), a);
                            mma16816<kBf>(sc, a, qb[kk][0], qb[kk][1]);
                        }
                    }
                    x[mt][0] = sc[0] * c0;
                    x[mt][1] = sc[1] * c1;
                    x[mt][2] = sc[2] * c0;
                    x[mt][3] = sc[3] * c1;
                    if (edge) {
                        const int ta = key0 + 16 * mt + (KV4 ? tok_r : r8);
                        if (!seen(ta)) x[mt][0] = x[mt][1] = -INFINITY;
                        if (!seen(ta + 8)) x[mt][2] = x[mt][3] = -INFINITY;
                    }
                }
                consumed(2 * k);
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
                const float z0 = m0 == -INFINITY ? 0.f : m0 - kWeightLog2;
                const float z1 = m1 == -INFINITY ? 0.f : m1 - kWeightLog2;
                uint32_t pb[kTiles][2];
#pragma unroll
                for (int mt = 0; mt < kTiles; ++mt) {
                    const float p0 = ex2_approx(x[mt][0] - z0), p1 = ex2_approx(x[mt][1] - z1);
                    const float p2 = ex2_approx(x[mt][2] - z0), p3 = ex2_approx(x[mt][3] - z1);
                    l0 += p0 + p2;
                    l1 += p1 + p3;
                    pb[mt][0] = transpose8x8(pack2<kBf>(p0, p1));
                    pb[mt][1] = transpose8x8(pack2<kBf>(p2, p3));
                }
                stage = arrived(2 * k + 1);
                if (!stage) break;
#pragma unroll
                for (int mt = 0; mt < kTiles; ++mt) {
                    const uint32_t pb0 = pb[mt][0], pb1 = pb[mt][1];
                    if constexpr (KV4) {
                        // tokens 2 j4, 2 j4 + 1 and eight further, as K's rows name them
                        const int ta = 16 * mt + (2 * j4 ^ (j4 & 1)), tb = 16 * mt + ((2 * j4 + 1) ^ (j4 & 1));
                        const uint8_t* vc = stage;
                        const uint8_t* vs = vc + R::kCodes;
                        const int gi = D == 128 ? r8 : r8 >> 1;
                        uint32_t e8[4] = {vs[ta * (D / 16) + gi], vs[tb * (D / 16) + gi], vs[(ta + 8) * (D / 16) + gi],
                                          vs[(tb + 8) * (D / 16) + gi]};
                        if (edge) {
                            // a weight of 0 must not meet the NaN that a masked row's scale may be
                            if (!seen(key0 + ta)) e8[0] = 0;
                            if (!seen(key0 + tb)) e8[1] = 0;
                            if (!seen(key0 + ta + 8)) e8[2] = 0;
                            if (!seen(key0 + tb + 8)) e8[3] = 0;
                        }
                        const uint32_t sx = e4m3x2_to_f16(e8[0] | e8[1] << 8), sy = e4m3x2_to_f16(e8[2] | e8[3] << 8);
                        uint32_t v4[4][D / 64];                     // four tokens' D / 8 channels
                        const int rows[4] = {ta, tb, ta + 8, tb + 8};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const uint8_t* src = vc + rows[e] * (D / 2) + r8 * (D / 16);
                            if constexpr (D == 128) *reinterpret_cast<uint2*>(v4[e]) = *reinterpret_cast<const uint2*>(src);
                            else v4[e][0] = *reinterpret_cast<const uint32_t*>(src);
                        }
#pragma unroll
                        for (int w = 0; w < D / 64; ++w) {
                            const uint32_t u0 = v4[0][w], u1 = v4[1][w], u2 = v4[2][w], u3 = v4[3][w];
                            // byte i of ev / od: the even / odd channel of byte i, of two tokens
                            uint32_t ev0[4], od0[4], ev1[4], od1[4];
                            constexpr uint32_t kLow = 0x0f0f0f0fu;
                            e2m1_word_to_f16((u0 & kLow) | ((u1 << 4) & ~kLow), ev0[0], ev0[1], ev0[2], ev0[3]);
                            e2m1_word_to_f16(((u0 >> 4) & kLow) | (u1 & ~kLow), od0[0], od0[1], od0[2], od0[3]);
                            e2m1_word_to_f16((u2 & kLow) | ((u3 << 4) & ~kLow), ev1[0], ev1[1], ev1[2], ev1[3]);
                            e2m1_word_to_f16(((u2 >> 4) & kLow) | (u3 & ~kLow), od1[0], od1[1], od1[2], od1[3]);
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t a[4] = {hmul2_u32(ev0[i], sx), hmul2_u32(od0[i], sx),
                                                       hmul2_u32(ev1[i], sy), hmul2_u32(od1[i], sy)};
                                mma16816<false>(o[4 * w + i], a, pb0, pb1);
                            }
                        }
                    } else {
                        if (edge && mt == 0) {
                            // tokens that are not visible may hold anything: zero their V rows, so that
                            // a weight of 0 cannot meet a NaN
                            for (int e = lane; e < kTok * (D / 8); e += 32) {
                                const int r = e / (D / 8), col = (e % (D / 8)) * 8;
                                if (!seen(key0 + r))
                                    *reinterpret_cast<uint4*>(stage + (col >> 6) * (kTok * 128) +
                                                              sw128_offset(r, col & 63)) = make_uint4(0, 0, 0, 0);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                        }
                        const uint32_t vbase = smem_u32(stage);
                        const int mat = lane >> 3;
#pragma unroll
                        for (int dt = 0; dt < D / 16; ++dt) {
                            const int col = dt * 16 + (mat & 1) * 8;
                            uint32_t a[4];
                            ldsm4_t(vbase + (col >> 6) * (kTok * 128) +
                                        sw128_offset(16 * mt + (mat >> 1) * 8 + (lane & 7), col & 63), a);
                            mma16816<kBf>(o[dt], a, pb0, pb1);
                        }
                    }
                }
                consumed(2 * k + 1);
            }
        }
        if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.status, BSATTN_ERR_BAD_INDEX);
        if (!ok) {
            // let copies in flight land before their stages become something else
            const uint64_t dl = global_timer_ns() + 200000000ull;
            for (int a = max(base_seq, seq - kStages); a < seq; ++a)
                wait_parity_drain(&full[a % kStages], (a / kStages) & 1, dl);
        }
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, w);
            l1 += __shfl_xor_sync(0xffffffffu, l1, w);
        }
        __syncthreads();                            // every warp's ring is drained
        lost = *abort_flag != 0;                    // the same in the whole CTA: nobody raises it until the next piece
        if (lost) l0 = l1 = __int_as_float(0x7fffffff);

        // ---------------------------------------------------------------- joining the four warps
        {
            float* mw = reinterpret_cast<float*>(sm) + warp * (R::kJoinWarp / 4);
            const int h0 = 2 * j4;
            if (lane < 4) {
                mw[h0] = m0;
                mw[h0 + 1] = m1;
                mw[8 + h0] = l0;
                mw[8 + h0 + 1] = l1;
            }
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                if constexpr (KV4) {
                    // lane row r8 stands for channels r8 D/8 + 2 mt + {0, 1}; they are kept at 16 mt + 2 r8, so
                    // that a store's eight rows lie next to each other
                    *reinterpret_cast<float2*>(mw + 16 + h0 * R::kRow + 16 * mt + 2 * r8) = make_float2(o[mt][0], o[mt][2]);
                    *reinterpret_cast<float2*>(mw + 16 + (h0 + 1) * R::kRow + 16 * mt + 2 * r8) =
                        make_float2(o[mt][1], o[mt][3]);
                } else {
                    const int d0 = mt * 16 + r8;
                    mw[16 + h0 * R::kRow + d0] = o[mt][0];
                    mw[16 + (h0 + 1) * R::kRow + d0] = o[mt][1];
                    mw[16 + h0 * R::kRow + d0 + 8] = o[mt][2];
                    mw[16 + (h0 + 1) * R::kRow + d0 + 8] = o[mt][3];
                }
            }
        }
        __syncthreads();
        const bool whole = i0 == 0 && i1 == s.n;
        const size_t slot = (static_cast<size_t>(part) * 2 + (i0 == 0 ? 1 : 0)) * p.Hkv + g;
        const size_t row_base = static_cast<size_t>(b) * p.Hq + g * G;
        const float* join = reinterpret_cast<const float*>(sm);
        constexpr int kW = R::kJoinWarp / 4;
        for (int e = tid; e < G * (D / 4); e += kThreads) {
            const int row = e / (D / 4), c4 = e % (D / 4);
            float M = -INFINITY;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) M = fmaxf(M, join[w * kW + row]);
            float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
            float den = 0.f;
            const float ref = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                // a warp without a finite score has l = 0, or NaN if it met one: either way it counts
                const float mw = join[w * kW + row];
                const float wt = mw == -INFINITY ? 1.f : ex2_approx(mw - ref);
                const float* ow = join + w * kW + 16 + row * R::kRow;
                float4 ov;
                if constexpr (KV4) {
                    const int r = 4 * c4 / (D / 8), mt = (4 * c4 % (D / 8)) / 2;
                    const float2 lo2 = *reinterpret_cast<const float2*>(ow + 16 * mt + 2 * r);
                    const float2 hi2 = *reinterpret_cast<const float2*>(ow + 16 * mt + 16 + 2 * r);
                    ov = make_float4(lo2.x, lo2.y, hi2.x, hi2.y);
                } else {
                    ov = *reinterpret_cast<const float4*>(ow + 4 * c4);
                }
                num.x += wt * ov.x;
                num.y += wt * ov.y;
                num.z += wt * ov.z;
                num.w += wt * ov.w;
                den += wt * join[w * kW + 8 + row];
            }
            // den is 0 only for a row with no visible token (NaN stays NaN)
            const float inv = den == 0.f ? 0.f : 1.f / den;
            const float4 val = make_float4(num.x * inv, num.y * inv, num.z * inv, num.w * inv);
            if (whole) {
                const float u = p.v_unit;
                uint2 w2;
                w2.x = pack2<BF16>(val.x * u, val.y * u);
                w2.y = pack2<BF16>(val.z * u, val.w * u);
                *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + (row_base + row) * D + 4 * c4) = w2;
            } else {
                *reinterpret_cast<float4*>(p.o_part + (slot * G + row) * D + 4 * c4) = val;
                if (c4 == 0) p.lse_part[slot * 8 + row] = den == 0.f ? -INFINITY : M + log2f(den);
            }
        }
        if (!whole) {
            // ------------------------------------------------------------ joining the pieces
            const int c_first = apart ? first : static_cast<int>(before / chunk);
            const int c_last = apart ? first + static_cast<int>((s.n - 1) / chunk)
                                     : static_cast<int>((before + s.n - 1) / chunk);
            const int count = c_last - c_first + 1;
            __syncthreads();
            if (tid == 0) {
                int before_me;
                asm volatile("atom.acq_rel.gpu.global.add.s32 %0, [%1], 1;"
                             : "=r"(before_me)
                             : "l"(&p.tickets[c_first * p.Hkv + g])
                             : "memory");
                misc[1] = before_me == count - 1;
            }
            __syncthreads();
            if (misc[1]) {
                // read through L2 (an SM's L1 may hold an earlier call's lines), kBatch pieces at a time
                for (int e = tid; e < G * (D / 4); e += kThreads) {
                    const int row = e / (D / 4), c4 = e % (D / 4);
                    float M = -INFINITY, den = 0.f;
                    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
                    for (int c8 = 0; c8 < count; c8 += kBatch) {
                        float lv[kBatch];
                        float4 ov[kBatch];
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            const int c = c_first + c8 + k;
                            const size_t sl = (static_cast<size_t>(c) * 2 + (c == c_first ? 1 : 0)) * p.Hkv + g;
                            const bool in = c <= c_last;
                            lv[k] = in ? __ldcg(p.lse_part + sl * 8 + row) : -INFINITY;
                            ov[k] = in ? __ldcg(reinterpret_cast<const float4*>(p.o_part + (sl * G + row) * D) + c4)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                        float Mc = M;
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) Mc = fmaxf(Mc, lv[k]);
                        const float ref = Mc == -INFINITY ? 0.f : Mc;
                        const float r = ex2_approx(M - ref);
                        num.x *= r;
                        num.y *= r;
                        num.z *= r;
                        num.w *= r;
                        den *= r;
#pragma unroll
                        for (int k = 0; k < kBatch; ++k) {
                            const float wt = ex2_approx(lv[k] - ref);
                            num.x += wt * ov[k].x;
                            num.y += wt * ov[k].y;
                            num.z += wt * ov[k].z;
                            num.w += wt * ov[k].w;
                            den += wt;
                        }
                        M = Mc;
                    }
                    const float inv = (den == 0.f ? 0.f : 1.f / den) * p.v_unit;
                    uint2 w2;
                    w2.x = pack2<BF16>(num.x * inv, num.y * inv);
                    w2.y = pack2<BF16>(num.z * inv, num.w * inv);
                    *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + (row_base + row) * D + 4 * c4) = w2;
                }
                if (tid == 0) p.tickets[c_first * p.Hkv + g] = 0;         // ready for the next call
            }
        }
        // the rings' next copies (async proxy) come after the joining's shared-memory accesses
        fence_proxy_async_smem();
        __syncthreads();
        x = before + i1;
        if (i1 == s.n) {
            before += s.n;
            ++b;
        }
    }
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

struct WsLayout {
    size_t tickets, lse, opart, total;
};

int parts_of(int Hkv, int ctas_per_sm) {
    int sms = num_sms_of_current_device();
    if (sms <= 0) sms = 148;
    const int parts = ctas_per_sm * sms / Hkv;
    return parts < 1 ? 1 : parts;
}

WsLayout ws_layout(int Hq, int Hkv, int d, int parts) {
    WsLayout w{};
    w.tickets = kHeader;
    w.lse = w.tickets + sizeof(int) * kMaxTickets;
    w.opart = w.lse + align256(sizeof(float) * 2 * static_cast<size_t>(parts) * Hkv * 8);
    w.total = w.opart + align256(sizeof(float) * 2 * static_cast<size_t>(parts) * Hq * d);
    return w;
}

template <int D, bool BF16, bool KV4>
int launch(const CUtensorMap& tk, const CUtensorMap& tv, const StreamParams& prm, cudaStream_t stream) {
    using R = Ring<D, KV4>;
    auto kern = stream_kernel<D, BF16, KV4>;
    static std::atomic<unsigned long long> raised{0};
    const int rc = raise_smem_limit(reinterpret_cast<const void*>(kern), R::kBytes, raised);
    if (rc) return rc;
    kern<<<static_cast<unsigned>(prm.parts) * prm.Hkv, kThreads, R::kBytes, stream>>>(tk, tv, prm);
    return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

// Checks, workspace and launch shared by the entry points.  `k16` / `v16`: 16-bit caches, or null.
int decode_stream(StreamParams prm, const void* k16, const void* v16, int d, bsattn_dtype dtype,
                  void* workspace, size_t workspace_bytes, cudaStream_t st) {
    const bool kv4 = prm.kc != nullptr;
    if (prm.B < 0 || prm.Hq <= 0 || prm.Hkv <= 0 || prm.window < 0 || prm.sinks < 0 || prm.max_sel < 0)
        return BSATTN_ERR_INVALID_ARG;
    if (prm.Hq % prm.Hkv) return BSATTN_ERR_INVALID_ARG;
    if (prm.Hq / prm.Hkv > 8) return BSATTN_ERR_UNSUPPORTED;
    if (d != 64 && d != 128) return BSATTN_ERR_UNSUPPORTED;
    if (dtype != BSATTN_F16 && dtype != BSATTN_BF16) return BSATTN_ERR_UNSUPPORTED;
    if (prm.Hkv > kMaxTickets) return BSATTN_ERR_UNSUPPORTED;
    if (!workspace) return BSATTN_ERR_INVALID_ARG;
    if (prm.B == 0) return BSATTN_OK;
    if (!prm.q || !prm.out || !prm.seqlens || !aligned16(prm.q) || !aligned16(prm.out)) return BSATTN_ERR_INVALID_ARG;
    if (!kv4 && !prm.table && prm.Smax == 0)
        return cudaMemsetAsync(prm.out, 0, static_cast<size_t>(prm.B) * prm.Hq * d * 2, st) == cudaSuccess
                   ? BSATTN_OK
                   : BSATTN_ERR_CUDA;
    // a CTA writes its rows while others still read: out may be q itself, whose rows have then been read
    const size_t out_bytes = static_cast<size_t>(prm.B) * prm.Hq * d * 2;
    const size_t rows = prm.table ? static_cast<size_t>(prm.num_pages) * prm.page_size
                                  : static_cast<size_t>(prm.B) * prm.Smax;
    const size_t values = rows * prm.Hkv * d;
    if ((prm.out != prm.q && overlap(prm.out, out_bytes, prm.q, out_bytes)) ||
        (kv4 && (overlap(prm.out, out_bytes, prm.kc, values / 2) || overlap(prm.out, out_bytes, prm.vc, values / 2) ||
                 overlap(prm.out, out_bytes, prm.ks, values / kGroup4) ||
                 overlap(prm.out, out_bytes, prm.vs, values / kGroup4))) ||
        (!kv4 && (overlap(prm.out, out_bytes, k16, 2 * values) || overlap(prm.out, out_bytes, v16, 2 * values))))
        return BSATTN_ERR_INVALID_ARG;
    const int parts = parts_of(prm.Hkv, kv4 ? Ring<128, true>::kCtas : Ring<128, false>::kCtas);
    if (static_cast<long long>(parts) * prm.Hkv > kMaxTickets) return BSATTN_ERR_UNSUPPORTED;
    const WsLayout w = ws_layout(prm.Hq, prm.Hkv, d, parts);
    if (workspace_bytes < w.total || !aligned16(workspace)) return BSATTN_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    prm.parts = parts;
    prm.status = status_word(ws);
    prm.tickets = reinterpret_cast<int*>(ws + w.tickets);
    prm.lse_part = reinterpret_cast<float*>(ws + w.lse);
    prm.o_part = reinterpret_cast<float*>(ws + w.opart);
    prm.score_log2 *= static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
    prm.budget_ns = wait_budget_ns();
    const bool bf16 = dtype == BSATTN_BF16;
    CUtensorMap tk{}, tv{};
    if (!kv4) {
        const uint64_t row_bytes = uint64_t(prm.Hkv) * d * 2;
        int rc = encode_3d(&tk, k16, bf16, d, prm.Hkv, rows, d * 2ull, row_bytes, 64, 1, Ring<128, false>::kTok, true);
        rc |= encode_3d(&tv, v16, bf16, d, prm.Hkv, rows, d * 2ull, row_bytes, 64, 1, Ring<128, false>::kTok, true);
        if (rc) return rc;
        if (d == 64) return bf16 ? launch<64, true, false>(tk, tv, prm, st) : launch<64, false, false>(tk, tv, prm, st);
        return bf16 ? launch<128, true, false>(tk, tv, prm, st) : launch<128, false, false>(tk, tv, prm, st);
    }
    if (d == 64) return bf16 ? launch<64, true, true>(tk, tv, prm, st) : launch<64, false, true>(tk, tv, prm, st);
    return bf16 ? launch<128, true, true>(tk, tv, prm, st) : launch<128, false, true>(tk, tv, prm, st);
}

int page_check(int num_pages, int page_size, int max_pages) {
    if (page_size <= 0 || num_pages <= 0 || max_pages <= 0) return BSATTN_ERR_INVALID_ARG;
    if (page_size % 64) return BSATTN_ERR_UNSUPPORTED;
    return BSATTN_OK;
}

}  // namespace
}  // namespace bsattn

extern "C" size_t bsattn_decode_window_workspace_size(int Hq, int Hkv, int d) {
    using namespace bsattn;
    if (Hq <= 0 || Hkv <= 0 || d <= 0) return kHeader;
    return ws_layout(Hq, Hkv, d, parts_of(Hkv, Ring<128, false>::kCtas)).total;
}

extern "C" size_t bsattn_decode_kv4_workspace_size(int Hq, int Hkv, int d) {
    using namespace bsattn;
    if (Hq <= 0 || Hkv <= 0 || d <= 0) return kHeader;
    return ws_layout(Hq, Hkv, d, parts_of(Hkv, Ring<128, true>::kCtas)).total;
}

extern "C" int bsattn_decode_window(const void* q, const void* k, const void* v,
                                    const int32_t* cache_seqlens, int window, int sinks, void* out,
                                    int B, int Hq, int Hkv, int Smax, int d, bsattn_dtype dtype,
                                    void* workspace, size_t workspace_bytes, void* stream) {
    using namespace bsattn;
    if (window < 1 || Smax < 0) return BSATTN_ERR_INVALID_ARG;
    if (B > 0 && Smax > 0 && (!k || !v || !aligned16(k) || !aligned16(v))) return BSATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(B) * Smax > 0x7fffffffLL) return BSATTN_ERR_UNSUPPORTED;
    StreamParams prm{};
    prm.q = q;
    prm.seqlens = cache_seqlens;
    prm.window = window;
    prm.sinks = sinks;
    prm.out = out;
    prm.B = B;
    prm.Hq = Hq;
    prm.Hkv = Hkv;
    prm.Smax = Smax;
    prm.score_log2 = 1.f;
    prm.v_unit = 1.f;
    return decode_stream(prm, k, v, d, dtype, workspace, workspace_bytes, static_cast<cudaStream_t>(stream));
}

extern "C" int bsattn_decode_window_paged(const void* q, const void* k_pages, const void* v_pages,
                                          const int32_t* cache_seqlens, const int32_t* block_table,
                                          int window, int sinks, void* out, int B, int Hq, int Hkv,
                                          int num_pages, int page_size, int max_pages_per_seq, int d,
                                          bsattn_dtype dtype, void* workspace, size_t workspace_bytes,
                                          void* stream) {
    using namespace bsattn;
    if (window < 1) return BSATTN_ERR_INVALID_ARG;
    const int rc = page_check(num_pages, page_size, max_pages_per_seq);
    if (rc) return rc;
    if (B > 0 && (!k_pages || !v_pages || !block_table || !aligned16(k_pages) || !aligned16(v_pages)))
        return BSATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL) return BSATTN_ERR_UNSUPPORTED;
    StreamParams prm{};
    prm.q = q;
    prm.seqlens = cache_seqlens;
    prm.table = block_table;
    prm.window = window;
    prm.sinks = sinks;
    prm.out = out;
    prm.B = B;
    prm.Hq = Hq;
    prm.Hkv = Hkv;
    prm.num_pages = num_pages;
    prm.page_size = page_size;
    prm.max_pages = max_pages_per_seq;
    prm.score_log2 = 1.f;
    prm.v_unit = 1.f;
    return decode_stream(prm, k_pages, v_pages, d, dtype, workspace, workspace_bytes,
                         static_cast<cudaStream_t>(stream));
}

extern "C" int bsattn_decode_paged_kv4(const void* q, const uint8_t* k_codes, const uint8_t* k_scales,
                                       const uint8_t* v_codes, const uint8_t* v_scales, float k_scale,
                                       float v_scale, const int32_t* cache_seqlens,
                                       const int32_t* block_indices, const int32_t* block_table,
                                       int window, int sinks, void* out, int B, int Hq, int Hkv,
                                       int num_pages, int page_size, int max_pages_per_seq, int d,
                                       int max_sel, bsattn_dtype dtype, void* workspace,
                                       size_t workspace_bytes, void* stream) {
    using namespace bsattn;
    const int rc = page_check(num_pages, page_size, max_pages_per_seq);
    if (rc) return rc;
    if (!unit_ok4(k_scale) || !unit_ok4(v_scale)) return BSATTN_ERR_INVALID_ARG;
    if (block_indices && window) return BSATTN_ERR_INVALID_ARG;       // one rule of visibility a call
    if (!k_codes || !k_scales || !v_codes || !v_scales || (B > 0 && !block_table)) return BSATTN_ERR_INVALID_ARG;
    if (!aligned16(k_codes) || !aligned16(k_scales) || !aligned16(v_codes) || !aligned16(v_scales))
        return BSATTN_ERR_INVALID_ARG;
    if (max_sel < 0 || max_sel > (1 << 26)) return BSATTN_ERR_INVALID_ARG;
    StreamParams prm{};
    prm.q = q;
    prm.kc = k_codes;
    prm.ks = k_scales;
    prm.vc = v_codes;
    prm.vs = v_scales;
    prm.seqlens = cache_seqlens;
    prm.chosen = block_indices;
    prm.table = block_table;
    prm.window = window;
    prm.sinks = sinks;
    prm.out = out;
    prm.B = B;
    prm.Hq = Hq;
    prm.Hkv = Hkv;
    prm.max_sel = max_sel;
    prm.num_pages = num_pages;
    prm.page_size = page_size;
    prm.max_pages = max_pages_per_seq;
    prm.score_log2 = k_scale;
    prm.v_unit = v_scale;
    return decode_stream(prm, nullptr, nullptr, d, dtype, workspace, workspace_bytes,
                         static_cast<cudaStream_t>(stream));
}
