// block_select.cu -- the key blocks of a decode query, and the block mask of a prompt, by the product of
// 8-bit summaries (summary.cuh), sm_103a.
//
// The score of a key block for a query is (their codes' whole-number product) * (query scale) * (key scale),
// two 32-bit roundings; a decode's kv head takes the largest of its query heads' first products.  Chosen
// are blocks that are asked for whatever their score (the first ones, the last ones), then the best others
// up to the wanted number, the lower block first among equals.
//
// The choice is a search for the score that the wanted number of blocks reach: counts of blocks at or above
// four thresholds a trip, which cut what lies between into five, until a count is right or one score is left.  With
// scores spread evenly it takes some six trips for a thousand blocks.
#include <algorithm>

#include "host_internal.h"
#include "mma16.cuh"
#include "ptx.cuh"
#include "summary.cuh"

namespace bsattn {
namespace {

// ------------------------------------------------------------------------------------------ decode
//
// A (sequence, kv head) is a CTA's, or that of a cluster whose CTAs have a stretch of its blocks each.
// A warp scores 32 blocks at a time, S [16 blocks x 8 heads] = K Q^T twice by mma.sync m16n8k16 in fp16: a code c enters
// as 1152 + c, which takes one byte permutation for two codes (1024 + byte is an fp16 number with that byte for its
// lowest), and the sums begin at -1152 times the query's codes.  Whole numbers below 2^23 in magnitude throughout, 32
// channels a sum: exact.  (64 sequences of up to 1024 blocks, d = 128: 17.6 us; 16 blocks at a time 21.1, as the way from
// the products to a key is a chain of latencies; by 8-bit products, which the tensor core does at an m16n8k32 in 17
// cycles an SM, 21.3; by dp4a, with the adding of eight lanes' sums, 28.)
// Which channel a matrix index stands for is free, so a lane reads 16 consecutive codes of a row.  Keys stay in shared
// memory, the first kHeld of a thread in registers.  A trip of the search counts at four thresholds at once: a count is
// mostly the way through the barrier.
// The index is read once (41 MB there, 5.9 us at the copy rate); what bounds this is the longest row's chain: lengths,
// table and index 4 us, then 8 times 32 blocks a warp, six counts, the writing.

constexpr int kMaxBlocks = 46875;               // of a sequence: their keys lie in shared memory
constexpr int kHeld = 8;                        // keys of a thread in registers

struct SelectParams {
    const void* q;
    const int8_t* codes;
    const float* scales;
    const int32_t* seqlens;
    const int32_t* table;
    int32_t* out;
    int* status;
    int Hq, Hkv, page_size, max_pages, num_pages, max_sel, sinks, recent;
};

// What the CTA's warps add up, or the cluster's CTAs.
struct Shares {
    uint32_t range[2];                          // largest of ~key, and of key
    int there, forced;                          // blocks that may be chosen, blocks that have to be
    int counts[3][4];
};

__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
    return n;
}
__device__ __forceinline__ void cluster_arrive() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// The word of CTA `rank` that stands where `mine` does here.
__device__ __forceinline__ uint32_t word_of(const void* mine, uint32_t rank) {
    uint32_t at;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(mine)), "r"(rank));
    return at;
}
__device__ __forceinline__ void add_to(uint32_t at, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}
__device__ __forceinline__ void max_to(uint32_t at, uint32_t v) {
    asm volatile("red.relaxed.cluster.shared::cluster.max.u32 [%0], %1;" ::"r"(at), "r"(v) : "memory");
}

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
}

constexpr int kDepth = 2;                       // times 32 blocks whose index rows a warp has on their way
constexpr int kMaxCluster = 8;

template <int D, bool BF16, int TH>
__global__ void __launch_bounds__(TH, TH == 128 ? 4 : 1) select_kernel(const SelectParams p) {
    constexpr int kWarps = TH / 32;
    constexpr int kSteps = D / 16, kSums = kSteps / 2;      // k16 steps, and sums of two of them
    constexpr uint32_t kGroup = 32 * D + 128;               // 32 index rows: codes, scales
    extern __shared__ __align__(16) uint8_t sel_smem[];
    uint32_t* keys = reinterpret_cast<uint32_t*>(sel_smem + kWarps * kDepth * kGroup);   // of the CTA's blocks; first their index rows
    __shared__ uint2 qb[kSteps][32];                        // the queries' codes as a lane's operands, head lane / 4
    __shared__ float qscale[8], qbase[kSums][8];            // of the query heads: scale, where sums begin
    __shared__ Shares own, all;                             // the CTA's, the cluster's
    __shared__ int above[kWarps], level[kWarps];
    __shared__ int at_rank[2][kMaxCluster];                 // chosen blocks of each CTA: above the threshold, at it
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int CL = static_cast<int>(cluster_size()), rank = static_cast<int>(blockIdx.x) % CL;
    const int row = static_cast<int>(blockIdx.x) / CL, b = row / p.Hkv, g = row - b * p.Hkv, G = p.Hq / p.Hkv;

    const int asked = p.seqlens[b];
    // a warp a query head: its codes and scale
    for (int head = warp; head < G; head += kWarps) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.q) +
                                                                (static_cast<size_t>(b) * p.Hq + g * G + head) * D);
        float x[D / 32], top = 0.f;
        bool finite = true;
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
            const float2 f = mma16::unpack2<BF16>(src[lane * (D / 64) + w]);
            x[2 * w] = f.x;
            x[2 * w + 1] = f.y;
        }
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            const float a = fabsf(x[e]);
            finite = finite && a <= FLT_MAX;
            top = fmaxf(top, a);
        }
        finite = __all_sync(0xffffffffu, finite);
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        const float scale = scale8(top, finite);
        int sum = 0;
#pragma unroll
        for (int e = 0; e < D / 32; ++e) {
            const int c = code8(x[e], scale, finite);
            x[e] = static_cast<float>(c);
            sum += c;
        }
        // (channels 2 i, 2 i + 1 of head h: half of the operands of lane 4 h + j in step k, as below)
#pragma unroll
        for (int e = 0; e < D / 64; ++e) {
            const int ch = lane * (D / 32) + 2 * e, k = ch / 64 * 4 + ch % 16 / 4;
            reinterpret_cast<uint32_t*>(&qb[k][4 * head + ch % 64 / 16])[ch % 4 / 2] = mma16::pack2<false>(x[2 * e], x[2 * e + 1]);
        }
        // Step k has channels 64 (k / 4) + 16 j + 4 (k % 4) + 0 .. 3 of a lane j of a quad, a sum two steps: those of
        // lanes with the same bit 4 and bit 1 (d = 128: four channels a lane) or the same bit 2 (d = 64: two).
#pragma unroll
        for (int m = 1; m < 32; m <<= 1)
            if (D == 128 ? m != 16 && m != 2 : m != 4) sum += __shfl_xor_sync(0xffffffffu, sum, m);
        if (D == 128 ? (lane & ~18) == 0 : (lane & ~4) == 0)
            qbase[D == 128 ? lane >> 4 << 1 | (lane >> 1 & 1) : lane >> 2][head] = -1152.f * static_cast<float>(sum);
        if (lane == 0) qscale[head] = finite ? scale : 0.f;         // a query that is not finite scores 0
    }
    const int blocks_a_page = p.page_size / kBlockRows;
    const int room = p.max_pages * blocks_a_page;
    const bool far = asked < 0 || asked > static_cast<long long>(p.max_pages) * p.page_size;
    const int all_n = asked <= 0 ? 0 : min(asked / kBlockRows + (asked % kBlockRows != 0), room);
    // the CTA's blocks: n from block0 on
    const int each = ((all_n + CL - 1) / CL + 31) & ~31;
    const int block0 = min(rank * each, all_n), n = min(each, all_n - block0);
    if (tid < static_cast<int>(sizeof(Shares) / 4)) {
        reinterpret_cast<uint32_t*>(&own)[tid] = 0;
        reinterpret_cast<uint32_t*>(&all)[tid] = 0;
    }
    if (CL > 1) cluster_arrive();                           // what the others add to is 0
    // (heads that there are not: codes 0)
    for (int i = tid; i < kSteps * 32; i += TH)
        if (i % 32 / 4 >= G) qb[i / 32][i % 32] = make_uint2(0, 0);
    if (tid < 8 * kSums && tid % 8 >= G) qbase[tid / 8][tid % 8] = 0.f;
    // the index row of each block, or -1
    bool bad = far;
    for (int i = tid; i < n; i += TH) {
        const int j = block0 + i, lp = j / blocks_a_page;
        const int page = __ldg(p.table + static_cast<size_t>(b) * p.max_pages + lp);
        const bool in = page >= 0 && page < p.num_pages;
        bad = bad || !in;
        keys[i] = in ? static_cast<uint32_t>(page * blocks_a_page + j - lp * blocks_a_page) : 0xffffffffu;
    }
    if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(p.status, BSATTN_ERR_BAD_INDEX);
    __syncthreads();

    // ---------------------------------------------------------------- scores
    {
        const int first_recent = max(all_n - p.recent, 0);
        const int r8 = lane >> 2, j4 = lane & 3, h0 = 2 * j4;
        float sq[2];                                        // (NaN of a head that there is not: no maximum takes it)
#pragma unroll
        for (int e = 0; e < 2; ++e) sq[e] = h0 + e < G ? qscale[h0 + e] : __int_as_float(0x7fffffff);
        uint32_t least = 0, most = 0;                       // of ~key, and of key
        int there = 0;                                      // and the forced ones, 2^16 each
        // Groups of 32 blocks in turn: the warp's m-th is group kWarps m + warp.  Where rows are 128 bytes, the two
        // halves of every second one change places, so that a quad's 16-byte reads of two rows meet no bank twice.
        uint8_t* ring = sel_smem + warp * kDepth * kGroup;
        const int groups = ((n + 31) / 32 - warp + kWarps - 1) / kWarps;
        constexpr int kChunks = D / 16, kRows = 32 / kChunks;       // of 16 bytes in a row; rows that a warp copies at once
        const int r_in = lane / kChunks, chunk = lane % kChunks;
        const int8_t* codes = p.codes + static_cast<size_t>(g) * D + chunk * 16;
        const size_t row_bytes = static_cast<size_t>(p.Hkv) * D;
        const uint32_t put = r_in * D + (D == 128 ? chunk ^ (r_in & 1) << 2 : chunk) * 16;
        const auto fetch = [&](int m) {
            if (m < groups) {
                const uint32_t to = smem_u32(ring + (m % kDepth) * kGroup);
                const int at = (m * kWarps + warp) * 32 + lane;
                uint32_t row = at < n ? keys[at] : 0u;
                if (row == 0xffffffffu) row = 0u;
#pragma unroll
                for (int e = 0; e < kChunks; ++e)
                    copy16(to + e * kRows * D + put, codes + __shfl_sync(0xffffffffu, row, kRows * e + r_in) * row_bytes);
                copy4(to + 32 * D + 4 * lane, p.scales + static_cast<size_t>(row) * p.Hkv + g);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        uint2 q2[kSteps];
#pragma unroll
        for (int k = 0; k < kSteps; ++k) q2[k] = qb[k][lane];
        float2 begin[kSums];
#pragma unroll
        for (int k = 0; k < kSums; ++k) begin[k] = *reinterpret_cast<const float2*>(&qbase[k][h0]);
#pragma unroll
        for (int m = 0; m < kDepth; ++m) fetch(m);
        for (int m = 0; m < groups; ++m) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
            __syncwarp();
            const uint8_t* stage = ring + (m % kDepth) * kGroup;
            float best[2][2];                                       // of blocks 16 t + 8 e + r8, over two heads
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                uint4 kc[2][D / 64];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int w = 0; w < D / 64; ++w) {
                        const int c = D == 128 ? (j4 + 4 * w) ^ (r8 & 1) << 2 : j4;
                        kc[e][w] = *reinterpret_cast<const uint4*>(stage + (16 * t + 8 * e + r8) * D + 16 * c);
                    }
                float c[kSums][4];
#pragma unroll
                for (int k = 0; k < kSums; ++k) {
                    c[k][0] = c[k][2] = begin[k].x;
                    c[k][1] = c[k][3] = begin[k].y;
                }
#pragma unroll
                for (int k = 0; k < kSteps; ++k) {
                    uint32_t a[4];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint4 v = kc[e][k / 4];
                        const uint32_t w = (k % 4 == 0 ? v.x : k % 4 == 1 ? v.y : k % 4 == 2 ? v.z : v.w) ^ 0x80808080u;
                        a[e] = __byte_perm(w, 0x64646464u, 0x4140);
                        a[e + 2] = __byte_perm(w, 0x64646464u, 0x4342);
                    }
                    mma16::mma16816<false>(c[k / 2], a, q2[k].x, q2[k].y);
                }
#pragma unroll
                for (int k = 1; k < kSums; ++k)
#pragma unroll
                    for (int e = 0; e < 4; ++e) c[0][e] += c[k][e];
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    best[t][e] = fmaxf(__fmul_rn(c[0][2 * e], sq[0]), __fmul_rn(c[0][2 * e + 1], sq[1]));
            }
            // over all heads, lane j of a quad block 16 (j / 2) + 8 (j % 2) + r8
            float top[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const float got = __shfl_xor_sync(0xffffffffu, j4 & 2 ? best[0][e] : best[1][e], 2);
                top[e] = fmaxf(j4 & 2 ? best[1][e] : best[0][e], got);
            }
            const float last = __shfl_xor_sync(0xffffffffu, j4 & 1 ? top[0] : top[1], 1);
            const float score = fmaxf(j4 & 1 ? top[1] : top[0], last);
            const int in_group = 8 * j4 + r8, i = (m * kWarps + warp) * 32 + in_group;
            const float sk = *reinterpret_cast<const float*>(stage + 32 * D + 4 * in_group);
            if (i < n) {
                uint32_t key = 0;
                if (keys[i] != 0xffffffffu) {
                    ++there;
                    if (block0 + i < p.sinks || block0 + i >= first_recent) {
                        key = kForced;
                        there += 1 << 16;
                    } else {
                        key = key_of(sk == INFINITY ? INFINITY : __fmul_rn(score, sk));
                        least = max(least, ~key);
                        most = max(most, key);
                    }
                }
                keys[i] = key;
            }
            __syncwarp();                                           // the stage is read
            fetch(m + kDepth);
        }
        // (a warp has fewer than 2^16 blocks)
        there = __reduce_add_sync(0xffffffffu, there);
        least = __reduce_max_sync(0xffffffffu, least);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            atomicMax(&own.range[0], least);
            atomicMax(&own.range[1], most);
            atomicAdd(&own.there, there & 0xffff);
            atomicAdd(&own.forced, there >> 16);
        }
    }
    __syncthreads();
    Shares& sh = CL > 1 ? all : own;
    if (CL > 1) {
        cluster_wait();
        // a lane a word of a CTA
        if (warp == 0 && lane / 4 < CL) {
            const uint32_t v = reinterpret_cast<const uint32_t*>(&own)[lane & 3];
            const uint32_t to = word_of(reinterpret_cast<const uint32_t*>(&all) + (lane & 3), lane / 4);
            if (lane & 2) add_to(to, v);
            else max_to(to, v);
        }
        cluster_arrive();
        cluster_wait();
    }

    // ---------------------------------------------------------------- the score that max_sel blocks reach
    uint32_t lo = 1;
    int spare = all_n;                                      // places for blocks whose score is lo itself
    const int there = sh.there;
    if (there > p.max_sel) {
        int c_hi = sh.forced;
        if (c_hi >= p.max_sel) {
            lo = kForced;                                   // the forced blocks take all places
        } else {
            uint32_t held[kHeld];
#pragma unroll
            for (int i = 0; i < kHeld; ++i) held[i] = i * TH + tid < n ? keys[i * TH + tid] : 0u;
            // count(lo) > max_sel > count(hi)
            lo = ~sh.range[0];
            uint32_t hi = sh.range[1] + 1;
            int c_lo = there;
            for (int step = 0; c_lo != p.max_sel && hi - lo > 1; ++step) {
                uint32_t t[4];
                thresholds(lo, hi, step, t);
                int c[2] = {0, 0};                          // two counts each, 2^16 apart
                const auto count = [&](uint32_t k) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) c[i] += (k >= t[2 * i] ? 1 : 0) + (k >= t[2 * i + 1] ? 0x10000 : 0);
                };
#pragma unroll
                for (int i = 0; i < kHeld; ++i) {
                    if (i * TH >= n) break;
                    count(held[i]);
                }
                for (int i = kHeld * TH + tid; i < n; i += TH) count(keys[i]);
                int* to = own.counts[step % 3];
                const int s0 = __reduce_add_sync(0xffffffffu, c[0]), s1 = __reduce_add_sync(0xffffffffu, c[1]);
                if (lane < 4) {
                    const int s = lane & 2 ? s1 : s0, v = lane & 1 ? s >> 16 : s & 0xffff;
                    if (v) atomicAdd(&to[lane], v);
                }
                __syncthreads();
                if (CL > 1) {
                    if (warp == 0 && lane / 4 < CL) add_to(word_of(&all.counts[step % 3][lane & 3], lane / 4), to[lane & 3]);
                    cluster_arrive();
                    cluster_wait();
                    to = all.counts[step % 3];
                }
                // the last threshold that max_sel blocks reach, and the first that fewer do
                int now[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) now[i] = static_cast<volatile int*>(to)[i];
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (now[i] >= p.max_sel) {
                        lo = t[i];
                        c_lo = now[i];
                    }
#pragma unroll
                for (int i = 3; i >= 0; --i)
                    if (now[i] < p.max_sel) {
                        hi = t[i];
                        c_hi = now[i];
                    }
                // everybody has read the counts of the trip before, which are those of the trip after next
                if (tid < 4) own.counts[(step + 2) % 3][tid] = all.counts[(step + 2) % 3][tid] = 0;
            }
            if (c_lo != p.max_sel) spare = p.max_sel - c_hi;
        }
    }

    // ---------------------------------------------------------------- the chosen blocks in order
    // warp w has the blocks [w * span, (w + 1) * span)
    const int span = ((n + kWarps - 1) / kWarps + 31) & ~31;
    const int j0 = min(warp * span, n), j1 = min(j0 + span, n);
    int over = 0, equal = 0;
    for (int j = j0 + lane; j < j1; j += 32) {
        over += keys[j] > lo;
        equal += keys[j] == lo;
    }
    over = __reduce_add_sync(0xffffffffu, over);
    equal = __reduce_add_sync(0xffffffffu, equal);
    if (lane == 0) {
        above[warp] = over;
        level[warp] = equal;
    }
    __syncthreads();
    int over_before = 0, equal_before = 0;
    if (CL > 1) {
        if (warp == 0) {
            const int o = __reduce_add_sync(0xffffffffu, lane < kWarps ? above[lane] : 0);
            const int e = __reduce_add_sync(0xffffffffu, lane < kWarps ? level[lane] : 0);
            if (lane < 2 * CL)
                asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(word_of(&at_rank[lane & 1][rank], lane >> 1)), "r"(lane & 1 ? e : o)
                             : "memory");
        }
        cluster_arrive();
        cluster_wait();
        for (int r = 0; r < rank; ++r) {
            over_before += at_rank[0][r];
            equal_before += at_rank[1][r];
        }
    }
    for (int w = 0; w < warp; ++w) {
        over_before += above[w];
        equal_before += level[w];
    }
    int32_t* out = p.out + static_cast<size_t>(row) * p.max_sel;
    const uint32_t below = (1u << lane) - 1u;
    for (int j = j0; j < j1; j += 32) {
        const uint32_t key = j + lane < j1 ? keys[j + lane] : 0u;
        const uint32_t is_over = __ballot_sync(0xffffffffu, key > lo);
        const uint32_t is_equal = __ballot_sync(0xffffffffu, key == lo);
        const int eq = equal_before + __popc(is_equal & below);
        const int at = over_before + __popc(is_over & below) + min(eq, spare);
        if (key > lo || (key == lo && eq < spare)) out[at] = block0 + j + lane;
        over_before += __popc(is_over);
        equal_before += __popc(is_equal);
    }
    // (the last warp has passed all blocks)
    if (rank == CL - 1 && warp == kWarps - 1)
        for (int j = over_before + min(equal_before, spare) + lane; j < p.max_sel; j += 32) out[j] = -1;
}

template <int D, bool BF16, int TH>
int launch_select(const SelectParams& prm, long long rows, int cluster, cudaStream_t st) {
    auto kern = select_kernel<D, BF16, TH>;
    const int blocks = prm.max_pages * (prm.page_size / kBlockRows);
    static std::atomic<unsigned long long> raised{0};
    int rc = raise_smem_limit(reinterpret_cast<const void*>(kern), 224 * 1024, raised);
    if (rc) return rc;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(rows * cluster));
    cfg.blockDim = dim3(TH);
    cfg.dynamicSmemBytes = TH / 32 * kDepth * (32 * D + 128) + 4 * static_cast<size_t>(((blocks + cluster - 1) / cluster + 31) & ~31);
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = static_cast<unsigned>(cluster);
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, prm) == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

template <int D, bool BF16>
int select(const SelectParams& prm, int B, cudaStream_t st) {
    int sms = num_sms_of_current_device();
    if (sms <= 0) sms = 148;
    const long long rows = static_cast<long long>(B) * prm.Hkv;
    const int blocks = prm.max_pages * (prm.page_size / kBlockRows);
    // Where a row can have an SM to itself, a CTA has 512 threads, and a long row a cluster of as many SMs as there are,
    // with 512 blocks a CTA at least (1 sequence of 8192 blocks, 8 kv heads: 12.9 us by clusters of eight, 35 by one
    // CTA; 2048 blocks: 11.1 by four, 12.5 by two; but 1024: 10.9 by two, 9.7 by one).  With few blocks the way through
    // its barriers is longer than the counts (512 blocks: 8.4 us, 7.9 by 128 threads; 257: 7.3 and 6.2).
    int cluster = 1;
    if (rows <= sms && blocks > 768) {
        while (cluster < kMaxCluster && rows * cluster * 2 <= sms && blocks >= std::max(1024 * cluster, 2048)) cluster *= 2;
        // (the rings of many warps and the keys of more blocks do not both fit)
        if (blocks <= 16384 * cluster) return launch_select<D, BF16, 512>(prm, rows, cluster, st);
    }
    // Small CTAs, four an SM: 192 rows of 512 blocks take 9.8 us, 15.5 by 512 threads.  Two to a row where they are at
    // once on the GPU and long (192 rows of 2048 blocks: 21.4 us, 23.5 by one; but 304 of 1024 18.8 and 16.3).
    cluster = rows * 2 <= 4 * sms && blocks >= 2048 ? 2 : 1;
    return launch_select<D, BF16, 128>(prm, rows, cluster, st);
}

// ------------------------------------------------------------------------------------------ prompts
//
// Two kernels.  One summarises the blocks of q and k, a warp each, HBM-bound (32 heads of 16384 tokens, d = 128, 268
// MB: 45 us, 6 TB/s); codes are kept as 16-bit whole numbers for the other, which takes 16 query blocks of a head a
// CTA: products by mma.sync m16n8k16 (whole numbers: exact), keys of the 16 rows in shared memory, then a warp a row
// to find its threshold and write its bytes (16 us there, a chain of latencies).  Under the causal rule a CTA goes no
// further than its rows see.


struct MaskParams {
    const void* x[2];                    // q, k
    long long sb[2], sh[2], ss[2];       // element strides: batch, head, row
    int H[2], S[2], n[2];                // heads, rows, blocks
    uint16_t* codes[2];                  // [B, H, n, d] bf16 whole numbers
    float* scales[2];                    // [B, H, n]
    uint8_t* mask;
    int B, topk, sinks, recent, dense, causal;
    int rows;                            // query blocks of a CTA: 16, or 8 where 16 rows of keys do not fit
    int pitch;                           // keys of a row: a multiple of 128, and 8 for the banks
    int wide;                            // four bytes of the mask can be written at once
};

template <int D, bool BF16, int WARPS, int BYTES>
__global__ void __launch_bounds__(32 * WARPS, 1) summarise_kernel(const MaskParams p) {
    using Ring = BlockRing<D, BYTES>;
    extern __shared__ __align__(128) uint8_t ring_smem[];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t of_q = static_cast<uint32_t>(p.B) * p.H[0] * p.n[0];
    const uint32_t tasks = of_q + static_cast<uint32_t>(p.B) * p.H[1] * p.n[1];
    const uint32_t stride = gridDim.x * WARPS;
    const Ring ring(ring_smem + warp * Ring::kBytes);
    struct Task {
        int t, b, h, j, count;
    };
    // neighbouring heads next to each other: in a projection's output their rows are neighbours
    const auto task_of = [&](uint32_t u) {
        Task k;
        k.t = u < of_q ? 0 : 1;
        if (k.t) u -= of_q;
        const uint32_t r = u / static_cast<uint32_t>(p.H[k.t]);
        k.h = static_cast<int>(u - r * p.H[k.t]);
        k.b = static_cast<int>(r / static_cast<uint32_t>(p.n[k.t]));
        k.j = static_cast<int>(r - static_cast<uint32_t>(k.b) * p.n[k.t]);
        k.count = min(p.S[k.t] - k.j * kBlockRows, kBlockRows);
        return k;
    };
    const auto fetch = [&](uint32_t u, int stage) {
        if (u < tasks) {
            const Task k = task_of(u);
            const uint16_t* src = static_cast<const uint16_t*>(p.x[k.t]) + k.b * p.sb[k.t] + k.h * p.sh[k.t] +
                                  static_cast<long long>(k.j) * kBlockRows * p.ss[k.t] + 8 * (lane % (D / 8));
            ring.fetch(stage, reinterpret_cast<const char*>(src), 2 * p.ss[k.t], k.count);
        }
        Ring::commit();
    };
    // (fewer than 2^31 tasks, and a stride below 2^16: nothing wraps)
    uint32_t u = blockIdx.x + gridDim.x * warp, ahead = u;
#pragma unroll
    for (int m = 0; m < Ring::kDepth; ++m, ahead += stride) fetch(ahead, m);
    for (int stage = 0; u < tasks; u += stride, ahead += stride, stage = (stage + 1) % Ring::kDepth) {
        Ring::wait();
        const Task k = task_of(u);
        float s[8];
        ring.template sum<BF16>(stage, s);
        fetch(ahead, stage);
        int code[8];
        const float scale = summarise<D>(s, k.count, code);
        const size_t to = (static_cast<size_t>(k.b) * p.H[k.t] + k.h) * p.n[k.t] + k.j;
        if (lane < D / 8) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 v = __floats2bfloat162_rn(static_cast<float>(code[2 * e]), static_cast<float>(code[2 * e + 1]));
                w[e] = *reinterpret_cast<const uint32_t*>(&v);
            }
            *reinterpret_cast<uint4*>(p.codes[k.t] + to * D + 8 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
            if (lane == 0) p.scales[k.t][to] = scale;
        }
    }
}

template <int D, int TH>
__global__ void __launch_bounds__(TH, TH == 256 ? 3 : 1) mask_kernel(const MaskParams p) {
    constexpr int kMaskWarps = TH / 32;
    extern __shared__ __align__(16) uint32_t keys[];        // [rows][pitch]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int nq = p.n[0], nk = p.n[1];
    const int strips = (nq + p.rows - 1) / p.rows;
    // the last rows, which see the most, first
    const int strip = strips - 1 - static_cast<int>(blockIdx.x) / (p.B * p.H[0]);
    const int bh = static_cast<int>(blockIdx.x) % (p.B * p.H[0]);
    const int b = bh / p.H[0], h = bh - b * p.H[0], kvh = h / (p.H[0] / p.H[1]);
    const int row0 = strip * p.rows, past = p.S[1] - p.S[0];
    // how many key blocks row r sees
    const auto seen = [&](int r) {
        if (!p.causal) return nk;
        const int last = min(r * kBlockRows + kBlockRows, p.S[0]) - 1 + past;
        return last < 0 ? 0 : last / kBlockRows + 1;
    };
    const int widest = seen(min(row0 + p.rows, nq) - 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");      // the summaries are there
    // ---------------------------------------------------------------- keys: a warp takes eight key blocks at a time
    {
        const int r8 = lane >> 2, j4 = lane & 3;
        // which channel a matrix index stands for is free: a lane of a quad takes D / 4 consecutive ones
        uint32_t a[D / 16][4];
        float sq[2];
        const size_t qbase = static_cast<size_t>(b) * p.H[0] + h;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int r = row0 + r8 + 8 * half;
            const bool on = r < nq && r8 + 8 * half < p.rows;
            const uint4* src = reinterpret_cast<const uint4*>(p.codes[0] + (qbase * nq + (on ? r : 0)) * D + j4 * (D / 4));
#pragma unroll
            for (int w = 0; w < D / 32; ++w) {
                const uint4 v = on ? src[w] : make_uint4(0, 0, 0, 0);
                a[2 * w][half] = v.x;
                a[2 * w][half + 2] = v.y;
                a[2 * w + 1][half] = v.z;
                a[2 * w + 1][half + 2] = v.w;
            }
            const float s = on ? p.scales[0][qbase * nq + r] : 0.f;
            sq[half] = s == INFINITY ? 0.f : s;             // a query block that is not finite scores 0
        }
        const size_t kbase = (static_cast<size_t>(b) * p.H[1] + kvh) * nk;
        // (the padding of a row stays unwritten)
        const int tiles = p.pitch / 8 - 1;
        uint4 next[D / 32];                                 // the next tile's codes and scales, on their way
        float next_scale[2];
        const auto fetch = [&](int tile) {
            const int c0 = 8 * tile;
            if (c0 >= widest) return;
            const uint4* src = reinterpret_cast<const uint4*>(p.codes[1] + (kbase + min(c0 + r8, nk - 1)) * D + j4 * (D / 4));
#pragma unroll
            for (int w = 0; w < D / 32; ++w) next[w] = src[w];
#pragma unroll
            for (int e = 0; e < 2; ++e) next_scale[e] = p.scales[1][kbase + min(c0 + 2 * j4 + e, nk - 1)];
        };
        fetch(warp);
        for (int tile = warp; tile < tiles; tile += kMaskWarps) {
            const int c0 = 8 * tile;
            uint2 put[2] = {};
            if (c0 < widest) {
                float c[4] = {};
                const float sk[2] = {next_scale[0], next_scale[1]};
                uint4 kv[D / 32];
#pragma unroll
                for (int w = 0; w < D / 32; ++w) kv[w] = next[w];
                fetch(tile + kMaskWarps);
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    mma16::mma16816<true>(c, a[2 * w], kv[w].x, kv[w].y);
                    mma16::mma16816<true>(c, a[2 * w + 1], kv[w].z, kv[w].w);
                }
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const int r = row0 + r8 + 8 * half;
                    const int n = r < nq ? seen(r) : 0;
                    uint32_t k2[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int at = c0 + 2 * j4 + e;
                        k2[e] = key_of(sk[e] == INFINITY ? INFINITY : __fmul_rn(__fmul_rn(c[2 * half + e], sq[half]), sk[e]));
                        if (at < p.sinks || at >= n - p.recent || (p.dense && r >= nq - 2)) k2[e] = kForced;
                        if (at >= n) k2[e] = 0;
                    }
                    put[half] = make_uint2(k2[0], k2[1]);
                }
            }
#pragma unroll
            for (int half = 0; half < 2; ++half)
                if (r8 + 8 * half < p.rows)
                    *reinterpret_cast<uint2*>(keys + static_cast<size_t>(r8 + 8 * half) * p.pitch + c0 + 2 * j4) = put[half];
        }
    }
    __syncthreads();
    // ---------------------------------------------------------------- a warp a row
    for (int i = warp; i < p.rows && row0 + i < nq; i += kMaskWarps) {
        const uint32_t* mine = keys + static_cast<size_t>(i) * p.pitch;
        const int n = seen(row0 + i);
        uint32_t lo = 1;
        int spare = nk;
        // the lane's keys: four of every 128, those of the first 256 in registers; 0 where there is none
        uint4 held[2];
#pragma unroll
        for (int c = 0; c < 2; ++c)
            held[c] = 128 * c < n ? *reinterpret_cast<const uint4*>(mine + 128 * c + 4 * lane) : make_uint4(0, 0, 0, 0);
        const auto every = [&](const auto& f) {
            f(held[0]);
            if (n > 128) f(held[1]);
            for (int j = 256 + 4 * lane; j < n; j += 128) f(*reinterpret_cast<const uint4*>(mine + j));
        };
        if (n > p.topk) {
            uint32_t least = 0xffffffffu, most = 0;
            int forced = 0;
            every([&](const uint4& k4) {
                const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    forced += k[e] == kForced;
                    if (k[e] != kForced) most = max(most, k[e]);
                    least = min(least, k[e] - 1u);          // (0 becomes the largest)
                }
            });
            forced = __reduce_add_sync(0xffffffffu, forced);
            least = __reduce_min_sync(0xffffffffu, least) + 1u;
            most = __reduce_max_sync(0xffffffffu, most);
            if (forced >= p.topk) {
                lo = kForced;
            } else {
                // count(lo) > topk > count(hi)
                lo = least;
                uint32_t hi = most + 1;
                int c_lo = n, c_hi = forced;
                for (int step = 0; c_lo != p.topk && hi - lo > 1; ++step) {
                    uint32_t t[4];
                    thresholds(lo, hi, step, t);
                    int c[2] = {0, 0};                      // two counts each, 2^16 apart
                    every([&](const uint4& k4) {
                        const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e)
#pragma unroll
                            for (int i = 0; i < 2; ++i) c[i] += (k[e] >= t[2 * i] ? 1 : 0) + (k[e] >= t[2 * i + 1] ? 0x10000 : 0);
                    });
#pragma unroll
                    for (int i = 0; i < 2; ++i) c[i] = __reduce_add_sync(0xffffffffu, c[i]);
                    const int now[4] = {c[0] & 0xffff, c[0] >> 16, c[1] & 0xffff, c[1] >> 16};
                    // the last threshold that topk blocks reach, and the first that fewer do
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (now[i] >= p.topk) {
                            lo = t[i];
                            c_lo = now[i];
                        }
#pragma unroll
                    for (int i = 3; i >= 0; --i)
                        if (now[i] < p.topk) {
                            hi = t[i];
                            c_hi = now[i];
                        }
                }
                if (c_lo != p.topk) spare = p.topk - c_hi;
            }
        }
        uint8_t* out = p.mask + (static_cast<size_t>(bh) * nq + row0 + i) * nk;
        const uint32_t below = (1u << lane) - 1u;
        int equal_before = 0;
        for (int j = 4 * lane; j - 4 * lane < nk; j += 128) {
            const uint4 k4 = j < 128 ? held[0] : j < 256 ? held[1] : j < n ? *reinterpret_cast<const uint4*>(mine + j) : make_uint4(0, 0, 0, 0);
            const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
            uint32_t equal[4];
            int rank = equal_before;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                equal[e] = __ballot_sync(0xffffffffu, k[e] == lo);
                rank += __popc(equal[e] & below);
                equal_before += __popc(equal[e]);
            }
            uint32_t on = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if (k[e] > lo || (k[e] == lo && rank < spare)) on |= 1u << 8 * e;
                rank += k[e] == lo;
            }
            if (p.wide) {
                if (j < nk) *reinterpret_cast<uint32_t*>(out + j) = on;
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (j + e < nk) out[j + e] = static_cast<uint8_t>(on >> 8 * e);
            }
        }
    }
}

// Byte offsets of the workspace: summaries of q, then of k.
struct MaskLayout {
    size_t codes[2], scales[2], total;
};

MaskLayout mask_layout(int B, int Hq, int Hkv, int Sq, int Sk, int d) {
    const auto blocks = [](int rows) { return (static_cast<size_t>(rows) + kBlockRows - 1) / kBlockRows; };
    const size_t n[2] = {static_cast<size_t>(B) * Hq * blocks(Sq), static_cast<size_t>(B) * Hkv * blocks(Sk)};
    MaskLayout w{};
    size_t at = 256;
    for (int t = 0; t < 2; ++t) {
        w.codes[t] = at;
        at += up256(n[t] * d * 2);
        w.scales[t] = at;
        at += up256(n[t] * 4);
    }
    w.total = at;
    return w;
}

template <int D, int TH>
int launch_rows(const MaskParams& prm, cudaStream_t st) {
    auto kern = mask_kernel<D, TH>;
    static std::atomic<unsigned long long> raised{0};
    const int rc = raise_smem_limit(reinterpret_cast<const void*>(kern), 224 * 1024, raised);
    if (rc) return rc;
    const int strips = (prm.n[0] + prm.rows - 1) / prm.rows;
    // launched while the summaries are still being made: it waits for them itself
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(strips) * prm.B * prm.H[0]);
    cfg.blockDim = dim3(TH);
    cfg.dynamicSmemBytes = static_cast<size_t>(prm.rows) * prm.pitch * 4;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, prm) == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

template <int D, bool BF16, int WARPS, int BYTES>
int launch_summaries(const MaskParams& prm, long long tasks, int sms, cudaStream_t st) {
    auto kern = summarise_kernel<D, BF16, WARPS, BYTES>;
    static std::atomic<unsigned long long> raised{0};
    const int rc = raise_smem_limit(reinterpret_cast<const void*>(kern), WARPS * BYTES, raised);
    if (rc) return rc;
    // a task a CTA first, then more
    kern<<<static_cast<unsigned>(std::min<long long>(tasks, sms)), 32 * WARPS, WARPS * BYTES, st>>>(prm);
    return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

template <int D, bool BF16>
int launch_mask(const MaskParams& prm, cudaStream_t st) {
    const long long tasks = static_cast<long long>(prm.B) * (static_cast<long long>(prm.H[0]) * prm.n[0] +
                                                             static_cast<long long>(prm.H[1]) * prm.n[1]);
    int sms = num_sms_of_current_device();
    if (sms <= 0) sms = 148;
    // Seven warps with 32 KB each where a warp has few blocks, and the way of the last one counts (2048 blocks: 13.4 us
    // for both kernels, 14.7 by four warps), four with 48 KB where it has many (16384 blocks: 60.8 us, 62.7 by seven).
    const int rc = tasks < 32LL * sms ? launch_summaries<D, BF16, 7, 32768>(prm, tasks, sms, st)
                                      : launch_summaries<D, BF16, 4, 49152>(prm, tasks, sms, st);
    if (rc) return rc;
    // 16 rows by 16 warps where every CTA has an SM to itself (64 CTAs of 64 key blocks: 13.5 us for both kernels, 15.5
    // by 8 warps), by 8 where there are more (512 CTAs of 256 key blocks: 61 us, 69 by 16 warps)
    const long long ctas = static_cast<long long>((prm.n[0] + prm.rows - 1) / prm.rows) * prm.B * prm.H[0];
    return ctas <= sms ? launch_rows<D, 512>(prm, st) : launch_rows<D, 256>(prm, st);
}

}  // namespace
}  // namespace bsattn

extern "C" int bsattn_decode_select(const void* q, const int8_t* codes, const float* scales,
                                    const int32_t* cache_seqlens, const int32_t* block_table, int sinks, int recent,
                                    int32_t* block_indices, int B, int Hq, int Hkv, int num_pages, int page_size,
                                    int max_pages_per_seq, int d, int max_sel, bsattn_dtype dtype, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    using namespace bsattn;
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || num_pages <= 0 || page_size <= 0 || max_pages_per_seq <= 0 ||
        max_sel <= 0 || sinks < 0 || recent < 0 || sinks > max_sel - std::min(recent, max_sel))
        return BSATTN_ERR_INVALID_ARG;
    if (recent > max_sel) return BSATTN_ERR_INVALID_ARG;
    if (Hq / Hkv > 8 || page_size % kBlockRows || (d != 64 && d != 128)) return BSATTN_ERR_UNSUPPORTED;
    if (dtype != BSATTN_F16 && dtype != BSATTN_BF16) return BSATTN_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < 256 || !aligned16(workspace)) return BSATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL || max_sel > (1 << 26) ||
        static_cast<long long>(max_pages_per_seq) * (page_size / kBlockRows) > kMaxBlocks ||
        static_cast<long long>(B) * Hkv > 0x7fffffffLL)
        return BSATTN_ERR_UNSUPPORTED;
    if (B == 0) return BSATTN_OK;
    if (!q || !codes || !scales || !cache_seqlens || !block_table || !block_indices) return BSATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(codes) || !aligned16(scales)) return BSATTN_ERR_INVALID_ARG;
    const size_t blocks = static_cast<size_t>(num_pages) * (page_size / kBlockRows) * Hkv;
    const size_t out_bytes = sizeof(int32_t) * B * Hkv * max_sel, lens = sizeof(int32_t) * B;
    if (overlap(block_indices, out_bytes, q, static_cast<size_t>(B) * Hq * d * 2) ||
        overlap(block_indices, out_bytes, codes, blocks * d) || overlap(block_indices, out_bytes, scales, blocks * 4) ||
        overlap(block_indices, out_bytes, cache_seqlens, lens) ||
        overlap(block_indices, out_bytes, block_table, lens * max_pages_per_seq))
        return BSATTN_ERR_INVALID_ARG;
    SelectParams prm{};
    prm.q = q;
    prm.codes = codes;
    prm.scales = scales;
    prm.seqlens = cache_seqlens;
    prm.table = block_table;
    prm.out = block_indices;
    prm.status = status_word(workspace);
    prm.Hq = Hq;
    prm.Hkv = Hkv;
    prm.page_size = page_size;
    prm.max_pages = max_pages_per_seq;
    prm.num_pages = num_pages;
    prm.max_sel = max_sel;
    prm.sinks = sinks;
    prm.recent = recent;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == BSATTN_BF16;
    if (d == 64) return bf16 ? select<64, true>(prm, B, st) : select<64, false>(prm, B, st);
    return bf16 ? select<128, true>(prm, B, st) : select<128, false>(prm, B, st);
}

extern "C" size_t bsattn_mask_from_qk_workspace_size(int B, int Hq, int Hkv, int Sq, int Sk, int d) {
    if (B <= 0 || Hq <= 0 || Hkv <= 0 || Sq <= 0 || Sk <= 0 || d <= 0) return 256;
    return bsattn::mask_layout(B, Hq, Hkv, Sq, Sk, d).total;
}

extern "C" int bsattn_mask_from_qk(const void* q, const void* k, int topk, int sinks, int recent,
                                   int use_dense_for_last_block, int is_causal, uint8_t* mask_out, int B, int Hq,
                                   int Hkv, int Sq, int Sk, int d, const int64_t* strides, bsattn_dtype dtype,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    using namespace bsattn;
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || Sq < 0 || Sk < 0 || topk < 0 || sinks < 0 || recent < 0)
        return BSATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return BSATTN_ERR_UNSUPPORTED;
    if (dtype != BSATTN_F16 && dtype != BSATTN_BF16) return BSATTN_ERR_UNSUPPORTED;
    if (Sq > (1 << 30) || Sk > (1 << 30)) return BSATTN_ERR_UNSUPPORTED;
    if (!workspace || !aligned16(workspace)) return BSATTN_ERR_INVALID_ARG;
    if (B == 0 || Sq == 0 || Sk == 0) return BSATTN_OK;         // an empty mask
    const MaskLayout w = mask_layout(B, Hq, Hkv, Sq, Sk, d);
    if (workspace_bytes < w.total) return BSATTN_ERR_INVALID_ARG;
    if (!q || !k || !mask_out || !aligned16(q) || !aligned16(k)) return BSATTN_ERR_INVALID_ARG;
    const int64_t dense_q[3] = {int64_t(Hq) * Sq * d, int64_t(Sq) * d, d}, dense_k[3] = {int64_t(Hkv) * Sk * d, int64_t(Sk) * d, d};
    const int64_t* st[2] = {strides ? strides : dense_q, strides ? strides + 3 : dense_k};
    MaskParams prm{};
    const int H[2] = {Hq, Hkv}, S[2] = {Sq, Sk};
    const void* x[2] = {q, k};
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    for (int t = 0; t < 2; ++t) {
        const int entries[3] = {B, H[t], S[t]};
        long long s[3];
        for (int e = 0; e < 3; ++e) {
            s[e] = entries[e] > 1 ? st[t][e] : 0;               // the stride of a dimension of one entry is never used
            if (s[e] < 0 || (s[e] & 7) || s[e] > (1LL << 40)) return BSATTN_ERR_INVALID_ARG;
        }
        prm.x[t] = x[t];
        prm.sb[t] = s[0];
        prm.sh[t] = s[1];
        prm.ss[t] = s[2];
        prm.H[t] = H[t];
        prm.S[t] = S[t];
        prm.n[t] = (S[t] + kBlockRows - 1) / kBlockRows;
        prm.codes[t] = reinterpret_cast<uint16_t*>(ws + w.codes[t]);
        prm.scales[t] = reinterpret_cast<float*>(ws + w.scales[t]);
    }
    const size_t mask_bytes = static_cast<size_t>(B) * Hq * prm.n[0] * prm.n[1];
    for (int t = 0; t < 2; ++t) {
        const size_t span = 2 * (static_cast<size_t>(B - 1) * prm.sb[t] + static_cast<size_t>(H[t] - 1) * prm.sh[t] +
                                 static_cast<size_t>(S[t] - 1) * prm.ss[t] + d);
        if (overlap(mask_out, mask_bytes, x[t], span) || overlap(ws, w.total, x[t], span)) return BSATTN_ERR_INVALID_ARG;
    }
    if (overlap(mask_out, mask_bytes, ws, w.total)) return BSATTN_ERR_INVALID_ARG;
    prm.mask = mask_out;
    prm.B = B;
    prm.topk = topk;
    prm.sinks = sinks;
    prm.recent = recent;
    prm.dense = use_dense_for_last_block != 0;
    prm.causal = is_causal != 0;
    prm.pitch = ((prm.n[1] + 127) & ~127) + 8;
    prm.wide = prm.n[1] % 4 == 0 && reinterpret_cast<uintptr_t>(mask_out) % 4 == 0;
    // 16 rows of keys, or 8 where they do not fit
    prm.rows = 16 * 4LL * prm.pitch <= 224 * 1024 ? 16 : 8;
    if (static_cast<long long>(prm.rows) * 4 * prm.pitch > 224 * 1024) return BSATTN_ERR_UNSUPPORTED;
    const long long tasks = static_cast<long long>(B) * (static_cast<long long>(Hq) * prm.n[0] + static_cast<long long>(Hkv) * prm.n[1]);
    if (tasks > 0x7fffffffLL) return BSATTN_ERR_UNSUPPORTED;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == BSATTN_BF16;
    if (d == 64) return bf16 ? launch_mask<64, true>(prm, cs) : launch_mask<64, false>(prm, cs);
    return bf16 ? launch_mask<128, true>(prm, cs) : launch_mask<128, false>(prm, cs);
}
