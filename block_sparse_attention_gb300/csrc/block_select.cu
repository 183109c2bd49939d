// block_select.cu -- the key blocks of a decode query, and the block mask of a prompt, by the product of
// 8-bit summaries (summary.cuh), sm_103a.
//
// The score of a key block for a query is (their codes' whole-number product) * (query scale) * (key scale),
// two 32-bit roundings; a decode's kv head takes the largest of its query heads' first products.  Chosen
// are blocks that are asked for whatever their score (the first ones, the last ones), then the best others
// up to the wanted number, the lower block first among equals.
//
// The choice is a search for the score that the wanted number of blocks reach: counts of blocks at or above
// a threshold, halving what lies between, until the count is right or one score is left.  With scores spread
// evenly it takes about as many counts as the number of blocks has bits.
#include <algorithm>

#include "host_internal.h"
#include "ptx.cuh"
#include "summary.cuh"

namespace bsattn {
namespace {

// ------------------------------------------------------------------------------------------ decode
//
// One CTA a (sequence, kv head).  An index row (codes of a block of one head) is read by d / 16 lanes, 16
// bytes each, against the query heads' codes in registers: four whole-number products an instruction
// (dp4a), and the lanes' sums added by exchanging halves (V values over L lanes in V - V / L exchanges).
// The index is read once, which bounds a large batch; a small one is a chain of latencies: lengths, table,
// index, then the counts.

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kMaxBlocks = 51200;               // of a sequence: their keys lie in shared memory

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

// The sum of `mine` over the CTA, the same in all threads.  Counters are used in turn, `nth` counting the calls.
__device__ __forceinline__ int cta_sum(int mine, int (&counter)[3], int nth) {
    const int w = __reduce_add_sync(0xffffffffu, mine);
    if ((threadIdx.x & 31) == 0 && w) atomicAdd(&counter[nth % 3], w);
    __syncthreads();
    // everybody has read the counter of the call before, which is the one of the call after next
    if (threadIdx.x == 0) counter[(nth + 2) % 3] = 0;
    return *static_cast<volatile int*>(&counter[nth % 3]);
}

// GP: query heads of a kv head, rounded up to a power of two.
template <int D, bool BF16, int GP>
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectParams p) {
    constexpr int kLanes = D / 16;                          // of an index row
    constexpr int kRows = 32 / kLanes;                      // that a warp reads at once
    constexpr int kPasses = kLanes > GP ? kLanes / GP : 1;  // reads whose sums are added together
    constexpr int kV = kPasses * GP, kR = kV / kLanes;      // values, and those a lane is left with
    constexpr int kUnroll = kPasses >= 4 ? 1 : (kPasses == 2 ? 2 : 4);
    extern __shared__ uint32_t keys[];                      // first each block's index row, then its key
    __shared__ __align__(16) int8_t qcodes[8][D];
    __shared__ float qscale[8];
    __shared__ int counter[3];
    __shared__ uint32_t range[2];                           // smallest and largest key
    __shared__ int above[kSelWarps], level[kSelWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int b = blockIdx.x / p.Hkv, g = blockIdx.x - b * p.Hkv, G = p.Hq / p.Hkv;

    const int asked = p.seqlens[b];
    const int blocks_a_page = p.page_size / kBlockRows;
    const int room = p.max_pages * blocks_a_page;
    const bool far = asked < 0 || asked > static_cast<long long>(p.max_pages) * p.page_size;
    const int n = asked <= 0 ? 0 : min(asked / kBlockRows + (asked % kBlockRows != 0), room);
    if (tid < 3) counter[tid] = 0;
    if (tid == 0) {
        range[0] = 0xffffffffu;
        range[1] = 0;
    }
    // the index row of each block, or -1
    bool bad = far;
    for (int j = tid; j < n; j += kSelThreads) {
        const int lp = j / blocks_a_page;
        const int page = p.table[static_cast<size_t>(b) * p.max_pages + lp];
        const bool in = page >= 0 && page < p.num_pages;
        bad = bad || !in;
        keys[j] = in ? static_cast<uint32_t>(page * blocks_a_page + j - lp * blocks_a_page) : 0xffffffffu;
    }
    if (bad && (lane == 0 || !far)) atomicOr(p.status, BSATTN_ERR_BAD_INDEX);
    // a warp a query head: its codes and scale
    if (warp < G) {
        const uint32_t* src = reinterpret_cast<const uint32_t*>(static_cast<const uint16_t*>(p.q) +
                                                                (static_cast<size_t>(b) * p.Hq + g * G + warp) * D);
        float x[D / 32], top = 0.f;
        bool finite = true;
#pragma unroll
        for (int w = 0; w < D / 64; ++w) {
            const float2 f = two_floats<BF16>(src[lane * (D / 64) + w]);
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
#pragma unroll
        for (int e = 0; e < D / 32; ++e) qcodes[warp][lane * (D / 32) + e] = static_cast<int8_t>(code8(x[e], scale, finite));
        if (lane == 0) qscale[warp] = finite ? scale : 0.f;         // a query that is not finite scores 0
    }
    __syncthreads();

    // ---------------------------------------------------------------- scores
    const int first_recent = max(n - p.recent, 0);
    {
        const int sub = lane / kLanes, part = lane % kLanes;
        int4 qc[GP];
#pragma unroll
        for (int h = 0; h < GP; ++h)
            qc[h] = h < G ? *reinterpret_cast<const int4*>(&qcodes[h][16 * part]) : make_int4(0, 0, 0, 0);
        // after the exchanges a lane has values kR part + {0 .. kR - 1}: value v is head v % GP of read v / GP
        const int my_pass = kR * part / GP, my_head = kR * part % GP;
        float sq[kR];
#pragma unroll
        for (int r = 0; r < kR; ++r) sq[r] = my_head + r < G ? qscale[my_head + r] : 0.f;
        uint32_t least = 0xffffffffu, most = 0;
        constexpr int kStep = kRows * kPasses;              // blocks of a warp at a time
        for (int base = warp * kStep; base < n; base += kSelWarps * kStep * kUnroll) {
            int4 kc[kUnroll][kPasses];
            float sk[kUnroll];
            uint32_t row_of_mine[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int at = base + u * kSelWarps * kStep;
#pragma unroll
                for (int i = 0; i < kPasses; ++i) {
                    const int j = at + i * kRows + sub;
                    const uint32_t row = j < n ? keys[j] : 0xffffffffu;
                    kc[u][i] = make_int4(0, 0, 0, 0);
                    if (row != 0xffffffffu)
                        kc[u][i] = __ldg(reinterpret_cast<const int4*>(p.codes + (static_cast<size_t>(row) * p.Hkv + g) * D) + part);
                }
                const int j = at + my_pass * kRows + sub;
                row_of_mine[u] = j < n ? keys[j] : 0xffffffffu;
                sk[u] = row_of_mine[u] != 0xffffffffu ? __ldg(p.scales + static_cast<size_t>(row_of_mine[u]) * p.Hkv + g) : 0.f;
            }
            __syncwarp();                                   // the rows are read: keys may take their places
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                int v[kV];
#pragma unroll
                for (int i = 0; i < kPasses; ++i)
#pragma unroll
                    for (int h = 0; h < GP; ++h) {
                        int s = __dp4a(kc[u][i].x, qc[h].x, 0);
                        s = __dp4a(kc[u][i].y, qc[h].y, s);
                        s = __dp4a(kc[u][i].z, qc[h].z, s);
                        v[i * GP + h] = __dp4a(kc[u][i].w, qc[h].w, s);
                    }
#pragma unroll
                for (int m = kLanes / 2, half = kV / 2; m > 0; m >>= 1, half >>= 1) {
                    const bool upper = (lane & m) != 0;
#pragma unroll
                    for (int i = 0; i < half; ++i) {
                        const int keep = upper ? v[i + half] : v[i], give = upper ? v[i] : v[i + half];
                        v[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
                    }
                }
                float best = -INFINITY;
#pragma unroll
                for (int r = 0; r < kR; ++r)
                    if (my_head + r < G) best = fmaxf(best, __fmul_rn(static_cast<float>(v[r]), sq[r]));
#pragma unroll
                for (int m = 1; m < GP / kR; m <<= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, m));
                const int j = base + u * kSelWarps * kStep + my_pass * kRows + sub;
                if (my_head == 0 && j < n) {
                    uint32_t key = 0;
                    if (row_of_mine[u] != 0xffffffffu) {
                        key = key_of(sk[u] == INFINITY ? INFINITY : __fmul_rn(best, sk[u]));
                        if (j < p.sinks || j >= first_recent) {
                            key = kForced;
                        } else {
                            least = min(least, key);
                            most = max(most, key);
                        }
                    }
                    keys[j] = key;
                }
            }
        }
        least = __reduce_min_sync(0xffffffffu, least);
        most = __reduce_max_sync(0xffffffffu, most);
        if (lane == 0) {
            atomicMin(&range[0], least);
            atomicMax(&range[1], most);
        }
    }
    __syncthreads();

    // ---------------------------------------------------------------- the score that max_sel blocks reach
    int nth = 0;
    const auto count = [&](uint32_t t) {
        int c = 0;
        for (int j = tid; j < n; j += kSelThreads) c += keys[j] >= t;
        return cta_sum(c, counter, nth++);
    };
    uint32_t lo = 1;
    int spare = n;                                          // places for blocks whose score is lo itself
    if (n > p.max_sel) {
        int c_lo = count(1);
        if (c_lo > p.max_sel) {
            // count(lo) >= max_sel > count(hi), hi = most + 1 (there are no more forced blocks than places)
            lo = range[0];
            uint32_t hi = range[1] + 1;
            int c_hi = count(hi);
            if (c_hi >= p.max_sel) {                        // the forced blocks take all places
                lo = hi;
                c_lo = c_hi;
            }
            for (int step = 0; c_lo != p.max_sel && hi - lo > 1; ++step) {
                const uint32_t mid = between(lo, hi, step);
                const int c = count(mid);
                if (c >= p.max_sel) {
                    lo = mid;
                    c_lo = c;
                } else {
                    hi = mid;
                    c_hi = c;
                }
            }
            if (c_lo != p.max_sel) spare = p.max_sel - c_hi;
        }
    }

    // ---------------------------------------------------------------- the chosen blocks in order
    // warp w has the blocks [w * each, (w + 1) * each)
    const int each = ((n + kSelWarps - 1) / kSelWarps + 31) & ~31;
    const int j0 = min(warp * each, n), j1 = min(j0 + each, n);
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
    int over_before = 0, equal_before = 0, all = 0, all_equal = 0;
#pragma unroll
    for (int w = 0; w < kSelWarps; ++w) {
        if (w == warp) {
            over_before = all;
            equal_before = all_equal;
        }
        all += above[w];
        all_equal += level[w];
    }
    int32_t* out = p.out + static_cast<size_t>(blockIdx.x) * p.max_sel;
    const uint32_t below = (1u << lane) - 1u;
    for (int j = j0; j < j1; j += 32) {
        const uint32_t key = j + lane < j1 ? keys[j + lane] : 0u;
        const uint32_t is_over = __ballot_sync(0xffffffffu, key > lo);
        const uint32_t is_equal = __ballot_sync(0xffffffffu, key == lo);
        const int eq = equal_before + __popc(is_equal & below);
        const int at = over_before + __popc(is_over & below) + min(eq, spare);
        if (key > lo || (key == lo && eq < spare)) out[at] = j + lane;
        over_before += __popc(is_over);
        equal_before += __popc(is_equal);
    }
    for (int j = all + min(all_equal, spare) + tid; j < p.max_sel; j += kSelThreads) out[j] = -1;
}

template <int D, bool BF16, int GP>
int launch_select(const SelectParams& prm, int B, cudaStream_t st) {
    auto kern = select_kernel<D, BF16, GP>;
    const int blocks = prm.max_pages * (prm.page_size / kBlockRows);
    static std::atomic<unsigned long long> raised{0};
    const int rc = raise_smem_limit(reinterpret_cast<const void*>(kern), 4 * kMaxBlocks, raised);
    if (rc) return rc;
    kern<<<static_cast<unsigned>(B) * prm.Hkv, kSelThreads, 4 * static_cast<size_t>(blocks), st>>>(prm);
    return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

// ------------------------------------------------------------------------------------------ prompts
//
// Two kernels: one summarises the blocks of q and k (a warp each, HBM-bound), codes kept as 16-bit whole
// numbers for the second, which takes 16 query blocks of a head a CTA: products by mma.sync m16n8k16 (whole
// numbers: exact), keys of the 16 rows in shared memory, then a warp a row to find its threshold and write
// its bytes.  Under the causal rule a CTA goes no further than its rows see.

constexpr int kMaskThreads = 512;
constexpr int kMaskWarps = kMaskThreads / 32;

struct MaskParams {
    const void* x[2];                    // q, k
    long long sb[2], sh[2], ss[2];       // element strides: batch, head, row
    int H[2], S[2], n[2];                // heads, rows, blocks
    uint16_t* codes[2];                  // [B, H, n, d] bf16 whole numbers
    float* scales[2];                    // [B, H, n]
    uint8_t* mask;
    int B, topk, sinks, recent, dense, causal;
    int rows;                            // query blocks of a CTA: 16, or 8 where 16 rows of keys do not fit
    int pitch;                           // keys of a row, a multiple of 128
};

template <int D, bool BF16>
__global__ void __launch_bounds__(256) summarise_kernel(const MaskParams p) {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const int lane = threadIdx.x & 31;
    long long task = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const long long of_q = static_cast<long long>(p.B) * p.H[0] * p.n[0];
    const int t = task < of_q ? 0 : 1;
    if (t) task -= of_q;
    const int H = p.H[t], n = p.n[t];
    if (task >= static_cast<long long>(p.B) * H * n) return;
    // neighbouring heads next to each other: in a projection's output their rows are neighbours
    const uint32_t u = static_cast<uint32_t>(task);
    const int h = static_cast<int>(u % static_cast<uint32_t>(H));
    const uint32_t r = u / static_cast<uint32_t>(H);
    const int j = static_cast<int>(r % static_cast<uint32_t>(n)), b = static_cast<int>(r / static_cast<uint32_t>(n));
    const int count = min(p.S[t] - j * kBlockRows, kBlockRows);
    const uint16_t* src = static_cast<const uint16_t*>(p.x[t]) + b * p.sb[t] + h * p.sh[t] +
                          static_cast<long long>(j) * kBlockRows * p.ss[t] + 8 * (lane % (D / 8));
    const long long step = p.ss[t];
    float s[8];
    block_sum<D, BF16>([&](int row) { return reinterpret_cast<const uint4*>(src + row * step); }, count, s);
    int code[8];
    const float scale = summarise<D>(s, count, code);
    const size_t to = (static_cast<size_t>(b) * H + h) * n + j;
    if (lane < D / 8) {
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(static_cast<float>(code[2 * e]), static_cast<float>(code[2 * e + 1]));
            w[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        *reinterpret_cast<uint4*>(p.codes[t] + to * D + 8 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
        if (lane == 0) p.scales[t][to] = scale;
    }
}

__device__ __forceinline__ void mma_whole(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D>
__global__ void __launch_bounds__(kMaskThreads) mask_kernel(const MaskParams p) {
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
        const int tiles = p.pitch / 8;
        for (int tile = warp; tile < tiles; tile += kMaskWarps) {
            const int c0 = 8 * tile;
            uint2 put[2] = {};
            if (c0 < widest) {
                const int col = min(c0 + r8, nk - 1);
                const uint4* src = reinterpret_cast<const uint4*>(p.codes[1] + (kbase + col) * D + j4 * (D / 4));
                uint4 kv[D / 32];
#pragma unroll
                for (int w = 0; w < D / 32; ++w) kv[w] = src[w];
                float sk[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) sk[e] = p.scales[1][kbase + min(c0 + 2 * j4 + e, nk - 1)];
                float c[4] = {};
#pragma unroll
                for (int w = 0; w < D / 32; ++w) {
                    mma_whole(c, a[2 * w], kv[w].x, kv[w].y);
                    mma_whole(c, a[2 * w + 1], kv[w].z, kv[w].w);
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
        if (n > p.topk) {
            uint32_t least = 0xffffffffu, most = 0;
            int forced = 0;
            for (int j = 4 * lane; j < n; j += 128) {
                const uint4 k4 = *reinterpret_cast<const uint4*>(mine + j);
                const uint32_t k[4] = {k4.x, k4.y, k4.z, k4.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (k[e] == kForced) {
                        ++forced;
                    } else if (k[e] != 0) {
                        least = min(least, k[e]);
                        most = max(most, k[e]);
                    }
                }
            }
            forced = __reduce_add_sync(0xffffffffu, forced);
            least = __reduce_min_sync(0xffffffffu, least);
            most = __reduce_max_sync(0xffffffffu, most);
            if (forced >= p.topk) {
                lo = kForced;
            } else {
                // count(lo) > topk > count(hi)
                lo = least;
                uint32_t hi = most + 1;
                int c_lo = n, c_hi = forced;
                for (int step = 0; c_lo != p.topk && hi - lo > 1; ++step) {
                    const uint32_t mid = between(lo, hi, step);
                    int c = 0;
                    for (int j = 4 * lane; j < n; j += 128) {
                        const uint4 k4 = *reinterpret_cast<const uint4*>(mine + j);
                        c += (k4.x >= mid) + (k4.y >= mid) + (k4.z >= mid) + (k4.w >= mid);
                    }
                    c = __reduce_add_sync(0xffffffffu, c);
                    if (c >= p.topk) {
                        lo = mid;
                        c_lo = c;
                    } else {
                        hi = mid;
                        c_hi = c;
                    }
                }
                if (c_lo != p.topk) spare = p.topk - c_hi;
            }
        }
        uint8_t* out = p.mask + (static_cast<size_t>(bh) * nq + row0 + i) * nk;
        const uint32_t below = (1u << lane) - 1u;
        int equal_before = 0;
        for (int j = 0; j < nk; j += 32) {
            const uint32_t key = j + lane < n ? mine[j + lane] : 0u;
            const uint32_t is_equal = __ballot_sync(0xffffffffu, key == lo);
            const bool on = key > lo || (key == lo && equal_before + __popc(is_equal & below) < spare);
            if (j + lane < nk) out[j + lane] = on ? 1 : 0;
            equal_before += __popc(is_equal);
        }
    }
}

// Byte offsets of the workspace: summaries of q, then of k.
struct MaskLayout {
    size_t codes[2], scales[2], total;
};

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

MaskLayout mask_layout(int B, int Hq, int Hkv, int Sq, int Sk, int d) {
    const size_t n[2] = {static_cast<size_t>(B) * Hq * ((Sq + kBlockRows - 1) / kBlockRows),
                         static_cast<size_t>(B) * Hkv * ((Sk + kBlockRows - 1) / kBlockRows)};
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

template <int D, bool BF16>
int launch_mask(const MaskParams& prm, cudaStream_t st) {
    const long long tasks = static_cast<long long>(prm.B) * (static_cast<long long>(prm.H[0]) * prm.n[0] +
                                                             static_cast<long long>(prm.H[1]) * prm.n[1]);
    summarise_kernel<D, BF16><<<static_cast<unsigned>((tasks + 7) / 8), 256, 0, st>>>(prm);
    if (cudaGetLastError() != cudaSuccess) return BSATTN_ERR_CUDA;
    static std::atomic<unsigned long long> raised{0};
    const int rc = raise_smem_limit(reinterpret_cast<const void*>(mask_kernel<D>), 220 * 1024, raised);
    if (rc) return rc;
    const int strips = (prm.n[0] + prm.rows - 1) / prm.rows;
    // launched while the summaries are still being made: it waits for them itself
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(strips) * prm.B * prm.H[0]);
    cfg.blockDim = dim3(kMaskThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(prm.rows) * prm.pitch * 4;
    cfg.stream = st;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, mask_kernel<D>, prm) == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
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
    const auto run = [&](auto dim, auto bf16) {
        constexpr int D = decltype(dim)::value;
        constexpr bool BF16 = decltype(bf16)::value;
        const int G = Hq / Hkv;
        if (G == 1) return launch_select<D, BF16, 1>(prm, B, st);
        if (G == 2) return launch_select<D, BF16, 2>(prm, B, st);
        if (G <= 4) return launch_select<D, BF16, 4>(prm, B, st);
        return launch_select<D, BF16, 8>(prm, B, st);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (d == 64) return dtype == BSATTN_BF16 ? run(D64{}, std::true_type{}) : run(D64{}, std::false_type{});
    return dtype == BSATTN_BF16 ? run(D128{}, std::true_type{}) : run(D128{}, std::false_type{});
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
    prm.pitch = (prm.n[1] + 127) & ~127;
    // 16 rows of keys, or 8 where they do not fit
    prm.rows = 16 * 4LL * prm.pitch <= 220 * 1024 ? 16 : 8;
    if (static_cast<long long>(prm.rows) * 4 * prm.pitch > 220 * 1024) return BSATTN_ERR_UNSUPPORTED;
    const long long tasks = static_cast<long long>(B) * (static_cast<long long>(Hq) * prm.n[0] + static_cast<long long>(Hkv) * prm.n[1]);
    if (tasks > 0x7fffffffLL) return BSATTN_ERR_UNSUPPORTED;
    const cudaStream_t cs = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == BSATTN_BF16;
    if (d == 64) return bf16 ? launch_mask<64, true>(prm, cs) : launch_mask<64, false>(prm, cs);
    return bf16 ? launch_mask<128, true>(prm, cs) : launch_mask<128, false>(prm, cs);
}
