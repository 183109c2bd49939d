// block_index.cu -- 8-bit summaries of the 64-token key blocks of a paged cache, sm_103a.
//
// For every sequence, each block that holds one of its last new_lens[b] tokens is summarised again from its
// rows in the cache (summary.cuh): codes [pages, page_size / 64, Hkv, d] and a scale for each block and head.
//
// Each row is read once and 1/128 of it written, so HBM bandwidth bounds this, and for the few blocks of a
// decode step a chain of latencies.  A warp takes a (block, kv head), its neighbour the next head, as rows of
// neighbouring heads lie next to each other.  The lanes look up where 32 of a warp's blocks lie at once, and the
// warp has the rows of two (d = 64: four) on their way while it adds up another's.  16 prompts of 512 to 8191 tokens, 8
// heads, d = 128: 144 MB in 29 us (31.4 with sixteen 16-byte loads a lane in registers instead), 5 of them until
// the first rows are on their way; a step of 64 sequences: 4.5 us (5.0 with
// its 512 blocks on half of the SMs).
#include <algorithm>
#include <climits>

#include "host_internal.h"
#include "summary.cuh"

namespace bsattn {
namespace {

constexpr int kWarps = 7;                       // 32 KB of shared memory each
constexpr int kThreads = 32 * kWarps;
constexpr int kStretches = 256;                 // of sequences, a thread each; the last ones are empty
static_assert(kThreads <= kStretches, "a thread a stretch");

struct UpdateParams {
    const void* k;
    const int32_t* seqlens;
    const int32_t* new_lens;
    const int32_t* table;
    int8_t* codes;
    float* scales;
    int* status;
    int B, Hkv, page_size, max_pages, num_pages;
};

// The blocks of a sequence that are to be summarised: n from block `first` on; lengths out of range are
// cut to what there can be, and reported.
struct Touched {
    int len, first, n;
    bool bad;
};

__device__ __forceinline__ Touched touched(const UpdateParams& p, int b) {
    Touched t;
    int len = p.seqlens[b], fresh = p.new_lens[b];
    const long long room = static_cast<long long>(p.max_pages) * p.page_size;
    t.bad = len < 0 || fresh < 0 || fresh > len || len > room;
    len = max(len, 0);
    fresh = max(min(fresh, len), 0);
    t.first = (len - fresh) / kBlockRows;
    len = static_cast<int>(min(static_cast<long long>(len), room));
    t.len = len;
    t.n = fresh > 0 ? max(len / kBlockRows + (len % kBlockRows != 0) - t.first, 0) : 0;
    return t;
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads, 1) update_kernel(const UpdateParams p) {
    using Ring = BlockRing<D>;
    extern __shared__ __align__(128) uint8_t ring_smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // thread t has the blocks of its stretch of sequences; upto[t]: of all stretches to its end
    __shared__ long long upto[kStretches];
    __shared__ long long warp_sums[kWarps];
    const int per = (p.B + kThreads - 1) / kThreads;
    long long sum = 0;
    for (int k = 0; k < per; ++k) {
        const int b = tid * per + k;
        if (b >= p.B) break;
        const Touched t = touched(p, b);
        sum += t.n;
        if (t.bad && blockIdx.x == 0) atomicOr(p.status, BSATTN_ERR_BAD_INDEX);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += u;
    }
    if (lane == 31) warp_sums[warp] = sum;
    __syncthreads();
    for (int w = 0; w < warp; ++w) sum += warp_sums[w];
    upto[tid] = sum;
    if (tid + kThreads < kStretches) upto[tid + kThreads] = LLONG_MAX;
    __syncthreads();
    const long long tasks = upto[kThreads - 1] * p.Hkv;
    const int blocks_a_page = p.page_size / kBlockRows;
    const long long stride = static_cast<long long>(gridDim.x) * kWarps;
    const long long step = static_cast<long long>(p.Hkv) * D * 2;
    const Ring ring(ring_smem + warp * Ring::kBytes);
    bool bad = false;
    // (few tasks: one a CTA first)
    for (long long base = blockIdx.x + static_cast<long long>(gridDim.x) * warp; base < tasks; base += 32 * stride) {
        // ---------------------------------------------------------------- lane l: where the warp's l-th block lies
        const long long task = base + lane * stride;
        int of_block = -1, count = 0;                       // its place in the index over Hkv, and its rows
        int g = 0;
        if (task < tasks) {
            long long nth;
            if (tasks <= 0xffffffffLL) {
                const uint32_t q = static_cast<uint32_t>(task) / static_cast<uint32_t>(p.Hkv);
                nth = q;
                g = static_cast<int>(static_cast<uint32_t>(task) - q * static_cast<uint32_t>(p.Hkv));
            } else {
                nth = task / p.Hkv;
                g = static_cast<int>(task - nth * p.Hkv);
            }
            // the first stretch that ends past it
            int at = 0;
#pragma unroll
            for (int half = kStretches / 2; half > 0; half >>= 1)
                if (upto[at + half - 1] <= nth) at += half;
            long long before = at > 0 ? upto[at - 1] : 0;
            int b = at * per;
            Touched t = touched(p, b);
            while (nth >= before + t.n) {
                before += t.n;
                t = touched(p, ++b);
            }
            const int block = t.first + static_cast<int>(nth - before);
            const int lp = block / blocks_a_page, sub = block - lp * blocks_a_page;
            const int page = p.table[static_cast<size_t>(b) * p.max_pages + lp];
            if (page < 0 || page >= p.num_pages) {
                bad = true;
            } else {
                of_block = page * blocks_a_page + sub;
                count = min(t.len - block * kBlockRows, kBlockRows);
            }
        }
        const int n = static_cast<int>(min((tasks - base + stride - 1) / stride, 32LL));
        // ---------------------------------------------------------------- the blocks one after another
        const auto fetch = [&](int m) {
            const int at = __shfl_sync(0xffffffffu, of_block, m & 31), head = __shfl_sync(0xffffffffu, g, m & 31);
            const int rows = __shfl_sync(0xffffffffu, count, m & 31);
            if (m < n && at >= 0)
                ring.fetch(m % Ring::kDepth, static_cast<const char*>(p.k) +
                           (static_cast<size_t>(at) * kBlockRows * p.Hkv + head) * (D * 2) + 16 * (lane % (D / 8)), step, rows);
            Ring::commit();
        };
#pragma unroll
        for (int m = 0; m < Ring::kDepth; ++m) fetch(m);
        for (int m = 0; m < n; ++m) {
            const int at = __shfl_sync(0xffffffffu, of_block, m), head = __shfl_sync(0xffffffffu, g, m);
            const int rows = __shfl_sync(0xffffffffu, count, m);
            Ring::wait();
            if (at >= 0) {
                float s[8];
                ring.template sum<BF16>(m % Ring::kDepth, s);
                int code[8];
                const float scale = summarise<D>(s, rows, code);
                const size_t to = static_cast<size_t>(at) * p.Hkv + head;
                if (lane < D / 8) {
                    uint32_t w[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        w[h] = (code[4 * h] & 255) | (code[4 * h + 1] & 255) << 8 | (code[4 * h + 2] & 255) << 16 |
                               static_cast<uint32_t>(code[4 * h + 3]) << 24;
                    *reinterpret_cast<uint2*>(p.codes + to * D + 8 * lane) = make_uint2(w[0], w[1]);
                    if (lane == 0) p.scales[to] = scale;
                }
            }
            fetch(m + Ring::kDepth);
        }
    }
    if (bad) atomicOr(p.status, BSATTN_ERR_BAD_INDEX);
}

template <int D, bool BF16>
int launch(const UpdateParams& prm, int sms, cudaStream_t st) {
    auto kern = update_kernel<D, BF16>;
    constexpr int kSmem = kWarps * BlockRing<D>::kBytes;
    static std::atomic<unsigned long long> raised{0};
    const int rc = raise_smem_limit(reinterpret_cast<const void*>(kern), kSmem, raised);
    if (rc) return rc;
    // a warp a task, and no more CTAs than the GPU holds at once
    const long long most = static_cast<long long>(prm.B) * prm.max_pages * (prm.page_size / kBlockRows) * prm.Hkv;
    const long long grid = std::min<long long>((most + kWarps - 1) / kWarps, sms);
    kern<<<static_cast<unsigned>(grid), kThreads, kSmem, st>>>(prm);
    return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

}  // namespace
}  // namespace bsattn

extern "C" int bsattn_index_update(const void* k_pages, const int32_t* cache_seqlens, const int32_t* new_lens,
                                   const int32_t* block_table, int8_t* codes, float* scales, int B, int Hkv,
                                   int num_pages, int page_size, int max_pages_per_seq, int d, bsattn_dtype dtype,
                                   void* workspace, size_t workspace_bytes, void* stream) {
    using namespace bsattn;
    if (B < 0 || Hkv <= 0 || num_pages <= 0 || page_size <= 0 || max_pages_per_seq <= 0) return BSATTN_ERR_INVALID_ARG;
    if (page_size % kBlockRows || (d != 64 && d != 128)) return BSATTN_ERR_UNSUPPORTED;
    if (dtype != BSATTN_F16 && dtype != BSATTN_BF16) return BSATTN_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < 256 || !aligned16(workspace)) return BSATTN_ERR_INVALID_ARG;
    if (B == 0) return BSATTN_OK;
    if (!k_pages || !cache_seqlens || !new_lens || !block_table || !codes || !scales) return BSATTN_ERR_INVALID_ARG;
    if (!aligned16(k_pages) || !aligned16(codes) || !aligned16(scales)) return BSATTN_ERR_INVALID_ARG;
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL) return BSATTN_ERR_UNSUPPORTED;
    const size_t rows = static_cast<size_t>(num_pages) * page_size, blocks = rows / kBlockRows * Hkv;
    const size_t lens = sizeof(int32_t) * B, entries = lens * max_pages_per_seq;
    const void* in[4] = {k_pages, cache_seqlens, new_lens, block_table};
    const size_t in_bytes[4] = {rows * Hkv * d * 2, lens, lens, entries};
    for (int i = 0; i < 4; ++i)
        if (overlap(codes, blocks * d, in[i], in_bytes[i]) || overlap(scales, blocks * 4, in[i], in_bytes[i]))
            return BSATTN_ERR_INVALID_ARG;
    if (overlap(codes, blocks * d, scales, blocks * 4)) return BSATTN_ERR_INVALID_ARG;
    UpdateParams prm{};
    prm.k = k_pages;
    prm.seqlens = cache_seqlens;
    prm.new_lens = new_lens;
    prm.table = block_table;
    prm.codes = codes;
    prm.scales = scales;
    prm.status = status_word(workspace);
    prm.B = B;
    prm.Hkv = Hkv;
    prm.page_size = page_size;
    prm.max_pages = max_pages_per_seq;
    prm.num_pages = num_pages;
    int sms = num_sms_of_current_device();
    if (sms <= 0) sms = 148;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == BSATTN_BF16;
    if (d == 64) return bf16 ? launch<64, true>(prm, sms, st) : launch<64, false>(prm, sms, st);
    return bf16 ? launch<128, true>(prm, sms, st) : launch<128, false>(prm, sms, st);
}
