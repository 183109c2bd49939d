// block_index.cu -- 8-bit summaries of the 64-token key blocks of a paged cache, sm_103a.
//
// For every sequence, each block that holds one of its last new_lens[b] tokens is summarised again from its
// rows in the cache (summary.cuh): codes [pages, page_size / 64, Hkv, d] and a scale for each block and head.
//
// Each row is read once and 1/128 of it written, so HBM bandwidth bounds this, and for the few blocks of a
// decode step a chain of latencies.  A warp takes a (block, kv head), a warp's next to its neighbour's head,
// as rows of neighbouring heads lie next to each other: sixteen 16-byte loads a lane in flight.
#include <algorithm>

#include "host_internal.h"
#include "summary.cuh"

namespace bsattn {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

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
__global__ void __launch_bounds__(kThreads) update_kernel(const UpdateParams p) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // thread t has the blocks of its stretch of sequences; upto[t]: of all stretches to its end
    __shared__ long long upto[kThreads];
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
    __syncthreads();
    const long long tasks = upto[kThreads - 1] * p.Hkv;
    const int blocks_a_page = p.page_size / kBlockRows;
    bool bad = false;
    for (long long task = static_cast<long long>(blockIdx.x) * kWarps + warp; task < tasks;
         task += static_cast<long long>(gridDim.x) * kWarps) {
        long long nth;
        int g;
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
        for (int step = kThreads / 2; step > 0; step >>= 1)
            if (upto[at + step - 1] <= nth) at += step;
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
            continue;
        }
        const int count = min(t.len - block * kBlockRows, kBlockRows);
        const size_t row0 = static_cast<size_t>(page) * p.page_size + sub * kBlockRows;
        const uint16_t* src = static_cast<const uint16_t*>(p.k) + (row0 * p.Hkv + g) * D + 8 * (lane % (D / 8));
        float s[8];
        block_sum<D, BF16>([&](int r) { return reinterpret_cast<const uint4*>(src + static_cast<size_t>(r) * p.Hkv * D); },
                           count, s);
        int code[8];
        const float scale = summarise<D>(s, count, code);
        const size_t to = (static_cast<size_t>(page) * blocks_a_page + sub) * p.Hkv + g;
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
    if (bad && lane == 0) atomicOr(p.status, BSATTN_ERR_BAD_INDEX);
}

template <int D, bool BF16>
int launch(const UpdateParams& prm, int sms, cudaStream_t st) {
    // a warp a task, and no more CTAs than the GPU holds at once (three an SM)
    const long long most = static_cast<long long>(prm.B) * prm.max_pages * (prm.page_size / kBlockRows) * prm.Hkv;
    const long long grid = std::min<long long>((most + kWarps - 1) / kWarps, 3LL * sms);
    update_kernel<D, BF16><<<static_cast<unsigned>(grid), kThreads, 0, st>>>(prm);
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
