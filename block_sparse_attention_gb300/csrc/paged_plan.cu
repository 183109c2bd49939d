// paged_plan.cu -- block tables and slot maps for a paged cache, built on the GPU from request
// lengths, sm_103a.
//
// Per call every sequence b brings new_lens[b] tokens to the cached_lens[b] it holds.  With
//     end_b  = new_0 + ... + new_b                        (place of its tokens in the packed batch)
//     held_b = ceil(cached_b / page), need_b = ceil((cached_b + new_b) / page)
//     a_b    = need_b - held_b, A_b = a_0 + ... + a_b     (0 for a sequence that cannot fit)
// sequence b takes the pages free[count - 1 - (A_b - a_b) - k], k < a_b, off the top of the free
// list, and token t of it goes to slot table[pos / page] * page + pos % page, pos = cached_b + i.
//
// The work is a few bytes a sequence and 8 bytes a token, so a small call is bound by its launch
// and by the two dependent prefix sums.  Every CTA therefore scans all sequences itself (they are
// L2-resident and few) and keeps the results in shared memory: one launch, no workspace that two
// calls could disturb, no CTA that waits on another.  Tokens are dealt out over the CTAs and find
// their sequence by bisection in shared memory; a new page's number is read from the free list, not
// from the table, so that nothing is read that another CTA writes.  A step of 8 sequences takes 4.6 us,
// a tick of 2000 with 493k slots (4 MB written) 9.9 us: the launch, one trip to L2 and the scans.
#include <climits>

#include "host_internal.h"
#include "ptx.cuh"

namespace bsattn {
namespace {

constexpr int kThreads = 512;
constexpr int kPerThread = 16;
constexpr int kMaxSeqs = kThreads * kPerThread;
// Tokens in a row a thread writes the slots of: four where there are enough to keep the threads busy (a
// tick of 2000 sequences, 493k slots: 9.6 us against 11.0 with one), one for a step of a few tokens (eight
// of them: 4.6 us against 6.0 with four, whose look-ups follow one another).
constexpr int kLongRun = 4;
constexpr int kLongFrom = 16 * kThreads;

struct PlanParams {
    const int32_t* cached;
    const int32_t* fresh;
    const int32_t* free_pages;
    const int32_t* free_count;
    int32_t* table;
    int64_t* slots;
    int32_t* starts;
    int32_t* lens;
    int32_t* free_left;
    int* status;
    int B, page, max_pages, free_cap, max_tokens;
};

// Sums above INT_MAX stay there: the operands are not negative, so the sum is still associative.
__device__ __forceinline__ int sat_add(int a, int b) {
    const unsigned s = static_cast<unsigned>(a) + static_cast<unsigned>(b);
    return s > 0x7fffffffu ? 0x7fffffff : static_cast<int>(s);
}

// Inclusive prefix sum over the CTA's threads.
__device__ __forceinline__ int block_scan(int v, int* warp_sums) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v = sat_add(v, u);
    }
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    int before = 0;
    if (warp > 0) {
        int s = lane < warp ? warp_sums[lane] : 0;      // at most 16 warps
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s = sat_add(s, __shfl_xor_sync(0xffffffffu, s, o));
        before = s;
    }
    __syncthreads();
    return sat_add(before, v);
}

template <int kRun>
__global__ void __launch_bounds__(kThreads) plan_kernel(const PlanParams p) {
    extern __shared__ int sm[];
    __shared__ int warp_sums[kThreads / 32];
    __shared__ int used_max;
    int* end_of = sm;                    // [B] end of the sequence's tokens in the packed batch
    int* first_of = sm + p.B;            // [B] its first place in the free list's order, -1 = not served
    const int tid = threadIdx.x;
    const int per = (p.B + kThreads - 1) / kThreads;      // <= kPerThread
    const int b0 = tid * per;
    int room = *p.free_count;
    int flags = 0;
    if (room < 0 || room > p.free_cap) {
        flags |= BSATTN_ERR_BAD_INDEX;
        room = room < 0 ? 0 : p.free_cap;
    }
    if (tid == 0) used_max = 0;

    int have[kPerThread], more[kPerThread];
    int sum = 0;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int b = b0 + k;
        have[k] = more[k] = 0;
        if (k < per && b < p.B) {
            have[k] = p.cached[b];
            more[k] = p.fresh[b];
            sum = sat_add(sum, max(more[k], 0));
        }
    }
    int end = block_scan(sum, warp_sums);
    if (blockIdx.x == 0 && tid == kThreads - 1) {
        p.starts[0] = 0;
    }
    // tokens: walk the thread's sequences forward from the tokens before them
    int before = 0;
    {
        __shared__ int excl[kThreads];
        excl[tid] = end;
        __syncthreads();
        before = tid > 0 ? excl[tid - 1] : 0;
        __syncthreads();
    }
    int asked[kPerThread];
    int pages = 0, at = before;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int b = b0 + k;
        asked[k] = -1;                                    // -1: cannot be served
        if (k < per && b < p.B) {
            const bool sane = have[k] >= 0 && more[k] >= 0;
            at = sat_add(at, max(more[k], 0));
            end_of[b] = at;
            if (!sane) {
                flags |= BSATTN_ERR_BAD_INDEX;
            } else {
                const long long total = static_cast<long long>(have[k]) + more[k];
                const long long need = (total + p.page - 1) / p.page;
                const int held = have[k] / p.page + (have[k] % p.page != 0);
                if (need <= p.max_pages && at <= p.max_tokens && at < INT_MAX && total <= INT_MAX) {
                    asked[k] = static_cast<int>(need) - held;
                    pages = sat_add(pages, asked[k]);
                } else {
                    flags |= BSATTN_ERR_NO_SPACE;
                }
            }
        }
    }
    const int upto = block_scan(pages, warp_sums);
    int first = 0;
    {
        __shared__ int excl[kThreads];
        excl[tid] = upto;
        __syncthreads();
        first = tid > 0 ? excl[tid - 1] : 0;
    }
    int used = 0;
#pragma unroll
    for (int k = 0; k < kPerThread; ++k) {
        const int b = b0 + k;
        if (k < per && b < p.B) {
            const int a = asked[k];
            const int last = sat_add(first, max(a, 0));
            const bool served = a >= 0 && (a == 0 || last <= room);
            if (a >= 0 && !served) flags |= BSATTN_ERR_NO_SPACE;
            first_of[b] = served ? first : -1;
            if (served && a > 0) used = last;
            first = last;
            if (blockIdx.x == 0) {
                p.starts[b + 1] = end_of[b];
                p.lens[b] = served ? have[k] + more[k] : have[k];
            }
        }
    }
    if (blockIdx.x == 0) {
        if (flags) atomicOr(p.status, flags);
        if (used) atomicMax(&used_max, used);
    }
    __syncthreads();
    if (blockIdx.x == 0 && tid == 0) *p.free_left = room - used_max;

    // new table entries: a warp a sequence, the sequences dealt out over the grid
    const int lane = tid & 31;
    for (int b = blockIdx.x * (kThreads / 32) + (tid >> 5); b < p.B; b += gridDim.x * (kThreads / 32)) {
        const int f = first_of[b];
        if (f < 0) continue;
        const int have_b = p.cached[b], more_b = p.fresh[b];
        const int held = have_b / p.page + (have_b % p.page != 0);
        const int need = static_cast<int>((static_cast<long long>(have_b) + more_b + p.page - 1) / p.page);
        int32_t* row = p.table + static_cast<size_t>(b) * p.max_pages;
        for (int c = held + lane; c < need; c += 32) row[c] = p.free_pages[room - 1 - (f + c - held)];
    }

    // slots: a thread takes kRun tokens in a row, finds the sequence of the first by bisection and walks
    // on from there: most runs stay in one sequence and one page, whose number is looked up once
    bool unmapped = false;
    const long long stride = static_cast<long long>(gridDim.x) * kThreads * kRun;
    for (long long t0 = (static_cast<long long>(blockIdx.x) * kThreads + tid) * kRun; t0 < p.max_tokens; t0 += stride) {
        int lo = 0, hi = p.B;                     // first sequence that ends after t0
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (end_of[mid] > t0) hi = mid;
            else lo = mid + 1;
        }
        int64_t slot[kRun];
        int have_b = 0, begin = 0, held = 0, first_b = -1, chunk = -1, page = -1;
        bool fresh_seq = true;
#pragma unroll
        for (int k = 0; k < kRun; ++k) {
            const int t = static_cast<int>(min(t0 + k, static_cast<long long>(INT_MAX)));
            while (lo < p.B && end_of[lo] <= t) {
                ++lo;
                fresh_seq = true;
            }
            slot[k] = -1;
            if (lo >= p.B) continue;
            if (fresh_seq) {
                fresh_seq = false;
                have_b = p.cached[lo];
                begin = lo > 0 ? end_of[lo - 1] : 0;
                held = have_b / p.page + (have_b % p.page != 0);
                first_b = first_of[lo];
                chunk = -1;
            }
            if (first_b < 0) continue;
            const int pos = have_b + (t - begin);
            const int c = pos / p.page;
            if (c != chunk) {
                chunk = c;
                page = c < held ? p.table[static_cast<size_t>(lo) * p.max_pages + c]
                                : p.free_pages[room - 1 - (first_b + c - held)];
            }
            if (page >= 0) slot[k] = static_cast<int64_t>(page) * p.page + (pos - c * p.page);
            else if (t0 + k < p.max_tokens) unmapped = true;
        }
        if (kRun > 1 && t0 + kRun <= p.max_tokens && (reinterpret_cast<uintptr_t>(p.slots) & 15) == 0) {
#pragma unroll
            for (int k = 0; k + 1 < kRun; k += 2)
                *reinterpret_cast<longlong2*>(p.slots + t0 + k) = make_longlong2(slot[k], slot[k + 1]);
        } else {
#pragma unroll
            for (int k = 0; k < kRun; ++k)
                if (t0 + k < p.max_tokens) p.slots[t0 + k] = slot[k];
        }
    }
    if (unmapped) atomicOr(p.status, BSATTN_ERR_BAD_INDEX);
}

}  // namespace
}  // namespace bsattn

extern "C" int bsattn_paged_plan(const int32_t* cached_lens, const int32_t* new_lens,
                                 const int32_t* free_pages, const int32_t* free_count,
                                 int32_t* block_table, int64_t* slots, int32_t* starts,
                                 int32_t* seqlens, int32_t* free_left, int B, int page_size,
                                 int max_pages_per_seq, int free_capacity, int max_tokens,
                                 void* workspace, size_t workspace_bytes, void* stream) {
    using namespace bsattn;
    if (B < 0 || page_size <= 0 || max_pages_per_seq <= 0 || free_capacity < 0 || max_tokens < 0)
        return BSATTN_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < 256 || !aligned16(workspace) || !starts || !free_left || !free_count)
        return BSATTN_ERR_INVALID_ARG;
    if ((B > 0 && (!cached_lens || !new_lens || !block_table || !seqlens)) ||
        (max_tokens > 0 && !slots) || (free_capacity > 0 && !free_pages))
        return BSATTN_ERR_INVALID_ARG;
    if (B > kMaxSeqs) return BSATTN_ERR_UNSUPPORTED;
    // every CTA reads the inputs while CTA 0 writes the new lengths: no output may be an input
    const size_t nb = sizeof(int32_t) * static_cast<size_t>(B);
    const void* in[4] = {cached_lens, new_lens, free_pages, free_count};
    const size_t in_bytes[4] = {nb, nb, sizeof(int32_t) * static_cast<size_t>(free_capacity), sizeof(int32_t)};
    const void* out[5] = {block_table, slots, starts, seqlens, free_left};
    const size_t out_bytes[5] = {nb * max_pages_per_seq, sizeof(int64_t) * static_cast<size_t>(max_tokens),
                                 nb + sizeof(int32_t), nb, sizeof(int32_t)};
    for (int i = 0; i < 5; ++i) {
        for (int j = 0; j < 4; ++j)
            if (overlap(out[i], out_bytes[i], in[j], in_bytes[j]))
                return BSATTN_ERR_INVALID_ARG;
        for (int j = i + 1; j < 5; ++j)
            if (overlap(out[i], out_bytes[i], out[j], out_bytes[j]))
                return BSATTN_ERR_INVALID_ARG;
    }
    PlanParams p{cached_lens, new_lens, free_pages, free_count, block_table, slots, starts, seqlens,
                 free_left, status_word(workspace), B, page_size, max_pages_per_seq, free_capacity,
                 max_tokens};
    int sms = num_sms_of_current_device();
    if (sms <= 0) sms = 148;
    const bool long_runs = max_tokens >= kLongFrom;
    const long long per_cta = static_cast<long long>(kThreads) * (long_runs ? kLongRun : 1);
    long long grid = (max_tokens + per_cta - 1) / per_cta;
    grid = grid < 1 ? 1 : (grid > sms ? sms : grid);
    auto kern = long_runs ? plan_kernel<kLongRun> : plan_kernel<1>;
    const size_t smem = 2 * nb;
    if (smem > 32 * 1024 &&
        cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 64 * 1024) != cudaSuccess)
        return BSATTN_ERR_CUDA;
    kern<<<static_cast<unsigned>(grid), kThreads, smem, static_cast<cudaStream_t>(stream)>>>(p);
    return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}
