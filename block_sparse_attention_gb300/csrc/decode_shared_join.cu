// decode_shared_join.cu -- a decode over shared prefixes: the joining of all pieces, sm_103a.
//
// A warp a row: with (O, L) of each piece, out = sum O 2^(L - M) / sum 2^(L - M), in a fixed order.  What there is to
// read is in L2, so a chain of latencies bounds this: the L of 32 pieces come at once, and the O of eight with them.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "decode_shared.cuh"
#include "host_internal.h"
#include "mma16.cuh"
#include "ptx.cuh"

namespace bsattn {
namespace {

using namespace mma16;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kBatch = 8;                // pieces that a warp joins in one trip to L2

// WARPS: of a row, each with every WARPS-th piece: four where the rows are few, as a trip more costs more than joining
// their four results.
template <int D, bool BF16, int WARPS>
__global__ void __launch_bounds__(kThreads) join_kernel(const SharedCall p) {
    constexpr int kC = D / 32;                           // channels of a lane
    using V = std::conditional_t<kC == 4, float4, float2>;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int row = static_cast<int>(blockIdx.x) * (kWarps / WARPS) + warp / WARPS, share = warp % WARPS;
    const int b = row / p.Hq, h = row - b * p.Hq;
    if (b >= p.B) return;                                // (with four warps a row, none or all)
    const int G = p.Hq / p.Hkv, kvh = h / G;
    // the prefix whose sequences begin last before or at b
    int prefix = 0;
    for (int i = 1; i <= p.P; i += 32)
        prefix += __reduce_add_sync(0xffffffffu, i + lane <= p.P && p.starts[i + lane] <= b ? 1 : 0);
    PrefixGroup group{};
    int i = -1;
    if (prefix < p.P) {
        group = prefix_group(p, prefix);
        i = b - group.start;
    }
    const int mine = own_units(own_len(p, b));
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // pieces 0 .. shared - 1 are the prefix's, those up to `count` of the sequence's own tokens
    int shared = 0, count = 0, other = 0;
    long long first = 0, by = 0, own = 0;
    if (i >= 0 && i < group.n && group.tiles > 0) {
        const long long chunk = p.prefix_info[0], units = p.prefix_info[1 + prefix];
        const int t = i / p.seqs, each = p.halves ? 2 : 1;
        const long long from = units + (static_cast<long long>(t / p.deep) * (p.Hkv / p.side) + kvh / p.side) * group.tiles;
        const long long c0 = from / chunk;
        shared = static_cast<int>((from + group.tiles - 1) / chunk - c0 + 1) * each;
        by = static_cast<long long>(p.part_rows) * each;
        first = prefix_place(p, group, static_cast<int>(c0), t, kvh, other) + (i - t * p.seqs) * G + (h - kvh * G);
    }
    count = shared;
    if (mine > 0) {
        const long long chunk = p.own_info[0], from = p.own_info[1 + b], c0 = from / chunk;
        count += static_cast<int>((from + mine - 1) / chunk - c0 + 1);
        own = ((c0 + b) * p.Hkv + kvh) * G + (h - kvh * G);
    }
    float num[kC] = {};
    float M = -INFINITY, den = 0.f;
    const auto place = [&](int n) -> long long {
        return n >= shared ? own + static_cast<long long>(n - shared) * p.Hq
               : p.halves  ? first + (n >> 1) * by + (n & 1) * other
                           : first + n * by;
    };
    // 32 pieces at a time: their L, one a lane, and with them the O of the first eight
    for (int k0 = share; k0 < count; k0 += 32 * WARPS) {
        const int here = min((count - k0 + WARPS - 1) / WARPS, 32);
        V ov[kBatch];
        const auto fetch = [&](int k1) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                ov[k] = V{};
                if (k1 + k < here) {
                    const int at = k0 + (k1 + k) * WARPS;
                    ov[k] = __ldcg(reinterpret_cast<const V*>((at < shared ? p.prefix_o : p.own_o) + place(at) * D) + lane);
                }
            }
        };
        const int n = k0 + lane * WARPS;
        const float mine_l = n < count ? __ldcg((n < shared ? p.prefix_lse : p.own_lse) + place(n)) : -INFINITY;
        fetch(0);
        float top = mine_l;
#pragma unroll
        for (int w = 1; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
        top = fmaxf(top, M);
        const float ref = top == -INFINITY ? 0.f : top, down = ex2_approx(M - ref);
        M = top;
        den *= down;
#pragma unroll
        for (int e = 0; e < kC; ++e) num[e] *= down;
        const float weight = mine_l == -INFINITY ? 0.f : ex2_approx(mine_l - ref);
        den += weight;                                   // of this lane's pieces
        for (int k1 = 0;;) {
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const float w = __shfl_sync(0xffffffffu, weight, (k1 + k) & 31);
                // (where a row has met no finite score O may not have been written)
                if (k1 + k >= here || w == 0.f) continue;
                const float* v = reinterpret_cast<const float*>(&ov[k]);
#pragma unroll
                for (int e = 0; e < kC; ++e) num[e] = fmaf(w, v[e], num[e]);
            }
            k1 += kBatch;
            if (k1 >= here) break;
            fetch(k1);
        }
    }
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) den += __shfl_xor_sync(0xffffffffu, den, w);
    if constexpr (WARPS > 1) {
        __shared__ float top_of[WARPS], den_of[WARPS];
        __shared__ V num_of[WARPS][32];
        V* to = &num_of[share][lane];
#pragma unroll
        for (int e = 0; e < kC; ++e) reinterpret_cast<float*>(to)[e] = num[e];
        if (lane == 0) {
            top_of[share] = M;
            den_of[share] = den;
        }
        __syncthreads();
        if (share > 0) return;
        float top = -INFINITY;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) top = fmaxf(top, top_of[w]);
        const float ref = top == -INFINITY ? 0.f : top;
        den = 0.f;
#pragma unroll
        for (int e = 0; e < kC; ++e) num[e] = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            // a warp without a finite L has a sum of 0, or NaN if it met one: either way it counts
            const float by = top_of[w] == -INFINITY ? 1.f : ex2_approx(top_of[w] - ref);
            const V v = num_of[w][lane];
#pragma unroll
            for (int e = 0; e < kC; ++e) num[e] = fmaf(by, reinterpret_cast<const float*>(&v)[e], num[e]);
            den = fmaf(by, den_of[w], den);
        }
    }
    const float inv = den == 0.f ? 0.f : 1.f / den;
    uint32_t w[kC / 2];
#pragma unroll
    for (int e = 0; e < kC / 2; ++e) w[e] = pack2<BF16>(num[2 * e] * inv, num[2 * e + 1] * inv);
    uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(p.out) + static_cast<size_t>(row) * D + kC * lane);
    if constexpr (kC == 4) *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
    else out[0] = w[0];
}

// Launches a kernel that may start while the one before it on the stream still runs, and waits for that one by itself.
template <typename Kernel>
int launch_early(Kernel kern, unsigned grid, cudaStream_t stream, const SharedCall& call) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kern, call) == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

}  // namespace

int launch_join(const SharedCall& p, int d, bool bf16, cudaStream_t st) {
    const long long rows = static_cast<long long>(p.B) * p.Hq;
    // (the whole call with four warps a row and with one: 128 rows 18.1 and 20.1 us, 2048 rows 71.4 and 67.6)
    const bool few = rows <= 1024;
    const unsigned grid = static_cast<unsigned>(few ? rows : (rows + kWarps - 1) / kWarps);
    const auto run = [&](auto dim, auto type) {
        constexpr int D = decltype(dim)::value;
        constexpr bool BF16 = decltype(type)::value;
        return few ? launch_early(join_kernel<D, BF16, kWarps>, grid, st, p)
                   : launch_early(join_kernel<D, BF16, 1>, grid, st, p);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (d == 64) return bf16 ? run(D64{}, std::true_type{}) : run(D64{}, std::false_type{});
    return bf16 ? run(D128{}, std::true_type{}) : run(D128{}, std::false_type{});
}

}  // namespace bsattn
