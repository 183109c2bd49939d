// kv4.cu -- writing K and V rows into the paged 4-bit cache and reading rows back, sm_103a.
//
// Append: token t of the packed batch goes to slot slots[t]: page slot / page_size, row slot %
// page_size of codes [pages, Hkv, page_size, d / 2] and scales [pages, Hkv, page_size, d / 16].  A
// group of 16 channels x becomes
//     s = e4m3(amax / 6),  code = e2m1(x / s)          (x in units of the cache's power of two)
// both rounded to nearest, ties to even.  The codes are those of exact arithmetic: amax / 6 and
// x / s can only lie on a rounding border when they are representable, since x has at most 11
// significant bits and a border times s at most 7; so the nearest 32-bit quotient decides amax / 6
// rightly, and x / s is taken as x * (1 / s) rounded to a multiple of 2^-16 (adding and taking off
// 192): that is on the border exactly when x / s is, as other quotients are 2^-13 or more away.
//
// Gather is the way back: code * s * u rounded to the output type.
//
// Both move each byte once and are bound by memory: 2 bytes a channel one way, 0.5625 the other.  65521
// rows of 8 heads, d = 128, keys and values (344 MB each way): append 58 us and gather 57 us, 5.9 and 6.1
// TB/s; 61 rows: both in 4.8 us.
// A warp takes a token, so that the slot's division is made once a token.  On the way in a lane takes
// a group, two of keys and two of values at a time (128 bytes a lane in flight); on the way out half a
// group, so that a warp's 16-byte stores are contiguous, four of each.  Writing whole groups out, two
// stores 32 bytes apart a lane, took 73 us for 65521 rows of 8 heads, d = 128, against 57; reading half
// groups in works out each scale twice and took 76 us against 60.
#include "host_internal.h"
#include "kv4.cuh"
#include "ptx.cuh"

namespace bsattn {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct Kv4Params {
    const void* k;            // append: new keys; gather: output keys
    const void* v;
    long long k_token, k_head, v_token, v_head;    // strides in elements
    const int64_t* slots;
    uint8_t* kc;
    uint8_t* ks;
    uint8_t* vc;
    uint8_t* vs;
    float k_unit, v_unit;
    int T, Hkv, page;
    long long num_slots;
    int* status;
};

// The page row a token's slot names; false for padding (negative) and for a slot outside the cache,
// which is recorded.
__device__ __forceinline__ bool locate(const Kv4Params& p, int64_t slot, long long& page, int& row) {
    if (slot < 0) return false;
    if (slot >= p.num_slots) {
        if ((threadIdx.x & 31) == 0) atomicOr(p.status, BSATTN_ERR_BAD_INDEX);
        return false;
    }
    if (p.num_slots <= 0xffffffffLL) {
        const uint32_t s = static_cast<uint32_t>(slot), pg = s / static_cast<uint32_t>(p.page);
        page = pg;
        row = static_cast<int>(s - pg * static_cast<uint32_t>(p.page));
    } else {
        page = slot / p.page;
        row = static_cast<int>(slot - page * p.page);
    }
    return true;
}

template <bool BF16>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if constexpr (BF16) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    } else {
        return __half22float2(*reinterpret_cast<__half2*>(&w));
    }
}

// 16 values (eight words of two) to eight bytes of codes and a scale.
template <bool BF16>
__device__ __forceinline__ uint2 quantise(const uint32_t (&w)[8], float per_unit, uint32_t& scale) {
    // the largest magnitude: 16-bit floats without their sign bit order as whole numbers
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __vmaxu2(top, w[i] & 0x7fff7fffu);
    top = max(top & 0xffffu, top >> 16);
    const bool finite = top < (BF16 ? 0x7f80u : 0x7c00u);
    const float amax = unpack2<BF16>(top).x * per_unit;
    scale = f32_to_e4m3(__fdiv_rn(amax, 6.f));
    const uint32_t sh = e4m3x2_to_f16(scale);
    const float s = __half22float2(*reinterpret_cast<const __half2*>(&sh)).x;
    const float by = s > 0.f ? __fdiv_rn(1.f, s) * per_unit : 0.f;
    uint32_t out[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        float q[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 x = unpack2<BF16>(w[4 * h + i]);
            q[2 * i] = __fadd_rn(__fmaf_rn(x.x, by, 192.f), -192.f);
            q[2 * i + 1] = __fadd_rn(__fmaf_rn(x.y, by, 192.f), -192.f);
        }
        // a negative value that rounds to 0 gets code 0, not 8: clear the sign of zero codes
        const uint32_t c = f32x8_to_e2m1(q);
        const uint32_t nonzero = (c | c >> 1 | c >> 2) & 0x11111111u;
        out[h] = c & (0x77777777u | nonzero << 3);
    }
    if (!finite) {
        scale = kNanScale4;
        out[0] = out[1] = 0;
    }
    return make_uint2(out[0], out[1]);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) append_kernel(const Kv4Params p) {
    constexpr int kG = D / kGroup4;                 // groups of a head
    const int lane = threadIdx.x & 31;
    const int t = static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    long long page;
    int row;
    if (!locate(p, p.slots[t], page, row)) return;
    const uint16_t* k = static_cast<const uint16_t*>(p.k) + t * p.k_token;
    const uint16_t* v = static_cast<const uint16_t*>(p.v) + t * p.v_token;
    const int groups = p.Hkv * kG;
    for (int g0 = lane; g0 < groups; g0 += 64) {
        // [key | value][group g0 | g0 + 32]
        uint32_t w[2][2][8];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int g = g0 + 32 * u;
            if (g < groups) {
                const int head = g / kG, c = (g % kG) * kGroup4;
                const uint4* a = reinterpret_cast<const uint4*>(k + head * p.k_head + c);
                const uint4* b = reinterpret_cast<const uint4*>(v + head * p.v_head + c);
                *reinterpret_cast<uint4*>(&w[0][u][0]) = __ldg(a);
                *reinterpret_cast<uint4*>(&w[0][u][4]) = __ldg(a + 1);
                *reinterpret_cast<uint4*>(&w[1][u][0]) = __ldg(b);
                *reinterpret_cast<uint4*>(&w[1][u][4]) = __ldg(b + 1);
            }
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int g = g0 + 32 * u;
            if (g < groups) {
                const int head = g / kG, gi = g % kG;
                const long long at = (page * p.Hkv + head) * p.page + row;
                uint32_t scale;
                const uint2 kq = quantise<BF16>(w[0][u], p.k_unit, scale);
                *reinterpret_cast<uint2*>(p.kc + at * (D / 2) + gi * 8) = kq;
                p.ks[at * kG + gi] = static_cast<uint8_t>(scale);
                const uint2 vq = quantise<BF16>(w[1][u], p.v_unit, scale);
                *reinterpret_cast<uint2*>(p.vc + at * (D / 2) + gi * 8) = vq;
                p.vs[at * kG + gi] = static_cast<uint8_t>(scale);
            }
        }
    }
}

// Four bytes of codes and their scale back to eight values of the output type.
template <bool BF16>
__device__ __forceinline__ uint4 expand(uint32_t codes, uint32_t scale, float unit) {
    const uint32_t s2 = e4m3x2_to_f16(scale | scale << 8);
    uint32_t r[4], o[4];
    e2m1_word_to_f16(codes, r[0], r[1], r[2], r[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t m = hmul2_u32(r[i], s2);          // exact
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&m));
        if constexpr (BF16) {
            const __nv_bfloat162 y = __floats2bfloat162_rn(f.x * unit, f.y * unit);
            o[i] = *reinterpret_cast<const uint32_t*>(&y);
        } else {
            const __half2 y = __floats2half2_rn(f.x * unit, f.y * unit);
            o[i] = *reinterpret_cast<const uint32_t*>(&y);
        }
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D, bool BF16>
__global__ void __launch_bounds__(kThreads) gather_kernel(const Kv4Params p) {
    constexpr int kH = D / 8;
    const int lane = threadIdx.x & 31;
    const int t = static_cast<int>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (t >= p.T) return;
    long long page = 0;
    int row = 0;
    const bool held = locate(p, p.slots[t], page, row);
    const int halves = p.Hkv * kH;
    uint4* k = static_cast<uint4*>(const_cast<void*>(p.k)) + static_cast<long long>(t) * halves;
    uint4* v = static_cast<uint4*>(const_cast<void*>(p.v)) + static_cast<long long>(t) * halves;
    for (int g0 = lane; g0 < halves; g0 += 128) {
        uint32_t c[2][4], s[2][4];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int h = g0 + 32 * u;
            c[0][u] = c[1][u] = s[0][u] = s[1][u] = 0;
            if (held && h < halves) {
                const long long at = (page * p.Hkv + h / kH) * p.page + row;
                const int hi = h % kH;
                c[0][u] = *reinterpret_cast<const uint32_t*>(p.kc + at * (D / 2) + hi * 4);
                c[1][u] = *reinterpret_cast<const uint32_t*>(p.vc + at * (D / 2) + hi * 4);
                s[0][u] = p.ks[at * (D / kGroup4) + hi / 2];
                s[1][u] = p.vs[at * (D / kGroup4) + hi / 2];
            }
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int h = g0 + 32 * u;
            if (h < halves) {
                k[h] = expand<BF16>(c[0][u], s[0][u], p.k_unit);
                v[h] = expand<BF16>(c[1][u], s[1][u], p.v_unit);
            }
        }
    }
}

// Checks shared by append and gather; BSATTN_OK with p.T == 0 means nothing to do.
int check(const Kv4Params& p, int num_pages, int d, bsattn_dtype dtype, const void* workspace,
          size_t workspace_bytes) {
    if (p.T < 0 || p.Hkv <= 0 || num_pages <= 0 || p.page <= 0) return BSATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return BSATTN_ERR_UNSUPPORTED;
    if (dtype != BSATTN_F16 && dtype != BSATTN_BF16) return BSATTN_ERR_UNSUPPORTED;
    if (p.Hkv > (1 << 20) || p.T > (1 << 30)) return BSATTN_ERR_UNSUPPORTED;
    if (!unit_ok4(p.k_unit) || !unit_ok4(p.v_unit)) return BSATTN_ERR_INVALID_ARG;
    if (!workspace || workspace_bytes < 256 || !aligned16(workspace)) return BSATTN_ERR_INVALID_ARG;
    if (p.T == 0) return BSATTN_OK;
    if (!p.k || !p.v || !p.slots || !p.kc || !p.ks || !p.vc || !p.vs) return BSATTN_ERR_INVALID_ARG;
    if (!aligned16(p.k) || !aligned16(p.v) || !aligned16(p.kc) || !aligned16(p.ks) || !aligned16(p.vc) ||
        !aligned16(p.vs))
        return BSATTN_ERR_INVALID_ARG;
    return BSATTN_OK;
}

}  // namespace
}  // namespace bsattn

extern "C" int bsattn_kv4_append(const void* k, const void* v, long long k_token_stride,
                                 long long k_head_stride, long long v_token_stride,
                                 long long v_head_stride, const int64_t* slots, uint8_t* k_codes,
                                 uint8_t* k_scales, uint8_t* v_codes, uint8_t* v_scales, float k_scale,
                                 float v_scale, int T, int Hkv, int num_pages, int page_size, int d,
                                 bsattn_dtype dtype, void* workspace, size_t workspace_bytes,
                                 void* stream) {
    using namespace bsattn;
    Kv4Params p{k, v, k_token_stride, k_head_stride, v_token_stride, v_head_stride, slots, k_codes,
                k_scales, v_codes, v_scales, k_scale, v_scale, T, Hkv, page_size,
                static_cast<long long>(num_pages) * page_size, status_word(workspace)};
    const int rc = check(p, num_pages, d, dtype, workspace, workspace_bytes);
    if (rc || T == 0) return rc;
    // the stride of a dimension of one entry is never used
    if ((T > 1 && ((k_token_stride | v_token_stride) & 7)) || (Hkv > 1 && ((k_head_stride | v_head_stride) & 7)))
        return BSATTN_ERR_INVALID_ARG;
    p.k_unit = 1.f / k_scale;                      // a power of two: exact
    p.v_unit = 1.f / v_scale;
    const unsigned grid = (static_cast<unsigned>(T) + kWarps - 1) / kWarps;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == BSATTN_BF16;
    if (d == 64) {
        if (bf16) append_kernel<64, true><<<grid, kThreads, 0, st>>>(p);
        else append_kernel<64, false><<<grid, kThreads, 0, st>>>(p);
    } else {
        if (bf16) append_kernel<128, true><<<grid, kThreads, 0, st>>>(p);
        else append_kernel<128, false><<<grid, kThreads, 0, st>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

extern "C" int bsattn_kv4_gather(const int64_t* slots, const uint8_t* k_codes, const uint8_t* k_scales,
                                 const uint8_t* v_codes, const uint8_t* v_scales, float k_scale,
                                 float v_scale, void* k, void* v, int T, int Hkv, int num_pages,
                                 int page_size, int d, bsattn_dtype dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
    using namespace bsattn;
    Kv4Params p{k, v, 0, 0, 0, 0, slots, const_cast<uint8_t*>(k_codes), const_cast<uint8_t*>(k_scales),
                const_cast<uint8_t*>(v_codes), const_cast<uint8_t*>(v_scales), k_scale, v_scale, T, Hkv,
                page_size, static_cast<long long>(num_pages) * page_size, status_word(workspace)};
    const int rc = check(p, num_pages, d, dtype, workspace, workspace_bytes);
    if (rc || T == 0) return rc;
    const unsigned grid = (static_cast<unsigned>(T) + kWarps - 1) / kWarps;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool bf16 = dtype == BSATTN_BF16;
    if (d == 64) {
        if (bf16) gather_kernel<64, true><<<grid, kThreads, 0, st>>>(p);
        else gather_kernel<64, false><<<grid, kThreads, 0, st>>>(p);
    } else {
        if (bf16) gather_kernel<128, true><<<grid, kThreads, 0, st>>>(p);
        else gather_kernel<128, false><<<grid, kThreads, 0, st>>>(p);
    }
    return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}
