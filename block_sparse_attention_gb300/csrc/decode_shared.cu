// decode_shared.cu -- one query token per sequence over a prefix that sequences share and each one's own tokens,
// 16-bit paged cache, sm_103a.
//
//     out = softmax_j(q . k_j / sqrt(d)) v_j,   j over the prefix's tokens and the sequence's own
//
// The softmax over both is joined from its parts: with (O, L) the result and log-sum-exp of a part,
// out = sum O 2^(L - M) / sum 2^(L - M).  One kernel makes the parts, and each of its CTAs has one of two roles.
// Some have the sequences' own tokens (decode_shared_own.cuh).  The others have the prefixes: the query heads of a kv
// head of all sequences that share one are the rows of its products, so K and V of a prefix are read once for up to
// 256 rows and not once a sequence.  Own tokens are bound by HBM bandwidth, prefixes with many rows by the tensor core
// (256 rows of d = 128: 256 operations a byte against the 280 that the two peaks divide to), so they run beside each
// other: 256 sequences of 1000 own tokens on the average over 65521, 32 / 8 heads, take 259 us (276 once the GPU is warm);
// 178 to 193 with prefixes alone, 169 with own tokens alone, and 363 by two kernels one after the other.  A CTA learns its
// role from the lengths, which every CTA adds up for itself (3 us).
//
// The rows of a prefix stand in two tcgen05 tiles a CTA:
//     S_x = Q_x K^T    M=128 N=128 K=d, fp32 in TMEM
//     P_x              exp2 online softmax, one thread a row, written over S_x as the 16-bit type
//     O_x += P_x V     M=128 N=d K=128, A = P_x from TMEM
// as in prefill_window.cu, with its roles (warps 0-3 and 4-7 softmax of tile 0 and 1, warps 8 and 9 their
// products, warp 10 the copies), its turns, its halves of P and its rule that the reference maximum moves only
// when it has grown by 2^8.  Where a prefix has no more than 128 rows, both tiles are the same rows and take
// every second key tile each, without turns.
// The prefixes' keys, end to end, are cut into equal parts, one a CTA, so that one long prefix and many
// short ones both fill their share of the GPU (decode_shared.cuh); a CTA goes from one piece to the next without a
// break.  With few rows the way to the first tile's end (lengths, page table, queries and keys, and this code, which has
// to come to every SM too: 10 us of 58 for 64 sequences over 32768 tokens) and the joining (9 us) are what shows.
//
// TMEM: S_0 0-127, S_1 128-255, O_0 256.., O_1 256 + d...  Every wait is bounded: on expiry the CTA records
// BSATTN_ERR_TIMEOUT, hands its remaining pieces over as NaN, drains what is in flight and leaves.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include "decode_shared.cuh"
#include "decode_shared_own.cuh"
#include "host_internal.h"
#include "tile128.cuh"

namespace bsattn {
namespace {

constexpr int kThreads = kSharedThreads;
constexpr int kMmaWarp = 8;              // and 9
constexpr int kLoadWarp = 10;
constexpr int kRegsSoftmax = 208, kRegsOther = 88;       // registers a thread: two warpgroups, and the third
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256;
constexpr float kRescaleLog2 = 8.0f;
constexpr int kLeastOwn = 2;             // units of own tokens that a warp has at least
// Notes of key tiles, in turn: the loader is never this many tiles ahead of the last warp of a softmax.
constexpr int kNotes = 16;

template <int D>
struct Cfg {
    static constexpr int kStages = D == 64 ? 10 : 5;             // one 128-row tile of K or V each
    static constexpr uint32_t kTile = 128 * D * 2;
    static constexpr uint32_t kKV = 2 * kTile;                   // after two query tiles
    static constexpr uint32_t kBars = kKV + kStages * kTile > OwnRing<D>::kBytes ? kKV + kStages * kTile : OwnRing<D>::kBytes;
    // q_full[2] q_free[2] full[stages] empty[stages] s_full[2] p_half[2] p_full[2] o_full[2] o_free[2] fin[2] turn[2]
    static constexpr uint32_t kNumBars = 4 + 2 * kStages + 14;
    static constexpr uint32_t kMisc = (kBars + 8 * kNumBars + 15) & ~15u;   // tmem base, abort flag, first prefix
    static constexpr uint32_t kMissing = kMisc + 16;             // [kNotes]: which halves of a key tile are not there
    static constexpr uint32_t kBytes = 1024 + kMissing + 4 * kNotes;
    static_assert(kBytes <= 226 * 1024, "shared memory");        // the scan's static arrays beside it
    // What a unit of a prefix costs, in units of own tokens: 1.6 us a CTA, while its 12 warps would have that many of the
    // others.  (256 sequences of 1000 own tokens over 65521: 267 us with 12, 273 with 13, 277 with 14, 292 with 15, where two
    // runs of the same are 5 apart; 64 over 32768: 59.0, 57.5, 57.1, 57.0; d = 64, 192 over 6 prefixes: 70.6 with 16, 69.4
    // with 18, 71.3 with 20, 74.2 with 22.)
    static constexpr float kCost = D == 128 ? 13.f : 18.f;
};

struct PrefixParams {
    SharedCall s;
    int q_bytes;                         // of a query tile
};

// Which CTAs have what.
struct Split {
    int prefix_ctas;                     // the first ones; the others have own tokens
    long long prefix_chunk;              // units of a (CTA, lane)
    int own_parts;                       // for each kv head
    long long own_chunk;
};

// The prefixes and the own tokens get CTAs in proportion to what they cost, but none more than it has use for.
template <int D, bool HALVES>
__device__ __forceinline__ Split split_of(const SharedCall& s, long long prefix_total, long long own_total) {
    const int n = static_cast<int>(gridDim.x), least = HALVES ? 2 : 1, lanes = s.side * s.deep;
    const float cost = static_cast<float>(prefix_total) * lanes * (HALVES ? 0.5f * Cfg<D>::kCost : Cfg<D>::kCost);
    const float own_cost = static_cast<float>(own_total) * s.Hkv;
    // (a warp a kv head at least; the launch has as many CTAs as that and a lane each take)
    const int most = (n - (own_total > 0 ? (s.Hkv + kOwnWarps - 1) / kOwnWarps : 0)) / lanes;
    const long long use = min((prefix_total + least - 1) / least, static_cast<long long>(most));
    const long long own_use = ((own_total + kLeastOwn - 1) / kLeastOwn * s.Hkv + kOwnWarps - 1) / kOwnWarps;
    long long parts = cost > 0.f ? max(static_cast<long long>(n * (cost / (cost + own_cost)) / lanes + 0.5f), 1LL) : 0LL;
    parts = min(max(parts, (n - min(own_use, static_cast<long long>(n))) / lanes), use);
    Split x;
    x.prefix_ctas = static_cast<int>(parts) * lanes;
    x.prefix_chunk = parts > 0 ? max((prefix_total + parts - 1) / parts, static_cast<long long>(least)) : least;
    x.own_parts = (n - x.prefix_ctas) * kOwnWarps / s.Hkv;
    x.own_chunk = x.own_parts > 0 ? max((own_total + x.own_parts - 1) / x.own_parts, static_cast<long long>(kLeastOwn)) : kLeastOwn;
    return x;
}

// A CTA's walk over its units, from piece to piece.
struct Walk {
    long long at, end, base;             // units done, the last one, units before prefix p
    int p;
};

struct Piece {
    int p, b0, kvh;                      // prefix, first of the item's sequences, kv head
    int k0, k1, len;                     // key tiles [k0, k1), keys of the prefix
    int rows;                            // of the item
    long long place;                     // of the first one
};

__device__ __forceinline__ bool next_piece(const PrefixParams& prm, int part, int beside, Walk& w, Piece& x) {
    while (w.at < w.end) {
        PrefixGroup g = prefix_group(prm.s, w.p);
        for (;;) {
            const long long units = prefix_units(prm.s, g);
            if (w.at < w.base + units) break;
            w.base += units;
            g = prefix_group(prm.s, ++w.p);
        }
        const long long local = w.at - w.base;
        const long long item = local <= 0x7fffffffLL ? static_cast<int>(local) / g.tiles : local / g.tiles;
        x.p = w.p;
        x.k0 = static_cast<int>(local - item * g.tiles);
        x.k1 = static_cast<int>(min(static_cast<long long>(g.tiles), x.k0 + (w.end - w.at)));
        w.at += x.k1 - x.k0;
        const int along = prm.s.Hkv / prm.s.side, m = static_cast<int>(item / along), side = beside % prm.s.side;
        const int t = m * prm.s.deep + beside / prm.s.side;
        if (t * prm.s.seqs >= g.n) continue;                  // the other lanes have one time more
        x.kvh = static_cast<int>(item - static_cast<long long>(m) * along) * prm.s.side + side;
        x.b0 = g.start + t * prm.s.seqs;
        x.len = g.len;
        x.place = prefix_place(prm.s, g, part, t, x.kvh, x.rows);
        return true;
    }
    return false;
}

// HALVES: both query tiles are the same rows, tile 0 takes the even key tiles of a piece and tile 1 the odd ones.
template <int D, bool BF16, bool HALVES>
__global__ void __launch_bounds__(kThreads, 1)
    shared_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap own_k,
                  const __grid_constant__ CUtensorMap own_v, const PrefixParams p) {
    using C = Cfg<D>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sq = sm;
    uint8_t* skv = sm + C::kKV;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + C::kBars);   // [2]
    uint64_t* q_free = q_full + 2;                                    // [2]
    uint64_t* full = q_free + 2;                                      // [stages]
    uint64_t* empty = full + kStages;                                 // [stages] both query tiles
    uint64_t* s_full = empty + kStages;                               // [2] the product, and its issuer
    uint64_t* p_half = s_full + 2;                                    // [2] four warps: P of the first 64 keys
    uint64_t* p_full = p_half + 2;                                    // [2] four warps
    uint64_t* o_full = p_full + 2;                                    // [2] a piece's last P V
    uint64_t* o_free = o_full + 2;                                    // [2] four warps
    uint64_t* fin = o_free + 2;                                       // [2]
    uint64_t* turn = fin + 2;                                         // [2] the other has issued
    int* misc = reinterpret_cast<int*>(sm + C::kMisc);
    int* missing = reinterpret_cast<int*>(sm + C::kMissing);
    volatile int* abort_flag = &misc[1];
    int* status = p.s.status;
    __shared__ long long warp_sums[2][kThreads / 32];
    __shared__ long long first_base;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int lanes = p.s.side * p.s.deep, part = static_cast<int>(blockIdx.x) / lanes, beside = static_cast<int>(blockIdx.x) - part * lanes;

    // The kernel that joins may start wherever there is room (and waits for this one by itself).  With the leave to
    // start given at the top, its CTAs come to wait beside this one's.
    const auto leave = [] { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); };

    if (tid == 32 * kLoadWarp) {
        tma_prefetch_desc(&tm_q);
        tma_prefetch_desc(&tm_k);
        tma_prefetch_desc(&tm_v);
        tma_prefetch_desc(&own_k);
        tma_prefetch_desc(&own_v);
    }

    // ------------------------------------------------------------ this CTA's part of all units
    Walk start;
    {
        // a thread a stretch of prefixes, and one of sequences
        const int per = (p.s.P + kThreads - 1) / kThreads, own_per = (p.s.B + kThreads - 1) / kThreads;
        long long sum = 0, own_sum = 0;
        for (int k = 0; k < own_per; ++k) {
            const int b = tid * own_per + k;
            if (b >= p.s.B) break;
            const int len = p.s.own_lens[b];
            own_sum += own_units(max(min(len, p.s.own_room), 0));
            if ((len < 0 || len > p.s.own_room) && blockIdx.x == 0) atomicOr(status, BSATTN_ERR_BAD_INDEX);
        }
        for (int k = 0; k < per; ++k) {
            const int i = tid * per + k;
            if (i >= p.s.P) break;
            const PrefixGroup g = prefix_group(p.s, i);
            sum += prefix_units(p.s, g);
            if (g.bad && blockIdx.x == 0) atomicOr(status, BSATTN_ERR_BAD_INDEX);
        }
        long long upto = sum, own_upto = own_sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long u = __shfl_up_sync(0xffffffffu, upto, o), v = __shfl_up_sync(0xffffffffu, own_upto, o);
            if (lane >= o) {
                upto += u;
                own_upto += v;
            }
        }
        if (lane == 31) {
            warp_sums[0][warp] = upto;
            warp_sums[1][warp] = own_upto;
        }
        __syncthreads();
        long long total = 0, own_total = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) {
                upto += warp_sums[0][w];
                own_upto += warp_sums[1][w];
            }
            total += warp_sums[0][w];
            own_total += warp_sums[1][w];
        }
        const Split split = split_of<D, HALVES>(p.s, total, own_total);
        if (blockIdx.x == 0) {
            long long before = upto - sum;
            for (int k = 0; k < per; ++k) {
                const int i = tid * per + k;
                if (i >= p.s.P) break;
                p.s.prefix_info[1 + i] = before;
                before += prefix_units(p.s, prefix_group(p.s, i));
            }
            before = own_upto - own_sum;
            for (int k = 0; k < own_per; ++k) {
                const int b = tid * own_per + k;
                if (b >= p.s.B) break;
                p.s.own_info[1 + b] = before;
                before += own_units(own_len(p.s, b));
            }
            if (tid == 0) {
                p.s.prefix_info[0] = split.prefix_chunk;
                p.s.own_info[0] = split.own_chunk;
            }
        }
        if (static_cast<int>(blockIdx.x) >= split.prefix_ctas) {
            // ------------------------------------------------------------ own tokens
            using R = OwnRing<D>;
            long long* upto_of = reinterpret_cast<long long*>(sm + R::kUpto);
            upto_of[tid] = own_upto;
            if (tid + kThreads < kStretches) upto_of[tid + kThreads] = LLONG_MAX;
            if (tid < kOwnWarps * R::kStages) mbar_init(reinterpret_cast<uint64_t*>(sm + R::kBars) + tid, 1);
            fence_barrier_init();
            if (tid == 0) misc[1] = 0;
            __syncthreads();
            // neighbouring warps have the same tokens of neighbouring kv heads, which lie next to each other
            const int id = (static_cast<int>(blockIdx.x) - split.prefix_ctas) * kOwnWarps + warp, mine = id / p.s.Hkv;
            if (mine < split.own_parts)
                own_tokens<D, BF16>(&own_k, &own_v, p.s, sm, abort_flag, mine, id - mine * p.s.Hkv, split.own_chunk, own_total);
            leave();
            return;
        }
        const long long chunk = split.prefix_chunk;
        start.at = part * chunk;
        start.end = min(start.at + chunk, total);
        if (start.at >= total) {                              // the whole CTA
            leave();
            return;
        }
        if (upto - sum <= start.at && start.at < upto) {
            int i = tid * per;
            long long before = upto - sum;
            for (;; ++i) {
                const long long n = prefix_units(p.s, prefix_group(p.s, i));
                if (start.at < before + n) break;
                before += n;
            }
            misc[2] = i;
            first_base = before;
        }
    }

    if (tid == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 1);
            mbar_init(&q_free[x], 1);
            mbar_init(&s_full[x], 2);
            mbar_init(&p_half[x], 4);
            mbar_init(&p_full[x], 4);
            mbar_init(&o_full[x], 1);
            mbar_init(&o_free[x], 4);
            mbar_init(&fin[x], 1);
            mbar_init(&turn[x], 1);
        }
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);
        }
        misc[1] = 0;
        fence_barrier_init();
    }
    if (warp == kMmaWarp) {
        tmem_alloc(reinterpret_cast<uint32_t*>(&misc[0]), kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tbase = static_cast<uint32_t>(misc[0]);
    start.p = misc[2];
    start.base = first_base;
    // key tiles of query tile x in a piece of n
    const auto tiles_of = [](int x, int n) { return HALVES ? (n + 1 - x) / 2 : n; };

    // The softmax keeps a row of 128 scores a thread: its two warpgroups take 208 of the registers that the
    // launch gave, the third is left 88.  (launch() has checked that the launch gave that many.)
    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        Walk walk = start;
        Piece piece;
        if (warp == kLoadWarp) {
            // ------------------------------------------------------------ TMA
            // K and V of the prefixes and of the own tokens are streamed past what is in L2 and read again: this code,
            // which every SM fetches at the start, the pieces, the tables (64 sequences over 32768 tokens: 57.5 us, 68.0
            // without; a few tokens' worth only: the same).
            const uint64_t once = l2_evict_first();
            int g = 0;                                   // tiles loaded, K and V counted apart
            int nq[2] = {0, 0};                          // Q tiles loaded
            bool ok = true, bad = false;
            while (ok && next_piece(p, part, beside, walk, piece)) {
                const int n = piece.k1 - piece.k0;
                const auto queries = [&] {
                    for (int x = 0; ok && x < 2; ++x) {
                        if (tiles_of(x, n) == 0) continue;
                        ok = nq[x] == 0 || warp_wait_within(&q_free[x], (nq[x] - 1) & 1, p.s.budget_ns, abort_flag, status);
                        if (!ok) break;
                        if (lane == 0) {
                            mbar_arrive_expect_tx(&q_full[x], static_cast<uint32_t>(p.q_bytes));
                            const int b = piece.b0 + (HALVES ? 0 : x * (p.s.seqs / 2));
#pragma unroll
                            for (int h = 0; h < D / 64; ++h)
                                tma_load_4d(sq + x * C::kTile + h * 16384, &tm_q, &q_full[x], h * 64, 0, piece.kvh, b);
                        }
                        ++nq[x];
                    }
                };
                // (of a later piece they come after its first K, as they wait for the tiles before it)
                const bool at_once = nq[0] == 0 && nq[1] == 0;
                if (at_once) queries();
                int look = -1;
                for (int i = 0; ok && i < n; ++i) {
                    if ((i & 15) == 0) {
                        // the cache rows of the next 32 blocks of 64 keys
                        const int key = 2 * (piece.k0 + i) * 64 + 64 * lane;
                        look = -1;
                        if (key < piece.len && key < 128 * piece.k1) {
                            const int lp = key / p.s.page_size;
                            const int page = p.s.prefix_table[static_cast<size_t>(piece.p) * p.s.prefix_pages + lp];
                            if (page >= 0 && page < p.s.num_pages) look = page * p.s.page_size + key - lp * p.s.page_size;
                            else bad = true;
                        }
                    }
                    const int r0 = __shfl_sync(0xffffffffu, look, 2 * (i & 15));
                    const int r1 = __shfl_sync(0xffffffffu, look, 2 * (i & 15) + 1);
                    // rows past the cache's end are filled with zeros
                    const int none = p.s.num_pages * p.s.page_size;
#pragma unroll 1
                    for (int v = 0; ok && v < 2; ++v) {
                        const int st = g % kStages;
                        ok = g < kStages || warp_wait_within(&empty[st], (g / kStages - 1) & 1, p.s.budget_ns, abort_flag, status);
                        if (!ok) break;
                        if (lane == 0) {
                            if (v == 0) missing[(g >> 1) % kNotes] = (r0 < 0 ? 1 : 0) | (r1 < 0 ? 2 : 0);
                            mbar_arrive_expect_tx(&full[st], C::kTile);
#pragma unroll
                            for (int h = 0; h < D / 64; ++h) {
                                uint8_t* dst = skv + st * C::kTile + h * 16384;
                                tma_load_3d(dst, v ? &tm_v : &tm_k, &full[st], h * 64, piece.kvh, r0 < 0 ? none : r0, once);
                                tma_load_3d(dst + 8192, v ? &tm_v : &tm_k, &full[st], h * 64, piece.kvh, r1 < 0 ? none : r1, once);
                            }
                        }
                        ++g;
                        if (i > 0 || v > 0 || at_once) continue;
                        queries();
                    }
                }
            }
            if (__any_sync(0xffffffffu, bad) && lane == 0) atomicOr(status, BSATTN_ERR_BAD_INDEX);
            // copies in flight land before the shared memory is released, whoever has given up on them
            const uint64_t dl = global_timer_ns() + 200000000ull;
            for (int x = 0; x < 2; ++x)
                if (nq[x] > 0) wait_parity_drain(&q_full[x], (nq[x] - 1) & 1, dl);
            for (int j = max(0, g - kStages); j < g; ++j) wait_parity_drain(&full[j % kStages], (j / kStages) & 1, dl);
            __syncwarp();
        } else if (warp == kMmaWarp || warp == kMmaWarp + 1) {
            // ------------------------------------------------------------ products of query tile x
            const int x = static_cast<int>(uniform(static_cast<uint32_t>(warp - kMmaWarp)));
            const bool lead = elect_one_sync();
            constexpr uint32_t idS = idesc_f16(128, 128, BF16, false);
            constexpr uint32_t idO = idesc_f16(128, D, BF16, true);
            const uint64_t q_desc = uniform(sdesc_sw128(smem_u32(sq + x * C::kTile), 16, 1024));
            const uint64_t k_desc = sdesc_sw128(smem_u32(skv), 16, 1024);
            const uint64_t v_desc = sdesc_sw128(smem_u32(skv), 16384, 1024);
            constexpr uint32_t kTileDesc = C::kTile >> 4;
            const uint32_t ts = uniform(tbase + 128 * x), to = uniform(tbase + kOCol + D * x);
            int blk = 0, items = 0, outs = 0;                // tiles, pieces (S begun, O begun) so far
            const auto wait = [&](uint64_t* bar, int parity) {
                return warp_wait_within(bar, static_cast<uint32_t>(parity & 1), p.s.budget_ns, abort_flag, status);
            };
            bool ok = true;
            // rows of a V tile past the prefix's end may hold anything, and a weight of 0 must not meet a NaN
            // (both issuers may clear them: they write the same)
            const auto clear_tail = [&](int st, int valid) {
                for (int e = lane; e < (128 - valid) * (D / 8); e += 32) {
                    const int r = valid + e / (D / 8), c = e % (D / 8);
                    *reinterpret_cast<uint4*>(skv + st * C::kTile + (c >> 3) * 16384 + r * 128 + (c & 7) * 16) =
                        make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async_smem();
                __syncwarp();
            };
            const auto issue_s = [&](int st) {
                const uint64_t kb = uniform(k_desc + static_cast<uint32_t>(st) * kTileDesc);
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < D / 16; ++kk) {
                    const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                    mma_f16_ss_if(lead, ts, q_desc + off, kb + off, idS, kk > 0 ? 1u : 0u);
                }
                mma_commit_if(lead, &s_full[x]);
                // passes on what the loader has noted, which this warp has seen by its wait for the tile
                mbar_arrive_if(lead, &s_full[x]);
            };
            // half of P V, which the softmax hands over while it works on the rest
            const auto issue_pv = [&](uint64_t vb, int half, bool begins) {
                tc_fence_after();
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int kk = 4 * half + e;
                    mma_f16_ts_if(lead, to, ts + 8 * kk, vb + ((kk * 2048) >> 4), idO, (!begins || half > 0 || e > 0) ? 1u : 0u);
                }
            };
            if constexpr (HALVES) {
                // Every stage is waited for in turn, the other tile's too, which are given back here as they are
                // not read.  V is given back by the product itself, so that the next tiles can come early.
                int g = 0;                                   // ring position: K at g, V after it
                while (ok && next_piece(p, part, beside, walk, piece)) {
                    const int n = piece.k1 - piece.k0, mine = tiles_of(x, n);
                    int done = 0;
                    for (int i = 0; ok && i < n; ++i, g += 2) {
                        const int sk = g % kStages, sv = (g + 1) % kStages;
                        if (!(ok = wait(&full[sk], g / kStages))) break;
                        if ((i & 1) != x) {
                            mbar_arrive_if(lead, &empty[sk]);
                            if (!(ok = wait(&full[sv], (g + 1) / kStages))) break;
                            mbar_arrive_if(lead, &empty[sv]);
                            continue;
                        }
                        if (done == 0 && !(ok = wait(&q_full[x], items++))) break;
                        issue_s(sk);
                        ++blk;
                        if (!(ok = wait(&full[sv], (g + 1) / kStages))) break;
                        const int valid = piece.len - 128 * (piece.k0 + i);
                        if (valid < 128) clear_tail(sv, valid);
                        if (done == 0 && outs++ > 0 && !(ok = wait(&o_free[x], outs - 2))) break;
                        const uint64_t vb = uniform(v_desc + static_cast<uint32_t>(sv) * kTileDesc);
                        if (!(ok = wait(&p_half[x], blk - 1))) break;
                        issue_pv(vb, 0, done == 0);
                        if (!(ok = wait(&p_full[x], blk - 1))) break;
                        issue_pv(vb, 1, done == 0);
                        if (++done == mine) mma_commit_if(lead, &o_full[x]);
                        mma_commit_if(lead, &empty[sv]);
                    }
                }
            } else {
                int g = 0, rounds = 0;
                bool pend = false, begins = false, ends = false; // a tile awaits its P V, which begins / ends its O
                int valid = 128;                                 // its rows of V that are the prefix's
                // One round: P V of the tile before, be it of the piece before, and S of the tile at position g,
                // if there is one.  None of its waits waits for what comes after it: K of position g takes
                // the stage of position g - 5 or an earlier one, which the softmax gave back for a round before.
                auto round = [&](bool tile, bool first, bool last, int rows) {
                    const int sk = g % kStages, sv = (g + kStages - 1) % kStages;
                    if (pend && !wait(&full[sv], (g - 1) / kStages)) return false;
                    if (pend && valid < 128) clear_tail(sv, valid);
                    if (tile && !wait(&full[sk], g / kStages)) return false;
                    const uint64_t vb = uniform(v_desc + static_cast<uint32_t>(sv) * kTileDesc);
                    if (tile && first && !wait(&q_full[x], items++)) return false;
                    // tile 0's round comes after tile 1's round before, tile 1's after tile 0's
                    if (rounds + x > 0 && !wait(&turn[x], rounds + x + 1)) return false;
                    ++rounds;
                    if (pend) {
                        if (begins && outs++ > 0 && !wait(&o_free[x], outs - 2)) return false;
                        if (!wait(&p_half[x], blk - 1)) return false;
                        issue_pv(vb, 0, begins);
                        if (!wait(&p_full[x], blk - 1)) return false;
                        issue_pv(vb, 1, begins);
                        if (ends) mma_commit_if(lead, &o_full[x]);
                        pend = false;
                    }
                    if (tile) {
                        issue_s(sk);
                        ++blk;
                        pend = true;
                        begins = first;
                        ends = last;
                        valid = rows;
                    }
                    mbar_arrive_if(lead, &turn[1 - x]);
                    return true;
                };
                while (ok && next_piece(p, part, beside, walk, piece))
                    for (int k = piece.k0; ok && k < piece.k1; ++k, g += 2)
                        ok = round(true, k == piece.k0, k == piece.k1 - 1, piece.len - 128 * k);
                if (ok) round(false, false, false, 0);
            }
            mma_commit_if(lead, &fin[x]);
            wait_parity_drain(&fin[x], 0, global_timer_ns() + 200000000ull);
            __syncwarp();
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ------------------------------------------------------------ softmax of query tile x
        const int x = warp >> 2;
        const int lrow = 32 * (warp & 3) + lane;
        const uint32_t lanes = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t ts = tbase + lanes + 128 * x, to = tbase + lanes + kOCol + D * x;
        const float c = p.s.scale_log2;
        // A weight is exp2(x c - reference(m)), m the maximum that the row goes by.  fp16 ones are taken 2^kUp times as large,
        // so that those down to 2^-32 of the largest (2^-25, half of the smallest subnormal, for 2^7) count in O as they
        // do in l: ten thousand keys of 2^-25 each would else be lost from O alone.  m may lag by kRescaleLog2, so none
        // passes 2^15; where scores are so large that their rounding shows, m does not lag and the reference is
        // rounded up.  bf16 reaches far enough as it is.
        constexpr float kUp = BF16 ? 0.f : 7.f, kLagBelow = 1048576.f;
        static_assert(BF16 || kUp + kRescaleLog2 <= 15.f, "weights below 65504");
        const auto reference = [c](float m) { return BF16 ? m * c : __fmaf_ru(m, c, -kUp); };
        const bool speaks = (warp & 3) == 0 && lane == 0;
        const int tile_rows = HALVES ? p.s.part_rows : p.s.part_rows / 2;
        const int irow = HALVES ? lrow : x * tile_rows + lrow;       // row of the item
        int blk = 0, items = 0, g = 0;
        bool ok = true;
        Walk walk = start;
        Piece piece;
        while (next_piece(p, part, beside, walk, piece)) {
            const int pieces = piece.k1 - piece.k0, n = tiles_of(x, pieces);
            const int g0 = g;                            // ring position of the piece's first K tile
            g += 2 * pieces;
            const bool mine = lrow < tile_rows && irow < piece.rows;
            const size_t at = piece.place + (HALVES ? x * piece.rows + lrow : irow);
            float m_used = -INFINITY, l = 0.f;
            int v_read = -1;                             // stage of the V tile to give back when it is read
            for (int i = 0; ok && i < n; ++i, ++blk) {
                const int u = HALVES ? 2 * i + x : i;
                const int st = (g0 + 2 * u) % kStages;
                if (!warp_wait_within(&s_full[x], blk & 1, p.s.budget_ns, abort_flag, status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const int gone = missing[((g0 >> 1) + u) % kNotes];
                if (speaks) {
                    // S of this tile is there: its K tile has been read, and V of the tile before
                    if (!HALVES && v_read >= 0) mbar_arrive(&empty[v_read]);
                    mbar_arrive(&empty[st]);
                    v_read = (g0 + 2 * u + 1) % kStages;
                    if (i == n - 1) mbar_arrive(&q_free[x]);
                }
                __syncwarp();
                float s[128];
#pragma unroll
                for (int h = 0; h < 4; ++h) tmem_ld_row32(ts + 32 * h, reinterpret_cast<uint32_t*>(s) + 32 * h);
                tmem_wait_ld();
                const int valid = piece.len - 128 * (piece.k0 + u);
                if (valid < 128 || gone != 0) {
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const uint32_t on = gone >> (h >> 1) & 1 ? 0u : below(valid - 32 * h);
                        if (on == 0xffffffffu) continue;
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            if (!((on >> e) & 1u)) s[32 * h + e] = -INFINITY;
                    }
                }
                float mx;
                {
                    float m4[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        m4[j] = max3f(s[j], s[j + 4], s[j + 8]);
#pragma unroll
                        for (int e = 12; e + 4 < 128; e += 8) m4[j] = max3f(m4[j], s[j + e], s[j + e + 4]);
                        m4[j] = fmaxf(m4[j], s[j + 124]);
                    }
                    mx = fmaxf(max3f(m4[0], m4[1], m4[2]), m4[3]);
                }
                const float used = m_used * c;
                const bool grow = mx * c > used + kRescaleLog2 || (!BF16 && mx > m_used && !(fabsf(used) < kLagBelow));
                const float m_new = grow ? mx : m_used;
                const float alpha = grow ? ex2_approx((m_used - m_new) * c) : 1.f;
                const bool rescale = grow && m_used != -INFINITY;
                m_used = m_new;
                const float mc = m_new == -INFINITY ? 0.f : reference(m_new);
                if (__any_sync(0xffffffffu, rescale)) {
                    // O holds every tile before this one: their P V ran before this tile's S
#pragma unroll 1
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o[32];
                        tmem_ld_row32(to + c0, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                        tmem_st_row32(to + c0, o);
                    }
                }
                float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f),
                                 make_float2(0.f, 0.f)};
#pragma unroll
                for (int h = 0; h < 4; ++h) {
                    uint32_t pv[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        const float2 y = fma2f(make_float2(s[32 * h + 2 * e], s[32 * h + 2 * e + 1]), make_float2(c, c),
                                               make_float2(-mc, -mc));
                        const float2 ev = make_float2(ex2_approx(y.x), ex2_approx(y.y));
                        acc[e & 3] = add2f(acc[e & 3], ev);
                        pv[e] = pack2<BF16>(ev.x, ev.y);
                    }
                    tmem_st_row16(ts + 16 * h, pv);
                    if (h == 1) {
                        tmem_wait_st();
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&p_half[x]);
                    }
                }
                const float2 a2 = add2f(add2f(acc[0], acc[1]), add2f(acc[2], acc[3]));
                l = l * alpha + (a2.x + a2.y);
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[x]);
            }
            // ---- the piece's O / l and log-sum-exp (base 2)
            if (ok && n > 0) {
                ok = warp_wait_within(&o_full[x], items & 1, p.s.budget_ns, abort_flag, status);
                ++items;
            }
            if (!ok) {
                // (and so for the pieces after it: what lacks a part shows it)
                if (mine) p.s.prefix_lse[at] = __int_as_float(0x7fffffff);
                continue;
            }
            if (n == 0) {
                if (mine) p.s.prefix_lse[at] = -INFINITY;
                continue;
            }
            tc_fence_after();
            if (!HALVES && speaks) mbar_arrive(&empty[v_read]);
            __syncwarp();
            // a row without a finite score has l = 0, or NaN if it met one
            const float inv = l == 0.f ? 0.f : 1.f / l;
            const uint32_t rows = __ballot_sync(0xffffffffu, mine);
            // Four lanes exchange their pairs of columns, so that they write 64 bytes of a row (a row a lane would
            // be 32 lines a store: 4.3 us for 256 rows of 128, against 1.3).
            float* out = p.s.prefix_o + (at - lane) * D + 4 * (lane & 1) + 8 * (lane >> 1 & 1);
            const bool upper = (lane & 2) != 0, odd = (lane & 1) != 0;
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
                // a lane holds rows lane / 4 + 8 {0, 1} of 16, two neighbouring columns of every eight
                uint32_t o[D / 2];
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 64) tmem_ld_16x256b_x8(to + (static_cast<uint32_t>(16 * hf) << 16) + c0, o + c0 / 2);
                tmem_wait_ld();
                if (hf == 1) {
                    // O is in registers: the next piece's first P V may overwrite it
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&o_free[x]);
                }
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int row = 16 * hf + 8 * r + (lane >> 2);
                    const float by = __shfl_sync(0xffffffffu, inv, row);
                    const bool there = (rows >> row & 1u) != 0u;
#pragma unroll
                    for (int i = 0; i < D / 16; ++i) {
                        float f[2], g2[2];               // the lane's first and second pair
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float a = __uint_as_float(o[8 * i + 2 * r + e]) * by;
                            const float b = __uint_as_float(o[8 * i + 4 + 2 * r + e]) * by;
                            const float got = __shfl_xor_sync(0xffffffffu, upper ? a : b, 2);
                            f[e] = upper ? got : a;
                            g2[e] = upper ? b : got;
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const float got = __shfl_xor_sync(0xffffffffu, odd ? f[e] : g2[e], 1);
                            if (odd) f[e] = got;
                            else g2[e] = got;
                        }
                        if (there) *reinterpret_cast<float4*>(out + row * D + 16 * i) = make_float4(f[0], f[1], g2[0], g2[1]);
                    }
                }
            }
            if (mine) {
                p.s.prefix_lse[at] = l == 0.f ? -INFINITY : reference(m_used) + log2f(l);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tbase, kTmemCols);
    }
    leave();
}

template <int D, bool BF16, bool HALVES>
int launch(const CUtensorMap (&maps)[5], const PrefixParams& prm, int grid, cudaStream_t stream) {
    auto kern = shared_kernel<D, BF16, HALVES>;
    static std::atomic<unsigned long long> raised{0};
    const int rc = raise_smem_limit(reinterpret_cast<const void*>(kern), Cfg<D>::kBytes, raised);
    if (rc) return rc;
    // the warpgroups' register shares come out of the launch's: with fewer, the larger ones would never come
    static const bool enough = [kern] {
        cudaFuncAttributes a{};
        return cudaFuncGetAttributes(&a, kern) == cudaSuccess &&
               a.numRegs * kThreads >= 128 * (2 * kRegsSoftmax + kRegsOther);
    }();
    if (!enough) return BSATTN_ERR_CUDA;
    kern<<<static_cast<unsigned>(grid), kThreads, Cfg<D>::kBytes, stream>>>(maps[0], maps[1], maps[2], maps[3], maps[4], prm);
    return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

// Byte offsets of the workspace, behind the status word, and what depends on the shape and the GPU alone.
struct Layout {
    size_t prefix_info, own_info, prefix_lse, prefix_o, own_lse, own_o, total;
    int halves, seqs, part_rows, side, deep, prefix_parts, own_parts, grid;
    long long lane_rows;
};

Layout layout_of(int B, int P, int Hq, int Hkv, int d, int sms) {
    Layout w{};
    const int G = Hq / Hkv, tile = 128 / G;              // sequences of a 128-row tile
    // A prefix with no more than a tile of rows, on the average, has both query tiles of a CTA to itself (192 sequences
    // over 6 prefixes, d = 64: 69 us, and 88 with one of the tiles empty).
    w.halves = (static_cast<long long>(B) + P - 1) / P <= tile;
    w.seqs = w.halves ? tile : 2 * tile;
    w.part_rows = w.seqs * G;
    // A prefix with no more rows than a CTA has is read once: all its kv heads at the same keys at the same time, as
    // those lie next to each other in the cache (64 sequences over 32768 tokens: 57.5 us for 62.4).  One prefix with more is
    // read several times: at the same time, so that all but one reading comes from L2 (256 sequences over 65521: 273 us
    // for 335).
    const int times = (B + w.seqs - 1) / w.seqs;
    w.side = (static_cast<long long>(B) + P - 1) / P <= w.seqs && 2 * Hkv <= sms ? Hkv : 1;
    w.deep = P == 1 && times > 1 ? (times + (times + 7) / 8 - 1) / ((times + 7) / 8) : 1;
    // a CTA an SM, and no fewer than one for each lane and a warp for the own tokens of each kv head
    const int lanes = w.side * w.deep;
    w.grid = std::max(sms, lanes + (Hkv + kOwnWarps - 1) / kOwnWarps);
    w.prefix_parts = w.grid / lanes;                     // if all CTAs had prefixes, or own tokens
    w.own_parts = w.grid * kOwnWarps / Hkv;
    const long long of_items = w.deep > 1 ? static_cast<long long>((times + w.deep - 1) / w.deep) * w.seqs : B;
    w.lane_rows = static_cast<long long>(w.prefix_parts) * w.part_rows + of_items * G * (Hkv / w.side);
    const size_t rows = static_cast<size_t>(w.lane_rows) * lanes * (w.halves ? 2 : 1);
    const size_t own = (static_cast<size_t>(B) + w.own_parts) * Hq;
    size_t at = 256;
    const auto take = [&at](size_t bytes) {
        const size_t here = at;
        at += up256(bytes);
        return here;
    };
    w.prefix_info = take(sizeof(long long) * (static_cast<size_t>(P) + 1));
    w.own_info = take(sizeof(long long) * (static_cast<size_t>(B) + 1));
    w.prefix_lse = take(sizeof(float) * rows);
    w.prefix_o = take(sizeof(float) * rows * d);
    w.own_lse = take(sizeof(float) * own);
    w.own_o = take(sizeof(float) * own * d);
    w.total = at;
    return w;
}

int sms_of_device() {
    const int n = num_sms_of_current_device();
    return n > 0 ? n : 148;
}

}  // namespace
}  // namespace bsattn

extern "C" size_t bsattn_decode_shared_workspace_size(int B, int P, int Hq, int Hkv, int d) {
    using namespace bsattn;
    if (B <= 0 || P <= 0 || Hq <= 0 || Hkv <= 0 || d <= 0 || Hq % Hkv || Hq / Hkv > 8) return 256;
    return layout_of(B, P, Hq, Hkv, d, sms_of_device()).total;
}

extern "C" int bsattn_decode_shared(const void* q, const void* k_pages, const void* v_pages,
                                    const int32_t* prefix_lens, const int32_t* prefix_table,
                                    const int32_t* group_starts, const int32_t* cache_seqlens,
                                    const int32_t* block_table, void* out, int B, int P, int Hq, int Hkv,
                                    int num_pages, int page_size, int max_pages_per_prefix, int max_pages_per_seq,
                                    int d, bsattn_dtype dtype, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace bsattn;
    if (B < 0 || P <= 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || num_pages <= 0 || page_size <= 0 ||
        max_pages_per_prefix <= 0 || max_pages_per_seq <= 0)
        return BSATTN_ERR_INVALID_ARG;
    if (Hq / Hkv > 8 || page_size % 64 || (d != 64 && d != 128)) return BSATTN_ERR_UNSUPPORTED;
    if (dtype != BSATTN_F16 && dtype != BSATTN_BF16) return BSATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(num_pages) * page_size > 0x7fffffffLL - 128) return BSATTN_ERR_UNSUPPORTED;
    if (static_cast<long long>(B) * Hq > 0x7fffffffLL || P > (1 << 24) || Hkv > 1024) return BSATTN_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < 256 || !aligned16(workspace)) return BSATTN_ERR_INVALID_ARG;
    if (B == 0) return BSATTN_OK;
    if (!q || !out || !k_pages || !v_pages || !prefix_lens || !prefix_table || !group_starts || !cache_seqlens ||
        !block_table)
        return BSATTN_ERR_INVALID_ARG;
    if (!aligned16(q) || !aligned16(out) || !aligned16(k_pages) || !aligned16(v_pages)) return BSATTN_ERR_INVALID_ARG;
    // out is written by the last kernel, which reads neither q nor the cache: it may be q itself
    const size_t out_bytes = static_cast<size_t>(B) * Hq * d * 2;
    const uint64_t rows = uint64_t(num_pages) * page_size, row_bytes = uint64_t(Hkv) * d * 2;
    if ((out != q && overlap(out, out_bytes, q, out_bytes)) || overlap(out, out_bytes, k_pages, rows * row_bytes) ||
        overlap(out, out_bytes, v_pages, rows * row_bytes))
        return BSATTN_ERR_INVALID_ARG;
    const int sms = sms_of_device();
    const Layout w = layout_of(B, P, Hq, Hkv, d, sms);
    if (workspace_bytes < w.total) return BSATTN_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    PrefixParams prm{};
    SharedCall& s = prm.s;
    s.q = q;
    s.out = out;
    s.starts = group_starts;
    s.prefix_lens = prefix_lens;
    s.own_lens = cache_seqlens;
    s.prefix_table = prefix_table;
    s.own_table = block_table;
    s.prefix_info = reinterpret_cast<long long*>(ws + w.prefix_info);
    s.own_info = reinterpret_cast<long long*>(ws + w.own_info);
    s.prefix_lse = reinterpret_cast<float*>(ws + w.prefix_lse);
    s.prefix_o = reinterpret_cast<float*>(ws + w.prefix_o);
    s.own_lse = reinterpret_cast<float*>(ws + w.own_lse);
    s.own_o = reinterpret_cast<float*>(ws + w.own_o);
    s.status = status_word(workspace);
    s.B = B;
    s.P = P;
    s.Hq = Hq;
    s.Hkv = Hkv;
    s.seqs = w.seqs;
    s.part_rows = w.part_rows;
    s.halves = w.halves;
    s.side = w.side;
    s.deep = w.deep;
    s.lane_rows = w.lane_rows;
    s.page_size = page_size;
    s.num_pages = num_pages;
    s.prefix_pages = max_pages_per_prefix;
    s.own_pages = max_pages_per_seq;
    s.prefix_room = static_cast<int>(std::min(static_cast<long long>(max_pages_per_prefix) * page_size, 1LL << 30));
    s.own_room = static_cast<int>(std::min(static_cast<long long>(max_pages_per_seq) * page_size, 1LL << 30));
    s.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
    s.budget_ns = wait_budget_ns();
    const int G = Hq / Hkv, tile = 128 / G;
    prm.q_bytes = tile * G * d * 2;
    const bool bf16 = dtype == BSATTN_BF16;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    CUtensorMap maps[5];                                 // q, K, V, and K, V as own tokens are read
    const uint64_t dq[4] = {uint64_t(d), uint64_t(G), uint64_t(Hkv), uint64_t(B)};
    const uint64_t sq[3] = {d * 2ull, uint64_t(G) * d * 2, uint64_t(Hq) * d * 2};
    const uint32_t bq[4] = {64, uint32_t(G), 1, uint32_t(tile)};
    int rc = encode_4d(&maps[0], q, bf16, dq, sq, bq);
    for (int e = 0; e < 4 && !rc; ++e)
        rc = encode_3d(&maps[1 + e], e & 1 ? v_pages : k_pages, bf16, d, Hkv, rows, d * 2ull, row_bytes, 64, 1, e < 2 ? 64 : kTok, true);
    if (rc) return rc;
    const auto run = [&](auto dim, auto halves) {
        constexpr int D = decltype(dim)::value;
        constexpr bool HALVES = decltype(halves)::value;
        return bf16 ? launch<D, true, HALVES>(maps, prm, w.grid, st) : launch<D, false, HALVES>(maps, prm, w.grid, st);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (w.halves) rc = d == 64 ? run(D64{}, std::true_type{}) : run(D128{}, std::true_type{});
    else rc = d == 64 ? run(D64{}, std::false_type{}) : run(D128{}, std::false_type{});
    return rc ? rc : launch_join(s, d, bf16, st);
}
