// prefill_window.cu -- causal attention with a sliding window and a few first tokens that stay
// visible (sinks), forward, sm_103a.
//
// Query row i stands at position p = i + (Sk - Sq) and sees key j iff j <= p and (j < sinks or
// j > p - window); out_i = softmax_j(q_i . k_j / sqrt(d)) v_j over those keys, 0 where there is none.
//
// Both products are tensor-core work: 4 d operations a visible pair, against which the reads are
// small as long as a K/V tile serves many rows.  One CTA per SM therefore takes two 128-row query
// tiles that see (nearly) the same keys, two query heads of a kv head at the same rows or, where
// heads do not pair up, two neighbouring row blocks of a head, and runs them against one stream of
// 128-key K/V tiles: half the L2 traffic of one tile a CTA, and while the softmax of one query tile
// works the tensor core has the other's products.  With no more query tiles than SMs both are the same
// tile instead, each over every second of its key tiles, without turns; their O and sums are joined at the
// end.
//     S_x = Q_x K^T    tcgen05.mma M=128 N=128 K=d, fp32 in TMEM (N = 128: both operands' shared
//                      memory reads then take no longer than the products themselves)
//     P_x              exp2 online softmax, one thread a row, written over S_x as the 16-bit type
//     O_x += P_x V     tcgen05.mma M=128 N=d K=128, A = P_x from TMEM
// The row maximum used is raised, and O_x rescaled, only when it grows by more than 2^8: weights stay
// below 2^8 and the sum and O share the reference, so nothing is lost.  P is rounded to the input
// type (the products of kind::f16 take one type); statistics, sums and O are 32-bit.
//
// 384 threads:
//   warps 0-3 / 4-7   softmax and epilogue of query tile 0 / 1 (TMEM lane = row)
//   warps 8 / 9       issue the products of query tile 0 / 1, P V(j) and S(j + 1) in turn, j counting on
//                     from one item to the next.  One issuer's products run in order: S(j + 1) may
//                     overwrite P(j) without a wait
//   warp 10           TMA: Q tiles, then K and V tiles through one ring of stages (warp 11 idles)
// P is handed over in two halves of 64 keys, so that half of P V runs under the rest of the softmax.
// The two issuers take turns, a P V and an S each, which keeps the query tiles half a period apart, one's
// softmax under the other's products; left alone they fall into step and stay there (4500 cycles a round).
// All other waits of an issuer come before the one for P, where they overlap the softmax.
//
// What bounds it, d = 128: the tensor core, in use 67 % of the time (the rest is the hand-over from S to P
// and back, in part under the other query tile's products).  32 heads over 8 kv heads, 16384 tokens, window
// 4096, bf16: 660 us, 1459 TFLOP/s, in short runs, 700 us when run for seconds.
// d = 64: one query tile's chain.  P is written over S, so its next S comes after its P V: S, hand-over,
// softmax, hand-over and P V follow one another, and only the other query tile's chain runs beside them.  A
// round (a key tile of both) takes some 2700 cycles against 1024 of products (4 x 16 heads, 8191 tokens,
// window 1024, fp16: 210 us, 616 TFLOP/s; the busiest CTA has 14 items and 144 rounds).  Clock stamps, which
// stretch a round to 3200, find of the 3560 cycles from one tile of a warp to its next: 870 waiting for S,
// 300 TMEM loads, 450 masking (250 where nothing is masked), 300 maximum, 1120 exponentials and P, 520 for
// the change of items.  Without sinks, which cost a whole key tile of 11 there, it takes 178 us for 202 (N(0, 1)
// inputs).  S of the next item under the epilogue and the next item worked out while the last P V runs took
// 220 us to 213, the look at O for NaN 213 to 216.
//
// TMEM: S_0 0-127, S_1 128-255, O_0 256.., O_1 256 + d...  Items are dealt out round-robin, last
// rows first (they see the most keys), so CTAs at work at one time share K/V in L2.  Every wait is
// bounded: on expiry the CTA records BSATTN_ERR_TIMEOUT, drains what is in flight and leaves.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "host_internal.h"
#include "ptx.cuh"
#include "strided.h"

namespace bsattn {
namespace {

constexpr int kThreads = 384;
constexpr int kMmaWarp = 8;              // and 9
constexpr int kLoadWarp = 10;
constexpr int kRegsSoftmax = 208, kRegsOther = 88;       // registers a thread: two warpgroups, and the third
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kOCol = 256;
constexpr float kRescaleLog2 = 8.0f;

template <int D>
struct Cfg {
    static constexpr int kStages = D == 64 ? 10 : 5;             // one 128-row tile of K or V each
    static constexpr uint32_t kTile = 128 * D * 2;
    static constexpr uint32_t kQ = 0;                            // two query tiles
    static constexpr uint32_t kKV = 2 * kTile;
    static constexpr uint32_t kBars = kKV + kStages * kTile;
    // q_full[2] q_free[2] full[stages] empty[stages] s_full[2] p_half[2] p_full[2] o_full[2] o_free[2] fin[2] turn[2] joined
    static constexpr uint32_t kNumBars = 4 + 2 * kStages + 15;
    static constexpr uint32_t kMisc = (kBars + 8 * kNumBars + 15) & ~15u;   // tmem base, abort flag
    static constexpr uint32_t kHalf = kMisc + 16;                // (m, l) of query tile 1's rows
    static constexpr uint32_t kBytes = 1024 + kHalf + 128 * 8;
    static_assert(kBytes <= 227 * 1024, "shared memory");
};

// What the two query tiles of an item are: two heads of a kv head at the same rows, two neighbouring row
// blocks of a head, or one tile whose keys are shared out between them.  (The last has kernels of its own:
// decided at run time it would cost the other two 2 % at d = 64.)
enum Pairing { kHeads, kRows, kSplit };

struct WindowParams {
    void* out;
    int* status;
    long long out_b, out_h, out_s;       // element strides of out
    const void* q;                       // what the tensor maps show, for rows that are worked out again
    const void* k;
    const void* v;
    long long q_b, q_h, q_s, k_b, k_h, k_s, v_b, v_h, v_s;
    int B, Hq, Hkv, Sq, Sk;
    int window, sinks;
    int nq;                              // 128-row query blocks
    int pairing;                         // what an item's two query tiles are
    int pairs;                           // items per (batch, item row): head pairs, or heads
    int rows;                            // item rows: row blocks, or pairs of them
    int total_items, sms;
    float scale_log2;
    unsigned long long budget_ns;
};

__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int c0, int c1,
                                            int c2, int c3) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
        : "memory");
}

__device__ __forceinline__ float max3f(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

__device__ __forceinline__ float2 fma2f(float2 a, float2 b, float2 c) {
    unsigned long long ra, rb, rc, rd;
    asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(rc) : "f"(c.x), "f"(c.y));
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(rd) : "l"(ra), "l"(rb), "l"(rc));
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
    return d;
}

__device__ __forceinline__ float2 add2f(float2 a, float2 b) {
    unsigned long long ra, rb, rd;
    asm("mov.b64 %0, {%1, %2};" : "=l"(ra) : "f"(a.x), "f"(a.y));
    asm("mov.b64 %0, {%1, %2};" : "=l"(rb) : "f"(b.x), "f"(b.y));
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(rd) : "l"(ra), "l"(rb));
    float2 d;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(d.x), "=f"(d.y) : "l"(rd));
    return d;
}

template <bool BF16>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (BF16) {
        __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
    } else {
        __half2 v = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&v);
    }
}

// 32 TMEM lanes x 32 columns, one accumulator row a thread.
__device__ __forceinline__ void tmem_ld_row32(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),
          "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),
          "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]),
          "=r"(r[31])
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_row32(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st_row16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
        ::"r"(taddr), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]),
        "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}

// A value that is the same in all lanes, in a form the compiler knows to be so: descriptors and TMEM
// addresses made from it stay in uniform registers.  An MMA then takes one issue slot or two instead of a
// dozen, which decides its rate when the softmax warps contend for the slots: 64 cycles an M128 N128 K16
// MMA against 71 alone and 110 beside a warp that issues every cycle.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ uint64_t uniform(uint64_t v) {
    return static_cast<uint64_t>(uniform(static_cast<uint32_t>(v >> 32))) << 32 | uniform(static_cast<uint32_t>(v));
}

// D[tmem] (+)= A[tmem] * B[smem], kind::f16, by one lane of a converged warp under a guard predicate.
__device__ __forceinline__ void mma_f16_ts_if(bool lead, uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                              uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(lead ? 1u : 0u)
        : "memory");
}

// The 128-key tiles one query tile visits: [0, sink) and [lo, hi); hi = 0: none.
struct Tiles {
    int head, qb;          // query head, row block (past the last one: no rows)
    int lo, hi, sink;
    __device__ __forceinline__ int tile(int i) const { return i < sink ? i : lo + (i - sink); }
    __device__ __forceinline__ int count() const { return hi > 0 ? sink + hi - lo : 0; }
};

// One item: the two query tiles and the tiles their union visits.  SPLIT: both are one query tile, which
// visits that union, tile 0 the even positions in it and tile 1 the odd ones.
template <bool SPLIT>
struct Item {
    int b, kvh;
    Tiles x[2], both;
    __device__ __forceinline__ int count() const { return both.count(); }
    __device__ __forceinline__ int tile(int i) const { return both.tile(i); }
    __device__ __forceinline__ int count(int w) const {
        if (SPLIT) return (both.count() + 1 - w) / 2;
        return w ? x[1].count() : x[0].count();
    }
    // whether query tile w visits position i, which holds tile t
    __device__ __forceinline__ bool has(int w, int i, int t) const {
        if (SPLIT) return (i & 1) == w;
        const Tiles& me = w ? x[1] : x[0];
        return t < me.hi && (t < me.sink || t >= me.lo);
    }
    // position of the m-th tile of query tile w, which is t
    __device__ __forceinline__ int at(int w, int m, int t) const {
        if (SPLIT) return 2 * m + w;
        return t < both.sink ? t : both.sink + t - both.lo;
    }
};

__device__ __forceinline__ Tiles tiles_of(const WindowParams& p, int head, int qb) {
    Tiles x;
    x.head = head;
    x.qb = qb;
    x.lo = x.hi = x.sink = 0;
    if (qb < p.nq) {
        const int past = p.Sk - p.Sq;
        const int first = qb * 128 + past, last = min(qb * 128 + 127, p.Sq - 1) + past;
        if (last >= 0) {
            const long long low = static_cast<long long>(first) - p.window + 1;
            x.lo = low > 0 ? static_cast<int>(low / 128) : 0;
            x.hi = last / 128 + 1;
            x.sink = min(p.sinks / 128 + (p.sinks % 128 != 0), x.lo);
        }
    }
    return x;
}

template <bool SPLIT>
__device__ __forceinline__ Item<SPLIT> item_of(const WindowParams& p, int t) {
    // last rows first; at a row, all pairs of all batches next to each other
    Item<SPLIT> it;
    const int per_row = p.B * p.pairs;
    const int row = p.rows - 1 - t / per_row;
    const int r = t - (t / per_row) * per_row;
    it.b = r / p.pairs;
    const int pair = r - it.b * p.pairs;
    const int group = p.Hq / p.Hkv;
    if (!SPLIT && p.pairing == kHeads) {
        it.kvh = 2 * pair / group;
        it.x[0] = tiles_of(p, 2 * pair, row);
        it.x[1] = it.x[0];
        it.x[1].head = 2 * pair + 1;
        it.both = it.x[0];
    } else if (!SPLIT) {
        it.kvh = pair / group;
        it.x[0] = tiles_of(p, pair, 2 * row);
        it.x[1] = tiles_of(p, pair, 2 * row + 1);
        // the second block is the later one: its keys start and end no earlier
        it.both = it.x[0].hi > 0 ? it.x[0] : it.x[1];
        it.both.hi = max(it.x[0].hi, it.x[1].hi);
    } else {
        it.kvh = pair / group;
        it.both = it.x[0] = it.x[1] = tiles_of(p, pair, row);
    }
    return it;
}

// P V takes all 128 keys of a tile, those that a row does not see with weight 0, and 0 times an infinity or
// a NaN is NaN.  Where V holds one in a tile that a row sees in part, rows come out NaN that do not see it.
// Those are found by their O and worked out again by a warp, 16 rows at a time, m and 1 / l being known, with such
// values taken for 0; a row that does see one is left as it is.  Keys are taken from the last one back, as a
// padded end, where all rows see such values, is then done with at once.  (Looking V over before the product
// instead, in partly seen tiles alone, cost calls without any 8 to 24 %; the look at O costs 1 to 3 %.  4 x 16
// heads of 8191 tokens, window 1024, N(0, 1) inputs, V's last 1000 all NaN: 448 us against 202.)
template <bool BF16>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (BF16) {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    } else {
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}

__device__ __forceinline__ uint32_t below(int n) { return n >= 32 ? 0xffffffffu : (n <= 0 ? 0u : (1u << n) - 1u); }

// Visits the steps of 16 keys that rows row0 .. row0 + 15 see some of, the last one first, until f is false.
template <typename F>
__device__ __forceinline__ void key_steps(const WindowParams& p, int row0, F f) {
    const int at = row0 + p.Sk - p.Sq, first = at >= p.window ? at - p.window + 1 : 0;
    const int near = first / 16, sink = min(p.sinks / 16 + (p.sinks % 16 != 0), near);
#pragma unroll 1
    for (int st = min(at + 15, p.Sk - 1) / 16; st >= 0; --st) {
        if (st < near && st >= sink) st = sink - 1;
        if (st < 0 || !f(16 * st)) break;
    }
}

// Which of 16 keys from key0 on the row at `pos` sees.
__device__ __forceinline__ uint32_t seen_of(const WindowParams& p, int pos, int key0) {
    const int lo = pos >= p.window ? pos - p.window + 1 : 0;
    return below(pos + 1 - key0) & (~below(lo - key0) | below(p.sinks - key0)) & 0xffffu;
}

// Of the rows row0 + r with bit r in `want`, those that see no infinity or NaN in V.
template <int D, bool BF16>
__device__ __noinline__ uint32_t unmet_rows(const WindowParams& p, int b, int head, int row0, uint32_t want) {
    constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
    const int lane = threadIdx.x & 31;
    const uint16_t* v = static_cast<const uint16_t*>(p.v) + b * p.v_b + head / (p.Hq / p.Hkv) * p.v_h + D / 2 * (lane & 1);
    const int pos = row0 + (lane & 15) + p.Sk - p.Sq;
    key_steps(p, row0, [&](int key0) {
        // two lanes a key
        const uint4* row = reinterpret_cast<const uint4*>(v + min(key0 + (lane >> 1), p.Sk - 1) * p.v_s);
        bool bad = false;
#pragma unroll
        for (int e = 0; e < D / 16; ++e) {
            const uint4 w = row[e];
            const uint32_t w4[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) bad = bad || (w4[c] & kExp) == kExp || (w4[c] >> 16 & kExp) == kExp;
        }
        const uint32_t lanes = __ballot_sync(0xffffffffu, bad);
        if (lanes != 0u) {
            uint32_t keys = 0;
            for (int e = 0; e < 16; ++e) keys |= (lanes >> (2 * e) & 3u ? 1u : 0u) << e;
            want &= ~__ballot_sync(0xffffffffu, (seen_of(p, pos, key0) & keys) != 0u);
        }
        return want != 0u;
    });
    return want;
}

// Rows row0 + r with bit r in `want`; m and inv are of the lane's row, and row0 is lane `lane0`'s.
template <int D, bool BF16>
__device__ __noinline__ void mend_rows(const WindowParams& p, int b, int head, int row0, int lane0, uint32_t want,
                                           float m, float inv) {
    const int lane = threadIdx.x & 31, r = lane >> 2, j = lane & 3, kvh = head / (p.Hq / p.Hkv);
    const uint16_t* q = static_cast<const uint16_t*>(p.q) + b * p.q_b + head * p.q_h;
    const uint16_t* k = static_cast<const uint16_t*>(p.k) + b * p.k_b + kvh * p.k_h;
    const uint16_t* v = static_cast<const uint16_t*>(p.v) + b * p.v_b + kvh * p.v_h;
    // a lane has rows r and r + 8 of the products
    const float m0 = __shfl_sync(0xffffffffu, m, lane0 + r), m1 = __shfl_sync(0xffffffffu, m, lane0 + r + 8);
    const float inv0 = __shfl_sync(0xffffffffu, inv, lane0 + r), inv1 = __shfl_sync(0xffffffffu, inv, lane0 + r + 8);
    const int pos0 = row0 + r + p.Sk - p.Sq, pos1 = pos0 + 8;
    uint32_t qa[D / 16][4];
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            qa[kk][e] = *reinterpret_cast<const uint32_t*>(q + min(row0 + r + 8 * (e & 1), p.Sq - 1) * p.q_s + 16 * kk +
                                                           8 * (e >> 1) + 2 * j);
    float o[D / 8][4] = {};
    key_steps(p, row0, [&](int key0) {
        float sc[2][4] = {};
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const uint16_t* kr = k + min(key0 + 8 * t + r, p.Sk - 1) * p.k_s + 2 * j;
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk)
                mma16816<BF16>(sc[t], qa[kk], *reinterpret_cast<const uint32_t*>(kr + 16 * kk),
                               *reinterpret_cast<const uint32_t*>(kr + 16 * kk + 8));
        }
        const uint32_t on0 = seen_of(p, pos0, key0), on1 = seen_of(p, pos1, key0);
        uint32_t pa[4];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int bit = 8 * t + 2 * j;
            pa[2 * t] = pack2<BF16>(on0 >> bit & 1u ? ex2_approx((sc[t][0] - m0) * p.scale_log2) : 0.f,
                                    on0 >> (bit + 1) & 1u ? ex2_approx((sc[t][1] - m0) * p.scale_log2) : 0.f);
            pa[2 * t + 1] = pack2<BF16>(on1 >> bit & 1u ? ex2_approx((sc[t][2] - m1) * p.scale_log2) : 0.f,
                                        on1 >> (bit + 1) & 1u ? ex2_approx((sc[t][3] - m1) * p.scale_log2) : 0.f);
        }
        // keys 2 j, 2 j + 1 and eight further, channels 8 n + r
        const uint16_t* vr[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) vr[e] = v + min(key0 + 2 * j + (e & 1) + 8 * (e >> 1), p.Sk - 1) * p.v_s + r;
        constexpr uint32_t kExp = BF16 ? 0x7f80u : 0x7c00u;
#pragma unroll
        for (int n = 0; n < D / 8; ++n) {
            uint32_t u[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                u[e] = vr[e][8 * n];
                if ((u[e] & kExp) == kExp) u[e] = 0u;
            }
            mma16816<BF16>(o[n], pa, u[0] | u[1] << 16, u[2] | u[3] << 16);
        }
        return true;
    });
    const bool write0 = want >> r & 1u, write1 = want >> (r + 8) & 1u;
    uint16_t* out = static_cast<uint16_t*>(p.out) + b * p.out_b + head * p.out_h + 2 * j;
#pragma unroll
    for (int n = 0; n < D / 8; ++n) {
        if (write0)
            *reinterpret_cast<uint32_t*>(out + (row0 + r) * p.out_s + 8 * n) = pack2<BF16>(o[n][0] * inv0, o[n][1] * inv0);
        if (write1)
            *reinterpret_cast<uint32_t*>(out + (row0 + r + 8) * p.out_s + 8 * n) = pack2<BF16>(o[n][2] * inv1, o[n][3] * inv1);
    }
}

template <int D, bool BF16, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1)
    window_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v, const WindowParams p) {
    using C = Cfg<D>;
    using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
    constexpr int kStages = C::kStages;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sq = sm + C::kQ;
    uint8_t* skv = sm + C::kKV;
    uint64_t* q_full = reinterpret_cast<uint64_t*>(sm + C::kBars);   // [2]
    uint64_t* q_free = q_full + 2;                                    // [2]
    uint64_t* full = q_free + 2;                                      // [stages]
    uint64_t* empty = full + kStages;                                 // [stages] both query tiles
    uint64_t* s_full = empty + kStages;                               // [2]
    uint64_t* p_half = s_full + 2;                                    // [2] four warps: P of the first 64 keys
    uint64_t* p_full = p_half + 2;                                    // [2] four warps
    uint64_t* o_full = p_full + 2;                                    // [2] an item's last P V
    uint64_t* o_free = o_full + 2;                                    // [2] four warps
    uint64_t* fin = o_free + 2;                                       // [2]
    uint64_t* turn = fin + 2;                                         // [2] the other has issued
    uint64_t* joined = turn + 2;                                      // four warps: query tile 1's (m, l)
    int* misc = reinterpret_cast<int*>(sm + C::kMisc);
    float2* half_ml = reinterpret_cast<float2*>(sm + C::kHalf);
    volatile int* abort_flag = &misc[1];
    int* status = p.status;

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // of the waits of an item: a call over long sequences may itself take longer than a wait's budget
    uint64_t deadline = global_timer_ns() + p.budget_ns;

    if (tid == 0) {
        for (int x = 0; x < 2; ++x) {
            mbar_init(&q_full[x], 1);
            mbar_init(&q_free[x], 1);
            mbar_init(&s_full[x], 1);
            mbar_init(&p_half[x], 4);
            mbar_init(&p_full[x], 4);
            mbar_init(&o_full[x], 1);
            mbar_init(&o_free[x], 4);
            mbar_init(&fin[x], 1);
            mbar_init(&turn[x], 1);
        }
        mbar_init(joined, 4);
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

    // The softmax keeps a row of 128 scores a thread: its two warpgroups take 208 of the registers that the
    // launch gave, the third is left 88.  (launch() has checked that the launch gave that many.)
    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
        if (warp == kLoadWarp) {
            // ------------------------------------------------------------ TMA
            if (lane == 0) {
                tma_prefetch_desc(&tm_q);
                tma_prefetch_desc(&tm_k);
                tma_prefetch_desc(&tm_v);
                int g = 0;                                   // tiles loaded, K and V counted apart
                int nq[2] = {0, 0};                          // Q tiles loaded
                bool ok = true;
                auto load = [&](const CUtensorMap* map, int tile, const Item<SPLIT>& it) {
                    const int st = g % kStages;
                    if (g >= kStages && !wait_parity(&empty[st], (g / kStages - 1) & 1, deadline, abort_flag, status))
                        return false;
                    mbar_arrive_expect_tx(&full[st], C::kTile);
                    for (int h = 0; h < D / 64; ++h)
                        tma_load_4d(skv + st * C::kTile + h * 16384, map, &full[st], h * 64, tile * 128, it.kvh, it.b);
                    ++g;
                    return true;
                };
                for (int t = blockIdx.x; ok && t < p.total_items; t += gridDim.x) {
                    const Item<SPLIT> it = item_of<SPLIT>(p, t);
                    deadline = global_timer_ns() + p.budget_ns;
                    const int n = it.count();
                    for (int i = 0; ok && i < n; ++i) {
                        ok = load(&tm_k, it.tile(i), it);
                        if (i == 0) {
                            for (int x = 0; ok && x < 2; ++x) {
                                if (it.count(x) == 0) continue;
                                if (nq[x] > 0 && !wait_parity(&q_free[x], (nq[x] - 1) & 1, deadline, abort_flag, status)) {
                                    ok = false;
                                    break;
                                }
                                mbar_arrive_expect_tx(&q_full[x], C::kTile);
                                for (int h = 0; h < D / 64; ++h)
                                    tma_load_4d(sq + x * C::kTile + h * 16384, &tm_q, &q_full[x], h * 64,
                                                it.x[x].qb * 128, it.x[x].head, it.b);
                                ++nq[x];
                            }
                        }
                        ok = ok && load(&tm_v, it.tile(i), it);
                    }
                }
                if (*abort_flag) {
                    // copies in flight land before the shared memory is released
                    const uint64_t dl = global_timer_ns() + 200000000ull;
                    for (int x = 0; x < 2; ++x)
                        if (nq[x] > 0) wait_parity_drain(&q_full[x], (nq[x] - 1) & 1, dl);
                    for (int j = max(0, g - kStages); j < g; ++j) wait_parity_drain(&full[j % kStages], (j / kStages) & 1, dl);
                }
            }
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
            if constexpr (SPLIT) {
                // One item, key tiles taken alternately: neither query tile waits for the other.  Every stage is
                // waited for in turn, the other's too, which are given back here as they are not read.  V is given
                // back by the product itself: the ring holds no more than five tiles, and the next K tiles
                // wait for its place.
                // Nothing waits for a later tile: K of tile i takes the place of V of tile i - 3 or an earlier
                // one, V that of K of tile i - 2.
                const Item<SPLIT> it = item_of<SPLIT>(p, blockIdx.x);
                const int n = it.count();
                int blk = 0;                                 // S issued
                bool ok = it.count(x) == 0 || warp_wait_parity(&q_full[x], 0, deadline, abort_flag, status);
                for (int i = 0; ok && i < n; ++i) {
                    const int sk = 2 * i % kStages, sv = (2 * i + 1) % kStages;
                    ok = warp_wait_parity(&full[sk], (2 * i / kStages) & 1, deadline, abort_flag, status);
                    if (!ok) break;
                    const bool mine = (i & 1) == x;
                    if (mine) {
                        const uint64_t kb = uniform(k_desc + static_cast<uint32_t>(sk) * kTileDesc);
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                            mma_f16_ss_if(lead, ts, q_desc + off, kb + off, idS, kk > 0 ? 1u : 0u);
                        }
                        mma_commit_if(lead, &s_full[x]);
                        ++blk;
                    } else {
                        mbar_arrive_if(lead, &empty[sk]);
                    }
                    ok = warp_wait_parity(&full[sv], ((2 * i + 1) / kStages) & 1, deadline, abort_flag, status);
                    if (!ok) break;
                    if (!mine) mbar_arrive_if(lead, &empty[sv]);
                    // P V of the last tile of its own, once the other's after it is passed
                    const int own = mine ? i : i - 1;
                    if (own < 0 || (mine && i + 1 < n)) continue;
                    const uint32_t so = static_cast<uint32_t>(2 * own + 1) % kStages;
                    const uint64_t vb = uniform(v_desc + so * kTileDesc);
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        ok = ok && warp_wait_parity(half ? &p_full[x] : &p_half[x], (blk - 1) & 1, deadline, abort_flag, status);
                        if (!ok) break;
                        tc_fence_after();
#pragma unroll
                        for (int kk = 4 * half; kk < 4 * half + 4; ++kk)
                            mma_f16_ts_if(lead, to, ts + 8 * kk, vb + ((kk * 2048) >> 4), idO, (blk > 1 || kk > 0) ? 1u : 0u);
                    }
                    if (!ok) break;
                    if (blk == it.count(x)) mma_commit_if(lead, &o_full[x]);
                    mma_commit_if(lead, &empty[so]);
                }
            } else {
                int g = 0;                                       // ring position: K of tile i of all items' at 2 i, V after it
                int blk = 0, items = 0, outs = 0, rounds = 0;    // tiles, items (S begun, O begun) and rounds so far
                bool pend = false, begins = false, ends = false; // a tile awaits its P V, which begins / ends its O
                bool passed = false;                             // the tile before is not this query tile's
                bool ok = true;
                // One round: P V of the tile before, be it of the item before, and S of the tile at position g, if
                // there is one and this query tile visits it.  A commit takes its turn among the products, so there
                // is only S's and the last P V's: the softmax warps pass on what it says about the stages and Q.
                // Every stage is waited for in turn, visited or not: a parity tells two of its uses apart, no more.
                // A stage that this query tile does not read it gives back here, but only once it is loaded: an arrival
                // before that could count for the stage's use before.
                // None of the waits waits for what comes after its own round: K of position g takes the stage
                // of position g - 5 or an earlier one, which the softmax gave back for a round before.
                auto round = [&](bool tile, bool visit, bool first, bool last) {
                    const int sk = g % kStages;
                    if (g > 0 && !warp_wait_parity(&full[(g - 1) % kStages], ((g - 1) / kStages) & 1, deadline, abort_flag, status))
                        return false;
                    if (passed) mbar_arrive_if(lead, &empty[(g - 1) % kStages]);
                    if (tile && !warp_wait_parity(&full[sk], (g / kStages) & 1, deadline, abort_flag, status)) return false;
                    passed = tile && !visit;
                    if (passed) mbar_arrive_if(lead, &empty[sk]);
                    const uint64_t vb = uniform(v_desc + static_cast<uint32_t>((g + kStages - 1) % kStages) * kTileDesc);
                    const uint64_t kb = uniform(k_desc + static_cast<uint32_t>(sk) * kTileDesc);
                    if (visit && first) {
                        if (!warp_wait_parity(&q_full[x], items & 1, deadline, abort_flag, status)) return false;
                        ++items;
                    }
                    // tile 0's round comes after tile 1's round before, tile 1's after tile 0's
                    if (rounds + x > 0 && !warp_wait_parity(&turn[x], (rounds + x + 1) & 1, deadline, abort_flag, status))
                        return false;
                    ++rounds;
                    if (pend) {
                        if (begins) {
                            if (outs > 0 && !warp_wait_parity(&o_free[x], (outs - 1) & 1, deadline, abort_flag, status))
                                return false;
                            ++outs;
                        }
                        if (!warp_wait_parity(&p_half[x], (blk - 1) & 1, deadline, abort_flag, status)) return false;
                        // the first half of P V runs under the second half of the softmax
                        tc_fence_after();
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_f16_ts_if(lead, to, ts + 8 * kk, vb + ((kk * 2048) >> 4), idO, (!begins || kk > 0) ? 1u : 0u);
                        if (!warp_wait_parity(&p_full[x], (blk - 1) & 1, deadline, abort_flag, status)) return false;
                    }
                    tc_fence_after();
                    if (pend) {
#pragma unroll
                        for (int kk = 4; kk < 8; ++kk)
                            mma_f16_ts_if(lead, to, ts + 8 * kk, vb + ((kk * 2048) >> 4), idO, 1u);
                        if (ends) mma_commit_if(lead, &o_full[x]);
                        pend = false;
                    }
                    if (visit) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t off = ((kk >> 2) * 16384 + (kk & 3) * 32) >> 4;
                            mma_f16_ss_if(lead, ts, q_desc + off, kb + off, idS, kk > 0 ? 1u : 0u);
                        }
                        mma_commit_if(lead, &s_full[x]);
                        ++blk;
                        pend = true;
                        begins = first;
                        ends = last;
                    }
                    mbar_arrive_if(lead, &turn[1 - x]);
                    return true;
                };
                for (int t = blockIdx.x; ok && t < p.total_items; t += gridDim.x) {
                    const Item<SPLIT> it = item_of<SPLIT>(p, t);
                    deadline = global_timer_ns() + p.budget_ns;
                    const int n = it.count(), mine = it.count(x);
                    int done = 0;                                // S issued in this item
                    for (int i = 0; ok && i < n; ++i, g += 2) {
                        const bool visit = it.has(x, i, it.tile(i));
                        ok = round(true, visit, done == 0, done == mine - 1);
                        done += visit;
                    }
                }
                if (ok) {
                    deadline = global_timer_ns() + p.budget_ns;
                    round(false, false, false, false);
                }
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
        const float c = p.scale_log2;
        int blk = 0, items = 0, g = 0;
        bool ok = true;
        Item<SPLIT> it = item_of<SPLIT>(p, blockIdx.x);
        for (int t = blockIdx.x; ok && t < p.total_items; t += gridDim.x) {
            const Tiles me = x ? it.x[1] : it.x[0];
            const int n = it.count(x);
            const int g0 = g;                            // ring position of the item's first K tile
            g += 2 * it.count();
            const bool speaks = (warp & 3) == 0 && lane == 0;
            int v_read = -1;                             // stage of the V tile to give back when it is read
            const int row = me.qb * 128 + lrow;
            const int pos = row + p.Sk - p.Sq;
            T* out = reinterpret_cast<T*>(p.out) + it.b * p.out_b + me.head * p.out_h + row * p.out_s;
            if (n == 0 && !SPLIT) {
                // no key, or (the partner of an odd last row block) no row
                if (row < p.Sq)
                    for (int e = 0; e < D / 8; ++e) reinterpret_cast<uint4*>(out)[e] = make_uint4(0, 0, 0, 0);
                it = item_of<SPLIT>(p, t + gridDim.x);
                deadline = global_timer_ns() + p.budget_ns;
                continue;
            }
            // keys [lo, pos] and, below lo, those before the sinks
            const int lo = pos >= p.window ? pos - p.window + 1 : 0;
            float m_used = -INFINITY, l = 0.f;
            for (int i = 0; i < n; ++i, ++blk) {
                const int tile = SPLIT ? it.tile(2 * i + x) : me.tile(i);
                const int key0 = 128 * tile;
                const int u = it.at(x, i, tile);
                if (!warp_wait_parity(&s_full[x], blk & 1, deadline, abort_flag, status)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                if (speaks) {
                    // S of this tile is there: its K tile has been read, and V of the tile before
                    if (!SPLIT && v_read >= 0) mbar_arrive(&empty[v_read]);
                    const int at = g0 + 2 * u;
                    mbar_arrive(&empty[at % kStages]);
                    v_read = (at + 1) % kStages;
                    if (i == n - 1) mbar_arrive(&q_free[x]);
                }
                __syncwarp();
                float s[128];
#pragma unroll
                for (int h = 0; h < 4; ++h) tmem_ld_row32(ts + 32 * h, reinterpret_cast<uint32_t*>(s) + 32 * h);
                tmem_wait_ld();
                const bool edge = key0 + 127 > pos || (key0 < lo && key0 + 128 > p.sinks);
                if (__any_sync(0xffffffffu, edge)) {
                    // 32 keys at a time, as most of them are visible to all of a warp's rows or to none
#pragma unroll
                    for (int h = 0; h < 4; ++h) {
                        const int k0 = key0 + 32 * h;
                        // bit e: key k0 + e is visible
                        const uint32_t on = below(pos + 1 - k0) & (~below(lo - k0) | below(p.sinks - k0));
                        if (__all_sync(0xffffffffu, on == 0xffffffffu)) continue;
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
                const bool grow = mx * c > m_used * c + kRescaleLog2;
                const float m_new = grow ? mx : m_used;
                const float alpha = grow ? ex2_approx((m_used - m_new) * c) : 1.f;
                const bool rescale = grow && m_used != -INFINITY;
                m_used = m_new;
                const float mc = m_new == -INFINITY ? 0.f : m_new * c;
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
            if (!ok) break;
            // the next item (past the last one: unused) is worked out while the last P V runs
            const Item<SPLIT> after = item_of<SPLIT>(p, t + gridDim.x);
            deadline = global_timer_ns() + p.budget_ns;
            // ---- O / l to memory
            if ((!SPLIT || n > 0) && !warp_wait_parity(&o_full[x], items & 1, deadline, abort_flag, status)) {
                ok = false;
                break;
            }
            if (!SPLIT || n > 0) ++items;
            tc_fence_after();
            if (!SPLIT && speaks) mbar_arrive(&empty[v_read]);
            __syncwarp();
            float scale0 = 1.f, scale1 = 0.f;
            if (SPLIT) {
                // query tile 0's threads join both halves of a row: tile 1's O is in the same TMEM lane.  (A CTA
                // has one item then, so nothing overwrites it.)
                if (x == 1) {
                    half_ml[lrow] = make_float2(m_used, l);
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(joined);
                    continue;
                }
                if (!warp_wait_parity(joined, 0, deadline, abort_flag, status) ||
                    (it.count(1) > 0 && !warp_wait_parity(&o_full[1], 0, deadline, abort_flag, status))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const float2 other = half_ml[lrow];
                const float top = fmaxf(m_used, other.x);
                const float ref = top == -INFINITY ? 0.f : top;
                // a half without a finite score has l = 0, or NaN if it met one: either way it counts
                scale0 = m_used == -INFINITY ? 1.f : ex2_approx((m_used - ref) * c);
                scale1 = other.x == -INFINITY ? 1.f : ex2_approx((other.x - ref) * c);
                l = l * scale0 + other.y * scale1;
                m_used = top;
            }
            const bool two = SPLIT && it.count(1) > 0;
            const float inv = l == 0.f ? 0.f : 1.f / l;         // NaN stays NaN
            uint32_t o[D];
#pragma unroll
            for (int c0 = 0; c0 < D; c0 += 32) tmem_ld_row32(to + c0, o + c0);
            tmem_wait_ld();
            if (SPLIT) {
                if (n == 0) {
#pragma unroll
                    for (int e = 0; e < D; ++e) o[e] = 0u;
                }
                if (two) {
#pragma unroll
                    for (int c0 = 0; c0 < D; c0 += 32) {
                        uint32_t o1[32];
                        tmem_ld_row32(to + D + c0, o1);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            o[c0 + e] = __float_as_uint(__uint_as_float(o[c0 + e]) * scale0 + __uint_as_float(o1[e]) * scale1);
                    }
                }
            }
            // O is in registers: the next item's first P V may overwrite it
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&o_free[x]);
            float2 zero[4] = {};                                // or NaN
#pragma unroll
            for (int e = 0; e < D; e += 2)
                zero[e / 2 & 3] = fma2f(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), make_float2(0.f, 0.f), zero[e / 2 & 3]);
            const float2 sum = add2f(add2f(zero[0], zero[1]), add2f(zero[2], zero[3]));
            // (a NaN in l is the row's own: of a score)
            const uint32_t rows = __ballot_sync(0xffffffffu, sum.x + sum.y != 0.f && l > 0.f && row < p.Sq);
            uint32_t mend = 0u;
#pragma unroll 1
            for (int at = 0; rows != 0u && at < 32; at += 16)
                if (rows >> at & 0xffffu) mend |= unmet_rows<D, BF16>(p, it.b, me.head, row - lane + at, rows >> at & 0xffffu) << at;
            if (row < p.Sq && !(mend >> lane & 1u)) {
#pragma unroll
                for (int c0 = 0; c0 < D; c0 += 8) {
                    uint32_t ob[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        ob[e] = l == 0.f ? 0u : pack2<BF16>(__uint_as_float(o[c0 + 2 * e]) * inv, __uint_as_float(o[c0 + 2 * e + 1]) * inv);
                    reinterpret_cast<uint4*>(out)[c0 / 8] = make_uint4(ob[0], ob[1], ob[2], ob[3]);
                }
            }
#pragma unroll 1
            for (int at = 0; mend != 0u && at < 32; at += 16)
                if (mend >> at & 0xffffu)
                    mend_rows<D, BF16>(p, it.b, me.head, row - lane + at, at, mend >> at & 0xffffu, m_used, inv);
            it = after;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        tc_fence_after();
        tmem_dealloc(tbase, kTmemCols);
    }
}

// Strides (elements) of a [B, H, S, d] tensor as a tensor map wants them: a dimension of one entry may
// carry any stride, so it gets one that is always valid.  False: not a layout the map can hold.
bool map_strides(const int64_t* st, int B, int H, int S, int d, uint64_t (&bytes)[3]) {
    const int64_t in[3] = {st[2], st[1], st[0]};         // rows, heads, batches
    const int n[3] = {S, H, B};
    for (int i = 0; i < 3; ++i) {
        if (n[i] == 1) {
            bytes[i] = static_cast<uint64_t>(d) * 2;
            continue;
        }
        if (in[i] <= 0 || (in[i] & 7) || in[i] >= (int64_t(1) << 38)) return false;
        bytes[i] = static_cast<uint64_t>(in[i]) * 2;
    }
    return true;
}

template <int D, bool BF16, bool SPLIT>
int launch(const void* q, const void* k, const void* v, const int64_t (&st)[12], const WindowParams& prm,
           cudaStream_t stream) {
    uint64_t qs[3], ks[3], vs[3];
    const int sk = prm.Sk > 0 ? prm.Sk : 1, hk = prm.Sk > 0 ? prm.Hkv : 1, bk = prm.Sk > 0 ? prm.B : 1;
    if (!map_strides(st, prm.B, prm.Hq, prm.Sq, D, qs) || !map_strides(st + 3, bk, hk, sk, D, ks) ||
        !map_strides(st + 6, bk, hk, sk, D, vs))
        return BSATTN_ERR_INVALID_ARG;
    CUtensorMap tq, tk, tv;
    const uint64_t dq[4] = {D, uint64_t(prm.Sq), uint64_t(prm.Hq), uint64_t(prm.B)};
    const uint64_t dk[4] = {D, uint64_t(sk), uint64_t(hk), uint64_t(bk)};
    const uint32_t box[4] = {64, 128, 1, 1};
    int rc = encode_4d(&tq, q, BF16, dq, qs, box);
    if (!rc) rc = encode_4d(&tk, k, BF16, dk, ks, box);
    if (!rc) rc = encode_4d(&tv, v, BF16, dk, vs, box);
    if (rc) return rc;
    auto kern = window_kernel<D, BF16, SPLIT>;
    static std::atomic<unsigned long long> raised{0};
    rc = raise_smem_limit(reinterpret_cast<const void*>(kern), Cfg<D>::kBytes, raised);
    if (rc) return rc;
    // the warpgroups' register shares come out of the launch's: with fewer, the larger ones would never come
    static const bool enough = [kern] {
        cudaFuncAttributes a{};
        return cudaFuncGetAttributes(&a, kern) == cudaSuccess &&
               a.numRegs * kThreads >= 128 * (2 * kRegsSoftmax + kRegsOther);
    }();
    if (!enough) return BSATTN_ERR_CUDA;
    const int grid = prm.total_items < prm.sms ? prm.total_items : prm.sms;
    kern<<<static_cast<unsigned>(grid), kThreads, Cfg<D>::kBytes, stream>>>(tq, tk, tv, prm);
    return cudaGetLastError() == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

}  // namespace
}  // namespace bsattn

extern "C" int bsattn_prefill_window(const void* q, const void* k, const void* v, int window, int sinks,
                                     void* out, int B, int Hq, int Hkv, int Sq, int Sk, int d,
                                     const int64_t* strides, bsattn_dtype dtype, void* workspace,
                                     size_t workspace_bytes, void* stream) {
    using namespace bsattn;
    if (B < 0 || Hq <= 0 || Hkv <= 0 || Sq < 0 || Sk < 0 || window < 1 || sinks < 0) return BSATTN_ERR_INVALID_ARG;
    if (Hq % Hkv) return BSATTN_ERR_INVALID_ARG;
    if (d != 64 && d != 128) return BSATTN_ERR_UNSUPPORTED;
    if (dtype != BSATTN_F16 && dtype != BSATTN_BF16) return BSATTN_ERR_UNSUPPORTED;
    if (!workspace || workspace_bytes < 256 || !aligned16(workspace)) return BSATTN_ERR_INVALID_ARG;
    if (B == 0 || Sq == 0) return BSATTN_OK;
    if (!q || !out || !aligned16(q) || !aligned16(out)) return BSATTN_ERR_INVALID_ARG;
    if (Sk > 0 && (!k || !v || !aligned16(k) || !aligned16(v))) return BSATTN_ERR_INVALID_ARG;
    if (Sq > (1 << 30) || Sk > (1 << 30)) return BSATTN_ERR_UNSUPPORTED;
    int64_t st[12];
    if (strides) {
        for (int i = 0; i < 12; ++i) st[i] = strides[i];
    } else {
        const int64_t H[4] = {Hq, Hkv, Hkv, Hq}, S[4] = {Sq, Sk, Sk, Sq};
        for (int i = 0; i < 4; ++i) {
            st[3 * i] = H[i] * S[i] * d;
            st[3 * i + 1] = S[i] * d;
            st[3 * i + 2] = d;
        }
    }
    // out is written with 16-byte stores while other CTAs still read q, k and v: its rows must not share
    // memory with one another, with k or v, or with q unless it is q itself (a row block of q has been read
    // when its outputs are written)
    const int64_t on[3] = {B, Hq, Sq};
    for (int i = 0; i < 3; ++i)
        if (on[i] > 1 && (st[9 + i] < d || (st[9 + i] & 7))) return BSATTN_ERR_INVALID_ARG;
    const auto tensor = [&](const void* base, int heads, int rows, int at) {
        return Strided{base, {B, heads, rows}, {st[at], st[at + 1], st[at + 2]}};
    };
    const Strided to = tensor(out, Hq, Sq, 9), from[3] = {tensor(q, Hq, Sq, 0), tensor(k, Hkv, Sk, 3), tensor(v, Hkv, Sk, 6)};
    if (overlaps_itself(to, d)) return BSATTN_ERR_INVALID_ARG;
    for (int i = 0; i < (Sk > 0 ? 3 : 1); ++i) {
        for (int e = 0; e < 3; ++e)
            if (from[i].n[e] > 1 && from[i].stride[e] <= 0) return BSATTN_ERR_INVALID_ARG;
        if (!(i == 0 && to.same_as(from[0])) && overlap(to, from[i], d)) return BSATTN_ERR_INVALID_ARG;
    }
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    WindowParams prm{};
    prm.out = out;
    prm.q = q;
    prm.k = k;
    prm.v = v;
    const auto stride = [&](int at, int entries) -> long long { return entries > 1 ? st[at] : 0; };
    prm.q_b = stride(0, B);
    prm.q_h = stride(1, Hq);
    prm.q_s = stride(2, Sq);
    prm.k_b = stride(3, B);
    prm.k_h = stride(4, Hkv);
    prm.k_s = stride(5, Sk);
    prm.v_b = stride(6, B);
    prm.v_h = stride(7, Hkv);
    prm.v_s = stride(8, Sk);
    prm.status = status_word(workspace);
    prm.out_b = stride(9, B);
    prm.out_h = stride(10, Hq);
    prm.out_s = stride(11, Sq);
    prm.B = B;
    prm.Hq = Hq;
    prm.Hkv = Hkv;
    prm.Sq = Sq;
    prm.Sk = Sk;
    prm.window = window;
    prm.sinks = sinks;
    prm.nq = (Sq + 127) / 128;
    // Where there is an SM for every query tile, both tiles of a CTA are the same one, each with half of its
    // keys (257 rows of 8 heads after 8192 cached tokens, window 1024: 15.5 us against 23.7).
    int sms = num_sms_of_current_device();
    if (sms <= 0) sms = 148;
    if (static_cast<long long>(B) * Hq * prm.nq <= sms) {
        prm.pairing = kSplit;
        prm.pairs = Hq;
        prm.rows = prm.nq;
    } else if ((Hq / Hkv) % 2 == 0) {
        prm.pairing = kHeads;
        prm.pairs = Hq / 2;
        prm.rows = prm.nq;
    } else {
        prm.pairing = kRows;
        prm.pairs = Hq;
        prm.rows = (prm.nq + 1) / 2;
    }
    const long long items = static_cast<long long>(B) * prm.pairs * prm.rows;
    if (items > 0x3fffffffLL) return BSATTN_ERR_UNSUPPORTED;
    prm.total_items = static_cast<int>(items);
    prm.sms = sms;
    prm.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
    prm.budget_ns = wait_budget_ns();
    if (Sk == 0) k = v = q;                     // no row sees a key: K and V are not read, only mapped
    const bool bf16 = dtype == BSATTN_BF16;
    const auto run = [&](auto dim, auto split) {
        constexpr int D = decltype(dim)::value;
        constexpr bool SPLIT = decltype(split)::value;
        return bf16 ? launch<D, true, SPLIT>(q, k, v, st, prm, cs) : launch<D, false, SPLIT>(q, k, v, st, prm, cs);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (prm.pairing == kSplit) return d == 64 ? run(D64{}, std::true_type{}) : run(D128{}, std::true_type{});
    return d == 64 ? run(D64{}, std::false_type{}) : run(D128{}, std::false_type{});
}
