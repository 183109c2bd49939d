// decode_shared.cuh -- what the kernels of a decode over shared prefixes know of a call, and where its pieces lie:
// decode_shared.cu makes them (those of the sequences' own tokens by decode_shared_own.cuh), decode_shared_join.cu
// joins them.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "bsattn.h"

namespace bsattn {

constexpr int kSharedThreads = 384;

// A piece is the result over some keys: for each of its rows O / l (fp32) and the base-2 log-sum-exp, -infinity
// where the row has met no finite score (O is not written then, or is 0).
//
// Prefixes.  Sequences starts[p] .. starts[p + 1] - 1 share prefix p.  `side` kv heads and `deep` times up to `seqs`
// sequences are worked side by side at the same keys, by CTAs of their own, the lanes.  An item is up to `seqs`
// sequences and one kv head, those of a lane: a multiple of `deep` or `side` on from the lane's first.  A unit is 128
// keys of an item.  A lane's units, in the order prefix, sequences, kv heads, keys, are cut into equal parts, one a CTA.
// What part c has of an item is a piece; its row r stands at
//     c * part_rows + (the lane's rows of all items before) + r
// of the lane's, or twice as far apart where `halves`: a piece is then two, of every second key tile each.  (Going
// from a piece to the next one moves on by the item's rows or by part_rows, which is no less, or by both: no two
// share a place.)
//
// Own tokens.  A unit is 32 keys of a sequence.  The units of all sequences, end to end, are cut into equal parts,
// one a (warp, kv head).  What part c has of sequence b is a piece at c + b: [kv head][its query heads].
struct SharedCall {
    const void* q;
    void* out;
    const int32_t* starts;       // [P + 1]
    const int32_t* prefix_lens;  // [P]
    const int32_t* own_lens;     // [B]
    const int32_t* prefix_table; // [P, prefix_pages]
    const int32_t* own_table;    // [B, own_pages]
    long long* prefix_info;      // [0] units of a part; [1 + p] units before prefix p
    long long* own_info;         // [0] units of a part; [1 + b] units before sequence b
    float* prefix_lse;
    float* prefix_o;
    float* own_lse;
    float* own_o;
    int* status;
    int B, P, Hq, Hkv;
    int seqs, part_rows, halves;
    long long lane_rows;         // of all pieces of a lane
    int side, deep;
    int page_size, num_pages, prefix_pages, own_pages;
    int prefix_room, own_room;   // tokens that a table has room for
    float scale_log2;
    unsigned long long budget_ns;
};

struct PrefixGroup {
    int start, n;                // sequences
    int len, tiles;              // keys
    bool bad;
};

// Entries out of range are cut to what there can be, and reported.
__device__ __forceinline__ PrefixGroup prefix_group(const SharedCall& s, int p) {
    PrefixGroup g;
    const int from = s.starts[p], to = s.starts[p + 1], len = s.prefix_lens[p];
    g.bad = from < 0 || to < from || to > s.B || len < 0 || len > s.prefix_room || (p == 0 && from != 0) ||
            (p == s.P - 1 && to != s.B);
    g.start = max(min(from, s.B), 0);
    g.n = max(max(min(to, s.B), 0) - g.start, 0);
    g.len = max(min(len, s.prefix_room), 0);
    g.tiles = g.len / 128 + (g.len % 128 != 0);
    return g;
}

__device__ __forceinline__ long long prefix_units(const SharedCall& s, const PrefixGroup& g) {
    const int times = (g.n + s.seqs - 1) / s.seqs;
    return static_cast<long long>((times + s.deep - 1) / s.deep) * (s.Hkv / s.side) * g.tiles;
}

// Where part c's rows of an item (the t-th sequences of a group, kv head h) begin, and how many there are.
__device__ __forceinline__ long long prefix_place(const SharedCall& s, const PrefixGroup& g, int c, int t, int h, int& rows) {
    const int G = s.Hq / s.Hkv, lane = t % s.deep * s.side + h % s.side, along = s.Hkv / s.side;
    rows = min(s.seqs, g.n - t * s.seqs) * G;
    // (there is one prefix only where deep > 1)
    const long long before = (s.deep > 1 ? 0LL : g.start) + t / s.deep * s.seqs;
    return (lane * s.lane_rows + static_cast<long long>(c) * s.part_rows + before * G * along +
            static_cast<long long>(h / s.side) * rows) *
           (s.halves ? 2 : 1);
}

__device__ __forceinline__ int own_len(const SharedCall& s, int b) { return max(min(s.own_lens[b], s.own_room), 0); }
__device__ __forceinline__ int own_units(int len) { return len / 32 + (len % 32 != 0); }

// The launch of decode_shared_join.cu, second on the stream.
int launch_join(const SharedCall& call, int d, bool bf16, cudaStream_t stream);

}  // namespace bsattn
