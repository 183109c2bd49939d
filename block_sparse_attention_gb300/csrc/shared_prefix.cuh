// shared_prefix.cuh -- where the results over shared prefixes lie, for the kernel that makes them
// (decode_shared.cu) and the one that joins them with each sequence's own tokens (decode_stream.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "bsattn.h"

namespace bsattn {

// Sequences starts[p] .. starts[p + 1] - 1 share prefix p.  An item is a kv head's query rows of up to `seqs`
// of them; a unit is 128 keys of an item.  The units of all items, in the order prefix, sequences, kv head,
// keys, are cut into equal parts, one a CTA.  What part c has of an item is a piece of it: a row each of
// O / l and log2-sum-exp, at
//     (c * part_rows + rows of all items before + row)          twice as far apart where `halves`: a piece is
// then two, of every second key tile.  (Going from a piece to the next one moves on by the item's rows or by
// part_rows, which is no less, or by both: no two share a place.)
struct PrefixPieces {
    const int32_t* starts;       // [P + 1]
    const int32_t* lens;         // [P]
    long long* info;             // [0] units of a part; [1 + p] units before prefix p
    float* lse;
    float* o;
    int P, B, Hq, Hkv, seqs;
    int room;                    // tokens that a prefix's table has room for
    int part_rows;               // seqs * Hq / Hkv
    int halves;
    long long rows;              // places there are
};

struct PrefixGroup {
    int start, n;                // sequences
    int len, tiles;              // keys
    bool bad;
};

// Entries out of range are cut to what there can be, and reported.
__device__ __forceinline__ PrefixGroup prefix_group(const PrefixPieces& s, int p) {
    PrefixGroup g;
    const int from = s.starts[p], to = s.starts[p + 1], len = s.lens[p];
    g.bad = from < 0 || to < from || to > s.B || len < 0 || len > s.room || (p == 0 && from != 0) ||
            (p == s.P - 1 && to != s.B);
    g.start = max(min(from, s.B), 0);
    g.n = max(max(min(to, s.B), 0) - g.start, 0);
    g.len = max(min(len, s.room), 0);
    g.tiles = g.len / 128 + (g.len % 128 != 0);
    return g;
}

__device__ __forceinline__ long long prefix_units(const PrefixPieces& s, const PrefixGroup& g) {
    return static_cast<long long>((g.n + s.seqs - 1) / s.seqs) * s.Hkv * g.tiles;
}

// Rows of all items before item (sequences t, kv head h) of a group, and the item's own.
__device__ __forceinline__ long long prefix_rows_before(const PrefixPieces& s, const PrefixGroup& g, int t, int h, int& rows) {
    rows = min(s.seqs, g.n - t * s.seqs) * (s.Hq / s.Hkv);
    return (static_cast<long long>(g.start) + static_cast<long long>(t) * s.seqs) * s.Hq + static_cast<long long>(h) * rows;
}

// The arguments of a stream decode over a 16-bit paged cache.
struct StreamCall {
    const void* q;
    const void* k;
    const void* v;
    const int32_t* seqlens;
    const int32_t* table;
    void* out;
    int B, Hq, Hkv, num_pages, page_size, max_pages, d;
    bsattn_dtype dtype;
    void* workspace;
    size_t workspace_bytes;
};

// The sequences' own tokens, joined with what the kernel launched before it on the stream has written to `pieces`;
// with `check`, nothing but the checks of its arguments.  (decode_stream.cu)
int decode_stream_shared(const StreamCall& call, const PrefixPieces& pieces, bool check, cudaStream_t stream);

}  // namespace bsattn
