// decode_shared.cuh -- what the kernels of a decode over shared prefixes know of a call, and where its pieces lie:
// decode_shared.cu makes those of the prefixes, decode_shared_own.cu those of the sequences' own tokens, and joins.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "bsattn.h"

namespace bsattn {

// A piece is the result over some keys: for each of its rows O / l (fp32) and the base-2 log-sum-exp, -infinity
// where the row has met no finite score (O is not written then, or is 0).
//
// Prefixes.  Sequences starts[p] .. starts[p + 1] - 1 share prefix p.  A CTA's kv head is its lane among `side` kv
// heads side by side, plus a multiple of `side`.  An item is up to `seqs` sequences and one such multiple; a unit is
// 128 keys of an item.  The units of all items, in the order prefix, sequences, kv heads, keys, are cut into equal
// parts, one a (CTA, lane).  What part c has of an item is a piece; its row r stands at
//     c * part_rows + (the lane's rows of all items before) + r
// of the lane's, or twice as far apart where `halves`: a piece is then two, of every second key tile each.  (Going
// from a piece to the next one moves on by the item's rows or by part_rows, which is no less, or by both: no two
// share a place.)
//
// Own tokens.  A unit is 32 keys of a sequence.  The units of all sequences, end to end, are cut into equal parts,
// one a (warp, kv head).  What part c has of sequence b is a piece at c + b: [kv head][its query heads].
struct SharedCall {
    const void* q;
    const void* k;
    const void* v;
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
    int side, prefix_parts, own_parts;
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
    return static_cast<long long>((g.n + s.seqs - 1) / s.seqs) * (s.Hkv / s.side) * g.tiles;
}

// Where part c's rows of an item (the t-th sequences of a group, kv head h) begin, and how many there are.
__device__ __forceinline__ long long prefix_place(const SharedCall& s, const PrefixGroup& g, int c, int t, int h, int& rows) {
    const int G = s.Hq / s.Hkv, lane = h % s.side, along = s.Hkv / s.side;
    rows = min(s.seqs, g.n - t * s.seqs) * G;
    const long long of_lane = static_cast<long long>(s.prefix_parts) * s.part_rows + static_cast<long long>(s.B) * G * along;
    return (lane * of_lane + static_cast<long long>(c) * s.part_rows +
            (static_cast<long long>(g.start) + t * s.seqs) * G * along + static_cast<long long>(h / s.side) * rows) *
           (s.halves ? 2 : 1);
}

__device__ __forceinline__ int own_len(const SharedCall& s, int b) { return max(min(s.own_lens[b], s.own_room), 0); }
__device__ __forceinline__ int own_units(int len) { return len / 32 + (len % 32 != 0); }

// Launches of decode_shared_own.cu.  The own tokens' kernel comes first on the stream; that of the prefixes does
// not end before it (so that the joining one, launched third, need only wait for the second).
int launch_own_tokens(const SharedCall& call, int d, bool bf16, cudaStream_t stream);
int launch_join(const SharedCall& call, int d, bool bf16, cudaStream_t stream);

// Launches a kernel; `early`: it may start while the one before it on the stream still runs, and waits for that one
// by itself.
template <typename Kernel, typename... Args>
int launch_on(bool early, Kernel kern, unsigned grid, int threads, size_t smem, cudaStream_t stream, const Args&... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &at;
    cfg.numAttrs = early ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? BSATTN_OK : BSATTN_ERR_CUDA;
}

}  // namespace bsattn
