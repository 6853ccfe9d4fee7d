// Device-side view of a paged cache and of the sequences whose tokens it holds.
//
// A cache's pages hold 64 tokens each, per key/value head apart: keys as E4M3 codes [64][D], values turned,
// [D][64] (the attention's second product sums over tokens: a lane's codes are then neighbours in memory), and one
// E8M0 scale byte for the keys and one for the values of a (page, head). Token t of sequence s is slot t % 64 of page
// table[s][t / 64].
//
// Lengths, starts and pages are device data that the host does not see; whatever they hold, the functions here
// keep every index inside its array: a start is clamped to the tokens there are, a length to what the table's
// row can hold, and a page outside the cache is no page (-1).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "launch.hpp"

namespace nvfp4 {

constexpr int kPage = 64;  // tokens

// Sequence s: its tokens in the call are rows first .. first + n - 1, the last n of its `len` tokens.
struct Seq {
    int first, n, len;
};

__device__ __forceinline__ Seq sequence(const SeqArgs &a, int s) {
    Seq q;
    q.len = min(max(a.lengths[s], 0), a.width * kPage);
    if (a.starts) {
        q.first = min(max(a.starts[s], 0), a.tokens);
        q.n = min(max(a.starts[s + 1], q.first), a.tokens) - q.first;
    } else {
        q.first = s;
        q.n = 1;
    }
    return q;
}

__device__ __forceinline__ int page_of(const SeqArgs &a, int s, int block) {
    const int p = a.table[(int64_t)s * a.ldt + block];
    return p >= 0 && p < a.pages ? p : -1;
}

// The pieces of `size` rows that a call's sequences are cut into, numbered: those of sequence s, of rows_per rows a
// token, begin at base(s) = floor(first rows_per / size) + extra s. floor(a + b) + 1 >= floor(a) + ceil(b), so with extra
// = 1 no two pieces share a number, and no number reaches piece_bound; extra = 2 leaves room for one piece more per
// sequence. Some numbers have no piece. size = 2^log2.
__device__ __forceinline__ int log2_of(int size) { return __ffs(size) - 1; }
__device__ __forceinline__ int piece_base(const SeqArgs &a, int s, int rows_per, int log2, int extra) {
    const int first = a.starts ? min(max(a.starts[s], 0), a.tokens) : s;
    return (int)((uint64_t)first * (uint32_t)rows_per >> log2) + extra * s;
}

// The last sequence whose base is not past `piece` (the bases ascend). Called by whole waves, all lanes alike.
__device__ __forceinline__ int piece_sequence(const SeqArgs &a, int piece, int rows_per, int log2, int extra) {
    const int lane = threadIdx.x & 63;
    int s = 0;
    for (int s0 = 0; s0 < a.seqs; s0 += 64) {
        const bool in = s0 + lane < a.seqs && piece_base(a, s0 + lane, rows_per, log2, extra) <= piece;
        const int n = __popcll(__ballot(in));
        if (n) s = s0 + n - 1;
        if (n < 64) break;
    }
    return __builtin_amdgcn_readfirstlane(s);
}

}  // namespace nvfp4
