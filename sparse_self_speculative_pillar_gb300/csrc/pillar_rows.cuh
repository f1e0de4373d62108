// pillar_rows.cuh -- where the tokens of a packed batch live in the cache.
//
// Packed row t belongs to the request b with off[b] <= t < off[b+1]; its
// position is counted from the request's first one (a read) or up to its last
// one (an append), and its place is row position % 16 of block
// block_table[b, position / 16].
#pragma once

#include "pillar_device.cuh"

namespace pillar {

struct RowMap {
    const int *off;    // [B+1], ascending from 0
    const int *base;   // [B]: lengths that include the rows (ends), or positions of the first rows
    const int *table;  // [B, max_blocks]
    int *flags;        // device error word, or null
    int n, B, max_blocks, num_blocks, max_len;
    bool ends;
};

constexpr int kMapRows = 32;  // rows that one call maps, at most

// The places of rows [t0, t0 + rows) as block * 16 + row of the block, or -1, by one warp.  The request of row t0 is found
// 32 offsets at a time (two dependent rounds for a thousand requests), the others' by the offsets that follow it.
__device__ __forceinline__ void find_rows(const RowMap &m, int t0, int rows, long long *place) {
    const int lane = threadIdx.x & 31;
    const long long t = (long long)t0 + lane;
    const int all = min(m.n, __ldg(m.off + m.B));
    int lo = 0;
    for (int n = m.B; n > 1;) {  // the last offset at or below t0 is one of n from lo on
        const int step = (n + 31) / 32, i = lo + lane * step;
        const unsigned le = __ballot_sync(0xffffffffu, lane * step < n && __ldg(m.off + i) <= t0);
        const int k = max(31 - __clz(le), 0);
        n = min(step, n - k * step);
        lo += k * step;
    }
    // (more than 32 requests begin within the rows only when some of them are empty: the loop below)
    const int behind = lo + 1 + lane <= m.B ? __ldg(m.off + lo + 1 + lane) : 0x7fffffff;
    int b = lo;
    for (int i = 0; i < rows; ++i) {
        const int at = __popc(__ballot_sync(0xffffffffu, behind <= t0 + i));
        if (lane == i) b = lo + at;
    }
    if (lane >= rows) return;
    long long at = -1;
    if (t < all) {
        for (b = min(b, m.B - 1); b + 1 < m.B && __ldg(m.off + b + 1) <= t;) ++b;
        const int first = __ldg(m.off + b), end = __ldg(m.off + b + 1), base = __ldg(m.base + b);
        // (64 bits: a length near the lowest int would wrap)
        const long long start = m.ends ? (long long)base - ((long long)end - first) : base, pos = start + (t - first);
        int bad = 0;
        if (first < 0 || t < first || t >= end || end > m.n || start < 0 || start + ((long long)end - first) > m.max_len ||
            pos / PILLAR_KV_BLOCK >= m.max_blocks) {
            bad = PILLAR_FLAG_REQUEST;
        } else {
            const int block = __ldg(m.table + (size_t)b * m.max_blocks + pos / PILLAR_KV_BLOCK);
            if (block < 0 || block >= m.num_blocks) bad = PILLAR_FLAG_SLOT;
            else at = (long long)block * PILLAR_KV_BLOCK + pos % PILLAR_KV_BLOCK;
        }
        if (bad && m.flags) atomicOr(m.flags, bad);
    }
    place[lane] = at;
}

// A packed batch is worked on in pieces of 16 bytes of bf16 (eight values): piece j of a token, K's first, then V's.  A
// CTA's threads walk over the pieces of its tokens; the pair (token, piece) moves on without a division.
struct Walk {
    int token, piece, dt, dp, pieces;
    __device__ __forceinline__ Walk(int threads, int pieces_) : pieces(pieces_) {
        token = threadIdx.x / pieces;
        piece = threadIdx.x - token * pieces;
        dt = threads / pieces;
        dp = threads - dt * pieces;
    }
    __device__ __forceinline__ void next() {
        token += dt;
        piece += dp;
        if (piece >= pieces) piece -= pieces, ++token;
    }
};

}  // namespace pillar
