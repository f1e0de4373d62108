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
    int n, B, Hkv, max_blocks, num_blocks, max_len;
    bool ends;
};

constexpr int kMapRows = 32;  // rows that one call maps, at most

// The places of rows [t0, t0 + rows), for KV head 0, as rows of the pools (block * Hkv * 16 + row of the block; head h lies 16 h
// further on), or -1, by one warp.  The request of row t0 is found 32 offsets at a time (two dependent rounds for a thousand
// requests), the others' by the offsets that follow it.
__device__ __forceinline__ void find_rows(const RowMap &m, long long t0, int rows, int *place) {
    const int lane = threadIdx.x & 31;
    const long long t = t0 + lane;
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
    int at = -1;
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
            else at = block * m.Hkv * PILLAR_KV_BLOCK + (int)(pos % PILLAR_KV_BLOCK);
        }
        if (bad && m.flags) atomicOr(m.flags, bad);
    }
    place[lane] = at;
}

// A packed batch is worked on in pieces of sixteen values (32 bytes of bf16), K's by the first half of a CTA's workers, V's by
// the second.  The pair (token, piece of the token) of a thread moves on by that many threads without a division.
struct Walk {
    int token, piece, dt, dp, pieces;
    __device__ __forceinline__ Walk(int thread, int threads, int pieces_) : pieces(pieces_) {
        token = thread / pieces;
        piece = thread - token * pieces;
        dt = threads / pieces;
        dp = threads - dt * pieces;
    }
    __device__ __forceinline__ void next() {
        token += dt;
        piece += dp;
        if (piece >= pieces) piece -= pieces, ++token;
    }
};

// 32 bytes; kWide: at a multiple of 32.
struct Half16 {
    uint32_t w[8];
};
template <bool kWide>
__device__ __forceinline__ Half16 load32(const uint16_t *src) {
    Half16 x;
    if (kWide) {
        asm volatile("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(x.w[0]), "=r"(x.w[1]), "=r"(x.w[2]), "=r"(x.w[3]), "=r"(x.w[4]), "=r"(x.w[5]), "=r"(x.w[6]), "=r"(x.w[7])
                     : "l"(src));
    } else {
        const uint4 a = __ldg(reinterpret_cast<const uint4 *>(src)), b = __ldg(reinterpret_cast<const uint4 *>(src) + 1);
        x = {{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
    }
    return x;
}
template <bool kWide>
__device__ __forceinline__ void store32(uint16_t *dst, const uint32_t (&w)[8]) {
    if (kWide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}
// Rows of both tensors at multiples of 32 bytes.
inline bool rows_wide(const void *k, const void *v, long long k_stride, long long v_stride) {
    return ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31) == 0 && ((k_stride | v_stride) & 15) == 0;
}

// CTAs of eight warps that work and one that finds the rows of the next `most` tokens meanwhile (a chain of four or five
// dependent loads).  Each goes through a range of the batch of its own, all of nearly one length.
constexpr int kRowWorkers = 256, kRowThreads = kRowWorkers + 32;
template <typename Work>
__device__ __forceinline__ void for_rows(const RowMap &m, int most, Work work) {
    __shared__ int s_place[2][kMapRows];
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int end = (int)((long long)m.n * (blockIdx.x + 1) / gridDim.x);
    int buf = 0;
    for (int t0 = (int)((long long)m.n * blockIdx.x / gridDim.x); t0 < end; buf ^= 1) {
        const int rows = min(most, end - t0);
        if (threadIdx.x >= kRowWorkers) find_rows(m, t0, rows, s_place[buf]);
        __syncthreads();  // (and the rows before last have been worked on)
        if (threadIdx.x < kRowWorkers) work((long long)t0, rows, s_place[buf]);
        t0 += rows;
    }
}
// Most rows of a CTA's turn, and CTAs: one row while that many CTAs are resident at once (a decode step), else sixteen (26 K rows
// stored and read back: 53.5 us; eight 54.6, thirty-two 53.8), and no more CTAs than are resident.  (Ten in a graph, 8 heads of
// D = 128.  Appends of 608 rows, one to a CTA: 39 us; of 760 60 in turns of sixteen rows, 63 one by one; of 2432 62 and 122.  Reads of
// 760 rows, one to a CTA: 41, in turns of sixteen 55; of 912 56 and 60; of 2432 60 and 109.)
inline int rows_of_turn(int n, int resident, int nsm) { return n <= resident * nsm ? 1 : 16; }
inline unsigned row_ctas(int n, int rows, int resident, int nsm) {
    const long long groups = ((long long)n + rows - 1) / rows, most = (long long)resident * nsm;
    return (unsigned)(groups < most ? groups : most);
}
// (Launched while the kernel before on the stream still runs: its launch is over when that kernel is.)
template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args, int), const Args &a, int rows, unsigned grid, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kRowThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a, rows);
}

}  // namespace pillar
