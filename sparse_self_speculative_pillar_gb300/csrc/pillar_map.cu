// pillar_map.cu -- block tables and slot maps from request lengths.
//
// With n_b = ceil(len_b / 16) and m_b = ceil(prev_b / 16), request b takes
// max(n_b - m_b, 0) blocks from the free ring and gives max(m_b - n_b, 0)
// back.  Everything else is prefix sums over the batch: where its blocks
// start in the ring, where its released blocks go, where its positions start
// in the slot table (kv_off) and its new tokens in new_slots (new_off).
//
// Two kernels:
//   1. map_scan: one CTA, a thread per request (1024 at a time, with carries),
//      two block scans -- the demand first, since it decides which requests
//      are granted, then the other sums -- and the records the expansion
//      needs.  It also advances the ring's state: the expansion works from
//      the copy in the workspace.  Latency-bound.
//   2. map_expand: slot_table[kv_off[b] + t] = block * 16 + t % 16, four slots
//      per thread and store, 4096 per CTA tile; the requests of a tile are
//      found by one warp (32-way search of kv_off) and shared.  A position at
//      the start of a newly taken block also writes the block table's entry.
//      Bound by the stores: 4 bytes per position.
// The ring is first in, first out and never holds more than its size, so the
// places popped in a call (from head) and the places pushed (from head +
// count) are distinct: taking and giving need no order between them.
#include "pillar_device.cuh"
#include "pillar_map.h"

namespace pillar {

namespace {

constexpr int kScanThreads = 1024;
constexpr int kExpandThreads = 256;
constexpr int kExpandTile = 4096;  // slots per CTA tile: four int4 stores per thread
constexpr int kBlock = PILLAR_KV_BLOCK;

__device__ __forceinline__ long long warp_scan(long long x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if ((threadIdx.x & 31) >= o) x += y;
    }
    return x;
}

// Exclusive scan of N values per thread over the CTA; tot[] gets the totals.
template <int N>
__device__ void block_scan(long long (&v)[N], long long (&tot)[N]) {
    __shared__ long long sums[N][kScanThreads / 32];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    long long x[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        x[i] = warp_scan(v[i]);
        if (lane == 31) sums[i][wid] = x[i];
    }
    __syncthreads();
    if (wid < N) {
        const long long own = sums[wid][lane];
        sums[wid][lane] = warp_scan(own);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        tot[i] = sums[i][kScanThreads / 32 - 1];
        v[i] = x[i] - v[i] + (wid ? sums[i][wid - 1] : 0);
    }
    __syncthreads();
}

__global__ void __launch_bounds__(kScanThreads, 1) map_scan(const MapArgs a) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    MapHeader *hdr = reinterpret_cast<MapHeader *>(a.ws);
    MapRequest *rec = reinterpret_cast<MapRequest *>(a.ws + sizeof(MapHeader));
    int head = a.state[0], count = a.state[1];
    int bad = 0;
    const bool ring_ok = head >= 0 && head < a.num_blocks && count >= 0 && count <= a.num_blocks;
    if (!ring_ok) bad |= PILLAR_FLAG_BLOCK, head = 0, count = 0;
    __shared__ int s_bad;
    if (threadIdx.x == 0) s_bad = 0;
    long long c_want = 0, c_used = 0, c_len = 0, c_new = 0, c_give = 0;  // carries (the same in every thread)
    for (int base = 0; base < a.B; base += kScanThreads) {
        const int b = base + threadIdx.x;
        const bool live = b < a.B;
        int prev = live ? a.prev_len[b] : 0, len = live ? a.req_len[b] : 0;
        const long long most = min((long long)a.max_len, (long long)a.max_blocks * kBlock);
        if (prev < 0 || prev > most) bad |= PILLAR_FLAG_REQUEST, prev = 0, len = 0;
        if (len < 0 || len > most) bad |= PILLAR_FLAG_REQUEST, len = prev;
        const int m = (prev + kBlock - 1) / kBlock;
        int n = (len + kBlock - 1) / kBlock;
        long long want[1] = {n > m ? n - m : 0}, wtot[1];
        const long long own = want[0];
        block_scan<1>(want, wtot);
        const long long first = c_want + want[0];
        if (own > 0 && first + own > count) bad |= PILLAR_FLAG_BLOCK, len = prev, n = m;
        const int fresh = len > prev ? len - prev : 0, back = m > n ? m - n : 0;
        long long v[4] = {len, fresh, back, n > m ? n - m : 0}, tot[4];
        block_scan<4>(v, tot);
        if (live) {
            const long long no = c_new + v[1];
            if (no + fresh > 0x7fffffffll) bad |= PILLAR_FLAG_COUNT;
            MapRequest r;
            r.kv_off = c_len + v[0];
            r.new_off = (int)min(no, 0x7fffffffll);
            r.prev = prev;
            r.blocks = n;
            r.kept = min(n, m);
            r.take = (int)(c_used + v[3]);  // (the granted requests' demands come first)
            r.give = (int)min(c_give + v[2], 0x7fffffffll);
            r.give_end = (int)min(c_give + v[2] + back, 0x7fffffffll);
            r.pad = 0;
            rec[b] = r;
            a.granted[b] = len;
            a.kv_off[b] = r.kv_off;
            a.new_off[b] = r.new_off;
        }
        c_want += wtot[0];
        c_len += tot[0];
        c_new += tot[1];
        c_give += tot[2];
        c_used += tot[3];
    }
    const long long left = (long long)count - c_used + c_give;
    if (left > a.num_blocks) bad |= PILLAR_FLAG_BLOCK;  // more given back than the pool has
    if (bad) atomicOr(&s_bad, bad);
    __syncthreads();
    if (threadIdx.x == 0) {
        if (c_len > a.slot_capacity || c_new > a.new_capacity) s_bad |= PILLAR_FLAG_COUNT;
        hdr->err = s_bad;
        hdr->head = head;
        hdr->count = count;
        hdr->total = c_len;
        hdr->total_new = c_new;
        hdr->released = ring_ok ? c_give : 0;
        a.kv_off[a.B] = c_len;
        a.new_off[a.B] = (int)min(c_new, 0x7fffffffll);
        if (ring_ok) {
            a.state[0] = (int)((head + c_used) % a.num_blocks);
            a.state[1] = (int)min(left, (long long)a.num_blocks);
        }
    }
}

// The last request whose offset is at or below x (the offsets ascend from 0;
// x is below the total), by the whole warp: 32 probes a round.
template <typename F>
__device__ __forceinline__ int warp_find(int B, long long x, F off) {
    int lo = 0, n = B;  // the answer lies in [lo, lo + n)
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int i = lo + (int)(threadIdx.x & 31) * step;
        const unsigned le = __ballot_sync(0xffffffffu, i < lo + n && off(i) <= x);
        const int k = 31 - __clz(le);  // (lane 0 probes lo, which holds)
        const int end = lo + n;
        lo += k * step;
        n = min(step, end - lo);
    }
    return lo;
}

// The slot of position t of request b, its block taken from the ring when it
// is new (and then entered into the table by the thread that writes it).
struct Slots {
    const MapArgs &a;
    int head;
    int *bad;
    __device__ __forceinline__ int block(const MapRequest &r, int b, int i, bool enter) const {
        int blk;
        if (i < r.kept) {
            blk = a.table[(size_t)b * a.max_blocks + i];
        } else {
            long long at = (long long)head + r.take + (i - r.kept);
            if (at >= a.num_blocks) at -= a.num_blocks;
            blk = a.ring[at];
            if (enter) a.table[(size_t)b * a.max_blocks + i] = blk;
        }
        return blk;
    }
    __device__ __forceinline__ int slot(int blk, int t) const {
        if (blk < 0 || blk >= a.num_blocks) {
            *bad |= PILLAR_FLAG_SLOT;
            return -1;
        }
        return blk * kBlock + (t & (kBlock - 1));
    }
};

__global__ void __launch_bounds__(kExpandThreads) map_expand(const MapArgs a) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    MapHeader *hdr = reinterpret_cast<MapHeader *>(a.ws);
    const MapRequest *rec = reinterpret_cast<const MapRequest *>(a.ws + sizeof(MapHeader));
    __shared__ int s_first;
    int bad = 0;
    const Slots sl{a, hdr->head, &bad};
    // --- the slot table.  Every block of every request is entered here, whatever the capacity.
    const long long total = hdr->total;
    for (long long t0 = (long long)blockIdx.x * kExpandTile; t0 < total; t0 += (long long)gridDim.x * kExpandTile) {
        if (threadIdx.x < 32) {
            const int f = warp_find(a.B, t0, [&](int i) { return rec[i].kv_off; });
            if (threadIdx.x == 0) s_first = f;
        }
        __syncthreads();
        int b = s_first;
        __syncthreads();
        MapRequest r = rec[b];
        long long end = b + 1 < a.B ? rec[b + 1].kv_off : total;
        int blk = -1, at = -1;  // the block of the last position
#pragma unroll
        for (int q = 0; q < kExpandTile / (4 * kExpandThreads); ++q) {
            const long long i0 = t0 + ((long long)q * kExpandThreads + threadIdx.x) * 4;
            if (i0 >= total) break;
            int v[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const long long i = i0 + e;
                if (i >= total) break;
                while (i >= end) {  // (requests ahead, empty ones included)
                    r = rec[++b];
                    end = b + 1 < a.B ? rec[b + 1].kv_off : total;
                    at = -1;
                }
                const int t = (int)(i - r.kv_off);
                if (t / kBlock != at) {
                    at = t / kBlock;
                    blk = sl.block(r, b, at, (t & (kBlock - 1)) == 0);
                }
                v[e] = sl.slot(blk, t);
            }
            if (i0 + 4 <= min(total, a.slot_capacity)) {
                *reinterpret_cast<int4 *>(a.slots + i0) = make_int4(v[0], v[1], v[2], v[3]);
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (i0 + e < total && i0 + e < a.slot_capacity) a.slots[i0 + e] = v[e];
            }
        }
    }
    // --- the new tokens' slots
    const int warp = (int)((blockIdx.x * kExpandThreads + threadIdx.x) >> 5), lane = threadIdx.x & 31;
    const int warps = (int)(gridDim.x * kExpandThreads >> 5);
    const long long nnew = min(min(hdr->total_new, a.new_capacity), 0x7fffffffll);
    for (long long i0 = (long long)warp * 32; i0 < nnew; i0 += (long long)warps * 32) {
        int b = warp_find(a.B, i0, [&](int i) { return (long long)rec[i].new_off; });
        const long long i = i0 + lane;
        if (i < nnew) {
            while (b + 1 < a.B && rec[b + 1].new_off <= i) ++b;
            const MapRequest r = rec[b];
            const int t = r.prev + (int)(i - r.new_off);
            a.new_slots[i] = sl.slot(sl.block(r, b, t / kBlock, false), t);
        }
    }
    // --- the blocks given back
    const long long nback = hdr->released;
    for (long long i0 = (long long)warp * 32; i0 < nback; i0 += (long long)warps * 32) {
        int b = warp_find(a.B, i0, [&](int i) { return (long long)rec[i].give; });
        const long long i = i0 + lane;
        if (i < nback) {
            while (b + 1 < a.B && rec[b].give_end <= i) ++b;
            const MapRequest r = rec[b];
            const int blk = a.table[(size_t)b * a.max_blocks + r.blocks + (int)(i - r.give)];
            if (blk < 0 || blk >= a.num_blocks) bad |= PILLAR_FLAG_SLOT;
            a.ring[((long long)hdr->head + hdr->count + i) % a.num_blocks] = blk;
        }
    }
    if (bad) atomicOr(&hdr->err, bad);
}

}  // namespace

cudaError_t launch_block_map(const MapArgs &a, int nsm, cudaStream_t st) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kScanThreads);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, map_scan, a);
    if (e != cudaSuccess) return e;
    // as many CTAs as the batch could need at its longest, up to four per SM (the totals are on the device)
    const long long most = (long long)a.B * a.max_len;
    long long grid = (most + kExpandTile - 1) / kExpandTile;
    grid = grid < 1 ? 1 : grid > 4ll * nsm ? 4ll * nsm : grid;
    cfg.gridDim = dim3((unsigned)grid);
    cfg.blockDim = dim3(kExpandThreads);
    return cudaLaunchKernelEx(&cfg, map_expand, a);
}

}  // namespace pillar
