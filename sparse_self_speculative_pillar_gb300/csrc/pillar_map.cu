// pillar_map.cu -- block tables and slot maps from request lengths.
//
// With n_b = ceil(len_b / 16) and m_b = ceil(prev_b / 16), request b takes
// max(n_b - m_b, 0) blocks from the free ring and gives max(m_b - n_b, 0)
// back.  Everything else is prefix sums over the batch: where its blocks
// start in the ring, where its released blocks go, where its positions start
// in the slot table (kv_off) and its new tokens in new_slots (new_off).
//
// Two kernels, 19 us a call for 2048 requests of 1024 to 16384 positions (11.2 million):
//   1. map_scan: one CTA, two requests a thread (2048 at a time, with carries), one
//      block scan of the four sums; only when the ring runs short does the demand
//      decide first, with a scan of its own.  It writes the records that the
//      expansion needs beyond the call's own arrays (8 bytes a request: with
//      whole records one SM took as long to write them as for all the rest), and
//      advances the ring's state: the expansion works from the
//      copy in the workspace.  Latency-bound, some 4 us for 2048 requests.
//   2. map_expand: slot_table[kv_off[b] + t] = block * 16 + t % 16.  A grid row of CTAs
//      per request, a warp per 512 positions: one coalesced load of 32 blocks, then
//      16-byte stores whose blocks come by shuffle.  (A flat grid over the slots, each
//      tile searching its request, took 55 us for those slots where this takes
//      13, 3.5 TB/s.)  Blocks that were taken are entered into the
//      table on the way.  It writes 4 bytes per position, at 0.52 of a copy's rate: with
//      2048 requests each has one CTA, whose warps go through one to four
//      dependent rounds of table line and stores.
// The ring is first in, first out, and blocks are given back only when those
// in it before the call and those given back together fit (they always do
// when the tables and the ring agree on who holds what), so the places popped
// in a call (from head) and the places pushed (from head + count) are
// distinct: taking and giving need no order between them.
#include "pillar_device.cuh"
#include "pillar_map.h"

namespace pillar {

namespace {

constexpr int kScanThreads = 1024;
constexpr int kPerThread = 2;      // requests a scan thread takes
constexpr int kExpandThreads = 256;
constexpr int kBlock = PILLAR_KV_BLOCK;

// (len + 15 would pass 31 bits for the longest lengths)
__device__ __forceinline__ int blocks_of(int len) { return len / kBlock + (len % kBlock != 0); }

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
    const long long most = min((long long)a.max_len, (long long)a.max_blocks * kBlock);
    for (int base = 0; base < a.B; base += kScanThreads * kPerThread) {
        const int b0 = base + threadIdx.x * kPerThread;
        int prev[kPerThread], len[kPerThread];
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            prev[i] = b0 + i < a.B ? a.prev_len[b0 + i] : 0;
            len[i] = b0 + i < a.B ? a.req_len[b0 + i] : 0;
        }
        long long v[4] = {0, 0, 0, 0}, tot[4];  // positions, new tokens, blocks given back, blocks taken
        auto add = [&](int i) {
            const int m = blocks_of(prev[i]), n = blocks_of(len[i]);
            v[0] += len[i];
            v[1] += max(len[i] - prev[i], 0);
            v[2] += max(m - n, 0);
            v[3] += max(n - m, 0);
        };
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            if (prev[i] < 0 || prev[i] > most) bad |= PILLAR_FLAG_REQUEST, prev[i] = 0, len[i] = 0;
            if (len[i] < 0 || len[i] > most) bad |= PILLAR_FLAG_REQUEST, len[i] = prev[i];
            add(i);
        }
        block_scan<4>(v, tot);
        const long long before = c_want;
        c_want += tot[3];
        if (c_want > count) {  // (the same in every thread) the ring runs short: the first whose blocks do not fit and
                               // all later ones that need some stay as they are
            long long want = before + v[3];
            v[0] = v[1] = v[2] = v[3] = 0;
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                const int own = max(blocks_of(len[i]) - blocks_of(prev[i]), 0);
                want += own;
                if (own > 0 && want > count) bad |= PILLAR_FLAG_BLOCK, len[i] = prev[i];
                add(i);
            }
            block_scan<4>(v, tot);
        }
        long long kv = c_len + v[0], no = c_new + v[1], give = c_give + v[2], take = c_used + v[3];
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) {
            const int b = b0 + i, m = blocks_of(prev[i]), n = blocks_of(len[i]), fresh = max(len[i] - prev[i], 0);
            if (b < a.B) {
                if (no + fresh > 0x7fffffffll) bad |= PILLAR_FLAG_COUNT;
                // (the granted requests' demands come first in the ring)
                rec[b] = MapRequest{(int)take, (int)min(give, 0x7fffffffll)};
                a.granted[b] = len[i];
                a.kv_off[b] = kv;
                a.new_off[b] = (int)min(no, 0x7fffffffll);
            }
            kv += len[i];
            no += fresh;
            give += max(m - n, 0);
            take += max(n - m, 0);
        }
        c_len += tot[0];
        c_new += tot[1];
        c_give += tot[2];
        c_used += tot[3];
    }
    // more given back than the ring has room for beside what it held: none is (a block would land in a place that is being
    // popped)
    const bool fits = count + c_give <= a.num_blocks;
    if (!fits) bad |= PILLAR_FLAG_BLOCK;
    if (bad) atomicOr(&s_bad, bad);
    __syncthreads();
    if (threadIdx.x == 0) {
        if (c_len > a.slot_capacity || c_new > a.new_capacity) s_bad |= PILLAR_FLAG_COUNT;
        hdr->err = s_bad;
        hdr->head = head;
        hdr->count = count;
        hdr->released = ring_ok && fits ? c_give : 0;
        a.kv_off[a.B] = c_len;
        a.new_off[a.B] = (int)min(c_new, 0x7fffffffll);
        if (ring_ok) {
            a.state[0] = (int)((head + c_used) % a.num_blocks);
            a.state[1] = (int)(count - c_used + (fits ? c_give : 0));
        }
    }
}

__global__ void __launch_bounds__(kExpandThreads) map_expand(const MapArgs a) {
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    MapHeader *hdr = reinterpret_cast<MapHeader *>(a.ws);
    const MapRequest *rec = reinterpret_cast<const MapRequest *>(a.ws + sizeof(MapHeader));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int head = hdr->head, count = hdr->count;
    int bad = 0;
    auto slot0 = [&](int blk) {  // first slot of a block
        if (blk >= 0 && blk < a.num_blocks) return blk * kBlock;
        bad |= PILLAR_FLAG_SLOT;
        return -1;
    };
    const int most = (int)min((long long)a.max_len, (long long)a.max_blocks * kBlock);
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const MapRequest r = rec[b];
        const int len = a.granted[b], given = a.prev_len[b];
        const long long off = a.kv_off[b];
        const int prev = given < 0 || given > most ? 0 : given;
        const int blocks = blocks_of(len), had = blocks_of(prev), kept = min(blocks, had);
        int *row = a.table + (size_t)b * a.max_blocks;
        auto block = [&](int i) {  // (those past `kept` are being taken)
            if (i < kept) return row[i];
            const long long at = (long long)head + r.take + (i - kept);
            return a.ring[at >= a.num_blocks ? at - a.num_blocks : at];
        };
        // output aligned to four slots: `lead` single ones, then 16-byte stores, which may span two blocks
        const int lead = (int)(-off & 3);
        for (int i0 = (blockIdx.y * (kExpandThreads / 32) + warp) * 32; i0 < blocks;
             i0 += gridDim.y * (kExpandThreads / 32) * 32) {
            const int i = i0 + lane;
            const int blk = i < blocks ? block(i) : 0, behind = i0 + 32 < blocks ? block(i0 + 32) : 0;
            if (i >= kept && i < blocks) row[i] = blk;
            const int first = i < blocks ? slot0(blk) : 0, next = i0 + 32 < blocks ? slot0(behind) : 0;
            const int t0 = i0 * kBlock;
            int *out = a.slots + off + t0;
            const int n = (int)max(0ll, min((long long)len - t0, a.slot_capacity - off - t0));  // slots to write from t0 on
            const int s0 = __shfl_sync(0xffffffffu, first, 0);
            if (i0 == 0 && lane < lead && lane < n) out[lane] = s0 < 0 ? -1 : s0 + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int t = lead + 128 * e + 4 * lane, j = t / kBlock, j3 = (t + 3) / kBlock;
                const int sa = __shfl_sync(0xffffffffu, first, j & 31), sb = __shfl_sync(0xffffffffu, first, j3 & 31);
                const int xa = j < 32 ? sa : next, xb = j3 < 32 ? sb : next;
                int v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int x = (t + q) / kBlock == j ? xa : xb;
                    v[q] = x < 0 ? -1 : x + (t + q) % kBlock;
                }
                if (t + 4 <= n) {
                    *reinterpret_cast<int4 *>(out + t) = make_int4(v[0], v[1], v[2], v[3]);
                } else {
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        if (t + q < n) out[t + q] = v[q];
                }
            }
        }
        if (blockIdx.y == 0) {
            // the new tokens' slots
            const int no = a.new_off[b];
            for (int i = threadIdx.x; i < len - prev && (long long)no + i < a.new_capacity; i += kExpandThreads) {
                const int t = prev + i, s = slot0(block(t / kBlock));
                a.new_slots[(long long)no + i] = s < 0 ? -1 : s + t % kBlock;
            }
            // the blocks given back
            if (hdr->released)
                for (int i = threadIdx.x; i < had - blocks; i += kExpandThreads) {
                    const int blk = row[blocks + i];
                    slot0(blk);
                    a.ring[((long long)head + count + r.give + i) % a.num_blocks] = blk;
                }
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
    // per request, CTAs for its longest possible table, as long as that stays within 16 a SM
    // (in a graph, 2048 requests of 1024 to 16384 positions: 17.8 us a call with 16, 18.7 with 32, 22.1 with 64; of 8000
    // each: 19.1, 21.4 and 21.4; 256 of 8000: 6.8 with all three)
    const int per_cta = kExpandThreads * kBlock;
    int rows = (int)(((long long)a.max_len + per_cta - 1) / per_cta);
    const int most = 16 * nsm / a.B;
    rows = rows < most ? rows : most;
    cfg.gridDim = dim3((unsigned)(a.B < 65536 ? a.B : 65536), (unsigned)(rows < 1 ? 1 : rows < 65535 ? rows : 65535));
    cfg.blockDim = dim3(kExpandThreads);
    return cudaLaunchKernelEx(&cfg, map_expand, a);
}

}  // namespace pillar
