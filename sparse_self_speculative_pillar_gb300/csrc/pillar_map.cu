// pillar_map.cu -- block tables and slot maps from request lengths.
//
// With n_b = ceil(len_b / 16) and m_b = ceil(prev_b / 16), request b takes
// max(n_b - m_b, 0) blocks from the free ring and gives max(m_b - n_b, 0)
// back.  Everything else is prefix sums over the batch: where its blocks
// start in the ring, where its released blocks go, where its positions start
// in the slot table (kv_off) and its new tokens in new_slots (new_off).
//
// Two kernels:
//   1. map_scan: one CTA, four requests a thread (4096 at a time, with carries), one
//      block scan of the four sums; only when the ring runs short does the demand
//      decide first, with a scan of its own.  It writes the records that the
//      expansion needs and advances the ring's state: the expansion works from the
//      copy in the workspace.  Latency-bound.
//   2. map_expand: slot_table[kv_off[b] + t] = block * 16 + t % 16.  A grid row of CTAs
//      per request, a warp per 512 positions: one coalesced load of 32 blocks, then
//      16-byte stores whose block comes by shuffle.  (A flat grid over the slots, each
//      tile searching its request, took 55 us for 17 million slots where this takes
//      9, with 67 MB to write.)  Blocks that were taken are entered into the
//      table on the way.  Bound by the stores: 4 bytes per position.
// The ring is first in, first out and never holds more than its size, so the
// places popped in a call (from head) and the places pushed (from head +
// count) are distinct: taking and giving need no order between them.
#include "pillar_device.cuh"
#include "pillar_map.h"

namespace pillar {

namespace {

constexpr int kScanThreads = 1024;
constexpr int kPerThread = 4;      // requests a scan thread takes
constexpr int kExpandThreads = 256;
constexpr int kWarpBlocks = 32;    // blocks a warp expands at a time (64: 5 % slower, 128: 15 %)
constexpr int kBlock = PILLAR_KV_BLOCK;

__device__ __forceinline__ int blocks_of(int len) { return (len + kBlock - 1) / kBlock; }

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
                MapRequest r;
                r.kv_off = kv;
                r.new_off = (int)min(no, 0x7fffffffll);
                r.prev = prev[i];
                r.blocks = n;
                r.kept = min(n, m);
                r.take = (int)take;  // (the granted requests' demands come first)
                r.give = (int)min(give, 0x7fffffffll);
                r.give_end = (int)min(give + max(m - n, 0), 0x7fffffffll);
                r.len = len[i];
                rec[b] = r;
                a.granted[b] = len[i];
                a.kv_off[b] = kv;
                a.new_off[b] = r.new_off;
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
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const MapRequest r = rec[b];
        const int len = r.len;
        int *row = a.table + (size_t)b * a.max_blocks;
        auto ring = [&](int i) {  // the i-th block, when it was taken
            const long long at = (long long)head + r.take + (i - r.kept);
            return a.ring[at >= a.num_blocks ? at - a.num_blocks : at];
        };
        for (int i0 = (blockIdx.y * (kExpandThreads / 32) + warp) * kWarpBlocks; i0 < r.blocks;
             i0 += gridDim.y * (kExpandThreads / 32) * kWarpBlocks) {
            int blk[kWarpBlocks / 32];
#pragma unroll
            for (int q = 0; q < kWarpBlocks / 32; ++q) {
                const int i = i0 + 32 * q + lane;
                blk[q] = i >= r.blocks ? 0 : i < r.kept ? row[i] : ring(i);
            }
#pragma unroll
            for (int q = 0; q < kWarpBlocks / 32; ++q) {
                const int i = i0 + 32 * q + lane;
                if (i >= r.kept && i < r.blocks) row[i] = blk[q];
                const int first = i < r.blocks ? slot0(blk[q]) : 0;
                const int t0 = (i0 + 32 * q) * kBlock;  // position of the 32 blocks' first slot
                const long long at = r.kv_off + t0;
                if ((at & 3) == 0 && t0 + 32 * kBlock <= len && at + 32 * kBlock <= a.slot_capacity) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {  // eight blocks a store, four lanes each
                        const int s = __shfl_sync(0xffffffffu, first, 8 * e + (lane >> 2)), o = (lane & 3) * 4;
                        *reinterpret_cast<int4 *>(a.slots + at + 128 * e + 4 * lane) =
                            s < 0 ? make_int4(-1, -1, -1, -1) : make_int4(s + o, s + o + 1, s + o + 2, s + o + 3);
                    }
                } else {
#pragma unroll 4
                    for (int e = 0; e < 16; ++e) {  // two blocks a store
                        const int s = __shfl_sync(0xffffffffu, first, 2 * e + (lane >> 4)), t = 32 * e + lane;
                        if (t0 + t < len && at + t < a.slot_capacity) a.slots[at + t] = s < 0 ? -1 : s + (lane & 15);
                    }
                }
            }
        }
        if (blockIdx.y == 0) {
            // the new tokens' slots
            for (int i = threadIdx.x; i < len - r.prev && (long long)r.new_off + i < a.new_capacity; i += kExpandThreads) {
                const int t = r.prev + i, j = t / kBlock, s = slot0(j < r.kept ? row[j] : ring(j));
                a.new_slots[(long long)r.new_off + i] = s < 0 ? -1 : s + t % kBlock;
            }
            // the blocks given back
            if (hdr->released)
                for (int i = threadIdx.x; i < r.give_end - r.give; i += kExpandThreads) {
                    const int blk = row[r.blocks + i];
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
    // per request, CTAs for its longest possible table, as long as that stays within 32 a SM
    const int per_cta = kExpandThreads / 32 * kWarpBlocks * kBlock;
    int rows = (int)(((long long)a.max_len + per_cta - 1) / per_cta);
    const int most = 32 * nsm / a.B;
    rows = rows < most ? rows : most;
    cfg.gridDim = dim3((unsigned)(a.B < 65536 ? a.B : 65536), (unsigned)(rows < 1 ? 1 : rows < 65535 ? rows : 65535));
    cfg.blockDim = dim3(kExpandThreads);
    return cudaLaunchKernelEx(&cfg, map_expand, a);
}

}  // namespace pillar
