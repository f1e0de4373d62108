// pillar_attn_kv4.cu -- the unified draft/verify attention over the 4-bit cache.
//
// For query row r and key t, with K and V rows e2m1(code) * scale (pillar_kv4.cuh):
//     s[r, t] = scale * (q_r . k_t),   o[r] = sum_t e^(s[r, t] - m) v_t / sum_t e^(s[r, t] - m)
// The planner, its work items, the partial records and the merge of split
// units are those of the bf16 step; only the kernel between them differs.
//
// Every cache value is an f16 value (six significant bits within 2^-18 ..
// 61440), and so is a bf16 query row divided by a power of two (its largest
// magnitude brought to [2^14, 2^15)), but for elements 2^-28 below that.  So
// both products take f16 operands and the scores are sums of exact products.
//
// Here are the verify items of more than sixteen rows (24 without a dump of logits);
// pillar_attn_kv4_few.cu has the others.  One persistent CTA an SM, 128 keys a tile, the keys on the M of
// tcgen05:
//     S^T [keys x rows] = K Q^T      K from tensor memory, Q from shared memory
//     O^T [D x rows]   += V^T P^T    V and P from shared memory
// so that a key's row is made into an operand once, whatever the number of
// query rows.
// A row is (head, query token), the tokens of a head together: the rows' logits
// lie one after another.
//   * The resolver warp takes items from the planner's queue and turns their
//     keys into rows of the pools, 512 at a time.
//   * Four warps each for K and V copy the rows of the tiles ahead (16 bytes a
//     lane), turn a key's codes into f16 and write them to tensor memory (K: lane
//     = key) or swizzled shared memory (V: keys x D, MN-major).
//   * One warp issues the products of S^T, another one those of O^T.
//   * Sixteen softmax warps, a key a thread: two sets that take tiles in turn, each
//     with an O and reference maxima of its own, of two groups that share the rows,
//     eight at a time.  A reference maximum moves only when a score passes it by
//     more than 2^8, which a vote of the group finds out.
//   * Four warps write finished items, one stages queries.
//
// What bounds it: issue slots.  On 128 requests of 6144 to 10240 tokens, 15 of them verifying 36 rows a KV head, logits dumped (145 us
// a call, 2.3 TB/s; the bf16 step 170, the 8-bit one 200), an SM's schedulers issue 0.63 of their cycles: a tile takes some 4200
// instructions and 520 more for eight rows (conversions and operand stores, softmax, the dump's stores).  The tensor cores are
// at 0.11, DRAM at 0.27.  Keys rather than rows on the M: a tile's products then cost what its rows do, and K goes from a
// thread's registers to tensor memory without a transpose.  With mma.sync at 36 rows (five row tiles a warp) the call took 216 us
// where this took 158; with blocks of codes copied by TMA into the same roles 160 where this took 146; items of 1024 keys took 164
// where those of 2048 took 158.
#include "pillar_attn_kv4.cuh"

namespace pillar {

namespace {

constexpr int kTile = 128;                   // keys of a tile
constexpr int kChunkTiles = 4;               // tiles whose rows are resolved together
constexpr int kChunkKeys = kTile * kChunkTiles;
// Chunks in flight between the resolver and their readers.  K and V warps look for the rows of tile x + 4 before they work on
// tile x.  With items of one tile, each a chunk, those are free once the softmax warps have come to tile x + 4 - kChunks, and
// to tile x they come without these: kChunks >= 4.
constexpr int kChunks = 5;
constexpr int kItems = 6;                    // items in flight (tile x + 4 may belong to item i + 4: as for kChunks, at least 5)
constexpr int kStages = 4;                   // tiles of codes in shared memory
constexpr int kWarps = 32, kGroups = 4;       // groups of softmax warps
constexpr int kThreads4 = kWarps * 32;
// tensor memory: two tiles of K, two of S^T, the O^T of each set, sums of weights (a key's lane, a column per row) of each set
constexpr uint32_t kTmemCols = 512, kTmemK = 0, kTmemS = 128, kTmemO = 256, kTmemL = 384;

// A work item in shared memory.
struct alignas(16) ItemRec {
    int stop;            // no more items
    int tiles, n, begin; // its tiles, keys, first position
    int L, g;            // context length, KV head
    int q_off, vidx, nsplit, rec;
    long long logit_off;
};

template <int D>
struct Smem4 {
    static constexpr int kRow = D / 2, kScales = D / kGroup4;  // bytes of a key's codes and scales
    alignas(1024) uint8_t v[2][kTile * D * 2];  // V operands: 64-dimension halves of [128 keys][128 bytes], 128-byte swizzle
    alignas(1024) uint8_t p[2][kTile * 128];    // P operands: 16-row groups of [128 keys][32 bytes], 32-byte swizzle
    alignas(1024) uint8_t q[2][kMaxRows * D * 2];  // Q operands: 64-dimension halves of [64 rows][128 bytes], 128-byte swizzle
    alignas(128) uint8_t codes[2][kStages][kTile * kRow];    // K, V
    alignas(16) uint8_t scales[2][kStages][kTile * kScales];
    alignas(16) int row[kChunks][kChunkKeys];   // rows of the pools ((block * Hkv + g) * 16 + position % 16), or -1
    int chunk_tiles[kChunks];                   // 0: no more
    ItemRec item[kItems];
    // per query row: logit = sum * fac, in base-2 units sum * fac2; last position seen
    alignas(16) float fac[kItems][kMaxRows], fac2[kItems][kMaxRows];
    int lim[kItems][kMaxRows];
    // per item (in turn), set and row: kLift - reference maximum (base 2); sums of weights, by the keys' warp of a tile
    alignas(16) float nref[2][2][kMaxRows], sum[2][2][4][kMaxRows];
    float top[kGroups][4][32];                  // a group's largest scores, per warp
    uint64_t item_full[kItems], item_empty[kItems], fac_full[kItems];
    uint64_t rows_full[kChunks], rows_empty[kChunks];
    uint64_t q_full[2], q_empty[2], k_full[2], s_full[2], p_full[2], v_full[2], pv_done[2];
    uint64_t o_full[2], o_empty[2], epi_full[2], epi_empty[2], drain[2];
    uint32_t tmem;
    int abort;  // a wait has given up
};
static_assert(sizeof(Smem4<128>) <= 227 * 1024, "shared memory of a CTA");
static_assert(sizeof(Smem4<64>) > 114 * 1024, "never two CTAs on an SM: each takes all of its tensor memory");

// A wait by a whole warp, a few instructions long (every wait that is inlined costs the roles' shared instruction cache; with
// the clock in each, plain decoding took 227 us here, and 215 without).  The products' warps watch the clock for all: nothing
// moves in a CTA for long without them, and one that has had nothing to do for the bound raises the abort flag.  A count of polls
// bounds the waits that outlive it, whatever the caller's bound is (an item takes microseconds).
constexpr int kMostPolls = 1 << 22;
template <int D>
__device__ __forceinline__ bool wait4(uint64_t *bar, uint32_t parity, Smem4<D> &sm) {
#pragma unroll 1
    for (int n = 0; !mbar_try_wait_warp(bar, parity); ++n)
        if (__any_sync(0xffffffffu, *static_cast<volatile int *>(&sm.abort) | (n > kMostPolls))) {
            sm.abort = 1;
            return false;
        }
    return true;
}
// The same for two barriers, by the warps that watch the clock.  (By the whole warp, too: one thread's tests of a barrier come back
// at once, 40 cycles apart, and took a third of its scheduler's issue slots.)
template <int D>
__device__ __forceinline__ bool watch4(uint64_t *bar, uint32_t parity, uint64_t *bar2, uint32_t parity2, Smem4<D> &sm,
                                       unsigned long long ns) {
    unsigned long long t0 = 0;
#pragma unroll 1
    for (;;) {
        const bool one = mbar_try_wait(bar, parity), two = mbar_try_wait(bar2, parity2);  // (the tests' latencies overlap)
        if (__all_sync(0xffffffffu, one && two)) return true;
        const unsigned long long now = global_timer_ns();
        if (t0 == 0) t0 = now;
        if (__any_sync(0xffffffffu, *static_cast<volatile int *>(&sm.abort) | (now - t0 > ns))) {
            sm.abort = 1;
            return false;
        }
    }
}

__device__ __forceinline__ void arrive_lane0(uint64_t *bar, uint32_t count = 1) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive_cnt(bar, count);
}
__device__ __forceinline__ bool elect_one4() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
template <int kOff>
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {  // to dst + kOff
    asm volatile("cp.async.cg.shared.global [%0+%2], [%1], 16;" ::"r"(dst), "l"(src), "n"(kOff) : "memory");
}
template <int kOff>
__device__ __forceinline__ int lds_int(uint32_t at) {
    int v;
    asm volatile("ld.shared.s32 %0, [%1+%2];" : "=r"(v) : "r"(at), "n"(kOff) : "memory");
    return v;
}
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(N) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Columns of this thread's tensor-memory lane; the loads and stores are waited for together.
__device__ __forceinline__ void tmem_ld8(uint32_t taddr, float *v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "f"(v[0]), "f"(v[1]),
                 "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The rows' chunks of eight are dealt out to the two groups of a softmax set: group h has chunks h, h + 2, ..
static_assert(kMaxRows == 64 && kGroups == 4, "four chunks of eight rows a group, at most: a lane a row");

// ------------------------------------------------------------------ resolver warp

// A CTA's share of the drafts' lists and of the block tables into L2, as it runs out of verify items: the drafts' kernel begins with
// chains of loads from them (128 requests, 15 verify: 147.5 us -> 146.4; five query heads a KV head, contexts of 4096 to 24576: 190.9 ->
// 190.2; medians of five runs of either, which lie within 0.2).  Arrays so large that a call may well read only a fraction of them are
// left out.
constexpr long long kPrefetchBytes = 8 << 20;
__device__ __forceinline__ void prefetch_lists(const Kv4Params &p, int lane) {
    const long long list = (long long)p.B * p.Hkv * p.max_sparse * 4, table = (long long)p.B * p.c.max_blocks * 4;
    const int first = blockIdx.x * 32 + lane, n = gridDim.x * 32;
    if (list <= kPrefetchBytes)
        for (int l = first; l * 128ll < list; l += n) l2_prefetch(reinterpret_cast<const char *>(p.sparse_idx) + l * 128ll);
    if (table <= kPrefetchBytes)
        for (int l = first; l * 128ll < table; l += n) l2_prefetch(reinterpret_cast<const char *>(p.c.table) + l * 128ll);
}

template <int D>
__device__ void resolver4(const Kv4Params &p, Smem4<D> &sm, int lane) {
    const int num_items = *reinterpret_cast<volatile int *>(&p.hdr->num_verify_items);
    int slot = 0;  // of the next chunk
    uint32_t phase = 0;
#pragma unroll 1
    for (int i = 0;; ++i) {
        const int is = i % kItems;
        if (!wait4(&sm.item_empty[is], (i / kItems & 1) ^ 1, sm)) return;
        int it = 0;
        if (lane == 0) it = atomicAdd(&p.hdr->item_counter, 1);
        it = __shfl_sync(0xffffffffu, it, 0);
        if (it >= num_items) {
            if (lane == 0) sm.item[is].stop = 1;
            arrive_lane0(&sm.item_full[is]);
            if (p.hdr->num_items > num_items) prefetch_lists(p, lane);
            if (!wait4(&sm.rows_empty[slot], phase ^ 1, sm)) return;
            if (lane == 0) sm.chunk_tiles[slot] = 0;
            arrive_lane0(&sm.rows_full[slot]);
            return;
        }
        const Item itm = p.items[it];
        const int b = itm.unit / p.Hkv, g = itm.unit - b * p.Hkv;
        const ReqInfo ri = p.req[b];
        const UnitInfo ui = p.unit[itm.unit];
        const int n = itm.end - itm.begin, tiles = max(1, (n + kTile - 1) / kTile);
        if (lane == 0) {
            ItemRec r;
            r.stop = 0;
            r.tiles = tiles;
            r.n = n;
            r.begin = itm.begin;
            r.L = ri.len;
            r.g = g;
            r.q_off = ri.q_off;
            r.vidx = ri.vidx;
            r.nsplit = ui.nsplit;
            r.rec = ui.rec_base + itm.split * ui.rec_rows;
            r.logit_off = p.logit_off[b];
            sm.item[is] = r;
        }
        arrive_lane0(&sm.item_full[is]);
        const int *table = p.c.table + (size_t)b * p.c.max_blocks;
        int bad = 0;
#pragma unroll 1
        for (int k0 = 0; k0 < tiles * kTile; k0 += kChunkKeys) {
            if (!wait4(&sm.rows_empty[slot], phase ^ 1, sm)) return;
            int *rows = sm.row[slot];
            {  // (items begin at multiples of 64: a lane has the sixteen keys of a block)
                const int k = k0 + lane * PILLAR_KV_BLOCK, pos = (itm.begin + k) / PILLAR_KV_BLOCK;
                int row = -1;
                if (k < n) {
                    const int blk = pos < p.c.max_blocks ? __ldg(table + pos) : -1;
                    if (blk >= 0 && blk < p.c.num_blocks) row = (blk * p.Hkv + g) * PILLAR_KV_BLOCK;
                    else bad |= PILLAR_FLAG_SLOT;
                }
                const int m = row >= 0 ? n - k : 0;
#pragma unroll
                for (int e = 0; e < PILLAR_KV_BLOCK; e += 4)
                    *reinterpret_cast<int4 *>(rows + lane * PILLAR_KV_BLOCK + e) =
                        make_int4(e < m ? row + e : -1, e + 1 < m ? row + e + 1 : -1, e + 2 < m ? row + e + 2 : -1,
                                  e + 3 < m ? row + e + 3 : -1);
            }
            if (lane == 0) sm.chunk_tiles[slot] = min(kChunkTiles, tiles - k0 / kTile);
            arrive_lane0(&sm.rows_full[slot]);
            if (++slot == kChunks) slot = 0, phase ^= 1;
        }
        if (bad) atomicOr(&p.hdr->err, bad);
    }
}

// ------------------------------------------------------------------ K and V warps

// Shared-memory accesses at an address and a constant.
template <int kOff>
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4+%5];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at), "n"(kOff));
    return v;
}
template <int kOff>
__device__ __forceinline__ void sts128(uint32_t at, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.u32 [%0+%5], {%1, %2, %3, %4};" ::"r"(at), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "n"(kOff) : "memory");
}

// Warp w of the four that turn K (or V) into operands: keys 32 w .. 32 w + 31 of every tile, from the copies on.  (Code is kept
// small here and below, rolled where it can be: the roles run at once and share the instruction cache.)
template <int D, bool kValue>
__device__ void convert4(const Kv4Params &p, Smem4<D> &sm, uint32_t tm, int w, int lane) {
    using S = Smem4<D>;
    constexpr int RC = S::kRow / 16;  // 16-byte pieces of a row of codes
    const int key = 32 * w + lane;
    // Piece c of row r lies at c ^ flip(r): eight lanes that read eight rows' pieces c meet no bank twice.  A lane copies piece
    // lane % RC of rows lane / RC + i * 32 / RC, whose flip is the same for all i.
    auto flip = [](int r) { return RC == 4 ? (r >> 1) & 3 : (r >> 2) & 1; };
    const int c = lane % RC, r0 = lane / RC;
    const uint8_t *codes = (kValue ? p.c.v4 : p.c.k4) + c * 16, *scales = kValue ? p.c.v_scale : p.c.k_scale;
    const uint32_t to_codes = smem_u32(sm.codes[kValue][0] + (32 * w + r0) * S::kRow + ((c ^ flip(r0)) << 4));
    const uint32_t to_scales = smem_u32(sm.scales[kValue][0] + key * S::kScales);
    const uint32_t from = smem_u32(sm.codes[kValue][0] + key * S::kRow + (flip(key) << 4));
    const uint32_t out = smem_u32(sm.v[0] + key * 128 + ((key & 7) << 4));
    int slot = 0, at = 0, tiles = 0;  // the chunk that loads go through: its slot, tile and tiles
    uint32_t phase = 0;
    int issued = 0;
    bool more = true;
#pragma unroll 1
    for (int x = -kStages; x < 0 || x < issued; ++x) {  // (four tiles ahead)
        const uint32_t st = (uint32_t)x % kStages;
        uint4 y[RC];
        uint32_t sc[2] = {0, 0};
        if (x >= 0) {
            copies_wait<kStages - 1>();
            __syncwarp();
            const uint32_t src = from + st * (kTile * S::kRow);
#pragma unroll
            for (int i = 0; i < RC; ++i) y[i] = lds128<0>(src ^ (i << 4));
            const uint32_t *sp = reinterpret_cast<const uint32_t *>(sm.scales[kValue][st] + key * S::kScales);
            if (D == 128) {
                const uint2 z = *reinterpret_cast<const uint2 *>(sp);
                sc[0] = z.x, sc[1] = z.y;
            } else {
                sc[0] = *sp;
            }
            __syncwarp();
        }
        if (more && at == tiles) {
            tiles = wait4(&sm.rows_full[slot], phase, sm) ? sm.chunk_tiles[slot] : 0;
            at = 0;
            more = tiles > 0;
        }
        if (more) {
            const uint32_t rows = smem_u32(sm.row[slot] + at * kTile + 32 * w), mine = rows + r0 * 4, dst = to_codes + st * (kTile * S::kRow);
            constexpr int RP = 32 / RC;  // (the codes of a key that is not there: any, its scales are 0)
            copy16<0>(dst, codes + (size_t)(uint32_t)max(lds_int<0>(mine), 0) * S::kRow);
            copy16<RP * S::kRow>(dst, codes + (size_t)(uint32_t)max(lds_int<4 * RP>(mine), 0) * S::kRow);
            if (RC == 4) {
                copy16<2 * RP * S::kRow>(dst, codes + (size_t)(uint32_t)max(lds_int<8 * RP>(mine), 0) * S::kRow);
                copy16<3 * RP * S::kRow>(dst, codes + (size_t)(uint32_t)max(lds_int<12 * RP>(mine), 0) * S::kRow);
            }
            const int row = lds_int<0>(rows + lane * 4);
            copy_small<S::kScales>(to_scales + st * (kTile * S::kScales), scales + (size_t)(uint32_t)max(row, 0) * S::kScales,
                                   row >= 0 ? S::kScales : 0);
            ++issued;
            if (++at == tiles) {
                arrive_lane0(&sm.rows_empty[slot]);
                if (++slot == kChunks) slot = 0, phase ^= 1;
            }
        }
        copies_commit();
        if (x < 0) continue;
        const int buf = x & 1;
        // the operand's buffer is free: the scores (the outputs) of the tile before last are done
        if (!wait4(kValue ? &sm.pv_done[buf] : &sm.s_full[buf], (x >> 1 & 1) ^ 1, sm)) break;
        tc_fence_after();
        const uint32_t into = out + buf * (kTile * D * 2), columns = tm + ((uint32_t)w << 21) + kTmemK + buf * 64;
#pragma unroll
        for (int i = 0; i < RC; ++i) {
            const uint32_t word[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
            uint32_t h[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f16_of_e2m1(word[e], h[e]);
                const uint32_t s = scale_pair(sc[i >> 1], (2 * i + (e >> 1)) & 3);
#pragma unroll
                for (int d = 0; d < 4; ++d) h[e][d] = mul_f16x2(h[e][d], s);
            }
            if (kValue) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t to = into ^ (((i & 1) * 4 + e) << 4);
                    if (i < 2) sts128<0>(to, h[e]);
                    else sts128<kTile * 128>(to, h[e]);
                }
            } else {
                tmem_st16(columns + i * 16, &h[0][0]);
            }
        }
        if (kValue) {
            fence_proxy_async_smem();
        } else {
            tmem_wait_st();
            tc_fence_before();
        }
        arrive_lane0(kValue ? &sm.v_full[buf] : &sm.k_full[buf]);
    }
    copies_wait<0>();
}

// ------------------------------------------------------------------ products

constexpr uint32_t kId4 = (1u << 4) | ((uint32_t)(kTile >> 4) << 24);  // f16 operands, fp32 sums, M = 128; N / 8 from bit 17 on

// K-step descriptors of the 32-byte-swizzled P operand: rows (N) contiguous, 16 of them 32 bytes a key; groups of 16 rows
// 4096 bytes apart, of 8 keys 256.
__device__ __forceinline__ uint64_t p_desc(uint32_t saddr) { return umma_sdesc(saddr, kTile * 32, 256) | ((uint64_t)6 << 61); }

// Every product has completed before its thread lets the tensor memory be freed.
template <int D>
__device__ __forceinline__ void drain4(Smem4<D> &sm, int which) {
    umma_commit(&sm.drain[which]);
    const unsigned long long t0 = global_timer_ns();
#pragma unroll 1
    while (!mbar_try_wait(&sm.drain[which], 0))
        if (global_timer_ns() - t0 > kWaitTimeoutNs) break;
}

// S^T of every tile.  (The products of a tile take 250 and 440 cycles, O^T's waiting for its operands in shared memory; one warp
// for both, with the tests of its waits between them, took 1900 a tile.)
template <int D>
__device__ void scores4(const Kv4Params &p, Smem4<D> &sm, uint32_t tm) {
    const uint32_t id = kId4 | ((uint32_t)(p.M + 15) / 16 << 18);
    uint32_t x = 0;
#pragma unroll 1
    for (int i = 0;; ++i) {
        const int is = i % kItems;
        if (!watch4(&sm.item_full[is], i / kItems & 1, &sm.item_full[is], i / kItems & 1, sm, p.wait_ns)) break;
        // (a reduction leaves its result in a uniform register, as the products' operands have to be)
        const int tiles = __reduce_or_sync(0xffffffffu, (unsigned)(sm.item[is].stop ? 0 : sm.item[is].tiles));
        if (tiles == 0) break;
        arrive_lane0(&sm.item_empty[is]);
        if (!watch4(&sm.q_full[i & 1], i >> 1 & 1, &sm.q_full[i & 1], i >> 1 & 1, sm, p.wait_ns)) break;
        const uint64_t dq = umma_sdesc_sw128(smem_u32(sm.q[i & 1]), 16, 1024);
        int t = 0;
#pragma unroll 1
        for (; t < tiles; ++t, ++x) {
            const int b = x & 1;
            const uint32_t ph = x >> 1 & 1;
            // (the scores of the tile before last have been read: its P is there)
            if (!watch4(&sm.k_full[b], ph, &sm.p_full[b], ph ^ 1, sm, p.wait_ns)) break;
            tc_fence_after();
            if (elect_one4()) {
#pragma unroll
                for (int ks = 0; ks < D / 16; ++ks)
                    umma_bf16_ts(tm + kTmemS + b * 64, tm + kTmemK + b * 64 + ks * 8,
                                 dq + (uint64_t)((ks >> 2) * (kMaxRows * 128 / 16) + (ks & 3) * 2), id, ks > 0 ? 1u : 0u);
                umma_commit(&sm.s_full[b]);
                if (t + 1 == tiles) umma_commit(&sm.q_empty[i & 1]);
            }
            __syncwarp();
        }
        if (t < tiles) break;
    }
    if (x > 0 && elect_one4()) drain4(sm, 0);
    __syncwarp();
}

// O^T of every tile.
template <int D>
__device__ void outputs4(const Kv4Params &p, Smem4<D> &sm, uint32_t tm) {
    const uint32_t id = kId4 | (1u << 15) | (1u << 16) | ((uint32_t)(p.M + 15) / 16 << 18);
    uint32_t x = 0;
#pragma unroll 1
    for (int i = 0;; ++i) {
        const int is = i % kItems;
        if (!watch4(&sm.item_full[is], i / kItems & 1, &sm.item_full[is], i / kItems & 1, sm, p.wait_ns)) break;
        const int tiles = __reduce_or_sync(0xffffffffu, (unsigned)(sm.item[is].stop ? 0 : sm.item[is].tiles));
        if (tiles == 0) break;
        arrive_lane0(&sm.item_empty[is]);
        // (the item before has been written: O is not kept twice)
        if (i > 0 && !watch4(&sm.o_empty[(i & 1) ^ 1], (i - 1) >> 1 & 1, &sm.o_empty[(i & 1) ^ 1], (i - 1) >> 1 & 1, sm, p.wait_ns)) break;
        int t = 0;
#pragma unroll 1
        for (; t < tiles; ++t, ++x) {
            const int b = x & 1;
            const uint32_t ph = x >> 1 & 1;
            if (!watch4(&sm.v_full[b], ph, &sm.p_full[b], ph, sm, p.wait_ns)) break;
            tc_fence_after();
            if (elect_one4()) {
                // V: M (dimensions) in halves of 64; for D = 64 the second half is whatever follows, and nobody reads its O
                const uint64_t dv = umma_sdesc_sw128(smem_u32(sm.v[b]), kTile * 128, 1024), dp = p_desc(smem_u32(sm.p[b]));
                const uint32_t to = tm + kTmemO + b * 64, add = t > 1;
#pragma unroll
                for (int ks = 0; ks < kTile / 16; ++ks)
                    umma_bf16(to, dv + (uint64_t)(ks * 128), dp + (uint64_t)(ks * 32), id, ks > 0 ? 1u : add);
                umma_commit(&sm.pv_done[b]);
                if (t + 1 == tiles) umma_commit(&sm.o_full[i & 1]);
            }
            __syncwarp();
        }
        if (t < tiles) break;
    }
    if (x > 0 && elect_one4()) drain4(sm, 1);
    __syncwarp();
}

// ------------------------------------------------------------------ softmax warps

// True when it is for any thread of the group (which all reach it).
__device__ __forceinline__ bool group_any(int grp, bool x) {
    uint32_t y;
    asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %2, 0;\n\tbarrier.cta.red.or.pred q, %1, 128, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
                 : "=r"(y)
                 : "r"(grp + 1), "r"((uint32_t)x)
                 : "memory");
    return y != 0;
}
__device__ __forceinline__ float warp_max(float x) {  // (a NaN is passed over)
    float y;
    asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
    return y;
}

// (Without a clobber of memory: other loads need not wait for it.)
__device__ __forceinline__ void store_global(float *dst, float v) { asm volatile("st.global.f32 [%0], %1;" ::"l"(dst), "f"(v)); }
__device__ __forceinline__ void load8(const float *src, float *v) {
    const float4 a = reinterpret_cast<const float4 *>(src)[0], b = reinterpret_cast<const float4 *>(src)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

// Eight rows' scores of a thread's key, with those that do not count at -inf.
struct Key4 {
    bool there, part;  // there is such a key; some row does not see it
    int pos;
};
__device__ __forceinline__ void scores8(uint32_t taddr, const Key4 &k, const int *lim, float (&s)[8]) {
    tmem_ld8(taddr, s);
    tmem_wait_ld();
    if (k.part) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (!k.there || k.pos > lim[e]) s[e] = neg_inf();
    }
}

// Group `half` of set `set`; its chunk ch is rows [8 half + 16 ch, + 8).
template <int D>
__device__ void softmax4(const Kv4Params &p, Smem4<D> &sm, uint32_t tm, int grp, int w, int lane) {
    const int key = 32 * w + lane, set = grp >> 1, half = grp & 1;
    const uint32_t quad = tm + ((uint32_t)w << 21) + set * 64 + half * 8;
    const int rows = p.M, nch = ((rows + 7) / 8 - half + 1) / 2;
    const int mine = 8 * half + 16 * (lane >> 3) + (lane & 7);  // the row that this lane looks after
    uint32_t x = 0;  // tile
    int slot = 0;    // of the chunk
    uint32_t phase = 0;
    bool dead = false;  // a wait has given up: the group leaves together, at its next vote
#pragma unroll 1
    for (int i = 0;; ++i) {
        const int is = i % kItems, sl = i & 1;
        dead |= !wait4(&sm.item_full[is], i / kItems & 1, sm);
        if (group_any(grp, dead)) return;
        const ItemRec &rec = sm.item[is];
        if (rec.stop) return;
        const int tiles = rec.tiles, last = rec.n - key;  // (the key is there in tiles that begin before `last`)
        const int sure = rec.L - (p.k + 1);               // every row sees up to here
        dead |= !wait4(&sm.fac_full[is], i / kItems & 1, sm);
        dead |= !wait4(&sm.epi_empty[sl], (i >> 1 & 1) ^ 1, sm);
        const float *fac2 = sm.fac2[is] + 8 * half;
        const int *lim = sm.lim[is] + 8 * half;
        float *nref = sm.nref[sl][set] + 8 * half;
        float m = neg_inf();  // the reference maximum of row `mine`, in every warp
        bool fresh = true, first = true;  // some row has none yet; nothing has been added to O
        {
            const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
            for (int ch = 0; ch < nch; ++ch) tmem_st8(quad + kTmemL + 16 * ch, zero);
            tmem_wait_st();
            if (w == 0 && mine < kMaxRows) sm.nref[sl][set][mine] = kLift;
        }
        Key4 kk;
        kk.pos = rec.begin + key;
        const long long row_logits = rec.L;
        float *logits = p.logits + (rec.logit_off + ((long long)rec.g * rows + 8 * half) * row_logits + kk.pos);  // of row 8 half
#pragma unroll 1
        for (int t = 0; t < tiles; ++t, ++x, kk.pos += kTile, logits += kTile) {
            if (t % kChunkTiles == 0) dead |= !wait4(&sm.rows_full[slot], phase, sm);
            kk.there = sm.row[slot][t % kChunkTiles * kTile + key] >= 0;
            if (t % kChunkTiles == kChunkTiles - 1 || t == tiles - 1) {
                arrive_lane0(&sm.rows_empty[slot]);
                if (++slot == kChunks) slot = 0, phase ^= 1;
            }
            if ((x & 1) != set) continue;
            const uint32_t ph = x >> 1 & 1;
            kk.part = !kk.there || kk.pos > sure;
            dead |= !wait4(&sm.s_full[set], ph, sm);
            tc_fence_after();
            float most = neg_inf();
#pragma unroll 1
            for (int ch = 0; ch < nch; ++ch) {
                float s[8], f[8], r[8];
                load8(fac2 + 16 * ch, f);
                load8(nref + 16 * ch, r);
                scores8(quad + kTmemS + 16 * ch, kk, lim + 16 * ch, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) most = fmaxf(most, fmaf(s[e], f[e], r[e]));
            }
            if (group_any(grp, most > kGrow || fresh || dead)) {  // rare: new reference maxima
                if (group_any(grp, dead)) return;
                float mx = neg_inf();
#pragma unroll 1
                for (int ch = 0; ch < nch; ++ch) {
                    float s[8], f[8];
                    load8(fac2 + 16 * ch, f);
                    scores8(quad + kTmemS + 16 * ch, kk, lim + 16 * ch, s);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = warp_max(s[e] * f[e]);
                        if (lane == ch * 8 + e) mx = y;
                    }
                }
                sm.top[grp][w][lane] = mx;
                if (!first) {  // what has been added to O so far is done: its rows are scaled below
                    dead |= !wait4(&sm.pv_done[set], ph ^ 1, sm);
                    tc_fence_after();
                }
                group_any(grp, false);
                mx = fmaxf(fmaxf(sm.top[grp][0][lane], sm.top[grp][1][lane]), fmaxf(sm.top[grp][2][lane], sm.top[grp][3][lane]));
                // (a row's reference goes by its own scores alone: one whose scores stayed within the bound keeps its)
                const float to_m = m == neg_inf() || mx > m + (kGrow - kLift) ? fmaxf(mx, m) : m;
                const float f = m == neg_inf() || to_m == m ? 1.f : ex2_approx(m - to_m);
                m = to_m;
                if (w == 0 && lane < 8 * nch) sm.nref[sl][set][mine] = kLift - (m == neg_inf() ? 0.f : m);
                fresh = __any_sync(0xffffffffu, lane < 8 * nch && mine < rows && m == neg_inf());
                if (!first) {
#pragma unroll 1
                    for (int ch = 0; ch < nch; ++ch) {
                        float o[8], l[8];
                        tmem_ld8(quad + kTmemO + 16 * ch, o);
                        tmem_ld8(quad + kTmemL + 16 * ch, l);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float fe = __shfl_sync(0xffffffffu, f, ch * 8 + e);
                            l[e] *= fe;
                            o[e] *= fe;
                        }
                        tmem_st8(quad + kTmemO + 16 * ch, o);
                        tmem_st8(quad + kTmemL + 16 * ch, l);
                    }
                    tmem_wait_st();
                }
                group_any(grp, false);
            }
            first = false;
            dead |= !wait4(&sm.pv_done[set], ph ^ 1, sm);  // the P of this set's tile before has been read
            uint8_t *dst = sm.p[set] + key * 32 + ((half ^ ((key >> 2) & 1)) << 4);
            const bool dump = p.logits && t * kTile < last;
#pragma unroll 1
            for (int ch = 0; ch < nch; ++ch) {
                float s[8], f[8], r[8], l[8];
                load8(fac2 + 16 * ch, f);
                load8(nref + 16 * ch, r);
                tmem_ld8(quad + kTmemL + 16 * ch, l);
                scores8(quad + kTmemS + 16 * ch, kk, lim + 16 * ch, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    r[e] = ex2_approx(fmaf(s[e], f[e], r[e]));
                    l[e] += r[e];
                }
                tmem_st8(quad + kTmemL + 16 * ch, l);
                *reinterpret_cast<uint4 *>(dst + ch * (kTile * 32)) =
                    make_uint4(pack_f16x2(r[0], r[1]), pack_f16x2(r[2], r[3]), pack_f16x2(r[4], r[5]), pack_f16x2(r[6], r[7]));
                if (dump) {
                    const int r0 = 8 * half + 16 * ch;
                    float *to = logits + 16 * ch * row_logits;
                    load8(sm.fac[is] + r0, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e, to += row_logits)
                        if (r0 + e < rows) store_global(to, s[e] * f[e]);
                }
            }
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            arrive_lane0(&sm.p_full[set]);
        }
        // the sums of weights over the warp's keys: of eight rows at a time, each lane ends up with one
#pragma unroll 1
        for (int ch = 0; ch < nch; ++ch) {
            float l[8], z;
            tmem_ld8(quad + kTmemL + 16 * ch, l);
            tmem_wait_ld();
#pragma unroll
            for (int h = 16, k = 4; k; h >>= 1, k >>= 1)
#pragma unroll
                for (int e = 0; e < k; ++e) {
                    const bool up = lane & h;
                    const float keep = up ? l[k + e] : l[e], give = up ? l[e] : l[k + e];
                    l[e] = keep + __shfl_xor_sync(0xffffffffu, give, h);
                }
            z = l[0];
            z += __shfl_xor_sync(0xffffffffu, z, 2);
            z += __shfl_xor_sync(0xffffffffu, z, 1);
            if ((lane & 3) == 0)
                sm.sum[sl][set][w][8 * half + 16 * ch + (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1)] = z;
        }
        arrive_lane0(&sm.epi_full[sl]);
        arrive_lane0(&sm.item_empty[is]);
    }
}

// ------------------------------------------------------------------ query warp

// The f16 query operands of an item (four rows at a time) and what the softmax warps know about its rows.
template <int D>
__device__ void queries4(const Kv4Params &p, Smem4<D> &sm, int lane) {
    constexpr int W = D / 64;  // words of a lane
#pragma unroll 1
    for (int i = 0;; ++i) {
        const int is = i % kItems;
        if (!wait4(&sm.item_full[is], i / kItems & 1, sm)) return;
        const ItemRec rec = sm.item[is];
        if (rec.stop) return;
        if (!wait4(&sm.q_empty[i & 1], (i >> 1 & 1) ^ 1, sm)) return;
#pragma unroll 1
        for (int r0 = 0; r0 < (p.M + 7) / 8 * 8; r0 += 4) {
            // (lane l looks after row r0 + l % 4)
            const int my = r0 + (lane & 3), gi = my / (p.k + 1), j = my - gi * (p.k + 1);
            const int at = my < p.M ? (rec.q_off + j) * p.Hq + rec.g * p.G + gi : -1;
            uint32_t x[4][W], mine = 0;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int row = __shfl_sync(0xffffffffu, at, e);
#pragma unroll
                for (int a = 0; a < W; ++a) x[e][a] = 0;
                if (row >= 0) {
                    const uint32_t *src = reinterpret_cast<const uint32_t *>(p.q + (size_t)row * D) + lane * W;
                    if (W == 2) {
                        const uint2 y = __ldg(reinterpret_cast<const uint2 *>(src));
                        x[e][0] = y.x, x[e][W - 1] = y.y;
                    } else {
                        x[e][0] = __ldg(src);
                    }
                }
            }
            uint8_t *dst = sm.q[i & 1] + (lane * W / 32) * (kMaxRows * 128) + r0 * 128 + lane * W % 4 * 4;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                uint32_t mx = x[e][0] & 0x7fff7fffu;
                if (W == 2) mx = __vmaxu2(mx, x[e][W - 1] & 0x7fff7fffu);
                mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
                if ((lane & 3) == e) mine = mx;
                float up, down;
                query_scale(mx, &up, &down);
                uint8_t *to = dst + e * 128 + (((lane * W % 32 / 4) ^ ((r0 + e) & 7)) << 4);
                if (W == 2)
                    *reinterpret_cast<uint2 *>(to) = make_uint2(pack_f16x2(bf16lo(x[e][0]) * up, bf16hi(x[e][0]) * up),
                                                                pack_f16x2(bf16lo(x[e][W - 1]) * up, bf16hi(x[e][W - 1]) * up));
                else
                    *reinterpret_cast<uint32_t *>(to) = pack_f16x2(bf16lo(x[e][0]) * up, bf16hi(x[e][0]) * up);
            }
            if (lane < 4) {
                float up, down;
                query_scale(mine, &up, &down);
                const float fac = fmaxf(down * p.scale, __int_as_float(1));  // (above 0: a masked score stays -inf)
                sm.fac[is][my] = fac;
                const int lim = my < p.M ? rec.L - (p.k + 1) + j : 0x7fffffff;
                sm.fac2[is][my] = softmax_factor(fac, mine, lim);
                sm.lim[is][my] = lim;
            }
        }
        fence_proxy_async_smem();
        arrive_lane0(&sm.q_full[i & 1]);
        arrive_lane0(&sm.fac_full[is]);
        arrive_lane0(&sm.item_empty[is]);
    }
}

// ------------------------------------------------------------------ epilogue warps

template <int D>
__device__ void epilogue4(const Kv4Params &p, Smem4<D> &sm, uint32_t tm, int w, int lane) {
    const int d = 32 * w + lane;
#pragma unroll 1
    for (int i = 0;; ++i) {
        const int is = i % kItems, sl = i & 1;
        if (!wait4(&sm.item_full[is], i / kItems & 1, sm)) return;
        const ItemRec rec = sm.item[is];
        if (rec.stop) return;
        if (!wait4(&sm.epi_full[sl], i >> 1 & 1, sm) || !wait4(&sm.o_full[sl], i >> 1 & 1, sm)) return;
        tc_fence_after();
        const bool whole = rec.nsplit == 1;
#pragma unroll 1
        for (int h = 0; h < p.M; h += 32) {
            // row h + lane: where it goes (-1: there is none), and what the sets' O are multiplied by
            const int r = h + lane, gi = r / (p.k + 1), j = r - gi * (p.k + 1);
            int at = -1;
            float f0 = 0.f, f1 = 0.f;
            if (r < p.M) {
                at = whole ? (rec.q_off + j) * p.Hq + rec.g * p.G + gi : rec.rec + j * p.G + gi;
                const float *s0 = &sm.sum[sl][0][0][r], *s1 = &sm.sum[sl][1][0][r];
                const float l0 = s0[0] + s0[kMaxRows] + s0[2 * kMaxRows] + s0[3 * kMaxRows], ref0 = -sm.nref[sl][0][r];
                const float l1 = s1[0] + s1[kMaxRows] + s1[2 * kMaxRows] + s1[3 * kMaxRows], ref1 = -sm.nref[sl][1][r];
                // (a sum of 0 has no reference)
                const float ref = l0 == 0.f ? ref1 : l1 == 0.f ? ref0 : fmaxf(ref0, ref1);
                f0 = l0 == 0.f ? 0.f : ex2_approx(ref0 - ref);
                f1 = l1 == 0.f ? 0.f : ex2_approx(ref1 - ref);
                const float l = __fadd_rn(__fmul_rn(l0, f0), __fmul_rn(l1, f1));  // (the same whichever set began)
                const float inv = l == 0.f ? 0.f : __frcp_rn(l);
                // (what is 0 stays it under a NaN sum: an O that nobody wrote is not read)
                if (f0 != 0.f) f0 *= inv;
                if (f1 != 0.f) f1 *= inv;
                if (w == 0) {
                    const float z = l > 0.f ? ref * 0.69314718f + logf(l) : (l == 0.f ? neg_inf() : l);  // (a NaN sum stays one)
                    if (!whole) p.part_lse[at] = z;
                    else p.lse[(size_t)rec.vidx * p.Hq * (p.k + 1) + (size_t)rec.g * p.M + r] = z;
                }
            }
            // (an item of one tile has one O: the set that met no tile has sums of 0)
            const bool any0 = __any_sync(0xffffffffu, f0 != 0.f), any1 = __any_sync(0xffffffffu, f1 != 0.f);
#pragma unroll 1
            for (int r0 = 0; r0 < min(32, p.M - h); r0 += 8) {
                float o[8], o1[8];
                const uint32_t from = tm + ((uint32_t)w << 21) + kTmemO + h + r0;
                tmem_ld8(from, o);
                tmem_ld8(from + 64, o1);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float a0 = __shfl_sync(0xffffffffu, f0, r0 + e), a1 = __shfl_sync(0xffffffffu, f1, r0 + e);
                    const int row = __shfl_sync(0xffffffffu, at, r0 + e);
                    const float y = __fadd_rn(any0 ? __fmul_rn(o[e], a0) : 0.f, any1 ? __fmul_rn(o1[e], a1) : 0.f);
                    if (row >= 0 && d < D) {
                        const size_t to = (size_t)row * D + d;
                        if (whole) p.out[to] = (uint16_t)pack_bf16x2(y, 0.f);
                        else p.part_o[to] = y;
                    }
                }
            }
        }
        tc_fence_before();
        arrive_lane0(&sm.o_empty[sl]);
        arrive_lane0(&sm.epi_empty[sl]);
        arrive_lane0(&sm.item_empty[is]);
    }
}

// ------------------------------------------------------------------ kernel

template <int D>
__global__ void __launch_bounds__(kThreads4, 1) attn_kv4_kernel(const __grid_constant__ Kv4Params p) {
    extern __shared__ __align__(1024) char smem[];
    Smem4<D> &sm = *reinterpret_cast<Smem4<D> *>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, w = warp & 3;
    if (threadIdx.x == 0) {
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&sm.item_full[i], 1);
            mbar_init(&sm.item_empty[i], 4 * kGroups + 4 + 1 + 2);  // softmax, epilogue and query warps, the products' warps
            mbar_init(&sm.fac_full[i], 1);
        }
        for (int i = 0; i < kChunks; ++i) {
            mbar_init(&sm.rows_full[i], 1);
            mbar_init(&sm.rows_empty[i], 8 + 4 * kGroups);  // K, V and softmax warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 1);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.k_full[i], 4);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.p_full[i], 2 * kGroups);
            mbar_init(&sm.v_full[i], 4);
            mbar_init(&sm.pv_done[i], 1);
            mbar_init(&sm.o_full[i], 1);
            mbar_init(&sm.o_empty[i], 4);
            mbar_init(&sm.epi_full[i], 4 * kGroups);
            mbar_init(&sm.epi_empty[i], 4);
        }
        for (int i = 0; i < 2; ++i) mbar_init(&sm.drain[i], 1);
        sm.abort = 0;
        mbar_init_fence();
    }
    if (warp == 0) tmem_alloc(&sm.tmem, kTmemCols);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    pdl_wait_prerequisites();  // the plan's output is read only from here on
    pdl_launch_dependents();   // (the merge waits for this kernel's completion itself)
    const int wg = warp >> 2;
    if (wg < kGroups) {
        softmax4<D>(p, sm, tm, wg, w, lane);
    } else if (wg == kGroups) {
        convert4<D, false>(p, sm, tm, w, lane);
    } else if (wg == kGroups + 1) {
        convert4<D, true>(p, sm, tm, w, lane);
    } else if (wg == kGroups + 2) {
        if (w == 0) resolver4<D>(p, sm, lane);
        else if (w == 3) queries4<D>(p, sm, lane);
        else if (w == 1) scores4<D>(p, sm, tm);
        else outputs4<D>(p, sm, tm);
    } else {
        epilogue4<D>(p, sm, tm, w, lane);
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && sm.abort) atomicOr(&p.hdr->err, PILLAR_FLAG_TIMEOUT);
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm, kTmemCols);
    }
}

template <int D>
cudaError_t launch_t(const Kv4Params &p, int nsm, cudaStream_t st) {
    constexpr int kSmem = (int)sizeof(Smem4<D>);
    static unsigned long long configured[kMaxDevices] = {};
    int dev = 0;
    unsigned long long ctx = 0;
    cudaError_t e = current_device_context(&dev, &ctx);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (ctx == 0 || __atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE) != ctx) {
        e = cudaFuncSetAttribute(attn_kv4_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_kv4_kernel<D>, kThreads4, kSmem);
        if (e != cudaSuccess) return e;
        if (n != 1) return cudaErrorInvalidConfiguration;  // a CTA takes all of its SM's tensor memory
        e = current_device_context(&dev, &ctx);  // (the calls above made a context current)
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], ctx, __ATOMIC_RELEASE);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nsm);
    cfg.blockDim = dim3(kThreads4);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_kv4_kernel<D>, p);
}

}  // namespace

cudaError_t launch_attn_kv4(const AttnArgs &a, const Kv4Cache &c, bool whole, int nsm, cudaStream_t st) {
    Kv4Params p;
    p.q = a.q;
    p.c = c;
    p.sparse_idx = a.sparse_idx;
    p.out = a.out;
    p.logits = a.logits;
    p.lse = a.lse;
    p.hdr = reinterpret_cast<WsHeader *>(a.ws);
    p.req = reinterpret_cast<const ReqInfo *>(a.ws + a.lay.req);
    p.logit_off = reinterpret_cast<const long long *>(a.ws + a.lay.logit_off);
    p.unit = reinterpret_cast<const UnitInfo *>(a.ws + a.lay.unit);
    p.items = reinterpret_cast<const Item *>(a.ws + a.lay.items);
    p.part_o = reinterpret_cast<float *>(a.ws + a.lay.part_o);
    p.part_lse = reinterpret_cast<float *>(a.ws + a.lay.part_lse);
    p.B = a.B;
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.k = a.k;
    p.M = (a.k + 1) * p.G;
    p.max_sparse = a.max_sparse;
    p.scale = a.scale;
    p.wait_ns = a.wait_ns;
    // All items have at most eight rows, or those of verify requests go first, in a kernel whose CTAs the others take the place
    // of as these end.
    cudaError_t e = cudaSuccess;
    if (p.M <= 8 || a.schedule == PILLAR_SCHEDULE_DRAFT_ONLY) {
        e = launch_attn_kv4_few(p, a.D, 8, 0, false, nsm, st);
    } else {
        e = p.M <= (p.logits ? kFewRowsDumped : kFewRows) ? launch_attn_kv4_few(p, a.D, p.M, 1, false, nsm, st)
            : a.D == 128                                  ? launch_t<128>(p, nsm, st)
                                                          : launch_t<64>(p, nsm, st);
        if (e == cudaSuccess && a.schedule != PILLAR_SCHEDULE_VERIFY_ONLY) e = launch_attn_kv4_few(p, a.D, 8, 2, true, nsm, st);
    }
    // Nothing to merge where no item is split (two draft and two verify requests, as a graph: 22.6 us -> 20.7); the kernels of few rows have set the queues
    // up for the next run, which those of the many verify rows alone leave to the merge.
    const bool queues = p.M <= kFewRowsDumped || a.schedule != PILLAR_SCHEDULE_VERIFY_ONLY;
    return e == cudaSuccess && !(whole && queues) ? launch_merge(a, nsm, st) : e;
}

}  // namespace pillar
