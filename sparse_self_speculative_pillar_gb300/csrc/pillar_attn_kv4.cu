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
// One persistent CTA an SM, 128 keys a tile, the keys on the M of tcgen05:
//     S^T [keys x rows] = K Q^T      K from tensor memory, Q from shared memory
//     O^T [D x rows]   += V^T P^T    V and P from shared memory
// so that a key's row is made into an operand once, whatever the number of
// query rows, and a few rows (N is a multiple of 16) cost little.
//   * The resolver warp takes items from the planner's queue and turns their
//     keys into rows of the pools, 512 at a time.
//   * Four warps each for K and V copy the rows of the tiles ahead (16 bytes a
//     lane), turn a key's 64 bytes of codes into f16 and write them to tensor
//     memory (K: lane = key) or swizzled shared memory (V: keys x D, MN-major).
//   * One warp issues all products.
//   * Eight softmax warps, a key a thread: two groups of four that take tiles in
//     turn where an item has at most 16 rows (each with its own O and reference
//     maxima), and share the rows of every tile where it has more.  A reference
//     maximum moves only when a score passes it by more than 2^8, which a vote of
//     the group finds out.  P is rounded to f16 relative to it: weights are at
//     most 2^14, and 2^6 or more for a row's largest.
//   * Four warps write finished items, two stage queries.
#include "pillar_attn_kv4.cuh"

namespace pillar {

namespace {

constexpr int kTile = 128;                   // keys of a tile
constexpr int kChunkTiles = 4;               // tiles whose rows are resolved together
constexpr int kChunkKeys = kTile * kChunkTiles;
constexpr int kChunks = 3;                   // chunks in flight between the resolver and their readers
constexpr int kItems = 8;                    // items in flight
constexpr int kStages = 4;                   // tiles of codes in shared memory
constexpr int kWarps = 24;
constexpr int kThreads4 = kWarps * 32;
// tensor memory: two tiles of K, two of S^T, the O^T of two items, sums of weights (a key's lane, a column per row)
constexpr uint32_t kTmemCols = 512, kTmemK = 0, kTmemS = 128, kTmemO = 256, kTmemL = 384;

// A work item in shared memory.
struct alignas(16) ItemRec {
    int stop;               // no more items
    int tiles, rows, verify;
    int n, begin, L, g;     // keys; first one (verify: its position); context length; KV head
    int q_off, vidx, nsplit, rec;
    long long logit_off;
    int pad[2];
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
    // per query row: logit = sum * fac, in base-2 units sum * fac2; last position seen; its logits, or null
    alignas(16) float fac[kItems][kMaxRows], fac2[kItems][kMaxRows];
    int lim[kItems][kMaxRows];
    float *lb[kItems][kMaxRows];
    // per item (in turn), group and row of the group: kLift - reference maximum (base 2); sums of weights per warp
    alignas(16) float nref[2][2][32], sum[2][2][4][32];
    float top[2][4][32];                        // a group's largest scores, per warp
    uint64_t item_full[kItems], item_empty[kItems], fac_full[kItems];
    uint64_t rows_full[kChunks], rows_empty[kChunks];
    uint64_t q_full[2], q_empty[2], k_full[2], s_full[2], s_empty[2], p_full[2], v_full[2], pv_done[2];
    uint64_t o_full[2], o_empty[2], epi_full[2], epi_empty[2], drain;
    uint32_t tmem;
    int abort;  // a wait has given up
};
static_assert(sizeof(Smem4<128>) <= 227 * 1024, "shared memory of a CTA");
static_assert(sizeof(Smem4<64>) > 114 * 1024, "never two CTAs on an SM: each takes all of its tensor memory");

// A wait by a whole warp, a few instructions long (every wait that is inlined costs the roles' shared instruction cache; with
// the clock in each, plain decoding took 227 us where this took XXX).  The products' warp watches the clock for all: nothing
// moves in a CTA for long without it, and when it has had nothing to do for the bound it raises the abort flag.  A count of polls
// bounds the waits that outlive it.
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
constexpr int kRegsSoftmax = 104, kRegsConvert = 72, kRegsRest = 64;
static_assert(2 * kRegsSoftmax + 2 * kRegsConvert + 2 * kRegsRest <= kThreads4 / 128 * 80, "the registers at launch");

__device__ __forceinline__ void arrive_lane0(uint64_t *bar, uint32_t count = 1) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive_cnt(bar, count);
}
__device__ __forceinline__ bool elect_one4() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ bool test4(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_test_wait(bar, parity));
}

__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
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

// How an item's query rows are shared by the softmax groups: at most 16 rows, the groups take tiles in turn; else group 0
// has the first `first` chunks of eight rows and group 1 the others.
__device__ __forceinline__ bool takes_turns(int rows) { return rows <= 16; }
__device__ __forceinline__ int first_chunks(int rows) { return ((rows + 7) / 8 + 1) / 2; }

// ------------------------------------------------------------------ resolver warp

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
            if (!wait4(&sm.rows_empty[slot], phase ^ 1, sm)) return;
            if (lane == 0) sm.chunk_tiles[slot] = 0;
            arrive_lane0(&sm.rows_full[slot]);
            return;
        }
        const Item itm = p.items[it];
        const int b = itm.unit / p.Hkv, g = itm.unit - b * p.Hkv;
        const ReqInfo ri = p.req[b];
        const UnitInfo ui = p.unit[itm.unit];
        const bool verify = ri.mode == 1;
        const int n = itm.end - itm.begin, tiles = max(1, (n + kTile - 1) / kTile);
        if (lane == 0) {
            ItemRec r;
            r.stop = 0;
            r.tiles = tiles;
            r.rows = verify ? p.M : p.G;
            r.verify = verify;
            r.n = n;
            r.begin = itm.begin;
            r.L = ri.len;
            r.g = g;
            r.q_off = ri.q_off;
            r.vidx = ri.vidx;
            r.nsplit = ui.nsplit;
            r.rec = ui.rec_base + itm.split * ui.rec_rows;
            r.logit_off = verify ? p.logit_off[b] : 0;
            sm.item[is] = r;
        }
        arrive_lane0(&sm.item_full[is]);
        const int *list = p.sparse_idx + ((size_t)b * p.Hkv + g) * p.max_sparse + itm.begin;
        const int *table = p.c.table + (size_t)b * p.c.max_blocks;
        int bad = 0;
#pragma unroll 1
        for (int k0 = 0; k0 < tiles * kTile; k0 += kChunkKeys) {
            if (!wait4(&sm.rows_empty[slot], phase ^ 1, sm)) return;
            int *rows = sm.row[slot];
            if (verify) {  // (items begin at multiples of 64: a lane has the sixteen keys of a block)
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
            } else {
                // (the loads without conditions, eight in flight: past the end, and for bad positions, of a key that there is)
#pragma unroll 1
              for (int k1 = 0; k1 < kChunkKeys && k0 + k1 < tiles * kTile; k1 += 256) {
                int pos[8], blk[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) pos[e] = n > 0 ? __ldg(list + min(k0 + k1 + e * 32 + lane, n - 1)) : -1;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if ((unsigned)pos[e] >= (unsigned)ri.len) bad |= PILLAR_FLAG_INDEX * (n > 0), pos[e] = -1;
                    blk[e] = __ldg(table + min((unsigned)max(pos[e], 0) / PILLAR_KV_BLOCK, (unsigned)p.c.max_blocks - 1));
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    int row = -1;
                    if (pos[e] >= 0) {
                        if ((unsigned)blk[e] < (unsigned)p.c.num_blocks && pos[e] / PILLAR_KV_BLOCK < p.c.max_blocks)
                            row = (blk[e] * p.Hkv + g) * PILLAR_KV_BLOCK + pos[e] % PILLAR_KV_BLOCK;
                        else bad |= PILLAR_FLAG_SLOT;
                    }
                    rows[k1 + e * 32 + lane] = k0 + k1 + e * 32 + lane < n ? row : -1;
                }
              }
            }
            if (lane == 0) sm.chunk_tiles[slot] = min(kChunkTiles, tiles - k0 / kTile);
            arrive_lane0(&sm.rows_full[slot]);
            if (++slot == kChunks) slot = 0, phase ^= 1;
        }
        if (bad) atomicOr(&p.hdr->err, bad);
    }
}

// ------------------------------------------------------------------ K and V warps

// Warp w of K's (or V's) four: keys 32 w .. 32 w + 31 of every tile, from the copies to the operand.  (Code is kept small here
// and below, rolled where it can be: the roles run at once and share the instruction cache.)
template <int D, bool kValue>
__device__ void convert4(const Kv4Params &p, Smem4<D> &sm, uint32_t tm, int w, int lane) {
    using S = Smem4<D>;
    constexpr int RC = S::kRow / 16;                            // 16-byte pieces of a row of codes
    const uint8_t *codes = kValue ? p.c.v4 : p.c.k4, *scales = kValue ? p.c.v_scale : p.c.k_scale;
    const int key = 32 * w + lane;
    // piece c of row r lies at c ^ flip(r): eight lanes that read eight rows' pieces c meet no bank twice
    auto flip = [](int r) { return RC == 4 ? (r >> 1) & 3 : (r >> 2) & 1; };
    int slot = 0, at = 0, tiles = 0;  // the chunk that loads go through: its slot, tile and tiles (0: the next one has to come)
    uint32_t phase = 0;
    int issued = 0;
    bool more = true, ok = true;
#pragma unroll 1
    for (int x = 1 - kStages; ok; ++x) {
        // the loads of tile x + kStages - 1
        if (more && at == tiles) {
            ok = wait4(&sm.rows_full[slot], phase, sm);
            tiles = ok ? sm.chunk_tiles[slot] : 0;
            at = 0;
            more = tiles > 0;
        }
        if (more) {
            const int st = issued % kStages;
            const int *rows = sm.row[slot] + at * kTile + 32 * w;
            const uint32_t dst = smem_u32(sm.codes[kValue][st] + 32 * w * S::kRow);
            const int c = lane % RC;
#pragma unroll
            for (int i = 0; i < RC; ++i) {
                const int r = i * (32 / RC) + lane / RC, row = rows[r];
                copy16(dst + r * S::kRow + ((c ^ flip(r)) << 4), codes + (size_t)max(row, 0) * S::kRow + c * 16, row >= 0 ? 16 : 0);
            }
            const int row = rows[lane];
            copy_small<S::kScales>(smem_u32(sm.scales[kValue][st] + key * S::kScales), scales + (size_t)max(row, 0) * S::kScales,
                                   row >= 0 ? S::kScales : 0);
            ++issued;
            if (++at == tiles) {
                arrive_lane0(&sm.rows_empty[slot]);
                if (++slot == kChunks) slot = 0, phase ^= 1;
            }
        }
        copies_commit();
        if (x < 0) continue;
        if (x == issued) break;
        copies_wait<kStages - 1>();
        __syncwarp();
        const int st = x % kStages, buf = x & 1;
        // the operand's buffer is free: the scores (the outputs) of the tile before last are done
        ok = wait4(kValue ? &sm.pv_done[buf] : &sm.s_full[buf], (x >> 1 & 1) ^ 1, sm);
        if (!ok) break;
        tc_fence_after();
        const uint8_t *src = sm.codes[kValue][st] + key * S::kRow;
        const uint8_t *sc = sm.scales[kValue][st] + key * S::kScales;
        uint8_t *dst = sm.v[buf] + key * 128;
#pragma unroll 1
        for (int i = 0; i < RC; ++i) {
            const uint4 y = *reinterpret_cast<const uint4 *>(src + ((i ^ flip(key)) << 4));
            const uint32_t two = *reinterpret_cast<const uint16_t *>(sc + 2 * i);
            const uint32_t s0 = scale_pair(two, 0), s1 = scale_pair(two, 1);
            const uint32_t word[4] = {y.x, y.y, y.z, y.w};
            uint32_t h[4][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                f16_of_e2m1(word[e], h[e]);
#pragma unroll
                for (int d = 0; d < 4; ++d) h[e][d] = mul_f16x2(h[e][d], e < 2 ? s0 : s1);
            }
            if (kValue) {
                uint8_t *half = dst + (i >> 1) * (kTile * 128);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    *reinterpret_cast<uint4 *>(half + ((((i & 1) * 4 + e) ^ (key & 7)) << 4)) =
                        make_uint4(h[e][0], h[e][1], h[e][2], h[e][3]);
            } else {
                tmem_st16(tm + ((uint32_t)w << 21) + kTmemK + buf * 64 + i * 16, &h[0][0]);
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

// ------------------------------------------------------------------ MMA warp

// K-step descriptors of the 32-byte-swizzled P operand: rows (N) contiguous, 16 of them 32 bytes a key; groups of 16 rows
// 4096 bytes apart, of 8 keys 256.
__device__ __forceinline__ uint64_t p_desc(uint32_t saddr) { return umma_sdesc(saddr, kTile * 32, 256) | ((uint64_t)6 << 61); }

template <int D>
__device__ void mma4(const Kv4Params &p, Smem4<D> &sm, uint32_t tm) {
    constexpr uint32_t kId = (1u << 4) | ((uint32_t)(kTile >> 4) << 24);  // f16 operands, fp32 sums, M = 128
    uint32_t vs = 0, vp = 0;            // tiles whose scores, whose outputs have been issued
    int si = 0, st = 0, sT = 0, sN = 0;  // scores: item, tile of it, its tiles (0: to come), its rows
    int oi = 0, ot = 0, oT = 0, orows = 0;
    bool stop = false, issued = false;
    unsigned long long idle = 0;
#pragma unroll 1
    for (uint32_t spin = 0;; ++spin) {
        bool progress = false;
        if (!stop && vs - vp < 2) {
            if (sT == 0 && test4(&sm.item_full[si % kItems], si / kItems & 1)) {
                const ItemRec &r = sm.item[si % kItems];
                if (r.stop) stop = true;
                else sT = r.tiles, sN = (r.rows + 15) / 16 * 16, st = 0;
            }
            const int b = vs & 1;
            if (sT > 0 && test4(&sm.k_full[b], vs >> 1 & 1) && test4(&sm.s_empty[b], (vs >> 1 & 1) ^ 1) &&
                (st > 0 || test4(&sm.q_full[si & 1], si >> 1 & 1))) {
                tc_fence_after();
                if (elect_one4()) {
                    const uint64_t dq = umma_sdesc_sw128(smem_u32(sm.q[si & 1]), 16, 1024);
                    const uint32_t id = kId | ((uint32_t)sN >> 3 << 17);
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        umma_bf16_ts(tm + kTmemS + b * 64, tm + kTmemK + b * 64 + ks * 8,
                                     dq + (uint64_t)((ks >> 2) * (kMaxRows * 128 / 16) + (ks & 3) * 2), id, ks > 0 ? 1u : 0u);
                    umma_commit(&sm.s_full[b]);
                    if (st + 1 == sT) umma_commit(&sm.q_empty[si & 1]);
                }
                __syncwarp();
                issued = progress = true;
                ++vs;
                if (++st == sT) sT = 0, ++si;
            }
        }
        if (vp < vs) {
            if (oT == 0) {  // (its scores have been issued: the record is there)
                const ItemRec &r = sm.item[oi % kItems];
                oT = r.tiles, orows = r.rows, ot = 0;
            }
            const int b = vp & 1;
            if (test4(&sm.p_full[b], vp >> 1 & 1) && test4(&sm.v_full[b], vp >> 1 & 1) &&
                (ot > 0 || test4(&sm.o_empty[oi & 1], (oi >> 1 & 1) ^ 1))) {
                tc_fence_after();
                const bool turns = takes_turns(orows), add = ot >= (turns ? 2 : 1);
                if (elect_one4()) {
                    // V: M (dimensions) in halves of 64; for D = 64 the second half is whatever follows, and nobody reads its O
                    const uint64_t dv = umma_sdesc_sw128(smem_u32(sm.v[b]), kTile * 128, 1024), dp = p_desc(smem_u32(sm.p[b]));
                    const uint32_t id = kId | (1u << 15) | (1u << 16) | ((uint32_t)((orows + 15) / 16 * 16) >> 3 << 17);
                    const uint32_t to = tm + kTmemO + (oi & 1) * 64 + (turns ? b * 16 : 0);
#pragma unroll
                    for (int ks = 0; ks < kTile / 16; ++ks)
                        umma_bf16(to, dv + (uint64_t)(ks * 128), dp + (uint64_t)(ks * 32), id, add || ks > 0 ? 1u : 0u);
                    umma_commit(&sm.pv_done[b]);
                    if (ot + 1 == oT) umma_commit(&sm.o_full[oi & 1]);
                }
                __syncwarp();
                progress = true;
                ++vp;
                if (++ot == oT) {
                    oT = 0;
                    arrive_lane0(&sm.item_empty[oi % kItems]);
                    ++oi;
                }
            }
        }
        if (stop && vp == vs) break;
        if (progress) {
            idle = 0;
            continue;
        }
        if ((spin & 63) == 0) {
            const unsigned long long now = global_timer_ns();
            if (idle == 0) idle = now;
            if (__any_sync(0xffffffffu, now - idle > p.wait_ns || *static_cast<volatile int *>(&sm.abort))) {
                *static_cast<volatile int *>(&sm.abort) = 1;
                break;
            }
        }
    }
    if (issued && elect_one4()) {  // every product has completed before the tensor memory is freed
        umma_commit(&sm.drain);
        const unsigned long long t0 = global_timer_ns();
        while (!mbar_try_wait(&sm.drain, 0))
            if (global_timer_ns() - t0 > kWaitTimeoutNs) break;
    }
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

// Eight rows' scores of a thread's key, with those that do not count at -inf.
struct Key4 {
    bool there, part;  // there is such a key; some row does not see it
    int pos;
    const int *lim;
};
__device__ __forceinline__ void scores8(uint32_t taddr, const Key4 &k, int ch, float (&s)[8]) {
    tmem_ld8(taddr + ch * 8, s);
    tmem_wait_ld();
    if (k.part) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            if (!k.there || k.pos > k.lim[ch * 8 + e]) s[e] = neg_inf();
    }
}
__device__ __forceinline__ void load8(const float *src, float (&v)[8]) {
    const float4 a = reinterpret_cast<const float4 *>(src)[0], b = reinterpret_cast<const float4 *>(src)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

template <int D>
__device__ void softmax4(const Kv4Params &p, Smem4<D> &sm, uint32_t tm, int grp, int w, int lane) {
    const int key = 32 * w + lane;
    const uint32_t quad = tm + ((uint32_t)w << 21);
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
        const int tiles = rec.tiles, rows = rec.rows, n = rec.n;
        const bool verify = rec.verify, turns = takes_turns(rows), dump = verify && p.logits;
        const int sure = verify ? rec.L - (p.k + 1) : 0x7fffffff;  // every row sees up to here
        const int c0 = !turns && grp ? 8 * first_chunks(rows) : 0;
        const int mine = !turns && !grp ? min(rows, 8 * first_chunks(rows)) : rows - c0, nch = (mine + 7) / 8;
        dead |= !wait4(&sm.fac_full[is], i / kItems & 1, sm);
        dead |= !wait4(&sm.epi_empty[sl], (i >> 1 & 1) ^ 1, sm);
        // Where both groups use both buffers, the other one is done with the item before: its tiles' phases are over, and a
        // wait for the next phase of a buffer that this group has not watched is one for the right one.
        if (!turns && i > 0) dead |= !wait4(&sm.epi_full[sl ^ 1], (i - 1) >> 1 & 1, sm);
        const float *fac2 = sm.fac2[is] + c0;
        float *nref = sm.nref[sl][grp];
        if (w == 0) nref[lane] = kLift;
        const uint32_t tl = quad + kTmemL + grp * 32, to = quad + kTmemO + sl * 64 + (turns ? grp * 16 : c0);
        float m = neg_inf();  // the reference maximum of row `lane` of the group, in every warp
        bool fresh = true, first = true;  // some row has none yet; nothing has been added to O
        Key4 kk;
        kk.pos = rec.begin + key;
        kk.lim = sm.lim[is] + c0;
#pragma unroll 1
        for (int t = 0; t < tiles; ++t, ++x, kk.pos += kTile) {
            if (t % kChunkTiles == 0) dead |= !wait4(&sm.rows_full[slot], phase, sm);
            kk.there = sm.row[slot][t % kChunkTiles * kTile + key] >= 0;
            if (t % kChunkTiles == kChunkTiles - 1 || t == tiles - 1) {
                arrive_lane0(&sm.rows_empty[slot]);
                if (++slot == kChunks) slot = 0, phase ^= 1;
            }
            const int b = x & 1;
            if (turns && b != grp) continue;
            const uint32_t ph = x >> 1 & 1, ts = quad + kTmemS + b * 64 + c0;
            kk.part = !kk.there || (verify && kk.pos > sure);
            dead |= !wait4(&sm.s_full[b], ph, sm);
            tc_fence_after();
            float most = neg_inf();
#pragma unroll 1
            for (int ch = 0; ch < nch; ++ch) {
                float s[8], f[8], r[8];
                load8(fac2 + ch * 8, f);
                load8(nref + ch * 8, r);
                scores8(ts, kk, ch, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) most = fmaxf(most, fmaf(s[e], f[e], r[e]));
            }
            if (group_any(grp, most > kGrow || fresh || dead)) {  // rare: new reference maxima
                if (group_any(grp, dead)) return;
                float mx = neg_inf();
#pragma unroll 1
                for (int ch = 0; ch < nch; ++ch) {
                    float s[8], f[8];
                    load8(fac2 + ch * 8, f);
                    scores8(ts, kk, ch, s);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float y = warp_max(s[e] * f[e]);
                        if (lane == ch * 8 + e) mx = y;
                    }
                }
                sm.top[grp][w][lane] = mx;
                if (!first) {  // what has been added to O so far is done: its rows are scaled below
                    const uint32_t y = turns ? x - 2 : x - 1;
                    dead |= !wait4(&sm.pv_done[y & 1], y >> 1 & 1, sm);
                    tc_fence_after();
                }
                group_any(grp, false);
                mx = fmaxf(fmaxf(sm.top[grp][0][lane], sm.top[grp][1][lane]), fmaxf(sm.top[grp][2][lane], sm.top[grp][3][lane]));
                // (a row's reference goes by its own scores alone: one whose scores stayed within the bound keeps its)
                const float to_m = m == neg_inf() || mx > m + (kGrow - kLift) ? fmaxf(mx, m) : m;
                const float f = m == neg_inf() || to_m == m ? 1.f : ex2_approx(m - to_m);
                m = to_m;
                if (w == 0) nref[lane] = kLift - (m == neg_inf() ? 0.f : m);
                fresh = __any_sync(0xffffffffu, lane < mine && m == neg_inf());
                if (!first) {
#pragma unroll 1
                    for (int ch = 0; ch < nch; ++ch) {
                        float o[8], l[8];
                        tmem_ld8(to + ch * 8, o);
                        tmem_ld8(tl + ch * 8, l);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 8; ++e) {
                            const float fe = __shfl_sync(0xffffffffu, f, ch * 8 + e);
                            l[e] *= fe;
                            o[e] *= fe;
                        }
                        tmem_st8(to + ch * 8, o);
                        tmem_st8(tl + ch * 8, l);
                    }
                    tmem_wait_st();
                }
                group_any(grp, false);
            }
            dead |= !wait4(&sm.pv_done[b], ph ^ 1, sm);  // the P of the tile before last has been read
            uint8_t *dst = sm.p[b] + key * 32;
            const bool write = dump && t * kTile + key < n;
#pragma unroll 1
            for (int ch = 0; ch < nch; ++ch) {
                float s[8], f[8], r[8], l[8];
                load8(fac2 + ch * 8, f);
                load8(nref + ch * 8, r);
                tmem_ld8(tl + ch * 8, l);
                scores8(ts, kk, ch, s);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    r[e] = ex2_approx(fmaf(s[e], f[e], r[e]));
                    l[e] = r[e] + (first ? 0.f : l[e]);
                }
                tmem_st8(tl + ch * 8, l);
                const int cc = c0 / 8 + ch;
                *reinterpret_cast<uint4 *>(dst + (cc >> 1) * (kTile * 32) + (((cc & 1) ^ ((key >> 2) & 1)) << 4)) =
                    make_uint4(pack_f16x2(r[0], r[1]), pack_f16x2(r[2], r[3]), pack_f16x2(r[4], r[5]), pack_f16x2(r[6], r[7]));
                if (write) {
                    load8(sm.fac[is] + c0 + ch * 8, f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float *row = sm.lb[is][c0 + ch * 8 + e];
                        if (row) row[kk.pos] = s[e] * f[e];
                    }
                }
            }
            first = false;
            tmem_wait_st();
            fence_proxy_async_smem();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive_cnt(&sm.p_full[b], turns ? 2 : 1);
                mbar_arrive_cnt(&sm.s_empty[b], turns ? 2 : 1);
            }
            __syncwarp();
        }
        // the sums of weights over the warp's keys: of eight rows at a time, each lane ends up with one
#pragma unroll 1
        for (int ch = 0; ch < nch; ++ch) {
            float l[8], z;
            tmem_ld8(tl + ch * 8, l);
            tmem_wait_ld();
#pragma unroll
            for (int h = 16, k = 4; k; h >>= 1, k >>= 1)
#pragma unroll
                for (int e = 0; e < k; ++e) {
                    const bool up = lane & h;
                    const float keep = up ? l[k + e] : l[e], give = up ? l[e] : l[k + e];
                    l[e] = keep + __shfl_xor_sync(0xffffffffu, give, h);
                }
            z = first ? 0.f : l[0];
            z += __shfl_xor_sync(0xffffffffu, z, 2);
            z += __shfl_xor_sync(0xffffffffu, z, 1);
            if ((lane & 3) == 0) sm.sum[sl][grp][w][ch * 8 + (lane >> 4 & 1) * 4 + (lane >> 3 & 1) * 2 + (lane >> 2 & 1)] = z;
        }
        arrive_lane0(&sm.epi_full[sl]);
        arrive_lane0(&sm.item_empty[is]);
    }
}

// ------------------------------------------------------------------ query warps

// The f16 query operands of an item (two warps, four rows at a time each) and what the softmax warps know about its rows.
template <int D>
__device__ void queries4(const Kv4Params &p, Smem4<D> &sm, int w, int lane) {
    constexpr int W = D / 64;  // words of a lane
#pragma unroll 1
    for (int i = 0;; ++i) {
        const int is = i % kItems;
        if (!wait4(&sm.item_full[is], i / kItems & 1, sm)) return;
        const ItemRec rec = sm.item[is];
        if (rec.stop) return;
        if (!wait4(&sm.q_empty[i & 1], (i >> 1 & 1) ^ 1, sm)) return;
#pragma unroll 1
        for (int r0 = 4 * w; r0 < (rec.rows + 7) / 8 * 8; r0 += 8) {
            // (lane l looks after row r0 + l % 4)
            const int my = r0 + (lane & 3), j = rec.verify ? my / p.G : 0, gi = my - j * p.G;
            const int at = my < rec.rows ? (rec.q_off + j) * p.Hq + rec.g * p.G + gi : -1;
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
                mx = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16)) >> 7;
                mx = max(mx, 15u);                                     // biased exponent, such that 2^(141 - mx) is finite
                if ((lane & 3) == e) mine = mx;
                const float up = __uint_as_float((268u - mx) << 23);   // 2^(141 - mx): the largest comes to [2^14, 2^15)
                uint8_t *to = dst + e * 128 + (((lane * W % 32 / 4) ^ ((r0 + e) & 7)) << 4);
                if (W == 2)
                    *reinterpret_cast<uint2 *>(to) = make_uint2(pack_f16x2(bf16lo(x[e][0]) * up, bf16hi(x[e][0]) * up),
                                                                pack_f16x2(bf16lo(x[e][W - 1]) * up, bf16hi(x[e][W - 1]) * up));
                else
                    *reinterpret_cast<uint32_t *>(to) = pack_f16x2(bf16lo(x[e][0]) * up, bf16hi(x[e][0]) * up);
            }
            if (lane < 4) {
                const float down = __uint_as_float((mine - 14u) << 23);
                const float fac = fmaxf(down * p.scale, __int_as_float(1));  // (above 0: a masked score stays -inf)
                sm.fac[is][my] = fac;
                sm.fac2[is][my] = fmaxf(fac * kLog2e, __int_as_float(1));
                sm.lim[is][my] = rec.verify && my < rec.rows ? rec.L - (p.k + 1) + j : 0x7fffffff;
                sm.lb[is][my] = my < rec.rows && rec.verify && p.logits
                                    ? p.logits + (rec.logit_off + ((long long)(rec.g * p.G + gi) * (p.k + 1) + j) * rec.L) : nullptr;
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
        const bool turns = takes_turns(rec.rows), whole = rec.nsplit == 1;
        const int split = 8 * first_chunks(rec.rows);
#pragma unroll 1
        for (int h = 0; h < rec.rows; h += 32) {
            // row h + lane: where it goes (-1: there is none), and what the (two) accumulators are multiplied by
            const int r = h + lane, j = rec.verify ? r / p.G : 0, gi = r - j * p.G;
            int at = -1;
            float f0 = 0.f, f1 = 0.f;
            if (r < rec.rows) {
                at = whole ? (rec.q_off + j) * p.Hq + rec.g * p.G + gi : rec.rec + r;
                const int grp = !turns && r >= split, c = r - (grp ? split : 0);
                const float *s0 = &sm.sum[sl][grp][0][c];
                float l = s0[0] + s0[32] + s0[64] + s0[96], ref = -sm.nref[sl][grp][c];
                f0 = 1.f;
                if (turns) {
                    const float *s1 = &sm.sum[sl][1][0][c];
                    const float l1 = s1[0] + s1[32] + s1[64] + s1[96], ref1 = -sm.nref[sl][1][c];
                    // (a sum of 0 has no reference)
                    const float top = l == 0.f ? ref1 : l1 == 0.f ? ref : fmaxf(ref, ref1);
                    f0 = l == 0.f ? 0.f : ex2_approx(ref - top);
                    f1 = l1 == 0.f ? 0.f : ex2_approx(ref1 - top);
                    l = __fadd_rn(__fmul_rn(l, f0), __fmul_rn(l1, f1));  // (the same whichever group began)
                    ref = top;
                }
                const float inv = l == 0.f ? 0.f : __frcp_rn(l);
                // (what is 0 stays it under a NaN sum: an accumulator that nobody wrote is not read)
                if (f0 != 0.f) f0 *= inv;
                if (f1 != 0.f) f1 *= inv;
                if (w == 0) {
                    const float z = l > 0.f ? ref * 0.69314718f + logf(l) : (l == 0.f ? neg_inf() : l);  // (a NaN sum stays one)
                    if (!whole) p.part_lse[at] = z;
                    else if (rec.verify) p.lse[((size_t)rec.vidx * p.Hq + (size_t)rec.g * p.G + gi) * (p.k + 1) + j] = z;
                }
            }
            // (in turns, an item of one tile has one accumulator: a group that met no tile has sums of 0)
            const bool any0 = !turns || __any_sync(0xffffffffu, f0 != 0.f), any1 = __any_sync(0xffffffffu, f1 != 0.f);
#pragma unroll 1
            for (int r0 = 0; r0 < min(32, rec.rows - h); r0 += 8) {
                float o[8], o1[8];
                const uint32_t from = tm + ((uint32_t)w << 21) + kTmemO + sl * 64 + h + r0;
                tmem_ld8(from, o);
                tmem_ld8(from + (turns ? 16 : 0), o1);
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
            mbar_init(&sm.item_empty[i], 8 + 4 + 2 + 1);  // softmax, epilogue and query warps, the products' warp
            mbar_init(&sm.fac_full[i], 2);
        }
        for (int i = 0; i < kChunks; ++i) {
            mbar_init(&sm.rows_full[i], 1);
            mbar_init(&sm.rows_empty[i], 16);  // K, V and softmax warps
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.q_full[i], 2);
            mbar_init(&sm.q_empty[i], 1);
            mbar_init(&sm.k_full[i], 4);
            mbar_init(&sm.s_full[i], 1);
            mbar_init(&sm.s_empty[i], 8);
            mbar_init(&sm.p_full[i], 8);
            mbar_init(&sm.v_full[i], 4);
            mbar_init(&sm.pv_done[i], 1);
            mbar_init(&sm.o_full[i], 1);
            mbar_init(&sm.o_empty[i], 4);
            mbar_init(&sm.epi_full[i], 8);
            mbar_init(&sm.epi_empty[i], 4);
        }
        mbar_init(&sm.drain, 1);
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
    // the registers go to the softmax warps: 80 a thread at launch
    switch (warp >> 2) {
        case 0:
        case 1:
            asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
            softmax4<D>(p, sm, tm, warp >> 2, w, lane);
            break;
        case 2:
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
            convert4<D, false>(p, sm, tm, w, lane);
            break;
        case 3:
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
            convert4<D, true>(p, sm, tm, w, lane);
            break;
        case 4:
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
            if (w == 0) resolver4<D>(p, sm, lane);
            else if (w == 1) mma4<D>(p, sm, tm);
            else queries4<D>(p, sm, w - 2, lane);
            break;
        default:
            asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
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

cudaError_t launch_attn_kv4(const AttnArgs &a, const Kv4Cache &c, int nsm, cudaStream_t st) {
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
    p.Hq = a.Hq;
    p.Hkv = a.Hkv;
    p.G = a.Hq / a.Hkv;
    p.k = a.k;
    p.M = (a.k + 1) * p.G;
    p.max_sparse = a.max_sparse;
    p.scale = a.scale;
    p.wait_ns = a.wait_ns;
    // Verify items of more than eight rows and then the others, whose CTAs take the place of the first ones as these end.
    const bool many = p.M > kFewRows && a.schedule != PILLAR_SCHEDULE_DRAFT_ONLY;
    cudaError_t e = cudaSuccess;
    if (many) e = a.D == 128 ? launch_t<128>(p, nsm, st) : launch_t<64>(p, nsm, st);
    if (e == cudaSuccess && (!many || a.schedule != PILLAR_SCHEDULE_VERIFY_ONLY))
        e = launch_attn_kv4_few(p, a.D, many, nsm, st);
    return e == cudaSuccess ? launch_merge(a, nsm, st) : e;
}

}  // namespace pillar
