// pillar_prompt.cu -- causal attention over whole prompts, packed one after
// another, with grouped heads.
//
//   out[i, h] = sum_{j <= i} softmax_j(scale q_ih . k_j,h/G) v_j,h/G   (j in i's sequence)
//   lse[i, h] = log sum_{j <= i} e^(scale q_ih . k_j,h/G)
//
// A planner lists the sequences' row tiles, those with the most keys first.  The
// attention kernel is persistent, one CTA per SM; CTA c takes units c, 2 G - 1 - c,
// 2 G + c, ... of the G CTAs' rounds: over many rounds their slopes cancel, over two
// or three they do not (see below).  A unit is
// two tiles of 128 query rows against the 128-key tiles up to the diagonal: the same
// rows for two heads that share a KV head, or, when a group has an odd number of
// heads, 256 consecutive rows of one:
//   * a load thread brings Q, K and V tiles by TMA (128-byte swizzle; K and V through
//     one ring, in the order in which they are used);
//   * an MMA warp issues S_b = Q_b K^T (128 x 128, tcgen05, both operands in shared
//     memory, fp32 in tensor memory) and O_b += P_b V (P from tensor memory, over
//     its scores) for the two row tiles b in turn: while the softmax of one is at
//     work, the tensor cores have the other's products;
//   * two warpgroups, one per row tile, a row per thread: the whole row of scores
//     in registers, its maximum, exponentials and sum without a shuffle, and
//     bf16 probabilities back to tensor memory (the products take both operands in one
//     type, and V's range needs bf16; the sum is of the unrounded ones.  It costs what
//     the bf16 step pays too: 0.0018 to 0.0020 of the output's norm, where rounding the
//     output alone costs 0.0015).  O is rescaled only when a row's
//     maximum grew by more than 2^8.  At a unit's end they normalise O and write it
//     through a 4 KB buffer a warp, so that eight lanes store 128 bytes of a row (each
//     lane storing its own row, 16 bytes at a time, took 3000 to 4400 cycles a unit).
// What bounds it: the tensor cores (4 D flops a visible pair; half of the diagonal
// tile is computed and masked): 16384 tokens, 32 heads on 8, D = 128 take 1473 to 1493 us,
// 1.48 PFLOP/s of visible pairs, 0.79 of a library matrix product's rate; S reads both operands
// from shared memory.  Batches of few rounds are bound by their longest CTA and by each
// unit's ends: 24 sequences of 1 to 2047 tokens, the same heads, 73 us, where the busiest
// CTA has 31 key tiles of two row tiles, the mean is 26, and an SM is active for 0.86 of
// the longest's cycles; 12 of 300 to 4100, D = 64, four heads on one, 55 us, 37 against a
// mean of 28, 0.79 of the cycles, the exponentials' pipe busy for 0.37 of an SM's own and
// the tensor cores for 0.34.  Keys behind a sequence's end lie in the next one:
// their scores are behind the diagonal for every row that counts, and their values
// are zeroed in shared memory, since 0 * NaN would carry over.
#include <cuda.h>  // CUtensorMap

#include "pillar_device.cuh"
#include "pillar_prompt.h"

namespace pillar {

namespace {

constexpr int kPlanThreadsP = 1024;
constexpr int kLevels = 1024;  // bins of the longest-first order

// Lists the tiles, those with the most keys first.
__global__ void __launch_bounds__(kPlanThreadsP) prompt_plan(const int *seq_off, int B, int n, int max_len, int rows, int room,
                                                             PromptHeader *hdr, PromptTile *tiles) {
    __shared__ int s_bin[kLevels];
    __shared__ int s_warp[32];
    __shared__ int s_bad;
    __shared__ long long s_tiles[32];
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    s_bin[tid] = 0;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    // bin of tile i of a sequence: larger i first
    const int most = (min(max_len, n) - 1) / rows + 1;
    int shift = 0;
    while ((most >> shift) >= kLevels) ++shift;
    auto level = [&](int i) { return kLevels - 1 - (i >> shift); };
    auto tiles_of = [&](int b, int *first, int *len) {
        const int lo = seq_off[b], hi = seq_off[b + 1];
        if (lo < 0 || hi < lo || hi > n || hi - lo > max_len) {
            s_bad = PILLAR_FLAG_REQUEST;
            return 0;
        }
        *first = lo;
        *len = hi - lo;
        return (hi - lo) / rows + ((hi - lo) % rows != 0);
    };
    int first = 0, len = 0;
    long long mine = 0;  // tiles of this warp's sequences
    for (int b = wid; b < B && mine <= room; b += 32) {
        const int nt = tiles_of(b, &first, &len);
        mine += nt;
        for (int i = lane; i < nt && mine <= room; i += 32) atomicAdd(&s_bin[level(i)], 1);
    }
    if (lane == 0) s_tiles[wid] = mine;
    __syncthreads();
    const long long part = s_tiles[lane];
    const long long total = ((long long)__reduce_add_sync(0xffffffffu, (unsigned)(part >> 16)) << 16) +
                            __reduce_add_sync(0xffffffffu, (unsigned)part & 0xffffu);
    if (total > room) {  // only sequences that overlap list more than there is room for
        if (tid == 0) {
            hdr->num_tiles = 0;
            hdr->err = PILLAR_FLAG_REQUEST;
        }
        return;
    }
    const int own = s_bin[tid];
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[wid] = x;
    __syncthreads();
    const int before = (int)__reduce_add_sync(0xffffffffu, lane < wid ? (unsigned)s_warp[lane] : 0u);
    s_bin[tid] = before + x - own;
    __syncthreads();
    for (int b = wid; b < B; b += 32) {
        const int nt = tiles_of(b, &first, &len);
        for (int i = lane; i < nt; i += 32) {
            tiles[atomicAdd(&s_bin[level(i)], 1)] = PromptTile{first, len, i, 0};
        }
    }
    __syncthreads();
    if (tid == 0) {
        hdr->num_tiles = (int)total;
        hdr->err = s_bad;
    }
}

constexpr int kSoftmaxWarps = 8;
constexpr int kThreadsP = (kSoftmaxWarps + 4) * 32;  // and the MMA warp, the load warp, two idle ones
constexpr uint32_t kSoftmaxRegs = 208, kOtherRegsP = 80;
static_assert(kSoftmaxWarps * 32 * kSoftmaxRegs + 128 * kOtherRegsP <= kThreadsP * 168, "registers of the launch");
constexpr int kTileP = kPromptRows;  // query rows of a row tile, keys of a key tile
constexpr uint32_t kTmemColsP = 512;
constexpr float kRescaleLog2P = 8.f;

struct PromptParams {
    CUtensorMap q, k, v;  // [n, heads, D] bf16, box 128 tokens x 1 head x 64 columns, 128-byte swizzle
    uint16_t *out;
    float *lse;
    PromptHeader *hdr;
    const PromptTile *tiles;
    int Hq, G;
    int rows;       // of a planned tile
    int per_tile;   // units of a planned tile: Hq / 2 pairs of heads, or Hq heads
    float scale;
    unsigned long long wait_ns;
};

template <int D>
struct SmemP {
    static constexpr int kTileBytes = kTileP * D * 2;
    static constexpr int kSlots = D == 128 ? 4 : 6;  // K and V tiles in shared memory (three: 6 % slower on long prompts)
    alignas(1024) uint8_t q[2][kTileBytes];
    uint8_t kv[kSlots][kTileBytes];
    uint8_t out[kSoftmaxWarps][32 * 128];  // 32 rows of 64 columns, on their way to memory
    uint64_t qfull[2], qempty[2], kvfull[kSlots], kvempty[kSlots];
    uint64_t sfull[2], pfull[2], pvdone[2], ofree[2], cexit, drain;
    uint32_t tmem;
    int abort;
};
static_assert(sizeof(SmemP<128>) <= 227 * 1024, "shared memory of a CTA");
static_assert(sizeof(SmemP<64>) > 114 * 1024, "never two CTAs on an SM: each takes all of its tensor memory");

struct BoundsP {
    volatile int *abort;
    int *err;
    unsigned long long ns;
};
__device__ __forceinline__ bool waitp(uint64_t *bar, uint32_t parity, const BoundsP &b) {
    return mbar_wait(bar, parity, b.abort, b.err, b.ns);
}
__device__ __forceinline__ bool waitw(uint64_t *bar, uint32_t parity, const BoundsP &b) {  // by a whole warp
    return mbar_wait_warp(bar, parity, b.abort, b.err, b.ns);
}
// Bounded wait for copies or products already in flight, whatever the pipeline's bound and the abort flag say.
__device__ __forceinline__ void drainp(uint64_t *bar, uint32_t parity) {
    const unsigned long long t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity))
        if (global_timer_ns() - t0 > kWaitTimeoutNs) return;
}

// Columns [x, x + 64) of head y of tokens z .. z + 127.
__device__ __forceinline__ void tma_load3(void *dst, const void *map, int x, int y, int z, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
            smem_u32(dst)),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}

// A unit of a CTA: row tiles 0 and 1.
struct Unit {
    int row0, len;  // the sequence's first row and length
    int q0, h;      // first row (in the sequence) and head of row tile 0
    int dq, dh;     // what row tile 1 adds to them
    int na, nb;     // key tiles of the row tiles (nb 0: there is no second one)
    __device__ __forceinline__ int nk() const { return max(na, nb); }
    __device__ __forceinline__ int of(int b) const { return b ? nb : na; }
};
// The units of a CTA in order; the record of the one after the next loads while the next is worked on.
struct Units {
    const PromptParams &p;
    int total, round, t, x;  // units in all; the round, tile and place in the tile of `ahead`
    PromptTile ahead;
    __device__ __forceinline__ Units(const PromptParams &q, int n) : p(q), total(n), round(-1), t(-1) { fetch(); }
    __device__ __forceinline__ void fetch() {
        ++round;
        const int c = blockIdx.x, G = gridDim.x;
        const long long r = (long long)round * G + ((round & 1) ? G - 1 - c : c);
        t = r < total ? (int)(r / p.per_tile) : -1;  // (only the last round can be incomplete)
        x = (int)(r - (long long)t * p.per_tile);
        if (t >= 0) ahead = p.tiles[t];
    }
    __device__ __forceinline__ bool next(Unit *u) {
        if (t < 0) return false;
        u->row0 = ahead.row0;
        u->len = ahead.len;
        u->q0 = ahead.tile * p.rows;
        u->na = u->q0 / kTileP + 1;
        if (p.rows == kTileP) {
            u->h = 2 * x;
            u->dq = 0, u->dh = 1;
            u->nb = u->na;
        } else {
            u->h = x;
            u->dq = kTileP, u->dh = 0;
            u->nb = u->q0 + kTileP < ahead.len ? u->na + 1 : 0;
        }
        fetch();
        return true;
    }
};

// ------------------------------------------------------------------ load thread

template <int D>
__device__ void load_role(const PromptParams &p, SmemP<D> &sm, const BoundsP &bd, int total) {
    using S = SmemP<D>;
    int slot = 0;
    uint32_t phase = 0, qph[2] = {0, 0}, issued = 0, parity = 0, qissued = 0, qparity = 0;
    bool ok = true;
    auto tile = [&](uint8_t *dst, const CUtensorMap *m, int head, int row, uint64_t *bar) {
        mbar_arrive_expect_tx(bar, S::kTileBytes);
#pragma unroll
        for (int x = 0; x < D; x += 64) tma_load3(dst + x * (kTileP * 2), m, x, head, row, bar);
    };
    auto kv = [&](const CUtensorMap *m, int head, int row) {
        ok = waitp(&sm.kvempty[slot], phase ^ 1, bd);
        if (!ok) return;
        tile(sm.kv[slot], m, head, row, &sm.kvfull[slot]);
        issued |= 1u << slot;
        parity = (parity & ~(1u << slot)) | (phase << slot);
        if (++slot == S::kSlots) slot = 0, phase ^= 1;
    };
    auto query = [&](const Unit &u, int b) {
        ok = waitp(&sm.qempty[b], qph[b] ^ 1, bd);
        if (!ok) return;
        tile(sm.q[b], &p.q, u.h + b * u.dh, u.row0 + u.q0 + b * u.dq, &sm.qfull[b]);
        qissued |= 1u << b;
        qparity = (qparity & ~(1u << b)) | (qph[b] << b);
        qph[b] ^= 1;
    };
    Units units(p, total);
    for (Unit u; ok && units.next(&u);) {
        query(u, 0);
        for (int j = 0; j < u.nk() && ok; ++j) {
            kv(&p.k, u.h / p.G, u.row0 + j * kTileP);
            if (ok && j == 0 && u.nb) query(u, 1);
            if (ok) kv(&p.v, u.h / p.G, u.row0 + j * kTileP);
        }
    }
    // Every copy lands before the CTA can exit, whoever gave up: another role can do so when this one has issued its last
    // copies and waits for nothing more.  (Nothing else arrives on these barriers: a slot's last phase stays testable.)
    for (int s = 0; s < S::kSlots; ++s)
        if ((issued >> s) & 1) drainp(&sm.kvfull[s], (parity >> s) & 1);
    for (int b = 0; b < 2; ++b)
        if ((qissued >> b) & 1) drainp(&sm.qfull[b], (qparity >> b) & 1);
}

// ------------------------------------------------------------------ MMA warp

// True for one lane of a converged warp, the same each time.  (Where a branch on the lane's number chose the issuing
// thread, the compiler moved every operand of every product to the uniform registers lane by lane: 4900 cycles a step of
// four 128 x 128 products instead of 3700.)
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(one));
    return one != 0;
}

template <int D>
__device__ void mma_role(const PromptParams &p, SmemP<D> &sm, const BoundsP &bd, int total, uint32_t tm, int lane) {
    using S = SmemP<D>;
    constexpr uint32_t idS = umma_idesc_bf16(kTileP, kTileP, 0, 0), idO = umma_idesc_bf16(kTileP, D, 0, 1);
    uint32_t qph[2] = {0, 0}, pph[2] = {0, 0}, oph[2] = {0, 0};
    int slot0 = 0;        // slot of the next unit's first K tile
    uint32_t phase0 = 0;  // and its phase
    bool issued = false;
    auto slot_of = [&](int i, uint32_t *ph) {  // i-th K or V tile of the unit (K_j: 2 j, V_j: 2 j + 1)
        const int x = slot0 + i;
        *ph = (phase0 + x / S::kSlots) & 1;
        return x % S::kSlots;
    };
    auto scores = [&](int b, int slot) {
        const uint64_t dq = umma_sdesc_sw128(smem_u32(sm.q[b]), 16, 1024), dk = umma_sdesc_sw128(smem_u32(sm.kv[slot]), 16, 1024);
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t step = (uint64_t)((ks >> 2) * (kTileP * 128 / 16) + (ks & 3) * 2);
            umma_bf16(tm + b * kTileP, dq + step, dk + step, idS, ks > 0 ? 1u : 0u);
        }
    };
    auto output = [&](int b, int slot, bool first) {
        const uint64_t dv = umma_sdesc_sw128(smem_u32(sm.kv[slot]), kTileP * 128, 1024);
#pragma unroll
        for (int ks = 0; ks < kTileP / 16; ++ks)  // 16 keys: two 8-key atoms of 1024 bytes
            umma_bf16_ts(tm + 2 * kTileP + b * D, tm + b * kTileP + ks * 8, dv + (uint64_t)(ks * 128), idO,
                         first && ks == 0 ? 0u : 1u);
    };
    Units units(p, total);
    for (Unit u; units.next(&u);) {
        const int nk = u.nk();
        uint32_t ph;
        int s = slot_of(0, &ph);
        bool ok = waitw(&sm.kvfull[s], ph, bd);
        for (int b = 0; b < 2 && ok; ++b) {
            if (!u.of(b)) continue;
            ok = waitw(&sm.qfull[b], qph[b], bd);
            if (!ok) break;
            qph[b] ^= 1;
            tc_fence_after();
            if (elect_one()) {
                scores(b, s);
                umma_commit(&sm.sfull[b]);
                if (u.of(b) == 1) umma_commit(&sm.qempty[b]);
            }
            issued = true;
        }
        if (ok && elect_one()) umma_commit(&sm.kvempty[s]);
        for (int j = 0; j < nk && ok; ++j) {
            const int vs = slot_of(2 * j + 1, &ph);
            ok = waitw(&sm.kvfull[vs], ph, bd);
            if (!ok) break;
            const int tail = u.len - j * kTileP;  // keys of the sequence in this tile
            if (tail < kTileP) {
#pragma unroll
                for (int x = 0; x < D; x += 64)
                    for (int i = tail * 128 + lane * 16; i < kTileP * 128; i += 32 * 16)
                        *reinterpret_cast<uint4 *>(sm.kv[vs] + x * (kTileP * 2) + i) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_smem();
                __syncwarp();
            }
            const int ks = slot_of(2 * j + 2, &ph);
            bool have_k = false;
            for (int b = 0; b < 2 && ok; ++b) {
                if (j >= u.of(b)) continue;
                if (j == 0) {  // O of this row tile has been read out
                    ok = waitw(&sm.ofree[b], oph[b] ^ 1, bd);
                    if (!ok) break;
                    oph[b] ^= 1;
                }
                ok = waitw(&sm.pfull[b], pph[b], bd);
                if (!ok) break;
                pph[b] ^= 1;
                tc_fence_after();
                if (elect_one()) {
                    output(b, vs, j == 0);
                    umma_commit(&sm.pvdone[b]);
                }
                if (j + 1 < u.of(b)) {
                    if (!have_k) {
                        ok = waitw(&sm.kvfull[ks], ph, bd);
                        if (!ok) break;
                        have_k = true;
                        tc_fence_after();
                    }
                    if (elect_one()) {  // over P: the tensor cores take the products in the order of their issue
                        scores(b, ks);
                        umma_commit(&sm.sfull[b]);
                        if (j + 2 == u.of(b)) umma_commit(&sm.qempty[b]);
                    }
                }
            }
            if (!ok) break;
            if (elect_one()) {
                umma_commit(&sm.kvempty[vs]);
                if (have_k) umma_commit(&sm.kvempty[ks]);
            }
        }
        if (!ok) break;
        slot0 += 2 * nk;
        phase0 = (phase0 + slot0 / S::kSlots) & 1;
        slot0 %= S::kSlots;
    }
    if (issued && elect_one()) {  // every product has completed before the tensor memory is freed
        umma_commit(&sm.drain);
        drainp(&sm.drain, 0);
    }
    __syncwarp();
}

// ------------------------------------------------------------------ softmax warpgroups

__device__ __forceinline__ float max3(float a, float b, float c) {
    float d;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// 32 columns of this thread's lane, without the wait.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float *v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]),
          "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]),
          "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
        : "r"(taddr));
}
__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Scales this thread's row of O by f (rare).
template <int D>
__device__ __noinline__ void rescale_row(uint32_t tO, float f) {
#pragma unroll 1
    for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(tO + c, o);
#pragma unroll
        for (int i = 0; i < 32; ++i) o[i] *= f;
        tmem_st32(tO + c, o);
    }
}

template <int D>
__device__ void softmax_role(const PromptParams &p, SmemP<D> &sm, const BoundsP &bd, int total, uint32_t tm, int warp, int lane) {
    const int b = warp >> 2, row = (warp & 3) * 32 + lane;  // row tile, row in it
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tm + b * kTileP + lanes, tO = tm + 2 * kTileP + b * D + lanes;
    const float c2 = p.scale * kLog2e;
    uint32_t n = 0;  // key tiles this warpgroup has done
    Units units(p, total);
    for (Unit u; units.next(&u);) {
        const int nk = u.of(b);
        if (!nk) continue;
        float m = neg_inf(), l = 0.f;  // reference maximum (base 2, scaled) and sum
#pragma unroll 1
        for (int j = 0; j < nk; ++j, ++n) {
            if (!waitw(&sm.sfull[b], n & 1, bd)) return;
            tc_fence_after();
            float s[kTileP];
#pragma unroll
            for (int i = 0; i < kTileP; i += 32) tmem_ld32_async(tS + i, s + i);
            tmem_ld_wait();
            if (j == nk - 1) {  // the diagonal tile
#pragma unroll
                for (int i = 0; i < kTileP; ++i)
                    if (i > row) s[i] = neg_inf();
            }
            float m4[4] = {s[0], s[1], s[2], s[3]};
#pragma unroll
            for (int i = 4; i < kTileP - 4; i += 8)
#pragma unroll
                for (int e = 0; e < 4; ++e) m4[e] = max3(m4[e], s[i + e], s[i + 4 + e]);
#pragma unroll
            for (int e = 0; e < 4; ++e) m4[e] = fmaxf(m4[e], s[kTileP - 4 + e]);
            const float mt = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * c2;
            bool grow = false;
            float f = 1.f;
            if (m == neg_inf()) {
                m = mt;
            } else if (mt - m > kRescaleLog2P) {
                f = ex2_approx(m - mt);
                l *= f;
                m = mt;
                grow = true;
            }
            if (__any_sync(0xffffffffu, grow)) {  // (a row grows only behind an earlier tile's P V)
                if (!waitw(&sm.pvdone[b], (n - 1) & 1, bd)) return;
                tc_fence_after();
                rescale_row<D>(tO, f);
            }
            const float nb = m == neg_inf() ? 0.f : -m;
            const float2 k2 = make_float2(c2, c2), b2 = make_float2(nb, nb);
            float2 l4[4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t pw[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float2 x = ffma2(make_float2(s[64 * h + 2 * i], s[64 * h + 2 * i + 1]), k2, b2);
                    const float2 e = make_float2(ex2_approx(x.x), ex2_approx(x.y));
                    l4[i & 3] = h == 0 && i < 4 ? e : fadd2(l4[i & 3], e);
                    pw[i] = pack_bf16x2(e.x, e.y);
                }
                tmem_st32u(tS + 32 * h, pw);
            }
            const float2 ls = fadd2(fadd2(l4[0], l4[1]), fadd2(l4[2], l4[3]));
            l += ls.x + ls.y;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.pfull[b]);
        }
        // the unit's rows
        if (!waitw(&sm.pvdone[b], (n - 1) & 1, bd)) return;
        tc_fence_after();
        const int i0 = u.q0 + b * u.dq + (warp & 3) * 32, left = u.len - i0;  // this warp's first row; rows from there on
        const int h = u.h + b * u.dh;
        const long long at = ((long long)u.row0 + i0) * p.Hq + h;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        uint8_t *buf = sm.out[warp];
#pragma unroll 1
        for (int x = 0; x < D; x += 64) {
            float o[64];
            tmem_ld32_async(tO + x, o);
            tmem_ld32_async(tO + x + 32, o + 32);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 8; ++e)  // 16-byte pieces, XOR-ed with the row: no bank twice, either way
                *reinterpret_cast<uint4 *>(buf + lane * 128 + ((e ^ (lane & 7)) * 16)) =
                    make_uint4(pack_bf16x2(o[8 * e] * inv, o[8 * e + 1] * inv), pack_bf16x2(o[8 * e + 2] * inv, o[8 * e + 3] * inv),
                               pack_bf16x2(o[8 * e + 4] * inv, o[8 * e + 5] * inv),
                               pack_bf16x2(o[8 * e + 6] * inv, o[8 * e + 7] * inv));
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                const int rr = 4 * q + (lane >> 3), ch = lane & 7;
                const uint4 v = *reinterpret_cast<const uint4 *>(buf + rr * 128 + ((ch ^ (rr & 7)) * 16));
                if (rr < left) *reinterpret_cast<uint4 *>(p.out + (at + (long long)rr * p.Hq) * D + x + ch * 8) = v;
            }
            __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.ofree[b]);
        if (lane < left && p.lse)
            p.lse[at + (long long)lane * p.Hq] = l > 0.f ? m * 0.6931471805599453f + logf(l) : (l == 0.f ? neg_inf() : l);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreadsP, 1) prompt_kernel(const __grid_constant__ PromptParams p) {
    extern __shared__ __align__(1024) uint8_t smem_p[];
    SmemP<D> &sm = *reinterpret_cast<SmemP<D> *>(smem_p);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.qfull[i], 1);
            mbar_init(&sm.qempty[i], 1);
            mbar_init(&sm.sfull[i], 1);
            mbar_init(&sm.pfull[i], 4);
            mbar_init(&sm.pvdone[i], 1);
            mbar_init(&sm.ofree[i], 4);
        }
        for (int i = 0; i < SmemP<D>::kSlots; ++i) {
            mbar_init(&sm.kvfull[i], 1);
            mbar_init(&sm.kvempty[i], 1);
        }
        mbar_init(&sm.cexit, kSoftmaxWarps + 1);
        mbar_init(&sm.drain, 1);
        sm.abort = 0;
        mbar_init_fence();
    }
    if (warp == 0) tmem_alloc(&sm.tmem, kTmemColsP);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = sm.tmem;
    pdl_wait_prerequisites();  // the tiles are the planner's
    pdl_launch_dependents();
    const int total = *reinterpret_cast<volatile int *>(&p.hdr->num_tiles) * p.per_tile;
    const BoundsP bd{&sm.abort, &p.hdr->err, p.wait_ns};
    if (warp < kSoftmaxWarps) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        softmax_role<D>(p, sm, bd, total, tm, warp, lane);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.cexit);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegsP));
        if (warp == kSoftmaxWarps) {
            mma_role<D>(p, sm, bd, total, tm, lane);
            tc_fence_before();
            if (lane == 0) mbar_arrive(&sm.cexit);
        } else if (warp == kSoftmaxWarps + 1 && lane == 0) {
            load_role<D>(p, sm, bd, total);
        }
        __syncwarp();
    }
    if (warp == 0) {  // everyone is done with the tensor memory
        drainp(&sm.cexit, 0);
        tc_fence_after();
        tmem_dealloc(tm, kTmemColsP);
    }
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// Token rows of `heads` x D bf16, `stride` elements apart.  Tokens behind the last read as zeros.
cudaError_t token_map(CUtensorMap *m, const uint16_t *base, int n, int heads, int D, long long stride) {
    static const EncodeTiledFn fn = reinterpret_cast<EncodeTiledFn>(driver_entry("cuTensorMapEncodeTiled", 12000));
    if (!fn) return cudaErrorNotSupported;
    const cuuint64_t dim[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)n};
    const cuuint64_t step[2] = {(cuuint64_t)D * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, kTileP}, one[3] = {1, 1, 1};
    const CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint16_t *>(base), dim, step, box, one,
                          CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D>
cudaError_t launch_t(const PromptParams &p, int grid, cudaLaunchConfig_t &cfg) {
    static unsigned long long configured[kMaxDevices] = {};  // launch attributes, once per device context
    int dev = 0;
    unsigned long long ctx = 0;
    cudaError_t e = current_device_context(&dev, &ctx);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (ctx == 0 || __atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE) != ctx) {
        e = cudaFuncSetAttribute(prompt_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SmemP<D>));
        if (e != cudaSuccess) return e;
        e = current_device_context(&dev, &ctx);  // (the call above made a context current)
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], ctx, __ATOMIC_RELEASE);
    }
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreadsP);
    cfg.dynamicSmemBytes = sizeof(SmemP<D>);
    return cudaLaunchKernelEx(&cfg, prompt_kernel<D>, p);
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs &a, int nsm, cudaStream_t st) {
    PromptParams p;
    cudaError_t e = token_map(&p.q, a.q, a.n, a.Hq, a.D, a.q_stride);
    if (e == cudaSuccess) e = token_map(&p.k, a.k, a.n, a.Hkv, a.D, a.k_stride);
    if (e == cudaSuccess) e = token_map(&p.v, a.v, a.n, a.Hkv, a.D, a.v_stride);
    if (e != cudaSuccess) return e;
    p.hdr = reinterpret_cast<PromptHeader *>(a.ws);
    PromptTile *tiles = reinterpret_cast<PromptTile *>(a.ws + sizeof(PromptHeader));
    p.tiles = tiles;
    p.out = a.out;
    p.lse = a.lse;
    p.Hq = a.Hq;
    p.G = a.Hq / a.Hkv;
    p.rows = prompt_tile_rows(p.G);
    p.per_tile = p.rows == kTileP ? a.Hq / 2 : a.Hq;
    p.scale = a.scale;
    p.wait_ns = a.wait_ns;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreadsP);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const int room = (int)prompt_max_tiles(a.B, a.n);
    e = cudaLaunchKernelEx(&cfg, prompt_plan, a.seq_off, a.B, a.n, a.max_len, p.rows, room, p.hdr, tiles);
    if (e != cudaSuccess) return e;
    const long long units = (long long)room * p.per_tile;
    const int grid = (int)(units < nsm ? units : nsm);
    return a.D == 128 ? launch_t<128>(p, grid, cfg) : launch_t<64>(p, grid, cfg);
}

}  // namespace pillar
