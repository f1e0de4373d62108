// pillar_attn_kv4_few.cu -- the 4-bit attention's items of at most eight query rows: drafts and plain decoding.
//
// Every warp works alone on 16 keys at a time: S^T = K Q^T and O^T = V^T P^T
// with m16n8k16, the keys (the dimensions) on m and the rows on n, both
// operands f16 (every cache value is one).  Nothing waits for another warp
// before an item's end, where the eight warps of the CTA, which share its keys,
// join through shared memory.
//   * The codes come by 16-byte asynchronous copies into three slots of the warp's
//     own.  K: lane c of four has dimensions [32c, 32c + 32) of its key, 16 bytes
//     that hold the operands of all steps.  V: a lane has 16 (D = 128) dimensions of
//     four keys, and two keys' codes are paired into bytes that convert at once.
//   * Among 16 keys m = g and g + 8 are keys 2g and 2g + 1, so that a lane holds
//     neighbours: their logits are one store.  P is transposed between the products
//     by movmatrix.
//   * Each warp has reference maxima of its own; one moves when a score passes it
//     by more than 2^8, which a vote of the warp finds out.
#include "pillar_attn_kv4.cuh"

namespace pillar {

namespace {

constexpr int kThreadsF = 256, kWarpsF = kThreadsF / 32;
constexpr int kCtasF = 2;                        // CTAs of an SM
constexpr int kSlotsF = 3;                       // 16-key pieces of a warp: one being read, two on their way
constexpr int kPieces = kMaxChunk / (16 * kWarpsF);  // of a warp in an item, at most
static_assert(kPieces <= 16, "a lane keeps what it knows of a piece, lists fill 16");

template <int D>
struct PieceF {
    static constexpr int kRow = D / 2, kScales = D / kGroup4;
    alignas(128) uint8_t k[16 * kRow];
    uint8_t v[16 * kRow], ks[16 * kScales], vs[16 * kScales];
};

// A work item (in shared memory).
struct WorkF {
    int b, g, begin, n, L, q_off, vidx, nsplit, rec, verify;
    long long logit_off;
};

template <int D>
struct SmemF {
    PieceF<D> piece[kWarpsF][kSlotsF];
    float o[kWarpsF][8][D + 4], m[kWarpsF][8], l[kWarpsF][8];  // the warps' parts of an item's rows
    int row[kWarpsF][kPieces * 16];                            // lists: rows of the pools, or -1
    struct alignas(16) {
        Item item;
        ReqInfo req;
        UnitInfo unit;
    } ahead;     // the next item's records
    float *lb[8];  // where the logits of the item's rows at position 0 go, or null
    WorkF w[2];  // this item and the next, in turn
    int item;
};

struct FewParams {
    Kv4Params p;
    int *counter;
    bool few_only, after;
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_scales(uint32_t dst, const void *src, int bytes) {  // (zeros behind `bytes`)
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(N) : "memory");
}
// Shared-memory loads at an address and a constant.
template <int kOff>
__device__ __forceinline__ uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4+%5];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at), "n"(kOff));
    return v;
}
template <int kOff>
__device__ __forceinline__ uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2+%3];" : "=r"(v.x), "=r"(v.y) : "r"(at), "n"(kOff));
    return v;
}
template <int kOff>
__device__ __forceinline__ uint32_t lds32(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1+%2];" : "=r"(v) : "r"(at), "n"(kOff));
    return v;
}
template <int kOff>
__device__ __forceinline__ uint32_t lds8(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u8 %0, [%1+%2];" : "=r"(v) : "r"(at), "n"(kOff));
    return v;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Byte offset of 16-byte chunk ch of row r in a piece's K and V codes.  K: lanes read the rows 2g together, two at a time (four
// for D = 64); V: the rows 4c, a part each.  Rows change places, or chunks under an XOR, so that they meet no bank twice.
template <int D>
__device__ __forceinline__ int k_at(int r, int ch) {
    if (D == 128) return (r ^ ((r >> 1) & 1)) * 64 + ch * 16;
    return (r ^ ((r >> 2) & 1)) * 32 + ch * 16;
}
template <int D>
__device__ __forceinline__ int v_at(int r, int ch) {
    const int flip = ((r >> 2) & 3) << 1;
    if (D == 128) return (r >> 1) * 128 + ((((r & 1) << 2) | ch) ^ flip) * 16;
    return (r >> 2) * 128 + ((((r & 3) << 1) | ch) ^ flip) * 16;
}

// What a lane keeps through an item; rows 2c and 2c + 1 of the item are those of accumulator columns 0 and 1.
template <int D>
struct StateF {
    uint32_t q[D / 16][2];             // query operands
    float o[D / 16][4];                // O^T: dimensions (D / 8) g + 2i and the next, rows 2c and 2c + 1
    float fac[2], fac2[2], nref[2], l[2];  // logit = sum * fac, fac2 in base 2; kLift - reference; this lane's weights
    int lim[2];                        // last position seen
    bool fresh;                        // a row has no reference yet
};

// Where a lane's parts of a piece lie, from the piece's first byte on.
template <int D>
struct PlaceF {
    uint32_t k, ks, v, vs;
    __device__ __forceinline__ PlaceF(int g, int c) {
        using Pc = PieceF<D>;
        k = D == 128 ? k_at<D>(2 * g, c) : k_at<D>(2 * g, c >> 1) + (c & 1) * 8;  // (row 2g + 1: ^ Pc::kRow)
        v = 16 * Pc::kRow + (D == 128 ? v_at<D>(4 * c, g >> 1) + (g & 1) * 8 : v_at<D>(4 * c, g >> 2) + (g & 3) * 4);
        ks = 32 * Pc::kRow + 2 * g * Pc::kScales + c * Pc::kScales / 4;
        vs = 32 * Pc::kRow + 16 * Pc::kScales + 4 * c * Pc::kScales + g * Pc::kScales / 8;
    }
};

// 16 keys: those of `vis`; all: every row sees them all; pos0: position of the first (verify); left: keys of the item from
// it on; logits: where the logits of rows 2c and 2c + 1 at position 0 go (each null for no such row), or null.
template <int D>
__device__ __forceinline__ void keys16(uint32_t pc, const PlaceF<D> &at, unsigned vis, bool all, int pos0, int left,
                                       float *const *logits, StateF<D> &a) {
    using Pc = PieceF<D>;
    float s[4] = {0.f, 0.f, 0.f, 0.f};  // keys 2g (rows 2c, 2c + 1) and 2g + 1
    {
        constexpr int W = D / 32;  // words of a lane's part of a row
        constexpr uint32_t kBoth = 0x00800080u;  // (a scale byte in bits 7 to 14 is its f16 value)
        uint32_t x[2][W];
        const uint32_t k0 = pc + at.k, k1 = pc + (at.k ^ Pc::kRow), ks = pc + at.ks;
        if (D == 128) {
            const uint4 y0 = lds128<0>(k0), y1 = lds128<0>(k1);
            x[0][0] = y0.x, x[0][1] = y0.y, x[0][W - 2] = y0.z, x[0][W - 1] = y0.w;
            x[1][0] = y1.x, x[1][1] = y1.y, x[1][W - 2] = y1.z, x[1][W - 1] = y1.w;
        } else {
            const uint2 y0 = lds64<0>(k0), y1 = lds64<0>(k1);
            x[0][0] = y0.x, x[0][1] = y0.y, x[1][0] = y1.x, x[1][1] = y1.y;
        }
        uint32_t sc[2][2];
        sc[0][0] = lds8<0>(ks) * kBoth;
        sc[1][0] = lds8<Pc::kScales>(ks) * kBoth;
        if (D == 128) {
            sc[0][1] = lds8<1>(ks) * kBoth;
            sc[1][1] = lds8<Pc::kScales + 1>(ks) * kBoth;
        }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            uint32_t h0[4], h1[4];
            f16_of_e2m1(x[0][i], h0);
            f16_of_e2m1(x[1][i], h1);
#pragma unroll
            for (int e = 0; e < 4; ++e) h0[e] = mul_f16x2(h0[e], sc[0][i >> 1]), h1[e] = mul_f16x2(h1[e], sc[1][i >> 1]);
            mma16816(s, h0[0], h1[0], h0[1], h1[1], a.q[2 * i][0], a.q[2 * i][1]);
            mma16816(s, h0[2], h1[2], h0[3], h1[3], a.q[2 * i + 1][0], a.q[2 * i + 1][1]);
        }
    }
    // V: this lane's D / 8 dimensions of keys 4c .. 4c + 3 (k = 2c, 2c + 8, 2c + 1, 2c + 9)
    constexpr int W = D / 64;  // words per key
    uint32_t x[4][W], s02, s13;
    {
        const uint32_t v0 = pc + at.v, vs = pc + at.vs;
        if (D == 128) {
            const uint32_t v1 = pc + (at.v ^ 64);
            const uint2 y0 = lds64<0>(v0), y1 = lds64<0>(v1), y2 = lds64<128>(v0), y3 = lds64<128>(v1);
            x[0][0] = y0.x, x[0][W - 1] = y0.y, x[1][0] = y1.x, x[1][W - 1] = y1.y;
            x[2][0] = y2.x, x[2][W - 1] = y2.y, x[3][0] = y3.x, x[3][W - 1] = y3.y;
        } else {
#pragma unroll
            for (int u = 0; u < 4; ++u) x[u][0] = lds32<0>(pc + (at.v ^ (32 * u)));
        }
        s02 = lds8<0>(vs) * 0x80u + lds8<2 * Pc::kScales>(vs) * 0x800000u;
        s13 = lds8<Pc::kScales>(vs) * 0x80u + lds8<3 * Pc::kScales>(vs) * 0x800000u;
    }
    if (!all) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const int key = 2 * g + (e >> 1);
            if (!((vis >> key) & 1) || pos0 + key > a.lim[e & 1]) s[e] = neg_inf();
        }
    }
    if (logits) {
        const int lane = threadIdx.x & 31, g = lane >> 2;
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
            float *dst = logits[e];
            if (!dst) continue;
            dst += pos0 + 2 * g;  // eight lanes write 64 bytes of a row
            const float fac = e ? a.fac[1] : a.fac[0], y0 = (e ? s[1] : s[0]) * fac, y1 = (e ? s[3] : s[2]) * fac;
            if (2 * g + 2 <= left && !(reinterpret_cast<uintptr_t>(dst) & 7)) {
                *reinterpret_cast<float2 *>(dst) = make_float2(y0, y1);
            } else {
                if (2 * g < left) dst[0] = y0;
                if (2 * g + 1 < left) dst[1] = y1;
            }
        }
    }
    float w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = fmaf(s[e], a.fac2[e & 1], a.nref[e & 1]);
    if (__any_sync(0xffffffffu, a.fresh || fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3])) > kGrow)) {  // rare: new references
        bool none = false;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float mx = fmaxf(s[e] * a.fac2[e], s[e + 2] * a.fac2[e]);
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            // (a row without one has nref = kLift + inf, which no key of weight has come by)
            const bool had = a.nref[e] < __int_as_float(0x7f800000);
            const float was = kLift - a.nref[e], to = !had || mx > was + (kGrow - kLift) ? fmaxf(mx, was) : was;
            const float f = !had || to == was ? 1.f : ex2_approx(was - to);
            a.nref[e] = kLift - to;
            none |= to == neg_inf();
            a.l[e] *= f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) a.o[i][e] *= f, a.o[i][e + 2] *= f;
#pragma unroll
            for (int k = 0; k < 2; ++k) w[2 * k + e] = fmaf(s[2 * k + e], a.fac2[e], to == neg_inf() ? 0.f : a.nref[e]);
        }
        a.fresh = none;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = ex2_approx(w[e]);
    a.l[0] += w[0] + w[2];
    a.l[1] += w[1] + w[3];
    const uint32_t b0 = transpose8x8(pack_f16x2(w[0], w[1])), b1 = transpose8x8(pack_f16x2(w[2], w[3]));
#pragma unroll
    for (int i = 0; i < W; ++i) {
        constexpr uint32_t kLow = 0x0f0f0f0fu;
        uint32_t he[2][4], ho[2][4];  // [keys 0, 2 | 1, 3]: even dimensions, odd ones
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const uint32_t lo = x[e][i], hi = x[e + 2][i];
            f16_of_e2m1((lo & kLow) | (hi << 4 & ~kLow), he[e]);
            f16_of_e2m1((lo >> 4 & kLow) | (hi & ~kLow), ho[e]);
#pragma unroll
            for (int d = 0; d < 4; ++d) he[e][d] = mul_f16x2(he[e][d], e ? s13 : s02), ho[e][d] = mul_f16x2(ho[e][d], e ? s13 : s02);
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) mma16816(a.o[4 * i + d], he[0][d], ho[0][d], he[1][d], ho[1][d], b0, b1);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreadsF, kCtasF) attn_kv4_few_kernel(const __grid_constant__ FewParams fp) {
    using Pc = PieceF<D>;
    extern __shared__ __align__(128) char smem[];
    SmemF<D> &sm = *reinterpret_cast<SmemF<D> *>(smem);
    const Kv4Params &p = fp.p;
    // (behind the verify items' kernel: its CTAs let this one start once the plan is complete)
    if (!fp.after) pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int first = fp.few_only ? 0 : __ldcg(&p.hdr->num_verify_items), num_items = __ldcg(&p.hdr->num_items);
    int bad = 0;
    // thread 0 takes the next item one step at a time: its index, its record, the records that names
    int step = 0, next = 0;
    auto advance = [&]() {
        if (step == 0) {
            next = first + atomicAdd(fp.counter, 1);
        } else if (next < num_items) {
            if (step == 1) {
                copy16(smem_u32(&sm.ahead.item), p.items + next);
            } else if (step == 4) {  // (copies of this step come with the pieces of two steps on)
                const int unit = sm.ahead.item.unit;
                copy16(smem_u32(&sm.ahead.req), p.req + unit / p.Hkv);
                copy16(smem_u32(&sm.ahead.unit), p.unit + unit);
            }
        }
        ++step;
    };
    static_assert(sizeof(Item) == 16 && sizeof(ReqInfo) == 16 && sizeof(UnitInfo) == 16, "records of 16 bytes");
    static_assert(kSlotsF == 3, "a copy is there two steps later");
    auto open = [&](WorkF &w) {  // the next item's record, by thread 0
#pragma unroll 1
        while (step < 5) {
            if (step == 4) asm volatile("cp.async.wait_all;" ::: "memory");
            advance();
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
        step = 0;
        sm.item = next;
        if (next >= num_items) return;
        const Item itm = sm.ahead.item;
        const ReqInfo rq = sm.ahead.req;
        const UnitInfo un = sm.ahead.unit;
        w.b = itm.unit / p.Hkv;
        w.g = itm.unit - w.b * p.Hkv;
        w.begin = itm.begin;
        w.n = itm.end - itm.begin;
        w.q_off = rq.q_off;
        w.vidx = rq.vidx;
        w.L = rq.len;
        w.verify = rq.mode == 1;
        w.nsplit = un.nsplit;
        w.rec = un.rec_base + itm.split * un.rec_rows;
        w.logit_off = w.verify && p.logits ? __ldcg(p.logit_off + w.b) : 0;
    };
    if (tid == 0) open(sm.w[0]);
    __syncthreads();
    // Of its pieces of the item (warp, warp + 8, ..): a lane keeps the first row of piece `lane` (contexts) and which of its
    // keys there are; lists have their rows in shared memory.
    int base = 0;
    unsigned vis = 0;
    StateF<D> a;
    const PlaceF<D> at(g, c);
    uint4 qx[D / 64][2];  // the next item's queries, on their way
    int qrow = -1;
    auto look_up = [&](const WorkF &w) {  // an item's rows and queries: loads only as far as they depend on none of the others
        const int rows = w.verify ? p.M : p.G, j = w.verify ? g / p.G : 0;
        qrow = g < rows ? (w.q_off + j) * p.Hq + w.g * p.G + g - j * p.G : -1;
        const uint16_t *src = p.q + (size_t)max(qrow, 0) * D + c * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            qx[i][0] = qrow >= 0 ? __ldg(reinterpret_cast<const uint4 *>(src + 16 * i)) : make_uint4(0, 0, 0, 0);
            qx[i][1] = qrow >= 0 ? __ldg(reinterpret_cast<const uint4 *>(src + 16 * i + 8)) : make_uint4(0, 0, 0, 0);
        }
        const int *table = p.c.table + (size_t)w.b * p.c.max_blocks;
        vis = 0;
        if (w.verify) {  // (items begin at multiples of 64: a piece is a block)
            const int k = (warp + lane * kWarpsF) * 16, pos = (w.begin + k) / PILLAR_KV_BLOCK;
            base = -1;
            if (lane < kPieces && k < w.n) {
                const int blk = pos < p.c.max_blocks ? __ldg(table + pos) : -1;
                if (blk >= 0 && blk < p.c.num_blocks) {
                    base = (blk * p.Hkv + w.g) * PILLAR_KV_BLOCK;
                    vis = w.n - k >= 16 ? 0xffffu : (1u << (w.n - k)) - 1;
                } else {
                    bad |= PILLAR_FLAG_SLOT;
                }
            }
        } else {
            const int *list = p.sparse_idx + ((size_t)w.b * p.Hkv + w.g) * p.max_sparse + w.begin;
            // two pieces at a time, four times that in flight
#pragma unroll 1
            for (int m0 = 0; m0 < kPieces / 2 && (warp + 2 * m0 * kWarpsF) * 16 < w.n; m0 += 4) {
                int pos[4], blk[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int k = (warp + (2 * (m0 + m) + (lane >> 4)) * kWarpsF) * 16 + (lane & 15);
                    pos[m] = k < w.n ? __ldg(list + k) : -1;
                    if (k < w.n && (unsigned)pos[m] >= (unsigned)w.L) bad |= PILLAR_FLAG_INDEX, pos[m] = -1;
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    blk[m] = 0;
                    if (pos[m] >= 0) blk[m] = pos[m] / PILLAR_KV_BLOCK < p.c.max_blocks ? __ldg(table + pos[m] / PILLAR_KV_BLOCK) : -1;
                }
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    if ((unsigned)blk[m] >= (unsigned)p.c.num_blocks) bad |= PILLAR_FLAG_SLOT, pos[m] = -1;
                    sm.row[warp][(m0 + m) * 32 + lane] =
                        pos[m] >= 0 ? (blk[m] * p.Hkv + w.g) * PILLAR_KV_BLOCK + pos[m] % PILLAR_KV_BLOCK : -1;
                    const unsigned there = __ballot_sync(0xffffffffu, pos[m] >= 0);
                    if (lane >> 1 == m0 + m) vis = lane & 1 ? there >> 16 : there & 0xffffu;
                }
            }
            __syncwarp();
        }
    };
    if (sm.item < num_items) look_up(sm.w[0]);
    for (int turn = 0; sm.item < num_items; turn ^= 1) {
        const WorkF &w = sm.w[turn];
        const bool verify = w.verify;
        const int n = w.n, rows = verify ? p.M : p.G;
        const int pieces = (n - warp * 16 + kWarpsF * 16 - 1) / (kWarpsF * 16);  // (0 or less: none)
        constexpr uint32_t kBytes = sizeof(Pc);
        const uint32_t slots = smem_u32(sm.piece[warp]);
        auto fetch = [&](int j, uint32_t dst) {
            if (j >= pieces) return;
            constexpr int RC = Pc::kRow / 16, RP = 32 / RC;  // 16-byte pieces of a row, rows of a pass
            const unsigned there = __shfl_sync(0xffffffffu, vis, j);
            const int r = lane / RC, ch = lane % RC, sr = lane & 15;
            const uint32_t to_s = dst + 32 * Pc::kRow + lane * Pc::kScales, bytes = (there >> sr) & 1 ? Pc::kScales : 0;
            const uint8_t *scales = lane < 16 ? p.c.k_scale : p.c.v_scale;
            // (the codes of a key that is not there: any, its scales are 0)
            if (verify) {
                const int row = max(__shfl_sync(0xffffffffu, base, j), 0);
                const size_t src = (size_t)(unsigned)row * Pc::kRow + lane * 16;
#pragma unroll
                for (int i = 0; i < 16 / RP; ++i) {
                    copy16(dst + k_at<D>(i * RP + r, ch), p.c.k4 + src + i * 512);
                    copy16(dst + 16 * Pc::kRow + v_at<D>(i * RP + r, ch), p.c.v4 + src + i * 512);
                }
                copy_scales<Pc::kScales>(to_s, scales + (size_t)(unsigned)(row + sr) * Pc::kScales, bytes);
            } else {
                const int *rows = sm.row[warp] + j * 16;
#pragma unroll
                for (int i = 0; i < 16 / RP; ++i) {
                    const size_t src = (size_t)(unsigned)max(rows[i * RP + r], 0) * Pc::kRow + ch * 16;
                    copy16(dst + k_at<D>(i * RP + r, ch), p.c.k4 + src);
                    copy16(dst + 16 * Pc::kRow + v_at<D>(i * RP + r, ch), p.c.v4 + src);
                }
                copy_scales<Pc::kScales>(to_s, scales + (size_t)(unsigned)max(rows[sr], 0) * Pc::kScales, bytes);
            }
        };
#pragma unroll
        for (int j = 0; j < kSlotsF - 1; ++j) {
            fetch(j, slots + j * kBytes);
            asm volatile("cp.async.commit_group;" ::: "memory");
        }
        // the queries' operands
        {
            uint32_t mx = 0;
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    mx = __vmaxu2(__vmaxu2(__vmaxu2(mx, qx[i][h].x & 0x7fff7fffu), __vmaxu2(qx[i][h].y & 0x7fff7fffu, qx[i][h].z & 0x7fff7fffu)),
                                  qx[i][h].w & 0x7fff7fffu);
            mx = max(mx & 0xffffu, mx >> 16);
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            float up, down;
            query_scale(mx, &up, &down);
#pragma unroll
            for (int i = 0; i < D / 64; ++i)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const uint32_t wd[4] = {qx[i][h].x, qx[i][h].y, qx[i][h].z, qx[i][h].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        a.q[4 * i + 2 * h + (e >> 1)][e & 1] = pack_f16x2(bf16lo(wd[e]) * up, bf16hi(wd[e]) * up);
                }
            float fac = fmaxf(down * p.scale, __int_as_float(1));  // (above 0: a masked score stays -inf)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                a.fac[e] = __shfl_sync(0xffffffffu, fac, 4 * (2 * c + e));
                a.fac2[e] = fmaxf(a.fac[e] * kLog2e, __int_as_float(1));
                a.nref[e] = -neg_inf();
                a.l[e] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.o[i][e] = 0.f;
            a.fresh = true;
        }
        const int sure = verify ? w.L - (p.k + 1) : 0x7fffffff;  // every row sees up to here
        const bool dump = verify && p.logits;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int r = 2 * c + e;
            a.lim[e] = verify && r < rows ? sure + r / p.G : 0x7fffffff;
        }
        if (dump) {
            if (tid < 8) {
                const int j = tid / p.G, gi = tid - j * p.G;
                sm.lb[tid] = tid < rows ? p.logits + w.logit_off + ((long long)(w.g * p.G + gi) * (p.k + 1) + j) * w.L : nullptr;
            }
            __syncthreads();
        }
        uint32_t here = slots, there_to = slots + (kSlotsF - 1) * kBytes;  // the slots of piece j, of the one fetched
#pragma unroll 1
        for (int j = 0; j < pieces; ++j) {
            if (tid == 0 && j + 6 >= pieces && step < 5) advance();  // (not before it is needed: no item waits behind a long one)
            fetch(j + kSlotsF - 1, there_to);
            asm volatile("cp.async.commit_group;\n\tcp.async.wait_group %0;" ::"n"(kSlotsF - 1) : "memory");
            __syncwarp();
            const int k0 = (warp + j * kWarpsF) * 16;
            const unsigned there = __shfl_sync(0xffffffffu, vis, j);
            const int pos0 = verify ? w.begin + k0 : 0;
            keys16<D>(here, at, there, there == 0xffffu && (!verify || pos0 + 15 <= sure), pos0, n - k0, dump ? sm.lb + 2 * c : nullptr, a);
            __syncwarp();
            there_to = here;
            here = here == slots + (kSlotsF - 1) * kBytes ? slots : here + kBytes;
        }
        // --- the item's rows: the warps' parts
        __syncthreads();  // (those of the item before have been read)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            float *dst = &sm.o[warp][2 * c + e][g * (D / 8)];
#pragma unroll
            for (int i = 0; i < D / 16; i += 2)
                *reinterpret_cast<float4 *>(dst + 2 * i) = make_float4(a.o[i][e], a.o[i][e + 2], a.o[i + 1][e], a.o[i + 1][e + 2]);
            float l = a.l[e];
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
            if (g == 0) sm.m[warp][2 * c + e] = -a.nref[e], sm.l[warp][2 * c + e] = l;
        }
        if (tid == 0) open(sm.w[turn ^ 1]);
        __syncthreads();
        if (sm.item < num_items) look_up(sm.w[turn ^ 1]);
        constexpr int C4 = D / 4;  // four dimensions a thread
        if (tid < 8 * C4) {
            const int r = tid / C4, d = (tid - r * C4) * 4;
            if (r < rows) {
                float mx = neg_inf(), l = 0.f;
#pragma unroll
                for (int s = 0; s < kWarpsF; ++s)
                    if (sm.l[s][r] != 0.f) mx = fmaxf(mx, sm.m[s][r]);  // (a sum of 0 has no reference)
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int s = 0; s < kWarpsF; ++s) {
                    const float ls = sm.l[s][r], f = ls == 0.f ? 0.f : ex2_approx(sm.m[s][r] - mx);
                    const float4 o = *reinterpret_cast<const float4 *>(&sm.o[s][r][d]);
                    l += f * ls;
                    v.x += f * o.x, v.y += f * o.y, v.z += f * o.z, v.w += f * o.w;
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
                v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
                const int j = w.verify ? r / p.G : 0, gi = r - j * p.G;
                if (w.nsplit == 1)
                    *reinterpret_cast<uint2 *>(p.out + ((size_t)(w.q_off + j) * p.Hq + (size_t)w.g * p.G + gi) * D + d) =
                        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                else
                    *reinterpret_cast<float4 *>(p.part_o + ((size_t)w.rec + r) * D + d) = v;
                if (d == 0) {
                    const float z = l > 0.f ? mx * 0.69314718f + logf(l) : (l == 0.f ? neg_inf() : l);  // (a NaN sum stays one)
                    if (w.nsplit > 1) p.part_lse[(size_t)w.rec + r] = z;
                    else if (w.verify) p.lse[((size_t)w.vidx * p.Hq + (size_t)w.g * p.G + gi) * (p.k + 1) + j] = z;
                }
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (bad) atomicOr(&p.hdr->err, bad);
    // (what follows on the stream waits for this kernel: let that mean the verify items' kernel, too)
    if (fp.after) pdl_wait_prerequisites();
}

template <int D>
cudaError_t launch_t(const FewParams &p, int nsm, cudaStream_t st) {
    constexpr int kSmem = (int)sizeof(SmemF<D>);
    static_assert(kCtasF * (kSmem + 1024) <= 228 * 1024, "the CTAs of an SM");
    static unsigned long long configured[kMaxDevices] = {};
    int dev = 0;
    unsigned long long ctx = 0;
    cudaError_t e = current_device_context(&dev, &ctx);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (ctx == 0 || __atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE) != ctx) {
        e = cudaFuncSetAttribute(attn_kv4_few_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        e = current_device_context(&dev, &ctx);  // (the calls above made a context current)
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], ctx, __ATOMIC_RELEASE);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtasF * nsm);
    cfg.blockDim = dim3(kThreadsF);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_kv4_few_kernel<D>, p);
}

}  // namespace

cudaError_t launch_attn_kv4_few(const Kv4Params &p, int D, bool after, int nsm, cudaStream_t st) {
    FewParams f;
    f.p = p;
    f.few_only = p.M <= kFewRows;
    f.counter = f.few_only ? &p.hdr->item_counter : &p.hdr->draft_counter;
    f.after = after;
    return D == 128 ? launch_t<128>(f, nsm, st) : launch_t<64>(f, nsm, st);
}

}  // namespace pillar
