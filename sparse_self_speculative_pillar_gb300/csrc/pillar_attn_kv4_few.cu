// pillar_attn_kv4_few.cu -- the 4-bit attention's items of at most 24 query rows: drafts, plain decoding, short verify
// steps.
//
// Every warp works alone on 16 keys at a time: S^T = K Q^T and O^T = V^T P^T
// with m16n8k16, the keys (the dimensions) on m and one to three tiles of eight
// rows on n, both operands f16 (every cache value is one).  Nothing waits for
// another warp before an item's end, where the four warps of the CTA, which share
// its keys, join through shared memory.
//   * The codes come by 16-byte asynchronous copies into three slots of the warp's
//     own.  K: lane c of four has dimensions [32c, 32c + 32) of its key, 16 bytes
//     that hold the operands of all steps.  V: a lane has 16 (D = 128) dimensions of
//     four keys, and two keys' codes are paired into bytes that convert at once.
//   * Among 16 keys m = g and g + 8 are keys 2g and 2g + 1, so that a lane holds
//     neighbours: their logits are one store.  P is transposed between the products
//     by movmatrix.
//   * Each warp has reference maxima of its own; one moves when a score passes it
//     by more than 2^8, which a vote of the warp finds out.
//
// What bounds it.  64 contexts of 1000 to 30000 keys, four rows (32 heads on 8, D = 128): 138 us a call, 549 MB, 4.0 TB/s; some
// 370 instructions for 16 keys, issued in 0.65 of the schedulers' cycles by sixteen warps an SM (per issue 1.3 warps wait for
// fixed latencies, 0.16 for memory).  Lists (128 requests, 300 to 520 keys each): 52 us a call for 63 MB, the chain of queue, list,
// table and rows at an item's start and accesses of 64 bytes; issue 0.37.  One row tile on tcgen05 with the roles of
// pillar_attn_kv4.cu: 215 us where this took 184.  Two CTAs of eight warps instead of four of four: 157 where this took 143.
#include "pillar_attn_kv4.cuh"

namespace pillar {

namespace {

constexpr int kWarps = 4, kThreads = kWarps * 32;
template <int NT>
constexpr int kCtas = 5 - NT;  // CTAs of an SM (more would take the registers that hold O)
constexpr int kSlots = 3;  // 16-key pieces of a warp: one being read, two on their way (four and five of one row tile: no case faster)
constexpr int kPieces = kMaxChunk / 16 / kWarps;  // of a warp in an item, at most
static_assert(kPieces <= 32, "a lane keeps what it knows of a piece");

template <int D>
struct Piece4 {
    static constexpr int kRow = D / 2, kScales = D / kGroup4;
    alignas(128) uint8_t k[16 * kRow];
    uint8_t v[16 * kRow], ks[16 * kScales], vs[16 * kScales];
};

// A work item (in shared memory).
struct Work4 {
    int b, g, begin, n, L, q_off, vidx, nsplit, rec, verify;
    long long logit_off;
};

template <int D, int NT>
struct Smem4 {
    static constexpr int kRows = 8 * NT;
    Piece4<D> piece[kWarps][kSlots];
    // the warps' parts of a row tile; of items of one, O takes the place of its warp's pieces
    float own_o[NT == 1 ? 1 : kWarps][8][NT == 1 ? 4 : D + 4], m[kWarps][8], l[kWarps][8];
    __device__ __forceinline__ float *o(int w, int row) {
        return NT == 1 ? reinterpret_cast<float *>(piece[w]) + row * (D + 4) : own_o[NT == 1 ? 0 : w][row];
    }
    static_assert(8 * (D + 4) * sizeof(float) <= kSlots * sizeof(Piece4<D>), "O in the place of the pieces");
    uint2 q[NT][NT == 1 ? 1 : D / 16][32];                  // more than one row tile: query operands by row tile, step, lane
    alignas(8) float fac[kRows], fac2[kRows];               // per row: logit = sum * fac, fac2 in base 2
    int lim[kRows];                                         // last position seen
    float *lb[kRows];                                       // where its logits at position 0 go, or null
    int row[kWarps][NT == 1 ? kPieces * 16 : 1];            // lists (one row tile): rows of the pools, or -1
    struct alignas(16) {
        Item item;
        ReqInfo req;
        UnitInfo unit;
    } ahead;     // the next item's records
    Work4 w[2];  // this item and the next, in turn
    int item;
};

struct FewParams {
    Kv4Params p;
    int *counter;  // of the items taken
    int part;      // 0: all items, 1: those of verify requests, 2: the others
    bool after;    // launched behind a kernel of the verify items
};

__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global.L2::64B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_scales(uint32_t dst, const void *src, int bytes) {  // (zeros behind `bytes`)
    asm volatile("cp.async.ca.shared.global.L2::64B [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(N) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

// Where a lane's parts of a piece lie, from the piece's first byte on.
template <int D>
struct Place4 {
    uint32_t k, ks, v, vs;
    __device__ __forceinline__ Place4(int g, int c) {
        using Pc = Piece4<D>;
        k = D == 128 ? k_at<D>(2 * g, c) : k_at<D>(2 * g, c >> 1) + (c & 1) * 8;  // (row 2g + 1: ^ Pc::kRow)
        v = 16 * Pc::kRow + (D == 128 ? v_at<D>(4 * c, g >> 1) + (g & 1) * 8 : v_at<D>(4 * c, g >> 2) + (g & 3) * 4);
        ks = 32 * Pc::kRow + 2 * g * Pc::kScales + c * Pc::kScales / 4;
        vs = 32 * Pc::kRow + 16 * Pc::kScales + 4 * c * Pc::kScales + g * Pc::kScales / 8;
    }
};

// What a lane keeps through an item; of row tile t, rows 2c and 2c + 1 are those of accumulator columns 0 and 1.
template <int D, int NT>
struct State4 {
    uint32_t q[NT == 1 ? D / 16 : 1][2];  // query operands (of one row tile)
    float o[NT][D / 16][4];               // O^T: dimensions (D / 8) g + 2i and the next, rows 2c and 2c + 1
    float nref[NT][2], l[NT][2];          // kLift - reference (infinite: none yet); this lane's weights
    bool fresh;                           // a row has no reference yet
};

// 16 keys: those of `vis`; all: every row sees them all; pos0: position of the first (verify); left: keys of the item from it
// on.  dump: the logits are wanted.
template <int D, int NT>
__device__ __forceinline__ void keys16(const Smem4<D, NT> &sm, uint32_t pc, const Place4<D> &at, unsigned vis, bool all, int pos0,
                                       int left, bool dump, State4<D, NT> &a) {
    using Pc = Piece4<D>;
    const int lane = threadIdx.x & 31, c = lane & 3;
    float s[NT][4];  // keys 2g (rows 2c, 2c + 1) and 2g + 1
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] = 0.f;
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
        const uint2 *q = &sm.q[0][0][lane];  // (more than one row tile)
#pragma unroll
        for (int i = 0; i < W; ++i) {
            uint32_t h0[4], h1[4];
            f16_of_e2m1(x[0][i], h0);
            f16_of_e2m1(x[1][i], h1);
#pragma unroll
            for (int e = 0; e < 4; ++e) h0[e] = mul_f16x2(h0[e], sc[0][i >> 1]), h1[e] = mul_f16x2(h1[e], sc[1][i >> 1]);
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int t = 0; t < NT; ++t) {
                    const int j = 2 * i + h;
                    uint2 b;
                    if (NT == 1) b = make_uint2(a.q[NT == 1 ? j : 0][0], a.q[NT == 1 ? j : 0][1]);
                    else b = q[(t * (D / 16) + j) * 32];
                    mma16816(s[t], h0[2 * h], h1[2 * h], h0[2 * h + 1], h1[2 * h + 1], b.x, b.y);
                }
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
        const int g = lane >> 2;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int key = 2 * g + (e >> 1);
                if (!((vis >> key) & 1) || pos0 + key > sm.lim[8 * t + 2 * c + (e & 1)]) s[t][e] = neg_inf();
            }
    }
    if (dump) {
        const int g = lane >> 2;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int r = 8 * t + 2 * c + e;
                float *dst = sm.lb[r];
                if (!dst) continue;
                dst += pos0 + 2 * g;  // eight lanes write 64 bytes of a row
                const float fac = sm.fac[r], y0 = s[t][e] * fac, y1 = s[t][e + 2] * fac;
                if (2 * g + 2 <= left && !(reinterpret_cast<uintptr_t>(dst) & 7)) {
                    asm volatile("st.global.v2.f32 [%0], {%1, %2};" ::"l"(dst), "f"(y0), "f"(y1));
                } else {
                    if (2 * g < left) dst[0] = y0;
                    if (2 * g + 1 < left) dst[1] = y1;
                }
            }
    }
    bool grow = a.fresh;
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        const float2 f = *reinterpret_cast<const float2 *>(&sm.fac2[8 * t + 2 * c]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s[t][e] *= e & 1 ? f.y : f.x;
        grow |= fmaxf(fmaxf(s[t][0], s[t][2]) + a.nref[t][0], fmaxf(s[t][1], s[t][3]) + a.nref[t][1]) > kGrow;
    }
    if (__any_sync(0xffffffffu, grow)) {  // rare: new references
        bool none = false;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = fmaxf(s[t][e], s[t][e + 2]);
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                // (a row's reference goes by its own scores alone; one without has nref = kLift + inf)
                const bool had = a.nref[t][e] < __int_as_float(0x7f800000);
                const float was = kLift - a.nref[t][e], to = !had || mx > was + (kGrow - kLift) ? fmaxf(mx, was) : was;
                const float f = !had || to == was ? 1.f : ex2_approx(was - to);
                a.nref[t][e] = kLift - to;
                none |= to == neg_inf();
                a.l[t][e] *= f;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) a.o[t][i][e] *= f, a.o[t][i][e + 2] *= f;
            }
        a.fresh = none;
    }
    uint32_t pb[NT][2];  // P^T operands
#pragma unroll
    for (int t = 0; t < NT; ++t) {
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // (without a reference a score is -inf, whose weight is 0, or NaN)
            const float ref = a.nref[t][e & 1];
            w[e] = ex2_approx(s[t][e] + (ref == __int_as_float(0x7f800000) ? 0.f : ref));
        }
        a.l[t][0] += w[0] + w[2];
        a.l[t][1] += w[1] + w[3];
        pb[t][0] = transpose8x8(pack_f16x2(w[0], w[1]));
        pb[t][1] = transpose8x8(pack_f16x2(w[2], w[3]));
    }
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
        for (int d = 0; d < 4; ++d)
#pragma unroll
            for (int t = 0; t < NT; ++t) mma16816(a.o[t][4 * i + d], he[0][d], ho[0][d], he[1][d], ho[1][d], pb[t][0], pb[t][1]);
    }
}

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, kCtas<NT>) attn_kv4_few_kernel(const __grid_constant__ FewParams fp) {
    using Pc = Piece4<D>;
    extern __shared__ __align__(128) char smem[];
    Smem4<D, NT> &sm = *reinterpret_cast<Smem4<D, NT> *>(smem);
    const Kv4Params &p = fp.p;
    // (behind the verify items' kernel: its CTAs let this one start once the plan is complete)
    if (!fp.after) pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int first = fp.part == 2 ? __ldcg(&p.hdr->num_verify_items) : 0;
    const int num_items = fp.part == 1 ? __ldcg(&p.hdr->num_verify_items) : __ldcg(&p.hdr->num_items);
    int bad = 0;
    // thread 0 takes the next item one step at a time: its index, its record, the records that names
    int step = 0, next = 0;
    auto advance = [&]() {
        if (step == 0) {
            next = first + atomicAdd(fp.counter, 1);
        } else if (next < num_items) {
            if (step == 1) {
                copy16(smem_u32(&sm.ahead.item), p.items + next);
            } else if (step == kSlots + 1) {  // (a copy is there with the pieces of kSlots - 1 steps on)
                const int unit = sm.ahead.item.unit;
                copy16(smem_u32(&sm.ahead.req), p.req + unit / p.Hkv);
                copy16(smem_u32(&sm.ahead.unit), p.unit + unit);
            }
        }
        ++step;
    };
    static_assert(sizeof(Item) == 16 && sizeof(ReqInfo) == 16 && sizeof(UnitInfo) == 16, "records of 16 bytes");
    auto open = [&](Work4 &w) {  // the next item's record, by thread 0
#pragma unroll 1
        while (step < kSlots + 2) {
            if (step == kSlots + 1) copies_commit(), copies_wait<0>();
            advance();
        }
        copies_commit();
        copies_wait<0>();
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
    // Of its pieces of the item (warp, warp + 4, ..) a lane keeps the first row of piece `lane` (contexts) and which of its keys
    // there are; lists have their rows in shared memory.
    unsigned base = 0, vis = 0;
    State4<D, NT> a;
    const Place4<D> at(g, c);
    uint4 qx[D / 64][2];  // the next item's queries, on their way: row tile `warp` (row tile 0, one only)
    const int qtile = NT == 1 ? 0 : warp;
    auto look_up = [&](const Work4 &w) {  // an item's rows and queries: loads only as far as they depend on none of the others
        const int rows = w.verify ? p.M : p.G, r = qtile * 8 + g, j = w.verify ? r / p.G : 0;
        const int qrow = r < rows ? (w.q_off + j) * p.Hq + w.g * p.G + r - j * p.G : -1;
        const uint16_t *src = p.q + (size_t)max(qrow, 0) * D + c * (D / 4);
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            qx[i][0] = qrow >= 0 ? __ldg(reinterpret_cast<const uint4 *>(src + 16 * i)) : make_uint4(0, 0, 0, 0);
            qx[i][1] = qrow >= 0 ? __ldg(reinterpret_cast<const uint4 *>(src + 16 * i + 8)) : make_uint4(0, 0, 0, 0);
        }
        const int *table = p.c.table + (size_t)w.b * p.c.max_blocks;
        vis = 0;
        if (NT > 1 || w.verify) {  // (items begin at multiples of 64: a piece is a block)
            const int k = (warp + lane * kWarps) * 16, pos = (w.begin + k) / PILLAR_KV_BLOCK;
            base = 0;
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
            for (int m0 = 0; (warp + 2 * m0 * kWarps) * 16 < w.n; m0 += 4) {
                int pos[4], blk[4];
#pragma unroll
                for (int m = 0; m < 4; ++m) {
                    const int k = (warp + (2 * (m0 + m) + (lane >> 4)) * kWarps) * 16 + (lane & 15);
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
    constexpr uint32_t kBytes = sizeof(Pc);
    const uint32_t slots = smem_u32(sm.piece[warp]);
    // A lane copies 16 bytes of rows r and r + RP .. of a piece, K's and V's, and the scales of one key of either.
    constexpr int RC = Pc::kRow / 16, RP = 32 / RC;  // 16-byte pieces of a row, rows of a pass
    const int cr = lane / RC, ch = lane % RC, sr = lane & 15;
    const uint8_t *const k_from = p.c.k4 + lane * 16, *const v_from = p.c.v4 + lane * 16;
    const uint8_t *const s_from = (lane < 16 ? p.c.k_scale : p.c.v_scale) + sr * Pc::kScales;
    const uint32_t s_to = 32 * Pc::kRow + lane * Pc::kScales;
    auto fetch = [&](int j, int pieces, bool verify, uint32_t dst) {
        if (j >= pieces) return;
        const uint32_t bytes = (__shfl_sync(0xffffffffu, vis, j) >> sr & 1) * Pc::kScales;
        // (the codes of a key that is not there: any, its scales are 0)
        if (NT > 1 || verify) {
            const uint32_t row = __shfl_sync(0xffffffffu, base, j);
            const uint8_t *k = k_from + (size_t)row * Pc::kRow, *v = v_from + (size_t)row * Pc::kRow;
#pragma unroll
            for (int i = 0; i < 16 / RP; ++i) {
                copy16(dst + k_at<D>(i * RP + cr, ch), k + i * 512);
                copy16(dst + 16 * Pc::kRow + v_at<D>(i * RP + cr, ch), v + i * 512);
            }
            copy_scales<Pc::kScales>(dst + s_to, s_from + (size_t)row * Pc::kScales, bytes);
        } else {
            const int *rows = sm.row[warp] + j * 16;
#pragma unroll
            for (int i = 0; i < 16 / RP; ++i) {
                const size_t src = (size_t)(unsigned)max(rows[i * RP + cr], 0) * Pc::kRow + ch * 16;
                copy16(dst + k_at<D>(i * RP + cr, ch), p.c.k4 + src);
                copy16(dst + 16 * Pc::kRow + v_at<D>(i * RP + cr, ch), p.c.v4 + src);
            }
            copy_scales<Pc::kScales>(dst + s_to, (lane < 16 ? p.c.k_scale : p.c.v_scale) + (size_t)(unsigned)max(rows[sr], 0) * Pc::kScales, bytes);
        }
    };
    auto pieces_of = [&](const Work4 &w) { return (w.n - warp * 16 + kWarps * 16 - 1) / (kWarps * 16); };  // (0 or less: none)
    auto begin_item = [&](const Work4 &w) {  // its first pieces
        const int pieces = pieces_of(w);
#pragma unroll 1
        for (int j = 0; j < kSlots - 1; ++j) {
            fetch(j, pieces, w.verify, slots + j * kBytes);
            copies_commit();
        }
    };
    // The queries of row tile qtile as operands: in registers (one row tile), or by its warp to shared memory, with what
    // the item's rows go by.
    auto queries = [&](const Work4 &w) {
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
                for (int e = 0; e < 4; e += 2) {
                    const uint32_t b0 = pack_f16x2(bf16lo(wd[e]) * up, bf16hi(wd[e]) * up);
                    const uint32_t b1 = pack_f16x2(bf16lo(wd[e + 1]) * up, bf16hi(wd[e + 1]) * up);
                    const int j = 4 * i + 2 * h + (e >> 1);
                    if (NT == 1) a.q[NT == 1 ? j : 0][0] = b0, a.q[NT == 1 ? j : 0][1] = b1;
                    else sm.q[qtile][j][lane] = make_uint2(b0, b1);
                }
            }
        if (c == 0 && (NT > 1 || warp == 0)) {
            const int rows = w.verify ? p.M : p.G, r = qtile * 8 + g, j = w.verify ? r / p.G : 0, gi = r - j * p.G;
            const float fac = fmaxf(down * p.scale, __int_as_float(1));  // (above 0: a masked score stays -inf)
            sm.fac[r] = fac;
            const int lim = w.verify && r < rows ? w.L - (p.k + 1) + j : 0x7fffffff;
            sm.fac2[r] = softmax_factor(fac, mx, lim);
            sm.lim[r] = lim;
            sm.lb[r] = w.verify && p.logits && r < rows
                           ? p.logits + w.logit_off + ((long long)(w.g * p.G + gi) * (p.k + 1) + j) * w.L : nullptr;
        }
    };
    const bool stages = qtile < NT;  // (rows that there are not, too: zeros)
    bool more = sm.item < num_items;  // (read between two barriers: thread 0 may have the item after next before others start)
    if (more) {
        look_up(sm.w[0]);
        begin_item(sm.w[0]);
        if (stages) queries(sm.w[0]);
    }
    __syncthreads();
    for (int turn = 0; more; turn ^= 1) {
        const Work4 &w = sm.w[turn];
        const bool verify = w.verify, dump = verify && p.logits;
        const int n = w.n, rows = verify ? p.M : p.G, pieces = pieces_of(w);
        const int sure = verify ? w.L - (p.k + 1) : 0x7fffffff;  // every row sees up to here
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) a.nref[t][e] = -neg_inf(), a.l[t][e] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.o[t][i][e] = 0.f;
        }
        a.fresh = true;
        uint32_t here = slots, into = slots + (kSlots - 1) * kBytes;  // the slots of piece j, of the one fetched
#pragma unroll 1
        for (int j = 0; j < pieces; ++j) {
            // (not before it is needed: no item waits behind a long one)
            if (tid == 0 && j + kSlots + 3 >= pieces && step < kSlots + 2) advance();
            fetch(j + kSlots - 1, pieces, verify, into);
            copies_commit();
            copies_wait<kSlots - 1>();
            __syncwarp();
            const int k0 = (warp + j * kWarps) * 16;
            const unsigned there = __shfl_sync(0xffffffffu, vis, j);
            const int pos0 = verify ? w.begin + k0 : 0;
            keys16<D, NT>(sm, here, at, there, there == 0xffffu && (!verify || pos0 + 15 <= sure), pos0, n - k0, dump, a);
            __syncwarp();
            into = here;
            here = here == slots + (kSlots - 1) * kBytes ? slots : here + kBytes;
        }
        if (tid == 0) open(sm.w[turn ^ 1]);
        // --- the item's rows: the warps' parts, one row tile of each group at a time
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            __syncthreads();  // (the parts before have been read; the next item's record is there)
            if (t == 0) more = sm.item < num_items;
            if (t == 0 && more) look_up(sm.w[turn ^ 1]);
            if (t == 1 && more) begin_item(sm.w[turn ^ 1]);  // (what it looked up has come meanwhile)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float *dst = sm.o(warp, 2 * c + e) + g * (D / 8);
#pragma unroll
                for (int i = 0; i < D / 16; i += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * i) =
                        make_float4(a.o[t][i][e], a.o[t][i][e + 2], a.o[t][i + 1][e], a.o[t][i + 1][e + 2]);
                float l = a.l[t][e];
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                if (g == 0) sm.m[warp][2 * c + e] = -a.nref[t][e], sm.l[warp][2 * c + e] = l;
            }
            __syncthreads();
            constexpr int C4 = D / 4;  // four dimensions a thread
#pragma unroll 1
            for (int y = tid; y < 8 * C4; y += kThreads) {
                const int lr = y / C4, d = (y % C4) * 4, r = 8 * t + lr;
                if (r >= rows) continue;
                float mx = neg_inf(), l = 0.f;
#pragma unroll 4
                for (int s = 0; s < kWarps; ++s)
                    if (sm.l[s][lr] != 0.f) mx = fmaxf(mx, sm.m[s][lr]);  // (a sum of 0 has no reference)
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
                for (int s = 0; s < kWarps; ++s) {
                    const float ls = sm.l[s][lr], f = ls == 0.f ? 0.f : ex2_approx(sm.m[s][lr] - mx);
                    const float4 o = *reinterpret_cast<const float4 *>(sm.o(s, lr) + d);
                    l += f * ls;
                    v.x += f * o.x, v.y += f * o.y, v.z += f * o.z, v.w += f * o.w;
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
                v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
                const int j = verify ? r / p.G : 0, gi = r - j * p.G;
                if (w.nsplit == 1)
                    *reinterpret_cast<uint2 *>(p.out + ((size_t)(w.q_off + j) * p.Hq + (size_t)w.g * p.G + gi) * D + d) =
                        make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                else
                    *reinterpret_cast<float4 *>(p.part_o + ((size_t)w.rec + r) * D + d) = v;
                if (d == 0) {
                    const float z = l > 0.f ? mx * 0.69314718f + logf(l) : (l == 0.f ? neg_inf() : l);  // (a NaN sum stays one)
                    if (w.nsplit > 1) p.part_lse[(size_t)w.rec + r] = z;
                    else if (verify) p.lse[((size_t)w.vidx * p.Hq + (size_t)w.g * p.G + gi) * (p.k + 1) + j] = z;
                }
            }
        }
        if (more) {
            if (NT == 1) {
                __syncthreads();  // (O has been read; `more` is every thread's)
                begin_item(sm.w[turn ^ 1]);
            }
            if (stages) queries(sm.w[turn ^ 1]);
        }
        __syncthreads();  // (the next item's queries and rows are there)
    }
    copies_wait<0>();
    // (each CTA has drawn one number past the items: who has the last of these sets the queue up for the next run on the plan)
    if (tid == 0 && sm.item == num_items + (int)gridDim.x - 1) *fp.counter = 0;
    if (bad) atomicOr(&p.hdr->err, bad);
    // (what follows on the stream waits for this kernel: let that mean the verify items' kernel, too)
    if (fp.after) {
        pdl_wait_prerequisites();
        if (blockIdx.x == 0 && tid == 0) p.hdr->item_counter = 0;
    }
}

template <int D, int NT>
cudaError_t launch_t(const FewParams &p, int nsm, cudaStream_t st) {
    constexpr int kSmem = (int)sizeof(Smem4<D, NT>);
    static_assert(kCtas<NT> * (kSmem + 1024) <= 228 * 1024, "the CTAs of an SM");
    static unsigned long long configured[kMaxDevices] = {};
    int dev = 0;
    unsigned long long ctx = 0;
    cudaError_t e = current_device_context(&dev, &ctx);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (ctx == 0 || __atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE) != ctx) {
        e = cudaFuncSetAttribute(attn_kv4_few_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        e = current_device_context(&dev, &ctx);  // (the calls above made a context current)
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], ctx, __ATOMIC_RELEASE);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas<NT> * nsm);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_kv4_few_kernel<D, NT>, p);
}

}  // namespace

cudaError_t launch_attn_kv4_few(const Kv4Params &p, int D, int rows, int part, bool after, int nsm, cudaStream_t st) {
    FewParams f;
    f.p = p;
    f.part = part;
    f.counter = part == 2 ? &p.hdr->draft_counter : &p.hdr->item_counter;
    f.after = after;
    if (rows <= 8) return D == 128 ? launch_t<128, 1>(f, nsm, st) : launch_t<64, 1>(f, nsm, st);
    if (rows <= 16) return D == 128 ? launch_t<128, 2>(f, nsm, st) : launch_t<64, 2>(f, nsm, st);
    return D == 128 ? launch_t<128, 3>(f, nsm, st) : launch_t<64, 3>(f, nsm, st);
}

}  // namespace pillar
