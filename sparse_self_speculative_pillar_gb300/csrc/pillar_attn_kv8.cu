// pillar_attn_kv8.cu -- the unified draft/verify attention over the 8-bit cache.
//
// The step of pillar_attn.cu with K and V read as e4m3 codes and a scale per
// (block of 16 tokens, KV head): for query row r and key t in block j
//     s[r, t] = scale * ks[j, g] * (q_r . k8_t)
//     o[r]    = sum_t e^(s[r, t] - m) vs[j, g] v8_t / sum_t e^(s[r, t] - m)
// The planner, its work items, the partial records and the merge of split
// units are those of the bf16 step; only the kernel between them differs.
//
// What bounds it: the bytes of the cache (2 D per key and head) and, for
// verify rows, the fp32 logits; and next to them the work of turning 8-bit codes
// into tensor-core operands, which decided the shape of the kernel:
//   * Every e4m3 value is an f16 value, and a bf16 query row divided by a power of
//     two (its largest magnitude brought to [2^14, 2^15)) is one too, but for
//     elements 2^-28 below that, whose rounding (2^-39 of it) fp32 would not see.
//     So q . k8 is a sum of exact products with f16 operands, as with bf16 keys.
//     (mma with e4m3 operands would take the codes as they are, but this GPU
//     converts them to f16 inside the instruction, for every use: measured 590 to
//     700 pairs a cycle and SM with operands that change, 960 with f16 ones; a
//     kernel on it took 447 us where this one takes 211.  tcgen05 takes the codes
//     as they are, with the keys on its M and queries and probabilities split into
//     two and three e4m3 values: a kernel of specialised warps on it took 250 us,
//     and 202 for the second batch below (this one: 200); its roles' code did not fit the
//     instruction cache together, and it is not kept.)
//   * The keys are the m of m16n8k16, the query rows its n: S^T = K Q^T and
//     O^T = V^T P^T.  A tile of eight rows wastes little, its O^T is 32 registers a
//     lane, and above all an operand made of K or V serves every row tile of its
//     warp.
//   * The order of the reduction index is free as long as both operands use the
//     same one.  Within a row, lane c of four takes bytes [16c, 16c + 16) (and
//     the same 64 further on), so that a 16-byte load holds the lane's part of
//     four steps; V's rows are read whole by eight lanes, a byte permute pairs two
//     keys' values of a dimension, and one conversion makes an operand register.
//     Among 16 keys, m = g and g + 8 are keys 2g and 2g + 1, so that a lane holds
//     neighbours: their scales are one load, their logits one store.
//     P is transposed between the products by movmatrix.
//   * K and V rows land in shared memory by 16-byte asynchronous copies, their
//     16-byte chunks XOR-ed with the row so that these loads meet no bank twice.
//   * P is rounded to f16 with the scale of its key's values in it, relative to
//     the largest value scale its warp has met: weights are at most 2^15, and at
//     least 2^7 for the row's largest probability at the largest scale.  A row's
//     reference maximum moves only when a score passes it by more than 2^8, which
//     a vote of the warp finds out: no reductions on most steps.
// Two CTAs of eight warps per SM (three where items have at most eight rows: 211 us
// against 233 for the first batch below) work through items of the planner's queue, 128
// keys at a time out of a ring of 64-key stages that all threads fill.  The warps
// share an item's row tiles, two each, and its keys, 16 at a time, and join
// through shared memory at the item's end; meanwhile the other CTA's loads keep
// coming.  Five or six row tiles are three groups of three, three and two warps (in
// four groups of two, one of them idle, the second batch below took 254 us where
// this took 237).  The time of a step is the latency of its chain of conversions,
// products and exponentials, about 3000 cycles for 32 keys: sixteen warps of two row
// tiles hide it better than eight to twelve of three, which one CTA with loader warps
// of its own had (345 us against 233 with two CTAs).
// Measured (32 heads on 8, D = 128): 64 single rows over contexts of 1000 to 30000
// tokens 211 us, 4.6 TB/s of cache or 0.69 of a copy's rate; 128 requests with contexts
// of 6144 to 10240, one ninth of them verify with 9 tokens, 200 us, 0.36: slower than the
// bf16 step, which takes 170 on the same batch.  Drafts alone (the same lengths, lists of a
// twentieth) take 61 us, the bf16 step 63; D = 64, the second batch 150 (150) and the first
// 150 (352, with the dump that the bf16 step always writes).  Copies of this
// kernel that leave out the products, or the copies, say which side it is: 134 and
// 145 of 170 us for single rows over 4000 to 6000 tokens (two CTAs), 100 and 222 of 238
// for the second batch (before its last two steps).
#include "pillar_device.cuh"

namespace pillar {

namespace {

constexpr int kThreads8 = 256;
constexpr int kWarps8 = kThreads8 / 32;
constexpr int kStep = 128;          // keys between two barriers
constexpr int kPairs = 4;           // steps whose rows are resolved ahead
constexpr int kLead = 3;            // steps before its end at which an item's successor is taken from the queue (at its start,
                                    // it waits behind a long item: 237 us for the second batch above where this then took 214)
// The kernel's two forms.  Where an item has at most eight rows (kOne: plain decoding, short drafts) a warp's accumulators
// are half as many, and three CTAs of four stages fit on an SM.
template <bool kOne>
struct Form {
    static constexpr int kCtas = kOne ? 3 : 2;
    static constexpr int kStages = kOne ? 4 : 5;        // 64-key stages: two being read, the others in flight
    static constexpr int kItemTiles = kOne ? 1 : kMaxRows / 8;  // row tiles of an item
    static constexpr int kTiles = kOne ? 1 : 2;         // row tiles of a warp, at most
};
constexpr int kBlk = PILLAR_KV_BLOCK;
constexpr float kGrowLog2 = 8.f;    // a row's reference maximum moves once a score passes it by more than 2^8
constexpr float kWeight = 128.f;    // weight of a probability of 1 at the largest value scale: times 2^8 it is 2^15

struct Kv8Params {
    const uint16_t *q;
    Kv8Cache c;
    const int *sparse_idx;
    uint16_t *out;
    float *logits, *lse;  // logits may be null
    WsHeader *hdr;
    const ReqInfo *req;
    const long long *logit_off;
    const UnitInfo *unit;
    const Item *items;
    float *part_o, *part_lse;
    int Hq, Hkv, G, k, M, max_sparse;
    float scale;
};

// A work item (in shared memory: the registers are needed elsewhere).
struct Work {
    int b, g, begin, n, L, q_off, vidx, nsplit, rec, verify;
    long long logit_off;
};

struct RowInfo {
    long long logits;  // offset of the row's logit at position 0 (-1: none to write)
    int lim;           // last position it sees
    int pad;
};

// The records of the item after this one, copied while this one runs.
struct alignas(16) Ahead {
    Item item;
    ReqInfo req;
    UnitInfo unit;
    long long logit_off;
};

template <int D>
struct Stage8 {
    alignas(128) uint8_t k[kTileKeys * D];
    uint8_t v[kTileKeys * D];
    float ks[kTileKeys], vs[kTileKeys];
};

template <int D, bool kOne>
struct Smem8 {
    Stage8<D> stage[Form<kOne>::kStages];
    uint2 q[Form<kOne>::kItemTiles][D / 16][32];    // query operands: row tile, step, lane
    float fac[kMaxRows];               // per row: logit = sum * fac * ks
    RowInfo rows[kMaxRows];
    int row[kPairs][kStep];            // rows of the pools ((block * Hkv + g) * 16 + position % 16), or -1
    unsigned mask[kPairs][kStep / 32]; // which of 32 keys there are
    Ahead ahead;
    Work w[2];                         // this item and the next, in turn
    int item;                          // index of the next one
};

// How an item's row tiles are shared out: `groups` of warps, `tiles` row tiles each.  A group's warps share the keys; of
// three groups the last has two warps, the others three.
struct Split {
    int tiles, groups;
    __device__ __forceinline__ int of(int warp) const { return warp * groups / kWarps8; }
    __device__ __forceinline__ int first(int gr) const { return groups == 3 ? 3 * gr : gr * (kWarps8 / groups); }
    __device__ __forceinline__ int warps(int gr) const { return groups == 3 ? (gr == 2 ? 2 : 3) : kWarps8 / groups; }
};
static_assert(kWarps8 == 8 && kMaxRows == 64 && Form<false>::kTiles == 2, "one to four groups of eight warps");
__device__ __forceinline__ Split split_of(int rows) {
    const int nrt = (rows + 7) / 8;
    return {min(nrt, 2), (nrt + 1) / 2};
}

// Byte offset of 16-byte chunk c of row r.  K: the two rows that eight lanes read together differ in bit 1
// of r; V: the four rows differ in bits 2 and 3.  (At D = 64 two rows make one 128-byte line.)  The XORs do
// not depend on multiples of 16 of the row, so an offset is a lane's base plus a constant.
template <int D>
__device__ __forceinline__ int k_chunk(int r, int c) {
    if (D == 128) return r * 128 + (c ^ ((r & 2) << 1)) * 16;
    return (r >> 1) * 128 + ((((r & 1) << 2) | c) ^ ((r & 2) << 1)) * 16;
}
template <int D>
__device__ __forceinline__ int v_chunk(int r, int c) {
    if (D == 128) return r * 128 + (c ^ (((r >> 2) & 3) << 1)) * 16;
    return (r >> 1) * 128 + ((((r & 1) << 2) | c) ^ (((r >> 2) & 3) << 1)) * 16;
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp8(uint32_t dst, const void *src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Two e4m3 codes (low half of the word) as f16 values.
__device__ __forceinline__ uint32_t f16x2_of(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    return h;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    return h;
}
// The transpose of an 8 x 8 tile of 16-bit values (lane t: row t / 4, columns 2 (t % 4) and the next).
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

// Rows 2c and 2c + 1 of each row tile, as the eight lanes with this c hold them.
template <int D, int kTiles>
struct Acc {
    float o[kTiles][D / 16][4];  // O^T: dimension of lane g and the next one, rows 2c and 2c + 1
    float m[kTiles][2], l[kTiles][2], fac[kTiles][2];  // reference maximum, this lane's part of the sum
    float wsc, vmax;                 // weight of a probability = p * vs * wsc; largest |vs| so far
};

// What a warp knows about its item beyond the record.
struct Part {
    int rows, row0;  // rows of the item, first row of this warp's tiles
    int share, kg;   // warps that share the keys, this one's number among them
    int sure;        // every row sees up to here
};

// 16 NK keys of a stage, from its row r0 on, for the first NT row tiles of a warp.  vis: which of 32 keys from
// r0 on there are; all: the rows see every one; pos0: position of the first (verify); left: keys of the item from
// the first one on.
template <int D, int NT, int NK, int kTiles>
__device__ __forceinline__ void keys8(const Kv8Params &p, const Stage8<D> &st, int r0,
                                      unsigned vis, bool all, int pos0, int left, const uint2 (*q)[D / 16][32],
                                      const RowInfo *rows, bool dump, Acc<D, kTiles> &a) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    float s[NK][NT][4];  // keys 16 h + 2 g and the next, rows 2c and 2c + 1
#pragma unroll
    for (int h = 0; h < NK; ++h)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][t][e] = 0.f;
    const uint8_t *kb = st.k + r0 * D + k_chunk<D>(2 * g, c);
    const int flip = (g & 1) ? -64 : 64;                // the chunk four further on, under the XOR,
    const int odd = D == 128 ? D : flip;                // and the next key
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        uint4 x[NK][2];
#pragma unroll
        for (int h = 0; h < NK; ++h)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                x[h][e] = *reinterpret_cast<const uint4 *>(kb + (i ? flip : 0) + 16 * h * D + (e ? odd : 0));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint2 b[NT];
#pragma unroll
            for (int t = 0; t < NT; ++t) b[t] = q[t][4 * i + j][lane];
#pragma unroll
            for (int h = 0; h < NK; ++h) {
                const uint32_t w0 = j == 0 ? x[h][0].x : j == 1 ? x[h][0].y : j == 2 ? x[h][0].z : x[h][0].w;
                const uint32_t w1 = j == 0 ? x[h][1].x : j == 1 ? x[h][1].y : j == 2 ? x[h][1].z : x[h][1].w;
                const uint32_t a0 = f16x2_of(w0), a1 = f16x2_of(w1), a2 = f16x2_of(w0 >> 16), a3 = f16x2_of(w1 >> 16);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(s[h][t], a0, a1, a2, a3, b[t].x, b[t].y);
            }
        }
    }
    // scale, mask, dump; does a score pass its row's reference?
    bool grow = false;
#pragma unroll
    for (int h = 0; h < NK; ++h) {
        const float2 ks = *reinterpret_cast<const float2 *>(st.ks + r0 + 16 * h + 2 * g);
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) s[h][t][e] *= a.fac[t][e & 1] * (e < 2 ? ks.x : ks.y);
            if (!all) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = 16 * h + 2 * g + (e >> 1);
                    if (!((vis >> key) & 1) || pos0 + key > rows[8 * t + 2 * c + (e & 1)].lim) s[h][t][e] = neg_inf();
                }
            }
#pragma unroll
            for (int e = 0; e < 2; ++e)
                grow |= (fmaxf(s[h][t][e], s[h][t][e + 2]) - a.m[t][e]) * kLog2e > kGrowLog2;
        }
    }
    if (dump) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const long long lb = rows[8 * t + 2 * c + e].logits;
                if (lb < 0) continue;
                float *dst = p.logits + lb + pos0 + 2 * g;  // eight lanes write 64 bytes of a row
#pragma unroll
                for (int h = 0; h < NK; ++h) {
                    const int key = 16 * h + 2 * g;
                    if (key + 2 <= left && !(reinterpret_cast<uintptr_t>(dst) & 7)) {
                        *reinterpret_cast<float2 *>(dst + 16 * h) = make_float2(s[h][t][e], s[h][t][e + 2]);
                    } else {
                        if (key < left) dst[16 * h] = s[h][t][e];
                        if (key + 1 < left) dst[16 * h + 1] = s[h][t][e + 2];
                    }
                }
            }
    }
    // the value scales of the keys
    float vw[NK][2];
    float tm = 0.f;
#pragma unroll
    for (int h = 0; h < NK; ++h)
    {
        const float2 x = *reinterpret_cast<const float2 *>(st.vs + r0 + 16 * h + 2 * g);
        vw[h][0] = x.x, vw[h][1] = x.y;
        tm = fmaxf(tm, fmaxf(fabsf(x.x), fabsf(x.y)));
    }
    grow |= tm > a.vmax;
    if (__any_sync(0xffffffffu, grow)) {  // rare: new reference maxima, a larger value scale
        tm = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(tm)));
        float vf = 1.f;
        if (tm > a.vmax) {
            const float wn = fminf(kWeight / tm, 0x1p126f);
            if (a.vmax > 0.f) vf = wn / a.wsc;
            a.vmax = tm;
            a.wsc = wn;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float f[2];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float mx = a.m[t][e];
#pragma unroll
                for (int h = 0; h < NK; ++h) mx = fmaxf(mx, fmaxf(s[h][t][e], s[h][t][e + 2]));
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
                const float was = a.m[t][e], fl = was == neg_inf() ? 1.f : ex2_approx((was - mx) * kLog2e);
                a.l[t][e] *= fl;
                f[e] = fl * vf;
                a.m[t][e] = mx;
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
                a.o[t][i][0] *= f[0], a.o[t][i][1] *= f[1];
                a.o[t][i][2] *= f[0], a.o[t][i][3] *= f[1];
            }
        }
    }
    uint32_t pb[NK][NT][2];  // P^T operands
#pragma unroll
    for (int h = 0; h < NK; ++h) {
        const float w0 = vw[h][0] * a.wsc, w1 = vw[h][1] * a.wsc;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            float e4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float ref = a.m[t][e & 1];
                e4[e] = ex2_approx(fmaf(s[h][t][e], kLog2e, -(ref == neg_inf() ? 0.f : ref) * kLog2e));
            }
            a.l[t][0] += e4[0] + e4[2];
            a.l[t][1] += e4[1] + e4[3];
            pb[h][t][0] = transpose8x8(pack_f16x2(e4[0] * w0, e4[1] * w0));
            pb[h][t][1] = transpose8x8(pack_f16x2(e4[2] * w1, e4[3] * w1));
        }
    }
    // V: this lane's dimensions (16 at D = 128, 8 at D = 64) of keys 4c .. 4c + 3 (k = 2c, 2c + 8, 2c + 1, 2c + 9)
    constexpr int W = D / 32;  // words per key
    const uint8_t *vb = st.v + r0 * D + (D == 128 ? v_chunk<D>(4 * c, g) : v_chunk<D>(4 * c, g >> 1) + (g & 1) * 8);
    const int next = D == 128 ? 128 : ((c & 2) ? -64 : 64);  // (D = 64: the other half of the line, under the XOR)
#pragma unroll
    for (int h = 0; h < NK; ++h) {
        uint32_t x[4][W];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const uint8_t *src = vb + (16 * h + 2 * (u & 1)) * D + ((u >> 1) ? next : 0);  // key 4c + 2 (u % 2) + u / 2
            if (D == 128) {
                const uint4 y = *reinterpret_cast<const uint4 *>(src);
                x[u][0] = y.x, x[u][1] = y.y, x[u][W - 2] = y.z, x[u][W - 1] = y.w;
            } else {
                const uint2 y = *reinterpret_cast<const uint2 *>(src);
                x[u][0] = y.x, x[u][1] = y.y;
            }
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {  // dimensions 4 i + 2 hf and the next
                const uint32_t ab = __byte_perm(x[0][i], x[1][i], hf ? 0x7362 : 0x5140);
                const uint32_t cd = __byte_perm(x[2][i], x[3][i], hf ? 0x7362 : 0x5140);
                const uint32_t a0 = f16x2_of(ab), a1 = f16x2_of(ab >> 16), a2 = f16x2_of(cd), a3 = f16x2_of(cd >> 16);
#pragma unroll
                for (int t = 0; t < NT; ++t) mma16816(a.o[t][2 * i + hf], a0, a1, a2, a3, pb[h][t][0], pb[h][t][1]);
            }
    }
}

// Dimensions [d, d + 4) of the normalised output of row `row` (query token j, head gi of the group).
__device__ __forceinline__ void store4(const Kv8Params &p, const Work &w, int D, int row, int j, int gi, int d, float4 v) {
    if (w.nsplit == 1)
        *reinterpret_cast<uint2 *>(p.out + ((size_t)(w.q_off + j) * p.Hq + (size_t)w.g * p.G + gi) * D + d) =
            make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    else
        *reinterpret_cast<float4 *>(p.part_o + ((size_t)w.rec + row) * D + d) = v;
}

__device__ __forceinline__ void store_lse(const Kv8Params &p, const Work &w, int row, int j, int gi, float m, float l) {
    const float z = l > 0.f ? m + logf(l) : (l == 0.f ? neg_inf() : l);  // (a NaN sum stays one)
    if (w.nsplit > 1) p.part_lse[(size_t)w.rec + row] = z;
    else if (w.verify) p.lse[((size_t)w.vidx * p.Hq + (size_t)w.g * p.G + gi) * (p.k + 1) + j] = z;
}

// The f16 query operands of row tile t, by one warp: step j, lane (g, c): four elements of row 8 t + g, taken as the K
// loads take bytes (64 (j / 4) + 16 c + 4 (j % 4) on).
template <int D, bool kOne>
__device__ __forceinline__ void stage_queries(const Kv8Params &p, const Work &w, Smem8<D, kOne> &sm, int t, int rows) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3, row = t * 8 + g;
    uint4 x[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x[i] = make_uint4(0, 0, 0, 0);
    if (row < rows) {
        const int j = w.verify ? row / p.G : 0;
        const uint16_t *src = p.q + ((size_t)(w.q_off + j) * p.Hq + (size_t)w.g * p.G + row - j * p.G) * D + c * 16;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            x[2 * i] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * i));
            x[2 * i + 1] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * i + 8));
        }
    }
    uint32_t mx = 0;  // the row's largest magnitude, over the four lanes that share it
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        mx = __vmaxu2(__vmaxu2(__vmaxu2(mx, x[i].x & 0x7fff7fffu), __vmaxu2(x[i].y & 0x7fff7fffu, x[i].z & 0x7fff7fffu)),
                      x[i].w & 0x7fff7fffu);
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = max((int)(mx >> 7), 15);                // biased exponent, such that 2^(141 - e) is finite
    const float up = __int_as_float((268 - e) << 23);     // 2^(141 - e): the largest comes to [2^14, 2^15)
    const float down = __int_as_float((e - 14) << 23);
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const uint32_t wd[8] = {x[2 * i].x,     x[2 * i].y,     x[2 * i].z,     x[2 * i].w,
                                x[2 * i + 1].x, x[2 * i + 1].y, x[2 * i + 1].z, x[2 * i + 1].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sm.q[t][4 * i + j][lane] = make_uint2(pack_f16x2(bf16lo(wd[2 * j]) * up, bf16hi(wd[2 * j]) * up),
                                                  pack_f16x2(bf16lo(wd[2 * j + 1]) * up, bf16hi(wd[2 * j + 1]) * up));
    }
    if (c == 0) {
        sm.fac[row] = down * p.scale;
        RowInfo ri;
        const int j = w.verify ? row / p.G : 0, gi = row - j * p.G;
        ri.logits = row < rows && w.verify && p.logits
                        ? w.logit_off + ((long long)(w.g * p.G + gi) * (p.k + 1) + j) * w.L : -1;
        ri.lim = w.verify ? w.L - (p.k + 1) + j : 0x7fffffff;
        ri.pad = 0;
        sm.rows[row] = ri;
    }
}

template <int D, bool kOne>
__global__ void __launch_bounds__(kThreads8, Form<kOne>::kCtas) attn_kv8_kernel(const __grid_constant__ Kv8Params p) {
    constexpr int kStages = Form<kOne>::kStages, kTiles = Form<kOne>::kTiles;
    extern __shared__ __align__(128) char smem[];
    Smem8<D, kOne> &sm = *reinterpret_cast<Smem8<D, kOne> *>(smem);
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int num_items = *reinterpret_cast<volatile int *>(&p.hdr->num_items);
    int bad = 0;
    // (thread 0 alone copies the records ahead and reads them)
    auto copy_item = [&](int it) { cp16(smem_u32(&sm.ahead.item), p.items + it, 16); };
    auto copy_unit = [&]() {
        const int unit = sm.ahead.item.unit, b = unit / p.Hkv;
        cp16(smem_u32(&sm.ahead.req), p.req + b, 16);
        cp16(smem_u32(&sm.ahead.unit), p.unit + unit, 16);
        cp8(smem_u32(&sm.ahead.logit_off), p.logit_off + b);
    };
    auto open_item = [&](Work &w) {  // from the records ahead
        const Ahead &n = sm.ahead;
        w.b = n.item.unit / p.Hkv;
        w.g = n.item.unit - w.b * p.Hkv;
        w.begin = n.item.begin;
        w.n = n.item.end - n.item.begin;
        w.L = n.req.len;
        w.q_off = n.req.q_off;
        w.vidx = n.req.vidx;
        w.nsplit = n.unit.nsplit;
        w.rec = n.unit.rec_base + n.item.split * n.unit.rec_rows;
        w.verify = n.req.mode == 1;
        w.logit_off = w.verify ? n.logit_off : 0;
    };
    int next = 0, done = 0;  // how far thread 0 is with the next item: 0 nothing, 1 its index, 2 its item record, 3 all of them
    if (tid == 0) {
        const int it = atomicAdd(&p.hdr->item_counter, 1);
        sm.item = it;
        if (it < num_items) {
            copy_item(it);
            cp_wait<0>();  // (thread 0 has committed nothing: the next line does)
            cp_commit();
            cp_wait<0>();
            copy_unit();
            cp_commit();
            cp_wait<0>();
            open_item(sm.w[0]);
        }
    }
    __syncthreads();
    auto position = [&](const Work &w, int t) {  // of key tid of step t; -1: no such key
        const int i = t * kStep + tid;
        if (i >= w.n) return -1;
        if (w.verify) return w.begin + i;
        const int pos = __ldg(p.sparse_idx + ((size_t)w.b * p.Hkv + w.g) * p.max_sparse + w.begin + i);
        if (pos < 0 || pos >= w.L) {
            bad |= PILLAR_FLAG_INDEX;
            return -1;
        }
        return pos;
    };
    auto block = [&](const Work &w, int pos) {
        return pos >= 0 && pos / kBlk < p.c.max_blocks ? __ldg(p.c.table + (size_t)w.b * p.c.max_blocks + pos / kBlk) : -1;
    };
    // the positions of an item's first steps: looked up while the item before is being joined
    int pos[5];
    const bool finds = tid < kStep;
    auto positions = [&](const Work &w) {
        const bool any = finds && sm.item < num_items;
#pragma unroll
        for (int t = 0; t < 5; ++t) pos[t] = any ? position(w, t) : -1;
    };
    positions(sm.w[0]);
    for (int turn = 0; sm.item < num_items; turn ^= 1) {
        const Work &w = sm.w[turn];
        done = 0;
        const int steps = (w.n + kStep - 1) / kStep;
        // --- the loads.  Thread tid < 128 finds key tid of each step: its position, its block, its row of the
        // pools, one link of that chain a step, so that each has a step's time to arrive.  The rows go
        // through shared memory to the copies, in which the 16-byte pieces of a row belong to adjacent lanes.
        auto resolve = [&](int t, int pos, int blk) {  // (the first four warps, whole)
            const bool ok = pos >= 0 && blk >= 0 && blk < p.c.num_blocks;
            if (pos >= 0 && !ok) bad |= PILLAR_FLAG_SLOT;
            sm.row[t % kPairs][tid] = ok ? (blk * p.Hkv + w.g) * kBlk + pos % kBlk : -1;
            const unsigned m = __ballot_sync(0xffffffffu, ok);
            if (lane == 0) sm.mask[t % kPairs][warp] = m;
        };
        auto fetch = [&](int s) {  // 64-key stage s of the item
            constexpr int RL = D / 16, RP = kThreads8 / RL;  // lanes of a row, rows of a pass
            Stage8<D> &st = sm.stage[s % kStages];
            const int *rows = sm.row[(s >> 1) % kPairs] + (s & 1) * kTileKeys;
            const int ch = tid % RL;
            const uint32_t kd = smem_u32(st.k), vd = smem_u32(st.v);
#pragma unroll
            for (int i = 0; i < kTileKeys / RP; ++i) {
                const int r = i * RP + tid / RL, at = rows[r];
                const size_t src = (size_t)max(at, 0) * D + ch * 16;
                const int bytes = at >= 0 ? 16 : 0;  // (no key: zeros)
                cp16(kd + k_chunk<D>(r, ch), p.c.k8 + src, bytes);
                cp16(vd + v_chunk<D>(r, ch), p.c.v8 + src, bytes);
            }
            if (tid < 2 * kTileKeys) {
                const int r = tid & (kTileKeys - 1), at = rows[r], unit = max(at, 0) / kBlk, bytes = at >= 0 ? 4 : 0;
                if (tid < kTileKeys) cp4(smem_u32(&st.ks[r]), p.c.k_scale + unit, bytes);
                else cp4(smem_u32(&st.vs[r]), p.c.v_scale + unit, bytes);
            }
        };
        int pos_r = -1, blk_r = -1, pos_b = -1;
        if (finds) {
            int blk[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) blk[t] = block(w, pos[t]);
#pragma unroll
            for (int t = 0; t < 3; ++t) resolve(t, pos[t], blk[t]);
            pos_r = pos[3], blk_r = blk[3], pos_b = pos[4];
        }
        __syncthreads();
#pragma unroll
        for (int s = 0; s < kStages - 2; ++s) {
            if (s < 2 * steps) fetch(s);
            cp_commit();
        }
        Part pt;
        pt.rows = w.verify ? p.M : p.G;
        const Split sp = split_of(pt.rows);
        const int gr = sp.of(warp);
        pt.kg = warp - sp.first(gr);
        pt.share = sp.warps(gr);
        pt.row0 = gr * sp.tiles * 8;
        pt.sure = w.verify ? w.L - (p.k + 1) : 0x7fffffff;
        if (warp < sp.groups * sp.tiles) stage_queries<D, kOne>(p, w, sm, warp, pt.rows);  // (rows of the groups' last tiles that there are not, too)
        __syncthreads();
        Acc<D, kTiles> a;
        a.wsc = 0x1p126f;
        a.vmax = 0.f;
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                a.m[t][e] = neg_inf();
                a.l[t][e] = 0.f;
                a.fac[t][e] = t < sp.tiles ? sm.fac[pt.row0 + 8 * t + 2 * c + e] : 0.f;
            }
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) a.o[t][i][e] = 0.f;
        }
        const uint2(*q)[D / 16][32] = &sm.q[pt.row0 / 8];
        const RowInfo *rinfo = sm.rows + pt.row0;
        const bool dump = w.verify && p.logits, one = pt.rows - pt.row0 <= 8;
        for (int t = 0; t < steps; ++t) {
            cp_wait<kStages - 4>();
            __syncthreads();  // stages 2t and 2t+1 are in shared memory, and those of step t-1 are free
            // the next item, one link a step; not before it is needed, so that no item waits behind a long one
            if (tid == 0 && t + kLead >= steps && done < 3) {
                if (done == 0) next = atomicAdd(&p.hdr->item_counter, 1);
                else if (next < num_items) done == 1 ? copy_item(next) : copy_unit();
                ++done;
            }
#pragma unroll
            for (int s = 2 * t + kStages - 2; s < 2 * t + kStages; ++s) {
                if (s < 2 * steps) fetch(s);
                cp_commit();
            }
            if (finds) {
                resolve(t + 3, pos_r, blk_r);
                pos_r = pos_b;
                blk_r = block(w, pos_b);
                pos_b = position(w, t + 5);
            }
#pragma unroll 1
            for (int q16 = pt.kg; q16 < kStep / 16; q16 += pt.share) {
                const int k0 = t * kStep + 16 * q16;
                if (k0 >= w.n) break;
                const unsigned vis = (sm.mask[t % kPairs][q16 >> 1] >> (16 * (q16 & 1))) & 0xffffu;
                const int pos0 = w.verify ? w.begin + k0 : 0;
                const bool all = vis == 0xffffu && (!w.verify || pos0 + 15 <= pt.sure);
                const Stage8<D> &st = sm.stage[(2 * t + (q16 >> 2)) % kStages];
                if constexpr (!kOne) {
                    if (!one) {
                        keys8<D, 2, 1>(p, st, 16 * (q16 & 3), vis, all, pos0, w.n - k0, q, rinfo, dump, a);
                        continue;
                    }
                }
                keys8<D, 1, 1>(p, st, 16 * (q16 & 3), vis, all, pos0, w.n - k0, q, rinfo, dump, a);
            }
        }
        if (tid == 0) {  // (a short item: the rest of the next one's records)
            if (done == 0) next = atomicAdd(&p.hdr->item_counter, 1);
            sm.item = next;
            if (next < num_items) {
                cp_wait<0>();
                if (done <= 1) {
                    copy_item(next);
                    cp_commit();
                    cp_wait<0>();
                }
                if (done <= 2) copy_unit();
                cp_commit();
                cp_wait<0>();
                open_item(sm.w[turn ^ 1]);
            }
        }
        // --- the item's rows: the warps that shared the keys of a row tile join, one tile of each group at a time
        const float unw = 1.f / a.wsc;
        float(*so)[8][D + 4] = reinterpret_cast<float(*)[8][D + 4]>(sm.stage);  // [warps][8][D + 4]
        float(*smx)[8] = reinterpret_cast<float(*)[8]>(so + kWarps8), (*sl)[8] = smx + kWarps8;
        static_assert(sizeof(float) * kWarps8 * 8 * (D + 6) <= sizeof(sm.stage), "the join fits into the stages");
        cp_wait<0>();
        __syncthreads();  // (the keys are done with, the next item is there)
        positions(sm.w[turn ^ 1]);
#pragma unroll
        for (int t = 0; t < kTiles; ++t) {
            if (t >= sp.tiles) break;
            if (t > 0) __syncthreads();
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float *dst = &so[warp][2 * c + e][g * (D / 8)];
#pragma unroll
                for (int i = 0; i < D / 16; i += 2)
                    *reinterpret_cast<float4 *>(dst + 2 * i) =
                        make_float4(a.o[t][i][e] * unw, a.o[t][i][e + 2] * unw, a.o[t][i + 1][e] * unw,
                                    a.o[t][i + 1][e + 2] * unw);
                float l = a.l[t][e];
#pragma unroll
                for (int o = 4; o <= 16; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
                if (g == 0) smx[warp][2 * c + e] = a.m[t][e], sl[warp][2 * c + e] = l;
            }
            __syncthreads();
            constexpr int C4 = D / 4;  // four dimensions a thread
            for (int x = tid; x < sp.groups * 8 * C4; x += kThreads8) {
                const int gr = x / (8 * C4), y = x - gr * 8 * C4, lr = y / C4, d = (y - lr * C4) * 4;
                const int row = (gr * sp.tiles + t) * 8 + lr, w0 = sp.first(gr), share = sp.warps(gr);
                if (row >= pt.rows) continue;
                float mx = neg_inf(), l = 0.f;
                for (int s = 0; s < share; ++s) mx = fmaxf(mx, smx[w0 + s][lr]);
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                if (mx > neg_inf()) {
                    for (int s = 0; s < share; ++s) {
                        const float f = ex2_approx((smx[w0 + s][lr] - mx) * kLog2e);
                        const float4 o = *reinterpret_cast<const float4 *>(&so[w0 + s][lr][d]);
                        l += f * sl[w0 + s][lr];
                        v.x += f * o.x, v.y += f * o.y, v.z += f * o.z, v.w += f * o.w;
                    }
                } else {
                    for (int s = 0; s < share; ++s) l += sl[w0 + s][lr];  // 0, or a NaN
                }
                const float inv = l == 0.f ? 0.f : 1.f / l;
                v.x *= inv, v.y *= inv, v.z *= inv, v.w *= inv;
                const int j = w.verify ? row / p.G : 0, gi = row - j * p.G;
                store4(p, w, D, row, j, gi, d, v);
                if (d == 0) store_lse(p, w, row, j, gi, mx, l);
            }
        }
    }
    if (bad) atomicOr(&p.hdr->err, bad);
}

template <int D, bool kOne>
cudaError_t launch_t(const Kv8Params &p, int nsm, cudaStream_t st) {
    constexpr int kSmem = (int)sizeof(Smem8<D, kOne>);
    static_assert(Form<kOne>::kCtas * (kSmem + 1024) <= 228 * 1024, "the CTAs of an SM");
    static unsigned long long configured[kMaxDevices] = {};
    int dev = 0;
    unsigned long long ctx = 0;
    cudaError_t e = current_device_context(&dev, &ctx);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (ctx == 0 || __atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE) != ctx) {
        e = cudaFuncSetAttribute(attn_kv8_kernel<D, kOne>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        e = current_device_context(&dev, &ctx);  // (the calls above made a context current)
        if (e != cudaSuccess) return e;
        __atomic_store_n(&configured[dev], ctx, __ATOMIC_RELEASE);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(Form<kOne>::kCtas * nsm);
    cfg.blockDim = dim3(kThreads8);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_kv8_kernel<D, kOne>, p);
}

}  // namespace

cudaError_t launch_attn_kv8(const AttnArgs &a, const Kv8Cache &c, int nsm, cudaStream_t st) {
    Kv8Params p;
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
    const cudaError_t e = p.M <= 8 ? (a.D == 128 ? launch_t<128, true>(p, nsm, st) : launch_t<64, true>(p, nsm, st))
                                : (a.D == 128 ? launch_t<128, false>(p, nsm, st) : launch_t<64, false>(p, nsm, st));
    return e == cudaSuccess ? launch_merge(a, nsm, st) : e;
}

}  // namespace pillar
