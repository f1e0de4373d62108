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
// verify rows, the fp32 logits.  The arithmetic is small next to them -- at
// most 64 rows per key -- but an 8-bit code has to become a tensor-core
// operand first, so the kernel is built around converting each byte in the
// registers it is consumed from:
//   * mma.m16n8k16 with f16 operands and fp32 accumulators.  Every e4m3 value
//     is an f16 value; a bf16 query row divided by a power of two (its largest
//     magnitude brought to [2^14, 2^15)) is one too, except for elements 2^-28
//     below the row's largest, whose rounding (2^-39 of it) fp32 would not see
//     either.  So q . k8 is a sum of exact products, as with bf16 keys.
//     tcgen05 would want the converted tile written back to shared memory,
//     twice the bytes that the loads bring in, to fill an M of 64 or 128 that
//     at most 64 rows use.
//   * The order of the reduction index is free as long as both operands use the
//     same one.  Within a row, lane c of four takes bytes [16c, 16c + 16) (and
//     the same 64 further on), so a lane's 16-byte loads hold whole operand
//     registers of consecutive steps; within 16 keys, columns n of the two
//     8-key tiles are keys 4 (n / 2) + n % 2 and two further on, so a lane owns
//     four consecutive keys: one 16-byte load of their scales, one 16-byte store
//     of their logits, and its probabilities are in place for the second
//     product.  V's rows are read whole by eight lanes, and one byte permute
//     pairs two keys' values of a dimension.
//   * K and V rows land in shared memory by 16-byte asynchronous copies, their
//     16-byte chunks XOR-ed with the row so that these loads meet no bank twice.
//   * P is rounded to f16 with the scale of its key's values in it, relative to
//     the largest value scale met so far (the accumulator is rescaled when that
//     grows, as it is when the row maximum does): weights stay in [0, 2^15], and
//     those down to 2^-29 of it keep all eleven bits.
// A CTA of four warps works through items of the planner's queue, 64 keys a
// tile.  Rows are padded to tiles of 16: with one such tile each warp takes 16
// of the 64 keys, with two 32, with more all of them, and the warps of a tile
// join at the item's end.
#include "pillar_device.cuh"

namespace pillar {

namespace {

constexpr int kThreads8 = 128;
constexpr int kStages8 = 4;
constexpr int kBlk = PILLAR_KV_BLOCK;
constexpr float kGrowLog2 = 8.f;    // O is rescaled once a row maximum grew by more than 2^8
constexpr float kWeight = 128.f;    // weight of a probability of 1 at the largest value scale: 2^7 * 2^8 <= 2^15
constexpr int kNever = 0x7fffffff;  // position of a key that no row sees

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

template <int D>
struct Stage8 {
    alignas(16) uint8_t k[kTileKeys * D];
    uint8_t v[kTileKeys * D];
    float ks[kTileKeys], vs[kTileKeys];
    int pos[kTileKeys];  // position (verify), 0 (draft), or kNever
};

// Byte offset of 16-byte chunk c of row r.
template <int D>
__device__ __forceinline__ int k_chunk(int r, int c) {
    return D == 128 ? r * 128 + (c ^ ((r & 1) << 2)) * 16 : r * 64 + c * 16;
}
template <int D>
__device__ __forceinline__ int v_chunk(int r, int c) {
    if (D == 128) return r * 128 + (c ^ (((r >> 2) & 3) << 1)) * 16;
    return (r >> 1) * 128 + ((((r & 1) << 2) | c) ^ (((r >> 2) & 3) << 1)) * 16;
}

__device__ __forceinline__ void cp16(void *dst, const void *src, bool ok) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp4(void *dst, const void *src, bool ok) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(ok ? 4 : 0) : "memory");
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
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A work item as every thread of the CTA holds it.
struct Work {
    int b, g, begin, n, L, q_off, vidx, nsplit, rec;
    long long logit_off;
    bool verify;
};

// One of the two query rows of a thread.
struct Row8 {
    int lim;         // last position it sees (-1: no row of the item)
    int j, gi;       // query token, head of the group
    float fac;       // logit = accumulator * fac * ks
    float m, l;      // reference maximum, this thread's part of the sum
    long long lb;    // its logits (-1: none to write)
};

template <int D>
struct Acc {
    float o[D / 8][4];
    Row8 r[2];
    uint32_t q[D / 16][4];
    float wsc;       // weight of a probability = p * vs * wsc
    float vmax;      // largest |vs| so far
};

// Query row `row` of the item as f16 operand registers: q[step][h], q[step][h + 2].
template <int D, int H>
__device__ __forceinline__ void load_row(const Kv8Params &p, const Work &w, int row, int rows, int c, Acc<D> &a) {
    Row8 &r = a.r[H];
    r.lim = -1;
    r.j = r.gi = 0;
    r.fac = 0.f;
    r.m = neg_inf();
    r.l = 0.f;
    r.lb = -1;
    uint4 x[D / 32];
#pragma unroll
    for (int i = 0; i < D / 32; ++i) x[i] = make_uint4(0, 0, 0, 0);
    if (row < rows) {
        r.j = w.verify ? row / p.G : 0;
        r.gi = row - r.j * p.G;
        r.lim = w.verify ? w.L - (p.k + 1) + r.j : kNever - 1;
        const uint16_t *src = p.q + ((size_t)(w.q_off + r.j) * p.Hq + (size_t)w.g * p.G + r.gi) * D + c * 16;
#pragma unroll
        for (int i = 0; i < D / 64; ++i) {
            x[2 * i] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * i));
            x[2 * i + 1] = __ldg(reinterpret_cast<const uint4 *>(src + 64 * i + 8));
        }
        if (w.verify && p.logits) r.lb = w.logit_off + ((long long)(w.g * p.G + r.gi) * (p.k + 1) + r.j) * w.L;
    }
    // the row's largest magnitude, over the four lanes that share it
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
        mx = __vmaxu2(__vmaxu2(__vmaxu2(mx, x[i].x & 0x7fff7fffu), __vmaxu2(x[i].y & 0x7fff7fffu, x[i].z & 0x7fff7fffu)),
                      x[i].w & 0x7fff7fffu);
    mx = max(mx & 0xffffu, mx >> 16);
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const int e = max((int)(mx >> 7), 15);               // biased exponent; 2^(141 - e) stays finite
    const float up = __int_as_float((141 - e + 127) << 23);  // brings it to 2^14
    const float down = __int_as_float((e - 141 + 127) << 23);
    r.fac = down * p.scale;
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        const uint32_t wd[8] = {x[2 * i].x,     x[2 * i].y,     x[2 * i].z,     x[2 * i].w,
                                x[2 * i + 1].x, x[2 * i + 1].y, x[2 * i + 1].z, x[2 * i + 1].w};
#pragma unroll
        for (int s = 0; s < 4; ++s) {  // elements 4s .. 4s+3 of the lane's 16
            a.q[4 * i + s][H] = pack_f16x2(bf16lo(wd[2 * s]) * up, bf16hi(wd[2 * s]) * up);
            a.q[4 * i + s][H + 2] = pack_f16x2(bf16lo(wd[2 * s + 1]) * up, bf16hi(wd[2 * s + 1]) * up);
        }
    }
}

// NG groups of 16 keys of a staged tile, starting with key k0 of the tile.
template <int D, int NG>
__device__ __forceinline__ void tile_keys(const Kv8Params &p, const Work &w, const Stage8<D> &st, int k0, int tile0, int nk,
                                          Acc<D> &a) {
    const int lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    float s[NG][2][4];
#pragma unroll
    for (int q = 0; q < NG; ++q)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            const int row = k0 + q * 16 + 4 * (g >> 1) + (g & 1) + 2 * t;
            uint32_t kw[D / 16];
#pragma unroll
            for (int i = 0; i < D / 64; ++i) {
                const uint4 x = *reinterpret_cast<const uint4 *>(st.k + k_chunk<D>(row, 4 * i + c));
                kw[4 * i] = x.x, kw[4 * i + 1] = x.y, kw[4 * i + 2] = x.z, kw[4 * i + 3] = x.w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) s[q][t][e] = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i) mma16816(s[q][t], a.q[i], f16x2_of(kw[i]), f16x2_of(kw[i] >> 16));
        }
    // scale, mask, dump; the rows' maxima
    float mt[2] = {neg_inf(), neg_inf()};
#pragma unroll
    for (int q = 0; q < NG; ++q) {
        const int kb = k0 + q * 16 + 4 * c;  // this lane's four keys: kb .. kb+3
        const float4 ks = *reinterpret_cast<const float4 *>(st.ks + kb);
        const int4 ps = *reinterpret_cast<const int4 *>(st.pos + kb);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const Row8 &r = a.r[h];
            float v0 = s[q][0][2 * h] * r.fac * ks.x, v1 = s[q][0][2 * h + 1] * r.fac * ks.y;
            float v2 = s[q][1][2 * h] * r.fac * ks.z, v3 = s[q][1][2 * h + 1] * r.fac * ks.w;
            if (ps.x > r.lim) v0 = neg_inf();
            if (ps.y > r.lim) v1 = neg_inf();
            if (ps.z > r.lim) v2 = neg_inf();
            if (ps.w > r.lim) v3 = neg_inf();
            s[q][0][2 * h] = v0, s[q][0][2 * h + 1] = v1, s[q][1][2 * h] = v2, s[q][1][2 * h + 1] = v3;
            mt[h] = fmaxf(mt[h], fmaxf(fmaxf(v0, v1), fmaxf(v2, v3)));
            if (r.lb >= 0) {
                float *dst = p.logits + r.lb + w.begin + tile0 + kb;
                const int odd = (int)(reinterpret_cast<uintptr_t>(dst) & 15);
                if (kb + 4 <= nk && (odd & 7) == 0) {
                    if (odd == 0) {
                        *reinterpret_cast<float4 *>(dst) = make_float4(v0, v1, v2, v3);
                    } else {
                        *reinterpret_cast<float2 *>(dst) = make_float2(v0, v1);
                        *reinterpret_cast<float2 *>(dst + 2) = make_float2(v2, v3);
                    }
                } else {
                    if (kb < nk) dst[0] = v0;
                    if (kb + 1 < nk) dst[1] = v1;
                    if (kb + 2 < nk) dst[2] = v2;
                    if (kb + 3 < nk) dst[3] = v3;
                }
            }
        }
    }
    float f[2] = {1.f, 1.f};
    bool grow = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        Row8 &r = a.r[h];
        mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], 1));
        mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], 2));
        const float mn = fmaxf(r.m, mt[h]);
        if (r.m == neg_inf()) {
            r.m = mn;
        } else if ((mn - r.m) * kLog2e > kGrowLog2) {
            f[h] = ex2_approx((r.m - mn) * kLog2e);
            r.l *= f[h];
            r.m = mn;
            grow = true;
        }
    }
    // the value scales of the tile
    {
        const float2 vs = *reinterpret_cast<const float2 *>(st.vs + 2 * lane);
        const float tm = __uint_as_float(__reduce_max_sync(
            0xffffffffu, max(__float_as_uint(vs.x) & 0x7fffffffu, __float_as_uint(vs.y) & 0x7fffffffu)));
        if (tm > a.vmax) {  // (the same in every warp of the CTA)
            const float wn = fminf(kWeight / tm, 0x1p126f);
            if (a.vmax > 0.f) {
                const float ratio = wn / a.wsc;
                f[0] *= ratio;
                f[1] *= ratio;
                grow = true;
            }
            a.vmax = tm;
            a.wsc = wn;
        }
    }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
            a.o[i][0] *= f[0], a.o[i][1] *= f[0];
            a.o[i][2] *= f[1], a.o[i][3] *= f[1];
        }
    }
#pragma unroll
    for (int q = 0; q < NG; ++q) {
        const int kb = k0 + q * 16 + 4 * c;
        float4 ws = *reinterpret_cast<const float4 *>(st.vs + kb);
        ws.x *= a.wsc, ws.y *= a.wsc, ws.z *= a.wsc, ws.w *= a.wsc;
        uint32_t pa[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            Row8 &r = a.r[h];
            const float nb = -(r.m == neg_inf() ? 0.f : r.m) * kLog2e;
            const float p0 = ex2_approx(fmaf(s[q][0][2 * h], kLog2e, nb)), p1 = ex2_approx(fmaf(s[q][0][2 * h + 1], kLog2e, nb));
            const float p2 = ex2_approx(fmaf(s[q][1][2 * h], kLog2e, nb)), p3 = ex2_approx(fmaf(s[q][1][2 * h + 1], kLog2e, nb));
            r.l += (p0 + p1) + (p2 + p3);
            pa[h] = pack_f16x2(p0 * ws.x, p1 * ws.y);
            pa[h + 2] = pack_f16x2(p2 * ws.z, p3 * ws.w);
        }
        // V: this lane's dimensions of its four keys (a whole 16-byte chunk at D = 128, half of one at D = 64)
        constexpr int W = D / 32;  // words per key
        uint32_t vw[4][W];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            if (D == 128) {
                const uint4 x = *reinterpret_cast<const uint4 *>(st.v + v_chunk<D>(kb + u, g));
                vw[u][0] = x.x, vw[u][1] = x.y, vw[u][W - 2] = x.z, vw[u][W - 1] = x.w;
            } else {
                const uint2 x = *reinterpret_cast<const uint2 *>(st.v + v_chunk<D>(kb + u, g >> 1) + (g & 1) * 8);
                vw[u][0] = x.x, vw[u][1] = x.y;
            }
        }
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {  // two dimensions at a time: bytes (2 hf, 2 hf + 1) of the word
                const uint32_t ab = __byte_perm(vw[0][i], vw[1][i], hf ? 0x7362 : 0x5140);
                const uint32_t cd = __byte_perm(vw[2][i], vw[3][i], hf ? 0x7362 : 0x5140);
                mma16816(a.o[4 * i + 2 * hf], pa, f16x2_of(ab), f16x2_of(cd));
                mma16816(a.o[4 * i + 2 * hf + 1], pa, f16x2_of(ab >> 16), f16x2_of(cd >> 16));
            }
    }
}

// Where the rows of an item go: row r, dimensions [d, d + N) of the normalised output.
template <int D>
__device__ __forceinline__ void store_row(const Kv8Params &p, const Work &w, int row, int j, int gi, int d, const float *v,
                                          int n) {
    if (w.nsplit == 1) {
        uint16_t *dst = p.out + ((size_t)(w.q_off + j) * p.Hq + (size_t)w.g * p.G + gi) * D + d;
        for (int i = 0; i < n; i += 8)
            *reinterpret_cast<uint4 *>(dst + i) =
                make_uint4(pack_bf16x2(v[i], v[i + 1]), pack_bf16x2(v[i + 2], v[i + 3]), pack_bf16x2(v[i + 4], v[i + 5]),
                           pack_bf16x2(v[i + 6], v[i + 7]));
    } else {
        float *dst = p.part_o + ((size_t)w.rec + row) * D + d;
        for (int i = 0; i < n; i += 4) *reinterpret_cast<float4 *>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
    }
}

__device__ __forceinline__ void store_lse(const Kv8Params &p, const Work &w, int row, int j, int gi, float m, float l) {
    const float z = l > 0.f ? m + logf(l) : (l == 0.f ? neg_inf() : l);  // (a NaN sum stays one)
    if (w.nsplit > 1) p.part_lse[(size_t)w.rec + row] = z;
    else if (w.verify) p.lse[((size_t)w.vidx * p.Hq + (size_t)w.g * p.G + gi) * (p.k + 1) + j] = z;
}

template <int D>
__global__ void __launch_bounds__(kThreads8, 3) attn_kv8_kernel(const __grid_constant__ Kv8Params p) {
    extern __shared__ __align__(16) char smem[];
    Stage8<D> *stage = reinterpret_cast<Stage8<D> *>(smem);
    __shared__ int s_item;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, c = lane & 3;
    const int num_items = *reinterpret_cast<volatile int *>(&p.hdr->num_items);
    int bad = 0;
    if (tid == 0) s_item = atomicAdd(&p.hdr->item_counter, 1);
    __syncthreads();
    int it = s_item;
    while (it < num_items) {
        __syncthreads();  // everyone has read s_item, and the last item's shared memory
        if (tid == 0) s_item = atomicAdd(&p.hdr->item_counter, 1);  // the item after this one
        Work w;
        {
            const Item itm = p.items[it];
            w.b = itm.unit / p.Hkv;
            w.g = itm.unit - w.b * p.Hkv;
            const ReqInfo ri = p.req[w.b];
            const UnitInfo ui = p.unit[itm.unit];
            w.begin = itm.begin;
            w.n = itm.end - itm.begin;
            w.L = ri.len;
            w.q_off = ri.q_off;
            w.vidx = ri.vidx;
            w.nsplit = ui.nsplit;
            w.rec = ui.rec_base + itm.split * ui.rec_rows;
            w.verify = ri.mode == 1;
            w.logit_off = w.verify ? p.logit_off[w.b] : 0;
        }
        const int ntiles = (w.n + kTileKeys - 1) / kTileKeys;
        // --- the loads: thread tid fetches half of row tid / 2 of every tile.  The chain of a key -- its
        // position, its block, its rows -- is spread over the tiles ahead.
        const int lr = tid >> 1, lh = tid & 1;
        const int *list = p.sparse_idx + ((size_t)w.b * p.Hkv + w.g) * p.max_sparse + w.begin;
        const int *tab = p.c.table + (size_t)w.b * p.c.max_blocks;
        auto position = [&](int t) {  // -1: no such key
            const int i = t * kTileKeys + lr;
            if (i >= w.n) return -1;
            if (w.verify) return w.begin + i;
            const int pos = __ldg(list + i);
            if (pos < 0 || pos >= w.L) {
                bad |= PILLAR_FLAG_INDEX;
                return -1;
            }
            return pos;
        };
        auto block = [&](int pos) { return pos >= 0 && pos / kBlk < p.c.max_blocks ? __ldg(tab + pos / kBlk) : -1; };
        auto fetch = [&](int t, int pos, int blk) {
            Stage8<D> &st = stage[t % kStages8];
            const bool ok = blk >= 0 && blk < p.c.num_blocks;
            if (pos >= 0 && !ok) bad |= PILLAR_FLAG_SLOT;
            const size_t unit = ok ? (size_t)blk * p.Hkv + w.g : 0;
            const size_t row = (unit * kBlk + (ok ? pos % kBlk : 0)) * D;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int ch = lh * (D / 32) + i;
                cp16(st.k + k_chunk<D>(lr, ch), p.c.k8 + row + ch * 16, ok);
                cp16(st.v + v_chunk<D>(lr, ch), p.c.v8 + row + ch * 16, ok);
            }
            if (lh == 0) {
                cp4(&st.ks[lr], p.c.k_scale + unit, ok);
                st.pos[lr] = !ok ? kNever : (w.verify ? pos : 0);
            } else {
                cp4(&st.vs[lr], p.c.v_scale + unit, ok);
            }
        };
        int posv[kStages8 + 1], blkv[kStages8];
#pragma unroll
        for (int t = 0; t < kStages8 + 1; ++t) posv[t] = position(t);
#pragma unroll
        for (int t = 0; t < kStages8; ++t) blkv[t] = block(posv[t]);
        Acc<D> a;
        const int rows = w.verify ? p.M : p.G;
        const int mt = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;  // row tiles (as warps share them out)
        const int mtile = warp & (mt - 1), kg = warp / mt;   // this warp's row tile, its share of the keys
        const bool active = mtile * 16 < rows;
#pragma unroll
        for (int t = 0; t < kStages8 - 1; ++t) {
            if (t < ntiles) fetch(t, posv[t], blkv[t]);
            cp_commit();
        }
        int blk_next = blkv[kStages8 - 1], pos_next = posv[kStages8 - 1], pos_after = posv[kStages8];
        load_row<D, 0>(p, w, mtile * 16 + g, rows, c, a);
        load_row<D, 1>(p, w, mtile * 16 + g + 8, rows, c, a);
        a.wsc = 0x1p126f;
        a.vmax = 0.f;
#pragma unroll
        for (int i = 0; i < D / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) a.o[i][e] = 0.f;
        for (int t = 0; t < ntiles; ++t) {
            cp_wait<kStages8 - 2>();
            __syncthreads();  // tile t is in shared memory, and tile t-1's stage is free
            if (t + kStages8 - 1 < ntiles) fetch(t + kStages8 - 1, pos_next, blk_next);
            cp_commit();
            pos_next = pos_after;
            blk_next = block(pos_next);
            pos_after = position(t + kStages8 + 1);
            if (active) {
                const Stage8<D> &st = stage[t % kStages8];
                const int t0 = t * kTileKeys, nk = min(kTileKeys, w.n - t0);
                if (mt == 1) tile_keys<D, 1>(p, w, st, kg * 16, t0, nk, a);
                else if (mt == 2) tile_keys<D, 2>(p, w, st, kg * 32, t0, nk, a);
                else tile_keys<D, 2>(p, w, st, 0, t0, nk, a), tile_keys<D, 2>(p, w, st, 32, t0, nk, a);
            }
        }
        // --- the item's rows
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            a.r[h].l += __shfl_xor_sync(0xffffffffu, a.r[h].l, 1);
            a.r[h].l += __shfl_xor_sync(0xffffffffu, a.r[h].l, 2);
        }
        const float unw = 1.f / a.wsc;
        if (mt == 4) {
            if (active) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const Row8 &r = a.r[h];
                    const int row = mtile * 16 + g + 8 * h;
                    if (row >= rows) continue;
                    const float inv = r.l == 0.f ? 0.f : 1.f / r.l;
                    float v[D / 4];
#pragma unroll
                    for (int i = 0; i < D / 8; ++i) {
                        v[i] = a.o[i][2 * h] * inv * unw;
                        v[D / 8 + i] = a.o[i][2 * h + 1] * inv * unw;
                    }
                    store_row<D>(p, w, row, r.j, r.gi, c * (D / 4), v, D / 4);
                    if (c == 0) store_lse(p, w, row, r.j, r.gi, r.m, r.l);
                }
            }
        } else {  // the warps that shared a row tile's keys: m, l and O through shared memory
            constexpr int LD = D + 4;
            float *so = reinterpret_cast<float *>(smem);           // [4 warps][16][LD]
            float *sm = so + 4 * 16 * LD, *sl = sm + 4 * 16;       // [4 warps][16]
            cp_wait<0>();
            __syncthreads();
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int lrow = g + 8 * h;
                float *dst = so + (warp * 16 + lrow) * LD + c * (D / 4);
#pragma unroll
                for (int i = 0; i < D / 8; ++i) {
                    dst[i] = a.o[i][2 * h];
                    dst[D / 8 + i] = a.o[i][2 * h + 1];
                }
                if (c == 0) sm[warp * 16 + lrow] = a.r[h].m, sl[warp * 16 + lrow] = a.r[h].l;
            }
            __syncthreads();
            const int share = 4 / mt;
            constexpr int C8 = D / 8;
            for (int x = tid; x < rows * C8; x += kThreads8) {
                const int row = x / C8, d = (x - row * C8) * 8;
                const int tile = row >> 4, lrow = row & 15;
                float m = neg_inf(), l = 0.f;
                for (int s = 0; s < share; ++s) m = fmaxf(m, sm[(s * mt + tile) * 16 + lrow]);
                float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
                if (m > neg_inf()) {
                    for (int s = 0; s < share; ++s) {
                        const int at = (s * mt + tile) * 16 + lrow;
                        const float f = ex2_approx((sm[at] - m) * kLog2e);
                        l += f * sl[at];
#pragma unroll
                        for (int i = 0; i < 8; ++i) v[i] += f * so[at * LD + d + i];
                    }
                } else {
                    for (int s = 0; s < share; ++s) l += sl[(s * mt + tile) * 16 + lrow];  // 0, or a NaN
                }
                const float inv = l == 0.f ? 0.f : unw / l;
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] *= inv;
                const int j = w.verify ? row / p.G : 0;
                store_row<D>(p, w, row, j, row - j * p.G, d, v, 8);
                if (d == 0) store_lse(p, w, row, j, row - j * p.G, m, l);
            }
        }
        __syncthreads();  // (an item without keys has had no barrier since s_item was written)
        it = s_item;
    }
    if (bad) atomicOr(&p.hdr->err, bad);
}

template <int D>
cudaError_t launch_t(const Kv8Params &p, int nsm, cudaStream_t st) {
    constexpr int kSmem = kStages8 * (int)sizeof(Stage8<D>);
    static_assert(4 * 16 * (D + 4) * 4 + 2 * 4 * 16 * 4 <= kSmem, "the join fits into the stages");
    static int occupancy[kMaxDevices];
    static unsigned long long configured[kMaxDevices] = {};
    int dev = 0;
    unsigned long long ctx = 0;
    cudaError_t e = current_device_context(&dev, &ctx);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    if (ctx == 0 || __atomic_load_n(&configured[dev], __ATOMIC_ACQUIRE) != ctx) {
        e = cudaFuncSetAttribute(attn_kv8_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        int n = 0;
        e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, attn_kv8_kernel<D>, kThreads8, kSmem);
        if (e != cudaSuccess) return e;
        if (n < 1) return cudaErrorInvalidConfiguration;
        e = current_device_context(&dev, &ctx);  // (the calls above made a context current)
        if (e != cudaSuccess) return e;
        __atomic_store_n(&occupancy[dev], n, __ATOMIC_RELAXED);
        __atomic_store_n(&configured[dev], ctx, __ATOMIC_RELEASE);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(nsm * __atomic_load_n(&occupancy[dev], __ATOMIC_RELAXED));
    cfg.blockDim = dim3(kThreads8);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attn_kv8_kernel<D>, p);
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
    const cudaError_t e = a.D == 128 ? launch_t<128>(p, nsm, st) : launch_t<64>(p, nsm, st);
    return e == cudaSuccess ? launch_merge(a, nsm, st) : e;
}

}  // namespace pillar
