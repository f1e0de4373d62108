// pillar_attn_kv4.cu -- the unified draft/verify attention over the 4-bit cache.
//
// For query row r and key t, with K and V rows e2m1(code) * scale (pillar_kv4.cuh):
//     s[r, t] = scale * (q_r . k_t),   o[r] = sum_t e^(s[r, t] - m) v_t / sum_t e^(s[r, t] - m)
// The planner, its work items, the partial records and the merge of split
// units are those of the bf16 step; only the kernel between them differs.
//
// A warp has a query row of an item, a lane D / 32 of its dimensions, and
// walks over the keys with a running maximum and sum.
#include "pillar_kv4.cuh"

namespace pillar {

namespace {

constexpr int kThreads4 = 256;

struct Kv4Params {
    const uint16_t *q;
    Kv4Cache c;
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

// Dimensions [N lane, N lane + N) of a cache row.
template <int N>
__device__ __forceinline__ void row_values(const uint8_t *codes, const uint8_t *scale, size_t row, int lane, float (&v)[N]) {
    const uint8_t *src = codes + row * (N * 16) + lane * (N / 2);
    const uint32_t w = N == 4 ? *reinterpret_cast<const uint16_t *>(src) : *src;
    uint32_t h[4];
    f16_of_e2m1(w, h);
    const uint32_t s = scale_pair(scale[row * (N * 32 / kGroup4) + lane * N / kGroup4], 0);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const uint32_t x = mul_f16x2(h[i], s);
        asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
            : "=f"(v[2 * i]), "=f"(v[2 * i + 1])
            : "r"(x));
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads4) attn_kv4_kernel(const __grid_constant__ Kv4Params p) {
    constexpr int N = D / 32;
    __shared__ int s_item;
    pdl_wait_prerequisites();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int num_items = *reinterpret_cast<volatile int *>(&p.hdr->num_items);
    int bad = 0;
    for (;;) {
        __syncthreads();
        if (threadIdx.x == 0) s_item = atomicAdd(&p.hdr->item_counter, 1);
        __syncthreads();
        if (s_item >= num_items) break;
        const Item it = p.items[s_item];
        const int b = it.unit / p.Hkv, g = it.unit - b * p.Hkv;
        const ReqInfo req = p.req[b];
        const UnitInfo unit = p.unit[it.unit];
        const bool verify = req.mode == 1;
        const int rows = verify ? p.M : p.G, rec = unit.rec_base + it.split * unit.rec_rows;
        for (int r = warp; r < rows; r += kThreads4 / 32) {
            const int j = verify ? r / p.G : 0, gi = r - j * p.G;
            const size_t orow = (size_t)(req.q_off + j) * p.Hq + (size_t)g * p.G + gi;
            const long long lb = verify && p.logits
                                     ? p.logit_off[b] + ((long long)(g * p.G + gi) * (p.k + 1) + j) * req.len : -1;
            const int lim = verify ? req.len - (p.k + 1) + j : 0x7fffffff;
            float q[N], o[N] = {}, m = neg_inf(), l = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) q[i] = bf16lo(p.q[orow * D + lane * N + i]);
            for (int t = it.begin; t < it.end; ++t) {
                int pos = t;
                if (!verify) pos = p.sparse_idx[((size_t)b * p.Hkv + g) * p.max_sparse + t];
                float s = neg_inf();
                size_t row = 0;
                if (pos < 0 || pos >= req.len) {
                    bad |= PILLAR_FLAG_INDEX;
                } else {
                    const int blk = pos / PILLAR_KV_BLOCK < p.c.max_blocks
                                        ? p.c.table[(size_t)b * p.c.max_blocks + pos / PILLAR_KV_BLOCK] : -1;
                    if (blk < 0 || blk >= p.c.num_blocks) {
                        bad |= PILLAR_FLAG_SLOT;
                    } else if (pos <= lim) {
                        row = ((size_t)blk * p.Hkv + g) * PILLAR_KV_BLOCK + pos % PILLAR_KV_BLOCK;
                        float k[N];
                        row_values<N>(p.c.k4, p.c.k_scale, row, lane, k);
                        s = 0.f;
#pragma unroll
                        for (int i = 0; i < N; ++i) s += q[i] * k[i];
#pragma unroll
                        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
                        s *= p.scale;
                    }
                }
                if (lb >= 0 && lane == 0) p.logits[lb + pos] = s;
                if (s == neg_inf()) continue;
                const float mn = fmaxf(m, s), f = m == neg_inf() ? 0.f : expf(m - mn), e = expf(s - mn);
                float v[N];
                row_values<N>(p.c.v4, p.c.v_scale, row, lane, v);
                l = l * f + e;
#pragma unroll
                for (int i = 0; i < N; ++i) o[i] = o[i] * f + e * v[i];
                m = mn;
            }
            const float inv = l == 0.f ? 0.f : 1.f / l, z = l > 0.f ? m + logf(l) : (l == 0.f ? neg_inf() : l);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                if (unit.nsplit > 1) p.part_o[((size_t)rec + r) * D + lane * N + i] = o[i] * inv;
                else p.out[orow * D + lane * N + i] = (uint16_t)pack_bf16x2(o[i] * inv, 0.f);
            }
            if (lane == 0) {
                if (unit.nsplit > 1) p.part_lse[(size_t)rec + r] = z;
                else if (verify) p.lse[((size_t)req.vidx * p.Hq + (size_t)g * p.G + gi) * (p.k + 1) + j] = z;
            }
        }
    }
    if (bad) atomicOr(&p.hdr->err, bad);
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
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(4 * nsm);
    cfg.blockDim = dim3(kThreads4);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = a.D == 128 ? cudaLaunchKernelEx(&cfg, attn_kv4_kernel<128>, p) : cudaLaunchKernelEx(&cfg, attn_kv4_kernel<64>, p);
    return e == cudaSuccess ? launch_merge(a, nsm, st) : e;
}

}  // namespace pillar
