// pillar_prompt.cu -- causal attention over whole prompts, packed one after
// another, with grouped heads.
//
//   out[i, h] = sum_{j <= i} softmax_j(scale q_ih . k_j,h/G) v_j,h/G   (j in i's sequence)
//   lse[i, h] = log sum_{j <= i} e^(scale q_ih . k_j,h/G)
//
// A planner lists the sequences' 256-row tiles, longest first.  The attention
// kernel: one warp per (row, head), a running maximum and sum over the keys.
#include "pillar_device.cuh"
#include "pillar_prompt.h"

namespace pillar {

namespace {

constexpr int kPlanThreadsP = 1024;
constexpr int kLevels = 1024;  // bins of the longest-first order

// Lists the tiles, those with the most keys first.
__global__ void __launch_bounds__(kPlanThreadsP) prompt_plan(const int *seq_off, int B, int n, int max_len, int room, PromptHeader *hdr,
                                                             PromptTile *tiles) {
    __shared__ int s_bin[kLevels];
    __shared__ int s_warp[32];
    __shared__ int s_bad;
    pdl_wait_prerequisites();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
    s_bin[tid] = 0;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    // bin of tile i of a sequence: larger i first
    const int most = (max_len + kPromptRows - 1) / kPromptRows;
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
        return (hi - lo + kPromptRows - 1) / kPromptRows;
    };
    int first = 0, len = 0;
    for (int b = wid; b < B; b += 32) {
        const int nt = tiles_of(b, &first, &len);
        for (int i = lane; i < nt; i += 32) atomicAdd(&s_bin[level(i)], 1);
    }
    __syncthreads();
    const int own = s_bin[tid];
    int x = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_warp[wid] = x;
    __syncthreads();
    int before = 0;
    for (int i = 0; i < wid; ++i) before += s_warp[i];
    s_bin[tid] = before + x - own;
    __syncthreads();
    for (int b = wid; b < B; b += 32) {
        const int nt = tiles_of(b, &first, &len);
        for (int i = lane; i < nt; i += 32) {
            const int at = atomicAdd(&s_bin[level(i)], 1);
            if (at < room) tiles[at] = PromptTile{first, len, i, 0};
            else s_bad = PILLAR_FLAG_REQUEST;  // (overlapping sequences list more than there is room for)
        }
    }
    __syncthreads();
    if (tid == 0) {
        int total = 0;
        for (int i = 0; i < 32; ++i) total += s_warp[i];
        hdr->num_tiles = min(total, room);
        hdr->err = s_bad;
    }
}

template <int D>
__global__ void __launch_bounds__(256) prompt_kernel(const PromptArgs a, const PromptHeader *hdr, const PromptTile *tiles) {
    pdl_wait_prerequisites();
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31, G = a.Hq / a.Hkv;
    const long long warps = (long long)gridDim.x * 8;
    const long long total = (long long)hdr->num_tiles * kPromptRows * a.Hq;
    for (long long w = (long long)blockIdx.x * 8 + (threadIdx.x >> 5); w < total; w += warps) {
        const int h = (int)(w % a.Hq);
        const long long x = w / a.Hq;
        const PromptTile t = tiles[x / kPromptRows];
        const int i = t.tile * kPromptRows + (int)(x % kPromptRows);
        if (i >= t.len) continue;
        auto at = [&](const uint16_t *p, long long stride, long long row, int head, int e) {
            return __uint_as_float((uint32_t)__ldg(p + row * stride + (long long)head * D + lane * E + e) << 16);
        };
        float q[E], o[E] = {};
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = at(a.q, a.q_stride, (long long)t.row0 + i, h, e);
        float m = neg_inf(), l = 0.f;
        for (int j = 0; j <= i; ++j) {
            float s = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) s = fmaf(q[e], at(a.k, a.k_stride, (long long)t.row0 + j, h / G, e), s);
#pragma unroll
            for (int d = 16; d >= 1; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
            s *= a.scale;
            const float mn = fmaxf(m, s), f = m == neg_inf() ? 0.f : expf(m - mn), p = expf(s - (mn == neg_inf() ? 0.f : mn));
            l = l * f + p;
#pragma unroll
            for (int e = 0; e < E; ++e) o[e] = o[e] * f + p * at(a.v, a.v_stride, (long long)t.row0 + j, h / G, e);
            m = mn;
        }
        const long long row = ((long long)t.row0 + i) * a.Hq + h;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const __nv_bfloat16 b = __float2bfloat16_rn(o[e] * inv);
            a.out[row * D + lane * E + e] = *reinterpret_cast<const uint16_t *>(&b);
        }
        if (a.lse && lane == 0) a.lse[row] = l > 0.f ? m + logf(l) : (l == 0.f ? neg_inf() : l);
    }
}

}  // namespace

cudaError_t launch_prompt(const PromptArgs &a, int nsm, cudaStream_t st) {
    PromptHeader *hdr = reinterpret_cast<PromptHeader *>(a.ws);
    PromptTile *tiles = reinterpret_cast<PromptTile *>(a.ws + sizeof(PromptHeader));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kPlanThreadsP);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, prompt_plan, a.seq_off, a.B, a.n, a.max_len,
                                       (int)prompt_max_tiles(a.B, a.n), hdr, tiles);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3(nsm * 8);
    cfg.blockDim = dim3(256);
    return a.D == 128 ? cudaLaunchKernelEx(&cfg, prompt_kernel<128>, a, (const PromptHeader *)hdr, (const PromptTile *)tiles)
                      : cudaLaunchKernelEx(&cfg, prompt_kernel<64>, a, (const PromptHeader *)hdr, (const PromptTile *)tiles);
}

}  // namespace pillar
