// pillar_kv8.cu -- appending new K/V rows to the 8-bit cache.
//
// The cache holds e4m3 codes [num_blocks, Hkv, 16, D] and one fp32 scale per
// (block, KV head), for K and for V: value = code * scale.  For the new rows x
// of one (block, head), with a = max |x|:
//     e      = the smallest integer >= -126 with a <= 448 * 2^e
//     scale' = 2^e                    when the block's first row is among them
//            = max(scale, 2^e)        when it holds earlier rows
//     code   = rne_e4m3(x / scale'),  and where the scale grew, the block's other rows:
//              rne_e4m3(code * scale / scale')
// The scale is a power of two: e4m3 is a floating-point format, so a tighter
// scale would gain at most one of its eighteen binades and no precision, while
// with a power of two the division is exact, each value is rounded once, and
// rounding other rows again changes only values that leave the normal range.
//
// One warp per (block with new rows, head, K or V): the block's new rows are
// at most 16 x 256 bytes, held in registers as one load of 16 bytes per lane
// and row group, so they are read once, reduced to their maximum and written
// as codes.  A block is found from the first of its new rows: a CTA takes
// `rows` consecutive packed rows and collects those that start a block or a
// request's new tokens.  With few tokens (a decode step) a CTA takes one row,
// so that all blocks are in flight together; with many (a prompt) sixteen, so
// that the request search is shared.  A prefill batch (32 prompts of 100 to 4000
// tokens, 8 heads of 128 for K and for V: 2 bytes read and 1 written per
// element) takes 32.7 us, 4.96 TB/s or 0.73 of a copy's rate.  No unit is full (ALU
// 0.38, issue 0.49, HBM 0.55 of the peak rates in a cold launch): of 13.9 warps per issue 5.5
// wait for loads and 2.7 for the first warp, whose chain of offsets, lengths and
// table opens every CTA, and a CTA has two blocks' work a warp before it ends.  A
// decode step (128 requests) takes 10 us: launch and the latency of the dependent
// loads (offsets, table, rows).
#include "pillar_device.cuh"
#include "pillar_kv8.h"

namespace pillar {

namespace {

constexpr int kThreadsPerCta = 256;
constexpr int kWarps = kThreadsPerCta / 32;
constexpr int kMaxCtaRows = 16;
constexpr int kBlock = PILLAR_KV_BLOCK;

// Two fp32 values as e4m3 codes (round to nearest even, saturating at 448).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes as fp32 values.
__device__ __forceinline__ float2 from_e4m3x2(uint32_t codes) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
    float2 v;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(v.x), "=f"(v.y)
        : "r"(h));
    return v;
}

// e of the scale 2^e for a largest magnitude given as bf16 bits (finite):
// with a = (1 + M/128) 2^(E-127), a <= 1.75 * 2^(8+e) <=> e >= E - 135, one
// more when 1 + M/128 > 1.75.
__device__ __forceinline__ int scale_exponent(uint32_t bits) {
    const int E = (int)(bits >> 7), M = (int)(bits & 127);
    return max(E - 135 + (M > 96 ? 1 : 0), -126);
}
__device__ __forceinline__ float pow2(int e) { return __int_as_float((e + 127) << 23); }

// The larger magnitudes of two pairs of bf16 values; a NaN stays one.
__device__ __forceinline__ uint32_t max_abs2(uint32_t m, uint32_t x) {
    uint32_t d;
    asm("{\n\t.reg .b32 t;\n\tabs.bf16x2 t, %2;\n\tmax.NaN.bf16x2 %0, %1, t;\n\t}" : "=r"(d) : "r"(m), "r"(x));
    return d;
}
// The low bf16 value of a pair, by a multiplication: the shifts and masks of this kernel keep the ALU busy.
__device__ __forceinline__ float low_of(uint32_t w) { return __uint_as_float(w * 65536u); }

struct Owner {
    int token;  // the first of the block's new rows
    int block;
    int row;    // its row of the block
    int rows;   // new rows in the block
};

// NaN becomes 0; an infinity stays (it saturates).
__device__ __forceinline__ float clean(float x) { return x == x ? x : 0.f; }

template <int D>
__device__ void append_block(const Kv8AppendArgs &a, const Owner &o, int h, bool value) {
    constexpr int RL = D / 8;                // lanes of a row (16 bytes each)
    constexpr int RW = 32 / RL;              // rows of a warp load
    constexpr int NL = kBlock / RW;          // loads of a whole block
    const int lane = threadIdx.x & 31, c = lane % RL, rl = lane / RL;
    const uint16_t *src = (value ? a.v_new : a.k_new) + (long long)o.token * (value ? a.v_stride : a.k_stride) +
                          (long long)h * D + c * 8;
    const long long stride = value ? a.v_stride : a.k_stride;
    const size_t unit = (size_t)o.block * a.Hkv + h;
    uint8_t *dst = (value ? a.v8 : a.k8) + unit * (kBlock * D);
    float *scale = (value ? a.v_scale : a.k_scale) + unit;
    const float before = o.row > 0 ? *scale : 0.f;
    uint4 x[NL];
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        const int r = i * RW + rl;
        x[i] = r < o.rows ? __ldg(reinterpret_cast<const uint4 *>(src + r * stride)) : make_uint4(0, 0, 0, 0);
    }
    // the largest magnitude, then as bits: positive bf16 values order as integers, NaN last
    uint32_t mx = 0;
#pragma unroll
    for (int i = 0; i < NL; ++i) {
        mx = max_abs2(max_abs2(max_abs2(max_abs2(mx, x[i].x), x[i].y), x[i].z), x[i].w);
    }
    uint32_t amax = __reduce_max_sync(0xffffffffu, max(mx & 0xffffu, mx >> 16));
    bool odd = false;
    if (amax >= 0x7f80u) {  // infinities or NaN: the largest finite magnitude decides the scale
        odd = true;
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const uint32_t lo = w[q] & 0x7fffu, hi = (w[q] >> 16) & 0x7fffu;
                m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
            }
        }
        amax = __reduce_max_sync(0xffffffffu, m);
    }
    float s = pow2(scale_exponent(amax));
    if (o.row > 0) {
        const bool good = before >= 0.f && before < __int_as_float(0x7f800000);
        if (!good && lane == 0 && a.flags) atomicOr(a.flags, PILLAR_FLAG_VALUE);
        const float old = good ? before : 0.f;
        if (old >= s) {
            s = old;
        } else {  // the block's other rows under the larger scale
            const float ratio = old / s;
            for (int i = lane * 16; i < kBlock * D; i += 32 * 16) {
                const int r = i / D;
                if (r >= o.row && r < o.row + o.rows) continue;
                uint4 w = *reinterpret_cast<const uint4 *>(dst + i);
                uint32_t *u = reinterpret_cast<uint32_t *>(&w);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const float2 lo = from_e4m3x2(u[q] & 0xffffu), hi = from_e4m3x2(u[q] >> 16);
                    u[q] = e4m3x2(lo.x * ratio, lo.y * ratio) | e4m3x2(hi.x * ratio, hi.y * ratio) << 16;
                }
                *reinterpret_cast<uint4 *>(dst + i) = w;
            }
        }
    }
    // multiplying by 1/s is exact for the powers of two that this kernel writes; a scale that came
    // from elsewhere divides
    uint8_t *out = dst + (size_t)(o.row + rl) * D + c * 8;
    if (!odd && (__float_as_uint(s) & 0x7fffffu) == 0) {
        const float inv = 1.f / s;
#pragma unroll
        for (int i = 0; i < NL; ++i) {
            if (i * RW + rl >= o.rows) continue;
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
            uint32_t c2[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) c2[q] = e4m3x2(low_of(w[q]) * inv, bf16hi(w[q]) * inv);
            *reinterpret_cast<uint2 *>(out + i * RW * D) = make_uint2(c2[0] | c2[1] << 16, c2[2] | c2[3] << 16);
        }
    } else {  // (rare: not unrolled, the rows read again)
#pragma unroll 1
        for (int r = rl; r < o.rows; r += RW) {
            const uint4 y = __ldg(reinterpret_cast<const uint4 *>(src + r * stride));
            const uint32_t w[4] = {y.x, y.y, y.z, y.w};
            uint32_t c2[4];
#pragma unroll
            for (int q = 0; q < 4; ++q)
                c2[q] = e4m3x2(__fdiv_rn(clean(low_of(w[q])), s), __fdiv_rn(clean(bf16hi(w[q])), s));
            *reinterpret_cast<uint2 *>(out + (r - rl) * D) = make_uint2(c2[0] | c2[1] << 16, c2[2] | c2[3] << 16);
        }
    }
    if (lane == 0) {
        if (o.row == 0 || s != before) *scale = s;
        if (odd && a.flags) atomicOr(a.flags, PILLAR_FLAG_VALUE);
    }
}

template <int D>
__global__ void __launch_bounds__(kThreadsPerCta, 4) kv8_append_kernel(const Kv8AppendArgs a, int rows) {
    __shared__ Owner s_own[kMaxCtaRows];
    __shared__ int s_n;
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x;
        const int t0 = blockIdx.x * rows, t = t0 + lane;
        const int all = min(a.n, __ldg(a.new_off + a.B));
        // the request of row t0: 32 offsets a round
        int lo = 0;
        for (int n = a.B; n > 1;) {  // the last offset at or below t0 is one of n from lo on
            const int step = (n + 31) / 32, i = lo + lane * step;
            const unsigned le = __ballot_sync(0xffffffffu, lane * step < n && __ldg(a.new_off + i) <= t0);
            const int k = max(31 - __clz(le), 0);
            n = min(step, n - k * step);
            lo += k * step;
        }
        // the others' by the offsets that follow it (more than 32 requests begin within 16 rows only when some are empty)
        const int behind = lo + 1 + lane <= a.B ? __ldg(a.new_off + lo + 1 + lane) : 0x7fffffff;
        int b = lo;
        for (int i = 0; i < rows; ++i) {
            const int at = __popc(__ballot_sync(0xffffffffu, behind <= t0 + i));
            if (lane == i) b = lo + at;
        }
        if (lane < rows)
            for (b = min(b, a.B - 1); b + 1 < a.B && __ldg(a.new_off + b + 1) <= t;) ++b;
        bool own = false;
        Owner o = {};
        int bad = 0;
        if (lane < rows && t < all) {
            const int first = __ldg(a.new_off + b), end = __ldg(a.new_off + b + 1), len = __ldg(a.req_len + b);
            const long long pos = (long long)len - end + t;
            // (len - (end - first) would pass 31 bits for the lowest lengths)
            if (first < 0 || t < first || t >= end || end > a.n || len > a.max_len || len < end - first ||
                pos / kBlock >= a.max_blocks) {
                bad = PILLAR_FLAG_REQUEST;
            } else if (pos % kBlock == 0 || t == first) {
                o.token = t;
                o.row = (int)(pos % kBlock);
                o.rows = min(kBlock - o.row, end - t);
                o.block = a.table[(size_t)b * a.max_blocks + pos / kBlock];
                if (o.block < 0 || o.block >= a.num_blocks) bad = PILLAR_FLAG_SLOT;
                else own = true;
            }
        }
        if (bad && a.flags) atomicOr(a.flags, bad);
        const unsigned owners = __ballot_sync(0xffffffffu, own);
        if (own) s_own[__popc(owners & ((1u << lane) - 1))] = o;
        if (lane == 0) s_n = __popc(owners);
    }
    __syncthreads();
    const int work = s_n * a.Hkv * 2;
    for (int w = threadIdx.x >> 5; w < work; w += kWarps) {
        const int h2 = w % (a.Hkv * 2);
        append_block<D>(a, s_own[w / (a.Hkv * 2)], h2 >> 1, h2 & 1);
    }
}

}  // namespace

cudaError_t launch_kv8_append(const Kv8AppendArgs &a, int nsm, cudaStream_t st) {
    // one row per CTA while that gives every SM at most sixteen CTAs, sixteen beyond
    const int rows = a.n <= 16 * nsm ? 1 : kMaxCtaRows;
    const unsigned grid = (unsigned)((a.n + (long long)rows - 1) / rows);
    if (a.D == 128) kv8_append_kernel<128><<<grid, kThreadsPerCta, 0, st>>>(a, rows);
    else kv8_append_kernel<64><<<grid, kThreadsPerCta, 0, st>>>(a, rows);
    return cudaGetLastError();
}

}  // namespace pillar
