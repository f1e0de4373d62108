// pillar_kv4.cu -- appending new K/V rows to the 4-bit cache.
//
// For 16 neighbouring values x of a row, with a = max |x|:
//     s    = the smallest scale with a <= 6 s, from 2^-17 to 10240
//     code = the e2m1 value nearest to x / s (ties to even, saturating at 6)
// A row's scales are its own, so an append touches no earlier row, whatever
// the values are.
//
// One thread has eight values (16 bytes of the row), two neighbours share a
// scale.  What bounds it: memory, 2 bytes read and 0.56 written per value.
#include "pillar_kv4.cuh"
#include "pillar_kv4.h"
#include "pillar_rows.cuh"

namespace pillar {

namespace {

constexpr int kThreads4 = 256;
constexpr int kMaxCtaRows4 = 16;

// The scale byte of a largest magnitude a (finite, >= 0).  a / 6 by the reciprocal rounded down: at most a relative 2^-23
// below, so that a = 6 s comes to s or just below it, and, as a has eight significant bits and s four, any a > 6 s stays above.
__device__ __forceinline__ uint32_t scale_byte(float a) {
    const float u = a * 0x1.555554p-3f;
    const uint32_t normal = ((__float_as_uint(u) + 0xfffffu) >> 20) - (112u << 3);  // four significant bits, rounded up
    const uint32_t small = (uint32_t)__float2int_ru(u * 0x1p17f);                   // steps of 2^-17 below 2^-14
    return min(max(u >= 0x1p-14f ? normal : small, 1u), (uint32_t)kTopScale);
}
__device__ __forceinline__ float scale_value(uint32_t byte) {
    return byte >= 8 ? __uint_as_float((byte + (112u << 3)) << 20) : (float)byte * 0x1p-17f;
}

// Eight values x / s as codes.  x has eight significant bits and s four, so that x / s is a tie between two codes or at
// least 2^-10 away from one; the product with 1 / s, within 2^-20 of the quotient, is rounded to a multiple of 2^-14 first
// (the addition of 768), which makes ties exact.
__device__ __forceinline__ uint32_t codes_of(const uint4 &x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t out;
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __fadd_rn(__fmaf_rn(bf16lo(w[i]), inv, 768.f), -768.f);
        v[2 * i + 1] = __fadd_rn(__fmaf_rn(bf16hi(w[i]), inv, 768.f), -768.f);
    }
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(out)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return out;
}

// Rare: a NaN becomes 0; infinities stay (they saturate) and are left out of the largest magnitude.
__device__ __noinline__ uint32_t clean(uint4 &x) {
    uint32_t *w = &x.x, m = 0;
    for (int i = 0; i < 4; ++i) {
        uint32_t lo = w[i] & 0xffffu, hi = w[i] >> 16;
        if ((lo & 0x7fffu) > 0x7f80u) lo = 0;
        if ((hi & 0x7fffu) > 0x7f80u) hi = 0;
        w[i] = lo | hi << 16;
        lo &= 0x7fffu, hi &= 0x7fffu;
        m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
    }
    return m;
}

template <int D>
__global__ void __launch_bounds__(kThreads4) kv4_append_kernel(const Kv4AppendArgs a, int rows) {
    __shared__ long long s_place[kMapRows];
    const int t0 = blockIdx.x * rows;
    if (threadIdx.x < 32) {
        const RowMap m{a.new_off, a.req_len, a.table, a.flags, a.n, a.B, a.max_blocks, a.num_blocks, a.max_len, true};
        find_rows(m, t0, rows, s_place);
    }
    __syncthreads();
    constexpr int PR = D / 8;  // pieces of a row
    const int half = a.Hkv * PR;
    int bad = 0;
    // (all lanes of a warp stay in the loop together: neighbours exchange their largest magnitudes)
    Walk w(kThreads4, 2 * half);
    const int total = rows * 2 * half;
    for (int base = 0; base < total; base += kThreads4, w.next()) {
        const bool in = base + (int)threadIdx.x < total;
        const long long place = in ? s_place[w.token] : -1;
        const bool value = w.piece >= half;
        const int p = value ? w.piece - half : w.piece;
        uint4 x = make_uint4(0, 0, 0, 0);
        if (place >= 0) {
            const uint16_t *src = (value ? a.v_new : a.k_new) + (long long)(t0 + w.token) * (value ? a.v_stride : a.k_stride) +
                                  (long long)p * 8;
            x = __ldg(reinterpret_cast<const uint4 *>(src));
        }
        const uint32_t m2 = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
        uint32_t mx = max(m2 & 0xffffu, m2 >> 16);
        if (mx >= 0x7f80u) {
            mx = clean(x);
            bad = PILLAR_FLAG_VALUE;
        }
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        if (place < 0) continue;
        if (mx > 0x4770u) bad = PILLAR_FLAG_VALUE;  // 61440: the largest value the cache holds
        const uint32_t byte = scale_byte(__uint_as_float(mx << 16));
        const uint32_t codes = codes_of(x, 1.f / scale_value(byte));
        const int h = p / PR, c = p - h * PR;
        const size_t row = ((size_t)(place / PILLAR_KV_BLOCK) * a.Hkv + h) * PILLAR_KV_BLOCK + place % PILLAR_KV_BLOCK;
        *reinterpret_cast<uint32_t *>((value ? a.v4 : a.k4) + row * (D / 2) + c * 4) = codes;
        if (!(c & 1)) ((value ? a.v_scale : a.k_scale) + row * (D / kGroup4))[c >> 1] = (uint8_t)byte;
    }
    if (bad && a.flags) atomicOr(a.flags, bad);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs &a, int nsm, cudaStream_t st) {
    const int rows = a.n <= 16 * nsm ? 1 : kMaxCtaRows4;
    const unsigned grid = (unsigned)((a.n + (long long)rows - 1) / rows);
    if (a.D == 128) kv4_append_kernel<128><<<grid, kThreads4, 0, st>>>(a, rows);
    else kv4_append_kernel<64><<<grid, kThreads4, 0, st>>>(a, rows);
    return cudaGetLastError();
}

}  // namespace pillar
