// pillar_kv4.cu -- appending new K/V rows to the 4-bit cache.
//
// For 16 neighbouring values x of a row, with a = max |x|:
//     s    = the smallest scale with a <= 6 s, from 2^-17 to 10240
//     code = the e2m1 value nearest to x / s (ties to even, saturating at 6)
// A row's scales are its own, so an append touches no earlier row, whatever
// the values are.
//
// One thread has the sixteen values of a scale, two at a time.  What bounds it: memory, 2 bytes read and 0.56 written per
// value.  Of 14 warps per issue 5.7 wait for loads and 2.8 at a turn's end, the ALU is at 0.49.  26 K rows of K and V (8 heads,
// D = 128) stored and read back take 53.5 us, 4.6 TB/s; with turns dealt out one by one instead of a range to a CTA, and launches that wait for the
// kernel before, 59.5; with 8-byte pieces of four values a thread 80.  (Three CTAs of four pieces a thread: 52 to 54 us; two of
// eight: 63; five of two, with 40 registers: 59.)
#include "pillar_kv4.cuh"
#include "pillar_kv4.h"
#include "pillar_rows.cuh"

namespace pillar {

namespace {

constexpr int kResident = 4, kUnroll = 2;  // CTAs of an SM, pieces of a thread in flight

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(d)
        : "l"(*reinterpret_cast<unsigned long long *>(&a)), "l"(*reinterpret_cast<unsigned long long *>(&b)),
          "l"(*reinterpret_cast<unsigned long long *>(&c)));
    return *reinterpret_cast<float2 *>(&d);
}

// The scale byte of a largest magnitude a (finite, >= 0), and the scale's inverse.  a / 6 by the reciprocal rounded down: at most
// a relative 2^-23 below, so that a = 6 s comes to s or just below it, and, as a has eight significant bits and s four, any
// a > 6 s stays above.
__device__ __forceinline__ uint32_t scale_byte(float a, float *inv) {
    const float u = a * 0x1.555554p-3f;
    const uint32_t up = __float_as_uint(u) + 0xfffffu;            // four significant bits, rounded up
    const uint32_t small = (uint32_t)__float2int_ru(u * 0x1p17f);  // steps of 2^-17 below 2^-14
    const uint32_t byte = min(max(u >= 0x1p-14f ? (up >> 20) - (112u << 3) : small, 1u), (uint32_t)kTopScale);
    const float s = byte >= 8 ? __uint_as_float((byte + (112u << 3)) << 20) : (float)byte * 0x1p-17f;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(*inv) : "f"(s));  // (within 2^-23)
    return byte;
}

// Eight values x / s as codes.  x has eight significant bits and s four, so that x / s is a tie between two codes or at
// least 2^-10 away from one; the product with 1 / s, within 2^-20 of the quotient, is rounded to a multiple of 2^-14 first
// (the addition of 768), which makes ties exact.
__device__ __forceinline__ uint32_t codes_of(const uint32_t *w, float inv) {
    const float2 i2 = make_float2(inv, inv), big = make_float2(768.f, 768.f), less = make_float2(-768.f, -768.f);
    uint32_t out;
    float2 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = fadd2(fma2(make_float2(bf16lo(w[i]), bf16hi(w[i])), i2, big), less);
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(out)
        : "f"(v[0].x), "f"(v[0].y), "f"(v[1].x), "f"(v[1].y), "f"(v[2].x), "f"(v[2].y), "f"(v[3].x), "f"(v[3].y));
    return out;
}

// Rare: NaN becomes 0; infinities stay (they saturate) and are left out of the largest magnitude, which is returned.
__device__ __forceinline__ uint32_t clean(Half16 &x) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t lo = x.w[i] & 0xffffu, hi = x.w[i] >> 16;
        if ((lo & 0x7fffu) > 0x7f80u) lo = 0;
        if ((hi & 0x7fffu) > 0x7f80u) hi = 0;
        x.w[i] = lo | hi << 16;
        lo &= 0x7fffu, hi &= 0x7fffu;
        m = max(m, max(lo < 0x7f80u ? lo : 0u, hi < 0x7f80u ? hi : 0u));
    }
    return m;
}

template <int D, bool kWide>
__global__ void __launch_bounds__(kRowThreads, kResident) kv4_append_kernel(Kv4AppendArgs a, int most) {
    constexpr int PR = D / kGroup4;  // pieces of a row
    int bad = 0;
    const bool value = threadIdx.x >= kRowWorkers / 2;
    const uint16_t *const from = value ? a.v_new : a.k_new;
    const long long stride = value ? a.v_stride : a.k_stride;
    uint8_t *const codes = value ? a.v4 : a.k4, *const scales = value ? a.v_scale : a.k_scale;
    const RowMap m{a.new_off, a.req_len, a.table, a.flags, a.n, a.B, a.Hkv, a.max_blocks, a.num_blocks, a.max_len, true};
    for_rows(m, most, [&](long long t0, int rows, const int *place) {
        Walk w(threadIdx.x % (kRowWorkers / 2), kRowWorkers / 2, a.Hkv * PR);
        while (w.token < rows) {
            Half16 x[kUnroll];
            int at[kUnroll], piece[kUnroll];  // row of the pools for head 0, or -1
#pragma unroll
            for (int i = 0; i < kUnroll; ++i, w.next()) {
                at[i] = w.token < rows ? place[w.token] : -1;
                piece[i] = w.piece;
                if (at[i] >= 0) x[i] = load32<kWide>(from + (t0 + w.token) * stride + w.piece * kGroup4);
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                if (at[i] < 0) continue;
                uint32_t m2 = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) m2 = __vmaxu2(m2, x[i].w[e] & 0x7fff7fffu);
                uint32_t mx = max(m2 & 0xffffu, m2 >> 16);
                if (mx > 0x4770u) {  // past 61440, the largest value the cache holds
                    bad = PILLAR_FLAG_VALUE;
                    if (mx >= 0x7f80u) mx = clean(x[i]);
                }
                float inv;
                const uint32_t byte = scale_byte(__uint_as_float(mx << 16), &inv);
                const int h = piece[i] / PR, c = piece[i] % PR;
                const size_t row = (size_t)(unsigned)(at[i] + h * PILLAR_KV_BLOCK);
                *reinterpret_cast<uint2 *>(codes + row * (D / 2) + c * 8) = make_uint2(codes_of(x[i].w, inv), codes_of(x[i].w + 4, inv));
                scales[row * PR + c] = (uint8_t)byte;
            }
        }
    });
    if (bad && a.flags) atomicOr(a.flags, bad);
}

}  // namespace

cudaError_t launch_kv4_append(const Kv4AppendArgs &a, int nsm, cudaStream_t st) {
    const int rows = rows_of_turn(a.n, kResident, nsm);
    const unsigned grid = row_ctas(a.n, rows, kResident, nsm);
    const bool wide = rows_wide(a.k_new, a.v_new, a.k_stride, a.v_stride);
    const auto f = a.D == 128 ? (wide ? kv4_append_kernel<128, true> : kv4_append_kernel<128, false>)
                              : (wide ? kv4_append_kernel<64, true> : kv4_append_kernel<64, false>);
    return launch_rows(f, a, rows, grid, st);
}

}  // namespace pillar
