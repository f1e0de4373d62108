// pillar_kv_read.cu -- positions of the quantised caches as bf16 rows.
//
// 4 bits: e2m1(code) * scale, exact in bf16.  8 bits: e4m3(code) * scale, one
// rounding (none under the power-of-two scales that the append writes, short of
// the ends of bf16's range).
//
// One thread has sixteen values (32 bytes of output), two at a time.  What bounds it: memory, mostly the rows written (2 bytes a
// value, after 0.56 or 1 read).  1.3 GB of 4-bit codes and rows take 207 us and 1.5 GB of 8-bit ones 240: 6.2 and 6.3 TB/s, 0.92
// and 0.93 of a plain copy's rate (16-byte accesses: 235 and 291).  (Three CTAs of four pieces a thread: 205 and 239 us; six of two,
// with 32 registers: 246 and 278.)
#include "pillar_kv4.cuh"
#include "pillar_kv4.h"
#include "pillar_rows.cuh"

namespace pillar {

namespace {

constexpr int kResident = 5, kUnroll = 2;  // CTAs of an SM, pieces of a thread in flight

__device__ __forceinline__ float2 f32_of(uint32_t h) {
    float2 v;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(v.x), "=f"(v.y)
        : "r"(h));
    return v;
}

template <int D, int kBits, bool kWide>
__global__ void __launch_bounds__(kRowThreads, kResident) kv_read_kernel(KvReadArgs a, int most) {
    constexpr int PR = D / 16;  // pieces of a row
    const bool value = threadIdx.x >= kRowWorkers / 2;
    uint16_t *const out = value ? a.v_out : a.k_out;
    const long long stride = value ? a.v_stride : a.k_stride;
    const uint8_t *const from = value ? a.v : a.k;
    const void *const scales = value ? a.v_scale : a.k_scale;
    const RowMap m{a.out_off, a.first, a.table, a.flags, a.n, a.B, a.Hkv, a.max_blocks, a.num_blocks, a.max_len, false};
    for_rows(m, most, [&](long long t0, int rows, const int *place) {
        Walk w(threadIdx.x % (kRowWorkers / 2), kRowWorkers / 2, a.Hkv * PR);
        while (w.token < rows) {
            uint4 codes[kUnroll];
            uint32_t scale[kUnroll];
            uint16_t *dst[kUnroll];
#pragma unroll
            for (int i = 0; i < kUnroll; ++i, w.next()) {
                dst[i] = nullptr;
                const int at = w.token < rows ? place[w.token] : -1;
                if (at < 0) continue;
                const int h = w.piece / PR, c = w.piece % PR;
                const size_t row = (size_t)(unsigned)(at + h * PILLAR_KV_BLOCK);
                dst[i] = out + (t0 + w.token) * stride + w.piece * 16;
                if (kBits == 4) {
                    const uint2 y = __ldg(reinterpret_cast<const uint2 *>(from + row * (D / 2)) + c);
                    codes[i].x = y.x, codes[i].y = y.y;
                    scale[i] = __ldg(static_cast<const uint8_t *>(scales) + row * PR + c);
                } else {
                    codes[i] = __ldg(reinterpret_cast<const uint4 *>(from + row * D) + c);
                    scale[i] = __ldg(static_cast<const uint32_t *>(scales) + row / PILLAR_KV_BLOCK);
                }
            }
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                if (!dst[i]) continue;
                uint32_t o[8];
                if (kBits == 4) {
                    const uint32_t s = scale[i] * 0x00800080u;  // (a scale byte in bits 7 to 14 is its f16 value)
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t x[4];
                        f16_of_e2m1(q ? codes[i].y : codes[i].x, x);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 v = f32_of(mul_f16x2(x[e], s));
                            o[4 * q + e] = pack_bf16x2(v.x, v.y);
                        }
                    }
                } else {
                    const float s = __uint_as_float(scale[i]);
                    const uint32_t wd[4] = {codes[i].x, codes[i].y, codes[i].z, codes[i].w};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        uint32_t x;
                        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"((uint16_t)(wd[e >> 1] >> (16 * (e & 1)))));
                        const float2 v = f32_of(x);
                        o[e] = pack_bf16x2(v.x * s, v.y * s);
                    }
                }
                store32<kWide>(dst[i], o);
            }
        }
    });
}

}  // namespace

cudaError_t launch_kv_read(const KvReadArgs &a, int nsm, cudaStream_t st) {
    const int rows = rows_of_turn(a.n, kResident, nsm);
    const unsigned grid = row_ctas(a.n, rows, kResident, nsm);
    const bool wide = rows_wide(a.k_out, a.v_out, a.k_stride, a.v_stride);
    const auto f = a.bits == 4 ? (a.D == 128 ? (wide ? kv_read_kernel<128, 4, true> : kv_read_kernel<128, 4, false>)
                                             : (wide ? kv_read_kernel<64, 4, true> : kv_read_kernel<64, 4, false>))
                               : (a.D == 128 ? (wide ? kv_read_kernel<128, 8, true> : kv_read_kernel<128, 8, false>)
                                             : (wide ? kv_read_kernel<64, 8, true> : kv_read_kernel<64, 8, false>));
    return launch_rows(f, a, rows, grid, st);
}

}  // namespace pillar
