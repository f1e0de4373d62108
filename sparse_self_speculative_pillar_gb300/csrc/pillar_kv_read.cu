// pillar_kv_read.cu -- positions of the quantised caches as bf16 rows.
//
// 4 bits: e2m1(code) * scale, exact in bf16.  8 bits: e4m3(code) * scale, one
// rounding (none under the power-of-two scales that the append writes, short of
// the ends of bf16's range).
//
// One thread has eight values (16 bytes of output).  What bounds it: memory,
// mostly the rows written (2 bytes a value, after 0.56 or 1 read).
#include "pillar_kv4.cuh"
#include "pillar_kv4.h"
#include "pillar_rows.cuh"

namespace pillar {

namespace {

constexpr int kThreadsR = 256;
constexpr int kMaxCtaRowsR = 16;

__device__ __forceinline__ float2 f32_of(uint32_t h) {
    float2 v;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
        : "=f"(v.x), "=f"(v.y)
        : "r"(h));
    return v;
}

template <int D, int kBits>
__global__ void __launch_bounds__(kThreadsR) kv_read_kernel(const KvReadArgs a, int rows) {
    __shared__ long long s_place[kMapRows];
    const int t0 = blockIdx.x * rows;
    if (threadIdx.x < 32) {
        const RowMap m{a.out_off, a.first, a.table, a.flags, a.n, a.B, a.max_blocks, a.num_blocks, a.max_len, false};
        find_rows(m, t0, rows, s_place);
    }
    __syncthreads();
    constexpr int PR = D / 8;
    const int half = a.Hkv * PR;
    for (Walk w(kThreadsR, 2 * half); w.token < rows; w.next()) {
        const long long place = s_place[w.token];
        if (place < 0) continue;
        const bool value = w.piece >= half;
        const int p = value ? w.piece - half : w.piece, h = p / PR, c = p - h * PR;
        const size_t unit = (size_t)(place / PILLAR_KV_BLOCK) * a.Hkv + h, row = unit * PILLAR_KV_BLOCK + place % PILLAR_KV_BLOCK;
        uint32_t o[4];
        if (kBits == 4) {
            const uint32_t codes = __ldg(reinterpret_cast<const uint32_t *>((value ? a.v : a.k) + row * (D / 2) + c * 4));
            const uint32_t byte = __ldg(static_cast<const uint8_t *>(value ? a.v_scale : a.k_scale) + row * (D / kGroup4) + (c >> 1));
            const uint32_t s = scale_pair(byte, 0);
            uint32_t x[4];
            f16_of_e2m1(codes, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 v = f32_of(mul_f16x2(x[i], s));
                o[i] = pack_bf16x2(v.x, v.y);
            }
        } else {
            const uint2 codes = __ldg(reinterpret_cast<const uint2 *>((value ? a.v : a.k) + row * D + c * 8));
            const float s = __ldg(static_cast<const float *>(value ? a.v_scale : a.k_scale) + unit);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t two = (i < 2 ? codes.x : codes.y) >> (16 * (i & 1));
                uint32_t x;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(x) : "h"((uint16_t)two));
                const float2 v = f32_of(x);
                o[i] = pack_bf16x2(v.x * s, v.y * s);
            }
        }
        uint16_t *dst = (value ? a.v_out : a.k_out) + (long long)(t0 + w.token) * (value ? a.v_stride : a.k_stride) + (long long)p * 8;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

}  // namespace

cudaError_t launch_kv_read(const KvReadArgs &a, int nsm, cudaStream_t st) {
    const int rows = a.n <= 16 * nsm ? 1 : kMaxCtaRowsR;
    const unsigned grid = (unsigned)((a.n + (long long)rows - 1) / rows);
    if (a.bits == 4) {
        if (a.D == 128) kv_read_kernel<128, 4><<<grid, kThreadsR, 0, st>>>(a, rows);
        else kv_read_kernel<64, 4><<<grid, kThreadsR, 0, st>>>(a, rows);
    } else {
        if (a.D == 128) kv_read_kernel<128, 8><<<grid, kThreadsR, 0, st>>>(a, rows);
        else kv_read_kernel<64, 8><<<grid, kThreadsR, 0, st>>>(a, rows);
    }
    return cudaGetLastError();
}

}  // namespace pillar
