// pillar_attn_kv4.cuh -- what the two kernels of the 4-bit attention share: items of few query rows
// (pillar_attn_kv4_few.cu) and the others (pillar_attn_kv4.cu).
#pragma once

#include "pillar_kv4.cuh"

namespace pillar {

// Verify items of at most so many rows, without a dump of logits and with one, go to warps of mma.sync; the others to tcgen05,
// whose work for a key is the same whatever the rows.  (128 requests of 8192 tokens, 32 heads on 8, one in k + 1 of them
// verifying, the others on lists of 410; mma.sync first, repeats within 1 us, floors of 52, 44 and 39 us, with a dump 72, 64 and 59.
// 16 rows: 122 us and 155, with a dump 143 and 166; 20: 137 and 148, with one 171 and 159; 24: 125 and 138, with one 150 and 149.  32
// requests that all verify: 113 and 129, with one 137 both; 143 and 144, with one 191 and 156; 145 both, with one 192 and 158.)
constexpr int kFewRows = 24, kFewRowsDumped = 16;

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
    int B, Hq, Hkv, G, k, M, max_sparse;
    float scale;
    unsigned long long wait_ns;
};

// A weight is 2^(s - m + kLift) for a score s and its row's reference maximum m (base 2); the reference moves once a weight
// passes 2^kGrow.  So f16 weights are at most 2^14, and 2^6 or more for a row's largest.
constexpr float kLift = 6.f, kGrow = 8.f + kLift;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t h;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
    return h;
}

// The power of two that brings a query row, whose largest magnitude has the bf16 bits mx, to [2^14, 2^15), and its inverse.
__device__ __forceinline__ void query_scale(uint32_t mx, float *up, float *down) {
    const uint32_t e = max(mx >> 7, 15u);          // biased exponent, such that 2^(141 - e) is finite
    *up = __uint_as_float((268u - e) << 23);       // 2^(141 - e)
    *down = __uint_as_float((e - 14u) << 23);
}

// A row's factor in base 2 (scores = sum * factor), above 0 so that a masked score stays -inf.  mx as above, lim the last position
// that the row sees.  NaN for a row with a NaN or an infinity that sees any: its scores are infinite or NaN, and where all of them
// are -inf their weights alone would not tell them from masked ones.
__device__ __forceinline__ float softmax_factor(float fac, uint32_t mx, int lim) {
    return mx >= 0x7f80u && lim >= 0 ? __int_as_float(0x7fffffff) : fmaxf(fac * kLog2e, __int_as_float(1));
}

// The items of part 0 (all), 1 (of verify requests) or 2 (the others), of `rows` <= kFewRows rows at most.  after: another
// kernel on this stream has the verify items, and is the one waited for at the end.
cudaError_t launch_attn_kv4_few(const Kv4Params &p, int D, int rows, int part, bool after, int nsm, cudaStream_t st);

}  // namespace pillar
