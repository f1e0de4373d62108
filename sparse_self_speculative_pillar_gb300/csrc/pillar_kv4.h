// pillar_kv4.h -- host-side launches of the 4-bit cache's append (pillar_kv4.cu) and of the reads of both
// quantised caches (pillar_kv_read.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace pillar {

struct Kv4AppendArgs {
    const uint16_t *k_new, *v_new;
    long long k_stride, v_stride;  // elements between two tokens' rows
    const int *req_len, *new_off, *table;
    uint8_t *k4, *v4, *k_scale, *v_scale;
    int *flags;  // device error word, or null
    int n, B, Hkv, D, max_blocks, num_blocks, max_len;
};
cudaError_t launch_kv4_append(const Kv4AppendArgs &a, int nsm, cudaStream_t st);

struct KvReadArgs {
    const uint8_t *k, *v;          // codes
    const void *k_scale, *v_scale; // 4 bits: bytes, a scale per 16 values; 8 bits: fp32, one per (block, KV head)
    const int *first, *out_off, *table;
    uint16_t *k_out, *v_out;
    long long k_stride, v_stride;  // elements between two tokens' rows
    int *flags;
    int n, B, Hkv, D, max_blocks, num_blocks, max_len;
    int bits;                      // 4 or 8
};
cudaError_t launch_kv_read(const KvReadArgs &a, int nsm, cudaStream_t st);

}  // namespace pillar
