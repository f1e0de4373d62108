// pillar_kv8.h -- host-side launch of the append to the 8-bit cache (pillar_kv8.cu).
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

namespace pillar {

struct Kv8AppendArgs {
    const uint16_t *k_new, *v_new;
    long long k_stride, v_stride;  // elements between two tokens' rows
    const int *req_len, *new_off, *table;
    uint8_t *k8, *v8;
    float *k_scale, *v_scale;
    int *flags;  // device error word, or null
    int n, B, Hkv, D, max_blocks, num_blocks, max_len;
};
cudaError_t launch_kv8_append(const Kv8AppendArgs &a, int nsm, cudaStream_t st);

}  // namespace pillar
