// pillar_map.h -- host-side launch of the block map (pillar_map.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace pillar {

// What the scan leaves for the expansion beside the call's own arrays: one record for the call, one per request.
struct MapHeader {
    int err;          // PILLAR_FLAG_* bits
    int head, count;  // the ring's state when the call began
    int pad;
    long long released;  // blocks given back
    long long pad2[29];  // keeps the records 256-byte aligned
};
static_assert(sizeof(MapHeader) == 256, "header size");

struct MapRequest {
    int take;  // its first block from the ring: head + take
    int give;  // its first released block: pushed at head + count + give
};

inline size_t map_ws_bytes(int B) {
    return (sizeof(MapHeader) + sizeof(MapRequest) * (size_t)B + 255) & ~size_t(255);
}

struct MapArgs {
    const int *req_len, *prev_len;
    int *table, *ring, *state, *granted;
    long long *kv_off;
    int *slots;
    long long slot_capacity;
    int *new_off, *new_slots;
    long long new_capacity;
    char *ws;
    int B, max_blocks, max_len, num_blocks;
};
cudaError_t launch_block_map(const MapArgs &a, int nsm, cudaStream_t st);

}  // namespace pillar
