// pillar_prompt.h -- host-side launch of the attention over prompts (pillar_prompt.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace pillar {

constexpr int kPromptRows = 128;  // query rows of a row tile

struct PromptHeader {
    int err;        // PILLAR_FLAG_* bits
    int num_tiles;
    int pad[62];
};
static_assert(sizeof(PromptHeader) == 256, "header size");

// `rows` consecutive query rows of one sequence: one row tile, taken for two heads of a KV group at once, or
// two row tiles of one head when the groups have no pairs.
struct PromptTile {
    int row0;  // the sequence's first row
    int len;   // its length
    int tile;  // rows rows * tile .. rows * (tile + 1) - 1 of it
    int pad;
};
inline int prompt_tile_rows(int G) { return G % 2 == 0 ? kPromptRows : 2 * kPromptRows; }

inline long long prompt_max_tiles(int B, int n) { return (long long)n / kPromptRows + B; }
inline size_t prompt_ws_bytes(int B, int n) {
    return (sizeof(PromptHeader) + sizeof(PromptTile) * (size_t)prompt_max_tiles(B, n) + 255) & ~size_t(255);
}

struct PromptArgs {
    const uint16_t *q, *k, *v;
    long long q_stride, k_stride, v_stride;  // elements between two tokens' rows
    const int *seq_off;
    uint16_t *out;
    float *lse;  // or null
    char *ws;
    int B, n, Hq, Hkv, D, max_len;
    float scale;
    unsigned long long wait_ns;
};
cudaError_t launch_prompt(const PromptArgs &a, int nsm, cudaStream_t st);

}  // namespace pillar
