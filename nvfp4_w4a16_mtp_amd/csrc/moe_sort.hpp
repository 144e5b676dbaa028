// What the sorted-token MoE kernels share: the sort's launches and the tile map that
// it leaves for the experts' products.
#pragma once

#include "common.hpp"

namespace nvfp4 {

constexpr int kMaxExperts = 1024, kMaxTopK = 16;

// Row tiles of the experts' products, in expert order: tile i holds rows
// [row, row + tile height) of the sorted pairs, cut at the expert's end.
struct MoeTile {
    int32_t expert, row;
};

struct SortArgs {
    const float *logits;     // [m][experts], or NULL: ids are given
    int m, experts, top_k;
    int32_t *ids;            // [m][top_k]
    float *w;                // [m][top_k]
    int32_t *offsets;        // [experts + 1]
    int32_t *order, *place;  // [m * top_k]
    int32_t *hist;           // [blocks][(experts + 1) / 2], two experts a word
    int per_block;           // tokens a block of the counting launch
    MoeTile *tiles;          // NULL, or the tile map
    int32_t *tile_count;     // [1], with tiles
    int tile_rows;
};

size_t moe_sort_hist_bytes(int m, int experts);
void launch_moe_sort(SortArgs a, hipStream_t s);

// Element types of rows: fp32 or bf16.
void launch_moe_combine(const void *ys, bool ys_bf16, int m, int hidden, int top_k, const int32_t *place, const float *w,
                        void *y, bool y_bf16, hipStream_t s);

int check_moe_sizes(int m, int experts, int top_k, const char *who);

}  // namespace nvfp4
