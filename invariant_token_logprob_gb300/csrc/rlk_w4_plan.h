// rlk_w4_plan.h -- how the product with a 4-bit weight (rlk_w4_linear.cu) cuts K, and which
// words of the scales and zero points it copies: plain arithmetic without CUDA, so that a host
// compiler can check it.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define RLK_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define RLK_HOST_DEVICE inline
#endif

namespace rlk {

constexpr int kW4TileN = 128;        // rows of W per tile
constexpr int kW4ScaleGroups = 32;   // groups of a tile's rows copied together: a chunk

// Words per row that a chunk's values of `size` bytes fill, and one more for rows that start
// inside a word.
constexpr int w4_chunk_words(int size) { return kW4ScaleGroups * size / 4 + 1; }

// Byte offset of word w of a tile row's chunk, in an array of row_values values of `size`
// bytes per row; value `from` is the chunk's first one of the tile's first row.
RLK_HOST_DEVICE int64_t w4_chunk_word(int64_t from, int row, int row_values, int size, int w) {
    return ((from + int64_t(row) * row_values) * size & ~int64_t(3)) + w * 4;
}

// Whether all words of a tile's chunk lie inside an array of n_rows rows: the last word of the
// last row does.  (A row's words always span kW4ScaleGroups values and more, which are many
// rows where a row has few groups, so a distance in rows would not tell.)
RLK_HOST_DEVICE bool w4_chunk_inside(int64_t from, int row_values, int64_t n_rows, int size) {
    return w4_chunk_word(from, kW4TileN - 1, row_values, size, w4_chunk_words(size) - 1) + 4 <=
           n_rows * row_values * size;
}

// Parts of K per tile: the fewest rounds of stages over the SMs, counting a few stages'
// time for a part's beginning and end.  The cut decides the order of the sums, so it follows
// from the weight's shape alone: the number of SMs is the GB300's, whatever the device has.
constexpr int kW4MaxParts = 8;
constexpr int kW4PlanSms = 152;
inline int w4_parts_of_k(int tiles, int num_stages) {
    int best = 1;
    int64_t best_cost = INT64_MAX;
    for (int s = 1; s <= kW4MaxParts && s <= num_stages; ++s) {
        const int64_t rounds = (int64_t(tiles) * s + kW4PlanSms - 1) / kW4PlanSms;
        const int64_t cost = rounds * ((num_stages + s - 1) / s + 3 + (s > 1 ? 1 : 0));
        if (cost < best_cost) {
            best_cost = cost;
            best = s;
        }
    }
    return best;
}

}  // namespace rlk
