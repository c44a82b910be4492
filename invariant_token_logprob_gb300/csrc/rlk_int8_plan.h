// rlk_int8_plan.h -- how the product of 8-bit integers (rlk_int8_linear.cu) cuts x's rows, K and
// shared and tensor memory: plain arithmetic without CUDA, so that a host compiler can check it.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace rlk {

constexpr int kInt8TileN = 128;    // channels per tile = UMMA M = TMEM lanes
constexpr int kInt8StageK = 128;   // k per stage
constexpr int kInt8MaxParts = 8;   // parts of K per tile (CTAs of a cluster)
constexpr int kInt8SumStages = 8;  // stages per fp32 sum: 1024 k, |sum| <= 128^2 1024 = 2^24

// Rows of x that a tile has room for.
constexpr int int8_room(int64_t rows) {
    return rows <= 16 ? 16 : rows <= 32 ? 32 : rows <= 64 ? 64 : rows <= 128 ? 128 : 192;
}
// Sets of four warps that add the sums up, 64 columns each; teams of four that turn codes into
// numbers; the accumulators' (two) and the numbers' buffers in tensor memory's 512 columns.
constexpr int int8_sets(int room) { return room <= 64 ? 1 : room / 64; }
constexpr int int8_teams(int room) { return room <= 128 ? 3 : 2; }
constexpr int int8_warps(int room) { return 2 + 4 * (int8_sets(room) + int8_teams(room)); }
constexpr int kInt8NumberCols = kInt8StageK / 2;  // a stage's numbers, two to a column
constexpr int int8_number_bufs(int room) { return room <= 128 ? 4 : 2; }
constexpr int int8_tmem_cols(int room) { return 2 * room + int8_number_bufs(room) * kInt8NumberCols; }

constexpr int kInt8CodeBytes = kInt8TileN * kInt8StageK;
constexpr int int8_stage_bytes(int room) { return kInt8CodeBytes + room * kInt8StageK * 2; }
constexpr int int8_stages(int room) {
    return room == 16 ? 10 : room == 32 ? 8 : room == 64 ? 6 : room == 128 ? 4 : 3;
}
constexpr int kInt8MaxBarriers = 2 * 10 + 2 * 4 + 2 * 2 + 1;
constexpr size_t int8_smem_bytes(int room) {
    return 1024 + size_t(int8_stages(room)) * int8_stage_bytes(room) + kInt8MaxBarriers * 8 + 16;
}

struct Int8Plan {
    int chunks;    // of x's rows
    int rows;      // of x per chunk (the last one may be short)
    int room;
    int mma_n;     // columns of the products: rows, rounded up to 16
    int tiles;     // of channels
    int stages;    // of the whole K
    int parts;     // of K
};

// The parts of K follow the fewest rounds of stages over the SMs, counting a few stages' time
// for a part's beginning and end.  (No bit depends on any of this: the sums are exact.)
inline Int8Plan int8_plan(int64_t T, int64_t N, int64_t K, int num_sms) {
    Int8Plan p = {};
    p.chunks = int((T + 191) / 192);
    p.rows = int((T + p.chunks - 1) / p.chunks);
    p.room = int8_room(p.rows);
    p.mma_n = (p.rows + 15) / 16 * 16;
    p.tiles = int((N + kInt8TileN - 1) / kInt8TileN);
    p.stages = int((K + kInt8StageK - 1) / kInt8StageK);
    const int64_t items = int64_t(p.tiles) * p.chunks;
    p.parts = 1;
    int64_t best = INT64_MAX;
    for (int s = 1; s <= kInt8MaxParts && s <= p.stages; ++s) {
        const int64_t rounds = (items * s + num_sms - 1) / num_sms;
        const int64_t cost = rounds * ((p.stages + s - 1) / s + 4 + (s > 1 ? 2 : 0));
        if (cost < best) {
            best = cost;
            p.parts = s;
        }
    }
    return p;
}

}  // namespace rlk
