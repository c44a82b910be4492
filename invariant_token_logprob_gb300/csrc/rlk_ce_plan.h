// rlk_ce_plan.h -- how the cross entropy's backward (rlk_cross_entropy_backward) cuts the
// vocabulary into pieces and a piece into ranges: plain arithmetic without CUDA, so that a host
// compiler can check it.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace rlk {

struct CePlan {
    int64_t rows;   // vocabulary entries of a piece (a multiple of 256; the last one may be short)
    int64_t pieces;
    int parts;      // ranges of a piece's entries whose grad_h sums are held apart
};

constexpr int64_t kCeTile = 256;         // rows and columns of a unit of each product
constexpr int64_t kCeBlock = 64;         // k of a block
constexpr int64_t kCePairs = 76;         // CTA pairs of a GB300 (whatever the device has)
constexpr int kCeMaxParts = 8;
constexpr double kCeLaunchUs = 3.0;
// Bytes that a piece's dz and its transpose may take together.
constexpr int64_t kCeBytes = int64_t(1) << 29;

inline int64_t ce_cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t ce_row_stride(int64_t n) { return ce_cdiv(n, 8) * 8; }

// Estimated time (us) of one piece with `rows` entries: whole rounds of units over the pairs for
// the scores and for both products, 0.27 us per block of k, and the partial sums of grad_h,
// which are read and written once per piece, half of it behind the products.
inline double ce_piece_cost(int64_t T, int64_t H, int64_t rows, int parts) {
    const double block_us = 0.27, bytes_per_us = 6.7e6;
    const int64_t mt = ce_cdiv(T, kCeTile), nt = ce_cdiv(H, kCeTile), vt = ce_cdiv(rows, kCeTile);
    const double scores = double(ce_cdiv(mt * vt, kCePairs)) * double(ce_cdiv(H, kCeBlock));
    const double weight = double(ce_cdiv(vt * nt, kCePairs)) * double(ce_cdiv(T, kCeBlock));
    const double hidden = double(ce_cdiv(mt * nt * parts, kCePairs)) *
                          double(ce_cdiv(ce_cdiv(rows, kCeBlock), parts));
    return (scores + weight + hidden) * block_us + 3 * kCeLaunchUs +
           double(parts) * double(T) * double(H) * 4.0 / bytes_per_us;
}

// Entries of a range, and ranges that hold any (those of the first, whole piece).
inline int64_t ce_part_rows(const CePlan& p) {
    return ce_cdiv(ce_cdiv(p.rows, kCeBlock), p.parts) * kCeBlock;
}

// From the shape alone, so that the order of grad_h's sums is.
inline CePlan ce_plan(int64_t T, int64_t H, int64_t V) {
    int64_t most = kCeBytes / (4 * ce_row_stride(T)) / kCeTile * kCeTile;
    if (most < kCeTile) most = kCeTile;
    const int64_t fewest = ce_cdiv(V, most);
    CePlan best = {};
    double best_cost = 0;
    for (int64_t n = fewest; n <= (fewest == 1 ? 1 : 2 * fewest); ++n) {
        const int64_t rows = ce_cdiv(ce_cdiv(V, n), kCeTile) * kCeTile;
        const int64_t pieces = ce_cdiv(V, rows);
        for (int parts = 1; parts <= kCeMaxParts; ++parts) {
            if (parts > 1 && ce_cdiv(ce_cdiv(rows, kCeBlock), parts) < 8) break;
            double cost = double(pieces) * ce_piece_cost(T, H, rows, parts);
            if (pieces == 1 && parts == 1) cost -= kCeLaunchUs;  // grad_h comes without a sum
            if (best.rows == 0 || cost < best_cost * 0.995) {
                best = {rows, pieces, parts};
                best_cost = cost;
            }
        }
    }
    return best;
}

// Workspace of the backward, from the first address in it that is a multiple of kCeAlign: dz
// [T][rows] and its transpose, 16 bits each, grad_h's sums [parts][T][H] in fp32, h in fp16, and
// what belongs to a row (32 bytes and 4) and to all.
constexpr size_t kCeAlign = 256;
struct CeLayout {
    size_t dzt, sums, h, rows, tops, top, bytes;  // offsets; dz lies at 0
};
inline CeLayout ce_layout(int64_t T, int64_t H, const CePlan& p) {
    auto round = [](size_t b) { return (b + 255) / 256 * 256; };
    CeLayout l;
    l.dzt = round(size_t(T) * size_t(p.rows) * 2);
    l.sums = l.dzt + round(size_t(p.rows) * size_t(ce_row_stride(T)) * 2);
    l.h = l.sums + round(size_t(p.parts) * size_t(T) * size_t(H) * 4);
    l.rows = l.h + round(size_t(T) * size_t(H) * 2);
    l.tops = l.rows + round(size_t(T) * 32);
    l.top = l.tops + round(size_t(T) * 4);
    l.bytes = l.top + 256;
    return l;
}

}  // namespace rlk
