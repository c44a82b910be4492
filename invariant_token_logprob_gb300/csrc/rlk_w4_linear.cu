// rlk_w4_linear.cu -- y [T][N] = x [T][K] . W^T for a weight in 4 bits with group scales
// (the format of rlk_w4.cu), on the tensor cores:
//   y[t][n] = sum_g s[n][g] * sum_{k in g} (q[n][k] - z[n][g]) x[t][k]
// q - z is a whole number up to 15 in magnitude, exact in bf16 and fp16, so a group's sum
// runs on the tensor core on 16-bit operands with exact products, and the group's scale
// meets it once, in fp32, on the CUDA cores.
//
// What bounds it: the codes, N K / 2 bytes, read once.  x is small.  The codes must become
// 16-bit numbers on the way (11 instructions per 8 codes), so a plain row-times-vector
// kernel would spend twice the instructions on the products alone; and a tile of numbers
// written to shared memory for the tensor core and read back by it would take more
// shared-memory time than the codes take from HBM.  So the tile goes through tensor memory:
// a thread owns one row of a 128-row tile, turns the row's codes into numbers in registers
// and stores them to its TMEM lane, from where they are the A operand.  x is B (N = the
// rows of x, 16, 32 or 64 at a time).
// N = 151936, K = 4096, group 128, bf16: T = 1 58 us (5.5 TB/s, 0.81 of a copy), T = 32 65 us,
// T = 64 80 us (83 with zero points), where the x that comes in again for every tile, 32 KB a stage next to 16 KB of
// codes, costs more than the codes.  N = K = 4096, T = 1: 6.4 us.
//
// One CTA per SM; a tile's K goes by in stages of 256 k:
//   warp 0       TMA producer: the stage's codes (16 KB) and x
//   warp 1       MMA issuer: per stage and group its MMAs into a D buffer, fresh
//   warp 2       copies the scales and zero points, 32 groups of the tile's rows at a time,
//                into shared memory, where a thread finds its row's: straight from global
//                memory every lane of a warp would touch another row, 32 sectors a load.
//                Word by word, so that any number of groups per row will do: a row's words
//                are those that hold its groups, its values lie from its own shift on
//   warps 3..    products, one or two sets of four: a thread keeps a row's running sums, one
//                per row of x (of half of them):
//                acc = fma(D, scale, acc), stage after stage, group after group
//   the others   two or three teams of four warps, which take the stages in turn: a thread
//                turns its row's codes into numbers and stores them to the team's A buffer
// Turning codes into numbers takes 5 instructions of the half-rate integer pipe per 8 codes,
// about 21 us of the SMs' time for 622 M codes next to 47 us of HBM's: the teams are there so
// that one's waits are the others' work.
//
// Few tiles (N of some thousands): the K range of a tile is cut into `splits` parts, one
// per CTA of a cluster, whose sums meet through distributed shared memory in the order of k.
// The cut follows from N and K (rlk_w4_plan.h); tiles, stages and the order of the sums are fixed; a row of
// x is one column of D.  So a row's bits do not depend on T.
//
// Every wait is bounded (2 s); on expiry the kernel records it, waits for its copies and
// products under way and returns.
#include <atomic>

#include "rlk_logits.cuh"
#include "rlk_logits_w4.h"
#include "rlk_ptx.cuh"
#include "rlk_w4.cuh"
#include "rlk_w4_plan.h"

namespace rlk {
namespace {

constexpr int kTileN = kW4TileN;             // rows of W per tile = UMMA M = TMEM lanes
constexpr int kStageK = 256;                 // k per stage
constexpr int kCodeBytes = kTileN * kStageK / 2;
constexpr int kTeamWarps = 4;
constexpr int kFirstProductWarp = 3;
// Sets of four product warps, which share the columns: 64 in one set's registers leave none to
// load ahead with (N = 151936, K = 4096, T = 64: group 128 83 us, group 32 176 us; two sets
// 80 and 166 us).
constexpr int product_sets(int cols) { return cols < 64 ? 1 : 2; }
constexpr int first_team_warp(int cols) { return kFirstProductWarp + 4 * product_sets(cols); }
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kABufCols = kStageK / 2;  // two 16-bit numbers per column
constexpr int kMaxSplits = kW4MaxParts;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 200000000ull;

__device__ unsigned int g_w4_error;  // bit 0: a wait ran out; bit 1: a teardown wait ran out

// Scales and zero points of kScaleGroups groups of a tile's rows, in words (one more than
// they fill, for rows that start inside a word).  The rows lie an odd number of words apart,
// so 32 rows' values of one group lie in 32 banks.
constexpr int kScaleGroups = kW4ScaleGroups;
constexpr int kScaleWords = w4_chunk_words(2);
constexpr int kZeroWords = w4_chunk_words(1);
static_assert(kScaleWords % 2 == 1 && kZeroWords % 2 == 1, "banks");
constexpr int kScaleBytes = kTileN * (kScaleWords + kZeroWords) * 4;

// Rows of x a CTA takes at a time, and the MMA's N (at least 16).
constexpr int mma_n(int cols) { return cols < 16 ? 16 : cols; }
constexpr int stage_bytes(int cols) { return kCodeBytes + mma_n(cols) * kStageK * 2; }
// Groups of 32 run through a chunk of scales in four stages: two more buffers, a stage less.
constexpr int scale_bufs_of(int groups) { return groups == 8 ? 4 : 2; }
constexpr int stages(int cols, int groups) {
    return (cols <= 16 ? 8 : cols == 32 ? 6 : 4) - (groups == 8 ? 1 : 0);
}
// Tensor memory: A buffers (one per team) first, then the D buffers, `cols` columns for
// each of some groups of a stage, 128 columns at most: two buffers have to fit, or the products
// wait for the MMAs and the MMAs for them (N = 151936, K = 4096, T = 64, a stage's groups
// together: group 64 126 us, by twos 108 us).
constexpr int d_groups(int cols, int groups) {
    return groups < 128 / mma_n(cols) ? groups : 128 / mma_n(cols);
}
constexpr int d_cols(int cols, int groups) { return mma_n(cols) * d_groups(cols, groups); }
constexpr int num_teams(int cols, int groups) { return d_cols(cols, groups) <= 64 ? 3 : 2; }
constexpr int num_d(int cols, int groups) {
    return (int(kTmemCols) - num_teams(cols, groups) * int(kABufCols)) / d_cols(cols, groups) < 4
               ? (int(kTmemCols) - num_teams(cols, groups) * int(kABufCols)) / d_cols(cols, groups)
               : 4;
}
constexpr int kMaxBarriers = 2 * 8 + 2 * 3 + 2 * 4 + 2 * 4 + 1;
constexpr size_t smem_bytes(int cols, int groups) {
    return 1024 + size_t(stages(cols, groups)) * stage_bytes(cols) +
           scale_bufs_of(groups) * kScaleBytes + kMaxBarriers * 8 + 16;
}
static_assert(smem_bytes(64, 4) <= 227 * 1024 && smem_bytes(64, 8) <= 227 * 1024 &&
                  smem_bytes(64, 2) <= 227 * 1024 && smem_bytes(32, 8) <= 227 * 1024 &&
                  smem_bytes(16, 8) <= 227 * 1024 && smem_bytes(32, 4) <= 227 * 1024 &&
                  smem_bytes(16, 4) <= 227 * 1024,
              "shared memory per CTA");
static_assert((64 + kMaxSplits) * kTileN * 4 <= stages(8, 8) * stage_bytes(8) &&
                  (64 + kMaxSplits) * kTileN * 4 <= stages(64, 8) * stage_bytes(64),
              "the parts' sums take the stages' place");

struct Args {
    const void* scales;
    const uint8_t* zeros;
    void* y;
    int64_t T;
    int N, num_groups;
    int chunks;        // of `cols` rows of x
    int items;         // tiles * chunks
    int num_stages;    // of the whole K
    int splits;
    int x_rows;        // rows of an x box: fewer than the MMA's N where T is (the others'
                       // columns hold what the shared memory held and are never read)
    int stall_selftest;  // bounded-wait self-test: 1, the producer issues no copies; 2, the MMA
                         // issuer consumes no stage
};

// By whole warps or single lanes; the usual wait finds its phase complete.
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity,
                                             volatile int* abort_flag) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = global_timer_ns();
    uint32_t spins = 0;
    while (true) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((++spins & 63u) == 0) {
            if (*abort_flag) return false;
            if (global_timer_ns() - t0 > kWaitLimitNs) {
                *abort_flag = 1;
                atomicOr(&g_w4_error, 1u);
                return false;
            }
        }
    }
}

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > kDrainLimitNs) {
            atomicOr(&g_w4_error, 2u);
            return;
        }
    }
}

template <typename Elem>
__device__ __forceinline__ void numbers(const uint4& words, const Numbers<Elem>& minus,
                                        uint32_t (&r)[16]) {
    const uint32_t w[4] = {words.x, words.y, words.z, words.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        minus.pair(w[i], r[4 * i], r[4 * i + 1]);
        minus.pair(w[i] >> 8, r[4 * i + 2], r[4 * i + 3]);
    }
}

// kGroups groups, kStride columns apart, of N (8, 16 or 32) fp32 columns of this thread's lane,
// each group scaled into acc.  A piece is loaded while the one before is added.
template <int N, int kGroups, int kStride>
__device__ __forceinline__ void add_products(uint32_t taddr, const float* scale, F2 (&acc)[N / 2]) {
    constexpr int kPiece = N < 16 ? N : 16, kPieces = N / kPiece;
    uint32_t r[2][kPiece];
    auto load = [&](int i) {
        const uint32_t at = taddr + i / kPieces * kStride + i % kPieces * kPiece;
        if constexpr (kPiece == 8)
            tmem_ld8(at, r[i % 2]);
        else
            tmem_ld16(at, r[i % 2]);
    };
    load(0);
#pragma unroll
    for (int i = 0; i < kGroups * kPieces; ++i) {
        tmem_ld_wait();
        if (i + 1 < kGroups * kPieces) load(i + 1);
        const F2 s = pack2(scale[i / kPieces], scale[i / kPieces]);
        const int c = i % kPieces * kPiece;
#pragma unroll
        for (int j = 0; j < kPiece; j += 2)
            acc[(c + j) / 2] = fma2(pack2(__uint_as_float(r[i % 2][j]), __uint_as_float(r[i % 2][j + 1])),
                                    s, acc[(c + j) / 2]);
    }
}

// Copies kScaleGroups values of kSize bytes of each of a tile's rows, value `from` of an
// array of n_rows rows on and row_values further per row, as the words that hold them.  A warp
// takes whole rows side by side: rows four (kSize 1) or two apart start at the same place
// of a word, so a lane's words lie a fixed step apart.  The word behind comes at the end.
template <int kSize>
__device__ __forceinline__ void copy_groups(const uint8_t* base, int64_t from, int row_values,
                                            int64_t n_rows, int lane, uint32_t to) {
    constexpr int kWords = kScaleGroups * kSize / 4;  // and one more
    constexpr int kRows = 32 / kWords;                // at once
    static_assert(kRows * kSize % 4 == 0, "the rows of a step start at the same place of a word");
    auto word = [&](int row, int w) { return w4_chunk_word(from, row, row_values, kSize, w); };
    const int64_t at = word(lane / kWords, lane % kWords);
    const uint32_t dst = to + ((lane / kWords) * (kWords + 1) + lane % kWords) * 4;
    const int64_t step = int64_t(kRows) * row_values * kSize;
    // one warp keeps up with all others only with few instructions per word
    if (w4_chunk_inside(from, row_values, n_rows, kSize)) {
        const uint8_t* src = base + at;
        uint32_t d = dst;
#pragma unroll 8
        for (int r = 0; r < kTileN; r += kRows) {
            copy_word_async(d, src, 4);
            src += step;
            d += kRows * (kWords + 1) * 4;
        }
#pragma unroll 1
        for (int r = 0; r < kTileN; r += 32)
            copy_word_async(to + ((r + lane) * (kWords + 1) + kWords) * 4,
                            base + word(r + lane, kWords), 4);
        return;
    }
    const int64_t end = n_rows * row_values * kSize;
    auto copy = [&](int64_t src, uint32_t d) {
        const int64_t left = end - src;
        const uint32_t bytes = left <= 0 ? 0u : left < 4 ? uint32_t(left) : 4u;
        copy_word_async(d, bytes ? base + src : base, bytes);
    };
    int64_t src = at;
    uint32_t d = dst;
#pragma unroll 4
    for (int r = 0; r < kTileN; r += kRows) {
        copy(src, d);
        src += step;
        d += kRows * (kWords + 1) * 4;
    }
#pragma unroll
    for (int r = lane; r < kTileN; r += 32)
        copy(word(r, kWords), to + (r * (kWords + 1) + kWords) * 4);
}

// kCols: rows of x at a time; kGroups: groups per stage.
template <typename Elem, typename Out, int kCols, int kGroups, bool kZeros>
__global__ void __launch_bounds__(32 * (first_team_warp(kCols) + kTeamWarps * num_teams(kCols, kGroups)), 1)
    linear_w4_kernel(const __grid_constant__ CUtensorMap tmap_w,
                     const __grid_constant__ CUtensorMap tmap_x, const Args p) {
    constexpr int kN = mma_n(kCols);
    constexpr int kStages = stages(kCols, kGroups);
    constexpr int kScaleBufs = scale_bufs_of(kGroups);
    constexpr int kStageBytes = stage_bytes(kCols);
    constexpr int kTeams = num_teams(kCols, kGroups);
    constexpr int kDs = num_d(kCols, kGroups);
    constexpr uint32_t kDBase = kTeams * kABufCols;
    constexpr uint32_t kDBufCols = d_cols(kCols, kGroups);
    constexpr int kDGroups = d_groups(kCols, kGroups);
    constexpr int kSets = product_sets(kCols), kMine = kCols / kSets;  // a product warp's columns
    constexpr int kProductWarps = 4 * kSets, kFirstTeamWarp = first_team_warp(kCols);
    constexpr int kChunkStages = kScaleGroups / kGroups;  // stages per chunk of scales
    constexpr float kUnit = Numbers<Elem>::kUnit;  // (a power of two: dividing is exact)
    constexpr uint32_t kIdesc =
        std::is_same<Elem, __half>::value ? idesc_f16_f32(kTileN, kN) : idesc_bf16_f32(kTileN, kN);
    static_assert(kDs >= 2 && kGroups % kDGroups == 0 && kDBase + kDs * kDBufCols <= kTmemCols, "tensor memory");
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t stage0 = raw_addr + pad;
    uint8_t* scale_bufs = smem + size_t(kStages) * kStageBytes;
    uint64_t* bars = reinterpret_cast<uint64_t*>(scale_bufs + kScaleBufs * kScaleBytes);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kMaxBarriers);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const uint32_t bar0 = smem_u32(bars);
    auto full_bar = [&](uint32_t s) { return bar0 + 8 * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8 * (kStages + s); };
    constexpr int kA = 2 * kStages, kD = kA + 2 * kTeams, kS = kD + 2 * kDs;
    static_assert(kS + 2 * kScaleBufs + 1 <= kMaxBarriers, "barriers");
    auto a_full = [&](uint32_t team) { return bar0 + 8 * (kA + team); };
    auto a_empty = [&](uint32_t team) { return bar0 + 8 * (kA + kTeams + team); };
    auto d_full = [&](uint32_t d) { return bar0 + 8 * (kD + d); };
    auto d_empty = [&](uint32_t d) { return bar0 + 8 * (kD + kDs + d); };
    auto s_full = [&](uint32_t buf) { return bar0 + 8 * (kS + buf); };
    auto s_empty = [&](uint32_t buf) { return bar0 + 8 * (kS + kScaleBufs + buf); };
    const uint32_t drain_bar = bar0 + 8 * (kS + 2 * kScaleBufs);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), kTeamWarps + 1);  // the codes' readers, and the MMAs
        }
        for (int i = 0; i < kTeams; ++i) {
            mbar_init(a_full(i), kTeamWarps);
            mbar_init(a_empty(i), 1);
        }
        for (int i = 0; i < kDs; ++i) {
            mbar_init(d_full(i), 1);
            mbar_init(d_empty(i), kProductWarps);
        }
        for (int i = 0; i < kScaleBufs; ++i) {
            mbar_init(s_full(i), 32);  // the copying warp's lanes
            mbar_init(s_empty(i), kProductWarps + (kZeros ? kTeams * kTeamWarps : 0));
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmap_w);
        tma_prefetch_desc(&tmap_x);
    }
    if (warp == 1) {
        tmem_alloc<1>(smem_u32(tmem_slot), kTmemCols);
        tmem_relinquish<1>();
    }
    tc_fence_before_sync();
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    grid_dependency_wait();
    grid_launch_dependents();

    // A cluster takes one item, a CTA alone every gridDim.x-th; either way these stages of K.
    const int rank = p.splits > 1 ? int(cluster_ctarank()) : 0;
    const int first_item = p.splits > 1 ? int(blockIdx.x) / p.splits : int(blockIdx.x);
    const int item_step = p.splits > 1 ? p.items : int(gridDim.x);
    const int k_first = int(int64_t(p.num_stages) * rank / p.splits);
    const int k_last = int(int64_t(p.num_stages) * (rank + 1) / p.splits);

    const int row_in_tile = (warp & 3) * 32 + lane;  // (a warp reaches the lanes of its quadrant)
    const uint32_t lane_base = tmem_base + (uint32_t((warp & 3) * 32) << 16);
    F2 acc[kMine / 2];  // of the product warps: the sums of columns mine0 ..
    const int mine0 = kSets > 1 ? (warp - kFirstProductWarp) / 4 * kMine : 0;

    // By a whole warp: all lanes wait, all learn the outcome.
    auto warp_wait = [&](uint32_t bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_bounded(bar, parity, abort_flag)) != 0;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ producer
        if (lane == 0) {
            uint32_t stage = 0, phase = 0;
            int issued = 0;
            bool ok = true;
            const int items = p.stall_selftest == 1 ? 0 : p.items;
            for (int item = first_item; ok && item < items; item += item_step) {
                const int tile = item / p.chunks;
                const int chunk = item - tile * p.chunks;
                for (int ks = k_first; ks < k_last; ++ks) {
                    if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = stage0 + stage * kStageBytes;
                    mbar_arrive_expect_tx(full_bar(stage), kCodeBytes + uint32_t(p.x_rows) * kStageK * 2);
                    tma_load_2d(&tmap_w, full_bar(stage), at, ks * (kStageK / 2), tile * kTileN);
#pragma unroll
                    for (int i = 0; i < kStageK / 64; ++i)
                        tma_load_2d(&tmap_x, full_bar(stage), at + kCodeBytes + i * kN * 128,
                                    ks * kStageK + i * 64, chunk * kCols);
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // The copies this thread started land before the CTA exits, whichever role gave up:
            // the others may stop waiting for them after the last one was issued.  (Usually
            // they have landed, or the others wait for them too.)
            for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i) {
                const uint32_t bar = full_bar(i % kStages), parity = uint32_t(i / kStages) & 1u;
                if (!wait_bounded(bar, parity, abort_flag)) wait_drain(bar, parity);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // The whole warp runs the loop and one elected lane issues: addresses and
        // descriptors then are warp-uniform, which single-lane code does not let them be.
        const bool leader = elect_one();
        uint32_t stage = 0, phase = 0, team = 0, team_phase = 0, d = 0, d_phase = 0;
        bool ok = true;
        const int items = p.stall_selftest == 2 ? 0 : p.items;
        for (int item = first_item; ok && item < items; item += item_step) {
            for (int ks = k_first; ks < k_last; ++ks) {
                ok = warp_wait(full_bar(stage), phase) && warp_wait(a_full(team), team_phase);
                if (!ok) break;
                const uint64_t x_desc = sw128_kmajor_desc(stage0 + stage * kStageBytes + kCodeBytes);
                const uint32_t a_tmem = tmem_base + team * kABufCols;
#pragma unroll
                for (int g0 = 0; g0 < kGroups; g0 += kDGroups) {
                    ok = warp_wait(d_empty(d), d_phase ^ 1u);
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint32_t d_tmem = tmem_base + kDBase + d * kDBufCols;
                    if (leader) {
                        constexpr int kPerGroup = kStageK / 16 / kGroups;
#pragma unroll
                        for (int i = g0 * kPerGroup; i < (g0 + kDGroups) * kPerGroup; ++i) {
                            const uint64_t off = uint64_t((i / 4 * kN * 128 + i % 4 * 32) >> 4);
                            umma_f16_tmem_a(d_tmem + (i / kPerGroup - g0) * kN, a_tmem + i * 8,
                                            x_desc + off, kIdesc, i % kPerGroup != 0 ? 1u : 0u);
                        }
                        umma_commit(d_full(d));
                    }
                    if (++d == kDs) {
                        d = 0;
                        d_phase ^= 1u;
                    }
                }
                if (!ok) break;
                if (leader) {
                    umma_commit(a_empty(team));
                    umma_commit(empty_bar(stage));
                }
                __syncwarp();
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++team == kTeams) {
                    team = 0;
                    team_phase ^= 1u;
                }
            }
        }
        if (leader) {
            umma_commit(drain_bar);  // no MMA may still run when TMEM is freed
            wait_drain(drain_bar, 0);
        }
        __syncwarp();
    } else if (warp == 2) {
        // ------------------------------------------------------------ scales
        uint32_t buf = 0, buf_phase = 0;
        bool ok = true;
        for (int item = first_item; ok && item < p.items; item += item_step) {
            const int64_t n0 = int64_t(item / p.chunks) * kTileN;
            for (int ks = k_first; ks < k_last; ks += kChunkStages) {
                ok = warp_wait(s_empty(buf), buf_phase ^ 1u);
                if (!ok) break;
                const uint32_t to = smem_u32(scale_bufs + buf * kScaleBytes);
                const int64_t from = n0 * p.num_groups + ks * kGroups;  // the first row's first group
                copy_groups<2>(static_cast<const uint8_t*>(p.scales), from, p.num_groups, p.N, lane, to);
                if (kZeros)
                    copy_groups<1>(p.zeros, from, p.num_groups, p.N, lane, to + kTileN * kScaleWords * 4);
                copy_words_arrive(s_full(buf));
                if (++buf == kScaleBufs) {
                    buf = 0;
                    buf_phase ^= 1u;
                }
            }
        }
        copy_words_wait_all();  // (no copy outlives the CTA)
        __syncwarp();
    } else if (warp < kFirstTeamWarp) {
        // ------------------------------------------------------------ products
        uint32_t d = 0, d_phase = 0, buf = 0, buf_phase = 0;
        bool ok = true;
        for (int item = first_item; ok && item < p.items; item += item_step) {
            const int tile = item / p.chunks;
            const int chunk = item - tile * p.chunks;
            const int n = tile * kTileN + row_in_tile;
            const uint32_t row_first = uint32_t(n) * uint32_t(p.num_groups);  // (its low bit counts)
#pragma unroll
            for (int t = 0; t < kMine / 2; ++t) acc[t] = pack2(0.0f, 0.0f);
            for (int ks0 = k_first; ok && ks0 < k_last; ks0 += kChunkStages) {
                ok = warp_wait(s_full(buf), buf_phase);
                const Elem* scales = reinterpret_cast<const Elem*>(scale_bufs + buf * kScaleBytes +
                                                                   row_in_tile * kScaleWords * 4) +
                                     ((row_first + uint32_t(ks0 * kGroups)) & 1u);
                const int stop = min(k_last, ks0 + kChunkStages);
                for (int ks = ks0; ok && ks < stop; ++ks) {
#pragma unroll 1
                    for (int g0 = 0; g0 < kGroups; g0 += kDGroups) {
                        float scale[kDGroups];
#pragma unroll
                        for (int g = 0; g < kDGroups; ++g)  // (0 behind the row's last group)
                            scale[g] = ks * kGroups + g0 + g < p.num_groups
                                           ? to_float(scales[(ks - ks0) * kGroups + g0 + g]) : 0.0f;
                        ok = warp_wait(d_full(d), d_phase);
                        if (!ok) break;
                        tc_fence_after_sync();
                        add_products<kMine, kDGroups, kN>(lane_base + kDBase + d * kDBufCols + mine0, scale, acc);
                        tc_fence_before_sync();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(d_empty(d));
                        if (++d == kDs) {
                            d = 0;
                            d_phase ^= 1u;
                        }
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(s_empty(buf));
                if (++buf == kScaleBufs) {
                    buf = 0;
                    buf_phase ^= 1u;
                }
            }
            if (p.splits == 1 && n < p.N && ok) {
                const int64_t t0 = int64_t(chunk) * kCols + mine0;
                Out* y = static_cast<Out*>(p.y) + t0 * p.N + n;
#pragma unroll
                for (int t = 0; t < kMine; t += 2) {
                    const float2 v = unpack2(acc[t / 2]);
                    if (t0 + t < p.T) y[int64_t(t) * p.N] = from_float<Out>(v.x / kUnit);
                    if (t0 + t + 1 < p.T) y[int64_t(t + 1) * p.N] = from_float<Out>(v.y / kUnit);
                }
            }
        }
    } else {
        // ------------------------------------------------------------ numbers
        const int team = (warp - kFirstTeamWarp) / kTeamWarps;
        const uint32_t a_tmem = lane_base + team * kABufCols;
        // The CTA's stages are numbered through all items; number i lies in ring place
        // i % kStages and belongs to team i % kTeams.
        uint32_t stage = 0, phase = 0, turn = 0, a_phase = 0, buf = 0, buf_phase = 0;
        bool ok = true;
        for (int item = first_item; ok && item < p.items; item += item_step) {
            const int n = item / p.chunks * kTileN + row_in_tile;
            const uint32_t row_first = uint32_t(n) * uint32_t(p.num_groups);  // (its low bits count)
            for (int ks = k_first; ok && ks < k_last; ++ks) {
                const int in_chunk = (ks - k_first) % kChunkStages;
                if (kZeros && in_chunk == 0) ok = warp_wait(s_full(buf), buf_phase);
                const uint8_t* zeros = scale_bufs + buf * kScaleBytes + kTileN * kScaleWords * 4 +
                                       row_in_tile * kZeroWords * 4;
                if (ok && turn == uint32_t(team)) {
                    uint32_t zero[kGroups];  // (the row's values lie behind the shift of its first word)
#pragma unroll
                    for (int g = 0; g < kGroups; ++g)
                        zero[g] = kZeros ? zeros[((row_first + uint32_t((ks - in_chunk) * kGroups)) & 3u) +
                                                 in_chunk * kGroups + g]
                                         : 8u;
                    ok = warp_wait(full_bar(stage), phase) && warp_wait(a_empty(team), a_phase ^ 1u);
                    if (!ok) break;
                    tc_fence_after_sync();  // the MMAs that read the buffer come before the stores
                    // 16-byte pieces of the row, swizzled by its place among eight
                    const uint32_t codes = stage0 + stage * kStageBytes + row_in_tile * 128 +
                                           ((row_in_tile & 7) << 4);
                    uint4 next = load_shared_v4(codes);
#pragma unroll
                    for (int g = 0; g < kGroups; ++g) {
                        const Numbers<Elem> minus(zero[g]);
#pragma unroll
                        for (int c = g * 8 / kGroups; c < (g + 1) * 8 / kGroups; ++c) {
                            const uint4 words = next;
                            next = load_shared_v4(codes ^ ((c < 7 ? c + 1 : 7) << 4));
                            uint32_t r[16];
                            numbers<Elem>(words, minus, r);
                            tmem_st16(a_tmem + c * 16, r);
                        }
                    }
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(a_full(team));
                        mbar_arrive(empty_bar(stage));
                    }
                    a_phase ^= 1u;
                }
                if (kZeros && (in_chunk == kChunkStages - 1 || ks + 1 == k_last)) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(s_empty(buf));
                    if (++buf == kScaleBufs) {
                        buf = 0;
                        buf_phase ^= 1u;
                    }
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++turn == kTeams) turn = 0;
            }
        }
    }

    if (p.splits > 1) {
        // Each CTA ends a share of the columns: sums of all parts, in the order of k, in
        // the place of the stages.
        float* parts = reinterpret_cast<float*>(smem);
        cluster_sync();  // no CTA uses its stages any more
        const int share = (kCols + p.splits - 1) / p.splits;
        if (warp >= kFirstProductWarp && warp < kFirstTeamWarp) {
#pragma unroll
            for (int t = 0; t < kMine; ++t) {
                const int owner = (mine0 + t) / share;
                const int place = rank * share + (mine0 + t - owner * share);
                const uint32_t to = mapa_shared(smem_u32(parts + place * kTileN + row_in_tile), owner);
                const float2 v = unpack2(acc[t / 2]);
                st_shared_cluster_u32(to, __float_as_uint(t & 1 ? v.y : v.x));
            }
        }
        cluster_sync();
        const int tile = first_item / p.chunks;
        const int chunk = first_item - tile * p.chunks;
        const int n = tile * kTileN + row_in_tile;
        if (warp >= kFirstProductWarp && n < p.N) {
            for (int i = (warp - kFirstProductWarp) / 4; i < share; i += kSets + kTeams) {
                const int64_t t = int64_t(chunk) * kCols + rank * share + i;
                if (rank * share + i >= kCols || t >= p.T) break;
                float sum = parts[i * kTileN + row_in_tile];
                for (int s = 1; s < p.splits; ++s)
                    sum += parts[(s * share + i) * kTileN + row_in_tile];
                static_cast<Out*>(p.y)[t * p.N + n] = from_float<Out>(sum / kUnit);
            }
        }
    }

    tc_fence_before_sync();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc<1>(tmem_base, kTmemCols);
    }
}

template <typename Elem, typename Out, int kCols, int kGroups, bool kZeros>
cudaError_t launch(const CUtensorMap& tw, const CUtensorMap& tx, const Args& p, int num_sms,
                   cudaStream_t stream) {
    auto kernel = linear_w4_kernel<Elem, Out, kCols, kGroups, kZeros>;
    constexpr size_t smem = smem_bytes(kCols, kGroups);
    static std::atomic<int> configured[64];  // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!configured[dev].load()) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
        if (e != cudaSuccess) return e;
        configured[dev].store(1);
    }
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(p.splits);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    const int64_t ctas = p.splits > 1 ? int64_t(p.items) * p.splits
                                      : (p.items < num_sms ? p.items : num_sms);
    cfg.gridDim = dim3(unsigned(ctas), 1, 1);
    cfg.blockDim = dim3(32 * (first_team_warp(kCols) + kTeamWarps * num_teams(kCols, kGroups)), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = p.splits > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, tw, tx, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

// (fp16 and bf16 are copied alike)
bool encode_maps(const uint32_t* codes, const void* x, int64_t T, int64_t N, int64_t K, int x_rows,
                 CUtensorMap* tw, CUtensorMap* tx) {
    return encode_tensor_map_2d(tw, codes, uint64_t(K / 2), uint64_t(N), uint64_t(K / 2),
                                kStageK / 2, kTileN, true) &&
           encode_tensor_map_2d(tx, x, uint64_t(K), uint64_t(T), uint64_t(K) * 2, 64,
                                uint32_t(x_rows), false);
}

// Rows of x per pass over the codes.
int columns(int64_t T) { return T <= 8 ? 8 : T <= 16 ? 16 : T <= 32 ? 32 : 64; }

template <typename Elem, typename Out, bool kZeros>
cudaError_t launch_cols(int cols, int groups, const CUtensorMap& tw, const CUtensorMap& tx,
                        const Args& p, int num_sms, cudaStream_t s) {
    auto go = [&](auto c) {
        constexpr int kCols = decltype(c)::value;
        if (groups == 2) return launch<Elem, Out, kCols, 2, kZeros>(tw, tx, p, num_sms, s);
        if (groups == 4) return launch<Elem, Out, kCols, 4, kZeros>(tw, tx, p, num_sms, s);
        if (groups == 8) return launch<Elem, Out, kCols, 8, kZeros>(tw, tx, p, num_sms, s);
        return cudaErrorInvalidValue;
    };
    if (cols == 8) return go(std::integral_constant<int, 8>());
    if (cols == 16) return go(std::integral_constant<int, 16>());
    if (cols == 32) return go(std::integral_constant<int, 32>());
    return go(std::integral_constant<int, 64>());
}

}  // namespace

cudaError_t launch_linear_w4(const void* x, ElemType type, const uint32_t* codes,
                             const void* scales, const uint8_t* zeros, int64_t T, int64_t N,
                             int64_t K, int group, void* y, ElemType y_type, int num_sms,
                             cudaStream_t stream) {
    const int groups = kStageK / group;  // per stage
    const int cols = columns(T);
    const int64_t tiles = (N + kTileN - 1) / kTileN;
    const int64_t chunks = (T + cols - 1) / cols;
    if (tiles * chunks * kMaxSplits > INT32_MAX) return cudaErrorInvalidValue;
    Args p = {scales, zeros, y, T, int(N), int((K + group - 1) / group), int(chunks),
              int(tiles * chunks), int((K + kStageK - 1) / kStageK), 1,
              int(T < mma_n(cols) ? T : mma_n(cols)), 0};
    p.splits = w4_parts_of_k(int(tiles), p.num_stages);
    CUtensorMap tw, tx;
    if (!encode_maps(codes, x, T, N, K, p.x_rows, &tw, &tx)) return cudaErrorInvalidValue;
    auto go = [&](auto elem, auto out) {
        using Elem = decltype(elem);
        using Out = decltype(out);
        return zeros ? launch_cols<Elem, Out, true>(cols, groups, tw, tx, p, num_sms, stream)
                     : launch_cols<Elem, Out, false>(cols, groups, tw, tx, p, num_sms, stream);
    };
    const bool wide = y_type == ElemType::kFp32;
    if (type == ElemType::kBf16)
        return wide ? go(__nv_bfloat16(), float()) : go(__nv_bfloat16(), __nv_bfloat16());
    return wide ? go(__half(), float()) : go(__half(), __half());
}

cudaError_t launch_linear_w4_stall_selftest(const void* x, const uint32_t* codes,
                                            const void* scales, float* y, int mode, int num_sms,
                                            cudaStream_t stream) {
    // one tile and four stages: all copies are issued before a wait can run out
    constexpr int64_t T = 1, N = kTileN, K = 4 * kStageK;
    constexpr int kCols = 8, kGroup = 128;
    static_assert(K / kStageK <= stages(kCols, kStageK / kGroup), "the ring holds every stage");
    const Args p = {scales, nullptr, y, T, int(N), int(K / kGroup), 1, 1, int(K / kStageK), 1, 1, mode};
    CUtensorMap tw, tx;
    if (!encode_maps(codes, x, T, N, K, p.x_rows, &tw, &tx)) return cudaErrorInvalidValue;
    return launch<__nv_bfloat16, float, kCols, kStageK / kGroup, false>(tw, tx, p, num_sms, stream);
}

cudaError_t linear_w4_take_error(unsigned int* out) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_w4_error, sizeof v);
    if (e != cudaSuccess) return e;
    if (v) e = cudaMemcpyToSymbol(g_w4_error, &zero, sizeof zero);
    *out = v;
    return e;
}

}  // namespace rlk
