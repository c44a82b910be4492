// rlk_int8_linear.cu -- y [T][N] = x [T][K] . W^T for both in 8-bit whole numbers (rlk_int8.cu):
//   y[t][n] = float(sum_k qx[t][k] qw[n][k]) * sx[t] * sw[n]
// with an exact sum.  This GPU's tensor cores have no product of 8-bit integers of their own, but
// 8-bit integers are exact in fp16 and so are their products in fp32, and a sum of 1024 of them
// stays within 2^24, where fp32 holds every whole number: so the codes run through
// tcgen05.mma kind::f16, and every 1024 k the fp32 sums go over into 32-bit integers.  No
// order of the sums can change a bit, so tiles and the cut of K are free.
//
// What bounds it: few rows of x, the codes of W, N K bytes read once; many rows, the 16-bit
// products.  x, small, is made fp16 by the quantiser before.  W's codes become fp16 in registers
// (5 instructions per 4 codes: the code's byte under the exponent of 1024, minus 1152) and go to
// tensor memory, from where they are the A operand, so shared memory carries one byte per code.
//
// One CTA per SM; a tile is 128 channels by up to 192 rows of x, its K goes by in stages of 128:
//   warp 0     TMA producer: the stage's codes (16 KB) and x
//   warp 1     MMA issuer: 8 MMAs per stage, accumulators for 1024 k, two of them
//   sets       of four warps, 64 columns each: a thread adds its channel's sums up in integers
//   teams      of four warps, which take the stages in turn: a thread turns its channel's codes
//              into numbers and stores them to one of two or four A buffers
// A team meets only every second or third stage, and a barrier tells two phases apart, not three: that
// the phase before the one it waits for is over must be known.  So it waits for its buffer first.
// That the MMAs of the stage that had the buffer before are done (stage i - buffers) says that all
// copies up to that stage's have come, and the ring place of stage i held no later one (i - stages).
//
// Few tiles: K is cut into parts, one per CTA of a cluster, whose integers meet through
// distributed shared memory.
//
// Every wait is bounded (2 s); on expiry the kernel records it, waits for its copies and
// products under way and returns.
//
// Why 192 rows at most: two accumulators and two buffers of numbers are tensor memory's 512 columns.
// A product of N columns takes about 60 + N/4 cycles here (A from tensor memory), so tiles are as
// wide as fit: 160 columns, with three buffers of numbers, were slower at T = 4096.
// Measured (codes rotated past L2; us), N = 151936, K = 4096: T = 1 94 (6.6 TB/s, 0.97 of a copy),
// 16 99, 32 101, 64 112-114, 128 143; N = 16384, K = 4096: T = 512 64, T = 4096 339 (1.62 PFLOP/s,
// 0.86 of the measured bf16 rate); N = K = 4096: T = 4096 104.  By dot products of codes on the CUDA
// cores: T = 1 196, T = 64 2149, T = 4096 21735.
#include <atomic>

#include "rlk_int8_plan.h"
#include "rlk_logits.cuh"
#include "rlk_ptx.cuh"
#include "rlk_train_int8.h"

namespace rlk {
namespace {

constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint64_t kDrainLimitNs = 200000000ull;

constexpr bool fits(int room) {
    return int8_smem_bytes(room) <= 227 * 1024 && int8_tmem_cols(room) <= int(kTmemCols) &&
           2 * (int8_stages(room) + int8_number_bufs(room) + 2) + 1 <= kInt8MaxBarriers &&
           (room + kInt8MaxParts) * kInt8TileN * 4 <= int8_stages(room) * int8_stage_bytes(room);
}
static_assert(fits(16) && fits(32) && fits(64) && fits(128) && fits(192), "memory per CTA");
// (see above; and for the buffers' own phases: a team's last buffer was freed by stage
// i - teams - buffers)
constexpr bool phases_known(int room) {
    return int8_stages(room) >= int8_number_bufs(room) && int8_number_bufs(room) >= int8_teams(room);
}
static_assert(phases_known(16) && phases_known(32) && phases_known(64) && phases_known(128) &&
                  phases_known(192),
              "a team's waits are for the next phase");

__device__ unsigned int g_int8_error;  // bit 0: a wait ran out; bit 1: a teardown wait ran out

struct Args {
    const float* x_scales;
    const float* scales;
    void* y;
    int64_t T;
    int N;
    Int8Plan plan;
    int items;           // tiles * chunks
    int stall_selftest;  // bounded-wait self-test: 1, the producer issues no copies; 2, the MMA
                         // issuer consumes no stage
};

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
                atomicOr(&g_int8_error, 1u);
                return false;
            }
        }
    }
}

__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity) {
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(bar, parity)) {
        if (global_timer_ns() - t0 > kDrainLimitNs) {
            atomicOr(&g_int8_error, 2u);
            return;
        }
    }
}

// Four codes as two pairs of fp16 numbers: byte b of (codes ^ 0x80) is the code plus 128, and
// 0x64 above it makes it the fp16 number 1024 + b; 1152 less is the code, exactly.
__device__ __forceinline__ void numbers(uint32_t codes, uint32_t& lo, uint32_t& hi) {
    const uint32_t u = codes ^ 0x80808080u;
    const uint32_t less = 0x64806480u;
    auto sub = [&](uint32_t a) {
        const __half2 d = __hsub2(*reinterpret_cast<const __half2*>(&a),
                                  *reinterpret_cast<const __half2*>(&less));
        return *reinterpret_cast<const uint32_t*>(&d);
    };
    lo = sub(__byte_perm(u, 0x64646464u, 0x4140));
    hi = sub(__byte_perm(u, 0x64646464u, 0x4342));
}

template <typename Out, int kRoom>
__global__ void __launch_bounds__(32 * int8_warps(kRoom), 1)
    linear_int8_kernel(const __grid_constant__ CUtensorMap tmap_w,
                       const __grid_constant__ CUtensorMap tmap_x, const Args p) {
    constexpr int kStages = int8_stages(kRoom);
    constexpr int kStageBytes = int8_stage_bytes(kRoom);
    constexpr int kTeams = int8_teams(kRoom), kSets = int8_sets(kRoom);
    constexpr int kBufs = int8_number_bufs(kRoom);
    constexpr uint32_t kNumberCols = kInt8NumberCols;
    constexpr int kMine = kRoom / kSets;  // columns of a set
    constexpr int kLaneRows = (kMine + 31) / 32;
    constexpr int kPiece = kSets > 1 ? 8 : 16;  // (registers)
    constexpr int kFirstTeamWarp = 2 + 4 * kSets;
    constexpr uint32_t kDBase = kBufs * kNumberCols;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    const uint32_t pad = (1024u - (raw_addr & 1023u)) & 1023u;
    uint8_t* smem = smem_raw + pad;
    const uint32_t stage0 = raw_addr + pad;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + size_t(kStages) * kStageBytes);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kInt8MaxBarriers);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const uint32_t bar0 = smem_u32(bars);
    constexpr int kA = 2 * kStages, kD = kA + 2 * kBufs;
    auto full_bar = [&](uint32_t s) { return bar0 + 8 * s; };
    auto empty_bar = [&](uint32_t s) { return bar0 + 8 * (kStages + s); };
    auto a_full = [&](uint32_t buf) { return bar0 + 8 * (kA + buf); };
    auto a_empty = [&](uint32_t buf) { return bar0 + 8 * (kA + kBufs + buf); };
    auto d_full = [&](uint32_t d) { return bar0 + 8 * (kD + d); };
    auto d_empty = [&](uint32_t d) { return bar0 + 8 * (kD + 2 + d); };
    const uint32_t drain_bar = bar0 + 8 * (kD + 4);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 4 + 1);  // the codes' readers, and the MMAs
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(a_full(i), 4);
            mbar_init(a_empty(i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(d_full(i), 1);
            mbar_init(d_empty(i), 4 * kSets);
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

    // A cluster takes one item, a CTA alone every gridDim.x-th; either way these stages of K.
    const Int8Plan& plan = p.plan;
    // (from blockIdx: the compiler then knows that all that follows is the same in a warp, which the
    // issue of MMAs needs to be quick)
    const int rank = int(blockIdx.x) % plan.parts;
    const int first_item = plan.parts > 1 ? int(blockIdx.x) / plan.parts : int(blockIdx.x);
    const int item_step = plan.parts > 1 ? p.items : int(gridDim.x);
    const int k_first = int(int64_t(plan.stages) * rank / plan.parts);
    const int k_last = int(int64_t(plan.stages) * (rank + 1) / plan.parts);

    grid_dependency_wait();
    grid_launch_dependents();

    const int row_in_tile = (warp & 3) * 32 + lane;  // (a warp reaches the lanes of its quadrant)
    const uint32_t lane_base = tmem_base + (uint32_t((warp & 3) * 32) << 16);
    int sum[kMine];  // of the sets' warps: columns mine0 ..
    const int mine0 = (warp - 2) / 4 * kMine;

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
                const int tile = item / plan.chunks;
                const int chunk = item - tile * plan.chunks;
                for (int ks = k_first; ks < k_last; ++ks) {
                    if (!wait_bounded(empty_bar(stage), phase ^ 1u, abort_flag)) {
                        ok = false;
                        break;
                    }
                    const uint32_t at = stage0 + stage * kStageBytes;
                    mbar_arrive_expect_tx(full_bar(stage), kInt8CodeBytes +
                                                               uint32_t(plan.rows) * kInt8StageK * 2);
                    tma_load_2d(&tmap_w, full_bar(stage), at, ks * kInt8StageK, tile * kInt8TileN);
#pragma unroll
                    for (int i = 0; i < kInt8StageK / 64; ++i)
                        tma_load_2d(&tmap_x, full_bar(stage), at + kInt8CodeBytes + i * kRoom * 128,
                                    ks * kInt8StageK + i * 64, chunk * plan.rows);
                    ++issued;
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            // The copies this thread started land before the CTA exits, whichever role gave up.
            for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i) {
                const uint32_t bar = full_bar(i % kStages), parity = uint32_t(i / kStages) & 1u;
                if (!wait_bounded(bar, parity, abort_flag)) wait_drain(bar, parity);
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issuer
        // (the whole warp runs the loop and one lane issues: addresses from outside that lane's branch
        // are warp-uniform, as the instructions want them)
        const bool leader = elect_one();
        const uint32_t idesc = idesc_f16_f32(kInt8TileN, plan.mma_n);
        uint32_t stage = 0, phase = 0, buf = 0, buf_phase = 0, d = 0, d_phase = 0;
        bool ok = true;
        const int items = p.stall_selftest == 2 ? 0 : p.items;
        for (int item = first_item; ok && item < items; item += item_step) {
            for (int ks = k_first; ks < k_last; ++ks) {
                const bool opens = (ks - k_first) % kInt8SumStages == 0;
                const bool closes = (ks - k_first) % kInt8SumStages == kInt8SumStages - 1 || ks + 1 == k_last;
                ok = warp_wait(full_bar(stage), phase) && warp_wait(a_full(buf), buf_phase) &&
                     (!opens || warp_wait(d_empty(d), d_phase ^ 1u));
                if (!ok) break;
                tc_fence_after_sync();
                const uint64_t x_desc =
                    sw128_kmajor_desc(stage0 + stage * kStageBytes + kInt8CodeBytes);
                const uint32_t a_tmem = tmem_base + buf * kNumberCols;
                const uint32_t d_tmem = tmem_base + kDBase + d * kRoom;
                const uint32_t a_done = a_empty(buf), stage_done = empty_bar(stage), d_done = d_full(d);
                const uint32_t more = opens ? 0u : 1u;
                if (leader) {
#pragma unroll
                    for (int i = 0; i < kInt8StageK / 16; ++i)
                        umma_f16_tmem_a(d_tmem, a_tmem + i * 8,
                                        x_desc + uint64_t((i / 4 * kRoom * 128 + i % 4 * 32) >> 4),
                                        idesc, i == 0 ? more : 1u);
                    umma_commit(a_done);
                    umma_commit(stage_done);
                    if (closes) umma_commit(d_done);
                }
                __syncwarp();
                if (++buf == kBufs) {
                    buf = 0;
                    buf_phase ^= 1u;
                }
                if (closes && ++d == 2) {
                    d = 0;
                    d_phase ^= 1u;
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
            }
        }
        if (leader) {
            umma_commit(drain_bar);  // no MMA may still run when TMEM is freed
            wait_drain(drain_bar, 0);
        }
        __syncwarp();
    } else if (warp < kFirstTeamWarp) {
        // ------------------------------------------------------------ sums
        uint32_t d = 0, d_phase = 0;
        bool ok = true;
        for (int item = first_item; ok && item < p.items; item += item_step) {
            const int tile = item / plan.chunks;
            const int chunk = item - tile * plan.chunks;
            const int n = tile * kInt8TileN + row_in_tile;
            const int first = chunk * plan.rows + mine0;
            const int rows = int(min(int64_t(plan.rows), p.T - chunk * plan.rows)) - mine0;  // mine
            // the scales that the stores will want, a lane one of every 32 rows'
            float scale = 0.0f, x_scale[kLaneRows];
            if (plan.parts == 1) {
                scale = n < p.N ? __ldg(p.scales + n) : 0.0f;
#pragma unroll
                for (int j = 0; j < kLaneRows; ++j)
                    x_scale[j] = 32 * j + lane < rows ? __ldg(p.x_scales + first + 32 * j + lane) : 0.0f;
            }
#pragma unroll
            for (int t = 0; t < kMine; ++t) sum[t] = 0;
            for (int ks = k_first; ks < k_last; ks += kInt8SumStages) {
                ok = warp_wait(d_full(d), d_phase);
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t at = lane_base + kDBase + d * kRoom + mine0;
#pragma unroll
                for (int c = 0; c < kMine; c += kPiece) {
                    uint32_t r[kPiece];
                    if constexpr (kPiece == 8)
                        tmem_ld8(at + c, r);
                    else
                        tmem_ld16(at + c, r);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < kPiece; ++j) sum[c + j] += __float2int_rn(__uint_as_float(r[j]));
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(d_empty(d));
                if (++d == 2) {
                    d = 0;
                    d_phase ^= 1u;
                }
            }
            if (plan.parts == 1 && ok) {
                // (stores one after the other, without a load or a branch between: the next item's
                // sums wait for them)
                Out* y = static_cast<Out*>(p.y) + int64_t(first) * p.N + n;
                const bool there = n < p.N;
#pragma unroll
                for (int t = 0; t < kMine; ++t) {
                    const float xs = __shfl_sync(0xffffffffu, x_scale[t / 32], t % 32);
                    if (there && t < rows) *y = from_float<Out>(__fmul_rn(__fmul_rn(float(sum[t]), xs), scale));
                    y += p.N;
                }
            }
        }
    } else {
        // ------------------------------------------------------------ numbers
        const uint32_t team = uint32_t(warp - kFirstTeamWarp) / 4;
        // The CTA's stages are numbered through all items; number i lies in ring place i % kStages,
        // belongs to team i % kTeams and goes to buffer i % kBufs.
        uint32_t stage = 0, phase = 0, turn = 0, buf = 0, buf_phase = 0;
        bool ok = true;
        for (int item = first_item; ok && item < p.items; item += item_step) {
            for (int ks = k_first; ks < k_last; ++ks) {
                if (turn == team) {
                    // (the buffer first: see the top)
                    ok = warp_wait(a_empty(buf), buf_phase ^ 1u) && warp_wait(full_bar(stage), phase);
                    if (!ok) break;
                    // 16-byte pieces of the row, swizzled by its place among eight
                    const uint32_t codes = stage0 + stage * kStageBytes + row_in_tile * 128 +
                                           ((row_in_tile & 7) << 4);
                    const uint32_t a_tmem = lane_base + buf * kNumberCols;
                    tc_fence_after_sync();  // the MMAs that read the buffer come before the stores
#pragma unroll
                    for (int c = 0; c < 8; c += 2) {
                        const uint4 v[2] = {load_shared_v4(codes ^ (c << 4)),
                                            load_shared_v4(codes ^ ((c + 1) << 4))};
                        uint32_t r[16];
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            numbers(v[i].x, r[8 * i], r[8 * i + 1]);
                            numbers(v[i].y, r[8 * i + 2], r[8 * i + 3]);
                            numbers(v[i].z, r[8 * i + 4], r[8 * i + 5]);
                            numbers(v[i].w, r[8 * i + 6], r[8 * i + 7]);
                        }
                        tmem_st16(a_tmem + c * 8, r);
                    }
                    tmem_st_wait();
                    tc_fence_before_sync();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(a_full(buf));
                        mbar_arrive(empty_bar(stage));
                    }
                }
                if (++stage == kStages) {
                    stage = 0;
                    phase ^= 1u;
                }
                if (++buf == kBufs) {
                    buf = 0;
                    buf_phase ^= 1u;
                }
                if (++turn == kTeams) turn = 0;
            }
        }
    }

    if (plan.parts > 1) {
        // Each CTA ends a share of the columns: the integers of all parts, in the place of the
        // stages.
        int* sums = reinterpret_cast<int*>(smem);
        cluster_sync();  // no CTA uses its stages any more
        const int share = (kRoom + plan.parts - 1) / plan.parts;
        if (warp >= 2 && warp < kFirstTeamWarp) {
#pragma unroll
            for (int t = 0; t < kMine; ++t) {
                const int owner = (mine0 + t) / share;
                const int place = rank * share + (mine0 + t - owner * share);
                st_shared_cluster_u32(
                    mapa_shared(smem_u32(sums + place * kInt8TileN + row_in_tile), owner),
                    uint32_t(sum[t]));
            }
        }
        cluster_sync();
        const int tile = first_item / plan.chunks;
        const int chunk = first_item - tile * plan.chunks;
        const int n = tile * kInt8TileN + row_in_tile;
        if (warp >= 2 && n < p.N) {
            const float s = __ldg(p.scales + n);
            for (int i = (warp - 2) / 4; i < share; i += kSets + kTeams) {
                const int column = rank * share + i;
                const int64_t t = int64_t(chunk) * plan.rows + column;
                if (column >= plan.rows || t >= p.T) break;
                int total = sums[i * kInt8TileN + row_in_tile];
                for (int part = 1; part < plan.parts; ++part)
                    total += sums[(part * share + i) * kInt8TileN + row_in_tile];
                static_cast<Out*>(p.y)[t * p.N + n] =
                    from_float<Out>(__fmul_rn(__fmul_rn(float(total), __ldg(p.x_scales + t)), s));
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

// The kernels of an output type may have their shared memory: set for every room by the type's first call
// on a device, whichever room it takes (a call in a graph's capture then meets no kernel for the first time).
template <typename Out>
cudaError_t configure() {
    static std::atomic<int> configured[64];  // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (configured[dev].load()) return cudaSuccess;
    auto allow = [&](auto kernel, int room) {
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     int(int8_smem_bytes(room)));
    };
    allow(linear_int8_kernel<Out, 16>, 16);
    allow(linear_int8_kernel<Out, 32>, 32);
    allow(linear_int8_kernel<Out, 64>, 64);
    allow(linear_int8_kernel<Out, 128>, 128);
    allow(linear_int8_kernel<Out, 192>, 192);
    if (e == cudaSuccess) configured[dev].store(1);
    return e;
}

template <typename Out, int kRoom>
cudaError_t launch(const CUtensorMap& tw, const CUtensorMap& tx, const Args& p, int num_sms,
                   cudaStream_t stream) {
    auto kernel = linear_int8_kernel<Out, kRoom>;
    constexpr size_t smem = int8_smem_bytes(kRoom);
    cudaError_t e = configure<Out>();
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = unsigned(p.plan.parts);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    const int64_t ctas = p.plan.parts > 1 ? int64_t(p.items) * p.plan.parts
                                          : (p.items < num_sms ? p.items : num_sms);
    cfg.gridDim = dim3(unsigned(ctas), 1, 1);
    cfg.blockDim = dim3(32 * int8_warps(kRoom), 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = p.plan.parts > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, kernel, tw, tx, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

template <typename Out>
cudaError_t launch_room(const CUtensorMap& tw, const CUtensorMap& tx, const Args& p, int num_sms,
                        cudaStream_t s) {
    switch (p.plan.room) {
        case 16: return launch<Out, 16>(tw, tx, p, num_sms, s);
        case 32: return launch<Out, 32>(tw, tx, p, num_sms, s);
        case 64: return launch<Out, 64>(tw, tx, p, num_sms, s);
        case 128: return launch<Out, 128>(tw, tx, p, num_sms, s);
        default: return launch<Out, 192>(tw, tx, p, num_sms, s);
    }
}

// (fp16 and bf16 are copied alike)
bool encode_maps(const int8_t* codes, const void* x, int64_t T, int64_t N, int64_t K, int x_rows,
                 CUtensorMap* tw, CUtensorMap* tx) {
    return encode_tensor_map_2d(tw, codes, uint64_t(K), uint64_t(N), uint64_t(K), kInt8StageK,
                                kInt8TileN, true) &&
           encode_tensor_map_2d(tx, x, uint64_t(K), uint64_t(T), uint64_t(K) * 2, 64,
                                uint32_t(x_rows), false);
}

}  // namespace

cudaError_t launch_linear_int8(const void* x_fp16, const float* x_scales, const int8_t* codes,
                               const float* scales, int64_t T, int64_t N, int64_t K, void* y,
                               ElemType y_type, int num_sms, cudaStream_t stream) {
    if ((N + kInt8TileN - 1) / kInt8TileN * ((T + 191) / 192) * kInt8MaxParts > INT32_MAX)
        return cudaErrorInvalidValue;
    Args p = {x_scales, scales, y, T, int(N), int8_plan(T, N, K, num_sms), 0, 0};
    p.items = p.plan.tiles * p.plan.chunks;
    CUtensorMap tw, tx;
    if (!encode_maps(codes, x_fp16, T, N, K, p.plan.rows, &tw, &tx)) return cudaErrorInvalidValue;
    if (y_type == ElemType::kBf16) return launch_room<__nv_bfloat16>(tw, tx, p, num_sms, stream);
    if (y_type == ElemType::kFp16) return launch_room<__half>(tw, tx, p, num_sms, stream);
    return launch_room<float>(tw, tx, p, num_sms, stream);
}

cudaError_t launch_linear_int8_stall_selftest(const void* x_fp16, const float* x_scales,
                                              const int8_t* codes, const float* scales, float* y,
                                              int mode, int num_sms, cudaStream_t stream) {
    // one tile and four stages: all copies are issued before a wait can run out
    constexpr int64_t T = 1, N = kInt8TileN, K = 4 * kInt8StageK;
    static_assert(K / kInt8StageK <= int8_stages(16), "the ring holds every stage");
    Args p = {x_scales, scales, y, T, int(N), int8_plan(T, N, K, num_sms), 1, mode};
    p.plan.parts = 1;
    CUtensorMap tw, tx;
    if (!encode_maps(codes, x_fp16, T, N, K, p.plan.rows, &tw, &tx)) return cudaErrorInvalidValue;
    return launch<float, 16>(tw, tx, p, num_sms, stream);
}

cudaError_t linear_int8_take_error(unsigned int* out) {
    unsigned int v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_int8_error, sizeof v);
    if (e != cudaSuccess) return e;
    if (v) e = cudaMemcpyToSymbol(g_int8_error, &zero, sizeof zero);
    *out = v;
    return e;
}

}  // namespace rlk
