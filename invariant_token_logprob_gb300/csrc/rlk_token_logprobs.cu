// rlk_token_logprobs.cu -- log probabilities of given tokens from logits, with
// the log-sum-exp, the entropy and the top alternatives, and their gradient.
//
// Per row, with z = x * inv_temp over the tokens that are allowed and above -inf:
//   m = max z, S = sum exp(z - m), U = sum exp(z - m) (z - m)
//   lse = m + log S, entropy = log S - U / S, logp = z[target] - lse
// and the gradient of those outputs with respect to x (p = exp(z - lse)):
//   dx[v] = inv_temp * ( p[v] (g_lse - G - g_H (z[v] - lse + H))
//                        + [v == target] g_logp + sum_j [v == id_j] g_top_j ),
//   G = g_logp + sum_j g_top_j
//
// Forward: one pass over the row and one launch.  A row is dealt to 64 strips of 32
// lanes: lane l of strip s takes the eight elements from 256 s + 8 l on, and those
// 16384, 2 * 16384, ... behind, and keeps a reference and the two sums about it.  A
// strip is read by one warp.  The 64 x 32 partial sums meet in one binary tree, strips
// first (inside a block of eight, then the blocks), lanes last.  Strips, lanes and tree
// follow from V alone, so a row's bits depend on that row only, while the launch is free
// to give a row to one CTA (many rows) or to a cluster of two, four or eight (few rows).
//
// Alternatives: what one lane of one strip reads is a cell, and its maximum is known
// anyway.  Order tokens by (larger logit, lower index) and cells by (larger maximum,
// lower place of it).  If K cells reach a bound, the top K tokens lie in cells that
// reach it and reach it themselves: a token below it would have K tokens before it, one
// in each of those cells.  So after the pass a bound is taken from the warps' best
// cells, the cells that reach it (some tens of 2048) are read again, and their tokens
// that reach it, hardly more, are ranked by counting.
//
// The pass is bound by the reads of the logits where rows are many (T = 4096, V = 151936,
// bf16: 206 us, 6.0 TB/s; with 20 alternatives 249 us; T = 1024, fp32: 95 us, 6.6 TB/s),
// by the latency of its steps where they are few (T = 1, fp32, 20 alternatives: 8.4 us).
// The gradient reads and writes each logit once (T = 4096, bf16: 361 us, 6.9 TB/s).
#include <float.h>
#include <limits.h>

#include <atomic>

#include "rlk_logits.cuh"
#include "rlk_logits_w4.h"
#include "rlk_lse.cuh"
#include "rlk_ptx.cuh"

namespace rlk {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kStrips = 64;             // of a row: kBlocks blocks of kWarps
constexpr int kBlocks = kStrips / kWarps;  // also the largest cluster
constexpr int kGroup = 8;               // neighbouring elements per lane
constexpr int kStep = 32 * kGroup;      // elements of a strip side by side
constexpr int kStride = kStrips * kStep;  // from a lane's group to its next one
constexpr int kCells = kStrips * 32;
constexpr uint32_t kNoStrip = uint32_t(INT_MAX) / kStep + 1;
constexpr float kLn2 = 0.6931471805599453f;

// Rows whose target was >= V, counted since the last read on this device.
__device__ unsigned long long g_range_rows;

__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Sums about a reference m (a raw logit; -FLT_MAX, the identity, before any token), in
// units of log 2: t = (x - m) * inv_temp * log2 e, s = sum 2^t, u = sum 2^t t.
struct Sums {
    float m, s, u;
};

// Far below: where 2^t is 0, t is cut off there so that 0 * t is 0.  kFar cuts the
// step between two references, which multiplies a whole sum.
constexpr float kFarBelow = -200.0f;
constexpr float kFar = -1e30f;

__device__ __forceinline__ Sums combine(Sums a, Sums b, float c2) {
    const float m = fmaxf(a.m, b.m);
    const float da = max_nan((a.m - m) * c2, kFar), db = max_nan((b.m - m) * c2, kFar);
    const float ea = ex2(da), eb = ex2(db);
    Sums r;
    r.m = m;
    r.s = fmaf(a.s, ea, b.s * eb);
    r.u = fmaf(ea, fmaf(da, a.s, a.u), eb * fmaf(db, b.s, b.u));
    return r;
}

// Orders fp32 values as unsigned integers (larger value, larger integer; the zeros are
// equal; 0 is below every value).
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
    return __uint_as_float((k >> 31) ? (k & 0x7fffffffu) : ~k);
}
// (value, place): larger value first, lower place first among equals; 0 is none.
__device__ __forceinline__ uint64_t order_key(float x, uint32_t place) {
    return (uint64_t(ordered(x)) << 32) | (~place);
}
__device__ __forceinline__ uint32_t key_place(uint64_t k) { return ~uint32_t(k); }

constexpr int kCellList = 256;   // cells read again
constexpr int kTokenList = 512;  // tokens ranked by counting
constexpr int kGroupsAtOnce = 2 * kThreads;  // groups of cells looked through together

struct Shared {
    uint64_t cells[kCells];              // the CTA's cells; 0: no token
    Sums strip_sums[kBlocks][kWarps][32];
    Sums block_sums[kBlocks][32];        // rank 0: of the whole row
    uint64_t cell_list[kCellList];
    uint32_t group_list[kGroupsAtOnce];
    uint64_t chosen[kMaxTopK];           // the CTA's, then the row's best tokens
    uint32_t warp_bound[kWarps];
    Sums row;
    int count, tokens, groups;

    // Tokens to rank, in the cells' place once the list of cells is complete.
    __device__ __forceinline__ uint64_t* token_list() { return cells; }
    // Rank 0: the best tokens of every CTA, in the place of a block of strip sums that only
    // a CTA without a cluster has.
    __device__ __forceinline__ uint64_t* gathered() {
        return reinterpret_cast<uint64_t*>(strip_sums[kBlocks - 1]);
    }
};
static_assert(sizeof(Shared) <= 48 * 1024, "no opt-in for shared memory");
static_assert(kBlocks * kMaxTopK * 8 <= sizeof(Sums) * kWarps * 32, "one block of strip sums");
static_assert(kTokenList <= kCells && kCellList >= kMaxTopK && kTokenList % 4 == 0, "lists");

struct Args {
    const void* logits;
    int64_t row_stride;
    const int32_t* targets;
    const uint32_t* allowed;
    int64_t allowed_stride;
    int V, top_k;
    float inv_temp;
    float *out_logp, *out_lse, *out_entropy, *out_top;
    int32_t* out_ids;
};

// Adds eight elements to the sums about m.  kCut: elements at -inf may be among them
// (0 * -inf must not reach u).
template <bool kCut, typename Elem>
__device__ __forceinline__ void add_eight(const Packed8<Elem>& x, F2 low, F2 scale, F2& s, F2& u) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const float2 xx = x.pair(j);
        F2 t = mul2(add2(pack2(xx.x, xx.y), low), scale);
        float2 f = unpack2(t);
        if (kCut) {
            f = make_float2(max_nan(f.x, kFarBelow), max_nan(f.y, kFarBelow));
            t = pack2(f.x, f.y);
        }
        const F2 p = pack2(ex2(f.x), ex2(f.y));
        s = add2(s, p);
        u = fma2(p, t, u);
    }
}

// The running state of one lane of one strip.  The reference m is the maximum of the
// first unit of groups with a token; it moves on only where a later unit's maximum lies
// more than kLead above it (2^kLead times the elements stay far inside fp32), so that the
// usual unit has no step between references.
constexpr float kLead = 8.0f;

struct LaneState {
    float top, m;
    uint32_t place;
    F2 s, u;

    // Looks at a unit of N groups, the first one `group` of the row, kStride apart.
    template <int N, typename Elem>
    __device__ __forceinline__ void look(const Packed8<Elem>* x, uint32_t group, float c2) {
        float most = -INFINITY;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float g = x[i].max();
            if (g > top) {
                top = g;
                place = group + i * (kStride / kGroup);
            }
            most = fmaxf(most, g);
        }
        if ((most - m) * c2 > kLead) {
            const float d = max_nan((m - most) * c2, kFar);
            const float f = ex2(d);
            const F2 ff = pack2(f, f), dd = pack2(d, d);
            u = mul2(ff, fma2(dd, s, u));
            s = mul2(ff, s);
            m = most;
        }
    }
    // Adds them.  summed(k) follows the k-th group; again(group) loads one that holds an
    // element at -inf, which is cut then.
    template <bool kCut, typename Elem, int N, typename Summed, typename Again>
    __device__ __forceinline__ void add(const Packed8<Elem> (&x)[N], uint32_t group, float c2,
                                        Summed&& summed, Again&& again) {
        look<N>(x, group, c2);
        const F2 low = pack2(-m, -m), scale = pack2(c2, c2);
        F2 us = pack2(0.0f, 0.0f), uu = us;
#pragma unroll
        for (int k = 0; k < N; ++k) {
            add_eight<kCut>(x[k], low, scale, us, uu);
            summed(k);
        }
        if (!kCut && !finite(uu)) {
            us = uu = pack2(0.0f, 0.0f);
#pragma unroll 1
            for (int k = 0; k < N; ++k)
                add_eight<true>(again(group + k * (kStride / kGroup)), low, scale, us, uu);
        }
        s = add2(s, us);
        u = add2(u, uu);
    }
    // False where an element at -inf (or a NaN) was added without a cut.
    static __device__ __forceinline__ bool finite(F2 uu) {
        const float2 test = unpack2(uu);
        return test.x + test.y == test.x + test.y;
    }
};

// How a strip's groups are taken: rows of 32 groups (one per lane, kStride apart) in units of
// kUnitOf<Elem> rows as long as they lie whole in the row, what is left of the whole ones one
// at a time, and then the row's end.  It follows from V and the type alone (a unit's maximum
// decides the rounding), not from the row's alignment.
template <typename Elem>
constexpr int kUnitOf = 8 / int(sizeof(Elem));  // 64 bytes per lane; bf16, T = 4096,
                                                // V = 151936: 205 us, with 32 bytes 240 us

struct StripPlan {
    uint32_t base;   // the strip's first element
    uint32_t whole;  // rows of groups whose vectors, and the longest shift, lie in the row
    __device__ __forceinline__ StripPlan(uint32_t strip, uint32_t V)
        : base(strip * kStep),
          whole(base + kStep + kGroup <= V ? (V - base - kStep - kGroup) / kStride + 1 : 0) {}
};

// The loads of one unit (or of the whole rows left behind the last one), under way from load()
// until take() gives their elements.  Rows at 16-byte boundaries wait in registers.
template <typename Elem, bool kShifted, bool kMasked>
struct Unit {
    static constexpr int N = kUnitOf<Elem>;
    Vectors<Elem, false> in[N];
    uint32_t b[N];
    // Row first + k of the strip, if it is whole.
    __device__ __forceinline__ void load(int k, const Elem* row, const uint8_t* bits, int lane,
                                         const StripPlan& plan, uint32_t first) {
        if (first + k >= plan.whole) return;
        const uint32_t e = plan.base + lane * kGroup + (first + k) * kStride;
        in[k].load(row, e, 0);
        if (kMasked) b[k] = bits[e / kGroup];
    }
};

// Shifted rows wait in the warp's slots in shared memory: a second vector per lane would make
// their loads too many registers (T = 4096, V = 151935, bf16: 262 us; in registers 294 us, and
// 443 us with spills at four CTAs per SM).  The lanes copy the strip's vectors and lane 0 the
// one behind it; each then reads those that cover its elements.
template <typename Elem, bool kMasked>
struct Unit<Elem, true, kMasked> {
    static constexpr int N = kUnitOf<Elem>;
    static constexpr int kOwn = kGroup / kVecElems<Elem>;    // vectors of a lane
    static constexpr int kVecs = 32 * kOwn + 1;              // of a row of groups
    uint4* slots;
    uint32_t b[N];
    __device__ __forceinline__ Unit(uint4* ring, int warp) : slots(ring + warp * (N * kVecs)) {}
    __device__ __forceinline__ void load(const Elem* row, const uint8_t* bits, int shift, int lane,
                                         const StripPlan& plan, uint32_t first) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            if (first + k >= plan.whole) break;
            const uint32_t e = plan.base + (first + k) * kStride;
            const uint4* from = reinterpret_cast<const uint4*>(row + e - shift);
            const uint32_t to = smem_u32(slots + k * kVecs);
#pragma unroll
            for (int i = 0; i < kOwn; ++i) {
                // (the row's first vector may begin in front of the tensor)
                const int v = i * 32 + lane;
                if (e + v > 0) copy_vector_async(to + v * 16, from + v);
            }
            if (lane == 0) copy_vector_async(to + 32 * kOwn * 16, from + 32 * kOwn);
            if (kMasked) b[k] = bits[e / kGroup + lane];
        }
    }
    template <int M>
    __device__ __forceinline__ void take(Packed8<Elem> (&x)[M], uint32_t first, int shift, int lane) {
        copy_words_wait_all();
        __syncwarp();
        Vectors<Elem, true> in[M];
#pragma unroll
        for (int k = 0; k < M; ++k)
#pragma unroll
            for (int i = 0; i <= kOwn; ++i) in[k].v[i] = slots[(first + k) * kVecs + lane * kOwn + i];
        unshift(in, shift, x);
        __syncwarp();  // the slots may be loaded again
    }
};

// The eight elements from e0 on, wherever they lie in the row.
template <typename Elem, bool kShifted>
__device__ __forceinline__ Packed8<Elem> load_group(const Elem* row, int64_t e0, int shift, int64_t V) {
    Packed8<Elem> x[1];
    if (Vectors<Elem, kShifted>::inside(e0, shift, V)) {
        Vectors<Elem, kShifted> in[1];
        in[0].load(row, e0, shift);
        unshift(in, shift, x);
    } else {
        x[0].load_single(row, e0, V);
    }
    return x[0];
}

// One strip's lane: its sums, and its cell's key.  `unit` holds the loads of its first unit,
// on return those of the next strip's.
template <typename Elem, bool kShifted, bool kMasked>
__device__ __forceinline__ Sums read_strip(const Elem* row, int shift, const uint8_t* bits,
                                           uint32_t V, const StripPlan& plan, const StripPlan& next,
                                           Unit<Elem, kShifted, kMasked>& unit, int lane, float c2,
                                           uint64_t* cell) {
    constexpr int N = kUnitOf<Elem>;
    constexpr uint32_t kRow = kStride / kGroup;
    LaneState st = {-INFINITY, -FLT_MAX, 0u, pack2(0.0f, 0.0f), pack2(0.0f, 0.0f)};
    const uint32_t group = (plan.base + lane * kGroup) / kGroup;
    // The unit's groups from the k-th on, which is row i + k; `last`: loads what comes next.
    auto take = [&](auto& x, uint32_t i, auto k, bool last, bool more) {
        constexpr int K = decltype(k)::value, M = sizeof(x) / sizeof(x[0]);
        if constexpr (kShifted) {
            unit.take(x, K, shift, lane);
            if (group + i + K == 0) x[0].load_single(row, 0, V);
        } else {
#pragma unroll
            for (int j = 0; j < M; ++j) unit.in[K + j].template get<0>(x[j]);
        }
        if (kMasked) {
#pragma unroll
            for (int j = 0; j < M; ++j) x[j].keep(unit.b[K + j]);
        }
        if constexpr (kShifted) {
            if (last) unit.load(row, bits, shift, lane, more ? plan : next, more ? i + N : 0);
        }
    };
    constexpr std::integral_constant<int, 0> k0;
    constexpr std::integral_constant<int, (N > 2 ? 2 : 0)> k2;
    auto again = [&](uint32_t g) {
        return load_group<Elem, kShifted>(row, int64_t(g) * kGroup, shift, V);
    };
    uint32_t i = 0;
    for (; i + N <= plan.whole; i += N) {
        const bool more = i + N < plan.whole;
        Packed8<Elem> x[N];
        take(x, i, k0, true, more);
        st.template add<kMasked>(x, group + i * kRow, c2, [&](int k) {
            // (a group's registers take the next unit's loads once it is summed)
            if constexpr (!kShifted) {
                if (more)
                    unit.load(k, row, bits, lane, plan, i + N);
                else
                    unit.load(k, row, bits, lane, next, 0);
            }
        }, again);
    }
    // What is left of the whole rows, and the next strip's first unit.
    const uint32_t left = plan.whole - i;
    if (left > 0) {
        if (N > 2 && left >= 2) {
            Packed8<Elem> x[2];
            take(x, i, k0, left == 2, false);
            st.template add<kMasked>(x, group + i * kRow, c2, [](int) {}, again);
        }
        if (left % 2 != 0) {
            Packed8<Elem> x[1];
            if (left > 1)
                take(x, i, k2, true, false);
            else
                take(x, i, k0, true, false);
            st.template add<kMasked>(x, group + (plan.whole - 1) * kRow, c2, [](int) {}, again);
        }
        if constexpr (!kShifted) {
#pragma unroll
            for (int k = 0; k < N; ++k) unit.load(k, row, bits, lane, next, 0);
        }
    }
    for (i = plan.whole; int64_t(plan.base) + int64_t(i) * kStride < V; ++i) {  // the row's end
        const int64_t e0 = (int64_t(group) + i * kRow) * kGroup;
        Packed8<Elem> x = load_group<Elem, kShifted>(row, e0, shift, V);
        if (kMasked) x.keep(e0 < V ? bits[e0 / kGroup] : 0u);
        Packed8<Elem> one[1] = {x};
        st.template add<true>(one, uint32_t(e0 / kGroup), c2, [](int) {}, again);
    }
    *cell = st.top > -INFINITY ? order_key(st.top, st.place) : 0;
    const float2 s1 = unpack2(st.s), u1 = unpack2(st.u);
    return {st.m, s1.x + s1.y, u1.x + u1.y};
}

// Eight sums of a lane in a binary tree.
__device__ __forceinline__ Sums combine_eight(const Sums (*w)[32], int lane, float c2) {
    Sums a[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = w[i][lane];
#pragma unroll
    for (int n = 1; n < 8; n *= 2)
#pragma unroll
        for (int i = 0; i < 8; i += 2 * n) a[i] = combine(a[i], a[i + n], c2);
    return a[0];
}

// One element of the row, -inf where the mask leaves it out.
template <typename Elem>
__device__ __forceinline__ float element(const Elem* row, const uint8_t* bits, int64_t v) {
    if (bits && !((bits[v >> 3] >> (v & 7)) & 1u)) return -INFINITY;
    return to_float(row[v]);
}

// Puts the top_k largest keys of list[0 .. n), larger first, into out (zeroed before); the
// list is zero up to the next multiple of four.  By the threads from `first` on.
__device__ __forceinline__ void rank_keys(const uint64_t* list, int n, int top_k, uint64_t* out,
                                          int first = 0) {
    for (int i = int(threadIdx.x) - first; i < n; i += kThreads - first) {
        if (i < 0) return;
        const uint64_t k = list[i];
        int rank = 0;
#pragma unroll 4
        for (int o = 0; o < n; o += 4) {
            const ulonglong2 a = *reinterpret_cast<const ulonglong2*>(list + o);
            const ulonglong2 b = *reinterpret_cast<const ulonglong2*>(list + o + 2);
            rank += (a.x > k) + (a.y > k) + (b.x > k) + (b.y > k);
        }
        if (k != 0 && rank < top_k) out[rank] = k;
    }
}

// Collects the keys at or above `bound` out of those that each(f, bound) calls f with, into
// `list` (of kSize, zero up to the next multiple of four); returns their number.  If they
// are more than the list holds, the top_k-th of those that it got is a higher bound that
// still keeps the top_k best, and leaves out all but top_k of the list: the collection
// starts again with that.  *count and sh.chosen are 0 before and after.
template <int kSize, typename Each>
__device__ __forceinline__ int collect(Shared& sh, uint64_t* list, int* count, uint64_t& bound,
                                       int top_k, Each&& each) {
    while (true) {
        each([&](uint64_t k) {
            const int at = atomicAdd(count, 1);
            if (at < kSize) list[at] = k;
        }, bound);
        __syncthreads();
        const int n = *count;
        if (n <= kSize) {
            if (threadIdx.x < 4 && n + threadIdx.x < kSize) list[n + threadIdx.x] = 0;
            __syncthreads();
            return n;
        }
        rank_keys(list, kSize, top_k, sh.chosen);
        __syncthreads();
        bound = sh.chosen[top_k - 1];
        __syncthreads();
        if (threadIdx.x == 0) *count = 0;
        if (threadIdx.x < kMaxTopK) sh.chosen[threadIdx.x] = 0;
        __syncthreads();
    }
}

// Lists the CTA's cells that may hold one of its top_k best tokens; returns their number and
// the lowest token key that they are to be searched for.
__device__ __forceinline__ int best_cells(Shared& sh, int cells, int top_k, uint64_t& bound) {
    // A value that at least top_k cells reach: the lowest of the warps' r-th best lanes.
    uint32_t mine = 0;
    for (int i = threadIdx.x; i < cells; i += kThreads) mine = max(mine, uint32_t(sh.cells[i] >> 32));
    uint32_t low = 0;
    for (int r = 0; r < (top_k + kWarps - 1) / kWarps; ++r) {
        low = __reduce_max_sync(0xffffffffu, mine);
        if (mine == low) mine = 0;
    }
    if ((threadIdx.x & 31) == 0) sh.warp_bound[threadIdx.x >> 5] = low;
    if (threadIdx.x == 0) sh.count = sh.tokens = sh.groups = 0;
    if (threadIdx.x < kMaxTopK) sh.chosen[threadIdx.x] = 0;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) low = min(low, sh.warp_bound[w]);
    bound = max(uint64_t(low) << 32, uint64_t(1));
    const int n = collect<kCellList>(sh, sh.cell_list, &sh.count, bound, top_k,
                                     [&](auto&& f, uint64_t at_least) {
        for (int i = threadIdx.x; i < cells; i += kThreads) {
            const uint64_t k = sh.cells[i];
            if (k >= at_least) f(k);
        }
    });
    // a cell's key places its group: the last element of that group
    bound = uint32_t(bound) == 0 || bound == 1
                ? bound
                : (bound & ~uint64_t(0xffffffffu)) | uint32_t(~(key_place(bound) * kGroup + kGroup - 1));
    return n;
}

// Calls f(key) for the tokens of the listed cells that are not below `bound`.  The cells'
// groups are dealt to the threads, kGroupsAtOnce at a time: first the groups whose vectors
// hold an element that high (their neighbours' elements among them, and forbidden ones) are
// listed, then the elements of those are looked at one by one.  All threads call it.
//
// This and what follows runs once per row, so its instructions are rarely in the cache:
// short loops beat unrolled code.
template <typename Elem, typename F>
__device__ __forceinline__ void each_token(Shared& sh, const Elem* row, int shift,
                                           const uint8_t* bits, uint32_t V, int cells,
                                           uint64_t bound, F&& f) {
    using In = Vectors<Elem, true>;
    const uint32_t per_cell = (V - 1) / kStride + 1;
    const uint32_t total = cells * per_cell;
    for (uint32_t from = 0; from < total; from += kGroupsAtOnce) {
        uint32_t e0[2];
        In in[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t g = from + threadIdx.x + i * kThreads;
            const uint32_t c = g / per_cell;
            const uint64_t e = uint64_t(key_place(sh.cell_list[min(c, uint32_t(cells - 1))]) % kCells) * kGroup +
                               uint64_t(g - c * per_cell) * kStride;
            e0[i] = g < total && e < V ? uint32_t(e) : UINT32_MAX;
            if (e0[i] != UINT32_MAX && In::inside(e0[i], shift, V)) in[i].load(row, e0[i], shift);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (e0[i] == UINT32_MAX) continue;
            float top = INFINITY;
            if (In::inside(e0[i], shift, V)) {
                top = -INFINITY;
#pragma unroll
                for (int j = 0; j < In::kVecs; ++j) top = max_of<Elem>(top, in[i].v[j]);
            }
            if (ordered(top) >= uint32_t(bound >> 32)) sh.group_list[atomicAdd(&sh.groups, 1)] = e0[i];
        }
        __syncthreads();
        const int n = sh.groups * kGroup;
#pragma unroll 1
        for (int i = threadIdx.x; i < n; i += kThreads) {
            const uint32_t e = sh.group_list[i / kGroup] + i % kGroup;
            const float x = e < V ? element(row, bits, e) : -INFINITY;
            const uint64_t k = order_key(x, e);
            if (x > -INFINITY && k >= bound) f(k);
        }
        __syncthreads();
        if (threadIdx.x == 0) sh.groups = 0;
        if (from + kGroupsAtOnce < total) __syncthreads();
    }
}

// CTAs per SM: four by registers; the slots of shifted rows leave shared memory for three.
template <bool kShifted>
constexpr int kCtasPerSm = kShifted ? 3 : 4;
// Shared memory of a CTA.
constexpr int kSharedBytes = (int(sizeof(Shared)) + 15) / 16 * 16;

// Grid: T clusters of `ranks` CTAs (1, 2, 4 or 8).  kShifted: not every row starts at a
// 16-byte boundary.
template <typename Elem, bool kShifted, bool kMasked>
__global__ void __launch_bounds__(kThreads, kCtasPerSm<kShifted>)
    token_logprobs_kernel(const Args p, int ranks) {
    extern __shared__ __align__(16) uint8_t smem[];
    Shared& sh = *reinterpret_cast<Shared*>(smem);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // Launched with programmatic overlap: the kernel ahead in the stream may still be writing
    // the logits (or reading the outputs) until here.
    grid_dependency_wait();
    grid_launch_dependents();
    const int rank = ranks > 1 ? int(cluster_ctarank()) : 0;
    const int64_t t = blockIdx.x / unsigned(ranks);
    const Elem* row = static_cast<const Elem*>(p.logits) + t * p.row_stride;
    const uint8_t* bits =
        kMasked ? reinterpret_cast<const uint8_t*>(p.allowed + t * p.allowed_stride) : nullptr;
    // (below infinity, as 0 times it has to be 0; what the limit cuts off only logits that
    // differ by less than 1e-36 could tell)
    const float c2 = fminf(p.inv_temp * kLog2e, FLT_MAX);
    const int shift = kShifted ? row_shift(row) : 0;
    if (ranks > 1) cluster_arrive_relaxed();  // every CTA runs before another writes to it
    int32_t target = -1;
    if (rank == 0 && threadIdx.x == 0) target = p.targets[t];

    // A block of eight strips at a time, one strip per warp.
    const int blocks = kBlocks / ranks;
    const int first = rank * blocks * kWarps + warp;
    StripPlan plan(first, p.V);
    using Loads = Unit<Elem, kShifted, kMasked>;
    Loads unit = [&] {
        if constexpr (kShifted) return Loads(reinterpret_cast<uint4*>(smem + kSharedBytes), warp);
        else return Loads();
    }();
    if constexpr (kShifted) {
        unit.load(row, bits, shift, lane, plan, 0);
    } else {
#pragma unroll
        for (int k = 0; k < Loads::N; ++k) unit.load(k, row, bits, lane, plan, 0);
    }
    for (int j = 0; j < blocks; ++j) {
        // (behind the last block: a strip behind every row's end)
        const StripPlan next(j + 1 < blocks ? first + (j + 1) * kWarps : kNoStrip, p.V);
        uint64_t cell = 0;
        sh.strip_sums[j][warp][lane] = read_strip<Elem, kShifted, kMasked>(
            row, shift, bits, uint32_t(p.V), plan, next, unit, lane, c2, &cell);
        if (p.top_k > 0) sh.cells[(j * kWarps + warp) * 32 + lane] = cell;
        plan = next;
    }
    float target_x = -INFINITY;
    if (target >= 0 && target < p.V) target_x = element(row, bits, target);
    __syncthreads();

    uint64_t bound = 0;
    int cells = 0, tokens = 0;
    if (p.top_k > 0) cells = best_cells(sh, kCells / ranks, p.top_k, bound);
    Sums sum;
    if (warp < blocks) {
        sum = combine_eight(sh.strip_sums[warp], lane, c2);
        if (ranks == 1) sh.block_sums[warp][lane] = sum;
    }
    if (p.top_k > 0)
        tokens = collect<kTokenList>(sh, sh.token_list(), &sh.tokens, bound, p.top_k,
                                     [&](auto&& f, uint64_t at_least) {
            each_token(sh, row, shift, bits, uint32_t(p.V), cells, at_least, f);
        });

    const int handed = (p.top_k + 3) / 4 * 4;  // keys each CTA hands over, zeros at the end
    if (ranks > 1) {
        if (p.top_k > 0) {
            rank_keys(sh.token_list(), tokens, p.top_k, sh.chosen);
            __syncthreads();
        }
        cluster_wait();
        if (warp < blocks) {
            const uint32_t to = mapa_shared(smem_u32(&sh.block_sums[rank * blocks + warp][lane]), 0);
            st_shared_cluster_u32(to, __float_as_uint(sum.m));
            st_shared_cluster_u32(to + 4, __float_as_uint(sum.s));
            st_shared_cluster_u32(to + 8, __float_as_uint(sum.u));
        }
        if (warp == kWarps - 1 && lane < handed) {
            const uint64_t k = sh.chosen[lane];
            const uint32_t to = mapa_shared(smem_u32(&sh.gathered()[rank * handed + lane]), 0);
            st_shared_cluster_u32(to, uint32_t(k));
            st_shared_cluster_u32(to + 4, uint32_t(k >> 32));
        }
        cluster_sync();
        if (rank != 0) return;
        if (threadIdx.x < kMaxTopK) sh.chosen[threadIdx.x] = 0;
    }
    __syncthreads();
    if (warp > 0) {  // the other warps rank the tokens while the first one ends the sums
        if (ranks == 1)
            rank_keys(sh.token_list(), tokens, p.top_k, sh.chosen, 32);
        else
            rank_keys(sh.gathered(), ranks * handed, p.top_k, sh.chosen, 32);
    } else {
        sum = combine_eight(sh.block_sums, lane, c2);
#pragma unroll 1
        for (int off = 16; off > 0; off >>= 1) {
            Sums o;
            o.m = __shfl_xor_sync(0xffffffffu, sum.m, off);
            o.s = __shfl_xor_sync(0xffffffffu, sum.s, off);
            o.u = __shfl_xor_sync(0xffffffffu, sum.u, off);
            sum = combine(sum, o, c2);
        }
        if (lane == 0) {
            sh.row = sum;
            const float logs = logf(sum.s);
            const float lse = fmaf(sum.m, p.inv_temp, logs);
            const bool empty = sum.s == 0.0f || lse == -INFINITY;
            p.out_lse[t] = empty ? -INFINITY : lse;
            p.out_entropy[t] = empty ? 0.0f : logs - kLn2 * (sum.u / sum.s);
            float lp = 0.0f;
            if (target >= 0 && target < p.V)
                lp = target_x == -INFINITY || empty ? -INFINITY
                                                    : (target_x - sum.m) * p.inv_temp - logs;
            else if (target >= p.V)
                atomicAdd(&g_range_rows, 1ull);
            p.out_logp[t] = lp;
        }
    }
    if (p.top_k == 0) return;
    __syncthreads();
    if (threadIdx.x < p.top_k) {
        const uint64_t k = sh.chosen[threadIdx.x];
        const float logs = logf(sh.row.s);
        const bool empty = fmaf(sh.row.m, p.inv_temp, logs) == -INFINITY;
        const int64_t at = t * p.top_k + threadIdx.x;
        p.out_ids[at] = k == 0 ? -1 : int32_t(key_place(k));
        p.out_top[at] = k == 0 || empty
                            ? -INFINITY
                            : (from_ordered(uint32_t(k >> 32)) - sh.row.m) * p.inv_temp - logs;
    }
}

struct BackwardArgs {
    const void* logits;
    int64_t row_stride;
    const int32_t* targets;
    const uint32_t* allowed;
    int64_t allowed_stride;
    int V, top_k;
    float inv_temp;
    const float *lse, *entropy, *g_logp, *g_lse, *g_entropy, *g_top;
    const int32_t* top_ids;
    void* grad;
    int64_t grad_stride;
    int parts, part_length;  // CTAs per row and elements of each (a multiple of kGroup)
};

// dx = p (a - b (z - lse)) with a, b scaled by inv_temp, for the tokens of a row.
struct RowGradient {
    float it, lse, a, b;
    __device__ __forceinline__ float operator()(float x) const {
        const float lp = max_nan(fmaf(x, it, -lse), kFarBelow);
        return ex2(lp * kLog2e) * fmaf(lp, -b, a);
    }
    template <typename Elem>
    __device__ __forceinline__ void operator()(const Packed8<Elem>& in, float (&x)[8]) const {
        const F2 it2 = pack2(it, it), lse2 = pack2(-lse, -lse), a2 = pack2(a, a), b2 = pack2(-b, -b);
        const F2 l2e = pack2(kLog2e, kLog2e);
#pragma unroll
        for (int j = 0; j < 8; j += 2) {
            const float2 xx = in.pair(j / 2);
            const float2 lp = unpack2(fma2(pack2(xx.x, xx.y), it2, lse2));
            const F2 l = pack2(max_nan(lp.x, kFarBelow), max_nan(lp.y, kFarBelow));
            const float2 t = unpack2(mul2(l, l2e));
            const float2 d = unpack2(mul2(pack2(ex2(t.x), ex2(t.y)), fma2(l, b2, a2)));
            x[j] = d.x;
            x[j + 1] = d.y;
        }
    }
};

__device__ __forceinline__ void store_eight(float* out, const float (&x)[8]) {
    reinterpret_cast<float4*>(out)[0] = make_float4(x[0], x[1], x[2], x[3]);
    reinterpret_cast<float4*>(out)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store_eight(__half* out, const float (&x)[8]) {
    __half2 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2half2_rn(x[2 * j], x[2 * j + 1]);
    *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(h);
}
__device__ __forceinline__ void store_eight(__nv_bfloat16* out, const float (&x)[8]) {
    __nv_bfloat162 h[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
    *reinterpret_cast<uint4*>(out) = *reinterpret_cast<const uint4*>(h);
}

// Eight mask bits from element e0 on (e0 + 7 lies in the row).
__device__ __forceinline__ uint32_t eight_bits(const uint8_t* bits, int64_t e0) {
    const int64_t b = e0 >> 3;
    const int off = int(e0 & 7);
    return off ? (uint32_t(bits[b]) | uint32_t(bits[b + 1]) << 8) >> off : bits[b];
}

// One part of a row: elementwise in groups of eight that start at 16-byte boundaries of
// the gradient's row, then the few tokens with a gradient of their own (the target, the
// alternatives) once more, whole.  Those are read before anything is written, so the
// gradient may take the logits' place.
template <typename Elem, bool kMasked>
__global__ void __launch_bounds__(kThreads, 4)
    token_logprobs_backward_kernel(const BackwardArgs p) {
    const int lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t t = blockIdx.x / unsigned(p.parts);
    const int part = int(blockIdx.x - t * p.parts);
    const Elem* row = static_cast<const Elem*>(p.logits) + t * p.row_stride;
    Elem* out = static_cast<Elem*>(p.grad) + t * p.grad_stride;
    const uint8_t* bits =
        kMasked ? reinterpret_cast<const uint8_t*>(p.allowed + t * p.allowed_stride) : nullptr;
    const int head = (kVecElems<Elem> - row_shift(out)) % kVecElems<Elem>;
    const int begin = part == 0 ? 0 : head + part * p.part_length;
    const int end = int(min(int64_t(head) + int64_t(part + 1) * p.part_length, int64_t(p.V)));

    const int32_t target = p.targets[t];
    const float g_target = p.g_logp && target >= 0 && target < p.V ? p.g_logp[t] : 0.0f;
    int32_t id = -1;
    float g_id = 0.0f;
    if (lane < p.top_k) {
        id = p.top_ids[t * p.top_k + lane];
        if (id >= 0 && id < p.V)
            g_id = p.g_top[t * p.top_k + lane];
        else
            id = -1;
    }
    float total = g_id;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) total += __shfl_xor_sync(0xffffffffu, total, off);
    total += g_target;
    const float g_ent = p.g_entropy ? p.g_entropy[t] : 0.0f;
    const float H = p.g_entropy ? p.entropy[t] : 0.0f;
    RowGradient f;
    f.it = p.inv_temp;
    f.lse = p.lse[t];
    f.b = p.inv_temp * g_ent;
    f.a = p.inv_temp * ((p.g_lse ? p.g_lse[t] : 0.0f) - total - g_ent * H);
    const bool empty = f.lse == -INFINITY;
    // A token at -inf (masked or not) has gradient 0.  Its p is 0, but 0 times a factor that is
    // not finite would not be: rows whose factors reach fp32's end at the cut, or whose lse is
    // NaN, compare each element, one by one as the rows without tokens.
    const bool special = empty || !(fabsf(f.a) - kFarBelow * fabsf(f.b) <= FLT_MAX) || f.lse != f.lse;

    // Tokens of this part with a gradient of their own: lane j the j-th alternative (the
    // first of equal ids for all of them), lane 0 of warp 1 the target.
    const bool own_target = target >= begin && target < end;
    int own = -1;
    float own_x = -INFINITY, own_g = 0.0f;
    if (p.top_k > 0 || own_target) {
        bool taken = false;
        for (int j = 0; j < p.top_k; ++j) {
            const int32_t other = __shfl_sync(0xffffffffu, id, j);
            const float g = __shfl_sync(0xffffffffu, g_id, j);
            taken |= other == target;
            if (other == id) {
                own_g += g;
                if (j < lane) own_g = NAN;  // an earlier lane has it
            }
        }
        if (threadIdx.x < 32) {
            if (id >= begin && id < end && own_g == own_g) own = id;
            if (id == target) own_g += g_target;
        } else if (threadIdx.x == 32 && own_target && !taken) {
            own = target;
            own_g = g_target;
        }
        if (own >= 0) own_x = element(row, bits, own);
        __syncthreads();
    }

    const int first = head + part * p.part_length;
    const int shift = (row_shift(row) + head) % kVecElems<Elem>;
    auto body = [&](auto shifted) {
        using In = Vectors<Elem, decltype(shifted)::value>;
        constexpr int kBatch = 8 / int(sizeof(Elem));
        for (int64_t e = int64_t(first) + threadIdx.x * kGroup; e < end;
             e += kBatch * kThreads * kGroup) {
            In in[kBatch];
            Packed8<Elem> raw[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t e0 = e + i * kThreads * kGroup;
                if (e0 < end && In::inside(e0, shift, p.V)) in[i].load(row, e0, shift);
            }
            unshift(in, shift, raw);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const int64_t e0 = e + i * kThreads * kGroup;
                if (e0 >= end) break;
                if (In::inside(e0, shift, p.V)) {
                    if (kMasked) raw[i].keep(eight_bits(bits, e0));
                    float x[8];
                    f(raw[i], x);
                    store_eight(out + e0, x);
                } else {
                    for (int j = 0; j < 8 && e0 + j < p.V; ++j)
                        out[e0 + j] = from_float<Elem>(f(element(row, bits, e0 + j)));
                }
            }
        }
    };
    if (special) {
        for (int64_t e = int64_t(begin) + threadIdx.x; e < end; e += kThreads) {
            const float x = empty ? -INFINITY : element(row, bits, e);
            out[e] = from_float<Elem>(x == -INFINITY ? 0.0f : f(x));
        }
    } else {
        if (shift == 0)
            body(std::false_type());
        else
            body(std::true_type());
        if (part == 0 && threadIdx.x < min(head, p.V))
            out[threadIdx.x] = from_float<Elem>(f(element(row, bits, threadIdx.x)));
    }

    if (p.top_k > 0 || own_target) {
        __syncthreads();
        if (own >= 0 && own_x != -INFINITY && !empty)
            out[own] = from_float<Elem>(fmaf(f.it, own_g, f(own_x)));
    }
}

}  // namespace

cudaError_t token_logprobs_take_range_rows(unsigned long long* out) {
    unsigned long long v = 0, zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(&v, g_range_rows, sizeof v);
    if (e != cudaSuccess) return e;
    if (v) e = cudaMemcpyToSymbol(g_range_rows, &zero, sizeof zero);
    *out = v;
    return e;
}

cudaError_t launch_token_logprobs(const void* logits, ElemType type, int64_t row_stride,
                                  const int32_t* targets, const uint32_t* allowed,
                                  int64_t allowed_stride, int64_t T, int64_t V, float inv_temp,
                                  int top_k, float* out_logp, float* out_lse, float* out_entropy,
                                  int32_t* out_ids, float* out_top, int num_sms, cudaStream_t stream) {
    const Args p = {logits, row_stride, targets, allowed, allowed_stride, int(V), top_k, inv_temp,
                    out_logp, out_lse, out_entropy, out_top, out_ids};
    const int64_t elem = type == ElemType::kFp32 ? 4 : 2;
    const bool shifted = reinterpret_cast<uintptr_t>(logits) % 16 != 0 ||
                         (T > 1 && row_stride * elem % 16 != 0);
    // CTAs per row: as many as keep the launch within what the SMs hold at once (four
    // CTAs each; a little less with alternatives, whose selection every CTA pays for, and
    // then at least 8192 elements per CTA).
    int ranks = 8;
    while (ranks > 1 && (2 * T * ranks > (top_k ? 7 : 8) * int64_t(num_sms) ||
                         (top_k && V < 8192 * int64_t(ranks))))
        ranks /= 2;
    auto go = [&](auto kernel, int slots, int which) {
        const int smem = kSharedBytes + slots;
        // per device: the kernels that may have that much
        static std::atomic<uint8_t> configured[64];
        if (slots > 0) {
            int dev = 0;
            cudaError_t e = cudaGetDevice(&dev);
            if (e != cudaSuccess) return e;
            if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
            if (!(configured[dev].load() >> which & 1)) {
                e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
                if (e != cudaSuccess) return e;
                configured[dev].fetch_or(uint8_t(1 << which));
            }
        }
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[2];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = unsigned(ranks);
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.gridDim = dim3(unsigned(T * ranks), 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = ranks > 1 ? 2 : 1;
        cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p, ranks);
        return e != cudaSuccess ? e : cudaGetLastError();
    };
    auto pick = [&](auto elem) {
        using Elem = decltype(elem);
        constexpr int kSlots = kWarps * kUnitOf<Elem> * Unit<Elem, true, false>::kVecs * 16;
        const int which = int(type) * 2;
        if (shifted)
            return allowed ? go(token_logprobs_kernel<Elem, true, true>, kSlots, which + 1)
                           : go(token_logprobs_kernel<Elem, true, false>, kSlots, which);
        return allowed ? go(token_logprobs_kernel<Elem, false, true>, 0, 0)
                       : go(token_logprobs_kernel<Elem, false, false>, 0, 0);
    };
    if (type == ElemType::kBf16) return pick(__nv_bfloat16());
    if (type == ElemType::kFp16) return pick(__half());
    return pick(float());
}

cudaError_t launch_token_logprobs_backward(const void* logits, ElemType type, int64_t row_stride,
                                           const int32_t* targets, const uint32_t* allowed,
                                           int64_t allowed_stride, int64_t T, int64_t V,
                                           float inv_temp, const float* lse, const float* entropy,
                                           const float* g_logp, const float* g_lse,
                                           const float* g_entropy, const int32_t* top_ids,
                                           const float* g_top, int top_k, void* grad,
                                           int64_t grad_stride, int num_sms, cudaStream_t stream) {
    BackwardArgs p = {logits, row_stride, targets, allowed, allowed_stride, int(V), top_k, inv_temp,
                      lse, entropy, g_logp, g_lse, g_entropy, g_top, top_ids, grad, grad_stride, 1, 0};
    int64_t want = 32768;
    while (want > 2048 && T * ((V + want - 1) / want) < 8 * int64_t(num_sms)) want /= 2;
    p.part_length = int(want);
    p.parts = int((V + want - 1) / want);
    auto go = [&](auto kernel) {
        cudaLaunchConfig_t cfg = {};
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[0].val.programmaticStreamSerializationAllowed = 1;
        cfg.gridDim = dim3(unsigned(T * p.parts), 1, 1);
        cfg.blockDim = dim3(kThreads, 1, 1);
        cfg.stream = stream;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
        return e != cudaSuccess ? e : cudaGetLastError();
    };
    if (type == ElemType::kBf16)
        return allowed ? go(token_logprobs_backward_kernel<__nv_bfloat16, true>)
                       : go(token_logprobs_backward_kernel<__nv_bfloat16, false>);
    if (type == ElemType::kFp16)
        return allowed ? go(token_logprobs_backward_kernel<__half, true>)
                       : go(token_logprobs_backward_kernel<__half, false>);
    return allowed ? go(token_logprobs_backward_kernel<float, true>)
                   : go(token_logprobs_backward_kernel<float, false>);
}

}  // namespace rlk
