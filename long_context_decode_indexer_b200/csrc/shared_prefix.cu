// shared_prefix.cu -- dense MQA-mode MLA attention of a batch whose queries
// share long prefixes, on sm_100a.
//
//   out = softmax(scale q . c) c[:512] over all positions of a query, the
//   first group_n of which are the same cache rows for its whole group.
//
// All heads of all queries of a group read the same prefix rows, so the
// group's (query, head) pairs are the rows of one matrix product: 128 of them
// at a time stream the prefix.  What a query has behind the prefix is a
// product of its own with its h rows.  Both are the same work: a row tile
// (up to 128 rows of q) over a range of positions, cut into pieces over the
// CTA pairs and merged by log-sum-exp.
//
// k17_prefix_plan  one CTA: the row tiles, and where each pair's work starts.
// k18_prefix_attn  a persistent kernel, one CTA pair per two SMs.
// k19_prefix_join  merges the pieces of every query row.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "dsa.h"
#include "kernels.h"
#include "ptx.cuh"
#include "ptx_pair.cuh"
#include "serving.h"

namespace dsa {

// ---------------------------------------------------------------------------
// k17: the plan.  Segments are the groups' shared ranges (all of a group's
// rows) followed by every query's own range.  A query whose history ends
// inside the prefix takes no part in the shared tile (its rows there are
// computed and dropped): the positions it does not see then cannot reach it,
// whatever they hold.  The cost axis is the row tiles one behind the other,
// tiles + kPfxOverhead each, cut into equal shares; while there are fewer
// tiles than pairs every pair takes one (starting up then costs less than
// working them off one by one).
//
// Where row tiles of one prefix are cut at different places, their pairs
// would read it at as many places at once, and a prefix larger than L2 would
// come from HBM again and again (889 MB for a 113 MB prefix and 16 row tiles).
// So each row tile takes its tiles in an order that starts where its first
// inner cut lies: the pairs that start there all read tile 0 first, the pairs
// behind them tile s, 2 s, .. (s tiles a share), and go on in step.  The sums
// do not depend on the order.
//
// One load of the inputs, the rest in shared
// memory: the latency of this kernel is the latency of small calls.
// ---------------------------------------------------------------------------
namespace {

constexpr int kPlanThreads = 1024;
// The plan's arrays, carved from dynamic shared memory of the call's own size
// (a large request would make the launch wait for an SM to be empty).
struct PlanSmem {
    long long *tile0;   // [segments + 1] position tiles (of all row tiles) before the segment
    int32_t *rt0;       // [segments + 1] first row tile
    int32_t *n;         // [nq] visible positions, clamped
    int32_t *seq;       // [nq]
    int32_t *grp;       // [nq] group of a query, or -1
    int32_t *q0;        // [groups + 1]
    int32_t *prefix;    // [groups] clamped
    int32_t *used;      // [groups] some query sees the whole prefix
    __host__ __device__ static size_t bytes(int nq, int groups) {
        return (static_cast<size_t>(nq) + groups + 1) * 12 + static_cast<size_t>(nq) * 12 +
               (static_cast<size_t>(groups) + 1) * 12;
    }
    __device__ PlanSmem(void *base, int nq, int groups) {
        const int segs = nq + groups + 1;
        tile0 = static_cast<long long *>(base);
        rt0 = reinterpret_cast<int32_t *>(tile0 + segs);
        n = rt0 + segs;
        seq = n + nq;
        grp = seq + nq;
        q0 = grp + nq;
        prefix = q0 + groups + 1;
        used = prefix + groups + 1;
    }
};

// a / b of non-negative numbers, in 32 bits where they fit (a 64-bit division
// is a hundred instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

}  // namespace

__global__ void __launch_bounds__(kPlanThreads) k17_prefix_plan(const PrefixParams a) {
    extern __shared__ __align__(16) uint8_t plan_raw[];
    __shared__ long long warp_tiles[kPlanThreads / 32];
    __shared__ int32_t warp_rt[kPlanThreads / 32];
    // the cuts, and the tiles before each
    __shared__ long long cut[kPfxMaxPairs + 1], raw[kPfxMaxPairs + 1];
    __shared__ long long cut_at[kPfxMaxPairs + 1], raw_at[kPfxMaxPairs + 1];
    __shared__ int32_t any_bad, n_cuts;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // k18 may set itself up meanwhile; everything below waits for the kernel
    // ahead of this one
    grid_launch_dependents();
    grid_dependency_wait();
    const int G = a.ngroups, nseg = G + a.nq;
    const PlanSmem sm(plan_raw, a.nq, G);
    if (tid == 0) any_bad = 0;
    for (int i = tid; i < a.nq; i += kPlanThreads) {
        const int n = a.q_n[i];
        sm.seq[i] = a.q_seq[i];
        sm.n[i] = min(max(n, 0), a.max_n);
        sm.grp[i] = -1;
        if (n < 0 || n > a.max_n) record_status(a.status, DSA_ERR_DEVICE_CHECK);
    }
    for (int g = tid; g <= G; g += kPlanThreads) {
        sm.q0[g] = a.group_q0[g];
        if (g == G) break;
        const int n = a.group_n[g];
        sm.prefix[g] = min(max(n, 0), a.max_n);
        sm.used[g] = 0;
        if (n < 0 || n > a.max_n) record_status(a.status, DSA_ERR_DEVICE_CHECK);
    }
    __syncthreads();
    for (int g = tid; g <= G; g += kPlanThreads)
        if (g == G ? sm.q0[g] != a.nq : (sm.q0[g] < 0 || sm.q0[g + 1] < sm.q0[g] || (g == 0 && sm.q0[g] != 0))) any_bad = 1;
    __syncthreads();
    const bool bad = any_bad != 0;  // no usable groups: every query on its own
    if (bad && tid == 0) record_status(a.status, DSA_ERR_DEVICE_CHECK);
    if (!bad)
        for (int g = warp; g < G; g += kPlanThreads / 32) {
            const int p = sm.prefix[g];
            bool any = false;
            for (int i = sm.q0[g] + lane; i < sm.q0[g + 1]; i += 32) {
                sm.grp[i] = g;
                any |= sm.n[i] >= p;
            }
            if (__any_sync(0xffffffffu, any) && lane == 0) sm.used[g] = p > 0;
        }
    __syncthreads();
    // segment s -> rows, range, sequence
    auto segment = [&](int s, PrefixTile &t) {
        t.row0 = t.nrows = t.lo = t.hi = t.seq = t.pieces = t.turn = 0;
        if (s < G) {
            if (!bad && sm.used[s]) {
                t.row0 = sm.q0[s] * a.h;
                t.nrows = (sm.q0[s + 1] - sm.q0[s]) * a.h;
                t.hi = sm.prefix[s];
                t.seq = sm.seq[sm.q0[s]];
            }
        } else {
            const int i = s - G, g = sm.grp[i], n = sm.n[i];
            const int p = g >= 0 ? sm.prefix[g] : 0;
            t.row0 = i * a.h;
            t.nrows = a.h;
            t.lo = n >= p ? p : 0;
            t.hi = n;
            // a history inside the prefix is read where the prefix is
            t.seq = sm.seq[n >= p ? i : sm.q0[g]];
        }
        t.base = a.page_table ? t.lo & ~63 : t.lo;
        t.tiles = t.hi > t.lo ? (t.hi - t.base + kPfxTile - 1) / kPfxTile : 0;
        if (t.tiles == 0) t.nrows = 0;
    };
    const int per = (nseg + kPlanThreads - 1) / kPlanThreads;
    const int s0 = min(tid * per, nseg), s1 = min(s0 + per, nseg);
    long long tiles = 0;
    int rts = 0;
    for (int s = s0; s < s1; ++s) {
        PrefixTile t;
        segment(s, t);
        const int r = (t.nrows + kPfxRows - 1) / kPfxRows;
        rts += r;
        tiles += static_cast<long long>(r) * t.tiles;
    }
    long long it = tiles;
    int ir = rts;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long x = __shfl_up_sync(0xffffffffu, it, o);
        const int y = __shfl_up_sync(0xffffffffu, ir, o);
        if (lane >= o) {
            it += x;
            ir += y;
        }
    }
    if (lane == 31) {
        warp_tiles[warp] = it;
        warp_rt[warp] = ir;
    }
    __syncthreads();
    long long total_tiles = 0, bt = it - tiles;
    int total_rt = 0, br = ir - rts;
    const int warps = min((nseg + per - 1) / per / 32 + 1, kPlanThreads / 32);  // those that have segments
    for (int w = 0; w < warps; ++w) {
        if (w < warp) {
            bt += warp_tiles[w];
            br += warp_rt[w];
        }
        total_tiles += warp_tiles[w];
        total_rt += warp_rt[w];
    }
    for (int s = s0; s < s1; ++s) {
        PrefixTile t;
        segment(s, t);
        const int r = (t.nrows + kPfxRows - 1) / kPfxRows;
        sm.tile0[s] = bt;
        sm.rt0[s] = br;
        bt += static_cast<long long>(r) * t.tiles;
        br += r;
    }
    if (tid == 0) {
        sm.tile0[nseg] = total_tiles;
        sm.rt0[nseg] = total_rt;
    }
    __syncthreads();
    // the cuts: one tile each, or equal shares of the cost axis
    const int over = total_tiles <= a.pairs ? 0 : kPfxOverhead;
    const int pairs = total_tiles <= a.pairs ? static_cast<int>(total_tiles) : a.pairs;
    auto start_of = [&](int s) { return sm.tile0[s] + static_cast<long long>(over) * sm.rt0[s]; };
    if (tid <= pairs) {
        long long key = static_cast<long long>(total_rt) << 32, at = total_tiles;
        if (tid < pairs) {
            const long long x = quotient(start_of(nseg) * tid, pairs);
            int lo = 0, hi = nseg;  // the last segment that starts at or before x: it is not empty
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (start_of(mid) <= x) lo = mid;
                else hi = mid;
            }
            const long long begin = start_of(lo);
            const long long unit = quotient(start_of(lo + 1) - begin, sm.rt0[lo + 1] - sm.rt0[lo]);
            const long long rt = quotient(x - begin, unit);
            const int t = max(static_cast<int>(x - begin - rt * unit) - over, 0);
            key = (sm.rt0[lo] + rt) << 32 | t;
            at = sm.tile0[lo] + rt * (unit - over) + t;
        }
        raw[tid] = key;
        raw_at[tid] = at;
    }
    __syncthreads();
    // pairs without work go: a piece's pairs are then consecutive
    if (warp == 0) {
        int n = 0;
        for (int w0 = 0; w0 < pairs; w0 += 32) {
            const int w = w0 + lane;
            const bool keep = w < pairs && raw[w] < raw[w + 1];
            const uint32_t m = __ballot_sync(0xffffffffu, keep);
            if (keep) {
                cut[n + __popc(m & ((1u << lane) - 1u))] = raw[w];
                cut_at[n + __popc(m & ((1u << lane) - 1u))] = raw_at[w];
            }
            n += __popc(m);
        }
        if (lane == 0) n_cuts = n;
        for (int w = n + lane; w <= a.pairs; w += 32) cut[w] = static_cast<long long>(total_rt) << 32;
    }
    __syncthreads();
    for (int w = tid; w <= a.pairs; w += kPlanThreads) a.cut[w] = cut[w];
    // row tiles, each with its pairs
    auto pair_of = [&](long long key) {  // the pair whose range holds key
        int lo = 0, hi = n_cuts;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (cut[mid] <= key) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    for (int rt = tid; rt < total_rt; rt += kPlanThreads) {
        int lo = 0, hi = nseg;  // its segment: the last that starts at or before rt
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (sm.rt0[mid] <= rt) lo = mid;
            else hi = mid;
        }
        PrefixTile t;
        segment(lo, t);
        const int k = rt - sm.rt0[lo];
        const long long begin = static_cast<long long>(rt) << 32;
        const int first = pair_of(begin), end = pair_of(begin | (t.tiles - 1));
        t.row0 += k * kPfxRows;
        t.nrows = min(t.nrows - k * kPfxRows, kPfxRows);
        t.pieces = first | (end - first + 1) << 16;
        if (lo < G) {
            // the first cut inside, or how far its one pair is when it starts
            const int inner = static_cast<int>(cut[first + 1] & 0xffffffff);
            const long long ahead = sm.tile0[lo] + static_cast<long long>(k) * t.tiles - cut_at[first];
            t.turn = first < end ? (cut[first] == begin ? 0 : t.tiles - inner)
                                 : static_cast<int>(ahead - quotient(ahead, t.tiles) * t.tiles);
        }
        a.tiles[rt] = t;
    }
    for (int i = tid; i < a.nq; i += kPlanThreads) {
        const int g = sm.grp[i];
        int at = -1;
        if (g >= 0 && sm.used[g] && sm.n[i] >= sm.prefix[g]) {
            const int row = (i - sm.q0[g]) * a.h;
            at = (sm.rt0[g] + row / kPfxRows) << 7 | (row % kPfxRows);
        }
        a.q_shared[i] = at;
        a.q_own[i] = sm.rt0[G + i + 1] > sm.rt0[G + i] ? sm.rt0[G + i] : -1;
    }
}

// ---------------------------------------------------------------------------
// k18: a CTA pair (cluster of two) works on a row tile of 128 query rows, 64
// in each CTA, and tiles of 256 positions:
//   S = Q K^T   M = 128, N = 256 positions (each CTA supplies 128), K = 576
//   O += P V    M = 128, N = 512 value columns (each CTA supplies 256), K = 256
// With 64 rows a CTA, O takes 256 of its 512 TMEM columns, which leaves room
// for two S buffers: S(j+1) is computed while the softmax of tile j runs.
// (128 rows a CTA would fill TMEM with O alone.)  An M = 128 MMA of a pair
// takes 70 cycles whether N is 128 or 256, hence 256 positions.
//   warp 0      TMA into one ring of 16 KB stages, in the order the MMAs take
//               them: a K stage is 128 positions x 64 columns, a V stage 64
//               positions x 128 value columns (128B swizzle)
//   warp 1      the leader's elected lane issues every MMA of the pair
//   warps 2-9   softmax: TMEM lane = row + 64 * (position half); two warps a
//               lane quarter, 64 positions each.  The row maximum is merged
//               over the four threads of a row; it is raised only past 2^8,
//               then O is rescaled.  P goes to shared memory in bf16.
// 64 queries x 128 heads over a shared 32K prefix take 484-499 us, 1.20-1.23
// PFLOP/s: 0.71-0.73 of the measured bf16 rate, at the chip's power limit.  P as a bf16 pair
// (hi + lo, as in the sparse attention) took 27% more.  A tile takes about
// 4900 cycles, its 68 MMAs at least 4760.
// ---------------------------------------------------------------------------
namespace {

constexpr uint32_t kChunk = 64 * 128;          // 64 rows x 64 bf16 columns
constexpr uint32_t kStage = 2 * kChunk;
constexpr int kQChunks = kDqk / 64;            // 9
constexpr int kStages = 7;
constexpr uint32_t kOffP = kQChunks * kChunk;  // P: four chunks of 64 positions
constexpr uint32_t kOffRing = kOffP + 4 * kChunk;
constexpr uint32_t kOffMisc = kOffRing + kStages * kStage;
constexpr uint32_t kColO = 0, kColS = 256;     // TMEM columns: O, then two S buffers of 128
constexpr float kRaise = 8.f;                  // the running maximum is raised past 2^8 only

struct PfxSmem {
    uint64_t full[kStages], empty[kStages];
    uint64_t q_full, q_empty, s_full[2], p_full, pv_done, o_empty, edge, mma_done;
    uint32_t tmem_base;
    volatile int32_t abort;
    float xch[2][4][64];  // exchange between the four threads of a row
};
constexpr uint32_t kPfxSmemBytes = kOffMisc + sizeof(PfxSmem);
static_assert(kPfxSmemBytes <= 232448, "shared memory of k18");

__device__ __forceinline__ bool bar_and(int id, int count, bool pred) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "bar.red.and.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(static_cast<uint32_t>(pred)), "r"(id), "r"(count)
        : "memory");
    return r != 0;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// First position of the j-th tile that is taken.
__device__ __forceinline__ int tile_start(const PrefixTile &t, int j) {
    const int at = j + t.turn;
    return t.base + (at < t.tiles ? at : at - t.tiles) * kPfxTile;
}
// 64-position groups of a tile that hold positions before the end.
__device__ __forceinline__ int groups_of(const PrefixTile &t, int j) {
    return min((t.hi - tile_start(t, j) + 63) >> 6, kPfxTile / 64);
}

// A pair's walk over its pieces: row tile rt, position tiles [t0, t1).
struct PieceWalk {
    int64_t key, end;
    __device__ bool next(const PrefixTile *tiles, int &rt, int &t0, int &t1, PrefixTile &t) {
        if (key >= end) return false;
        rt = static_cast<int>(key >> 32);
        t0 = static_cast<int>(key & 0xffffffff);
        t = tiles[rt];
        const int64_t row_end = static_cast<int64_t>(rt) << 32 | t.tiles;
        t1 = end < row_end ? static_cast<int>(end & 0xffffffff) : t.tiles;
        key = static_cast<int64_t>(rt + 1) << 32;
        return true;
    }
};

}  // namespace

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPfxThreads, 1)
    k18_prefix_attn(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                    const __grid_constant__ CUtensorMap vmap, const PrefixParams a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    PfxSmem &sm = *reinterpret_cast<PfxSmem *>(smem + kOffMisc);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const uint32_t cta = cluster_rank();
    const int pair = blockIdx.x >> 1;

    if (tid == 0) {
        prefetch_map(&qmap);
        prefetch_map(&kmap);
        prefetch_map(&vmap);
        sm.abort = 0;
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&sm.full[s], 2);   // both producers
            mbar_init(&sm.empty[s], 1);
        }
        mbar_init(&sm.q_full, 2);
        mbar_init(&sm.q_empty, 1);
        mbar_init(&sm.s_full[0], 1);
        mbar_init(&sm.s_full[1], 1);
        mbar_init(&sm.p_full, 16);  // the softmax warps of both CTAs
        mbar_init(&sm.pv_done, 1);
        mbar_init(&sm.o_empty, 16);
        mbar_init(&sm.edge, 1);
        mbar_init(&sm.mma_done, 1);
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(&sm.tmem_base, 512);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem = sm.tmem_base;
    grid_dependency_wait();  // the plan

    PieceWalk walk{a.cut[pair], a.cut[pair + 1]};
    PrefixTile t;
    int rt, t0, t1;

    if (warp == 0) {
        // ------------------------------------------------ TMA, both CTAs
        int s = 0, pieces = 0;
        uint32_t ph = 0, eph = 0;
        bool ok = true;
        const uint32_t full0 = remote_smem(&sm.full[0], 0), q_full = remote_smem(&sm.q_full, 0);
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            return __all_sync(0xffffffffu, mbar_wait(bar, parity, a.wait_budget) && !sm.abort) != 0;
        };
        bool ahead = mbar_test(&sm.empty[0], 1u);  // this stage is free (looked at one stage ahead)
        auto wait_empty = [&]() { return __all_sync(0xffffffffu, ahead) || wait(&sm.empty[s], ph ^ 1u); };
        auto advance = [&]() {
            if (++s == kStages) {
                s = 0;
                ph ^= 1u;
            }
            ahead = mbar_test(&sm.empty[s], ph ^ 1u);
        };
        while (ok && walk.next(a.tiles, rt, t0, t1, t)) {
            // cache rows of the four 64-position groups of tile j (lanes
            // 0-3): the table entries are loaded two tiles ahead and turned
            // into rows one tile ahead.  Groups behind the end, or outside
            // the cache, come from past the tensor's end and read as zero.
            const int64_t row_base = a.page_table ? 0 : a.seq_row0[t.seq];
            const int32_t *table = a.page_table ? a.page_table + static_cast<int64_t>(t.seq) * a.max_pages : nullptr;
            auto page_of = [&](int j) {
                const int p = tile_start(t, j) + 64 * lane;
                return table && lane < 4 && j < t1 && p < t.hi ? table[p >> a.page_shift] : 0;
            };
            auto rows_of = [&](int j, int page) {
                const int p = tile_start(t, j) + 64 * lane;
                int row = static_cast<int>(a.cache_rows);
                if (lane < 4 && j < t1 && p < t.hi) {
                    const int64_t r = table ? (static_cast<int64_t>(page) << a.page_shift) + (p & ((1 << a.page_shift) - 1))
                                            : row_base + p;
                    const int64_t last = r + min(64, t.hi - p);  // rows in use, at most
                    if (r >= 0 && last <= a.cache_rows) row = static_cast<int>(r);
                    else record_status(a.status, DSA_ERR_DEVICE_CHECK);
                }
                return row;
            };
            const int page0 = page_of(t0), page1 = page_of(t0 + 1);
            int r_cur = rows_of(t0, page0), r_next = rows_of(t0 + 1, page1);
            // this CTA's half of a tile's positions, all 576 columns
            auto load_k = [&](int rows) {
                const int r0 = __shfl_sync(0xffffffffu, rows, 2 * static_cast<int>(cta));
                const int r1 = __shfl_sync(0xffffffffu, rows, 2 * static_cast<int>(cta) + 1);
                for (int c = 0; c < kQChunks; ++c) {
                    if (!wait_empty()) return false;
                    if (elect_one()) {
                        uint8_t *dst = smem + kOffRing + s * kStage;
                        cluster_arrive_expect_tx(full0 + s * 8, kStage);
                        tma_load_2d_pair(dst, &kmap, full0 + s * 8, c * 64, r0);
                        tma_load_2d_pair(dst + kChunk, &kmap, full0 + s * 8, c * 64, r1);
                    }
                    advance();
                }
                return true;
            };
            // all groups of positions, this CTA's half of each 256 value columns
            auto load_v = [&](int rows, int j) {
                const int groups = groups_of(t, j);
                for (int g = 0; g < groups; ++g) {
                    const int row = __shfl_sync(0xffffffffu, rows, g);
                    const int p = tile_start(t, j) + 64 * g;
                    const int z0 = max(t.lo - p, 0), z1 = min(t.hi - p, 64);
                    for (int nh = 0; nh < 2; ++nh) {
                        const int block = nh * 4 + static_cast<int>(cta) * 2;
                        if (!wait_empty()) return false;
                        uint8_t *dst = smem + kOffRing + s * kStage;
                        if (z0 == 0 && z1 == 64) {
                            if (elect_one()) {
                                cluster_arrive_expect_tx(full0 + s * 8, kStage);
                                tma_load_3d_pair(dst, &vmap, full0 + s * 8, 0, row, block);
                            }
                        } else {
                            // rows outside [lo, hi) may hold anything, and 0 *
                            // NaN is NaN: clear them before the MMA reads
                            if (elect_one()) {
                                mbar_arrive_expect_tx(&sm.edge, kStage);
                                tma_load_3d(dst, &vmap, &sm.edge, 0, row, block);
                            }
                            __syncwarp();
                            if (!wait(&sm.edge, eph)) return false;
                            eph ^= 1u;
                            for (int i = lane >> 3; i < 128; i += 4) {
                                const int r = i & 63;
                                if (r < z0 || r >= z1)
                                    *reinterpret_cast<uint4 *>(dst + (i >> 6) * kChunk + r * 128 + (lane & 7) * 16) =
                                        make_uint4(0u, 0u, 0u, 0u);
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (elect_one()) {
                                cluster_release_smem();
                                cluster_arrive(full0 + s * 8);
                            }
                        }
                        advance();
                    }
                }
                return true;
            };
            // q: 64 rows x 576, once the last piece's S products are done
            if (pieces > 0 && !(ok = wait(&sm.q_empty, static_cast<uint32_t>(pieces - 1) & 1u))) break;
            if (elect_one()) {
                cluster_arrive_expect_tx(q_full, kQChunks * kChunk);
                for (int c = 0; c < kQChunks; ++c)
                    tma_load_2d_pair(smem + c * kChunk, &qmap, q_full, c * 64, t.row0 + static_cast<int>(cta) * 64);
            }
            __syncwarp();
            ++pieces;
            // in the order the MMAs take them: K(0), K(1), V(0), K(2), V(1), ...
            ok = load_k(r_cur);
            for (int j = t0; ok && j < t1; ++j) {
                const int page_after = page_of(j + 2);
                if (j + 1 < t1) ok = load_k(r_next);
                if (ok) ok = load_v(r_cur, j);
                r_cur = r_next;
                r_next = rows_of(j + 2, page_after);
            }
        }
        if (!ok && lane == 0) {
            record_status(a.status, DSA_ERR_TIMEOUT);
            sm.abort = 1;
        }
        // A load in flight must land before its CTA exits.  The MMAs took them
        // all, unless the work was abandoned: then the barriers that count
        // them may miss the other CTA's arrival, so the wait is a time (50 us,
        // far above what a load takes).
        if (!ok) {
            const long long begin = clock64();
            while (clock64() - begin < 100000) __nanosleep(1000);
        }
    } else if (warp == 1 && cta == 0) {
        // ------------------------------------------------ MMA, the leader
        constexpr uint32_t idesc_s = make_idesc(1, 1, 0, 0, 128, 256);
        constexpr uint32_t idesc_pv = make_idesc(1, 1, 0, 1, 128, 256);
        // descriptors of offset 0; an offset of b bytes adds b / 16
        const uint64_t q_desc = make_sdesc(smem_u32(smem), 16, 1024, kSwizzle128B);
        const uint64_t p_desc = make_sdesc(smem_u32(smem + kOffP), 16, 1024, kSwizzle128B);
        const uint64_t k_desc = make_sdesc(smem_u32(smem + kOffRing), 16, 1024, kSwizzle128B);
        const uint64_t v_desc = make_sdesc(smem_u32(smem + kOffRing), kChunk, 1024, kSwizzle128B);
        int s = 0, pieces = 0;
        uint32_t ph = 0, it = 0;  // it: tiles so far
        bool ok = true;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            const bool w = __all_sync(0xffffffffu, mbar_wait(bar, parity, a.wait_budget) && !sm.abort) != 0;
            tc_fence_after();
            return w;
        };
        // the same where the other CTA's threads have written
        auto wait_peer = [&](uint64_t *bar, uint32_t parity) {
            const bool w = __all_sync(0xffffffffu, mbar_wait_cluster(bar, parity, a.wait_budget) && !sm.abort) != 0;
            tc_fence_after();
            return w;
        };
        bool ahead = false;  // the next stage has arrived (looked at one stage ahead)
        auto wait_full = [&]() {
            if (!__all_sync(0xffffffffu, ahead)) return wait(&sm.full[s], ph);
            tc_fence_after();
            return true;
        };
        auto advance = [&]() {
            if (++s == kStages) {
                s = 0;
                ph ^= 1u;
            }
            ahead = mbar_test(&sm.full[s], ph);
        };
        auto issue_s = [&](uint32_t tile) {
            const uint32_t d = tmem + kColS + (tile & 1u) * 128;
            for (int c = 0; c < kQChunks; ++c) {
                if (!wait_full()) return false;
                if (elect_one()) {
                    const uint64_t ad = q_desc + c * (kChunk / 16), bd = k_desc + s * (kStage / 16);
                    if (c == 0) mma_bf16_ss_pair<false>(d, ad, bd, idesc_s);
                    else mma_bf16_ss_pair<true>(d, ad, bd, idesc_s);
#pragma unroll
                    for (int kk = 1; kk < 4; ++kk) mma_bf16_ss_pair<true>(d, ad + kk * 2, bd + kk * 2, idesc_s);
                    tc_commit_pair(&sm.empty[s]);
                    if (c == kQChunks - 1) tc_commit_pair(&sm.s_full[tile & 1u]);
                }
                __syncwarp();
                advance();
            }
            return true;
        };
        while (ok && walk.next(a.tiles, rt, t0, t1, t)) {
            if (!(ok = wait(&sm.q_full, static_cast<uint32_t>(pieces) & 1u))) break;
            if (!(ok = issue_s(it))) break;
            if (t1 - t0 == 1 && elect_one()) tc_commit_pair(&sm.q_empty);
            __syncwarp();
            for (int j = t0; j < t1; ++j, ++it) {
                if (j + 1 < t1) {
                    if (!(ok = issue_s(it + 1))) break;
                    if (j + 2 == t1 && elect_one()) tc_commit_pair(&sm.q_empty);
                    __syncwarp();
                }
                // P(j) written (so S(j) read, and O rescaled); the first tile
                // of a piece overwrites O, which the last piece's epilogue
                // must have read
                ok = wait_peer(&sm.p_full, it & 1u);
                if (ok && j == t0 && pieces > 0) ok = wait_peer(&sm.o_empty, static_cast<uint32_t>(pieces - 1) & 1u);
                if (!ok) break;
                const int groups = groups_of(t, j);
                for (int g = 0; g < groups; ++g) {
                    // a group with rows cleared by the loading warps themselves
                    const int p = tile_start(t, j) + 64 * g;
                    const bool edge = p < t.lo || p + 64 > t.hi;
                    for (int nh = 0; nh < 2; ++nh) {
                        if (!(ok = edge ? wait_peer(&sm.full[s], ph) : wait_full())) break;
                        if (elect_one()) {
                            const uint32_t d = tmem + kColO + nh * 128;
                            const uint64_t ad = p_desc + g * (kChunk / 16), bd = v_desc + s * (kStage / 16);
                            if (j == t0 && g == 0) mma_bf16_ss_pair<false>(d, ad, bd, idesc_pv);
                            else mma_bf16_ss_pair<true>(d, ad, bd, idesc_pv);
#pragma unroll
                            for (int kk = 1; kk < 4; ++kk)  // 16 positions: two 8-row groups of the stage
                                mma_bf16_ss_pair<true>(d, ad + kk * 2, bd + kk * 128, idesc_pv);
                            tc_commit_pair(&sm.empty[s]);
                        }
                        __syncwarp();
                        advance();
                    }
                    if (!ok) break;
                }
                if (!ok) break;
                if (elect_one()) tc_commit_pair(&sm.pv_done);
                __syncwarp();
            }
            ++pieces;
        }
        if (!ok && lane == 0) {
            record_status(a.status, DSA_ERR_TIMEOUT);
            sm.abort = 1;
        }
        if (elect_one()) tc_commit_pair(&sm.mma_done);
        __syncwarp();
    } else if (warp >= 2) {
        // ------------------------------------------------ softmax, both CTAs
        const int quarter = warp & 3;          // TMEM lanes 32 * quarter ..
        const int hf = (warp - 2) >> 2;        // which 64 of the 128 S columns; which 128 of the 256 O columns
        const int ph = quarter >> 1;           // position half of the tile / 128-column part of each V half
        const int rg = quarter & 1;            // row group: its four warps exchange under one barrier
        const int r = rg * 32 + lane;          // row of this CTA
        const int part = ph * 2 + hf;          // the 64 positions of a tile this thread has
        const uint32_t lane_addr = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t p_full = remote_smem(&sm.p_full, 0), o_empty = remote_smem(&sm.o_empty, 0);
        uint8_t *prow = smem + kOffP + part * kChunk + r * 128;
        uint32_t it = 0;
        bool ok = true;
        bool skip = a.inject && pair == 0 && cta == 0 && warp == 2;
        auto wait = [&](uint64_t *bar, uint32_t parity) {
            const bool w = __all_sync(0xffffffffu, mbar_wait(bar, parity, a.wait_budget) && !sm.abort) != 0;
            tc_fence_after();
            return w;
        };
        while (ok && walk.next(a.tiles, rt, t0, t1, t)) {
            float m = -INFINITY, l = 0.f;
            for (int j = t0; j < t1; ++j, ++it) {
                if (ok) ok = wait(&sm.s_full[it & 1u], (it >> 1) & 1u);
                float x[64];
                float mx = -INFINITY, unit = a.scale_log2;
                if (ok) {
                    uint32_t(&u0)[32] = *reinterpret_cast<uint32_t(*)[32]>(x);
                    uint32_t(&u1)[32] = *reinterpret_cast<uint32_t(*)[32]>(x + 32);
                    tmem_ld32(lane_addr + kColS + (it & 1u) * 128 + hf * 64, u0);
                    tmem_ld32(lane_addr + kColS + (it & 1u) * 128 + hf * 64 + 32, u1);
                    tmem_wait_ld();
                    const int p = tile_start(t, j) + part * 64;
                    if (p >= t.lo && p + 64 <= t.hi) {
                        if (unit >= 0.f) {
#pragma unroll
                            for (int c = 0; c < 64; ++c) mx = fmaxf(mx, x[c]);
                        } else {
                            mx = INFINITY;
#pragma unroll
                            for (int c = 0; c < 64; ++c) mx = fminf(mx, x[c]);
                        }
                        mx *= unit;
                    } else {
#pragma unroll
                        for (int c = 0; c < 64; ++c) {
                            x[c] = (p + c >= t.lo && p + c < t.hi) ? x[c] * unit : -INFINITY;
                            mx = fmaxf(mx, x[c]);
                        }
                        unit = 1.f;  // scaled already
                    }
                    sm.xch[it & 1u][part][r] = mx;
                }
                ok = bar_and(1 + rg, 128, ok);
                if (!ok) break;
                mx = fmaxf(fmaxf(sm.xch[it & 1u][0][r], sm.xch[it & 1u][1][r]),
                           fmaxf(sm.xch[it & 1u][2][r], sm.xch[it & 1u][3][r]));
                float alpha = 1.f;
                bool rescale = false;
                if (mx > m + kRaise || (m == -INFINITY && mx > m)) {
                    rescale = m != -INFINITY;
                    alpha = rescale ? fast_exp2(m - mx) : 1.f;
                    m = mx;
                    l *= alpha;
                }
                const float mm = m == -INFINITY ? 0.f : m;  // nothing but -inf so far: every weight is 0
                // a weight is rounded to bf16 once, for its product; the sum
                // takes it unrounded
                uint32_t w2[32];
                float2 sum = make_float2(0.f, 0.f);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float2 y = fma2(make_float2(x[2 * e], x[2 * e + 1]), make_float2(unit, unit), make_float2(-mm, -mm));
                    const float2 w = make_float2(fast_exp2(y.x), fast_exp2(y.y));
                    sum.x += w.x;
                    sum.y += w.y;
                    w2[e] = pack_bf16(w.x, w.y);
                }
                l += sum.x + sum.y;
                // P and O are free once the last tile's product is done
                if (j > t0) ok = wait(&sm.pv_done, (it - 1) & 1u);
                if (ok && j > t0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
                    for (int c = hf * 128; c < hf * 128 + 128; c += 32) {
                        uint32_t o[32];
                        tmem_ld32(lane_addr + kColO + c, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                        tmem_st32(lane_addr + kColO + c, o);
                    }
                    tmem_wait_st();
                }
                if (ok) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const int at = (k ^ (r & 7)) * 16;
                        *reinterpret_cast<uint4 *>(prow + at) = make_uint4(w2[4 * k], w2[4 * k + 1], w2[4 * k + 2], w2[4 * k + 3]);
                    }
                    fence_proxy_async_smem();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0 && !skip) {
                        cluster_release_smem();
                        cluster_arrive(p_full);
                    }
                    skip = false;
                }
            }
            // epilogue: the piece's O / l and log-sum-exp
            if (ok) ok = wait(&sm.pv_done, (it - 1) & 1u);
            sm.xch[it & 1u][part][r] = l;
            ok = bar_and(1 + rg, 128, ok);
            if (!ok) break;
            const float lt = (sm.xch[it & 1u][0][r] + sm.xch[it & 1u][1][r]) + (sm.xch[it & 1u][2][r] + sm.xch[it & 1u][3][r]);
            bar_and(1 + rg, 128, true);  // read before the next piece's first exchange
            const float inv = lt == 0.f ? 0.f : 1.f / lt;
            const int64_t slot = rt + pair;
            const int row = static_cast<int>(cta) * 64 + r;
            // through this warp's part of the P buffer, so that a store covers
            // whole 128-byte lines: 32 rows x 32 columns at a time
            uint8_t *stage = smem + kOffP + (warp - 2) * 4096;
            float *dst = a.part_o + (slot * kPfxRows + static_cast<int>(cta) * 64 + rg * 32) * kDv + hf * 256 + ph * 128;
            const int rows_left = t.nrows - static_cast<int>(cta) * 64 - rg * 32;
#pragma unroll 1
            for (int c = 0; c < 128 && rows_left > 0; c += 32) {
                uint32_t o[32];
                tmem_ld32(lane_addr + kColO + hf * 128 + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4 *>(stage + lane * 128 + ((i ^ (lane & 7)) * 16)) =
                        make_float4(__uint_as_float(o[4 * i]) * inv, __uint_as_float(o[4 * i + 1]) * inv,
                                    __uint_as_float(o[4 * i + 2]) * inv, __uint_as_float(o[4 * i + 3]) * inv);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int q = i * 4 + (lane >> 3);
                    if (q < rows_left)
                        *reinterpret_cast<float4 *>(dst + static_cast<int64_t>(q) * kDv + c + (lane & 7) * 4) =
                            *reinterpret_cast<const float4 *>(stage + q * 128 + (((lane & 7) ^ (q & 7)) * 16));
                }
                __syncwarp();
            }
            if (part == 0 && row < t.nrows)
                a.part_lse[slot * kPfxRows + row] = lt == 0.f ? -INFINITY : (m + log2f(lt)) * 0.6931471805599453f;
            tc_fence_before();
            __syncwarp();
            if (lane == 0) cluster_arrive(o_empty);
        }
        if (!ok && lane == 0) {
            record_status(a.status, DSA_ERR_TIMEOUT);
            sm.abort = 1;
        }
    }

    grid_launch_dependents();
    // every MMA of the pair is done before TMEM is freed and either CTA exits
    __syncthreads();
    if (warp == 1 && lane == 0) mbar_wait(&sm.mma_done, 0, a.wait_budget);
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) tmem_dealloc_pair(tmem, 512);
}

// ---------------------------------------------------------------------------
// k19: one warp merges the pieces of one query row, or (C = 1) of a quarter of
// its columns: those of its shared row tile and of its own, each worked on by
// consecutive pairs; a piece's slot is row tile + pair.  With few rows there
// can be 74 pieces to a row, and the quarters keep more of them in flight.
// ---------------------------------------------------------------------------
template <int C>
__global__ void __launch_bounds__(256) k19_prefix_join(const PrefixParams a) {
    grid_dependency_wait();
    constexpr int kAhead = 16 / C;  // pieces loaded together
    const int lane = threadIdx.x & 31;
    const int64_t unit = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    const int64_t row = C == 4 ? unit : unit >> 2;
    const int col = C == 4 ? 0 : static_cast<int>(unit & 3) * 128;  // first of the warp's columns
    if (row >= static_cast<int64_t>(a.nq) * a.h) return;
    const int i = static_cast<int>(row / a.h), head = static_cast<int>(row % a.h);
    const int sh = a.q_shared[i], own = a.q_own[i];
    // shared tile (the group's rows run on over tiles), own tile
    int rt[2] = {sh >= 0 ? (sh >> 7) + ((sh & 127) + head) / kPfxRows : -1, own};
    const int at[2] = {((sh & 127) + head) % kPfxRows, head};
    int count[2];
    int64_t slot[2];  // of the first piece
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const int p = rt[k] >= 0 ? a.tiles[rt[k]].pieces : 0;
        count[k] = p >> 16;
        slot[k] = static_cast<int64_t>(rt[k] + (p & 0xffff)) * kPfxRows + at[k];
    }
    const int pieces = count[0] + count[1];
    auto slot_of = [&](int p) { return p < count[0] ? slot[0] + static_cast<int64_t>(p) * kPfxRows
                                                    : slot[1] + static_cast<int64_t>(p - count[0]) * kPfxRows; };
    float top = -INFINITY;
    for (int p = lane; p < pieces; p += 32) top = fmaxf(top, a.part_lse[slot_of(p)]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const float base = top == -INFINITY ? 0.f : top;
    float4 acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f;
    for (int p0 = 0; p0 < pieces; p0 += 32) {
        const float mine = p0 + lane < pieces ? expf(a.part_lse[slot_of(p0 + lane)] - base) : 0.f;
        const int n = min(32, pieces - p0);
        for (int p = 0; p < n; p += kAhead) {
            float4 v[kAhead][C];
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (p + k < n) {
                    const float4 *o = reinterpret_cast<const float4 *>(a.part_o + slot_of(p0 + p + k) * kDv + col);
#pragma unroll
                    for (int c = 0; c < C; ++c) v[k][c] = __ldcg(o + c * 32 + lane);
                }
#pragma unroll
            for (int k = 0; k < kAhead; ++k)
                if (p + k < n) {
                    const float f = __shfl_sync(0xffffffffu, mine, p + k);
                    total += f;
#pragma unroll
                    for (int c = 0; c < C; ++c) {
                        acc[c].x += f * v[k][c].x;
                        acc[c].y += f * v[k][c].y;
                        acc[c].z += f * v[k][c].z;
                        acc[c].w += f * v[k][c].w;
                    }
                }
        }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    uint2 *out = reinterpret_cast<uint2 *>(a.out + row * kDv + col);
#pragma unroll
    for (int c = 0; c < C; ++c)
        out[c * 32 + lane] = make_uint2(pack_bf16(acc[c].x * inv, acc[c].y * inv), pack_bf16(acc[c].z * inv, acc[c].w * inv));
    if (lane == 0 && col == 0) a.lse[row] = total == 0.f ? -INFINITY : base + logf(total);
}

cudaError_t launch_shared_prefix(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                 const PrefixParams &a, cudaStream_t st) {
    const size_t plan_bytes = PlanSmem::bytes(a.nq, a.ngroups);
    cudaError_t e = cudaFuncSetAttribute(k17_prefix_plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         static_cast<int>(PlanSmem::bytes(kPfxMaxQueries, kPfxMaxGroups)));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(k18_prefix_attn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kPfxSmemBytes));
    if (e != cudaSuccess) return e;
    e = launch_dependent(k17_prefix_plan, 1, kPlanThreads, plan_bytes, st, a);
    if (e != cudaSuccess) return e;
    e = launch_dependent(k18_prefix_attn, 2 * a.pairs, kPfxThreads, kPfxSmemBytes, st, qmap, kmap, vmap, a);
    if (e != cudaSuccess) return e;
    // quarters of few rows (64 rows of 74 pieces: the call 52 -> 41 us), whole
    // rows where there are more (864 rows of two pieces: 24 -> 21 us)
    const int64_t rows = static_cast<int64_t>(a.nq) * a.h;
    if (rows <= 256) return launch_dependent(k19_prefix_join<1>, static_cast<int>((rows + 1) / 2), 256, 0, st, a);
    return launch_dependent(k19_prefix_join<4>, static_cast<int>((rows + 7) / 8), 256, 0, st, a);
}

}  // namespace dsa
