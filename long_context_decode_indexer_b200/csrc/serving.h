// serving.h -- launch parameters of the serving kernels: page tables and slot
// maps, rotary positions, the latent cache append and the shared-prefix
// attention; shared by the host-side API (serving_api.cu) and the kernels.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace dsa {

// Launch as a programmatic dependent of the kernel ahead in the stream: the
// kernel may start early and waits (grid_dependency_wait) before it reads.
template <class... KArgs, class... Args>
inline cudaError_t launch_dependent(void (*kern)(KArgs...), int grid, int block, size_t smem, cudaStream_t st,
                                    const Args &...args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// ------------------------------------------------- page tables and slot maps
constexpr int kTabThreads = 512;
constexpr int kTabMaxSeq = 16384;  // three int32 per sequence in shared memory: 192 KB

// kv_len is seq_len, or free_head_out is free_head: written behind a barrier of
// the cluster that is the whole grid, or by a second kernel.
enum { kTabApart = 0, kTabAdvanceCluster = 1, kTabAdvanceLater = 2 };
constexpr int kTabCluster = 8;

struct TableParams {
    const int32_t *seq_len, *new_len, *fork_src, *free_pages, *free_head;
    int32_t *page_table, *q_start, *q_seq, *positions, *q_n, *slots, *kv_len, *free_head_out;
    int32_t nseq, nt, page_size, max_pages, n_free, sees_self;
    int32_t page_shift;  // page_size = 1 << page_shift, or -1
    int32_t vec;         // the token arrays are 16-byte aligned
    int32_t in_place;    // kTabApart, or how lengths and head are advanced in place
    int64_t n_pages;     // page ids are 0..n_pages-1
    int32_t *taken;      // ws: pages handed out, from k13 to k13_advance (in place)
    int *status;
};
cudaError_t launch_build_tables(const TableParams &a, int grid, cudaStream_t st);

// --------------------------------------------------------- rotary positions
constexpr int kRopeMaxPairs = 128;
constexpr int kLatent = 512;   // c_kv width of a latent row
constexpr int kRopeRow = 64;   // rope part of a latent row

struct RopeTurns {
    double turn[kRopeMaxPairs];  // turns (angle / 2 pi) per position of each pair
    double mscale;
};

struct RopeParams {
    const void *x;   // source (dy of the backward pass)
    void *y;
    const int32_t *positions;
    int64_t xt, xh, yt, yh;  // token and head strides of source and destination, elements
    int32_t nt, h;           // heads of the wider side
    int32_t begin, rot, d;
    int32_t in_place;        // source and destination are the same array
    int32_t transpose;       // backward: the inverse turn, padding tokens get 0
    int32_t units_rope, units;  // work units of a head: rotated, all
    int32_t tp, hp;          // tokens of a block; heads of a step (k14), threads summing a unit (k15)
    int32_t ub, iters;       // k14: units of a block, steps
    RopeTurns tb;
};
// vec: 16-byte accesses (pointers, strides and ranges allow them);
// shared: 0 heads map one to one, 1 one source head to all (forward), 2 all
// source heads summed into one (backward)
cudaError_t launch_rope(const RopeParams &a, int dtype, bool half_layout, bool vec, int shared, cudaStream_t st);

struct AppendParams {
    const uint16_t *c_kv, *k_pe;
    int64_t c_stride, pe_stride;
    const int32_t *positions, *slots;
    void *cache;
    int64_t row_stride;   // bf16 elements, or bytes of an FP8 row
    float *kv_scale;      // FP8: [cache_rows]
    int64_t cache_rows;
    int32_t nt, half_layout;
    int *status;
    RopeTurns tb;
};
cudaError_t launch_latent_append(const AppendParams &a, bool fp8, cudaStream_t st);

// -------------------------------------------------- shared-prefix attention
constexpr int kPfxRows = 128;       // query rows per row tile, 64 in each CTA of a pair
constexpr int kPfxTile = 256;       // positions per tile
constexpr int kPfxOverhead = 2;     // cost of starting and ending a piece, in tiles
constexpr int kPfxMaxPairs = 128;   // CTA pairs of the grid (74 on 148 SMs)
constexpr int kPfxMaxQueries = 4096;
constexpr int kPfxMaxGroups = 4096;
constexpr int kPfxThreads = 320;    // warp 0 loads, warp 1 MMA, warps 2-9 softmax

// One tile of query rows over one range of positions, as the plan lays it out.
struct PrefixTile {
    int32_t row0, nrows;   // query rows (query * h + head), at most 128
    int32_t lo, hi;        // positions [lo, hi) of the sequence the rows attend to
    int32_t seq;           // read through this sequence's table
    int32_t base;          // first position of tile 0 (64-aligned in pages, else lo)
    int32_t tiles;         // position tiles from base to hi
    int32_t pieces;        // its first pair | pairs that work on it << 16
    int32_t turn;          // the tiles are taken in the order turn, turn + 1, .., tiles - 1, 0, .., turn - 1
};

struct PrefixParams {
    const int32_t *q_seq, *q_n;
    const int64_t *seq_row0;
    const int32_t *page_table;
    int32_t max_pages, page_shift;  // page_size = 1 << page_shift
    int64_t cache_rows;
    const int32_t *group_q0, *group_n;
    int32_t ngroups, nq, h, max_n;
    int32_t pairs;            // CTA pairs of the grid
    float scale_log2;
    uint16_t *out;
    float *lse;
    // workspace
    int64_t *cut;             // [pairs + 1] where each pair's work starts: row tile << 32 | tile (in its order)
    PrefixTile *tiles;        // row tiles, in order
    int32_t *q_shared;        // [nq] the query's shared row tile << 7 | its first row there, or -1
    int32_t *q_own;           // [nq] the query's own row tile, or -1
    float *part_o;            // [row tiles + pairs, 128, 512] normalised partial outputs
    float *part_lse;          // [row tiles + pairs, 128]
    int *status;
    long long wait_budget;
    int32_t inject;           // tests only: the first pair leaves out one arrival
};
cudaError_t launch_shared_prefix(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                 const PrefixParams &a, cudaStream_t st);

}  // namespace dsa
