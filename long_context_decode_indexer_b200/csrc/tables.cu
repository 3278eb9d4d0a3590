// tables.cu -- page tables and slot maps of one serving step, built on the
// GPU from the requests' lengths, so that no step waits for the host.
//
// With seq_b positions cached and new_b to come, sequence b needs
//   need_b = ceil((seq_b + new_b) / ps) - ceil(seq_b / ps)
// pages; its tokens and its pages start at the exclusive prefix sums of new
// and need.  Everything else is a lookup: token j of sequence b has position
// seq_b + j and row page * ps + position % ps, its page an entry of the table
// (the last, partly filled page) or of the free list (a new one).
//
// One kernel.  Every CTA computes both prefix sums itself (nseq lengths are a
// few KB and stay in L2; a second launch would cost more than the repeated
// scan), then takes its share of the tokens (each finds its sequence by a
// binary search in shared memory) and of the sequences (one warp each, for
// the table entries).  Nothing a CTA reads is written by another.  Where the
// new lengths or the new head replace the old ones, every CTA has to have read
// them first: up to eight CTAs are one cluster and meet at its barrier (128
// idle sequences: 3.6 us apart, 4.25 in place, 4.7 with a second kernel); more
// leave it to a small second kernel (4096: 6.2 and 7.5 us).  A counter of
// finished CTAs (4.3 and 7.6 us) would rely on what earlier calls left in the
// workspace.  What bounds it is the chain of dependent loads: lengths,
// shared-memory search, page (4.5 us for 128 sequences of two tokens, 10.8 us
// for 4096 sequences and 100000 tokens).
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsa.h"
#include "ptx.cuh"
#include "ptx_pair.cuh"
#include "serving.h"

namespace dsa {

namespace {

// First index in start[0..n] whose value exceeds t, minus one: the sequence
// of token t (empty sequences are skipped).
__device__ __forceinline__ int seq_of(const int32_t *start, int n, int t) {
    int lo = 0, hi = n;  // start[lo] <= t < start[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

// One warp writes to[0..n) = id of each from[i], eight loads at a time (a
// fork of a 128K history copies 2048 entries).
template <class F>
__device__ __forceinline__ void copy_entries(int32_t *to, const int32_t *from, int n, int lane, F id) {
    for (int i = lane; i < n; i += 8 * 32) {
        int v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + 32 * k < n) v[k] = from[i + 32 * k];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (i + 32 * k < n) to[i + 32 * k] = id(v[k]);
    }
}

}  // namespace

__global__ void __launch_bounds__(kTabThreads, 1) k13_build_tables(const TableParams a) {
    extern __shared__ int32_t sm_tab[];
    int32_t *tok0 = sm_tab;                    // [nseq + 1] new_len, then the first token of each sequence
    int32_t *page0 = sm_tab + a.nseq + 1;      // [nseq + 1] pages needed, then the first new page
    int32_t *len = sm_tab + 2 * (a.nseq + 1);  // [nseq] cached positions
    __shared__ uint32_t warp_tok[kTabThreads / 32], warp_page[kTabThreads / 32];
    __shared__ int bad_any;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int ps = a.page_size;
    const int head = *a.free_head;
    // x / page_size (a division is forty instructions, a shift one)
    auto pages_of = [&](int x) { return a.page_shift >= 0 ? x >> a.page_shift : x / ps; };
    if (tid == 0) bad_any = 0;
    __syncthreads();

    // ---- lengths, checked one by one; 0 where refused, so that the sums
    // below stay defined
    bool bad = false;
#pragma unroll 4
    for (int b = tid; b < a.nseq; b += kTabThreads) {
        const int64_t s = a.seq_len[b], n = a.new_len[b];
        const bool ok = s >= 0 && n >= 0 && n <= a.nt && s + n <= static_cast<int64_t>(a.max_pages) * ps;
        bad |= !ok;
        const int si = ok ? static_cast<int>(s) : 0, ni = ok ? static_cast<int>(n) : 0;
        len[b] = si;
        tok0[b] = ni;
        page0[b] = pages_of(si + ni + ps - 1) - pages_of(si + ps - 1);
    }
    __syncthreads();
    if (a.fork_src) {
#pragma unroll 4
        for (int b = tid; b < a.nseq; b += kTabThreads) {
            const int src = a.fork_src[b];
            if (src >= 0)
                bad |= src >= a.nseq || src == b || a.fork_src[src] >= 0 || len[b] % ps != 0 || len[b] > len[src];
        }
    }
    if (bad) bad_any = 1;
    // ---- prefix sums.  A warp takes consecutive sequences, 32 at a time.
    // Sums stop at 2^30: more than any batch that fits, and no overflow.
    auto add = [](uint32_t x, uint32_t y) { return min(x + y, 1u << 30); };
    const int per = (a.nseq + kTabThreads - 1) / kTabThreads * 32;
    const int b0 = min(warp * per, a.nseq), b1 = min(b0 + per, a.nseq);
    uint32_t tok = 0, pages = 0;  // of the warp's sequences so far
    for (int b = b0 + lane; b - lane < b1; b += 32) {
        const uint32_t n = b < b1 ? tok0[b] : 0u, need = b < b1 ? page0[b] : 0u;
        uint32_t x = n, y = need;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(0xffffffffu, x, o), v = __shfl_up_sync(0xffffffffu, y, o);
            if (lane >= o) {
                x = add(x, u);
                y = add(y, v);
            }
        }
        if (b < b1) {
            tok0[b] = static_cast<int32_t>(add(tok, x - n));
            page0[b] = static_cast<int32_t>(add(pages, y - need));
        }
        tok = add(tok, __shfl_sync(0xffffffffu, x, 31));
        pages = add(pages, __shfl_sync(0xffffffffu, y, 31));
    }
    if (lane == 0) {
        warp_tok[warp] = tok;
        warp_page[warp] = pages;
    }
    __syncthreads();
    uint32_t total_t = 0, total_p = 0, base_t = 0, base_p = 0;
#pragma unroll
    for (int w = 0; w < kTabThreads / 32; ++w) {
        if (w == warp) {
            base_t = total_t;
            base_p = total_p;
        }
        total_t = add(total_t, warp_tok[w]);
        total_p = add(total_p, warp_page[w]);
    }
    const bool refuse = bad_any || total_t > static_cast<uint32_t>(a.nt) || head < 0 || head > a.n_free ||
                        total_p > static_cast<uint32_t>(a.n_free - head);
    if (!refuse) {
        for (int b = b0 + lane; b < b1; b += 32) {
            tok0[b] += static_cast<int32_t>(base_t);
            page0[b] += static_cast<int32_t>(base_p);
        }
        if (tid == 0) {
            tok0[a.nseq] = static_cast<int32_t>(total_t);
            page0[a.nseq] = static_cast<int32_t>(total_p);
        }
    } else if (tid == 0) {
        record_status(a.status, DSA_ERR_DEVICE_CHECK);
    }
    __syncthreads();

    const int gtid = blockIdx.x * kTabThreads + tid, gthreads = gridDim.x * kTabThreads;
    const int ntok = refuse ? 0 : static_cast<int>(total_t);
    // ---- tokens, four adjacent ones a thread (one search, then steps) where
    // there are more than threads
    const int chunk = a.nt > gthreads ? 4 : 1;
    for (int64_t first = static_cast<int64_t>(gtid) * chunk; first < a.nt; first += static_cast<int64_t>(gthreads) * chunk) {
        const int t0 = static_cast<int>(first), count = min(chunk, a.nt - t0);
        int seq[4], pos[4], n[4], page[4], slot[4];
        int b = t0 < ntok ? seq_of(tok0, a.nseq, t0) : 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int t = t0 + k;
            seq[k] = 0;
            pos[k] = slot[k] = -1;
            n[k] = 0;
            page[k] = 0;
            if (k < count && t < ntok) {
                while (tok0[b + 1] <= t) ++b;  // sequences without tokens are passed
                const int s = len[b];
                seq[k] = b;
                pos[k] = s + (t - tok0[b]);
                n[k] = pos[k] + a.sees_self;
                const int held = pages_of(s + ps - 1), at = pages_of(pos[k]);
                page[k] = at < held ? a.page_table[static_cast<int64_t>(b) * a.max_pages + at]
                                    : a.free_pages[head + page0[b] + (at - held)];
            }
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < count && t0 + k < ntok) {
                if (page[k] >= 0 && page[k] < a.n_pages) slot[k] = page[k] * ps + (pos[k] - pages_of(pos[k]) * ps);
                else record_status(a.status, DSA_ERR_DEVICE_CHECK);
            }
        if (a.vec && count == 4) {
            *reinterpret_cast<int4 *>(a.q_seq + t0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
            *reinterpret_cast<int4 *>(a.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4 *>(a.q_n + t0) = make_int4(n[0], n[1], n[2], n[3]);
            *reinterpret_cast<int4 *>(a.slots + t0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
        } else {
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (k < count) {
                    a.q_seq[t0 + k] = seq[k];
                    a.positions[t0 + k] = pos[k];
                    a.q_n[t0 + k] = n[k];
                    a.slots[t0 + k] = slot[k];
                }
        }
    }
    // ---- sequences: offsets, table entries, lengths
    for (int b = gtid; b < a.nseq; b += gthreads) a.q_start[b] = refuse ? 0 : tok0[b];
    if (gtid == 0) a.q_start[a.nseq] = ntok;
    if (!refuse)
        for (int b = gtid >> 5; b < a.nseq; b += gthreads >> 5) {
            const int held = pages_of(len[b] + ps - 1), need = page0[b + 1] - page0[b];
            int32_t *row = a.page_table + static_cast<int64_t>(b) * a.max_pages;
            const int src = a.fork_src ? a.fork_src[b] : -1;
            if (src >= 0)
                copy_entries(row, a.page_table + static_cast<int64_t>(src) * a.max_pages, held, lane, [](int p) { return p; });
            copy_entries(row + held, a.free_pages + head + page0[b], need, lane,
                         [&](int p) { return p >= 0 && p < a.n_pages ? p : -1; });
        }
    const int32_t taken = refuse ? 0 : static_cast<int32_t>(total_p);
    if (a.in_place == kTabAdvanceLater) {
        if (gtid == 0) *a.taken = taken;
        return;
    }
    if (a.in_place == kTabAdvanceCluster) {
        __syncthreads();
        cluster_sync_all();
    }
    for (int b = gtid; b < a.nseq; b += gthreads)
        a.kv_len[b] = refuse ? a.seq_len[b] : len[b] + (tok0[b + 1] - tok0[b]);
    if (gtid == 0) *a.free_head_out = head + taken;
}

// The lengths and the head in place, after k13: a refused batch has offsets
// of 0 throughout, so its lengths stay.
__global__ void __launch_bounds__(kTabThreads) k13_advance(const TableParams a) {
    grid_dependency_wait();
    const int b = blockIdx.x * kTabThreads + threadIdx.x;
    if (b < a.nseq) a.kv_len[b] = a.seq_len[b] + (a.q_start[b + 1] - a.q_start[b]);
    if (b == 0) *a.free_head_out = *a.free_head + *a.taken;
}

cudaError_t launch_build_tables(const TableParams &a, int grid, cudaStream_t st) {
    const size_t smem = static_cast<size_t>(a.nseq + 1) * 12;
    if (smem > 48 * 1024 - 1024) {  // beside the kernel's static shared memory
        cudaError_t e = cudaFuncSetAttribute(k13_build_tables, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (kTabMaxSeq + 1) * 12);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kTabThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = grid;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.in_place == kTabAdvanceCluster ? 1 : 0;
    cudaError_t e = cudaLaunchKernelEx(&cfg, k13_build_tables, a);
    if (e == cudaSuccess) e = cudaGetLastError();
    if (e != cudaSuccess || a.in_place != kTabAdvanceLater) return e;
    return launch_dependent(k13_advance, a.nseq > 0 ? (a.nseq + kTabThreads - 1) / kTabThreads : 1, kTabThreads, 0, st, a);
}

}  // namespace dsa
