// serving_api.cu -- the C ABI of the serving operators declared in
// include/dsa.h: page tables and slot maps, rotary positions, the latent
// cache append, the shared-prefix attention.  Argument validation, planning
// and launches; the work is in tables.cu, rope.cu and shared_prefix.cu.
#include <cuda_runtime.h>
#include <math.h>
#include <string.h>

#include "api_util.h"
#include "dsa.h"
#include "kernels.h"
#include "serving.h"

using namespace dsa;

namespace {

int check_status_ws(void *ws, size_t ws_bytes, size_t need) {
    if (!ws) return fail(DSA_ERR_WORKSPACE, "ws is NULL");
    if (!aligned(ws, 256)) return fail(DSA_ERR_WORKSPACE, "ws must be 256-byte aligned");
    if (ws_bytes < need) return fail(DSA_ERR_WORKSPACE, "ws_bytes %zu < required %zu", ws_bytes, need);
    return DSA_OK;
}

// ------------------------------------------------- page tables and slot maps
int check_tables(const dsa_table_params *tp) {
    if (!tp) return fail(DSA_ERR_INVALID_ARG, "params is NULL");
    if (tp->nseq < 0 || tp->nseq > kTabMaxSeq) return fail(DSA_ERR_INVALID_ARG, "nseq must be in [0, %d]", kTabMaxSeq);
    if (tp->nt < 0 || tp->nt > (1 << 27)) return fail(DSA_ERR_INVALID_ARG, "nt must be in [0, 2^27]");
    if (tp->page_size < 1 || tp->page_size > 65536) return fail(DSA_ERR_INVALID_ARG, "page_size must be in [1, 65536]");
    if (tp->max_pages < 1 || static_cast<int64_t>(tp->max_pages) * tp->page_size > (int64_t(1) << 30))
        return fail(DSA_ERR_INVALID_ARG, "max_pages must be >= 1 and max_pages * page_size <= 2^30");
    if (tp->n_free < 0) return fail(DSA_ERR_INVALID_ARG, "n_free < 0");
    if (tp->sees_self != 0 && tp->sees_self != 1) return fail(DSA_ERR_INVALID_ARG, "sees_self must be 0 or 1");
    if (tp->cache_rows < 1 || tp->cache_rows >= (int64_t(1) << 31))
        return fail(DSA_ERR_INVALID_ARG, "cache_rows must be in [1, 2^31)");
    return DSA_OK;
}

// ---------------------------------------------------------- rotary positions
int check_rope(const dsa_rope_spec *rs) {
    if (!rs) return fail(DSA_ERR_INVALID_ARG, "rope spec is NULL");
    if (rs->rope_dim < 0 || rs->rope_dim > 2 * kRopeMaxPairs || (rs->rope_dim & 1))
        return fail(DSA_ERR_INVALID_ARG, "rope_dim must be even and in [0, %d]", 2 * kRopeMaxPairs);
    if (rs->layout != DSA_ROPE_INTERLEAVED && rs->layout != DSA_ROPE_HALF)
        return fail(DSA_ERR_INVALID_ARG, "unknown rope layout %d", rs->layout);
    if (rs->scaling < DSA_ROPE_SCALE_NONE || rs->scaling > DSA_ROPE_SCALE_YARN)
        return fail(DSA_ERR_INVALID_ARG, "unknown rope scaling %d", rs->scaling);
    if (!isfinite(rs->theta) || !(rs->theta > 0)) return fail(DSA_ERR_INVALID_ARG, "theta must be finite and > 0");
    if (!isfinite(rs->mscale)) return fail(DSA_ERR_INVALID_ARG, "mscale must be finite");
    if (rs->scaling != DSA_ROPE_SCALE_NONE && (!isfinite(rs->factor) || !(rs->factor > 0)))
        return fail(DSA_ERR_INVALID_ARG, "factor must be finite and > 0");
    if (rs->scaling == DSA_ROPE_SCALE_YARN &&
        (!(rs->theta > 1) || rs->orig_max_pos < 1 || !isfinite(rs->beta_fast) || !(rs->beta_slow > 0) ||
         !(rs->beta_fast >= rs->beta_slow)))
        return fail(DSA_ERR_INVALID_ARG, "YaRN needs theta > 1, orig_max_pos >= 1 and beta_fast >= beta_slow > 0");
    return DSA_OK;
}

// The speed of every pair, in turns per position.  Powers of theta for every
// eighth pair times those of the seven steps between (eleven powers for 32
// pairs, 25 ns each); products and scaling are carried in more bits and
// rounded once.  False where a speed is not finite: its sines would be NaN.
bool fill_turns(const dsa_rope_spec *rs, RopeTurns &tb) {
    constexpr double kTwoPi = 6.283185307179586476925286766559;
    constexpr int kStep = 8;
    const int rot = rs->rope_dim;
    const double d = rot;
    double theta = rs->theta;
    if (rs->scaling == DSA_ROPE_SCALE_BASE && rot > 2) theta *= pow(rs->factor, d / (d - 2.0));
    double lo = 0, hi = 0;
    if (rs->scaling == DSA_ROPE_SCALE_YARN) {
        const double span = rs->orig_max_pos / kTwoPi, two_ln = 2.0 * log(rs->theta);
        lo = floor(d * log(span / rs->beta_fast) / two_ln);
        hi = ceil(d * log(span / rs->beta_slow) / two_ln);
        if (lo < 0) lo = 0;
        if (hi > d - 1) hi = d - 1;
    }
    memset(&tb, 0, sizeof tb);
    tb.mscale = rs->mscale;
    double step[kStep] = {1.0}, anchor = 1.0;
    for (int k = 1; k < kStep && k < rot / 2; ++k) step[k] = pow(theta, -2.0 * k / d);
    for (int i = 0; i < rot / 2; ++i) {
        if (i > 0 && i % kStep == 0) anchor = pow(theta, -2.0 * i / d);
        long double f = static_cast<long double>(anchor) * step[i % kStep];
        if (rs->scaling == DSA_ROPE_SCALE_LINEAR) f /= rs->factor;
        if (rs->scaling == DSA_ROPE_SCALE_YARN) {
            const double width = hi - lo > 0.001 ? hi - lo : 0.001;
            double r = (i - lo) / width;
            r = r < 0 ? 0 : (r > 1 ? 1 : r);
            f = f * (1 - r) + f / rs->factor * r;
        }
        tb.turn[i] = static_cast<double>(f * 0.159154943091895335768883763372514362L);
        if (!(tb.turn[i] <= 1e290)) return false;
    }
    return true;
}

int rope_common(const dsa_rope_spec *rs, const dsa_rope_params *rp, const void *src, const int32_t *positions,
                void *dst, bool backward, void *stream) {
    int rc = check_rope(rs);
    if (rc) return rc;
    if (!rp) return fail(DSA_ERR_INVALID_ARG, "params is NULL");
    if (rp->nt < 0 || rp->nt > (1 << 27)) return fail(DSA_ERR_INVALID_ARG, "nt must be in [0, 2^27]");
    if (rp->h < 1 || rp->h > 65535) return fail(DSA_ERR_INVALID_ARG, "h must be in [1, 65535]");
    if (rp->x_heads != rp->h && rp->x_heads != 1) return fail(DSA_ERR_INVALID_ARG, "x_heads must be h or 1");
    if (rp->d < 1 || rp->d > 1024) return fail(DSA_ERR_INVALID_ARG, "d must be in [1, 1024]");
    if (rp->begin < 0 || rp->begin > rp->d - rs->rope_dim)
        return fail(DSA_ERR_INVALID_ARG, "[begin, begin + rope_dim) must lie in [0, d)");
    if (rp->dtype != DSA_DTYPE_BF16 && rp->dtype != DSA_DTYPE_FP16 && rp->dtype != DSA_DTYPE_FP32)
        return fail(DSA_ERR_INVALID_ARG, "unknown dtype %d", rp->dtype);
    if (rp->x_token_stride < 0 || rp->x_head_stride < 0 || rp->y_token_stride < 0 || rp->y_head_stride < 0)
        return fail(DSA_ERR_INVALID_ARG, "strides must be >= 0");
    // the rows of the side that is written are distinct: tokens outside heads
    // or heads outside tokens
    const bool shared = rp->x_heads != rp->h;
    const int64_t wt = backward ? rp->x_token_stride : rp->y_token_stride;
    const int64_t wh = backward ? rp->x_head_stride : rp->y_head_stride;
    const int64_t heads = backward ? rp->x_heads : rp->h;
    if ((heads > 1 && wh < rp->d) || (rp->nt > 1 && wt < rp->d) ||
        (heads > 1 && rp->nt > 1 && (wt < rp->d || (wt - rp->d) / (heads - 1) < wh) &&
         (wh < rp->d || (wh - rp->d) / (rp->nt - 1) < wt)))
        return fail(DSA_ERR_INVALID_ARG, "rows of the output overlap");
    if (rp->nt == 0) return DSA_OK;
    const size_t size = rp->dtype == DSA_DTYPE_FP32 ? 4 : 2;
    if (!src || !dst || !positions) return fail(DSA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(src, size) || !aligned(dst, size)) return fail(DSA_ERR_INVALID_ARG, "tensors must be aligned to their type");
    const bool in_place = src == dst;
    if (in_place && (shared || rp->x_token_stride != rp->y_token_stride || rp->x_head_stride != rp->y_head_stride))
        return fail(DSA_ERR_INVALID_ARG, "in place needs x_heads = h and equal strides");
    if (int frc = host_fault("rope")) return frc;
    RopeParams a;
    memset(&a, 0, sizeof a);
    a.x = src;
    a.y = dst;
    a.positions = positions;
    a.xt = backward ? rp->y_token_stride : rp->x_token_stride;
    a.xh = backward ? rp->y_head_stride : rp->x_head_stride;
    a.yt = backward ? rp->x_token_stride : rp->y_token_stride;
    a.yh = backward ? rp->x_head_stride : rp->y_head_stride;
    a.nt = rp->nt;
    a.h = rp->h;
    a.begin = rp->begin;
    a.rot = rs->rope_dim;
    a.d = rp->d;
    a.in_place = in_place;
    a.transpose = backward;
    if (!fill_turns(rs, a.tb)) return fail(DSA_ERR_INVALID_ARG, "theta and factor give speeds that are not finite");
    const int v = static_cast<int>(16 / size);
    const bool half = rs->layout == DSA_ROPE_HALF;
    const bool vec = aligned(src, 16) && aligned(dst, 16) && a.xt % v == 0 && a.xh % v == 0 && a.yt % v == 0 &&
                     a.yh % v == 0 && a.begin % v == 0 && a.d % v == 0 && a.rot % (half ? 2 * v : v) == 0;
    cudaError_t e = launch_rope(a, rp->dtype, half, vec, !shared ? 0 : (backward ? 2 : 1), static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "rotary positions launch");
    return DSA_OK;
}

int append_common(const dsa_rope_spec *rs, int32_t nt, const void *c_kv, int64_t c_stride, const void *k_pe,
                  int64_t pe_stride, const int32_t *positions, const int32_t *slots, void *cache, int64_t row_stride,
                  float *kv_scale, bool fp8, int64_t cache_rows, void *ws, size_t ws_bytes, void *stream) {
    int rc = check_rope(rs);
    if (rc) return rc;
    if (rs->rope_dim != kRopeRow) return fail(DSA_ERR_UNSUPPORTED, "the rope part of a latent row is %d wide", kRopeRow);
    if (nt < 0 || nt > (1 << 27)) return fail(DSA_ERR_INVALID_ARG, "nt must be in [0, 2^27]");
    if (cache_rows < 1 || cache_rows >= (int64_t(1) << 31)) return fail(DSA_ERR_INVALID_ARG, "cache_rows must be in [1, 2^31)");
    const int64_t unit = fp8 ? 16 : 8;
    if (row_stride < kDqk || row_stride % unit != 0)
        return fail(DSA_ERR_INVALID_ARG, "cache rows must be >= 576 apart, a multiple of %d", static_cast<int>(unit));
    rc = check_status_ws(ws, ws_bytes, DSA_WS_STATUS_BYTES);
    if (rc) return rc;
    if (nt == 0) return DSA_OK;
    if (!c_kv || !k_pe || !positions || !slots || !cache || (fp8 && !kv_scale))
        return fail(DSA_ERR_INVALID_ARG, "a required pointer is NULL");
    if (!aligned(c_kv, 16) || !aligned(k_pe, 16) || !aligned(cache, 16))
        return fail(DSA_ERR_INVALID_ARG, "c_kv, k_pe and the cache must be 16-byte aligned");
    if (nt > 1 && (c_stride < kLatent || pe_stride < kRopeRow))
        return fail(DSA_ERR_INVALID_ARG, "rows of c_kv or k_pe overlap");
    if (nt > 1 && (c_stride % 8 != 0 || pe_stride % 8 != 0)) return fail(DSA_ERR_INVALID_ARG, "input strides must be multiples of 8");
    if (int frc = host_fault("append")) return frc;
    AppendParams a;
    memset(&a, 0, sizeof a);
    a.c_kv = static_cast<const uint16_t *>(c_kv);
    a.k_pe = static_cast<const uint16_t *>(k_pe);
    a.c_stride = c_stride;
    a.pe_stride = pe_stride;
    a.positions = positions;
    a.slots = slots;
    a.cache = cache;
    a.row_stride = row_stride;
    a.kv_scale = kv_scale;
    a.cache_rows = cache_rows;
    a.nt = nt;
    a.half_layout = rs->layout == DSA_ROPE_HALF;
    a.status = at<int>(ws, 0);
    if (!fill_turns(rs, a.tb)) return fail(DSA_ERR_INVALID_ARG, "theta and factor give speeds that are not finite");
    cudaError_t e = launch_latent_append(a, fp8, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "latent append launch");
    return DSA_OK;
}

// ------------------------------------------------- shared-prefix attention
int check_prefix(const dsa_params *p, const dsa_kv *kv, int32_t ngroups) {
    int rc = check_params(p);
    if (!rc) rc = check_kv(p, kv);
    if (rc) return rc;
    if (p->nq > kPfxMaxQueries)
        return fail(DSA_ERR_UNSUPPORTED, "shared-prefix attention takes at most %d queries", kPfxMaxQueries);
    if (p->nq > 0 && (ngroups < 1 || ngroups > kPfxMaxGroups))
        return fail(DSA_ERR_INVALID_ARG, "ngroups must be in [1, %d]", kPfxMaxGroups);
    return DSA_OK;
}

struct PrefixLayout {
    size_t cut, tiles, q_shared, q_own, part_o, part_lse, total;
    int pairs;
};

PrefixLayout plan_prefix(const dsa_params *p, int32_t ngroups) {
    PrefixLayout w;
    memset(&w, 0, sizeof w);
    w.pairs = num_sms() / 2 < kPfxMaxPairs ? num_sms() / 2 : kPfxMaxPairs;
    // row tiles: each group's rows in 128s, and one for every query's own part
    const int64_t full = (static_cast<int64_t>(p->nq) * p->h) / kPfxRows;
    const int64_t groups = ngroups < p->nq ? ngroups : p->nq;
    const size_t row_tiles = static_cast<size_t>(full + groups + p->nq);
    const size_t slots = row_tiles + static_cast<size_t>(w.pairs);
    size_t off = DSA_WS_STATUS_BYTES;
    w.cut = off;
    off = up(off + static_cast<size_t>(w.pairs + 1) * 8, 256);
    w.tiles = off;
    off = up(off + row_tiles * sizeof(PrefixTile), 256);
    w.q_shared = off;
    off = up(off + static_cast<size_t>(p->nq) * 4, 256);
    w.q_own = off;
    off = up(off + static_cast<size_t>(p->nq) * 4, 256);
    w.part_o = off;
    off = up(off + slots * kPfxRows * kDv * 4, 256);
    w.part_lse = off;
    off = up(off + slots * kPfxRows * 4, 256);
    w.total = off;
    return w;
}

}  // namespace

extern "C" {

int dsa_table_workspace_size(const dsa_table_params *tp, size_t *bytes) {
    int rc = check_tables(tp);
    if (rc) return rc;
    if (!bytes) return fail(DSA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 512;  // status word; pages handed out
    return DSA_OK;
}

int dsa_build_tables(const dsa_table_params *tp, const int32_t *seq_len, const int32_t *new_len,
                     const int32_t *fork_src, const int32_t *free_pages, const int32_t *free_head,
                     int32_t *page_table, int32_t *q_start, int32_t *q_seq, int32_t *positions, int32_t *q_n,
                     int32_t *slots, int32_t *kv_len, int32_t *free_head_out, void *ws, size_t ws_bytes,
                     void *stream) {
    int rc = check_tables(tp);
    if (!rc) rc = check_status_ws(ws, ws_bytes, 512);
    if (rc) return rc;
    if (!q_start || !free_head || !free_head_out) return fail(DSA_ERR_INVALID_ARG, "q_start / free_head / free_head_out is NULL");
    if (tp->nseq > 0 && (!seq_len || !new_len || !page_table || !kv_len))
        return fail(DSA_ERR_INVALID_ARG, "seq_len / new_len / page_table / kv_len is NULL");
    if (tp->n_free > 0 && !free_pages) return fail(DSA_ERR_INVALID_ARG, "free_pages is NULL");
    if (tp->nt > 0 && (!q_seq || !positions || !q_n || !slots))
        return fail(DSA_ERR_INVALID_ARG, "q_seq / positions / q_n / slots is NULL");
    if (int frc = host_fault("tables")) return frc;
    TableParams a;
    memset(&a, 0, sizeof a);
    a.seq_len = seq_len;
    a.new_len = new_len;
    a.fork_src = fork_src;
    a.free_pages = free_pages;
    a.free_head = free_head;
    a.page_table = page_table;
    a.q_start = q_start;
    a.q_seq = q_seq;
    a.positions = positions;
    a.q_n = q_n;
    a.slots = slots;
    a.kv_len = kv_len;
    a.free_head_out = free_head_out;
    a.nseq = tp->nseq;
    a.nt = tp->nt;
    a.page_size = tp->page_size;
    a.max_pages = tp->max_pages;
    a.n_free = tp->n_free;
    a.sees_self = tp->sees_self;
    a.page_shift = -1;
    for (int i = 0; i <= 16; ++i)
        if (tp->page_size == 1 << i) a.page_shift = i;
    a.vec = aligned(q_seq, 16) && aligned(positions, 16) && aligned(q_n, 16) && aligned(slots, 16);
    a.n_pages = tp->cache_rows / tp->page_size;
    a.status = at<int>(ws, 0);
    a.taken = at<int32_t>(ws, 256);
    // a CTA for every 2048 tokens or 64 sequences, at most one per SM
    const int by_tokens = (tp->nt + 4 * kTabThreads - 1) / (4 * kTabThreads), by_seqs = (tp->nseq + 63) / 64;
    int grid = by_tokens > by_seqs ? by_tokens : by_seqs;
    grid = grid < 1 ? 1 : (grid > num_sms() ? num_sms() : grid);
    if (kv_len == seq_len || free_head_out == free_head) {
        a.in_place = grid <= kTabCluster ? kTabAdvanceCluster : kTabAdvanceLater;
        if (grid <= kTabCluster)
            for (int g = 1; g < 2 * kTabCluster; g *= 2)  // a cluster of 1, 2, 4 or 8
                if (g >= grid) {
                    grid = g;
                    break;
                }
    }
    cudaError_t e = launch_build_tables(a, grid, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "page table launch");
    return DSA_OK;
}

int dsa_rope(const dsa_rope_spec *rs, const dsa_rope_params *rp, const void *x, const int32_t *positions, void *y,
             void *stream) {
    return rope_common(rs, rp, x, positions, y, false, stream);
}

int dsa_rope_backward(const dsa_rope_spec *rs, const dsa_rope_params *rp, const void *dy, const int32_t *positions,
                      void *dx, void *stream) {
    return rope_common(rs, rp, dy, positions, dx, true, stream);
}

int dsa_latent_append(const dsa_rope_spec *rs, int32_t nt, const void *c_kv, int64_t c_kv_stride, const void *k_pe,
                      int64_t k_pe_stride, const int32_t *positions, const int32_t *slots, void *kv_cache,
                      int64_t kv_row_stride, int64_t cache_rows, void *ws, size_t ws_bytes, void *stream) {
    return append_common(rs, nt, c_kv, c_kv_stride, k_pe, k_pe_stride, positions, slots, kv_cache, kv_row_stride,
                         nullptr, false, cache_rows, ws, ws_bytes, stream);
}

int dsa_latent_append_fp8(const dsa_rope_spec *rs, int32_t nt, const void *c_kv, int64_t c_kv_stride,
                          const void *k_pe, int64_t k_pe_stride, const int32_t *positions, const int32_t *slots,
                          void *kv8_cache, int64_t kv8_row_bytes, float *kv_scale, int64_t cache_rows, void *ws,
                          size_t ws_bytes, void *stream) {
    return append_common(rs, nt, c_kv, c_kv_stride, k_pe, k_pe_stride, positions, slots, kv8_cache, kv8_row_bytes,
                         kv_scale, true, cache_rows, ws, ws_bytes, stream);
}

int dsa_shared_prefix_workspace_size(const dsa_params *p, const dsa_kv *kv, int32_t ngroups, size_t *bytes) {
    int rc = check_prefix(p, kv, ngroups);
    if (rc) return rc;
    if (!bytes) return fail(DSA_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = plan_prefix(p, ngroups).total;
    return DSA_OK;
}

int dsa_mla_shared_prefix(const dsa_params *p, const dsa_kv *kv, int32_t ngroups, const int32_t *group_q0,
                          const int32_t *group_n, const void *q, const void *kv_cache, int64_t kv_row_stride,
                          void *out, float *lse, void *ws, size_t ws_bytes, void *stream) {
    int rc = check_prefix(p, kv, ngroups);
    if (rc) return rc;
    const PrefixLayout w = plan_prefix(p, ngroups);
    rc = check_status_ws(ws, ws_bytes, w.total);
    if (rc) return rc;
    if (p->nq == 0) return DSA_OK;
    if (!group_q0 || !group_n || !q || !kv_cache || !out || !lse)
        return fail(DSA_ERR_INVALID_ARG, "group_q0 / group_n / q / kv_cache / out / lse is NULL");
    if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16))
        return fail(DSA_ERR_INVALID_ARG, "q / kv_cache / out must be 16-byte aligned");
    if (kv_row_stride < kDqk || kv_row_stride % 8 != 0)
        return fail(DSA_ERR_INVALID_ARG, "kv_row_stride must be >= 576 and a multiple of 8");
    if (int frc = host_fault("shared_prefix")) return frc;
    PrefixParams a;
    memset(&a, 0, sizeof a);
    a.q_seq = kv->q_seq;
    a.q_n = kv->q_n;
    a.seq_row0 = kv->seq_row0;
    a.page_table = kv->page_table;
    a.max_pages = kv->max_pages;
    a.page_shift = kv->page_size == 128 ? 7 : 6;
    a.cache_rows = kv->cache_rows;
    a.group_q0 = group_q0;
    a.group_n = group_n;
    a.ngroups = ngroups;
    a.nq = p->nq;
    a.h = p->h;
    a.max_n = p->max_n;
    a.pairs = w.pairs;
    a.scale_log2 = p->scale * 1.4426950408889634f;
    a.out = static_cast<uint16_t *>(out);
    a.lse = lse;
    a.cut = at<int64_t>(ws, w.cut);
    a.tiles = at<PrefixTile>(ws, w.tiles);
    a.q_shared = at<int32_t>(ws, w.q_shared);
    a.q_own = at<int32_t>(ws, w.q_own);
    a.part_o = at<float>(ws, w.part_o);
    a.part_lse = at<float>(ws, w.part_lse);
    a.status = at<int>(ws, 0);
    a.wait_budget = kWaitBudgetCycles;
    if (inject_timeout("shared_prefix")) {
        a.wait_budget = kTestWaitBudget;
        a.inject = 1;
    }
    // boxes of 64 rows x 64 columns: one swizzled chunk
    CUtensorMap qmap, kmap, vmap;
    rc = make_map_2d(&qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, q, kDqk, static_cast<uint64_t>(p->nq) * p->h, kDqk * 2, 64,
                     64, CU_TENSOR_MAP_SWIZZLE_128B);
    if (!rc)
        rc = make_map_2d(&kmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kv_cache, kDqk, static_cast<uint64_t>(kv->cache_rows),
                         static_cast<uint64_t>(kv_row_stride) * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
    // the value columns in blocks of 64, two blocks a box
    if (!rc)
        rc = make_map_3d(&vmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, kv_cache,
                         {64, static_cast<uint64_t>(kv->cache_rows), kDv / 64},
                         {static_cast<uint64_t>(kv_row_stride) * 2, 128}, {64, 64, 2}, CU_TENSOR_MAP_SWIZZLE_128B);
    if (rc) return rc;
    cudaError_t e = launch_shared_prefix(qmap, kmap, vmap, a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "shared-prefix attention launch");
    return DSA_OK;
}

}  // extern "C"
