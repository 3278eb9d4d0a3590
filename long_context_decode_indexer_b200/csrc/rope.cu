// rope.cu -- rotary positions and the latent cache append.
//
// Pair i of a head turns by the angle pos * f_i.  The host passes f_i / 2 pi
// in 64 bits (the scaling for long contexts is all in these numbers), so a
// thread gets an angle from one 64-bit product.  The speed's own rounding and
// the product's leave a few 2^-53 of the angle: 2e-8 rad at position 2^27 and
// f = 1, a third of an fp32 step.  sincospif takes its fractional part rounded
// to fp32, and what that rounding left out (up to 9e-8 rad) turns the result
// once more, to first order.  No table of cosines is read or kept.
//
// All three kernels move bytes and little else: the floor is x read and y
// written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "api_util.h"
#include "dsa.h"
#include "ptx.cuh"
#include "serving.h"

namespace dsa {

namespace {

template <class T>
__device__ __forceinline__ float to_f(T v);
template <>
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f(float v) { return v; }
template <class T>
__device__ __forceinline__ T from_f(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_f(float v) { return v; }

// N adjacent elements, as one 16-byte access (N * sizeof(T) == 16) or one by one.
template <class T, int N>
struct alignas(N * sizeof(T) == 16 ? 16 : sizeof(T)) Pack {
    T v[N];
};
template <class T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T *p) {
    Pack<T, N> r;
    if constexpr (N * sizeof(T) == 16) {
        *reinterpret_cast<uint4 *>(&r) = __ldcg(reinterpret_cast<const uint4 *>(p));  // no reuse: not through L1
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) r.v[i] = p[i];
    }
    return r;
}
template <class T, int N>
__device__ __forceinline__ void store_pack(T *p, const Pack<T, N> &r) {
    if constexpr (N * sizeof(T) == 16) {
        __stcg(reinterpret_cast<uint4 *>(p), *reinterpret_cast<const uint4 *>(&r));
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) p[i] = r.v[i];
    }
}

// sin and cos of pos * turn turns.
__device__ __forceinline__ void turn_sincos(int pos, double turn, float &s, float &c) {
    const double t = static_cast<double>(pos) * turn, half_turns = 2.0 * (t - rint(t));
    const float near = static_cast<float>(half_turns);
    float s0, c0;
    sincospif(near, &s0, &c0);
    const float rest = static_cast<float>(half_turns - near) * 3.14159265f;  // radians
    s = fmaf(c0, rest, s0);
    c = fmaf(-s0, rest, c0);
}

}  // namespace

// A head is cut into units.  A rotated unit is P pairs: 2P adjacent elements
// (interleaved), or P elements at i and P at i + rot / 2 (half); every other
// unit is W adjacent elements to copy.  With 16-byte accesses W is one of
// them; the element form (P = W = 1) serves every other alignment.
template <class T, bool HALF, bool VEC>
struct RopeShape {
    static constexpr int kVec = 16 / sizeof(T);
    static constexpr int P = VEC ? (HALF ? kVec : kVec / 2) : 1;
    static constexpr int W = VEC ? kVec : 1;
    static constexpr int N0 = HALF ? P : 2 * P;  // elements of a rotated unit's first access
};
constexpr int kRopeThreads = 256;
constexpr int kRopeMaxTokens = 32;  // of a block of k14

// First element of unit u: rotated units first, then the copied ones in order.
template <class S>
__device__ __forceinline__ int unit_offset(const RopeParams &a, int u) {
    if (u < a.units_rope) return a.begin + u * S::N0;
    const int e = (u - a.units_rope) * S::W;
    return e < a.begin ? e : e + a.rot;
}

// The sines and cosines of a block's tokens, times mscale: table[token][pair].
__device__ __forceinline__ void fill_table(float2 *table, const RopeParams &a, int64_t t0, int tokens) {
    const int pairs = a.rot / 2;
    const float ms = static_cast<float>(a.tb.mscale);
    for (int i = threadIdx.x; i < tokens * pairs; i += blockDim.x) {
        const int64_t t = t0 + i / pairs;
        if (t >= a.nt) break;
        float s, c;
        turn_sincos(a.positions[t], a.tb.turn[i % pairs], s, c);
        table[i] = make_float2(c * ms, a.transpose ? -s * ms : s * ms);
    }
}

// k14: y = R x head by head, or (SHARED) one source head to every head of y.
// A thread keeps one unit of one token over its heads (hp heads apart), so
// its sines stay in registers; consecutive threads take consecutive units,
// then heads, then tokens, so that a step covers adjacent memory.  The sines
// are computed once a block, while the first loads are in flight: threads
// that computed their own spent more on them than on their bytes (92 us
// instead of 43 for 8191 x 128 x 64 bf16 in place; the bytes take 42).
template <class T, bool HALF, bool VEC, bool SHARED>
__global__ void __launch_bounds__(kRopeThreads) k14_rope(const __grid_constant__ RopeParams a) {
    using S = RopeShape<T, HALF, VEC>;
    constexpr int P = S::P, W = S::W, N0 = S::N0;
    constexpr int kAhead = 4;
    extern __shared__ float2 table[];
    __shared__ bool padding[kRopeMaxTokens];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tp;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tp), a.nt - t0));
    const int u = blockIdx.z * kRopeThreads + threadIdx.x % a.ub;
    const int r = threadIdx.x / a.ub, ts = r / a.hp;
    const bool live = ts < tokens && u < a.units;
    const bool rope = u < a.units_rope;
    const int h0 = blockIdx.y * (a.hp * a.iters) + r % a.hp;
    const int h_end = live ? min(a.h, static_cast<int>(blockIdx.y + 1) * a.hp * a.iters) : 0;
    const int e = unit_offset<S>(a, u);
    const T *x = static_cast<const T *>(a.x) + (t0 + ts) * a.xt + e;
    T *y = static_cast<T *>(a.y) + (t0 + ts) * a.yt + e;
    Pack<T, N0> v0[kAhead];
    Pack<T, HALF ? P : 1> v1[kAhead];
    auto load = [&](int h) {
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (h + k * a.hp < h_end) {
                const T *src = x + (SHARED ? 0 : (h + k * a.hp) * a.xh);
                if (rope) {
                    v0[k] = load_pack<T, N0>(src);
                    if constexpr (HALF) v1[k] = load_pack<T, P>(src + a.rot / 2);
                } else {
                    *reinterpret_cast<Pack<T, W> *>(&v0[k]) = load_pack<T, W>(src);
                }
            }
    };
    load(h0);
    fill_table(table, a, t0, tokens);
    if (threadIdx.x < tokens) padding[threadIdx.x] = a.positions[t0 + threadIdx.x] < 0;
    __syncthreads();
    if (!live) return;
    // padding: left as it was (forward) or zeros (gradient); in place the
    // elements to copy are there already
    const bool pad = padding[ts];
    if (pad ? !a.transpose : (!rope && a.in_place)) return;
    float2 cs[P];
    if (rope) {
#pragma unroll
        for (int p = 0; p < P; ++p) cs[p] = table[ts * (a.rot / 2) + u * P + p];
    }
    for (int h = h0; h < h_end; h += kAhead * a.hp) {
        if (h != h0) load(h);
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            if (h + k * a.hp >= h_end) break;
            T *dst = y + (h + k * a.hp) * a.yh;
            if (!rope) {
                store_pack(dst, pad ? Pack<T, W>{} : *reinterpret_cast<const Pack<T, W> *>(&v0[k]));
                continue;
            }
#pragma unroll
            for (int p = 0; p < P; ++p) {
                T &p0 = HALF ? v0[k].v[p] : v0[k].v[2 * p];
                T &p1 = HALF ? v1[k].v[HALF ? p : 0] : v0[k].v[HALF ? 0 : 2 * p + 1];
                const float a0 = to_f(p0), a1 = to_f(p1);
                p0 = from_f<T>(pad ? 0.f : a0 * cs[p].x - a1 * cs[p].y);
                p1 = from_f<T>(pad ? 0.f : a0 * cs[p].y + a1 * cs[p].x);
            }
            store_pack(dst, v0[k]);
            if constexpr (HALF) store_pack(dst + a.rot / 2, v1[k]);
        }
    }
}

// k14 for heads that are adjacent in memory but whose rotated range does not
// start or end on 16 bytes (or whose width is odd): a block moves the whole
// heads [h0, h0 + hp) of a token through shared memory, in and out by 16
// bytes, and turns the pairs there.  11473 x 64 x 128 fp16 with 86 rotated:
// 94 us, element by element 308.
template <class T, bool HALF>
__global__ void __launch_bounds__(kRopeThreads) k14_rope_staged(const __grid_constant__ RopeParams a) {
    extern __shared__ float2 table[];  // [pairs], then the heads
    constexpr int kVec = 16 / sizeof(T);
    const int pairs = a.rot / 2;
    T *buf = reinterpret_cast<T *>(reinterpret_cast<uint8_t *>(table) + (pairs * 8 + 15) / 16 * 16);
    const int64_t t = blockIdx.x;
    const int h0 = blockIdx.y * a.hp, heads = min(a.hp, a.h - h0), span = heads * a.d;
    const int pos = a.positions[t];
    if (pos < 0 && !a.transpose) return;
    const T *x = static_cast<const T *>(a.x) + t * a.xt + static_cast<int64_t>(h0) * a.d;
    T *y = static_cast<T *>(a.y) + t * a.yt + static_cast<int64_t>(h0) * a.d;
    if (pos < 0) {
        for (int i = threadIdx.x; i < span; i += kRopeThreads) y[i] = from_f<T>(0.f);
        return;
    }
    const int whole = span / kVec;
#pragma unroll 4
    for (int i = threadIdx.x; i < whole; i += kRopeThreads)
        reinterpret_cast<uint4 *>(buf)[i] = __ldcg(reinterpret_cast<const uint4 *>(x) + i);
    for (int i = whole * kVec + threadIdx.x; i < span; i += kRopeThreads) buf[i] = x[i];
    fill_table(table, a, t, 1);
    __syncthreads();
    for (int i = threadIdx.x; i < heads * pairs; i += kRopeThreads) {
        const int h = i / pairs, p = i - h * pairs;
        T *e = buf + h * a.d + a.begin;
        T &p0 = e[HALF ? p : 2 * p], &p1 = e[HALF ? p + pairs : 2 * p + 1];
        const float2 cs = table[p];
        const float a0 = to_f(p0), a1 = to_f(p1);
        p0 = from_f<T>(a0 * cs.x - a1 * cs.y);
        p1 = from_f<T>(a0 * cs.y + a1 * cs.x);
    }
    __syncthreads();
#pragma unroll 4
    for (int i = threadIdx.x; i < whole; i += kRopeThreads)
        __stcg(reinterpret_cast<uint4 *>(y) + i, reinterpret_cast<const uint4 *>(buf)[i]);
    for (int i = whole * kVec + threadIdx.x; i < span; i += kRopeThreads) y[i] = buf[i];
}

// k15: the gradient of a head that all heads share: dx = R^T sum_h dy_h.  The
// turn is linear and the same for every head, so the heads are summed first
// and turned once: hp threads a unit each sum their heads in order (fp32), a
// thread per element adds the hp partial sums in order, and one thread a unit
// turns the result.
template <class T, bool HALF, bool VEC>
__global__ void __launch_bounds__(kRopeThreads) k15_rope_sum(const __grid_constant__ RopeParams a) {
    using S = RopeShape<T, HALF, VEC>;
    constexpr int P = S::P, W = S::W, N0 = S::N0;
    extern __shared__ float2 table[];  // [tp][pairs], then float sums [tp][hp][d]
    float *sums = reinterpret_cast<float *>(table + a.tp * (a.rot / 2));
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * a.tp;
    const int tokens = static_cast<int>(min(static_cast<int64_t>(a.tp), a.nt - t0));
    for (int i = threadIdx.x; i < tokens * a.hp * a.units; i += kRopeThreads) {
        const int u = i % a.units, part = i / a.units % a.hp, t = i / a.units / a.hp;
        const bool rope = u < a.units_rope;
        const int e = unit_offset<S>(a, u);
        float acc[2 * P];
#pragma unroll
        for (int k = 0; k < 2 * P; ++k) acc[k] = 0.f;
        if (a.positions[t0 + t] >= 0) {
            const T *x = static_cast<const T *>(a.x) + (t0 + t) * a.xt + e;
            if (rope) {
#pragma unroll (VEC ? 4 : 16)
                for (int h = part; h < a.h; h += a.hp) {
                    const Pack<T, N0> v = load_pack<T, N0>(x + h * a.xh);
#pragma unroll
                    for (int k = 0; k < N0; ++k) acc[k] += to_f(v.v[k]);
                    if constexpr (HALF) {
                        const Pack<T, P> w = load_pack<T, P>(x + h * a.xh + a.rot / 2);
#pragma unroll
                        for (int k = 0; k < P; ++k) acc[P + k] += to_f(w.v[k]);
                    }
                }
            } else {
#pragma unroll (VEC ? 4 : 16)
                for (int h = part; h < a.h; h += a.hp) {
                    const Pack<T, W> v = load_pack<T, W>(x + h * a.xh);
#pragma unroll
                    for (int k = 0; k < W; ++k) acc[k] += to_f(v.v[k]);
                }
            }
        }
        float *row = sums + (t * a.hp + part) * a.d;
        if (rope) {
#pragma unroll
            for (int k = 0; k < 2 * P; ++k) row[HALF && k >= P ? e + a.rot / 2 + k - P : e + k] = acc[k];
        } else {
#pragma unroll
            for (int k = 0; k < W; ++k) row[e + k] = acc[k];
        }
    }
    fill_table(table, a, t0, tokens);
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * a.d; i += kRopeThreads) {
        float *col = sums + (i / a.d) * a.hp * a.d + i % a.d;
        float sum = col[0];
        for (int p = 1; p < a.hp; ++p) sum += col[p * a.d];
        col[0] = sum;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < tokens * a.units; i += kRopeThreads) {
        const int u = i % a.units, t = i / a.units, e = unit_offset<S>(a, u);
        const float *row = sums + t * a.hp * a.d;
        T *y = static_cast<T *>(a.y) + (t0 + t) * a.yt + e;
        if (u >= a.units_rope) {
            Pack<T, W> v;
#pragma unroll
            for (int k = 0; k < W; ++k) v.v[k] = from_f<T>(row[e + k]);
            store_pack(y, v);
            continue;
        }
        Pack<T, N0> v0;
        Pack<T, HALF ? P : 1> v1;
        const bool pad = a.positions[t0 + t] < 0;
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const float2 cs = table[t * (a.rot / 2) + u * P + p];
            const int e0 = HALF ? e + p : e + 2 * p, e1 = HALF ? e + a.rot / 2 + p : e + 2 * p + 1;
            const T d0 = from_f<T>(pad ? 0.f : row[e0] * cs.x - row[e1] * cs.y);
            const T d1 = from_f<T>(pad ? 0.f : row[e0] * cs.y + row[e1] * cs.x);
            if constexpr (HALF) {
                v0.v[p] = d0;
                v1.v[p] = d1;
            } else {
                v0.v[2 * p] = d0;
                v0.v[2 * p + 1] = d1;
            }
        }
        store_pack(y, v0);
        if constexpr (HALF) store_pack(y + a.rot / 2, v1);
    }
}

namespace {

template <class T, bool HALF, bool VEC>
cudaError_t launch_rope_t(RopeParams a, int shared, cudaStream_t st) {
    using S = RopeShape<T, HALF, VEC>;
    a.units_rope = a.rot / 2 / S::P;
    // in place only the rotated range moves (a padding token's gradient is
    // cleared whole)
    a.units = a.units_rope + (a.in_place && !a.transpose ? 0 : (a.d - a.rot) / S::W);
    if (a.units == 0) return cudaSuccess;
    if (shared == 2) {
        a.hp = kRopeThreads / a.units < 1 ? 1 : (kRopeThreads / a.units > a.h ? a.h : kRopeThreads / a.units);
        // few threads a unit where there are many tokens (4, 8, 32: 29, 31, 45
        // us for 8191 x 128 x 64 bf16), many where there are few
        const int most = static_cast<int64_t>(a.nt) * a.units < num_sms() * kRopeThreads / 8 ? 32 : 4;
        if (a.hp > most) a.hp = most;
        a.tp = kRopeThreads / (a.units * a.hp) < 1 ? 1 : kRopeThreads / (a.units * a.hp);
        const int64_t grid = (static_cast<int64_t>(a.nt) + a.tp - 1) / a.tp;
        // at most 48 KB: tp * hp * units <= 256 threads (or one row of 1024)
        // of up to 16 sums each, and tp tables of 1 KB
        const size_t smem = static_cast<size_t>(a.tp) * (a.rot / 2 * 8 + static_cast<size_t>(a.hp) * a.d * 4);
        k15_rope_sum<T, HALF, VEC><<<static_cast<unsigned>(grid), kRopeThreads, smem, st>>>(a);
        return cudaGetLastError();
    }
    if constexpr (!VEC) {
        // heads of about 8 KB a block, a number of them that is whole 16 bytes
        const int64_t head = static_cast<int64_t>(a.d) * sizeof(T);
        int step = 1;
        while (head * step % 16 != 0) step *= 2;
        const bool dense = (a.h == 1 || (a.xh == a.d && a.yh == a.d)) &&
                           (a.nt == 1 || (a.xt * sizeof(T) % 16 == 0 && a.yt * sizeof(T) % 16 == 0)) &&
                           reinterpret_cast<uintptr_t>(a.x) % 16 == 0 && reinterpret_cast<uintptr_t>(a.y) % 16 == 0;
        // in place only where most of a head is rotated
        if (shared == 0 && dense && a.rot > 0 && (!a.in_place || 2 * a.rot >= a.d)) {
            const int64_t fit = 8192 / (head * step) * step;
            a.hp = static_cast<int>(fit < step ? step : (fit > a.h ? a.h : fit));
            const size_t smem = (a.rot / 2 * 8 + 15) / 16 * 16 + static_cast<size_t>(a.hp) * head;
            k14_rope_staged<T, HALF><<<dim3(a.nt, (a.h + a.hp - 1) / a.hp), kRopeThreads, smem, st>>>(a);
            return cudaGetLastError();
        }
    }
    a.ub = a.units < kRopeThreads ? a.units : kRopeThreads;
    const int gz = (a.units + kRopeThreads - 1) / kRopeThreads;
    // blocks of about 128 threads of four heads each: one batch of loads, and
    // many blocks on an SM at different points of it (256 threads of 16 heads
    // took 90 us for 4096 x 128 x 192 bf16, these 76)
    const int room = a.ub < 128 ? 128 / a.ub : 1;  // heads x tokens a step
    a.hp = room < a.h ? room : a.h;
    a.tp = room / a.hp < kRopeMaxTokens ? room / a.hp : kRopeMaxTokens;
    const int64_t gx = (static_cast<int64_t>(a.nt) + a.tp - 1) / a.tp;
    int iters = (a.h + a.hp - 1) / a.hp;  // fewer than four heads while the grid is small
    if (iters > 4) iters = 4;
    while (iters > 1 && gx * gz * ((a.h + a.hp * iters - 1) / (a.hp * iters)) < num_sms() * 4) iters = (iters + 1) / 2;
    a.iters = iters;
    const dim3 grid(static_cast<unsigned>(gx), static_cast<unsigned>((a.h + a.hp * iters - 1) / (a.hp * iters)), gz);
    const int threads = a.ub * a.hp * a.tp;
    const size_t smem = static_cast<size_t>(a.tp) * (a.rot / 2) * 8;
    if (shared == 1) k14_rope<T, HALF, VEC, true><<<grid, threads, smem, st>>>(a);
    else k14_rope<T, HALF, VEC, false><<<grid, threads, smem, st>>>(a);
    return cudaGetLastError();
}

template <class T>
cudaError_t launch_rope_d(const RopeParams &a, bool half, bool vec, int shared, cudaStream_t st) {
    if (half) return vec ? launch_rope_t<T, true, true>(a, shared, st) : launch_rope_t<T, true, false>(a, shared, st);
    return vec ? launch_rope_t<T, false, true>(a, shared, st) : launch_rope_t<T, false, false>(a, shared, st);
}

}  // namespace

cudaError_t launch_rope(const RopeParams &a, int dtype, bool half_layout, bool vec, int shared, cudaStream_t st) {
    if (dtype == DSA_DTYPE_BF16) return launch_rope_d<__nv_bfloat16>(a, half_layout, vec, shared, st);
    if (dtype == DSA_DTYPE_FP16) return launch_rope_d<__half>(a, half_layout, vec, shared, st);
    return launch_rope_d<float>(a, half_layout, vec, shared, st);
}

// ---------------------------------------------------------------------------
// k16: one warp appends one token's latent row.  Lane l moves c_kv elements
// [16 l, 16 l + 16) (two 16-byte loads) and turns pair l of the rope part.
// FP8: the row's amax by a warp reduction, its scale the smallest power of
// two with amax / s <= 448.
// ---------------------------------------------------------------------------
namespace {

// 2^e with amax / 2^e <= 448, e as small as possible and at least -126, from
// the bits of amax: 448 is 1.75 * 2^8.
__device__ __forceinline__ float row_scale(float amax) {
    if (!(amax > 0.f)) return 1.f;
    const uint32_t bits = __float_as_uint(amax);
    const int e = static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, -126) + 127) << 23);
}

// v in fp32 with its lost bits folded into the last one (round to odd), so
// that a later rounding to few bits is that of v itself.
__device__ __forceinline__ float odd_float(double v) {
    const float f = __double2float_rz(v);
    return static_cast<double>(f) == v ? f : __uint_as_float(__float_as_uint(f) | 1u);
}

__device__ __forceinline__ uint32_t e4m3_pair(float lo, float hi) {
    return static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}

}  // namespace

template <bool FP8>
__global__ void __launch_bounds__(128) k16_latent_append(const __grid_constant__ AppendParams a) {
    const int t = blockIdx.x * 4 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= a.nt) return;
    // every load is issued before the slot is looked at
    const int slot = a.slots[t], pos = a.positions[t];
    const uint4 *cp = reinterpret_cast<const uint4 *>(a.c_kv + static_cast<int64_t>(t) * a.c_stride) + 2 * lane;
    const uint4 c0 = __ldcg(cp), c1 = __ldcg(cp + 1);
    const uint16_t *pe = a.k_pe + static_cast<int64_t>(t) * a.pe_stride;
    const int i0 = a.half_layout ? lane : 2 * lane, i1 = a.half_layout ? lane + kRopeRow / 2 : 2 * lane + 1;
    const float x0 = bf16_bits_to_float(pe[i0]), x1 = bf16_bits_to_float(pe[i1]);
    if (slot == -1) return;
    if (slot < 0 || slot >= a.cache_rows) {
        if (lane == 0) record_status(a.status, DSA_ERR_DEVICE_CHECK);
        return;
    }
    if constexpr (!FP8) {
        float s, c;
        turn_sincos(pos, a.tb.turn[lane], s, c);
        const float ms = static_cast<float>(a.tb.mscale);
        s *= ms;
        c *= ms;
        uint16_t *row = static_cast<uint16_t *>(a.cache) + static_cast<int64_t>(slot) * a.row_stride;
        reinterpret_cast<uint4 *>(row)[2 * lane] = c0;
        reinterpret_cast<uint4 *>(row)[2 * lane + 1] = c1;
        row[kLatent + i0] = __bfloat16_as_ushort(__float2bfloat16_rn(x0 * c - x1 * s));
        row[kLatent + i1] = __bfloat16_as_ushort(__float2bfloat16_rn(x0 * s + x1 * c));
    } else {
        // in 64 bits: a value next to a rounding border gets its own code
        const double turns = static_cast<double>(pos) * a.tb.turn[lane];
        double s, c;
        sincospi(2.0 * (turns - rint(turns)), &s, &c);
        s *= a.tb.mscale;
        c *= a.tb.mscale;
        const double y0 = x0 * c - x1 * s, y1 = x0 * s + x1 * c;
        float v[16];
        const uint32_t w[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
        float amax = 0.f;  // of the finite values
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) amax = fabsf(v[i]) < INFINITY ? fmaxf(amax, fabsf(v[i])) : amax;
        // rounded up: the borders between scales are fp32 numbers, so a value
        // above one stays above and one at or below stays
        const float r0 = __double2float_ru(fabs(y0)), r1 = __double2float_ru(fabs(y1));
        amax = r0 < INFINITY ? fmaxf(amax, r0) : amax;
        amax = r1 < INFINITY ? fmaxf(amax, r1) : amax;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float scale = row_scale(amax);
        const float inv = 1.f / scale;  // exact: a power of two between 2^-120 and 2^126
        uint32_t code[4];
#pragma unroll
        for (int g = 0; g < 4; ++g)
            code[g] = e4m3_pair(v[4 * g] * inv, v[4 * g + 1] * inv) |
                      e4m3_pair(v[4 * g + 2] * inv, v[4 * g + 3] * inv) << 16;
        uint8_t *row = static_cast<uint8_t *>(a.cache) + static_cast<int64_t>(slot) * a.row_stride;
        reinterpret_cast<uint4 *>(row)[lane] = make_uint4(code[0], code[1], code[2], code[3]);
        const uint32_t pair = e4m3_pair(odd_float(y0 * inv), odd_float(y1 * inv));
        if (a.half_layout) {
            row[kLatent + i0] = static_cast<uint8_t>(pair);
            row[kLatent + i1] = static_cast<uint8_t>(pair >> 8);
        } else {
            reinterpret_cast<uint16_t *>(row + kLatent)[lane] = static_cast<uint16_t>(pair);
        }
        if (lane == 0) a.kv_scale[slot] = scale;
    }
}

cudaError_t launch_latent_append(const AppendParams &a, bool fp8, cudaStream_t st) {
    const int grid = (a.nt + 3) / 4;
    if (fp8) k16_latent_append<true><<<grid, 128, 0, st>>>(a);
    else k16_latent_append<false><<<grid, 128, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace dsa
