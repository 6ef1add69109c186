// Causal depthwise convolution over a few rows: forward, backward, one row.
//
// A thread owns V = 4 neighbouring channels (2 in the backward pass, which keeps
// two windows and the sums of dw) and
// walks a run of rows with the last rows in registers, so each row is read once
// (plus taps - 1 rows in front of each run, out of the cache).  Bound by memory
// traffic: 2 K multiply-adds per 2 elements moved; 8 x 2048 x 4096 bf16 with 4
// taps takes 52 us forward (5.2 TB/s) and 107 backward, whose second window and
// sums of dw leave less in flight (4, 5 or 6 waves a SIMD and chunks of 64 rows
// measure the same).
#pragma once

#include "causal_conv.hpp"
#include "column_sum.hpp"
#include "launch.hpp"
#include "row_walk.hpp"

namespace canon {
namespace seq {

constexpr int kConvV = 4;

template <typename T, int V>
__device__ __forceinline__ void unpack(const Vec<T, V>& x, float (&v)[V])
{
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = T::load(x.e[i]);
}

template <typename T, int K, int V>
struct ConvParams {
    float w[K][V], b[V];

    __device__ __forceinline__ void load(const ConvArgs& a, int32_t ch)
    {
        // the channels' taps are consecutive: one branch, so that the loads merge
        if (a.param_f32)
            fill<F32>(a, ch);
        else
            fill<T>(a, ch);
    }
    template <typename P>
    __device__ __forceinline__ void fill(const ConvArgs& a, int32_t ch)
    {
        const typename P::store_t* pw =
            static_cast<const typename P::store_t*>(a.weight) + (int64_t)ch * K;
        const typename P::store_t* pb = static_cast<const typename P::store_t*>(a.bias) + ch;
#pragma unroll
        for (int i = 0; i < V; ++i)
#pragma unroll
            for (int k = 0; k < K; ++k) w[k][i] = P::load(pw[i * K + k]);
#pragma unroll
        for (int i = 0; i < V; ++i) b[i] = 0.f;
        if (a.bias)
#pragma unroll
            for (int i = 0; i < V; ++i) b[i] = P::load(pb[i]);
    }
};

// Row t of the sequence, or of the initial state in front of it (t < 0).
template <typename T, int K, int V>
__device__ __forceinline__ void conv_row(const ConvArgs& a, const typename T::store_t* x,
                                         int64_t s, int32_t t, int32_t ch, float (&v)[V])
{
    if (t >= 0) {
        unpack<T, V>(ld_vec<T, V>(x + (int64_t)t * a.x.row), v);
    } else if (a.init) {
        const typename T::store_t* p = static_cast<const typename T::store_t*>(a.init);
        unpack<T, V>(ld_vec<T, V>(p + (s * (K - 1) + (K - 1 + t)) * a.channels + ch), v);
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = 0.f;
    }
}

template <int K, int V>
__device__ __forceinline__ float conv_sum(const float (&win)[K][V], const float (&w)[K][V],
                                          float b, int i)
{
    float p = b;
#pragma unroll
    for (int k = 0; k < K; ++k) p = fma32(w[k][i], win[k][i], p);
    return p;
}

// RUN rows per thread (at least K - 1, so that only a sequence's first run
// reads the initial state).
template <typename T, int K, int V, int RUN>
__global__ __launch_bounds__(256, K <= 4 ? 4 : 2) void k_causal_conv(ConvArgs a)
{
    const int32_t nv = a.channels / V;  // whole vectors, or V = 1
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t slot = i / nv;
    const int32_t ch = (int32_t)(i - slot * nv) * V;
    if (slot >= slot_count<RUN>(a.q.seqs, a.q.rows, a.q.starts != nullptr)) return;
    const Chunk ck = slot_chunk<RUN>(a.q, slot);
    if (ck.row > 0 && ck.len <= 0) return;
    const typename T::store_t* x = rows_ptr<T>(a.x, ck.s, a.q, ck.span.first) + ch;
    typename T::store_t* out = rows_ptr<T>(a.out, ck.s, a.q, ck.span.first) + ch;

    float win[K][V];  // the rows up to the current one, oldest first
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) conv_row<T, K, V>(a, x, ck.s, ck.row - (K - 1) + k, ch, win[k + 1]);

    if (a.final && ck.row == 0) {
        // By the thread that has read the initial state, which may be the
        // same buffer: the last K - 1 rows of initial state and sequence.
        typename T::store_t* f =
            static_cast<typename T::store_t*>(a.final) + ck.s * (K - 1) * a.channels + ch;
#pragma unroll
        for (int k = 0; k + 1 < K; ++k) {
            const int32_t t = ck.span.len - (K - 1) + k;
            float v[V];
            if (t >= 0) {
                conv_row<T, K, V>(a, x, ck.s, t, ch, v);
            } else {  // row K - 1 + t of the initial state, in win[K + t]
#pragma unroll
                for (int m = 0; m + 1 < K; ++m)
                    if (m == K - 1 + t)
#pragma unroll
                        for (int j = 0; j < V; ++j) v[j] = win[m + 1][j];
            }
            st_vec<T, V>(f + (int64_t)k * a.channels, v);
        }
    }

    // Rows r0 .. r0 + U - 1 are computed while the next U are on their way.  Runs
    // that are full in every lane of the wave need no checks.
    constexpr int U = 4;
    Vec<T, V> in[2][U];
    const typename T::store_t* xr = x + (int64_t)ck.row * a.x.row;
    typename T::store_t* outr = out + (int64_t)ck.row * a.out.row;
    auto fetch = [&](int b, int32_t r0, bool full) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t r = full || r0 + u < ck.len ? r0 + u : ck.len - 1;
            in[b][u] = ld_vec<T, V>(xr + (int64_t)r * a.x.row);
        }
    };
    if (ck.len > 0) fetch(0, 0, false);
    ConvParams<T, K, V> p;
    p.load(a, ch);
    auto rows = [&](int b, int32_t r0, bool full) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (!full && r0 + u >= ck.len) break;
#pragma unroll
            for (int k = 0; k + 1 < K; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) win[k][j] = win[k + 1][j];
            unpack<T, V>(in[b][u], win[K - 1]);
            float y[V];
#pragma unroll
            for (int j = 0; j < V; ++j) y[j] = conv_sum<K, V>(win, p.w, p.b[j], j);
            if (a.silu)
#pragma unroll
                for (int j = 0; j < V; ++j) y[j] = silu_f(y[j], sigmoid_f<T>(y[j]));
            st_vec<T, V>(outr + (int64_t)(r0 + u) * a.out.row, y);
        }
    };
    if (__all(ck.len == RUN)) {
#pragma unroll 1
        for (int32_t r0 = 0; r0 < RUN; r0 += 2 * U) {
            fetch(1, r0 + U, true);
            rows(0, r0, true);
            if (r0 + 2 * U < RUN) fetch(0, r0 + 2 * U, true);
            rows(1, r0 + U, true);
        }
    } else {
#pragma unroll 1
        for (int32_t r0 = 0; r0 < ck.len; r0 += U) {
            if (r0 > 0) fetch(0, r0, false);
            rows(0, r0, false);
        }
    }
}

// Backward: with dp = dout silu'(p), dx[t] = sum_k w[k] dp[t + K - 1 - k].  A
// thread walks its run and K - 1 rows beyond it, p recomputed from x.
// Its rows' part of dw and db goes to the workspace, per slot.
template <typename T, int K, int V>
__global__ __launch_bounds__(256, K <= 4 ? 5 : 2) void k_causal_conv_grad(ConvArgs a)
{
    constexpr int RUN = CANON_CONV_CHUNK;
    const int32_t nv = a.channels / V;  // whole vectors, or V = 1
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t slot = i / nv;
    const int32_t ch = (int32_t)(i - slot * nv) * V;
    if (slot >= slot_count<RUN>(a.q.seqs, a.q.rows, a.q.starts != nullptr)) return;
    const Chunk ck = slot_chunk<RUN>(a.q, slot);
    float dw[K][V], db[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        db[j] = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) dw[k][j] = 0.f;
    }
    if (ck.row == 0 || ck.len > 0) {
        const int64_t first = ck.span.first;
        const typename T::store_t* x = rows_ptr<T>(a.x, ck.s, a.q, first) + ch;
        const typename T::store_t* go = rows_ptr<T>(a.dout, ck.s, a.q, first) + ch;
        typename T::store_t* dx = rows_ptr<T>(a.dx, ck.s, a.q, first) + ch;
        const typename T::store_t* df =
            a.dfinal ? static_cast<const typename T::store_t*>(a.dfinal) +
                           ck.s * (K - 1) * a.channels + ch
                     : nullptr;
        typename T::store_t* di = a.dinit ? static_cast<typename T::store_t*>(a.dinit) +
                                                ck.s * (K - 1) * a.channels + ch
                                          : nullptr;
        float win[K][V], dp[K][V];
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < V; ++j) win[k][j] = dp[k][j] = 0.f;
        if (ck.len > 0)
#pragma unroll
            for (int k = 0; k + 1 < K; ++k)
                conv_row<T, K, V>(a, x, ck.s, ck.row - (K - 1) + k, ch, win[k + 1]);
        const int32_t len = ck.span.len;
        const int32_t end = ck.row + ck.len;  // of the run
        const int32_t stop = end + K - 1;
        // As in the forward kernel; a run without a sequence's end or start near
        // it (INNER, in every lane of the wave) needs no checks but r's.
        constexpr int U = 4;
        Vec<T, V> in[2][U], gin[2][U];
        auto fetch = [&](int b, int32_t r0, bool inner) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t t = ck.row + r0 + u;
                const int64_t row = inner || t < len ? t : len - 1;
                in[b][u] = ld_vec<T, V>(x + row * a.x.row);
                gin[b][u] = ld_vec<T, V>(go + row * a.dout.row);
            }
        };
        if (len > 0) fetch(0, 0, false);
        ConvParams<T, K, V> p;
        p.load(a, ch);
        // r: the row within the run; row r - (K - 1) gets its gradient at row r
        auto one_row = [&](int b, int u, int32_t r, bool inner) {
            const int32_t t = ck.row + r;
#pragma unroll
            for (int k = 0; k + 1 < K; ++k)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    win[k][j] = win[k + 1][j];
                    dp[k][j] = dp[k + 1][j];
                }
            if (inner || t < len) {
                unpack<T, V>(in[b][u], win[K - 1]);
                unpack<T, V>(gin[b][u], dp[K - 1]);
                if (a.silu)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float s = conv_sum<K, V>(win, p.w, p.b[j], j);
                        dp[K - 1][j] *= silu_slope(s, sigmoid_f<T>(s));
                    }
                if (inner ? r < RUN : t < end)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        db[j] += dp[K - 1][j];
#pragma unroll
                        for (int k = 0; k < K; ++k)
                            dw[k][j] = fma32(dp[K - 1][j], win[k][j], dw[k][j]);
                    }
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) dp[K - 1][j] = 0.f;
            }
            // row m has all of dp[m .. t]: w[K - 1] dp[m] first
            const int32_t m = t - (K - 1);
            const bool initial = !inner && m < 0;
            if (initial ? di == nullptr : r < K - 1) return;
            float y[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                y[j] = p.w[K - 1][j] * dp[0][j];
#pragma unroll
                for (int k = 1; k < K; ++k) y[j] = fma32(p.w[K - 1 - k][j], dp[k][j], y[j]);
            }
            // the final state's row that is row m
            const int32_t f = m - (len - (K - 1));
            if (!inner && df && f >= 0) {
                float g[V];
                unpack<T, V>(ld_vec<T, V>(df + (int64_t)f * a.channels), g);
#pragma unroll
                for (int j = 0; j < V; ++j) y[j] += g[j];
            }
            if (initial)
                st_vec<T, V>(di + (int64_t)(K - 1 + m) * a.channels, y);
            else
                st_vec<T, V>(dx + (int64_t)m * a.dx.row, y);
        };
        constexpr int ALL = RUN + K - 1;
        constexpr int READ = (ALL + U - 1) / U * U;  // rows that whole fetches read
        if (__all(ck.len == RUN && ck.row > 0 && ck.row + READ <= len)) {
            // exactly ALL rows: the run's last row is r = ALL - 1's, and the rows of dx
            // behind it are the next run's to store
            walk_rows<ALL, U>([&](int b, int32_t r0) { fetch(b, r0, true); },
                              [&](int b, int u, int32_t r) { one_row(b, u, r, true); });
        } else {
#pragma unroll 1
            for (int32_t r0 = 0; r0 < stop - ck.row; r0 += U) {
                if (r0 > 0 && len > 0) fetch(0, r0, false);
#pragma unroll
                for (int u = 0; u < U; ++u)
                    if (r0 + u < stop - ck.row) one_row(0, u, r0 + u, false);
            }
        }
    }
    float* pw = a.ws_w + (slot * a.channels + ch) * K;
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
        for (int k = 0; k < K; ++k) pw[j * K + k] = dw[k][j];
    if (a.dbias)
#pragma unroll
        for (int j = 0; j < V; ++j) a.ws_b[slot * a.channels + ch + j] = db[j];
}

// One row of each sequence; the state's rows move up by one.
template <typename T, int K, int V>
__global__ __launch_bounds__(256) void k_causal_conv_step(ConvArgs a)
{
    const int32_t nv = a.channels / V;  // whole vectors, or V = 1
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t s = i / nv;
    const int32_t ch = (int32_t)(i - s * nv) * V;
    if (s >= a.q.seqs) return;
    const typename T::store_t* x = static_cast<typename T::store_t*>(a.x.p) + s * a.x.seq + ch;
    float win[K][V];
#pragma unroll
    for (int k = 0; k + 1 < K; ++k) conv_row<T, K, V>(a, x, s, k - (K - 1), ch, win[k]);
    const Vec<T, V> in = ld_vec<T, V>(x);
    unpack<T, V>(in, win[K - 1]);
    ConvParams<T, K, V> p;
    p.load(a, ch);
    float y[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
        y[j] = conv_sum<K, V>(win, p.w, p.b[j], j);
        if (a.silu) y[j] = silu_f(y[j], sigmoid_f<T>(y[j]));
    }
    if (a.final) {
        typename T::store_t* f =
            static_cast<typename T::store_t*>(a.final) + s * (K - 1) * a.channels + ch;
#pragma unroll
        for (int k = 0; k + 1 < K; ++k)
            st_vec<T, V>(f + (int64_t)k * a.channels, win[k + 1]);
    }
    st_vec<T, V>(static_cast<typename T::store_t*>(a.out.p) + s * a.out.seq + ch, y);
}

// --------------------------------------------------------------------- launches
template <int RUN>
unsigned conv_grid(const ConvArgs& a, int v)
{
    const int64_t slots = slot_count<RUN>(a.q.seqs, a.q.rows, a.q.starts != nullptr);
    return (unsigned)((slots * (a.channels / v) + 255) / 256);
}

template <typename T, int K, int V>
hipError_t launch_conv_v(const ConvArgs& a, hipStream_t st)
{
    // Long runs read fewer rows twice; short ones are for launches that would
    // leave compute units without work.  Measured for 2048, 4096, 8192, 16384 rows
    // of 4096 bf16 channels (64 to 512 threads x 1024), us: runs of 32 rows 10.9,
    // 16.4, 24.0, 45.7; of 8 rows 9.1, 15.1, 26.5, 47.7.
    const int64_t threads = slot_count<32>(a.q.seqs, a.q.rows, a.q.starts != nullptr) *
                            (a.channels / V);
    if (threads >= (int64_t)device_cus() * 768)
        k_causal_conv<T, K, V, 32><<<dim3(conv_grid<32>(a, V)), dim3(256), 0, st>>>(a);
    else
        k_causal_conv<T, K, V, 8><<<dim3(conv_grid<8>(a, V)), dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

template <typename T, int K, int V>
hipError_t launch_conv_grad_v(const ConvArgs& a, hipStream_t st)
{
    const int64_t slots =
        slot_count<CANON_CONV_CHUNK>(a.q.seqs, a.q.rows, a.q.starts != nullptr);
    const unsigned grid = conv_grid<CANON_CONV_CHUNK>(a, V);
    if (grid) k_causal_conv_grad<T, K, V><<<dim3(grid), dim3(256), 0, st>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    const int64_t d = a.channels;
    return launch_column_sums({{{a.ws_w, d * K, K, K, a.dweight}, {a.ws_b, d, 1, 1, a.dbias}, {}},
                               slots},
                              st);
}

template <typename T, int K, int V>
hipError_t launch_conv_step_v(const ConvArgs& a, hipStream_t st)
{
    const int64_t n = a.q.seqs * (a.channels / V);
    k_causal_conv_step<T, K, V><<<dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

#define CANON_CONV_TAPS(FN, V)                 \
    switch (taps) {                            \
        case 1: return FN<T, 1, V>(a, st);     \
        case 2: return FN<T, 2, V>(a, st);     \
        case 3: return FN<T, 3, V>(a, st);     \
        case 4: return FN<T, 4, V>(a, st);     \
        case 5: return FN<T, 5, V>(a, st);     \
        case 6: return FN<T, 6, V>(a, st);     \
        case 7: return FN<T, 7, V>(a, st);     \
        default: return FN<T, 8, V>(a, st);    \
    }

// V channels a thread, or one where they are not aligned to that.  Vectors read and
// written as they lie gain and lose too little to be worth theirs: 4 taps, single
// channels and such vectors, us: forward float32 16384 x 4095 137 and 129, 16384 x
// 1001 25.6 and 26.7, 2048 x 4095 13.1 and 15.4; backward bf16 16384 x 4095 123 and
// 136, 16384 x 2047 60.7 and 58.2, 2048 x 2047 19.7 and 22.8; single rows float32
// 2048 x 4095 45.5 and 42.3, 2048 x 1001 12.8 and 13.3.
#define CANON_CONV_LAUNCH(NAME, FN, V)                              \
    template <typename T>                                           \
    hipError_t NAME(const ConvArgs& a, int taps, hipStream_t st)    \
    {                                                               \
        if (a.vec) CANON_CONV_TAPS(FN, V)                           \
        CANON_CONV_TAPS(FN, 1)                                      \
    }
CANON_CONV_LAUNCH(launch_causal_conv, launch_conv_v, kConvV)
CANON_CONV_LAUNCH(launch_causal_conv_grad, launch_conv_grad_v, 2)
CANON_CONV_LAUNCH(launch_causal_conv_step, launch_conv_step_v, kConvV)
#undef CANON_CONV_LAUNCH
#undef CANON_CONV_TAPS

}  // namespace seq
}  // namespace canon
