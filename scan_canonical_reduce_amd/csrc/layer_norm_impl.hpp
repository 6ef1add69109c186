// Layer norm: forward, and backward with the sums over rows.
#pragma once

#include "column_sum.hpp"
#include "launch.hpp"
#include "layer_norm.hpp"

namespace canon {
namespace seq {

template <typename T>
constexpr int kNormV = 16 / sizeof(typename T::store_t);

// Columns [col, col + V) of a row as 32-bit values, 0 beyond its width.
template <typename T, int V>
__device__ __forceinline__ void ld_cols(const typename T::store_t* p, int col, int width,
                                        float (&v)[V])
{
    if (col + V <= width) {
        const Vec<T, V> r = ld_any<T, V, false>(p + col);
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = T::load(r.e[j]);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = col + j < width ? T::load(p[col + j]) : 0.f;
    }
}

template <typename T, int V>
__device__ __forceinline__ void st_cols(typename T::store_t* p, int col, int width,
                                        const float (&v)[V])
{
    if (col + V <= width) {
        st_any<T, V, false>(p + col, v);
    } else {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (col + j < width) p[col + j] = T::round(v[j]);
    }
}

template <int V>
__device__ __forceinline__ float tree(const float (&v)[V])
{
    float t[V];
#pragma unroll
    for (int j = 0; j < V; ++j) t[j] = v[j];
#pragma unroll
    for (int d = 1; d < V; d *= 2)
#pragma unroll
        for (int j = 0; j + d < V; j += 2 * d) t[j] += t[j + d];
    return t[0];
}

// The pairwise tree over the lanes of a team (a power of two of lanes that lie
// together, whole waves beyond 64), in every lane.  lds: the team's waves' values;
// not to be used again before the next barrier but one.
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float* lds)
{
#pragma unroll
    for (int d = 1; d < (TEAM < 64 ? TEAM : 64); d *= 2) v += __shfl_xor(v, d);
    if constexpr (TEAM > 64) {
        constexpr int W = TEAM / 64;
        if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
        __syncthreads();
        float w[W];
#pragma unroll
        for (int i = 0; i < W; ++i) w[i] = lds[i];
        v = tree(w);
    }
    return v;
}

template <typename T>
__device__ __forceinline__ typename T::store_t* norm_row(const canon_rows_t& r, const NormArgs& a,
                                                         int32_t row)
{
    int64_t s = 0;
    if (row >= a.rows) {
        s = (uint32_t)row / (uint32_t)a.rows;
        row -= (int32_t)s * a.rows;
    }
    return static_cast<typename T::store_t*>(r.p) + s * r.seq + row * r.row;
}

// One workgroup per row, which is read again for each sum: any width.
template <typename T, typename P>
__global__ __launch_bounds__(256) void k_norm_loop(NormArgs a)
{
    constexpr int V = kNormV<T>, STEP = 256 * V;
    using E = typename T::store_t;
    using W = typename P::store_t;
    __shared__ float lds[2][4];
    const int c0 = threadIdx.x * V;
    for (int32_t row = blockIdx.x; row < a.total; row += gridDim.x) {
        const E* x = norm_row<T>(a.x, a, row);
        const E* res = a.residual.p ? norm_row<T>(a.residual, a, row) : nullptr;
        E* sum = a.sum.p ? norm_row<T>(a.sum, a, row) : nullptr;
        E* out = norm_row<T>(a.out, a, row);
        auto load = [&](int c, float(&v)[V]) {
            ld_cols<T, V>(x, c, a.width, v);
            if (!res) return;
            float r[V];
            ld_cols<T, V>(res, c, a.width, r);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = T::load(T::round(v[j] + r[j]));
        };
        float s = 0.f, q = 0.f;
        for (int c = c0; c < a.width; c += STEP) {
            float v[V];
            load(c, v);
            s += tree(v);
        }
        const float mean = team_sum<256>(s, lds[0]) * a.inv_width;
        for (int c = c0; c < a.width; c += STEP) {
            float v[V];
            load(c, v);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[j] = c + j < a.width ? v[j] - mean : 0.f;
                v[j] *= v[j];
            }
            q += tree(v);
        }
        const float rstd =
            __builtin_amdgcn_rsqf(fma32(team_sum<256>(q, lds[1]), a.inv_width, a.eps));
        if (a.stats && threadIdx.x == 0) {
            a.stats[2 * (int64_t)row] = mean;
            a.stats[2 * (int64_t)row + 1] = rstd;
        }
        for (int c = c0; c < a.width; c += STEP) {
            float v[V], w[V], b[V] = {};
            load(c, v);
            if (sum) st_cols<T, V>(sum, c, a.width, v);
            ld_cols<P, V>(static_cast<const W*>(a.weight), c, a.width, w);
            if (a.bias) ld_cols<P, V>(static_cast<const W*>(a.bias), c, a.width, b);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = fma32((v[j] - mean) * rstd, w[j], b[j]);
            st_cols<T, V>(out, c, a.width, v);
        }
    }
}

// dx of a row by one workgroup, which reads the row twice: any width.
template <typename T, typename P>
__global__ __launch_bounds__(256) void k_norm_dx_loop(NormArgs a)
{
    constexpr int V = kNormV<T>, STEP = 256 * V;
    using E = typename T::store_t;
    using W = typename P::store_t;
    __shared__ float lds[2][4];
    const int c0 = threadIdx.x * V;
    for (int32_t row = blockIdx.x; row < a.total; row += gridDim.x) {
        const E* x = norm_row<T>(a.x, a, row);
        const E* dout = norm_row<T>(a.dout, a, row);
        const E* dsum = a.dsum.p ? norm_row<T>(a.dsum, a, row) : nullptr;
        E* dx = norm_row<T>(a.dx, a, row);
        const float mean = a.stats[2 * (int64_t)row], rstd = a.stats[2 * (int64_t)row + 1];
        float s = 0.f, q = 0.f;
        for (int c = c0; c < a.width; c += STEP) {
            float v[V], g[V], w[V];
            ld_cols<T, V>(x, c, a.width, v);
            ld_cols<T, V>(dout, c, a.width, g);
            ld_cols<P, V>(static_cast<const W*>(a.weight), c, a.width, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                g[j] *= w[j];
                v[j] = c + j < a.width ? (v[j] - mean) * rstd * g[j] : 0.f;
            }
            s += tree(g);
            q += tree(v);
        }
        s = team_sum<256>(s, lds[0]) * a.inv_width;
        q = team_sum<256>(q, lds[1]) * a.inv_width;
        for (int c = c0; c < a.width; c += STEP) {
            float v[V], g[V], w[V], d[V] = {};
            ld_cols<T, V>(x, c, a.width, v);
            ld_cols<T, V>(dout, c, a.width, g);
            if (dsum) ld_cols<T, V>(dsum, c, a.width, d);
            ld_cols<P, V>(static_cast<const W*>(a.weight), c, a.width, w);
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float n = (v[j] - mean) * rstd;
                v[j] = fma32(rstd, fma32(-n, q, fma32(g[j], w[j], -s)), d[j]);
            }
            st_cols<T, V>(dx, c, a.width, v);
        }
    }
}

// Sums of a chunk of rows, a vector of columns a thread.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_dw(NormArgs a, int32_t chunk, int32_t tiles)
{
    constexpr int V = kNormV<T>;
    const int32_t k = blockIdx.x / (uint32_t)tiles, tile = blockIdx.x - k * tiles;
    const int c = (tile * 256 + threadIdx.x) * V;
    if (c >= a.width) return;
    float dw[V] = {}, db[V] = {};
    const int32_t end = a.total - k * chunk < chunk ? a.total : (k + 1) * chunk;
    for (int32_t row = k * chunk; row < end; ++row) {
        float v[V], g[V];
        ld_cols<T, V>(norm_row<T>(a.x, a, row), c, a.width, v);
        ld_cols<T, V>(norm_row<T>(a.dout, a, row), c, a.width, g);
        const float mean = a.stats[2 * (int64_t)row], rstd = a.stats[2 * (int64_t)row + 1];
#pragma unroll
        for (int j = 0; j < V; ++j) {
            dw[j] = fma32((v[j] - mean) * rstd, g[j], dw[j]);
            db[j] += g[j];
        }
    }
    st_cols<F32, V>(a.ws_w + (int64_t)k * a.width, c, a.width, dw);
    if (a.dbias) st_cols<F32, V>(a.ws_b + (int64_t)k * a.width, c, a.width, db);
}

template <typename T, typename P>
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t st)
{
    const int64_t most = (int64_t)resident_grid<&k_norm_loop<T, P>>(256);
    const unsigned grid = (unsigned)(a.total < most ? a.total : most);
    k_norm_loop<T, P><<<dim3(grid), dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

template <typename T, typename P>
hipError_t launch_layer_norm_grad(const NormArgs& a, hipStream_t st)
{
    const int64_t chunk = norm_chunk(a.total), chunks = (a.total + chunk - 1) / chunk;
    if (a.total > 0) {
        constexpr int64_t cols = 256 * kNormV<T>;
        const int64_t tiles = (a.width + cols - 1) / cols;
        k_norm_dw<T><<<dim3((unsigned)(chunks * tiles)), dim3(256), 0, st>>>(a, (int32_t)chunk,
                                                                           (int32_t)tiles);
        if (hipError_t e = hipGetLastError()) return e;
        // after the sums, which read dout: dx may be in its place
        const int64_t most = (int64_t)resident_grid<&k_norm_dx_loop<T, P>>(256);
        k_norm_dx_loop<T, P><<<dim3((unsigned)(a.total < most ? a.total : most)), dim3(256), 0,
                               st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    ColumnSums sums{{{a.ws_w, a.width, 1, 1, a.dweight}, {a.ws_b, a.width, 1, 1, a.dbias}, {}},
                    a.total > 0 ? chunks : 0};
    return launch_column_sums(sums, st);
}

}  // namespace seq
}  // namespace canon
