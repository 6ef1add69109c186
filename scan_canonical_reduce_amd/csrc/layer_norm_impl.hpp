// Layer norm: forward, and backward with the sums over rows.
#pragma once

#include <type_traits>

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

// The columns of lane l of a team are the vectors l, l + TEAM, ... of a row, NV of them
// in registers.  A row's sum adds each vector by a tree, a lane's vectors in order, and
// the lanes by the pairwise tree: the team, and with it the expression, goes by the
// width and the type alone.
template <typename T, int NV>
using Raw = Vec<T, kNormV<T>>[NV];

template <typename T, int TEAM, int NV>
__device__ __forceinline__ void ld_row(const typename T::store_t* p, int lane, int width,
                                       Raw<T, NV>& r)
{
    constexpr int V = kNormV<T>;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * TEAM + lane) * V;
        if (c + V <= width) {
            r[k] = ld_any<T, V, false>(p + c);
        } else {
            r[k] = Vec<T, V>{};
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (c + j < width) r[k].e[j] = p[c + j];
        }
    }
}

// Rows of up to TEAM NV vectors.  A workgroup walks its rows with the parameters and the
// next row in registers (16384 x 4096 bf16 with a residual: XX).
template <typename T, typename P, int TEAM, int NV, bool RES>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void k_norm(NormArgs a)
{
    constexpr int V = kNormV<T>, THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM;
    using E = typename T::store_t;
    using W = typename P::store_t;
    __shared__ float lds[2][THREADS / 64];
    const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    float w[NV][V], b[NV][V];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
        const int c = (k * TEAM + lane) * V;
        ld_cols<P, V>(static_cast<const W*>(a.weight), c, a.width, w[k]);
#pragma unroll
        for (int j = 0; j < V; ++j) b[k][j] = 0.f;
        if (a.bias) ld_cols<P, V>(static_cast<const W*>(a.bias), c, a.width, b[k]);
    }
    const int32_t step = gridDim.x * TEAMS;
    int32_t row = blockIdx.x * TEAMS + team;
    Raw<T, NV> x, res;
    auto fetch = [&](int32_t at) {
        ld_row<T, TEAM, NV>(norm_row<T>(a.x, a, at), lane, a.width, x);
        if (RES) ld_row<T, TEAM, NV>(norm_row<T>(a.residual, a, at), lane, a.width, res);
    };
    if (row < a.total) fetch(row);
    for (; row < a.total; row += step) {
        float v[NV][V], s = 0.f, q = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[k][j] = T::load(x[k].e[j]);
                if (RES) v[k][j] = T::load(T::round(v[k][j] + T::load(res[k].e[j])));
            }
            s += tree(v[k]);
        }
        if (RES && a.sum.p) {
            E* p = norm_row<T>(a.sum, a, row);
#pragma unroll
            for (int k = 0; k < NV; ++k) st_cols<T, V>(p, (k * TEAM + lane) * V, a.width, v[k]);
        }
        if (row + step < a.total) fetch(row + step);
        const float mean = team_sum<TEAM>(s, lds[0]) * a.inv_width;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float d[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                v[k][j] = (k * TEAM + lane) * V + j < a.width ? v[k][j] - mean : 0.f;
                d[j] = v[k][j] * v[k][j];
            }
            q += tree(d);
        }
        const float rstd =
            __builtin_amdgcn_rsqf(fma32(team_sum<TEAM>(q, lds[1]), a.inv_width, a.eps));
        if (a.stats && lane == 0) {
            a.stats[2 * (int64_t)row] = mean;
            a.stats[2 * (int64_t)row + 1] = rstd;
        }
        E* out = norm_row<T>(a.out, a, row);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j) v[k][j] = fma32(v[k][j] * rstd, w[k][j], b[k][j]);
            st_cols<T, V>(out, (k * TEAM + lane) * V, a.width, v[k]);
        }
    }
}

// Backward for rows of up to TEAM NV vectors, with the sums of dweight and dbias over a
// chunk of rows in registers: row i of the chunk to team i mod TEAMS, the teams by the
// pairwise tree.
template <typename T, typename P, int TEAM, int NV>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void k_norm_grad(NormArgs a, int32_t chunk)
{
    constexpr int V = kNormV<T>, THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM;
    using E = typename T::store_t;
    using W = typename P::store_t;
    __shared__ float lds[2][THREADS / 64];
    __shared__ float part[TEAMS > 1 ? THREADS * V : 1];
    const int lane = threadIdx.x % TEAM, team = threadIdx.x / TEAM;
    float w[NV][V], dw[NV][V] = {}, db[NV][V] = {};
#pragma unroll
    for (int k = 0; k < NV; ++k)
        ld_cols<P, V>(static_cast<const W*>(a.weight), (k * TEAM + lane) * V, a.width, w[k]);
    const int32_t first = blockIdx.x * chunk;
    const int32_t end = a.total - first < chunk ? a.total : first + chunk;
    Raw<T, NV> x, g, ds;
    auto fetch = [&](int32_t at) {
        ld_row<T, TEAM, NV>(norm_row<T>(a.x, a, at), lane, a.width, x);
        ld_row<T, TEAM, NV>(norm_row<T>(a.dout, a, at), lane, a.width, g);
        if (a.dsum.p) ld_row<T, TEAM, NV>(norm_row<T>(a.dsum, a, at), lane, a.width, ds);
    };
    int32_t row = first + team;
    if (row < end) fetch(row);
    for (; row < end; row += TEAMS) {
        const float mean = a.stats[2 * (int64_t)row], rstd = a.stats[2 * (int64_t)row + 1];
        float n[NV][V], d[NV][V], e[NV][V], s = 0.f, q = 0.f;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            float t[V];
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const float dout = T::load(g[k].e[j]);
                n[k][j] = (T::load(x[k].e[j]) - mean) * rstd;
                dw[k][j] = fma32(n[k][j], dout, dw[k][j]);
                db[k][j] += dout;
                d[k][j] = dout * w[k][j];
                t[j] = n[k][j] * d[k][j];
                e[k][j] = a.dsum.p ? T::load(ds[k].e[j]) : 0.f;
            }
            s += tree(d[k]);
            q += tree(t);
        }
        if (row + TEAMS < end) fetch(row + TEAMS);
        s = team_sum<TEAM>(s, lds[0]) * a.inv_width;
        q = team_sum<TEAM>(q, lds[1]) * a.inv_width;
        E* dx = norm_row<T>(a.dx, a, row);
#pragma unroll
        for (int k = 0; k < NV; ++k) {
#pragma unroll
            for (int j = 0; j < V; ++j)
                d[k][j] = fma32(rstd, fma32(-n[k][j], q, d[k][j] - s), e[k][j]);
            st_cols<T, V>(dx, (k * TEAM + lane) * V, a.width, d[k]);
        }
    }
    // the teams' sums, a vector at a time
#pragma unroll
    for (int k = 0; k < 2 * NV; ++k) {
        float(&sum)[V] = k < NV ? dw[k % NV] : db[k % NV];
        if (k >= NV && !a.dbias) break;
        if (TEAMS > 1) {
#pragma unroll
            for (int d = 1; d < TEAMS; d *= 2) {
                __syncthreads();
                if (team & d)
#pragma unroll
                    for (int j = 0; j < V; ++j) part[j * THREADS + threadIdx.x] = sum[j];
                __syncthreads();
                if (!(team & d))
#pragma unroll
                    for (int j = 0; j < V; ++j) sum[j] += part[j * THREADS + threadIdx.x + d * TEAM];
            }
        }
        if (team == 0)
            st_cols<F32, V>((k < NV ? a.ws_w : a.ws_b) + (int64_t)blockIdx.x * a.width,
                            (k % NV * TEAM + lane) * V, a.width, sum);
    }
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

// The team for rows of a width: 16 columns a lane (of 32 bits, four vectors; of 16,
// two), whole rows in registers up to 16384 columns.
template <class F>
hipError_t with_team(int32_t width, F&& f)
{
    if (width <= 256) return f(std::integral_constant<int, 16>{});
    if (width <= 1024) return f(std::integral_constant<int, 64>{});
    if (width <= 4096) return f(std::integral_constant<int, 256>{});
    if (width <= 16384) return f(std::integral_constant<int, 1024>{});
    return f(std::integral_constant<int, 0>{});
}

template <auto KERN>
hipError_t launch_norm_rows(const NormArgs& a, int threads, int32_t teams, hipStream_t st)
{
    const int64_t most = (int64_t)resident_grid<KERN>(threads);
    const int64_t need = (a.total + teams - 1) / teams;
    KERN<<<dim3((unsigned)(need < most ? need : most)), dim3(threads), 0, st>>>(a);
    return hipGetLastError();
}

template <typename T, typename P>
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t st)
{
    return with_team(a.width, [&](auto t) {
        constexpr int TEAM = decltype(t)::value, NV = 16 / kNormV<T>;
        if constexpr (TEAM == 0) {
            return launch_norm_rows<&k_norm_loop<T, P>>(a, 256, 1, st);
        } else {
            constexpr int THREADS = TEAM < 256 ? 256 : TEAM;
            if (a.residual.p)
                return launch_norm_rows<&k_norm<T, P, TEAM, NV, true>>(a, THREADS, THREADS / TEAM, st);
            return launch_norm_rows<&k_norm<T, P, TEAM, NV, false>>(a, THREADS, THREADS / TEAM, st);
        }
    });
}

template <typename T, typename P>
hipError_t launch_layer_norm_grad(const NormArgs& a, hipStream_t st)
{
    const int64_t chunk = norm_chunk(a.total), chunks = (a.total + chunk - 1) / chunk;
    if (a.total > 0) {
        const hipError_t e = with_team(a.width, [&](auto t) {
            // the sums take 32 registers more: no more than 512 threads, 8192 columns
            constexpr int WIDE = decltype(t)::value, TEAM = WIDE < 1024 ? WIDE : 512;
            constexpr int NV = 16 / kNormV<T>;
            if (TEAM == 0 || a.width > TEAM * 16) {
                constexpr int64_t cols = 256 * kNormV<T>;
                const int64_t tiles = (a.width + cols - 1) / cols;
                k_norm_dw<T><<<dim3((unsigned)(chunks * tiles)), dim3(256), 0, st>>>(
                    a, (int32_t)chunk, (int32_t)tiles);
                if (hipError_t e = hipGetLastError()) return e;
                // after the sums, which read dout: dx may be in its place
                return launch_norm_rows<&k_norm_dx_loop<T, P>>(a, 256, 1, st);
            }
            if constexpr (TEAM > 0) {
                k_norm_grad<T, P, TEAM, NV><<<dim3((unsigned)chunks), dim3(TEAM < 256 ? 256 : TEAM),
                                              0, st>>>(a, (int32_t)chunk);
            }
            return hipGetLastError();
        });
        if (e) return e;
    }
    ColumnSums sums{{{a.ws_w, a.width, 1, 1, a.dweight}, {a.ws_b, a.width, 1, 1, a.dbias}, {}},
                    a.total > 0 ? chunks : 0};
    return launch_column_sums(sums, st);
}

}  // namespace seq
}  // namespace canon
