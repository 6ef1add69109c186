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

// 16 bytes of a row, as words: kNormV elements.
typedef uint32_t Words16 __attribute__((ext_vector_type(4)));

template <typename T>
__device__ __forceinline__ float element(const Words16& w, int j)
{
    if constexpr (std::is_same<T, F32>::value)
        return __uint_as_float(w[j]);
    else if constexpr (std::is_same<T, BF16>::value)
        return __uint_as_float(j & 1 ? w[j / 2] & 0xffff0000u : w[j / 2] << 16);
    else
        return T::load((uint16_t)(w[j / 2] >> 16 * (j & 1)));
}
template <typename T>
__device__ __forceinline__ Words16 rounded(const float* v)
{
    Words16 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (std::is_same<T, F32>::value)
            w[i] = __float_as_uint(v[i]);
        else
            w[i] = T::round(v[2 * i]) | (uint32_t)T::round(v[2 * i + 1]) << 16;
    }
    return w;
}
// The words moved up by one element, and down.
template <typename T>
__device__ __forceinline__ Words16 push(Words16 w, typename T::store_t e)
{
    if constexpr (std::is_same<T, F32>::value) return Words16{__float_as_uint(e), w.x, w.y, w.z};
    return Words16{w.x << 16 | (uint32_t)e, w.y << 16 | w.x >> 16, w.z << 16 | w.y >> 16,
                   w.w << 16 | w.z >> 16};
}
template <typename T>
__device__ __forceinline__ Words16 pop(Words16 w)
{
    if constexpr (std::is_same<T, F32>::value) return Words16{w.y, w.z, w.w, 0};
    return Words16{w.x >> 16 | w.y << 16, w.y >> 16 | w.z << 16, w.z >> 16 | w.w << 16, w.w >> 16};
}

// Element c of a row: a base that a wave shares and an offset of 32 bits (a width is
// below 2^24), so that no lane holds addresses of 64 bits.
template <typename E>
__device__ __forceinline__ E* row_at(E* row, int c)
{
    return (E*)((char*)row + (uint32_t)(c * (int)sizeof(E)));
}

// The 16 bytes from column c on, zero beyond the row's width; and their store.  The
// elements of a vector that the row's end cuts are taken one by one.
template <typename T>
__device__ __forceinline__ Words16 ld16(const typename T::store_t* row, int c, int width)
{
    constexpr int V = kNormV<T>;
    Words16 w = {0, 0, 0, 0};
    if (c + V <= width) {
        __builtin_memcpy(&w, row_at(row, c), 16);
    } else if (c < width) {
#pragma unroll 1
        for (int j = width - 1; j >= c; --j) w = push<T>(w, *row_at(row, j));
    }
    return w;
}
template <typename T>
__device__ __forceinline__ void st16(typename T::store_t* row, int c, int width, Words16 w)
{
    constexpr int V = kNormV<T>;
    if (c + V <= width) {
        __builtin_memcpy(row_at(row, c), &w, 16);
    } else {
#pragma unroll 1
        for (; c < width; ++c, w = pop<T>(w)) {
            if constexpr (std::is_same<T, F32>::value)
                *row_at(row, c) = __uint_as_float(w.x);
            else
                *row_at(row, c) = (uint16_t)w.x;
        }
    }
}

// Columns [c, c + V) as 32-bit values, 0 beyond the row's width; and their store.
template <typename T, int V>
__device__ __forceinline__ void ld_cols(const typename T::store_t* row, int c, int width,
                                        float (&v)[V])
{
    constexpr int N = kNormV<T>;
#pragma unroll
    for (int h = 0; h < V; h += N) {
        const Words16 w = ld16<T>(row, c + h, width);
#pragma unroll
        for (int j = 0; j < N; ++j) v[h + j] = element<T>(w, j);
    }
}
template <typename T, int V>
__device__ __forceinline__ void st_cols(typename T::store_t* row, int c, int width,
                                        const float (&v)[V])
{
#pragma unroll
    for (int h = 0; h < V; h += kNormV<T>) st16<T>(row, c + h, width, rounded<T>(v + h));
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

// Sums over the lanes of a team (a power of two of lanes that lie together, whole waves
// beyond 64) by the pairwise tree, in every lane, N of them with one barrier.  lds: each
// wave's sums; not to be used again before the next barrier but one.
template <int TEAM, int N>
__device__ __forceinline__ void team_sums(float (&v)[N], float (*lds)[N])
{
    static_assert(TEAM >= 16, "rows of 16 lanes");
#pragma unroll
    for (int i = 0; i < N; ++i) {
        v[i] += dpp<0xb1>(v[i]);   // quads: the neighbour,
        v[i] += dpp<0x4e>(v[i]);   // the other pair;
        v[i] += dpp<0x141>(v[i]);  // the other quad of eight, mirrored,
        v[i] += dpp<0x140>(v[i]);  // the other eight of sixteen
        if constexpr (TEAM >= 64) {
            v[i] = fold_rows(v[i], v[i]);
            v[i] = fold_halves(v[i], v[i]);
        }
    }
    if constexpr (TEAM > 64) {
        constexpr int W = TEAM / 64;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) lds[threadIdx.x >> 6][i] = v[i];
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float w[W];
#pragma unroll
            for (int j = 0; j < W; ++j) w[j] = lds[j][i];
            v[i] = tree(w);
        }
    }
}
template <int TEAM>
__device__ __forceinline__ float team_sum(float v, float (*lds)[1])
{
    float s[1] = {v};
    team_sums<TEAM>(s, lds);
    return s[0];
}

// Deviations whose squares are beyond 32 bits, or too small for them, are squared again
// times a power of two: from z, the mean square and eps (NaN in a row that has one), the
// factor, which is the same in a whole team.
__device__ __forceinline__ bool norm_fits(float z) { return z >= 0x1p-100f && z <= kMaxF; }
__device__ __forceinline__ float norm_factor(float z) { return z < 1.f ? 0x1p100f : 0x1p-80f; }

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
template <int NV>
using Raw = Words16[NV];

template <typename T, int TEAM, int NV>
__device__ __forceinline__ void ld_row(const typename T::store_t* row, int lane, int width,
                                       Raw<NV>& r)
{
#pragma unroll
    for (int k = 0; k < NV; ++k) r[k] = ld16<T>(row, (k * TEAM + lane) * kNormV<T>, width);
}

// The same values, as if loaded again: what was computed from them before is computed
// anew instead of waiting in registers.
template <int NV>
__device__ __forceinline__ void afresh(Raw<NV>& r)
{
#pragma unroll
    for (int k = 0; k < NV; ++k) asm("" : "+v"(r[k]));
}

// Rows of up to TEAM NV vectors.  A workgroup walks its rows with the parameters and the
// next row in registers (16384 x 4096 bf16 with a residual: 95 us, 5.7 TB/s).
template <typename T, typename P, int TEAM, int NV, bool RES>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void k_norm(NormArgs a)
{
    constexpr int V = kNormV<T>, THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM;
    using E = typename T::store_t;
    using W = typename P::store_t;
    __shared__ float lds[3][THREADS / 64][1];
    const int lane = threadIdx.x % TEAM;
    const int team = TEAM < 64 ? threadIdx.x / TEAM : uniform((int32_t)(threadIdx.x / TEAM));
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
    Raw<NV> x, res;
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
                v[k][j] = element<T>(x[k], j);
                if (RES) v[k][j] = T::load(T::round(v[k][j] + element<T>(res[k], j)));
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
        const float z = fma32(team_sum<TEAM>(q, lds[1]), a.inv_width, a.eps);
        float rstd = __builtin_amdgcn_rsqf(z);
        if (!norm_fits(z)) {
            const float c = norm_factor(z);
            q = 0.f;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float d[V];
#pragma unroll
                for (int j = 0; j < V; ++j) d[j] = v[k][j] * c * (v[k][j] * c);
                q += tree(d);
            }
            q = team_sum<TEAM>(q, lds[2]);
            rstd = __builtin_amdgcn_rsqf(fma32(q, a.inv_width, a.eps * c * c)) * c;
        }
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
// pairwise tree.  A team takes RB rows at a time, whose sums share a barrier, while the
// next ones arrive.  Memory bounds it: 16384 x 4096 bf16 with dsum 117 us, 4.6 TB/s.
template <typename T, int NV, int RB>
struct NormRows {
    Raw<NV> x[RB], g[RB], ds[RB];
    float mean[RB], rstd[RB];
};
template <typename T, typename P, int TEAM, int NV, int RB>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void k_norm_grad(NormArgs a, int32_t chunk)
{
    constexpr int V = kNormV<T>, THREADS = TEAM < 256 ? 256 : TEAM, TEAMS = THREADS / TEAM;
    using E = typename T::store_t;
    using W = typename P::store_t;
    __shared__ float lds[2][THREADS / 64][2 * RB];
    __shared__ float part[TEAMS > 1 ? 2 : 1][TEAMS][TEAMS > 1 ? TEAM * NV * V : 1];
    const int lane = threadIdx.x % TEAM;
    const int team = TEAM < 64 ? threadIdx.x / TEAM : uniform((int32_t)(threadIdx.x / TEAM));
    const int32_t first = blockIdx.x * chunk;
    const int32_t end = a.total - first < chunk ? a.total : first + chunk;
    auto fetch = [&](NormRows<T, NV, RB>& r, int32_t row) {
#pragma unroll
        for (int u = 0; u < RB; ++u) {
            const int32_t at = row + u * TEAMS;
            if (at >= end) break;
            r.mean[u] = a.stats[2 * (int64_t)at];
            r.rstd[u] = a.stats[2 * (int64_t)at + 1];
            ld_row<T, TEAM, NV>(norm_row<T>(a.x, a, at), lane, a.width, r.x[u]);
            ld_row<T, TEAM, NV>(norm_row<T>(a.dout, a, at), lane, a.width, r.g[u]);
            if (a.dsum.p) ld_row<T, TEAM, NV>(norm_row<T>(a.dsum, a, at), lane, a.width, r.ds[u]);
        }
    };
    // whole waves that need no barrier hide their loads behind each other's work
    constexpr bool AHEAD = TEAM > 64;
    NormRows<T, NV, RB> now, next;
    int32_t row = first + team;
    if (AHEAD) fetch(next, row);
    float w[NV][V], dw[NV][V] = {}, db[NV][V] = {};
#pragma unroll
    for (int k = 0; k < NV; ++k)
        ld_cols<P, V>(static_cast<const W*>(a.weight), (k * TEAM + lane) * V, a.width, w[k]);
    for (int buf = 0; row < end; row += RB * TEAMS, buf ^= 1) {
        if (AHEAD) {
            now = next;
            if (row + RB * TEAMS < end) fetch(next, row + RB * TEAMS);
        } else {
            fetch(now, row);
        }
        float sums[2 * RB] = {};
#pragma unroll
        for (int u = 0; u < RB; ++u) {
            if (row + u * TEAMS >= end) break;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float d[V], t[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float dout = element<T>(now.g[u][k], j);
                    const float n = (element<T>(now.x[u][k], j) - now.mean[u]) * now.rstd[u];
                    dw[k][j] = fma32(n, dout, dw[k][j]);
                    db[k][j] += dout;
                    d[j] = dout * w[k][j];
                    t[j] = n * d[j];
                }
                sums[2 * u] += tree(d);
                sums[2 * u + 1] += tree(t);
            }
        }
        team_sums<TEAM>(sums, lds[buf]);
#pragma unroll
        for (int u = 0; u < RB; ++u) {
            if (row + u * TEAMS >= end) break;
            afresh<NV>(now.x[u]);
            afresh<NV>(now.g[u]);
            E* dx = norm_row<T>(a.dx, a, row + u * TEAMS);
            const float s = sums[2 * u] * a.inv_width, q = sums[2 * u + 1] * a.inv_width;
#pragma unroll
            for (int k = 0; k < NV; ++k) {
                float d[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float n = (element<T>(now.x[u][k], j) - now.mean[u]) * now.rstd[u];
                    const float g = fma32(-n, q, element<T>(now.g[u][k], j) * w[k][j] - s);
                    d[j] = fma32(now.rstd[u], g, a.dsum.p ? element<T>(now.ds[u][k], j) : 0.f);
                }
                st_cols<T, V>(dx, (k * TEAM + lane) * V, a.width, d);
            }
        }
    }
    if constexpr (TEAMS == 1) {
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * TEAM + lane) * V;
            const int64_t at = (int64_t)blockIdx.x * a.width;
            st_cols<F32, V>(a.ws_w + at, c, a.width, dw[k]);
            if (a.dbias) st_cols<F32, V>(a.ws_b + at, c, a.width, db[k]);
        }
    } else {
        constexpr int COLS = TEAM * NV * V;
#pragma unroll
        for (int k = 0; k < NV; ++k) {
            const int c = (k * TEAM + lane) * V;
#pragma unroll
            for (int j = 0; j < V; ++j) {
                part[0][team][c + j] = dw[k][j];
                part[1][team][c + j] = db[k][j];
            }
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 2 * COLS; i += THREADS) {
            const int which = i / COLS, c = i % COLS;
            if (c >= a.width || (which && !a.dbias)) continue;
            float v[TEAMS];
#pragma unroll
            for (int t = 0; t < TEAMS; ++t) v[t] = part[which][t][c];
            (which ? a.ws_b : a.ws_w)[(int64_t)blockIdx.x * a.width + c] = tree(v);
        }
    }
}

// Rows of any width, a workgroup each: the first U vectors of a lane in registers, the
// others read again for each sum (from the caches), U of them in flight.  777 x 20000
// float32: 34 us warm, 43 cold (47 with all read again, 47 and more with all in registers,
// which spill or leave a lane too few in flight).
constexpr int kLoopU = 4;

template <typename T, typename P>
__global__ __launch_bounds__(1024) void k_norm_loop(NormArgs a)
{
    constexpr int V = kNormV<T>, STEP = 1024 * V, U = kLoopU;
    using E = typename T::store_t;
    using W = typename P::store_t;
    __shared__ float lds[3][16][1];
    const int c0 = threadIdx.x * V;
    for (int32_t row = blockIdx.x; row < a.total; row += gridDim.x) {
        const E* x = norm_row<T>(a.x, a, row);
        const E* res = a.residual.p ? norm_row<T>(a.residual, a, row) : nullptr;
        E* sum = a.sum.p ? norm_row<T>(a.sum, a, row) : nullptr;
        E* out = norm_row<T>(a.out, a, row);
        // the vectors s of a lane from c on
        auto fetch = [&](int c, Words16(&w)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) w[u] = ld16<T>(x, c + u * STEP, a.width);
            if (res) {
                Words16 r[U];
#pragma unroll
                for (int u = 0; u < U; ++u) r[u] = ld16<T>(res, c + u * STEP, a.width);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float v[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] = element<T>(w[u], j) + element<T>(r[u], j);
                    w[u] = rounded<T>(v);
                }
            }
        };
        Words16 kept[U];
        fetch(c0, kept);
        // f(column, the vector s there), in order
        auto each = [&](auto f) {
            auto use = [&](int c, const Words16(&w)[U]) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (c + u * STEP >= a.width) break;
                    float v[V];
#pragma unroll
                    for (int j = 0; j < V; ++j) v[j] = element<T>(w[u], j);
                    f(c + u * STEP, v);
                }
            };
            use(c0, kept);
            for (int c = c0 + U * STEP; c < a.width; c += U * STEP) {
                Words16 w[U];
                fetch(c, w);
                use(c, w);
            }
        };
        float s = 0.f, q = 0.f;
        each([&](int, float(&v)[V]) { s += tree(v); });
        const float mean = team_sum<1024>(s, lds[0]) * a.inv_width;
        auto squares = [&](float by) {
            q = 0.f;
            each([&](int c, float(&v)[V]) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    v[j] = c + j < a.width ? (v[j] - mean) * by : 0.f;
                    v[j] *= v[j];
                }
                q += tree(v);
            });
            return q;
        };
        const float z = fma32(team_sum<1024>(squares(1.f), lds[1]), a.inv_width, a.eps);
        float rstd = __builtin_amdgcn_rsqf(z);
        if (!norm_fits(z)) {
            const float by = norm_factor(z);
            q = team_sum<1024>(squares(by), lds[2]);
            rstd = __builtin_amdgcn_rsqf(fma32(q, a.inv_width, a.eps * by * by)) * by;
        }
        if (a.stats && threadIdx.x == 0) {
            a.stats[2 * (int64_t)row] = mean;
            a.stats[2 * (int64_t)row + 1] = rstd;
        }
        each([&](int c, float(&v)[V]) {
            float w[V], b[V] = {};
            if (sum) st_cols<T, V>(sum, c, a.width, v);
            ld_cols<P, V>(static_cast<const W*>(a.weight), c, a.width, w);
            if (a.bias) ld_cols<P, V>(static_cast<const W*>(a.bias), c, a.width, b);
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] = fma32((v[j] - mean) * rstd, w[j], b[j]);
            st_cols<T, V>(out, c, a.width, v);
        });
    }
}

// dx of such rows, the first vectors of x and dout in registers: 43 us, 4.3 TB/s (54 with
// all read again).
template <typename T, typename P>
__global__ __launch_bounds__(1024) void k_norm_dx_loop(NormArgs a)
{
    constexpr int V = kNormV<T>, STEP = 1024 * V, U = kLoopU;
    using E = typename T::store_t;
    using W = typename P::store_t;
    __shared__ float lds[2][16][2];
    const int c0 = threadIdx.x * V;
    int buf = 0;
    for (int32_t row = blockIdx.x; row < a.total; row += gridDim.x, buf ^= 1) {
        const E* x = norm_row<T>(a.x, a, row);
        const E* dout = norm_row<T>(a.dout, a, row);
        const E* dsum = a.dsum.p ? norm_row<T>(a.dsum, a, row) : nullptr;
        E* dx = norm_row<T>(a.dx, a, row);
        const float mean = a.stats[2 * (int64_t)row], rstd = a.stats[2 * (int64_t)row + 1];
        auto fetch = [&](int c, Words16(&v)[U], Words16(&g)[U]) {
#pragma unroll
            for (int u = 0; u < U; ++u) v[u] = ld16<T>(x, c + u * STEP, a.width);
#pragma unroll
            for (int u = 0; u < U; ++u) g[u] = ld16<T>(dout, c + u * STEP, a.width);
        };
        Words16 kept_x[U], kept_g[U];
        fetch(c0, kept_x, kept_g);
        // f(column, n and dout weight there), in order
        auto each = [&](auto f) {
            auto use = [&](int c, const Words16(&v)[U], const Words16(&g)[U]) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const int at = c + u * STEP;
                    if (at >= a.width) break;
                    float n[V], d[V], w[V];
                    ld_cols<P, V>(static_cast<const W*>(a.weight), at, a.width, w);
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        n[j] = (element<T>(v[u], j) - mean) * rstd;
                        d[j] = element<T>(g[u], j) * w[j];
                    }
                    f(at, n, d);
                }
            };
            use(c0, kept_x, kept_g);
            for (int c = c0 + U * STEP; c < a.width; c += U * STEP) {
                Words16 v[U], g[U];
                fetch(c, v, g);
                use(c, v, g);
            }
        };
        float sums[2] = {0.f, 0.f};
        each([&](int, float(&n)[V], float(&d)[V]) {
            sums[0] += tree(d);
#pragma unroll
            for (int j = 0; j < V; ++j) n[j] *= d[j];  // 0 beyond the width, as d is
            sums[1] += tree(n);
        });
        team_sums<1024>(sums, lds[buf]);
        const float s = sums[0] * a.inv_width, q = sums[1] * a.inv_width;
        each([&](int c, float(&n)[V], float(&d)[V]) {
            float e[V] = {};
            if (dsum) ld_cols<T, V>(dsum, c, a.width, e);
#pragma unroll
            for (int j = 0; j < V; ++j) n[j] = fma32(rstd, fma32(-n[j], q, d[j] - s), e[j]);
            st_cols<T, V>(dx, c, a.width, n);
        });
    }
}

// Sums of a chunk of rows, a vector of columns a thread: x and dout are read once more,
// 21 us at 6 TB/s (24 in chunks of a quarter, whose sums are as many more).
template <typename T>
__global__ __launch_bounds__(256) void k_norm_dw(NormArgs a, int32_t chunk, int32_t tiles)
{
    constexpr int V = kNormV<T>;
    const int32_t k = blockIdx.x / (uint32_t)tiles, tile = blockIdx.x - k * tiles;
    const int c = (tile * 256 + threadIdx.x) * V;
    if (c >= a.width) return;
    float dw[V] = {}, db[V] = {};
    const int32_t end = a.total - k * chunk < chunk ? a.total : (k + 1) * chunk;
#pragma unroll 4
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

template <class F>
hipError_t with_grad_team(int32_t width, F&& f)
{
    if (width <= 256) return f(std::integral_constant<int, 16>{});
    if (width <= 1024) return f(std::integral_constant<int, 64>{});
    if (width <= 2048) return f(std::integral_constant<int, 256>{});
    if (width <= 4096) return f(std::integral_constant<int, 512>{});
    if (width <= kNormGradWide) return f(std::integral_constant<int, 1024>{});
    return f(std::integral_constant<int, 0>{});
}

template <auto KERN>
hipError_t launch_norm_rows(const NormArgs& a, int threads, int32_t teams, hipStream_t st)
{
    const int64_t most = (int64_t)resident_grid<KERN>(threads);
    const int64_t need = (a.total + teams - 1) / teams;
    const dim3 grid((unsigned)capped_grid(need < most ? need : most));
    KERN<<<grid, dim3(threads), 0, st>>>(a);
    return hipGetLastError();
}

template <typename T, typename P>
hipError_t launch_layer_norm(const NormArgs& a, hipStream_t st)
{
    return with_team(a.width, [&](auto t) {
        constexpr int TEAM = decltype(t)::value, NV = 16 / kNormV<T>;
        if constexpr (TEAM == 0) {
            return launch_norm_rows<&k_norm_loop<T, P>>(a, 1024, 1, st);
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
    const int64_t chunk = norm_chunk(a.total, a.width), chunks = (a.total + chunk - 1) / chunk;
    if (a.total > 0) {
        const hipError_t e = with_grad_team(a.width, [&](auto t) {
            constexpr int TEAM = decltype(t)::value, NV = (TEAM < 256 ? 16 : 8) / kNormV<T>;
            if constexpr (TEAM == 0) {
                constexpr int64_t cols = 256 * kNormV<T>;
                const int64_t tiles = (a.width + cols - 1) / cols;
                k_norm_dw<T><<<dim3((unsigned)(chunks * tiles)), dim3(256), 0, st>>>(
                    a, (int32_t)chunk, (int32_t)tiles);
                if (hipError_t e = hipGetLastError()) return e;
                // after the sums, which read dout: dx may be in its place
                return launch_norm_rows<&k_norm_dx_loop<T, P>>(a, 1024, 1, st);
            }
            if constexpr (TEAM > 0) {
                constexpr int RB = TEAM < 256 || TEAM == 1024 || sizeof(typename T::store_t) == 4 ? 1 : 2;
                k_norm_grad<T, P, TEAM, NV, RB><<<dim3((unsigned)chunks),
                                                  dim3(TEAM < 256 ? 256 : TEAM), 0, st>>>(
                    a, (int32_t)chunk);
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
