// Sampling of the next token, a workgroup for each row.
//
// A weight w = exp((logit - max) / temperature) <= 1 is computed in 64 bits and held
// as an integer multiple of 2^-bits, so that the sum of a whole row fits 62 bits:
// integer sums are the same in any order, so a row can be cut and its filters'
// borders searched in any way without changing which token u picks.
//
// No sort: what top_k and top_p keep are the tokens up to a border (key, index) in
// the order of descending keys, which ascend with the logit, and ascending indexes.
//   1. Each thread's largest logit, and the row's.
//   2. With a filter, tokens counted in kBins equal steps of the logit from the largest
//      down.  For top_k the threads' largest ones suffice: where k of them lie, k
//      tokens do, and not many more.  For a larger k all are counted; for top_p their
//      weights are added up, to 14 bits, which tells the border's step (or two).
//   3. The tokens in question go to a list in LDS: for top_k all from the border's step
//      up, for top_p those of its steps, while all weights are summed.
//   4. In a short list every token is compared with every other; in a longer one the
//      border is found digit by digit, by counts or sums of weights.
//   5. Sums of the kept weights by pieces of the row in index order, the piece in
//      which u's share falls, and the token in it.
// Where a list does not fit (thousands of tokens in a step, as where all are equal),
// the whole row is read again for every digit instead.
//
// What bounds it: passes over a row by one compute unit, and in those over weights vector
// issue (27 instructions in 64 bits a token).  256 rows of 131072 in bfloat16, which fill
// the chip, and one such row: the largest logit alone 18 and 11 us, no filter 48 and 34,
// top_k 50 31 and 22, top_p 0.9 86 and 70, which goes over the row for the steps and again
// for their list.  64 rows of 32000: 6, 15, 13 and 32.  (In an earlier version, where top_p
// 0.5 took 92 us and 0.9 100, adding up the weights themselves by steps with 64-bit atomics,
// so that they need not be computed again, took 88 and 119.)
#pragma once

#include <type_traits>

#include "launch.hpp"
#include "sample.hpp"

namespace canon {
namespace seq {

typedef unsigned long long u64;

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / 64;
constexpr int kBins = 4 * kSampleThreads;
constexpr int kList = 6144;
constexpr int kRank = 256;  // tokens of a list that are compared with each other
constexpr int kSums = 8 * kSampleWaves;
constexpr float kInf = __builtin_inff();

// The key of a logit that is not masked: ascending, one for both zeros, as wide as the
// type; and the logit of a key.
template <typename T>
__device__ __forceinline__ uint32_t logit_key(float x)
{
    constexpr bool wide = sizeof(typename T::store_t) == 4;
    uint32_t b;
    if constexpr (wide)
        b = __float_as_uint(x + 0.f);
    else
        b = (uint32_t)T::round(x + 0.f) << 16;
    const uint32_t k = b >> 31 ? ~b : b | 0x80000000u;
    return wide ? k : k >> 16;
}
template <typename T>
__device__ __forceinline__ float key_logit(uint32_t k)
{
    if constexpr (sizeof(typename T::store_t) == 4)
        return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
    else
        return T::load((uint16_t)(k >> 15 ? k & 0x7fffu : ~k));
}

// A row's weights.  2^y, y = (x - max) / temperature in binary steps, is 2^n times the
// polynomial of degree 10 whose largest error on [-1/2, 1/2] is smallest (2^-51.5
// relative with its rounded coefficients; 1 at 0).  Adding 2^(52 - bits) leaves the
// rounded multiple of 2^-bits in the low bits of the sum: 0 below 2^-60, where y is
// cut off, and for a masked logit.  Beside an infinite logit only such are kept; its y
// is not a number, and the cut makes it 0.
struct Weights {
    double max, scale, unit;  // scale: log2(e) / temperature
    double cut;               // -60, or 0 where the largest is infinite
    __device__ __forceinline__ u64 operator()(float x) const
    {
        const double y = __builtin_fmax(((double)x - max) * scale, cut);  // cut for a NaN
        const double t = y + 0x1.8p52, r = y - (t - 0x1.8p52);
        double p = 0x1.e6063f7217bc6p-28;
        p = __builtin_fma(p, r, 0x1.b675bca4eeebbp-24);
        p = __builtin_fma(p, r, 0x1.62bfd47773353p-20);
        p = __builtin_fma(p, r, 0x1.ffcb54062e698p-17);
        p = __builtin_fma(p, r, 0x1.430913096fd9fp-13);
        p = __builtin_fma(p, r, 0x1.5d87fe9d7a584p-10);
        p = __builtin_fma(p, r, 0x1.3b2ab6fba1ddap-7);
        p = __builtin_fma(p, r, 0x1.c6b08d703ce49p-5);
        p = __builtin_fma(p, r, 0x1.ebfbdff82c598p-3);
        p = __builtin_fma(p, r, 0x1.62e42fefa3a19p-1);
        p = __builtin_fma(p, r, 1.0);
        const u64 n = __builtin_bit_cast(u64, t) << 52;  // y's integer, as an exponent
        const double w = __builtin_bit_cast(double, __builtin_bit_cast(u64, p) + n);
        return __builtin_bit_cast(u64, w + unit) & 0xfffffffffffffull;
    }
};

// The kept tokens: those above the logit, and at it up to the index.
struct Border {
    float x;
    uint32_t idx;
    __device__ __forceinline__ bool keeps(float v, uint32_t i) const
    {
        return v > x || (v == x && i <= idx);
    }
};

// The weights that a share p of sum takes at least: one unit, and no more than all.
__device__ __forceinline__ u64 min_share(double p, u64 sum)
{
    const double want = __builtin_ceil(p * (double)sum);
    const u64 v = want >= 1. ? (u64)want : 1;
    return v < sum ? v : sum;
}

// ------------------------------------------------------------------- wave scans
template <int CTRL, int ROWS, typename V>
__device__ __forceinline__ V dpp_or_0(V v)
{
    if constexpr (sizeof(V) == 8) {
        const u64 b = __builtin_bit_cast(u64, v);
        const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, ROWS,
                                                                  0xf, false);
        const uint32_t hi =
            (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(b >> 32), CTRL, ROWS, 0xf, false);
        return __builtin_bit_cast(V, (u64)hi << 32 | lo);
    } else {
        return __builtin_bit_cast(V, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v),
                                                                 CTRL, ROWS, 0xf, false));
    }
}
// the sum over the lanes up to this one
template <typename V>
__device__ __forceinline__ V wave_upto(V v)
{
    v += dpp_or_0<0x111, 0xf>(v);  // from 1, 2, 4, 8 lanes below in a row of 16
    v += dpp_or_0<0x112, 0xf>(v);
    v += dpp_or_0<0x114, 0xf>(v);
    v += dpp_or_0<0x118, 0xf>(v);
    v += dpp_or_0<0x142, 0xa>(v);  // the last lane of a row to the odd rows
    v += dpp_or_0<0x143, 0xc>(v);  // and of the first half to the second
    return v;
}
__device__ __forceinline__ u64 lane64(u64 v, int lane)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)v, lane);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(v >> 32), lane);
    return (u64)hi << 32 | lo;
}

// From the highest of 256 bins down, the first at which the sum reaches target (which
// is at most the whole sum): its number, the sum above it and its own.  By one wave.
struct Picked {
    int bin;
    u64 above, here;
};
__device__ __forceinline__ void pick_bin(const u64* hist, u64 target, Picked* out)
{
    const int lane = threadIdx.x & 63, b0 = 255 - 4 * lane;
    u64 v[4], sum = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += v[i] = hist[b0 - i];
    const u64 upto = wave_upto(sum);
    u64 before = upto - sum;
    if (before >= target || upto < target) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (before + v[i] >= target) {
            *out = Picked{b0 - i, before, v[i]};
            return;
        }
        before += v[i];
    }
}

// The sums over the threads before this one, and of all, of N values at once.  lds: a
// value of each a wave, not to be used again before the next barrier.
template <typename V, int N>
__device__ __forceinline__ void scan_before(V (&v)[N], V (*lds)[kSampleWaves], V (&all)[N])
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const V upto = wave_upto(v[i]);
        if (lane == 63) lds[i][wave] = upto;
        v[i] = upto - v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) {
        // lane w of a row holds wave w's sum
        const V upto = wave_upto(lane < kSampleWaves ? lds[i][lane] : V(0));
        if constexpr (sizeof(V) == 8) {
            const u64 b = __builtin_bit_cast(u64, upto);
            all[i] = __builtin_bit_cast(V, lane64(b, kSampleWaves - 1));
            if (wave > 0) v[i] += __builtin_bit_cast(V, lane64(b, wave - 1));
        } else {
            const int b = __builtin_bit_cast(int, upto);
            all[i] = __builtin_bit_cast(V, __builtin_amdgcn_readlane(b, kSampleWaves - 1));
            if (wave > 0) v[i] += __builtin_bit_cast(V, __builtin_amdgcn_readlane(b, wave - 1));
        }
    }
}

// A row in pieces of 64 vectors.  Wave w has the pieces (16 g + w) G ... + G - 1 of
// each group g, so that sums by (g, w) are sums of stretches in index order.
template <typename T>
struct Row {
    using E = typename T::store_t;
    static constexpr int V = 16 / sizeof(E), kPiece = 64 * V, U = 2;
    const E* x;
    int32_t n, G, groups;
    // the vector of this lane in a piece that starts at `first` (below n)
    __device__ __forceinline__ Vec<T, V> load(int32_t first) const
    {
        const int32_t at = first + (threadIdx.x & 63) * V;
        if (first + kPiece <= n) return ld_any<T, V, false>(x + at);
        Vec<T, V> v;
#pragma unroll
        for (int e = 0; e < V; ++e) v.e[e] = at + e < n ? x[at + e] : T::round(-kInf);
        return v;
    }
    // f(g, index of the vector's first token, vector) over the wave's vectors
    template <class F>
    __device__ __forceinline__ void each(F&& f) const
    {
        const int wave = uniform((int32_t)(threadIdx.x >> 6));
        int g = 0, i = 0;
        struct Batch {
            Vec<T, V> v[U];
            int32_t first[U];
            int gs[U];
        };
        auto fetch = [&](Batch& b) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                b.first[u] = ((g * kSampleWaves + wave) * G + i) * kPiece;
                b.gs[u] = g < groups && b.first[u] < n ? g : -1;
                if (b.gs[u] >= 0) b.v[u] = load(b.first[u]);
                if (++i == G) i = 0, ++g;
            }
        };
        auto use = [&](const Batch& b) {
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (b.gs[u] >= 0) f(b.gs[u], b.first[u] + (int32_t)(threadIdx.x & 63) * V, b.v[u]);
        };
        Batch x, y;
        fetch(x);
        while (x.gs[0] >= 0) {
            fetch(y);
            use(x);
            x = y;
        }
    }
};

template <typename T>
__global__ __launch_bounds__(kSampleThreads) void k_sample(SampleArgs a)
{
    using R = Row<T>;
    using E = typename T::store_t;
    constexpr int V = R::V, kDigits = sizeof(E);
    __shared__ union {
        uint32_t bins[kBins + 64];  // and one a lane for what has no step
        u64 sums[kSums];
    } sh;
    __shared__ uint32_t lkey[kList], lidx[kList];
    __shared__ u64 hist[256], wave64[3][kSampleWaves];
    __shared__ double bounds[1][kSampleWaves];
    __shared__ struct {
        u64 place, weight;
    } entry[kRank];
    __shared__ Border s_border;
    __shared__ uint32_t wave32[1][kSampleWaves];
    // not one array: a wave may be at the minimum while others still read the maxima
    __shared__ float wave_max[kSampleWaves], wave_min[kSampleWaves];
    __shared__ Picked picked;
    __shared__ uint32_t s_n, s_first, s_b1, s_b2, s_c2;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform((int32_t)(tid >> 6));
    R r;
    r.x = static_cast<const E*>(a.logits) + row * a.ld;
    r.n = a.vocab;
    const int32_t pieces = (r.n + R::kPiece - 1) / R::kPiece;
    r.G = (pieces + kSums - 1) / kSums;
    r.groups = r.G ? (pieces + kSampleWaves * r.G - 1) / (kSampleWaves * r.G) : 0;

    // 1. the largest (a maximum takes the operand that is not NaN)
    float mine = -kInf;
    r.each([&](int, int32_t, const Vec<T, V>& v) {
#pragma unroll
        for (int e = 0; e < V; ++e) mine = __builtin_fmaxf(mine, T::load(v.e[e]));
    });
    float top = mine;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) top = __builtin_fmaxf(top, __shfl_xor(top, d));
    if (lane == 0) wave_max[wave] = top;
    for (int b = tid; b < kBins; b += kSampleThreads) sh.bins[b] = 0;
    if (tid == 0) s_n = 0, s_first = 0xffffffffu, s_b1 = s_b2 = kBins - 1;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) top = __builtin_fmaxf(top, wave_max[w]);
    auto put = [&](int64_t id) {
        if (a.ids64)
            static_cast<int64_t*>(a.ids)[row] = id;
        else
            static_cast<int32_t*>(a.ids)[row] = (int32_t)id;
    };
    if (top == -kInf) {
        if (tid == 0) put(-1);
        return;
    }
    const double t = a.temperature ? a.temperature[row] : a.temperature_all;
    const int32_t k = !(t > 0.) ? 1 : a.top_k ? a.top_k[row] : a.top_k_all;
    const double p = a.top_p ? a.top_p[row] : a.top_p_all;
    const double min_p = a.min_p ? a.min_p[row] : a.min_p_all;
    // f(x, index) over the row
    auto whole = [&](auto f) {
        r.each([&](int, int32_t at, const Vec<T, V>& v) {
#pragma unroll
            for (int e = 0; e < V; ++e) f(T::load(v.e[e]), (uint32_t)(at + e));
        });
    };
    if (k == 1) {  // the largest, whatever the other settings; in the waves that saw it
        if (__ballot(mine == top)) {
            uint32_t first = 0xffffffffu;
            whole([&](float x, uint32_t i) { first = x == top && i < first ? i : first; });
            if (first != 0xffffffffu) atomicMin(&s_first, first);
        }
        __syncthreads();
        if (tid == 0) put(s_first);
        return;
    }

    const Weights weigh{(double)top, __builtin_fmin(1.4426950408889634 / t, 1e300),
                        __builtin_amdgcn_ldexp(1., 52 - a.bits), top < kInf ? -60. : 0.};
    const u64 one = 1ull << a.bits;
    const u64 least = !(min_p > 0.) ? 0 : min_p < 1. ? (u64)__builtin_ceil(min_p * (double)one) : one;
    // the row's unmasked tokens; beside an infinite one, those alone
    Border border{top == kInf ? kInf : -kMaxF, 0xffffffffu};
    bool in_list = false;  // the list holds all tokens that are still in question

    auto tokens = [&](auto f) {
        if (!in_list) return whole(f);
        for (uint32_t i = tid; i < s_n; i += kSampleThreads) f(key_logit<T>(lkey[i]), lidx[i]);
    };
    auto append = [&](float x, uint32_t i) {
        const uint32_t at = atomicAdd(&s_n, 1u);
        if (at < kList) lkey[at] = logit_key<T>(x), lidx[at] = i;
    };
    // 4. the first tokens in order, of those in question and kept by the border, whose
    // values add up to target (at most the sum of all): the border behind them
    auto select = [&](auto weighted, u64 target) {
        uint32_t prefix = 0;
        u64 above = 0, here = 0;
        auto digit = [&](auto f) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            tokens(f);
            __syncthreads();
            if (wave == 0) pick_bin(hist, target - above, &picked);
            __syncthreads();
            above += picked.above;
            here = picked.here;
            return (uint32_t)picked.bin;
        };
#pragma unroll 1
        for (int shift = 8 * (kDigits - 1); shift >= 0; shift -= 8)
            prefix |= digit([&](float x, uint32_t i) {
                          const uint32_t key = logit_key<T>(x);
                          if (border.keeps(x, i) &&
                              (u64)key >> (shift + 8) == (u64)prefix >> (shift + 8))
                              atomicAdd(&hist[key >> shift & 255], weighted.value ? weigh(x) : 1ull);
                      })
                      << shift;
        const float at = key_logit<T>(prefix);
        u64 need = target - above;
        if (weighted.value) {
            const u64 each = weigh(at);
            need = (need + each - 1) / each;
            here /= each;
        }
        uint32_t idx = at == border.x ? border.idx : 0xffffffffu;
        if (need < here) {  // the lowest indexes of the ones at the logit
            idx = 0;
            target = need;
            above = 0;
#pragma unroll 1
            for (int shift = 16; shift >= 0; shift -= 8) {
                if (r.n <= 1 << shift) continue;
                idx |= (255u - digit([&](float x, uint32_t i) {
                            if (x == at && border.keeps(x, i) &&
                                i >> (shift + 8) == idx >> (shift + 8))
                                atomicAdd(&hist[255 - (i >> shift & 255)], 1ull);
                        }))
                       << shift;
            }
        }
        border = Border{at, idx};
    };
    // the same for a list of up to kRank tokens, all kept by the border so far: the
    // first `most` of them (at least one), and with by_p of those the first whose
    // weights, with those outside the list, make target (0: their share p)
    auto rank = [&](uint32_t most, bool by_p, u64 target, u64 outside) {
        const uint32_t n = s_n;
        int each = kSampleThreads / kRank;  // threads a token
        while (n * each * 2 <= kSampleThreads && each < 64) each *= 2;
        const uint32_t i = tid / each, q = tid & (each - 1);
        if (tid < n) {
            entry[tid].place = (u64)lkey[tid] << 32 | ~lidx[tid];
            entry[tid].weight = weigh(key_logit<T>(lkey[tid]));
        }
        __syncthreads();
        const bool on = i < n;
        const u64 place = on ? entry[i].place : 0;
        u64 before = 0;
        uint32_t place_no = 0;
        for (uint32_t j = q; j < n; j += each) {
            const bool first = entry[j].place > place;
            before += first ? entry[j].weight : 0;
            place_no += first;
        }
        for (int d = 1; d < each; d *= 2) {
            before += __shfl_xor(before, d);
            place_no += __shfl_xor(place_no, d);
        }
        const u64 mine = on ? entry[i].weight : 0;
        most = most < n ? most : n;
        const bool first = on && q == 0 && place_no < most;
        if (by_p && target == 0) {
            u64 v[1] = {first ? mine : 0}, all[1];
            scan_before(v, wave64, all);
            target = min_share(p, all[0]);
        }
        if (first && (!by_p || outside + before < target) &&
            (place_no + 1 == most || (by_p && outside + before + mine >= target)))
            s_border = Border{key_logit<T>((uint32_t)(place >> 32)), ~(uint32_t)place};
        __syncthreads();
        border = s_border;
    };
    // sums of value(first index, vector) by group
    auto group_sums = [&](auto value) {
        for (int i = tid; i < kSums; i += kSampleThreads) sh.sums[i] = 0;
        __syncthreads();
        int of = -1;
        u64 sum = 0;
        auto flush = [&]() {
            sum = wave_upto(sum);
            if (lane == 63 && of >= 0) sh.sums[of * kSampleWaves + wave] = sum;
            sum = 0;
        };
        r.each([&](int g, int32_t at, const Vec<T, V>& v) {
            if (g != of) flush();
            of = g;
            sum += value(at, v);
        });
        flush();
        __syncthreads();
    };

    auto by_least = [&](auto f) {  // f(whether no weight is too small)
        if (least == 0)
            f(std::true_type{});
        else
            f(std::false_type{});
    };

    // 2. and 3.
    bool summed = false;  // weights outside the list are in the groups' sums
    const bool by_p = p < 1.;
    bool by_k = k > 0 && k < r.n;
    if (by_k || by_p) {
        // steps as far as weights are not 0, or over the row's range where that is less
        double span = 36. * t;
        float per = (float)(kBins / span);
        if (span > 512.) {
            float least_x = kInf;
            whole([&](float x, uint32_t) {
                least_x = __builtin_fminf(least_x, x > -kInf ? x : kInf);
            });
#pragma unroll
            for (int d = 1; d < 64; d *= 2) least_x = __builtin_fminf(least_x, __shfl_xor(least_x, d));
            if (lane == 0) wave_min[wave] = least_x;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kSampleWaves; ++w) least_x = __builtin_fminf(least_x, wave_min[w]);
            const double range = weigh.max - least_x;
            if (range < span) {
                span = range;
                per = (float)((kBins - 1) / span);
            }
        }
        // differences of logits within the span are 32-bit numbers, not infinite
        const bool stepped = top < kInf && span > 0. && span <= (double)kMaxF && per < kInf;
        // descending with x; kBins for a masked one or one of no weight
        auto bin = [&](float x) {
            return (uint32_t)__builtin_fminf((top - x) * per, (float)kBins);
        };
        // the step in which the k-th counted token lies goes to s_b2; or false
        auto find_k = [&]() {
            uint32_t c[4], sum[1] = {0}, all[1];
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[0] += c[j] = sh.bins[4 * tid + j];
            scan_before(sum, wave32, all);
            uint32_t at = sum[0];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (at < (uint32_t)k && at + c[j] >= (uint32_t)k) s_b2 = 4 * tid + j, s_c2 = at + c[j];
                at += c[j];
            }
            __syncthreads();
            return all[0] >= (uint32_t)k;
        };
        auto list_to = [&](uint32_t last) {
            whole([&](float x, uint32_t i) {
                if ((top - x) * per < (float)(last + 1)) append(x, i);
            });
            __syncthreads();
            in_list = s_n <= kList;
        };
        auto clear = [&]() {
            __syncthreads();
            for (int b = tid; b < kBins; b += kSampleThreads) sh.bins[b] = 0;
            if (tid == 0) s_n = 0, s_b2 = kBins - 1;
            __syncthreads();
        };
        if (by_k && stepped) {
            if (k <= kSampleThreads) {
                if (const uint32_t b = bin(mine); b < kBins) atomicAdd(&sh.bins[b], 1u);
                __syncthreads();
                if (find_k()) list_to(s_b2);
            }
            if (!in_list) {
                clear();
                whole([&](float x, uint32_t) {
                    if (const uint32_t b = bin(x); b < kBins) atomicAdd(&sh.bins[b], 1u);
                });
                __syncthreads();
                by_k = find_k();  // else all that have a weight
                if (by_k && s_c2 <= kList) list_to(s_b2);
            }
        } else if (by_k) {
            u64 n[1] = {0}, all[1];
            whole([&](float x, uint32_t i) { n[0] += border.keeps(x, i); });
            __syncthreads();
            scan_before(n, wave64, all);
            by_k = all[0] > (u64)k;
        }
        if (by_k && in_list && s_n <= kRank) {
            rank((uint32_t)k, by_p, 0, 0);
        } else {
            if (by_k) select(std::false_type{}, (u64)k);
            u64 target = 0, outside = 0;  // weights; outside: of those above the list's
            if (by_p && !by_k && stepped) {
                clear();
                // A weight is its step's largest, 2^(-step b), times 1 - frac step ln 2, less
                // than 2^-14 off (a step is 52 / 4096 at most): integers again, whose
                // sums stay below 2^32 (adding 32-bit floats here takes 10 times as long)
                const float step = (float)(weigh.scale / (double)per);
                const float whole_step = __uint_as_float((uint32_t)(127 + a.share_bits) << 23);
                const float slope = -step * kLn2 * whole_step;
                whole([&](float x, uint32_t) {
                    const float d = (top - x) * per;
                    const uint32_t b = d < (float)kBins ? (uint32_t)d : kBins + lane;
                    atomicAdd(&sh.bins[b],
                              (uint32_t)fma32(__builtin_amdgcn_fractf(d), slope, whole_step));
                });
                __syncthreads();
                double c[4], sum[1] = {0.}, all[1];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    c[j] = (double)sh.bins[4 * tid + j] *
                           (double)exp2_hw(-step * (float)(4 * tid + j));
                    sum[0] += c[j];
                }
                scan_before(sum, bounds, all);
                // (beyond some 2^19 tokens a share's rounding may pass these margins, and
                // the border lie outside the steps: then the whole row is searched)
                uint32_t b1 = kBins - 1, b2 = kBins - 1;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    sum[0] += c[j];
                    if (sum[0] >= p * 0.9999 * all[0] && b1 == kBins - 1) b1 = 4 * tid + j;
                    if (sum[0] >= p * 1.0001 * all[0] && b2 == kBins - 1) b2 = 4 * tid + j;
                }
                if (b1 < kBins - 1) atomicMin(&s_b1, b1);
                if (b2 < kBins - 1) atomicMin(&s_b2, b2);
                __syncthreads();
                u64 w[3] = {0, 0, 0}, sums[3];  // of all, above the list, in it
                const float f1 = (float)s_b1, f2 = (float)(s_b2 + 1);
                by_least([&](auto all) {
                    group_sums([&](int32_t at, const Vec<T, V>& x) {
                        u64 up = 0;
                        u64 any = 0;  // lanes with tokens in the steps, which are seen to
                                      // afterwards: a branch for each holds up the others'
                                      // weights (100 us against 90)
#pragma unroll
                        for (int e = 0; e < V; ++e) {
                            const float y = T::load(x.e[e]);
                            const u64 v = weigh(y);
                            const float d = (top - y) * per;
                            const u64 above = d < f1 ? v : 0;
                            w[0] += v;
                            if (!all.value) w[1] += above;
                            up += all.value || above >= least ? above : 0;
                            any |= __ballot(d >= f1 && d < f2);
                        }
                        if (any) {
#pragma unroll
                            for (int e = 0; e < V; ++e) {
                                const float y = T::load(x.e[e]), d = (top - y) * per;
                                if (!(d >= f1 && d < f2)) continue;
                                w[2] += weigh(y);
                                append(y, (uint32_t)(at + e));
                            }
                        }
                        return up;
                    });
                });
                if (least == 0) w[1] = tid < kSums ? sh.sums[tid] : 0;
                scan_before(w, wave64, sums);
                target = min_share(p, sums[0]);
                // the steps' sums are rounded: these decide
                in_list = summed =
                    s_n <= kList && sums[1] < target && target - sums[1] <= sums[2];
                if (in_list) outside = sums[1];
            } else if (by_p) {
                u64 w[1] = {0}, all[1];
                tokens([&](float x, uint32_t i) { w[0] += border.keeps(x, i) ? weigh(x) : 0; });
                __syncthreads();
                scan_before(w, wave64, all);
                target = min_share(p, all[0]);
            }
            if (by_p && summed && s_n <= kRank)
                rank(kRank, true, target, outside);
            else if (by_p)
                select(std::true_type{}, target - outside);
        }
    }

    // 5. sums of what is kept
    auto kept = [&](float x, uint32_t i) -> u64 {
        if (!border.keeps(x, i)) return 0;
        const u64 v = weigh(x);
        return v >= least ? v : 0;
    };
    __syncthreads();
    if (in_list) {
        if (!summed)
            for (int i = tid; i < kSums; i += kSampleThreads) sh.sums[i] = 0;
        __syncthreads();
        tokens([&](float x, uint32_t i) {
            if (const u64 v = kept(x, i)) atomicAdd(&sh.sums[i / R::kPiece / r.G], v);
        });
        __syncthreads();
    } else if (border.x == -kMaxF && border.idx == 0xffffffffu) {  // all, masked ones weigh 0
        by_least([&](auto all) {
            group_sums([&](int32_t, const Vec<T, V>& x) {
                u64 sum = 0;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const u64 v = weigh(T::load(x.e[e]));
                    sum += all.value || v >= least ? v : 0;
                }
                return sum;
            });
        });
    } else {
        group_sums([&](int32_t at, const Vec<T, V>& x) {
            u64 sum = 0;
#pragma unroll
            for (int e = 0; e < V; ++e) sum += kept(T::load(x.e[e]), (uint32_t)(at + e));
            return sum;
        });
    }
    // each wave finds the group, whose wave goes on
    static_assert(kSums == 128, "two sums a lane");
    const u64 s0 = sh.sums[2 * lane], s1 = sh.sums[2 * lane + 1];
    const u64 upto = wave_upto(s0 + s1), sum = lane64(upto, 63);
    double share = (double)a.u[row];
    share = share > 0. ? share : 0.;
    u64 target = share < 1. ? (u64)(share * (double)sum) : sum - 1;
    target = target < sum ? target : sum - 1;
    const int win = __builtin_ctzll(__ballot(upto > target));
    u64 before = upto - s0 - s1;
    const bool second = before + s0 <= target;
    if (second) before += s0;
    const int group = __builtin_amdgcn_readlane(2 * lane + second, win);
    before = lane64(before, win);
    if (group % kSampleWaves != wave) return;
    for (int32_t i = 0; i < r.G; ++i) {
        const int32_t first = (group * r.G + i) * R::kPiece, at = first + lane * V;
        if (first >= r.n) return;
        const Vec<T, V> v = r.load(first);
        u64 x[V], mine = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) mine += x[e] = kept(T::load(v.e[e]), (uint32_t)(at + e));
        const u64 up = wave_upto(mine);
        const u64 mask = __ballot(before + up > target);
        if (mask) {
            if (lane != __builtin_ctzll(mask)) return;
            before += up - mine;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                if (before + x[e] > target) {
                    put(at + e);
                    return;
                }
                before += x[e];
            }
        }
        before += lane64(up, 63);
    }
}

template <typename T>
hipError_t launch_sample(const SampleArgs& a, hipStream_t st)
{
    k_sample<T><<<dim3((unsigned)a.rows), dim3(kSampleThreads), 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace seq
}  // namespace canon
