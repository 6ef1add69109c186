// Sampling of the next token, a workgroup for each row.
//
// A weight w = exp((logit - max) / temperature) <= 1 is computed in 64 bits and held
// as an integer multiple of 2^-bits, so that the sum of a whole row fits 62 bits:
// integer sums are the same in any order, so a row can be cut and its filters'
// borders searched in any way without changing which token u picks.
//
// No sort: what top_k and top_p keep are the tokens up to a border (key, index) in
// the order of descending keys, which ascend with the logit, and ascending indexes.
//   1. The row's largest and smallest logit.
//   2. With a filter, the tokens counted in kBins equal steps of the logit from the
//      largest down.  The counts tell in which step the top_k-th token lies, and, as a
//      step's weights are known to a step, between which two the top_p border lies.
//   3. Those tokens go to a list in LDS: for top_k all from the border's step up, for
//      top_p alone those of the steps in question, while all weights are summed.
//   4. The border is found in the list digit by digit, by counts or sums of weights.
//   5. Sums of the kept weights by pieces of the row in index order, the piece in
//      which u's share falls, and the token in it.
// Where a list does not fit (thousands of tokens in a step, as where all are equal),
// the whole row is read again for every digit instead.
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
constexpr int kSums = 8 * kSampleWaves;

// The key of a logit: ascending, one for both zeros, 0 for a masked one (NaN, minus
// infinity); and the logit of a key that is not 0.  As wide as the type.
template <typename T>
__device__ __forceinline__ uint32_t logit_key(typename T::store_t raw)
{
    if constexpr (sizeof(raw) == 4) {
        const uint32_t b = __float_as_uint(raw + 0.f);
        const uint32_t k = b >> 31 ? ~b : b | 0x80000000u;
        return raw > -__builtin_inff() ? k : 0u;
    } else {
        const uint32_t b = raw == 0x8000u ? 0u : raw;
        const uint32_t k = b >> 15 ? ~b & 0xffffu : b | 0x8000u;
        return T::load(raw) > -__builtin_inff() ? k : 0u;
    }
}
template <typename T>
__device__ __forceinline__ float key_logit(uint32_t k)
{
    if constexpr (sizeof(typename T::store_t) == 4)
        return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
    else
        return T::load((uint16_t)(k >> 15 ? k & 0x7fffu : ~k));
}
template <typename T>
__device__ __forceinline__ typename T::store_t masked_logit()
{
    if constexpr (sizeof(typename T::store_t) == 4)
        return -__builtin_inff();
    else
        return T::round(-__builtin_inff());
}

// A row's weights.  2^y, y = (x - max) / temperature in binary steps, is 2^n times the
// polynomial of degree 10 whose largest error on [-1/2, 1/2] is smallest (2^-51.5
// relative with its rounded coefficients; 1 at 0).  Adding 2^(52 - bits) leaves the
// rounded multiple of 2^-bits in the low bits of the sum.  Below 2^-60 it is 0.
struct Weights {
    double max, scale, unit;  // scale: log2(e) / temperature
    __device__ __forceinline__ u64 operator()(float x) const
    {
        // plus infinity as the largest number: where one is there, only such are kept
        const double d = (double)__builtin_fminf(x, kMaxF) - max;
        const double y = __builtin_fmax(d * scale, -60.);  // -60 for a NaN
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

// The kept tokens: those above the key, and at it up to the index.
struct Border {
    uint32_t key, idx;
    __device__ __forceinline__ bool keeps(uint32_t k, uint32_t i) const
    {
        return k > key || (k == key && i <= idx);
    }
};

// The weights that a share p of sum takes at least: one unit, and no more than all.
__device__ __forceinline__ u64 min_share(double p, u64 sum)
{
    const double want = __builtin_ceil(p * (double)sum);
    const u64 v = want >= 1. ? (u64)want : 1;
    return v < sum ? v : sum;
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
    u64 upto = sum;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const u64 o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
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

// The sum over the threads before this one, and of all.  lds: a value a wave, not to
// be used again before the next barrier.
template <typename V>
__device__ __forceinline__ V scan_before(V v, V* lds, V& all)
{
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    V upto = v;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const V o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    if (lane == 63) lds[wave] = upto;
    __syncthreads();
    V before = upto - v;
    all = 0;
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        const V s = lds[w];
        if (w < wave) before += s;
        all += s;
    }
    return before;
}

// A row in pieces of 64 vectors.  Wave w has the pieces (16 g + w) G ... + G - 1 of
// each group g, so that sums by (g, w) are sums of stretches in index order.
template <typename T>
struct Row {
    using E = typename T::store_t;
    static constexpr int V = 16 / sizeof(E), kPiece = 64 * V, U = 4;
    const E* x;
    int32_t n, G, groups;
    __device__ __forceinline__ int32_t piece(int g, int w) const
    {
        return (g * kSampleWaves + w) * G;
    }
    __device__ __forceinline__ Vec<T, V> load(int32_t at) const
    {
        if (at + V <= n) return ld_any<T, V, false>(x + at);
        Vec<T, V> v;
#pragma unroll
        for (int e = 0; e < V; ++e) v.e[e] = at + e < n ? x[at + e] : masked_logit<T>();
        return v;
    }
    // f(g, index of the vector's first token, vector) over the wave's vectors
    template <class F>
    __device__ __forceinline__ void each(F&& f) const
    {
        const int lane = threadIdx.x & 63, wave = uniform((int32_t)(threadIdx.x >> 6));
        int g = 0, i = 0;
        while (g < groups) {
            Vec<T, V> v[U];
            int32_t at[U];
            int gs[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int32_t first = (piece(g, wave) + i) * kPiece;
                gs[u] = g < groups && first < n ? g : -1;
                at[u] = first + lane * V;
                if (gs[u] >= 0) v[u] = load(at[u]);
                if (++i == G) i = 0, ++g;
            }
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (gs[u] >= 0) f(gs[u], at[u], v[u]);
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
        uint32_t bins[kBins];
        u64 sums[kSums];
    } sh;
    __shared__ uint32_t lkey[kList], lidx[kList];
    __shared__ u64 hist[256], wave64[kSampleWaves];
    __shared__ double wave_lo[kSampleWaves], wave_hi[kSampleWaves];
    __shared__ uint32_t wave_a[kSampleWaves], wave_b[kSampleWaves];
    __shared__ Picked picked;
    __shared__ uint32_t s_n, s_first, s_b1, s_b2, s_c1, s_c2;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    R r;
    r.x = static_cast<const E*>(a.logits) + row * a.ld;
    r.n = a.vocab;
    const int32_t pieces = (r.n + R::kPiece - 1) / R::kPiece;
    r.G = (pieces + kSums - 1) / kSums;
    r.groups = r.G ? (pieces + kSampleWaves * r.G - 1) / (kSampleWaves * r.G) : 0;

    // 1. the largest and the smallest key
    uint32_t top = 0, low = 0xffffffffu;
    r.each([&](int, int32_t, const Vec<T, V>& v) {
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const uint32_t k = logit_key<T>(v.e[e]);
            top = k > top ? k : top;
            low = k - 1 < low ? k - 1 : low;  // a masked one is the largest here
        }
    });
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_xor(top, d), p = __shfl_xor(low, d);
        top = o > top ? o : top;
        low = p < low ? p : low;
    }
    if (lane == 0) wave_a[wave] = top, wave_b[wave] = low;
    for (int b = tid; b < kBins; b += kSampleThreads) sh.bins[b] = 0;
    if (tid == 0) s_n = 0, s_first = 0xffffffffu, s_b1 = s_b2 = kBins - 1;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) {
        top = wave_a[w] > top ? wave_a[w] : top;
        low = wave_b[w] < low ? wave_b[w] : low;
    }
    auto put = [&](int64_t id) {
        if (a.ids64)
            static_cast<int64_t*>(a.ids)[row] = id;
        else
            static_cast<int32_t*>(a.ids)[row] = (int32_t)id;
    };
    if (top == 0) {
        if (tid == 0) put(-1);
        return;
    }
    const double t = a.temperature ? a.temperature[row] : a.temperature_all;
    const int32_t k = !(t > 0.) ? 1 : a.top_k ? a.top_k[row] : a.top_k_all;
    const double p = a.top_p ? a.top_p[row] : a.top_p_all;
    const double min_p = a.min_p ? a.min_p[row] : a.min_p_all;
    auto whole = [&](auto token) {
        r.each([&](int, int32_t at, const Vec<T, V>& v) {
#pragma unroll
            for (int e = 0; e < V; ++e) token(logit_key<T>(v.e[e]), (uint32_t)(at + e));
        });
    };
    if (k == 1) {  // the largest, whatever the other settings
        uint32_t first = 0xffffffffu;
        whole([&](uint32_t key, uint32_t i) { first = key == top && i < first ? i : first; });
        if (first != 0xffffffffu) atomicMin(&s_first, first);
        __syncthreads();
        if (tid == 0) put(s_first);
        return;
    }

    const float fmax = key_logit<T>(top), fmin = key_logit<T>(low + 1);
    const Weights weigh{(double)__builtin_fminf(fmax, kMaxF),
                        __builtin_fmin(1.4426950408889634 / t, 1e300),
                        __builtin_amdgcn_ldexp(1., 52 - a.bits)};
    const u64 one = 1ull << a.bits;
    const u64 least = !(min_p > 0.) ? 0 : min_p < 1. ? (u64)__builtin_ceil(min_p * (double)one) : one;
    // the row's unmasked tokens; beside an infinite one, those alone
    const bool infinite = fmax == __builtin_inff();
    Border border{infinite ? top : 1u, 0xffffffffu};
    bool in_list = false;  // the list holds all tokens that are still in question

    auto tokens = [&](auto token) {
        if (!in_list) return whole(token);
        for (uint32_t i = tid; i < s_n; i += kSampleThreads) token(lkey[i], lidx[i]);
    };
    auto append = [&](uint32_t key, uint32_t i) {
        const uint32_t at = atomicAdd(&s_n, 1u);
        if (at < kList) lkey[at] = key, lidx[at] = i;
    };
    auto sum_all = [&](u64 v) {
        u64 sum;
        __syncthreads();
        scan_before(v, wave64, sum);
        return sum;
    };
    // 4. the first tokens in order, of those in question and kept by the border, whose
    // values add up to target (at most the sum of all): the border behind them
    auto select = [&](auto weighted, u64 target) {
        uint32_t prefix = 0;
        u64 above = 0, here = 0;
        auto digit = [&](auto token) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            tokens(token);
            __syncthreads();
            if (wave == 0) pick_bin(hist, target - above, &picked);
            __syncthreads();
            above += picked.above;
            here = picked.here;
            return (uint32_t)picked.bin;
        };
#pragma unroll 1
        for (int shift = 8 * (kDigits - 1); shift >= 0; shift -= 8)
            prefix |= digit([&](uint32_t key, uint32_t i) {
                          if (border.keeps(key, i) &&
                              (u64)key >> (shift + 8) == (u64)prefix >> (shift + 8))
                              atomicAdd(&hist[key >> shift & 255],
                                        weighted.value ? weigh(key_logit<T>(key)) : 1ull);
                      })
                      << shift;
        u64 need = target - above;
        if (weighted.value) {
            const u64 each = weigh(key_logit<T>(prefix));
            need = (need + each - 1) / each;
            here /= each;
        }
        uint32_t idx = prefix == border.key ? border.idx : 0xffffffffu;
        if (need < here) {  // the lowest indexes of the ones at the key
            idx = 0;
            target = need;
            above = 0;
#pragma unroll 1
            for (int shift = 16; shift >= 0; shift -= 8) {
                if (r.n <= 1 << shift) continue;
                idx |= (255u - digit([&](uint32_t key, uint32_t i) {
                            if (key == prefix && border.keeps(key, i) &&
                                i >> (shift + 8) == idx >> (shift + 8))
                                atomicAdd(&hist[255 - (i >> shift & 255)], 1ull);
                        }))
                       << shift;
            }
        }
        border = Border{prefix, idx};
    };
    // sums of value(raw logit, index) by group
    auto group_sums = [&](auto value) {
        for (int i = tid; i < kSums; i += kSampleThreads) sh.sums[i] = 0;
        __syncthreads();
        int of = -1;
        u64 sum = 0;
        auto flush = [&]() {
#pragma unroll
            for (int d = 1; d < 64; d *= 2) sum += __shfl_xor(sum, d);
            if (lane == 0 && of >= 0) sh.sums[of * kSampleWaves + wave] = sum;
            sum = 0;
        };
        r.each([&](int g, int32_t at, const Vec<T, V>& v) {
            if (g != of) flush();
            of = g;
#pragma unroll
            for (int e = 0; e < V; ++e) sum += value(v.e[e], (uint32_t)(at + e));
        });
        flush();
        __syncthreads();
    };

    // 2. and 3.
    bool summed = false;  // weights outside the list are in the groups' sums
    const bool by_p = p < 1.;
    if ((k > 0 && k < r.n) || by_p) {
        // steps over the row's range, or as far as weights are not 0
        const double range = weigh.max - fmin, reach = 36. * t;
        const double span = infinite ? 0. : range < reach ? range : reach;
        const float per = (float)(kBins / span);
        auto bin = [&](uint32_t key) {
            const float b = (fmax - key_logit<T>(key)) * per;
            return (uint32_t)(b < (float)(kBins - 1) ? (int)b : b == b ? kBins - 1 : 0);
        };
        whole([&](uint32_t key, uint32_t i) {
            if (border.keeps(key, i)) atomicAdd(&sh.bins[bin(key)], 1u);
        });
        __syncthreads();
        uint32_t c[4], sum = 0, total;
#pragma unroll
        for (int j = 0; j < 4; ++j) sum += c[j] = sh.bins[4 * tid + j];
        const uint32_t before = scan_before(sum, wave_a, total);
        const bool by_k = k > 0 && total > (uint32_t)k;
        u64 outside = 0;  // weights above the list's
        u64 target = 0;
        if (by_k) {
            uint32_t at = before;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (at < (uint32_t)k && at + c[j] >= (uint32_t)k) s_b2 = 4 * tid + j, s_c2 = at + c[j];
                at += c[j];
            }
            __syncthreads();
            if (s_c2 <= kList) {
                const uint32_t b2 = s_b2;
                whole([&](uint32_t key, uint32_t i) {
                    if (border.keeps(key, i) && bin(key) <= b2) append(key, i);
                });
                __syncthreads();
                in_list = true;
            }
            select(std::false_type{}, (u64)k);
            if (by_p) {
                u64 s = 0;
                tokens([&](uint32_t key, uint32_t i) {
                    if (border.keeps(key, i)) s += weigh(key_logit<T>(key));
                });
                target = sum_all(s);
            }
        } else if (by_p) {
            // bounds of the weights of each step, and of their sums
            const float step = (float)(span * weigh.scale / kBins);
            double lo[4], hi[4], lo4 = 0., hi4 = 0., lo_all, hi_all;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float b = (float)(4 * tid + j);
                lo[j] = b < (float)(kBins - 1) ? c[j] * (double)exp2_hw(-step * (b + 1.f)) * 0.9999 : 0.;
                hi[j] = c[j] * (double)exp2_hw(-step * b) * 1.0001;
                lo4 += lo[j];
                hi4 += hi[j];
            }
            double l = scan_before(lo4, wave_lo, lo_all), h = scan_before(hi4, wave_hi, hi_all);
            uint32_t b1 = kBins - 1, b2 = kBins - 1;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                l += lo[j];
                h += hi[j];
                if (h >= p * lo_all && b1 == kBins - 1) b1 = 4 * tid + j;
                if (l >= p * hi_all && b2 == kBins - 1) b2 = 4 * tid + j;
            }
            atomicMin(&s_b1, b1);
            atomicMin(&s_b2, b2);
            __syncthreads();
            b1 = s_b1;
            b2 = s_b2;
            uint32_t at = before;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if ((uint32_t)(4 * tid + j) == b1) s_c1 = at;
                at += c[j];
                if ((uint32_t)(4 * tid + j) == b2) s_c2 = at;
            }
            __syncthreads();
            const bool fits = s_c2 - s_c1 <= kList;
            u64 weights = 0, listed = 0;
            group_sums([&](E raw, uint32_t i) -> u64 {
                const uint32_t key = logit_key<T>(raw);
                if (!border.keeps(key, i)) return 0;
                const u64 v = weigh(T::load(raw));
                const uint32_t b = bin(key);
                weights += v;
                if (b < b1) {
                    outside += v;
                } else if (b <= b2) {
                    listed += v;
                    if (fits) append(key, i);
                }
                return b < b1 && v >= least ? v : 0;
            });
            target = sum_all(weights);
            outside = sum_all(outside);
            listed = sum_all(listed);
            const u64 want = min_share(p, target);
            // the bounds are rounded: the sums decide
            in_list = summed = fits && outside < want && want - outside <= listed;
            if (!in_list) outside = 0;
        }
        if (by_p) select(std::true_type{}, min_share(p, target) - outside);
    }

    // 5. sums of what is kept
    auto kept = [&](uint32_t key, uint32_t i) -> u64 {
        if (!border.keeps(key, i)) return 0;
        const u64 v = weigh(key_logit<T>(key));
        return v >= least ? v : 0;
    };
    if (in_list) {
        if (!summed) {
            __syncthreads();
            for (int i = tid; i < kSums; i += kSampleThreads) sh.sums[i] = 0;
        }
        __syncthreads();
        tokens([&](uint32_t key, uint32_t i) {
            if (const u64 v = kept(key, i)) atomicAdd(&sh.sums[i / R::kPiece / r.G], v);
        });
        __syncthreads();
    } else {
        __syncthreads();
        group_sums([&](E raw, uint32_t i) { return kept(logit_key<T>(raw), i); });
    }
    // each wave finds the group, whose wave goes on
    static_assert(kSums == 128, "two sums a lane");
    const u64 s0 = sh.sums[2 * lane], s1 = sh.sums[2 * lane + 1];
    u64 upto = s0 + s1;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const u64 o = __shfl_up(upto, d);
        if (lane >= d) upto += o;
    }
    const u64 sum = __shfl(upto, 63);
    double share = (double)a.u[row];
    share = share > 0. ? share : 0.;
    u64 target = share < 1. ? (u64)(share * (double)sum) : sum - 1;
    target = target < sum ? target : sum - 1;
    const u64 hit = __ballot(upto > target);
    const int win = __builtin_ctzll(hit);
    u64 before = upto - s0 - s1;
    const bool second = before + s0 <= target;
    if (second) before += s0;
    const int group = __shfl(2 * lane + second, win);
    before = __shfl(before, win);
    if (group % kSampleWaves != wave) return;
    for (int32_t i = 0; i < r.G; ++i) {
        const int32_t at = (group * r.G + i) * R::kPiece + lane * V;
        const Vec<T, V> v = r.load(at);
        u64 x[V], mine = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) mine += x[e] = kept(logit_key<T>(v.e[e]), (uint32_t)(at + e));
        u64 up = mine;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const u64 o = __shfl_up(up, d);
            if (lane >= d) up += o;
        }
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
        before += __shfl(up, 63);
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
