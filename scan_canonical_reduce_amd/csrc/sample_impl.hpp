// Sampling of the next token.
//
// A weight w = exp((logit - max) / temperature) <= 1 is computed in 64 bits and held
// as an integer multiple of 2^-bits, so that the sum of a whole row fits 62 bits:
// integer sums are the same in any order, so a row can be cut and its filters'
// borders searched in any way without changing which token u picks.
//
// No sort: the tokens that top_k and top_p keep are the ones above a threshold logit
// and some of those at it, lowest index first.  The threshold is found digit by digit
// of its ordered 32-bit key, from counts (top_k) or sums of weights (top_p) by digit.
#pragma once

#include "launch.hpp"
#include "sample.hpp"

namespace canon {
namespace seq {

typedef unsigned long long u64;

// Ascending with the logit; 0 for a masked one (NaN, minus infinity).
__device__ __forceinline__ uint32_t logit_key(float x)
{
    const uint32_t b = __float_as_uint(x + 0.f);  // one zero
    const uint32_t k = b >> 31 ? ~b : b | 0x80000000u;
    return x > -__builtin_inff() ? k : 0u;
}
__device__ __forceinline__ float key_logit(uint32_t k)
{
    return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k);
}

// 2^y for y <= 0 as a multiple of 2^-bits, and its value.  The polynomial is the one of
// degree 10 whose largest error on [-1/2, 1/2] is smallest (2^-51.5 relative with the
// rounded coefficients); adding 2^52 leaves the rounded integer in the low bits.
__device__ __forceinline__ double exp2_64(double y)
{
    const double n = __builtin_rint(y), r = y - n;
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
    return __builtin_amdgcn_ldexp(p, (int)n);
}
__device__ __forceinline__ u64 fixed(double w, int bits)
{
    const double v = __builtin_amdgcn_ldexp(w, bits) + 0x1p52;
    return __builtin_bit_cast(u64, v) & 0xfffffffffffffull;
}

// A row's weights.
struct Weights {
    double max, scale, least;  // scale: log2(e) / temperature; least: min_p
    int bits;
    __device__ __forceinline__ u64 operator()(uint32_t key) const
    {
        if (key == 0) return 0;
        const double x = key_logit(key);
        double y = x == max ? 0. : (x - max) * scale;  // infinities
        if (!(y >= -60.)) return 0;                     // rounds to 0
        const double w = exp2_64(y);
        return w >= least ? fixed(w, bits) : 0;
    }
};

constexpr int kSampleThreads = 1024;
constexpr int kSampleWaves = kSampleThreads / 64;

// From the highest of 256 bins down, the first at which the sum reaches target (which
// is at most the whole sum): its number and the sum above it.  One wave; hist is
// overwritten by nobody meanwhile.
__device__ __forceinline__ void pick_bin(const u64* hist, u64 target, int* bin, u64* above)
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
    int i = 0;
#pragma unroll
    for (; i < 3; ++i) {
        if (before + v[i] >= target) break;
        before += v[i];
    }
    *bin = b0 - i;
    *above = before;
}

template <typename T>
__global__ __launch_bounds__(kSampleThreads) void k_sample(SampleArgs a)
{
    __shared__ u64 hist[256];
    __shared__ u64 wsum[kSampleWaves];
    __shared__ uint32_t wmax[kSampleWaves];
    __shared__ int s_bin;
    __shared__ u64 s_above;
    const int64_t row = blockIdx.x;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const typename T::store_t* x =
        static_cast<const typename T::store_t*>(a.logits) + row * a.ld;
    const int32_t n = a.vocab;

    // the largest
    uint32_t top = 0;
    for (int32_t i = tid; i < n; i += kSampleThreads) {
        const uint32_t k = logit_key(ld<T>(x + i));
        top = k > top ? k : top;
    }
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const uint32_t o = __shfl_xor(top, d);
        top = o > top ? o : top;
    }
    if (lane == 0) wmax[wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSampleWaves; ++w) top = wmax[w] > top ? wmax[w] : top;
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
    int32_t k = a.top_k ? a.top_k[row] : a.top_k_all;
    const double p = a.top_p ? a.top_p[row] : a.top_p_all;
    double least = a.min_p ? a.min_p[row] : a.min_p_all;
    least = !(least > 0.) ? 0. : least < 1. ? least : 1.;
    Weights w{key_logit(top), 1.4426950408889634 / t, least, a.bits};
    if (!(t > 0.)) {
        w.scale = 0.;
        k = 1;
    }

    // the threshold key and how many tokens at it are kept
    uint32_t limit = 0;
    int32_t ties = 0x7fffffff;
    // digit by digit; value(key): what a token counts; tie_at, tie_sum: the key whose
    // tokens count tie_sum together
    auto select = [&](u64 target, auto value, uint32_t tie_at, u64 tie_sum) {
        uint32_t prefix = 0;
        u64 above = 0;
        for (int shift = 24; shift >= 0; shift -= 8) {
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            auto mine = [&](uint32_t key) {
                return shift == 24 || (key >> shift >> 8) == (prefix >> shift >> 8);
            };
            for (int32_t i = tid; i < n; i += kSampleThreads) {
                const uint32_t key = logit_key(ld<T>(x + i));
                if (key <= tie_at || !mine(key)) continue;
                if (const u64 v = value(key)) atomicAdd(&hist[key >> shift & 255], v);
            }
            if (tid == 0 && tie_at && mine(tie_at))
                atomicAdd(&hist[tie_at >> shift & 255], tie_sum);
            __syncthreads();
            if (wave == 0) pick_bin(hist, target - above, &s_bin, &s_above);
            __syncthreads();
            prefix |= (uint32_t)s_bin << shift;
            above += s_above;
            __syncthreads();
        }
        limit = prefix;
        return target - above;  // what the tokens at the limit have to give
    };
    // sum over the row's tokens, in every thread
    auto total = [&](auto value) {
        u64 s = 0;
        for (int32_t i = tid; i < n; i += kSampleThreads) s += value(logit_key(ld<T>(x + i)));
#pragma unroll
        for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
        __syncthreads();
        if (lane == 0) wsum[wave] = s;
        __syncthreads();
        s = 0;
#pragma unroll
        for (int v = 0; v < kSampleWaves; ++v) s += wsum[v];
        return s;
    };
    if (k > 0 && k < n) {
        auto one = [](uint32_t key) { return (u64)(key != 0); };
        if (total(one) > (u64)k) ties = (int32_t)select((u64)k, one, 0, 0);
    }
    Weights all = w;  // without min_p, which comes after top_p
    all.least = 0.;
    auto kept_sum = [&](const Weights& f) {
        u64 s = total([&](uint32_t key) { return key > limit ? f(key) : 0; });
        return limit ? s + ties * f(limit) : s;
    };
    if (p < 1.) {
        const u64 sum = kept_sum(all);
        const double want = __builtin_ceil(p * (double)sum);
        u64 target = want >= 1. ? (u64)want : 1;
        target = target < sum ? target : sum;
        const uint32_t at = limit;
        const u64 left =
            select(target, all, at, at ? ties * all(at) : 0);
        const u64 each = all(limit);
        const u64 need = (left + each - 1) / each;
        ties = limit == at && need > (u64)ties ? ties : (int32_t)need;
    }

    // the kept tokens in index order: each wave a stretch
    const u64 sum = kept_sum(w);
    double at = (double)(a.u ? a.u[row] : 0.f);
    at = at > 0. ? at : 0.;
    const double want = at * (double)sum;
    u64 target = (u64)want;  // up to 2^62: no overflow
    target = at < 1. && target < sum ? target : sum - 1;
    const int32_t part = (n + kSampleWaves * 64 - 1) / (kSampleWaves * 64) * 64;
    const int32_t i0 = wave * part, i1 = i0 + part < n ? i0 + part : n;
    // tokens at the limit before this wave's stretch
    __syncthreads();
    uint32_t mine = 0;
    for (int32_t i = i0 + lane; i < i1; i += 64) mine += logit_key(ld<T>(x + i)) == limit;
#pragma unroll
    for (int d = 1; d < 64; d *= 2) mine += __shfl_xor(mine, d);
    if (lane == 0) wmax[wave] = mine;
    __syncthreads();
    uint32_t rank0 = 0;
    for (int v = 0; v < wave; ++v) rank0 += wmax[v];
    auto value = [&](int32_t i, uint32_t& rank) {
        const uint32_t key = i < i1 ? logit_key(ld<T>(x + i)) : 0;
        const bool tie = limit != 0 && key == limit;
        const u64 mask = __ballot(tie);
        const uint32_t r = rank + __popcll(mask & ((1ull << lane) - 1));
        rank += __popcll(mask);
        return key > limit || (tie && r < (uint32_t)ties) ? w(key) : 0;
    };
    u64 s = 0;
    uint32_t rank = rank0;
    for (int32_t i = i0; i < i1; i += 64) s += value(i + lane, rank);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) s += __shfl_xor(s, d);
    if (lane == 0) wsum[wave] = s;
    __syncthreads();
    u64 before = 0;
    for (int v = 0; v < wave; ++v) before += wsum[v];
    if (target < before || target >= before + s) return;  // another wave's
    rank = rank0;
    for (int32_t i = i0; i < i1; i += 64) {
        const u64 v = value(i + lane, rank);
        u64 upto = v;
#pragma unroll
        for (int d = 1; d < 64; d *= 2) {
            const u64 o = __shfl_up(upto, d);
            if (lane >= d) upto += o;
        }
        const u64 hit = __ballot(before + upto > target);
        if (hit) {
            if (lane == __builtin_ctzll(hit)) put(i + lane);
            return;
        }
        before += __shfl(upto, 63);
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
