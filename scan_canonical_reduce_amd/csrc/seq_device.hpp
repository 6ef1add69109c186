// Device helpers of the sequence operators (canon_seq.h): element types,
// scalar functions, lane moves and the walk over sequences.
#pragma once

#include <hip/hip_bf16.h>
#include <hip/hip_fp16.h>
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/canon_seq.h"

namespace canon {
namespace seq {

// ---------------------------------------------------------------- element types
struct F32 {
    using store_t = float;
    static __device__ __forceinline__ float load(float v) { return v; }
    static __device__ __forceinline__ float round(float v) { return v; }
};
struct BF16 {
    using store_t = uint16_t;
    static __device__ __forceinline__ float load(uint16_t v)
    {
        return __uint_as_float((uint32_t)v << 16);
    }
    // to nearest even; a NaN keeps its upper bits and stays a NaN
    static __device__ __forceinline__ uint16_t round(float v)
    {
        return __builtin_bit_cast(uint16_t, (__bf16)v);
    }
};
struct F16 {
    using store_t = uint16_t;
    static __device__ __forceinline__ float load(uint16_t v)
    {
        return (float)__builtin_bit_cast(_Float16, v);
    }
    // The empty asm keeps the 32-bit value a value: without it a product before
    // the conversion becomes one mixed-precision FMA, which rounds the exact
    // product to 16 bits, and the stored bits would depend on the code around.
    static __device__ __forceinline__ uint16_t round(float v)
    {
        asm("" : "+v"(v));
        return __builtin_bit_cast(uint16_t, (_Float16)v);
    }
};

template <typename T>
__device__ __forceinline__ float ld(const typename T::store_t* p)
{
    return T::load(*p);
}

template <typename T>
__device__ __forceinline__ void st(typename T::store_t* p, float v)
{
    *p = T::round(v);
}

// V consecutive elements as one (or, for 32-bit elements beyond 16 bytes,
// several) vector accesses; p aligned to min(16, V * sizeof) bytes.
template <typename T, int V>
struct alignas((V * sizeof(typename T::store_t) < 16) ? V * sizeof(typename T::store_t) : 16) Vec {
    typename T::store_t e[V];
};

template <int BYTES>
struct Words {
    typedef uint32_t type __attribute__((ext_vector_type(BYTES / 4)));
};
template <>
struct Words<4> {
    typedef uint32_t type;
};
template <>
struct Words<2> {
    typedef uint16_t type;
};
template <>
struct Words<32> {  // two accesses, aligned to 16
    typedef uint32_t type __attribute__((ext_vector_type(8), aligned(16)));
};
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> ld_vec(const typename T::store_t* p)
{
    using W = typename Words<sizeof(Vec<T, V>)>::type;
    return __builtin_bit_cast(Vec<T, V>, *reinterpret_cast<const W*>(p));
}

template <typename T, int V>
__device__ __forceinline__ void st_vec(typename T::store_t* p, const float (&v)[V])
{
    Vec<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.e[i] = T::round(v[i]);
    *reinterpret_cast<Vec<T, V>*>(p) = o;
}

// V elements as one access, at its own alignment (AL) or the element's.
template <typename T, int V, bool AL>
__device__ __forceinline__ Vec<T, V> ld_any(const typename T::store_t* p)
{
    if constexpr (AL) {
        return ld_vec<T, V>(p);
    } else {
        typename Words<sizeof(Vec<T, V>)>::type w;
        __builtin_memcpy(&w, p, sizeof(w));
        return __builtin_bit_cast(Vec<T, V>, w);
    }
}
// A loaded vector as one value, where its elements are used: else the compiler may
// split the load by how they are.
template <typename T, int V>
__device__ __forceinline__ Vec<T, V> whole(const Vec<T, V>& v)
{
    auto w = __builtin_bit_cast(typename Words<sizeof(Vec<T, V>)>::type, v);
    asm("" : "+v"(w));
    return __builtin_bit_cast(Vec<T, V>, w);
}
template <typename T, int V, bool AL>
__device__ __forceinline__ void st_any(typename T::store_t* p, const float (&v)[V])
{
    Vec<T, V> o;
#pragma unroll
    for (int i = 0; i < V; ++i) o.e[i] = T::round(v[i]);
    if constexpr (AL)
        *reinterpret_cast<Vec<T, V>*>(p) = o;
    else
        __builtin_memcpy(p, &o, sizeof(o));
}

// The column of a lane's vector: where rows are not whole vectors (they are at
// least one) the last one is moved back over the one before it.
template <int V, bool AL>
__device__ __forceinline__ int64_t vec_col(int64_t col, int64_t width)
{
    return AL || col + V <= width ? col : width - V;
}

// --------------------------------------------------------------- scalar functions
constexpr float kLog2e = 0x1.715476p+0f;     // log2(e) to 24 bits
constexpr float kLog2eLo = 0x1.4ae0bep-26f;  // and the rest
constexpr float kLn2 = 0x1.62e43p-1f;

__device__ __forceinline__ float fma32(float a, float b, float c) { return __builtin_fmaf(a, b, c); }
__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }
// 1 / x to 1 ulp
__device__ __forceinline__ float rcp_hw(float x) { return __builtin_amdgcn_rcpf(x); }

// Limits are taken by clamps (one instruction), not by comparison and selection
// (two).
constexpr float kMaxF = 0x1.fffffep+127f;
__device__ __forceinline__ float clamp_f(float x, float lo, float hi)
{
    return __builtin_amdgcn_fmed3f(x, lo, hi);  // lo for a NaN
}

// exp(x).  float32 activations: to about 2 ulp, with the product x log2(e) in
// two parts, the lower one, below 2^-16, through exp2(r) = 1 + r ln 2.  16-bit
// activations: the high part alone, whose relative error, |x| 2^-24 and the
// exponential's ulp, is far below theirs.
template <typename T>
__device__ __forceinline__ float exp_f(float x)
{
    const float e = exp2_hw(x * kLog2e);  // 0, infinity or NaN included
    if (sizeof(typename T::store_t) == 2) return e;
    const float c = clamp_f(x, -200.f, 200.f);
    const float r = fma32(c, kLog2eLo, fma32(c, kLog2e, -(c * kLog2e)));
    return e * fma32(r, kLn2, 1.f);
}

// 1 / (1 + exp(-x)): 0 and 1 in the limits
template <typename T>
__device__ __forceinline__ float sigmoid_f(float x)
{
    return rcp_hw(1.f + exp_f<T>(-x));
}

// softplus(x) = max(x, 0) + log(1 + e), e = exp(-|x|) <= 1, with the logarithm
// as 2 artanh(s) = s P(s^2), s = e / (2 + e) <= 1/3.  P is the polynomial of
// degree 4 whose largest relative error on [0, 1/9] is smallest (found by exchange
// on 2 artanh(sqrt v) / sqrt v; 0.13 2^-24 with the coefficients rounded to 32 bits).  No cancellation at any x,
// so small step sizes keep their relative precision.
template <typename T>
__device__ __forceinline__ float softplus_f(float x)
{
    const float e = exp_f<T>(-__builtin_fabsf(x));
    const float s = e * rcp_hw(2.f + e);
    const float v = s * s;
    float p = fma32(v, 0x1.208bdp-2f, 0x1.1e510ap-2f);
    p = fma32(p, v, 0x1.99dae6p-2f);
    p = fma32(p, v, 0x1.5554e0p-1f);
    p = fma32(p, v, 2.f);
    return fma32(s, p, clamp_f(x, 0.f, __builtin_inff()));  // a NaN is one in s
}

// x sigmoid(x) given q = sigmoid(x): 0, not a NaN, at minus infinity
__device__ __forceinline__ float silu_f(float x, float q)
{
    return clamp_f(x, -kMaxF, __builtin_inff()) * q;
}

// d/dx of x sigmoid(x), given q = sigmoid(x): q + x q (1 - q), with its limits
// 0 and 1 where x is infinite
__device__ __forceinline__ float silu_slope(float x, float q)
{
    return fma32(clamp_f(x, -kMaxF, kMaxF), q - q * q, q);
}

// Keeps the compiler from putting off the computation of x: a sum that is only
// read after a loop or a branch would be added up there, its terms all kept in
// registers until then.
__device__ __forceinline__ void pin(float& x) { asm volatile("" : "+v"(x)); }

// ------------------------------------------------------------------- lane moves
template <int CTRL>
__device__ __forceinline__ float dpp(float v)
{
    return __uint_as_float((uint32_t)__builtin_amdgcn_update_dpp(
        0, (int)__float_as_uint(v), CTRL, 0xf, 0xf, true));
}

// lane T of each row of 16 lanes, to the whole row
template <int T>
__device__ __forceinline__ float row_bcast(float v)
{
    return dpp<0x150 + T>(v);
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// lower half wave: x summed over lane and lane + 32; upper half: y likewise
__device__ __forceinline__ float fold_halves(float x, float y)
{
    const u32x2 r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(y), false,
                                                     false);
    return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// even rows of 16 lanes: x summed over the row and the next; odd rows: y
// likewise over the row and the one before
__device__ __forceinline__ float fold_rows(float x, float y)
{
    const u32x2 r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(y), false,
                                                     false);
    return __uint_as_float(r.x) + __uint_as_float(r.y);
}

// Rows of a wave's lanes hold partial sums of four values; row q gets the
// total of value q.
__device__ __forceinline__ float fold_quad(float v0, float v1, float v2, float v3)
{
    return fold_rows(fold_halves(v0, v2), fold_halves(v1, v3));
}

// Orders a wave's shared-memory writes before its later reads of them by
// other lanes (the hardware keeps a wave's LDS accesses in order; this keeps
// the compiler from moving them).
__device__ __forceinline__ void wave_lds_fence()
{
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// ------------------------------------------------------------------- sequences
struct Seqs {
    int64_t seqs, rows;
    const int32_t* starts;
};

// Rows [first, first + len) of a sequence (first: 0 unless packed).
struct Span {
    int64_t first;
    int32_t len;
};

__device__ __forceinline__ int32_t clamp_start(const Seqs& q, int64_t s)
{
    const int32_t v = q.starts[s];
    return v < 0 ? 0 : (v > (int32_t)q.rows ? (int32_t)q.rows : v);
}

__device__ __forceinline__ Span seq_span(const Seqs& q, int64_t s)
{
    if (q.starts == nullptr) return Span{0, (int32_t)q.rows};
    const int32_t a = clamp_start(q, s), b = clamp_start(q, s + 1);
    return Span{a, b > a ? b - a : 0};
}

// Chunks of CH rows from each sequence's start have slots of their own,
// numbered without a prefix sum: chunk c of sequence s has slot base(s) + c,
// with base(s) = s max(1, ceil(rows / CH)), or, packed, s + floor(starts[s] /
// CH) (a sequence of n rows from row a takes ceil(n / CH) <= floor((a + n) /
// CH) - floor(a / CH) + 1 slots).  Every sequence has a slot; some slots stay
// empty.
template <int CH>
__host__ __device__ __forceinline__ int64_t chunks_per_seq(int64_t rows)
{
    return rows > CH ? (rows + CH - 1) / CH : 1;
}

template <int CH>
__host__ __device__ __forceinline__ int64_t slot_count(int64_t seqs, int64_t rows, bool packed)
{
    if (seqs == 0) return 0;  // rows of no sequence
    return packed ? seqs + rows / CH : seqs * chunks_per_seq<CH>(rows);
}

template <int CH>
__device__ __forceinline__ int64_t slot_base(const Seqs& q, int64_t s)
{
    if (q.starts == nullptr) return s * chunks_per_seq<CH>(q.rows);
    return s + clamp_start(q, s) / CH;
}

// The chunk of a slot: its sequence, rows [row, row + len) of it (row counted
// from the sequence's start) and the sequence's span; len <= 0 for an empty
// slot.
struct Chunk {
    int64_t s;
    Span span;
    int32_t row;
    int32_t len;
};

// Chunk `slot - base` of sequence s, packed.
template <int CH>
__device__ __forceinline__ Chunk packed_chunk(const Seqs& q, int64_t s, int64_t slot)
{
    Chunk c;
    c.s = s;
    c.span = seq_span(q, s);
    const int64_t k = slot - s - c.span.first / CH;
    c.row = k < 0 || k > (int64_t)(0x7fffffff / CH) ? 0x7fffffff / CH * CH : (int32_t)k * CH;
    const int32_t left = c.span.len - c.row;
    c.len = left < CH ? left : CH;
    return c;
}

template <int CH>
__device__ __forceinline__ Chunk even_chunk(const Seqs& q, int64_t slot)
{
    Chunk c;
    const int64_t per = chunks_per_seq<CH>(q.rows);
    c.s = slot / per;
    c.span = Span{0, (int32_t)q.rows};
    c.row = (int32_t)((slot - c.s * per) * CH);
    const int32_t left = c.span.len - c.row;
    c.len = left < CH ? left : CH;
    return c;
}

template <int CH>
__device__ __forceinline__ Chunk slot_chunk(const Seqs& q, int64_t slot)
{
    if (q.starts == nullptr) return even_chunk<CH>(q, slot);
    int64_t lo = 0, hi = q.seqs - 1;  // the last sequence with base <= slot
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (slot_base<CH>(q, mid) <= slot)
            lo = mid;
        else
            hi = mid - 1;
    }
    return packed_chunk<CH>(q, lo, slot);
}

// The value of a wave's first lane, in scalar registers: for values that are
// the same in every lane but were read or computed lane by lane.
__device__ __forceinline__ int32_t uniform(int32_t v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ int64_t uniform(int64_t v)
{
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int32_t)(uint32_t)v);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int32_t)(v >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ Span uniform(Span s) { return Span{uniform(s.first), uniform(s.len)}; }
__device__ __forceinline__ Chunk uniform(Chunk c)
{
    return Chunk{uniform(c.s), uniform(c.span), uniform(c.row), uniform(c.len)};
}

// slot_chunk for a slot that is the same in all lanes of a wave: 64 sequences are
// looked at at a time, so that up to 64 take one load instead of one after the
// other.
template <int CH>
__device__ __forceinline__ Chunk wave_slot_chunk(const Seqs& q, int64_t slot)
{
    if (q.starts == nullptr) return even_chunk<CH>(q, slot);
    const int lane = threadIdx.x & 63;
    int64_t lo = 0, n = q.seqs;  // it is one of the n sequences from lo on
    while (n > 1) {
        const int64_t step = (n + 63) / 64, at = lane * step;
        const uint64_t hit = __ballot(at < n && slot_base<CH>(q, lo + (at < n ? at : 0)) <= slot);
        const int64_t k = hit ? (63 - __builtin_clzll(hit)) * step : 0;
        lo += k;
        n = n - k < step ? n - k : step;
    }
    return uniform(packed_chunk<CH>(q, lo, slot));
}

template <typename T>
__device__ __forceinline__ typename T::store_t* rows_ptr(const canon_rows_t& r, int64_t s,
                                                         const Seqs& q, int64_t first)
{
    return static_cast<typename T::store_t*>(r.p) + (q.starts ? 0 : s * r.seq) + first * r.row;
}

}  // namespace seq
}  // namespace canon
