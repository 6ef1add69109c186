// The gated linear recurrence h[t] = a h[t-1] + c i x[t], elementwise over the
// channels: forward, backward and single rows.
//
// A lane holds V channels; a wave walks a chunk of 8 rows, whose inputs it loads at
// once.  The 16 waves of a workgroup take the chunks of a round (128 rows), fold each
// from zero, exchange the folds through LDS, and fold again from their chunks' start
// states, with e = a - 1 and v = c i x still in registers: one pass over memory.  Rounds
// of a block (512 rows) follow each other in the workgroup; forward, a row of the next
// round is loaded where one of this round has been used.
//
// Memory bounds it, and vector issue nearly as much: 38 instructions a value forward (69%
// of the time), 86 backward (81%).  8 x 2048 x 4096 bf16, both gates: forward 113 us (4.8
// TB/s), backward 227 (4.1).  8 waves of 16 rows, at 256 registers a lane, took 131 and
// 255 where these then took 122 and 243; rows of the next round in flight in the backward
// pass too cost spilled registers at 16 waves (338), and gained nothing at 8 (260).
//
// a is near 1 for a long memory, so it is kept as its difference from 1: with e = a - 1,
//   h <- (h + e h) + v,   and for the product of a, Q = P - 1:  Q <- Q + (e Q + e),
// h + e h with one rounding.  An a of 0 (e and Q of -1, which the folds keep exactly) so
// leaves nothing of any finite h, as h + (e h + v), whose rounding is that of e h, would.
// The start states of rounds and chunks are folded in 64 bits inside a block and rounded to
// 32 between blocks: an h that loses less than its last bit in a chunk would stay as it is
// otherwise.  (Chunks of a round folded on in 32 bits take 2 us less of the backward pass.)
#pragma once

#include <type_traits>

#include "column_sum.hpp"
#include "launch.hpp"
#include "recurrence.hpp"

namespace canon {
namespace seq {

constexpr int kCh = CANON_RECUR_CHUNK;

__device__ __forceinline__ double fma64(double a, double b, double c) { return __builtin_fma(a, b, c); }

// exp(l) - 1 for l <= 0: down to -1 by l + l^2 q(l), where q interpolates
// (exp(l) - 1 - l) / l^2 at the Chebyshev nodes of [-1, 0] (off by 2^-25 of the result);
// below it the exponential less 1, which loses less than a bit there.
template <typename T, bool NEAR>
__device__ __forceinline__ float expm1_f(float l)
{
    float p = fma32(l, 0x1.20330cp-13f, 0x1.5b4b08p-10f);
    p = fma32(p, l, 0x1.100344p-7f);
    p = fma32(p, l, 0x1.5545cap-5f);
    p = fma32(p, l, 0x1.5555p-3f);
    p = fma32(p, l, 0.5f);
    const float near = fma32(l * l, p, l);
    if (NEAR) return near;
    return l >= -1.f ? near : exp_f<T>(l) - 1.f;
}

// The decays of a lane's channels, and whether no lane of the wave has one above 1:
// then the logarithm of a, between -decay and 0, needs the polynomial alone.
template <int V>
struct Decay {
    float d[V];
    bool near;
};
template <bool DECAY, int V>
__device__ __forceinline__ Decay<V> load_decay(const float* decay, int32_t ch)
{
    Decay<V> d{{}, DECAY};
    if (DECAY) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            d.d[k] = decay[ch + k];
            d.near = d.near && __ballot(d.d[k] <= 1.f) == ~0ull;
        }
    }
    return d;
}

// e = a - 1
template <typename T, bool DECAY, bool NEAR>
__device__ __forceinline__ float gate_e(float gate, float decay)
{
    if (!DECAY) return -sigmoid_f<T>(-gate);
    return expm1_f<T, NEAR>(-decay * sigmoid_f<T>(gate));
}
// sqrt(1 - a^2) = sqrt((1 - a)(1 + a)), or 1 - a
template <bool DECAY>
__device__ __forceinline__ float factor(float e)
{
    return DECAY ? __builtin_amdgcn_sqrtf(-e * (2.f + e)) : -e;
}

// A wave's channels and place in its workgroup.
struct Lane {
    int lane, wave;
    int32_t c, ch;  // the lane's first channel, and one from which V may be read
    bool on;        // c is a channel
};
template <int V>
__device__ __forceinline__ Lane recur_lane(const RecurArgs& a, int32_t slab)
{
    Lane l;
    l.lane = threadIdx.x & 63;
    l.wave = uniform((int32_t)(threadIdx.x >> 6));
    l.c = (slab * 64 + l.lane) * V;
    l.on = l.c < a.channels;
    l.ch = l.on ? l.c : a.channels - V;
    return l;
}

// A float of each of the lane's channels.
template <int V>
__device__ __forceinline__ void ld_channels(const float* p, float (&v)[V])
{
#pragma unroll
    for (int k = 0; k < V; ++k) v[k] = p[k];
}
template <int V>
__device__ __forceinline__ void st_channels(float* p, const float (&v)[V])
{
#pragma unroll
    for (int k = 0; k < V; ++k) p[k] = v[k];
}

// The rows of a chunk in the lane's channels, a register each (V is 1, or 2 of 16 bits).
// Byte offsets within a chunk are 32-bit: fewer than 8 rows of a pitch below 2^24
// elements, and a channel below 2^24 (the host checks both).
template <typename T, int V>
struct ChunkRows {
    using E = typename T::store_t;
    static constexpr int kBytes = V * sizeof(E);
    uint32_t v[kCh];  // bits

    // from the rows at b, of which n are valid, at least one; the others are a copy of
    // the last
    __device__ __forceinline__ void load_row(__amdgpu_buffer_rsrc_t b, const canon_rows_t& a,
                                             const Lane& l, int r, int n)
    {
        v[r] = bits(b, (uint32_t)l.ch * (uint32_t)sizeof(E),
                    (r < n ? r : n - 1) * ((uint32_t)a.row * (uint32_t)sizeof(E)));
    }
    __device__ __forceinline__ void load(const canon_rows_t& a, const Seqs& q, int64_t s, int64_t row,
                                         const Lane& l, int n)
    {
        const __amdgpu_buffer_rsrc_t b = tile_rsrc(rows_ptr<T>(a, s, q, row));
#pragma unroll
        for (int r = 0; r < kCh; ++r) load_row(b, a, l, r, n);
    }
    static __device__ __forceinline__ uint32_t bits(__amdgpu_buffer_rsrc_t b, uint32_t off,
                                                    uint32_t row)
    {
        if constexpr (kBytes == 2)
            return __builtin_amdgcn_raw_buffer_load_b16(b, off, row, 0);
        else
            return __builtin_amdgcn_raw_buffer_load_b32(b, off, row, 0);
    }
    __device__ __forceinline__ float get(int r, int k) const
    {
        if constexpr (sizeof(E) == 4)
            return __uint_as_float(v[r]);
        else
            return T::load((uint16_t)(v[r] >> 16 * k));
    }
    __device__ __forceinline__ void set(int r, float x)
    {
        v[r] = __float_as_uint(x);
        if constexpr (sizeof(E) == 2) v[r] = T::round(x) * 0x10001u;
    }
    // The same values, as if loaded again: what was computed from them before is
    // computed anew instead of waiting in registers.
    __device__ __forceinline__ void afresh()
    {
#pragma unroll
        for (int r = 0; r < kCh; ++r) asm("" : "+v"(v[r]));
    }
};

// Two values rounded to 16 bits, the first in the lower half.
__device__ __forceinline__ uint32_t round_two(BF16, float a, float b)
{
    typedef float f32x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}
__device__ __forceinline__ uint32_t round_two(F16, float a, float b)
{
    return (uint32_t)F16::round(a) | (uint32_t)F16::round(b) << 16;
}

// The n rows of a chunk of an output.  Every lane stores every row, with an offset out
// of the buffer's range, which drops it, where there is no such row or channel: without
// branches the loads in flight are waited for by their number.  Stores go past the caches,
// which rows that are read again have a use for (4 x 2048 x 4096 bf16 backward 138 -> 119
// us, 8 x 2048 x 4096 127 + 247 -> 122 + 243; small calls, and a call together with the
// next one that reads its outputs, take the same within 3%).
template <typename T, int V>
struct ChunkOut {
    using E = typename T::store_t;
    static constexpr uint32_t kDropped = 0x80000000u;
    __amdgpu_buffer_rsrc_t b;
    uint32_t pitch, off;
    int n;
    __device__ __forceinline__ ChunkOut(const canon_rows_t& a, const Seqs& q, int64_t s, int64_t row,
                                        const Lane& l, int rows)
        : b(__builtin_amdgcn_make_buffer_rsrc(rows_ptr<T>(a, s, q, row), 0, 0x7fffffff, 0x00020000)),
          pitch((uint32_t)a.row * (uint32_t)sizeof(E)),
          off(l.on ? (uint32_t)l.c * (uint32_t)sizeof(E) : kDropped),
          n(rows)
    {
    }
    __device__ __forceinline__ void store(int r, const float (&y)[V]) const
    {
        const uint32_t to = r < n ? off : kDropped;
        constexpr int PAST = 2;
        if constexpr (V == 2)
            __builtin_amdgcn_raw_buffer_store_b32(round_two(T{}, y[0], y[1]), b, to, r * pitch, PAST);
        else if constexpr (sizeof(E) == 4)
            __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(y[0]), b, to, r * pitch, PAST);
        else
            __builtin_amdgcn_raw_buffer_store_b16(T::round(y[0]), b, to, r * pitch, PAST);
    }
};

// What a chunk reads, and where its rows are.
template <typename T, int V>
struct ChunkIn {
    ChunkRows<T, V> g, x, in;
    __device__ __forceinline__ void load(const RecurArgs& a, const Lane& l, int64_t s, int64_t row,
                                         int n)
    {
        const From from(a, s, row);
#pragma unroll
        for (int r = 0; r < kCh; ++r) load_row(a, l, from, r, n);
    }
    struct From {
        __amdgpu_buffer_rsrc_t g, x, in;
        __device__ __forceinline__ From(const RecurArgs& a, int64_t s, int64_t row)
            : g(tile_rsrc(rows_ptr<T>(a.gate, s, a.q, row))),
              x(tile_rsrc(rows_ptr<T>(a.x, s, a.q, row))),
              in(tile_rsrc(rows_ptr<T>(a.input, s, a.q, row)))
        {
        }
    };
    __device__ __forceinline__ void load_row(const RecurArgs& a, const Lane& l, const From& f, int r,
                                             int n)
    {
        g.load_row(f.g, a.gate, l, r, n);
        x.load_row(f.x, a.x, l, r, n);
        if (a.input.p) in.load_row(f.in, a.input, l, r, n);
    }
};

// e and v of a chunk's n rows; those beyond leave the state as it is.  after(r) follows
// the last use of row r.
template <typename T, int V, bool DECAY, bool NEAR, bool INPUT, class F>
__device__ __forceinline__ void chunk_values(ChunkIn<T, V>& c, int n, const Decay<V>& d,
                                             float (&e)[kCh][V], float (&v)[kCh][V], F&& after)
{
#pragma unroll
    for (int r = 0; r < kCh; ++r) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            e[r][k] = gate_e<T, DECAY, NEAR>(c.g.get(r, k), d.d[k]);
            v[r][k] = factor<DECAY>(e[r][k]) * c.x.get(r, k);
            if (INPUT) v[r][k] *= sigmoid_f<T>(c.in.get(r, k));
        }
        after(r);
    }
    if (n < kCh) {
#pragma unroll
        for (int r = 0; r < kCh; ++r)
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (r >= n) e[r][k] = v[r][k] = 0.f;
    }
}
template <typename T, int V, bool DECAY, class F>
__device__ __forceinline__ void chunk_values(const RecurArgs& a, ChunkIn<T, V>& c, int n,
                                             const Decay<V>& d, float (&e)[kCh][V],
                                             float (&v)[kCh][V], F&& after)
{
    if (DECAY && d.near) {
        if (a.input.p)
            chunk_values<T, V, DECAY, true, true>(c, n, d, e, v, after);
        else
            chunk_values<T, V, DECAY, true, false>(c, n, d, e, v, after);
    } else {
        if (a.input.p)
            chunk_values<T, V, DECAY, false, true>(c, n, d, e, v, after);
        else
            chunk_values<T, V, DECAY, false, false>(c, n, d, e, v, after);
    }
}

// A value at the start of the next block, given the block's Q and S.
__device__ __forceinline__ float carry(float h, float q, float s)
{
    return (float)(fma64(q, h, h) + s);
}

// A value further on in a block that starts with h, given the Q and S between; past
// the block's end it is rounded to 32 bits.
__device__ __forceinline__ double carried(float h, double q, double s, bool end)
{
    return end ? (double)carry(h, (float)q, (float)s) : fma64(q, h, h) + s;
}

// The state that a block starts with, given those of the first one in ws_h: where
// sequences have few blocks, from the folds of the n before it, which are step slots apart
// (else k_recur_carry has folded them, into its own ws_h).  The reads grow with the square;
// kRecurFold has both ways' times.
template <int V>
__device__ __forceinline__ void block_start(const RecurArgs& a, const Lane& l, int64_t slot, int32_t n,
                                            int32_t step, float (&h)[V])
{
    if (a.carry) n = 0;
    ld_channels<V>(a.ws_h + (slot + (int64_t)n * step) * a.channels + l.ch, h);
    constexpr int U = 8;
    for (int32_t left = n; left > 0; left -= U) {
        float q[U][V], s[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t i = (slot + (int64_t)(left - u > 1 ? left - u : 1) * step) * a.channels + l.ch;
            ld_channels<V>(a.ws_q + i, q[u]);
            ld_channels<V>(a.ws_s + i, s[u]);
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int j = 0; j < V; ++j)
                if (u < left) h[j] = carry(h[j], q[u][j], s[u][j]);
    }
}

// Rows of a wave in the round that starts at `from`, of those before `end`.
__device__ __forceinline__ int chunk_rows(const Lane& l, int32_t from, int32_t end)
{
    const int32_t left = end - from - l.wave * kCh;
    return left < kCh ? left : kCh;
}

enum { kRecurSum, kRecurOut, kRecurWhole, kRecurSpreadOut };

// The block and round of a workgroup, where each round has one; false if there are no
// such rows.
struct Round {
    Chunk k;
    int32_t rd, rounds;  // of the block
    bool some;
};
__device__ __forceinline__ Round round_of(const RecurArgs& a, int32_t job)
{
    Round r;
    r.k = wave_slot_chunk<CANON_RECUR_BLOCK>(a.q, job / kRecurRounds);
    r.rd = job % kRecurRounds;
    if (r.k.len < 0) r.k.len = 0;
    r.rounds = (r.k.len + kRecurRound - 1) / kRecurRound;
    r.some = r.rd < r.rounds;
    return r;
}

// Q and S of a wave's chunks of a slot, n of them from c on (step 1), or up to c (step
// -1), from their folds in ws_cq and ws_cs.
__device__ __forceinline__ void fold_chunks(const RecurArgs& a, const Lane& l, int64_t slot, int c,
                                            int n, int step, double& Q, double& S)
{
    constexpr int U = 16;  // of a round
    Q = S = 0.;
    for (; n > 0; n -= U) {
        float q[U], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u, c += step) {
            const int64_t i = (slot * kRecurBlockChunks + c) * a.channels + l.ch;
            q[u] = a.ws_cq[i];
            s[u] = a.ws_cs[i];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            S = fma64(q[u], S, S) + s[u];
            Q += fma64(q[u], Q, q[u]);
        }
    }
}

// The folds of the chunks of each round, for k_recurrence and k_recurrence_grad with a
// workgroup for each round; those that serve no other are left out.  999 x 520 float32: 4.7
// us forward and 4.4 backward, before 6.5 and 9.8 of outputs; a workgroup for each block
// took 11 + 13 and 4 + 21.
template <typename T, bool DECAY, bool BACK>
__global__ __launch_bounds__(64 * kRecurWaves) void k_recur_chunks(RecurArgs a)
{
    const int32_t job = uniform((int32_t)(blockIdx.x / (uint32_t)a.slabs));
    const Lane l = recur_lane<1>(a, blockIdx.x - job * a.slabs);
    const Round r = round_of(a, job);
    if (!r.some) return;
    const Chunk& k = r.k;
    const int64_t slot = job / kRecurRounds;
    const int32_t from = k.row + r.rd * kRecurRound, end = k.row + k.len;
    const bool first = from == 0, last = from + kRecurRound >= k.span.len;
    // the last workgroup of a sequence may overwrite init with final while others begin
    if (!BACK && first && l.wave == 0 && l.on)
        a.ws_h[slot * a.channels + l.c] = a.init ? a.init[k.s * a.channels + l.c] : 0.f;
    if (BACK ? first : last) return;
    const int n = chunk_rows(l, from, end);
    const int64_t row = k.span.first + from + l.wave * kCh;
    const Decay<1> decay = load_decay<DECAY, 1>(a.decay, l.ch);
    float q = 0.f, s = 0.f;
    if (n > 0 && !BACK) {
        ChunkIn<T, 1> in;
        float e[kCh][1], v[kCh][1];
        in.load(a, l, k.s, row, n);
        chunk_values<T, 1, DECAY>(a, in, n, decay, e, v, [](int) {});
#pragma unroll
        for (int i = 0; i < kCh; ++i) {
            s = fma32(e[i][0], s, s) + v[i][0];
            q += fma32(e[i][0], q, e[i][0]);
        }
    }
    if (n > 0 && BACK) {
        ChunkRows<T, 1> g, d;
        g.load(a.gate, a.q, k.s, row, l, n);
        d.load(a.dout, a.q, k.s, row, l, n);
#pragma unroll
        for (int i = kCh - 1; i >= 0; --i) {
            if (i >= n) continue;
            const float e = gate_e<T, DECAY, false>(g.get(i, 0), decay.d[0]);
            const float lam = d.get(i, 0) + s;
            s = fma32(e, lam, lam);
            q += fma32(e, q, e);
        }
    }
    if (!l.on) return;
    const int64_t i = (slot * kRecurBlockChunks + r.rd * kRecurWaves + l.wave) * a.channels + l.c;
    a.ws_cq[i] = q;
    a.ws_cs[i] = s;
}

// kRecurSum: Q and S of each block.  kRecurOut: the outputs of each block, from its
// start state.  kRecurWhole: the outputs of whole sequences, block after block.
// Wave 0 carries the state from round to round.  kRecurSpreadOut: the outputs of each
// round, to whose start the waves fold what is before, a block each.
template <typename T, int V, bool DECAY, int MODE>
__global__ __launch_bounds__(64 * kRecurWaves) void k_recurrence(RecurArgs a)
{
    constexpr int W = 64 * V;
    __shared__ float lq[2][kRecurWaves][W], ls[2][kRecurWaves][W];
    __shared__ double lh[2][W], lc[MODE == kRecurSpreadOut ? kRecurWaves : 1][2][W];
    const int32_t job = uniform((int32_t)(blockIdx.x / (uint32_t)a.slabs));
    const Lane l = recur_lane<V>(a, blockIdx.x - job * a.slabs);
    const int at_lds = l.lane * V;
    Chunk k;
    int32_t rd = 0;
    int64_t slot = job;
    if (MODE == kRecurWhole) {
        k = Chunk{job, Span{0, (int32_t)a.q.rows}, 0, (int32_t)a.q.rows};
        if (k.len > CANON_RECUR_BLOCK) k.len = CANON_RECUR_BLOCK;
        slot = job * chunks_per_seq<CANON_RECUR_BLOCK>(a.q.rows);
    } else if (MODE == kRecurSpreadOut) {
        const Round r = round_of(a, job);
        if (!r.some && (r.k.row != 0 || r.rd != 0)) return;
        k = r.k;
        rd = r.rd;
        slot = job / kRecurRounds;
    } else {
        k = wave_slot_chunk<CANON_RECUR_BLOCK>(a.q, slot);
        if (k.len <= 0 && k.row != 0) return;  // no block has this slot
        if (k.len < 0) k.len = 0;
        // the last block's fold serves no other
        if (MODE == kRecurSum && k.row + k.len >= k.span.len) return;
    }
    const int32_t end = MODE == kRecurWhole ? k.span.len : k.row + k.len;
    const int32_t start = k.row + rd * kRecurRound;
    ChunkIn<T, V> in;
    if (const int n = chunk_rows(l, start, end); n > 0)
        in.load(a, l, k.s, k.span.first + start + l.wave * kCh, n);
    const Decay<V> decay = load_decay<DECAY, V>(a.decay, l.ch);
    float h0[V] = {};
    // Where there are more blocks, the first one's fold keeps init in ws_h: the last one's
    // outputs may overwrite init with final while others begin.
    const bool cut = MODE != kRecurWhole && k.span.len > CANON_RECUR_BLOCK;
    const int32_t before = k.row / CANON_RECUR_BLOCK;
    if (MODE == kRecurSpreadOut) {
        if (k.len == 0) {
            if (a.init) ld_channels<V>(a.init + k.s * a.channels + l.ch, h0);
            if (a.final && l.wave == 0 && l.on)
                st_channels<V>(a.final + k.s * a.channels + l.c, h0);
            return;
        }
        ld_channels<V>(a.ws_h + (slot - before) * a.channels + l.ch, h0);
        if (l.wave <= before) {
            double Q, S;
            fold_chunks(a, l, slot - before + l.wave, 0,
                        l.wave < before ? kRecurBlockChunks : rd * kRecurWaves, 1, Q, S);
            lc[l.wave][0][at_lds] = Q;
            lc[l.wave][1][at_lds] = S;
        }
    } else if (MODE == kRecurOut && cut) {
        if (l.wave == 0) block_start<V>(a, l, slot, k.row / CANON_RECUR_BLOCK, -1, h0);
    } else if (a.init && (MODE != kRecurSum || k.row == 0)) {
        ld_channels<V>(a.init + k.s * a.channels + l.ch, h0);
    }
    if (MODE == kRecurSum && k.row == 0 && l.wave == 0 && l.on)
        st_channels<V>(a.ws_h + slot * a.channels + l.c, h0);
    if (MODE != kRecurSum && MODE != kRecurSpreadOut && l.wave == 0) {
#pragma unroll
        for (int j = 0; j < V; ++j) lh[0][at_lds + j] = h0[j];
    }
    int buf = 0;
    for (;;) {
        double Q[V] = {}, S[V] = {};  // in wave 0
        for (int32_t from = MODE == kRecurSpreadOut ? start : k.row; from < k.row + k.len;
             from += kRecurRound, buf ^= 1) {
            const int32_t at = from + l.wave * kCh;
            const int n = chunk_rows(l, from, end);
            float e[kCh][V], v[kCh][V];
            if (n > 0) {
                // The next round's row takes the place of the one just used; where there is
                // none the last row is read again.
                const int32_t to = at + kRecurRound < end ? at + kRecurRound : end - 1;
                const int m = end - to < kCh ? end - to : kCh;
                const typename ChunkIn<T, V>::From rows(a, k.s, k.span.first + to);
                chunk_values<T, V, DECAY>(a, in, n, decay, e, v, [&](int r) {
                    if (MODE != kRecurSpreadOut) in.load_row(a, l, rows, r, m);
                });
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float q = 0.f, s = 0.f;
#pragma unroll
                    for (int r = 0; r < kCh; ++r) {
                        s = fma32(e[r][j], s, s) + v[r][j];
                        q += fma32(e[r][j], q, e[r][j]);
                    }
                    lq[buf][l.wave][at_lds + j] = q;
                    ls[buf][l.wave][at_lds + j] = s;
                }
            }
            __syncthreads();
            if (MODE == kRecurSpreadOut) {
                for (int32_t b = 0; b < before; ++b)
                    h0[0] = carry(h0[0], (float)lc[b][0][at_lds], (float)lc[b][1][at_lds]);
                Q[0] = lc[before][0][at_lds];
                S[0] = lc[before][1][at_lds];
            }
            float y[V];
            if (MODE != kRecurSum) {
                double h[V];
#pragma unroll
                for (int j = 0; j < V; ++j)
                    h[j] = MODE != kRecurSpreadOut ? lh[buf][at_lds + j]
                           : rd                    ? carried(h0[j], Q[j], S[j], false)
                                                   : (double)h0[j];
#pragma unroll 2
                for (int c = 0; c < l.wave; ++c)
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        h[j] = fma64(lq[buf][c][at_lds + j], h[j], h[j]) + ls[buf][c][at_lds + j];
#pragma unroll
                for (int j = 0; j < V; ++j) y[j] = (float)h[j];
            }
            const bool ends = from + kRecurRound >= k.span.len;
            if (l.wave == 0 && a.kept && l.on && MODE == kRecurSpreadOut)
                st_channels<V>(a.kept + (slot * kRecurRounds + rd) * a.channels + l.c, y);
            if (l.wave == 0 && (MODE != kRecurSpreadOut || ends)) {
                if (MODE != kRecurSum && MODE != kRecurSpreadOut && a.kept && l.on)
                    st_channels<V>(a.kept + (slot * kRecurRounds + (from - k.row) / kRecurRound) *
                                                a.channels + l.c, y);
                const int32_t rows = k.row + k.len - from;
                const int chunks = rows < kRecurRound ? (rows + kCh - 1) / kCh : kRecurWaves;
#pragma unroll 2
                for (int c = 0; c < chunks; ++c)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const double q = lq[buf][c][at_lds + j], s = ls[buf][c][at_lds + j];
                        S[j] = fma64(q, S[j], S[j]) + s;
                        Q[j] += fma64(q, Q[j], q);
                    }
                const bool done = from + kRecurRound >= k.row + k.len;  // the block's end
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    if (MODE == kRecurSum) continue;
                    const double hn = carried(h0[j], Q[j], S[j], done);
                    if (done) h0[j] = (float)hn;
                    if (MODE != kRecurSpreadOut) lh[buf ^ 1][at_lds + j] = hn;
                }
            }
            if (MODE != kRecurSum && n > 0) {
                const ChunkOut<T, V> out(a.out, a.q, k.s, k.span.first + at, l, n);
#pragma unroll
                for (int r = 0; r < kCh; ++r) {
#pragma unroll
                    for (int j = 0; j < V; ++j) y[j] = fma32(e[r][j], y[j], y[j]) + v[r][j];
                    out.store(r, y);
                }
            }
            if (MODE == kRecurSpreadOut) {
                if (ends && l.wave == 0 && l.on && a.final)
                    st_channels<V>(a.final + k.s * a.channels + l.c, h0);
                return;
            }
        }
        const bool last = k.row + k.len >= k.span.len;
        if (l.wave == 0 && l.on) {
            if (MODE == kRecurSum) {
                float q[V], s[V];
#pragma unroll
                for (int j = 0; j < V; ++j) q[j] = (float)Q[j], s[j] = (float)S[j];
                st_channels<V>(a.ws_q + slot * a.channels + l.c, q);
                st_channels<V>(a.ws_s + slot * a.channels + l.c, s);
            } else if (last && a.final) {
                st_channels<V>(a.final + k.s * a.channels + l.c, h0);
            }
        }
        if (MODE != kRecurWhole || last) return;
        k.row += CANON_RECUR_BLOCK;
        k.len = k.span.len - k.row < CANON_RECUR_BLOCK ? k.span.len - k.row : CANON_RECUR_BLOCK;
        ++slot;
    }
}

// The start states of each sequence's blocks from the first one's (in ws_h) and the
// blocks' Q and S (in ws_q, ws_s), into ws_h; backwards: the gradients that come in past
// their ends.  Latency: a chain of loads, eight blocks at a time (6 us for 32 blocks of
// 2048 channels).
template <bool BACK>
__global__ __launch_bounds__(64) void k_recur_carry(RecurArgs a)
{
    const uint32_t slabs = (a.channels + 63) / 64;
    const int64_t s = blockIdx.x / slabs;
    const int32_t c = (blockIdx.x - (uint32_t)s * slabs) * 64 + threadIdx.x;
    if (c >= a.channels) return;
    const Span span = seq_span(a.q, s);
    const int64_t slot = slot_base<CANON_RECUR_BLOCK>(a.q, s);
    const int32_t blocks = (span.len + CANON_RECUR_BLOCK - 1) / CANON_RECUR_BLOCK;
    if (blocks < 2) return;
    float h = a.ws_h[(slot + (BACK ? blocks - 1 : 0)) * a.channels + c];
    constexpr int U = 8;
    for (int32_t b0 = 0; b0 < blocks - 1; b0 += U) {
        float q[U], v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t b = b0 + u < blocks - 1 ? b0 + u : blocks - 2;
            const int64_t i = (slot + (BACK ? blocks - 1 - b : b)) * a.channels + c;
            q[u] = a.ws_q[i];
            v[u] = a.ws_s[i];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t b = b0 + u;
            if (b >= blocks - 1) break;
            h = carry(h, q[u], v[u]);
            a.ws_h[(slot + (BACK ? blocks - 2 - b : b + 1)) * a.channels + c] = h;
        }
    }
}

// One row of each sequence, a thread a channel: 256 x 4096 bf16 6.0 us, 2.8 TB/s.
template <typename T, bool DECAY>
__global__ __launch_bounds__(256) void k_recurrence_step(RecurArgs a)
{
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t s = i / a.channels;
    const int32_t c = (int32_t)(i - s * a.channels);
    if (s >= a.q.seqs) return;
    auto row = [&](const canon_rows_t& r) {
        return static_cast<typename T::store_t*>(r.p) + s * r.seq + c;
    };
    const float e = gate_e<T, DECAY, false>(ld<T>(row(a.gate)), DECAY ? a.decay[c] : 0.f);
    float v = factor<DECAY>(e) * ld<T>(row(a.x));
    if (a.input.p) v *= sigmoid_f<T>(ld<T>(row(a.input)));
    float h = a.init ? a.init[i] : 0.f;
    h = fma32(e, h, h) + v;
    st<T>(row(a.out), h);
    if (a.final) a.final[i] = h;
}

// Backward.  With lam[t] = dout[t] + a[t+1] lam[t+1], the gradient of h[t]:
//   dx = lam c i,   da = lam h[t-1],   d(c i x) = lam,
// where h is folded again from the states kept at every round.  The fold of lam goes
// backwards over chunks, rounds and blocks just as h's does forwards; the last wave
// carries it.
// k_recur_back_sum: Q and the fold from zero of each block.
template <typename T, int V, bool DECAY>
__global__ __launch_bounds__(64 * kRecurWaves) void k_recur_back_sum(RecurArgs a)
{
    constexpr int W = 64 * V;
    __shared__ float lq[2][kRecurWaves][W], lt[2][kRecurWaves][W];
    const int64_t slot = uniform((int32_t)(blockIdx.x / (uint32_t)a.slabs));
    const Lane l = recur_lane<V>(a, blockIdx.x - (int32_t)slot * a.slabs);
    const int at_lds = l.lane * V;
    const Decay<V> decay = load_decay<DECAY, V>(a.decay, l.ch);
    const Chunk k = wave_slot_chunk<CANON_RECUR_BLOCK>(a.q, slot);
    if (k.len <= 0 || k.row == 0) return;  // the first block's fold serves no other
    if (k.row + k.len >= k.span.len && l.wave == 0 && l.on) {
        float g0[V] = {};
        if (a.dfinal) ld_channels<V>(a.dfinal + k.s * a.channels + l.c, g0);
        st_channels<V>(a.ws_h + slot * a.channels + l.c, g0);
    }
    double Q[V] = {}, G[V] = {};
    int buf = 0;
    for (int rd = (k.len - 1) / kRecurRound; rd >= 0; --rd, buf ^= 1) {
        const int32_t from = k.row + rd * kRecurRound, at = from + l.wave * kCh;
        const int n = chunk_rows(l, from, k.row + k.len);
        float q[V] = {}, t[V] = {};
        if (n > 0) {
            ChunkRows<T, V> g, d;
            g.load(a.gate, a.q, k.s, k.span.first + at, l, n);
            d.load(a.dout, a.q, k.s, k.span.first + at, l, n);
#pragma unroll
            for (int r = kCh - 1; r >= 0; --r)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float e = r < n ? gate_e<T, DECAY, false>(g.get(r, j), decay.d[j]) : 0.f;
                    const float lam = r < n ? d.get(r, j) + t[j] : t[j];
                    t[j] = fma32(e, lam, lam);
                    q[j] += fma32(e, q[j], e);
                }
        }
        st_channels<V>(&lq[buf][l.wave][at_lds], q);
        st_channels<V>(&lt[buf][l.wave][at_lds], t);
        __syncthreads();
        if (l.wave == 0)
            for (int c = kRecurWaves - 1; c >= 0; --c)
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const double cq = lq[buf][c][at_lds + j], ct = lt[buf][c][at_lds + j];
                    G[j] = fma64(cq, G[j], G[j]) + ct;
                    Q[j] += fma64(cq, Q[j], cq);
                }
    }
    if (l.wave == 0 && l.on) {
        float q[V], g[V];
#pragma unroll
        for (int j = 0; j < V; ++j) q[j] = (float)Q[j], g[j] = (float)G[j];
        st_channels<V>(a.ws_q + slot * a.channels + l.c, q);
        st_channels<V>(a.ws_s + slot * a.channels + l.c, g);
    }
}

// sigmoid(y) and 1 - sigmoid(y), the latter without cancellation.
struct Sigmoid {
    float s, rest;
};
template <typename T>
__device__ __forceinline__ Sigmoid sigmoid_both(float y)
{
    const float e = exp_f<T>(-y), s = rcp_hw(1.f + e);
    return Sigmoid{s, clamp_f(e, 0.f, kMaxF) * s};
}

// The gradients, block by block (MODE kRecurOut) or of whole sequences (kRecurWhole).
// A row keeps e and v = c i x in registers, and h[t-1] in LDS;
//   d log a = lam (a h[t-1] - a^2 v / c^2),   c^2 = -e (2 + e),   and without decay
//   d gate  = lam a (c h[t-1] - v).
template <typename T, int V, bool DECAY, int MODE>
__global__ __launch_bounds__(64 * kRecurWaves) void k_recurrence_grad(RecurArgs a)
{
    constexpr int W = 64 * V;
    __shared__ float lq[2][kRecurWaves][W], ls[2][kRecurWaves][W], lt[2][kRecurWaves][W],
        ldd[kRecurWaves][W], before[kRecurWaves][kCh][W];
    __shared__ double lg[2][W], lc[MODE == kRecurSpreadOut ? kRecurWaves : 1][2][W];
    const int32_t job = uniform((int32_t)(blockIdx.x / (uint32_t)a.slabs));
    const Lane l = recur_lane<V>(a, blockIdx.x - job * a.slabs);
    const int at_lds = l.lane * V;
    const bool carrier = l.wave == kRecurWaves - 1;
    Chunk k;
    int64_t slot = job;
    int32_t mine = 0;  // the round, where each has a workgroup
    if (MODE == kRecurSpreadOut) {
        const Round r = round_of(a, job);
        k = r.k;
        slot = job / kRecurRounds;
        mine = r.rd;
        if (!r.some) {
            if (!l.on || l.wave != 0) return;
            if (DECAY) a.ws_dd[(int64_t)job * a.channels + l.c] = 0.f;
            if (k.row == 0 && mine == 0 && a.dinit)  // an empty sequence
                a.dinit[k.s * a.channels + l.c] =
                    a.dfinal ? a.dfinal[k.s * a.channels + l.c] : 0.f;
            return;
        }
    } else if (MODE == kRecurWhole) {
        const int32_t rows = (int32_t)a.q.rows;
        const int32_t blocks = (int32_t)chunks_per_seq<CANON_RECUR_BLOCK>(rows);
        const int32_t row = (blocks - 1) * CANON_RECUR_BLOCK;
        k = Chunk{job, Span{0, rows}, row, rows - row};
        slot = job * blocks + blocks - 1;
    } else {
        k = wave_slot_chunk<CANON_RECUR_BLOCK>(a.q, slot);
        if (k.len < 0) k.len = 0;
        if (k.len == 0 && k.row != 0) {  // no block has this slot
            const float zero[V] = {};
            if (DECAY && l.wave == 0 && l.on)
                st_channels<V>(a.ws_dd + slot * a.channels + l.c, zero);
            return;
        }
    }
    const int32_t end = k.row + k.len;
    const Decay<V> decay = load_decay<DECAY, V>(a.decay, l.ch);
    float g0[V] = {};
    const int32_t rounds = (k.len + kRecurRound - 1) / kRecurRound;
    const int32_t behind = (k.span.len - 1) / CANON_RECUR_BLOCK - k.row / CANON_RECUR_BLOCK;
    if (MODE == kRecurSpreadOut) {
        if (a.dfinal) ld_channels<V>(a.dfinal + k.s * a.channels + l.ch, g0);
        if (l.wave <= behind) {  // from the last block on
            const bool own = l.wave == behind;
            const int32_t row = own ? k.row : k.row + (behind - l.wave) * CANON_RECUR_BLOCK;
            const int32_t len =
                k.span.len - row < CANON_RECUR_BLOCK ? k.span.len - row : CANON_RECUR_BLOCK;
            const int32_t chunks = (len + kRecurRound - 1) / kRecurRound * kRecurWaves;
            double Q, S;
            fold_chunks(a, l, slot + behind - l.wave, chunks - 1,
                        own ? chunks - (mine + 1) * kRecurWaves : chunks, -1, Q, S);
            lc[l.wave][0][at_lds] = Q;
            lc[l.wave][1][at_lds] = S;
        }
    } else if (MODE == kRecurOut && k.span.len > CANON_RECUR_BLOCK) {
        const int32_t last = (k.span.len - 1) / CANON_RECUR_BLOCK;
        if (carrier) block_start<V>(a, l, slot, last - k.row / CANON_RECUR_BLOCK, 1, g0);
    } else if (a.dfinal)
        ld_channels<V>(a.dfinal + k.s * a.channels + l.ch, g0);
    if (carrier && MODE != kRecurSpreadOut) {
#pragma unroll
        for (int j = 0; j < V; ++j) lg[0][at_lds + j] = g0[j];
    }
    int buf = 0;
    for (;;) {
        double Q[V] = {}, S[V] = {};  // in the carrier
        float dd[V] = {};
        for (int rd = MODE == kRecurSpreadOut ? mine : (k.len + kRecurRound - 1) / kRecurRound - 1;
             rd >= (MODE == kRecurSpreadOut ? mine : 0); --rd, buf ^= 1) {
            const int32_t from = k.row + rd * kRecurRound;
            const int n = chunk_rows(l, from, end);
            const int64_t row = k.span.first + from + l.wave * kCh;
            ChunkIn<T, V> in;
            ChunkRows<T, V> dout;
            float e[kCh][V], v[kCh][V], kept[V];
            float q[V] = {}, s[V] = {}, t[V] = {};
            if (n > 0) {
                in.load(a, l, k.s, row, n);
                dout.load(a.dout, a.q, k.s, row, l, n);
                ld_channels<V>(a.kept + (slot * kRecurRounds + rd) * a.channels + l.ch, kept);
                chunk_values<T, V, DECAY>(a, in, n, decay, e, v, [](int) {});
                if (n < kCh) {  // rows that add nothing to lam or to the decay's gradient
#pragma unroll
                    for (int r = 1; r < kCh; ++r)
                        if (r >= n) dout.set(r, 0.f), in.g.set(r, -__builtin_inff());
                }
#pragma unroll
                for (int r = 0; r < kCh; ++r)
#pragma unroll
                    for (int j = 0; j < V; ++j) s[j] = fma32(e[r][j], s[j], s[j]) + v[r][j];
#pragma unroll
                for (int r = kCh - 1; r >= 0; --r)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const float lam = dout.get(r, j) + t[j];
                        t[j] = fma32(e[r][j], lam, lam);
                        q[j] += fma32(e[r][j], q[j], e[r][j]);
                    }
            }
            st_channels<V>(&lq[buf][l.wave][at_lds], q);
            st_channels<V>(&ls[buf][l.wave][at_lds], s);
            st_channels<V>(&lt[buf][l.wave][at_lds], t);
            __syncthreads();
            double G[V];  // what reaches h[t] from the rows behind
            if (MODE == kRecurSpreadOut) {
                for (int32_t b = 0; b < behind; ++b)
                    g0[0] = carry(g0[0], (float)lc[b][0][at_lds], (float)lc[b][1][at_lds]);
                Q[0] = lc[behind][0][at_lds];
                S[0] = lc[behind][1][at_lds];
                G[0] = rd < rounds - 1 ? carried(g0[0], Q[0], S[0], false) : (double)g0[0];
            } else {
#pragma unroll
                for (int j = 0; j < V; ++j) G[j] = lg[buf][at_lds + j];
            }
            if (carrier && (MODE != kRecurSpreadOut || from == 0)) {
#pragma unroll 2
                for (int c = kRecurWaves - 1; c >= 0; --c)
#pragma unroll
                    for (int j = 0; j < V; ++j) {
                        const double cq = lq[buf][c][at_lds + j], ct = lt[buf][c][at_lds + j];
                        S[j] = fma64(cq, S[j], S[j]) + ct;
                        Q[j] += fma64(cq, Q[j], cq);
                    }
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const double gn = carried(g0[j], Q[j], S[j], rd == 0);  // the block's start
                    if (rd == 0) g0[j] = (float)gn;
                    if (MODE != kRecurSpreadOut) lg[buf ^ 1][at_lds + j] = gn;
                }
            }
            if (n <= 0) continue;
#pragma unroll 2
            for (int c = kRecurWaves - 1; c > l.wave; --c)
#pragma unroll
                for (int j = 0; j < V; ++j)
                    G[j] = fma64(lq[buf][c][at_lds + j], G[j], G[j]) + lt[buf][c][at_lds + j];
            float R[V], y[V];
            {
                double h[V];
#pragma unroll
                for (int j = 0; j < V; ++j) h[j] = kept[j];
#pragma unroll 2
                for (int c = 0; c < l.wave; ++c)
#pragma unroll
                    for (int j = 0; j < V; ++j)
                        h[j] = fma64(lq[buf][c][at_lds + j], h[j], h[j]) + ls[buf][c][at_lds + j];
#pragma unroll
                for (int j = 0; j < V; ++j) R[j] = (float)G[j], y[j] = (float)h[j];
            }
#pragma unroll
            for (int r = 0; r < kCh; ++r) {
                st_channels<V>(&before[l.wave][r][at_lds], y);
#pragma unroll
                for (int j = 0; j < V; ++j) y[j] = fma32(e[r][j], y[j], y[j]) + v[r][j];
            }
            in.g.afresh();
            if (a.input.p) in.in.afresh();
            dout.afresh();
            const ChunkOut<T, V> dx(a.dx, a.q, k.s, row, l, n), dg(a.dgate, a.q, k.s, row, l, n),
                di(a.dinput, a.q, k.s, row, l, n);
#pragma unroll
            for (int r = kCh - 1; r >= 0; --r) {
                // rows side by side would need more registers than there are
                if (r % 2) __builtin_amdgcn_sched_barrier(0);
                float out[V], m[V], dinput[V];
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    const float lam = dout.get(r, j) + R[j], hp = before[l.wave][r][at_lds + j];
                    const float er = e[r][j], vr = v[r][j];
                    R[j] = fma32(er, lam, lam);
                    const Sigmoid g = sigmoid_both<T>(in.g.get(r, j));
                    if (DECAY) {
                        // a itself, which 1 + e loses where it is small; by the channel's
                        // decay alone, not its wave's
                        float al = 1.f + er;
                        if (!decay.near && decay.d[j] > 1.f) al = exp_f<T>(-decay.d[j] * g.s);
                        const float z = -er * (2.f + er);
                        // 1 / c; where c is 0, so is v, and the slope counts as 0
                        const float rc = __builtin_amdgcn_rsqf(__builtin_fmaxf(z, 0x1p-126f));
                        const float q1 = al * rc;
                        const float rr = lam * fma32(al, hp, -(q1 * q1 * vr)) * g.s;
                        dd[j] -= rr;
                        out[j] = -decay.d[j] * rr * g.rest;
                        m[j] = z * rc;
                    } else {
                        out[j] = lam * g.s * fma32(-er, hp, -vr);
                        m[j] = -er;
                    }
                    if (a.input.p) {
                        const Sigmoid i = sigmoid_both<T>(in.in.get(r, j));
                        m[j] *= i.s;
                        dinput[j] = lam * vr * i.rest;
                    }
                    m[j] *= lam;
                }
                dg.store(r, out);
                if (a.input.p) di.store(r, dinput);
                dx.store(r, m);
            }
        }
        if (DECAY) {
            st_channels<V>(&ldd[l.wave][at_lds], dd);
            __syncthreads();
            if (l.wave == 0 && l.on) {
#pragma unroll
                for (int j = 0; j < V; ++j) {
                    float v[kRecurWaves];
#pragma unroll
                    for (int w = 0; w < kRecurWaves; ++w) v[w] = ldd[w][at_lds + j];
#pragma unroll
                    for (int p = 1; p < kRecurWaves; p *= 2)
#pragma unroll
                        for (int w = 0; w < kRecurWaves; w += 2 * p) v[w] += v[w + p];
                    dd[j] = v[0];
                }
                st_channels<V>(a.ws_dd + (MODE == kRecurSpreadOut ? job : slot) * a.channels + l.c,
                               dd);
            }
        }
        const bool first = MODE == kRecurSpreadOut ? k.row == 0 && mine == 0 : k.row == 0;
        if (carrier && first && a.dinit && l.on)
            st_channels<V>(a.dinit + k.s * a.channels + l.c, g0);
        if (MODE != kRecurWhole || first) return;
        k.row -= CANON_RECUR_BLOCK;
        k.len = CANON_RECUR_BLOCK;
        --slot;
    }
}

// f(a, DECAY, V, whole): how the work is laid over the compute units, of which a workgroup
// takes one.
//
// Sequences of several blocks are walked whole by a workgroup each, where three quarters of
// the units get one, or else in blocks side by side, for which the folds of the blocks take
// a second pass over x and the gates.  2048 rows of 4096 channels, bf16, both gates, forward
// and backward, whole against side by side: 6 sequences 93 + 203 us against 145 + 210, 3
// sequences 58 + 128 against 88 + 126; but 2 sequences 56 + 114 against 49 + 73.  (Lengths of
// packed sequences are not known here.)
//
// A lane takes two channels where they fill a register and are aligned in every row, but
// one where that leaves no unit two workgroups: 8 sequences 124 + 235 us with two and
// 132 + 263 with one, 4 sequences 80 + 179 and 61 + 132; side by side, 2
// sequences 49 + 73 and 61 + 83, one of 2048 channels 44 + 66 and 33 + 47.
template <typename T, class F>
hipError_t with_recur(RecurArgs a, F&& f)
{
    const int64_t cus = device_cus();
    const bool packed = a.q.starts != nullptr;
    // about as many as have rows: the last block of a packed sequence is short
    const int64_t blocks = slot_count<CANON_RECUR_BLOCK>(a.q.seqs, a.q.rows, packed) -
                           (packed ? a.q.seqs / 2 : 0);
    auto slabs = [&](int v) { return (a.channels + 64 * v - 1) / (64 * v); };
    const bool whole = a.ws_h && !a.spread && !packed && a.q.seqs * slabs(1) >= cus - cus / 4;
    const int v = a.pairs && !a.spread && (whole ? a.q.seqs : blocks) * slabs(1) > cus ? 2 : 1;
    a.slabs = slabs(v);
    if constexpr (sizeof(typename T::store_t) == 2) {
        using Two = std::integral_constant<int, 2>;
        if (v == 2)
            return a.decay ? f(a, std::true_type{}, Two{}, whole)
                           : f(a, std::false_type{}, Two{}, whole);
    }
    using One = std::integral_constant<int, 1>;
    return a.decay ? f(a, std::true_type{}, One{}, whole) : f(a, std::false_type{}, One{}, whole);
}

template <typename T, bool DECAY, int V>
hipError_t launch_recurrence_t(const RecurArgs& a, bool whole, hipStream_t st)
{
    const dim3 threads(64 * kRecurWaves);
    const unsigned seqs = (unsigned)(a.q.seqs * a.slabs);
    const unsigned carries = (unsigned)(a.q.seqs * ((a.channels + 63) / 64));
    const int64_t slots = slot_count<CANON_RECUR_BLOCK>(a.q.seqs, a.q.rows, a.q.starts != nullptr);
    const unsigned blocks = (unsigned)(slots * a.slabs);
    if constexpr (V == 1) {
        if (a.spread) {
            const dim3 rounds((unsigned)(blocks * kRecurRounds));
            k_recur_chunks<T, DECAY, false><<<rounds, threads, 0, st>>>(a);
            if (hipError_t e = hipGetLastError()) return e;
            k_recurrence<T, 1, DECAY, kRecurSpreadOut><<<rounds, threads, 0, st>>>(a);
            return hipGetLastError();
        }
    }
    if (whole) {
        k_recurrence<T, V, DECAY, kRecurWhole><<<dim3(seqs), threads, 0, st>>>(a);
        return hipGetLastError();
    }
    if (a.ws_h) {
        k_recurrence<T, V, DECAY, kRecurSum><<<dim3(blocks), threads, 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
        if (a.carry) k_recur_carry<false><<<dim3(carries), dim3(64), 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    k_recurrence<T, V, DECAY, kRecurOut><<<dim3(blocks), threads, 0, st>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_recurrence(const RecurArgs& a, hipStream_t st)
{
    return with_recur<T>(a, [&](const RecurArgs& b, auto d, auto v, bool whole) {
        return launch_recurrence_t<T, decltype(d)::value, decltype(v)::value>(b, whole, st);
    });
}

template <typename T, bool DECAY, int V>
hipError_t launch_recurrence_grad_t(const RecurArgs& a, bool whole, hipStream_t st)
{
    const dim3 threads(64 * kRecurWaves);
    const unsigned seqs = (unsigned)(a.q.seqs * a.slabs);
    const unsigned carries = (unsigned)(a.q.seqs * ((a.channels + 63) / 64));
    const int64_t slots = slot_count<CANON_RECUR_BLOCK>(a.q.seqs, a.q.rows, a.q.starts != nullptr);
    const unsigned blocks = (unsigned)(slots * a.slabs);
    if (a.spread) {
        if constexpr (V == 1) {
            const dim3 rounds((unsigned)(blocks * kRecurRounds));
            k_recur_chunks<T, DECAY, true><<<rounds, threads, 0, st>>>(a);
            if (hipError_t e = hipGetLastError()) return e;
            k_recurrence_grad<T, 1, DECAY, kRecurSpreadOut><<<rounds, threads, 0, st>>>(a);
        }
    } else if (whole) {
        k_recurrence_grad<T, V, DECAY, kRecurWhole><<<dim3(seqs), threads, 0, st>>>(a);
    } else if (slots > 0) {
        if (a.ws_h) {
            k_recur_back_sum<T, V, DECAY><<<dim3(blocks), threads, 0, st>>>(a);
            if (hipError_t e = hipGetLastError()) return e;
            if (a.carry) k_recur_carry<true><<<dim3(carries), dim3(64), 0, st>>>(a);
            if (hipError_t e = hipGetLastError()) return e;
        }
        k_recurrence_grad<T, V, DECAY, kRecurOut><<<dim3(blocks), threads, 0, st>>>(a);
    }
    if (hipError_t e = hipGetLastError()) return e;
    if (!DECAY) return hipSuccess;
    ColumnSums sums{{{a.ws_dd, a.channels, 1, 1, a.ddecay}, {}, {}},
                    a.spread ? slots * kRecurRounds : slots};
    return launch_column_sums(sums, st);
}

template <typename T>
hipError_t launch_recurrence_grad(const RecurArgs& a, hipStream_t st)
{
    return with_recur<T>(a, [&](const RecurArgs& b, auto d, auto v, bool whole) {
        return launch_recurrence_grad_t<T, decltype(d)::value, decltype(v)::value>(b, whole, st);
    });
}

template <typename T>
hipError_t launch_recurrence_step(const RecurArgs& a, hipStream_t st)
{
    const dim3 grid((unsigned)((a.q.seqs * a.channels + 255) / 256));
    if (a.decay)
        k_recurrence_step<T, true><<<grid, dim3(256), 0, st>>>(a);
    else
        k_recurrence_step<T, false><<<grid, dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

}  // namespace seq
}  // namespace canon
