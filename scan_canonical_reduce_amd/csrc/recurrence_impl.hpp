// The gated linear recurrence h[t] = a h[t-1] + c i x[t], elementwise over the
// channels: forward, backward and single rows.
//
// A lane holds one channel; a wave walks a chunk of 16 rows, whose inputs it loads
// at once.  The waves of a workgroup take the chunks of a round (128 rows), fold
// each from zero, exchange the folds through LDS, and fold again from their chunks'
// start states, with e = a - 1 and v = c i x still in registers: one pass over
// memory.  Rounds of a block (512 rows) follow each other in the workgroup.
//
// a is near 1 for a long memory, and a rounding of h at every row would add up over
// that memory.  So everything is kept as differences from 1: with e = a - 1,
//   h <- h + (e h + v),   and for the product of a, Q = P - 1:  Q <- Q + (e Q + e),
// and the start states of chunks, which see one rounding per chunk, are carried in 64
// bits inside a block and rounded to 32 between blocks.
#pragma once

#include <type_traits>

#include "column_sum.hpp"
#include "launch.hpp"
#include "recurrence.hpp"

namespace canon {
namespace seq {

constexpr int kCh = CANON_RECUR_CHUNK;

__device__ __forceinline__ double fma64(double a, double b, double c) { return __builtin_fma(a, b, c); }

// exp(l) - 1 for l <= 0: the series, whose next term is below 2^-25 of l up to
// 0.35, or the exponential less 1, which loses a bit and a half there.
template <typename T>
__device__ __forceinline__ float expm1_f(float l, bool near_only)
{
    float p = fma32(l, 0x1.a01a02p-13f, 0x1.6c16c2p-10f);  // 1/7!, 1/6!
    p = fma32(p, l, 0x1.111112p-7f);
    p = fma32(p, l, 0x1.555556p-5f);
    p = fma32(p, l, 0x1.555556p-3f);
    p = fma32(p, l, 0.5f);
    const float near = fma32(l * l, p, l);
    if (near_only) return near;
    return l > -0.35f ? near : exp_f<T>(l) - 1.f;
}

// A channel's decay, and whether no lane of the wave has one above 0.35: then the
// logarithm of a, between -decay and 0, needs the series alone.
struct Decay {
    float d;
    bool near_only;
};
template <bool DECAY>
__device__ __forceinline__ Decay load_decay(const float* decay, int32_t ch)
{
    if (!DECAY) return Decay{0.f, false};
    const float d = decay[ch];
    return Decay{d, __ballot(d < 0.35f) == ~0ull};
}

// e = a - 1
template <typename T, bool DECAY>
__device__ __forceinline__ float gate_e(float gate, const Decay& d)
{
    if (!DECAY) return -sigmoid_f<T>(-gate);
    return expm1_f<T>(-d.d * sigmoid_f<T>(gate), d.near_only);
}
// sqrt(1 - a^2) = sqrt((1 - a)(1 + a)), or 1 - a
template <bool DECAY>
__device__ __forceinline__ float factor(float e)
{
    return DECAY ? __builtin_amdgcn_sqrtf(-e * (2.f + e)) : -e;
}

// A wave's channel and place in its workgroup.
struct Lane {
    int lane, wave;
    int32_t c, ch;  // channel, and one that may be read
    bool on;        // c is a channel
};
__device__ __forceinline__ Lane recur_lane(const RecurArgs& a, int32_t slab)
{
    Lane l;
    l.lane = threadIdx.x & 63;
    l.wave = uniform((int32_t)(threadIdx.x >> 6));
    l.c = slab * 64 + l.lane;
    l.on = l.c < a.channels;
    l.ch = l.on ? l.c : a.channels - 1;
    return l;
}

// The rows of a chunk in the lane's channel.  Byte offsets within a chunk are 32-bit:
// fewer than 16 rows of a pitch below 2^24 elements, and a channel below 2^24 (the host
// checks both).
template <typename T>
struct ChunkRows {
    using E = typename T::store_t;
    uint32_t v[kCh];  // bits

    // n rows are valid, at least one; the others are a copy of the last
    __device__ __forceinline__ void load(const canon_rows_t& a, const Seqs& q, int64_t s, int64_t row,
                                         const Lane& l, int n)
    {
        const __amdgpu_buffer_rsrc_t b = tile_rsrc(rows_ptr<T>(a, s, q, row));
        const uint32_t pitch = (uint32_t)a.row * (uint32_t)sizeof(E);
        const uint32_t off = (uint32_t)l.ch * (uint32_t)sizeof(E);
        if (n >= kCh) {
#pragma unroll
            for (int r = 0; r < kCh; ++r) v[r] = bits(b, off, r * pitch);
        } else {
#pragma unroll
            for (int r = 0; r < kCh; ++r) v[r] = bits(b, off, (r < n ? r : n - 1) * pitch);
        }
    }
    static __device__ __forceinline__ uint32_t bits(__amdgpu_buffer_rsrc_t b, uint32_t off,
                                                    uint32_t row)
    {
        if constexpr (sizeof(E) == 2)
            return __builtin_amdgcn_raw_buffer_load_b16(b, off, row, 0);
        else
            return __builtin_amdgcn_raw_buffer_load_b32(b, off, row, 0);
    }
    __device__ __forceinline__ float operator[](int r) const
    {
        if constexpr (sizeof(E) == 2)
            return T::load((uint16_t)v[r]);
        else
            return __uint_as_float(v[r]);
    }
    // The same values, as if loaded again: what was computed from them before is
    // computed anew instead of waiting in registers.
    __device__ __forceinline__ void afresh()
    {
#pragma unroll
        for (int r = 0; r < kCh; ++r) asm("" : "+v"(v[r]));
    }
};

// The rows of a chunk of an output.
template <typename T>
struct ChunkOut {
    using E = typename T::store_t;
    __amdgpu_buffer_rsrc_t b;
    uint32_t pitch, off;
    __device__ __forceinline__ ChunkOut(const canon_rows_t& a, const Seqs& q, int64_t s, int64_t row,
                                        const Lane& l)
        : b(tile_rsrc(rows_ptr<T>(a, s, q, row))),
          pitch((uint32_t)a.row * (uint32_t)sizeof(E)),
          off((uint32_t)l.c * (uint32_t)sizeof(E))
    {
    }
    __device__ __forceinline__ void store(int r, float v) const
    {
        rsrc_store(b, off, r * pitch, T::round(v));
    }
};

// What a chunk reads.
template <typename T>
struct ChunkIn {
    ChunkRows<T> x, g, in;
    __device__ __forceinline__ void load(const RecurArgs& a, const Lane& l, int64_t s, int64_t row,
                                         int n)
    {
        g.load(a.gate, a.q, s, row, l, n);
        x.load(a.x, a.q, s, row, l, n);
        if (a.input.p) in.load(a.input, a.q, s, row, l, n);
    }
};

// e and m = c i of a chunk's rows; rows beyond n leave the state as it is.
template <typename T, bool DECAY>
__device__ __forceinline__ void chunk_gates(const RecurArgs& a, const ChunkIn<T>& c, int n,
                                            const Decay& d, float (&e)[kCh], float (&m)[kCh])
{
#pragma unroll
    for (int r = 0; r < kCh; ++r) {
        if (r % 4 == 0) __builtin_amdgcn_sched_barrier(0);  // else more registers
        e[r] = gate_e<T, DECAY>(c.g[r], d);
        m[r] = factor<DECAY>(e[r]);
    }
    if (a.input.p) {
#pragma unroll
        for (int r = 0; r < kCh; ++r) m[r] *= sigmoid_f<T>(c.in[r]);
    }
    if (n < kCh) {
#pragma unroll
        for (int r = 0; r < kCh; ++r)
            if (r >= n) e[r] = m[r] = 0.f;
    }
}

// A value at the start of the next block, given the block's Q and S.
__device__ __forceinline__ float carry(float h, float q, float s)
{
    return (float)((double)h + fma64(q, h, s));
}

enum { kRecurSum, kRecurOut, kRecurWhole };

// kRecurSum: Q and S of each block.  kRecurOut: the outputs of each block, from its
// start state.  kRecurWhole: the outputs of whole sequences, block after block.
template <typename T, bool DECAY, int MODE>
__global__ __launch_bounds__(64 * kRecurWaves, 4) void k_recurrence(RecurArgs a)
{
    __shared__ float lq[2][kRecurWaves][64], ls[2][kRecurWaves][64], lh[64];
    const int64_t job = blockIdx.x / (uint32_t)a.slabs;
    const Lane l = recur_lane(a, blockIdx.x - (uint32_t)job * a.slabs);
    const Decay decay = load_decay<DECAY>(a.decay, l.ch);
    Chunk k;
    int64_t slot = job;
    if (MODE == kRecurWhole) {
        k = Chunk{job, Span{0, (int32_t)a.q.rows}, 0, (int32_t)a.q.rows};
        if (k.len > CANON_RECUR_BLOCK) k.len = CANON_RECUR_BLOCK;
        slot = job * chunks_per_seq<CANON_RECUR_BLOCK>(a.q.rows);
    } else {
        k = wave_slot_chunk<CANON_RECUR_BLOCK>(a.q, slot);
        if (k.len <= 0 && k.row != 0) return;  // no block has this slot
        if (k.len < 0) k.len = 0;
        // the last block's fold serves no other
        if (MODE == kRecurSum && k.row + k.len >= k.span.len) return;
    }
    float h0 = 0.f;
    // a block reads its start state where k_recur_carry has put it, also the first one:
    // the last one's workgroup may have overwritten init with final
    if (MODE == kRecurOut && a.ws_h)
        h0 = a.ws_h[slot * a.channels + l.ch];
    else if (MODE != kRecurSum && a.init)
        h0 = a.init[k.s * a.channels + l.ch];
    // the wave's rows of the round at `from`, none beyond `end`
    const int32_t end = MODE == kRecurWhole ? k.span.len : k.row + k.len;
    auto rows_of = [&](int32_t from) {
        const int32_t left = end - from - l.wave * kCh;
        return left < kCh ? left : kCh;
    };
    int buf = 0;
    ChunkIn<T> in;
    if (const int n = rows_of(k.row); n > 0)
        in.load(a, l, k.s, k.span.first + k.row + l.wave * kCh, n);
    for (;;) {
        double h = h0, Q = 0., S = 0.;
        const int rounds = (k.len + kRecurRound - 1) / kRecurRound;
        for (int rd = 0; rd < rounds; ++rd, buf ^= 1) {
            const int32_t from = k.row + rd * kRecurRound, at = from + l.wave * kCh;
            const int n = rows_of(from);
            float e[kCh], v[kCh];
            if (n > 0) {
                chunk_gates<T, DECAY>(a, in, n, decay, e, v);
#pragma unroll
                for (int r = 0; r < kCh; ++r) v[r] *= in.x[r];
                // the next round's rows arrive meanwhile
                if (const int m = rows_of(from + kRecurRound); m > 0)
                    in.load(a, l, k.s, k.span.first + at + kRecurRound, m);
                float q = 0.f, s = 0.f;
#pragma unroll
                for (int r = 0; r < kCh; ++r) {
                    s += fma32(e[r], s, v[r]);
                    q += fma32(e[r], q, e[r]);
                }
                lq[buf][l.wave][l.lane] = q;
                ls[buf][l.wave][l.lane] = s;
            }
            __syncthreads();
            if (MODE != kRecurSum && a.kept && l.wave == 0 && l.on)
                a.kept[(slot * kRecurRounds + rd) * a.channels + l.c] = (float)h;
            const int32_t rows_left = k.len - rd * kRecurRound;
            const int chunks =
                rows_left < kRecurRound ? (rows_left + kCh - 1) / kCh : kRecurWaves;
            double mine = h;
#pragma unroll 1
            for (int c = 0; c < chunks; ++c) {
                const double q = lq[buf][c][l.lane], s = ls[buf][c][l.lane];
                if (MODE != kRecurSum) {
                    if (c == l.wave) mine = h;
                    h += fma64(q, h, s);
                }
                if (l.wave == 0) {
                    S += fma64(q, S, s);
                    Q += fma64(q, Q, q);
                }
            }
            if (MODE != kRecurSum && n > 0) {
                float y = (float)mine;
                const ChunkOut<T> out(a.out, a.q, k.s, k.span.first + at, l);
#pragma unroll
                for (int r = 0; r < kCh; ++r) {
                    y += fma32(e[r], y, v[r]);
                    v[r] = y;
                }
                if (l.on) {
                    if (n >= kCh) {
#pragma unroll
                        for (int r = 0; r < kCh; ++r) out.store(r, v[r]);
                    } else {
#pragma unroll
                        for (int r = 0; r < kCh; ++r)
                            if (r < n) out.store(r, v[r]);
                    }
                }
            }
        }
        const bool last = k.row + k.len >= k.span.len;
        if (MODE == kRecurSum) {
            if (l.wave == 0 && l.on) {
                a.ws_q[slot * a.channels + l.c] = (float)Q;
                a.ws_s[slot * a.channels + l.c] = (float)S;
            }
            return;
        }
        if (l.wave == 0) {
            if (k.len > 0) h0 = carry(h0, (float)Q, (float)S);
            if (last && a.final && l.on) a.final[k.s * a.channels + l.c] = h0;
        }
        if (MODE == kRecurOut || last) return;
        // wave 0's value for all; the next round's barrier is before the next write
        if (l.wave == 0) lh[l.lane] = h0;
        __syncthreads();
        h0 = lh[l.lane];
        k.row += CANON_RECUR_BLOCK;
        k.len = k.span.len - k.row < CANON_RECUR_BLOCK ? k.span.len - k.row : CANON_RECUR_BLOCK;
        ++slot;
    }
}

// The start states of each sequence's blocks from the blocks' Q and S (in ws_q,
// ws_s), into ws_h; backwards: the gradients that come in past their ends.
template <bool BACK>
__global__ __launch_bounds__(64) void k_recur_carry(RecurArgs a)
{
    const int64_t s = blockIdx.x / (uint32_t)a.slabs;
    const int32_t c = (blockIdx.x - (uint32_t)s * a.slabs) * 64 + threadIdx.x;
    if (c >= a.channels) return;
    const Span span = seq_span(a.q, s);
    const int64_t slot = slot_base<CANON_RECUR_BLOCK>(a.q, s);
    const int32_t blocks = (span.len + CANON_RECUR_BLOCK - 1) / CANON_RECUR_BLOCK;
    const float* from = BACK ? a.dfinal : a.init;
    float h = from ? from[s * a.channels + c] : 0.f;
    a.ws_h[(slot + (BACK && blocks > 0 ? blocks - 1 : 0)) * a.channels + c] = h;
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
    const float e = gate_e<T, DECAY>(ld<T>(row(a.gate)), Decay{DECAY ? a.decay[c] : 0.f, false});
    float v = factor<DECAY>(e) * ld<T>(row(a.x));
    if (a.input.p) v *= sigmoid_f<T>(ld<T>(row(a.input)));
    float h = a.init ? a.init[i] : 0.f;
    h += fma32(e, h, v);
    st<T>(row(a.out), h);
    if (a.final) a.final[i] = h;
}

// Backward.  With lam[t] = dout[t] + a[t+1] lam[t+1], the gradient of h[t]:
//   dx = lam c i,   da = lam h[t-1],   d(c i x) = lam,
// where h is folded again from the states kept at every round.  The fold of lam goes
// backwards over chunks, rounds and blocks just as h's does forwards.
// k_recur_back_sum: Q and the fold from zero of each block.
template <typename T, bool DECAY>
__global__ __launch_bounds__(64 * kRecurWaves) void k_recur_back_sum(RecurArgs a)
{
    __shared__ float lq[2][kRecurWaves][64], lt[2][kRecurWaves][64];
    const int64_t slot = blockIdx.x / (uint32_t)a.slabs;
    const Lane l = recur_lane(a, blockIdx.x - (uint32_t)slot * a.slabs);
    const Decay decay = load_decay<DECAY>(a.decay, l.ch);
    const Chunk k = wave_slot_chunk<CANON_RECUR_BLOCK>(a.q, slot);
    if (k.len <= 0 || k.row == 0) return;  // the first block's fold serves no other
    double Q = 0., G = 0.;
    int buf = 0;
    for (int rd = (k.len - 1) / kRecurRound; rd >= 0; --rd, buf ^= 1) {
        const int32_t at = k.row + rd * kRecurRound + l.wave * kCh;
        const int32_t left = k.row + k.len - at;
        const int n = left < kCh ? left : kCh;
        float q = 0.f, t = 0.f;
        if (n > 0) {
            ChunkRows<T> g, d;
            g.load(a.gate, a.q, k.s, k.span.first + at, l, n);
            d.load(a.dout, a.q, k.s, k.span.first + at, l, n);
#pragma unroll
            for (int r = kCh - 1; r >= 0; --r) {
                const float e = r < n ? gate_e<T, DECAY>(g[r], decay) : 0.f;
                const float lam = r < n ? d[r] + t : t;
                t = fma32(e, lam, lam);
                q += fma32(e, q, e);
            }
        }
        lq[buf][l.wave][l.lane] = q;
        lt[buf][l.wave][l.lane] = t;
        __syncthreads();
        if (l.wave == 0)
            for (int c = kRecurWaves - 1; c >= 0; --c) {
                const double cq = lq[buf][c][l.lane], ct = lt[buf][c][l.lane];
                G += fma64(cq, G, ct);
                Q += fma64(cq, Q, cq);
            }
    }
    if (l.wave == 0 && l.on) {
        a.ws_q[slot * a.channels + l.c] = (float)Q;
        a.ws_s[slot * a.channels + l.c] = (float)G;
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
template <typename T, bool DECAY, int MODE>
__global__ __launch_bounds__(64 * kRecurWaves, sizeof(typename T::store_t) == 2 ? 4 : 2) void
k_recurrence_grad(RecurArgs a)
{
    __shared__ float lq[2][kRecurWaves][64], ls[2][kRecurWaves][64], lt[2][kRecurWaves][64],
        lh[64], ldd[kRecurWaves][64], before[kRecurWaves][kCh][64];
    const int64_t job = blockIdx.x / (uint32_t)a.slabs;
    const Lane l = recur_lane(a, blockIdx.x - (uint32_t)job * a.slabs);
    const Decay decay = load_decay<DECAY>(a.decay, l.ch);
    Chunk k;
    int64_t slot = job;
    if (MODE == kRecurWhole) {
        const int32_t rows = (int32_t)a.q.rows;
        const int32_t blocks = (int32_t)chunks_per_seq<CANON_RECUR_BLOCK>(rows);
        const int32_t row = (blocks - 1) * CANON_RECUR_BLOCK;
        k = Chunk{job, Span{0, rows}, row, rows - row};
        slot = job * blocks + blocks - 1;
    } else {
        k = wave_slot_chunk<CANON_RECUR_BLOCK>(a.q, slot);
        if (k.len < 0) k.len = 0;
        if (k.len == 0 && k.row != 0) {  // no block has this slot
            if (DECAY && l.wave == 0 && l.on) a.ws_dd[slot * a.channels + l.c] = 0.f;
            return;
        }
    }
    float g0 = 0.f;
    if (MODE == kRecurOut && a.ws_h)
        g0 = a.ws_h[slot * a.channels + l.ch];
    else if (a.dfinal)
        g0 = a.dfinal[k.s * a.channels + l.ch];
    int buf = 0;
    for (;;) {
        double G = g0, Q = 0., S = 0.;
        float dd = 0.f;
        for (int rd = (k.len + kRecurRound - 1) / kRecurRound - 1; rd >= 0; --rd, buf ^= 1) {
            const int32_t at = k.row + rd * kRecurRound + l.wave * kCh;
            const int32_t left = k.row + k.len - at;
            const int n = left < kCh ? left : kCh;
            const int64_t row = k.span.first + at;
            ChunkIn<T> in;
            ChunkRows<T> dout;
            float e[kCh], v[kCh];
            float q = 0.f, s = 0.f, t = 0.f;
            if (n > 0) {
                in.load(a, l, k.s, row, n);
                dout.load(a.dout, a.q, k.s, row, l, n);
                chunk_gates<T, DECAY>(a, in, n, decay, e, v);
#pragma unroll
                for (int r = 0; r < kCh; ++r) {
                    if (r % 4 == 0) __builtin_amdgcn_sched_barrier(0);
                    v[r] *= in.x[r];
                    s += fma32(e[r], s, v[r]);
                }
#pragma unroll
                for (int r = kCh - 1; r >= 0; --r) {
                    if (r % 4 == 3) __builtin_amdgcn_sched_barrier(0);
                    const float lam = r < n ? dout[r] + t : t;
                    t = fma32(e[r], lam, lam);
                    q += fma32(e[r], q, e[r]);
                }
            }
            lq[buf][l.wave][l.lane] = q;
            ls[buf][l.wave][l.lane] = s;
            lt[buf][l.wave][l.lane] = t;
            __syncthreads();
            double h = a.kept[(slot * kRecurRounds + rd) * a.channels + l.ch];
#pragma unroll 1
            for (int c = 0; c < l.wave; ++c)
                h += fma64(lq[buf][c][l.lane], h, ls[buf][c][l.lane]);
            double mine = G;
#pragma unroll 1
            for (int c = kRecurWaves - 1; c >= 0; --c) {
                const double cq = lq[buf][c][l.lane], ct = lt[buf][c][l.lane];
                if (c == l.wave) mine = G;
                G += fma64(cq, G, ct);
                if (l.wave == 0) {
                    S += fma64(cq, S, ct);
                    Q += fma64(cq, Q, cq);
                }
            }
            if (n <= 0) continue;
            float y = (float)h;
#pragma unroll
            for (int r = 0; r < kCh; ++r) {
                before[l.wave][r][l.lane] = y;
                y += fma32(e[r], y, v[r]);
            }
            in.g.afresh();
            if (a.input.p) in.in.afresh();
            dout.afresh();
            const ChunkOut<T> dx(a.dx, a.q, k.s, row, l), dg(a.dgate, a.q, k.s, row, l),
                di(a.dinput, a.q, k.s, row, l);
            float R = (float)mine;  // what reaches h[t] from the rows behind
#pragma unroll
            for (int r = kCh - 1; r >= 0; --r) {
                if (r >= n) continue;
                // rows side by side would need more registers than there are
                if (r % 2) __builtin_amdgcn_sched_barrier(0);
                const float lam = dout[r] + R, hp = before[l.wave][r][l.lane];
                R = fma32(e[r], lam, lam);
                const Sigmoid g = sigmoid_both<T>(in.g[r]);
                float out, m;
                if (DECAY) {
                    const float al = 1.f + e[r], z = -e[r] * (2.f + e[r]);
                    const float slope = z > 0.f ? al * al * rcp_hw(z) : 0.f;
                    const float rr = lam * fma32(al, hp, -(slope * v[r])) * g.s;
                    dd -= rr;
                    out = -decay.d * rr * g.rest;
                    m = __builtin_amdgcn_sqrtf(z);
                } else {
                    // a itself, which 1 + e loses where it is small
                    out = lam * g.s * fma32(-e[r], hp, -v[r]);
                    m = -e[r];
                }
                if (l.on) {
                    dg.store(r, out);
                    if (a.input.p) {
                        const Sigmoid i = sigmoid_both<T>(in.in[r]);
                        m *= i.s;
                        di.store(r, lam * v[r] * i.rest);
                    }
                    dx.store(r, lam * m);
                }
            }
        }
        if (DECAY) {
            ldd[l.wave][l.lane] = dd;
            __syncthreads();
            if (l.wave == 0 && l.on) {
                float v[kRecurWaves];
#pragma unroll
                for (int w = 0; w < kRecurWaves; ++w) v[w] = ldd[w][l.lane];
#pragma unroll
                for (int p = 1; p < kRecurWaves; p *= 2)
#pragma unroll
                    for (int w = 0; w < kRecurWaves; w += 2 * p) v[w] += v[w + p];
                a.ws_dd[slot * a.channels + l.c] = v[0];
            }
        }
        const bool first = k.row == 0;
        if (l.wave == 0) {
            if (k.len > 0) g0 = carry(g0, (float)Q, (float)S);
            if (first && a.dinit && l.on) a.dinit[k.s * a.channels + l.c] = g0;
        }
        if (MODE == kRecurOut || first) return;
        if (l.wave == 0) lh[l.lane] = g0;
        __syncthreads();
        g0 = lh[l.lane];
        k.row -= CANON_RECUR_BLOCK;
        k.len = CANON_RECUR_BLOCK;
        --slot;
    }
}

// Sequences that are walked whole by a workgroup each: where that gives every
// compute unit one.  Packed ones never are (their lengths are not known here).
inline bool recur_whole(const RecurArgs& a)
{
    return a.q.starts == nullptr && a.q.seqs * a.slabs >= (int64_t)device_cus();
}

template <typename T, bool DECAY>
hipError_t launch_recurrence_t(const RecurArgs& a, hipStream_t st)
{
    const dim3 threads(64 * kRecurWaves);
    const unsigned seqs = (unsigned)(a.q.seqs * a.slabs);
    const int64_t slots = slot_count<CANON_RECUR_BLOCK>(a.q.seqs, a.q.rows, a.q.starts != nullptr);
    const unsigned blocks = (unsigned)(slots * a.slabs);
    if (a.ws_h && recur_whole(a)) {
        k_recurrence<T, DECAY, kRecurWhole><<<dim3(seqs), threads, 0, st>>>(a);
        return hipGetLastError();
    }
    if (a.ws_h) {
        k_recurrence<T, DECAY, kRecurSum><<<dim3(blocks), threads, 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
        k_recur_carry<false><<<dim3(seqs), dim3(64), 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    k_recurrence<T, DECAY, kRecurOut><<<dim3(blocks), threads, 0, st>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_recurrence(const RecurArgs& a, hipStream_t st)
{
    return a.decay ? launch_recurrence_t<T, true>(a, st) : launch_recurrence_t<T, false>(a, st);
}

template <typename T, bool DECAY>
hipError_t launch_recurrence_grad_t(const RecurArgs& a, hipStream_t st)
{
    const dim3 threads(64 * kRecurWaves);
    const unsigned seqs = (unsigned)(a.q.seqs * a.slabs);
    const int64_t slots = slot_count<CANON_RECUR_BLOCK>(a.q.seqs, a.q.rows, a.q.starts != nullptr);
    const unsigned blocks = (unsigned)(slots * a.slabs);
    if (a.ws_h && recur_whole(a)) {
        k_recurrence_grad<T, DECAY, kRecurWhole><<<dim3(seqs), threads, 0, st>>>(a);
    } else if (slots > 0) {
        if (a.ws_h) {
            k_recur_back_sum<T, DECAY><<<dim3(blocks), threads, 0, st>>>(a);
            if (hipError_t e = hipGetLastError()) return e;
            k_recur_carry<true><<<dim3(seqs), dim3(64), 0, st>>>(a);
            if (hipError_t e = hipGetLastError()) return e;
        }
        k_recurrence_grad<T, DECAY, kRecurOut><<<dim3(blocks), threads, 0, st>>>(a);
    }
    if (hipError_t e = hipGetLastError()) return e;
    if (!DECAY) return hipSuccess;
    ColumnSums sums{{{a.ws_dd, a.channels, 1, 1, a.ddecay}, {}, {}}, slots};
    return launch_column_sums(sums, st);
}

template <typename T>
hipError_t launch_recurrence_grad(const RecurArgs& a, hipStream_t st)
{
    return a.decay ? launch_recurrence_grad_t<T, true>(a, st)
                   : launch_recurrence_grad_t<T, false>(a, st);
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
