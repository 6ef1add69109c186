// Selective state space scan: forward pass and single rows.
//
// A wave holds 16 channels.  Its lanes are four rows of 16: lane c of row q
// keeps channel c's states KS q .. KS q + KS - 1 (KS = 1, 2, 4 for up to 4,
// 8, 16 states) in registers and walks the rows of the sequence in order.
// Every wave is independent; nothing is exchanged between waves:
//   - A tile is 16 sequence rows.  For the values of one (row, channel), lane
//     c of row q takes sequence rows 4 r + q, r < 4, so each softplus, gate
//     and store is done once; dl and dl u reach the other lanes of the channel
//     through 2 KiB of LDS that only this wave uses (no barrier).
//   - B and C of sequence row t are held by lane t of each row of lanes and
//     reach the others as the DPP operand of the multiplication itself
//     (row_newbcast), without LDS or an instruction of their own.
//   - y is summed over a lane's states, then over the four rows of lanes, four
//     sequence rows at a time (permlane swaps: 6 instructions for 4 rows),
//     which leaves it where the gate and the store want it.
// Per (row, channel, state) that is 2 multiplications, 1 exponential and 2 FMAs
// (3 in the kernel that walks whole sequences).  Measured on one SIMD of an
// MI355X, in cycles a wave: FMA or product of vector registers 2.8, with a DPP
// operand 4.5, exponential 8.4, lane swap 8; so about 23 cycles for 64 values,
// and the kernel is bound by vector issue, not by memory: at 8 x 2048 x 4096 and
// 16 states the values alone take 170 us of the 400 (whole sequences, which also
// save the states for the backward pass), of 142 for one sequence of 16384 x 2048
// in chunks, whose sums from zero take another 107.
#pragma once

#include "launch.hpp"
#include "selective_scan.hpp"

namespace canon {
namespace seq {

constexpr int kCh = CANON_SCAN_CHUNK;
constexpr int kSubs = kCh / kSub;

enum ScanMode {
    kSum,   // each chunk's fold from zero and sum of dl, to the workspace
    kEmit,  // one chunk from its start state in the workspace
    kSeq    // a whole sequence, chunk after chunk, the state carried
};

// The lane's place: channel and states.
struct Lane {
    int q, c;
    int32_t ch;    // channel (a valid one also where the lane has none)
    bool active;
    int32_t wch;   // the wave's first channel within the group
    int32_t g;
};

__device__ __forceinline__ Lane lane_place(const ScanArgs& a, int slab)
{
    Lane l;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    l.q = lane >> 4;
    l.c = lane & 15;
    l.g = slab / a.slabs;
    l.wch = (slab - l.g * a.slabs) * kSlab + w * 16;
    const int32_t in_g = l.wch + l.c;
    l.active = in_g < a.dg;
    l.ch = l.g * a.dg + (l.active ? in_g : a.dg - 1);
    return l;
}

template <typename T>
__device__ __forceinline__ uint32_t tile_off(const canon_rows_t& r, uint32_t t, uint32_t col)
{
    return (t * (uint32_t)r.row + col) * (uint32_t)sizeof(typename T::store_t);
}

// A lane's rows 4 r + q of one activation's current 16-row tile.
template <typename T>
struct LaneRows {
    using E = typename T::store_t;
    E* base;        // the tile's first row (wave-uniform)
    uint32_t step;  // 4 rows, in bytes
    uint32_t off;   // row q, this lane's channel

    __device__ __forceinline__ void init(const canon_rows_t& r, const Lane& l, int64_t s,
                                         const Seqs& q, int64_t first)
    {
        base = rows_ptr<T>(r, s, q, first);
        step = tile_off<T>(r, 4, 0);
        off = tile_off<T>(r, l.q, l.ch);
    }
    __device__ __forceinline__ void next() { base += 4 * (uint64_t)step / sizeof(E); }
    __device__ __forceinline__ void prev() { base -= 4 * (uint64_t)step / sizeof(E); }
    // rows past the sequence's end are read as its last row and not used
    __device__ __forceinline__ void load(const canon_rows_t& a, const Lane& l, int32_t len,
                                         E (&v)[4]) const
    {
        const __amdgpu_buffer_rsrc_t b = tile_rsrc(base);
        if (len >= kSub) {
#pragma unroll
            for (int r = 0; r < 4; ++r) rsrc_load(b, off, r * step, v[r]);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int t = 4 * r + l.q < len ? 4 * r + l.q : len - 1;
                rsrc_load(b, tile_off<T>(a, t, l.ch), 0, v[r]);
            }
        }
    }
    __device__ __forceinline__ void store(const Lane& l, int32_t len, const float (&v)[4]) const
    {
        if (!l.active) return;
        const __amdgpu_buffer_rsrc_t b = tile_rsrc(base);
        if (len >= kSub) {
#pragma unroll
            for (int r = 0; r < 4; ++r) rsrc_store(b, off, r * step, T::round(v[r]));
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (4 * r + l.q < len) rsrc_store(b, off, r * step, T::round(v[r]));
        }
    }
};

// B or C of the tile's row c: this lane's states (0 beyond the last one, and
// for rows past the end).
template <typename T, int KS>
struct LaneBC {
    using E = typename T::store_t;
    E* base;
    int64_t step;  // 16 rows
    uint32_t off;
    Vec<T, KS> x;

    __device__ __forceinline__ void init(const ScanArgs& a, const canon_rows_t& r, const Lane& l,
                                         int64_t s, int64_t first)
    {
        base = rows_ptr<T>(r, s, a.q, first);
        step = kSub * r.row;
        off = tile_off<T>(r, l.c, l.g * a.states + l.q * KS);
    }
    __device__ __forceinline__ void next() { base += step; }
    __device__ __forceinline__ void prev() { base -= step; }
    __device__ __forceinline__ void load(const ScanArgs& a, const Lane& l, int32_t len)
    {
        x = Vec<T, KS>{};
        if (l.c >= len || l.q * KS >= a.states) return;
        if (a.bc_vec) {
            x = ld_vec<T, KS>(reinterpret_cast<const E*>(reinterpret_cast<const char*>(base) + off));
        } else {
            const __amdgpu_buffer_rsrc_t b = tile_rsrc(base);
#pragma unroll
            for (int i = 0; i < KS; ++i)
                if (l.q * KS + i < a.states) rsrc_load(b, off, i * sizeof(E), x.e[i]);
        }
    }
    __device__ __forceinline__ void get(float (&v)[KS]) const
    {
#pragma unroll
        for (int i = 0; i < KS; ++i) v[i] = T::load(x.e[i]);
    }
};

// The inputs of a tile as this lane loads them.
template <typename T, int KS, bool EMIT>
struct Tile {
    LaneRows<T> ru, rd, rz;
    typename T::store_t u[4], dl[4], z[4];
    LaneBC<T, KS> B, C;

    __device__ __forceinline__ void init(const ScanArgs& a, const Lane& l, int64_t s,
                                         int64_t first)
    {
        ru.init(a.u, l, s, a.q, first);
        rd.init(a.delta, l, s, a.q, first);
        B.init(a, a.B, l, s, first);
        if (!EMIT) return;
        rz.init(a.z, l, s, a.q, first);
        C.init(a, a.C, l, s, first);
    }
    __device__ __forceinline__ void load(const ScanArgs& a, const Lane& l, int32_t len, bool gate)
    {
        ru.load(a.u, l, len, u);
        rd.load(a.delta, l, len, dl);
        if (EMIT && gate) rz.load(a.z, l, len, z);
        B.load(a, l, len);
        if (EMIT) C.load(a, l, len);
        ru.next();
        rd.next();
        B.next();
        if (!EMIT) return;
        rz.next();
        C.next();
    }
};

// dl of a lane's four rows.
template <typename T>
__device__ __forceinline__ void step_sizes(const ScanArgs& a, const typename T::store_t (&x)[4],
                                           float bias, float (&raw)[4], float (&dl)[4])
{
#pragma unroll
    for (int r = 0; r < 4; ++r) dl[r] = raw[r] = T::load(x[r]) + bias;
    if (a.softplus)
#pragma unroll
        for (int r = 0; r < 4; ++r) dl[r] = softplus_f<T>(raw[r]);
}

// sum over i of lane T's b[i] (of each row of 16 lanes) times x[i], as one
// product and KS - 1 FMAs that take b through DPP; the compiler would broadcast
// each b[i] by an instruction of its own.  DPP and lane swaps read a register
// only two wait states after a vector instruction wrote it, and the compiler
// does not see into these blocks: the first s_nop is for a b[i] written just
// before, the last for a user of the result.  (Every block of this kind here
// and in the backward pass opens and closes so.)
template <int T, int KS>
__device__ __forceinline__ float bcast_dot(const float (&b)[KS], const float (&x)[KS])
{
    float y;
    if constexpr (KS == 4)
        asm("s_nop 1\n\t"
            "v_mul_f32_dpp %0, %1, %5 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %2, %6 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %3, %7 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %4, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
            "s_nop 1"
            : "=&v"(y)
            : "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "v"(x[0]), "v"(x[1]), "v"(x[2]),
              "v"(x[3]), "n"(T));
    else if constexpr (KS == 2)
        asm("s_nop 1\n\t"
            "v_mul_f32_dpp %0, %1, %3 row_newbcast:%5 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %0, %2, %4 row_newbcast:%5 row_mask:0xf bank_mask:0xf\n\t"
            "s_nop 1"
            : "=&v"(y)
            : "v"(b[0]), "v"(b[1]), "v"(x[0]), "v"(x[1]), "n"(T));
    else
        y = row_bcast<T>(b[0]) * x[0];
    return y;
}

// One step of the recurrence for row T of the tile; x = dl, dl u.
template <int KS, int MODE, int T>
__device__ __forceinline__ float scan_row(const float2 x, const float (&A2)[KS],
                                          const float (&B)[KS], const float (&C)[KS],
                                          float (&h)[KS], float (&S)[KS], float& sdl)
{
    if (MODE != kEmit) sdl += x.x;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const float e = exp2_hw(x.x * A2[i]);
        const float b = row_bcast<T>(B[i]) * x.y;
        if (MODE != kEmit) S[i] = fma32(e, S[i], b);
        if (MODE != kSum) h[i] = fma32(e, h[i], b);
        if (MODE == kSeq) pin(S[i]);
    }
    if (MODE == kSeq) pin(sdl);
    return MODE != kSum ? bcast_dot<T, KS>(C, h) : 0.f;
}

// Rows 4 R .. 4 R + 3 of the tile, whose values x are in registers; the next
// four are read from LDS meanwhile.
template <int KS, int MODE, int R>
__device__ __forceinline__ void scan_rows4(const float2 (*ex)[16], int c, float2 (&x)[4],
                                           const float (&A2)[KS], const float (&B)[KS],
                                           const float (&C)[KS], float (&h)[KS], float (&S)[KS],
                                           float& sdl, float (&yr)[4])
{
    float2 nx[4];
    if constexpr (R < 3)
#pragma unroll
        for (int k = 0; k < 4; ++k) nx[k] = ex[4 * R + 4 + k][c];
    const float y0 = scan_row<KS, MODE, 4 * R + 0>(x[0], A2, B, C, h, S, sdl);
    const float y1 = scan_row<KS, MODE, 4 * R + 1>(x[1], A2, B, C, h, S, sdl);
    const float y2 = scan_row<KS, MODE, 4 * R + 2>(x[2], A2, B, C, h, S, sdl);
    const float y3 = scan_row<KS, MODE, 4 * R + 3>(x[3], A2, B, C, h, S, sdl);
    if (MODE != kSum) yr[R] = fold_quad(y0, y1, y2, y3);
    if constexpr (R < 3)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = nx[k];
}

template <int KS>
struct alignas(KS * 4) StateVec {
    float e[KS];
};

template <int KS>
__device__ __forceinline__ void ld_states(const float* p, float (&v)[KS])
{
    const StateVec<KS> x = *reinterpret_cast<const StateVec<KS>*>(p);
#pragma unroll
    for (int i = 0; i < KS; ++i) v[i] = x.e[i];
}

template <int KS>
__device__ __forceinline__ void st_states(float* p, const float (&v)[KS])
{
    StateVec<KS> x;
#pragma unroll
    for (int i = 0; i < KS; ++i) x.e[i] = v[i];
    *reinterpret_cast<StateVec<KS>*>(p) = x;
}

// log2(e) A.  Minus infinity becomes the lowest finite value: the same
// exponential, 0, of any step size above zero, and 1 of the rows past the end,
// whose step size is 0.
__device__ __forceinline__ float decay_rate(float A)
{
    const float x = A * kLog2e;
    return x < -kMaxF ? -kMaxF : x;
}

// A chunk's effect on the state that enters it: 2^x H + S, x = log2(e) A sum dl.
// A zero state stays S where 2^x overflows (A above zero).
__device__ __forceinline__ float next_state(float x, float H, float S)
{
    return H == 0.f ? S : fma32(exp2_hw(x), H, S);
}

template <typename T, int KS, int MODE>
__global__ __launch_bounds__(256, 4) void k_selective_scan(ScanArgs a)
{
    constexpr int NP = 4 * KS;
    __shared__ float2 ex_all[4][kSub][16];
    const int slabs = a.slabs * (a.channels / a.dg);
    const int64_t slot_id = blockIdx.x / slabs;
    const Lane l = lane_place(a, (int)(blockIdx.x - slot_id * slabs));
    if (l.wch >= a.dg) return;
    float2(*ex)[16] = ex_all[threadIdx.x >> 6];

    int64_t s, slot = slot_id;  // the sequence, and the slot of its chunk
    int32_t lo, hi;             // rows of the sequence
    Span span;
    if (MODE == kSeq) {
        s = slot_id;
        span = uniform(seq_span(a.q, s));
        slot = uniform(slot_base<kCh>(a.q, s));
        lo = 0;
        hi = span.len;
    } else {
        const Chunk ck = wave_slot_chunk<kCh>(a.q, slot);
        if (ck.len <= 0) return;
        s = ck.s;
        span = ck.span;
        lo = ck.row;
        hi = ck.row + ck.len;
    }

    float A2[KS], h[KS], S[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const int n = l.q * KS + i;
        A2[i] = n < a.states ? decay_rate(a.A[(int64_t)l.ch * a.states + n]) : 0.f;
        h[i] = 0.f;
        S[i] = 0.f;
        if (MODE == kSeq && a.init && n < a.states)
            h[i] = a.init[(s * a.channels + l.ch) * a.states + n];
    }
    const float bias = a.bias ? a.bias[l.ch] : 0.f;
    const float Dc = MODE != kSum && a.D ? a.D[l.ch] : 0.f;
    const bool gate = a.z.p != nullptr;
    if (MODE == kEmit)
        ld_states<KS>(a.ws_state + (slot * a.channels + l.ch) * NP + l.q * KS, h);
    float H[KS];  // the chunk's start state
#pragma unroll
    for (int i = 0; i < KS; ++i) H[i] = h[i];

    Tile<T, KS, MODE != kSum> tile;
    tile.init(a, l, s, span.first + lo);
    LaneRows<T> ro;
    ro.init(a.out, l, s, a.q, span.first + lo);
    if (lo < hi) tile.load(a, l, hi - lo, gate);
    float sdl = 0.f;
#pragma unroll 1
    for (int32_t row = lo; row < hi; row += kSub) {
        const int32_t len = hi - row;
        const int sub = row / kSub % kSubs;
        float u[4], dl[4], raw[4], dlu[4], gz[4], B[KS], C[KS];
        step_sizes<T>(a, tile.dl, bias, raw, dl);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            u[r] = T::load(tile.u[r]);
            dlu[r] = dl[r] * u[r];
        }
        if (len < kSub)  // rows past the end: exp(0) = 1 and nothing added
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (4 * r + l.q >= len) dl[r] = dlu[r] = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) ex[4 * r + l.q][l.c] = make_float2(dl[r], dlu[r]);
        if (MODE != kSum && gate)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float z = T::load(tile.z[r]);
                gz[r] = silu_f(z, sigmoid_f<T>(z));
            }
        tile.B.get(B);
        if (MODE != kSum) tile.C.get(C);
        wave_lds_fence();
        if (MODE != kSum && a.cs && l.active)
            st_states<KS>(a.cs + ((slot * kSubs + sub) * a.channels + l.ch) * NP + l.q * KS, h);
        // the next tile's loads, in flight while this one is computed
        if (len > kSub) tile.load(a, l, len - kSub, gate);

        float y[4];
        float2 x[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = ex[k][l.c];
        scan_rows4<KS, MODE, 0>(ex, l.c, x, A2, B, C, h, S, sdl, y);
        scan_rows4<KS, MODE, 1>(ex, l.c, x, A2, B, C, h, S, sdl, y);
        scan_rows4<KS, MODE, 2>(ex, l.c, x, A2, B, C, h, S, sdl, y);
        scan_rows4<KS, MODE, 3>(ex, l.c, x, A2, B, C, h, S, sdl, y);
        wave_lds_fence();
        if (MODE != kSum) {
#pragma unroll
            for (int r = 0; r < 4; ++r) y[r] = fma32(Dc, u[r], y[r]);
            if (gate)
#pragma unroll
                for (int r = 0; r < 4; ++r) y[r] *= gz[r];
            ro.store(l, len, y);
            ro.next();
        }
        if (MODE == kSeq && (sub == kSubs - 1 || len <= kSub)) {
#pragma unroll
            for (int i = 0; i < KS; ++i) {  // the next chunk's start state
                H[i] = next_state(sdl * A2[i], H[i], S[i]);
                h[i] = H[i];
                S[i] = 0.f;
            }
            sdl = 0.f;
            ++slot;
        }
    }
    if (!l.active) return;
    if (MODE == kSum) {
        st_states<KS>(a.ws_state + (slot * a.channels + l.ch) * NP + l.q * KS, S);
        if (l.q == 0) a.ws_dl[slot * a.channels + l.ch] = sdl;
    }
    if (MODE == kSeq && a.final) {
#pragma unroll
        for (int i = 0; i < KS; ++i)
            if (l.q * KS + i < a.states)
                a.final[(s * a.channels + l.ch) * a.states + l.q * KS + i] = h[i];
    }
}

// The states between chunks, one thread per (sequence, channel, state):
// carry <- exp(A sum dl) carry + S over the chunks in order, each chunk's S in
// the workspace replaced by the carry that enters it.  REV: from the last
// chunk to the first, for the gradient (S: the chunk's backward fold).  The
// chain is one FMA per chunk; the loads of the next chunks are in flight while
// the carry passes through these.  Workgroups of one wave, so that few states
// spread over all compute units.
template <int NP, bool REV>
__global__ __launch_bounds__(64) void k_scan_carry(ScanArgs a, const float* __restrict__ first,
                                                   float* __restrict__ last)
{
    const int64_t dn = (int64_t)a.channels * NP;
    const int64_t per = (dn + 63) / 64;
    const int64_t s = blockIdx.x / per;
    const int64_t i = (blockIdx.x - s * per) * 64 + threadIdx.x;
    if (i >= dn) return;
    const int64_t d = i / NP;
    const int n = (int)(i - d * NP);
    const bool real = n < a.states;
    const Span span = uniform(seq_span(a.q, s));
    const int64_t base = uniform(slot_base<kCh>(a.q, s));
    const int32_t chunks = (span.len + kCh - 1) / kCh;
    const float A2 = real ? decay_rate(a.A[d * a.states + n]) : 0.f;
    const int64_t own = (s * a.channels + d) * a.states + n;
    float carry = first && real ? first[own] : 0.f;
    constexpr int U = 16;
    const int64_t step = REV ? -1 : 1;
    const int64_t at = base + (REV ? chunks - 1 : 0);
    float* state = a.ws_state + at * dn + i;  // the next chunk to store
    const float* ps = state;                  // the next to load
    const float* pd = a.ws_dl + at * a.channels + d;
    float S[2][U], P[2][U];
    auto load = [&](int b, int32_t k0) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            S[b][j] = *ps;
            P[b][j] = *pd;
            if (k0 + j + 1 < chunks) {
                ps += step * dn;
                pd += step * a.channels;
            }
        }
    };
    auto pass = [&](int b, int32_t k0) {
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k0 + j >= chunks) break;
            *state = carry;
            state += step * dn;
            carry = next_state(P[b][j] * A2, carry, S[b][j]);
        }
    };
    if (chunks > 0) {
        load(0, 0);
        for (int32_t k0 = 0; k0 < chunks; k0 += 2 * U) {
            if (k0 + U < chunks) load(1, k0 + U);
            pass(0, k0);
            if (k0 + 2 * U < chunks) load(0, k0 + 2 * U);
            pass(1, k0 + U);
        }
    }
    if (last && real) last[own] = carry;
}

template <int NP, bool REV>
hipError_t launch_scan_carry(const ScanArgs& a, const float* first, float* last, hipStream_t st)
{
    const int64_t per = ((int64_t)a.channels * NP + 63) / 64;
    if (a.q.seqs * per == 0) return hipSuccess;
    k_scan_carry<NP, REV><<<dim3((unsigned)(a.q.seqs * per)), dim3(64), 0, st>>>(a, first, last);
    return hipGetLastError();
}

// One row of each sequence: a lane holds KS states of a channel and four
// neighbouring lanes a channel, so a wave's state accesses are contiguous; the
// state is read and written once, which is nearly all of the traffic.  A thread
// takes SEQS sequences, all their loads in flight together.
template <typename T, int KS, int SEQS>
__global__ __launch_bounds__(256) void k_selective_scan_step(ScanArgs a)
{
    const int slabs = a.slabs * (a.channels / a.dg);
    const int64_t part = blockIdx.x / slabs;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int slab = (int)(blockIdx.x - part * slabs);
    Lane l{};
    l.g = slab / a.slabs;
    l.q = lane & 3;
    const int32_t in_g = (slab - l.g * a.slabs) * kSlab + w * 16 + (lane >> 2);
    if (in_g >= a.dg) return;  // whole groups of four lanes
    const int32_t ch = l.g * a.dg + in_g;
    const int64_t s0 = part * SEQS;
    const int seqs = a.q.seqs - s0 < SEQS ? (int)(a.q.seqs - s0) : SEQS;
    const int64_t at = ch * (int64_t)a.states + l.q * KS;
    const int64_t per = (int64_t)a.channels * a.states;
    const bool gate = a.z.p != nullptr;

    typename T::store_t u[SEQS], dl[SEQS], z[SEQS];
    LaneBC<T, KS> B[SEQS], C[SEQS];
    float h[SEQS][KS], A2[KS];
#pragma unroll
    for (int j = 0; j < SEQS; ++j) {
        const int64_t s = s0 + (j < seqs ? j : 0);
        u[j] = static_cast<typename T::store_t*>(a.u.p)[s * a.u.seq + ch];
        dl[j] = static_cast<typename T::store_t*>(a.delta.p)[s * a.delta.seq + ch];
        if (gate) z[j] = static_cast<typename T::store_t*>(a.z.p)[s * a.z.seq + ch];
        B[j].init(a, a.B, l, s, 0);
        C[j].init(a, a.C, l, s, 0);
        B[j].load(a, l, 1);
        C[j].load(a, l, 1);
#pragma unroll
        for (int i = 0; i < KS; ++i) h[j][i] = 0.f;
        if (a.init) {
            if (a.st_vec) {
                ld_states<KS>(a.init + s * per + at, h[j]);
            } else {
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    if (l.q * KS + i < a.states) h[j][i] = a.init[s * per + at + i];
            }
        }
    }
    if (a.st_vec) {
        ld_states<KS>(a.A + at, A2);
    } else {
#pragma unroll
        for (int i = 0; i < KS; ++i) A2[i] = l.q * KS + i < a.states ? a.A[at + i] : 0.f;
    }
#pragma unroll
    for (int i = 0; i < KS; ++i) A2[i] = decay_rate(A2[i]);
    const float bias = a.bias ? a.bias[ch] : 0.f, Dc = a.D ? a.D[ch] : 0.f;
#pragma unroll
    for (int j = 0; j < SEQS; ++j) {
        if (j >= seqs) break;
        const int64_t s = s0 + j;
        const float x = T::load(u[j]), raw = T::load(dl[j]) + bias;
        const float d = a.softplus ? softplus_f<T>(raw) : raw;
        const float du = d * x;
        float b[KS], c[KS], y = 0.f;
        B[j].get(b);
        C[j].get(c);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            h[j][i] = fma32(exp2_hw(d * A2[i]), h[j][i], b[i] * du);
            y = i == 0 ? c[i] * h[j][i] : fma32(c[i], h[j][i], y);
        }
        if (a.final) {
            if (a.st_vec) {
                st_states<KS>(a.final + s * per + at, h[j]);
            } else {
#pragma unroll
                for (int i = 0; i < KS; ++i)
                    if (l.q * KS + i < a.states) a.final[s * per + at + i] = h[j][i];
            }
        }
        y += dpp<0xb1>(y);  // lanes of the channel: neighbour, then pair
        y += dpp<0x4e>(y);
        y = fma32(Dc, x, y);
        if (gate) {
            const float zz = T::load(z[j]);
            y *= silu_f(zz, sigmoid_f<T>(zz));
        }
        if (l.q == 0) static_cast<typename T::store_t*>(a.out.p)[s * a.out.seq + ch] = T::round(y);
    }
}

// ---------------------------------------------------------------------- launches
// Whole sequences take one exponential per value instead of two, but need
// enough of them: a workgroup holds 64 channels of one, and 256 compute units
// fill in steps.  Measured for 1024 rows of 4096 channels (bf16, 16 states), in
// us, at 64, 128, 192, 256, 320, 384, 512, 576, 1024 workgroups: whole 123, 124,
// 124, 123, 177, 179, 180, 242, 310; in chunks 47, 78, 106, 132, 162, 187, 242,
// 273, 470; and in the same proportion for 256 rows (34 and 22 at 64 workgroups,
// 48 and 79 at 512).  float32 and 8 or 4 states change sides within 64 workgroups of
// that: the other way would at most save 10% (4 states at 256: whole 77, in chunks
// 70).  Packed sequences' lengths are not known here.
inline bool scan_whole_sequences(const ScanArgs& a, int64_t slabs)
{
    const int64_t w = a.q.seqs * slabs;
    if (a.q.rows <= kShortRows) return true;
    return a.q.starts == nullptr && 60 + 62 * ((w + 255) / 256) <= 18 + w * 57 / 128;
}

template <typename T, int KS>
hipError_t launch_scan_ks(const ScanArgs& a, int64_t groups, hipStream_t st)
{
    const int64_t slabs = groups * a.slabs;
    if (scan_whole_sequences(a, slabs)) {
        k_selective_scan<T, KS, kSeq><<<dim3((unsigned)(a.q.seqs * slabs)), dim3(256), 0, st>>>(a);
        return hipGetLastError();
    }
    const int64_t slots = slot_count<kCh>(a.q.seqs, a.q.rows, a.q.starts != nullptr);
    const unsigned grid = (unsigned)(slots * slabs);
    k_selective_scan<T, KS, kSum><<<dim3(grid), dim3(256), 0, st>>>(a);
    if (hipError_t e = hipGetLastError()) return e;
    if (hipError_t e = launch_scan_carry<4 * KS, false>(a, a.init, a.final, st)) return e;
    k_selective_scan<T, KS, kEmit><<<dim3(grid), dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_selective_scan(const ScanArgs& a, int64_t groups, hipStream_t st)
{
    switch (scan_ks(a.states)) {
        case 1: return launch_scan_ks<T, 1>(a, groups, st);
        case 2: return launch_scan_ks<T, 2>(a, groups, st);
        default: return launch_scan_ks<T, 4>(a, groups, st);
    }
}

template <typename T, int KS>
hipError_t launch_scan_step_ks(const ScanArgs& a, int64_t groups, hipStream_t st)
{
    const int64_t slabs = groups * a.slabs;
    // Four sequences a thread once that still gives every compute unit several
    // workgroups.  4096 channels, 16 states, bf16: 256 sequences (16384 workgroups
    // of one each) 34 us with one, 26 with four, 5.6 TB/s; 127 with one 15.3, 128
    // with four 14.4.
    if (a.q.seqs * slabs >= 8192)
        k_selective_scan_step<T, KS, 4>
            <<<dim3((unsigned)((a.q.seqs + 3) / 4 * slabs)), dim3(256), 0, st>>>(a);
    else
        k_selective_scan_step<T, KS, 1><<<dim3((unsigned)(a.q.seqs * slabs)), dim3(256), 0, st>>>(a);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_selective_scan_step(const ScanArgs& a, int64_t groups, hipStream_t st)
{
    switch (scan_ks(a.states)) {
        case 1: return launch_scan_step_ks<T, 1>(a, groups, st);
        case 2: return launch_scan_step_ks<T, 2>(a, groups, st);
        default: return launch_scan_step_ks<T, 4>(a, groups, st);
    }
}

}  // namespace seq
}  // namespace canon
