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
// Per (row, channel, state) that is 2 multiplications, 1 exponential (two
// issue slots) and 2 FMAs, so the kernel is bound by vector issue: a pass
// without recomputation needs 6 slots of 4 cycles for 64 lanes.
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

// B or C of one sequence row, this lane's states (0 beyond the last one).
template <typename T, int KS>
__device__ __forceinline__ void load_bc(const ScanArgs& a, const typename T::store_t* p, int q,
                                        bool valid, float (&v)[KS])
{
    if (a.bc_vec) {
        Vec<T, KS> x{};
        if (q * KS < a.states) x = ld_vec<T, KS>(p + q * KS);
#pragma unroll
        for (int i = 0; i < KS; ++i) v[i] = valid ? T::load(x.e[i]) : 0.f;
    } else {
#pragma unroll
        for (int i = 0; i < KS; ++i)
            v[i] = valid && q * KS + i < a.states ? ld<T>(p + q * KS + i) : 0.f;
    }
}

// The inputs of a tile as this lane loads them: rows 4 r + q of its channel,
// and B and C of row c.
template <typename T, int KS, bool EMIT>
struct Tile {
    typename T::store_t u[4], dl[4], z[4];
    float B[KS], C[KS];

    __device__ __forceinline__ void load(const ScanArgs& a, const Lane& l, int64_t s,
                                         const Span& span, int32_t row, int32_t len, bool gate)
    {
        // rows past the sequence's end are read as its last row and not used
        const typename T::store_t* pu = rows_ptr<T>(a.u, s, a.q, span.first + row) + l.ch;
        const typename T::store_t* pd = rows_ptr<T>(a.delta, s, a.q, span.first + row) + l.ch;
        const typename T::store_t* pz =
            gate ? rows_ptr<T>(a.z, s, a.q, span.first + row) + l.ch : nullptr;
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int64_t t = 4 * r + l.q < len ? 4 * r + l.q : len - 1;
            u[r] = pu[t * a.u.row];
            dl[r] = pd[t * a.delta.row];
            if (EMIT && gate) z[r] = pz[t * a.z.row];
        }
        const int64_t t = l.c < len ? l.c : len - 1;
        load_bc<T, KS>(a,
                       rows_ptr<T>(a.B, s, a.q, span.first + row + t) + (int64_t)l.g * a.states,
                       l.q, l.c < len, B);
        if (EMIT)
            load_bc<T, KS>(
                a, rows_ptr<T>(a.C, s, a.q, span.first + row + t) + (int64_t)l.g * a.states, l.q,
                l.c < len, C);
    }
};

// One step of the recurrence for row T of the tile.
template <int KS, int MODE, int T>
__device__ __forceinline__ void scan_row(const float2 (*ex)[16], int c, const float (&A2)[KS],
                                         const float (&B)[KS], const float (&C)[KS],
                                         float (&h)[KS], float (&S)[KS], float& sdl,
                                         float (&y)[4])
{
    const float2 x = ex[T][c];  // dl, dl u
    if (MODE != kEmit) sdl += x.x;
    float acc = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const float e = exp2_hw(x.x * A2[i]);
        const float b = row_bcast<T>(B[i]) * x.y;
        if (MODE != kEmit) S[i] = fma32(e, S[i], b);
        if (MODE != kSum) {
            h[i] = fma32(e, h[i], b);
            acc = i == 0 ? row_bcast<T>(C[i]) * h[i] : fma32(row_bcast<T>(C[i]), h[i], acc);
        }
    }
    if (MODE != kSum) y[T & 3] = acc;
}

template <int KS, int MODE, int R>
__device__ __forceinline__ void scan_rows4(const float2 (*ex)[16], int c, const float (&A2)[KS],
                                           const float (&B)[KS], const float (&C)[KS],
                                           float (&h)[KS], float (&S)[KS], float& sdl,
                                           float (&yr)[4])
{
    float y[4];
    scan_row<KS, MODE, 4 * R + 0>(ex, c, A2, B, C, h, S, sdl, y);
    scan_row<KS, MODE, 4 * R + 1>(ex, c, A2, B, C, h, S, sdl, y);
    scan_row<KS, MODE, 4 * R + 2>(ex, c, A2, B, C, h, S, sdl, y);
    scan_row<KS, MODE, 4 * R + 3>(ex, c, A2, B, C, h, S, sdl, y);
    if (MODE != kSum) yr[R] = fold_quad(y[0], y[1], y[2], y[3]);
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

template <typename T, int KS, int MODE>
__global__ __launch_bounds__(256) void k_selective_scan(ScanArgs a)
{
    constexpr int NP = 4 * KS;
    __shared__ float2 ex_all[4][kSub][16];
    const int slabs = a.slabs * (a.channels / a.dg);
    const int64_t slot_id = blockIdx.x / slabs;
    const Lane l = lane_place(a, (int)(blockIdx.x - slot_id * slabs));
    if (l.wch >= a.dg) return;
    float2(*ex)[16] = ex_all[threadIdx.x >> 6];

    Chunk ck;
    int64_t slot = slot_id;
    if (MODE == kSeq) {
        ck.s = slot_id;
        ck.span = seq_span(a.q, ck.s);
        slot = slot_base<kCh>(a.q, ck.s);
        ck.row = 0;
        ck.len = ck.span.len < kCh ? ck.span.len : kCh;
    } else {
        ck = slot_chunk<kCh>(a.q, slot);
        if (ck.len <= 0) return;
    }

    float A2[KS], h[KS], S[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const int n = l.q * KS + i;
        A2[i] = n < a.states ? a.A[(int64_t)l.ch * a.states + n] * kLog2e : 0.f;
        h[i] = 0.f;
        S[i] = 0.f;
        if (MODE == kSeq && a.init && n < a.states)
            h[i] = a.init[(ck.s * a.channels + l.ch) * a.states + n];
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
    if (ck.len > 0) tile.load(a, l, ck.s, ck.span, ck.row, ck.len, gate);
    float sdl = 0.f;
    while (ck.len > 0) {
        typename T::store_t* po =
            MODE != kSum ? rows_ptr<T>(a.out, ck.s, a.q, ck.span.first + ck.row) + l.ch : nullptr;
        for (int sub = 0; sub * kSub < ck.len; ++sub) {
            const int32_t row = ck.row + sub * kSub, len = ck.len - sub * kSub;
            float u[4], z[4], B[KS], C[KS];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const bool valid = 4 * r + l.q < len;
                u[r] = T::load(tile.u[r]);
                if (MODE != kSum && gate) z[r] = T::load(tile.z[r]);
                const float raw = T::load(tile.dl[r]) + bias;
                const float d = a.softplus ? softplus_f(raw, nullptr) : raw;
                // a row past the end: exp(0) = 1 and nothing added
                ex[4 * r + l.q][l.c] = valid ? make_float2(d, d * u[r]) : make_float2(0.f, 0.f);
            }
#pragma unroll
            for (int i = 0; i < KS; ++i) {
                B[i] = tile.B[i];
                if (MODE != kSum) C[i] = tile.C[i];
            }
            wave_lds_fence();
            if (MODE != kSum && a.cs && l.active)
                st_states<KS>(a.cs + ((slot * kSubs + sub) * a.channels + l.ch) * NP + l.q * KS, h);
            // the next tile's loads, in flight while this one is computed
            const int32_t left = ck.span.len - row - kSub;
            if (left > 0 && (MODE == kSeq || sub + 1 < kSubs))
                tile.load(a, l, ck.s, ck.span, row + kSub, left, gate);

            float yr[4];
            scan_rows4<KS, MODE, 0>(ex, l.c, A2, B, C, h, S, sdl, yr);
            scan_rows4<KS, MODE, 1>(ex, l.c, A2, B, C, h, S, sdl, yr);
            scan_rows4<KS, MODE, 2>(ex, l.c, A2, B, C, h, S, sdl, yr);
            scan_rows4<KS, MODE, 3>(ex, l.c, A2, B, C, h, S, sdl, yr);
            wave_lds_fence();
            if (MODE != kSum) {
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    float y = fma32(Dc, u[r], yr[r]);
                    if (gate) y *= silu_f(z[r], sigmoid_f(z[r]));
                    if (l.active && 4 * r + l.q < len)
                        st<T>(po + (int64_t)(sub * kSub + 4 * r + l.q) * a.out.row, y);
                }
            }
        }
        if (MODE != kSeq) break;
#pragma unroll
        for (int i = 0; i < KS; ++i) {  // the next chunk's start state
            H[i] = fma32(exp2_hw(sdl * A2[i]), H[i], S[i]);
            h[i] = H[i];
            S[i] = 0.f;
        }
        sdl = 0.f;
        ++slot;
        ck.row += kCh;
        ck.len = ck.span.len - ck.row < kCh ? ck.span.len - ck.row : kCh;
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
                a.final[(ck.s * a.channels + l.ch) * a.states + l.q * KS + i] = h[i];
    }
}

// The states between chunks, one thread per (sequence, channel, state):
// carry <- exp(A sum dl) carry + S over the chunks in order, each chunk's S in
// the workspace replaced by the carry that enters it.  REV: from the last
// chunk to the first, for the gradient (S: the chunk's backward fold).
template <int NP, bool REV>
__global__ __launch_bounds__(256) void k_scan_carry(ScanArgs a, const float* __restrict__ first,
                                                    float* __restrict__ last)
{
    const int64_t dn = (int64_t)a.channels * NP;
    const int64_t per = (dn + 255) / 256;
    const int64_t s = blockIdx.x / per;
    const int64_t i = (blockIdx.x - s * per) * 256 + threadIdx.x;
    if (i >= dn) return;
    const int64_t d = i / NP;
    const int n = (int)(i - d * NP);
    const bool real = n < a.states;
    const Span span = seq_span(a.q, s);
    const int64_t chunks = (span.len + kCh - 1) / kCh, base = slot_base<kCh>(a.q, s);
    const float A2 = real ? a.A[d * a.states + n] * kLog2e : 0.f;
    const int64_t own = (s * a.channels + d) * a.states + n;
    float carry = first && real ? first[own] : 0.f;
    constexpr int U = 8;
    for (int64_t k0 = 0; k0 < chunks; k0 += U) {
        float S[U], P[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int64_t k = k0 + j < chunks ? k0 + j : chunks - 1;
            const int64_t slot = base + (REV ? chunks - 1 - k : k);
            S[j] = a.ws_state[slot * dn + i];
            P[j] = exp2_hw(a.ws_dl[slot * a.channels + d] * A2);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (k0 + j >= chunks) break;
            const int64_t slot = base + (REV ? chunks - 1 - k0 - j : k0 + j);
            a.ws_state[slot * dn + i] = carry;
            carry = fma32(P[j], carry, S[j]);
        }
    }
    if (last && real) last[own] = carry;
}

template <int NP, bool REV>
hipError_t launch_scan_carry(const ScanArgs& a, const float* first, float* last, hipStream_t st)
{
    const int64_t per = ((int64_t)a.channels * NP + 255) / 256;
    if (a.q.seqs * per == 0) return hipSuccess;
    k_scan_carry<NP, REV><<<dim3((unsigned)(a.q.seqs * per)), dim3(256), 0, st>>>(a, first, last);
    return hipGetLastError();
}

// One row of each sequence: a lane holds KS states of a channel and four rows
// of lanes a channel, as above; the state is read and written once, which is
// nearly all of the traffic.
template <typename T, int KS>
__global__ __launch_bounds__(256) void k_selective_scan_step(ScanArgs a)
{
    const int slabs = a.slabs * (a.channels / a.dg);
    const int64_t s = blockIdx.x / slabs;
    // states of a channel in neighbouring lanes, so a wave's state accesses are
    // contiguous: q = lane mod 4 here
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int slab = (int)(blockIdx.x - s * slabs);
    const int g = slab / a.slabs, q = lane & 3;
    const int32_t in_g = (slab - g * a.slabs) * kSlab + w * 16 + (lane >> 2);
    if (in_g >= a.dg) return;  // whole groups of four lanes
    const int32_t ch = g * a.dg + in_g;

    const float u = ld<T>(static_cast<typename T::store_t*>(a.u.p) + s * a.u.seq + ch);
    float raw = ld<T>(static_cast<typename T::store_t*>(a.delta.p) + s * a.delta.seq + ch);
    if (a.bias) raw += a.bias[ch];
    const float d = a.softplus ? softplus_f(raw, nullptr) : raw;
    const float du = d * u;
    float B[KS], C[KS];
    const int64_t gb = (int64_t)g * a.states;
    load_bc<T, KS>(a, static_cast<typename T::store_t*>(a.B.p) + s * a.B.seq + gb, q, true, B);
    load_bc<T, KS>(a, static_cast<typename T::store_t*>(a.C.p) + s * a.C.seq + gb, q, true, C);
    const int64_t at = (s * a.channels + ch) * a.states + q * KS;
    const bool vec = a.st_vec;
    float h[KS], A2[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) h[i] = 0.f;
    if (vec) {
        ld_states<KS>(a.A + (int64_t)ch * a.states + q * KS, A2);
        if (a.init) ld_states<KS>(a.init + at, h);
    } else {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const bool real = q * KS + i < a.states;
            A2[i] = real ? a.A[(int64_t)ch * a.states + q * KS + i] : 0.f;
            if (a.init && real) h[i] = a.init[at + i];
        }
    }
    float y = 0.f;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        h[i] = fma32(exp2_hw(d * (A2[i] * kLog2e)), h[i], B[i] * du);
        y = i == 0 ? C[i] * h[i] : fma32(C[i], h[i], y);
    }
    if (a.final) {
        if (vec) {
            st_states<KS>(a.final + at, h);
        } else {
#pragma unroll
            for (int i = 0; i < KS; ++i)
                if (q * KS + i < a.states) a.final[at + i] = h[i];
        }
    }
    y += dpp<0xb1>(y);  // lanes of the channel: neighbour, then pair
    y += dpp<0x4e>(y);
    if (q != 0) return;
    if (a.D) y = fma32(a.D[ch], u, y);
    if (a.z.p) {
        const float z = ld<T>(static_cast<typename T::store_t*>(a.z.p) + s * a.z.seq + ch);
        y *= silu_f(z, sigmoid_f(z));
    }
    st<T>(static_cast<typename T::store_t*>(a.out.p) + s * a.out.seq + ch, y);
}

// ---------------------------------------------------------------------- launches
template <typename T, int KS>
hipError_t launch_scan_ks(const ScanArgs& a, int64_t groups, hipStream_t st)
{
    const int64_t slots = slot_count<kCh>(a.q.seqs, a.q.rows, a.q.starts != nullptr);
    const unsigned grid = (unsigned)(slots * groups * a.slabs);
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

template <typename T>
hipError_t launch_selective_scan_step(const ScanArgs& a, int64_t groups, hipStream_t st)
{
    const dim3 grid((unsigned)(a.q.seqs * groups * a.slabs)), block(256);
    switch (scan_ks(a.states)) {
        case 1: k_selective_scan_step<T, 1><<<grid, block, 0, st>>>(a); break;
        case 2: k_selective_scan_step<T, 2><<<grid, block, 0, st>>>(a); break;
        default: k_selective_scan_step<T, 4><<<grid, block, 0, st>>>(a); break;
    }
    return hipGetLastError();
}

}  // namespace seq
}  // namespace canon
