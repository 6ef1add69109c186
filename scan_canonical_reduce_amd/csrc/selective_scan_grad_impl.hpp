// Selective state space scan: backward pass.
//
// With lam[t] the gradient of h[t] and R[t] = a[t+1] lam[t+1] what reaches
// h[t] from later rows,
//   lam = C dy + R,  R[t-1] = a lam,  dy = dout z sigmoid(z)
//   dB[t,n] = sum_d lam dl u      dC[t,n] = sum_d dy h
//   through = sum_n B lam         decay   = R[t-1] h[t-1]  (= a h[t-1] lam)
//   du  = through dl + D dy       ddl = sum_n A decay + through u
//   dA  = sum_t dl decay          dD  = sum_t dy u        dz = dout y silu'(z)
// Three passes over chunks of 64 rows: each chunk's fold of lam from zero,
// backwards; the carries R between chunks; then each chunk with its carry.
// The last pass reads the h that the forward pass saved every 16 rows, keeps
// a and h of 16 rows in registers (lane layout of selective_scan_impl.hpp) and
// walks them backwards.
//
// dB and dC are sums over channels, i.e. across the 16 lanes of a row of
// lanes: sequence rows are folded into lanes two at a time (each level halves
// both the number of values and the lanes a value is spread over: 15 additions
// for 16 values where a plain butterfly takes 64), which leaves lane c with
// sequence row bitrev(c).  The four waves of a workgroup are summed through LDS
// and the workgroups' sums by a second kernel, in slab order.
//
// 8 x 2048 x 4096, 16 states, bf16: 935 us, of which vector instructions issue for
// 70 to 75%; a and h of 16 rows take 240 to 255 registers, so two waves a SIMD.
// Sums over the slabs and chunks: 42 us more.
#pragma once

#include "column_sum.hpp"
#include "selective_scan_impl.hpp"

namespace canon {
namespace seq {

// Inputs of a 16-row tile of the backward passes, loaded as in Tile, from the
// last tile to the first.
template <typename T, int KS, bool MAIN>
struct GradTile {
    LaneRows<T> ru, rd, rz, rg;
    typename T::store_t u[4], dl[4], z[4], go[4];
    LaneBC<T, KS> B, C;

    __device__ __forceinline__ void init(const ScanArgs& a, const Lane& l, int64_t s,
                                         int64_t first)
    {
        if (MAIN) ru.init(a.u, l, s, a.q, first);
        rd.init(a.delta, l, s, a.q, first);
        rz.init(a.z, l, s, a.q, first);
        rg.init(a.dout, l, s, a.q, first);
        if (MAIN) B.init(a, a.B, l, s, first);
        C.init(a, a.C, l, s, first);
    }
    __device__ __forceinline__ void load(const ScanArgs& a, const Lane& l, int32_t len, bool gate)
    {
        if (MAIN) ru.load(a.u, l, len, u);
        rd.load(a.delta, l, len, dl);
        rg.load(a.dout, l, len, go);
        if (gate) rz.load(a.z, l, len, z);
        C.load(a, l, len);
        if (MAIN) B.load(a, l, len);
        if (MAIN) ru.prev();
        rd.prev();
        rg.prev();
        rz.prev();
        C.prev();
        if (MAIN) B.prev();
    }
};

// b[i] of lane T times x, added to y[i]
template <int T, int KS>
__device__ __forceinline__ void bcast_fma(const float (&b)[KS], float x, float (&y)[KS])
{
    if constexpr (KS == 4)
        asm("s_nop 1\n\t"
            "v_fmac_f32_dpp %0, %4, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %1, %5, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %2, %6, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
            "v_fmac_f32_dpp %3, %7, %8 row_newbcast:%9 row_mask:0xf bank_mask:0xf\n\t"
            "s_nop 1"
            : "+v"(y[0]), "+v"(y[1]), "+v"(y[2]), "+v"(y[3])
            : "v"(b[0]), "v"(b[1]), "v"(b[2]), "v"(b[3]), "v"(x), "n"(T));
    else
#pragma unroll
        for (int i = 0; i < KS; ++i) y[i] = fma32(row_bcast<T>(b[i]), x, y[i]);
}

template <int KS, int T>
__device__ __forceinline__ void back_row(const float2 (*ex)[16], int c, const float (&A2)[KS],
                                         const float (&C)[KS], float (&R)[KS], float& sdl)
{
    const float2 x = ex[T][c];  // dl, dy
    sdl += x.x;
    bcast_fma<T, KS>(C, x.y, R);
#pragma unroll
    for (int i = 0; i < KS; ++i) R[i] *= exp2_hw(x.x * A2[i]);
}

template <int KS, int T>
__device__ __forceinline__ void back_rows(const float2 (*ex)[16], int c, const float (&A2)[KS],
                                          const float (&C)[KS], float (&R)[KS], float& sdl)
{
    back_row<KS, T>(ex, c, A2, C, R, sdl);
    if constexpr (T > 0) back_rows<KS, T - 1>(ex, c, A2, C, R, sdl);
}

// Each chunk's backward fold from zero, and its sum of dl.
template <typename T, int KS>
__global__ __launch_bounds__(256) void k_scan_back_sum(ScanArgs a)
{
    constexpr int NP = 4 * KS;
    __shared__ float2 ex_all[4][kSub][16];
    const int slabs = a.slabs * (a.channels / a.dg);
    const int64_t slot = blockIdx.x / slabs;
    const Lane l = lane_place(a, (int)(blockIdx.x - slot * slabs));
    if (l.wch >= a.dg) return;
    float2(*ex)[16] = ex_all[threadIdx.x >> 6];
    const Chunk ck = wave_slot_chunk<kCh>(a.q, slot);
    if (ck.len <= 0) return;

    float A2[KS], R[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const int n = l.q * KS + i;
        A2[i] = n < a.states ? decay_rate(a.A[(int64_t)l.ch * a.states + n]) : 0.f;
        R[i] = 0.f;
    }
    const float bias = a.bias ? a.bias[l.ch] : 0.f;
    const bool gate = a.z.p != nullptr;
    float sdl = 0.f;
    int sub = (ck.len - 1) / kSub;
    GradTile<T, KS, false> tile;
    tile.init(a, l, ck.s, ck.span.first + ck.row + sub * kSub);
    tile.load(a, l, ck.len - sub * kSub, gate);
    for (; sub >= 0; --sub) {
        const int32_t len = ck.len - sub * kSub;
        float C[KS], dl[4], raw[4], dy[4];
        tile.C.get(C);
        step_sizes<T>(a, tile.dl, bias, raw, dl);
#pragma unroll
        for (int r = 0; r < 4; ++r) dy[r] = T::load(tile.go[r]);
        if (gate)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const float z = T::load(tile.z[r]);
                dy[r] *= silu_f(z, sigmoid_f<T>(z));
            }
        if (len < kSub)
#pragma unroll
            for (int r = 0; r < 4; ++r)
                if (4 * r + l.q >= len) dl[r] = dy[r] = 0.f;
#pragma unroll
        for (int r = 0; r < 4; ++r) ex[4 * r + l.q][l.c] = make_float2(dl[r], dy[r]);
        wave_lds_fence();
        if (sub > 0) tile.load(a, l, kSub, gate);
        back_rows<KS, kSub - 1>(ex, l.c, A2, C, R, sdl);
        wave_lds_fence();
    }
    if (!l.active) return;
    st_states<KS>(a.ws_state + (slot * a.channels + l.ch) * NP + l.q * KS, R);
    if (l.q == 0) a.ws_dl[slot * a.channels + l.ch] = sdl;
}

// One level of the sum over a row's 16 lanes, for KS values: a lane without the
// level's bit of c gets x plus the mirrored lane's x, a lane with it y plus the
// mirrored lane's y.  Mirrors over 16 and 8 lanes pair whole banks of four, so
// both sums write their own banks of the result, two instructions a value; below
// that the lanes select first, three instructions, by masks that are constants
// in scalar registers.
#define CANON_FOLD_BANKS(NAME, CTRL, LOWER, UPPER)                                              \
    template <int KS>                                                                           \
    __device__ __forceinline__ void NAME(const float (&x)[KS], const float (&y)[KS],            \
                                         float (&r)[KS])                                        \
    {                                                                                           \
        if constexpr (KS == 4)                                                                  \
            asm("s_nop 1\n\t"                                                                   \
                "v_add_f32_dpp %0, %4, %4 " CTRL " row_mask:0xf bank_mask:" LOWER "\n\t"        \
                "v_add_f32_dpp %1, %5, %5 " CTRL " row_mask:0xf bank_mask:" LOWER "\n\t"        \
                "v_add_f32_dpp %2, %6, %6 " CTRL " row_mask:0xf bank_mask:" LOWER "\n\t"        \
                "v_add_f32_dpp %3, %7, %7 " CTRL " row_mask:0xf bank_mask:" LOWER "\n\t"        \
                "v_add_f32_dpp %0, %8, %8 " CTRL " row_mask:0xf bank_mask:" UPPER "\n\t"        \
                "v_add_f32_dpp %1, %9, %9 " CTRL " row_mask:0xf bank_mask:" UPPER "\n\t"        \
                "v_add_f32_dpp %2, %10, %10 " CTRL " row_mask:0xf bank_mask:" UPPER "\n\t"      \
                "v_add_f32_dpp %3, %11, %11 " CTRL " row_mask:0xf bank_mask:" UPPER "\n\t"      \
                "s_nop 1"                                                                       \
                : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3])                            \
                : "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]), "v"(y[0]), "v"(y[1]), "v"(y[2]),  \
                  "v"(y[3]));                                                                   \
        else                                                                                    \
            for (int i = 0; i < KS; ++i)                                                        \
                asm("s_nop 1\n\t"                                                               \
                    "v_add_f32_dpp %0, %1, %1 " CTRL " row_mask:0xf bank_mask:" LOWER "\n\t"    \
                    "v_add_f32_dpp %0, %2, %2 " CTRL " row_mask:0xf bank_mask:" UPPER "\n\t"    \
                    "s_nop 1"                                                                   \
                    : "=&v"(r[i])                                                               \
                    : "v"(x[i]), "v"(y[i]));                                                    \
    }
CANON_FOLD_BANKS(fold16, "row_mirror", "0x3", "0xc")
CANON_FOLD_BANKS(fold8, "row_half_mirror", "0x5", "0xa")
#undef CANON_FOLD_BANKS

#define CANON_FOLD_SELECT(NAME, CTRL, MASK)                                                     \
    template <int KS>                                                                           \
    __device__ __forceinline__ void NAME(const float (&x)[KS], const float (&y)[KS],            \
                                         float (&r)[KS])                                        \
    {                                                                                           \
        const uint64_t upper = MASK;                                                            \
        float t[KS];                                                                            \
        if constexpr (KS == 4)                                                                  \
            asm("v_cndmask_b32_e64 %4, %12, %8, %16\n\t"                                        \
                "v_cndmask_b32_e64 %5, %13, %9, %16\n\t"                                        \
                "v_cndmask_b32_e64 %6, %14, %10, %16\n\t"                                       \
                "v_cndmask_b32_e64 %7, %15, %11, %16\n\t"                                       \
                "v_cndmask_b32_e64 %0, %8, %12, %16\n\t"                                        \
                "v_cndmask_b32_e64 %1, %9, %13, %16\n\t"                                        \
                "v_cndmask_b32_e64 %2, %10, %14, %16\n\t"                                       \
                "v_cndmask_b32_e64 %3, %11, %15, %16\n\t"                                       \
                "v_add_f32_dpp %0, %4, %0 " CTRL " row_mask:0xf bank_mask:0xf\n\t"              \
                "v_add_f32_dpp %1, %5, %1 " CTRL " row_mask:0xf bank_mask:0xf\n\t"              \
                "v_add_f32_dpp %2, %6, %2 " CTRL " row_mask:0xf bank_mask:0xf\n\t"              \
                "v_add_f32_dpp %3, %7, %3 " CTRL " row_mask:0xf bank_mask:0xf\n\t"              \
                "s_nop 1"                                                                       \
                : "=&v"(r[0]), "=&v"(r[1]), "=&v"(r[2]), "=&v"(r[3]), "=&v"(t[0]), "=&v"(t[1]), \
                  "=&v"(t[2]), "=&v"(t[3])                                                      \
                : "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]), "v"(y[0]), "v"(y[1]), "v"(y[2]),  \
                  "v"(y[3]), "s"(upper));                                                       \
        else                                                                                    \
            for (int i = 0; i < KS; ++i)                                                        \
                asm("v_cndmask_b32_e64 %1, %3, %2, %4\n\t"                                      \
                    "v_cndmask_b32_e64 %0, %2, %3, %4\n\t"                                      \
                    "s_nop 1\n\t"                                                               \
                    "v_add_f32_dpp %0, %1, %0 " CTRL " row_mask:0xf bank_mask:0xf\n\t"          \
                    "s_nop 1"                                                                   \
                    : "=&v"(r[i]), "=&v"(t[i])                                                  \
                    : "v"(x[i]), "v"(y[i]), "s"(upper));                                        \
    }
CANON_FOLD_SELECT(fold4, "quad_perm:[3,2,1,0]", 0xccccccccccccccccull)
CANON_FOLD_SELECT(fold2, "quad_perm:[1,0,3,2]", 0xaaaaaaaaaaaaaaaaull)
#undef CANON_FOLD_SELECT

// Sums over the lanes of a row, sequence rows arriving in descending order T =
// 15 .. 0; v[L] holds what waits for its partner at level L.
template <int KS>
struct LaneSum {
    float wait[4][KS];

    template <int T>
    __device__ __forceinline__ void add(float (&x)[KS])
    {
        if constexpr (T & 1) {
            copy(x, wait[0]);
        } else {
            float a[KS];
            fold16<KS>(x, wait[0], a);
            if constexpr (T & 2) {
                copy(a, wait[1]);
            } else {
                float b[KS];
                fold8<KS>(a, wait[1], b);
                if constexpr (T & 4) {
                    copy(b, wait[2]);
                } else {
                    float d[KS];
                    fold4<KS>(b, wait[2], d);
                    if constexpr (T & 8)
                        copy(d, wait[3]);
                    else
                        fold2<KS>(d, wait[3], x);
                }
            }
        }
    }
    static __device__ __forceinline__ void copy(const float (&x)[KS], float (&y)[KS])
    {
#pragma unroll
        for (int i = 0; i < KS; ++i) y[i] = x[i];
    }
};

// What a lane passes to the other lanes of its channel, per row, and keeps for
// itself until the row's sums are there: three arrays of pairs.
struct GradRows {
    float2 a[kSub][16];  // dl, dl u
    float2 b[kSub][16];  // dy (the gated gradient of y), u
    float2 c[kSub][16];  // d dl / d delta, dout silu'(z)
};

template <int KS>
struct GradRegs {
    float a[kSub][KS], h[kSub + 1][KS];  // h[t]: before row t
    float A2[KS], R[KS], dA[KS], B[KS], C[KS];
    float dBt[KS], dCt[KS];  // the tile's sums, once row 0 is folded
    LaneSum<KS> sb, sc;
    float th[4], dc[4], y[4];
};

template <int KS, int T>
__device__ __forceinline__ void grad_forward(const GradRows& ex, int c, bool gate,
                                             GradRegs<KS>& g, float (&y)[4])
{
    const float dl = ex.a[T][c].x, dlu = ex.a[T][c].y;
    float hn[KS];
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        g.a[T][i] = exp2_hw(dl * g.A2[i]);
        hn[i] = fma32(g.a[T][i], g.h[T][i], row_bcast<T>(g.B[i]) * dlu);
    }
    y[T & 3] = bcast_dot<T, KS>(g.C, hn);
#pragma unroll
    for (int i = 0; i < KS; ++i) g.h[T + 1][i] = hn[i];
    if constexpr ((T & 3) == 3) g.y[T >> 2] = fold_quad(y[0], y[1], y[2], y[3]);
    if constexpr (T + 1 < kSub) grad_forward<KS, T + 1>(ex, c, gate, g, y);
}

// What a row's backward step needs of the other lanes.
struct RowIn {
    float2 a;  // dl, dl u
    float dy;
};

template <int KS, int T>
__device__ __forceinline__ void grad_row(const RowIn& x, int c, GradRegs<KS>& g, float& th,
                                         float& dc)
{
    float b[KS], s[KS], decay = 0.f;
    bcast_fma<T, KS>(g.C, x.dy, g.R);  // lam
    th = bcast_dot<T, KS>(g.B, g.R);
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        b[i] = g.R[i] * x.a.y;
        s[i] = x.dy * g.h[T + 1][i];
        g.R[i] *= g.a[T][i];
        const float d = g.R[i] * g.h[T][i];
        g.dA[i] = fma32(x.a.x, d, g.dA[i]);
        pin(g.dA[i]);
        decay = i == 0 ? g.A2[i] * d : fma32(g.A2[i], d, decay);
    }
    dc = decay;
    g.sb.template add<T>(b);
    g.sc.template add<T>(s);
    if constexpr (T == 0) {
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            g.dBt[i] = b[i];
            g.dCt[i] = s[i];
        }
    }
}

template <int R>
__device__ __forceinline__ void read_rows(const GradRows& ex, int c, RowIn (&x)[4])
{
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[k].a = ex.a[4 * R + k][c];
        x[k].dy = ex.b[4 * R + k][c].x;
    }
}

// Rows 4 R + 3 .. 4 R, whose values x are in registers; the four before them
// are read from LDS meanwhile.
template <int KS, int R>
__device__ __forceinline__ void grad_rows4(const GradRows& ex, int c, RowIn (&x)[4],
                                           GradRegs<KS>& g)
{
    RowIn nx[4];
    if constexpr (R > 0) read_rows<R - 1>(ex, c, nx);
    float th[4], dc[4];
    grad_row<KS, 4 * R + 3>(x[3], c, g, th[3], dc[3]);
    grad_row<KS, 4 * R + 2>(x[2], c, g, th[2], dc[2]);
    grad_row<KS, 4 * R + 1>(x[1], c, g, th[1], dc[1]);
    grad_row<KS, 4 * R + 0>(x[0], c, g, th[0], dc[0]);
    g.th[R] = fold_quad(th[0], th[1], th[2], th[3]);
    g.dc[R] = fold_quad(dc[0], dc[1], dc[2], dc[3]);
    if constexpr (R > 0)
#pragma unroll
        for (int k = 0; k < 4; ++k) x[k] = nx[k];
}

// The partial sums of a slot without rows.
template <int KS>
__device__ __forceinline__ void zero_slot(const ScanArgs& a, const Lane& l, int64_t slot)
{
    const float zero[KS] = {};
    const int64_t at = slot * a.channels + l.ch;
    st_states<KS>(a.ws_state + at * (4 * KS) + l.q * KS, zero);
    if (l.q == 0) {
        a.ws_dD[at] = 0.f;
        a.ws_dbias[at] = 0.f;
    }
}

// One chunk, given the carry R that enters it from later rows (a.ws_state,
// which then takes the chunk's part of dA); or, SEQ, a whole sequence from its
// end, the carry kept in registers.
template <typename T, int KS, bool SEQ>
__global__ __launch_bounds__(256, 2) void k_selective_scan_grad(ScanArgs a)
{
    constexpr int NP = 4 * KS;
    __shared__ GradRows ex_all[4];
    // two buffers: one barrier a tile; rows padded by 16 bytes against bank conflicts
    alignas(16) __shared__ float bc[2][4][kSub][2 * NP + 4];
    const int slabs = a.slabs * (a.channels / a.dg);
    const int64_t id = blockIdx.x / slabs;
    const int slab = (int)(blockIdx.x - id * slabs);
    const Lane l = lane_place(a, slab);
    const int w = uniform((int32_t)(threadIdx.x >> 6));
    GradRows& ex = ex_all[w];
    int64_t s, slot;  // the sequence, and the slot of its chunk (SEQ: the last one)
    int32_t lo, hi;   // rows of the sequence
    Span span;
    if (SEQ) {
        s = id;
        span = uniform(seq_span(a.q, s));
        lo = 0;
        hi = span.len;
        slot = uniform(slot_base<kCh>(a.q, s)) + (hi > 0 ? (hi - 1) / kCh : 0);
    } else {
        slot = id;
        const Chunk ck = wave_slot_chunk<kCh>(a.q, slot);
        s = ck.s;
        span = ck.span;
        lo = ck.row;
        hi = ck.row + ck.len;
    }
    if (SEQ && a.q.starts && l.active) {
        // slots between this sequence's chunks and the next sequence's (the first
        // sequence: also those before it) take no part in the sums: zero
        const int64_t base = uniform(slot_base<kCh>(a.q, s));
        const int64_t end = s + 1 < a.q.seqs ? uniform(slot_base<kCh>(a.q, s + 1))
                                             : slot_count<kCh>(a.q.seqs, a.q.rows, true);
        for (int64_t k = s == 0 ? 0 : base; k < end; ++k)
            if (k < base || k > slot) zero_slot<KS>(a, l, k);
    }
    const int64_t own = ((SEQ ? s : slot) * a.channels + l.ch) * (SEQ ? a.states : NP) + l.q * KS;
    if (hi <= lo) {  // an empty slot: its partial sums are zero
        if (l.active) {
            zero_slot<KS>(a, l, slot);
            if (SEQ && a.dinit)
                for (int i = 0; i < KS; ++i)
                    if (l.q * KS + i < a.states) a.dinit[own + i] = a.dfinal ? a.dfinal[own + i] : 0.f;
        }
        return;
    }

    GradRegs<KS> g;
#pragma unroll
    for (int i = 0; i < KS; ++i) {
        const int n = l.q * KS + i;
        g.A2[i] = n < a.states ? decay_rate(a.A[(int64_t)l.ch * a.states + n]) : 0.f;
        g.R[i] = SEQ && a.dfinal && l.active && n < a.states ? a.dfinal[own + i] : 0.f;
        g.dA[i] = 0.f;
    }
    if (!SEQ && l.active) ld_states<KS>(a.ws_state + own, g.R);
    const float bias = a.bias ? a.bias[l.ch] : 0.f, Dc = a.D ? a.D[l.ch] : 0.f;
    const bool gate = a.z.p != nullptr;
    float dD = 0.f, dbias = 0.f;
    const int brev = (l.c & 1) << 3 | (l.c & 2) << 1 | (l.c & 4) >> 1 | (l.c & 8) >> 3;
    // the rows of the partial sums of dB and dC: packed rows, or sequence by sequence
    const int64_t bc_row = (a.q.starts ? 0 : s * a.q.rows) + span.first;
    const int64_t bc_rows = a.q.starts ? a.q.rows : a.q.seqs * a.q.rows;

    int32_t row = (hi - 1) / kSub * kSub;
    GradTile<T, KS, true> tile;
    tile.init(a, l, s, span.first + row);
    tile.load(a, l, hi - row, gate);
    LaneRows<T> o_du, o_dd, o_dz;
    o_du.init(a.du, l, s, a.q, span.first + row);
    o_dd.init(a.ddelta, l, s, a.q, span.first + row);
    o_dz.init(a.dz, l, s, a.q, span.first + row);
    for (; row >= lo; row -= kSub) {
        const int32_t len = hi - row;
        const int sub = row / kSub % kSubs;
        {
            float raw[4], dl[4], dy[4], slope[4], gw[4];
            step_sizes<T>(a, tile.dl, bias, raw, dl);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                dy[r] = T::load(tile.go[r]);
                slope[r] = 1.f;
                gw[r] = 0.f;
            }
            if (a.softplus)
#pragma unroll
                for (int r = 0; r < 4; ++r) slope[r] = sigmoid_f<T>(raw[r]);
            if (gate)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const float z = T::load(tile.z[r]), q = sigmoid_f<T>(z);
                    gw[r] = dy[r] * silu_slope(z, q);
                    dy[r] *= silu_f(z, q);
                }
            float u[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) u[r] = T::load(tile.u[r]);
            // rows past the end and channels past the last: nothing is added
            if (len < kSub || l.wch + 16 > a.dg)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!l.active || 4 * r + l.q >= len) dl[r] = u[r] = dy[r] = 0.f;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                ex.a[4 * r + l.q][l.c] = make_float2(dl[r], dl[r] * u[r]);
                ex.b[4 * r + l.q][l.c] = make_float2(dy[r], u[r]);
                ex.c[4 * r + l.q][l.c] = make_float2(slope[r], gw[r]);
            }
        }
        tile.B.get(g.B);
        tile.C.get(g.C);
#pragma unroll
        for (int i = 0; i < KS; ++i) g.h[0][i] = 0.f;
        if (l.active)
            ld_states<KS>(a.cs + ((slot * kSubs + sub) * a.channels + l.ch) * NP + l.q * KS, g.h[0]);
        wave_lds_fence();

        float t0[4];
        grad_forward<KS, 0>(ex, l.c, gate, g, t0);
        RowIn x[4];
        read_rows<3>(ex, l.c, x);
        grad_rows4<KS, 3>(ex, l.c, x, g);
        grad_rows4<KS, 2>(ex, l.c, x, g);
        // the next tile's loads, into the registers that half the rows have left
        __builtin_amdgcn_sched_barrier(0);
        if (row > lo) tile.load(a, l, kSub, gate);
        __builtin_amdgcn_sched_barrier(0);
        grad_rows4<KS, 1>(ex, l.c, x, g);
        grad_rows4<KS, 0>(ex, l.c, x, g);

        float(*mine)[2 * NP + 4] = bc[sub & 1][w];
        st_states<KS>(&mine[brev][l.q * KS], g.dBt);
        st_states<KS>(&mine[brev][NP + l.q * KS], g.dCt);
        float du[4], dd[4], dz[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const float row_dl = ex.a[4 * r + l.q][l.c].x;
            const float2 dy_u = ex.b[4 * r + l.q][l.c], sw = ex.c[4 * r + l.q][l.c];
            du[r] = fma32(g.th[r], row_dl, Dc * dy_u.x);
            dd[r] = fma32(g.th[r], dy_u.y, g.dc[r] * kLn2) * sw.x;
            dz[r] = sw.y * fma32(Dc, dy_u.y, g.y[r]);
            dD = fma32(dy_u.x, dy_u.y, dD);
            if (l.active && 4 * r + l.q < len) dbias += dd[r];
        }
        o_du.store(l, len, du);
        o_du.prev();
        o_dd.store(l, len, dd);
        o_dd.prev();
        if (gate) o_dz.store(l, len, dz);
        o_dz.prev();
        __syncthreads();
        for (int i = threadIdx.x; i < kSub * 2 * NP; i += 256) {
            const int t = i / (2 * NP), n = i - t * 2 * NP;
            const float v = (bc[sub & 1][0][t][n] + bc[sub & 1][1][t][n]) +
                            (bc[sub & 1][2][t][n] + bc[sub & 1][3][t][n]);
            if (t < len)
                a.ws_bc[((int64_t)slab * bc_rows + bc_row + row + t) * (2 * NP) + n] = v;
        }
        if (sub != 0) continue;
        // the chunk is done: its parts of the parameters' gradients
        const float sum_D = fold_quad(dD, dD, dD, dD);
        const float sum_b = fold_quad(dbias, dbias, dbias, dbias);
        if (l.active) {
            const int64_t part = slot * a.channels + l.ch;
            st_states<KS>(a.ws_state + part * NP + l.q * KS, g.dA);
            if (l.q == 0) {
                a.ws_dD[part] = sum_D;
                a.ws_dbias[part] = sum_b;
            }
        }
        if (!SEQ) continue;
        --slot;
        dD = dbias = 0.f;
#pragma unroll
        for (int i = 0; i < KS; ++i) g.dA[i] = 0.f;
    }
    if (SEQ && a.dinit && l.active)
#pragma unroll
        for (int i = 0; i < KS; ++i)
            if (l.q * KS + i < a.states) a.dinit[own + i] = g.R[i];
}

// What is left to sum, in one launch: the first workgroups take the parameters'
// gradients over the chunks, the others dB and dC of each row, the slabs' sums in
// order, rounded once.
template <typename T, int NP>
__global__ __launch_bounds__(1024) void k_scan_grad_sums(ScanArgs a, ColumnSums params,
                                                         uint32_t param_blocks, int groups)
{
    if (blockIdx.x < param_blocks) {
        column_sum_block(params, blockIdx.x);
        return;
    }
    const int64_t bc_rows = a.q.starts ? a.q.rows : a.q.seqs * a.q.rows;
    const int64_t i = (int64_t)(blockIdx.x - param_blocks) * 1024 + threadIdx.x;
    const int64_t rg = i / (2 * NP);
    const int n = (int)(i - rg * (2 * NP));
    const int64_t r = rg / groups;
    const int g = (int)(rg - r * groups);
    const int st_n = n < NP ? n : n - NP;
    if (r >= bc_rows || st_n >= a.states) return;
    int64_t s = 0, row = r;
    if (a.q.starts) {
        if (r < clamp_start(a.q, 0) || r >= clamp_start(a.q, a.q.seqs)) return;
    } else {
        s = r / a.q.rows;
        row = r - s * a.q.rows;
    }
    const float* p = a.ws_bc + ((int64_t)g * a.slabs * bc_rows + r) * (2 * NP) + n;
    const int64_t step = bc_rows * (2 * NP);
    float v = 0.f;
    int k = 0;
    for (; k + 8 <= a.slabs; k += 8) {
        float x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = p[(k + j) * step];
#pragma unroll
        for (int j = 0; j < 8; ++j) v += x[j];
    }
    for (; k < a.slabs; ++k) v += p[k * step];
    const canon_rows_t& o = n < NP ? a.dB : a.dC;
    st<T>(rows_ptr<T>(o, s, a.q, row) + (int64_t)g * a.states + st_n, v);
}

// Whole sequences save the pass that folds each chunk from zero, where there
// are enough for the chip's 512 places (two workgroups on each of 256 compute
// units).  Measured as for the forward pass, at 64, 128, 256, 320, 384, 448, 512,
// 576, 640, 768, 1024 workgroups: whole 323, 323, 344, 455, 459, 462, 467, 716,
// 725, 737, 911; in chunks 99, 167, 305, 378, 446, 515, 584, 655, 723, 862, 1146.
// The same for float32 and 8 states, within 5%; with 4 states whole sequences would
// gain at 640 already (bf16 329 and 370, float32 382 and 453).
inline bool grad_whole_sequences(const ScanArgs& a, int64_t slabs)
{
    const int64_t w = a.q.seqs * slabs, full = w / 512, rest = w % 512;
    if (a.q.rows <= kShortRows) return w > 0;
    const int64_t last = rest > 256 ? 455 : rest > 0 ? (full ? 265 : 330) : 0;
    return a.q.starts == nullptr && w > 0 && 467 * full + last <= 28 + w * 35 / 32;
}

template <typename T, int KS>
hipError_t launch_scan_grad_ks(const ScanArgs& a, int64_t groups, hipStream_t st)
{
    constexpr int NP = 4 * KS;
    const int64_t slots = slot_count<kCh>(a.q.seqs, a.q.rows, a.q.starts != nullptr);
    const int64_t slabs = groups * a.slabs;
    if (grad_whole_sequences(a, slabs)) {
        k_selective_scan_grad<T, KS, true>
            <<<dim3((unsigned)(a.q.seqs * slabs)), dim3(256), 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    } else {
        const unsigned grid = (unsigned)(slots * slabs);
        if (grid) k_scan_back_sum<T, KS><<<dim3(grid), dim3(256), 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
        if (hipError_t e = launch_scan_carry<NP, true>(a, a.dfinal, a.dinit, st)) return e;
        if (grid) k_selective_scan_grad<T, KS, false><<<dim3(grid), dim3(256), 0, st>>>(a);
        if (hipError_t e = hipGetLastError()) return e;
    }
    const int64_t d = a.channels;
    const ColumnSums params = {{{a.ws_state, d * NP, NP, a.states, a.dA},
                                {a.ws_dD, d, 1, 1, a.dD},
                                {a.ws_dbias, d, 1, 1, a.dbias}},
                               slots};
    const int64_t blocks = column_sum_blocks(params);
    const int64_t bc = (a.q.starts ? a.q.rows : a.q.seqs * a.q.rows) * groups * 2 * NP;
    k_scan_grad_sums<T, NP><<<dim3((unsigned)(blocks + (bc + 1023) / 1024)), dim3(1024), 0, st>>>(
        a, params, (uint32_t)blocks, (int)groups);
    return hipGetLastError();
}

template <typename T>
hipError_t launch_selective_scan_grad(const ScanArgs& a, int64_t groups, hipStream_t st)
{
    switch (scan_ks(a.states)) {
        case 1: return launch_scan_grad_ks<T, 1>(a, groups, st);
        case 2: return launch_scan_grad_ks<T, 2>(a, groups, st);
        default: return launch_scan_grad_ks<T, 4>(a, groups, st);
    }
}

}  // namespace seq
}  // namespace canon
