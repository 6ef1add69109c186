// C ABI of the sequence operators (canon_seq.h): argument checking, workspace
// layout, dispatch on the element type.
#include "../../include/canon_seq.h"
#include "api_impl.hpp"
#include "causal_conv.hpp"
#include "embedding.hpp"
#include "selective_scan.hpp"

using namespace canon;
using namespace canon::seq;
using canon::abi::check_ws;
using canon::abi::hip_status;
using canon::abi::round_up;

namespace {

size_t elem_bytes(int64_t dtype) { return dtype == CANON_F32 ? 4 : 2; }
bool is_dtype(int64_t d) { return d == CANON_F32 || d == CANON_BF16 || d == CANON_F16; }

// Launches are one-dimensional: fewer than 2^32 threads.  Row counts fit
// 32-bit indexes with room for a chunk; partial sums are kept below 2^47
// elements so that no size overflows.
constexpr int64_t kMaxRows = (int64_t)1 << 30;
constexpr int64_t kMaxGrid256 = (int64_t)1 << 24;

bool mul_fits(int64_t a, int64_t b, int64_t limit) { return a == 0 || b <= limit / a; }

template <class F>
canon_status_t with_dtype(int64_t dtype, F&& f)
{
    switch (dtype) {
        case CANON_F32: return f(F32{});
        case CANON_BF16: return f(BF16{});
        case CANON_F16: return f(F16{});
        default: return CANON_EINVAL;
    }
}

// Vectors of `bytes` at every row of r: base and strides.
bool rows_aligned(const canon_rows_t& r, size_t es, size_t bytes, bool one_row)
{
    if (r.p == nullptr) return true;
    const bool row_ok = one_row || (size_t)r.row * es % bytes == 0;
    return (uintptr_t)r.p % bytes == 0 && row_ok && (size_t)r.seq * es % bytes == 0;
}

bool ptr_aligned(const void* p, size_t bytes) { return (uintptr_t)p % bytes == 0; }

bool rows_valid(const canon_rows_t& r) { return r.p != nullptr && r.row >= 0 && r.seq >= 0; }
// rows of an output: no two may share elements, whether a sequence's rows lie
// together or the sequences are interleaved
bool out_valid(const canon_rows_t& r, int64_t cols, int64_t seqs, int64_t rows)
{
    if (!rows_valid(r)) return false;
    if (rows > 1 && r.row < cols) return false;
    if (seqs <= 1) return true;
    if (r.seq < cols) return false;
    return rows <= 1 || (r.seq - cols) / (rows - 1) >= r.row ||
           (r.row - cols) / (seqs - 1) >= r.seq;
}

// Bump allocation in the workspace.
struct Layout {
    size_t bytes = 0;
    size_t take(size_t n)
    {
        const size_t at = bytes;
        bytes += round_up(n, 256);
        return at;
    }
    template <typename T>
    static T* at(void* ws, size_t off)
    {
        return reinterpret_cast<T*>(static_cast<char*>(ws) + off);
    }
};

// ------------------------------------------------------------------ embedding
struct EmbedLayout : Layout {
    size_t order, offset, items, n_items, n_long, before, longs, part, part_last;
    int64_t ld;
    EmbedLayout(int64_t tokens, int64_t rows, int64_t width)
    {
        const size_t groups = (size_t)id_groups(rows);
        order = take(4 * (size_t)tokens);
        offset = take(4 * ((size_t)rows + 1));
        items = take(16 * (size_t)tokens);
        n_items = take(4 * groups);
        n_long = take(4 * groups);
        before = take(4 * groups);
        longs = take(4 * ((size_t)tokens / (kEmbedChunk + 1) + 1));
        ld = (width + 3) / 4 * 4;
        const size_t parts =
            tokens > kEmbedChunk ? ((size_t)tokens / kEmbedChunk + 1) * (size_t)ld * 4 : 0;
        part = take(parts);
        part_last = take(parts);
    }
};

bool embed_sizes_ok(size_t tokens, size_t rows, size_t width)
{
    return tokens < (size_t)kMaxRows && rows < ((size_t)1 << 31) && width < ((size_t)1 << 24);
}

bool embed_grad_sizes_ok(size_t tokens, size_t rows, size_t width)
{
    return embed_sizes_ok(tokens, rows, width) && rows <= (size_t)kEmbedGradRows;
}

// ---------------------------------------------------------------- convolution
struct ConvLayout : Layout {
    size_t w, b;
    ConvLayout(int64_t seqs, int64_t rows, bool packed, int64_t channels, int64_t taps)
    {
        const size_t slots = (size_t)slot_count<CANON_CONV_CHUNK>(seqs, rows, packed);
        w = take(4 * slots * (size_t)channels * (size_t)taps);
        b = take(4 * slots * (size_t)channels);
    }
};

// Sizes that every kernel can index and launch.
canon_status_t seq_sizes(int64_t seqs, int64_t rows, int64_t channels, bool packed)
{
    if (seqs < 0 || rows < 0 || channels < 0) return CANON_EINVAL;
    if (rows >= kMaxRows || seqs >= kMaxRows || channels >= (1 << 24)) return CANON_EUNSUPPORTED;
    const int64_t slots = slot_count<8>(seqs, rows, packed);
    if (!mul_fits(slots, channels, (int64_t)1 << 40)) return CANON_EUNSUPPORTED;
    return CANON_OK;
}

canon_status_t conv_args(const canon_conv_t* c, bool step, bool grad, ConvArgs* a)
{
    if (c == nullptr) return CANON_EINVAL;
    const bool packed = c->starts != nullptr;
    if (step && packed) return CANON_EINVAL;
    const int64_t rows = step ? 1 : c->rows;
    if (canon_status_t s = seq_sizes(c->seqs, rows, c->channels, packed)) return s;
    if (!is_dtype(c->dtype) || c->taps < 1 || (c->silu != 0 && c->silu != 1)) return CANON_EINVAL;
    if (c->param_dtype != c->dtype && c->param_dtype != CANON_F32) return CANON_EINVAL;
    if (c->taps > CANON_MAX_TAPS) return CANON_EUNSUPPORTED;
    if (c->weight == nullptr) return CANON_EINVAL;
    const bool some = c->seqs > 0 && rows > 0 && c->channels > 0;
    const int64_t out_seqs = packed ? 1 : c->seqs;
    if (some && !rows_valid(c->x)) return CANON_EINVAL;
    if (some && !grad && !out_valid(c->out, c->channels, out_seqs, rows)) return CANON_EINVAL;
    if (some && grad &&
        (!rows_valid(c->dout) || !out_valid(c->dx, c->channels, out_seqs, rows)))
        return CANON_EINVAL;
    if (grad && (c->dweight == nullptr || (c->dbias != nullptr && c->bias == nullptr)))
        return CANON_EINVAL;
    const size_t es = elem_bytes(c->dtype);
    *a = ConvArgs{};
    a->q = Seqs{c->seqs, rows, c->starts};
    a->x = c->x;
    a->out = c->out;
    a->weight = c->weight;
    a->bias = c->bias;
    a->init = c->taps > 1 ? c->init_state : nullptr;
    a->final = c->taps > 1 && !grad ? c->final_state : nullptr;
    a->channels = (int32_t)c->channels;
    a->param_f32 = c->param_dtype == CANON_F32;
    a->silu = c->silu != 0;
    a->dout = grad ? c->dout : canon_rows_t{};
    a->dx = grad ? c->dx : canon_rows_t{};
    if (grad) a->out = canon_rows_t{};
    a->dweight = c->dweight;
    a->dbias = c->dbias;
    a->dfinal = c->taps > 1 ? c->d_final_state : nullptr;
    a->dinit = c->taps > 1 ? c->d_init_state : nullptr;
    const size_t v = 4 * es;  // four channels
    a->vec = (size_t)c->channels * es % v == 0 && rows_aligned(a->x, es, v, false) &&
             rows_aligned(a->out, es, v, false) && rows_aligned(a->dout, es, v, false) &&
             rows_aligned(a->dx, es, v, false) && ptr_aligned(a->init, v) &&
             ptr_aligned(a->final, v) && ptr_aligned(a->dfinal, v) && ptr_aligned(a->dinit, v);
    // threads of the shortest runs: four channels each, two in the backward
    // pass, or (counted so wherever it can be) one
    const int64_t per = a->vec ? c->channels / (grad ? 2 : 4) : c->channels;
    if (!mul_fits(per, slot_count<8>(c->seqs, rows, packed), kMaxGrid256 * 255))
        return CANON_EUNSUPPORTED;
    return CANON_OK;
}

// ------------------------------------------------------------- selective scan
struct SelectiveScanLayout : Layout {
    size_t state, dl, dD = 0, dbias = 0, bc = 0;
    SelectiveScanLayout(int64_t seqs, int64_t rows, bool packed, int64_t channels, int64_t states,
               int64_t groups, bool grad)
    {
        const size_t slots = (size_t)slot_count<CANON_SCAN_CHUNK>(seqs, rows, packed);
        const size_t np = 4 * (size_t)scan_ks(states), d = (size_t)channels;
        state = take(4 * slots * d * np);
        dl = take(4 * slots * d);
        if (!grad) return;
        dD = take(4 * slots * d);
        dbias = take(4 * slots * d);
        const size_t slabs =
            (size_t)groups * (((size_t)channels / (size_t)groups + kSlab - 1) / kSlab);
        bc = take(4 * slabs * 2 * np * (size_t)(packed ? rows : seqs * rows));
    }
};

bool scan_query_ok(size_t seqs, size_t rows, size_t channels, size_t groups, size_t states)
{
    return seqs < (size_t)kMaxRows && rows < (size_t)kMaxRows && channels < (1u << 24) &&
           groups >= 1 && groups <= (channels > 1 ? channels : 1) && channels % groups == 0 &&
           states >= 1 && states <= CANON_MAX_STATES;
}

canon_status_t scan_args(const canon_selective_scan_t* c, bool step, bool grad, ScanArgs* a)
{
    if (c == nullptr) return CANON_EINVAL;
    const bool packed = c->starts != nullptr;
    if (step && packed) return CANON_EINVAL;
    const int64_t rows = step ? 1 : c->rows;
    if (canon_status_t s = seq_sizes(c->seqs, rows, c->channels, packed)) return s;
    if (!is_dtype(c->dtype) || (c->softplus != 0 && c->softplus != 1) || c->groups < 1 ||
        c->states < 1 || c->channels % c->groups != 0)
        return CANON_EINVAL;
    if (c->states > CANON_MAX_STATES) return CANON_EUNSUPPORTED;
    if (c->channels > 0 && c->A == nullptr) return CANON_EINVAL;
    const int64_t bc_cols = c->groups * c->states, out_seqs = packed ? 1 : c->seqs;
    const bool some = c->seqs > 0 && rows > 0 && c->channels > 0;
    if (some) {
        if (!rows_valid(c->u) || !rows_valid(c->delta) || !rows_valid(c->B) || !rows_valid(c->C))
            return CANON_EINVAL;
        if (c->z.p != nullptr && !rows_valid(c->z)) return CANON_EINVAL;
        if (!grad && !out_valid(c->out, c->channels, out_seqs, rows)) return CANON_EINVAL;
        if (grad && (!rows_valid(c->dout) || !out_valid(c->du, c->channels, out_seqs, rows) ||
                     !out_valid(c->ddelta, c->channels, out_seqs, rows) ||
                     (c->z.p != nullptr && !out_valid(c->dz, c->channels, out_seqs, rows)) ||
                     !out_valid(c->dB, bc_cols, out_seqs, rows) || !out_valid(c->dC, bc_cols, out_seqs, rows) ||
                     c->chunk_states == nullptr))
            return CANON_EINVAL;
    }
    // without channels nothing would be written to dB and dC
    if (grad && (c->channels == 0 || c->dA == nullptr || (c->dD != nullptr && c->D == nullptr) ||
                 (c->ddelta_bias != nullptr && c->delta_bias == nullptr)))
        return CANON_EINVAL;
    if (!ptr_aligned(c->chunk_states, 16)) return CANON_EINVAL;
    for (const canon_rows_t* r : {&c->u, &c->delta, &c->z, &c->out, &c->B, &c->C, &c->dout, &c->du,
                                  &c->ddelta, &c->dz, &c->dB, &c->dC})
        if (r->p != nullptr && r->row >= kMaxPitch) return CANON_EUNSUPPORTED;
    if (bc_cols >= ((int64_t)1 << 24)) return CANON_EUNSUPPORTED;
    const size_t es = elem_bytes(c->dtype);
    const int ks = scan_ks(c->states);
    *a = ScanArgs{};
    a->q = Seqs{c->seqs, rows, c->starts};
    a->u = c->u;
    a->delta = c->delta;
    a->z = c->z;
    a->out = c->out;
    a->B = c->B;
    a->C = c->C;
    a->A = c->A;
    a->D = c->D;
    a->bias = c->delta_bias;
    a->init = c->init_state;
    a->final = c->final_state;
    a->cs = c->chunk_states;
    a->channels = (int32_t)c->channels;
    a->dg = (int32_t)(c->channels / c->groups);
    a->slabs = (a->dg + kSlab - 1) / kSlab;
    a->states = (int32_t)c->states;
    a->softplus = c->softplus != 0;
    a->bc_vec = c->states % ks == 0 && rows_aligned(c->B, es, ks * es, false) &&
                rows_aligned(c->C, es, ks * es, false);
    a->st_vec = c->states == 4 * ks && ptr_aligned(c->A, 4 * ks) &&
                ptr_aligned(c->init_state, 4 * ks) && ptr_aligned(c->final_state, 4 * ks);
    a->dout = c->dout;
    a->du = c->du;
    a->ddelta = c->ddelta;
    a->dz = c->dz;
    a->dB = c->dB;
    a->dC = c->dC;
    a->dA = c->dA;
    a->dD = c->dD;
    a->dbias = c->ddelta_bias;
    a->dfinal = c->d_final_state;
    a->dinit = c->d_init_state;
    const int64_t slots =
        step ? c->seqs : slot_count<CANON_SCAN_CHUNK>(c->seqs, rows, packed);
    if (!mul_fits(slots, c->groups * a->slabs, kMaxGrid256 - 1) ||
        !mul_fits(c->seqs, (c->channels * 4 * ks + 63) / 64, 4 * kMaxGrid256 - 1) ||
        (grad && (!mul_fits((packed ? rows : c->seqs * rows), c->groups * 8 * ks,
                            (int64_t)1 << 31) ||
                  !mul_fits(c->channels, 4 * ks + 2, (int64_t)1 << 26))))  // column sums
        return CANON_EUNSUPPORTED;
    return CANON_OK;
}

}  // namespace

extern "C" {

int canon_seq_version(void) { return CANON_SEQ_VERSION; }

canon_status_t canon_embedding(int dtype, const void* weight, size_t ld_weight, size_t rows,
                               size_t width, const void* ids, int id_bytes, size_t tokens,
                               float scale, void* out, size_t ld_out, void* stream)
{
    if (!is_dtype(dtype) || (id_bytes != 4 && id_bytes != 8) || ld_weight < width ||
        ld_out < width)
        return CANON_EINVAL;
    if (tokens == 0 || width == 0) return CANON_OK;
    if (ids == nullptr || out == nullptr || (rows > 0 && weight == nullptr)) return CANON_EINVAL;
    const size_t es = elem_bytes(dtype);
    if (!embed_sizes_ok(tokens, rows, width) ||
        !mul_fits((int64_t)tokens, embed_accesses((int64_t)width, es),
                  (kMaxGrid256 - 1) * kEmbedGridAccesses))
        return CANON_EUNSUPPORTED;
    if (out == weight) return CANON_EINVAL;
    EmbedArgs a{weight, (int64_t)ld_weight, (int64_t)rows, (int64_t)width, ids, id_bytes == 8,
                false, (int64_t)tokens, scale, out, (int64_t)ld_out};
    a.vec = width * es % 16 == 0 && ptr_aligned(weight, 16) && ptr_aligned(out, 16) &&
            ld_weight * es % 16 == 0 && ld_out * es % 16 == 0;
    return with_dtype(dtype, [&](auto t) {
        return hip_status(launch_embedding<decltype(t)>(a, static_cast<hipStream_t>(stream)));
    });
}

size_t canon_embedding_grad_workspace_bytes(size_t tokens, size_t rows, size_t width)
{
    if (!embed_grad_sizes_ok(tokens, rows, width) || rows == 0 || width == 0) return 0;
    return EmbedLayout((int64_t)tokens, (int64_t)rows, (int64_t)width).bytes;
}

canon_status_t canon_embedding_grad(int dtype, const void* dout, size_t ld_dout, const void* ids,
                                    int id_bytes, size_t tokens, size_t rows, size_t width,
                                    float scale, int64_t padding_id, int accumulate, int dw_dtype,
                                    void* dw, size_t ld_dw, void* ws, size_t ws_bytes,
                                    void* stream)
{
    if (!is_dtype(dtype) || (dw_dtype != dtype && dw_dtype != CANON_F32) ||
        (id_bytes != 4 && id_bytes != 8) || (accumulate != 0 && accumulate != 1) ||
        ld_dout < width || ld_dw < width || padding_id < -1)
        return CANON_EINVAL;
    if (rows == 0 || width == 0) return CANON_OK;
    if (dw == nullptr || (tokens > 0 && (ids == nullptr || dout == nullptr))) return CANON_EINVAL;
    if (!embed_grad_sizes_ok(tokens, rows, width)) return CANON_EUNSUPPORTED;
    const EmbedLayout l((int64_t)tokens, (int64_t)rows, (int64_t)width);
    if (canon_status_t s = check_ws(ws, ws_bytes, l.bytes)) return s;
    if (tokens > 0 && dw == dout) return CANON_EINVAL;
    const size_t es = elem_bytes(dtype), gs = elem_bytes(dw_dtype);
    EmbedGradArgs a{};
    a.dout = dout;
    a.ld_dout = (int64_t)ld_dout;
    a.ids = ids;
    a.ids64 = id_bytes == 8;
    a.vec = width * es % 16 == 0 && ptr_aligned(dout, 16) && ptr_aligned(dw, 16) &&
            ld_dout * es % 16 == 0 && ld_dw * gs % 16 == 0;
    a.accumulate = accumulate != 0;
    a.tokens = (int64_t)tokens;
    a.rows = (int64_t)rows;
    a.width = (int64_t)width;
    a.scale = scale;
    a.padding_id = padding_id;
    a.dw = dw;
    a.ld_dw = (int64_t)ld_dw;
    a.order = l.at<int32_t>(ws, l.order);
    a.offset = l.at<int32_t>(ws, l.offset);
    a.items = l.at<int4>(ws, l.items);
    a.n_items = l.at<int32_t>(ws, l.n_items);
    a.n_long = l.at<int32_t>(ws, l.n_long);
    a.before = l.at<int32_t>(ws, l.before);
    a.longs = l.at<int32_t>(ws, l.longs);
    a.part = l.at<float>(ws, l.part);
    a.part_last = l.at<float>(ws, l.part_last);
    a.ld_part = l.ld;
    const hipStream_t st = static_cast<hipStream_t>(stream);
    switch (dtype) {
        case CANON_F32: return hip_status(launch_embedding_grad<F32, F32>(a, st));
        case CANON_BF16:
            return hip_status(dw_dtype == CANON_F32 ? launch_embedding_grad<BF16, F32>(a, st)
                                                    : launch_embedding_grad<BF16, BF16>(a, st));
        default:
            return hip_status(dw_dtype == CANON_F32 ? launch_embedding_grad<F16, F32>(a, st)
                                                    : launch_embedding_grad<F16, F16>(a, st));
    }
}

canon_status_t canon_causal_conv(const canon_conv_t* c, void* stream)
{
    ConvArgs a;
    if (canon_status_t s = conv_args(c, false, false, &a)) return s;
    if (a.q.seqs == 0 || a.channels == 0) return CANON_OK;
    // in place a run would read rows that its neighbour has overwritten
    if (a.q.rows > 0 && a.out.p == a.x.p) return CANON_EINVAL;
    return with_dtype(c->dtype, [&](auto t) {
        return hip_status(launch_causal_conv<decltype(t)>(a, (int)c->taps,
                                                          static_cast<hipStream_t>(stream)));
    });
}

size_t canon_causal_conv_grad_workspace_bytes(size_t seqs, size_t rows, int packed,
                                              size_t channels, size_t taps)
{
    if (seqs >= (size_t)kMaxRows || rows >= (size_t)kMaxRows || channels >= (1u << 24) ||
        taps < 1 || taps > CANON_MAX_TAPS)
        return 0;
    return ConvLayout((int64_t)seqs, (int64_t)rows, packed != 0, (int64_t)channels, (int64_t)taps)
        .bytes;
}

canon_status_t canon_causal_conv_grad(const canon_conv_t* c, void* ws, size_t ws_bytes,
                                      void* stream)
{
    ConvArgs a;
    if (canon_status_t s = conv_args(c, false, true, &a)) return s;
    if (a.channels == 0) return CANON_OK;
    const ConvLayout l(a.q.seqs, a.q.rows, a.q.starts != nullptr, a.channels, c->taps);
    if (canon_status_t s = check_ws(ws, ws_bytes, l.bytes)) return s;
    if (a.q.seqs > 0 && a.q.rows > 0 && (a.dx.p == a.x.p || a.dx.p == a.dout.p))
        return CANON_EINVAL;
    a.ws_w = l.at<float>(ws, l.w);
    a.ws_b = l.at<float>(ws, l.b);
    return with_dtype(c->dtype, [&](auto t) {
        return hip_status(launch_causal_conv_grad<decltype(t)>(a, (int)c->taps,
                                                               static_cast<hipStream_t>(stream)));
    });
}

canon_status_t canon_causal_conv_step(const canon_conv_t* c, void* stream)
{
    ConvArgs a;
    if (canon_status_t s = conv_args(c, true, false, &a)) return s;
    if (a.q.seqs == 0 || a.channels == 0) return CANON_OK;
    return with_dtype(c->dtype, [&](auto t) {
        return hip_status(launch_causal_conv_step<decltype(t)>(a, (int)c->taps,
                                                               static_cast<hipStream_t>(stream)));
    });
}

size_t canon_selective_scan_states(size_t seqs, size_t rows, int packed, size_t channels,
                                   size_t states)
{
    if (!scan_query_ok(seqs, rows, channels, 1, states)) return 0;
    return (size_t)slot_count<CANON_SCAN_CHUNK>((int64_t)seqs, (int64_t)rows, packed != 0) *
           (CANON_SCAN_CHUNK / kSub) * channels * 4 * (size_t)scan_ks((int64_t)states);
}

size_t canon_selective_scan_workspace_bytes(size_t seqs, size_t rows, int packed, size_t channels,
                                            size_t states)
{
    if (!scan_query_ok(seqs, rows, channels, 1, states)) return 0;
    return SelectiveScanLayout((int64_t)seqs, (int64_t)rows, packed != 0, (int64_t)channels,
                      (int64_t)states, 1, false)
        .bytes;
}

canon_status_t canon_selective_scan(const canon_selective_scan_t* c, void* ws, size_t ws_bytes,
                                    void* stream)
{
    ScanArgs a;
    if (canon_status_t s = scan_args(c, false, false, &a)) return s;
    if (a.q.seqs == 0 || a.channels == 0) return CANON_OK;
    const SelectiveScanLayout l(a.q.seqs, a.q.rows, a.q.starts != nullptr, a.channels, a.states, 1, false);
    if (canon_status_t s = check_ws(ws, ws_bytes, l.bytes)) return s;
    a.ws_state = l.at<float>(ws, l.state);
    a.ws_dl = l.at<float>(ws, l.dl);
    return with_dtype(c->dtype, [&](auto t) {
        return hip_status(launch_selective_scan<decltype(t)>(a, c->groups,
                                                             static_cast<hipStream_t>(stream)));
    });
}

size_t canon_selective_scan_grad_workspace_bytes(size_t seqs, size_t rows, int packed,
                                                 size_t channels, size_t groups, size_t states)
{
    if (!scan_query_ok(seqs, rows, channels, groups, states)) return 0;
    return SelectiveScanLayout((int64_t)seqs, (int64_t)rows, packed != 0, (int64_t)channels,
                      (int64_t)states, (int64_t)groups, true)
        .bytes;
}

canon_status_t canon_selective_scan_grad(const canon_selective_scan_t* c, void* ws,
                                         size_t ws_bytes, void* stream)
{
    ScanArgs a;
    if (canon_status_t s = scan_args(c, false, true, &a)) return s;
    const SelectiveScanLayout l(a.q.seqs, a.q.rows, a.q.starts != nullptr, a.channels, a.states, c->groups,
                       true);
    if (canon_status_t s = check_ws(ws, ws_bytes, l.bytes)) return s;
    a.ws_state = l.at<float>(ws, l.state);
    a.ws_dl = l.at<float>(ws, l.dl);
    a.ws_dD = l.at<float>(ws, l.dD);
    a.ws_dbias = l.at<float>(ws, l.dbias);
    a.ws_bc = l.at<float>(ws, l.bc);
    return with_dtype(c->dtype, [&](auto t) {
        return hip_status(launch_selective_scan_grad<decltype(t)>(
            a, c->groups, static_cast<hipStream_t>(stream)));
    });
}

canon_status_t canon_selective_scan_step(const canon_selective_scan_t* c, void* stream)
{
    ScanArgs a;
    if (canon_status_t s = scan_args(c, true, false, &a)) return s;
    if (a.q.seqs == 0 || a.channels == 0) return CANON_OK;
    return with_dtype(c->dtype, [&](auto t) {
        return hip_status(launch_selective_scan_step<decltype(t)>(
            a, c->groups, static_cast<hipStream_t>(stream)));
    });
}

}  // extern "C"
