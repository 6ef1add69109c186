// C ABI of the layer operators (canon_layer.h): argument checking, workspace
// layout, dispatch on the element type.
#include "../../include/canon_layer.h"
#include "layer_norm.hpp"
#include "recurrence.hpp"
#include "sample.hpp"
#include "seq_args.hpp"

using namespace canon;
using namespace canon::seq;
using canon::abi::check_ws;
using canon::abi::hip_status;

namespace {

// An output in an input's place: the same elements, not a shifted or strided view.
bool same_rows(const canon_rows_t& a, const canon_rows_t& b)
{
    return a.p == b.p && a.seq == b.seq && a.row == b.row;
}
bool in_place_ok(const canon_rows_t& out, const canon_rows_t& in)
{
    return in.p == nullptr || out.p != in.p || same_rows(out, in);
}

// ----------------------------------------------------------------- layer norm
// A row index and a step of the whole grid add up to less than 2^31.
bool norm_sizes_ok(int64_t seqs, int64_t rows, int64_t width)
{
    return seqs < kMaxRows && rows < kMaxRows && width < ((int64_t)1 << 24) &&
           mul_fits(seqs, rows, kMaxRows - 1);
}

int64_t norm_chunks(int64_t total, int64_t width)
{
    const int64_t chunk = norm_chunk(total, width);
    return (total + chunk - 1) / chunk;
}

struct NormLayout : Layout {
    size_t w, b;
    NormLayout(int64_t total, int64_t width)
    {
        const size_t part = 4 * (size_t)norm_chunks(total, width) * (size_t)width;
        w = take(part);
        b = take(part);
    }
};

canon_status_t norm_args(const canon_norm_t* c, bool grad, NormArgs* a)
{
    if (c == nullptr) return CANON_EINVAL;
    if (c->seqs < 0 || c->rows < 0 || c->width < 0 || !is_dtype(c->dtype) ||
        (c->param_dtype != c->dtype && c->param_dtype != CANON_F32))
        return CANON_EINVAL;
    if (!norm_sizes_ok(c->seqs, c->rows, c->width)) return CANON_EUNSUPPORTED;
    *a = NormArgs{};
    a->total = (int32_t)(c->seqs * c->rows);
    a->rows = (int32_t)c->rows;
    a->width = (int32_t)c->width;
    if (c->width > 0 && c->weight == nullptr) return CANON_EINVAL;
    if (grad && c->width > 0 && c->dweight == nullptr) return CANON_EINVAL;
    if (!grad && !(c->eps >= 0. && c->eps <= (double)kMaxF)) return CANON_EINVAL;  // NaN too
    if (a->total > 0 && a->width > 0) {
        auto out_ok = [&](const canon_rows_t& r) {
            return out_valid(r, c->width, c->seqs, c->rows);
        };
        if (!rows_valid(c->x)) return CANON_EINVAL;
        if (!grad) {
            const bool res = c->residual.p != nullptr, sum = c->sum.p != nullptr;
            if ((res && !rows_valid(c->residual)) || !out_ok(c->out) ||
                (sum && (!res || !out_ok(c->sum) || c->sum.p == c->out.p)))
                return CANON_EINVAL;
            for (const canon_rows_t* in : {&c->x, &c->residual})
                if (!in_place_ok(c->out, *in) || (sum && !in_place_ok(c->sum, *in)))
                    return CANON_EINVAL;
        } else {
            if (!rows_valid(c->dout) || !out_ok(c->dx) || c->stats == nullptr ||
                (c->dsum.p != nullptr && !rows_valid(c->dsum)) || c->dx.p == c->x.p ||
                !in_place_ok(c->dx, c->dout) || !in_place_ok(c->dx, c->dsum))
                return CANON_EINVAL;
        }
    }
    a->inv_width = a->width > 0 ? 1.f / (float)a->width : 0.f;
    a->eps = (float)c->eps;
    a->x = c->x;
    a->weight = c->weight;
    a->stats = c->stats;
    if (!grad) {
        a->residual = c->residual;
        a->sum = c->sum;
        a->out = c->out;
        a->bias = c->bias;
        return CANON_OK;
    }
    a->dout = c->dout;
    a->dsum = c->dsum;
    a->dx = c->dx;
    a->dweight = c->dweight;
    a->dbias = c->dbias;
    if (!mul_fits(norm_chunks(a->total, a->width), (c->width + 1023) / 1024, kMaxGrid256 - 1))
        return CANON_EUNSUPPORTED;
    return CANON_OK;
}

template <class F>
canon_status_t with_params(int64_t dtype, int64_t param, F&& f)
{
    switch (dtype) {
        case CANON_F32: return f(F32{}, F32{});
        case CANON_BF16: return param == CANON_F32 ? f(BF16{}, F32{}) : f(BF16{}, BF16{});
        case CANON_F16: return param == CANON_F32 ? f(F16{}, F32{}) : f(F16{}, F16{});
        default: return CANON_EINVAL;
    }
}

// ----------------------------------------------------------------- recurrence
struct RecurLayout : Layout {
    size_t q = 0, s = 0, h = 0, cq = 0, cs = 0, dd = 0;
    bool carried;  // some sequence may have more than one block
    bool launch;   // and some more than kRecurFold
    bool spread;
    RecurLayout(int64_t seqs, int64_t rows, bool packed, int64_t channels, bool grad)
        : carried(rows > CANON_RECUR_BLOCK && seqs > 0),
          launch(rows > CANON_RECUR_BLOCK * kRecurFold)
    {
        const int64_t slots = slot_count<CANON_RECUR_BLOCK>(seqs, rows, packed);
        const size_t n = 4 * (size_t)slots * (size_t)channels;
        spread = recur_spread(slots, rows, channels) && seqs > 0;
        if (spread) {
            cq = take(kRecurBlockChunks * n);
            cs = take(kRecurBlockChunks * n);
            if (!grad) h = take(n);
        } else if (carried) {
            q = take(n);
            s = take(n);
            h = take(n);
        }
        if (grad) dd = take(spread ? kRecurRounds * n : n);
    }
    void place(RecurArgs* a, void* ws) const
    {
        a->spread = spread;
        if (spread) {
            a->ws_cq = at<float>(ws, cq);
            a->ws_cs = at<float>(ws, cs);
            a->ws_h = at<float>(ws, h);
            return;
        }
        if (!carried) return;
        a->carry = launch;
        a->ws_q = at<float>(ws, q);
        a->ws_s = at<float>(ws, s);
        a->ws_h = at<float>(ws, h);
    }
};

bool recur_query_ok(size_t seqs, size_t rows, size_t channels)
{
    return seqs < (size_t)kMaxRows && rows < (size_t)kMaxRows && channels < ((size_t)1 << 24);
}

canon_status_t recur_args(const canon_recur_t* c, bool step, bool grad, RecurArgs* a)
{
    if (c == nullptr) return CANON_EINVAL;
    const bool packed = c->starts != nullptr, input = c->input_gate.p != nullptr;
    if (step && packed) return CANON_EINVAL;
    const int64_t rows = step ? 1 : c->rows, out_seqs = packed ? 1 : c->seqs;
    if (canon_status_t s = seq_sizes(c->seqs, rows, c->channels, packed)) return s;
    if (!is_dtype(c->dtype)) return CANON_EINVAL;
    auto out_ok = [&](const canon_rows_t& r) { return out_valid(r, c->channels, out_seqs, rows); };
    if (c->seqs > 0 && rows > 0 && c->channels > 0) {
        if (!rows_valid(c->x) || !rows_valid(c->gate) || (input && !rows_valid(c->input_gate)))
            return CANON_EINVAL;
        const canon_rows_t* in[] = {&c->x, &c->gate, &c->input_gate, &c->dout};
        const canon_rows_t* out[] = {grad ? &c->dx : &c->out, &c->dgate, &c->dinput_gate};
        const int outs = !grad ? 1 : input ? 3 : 2, ins = grad ? 4 : 3;
        if (grad && (!rows_valid(c->dout) || c->kept_states == nullptr)) return CANON_EINVAL;
        for (int o = 0; o < outs; ++o) {
            if (!out_ok(*out[o])) return CANON_EINVAL;
            // rows are read again by other workgroups, or by a second pass; single ones by
            // the thread that writes there
            for (int i = 0; i < ins; ++i)
                if (out[o]->p == in[i]->p &&
                    !(step && (c->seqs == 1 || out[o]->seq == in[i]->seq)))
                    return CANON_EINVAL;
            for (int p = 0; p < o; ++p)
                if (out[o]->p == out[p]->p) return CANON_EINVAL;
        }
    }
    if (grad && c->channels > 0 && (c->ddecay == nullptr) != (c->decay == nullptr))
        return CANON_EINVAL;
    if (grad && c->d_init_state != nullptr && c->d_init_state == c->d_final_state)
        return CANON_EINVAL;
    for (const canon_rows_t* r : {&c->x, &c->gate, &c->input_gate, &c->out, &c->dout, &c->dx,
                                  &c->dgate, &c->dinput_gate})
        if (r->p != nullptr && r->row >= kRecurPitch && !step) return CANON_EUNSUPPORTED;
    *a = RecurArgs{};
    a->q = Seqs{c->seqs, rows, c->starts};
    a->x = c->x;
    a->gate = c->gate;
    a->input = c->input_gate;
    a->decay = c->decay;
    a->channels = (int32_t)c->channels;
    a->kept = c->kept_states;
    if (!grad) {
        a->out = c->out;
        a->init = c->init_state;
        a->final = c->final_state;
    } else {
        a->dout = c->dout;
        a->dx = c->dx;
        a->dgate = c->dgate;
        a->dinput = c->dinput_gate;
        a->ddecay = c->ddecay;
        a->dfinal = c->d_final_state;
        a->dinit = c->d_init_state;
    }
    a->pairs = c->dtype != CANON_F32 && c->channels % 2 == 0;
    for (const canon_rows_t* r : {&a->x, &a->gate, &a->input, &a->out, &a->dout, &a->dx, &a->dgate,
                                  &a->dinput})
        a->pairs = a->pairs && rows_aligned(*r, 2, 4, false);
    const int64_t slots =
        step ? c->seqs : slot_count<CANON_RECUR_BLOCK>(c->seqs, rows, packed);
    if (!mul_fits(slots, (c->channels + 63) / 64, ((int64_t)1 << 22) - 1))
        return CANON_EUNSUPPORTED;
    return CANON_OK;
}

}  // namespace

extern "C" {

int canon_layer_version(void) { return CANON_LAYER_VERSION; }

canon_status_t canon_layer_norm(const canon_norm_t* c, void* stream)
{
    NormArgs a;
    if (canon_status_t s = norm_args(c, false, &a)) return s;
    if (a.total == 0 || a.width == 0) return CANON_OK;
    return with_params(c->dtype, c->param_dtype, [&](auto t, auto p) {
        return hip_status(launch_layer_norm<decltype(t), decltype(p)>(
            a, static_cast<hipStream_t>(stream)));
    });
}

size_t canon_layer_norm_grad_workspace_bytes(size_t seqs, size_t rows, size_t width)
{
    if (seqs >= (size_t)kMaxRows || rows >= (size_t)kMaxRows || width >= ((size_t)1 << 24) ||
        !norm_sizes_ok((int64_t)seqs, (int64_t)rows, (int64_t)width))
        return 0;
    return NormLayout((int64_t)(seqs * rows), (int64_t)width).bytes;
}

canon_status_t canon_layer_norm_grad(const canon_norm_t* c, void* ws, size_t ws_bytes,
                                     void* stream)
{
    NormArgs a;
    if (canon_status_t s = norm_args(c, true, &a)) return s;
    if (a.width == 0) return CANON_OK;
    const NormLayout l(a.total, a.width);
    if (canon_status_t s = check_ws(ws, ws_bytes, l.bytes)) return s;
    a.ws_w = l.at<float>(ws, l.w);
    a.ws_b = l.at<float>(ws, l.b);
    return with_params(c->dtype, c->param_dtype, [&](auto t, auto p) {
        return hip_status(launch_layer_norm_grad<decltype(t), decltype(p)>(
            a, static_cast<hipStream_t>(stream)));
    });
}

size_t canon_gated_recurrence_states(size_t seqs, size_t rows, int packed, size_t channels)
{
    if (!recur_query_ok(seqs, rows, channels)) return 0;
    return (size_t)slot_count<CANON_RECUR_BLOCK>((int64_t)seqs, (int64_t)rows, packed != 0) *
           kRecurRounds * channels;
}

size_t canon_gated_recurrence_workspace_bytes(size_t seqs, size_t rows, int packed,
                                              size_t channels)
{
    if (!recur_query_ok(seqs, rows, channels)) return 0;
    return RecurLayout((int64_t)seqs, (int64_t)rows, packed != 0, (int64_t)channels, false).bytes;
}

canon_status_t canon_gated_recurrence(const canon_recur_t* c, void* ws, size_t ws_bytes,
                                      void* stream)
{
    RecurArgs a;
    if (canon_status_t s = recur_args(c, false, false, &a)) return s;
    if (a.q.seqs == 0 || a.channels == 0) return CANON_OK;
    const RecurLayout l(a.q.seqs, a.q.rows, a.q.starts != nullptr, a.channels, false);
    if (canon_status_t s = check_ws(ws, ws_bytes, l.bytes)) return s;
    l.place(&a, ws);
    return with_dtype(c->dtype, [&](auto t) {
        return hip_status(launch_recurrence<decltype(t)>(a, static_cast<hipStream_t>(stream)));
    });
}

size_t canon_gated_recurrence_grad_workspace_bytes(size_t seqs, size_t rows, int packed,
                                                   size_t channels)
{
    if (!recur_query_ok(seqs, rows, channels)) return 0;
    return RecurLayout((int64_t)seqs, (int64_t)rows, packed != 0, (int64_t)channels, true).bytes;
}

canon_status_t canon_gated_recurrence_grad(const canon_recur_t* c, void* ws, size_t ws_bytes,
                                           void* stream)
{
    RecurArgs a;
    if (canon_status_t s = recur_args(c, false, true, &a)) return s;
    if (a.channels == 0) return CANON_OK;
    const RecurLayout l(a.q.seqs, a.q.rows, a.q.starts != nullptr, a.channels, true);
    if (canon_status_t s = check_ws(ws, ws_bytes, l.bytes)) return s;
    l.place(&a, ws);
    a.ws_dd = l.at<float>(ws, l.dd);
    return with_dtype(c->dtype, [&](auto t) {
        return hip_status(launch_recurrence_grad<decltype(t)>(a, static_cast<hipStream_t>(stream)));
    });
}

canon_status_t canon_gated_recurrence_step(const canon_recur_t* c, void* stream)
{
    RecurArgs a;
    if (canon_status_t s = recur_args(c, true, false, &a)) return s;
    if (a.q.seqs == 0 || a.channels == 0) return CANON_OK;
    return with_dtype(c->dtype, [&](auto t) {
        return hip_status(launch_recurrence_step<decltype(t)>(a, static_cast<hipStream_t>(stream)));
    });
}

size_t canon_sample_workspace_bytes(size_t rows, size_t vocab)
{
    (void)rows;
    (void)vocab;
    return 0;
}

canon_status_t canon_sample(const canon_sample_t* c, void* ws, size_t ws_bytes, void* stream)
{
    if (c == nullptr || c->rows < 0 || c->vocab < 0 || c->ld < 0 || !is_dtype(c->dtype) ||
        (c->id_bytes != 4 && c->id_bytes != 8))
        return CANON_EINVAL;
    if (c->rows >= ((int64_t)1 << 22) || c->vocab >= ((int64_t)1 << 24)) return CANON_EUNSUPPORTED;
    if (c->rows == 0) return CANON_OK;
    if (c->ids == nullptr || c->u == nullptr || (c->vocab > 0 && c->logits == nullptr))
        return CANON_EINVAL;
    if (canon_status_t s =
            check_ws(ws, ws_bytes, canon_sample_workspace_bytes((size_t)c->rows, (size_t)c->vocab)))
        return s;
    SampleArgs a{};
    a.logits = c->logits;
    a.ld = c->ld;
    a.rows = c->rows;
    a.vocab = (int32_t)c->vocab;
    int log = 0;
    while (((int64_t)1 << log) < c->vocab) ++log;
    a.bits = log < 12 ? 50 : 62 - log;
    a.share_bits = log < 16 ? 15 : 31 - log;
    a.u = c->u;
    a.temperature = c->temperature;
    a.top_p = c->top_p;
    a.min_p = c->min_p;
    a.top_k = c->top_k;
    a.temperature_all = c->temperature_all;
    a.top_p_all = c->top_p_all;
    a.min_p_all = c->min_p_all;
    a.top_k_all = (int32_t)(c->top_k_all < 0 ? 0 : c->top_k_all > c->vocab ? 0 : c->top_k_all);
    a.ids = c->ids;
    a.ids64 = c->id_bytes == 8;
    return with_dtype(c->dtype, [&](auto t) {
        return hip_status(launch_sample<decltype(t)>(a, static_cast<hipStream_t>(stream)));
    });
}

}  // extern "C"
