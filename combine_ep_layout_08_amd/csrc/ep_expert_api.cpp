// C ABI of the experts' products (include/ep_expert.h): argument checks and kernel
// launches.  Nothing here allocates, synchronises or keeps a pointer.
#include "ep_expert_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

ep_status hip_status(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_HIP; }

struct Span {
    const void *p;
    int64_t bytes;
};

// Whether an output and another buffer share memory; `same`: they may start at the same
// address.
bool clash(Span out, Span other, bool same = false) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(out.p),
                    b = reinterpret_cast<uintptr_t>(other.p);
    if (!a || !b || (same && a == b)) return false;
    return a < b + other.bytes && b < a + out.bytes;
}

// Whether any of the outputs shares memory with another one or with an input.
template <size_t N, size_t M>
bool clashes(const Span (&outs)[N], const Span (&ins)[M]) {
    for (size_t i = 0; i < N; ++i) {
        for (const Span &in : ins)
            if (clash(outs[i], in)) return true;
        for (size_t j = 0; j < i; ++j)
            if (clash(outs[i], outs[j])) return true;
    }
    return false;
}

// A handle from ep_handle_init (or a plain copy of one) that has a layout.
ep_status handle_status(const ep_handle *h) {
    if (!h) return EP_ERR_NULL;
    if (!h->counts || !h->psum || !h->dst_slot || !h->src_meta || !h->scalars ||
        h->num_topk < 1 || h->num_topk > ep::kMaxTopk || h->num_experts < 1 ||
        h->num_experts > ep::kMaxExperts || h->expert_alignment < 1 || h->capacity < 0 ||
        h->num_tokens < 0 || h->num_tokens > h->max_tokens)
        return EP_ERR_WORKSPACE;
    return h->laid_out ? EP_OK : EP_ERR_NOT_LAID_OUT;
}

ep_status size_status(int32_t size, int32_t unit, int32_t most) {
    if (size <= 0) return EP_ERR_SHAPE;
    if (size % unit != 0) return EP_ERR_MISALIGNED;
    return size <= most ? EP_OK : EP_ERR_UNSUPPORTED;
}

bool has_rows(const ep_handle *h) { return h->num_tokens > 0 && h->capacity > 0; }

ep::Segments segments(const ep_handle *h) {
    ep::Segments s{};
    s.counts = h->counts;
    s.psum = h->psum;
    s.src_meta = h->src_meta;
    s.scalars = h->scalars;
    s.num_experts = h->num_experts;
    s.num_topk = h->num_topk;
    s.num_tokens = h->num_tokens;
    s.capacity = h->capacity;
    return s;
}

int64_t x_rows(const ep_handle *h, int32_t token_rows) {
    return token_rows ? h->num_tokens : h->capacity;
}

}  // namespace

extern "C" {

ep_status ep_quantize_i8(const void *x, int32_t num_rows, int32_t channels, void *out_q,
                         float *out_scale, hipStream_t stream) {
    if (num_rows < 0) return EP_ERR_SHAPE;
    const ep_status st = size_status(channels, 16, ep::kMaxExpertChannels);
    if (st != EP_OK || num_rows == 0) return st;
    if (!x || !out_q || !out_scale) return EP_ERR_NULL;
    if (!aligned(x, 16) || !aligned(out_q, 16) || !aligned(out_scale, 4))
        return EP_ERR_MISALIGNED;
    const int64_t all = static_cast<int64_t>(num_rows) * channels;
    if (clashes<2, 1>({{out_q, all}, {out_scale, 4 * int64_t(num_rows)}}, {{x, 2 * all}}))
        return EP_ERR_UNSUPPORTED;
    ep::QuantI8Args a{};
    a.num_rows = num_rows;
    a.x = x;
    a.channels = channels;
    a.q = out_q;
    a.scale = out_scale;
    return hip_status(ep::launch_quantize_i8(a, stream));
}

ep_status ep_quantize_i8_rows(const ep_handle *h, const void *x, int32_t channels, void *out_q,
                              float *out_scale, hipStream_t stream) {
    ep_status st = handle_status(h);
    if (st != EP_OK) return st;
    st = size_status(channels, 16, ep::kMaxExpertChannels);
    if (st != EP_OK || !has_rows(h)) return st;
    if (!x || !out_q || !out_scale) return EP_ERR_NULL;
    if (!aligned(x, 16) || !aligned(out_q, 16) || !aligned(out_scale, 4))
        return EP_ERR_MISALIGNED;
    const int64_t all = h->capacity * channels;
    if (clashes<2, 1>({{out_q, all}, {out_scale, 4 * h->capacity}}, {{x, 2 * all}}))
        return EP_ERR_UNSUPPORTED;
    ep::QuantI8Args a{};
    a.dst = h->dst_slot;
    a.scalars = h->scalars;
    a.num_rows = static_cast<int64_t>(h->num_tokens) * h->num_topk;
    a.capacity = h->capacity;
    a.x = x;
    a.channels = channels;
    a.q = out_q;
    a.scale = out_scale;
    return hip_status(ep::launch_quantize_i8(a, stream));
}

ep_status ep_expert_i8(const ep_handle *h, const void *x, const float *x_scale,
                       int32_t token_rows, int32_t k, const void *w, const float *w_scale,
                       int32_t n, int32_t gated, const float *row_weights, void *out,
                       hipStream_t stream) {
    ep_status st = handle_status(h);
    if (st != EP_OK) return st;
    if ((token_rows != 0 && token_rows != 1) || (gated != 0 && gated != 1) ||
        (row_weights && !gated))
        return EP_ERR_UNSUPPORTED;
    st = size_status(k, 16, ep::kMaxExpertChannels);
    if (st != EP_OK) return st;
    st = size_status(n, gated ? 16 : 8, 2 * ep::kMaxExpertChannels);
    if (st != EP_OK) return st;
    const bool rows = has_rows(h);
    if (!w || !w_scale || (rows && (!x || !x_scale || !out))) return EP_ERR_NULL;
    if (!aligned(x, 16) || !aligned(x_scale, 4) || !aligned(w, 16) || !aligned(w_scale, 16) ||
        !aligned(row_weights, 4) || !aligned(out, 16))
        return EP_ERR_MISALIGNED;
    if (!rows) return EP_OK;
    const int64_t outputs = gated ? n / 2 : n, e = h->num_experts;
    const int64_t xr = x_rows(h, token_rows);
    if (clashes<1, 5>({{out, 2 * h->capacity * outputs}},
                      {{x, xr * k}, {x_scale, 4 * xr}, {w, e * n * k}, {w_scale, 4 * e * n},
                       {row_weights, 4 * h->capacity}}))
        return EP_ERR_UNSUPPORTED;
    ep::ExpertArgs a{};
    a.seg = segments(h);
    a.x = x;
    a.token_rows = token_rows != 0;
    a.k = k;
    a.w = w;
    a.n = static_cast<int32_t>(outputs);
    a.x_scale = x_scale;
    a.w_scale = w_scale;
    a.row_weights = row_weights;
    a.out = out;
    return hip_status(ep::launch_expert_i8(a, gated != 0, stream));
}

ep_status ep_expert_ffn(const ep_handle *h, const void *x, int32_t token_rows, int32_t hidden,
                        const void *w13, const void *w2, int32_t inter,
                        const float *row_weights, void *out_h, void *saved, void *out_y,
                        hipStream_t stream) {
    ep_status st = handle_status(h);
    if (st != EP_OK) return st;
    if (token_rows != 0 && token_rows != 1) return EP_ERR_UNSUPPORTED;
    st = size_status(hidden, 8, ep::kMaxExpertChannels);
    if (st != EP_OK) return st;
    st = size_status(inter, 8, ep::kMaxExpertChannels);
    if (st != EP_OK) return st;
    const bool rows = has_rows(h);
    if (!w13 || (rows && (!x || !out_h || !out_y != !w2)) || (out_y && !w2)) return EP_ERR_NULL;
    if (!aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) || !aligned(row_weights, 4) ||
        !aligned(out_h, 16) || !aligned(saved, 16) || !aligned(out_y, 16))
        return EP_ERR_MISALIGNED;
    if (!rows) return EP_OK;
    const int64_t e = h->num_experts, cap = h->capacity;
    const int64_t weight = e * hidden * inter;
    if (clashes<3, 4>({{out_h, 2 * cap * inter}, {saved, 4 * cap * inter}, {out_y, 2 * cap * hidden}},
                      {{x, 2 * x_rows(h, token_rows) * hidden}, {w13, 4 * weight}, {w2, 2 * weight},
                       {row_weights, 4 * cap}}))
        return EP_ERR_UNSUPPORTED;
    ep::ExpertArgs a{};
    a.seg = segments(h);
    a.x = x;
    a.token_rows = token_rows != 0;
    a.k = hidden;
    a.w = w13;
    a.n = inter;
    a.row_weights = row_weights;
    a.out = out_h;
    a.saved = saved;
    const hipError_t err = ep::launch_expert_gated(a, stream);
    if (err != hipSuccess || !out_y) return hip_status(err);
    ep::ExpertArgs b{};
    b.seg = a.seg;
    b.x = out_h;
    b.k = inter;
    b.w = w2;
    b.n = hidden;
    b.out = out_y;
    return hip_status(ep::launch_expert_product(b, stream));
}

size_t ep_expert_ffn_backward_workspace(const ep_handle *h, int32_t inter) {
    if (!h || h->capacity < 0 || size_status(inter, 8, ep::kMaxExpertChannels) != EP_OK) return 0;
    return sizeof(float) * static_cast<size_t>(h->capacity) *
           static_cast<size_t>(ep::gate_grad_tiles(inter));
}

ep_status ep_expert_ffn_backward(const ep_handle *h, const void *grad_y, const void *x,
                                 int32_t token_rows, int32_t hidden, const void *w13,
                                 const void *w2, int32_t inter, const float *row_weights,
                                 const void *saved, void *rows_h, int32_t remake_h,
                                 void *grad_gate_up, void *grad_x, ep_dtype grad_dtype,
                                 void *grad_w13, void *grad_w2, float *grad_row_weights,
                                 void *workspace, size_t ws_bytes, hipStream_t stream) {
    ep_status st = handle_status(h);
    if (st != EP_OK) return st;
    if (grad_dtype != EP_BF16 && grad_dtype != EP_F32) return EP_ERR_DTYPE;
    if ((token_rows != 0 && token_rows != 1) || (remake_h != 0 && remake_h != 1))
        return EP_ERR_UNSUPPORTED;
    st = size_status(hidden, 8, ep::kMaxExpertChannels);
    if (st != EP_OK) return st;
    st = size_status(inter, 8, ep::kMaxExpertChannels);
    if (st != EP_OK) return st;
    const bool rows = has_rows(h);
    if (!w2 || (grad_x && !w13)) return EP_ERR_NULL;
    if (rows && (!grad_y || !saved || !grad_gate_up || (grad_w13 && !x) ||
                 ((grad_w2 || remake_h) && !rows_h)))
        return EP_ERR_NULL;
    if (!aligned(grad_y, 16) || !aligned(x, 16) || !aligned(w13, 16) || !aligned(w2, 16) ||
        !aligned(row_weights, 4) || !aligned(saved, 16) || !aligned(rows_h, 16) ||
        !aligned(grad_gate_up, 16) || !aligned(grad_x, 16) || !aligned(grad_w13, 16) ||
        !aligned(grad_w2, 16) || !aligned(grad_row_weights, 4) || !aligned(workspace, 16))
        return EP_ERR_MISALIGNED;
    const int64_t e = h->num_experts, cap = h->capacity;
    const int64_t weight = e * hidden * inter, wide = grad_dtype == EP_F32 ? 4 : 2;
    const size_t need = grad_row_weights && rows ? ep_expert_ffn_backward_workspace(h, inter) : 0;
    if (need > 0 && (!workspace || ws_bytes < need)) return EP_ERR_WORKSPACE;
    const Span ws{need > 0 ? workspace : nullptr, static_cast<int64_t>(need)};
    const Span gate_up{saved, 4 * cap * inter}, made{rows_h, 2 * cap * inter};
    const Span none{nullptr, 0}, grads{grad_gate_up, 4 * cap * inter};
    const Span outs[] = {{grad_x, 2 * cap * hidden}, {grad_w13, 2 * wide * weight},
                         {grad_w2, wide * weight}, {grad_row_weights, 4 * cap}, ws,
                         remake_h ? made : none};
    const Span ins[] = {{grad_y, 2 * cap * hidden}, {x, 2 * x_rows(h, token_rows) * hidden},
                        {w13, 4 * weight}, {w2, 2 * weight}, {row_weights, 4 * cap},
                        remake_h ? none : made};
    if (clashes(outs, ins) || clash(grads, gate_up, true)) return EP_ERR_UNSUPPORTED;
    for (const Span &s : outs)
        if (clash(s, gate_up) || clash(s, grads)) return EP_ERR_UNSUPPORTED;
    for (const Span &s : ins)
        if (clash(grads, s)) return EP_ERR_UNSUPPORTED;
    hipError_t err = hipSuccess;
    if (rows) {
        ep::ExpertArgs a{};
        a.seg = segments(h);
        a.x = grad_y;
        a.k = hidden;
        a.w = w2;
        a.n = inter;
        a.row_weights = row_weights;
        a.out = remake_h ? rows_h : nullptr;
        a.gate_up = saved;
        a.grad_gate_up = grad_gate_up;
        a.partial = need > 0 ? static_cast<float *>(workspace) : nullptr;
        err = ep::launch_expert_gate_grad(a, grad_row_weights, h->dst_slot, stream);
        if (err == hipSuccess && grad_x) {
            ep::ExpertArgs b{};
            b.seg = a.seg;
            b.x = grad_gate_up;
            b.k = 2 * inter;
            b.w = w13;
            b.n = hidden;
            b.out = grad_x;
            err = ep::launch_expert_grad_rows(b, stream);
        }
    }
    // without rows every gradient of a weight is zero
    auto grad_weight = [&](const void *g, const void *by, int32_t tokens, int32_t n, int32_t k,
                           void *out) {
        if (err != hipSuccess || !out) return;
        ep::GradWeightArgs a{};
        a.seg = segments(h);
        if (!rows) a.seg.capacity = 0;
        a.g = g;
        a.x = by;
        a.token_rows = tokens != 0;
        a.n = n;
        a.k = k;
        a.f32 = grad_dtype == EP_F32;
        a.out = out;
        err = ep::launch_expert_grad_weight(a, stream);
    };
    grad_weight(grad_gate_up, x, token_rows, 2 * inter, hidden, grad_w13);
    grad_weight(grad_y, rows_h, 0, hidden, inter, grad_w2);
    return hip_status(err);
}

}  // extern "C"
