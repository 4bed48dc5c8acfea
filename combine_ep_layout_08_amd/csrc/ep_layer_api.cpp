// C ABI of the layer operators (include/ep_layer.h): argument checks and
// kernel launches.  Nothing here allocates, synchronises or keeps a pointer.
#include "../../include/ep_layer.h"

#include <cmath>

#include "ep_layer_internal.h"

namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

ep_status hip_status(hipError_t e) { return e == hipSuccess ? EP_OK : EP_ERR_HIP; }

bool known_format(ep_sf_format fmt) { return fmt == EP_SF_F32 || fmt == EP_SF_UE8M0; }

// Whether an output and another buffer, both rows of the given bytes, share memory: then
// a row's block would read what another has written.  `same`: the two may start at the same
// address, where each thread reads a place before it writes it.
struct Span {
    const void *p;
    int64_t bytes;
};

bool clash(Span out, Span other, bool same = false) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(out.p),
                    b = reinterpret_cast<uintptr_t>(other.p);
    if (!a || !b || (same && a == b)) return false;
    return a < b + other.bytes && b < a + out.bytes;
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

// Sizes of rows of `channels` channels, of which E4M3 ones come in whole
// blocks of 128.
ep_status channels_status(int32_t channels, bool fp8) {
    if (channels <= 0) return EP_ERR_SHAPE;
    if (channels % (fp8 ? 128 : 8) != 0) return EP_ERR_MISALIGNED;
    return channels <= ep::kMaxLayerHidden ? EP_OK : EP_ERR_UNSUPPORTED;
}

// An E4M3 buffer's scales; `used`: the call reads or writes some.
ep_status scales_status(ep_sf_format fmt, const void *p, int64_t ts, int64_t hs, bool used,
                        ep::Scales *out) {
    if (!known_format(fmt)) return EP_ERR_DTYPE;
    if (ts < 0 || hs < 0) return EP_ERR_SHAPE;
    if (used && !p) return EP_ERR_NULL;
    if (!aligned(p, 4)) return EP_ERR_MISALIGNED;
    out->p = static_cast<uint32_t *>(const_cast<void *>(p));
    out->ts = ts;
    out->hs = hs;
    out->ue8m0 = fmt == EP_SF_UE8M0;
    return EP_OK;
}

ep_status w4_status(int32_t num_experts, int32_t n, int32_t k, ep_w4_format fmt, int32_t group) {
    if (fmt != EP_W4_INT4 && fmt != EP_W4_MXFP4) return EP_ERR_DTYPE;
    if (num_experts < 1 || n < 1 || k < 1) return EP_ERR_SHAPE;
    if (num_experts > ep::kMaxExperts || k > ep::kMaxLayerHidden) return EP_ERR_UNSUPPORTED;
    if (group != 32 && (fmt == EP_W4_MXFP4 || (group != 64 && group != 128)))
        return EP_ERR_UNSUPPORTED;
    if (n % 8 != 0 || k % 128 != 0) return EP_ERR_MISALIGNED;
    return EP_OK;
}

size_t padded_n(int32_t n) { return (static_cast<size_t>(n) + 15) / 16 * 16; }

}  // namespace

extern "C" {

ep_status ep_add_rmsnorm(const void *x, const void *residual, const void *weight,
                         ep_dtype weight_dtype, float eps, int32_t num_tokens, int32_t hidden,
                         void *out_z, void *out_y, ep_sf_format fmt, void *out_q, void *out_sf,
                         int64_t out_sf_token_stride, int64_t out_sf_hidden_stride,
                         float *out_rstd, hipStream_t stream) {
    if (weight_dtype != EP_BF16 && weight_dtype != EP_F32) return EP_ERR_DTYPE;
    if (num_tokens < 0 || !(eps >= 0.0f) || std::isinf(eps)) return EP_ERR_SHAPE;
    ep_status st = channels_status(hidden, out_q != nullptr);
    if (st != EP_OK) return st;
    ep::NormArgs a{};
    if (out_q) {
        st = scales_status(fmt, out_sf, out_sf_token_stride, out_sf_hidden_stride,
                           num_tokens > 0, &a.sf);
        if (st != EP_OK) return st;
    }
    if (num_tokens == 0) return EP_OK;
    if (!x || !weight || (!out_z && !out_y && !out_q && !out_rstd)) return EP_ERR_NULL;
    if (!aligned(x, 16) || !aligned(residual, 16) || !aligned(weight, 16) ||
        !aligned(out_z, 16) || !aligned(out_y, 16) || !aligned(out_q, 16) ||
        !aligned(out_rstd, 4))
        return EP_ERR_MISALIGNED;
    const int64_t codes = static_cast<int64_t>(num_tokens) * hidden;
    const Span ins[] = {{x, 2 * codes}, {residual, 2 * codes}};
    const Span zs{out_z, 2 * codes}, ys{out_y, 2 * codes}, qs{out_q, codes};
    for (const Span &in : ins)
        if (clash(zs, in, true) || clash(ys, in) || clash(qs, in)) return EP_ERR_UNSUPPORTED;
    if (clash(ys, zs) || clash(qs, zs) || clash(qs, ys)) return EP_ERR_UNSUPPORTED;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.weight_bf16 = weight_dtype == EP_BF16;
    a.eps = eps;
    a.num_tokens = num_tokens;
    a.hidden = hidden;
    a.out_z = out_z;
    a.out_y = out_y;
    a.out_q = out_q;
    a.out_rstd = out_rstd;
    return hip_status(ep::launch_add_rmsnorm(a, stream));
}

size_t ep_add_rmsnorm_backward_workspace(int32_t num_tokens, int32_t hidden) {
    if (num_tokens < 0 || channels_status(hidden, false) != EP_OK) return 0;
    return sizeof(float) * static_cast<size_t>(hidden) *
           static_cast<size_t>(ep::norm_grad_blocks(num_tokens));
}

ep_status ep_add_rmsnorm_backward(const void *grad_y, const void *z, const void *weight,
                                  ep_dtype weight_dtype, const float *rstd, const void *grad_z,
                                  int32_t num_tokens, int32_t hidden, void *grad_x,
                                  float *grad_weight, void *workspace, size_t ws_bytes,
                                  hipStream_t stream) {
    if (weight_dtype != EP_BF16 && weight_dtype != EP_F32) return EP_ERR_DTYPE;
    if (num_tokens < 0) return EP_ERR_SHAPE;
    const ep_status st = channels_status(hidden, false);
    if (st != EP_OK) return st;
    if (!aligned(grad_y, 16) || !aligned(z, 16) || !aligned(weight, 16) || !aligned(rstd, 4) ||
        !aligned(grad_z, 16) || !aligned(grad_x, 16) || !aligned(grad_weight, 16) ||
        !aligned(workspace, 16))
        return EP_ERR_MISALIGNED;
    if (num_tokens > 0 && (!grad_y || !z || !weight || !rstd || (!grad_x && !grad_weight)))
        return EP_ERR_NULL;
    const int64_t bytes = 2 * static_cast<int64_t>(num_tokens) * hidden;
    const Span gx{grad_x, bytes};
    if (clash(gx, {grad_y, bytes}, true) || clash(gx, {z, bytes}, true) ||
        clash(gx, {grad_z, bytes}, true))
        return EP_ERR_UNSUPPORTED;
    const size_t need = grad_weight ? ep_add_rmsnorm_backward_workspace(num_tokens, hidden) : 0;
    if (need > 0 && (!workspace || ws_bytes < need)) return EP_ERR_WORKSPACE;
    ep::NormGradArgs a{};
    a.grad_y = grad_y;
    a.z = z;
    a.grad_z = grad_z;
    a.weight = weight;
    a.weight_bf16 = weight_dtype == EP_BF16;
    a.rstd = rstd;
    a.num_tokens = num_tokens;
    a.hidden = hidden;
    a.grad_x = grad_x;
    a.grad_weight = grad_weight;
    a.partial = static_cast<float *>(workspace);
    return hip_status(ep::launch_add_rmsnorm_backward(a, stream));
}

size_t ep_w4_code_bytes(int32_t num_experts, int32_t n, int32_t k) {
    if (w4_status(num_experts, n, k, EP_W4_MXFP4, 32) != EP_OK) return 0;
    return static_cast<size_t>(num_experts) * padded_n(n) * (static_cast<size_t>(k) / 2);
}

size_t ep_w4_scale_bytes(int32_t num_experts, int32_t n, int32_t k, ep_w4_format fmt,
                         int32_t group) {
    if (w4_status(num_experts, n, k, fmt, group) != EP_OK) return 0;
    return static_cast<size_t>(num_experts) * padded_n(n) * static_cast<size_t>(k / group) *
           (fmt == EP_W4_INT4 ? 2 : 1);
}

ep_status ep_w4_pack(const void *codes, const void *scales, int32_t num_experts, int32_t n,
                     int32_t k, ep_w4_format fmt, int32_t group, void *out_codes,
                     void *out_scales, hipStream_t stream) {
    const ep_status st = w4_status(num_experts, n, k, fmt, group);
    if (st != EP_OK) return st;
    if (!codes || !scales || !out_codes || !out_scales) return EP_ERR_NULL;
    if (!aligned(codes, 4) || !aligned(scales, 4) || !aligned(out_codes, 16) ||
        !aligned(out_scales, 16))
        return EP_ERR_MISALIGNED;
    return hip_status(ep::launch_w4_pack(codes, scales, num_experts, n, k, fmt, group, out_codes,
                                         out_scales, stream));
}

ep_status ep_expert_w4(const ep_handle *h, const void *x, ep_dtype x_dtype, int32_t token_rows,
                       int32_t k, const void *sf, ep_sf_format sf_fmt, int64_t sf_token_stride,
                       int64_t sf_hidden_stride, const void *codes, const void *scales,
                       ep_w4_format fmt, int32_t group, int32_t n, void *out,
                       hipStream_t stream) {
    ep_status st = handle_status(h);
    if (st != EP_OK) return st;
    if (x_dtype != EP_BF16 && x_dtype != EP_FP8_E4M3) return EP_ERR_DTYPE;
    if (token_rows != 0 && token_rows != 1) return EP_ERR_UNSUPPORTED;
    st = w4_status(h->num_experts, n, k, fmt, group);
    if (st != EP_OK) return st;
    const bool fp8 = x_dtype == EP_FP8_E4M3;
    const bool rows = h->num_tokens > 0 && h->capacity > 0;
    ep::W4Args a{};
    if (fp8) {
        st = scales_status(sf_fmt, sf, sf_token_stride, sf_hidden_stride, rows, &a.sf);
        if (st != EP_OK) return st;
    } else if (sf) {
        return EP_ERR_DTYPE;
    }
    if (!codes || !scales || (rows && (!x || !out))) return EP_ERR_NULL;
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(out, 16))
        return EP_ERR_MISALIGNED;
    if (!rows) return EP_OK;
    const int64_t x_rows = token_rows ? h->num_tokens : h->capacity;
    if (clash({out, 2 * int64_t(h->capacity) * n}, {x, x_rows * k * (fp8 ? 1 : 2)}))
        return EP_ERR_UNSUPPORTED;
    a.counts = h->counts;
    a.psum = h->psum;
    a.src_meta = h->src_meta;
    a.scalars = h->scalars;
    a.num_experts = h->num_experts;
    a.num_topk = h->num_topk;
    a.num_tokens = h->num_tokens;
    a.capacity = h->capacity;
    a.x = x;
    a.x_fp8 = fp8;
    a.token_rows = token_rows != 0;
    a.k = k;
    a.n = n;
    a.codes = codes;
    a.scales = scales;
    a.fmt = fmt;
    a.group = group;
    a.out = out;
    return hip_status(ep::launch_expert_w4(a, stream));
}

ep_status ep_swiglu(const ep_handle *h, const void *gate_up, int32_t inter,
                    const float *row_weights, ep_dtype h_dtype, void *out_h, ep_sf_format fmt,
                    void *out_sf, int64_t out_sf_token_stride, int64_t out_sf_hidden_stride,
                    void *saved, ep_sf_format saved_fmt, void *saved_sf,
                    int64_t saved_sf_token_stride, int64_t saved_sf_hidden_stride,
                    hipStream_t stream) {
    ep_status st = handle_status(h);
    if (st != EP_OK) return st;
    if (h_dtype != EP_BF16 && h_dtype != EP_FP8_E4M3) return EP_ERR_DTYPE;
    const bool h_fp8 = h_dtype == EP_FP8_E4M3;
    st = channels_status(inter, h_fp8 || saved);
    if (st != EP_OK) return st;
    const bool rows = h->num_tokens > 0 && h->capacity > 0;
    ep::ActArgs a{};
    if (h_fp8) {
        st = scales_status(fmt, out_sf, out_sf_token_stride, out_sf_hidden_stride, rows, &a.h_sf);
        if (st != EP_OK) return st;
    } else if (out_sf) {
        return EP_ERR_DTYPE;
    }
    if (saved) {
        st = scales_status(saved_fmt, saved_sf, saved_sf_token_stride, saved_sf_hidden_stride,
                           rows, &a.saved_sf);
        if (st != EP_OK) return st;
    } else if (saved_sf) {
        return EP_ERR_NULL;
    }
    if (rows && (!gate_up || !out_h)) return EP_ERR_NULL;
    if (!aligned(gate_up, 16) || !aligned(row_weights, 4) || !aligned(out_h, 16) ||
        !aligned(saved, 16))
        return EP_ERR_MISALIGNED;
    if (!rows) return EP_OK;
    const int64_t part = static_cast<int64_t>(h->capacity) * inter;
    const Span in{gate_up, 4 * part}, hs{out_h, part * (h_fp8 ? 1 : 2)}, ss{saved, 2 * part};
    if (clash(hs, in) || clash(ss, in) || clash(ss, hs)) return EP_ERR_UNSUPPORTED;
    a.dst = h->dst_slot;
    a.scalars = h->scalars;
    a.num_slots = static_cast<int64_t>(h->num_tokens) * h->num_topk;
    a.capacity = h->capacity;
    a.gate_up = gate_up;
    a.inter = inter;
    a.row_weights = row_weights;
    a.out_h = out_h;
    a.h_fp8 = h_fp8;
    a.saved = saved;
    return hip_status(ep::launch_swiglu(a, stream));
}

ep_status ep_swiglu_backward(const ep_handle *h, const void *grad_h, int32_t inter,
                             const float *row_weights, const void *saved, ep_dtype saved_dtype,
                             ep_sf_format saved_fmt, const void *saved_sf,
                             int64_t saved_sf_token_stride, int64_t saved_sf_hidden_stride,
                             void *grad_gate_up, float *grad_row_weights, void *out_h,
                             hipStream_t stream) {
    ep_status st = handle_status(h);
    if (st != EP_OK) return st;
    if (saved_dtype != EP_BF16 && saved_dtype != EP_FP8_E4M3) return EP_ERR_DTYPE;
    const bool fp8 = saved_dtype == EP_FP8_E4M3;
    st = channels_status(inter, fp8);
    if (st != EP_OK) return st;
    const bool rows = h->num_tokens > 0 && h->capacity > 0;
    ep::ActGradArgs a{};
    if (fp8) {
        st = scales_status(saved_fmt, saved_sf, saved_sf_token_stride, saved_sf_hidden_stride,
                           rows, &a.saved_sf);
        if (st != EP_OK) return st;
    } else if (saved_sf) {
        return EP_ERR_DTYPE;
    }
    if (rows && (!grad_h || !saved || !grad_gate_up)) return EP_ERR_NULL;
    if (!aligned(grad_h, 16) || !aligned(row_weights, 4) || !aligned(saved, 16) ||
        !aligned(grad_gate_up, 16) || !aligned(grad_row_weights, 4) || !aligned(out_h, 16))
        return EP_ERR_MISALIGNED;
    if (!rows) return EP_OK;
    const int64_t part = static_cast<int64_t>(h->capacity) * inter;
    const Span gh{grad_h, 2 * part}, in{saved, part * (fp8 ? 2 : 4)};
    const Span gg{grad_gate_up, 4 * part}, hs{out_h, 2 * part};
    if (clash(gg, gh) || clash(gg, in, !fp8) || clash(hs, gh, true) || clash(hs, in) ||
        clash(hs, gg))
        return EP_ERR_UNSUPPORTED;
    a.dst = h->dst_slot;
    a.scalars = h->scalars;
    a.num_slots = static_cast<int64_t>(h->num_tokens) * h->num_topk;
    a.capacity = h->capacity;
    a.grad_h = grad_h;
    a.inter = inter;
    a.row_weights = row_weights;
    a.saved = saved;
    a.saved_fp8 = fp8;
    a.grad_gate_up = grad_gate_up;
    a.grad_row_weights = grad_row_weights;
    a.out_h = out_h;
    return hip_status(ep::launch_swiglu_backward(a, stream));
}

}  // extern "C"
