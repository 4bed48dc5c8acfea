// Kernel arguments and launches of the layer operators (include/ep_layer.h).
#pragma once

#include "../../include/ep_layer.h"
#include "ep_internal.h"

namespace ep {

constexpr int kMaxLayerHidden = 32768;   // channels of a norm, activation or product row

// A scale buffer: 4-byte packs with a token and a pack stride.
struct Scales {
    uint32_t *p = nullptr;
    int64_t ts = 0, hs = 0;
    bool ue8m0 = false;
};

struct NormArgs {
    const void *x, *residual;    // bf16 [T, H]; residual may be null
    const void *weight;
    bool weight_bf16;
    float eps;
    int32_t num_tokens, hidden;
    void *out_z, *out_y;         // bf16 [T, H] or null
    void *out_q;                 // E4M3 [T, H] or null
    Scales sf;
    float *out_rstd;             // [T] or null
};

struct NormGradArgs {
    const void *grad_y, *z, *grad_z;
    const void *weight;
    bool weight_bf16;
    const float *rstd;
    int32_t num_tokens, hidden;
    void *grad_x;                // bf16 [T, H] or null
    float *grad_weight;          // [H] or null
    float *partial;              // [norm_grad_blocks, H] sums of grad_weight
};

struct ActArgs {
    const int32_t *dst, *scalars;
    int64_t num_slots, capacity;
    const void *gate_up;         // bf16 [capacity, 2 inter]
    int32_t inter;
    const float *row_weights;
    void *out_h;                 // bf16 or E4M3 [capacity, inter]
    bool h_fp8;
    Scales h_sf;
    void *saved;                 // E4M3 [capacity, 2 inter] or null
    Scales saved_sf;
};

struct ActGradArgs {
    const int32_t *dst, *scalars;
    int64_t num_slots, capacity;
    const void *grad_h;          // bf16 [capacity, inter]
    int32_t inter;
    const float *row_weights;
    const void *saved;           // bf16 or E4M3 [capacity, 2 inter]
    bool saved_fp8;
    Scales saved_sf;
    void *grad_gate_up;          // bf16 [capacity, 2 inter]
    float *grad_row_weights;     // [capacity] or null
    void *out_h;                 // bf16 [capacity, inter] or null
};

struct W4Args {
    const int32_t *counts, *psum, *src_meta, *scalars;
    int32_t num_experts, num_topk, num_tokens;
    int64_t capacity;
    const void *x;
    bool x_fp8, token_rows;
    Scales sf;
    int32_t k, n;
    const void *codes, *scales;
    int32_t fmt, group;
    void *out;                   // bf16 [capacity, n]
};

// Blocks whose sums of grad_weight the workspace holds (0: none are kept).
int norm_grad_blocks(int32_t num_tokens);

hipError_t launch_add_rmsnorm(const NormArgs &a, hipStream_t stream);
hipError_t launch_add_rmsnorm_backward(const NormGradArgs &a, hipStream_t stream);
hipError_t launch_swiglu(const ActArgs &a, hipStream_t stream);
hipError_t launch_swiglu_backward(const ActGradArgs &a, hipStream_t stream);
hipError_t launch_w4_pack(const void *codes, const void *scales, int32_t num_experts, int32_t n,
                          int32_t k, int32_t fmt, int32_t group, void *out_codes,
                          void *out_scales, hipStream_t stream);
hipError_t launch_expert_w4(const W4Args &a, hipStream_t stream);

}  // namespace ep
