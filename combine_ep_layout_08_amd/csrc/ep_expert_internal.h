// Kernel arguments and launches of the experts' products (include/ep_expert.h).
#pragma once

#include "../../include/ep_expert.h"
#include "ep_internal.h"

namespace ep {

constexpr int kMaxExpertChannels = 32768;    // of x, h and y

struct QuantI8Args {
    const int32_t *dst, *scalars;            // null: all rows
    int64_t num_rows;                        // or slots
    int64_t capacity;
    const void *x;
    int32_t channels;
    void *q;
    float *scale;
};

// What the tiles of every product on expert rows need of the handle.
struct Segments {
    const int32_t *counts, *psum, *src_meta, *scalars;
    int32_t num_experts, num_topk, num_tokens;
    int64_t capacity;
};

struct ExpertArgs {
    Segments seg;
    const void *x;                           // rows that are multiplied
    bool token_rows;
    int32_t k;                               // channels that are summed
    const void *w;
    int32_t n;                               // outputs (gated: of the activation)
    const float *x_scale, *w_scale;          // int8
    const float *row_weights;
    void *out;                               // bf16 [capacity, n]
    void *saved;                             // gated: bf16 [capacity, 2 n] or null
    // the activation's gradient
    const void *gate_up;                     // bf16 [capacity, 2 n]
    void *grad_gate_up;                      // bf16 [capacity, 2 n]
    float *partial;                          // [waves' columns, capacity] or null
};

struct GradWeightArgs {
    Segments seg;
    const void *g;                           // bf16 [capacity, n]
    const void *x;                           // bf16 rows of k channels
    bool token_rows;
    int32_t n, k;
    bool f32;
    void *out;                               // [E, n, k]
};

// At most so many waves' columns the gradient of `inter` activations is made in: a row has a
// sum of each for the gradient of its weight.
int gate_grad_tiles(int32_t inter);

hipError_t launch_quantize_i8(const QuantI8Args &a, hipStream_t stream);
hipError_t launch_expert_i8(const ExpertArgs &a, bool gated, hipStream_t stream);
hipError_t launch_expert_gated(const ExpertArgs &a, hipStream_t stream);
hipError_t launch_expert_product(const ExpertArgs &a, hipStream_t stream);
hipError_t launch_expert_gate_grad(const ExpertArgs &a, float *grad_row_weights, const int32_t *dst,
                                   hipStream_t stream);
hipError_t launch_expert_grad_rows(const ExpertArgs &a, hipStream_t stream);
hipError_t launch_expert_grad_weight(const GradWeightArgs &a, hipStream_t stream);

}  // namespace ep
