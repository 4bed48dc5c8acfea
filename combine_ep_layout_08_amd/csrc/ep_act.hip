// Gated activation of the expert rows with its 8-bit checkpoint, and its
// gradient, on gfx950 (include/ep_layer.h: ep_swiglu, ep_swiglu_backward).
#include "ep_layer_internal.h"
#include "ep_rows.h"

namespace ep {
namespace {

constexpr int kActThreads = 256;
constexpr int kActWaves = kActThreads / 64;
constexpr int64_t kActRows = 4096;       // rows from which a wave takes a whole one
constexpr int64_t kActBlocks = 1 << 22;  // most blocks of a launch; they walk the work behind

dim3 act_grid(int64_t waves) {
    const int64_t blocks = (waves + kActWaves - 1) / kActWaves;
    return dim3(static_cast<uint32_t>(blocks < kActBlocks ? blocks : kActBlocks));
}

// Exponent bytes of gate's and up's block b into a row of 2 * blocks bytes: up's
// need not start at a pack, so every block stores its own byte; the bytes behind the
// last block are zero.
__device__ inline void store_bytes(const Scales &sf, int64_t row, int b, int blocks,
                                   uint32_t gate, uint32_t up, int lane) {
    if ((lane & 15) != 0 || b >= blocks) return;
    char *base = reinterpret_cast<char *>(sf.p + row * sf.ts);
    auto store = [&](int i, uint32_t e) {
        base[4 * ((i >> 2) * sf.hs) + (i & 3)] = static_cast<char>(e);
    };
    store(b, gate);
    store(blocks + b, up);
    if (b == blocks - 1)
        for (int i = 2 * blocks; i & 3; ++i) store(i, 0);
}

// Row of slot i, or -1 where the slot is empty, outside the buffers, or the
// layout on the handle is void.  Slots and not rows are walked: every slot has a
// row, while gaps and the room behind the last row would have to be looked at (walked in
// memory order 32768 of 65280 rows took 113 us instead of 103, a decode batch 20 instead of 5).
__device__ inline int64_t slot_row(const int32_t *dst, const int32_t *scalars, int64_t i,
                                   int64_t capacity) {
    const int32_t r = dst[i];
    const uint32_t bits = static_cast<uint32_t>(scalars[EP_SCALAR_ERROR_BITS]);
    return r < 0 || r >= capacity || (bits & EP_ERRBIT_FATAL) ? -1 : r;
}

// One wave for a slot's row, 512 channels a step, 8 a lane: a row of 16 lanes is
// one scale block of gate, of up and of h.  gridDim.y waves share a row.
template <int HFMT, int SFMT>
__global__ __launch_bounds__(kActThreads) void act_kernel(const ActArgs a) {
#pragma clang fp contract(off)
    const int lane = threadIdx.x & 63;
    const int V = a.inter / 8, chunks = (V + 63) / 64, blocks = a.inter / 128;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kActWaves;
    for (int64_t slot = static_cast<int64_t>(blockIdx.x) * kActWaves +
                        __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
         slot < a.num_slots; slot += stride) {
        const int64_t row = slot_row(a.dst, a.scalars, slot, a.capacity);
        if (row < 0) continue;
        const float w = a.row_weights ? a.row_weights[row] : 1.0f;
        const u32x4 *src = static_cast<const u32x4 *>(a.gate_up) + row * 2 * V;
        for (int chunk = blockIdx.y; chunk < chunks; chunk += gridDim.y) {
            const int v = chunk * 64 + lane;
            const bool in = v < V;
            u32x4 gv = u32x4{0u, 0u, 0u, 0u}, uv = gv;
            if (in) {
                gv = src[v];
                uv = src[V + v];
            }
            float g[8], u[8], h[8];
            unpack8(gv, g);
            unpack8(uv, u);
#pragma unroll
            for (int j = 0; j < 8; ++j) h[j] = g[j] * sigmoid(g[j]) * u[j] * w;
            const int b0 = chunk * 4;
            uint32_t pack;
            if (HFMT == kSfNone) {
                if (in) (static_cast<u32x4 *>(a.out_h) + row * V)[v] = pack8(h);
            }
            uint32_t gm = 0, um = 0;
            if (SFMT != kSfNone) {
                constexpr int F = SFMT == kSfNone ? EP_SF_F32 : SFMT;
                gm = block_max_bits(gv);
                um = block_max_bits(uv);
                u32x2 *dst = static_cast<u32x2 *>(a.saved) + row * 2 * V;
                u32x2 q = e4m3_block8<F>(g, gm, &pack);
                const uint32_t gp = pack;
                if (in) dst[v] = q;
                q = e4m3_block8<F>(u, um, &pack);
                if (in) dst[V + v] = q;
                if (F == EP_SF_F32) {
                    store_packs<F>(a.saved_sf.p, a.saved_sf.ts, a.saved_sf.hs, row, b0, blocks, gp,
                                   lane);
                    const int b = b0 + (lane >> 4);
                    if ((lane & 15) == 0 && b < blocks)
                        a.saved_sf.p[row * a.saved_sf.ts + (blocks + b) * a.saved_sf.hs] = pack;
                } else {
                    store_bytes(a.saved_sf, row, b0 + (lane >> 4), blocks, gp, pack, lane);
                }
            }
            if (HFMT != kSfNone) {
                constexpr int F = HFMT == kSfNone ? EP_SF_F32 : HFMT;
                // with finite factors whose product stays finite h is finite too,
                // and its maximum takes half the operations
                const bool finite = SFMT != kSfNone &&
                    __builtin_fabsf(__uint_as_float(gm) * __uint_as_float(um)) < 3.4e38f &&
                    __builtin_fabsf(w) <= 1.0f;
                const uint32_t hm = finite ? finite_max_bits(h) : block_max_bits(h);
                const u32x2 q = e4m3_block8<F>(h, hm, &pack);
                if (in) (static_cast<u32x2 *>(a.out_h) + row * V)[v] = q;
                store_packs<F>(a.h_sf.p, a.h_sf.ts, a.h_sf.hs, row, b0, blocks, pack, lane);
            }
        }
    }
}

template <int HFMT>
hipError_t launch_act(const ActArgs &a, hipStream_t stream) {
    // Few rows: a wave for every 512 channels; many: one a row, which reads the slot and
    // the row weight once.
    const int chunks = (a.inter / 8 + 63) / 64;
    const bool few = a.num_slots < kActRows;
    dim3 grid = act_grid(a.num_slots);
    grid.y = few ? chunks : 1;
    const dim3 block(kActThreads);
    if (!a.saved) act_kernel<HFMT, kSfNone><<<grid, block, 0, stream>>>(a);
    else if (a.saved_sf.ue8m0) act_kernel<HFMT, EP_SF_UE8M0><<<grid, block, 0, stream>>>(a);
    else act_kernel<HFMT, EP_SF_F32><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

// One wave a slot's row, 512 channels a step, so the row weight's gradient is
// one wave's sum.
template <bool FP8>
__global__ __launch_bounds__(kActThreads) void act_grad_kernel(const ActGradArgs a) {
    const int lane = threadIdx.x & 63;
    const int V = a.inter / 8, blocks = a.inter / 128;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * kActWaves;
    for (int64_t slot = static_cast<int64_t>(blockIdx.x) * kActWaves + (threadIdx.x >> 6);
         slot < a.num_slots; slot += stride) {
        const int64_t row = slot_row(a.dst, a.scalars, slot, a.capacity);
        if (row < 0) continue;
        const float w = a.row_weights ? a.row_weights[row] : 1.0f;
        float total = 0.0f;
        for (int v = lane; v < V; v += 64) {
            float g[8], u[8], gh[8];
            unpack8((static_cast<const u32x4 *>(a.grad_h) + row * V)[v], gh);
            if (FP8) {
                const u32x2 *src = static_cast<const u32x2 *>(a.saved) + row * 2 * V;
                const u32x2 gq = src[v], uq = src[V + v];
                const float gs = load_scale(a.saved_sf.p, a.saved_sf.ts, a.saved_sf.hs, row, v >> 4,
                                            a.saved_sf.ue8m0);
                const float us = load_scale(a.saved_sf.p, a.saved_sf.ts, a.saved_sf.hs, row,
                                            blocks + (v >> 4), a.saved_sf.ue8m0);
                e4m3_values4(gq.x, g);
                e4m3_values4(gq.y, g + 4);
                e4m3_values4(uq.x, u);
                e4m3_values4(uq.y, u + 4);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    g[j] *= gs;
                    u[j] *= us;
                }
            } else {
                const u32x4 *src = static_cast<const u32x4 *>(a.saved) + row * 2 * V;
                unpack8(src[v], g);
                unpack8(src[V + v], u);
            }
            float og[8], ou[8], oh[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float s = sigmoid(g[j]);
                const float silu = g[j] * s;
                const float whole = silu * u[j];
                total = __builtin_fmaf(gh[j], whole, total);
                const float wg = w * gh[j];
                const float slope = s * __builtin_fmaf(g[j], 1.0f - s, 1.0f);
                og[j] = wg * u[j] * slope;
                ou[j] = wg * silu;
                oh[j] = w * whole;
            }
            u32x4 *dst = static_cast<u32x4 *>(a.grad_gate_up) + row * 2 * V;
            dst[v] = pack8(og);
            dst[V + v] = pack8(ou);
            if (a.out_h) (static_cast<u32x4 *>(a.out_h) + row * V)[v] = pack8(oh);
        }
        if (!a.grad_row_weights) continue;
        total = wave_sum(total);
        if (lane == 0) a.grad_row_weights[row] = total;
    }
}

}  // namespace

hipError_t launch_swiglu(const ActArgs &a, hipStream_t stream) {
    if (!a.h_fp8) return launch_act<kSfNone>(a, stream);
    return a.h_sf.ue8m0 ? launch_act<EP_SF_UE8M0>(a, stream) : launch_act<EP_SF_F32>(a, stream);
}

hipError_t launch_swiglu_backward(const ActGradArgs &a, hipStream_t stream) {
    const dim3 grid = act_grid(a.num_slots), block(kActThreads);
    if (a.saved_fp8) act_grad_kernel<true><<<grid, block, 0, stream>>>(a);
    else act_grad_kernel<false><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace ep
