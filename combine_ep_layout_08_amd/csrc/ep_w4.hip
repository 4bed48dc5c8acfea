// Products of the expert rows with 4-bit weights on gfx950
// (include/ep_layer.h: ep_w4_pack, ep_expert_w4).
//
// out[r, :] = x[r, :] . W[e]^T for the rows r of expert e, as matrix
// instructions of 16 rows x 16 outputs x 32 channels (v_mfma_f32_16x16x32_bf16;
// lane l holds row l % 16 of x, output l % 16 of W, channels 8 (l / 16) .. + 7 of
// each, and accumulates rows 4 (l / 16) .. + 3 of output l % 16).
//
// Packed weights: for every expert, tile of 16 outputs and step of 128
// channels, one record of 1 KB: lane l's 16 bytes at 16 l, dword j the eight
// codes of output l % 16, channels 32 j + 8 (l / 16) .. + 7, which is what lane l
// feeds to the j-th matrix instruction.  A wave reads a record in one load
// of consecutive addresses, and a tile's records follow each other.  Codes of
// EP_W4_INT4 are stored with channel 2i in nibble i and 2i + 1 in nibble i + 4, so
// that one shift and one and-or make a pair of bf16: 0x4300 | code is 128 + code
// exactly.  The 136 = 128 + 8 is taken off again by a product of x with the
// constant -136, which starts the same accumulator.  EP_W4_MXFP4 codes keep
// their order and become bf16 pairs, scaled, by v_cvt_scalef32_pk_bf16_fp4
// (exact: E2M1 times a power of two).
// Scales: [expert][tile][step][output][128 / group], so a lane's scales of a step
// are consecutive.
#include "ep_layer_internal.h"
#include "ep_rows.h"

namespace ep {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kMinus136 = 0xC308C308u;     // a pair of bf16

__device__ inline f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                   __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}

// Eight codes as 128 + code in bf16.
__device__ inline u32x4 int4_plus128(uint32_t w) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
    return o;
}

// Eight E2M1 codes times 2^(e - 127) in bf16; e = 255 gives NaN.
__device__ inline u32x4 mxfp4(uint32_t w, uint32_t e) {
    const float s = __uint_as_float(e == 0 ? 0x00400000u : e << 23);
    u32x4 o;
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    return o;
}

// Eight E4M3 codes as bf16 (exact).
__device__ inline u32x4 e4m3_bf16(u32x2 w) {
    u32x4 o;
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, 1.0f, false));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.x, 1.0f, true));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, 1.0f, false));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w.y, 1.0f, true));
    return o;
}

// ---------------------------------------------------------------- layout
// One thread a dword of the packed codes.
__global__ __launch_bounds__(256) void pack_codes_kernel(const uint8_t *codes, int64_t experts,
                                                         int n, int k, bool int4, uint32_t *out) {
    const int tiles = (n + 15) / 16, steps = k / 128;
    const int64_t total = experts * tiles * steps * 256;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += stride) {
        const int j = static_cast<int>(i & 3), lane = static_cast<int>(i >> 2) & 63;
        const int64_t record = i >> 8;
        const int64_t e = record / (static_cast<int64_t>(tiles) * steps);
        const int tile = static_cast<int>(record / steps % tiles);
        const int row = tile * 16 + (lane & 15);
        const int ch = static_cast<int>(record % steps) * 128 + 32 * j + 8 * (lane >> 4);
        uint32_t w = int4 ? 0x88888888u : 0u;                  // zeros
        if (row < n)
            w = *reinterpret_cast<const uint32_t *>(codes + (e * n + row) * (k / 2) + ch / 2);
        if (int4) {
            uint32_t o = 0;
#pragma unroll
            for (int c = 0; c < 8; ++c)
                o |= ((w >> (4 * c)) & 0xFu) << (4 * (c / 2 + 4 * (c & 1)));
            w = o;
        }
        out[i] = w;
    }
}

// One thread a scale; U: its bytes.
template <typename U>
__global__ __launch_bounds__(256) void pack_scales_kernel(const U *scales, int64_t experts, int n,
                                                          int groups, int per_step, U *out) {
    const int tiles = (n + 15) / 16, steps = groups / per_step;
    const int64_t total = experts * tiles * 16 * groups;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += stride) {
        const int g = static_cast<int>(i % per_step);
        const int64_t at = i / per_step;
        const int64_t record = at >> 4;
        const int64_t e = record / (static_cast<int64_t>(tiles) * steps);
        const int row = static_cast<int>(record / steps % tiles) * 16 + static_cast<int>(at & 15);
        const int group = static_cast<int>(record % steps) * per_step + g;
        out[i] = row < n ? scales[(e * n + row) * groups + group] : U(0);
    }
}

// ---------------------------------------------------------------- product
// The expert with the a-th smallest index among those that have rows (-1 if
// fewer have), its first row and its rows' count.  Every lane calls this.
__device__ inline int active_expert(const int32_t *counts, const int32_t *psum, int experts, int a,
                                    int lane, int *start, int *rows) {
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int e = e0 + lane;
        const int32_t c = e < experts ? counts[e] : 0;
        const int32_t p = e < experts ? psum[e] : 0;
        uint64_t some = __ballot(c > 0);
        const int n = __popcll(some);
        if (a >= n) {
            a -= n;
            continue;
        }
        for (; a > 0; --a) some &= some - 1;
        const int l = __ffsll(static_cast<unsigned long long>(some)) - 1;
        *start = __builtin_amdgcn_readlane(p, l);
        *rows = __builtin_amdgcn_readlane(c, l);
        return e0 + l;
    }
    return -1;
}

constexpr int kW4Threads = 256;

// One wave for a tile of 16 outputs of one expert, 16 rows at a time.
template <int FMT, int GROUP, bool FP8>
__global__ __launch_bounds__(kW4Threads) void w4_kernel(const W4Args a) {
    const int lane = threadIdx.x & 63, q = lane >> 4;
    const int tiles = (a.n + 15) / 16, steps = a.k / 128;
    const int tile = blockIdx.x * (kW4Threads / 64) + (threadIdx.x >> 6);
    if (tile >= tiles) return;
    if (static_cast<uint32_t>(a.scalars[EP_SCALAR_ERROR_BITS]) & EP_ERRBIT_FATAL) return;
    int start, rows;
    const int e = active_expert(a.counts, a.psum, a.num_experts, blockIdx.y, lane, &start, &rows);
    if (e < 0) return;
    constexpr int kPer = 128 / GROUP;
    const int64_t record = (static_cast<int64_t>(e) * tiles + tile) * steps;
    const u32x4 *codes = static_cast<const u32x4 *>(a.codes) + record * 64 + lane;
    const char *scales = static_cast<const char *>(a.scales) +
                         (record * 16 + (lane & 15)) * kPer * (FMT == EP_W4_INT4 ? 2 : 1);
    const int out_col = tile * 16 + (lane & 15);
    for (int m0 = 0; m0 < rows; m0 += 16) {
        const int m = m0 + (lane & 15) < rows ? m0 + (lane & 15) : rows - 1;
        const int64_t row = start + m;
        const int64_t src = a.token_rows ? a.src_meta[row] / a.num_topk : row;
        const char *x = static_cast<const char *>(a.x) + (src * a.k + 8 * q) * (FP8 ? 1 : 2);
        f32x4 total = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < steps; ++s) {
            const u32x4 w = codes[static_cast<int64_t>(s) * 64];
            u32x4 xs[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (FP8) xs[j] = e4m3_bf16(*reinterpret_cast<const u32x2 *>(x + s * 128 + 32 * j));
                else xs[j] = *reinterpret_cast<const u32x4 *>(x + (s * 128 + 32 * j) * 2);
            }
            f32x4 part = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if (FMT == EP_W4_MXFP4) {
                const uint32_t sc = *reinterpret_cast<const uint32_t *>(scales + s * 64);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    part = mfma(xs[j], mxfp4(w[j], (sc >> (8 * j)) & 0xFFu), part);
            } else {
                const uint16_t *sc = reinterpret_cast<const uint16_t *>(scales + s * 32 * kPer);
#pragma unroll
                for (int g = 0; g < kPer; ++g) {
                    f32x4 acc = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int j = g * 4 / kPer; j < (g + 1) * 4 / kPer; ++j) {
                        acc = mfma(xs[j], u32x4{kMinus136, kMinus136, kMinus136, kMinus136}, acc);
                        acc = mfma(xs[j], int4_plus128(w[j]), acc);
                    }
                    const float f = __uint_as_float(static_cast<uint32_t>(sc[g]) << 16);
#pragma unroll
                    for (int i = 0; i < 4; ++i) part[i] = __builtin_fmaf(f, acc[i], part[i]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (FP8) {
                    const int mi = m0 + 4 * q + i;
                    const int64_t ri = start + (mi < rows ? mi : rows - 1);
                    const int64_t si = a.token_rows ? a.src_meta[ri] / a.num_topk : ri;
                    total[i] = __builtin_fmaf(
                        load_scale(a.sf.p, a.sf.ts, a.sf.hs, si, s, a.sf.ue8m0), part[i], total[i]);
                } else {
                    total[i] += part[i];
                }
            }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int mi = m0 + 4 * q + i;
            if (mi < rows && out_col < a.n)
                static_cast<uint16_t *>(a.out)[static_cast<int64_t>(start + mi) * a.n + out_col] =
                    static_cast<uint16_t>(pack2(total[i], 0.0f));
        }
    }
}

template <int FMT, int GROUP>
hipError_t launch_w4(const W4Args &a, hipStream_t stream) {
    const int tiles = (a.n + 15) / 16;
    const int64_t slots = static_cast<int64_t>(a.num_tokens) * a.num_topk;
    const int active = static_cast<int>(slots < a.num_experts ? slots : a.num_experts);
    const dim3 grid((tiles + 3) / 4, active), block(kW4Threads);
    if (a.x_fp8) w4_kernel<FMT, GROUP, true><<<grid, block, 0, stream>>>(a);
    else w4_kernel<FMT, GROUP, false><<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_w4_pack(const void *codes, const void *scales, int32_t num_experts, int32_t n,
                          int32_t k, int32_t fmt, int32_t group, void *out_codes,
                          void *out_scales, hipStream_t stream) {
    const bool int4 = fmt == EP_W4_INT4;
    pack_codes_kernel<<<4096, 256, 0, stream>>>(static_cast<const uint8_t *>(codes), num_experts,
                                                n, k, int4, static_cast<uint32_t *>(out_codes));
    if (int4)
        pack_scales_kernel<uint16_t><<<1024, 256, 0, stream>>>(
            static_cast<const uint16_t *>(scales), num_experts, n, k / group, 128 / group,
            static_cast<uint16_t *>(out_scales));
    else
        pack_scales_kernel<uint8_t><<<1024, 256, 0, stream>>>(
            static_cast<const uint8_t *>(scales), num_experts, n, k / group, 128 / group,
            static_cast<uint8_t *>(out_scales));
    return hipGetLastError();
}

hipError_t launch_expert_w4(const W4Args &a, hipStream_t stream) {
    if (a.fmt == EP_W4_MXFP4) return launch_w4<EP_W4_MXFP4, 32>(a, stream);
    if (a.group == 32) return launch_w4<EP_W4_INT4, 32>(a, stream);
    if (a.group == 64) return launch_w4<EP_W4_INT4, 64>(a, stream);
    return launch_w4<EP_W4_INT4, 128>(a, stream);
}

}  // namespace ep
