// Device helpers of the layer operators: bf16 and E4M3 rows in 16-byte
// vectors, block scales, and sums over a wave.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "ep_internal.h"

namespace ep {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr int kSfNone = -1;   // no E4M3 output; otherwise an ep_sf_format

__device__ inline float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ inline float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ inline void unpack8(const u32x4 v, float f[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(v[i]);
        f[2 * i + 1] = bf16_hi(v[i]);
    }
}

// Two floats to packed bf16, nearest even (one v_cvt_pk_bf16_f32).
__device__ inline uint32_t pack2(float a, float b) {
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{a, b}), bf16x2));
}

__device__ inline u32x4 pack8(const float f[8]) {
    return u32x4{pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7])};
}

// Rotation by N within each row of 16 lanes.
template <int N>
__device__ inline uint32_t row_ror(uint32_t v) {
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(
        0, static_cast<int>(v), 0x120 | N, 0xF, 0xF, false));
}

// Largest value over each row of 16 lanes (a block of 128 channels, 8 a lane).
__device__ inline uint32_t row_max(uint32_t v) {
    uint32_t o;
    o = row_ror<8>(v); v = o > v ? o : v;
    o = row_ror<4>(v); v = o > v ? o : v;
    o = row_ror<2>(v); v = o > v ? o : v;
    o = row_ror<1>(v); v = o > v ? o : v;
    return v;
}

__device__ inline float row_sum(float v) {
    v += __uint_as_float(row_ror<8>(__float_as_uint(v)));
    v += __uint_as_float(row_ror<4>(__float_as_uint(v)));
    v += __uint_as_float(row_ror<2>(__float_as_uint(v)));
    v += __uint_as_float(row_ror<1>(__float_as_uint(v)));
    return v;
}

__device__ inline float lane_value(float v, int lane) {
    return __uint_as_float(static_cast<uint32_t>(
        __builtin_amdgcn_readlane(static_cast<int>(__float_as_uint(v)), lane)));
}

// Sum over the wave, the same in every lane.
__device__ inline float wave_sum(float v) {
    v = row_sum(v);
    return (lane_value(v, 0) + lane_value(v, 16)) + (lane_value(v, 32) + lane_value(v, 48));
}

template <int N>
__device__ inline double row_ror64(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = row_ror<N>(static_cast<uint32_t>(b));
    const uint64_t hi = row_ror<N>(static_cast<uint32_t>(b >> 32));
    return __builtin_bit_cast(double, lo | (hi << 32));
}

__device__ inline double lane_value64(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = static_cast<uint32_t>(
        __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(b)), lane));
    const uint64_t hi = static_cast<uint32_t>(
        __builtin_amdgcn_readlane(static_cast<int>(static_cast<uint32_t>(b >> 32)), lane));
    return __builtin_bit_cast(double, lo | (hi << 32));
}

__device__ inline double wave_sum64(double v) {
    v += row_ror64<8>(v);
    v += row_ror64<4>(v);
    v += row_ror64<2>(v);
    v += row_ror64<1>(v);
    return (lane_value64(v, 0) + lane_value64(v, 16)) +
           (lane_value64(v, 32) + lane_value64(v, 48));
}

// ---------------------------------------------------------------- E4M3 blocks
// The recipe of ep_quantize_fp8 on binary32 values: a row of 16 lanes holds a
// block of 128 channels, 8 a lane; every lane of the block calls this.
//   amax = largest |v| (NaN skipped), s = max(amax, 1e-12) / 448; UE8M0 rounds
//   s up to a power of two; code = E4M3 nearest to clamp(v / s, +-448).
// Finite blocks divide through one correctly rounded reciprocal y = 1/s and
// one remainder correction (Markstein's division), which gives the correctly
// rounded v / s wherever |v / s| >= 2^-11; smaller quotients have the zero
// code either way.  Those quotients lie within an ulp of +-448, so only
// blocks with an infinity or a NaN are clamped, and take true divisions.
// *pack: the scale's binary32 bits, or its exponent byte.
template <int FMT>
__device__ inline u32x2 e4m3_block8(const float v[8], uint32_t *pack) {
#pragma clang fp contract(off)
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        m = b > m ? b : m;
    }
    m = row_max(m);                        // non-negative floats order like their bits, NaN on top
    const bool finite = m < 0x7F800000u;
    if (!finite) {
        m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
            if (b <= 0x7F800000u && b > m) m = b;
        }
        m = row_max(m);
    }
    const float amax = __uint_as_float(m);
    float s = __fdiv_rn(amax > 1e-12f ? amax : 1e-12f, 448.0f);
    if (FMT == EP_SF_UE8M0) {
        uint32_t e = (__float_as_uint(s) >> 23) & 0xFFu;
        if (__float_as_uint(s) & 0x7FFFFFu) ++e;
        *pack = e;
        s = __uint_as_float(e << 23);
    } else {
        *pack = __float_as_uint(s);
    }
    float c[8];
    if (finite) {
        if (FMT == EP_SF_UE8M0) {
            // s = 2^k with -49 <= k <= 120: v * 2^-k is v / s
            const float y = __uint_as_float((254u << 23) - __float_as_uint(s));
#pragma unroll
            for (int i = 0; i < 8; ++i) c[i] = v[i] * y;
        } else {
            const float y = __fdiv_rn(1.0f, s);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q0 = v[i] * y;
                const float n = __builtin_fmaf(q0, s, -v[i]);
                c[i] = __builtin_fmaf(-n, y, q0);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            c[i] = __builtin_fminf(__builtin_fmaxf(__fdiv_rn(v[i], s), -448.0f), 448.0f);
    }
    uint32_t w[2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
        int word = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * g], c[4 * g + 1], 0, false);
        word = __builtin_amdgcn_cvt_pk_fp8_f32(c[4 * g + 2], c[4 * g + 3], word, true);
        w[g] = static_cast<uint32_t>(word);
    }
    if (!finite) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q = __fdiv_rn(v[i], s);
            if (q != q)
                w[i / 4] = (w[i / 4] & ~(0xFFu << (8 * (i % 4)))) | (0x7Fu << (8 * (i % 4)));
        }
    }
    return u32x2{w[0], w[1]};
}

// Stores the scale packs of a wave that holds 4 consecutive blocks starting
// at block b0 (a multiple of 4), one per row of 16 lanes, each lane's `pack`
// from e4m3_block8 (rows past the last block: anything).  `row` is the
// buffer's row.  Every lane of the wave calls this.
template <int FMT>
__device__ inline void store_packs(uint32_t *sf, int64_t ts, int64_t hs, int64_t row, int b0,
                                   int blocks, uint32_t pack, int lane) {
    if (FMT == EP_SF_F32) {
        const int b = b0 + (lane >> 4);
        if ((lane & 15) == 0 && b < blocks) sf[row * ts + b * hs] = pack;
    } else {
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t e = static_cast<uint32_t>(
                __builtin_amdgcn_readlane(static_cast<int>(pack), 16 * i));
            if (b0 + i < blocks) word |= e << (8 * i);
        }
        if (lane == 0 && b0 < blocks) sf[row * ts + (b0 >> 2) * hs] = word;
    }
}

// Scale of block b of a row: binary32 bits, or an exponent byte of a pack
// (byte 0 is 2^-127, byte 255 NaN).
__device__ inline float load_scale(const uint32_t *sf, int64_t ts, int64_t hs, int64_t row, int b,
                                   bool ue8m0) {
    if (!ue8m0) return __uint_as_float(sf[row * ts + b * hs]);
    const uint32_t e = (sf[row * ts + (b >> 2) * hs] >> (8 * (b & 3))) & 0xFFu;
    return __uint_as_float(e == 0 ? 0x00400000u : e == 255 ? 0x7FC00000u : e << 23);
}

// Values of four E4M3 codes.
__device__ inline void e4m3_values4(uint32_t w, float f[4]) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8(static_cast<int>(w), true);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y;
}

}  // namespace ep
