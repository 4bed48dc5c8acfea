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
// block of 128 channels, 8 a lane; every lane of the block calls these.
//   amax = largest |v| (NaN skipped), s = max(amax, 1e-12) / 448; UE8M0 rounds
//   s up to a power of two; code = E4M3 nearest to clamp(v / s, +-448).
// Divisions are Markstein's: with y the correctly rounded reciprocal of b and q0 = a y,
// q0 + (a - q0 b) y, each step one fused operation, is the correctly rounded a / b
// where nothing leaves the normal range; and y itself comes from the hardware's
// reciprocal (within an ulp) by one step y + (1 - b y) y.  (Compared with true divisions on
// MI355X over every significand of s at ten exponents, eight quotients each: no
// difference.)  Six operations a block and three a value, where a true division takes
// ten or more; with three blocks a lane they had the activation's vector units
// busy 87 % of the time, now 64 %.

// Largest |v| of the block as bits; NaN patterns (above infinity's) are kept.
__device__ inline uint32_t block_max_bits(const float v[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        m = b > m ? b : m;
    }
    return row_max(m);
}

// The same of bf16 values, two a word, with packed 16-bit maxima.
__device__ inline uint32_t block_max_bits(const u32x4 v) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = __builtin_bit_cast(u16x2, v.x & 0x7FFF7FFFu);
#pragma unroll
    for (int i = 1; i < 4; ++i)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
    const uint32_t w = __builtin_bit_cast(uint32_t, m);
    const uint32_t lo = w << 16, hi = w & 0xFFFF0000u;
    return row_max(lo > hi ? lo : hi);
}

// The same of values that are known to be neither NaN nor infinite.
__device__ inline uint32_t finite_max_bits(const float v[8]) {
    float m = __builtin_fabsf(v[0]);
#pragma unroll
    for (int i = 1; i < 8; ++i) m = __builtin_fmaxf(m, __builtin_fabsf(v[i]));
    return row_max(__float_as_uint(m));
}

__device__ inline float over_448(float amax) {
    const float y = 1.0f / 448.0f;
    const float q = amax * y;
    return __builtin_fmaf(__builtin_fmaf(-q, 448.0f, amax), y, q);
}

__device__ inline uint32_t e4m3_pack4(const float c[4]) {
    int word = __builtin_amdgcn_cvt_pk_fp8_f32(c[0], c[1], 0, false);
    word = __builtin_amdgcn_cvt_pk_fp8_f32(c[2], c[3], word, true);
    return static_cast<uint32_t>(word);
}

// A block's divisor from its scale max(amax, 1e-12) / 448, and what is stored: binary32
// bits or the exponent byte.
template <int FMT>
__device__ inline float block_divisor(float s, uint32_t *pack) {
    if (FMT == EP_SF_UE8M0) {
        uint32_t e = (__float_as_uint(s) >> 23) & 0xFFu;
        if (__float_as_uint(s) & 0x7FFFFFu) ++e;
        *pack = e;
        return __uint_as_float(e << 23);
    }
    *pack = __float_as_uint(s);
    return s;
}

__device__ inline float at_least(float amax) { return amax > 1e-12f ? amax : 1e-12f; }

// Codes of a block with an infinity or a NaN in it: true divisions, clamped, NaN codes.
template <int FMT>
__device__ inline u32x2 e4m3_special8(const float v[8], uint32_t *pack) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t b = __float_as_uint(v[i]) & 0x7FFFFFFFu;
        if (b <= 0x7F800000u && b > m) m = b;
    }
    const float s =
        block_divisor<FMT>(__fdiv_rn(at_least(__uint_as_float(row_max(m))), 448.0f), pack);
    float c[8];
    uint32_t nan[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q = __fdiv_rn(v[i], s);
        if (q != q) nan[i / 4] |= 0xFFu << (8 * (i % 4));
        c[i] = __builtin_fminf(__builtin_fmaxf(q, -448.0f), 448.0f);
    }
    const uint32_t lo = e4m3_pack4(c), hi = e4m3_pack4(c + 4);
    return u32x2{(lo & ~nan[0]) | (0x7F7F7F7Fu & nan[0]), (hi & ~nan[1]) | (0x7F7F7F7Fu & nan[1])};
}

// Codes of a block whose maximum has the bits `max_bits` (from one of the above):
// the quotients of a finite block lie within an ulp of +-448, so nothing is clamped.
// *pack: the scale's binary32 bits, or its exponent byte.
template <int FMT>
__device__ inline u32x2 e4m3_block8(const float v[8], uint32_t max_bits, uint32_t *pack) {
#pragma clang fp contract(off)
    if (__builtin_expect(max_bits >= 0x7F800000u, 0)) return e4m3_special8<FMT>(v, pack);
    const float s =
        block_divisor<FMT>(over_448(at_least(__uint_as_float(max_bits))), pack);
    float c[8];
    if (FMT == EP_SF_UE8M0) {
        // s = 2^k with -49 <= k <= 120: v * 2^-k is v / s
        const float y = __uint_as_float((254u << 23) - __float_as_uint(s));
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = v[i] * y;
    } else {
        const float y0 = __builtin_amdgcn_rcpf(s);
        const float y = __builtin_fmaf(__builtin_fmaf(-s, y0, 1.0f), y0, y0);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float q0 = v[i] * y;
            const float n = __builtin_fmaf(q0, s, -v[i]);
            c[i] = __builtin_fmaf(-n, y, q0);
        }
    }
    return u32x2{e4m3_pack4(c), e4m3_pack4(c + 4)};
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
