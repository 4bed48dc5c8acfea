// Products of the expert rows with 4-bit weights on gfx950
// (include/ep_layer.h: ep_w4_pack, ep_expert_w4).
//
// out[r, :] = x[r, :] . W[e]^T for the rows r of expert e, as matrix
// instructions of 16 rows x 16 outputs x 32 channels (v_mfma_f32_16x16x32_bf16;
// lane l holds row l % 16 of x, output l % 16 of W, channels 8 (l / 16) .. + 7 of
// each, and accumulates four of operand A's for one of operand B's).
//
// Packed weights: for every expert, tile of 16 outputs and step of 128
// channels, one record of 1 KB: lane l's 16 bytes at 16 l, dword j eight codes of
// output l % 16.  A wave reads a record in one load of consecutive addresses, and a
// tile's records follow each other, so a wave reads one stream (read this way
// 1 GB came in at 7.0 TB/s on MI355X; rows of codes as they are in a model's
// file, 16 rows by 128 bytes a wave, at 5.6 to 6.3).
//   EP_W4_INT4: dword j holds channels 32 j + 8 (l / 16) .. + 7, what lane l feeds to the
//   j-th instruction, channel 2i in nibble i and 2i + 1 in nibble i + 4: one shift
//   and one and-or make a pair of bf16, 0x4300 | code = 128 + code exactly.  The
//   136 = 128 + 8 is taken off by a product of x with the constant -136, from
//   which the accumulators of all tiles start; a group's sum is then
//   scaled and added to the total.  28 vector instructions a record: the
//   conversion is what bounds larger batches.
//   EP_W4_MXFP4: lane l holds channels 32 (l / 16) .. + 31, one scale group, in order;
//   v_cvt_scalef32_pk_bf16_fp4 makes pairs of bf16, scaled and exact.
// x in E4M3 is turned into bf16 (exactly) on its way into LDS.  The scaled instruction on 8-
// and 4-bit codes, v_mfma_scale_f32_16x16x128_f8f6f4, would take E4M3 and E2M1 as they are, but
// it drops what is small beside the largest products of its 128 channels (2688 - 2688 + 2^-10
// gives 0; rows whose large products cancel were off by 262 2^-24 of the sum of |x w|, with the
// bf16 instruction by less than 2 2^-24), which is less than the binary32 sums promised.
// Scales: [expert][tile][step], in a step [output][group] for EP_W4_INT4 and
// [group][output] for EP_W4_MXFP4, so a lane's scales of a step are consecutive.
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
// `mask` and `one28` hold 0x000F000F and 0x43004300 in registers of the two kinds that
// one v_and_or_b32 can take (it has no room for literals).
__device__ inline u32x4 int4_plus128(uint32_t w, uint32_t mask, uint32_t one28) {
    u32x4 o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = ((w >> (4 * i)) & mask) | one28;
    return o;
}

// Eight E2M1 codes times 2^(e - 127) in bf16; e = 255 gives NaN.
__device__ inline u32x4 mxfp4(uint32_t w, uint32_t e) {
    const float s = __uint_as_float(e << 23);      // only the exponent counts: 0 is 2^-127
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
// First of the eight channels that dword j of a lane's codes holds within a
// step: the scale groups of EP_W4_INT4 lie across a matrix instruction's lanes, the
// ones of EP_W4_MXFP4 within a lane.
__device__ inline int first_channel(bool int4, int j, int q) {
    return int4 ? 32 * j + 8 * q : 32 * q + 8 * j;
}

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
        const int row = static_cast<int>(record / steps % tiles) * 16 + (lane & 15);
        const int ch = static_cast<int>(record % steps) * 128 + first_channel(int4, j, lane >> 4);
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

// One thread a scale; U: its bytes.  A record's scales are [output][group] for
// EP_W4_INT4 and [group][output], lane by lane, for EP_W4_MXFP4.
template <typename U>
__global__ __launch_bounds__(256) void pack_scales_kernel(const U *scales, int64_t experts, int n,
                                                          int groups, int per_step, U *out) {
    const int tiles = (n + 15) / 16, steps = groups / per_step;
    const int64_t total = experts * tiles * 16 * groups;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < total; i += stride) {
        const int at = static_cast<int>(i % (16 * per_step));
        const int64_t record = i / (16 * per_step);
        const int64_t e = record / (static_cast<int64_t>(tiles) * steps);
        const bool int4 = sizeof(U) == 2;
        const int row = static_cast<int>(record / steps % tiles) * 16 +
                        (int4 ? at / per_step : at & 15);
        const int group = static_cast<int>(record % steps) * per_step +
                          (int4 ? at % per_step : at >> 4);
        out[i] = row < n ? scales[(e * n + row) * groups + group] : U(0);
    }
}

// ---------------------------------------------------------------- product
// Every expert's rows are taken in passes of `per` rows.  Pass number `pass` of all of
// them, experts in order: its expert (-1 behind the last pass), and where its rows
// lie.  Every lane of the wave calls this.
struct Pass {
    int expert, start, rows;
};

__device__ inline Pass find_pass(const int32_t *counts, const int32_t *psum, int experts, int pass,
                                 int per, int lane) {
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int e = e0 + lane;
        const int32_t c = e < experts ? counts[e] : 0;
        const int32_t p = e < experts ? psum[e] : 0;
        int upto = (c + per - 1) / per;              // passes up to and with this expert
        const uint64_t some = __ballot(upto > 0);
        if (__ballot(upto > 1) == 0) {
            upto = __popcll(some & ((uint64_t(2) << lane) - 1));
        } else {
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int below = __shfl_up(upto, d);
                if (lane >= d) upto += below;
            }
        }
        const int all = __builtin_amdgcn_readlane(upto, 63);
        if (pass >= all) {
            pass -= all;
            continue;
        }
        // the first lane whose sum is past the number
        const int l = __builtin_amdgcn_readfirstlane(
            __ffsll(static_cast<unsigned long long>(__ballot(upto > pass))) - 1);
        const int rows = __builtin_amdgcn_readlane(c, l);
        const int before = __builtin_amdgcn_readlane(upto, l) - (rows + per - 1) / per;
        const int first = (pass - before) * per;
        return {e0 + l, __builtin_amdgcn_readlane(p, l) + first,
                rows - first < per ? rows - first : per};
    }
    return {-1, 0, 0};
}

constexpr int kW4Threads = 256;
constexpr int kW4Waves = kW4Threads / 64;

// A barrier that orders LDS alone: loads of weights stay in flight across it.
__device__ inline void lds_barrier() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// What a wave has read of its weights for one step: NT records and their scales.
template <int FMT, int GROUP, int NT>
struct Records {
    static constexpr int kScaleWords = FMT == EP_W4_MXFP4 || GROUP > 32 ? 1 : 2;
    u32x4 w[NT];
    uint32_t sw[NT][kScaleWords];
};

// The value of the other lane of an even and an odd one.
__device__ inline uint32_t other_of_pair(uint32_t v) {
    return static_cast<uint32_t>(
        __builtin_amdgcn_update_dpp(0, static_cast<int>(v), 0xB1, 0xF, 0xF, true));
}

typedef __amdgpu_buffer_rsrc_t Buffer;

// A view of `bytes` bytes; loads behind them give 0.
__device__ inline Buffer bounded(const char *p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<char *>(p), 0, bytes, 0x00020000);
}

constexpr int kStream = 2;                       // non-temporal
constexpr uint32_t kNowhere = 0x80000000u;       // behind any view's end

// One block for one pass (MT tiles of 16 rows of one expert) and NW groups of NT
// tiles of 16 outputs: a group is one wave's, or KS waves take every KS-th step
// each and add up through LDS.
//   EP_W4_INT4: x is operand A and the weights operand B, so a lane has the sums of four rows
//   of one output and a group's sums one scale of the weights a lane.  (The other way
//   round, four scales a lane and group had to be unpacked and held: groups of 32, 64 outputs
//   of 32 rows spilled registers; 128 tokens 250 -> 219 us with groups of 32, 4 tokens 78 -> 69.)
//   EP_W4_MXFP4: the other way round, so a lane has four outputs of one row, one scale of x,
//   and stores 8 bytes; the weights' scales are the conversion's business.
//   x is brought by the block's waves together and handed over through LDS, in
//   the lanes' order (16 bytes a lane, no bank conflicts): loads of 16 rows by 64
//   bytes keep the address units busy for about 35 cycles each, as long as 400
//   bytes of weights take at the HBM's rate, and with every wave loading its own x a batch of
//   16 rows an expert took 125 us more (64 experts, 4096 x 7168, MXFP4; it takes 187).
//   The weights of the next D - 1 rounds stay in flight across the rounds'
//   barriers, which order LDS only.
//   HELD: a pass has `per` rows at most (one to four) and all of their x is brought to LDS
//   before the first step, which takes x's loads and the barriers out of the loop: one token
//   of 8 experts 24.5 -> 22.1 us, four tokens 78 -> 67, two experts of 4096 channels and
//   1024 outputs 8.5 -> 6.2 (7168 channels to 4096 outputs, EP_W4_INT4).
template <int FMT, int GROUP, bool FP8, int NT, int MT, int KS, int D, bool HELD>
__global__ __launch_bounds__(kW4Threads, 2) void w4_kernel(const W4Args a, int first_pass,
                                                           int per) {
    typedef Records<FMT, GROUP, NT> R;
    constexpr bool MX = FMT == EP_W4_MXFP4;
    constexpr int NW = kW4Waves / KS;
    constexpr int P = MX ? 1 : 128 / GROUP;      // groups of a step that are scaled afterwards
    constexpr int U = 4;                         // 16-byte units of x a lane, row and step
    constexpr int F = MT * U;                    // units of x a lane and round
    constexpr int PER = F > NW ? F / NW : 1;     // of them a wave brings
    constexpr int SPER = MT > NW ? MT / NW : 1;  // tiles' scales of x it brings
    constexpr int kXUnits = HELD ? 1 : D * KS * F * 64;
    constexpr int kSumUnits = KS == 1 || HELD ? 0 : kW4Waves * NT * MT * 64;
    __shared__ u32x4 ring[kXUnits > kSumUnits ? kXUnits : kSumUnits];
    alignas(16) __shared__ float ring_sf[FP8 && !HELD ? D * KS * MT * 16 : 1];
    extern __shared__ u32x4 all[];               // HELD: x, then the sums
    u32x4 *const lds = HELD ? all : ring;
    const int lane = threadIdx.x & 63, q = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int kg = wave % KS, nw = wave / KS;
    const int tiles = (a.n + 15) / 16, steps = a.k / 128;
    const int tile0 = (blockIdx.x * NW + nw) * NT;
    const uint32_t bits = static_cast<uint32_t>(a.scalars[EP_SCALAR_ERROR_BITS]);
    uint32_t mask = 0x000F000Fu, one28 = 0x43004300u;
    asm("" : "+s"(mask));
    asm("" : "+v"(one28));

    Pass pass = find_pass(a.counts, a.psum, a.num_experts, first_pass + blockIdx.y, per, lane);
    if (pass.expert < 0 || (bits & EP_ERRBIT_FATAL)) return;
    // no layout content sends a load or a store out of the rows' buffers
    if (pass.start < 0 || pass.start >= a.capacity) return;
    if (pass.rows > a.capacity - pass.start) pass.rows = static_cast<int>(a.capacity - pass.start);
    // The group's records are consecutive; tiles behind the last are read as the
    // last and not stored.
    constexpr int kScaleStep = MX ? 64 : 32 * P;                     // bytes of a record's scales
    const int first = tile0 < tiles ? tile0 : tiles - 1;
    const int mine = first + NT <= tiles ? NT : tiles - first;
    const int64_t record = (static_cast<int64_t>(pass.expert) * tiles + first) * steps;
    const Buffer codes = bounded(static_cast<const char *>(a.codes) + record * 1024,
                                 mine * steps * 1024);
    const Buffer scales = bounded(static_cast<const char *>(a.scales) + record * kScaleStep,
                                  mine * steps * kScaleStep);
    uint32_t code_at = 16 * lane;
    uint32_t scale_at = MX ? lane : 2 * P * (lane & 15);
    const int rounds = (steps + KS - 1) / KS;
    auto step = [&](int round) { return round * KS + kg; };
    auto held = [&](int s) { return s < steps ? s : steps - 1; };
    // Called for one round after the other: offsets and pointers are moved on in
    // place, as an address in a register of its own would be put where an
    // older load is still to arrive, and wait for it.  Rounds behind the last read nothing.
    auto load_w = [&](R &r, int round) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            const int at = (t < mine ? t : 0) * steps + held(step(round));
            r.w[t] = __builtin_amdgcn_raw_buffer_load_b128(codes, code_at, at * 1024, kStream);
            const int sat = at * kScaleStep;
            if (MX) {
                r.sw[t][0] = __builtin_amdgcn_raw_buffer_load_b8(scales, scale_at, sat, 0);
            } else if (P == 1) {
                r.sw[t][0] = __builtin_amdgcn_raw_buffer_load_b16(scales, scale_at, sat, 0);
            } else if (P == 2) {
                r.sw[t][0] = __builtin_amdgcn_raw_buffer_load_b32(scales, scale_at, sat, 0);
            } else {
                const u32x2 v = __builtin_amdgcn_raw_buffer_load_b64(scales, scale_at, sat, 0);
                r.sw[t][0] = v.x;
                r.sw[t][1 % R::kScaleWords] = v.y;
            }
        }
        if (round + 1 >= rounds) code_at = scale_at = kNowhere;
    };
    // the weights of the first rounds are on their way before anything of x is known
    R w[D];
#pragma unroll
    for (int d = 0; d + 1 < D; ++d) load_w(w[d], d);
    // Unit i = t * U + j of a step's x, and the scales of tile i, are brought by wave
    // i % NW (by several, the same values, where there are fewer units than waves).
    const char *xp[PER];
    const uint32_t *sp[SPER];
    auto row_of = [&](int m) {
        const int64_t row = pass.start + m;
        if (!a.token_rows) return row;
        // a call captured for fewer tokens than a later layout has reads the last of its own
        const int64_t token = a.src_meta[row] / a.num_topk;
        return token < 0 ? 0 : token < a.num_tokens ? token : a.num_tokens - 1;
    };
    auto source = [&](int t) {
        const int m = 16 * t + (lane & 15);
        return row_of(m < pass.rows ? m : pass.rows - 1);
    };
    if (!HELD)
#pragma unroll
    for (int p = 0; p < PER; ++p) {
        const int i = (p * NW + nw) % F, ch = first_channel(!MX, i % U, q);
        xp[p] = static_cast<const char *>(a.x) +
                (source(i / U) * a.k + held(kg) * 128 + ch) * (FP8 ? 1 : 2);
    }
    if (FP8 && !HELD) {
#pragma unroll
        for (int p = 0; p < SPER; ++p) {
            const int i = (p * NW + nw) % MT;
            sp[p] = a.sf.p + source(i) * a.sf.ts;
        }
    }
    struct X {
        u32x4 v[PER];
        float sf[SPER];
    };
    auto load_x = [&](X &r, int round) {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            if (FP8) {
                const u32x2 v = *reinterpret_cast<const u32x2 *>(xp[p]);
                r.v[p].x = v.x;
                r.v[p].y = v.y;
            } else {
                r.v[p] = *reinterpret_cast<const u32x4 *>(xp[p]);
            }
            // the row's last step stays the last
            xp[p] += step(round + 1) < steps ? KS * 128 * (FP8 ? 1 : 2) : 0;
        }
        if (FP8) {
#pragma unroll
            for (int p = 0; p < SPER; ++p)
                r.sf[p] = load_scale(sp[p], 0, a.sf.hs, 0, held(step(round)), a.sf.ue8m0);
        }
    };
    // Steps behind the last count as zeros.
    auto store_x = [&](const X &r, int round, int half) {
        const int buf = half * KS + kg;
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const uint32_t keep = step(round) < steps ? 0xFFFFFFFFu : 0u;
            const u32x4 v = FP8 ? e4m3_bf16(u32x2{r.v[p].x, r.v[p].y}) : r.v[p];
            lds[(buf * F + (p * NW + nw) % F) * 64 + lane] = v & keep;
        }
        if (FP8) {
#pragma unroll
            for (int p = 0; p < SPER; ++p)
                ring_sf[(buf * MT + (p * NW + nw) % MT) * 16 + (lane & 15)] =
                    step(round) < steps ? r.sf[p] : 0.0f;
        }
    };
    f32x4 total[MT][NT];
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u) total[t][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    // HELD: row m's units (8 channels in 16 bytes) start at m * pitch, an odd number so that rows
    // lie in different banks; behind the rows the zeros that steps behind the last read, and the
    // scales.
    constexpr int kStepUnits = 4 * U;
    const int pitch = steps * kStepUnits + 1, zeros = per * pitch;
    float *const held_sf = reinterpret_cast<float *>(all + zeros + kStepUnits);
    const int my_row = (lane & 15) < pass.rows ? lane & 15 : pass.rows - 1;
    auto compute = [&](const R &r, int half, int round) {
        const int s = step(round);
        const u32x4 *xl = HELD ? all + (s < steps ? my_row * pitch + s * kStepUnits : zeros) +
                                     (MX ? 4 * q : q)
                               : lds + (half * KS + kg) * F * 64 + lane;
        constexpr int kUnit = !HELD ? 64 : MX ? 1 : 4;      // from one unit to the next
        f32x4 sx[MT];                            // of the rows that a lane has sums of
        if (FP8)
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                const float *ring_at = ring_sf + ((half * KS + kg) * MT + t) * 16;
                if (MX) {
                    sx[t][0] = !HELD ? ring_at[lane & 15]
                               : s < steps ? held_sf[my_row * steps + s] : 0.0f;
                } else if (!HELD) {
                    sx[t] = *reinterpret_cast<const f32x4 *>(ring_at + 4 * q);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        sx[t][i] = s < steps ? held_sf[(i < pass.rows ? i : 0) * steps + s] : 0.0f;
                }
            }
#pragma unroll
        for (int g = 0; g < P; ++g) {
            constexpr int J = U / P;
            f32x4 acc[MT][NT];
            u32x4 xs[MT][J];
#pragma unroll
            for (int t = 0; t < MT; ++t)
#pragma unroll
                for (int j = 0; j < J; ++j) xs[t][j] = xl[(t * U + g * J + j) * kUnit];
#pragma unroll
            for (int t = 0; t < MT; ++t) {
                f32x4 from = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                if (!MX)
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        from = mfma(xs[t][j],
                                    u32x4{kMinus136, kMinus136, kMinus136, kMinus136}, from);
#pragma unroll
                for (int u = 0; u < NT; ++u) acc[t][u] = MX && !FP8 ? total[t][u] : from;
            }
#pragma unroll
            for (int j = 0; j < J; ++j)
#pragma unroll
                for (int u = 0; u < NT; ++u) {
                    const uint32_t w4 = r.w[u][(g * J + j) % 4];
                    const u32x4 w = MX ? mxfp4(w4, r.sw[u][0])
                                       : int4_plus128(w4, mask, one28);
#pragma unroll
                    for (int t = 0; t < MT; ++t)
                        acc[t][u] = MX ? mfma(w, xs[t][j], acc[t][u])
                                       : mfma(xs[t][j], w, acc[t][u]);
                }
#pragma unroll
            for (int u = 0; u < NT; ++u) {
                const uint32_t sw = r.sw[u][g / 2 % R::kScaleWords];
                const float f = MX ? 1.0f : g & 1 ? bf16_hi(sw) : bf16_lo(sw);
#pragma unroll
                for (int t = 0; t < MT; ++t) {
                    if (MX && !FP8) {
                        total[t][u] = acc[t][u];
                        continue;
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float m = MX ? sx[t][0] : FP8 ? f * sx[t][i] : f;
                        total[t][u][i] = __builtin_fmaf(m, acc[t][u][i], total[t][u][i]);
                    }
                }
            }
        }
    };
    // While a round is computed on, the weights of the next D - 1 are on their way
    // into registers, and their x into registers and then LDS.
    X x[D];
    if (HELD) {
        const int tid = threadIdx.x;
        for (int m = 0; m < pass.rows; ++m) {
            const int64_t from = row_of(m);
            const char *row = static_cast<const char *>(a.x) + from * a.k * (FP8 ? 1 : 2);
#pragma unroll 4
            for (int u = tid; u < steps * kStepUnits; u += kW4Threads)
                all[m * pitch + u] =
                    FP8 ? e4m3_bf16(reinterpret_cast<const u32x2 *>(row)[u])
                        : reinterpret_cast<const u32x4 *>(row)[u];
            if (FP8)
                for (int s = tid; s < steps; s += kW4Threads)
                    held_sf[m * steps + s] = load_scale(a.sf.p, a.sf.ts, a.sf.hs, from, s,
                                                        a.sf.ue8m0);
        }
        if (tid < kStepUnits) all[zeros + tid] = u32x4{0u, 0u, 0u, 0u};
    } else {
#pragma unroll
        for (int d = 0; d + 1 < D; ++d) load_x(x[d], d);
        store_x(x[0], 0, 0);
    }
    lds_barrier();
    for (int round = 0; round < rounds;) {
#pragma unroll
        for (int d = 0; d < D; ++d) {
            if (!HELD) load_x(x[(d + D - 1) % D], round + D - 1);
            load_w(w[(d + D - 1) % D], round + D - 1);
            __builtin_amdgcn_sched_barrier(0);
            compute(w[d], d, round);
            __builtin_amdgcn_sched_barrier(0);
            if (!HELD) {
                store_x(x[(d + 1) % D], round + 1, (d + 1) % D);
                lds_barrier();
            }
            if (++round == rounds) break;
        }
    }
    if (KS > 1) {
        lds_barrier();                       // x is read: its room becomes the sums'
#pragma unroll
        for (int t = 0; t < MT; ++t)
#pragma unroll
            for (int u = 0; u < NT; ++u)
                lds[((wave * MT + t) * NT + u) * 64 + lane] =
                    __builtin_bit_cast(u32x4, total[t][u]);
        lds_barrier();
    }
#pragma unroll
    for (int t = 0; t < MT; ++t)
#pragma unroll
        for (int u = 0; u < NT; ++u) {
            if ((t * NT + u) % KS != kg) continue;
            f32x4 v = total[t][u];
            if (KS > 1) {
                v = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int k = 0; k < KS; ++k)
                    v += __builtin_bit_cast(
                        f32x4, lds[(((nw * KS + k) * MT + t) * NT + u) * 64 + lane]);
            }
            uint16_t *out = static_cast<uint16_t *>(a.out) + static_cast<int64_t>(pass.start) * a.n;
            const uint32_t lo = pack2(v[0], v[1]), hi = pack2(v[2], v[3]);
            if (MX) {
                const int m = 16 * t + (lane & 15), col = (tile0 + u) * 16 + 4 * q;
                if (m < pass.rows && col < a.n)
                    *reinterpret_cast<u32x2 *>(out + static_cast<int64_t>(m) * a.n + col) =
                        u32x2{lo, hi};
                continue;
            }
            // two lanes' outputs of a row make a word: the even lane's of rows 0 and 2, the odd
            // one's of rows 1 and 3
            const int m = 16 * t + 4 * q + (lane & 1), col = (tile0 + u) * 16 + (lane & 14);
            const uint32_t pick = lane & 1 ? 0x03020706u : 0x05040100u;
            const uint32_t first_row = __builtin_amdgcn_perm(other_of_pair(lo), lo, pick);
            const uint32_t second_row = __builtin_amdgcn_perm(other_of_pair(hi), hi, pick);
            if (col >= a.n) continue;
            if (m < pass.rows)
                *reinterpret_cast<uint32_t *>(out + static_cast<int64_t>(m) * a.n + col) =
                    first_row;
            if (m + 2 < pass.rows)
                *reinterpret_cast<uint32_t *>(out + static_cast<int64_t>(m + 2) * a.n + col) =
                    second_row;
        }
}

template <int FMT, int GROUP, bool FP8, int NT, int MT, int KS, int D, bool HELD = false>
hipError_t launch_w4(const W4Args &a, int64_t active, int64_t slots, hipStream_t stream,
                     int per = 16 * MT, int held_bytes = 0) {
    constexpr int per_block = NT * (kW4Waves / KS);
    const int groups = ((a.n + 15) / 16 + per_block - 1) / per_block;
    // no more passes than these: every expert's last one may be partly filled
    const int64_t passes = active + slots / per;
    // a launch holds fewer than 2^32 threads, and 2^16 blocks along y
    int64_t most = (int64_t(1) << 23) / groups;
    most = most < 1 ? 1 : most > 32768 ? 32768 : most;
    for (int64_t p = 0; p < passes; p += most) {
        const dim3 grid(groups, static_cast<uint32_t>(passes - p < most ? passes - p : most));
        w4_kernel<FMT, GROUP, FP8, NT, MT, KS, D, HELD>
            <<<grid, kW4Threads, held_bytes, stream>>>(a, static_cast<int>(p), per);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

constexpr int kHeldBytes = 64 * 1024;            // two blocks a compute unit

// LDS of a pass of `per` rows held whole, room for the sums of the waves at least.
int held_bytes(int per, int steps, int tiles_a_wave, bool fp8) {
    const int64_t x = 16 * (per * (int64_t(steps) * 16 + 1) + 16) +
                      (fp8 ? int64_t(4) * per * steps : 0);
    const int sums = 16 * kW4Waves * tiles_a_wave * 64;
    return x > kHeldBytes ? kHeldBytes + 1 : x > sums ? static_cast<int>(x) : sums;
}

template <int FMT, int GROUP, bool FP8, int NT, int D>
hipError_t launch_held(const W4Args &a, int64_t active, int64_t slots, int per,
                       hipStream_t stream) {
    return launch_w4<FMT, GROUP, FP8, NT, 1, 4, D, true>(
        a, active, slots, stream, per,
        held_bytes(per, a.k / 128, NT, FP8));
}

// Tile and split, by the sizes that the host knows (us at 64 experts of 4096 x 7168 and
// EP_W4_INT4 groups of 128 unless said).  A grid is counted in tiles of 16 outputs of
// the passes that there will be at least; kBlocks is one and a half blocks a compute unit.
//   Few rows: x is held, in passes of up to four rows, while it takes at most 64 KB.  An expert
//   with more rows reads its weights again, which is the cost: EP_W4_INT4 153 without and
//   143 with at 2 rows an expert on average, 183 and 201 at 4; EP_W4_MXFP4 with E4M3 rows 100
//   and 98 at one, 129 and 127 at one and a half, 141 and 146 at two (9 tokens of 8 experts, 320 x
//   4224: 10.4 and 9.9).  Up to four tokens no expert
//   has more (4 tokens, 8 experts of 2192 x 6272, 2.5 rows: 22.5 and 19.2), and in a small grid
//   more passes fill the card (8 experts of 360 x 1920, 14 rows: 7.8 and 7.1; no longer with
//   1320 tiles: 312 x 5888, 33 rows, 14.9 and 17.5).  Four waves a group, 64 outputs a wave or,
//   below 1920 tiles, 32 (2048 tiles: 22.2 with 64 and 24.3 with 32; 1788 of 5248 channels: 18.0
//   and 16.8; 256: 10.8 and 8.8).
//   Otherwise, rows a pass: 16 or 32.  The codes' conversion and the weights' reading are paid
//   once a pass, an empty half of a wide one costs its matrix instructions.
//   EP_W4_INT4: 159 (16) and 184 (32) at 8 rows an expert on average, 189 and 189 at 12, 226
//   and 194 at 16; so 32 beyond 12.  EP_W4_MXFP4 converts less: with E4M3 rows 159 and 179 at 8
//   rows, 181 and 182 at 10, 225 and 189 at 16, with bf16 rows 159 and 168, 178 and 171, 224 and
//   181; so 32 beyond 9.  But only where wide passes fill the card too:
//   EP_W4_INT4 with 2304 tiles (32 experts, 1152 x 2304, 17.6 rows) 23.1 (16) and 25.1;
//   EP_W4_MXFP4 with 2052 tiles (16 experts, 1824 x 4480, 36 rows) 42.2 and 39.5, with 512 (8
//   experts, 1024 x 4096, 32 rows) 17.6 and 28.9.  64 rows gave
//   nothing (16 experts of 64 rows: 150 against 135).
//   Outputs a wave and waves a group: the widest that fills the card.  Short rows leave a
//   block little to do between its first and last loads, which more blocks a compute unit
//   hide: 64 outputs a wave from 32 steps on only (7168 x 2048, 16 steps, groups of 64, 4
//   rows: 87 with 64, 81 with 32).  Two waves a group below 8 kBlocks tiles (16 experts,
//   712 x 1152: 7.8, one wave 8.5), four below 768 if each has a few steps (8 experts, 312 x 5888:
//   14.9, two waves 17.5; 1208 x 1664, 13 steps: 9.1 and 7.9); of two or three steps one wave
//   takes all (16 experts of 512 x 256: 4.6, four waves 5.5).
//   Three steps in registers instead of two keep more of the weights in flight where a
//   block is short of waves.  With 64 outputs of 32 rows they cost waves: 16 rows an expert,
//   EP_W4_MXFP4 189 with two and 192 with three (25 rows, UE8M0 scales: 222 and 256), EP_W4_INT4
//   193 and 194, with groups of 32 217 and 228.
template <int FMT, int GROUP, bool FP8>
hipError_t choose_w4(const W4Args &a, hipStream_t stream) {
    constexpr bool MX = FMT == EP_W4_MXFP4;
    constexpr int64_t kBlocks = 384;
    const int64_t slots = static_cast<int64_t>(a.num_tokens) * a.num_topk, experts = a.num_experts;
    const int64_t active = slots < experts ? slots : experts;
    const int steps = a.k / 128;
    auto tiles_of = [&](int rows) {
        const int64_t passes = slots / rows;
        return (passes > active ? passes : active) * ((a.n + 15) / 16);
    };
    const int per = a.num_tokens < 4 ? a.num_tokens : 4;
    const bool few = a.num_tokens <= 4 || 2 * slots <= (MX ? 3 : 4) * experts ||
                     tiles_of(4) <= 2 * kBlocks;
    if (few && steps >= 4 && held_bytes(per, steps, 4, FP8) <= kHeldBytes)
        return tiles_of(per) >= 5 * kBlocks
                   ? launch_held<FMT, GROUP, FP8, 4, 2>(a, active, slots, per, stream)
                   : launch_held<FMT, GROUP, FP8, 2, 3>(a, active, slots, per, stream);
    const bool wide = slots > (MX ? 9 : 12) * experts && tiles_of(32) >= (MX ? 4 : 8) * kBlocks;
    const int64_t tiles = tiles_of(wide ? 32 : 16);
    if (tiles >= 16 * kBlocks && steps >= 32)
        return wide ? launch_w4<FMT, GROUP, FP8, 4, 2, 1, 2>(a, active, slots, stream)
                    : launch_w4<FMT, GROUP, FP8, 4, 1, 1, 2>(a, active, slots, stream);
    if (wide) return launch_w4<FMT, GROUP, FP8, 2, 2, 1, 2>(a, active, slots, stream);
    if (tiles >= 8 * kBlocks || steps < 4)
        return launch_w4<FMT, GROUP, FP8, 2, 1, 1, 2>(a, active, slots, stream);
    return tiles >= 2 * kBlocks || steps < 14
               ? launch_w4<FMT, GROUP, FP8, 2, 1, 2, 2>(a, active, slots, stream)
               : launch_w4<FMT, GROUP, FP8, 2, 1, 4, 3>(a, active, slots, stream);
}

template <int FMT, int GROUP>
hipError_t choose_x(const W4Args &a, hipStream_t stream) {
    return a.x_fp8 ? choose_w4<FMT, GROUP, true>(a, stream)
                   : choose_w4<FMT, GROUP, false>(a, stream);
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
    if (a.fmt == EP_W4_MXFP4) return choose_x<EP_W4_MXFP4, 32>(a, stream);
    if (a.group == 32) return choose_x<EP_W4_INT4, 32>(a, stream);
    if (a.group == 64) return choose_x<EP_W4_INT4, 64>(a, stream);
    return choose_x<EP_W4_INT4, 128>(a, stream);
}

}  // namespace ep
