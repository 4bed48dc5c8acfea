// Rows in 8-bit integers with one scale a row, on gfx950 (include/ep_expert.h:
// ep_quantize_i8, ep_quantize_i8_rows).
#include "ep_expert_internal.h"
#include "ep_rows.h"

namespace ep {
namespace {

typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

// Largest |v| of 8 bf16 values, bits of bf16 in two halves, and of what m holds; NaN patterns
// are larger than any number's.
__device__ inline u16x2 larger(u16x2 m, const u32x4 v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = v[i] & 0x7FFF7FFFu;
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, w));
    }
    return m;
}

__device__ inline uint32_t wave_max(uint32_t v) {
    v = row_max(v);
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16),
                   c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    const uint32_t e = a > b ? a : b, f = c > d ? c : d;
    return e > f ? e : f;
}

// Eight codes of one row: v / s, rounded to the nearest whole number.  q0 + (v - q0 s) y, each
// step one fused operation and y the correctly rounded reciprocal, is the correctly rounded
// quotient (Markstein, IBM Journal of Research and Development 34, 1990); adding 1.5 2^23 rounds it, and
// the sum's low byte is the code.
__device__ inline u32x2 codes8(const u32x4 v, float s, float y) {
#pragma clang fp contract(off)
    float f[8];
    unpack8(v, f);
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float q0 = f[i] * y;
        const float n = __builtin_fmaf(q0, s, -f[i]);
        const float q = __builtin_fmaf(-n, y, q0);
        c[i] = __float_as_uint(q + 12582912.0f);             // the code in the low byte
    }
    auto pack = [&](int i) {
        const uint32_t lo = __builtin_amdgcn_perm(c[i + 1], c[i], 0x0C0C0400u);
        const uint32_t hi = __builtin_amdgcn_perm(c[i + 3], c[i + 2], 0x0C0C0400u);
        return lo | (hi << 16);
    };
    return u32x2{pack(0), pack(4)};
}

// One row by W waves of a block of four, V vectors of 8 channels a lane in registers: read once,
// for its largest value and then its codes.  Bound by HBM: 32768 rows of 2048 channels 34.6 us, 5.8 of
// the 6.5 TB/s of a plain copy; one row of 7168 2.0 us, a launch and two round trips.  MANY rows are
// read past the caches, which are left to what is written (32768 rows of 2048: 42 -> 34.6 us;
// with the stores past them too 39).
template <int W, int V, bool MANY>
__global__ __launch_bounds__(256) void quant_i8_kernel(const QuantI8Args a, int64_t first) {
    __shared__ uint32_t tops[4];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int vecs = a.channels / 8, me = wave % W * 64 + lane;
    int64_t row = first + blockIdx.x * static_cast<int64_t>(4 / W) + wave / W;
    bool here = row < a.num_rows;
    if (a.dst && here) {
        const uint32_t bits = static_cast<uint32_t>(a.scalars[EP_SCALAR_ERROR_BITS]);
        row = a.dst[row];
        here = row >= 0 && row < a.capacity && !(bits & EP_ERRBIT_FATAL);
    }
    if (!here) return;                                       // W == 1, or the whole block
    const u32x4 *x = static_cast<const u32x4 *>(a.x) + row * vecs;
    u32x4 v[V];
    u16x2 m = u16x2{0, 0};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = i * 64 * W + me;
        if (at >= vecs) v[i] = u32x4{0u, 0u, 0u, 0u};
        else v[i] = MANY ? __builtin_nontemporal_load(x + at) : x[at];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) m = larger(m, v[i]);
    uint32_t top = wave_max(static_cast<uint32_t>(m.x > m.y ? m.x : m.y) << 16);
    if (W > 1) {
        if (lane == 0) tops[wave] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < W; ++i) top = top > tops[i] ? top : tops[i];
    }
    const bool fine = top < 0x7F800000u;
    const float amax = __uint_as_float(top);
    const float s = __fdiv_rn(amax > 1e-12f ? amax : 1e-12f, 127.0f);
    const float y = __fdiv_rn(1.0f, s);
    u32x2 *q = static_cast<u32x2 *>(a.q) + row * vecs;
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int at = i * 64 * W + me;
        if (at < vecs) q[at] = fine ? codes8(v[i], s, y) : u32x2{0u, 0u};
    }
    if (me == 0) a.scale[row] = fine ? s : __uint_as_float(0x7FC00000u);
}

template <int W, int V, bool MANY = false>
hipError_t launch_quant(const QuantI8Args &a, hipStream_t stream) {
    // rows of a launch: 2^22 blocks, so 2^30 threads whatever a row takes (HIP refuses 2^32)
    constexpr int64_t kMost = (int64_t(1) << 22) * (4 / W);
    for (int64_t r = 0; r < a.num_rows; r += kMost) {
        const int64_t n = a.num_rows - r < kMost ? a.num_rows - r : kMost;
        const int64_t blocks = (n * W + 3) / 4;
        quant_i8_kernel<W, V, MANY><<<static_cast<uint32_t>(blocks), 256, 0, stream>>>(a, r);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

}  // namespace

// Many rows: a wave each, which waits for no other one (32768 rows of 2048: 45 us by four waves).
// Few: four waves, as a row's latency is what counts.
hipError_t launch_quantize_i8(const QuantI8Args &a, hipStream_t stream) {
    const int vecs = a.channels / 8;
    const bool many = a.num_rows >= 2048;
    if (many) {
        if (vecs <= 64) return launch_quant<1, 1, true>(a, stream);
        if (vecs <= 128) return launch_quant<1, 2, true>(a, stream);
        if (vecs <= 256) return launch_quant<1, 4, true>(a, stream);
        if (vecs <= 512) return launch_quant<1, 8, true>(a, stream);
        if (vecs <= 1024) return launch_quant<4, 4, true>(a, stream);
        return launch_quant<4, 16, true>(a, stream);
    }
    if (vecs <= 64) return launch_quant<1, 1>(a, stream);
    if (vecs <= 256) return launch_quant<4, 1>(a, stream);
    if (vecs <= 512) return launch_quant<4, 2>(a, stream);
    if (vecs <= 1024) return launch_quant<4, 4>(a, stream);
    return launch_quant<4, 16>(a, stream);
}

}  // namespace ep
