// Sum with the residual, root-mean-square norm and E4M3 rows, and the norm's
// gradient, on gfx950 (include/ep_layer.h: ep_add_rmsnorm).
#include "ep_layer_internal.h"
#include "ep_rows.h"

namespace ep {
namespace {

constexpr int kNormBlocks = 1 << 18;     // most blocks of a launch; they walk the rows behind
// Rows up to which the gradient is one launch (us, two launches / one, host time of the
// second included: 512 x 7168 17.5 / 11.9, 1024 x 7168 21.0 / 18.0, 2048 x 7168 28.9 / 31.6;
// 1024 x 1280 15.8 / 11.7, 2048 x 1280 16.1 / 19.6).
constexpr int kFewRows = 1024;

// Channels [8v, 8v + 8) of the norm's weight as binary32.
__device__ inline void load_weight(const void *w, bool bf16, int v, float f[8]) {
    if (bf16) {
        unpack8(static_cast<const u32x4 *>(w)[v], f);
    } else {
        const f32x4 *p = static_cast<const f32x4 *>(w) + 2 * static_cast<int64_t>(v);
        const f32x4 a = p[0], b = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[i] = a[i];
            f[4 + i] = b[i];
        }
    }
}

// Stores a vector, past the caches with STREAM (a template argument: of two branches that
// differ in the hint alone the compiler makes one without it).
template <bool STREAM, typename T>
__device__ inline void put(void *base, int64_t at, T v) {
    if (STREAM) __builtin_nontemporal_store(v, static_cast<T *>(base) + at);
    else static_cast<T *>(base)[at] = v;
}

// ---------------------------------------------------------------- forward
// One block a row; thread t holds the row's 16-byte vectors t, t + threads,
// ... (VPT of them) in registers, so the row is read once.  A wave holds 512
// consecutive channels of each pass: four scale blocks, one a row of 16 lanes,
// and one whole UE8M0 pack.
template <int VPT, int FMT, bool STREAM>
__global__ __launch_bounds__(1024) void norm_kernel(const NormArgs a) {
#pragma clang fp contract(off)
    __shared__ double sums[2][16];
    const int V = a.hidden / 8;
    const int threads = blockDim.x, tid = threadIdx.x, lane = tid & 63;
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.num_tokens; row += gridDim.x, turn ^= 1) {
        const u32x4 *x = static_cast<const u32x4 *>(a.x) + row * V;
        const u32x4 *res = a.residual ? static_cast<const u32x4 *>(a.residual) + row * V : nullptr;
        u32x4 z[VPT];
        float w[VPT][8];
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * threads + tid;
            z[i] = u32x4{0u, 0u, 0u, 0u};
            if (v < V) {
                z[i] = x[v];
                if (res) {
                    float f[8], g[8];
                    unpack8(z[i], f);
                    unpack8(res[v], g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] += g[j];
                    z[i] = pack8(f);
                }
                load_weight(a.weight, a.weight_bf16, v, w[i]);
                if (a.out_z) put<STREAM>(a.out_z, row * V + v, z[i]);
            }
            float f[8];
            unpack8(z[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) sum = __builtin_fma(static_cast<double>(f[j]),
                                                            static_cast<double>(f[j]), sum);
        }
        sum = wave_sum64(sum);
        if (lane == 0) sums[turn][tid >> 6] = sum;
        __syncthreads();                   // the other half of sums is free until the next barrier
        sum = 0.0;
        for (int i = 0; i < threads / 64; ++i) sum += sums[turn][i];
        const float rstd = static_cast<float>(
            1.0 / __builtin_sqrt(sum / static_cast<double>(a.hidden) + static_cast<double>(a.eps)));
        if (a.out_rstd && tid == 0) a.out_rstd[row] = rstd;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * threads + tid;
            float y[8];
            unpack8(z[i], y);
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = v < V ? (y[j] * rstd) * w[i][j] : 0.0f;
            if (a.out_y && v < V) put<STREAM>(a.out_y, row * V + v, pack8(y));
            if (FMT != kSfNone) {
                uint32_t pack;
                const u32x2 q = e4m3_block8<FMT == kSfNone ? EP_SF_F32 : FMT>(
                    y, block_max_bits(y), &pack);
                if (v < V) put<STREAM>(a.out_q, row * V + v, q);
                store_packs<FMT == kSfNone ? EP_SF_F32 : FMT>(
                    a.sf.p, a.sf.ts, a.sf.hs, row, (v - lane) / 16, V / 16, pack, lane);
            }
        }
    }
}

// Bytes of outputs from which, and up to which, the rows are stored past the caches.
// Too many for the last-level cache (256 MB) beside the rows that are read, but few
// enough that ordinary stores would leave them there: then they go on to
// HBM late, in the way of the reads.  Rows of 7168, sum, bf16 and E4M3 rows, alone and with a
// router product and a dispatch behind it (ordinary / past the caches, us): 73 MB
// 31.0 / 22.7 and 93 / 96, 107 MB 42.4 / 35.0 and 128 / 124, 147 MB 54.2 / 51.0 and 158 / 153,
// 294 MB 100 / 95 and 294 / 302: the consumer decides.
constexpr int64_t kStreamFrom = int64_t(96) << 20, kStreamTo = int64_t(256) << 20;

template <int FMT>
hipError_t launch_norm(const NormArgs &a, hipStream_t stream) {
    const int64_t bytes = static_cast<int64_t>(a.num_tokens) * a.hidden *
                          ((a.out_z ? 2 : 0) + (a.out_y ? 2 : 0) + (a.out_q ? 1 : 0));
    const bool past = bytes >= kStreamFrom && bytes <= kStreamTo;
    const int V = a.hidden / 8;
    const int vpt = V <= 512 ? 1 : V <= 1024 ? 2 : 4;
    const int threads = ((V + vpt - 1) / vpt + 63) / 64 * 64;
    const dim3 grid(a.num_tokens < kNormBlocks ? a.num_tokens : kNormBlocks), block(threads);
    const auto kernel = vpt == 1   ? (past ? norm_kernel<1, FMT, true> : norm_kernel<1, FMT, false>)
                        : vpt == 2 ? (past ? norm_kernel<2, FMT, true> : norm_kernel<2, FMT, false>)
                                   : (past ? norm_kernel<4, FMT, true> : norm_kernel<4, FMT, false>);
    kernel<<<grid, block, 0, stream>>>(a);
    return hipGetLastError();
}

// ---------------------------------------------------------------- gradient
// Blocks walk the rows with the grid's stride; each thread keeps the weight
// and its sums of g * n for its channels in registers, so grad_weight costs
// one row of binary32 a block, added up by a second kernel in block order.
template <int VPT>
__global__ __launch_bounds__(1024) void norm_grad_kernel(const NormGradArgs a) {
    __shared__ float sums[2][16];
    const int V = a.hidden / 8;
    const int threads = blockDim.x, tid = threadIdx.x, lane = tid & 63;
    const float inv = 1.0f / static_cast<float>(a.hidden);
    float w[VPT][8], gw[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = i * threads + tid;
#pragma unroll
        for (int j = 0; j < 8; ++j) w[i][j] = gw[i][j] = 0.0f;
        if (v < V) load_weight(a.weight, a.weight_bf16, v, w[i]);
    }
    int turn = 0;
    for (int64_t row = blockIdx.x; row < a.num_tokens; row += gridDim.x, turn ^= 1) {
        const u32x4 *zr = static_cast<const u32x4 *>(a.z) + row * V;
        const u32x4 *gr = static_cast<const u32x4 *>(a.grad_y) + row * V;
        const float rstd = a.rstd[row];
        u32x4 z[VPT], g[VPT], more[VPT];
        float c = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * threads + tid;
            z[i] = g[i] = more[i] = u32x4{0u, 0u, 0u, 0u};
            if (v < V) {
                // read past the caches, as nothing reads them after this (49.9 -> 48.0 us
                // at 4096 x 7168 with the gradient along the residual)
                z[i] = __builtin_nontemporal_load(zr + v);
                g[i] = __builtin_nontemporal_load(gr + v);
                if (a.grad_z)
                    more[i] = __builtin_nontemporal_load(
                        static_cast<const u32x4 *>(a.grad_z) + row * V + v);
            }
        }
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            float zf[8], gf[8];
            unpack8(z[i], zf);
            unpack8(g[i], gf);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float gn = gf[j] * (zf[j] * rstd);
                gw[i][j] += gn;
                c = __builtin_fmaf(gn, w[i][j], c);
            }
        }
        if (!a.grad_x) continue;
        c = wave_sum(c);
        if (lane == 0) sums[turn][tid >> 6] = c;
        __syncthreads();               // the other half of sums is free until the next barrier
        c = 0.0f;
        for (int i = 0; i < threads / 64; ++i) c += sums[turn][i];
        c *= inv;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * threads + tid;
            if (v >= V) continue;
            float zf[8], gf[8], mf[8], o[8];
            unpack8(z[i], zf);
            unpack8(g[i], gf);
            unpack8(more[i], mf);
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = __builtin_fmaf(gf[j] * w[i][j] - (zf[j] * rstd) * c, rstd, mf[j]);
            (static_cast<u32x4 *>(a.grad_x) + row * V)[v] = pack8(o);
        }
    }
    if (!a.grad_weight) return;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
        const int v = i * threads + tid;
        if (v >= V) continue;
        f32x4 *p = reinterpret_cast<f32x4 *>(a.partial +
                                             static_cast<int64_t>(blockIdx.x) * a.hidden) + 2 * v;
        p[0] = f32x4{gw[i][0], gw[i][1], gw[i][2], gw[i][3]};
        p[1] = f32x4{gw[i][4], gw[i][5], gw[i][6], gw[i][7]};
    }
}

// Few rows: one launch.  The first blocks take a row each for grad_x; each of the
// others 64 channels of grad_weight over all rows, which reads g and z a second time (from the
// caches) instead of writing and reading sums.  8 lanes of 8 channels, the rest of the
// threads are groups that take every so many rows, added up in a fixed order.
template <int VPT>
__global__ __launch_bounds__(1024) void norm_grad_few_kernel(const NormGradArgs a,
                                                             int row_blocks) {
    __shared__ float sums[16][64];
    const int V = a.hidden / 8;
    const int threads = blockDim.x, tid = threadIdx.x, lane = tid & 63;
    if (static_cast<int>(blockIdx.x) < row_blocks) {
        const int64_t row = blockIdx.x;
        const float rstd = a.rstd[row];
        float zf[VPT][8], gf[VPT][8], mf[VPT][8];
        float c = 0.0f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * threads + tid;
            u32x4 z = u32x4{0u, 0u, 0u, 0u}, g = z, more = z;
            float w[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
            if (v < V) {
                z = (static_cast<const u32x4 *>(a.z) + row * V)[v];
                g = (static_cast<const u32x4 *>(a.grad_y) + row * V)[v];
                if (a.grad_z) more = (static_cast<const u32x4 *>(a.grad_z) + row * V)[v];
                load_weight(a.weight, a.weight_bf16, v, w);
            }
            unpack8(z, zf[i]);
            unpack8(g, gf[i]);
            unpack8(more, mf[i]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c = __builtin_fmaf(gf[i][j] * (zf[i][j] * rstd), w[j], c);
                gf[i][j] *= w[j];
            }
        }
        c = wave_sum(c);
        if (lane == 0) sums[tid >> 6][0] = c;
        __syncthreads();
        c = 0.0f;
        for (int i = 0; i < threads / 64; ++i) c += sums[i][0];
        c *= 1.0f / static_cast<float>(a.hidden);
#pragma unroll
        for (int i = 0; i < VPT; ++i) {
            const int v = i * threads + tid;
            float o[8];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                o[j] = __builtin_fmaf(gf[i][j] - (zf[i][j] * rstd) * c, rstd, mf[i][j]);
            if (v < V) (static_cast<u32x4 *>(a.grad_x) + row * V)[v] = pack8(o);
        }
        return;
    }
    const int v = (blockIdx.x - row_blocks) * 8 + (tid & 7);
    float s[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
    if (v < V) {
#pragma unroll 4
        for (int64_t row = tid >> 3; row < a.num_tokens; row += threads / 8) {
            const float rstd = a.rstd[row];
            float zf[8], gf[8];
            unpack8((static_cast<const u32x4 *>(a.z) + row * V)[v], zf);
            unpack8((static_cast<const u32x4 *>(a.grad_y) + row * V)[v], gf);
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] += gf[j] * (zf[j] * rstd);
        }
    }
#pragma unroll
    for (int d = 8; d < 64; d <<= 1)
#pragma unroll
        for (int j = 0; j < 8; ++j) s[j] += __shfl_xor(s[j], d);
    if (lane < 8)
#pragma unroll
        for (int j = 0; j < 8; ++j) sums[tid >> 6][lane * 8 + j] = s[j];
    __syncthreads();
    const int64_t ch = static_cast<int64_t>(blockIdx.x - row_blocks) * 64 + tid;
    if (tid >= 64 || ch >= a.hidden) return;
    float total = sums[0][tid];
    for (int w = 1; w < threads / 64; ++w) total += sums[w][tid];
    a.grad_weight[ch] = total;
}

// Sums of the blocks' rows, 32 channels a block: 8 lanes of 4 channels, 128 groups
// that take every 128th row.  A group's loads are independent of each other, so
// the kernel lasts a few memory latencies (8 groups of 64 loads in a chain took
// 8 to 10 us for 512 rows of 7168).
constexpr int kSumThreads = 1024;

__global__ __launch_bounds__(kSumThreads) void norm_grad_sum_kernel(const float *partial, int rows,
                                                                    int hidden, float *out) {
    __shared__ f32x4 sums[kSumThreads / 64][8];
    const int lane = threadIdx.x & 7, group = threadIdx.x >> 3;
    const int c = (blockIdx.x * 8 + lane) * 4;
    f32x4 s = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    if (c < hidden) {
#pragma unroll 4
        for (int r = group; r < rows; r += kSumThreads / 8)
            s += *reinterpret_cast<const f32x4 *>(partial + static_cast<int64_t>(r) * hidden + c);
    }
#pragma unroll
    for (int d = 8; d < 64; d <<= 1)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[i] += __shfl_xor(s[i], d);
    if ((threadIdx.x & 63) < 8) sums[threadIdx.x >> 6][lane] = s;
    __syncthreads();
    if (threadIdx.x >= 8 || c >= hidden) return;
    s = sums[0][lane];
#pragma unroll
    for (int w = 1; w < kSumThreads / 64; ++w) s += sums[w][lane];
    *reinterpret_cast<f32x4 *>(out + c) = s;
}

hipError_t launch_few(const NormGradArgs &a, int rows, int columns, hipStream_t stream) {
    const int V = a.hidden / 8, blocks = rows + columns;
    if (blocks == 0) return hipSuccess;
    if (V <= 512) norm_grad_few_kernel<1><<<blocks, 512, 0, stream>>>(a, rows);
    else if (V <= 1024) norm_grad_few_kernel<1><<<blocks, 1024, 0, stream>>>(a, rows);
    else norm_grad_few_kernel<4><<<blocks, 1024, 0, stream>>>(a, rows);
    return hipGetLastError();
}

// Whether two buffers of `bytes` bytes share some.
bool overlap(const void *p, const void *q, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return a < b + bytes && b < a + bytes;
}

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs &a, hipStream_t stream) {
    if (!a.out_q) return launch_norm<kSfNone>(a, stream);
    return a.sf.ue8m0 ? launch_norm<EP_SF_UE8M0>(a, stream) : launch_norm<EP_SF_F32>(a, stream);
}

// Two blocks a compute unit: 384 to 512 of them took 47 to 48 us at 4096 x 7168, 640 and
// more 53 and more (their sums' rows), 256 took 51.
int norm_grad_blocks(int32_t num_tokens) { return num_tokens <= kFewRows ? 0 : 512; }

hipError_t launch_add_rmsnorm_backward(const NormGradArgs &a, hipStream_t stream) {
    const int V = a.hidden / 8;
    if (a.num_tokens <= kFewRows) {
        const int rows = a.grad_x ? a.num_tokens : 0, columns = a.grad_weight ? (V + 7) / 8 : 0;
        // grad_x over grad_y would take from grad_weight's blocks what they have yet to read
        const int64_t bytes = static_cast<int64_t>(a.num_tokens) * a.hidden * 2;
        const bool apart = !overlap(a.grad_x, a.grad_y, bytes) && !overlap(a.grad_x, a.z, bytes);
        if (apart || rows == 0 || columns == 0) return launch_few(a, rows, columns, stream);
        const hipError_t e = launch_few(a, 0, columns, stream);
        return e != hipSuccess ? e : launch_few(a, rows, 0, stream);
    }
    const int blocks = norm_grad_blocks(a.num_tokens);
    const int vpt = V <= 512 ? 1 : V <= 1024 ? 2 : 4;
    const int threads = ((V + vpt - 1) / vpt + 63) / 64 * 64;
    if (vpt == 1) norm_grad_kernel<1><<<blocks, threads, 0, stream>>>(a);
    else if (vpt == 2) norm_grad_kernel<2><<<blocks, threads, 0, stream>>>(a);
    else norm_grad_kernel<4><<<blocks, threads, 0, stream>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.grad_weight) return e;
    norm_grad_sum_kernel<<<(a.hidden + 31) / 32, kSumThreads, 0, stream>>>(a.partial, blocks,
                                                                           a.hidden, a.grad_weight);
    return hipGetLastError();
}

}  // namespace ep
