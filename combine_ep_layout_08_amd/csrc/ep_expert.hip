// The experts' products on gfx950 (include/ep_expert.h): int8 rows and weights, the bf16
// gated feed-forward block, and its gradients.
#include "ep_expert_internal.h"
#include "ep_tile.h"

namespace ep {
namespace {

// 1 / (1 + exp(-g)), as ep_swiglu has it.
__device__ inline float sigmoid(float g) {
    return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g));
}

// ---------------------------------------------------------------- tiles of the experts' rows
// Every expert's rows are cut into as few row tiles of at most `per` rows as they need, about
// equal ones, and every row tile meets `across` tiles of outputs.
struct Place {
    int expert;              // -1: no such tile
    int start, rows;         // rows of the layout
    int column;              // tile of outputs
};

// Block `id` of those of a launch: blocks go round the 8 XCDs, each with an L2 of its own, so
// block id takes tile id / 8 of the (id % 8)-th part of all tiles.  An expert's tiles follow
// each other, row tiles fastest, so what is under way on an XCD at a time shares weights.
__device__ inline Place find_tile(const Segments &seg, int64_t id, int per, int across, int lane) {
    const int experts = seg.num_experts;
    int64_t all = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int e = e0 + lane;
        const int c = e < experts ? seg.counts[e] : 0;
        int t = c > 0 ? (c + per - 1) / per : 0;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) t += __shfl_xor(t, d);
        all += __builtin_amdgcn_readfirstlane(t);
    }
    all *= across;
    const int64_t part = (all + 7) / 8, tile = (id & 7) * part + (id >> 3);
    if ((id >> 3) >= part || tile >= all) return {-1, 0, 0, 0};
    int pass = static_cast<int>(tile / across);
    int64_t before = 0;      // row tiles of the experts so far
    for (int e0 = 0; e0 < experts; e0 += 64) {
        const int e = e0 + lane;
        const int c = e < experts ? seg.counts[e] : 0;
        const int mine = c > 0 ? (c + per - 1) / per : 0;
        int upto = mine;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int below = __shfl_up(upto, d);
            if (lane >= d) upto += below;
        }
        const int sum = __builtin_amdgcn_readlane(upto, 63);
        if (pass >= sum) {
            pass -= sum;
            before += sum;
            continue;
        }
        // the first lane whose sum is past the number
        const int l = __builtin_amdgcn_readfirstlane(
            __ffsll(static_cast<unsigned long long>(__ballot(upto > pass))) - 1);
        const int tiles = __builtin_amdgcn_readlane(mine, l);
        const int count = __builtin_amdgcn_readlane(c, l);
        before += __builtin_amdgcn_readlane(upto, l) - tiles;
        const int at = static_cast<int>(tile - before * across);
        const int size = ((count + tiles - 1) / tiles + 15) / 16 * 16;
        const int first = at % tiles * size;
        return {e0 + l, seg.psum[e0 + l] + first, count - first < size ? count - first : size,
                at / tiles};
    }
    return {-1, 0, 0, 0};
}

// The tile of a block of a launch, inside the rows' buffers whatever the layout holds.
__device__ inline bool block_tile(const Segments &seg, int64_t first, int per, int across,
                                  Place *p) {
    const uint32_t bits = static_cast<uint32_t>(seg.scalars[EP_SCALAR_ERROR_BITS]);
    *p = find_tile(seg, first + blockIdx.x, per, across, threadIdx.x & 63);
    if (p->expert < 0 || (bits & EP_ERRBIT_FATAL)) return false;
    // the same in every lane, which the compiler cannot see
    p->expert = __builtin_amdgcn_readfirstlane(p->expert);
    p->start = __builtin_amdgcn_readfirstlane(p->start);
    p->rows = __builtin_amdgcn_readfirstlane(p->rows);
    p->column = __builtin_amdgcn_readfirstlane(p->column);
    if (p->start < 0 || p->start >= seg.capacity) return false;
    if (p->rows > seg.capacity - p->start) p->rows = static_cast<int>(seg.capacity - p->start);
    return true;
}

// A tile that is full or nearly so has code of its own: what decides on the row tiles to leave out
// costs 2 %.
template <typename C, typename Q, typename P>
__device__ inline void expert_product(Q &q, P &p, int channels, int rows, uint32_t lds,
                                      typename C::Sums &sums) {
    if (C::TQ <= 2 || rows > C::M * C::WQ * (C::TQ - 2))
        tile_product<C, true>(q, p, channels, rows, lds, sums);
    else
        tile_product<C, false>(q, p, channels, rows, lds, sums);
}

enum Out { kPlain, kGated, kGateGrad };

// Products of expert rows: out[r, j] = sum_c x[r, c] w[e][j, c] (COLS: w[e][c, j]).
//   kPlain     rounded to bf16 (int8: times the scales first)
//   kGated     half of the tile's columns are gate's and half up's, wave by wave, so a lane
//              holds both: their activation is what is stored
//   kGateGrad  the sums are the gradient of the activation; gate and up are read, their
//              gradients stored
// The sums lie in the lanes as groups of four consecutive outputs of one row.  Where the weights
// are in rows, which weight goes to which place of the tile is free: a lane's outputs are made
// consecutive, and it stores 8 of them (16 bytes) at a time.
template <typename C, int OUT, bool COLS, bool GATHER>
__global__ __launch_bounds__(C::kThreads, C::kBlocks) void expert_kernel(const ExpertArgs a, int64_t first) {
    constexpr bool I8 = C::Type::kBytes == 1;
    constexpr int TQ = C::TQ, TP = C::TP;
    constexpr int BP = OUT == kGated ? C::BP / 2 : C::BP;    // outputs of a tile
    extern __shared__ u32x4 shared[];
    constexpr int M = C::M, kGroups = C::Type::kGroups;
    const int lane = threadIdx.x & 63, part = lane / M;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wq = wave / C::WP, wp = wave % C::WP;
    const int across = (a.n + BP - 1) / BP;
    Place at;
    if (!block_tile(a.seg, first, C::BQ, across, &at)) return;
    const int p0 = at.column * BP;
    const uint32_t lds = lds_address(shared);
    typename C::Sums sums;
    RowsOperand<C::BQ, C::kThreads, GATHER> q;
    const int64_t pitch = static_cast<int64_t>(a.k) * C::Type::kBytes;
    if (GATHER)
        q.init(a.x, [&](int r) {
            const int64_t row = at.start + (r < at.rows ? r : at.rows - 1);
            return token_of(a.seg.src_meta, row, a.seg.num_topk, a.seg.num_tokens) * pitch;
        });
    else
        q.init(static_cast<const char *>(a.x) + at.start * pitch, [&](int r) {
            return (r < at.rows ? r : at.rows - 1) * pitch;
        });
    const int64_t w_rows = (OUT == kGated ? 2 : 1) * static_cast<int64_t>(a.n);
    if constexpr (COLS) {
        ColsOperand<C::BP, C::kThreads, false> p;
        const char *w = static_cast<const char *>(a.w) +
                        at.expert * static_cast<int64_t>(a.k) * a.n * 2;
        p.init(w, 2 * static_cast<int64_t>(a.n), p0, a.n);
        expert_product<C>(q, p, a.k, at.rows, lds, sums);
    } else {
        RowsOperand<C::BP, C::kThreads, false> p;
        const char *w = static_cast<const char *>(a.w) + at.expert * w_rows * pitch;
        // LDS row i of the wave's tile t is what lane part i / 4 % (64 / M) has in group i M / 256;
        // gated, the tiles of the upper half are up's.
        p.init(w, [&](int r) {
            constexpr int G = OUT == kGated ? TP / 2 : TP, L = 64 / M;
            const int i = r % M, t = r / M % TP;
            int j = p0 + r / (M * TP) * M * G + i / 4 % L * 4 * kGroups * G +
                    t % G * 4 * kGroups + i / (4 * L) * 4 + i % 4;
            j = j < a.n ? j : a.n - 1;                       // computed on, and not stored
            return (j + (t < G ? 0 : a.n)) * pitch;
        });
        expert_product<C>(q, p, a.k, at.rows, lds, sums);
    }
    if constexpr (OUT == kGateGrad) {
        float *const parts = reinterpret_cast<float *>(shared);      // [WP][BQ]
        if (a.partial) block_barrier();                              // the ring is read
#pragma unroll
        for (int t = 0; t < TQ; ++t) {
            const int m = (t * C::WQ + wq) * M + lane % M;
            const bool in = m < at.rows;
            const int64_t row = at.start + (in ? m : 0);
            const float w = a.row_weights && in ? a.row_weights[row] : 1.0f;
            float total = 0.0f;
#pragma unroll
            for (int u = 0; u < TP * kGroups; ++u) {
                const int col = p0 + (wp * TP + u / kGroups) * M + u % kGroups * 8 + 4 * part;
                if (!in || col >= a.n) continue;
                const int64_t gate_at = row * 2 * a.n + col;
                const uint16_t *gu = static_cast<const uint16_t *>(a.gate_up) + gate_at;
                const u32x2 gv = *reinterpret_cast<const u32x2 *>(gu);
                const u32x2 uv = *reinterpret_cast<const u32x2 *>(gu + a.n);
                const float g[4] = {bf16_lo(gv.x), bf16_hi(gv.x), bf16_lo(gv.y), bf16_hi(gv.y)};
                const float up[4] = {bf16_lo(uv.x), bf16_hi(uv.x), bf16_lo(uv.y), bf16_hi(uv.y)};
                float og[4], ou[4], oh[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float gh = sums.v[t][u / kGroups][u % kGroups * 4 + i];
                    const float s = sigmoid(g[i]);
                    const float silu = g[i] * s, whole = silu * up[i];
                    total = __builtin_fmaf(gh, whole, total);
                    const float wg = w * gh;
                    og[i] = wg * up[i] * (s * __builtin_fmaf(g[i], 1.0f - s, 1.0f));
                    ou[i] = wg * silu;
                    oh[i] = w * whole;
                }
                uint16_t *gg = static_cast<uint16_t *>(a.grad_gate_up) + gate_at;
                *reinterpret_cast<u32x2 *>(gg) = u32x2{pack2(og[0], og[1]), pack2(og[2], og[3])};
                *reinterpret_cast<u32x2 *>(gg + a.n) =
                    u32x2{pack2(ou[0], ou[1]), pack2(ou[2], ou[3])};
                if (a.out)
                    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + row * a.n + col) =
                        u32x2{pack2(oh[0], oh[1]), pack2(oh[2], oh[3])};
            }
            if (a.partial) {
                if (M == 16) total += __shfl_xor(total, 16);
                total += __shfl_xor(total, 32);
                if (lane < M) parts[wp * C::BQ + m] = total;
            }
        }
        if (!a.partial) return;
        __syncthreads();
        for (int m = threadIdx.x; m < at.rows; m += C::kThreads) {
            float total = 0.0f;
#pragma unroll
            for (int i = 0; i < C::WP; ++i) total += parts[i * C::BQ + m];
            a.partial[static_cast<int64_t>(at.column) * a.seg.capacity + at.start + m] = total;
        }
        return;
    } else {
        constexpr int G = OUT == kGated ? TP / 2 : TP;       // tiles of outputs a lane has
        constexpr int R = 4 * kGroups;                       // outputs of a tile a lane has
        constexpr int V = COLS ? 4 : R * G;                  // consecutive outputs
        constexpr int U = V < 8 ? V : 8;                     // stored at a time
        const int64_t w_at = at.expert * w_rows;
#pragma unroll
        for (int t = 0; t < TQ; ++t) {
            const int m = (t * C::WQ + wq) * M + lane % M;
            if (m >= at.rows) continue;
            const int64_t row = at.start + m;
            float xs = 1.0f;
            if (I8)
                xs = a.x_scale[GATHER ? token_of(a.seg.src_meta, row, a.seg.num_topk,
                                                 a.seg.num_tokens)
                                      : row];
            const float w = OUT == kGated && a.row_weights ? a.row_weights[row] : 1.0f;
#pragma unroll
            for (int u = 0; u < R * G; u += U) {             // of the lane's outputs
                const int col = COLS ? p0 + (wp * TP + u / R) * M + u % R * 2 + 4 * part
                                     : p0 + wp * M * G + part * R * G + u;
                if (col >= a.n) continue;
                float v[U], up[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    v[i] = static_cast<float>(sums.v[t][(u + i) / R][(u + i) % R]);
                    if (OUT == kGated)
                        up[i] = static_cast<float>(sums.v[t][(G + (u + i) / R) % TP][(u + i) % R]);
                }
                if (I8) {
#pragma unroll
                    for (int i = 0; i < U; i += 4) {
                        const f32x4 s =
                            *reinterpret_cast<const f32x4 *>(a.w_scale + w_at + col + i);
                        f32x4 su = s;
                        if (OUT == kGated)
                            su = *reinterpret_cast<const f32x4 *>(a.w_scale + w_at + a.n + col + i);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[i + j] = v[i + j] * xs * s[j];
                            if (OUT == kGated) up[i + j] = up[i + j] * xs * su[j];
                        }
                    }
                }
                auto store = [&](void *to, int64_t place, const float *f) {
                    uint16_t *o = static_cast<uint16_t *>(to) + place;
                    if constexpr (U == 8)
                        *reinterpret_cast<u32x4 *>(o) = pack8(f);
                    else
                        *reinterpret_cast<u32x2 *>(o) =
                            u32x2{pack2(f[0], f[1]), pack2(f[2], f[3])};
                };
                if (OUT == kGated) {
                    if (a.saved) {
                        store(a.saved, row * 2 * a.n + col, v);
                        store(a.saved, row * 2 * a.n + a.n + col, up);
                    }
#pragma unroll
                    for (int i = 0; i < U; ++i) v[i] = v[i] * sigmoid(v[i]) * up[i] * w;
                }
                store(a.out, row * a.n + col, v);
            }
        }
    }
}

// Gradient of the weights: out[e][j, c] = sum over the expert's rows of g[r, j] x[r, c].  P are
// the columns of x, Q those of g, the rows what is summed.
template <typename C, bool GATHER, bool F32>
__global__ __launch_bounds__(C::kThreads, C::kBlocks) void grad_weight_kernel(const GradWeightArgs a,
                                                                     int64_t first) {
    extern __shared__ u32x4 shared[];
    constexpr int M = C::M, kGroups = C::Type::kGroups;
    const int lane = threadIdx.x & 63, part = lane / M;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wq = wave / C::WP, wp = wave % C::WP;
    const int down = (a.n + C::BQ - 1) / C::BQ, across = (a.k + C::BP - 1) / C::BP;
    const uint32_t bits = static_cast<uint32_t>(a.seg.scalars[EP_SCALAR_ERROR_BITS]);
    const int64_t all = static_cast<int64_t>(a.seg.num_experts) * down * across;
    const int64_t id = first + blockIdx.x, share = (all + 7) / 8;
    const int64_t tile = (id & 7) * share + (id >> 3);
    if ((id >> 3) >= share || tile >= all || (bits & EP_ERRBIT_FATAL)) return;
    const int expert = static_cast<int>(tile / (down * across));
    const int place = static_cast<int>(tile % (down * across));
    const int q0 = place % down * C::BQ, p0 = place / down * C::BP;
    // no layout content sends a load out of the rows' buffers
    int64_t start = __builtin_amdgcn_readfirstlane(a.seg.psum[expert]);
    int64_t rows = __builtin_amdgcn_readfirstlane(a.seg.counts[expert]);
    if (start < 0 || start >= a.seg.capacity || rows < 0) start = rows = 0;
    if (rows > a.seg.capacity - start) rows = a.seg.capacity - start;
    const uint32_t lds = lds_address(shared);
    typename C::Sums sums;
    ColsOperand<C::BQ, C::kThreads, false> q;
    ColsOperand<C::BP, C::kThreads, GATHER> p;
    q.init(static_cast<const char *>(a.g) + start * a.n * 2, 2 * static_cast<int64_t>(a.n), q0, a.n);
    p.init(static_cast<const char *>(a.x) + (GATHER ? 0 : start * a.k * 2),
           2 * static_cast<int64_t>(a.k), p0, a.k);
    if (GATHER) p.gather(a.seg.src_meta + start, a.seg.num_topk, a.seg.num_tokens);
    tile_product<C, true>(q, p, static_cast<int>(rows), C::BQ, lds, sums);
    const int64_t base = static_cast<int64_t>(expert) * a.n;
#pragma unroll
    for (int t = 0; t < C::TQ; ++t) {
        const int j = q0 + (t * C::WQ + wq) * M + lane % M;
        if (j >= a.n) continue;
#pragma unroll
        for (int u = 0; u < C::TP * kGroups; ++u) {
            const int c = p0 + (wp * C::TP + u / kGroups) * M + u % kGroups * 8 + 4 * part;
            if (c >= a.k) continue;
            f32x4 v;
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = sums.v[t][u / kGroups][u % kGroups * 4 + i];
            const int64_t to = (base + j) * a.k + c;
            if (F32)
                *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + to) = v;
            else
                *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(a.out) + to) =
                    u32x2{pack2(v[0], v[1]), pack2(v[2], v[3])};
        }
    }
}

// The row weights' gradients from the tiles' sums, in the tiles' order.  One thread a slot.
__global__ __launch_bounds__(256) void row_sums_kernel(const int32_t *dst, const int32_t *scalars,
                                                       int64_t num_slots, int64_t capacity,
                                                       const float *partial, int tiles,
                                                       float *out) {
    const uint32_t bits = static_cast<uint32_t>(scalars[EP_SCALAR_ERROR_BITS]);
    if (bits & EP_ERRBIT_FATAL) return;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 256;
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < num_slots;
         i += stride) {
        const int32_t row = dst[i];
        if (row < 0 || row >= capacity) continue;
        float v = 0.0f;
        for (int t = 0; t < tiles; ++t) v += partial[t * capacity + row];
        out[row] = v;
    }
}

// ---------------------------------------------------------------- launches
// Kernels with more than 64 KB of LDS have to say so once a device.
template <typename K>
hipError_t allow_lds(K kernel, int bytes) {
    return hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                               hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
}

constexpr int64_t kMostBlocks = int64_t(1) << 22;    // of a launch; a multiple of 8

template <typename C, typename K, typename A>
hipError_t launch_tiles(K kernel, const A &a, int64_t tiles, hipStream_t stream) {
    hipError_t e = allow_lds(kernel, C::kLds);
    if (e != hipSuccess) return e;
    const int64_t blocks = (tiles + 7) / 8 * 8;
    for (int64_t b = 0; b < blocks; b += kMostBlocks) {
        const int64_t n = blocks - b < kMostBlocks ? blocks - b : kMostBlocks;
        kernel<<<static_cast<uint32_t>(n), C::kThreads, C::kLds, stream>>>(a, b);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

int64_t slots_of(const Segments &s) { return static_cast<int64_t>(s.num_tokens) * s.num_topk; }

// No more row tiles than these: every expert's last one may be partly filled.
int64_t row_tiles(const Segments &s, int per) {
    const int64_t slots = slots_of(s);
    return (slots < s.num_experts ? slots : s.num_experts) + slots / per;
}

template <typename C, int OUT, bool COLS>
hipError_t launch_expert(const ExpertArgs &a, hipStream_t stream) {
    constexpr int BP = OUT == kGated ? C::BP / 2 : C::BP;
    const int64_t tiles = row_tiles(a.seg, C::BQ) * ((a.n + BP - 1) / BP);
    if constexpr (!COLS) {
        if (a.token_rows)
            return launch_tiles<C>(expert_kernel<C, OUT, COLS, true>, a, tiles, stream);
    }
    return launch_tiles<C>(expert_kernel<C, OUT, COLS, false>, a, tiles, stream);
}

template <template <int> class T, int OUT, bool COLS>
hipError_t choose_expert(const ExpertArgs &a, hipStream_t stream) {
    const int64_t slots = slots_of(a.seg), experts = a.seg.num_experts;
    if (slots > 64 * experts) return launch_expert<Tile<T<16>, 256, 256, 2, 4, 2, 3>, OUT, COLS>(a, stream);
    if (slots > 16 * experts) return launch_expert<Tile<T<16>, 64, 128, 2, 2, 3, 3>, OUT, COLS>(a, stream);
    if constexpr (COLS)
        return launch_expert<Tile<T<16>, 16, 128, 1, 4, 4, 4>, OUT, COLS>(a, stream);
    else
        return launch_expert<Tile<T<16>, 16, 128, 1, 4, 4, 4>, OUT, COLS>(a, stream);
}

}  // namespace

constexpr int kGateGradColumns = 256;

int gate_grad_tiles(int32_t inter) { return (inter + kGateGradColumns - 1) / kGateGradColumns; }

hipError_t launch_expert_i8(const ExpertArgs &a, bool gated, hipStream_t stream) {
    return gated ? choose_expert<Int8, kGated, false>(a, stream)
                 : choose_expert<Int8, kPlain, false>(a, stream);
}

hipError_t launch_expert_gated(const ExpertArgs &a, hipStream_t stream) {
    return choose_expert<Bf16, kGated, false>(a, stream);
}

hipError_t launch_expert_product(const ExpertArgs &a, hipStream_t stream) {
    return choose_expert<Bf16, kPlain, false>(a, stream);
}

hipError_t launch_expert_gate_grad(const ExpertArgs &a, float *grad_row_weights, const int32_t *dst,
                                   hipStream_t stream) {
    hipError_t e = launch_expert<Tile<Bf16<16>, 256, kGateGradColumns, 2, 4, 2, 3>, kGateGrad, true>(a, stream);
    if (e != hipSuccess || !grad_row_weights) return e;
    const int64_t slots = slots_of(a.seg), blocks = (slots + 255) / 256;
    row_sums_kernel<<<static_cast<uint32_t>(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(
        dst, a.seg.scalars, slots, a.seg.capacity, a.partial, gate_grad_tiles(a.n),
        grad_row_weights);
    return hipGetLastError();
}

hipError_t launch_expert_grad_rows(const ExpertArgs &a, hipStream_t stream) {
    return choose_expert<Bf16, kPlain, true>(a, stream);
}

hipError_t launch_expert_grad_weight(const GradWeightArgs &a, hipStream_t stream) {
    typedef Tile<Bf16<16>, 256, 256, 2, 4, 2, 3> C;
    const int64_t tiles = static_cast<int64_t>(a.seg.num_experts) * ((a.n + C::BQ - 1) / C::BQ) *
                          ((a.k + C::BP - 1) / C::BP);
    if (a.f32)
        return a.token_rows ? launch_tiles<C>(grad_weight_kernel<C, true, true>, a, tiles, stream)
                            : launch_tiles<C>(grad_weight_kernel<C, false, true>, a, tiles, stream);
    return a.token_rows ? launch_tiles<C>(grad_weight_kernel<C, true, false>, a, tiles, stream)
                        : launch_tiles<C>(grad_weight_kernel<C, false, false>, a, tiles, stream);
}

}  // namespace ep
