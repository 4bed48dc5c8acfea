// The experts' products on gfx950 (include/ep_expert.h): int8 rows and weights, the bf16
// gated feed-forward block, and its gradients.
#include <atomic>
#include <type_traits>

#include "ep_expert_internal.h"
#include "ep_tile.h"

namespace ep {
namespace {

// ---------------------------------------------------------------- tiles of the experts' rows
// Every expert's rows are cut into as few row tiles of at most `per` rows as they need, about
// equal ones, and every row tile meets `across` tiles of outputs.
struct Place {
    int expert;              // -1: no such tile
    int start, rows;         // rows of the layout
    int column;              // tile of outputs
    int tiles;               // row tiles of the expert
};

// Block `id` of those of a launch: blocks go round the 8 XCDs, each with an L2 of its own, so
// block id takes tile id / 8 of the (id % 8)-th part of all tiles.  An expert's tiles follow
// each other, row tiles fastest, so what is under way on an XCD at a time shares weights.
__device__ inline Place find_tile(const Segments &seg, int64_t id, int per, int across, int lane) {
    const int experts = seg.num_experts;
    int count = 0, upto = 0, start = 0;          // of the lane's expert; row tiles up to it
    auto load = [&](int e0) {
        const int e = e0 + lane;
        count = e < experts ? seg.counts[e] : 0;
        start = e < experts ? seg.psum[e] : 0;
        if (count < 0) count = 0;
        upto = (count + per - 1) / per;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int below = __shfl_up(upto, d);
            if (lane >= d) upto += below;
        }
    };
    int64_t all = 0;
    for (int e0 = 0; e0 < experts; e0 += 64) {
        load(e0);
        all += __builtin_amdgcn_readlane(upto, 63);
    }
    all *= across;
    const int64_t part = (all + 7) / 8, tile = (id & 7) * part + (id >> 3);
    if ((id >> 3) >= part || tile >= all) return {-1, 0, 0, 0, 0};
    int pass = static_cast<int>(tile / across);
    int64_t before = 0;      // row tiles of the experts so far
    for (int e0 = 0; e0 < experts; e0 += 64) {
        if (experts > 64) load(e0);
        const int sum = __builtin_amdgcn_readlane(upto, 63);
        if (pass >= sum) {
            pass -= sum;
            before += sum;
            continue;
        }
        // the first lane whose sum is past the number
        const int l = __builtin_amdgcn_readfirstlane(
            __ffsll(static_cast<unsigned long long>(__ballot(upto > pass))) - 1);
        const int rows = __builtin_amdgcn_readlane(count, l), tiles = (rows + per - 1) / per;
        before += __builtin_amdgcn_readlane(upto, l) - tiles;
        const int at = static_cast<int>(tile - before * across);
        const int size = ((rows + tiles - 1) / tiles + 15) / 16 * 16;
        const int first = at % tiles * size;
        return {e0 + l, __builtin_amdgcn_readlane(start, l) + first,
                rows - first < size ? rows - first : size, at / tiles, tiles};
    }
    return {-1, 0, 0, 0, 0};
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
    p->tiles = __builtin_amdgcn_readfirstlane(p->tiles);
    if (p->start < 0 || p->start >= seg.capacity) return false;
    if (p->rows > seg.capacity - p->start) p->rows = static_cast<int>(seg.capacity - p->start);
    return true;
}

// A tile that is full or nearly so has code of its own: what decides on the row tiles to leave out
// costs 2 %.
template <typename C, typename Q, typename P>
__device__ inline void expert_product(Q &q, P &p, int channels, int rows, uint32_t lds,
                                      typename C::Sums &sums) {
    if (C::TQ <= 2 || rows > 16 * C::WQ * (C::TQ - 2))
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
// The sums lie in the lanes as four outputs of one row from each matrix instruction.  Which weight
// goes to which place of the tile is free: a lane's outputs of two instructions are made consecutive,
// and it stores these 8 (16 bytes) at a time, the four lanes of a row 64 bytes that lie together.
// What bounds them (64 experts, 7168 channels, 2 x 2048 outputs and back, bf16): few rows an expert,
// the weights' bytes, 16 rows 543 us (6.9 TB/s; up and gate) and 298 (6.3; down); many rows, the
// matrix units and the clock that the card holds under them: 512 rows an expert 1.48 to 1.52 ms (1265
// to 1300 TFLOP/s; matrix units busy 73 % of the cycles at 1.7 to 1.8 of 2.4 GHz) and, as routing
// leaves them, not multiples of the tile, 1.61 to 1.70 (64 %).  GATHER's addresses are two registers
// a load: its tiles of 256 x 256 spill 6 or 7, around the last chunks (int8 prompt of 4096 tokens,
// 8 of 64 experts: 900 us from the tokens' own rows, 888 from expanded ones; the bf16 block 2583 and
// 2601).
template <typename C, int OUT, bool COLS, bool GATHER, bool ONCE>
struct ExpertTile {
    static constexpr bool I8 = C::Type::kBytes == 1;
    static constexpr int TQ = C::TQ, TP = C::TP;
    static constexpr int G = OUT == kGated ? TP / 2 : TP;    // matrix instructions of outputs
    static constexpr int BP = 16 * C::WP * G;                // outputs of a tile
    static constexpr int U = 4 * G < 8 ? 4 * G : 8;          // stored at a time
    typedef RowsOperand<C::BQ, C::kThreads, GATHER, false> Q;
    typedef std::conditional_t<COLS, ColsOperand<C::BP, C::kThreads, false, true, ONCE>,
                               RowsOperand<C::BP, C::kThreads, false, ONCE>> P;
    const ExpertArgs &a;
    const Place &at;

    __device__ void start_q(Q &q) const {
        const int64_t pitch = static_cast<int64_t>(a.k) * C::Type::kBytes;
        if constexpr (GATHER)
            q.init(a.x, [&](int r) {
                const int64_t row = at.start + (r < at.rows ? r : at.rows - 1);
                return token_of(a.seg.src_meta, row, a.seg.num_topk, a.seg.num_tokens) * pitch;
            });
        else
            q.init(static_cast<const char *>(a.x) + at.start * pitch, [&](int r) {
                return (r < at.rows ? r : at.rows - 1) * pitch;
            });
    }
    __device__ void start_p(P &p) const {
        const int64_t pitch = static_cast<int64_t>(a.k) * C::Type::kBytes;
        const int p0 = at.column * BP;
        const char *w = static_cast<const char *>(a.w) +
                        at.expert * ((OUT == kGated ? 2 : 1) * static_cast<int64_t>(a.n) * pitch);
        if constexpr (COLS) {
            p.init(w, 2 * static_cast<int64_t>(a.n), p0, a.n);
        } else {
            // LDS row i of a wave's instruction t is what lane part i / 4 has of it; gated, the
            // instructions of the upper half are up's
            p.init(w, [&](int r) {
                const int i = r % 16, t = r / 16 % TP;
                const int g = t % G * 4;                     // of the lane part's outputs
                int j = p0 + r / (16 * TP) * 16 * G + g / U * 4 * U + i / 4 * U + g % U + i % 4;
                j = j < a.n ? j : a.n - 1;                   // computed on, and not stored
                return (j + (t < G ? 0 : a.n)) * pitch;
            });
        }
    }
    static __device__ void store(void *to, int64_t place, const float *f) {
        uint16_t *o = static_cast<uint16_t *>(to) + place;
        if constexpr (U == 8)
            *reinterpret_cast<u32x4 *>(o) = pack8(f);
        else
            *reinterpret_cast<u32x2 *>(o) = u32x2{pack2(f[0], f[1]), pack2(f[2], f[3])};
    }
    static __device__ void load(const void *from, int64_t place, float *f) {
        const uint16_t *o = static_cast<const uint16_t *>(from) + place;
        if constexpr (U == 8) {
            unpack8(*reinterpret_cast<const u32x4 *>(o), f);
        } else {
            const u32x2 v = *reinterpret_cast<const u32x2 *>(o);
            f[0] = bf16_lo(v.x);
            f[1] = bf16_hi(v.x);
            f[2] = bf16_lo(v.y);
            f[3] = bf16_hi(v.y);
        }
    }
    __device__ void finish(const typename C::Sums &sums) const {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int wq = wave / C::WP, wp = wave % C::WP, lane = threadIdx.x & 63;
        const int col0 = at.column * BP + wp * 16 * G + (lane >> 4) * U;     // the lane's first output
        const int64_t w_at = at.expert * ((OUT == kGated ? 2 : 1) * static_cast<int64_t>(a.n));
#pragma unroll
        for (int t = 0; t < TQ; ++t) {
            const int m = (t * C::WQ + wq) * 16 + (lane & 15);
            const bool in = m < at.rows;
            if (OUT != kGateGrad && !in) continue;
            const int64_t row = at.start + (in ? m : 0);
            float xs = 1.0f, w = 1.0f, total = 0.0f;
            if (I8)
                xs = a.x_scale[GATHER ? token_of(a.seg.src_meta, row, a.seg.num_topk,
                                                 a.seg.num_tokens)
                                      : row];
            if (OUT != kPlain && a.row_weights && in) w = a.row_weights[row];
#pragma unroll
            for (int u = 0; u < 4 * G; u += U) {             // of the lane's outputs
                const int col = col0 + 4 * u;
                if (!in || col >= a.n) continue;
                float v[U], up[U];
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    v[i] = static_cast<float>(sums.v[t][(u + i) / 4][i % 4]);
                    if (OUT == kGated)
                        up[i] = static_cast<float>(sums.v[t][(G + (u + i) / 4) % TP][i % 4]);
                }
                if (I8) {
#pragma unroll
                    for (int i = 0; i < U; i += 4) {
                        const float *ws = a.w_scale + w_at + col + i;
                        const f32x4 s = *reinterpret_cast<const f32x4 *>(ws);
                        f32x4 su = s;
                        if (OUT == kGated) su = *reinterpret_cast<const f32x4 *>(ws + a.n);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            v[i + j] = v[i + j] * xs * s[j];
                            if (OUT == kGated) up[i + j] = up[i + j] * xs * su[j];
                        }
                    }
                }
                if (OUT == kGated) {
                    if (a.saved) {
                        store(a.saved, row * 2 * a.n + col, v);
                        store(a.saved, row * 2 * a.n + a.n + col, up);
                    }
#pragma unroll
                    for (int i = 0; i < U; ++i) v[i] = v[i] * sigmoid(v[i]) * up[i] * w;
                }
                if (OUT != kGateGrad) {
                    store(a.out, row * a.n + col, v);
                    continue;
                }
                float g[U], h[U], og[U], ou[U];
                load(a.gate_up, row * 2 * a.n + col, g);
                load(a.gate_up, row * 2 * a.n + a.n + col, up);
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    const float s = sigmoid(g[i]);
                    const float silu = g[i] * s, whole = silu * up[i];
                    total = __builtin_fmaf(v[i], whole, total);
                    const float wg = w * v[i];
                    og[i] = wg * up[i] * (s * __builtin_fmaf(g[i], 1.0f - s, 1.0f));
                    ou[i] = wg * silu;
                    h[i] = w * whole;
                }
                store(a.grad_gate_up, row * 2 * a.n + col, og);
                store(a.grad_gate_up, row * 2 * a.n + a.n + col, ou);
                if (a.out) store(a.out, row * a.n + col, h);
            }
            if (OUT == kGateGrad && a.partial) {
                total += __shfl_xor(total, 16);
                total += __shfl_xor(total, 32);
                if (lane < 16 && in)
                    a.partial[(at.column * C::WP + wp) * a.seg.capacity + row] = total;
            }
        }
    }
};

// The tile's sums, operands as E has them.
template <typename E, typename C>
__device__ inline void expert_sums(const ExpertArgs &a, const Place &at, uint32_t lds,
                                   typename C::Sums &sums) {
    const E tile{a, at};
    typename E::Q q;
    typename E::P p;
    tile.start_q(q);
    tile.start_p(p);
    expert_product<C>(q, p, a.k, at.rows, lds, sums);
}

template <typename C, int OUT, bool COLS, bool GATHER, bool ONCE>
__global__ __launch_bounds__(C::kThreads, C::kBlocks) void expert_kernel(const ExpertArgs a,
                                                                         int64_t first) {
    typedef ExpertTile<C, OUT, COLS, GATHER, ONCE> E;
    extern __shared__ u32x4 shared[];
    Place at;
    if (!block_tile(a.seg, first, C::BQ, (a.n + E::BP - 1) / E::BP, &at)) return;
    typename C::Sums sums;
    // row tiles that follow each other find an expert's weights in the L2 if the first left them there
    // (64 experts, 4 x 7168 x 2048, us: 2048 rows all on one 276 past the caches, 230 not; half of
    // 3040 on one 710 and 683; 96 tokens of 8 by popularity, 7168 x 2048 int8, where some experts
    // have two tiles: past the caches all 162, those of one tile 165, of one or two 159)
    if (ONCE && at.tiles > 2)
        expert_sums<ExpertTile<C, OUT, COLS, GATHER, false>, C>(a, at, lds_address(shared), sums);
    else
        expert_sums<E, C>(a, at, lds_address(shared), sums);
    E{a, at}.finish(sums);
}

// Gradient of the weights: out[e][j, c] = sum over the expert's rows of g[r, j] x[r, c].  P are
// the columns of x, Q those of g, the rows what is summed.  An expert's rows are few chunks, so a
// tile's sums are soon to be stored: the blocks walk the tiles in one stream of chunks, and the next
// tile's first ones are on their way while one is stored (64 experts of 512 rows, 4096 x 7168: 2.10 ms
// in place of 2.84 with a block a tile; 900 TFLOP/s beside 3.76 GB stored.  Without its stores the
// kernel takes 1.7: of the 0.6 ms that their bytes take a third is hidden).  The matrix units are busy
// 40 % of the cycles, at 2.1 GHz: products and stores of a compute unit's one block follow each other.
// Known to be left (4096 tokens, uneven rows, w13 of 7168 to 2 x 2048 channels):
//   an XCD's eighth of the tiles is of whole experts, so popular ones keep their XCD busy after the
//   others (popularity by rank^-1.2 beside uniform: 64 experts, 8 a token, 3.78 ms and 2.46; 16, 2 a
//   token, 1.20 and 0.58; 8, 1 a token, 0.65 and 0.31);
//   GATHER: a load's address is a token's number that is read just before, which waits for all loads
//   under way, four times a chunk (3.54 ms beside 2.46 from expanded rows);
//   fp32 gradients are twice the bytes (all gradients of the block 7.29 ms and 6.17; 128 tokens 3.01 and
//   2.15).
template <typename C, bool GATHER, bool F32>
struct GradWeightTiles {
    static constexpr int TQ = C::TQ, TP = C::TP;
    static constexpr int kStores = TQ * TP / (F32 ? 1 : 2);
    static_assert(TP % 2 == 0, "8 outputs a lane");
    struct At : Job {
        int expert, q0, p0;
        int start;
    };
    typedef ColsOperand<C::BQ, C::kThreads, false, false, false> Q;
    typedef ColsOperand<C::BP, C::kThreads, GATHER, true, false> P;
    const GradWeightArgs &a;
    const int down, across, wq, wp;
    int64_t id, all, share;
    int expert, start, rows;     // the expert that was looked up last

    __device__ explicit GradWeightTiles(const GradWeightArgs &args)
        : a(args), down((args.n + C::BQ - 1) / C::BQ), across((args.k + C::BP - 1) / C::BP),
          wq(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) / C::WP),
          wp(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6) % C::WP), id(blockIdx.x),
          expert(-1), start(0), rows(0) {
        const uint32_t bits = static_cast<uint32_t>(a.seg.scalars[EP_SCALAR_ERROR_BITS]);
        all = bits & EP_ERRBIT_FATAL ? 0
                                     : static_cast<int64_t>(a.seg.num_experts) * down * across;
        all = uniform(all);
        share = (all + 7) / 8;
    }
    // Tiles without rows are zeros, and are written here.
    EP_INLINE __device__ bool fetch(At &at) {
        for (;; id += gridDim.x) {
            if ((id >> 3) >= share) return false;
            const int64_t tile = (id & 7) * share + (id >> 3);
            if (tile >= all) continue;
            at.expert = static_cast<int>(tile / (down * across));
            const int place = static_cast<int>(tile % (down * across));
            // strips of 6 tiles of Q, tiles of P along them: the 32 that are under way on an XCD have
            // 12 operands between them, which its L2 holds (512 rows an expert, 4096 x 7168 and
            // 7168 x 2048: 2.25 and 1.04 ms with strips of all tiles, 2.21 and 1.03 with 8, 2.13 and
            // 1.02 with 6, 2.14 and 1.07 with 4)
            constexpr int kStrip = 6;
            const int strip = place / (kStrip * across), in = place % (kStrip * across);
            const int left = down - strip * kStrip, high = left < kStrip ? left : kStrip;
            at.q0 = (strip * kStrip + in % high) * C::BQ;
            at.p0 = in / high * C::BP;
            if (at.expert != expert) {
                expert = at.expert;
                // no layout content sends a load out of the rows' buffers
                start = __builtin_amdgcn_readfirstlane(a.seg.psum[expert]);
                rows = __builtin_amdgcn_readfirstlane(a.seg.counts[expert]);
                if (start < 0 || start >= a.seg.capacity || rows < 0) start = rows = 0;
                if (rows > a.seg.capacity - start) rows = static_cast<int>(a.seg.capacity - start);
            }
            at.start = start;
            at.channels = rows;
            if (rows > 0) {
                id += gridDim.x;
                return true;
            }
            clear(at);
        }
    }
    // Zeros, 16 bytes a lane along the rows (one token's gradients, 63 of 64 experts of 7168 and 2048
    // channels without rows: 1197 us stored as sums are, 1078; past the caches 1094).
    EP_INLINE __device__ void clear(const At &at) const {
        constexpr int kEach = F32 ? 4 : 8, kLanes = C::BP / kEach;
        const int thread = thread_here(), c = at.p0 + thread % kLanes * kEach;
        if (c >= a.k) return;
        for (int j = at.q0 + thread / kLanes; j < at.q0 + C::BQ && j < a.n;
             j += C::kThreads / kLanes) {
            const int64_t to = (static_cast<int64_t>(at.expert) * a.n + j) * a.k + c;
            *reinterpret_cast<u32x4 *>(static_cast<char *>(a.out) + to * (F32 ? 4 : 2)) =
                u32x4{0u, 0u, 0u, 0u};
        }
    }
    EP_INLINE __device__ void start_q(Q &q, const At &at) {
        q.init(static_cast<const char *>(a.g) + static_cast<int64_t>(at.start) * a.n * 2,
               2 * static_cast<int64_t>(a.n), at.q0, a.n);
    }
    EP_INLINE __device__ void start_p(P &p, const At &at) {
        p.init(static_cast<const char *>(a.x) +
                   (GATHER ? 0 : static_cast<int64_t>(at.start) * a.k * 2),
               2 * static_cast<int64_t>(a.k), at.p0, a.k);
        if (GATHER) p.gather(a.seg.src_meta + at.start, a.seg.num_topk, a.seg.num_tokens);
    }
    EP_INLINE __device__ bool finish(const At &at, const typename C::Sums &sums) {
        const int lane = thread_here() & 63;
        const int c0 = at.p0 + wp * 16 * TP + (lane >> 4) * 8;      // the lane's first column
#pragma unroll
        for (int t = 0; t < TQ; ++t) {
            const int j = at.q0 + (t * C::WQ + wq) * 16 + (lane & 15);
            if (j >= a.n) continue;
            const int64_t to = (static_cast<int64_t>(at.expert) * a.n + j) * a.k + c0;
#pragma unroll
            for (int u = 0; u < TP; u += 2) {
                if (c0 + 16 * u >= a.k) continue;
                const f32x4 v = sums.v[t][u], w = sums.v[t][u + 1];
                if (F32) {
                    f32x4 *o = reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + to + 16 * u);
                    o[0] = v;
                    o[1] = w;
                } else {
                    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(a.out) + to + 16 * u) =
                        u32x4{pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(w[0], w[1]),
                              pack2(w[2], w[3])};
                }
            }
        }
        return at.q0 + C::BQ <= a.n && at.p0 + C::BP <= a.k;
    }
};

template <typename C, bool GATHER, bool F32>
__global__ __launch_bounds__(C::kThreads, C::kBlocks) void grad_weight_kernel(
    const GradWeightArgs a) {
    extern __shared__ u32x4 shared[];
    GradWeightTiles<C, GATHER, F32> tiles(a);
    tile_stream<C>(tiles, lds_address(shared));
}

// The row weights' gradients from the waves' sums, in the order of their columns.  One thread a
// slot; bound by the latency of the sums' loads, eight of which are under way at a time
// (16 experts of 25 rows, 12 sums: the gradients of the block 43.3 us with one, 41.1).
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
        const float *p = partial + row;
        float v = 0.0f;
        int t = 0;
        for (; t + 8 <= tiles; t += 8, p += 8 * capacity) {
            float s[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) s[j] = p[j * capacity];
#pragma unroll
            for (int j = 0; j < 8; ++j) v += s[j];
        }
        for (; t < tiles; ++t, p += capacity) v += *p;
        out[row] = v;
    }
}

// ---------------------------------------------------------------- launches
// Kernels with more than 64 KB of LDS have to say so, once a device.
template <auto Kernel>
hipError_t allow_lds(int bytes) {
    static std::atomic<uint64_t> said{0};
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const uint64_t bit = uint64_t(1) << (dev & 63);
    if (dev < 64 && (said.load(std::memory_order_relaxed) & bit)) return hipSuccess;
    e = hipFuncSetAttribute(reinterpret_cast<const void *>(Kernel),
                            hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess && dev < 64) said.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

constexpr int64_t kMostBlocks = int64_t(1) << 22;    // of a launch; a multiple of 8

// A block for every tile.
template <typename C, auto Kernel>
hipError_t launch_tiles(const ExpertArgs &a, int64_t tiles, hipStream_t stream) {
    hipError_t e = allow_lds<Kernel>(C::kLds);
    if (e != hipSuccess) return e;
    const int64_t blocks = (tiles + 7) / 8 * 8;
    for (int64_t b = 0; b < blocks; b += kMostBlocks) {
        const int64_t n = blocks - b < kMostBlocks ? blocks - b : kMostBlocks;
        Kernel<<<static_cast<uint32_t>(n), C::kThreads, C::kLds, stream>>>(a, b);
        e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// A block for every compute unit, which walks the tiles.
template <typename C, auto Kernel>
hipError_t launch_stream(const GradWeightArgs &a, int64_t tiles, hipStream_t stream) {
    const hipError_t e = allow_lds<Kernel>(C::kLds);
    if (e != hipSuccess) return e;
    const int64_t blocks = (persistent_grid(tiles, C::kLds > 80 * 1024 ? 1 : 2) + 7) / 8 * 8;
    Kernel<<<static_cast<uint32_t>(blocks), C::kThreads, C::kLds, stream>>>(a);
    return hipGetLastError();
}

int64_t slots_of(const Segments &s) { return static_cast<int64_t>(s.num_tokens) * s.num_topk; }

// No more row tiles than these: every expert's last one may be partly filled.
int64_t row_tiles(const Segments &s, int per) {
    const int64_t slots = slots_of(s);
    return (slots < s.num_experts ? slots : s.num_experts) + slots / per;
}

// sums: of how many waves' columns a row's sums are, for kGateGrad.
template <typename C, int OUT, bool COLS, bool ONCE>
hipError_t launch_expert(const ExpertArgs &a, hipStream_t stream, int *sums) {
    constexpr int BP = OUT == kGated ? C::BP / 2 : C::BP;
    const int across = (a.n + BP - 1) / BP;
    const int64_t tiles = row_tiles(a.seg, C::BQ) * across;
    if (sums) *sums = across * C::WP;
    // the block's product back down reads h, which has no tokens' own rows
    if constexpr (!COLS && (OUT == kGated || C::Type::kBytes == 1)) {
        if (a.token_rows)
            return launch_tiles<C, expert_kernel<C, OUT, COLS, true, ONCE>>(a, tiles, stream);
    }
    return launch_tiles<C, expert_kernel<C, OUT, COLS, false, ONCE>>(a, tiles, stream);
}

// Tile by the rows an expert has on average and the size of the grid, in tiles that there will be
// at least (64 experts of 7168 channels and 2 x 2048 gated outputs, us; 3.76 GB of weights).
//   ONCE: experts have one row tile or two, and their weights are read past the caches: 16 rows 608
//   without and 544 with, 128 tokens of 8 experts 931 and 842 for the whole block.  With more row
//   tiles the others read them from the caches: 192 rows 793 and 775, but the product down 453 and
//   469, and the gradient of x 835 and 841.  Few weights may be in the 256 MB last-level cache from
//   the call before (22 MB: 14.3 without, 18.2 with).
//   32 rows by 128 outputs up to 16 rows an expert (16 by 128: 544 without ONCE at 2 rows and at 4,
//   652 at 16, where 32 by 128 takes 609), 64 by 128 up to 48 (24: 638 with 32 by 128, 613; 48: 777
//   and 629; 64: 746, 256 by 256 630), behind that 256 by 256 (128: 1052 with 64 by 128, 885 with 128
//   by 128, 780 with 128 by 256, 677).  Weights in columns are read in pieces of 512 bytes by tiles of
//   256 outputs, of 256 by tiles of 128: the gradient of the activation 16 rows 343 with 32 by 128,
//   316 with 256 by 256.
//   Large tiles from 256 of them on, one a compute unit.  Below that long sums would gain by them and
//   short ones lose (int8, 8 experts of 512 rows, 7168 to 2048 channels, 128 large tiles: 95 with 64 by
//   128, 81 with 256 by 256; 1024 to 2048 17 and 21; 64 large tiles, 7168 to 1024 37 and 68).
//   A grid that does not fill the card takes smaller tiles (16 experts, 25 rows, 648 channels, 2 x 360
//   outputs and back: 15.6 with 32 by 128, 14.3 with 16 by 128; one token of 8 experts 124 and 122).
template <typename T, int OUT, bool COLS>
hipError_t choose_expert(const ExpertArgs &a, hipStream_t stream, int *sums = nullptr) {
    const int64_t slots = slots_of(a.seg), experts = a.seg.num_experts;
    const int64_t active = slots < experts ? slots : experts;
    const int64_t columns = (OUT == kGated ? 2 : 1) * static_cast<int64_t>(a.n);
    auto tiles = [&](int rows, int cols) {
        return (slots / rows > active ? slots / rows : active) * ((columns + cols - 1) / cols);
    };
    const bool few = slots <= 48 * experts;
    const bool once = few && active * columns * a.k * T::kBytes > (int64_t(64) << 20);
    if ((COLS || !few) && tiles(256, 256) >= 256) {
        typedef Tile<T, 256, 256, 2, 4, 2, 3> C;
        if constexpr (COLS)
            if (once) return launch_expert<C, OUT, COLS, true>(a, stream, sums);
        return launch_expert<C, OUT, COLS, false>(a, stream, sums);
    }
    if (slots > 16 * experts && tiles(64, 128) >= 512) {
        typedef Tile<T, 64, 128, 2, 2, 3, 3> C;
        // in columns never once: up to 48 rows an expert 512 of these tiles are 256 large ones
        if constexpr (!COLS)
            if (once) return launch_expert<C, OUT, COLS, true>(a, stream, sums);
        return launch_expert<C, OUT, COLS, false>(a, stream, sums);
    }
    if (tiles(32, 128) >= 512) {
        typedef Tile<T, 32, 128, 1, 4, 4, 4> C;
        return once ? launch_expert<C, OUT, COLS, true>(a, stream, sums)
                    : launch_expert<C, OUT, COLS, false>(a, stream, sums);
    }
    typedef Tile<T, 16, 128, 1, 4, 4, 4> C;
    return once ? launch_expert<C, OUT, COLS, true>(a, stream, sums)
                : launch_expert<C, OUT, COLS, false>(a, stream, sums);
}

int64_t grad_tiles(const GradWeightArgs &a, int size) {
    return static_cast<int64_t>(a.seg.num_experts) * ((a.n + size - 1) / size) *
           ((a.k + size - 1) / size);
}

}  // namespace

// A wave's columns are 32 at least.
int gate_grad_tiles(int32_t inter) { return (inter + 127) / 128 * 4; }

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
    int tiles = 0;
    const hipError_t e = choose_expert<Bf16, kGateGrad, true>(a, stream, &tiles);
    if (e != hipSuccess || !grad_row_weights) return e;
    const int64_t slots = slots_of(a.seg), blocks = (slots + 255) / 256;
    row_sums_kernel<<<static_cast<uint32_t>(blocks < 4096 ? blocks : 4096), 256, 0, stream>>>(
        dst, a.seg.scalars, slots, a.seg.capacity, a.partial, tiles,
        grad_row_weights);
    return hipGetLastError();
}

hipError_t launch_expert_grad_rows(const ExpertArgs &a, hipStream_t stream) {
    return choose_expert<Bf16, kPlain, true>(a, stream);
}

template <typename C>
static hipError_t launch_grad_weight(const GradWeightArgs &a, hipStream_t stream) {
    const int64_t tiles = grad_tiles(a, C::BQ);
    if (a.f32)
        return a.token_rows ? launch_stream<C, grad_weight_kernel<C, true, true>>(a, tiles, stream)
                            : launch_stream<C, grad_weight_kernel<C, false, true>>(a, tiles, stream);
    return a.token_rows ? launch_stream<C, grad_weight_kernel<C, true, false>>(a, tiles, stream)
                        : launch_stream<C, grad_weight_kernel<C, false, false>>(a, tiles, stream);
}

// Tiles of 256 x 256 where they fill the card, else of 128 x 128 (16 experts of 128 rows, us: 144 large
// tiles 12.0 and 11.4, 128 15.2 and 11.5, 96 8.9 and 7.2; 256 13.7 and 13.9; 32 experts, 2048
// 105 and 116).
hipError_t launch_expert_grad_weight(const GradWeightArgs &a, hipStream_t stream) {
    return grad_tiles(a, 256) >= 192
               ? launch_grad_weight<Tile<Bf16, 256, 256, 2, 4, 2, 3>>(a, stream)
               : launch_grad_weight<Tile<Bf16, 128, 128, 2, 2, 2, 3>>(a, stream);
}

}  // namespace ep
