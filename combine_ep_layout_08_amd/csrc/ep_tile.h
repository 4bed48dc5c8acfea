// Matrix product of one block's tile on gfx950, for the experts' products.
//
// A tile of the output is BQ rows by BP columns: out[q, p] = sum_c Q(q, c) P(p, c), c the
// channels that are summed.  P gives the outputs' contiguous dimension.  In memory an operand
// lies either in rows of channels ("rows": x, or W times x) or channel by channel ("cols":
// W^T times a gradient, or both operands of a weight gradient, where the channels are the
// expert's rows).  A chunk is 128 bytes of channels: 64 in bf16, 128 in int8.
//
// Chunks go from memory straight to LDS (global_load_lds, 16 bytes a lane), `S` of them in a
// ring.  Rows operands: an LDS row is 128 bytes, its 16-byte units permuted by the row's number, so
// that the rows which LDS serves together are in different banks.  Cols operands: an LDS
// row is one channel's BQ or BP values; ds_read_b64_tr_b16 hands each lane the four channels of
// its own column.  The permutations are made by the addresses that the lanes load from, as the
// load's place in LDS is fixed by the lane.
#pragma once

#include "ep_layer_internal.h"
#include "ep_rows.h"

namespace ep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

#define EP_LDS __attribute__((address_space(3)))

// Matrix instructions of M x M outputs.  Lane l holds p = l % M of the first operand, q = l % M
// of the second, 16 bytes of channels at 16 (l / M) of both, and four consecutive outputs in
// each of `groups` groups: p = 4 (64 / M) g + 4 (l / M) + i of q = l % M.
template <int M_>
struct Bf16 {
    static constexpr int M = M_, kBytes = 2, kGroups = M * M / 256;
    typedef float Acc __attribute__((ext_vector_type(4 * kGroups)));
    static __device__ inline Acc mma(u32x4 p, u32x4 q, Acc c) {
        const bf16x8 a = __builtin_bit_cast(bf16x8, p), b = __builtin_bit_cast(bf16x8, q);
        if constexpr (M == 16) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
        else return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
    }
};

// Sums of 32768 products of codes stay below 2^30: nothing is rounded.
template <int M_>
struct Int8 {
    static constexpr int M = M_, kBytes = 1, kGroups = M * M / 256;
    typedef int32_t Acc __attribute__((ext_vector_type(4 * kGroups)));
    static __device__ inline Acc mma(u32x4 p, u32x4 q, Acc c) {
        const i32x4 a = __builtin_bit_cast(i32x4, p), b = __builtin_bit_cast(i32x4, q);
        if constexpr (M == 16) return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
        else return __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, c, 0, 0, 0);
    }
};

// A value that is the same in every lane, in a scalar register.
__device__ inline int64_t uniform(int64_t v) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
    const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
    return static_cast<int64_t>(lo | static_cast<uint64_t>(hi) << 32);
}

__device__ inline const char *uniform(const void *p) {
    return reinterpret_cast<const char *>(uniform(reinterpret_cast<int64_t>(p)));
}

// 16 bytes a lane from memory to LDS at `to` + 16 lane, `to` the same in all lanes.  The
// compiler does not count these loads: wait_loads() does.  (Its builtin makes it wait for all
// of them before any read of LDS.)  Lanes that are switched off write nothing.
__device__ inline void load_lds(uint32_t to, const char *base, uint32_t off) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :: "s"(to), "v"(off), "s"(base) : "memory");
}

__device__ inline void load_lds(uint32_t to, const char *from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :: "s"(to), "v"(from) : "memory");
}

// Until at most N of the wave's loads are under way, and its LDS stores are done.
template <int N>
__device__ inline void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" :: "n"(N) : "memory");
}

__device__ inline void block_barrier() {
    asm volatile("s_barrier" ::: "memory");
}

__device__ inline uint32_t lds_address(const void *p) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((EP_LDS const char *)p));
}

__device__ inline u32x4 read_lds(uint32_t at) {
    return *reinterpret_cast<EP_LDS u32x4 *>(static_cast<uintptr_t>(at));
}

__device__ inline void zero_lds(uint32_t at) {
    *reinterpret_cast<EP_LDS u32x4 *>(static_cast<uintptr_t>(at)) = u32x4{0u, 0u, 0u, 0u};
}

// Where the rows of a token-rows call lie: the slot's token, inside the batch whatever the
// layout holds (a call captured for fewer tokens than a later layout has reads the last of
// its own).
__device__ inline int64_t token_of(const int32_t *src_meta, int64_t row, int topk, int tokens) {
    const int64_t t = src_meta[row] / topk;
    return t < 0 ? 0 : t < tokens ? t : tokens - 1;
}

// ---------------------------------------------------------------- operands
// An operand of R rows in rows of channels.  `Threads` threads bring a chunk in kLoads loads
// each: load i takes row i * Threads / 8 + thread / 8.  `row_of(i)` gives the row's byte offset
// from `base` (GATHER: its address).
template <int R, int Threads, bool GATHER>
struct RowsOperand {
    static constexpr int kBytes = R * 128;
    static constexpr int kLoads = kBytes / (Threads * 16) > 0 ? kBytes / (Threads * 16) : 1;
    static constexpr bool kPart = kBytes < Threads * 16;     // not every wave loads
    static_assert(kBytes % (Threads * 16) == 0 || kPart, "whole loads");
    const char *base;
    uint32_t off[GATHER ? 1 : kLoads];
    const char *from[GATHER ? kLoads : 1];
    uint32_t to;             // of the wave's first load in a stage
    int unit;                // of 16 bytes in the chunk, the same in every load
    bool mine;

    static __device__ int row(int i) { return i * (Threads / 8) + threadIdx.x / 8; }
    static __device__ int swizzle(int r) { return (r & 7) ^ ((r >> 4) & 1); }

    template <typename RowOf>
    __device__ void init(const void *b, RowOf row_of) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        base = uniform(b);
        unit = (threadIdx.x & 7) ^ swizzle(threadIdx.x >> 3);
        to = wave * 1024;
        mine = !kPart || wave * 1024 < kBytes;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int64_t at = row_of(mine ? row(i) : 0) + unit * 16;
            if (GATHER) from[i] = base + at;
            else off[i] = static_cast<uint32_t>(at);
        }
    }
    // Load i of the next chunk to `stage`, all of its channels; advance() after the last one.
    __device__ void load(uint32_t stage, int i) {
        if (kPart && !mine) return;
        if (GATHER) {
            load_lds(stage + to + i * Threads * 16, from[i]);
            from[i] += 128;
        } else {
            load_lds(stage + to + i * Threads * 16, base, off[i]);
        }
    }
    __device__ void advance() {
        if (!GATHER) base += 128;
    }
    // The last chunk, of which T has `channels`; what is missing is zeros.
    template <typename T, int N>
    __device__ void load_end(uint32_t stage, int channels) {
        if (kPart && !mine) return;
        const bool in = unit * 16 < channels * T::kBytes;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t at = stage + to + i * Threads * 16;
            if (!in) zero_lds(at + (threadIdx.x & 63) * 16);
            else if (GATHER) load_lds(at, from[i]);
            else load_lds(at, base, off[i]);
        }
    }
    // The wave's operand of a matrix instruction: rows M t .., the k-th 1024 / M bytes of channels.
    template <int M>
    static __device__ u32x4 fragment(uint32_t stage, int t, int k) {
        const int lane = threadIdx.x & 63;
        return read_lds(stage + (M * t + lane % M) * 128 +
                        (((k * (64 / M) + lane / M) ^ swizzle(M * t + lane % M)) << 4));
    }
};

// An operand of C columns, channel by channel, in bf16.  `from(i)` gives the byte offset of the
// thread's 16 bytes in load i from `base`, or its address (GATHER).
template <int C, int Threads, bool GATHER>
struct ColsOperand {
    static constexpr int kRow = 2 * C;                       // bytes of a channel
    static constexpr int kBytes = 64 * kRow;
    static constexpr int kLoads = kBytes / (Threads * 16);
    static constexpr bool kPart = false, mine = true;
    static_assert(kBytes % (Threads * 16) == 0 && C >= 128, "whole loads");
    const char *base;
    int64_t pitch;           // bytes from a channel to the next
    uint32_t col;            // byte offset of the thread's unit in its channel, as loaded
    uint32_t off[kLoads];
    const int32_t *src_meta; // GATHER: of the segment's rows
    int topk, tokens;
    uint32_t to;

    static __device__ int channel(int i) { return (i * Threads + threadIdx.x) / (kRow / 16); }
    // Units of 32 bytes are permuted by these bits of the channel: a read takes 32 bytes of
    // four consecutive channels in each row of 16 lanes, rows of lanes being 8 channels apart.
    static __device__ int swizzle(int ch) { return (ch & 3) | ((ch >> 1) & 4); }

    // Columns `first` .. of `cols` (in a row of `pitch` bytes) from channel 0 at `b`.
    __device__ void init(const void *b, int64_t row_pitch, int first, int cols) {
        base = uniform(b);
        pitch = uniform(row_pitch);
        to = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int ch = channel(i);
            const int unit = (threadIdx.x % (kRow / 16)) ^ (swizzle(ch) << 1);
            int c = first + unit * 8;
            if (c >= cols) c = cols - 8;                     // computed on, and not stored
            off[i] = (GATHER ? 0u : static_cast<uint32_t>(ch * pitch)) + 2u * c;
        }
    }
    __device__ void gather(const int32_t *meta, int k, int t) {
        src_meta = meta;
        topk = k;
        tokens = t;
    }
    // Load i of the next chunk to `stage`, all of its channels; advance() after the last one.
    __device__ void load(uint32_t stage, int i) { load_one(stage + to + i * Threads * 16, i); }
    __device__ void advance() {
        if (GATHER) src_meta += 64;
        else base += 64 * pitch;
    }
    // The last chunk, of which `channels` are there; what is missing is zeros.
    template <typename T, int N>
    __device__ void load_end(uint32_t stage, int channels) {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t at = stage + to + i * Threads * 16;
            if (channel(i) < channels) load_one(at, i);
            else zero_lds(at + (threadIdx.x & 63) * 16);
        }
    }
    __device__ void load_one(uint32_t at, int i) {
        if (GATHER)
            load_lds(at, base + token_of(src_meta, channel(i), topk, tokens) * pitch + off[i]);
        else
            load_lds(at, base, off[i]);
    }
    template <int M>
    static __device__ u32x4 fragment(uint32_t stage, int t, int k) {
        const int lane = threadIdx.x & 63, j = lane & 15;
        const int ch = k * (512 / M) + lane / M * 8 + (j >> 2);
        const int unit = t * (M / 16) + lane % M / 16;       // 16 columns
        u32x4 v;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const int c = ch + 4 * i;
            const uint32_t at = stage + c * kRow + ((unit ^ swizzle(c)) << 5) + (j & 3) * 8;
            const u32x2 r = __builtin_bit_cast(
                u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                           reinterpret_cast<EP_LDS s16x4 *>(static_cast<uintptr_t>(at))));
            v[2 * i] = r.x;
            v[2 * i + 1] = r.y;
        }
        return v;
    }
};

// ---------------------------------------------------------------- main loop
template <int N>
struct Int {
    static constexpr int value = N;
};

// WQ x WP waves, each TQ x TP matrix instructions; rings of SQ chunks of Q and SP of P, SP being SQ
// or one more.
template <typename T, int BQ_, int BP_, int WQ_, int WP_, int SQ_, int SP_>
struct Tile {
    typedef T Type;
    static constexpr int BQ = BQ_, BP = BP_, WQ = WQ_, WP = WP_, SQ = SQ_, SP = SP_;
    static_assert(SQ >= 2 && (SP == SQ || SP == SQ + 1), "what the waits count on");
    static constexpr int M = T::M, TQ = BQ / M / WQ, TP = BP / M / WP;
    static constexpr int kThreads = 64 * WQ * WP;
    static constexpr int kBlocks = kThreads >= 512 || TQ * TP > 32 ? 1 : 512 / kThreads;
    typedef typename T::Acc Acc;
    struct Sums {
        Acc v[TQ][TP];
    };
    static constexpr int kStageQ = BQ * 128, kStageP = BP * 128;
    static constexpr int kRingQ = SQ * kStageQ, kLds = kRingQ + SP * kStageP;
    static_assert(kLds <= 160 * 1024, "LDS of a compute unit");
};

// Sums of the tile over `channels` channels, of its first `rows` rows at least (a wave has row
// tiles wq, WQ + wq, 2 WQ + wq .., and leaves out pairs of them that are behind the rows; ALL: none).
// `lds`: kLds bytes; when this returns a wave may still be reading them.
//
// A chunk is multiplied in two halves of 64 bytes.  While the first half of chunk c is
// multiplied its second half is read from LDS; then comes the chunk's one barrier (chunk c is
// read by all, chunk c + 1 has come), and while the second half is multiplied the first half
// of chunk c + 1 is read.  Q's loads of chunk c + SQ set out after the barrier, P's of chunk c + SP
// half a chunk later, into the room of chunk c.
template <typename C, bool ALL, typename Q, typename P>
__device__ inline void tile_product(Q &q, P &p, int channels, int rows, uint32_t lds,
                                    typename C::Sums &sums) {
    typedef typename C::Type T;
    constexpr int TQ = C::TQ, TP = C::TP, kPerChunk = 128 / T::kBytes;
    constexpr int NQ = Q::kLoads, NP = P::kLoads;
    static_assert(!P::kPart, "every wave loads of P");
    const int active = (rows + C::M * C::WQ - 1) / (C::M * C::WQ);       // row tiles a wave
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wq = wave / C::WP, wp = wave % C::WP;
    const int chunks = (channels + kPerChunk - 1) / kPerChunk, whole = channels / kPerChunk;
#pragma unroll
    for (int a = 0; a < C::TQ; ++a)
#pragma unroll
        for (int b = 0; b < TP; ++b) sums.v[a][b] = typename C::Acc(0);
    if (chunks == 0) return;
    const uint32_t ring_q = lds, ring_p = lds + C::kRingQ;
    auto load = [&](auto &o, auto count, int chunk, uint32_t stage) {
        constexpr int N = decltype(count)::value;
        if (chunk < whole) {
#pragma unroll
            for (int i = 0; i < N; ++i) o.load(stage, i);
            o.advance();
        } else if (chunk < chunks) {
            o.template load_end<T, N>(stage, channels - chunk * kPerChunk);
        }
    };
    // Until chunk c has come.  Behind its loads SQ - 2 chunks of Q and SP - 2 of P set out, in the
    // first wait one more (AHEAD); only whole chunks have a known number of loads.
    auto arrived = [&](int c, auto ahead) {
        constexpr int BQ = C::SQ - 2 + decltype(ahead)::value;
        constexpr int BP = C::SP - 2 + decltype(ahead)::value;
        if (c + BP >= whole) wait_loads<0>();
        else if (Q::kPart && !q.mine) wait_loads<BP * NP>();
        else wait_loads<BQ * NQ + BP * NP>();
    };
    constexpr int K = C::M / 16;                 // matrix instructions of 64 bytes of channels
    struct Half {
        u32x4 q[TQ][K], p[TP][K];
    };
    auto read = [&](Half &f, uint32_t stage_q, uint32_t stage_p, int half, int i) {
        const int k = i % K, t = i / K;
        if (t < TP)
            f.p[t][k] = P::template fragment<C::M>(stage_p, wp * TP + t, half * K + k);
        else
            f.q[t - TP][k] =
                Q::template fragment<C::M>(stage_q, (t - TP) * C::WQ + wq, half * K + k);
    };
    // Multiplies `now`, a row tile at a time, while `then` is read and, with LOAD, the N loads of
    // a chunk set out.  Issued all at once the loads take the address unit 16 cycles each, in
    // which nothing is multiplied; spread over all row tiles they come later (64 experts, 512 rows
    // each, 7168 to 4096 bf16 channels: 1.55 ms, 1.53 spread over all, 1.51 over a half).
    // Reads and loads of a tile that leaves out row tiles are made in those that are left.
    auto step = [&](const Half &now, Half &then, uint32_t stage_q, uint32_t stage_p, int half,
                    auto &o, auto count, uint32_t room, auto with) {
        constexpr int N = decltype(count)::value;
        // row tiles in which loads set out; the ones that are never left out
        constexpr int kMost = ALL ? (TQ + 1) / 2 : 2, kEarly = TQ < kMost ? TQ : kMost;
#pragma unroll
        for (int a = 0; a < TQ; ++a) {
            if (!ALL && a >= kEarly && a % 2 == 0 && a >= active) break;
            if constexpr (decltype(with)::value != 0) {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (i * kEarly / N == a) o.load(room, i);
                if (a == kEarly - 1) o.advance();
            }
#pragma unroll
            for (int i = 0; i < (TP + TQ) * K; ++i)
                if (ALL ? i * TQ / ((TP + TQ) * K) == a
                        : i < TP * K ? i * kEarly / (TP * K) == a : i / K - TP == a)
                    read(then, stage_q, stage_p, half, i);
#pragma unroll
            for (int k = 0; k < K; ++k)
#pragma unroll
                for (int b = 0; b < TP; ++b)
                    sums.v[a][b] = T::mma(now.p[b][k], now.q[a][k], sums.v[a][b]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    // in the order of the loop: P's chunk ahead of Q's by SP - SQ
    constexpr int D = C::SP - C::SQ;
#pragma unroll
    for (int i = 0; i < C::SP; ++i) {
        if (i >= D) load(q, Int<NQ>(), i - D, ring_q + (i - D) * C::kStageQ);
        load(p, Int<NP>(), i, ring_p + i * C::kStageP);
    }
    arrived(0, Int<1>());
    block_barrier();
    uint32_t at_q = ring_q, at_p = ring_p, free_p = 0;
    Half first, second;
#pragma unroll
    for (int i = 0; i < (TP + TQ) * K; ++i) read(first, at_q, at_p, 0, i);
    // `steady`: the chunks that set out are whole ones
    auto chunk = [&](int c, auto steady) {
        constexpr bool kSteady = decltype(steady)::value != 0;
        if (!kSteady && c > 0) load(p, Int<NP>(), c - 1 + C::SP, free_p);
        if (kSteady && c > 0) step(first, second, at_q, at_p, 1, p, Int<NP>(), free_p, Int<1>());
        else step(first, second, at_q, at_p, 1, p, Int<NP>(), free_p, Int<0>());
        arrived(c + 1, Int<0>());
        block_barrier();
        const uint32_t free_q = at_q;
        free_p = at_p;
        if (!kSteady) load(q, Int<NQ>(), c + C::SQ, free_q);
        at_q = at_q + C::kStageQ == ring_p ? ring_q : at_q + C::kStageQ;
        at_p = at_p + C::kStageP == lds + C::kLds ? ring_p : at_p + C::kStageP;
        // behind the last chunk nothing has come: what is read is not used
        step(second, first, at_q, at_p, 0, q, Int<NQ>(), free_q, Int<kSteady>());
    };
    int c = 0;
    chunk(c++, Int<0>());
    for (; c + C::SQ < whole && c + C::SP <= whole; ++c) chunk(c, Int<1>());
    for (; c < chunks; ++c) chunk(c, Int<0>());
}

}  // namespace ep
