// Matrix product of one block's tile on gfx950, for the experts' products.
//
// A tile of the output is BQ rows by BP columns: out[q, p] = sum_c Q(q, c) P(p, c), c the
// channels that are summed.  P gives the outputs' contiguous dimension.  In memory an operand
// lies either in rows of channels ("rows": x, or W times x) or channel by channel ("cols":
// W^T times a gradient, or both operands of a weight gradient, where the channels are the
// expert's rows).  A chunk is 128 bytes of channels: 64 in bf16, 128 in int8.
//
// Chunks go from memory straight to LDS (global_load_lds, 16 bytes a lane), `S` of them in a
// ring.  Rows operands: an LDS row is 128 bytes, its 16-byte units permuted by u ^ (row % 8), so
// that the rows which LDS serves together are in different banks.  Cols operands: an LDS
// row is one channel's BQ or BP values; ds_read_b64_tr_b16 hands each lane the four channels of
// its own column.  The permutations are made by the addresses that the lanes load from, as the
// load's place in LDS is fixed by the lane.
//
// In the largest tile, 256 x 256 by 8 waves of 128 x 64, a wave reads 12 KB of LDS for 32 matrix
// instructions in a half chunk: LDS is busy a quarter to a third of the cycles, the matrix units
// half of them (512 rows an expert, uneven, weights in columns) to 3 of 4 (even, in rows).  4 waves of 128 x 128 read less and are slower (512 rows an expert 1.56 ms and 1.55, the
// gradient of x 1.66 and 1.57): one wave a SIMD has nothing to run beside its own waits.
#pragma once

#include "ep_layer_internal.h"
#include "ep_rows.h"

namespace ep {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int32_t i32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

#define EP_LDS __attribute__((address_space(3)))
#define EP_INLINE __attribute__((always_inline))

// 16 x 16 outputs of 64 bytes of channels: lane l holds p = l % 16 of the first operand, q =
// l % 16 of the second, the 16 bytes of channels at 16 (l / 16) of both, and the outputs
// p = 4 (l / 16) + i of q = l % 16.  (Instructions of 32 x 32 outputs: 1.62 ms in place of 1.55 for
// 64 experts of 512 rows, 7168 to 4096 channels, at a clock 4 % lower; on zeros both run a sixth
// faster: the clock that the card holds, 1.7 to 1.8 of its 2.4 GHz here, is part of what bounds
// a product of these sizes.)
struct Bf16 {
    typedef f32x4 Acc;
    static constexpr int kBytes = 2;
    static __device__ inline Acc mma(u32x4 p, u32x4 q, Acc c) {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, p),
                                                       __builtin_bit_cast(bf16x8, q), c, 0, 0, 0);
    }
};

// Sums of 32768 products of codes stay below 2^30: nothing is rounded.
struct Int8 {
    typedef i32x4 Acc;
    static constexpr int kBytes = 1;
    static __device__ inline Acc mma(u32x4 p, u32x4 q, Acc c) {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, p),
                                                     __builtin_bit_cast(i32x4, q), c, 0, 0, 0);
    }
};

// The thread's number, as if it were new: what is worked out from it for one tile is not kept in
// registers over all of them.
__device__ inline int thread_here() {
    int t = threadIdx.x;
    asm volatile("" : "+v"(t));
    return t;
}

// A value that is worked out once and stays in a register.
__device__ inline uint32_t kept(uint32_t v) {
    asm volatile("" : "+v"(v));
    return v;
}

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
// ONCE: past the caches.
template <bool ONCE>
__device__ inline void load_lds(uint32_t to, const char *base, uint32_t off) {
    if constexpr (ONCE)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2 nt"
                     :: "s"(to), "v"(off), "s"(base) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                     :: "s"(to), "v"(off), "s"(base) : "memory", "m0");
}

__device__ inline void load_lds(uint32_t to, const char *from) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :: "s"(to), "v"(from) : "memory", "m0");
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

// What lanes load that have nothing to load: every chunk is then the same number of loads.
static __device__ const u32x4 kZeros = {0u, 0u, 0u, 0u};

// Where the rows of a token-rows call lie: the slot's token, inside the batch whatever the
// layout holds (a call captured for fewer tokens than a later layout has reads the last of
// its own).
__device__ inline int64_t token_of(const int32_t *src_meta, int64_t row, int topk, int tokens) {
    const int64_t t = src_meta[row] / topk;
    return t < 0 ? 0 : t < tokens ? t : tokens - 1;
}

// ---------------------------------------------------------------- operands
// An operand of R rows in rows of channels.  `Threads` threads bring a chunk in kLoads loads
// each: load i takes row i * Threads / 8 + thread / 8.  `row_of(r)` gives the bytes from `base` to
// row r, below 2^32 but with GATHER, where the lanes hold addresses.  ONCE: past the caches.
template <int R, int Threads, bool GATHER, bool ONCE>
struct RowsOperand {
    static constexpr int kBytes = R * 128;
    static constexpr int kLoads = kBytes / (Threads * 16) > 0 ? kBytes / (Threads * 16) : 1;
    static constexpr bool kPart = kBytes < Threads * 16;     // not every wave loads
    static_assert(kBytes % (Threads * 16) == 0 || kPart, "whole loads");
    const char *base;
    uint32_t off[GATHER ? 1 : kLoads];
    const char *from[GATHER ? kLoads : 1];
    uint32_t to;             // of the wave's first load in a stage
    bool mine;

    // The thread's 16 bytes in the chunk, the same in every load.
    static __device__ int unit(int thread) { return (thread & 7) ^ ((thread >> 3) & 7); }

    template <typename RowOf>
    __device__ void init(const void *b, RowOf row_of) {
        const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        base = uniform(b);
        const int thread = thread_here();
        to = wave * 1024;
        mine = !kPart || wave * 1024 < kBytes;
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int64_t at =
                row_of(mine ? i * (Threads / 8) + thread / 8 : 0) + unit(thread) * 16;
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
            load_lds<ONCE>(stage + to + i * Threads * 16, base, off[i]);
        }
    }
    __device__ void advance() {
        if (!GATHER) base += 128;
    }
    // Load i of a chunk of which T has `channels`; what is missing is zeros.
    template <typename T>
    __device__ void load_end(uint32_t stage, int i, int channels) {
        if (kPart && !mine) return;
        const char *at = GATHER ? from[GATHER ? i : 0] : base + off[GATHER ? 0 : i];
        const bool in = unit(thread_here()) * 16 < channels * T::kBytes;
        load_lds(stage + to + i * Threads * 16, in ? at : reinterpret_cast<const char *>(&kZeros));
    }
    // The wave's operands of N matrix instructions, i of rows 16 (first + i STEP) ..: where in a
    // stage the lane reads them, 64 bytes of channels `half` of them.
    template <int N, int STEP>
    struct Reader {
        uint32_t at[2];
        __device__ explicit Reader(int first) {
            const int lane = threadIdx.x & 63, r = 16 * first + (lane & 15);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                at[h] = kept(r * 128 + (((h * 4 + (lane >> 4)) ^ (r & 7)) << 4));
        }
        __device__ u32x4 read(uint32_t stage, int i, int half) const {
            return read_lds(stage + at[half] + i * STEP * 2048);
        }
    };
};

// An operand of C columns, channel by channel, in bf16.  CONSECUTIVE: the columns of two of a wave's
// matrix instructions are dealt out so that a lane's sums lie side by side, part l / 16 of the
// lanes having 8 of their 32, 4 in each instruction: the transposing read takes any four columns
// that lie together.
template <int C, int Threads, bool GATHER, bool CONSECUTIVE, bool ONCE>
struct ColsOperand {
    static constexpr int kRow = 2 * C;                       // bytes of a channel
    static constexpr int kBytes = 64 * kRow;
    static constexpr int kLoads = kBytes / (Threads * 16);
    static constexpr bool kPart = false, mine = true;
    static_assert(kBytes % (Threads * 16) == 0 && C >= 128, "whole loads");
    const char *base;
    int64_t pitch;           // bytes from a channel to the next
    uint32_t off[kLoads];
    const int32_t *src_meta; // GATHER: of the segment's rows
    int topk, tokens;
    uint32_t to;

    static __device__ int channel(int i, int thread) { return (i * Threads + thread) / (kRow / 16); }
    // Units of 16 bytes are permuted by these bits of the channel.  A read takes four times
    // 8 bytes of four consecutive channels in each row of 16 lanes: 32 bytes of a channel, or
    // CONSECUTIVE four pieces 16 bytes apart.
    static __device__ int swizzle(int ch) {
        return CONSECUTIVE ? (ch & 3) << 2 : ((ch & 3) | ((ch >> 1) & 4)) << 1;
    }

    // Columns `first` .. of `cols` (in a row of `pitch` bytes) from channel 0 at `b`.
    __device__ void init(const void *b, int64_t row_pitch, int first, int cols) {
        base = uniform(b);
        pitch = uniform(row_pitch);
        to = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) * 1024;
        const int thread = thread_here();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int ch = channel(i, thread);
            const int unit = (thread % (kRow / 16)) ^ swizzle(ch);
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
    __device__ void load(uint32_t stage, int i) {
        if (GATHER) load_lds(stage + to + i * Threads * 16, address(i));
        else load_lds<ONCE>(stage + to + i * Threads * 16, uniform(base), off[i]);
    }
    __device__ void advance() {
        if (GATHER) src_meta += 64;
        else base += 64 * pitch;
    }
    // Load i of a chunk of which `channels` are there; what is missing is zeros.
    template <typename T>
    __device__ void load_end(uint32_t stage, int i, int channels) {
        const char *at = reinterpret_cast<const char *>(&kZeros);
        if (channel(i, thread_here()) < channels) at = address(i);
        load_lds(stage + to + i * Threads * 16, at);
    }
    __device__ const char *address(int i) {
        const char *b = base;
        return GATHER ? b + token_of(src_meta, channel(i, thread_here()), topk, tokens) * pitch +
                            off[i]
                      : b + off[i];
    }
    // The wave's operands of N matrix instructions, i of columns 16 (first + i STEP) ... or their
    // consecutive order: where in a stage the lane reads them.  What the permutation leaves apart
    // has an address of its own, all others are constants away.
    template <int N, int STEP>
    struct Reader {
        static constexpr int kWays = CONSECUTIVE ? N / 2 : 4;
        static_assert(CONSECUTIVE ? STEP == 1 && N % 2 == 0 : STEP % 2 == 0,
                      "what the permutation does");
        uint32_t at[kWays];
        __device__ explicit Reader(int first) {
            const int lane = threadIdx.x & 63, j = lane & 15;
            const int ch = (lane >> 4) * 8 + (j >> 2);
#pragma unroll
            for (int w = 0; w < kWays; ++w) {
                // four columns, of 8 bytes
                const int piece = CONSECUTIVE ? first * 4 + (j & 3) * 2 + 8 * w
                                              : 4 * (first + w * STEP) + (j & 3);
                at[w] = kept(ch * kRow + (((piece >> 1) ^ swizzle(ch)) << 4) + (piece & 1) * 8);
            }
        }
        __device__ u32x4 read(uint32_t stage, int i, int half) const {
            const uint32_t from = stage + (CONSECUTIVE ? at[i / 2] : at[i % 4]) +
                                  (CONSECUTIVE ? i % 2 * 8 : i / 4 * (4 * STEP * 32)) +
                                  half * 32 * kRow;
            u32x4 v;
#pragma unroll
            for (int k = 0; k < 2; ++k) {                    // swizzle(ch + 4) is swizzle(ch)
                const u32x2 r = __builtin_bit_cast(
                    u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<EP_LDS s16x4 *>(
                               static_cast<uintptr_t>(from + k * 4 * kRow))));
                v[2 * k] = r.x;
                v[2 * k + 1] = r.y;
            }
            return v;
        }
    };
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
    static constexpr int TQ = BQ / 16 / WQ, TP = BP / 16 / WP;
    static constexpr int kThreads = 64 * WQ * WP;
    static constexpr int kBlocks = kThreads >= 512 ? 1 : 512 / kThreads;
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
    const int active = (rows + 16 * C::WQ - 1) / (16 * C::WQ);       // row tiles a wave
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
#pragma unroll
            for (int i = 0; i < N; ++i)
                o.template load_end<T>(stage, i, channels - chunk * kPerChunk);
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
    struct Half {
        u32x4 q[TQ], p[TP];
    };
    const typename Q::template Reader<TQ, C::WQ> from_q(wq);
    const typename P::template Reader<TP, 1> from_p(wp * TP);
    auto read = [&](Half &f, uint32_t stage_q, uint32_t stage_p, int half, int i) {
        if (i < TP) f.p[i] = from_p.read(stage_p, i, half);
        else f.q[i - TP] = from_q.read(stage_q, i - TP, half);
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
            for (int i = 0; i < TP + TQ; ++i)
                if (ALL ? i * TQ / (TP + TQ) == a
                        : i < TP ? i * kEarly / TP == a : i - TP == a)
                    read(then, stage_q, stage_p, half, i);
#pragma unroll
            for (int b = 0; b < TP; ++b) sums.v[a][b] = T::mma(now.p[b], now.q[a], sums.v[a][b]);
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
    for (int i = 0; i < TP + TQ; ++i) read(first, at_q, at_p, 0, i);
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

// A tile to be made: what its operands lie at is the source's business.
struct Job {
    int channels;            // that are summed
};

// Makes one tile after the other.  A source has
//   bool fetch(At &)               the block's next tile, if there is one (never one without channels)
//   void start_q(Q &, const At &)  sets an operand to a tile's first chunk
//   void start_p(P &, const At &)
//   bool finish(const At &, Sums &) stores a tile; whether every wave issued exactly kStores
//                                  store instructions
// with At derived from Job.  The chunks of all tiles are one stream: the next tile's first ones are
// on their way while a tile's last ones are multiplied and its sums stored.
// Otherwise as tile_product.
template <typename C, typename S>
__device__ inline void tile_stream(S &src, uint32_t lds) {
    typedef typename C::Type T;
    typedef typename S::Q Q;
    typedef typename S::P P;
    typedef typename S::At At;
    constexpr int TQ = C::TQ, TP = C::TP, kPerChunk = 128 / T::kBytes;
    constexpr int NQ = Q::kLoads, NP = P::kLoads;
    constexpr int BQ = C::SQ - 2, BP = C::SP - 2;
    static_assert(!Q::kPart && !P::kPart, "every wave loads");
    static_assert(BQ * NQ + BP * NP + S::kStores < 64, "what a wave can count");
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int wq = wave / C::WP, wp = wave % C::WP;
    const uint32_t ring_q = lds, ring_p = lds + C::kRingQ, end = lds + C::kLds;
    At now, then;
    auto fetch = [&](At &at) EP_INLINE {
        const int some = __builtin_amdgcn_readfirstlane(src.fetch(at) ? 1 : 0);
        at.channels = __builtin_amdgcn_readfirstlane(at.channels);
        return some != 0;
    };
    if (!fetch(now)) return;
    bool more = fetch(then);
    Q q;
    P p;
    src.start_q(q, now);
    src.start_p(p, now);
    // What is loaded next: so many channels are left of the tile that the operand is at, which
    // is `then` where `ahead`; `count` chunks have set out, the next goes to `room`.
    struct Loader {
        int left, count;
        bool ahead;
        uint32_t room;
    };
    Loader lq = {now.channels, 0, false, ring_q}, lp = {now.channels, 0, false, ring_p};
    // The channels of the next chunk, or 0 where there is none.
    auto next_q = [&]() EP_INLINE {
        if (lq.left <= 0 && !lq.ahead && more) {
            src.start_q(q, then);
            lq.left = then.channels;
            lq.ahead = true;
        }
        return lq.left;
    };
    auto next_p = [&]() EP_INLINE {
        if (lp.left <= 0 && !lp.ahead && more) {
            src.start_p(p, then);
            lp.left = then.channels;
            lp.ahead = true;
        }
        return lp.left;
    };
    // One of its loads (the branches are the same in all lanes).
    auto load_q = [&](int left, int i) EP_INLINE {
        if (left >= kPerChunk) q.load(lq.room, i);
        else if (left > 0) q.template load_end<T>(lq.room, i, left);
    };
    auto load_p = [&](int left, int i) EP_INLINE {
        if (left >= kPerChunk) p.load(lp.room, i);
        else if (left > 0) p.template load_end<T>(lp.room, i, left);
    };
    // After its last load.
    auto loaded_q = [&](int left) EP_INLINE {
        if (left <= 0) return;
        q.advance();
        lq.left -= kPerChunk;
        ++lq.count;
        lq.room = lq.room + C::kStageQ == ring_p ? ring_q : lq.room + C::kStageQ;
    };
    auto loaded_p = [&](int left) EP_INLINE {
        if (left <= 0) return;
        p.advance();
        lp.left -= kPerChunk;
        ++lp.count;
        lp.room = lp.room + C::kStageP == end ? ring_p : lp.room + C::kStageP;
    };
    // Chunks until so many have set out.
    auto fill_q = [&](int count) EP_INLINE {
#pragma clang loop unroll(disable)
        while (lq.count < count) {
            const int left = next_q();
            if (left <= 0) break;
#pragma unroll
            for (int i = 0; i < NQ; ++i) load_q(left, i);
            loaded_q(left);
        }
    };
    auto fill_p = [&](int count) EP_INLINE {
#pragma clang loop unroll(disable)
        while (lp.count < count) {
            const int left = next_p();
            if (left <= 0) break;
#pragma unroll
            for (int i = 0; i < NP; ++i) load_p(left, i);
            loaded_p(left);
        }
    };
    struct Half {
        u32x4 q[TQ], p[TP];
    };
    const typename Q::template Reader<TQ, C::WQ> from_q(wq);
    const typename P::template Reader<TP, 1> from_p(wp * TP);
    auto read = [&](Half &f, uint32_t stage_q, uint32_t stage_p, int half, int i) EP_INLINE {
        if (i < TP) f.p[i] = from_p.read(stage_p, i, half);
        else f.q[i - TP] = from_q.read(stage_q, i - TP, half);
    };
    typename C::Sums sums;
    // Multiplies `f`, a row tile at a time, while `b` is read and the N loads of a chunk set out.
    auto step = [&](const Half &f, Half &b, uint32_t stage_q, uint32_t stage_p, int half, auto count,
                    auto load) EP_INLINE {
        constexpr int N = decltype(count)::value;
        constexpr int kEarly = (TQ + 1) / 2;                 // row tiles in which loads set out
#pragma unroll
        for (int t = 0; t < TQ; ++t) {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (i * kEarly / N == t) load(i);
#pragma unroll
            for (int i = 0; i < TP + TQ; ++i)
                if (i * TQ / (TP + TQ) == t) read(b, stage_q, stage_p, half, i);
#pragma unroll
            for (int u = 0; u < TP; ++u) sums.v[t][u] = T::mma(f.p[u], f.q[t], sums.v[t][u]);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    fill_p(C::SP);
    fill_q(C::SQ);
    wait_loads<0>();
    block_barrier();
    uint32_t at_q = ring_q, at_p = ring_p;
    Half first, second;
#pragma unroll
    for (int i = 0; i < TP + TQ; ++i) read(first, at_q, at_p, 0, i);
    int g = 0;                                   // chunks before this one
    int stores = 0;
    for (;;) {
#pragma unroll
        for (int t = 0; t < TQ; ++t)
#pragma unroll
            for (int u = 0; u < TP; ++u) {
                sums.v[t][u] = typename C::Acc(0);
                asm("" : "+v"(sums.v[t][u]));    // zeros like others: no first chunk of its own
            }
        const int last = g + (now.channels + kPerChunk - 1) / kPerChunk;
#pragma clang loop unroll(disable)
        for (; g < last; ++g) {
            // the first chunk's were loaded above
            const int left_p = lp.count < g + C::SP ? next_p() : 0;
            step(first, second, at_q, at_p, 1, Int<NP>(), [&](int i) EP_INLINE { load_p(left_p, i); });
            loaded_p(left_p);
            // chunk g + 1 has come: BQ chunks of Q and BP of P (none where the tiles ahead have no
            // more) may still be on their way, and what was stored since
            const bool known = lq.count == g + C::SQ && stores >= 0;
            const bool all = known && lp.count == g + C::SP, next = known && lp.count == g + 2;
            if (all && stores > 0) wait_loads<BQ * NQ + BP * NP + S::kStores>();
            else if (all) wait_loads<BQ * NQ + BP * NP>();
            else if (next && stores > 0) wait_loads<BQ * NQ + S::kStores>();
            else wait_loads<0>();
            stores = 0;
            block_barrier();
            at_q = at_q + C::kStageQ == ring_p ? ring_q : at_q + C::kStageQ;
            at_p = at_p + C::kStageP == end ? ring_p : at_p + C::kStageP;
            // behind the last chunk nothing has come: what is read is not used
            const int left_q = next_q();
            step(second, first, at_q, at_p, 0, Int<NQ>(), [&](int i) EP_INLINE { load_q(left_q, i); });
            loaded_q(left_q);
        }
        // Tiles of few chunks: what the loaders could not see before sets out ahead of the stores,
        // which loads behind them would wait for (all gradients of the block, 64 experts of 16 rows,
        // 7168 and 2048 channels: 2212 -> 2146 us; of 512 rows 6266 -> 6236).
        const At done = now;
        const bool end = !more;
        if (!end) {
            now = then;                          // both operands have begun with it
            lq.ahead = lp.ahead = false;
            more = fetch(then);
            fill_q(g + C::SQ);
            fill_p(g + C::SP - 1);
        }
        stores = src.finish(done, sums) ? S::kStores : -1;
        if (end) return;
    }
}

}  // namespace ep
