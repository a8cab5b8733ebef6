// linattn_mma.cu -- linear attention with decay in chunks of 64 tokens on the
// tensor cores (bf16 inputs, head sizes 64 and 128).
//
// With S the state before a chunk of m <= 64 tokens and i, j in the chunk:
//   o_i = scale ( sum_{j<=i} g^(i-j) (q_i . k_j) v_j  +  g^(i+1) S^T q_i )
//   S  <- g^m S + sum_j g^(m-1-j) k_j v_j^T
// (a reversed call: g^i in place of g^(i+1), g^(m-j) of g^(m-1-j), see
// linattn.cuh). Everything is held transposed, M = dv = the 128 TMEM lanes:
//   P    = Q K^T                    64 x 64 scores, weighted, bf16
//   O^T  = S^T Q^T, aged, + V^T P^T in one accumulator (R)
//   S^T += (w V)^T K                the float32 state, which stays in TMEM
// so that S^T, read out once a chunk, goes back to TMEM as the bf16 A operand
// of its product with Q^T without passing shared memory, and 256 columns (128
// S; 64 bf16 S, then the scores; 64 R) let two blocks share an SM: while one
// waits for its chain of products the other works.
//
// Precision. Scores and the state are rounded to bf16 (once each) where they
// enter a product whose result is rounded to bf16 anyway. The state itself is
// float32 and may be an output: w V is split into bf16 parts whose products
// are exact in the float32 accumulation. Two parts keep 2^-17 of a term, three
// 2^-25; the third is spent where the final state is asked for and the term
// will still weigh more than 2^-8 in it (states of 2 to 300 tokens: 2.4e-6
// relative with two parts, 0.05e-6 to 1.1e-6 with three). The accumulation
// itself cuts off low bits instead of rounding them: measured, 2e-8 to 4e-8 of
// the state for each of these products, over the tokens that the decay
// remembers in a window.
//
// What bounds it. Measured at 16384 tokens, 32 heads of 128 in 16 sequences:
// 134 us, 4.2 TB/s of the tensors' bytes, 0.62 of the copy bandwidth; issue
// slots half busy, the tensor pipe 0.29. Shared memory and TMEM accesses
// pass one 128-byte-a-cycle path: a chunk needs about 1700 cycles of it for
// TMEM (S read 512, its bf16 form 256, R 512, scores 128, and S written back
// 512 when a frame ends) and 1900 for shared memory (tiles in 384, w V 384,
// the products' operands 1100), against 2700 that its 64 KB take from HBM at
// an SM's share. The rest is the chain of a chunk's steps at two blocks an
// SM. What cost time: registers spilled in the chunk loop (154 us with 60
// bytes spilled, 133 with 4; now none at head size 128 and 8 bytes at 64),
// branches around single elements (each serialises its load), eight working
// warps (193 us against 166 at the time), masking each score by a selection
// (8 us, against none for the sum of zeros that finds rows which need it).
// Loading the next tiles earlier made no difference.
//
// Seventeen warps: sixteen do the elementwise work (on TMEM, four to a
// quarter of the lanes, a quarter of the columns each); the last issues
// copies and products, each as soon as its operands are there and its target
// is free. A chunk's chain is S^T Q^T, Q K^T, weights, V^T P^T; beside the
// first two run the outputs of the chunk before and w V, beside the last the
// state's pass for the next chunk; the update runs beside the weights.
//
// A chunk of fewer than 64 tokens keeps its first row at row 0, in a reversed
// call its last row at row 63: the weights then depend on the row alone.
//
// Head size 64: the A operands repeat their 64 rows (a zero stride between
// the halves of M), lanes 64..127 hold copies.
#include <algorithm>
#include <atomic>
#include <cstddef>
#include <mutex>
#include <cudaTypedefs.h>

#include "ak_tcgen05.cuh"
#include "linattn.cuh"

namespace ak {
namespace la {

constexpr int kChunk = 64;

struct Maps {
    CUtensorMap q, k, v;
    int q_h, k_h, v_h;  // 0: one head shared by all
};
struct ChunkBatch {
    Maps maps[kMaxCalls];
    Batch b;
    uint64_t* error_word;
    uint64_t epoch;
    uint64_t wait_limit_ns;
};

// A wait here is for this block's own copies and products: microseconds, or as
// long as the device is taken away from the block. A shorter limit than this
// would end sound calls.
constexpr uint64_t kLeastWait = 100'000'000;

constexpr int kFrame = 16;  // chunks of a frame at most

// Barriers and tables of a block.
struct Small {
    // arrivals: copies of q and k, of v (a stage each), products (of
    // the state, the scores, of the values, the update), working warps (state
    // operand ready and accumulator read, w V ready, scores ready)
    uint64_t qk[2], v[2], inter, scores, values, update, state, wv, ready;
    uint64_t drained;  // everything issued before a wait ran out
    int64_t count;
    uint32_t tmem;
    int failed, w, t0, t1;  // w: window or sequence of the block, t0, t1: its span
    // weights: of row j in the update after a whole chunk; and, which a fold
    // pass does not have, of the state before the chunk at row i, and of the
    // score of rows i and j at kChunk + i - j
    float wrow[kChunk];
    alignas(16) float age[kChunk];
    float score[2 * kChunk];
    float up[kFrame], down[kFrame];  // g^64u, and g^-64(u+1) or 1 (see `frame`)
    int len[kRanked];
    // by the chunk's parity and column: where the first value that is not
    // finite stands (see `spoil`)
    int bad[2 * 128];
};

template <int D, int PARTS, bool FOLD>
struct Plan {
    static constexpr int kWork = 512;        // threads of the working warps
    static constexpr int kThreads = kWork + 32;
    static constexpr int kSplit = kWork / 128;             // working warps of a quarter of the lanes
    static constexpr int kCols = kChunk / kSplit;          // accumulator columns of a thread
    static constexpr int kStages = FOLD ? 2 : 1;           // of the key and value tiles
    // shared memory: the tiles, then Small
    static constexpr int kTileBytes = kChunk * D * 2;
    static constexpr int kQ = 0;
    static constexpr int kK = FOLD ? 0 : kTileBytes;
    static constexpr int kV = kK + kStages * kTileBytes;
    static constexpr int kP = kV + kStages * kTileBytes;
    static constexpr int kW = kP + (FOLD ? 0 : kChunk * kChunk * 2);
    static constexpr int kSmall = kW + PARTS * kTileBytes;
    static constexpr int kUsed = kSmall + (int)(FOLD ? offsetof(Small, age) : sizeof(Small));
    // two blocks of the main pass share an SM's TMEM: a third would only wait for it
    static constexpr int kSmem = kUsed < 80 * 1024 && !FOLD ? 80 * 1024 : kUsed;
    // columns: S, its bf16 form, accumulator, scores (over the bf16 form at D = 128)
    static constexpr uint32_t kS = 0, kB = D, kR = D + D / 2, kX = D == 128 ? kB : kR + 64;
    static constexpr uint32_t kTmem = FOLD ? D : 256;
};

// What a block walks: the chunks of the sequence pieces in its window.
struct Chunk {
    int n;        // sequence
    int at, end;  // first token; end of the piece (a call has less than 2^31)
    int stop;     // end of the sequence
    int m;        // tokens of the chunk
    bool first;   // of the piece
    bool valid;
};

// Two float32 operations an instruction.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t pair_of(uint32_t a, uint32_t b) { return pair(__uint_as_float(a), __uint_as_float(b)); }
// Two values rounded to bf16, the first in the low half.
__device__ __forceinline__ uint32_t bf16x2_of(uint64_t x) {
    const float2 f = unpair(x);
    const __nv_bfloat162 y = __floats2bfloat162_rn(f.x, f.y);
    uint32_t r;
    memcpy(&r, &y, 4);
    return r;
}
__device__ __forceinline__ uint64_t pair_of_bf16x2(uint32_t x) { return pair_of(x << 16, x & 0xffff0000u); }

// Adds up zeros, or NaN where a value is a NaN or infinite: x times zero.
__device__ __forceinline__ void add_zeros(uint32_t& sum, uint32_t x) {
    asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum) : "r"(x), "r"(0u));
}

// V^T P^T multiplies a value also by the zero weights of the tokens before it.
// Values that are not finite are therefore taken out of the tile (w V, and with
// it the state, has them), and `poison` makes the outputs of their column NaN
// from their token on. `bad` holds the chunk's end less their place in it,
// which lies above the chunk's first token: what earlier chunks left there
// never does, and of one chunk's places the first is the largest. A thread
// looks through `pieces` pieces of its own, `step` rows apart.
__device__ __noinline__ void spoil(unsigned char* at, int pieces, int step, int* bad, int end, int sign) {
#pragma unroll 1
    for (int i = 0; i < pieces; ++i, at += step * 128, end -= sign * step) {
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
            unsigned short* const x = reinterpret_cast<unsigned short*>(at) + e;
            if ((*x & 0x7f80) != 0x7f80) continue;
            atomicMax(&bad[e], end);
            *x = 0;
        }
    }
}
// The same of a row of scores, `n` of them from column j0 on: those of later
// tokens have a zero weight, and become zero.
__device__ __noinline__ void mask_scores(unsigned char* p, int row, int j0, int n, bool rev) {
#pragma unroll 1
    for (int j = j0; j < j0 + n; ++j)
        if (rev ? j < row : j > row) *reinterpret_cast<unsigned short*>(p + swz128(row, j / 8) + j % 8 * 2) = 0;
}
__device__ __noinline__ void poison(bf16* out, int64_t tok, int first, int last) {
    for (int i = first; i < last; ++i) *reinterpret_cast<unsigned short*>(out + i * tok) = 0x7fc0;
}

// A wait that the first poll did not end: until the limit, after which the
// block records that it gave up, and none of its waits waits any longer.
__device__ __noinline__ void wait_long(uint64_t* bar, uint32_t phase, int* failed, const ChunkBatch& batch) {
    if (*(volatile int*)failed) return;
    if (!mbar_wait(bar, phase, globaltimer_ns() + batch.wait_limit_ns)) {
        *(volatile int*)failed = 1;
        if (batch.error_word) *(volatile uint64_t*)batch.error_word = batch.epoch;
    }
}

template <int D, int PARTS, bool FOLD>
__global__ void __launch_bounds__(Plan<D, PARTS, FOLD>::kThreads, 2) k_chunks(const __grid_constant__ ChunkBatch batch) {
    using P = Plan<D, PARTS, FOLD>;
    constexpr int kWork = P::kWork, kMmaThreads = P::kThreads, kSplit = P::kSplit, kCols = P::kCols;
    extern __shared__ __align__(1024) unsigned char sm[];
    Small& t = *reinterpret_cast<Small*>(sm + P::kSmall);
    const Args& a = batch.b.a[blockIdx.z];
    const Maps& maps = batch.maps[blockIdx.z];
    const uint32_t sbase = smem_addr(sm);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, threadIdx.x / kWarp, 0), lane = tid % kWarp;
    const int h = blockIdx.x;
    if (tid == 0) t.w = blockIdx.y;
    if (!FOLD && a.ranked) {
        // block w takes the w-th longest sequence: the long ones start first
        for (int i = tid; i < a.seqs; i += kMmaThreads) t.len[i] = (int)(offset_at(a, i + 1) - offset_at(a, i));
        __syncthreads();
        for (int i = tid; i < a.seqs; i += kMmaThreads) {
            const int mine = t.len[i];
            int rank = 0;
            for (int j = 0; j < a.seqs; ++j) rank += t.len[j] > mine || (t.len[j] == mine && j < i);
            if (rank == blockIdx.y) t.w = i;
        }
    }
    __syncthreads();
    if (tid == 0) {
        int64_t from, to;
        block_span(a, t.w, &from, &to);
        t.t0 = (int)from, t.t1 = (int)to;
    }
    const float ld = a.log_decay[h];
    const bool rev = a.reverse;
    // The state's frame. S is held divided by the decay since the frame
    // began, `frame` chunks at most, so that a chunk reads it for its bf16
    // form but writes it back only when a frame ends: TMEM traffic, at the
    // 128 bytes a cycle that shared memory has too, is what these warps
    // spend most on, and the write was a fifth of it. A chunk's terms enter
    // divided by the decay up to its end. e^30 bounds that; a head that
    // decays faster scales its state in every chunk before it adds terms.
    const float per_chunk = fabsf(ld) * kChunk;
    const int frame = per_chunk <= 30.0f ? (per_chunk * kFrame <= 30.0f ? kFrame : (int)(30.0f / per_chunk)) : 0;

    if (warp == kWork / kWarp) {
        tmem_alloc(&t.tmem, P::kTmem);
        if (lane == 0) {
            for (int i = 0; i < P::kStages; ++i) {
                mbar_init(&t.qk[i], 1);
                mbar_init(&t.v[i], 1);
            }
            mbar_init(&t.inter, 1);
            mbar_init(&t.scores, 1);
            mbar_init(&t.values, 1);
            mbar_init(&t.update, 1);
            mbar_init(&t.state, kWork / kWarp);
            mbar_init(&t.wv, kWork / kWarp);
            mbar_init(&t.ready, kWork / kWarp);
            mbar_init(&t.drained, 1);
            fence_barrier_init();
            t.failed = 0;
            tma_prefetch_map(&maps.k);
            tma_prefetch_map(&maps.v);
            if (!FOLD) tma_prefetch_map(&maps.q);
        }
    }
    if (!FOLD && tid < 2 * kChunk) {
        const int gap = rev ? kChunk - tid : tid - kChunk;
        t.score[tid] = gap < 0 ? 0.0f : decay_pow(ld, gap) * a.in_scale * a.out_scale;
    }
    if (!FOLD && tid >= 2 * kChunk && tid < 2 * kChunk + kFrame) {
        const int u = tid - 2 * kChunk;
        t.up[u] = decay_pow(ld, u * kChunk);
        t.down[u] = frame == 0 ? 1.0f : decay_pow(ld, -(u + 1) * kChunk);
    }
    if (!FOLD && tid < 2 * 128) t.bad[tid] = 0;
    if (tid < kChunk) {
        if (!FOLD) t.age[tid] = decay_pow(ld, rev ? kChunk - 1 - tid : tid + 1) * a.out_scale;
        t.wrow[tid] = decay_pow(ld, rev ? tid + 1 : kChunk - 1 - tid) * a.in_scale;
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, t.tmem, 0);
    // Only now: the main pass's blocks take TMEM before they wait for this
    // pass, which must not wait for theirs.
    if (FOLD) griddep_launch_dependents();

    // Bounded waits: a warp that gives up records it; all skip their further
    // waits and leave by the ordinary way, the issuing warp before it asks for
    // another chunk.
    auto wait_at = [&](uint64_t* bar, uint32_t phase) {
        if (!mbar_try_wait(bar, phase)) wait_long(bar, phase, &t.failed, batch);
        __syncwarp();  // whole warps go on to the tensor-memory instructions
    };
    auto wait = [&](uint64_t* bar, uint32_t& phase) {
        wait_at(bar, phase);
        phase ^= 1;
    };
    // A working warp is done with a step: its shared-memory and tensor-memory
    // accesses come before what the issuing warp does next.
    auto arrive = [&](uint64_t* bar) {
        fence_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };

    const int64_t ssize = (int64_t)D * D;
    auto addr = [&](int t) { return rev ? (int)a.tokens - 1 - t : t; };
    auto offset = [&](int n) { return (int)offset_at(a, n); };
    auto seq_state = [&](int n) { return ((rev ? a.seqs - 1 - n : n) * a.heads + h) * ssize; };
    // natural token of row 0 (before the array's start for a short reversed chunk)
    auto low = [&](const Chunk& c) { return rev ? (int)a.tokens - c.at - kChunk : c.at; };
    const bool writer = tid < kWork;

    // tokens of no sequence get zeros
    auto blank = [&](int from, int to) {
        if (!FOLD && writer)
            for (int x = from + tid / D; x < to; x += kWork / D) static_cast<bf16*>(a.o)[h * a.o_head + (int64_t)addr(x) * a.o_tok + tid % D] = __float2bfloat16_rn(0.0f);
    };
    auto start = [&](int n, int begin, int end) {
        Chunk c;
        c.n = n;
        c.at = begin > t.t0 ? begin : t.t0;
        c.end = end < t.t1 ? end : t.t1;
        c.stop = end;
        c.m = c.end - c.at < kChunk ? c.end - c.at : kChunk;
        c.first = true;
        c.valid = true;
        return c;
    };
    // the first chunk of sequence n or a later one; pieces without tokens are
    // settled on the way
    auto seek = [&](int n, int covered) {  // covered: outputs are settled up to there
        Chunk c = {};
        for (; n < a.seqs; ++n) {
            const int begin = offset(n), end = offset(n + 1);
            if (a.by_seq ? n > t.w : begin >= t.t1 && t.w != a.windows - 1) break;
            if (begin > covered) {
                blank(covered, begin < t.t1 ? begin : t.t1);
                covered = begin;
            }
            c = start(n, begin, end);
            if (c.at < c.end) return c;
            if (writer && a.s_out && begin >= t.t0) {  // an empty sequence passes its state on
                for (int i = tid; i < D * D; i += kWork)
                    a.s_out[seq_state(n) + i] = !a.s_in ? 0.0f
                                                : a.s_in[seq_state(n) + (a.s_in_t ? (i % D) * D + i / D : i)];
            }
        }
        c.valid = false;
        if (covered < t.t1) blank(covered, t.t1);
        return c;
    };
    auto next = [&](const Chunk& c) {
        Chunk x = c;
        x.at += c.m;
        x.first = false;
        if (x.at < c.end) {
            x.m = c.end - x.at < kChunk ? c.end - x.at : kChunk;
            return x;
        }
        // at the window's end only empty sequences at the axis' end are left
        if (!FOLD && (c.end < t.t1 || t.w == a.windows - 1)) return seek(c.n + 1, c.end);
        x.valid = false;
        return x;
    };

    int n = (int)first_sequence<kMmaThreads>(a, t.w, t.t0, &t.count);
    if (!FOLD) griddep_wait();  // the carries; and nothing is written before
    Chunk c = {};
    int32_t kind = kNone;
    if (FOLD) {
        while (n < a.seqs && offset(n + 1) <= t.t1) ++n;
        const int begin = n < a.seqs ? offset(n) : t.t1;
        kind = begin >= t.t1 ? kNone : (begin >= t.t0 ? kFresh : kThrough);
        if (tid == 0 && h == 0) a.tail[t.w] = kind;
        if (kind != kNone) c = start(n, begin, offset(n + 1));
    } else {
        c = seek(n, t.t0);
    }
    // parts of w V that a chunk's terms need
    auto parts_of = [&](const Chunk& c) {
        return PARTS == 3 && ld * (float)(c.stop - c.at - c.m) > -5.55f ? 3 : 2;
    };
    // where the state before a piece comes from; null: zero
    auto source = [&](const Chunk& c, bool* transposed) -> const float* {
        *transposed = false;
        const bool here = FOLD ? kind == kFresh : offset(c.n) >= t.t0;
        if (!here) {
            *transposed = a.carry_t;
            return FOLD ? nullptr : a.carry + ((int64_t)t.w * a.heads + h) * ssize;
        }
        if (!a.s_in) return nullptr;
        // another block may already have written this sequence's result in place
        if (!FOLD && a.stash && c.end < c.stop) return a.stash + ((int64_t)t.w * a.heads + h) * ssize;
        *transposed = a.s_in_t;
        return a.s_in + seq_state(c.n);
    };

    if (warp == kWork / kWarp) {
        // ------------------------------------------------------------------
        // copies and products
        // ------------------------------------------------------------------
        const uint32_t leader = lane == 0;
        uint32_t stage = 0, phase = 0, state = 0, inter = 0, wv = 0, ready = 0, values = 0, update = 0;
        const uint64_t dq = smem_desc(sbase + P::kQ, 16), dp = smem_desc(sbase + P::kP, 16);
        const uint64_t dkk = smem_desc(sbase + P::kK, 16), dk = smem_desc(sbase + P::kK, 8192);
        const uint64_t dv = smem_desc(sbase + P::kV, D == 128 ? 8192 : 0);
        const uint64_t dw = smem_desc(sbase + P::kW, D == 128 ? 8192 : 0);
        // A wait ran out: no barrier is used for another copy then, whose last
        // one may still be under way. Asked once a chunk.
        auto lost = [&] { return __shfl_sync(0xffffffffu, *(volatile int*)&t.failed, 0) != 0; };
        auto load = [&](const Chunk& c, uint64_t* bar, uint32_t expect, const CUtensorMap* map, int head, int at) {
            if (leader) {
                if (expect) mbar_arrive_expect_tx(bar, expect);
#pragma unroll
                for (int b = 0; b < D / 64; ++b) tma_load_3d(sm + at + b * 8192, map, b * 64, h * head, low(c), bar);
            }
            __syncwarp();
        };
        // q announces its own bytes and those of k, which comes later
        auto load_q = [&](const Chunk& c) { load(c, &t.qk[0], 2 * P::kTileBytes, &maps.q, maps.q_h, P::kQ); };
        auto load_k = [&](const Chunk& c, int st) {
            load(c, &t.qk[st], FOLD ? P::kTileBytes : 0, &maps.k, maps.k_h, P::kK + st * P::kTileBytes);
        };
        auto load_v = [&](const Chunk& c, int st) {
            load(c, &t.v[st], P::kTileBytes, &maps.v, maps.v_h, P::kV + st * P::kTileBytes);
        };
        if (c.valid) {
            load_v(c, 0);
            if (!FOLD) load_q(c);
            load_k(c, 0);
        }
        bool zero = true;
        while (c.valid) {
            if (c.first) {
                bool tr;
                zero = source(c, &tr) == nullptr;
            }
            if (!FOLD) wait(&t.state, state);
            wait_at(&t.qk[stage], phase);
            if (!FOLD) {
                tc_fence_after();
                if (!zero) {
                    // S^T Q^T
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        mma_ts(tmem + P::kR, tmem + P::kB + s * 8, dq + (((s / 4) * 8192 + (s % 4) * 32) >> 4),
                               mma_idesc(128, 64, false, false), s > 0, leader);
                    mma_commit(&t.inter, leader);
                    if (P::kX == P::kB) wait(&t.inter, inter);  // its operand's columns are free
                }
                // Q K^T; rows 64..127 of M read on into the next tile and are not used
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint64_t off = ((s / 4) * 8192 + (s % 4) * 32) >> 4;
                    mma_ss(tmem + P::kX, dq + off, dkk + off, mma_idesc(128, 64, false, false), s > 0, leader);
                }
                mma_commit(&t.scores, leader);
            }
            const int parts = parts_of(c);
            const Chunk c2 = next(c);
            if (FOLD && lost()) break;
            if (FOLD && c2.valid) {  // the other stage was used up with the update before
                load_v(c2, stage ^ 1);
                load_k(c2, stage ^ 1);
            }
            wait_at(&t.v[stage], phase);
            wait(&t.wv, wv);
            tc_fence_after();
            // S^T += (w V)^T K
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                if (p < 2 || parts == 3)
#pragma unroll
                    for (int s = 0; s < kChunk / 16; ++s)
                        mma_ss(tmem + P::kS, dw + ((p * P::kTileBytes + s * 2048) >> 4), dk + ((stage * P::kTileBytes + s * 2048) >> 4),
                               mma_idesc(128, D, true, true), !zero || p > 0 || s > 0, leader);
            mma_commit(&t.update, leader);
            if (!FOLD) {
                wait(&t.ready, ready);
                tc_fence_after();
                // V^T P^T
#pragma unroll
                for (int s = 0; s < kChunk / 16; ++s)
                    mma_ss(tmem + P::kR, dv + (s * 2048 >> 4), dp + (s * 32 >> 4), mma_idesc(128, 64, true, false), !zero || s > 0, leader);
                mma_commit(&t.values, leader);
            }
            // the next chunk's tiles, each as soon as its buffer has been used
            if (!FOLD && lost()) break;
            if (!FOLD && c2.valid) load_q(c2);
            wait(&t.update, update);
            if (!FOLD) {
                if (c2.valid) load_k(c2, 0);
                wait(&t.values, values);
                if (c2.valid) load_v(c2, 0);
            }
            if (P::kStages == 2) stage ^= 1;
            if (stage == 0) phase ^= 1;
            zero = false;
            c = c2;
        }
        if (lost()) {
            // What is in flight ends (or runs into the limit once more) before
            // the block gives up the memory that it writes to: products, and
            // the copies of the chunk that was left.
            const uint64_t until = globaltimer_ns() + batch.wait_limit_ns;
            mma_commit(&t.drained, leader);
            mbar_wait(&t.drained, 0, until);
            if (c.valid) {
                mbar_wait(&t.v[stage], phase, until);
                mbar_wait(&t.qk[stage], phase, until);
            }
        }
        __syncwarp();
    } else {
        // ------------------------------------------------------------------
        // elementwise work
        // ------------------------------------------------------------------
        const int row = (warp % 4) * 32 + lane;  // TMEM lane
        const int part = warp / 4;               // which quarter of the columns
        const int dv = row % D;                  // state column (copies at D = 64)
        const uint32_t lanes = tmem + ((uint32_t)((warp % 4) * 32) << 16);
        uint32_t stage = 0, phase = 0;  // phase: of the stage; without stages, of every barrier of a chunk
        uint32_t update = 0;
        // S before a piece; false where it is zero
        auto load_state = [&](const Chunk& c) {
            bool tr;
            const float* src = source(c, &tr);
            if (!src) return false;
            // a fold ages its state once, not chunk by chunk
            const float age = FOLD ? decay_pow(ld, t.t1 - c.at) : 1.0f;
#pragma unroll 1
            for (int k0 = part * (D / kSplit); k0 < (part + 1) * (D / kSplit); k0 += 16) {
                uint32_t r[16];
                const float* p = tr ? src + dv * D + k0 : src + k0 * D + dv;
#pragma unroll
                for (int i = 0; i < 16; ++i, p += tr ? 1 : D) r[i] = __float_as_uint(*p);
                if (FOLD && a.stash && row < D) {
                    float* keep = a.stash + ((int64_t)t.w * a.heads + h) * ssize + k0 * D + dv;
#pragma unroll
                    for (int i = 0; i < 16; ++i) keep[i * D] = __uint_as_float(r[i]);
                }
                if (FOLD)
#pragma unroll
                    for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * age);
                tmem_st(lanes + P::kS + k0, r);
            }
            tmem_wait_st();
            return true;
        };
        auto store_state = [&](float* dst, float factor) {
            if (row < D) {
#pragma unroll 1
                for (int k0 = part * (D / kSplit); k0 < (part + 1) * (D / kSplit); k0 += 16) {
                    uint32_t r[16];
                    tmem_ld(r, lanes + P::kS + k0);
                    tmem_wait_ld(r);
                    float* to = dst + k0 * D + dv;
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[i * D] = __uint_as_float(r[i]) * factor;
                }
            }
            __syncwarp();
        };
        int in_frame = 0;  // chunks since the frame began
        // S^T as a bf16 operand before a chunk of m tokens
        auto pass_state = [&](int m) {
            constexpr int N = D / kSplit < kCols ? D / kSplit : kCols;
            if (frame > 0 && in_frame < frame) {
                const float w = t.up[in_frame];
                const uint64_t ww = pair(w, w);
#pragma unroll 1
                for (int k0 = part * (D / kSplit); k0 < (part + 1) * (D / kSplit); k0 += N) {
                    uint32_t r[N], p[N / 2];
                    tmem_ld(r, lanes + P::kS + k0);
                    tmem_wait_ld(r);
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) p[i] = bf16x2_of(mul2(pair_of(r[2 * i], r[2 * i + 1]), ww));
                    tmem_st(lanes + P::kB + k0 / 2, p);
                }
            } else {
                // a fast head takes its operand before, a frame's end after scaling
                in_frame = 0;
                const Factor f = decay_factor(ld, frame == 0 ? m : frame * kChunk);
                const uint64_t lo = pair(f.lo, f.lo), hi = pair(f.hi, f.hi);
#pragma unroll 1
                for (int k0 = part * (D / kSplit); k0 < (part + 1) * (D / kSplit); k0 += N) {
                    uint32_t r[N], p[N / 2];
                    tmem_ld(r, lanes + P::kS + k0);
                    tmem_wait_ld(r);
#pragma unroll
                    for (int i = 0; i < N / 2; ++i) {
                        const uint64_t x = pair_of(r[2 * i], r[2 * i + 1]), y = fma2(x, hi, mul2(x, lo));
                        p[i] = bf16x2_of(frame == 0 ? x : y);
                        const float2 z = unpair(y);
                        r[2 * i] = __float_as_uint(z.x), r[2 * i + 1] = __float_as_uint(z.y);
                    }
                    tmem_st(lanes + P::kB + k0 / 2, p);
                    tmem_st(lanes + P::kS + k0, r);
                }
            }
            tmem_wait_st();
        };
        // w V in bf16 parts: 16-byte pieces, a thread's all in one column of
        // pieces and in rows of equal swizzle
        constexpr int kRowStep = kWork / (D / 8);
        const int v_row = tid / (D / 8);
        unsigned char* const v_at = sm + P::kV + (tid % (D / 8) / 8) * 8192 + swz128(v_row, tid % 8);
        auto split_values = [&](const Chunk& c, auto whole_chunk, auto three) {
            constexpr bool kFull = decltype(whole_chunk)::value, kThree = decltype(three)::value;
            const int r0 = rev ? kChunk - c.m : 0, shift = rev ? -r0 : kChunk - c.m;
            // what the terms are divided by, or have left to the fold's end
            const float age = FOLD                    ? decay_pow(ld, t.t1 - c.at - c.m)
                              : kFull || frame == 0 ? t.down[in_frame]
                                                    : decay_pow(ld, -(in_frame * kChunk + c.m));
            uint32_t zeros = 0;
#pragma unroll
            for (int i = 0; i < kChunk / kRowStep; ++i) {
                const int r = v_row + i * kRowStep;
                uint4 in = *reinterpret_cast<const uint4*>(v_at + stage * P::kTileBytes + i * kRowStep * 128);
                float w = t.wrow[kFull ? r : (r + shift) & (kChunk - 1)];
                if (!kFull && (unsigned)(r - r0) >= (unsigned)c.m) in = make_uint4(0, 0, 0, 0);
                w *= age;
                const uint64_t ww = pair(w, w), minus = pair(-1.0f, -1.0f);
                uint32_t* const x = &in.x;
                uint32_t y[2][4], z[4];
                if (!FOLD)
#pragma unroll
                    for (int e = 0; e < 4; ++e) add_zeros(zeros, x[e]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    uint64_t wv = mul2(pair_of_bf16x2(x[e]), ww);
                    y[0][e] = bf16x2_of(wv);
                    wv = fma2(pair_of_bf16x2(y[0][e]), minus, wv);  // what the part leaves, exactly
                    y[1][e] = bf16x2_of(wv);
                    if (kThree) z[e] = bf16x2_of(fma2(pair_of_bf16x2(y[1][e]), minus, wv));
                }
                unsigned char* const to = v_at + (P::kW - P::kV) + i * kRowStep * 128;
                *reinterpret_cast<uint4*>(to) = make_uint4(y[0][0], y[0][1], y[0][2], y[0][3]);
                *reinterpret_cast<uint4*>(to + P::kTileBytes) = make_uint4(y[1][0], y[1][1], y[1][2], y[1][3]);
                if (kThree) *reinterpret_cast<uint4*>(to + 2 * P::kTileBytes) = make_uint4(z[0], z[1], z[2], z[3]);
            }
            if (!FOLD && (zeros & 0x7fff7fffu))
                spoil(v_at, kChunk / kRowStep, kRowStep, t.bad + phase * 128 + tid % (D / 8) * 8,
                      c.at + c.m - (rev ? kChunk - 1 - v_row : v_row), rev ? -1 : 1);
        };
        using Yes = std::true_type;
        using No = std::false_type;
        const float* const score_at = t.score + kChunk + row - part * kCols;
        // a warp's quarter of the scores' columns may lie after all of its rows
        const bool masked = rev ? (part + 1) * kCols <= row - lane : part * kCols > row - lane + 31;
        const bool scored = row < kChunk && !masked;
        if (!FOLD && row < kChunk && masked)
#pragma unroll
            for (int y = 0; y < kCols / 8; ++y)
                *reinterpret_cast<uint4*>(sm + P::kP + swz128(row, part * (kCols / 8) + y)) = make_uint4(0, 0, 0, 0);
        bool zero = true;
        if (c.valid) {
            zero = !load_state(c);
            if (!FOLD) {
                if (!zero) pass_state(c.m);
                arrive(&t.state);
            }
        }
        while (c.valid) {
            const bool full = c.m == kChunk;
            // ---- w V ----
            wait_at(&t.v[stage], phase);
            if (full) {
                if (parts_of(c) == 3) split_values(c, Yes{}, Yes{});
                else split_values(c, Yes{}, No{});
            } else {
                // the other rows belong to other sequences: whatever they hold
                // (a NaN times a zero weight is a NaN) must not enter sums
                wait_at(&t.qk[stage], phase);
                constexpr int kPerRow = D / 8;
                for (int i = tid; i < (kChunk - c.m) * kPerRow; i += kWork) {
                    const int r = (rev ? 0 : c.m) + i / kPerRow, x = i % kPerRow;
                    const int off = (x / 8) * 8192 + swz128(r, x % 8);
                    *reinterpret_cast<uint4*>(sm + P::kK + stage * P::kTileBytes + off) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(sm + P::kV + stage * P::kTileBytes + off) = make_uint4(0, 0, 0, 0);
                }
                if (PARTS == 3) split_values(c, No{}, Yes{});
                else split_values(c, No{}, No{});
            }
            arrive(&t.wv);
            if (!FOLD) {
                // ---- scores, and the state's part of the outputs ----
                wait_at(&t.scores, phase);
                tc_fence_after();
                if (scored) {
                    // a row, weighted by g^(i-j) (later tokens: zero)
                    uint32_t r[kCols];
                    tmem_ld(r, lanes + P::kX + part * kCols);
                    tmem_wait_ld(r);
                    uint32_t zeros = 0;
#pragma unroll
                    for (int y = 0; y < kCols / 8; ++y) {
                        uint32_t p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int j = y * 8 + e * 2;
                            p[e] = bf16x2_of(mul2(pair_of(r[j], r[j + 1]), pair(score_at[-j], score_at[-j - 1])));
                            add_zeros(zeros, p[e]);
                        }
                        *reinterpret_cast<uint4*>(sm + P::kP + swz128(row, part * (kCols / 8) + y)) = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                    // (the warp stays whole for what follows; rows without such scores have zeros there already)
                    if (__any_sync(0xffffffffu, zeros & 0x7fff7fffu)) mask_scores(sm + P::kP, row, part * kCols, kCols, rev);
                }
                if (!zero) {
                    // the state's part, aged, back into the accumulator: the
                    // values' product adds to it, and no registers hold it meanwhile
                    uint32_t r[kCols];
                    tmem_ld(r, lanes + P::kR + part * kCols);
                    tmem_wait_ld(r);
#pragma unroll
                    for (int i = 0; i < kCols; i += 4) {
                        const float4 g = *reinterpret_cast<const float4*>(&t.age[part * kCols + i]);
                        const float2 x = unpair(mul2(pair_of(r[i], r[i + 1]), pair(g.x, g.y)));
                        const float2 y = unpair(mul2(pair_of(r[i + 2], r[i + 3]), pair(g.z, g.w)));
                        r[i] = __float_as_uint(x.x), r[i + 1] = __float_as_uint(x.y);
                        r[i + 2] = __float_as_uint(y.x), r[i + 3] = __float_as_uint(y.y);
                    }
                    tmem_st(lanes + P::kR + part * kCols, r);
                    tmem_wait_st();
                }
                arrive(&t.ready);
            }
            // ---- the state after the chunk; that before the next one ----
            if (FOLD) wait(&t.update, update);
            else wait_at(&t.update, phase);
            tc_fence_after();
            if (c.at + c.m == c.end) {
                if (FOLD) store_state(a.carry + ((int64_t)t.w * a.heads + h) * ssize, 1.0f);
                else if (a.s_out && c.end == c.stop)
                    store_state(a.s_out + seq_state(c.n), frame == 0 ? 1.0f : decay_pow(ld, in_frame * kChunk + c.m));
            }
            const int m = c.m, base = low(c);
            c = next(c);
            in_frame = c.first ? 0 : in_frame + 1;
            bool zero2 = false;
            if (c.valid && c.first) zero2 = !load_state(c);
            if (!FOLD) {
                if (c.valid && !zero2) pass_state(c.m);
                // ---- outputs ----
                wait_at(&t.values, phase);
                tc_fence_after();
                uint32_t r[kCols];
                tmem_ld(r, lanes + P::kR + part * kCols);
                tmem_wait_ld(r);
                if (c.valid) arrive(&t.state);  // the accumulator is free
                if (row < D) {
                    bf16* out = static_cast<bf16*>(a.o) + h * a.o_head + (int64_t)(base + part * kCols) * a.o_tok + dv;
                    const int64_t tok = a.o_tok;
                    uint32_t z[kCols / 2];
#pragma unroll
                    for (int i = 0; i < kCols / 2; ++i) z[i] = bf16x2_of(pair_of(r[2 * i], r[2 * i + 1]));
                    auto put = [&](int i) {
                        const unsigned short x = (unsigned short)(i % 2 ? z[i / 2] >> 16 : z[i / 2]);
                        *reinterpret_cast<unsigned short*>(out) = x, out += tok;
                    };
                    if (m == kChunk) {
#pragma unroll
                        for (int i = 0; i < kCols; ++i) put(i);
                    } else {
#pragma unroll
                        for (int i = 0; i < kCols; ++i)
                            { if ((unsigned)(part * kCols + i - (rev ? kChunk - m : 0)) < (unsigned)m) put(i); else out += tok; }
                    }
                    // place of the column's first value that was not finite, or beyond the chunk
                    const int at = rev ? (int)a.tokens - kChunk - base : base;
                    const int bad = t.bad[phase * 128 + dv];
                    if (bad > at) {
                        const int place = at + m - bad, low = (rev ? kChunk - m : place) - part * kCols;
                        poison(out - kCols * tok, tok, max(low, 0), min((rev ? kChunk - place : m) - part * kCols, kCols));
                    }
                }
                __syncwarp();
            }
            if (P::kStages == 2) stage ^= 1;
            if (stage == 0) phase ^= 1;
            zero = zero2;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWork / kWarp) tmem_free(tmem, P::kTmem);
}

// ---------------------------------------------------------------------------
// launch
// ---------------------------------------------------------------------------

static PFN_cuTensorMapEncodeTiled_v12000 encoder() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
        else
            cudaGetLastError();
    });
    return fn;
}

static bool encode(CUtensorMap* map, const void* base, int64_t tok, int64_t head, int64_t tokens, int heads, int dim) {
    const bool shared = head == 0 || heads == 1;
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)(shared ? 1 : heads), (cuuint64_t)tokens};
    const cuuint64_t strides[2] = {(cuuint64_t)(shared ? dim : head) * 2, (cuuint64_t)(tokens == 1 ? dim : tok) * 2};
    const cuuint32_t box[3] = {64, 1, kChunk};
    const cuuint32_t estr[3] = {1, 1, 1};
    return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

static bool tma_rows(const void* p, int64_t tok, int64_t head, int64_t tokens, int heads) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && (tokens == 1 || (tok > 0 && tok % 8 == 0)) &&
           (heads == 1 || head % 8 == 0);
}

// Whether the chunked kernel takes a call of these roles.
bool mma_takes(const Args& a, ak_dtype dtype) {
    return dtype == AK_BF16 && a.o_tok < (1 << 30) && a.dk == a.dv && (a.dk == 64 || a.dk == 128) && a.tokens > 0 &&
           tma_rows(a.q, a.q_tok, a.q_head, a.tokens, a.heads) && tma_rows(a.k, a.k_tok, a.k_head, a.tokens, a.heads) &&
           tma_rows(a.v, a.v_tok, a.v_head, a.tokens, a.heads) && encoder() != nullptr;
}

template <int D, int PARTS, bool FOLD>
static ak_status launch(const ChunkBatch& c, cudaStream_t stream) {
    static std::atomic<uint64_t> ready{0};
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    constexpr int smem = Plan<D, PARTS, FOLD>::kSmem;
    if (!(ready.load() >> dev.device & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(k_chunks<D, PARTS, FOLD>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        if (e != cudaSuccess) return cuda_fail(e);
        ready.fetch_or(1ull << dev.device);
    }
    const Args& a = c.b.a[0];
    const dim3 grid((unsigned)a.heads, (unsigned)a.windows, (unsigned)(FOLD ? c.b.folds : c.b.count));
    if (!FOLD && a.windows > 1 && !a.by_seq)
        return launch_behind(k_chunks<D, PARTS, FOLD>, grid, Plan<D, PARTS, FOLD>::kThreads, smem, stream, c);
    k_chunks<D, PARTS, FOLD><<<grid, Plan<D, PARTS, FOLD>::kThreads, smem, stream>>>(c);
    count_launches(1);
    return check_launch();
}

template <int D, int PARTS>
static ak_status launch_passes(const ChunkBatch& c, cudaStream_t stream) {
    if (c.b.a[0].windows > 1 && !c.b.a[0].by_seq) {
        ak_status s = launch<D, PARTS, true>(c, stream);
        if (s == AK_OK) s = launch_join(c.b, stream);
        if (s != AK_OK) return s;
    }
    return launch<D, PARTS, false>(c, stream);
}

ak_status launch_chunks(const Batch& b, uint64_t* error_word, uint64_t epoch, uint64_t wait_limit_ns,
                        cudaStream_t stream) {
    ChunkBatch c;
    c.b = b;
    bool final = false;
    for (int i = 0; i < b.count; ++i) {
        const Args& a = b.a[i];
        Maps& m = c.maps[i];
        if (!encode(&m.q, a.q, a.q_tok, a.q_head, a.tokens, a.heads, a.dk) ||
            !encode(&m.k, a.k, a.k_tok, a.k_head, a.tokens, a.heads, a.dk) ||
            !encode(&m.v, a.v, a.v_tok, a.v_head, a.tokens, a.heads, a.dv))
            return AK_ERR_UNSUPPORTED;  // nothing was launched
        m.q_h = a.q_head != 0 && a.heads > 1, m.k_h = a.k_head != 0 && a.heads > 1, m.v_h = a.v_head != 0 && a.heads > 1;
        final = final || a.s_out;
    }
    c.error_word = error_word;
    c.epoch = epoch;
    c.wait_limit_ns = std::max(wait_limit_ns, kLeastWait);
    if (b.a[0].dk == 128) return final ? launch_passes<128, 3>(c, stream) : launch_passes<128, 2>(c, stream);
    return final ? launch_passes<64, 3>(c, stream) : launch_passes<64, 2>(c, stream);
}

}  // namespace la
}  // namespace ak
