// linattn_mma.cu -- linear attention with decay in chunks of 64 tokens on the
// tensor cores (bf16 inputs, head sizes 64 and 128).
//
// With S the state before a chunk of m <= 64 tokens and i, j in the chunk:
//   o_i = scale ( sum_{j<=i} g^(i-j) (q_i . k_j) v_j  +  g^(i+1) S^T q_i )
//   S  <- g^m S + sum_j g^(m-1-j) k_j v_j^T
// (a reversed call: g^i in place of g^(i+1), g^(m-j) of g^(m-1-j), see
// linattn.cuh). Everything is held transposed, M = dv = the 128 TMEM lanes:
//   P    = Q K^T                    64 x 64 scores, weighted, bf16
//   O^T  = V^T P^T  and  S^T Q^T    one accumulator (R) in turn, combined in registers
//   S^T += (w V)^T K                the float32 state, which stays in TMEM
// so that S^T, read out once a chunk to be scaled, goes back to TMEM as the
// bf16 A operand of its product with Q^T without passing shared memory, and
// 256 columns (128 S, 64 bf16 S, 64 R) let two blocks share an SM: while one
// waits for its chain of products the other uses the tensor core.
//
// Precision. Scores and the state are rounded to bf16 (once each) where they
// enter a product whose result is rounded to bf16 anyway. The state itself is
// float32 and may be an output: w V is split into bf16 parts whose products
// are exact in the float32 accumulation. Two parts keep 2^-17 of a term, three
// 2^-25; the third is spent where the final state is asked for and the term
// will still weigh more than 2^-8 in it.
//
// What bounds it: shared memory, whose 128 bytes a cycle serve the tensor
// core's operands, TMA and the working warps alike. A chunk of 64 tokens at
// D = 128 needs about 2000 cycles of it (tiles in 384, w V 384, its products
// 512, scores 450, the other two products 320), against 2700 that its 64 KB
// take from HBM at an SM's share.
//
// Seventeen warps: sixteen do the elementwise work (on TMEM, four to a
// quarter of the lanes, a quarter of the columns each); the last issues
// copies and products and never waits for more than they need. A chunk's chain: state operand; w V
// and the scores while S^T Q^T runs; V^T P^T; the outputs while the update
// runs.
//
// A chunk of fewer than 64 tokens keeps its first row at row 0, in a reversed
// call its last row at row 63: the weights then depend on the row alone.
//
// Head size 64: the A operands repeat their 64 rows (a zero stride between
// the halves of M), lanes 64..127 hold copies.
#include <algorithm>
#include <atomic>
#include <mutex>
#include <cudaTypedefs.h>

#include "ak_tcgen05.cuh"
#include "linattn.cuh"

namespace ak {
namespace la {

constexpr int kChunk = 64;
constexpr int kWork = 512;              // threads of the working warps
constexpr int kMmaThreads = kWork + 32;
constexpr int kScoreWarps = 6;           // of the sixteen; the others make w V

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

template <int D, int PARTS, bool FOLD>
struct Plan {
    static constexpr int kTileBytes = kChunk * D * 2;
    static constexpr int kQ = 0;
    static constexpr int kK = FOLD ? 0 : kTileBytes;
    static constexpr int kV = kK + kTileBytes;
    static constexpr int kP = kV + kTileBytes;
    static constexpr int kW = kP + (FOLD ? 0 : kChunk * kChunk * 2);
    static constexpr int kEnd = kW + PARTS * kTileBytes;
    // two blocks an SM share its TMEM: no third one may become resident
    static constexpr int kSmem = 1024 + (kEnd < 80 * 1024 && !FOLD ? 80 * 1024 : kEnd);
    static constexpr uint32_t kS = 0, kB = D, kR = D + D / 2;
    static constexpr uint32_t kCols = FOLD ? D : 256;
    static constexpr uint32_t kLoadBytes = (FOLD ? 2 : 3) * kTileBytes;
};

// What a block walks: the chunks of the sequence pieces in its window.
struct Chunk {
    int n;        // sequence
    int at, end;  // first token; end of the piece (a call has less than 2^31)
    int m;        // tokens of the chunk
    bool first;       // of the piece
    bool valid;
};

template <int D, int PARTS, bool FOLD>
__global__ void __launch_bounds__(kMmaThreads, 2) k_chunks(const __grid_constant__ ChunkBatch batch) {
    using P = Plan<D, PARTS, FOLD>;
    extern __shared__ unsigned char s_raw[];
    // arrivals: TMA (q and k, v), products (of the state, of the values, the
    // update), working warps (state operand ready, the other operands ready)
    __shared__ uint64_t s_qk, s_v, s_inter, s_values, s_update, s_state, s_ready;
    __shared__ uint32_t s_tmem;
    __shared__ int s_failed;
    __shared__ int64_t s_count;
    // g^n at kChunk + n, zeros below: times in_scale for the update, times
    // both scales for the scores
    __shared__ float s_pow_raw[2 * kChunk + 1], s_score_raw[2 * kChunk + 1];
    __shared__ alignas(16) float s_age[kChunk];  // weight of the state before the chunk at each row
    __shared__ int s_len[kRanked], s_rank;
    float* const s_pow = s_pow_raw + kChunk;
    float* const s_score = s_score_raw + kChunk;
    const Args& a = batch.b.a[blockIdx.z];
    const Maps& maps = batch.maps[blockIdx.z];
    unsigned char* sm = s_raw + ((1024 - (smem_addr(s_raw) & 1023)) & 1023);
    const uint32_t sbase = smem_addr(sm);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, threadIdx.x / kWarp, 0), lane = tid % kWarp;
    const int h = blockIdx.x;
    int w = blockIdx.y;
    if (a.by_seq && a.seqs <= kRanked) {
        // block w takes the w-th longest sequence: the long ones start first
        for (int i = tid; i < a.seqs; i += kMmaThreads) s_len[i] = (int)(offset_at(a, i + 1) - offset_at(a, i));
        __syncthreads();
        for (int i = tid; i < a.seqs; i += kMmaThreads) {
            const int mine = s_len[i];
            int rank = 0;
            for (int j = 0; j < a.seqs; ++j) rank += s_len[j] > mine || (s_len[j] == mine && j < i);
            if (rank == w) s_rank = i;
        }
        __syncthreads();
        w = s_rank;
    }
    int t0, t1;
    {
        int64_t from, to;
        block_span(a, w, &from, &to);
        t0 = (int)from, t1 = (int)to;
    }
    const float ld = a.log_decay[h];
    const bool rev = a.reverse;

    if (warp == kWork / kWarp) {
        tmem_alloc(&s_tmem, P::kCols);
        if (lane == 0) {
            mbar_init(&s_qk, 1);
            mbar_init(&s_v, 1);
            mbar_init(&s_inter, 1);
            mbar_init(&s_values, 1);
            mbar_init(&s_update, 1);
            mbar_init(&s_state, kWork / kWarp);
            mbar_init(&s_ready, kWork / kWarp);
            fence_barrier_init();
            s_failed = 0;
            tma_prefetch_map(&maps.k);
            tma_prefetch_map(&maps.v);
            if (!FOLD) tma_prefetch_map(&maps.q);
        }
    }
    if (tid <= 2 * kChunk) {
        const float x = tid < kChunk ? 0.0f : decay_pow(ld, tid - kChunk) * a.in_scale;
        s_pow_raw[tid] = x;
        s_score_raw[tid] = x * a.out_scale;
    }
    if (tid < kChunk) s_age[tid] = decay_pow(ld, rev ? kChunk - 1 - tid : tid + 1) * a.out_scale;
    if (!FOLD)  // scores after their row stay zero
        for (int i = tid; i < kChunk * kChunk / 8; i += kMmaThreads) *reinterpret_cast<uint4*>(sm + P::kP + i * 16) = make_uint4(0, 0, 0, 0);
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);

    // Bounded waits: a warp that gives up records it; all skip their further
    // waits and leave by the ordinary way.
    auto wait = [&](uint64_t* bar, uint32_t& phase) {
        if (!mbar_try_wait(bar, phase) && !*(volatile int*)&s_failed) {
            if (!mbar_wait(bar, phase, globaltimer_ns() + batch.wait_limit_ns)) {
                *(volatile int*)&s_failed = 1;
                if (batch.error_word) *(volatile uint64_t*)batch.error_word = batch.epoch;
            }
        }
        phase ^= 1;
        __syncwarp();  // whole warps go on to the tensor-memory instructions
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
    bf16* const o = static_cast<bf16*>(a.o) + h * a.o_head;
    auto addr = [&](int t) { return rev ? (int)a.tokens - 1 - t : t; };
    auto offset = [&](int n) { return (int)offset_at(a, n); };
    auto seq_state = [&](int n) { return ((rev ? a.seqs - 1 - n : n) * a.heads + h) * ssize; };
    // natural token of row 0 (before the array's start for a short reversed chunk)
    auto low = [&](const Chunk& c) { return rev ? (int)a.tokens - c.at - kChunk : c.at; };
    const bool writer = tid < kWork;

    // tokens of no sequence get zeros
    auto blank = [&](int from, int to) {
        if (!FOLD && writer)
            for (int t = from + tid / D; t < to; t += kWork / D) o[(int64_t)addr(t) * a.o_tok + tid % D] = __float2bfloat16_rn(0.0f);
    };
    int covered = t0;
    auto start = [&](int n, int begin, int end) {
        Chunk c;
        c.n = n;
        c.at = begin > t0 ? begin : t0;
        c.end = end < t1 ? end : t1;
        c.m = c.end - c.at < kChunk ? c.end - c.at : kChunk;
        c.first = true;
        c.valid = true;
        return c;
    };
    // the first chunk of sequence n or a later one; pieces without tokens are
    // settled on the way
    auto seek = [&](int n) {
        Chunk c = {};
        for (; n < a.seqs; ++n) {
            const int begin = offset(n), end = offset(n + 1);
            if (a.by_seq ? n > w : begin >= t1 && w != a.windows - 1) break;
            if (begin > covered) {
                blank(covered, begin < t1 ? begin : t1);
                covered = begin;
            }
            c = start(n, begin, end);
            if (c.at < c.end) {
                covered = c.end;
                return c;
            }
            if (writer && a.s_out && begin >= t0) {  // an empty sequence passes its state on
                for (int i = tid; i < D * D; i += kWork)
                    a.s_out[seq_state(n) + i] = !a.s_in ? 0.0f
                                                : a.s_in[seq_state(n) + (a.s_in_t ? (i % D) * D + i / D : i)];
            }
        }
        c.valid = false;
        if (covered < t1) blank(covered, t1);
        covered = t1;
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
        if (!FOLD && (c.end < t1 || w == a.windows - 1)) return seek(c.n + 1);
        x.valid = false;
        return x;
    };

    int n = (int)first_sequence<kMmaThreads>(a, w, t0, &s_count);
    Chunk c = {};
    int32_t kind = kNone;
    if (FOLD) {
        while (n < a.seqs && offset(n + 1) <= t1) ++n;
        const int begin = n < a.seqs ? offset(n) : t1;
        kind = begin >= t1 ? kNone : (begin >= t0 ? kFresh : kThrough);
        if (tid == 0 && h == 0) a.tail[w] = kind;
        if (kind != kNone) c = start(n, begin, t1);
    } else {
        c = seek(n);
    }
    // parts of w V that a chunk's terms need
    auto parts_of = [&](const Chunk& c) {
        return PARTS == 3 && ld * (float)(offset(c.n + 1) - c.at - c.m) > -5.55f ? 3 : 2;
    };
    // where the state before a piece comes from; null: zero
    auto source = [&](const Chunk& c, bool* transposed) -> const float* {
        *transposed = false;
        const bool here = FOLD ? kind == kFresh : offset(c.n) >= t0;
        if (!here) return FOLD ? nullptr : a.carry + ((int64_t)w * a.heads + h) * ssize;
        if (!a.s_in) return nullptr;
        // another block may already have written this sequence's result in place
        if (!FOLD && a.stash && c.end == t1 && offset(c.n + 1) > t1) return a.stash + ((int64_t)w * a.heads + h) * ssize;
        *transposed = a.s_in_t;
        return a.s_in + seq_state(c.n);
    };

    if (warp == kWork / kWarp) {
        // ------------------------------------------------------------------
        // copies and products
        // ------------------------------------------------------------------
        const uint32_t leader = lane == 0;
        uint32_t qk = 0, v = 0, state = 0, ready = 0, values = 0, update = 0;
        const uint64_t dq = smem_desc(sbase + P::kQ, 16), dp = smem_desc(sbase + P::kP, 16);
        const uint64_t dk = smem_desc(sbase + P::kK, 8192);
        const uint64_t dv = smem_desc(sbase + P::kV, D == 128 ? 8192 : 0);
        const uint64_t dw = smem_desc(sbase + P::kW, D == 128 ? 8192 : 0);
        auto load = [&](const Chunk& c, uint64_t* bar, uint32_t expect, const CUtensorMap* map, int head, int at) {
            if (leader) {
                if (expect) mbar_arrive_expect_tx(bar, expect);
#pragma unroll
                for (int b = 0; b < D / 64; ++b) tma_load_3d(sm + at + b * 8192, map, b * 64, h * head, low(c), bar);
            }
            __syncwarp();
        };
        // q announces its own bytes and those of k, which comes later
        auto load_q = [&](const Chunk& c) {
            if (!FOLD) load(c, &s_qk, 2 * P::kTileBytes, &maps.q, maps.q_h, P::kQ);
        };
        auto load_k = [&](const Chunk& c) { load(c, &s_qk, FOLD ? P::kTileBytes : 0, &maps.k, maps.k_h, P::kK); };
        auto load_v = [&](const Chunk& c) { load(c, &s_v, P::kTileBytes, &maps.v, maps.v_h, P::kV); };
        if (c.valid) {
            load_v(c);
            load_q(c);
            load_k(c);
        }
        bool zero = true;
        while (c.valid) {
            if (c.first) {
                bool t;
                zero = source(c, &t) == nullptr;
            }
            if (!FOLD && !zero) wait(&s_state, state);
            wait(&s_qk, qk);
            if (!FOLD && !zero) {
                // S^T Q^T
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < D / 16; ++s)
                    mma_ts(tmem + P::kR, tmem + P::kB + s * 8, dq + (((s / 4) * 8192 + (s % 4) * 32) >> 4),
                           mma_idesc(128, 64, false, false), s > 0, leader);
                mma_commit(&s_inter, leader);
            }
            const int parts = parts_of(c);
            const Chunk c2 = next(c);
            wait(&s_v, v);
            wait(&s_ready, ready);
            tc_fence_after();
            if (!FOLD) {
                // V^T P^T
#pragma unroll
                for (int s = 0; s < kChunk / 16; ++s)
                    mma_ss(tmem + P::kR, dv + (s * 2048 >> 4), dp + (s * 32 >> 4), mma_idesc(128, 64, true, false), s > 0, leader);
                mma_commit(&s_values, leader);
            }
            // S^T += (w V)^T K
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                if (p < 2 || parts == 3)
#pragma unroll
                    for (int s = 0; s < kChunk / 16; ++s)
                        mma_ss(tmem + P::kS, dw + ((p * P::kTileBytes + s * 2048) >> 4), dk + (s * 2048 >> 4),
                               mma_idesc(128, D, true, true), !zero || p > 0 || s > 0, leader);
            mma_commit(&s_update, leader);
            // the next chunk's tiles, each as soon as its buffer has been used
            if (c2.valid) load_q(c2);
            if (!FOLD) wait(&s_values, values);
            if (FOLD) wait(&s_update, update);
            if (c2.valid) load_v(c2);
            if (!FOLD) wait(&s_update, update);
            if (c2.valid) load_k(c2);
            zero = false;
            c = c2;
        }
    } else {
        // ------------------------------------------------------------------
        // elementwise work
        // ------------------------------------------------------------------
        const int row = (warp % 4) * 32 + lane;  // TMEM lane
        const int part = warp / 4;               // which quarter of the columns
        const int dv = row % D;                  // state column (copies at D = 64)
        const uint32_t lanes = tmem + ((uint32_t)((warp % 4) * 32) << 16);
        const Factor whole = decay_factor(ld, kChunk);
        uint32_t qk = 0, v = 0, inter_ = 0, values = 0, update = 0;
        bool zero = true;
        while (c.valid) {
            const int m = c.m;
            const int r0 = rev ? kChunk - m : 0;  // rows r0 .. r0 + m - 1 hold the chunk
            if (c.first) {
                bool tr;
                const float* src = source(c, &tr);
                zero = src == nullptr;
                if (src) {
                    // a fold ages its state once, not chunk by chunk
                    const float age = FOLD ? decay_pow(ld, t1 - c.at) : 1.0f;
#pragma unroll 1
                    for (int k0 = part * (D / 4); k0 < (part + 1) * (D / 4); k0 += 16) {
                        uint32_t r[16];
                        const float* p = tr ? src + dv * D + k0 : src + k0 * D + dv;
#pragma unroll
                        for (int i = 0; i < 16; ++i, p += tr ? 1 : D) r[i] = __float_as_uint(*p);
                        if (FOLD && a.stash && row < D) {
                            float* keep = a.stash + ((int64_t)w * a.heads + h) * ssize + k0 * D + dv;
#pragma unroll
                            for (int i = 0; i < 16; ++i) keep[i * D] = __uint_as_float(r[i]);
                        }
                        if (FOLD)
#pragma unroll
                            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * age);
                        tmem_st16(lanes + P::kS + k0, r);
                    }
                    tmem_wait_st();
                }
            }
            // S^T as a bf16 operand, and scaled by g^m
            if (!FOLD && !zero) {
                const Factor f = m == kChunk ? whole : decay_factor(ld, m);
#pragma unroll 1
                for (int k0 = part * (D / 4); k0 < (part + 1) * (D / 4); k0 += 16) {
                    uint32_t r[16], p[8];
                    tmem_ld16(r, lanes + P::kS + k0);
                    tmem_wait_ld(r);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                        memcpy(&p[i], &x, 4);
                    }
                    tmem_st8(lanes + P::kB + k0 / 2, p);
                    if (f.hi == 1.0f) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(fmaf(__uint_as_float(r[i]), f.lo, __uint_as_float(r[i])));
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f.hi);
                    }
                    tmem_st16(lanes + P::kS + k0, r);
                }
                tmem_wait_st();
                arrive(&s_state);
            }
            uint32_t inter[16];
            if (!FOLD && warp < kScoreWarps) {
                wait(&s_qk, qk);
                v ^= 1;
                // Scores: 32 x 16 a warp, on register-level matrix
                // instructions; the quarter of the tile after its rows stays
                // zero. The way through TMEM (issue, barrier, load: about 1300
                // cycles) would lie on the chunk's chain and wants 64 columns
                // that are not there.
                const int rb = (rev ? warp > 3 : warp > 1) * 32;
                const int cb = (rev ? (warp > 3 ? warp - 2 : warp) : (warp > 1 ? warp - 2 : warp)) * 16;
                float x[2][2][4] = {};
#pragma unroll
                for (int s = 0; s < D / 16; ++s) {
                    const uint32_t box = sbase + (s / 4) * 8192;
                    uint32_t qa[2][4], kb[4];
                    ldmatrix4(kb, box + P::kK + swz128(cb + lane % 8 + lane / 16 * 8, (s % 4) * 2 + lane / 8 % 2));
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        ldmatrix4(qa[u], box + P::kQ + swz128(rb + u * 16 + lane % 16, (s % 4) * 2 + lane / 16));
#pragma unroll
                        for (int t = 0; t < 2; ++t) mma_16x8x16(x[u][t], qa[u], kb[2 * t], kb[2 * t + 1]);
                    }
                }
                // weighted by g^(i-j); later tokens count nothing
                const int i0 = rb + lane / 4, j0 = cb + lane % 4 * 2;
                const int corner = rev ? j0 - i0 : i0 - j0;
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int di = u * 16 + e * 8, dj = t * 8;
                            const int gap = corner + (rev ? dj - di : di - dj), gap1 = rev ? gap + 1 : gap - 1;
                            const float wl = s_score[gap], wh = s_score[gap1];
                            const float lo = gap >= 0 ? x[u][t][2 * e] * wl : 0.0f;
                            const float hi = gap1 >= 0 ? x[u][t][2 * e + 1] * wh : 0.0f;
                            *reinterpret_cast<__nv_bfloat162*>(sm + P::kP + swz128(i0 + di, cb / 8 + t) + lane % 4 * 4) =
                                __floats2bfloat162_rn(lo, hi);
                        }
            } else {
                // w V in bf16 parts
                constexpr int kFirst = FOLD ? 0 : kScoreWarps * kWarp, kCount = kWork - kFirst;
                const int mine = tid - kFirst;
                wait(&s_v, v);
                if (m < kChunk) {
                    // the other rows belong to other sequences: whatever they hold
                    // (a NaN times a zero weight is a NaN) must not enter sums
                    wait(&s_qk, qk);
                    constexpr int kPerRow = D / 8;
                    for (int i = mine; i < (kChunk - m) * kPerRow; i += kCount) {
                        const int r = (rev ? 0 : m) + i / kPerRow, x = i % kPerRow;
                        const int off = (x / 8) * 8192 + swz128(r, x % 8);
                        *reinterpret_cast<uint4*>(sm + P::kK + off) = make_uint4(0, 0, 0, 0);
                        *reinterpret_cast<uint4*>(sm + P::kV + off) = make_uint4(0, 0, 0, 0);
                    }
                } else {
                    qk ^= 1;
                }
                const int parts = parts_of(c);
                const float* const pw = s_pow + (rev ? 1 - r0 : m - 1);
                const float age = FOLD ? decay_pow(ld, t1 - c.at - m) : 1.0f;
#pragma unroll 2
                for (int i = mine; i < kChunk * D / 8; i += kCount) {
                    const int r = i / (D / 8), x = i % (D / 8);
                    const int off = (x / 8) * 8192 + swz128(r, x % 8);
                    uint4 vv = *reinterpret_cast<const uint4*>(sm + P::kV + off);
                    if ((unsigned)(r - r0) >= (unsigned)m) vv = make_uint4(0, 0, 0, 0);
                    const float wt = pw[rev ? r : -r] * age;
                    const uint32_t in[4] = {vv.x, vv.y, vv.z, vv.w};
                    uint32_t part[2][4];
                    float rest[8];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float lo = __uint_as_float(in[e] << 16) * wt, hi = __uint_as_float(in[e] & 0xffff0000u) * wt;
#pragma unroll
                        for (int p = 0; p < 2; ++p) {
                            const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
                            memcpy(&part[p][e], &y, 4);
                            if (p == 0 || PARTS == 3) {
                                lo -= __uint_as_float(part[p][e] << 16);
                                hi -= __uint_as_float(part[p][e] & 0xffff0000u);
                            }
                        }
                        rest[2 * e] = lo, rest[2 * e + 1] = hi;
                    }
#pragma unroll
                    for (int p = 0; p < 2; ++p)
                        *reinterpret_cast<uint4*>(sm + P::kW + p * P::kTileBytes + off) =
                            make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
                    if (PARTS == 3 && parts == 3) {
                        uint32_t last[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const __nv_bfloat162 y = __floats2bfloat162_rn(rest[2 * e], rest[2 * e + 1]);
                            memcpy(&last[e], &y, 4);
                        }
                        *reinterpret_cast<uint4*>(sm + P::kW + 2 * P::kTileBytes + off) = make_uint4(last[0], last[1], last[2], last[3]);
                    }
                }
            }
            __syncwarp();
            if (!FOLD && !zero) {
                wait(&s_inter, inter_);
                tc_fence_after();
                if (row < D) {
                    tmem_ld16(inter, lanes + P::kR + part * 16);
                    tmem_wait_ld(inter);
                }
            }
            arrive(&s_ready);
            const Chunk c2 = next(c);
            if (!FOLD) {
                wait(&s_values, values);
                tc_fence_after();
                if (row < D) {
                    bf16* const out = o + (int64_t)(low(c) + part * 16) * a.o_tok + dv;
                    const int tok = (int)a.o_tok;
                    uint32_t r[16];
                    tmem_ld16(r, lanes + P::kR + part * 16);
                    tmem_wait_ld(r);
                    bf16 z[16];
#pragma unroll
                    for (int i = 0; i < 16; i += 4) {
                        const float4 g = *reinterpret_cast<const float4*>(&s_age[part * 16 + i]);
                        const float wt[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            float x = __uint_as_float(r[i + e]);
                            if (!zero) x = fmaf(__uint_as_float(inter[i + e]), wt[e], x);
                            z[i + e] = __float2bfloat16_rn(x);
                        }
                    }
                    if (m == kChunk) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) out[(int64_t)tok * i] = z[i];
                    } else {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if ((unsigned)(part * 16 + i - r0) < (unsigned)m) out[(int64_t)tok * i] = z[i];
                    }
                }
                __syncwarp();
            }
            wait(&s_update, update);  // the state is up to date; w V may be overwritten
            tc_fence_after();
            zero = false;
            // the state after the piece
            float* dst = nullptr;
            if (c.at + m == c.end) {
                if (FOLD) dst = a.carry + ((int64_t)w * a.heads + h) * ssize;
                else if (a.s_out && c.end == offset(c.n + 1)) dst = a.s_out + seq_state(c.n);
            }
            if (dst && row < D) {
#pragma unroll 1
                for (int k0 = part * (D / 4); k0 < (part + 1) * (D / 4); k0 += 16) {
                    uint32_t r[16];
                    tmem_ld16(r, lanes + P::kS + k0);
                    tmem_wait_ld(r);
                    float* to = dst + k0 * D + dv;
#pragma unroll
                    for (int i = 0; i < 16; ++i) to[i * D] = __uint_as_float(r[i]);
                }
            }
            __syncwarp();
            c = c2;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kWork / kWarp) tmem_free(tmem, P::kCols);
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
    const dim3 grid((unsigned)a.heads, (unsigned)a.windows, (unsigned)c.b.count);
    k_chunks<D, PARTS, FOLD><<<grid, kMmaThreads, smem, stream>>>(c);
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
    c.wait_limit_ns = wait_limit_ns;
    if (b.a[0].dk == 128) return final ? launch_passes<128, 3>(c, stream) : launch_passes<128, 2>(c, stream);
    return final ? launch_passes<64, 3>(c, stream) : launch_passes<64, 2>(c, stream);
}

}  // namespace la
}  // namespace ak
