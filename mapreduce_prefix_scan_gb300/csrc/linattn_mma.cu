// linattn_mma.cu -- linear attention with decay in chunks of 64 tokens on the
// tensor cores (bf16 inputs, head sizes 64 and 128).
//
// With S the state before a chunk of m <= 64 tokens and i, j in the chunk:
//   o_i = scale ( sum_{j<=i} g^(i-j) (q_i . k_j) v_j  +  g^(i+1) S^T q_i )
//   S  <- g^m S + sum_j g^(m-1-j) k_j v_j^T
// (a reversed call: g^i in place of g^(i+1), g^(m-j) of g^(m-1-j), see
// linattn.cuh). Everything is held transposed, M = dv = the 128 TMEM lanes:
//   P    = Q K^T                    64 x 64 scores (accumulator R)
//   O^T  = V^T P^T  and  S^T Q^T    two products, combined in registers (R)
//   S^T += (w V)^T K                the float32 state, which stays in TMEM
// so that S^T, read out once a chunk to be scaled, goes back to TMEM as the
// bf16 A operand of its product with Q^T without passing shared memory, and
// 256 columns (128 S, 64 bf16 S, 64 R) let two blocks share an SM: while one
// waits for its chain of products the other uses the tensor core.
//
// Precision. Scores and the state are rounded to bf16 (once each) where they
// enter a product whose result is rounded to bf16 anyway. The state itself is
// float32 and may be an output: w V is split into bf16 parts (hi, mid and,
// where the final state is asked for, lo), whose products are exact in the
// float32 accumulation, so it keeps 2^-17 (two parts) or 2^-25 (three) of
// each term.
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
constexpr int kMmaThreads = 256;

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
    int64_t n;        // sequence
    int64_t at, end;  // first token; end of the piece
    int m;            // tokens of the chunk
    bool first;       // of the piece
    bool valid;
};

template <int D, int PARTS, bool FOLD>
__global__ void __launch_bounds__(kMmaThreads, 2) k_chunks(const __grid_constant__ ChunkBatch batch) {
    using P = Plan<D, PARTS, FOLD>;
    extern __shared__ unsigned char s_raw[];
    __shared__ uint64_t s_full, s_mma, s_upd;
    __shared__ uint32_t s_tmem;
    __shared__ int s_failed;
    __shared__ int64_t s_count;
    // g^n at kChunk + n, zeros below; the second table holds g^n in_scale
    __shared__ float s_pow_raw[2 * kChunk + 1], s_pows_raw[2 * kChunk + 1];
    float* const s_pow = s_pow_raw + kChunk;
    float* const s_pows = s_pows_raw + kChunk;
    const Args& a = batch.b.a[blockIdx.z];
    const Maps& maps = batch.maps[blockIdx.z];
    unsigned char* sm = s_raw + ((1024 - (smem_addr(s_raw) & 1023)) & 1023);
    const uint32_t sbase = smem_addr(sm);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, threadIdx.x / kWarp, 0), lane = tid % kWarp;
    const uint32_t leader = lane == 0;  // of warp 0, which issues products and copies
    const int row = (warp % 4) * 32 + lane;  // TMEM lane
    const int half = warp / 4;               // which half of the columns
    const int dv = row % D;                  // state column (copies at D = 64)
    const int64_t w = blockIdx.x;
    const int h = blockIdx.y;
    int64_t t0, t1;
    block_span(a, w, &t0, &t1);
    const float ld = a.log_decay[h];
    const bool rev = a.reverse;
    const int64_t ssize = (int64_t)D * D;
    bf16* o = static_cast<bf16*>(a.o) + h * a.o_head;

    if (warp == 0) tmem_alloc(&s_tmem, P::kCols);
    if (tid == 0) {
        mbar_init(&s_full, 1);
        mbar_init(&s_mma, 1);
        mbar_init(&s_upd, 1);
        fence_barrier_init();
        s_failed = 0;
        tma_prefetch_map(&maps.k);
        tma_prefetch_map(&maps.v);
        if (!FOLD) tma_prefetch_map(&maps.q);
    }
    if (tid <= 2 * kChunk) {
        const float x = tid < kChunk ? 0.0f : decay_pow(ld, tid - kChunk);
        s_pow_raw[tid] = x;
        s_pows_raw[tid] = x * a.in_scale;
    }
    const Factor whole = decay_factor(ld, kChunk);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, s_tmem, 0);
    const uint32_t lanes = (uint32_t)((warp % 4) * 32) << 16;

    // Bounded waits: a block that gives up records it, skips its further
    // waits and leaves by the ordinary way.
    uint32_t full_phase = 0, mma_phase = 0, upd_phase = 0;
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

    auto addr = [&](int64_t t) { return rev ? a.tokens - 1 - t : t; };
    auto seq_state = [&](int64_t n) { return ((rev ? a.seqs - 1 - n : n) * a.heads + h) * ssize; };
    // first natural token of a chunk
    auto low = [&](const Chunk& c) { return rev ? a.tokens - c.at - c.m : c.at; };

    auto load_q = [&](const Chunk& c) {  // announces the whole chunk's bytes
        mbar_arrive_expect_tx(&s_full, P::kLoadBytes);
        if (!FOLD)
#pragma unroll
            for (int b = 0; b < D / 64; ++b)
                tma_load_3d(sm + P::kQ + b * 8192, &maps.q, b * 64, h * maps.q_h, (int)low(c), &s_full);
    };
    auto load_kv = [&](const Chunk& c) {
#pragma unroll
        for (int b = 0; b < D / 64; ++b) {
            tma_load_3d(sm + P::kK + b * 8192, &maps.k, b * 64, h * maps.k_h, (int)low(c), &s_full);
            tma_load_3d(sm + P::kV + b * 8192, &maps.v, b * 64, h * maps.v_h, (int)low(c), &s_full);
        }
    };

    // tokens of no sequence get zeros
    auto blank = [&](int64_t from, int64_t to) {
        if constexpr (!FOLD)
            for (int64_t t = from + tid / D; t < to; t += kMmaThreads / D)
                o[addr(t) * a.o_tok + tid % D] = __float2bfloat16_rn(0.0f);
    };
    // the next chunk after `c`; pieces without tokens are settled on the way
    int64_t covered = t0;
    auto start = [&](int64_t n, int64_t begin, int64_t end) {
        Chunk c;
        c.n = n;
        c.at = begin > t0 ? begin : t0;
        c.end = end < t1 ? end : t1;
        c.m = (int)(c.end - c.at < kChunk ? c.end - c.at : kChunk);
        c.first = true;
        c.valid = true;
        return c;
    };
    auto seek = [&](int64_t n) {
        Chunk c = {};
        for (; n < a.seqs; ++n) {
            const int64_t begin = offset_at(a, n), end = offset_at(a, n + 1);
            if (a.by_seq ? n > w : begin >= t1 && w != a.windows - 1) break;
            if (begin > covered) blank(covered, begin < t1 ? begin : t1);
            if (begin > covered) covered = begin;
            c = start(n, begin, end);
            if (c.at < c.end) {
                covered = c.end;
                return c;
            }
            if (a.s_out && begin >= t0) {  // an empty sequence passes its state on
                for (int64_t i = tid; i < ssize; i += kMmaThreads)
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
            x.m = (int)(c.end - x.at < kChunk ? c.end - x.at : kChunk);
            return x;
        }
        if (FOLD || c.end >= t1) {
            // nothing of a later sequence but empty ones at the axis' end
            if (!FOLD && w == a.windows - 1) return seek(c.n + 1);
            x.valid = false;
            return x;
        }
        return seek(c.n + 1);
    };

    int64_t n = first_sequence<kMmaThreads>(a, t0, &s_count);
    Chunk c;
    int32_t kind = kNone;
    if (FOLD) {
        while (n < a.seqs && offset_at(a, n + 1) <= t1) ++n;
        const int64_t begin = n < a.seqs ? offset_at(a, n) : t1;
        kind = begin >= t1 ? kNone : (begin >= t0 ? kFresh : kThrough);
        if (tid == 0 && h == 0) a.tail[w] = kind;
        c = {};
        if (kind != kNone) c = start(n, begin, t1);
    } else {
        c = seek(n);
    }
    if (tid == 0 && c.valid) {
        load_q(c);
        load_kv(c);
    }

    bool zero = true;  // the state before the chunk is zero
    while (c.valid) {
        if (c.first) {
            // the state before the piece
            const int64_t begin = FOLD ? (kind == kFresh ? c.at : c.at - 1) : offset_at(a, c.n);
            const float* src = nullptr;
            bool tr = false;
            if (begin >= t0) {
                if (a.s_in) src = a.s_in + seq_state(c.n), tr = a.s_in_t;
                // another block may already have written this one's result in place
                if (!FOLD && a.stash && c.end == t1 && offset_at(a, c.n + 1) > t1) src = a.stash + (w * a.heads + h) * ssize;
            } else if (!FOLD) {
                src = a.carry + (w * a.heads + h) * ssize;
            }
            zero = src == nullptr;
            if (src) {
#pragma unroll 1
                for (int b = 0; b < D / 64; ++b) {
                    const int k0 = half * (D / 2) + b * 32;
                    uint32_t r[32];
                    if (tr) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4) {
                            // rows of a transposed state are the caller's: 4-byte alignment is all that is known
                            const float* p = src + (int64_t)dv * D + k0 + i;
#pragma unroll
                            for (int e = 0; e < 4; ++e) r[i + e] = __float_as_uint(p[e]);
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(src[(int64_t)(k0 + i) * D + dv]);
                    }
                    tmem_st32(tmem + lanes + P::kS + k0, r);
                    if (FOLD && a.stash && row < D) {
                        float* keep = a.stash + (w * a.heads + h) * ssize;
#pragma unroll
                        for (int i = 0; i < 32; ++i) keep[(int64_t)(k0 + i) * D + dv] = __uint_as_float(r[i]);
                    }
                }
                tmem_wait_st();
            }
        }
        wait(&s_full, full_phase);
        const int m = c.m;
        if (m < kChunk) {
            // rows past the chunk belong to other sequences: whatever they
            // hold (a NaN times a zero weight is a NaN) must not enter sums
            constexpr int kPerRow = D / 8;
            for (int i = tid; i < (kChunk - m) * kPerRow; i += kMmaThreads) {
                const int r = m + i / kPerRow, x = i % kPerRow;
                const int off = (x / 8) * 8192 + swz128(r, x % 8);
                *reinterpret_cast<uint4*>(sm + P::kK + off) = make_uint4(0, 0, 0, 0);
                *reinterpret_cast<uint4*>(sm + P::kV + off) = make_uint4(0, 0, 0, 0);
            }
            fence_async_smem();
            __syncthreads();
        }
        if (!FOLD && warp == 0) {
            tc_fence_after();
            // P = Q K^T; rows 64..127 of M read on into the next tile and are not used
#pragma unroll
            for (int s = 0; s < D / 16; ++s) {
                const uint32_t off = (s / 4) * 8192 + (s % 4) * 32;
                mma_ss(tmem + P::kR, smem_desc(sbase + P::kQ + off, 16), smem_desc(sbase + P::kK + off, 16),
                       mma_idesc(128, 64, false, false), s > 0, leader);
            }
            mma_commit(&s_mma, leader);
        }
        // S^T as a bf16 operand, and scaled by g^m
        if (!zero) {
            const Factor f = m == kChunk ? whole : decay_factor(ld, m);
#pragma unroll 1
            for (int b = 0; b < D / 64; ++b) {
                const int k0 = half * (D / 2) + b * 32;
                uint32_t r[32];
                tmem_ld32(r, tmem + lanes + P::kS + k0);
                tmem_wait_ld(r);
                if (!FOLD) {
                    uint32_t p[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(r[2 * i]), __uint_as_float(r[2 * i + 1]));
                        memcpy(&p[i], &x, 4);
                    }
                    tmem_st16(tmem + lanes + P::kB + k0 / 2, p);
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
                tmem_st32(tmem + lanes + P::kS + k0, r);
            }
            tmem_wait_st();
        }
        // w V in bf16 parts
        constexpr int kChunks16 = kChunk * D / 8;
#pragma unroll
        for (int i = tid; i < kChunks16; i += kMmaThreads) {
            const int r = i / (D / 8), x = i % (D / 8);
            const int off = (x / 8) * 8192 + swz128(r, x % 8);
            const uint4 vv = *reinterpret_cast<const uint4*>(sm + P::kV + off);
            const float wt = s_pows[rev ? r + 1 : m - 1 - r];  // rows past the chunk are zeros
            const uint32_t in[4] = {vv.x, vv.y, vv.z, vv.w};
            uint32_t part[PARTS][4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                float lo = __uint_as_float(in[e] << 16) * wt, hi = __uint_as_float(in[e] & 0xffff0000u) * wt;
#pragma unroll
                for (int p = 0; p < PARTS; ++p) {
                    const __nv_bfloat162 y = __floats2bfloat162_rn(lo, hi);
                    memcpy(&part[p][e], &y, 4);
                    lo -= __uint_as_float(part[p][e] << 16);
                    hi -= __uint_as_float(part[p][e] & 0xffff0000u);
                }
            }
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
                *reinterpret_cast<uint4*>(sm + P::kW + p * P::kTileBytes + off) =
                    make_uint4(part[p][0], part[p][1], part[p][2], part[p][3]);
        }
        if (!FOLD) {
            wait(&s_mma, mma_phase);
            tc_fence_after();
            if (row < kChunk) {
                // a row of scores, weighted by g^(i-j); later tokens count nothing
                uint32_t r[32];
                tmem_ld32(r, tmem + lanes + P::kR + half * 32);
                const int step = rev ? 1 : -1;
                const int gap0 = rev ? half * 32 - row : row - half * 32;
                float wt[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) wt[j] = s_pows[gap0 + step * j];
                tmem_wait_ld(r);
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    uint32_t p[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int j = x * 8 + e * 2;
                        const float lo = gap0 + step * j >= 0 ? __uint_as_float(r[j]) * wt[j] : 0.0f;
                        const float hi = gap0 + step * (j + 1) >= 0 ? __uint_as_float(r[j + 1]) * wt[j + 1] : 0.0f;
                        const __nv_bfloat162 z = __floats2bfloat162_rn(lo, hi);
                        memcpy(&p[e], &z, 4);
                    }
                    *reinterpret_cast<uint4*>(sm + P::kP + swz128(row, half * 4 + x)) = make_uint4(p[0], p[1], p[2], p[3]);
                }
            }
        }
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        auto update = [&] {  // S^T += (w V)^T K
#pragma unroll
            for (int p = 0; p < PARTS; ++p)
#pragma unroll
                for (int s = 0; s < kChunk / 16; ++s)
                    mma_ss(tmem + P::kS, smem_desc(sbase + P::kW + p * P::kTileBytes + s * 2048, D == 128 ? 8192 : 0),
                           smem_desc(sbase + P::kK + s * 2048, 8192), mma_idesc(128, D, true, true), !zero || p > 0 || s > 0, leader);
        };
        Chunk c2;
        if (!FOLD) {
            uint32_t inter[32];
            if (zero) {
                c2 = next(c);
            } else {
                if (warp == 0) {
                    tc_fence_after();
#pragma unroll
                    for (int s = 0; s < D / 16; ++s)
                        mma_ts(tmem + P::kR, tmem + P::kB + s * 8,
                               smem_desc(sbase + P::kQ + (s / 4) * 8192 + (s % 4) * 32, 16),
                               mma_idesc(128, 64, false, false), s > 0, leader);
                    mma_commit(&s_mma, leader);
                }
                c2 = next(c);
                wait(&s_mma, mma_phase);
                tc_fence_after();
                if (row < D) {
                    tmem_ld32(inter, tmem + lanes + P::kR + half * 32);
                    tmem_wait_ld(inter);
                }
                tc_fence_before();
                __syncthreads();
            }
            if (warp == 0) {
                tc_fence_after();
#pragma unroll
                for (int s = 0; s < kChunk / 16; ++s)
                    mma_ss(tmem + P::kR, smem_desc(sbase + P::kV + s * 2048, D == 128 ? 8192 : 0),
                           smem_desc(sbase + P::kP + s * 32, 16), mma_idesc(128, 64, true, false), s > 0, leader);
                mma_commit(&s_mma, leader);
                update();
                mma_commit(&s_upd, leader);
                // the query tile has been used
                if (leader && c2.valid) load_q(c2);
            }
            wait(&s_mma, mma_phase);
            tc_fence_after();
            if (row < D) {
                uint32_t r[32];
                tmem_ld32(r, tmem + lanes + P::kR + half * 32);
                const float* const pw = s_pow + (rev ? m - 1 - half * 32 : 1 + half * 32);
                const int step = rev ? -1 : 1;
                float wt[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) wt[i] = pw[step * i];
                tmem_wait_ld(r);
                bf16 y[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                    const float x = zero ? __uint_as_float(r[i]) : fmaf(__uint_as_float(inter[i]), wt[i], __uint_as_float(r[i]));
                    y[i] = __float2bfloat16_rn(x * a.out_scale);
                }
                bf16* out = o + (low(c) + half * 32) * a.o_tok + dv;
                if (m == kChunk) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) out[i * a.o_tok] = y[i];
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        if (half * 32 + i < m) out[i * a.o_tok] = y[i];
                }
            }
            __syncwarp();
        } else {
            if (warp == 0) {
                tc_fence_after();
                update();
                mma_commit(&s_upd, leader);
            }
            c2 = next(c);
            if (tid == 0 && c2.valid) load_q(c2);
            __syncwarp();
        }
        wait(&s_upd, upd_phase);  // the update is done: k, v and w V are free
        tc_fence_after();
        if (tid == 0 && c2.valid) load_kv(c2);
        zero = false;
        // the state after the piece
        float* dst = nullptr;
        if (c.at + m == c.end) {
            if (FOLD) dst = a.carry + (w * a.heads + h) * ssize;
            else if (a.s_out && c.end == offset_at(a, c.n + 1)) dst = a.s_out + seq_state(c.n);
        }
        if (dst && row < D) {
#pragma unroll 1
            for (int b = 0; b < D / 64; ++b) {
                const int k0 = half * (D / 2) + b * 32;
                uint32_t r[32];
                tmem_ld32(r, tmem + lanes + P::kS + k0);
                tmem_wait_ld(r);
#pragma unroll
                for (int i = 0; i < 32; ++i) dst[(int64_t)(k0 + i) * D + dv] = __uint_as_float(r[i]);
            }
        }
        tc_fence_before();
        c = c2;
        __syncthreads();
    }
    __syncthreads();
    if (warp == 0) tmem_free(tmem, P::kCols);
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
    return dtype == AK_BF16 && a.dk == a.dv && (a.dk == 64 || a.dk == 128) && a.tokens > 0 &&
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
    const dim3 grid((unsigned)a.windows, (unsigned)a.heads, (unsigned)c.b.count);
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
