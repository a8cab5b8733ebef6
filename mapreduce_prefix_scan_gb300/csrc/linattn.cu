// linattn.cu -- linear attention with a decay for each head: the token-by-
// token kernel for every type and head size, the join of window states, the
// single-token step and the choice between the kernels (linattn.cuh has the
// mathematics; linattn_mma.cu the chunked tensor-core kernel).
#include <algorithm>

#include "linattn.cuh"

namespace ak {
namespace la {

__device__ __forceinline__ float as_f(float v) { return v; }
__device__ __forceinline__ float as_f(bf16 v) { return __bfloat162float(v); }
template <class T>
__device__ __forceinline__ T from_f(float v) {
    if constexpr (std::is_same_v<T, bf16>) return __float2bfloat16_rn(v);
    else return v;
}

// ---------------------------------------------------------------------------
// token by token
// ---------------------------------------------------------------------------
// A block holds 32 columns of the state of one head: 4 groups of DK / 4 rows
// x 32 columns, a column's rows of a group in one thread's registers, so the
// state is read and written once a sequence piece. k, q and v of kTile tokens
// pass through registers into shared memory, the next tile's loads in flight
// while one is worked on (k and q are read as 16-byte broadcasts); the groups'
// parts of each output are added in shared memory once a tile.
//
// The decay leaves the inner loop: with X = g S before a block of b tokens,
//   S_e = g^e (X + sum_{j<=e} g^-j k_j v_j^T),  e = 0 .. b - 1,
// so v enters scaled by g^-j, o leaves scaled by g^e, and the state is scaled
// once a block (by a two-float factor). b is the largest power of two up to
// kTile that keeps g^-j below e^40. That is 2 DK fused operations a column
// and token: bound by the FMA pipe for long inputs and by the chain of tokens
// for few heads (hence the windows). 2049 tokens, 8 heads of 80, float32:
// 85 us in three launches, where waiting for each tile's loads took 145 and
// asking after every token whether a block ends 91.
constexpr int kTile = 16;
constexpr int kGroups = 4;
constexpr int kThreads = 32 * kGroups;

template <class T, int DK, bool FOLD>
__global__ void __launch_bounds__(kThreads) k_tokens(const __grid_constant__ Batch batch) {
    constexpr int R = DK / kGroups;
    __shared__ alignas(16) float s_k[kTile][DK]; __shared__ alignas(16) float s_q[FOLD ? 1 : kTile][FOLD ? 4 : DK];
    __shared__ float s_v[kTile][32];
    __shared__ float s_w[kTile], s_inv[kTile];  // g^e of each token times the output's scale, g^-e times the input's
    __shared__ float s_o[FOLD ? 1 : kTile][kGroups][32];
    __shared__ int64_t s_count;
    const int col = threadIdx.x % 32, grp = threadIdx.x / 32;
    const int64_t w = blockIdx.x;
    const int h = blockIdx.y;
    const int calls = FOLD ? batch.folds : batch.count;
    const Args& a = batch.a[blockIdx.z % calls];
    const int c0 = blockIdx.z / calls * 32;
    if (FOLD) griddep_launch_dependents();
    if (c0 >= a.dv) return;  // the calls of a batch may differ in dv
    const bool live = c0 + col < a.dv;
    int64_t t0, t1;
    block_span(a, w, &t0, &t1);
    const float ld = a.log_decay[h];
    int block = kTile;
    while (block > 1 && !(fabsf(ld) * block <= 40.0f)) block /= 2;
    const Factor whole = decay_factor(ld, block);
    const T* q = static_cast<const T*>(a.q) + h * a.q_head;
    const T* k = static_cast<const T*>(a.k) + h * a.k_head;
    const T* v = static_cast<const T*>(a.v) + h * a.v_head;
    T* o = static_cast<T*>(a.o) + h * a.o_head;
    const int64_t ssize = (int64_t)a.dk * a.dv;
    float s[R];

    auto addr = [&](int64_t t) { return a.reverse ? a.tokens - 1 - t : t; };
    // tokens of no sequence get zeros
    auto blank = [&](int64_t from, int64_t to) {
        if (FOLD) return;
        for (int64_t t = from + grp; t < to; t += kGroups)
            if (live) o[addr(t) * a.o_tok + c0 + col] = from_f<T>(0.0f);
    };
    auto load_state = [&](const float* src, bool transposed) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = grp * R + i;
            s[i] = 0.0f;
            if (src && live && r < a.dk)
                s[i] = transposed ? src[(int64_t)(c0 + col) * a.dk + r] : src[(int64_t)r * a.dv + c0 + col];
        }
    };
    auto store_state = [&](float* dst) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = grp * R + i;
            if (live && r < a.dk) dst[(int64_t)r * a.dv + c0 + col] = s[i];
        }
    };
    auto seq_state = [&](int64_t n) {
        const int64_t m = a.reverse ? a.seqs - 1 - n : n;
        return (m * a.heads + h) * ssize;
    };
    if (threadIdx.x < kTile) {
        const int e = threadIdx.x & (block - 1);
        s_w[threadIdx.x] = decay_pow(ld, e) * a.out_scale;
        s_inv[threadIdx.x] = decay_pow(ld, -e) * a.in_scale;
    }
    // tokens [from, to) of one sequence
    constexpr int kLoads = kTile * DK / kThreads, kLoadsV = kTile * 32 / kThreads;
    float fk[kLoads], fq[FOLD ? 1 : kLoads], fv[kLoadsV];
    auto fetch = [&](int64_t tb, int m) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int x = threadIdx.x + i * kThreads, t = x / DK, r = x % DK;
            const bool in = t < m && r < a.dk;
            fk[i] = in ? as_f(k[addr(tb + t) * a.k_tok + r]) : 0.0f;
            if (!FOLD) fq[i] = in ? as_f(q[addr(tb + t) * a.q_tok + r]) : 0.0f;
        }
#pragma unroll
        for (int i = 0; i < kLoadsV; ++i) {
            const int t = grp + i * kGroups;
            fv[i] = t < m && live ? as_f(v[addr(tb + t) * a.v_tok + c0 + col]) : 0.0f;
        }
    };
    auto walk = [&](int64_t from, int64_t to) {
        if (!a.reverse) {
            const Factor one = decay_factor(ld, 1);
#pragma unroll
            for (int i = 0; i < R; ++i) s[i] = s[i] * one;
        }
        fetch(from, (int)(to - from < kTile ? to - from : kTile));
        for (int64_t tb = from; tb < to; tb += kTile) {
            const int m = (int)(to - tb < kTile ? to - tb : kTile);
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kLoads; ++i) {
                const int x = threadIdx.x + i * kThreads;
                s_k[x / DK][x % DK] = fk[i];
                if (!FOLD) s_q[x / DK][x % DK] = fq[i];
            }
#pragma unroll
            for (int i = 0; i < kLoadsV; ++i) s_v[grp + i * kGroups][col] = fv[i] * s_inv[grp + i * kGroups];
            __syncthreads();
            if (tb + kTile < to) fetch(tb + kTile, (int)(to - tb - kTile < kTile ? to - tb - kTile : kTile));
            auto token = [&](int t) {
                const float vv = s_v[t][col];
                float acc[4] = {};
#pragma unroll
                for (int i = 0; i < R; i += 4) {
                    const float4 kk = *reinterpret_cast<const float4*>(&s_k[t][grp * R + i]);
                    s[i] = fmaf(kk.x, vv, s[i]), s[i + 1] = fmaf(kk.y, vv, s[i + 1]);
                    s[i + 2] = fmaf(kk.z, vv, s[i + 2]), s[i + 3] = fmaf(kk.w, vv, s[i + 3]);
                    if (!FOLD) {
                        const float4 qq = *reinterpret_cast<const float4*>(&s_q[t][grp * R + i]);
                        acc[0] = fmaf(qq.x, s[i], acc[0]), acc[1] = fmaf(qq.y, s[i + 1], acc[1]);
                        acc[2] = fmaf(qq.z, s[i + 2], acc[2]), acc[3] = fmaf(qq.w, s[i + 3], acc[3]);
                    }
                }
                if (!FOLD) s_o[t][grp][col] = (acc[0] + acc[1]) + (acc[2] + acc[3]);
            };
            auto scale = [&](Factor f) {
#pragma unroll
                for (int i = 0; i < R; ++i) s[i] = s[i] * f;
            };
            if (block == kTile && tb + kTile < to) {
                // a whole tile in one block, with more to come: nothing to ask between its tokens
#pragma unroll 4
                for (int t = 0; t < kTile; ++t) token(t);
                scale(whole);
            } else {
                for (int t = 0; t < m; ++t) {
                    token(t);
                    const int e = t & (block - 1);
                    const bool last = tb + t == to - 1;
                    if (last || e == block - 1) {
                        // after the last token a forward state is S, not g S
                        const int power = last && !a.reverse ? e : e + 1;
                        scale(power == block ? whole : Factor{decay_pow(ld, power), 0.0f});
                    }
                }
            }
            if (!FOLD) {
                __syncthreads();
                for (int t = grp; t < m; t += kGroups) {
                    const float x = (s_o[t][0][col] + s_o[t][1][col]) + (s_o[t][2][col] + s_o[t][3][col]);
                    if (live) o[addr(tb + t) * a.o_tok + c0 + col] = from_f<T>(x * s_w[t]);
                }
            }
        }
    };

    int64_t n = first_sequence<kThreads>(a, w, t0, &s_count);
    if (!FOLD) griddep_wait();  // the carries; and nothing is written before
    if (FOLD) {
        // the sequence that crosses the window's end
        while (n < a.seqs && offset_at(a, n + 1) <= t1) ++n;
        const int64_t begin = n < a.seqs ? offset_at(a, n) : t1;
        const int32_t kind = begin >= t1 ? kNone : (begin >= t0 ? kFresh : kThrough);
        if (threadIdx.x == 0 && h == 0 && c0 == 0) a.tail[w] = kind;
        if (kind == kNone) return;
        load_state(kind == kFresh && a.s_in ? a.s_in + seq_state(n) : nullptr, a.s_in_t);
        if (a.stash && kind == kFresh) store_state(a.stash + (w * a.heads + h) * ssize);
        walk(begin > t0 ? begin : t0, t1);
        store_state(a.carry + (w * a.heads + h) * ssize);
        return;
    }
    int64_t at = t0;
    for (; n < a.seqs; ++n) {
        const int64_t begin = offset_at(a, n), end = offset_at(a, n + 1);
        if (a.by_seq ? n > w : begin >= t1 && w != a.windows - 1) break;
        if (begin > at) blank(at, begin < t1 ? begin : t1);
        const bool before = begin < t0;  // never, by sequence
        const int64_t from = before ? t0 : begin, to = end < t1 ? end : t1;
        if (before) load_state(a.carry + (w * a.heads + h) * ssize, a.carry_t);
        else if (a.stash && end > t1) load_state(a.stash + (w * a.heads + h) * ssize, false);
        else load_state(a.s_in ? a.s_in + seq_state(n) : nullptr, a.s_in_t);
        if (from < to) walk(from, to);
        if (end <= t1 && a.s_out) store_state(a.s_out + seq_state(n));
        if (to > at) at = to;
        if (end > t1) break;
    }
    if (at < t1) blank(at, t1);
}

// ---------------------------------------------------------------------------
// join of the windows' states
// ---------------------------------------------------------------------------
// carry[w] holds window w's last piece folded from its own start (or zero);
// on return it holds the state before window w. One thread takes E values of
// the state and walks the windows; kAhead loads are in flight before the
// chain needs them.
constexpr int kAhead = 16;

template <int E>
__global__ void __launch_bounds__(128) k_join(const __grid_constant__ Batch batch) {
    const Args& a = batch.a[blockIdx.y];
    const int64_t i = (int64_t)blockIdx.x * 128 + threadIdx.x;
    griddep_launch_dependents();
    const int64_t n = (int64_t)a.heads * a.dk * a.dv / E;
    if (i >= n) return;
    const int64_t per_head = (int64_t)a.dk * a.dv / E;
    const Factor g = decay_factor(a.log_decay[i / per_head], (int)a.window);
    griddep_wait();
    Raw<4 * E>* c = reinterpret_cast<Raw<4 * E>*>(a.carry) + i;
    Raw<4 * E> run = {};
    int32_t before = kNone;  // tail of the window before: kNone, and nothing reads the window's state
    for (int64_t w0 = 0; w0 < a.windows; w0 += kAhead) {
        Raw<4 * E> u[kAhead];
        int32_t kind[kAhead];
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            // (a slot that no fold wrote is read as well, and not used)
            const bool in = w0 + j < a.windows;
            kind[j] = in ? a.tail[w0 + j] : (int32_t)kNone;
            if (in) u[j] = c[(w0 + j) * n];
        }
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
            if (before != kNone) c[(w0 + j) * n] = run;
            before = kind[j];
            if (kind[j] == kFresh) run = u[j];
            if (kind[j] == kThrough)
#pragma unroll
                for (int e = 0; e < E; ++e)
                    run.w[e] = __float_as_uint(__uint_as_float(run.w[e]) * g + __uint_as_float(u[j].w[e]));
        }
    }
}

ak_status launch_join(const Batch& b, cudaStream_t stream) {
    const Args& a = b.a[0];
    const int64_t n = (int64_t)a.heads * a.dk * a.dv;
    const bool four = (int64_t)a.dk * a.dv % 4 == 0;
    const dim3 grid((unsigned)((n / (four ? 4 : 1) + 127) / 128), (unsigned)b.folds);
    return launch_behind(four ? k_join<4> : k_join<1>, grid, 128, 0, stream, b);
}

template <class T, int DK>
ak_status launch_tokens(const Batch& b, cudaStream_t stream) {
    const Args& a = b.a[0];
    const int dv = std::max(a.dv, b.count > 1 ? a.dk : 0);
    dim3 grid((unsigned)a.windows, (unsigned)a.heads, (unsigned)((dv + 31) / 32 * b.folds));
    const bool fold = a.windows > 1 && !a.by_seq;
    if (fold) {
        k_tokens<T, DK, true><<<grid, kThreads, 0, stream>>>(b);
        count_launches(1);
        ak_status s = check_launch();
        if (s == AK_OK) s = launch_join(b, stream);
        if (s != AK_OK) return s;
    }
    grid.z = (unsigned)((dv + 31) / 32 * b.count);
    if (fold) return launch_behind(k_tokens<T, DK, false>, grid, kThreads, 0, stream, b);
    k_tokens<T, DK, false><<<grid, kThreads, 0, stream>>>(b);
    count_launches(1);
    return check_launch();
}

template <class T>
ak_status launch_tokens_of(const Batch& b, cudaStream_t stream) {
    const int dk = std::max(b.a[0].dk, b.count > 1 ? b.a[0].dv : 0);
    if (dk <= 32) return launch_tokens<T, 32>(b, stream);
    if (dk <= 64) return launch_tokens<T, 64>(b, stream);
    if (dk <= 96) return launch_tokens<T, 96>(b, stream);
    if (dk <= 128) return launch_tokens<T, 128>(b, stream);
    return launch_tokens<T, 256>(b, stream);
}

// ---------------------------------------------------------------------------
// one token
// ---------------------------------------------------------------------------
// S = g S + k v^T; o = scale S^T q, the state updated in place: it is read
// and written once, which is all the traffic that counts. A block takes a
// request, a head and `cols` columns; a warp's lanes take four columns each
// of kStepRows rows in flight, and the rows' parts of o meet in shared
// memory. 256 requests, 32 heads of 128: 160 us, 6.7 TB/s; one request, 16
// heads: 2.9 us (a launch and two dependent loads).
constexpr int kStepThreads = 256;
constexpr int kStepRows = 8;  // rows a thread has in flight

struct StepArgs {
    const void *q, *k, *v;
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head, o_tok, o_head;
    void* o;
    const float* log_decay;
    float* state;
    const int32_t* slots;
    int64_t nslots;
    int heads, dk, dv, cols;
    float scale;
};

// VEC: dv is a multiple of 4 and the state 16-byte aligned.
template <class T, bool VEC>
__global__ void __launch_bounds__(kStepThreads) k_step(const StepArgs a) {
    constexpr int E = VEC ? 4 : 1;
    extern __shared__ float s_part[];  // [groups][cols], then k[dk], q[dk]
    const int64_t b = blockIdx.x;
    const int h = blockIdx.y;
    const int c0 = blockIdx.z * a.cols;
    const int cols = min(a.cols, a.dv - c0);
    const int lanes = a.cols / E;              // threads across the columns
    const int groups = kStepThreads / lanes;   // rows side by side
    float* s_k = s_part + groups * a.cols;
    float* s_q = s_k + a.dk;
    const int64_t slot = a.slots ? (int64_t)a.slots[b] : b;
    const int x = threadIdx.x % lanes, g = threadIdx.x / lanes;
    T* o = static_cast<T*>(a.o) + b * a.o_tok + h * a.o_head + c0;
    if (slot < 0 || slot >= a.nslots) {  // a padding entry
        for (int i = threadIdx.x; i < cols; i += kStepThreads) o[i] = from_f<T>(0.0f);
        return;
    }
    const bool live = g < groups && x * E < cols;
    float* s = a.state + (slot * a.heads + h) * ((int64_t)a.dk * a.dv) + c0 + x * E;
    const Factor w = decay_factor(a.log_decay[h], 1);
    float st[kStepRows][E];
    // the first rows are in flight while k, q and v arrive
    auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kStepRows; ++i) {
            const int r = r0 + i * groups;
            if (live && r < a.dk) {
                if constexpr (VEC) *reinterpret_cast<float4*>(st[i]) = *reinterpret_cast<const float4*>(s + (int64_t)r * a.dv);
                else st[i][0] = s[(int64_t)r * a.dv];
            }
        }
    };
    load(g);
    const T* q = static_cast<const T*>(a.q) + b * a.q_tok + h * a.q_head;
    const T* k = static_cast<const T*>(a.k) + b * a.k_tok + h * a.k_head;
    const T* v = static_cast<const T*>(a.v) + b * a.v_tok + h * a.v_head + c0;
    for (int i = threadIdx.x; i < a.dk; i += kStepThreads) {
        s_k[i] = as_f(k[i]);
        s_q[i] = as_f(q[i]);
    }
    float vv[E], acc[E];
#pragma unroll
    for (int j = 0; j < E; ++j) {
        vv[j] = live ? as_f(v[x * E + j]) : 0.0f;
        acc[j] = 0.0f;
    }
    __syncthreads();
    for (int r0 = g; r0 < a.dk; r0 += groups * kStepRows) {
        if (r0 != g) load(r0);
#pragma unroll
        for (int i = 0; i < kStepRows; ++i) {
            const int r = r0 + i * groups;
            if (live && r < a.dk) {
                const float kk = s_k[r], qq = s_q[r];
#pragma unroll
                for (int j = 0; j < E; ++j) {
                    st[i][j] = fmaf(st[i][j], w.hi, fmaf(st[i][j], w.lo, kk * vv[j]));
                    acc[j] = fmaf(qq, st[i][j], acc[j]);
                }
                if constexpr (VEC) *reinterpret_cast<float4*>(s + (int64_t)r * a.dv) = *reinterpret_cast<const float4*>(st[i]);
                else s[(int64_t)r * a.dv] = st[i][0];
            }
        }
    }
    if (g < groups) {
#pragma unroll
        for (int j = 0; j < E; ++j) s_part[g * a.cols + x * E + j] = acc[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < cols; i += kStepThreads) {
        float r = 0.0f;
        for (int j = 0; j < groups; ++j) r += s_part[j * a.cols + i];
        o[i] = from_f<T>(r * a.scale);
    }
}

template <class T>
ak_status launch_step(const StepArgs& a, int64_t batch, bool vec, cudaStream_t stream) {
    const int lanes = a.cols / (vec ? 4 : 1);
    const size_t smem = ((size_t)(kStepThreads / lanes) * a.cols + 2 * (size_t)a.dk) * 4;
    const dim3 grid((unsigned)batch, (unsigned)a.heads, (unsigned)((a.dv + a.cols - 1) / a.cols));
    if (vec) k_step<T, true><<<grid, kStepThreads, smem, stream>>>(a);
    else k_step<T, false><<<grid, kStepThreads, smem, stream>>>(a);
    count_launches(1);
    return check_launch();
}

}  // namespace la

// How the token axis is divided among blocks.
struct Division {
    bool by_seq, ranked;
    int64_t window, windows;
};

// `slots`: blocks that run at a time; `lanes`: blocks that a window takes
// (heads, calls of the launch, column slices). One wave of equal windows
// leaves no block waiting for a last one, and longer windows have fewer
// states to pass on. By sequence there is no fold of window states and no
// join, but the longest sequence, or the last ones to start, set the time:
// that is taken where it ends sooner. Times are estimated in steps of 64
// tokens. Fold and join cost half of the main pass where it is long (32771
// tokens, 16 heads of 128: 52 and 10 us beside 123) and more where it is
// short: 0.7 of the work over all, and `fixed` steps of launches and join, 6
// of the chunk kernel's (2.5 us) or 4 of the token kernel's (10 us).
// Both sides measured at 102 shapes (8 to 64 heads, 2 to 300 sequences, 4096 to
// 19200 tokens, bf16 heads of 64 and 128 and float32 of 64, forward and
// backward), us by sequence / by windows:
//   bf16, 32 heads of 128, 16 sequences, 16384 tokens   145 / 176
//   the same of 8 sequences                             184 / 187
//   the same of 2 sequences, 4096 tokens                154 / 68
//   bf16, 8 heads of 64, 16 sequences, 8192 tokens      33 / 42
//   float32, 64 heads of 64, 2 sequences, 4096 tokens   388 / 555
// The faster one is taken, or one within 3 % of it, at 94 of them; the others
// lose 4 to 6 %, and 19 and 23 % backward over 300 sequences, which blocks do
// not sort. (With 1.35 of the work and 4 steps for both kernels 12 lost, by up
// to 43 %; with 6 steps for the token kernel 2049 tokens of 5 sequences, 8 heads
// of 80, took 120 us by sequence in place of 88 by windows.)
constexpr int64_t kMaxWindows = 65535;  // a grid's second extent

static Division divide(const LinattnCall& c, int64_t slots, int64_t lanes, int fixed) {
    const int64_t unit = 64;
    Division d = {};
    const int64_t units = std::max<int64_t>(1, (c.tokens + unit - 1) / unit);
    int64_t want = c.windows > 0 ? c.windows : slots / lanes;
    want = std::max<int64_t>(1, std::min({want, units, kMaxWindows}));
    const int64_t per = (units + want - 1) / want;
    d.window = per * unit;
    d.windows = std::max<int64_t>(1, (c.tokens + d.window - 1) / d.window);
    if (c.windows > 0 || c.seqs < 2 || c.seqs > kMaxWindows) return d;
    const double work = (double)(units + c.seqs) * lanes / slots;  // steps of 64 tokens, spread evenly
    const double longest = (double)((c.max_len + unit - 1) / unit);
    // (the longest start first, see linattn_mma.cu; unsorted, a long one may start last)
    const double seq_steps = std::max(longest, work + (c.seqs <= la::kRanked ? 0.15 : 0.5) * longest);
    const double window_steps = d.windows == 1 ? (double)(units + c.seqs) * std::max<int64_t>(1, lanes / slots)
                                               : std::max(1.7 * work, (double)per) + fixed;
    if (seq_steps <= window_steps) {
        d.by_seq = true;
        // (sorting takes a block about 2 us, which a few chunks do not earn back)
        d.ranked = c.seqs <= la::kRanked && longest > 4;
        d.windows = c.seqs;
    }
    return d;
}

static int64_t token_slices(int dv) { return (dv + 31) / 32; }

// Divisions of the two kernels (the pointers decide between them later).
static Division divide_chunks(const LinattnCall& c, const DeviceInfo& dev, int calls) {
    return divide(c, 2 * dev.sm_count, (int64_t)c.heads * calls, 6);
}
static Division divide_tokens(const LinattnCall& c, const DeviceInfo& dev, int calls) {
    return divide(c, 3 * dev.sm_count, (int64_t)c.heads * calls * token_slices(std::max(c.dk, c.dv)), 4);
}

static size_t carry_bytes(const LinattnCall& c, const Division& d, int calls) {
    if (d.by_seq || d.windows == 1) return 0;
    const size_t state = (size_t)c.heads * c.dk * c.dv * 4;
    // one call may work in place and keeps its initial states beside the carries
    return calls * align_up((size_t)d.windows * 4, 256) + (calls == 1 ? 2 : calls) * align_up((size_t)d.windows * state, 256);
}

size_t linattn_workspace(const LinattnCall& c, const DeviceInfo& dev) {
    size_t most = 0;
    for (int calls = 1; calls <= la::kMaxCalls; calls += 2) {  // the forward pass, the backward pass
        if (c.dtype == AK_BF16 && c.dk == c.dv && (c.dk == 64 || c.dk == 128))
            most = std::max(most, carry_bytes(c, divide_chunks(c, dev, calls), calls));
        most = std::max(most, carry_bytes(c, divide_tokens(c, dev, calls), calls));  // rows that TMA cannot take
    }
    return kWsHeader + most;
}

static la::Args args_of(const LinattnCall& c) {
    la::Args a = {};
    a.log_decay = c.log_decay;
    a.offsets = c.offsets;
    a.tokens = c.tokens;
    a.seqs = c.seqs;
    a.heads = c.heads;
    return a;
}

static void roles(la::Args& a, const ak_heads& q, const ak_heads& k, const ak_heads& v, const ak_heads& o, int dk, int dv) {
    a.q = q.data, a.q_tok = q.token_stride, a.q_head = q.head_stride;
    a.k = k.data, a.k_tok = k.token_stride, a.k_head = k.head_stride;
    a.v = v.data, a.v_tok = v.token_stride, a.v_head = v.head_stride;
    a.o = o.data, a.o_tok = o.token_stride, a.o_head = o.head_stride;
    a.dk = dk, a.dv = dv;
}

static void log_batch(const la::Batch& b, const LinattnCall& c, const char* kernel) {
    if (!log_on()) return;
    const la::Args& a = b.a[0];
    log_call("linear_attention%s tokens=%lld seqs=%lld heads=%d dk=%d dv=%d in=%s: %s, %lld %s", b.count > 1 ? "_backward" : "",
             (long long)c.tokens, (long long)c.seqs, c.heads, c.dk, c.dv, c.dtype == AK_F32 ? "f32" : "bf16", kernel,
             (long long)a.windows, a.by_seq ? "sequence(s), a block each" : a.windows > 1 ? "windows (fold, join, main)" : "window");
}

static ak_status run_batch(la::Batch& b, const LinattnCall& c, const DeviceInfo& dev, void* ws, cudaStream_t s) {
    auto place = [&](const Division& d) {
        char* w = static_cast<char*>(ws) + kWsHeader;
        for (int i = 0; i < b.count; ++i) {
            la::Args& a = b.a[i];
            a.by_seq = d.by_seq, a.ranked = d.ranked, a.window = d.window, a.windows = d.windows;
            a.tail = reinterpret_cast<int32_t*>(w);
            w += align_up((size_t)d.windows * 4, 256);
            a.carry = reinterpret_cast<float*>(w);
            w += align_up((size_t)d.windows * c.heads * c.dk * c.dv * 4, 256);
            a.stash = nullptr;
        }
        // the third call of the backward pass folds the transposes of the second's states
        if (b.count == 3) b.a[2].carry = b.a[1].carry, b.a[2].tail = b.a[1].tail, b.a[2].carry_t = true;
        // the backward pass has room for three carries and never works in place
        la::Args& a = b.a[0];
        if (b.count == 1 && a.s_in && a.s_in == a.s_out && !d.by_seq && d.windows > 1) a.stash = reinterpret_cast<float*>(w);
    };
    bool chunks = true;
    for (int i = 0; i < b.count; ++i) chunks = chunks && la::mma_takes(b.a[i], c.dtype);
    if (chunks) {
        place(divide_chunks(c, dev, b.count));
        const ak_status r = la::launch_chunks(b, static_cast<uint64_t*>(ws), c.epoch, (uint64_t)c.wait_limit_ns, s);
        if (r != AK_ERR_UNSUPPORTED) {
            log_batch(b, c, "tensor-core chunks");
            return r;
        }
    }
    place(divide_tokens(c, dev, b.count));
    log_batch(b, c, "token by token");
    return c.dtype == AK_F32 ? la::launch_tokens_of<float>(b, s) : la::launch_tokens_of<bf16>(b, s);
}

ak_status run_linattn(const LinattnCall& c, void* ws, cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    la::Batch b = {};
    b.count = b.folds = 1;
    la::Args& a = b.a[0];
    a = args_of(c);
    roles(a, c.q, c.k, c.v, c.o, c.dk, c.dv);
    a.s_in = c.state_in, a.s_out = c.state_out;
    a.out_scale = c.scale, a.in_scale = 1.0f;
    return run_batch(b, c, dev, ws, stream);
}

ak_status run_linattn_backward(const LinattnCall& c, void* ws, cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    la::Batch b = {};
    b.count = 3, b.folds = 2;
    for (la::Args& a : b.a) a = args_of(c);
    // dq = F(do, v, k) from the transposed initial state
    roles(b.a[0], c.o, c.v, c.k, c.dq, c.dv, c.dk);
    b.a[0].s_in = c.state_in, b.a[0].s_in_t = true;
    b.a[0].out_scale = c.scale, b.a[0].in_scale = 1.0f;
    // dv = R(k, q, do) from dS_T, leaving dS_0
    roles(b.a[1], c.k, c.q, c.o, c.dvv, c.dk, c.dv);
    b.a[1].s_in = c.dstate_out, b.a[1].s_out = c.dstate_in;
    // dk = R(v, do, q) from dS_T transposed
    roles(b.a[2], c.v, c.o, c.q, c.dk_out, c.dv, c.dk);
    b.a[2].s_in = c.dstate_out, b.a[2].s_in_t = true;
    for (int i = 1; i < 3; ++i) b.a[i].reverse = true, b.a[i].out_scale = 1.0f, b.a[i].in_scale = c.scale;
    return run_batch(b, c, dev, ws, stream);
}

ak_status run_linattn_step(const LinattnCall& c, float* state, const int32_t* slots, int64_t nslots,
                           cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    la::StepArgs a = {};
    a.q = c.q.data, a.q_tok = c.q.token_stride, a.q_head = c.q.head_stride;
    a.k = c.k.data, a.k_tok = c.k.token_stride, a.k_head = c.k.head_stride;
    a.v = c.v.data, a.v_tok = c.v.token_stride, a.v_head = c.v.head_stride;
    a.o = c.o.data, a.o_tok = c.o.token_stride, a.o_head = c.o.head_stride;
    a.log_decay = c.log_decay;
    a.state = state, a.slots = slots, a.nslots = nslots;
    a.heads = c.heads, a.dk = c.dk, a.dv = c.dv, a.scale = c.scale;
    const bool vec = c.dv % 4 == 0 && reinterpret_cast<uintptr_t>(state) % 16 == 0;
    a.cols = 32;
    while (a.cols < c.dv && a.cols < 256) a.cols *= 2;
    // fewer blocks than SMs: narrower column slices (128 bytes a row at least)
    while (a.cols > 32 && c.tokens * c.heads * ((c.dv + a.cols - 1) / a.cols) < 2 * dev.sm_count) a.cols /= 2;
    if (log_on())
        log_call("linear_attention_step requests=%lld heads=%d dk=%d dv=%d: %d columns a block", (long long)c.tokens, c.heads,
                 c.dk, c.dv, a.cols);
    return c.dtype == AK_F32 ? la::launch_step<float>(a, c.tokens, vec, stream)
                             : la::launch_step<bf16>(a, c.tokens, vec, stream);
}

}  // namespace ak
