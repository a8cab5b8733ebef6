// linattn.cuh -- linear attention with a decay for each head: the scan whose
// state is a matrix.
//
//   S_t = g S_{t-1} + k_t v_t^T   (dk x dv, float32),   o_t = scale S_t^T q_t,   g = exp(log_decay[h])
//
// Gradients are the same operator with its roles exchanged:
//   dq = F(do, v, k) from S_0^T;  dv = R(k, q, do) from dS_T;  dk = R(v, do, q) from dS_T^T
// where R runs time backwards and dS_t = g dS_{t+1} + scale q_t do_t^T. In R
// the carried state X_t = g dS_t has decayed once more on leaving a token
// and once less on entering it (`shift` = 1), which makes the last X the
// gradient of the initial state.
//
// A forward call keeps S, a reversed one X.
//
// Work along the token axis. The packed axis is cut into `windows` of
// `window` tokens, whatever the sequences' lengths; a block takes one window
// and one head and walks the pieces of sequences in it. With more than one
// window the scan takes three launches, like this library's long-line scans:
// a fold of each window's last piece into its state, a join of the windows'
// states along the axis, and the main pass from the joined states. Where the
// sequences are many and even, a block takes a sequence instead (by_seq), and
// the main pass is all there is. The backward pass runs its three calls side
// by side in the same launches (Batch). Positions
// below are primed: token t' = T - 1 - t and sequence n' = N - 1 - n in a
// reversed call, so both directions share every line of this logic.
#pragma once

#include "ak_common.cuh"
#include "ak_internal.h"

namespace ak {
namespace la {

// A window's last piece and what it means for the next window's start:
// kNone: no sequence crosses the window's end; kFresh: it began inside the
// window; kThrough: the whole window belongs to it.
enum Tail : int32_t { kNone = 0, kFresh = 1, kThrough = 2 };

struct Args {
    const void *q, *k, *v;
    int64_t q_tok, q_head, k_tok, k_head, v_tok, v_head;  // element strides
    void* o;
    int64_t o_tok, o_head;
    const float* log_decay;
    const int32_t* offsets;  // N + 1, or null: one sequence of T tokens
    int64_t tokens, seqs;
    int heads, dk, dv;       // of the roles (dk = rows of the state, dv = columns)
    const float* s_in;       // [N][H][dk][dv] ([dv][dk] when s_in_t), or null
    float* s_out;            // [N][H][dk][dv], or null
    bool s_in_t;
    bool reverse;
    float out_scale, in_scale;
    bool by_seq;             // block w takes sequence w; windows = seqs
    bool ranked;             // block w takes the w-th longest sequence
    int64_t window, windows;
    float* carry;            // [windows][H][dk * dv]
    bool carry_t;            // the carry is another call's, transposed
    int32_t* tail;           // [windows]
    // states written in place (s_out == s_in): the fold pass keeps here what
    // the main pass needs after another block may have overwritten it, the
    // initial states of sequences that begin in a window and leave it
    float* stash;            // as carry, or null
};

// Calls of one launch: the same tokens, heads and windows.
constexpr int kMaxCalls = 3;
constexpr int kRanked = 256;  // sequences that blocks sort by length
struct Batch {
    Args a[kMaxCalls];
    int count;
    int folds;  // of them, from the first, have a fold and a join of their own
};

// Launches `kernel` so that it may start while the launch before it still
// runs: until griddep_wait() it touches nothing of that one's. A fold pass, the
// join and the main pass follow each other this way.
template <class K, class A>
inline ak_status launch_behind(K kernel, dim3 grid, int threads, size_t smem, cudaStream_t stream, const A& arg) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, arg);
    if (e != cudaSuccess) return cuda_fail(e);
    count_launches(1);
    return check_launch();
}

__device__ __forceinline__ int64_t offset_at(const Args& a, int64_t n) {
    if (!a.offsets) return n == 0 ? 0 : a.tokens;
    const int64_t m = a.reverse ? a.seqs - n : n;
    int64_t x = a.offsets[m];
    x = x < 0 ? 0 : (x > a.tokens ? a.tokens : x);
    return a.reverse ? a.tokens - x : x;
}

// g^n: 1 for n = 0 whatever the decay (a decay of zero keeps its own token).
// The rounding of ld * n would shift the exponent by up to |ld n| 2^-24; its
// remainder is put back to first order.
__device__ __forceinline__ float decay_pow(float ld, int64_t n) {
    if (n == 0) return 1.0f;
    const float m = (float)n, x = ld * m, r = expf(x);
    return isinf(x) ? r : fmaf(r, fmaf(ld, m, -x), r);
}

// g^n as a sum of two floats. A factor that multiplies the state again and
// again must not carry a rounding of its own: with a slow decay (memory of M
// factors) a relative error e in it grows to M e in the state. M is about
// 1 / |x| with x = ld n, and 1 + expm1(x) is good to |x| 2^-23; a fast decay
// forgets the error with the rest.
struct Factor {
    float hi, lo;
};
__device__ __forceinline__ Factor decay_factor(float ld, int n) {
    const float x = n == 0 ? 0.0f : ld * (float)n;
    Factor f;
    f.hi = fabsf(x) < 0.5f ? 1.0f : decay_pow(ld, n);
    f.lo = fabsf(x) < 0.5f ? expm1f(x) : 0.0f;
    return f;
}
__device__ __forceinline__ float operator*(float s, Factor f) { return fmaf(s, f.hi, s * f.lo); }

// First and last + 1 token of block w.
__device__ __forceinline__ void block_span(const Args& a, int64_t w, int64_t* t0, int64_t* t1) {
    if (a.by_seq) {  // the blocks at the ends also take what lies outside every sequence
        *t0 = w == 0 ? 0 : offset_at(a, w);
        *t1 = w == a.windows - 1 ? a.tokens : offset_at(a, w + 1);
    } else {
        *t0 = w * a.window;
        *t1 = w == a.windows - 1 ? a.tokens : *t0 + a.window;
    }
}

// The first sequence with tokens at or after t0, or that is empty at or
// after t0. All threads of the block take part.
template <int THREADS>
__device__ __forceinline__ int64_t first_sequence(const Args& a, int64_t w, int64_t t0, int64_t* s_count) {
    if (a.by_seq) return w;
    if (!a.offsets || t0 == 0) return 0;
    int64_t c = 0;
    for (int64_t n = threadIdx.x; n < a.seqs; n += THREADS)
        c += offset_at(a, n) < t0 && offset_at(a, n + 1) <= t0;
    __syncthreads();
    if (threadIdx.x == 0) *s_count = 0;
    __syncthreads();
    for (int d = kWarp / 2; d > 0; d >>= 1) c += __shfl_down_sync(0xffffffffu, c, d);
    if (threadIdx.x % kWarp == 0 && c) atomicAdd(reinterpret_cast<unsigned long long*>(s_count), (unsigned long long)c);
    __syncthreads();
    return *s_count;
}

// linattn.cu
ak_status launch_join(const Batch& b, cudaStream_t stream);
// linattn_mma.cu
bool mma_takes(const Args& a, ak_dtype dtype);
ak_status launch_chunks(const Batch& b, uint64_t* error_word, uint64_t epoch, uint64_t wait_limit_ns,
                        cudaStream_t stream);

}  // namespace la
}  // namespace ak
