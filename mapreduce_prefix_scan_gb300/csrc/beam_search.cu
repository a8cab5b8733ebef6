// beam_search.cu -- the step of a beam search over all beams and the
// vocabulary, and the reordering of states by its parents.
//
// Request r has beams of summed log probabilities s_k and logits x_k(v). Its
// candidates are
//   s_k + x_k(v) - log sum_w exp x_k(w)   for a beam that goes on
//   s_k, as token `end`                   for one that has ended
// ranked by their value over length^penalty; the best `keep` follow, ties by
// the lowest beam, then token.
//
// Within a beam the order of candidates is that of its logits, so one pass
// over a row gives its sum and its best `keep` logits, and the request's
// answer is among them. A cluster of blocks takes a request, a block a row
// or a slice of one at a time:
//  - pass: each thread folds its columns (16 bytes of them, then those kThreads
//    times as far on, three or four such groups in flight) to a maximum, its column and a
//    sum of exponentials; no list is kept beside it, so an element costs a
//    conversion, a maximum, an exponential and three halves of packed pairs;
//  - the `keep`-th best of the threads' maxima is a bound below which nothing
//    can be chosen, and only the (at most `keep`) threads whose maximum
//    reaches it hold candidates: their columns are read once more, from L2 (with
//    the least of the warps' maxima for a bound, found sooner, 20 threads hold
//    candidates for 8 beams, and 64 x 8 rows of 128000 take 58 us, not 44);
//  - lists of 32 lie in the lanes of a warp and are merged as bitonic
//    sequences; the cluster's first block merges the rows.
// Keys order by (logit, lowest column), so the answer does not depend on the
// order in which threads find them.
//
// Decisions lie next to one another: logits differ by little, and so do the
// beams' sums. Sums of exponentials are float32 with a running compensation,
// the logarithm, the totals and the ranks are 64-bit (a few for each row: the
// device adds 64-bit numbers 64 times slower than 32-bit ones). What is left is the
// exponentials' own error, 2^-22 and d 2^-22.8 at d below the largest logit, and their
// sums' in groups of 16 bytes: logarithms of 32003 to 262144 logits were off by 1e-8 to 8e-8 in the
// mean, 1.7e-7 at most, and 2.3e-7 in rows that rise, where every group has a larger logit
// and the sum is scaled each time. Only a choice between beams that near can turn on it.
//
// Bound by HBM and the exponentials while rows are folded (0.78 of the copy
// bandwidth with four rows an SM) and by a chain of latencies after them (about 10 us:
// the block's sort, the candidates' loads, the cluster's exchange, the logarithms,
// the ranks, the merge). Back to back: 64 x 8 rows of 128000 bf16 43 to 46 us, 32 x 8
// float32 35 us (0.55), 4 rows of 32003 float32 11.4 us. Blocks of 128 threads: 52, 53
// and 13 us, of 512: 51, 34 and 12; rows in twice as many slices: 58, 35 and 12; three
// blocks an SM with eight groups in flight: 87, 37 and 11.
// The reordering of 8 x 64 x 8 states of 2048 float32 takes 6.9 us.
#include <algorithm>
#include <cooperative_groups.h>

#include "ak_common.cuh"
#include "ak_internal.h"

namespace cg = cooperative_groups;

namespace ak {
namespace bs {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / kWarp;
constexpr int kMaxBeams = 32;     // of a request, before and after: a list is a warp
// candidates held at a time: all of a group (16 bytes, 8 bf16) a thread, which may be candidates every one
constexpr int kFound = kThreads * 8;

// Orders floats as unsigned integers; -0 and 0 are one value.
__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t o) {
    return __uint_as_float(o & 0x80000000u ? o & 0x7fffffffu : ~o);
}
__device__ __forceinline__ uint64_t ordered(double x) {
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}

// A logit and its column; larger is better, 0 is none.
__device__ __forceinline__ uint64_t key_of(float x, uint32_t col) {
    return x > -INFINITY ? (uint64_t)ordered(x) << 32 | (0xffffffffu - col) : 0;
}

// What the merge of the rows sorts: the rank, then the lowest beam and its own order.
struct Pick {
    uint64_t rank;   // 0: none
    uint32_t place;  // ~(beam * 32 + place in its list)
};

__device__ __forceinline__ bool over(uint64_t a, uint64_t b) { return a > b; }
__device__ __forceinline__ bool over(const Pick& a, const Pick& b) {
    return a.rank > b.rank || (a.rank == b.rank && a.place > b.place);
}
__device__ __forceinline__ uint64_t from_lane(uint64_t v, int mask) { return __shfl_xor_sync(0xffffffffu, v, mask); }
__device__ __forceinline__ Pick from_lane(const Pick& v, int mask) {
    Pick o;
    o.rank = __shfl_xor_sync(0xffffffffu, v.rank, mask);
    o.place = __shfl_xor_sync(0xffffffffu, v.place, mask);
    return o;
}

// Of this lane's and another's value the larger (or the smaller).
template <class K>
__device__ __forceinline__ void exchange(K& v, int mask, bool larger) {
    const K o = from_lane(v, mask);
    if (over(o, v) == larger) v = o;
}

// Lanes 0 .. 31 in decreasing order.
template <class K>
__device__ __forceinline__ void warp_sort(K& v, int lane) {
#pragma unroll
    for (int k = 2; k <= kWarp; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) exchange(v, j, ((lane & k) == 0) == ((lane & j) == 0));
}

// The best 32 of two lists in decreasing order, `o` given reversed (lane 31's first).
template <class K>
__device__ __forceinline__ void warp_merge(K& v, const K& reversed, int lane) {
    if (over(reversed, v)) v = reversed;
#pragma unroll
    for (int j = kWarp / 2; j > 0; j >>= 1) exchange(v, j, (lane & j) == 0);
}

// Adds 32 values in any order to a list.
template <class K>
__device__ __forceinline__ void warp_take(K& list, K v, int lane) {
    warp_sort(v, lane);
    warp_merge(list, from_lane(v, kWarp - 1), lane);
}

// Warp 0's list becomes the best 32 of the first `warps` warps' lists (a power of
// two). Ends in the block's sync, but for one warp: that has nothing to wait for here.
template <class K>
__device__ __forceinline__ void block_merge(K& list, K (*s_lists)[kWarp], int lane, int warp, int warps = kWarps) {
    for (int half = warps / 2; half > 0; half >>= 1) {
        if (warp >= half && warp < 2 * half) s_lists[warp][lane] = list;
        __syncthreads();
        if (warp < half) warp_merge(list, s_lists[warp + half][kWarp - 1 - lane], lane);
        __syncthreads();
    }
}

// 16 bytes of a row.
template <class T>
struct alignas(16) Group {
    static constexpr int kSize = 16 / (int)sizeof(T);
    uint32_t w[4];
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
        else return __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
    }
};

// Columns [col, col + kSize) of a row, -infinity from column `end` on. The columns of
// a group are the same whatever the row's alignment: equal rows give equal sums.
template <class T>
__device__ __forceinline__ Group<T> load_group(const T* row, uint64_t col, uint32_t end, bool wide) {
    constexpr int G = Group<T>::kSize;
    Group<T> g;
    if (wide && col + G <= end) {
        asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
            : "=r"(g.w[0]), "=r"(g.w[1]), "=r"(g.w[2]), "=r"(g.w[3]) : "l"(row + col));
        return g;
    }
    T v[G];
#pragma unroll
    for (int i = 0; i < G; ++i) v[i] = col + i < end ? row[col + i] : T(-INFINITY);
    memcpy(&g, v, sizeof g);
    return g;
}

// Two float32 sums or products at once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
__device__ __forceinline__ float low(uint64_t p) { return __uint_as_float((uint32_t)p); }
__device__ __forceinline__ float high(uint64_t p) { return __uint_as_float((uint32_t)(p >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A row's (or slice's) share of the answer, in the first block's shared memory.
struct Share {
    float top;         // the largest logit, or -infinity
    float sum, lost;   // of exp(x - top)
    uint64_t keys[kMaxBeams];
};

struct Shared {
    uint64_t lists[kWarps][kWarp];
    Pick picks[kWarps][kWarp];
    uint64_t found[kFound];
    int nfound, nchosen;
    int chosen[kMaxBeams];
    uint64_t bound;
    float tops[kWarps], sums[kWarps], losts[kWarps];
    double norm[kMaxBeams];   // length^penalty of a beam's candidates
    float score[kMaxBeams];   // (outputs may lie where these came from)
    int length[kMaxBeams];
    bool was[kMaxBeams];
    double base[kMaxBeams];   // minus the largest logit, minus log sum exp over it
    Share share[kMaxBeams];   // of the rows' slices (first block)
    float totals[kMaxBeams][kWarp];
    uint32_t tokens[kMaxBeams][kWarp];
};

constexpr float kLog2e = 1.4426950408889634f;

// sum += x with what rounding loses kept in `lost`.
__device__ __forceinline__ void add(float& sum, float& lost, float x) {
    const float t = sum + x, v = t - sum;
    lost += (sum - (t - v)) + (x - v);
    sum = t;
}

// Folds columns [first, last) of a row and writes its share.
template <class T>
__device__ void fold_row(const T* row, uint32_t first, uint32_t last, int keep, Shared& s, Share* out, bool& waited) {
    constexpr int G = Group<T>::kSize;
    constexpr uint64_t kStep = (uint64_t)kThreads * G;
    // groups in flight: what the registers of four blocks an SM leave. Four of bf16 (five runs of
    // either in turn, 64 x 8 x 128000, 32 x 8 x 152064, 128 x 4 x 262144, 4 x 16 x 128000): 44.6, 34.0, 69.3, 25.3 us,
    // three 42.9, 32.3, 67.1, 23.9, no two runs of which overlap
    constexpr int kAhead = sizeof(T) == 2 ? 3 : 4;
    const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
    const bool wide = (reinterpret_cast<uintptr_t>(row) & 15) == 0;
    float top = -INFINITY, ref = 0.0f, sum = 0.0f, lost = 0.0f;
    uint32_t at = 0;
    Group<T> next[kAhead];
    uint64_t c0 = first + (uint64_t)tid * G;
#pragma unroll
    for (int u = 0; u < kAhead; ++u) next[u] = load_group(row, c0 + u * kStep, last, wide);
    for (; c0 < last; c0 += kAhead * kStep) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const uint64_t col = c0 + u * kStep;
            float x[G];
#pragma unroll
            for (int i = 0; i < G; ++i) x[i] = next[u][i];
            next[u] = load_group(row, col + kAhead * kStep, last, wide);
            float m = x[0];
#pragma unroll
            for (int i = 1; i < G; ++i) m = fmaxf(m, x[i]);
            if (m > top) {
                const float f = exp2f((ref - m) * kLog2e);
                if (top > -INFINITY) sum *= f, lost *= f;
                top = ref = m;
                uint32_t i = 0;
#pragma unroll
                for (int j = G - 1; j >= 0; --j)
                    if (x[j] == m) i = j;
                at = (uint32_t)col + i;
            }
            const uint64_t less = pair(-ref, -ref), scale = pair(kLog2e, kLog2e);
            uint64_t e = 0;
#pragma unroll
            for (int i = 0; i < G; i += 2) {
                const uint64_t y = mul2(add2(pair(x[i], x[i + 1]), less), scale);
                const uint64_t z = pair(exp2_fast(low(y)), exp2_fast(high(y)));
                e = i == 0 ? z : add2(e, z);
            }
            add(sum, lost, low(e) + high(e));
        }
    }
    // ---- the block's maximum and sum; the threads' best, and the bound
    float best = top;
#pragma unroll
    for (int d = kWarp / 2; d > 0; d >>= 1) best = fmaxf(best, __shfl_xor_sync(0xffffffffu, best, d));
    if (lane == 0) s.tops[warp] = best;
    if (tid == 0) s.nchosen = 0;
    const uint64_t mine = key_of(top, at);
    uint64_t list = mine;
    warp_sort(list, lane);
    __syncthreads();
    best = s.tops[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) best = fmaxf(best, s.tops[w]);
    // (a NaN among the logits is in `sum` alone)
    const float f = top > -INFINITY ? exp2f((top - best) * kLog2e) : 1.0f;
    sum *= f, lost *= f;
#pragma unroll
    for (int d = kWarp / 2; d > 0; d >>= 1) {
        const float o = __shfl_xor_sync(0xffffffffu, sum, d), ol = __shfl_xor_sync(0xffffffffu, lost, d);
        lost += ol;
        add(sum, lost, o);
    }
    if (lane == 0) s.sums[warp] = sum, s.losts[warp] = lost;
    block_merge(list, s.lists, lane, warp);
    if (warp == 0) {
        const uint64_t b = __shfl_sync(0xffffffffu, list, keep - 1);
        if (lane == 0) s.bound = b;
    }
    __syncthreads();
    const uint64_t bound = s.bound;
    // (fewer than `keep` threads with a candidate: each of them is looked through)
    if (mine && mine >= bound) s.chosen[atomicAdd(&s.nchosen, 1)] = tid;
    __syncthreads();
    // ---- the chosen threads' columns again, 16 of them a thread at a time; where
    // more are candidates than there is room for, a group, for which there always is
    // (how many lie in few threads is the logits' affair: the bound leaves out
    // threads, not columns)
    static_assert(kThreads * G <= kFound, "a group of every thread has to fit");
    constexpr int kSome = 16 / G;
    const int chosen = s.nchosen;
    const uint32_t groups = (last - first + G - 1) / G, per = (groups + kThreads - 1) / kThreads;  // of a thread, at most
    const uint32_t all = per * (uint32_t)chosen;
    bool spread = false;  // more than warp 0 holds a list
    list = 0;
    for (uint32_t g0 = 0; g0 < all; g0 += kSome * kThreads) {
        Group<T> x[kSome];
        uint64_t col[kSome];
#pragma unroll
        for (int j = 0; j < kSome; ++j) {
            const uint32_t g = g0 + j * kThreads + tid;
            col[j] = g < all ? first + ((uint64_t)(g % per) * kThreads + s.chosen[g / per]) * G : last;
            x[j] = load_group(row, col[j], last, wide);
        }
        for (int only = -1; only < kSome; ++only) {
            if (tid == 0) s.nfound = 0;
            __syncthreads();
#pragma unroll
            for (int j = 0; j < kSome; ++j) {
                if (only >= 0 && only != j) continue;
#pragma unroll
                for (int i = 0; i < G; ++i) {
                    const uint64_t k = key_of(x[j][i], (uint32_t)col[j] + i);
                    if (k && k >= bound) {
                        const int to = atomicAdd(&s.nfound, 1);
                        if (to < kFound) s.found[to] = k;
                    }
                }
            }
            __syncthreads();
            const int n = s.nfound;
            if (n <= kFound) {
                spread |= n > kWarp;
                for (int b = warp * kWarp; b < n; b += kThreads) warp_take(list, b + lane < n ? s.found[b + lane] : uint64_t(0), lane);
            }
            __syncthreads();
            if (only < 0 && n <= kFound) break;
        }
    }
    if (spread) block_merge(list, s.lists, lane, warp);
    if (!waited) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");  // the first block runs
    waited = true;
    if (warp == 0) {
        out->keys[lane] = list;
        if (lane == 0) {
            sum = s.sums[0], lost = s.losts[0];
            for (int w = 1; w < kWarps; ++w) {
                lost += s.losts[w];
                add(sum, lost, s.sums[w]);
            }
            out->top = best;
            out->sum = sum;
            out->lost = lost;
        }
    }
    __syncthreads();
}

template <class T>
__global__ void __launch_bounds__(kThreads, 4) k_beam_select(const BeamCall c) {
    __shared__ Shared s;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), parts = (int)cl.num_blocks();
    const int64_t r = blockIdx.x / parts;
    const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
    const int n = c.beams, keep = c.keep, slices = c.slices;
    const float* scores = c.scores + r * n;
    const uint8_t* done = c.done ? c.done + r * n : nullptr;
    const int32_t* lengths = c.lengths ? c.lengths + r * n : nullptr;
    const uint32_t vocab = (uint32_t)c.vocab, slice = ((vocab + slices - 1) / slices + 7) / 8 * 8;

    if (parts > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    Shared* s0 = cl.map_shared_rank(&s, 0);
    if (rank == 0 && warp == kWarps - 1 && lane < n) {
        const bool was = done && done[lane];
        const int len = (lengths ? lengths[lane] : 0) + !was;
        s.score[lane] = scores[lane];
        s.was[lane] = was;
        s.length[lane] = len;
        s.norm[lane] = c.penalty == 1.0 || c.penalty == 0.0 ? (double)len : pow((double)len, c.penalty);
    }
    bool waited = parts == 1;
    for (int item = rank; item < n * slices; item += parts) {
        const int k = item / slices;
        const float sc = scores[k];
        if ((done && done[k]) || !(fabsf(sc) < INFINITY)) continue;  // no need of its logits
        const uint32_t first = min((uint64_t)(item % slices) * slice, (uint64_t)vocab), last = min(first + slice, vocab);
        fold_row(static_cast<const T*>(c.logits) + r * c.batch_stride + k * c.beam_stride, first, last, keep, s, &s0->share[item], waited);
    }
    if (!waited) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (parts > 1) cl.sync();
    else __syncthreads();
    if (rank != 0) return;

    // ---- the rows' logarithms
    if (tid < n) {
        const Share* h = s.share + tid * slices;
        float top = -INFINITY, sum = 0.0f, lost = 0.0f;
        for (int i = 0; i < slices; ++i) top = fmaxf(top, h[i].top);
        for (int i = 0; i < slices; ++i) {
            const float f = slices > 1 && h[i].top > -INFINITY ? exp2f((h[i].top - top) * kLog2e) : 1.0f;
            lost += h[i].lost * f;
            add(sum, lost, h[i].sum * f);
        }
        s.base[tid] = -(double)top - log((double)sum + lost);
    }
    __syncthreads();
    // ---- candidates of all rows, each a list in its own order
    Pick list = {0, 0};
    for (int k = warp; k < n; k += kWarps) {
        const float sc = s.score[k];
        const bool was = s.was[k];
        Pick v = {0, ~(uint32_t)(k * kWarp + lane)};
        if (fabsf(sc) < INFINITY) {
            double total = sc;
            bool any = lane == 0;
            uint32_t token = 0;
            if (!was) {
                uint64_t key = s.share[k * slices].keys[lane];
                for (int i = 1; i < slices; ++i) warp_merge(key, s.share[k * slices + i].keys[kWarp - 1 - lane], lane);
                any = key != 0 && lane < keep;
                token = 0xffffffffu - (uint32_t)key;
                // (x - top) first: the difference of neighbours is exact
                total += (double)value_of((uint32_t)(key >> 32)) + s.base[k];
            }
            const double q = c.penalty == 0.0 ? total : total / s.norm[k];
            any = any && (c.penalty == 0.0 || s.norm[k] >= 0.0);  // (below 0 it would turn the order of the logits round)
            if (any && q > -INFINITY && q < INFINITY) v.rank = ordered(q);
            s.totals[k][lane] = (float)total;
            s.tokens[k][lane] = token;
        }
        warp_merge(list, from_lane(v, kWarp - 1), lane);
    }
    int warps = 1;
    while (warps < kWarps && warps < n) warps *= 2;
    block_merge(list, s.picks, lane, warp, warps);
    __syncwarp();  // (one beam: the block has not met, and lanes read below what others wrote to s.totals, s.tokens)
    if (warp == 0 && lane < keep) {
        const int64_t o = r * keep + lane;
        int token = -1, parent = -1, length = 0;
        bool ended = true;
        float total = -INFINITY;
        if (list.rank) {
            const uint32_t place = ~list.place;
            parent = (int)(place / kWarp);
            token = (int)s.tokens[parent][place % kWarp];
            total = s.totals[parent][place % kWarp];
            const bool was = s.was[parent];
            if (was) token = c.end;
            ended = was || (c.end >= 0 && token == c.end);
            length = s.length[parent];
        }
        c.out_scores[o] = total;
        c.out_tokens[o] = token;
        c.out_parents[o] = parent;
        if (c.out_done) c.out_done[o] = ended;
        if (c.out_lengths) c.out_lengths[o] = length;
    }
}

// ---------------------------------------------------------------------------
// reordering
// ---------------------------------------------------------------------------

// One column (of U) of all beams of a request and outer index at a time: a
// thread reads what moves before it writes any of it, so beams may trade
// places in place.
template <class U, int MOST>
__global__ void __launch_bounds__(kThreads) k_beam_reorder(const ReorderCall c) {
    const int64_t units = c.inner / (int64_t)sizeof(U), chunks = (units + kThreads - 1) / kThreads;
    const int64_t all = c.outer * c.batch * chunks;
    for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
        const int64_t row = div_fast(w, chunks), u = (w - row * chunks) * kThreads + threadIdx.x;
        const int64_t o = div_fast(row, c.batch), r = row - o * c.batch;
        if (u >= units) continue;
        char* base = static_cast<char*>(c.state) + o * c.outer_stride + r * c.batch_stride + u * (int64_t)sizeof(U);
        const int32_t* parents = c.parents + r * c.beams;
        U v[MOST];
        uint32_t moved = 0;
#pragma unroll
        for (int k = 0; k < MOST; ++k) {
            if (k < c.beams) {
                const int p = parents[k];
                if (p != k && p >= 0 && p < c.beams) {
                    moved |= 1u << k;
                    v[k] = *reinterpret_cast<const U*>(base + p * c.beam_stride);
                }
            }
        }
#pragma unroll
        for (int k = 0; k < MOST; ++k)
            if (moved >> k & 1) *reinterpret_cast<U*>(base + k * c.beam_stride) = v[k];
    }
}

template <class U>
void launch_reorder(const ReorderCall& c, int sm_count, cudaStream_t stream) {
    const int64_t chunks = (c.inner / (int64_t)sizeof(U) + kThreads - 1) / kThreads;
    const unsigned grid = (unsigned)std::min<int64_t>(c.outer * c.batch * chunks, (int64_t)sm_count * 8);
    if (c.beams <= 4) k_beam_reorder<U, 4><<<grid, kThreads, 0, stream>>>(c);
    else if (c.beams <= 8) k_beam_reorder<U, 8><<<grid, kThreads, 0, stream>>>(c);
    else if (c.beams <= 16) k_beam_reorder<U, 16><<<grid, kThreads, 0, stream>>>(c);
    else k_beam_reorder<U, 32><<<grid, kThreads, 0, stream>>>(c);
}

}  // namespace bs

ak_status run_beam_select(BeamCall c, cudaStream_t stream) {
    using namespace bs;
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    auto* kernel = c.dtype == AK_F32 ? k_beam_select<float> : k_beam_select<bf16>;
    static ClusterLimit limits[2];
    int most = 0;
    const ak_status st = limits[c.dtype == AK_F32].get(reinterpret_cast<const void*>(kernel), kThreads, dev.device, &most);
    if (st != AK_OK) return st;
    // blocks of a request: as many as run at once over all requests, four an
    // SM; whole rows each, or each row in slices of a round of loads at least
    const int64_t room = std::max<int64_t>(1, std::min<int64_t>(most, 4 * dev.sm_count / c.batch));
    int parts = (int)std::min<int64_t>(room, c.beams);
    c.slices = 1;
    while ((c.slices + 1) * c.beams <= room && c.vocab / (c.slices + 1) >= kThreads * 4) ++c.slices;
    if (c.slices > 1) parts = c.slices * c.beams;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(c.batch * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (log_on())
        log_call("beam_select requests=%lld beams=%d vocab=%lld keep=%d: clusters of %d blocks, rows in %d slices",
                 (long long)c.batch, c.beams, (long long)c.vocab, c.keep, parts, c.slices);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, c);
    if (e != cudaSuccess) return cuda_fail(e);
    count_launches(1);
    return check_launch();
}

ak_status run_beam_reorder(const ReorderCall& c, cudaStream_t stream) {
    using namespace bs;
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    const uint64_t bits = (uint64_t)reinterpret_cast<uintptr_t>(c.state) | (uint64_t)c.inner | (uint64_t)c.beam_stride |
                          (uint64_t)c.batch_stride | (uint64_t)c.outer_stride;
    if (bits % 16 == 0) launch_reorder<int4>(c, dev.sm_count, stream);
    else if (bits % 4 == 0) launch_reorder<int32_t>(c, dev.sm_count, stream);
    else if (bits % 2 == 0) launch_reorder<int16_t>(c, dev.sm_count, stream);
    else launch_reorder<int8_t>(c, dev.sm_count, stream);
    count_launches(1);
    return check_launch();
}

}  // namespace ak
