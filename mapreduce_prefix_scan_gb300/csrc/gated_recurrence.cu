// gated_recurrence.cu -- the scan whose state is a vector and whose decay is a
// gate for every token and channel, over packed sequences: forward, gradients,
// and single tokens.
//
//   h_t = a_t h_{t-1} + b_t x_t,  channel by channel
//   decay form: a = exp(g), b = 1;   gate form: a = sigmoid(g), b = 1 - a
// Gradients, with G_t the gradient that reaches h_t and C_t = a_t G_t what it
// passes on to h_{t-1}:
//   G_t = dh_t + C_{t+1}
//   dx_t = b_t G_t
//   dg_t = C_t h_{t-1}  (decay),  G_t (h_{t-1} - x_t) a_t b_t  (gate)
// Both are affine scans along the packed token axis, the second in reversed
// time (virtual token v = tokens - 1 - t), with a reset where a sequence begins.
//
// A cluster of up to 16 blocks takes 64 channels and walks the whole packed
// axis, a tile of kTy x R tokens for each block and step, whatever the
// sequences' lengths: balance does not depend on them, each input is read once
// and each output written once. In a tile a thread holds R consecutive tokens of 4
// channels in registers and folds them to (A, B), h -> A h + B; 64 threads fold
// the tile's 16 pairs, hand the block's pair to every block of the cluster
// (distributed shared memory), and after the cluster's barrier fold the pairs
// before them onto the state carried from the last step. So a token is a few
// dozen roundings away from any earlier one, not one for each token between,
// the order of every sum is fixed, and there is neither a workspace nor a wait
// on another cluster. The next tile's loads are in flight meanwhile.
//
// Of a run's or tile's A both A and A - 1 are held, and one above 1/2 is applied
// as A - 1: a factor near one that is rounded itself is off by up to 3e-8, the
// same way each time where gates are equal, for every token (or run) of a memory
// of thousands. A - 1 comes from the sum of the gates (decay), or from the b_t
// (gate), and its error is relative to itself.
#include <algorithm>
#include <atomic>
#include <cooperative_groups.h>

#include "ak_common.cuh"
#include "ak_internal.h"

namespace cg = cooperative_groups;

namespace ak {
namespace gr {

constexpr int kThreads = 256;
constexpr int kVec = 4;                       // channels of a thread
constexpr int kLx = 16;                       // threads along the channels
constexpr int kCh = kVec * kLx;               // channels of a block
constexpr int kTy = kThreads / kLx;           // runs of tokens of a tile
constexpr int kMaxParts = 16;                 // blocks of a cluster

// Four neighbouring values as they lie in memory.
template <class T>
struct alignas(4 * sizeof(T)) Four {
    uint32_t w[sizeof(T)];
};

__device__ __forceinline__ float get(const Four<float>& f, int i) { return __uint_as_float(f.w[i]); }
__device__ __forceinline__ float get(const Four<bf16>& f, int i) {
    return __uint_as_float(i % 2 ? f.w[i / 2] & 0xffff0000u : f.w[i / 2] << 16);
}

__device__ __forceinline__ Four<float> ld_four(const float* p) {
    Four<float> f;
    asm("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
        : "=r"(f.w[0]), "=r"(f.w[1]), "=r"(f.w[2]), "=r"(f.w[3]) : "l"(p));
    return f;
}
__device__ __forceinline__ Four<bf16> ld_four(const bf16* p) {
    Four<bf16> f;
    asm("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(f.w[0]), "=r"(f.w[1]) : "l"(p));
    return f;
}

// Values [0, left) of four at p, zeros past them.
template <class T, bool WIDE>
__device__ __forceinline__ Four<T> load(const T* p, int left) {
    if constexpr (WIDE) {
        return ld_four(p);
    } else {
        T v[kVec];
#pragma unroll
        for (int i = 0; i < kVec; ++i) v[i] = i < left ? p[i] : T(0.0f);
        Four<T> f;
        memcpy(&f, v, sizeof f);
        return f;
    }
}

__device__ __forceinline__ void store_values(float* p, const float (&v)[kVec]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store_values(bf16* p, const float (&v)[kVec]) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v[0], v[1]), hi = __floats2bfloat162_rn(v[2], v[3]);
    uint2 u;
    memcpy(&u.x, &lo, 4);
    memcpy(&u.y, &hi, 4);
    *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ void set(float* p, float v) { *p = v; }
__device__ __forceinline__ void set(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

template <class T, bool WIDE>
__device__ __forceinline__ void store(T* p, const float (&v)[kVec], int left) {
    if constexpr (WIDE) store_values(p, v);
    else {
#pragma unroll
        for (int i = 0; i < kVec; ++i)
            if (i < left) set(p + i, v[i]);
    }
}

// 2^x; an infinity gives 0 or an infinity, a NaN itself.
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

constexpr float kLog2e = 1.4426950408889634f;

// a and b of a gate, both to their own relative precision: 2^-22 where the
// results are bf16, a rounding or two where they are float32 (twice the
// instructions, for twice the bytes). In the first, e stops at 2^126, where a
// has long been nothing beside b.
template <class T, int FORM>
__device__ __forceinline__ void weights(float g, float& a, float& b) {
    constexpr bool kFast = sizeof(T) == 2;
    if (FORM == AK_RECURRENCE_DECAY) {
        a = kFast ? exp2_fast(g * kLog2e) : expf(g);
        b = 1.0f;
    } else {
        if (kFast) {
            const float e = exp2_fast(min_nan(g * -kLog2e, 126.0f));
            a = rcp_fast(1.0f + e);
            b = e * a;
        } else {
            const float e = expf(-fabsf(g)), r = __frcp_rn(1.0f + e);
            a = g >= 0.0f ? r : e * r;
            b = g >= 0.0f ? e * r : r;
        }
    }
}

// A product of a's, and it less one.
template <int FORM>
struct Product {
    float p = FORM == AK_RECURRENCE_DECAY ? 0.0f : 1.0f, m = 0.0f;  // (decay: p is the sum of the gates until done)
    __device__ __forceinline__ void take(float g, float a, float b) {
        if (FORM == AK_RECURRENCE_DECAY) {
            p += g;
        } else {
            p *= a;
            m = fmaf(m, -b, m - b);  // (1 + m)(1 - b) - 1
        }
    }
    __device__ __forceinline__ void done() {
        if (FORM == AK_RECURRENCE_DECAY) {
            m = expm1f(p);
            p = expf(p);
        }
    }
};

// A map h -> A h + off at h, of A and A - 1.
__device__ __forceinline__ bool is_near(float p) { return p > 0.5f; }
__device__ __forceinline__ float apply(float f, bool near, float off, bool reset, float h) {
    return reset ? off : fmaf(f, h, off) + (near ? h : 0.0f);
}

// The sequences' borders along the virtual axis, boundary by boundary: one
// warp's window of 32 of them, moved on as the walk passes it.
template <bool REV>
struct Borders {
    const int32_t* offsets;
    int tokens, n;
    __device__ __forceinline__ int at(int i) const {  // 0 <= i <= n
        if (!offsets) return i == 0 ? 0 : tokens;
        const int o = min(max(offsets[REV ? n - i : i], 0), tokens);
        return REV ? tokens - o : o;
    }
    // a sequence's number in the arrays of states
    __device__ __forceinline__ int64_t seq(int j) const { return REV ? n - 1 - j : j; }
};

// What a tile's tokens begin and end: bits for each run of R tokens, and the
// sequence for each token that has one.
template <int R>
struct Marks {
    int any;  // of the tile, or a row of it lies outside every sequence
    uint32_t first[kTy], last[kTy];
    int seq_first[kTy * R], seq_last[kTy * R];
};

template <int R, bool REV>
struct Walk {
    Borders<REV> b;
    int base, v;
    __device__ __forceinline__ void window(int lane) { v = base + lane <= b.n ? b.at(base + lane) : 0x7fffffff; }
    // Marks of tile [t0, t0 + kTy R); tiles come in increasing order.
    __device__ __forceinline__ void mark(Marks<R>& k, int64_t t0, int lane, int lo, int hi) {
        constexpr int kTile = kTy * R;
        bool any = t0 < lo || t0 + kTile > hi;
        if (lane < kTy) k.first[lane] = k.last[lane] = 0;
        __syncwarp();
        while (true) {
            const int next = __shfl_down_sync(0xffffffffu, v, 1);
            if (lane < kWarp - 1 && base + lane < b.n && v < next) {
                const int64_t f = v - t0, l = next - 1 - t0;
                if (f >= 0 && f < kTile) {
                    any = true;
                    k.seq_first[f] = base + lane;
                    atomicOr(&k.first[f / R], 1u << (f % R));
                }
                if (l >= 0 && l < kTile) {
                    any = true;
                    k.seq_last[l] = base + lane;
                    atomicOr(&k.last[l / R], 1u << (l % R));
                }
            }
            const int end = __shfl_sync(0xffffffffu, v, kWarp - 1);
            if (end >= t0 + kTile || base + kWarp - 1 >= b.n) break;
            base += kWarp - 1;
            window(lane);
        }
        any = __any_sync(0xffffffffu, any);
        if (lane == 0) k.any = any;
        __syncwarp();
    }
};

template <int R>
struct Shared {
    float p[kTy][kCh], m[kTy][kCh], b[kTy][kCh];  // the runs' maps: factor, factor less one, offset
    float in[kTy][kCh];                           // the state before each run
    float2 peer[2][kMaxParts][kCh];               // the blocks' maps: factor (less one where `near`), offset
    uint32_t near[2][kMaxParts][kCh / kWarp];
    int reset[kTy], peer_reset[2][kMaxParts];     // whether a map forgets what was before
    Marks<R> marks[2];
};

template <bool B>
struct Is {
    static constexpr bool value = B;
};

template <class T, int FORM, int R, bool REV, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) k_recurrence(const RecurrenceCall c) {
    constexpr int kTile = kTy * R;
    constexpr bool kGate = FORM == AK_RECURRENCE_GATE;
    constexpr bool kRows = REV && !kGate;   // h_{t-1} is read for every token
    constexpr bool kAgain = REV && kGate;   // h_{t-1} is computed again from the one before the run
    constexpr int RZ = REV ? R : 1, RB = kAgain ? R : 1;
    __shared__ Shared<R> s;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), parts = (int)cl.num_blocks();
    const int tid = threadIdx.x, lane = tid % kWarp, warp = tid / kWarp;
    const int lx = tid % kLx, ty = tid / kLx;
    const int64_t c0 = (int64_t)(blockIdx.x / parts) * kCh;
    const int64_t ch = c0 + lx * kVec;
    const int left = (int)max((int64_t)0, min((int64_t)kVec, c.channels - ch));
    const int64_t tokens = c.tokens;
    Walk<R, REV> walk;
    walk.b.offsets = c.offsets;
    walk.b.tokens = (int)tokens;
    walk.b.n = (int)c.seqs;
    const int lo = walk.b.n ? walk.b.at(0) : 0, hi = walk.b.n ? walk.b.at(walk.b.n) : 0;
    const int steps = (int)((tokens + (int64_t)kTile * parts - 1) / ((int64_t)kTile * parts));
    const float* const first_state = REV ? c.dstate_out : c.state_in;
    float* const last_state = REV ? c.dstate_in : c.state_out;

    // sequences without tokens pass their state on
    if (last_state) {
        for (int j0 = (rank * (kThreads / kWarp) + warp) * kWarp; j0 < walk.b.n; j0 += parts * kThreads) {
            const int j = j0 + lane;
            unsigned empty = __ballot_sync(0xffffffffu, j < walk.b.n && walk.b.at(j) >= walk.b.at(j + 1));
            for (; empty; empty &= empty - 1) {
                const int64_t row = walk.b.seq(j0 + __ffs(empty) - 1) * c.channels;
                for (int64_t i = c0 + lane; i < min(c0 + kCh, c.channels); i += kWarp)
                    last_state[row + i] = first_state ? first_state[row + i] : 0.0f;
            }
        }
    }

    // this thread's first row of an array, and the way to its next one
    const int64_t t_first = (int64_t)rank * kTile, t_step = (int64_t)parts * kTile;
    const int64_t row0 = REV ? tokens - 1 - (t_first + ty * R) : t_first + ty * R;
    struct Rows {
        T* p;
        int64_t row, tile;
    };
    auto rows = [&](const ak_rows& r, int64_t shift) {
        const int64_t st = REV ? -r.token_stride : r.token_stride;
        return Rows{static_cast<T*>(r.data) + (row0 + shift) * r.token_stride + ch, st, st * t_step};
    };
    Rows gr = rows(c.gate, 0), ur = rows(REV ? c.dh : c.x, 0), zr = rows(kRows ? c.h : c.x, kRows ? -1 : 0);
    Rows br = rows(c.h, -R);  // the row before the run's first token in time
    Rows outr = rows(REV ? c.dx : c.out, 0), dgr = rows(c.dgate, 0);

    // raw inputs of one tile: the gate, what is scanned (x, or dh), and for
    // gradients h_{t-1} of each token, or x and the state before the run
    Four<T> rg[R], ru[R], rz[RZ], rb[1];
    auto fetch = [&](int64_t t0) {
        const int64_t v0 = t0 + ty * R;
        if (t0 + kTile < tokens) {  // (the last row of all has none before it)
            if (left > 0) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    rg[r] = load<T, WIDE>(gr.p + r * gr.row, left);
                    ru[r] = load<T, WIDE>(ur.p + r * ur.row, left);
                    if (REV) rz[r % RZ] = load<T, WIDE>(zr.p + r * zr.row, left);
                }
                if (kAgain) rb[0] = load<T, WIDE>(br.p, left);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int64_t v = v0 + r;
                rg[r] = ru[r] = Four<T>{};
                if (REV) rz[r % RZ] = Four<T>{};
                if (v < tokens && left > 0) {
                    rg[r] = load<T, WIDE>(gr.p + r * gr.row, left);
                    ru[r] = load<T, WIDE>(ur.p + r * ur.row, left);
                    if (REV && (kAgain || v + 1 < tokens)) rz[r % RZ] = load<T, WIDE>(zr.p + r * zr.row, left);
                }
            }
            rb[0] = Four<T>{};
            if (kAgain && v0 + R < tokens && left > 0) rb[0] = load<T, WIDE>(br.p, left);
        }
        gr.p += gr.tile, ur.p += ur.tile, zr.p += zr.tile, br.p += br.tile;
    };

    float carry = 0.0f;  // of channel c0 + tid, for tid < kCh
#pragma unroll
    for (int r = 0; r < R; ++r) {
        rg[r] = ru[r] = Four<T>{};
        if (REV) rz[r % RZ] = Four<T>{};
    }
    rb[0] = Four<T>{};
    fetch(t_first);
    constexpr int kMarker = kThreads / kWarp - 1;
    if (warp == kMarker) {
        walk.base = 0;
        walk.window(lane);
        walk.mark(s.marks[0], t_first, lane, lo, hi);
    }
    if (parts > 1) cl.sync();  // every block of the cluster runs before one writes to another
    else __syncthreads();

    float a[R][kVec], b[RB][kVec], u[R][kVec], z[RZ][kVec];
    // ---- the run's map; in a tile with marks, tokens that begin a sequence
    // take its state and forget what was before
    auto fold_run = [&](auto marked, const Marks<R>& mk) {
        constexpr bool M = decltype(marked)::value;
        const uint32_t first = M ? mk.first[ty] : 0, last = M ? mk.last[ty] : 0;
        float fold[kVec] = {};
        Product<FORM> prod[kVec];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool begins = M && (first >> r & 1);
            const float* from = begins && first_state ? first_state + walk.b.seq(mk.seq_first[ty * R + r]) * c.channels + ch : nullptr;
#pragma unroll
            for (int q = 0; q < kVec; ++q) {
                const float g = get(rg[r], q), in = get(ru[r], q);
                float w;
                weights<T, FORM>(g, a[r][q], w);
                const float s0 = M && from && q < left ? from[q] : 0.0f;
                if (REV) {
                    if (kAgain) b[r % RB][q] = w;
                    u[r][q] = begins ? in + s0 : in;
                    fold[q] = a[r][q] * (begins ? u[r][q] : u[r][q] + fold[q]);
                } else {
                    const float in_b = kGate ? w * in : in;
                    u[r][q] = begins ? fmaf(a[r][q], s0, in_b) : in_b;
                    fold[q] = begins || r == 0 ? u[r][q] : fmaf(a[r][q], fold[q], u[r][q]);
                }
                prod[q].take(g, a[r][q], w);
            }
        }
        if (REV) {  // h_{t-1} of each token
            float hh[kVec];
#pragma unroll
            for (int q = 0; q < kVec; ++q) hh[q] = kAgain ? get(rb[0], q) : 0.0f;
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {  // forward in time
                const bool begins = M && (last >> r & 1);  // the sequence's first token
                const float* from = begins && c.state_in ? c.state_in + walk.b.seq(mk.seq_last[ty * R + r]) * c.channels + ch : nullptr;
#pragma unroll
                for (int q = 0; q < kVec; ++q) {
                    const float s0 = M && from && q < left ? from[q] : 0.0f;
                    if (kRows) {
                        z[r % RZ][q] = begins ? s0 : get(rz[r % RZ], q);
                    } else {
                        const float bq = b[r % RB][q], x = get(rz[r % RZ], q);
                        if (begins) hh[q] = s0;
                        z[r % RZ][q] = (hh[q] - x) * (a[r][q] * bq);
                        hh[q] = fmaf(a[r][q], hh[q], bq * x);
                    }
                }
            }
        }
        float p[kVec], m[kVec];
#pragma unroll
        for (int q = 0; q < kVec; ++q) {
            prod[q].done();
            p[q] = prod[q].p, m[q] = prod[q].m;
        }
        store_values(&s.p[ty][lx * kVec], p);
        store_values(&s.m[ty][lx * kVec], m);
        store_values(&s.b[ty][lx * kVec], fold);
        if (lx == 0) s.reset[ty] = first != 0;
    };
    // ---- the run again, from its state
    auto finish_run = [&](auto marked, const Marks<R>& mk, int64_t t0) {
        constexpr bool M = decltype(marked)::value;
        const uint32_t first = M ? mk.first[ty] : 0, last = M ? mk.last[ty] : 0;
        float h[kVec];
#pragma unroll
        for (int q = 0; q < kVec; ++q) h[q] = s.in[ty][lx * kVec + q];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t v = t0 + ty * R + r;
            const bool begins = M && (first >> r & 1), inside = !M || (v >= lo && v < hi);
            float o[kVec], og[kVec];
#pragma unroll
            for (int q = 0; q < kVec; ++q) {
                if (REV) {
                    const float g = begins ? u[r][q] : u[r][q] + h[q];
                    h[q] = a[r][q] * g;
                    o[q] = kGate ? b[r % RB][q] * g : g;
                    og[q] = (kGate ? g : h[q]) * z[r % RZ][q];
                    if (!inside) og[q] = 0.0f;
                } else {
                    h[q] = begins ? u[r][q] : fmaf(a[r][q], h[q], u[r][q]);
                    o[q] = h[q];
                }
                if (!inside) o[q] = 0.0f;
            }
            if (left > 0 && (!M || v < tokens)) {
                store<T, WIDE>(outr.p + r * outr.row, o, left);
                if (REV) store<T, WIDE>(dgr.p + r * dgr.row, og, left);
            }
            if (M && (last >> r & 1) && last_state) {
                float* to = last_state + walk.b.seq(mk.seq_last[ty * R + r]) * c.channels + ch;
#pragma unroll
                for (int q = 0; q < kVec; ++q)
                    if (q < left) to[q] = h[q];
            }
        }
        outr.p += outr.tile, dgr.p += dgr.tile;
    };

    for (int i = 0; i < steps; ++i) {
        const int64_t t0 = i * t_step + t_first;
        const Marks<R>& mk = s.marks[i & 1];
        const bool marked = mk.any;
        if (marked) fold_run(Is<true>(), mk);
        else fold_run(Is<false>(), mk);
        if (i + 1 < steps) fetch(t0 + t_step);
        __syncthreads();
        if (warp == kMarker && i + 1 < steps) walk.mark(s.marks[(i + 1) & 1], t0 + t_step, lane, lo, hi);

        // ---- the runs' maps meet
        float2 map = {};
        uint32_t near = 0;
        int reset = 0;
        if (tid < kCh) {
            float p = 1.0f, m = 0.0f, off = 0.0f;
#pragma unroll
            for (int y = 0; y < kTy; ++y) {
                const float py = s.p[y][tid], my = s.m[y][tid];
                off = apply(is_near(py) ? my : py, is_near(py), s.b[y][tid], s.reset[y], off);
                p *= py;
                m = fmaf(m, my, m + my);
                reset |= s.reset[y];
            }
            near = __ballot_sync(0xffffffffu, is_near(p));
            map = make_float2(is_near(p) ? m : p, off);
            for (int k = 0; k < parts && parts > 1; ++k) {
                Shared<R>* o = cl.map_shared_rank(&s, k);
                o->peer[i & 1][rank][tid] = map;
                if (lane == 0) o->near[i & 1][rank][warp] = near;
                if (tid == 0) o->peer_reset[i & 1][rank] = reset;
            }
        }
        if (parts > 1) cl.sync();
        if (tid < kCh) {
            auto of_peer = [&](int k, float h) {
                const float2 f = s.peer[i & 1][k][tid];
                return apply(f.x, s.near[i & 1][k][warp] >> lane & 1, f.y, s.peer_reset[i & 1][k], h);
            };
            float h = carry;
            for (int k = 0; k < rank; ++k) h = of_peer(k, h);
            carry = apply(map.x, near >> lane & 1, map.y, reset != 0, h);
            for (int k = rank + 1; k < parts; ++k) carry = of_peer(k, carry);
#pragma unroll
            for (int y = 0; y < kTy; ++y) {
                const float py = s.p[y][tid];
                s.in[y][tid] = h;
                h = apply(is_near(py) ? s.m[y][tid] : py, is_near(py), s.b[y][tid], s.reset[y], h);
            }
        }
        __syncthreads();
        if (marked) finish_run(Is<true>(), mk, t0);
        else finish_run(Is<false>(), mk, t0);
    }
}

// One token of each request, on its state of a pool.
template <class T, int FORM, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_step(const RecurrenceCall c, float* state, const int32_t* slots, int64_t nslots) {
    const int64_t per = (c.channels + kVec - 1) / kVec;
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at >= per * c.tokens) return;
    const int64_t t = div_fast(at, per), ch = (at - t * per) * kVec;
    const int left = (int)min((int64_t)kVec, c.channels - ch);
    const Four<T> g = load<T, WIDE>(static_cast<const T*>(c.gate.data) + t * c.gate.token_stride + ch, left);
    const Four<T> x = load<T, WIDE>(static_cast<const T*>(c.x.data) + t * c.x.token_stride + ch, left);
    const int64_t slot = slots ? slots[t] : t;
    float h[kVec] = {};
    if (slot >= 0 && slot < nslots) {
        float* p = state + slot * c.channels + ch;
        if (WIDE) {
            const float4 v = *reinterpret_cast<const float4*>(p);
            h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
        } else {
#pragma unroll
            for (int q = 0; q < kVec; ++q) h[q] = q < left ? p[q] : 0.0f;
        }
#pragma unroll
        for (int q = 0; q < kVec; ++q) {
            float a, b;
            weights<float, FORM>(get(g, q), a, b);  // (states are float32)
            h[q] = fmaf(a, h[q], FORM == AK_RECURRENCE_GATE ? b * get(x, q) : get(x, q));
        }
        store<float, WIDE>(p, h, left);
    }
    store<T, WIDE>(static_cast<T*>(c.out.data) + t * c.out.token_stride + ch, h, left);
}

// Whether four neighbouring channels are one aligned load in every row.
template <class T>
bool wide(const RecurrenceCall& c, const ak_rows& r) {
    return r.data == nullptr || (aligned(r.data, 4 * sizeof(T)) && r.token_stride % 4 == 0);
}

template <class T, int FORM, int R, bool REV, bool WIDE>
ak_status launch(const RecurrenceCall& c, cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    auto* kernel = k_recurrence<T, FORM, R, REV, WIDE>;
    static std::atomic<uint64_t> ready{0};
    if (!(ready.load() >> dev.device & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e != cudaSuccess) return cuda_fail(e);
        ready.fetch_or(1ull << dev.device);
    }
    // blocks of a cluster: as many as run at once over all channels, two an SM,
    // and no more than there are tiles
    const int64_t groups = std::max<int64_t>(1, (c.channels + kCh - 1) / kCh);
    const int64_t tiles = std::max<int64_t>(1, (c.tokens + kTy * R - 1) / (kTy * R));
    const int64_t parts = std::max<int64_t>(1, std::min<int64_t>({(int64_t)kMaxParts, tiles, 2 * dev.sm_count / groups}));
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(groups * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (log_on())
        log_call("gated_recurrence%s tokens=%lld seqs=%lld channels=%lld: %lld clusters of %lld blocks", REV ? "_backward" : "",
                 (long long)c.tokens, (long long)c.seqs, (long long)c.channels, (long long)groups, (long long)parts);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, c);
    if (e != cudaSuccess) return cuda_fail(e);
    count_launches(1);
    return check_launch();
}

// Tokens of a run: as many bytes in flight for either type.
template <class T, bool REV>
constexpr int run_of() { return REV || sizeof(T) == 4 ? 4 : 8; }

template <class T, bool REV>
ak_status by_form(const RecurrenceCall& c, cudaStream_t stream) {
    constexpr int R = run_of<T, REV>();
    const bool w = c.channels % 4 == 0 && wide<T>(c, c.x) && wide<T>(c, c.gate) && wide<T>(c, c.h) && wide<T>(c, c.dh) &&
                   wide<T>(c, c.out) && wide<T>(c, c.dx) && wide<T>(c, c.dgate);
    if (c.form == AK_RECURRENCE_DECAY)
        return w ? launch<T, AK_RECURRENCE_DECAY, R, REV, true>(c, stream) : launch<T, AK_RECURRENCE_DECAY, R, REV, false>(c, stream);
    return w ? launch<T, AK_RECURRENCE_GATE, R, REV, true>(c, stream) : launch<T, AK_RECURRENCE_GATE, R, REV, false>(c, stream);
}

template <class T, int FORM>
ak_status step(const RecurrenceCall& c, float* state, const int32_t* slots, int64_t nslots, cudaStream_t stream) {
    const int64_t per = (c.channels + kVec - 1) / kVec;
    const unsigned grid = (unsigned)((per * c.tokens + kThreads - 1) / kThreads);
    const bool w = c.channels % 4 == 0 && aligned(state, 16) && wide<T>(c, c.x) && wide<T>(c, c.gate) && wide<T>(c, c.out);
    if (w) k_step<T, FORM, true><<<grid, kThreads, 0, stream>>>(c, state, slots, nslots);
    else k_step<T, FORM, false><<<grid, kThreads, 0, stream>>>(c, state, slots, nslots);
    count_launches(1);
    return check_launch();
}

}  // namespace gr

ak_status run_recurrence(const RecurrenceCall& c, cudaStream_t stream) {
    return c.dtype == AK_F32 ? gr::by_form<float, false>(c, stream) : gr::by_form<bf16, false>(c, stream);
}

ak_status run_recurrence_backward(const RecurrenceCall& c, cudaStream_t stream) {
    return c.dtype == AK_F32 ? gr::by_form<float, true>(c, stream) : gr::by_form<bf16, true>(c, stream);
}

ak_status run_recurrence_step(const RecurrenceCall& c, float* state, const int32_t* slots, int64_t nslots,
                              cudaStream_t stream) {
    if (c.form == AK_RECURRENCE_DECAY)
        return c.dtype == AK_F32 ? gr::step<float, AK_RECURRENCE_DECAY>(c, state, slots, nslots, stream)
                                 : gr::step<bf16, AK_RECURRENCE_DECAY>(c, state, slots, nslots, stream);
    return c.dtype == AK_F32 ? gr::step<float, AK_RECURRENCE_GATE>(c, state, slots, nslots, stream)
                             : gr::step<bf16, AK_RECURRENCE_GATE>(c, state, slots, nslots, stream);
}

}  // namespace ak
