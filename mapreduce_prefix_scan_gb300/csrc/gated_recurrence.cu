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
// A is carried as its logarithm (in the decay form the sum of the gates, whose
// error is relative to itself), and one above 1/2 is applied as A - 1: a factor
// near one that is rounded itself is off by up to 3e-8, the same way each time
// where gates are equal, for every token (or run) of a memory of thousands.
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

// a and b of a gate; both to their own relative precision.
template <int FORM>
__device__ __forceinline__ void weights(float g, float& a, float& b) {
    if (FORM == AK_RECURRENCE_DECAY) {
        a = expf(g);
        b = 1.0f;
    } else {
        const float e = expf(-fabsf(g)), r = __frcp_rn(1.0f + e);
        a = g >= 0.0f ? r : e * r;
        b = g >= 0.0f ? e * r : r;
    }
}

// A product of a's, by its logarithm.
template <int FORM>
struct Product {
    float l = 0.0f;               // decay: the sum of the gates
    float p = 1.0f, m = 0.0f;     // gate: the product, and the product less one
    __device__ __forceinline__ void take(float g, float a, float b) {
        if (FORM == AK_RECURRENCE_DECAY) {
            l += g;
        } else {
            p *= a;
            m = fmaf(m, -b, m - b);  // (1 + m)(1 - b) - 1
        }
    }
    __device__ __forceinline__ float log() const {
        if (FORM == AK_RECURRENCE_DECAY) return l;
        return p > 0.5f ? log1pf(m) : logf(p);
    }
};

// Whether the factor e^l is held less one, and a map's value at h.
__device__ __forceinline__ bool is_near(float l) { return l > -0.6931f; }
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
    uint32_t first[kTy], last[kTy];
    int seq_first[kTy * R], seq_last[kTy * R];
};

template <int R, bool REV>
struct Walk {
    Borders<REV> b;
    int base, v;
    __device__ __forceinline__ void window(int lane) { v = base + lane <= b.n ? b.at(base + lane) : 0x7fffffff; }
    // Marks of tile [t0, t0 + kTy R); tiles come in increasing order.
    __device__ __forceinline__ void mark(Marks<R>& k, int64_t t0, int lane) {
        constexpr int kTile = kTy * R;
        if (lane < kTy) k.first[lane] = k.last[lane] = 0;
        __syncwarp();
        while (true) {
            const int next = __shfl_down_sync(0xffffffffu, v, 1);
            if (lane < kWarp - 1 && base + lane < b.n && v < next) {
                const int64_t f = v - t0, l = next - 1 - t0;
                if (f >= 0 && f < kTile) {
                    k.seq_first[f] = base + lane;
                    atomicOr(&k.first[f / R], 1u << (f % R));
                }
                if (l >= 0 && l < kTile) {
                    k.seq_last[l] = base + lane;
                    atomicOr(&k.last[l / R], 1u << (l % R));
                }
            }
            const int end = __shfl_sync(0xffffffffu, v, kWarp - 1);
            if (end >= t0 + kTile || base + kWarp - 1 >= b.n) break;
            base += kWarp - 1;
            window(lane);
        }
        __syncwarp();
    }
};

template <int R>
struct Shared {
    float a[kTy][kCh], l[kTy][kCh], b[kTy][kCh];  // the runs' maps: factor (less one if near one), its logarithm, offset
    float in[kTy][kCh];                           // the state before each run
    float2 peer[2][kMaxParts][kCh];               // the blocks' maps: factor (less one where `near`), offset
    uint32_t near[2][kMaxParts][kCh / kWarp];
    int reset[kTy], peer_reset[2][kMaxParts];     // whether a map forgets what was before
    Marks<R> marks[2];
};

template <class T, int FORM, int R, bool REV, bool WIDE>
__global__ void __launch_bounds__(kThreads, 2) k_recurrence(const RecurrenceCall c) {
    constexpr int kTile = kTy * R;
    constexpr bool kGate = FORM == AK_RECURRENCE_GATE;
    constexpr bool kRows = REV && !kGate;   // h_{t-1} is read for every token
    constexpr bool kAgain = REV && kGate;   // h_{t-1} is computed again from the one before the run
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
    const int64_t steps = (tokens + (int64_t)kTile * parts - 1) / ((int64_t)kTile * parts);
    const float* const first_state = REV ? c.dstate_out : c.state_in;
    float* const last_state = REV ? c.dstate_in : c.state_out;

    const T* const xp = static_cast<const T*>(c.x.data) + ch;
    const T* const gp = static_cast<const T*>(c.gate.data) + ch;
    const T* const hp = static_cast<const T*>(c.h.data) + ch;
    const T* const dp = static_cast<const T*>(c.dh.data) + ch;

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

    auto row_of = [&](int64_t v) { return REV ? tokens - 1 - v : v; };
    // raw inputs of one tile: the gate, what is scanned (x, or dh), and for
    // gradients h_{t-1} of each token, or x and the state before the run
    Four<T> rg[R], ru[R], rz[REV ? R : 1], rb[1];
    auto fetch = [&](int64_t t0) {
        const int64_t v0 = t0 + ty * R;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t v = v0 + r, t = row_of(v);
            rg[r] = ru[r] = Four<T>{};
            if (REV) rz[r % (REV ? R : 1)] = Four<T>{};
            if (v < tokens && left > 0) {
                rg[r] = load<T, WIDE>(gp + t * c.gate.token_stride, left);
                ru[r] = REV ? load<T, WIDE>(dp + t * c.dh.token_stride, left) : load<T, WIDE>(xp + t * c.x.token_stride, left);
                if (kAgain) rz[r % (REV ? R : 1)] = load<T, WIDE>(xp + t * c.x.token_stride, left);
                if (kRows && t > 0) rz[r % (REV ? R : 1)] = load<T, WIDE>(hp + (t - 1) * c.h.token_stride, left);
            }
        }
        if (kAgain) {
            rb[0] = Four<T>{};
            const int64_t t = row_of(v0 + R - 1);
            if (t > 0 && t < tokens && left > 0) rb[0] = load<T, WIDE>(hp + (t - 1) * c.h.token_stride, left);
        }
    };

    float carry = 0.0f;  // of channel c0 + tid, for tid < kCh
    const int64_t t_first = (int64_t)rank * kTile, t_step = (int64_t)parts * kTile;
    fetch(t_first);
    constexpr int kMarker = kThreads / kWarp - 1;
    if (warp == kMarker) {
        walk.base = 0;
        walk.window(lane);
        walk.mark(s.marks[0], t_first, lane);
    }
    if (parts > 1) cl.sync();  // every block of the cluster runs before one writes to another
    else __syncthreads();

    for (int64_t i = 0; i < steps; ++i) {
        const int64_t t0 = i * t_step + t_first;
        const Marks<R>& mk = s.marks[i & 1];
        const uint32_t first = mk.first[ty], last = mk.last[ty];

        // ---- fold of the run: B in `fold`, A in `prod`
        float a[R][kVec], b[kGate && REV ? R : 1][kVec], u[R][kVec], z[REV ? R : 1][kVec], fold[kVec];
        Product<FORM> prod[kVec];
#pragma unroll
        for (int q = 0; q < kVec; ++q) fold[q] = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const bool begins = first >> r & 1;
            const float* from = begins && first_state ? first_state + walk.b.seq(mk.seq_first[ty * R + r]) * c.channels + ch : nullptr;
#pragma unroll
            for (int q = 0; q < kVec; ++q) {
                const float g = get(rg[r], q), in = get(ru[r], q);
                float w;
                weights<FORM>(g, a[r][q], w);
                const float s0 = from && q < left ? from[q] : 0.0f;
                if (REV) {
                    if (kGate) b[r % (kGate && REV ? R : 1)][q] = w;
                    u[r][q] = begins ? in + s0 : in;
                    fold[q] = a[r][q] * (begins ? u[r][q] : u[r][q] + fold[q]);
                } else {
                    const float in_b = kGate ? w * in : in;
                    u[r][q] = begins ? fmaf(a[r][q], s0, in_b) : in_b;
                    fold[q] = begins ? u[r][q] : fmaf(a[r][q], fold[q], u[r][q]);
                }
                prod[q].take(g, a[r][q], w);
            }
        }
        // ---- h_{t-1} of each token (gradients)
        if (REV) {
            float hh[kVec];
#pragma unroll
            for (int q = 0; q < kVec; ++q) hh[q] = kAgain ? get(rb[0], q) : 0.0f;
#pragma unroll
            for (int r = R - 1; r >= 0; --r) {  // forward in time
                const bool begins = last >> r & 1;  // the sequence's first token
                const float* from = begins && c.state_in ? c.state_in + walk.b.seq(mk.seq_last[ty * R + r]) * c.channels + ch : nullptr;
#pragma unroll
                for (int q = 0; q < kVec; ++q) {
                    const float s0 = from && q < left ? from[q] : 0.0f;
                    if (kRows) {
                        z[r % (REV ? R : 1)][q] = begins ? s0 : get(rz[r % (REV ? R : 1)], q);
                    } else {
                        const float bq = b[r % (kGate && REV ? R : 1)][q], x = get(rz[r % (REV ? R : 1)], q);
                        if (begins) hh[q] = s0;
                        z[r % (REV ? R : 1)][q] = (hh[q] - x) * a[r][q] * bq;
                        hh[q] = fmaf(a[r][q], hh[q], bq * x);
                    }
                }
            }
        }
        if (i + 1 < steps) fetch(t0 + t_step);

        // ---- the runs' maps meet
#pragma unroll
        for (int q = 0; q < kVec; ++q) {
            const float l = prod[q].log();
            s.l[ty][lx * kVec + q] = l;
            s.a[ty][lx * kVec + q] = is_near(l) ? expm1f(l) : expf(l);
            s.b[ty][lx * kVec + q] = fold[q];
        }
        if (lx == 0) s.reset[ty] = first != 0;
        __syncthreads();
        if (warp == kMarker && i + 1 < steps) walk.mark(s.marks[(i + 1) & 1], t0 + t_step, lane);
        float2 map = {};
        uint32_t near = 0, run_near = 0, run_reset = 0;
        if (tid < kCh) {
            float l = 0.0f, off = 0.0f;
#pragma unroll
            for (int y = 0; y < kTy; ++y) {
                const float ly = s.l[y][tid];
                run_reset |= (uint32_t)s.reset[y] << y;
                run_near |= (uint32_t)is_near(ly) << y;
                off = apply(s.a[y][tid], is_near(ly), s.b[y][tid], run_reset >> y & 1, off);
                l += ly;
            }
            near = __ballot_sync(0xffffffffu, is_near(l));
            map = make_float2(is_near(l) ? expm1f(l) : expf(l), off);
            for (int p = 0; p < parts && parts > 1; ++p) {
                Shared<R>* o = cl.map_shared_rank(&s, p);
                o->peer[i & 1][rank][tid] = map;
                if (lane == 0) o->near[i & 1][rank][warp] = near;
                if (tid == 0) o->peer_reset[i & 1][rank] = run_reset != 0;
            }
        }
        if (parts > 1) cl.sync();
        if (tid < kCh) {
            auto of_peer = [&](int p, float h) {
                const float2 m = s.peer[i & 1][p][tid];
                return apply(m.x, s.near[i & 1][p][warp] >> lane & 1, m.y, s.peer_reset[i & 1][p], h);
            };
            float h = carry;
            for (int p = 0; p < rank; ++p) h = of_peer(p, h);
            carry = apply(map.x, near >> lane & 1, map.y, run_reset != 0, h);
            for (int p = rank + 1; p < parts; ++p) carry = of_peer(p, carry);
#pragma unroll
            for (int y = 0; y < kTy; ++y) {
                s.in[y][tid] = h;
                h = apply(s.a[y][tid], run_near >> y & 1, s.b[y][tid], run_reset >> y & 1, h);
            }
        }
        __syncthreads();

        // ---- the run again, from its state
        float h[kVec];
#pragma unroll
        for (int q = 0; q < kVec; ++q) h[q] = s.in[ty][lx * kVec + q];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const int64_t v = t0 + ty * R + r, t = row_of(v);
            const bool begins = first >> r & 1, inside = v >= lo && v < hi;
            float o[kVec], og[kVec];
#pragma unroll
            for (int q = 0; q < kVec; ++q) {
                if (REV) {
                    const float g = begins ? u[r][q] : u[r][q] + h[q];
                    h[q] = a[r][q] * g;
                    o[q] = kGate ? b[r % (kGate && REV ? R : 1)][q] * g : g;
                    og[q] = kGate ? g * z[r % (REV ? R : 1)][q] : h[q] * z[r % (REV ? R : 1)][q];
                    if (!inside) og[q] = 0.0f;
                } else {
                    h[q] = begins ? u[r][q] : fmaf(a[r][q], h[q], u[r][q]);
                    o[q] = h[q];
                }
                if (!inside) o[q] = 0.0f;
            }
            if (v < tokens && left > 0) {
                if (REV) {
                    store<T, WIDE>(static_cast<T*>(c.dx.data) + ch + t * c.dx.token_stride, o, left);
                    store<T, WIDE>(static_cast<T*>(c.dgate.data) + ch + t * c.dgate.token_stride, og, left);
                } else {
                    store<T, WIDE>(static_cast<T*>(c.out.data) + ch + t * c.out.token_stride, o, left);
                }
            }
            if ((last >> r & 1) && last_state) {
                float* to = last_state + walk.b.seq(mk.seq_last[ty * R + r]) * c.channels + ch;
#pragma unroll
                for (int q = 0; q < kVec; ++q)
                    if (q < left) to[q] = h[q];
            }
        }
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
            weights<FORM>(get(g, q), a, b);
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
