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
// A cluster of up to 16 blocks takes 32 channels and walks the whole packed
// axis, a tile of 8 runs of R tokens for each block and step, whatever the
// sequences' lengths: balance does not depend on them, each input is read once
// and each output written once. In a tile a thread folds R consecutive tokens of a
// channel, which it keeps in registers, to a map h -> A h + B; a thread for each
// channel folds the tile's 8 maps, sends the block's map to every block of the
// cluster, and when theirs have come folds the maps before its own onto the
// state carried from the last step. So a token is a few dozen roundings away from
// any earlier one, not one for each token between, the order of every sum is fixed,
// and there is neither a workspace nor a wait on another cluster. The next two
// tiles' copies to shared memory are under way meanwhile. Maps travel as
// asynchronous stores that count on the receiver's barrier: a cluster-wide
// barrier after plain stores took 1500 to 2500 cycles of a step's 5500, most of
// them the fence before it.
//
// Of a run's or tile's A both A and A - 1 are held, and one above 1/2 is applied
// as A - 1: a factor near one that is rounded itself is off by up to 3e-8, the
// same way each time where gates are equal, for every token (or run) of a memory
// of thousands. A - 1 comes from the sum of the gates (decay), or from the b_t
// (gate), and its error is relative to itself. In float32 calls the tokens of a
// run whose factors are all above 1/2 are applied so as well.
//
// Bound by the latency of a step (fold, maps, chain, outputs: 4000 cycles for two
// tiles of 256 tokens x 32 channels bf16 an SM, 32 KB read and 16 written each),
// not by its loads. Back to back: 16384 x 4096 bf16 95 us (0.63 of the copy
// bandwidth), gradients of 8192 x 4096 bf16 93 us (0.53), 8192 x 4096 float32 77 to
// 79 us (0.76), 32771 x 640 float32 65 us (0.57) and its gradients 102 us, 331 x 1000
// in 64 sequences 6.6 us. Rows at odd addresses, 16384 x 1001: 38 us bf16, 63 float32
// (by 4-byte words 86 and 103). Steps: 256 x 4096 bf16 3.5 us (0.62), one request 2.2 us.
// Tried: 64 channels a cluster, two a thread (32771 x 640 float32: 96 us, and 60 so;
// 32768 x 2048 bf16 102 and 94; but 16384 x 4096 bf16 90 and 95); half the tile and
// three blocks an SM (115, and 105 at the time); tiles in registers, loaded one step
// ahead (141).
#include <algorithm>
#include <atomic>
#include <cooperative_groups.h>

#include "ak_common.cuh"
#include "ak_internal.h"
#include "ak_tma.cuh"

namespace cg = cooperative_groups;

namespace ak {
namespace gr {

constexpr int kThreads = 256;
constexpr int kPerSm = 2;                     // blocks of an SM
constexpr int kCh = kWarp;                    // channels of a cluster, one a thread of a warp
constexpr int kTy = kThreads / kCh;           // runs of tokens of a tile
constexpr int kMaxParts = 16;                 // blocks of a cluster
constexpr int kAhead = 4;                     // maps read before the first of them is applied
constexpr int kStages = 2;                    // tiles on their way

// 16 bytes (or the first `size` of them, zeros past them) into shared memory.
__device__ __forceinline__ void copy16(void* to, const void* from, int size) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(
                     static_cast<uint32_t>(__cvta_generic_to_shared(to))),
                 "l"(from), "r"(size)
                 : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ float as_float(float v) { return v; }
__device__ __forceinline__ float as_float(bf16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void set(float* p, float v) { *p = v; }
__device__ __forceinline__ void set(bf16* p, float v) { *p = __float2bfloat16_rn(v); }

// Neighbouring values as they lie in memory.
template <class T, int N>
struct alignas(N * sizeof(T)) Values {
    T v[N];
    __device__ __forceinline__ float operator[](int i) const {
        return as_float(v[i]);
    }
};

// Values [0, left) of v; in one store where `whole`.
template <class T, int N>
__device__ __forceinline__ void store(T* p, const float (&v)[N], int left, bool whole) {
    if (whole) {
        Values<T, N> o;
#pragma unroll
        for (int i = 0; i < N; ++i) set(&o.v[i], v[i]);
        *reinterpret_cast<Values<T, N>*>(p) = o;
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
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

// a and b of a gate, each to 2^-21 + |g| 2^-23 of itself (the exponential's instruction
// 2^-22, its argument's product and constant |g| 2^-23.7, a sum, a reciprocal and a
// product 2^-22); below 2^-126 they are 0. Where results are bf16 e stops at 2^126: a has
// long been nothing beside b there.
template <class T, int FORM>
__device__ __forceinline__ void weights(float g, float& a, float& b) {
    constexpr bool kFast = sizeof(T) == 2;
    if (FORM == AK_RECURRENCE_DECAY) {
        a = exp2_fast(g * kLog2e);
        b = 1.0f;
    } else {
        if (kFast) {
            const float e = exp2_fast(min_nan(g * -kLog2e, 126.0f));
            a = rcp_fast(1.0f + e);
            b = e * a;
        } else {
            const float e = exp2_fast(fabsf(g) * -kLog2e), r = rcp_fast(1.0f + e);
            a = g >= 0.0f ? r : e * r;
            b = g >= 0.0f ? e * r : r;
        }
    }
}

// e^l - 1, by its series where that is used as such (l within log 2 of 0: the
// terms left out are below 2^-23 of it); e^l is e.
__device__ __forceinline__ float less_one(float l, float e) {
    float m = 1.0f / 362880;
    m = fmaf(m, l, 1.0f / 40320);
    m = fmaf(m, l, 1.0f / 5040);
    m = fmaf(m, l, 1.0f / 720);
    m = fmaf(m, l, 1.0f / 120);
    m = fmaf(m, l, 1.0f / 24);
    m = fmaf(m, l, 1.0f / 6);
    m = fmaf(m, l, 0.5f);
    m = fmaf(m * l, l, l);
    return fabsf(l) < 0.6932f ? m : e - 1.0f;
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
            const float l = p;
            p = exp2_fast(l * kLog2e);
            m = less_one(l, p);
        }
    }
};

// h -> A h + off, or off alone (a value that is not finite must not pass a
// reset, so it is no factor of 0). A above 1/2 is one and f, else f alone.
struct Map {
    float f, one, off;
    uint32_t reset;
    __device__ __forceinline__ float operator()(float h) const {
        const float v = fmaf(one, h, fmaf(f, h, off));
        return reset ? off : v;
    }
};
// A product of such A's in the making: A and A - 1.
struct Factor {
    float p = 1.0f, m = 0.0f;
    // this one, then the factor of `o`
    __device__ __forceinline__ Factor then(const Map& o) const {
        const float om = o.f + (o.one - 1.0f);
        Factor r;
        r.p = p * (o.f + o.one);
        r.m = fmaf(m, om, m + om);
        return r;
    }
    __device__ __forceinline__ Map map(float off, uint32_t reset) const {
        const bool near = p > 0.5f;
        return {near ? m : p, near ? 1.0f : 0.0f, off, reset};
    }
};
// What a channel's maps are to the blocks of its cluster: asynchronous stores
// whose bytes count on the receiver's barrier.
__device__ __forceinline__ uint32_t in_block(uint32_t addr, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ void send(uint32_t to, uint32_t bar, const Map& m) {
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "r"(__float_as_uint(m.f)), "r"(__float_as_uint(m.one)), "r"(__float_as_uint(m.off)), "r"(m.reset), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ bool try_received(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// The call whose wait ran out last (its epoch): for opts->check.
__device__ uint64_t g_gave_up;

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

// Inputs of a tile: the gate, what is scanned (x, or dh), and for gradients
// h_{t-1} of each token (decay), or x and the state before each run (gate).
// Of rows that do not begin at multiples of 16 bytes the pieces of 16 that they lie
// in are copied, so a row begins up to 14 bytes into its place.
template <class T, int R, bool REV, bool AGAIN, bool WIDE>
struct Tile {
    static constexpr int kPitch = WIDE ? kCh : kCh + 16 / (int)sizeof(T);
    T g[kTy * R * kPitch], u[kTy * R * kPitch], z[REV ? kTy * R * kPitch : 8], before[AGAIN ? kTy * kPitch : 8];
};

template <class T, int R, bool REV, bool AGAIN, bool WIDE>
struct alignas(16) Shared {
    Tile<T, R, REV, AGAIN, WIDE> tile[kStages];
    float4 run[kTy][kCh];  // the runs' maps
    float in[kTy][kCh];    // the state before each run
    Marks<R> marks[2];
    uint64_t come[2];  // maps of the even and of the odd steps
    int lost;
    float4 peer[1];  // [2][parts][kCh]: the blocks' maps
};

template <class T, int FORM, int R, bool REV, bool WIDE>
__global__ void __launch_bounds__(kThreads, kPerSm) k_recurrence(const RecurrenceCall c) {
    constexpr int kTile = kTy * R;
    constexpr bool kGate = FORM == AK_RECURRENCE_GATE;
    constexpr bool kRows = REV && !kGate;   // h_{t-1} is read for every token
    constexpr bool kAgain = REV && kGate;   // h_{t-1} is computed again from the one before the run
    constexpr int RZ = REV ? R : 1, RB = kAgain ? R : 1;
    extern __shared__ __align__(16) unsigned char smem[];
    using S = Shared<T, R, REV, kAgain, WIDE>;
    using In = Tile<T, R, REV, kAgain, WIDE>;
    constexpr int kPitch = In::kPitch;
    S& s = *reinterpret_cast<S*>(smem);
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), parts = (int)cl.num_blocks();
    const int tid = threadIdx.x, lane = tid % kWarp, ty = tid / kWarp;
    const int64_t c0 = (int64_t)(blockIdx.x / parts) * kCh;
    const int64_t ch = c0 + lane;
    const bool some = ch < c.channels;
    const int64_t tokens = c.tokens;
    Walk<R, REV> walk;
    walk.b.offsets = c.offsets;
    walk.b.tokens = (int)tokens;
    walk.b.n = (int)c.seqs;
    const int lo = walk.b.n ? walk.b.at(0) : 0, hi = walk.b.n ? walk.b.at(walk.b.n) : 0;
    const int steps = (int)((tokens + (int64_t)kTile * parts - 1) / ((int64_t)kTile * parts));
    const float* const first_state = REV ? c.dstate_out : c.state_in;
    float* const last_state = REV ? c.dstate_in : c.state_out;
    const int64_t t_first = (int64_t)rank * kTile, t_step = (int64_t)parts * kTile;
    auto row_of = [&](int64_t v) { return REV ? tokens - 1 - v : v; };

    // `rows` rows of an array, `apart` virtual tokens apart from v0 on (row + shift in
    // memory), those below `end` of them; the others are zeros
    auto copy = [&](T* to, const ak_rows& from, int rows, int apart, int64_t v0, int shift, int64_t end) {
        const T* base = static_cast<const T*>(from.data) + c0;
        const int64_t way = (REV ? -1 : 1) * from.token_stride;
        if constexpr (WIDE) {
            constexpr int kPer = 16 / (int)sizeof(T), kRow = kCh / kPer;
            const int col = tid % kRow * kPer;
            const int bytes = (int)max((int64_t)0, min((int64_t)kPer, c.channels - c0 - col)) * (int)sizeof(T);
            int64_t v = v0 + (int64_t)(tid / kRow) * apart;
            const T* p = base + (row_of(v) + shift) * from.token_stride + col;
#pragma unroll
            for (int r = 0; r < rows; r += kThreads / kRow) {
                const bool in = v < end && bytes > 0;
                if (r + tid / kRow < rows) copy16(to + (r + tid / kRow) * kPitch + col, in ? p : base, in ? bytes : 0);
                v += (kThreads / kRow) * apart;
                p += way * ((kThreads / kRow) * apart);
            }
        } else {
            // the aligned pieces of 16 bytes that the row lies in, from the first one's
            // beginning (which is of the same allocation: those begin at such pieces)
            constexpr int kPer = 16 / (int)sizeof(T), kRow = 2 * kCh / kPer, kUsed = kCh / kPer + 1;
            const int piece = tid % kRow;
            const int64_t n = min((int64_t)kCh, c.channels - c0) * (int64_t)sizeof(T);
            const char* none = reinterpret_cast<const char*>(reinterpret_cast<uintptr_t>(from.data) & ~(uintptr_t)15);
            int64_t v = v0 + (int64_t)(tid / kRow) * apart;
            const T* p = base + (row_of(v) + shift) * from.token_stride;
#pragma unroll
            for (int r = 0; r < rows; r += kThreads / kRow) {
                const char* row = reinterpret_cast<const char*>(p);
                const int64_t lead = reinterpret_cast<uintptr_t>(row) & 15;
                const int size = v < end ? (int)max((int64_t)0, min((int64_t)16, n + lead - 16 * piece)) : 0;
                if (piece < kUsed && r + tid / kRow < rows)
                    copy16(to + (r + tid / kRow) * kPitch + piece * kPer, size ? row - lead + 16 * piece : none, size);
                v += (kThreads / kRow) * apart;
                p += way * ((kThreads / kRow) * apart);
            }
        }
    };
    auto fetch = [&](int i) {
        auto& t = s.tile[i % kStages];
        const int64_t v0 = t_first + i * t_step;
        if (i < steps) {
            copy(t.g, c.gate, kTile, 1, v0, 0, tokens);
            copy(t.u, REV ? c.dh : c.x, kTile, 1, v0, 0, tokens);
            if constexpr (kAgain) {
                copy(t.z, c.x, kTile, 1, v0, 0, tokens);
                // the row before the run's first token in time
                copy(t.before, c.h, kTy, R, v0 + R - 1, -1, tokens - 1);
            }
            if constexpr (kRows) copy(t.z, c.h, kTile, 1, v0, -1, tokens - 1);
        }
        copy_commit();
    };
    // value of this thread's channel in row r of a copied array whose row 0 is virtual token v0
    auto value = [&](const T* rows, const ak_rows& from, int r, int apart, int64_t v0, int shift) {
        int at = lane;
        if constexpr (!WIDE) {
            const uint32_t first = (uint32_t)(reinterpret_cast<uintptr_t>(from.data) / sizeof(T)) + (uint32_t)c0;
            const uint32_t row = (uint32_t)row_of(v0) + (uint32_t)shift + (uint32_t)((REV ? -1 : 1) * r * apart);
            at += (first + row * (uint32_t)from.token_stride) & (16 / sizeof(T) - 1);
        }
        return as_float(rows[r * kPitch + at]);
    };
    constexpr int kMarker = kTy - 1;
#pragma unroll
    for (int i = 0; i < kStages; ++i) fetch(i);
    if (ty == kMarker) {
        walk.base = 0;
        walk.window(lane);
        walk.mark(s.marks[0], t_first, lane);
    }
    // sequences without tokens pass their state on
    if (last_state) {
        for (int j0 = (rank * kTy + ty) * kWarp; j0 < walk.b.n; j0 += parts * kThreads) {
            const int j = j0 + lane;
            unsigned empty = __ballot_sync(0xffffffffu, j < walk.b.n && walk.b.at(j) >= walk.b.at(j + 1));
            for (; empty; empty &= empty - 1) {
                const int64_t at = walk.b.seq(j0 + __ffs(empty) - 1) * c.channels + ch;
                if (some) last_state[at] = first_state ? first_state[at] : 0.0f;
            }
        }
    }
    if (tid == 0) {
        s.lost = 0;
        if (parts > 1) {
            mbar_init(&s.come[0], 1);
            mbar_init(&s.come[1], 1);
            fence_barrier_init();
        }
    }
    if (parts > 1) cl.sync();  // every block of the cluster runs, with its barriers, before one sends to another

    // a token's factor is a + one: in runs of float32 calls whose factors are all
    // near one, a is held less one
    constexpr bool kNear = sizeof(T) == 4;
    float a[R] = {}, b[RB] = {}, u[R] = {}, z[RZ] = {}, one = 0.0f;
    auto times = [&](int r, float h) { return kNear ? fmaf(a[r], h, one * h) : a[r] * h; };
    auto step = [&](int r, float h) { return kNear ? fmaf(one, h, fmaf(a[r], h, u[r])) : fmaf(a[r], h, u[r]); };
    auto state_of = [&](const float* states, int64_t seq) { return states && some ? states[seq * c.channels + ch] : 0.0f; };
    // ---- the run's map. A token that begins a sequence takes its state, and its
    // factor is 0: it forgets what was before, which is dropped as well, as it may
    // not be finite. Such tokens are rare, but some tile of a step often has one, and
    // code for them that is unrolled over the run evicts the rest from the
    // instruction cache (2000 cycles a step). So they are taken one at a time in
    // rolled loops, and only the chains, two or three instructions a token, exist
    // with and without them. (A branch for every token would keep tokens from
    // overlapping.)
    auto fold_run = [&](const Marks<R>& mk, const In& t, int64_t t0) {
        const uint32_t first = mk.first[ty];
        [[maybe_unused]] const uint32_t last = mk.last[ty];
        const int64_t v0 = t0 + ty * R;
        const int at = ty * R * kPitch;
        Product<FORM> prod;
        [[maybe_unused]] float m[kNear ? R : 1], least = 1.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            const float g = value(t.g + at, c.gate, r, 1, v0, 0), in = value(t.u + at, REV ? c.dh : c.x, r, 1, v0, 0);
            float w;
            weights<T, FORM>(g, a[r], w);
            prod.take(g, a[r], w);
            u[r] = kGate && !REV ? w * in : in;
            if constexpr (kAgain) {
                b[r] = w;
                z[r] = value(t.z + at, c.x, r, 1, v0, 0);
            }
            if constexpr (kRows) z[r] = value(t.z + at, c.h, r, 1, v0, -1);
            if constexpr (kNear) {
                m[r] = kGate ? -w : less_one(g, a[r]);
                least = fminf(least, a[r]);
            }
        }
        if constexpr (kNear) {
            const bool near = least > 0.5f;
            one = near ? 1.0f : 0.0f;
#pragma unroll
            for (int r = 0; r < R; ++r) a[r] = near ? m[r] : a[r];
        }
        if constexpr (REV) {  // h_{t-1} of each token, forward in time
            float hh = 0.0f;
            if constexpr (kAgain) hh = value(t.before, c.h, ty, R, t0 + R - 1, -1);
            auto again = [&](int r) {
                if constexpr (kAgain) {
                    const float bx = b[r] * z[r], h = hh;
                    hh = kNear ? fmaf(one, h, fmaf(a[r], h, bx)) : fmaf(a[r], h, bx);
                    z[r] = (h - z[r]) * ((a[r] + one) * b[r]);
                }
            };
            if (kRows) {
#pragma unroll 1
                for (uint32_t m = last; m; m &= m - 1) {  // the sequences' first tokens
                    const int at = __ffs(m) - 1;
                    const float s0 = state_of(c.state_in, walk.b.seq(mk.seq_last[ty * R + at]));
#pragma unroll
                    for (int r = 0; r < R; ++r) z[r] = r == at ? s0 : z[r];
                }
            } else if (last) {
#pragma unroll
                for (int r = R - 1; r >= 0; --r) {
                    if (last & 1u << r) hh = state_of(c.state_in, walk.b.seq(mk.seq_last[ty * R + r]));
                    again(r);
                }
            } else {
#pragma unroll
                for (int r = R - 1; r >= 0; --r) again(r);
            }
        }
        float fold = 0.0f;
        auto add = [&](int r) { fold = REV ? times(r, u[r] + fold) : step(r, fold); };
#pragma unroll 1
        for (uint32_t m = first; m; m &= m - 1) {
            const int at = __ffs(m) - 1;
            const float s0 = state_of(first_state, walk.b.seq(mk.seq_first[ty * R + at]));
#pragma unroll
            for (int r = 0; r < R; ++r) {
                if (REV) {
                    u[r] = r == at ? u[r] + s0 : u[r];
                } else {
                    u[r] = r == at && first_state ? step(r, s0) : u[r];
                    a[r] = r == at ? 0.0f - one : a[r];
                }
            }
        }
        if (first) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                fold = first & 1u << r ? 0.0f : fold;
                add(r);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) add(r);
        }
        prod.done();
        const Map all = Factor{prod.p, prod.m}.map(fold, first != 0);
        s.run[ty][lane] = make_float4(all.f, all.one, all.off, __uint_as_float(all.reset));
    };
    // ---- the run again, from its state: u becomes h_t, or G_t
    T* const out = static_cast<T*>(REV ? c.dx.data : c.out.data) + ch;
    T* const out_g = static_cast<T*>(c.dgate.data) + ch;
    const int64_t out_stride = REV ? c.dx.token_stride : c.out.token_stride;
    auto finish_run = [&](const Marks<R>& mk, int64_t t0) {
        const uint32_t first = mk.first[ty], last = mk.last[ty];
        const int64_t v0 = t0 + ty * R;
        float h = s.in[ty][lane];
        auto move = [&](int r) {
            u[r] = REV ? u[r] + h : step(r, h);
            h = REV ? times(r, u[r]) : u[r];
        };
        if (first) {
#pragma unroll
            for (int r = 0; r < R; ++r) {
                h = first & 1u << r ? 0.0f : h;
                move(r);
            }
        } else {
#pragma unroll
            for (int r = 0; r < R; ++r) move(r);
        }
        if (last_state && some) {
#pragma unroll 1
            for (uint32_t m = last; m; m &= m - 1) {
                const int at = __ffs(m) - 1;
                float v = 0.0f;
#pragma unroll
                for (int r = 0; r < R; ++r) v = r == at ? (REV ? times(r, u[r]) : u[r]) : v;
                last_state[walk.b.seq(mk.seq_last[ty * R + at]) * c.channels + ch] = v;
            }
        }
        T *po = out + row_of(v0) * out_stride, *pg = out_g + row_of(v0) * c.dgate.token_stride;
        const int64_t next = REV ? -out_stride : out_stride, next_g = REV ? -c.dgate.token_stride : c.dgate.token_stride;
        auto put = [&](int r) {
            if constexpr (kAgain) set(po, b[r] * u[r]);
            else set(po, u[r]);
            if constexpr (REV) set(pg, (kGate ? u[r] : times(r, u[r])) * z[r]);
            po += next, pg += next_g;
        };
        if (v0 + R <= tokens) {
            if (some) {
#pragma unroll
                for (int r = 0; r < R; ++r) put(r);
            }
        } else if (some) {
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (v0 + r < tokens) put(r);
        }
        if (t0 < lo || t0 + kTile > hi) {  // rows outside every sequence
#pragma unroll 1
            for (int64_t v = v0; v < min(v0 + R, tokens); ++v) {
                if ((v >= lo && v < hi) || !some) continue;
                set(out + row_of(v) * out_stride, 0.0f);
                if (REV) set(out_g + row_of(v) * c.dgate.token_stride, 0.0f);
            }
        }
    };

    float carry = 0.0f;  // of this thread's channel (warp 0)
    for (int i = 0; i < steps; ++i) {
        const int64_t t0 = i * t_step + t_first;
        const Marks<R>& mk = s.marks[i & 1];
        copy_wait<kStages - 1>();
        __syncthreads();
        if (s.lost) break;
        fold_run(mk, s.tile[i % kStages], t0);
        __syncthreads();

        // ---- the runs' maps meet
        auto map_of = [](const float4& f) { return Map{f.x, f.y, f.z, __float_as_uint(f.w)}; };
        Map tile = {};
        if (ty == 0) {
            Factor fac;
            float off = 0.0f;
            uint32_t reset = 0;
#pragma unroll
            for (int y0 = 0; y0 < kTy; y0 += kAhead) {
                float4 f[kAhead];
#pragma unroll
                for (int y = 0; y < kAhead; ++y) f[y] = s.run[y0 + y][tid];
#pragma unroll
                for (int y = 0; y < kAhead; ++y) {
                    const Map m = map_of(f[y]);
                    fac = fac.then(m);
                    off = m(off);
                    reset |= m.reset;
                }
            }
            tile = fac.map(off, reset);
            if (parts > 1) {
                if (tid == 0) mbar_arrive_expect_tx(&s.come[i & 1], (uint32_t)(parts * kCh * sizeof(float4)));
                const uint32_t to = smem_addr(s.peer + ((i & 1) * parts + rank) * kCh + tid), bar = smem_addr(&s.come[i & 1]);
#pragma unroll 4
                for (int k = 0; k < parts && (int64_t)i * parts + rank != c.skip_tile; ++k) send(in_block(to, k), in_block(bar, k), tile);
            }
        }
        fetch(i + kStages);
        if (ty == kMarker && i + 1 < steps) walk.mark(s.marks[(i + 1) & 1], t0 + t_step, lane);
        if (ty == 0) {
            float h = carry;
            if (parts > 1) {
                const uint32_t parity = i >> 1 & 1;
                if (!try_received(&s.come[i & 1], parity)) {
                    const uint64_t deadline = globaltimer_ns() + c.wait_limit_ns;
                    while (!try_received(&s.come[i & 1], parity)) {
                        if (globaltimer_ns() > deadline) {
                            s.lost = 1;
                            g_gave_up = c.epoch;
                            break;
                        }
                    }
                }
                const float4* peer = s.peer + (i & 1) * parts * kCh + tid;
                float at = carry;
                for (int k0 = 0; k0 < parts; k0 += kAhead) {
                    float4 f[kAhead];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) f[k] = peer[min(k0 + k, parts - 1) * kCh];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        if (k0 + k == rank) h = at;
                        if (k0 + k < parts) at = map_of(f[k])(at);
                    }
                }
                carry = at;
            } else {
                carry = tile(carry);
            }
#pragma unroll
            for (int y0 = 0; y0 < kTy; y0 += kAhead) {
                float4 f[kAhead];
#pragma unroll
                for (int y = 0; y < kAhead; ++y) f[y] = s.run[y0 + y][tid];
#pragma unroll
                for (int y = 0; y < kAhead; ++y) {
                    s.in[y0 + y][tid] = h;
                    h = map_of(f[y])(h);
                }
            }
        }
        __syncthreads();
        finish_run(mk, t0);
    }
    copy_wait<0>();
    if (parts > 1) cl.sync();  // nothing is on its way to a block that has left
}

constexpr int kStepVec = 4;  // channels of a thread of the step

// Neighbouring values of a row, zeros from the left-th on.
template <class T, bool WIDE>
__device__ __forceinline__ Values<T, kStepVec> load(const T* p, int left) {
    if constexpr (WIDE) {
        return *reinterpret_cast<const Values<T, kStepVec>*>(p);
    } else {
        T v[kStepVec];
#pragma unroll
        for (int i = 0; i < kStepVec; ++i) v[i] = i < left ? p[i] : T(0.0f);
        Values<T, kStepVec> f;
        memcpy(&f, v, sizeof f);
        return f;
    }
}

// One token of each request, on its state of a pool.
template <class T, int FORM, bool WIDE>
__global__ void __launch_bounds__(kThreads) k_step(const RecurrenceCall c, float* state, const int32_t* slots, int64_t nslots) {
    const int64_t per = (c.channels + kStepVec - 1) / kStepVec;
    const int64_t at = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    if (at >= per * c.tokens) return;
    const int64_t t = div_fast(at, per), ch = (at - t * per) * kStepVec;
    const int left = (int)min((int64_t)kStepVec, c.channels - ch);
    const Values<T, kStepVec> g = load<T, WIDE>(static_cast<const T*>(c.gate.data) + t * c.gate.token_stride + ch, left);
    const Values<T, kStepVec> x = load<T, WIDE>(static_cast<const T*>(c.x.data) + t * c.x.token_stride + ch, left);
    const int64_t slot = slots ? slots[t] : t;
    float h[kStepVec] = {};
    if (slot >= 0 && slot < nslots) {
        float* p = state + slot * c.channels + ch;
        if (WIDE) {
            const float4 v = *reinterpret_cast<const float4*>(p);
            h[0] = v.x, h[1] = v.y, h[2] = v.z, h[3] = v.w;
        } else {
#pragma unroll
            for (int q = 0; q < kStepVec; ++q) h[q] = q < left ? p[q] : 0.0f;
        }
#pragma unroll
        for (int q = 0; q < kStepVec; ++q) {
            float a, b;
            weights<float, FORM>(g[q], a, b);  // (states are float32)
            const bool near = a > 0.5f && fabsf(h[q]) < INFINITY;  // ((a - 1) h + h of an infinity is none)
            const float less = FORM == AK_RECURRENCE_GATE ? -b : less_one(g[q], a), in = FORM == AK_RECURRENCE_GATE ? b * x[q] : x[q];
            h[q] = fmaf(near ? less : a, h[q], in) + (near ? h[q] : 0.0f);
        }
        store(p, h, left, WIDE);
    }
    store(static_cast<T*>(c.out.data) + t * c.out.token_stride + ch, h, left, WIDE);
}

// Whether every row of an array begins at a multiple of `bytes`.
template <class T>
bool rows_at(const ak_rows& r, size_t bytes) {
    return r.data == nullptr || (aligned(r.data, bytes) && r.token_stride * sizeof(T) % bytes == 0);
}

template <class T, int FORM, int R, bool REV, bool WIDE>
ak_status launch(const RecurrenceCall& c, cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    auto* kernel = k_recurrence<T, FORM, R, REV, WIDE>;
    using S = Shared<T, R, REV, REV && FORM == AK_RECURRENCE_GATE, WIDE>;
    auto smem_of = [](int64_t parts) { return sizeof(S) + 2 * (size_t)parts * kCh * sizeof(float4); };
    cudaLaunchConfig_t cfg = {};
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // clusters of each size that the device holds at once; asked for once
    static std::atomic<uint64_t> ready{0};
    static std::atomic<int> room[64][kMaxParts + 1];
    if (!(ready.load() >> dev.device & 1)) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem_of(kMaxParts));
        for (int p = 1; p <= kMaxParts && e == cudaSuccess; ++p) {
            int n = 0;
            cfg.gridDim = dim3((unsigned)p);
            cfg.dynamicSmemBytes = smem_of(p);
            attr[0].val.clusterDim.x = (unsigned)p;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            room[dev.device & 63][p] = n;
        }
        if (e != cudaSuccess) return cuda_fail(e);
        ready.fetch_or(1ull << dev.device);
    }
    // blocks of a cluster: the most with which the clusters of all channels run
    // at once, and no more than there are tiles
    const int64_t groups = std::max<int64_t>(1, (c.channels + kCh - 1) / kCh);
    const int64_t tiles = std::max<int64_t>(1, (c.tokens + kTy * R - 1) / (kTy * R));
    int64_t parts = std::min<int64_t>(kMaxParts, tiles);
    while (parts > 1 && room[dev.device & 63][parts] < groups) --parts;
    cfg.gridDim = dim3((unsigned)(groups * parts));
    cfg.dynamicSmemBytes = smem_of(parts);
    attr[0].val.clusterDim.x = (unsigned)parts;
    if (log_on())
        log_call("gated_recurrence%s tokens=%lld seqs=%lld channels=%lld: %lld clusters of %lld blocks", REV ? "_backward" : "",
                 (long long)c.tokens, (long long)c.seqs, (long long)c.channels, (long long)groups, (long long)parts);
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, c);
    if (e != cudaSuccess) return cuda_fail(e);
    count_launches(1);
    return check_launch();
}

template <class T, int FORM, bool REV>
ak_status by_length(const RecurrenceCall& c, cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    const bool w = rows_at<T>(c.x, 16) && rows_at<T>(c.gate, 16) && rows_at<T>(c.h, 16) && rows_at<T>(c.dh, 16);
    // tokens of a run: what the registers hold; fewer where the tiles would leave
    // SMs without a block
    constexpr int R = (sizeof(T) == 2 ? 32 : 16) / (REV ? 2 : 1), kShort = 8;
    const int64_t groups = (c.channels + kCh - 1) / kCh;
    if (R > kShort && groups * ((c.tokens + kTy * R - 1) / (kTy * R)) < dev.sm_count)
        return w ? launch<T, FORM, kShort, REV, true>(c, stream) : launch<T, FORM, kShort, REV, false>(c, stream);
    return w ? launch<T, FORM, R, REV, true>(c, stream) : launch<T, FORM, R, REV, false>(c, stream);
}

template <class T, bool REV>
ak_status by_form(const RecurrenceCall& c, cudaStream_t stream) {
    return c.form == AK_RECURRENCE_DECAY ? by_length<T, AK_RECURRENCE_DECAY, REV>(c, stream)
                                         : by_length<T, AK_RECURRENCE_GATE, REV>(c, stream);
}

template <class T, int FORM>
ak_status step(const RecurrenceCall& c, float* state, const int32_t* slots, int64_t nslots, cudaStream_t stream) {
    const int64_t per = (c.channels + kStepVec - 1) / kStepVec;
    const unsigned grid = (unsigned)((per * c.tokens + kThreads - 1) / kThreads);
    constexpr size_t kFour = 4 * sizeof(T);
    const bool w = c.channels % 4 == 0 && aligned(state, 16) && rows_at<T>(c.x, kFour) && rows_at<T>(c.gate, kFour) && rows_at<T>(c.out, kFour);
    if (w) k_step<T, FORM, true><<<grid, kThreads, 0, stream>>>(c, state, slots, nslots);
    else k_step<T, FORM, false><<<grid, kThreads, 0, stream>>>(c, state, slots, nslots);
    count_launches(1);
    return check_launch();
}

}  // namespace gr

ak_status recurrence_lost(uint64_t epoch, bool* lost) {
    uint64_t word = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(&word, gr::g_gave_up, sizeof word);
    if (e != cudaSuccess) return cuda_fail(e);
    *lost = word == epoch;
    return AK_OK;
}

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
