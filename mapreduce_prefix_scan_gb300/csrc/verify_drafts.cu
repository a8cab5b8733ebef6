// verify_drafts.cu -- verification of drafted tokens against the target's
// probabilities, from given random numbers.
//
// Request r drafted d_0 .. d_{m-1} from distributions q_j; the target gives
// p_0 .. p_m. With u_j uniform in [0, 1) and e_v exponential (> 0):
//   a = the first j < m with not (u_j q_j(d_j) < p_j(d_j)), or m
//   tokens 0 .. a-1 are the drafts; token a is
//     argmax_v max(p_a(v) - q_a(v), 0) / e_v   if a < m (a refusal)
//     argmax_v p_a(v) / e_v                    if a == m (the bonus token)
// The argmax of weights over exponential noise draws from the normalised
// weights, so no normalising sum and no prefix sum of the row is needed: one
// pass over one row of p, q and e for each request, the least that has to be
// read. Without draft distributions q_j is one at d_j and zero elsewhere.
// Where the difference leaves nothing (p == q up to rounding), p decides.
//
// A cluster of blocks takes one request: warp 0 of every block finds `a` by
// itself (a gather of m values of p and q each; cheaper than passing it on),
// the blocks fold a slice of the row each into (score, lowest index) and
// combine in distributed shared memory. One launch, no workspace, and the
// same result in any order of combination.
//
// Bound by HBM for many requests (192 of 128000 float32: 47 us, 0.85 of the
// copy bandwidth; bf16 37 us, 0.73, its elements' divisions beside its bytes;
// certain drafts, with a row less to read, 44 and 40) and by the chain of
// dependent loads (draft -> p, q at the draft -> row, then the cluster's
// exchange) for few (4 of 32003: 6.0 us).
#include <algorithm>
#include <cooperative_groups.h>

#include "ak_common.cuh"
#include "ak_internal.h"

namespace cg = cooperative_groups;

namespace ak {
namespace vd {

constexpr int kThreads = 512;
constexpr int kBlocksPerSm = 3;

__device__ __forceinline__ float as_f(float v) { return v; }
__device__ __forceinline__ float as_f(bf16 v) { return __bfloat162float(v); }

// (score, index) as one word that orders by score, then by lowest index;
// 0 = no candidate. Scores are >= 0, so their bits order as integers.
__device__ __forceinline__ void offer(uint64_t& best, float weight, float noise, uint32_t v) {
    if (!(weight > 0.0f)) return;
    const float s = __fdiv_rn(weight, noise);
    if (!(s >= 0.0f)) return;
    const uint64_t key = ((uint64_t)(__float_as_uint(s) & 0x7fffffffu) << 32) | (0xffffffffu - v);
    if (key > best) best = key;
}

// Weights of elements [v, v + n) of the row against the noise.
template <class T, int MODE>  // 0: p alone, 1: p - q, 2: p without the draft
__device__ __forceinline__ uint64_t fold(const T* p, const T* q, const float* e, int64_t first, int64_t last,
                                         int64_t draft, bool vec) {
    uint64_t best = 0;
    constexpr int V = 16 / sizeof(T);
    if (vec) {
        // first is a multiple of V; the row's ragged end is taken one by one
        const int64_t full = first + (last - first) / V * V;
#pragma unroll 2
        for (int64_t v = first + (int64_t)threadIdx.x * V; v < full; v += (int64_t)kThreads * V) {
            const Raw<16> a = ld_stream16(p + v);
            Raw<16> b;
            if (MODE == 1) b = ld_stream16(q + v);
            Raw<16> n[V / 4];
#pragma unroll
            for (int i = 0; i < V / 4; ++i) n[i] = ld_stream16(e + v + 4 * i);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float w = as_f(raw_get<T>(a, i));
                if (MODE == 1) w -= as_f(raw_get<T>(b, i));
                if (MODE == 2 && v + i == draft) w = 0.0f;
                offer(best, w, raw_get<float>(n[i / 4], i % 4), (uint32_t)(v + i));
            }
        }
        first = full;
    }
    // rows that 16-byte loads do not fit, and a row's end: one value a load,
    // kOnce of them in flight (the candidates' branches would keep the
    // compiler from starting one before the last is done with)
    constexpr int kOnce = 6;
    for (int64_t v = first + threadIdx.x; v < last; v += kOnce * kThreads) {
        float w[kOnce], x[kOnce], n[kOnce];
#pragma unroll
        for (int i = 0; i < kOnce; ++i) {
            const int64_t at = min(v + i * kThreads, last - 1);
            w[i] = as_f(p[at]);
            if (MODE == 1) x[i] = as_f(q[at]);
            n[i] = e[at];
        }
#pragma unroll
        for (int i = 0; i < kOnce; ++i) {
            const int64_t at = v + i * kThreads;
            if (MODE == 1) w[i] -= x[i];
            if (MODE == 2 && at == draft) w[i] = 0.0f;
            if (at < last) offer(best, w[i], n[i], (uint32_t)at);
        }
    }
    return best;
}

template <class T>
__global__ void __launch_bounds__(kThreads, kBlocksPerSm) k_verify(const VerifyCall c) {
    __shared__ uint64_t s_warp[kThreads / kWarp];
    __shared__ uint64_t s_best[2];
    __shared__ int s_taken, s_count;
    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), parts = (int)cl.num_blocks();
    const int64_t r = blockIdx.x / parts;
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    const T* p = static_cast<const T*>(c.p) + r * c.p_req;
    const T* q = c.q ? static_cast<const T*>(c.q) + r * c.q_req : nullptr;
    const float* e = c.noise + r * c.noise_stride;
    const int32_t* d = c.drafts + r * c.k;

    if (warp == 0) {
        // the first loads do not wait for the count
        int64_t t = lane < c.k ? d[lane] : -1;
        float u = lane < c.k ? c.uniform[r * c.k + lane] : 0.0f;
        int m = c.counts ? c.counts[r] : c.k;
        m = max(0, min(m, c.k));
        int taken = m;
        for (int j0 = 0; j0 < m; j0 += kWarp) {
            const int j = j0 + lane;
            if (j0 > 0 && j < m) t = d[j], u = c.uniform[r * c.k + j];
            bool ok = j < m && t >= 0 && t < c.vocab;
            if (ok) {
                const float pv = as_f(p[j * c.p_row + t]);
                const float qv = q ? as_f(q[j * c.q_row + t]) : 1.0f;
                ok = (double)u * qv < pv;  // exact: a rounded product may equal p and not be it
            }
            const unsigned refused = __ballot_sync(0xffffffffu, !ok && j < m);
            if (refused) {
                taken = j0 + __ffs(refused) - 1;
                break;
            }
        }
        if (lane == 0) {
            s_taken = taken;
            s_count = m;
        }
    }
    __syncthreads();
    const int taken = s_taken;
    const bool refused = taken < s_count;
    const T* row = p + taken * c.p_row;
    const T* qrow = refused && q ? q + taken * c.q_row : nullptr;
    const int64_t draft = refused && !q ? d[taken] : -1;
    constexpr int64_t kAlign = 16 / (int64_t)sizeof(T);
    const int64_t slice = ((c.vocab + parts - 1) / parts + kAlign - 1) / kAlign * kAlign;
    const int64_t first = min((int64_t)rank * slice, c.vocab), last = min(first + slice, c.vocab);
    const bool vec = ((reinterpret_cast<uintptr_t>(row) | reinterpret_cast<uintptr_t>(e) |
                       (qrow ? reinterpret_cast<uintptr_t>(qrow) : 0)) & 15) == 0;

    uint64_t best = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
        if (pass == 0 && qrow) best = fold<T, 1>(row, qrow, e, first, last, -1, vec);
        else if (pass == 0 && draft >= 0) best = fold<T, 2>(row, nullptr, e, first, last, draft, vec);
        else best = fold<T, 0>(row, nullptr, e, first, last, -1, vec);
#pragma unroll
        for (int s = kWarp / 2; s > 0; s >>= 1) {
            const uint64_t o = __shfl_down_sync(0xffffffffu, best, s);
            if (o > best) best = o;
        }
        if (lane == 0) s_warp[warp] = best;
        __syncthreads();
        if (warp == 0) {
            best = lane < kThreads / kWarp ? s_warp[lane] : 0;
#pragma unroll
            for (int s = kWarp / 2; s > 0; s >>= 1) {
                const uint64_t o = __shfl_down_sync(0xffffffffu, best, s);
                if (o > best) best = o;
            }
            if (lane == 0) s_best[pass] = best;
        }
        cl.sync();
        best = 0;
        for (int b = 0; b < parts; ++b) {
            const uint64_t o = *cl.map_shared_rank(&s_best[pass], b);
            if (o > best) best = o;
        }
        // nothing left of the difference: the target's own row
        if (best != 0 || !refused) break;
    }
    if (rank == 0) {
        int32_t* out = c.tokens + r * (c.k + 1);
        for (int j = threadIdx.x; j <= c.k; j += kThreads) {
            int32_t t = -1;
            if (j < taken) t = d[j];
            else if (j == taken && best != 0) t = (int32_t)(0xffffffffu - (uint32_t)best);
            out[j] = t;
        }
        if (threadIdx.x == 0) c.accepted[r] = taken;
    }
    cl.sync();  // every block has read the others' shared memory
}

}  // namespace vd

ak_status run_verify(const VerifyCall& c, cudaStream_t stream) {
    using namespace vd;
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    // blocks of a request: as many as run at once over all requests (three an
    // SM), each with at least one round of vector loads. 192 requests of
    // 128000 float32: 2 blocks 45 us, 4 blocks (a second wave) 51, 8 blocks 60.
    int parts = 1;
    while (parts < 8 && c.nreq * parts * 2 <= kBlocksPerSm * dev.sm_count && c.vocab / (2 * parts) >= kThreads * 4) parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(c.nreq * parts));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)parts;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = c.dtype == AK_F32 ? cudaLaunchKernelEx(&cfg, k_verify<float>, c)
                                            : cudaLaunchKernelEx(&cfg, k_verify<bf16>, c);
    if (e != cudaSuccess) return cuda_fail(e);
    count_launches(1);
    return check_launch();
}

}  // namespace ak
