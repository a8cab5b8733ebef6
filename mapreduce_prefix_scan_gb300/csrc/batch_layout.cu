// batch_layout.cu -- block tables, slot maps and packed offsets of a batch,
// built on the device from the requests' lengths.
//
// With ctx_r tokens of request r in the paged cache, new_r tokens to run and
// blocks of b tokens:
//   offsets[r]  = sum_{s<r} new_s                       (exclusive scan)
//   have_r      = ceil(ctx_r / b),  want_r = ceil((ctx_r + new_r) / b)
//   base_r      = sum_{s<r} (want_s - have_s)           (exclusive scan)
//   table[r][c] = free[base_r + c - have_r]             for have_r <= c < want_r
//   token t of request r (the r with offsets[r] <= t < offsets[r+1]):
//   pos = ctx_r + t - offsets[r],  slot = table[r][pos / b] * b + pos % b
//
// Both scans are one scan of packed pairs. Up to kSmallReqs requests one
// launch does everything: every block scans all lengths itself (16 KB at
// 2047 requests, from L2) and keeps both prefixes in shared memory, which is
// cheaper than a second launch that waits for the first; then it expands its
// share of the token axis, four consecutive tokens a thread (16-byte stores)
// after one binary search in shared memory. Slots of new blocks come from
// the free list directly, so no block waits for another's table entries.
// More requests take three launches: tile sums, prefixes, expansion.
//
// Bound by latency (a launch, two dependent loads, the block scan: 6.5 us for
// 256 requests of a token each, back to back) and, for a million tokens, by
// the instructions that expand them (12 us; 13 with blocks of 24 tokens, which
// divide; 16 MB are 2.4 us of HBM). 9000 requests, in three launches: 29 us
// with a token each, 62 with a million tokens.
#include <algorithm>
#include <atomic>

#include "ak_common.cuh"
#include "ak_internal.h"

namespace ak {
namespace bl {

constexpr int kThreads = 512;
constexpr int kPer = 8;                         // requests a thread scans
constexpr int kSmallReqs = kThreads * kPer;     // requests one block scans
constexpr int kTok = 4;                         // consecutive tokens a thread writes

// (new tokens, new blocks) of a range of requests, added as one word: both
// sums stay below 2^31, so the low half never carries into the high one.
__device__ __forceinline__ uint64_t pack(uint32_t tokens, uint32_t blocks) {
    return ((uint64_t)blocks << 32) | tokens;
}

struct Req {
    int ctx, fresh, have, want;
};

// Blocks that `tokens` fill. 32-bit, and a shift for powers of two: 64-bit
// divisions of every length in every block were half of this kernel's
// instructions.
__device__ __forceinline__ int blocks_of(const LayoutCall& c, uint32_t tokens) {
    const uint32_t b = (uint32_t)c.block_size;
    if (c.block_shift >= 0) return (int)((tokens >> c.block_shift) + ((tokens & (b - 1)) != 0));
    return (int)(tokens / b + (tokens % b != 0));
}

__device__ __forceinline__ Req request(const LayoutCall& c, int64_t r) {
    Req q;
    q.ctx = max(c.ctx_lens[r], 0);
    q.fresh = max(c.new_lens[r], 0);
    q.have = blocks_of(c, (uint32_t)q.ctx);
    q.want = blocks_of(c, (uint32_t)q.ctx + (uint32_t)q.fresh);
    return q;
}

// Inclusive block scan of one packed pair a thread.
__device__ __forceinline__ uint64_t block_scan(uint64_t v, uint64_t* s_warp) {
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    if (lane == kWarp - 1) s_warp[warp] = v;
    __syncthreads();
    uint64_t before = 0;
#pragma unroll
    for (int w = 0; w < kThreads / kWarp; ++w)
        if (w < warp) before += s_warp[w];
    __syncthreads();
    return v + before;
}

// New table entries of request r, one lane an entry.
__device__ __forceinline__ void append(const LayoutCall& c, int64_t r, const Req& q, uint32_t base, int lane, int lanes) {
    int32_t* row = c.table + r * c.table_stride;
    const int end = min(q.want, c.table_width);
    for (int col = q.have + lane; col < end; col += lanes) {
        const int64_t at = (int64_t)base + (col - q.have);
        row[col] = at < c.nfree ? c.free_blocks[at] : -1;
    }
}

// Slot of position pos of request r (ctx tokens already there, its new
// blocks starting at free[base]); -1 past the table or the free list.
__device__ __forceinline__ int64_t slot_of(const LayoutCall& c, int64_t r, int pos, int have, uint32_t base) {
    const int b = c.block_size;
    const int col = (c.block_shift >= 0) ? pos >> c.block_shift : pos / b;
    if ((unsigned)col >= (unsigned)c.table_width) return -1;
    int32_t id;
    if (col < have) {
        id = c.table[r * c.table_stride + col];
    } else {
        const int64_t at = (int64_t)base + (col - have);
        id = at < c.nfree ? c.free_blocks[at] : -1;
    }
    return id < 0 ? -1 : (int64_t)id * b + (pos - col * b);
}

// Tokens [first, last) of the token axis, kTok a thread. off, base: prefix
// arrays over the requests; ctx_of: their cached lengths (shared or global
// memory).
__device__ __forceinline__ void expand(const LayoutCall& c, const int32_t* off, const int32_t* base,
                                       const int32_t* ctx_of, int64_t first, int64_t last) {
    const int64_t n = c.nreq;
    const int64_t total = off[n];
    for (int64_t t0 = first + (int64_t)threadIdx.x * kTok; t0 < last; t0 += (int64_t)kThreads * kTok) {
        int64_t slot[kTok];
        int32_t pos[kTok], req[kTok];
        // the last r with off[r] <= t0 (requests without tokens are skipped)
        int64_t lo = 0, hi = n;
        if (t0 < total) {
            while (hi - lo > 1) {
                const int64_t mid = (lo + hi) >> 1;
                if (off[mid] <= t0) lo = mid;
                else hi = mid;
            }
        }
        int64_t r = lo;
        int64_t held = -1;
        int ctx = 0, have = 0, start = 0;
        uint32_t bs = 0;
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            const int64_t t = t0 + i;
            slot[i] = -1;
            pos[i] = 0;
            req[i] = -1;
            if (t < total && t < last) {
                while (r + 1 < n && off[r + 1] <= t) ++r;
                if (r != held) {
                    held = r;
                    ctx = max(ctx_of[r], 0);
                    have = blocks_of(c, (uint32_t)ctx);
                    start = off[r];
                    bs = (uint32_t)base[r];
                }
                pos[i] = ctx + (int)(t - start);
                req[i] = (int32_t)r;
                slot[i] = slot_of(c, r, pos[i], have, bs);
            }
        }
        if (c.vec && t0 + kTok <= last) {
            *reinterpret_cast<int4*>(c.positions + t0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
            *reinterpret_cast<int4*>(c.requests + t0) = make_int4(req[0], req[1], req[2], req[3]);
            *reinterpret_cast<longlong2*>(c.slots + t0) = make_longlong2(slot[0], slot[1]);
            *reinterpret_cast<longlong2*>(c.slots + t0 + 2) = make_longlong2(slot[2], slot[3]);
        } else {
            for (int i = 0; i < kTok && t0 + i < last; ++i) {
                c.positions[t0 + i] = pos[i];
                c.requests[t0 + i] = req[i];
                c.slots[t0 + i] = slot[i];
            }
        }
    }
}

// Scans requests [first, first + kThreads * per), per <= kPer of them a
// thread; off and base receive the prefixes, keep_ctx (where given) the
// cached lengths. Returns this thread's inclusive sum after its last request.
__device__ __forceinline__ uint64_t scan_tile(const LayoutCall& c, int64_t first, int per, uint64_t carry, int32_t* off,
                                              int32_t* base, int32_t* keep_ctx, uint64_t* s_warp) {
    uint64_t v[kPer], sum = 0;
    const int64_t r0 = first + (int64_t)threadIdx.x * per;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        v[i] = 0;
        if (i < per && r0 + i < c.nreq) {
            const Req q = request(c, r0 + i);
            v[i] = pack((uint32_t)q.fresh, (uint32_t)(q.want - q.have));
            if (keep_ctx) keep_ctx[r0 + i] = q.ctx;
        }
        sum += v[i];
    }
    const uint64_t incl = block_scan(sum, s_warp) + carry;
    uint64_t run = incl - sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        if (i < per && r0 + i < c.nreq && off) {
            off[r0 + i] = (int32_t)(uint32_t)run;
            base[r0 + i] = (int32_t)(run >> 32);
        }
        run += v[i];
    }
    return incl;
}

__global__ void __launch_bounds__(kThreads) k_layout_small(const LayoutCall c) {
    __shared__ uint64_t s_warp[kThreads / kWarp];
    extern __shared__ int32_t s_pre[];  // off[nreq + 1], base[nreq + 1], ctx[nreq]
    const int n = (int)c.nreq;
    int32_t* off = s_pre;
    int32_t* base = off + n + 1;
    int32_t* ctx = base + n + 1;
    const uint64_t incl = scan_tile(c, 0, (n + kThreads - 1) / kThreads, 0, off, base, ctx, s_warp);
    if (threadIdx.x == kThreads - 1) {
        off[n] = (int32_t)(uint32_t)incl;
        base[n] = (int32_t)(incl >> 32);
    }
    __syncthreads();
    if (blockIdx.x == 0) {
        for (int r = threadIdx.x; r <= n; r += kThreads) c.offsets[r] = off[r];
        if (threadIdx.x == 0) {
            c.counts[0] = off[n];
            c.counts[1] = base[n];
        }
    }
    // new table entries: a group of 8 lanes a request
    constexpr int G = 8;
    for (int64_t r = (int64_t)blockIdx.x * (kThreads / G) + threadIdx.x / G; r < n;
         r += (int64_t)gridDim.x * (kThreads / G)) {
        const Req q = request(c, r);
        append(c, r, q, (uint32_t)base[r], threadIdx.x % G, G);
    }
    const int64_t first = (int64_t)blockIdx.x * c.tokens_per_block;
    expand(c, off, base, ctx, first, min(first + c.tokens_per_block, c.max_tokens));
}

__global__ void __launch_bounds__(kThreads) k_layout_sums(const LayoutCall c) {
    __shared__ uint64_t s_warp[kThreads / kWarp];
    const uint64_t incl = scan_tile(c, (int64_t)blockIdx.x * kSmallReqs, kPer, 0, nullptr, nullptr, nullptr, s_warp);
    if (threadIdx.x == kThreads - 1) c.tile_sums[blockIdx.x] = incl;
}

__global__ void __launch_bounds__(kThreads) k_layout_prefix(const LayoutCall c) {
    __shared__ uint64_t s_warp[kThreads / kWarp];
    __shared__ uint64_t s_carry;
    // fold of the earlier tiles' sums
    uint64_t v = 0;
    for (int64_t i = threadIdx.x; i < blockIdx.x; i += kThreads) v += c.tile_sums[i];
    v = block_scan(v, s_warp);
    if (threadIdx.x == kThreads - 1) s_carry = v;
    __syncthreads();
    const int64_t first = (int64_t)blockIdx.x * kSmallReqs;
    const uint64_t incl = scan_tile(c, first, kPer, s_carry, c.offsets, c.base, nullptr, s_warp);
    if (blockIdx.x == gridDim.x - 1 && threadIdx.x == kThreads - 1) {
        c.offsets[c.nreq] = (int32_t)(uint32_t)incl;
        c.counts[0] = (int32_t)(uint32_t)incl;
        c.counts[1] = (int32_t)(incl >> 32);
    }
    __syncthreads();  // this block's base values are visible to its threads
    constexpr int G = 8;
    const int64_t end = min(first + kSmallReqs, c.nreq);
    for (int64_t r = first + threadIdx.x / G; r < end; r += kThreads / G)
        append(c, r, request(c, r), (uint32_t)c.base[r], threadIdx.x % G, G);
}

__global__ void __launch_bounds__(kThreads) k_layout_expand(const LayoutCall c) {
    const int64_t first = (int64_t)blockIdx.x * c.tokens_per_block;
    expand(c, c.offsets, c.base, c.ctx_lens, first, min(first + c.tokens_per_block, c.max_tokens));
}

}  // namespace bl

size_t layout_workspace(int64_t nreq) {
    if (nreq <= bl::kSmallReqs) return kWsHeader;
    const int64_t tiles = (nreq + bl::kSmallReqs - 1) / bl::kSmallReqs;
    return kWsHeader + align_up((size_t)tiles * 8, 256) + align_up((size_t)nreq * 4, 256);
}

ak_status run_layout(LayoutCall c, void* ws, cudaStream_t stream) {
    using namespace bl;
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    // blocks of one pass over their tokens, at most two an SM
    const int64_t per = (int64_t)kThreads * kTok;
    int64_t grid = std::max<int64_t>(1, std::min<int64_t>((c.max_tokens + per - 1) / per, 2 * dev.sm_count));
    c.tokens_per_block = align_up((size_t)((c.max_tokens + grid - 1) / grid), kTok);
    if (c.nreq <= kSmallReqs) {
        const size_t smem = (3 * (size_t)c.nreq + 2) * 4;
        static std::atomic<uint64_t> ready{0};
        if (smem > 40 * 1024 && !(ready.load() >> dev.device & 1)) {
            const cudaError_t e = cudaFuncSetAttribute(k_layout_small, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                       (3 * kSmallReqs + 2) * 4);
            if (e != cudaSuccess) return cuda_fail(e);
            ready.fetch_or(1ull << dev.device);
        }
        k_layout_small<<<(unsigned)grid, kThreads, smem, stream>>>(c);
        count_launches(1);
        return check_launch();
    }
    const int64_t tiles = (c.nreq + kSmallReqs - 1) / kSmallReqs;
    char* w = static_cast<char*>(ws) + kWsHeader;
    c.tile_sums = reinterpret_cast<uint64_t*>(w);
    c.base = reinterpret_cast<int32_t*>(w + align_up((size_t)tiles * 8, 256));
    k_layout_sums<<<(unsigned)tiles, kThreads, 0, stream>>>(c);
    k_layout_prefix<<<(unsigned)tiles, kThreads, 0, stream>>>(c);
    k_layout_expand<<<(unsigned)grid, kThreads, 0, stream>>>(c);
    count_launches(3);
    return check_launch();
}

}  // namespace ak
