// blocks.cu -- what a paged cache's blocks need when requests fork, end or
// change places: counts of references, fork with copy on write, the list of
// free blocks, compaction of the pool, copies of blocks.
//
// A request of len tokens holds the first ceil(len / b) entries of its row of
// the block table; a block may be held by several requests. How often a block
// is held is what the tables say, so no count is kept between calls:
//   refs[i]  = number of held entries that are i               (a histogram)
//   free     = the i with refs[i] == 0, in order                (stream compaction)
//   fork     = rows by parents; of the requests that end in the same partly
//              filled block all but one (or all, if it is held otherwise too) get
//              a block of their own, in order from the free list
//              (a scan of flags)
//   compact  = the n blocks in use move to 0 .. n-1: the i-th that lies past n to the
//              i-th hole before it                             (two scans of one count)
// The four that compute on tables are each one launch of one cluster of up to
// 16 blocks of 1024 threads, whose phases the cluster's barrier separates: such
// tables are some hundred KB, and a second launch would cost more than the rest of the
// device could save. Histogram and ownership use integer atomics, whose order
// does not show. Only the copies touch the pool's bytes; they take the whole device.
//
// Bound by latency: 8 requests / 512 requests of up to 250 blocks (a pool of 54920):
// fork 8.9 / 16.4 us, free list 4.7 / 8.3; 16 / 256 requests (304 / 64000 blocks): count
// 3.4 / 7.3, compaction 8.8 / 15.4. Copies: 143 blocks of 2 x 8 KB 3.1 us, 16024 of 8 KB
// 44 us (0.88 of the copy bandwidth).
#include <algorithm>
#include <cooperative_groups.h>

#include "ak_common.cuh"
#include "ak_internal.h"

namespace cg = cooperative_groups;

namespace ak {
namespace bk {

constexpr int kThreads = 1024;
constexpr int kWarps = kThreads / kWarp;
constexpr int kPart = 128;      // table entries a warp takes at a time
constexpr int kCopyThreads = 256;
constexpr int kCopyUnroll = 4;

// The cluster as one team of threads.
struct Team {
    int rank, size;
    __device__ __forceinline__ Team() {
        cg::cluster_group cl = cg::this_cluster();
        rank = (int)cl.block_rank(), size = (int)cl.num_blocks();
    }
    // every thread's writes before it are visible to every thread after it
    __device__ __forceinline__ void sync() const {
        __threadfence();
        cg::this_cluster().sync();
    }
    __device__ __forceinline__ int64_t thread() const { return (int64_t)rank * kThreads + threadIdx.x; }
    __device__ __forceinline__ int64_t threads() const { return (int64_t)size * kThreads; }
    __device__ __forceinline__ int64_t warp() const { return thread() / kWarp; }
    __device__ __forceinline__ int64_t warps() const { return threads() / kWarp; }
    // this block's share of n, in whole rounds of `grain`
    __device__ __forceinline__ void share(int64_t n, int64_t grain, int64_t& first, int64_t& last) const {
        const int64_t per = ((n + size - 1) / size + grain - 1) / grain * grain;
        first = min(per * rank, n), last = min(first + per, n);
    }
};

// What other blocks wrote in this launch is read past L1.
__device__ __forceinline__ int32_t ld_shared(const int32_t* p) { return __ldcg(p); }

// Entries that a request of `len` tokens holds.
__device__ __forceinline__ int64_t held(int32_t len, int32_t block, int64_t width) {
    return len <= 0 ? 0 : min(((int64_t)len + block - 1) / block, width);
}

// Pieces of a row that a warp takes; at least one, as a row without entries has a length.
__device__ __forceinline__ int64_t row_parts(int64_t width) { return max((int64_t)1, (width + kPart - 1) / kPart); }

// Exclusive sum over the block's threads and the total. Ends in sync.
__device__ __forceinline__ int block_scan(int v, int* s_warp, int& total) {
    const int lane = threadIdx.x % kWarp, warp = threadIdx.x / kWarp;
    int incl = v;
#pragma unroll
    for (int d = 1; d < kWarp; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == kWarp - 1) s_warp[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int w = s_warp[lane];
#pragma unroll
        for (int d = 1; d < kWarp; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, w, d);
            if (lane >= d) w += o;
        }
        s_warp[lane] = w;
    }
    __syncthreads();
    const int before = warp ? s_warp[warp - 1] : 0;
    total = s_warp[kWarps - 1];
    __syncthreads();
    return before + incl - v;
}

struct Sums {
    int warp[kWarps];
    int part[16];  // what each block of the cluster counted
};

// Hands `count` to every block; after the team's sync sums.part holds all.
__device__ __forceinline__ void publish(Sums& sums, const Team& team, int count) {
    if ((int)threadIdx.x < team.size)
        cg::this_cluster().map_shared_rank(&sums, threadIdx.x)->part[team.rank] = count;
}

// ---------------------------------------------------------------------------
// counts
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads) k_blocks_count(const BlocksCall c) {
    const Team team;
    for (int64_t i = team.thread(); i < c.blocks; i += team.threads()) c.refs[i] = 0;
    team.sync();
    const int lane = threadIdx.x % kWarp;
    const int64_t parts = row_parts(c.width);
    for (int64_t w = team.warp(); w < c.rows * parts; w += team.warps()) {
        const int64_t r = div_fast(w, parts), col = (w - r * parts) * kPart;
        const int64_t end = min(held(c.lens[r], c.block_size, c.width), col + kPart);
        const int32_t* row = c.table + r * c.table_stride;
        for (int64_t i = col + lane; i < end; i += kWarp) {
            const int32_t id = row[i];
            if (id >= 0 && id < c.blocks) atomicAdd(c.refs + id, 1);
        }
    }
}

// ---------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads) k_blocks_fork(const BlocksCall c) {
    __shared__ Sums sums;
    const Team team;
    const int lane = threadIdx.x % kWarp;
    // owner: rows - the lowest row that ends in the block, or 0; ends: how many do
    int32_t *owner = c.work, *ends = owner + c.blocks, *copied = ends + c.blocks;
    for (int64_t i = team.thread(); i < c.blocks; i += team.threads()) c.refs[i] = owner[i] = ends[i] = 0;
    for (int64_t i = team.thread(); i < 2 * c.rows; i += team.threads()) c.pairs[i] = -1;
    team.sync();

    const int64_t parts = row_parts(c.width);
    for (int64_t w = team.warp(); w < c.rows * parts; w += team.warps()) {
        const int64_t r = div_fast(w, parts), part = w - r * parts, col = part * kPart;
        const int32_t p = c.parents[r];
        const bool live = p >= 0 && p < c.old_rows;
        const int32_t len = live ? max(c.lens[p], 0) : 0;
        const int64_t used = held(len, c.block_size, c.width);
        const int32_t* row = c.table + (int64_t)p * c.table_stride;
        int32_t* to = c.out_table + r * c.out_stride;
        for (int64_t i = col + lane; i < min(col + kPart, (int64_t)c.width); i += kWarp) {
            const int32_t id = i < used ? row[i] : -1;
            to[i] = id;
            if (i < used && id >= 0 && id < c.blocks) {
                atomicAdd(c.refs + id, 1);
                if (i == len / c.block_size && len % c.block_size) {
                    atomicMax(owner + id, (int32_t)(c.rows - r));
                    atomicAdd(ends + id, 1);
                }
            }
        }
        if (part == 0 && lane == 0) c.out_lens[r] = len;
    }
    team.sync();

    // ---- which rows copy their last block; decided before any count changes
    int64_t first, last;
    team.share(c.rows, 1, first, last);
    int mine = 0;
    for (int64_t r = first + threadIdx.x; r < last; r += kThreads) {
        const int32_t len = ld_shared(c.out_lens + r), col = len / c.block_size;
        int32_t id = -1;
        if (len % c.block_size && col < c.width) id = ld_shared(c.out_table + r * c.out_stride + col);
        const bool copy = id >= 0 && id < c.blocks &&
                          !(c.rows - ld_shared(owner + id) == r && ld_shared(c.refs + id) <= ld_shared(ends + id));
        copied[r] = copy ? id : -1;
        mine += copy;
    }
    int total;
    block_scan(mine, sums.warp, total);
    publish(sums, team, total);
    team.sync();

    int64_t at = 0, all = 0;
    for (int p = 0; p < team.size; ++p) {
        if (p < team.rank) at += sums.part[p];
        all += sums.part[p];
    }
    if (team.thread() == 0) c.counts[0] = (int32_t)all;
    for (int64_t r0 = first; r0 < last; r0 += kThreads) {
        const int64_t r = r0 + threadIdx.x;
        const int32_t id = r < last ? copied[r] : -1;
        const int64_t i = at + block_scan(id >= 0, sums.warp, total);
        if (id >= 0) {
            int32_t to = i < c.nfree ? c.free_blocks[i] : -1;
            if (to >= c.blocks) to = -1;
            c.out_table[r * c.out_stride + ld_shared(c.out_lens + r) / c.block_size] = to < 0 ? -1 : to;
            atomicAdd(c.refs + id, -1);
            if (to >= 0) {
                atomicAdd(c.refs + to, 1);
                c.pairs[2 * i] = id;
                c.pairs[2 * i + 1] = to;
            }
        }
        at += total;
    }
}

// ---------------------------------------------------------------------------
// free list
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads) k_blocks_free(const BlocksCall c) {
    __shared__ Sums sums;
    const Team team;
    int64_t first, last;
    team.share(c.blocks, kWarp, first, last);
    int mine = 0, total;
    for (int64_t i = first + threadIdx.x; i < last; i += kThreads) mine += c.refs[i] <= 0;
    block_scan(mine, sums.warp, total);
    team.sync();  // every block of the cluster runs
    publish(sums, team, total);
    team.sync();
    int64_t at = 0, all = 0;
    for (int p = 0; p < team.size; ++p) {
        if (p < team.rank) at += sums.part[p];
        all += sums.part[p];
    }
    if (team.thread() == 0) c.counts[0] = (int32_t)all;
    for (int64_t i0 = first; i0 < last; i0 += kThreads) {
        const int64_t i = i0 + threadIdx.x;
        const bool free = i < last && c.refs[i] <= 0;
        const int64_t to = at + block_scan(free, sums.warp, total);
        if (free) c.out_free[to] = (int32_t)i;
        at += total;
    }
    for (int64_t i = all + team.thread(); i < c.blocks; i += team.threads()) c.out_free[i] = -1;
}

// ---------------------------------------------------------------------------
// compaction
// ---------------------------------------------------------------------------

__global__ void __launch_bounds__(kThreads) k_blocks_compact(const BlocksCall c) {
    __shared__ Sums sums;
    const Team team;
    const int64_t most = c.blocks / 2;  // moves: as many as holes before, and blocks after, the n-th
    int32_t *holes = c.work, *movers = holes + most, *to = movers + most;
    int64_t first, last;
    team.share(c.blocks, kWarp, first, last);
    int mine = 0, total;
    for (int64_t i = first + threadIdx.x; i < last; i += kThreads) mine += c.refs[i] > 0;
    block_scan(mine, sums.warp, total);
    team.sync();  // every block of the cluster runs
    publish(sums, team, total);
    team.sync();
    int64_t at = 0, n = 0;
    for (int p = 0; p < team.size; ++p) {
        if (p < team.rank) at += sums.part[p];
        n += sums.part[p];
    }
    team.sync();  // all have read the counts: they are published once more below
    // ---- holes before the n-th block by rank; blocks in use from there on by
    // how many follow
    int past = 0;
    for (int64_t i0 = first; i0 < last; i0 += kThreads) {
        const int64_t i = i0 + threadIdx.x;
        const bool used = i < last && c.refs[i] > 0;
        const int64_t before = at + block_scan(used, sums.warp, total);
        if (i < last && !used && i < n) holes[i - before] = (int32_t)i;
        if (used && i >= n) {
            movers[n - 1 - before] = (int32_t)i;
            ++past;
        }
        at += total;
    }
    block_scan(past, sums.warp, total);
    publish(sums, team, total);
    team.sync();
    int64_t moves = 0;
    for (int p = 0; p < team.size; ++p) moves += sums.part[p];
    if (team.thread() == 0) {
        c.counts[0] = (int32_t)moves;
        c.counts[1] = (int32_t)n;
    }
    for (int64_t i = team.thread(); i < most; i += team.threads()) {
        int32_t a = -1, b = -1;
        if (i < moves) {
            a = ld_shared(movers + (moves - 1 - i));
            b = ld_shared(holes + i);
            to[a] = b;
        }
        c.pairs[2 * i] = a;
        c.pairs[2 * i + 1] = b;
    }
    team.sync();
    // ---- the table's entries
    const int lane = threadIdx.x % kWarp;
    const bool in_place = c.out_table == c.table;
    const int64_t parts = row_parts(c.width);
    for (int64_t w = team.warp(); w < c.rows * parts; w += team.warps()) {
        const int64_t r = div_fast(w, parts), col = (w - r * parts) * kPart;
        const int64_t used = held(c.lens[r], c.block_size, c.width);
        const int64_t end = min(col + kPart, in_place ? used : (int64_t)c.width);
        const int32_t* row = c.table + r * c.table_stride;
        int32_t* out = c.out_table + r * c.out_stride;
        for (int64_t i = col + lane; i < end; i += kWarp) {
            int32_t id = row[i];
            if (i < used && id >= n && id < c.blocks && c.refs[id] > 0) id = ld_shared(to + id);
            out[i] = id;
        }
    }
}

// ---------------------------------------------------------------------------
// copies
// ---------------------------------------------------------------------------

template <class U>
__global__ void __launch_bounds__(kCopyThreads) k_blocks_copy(const BlocksCopyCall c) {
    constexpr int64_t kSpan = (int64_t)kCopyThreads * kCopyUnroll;
    const int64_t units = c.inner / (int64_t)sizeof(U), chunks = (units + kSpan - 1) / kSpan;
    int64_t pairs = c.npairs;
    if (c.count) pairs = min(pairs, (int64_t)max(c.count[0], 0));
    const int64_t all = pairs * c.outer * chunks;
    for (int64_t w = blockIdx.x; w < all; w += gridDim.x) {
        const int64_t q = div_fast(w, chunks), first = (w - q * chunks) * kSpan + threadIdx.x;
        const int64_t o = div_fast(q, pairs), i = q - o * pairs;
        const int32_t a = c.pairs[2 * i], b = c.pairs[2 * i + 1];
        if (a < 0 || b < 0 || a >= c.blocks || b >= c.blocks || a == b) continue;
        char* base = static_cast<char*>(c.cache) + o * c.outer_stride;
        const U* from = reinterpret_cast<const U*>(base + a * c.block_stride);
        U* to = reinterpret_cast<U*>(base + b * c.block_stride);
        U v[kCopyUnroll];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (first + u * kCopyThreads < units) v[u] = from[first + u * kCopyThreads];
#pragma unroll
        for (int u = 0; u < kCopyUnroll; ++u)
            if (first + u * kCopyThreads < units) to[first + u * kCopyThreads] = v[u];
    }
}

template <class U>
void launch_copy(const BlocksCopyCall& c, int sm_count, cudaStream_t stream) {
    constexpr int64_t kSpan = (int64_t)kCopyThreads * kCopyUnroll;
    const int64_t chunks = (c.inner / (int64_t)sizeof(U) + kSpan - 1) / kSpan;
    // the count of pairs is on the device: one wave at most
    const int64_t grid = std::min<int64_t>((int64_t)sm_count * 8, std::min<int64_t>(c.npairs, 1 << 20) * std::min<int64_t>(c.outer * chunks, 1 << 20));
    k_blocks_copy<U><<<(unsigned)grid, kCopyThreads, 0, stream>>>(c);
}

// One cluster of as many blocks as the work keeps busy.
ak_status launch(void (*kernel)(BlocksCall), ClusterLimit& limit, const BlocksCall& c, int64_t work, cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    int most = 0;
    const ak_status s = limit.get(reinterpret_cast<const void*>(kernel), kThreads, dev.device, &most);
    if (s != AK_OK) return s;
    int size = 1;
    while (size < most && work > (int64_t)size * kThreads) size *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)size);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)size;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, c);
    if (e != cudaSuccess) return cuda_fail(e);
    count_launches(1);
    return check_launch();
}

}  // namespace bk

size_t blocks_fork_workspace(int64_t rows, int64_t blocks) {
    return kWsHeader + align_up((size_t)(2 * blocks + rows) * 4, 256);
}
size_t blocks_compact_workspace(int64_t blocks) { return kWsHeader + align_up((size_t)(2 * (blocks / 2) + blocks) * 4, 256); }

ak_status run_blocks_count(const BlocksCall& c, cudaStream_t stream) {
    static ClusterLimit limit;
    return bk::launch(bk::k_blocks_count, limit, c, std::max(c.rows * c.width, c.blocks), stream);
}
ak_status run_blocks_fork(BlocksCall c, void* ws, cudaStream_t stream) {
    static ClusterLimit limit;
    c.work = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kWsHeader);
    return bk::launch(bk::k_blocks_fork, limit, c, std::max(c.rows * c.width, c.blocks), stream);
}
ak_status run_blocks_free(const BlocksCall& c, cudaStream_t stream) {
    static ClusterLimit limit;
    return bk::launch(bk::k_blocks_free, limit, c, c.blocks, stream);
}
ak_status run_blocks_compact(BlocksCall c, void* ws, cudaStream_t stream) {
    static ClusterLimit limit;
    c.work = reinterpret_cast<int32_t*>(static_cast<char*>(ws) + kWsHeader);
    return bk::launch(bk::k_blocks_compact, limit, c, std::max(c.rows * c.width, c.blocks), stream);
}
ak_status run_blocks_copy(const BlocksCopyCall& c, cudaStream_t stream) {
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    const uint64_t bits = (uint64_t)reinterpret_cast<uintptr_t>(c.cache) | (uint64_t)c.inner | (uint64_t)c.block_stride |
                          (uint64_t)c.outer_stride;
    if (bits % 16 == 0) bk::launch_copy<int4>(c, dev.sm_count, stream);
    else if (bits % 4 == 0) bk::launch_copy<int32_t>(c, dev.sm_count, stream);
    else bk::launch_copy<int8_t>(c, dev.sm_count, stream);
    count_launches(1);
    return check_launch();
}

}  // namespace ak
