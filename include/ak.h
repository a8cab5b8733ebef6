/*
 * ak.h -- C ABI of the GB300 (sm_103a) device-wide reduce / prefix-scan library.
 *
 * Three operations, as stated in the AcceleratedKernels.jl pull requests
 * this library re-designs for GB300:
 *
 *   ak_reduce       whole-array mapreduce(f, op, A) into a host scalar or a
 *                   one-element device array ("Finish whole-array reductions
 *                   on the device", PR #139, sections "What changes" and
 *                   "Compatibility");
 *   ak_reduce_dims  mapreducedim!(f, op, R, A) over a set of dimensions of a
 *                   dense column-major array, e.g. sum(x; dims=2) of a matrix
 *                   or of the middle dimension of a 3-d array (strided
 *                   reduction PR #176, first two lists);
 *   ak_accumulate   accumulate!(op, dst, src) / cumsum: the inclusive scan of
 *                   the whole array or along one dimension, including
 *                   operators with no neutral element and non-commutative
 *                   ones (tile-scan PR #202, first paragraph and paragraph
 *                   "Alternatives").
 *
 * More of them carry the same scans and folds into sequence models: the
 * layout of a batch from its request lengths (ak_batch_layout), linear
 * attention with a decay for each head (ak_linear_attention, its gradients
 * and its single-token step), a recurrence with a gate for every token and
 * channel (ak_gated_recurrence, likewise), the verification of drafted tokens
 * (ak_verify_drafts), the step of a beam search (ak_beam_select,
 * ak_beam_reorder), and the forking, freeing, compacting and copying of a
 * paged cache's blocks (ak_blocks_*).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Pointers. Arrays (src, dst, workspace) are DEVICE pointers to memory of the
 *   current CUDA device; init and dst_host are HOST pointers. The caller owns
 *   every buffer; the library allocates no device memory.
 * Layout. Arrays are dense and column-major: element (i1, i2, ..., id) of a
 *   shape (n1, ..., nd) sits at i1 + n1*(i2 + n2*(i3 + ...)) (0-based). This
 *   is the memory of a contiguous row-major tensor of the reversed shape.
 *   Dimensions are numbered from 0 (Julia's dims=2 is dimension 1 here).
 * Element types (ak_dtype). AK_BF16 is the bfloat16 bit pattern; AK_MAT2_MODP
 *   is a 2x2 matrix over Z/pZ, p = 2^31 - 1, stored as four uint32 entries in
 *   column-major order (a11, a21, a12, a22), each in [0, p); its only operator
 *   is AK_OP_MATMUL_MODP, the product mod p, with the left operand first.
 * Types of a call. `in` is the element type of src; `acc` the accumulator in
 *   which f is applied and op folds; `out` the type stored. Supported
 *   (in -> acc -> out): F32->F32->F32, F32->F64->{F64,F32}, F64->F64->F64,
 *   BF16->F32->{BF16,F32}, I32->I32->I32, I32->I64->I64, I64->I64->I64,
 *   MAT2->MAT2->MAT2. f32 -> bf16 and f64 -> f32 stores round to nearest
 *   even; integer accumulators wrap modulo 2^32 / 2^64.
 * Order. Results equal the left-to-right fold up to the rounding of a
 *   different association tree; non-commutative operators keep the element
 *   order exactly. max / min follow Julia: NaN wins (returned as the
 *   canonical quiet NaN) and +0.0 > -0.0.
 * init. A host pointer to ONE value of the accumulator type, applied exactly
 *   once, leftmost: op(init, ...).
 * Asynchrony. Calls enqueue work on `stream` (a cudaStream_t, NULL = legacy
 *   default stream) and return without waiting, except where stated. Calls
 *   that share a workspace must be ordered on one stream.
 * Workspace. A device buffer of at least the size the matching
 *   *_workspace_size function reports for the same arguments (16-byte
 *   aligned). Its contents on entry are arbitrary: no clearing is needed
 *   between calls.
 * Errors. Every call returns an ak_status. Arguments are validated before
 *   anything is launched, so invalid calls have no effect on the device.
 *   AK_ERR_CUDA keeps the CUDA error, readable with ak_last_cuda_error().
 * Logging. With AK_LOG set in the environment (and not "0"), every call
 *   prints one line to stderr naming the path it takes: the first-pass grid
 *   of a reduction, the dims kernel with its shape, tile and split, the
 *   scan kernel with its tile count, findall's tile count, the kernel and the
 *   division of the token axis of linear attention. The variable is read on
 *   every call.
 */
#ifndef AK_H
#define AK_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum ak_status {
    AK_OK = 0,
    AK_ERR_INVALID_ARG = 1,   /* bad pointer, size, enum, dims or store mode */
    AK_ERR_UNSUPPORTED = 2,   /* valid but unsupported type / op / map combination */
    AK_ERR_WORKSPACE = 3,     /* workspace missing, too small or misaligned */
    AK_ERR_EMPTY_NO_INIT = 4, /* empty reduction, no init and no neutral element */
    AK_ERR_CUDA = 5,          /* a CUDA runtime call failed */
    AK_ERR_TIMEOUT = 6        /* a bounded device-side wait ran out (scan look-back) */
} ak_status;

typedef enum ak_dtype {
    AK_F32 = 0,
    AK_F64 = 1,
    AK_BF16 = 2,
    AK_I32 = 3,
    AK_I64 = 4,
    AK_MAT2_MODP = 5,
    AK_U8 = 6  /* bytes (Julia Bool flags): findall input only */
} ak_dtype;

/* f, applied to each element in the accumulator type before op. */
typedef enum ak_map { AK_MAP_IDENTITY = 0, AK_MAP_ABS = 1, AK_MAP_ABS2 = 2 } ak_map;

/* f of a fused two-source element (ak_reduce2), in the accumulator type:
 * a*b, (a-b)^2, |a-b| (integers wrap). */
typedef enum ak_map2 { AK_MAP2_MUL = 0, AK_MAP2_SQDIFF = 1, AK_MAP2_ABSDIFF = 2 } ak_map2;

typedef enum ak_op {
    AK_OP_ADD = 0,
    AK_OP_MUL = 1,
    AK_OP_MAX = 2,
    AK_OP_MIN = 3,
    AK_OP_MATMUL_MODP = 4
} ak_op;

/* How a reduction's result r is stored into R (PR #139, "What changes": the
 * last pass applies init, folds into R's previous value, or writes):
 *   AK_STORE_OVERWRITE  R = r
 *   AK_STORE_INIT       R = op(init, r)    (init required)
 *   AK_STORE_FOLD       R = op(R_old, r)   (R_old converted to acc first) */
typedef enum ak_store { AK_STORE_OVERWRITE = 0, AK_STORE_INIT = 1, AK_STORE_FOLD = 2 } ak_store;

/* Kernel shape of a strided dims reduction (PR #176, item 1): one thread per
 * output, one pass over tiles of outputs, or tiles of outputs with the
 * reduction split across blocks and a second pass. AUTO chooses by the
 * number of outputs versus the reduction length. */
typedef enum ak_dims_shape {
    AK_SHAPE_AUTO = 0,
    AK_SHAPE_THREAD = 1,
    AK_SHAPE_TILED = 2,
    AK_SHAPE_COLUMNS = 3
} ak_dims_shape;

/* Options; pass NULL for defaults or fill with ak_opts_default(). */
typedef struct ak_opts {
    int32_t no_neutral;       /* 1: treat op as having no neutral element; partial results
                                 carry an Optional flag (e.g. 8 bytes for a Float32 acc) */
    int32_t target_blocks;    /* whole-array first pass / persistent scan grid; 0 = auto */
    int32_t items_per_thread; /* scan run length / reduce loads in flight; 0 = auto */
    int32_t dims_shape;       /* ak_dims_shape */
    int32_t check;            /* 1: synchronize `stream` before returning and report
                                 device-side failures (AK_ERR_TIMEOUT) */
    int32_t flags;            /* tuning switches, AK_FLAG_* (0 = none) */
    int32_t exclusive;        /* ak_accumulate: 1 = exclusive scan (see ak_accumulate) */
    int32_t reserved;         /* must be 0 */
    int64_t wait_limit_ns;    /* bound of each device-side wait of the scan; 0 = 1 s. Without
                                 `check` a wait that runs out is not reported by the call
                                 itself: read it with ak_scan_status. (Linear attention
                                 and the gated recurrence take at least 0.1 s, see
                                 there.) */
    int64_t debug_skip_publish_tile; /* fault injection for tests: the scan tile with this
                                 index never publishes its state, so its successors'
                                 bounded waits run out; -1 = off */
} ak_opts;

/* AK_FLAG_DIMS_CLUSTER: a strided dims reduction whose split fits 2..16
 * blocks runs each output tile's blocks as one thread-block cluster and
 * combines their partials in distributed shared memory (one kernel, no
 * workspace partials) instead of a workspace and a second pass, at any input
 * size. Without the flag the automatic shape does so only for inputs of at
 * most 16 MB, where saving the second launch pays on GB300; larger inputs
 * split through the workspace. */
#define AK_FLAG_DIMS_CLUSTER 1

void ak_opts_default(ak_opts* opts);

const char* ak_status_string(ak_status status);
/* Size in bytes of one element of the type; 0 for an invalid type. */
size_t ak_dtype_size(ak_dtype dtype);
/* The cudaError_t of the last AK_ERR_CUDA returned on this thread. */
int ak_last_cuda_error(void);
/* Number of kernels this library has launched in this process. */
uint64_t ak_kernel_launch_count(void);

/* ---------------------------------------------------------------------------
 * ak_reduce: r = op(f(src[0]), f(src[1]), ..., f(src[n-1])), then stored by
 * `mode` into a one-element device array and/or returned to the host.
 * PR #139, "What changes": a first pass of a bounded number of blocks, each
 * reducing its share of the input to one partial, and a one-block second
 * pass that reduces the partials and performs the store; a small input takes
 * one launch; for a host result the last pass stores the bare partial, which
 * is copied back and finished on the host.
 *
 *   src        device, n elements of `in` (n == 0 allowed)
 *   dst_dev    device, one element of `out`, or NULL
 *   dst_host   host, one element of `out`, or NULL; when given the call
 *              returns only once the result is there (with AK_STORE_FOLD,
 *              *dst_host holds R_old on entry, unless dst_dev is also
 *              given, in which case R is the device element). The last
 *              pass writes the bare partial straight into a small mapped,
 *              pinned host slot of the calling thread (64 bytes, allocated
 *              by its first host-result call and kept until the process
 *              exits), then the call's sequence number beside it after a
 *              system-scope fence. The host polls that word for about
 *              200 us, then synchronizes `stream` (which also reports any
 *              error on it), and finishes the partial. The call may thus
 *              return before the kernel has retired on the stream; later
 *              work on the stream is ordered after it as usual. An
 *              asynchronous error that strikes after the result landed
 *              surfaces on the next synchronizing call.
 *   At least one of dst_dev / dst_host must be non-NULL.
 * Empty input: AK_STORE_INIT stores init; AK_STORE_FOLD leaves R unchanged;
 *   AK_STORE_OVERWRITE stores the neutral element of op (0 for +, 1 for *,
 *   the identity matrix), or fails with AK_ERR_EMPTY_NO_INIT for max / min
 *   and under no_neutral.
 * ------------------------------------------------------------------------- */
ak_status ak_reduce_workspace_size(int64_t n, ak_dtype in, ak_dtype acc, const ak_opts* opts,
                                   size_t* bytes);
ak_status ak_reduce(const void* src, int64_t n, ak_dtype in, ak_map f, ak_op op, ak_dtype acc,
                    ak_dtype out, const void* init, ak_store mode, void* dst_dev, void* dst_host,
                    void* workspace, size_t workspace_bytes, const ak_opts* opts, void* stream);

/* ---------------------------------------------------------------------------
 * ak_reduce2: r = op(f(a[0], b[0]), ..., f(a[n-1], b[n-1])) over two sources
 * of n elements of `in` read side by side -- a fused (Broadcasted) source such
 * as sum(x .* y) or sum(abs2.(x .- y)), reduced without materialising the
 * elementwise array. PR #139, "What changes": a single-output reduction whose
 * source is a Broadcasted takes the whole-array path. Arguments, workspace
 * (ak_reduce_workspace_size with the same n, in, acc), store modes and empty
 * rules are ak_reduce's; f is an ak_map2; matrices are not supported. Sources
 * whose addresses differ by a multiple of 32 bytes are read with 32-byte
 * vectors, others element by element.
 * ------------------------------------------------------------------------- */
ak_status ak_reduce2(const void* src_a, const void* src_b, int64_t n, ak_dtype in, ak_map2 f, ak_op op,
                     ak_dtype acc, ak_dtype out, const void* init, ak_store mode, void* dst_dev,
                     void* dst_host, void* workspace, size_t workspace_bytes, const ak_opts* opts,
                     void* stream);

/* ---------------------------------------------------------------------------
 * ak_reduce_dims: R[kept index] = op over the reduced dimensions of
 * f(src[...]), folded in increasing column-major order of the reduced
 * indices. PR #176: strided reductions into contiguous outputs take a 2-d
 * block of outputs x reduction rows, split across blocks (plus a second
 * pass) only when the outputs alone do not fill the device; the middle
 * dimension of a 3-d array is handled as runs of contiguous outputs at the
 * offsets of the other kept dimensions. PR #139: a reduction to a single
 * output over one contiguous range takes the whole-array path; its tests
 * cover offset views, which strides describe here.
 *
 *   ndim, shape   1 <= ndim <= 8, column-major extents (>= 0)
 *   strides       element strides of src per dimension (>= 0): a strided
 *                 view (a sub-array, a transpose, a stepped slice); NULL =
 *                 dense column-major. Views whose kept innermost dimension
 *                 has unit stride take the strided / row kernels (16-byte
 *                 loads when src and the strides are 16-byte multiples);
 *                 others a general kernel (slower: it walks the reduced
 *                 indices per thread).
 *   dims_mask     bit d set = dimension d is reduced (bits >= ndim invalid)
 *   dst           device, DENSE column-major array of `out` with the shape
 *                 of src where reduced extents are 1
 * Empty reductions (a reduced extent is 0) follow ak_reduce's empty rules.
 * ------------------------------------------------------------------------- */
ak_status ak_reduce_dims_workspace_size(int ndim, const int64_t* shape, const int64_t* strides,
                                        uint32_t dims_mask, ak_dtype in, ak_dtype acc,
                                        const ak_opts* opts, size_t* bytes);
ak_status ak_reduce_dims(const void* src, int ndim, const int64_t* shape, const int64_t* strides,
                         uint32_t dims_mask, ak_dtype in, ak_map f, ak_op op, ak_dtype acc,
                         ak_dtype out, const void* init, ak_store mode, void* dst, void* workspace,
                         size_t workspace_bytes, const ak_opts* opts, void* stream);

/* ---------------------------------------------------------------------------
 * ak_accumulate: inclusive scan. Along a line x_1, x_2, ...:
 *   y_1 = op(init, x_1) (or x_1 without init), y_i = op(y_{i-1}, x_i).
 * dim = -1 scans the whole array as one line (column-major order); dim = d
 * scans every line along dimension d independently. PR #202, first
 * paragraph: a tile is loaded, each thread scans its own run of consecutive
 * elements, and the tile prefix is applied (runs of lines that fit one tile
 * sit at an odd stride in shared memory, as there; long lines are copied by
 * the TMA engine into a swizzled ring, or walked in 32-byte segments). Tiles
 * pass their prefixes on in a single pass from published tile aggregates
 * (after decoupled look-back, Merrill & Garland 2016); every wait is bounded.
 * Long-line calls clear their own tile state on `stream` first, so a call
 * captured in a CUDA graph is correct on every replay.
 *
 *   src, dst      device, same shape; dst may equal src (in place) but must
 *                 not otherwise overlap it
 * Exclusive scan (opts->exclusive = 1): element i holds the fold of init and
 *   the elements before it, y_1 = init, y_i = op(y_{i-1}, x_{i-1}). The pages
 *   describe inclusive scans only; this is its plain exclusive counterpart.
 *   Without init the neutral element stands for it (0 for +, 1 for *, the
 *   identity matrix); max / min and no_neutral then fail with
 *   AK_ERR_EMPTY_NO_INIT, since the first output has no value.
 * A wait that runs out (only possible through debug_skip_publish_tile or a
 * hardware fault) stops the kernel early; with opts->check set the call then
 * returns AK_ERR_TIMEOUT and dst is unspecified. Without check the call
 * returns AK_OK and the failure is recorded in the workspace: after the
 * stream has reached the end of the call, ak_scan_status(workspace) tells.
 * ------------------------------------------------------------------------- */
ak_status ak_accumulate_workspace_size(int ndim, const int64_t* shape, int dim, ak_dtype in,
                                       ak_dtype acc, ak_op op, const ak_opts* opts,
                                       size_t* bytes);
ak_status ak_accumulate(const void* src, void* dst, int ndim, const int64_t* shape, int dim,
                        ak_dtype in, ak_op op, ak_dtype acc, ak_dtype out, const void* init,
                        void* workspace, size_t workspace_bytes, const ak_opts* opts,
                        void* stream);
/* Outcome of the last ak_accumulate that used this workspace: AK_OK, or
 * AK_ERR_TIMEOUT when one of its bounded waits ran out. A blocking read of
 * the workspace's first word: call it once the caller's stream has passed the
 * scan (e.g. after cudaStreamSynchronize), not while it runs. */
ak_status ak_scan_status(const void* workspace);

/* ---------------------------------------------------------------------------
 * ak_findall: the indices of the nonzero elements of src, in increasing
 * order, and their count (Julia's findall over a Bool array, or over
 * x .!= 0). The tile-scan PR #202 counts findall among its scans (ratio
 * table; its tests paragraph): the output slot of a selected element is the
 * exclusive count of the selected elements before it. One pass: tiles count
 * their selected elements, publish the counts and derive their output
 * offsets by decoupled look-back (bounded waits), then store the indices.
 *
 *   src        device, n elements of `in`: AK_U8 (nonzero byte = true),
 *              AK_I32, AK_I64 (!= 0), AK_F32, AK_F64 (!= 0.0: -0.0 is
 *              false, NaN true)
 *   idx        device, room for n int64 (the count is at most n); receives
 *              the 0-based indices; entries past the count are untouched
 *   count_dev  device, one int64, or NULL
 *   count_host host, one int64, or NULL; when given the call synchronizes
 *              `stream` and returns the count there
 *   At least one of count_dev / count_host must be non-NULL.
 * The workspace is cleared by the call on its stream (graph-replay safe).
 * ------------------------------------------------------------------------- */
ak_status ak_findall_workspace_size(int64_t n, ak_dtype in, const ak_opts* opts, size_t* bytes);
ak_status ak_findall(const void* src, int64_t n, ak_dtype in, int64_t* idx, int64_t* count_dev,
                     int64_t* count_host, void* workspace, size_t workspace_bytes, const ak_opts* opts,
                     void* stream);

/* ---------------------------------------------------------------------------
 * ak_reduce_noalloc: ak_reduce for callers that cannot allocate device memory.
 * The pages have no counterpart to this entry point; it exists for callers
 * that must not call cudaMalloc or any allocating routine when they reduce:
 * a real-time loop that cannot afford the implicit device synchronisation
 * of cudaMalloc / cudaFree, a process whose device memory is already fully
 * reserved by another allocator, or code held to a fixed memory budget.
 *
 * Arguments, results, store and empty-input rules are those of ak_reduce;
 * the caller still passes src and dst_dev / dst_host. The scratch (first-pass
 * partials and the bare result slot) lives in a fixed array of
 * AK_NOALLOC_SCRATCH_BYTES inside the library's device image, so every GPU
 * that loads the library holds that much memory until the process exits. A
 * call whose plan needs more scratch than that (it grows with the SM count
 * and the partial size, about 20 KB on a 152-SM GPU) returns
 * AK_ERR_WORKSPACE without launching anything.
 *
 * The first call on each device looks up the array's device address
 * (cudaGetSymbolAddress, with that device current); make that first call
 * before any stream capture. The address is kept per device and CUDA
 * context: after a cudaDeviceReset the device's new context holds the array
 * at a new address, and the next call (again: outside any capture) looks it
 * up anew. Every call on a device shares the one array:
 * calls that may overlap on the GPU (different streams, no ordering) race
 * on it and give wrong results; order them on one stream. Nothing in the
 * array needs clearing between calls.
 * ------------------------------------------------------------------------- */
#define AK_NOALLOC_SCRATCH_BYTES 65536
ak_status ak_reduce_noalloc(const void* src, int64_t n, ak_dtype in, ak_map f, ak_op op, ak_dtype acc,
                            ak_dtype out, const void* init, ak_store mode, void* dst_dev, void* dst_host,
                            const ak_opts* opts, void* stream);

/* ---------------------------------------------------------------------------
 * Shape selector of ak_reduce_dims, exposed for inspection and tests (pure
 * host logic, no device needed). For a canonical strided problem of
 * `inner` contiguous outputs, reduction length `red_len` at stride `inner`
 * and `outer` output runs, elements of `elem_bytes` and vector width
 * `vec_elems`, on a device of `sm_count` SMs, writes the chosen shape, the
 * outputs per block along the contiguous dimension, the reduction rows per
 * block and the split factor.
 * ------------------------------------------------------------------------- */
ak_status ak_dims_select(int64_t inner, int64_t red_len, int64_t outer, int elem_bytes,
                         int vec_elems, int sm_count, int forced_shape, int32_t* shape_out,
                         int32_t* tile_outputs, int32_t* row_groups, int32_t* split);

/* ---------------------------------------------------------------------------
 * ak_batch_layout: block tables, slot maps and packed offsets of a batch,
 * from its requests' lengths, without the lengths ever reaching the host.
 * With ctx_r tokens of request r in a paged cache of blocks of b tokens and
 * new_r tokens to run:
 *   offsets[r] = new_0 + ... + new_{r-1}           (exclusive scan, nreq + 1 values)
 *   blocks ceil(ctx_r / b) .. ceil((ctx_r + new_r) / b) - 1 of request r are
 *     taken from free_blocks, front to back, in request order, and entered
 *     in its row of block_table (other entries stay as they are)
 *   token t of request r: positions[t] = ctx_r + t - offsets[r],
 *     requests[t] = r, slots[t] = block_table[r][pos / b] * b + pos % b
 *
 *   ctx_lens, new_lens  device, nreq int32 (negative values count as 0)
 *   block_table  device, nreq rows of table_width int32, table_stride apart
 *   free_blocks  device, nfree int32; not changed: counts[1] of them are used
 *   offsets      device, nreq + 1 int32
 *   slots        device, max_tokens int64; positions, requests: max_tokens
 *                int32. Entries past the batch's last token get slot -1,
 *                position 0 and request -1.
 *   counts       device, 2 int32: tokens of the batch, blocks it takes
 * What does not fit is never written: tokens past max_tokens are left out, a
 * block past the free list enters as -1, and a token in such a block or past
 * the table's width (or in a block whose entry is negative) gets slot -1;
 * the caller compares counts with max_tokens and nfree. The sums of tokens
 * and of blocks must stay below 2^31.
 * ------------------------------------------------------------------------- */
ak_status ak_batch_layout_workspace_size(int64_t nreq, const ak_opts* opts, size_t* bytes);
ak_status ak_batch_layout(const int32_t* ctx_lens, const int32_t* new_lens, int64_t nreq, int32_t* block_table,
                          int64_t table_stride, int32_t table_width, const int32_t* free_blocks, int64_t nfree,
                          int32_t block_size, int64_t max_tokens, int32_t* offsets, int64_t* slots,
                          int32_t* positions, int32_t* requests, int32_t* counts, void* workspace,
                          size_t workspace_bytes, const ak_opts* opts, void* stream);

/* ---------------------------------------------------------------------------
 * ak_verify_drafts: how many of its drafted tokens each request keeps, and
 * the token after them, from given random numbers. Request r drafted tokens
 * d_0 .. d_{m-1} (m = draft_counts[r], or k) from distributions q_j; the
 * target's are p_0 .. p_m. With
 *   a = the first j < m for which u_j * q_j(d_j) < p_j(d_j) is false, or m
 * accepted[r] = a and tokens[r] = d_0 .. d_{a-1}, x, -1, -1, ... with
 *   x = argmax_v max(p_a(v) - q_a(v), 0) / e_v   if a < m
 *   x = argmax_v p_a(v) / e_v                    if a = m
 * (ties: the lowest v), which, for u uniform in [0, 1) and e exponential,
 * leaves the emitted tokens distributed as the target's own.
 *
 *   target_probs  device, element (r, j, v) at r*target_req + j*target_row + v,
 *                 j <= k; AK_F32 or AK_BF16, as are the draft's
 *   draft_probs   device, likewise with j < k; NULL: each draft was certain
 *                 (q_j is 1 at d_j and 0 elsewhere)
 *   draft_tokens  device, nreq * k int32; a token outside [0, vocab) is
 *                 refused
 *   draft_counts  device, nreq int32, clamped to [0, k]; NULL: all k
 *   uniform       device, nreq * k float
 *   noise         device, one row of vocab float > 0 for each request,
 *                 noise_stride apart
 *   tokens        device, nreq * (k + 1) int32
 *   accepted      device, nreq int32
 * The product u_j q_j(d_j) is compared exactly; differences and quotients are
 * rounded to float32. Candidates need a weight
 * above zero; scores that are NaN are passed over. If the difference leaves
 * no candidate (p = q up to rounding), p alone decides; if that leaves none,
 * x is -1. k may be 0. No workspace.
 * ------------------------------------------------------------------------- */
ak_status ak_verify_drafts(const void* target_probs, int64_t target_req, int64_t target_row, const void* draft_probs,
                           int64_t draft_req, int64_t draft_row, ak_dtype dtype, const int32_t* draft_tokens,
                           const int32_t* draft_counts, const float* uniform, const float* noise,
                           int64_t noise_stride, int64_t nreq, int32_t k, int64_t vocab, int32_t* tokens,
                           int32_t* accepted, const ak_opts* opts, void* stream);

/* ---------------------------------------------------------------------------
 * Linear attention with a decay for each head: the scan whose state is a
 * matrix. For each head h and sequence, with g = exp(log_decay[h]):
 *   S_t = g * S_{t-1} + k_t v_t^T      (dk x dv, float32)
 *   o_t = scale * S_t^T q_t            (the token itself included)
 * Sequences are packed along the token axis: sequence n holds tokens
 * offsets[n] .. offsets[n+1]-1 (the offsets of ak_batch_layout), some may be
 * empty. S starts from state_in, or zero.
 *
 * ak_heads describes one [tokens][heads][dim] array: element (t, h, i) at
 * t*token_stride + h*head_stride + i (strides in elements, >= 0; a head
 * stride of 0 shares one head among all in an input).
 *
 * ak_linattn, the shape of a call:
 *   dtype     AK_F32 or AK_BF16: of q, k, v, o and their gradients; products
 *             are summed in float32, and states are float32 throughout
 *   tokens, seqs, heads; dk, dv in 1 .. 256
 *   max_len   a bound on the longest sequence, or 0 (unknown); it only
 *             guides how the token axis is cut
 *   scale     finite
 *
 *   log_decay  device, heads float, normally <= 0; -infinity: no memory
 *   offsets    device, seqs + 1 int32, non-decreasing; NULL: one sequence of
 *              all tokens (seqs = 1). Values are clamped to [0, tokens].
 *              Output rows of tokens outside every sequence are set to 0.
 *   state_in   device, seqs*heads matrices, dk x dv with dv contiguous, or NULL
 *   state_out  device, the states after each sequence's last token, or NULL;
 *              may be state_in
 * The tensor core's float32 accumulation cuts off rather than rounds, so
 * states of bf16 calls (heads of 64 and 128) come out too small: by up to 4e-8
 * for each of the three products that add 16 tokens, as far back as the decay
 * remembers and no further than the window's start. On normal inputs, relative
 * and in norm: up to 4e-7 + 7.5e-9 M with M the tokens remembered, at most
 * those of a window. Measured: 1.2e-6 at a memory of 256 tokens; without decay
 * 3.5e-6 over 1000 tokens, 5e-5 over 16000 and 1.9e-4 over 64000 in one window,
 * 4.2e-6 over 16000 in 30 windows. A caller who needs more cuts the axis
 * (opts->target_blocks = tokens / 1000: below 8e-6 at any length), or passes
 * float32 tensors, whose states round to nearest (2.3e-6 over 16000 tokens in
 * one window).
 * Range: within a block of tokens terms are held divided by up to e^30 of decay
 * (e^40 in float32 calls and for other head sizes), so products k v above 1e25
 * (1e21) in size may overflow where the recurrence would not.
 * Within the types' rounding the order of summation is fixed by the shape:
 * equal calls give equal bits. In bf16 calls weighted scores and the state
 * are rounded to bf16 where they enter a product with q or v. A NaN or
 * infinity in q reaches its own output; in k, v or a state it reaches, as a NaN
 * or infinity, what the recurrence takes it to: its sequence and head from its
 * token on. In gradients likewise, those of k and v backwards in time.
 *
 * ak_linear_attention_backward: the gradients of sum(o * do) +
 * sum(state_out * dstate_out), from the forward call's inputs; dq, dk, dv as
 * q, k, v are described; dstate_in (may be NULL) receives the gradient of
 * state_in. log_decay and scale are constants of the model and get none. A
 * head that the inputs share gets its gradient for each head that reads it
 * (dq, dk and dv have no head stride of 0); their sum is the caller's.
 * dstate_in is neither dstate_out nor state_in.
 *
 * ak_linear_attention_step: one token for each of `tokens` requests (seqs,
 * offsets and max_len unused), the state updated in place. Request b uses
 * matrices slots[b] of nslots in `state` (slots NULL: b). An index outside
 * [0, nslots) marks padding: its output is 0. Indices must not repeat.
 *
 * opts->target_blocks: windows the token axis is cut into (0 = automatic).
 * opts->check also reports a bounded device-side wait that ran out
 * (AK_ERR_TIMEOUT; the results are then undefined). The waits are for a
 * block's own copies and products, microseconds apart: one runs out if the
 * device faults, or is taken away from the block for longer than
 * opts->wait_limit_ns (0.1 s at least). Outputs overlap neither each other nor
 * an input, except as stated.
 * ------------------------------------------------------------------------- */
typedef struct ak_heads {
    void* data;
    int64_t token_stride, head_stride;
} ak_heads;

typedef struct ak_linattn {
    int64_t tokens, seqs, max_len;
    int32_t heads, dk, dv;
    int32_t dtype; /* ak_dtype */
    float scale;
    int32_t reserved; /* must be 0 */
} ak_linattn;

/* Enough for the forward and the backward pass of a shape. Where it is 256
 * bytes they only report a wait that ran out, and a call without opts->check
 * may pass NULL. */
ak_status ak_linear_attention_workspace_size(const ak_linattn* shape, const ak_opts* opts, size_t* bytes);
ak_status ak_linear_attention(const ak_linattn* shape, const ak_heads* q, const ak_heads* k, const ak_heads* v,
                              const float* log_decay, const int32_t* offsets, const float* state_in,
                              const ak_heads* o, float* state_out, void* workspace, size_t workspace_bytes,
                              const ak_opts* opts, void* stream);
ak_status ak_linear_attention_backward(const ak_linattn* shape, const ak_heads* d_o, const ak_heads* q,
                                       const ak_heads* k, const ak_heads* v, const float* log_decay,
                                       const int32_t* offsets, const float* state_in, const float* dstate_out,
                                       const ak_heads* dq, const ak_heads* dk, const ak_heads* dv,
                                       float* dstate_in, void* workspace, size_t workspace_bytes,
                                       const ak_opts* opts, void* stream);
ak_status ak_linear_attention_step(const ak_linattn* shape, const ak_heads* q, const ak_heads* k, const ak_heads* v,
                                   const float* log_decay, float* state, const int32_t* slots, int64_t nslots,
                                   const ak_heads* o, const ak_opts* opts, void* stream);

/* ---------------------------------------------------------------------------
 * Gated linear recurrence: the scan whose state is a vector, with a gate for
 * every token and channel. For each channel and sequence
 *   h_t = a_t * h_{t-1} + b_t * x_t
 *   AK_RECURRENCE_DECAY  a = exp(gate), b = 1          (gate: a log decay, <= 0)
 *   AK_RECURRENCE_GATE   a = sigmoid(gate), b = 1 - a  (gate: a logit)
 * Sequences are packed along the token axis as in ak_linear_attention; h
 * starts from state_in, or zero.
 *
 * ak_rows describes one [tokens][channels] array: element (t, i) at
 * t*token_stride + i (stride in elements, >= 0; 0 shares one row among all
 * tokens in an input).
 *
 * ak_recurrence, the shape of a call:
 *   dtype     AK_F32 or AK_BF16: of x, gate, h and their gradients; states are
 *             float32, and so is all arithmetic
 *   form      ak_recurrence_form
 *   tokens, seqs, channels (>= 1)
 *
 *   offsets    device, seqs + 1 int32, non-decreasing; NULL: one sequence of
 *              all tokens (seqs = 1). Values are clamped to [0, tokens].
 *              Output rows of tokens outside every sequence are set to 0.
 *   state_in   device, seqs rows of channels float, or NULL
 *   h          may be x itself (the same memory and stride): the call then works
 *              in place (the gate form's gradients need x as it was)
 *   state_out  device, the states after each sequence's last token, or NULL;
 *              may be state_in. A sequence without tokens hands its state on.
 * The order of summation is fixed by the shape: equal calls give equal bits.
 * A gate of -infinity forgets what was before; a NaN or infinity reaches, as a
 * NaN or infinity, what the recurrence takes it to: its sequence and channel from its
 * token on (in gradients backwards in time).
 * Precision: a state is rounded where a token's run of up to 32, its tile of 8
 * runs and its cluster's step of up to 16 tiles meet, a few dozen times and not at
 * each token between, and factors near one are applied less one. Where every gate is
 * the same, the worst for this, states were off by 2e-7 of their norm in the median
 * over gates (memories of 1 to 10^5 tokens) and by 1.3e-6 at the worst gate. bf16 calls,
 * whose factors within a run are rounded as they are, by 6e-7 and 3.5e-6 (1.4e-5 if each
 * rounding pushed as far as it may); their outputs round to bf16. A gate's own factor is
 * exact to 2^-21 + |gate| 2^-23 of itself, and below 2^-126 it is 0.
 * Range: factors of up to 256 tokens are multiplied before the state they meet, so
 * log decays above 0 that reach e^88 within a tile may give infinities or NaN where
 * the recurrence would not.
 *
 * ak_gated_recurrence_backward: the gradients of sum(h * dh) +
 * sum(state_out * dstate_out), from the forward call's inputs and its output
 * h; dstate_in (may be NULL) receives the gradient of state_in. In a bf16 call
 * the gates' gradients see h as it was stored, rounded to bf16 (in the gate
 * form: h before every 8th or 16th token). x is not read in the decay form and may
 * be NULL there. A row that an input shares among tokens gets its gradient
 * for each token (dx and dgate have no stride of 0); their sum is the caller's.
 *
 * ak_gated_recurrence_step: one token for each of `tokens` requests (seqs and
 * offsets unused), the state updated in place. Request b uses row slots[b] of
 * nslots in `state` (slots NULL: b). An index outside [0, nslots) marks padding: its
 * output is 0. Indices must not repeat. An infinite state is what a h + b x makes of it.
 *
 * opts->check also reports a bounded device-side wait that ran out
 * (AK_ERR_TIMEOUT; the results are then undefined). The waits are for the maps of
 * the other blocks of a cluster, microseconds apart, for opts->wait_limit_ns (0.1 s
 * at least); opts->debug_skip_publish_tile: the tile with this index sends none.
 * Of calls that run out at the same time on a device one is reported.
 * Outputs overlap neither each other nor an input, except as stated. No workspace.
 * ------------------------------------------------------------------------- */
typedef enum ak_recurrence_form { AK_RECURRENCE_DECAY = 0, AK_RECURRENCE_GATE = 1 } ak_recurrence_form;

typedef struct ak_rows {
    void* data;
    int64_t token_stride;
} ak_rows;

typedef struct ak_recurrence {
    int64_t tokens, seqs, channels;
    int32_t dtype; /* ak_dtype */
    int32_t form;  /* ak_recurrence_form */
} ak_recurrence;

ak_status ak_gated_recurrence(const ak_recurrence* shape, const ak_rows* x, const ak_rows* gate,
                              const int32_t* offsets, const float* state_in, const ak_rows* h, float* state_out,
                              const ak_opts* opts, void* stream);
ak_status ak_gated_recurrence_backward(const ak_recurrence* shape, const ak_rows* dh, const ak_rows* x,
                                       const ak_rows* gate, const ak_rows* h, const int32_t* offsets,
                                       const float* state_in, const float* dstate_out, const ak_rows* dx,
                                       const ak_rows* dgate, float* dstate_in, const ak_opts* opts, void* stream);
ak_status ak_gated_recurrence_step(const ak_recurrence* shape, const ak_rows* x, const ak_rows* gate, float* state,
                                   const int32_t* slots, int64_t nslots, const ak_rows* h, const ak_opts* opts,
                                   void* stream);

/* ---------------------------------------------------------------------------
 * ak_beam_select: one step of a beam search over `batch` requests. Beam k of a
 * request has the summed log probability scores[k] and the logits x_k of its next
 * token; its candidates are
 *   token v, total scores[k] + x_k(v) - log sum_w exp x_k(w), length lengths[k] + 1
 *   if the beam has ended (done[k] != 0): end_token alone, total scores[k],
 *   length lengths[k]; its logits are not read
 * and the request's best `keep` of all its beams' candidates, by
 * total / length^penalty, are its next beams, in decreasing order (ties: the
 * lowest beam, then the larger logit, then the lowest token).
 *
 *   logits     device, element (r, k, v) at r*batch_stride + k*beam_stride + v;
 *              AK_F32 or AK_BF16
 *   scores     device, batch * beams float
 *   done       device, batch * beams bytes; NULL: none has ended
 *   lengths    device, batch * beams int32; NULL: all 0
 *   end_token  the token that ends a beam, or -1
 *   penalty    finite; 0: candidates are ranked by their totals
 *   beams, keep  1 .. 32 (a first step has one beam and keeps several)
 *   out_scores, out_tokens, out_parents  device, batch * keep: total, token
 *              and the beam it extends
 *   out_done, out_lengths  device, likewise, or NULL
 * With keep = beams, out_scores, out_done and out_lengths may be scores, done and
 * lengths themselves (with another number of them, those of one request).
 * Exponentials are float32, as are their sums, with compensation; logarithms, totals
 * and their comparison are 64-bit, out_scores rounded from them. Within a beam logits
 * decide, exactly. Between beams a logarithm that is off may: by 2e-7 at most where logits lie
 * in any order, 2.3e-7 where they rise along the row (2^-21 + d 2^-22.8 + (m + 2) 2^-21.6, d the
 * mean distance of what is summed below the row's largest logit, m the larger logits
 * that one thread meets). A
 * logit of -infinity, and what has no finite rank, is no candidate; a row
 * that holds a NaN or +infinity, or a beam whose score is not finite or whose length^penalty
 * is below 0 (a negative length), has none.
 * Where a request has fewer than `keep` candidates the rest of its beams get score
 * -infinity, token and parent -1, length 0 and done 1. No workspace.
 *
 * ak_beam_reorder: state[b] = state[parents[b]] for the `beams` (1 .. 32) rows of
 * each request, in place: rows of inner_bytes at
 *   o*outer_stride + r*batch_stride + k*beam_stride   (bytes; o < outer, r < batch)
 * A row whose parent is outside [0, beams) stays as it is. Rows do not overlap.
 * ------------------------------------------------------------------------- */
ak_status ak_beam_select(const void* logits, int64_t batch_stride, int64_t beam_stride, ak_dtype dtype, int64_t batch,
                         int32_t beams, int64_t vocab, int32_t keep, const float* scores, const uint8_t* done,
                         const int32_t* lengths, int32_t end_token, double penalty, float* out_scores,
                         int32_t* out_tokens, int32_t* out_parents, uint8_t* out_done, int32_t* out_lengths,
                         const ak_opts* opts, void* stream);
ak_status ak_beam_reorder(void* state, int64_t outer, int64_t outer_stride, int64_t batch, int64_t batch_stride,
                          int32_t beams, int64_t beam_stride, int64_t inner_bytes, const int32_t* parents,
                          const ak_opts* opts, void* stream);

/* ---------------------------------------------------------------------------
 * Blocks of a paged cache that requests share. A request of lens[r] tokens
 * holds the first ceil(lens[r] / block_size) entries of its row of the block
 * table (at most table_width; further entries mean nothing), and several requests may hold
 * the same block. An entry outside [0, nblocks) holds none. Nothing is kept between
 * calls: how often a block is held is what the table says.
 *
 * ak_blocks_count: refs[i] = held entries that are i, for nblocks blocks.
 *
 * ak_blocks_fork: row r of the result goes on from row parents[r] (nnew rows from
 * nreq; a parent outside [0, nreq): an empty row): its length and its held
 * entries, -1 past them. Where the last block is partly filled, the row
 * will write into it next, so rows may not share it: of those that end in the
 * same block the lowest keeps it, if no other row holds it in another place,
 * and every other takes a block from free_blocks, front to back in row order,
 * enters it, and its copy is listed: pairs[i] = (from, to). counts[0] is how many copies
 * are wanted; past the free list (or at an entry of it outside [0, nblocks))
 * the table gets -1 and no pair is listed. Unused pairs are (-1, -1). refs as
 * ak_blocks_count would give for the result.
 *   out_table  device, nnew rows of table_width, out_stride apart; out_lens
 *              nnew int32; refs nblocks int32; pairs nnew * 2 int32; counts 1 int32
 *
 * ak_blocks_free: the blocks i with refs[i] <= 0 in increasing order, -1 past
 * them (free_blocks: nblocks int32), and their number (counts: 1 int32). The
 * list is one for ak_batch_layout and ak_blocks_fork.
 *
 * ak_blocks_compact: moves the n blocks in use (refs > 0) to 0 .. n-1: the
 * i-th of them that lies at n or past it, to the i-th free one before n. out_table
 * is the table with its held entries renamed (out_table may be block_table),
 * pairs (nblocks / 2 of them, unused ones (-1, -1)) the moves, counts[0] their number,
 * counts[1] n.
 *
 * ak_blocks_copy: copies blocks within a cache: for each pair (from, to) the
 * inner_bytes at o*outer_stride + from*block_stride to those at o*outer_stride +
 * to*block_stride, for all o < outer. Pairs with an id outside [0, nblocks)
 * are passed over, and those past count[0] (device; NULL: all npairs). No block that
 * is copied to is in another pair (those of fork and compact are such).
 *
 * Outputs overlap neither each other nor an input, except as stated. nblocks, nreq,
 * nnew below 2^30.
 * ------------------------------------------------------------------------- */
ak_status ak_blocks_count(const int32_t* block_table, int64_t table_stride, int32_t table_width, const int32_t* lens,
                          int64_t nreq, int32_t block_size, int64_t nblocks, int32_t* refs, const ak_opts* opts,
                          void* stream);
ak_status ak_blocks_fork_workspace_size(int64_t nnew, int64_t nblocks, const ak_opts* opts, size_t* bytes);
ak_status ak_blocks_fork(const int32_t* block_table, int64_t table_stride, int32_t table_width, const int32_t* lens,
                         int64_t nreq, const int32_t* parents, int64_t nnew, const int32_t* free_blocks, int64_t nfree,
                         int32_t block_size, int64_t nblocks, int32_t* out_table, int64_t out_stride,
                         int32_t* out_lens, int32_t* refs, int32_t* pairs, int32_t* counts, void* workspace,
                         size_t workspace_bytes, const ak_opts* opts, void* stream);
ak_status ak_blocks_free(const int32_t* refs, int64_t nblocks, int32_t* free_blocks, int32_t* counts,
                         const ak_opts* opts, void* stream);
ak_status ak_blocks_compact_workspace_size(int64_t nblocks, const ak_opts* opts, size_t* bytes);
ak_status ak_blocks_compact(const int32_t* block_table, int64_t table_stride, int32_t table_width, const int32_t* lens,
                            int64_t nreq, const int32_t* refs, int32_t block_size, int64_t nblocks,
                            int32_t* out_table, int64_t out_stride, int32_t* pairs, int32_t* counts, void* workspace,
                            size_t workspace_bytes, const ak_opts* opts, void* stream);
ak_status ak_blocks_copy(void* cache, int64_t outer, int64_t outer_stride, int64_t nblocks, int64_t block_stride,
                         int64_t inner_bytes, const int32_t* pairs, int64_t npairs, const int32_t* count,
                         const ak_opts* opts, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* AK_H */
