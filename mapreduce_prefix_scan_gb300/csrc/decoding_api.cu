// decoding_api.cu -- the C entry points of the gated recurrence, the beam
// search and the cache's blocks: argument validation before anything touches
// the device, workspace sizing, dispatch.
#include <cmath>

#include "ak_internal.h"

using namespace ak;

static constexpr int64_t kMost = 0x7fffffff;
static constexpr int64_t kMostRows = 1 << 30;

static ak_status finish(ak_status s, const ak_opts* opts, void* stream) {
    if (s != AK_OK || !resolve_opts(opts).check) return s;
    return sync_and_check(static_cast<cudaStream_t>(stream));
}

static bool word_ptr(const void* p, bool needed) { return p ? aligned(p, 4) : !needed; }

// ===========================================================================
// ak_gated_recurrence
// ===========================================================================

static ak_status check_shape(const ak_recurrence* a) {
    if (!a || a->tokens < 0 || a->seqs < 0 || a->channels < 1 || a->tokens > kMost || a->seqs > kMostRows ||
        a->channels > kMostRows)
        return AK_ERR_INVALID_ARG;
    if (a->form != AK_RECURRENCE_DECAY && a->form != AK_RECURRENCE_GATE) return AK_ERR_INVALID_ARG;
    if (a->dtype < AK_F32 || a->dtype > AK_U8) return AK_ERR_INVALID_ARG;
    return a->dtype == AK_F32 || a->dtype == AK_BF16 ? AK_OK : AK_ERR_UNSUPPORTED;
}

// An array of a call that has tokens; the rows of an output do not overlap.
static bool good(const ak_recurrence* a, const ak_rows* x, bool output) {
    if (!x) return false;
    if (a->tokens == 0) return true;
    if (!x->data || !aligned(x->data, ak_dtype_size((ak_dtype)a->dtype)) || x->token_stride < 0) return false;
    return !output || a->tokens == 1 || x->token_stride >= a->channels;
}

// A shorter wait could run out where nothing is wrong.
static constexpr int64_t kLeastWait = 100000000;

static RecurrenceCall call_of(const ak_recurrence* a, const ak_opts& o) {
    RecurrenceCall c = {};
    c.epoch = next_epoch();
    c.wait_limit_ns = o.wait_limit_ns > kLeastWait ? o.wait_limit_ns : kLeastWait;
    c.skip_tile = o.debug_skip_publish_tile;
    c.dtype = (ak_dtype)a->dtype;
    c.form = a->form;
    c.tokens = a->tokens, c.seqs = a->seqs, c.channels = a->channels;
    return c;
}

// With opts->check: waits for the call and reports a wait that ran out.
static ak_status finish_recurrence(ak_status s, const RecurrenceCall& c, const ak_opts* opts, void* stream) {
    s = finish(s, opts, stream);
    if (s != AK_OK || !resolve_opts(opts).check) return s;
    bool lost = false;
    s = recurrence_lost(c.epoch, &lost);
    return s == AK_OK && lost ? AK_ERR_TIMEOUT : s;
}

extern "C" ak_status ak_gated_recurrence(const ak_recurrence* a, const ak_rows* x, const ak_rows* gate,
                                         const int32_t* offsets, const float* state_in, const ak_rows* h,
                                         float* state_out, const ak_opts* opts, void* stream) {
    const ak_status s = check_shape(a);
    if (s != AK_OK) return s;
    if (!good(a, x, false) || !good(a, gate, false) || !good(a, h, true)) return AK_ERR_INVALID_ARG;
    // in place the rows lie where they lay: others would be written before they are read
    if (a->tokens > 1 && h->data == x->data && h->token_stride != x->token_stride) return AK_ERR_INVALID_ARG;
    if (!word_ptr(offsets, a->seqs != 1) || !word_ptr(state_in, false) || !word_ptr(state_out, false))
        return AK_ERR_INVALID_ARG;
    if (a->tokens == 0 && (a->seqs == 0 || !state_out)) return AK_OK;
    RecurrenceCall c = call_of(a, resolve_opts(opts));
    c.x = *x, c.gate = *gate, c.out = *h;
    c.offsets = offsets, c.state_in = state_in, c.state_out = state_out;
    return finish_recurrence(run_recurrence(c, static_cast<cudaStream_t>(stream)), c, opts, stream);
}

extern "C" ak_status ak_gated_recurrence_backward(const ak_recurrence* a, const ak_rows* dh, const ak_rows* x,
                                                  const ak_rows* gate, const ak_rows* h, const int32_t* offsets,
                                                  const float* state_in, const float* dstate_out, const ak_rows* dx,
                                                  const ak_rows* dgate, float* dstate_in, const ak_opts* opts,
                                                  void* stream) {
    const ak_status s = check_shape(a);
    if (s != AK_OK) return s;
    const bool reads_x = a->form == AK_RECURRENCE_GATE;
    if (!good(a, dh, false) || (reads_x && !good(a, x, false)) || !good(a, gate, false) || !good(a, h, false) ||
        !good(a, dx, true) || !good(a, dgate, true))
        return AK_ERR_INVALID_ARG;
    if (!word_ptr(offsets, a->seqs != 1) || !word_ptr(state_in, false) || !word_ptr(dstate_out, false) ||
        !word_ptr(dstate_in, false))
        return AK_ERR_INVALID_ARG;
    if (a->tokens == 0 && (a->seqs == 0 || !dstate_in)) return AK_OK;
    RecurrenceCall c = call_of(a, resolve_opts(opts));
    c.dh = *dh, c.gate = *gate, c.h = *h, c.dx = *dx, c.dgate = *dgate;
    if (reads_x) c.x = *x;
    c.offsets = offsets, c.state_in = state_in, c.dstate_out = dstate_out, c.dstate_in = dstate_in;
    return finish_recurrence(run_recurrence_backward(c, static_cast<cudaStream_t>(stream)), c, opts, stream);
}

extern "C" ak_status ak_gated_recurrence_step(const ak_recurrence* a, const ak_rows* x, const ak_rows* gate,
                                              float* state, const int32_t* slots, int64_t nslots, const ak_rows* h,
                                              const ak_opts* opts, void* stream) {
    const ak_status s = check_shape(a);
    if (s != AK_OK) return s;
    if (!good(a, x, false) || !good(a, gate, false) || !good(a, h, true)) return AK_ERR_INVALID_ARG;
    if (nslots < 0 || !word_ptr(state, nslots > 0) || !word_ptr(slots, false)) return AK_ERR_INVALID_ARG;
    // a thread takes four channels of a request
    if ((a->channels + 3) / 4 > kMost * 256 / (a->tokens ? a->tokens : 1)) return AK_ERR_INVALID_ARG;
    if (a->tokens == 0) return AK_OK;
    RecurrenceCall c = call_of(a, resolve_opts(opts));
    c.x = *x, c.gate = *gate, c.out = *h;
    if (log_on())
        log_call("gated_recurrence_step requests=%lld channels=%lld: one launch", (long long)a->tokens, (long long)a->channels);
    return finish(run_recurrence_step(c, state, slots, nslots, static_cast<cudaStream_t>(stream)), opts, stream);
}

// ===========================================================================
// ak_beam_select, ak_beam_reorder
// ===========================================================================

extern "C" ak_status ak_beam_select(const void* logits, int64_t batch_stride, int64_t beam_stride, ak_dtype dtype,
                                    int64_t batch, int32_t beams, int64_t vocab, int32_t keep, const float* scores,
                                    const uint8_t* done, const int32_t* lengths, int32_t end_token, double penalty,
                                    float* out_scores, int32_t* out_tokens, int32_t* out_parents, uint8_t* out_done,
                                    int32_t* out_lengths, const ak_opts* opts, void* stream) {
    if (dtype < AK_F32 || dtype > AK_U8 || batch < 0 || batch > kMost / 16 || beams < 1 || beams > 32 || keep < 1 ||
        keep > 32 || vocab < 1 || vocab > kMost || end_token < -1 || end_token >= vocab || !std::isfinite(penalty))
        return AK_ERR_INVALID_ARG;
    if (dtype != AK_F32 && dtype != AK_BF16) return AK_ERR_UNSUPPORTED;
    if (batch == 0) return AK_OK;
    if (!logits || !aligned(logits, ak_dtype_size(dtype)) || batch_stride < 0 || beam_stride < 0) return AK_ERR_INVALID_ARG;
    if (!word_ptr(scores, true) || !word_ptr(lengths, false) || !word_ptr(out_scores, true) || !word_ptr(out_tokens, true) ||
        !word_ptr(out_parents, true) || !word_ptr(out_lengths, false))
        return AK_ERR_INVALID_ARG;
    // one request's outputs would lie in another's inputs, which are read at another time
    if (batch > 1 && keep != beams && (out_scores == scores || (done && out_done == done) || (lengths && out_lengths == lengths)))
        return AK_ERR_INVALID_ARG;
    BeamCall c = {};
    c.logits = logits, c.batch_stride = batch_stride, c.beam_stride = beam_stride, c.dtype = dtype;
    c.batch = batch, c.vocab = vocab, c.beams = beams, c.keep = keep, c.end = end_token, c.penalty = penalty;
    c.scores = scores, c.done = done, c.lengths = lengths;
    c.out_scores = out_scores, c.out_tokens = out_tokens, c.out_parents = out_parents;
    c.out_done = out_done, c.out_lengths = out_lengths;
    return finish(run_beam_select(c, static_cast<cudaStream_t>(stream)), opts, stream);
}

extern "C" ak_status ak_beam_reorder(void* state, int64_t outer, int64_t outer_stride, int64_t batch,
                                     int64_t batch_stride, int32_t beams, int64_t beam_stride, int64_t inner_bytes,
                                     const int32_t* parents, const ak_opts* opts, void* stream) {
    if (outer < 0 || batch < 0 || outer > kMost || batch > kMost || beams < 1 || beams > 32 || inner_bytes < 0 ||
        outer_stride < 0 || batch_stride < 0 || beam_stride < 0)
        return AK_ERR_INVALID_ARG;
    if (outer == 0 || batch == 0 || inner_bytes == 0) return AK_OK;
    if (!state || !word_ptr(parents, true)) return AK_ERR_INVALID_ARG;
    // rows that lie in one another cannot be traded
    if ((beams > 1 && beam_stride < inner_bytes) || (batch > 1 && batch_stride < inner_bytes) ||
        (outer > 1 && outer_stride < inner_bytes))
        return AK_ERR_INVALID_ARG;
    ReorderCall c = {};
    c.state = state, c.outer = outer, c.outer_stride = outer > 1 ? outer_stride : 0;
    c.batch = batch, c.batch_stride = batch > 1 ? batch_stride : 0;
    c.beams = beams, c.beam_stride = beams > 1 ? beam_stride : 0;
    c.inner = inner_bytes, c.parents = parents;
    if (log_on())
        log_call("beam_reorder outer=%lld requests=%lld beams=%d bytes=%lld: one launch", (long long)outer, (long long)batch,
                 beams, (long long)inner_bytes);
    return finish(run_beam_reorder(c, static_cast<cudaStream_t>(stream)), opts, stream);
}

// ===========================================================================
// ak_blocks_*
// ===========================================================================

// A block table and its requests' lengths.
static bool good_table(const int32_t* table, int64_t stride, int32_t width, const int32_t* lens, int64_t nreq,
                       int32_t block_size, int64_t nblocks) {
    if (nreq < 0 || nreq > kMostRows || width < 0 || block_size < 1 || nblocks < 0 || nblocks > kMostRows) return false;
    if (nreq == 0) return true;
    return word_ptr(lens, true) && (width == 0 || (word_ptr(table, true) && (nreq == 1 || stride >= width)));
}

static BlocksCall table_call(const int32_t* table, int64_t stride, int32_t width, const int32_t* lens, int64_t nreq,
                             int32_t block_size, int64_t nblocks) {
    BlocksCall c = {};
    c.table = table, c.table_stride = stride, c.width = width;
    c.lens = lens, c.rows = c.old_rows = nreq;
    c.block_size = block_size, c.blocks = nblocks;
    return c;
}

static bool good_workspace(const void* ws, size_t ws_bytes, size_t need) {
    return ws && ws_bytes >= need && aligned(ws, 16);
}

extern "C" ak_status ak_blocks_count(const int32_t* table, int64_t stride, int32_t width, const int32_t* lens,
                                     int64_t nreq, int32_t block_size, int64_t nblocks, int32_t* refs,
                                     const ak_opts* opts, void* stream) {
    if (!good_table(table, stride, width, lens, nreq, block_size, nblocks) || !word_ptr(refs, nblocks > 0))
        return AK_ERR_INVALID_ARG;
    if (nblocks == 0) return AK_OK;
    BlocksCall c = table_call(table, stride, width, lens, nreq, block_size, nblocks);
    c.refs = refs;
    if (log_on()) log_call("blocks_count requests=%lld blocks=%lld: one launch", (long long)nreq, (long long)nblocks);
    return finish(run_blocks_count(c, static_cast<cudaStream_t>(stream)), opts, stream);
}

extern "C" ak_status ak_blocks_fork_workspace_size(int64_t nnew, int64_t nblocks, const ak_opts* opts, size_t* bytes) {
    (void)opts;
    if (!bytes || nnew < 0 || nnew > kMostRows || nblocks < 0 || nblocks > kMostRows) return AK_ERR_INVALID_ARG;
    *bytes = blocks_fork_workspace(nnew, nblocks);
    return AK_OK;
}

extern "C" ak_status ak_blocks_fork(const int32_t* table, int64_t stride, int32_t width, const int32_t* lens,
                                    int64_t nreq, const int32_t* parents, int64_t nnew, const int32_t* free_blocks,
                                    int64_t nfree, int32_t block_size, int64_t nblocks, int32_t* out_table,
                                    int64_t out_stride, int32_t* out_lens, int32_t* refs, int32_t* pairs,
                                    int32_t* counts, void* ws, size_t ws_bytes, const ak_opts* opts, void* stream) {
    if (!good_table(table, stride, width, lens, nreq, block_size, nblocks) || nnew < 0 || nnew > kMostRows || nfree < 0)
        return AK_ERR_INVALID_ARG;
    if (!word_ptr(counts, true) || !word_ptr(refs, nblocks > 0) || !word_ptr(free_blocks, nfree > 0)) return AK_ERR_INVALID_ARG;
    if (nnew > 0 && (!word_ptr(parents, true) || !word_ptr(out_lens, true) || !word_ptr(pairs, true) ||
                     (width > 0 && (!word_ptr(out_table, true) || out_table == table || (nnew > 1 && out_stride < width))) ||
                     (nreq > 0 && out_lens == lens)))
        return AK_ERR_INVALID_ARG;
    if (!good_workspace(ws, ws_bytes, blocks_fork_workspace(nnew, nblocks))) return AK_ERR_WORKSPACE;
    BlocksCall c = table_call(table, stride, width, lens, nreq, block_size, nblocks);
    c.rows = nnew;
    c.parents = parents, c.free_blocks = free_blocks, c.nfree = nfree;
    c.out_table = out_table, c.out_stride = out_stride, c.out_lens = out_lens;
    c.refs = refs, c.pairs = pairs, c.counts = counts;
    if (log_on())
        log_call("blocks_fork requests=%lld of %lld blocks=%lld: one launch", (long long)nnew, (long long)nreq, (long long)nblocks);
    return finish(run_blocks_fork(c, ws, static_cast<cudaStream_t>(stream)), opts, stream);
}

extern "C" ak_status ak_blocks_free(const int32_t* refs, int64_t nblocks, int32_t* free_blocks, int32_t* counts,
                                    const ak_opts* opts, void* stream) {
    if (nblocks < 0 || nblocks > kMostRows || !word_ptr(refs, nblocks > 0) || !word_ptr(free_blocks, nblocks > 0) ||
        !word_ptr(counts, true))
        return AK_ERR_INVALID_ARG;
    BlocksCall c = {};
    c.refs = const_cast<int32_t*>(refs), c.blocks = nblocks, c.out_free = free_blocks, c.counts = counts;
    if (log_on()) log_call("blocks_free blocks=%lld: one launch", (long long)nblocks);
    return finish(run_blocks_free(c, static_cast<cudaStream_t>(stream)), opts, stream);
}

extern "C" ak_status ak_blocks_compact_workspace_size(int64_t nblocks, const ak_opts* opts, size_t* bytes) {
    (void)opts;
    if (!bytes || nblocks < 0 || nblocks > kMostRows) return AK_ERR_INVALID_ARG;
    *bytes = blocks_compact_workspace(nblocks);
    return AK_OK;
}

extern "C" ak_status ak_blocks_compact(const int32_t* table, int64_t stride, int32_t width, const int32_t* lens,
                                       int64_t nreq, const int32_t* refs, int32_t block_size, int64_t nblocks,
                                       int32_t* out_table, int64_t out_stride, int32_t* pairs, int32_t* counts,
                                       void* ws, size_t ws_bytes, const ak_opts* opts, void* stream) {
    if (!good_table(table, stride, width, lens, nreq, block_size, nblocks)) return AK_ERR_INVALID_ARG;
    if (!word_ptr(counts, true) || !word_ptr(refs, nblocks > 0) || !word_ptr(pairs, nblocks > 1)) return AK_ERR_INVALID_ARG;
    if (nreq > 0 && width > 0 && (!word_ptr(out_table, true) || (nreq > 1 && out_stride < width))) return AK_ERR_INVALID_ARG;
    // in place the rows lie where they lay
    if (nreq > 1 && width > 0 && out_table == table && out_stride != stride) return AK_ERR_INVALID_ARG;
    if (!good_workspace(ws, ws_bytes, blocks_compact_workspace(nblocks))) return AK_ERR_WORKSPACE;
    BlocksCall c = table_call(table, stride, width, lens, nreq, block_size, nblocks);
    c.refs = const_cast<int32_t*>(refs);
    c.out_table = out_table, c.out_stride = out_stride, c.pairs = pairs, c.counts = counts;
    if (log_on()) log_call("blocks_compact requests=%lld blocks=%lld: one launch", (long long)nreq, (long long)nblocks);
    return finish(run_blocks_compact(c, ws, static_cast<cudaStream_t>(stream)), opts, stream);
}

extern "C" ak_status ak_blocks_copy(void* cache, int64_t outer, int64_t outer_stride, int64_t nblocks,
                                    int64_t block_stride, int64_t inner_bytes, const int32_t* pairs, int64_t npairs,
                                    const int32_t* count, const ak_opts* opts, void* stream) {
    if (outer < 0 || outer > kMost || outer_stride < 0 || nblocks < 0 || nblocks > kMostRows || block_stride < 0 ||
        inner_bytes < 0 || npairs < 0 || npairs > kMostRows || !word_ptr(count, false))
        return AK_ERR_INVALID_ARG;
    if (outer == 0 || nblocks == 0 || inner_bytes == 0 || npairs == 0) return AK_OK;
    if (!cache || !word_ptr(pairs, true) || (nblocks > 1 && block_stride < inner_bytes) || (outer > 1 && outer_stride < inner_bytes))
        return AK_ERR_INVALID_ARG;
    BlocksCopyCall c = {};
    c.cache = cache, c.outer = outer, c.outer_stride = outer > 1 ? outer_stride : 0;
    c.blocks = nblocks, c.block_stride = nblocks > 1 ? block_stride : 0, c.inner = inner_bytes;
    c.pairs = pairs, c.npairs = npairs, c.count = count;
    if (log_on())
        log_call("blocks_copy pairs=%lld outer=%lld bytes=%lld: one launch", (long long)npairs, (long long)outer, (long long)inner_bytes);
    return finish(run_blocks_copy(c, static_cast<cudaStream_t>(stream)), opts, stream);
}
