// sequence_api.cu -- the C entry points of the sequence operators (batch
// layout, draft verification, linear attention): argument validation before
// anything touches the device, workspace sizing, dispatch.
#include <cmath>

#include "ak_internal.h"

using namespace ak;

static constexpr int64_t kMaxGrid = 0x7fffffff;

static ak_status finish(ak_status s, const ak_opts* opts, void* stream) {
    if (s != AK_OK || !resolve_opts(opts).check) return s;
    return sync_and_check(static_cast<cudaStream_t>(stream));
}

// ===========================================================================
// ak_batch_layout
// ===========================================================================

extern "C" ak_status ak_batch_layout_workspace_size(int64_t nreq, const ak_opts* opts, size_t* bytes) {
    (void)opts;
    if (!bytes || nreq < 0 || nreq > kMaxGrid) return AK_ERR_INVALID_ARG;
    *bytes = layout_workspace(nreq);
    return AK_OK;
}

extern "C" ak_status ak_batch_layout(const int32_t* ctx_lens, const int32_t* new_lens, int64_t nreq,
                                     int32_t* block_table, int64_t table_stride, int32_t table_width,
                                     const int32_t* free_blocks, int64_t nfree, int32_t block_size,
                                     int64_t max_tokens, int32_t* offsets, int64_t* slots, int32_t* positions,
                                     int32_t* requests, int32_t* counts, void* ws, size_t ws_bytes,
                                     const ak_opts* opts, void* stream) {
    if (nreq < 0 || nreq > kMaxGrid || table_width < 0 || nfree < 0 || block_size < 1 || max_tokens < 0 ||
        max_tokens > kMaxGrid)
        return AK_ERR_INVALID_ARG;
    if (!offsets || !counts || !aligned(offsets, 4) || !aligned(counts, 4)) return AK_ERR_INVALID_ARG;
    if (nreq > 0 && (!ctx_lens || !new_lens || !aligned(ctx_lens, 4) || !aligned(new_lens, 4)))
        return AK_ERR_INVALID_ARG;
    if (nreq > 0 && table_width > 0 && (!block_table || !aligned(block_table, 4) || table_stride < table_width))
        return AK_ERR_INVALID_ARG;
    if (nfree > 0 && (!free_blocks || !aligned(free_blocks, 4))) return AK_ERR_INVALID_ARG;
    if (max_tokens > 0 && (!slots || !positions || !requests || !aligned(slots, 8) || !aligned(positions, 4) ||
                           !aligned(requests, 4)))
        return AK_ERR_INVALID_ARG;
    const size_t need = layout_workspace(nreq);
    if (need > kWsHeader && (!ws || ws_bytes < need || !aligned(ws, 16))) return AK_ERR_WORKSPACE;
    LayoutCall c = {};
    c.ctx_lens = ctx_lens, c.new_lens = new_lens, c.nreq = nreq;
    c.table = block_table, c.table_stride = table_stride, c.table_width = table_width;
    c.free_blocks = free_blocks, c.nfree = nfree;
    c.block_size = block_size;
    c.block_shift = -1;
    if ((block_size & (block_size - 1)) == 0)
        for (c.block_shift = 0; (1 << c.block_shift) < block_size;) ++c.block_shift;
    c.max_tokens = max_tokens;
    c.offsets = offsets, c.slots = slots, c.positions = positions, c.requests = requests, c.counts = counts;
    c.vec = aligned(slots, 16) && aligned(positions, 16) && aligned(requests, 16);
    if (log_on())
        log_call("batch_layout requests=%lld max_tokens=%lld block=%d: %s", (long long)nreq, (long long)max_tokens,
                 block_size, need > kWsHeader ? "three launches" : "one launch");
    return finish(run_layout(c, ws, static_cast<cudaStream_t>(stream)), opts, stream);
}

// ===========================================================================
// ak_verify_drafts
// ===========================================================================

extern "C" ak_status ak_verify_drafts(const void* p, int64_t p_req, int64_t p_row, const void* q, int64_t q_req,
                                      int64_t q_row, ak_dtype dtype, const int32_t* drafts, const int32_t* counts,
                                      const float* uniform, const float* noise, int64_t noise_stride, int64_t nreq,
                                      int32_t k, int64_t vocab, int32_t* tokens, int32_t* accepted,
                                      const ak_opts* opts, void* stream) {
    if (dtype < AK_F32 || dtype > AK_U8 || nreq < 0 || k < 0 || vocab < 1 || vocab > kMaxGrid || k == 0x7fffffff)
        return AK_ERR_INVALID_ARG;
    if (dtype != AK_F32 && dtype != AK_BF16) return AK_ERR_UNSUPPORTED;
    if (nreq > kMaxGrid / 8) return AK_ERR_INVALID_ARG;
    if (nreq == 0) return AK_OK;
    const size_t esz = ak_dtype_size(dtype);
    if (!p || !aligned(p, esz) || p_req < 0 || p_row < 0 || !noise || !aligned(noise, 4) || noise_stride < 0)
        return AK_ERR_INVALID_ARG;
    if (q && (!aligned(q, esz) || q_req < 0 || q_row < 0)) return AK_ERR_INVALID_ARG;
    if (k > 0 && (!drafts || !uniform || !aligned(drafts, 4) || !aligned(uniform, 4))) return AK_ERR_INVALID_ARG;
    if (counts && !aligned(counts, 4)) return AK_ERR_INVALID_ARG;
    if (!tokens || !accepted || !aligned(tokens, 4) || !aligned(accepted, 4)) return AK_ERR_INVALID_ARG;
    VerifyCall c = {};
    c.p = p, c.p_req = p_req, c.p_row = p_row;
    c.q = q, c.q_req = q_req, c.q_row = q_row;
    c.dtype = dtype;
    c.drafts = drafts, c.counts = counts, c.uniform = uniform;
    c.noise = noise, c.noise_stride = noise_stride;
    c.nreq = nreq, c.k = k, c.vocab = vocab;
    c.tokens = tokens, c.accepted = accepted;
    if (log_on())
        log_call("verify_drafts requests=%lld drafts=%d vocab=%lld: one launch", (long long)nreq, k, (long long)vocab);
    return finish(run_verify(c, static_cast<cudaStream_t>(stream)), opts, stream);
}

// ===========================================================================
// ak_linear_attention
// ===========================================================================

static ak_status check_shape(const ak_linattn* a) {
    if (!a || a->tokens < 0 || a->seqs < 0 || a->max_len < 0 || a->heads < 1 || a->heads > 65535 || a->dk < 1 ||
        a->dv < 1 || a->dk > 256 || a->dv > 256 || a->reserved != 0 || !std::isfinite(a->scale))
        return AK_ERR_INVALID_ARG;
    if (a->tokens > kMaxGrid || a->seqs > kMaxGrid) return AK_ERR_INVALID_ARG;
    if (a->dtype < AK_F32 || a->dtype > AK_U8) return AK_ERR_INVALID_ARG;
    return a->dtype == AK_F32 || a->dtype == AK_BF16 ? AK_OK : AK_ERR_UNSUPPORTED;
}

// An input or output array of a call that has tokens.
static bool good(const ak_linattn* a, const ak_heads* x, int dim, bool output) {
    if (!x) return false;
    if (a->tokens == 0) return true;
    const size_t esz = ak_dtype_size((ak_dtype)a->dtype);
    if (!x->data || !aligned(x->data, esz) || x->token_stride < 0 || x->head_stride < 0) return false;
    // rows of an output must not overlap: one of the two strides spans the other
    if (!output) return true;
    const int64_t t = x->token_stride, h = x->head_stride;
    const bool heads_inside = (a->heads == 1 || h >= dim) && (a->tokens == 1 || t >= h * (a->heads - 1) + dim);
    const bool tokens_inside = (a->tokens == 1 || t >= dim) && (a->heads == 1 || h >= t * (a->tokens - 1) + dim);
    return heads_inside || tokens_inside;
}

static LinattnCall call_of(const ak_linattn* a, const ak_opts& o) {
    LinattnCall c = {};
    c.dtype = (ak_dtype)a->dtype;
    c.tokens = a->tokens, c.seqs = a->seqs;
    c.max_len = a->max_len > 0 && a->max_len < a->tokens ? a->max_len : a->tokens;
    c.heads = a->heads, c.dk = a->dk, c.dv = a->dv;
    c.scale = a->scale;
    c.windows = o.target_blocks > 0 ? o.target_blocks : 0;
    c.epoch = next_epoch();
    c.wait_limit_ns = o.wait_limit_ns;
    return c;
}

// A call that needs no more than the header uses it only to report a wait that
// ran out: without `check` it may be missing.
static ak_status check_workspace(const LinattnCall& c, const void* ws, size_t ws_bytes, bool check) {
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    const size_t need = linattn_workspace(c, dev);
    if (!ws && need == kWsHeader && !check) return AK_OK;
    return !ws || ws_bytes < need || !aligned(ws, 16) ? AK_ERR_WORKSPACE : AK_OK;
}

// With opts->check: waits for the call and reports a wait that ran out.
static ak_status finish_attention(ak_status s, const LinattnCall& c, const void* ws, const ak_opts* opts, void* stream) {
    s = finish(s, opts, stream);
    if (s != AK_OK || !resolve_opts(opts).check) return s;
    uint64_t word = 0;
    const cudaError_t e = cudaMemcpy(&word, ws, sizeof word, cudaMemcpyDeviceToHost);
    if (e != cudaSuccess) return cuda_fail(e);
    return word == c.epoch ? AK_ERR_TIMEOUT : AK_OK;
}

extern "C" ak_status ak_linear_attention_workspace_size(const ak_linattn* a, const ak_opts* opts, size_t* bytes) {
    ak_status s = check_shape(a);
    if (s != AK_OK) return s;
    if (!bytes) return AK_ERR_INVALID_ARG;
    DeviceInfo dev;
    if (!current_device(&dev)) return AK_ERR_CUDA;
    *bytes = linattn_workspace(call_of(a, resolve_opts(opts)), dev);
    return AK_OK;
}

static bool float_ptr(const void* p, bool needed) { return p ? aligned(p, 4) : !needed; }

extern "C" ak_status ak_linear_attention(const ak_linattn* a, const ak_heads* q, const ak_heads* k, const ak_heads* v,
                                         const float* log_decay, const int32_t* offsets, const float* state_in,
                                         const ak_heads* o, float* state_out, void* ws, size_t ws_bytes,
                                         const ak_opts* opts, void* stream) {
    ak_status s = check_shape(a);
    if (s != AK_OK) return s;
    if (!good(a, q, a->dk, false) || !good(a, k, a->dk, false) || !good(a, v, a->dv, false) || !good(a, o, a->dv, true))
        return AK_ERR_INVALID_ARG;
    if (!float_ptr(log_decay, true) || !float_ptr(offsets, a->seqs != 1) || !float_ptr(state_in, false) ||
        !float_ptr(state_out, false))
        return AK_ERR_INVALID_ARG;
    if (a->tokens == 0 && (a->seqs == 0 || !state_out)) return AK_OK;
    LinattnCall c = call_of(a, resolve_opts(opts));
    c.q = *q, c.k = *k, c.v = *v, c.o = *o;
    c.log_decay = log_decay, c.offsets = offsets, c.state_in = state_in, c.state_out = state_out;
    if ((s = check_workspace(c, ws, ws_bytes, resolve_opts(opts).check != 0)) != AK_OK) return s;
    return finish_attention(run_linattn(c, ws, static_cast<cudaStream_t>(stream)), c, ws, opts, stream);
}

extern "C" ak_status ak_linear_attention_backward(const ak_linattn* a, const ak_heads* d_o, const ak_heads* q,
                                                  const ak_heads* k, const ak_heads* v, const float* log_decay,
                                                  const int32_t* offsets, const float* state_in,
                                                  const float* dstate_out, const ak_heads* dq, const ak_heads* dk,
                                                  const ak_heads* dv, float* dstate_in, void* ws, size_t ws_bytes,
                                                  const ak_opts* opts, void* stream) {
    ak_status s = check_shape(a);
    if (s != AK_OK) return s;
    if (!good(a, q, a->dk, false) || !good(a, k, a->dk, false) || !good(a, v, a->dv, false) ||
        !good(a, d_o, a->dv, false) || !good(a, dq, a->dk, true) || !good(a, dk, a->dk, true) ||
        !good(a, dv, a->dv, true))
        return AK_ERR_INVALID_ARG;
    if (!float_ptr(log_decay, true) || !float_ptr(offsets, a->seqs != 1) || !float_ptr(state_in, false) ||
        !float_ptr(dstate_out, false) || !float_ptr(dstate_in, false))
        return AK_ERR_INVALID_ARG;
    // the three gradients are computed side by side: none may write what another reads
    if (dstate_in && (dstate_in == dstate_out || dstate_in == state_in)) return AK_ERR_INVALID_ARG;
    if (a->tokens == 0 && (a->seqs == 0 || !dstate_in)) return AK_OK;
    LinattnCall c = call_of(a, resolve_opts(opts));
    c.q = *q, c.k = *k, c.v = *v, c.o = *d_o;
    c.dq = *dq, c.dk_out = *dk, c.dvv = *dv;
    c.log_decay = log_decay, c.offsets = offsets, c.state_in = state_in;
    c.dstate_out = dstate_out, c.dstate_in = dstate_in;
    if ((s = check_workspace(c, ws, ws_bytes, resolve_opts(opts).check != 0)) != AK_OK) return s;
    return finish_attention(run_linattn_backward(c, ws, static_cast<cudaStream_t>(stream)), c, ws, opts, stream);
}

extern "C" ak_status ak_linear_attention_step(const ak_linattn* a, const ak_heads* q, const ak_heads* k,
                                              const ak_heads* v, const float* log_decay, float* state,
                                              const int32_t* slots, int64_t nslots, const ak_heads* o,
                                              const ak_opts* opts, void* stream) {
    ak_status s = check_shape(a);
    if (s != AK_OK) return s;
    if (!good(a, q, a->dk, false) || !good(a, k, a->dk, false) || !good(a, v, a->dv, false) || !good(a, o, a->dv, true))
        return AK_ERR_INVALID_ARG;
    if (nslots < 0 || !float_ptr(log_decay, true) || !float_ptr(state, nslots > 0) || !float_ptr(slots, false))
        return AK_ERR_INVALID_ARG;
    if (a->tokens == 0) return AK_OK;
    LinattnCall c = call_of(a, resolve_opts(opts));
    c.q = *q, c.k = *k, c.v = *v, c.o = *o;
    c.log_decay = log_decay;
    return finish(run_linattn_step(c, state, slots, nslots, static_cast<cudaStream_t>(stream)), opts, stream);
}
