// gdn2_layer_api.cpp -- the extern "C" boundary of the operators around the recurrence: argument
// validation, workspace sizing and dispatch. Every check runs on the host before anything is
// enqueued, so a rejected call has no effect on the device.
#include <hip/hip_runtime.h>

#include <initializer_list>

#include "gdn2.h"
#include "gdn2_internal.h"

namespace {

using gdn2::report;
using gdn2::report_hip;

constexpr int64_t kMaxElems = (int64_t{1} << 40);    // bound on any tensor's element count
constexpr int64_t kMaxTokens = (int64_t{1} << 30);   // token arithmetic stays in 32 bits
constexpr int32_t kMaxChannels = 1 << 20;

gdn2_status ok() { return report(GDN2_OK, ""); }

gdn2_status done(hipError_t e, const char *where) {
    return e == hipSuccess ? ok() : report_hip(e, where);
}

bool dtype_ok(int32_t t) { return t == GDN2_F32 || t == GDN2_BF16; }

// An output that is the same buffer as an input or as another output. NULLs are not compared.
template <int NO, int NI>
bool aliases(const void *const (&outs)[NO], const void *const (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        if (!outs[i]) continue;
        for (int j = 0; j < NI; ++j)
            if (outs[i] == ins[j]) return true;
        for (int j = i + 1; j < NO; ++j)
            if (outs[i] == outs[j]) return true;
    }
    return false;
}

// The token layout shared by the prompt calls: dense, or packed with cu_seqlens.
gdn2_status check_tokens(int32_t batch, int32_t seqlen, int32_t num_seqs, bool packed) {
    if (seqlen < 0) return report(GDN2_ERR_BAD_SHAPE, "seqlen must be >= 0");
    if (packed) {
        if (batch != 1) return report(GDN2_ERR_BAD_SHAPE, "packed batches need batch = 1");
        if (num_seqs < 1) return report(GDN2_ERR_BAD_SHAPE, "num_seqs must be >= 1");
    } else if (batch < 1) {
        return report(GDN2_ERR_BAD_SHAPE, "batch must be >= 1");
    }
    if (static_cast<int64_t>(batch) * seqlen > kMaxTokens || num_seqs > kMaxTokens)
        return report(GDN2_ERR_BAD_SHAPE, "more than 2^30 tokens or sequences");
    return GDN2_OK;
}

gdn2::SeqMap seq_map(const int32_t *cu, int32_t batch, int32_t seqlen, int32_t num_seqs) {
    return gdn2::SeqMap{cu, cu ? num_seqs : batch, seqlen, batch * seqlen};
}

// A token stride: 0 means contiguous. False if it is too small or the tensor too large.
bool take_stride(int64_t given, int64_t row, int64_t tokens, int64_t *out) {
    *out = given == 0 ? row : given;
    return *out >= row && *out <= kMaxElems && (tokens <= 0 || *out <= kMaxElems / tokens);
}

// ---- short convolution -------------------------------------------------------------------

gdn2_status check_conv(const gdn2_conv_dims *d, bool packed, bool backward) {
    if (!d) return report(GDN2_ERR_NULL_ARG, "dims is NULL");
    if (!dtype_ok(d->dtype)) return report(GDN2_ERR_UNSUPPORTED, "dtype must be GDN2_F32 or GDN2_BF16");
    if (backward && d->grad_dtype != GDN2_F32 && d->grad_dtype != d->dtype)
        return report(GDN2_ERR_UNSUPPORTED, "grad_dtype must be GDN2_F32 or dtype");
    if (d->width < 2 || d->width > 4) return report(GDN2_ERR_UNSUPPORTED, "width must be 2, 3 or 4");
    if (d->channels < 1 || d->channels > kMaxChannels)
        return report(GDN2_ERR_BAD_SHAPE, "channels must be 1 .. 2^20");
    const gdn2_status st = check_tokens(d->batch, d->seqlen, d->num_seqs, packed);
    if (st != GDN2_OK) return st;
    int64_t s;
    if (!take_stride(d->x_stride, d->channels, static_cast<int64_t>(d->batch) * d->seqlen, &s))
        return report(GDN2_ERR_BAD_SHAPE, "x_stride is smaller than channels or the tensor too large");
    const int64_t nseq = packed ? d->num_seqs : d->batch;
    if (nseq * d->channels * 3 > kMaxElems) return report(GDN2_ERR_BAD_SHAPE, "state tensor too large");
    return GDN2_OK;
}

gdn2::ConvArgs conv_args(const gdn2_conv_dims *d, const void *x, const float *weight,
                         const float *bias, const float *state0, const int32_t *cu, bool backward) {
    gdn2::ConvArgs a;
    a.x = x; a.weight = weight; a.bias = bias; a.state0 = state0;
    a.map = seq_map(cu, d->batch, d->seqlen, d->num_seqs);
    a.x_stride = d->x_stride ? d->x_stride : d->channels;
    a.channels = d->channels; a.width = d->width;
    a.tile = gdn2::conv_tile(a.map.total, a.channels, backward);
    a.silu = d->silu != 0;
    a.bf16 = d->dtype == GDN2_BF16;
    return a;
}

// ---- selective scan ----------------------------------------------------------------------

gdn2_status check_scan(const gdn2_scan_dims *d, bool packed, bool backward) {
    if (!d) return report(GDN2_ERR_NULL_ARG, "dims is NULL");
    if (!dtype_ok(d->dtype)) return report(GDN2_ERR_UNSUPPORTED, "dtype must be GDN2_F32 or GDN2_BF16");
    if (backward && d->grad_dtype != GDN2_F32 && d->grad_dtype != d->dtype)
        return report(GDN2_ERR_UNSUPPORTED, "grad_dtype must be GDN2_F32 or dtype");
    if (d->channels < 1 || d->channels > kMaxChannels)
        return report(GDN2_ERR_BAD_SHAPE, "channels must be 1 .. 2^20");
    if (d->groups < 1 || d->channels % d->groups != 0)
        return report(GDN2_ERR_BAD_SHAPE, "channels must be a multiple of groups");
    if (d->d_state < 1) return report(GDN2_ERR_BAD_SHAPE, "d_state must be >= 1");
    if (d->d_state > 128) return report(GDN2_ERR_UNSUPPORTED, "d_state must be 1 .. 128");
    const gdn2_status st = check_tokens(d->batch, d->seqlen, d->num_seqs, packed);
    if (st != GDN2_OK) return st;
    const int64_t tokens = static_cast<int64_t>(d->batch) * d->seqlen;
    const int64_t bc = static_cast<int64_t>(d->groups) * d->d_state;
    int64_t s;
    if (!take_stride(d->x_stride, d->channels, tokens, &s) ||
        !take_stride(d->dt_stride, d->channels, tokens, &s) ||
        !take_stride(d->gate_stride, d->channels, tokens, &s) ||
        !take_stride(d->b_stride, bc, tokens, &s) || !take_stride(d->c_stride, bc, tokens, &s))
        return report(GDN2_ERR_BAD_SHAPE, "a stride is smaller than its row or a tensor too large");
    const int64_t nseq = packed ? d->num_seqs : d->batch;
    if (nseq * d->channels * d->d_state > kMaxElems)
        return report(GDN2_ERR_BAD_SHAPE, "state tensor too large");
    return GDN2_OK;
}

template <typename Args>
void scan_inputs(Args *a, const gdn2_scan_dims *d, const void *x, const void *dt, const float *A,
                 const void *B, const void *C, const float *D, const void *gate, const float *dt_bias) {
    a->x = x; a->dt = dt; a->A = A; a->B = B; a->C = C; a->D = D; a->gate = gate; a->dt_bias = dt_bias;
    const int64_t bc = static_cast<int64_t>(d->groups) * d->d_state;
    a->x_stride = d->x_stride ? d->x_stride : d->channels;
    a->dt_stride = d->dt_stride ? d->dt_stride : d->channels;
    a->gate_stride = d->gate_stride ? d->gate_stride : d->channels;
    a->b_stride = d->b_stride ? d->b_stride : bc;
    a->c_stride = d->c_stride ? d->c_stride : bc;
    a->channels = d->channels; a->d_state = d->d_state; a->groups = d->groups;
    a->softplus = d->dt_softplus != 0;
    a->bf16 = d->dtype == GDN2_BF16;
}

// Whether rows of d_state floats can be taken in pieces of 16 bytes.
bool d_state_pieces(const gdn2_scan_dims *d, std::initializer_list<const float *> rows) {
    if (d->d_state % 4 != 0) return false;
    for (const float *p : rows)
        if (reinterpret_cast<uintptr_t>(p) % 16 != 0) return false;
    return true;
}

constexpr size_t kAlign = 256;
size_t padded(size_t bytes) { return (bytes + kAlign - 1) / kAlign * kAlign; }

// Sizes of the workspace: the tiles' states, sums and pass flags; backward also the states'
// gradients, a second array of sums, and the workgroups' shares of dB and dC.
struct ScanPlan {
    int tile, tiles;
    bool chained;
    size_t states, sums, flags, shares, kept_h, kept_dt;
    ScanPlan(const gdn2_scan_dims *d, bool packed, bool backward = false) {
        tile = backward ? gdn2::scan_bwd_tile(d->channels, d->groups, d->d_state, d->batch, d->seqlen, packed)
                        : gdn2::scan_tile(d->channels, d->groups, d->d_state, d->batch, d->seqlen, packed);
        tiles = gdn2::scan_tiles(d->batch * d->seqlen, tile);
        chained = gdn2::scan_chained(d->batch, d->seqlen, packed, tile);
        states = padded(static_cast<size_t>(tiles) * d->d_state * d->channels * sizeof(float));
        sums = padded(static_cast<size_t>(tiles) * d->channels * sizeof(float));
        flags = padded(static_cast<size_t>(tiles) * sizeof(int32_t));
        shares = padded(static_cast<size_t>(gdn2::scan_blocks(d->channels, d->groups, gdn2::scan_bwd_parts(d->d_state))) *
                        d->batch * d->seqlen * 2 * d->d_state * sizeof(float));
        const size_t kept = static_cast<size_t>(d->batch) * d->seqlen / 8 + 1;
        kept_h = padded(kept * d->d_state * d->channels * sizeof(float));
        kept_dt = padded(kept * d->channels * sizeof(float));
    }
    size_t fwd_bytes() const { return chained ? states + sums + flags : 0; }
    size_t bwd_bytes() const { return 2 * states + 2 * sums + flags + shares + kept_h + kept_dt; }
};

gdn2_status check_workspace(const void *ws, size_t bytes, size_t need) {
    if (need == 0) return GDN2_OK;
    if (!ws) return report(GDN2_ERR_WORKSPACE, "workspace is NULL");
    if (bytes < need) return report(GDN2_ERR_WORKSPACE, "workspace is too small");
    if (reinterpret_cast<uintptr_t>(ws) % kAlign != 0)
        return report(GDN2_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return GDN2_OK;
}

// ---- block norm --------------------------------------------------------------------------

gdn2_status check_norm(const gdn2_norm_dims *d, bool backward) {
    if (!d) return report(GDN2_ERR_NULL_ARG, "dims is NULL");
    if (!dtype_ok(d->dtype)) return report(GDN2_ERR_UNSUPPORTED, "dtype must be GDN2_F32 or GDN2_BF16");
    if (d->residual_dtype != GDN2_F32 && d->residual_dtype != d->dtype)
        return report(GDN2_ERR_UNSUPPORTED, "residual_dtype must be GDN2_F32 or dtype");
    if (backward && d->grad_dtype != GDN2_F32 && d->grad_dtype != d->dtype)
        return report(GDN2_ERR_UNSUPPORTED, "grad_dtype must be GDN2_F32 or dtype");
    if (d->d < 1) return report(GDN2_ERR_BAD_SHAPE, "d must be >= 1");
    if (d->d > 16384) return report(GDN2_ERR_UNSUPPORTED, "d must be 1 .. 16384");
    if (d->rows < 0 || d->rows > INT32_MAX) return report(GDN2_ERR_BAD_SHAPE, "rows must be 0 .. 2^31-1");
    if (!(d->eps >= 0.f && d->eps <= 1e30f)) return report(GDN2_ERR_BAD_SHAPE, "eps must be finite and >= 0");
    int64_t s;
    if (!take_stride(d->x_stride, d->d, d->rows, &s) || !take_stride(d->gate_stride, d->d, d->rows, &s))
        return report(GDN2_ERR_BAD_SHAPE, "a stride is smaller than d or a tensor too large");
    return GDN2_OK;
}

gdn2::NormArgs norm_args(const gdn2_norm_dims *d, const void *x, const void *gate, const void *residual,
                         const float *norm_weight, const float *scale, const float *next_weight) {
    gdn2::NormArgs a;
    a.x = x; a.gate = gate; a.residual = residual;
    a.norm_weight = norm_weight; a.scale = scale; a.next_weight = next_weight;
    a.rows = d->rows; a.d = d->d; a.eps = d->eps;
    a.x_stride = d->x_stride ? d->x_stride : d->d;
    a.gate_stride = d->gate_stride ? d->gate_stride : d->d;
    a.bf16 = d->dtype == GDN2_BF16;
    a.residual_f32 = a.bf16 && d->residual_dtype == GDN2_F32;
    a.grad_bf16 = d->grad_dtype == GDN2_BF16;
    return a;
}

}  // namespace

extern "C" {

gdn2_status gdn2_short_conv_fwd(const void *x, const float *weight, const float *bias,
                                const float *state0, const int32_t *cu_seqlens, void *y,
                                float *state_T, const gdn2_conv_dims *dims, void *stream) {
    gdn2_status st = check_conv(dims, cu_seqlens != nullptr, false);
    if (st != GDN2_OK) return st;
    const bool tokens = dims->batch > 0 && dims->seqlen > 0;
    if (!weight || (tokens && (!x || !y)))
        return report(GDN2_ERR_NULL_ARG, "x, weight and y are required");
    const void *outs[] = {y, state_T}, *ins[] = {x, weight, bias, state0, cu_seqlens};
    if (aliases(outs, ins)) return report(GDN2_ERR_BAD_SHAPE, "an output aliases an input or the other output");
    if (!tokens && !state_T) return ok();
    gdn2::ConvArgs a = conv_args(dims, x, weight, bias, state0, cu_seqlens, false);
    a.y = y; a.state_T = state_T;
    return done(gdn2::launch_conv_fwd(a, static_cast<hipStream_t>(stream)), "gdn2_short_conv_fwd launch");
}

size_t gdn2_short_conv_bwd_workspace_bytes(const gdn2_conv_dims *dims) {
    if (!dims || check_conv(dims, dims->num_seqs > 0 && dims->batch == 1, true) != GDN2_OK) return 0;
    const int64_t tokens = static_cast<int64_t>(dims->batch) * dims->seqlen;
    const int64_t tiles = gdn2::conv_tiles(tokens, gdn2::conv_tile(tokens, dims->channels, true));
    return static_cast<size_t>(tiles) * (dims->width + 1) * dims->channels * sizeof(float);
}

gdn2_status gdn2_short_conv_bwd(const void *x, const float *weight, const float *bias,
                                const float *state0, const int32_t *cu_seqlens, const void *dy,
                                const float *dstate_T, void *dx, float *dweight, float *dbias,
                                float *dstate0, const gdn2_conv_dims *dims, void *workspace,
                                size_t workspace_bytes, void *stream) {
    gdn2_status st = check_conv(dims, cu_seqlens != nullptr, true);
    if (st != GDN2_OK) return st;
    const bool tokens = dims->batch > 0 && dims->seqlen > 0;
    if (!weight || !dweight || (tokens && (!x || !dy || !dx)))
        return report(GDN2_ERR_NULL_ARG, "x, weight, dy, dx and dweight are required");
    if (bias && !dbias) return report(GDN2_ERR_NULL_ARG, "a bias needs dbias");
    const void *outs[] = {dx, dweight, dbias, dstate0};
    const void *ins[] = {x, weight, bias, state0, cu_seqlens, dy, dstate_T, workspace};
    if (aliases(outs, ins)) return report(GDN2_ERR_BAD_SHAPE, "an output aliases an input, the workspace or another output");
    gdn2::ConvArgs a = conv_args(dims, x, weight, bias, state0, cu_seqlens, true);
    const size_t need = static_cast<size_t>(gdn2::conv_tiles(a.map.total, a.tile)) * (a.width + 1) *
                        a.channels * sizeof(float);
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != GDN2_OK) return st;
    a.dy = dy; a.dstate_T = dstate_T; a.dx = dx; a.dweight = dweight; a.dbias = dbias; a.dstate0 = dstate0;
    a.partial = static_cast<float *>(workspace);
    a.grad_bf16 = dims->grad_dtype == GDN2_BF16;
    return done(gdn2::launch_conv_bwd(a, static_cast<hipStream_t>(stream)), "gdn2_short_conv_bwd launch");
}

gdn2_status gdn2_short_conv_step(const void *x, const float *weight, const float *bias,
                                 float *conv_state, const int32_t *state_idx, int32_t num_slots,
                                 void *y, const gdn2_conv_dims *dims, void *stream) {
    if (dims && dims->batch == 0) {     // an empty batch: the other dims still have to be right
        gdn2_conv_dims one = *dims;
        one.batch = 1;
        const gdn2_status st = check_conv(&one, false, false);
        return st != GDN2_OK ? st : ok();
    }
    gdn2_status st = check_conv(dims, false, false);
    if (st != GDN2_OK) return st;
    if (dims->seqlen < 1) return report(GDN2_ERR_BAD_SHAPE, "seqlen (tokens per sequence) must be >= 1");
    if (num_slots < 0) return report(GDN2_ERR_BAD_SHAPE, "num_slots must be >= 0");
    if (!state_idx && num_slots < dims->batch)
        return report(GDN2_ERR_BAD_SHAPE, "without state_idx, num_slots must be >= batch");
    if (static_cast<int64_t>(num_slots) * dims->channels * 3 > kMaxElems)
        return report(GDN2_ERR_BAD_SHAPE, "state tensor too large");
    if (!x || !weight || !y || (num_slots > 0 && !conv_state))
        return report(GDN2_ERR_NULL_ARG, "x, weight, conv_state and y are required");
    const void *outs[] = {y, conv_state}, *ins[] = {x, weight, bias, state_idx};
    if (aliases(outs, ins)) return report(GDN2_ERR_BAD_SHAPE, "y or the state aliases an input or the other");
    gdn2::ConvStepArgs a;
    a.x = x; a.weight = weight; a.bias = bias; a.state = conv_state; a.idx = state_idx; a.y = y;
    a.x_stride = dims->x_stride ? dims->x_stride : dims->channels;
    a.num_seqs = dims->batch; a.ntok = dims->seqlen; a.num_slots = num_slots;
    a.channels = dims->channels; a.width = dims->width;
    a.silu = dims->silu != 0;
    a.bf16 = dims->dtype == GDN2_BF16;
    return done(gdn2::launch_conv_step(a, static_cast<hipStream_t>(stream)), "gdn2_short_conv_step launch");
}

size_t gdn2_selective_scan_fwd_workspace_bytes(const gdn2_scan_dims *dims) {
    if (!dims) return 0;
    const bool packed = dims->num_seqs > 0 && dims->batch == 1;
    if (check_scan(dims, packed, false) != GDN2_OK) return 0;
    // sized for whichever layout the caller may use
    const size_t dense = ScanPlan(dims, false).fwd_bytes(), pk = packed ? ScanPlan(dims, true).fwd_bytes() : 0;
    return dense > pk ? dense : pk;
}

gdn2_status gdn2_selective_scan_fwd(const void *x, const void *dt, const float *A, const void *B,
                                    const void *C, const float *D, const void *gate,
                                    const float *dt_bias, const float *S0, const int32_t *cu_seqlens,
                                    void *o, float *S_T, const gdn2_scan_dims *dims, void *workspace,
                                    size_t workspace_bytes, void *stream) {
    const bool packed = cu_seqlens != nullptr;
    gdn2_status st = check_scan(dims, packed, false);
    if (st != GDN2_OK) return st;
    const bool tokens = dims->batch > 0 && dims->seqlen > 0;
    if (!A || (tokens && (!x || !dt || !B || !C || !o)))
        return report(GDN2_ERR_NULL_ARG, "x, dt, A, B, C and o are required");
    const void *outs[] = {o, S_T};
    const void *ins[] = {x, dt, A, B, C, D, gate, dt_bias, S0, cu_seqlens, workspace};
    if (aliases(outs, ins)) return report(GDN2_ERR_BAD_SHAPE, "an output aliases an input, the workspace or the other output");
    if (!tokens && !S_T) return ok();
    const ScanPlan p(dims, packed);
    st = check_workspace(workspace, workspace_bytes, p.fwd_bytes());
    if (st != GDN2_OK) return st;
    gdn2::ScanArgs a;
    scan_inputs(&a, dims, x, dt, A, B, C, D, gate, dt_bias);
    a.S0 = S0; a.o = o; a.S_T = S_T;
    a.map = seq_map(cu_seqlens, dims->batch, dims->seqlen, dims->num_seqs);
    a.tile = p.tile; a.chained = p.chained;
    a.vec = d_state_pieces(dims, {A, S0, S_T});
    if (p.chained) {
        char *w = static_cast<char *>(workspace);
        a.tiles_h = reinterpret_cast<float *>(w);
        a.tiles_dt = reinterpret_cast<float *>(w + p.states);
        a.tiles_pass = reinterpret_cast<int32_t *>(w + p.states + p.sums);
    }
    return done(gdn2::launch_scan_fwd(a, static_cast<hipStream_t>(stream)), "gdn2_selective_scan_fwd launch");
}

size_t gdn2_selective_scan_bwd_workspace_bytes(const gdn2_scan_dims *dims) {
    if (!dims) return 0;
    const bool packed = dims->num_seqs > 0 && dims->batch == 1;
    if (check_scan(dims, packed, true) != GDN2_OK) return 0;
    const size_t dense = ScanPlan(dims, false, true).bwd_bytes();
    const size_t pk = packed ? ScanPlan(dims, true, true).bwd_bytes() : 0;
    return dense > pk ? dense : pk;
}

gdn2_status gdn2_selective_scan_bwd(const void *x, const void *dt, const float *A, const void *B,
                                    const void *C, const float *D, const void *gate,
                                    const float *dt_bias, const float *S0, const int32_t *cu_seqlens,
                                    const void *dO, const float *dS_T, void *dx, void *ddt, float *dA,
                                    void *dB, void *dC, float *dD, void *dgate, float *ddt_bias,
                                    float *dS0, const gdn2_scan_dims *dims, void *workspace,
                                    size_t workspace_bytes, void *stream) {
    const bool packed = cu_seqlens != nullptr;
    gdn2_status st = check_scan(dims, packed, true);
    if (st != GDN2_OK) return st;
    const bool tokens = dims->batch > 0 && dims->seqlen > 0;
    if (!A || !dA || (tokens && (!x || !dt || !B || !C || !dO || !dx || !ddt || !dB || !dC)))
        return report(GDN2_ERR_NULL_ARG, "the inputs, dO, dx, ddt, dA, dB and dC are required");
    if ((D && !dD) || (dt_bias && !ddt_bias) || (tokens && gate && !dgate))
        return report(GDN2_ERR_NULL_ARG, "D, dt_bias and a gate need their gradients");
    const void *outs[] = {dx, ddt, dA, dB, dC, dD, dgate, ddt_bias, dS0};
    const void *ins[] = {x, dt, A, B, C, D, gate, dt_bias, S0, cu_seqlens, dO, dS_T, workspace};
    if (aliases(outs, ins)) return report(GDN2_ERR_BAD_SHAPE, "an output aliases an input, the workspace or another output");
    const ScanPlan p(dims, packed, true);
    st = check_workspace(workspace, workspace_bytes, p.bwd_bytes());
    if (st != GDN2_OK) return st;
    gdn2::ScanArgs a;
    scan_inputs(&a, dims, x, dt, A, B, C, D, gate, dt_bias);
    a.S0 = S0; a.dO = dO; a.dS_T = dS_T;
    a.dx = dx; a.ddt = ddt; a.dA = dA; a.dB = dB; a.dC = dC; a.dS0 = dS0;
    a.dD = D ? dD : nullptr; a.dgate = gate ? dgate : nullptr; a.ddt_bias = dt_bias ? ddt_bias : nullptr;
    a.map = seq_map(cu_seqlens, dims->batch, dims->seqlen, dims->num_seqs);
    a.tile = p.tile; a.chained = p.chained;
    a.vec = d_state_pieces(dims, {A, S0, dS_T, dS0});
    a.grad_bf16 = dims->grad_dtype == GDN2_BF16;
    char *w = static_cast<char *>(workspace);
    auto take = [&w](size_t bytes) {
        char *at = w;
        w += bytes;
        return reinterpret_cast<float *>(at);
    };
    a.tiles_h = take(p.states);
    a.tiles_g = take(p.states);
    a.tiles_dt = take(p.sums);
    a.tiles_db = take(p.sums);
    a.tiles_pass = reinterpret_cast<int32_t *>(take(p.flags));
    a.part_bc = take(p.shares);
    a.kept_h = take(p.kept_h);
    a.kept_dt = take(p.kept_dt);
    return done(gdn2::launch_scan_bwd(a, static_cast<hipStream_t>(stream)), "gdn2_selective_scan_bwd launch");
}

gdn2_status gdn2_selective_scan_step(const void *x, const void *dt, const float *A, const void *B,
                                     const void *C, const float *D, const void *gate,
                                     const float *dt_bias, void *state, int32_t state_dtype,
                                     const int32_t *state_idx, int32_t num_slots, void *o,
                                     const gdn2_scan_dims *dims, void *stream) {
    if (!dims) return report(GDN2_ERR_NULL_ARG, "dims is NULL");
    gdn2_scan_dims d = *dims;
    if (d.batch == 0) d.batch = 1;      // an empty batch: the other dims still have to be right
    gdn2_status st = check_scan(&d, false, false);
    if (st != GDN2_OK) return st;
    if (state_dtype != GDN2_STATE_F32 && state_dtype != GDN2_STATE_BF16)
        return report(GDN2_ERR_UNSUPPORTED, "state_dtype must be GDN2_STATE_F32 or GDN2_STATE_BF16");
    if (dims->batch == 0) return ok();
    if (d.seqlen < 1) return report(GDN2_ERR_BAD_SHAPE, "seqlen (tokens per sequence) must be >= 1");
    if (num_slots < 0) return report(GDN2_ERR_BAD_SHAPE, "num_slots must be >= 0");
    if (!state_idx && num_slots < d.batch)
        return report(GDN2_ERR_BAD_SHAPE, "without state_idx, num_slots must be >= batch");
    if (static_cast<int64_t>(num_slots) * d.channels * d.d_state > kMaxElems)
        return report(GDN2_ERR_BAD_SHAPE, "state tensor too large");
    if (!x || !dt || !A || !B || !C || !o || (num_slots > 0 && !state))
        return report(GDN2_ERR_NULL_ARG, "x, dt, A, B, C, the state and o are required");
    const void *outs[] = {o, state}, *ins[] = {x, dt, A, B, C, D, gate, dt_bias, state_idx};
    if (aliases(outs, ins)) return report(GDN2_ERR_BAD_SHAPE, "o or the state aliases an input or the other");
    gdn2::ScanStepArgs a;
    scan_inputs(&a, dims, x, dt, A, B, C, D, gate, dt_bias);
    a.state = state; a.idx = state_idx; a.o = o;
    a.num_seqs = d.batch; a.ntok = d.seqlen; a.num_slots = num_slots;
    a.state_bf16 = state_dtype == GDN2_STATE_BF16;
    return done(gdn2::launch_scan_step(a, static_cast<hipStream_t>(stream)), "gdn2_selective_scan_step launch");
}

gdn2_status gdn2_block_norm_fwd(const void *x, const void *gate, const void *residual,
                                const float *norm_weight, const float *scale,
                                const float *next_weight, void *h, void *y,
                                const gdn2_norm_dims *dims, void *stream) {
    gdn2_status st = check_norm(dims, false);
    if (st != GDN2_OK) return st;
    if (dims->rows == 0) return ok();
    if (!x || !h) return report(GDN2_ERR_NULL_ARG, "x and h are required");
    if (next_weight && !y) return report(GDN2_ERR_NULL_ARG, "next_weight needs y");
    // h may be the residual's own buffer: every value is read before its place is written
    const void *outs[] = {h, next_weight ? y : nullptr}, *ins[] = {x, gate, norm_weight, scale, next_weight};
    if (aliases(outs, ins) || (outs[1] && y == residual))
        return report(GDN2_ERR_BAD_SHAPE, "an output aliases an input or the other output");
    gdn2::NormArgs a = norm_args(dims, x, gate, residual, norm_weight, scale, next_weight);
    a.h = h; a.y = y;
    return done(gdn2::launch_norm(a, false, static_cast<hipStream_t>(stream)), "gdn2_block_norm_fwd launch");
}

size_t gdn2_block_norm_bwd_workspace_bytes(const gdn2_norm_dims *dims) {
    if (check_norm(dims, true) != GDN2_OK) return 0;
    return static_cast<size_t>(gdn2::norm_parts(dims->rows, dims->d)) * 3 * dims->d * sizeof(float);
}

gdn2_status gdn2_block_norm_bwd(const void *x, const void *gate, const void *residual,
                                const float *norm_weight, const float *scale,
                                const float *next_weight, const void *dh, const void *dy, void *dx,
                                void *dgate, void *dresidual, float *dnorm_weight, float *dscale,
                                float *dnext_weight, const gdn2_norm_dims *dims, void *workspace,
                                size_t workspace_bytes, void *stream) {
    gdn2_status st = check_norm(dims, true);
    if (st != GDN2_OK) return st;
    const bool rows = dims->rows > 0;
    if (rows && (!x || !dx)) return report(GDN2_ERR_NULL_ARG, "x and dx are required");
    if (rows && next_weight && !dy) return report(GDN2_ERR_NULL_ARG, "next_weight needs dy");
    if (rows && !dh && !next_weight) return report(GDN2_ERR_NULL_ARG, "without next_weight, dh is required");
    if (rows && ((gate && !dgate) || (residual && !dresidual)))
        return report(GDN2_ERR_NULL_ARG, "a gate needs dgate and a residual dresidual");
    if ((norm_weight && !dnorm_weight) || (scale && !dscale) || (next_weight && !dnext_weight))
        return report(GDN2_ERR_NULL_ARG, "every weight and scale needs its gradient");
    const void *outs[] = {dx, dgate, dresidual, dnorm_weight, dscale, dnext_weight};
    const void *ins[] = {x, gate, residual, norm_weight, scale, next_weight, dh, dy, workspace};
    if (aliases(outs, ins)) return report(GDN2_ERR_BAD_SHAPE, "an output aliases an input, the workspace or another output");
    const bool params = norm_weight || scale || next_weight;
    st = check_workspace(workspace, workspace_bytes,
                         params ? static_cast<size_t>(gdn2::norm_parts(dims->rows, dims->d)) * 3 * dims->d * sizeof(float) : 0);
    if (st != GDN2_OK) return st;
    if (!rows && !params) return ok();
    gdn2::NormArgs a = norm_args(dims, x, gate, residual, norm_weight, scale, next_weight);
    a.dh = dh; a.dy = dy; a.dx = dx; a.dgate = dgate; a.dresidual = residual ? dresidual : nullptr;
    a.dnorm_weight = dnorm_weight; a.dscale = dscale; a.dnext_weight = dnext_weight;
    a.partial = static_cast<float *>(workspace);
    return done(gdn2::launch_norm(a, true, static_cast<hipStream_t>(stream)), "gdn2_block_norm_bwd launch");
}

}  // extern "C"
