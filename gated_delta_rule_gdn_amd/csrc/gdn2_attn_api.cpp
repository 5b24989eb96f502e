// gdn2_attn_api.cpp -- the extern "C" boundary of the attention layer of hybrid stacks: argument
// validation, workspace sizing and dispatch. Every check runs on the host before anything is
// enqueued, so a rejected call has no effect on the device.
#include <hip/hip_runtime.h>

#include <cmath>

#include "gdn2.h"
#include "gdn2_checks.h"
#include "gdn2_internal.h"

namespace {

using namespace gdn2::checks;
using gdn2::report;

constexpr int64_t kMaxPlaces = (int64_t{1} << 31) - 1;    // of a pool of pages

// ---- norms and rotation ------------------------------------------------------------------

gdn2_status check_rotary(const gdn2_rotary_dims *d, bool backward) {
    if (!d) return report(GDN2_ERR_NULL_ARG, "dims is NULL");
    if (!dtype_ok(d->dtype)) return report(GDN2_ERR_UNSUPPORTED, "dtype must be GDN2_F32 or GDN2_BF16");
    if (backward && d->grad_dtype != GDN2_F32 && d->grad_dtype != d->dtype)
        return report(GDN2_ERR_UNSUPPORTED, "grad_dtype must be GDN2_F32 or dtype");
    if (d->batch < 0 || d->seqlen < 0) return report(GDN2_ERR_BAD_SHAPE, "batch and seqlen must be >= 0");
    const int64_t tokens = static_cast<int64_t>(d->batch) * d->seqlen;
    if (tokens > kMaxTokens) return report(GDN2_ERR_BAD_SHAPE, "more than 2^30 tokens");
    if (d->d < 2 || d->d > 512 || d->d % 2 != 0) return report(GDN2_ERR_UNSUPPORTED, "d must be even, 2 .. 512");
    if (d->d_rot < 0 || d->d_rot > d->d || d->d_rot % 2 != 0)
        return report(GDN2_ERR_BAD_SHAPE, "d_rot must be even, 0 .. d");
    if (d->h_q < 1 || d->h_k < 0) return report(GDN2_ERR_BAD_SHAPE, "h_q must be >= 1 and h_k >= 0");
    if (static_cast<int64_t>(d->h_q) * d->d > kMaxChannels || static_cast<int64_t>(d->h_k) * d->d > kMaxChannels)
        return report(GDN2_ERR_BAD_SHAPE, "a token's heads hold more than 2^20 values");
    if (d->num_positions < (d->d_rot > 0 ? 1 : 0)) return report(GDN2_ERR_BAD_SHAPE, "num_positions must be >= 1");
    if (!(d->eps >= 0.f && d->eps <= 1e30f)) return report(GDN2_ERR_BAD_SHAPE, "eps must be finite and >= 0");
    const int64_t qrow = static_cast<int64_t>(d->h_q) * d->d, krow = static_cast<int64_t>(d->h_k) * d->d;
    int64_t s;
    if (!take_stride(d->q_stride, qrow, tokens, &s) || !take_stride(d->k_stride, krow, tokens, &s) ||
        !take_stride(d->v_stride, krow, tokens, &s))
        return report(GDN2_ERR_BAD_SHAPE, "a stride is smaller than its row or a tensor too large");
    return GDN2_OK;
}

gdn2::RotaryArgs rotary_args(const gdn2_rotary_dims *d, const void *q, const void *k, const float *cos_sin,
                             const int32_t *positions, const float *q_weight, const float *k_weight) {
    gdn2::RotaryArgs a;
    a.q = q; a.k = k; a.cos_sin = cos_sin; a.positions = positions;
    a.q_weight = q_weight; a.k_weight = k_weight;
    a.tokens = d->batch * d->seqlen; a.seqlen = d->seqlen;
    a.h_q = d->h_q; a.h_k = d->h_k; a.d = d->d; a.d_rot = d->d_rot; a.num_positions = d->num_positions;
    a.q_stride = d->q_stride ? d->q_stride : static_cast<int64_t>(d->h_q) * d->d;
    a.k_stride = d->k_stride ? d->k_stride : static_cast<int64_t>(d->h_k) * d->d;
    a.v_stride = 0;
    a.eps = d->eps;
    a.interleaved = d->interleaved != 0;
    a.bf16 = d->dtype == GDN2_BF16;
    return a;
}

// An input that its own output may replace: then it has to be contiguous, which one token always is.
bool in_place_ok(const gdn2_rotary_dims *d, const void *in, const void *out, int64_t stride, int64_t row) {
    return in != out || stride == 0 || stride == row || (d->batch == 1 && d->seqlen == 1);
}

size_t rotary_bwd_bytes(const gdn2_rotary_dims *d) {
    return static_cast<size_t>(gdn2::kRotaryParts) * 2 * d->d * sizeof(float);
}

// ---- attention ---------------------------------------------------------------------------

gdn2_status check_attention(const gdn2_attention_dims *d) {
    if (!d) return report(GDN2_ERR_NULL_ARG, "dims is NULL");
    if (!dtype_ok(d->dtype)) return report(GDN2_ERR_UNSUPPORTED, "dtype must be GDN2_F32 or GDN2_BF16");
    if (d->num_seqs < 0 || d->new_tokens < 1)
        return report(GDN2_ERR_BAD_SHAPE, "num_seqs must be >= 0 and new_tokens >= 1");
    if (d->h_q < 1 || d->h_k < 1 || d->h_q % d->h_k != 0)
        return report(GDN2_ERR_BAD_SHAPE, "h_q must be a multiple of h_k, both >= 1");
    if (d->d != 64 && d->d != 128 && d->d != 256) return report(GDN2_ERR_UNSUPPORTED, "d must be 64, 128 or 256");
    if (static_cast<int64_t>(d->h_q) * d->d > kMaxChannels)
        return report(GDN2_ERR_BAD_SHAPE, "a token's heads hold more than 2^20 values");
    const int64_t tokens = static_cast<int64_t>(d->num_seqs) * d->new_tokens;
    if (tokens > kMaxTokens || tokens * d->h_q > kMaxPlaces)
        return report(GDN2_ERR_BAD_SHAPE, "more than 2^30 tokens or 2^31 rows of queries");
    if (d->page_size < 1 || d->num_pages < 0 || d->max_pages < 0)
        return report(GDN2_ERR_BAD_SHAPE, "page_size must be >= 1, num_pages and max_pages >= 0");
    // (the first quotient keeps the product inside 64 bits)
    if (d->num_pages > kMaxPlaces / d->page_size || static_cast<int64_t>(d->num_pages) * d->page_size > kMaxPlaces / d->h_k)
        return report(GDN2_ERR_BAD_SHAPE, "num_pages * h_k * page_size must be at most 2^31 - 1");
    if (static_cast<int64_t>(d->max_pages) * d->page_size > (int64_t{1} << 29))
        return report(GDN2_ERR_BAD_SHAPE, "max_pages * page_size must be at most 2^29");
    if (static_cast<int64_t>(d->num_seqs) * d->max_pages > kMaxElems)
        return report(GDN2_ERR_BAD_SHAPE, "page_table is too large");
    if (d->window < 0) return report(GDN2_ERR_BAD_SHAPE, "window must be >= 0");
    if (!std::isfinite(d->scale)) return report(GDN2_ERR_BAD_SHAPE, "scale must be finite");
    int64_t s;
    if (!take_stride(d->q_stride, static_cast<int64_t>(d->h_q) * d->d, tokens, &s))
        return report(GDN2_ERR_BAD_SHAPE, "q_stride is smaller than a token's heads or q too large");
    const gdn2::AttentionPlan p = gdn2::attention_plan(*d);
    if (p.groups > (int64_t{1} << 23))
        return report(GDN2_ERR_BAD_SHAPE, "more than 2^23 workgroups: too many sequences, heads or new tokens");
    return GDN2_OK;
}

bool al16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Sizes of the workspace: the parts' sums, their maxima and totals, and the sequences' numbers of them.
struct AttentionBytes {
    size_t o = 0, ml = 0, info = 0;
    AttentionBytes(const gdn2_attention_dims *d, const gdn2::AttentionPlan &p) {
        if (p.budget == 0) return;
        const size_t rows = static_cast<size_t>(p.max_parts * d->h_k * p.row_blocks) * p.row_tiles * 16;
        o = padded(rows * d->d * sizeof(float));
        ml = padded(rows * 2 * sizeof(float));
        info = padded(static_cast<size_t>(d->num_seqs) * 2 * sizeof(int32_t));
    }
    size_t total() const { return o + ml + info; }
};

}  // namespace

extern "C" {

gdn2_status gdn2_qk_rotary_fwd(const void *q, const void *k, const float *cos_sin,
                               const int32_t *positions, const float *q_weight, const float *k_weight,
                               void *q_out, void *k_out, const gdn2_rotary_dims *dims, void *stream) {
    const gdn2_status st = check_rotary(dims, false);
    if (st != GDN2_OK) return st;
    if (dims->batch == 0 || dims->seqlen == 0) return ok();
    const bool keys = dims->h_k > 0;
    if (!q || !q_out || (keys && (!k || !k_out)) || (dims->d_rot > 0 && !cos_sin))
        return report(GDN2_ERR_NULL_ARG, "q, k, cos_sin and their outputs are required");
    const int64_t qrow = static_cast<int64_t>(dims->h_q) * dims->d, krow = static_cast<int64_t>(dims->h_k) * dims->d;
    const void *kout = keys ? k_out : nullptr;
    const void *qouts[] = {q_out}, *qins[] = {keys ? k : nullptr, kout, cos_sin, positions, q_weight, k_weight};
    const void *kouts[] = {kout}, *kins[] = {q, cos_sin, positions, q_weight, k_weight};
    if (aliases(qouts, qins) || aliases(kouts, kins))
        return report(GDN2_ERR_BAD_SHAPE, "an output aliases an input or the other output");
    if (!in_place_ok(dims, q, q_out, dims->q_stride, qrow) || (keys && !in_place_ok(dims, k, kout, dims->k_stride, krow)))
        return report(GDN2_ERR_BAD_SHAPE, "only a contiguous input may be its own output");
    gdn2::RotaryArgs a = rotary_args(dims, q, k, cos_sin, positions, q_weight, keys ? k_weight : nullptr);
    a.q_out = q_out; a.k_out = k_out;
    return done(gdn2::launch_rotary(a, static_cast<hipStream_t>(stream)), "gdn2_qk_rotary_fwd launch");
}

size_t gdn2_qk_rotary_bwd_workspace_bytes(const gdn2_rotary_dims *dims) {
    return check_rotary(dims, true) == GDN2_OK ? rotary_bwd_bytes(dims) : 0;
}

gdn2_status gdn2_qk_rotary_bwd(const void *q, const void *k, const float *cos_sin,
                               const int32_t *positions, const float *q_weight, const float *k_weight,
                               const void *dq_out, const void *dk_out, void *dq, void *dk,
                               float *dq_weight, float *dk_weight, const gdn2_rotary_dims *dims,
                               void *workspace, size_t workspace_bytes, void *stream) {
    gdn2_status st = check_rotary(dims, true);
    if (st != GDN2_OK) return st;
    const bool tokens = dims->batch > 0 && dims->seqlen > 0, keys = dims->h_k > 0;
    if (!keys && !dk_weight) k_weight = nullptr;
    if (tokens && (!q || !dq_out || !dq || (keys && (!k || !dk_out || !dk)) || (dims->d_rot > 0 && !cos_sin)))
        return report(GDN2_ERR_NULL_ARG, "q, k, cos_sin, the incoming gradients, dq and dk are required");
    if ((q_weight && !dq_weight) || (k_weight && !dk_weight))
        return report(GDN2_ERR_NULL_ARG, "every weight needs its gradient");
    const void *outs[] = {dq, keys ? dk : nullptr, q_weight ? dq_weight : nullptr, k_weight ? dk_weight : nullptr};
    const void *ins[] = {q, k, cos_sin, positions, q_weight, k_weight, dq_out, dk_out, workspace};
    if (aliases(outs, ins)) return report(GDN2_ERR_BAD_SHAPE, "an output aliases an input, the workspace or another output");
    const bool weights = q_weight || k_weight;
    st = check_workspace(workspace, workspace_bytes, weights ? rotary_bwd_bytes(dims) : 0);
    if (st != GDN2_OK) return st;
    if (!tokens && !weights) return ok();
    gdn2::RotaryArgs a = rotary_args(dims, q, k, cos_sin, positions, q_weight, k_weight);
    a.dq_out = dq_out; a.dk_out = dk_out; a.dq = dq; a.dk = dk;
    a.dq_weight = dq_weight; a.dk_weight = dk_weight;
    a.partial = static_cast<float *>(workspace);
    a.grad_bf16 = dims->grad_dtype == GDN2_BF16;
    return done(gdn2::launch_rotary_bwd(a, static_cast<hipStream_t>(stream)), "gdn2_qk_rotary_bwd launch");
}

gdn2_status gdn2_qk_rotary_append(const void *q, const void *k, const void *v, const float *cos_sin,
                                  const int32_t *positions, const float *q_weight,
                                  const float *k_weight, const int32_t *slots, void *q_out,
                                  void *k_pages, void *v_pages, int32_t num_pages, int32_t page_size,
                                  const gdn2_rotary_dims *dims, void *stream) {
    const gdn2_status st = check_rotary(dims, false);
    if (st != GDN2_OK) return st;
    if (dims->h_k < 1) return report(GDN2_ERR_BAD_SHAPE, "h_k must be >= 1");
    if (num_pages < 0 || page_size < 1) return report(GDN2_ERR_BAD_SHAPE, "num_pages must be >= 0 and page_size >= 1");
    const int64_t places = static_cast<int64_t>(num_pages) * page_size;
    const int64_t krow = static_cast<int64_t>(dims->h_k) * dims->d;
    if (places > kMaxPlaces || places > kMaxElems / krow)
        return report(GDN2_ERR_BAD_SHAPE, "num_pages * page_size must be at most 2^31 - 1, and the pool at most 2^40 values");
    if (dims->batch == 0 || dims->seqlen == 0) return ok();
    if (!q || !k || !v || !positions || !slots || !q_out || (places > 0 && (!k_pages || !v_pages)) ||
        (dims->d_rot > 0 && !cos_sin))
        return report(GDN2_ERR_NULL_ARG, "q, k, v, cos_sin, positions, slots, q_out and the pages are required");
    const void *qouts[] = {q_out}, *qins[] = {k, v, cos_sin, positions, q_weight, k_weight, slots, k_pages, v_pages};
    const void *pouts[] = {k_pages, v_pages}, *pins[] = {q, k, v, cos_sin, positions, q_weight, k_weight, slots};
    if (aliases(qouts, qins) || aliases(pouts, pins))
        return report(GDN2_ERR_BAD_SHAPE, "an output aliases an input or another output");
    if (!in_place_ok(dims, q, q_out, dims->q_stride, static_cast<int64_t>(dims->h_q) * dims->d))
        return report(GDN2_ERR_BAD_SHAPE, "only a contiguous input may be its own output");
    gdn2::RotaryArgs a = rotary_args(dims, q, k, cos_sin, positions, q_weight, k_weight);
    a.v = v; a.v_stride = dims->v_stride ? dims->v_stride : krow;
    a.q_out = q_out; a.k_out = k_pages; a.v_out = v_pages;
    a.slots = slots; a.num_places = places; a.page_size = page_size;
    return done(gdn2::launch_rotary(a, static_cast<hipStream_t>(stream)), "gdn2_qk_rotary_append launch");
}

size_t gdn2_paged_attention_step_workspace_bytes(const gdn2_attention_dims *dims) {
    if (check_attention(dims) != GDN2_OK || dims->num_seqs == 0) return 0;
    return AttentionBytes(dims, gdn2::attention_plan(*dims)).total();
}

gdn2_status gdn2_paged_attention_step(const void *q, const void *k_pages, const void *v_pages,
                                      const int32_t *page_table, const int32_t *seq_lens, void *o,
                                      float *lse, const gdn2_attention_dims *dims, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    gdn2_status st = check_attention(dims);
    if (st != GDN2_OK) return st;
    if (dims->num_seqs == 0) return ok();
    const bool cached = dims->num_pages > 0 && dims->max_pages > 0;
    if (!q || !seq_lens || !o || (cached && (!k_pages || !v_pages || !page_table)))
        return report(GDN2_ERR_NULL_ARG, "q, the pages, page_table, seq_lens and o are required");
    const void *outs[] = {o, lse}, *ins[] = {q, k_pages, v_pages, page_table, seq_lens, workspace};
    if (aliases(outs, ins)) return report(GDN2_ERR_BAD_SHAPE, "an output aliases an input, the workspace or the other output");
    if (!al16(k_pages) || !al16(v_pages) || !al16(o))
        return report(GDN2_ERR_BAD_SHAPE, "the pages and o must be 16-byte aligned");
    const gdn2::AttentionPlan p = gdn2::attention_plan(*dims);
    const AttentionBytes bytes(dims, p);
    st = check_workspace(workspace, workspace_bytes, bytes.total());
    if (st != GDN2_OK) return st;
    gdn2::AttentionArgs a;
    a.q = q; a.k_pages = k_pages; a.v_pages = v_pages; a.page_table = page_table; a.seq_lens = seq_lens;
    a.o = o; a.lse = lse;
    a.budget = static_cast<int>(p.budget);
    if (a.budget > 0) {
        char *w = static_cast<char *>(workspace);
        a.part_o = reinterpret_cast<float *>(w);
        a.part_ml = reinterpret_cast<float *>(w + bytes.o);
        a.part_info = reinterpret_cast<int32_t *>(w + bytes.o + bytes.ml);
    }
    a.num_seqs = dims->num_seqs; a.new_tokens = dims->new_tokens; a.h_q = dims->h_q; a.h_k = dims->h_k;
    a.d = dims->d; a.num_pages = dims->num_pages; a.page_size = dims->page_size;
    a.max_pages = cached ? dims->max_pages : 0;      // nothing cached: every sequence is empty
    a.window = dims->window;
    a.q_stride = dims->q_stride ? dims->q_stride : static_cast<int64_t>(dims->h_q) * dims->d;
    a.scale = dims->scale;
    a.bf16 = dims->dtype == GDN2_BF16;
    a.q_whole = al16(q) && a.q_stride % (a.bf16 ? 8 : 4) == 0;
    // with s = ceil(log2 p) and m = ceil(2^(31+s) / p), m p - 2^(31+s) < p <= 2^s: exact below 2^31
    int s = 0;
    while ((int64_t{1} << s) < dims->page_size) ++s;
    a.page_shift = 31 + s;
    a.page_mul = static_cast<uint32_t>(((uint64_t{1} << a.page_shift) + dims->page_size - 1) / dims->page_size);
    return done(gdn2::launch_attention(a, p, static_cast<hipStream_t>(stream)), "gdn2_paged_attention_step launch");
}

gdn2_status gdn2_pool_copy(void *const *pools, const int64_t *slot_bytes, int32_t num_pools,
                           int32_t num_slots, const int32_t *src, const int32_t *dst, int32_t count,
                           void *stream) {
    if (num_pools < 0 || num_slots < 0 || count < 0)
        return report(GDN2_ERR_BAD_SHAPE, "num_pools, num_slots and count must be >= 0");
    if (num_pools > 0 && (!pools || !slot_bytes)) return report(GDN2_ERR_NULL_ARG, "pools and slot_bytes are required");
    for (int p = 0; p < num_pools; ++p) {
        if (slot_bytes[p] < 1 || slot_bytes[p] > (int64_t{1} << 32) ||
            (num_slots > 0 && slot_bytes[p] > 4 * kMaxElems / num_slots))
            return report(GDN2_ERR_BAD_SHAPE, "slot_bytes must be 1 .. 2^32, and a pool at most 2^42 bytes");
        if (num_slots > 0 && !pools[p]) return report(GDN2_ERR_NULL_ARG, "a pool is NULL");
        for (int r = 0; r < p; ++r)
            if (num_slots > 0 && pools[r] == pools[p]) return report(GDN2_ERR_BAD_SHAPE, "a pool is given twice");
    }
    if (num_pools == 0 || num_slots == 0 || count == 0) return ok();
    if (!src || !dst) return report(GDN2_ERR_NULL_ARG, "src and dst are required");
    if (src == dst) return ok();      // every slot onto itself
    for (int p = 0; p < num_pools; ++p)
        if (pools[p] == src || pools[p] == dst) return report(GDN2_ERR_BAD_SHAPE, "a pool aliases src or dst");
    gdn2::CopyArgs a;
    a.src = src; a.dst = dst; a.num_slots = num_slots; a.count = count;
    for (int at = 0; at < num_pools; at += gdn2::kCopyPools) {
        a.num_pools = num_pools - at < gdn2::kCopyPools ? num_pools - at : gdn2::kCopyPools;
        for (int p = 0; p < a.num_pools; ++p) {
            a.pool[p] = pools[at + p];
            a.bytes[p] = slot_bytes[at + p];
        }
        const hipError_t e = gdn2::launch_pool_copy(a, static_cast<hipStream_t>(stream));
        if (e != hipSuccess) return gdn2::report_hip(e, "gdn2_pool_copy launch");
    }
    return ok();
}

}  // extern "C"
