// gdn2_internal.h -- host-side launch interface between the C ABI layer and the kernels.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn2.h"

namespace gdn2 {

// Records a failure message for gdn2_last_error() on this thread and returns `st`.
gdn2_status report(gdn2_status st, const char *msg);
gdn2_status report_hip(hipError_t e, const char *where);

constexpr int kChunk = 64;   // chunk size of the chunked forward

// Optional fusions (gdn2_fusion): q/k L2-norm before the recurrence, gated RMS norm after.
struct Fusion {
    bool qk_norm = false;
    float l2eps = 0.f;
    const void *gate = nullptr;      // [.., h_v, d_v] input dtype, or NULL
    const float *nw = nullptr;       // [d_v] fp32
    float neps = 0.f;
    const float *cw = nullptr;       // short convolution taps [C][4] fp32, or NULL
    float *cst = nullptr;            // conv state [num_slots][3][C] fp32
    bool csilu = false;
    int gmode = 0;                   // GateMode of the b / w arguments (0: GDN-2 gates)
    float *cks = nullptr;            // chunked forward: state entering every chunk, or NULL
    void *cks16 = nullptr;           // the same as bf16 fragments (64-token path), or NULL
    void *cku16 = nullptr;           // U of every chunk as bf16 fragments (64-token path), or NULL
    char *bops = nullptr;            // with o == NULL: the backward's reverse-pass operands
    const void *bdo = nullptr;       // dO for bops
    void *tmat = nullptr;            // chunked forward, bf16: T = (I + A)^-1 per record, or NULL
    const float *ck_in = nullptr;    // with bops (64-token path): the state entering every chunk,
                                     // given (fp32, the layout of cks): no chain, no segment pass
};

struct DecodeArgs {
    const void *q, *k, *v, *log_alpha, *b, *w;
    void *S;                 // state pool [num_slots][h_v][d_k][d_v], fp32 or bf16
    const int32_t *idx;      // slot of each sequence, or NULL (slot n)
    void *o;
    int num_seqs, ntok, num_slots, h_k, h_v, d_k, d_v;
    bool bf16;               // input dtype
    bool state_bf16;         // state dtype
    Fusion fu;
};

struct ChunkArgs {
    const void *q, *k, *v, *log_alpha, *b, *w;
    const float *S0;
    const int32_t *cu_seqlens;   // NULL: dense
    void *o;
    float *S_T;
    char *workspace;
    int batch, seqlen, num_seqs, h_k, h_v, d_k, d_v;
    int chunk = kChunk;          // chunk size: 32, 64 or 128
    bool bf16;
    Fusion fu;
};

// Workspace layout of the chunked forward (all offsets 256-byte aligned):
//   [chunk map: int32[num_seqs + 1], packed batches only]
//   [per (chunk, value head) record of chunk_record_bytes()]
size_t chunk_record_bytes(int chunk, int d_k, int d_v, bool bf16);
int64_t chunk_upper_bound(int chunk, int batch, int seqlen, int num_seqs, bool packed);
size_t chunk_map_bytes(int num_seqs, bool packed);
size_t chunk_workspace_bytes(int chunk, int batch, int seqlen, int num_seqs, int h_v, int d_k,
                             int d_v, bool bf16, bool packed);
bool chunk_size_built(int chunk);

// Chunked backward (gdn2_chunk_bwd). Workspace: the forward's, then the state entering every
// chunk (fp32), a scratch o, then a per-record fp32 scratch.
struct BwdArgs {
    const void *q, *k, *v, *log_alpha, *b, *w;
    const float *S0;
    const int32_t *cu_seqlens;
    const void *dO;
    const float *dS_T;
    float *dq, *dk, *dv, *dw, *dla, *db, *dS0;
    char *workspace;
    int batch, seqlen, num_seqs, h_k, h_v, d_k, d_v;
    bool bf16;
    const float *ck_in = nullptr;    // the state entering every 64-token chunk, from the forward
                                     // (bf16 inputs: used instead of the re-run's chain), or NULL
};
size_t chunk_bwd_workspace_bytes(int batch, int seqlen, int num_seqs, int h_v, int d_k, int d_v,
                                 bool bf16, bool packed);
hipError_t launch_chunk_bwd(const BwdArgs &a, hipStream_t st);
// bf16 inputs (gdn2_bwd16.hip): the backward on bf16 matrix cores, with its own workspace.
size_t chunk_bwd16_workspace_bytes(int batch, int seqlen, int num_seqs, int h_v, int d_k, int d_v,
                                   bool packed);
hipError_t launch_chunk_bwd16(const BwdArgs &a, hipStream_t st);

// Gate mappings of other delta-rule variants onto the GDN-2 inputs (gdn2_map_gates).
enum GateMode { GATES_GDN2 = 0, GATES_KDA = 1, GATES_FG2 = 2, GATES_FG2_PLUS = 3, GATES_GDN = 4 };

struct GateArgs {
    int mode;
    const void *q, *k, *v, *log_alpha, *beta, *beta_v;
    void *q_out, *k_out, *v_out, *log_alpha_out, *b_out, *w_out;
    int64_t rows;            // tokens: batch x seqlen
    int h_k, h_v, d_k, d_v;
    bool bf16;
};

// The chain rule back through a gate mapping (gdn2_map_gates_bwd): the forward's k, v,
// beta, beta_v (input dtype), the fp32 gradients of the mapped inputs, the fp32 outputs.
struct GateBwdArgs {
    int mode;
    const void *k, *v, *beta, *beta_v;
    const float *dq_m, *dk_m, *dv_m, *dla_m, *db_m, *dw_m;
    float *dq, *dk, *dv, *dla, *dbeta, *dbeta_v;
    int64_t rows;
    int h_k, h_v, d_k, d_v;
    bool bf16;
};

// The sequences on a token axis of `total` tokens: n of them, packed (offsets cu[n + 1] in
// device memory) or dense (cu NULL, seqlen tokens each).
struct SeqMap {
    const int32_t *cu;
    int n, seqlen, total;
};

// The short convolution over prompts (gdn2_short_conv_fwd, gdn2_short_conv_bwd).
struct ConvArgs {
    const void *x = nullptr, *dy = nullptr;
    const float *weight = nullptr, *bias = nullptr, *state0 = nullptr, *dstate_T = nullptr;
    void *y = nullptr, *dx = nullptr;
    float *state_T = nullptr, *dstate0 = nullptr, *dweight = nullptr, *dbias = nullptr;
    float *partial = nullptr;        // [tiles][width + 1][channels] sums of a backward call
    SeqMap map;
    int64_t x_stride;                // elements from one token of x to the next
    int channels, width, tile;
    bool silu, bf16, grad_bf16 = false;
};
int conv_tile(int64_t tokens, int channels, bool backward);    // tokens a wave takes
int64_t conv_tiles(int64_t tokens, int tile);            // at least one
hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t st);
hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t st);

// The short convolution of single tokens (gdn2_short_conv_step).
struct ConvStepArgs {
    const void *x;
    const float *weight, *bias;
    float *state;                    // [num_slots][width - 1][channels]
    const int32_t *idx;
    void *y;
    int64_t x_stride;
    int num_seqs, ntok, num_slots, channels, width;
    bool silu, bf16;
};
hipError_t launch_conv_step(const ConvStepArgs &a, hipStream_t st);

// The selective scan over prompts (gdn2_selective_scan_fwd, gdn2_selective_scan_bwd).
struct ScanArgs {
    const void *x, *dt, *B, *C, *gate;
    const float *A, *D, *dt_bias, *S0;
    void *o = nullptr;
    float *S_T = nullptr;
    SeqMap map;
    int64_t x_stride, dt_stride, b_stride, c_stride, gate_stride;
    int channels, d_state, groups, tile;
    bool softplus, bf16;
    bool vec;                        // rows of d_state floats can be taken in whole pieces of four
    bool chained;                    // sequences reach over tiles: the arrays below are used
    float *tiles_h = nullptr;        // [tiles][d_state][channels]: states reached, then entering
    float *tiles_dt = nullptr;       // [tiles][channels]: sums of dt
    int32_t *tiles_pass = nullptr;   // [tiles]: whether one sequence passes through the whole tile
    // the backward: gradients in and out, and its own workspace
    const void *dO = nullptr;
    const float *dS_T = nullptr;
    void *dx = nullptr, *ddt = nullptr, *dB = nullptr, *dC = nullptr, *dgate = nullptr;
    float *dA = nullptr, *dD = nullptr, *ddt_bias = nullptr, *dS0 = nullptr;
    bool grad_bf16 = false;
    float *tiles_g = nullptr;        // as tiles_h, of the states' gradients from the back
    float *tiles_db = nullptr;       // [tiles][channels]: sums for ddt_bias
    float *kept_h = nullptr;         // [tokens / 8 + 1][d_state][channels]: states on the way
    float *kept_dt = nullptr;        // [tokens / 8 + 1][channels]: sums of dt up to them
    float *part_bc = nullptr;        // [workgroups across channels][tokens][2][d_state]
};
constexpr int kScanMaxBwdTile = 64;  // tokens of a tile of the backward, which LDS holds whole
int scan_parts(int d_state);                              // lanes that share a channel's states
int scan_blocks(int channels, int groups, int parts);     // workgroups across the channels
int scan_tile(int channels, int groups, int d_state, int batch, int seqlen, bool packed);
int scan_tiles(int total, int tile);
bool scan_chained(int batch, int seqlen, bool packed, int tile);
int scan_bwd_parts(int d_state);                          // the same in the backward
int scan_bwd_tile(int channels, int groups, int d_state, int batch, int seqlen, bool packed);
hipError_t launch_scan_fwd(const ScanArgs &a, hipStream_t st);
hipError_t launch_scan_bwd(const ScanArgs &a, hipStream_t st);

// The selective scan of single tokens (gdn2_selective_scan_step).
struct ScanStepArgs {
    const void *x, *dt, *B, *C, *gate;
    const float *A, *D, *dt_bias;
    void *state;                     // [num_slots][channels][d_state], fp32 or bf16
    const int32_t *idx;
    void *o;
    int64_t x_stride, dt_stride, b_stride, c_stride, gate_stride;
    int num_seqs, ntok, num_slots, channels, d_state, groups;
    bool softplus, bf16, state_bf16;
};
hipError_t launch_scan_step(const ScanStepArgs &a, hipStream_t st);

// The norms around a block (gdn2_block_norm_fwd, gdn2_block_norm_bwd).
struct NormArgs {
    const void *x, *gate, *residual;
    const float *norm_weight, *scale, *next_weight;
    void *h = nullptr, *y = nullptr;
    const void *dh = nullptr, *dy = nullptr;
    void *dx = nullptr, *dgate = nullptr, *dresidual = nullptr;
    float *dnorm_weight = nullptr, *dscale = nullptr, *dnext_weight = nullptr;
    float *partial = nullptr;        // [norm_parts()][3][d] sums of a backward call
    int64_t rows, x_stride, gate_stride;
    int d;
    float eps;
    bool bf16, residual_f32, grad_bf16 = false;
};
int norm_lanes(int d);                        // lanes that hold a row
int64_t norm_sets(int64_t rows, int d);       // workgroups that hold all rows
int64_t norm_parts(int64_t rows, int d);      // rows of the partial sums
hipError_t launch_norm(const NormArgs &a, bool backward, hipStream_t st);

// Norms of queries and keys with the rotation by position (gdn2_qk_rotary_fwd, _bwd, _append).
struct RotaryArgs {
    const void *q, *k, *v = nullptr;
    const float *cos_sin;            // [num_positions][d_rot]
    const int32_t *positions;        // NULL: token t % seqlen
    const float *q_weight, *k_weight;
    void *q_out = nullptr, *k_out = nullptr;       // k_out, v_out: the pages with `slots`
    void *v_out = nullptr;
    const int32_t *slots = nullptr;
    int64_t num_places = 0;          // num_pages * page_size
    int page_size = 1;
    const void *dq_out = nullptr, *dk_out = nullptr;
    void *dq = nullptr, *dk = nullptr;
    float *dq_weight = nullptr, *dk_weight = nullptr;
    float *partial = nullptr;        // [kRotaryParts][2][d] sums of a backward call
    int64_t q_stride, k_stride, v_stride = 0;
    int tokens, seqlen, h_q, h_k, d, d_rot, num_positions;
    int row_heads = 0;               // heads of a token that a wave takes at once: a power of two
    float eps, inv_d = 0.f;
    bool interleaved, bf16, grad_bf16 = false;
};
// Most rows of the partial sums: workgroups of a backward call, four per CU. (Three with accesses of eight
// values, where the fourth would wait: 8,192 tokens x 32 heads of 128 47.9 us in place of 40.9.)
constexpr int kRotaryParts = 1024;
hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st);
hipError_t launch_rotary_bwd(const RotaryArgs &a, hipStream_t st);

// Attention of new tokens over a paged cache (gdn2_paged_attention_step).
struct AttentionArgs {
    const void *q, *k_pages, *v_pages;
    const int32_t *page_table, *seq_lens;
    void *o;
    float *lse;
    float *part_o = nullptr;         // [workgroups][rows of a workgroup][d]: sums of a part of a sequence
    float *part_ml = nullptr;        // [workgroups][rows of a workgroup][2]: their maxima and totals
    int32_t *part_info = nullptr;    // [num_seqs][2]: a sequence's first part, and its number of parts
    int budget = 0;                  // of the plan
    int64_t q_stride;
    int num_seqs, new_tokens, h_q, h_k, d, num_pages, page_size, max_pages, window;
    uint32_t page_mul;               // x / page_size = x * page_mul >> page_shift for x < 2^31
    int page_shift;
    float scale;
    bool bf16;
    bool q_whole;                    // rows of q can be taken in whole pieces of 16 bytes
};
struct AttentionPlan {
    int row_tiles;                   // tiles of 16 rows that a workgroup takes
    int64_t row_blocks;              // workgroups that share a (sequence, key head)'s rows
    int64_t budget;                  // parts of sequences that run at once; 0: no sequence is cut
    int64_t max_parts;               // most parts that all sequences together are cut into
    int64_t groups;                  // workgroups: a part's key heads in eights, times row_blocks
};
AttentionPlan attention_plan(const gdn2_attention_dims &d);
hipError_t launch_attention(const AttentionArgs &a, const AttentionPlan &p, hipStream_t st);

// Slots of pools copied (gdn2_pool_copy).
constexpr int kCopyPools = 64;       // pools of one launch
struct CopyArgs {
    void *pool[kCopyPools];
    int64_t bytes[kCopyPools];       // of a slot
    int32_t first_piece[kCopyPools];     // of the workgroups that copy a pair: a pool's first one
    const int32_t *src, *dst;
    int num_pools, num_slots, count;
    int pieces, same_pieces;         // of all pools; of each, if they have the same, or 0
};
hipError_t launch_pool_copy(const CopyArgs &a, hipStream_t st);

hipError_t launch_decode(const DecodeArgs &a, hipStream_t st);
hipError_t launch_map_gates(const GateArgs &a, hipStream_t st);
hipError_t launch_map_gates_bwd(const GateBwdArgs &a, hipStream_t st);
hipError_t launch_chunk_fwd(const ChunkArgs &a, hipStream_t st);

}  // namespace gdn2
