// gdn2_scan.hip -- the selective state space scan over prompts, and of single tokens against a
// pool of states.
//
// Per channel d and state n, with the step dt_t[d] = softplus(dt_raw + dt_bias) (or their sum):
//     h_t = exp(dt_t A) h_{t-1} + dt_t B_t[n] x_t,   y_t = sum_n C_t[n] h_t + D x_t,
//     o_t = y_t silu(gate_t).
// The recurrence is elementwise in (d, n), with a decay of its own per token, channel and state,
// so it has no matrix form: its cost is one exp2 and four fp32 operations per (t, d, n) on the
// vector unit, about four times the time that x, dt, gate and o take from memory at 16 states.
//
// A lane owns one channel and up to 16 of its states, which makes the sum over n free of
// exchanges, and keeps h in registers along the tokens; B and C of eight tokens are staged in LDS
// for the workgroup's four waves and read by broadcast. Where channels and sequences alone do not
// fill the chip, the token axis is cut into tiles (packed sequences start and end anywhere in a
// tile): one pass forms each tile's state from zero and its sum of dt (the decay over a tile is
// exp(A sum dt)), a second chains the tiles, a third runs them from their true states. That costs
// the exp2 and three operations once more, so the rule takes it only when it is the faster.
//
// Measured: prompt of 4,096 tokens x 4,096 channels x 16 states, bf16, 131-146 us with the clock (59
// for the first pass, 8 for the chain, 78 for the last when they are timed one by one). The passes
// keep the vector unit 84 % busy: the states' own operations take 47 us in a scan run once, 86 us
// with the first pass, and the bytes 26 us. 16,384 x 2,048 packed 259-276 us.
#include <type_traits>

#include "gdn2_internal.h"
#include "gdn2_layer.h"
#include "gdn2_scan.h"

namespace gdn2 {

namespace {

constexpr int kFew = 4;      // states per lane where there are few tokens: see few()

// FINAL: runs a tile from its true state and writes o (and S_T). Otherwise: runs it from zero
// and writes its state, its sum of dt and whether one sequence passes through all of it.
// A batch of kB tokens has no branch between its tokens, so their LDS reads and arithmetic
// overlap; in a sequence's last batch the missing tokens take steps of zero, which leave h as
// it is.
template <typename T, int NS, int S, bool FINAL>
__global__ __launch_bounds__(256, FINAL ? 3 : 4) void scan_fwd_kernel(ScanArgs a) {
    using Lane = ScanLane<NS, S>;
    constexpr int NP = Lane::NP, ROW = FINAL ? 2 * NP : NP;
    __shared__ __align__(16) float s_bc[2][kB * ROW];
    const Lane l(a, blockIdx.x);
    const int64_t tile = tile_index();
    if (tile * a.tile >= a.map.total && tile > 0) return;      // the whole workgroup
    const int t0 = static_cast<int>(tile * a.tile);
    const int t1 = a.map.total - t0 < a.tile ? a.map.total : t0 + a.tile;
    const uint32_t c = l.c;
    const bool gated = FINAL && a.gate;
    float A2[NS], h[NS];
    load_rates(a, l, A2);
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.D ? a.D[c] : 0.f;
    float sum = 0.f;
    bool pass = false;
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = 0.f;
    for_spans(a.map, t0, t1, [&](const Span &s) {
        if (!s.starts && FINAL) {
            if constexpr (NS == kFew) walk_tiles(a, l, s, tile, A2, h);
            else load_tile(a, l, a.tiles_h, tile, h);
        } else if (s.starts && a.S0) {
            load_state<S == 1 || NS == kFew>(a, l, a.S0, s.i, h);
        } else {
#pragma unroll
            for (int n = 0; n < NS; ++n) h[n] = 0.f;
        }
        pass = !s.starts && !s.ends;
        Stage<T, NP, FINAL> st;
        T xr[kB], dr[kB], gr[kB];
        auto fetch = [&](int t) {
            const int m = s.hi - t;
            st.take(a, l.g, t, m);
            fetch_rows(static_cast<const T *>(a.dt) + t * a.dt_stride, a.dt_stride, c, m, dr);
            fetch_rows(static_cast<const T *>(a.x) + t * a.x_stride, a.x_stride, c, m, xr);
            if (gated) fetch_rows(static_cast<const T *>(a.gate) + t * a.gate_stride, a.gate_stride, c, m, gr);
        };
        if (s.lo < s.hi) {
            fetch(s.lo);
            st.put(s_bc[0]);
            __syncthreads();
        }
        int buf = 0;
        for (int t = s.lo; t < s.hi; t += kB, buf ^= 1) {
            float x[kB], d[kB], g[kB], y[kB] = {};
            widen(dr, d);
            widen(xr, x);
            if (gated) widen(gr, g);
            const int m = s.hi - t;
            if (m > kB) fetch(t + kB);
#pragma unroll
            for (int k = 0; k < kB; ++k) d[k] += bias;
            if (a.softplus)
#pragma unroll
                for (int k = 0; k < kB; ++k) d[k] = softplus(d[k]);
            if (m < kB)
#pragma unroll
                for (int k = 1; k < kB; ++k)
                    if (k >= m) d[k] = x[k] = 0.f;
            const float *bc = s_bc[buf] + l.n0;
#pragma unroll
            for (int k = 0; k < kB; ++k) {
                float b[NS];
                lds_row<NS>(bc + k * ROW, b);
                const float u = d[k] * x[k];
#pragma unroll
                for (int n = 0; n < NS; ++n)
                    h[n] = fmaf(__builtin_amdgcn_exp2f(d[k] * A2[n]), h[n], u * b[n]);
                if constexpr (FINAL) {
                    float cv[NS];
                    lds_row<NS>(bc + k * ROW + NP, cv);
                    y[k] = 0.f;
#pragma unroll
                    for (int n = 0; n < NS; ++n) y[k] = fmaf(cv[n], h[n], y[k]);
                } else {
                    sum += d[k];
                }
            }
            pin(h);
            if (FINAL) pin(y);
            if constexpr (FINAL) {
#pragma unroll
                for (int k = 0; k < kB; ++k) y[k] = fmaf(skip, x[k], sum_parts<S>(y[k]));
                if (gated)
#pragma unroll
                    for (int k = 0; k < kB; ++k) y[k] *= silu(g[k]);
                pin(y);
                if (l.on && l.part == 0) {
                    T *row = static_cast<T *>(a.o) + t * static_cast<int64_t>(a.channels);
#pragma unroll
                    for (int k = 0; k < kB; ++k) {
                        if (k < m) io<T>::st(elem(row, c), y[k]);
                        row += a.channels;
                    }
                }
            }
            if (m > kB) st.put(s_bc[buf ^ 1]);
            __syncthreads();
        }
        if (FINAL && s.ends && a.S_T) store_state(a, l, a.S_T, s.i, h);
    });
    if constexpr (!FINAL) {
        store_tile(a, l, a.tiles_h, tile, h);
        if (l.on && l.part == 0) a.tiles_dt[tile * a.channels + c] = sum;
        if (blockIdx.x == 0 && threadIdx.x == 0) a.tiles_pass[tile] = pass ? 1 : 0;
    }
}

// Chains the tiles: one thread per (state, channel).
__global__ __launch_bounds__(256) void scan_chain_kernel(ScanArgs a, int tiles) {
    chain_tiles<1>(a, a.tiles_h, tiles);
}

// Four of a channel's states, or of a row of B or C, from state n0 on: loaded without a condition
// (places behind the last state repeat one) and widened, with zeros there, when they are used. So
// a token's loads are all in flight before the first is waited for.
template <typename E, bool VEC>
struct Four {
    Raw<E, 4> v;
    __device__ __forceinline__ void load(const E *row, int n0, int states) {
        v.load(row + (n0 < states ? n0 : 0));
    }
    __device__ __forceinline__ void get(float (&x)[4], int n0, int states) const {
        v.get(x);
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = n0 < states ? x[j] : 0.f;
    }
};
template <typename E>
struct Four<E, false> {
    E v[4];
    __device__ __forceinline__ void load(const E *row, int n0, int states) {
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = row[n0 + j < states ? n0 + j : states - 1];
    }
    __device__ __forceinline__ void get(float (&x)[4], int n0, int states) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = n0 + j < states ? io<E>::val(v[j]) : 0.f;
    }
};

// T tokens of every sequence against its slot of a pool [num_slots][channels][d_state]. LP lanes
// per channel, four consecutive states per lane: a wave reads and writes 1 KiB of states in a
// row. Bound by that traffic; each state is read once and written once per call: 64 sequences x
// 4,096 channels x 16 fp32 states 12.3 us (36 MB, 2.9 TB/s). A workgroup
// keeps its channels' rates for several sequences, and loads the next one's state and token
// while it works on one. VEC: states, B and C are read in pieces of four.
template <typename T, typename TS, int LP, bool VEC>
__global__ __launch_bounds__(256) void scan_step_kernel(ScanStepArgs a) {
    constexpr int PER = 256 / LP;
    const int part = threadIdx.x & (LP - 1), n0 = 4 * part, states = a.d_state;
    const int c = blockIdx.x * PER + threadIdx.x / LP;
    const bool on = c < a.channels;
    const uint32_t cc = on ? c : a.channels - 1;
    const uint32_t bc = cc / (a.channels / a.groups) * states;       // in a row of B or C
    struct Token { T x, dt, gate; Four<T, VEC> b, c; };
    auto token = [&](int64_t row, Token &k) {
        k.x = *elem(static_cast<const T *>(a.x) + row * a.x_stride, cc);
        k.dt = *elem(static_cast<const T *>(a.dt) + row * a.dt_stride, cc);
        k.gate = T{};
        if (a.gate) k.gate = *elem(static_cast<const T *>(a.gate) + row * a.gate_stride, cc);
        k.b.load(static_cast<const T *>(a.B) + row * a.b_stride + bc, n0, states);
        k.c.load(static_cast<const T *>(a.C) + row * a.c_stride + bc, n0, states);
    };
    auto slot_of = [&](int64_t i) { return a.idx ? a.idx[i] : static_cast<int>(i); };
    auto in_pool = [&](int slot) { return slot >= 0 && slot < a.num_slots; };
    auto state_of = [&](int slot) {
        return static_cast<TS *>(a.state) + (static_cast<int64_t>(slot) * a.channels + cc) * states;
    };
    int64_t i = blockIdx.y;
    int slot = slot_of(i);
    Four<float, false> rates;
    Four<TS, VEC> next;
    Token first;
    rates.load(a.A + static_cast<int64_t>(cc) * states, n0, states);
    token(i * a.ntok, first);
    if (in_pool(slot)) next.load(state_of(slot), n0, states);
    const float bias = a.dt_bias ? a.dt_bias[cc] : 0.f, skip = a.D ? a.D[cc] : 0.f;
    float A2[4];
    rates.get(A2, n0, states);
#pragma unroll
    for (int j = 0; j < 4; ++j) A2[j] = rate2(A2[j]);
    for (; i < a.num_seqs; i += gridDim.y) {
        const int mine = slot;
        const Four<TS, VEC> old = next;
        Token k = first;
        if (i + gridDim.y < a.num_seqs) {
            slot = slot_of(i + gridDim.y);
            token((i + gridDim.y) * a.ntok, first);
            if (in_pool(slot)) next.load(state_of(slot), n0, states);
        }
        T *o = static_cast<T *>(a.o) + i * a.ntok * a.channels;
        if (!in_pool(mine)) {
            if (on && part == 0)
                for (int t = 0; t < a.ntok; ++t) io<T>::st(elem(o + t * static_cast<int64_t>(a.channels), cc), 0.f);
            continue;
        }
        float h[4];
        old.get(h, n0, states);
        for (int t = 0; t < a.ntok; ++t) {
            float b[4], cv[4];
            k.b.get(b, n0, states);
            k.c.get(cv, n0, states);
            const float x = io<T>::val(k.x), g = io<T>::val(k.gate);
            float d = io<T>::val(k.dt) + bias, y = 0.f;
            if (t + 1 < a.ntok) token(i * a.ntok + t + 1, k);
            if (a.softplus) d = softplus(d);
            const float u = d * x;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                h[j] = fmaf(__builtin_amdgcn_exp2f(d * A2[j]), h[j], u * b[j]);
                y = fmaf(cv[j], h[j], y);
            }
#pragma unroll
            for (int m = 1; m < LP; m <<= 1) y += __shfl_xor(y, m);
            y = fmaf(skip, x, y);
            if (a.gate) y *= silu(g);
            if (on && part == 0) io<T>::st(elem(o + t * static_cast<int64_t>(a.channels), cc), y);
        }
        TS *st = state_of(mine) + n0;
        if constexpr (VEC) {
            if (on && n0 < states) stv<TS, 4>(st, h);
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (on && n0 + j < states) io<TS>::st(st + j, h[j]);
        }
    }
}

template <typename T, int NS, int S>
hipError_t launch_fwd(const ScanArgs &a, hipStream_t st) {
    const int tiles = scan_tiles(a.map.total, a.tile);
    const int blocks = scan_blocks(a.channels, a.groups, S);
    const dim3 grid = scan_grid(blocks, tiles);
    if (a.chained) {        // what the last tile reaches goes nowhere
        hipLaunchKernelGGL((scan_fwd_kernel<T, NS, S, false>), scan_grid(blocks, tiles - 1), dim3(256), 0, st, a);
        const int64_t cols = static_cast<int64_t>(a.d_state) * a.channels;
        if constexpr (NS != kFew)
            hipLaunchKernelGGL(scan_chain_kernel, dim3(static_cast<unsigned>((cols + 255) / 256)), dim3(256),
                               0, st, a, tiles);
    }
    hipLaunchKernelGGL((scan_fwd_kernel<T, NS, S, true>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

// Few tokens leave most of the chip idle with 16 states per lane, and a call's time is that of its
// waves' start, one tile and the launches. With four states per lane a tile takes a third of the
// time, and the last pass chains the tiles itself (walk_tiles) instead of a launch in between:
// 197 tokens x 768 channels x 16 states 15.1 us against 21.9 us; 4 tokens 5.9 against 10.4 us. Taken
// up to three waves per SIMD and 32 tiles (320 x 1,536 x 16, 1,920 waves: 19.5 against 24.5 us; 197
// x 4,096, 3,328 waves: 21.9 against 22.7; 256 x 4,096, 4,096 waves: 25.8 against 23.9; 700 x 768, 44
// tiles: 26.9 both). At 32 lanes per channel a wave reads only eight neighbouring bytes of a tile's
// states, so that six tiles are the limit (96 tokens x 256 channels x 128 states 20.2 against 27.7 us;
// 197 tokens, 13 tiles, 30.7 against 28.4).
int few_parts(int d_state) {
    return d_state <= 8 ? 2 : d_state <= 16 ? 4 : d_state <= 32 ? 8 : d_state <= 64 ? 16 : 32;
}
bool few(const ScanArgs &a) {
    const int parts = few_parts(a.d_state), tiles = scan_tiles(a.map.total, a.tile);
    if (a.chained ? tiles > (parts < 32 ? 32 : 6) : a.tile > 16) return false;
    return static_cast<int64_t>(scan_blocks(a.channels, a.groups, parts)) * tiles * kScanWaves <= 3 * kSimds;
}

template <typename T>
hipError_t launch_fwd_t(const ScanArgs &a, hipStream_t st) {
    if (few(a)) {
        switch (few_parts(a.d_state)) {
        case 2: return launch_fwd<T, kFew, 2>(a, st);
        case 4: return launch_fwd<T, kFew, 4>(a, st);
        case 8: return launch_fwd<T, kFew, 8>(a, st);
        case 16: return launch_fwd<T, kFew, 16>(a, st);
        default: return launch_fwd<T, kFew, 32>(a, st);
        }
    }
    switch (scan_parts(a.d_state)) {
    case 1: return a.d_state <= 8 ? launch_fwd<T, 8, 1>(a, st) : launch_fwd<T, 16, 1>(a, st);
    case 2: return launch_fwd<T, 16, 2>(a, st);
    case 4: return launch_fwd<T, 16, 4>(a, st);
    default: return launch_fwd<T, 16, 8>(a, st);
    }
}

template <typename T, typename TS, int LP>
hipError_t launch_step(const ScanStepArgs &a, hipStream_t st) {
    // about 1,024 workgroups, four waves per SIMD, each with as many sequences as that leaves
    // (64 sequences x 4,096 channels x 16 states: 12.3 us; 512 14.7 us, one each 14.8 us)
    const int wide = (a.channels + 256 / LP - 1) / (256 / LP);
    int rows = (1024 + wide - 1) / wide;
    if (rows > a.num_seqs) rows = a.num_seqs;
    const dim3 grid(wide, rows);
    auto whole = [](const void *p, int64_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; };
    const bool vec = a.d_state % 4 == 0 && a.b_stride % 4 == 0 && a.c_stride % 4 == 0 &&
                     whole(a.state, 4 * sizeof(TS)) && whole(a.B, 4 * sizeof(T)) && whole(a.C, 4 * sizeof(T));
    if (vec) hipLaunchKernelGGL((scan_step_kernel<T, TS, LP, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((scan_step_kernel<T, TS, LP, false>), grid, dim3(256), 0, st, a);
    return hipGetLastError();
}

template <typename T, typename TS>
hipError_t launch_step_t(const ScanStepArgs &a, hipStream_t st) {
    if (a.d_state <= 4) return launch_step<T, TS, 1>(a, st);
    if (a.d_state <= 8) return launch_step<T, TS, 2>(a, st);
    if (a.d_state <= 16) return launch_step<T, TS, 4>(a, st);
    if (a.d_state <= 32) return launch_step<T, TS, 8>(a, st);
    if (a.d_state <= 64) return launch_step<T, TS, 16>(a, st);
    return launch_step<T, TS, 32>(a, st);
}

}  // namespace

int scan_parts(int d_state) { return d_state <= 16 ? 1 : d_state <= 32 ? 2 : d_state <= 64 ? 4 : 8; }

int scan_blocks(int channels, int groups, int parts) {
    const int per = channels / groups, w = kScanWaves * 64 / parts;
    return groups * ((per + w - 1) / w);
}

int scan_tiles(int total, int tile) { return total > tile ? (total + tile - 1) / tile : 1; }

// Tokens per tile. A dense batch whose sequences alone give 1,024 waves (one per SIMD) is not
// cut, waves without a channel counted as the others, since they take as long (see ScanLane): its
// tile is a sequence (16 x 1,024 tokens x 4,096 channels, 1,024 waves: 429 us against
// 503 us cut; 64 x 128 x 2,048, 2,048 waves: 81 against 140; but 12 x 512 x 4,096, 768 waves: 215
// against 182). Otherwise about three waves per SIMD, 16 tokens at least.
int scan_tile(int channels, int groups, int d_state, int batch, int seqlen, bool packed) {
    const int64_t total = static_cast<int64_t>(batch) * seqlen;
    const int64_t waves = static_cast<int64_t>(kScanWaves) * scan_blocks(channels, groups, scan_parts(d_state));
    if (!packed && (batch * waves >= kSimds || seqlen <= 16)) return seqlen > 0 ? seqlen : 1;
    const int64_t t = (total * waves / (3 * kSimds) + kB - 1) / kB * kB;
    return t < 16 ? 16 : static_cast<int>(t);
}

// Whether some sequence may reach over a tile's end.
bool scan_chained(int batch, int seqlen, bool packed, int tile) {
    return static_cast<int64_t>(batch) * seqlen > tile && (packed || tile != seqlen);
}

hipError_t launch_scan_fwd(const ScanArgs &a, hipStream_t st) {
    return a.bf16 ? launch_fwd_t<bf16_t>(a, st) : launch_fwd_t<float>(a, st);
}

hipError_t launch_scan_step(const ScanStepArgs &a, hipStream_t st) {
    if (a.bf16) return a.state_bf16 ? launch_step_t<bf16_t, bf16_t>(a, st) : launch_step_t<bf16_t, float>(a, st);
    return a.state_bf16 ? launch_step_t<float, bf16_t>(a, st) : launch_step_t<float, float>(a, st);
}

}  // namespace gdn2
