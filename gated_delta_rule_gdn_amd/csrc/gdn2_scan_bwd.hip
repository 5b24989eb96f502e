// gdn2_scan_bwd.hip -- gradients of the selective scan.
//
// With dy = dO silu(gate), a_t = exp(dt_t A), and gh_t the gradient of the state h_t:
//     gh_t   = C_t dy_t + a_{t+1} gh_{t+1}          (dS_T after a sequence's last token)
//     dC_t   = sum_d dy h_t,                        dB_t = sum_d gh_t dt_t x_t
//     dx_t   = D dy + dt_t sum_n gh_t B_t,          dD = sum_t dy x
//     ddt_t  = x_t sum_n gh_t B_t + sum_n gh_t a_t h_{t-1} A,   through softplus' for the input
//     dA     = sum_t gh_t a_t h_{t-1} dt_t,         dS0 = a_0 gh_0,   dgate = dO y silu'(gate)
// Nothing but the inputs is kept from the forward. Four launches:
//   1. per tile of tokens: the state it reaches from zero, every eighth on the way, its sum of dt,
//      and what its outputs alone give back to the state that enters it
//      (sum_t prod_{s<=t} a_s C_t dy_t);
//   2. both chained over the tiles, one from the front, one from the back;
//   3. per tile, back over groups of eight tokens: their states again into registers, and the
//      gradients from the last to the first;
//   4. the sums over tiles (dA, dD, ddt_bias) and over workgroups of channels (dB, dC).
// Every sum has a fixed order: the same bits at every call.
//
// dB and dC sum over channels, which lie across the lanes. A wave reduces and spreads at once:
// each step sends half of a lane's values to the partner lane and adds the other half, so 8
// values over 32 lanes cost about 19 operations instead of 40 (reduce_spread).
//
// Bound by the vector unit: 4,096 tokens x 2,048 channels x 16 states, bf16, 239-250 us (180 for
// launch 3, at 75 % of the unit's issue, 62 for launch 1, 11 for the chain when they are timed one
// by one), against 120 us for the states' own operations and 23 us for the bytes.
#include "gdn2_internal.h"
#include "gdn2_layer.h"
#include "gdn2_scan.h"

namespace gdn2 {

namespace {

constexpr int kG = 8;        // tokens whose states are in registers together

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}

// x of the partner lane in a sum over lane bit BIT of a row of 16: rotation by 8, the mirror of
// eight lanes, and the two exchanges inside four. (The mirror pairs lane l with 7 - l: another
// lane of the other four, which is as good, since the sum goes on over those.)
template <int BIT>
__device__ __forceinline__ float partner(float x) {
    if constexpr (BIT == 3) return dpp<0x128>(x);          // row_ror:8
    else if constexpr (BIT == 2) return dpp<0x141>(x);     // row_half_mirror
    else if constexpr (BIT == 1) return dpp<0x4e>(x);      // quad_perm [2,3,0,1]
    else return dpp<0xb1>(x);                              // quad_perm [1,0,3,2]
}

// One step of the reduction over lane bit BIT of M values: where M > 1, lanes with the bit clear
// keep the sums of the first half, the others those of the second.
template <int BIT, int M>
__device__ __forceinline__ void spread_step(float *v) {
    if constexpr (BIT >= 4) {
        // swaps the upper half (of 64 lanes, or of each 32) of one register with the lower half
        // of the other, which is both lanes' share of the exchange
        constexpr int H = M > 1 ? M / 2 : 1;
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const uint32_t lo = __float_as_uint(v[i]), hi = __float_as_uint(v[M > 1 ? i + H : i]);
            const auto r = BIT == 5 ? __builtin_amdgcn_permlane32_swap(lo, hi, false, false)
                                    : __builtin_amdgcn_permlane16_swap(lo, hi, false, false);
            v[i] = __uint_as_float(r[0]) + __uint_as_float(r[1]);
        }
    } else if constexpr (M > 1) {
        const bool up = (threadIdx.x >> BIT) & 1;
#pragma unroll
        for (int i = 0; i < M / 2; ++i) {
            const float keep = up ? v[i + M / 2] : v[i], send = up ? v[i] : v[i + M / 2];
            v[i] = keep + partner<BIT>(send);
        }
    } else {
        v[0] += partner<BIT>(v[0]);
    }
}

// Sums M values over the CW channel lanes of a wave. What is left in v[0] (and on, where M is
// above CW: spread_left() values) are the sums of the values from spread_index() on.
template <int BIT, int M>
__device__ __forceinline__ void reduce_spread(float *v) {
    spread_step<BIT, M>(v);
    if constexpr (BIT > 0) reduce_spread<BIT - 1, (M > 1 ? M / 2 : 1)>(v);
}
constexpr int spread_left(int lanes, int m) { return m > lanes ? m / lanes : 1; }
template <int CW, int M>
__device__ __forceinline__ int spread_index(bool *writes) {
    int n = 0, m = M, free = 0;
    for (int bit = __builtin_ctz(CW) - 1; bit >= 0; --bit) {
        const int b = (threadIdx.x >> bit) & 1;
        if (m > 1) {        // lanes with the bit set keep the upper half
            m /= 2;
            n += b * m;
        } else {
            free |= b;
        }
    }
    *writes = free == 0;
    return n;
}

// Launch 1. See the head of the file; `chain` is the running product of decays. Only the sequence
// that enters the tile gives anything back, which is stored where that sequence's share ends, so
// that nothing of the next one can reach it. Also keeps the state
// before every eighth token of a sequence's share of the tile, and the sum of dt up to there. Such
// places are at least eight tokens apart, so token t's are kept at t / 8.
template <typename T, typename TG, int NS, int S>
__global__ __launch_bounds__(256, 2) void scan_bwd_tile_kernel(ScanArgs a) {
    using Lane = ScanLane<NS, S>;
    constexpr int NP = Lane::NP;
    __shared__ __align__(16) float s_bc[2][kB * 2 * NP];
    const Lane l(a, blockIdx.x);
    const int64_t tile = tile_index();
    if (tile * a.tile >= a.map.total && tile > 0) return;      // the whole workgroup
    const int t0 = static_cast<int>(tile * a.tile);
    const int t1 = a.map.total - t0 < a.tile ? a.map.total : t0 + a.tile;
    const uint32_t c = l.c;
    float A2[NS], h[NS], back[NS], chain[NS];
    load_rates(a, l, A2);
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f;
    float sum = 0.f;
    bool pass = false, entered = false;
#pragma unroll
    for (int n = 0; n < NS; ++n) { h[n] = 0.f; back[n] = 0.f; chain[n] = 1.f; }
    for_spans(a.map, t0, t1, [&](const Span &s) {
        if (s.starts) {
            if (a.S0) load_state(a, l, a.S0, s.i, h);
            else
#pragma unroll
                for (int n = 0; n < NS; ++n) h[n] = 0.f;
        }
        pass = !s.starts && !s.ends;
        Stage<T, NP, true> st;
        T xr[kB], dr[kB], gr[kB];
        TG yr[kB];
        auto fetch = [&](int t) {
            const int m = s.hi - t;
            st.take(a, l.g, t, m);
            fetch_rows(static_cast<const T *>(a.dt) + t * a.dt_stride, a.dt_stride, c, m, dr);
            fetch_rows(static_cast<const T *>(a.x) + t * a.x_stride, a.x_stride, c, m, xr);
            fetch_rows(static_cast<const TG *>(a.dO) + t * static_cast<int64_t>(a.channels), a.channels, c, m, yr);
            if (a.gate) fetch_rows(static_cast<const T *>(a.gate) + t * a.gate_stride, a.gate_stride, c, m, gr);
        };
        if (s.lo < s.hi) {
            fetch(s.lo);
            st.put(s_bc[0]);
            __syncthreads();
        }
        int buf = 0;
        for (int t = s.lo; t < s.hi; t += kB, buf ^= 1) {
            float x[kB], d[kB], dy[kB];
            widen(dr, d);
            widen(xr, x);
            widen(yr, dy);
            if (a.gate)
#pragma unroll
                for (int k = 0; k < kB; ++k) dy[k] *= silu(io<T>::val(gr[k]));
            const int m = s.hi - t;
            if (m > kB) fetch(t + kB);
            if (t > s.lo) {
                store_tile(a, l, a.kept_h, t / kG, h);
                if (l.on && l.part == 0) a.kept_dt[(t / kG) * static_cast<int64_t>(a.channels) + c] = sum;
            }
#pragma unroll
            for (int k = 0; k < kB; ++k) d[k] += bias;
            if (a.softplus) softplus_shared<S>(d);
            if (m < kB)         // steps of zero: h and chain stay, and nothing comes back
#pragma unroll
                for (int k = 1; k < kB; ++k)
                    if (k >= m) d[k] = x[k] = dy[k] = 0.f;
            const float *bc = s_bc[buf] + l.n0;
#pragma unroll
            for (int k = 0; k < kB; ++k) {
                float b[NS], cv[NS];
                lds_row<NS>(bc + k * 2 * NP, b);
                lds_row<NS>(bc + k * 2 * NP + NP, cv);
                const float u = d[k] * x[k];
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    const float decay = __builtin_amdgcn_exp2f(d[k] * A2[n]);
                    h[n] = fmaf(decay, h[n], u * b[n]);
                    chain[n] *= decay;
                    back[n] = fmaf(chain[n], cv[n] * dy[k], back[n]);
                }
                sum += d[k];
            }
            pin(h);
            pin(chain);
            pin(back);
            if (m > kB) st.put(s_bc[buf ^ 1]);
            __syncthreads();
        }
        if (!s.starts) {
            if (s.ends && a.dS_T) {
                float g[NS];
                load_state(a, l, a.dS_T, s.i, g);
#pragma unroll
                for (int n = 0; n < NS; ++n) back[n] = fmaf(chain[n], g[n], back[n]);
            }
            store_tile(a, l, a.tiles_g, tile, back);
            entered = true;
        }
    });
    store_tile(a, l, a.tiles_h, tile, h);
    if (!entered) {
#pragma unroll
        for (int n = 0; n < NS; ++n) back[n] = 0.f;
        store_tile(a, l, a.tiles_g, tile, back);
    }
    if (l.on && l.part == 0) a.tiles_dt[tile * a.channels + c] = sum;
    if (blockIdx.x == 0 && threadIdx.x == 0) a.tiles_pass[tile] = pass ? 1 : 0;
}

// Launch 2: the states from the front, the gradients from the back.
__global__ __launch_bounds__(256) void scan_bwd_chain_kernel(ScanArgs a, int tiles) {
    if (blockIdx.y == 0) chain_tiles<1>(a, a.tiles_h, tiles);
    else chain_tiles<-1>(a, a.tiles_g, tiles);
}

// Launch 3. As in the forward, a group of kG tokens has no branch between its tokens: the ones
// missing from a sequence's last group take steps of zero, with no input and no gradient.
template <typename T, typename TG, int NS, int S>
__global__ __launch_bounds__(256, 2) void scan_bwd_kernel(ScanArgs a) {
    using Lane = ScanLane<NS, S>;
    constexpr int NP = Lane::NP, CW = Lane::CW, TOP = __builtin_ctz(CW) - 1;
    constexpr int LEFT = spread_left(CW, NS);
    extern __shared__ __align__(16) float lds[];
    // B and C of the tile [groups * kG][2][NP]; the waves' dB and dC, for two groups in turn
    // [2][waves][kG][2][NP], and a place for what lanes without a result of their own write
    constexpr int RED = kG * 2 * NP;
    float *s_bc = lds, *s_red = s_bc + (a.tile + kG - 1) / kG * RED, *s_none = s_red + 2 * kScanWaves * RED;
    const Lane l(a, blockIdx.x);
    const int64_t tile = tile_index();
    if (tile * a.tile >= a.map.total && tile > 0) return;      // the whole workgroup
    const int t0 = static_cast<int>(tile * a.tile);
    const int t1 = a.map.total - t0 < a.tile ? a.map.total : t0 + a.tile;
    const uint32_t c = l.c;
    float A2[NS], dA[NS];
    load_rates(a, l, A2);
#pragma unroll
    for (int n = 0; n < NS; ++n) dA[n] = 0.f;
    const float bias = a.dt_bias ? a.dt_bias[c] : 0.f, skip = a.D ? a.D[c] : 0.f;
    float dD = 0.f, dbias = 0.f;
    bool writes;
    float *my_red = s_red + l.wave * RED + l.n0 + spread_index<CW, NS>(&writes);
    const int other = writes ? kScanWaves * RED : 0;
    if (!writes) my_red = s_none + (threadIdx.x & 63);
    int turn = 0;
    const bool gated = a.gate != nullptr;
    // the step sizes of a group, zero from m on and in lanes without a channel (which then add
    // nothing to the sums over channels)
    auto steps = [&](float (&d)[kG], int m) {
        if (a.softplus) softplus_shared<S>(d);
        if (m < kG)
#pragma unroll
            for (int k = 1; k < kG; ++k)
                if (k >= m) d[k] = 0.f;
        if (!l.on)
#pragma unroll
            for (int k = 0; k < kG; ++k) d[k] = 0.f;
    };
    for_spans(a.map, t0, t1, [&](const Span &s) {
        float g[NS];        // the gradient that comes to h_t from behind, a_{t+1} gh_{t+1}
        if (!s.ends) {
            load_tile(a, l, a.tiles_g, tile, g);
        } else if (a.dS_T) {
            load_state<false>(a, l, a.dS_T, s.i, g);
        } else {
#pragma unroll
            for (int n = 0; n < NS; ++n) g[n] = 0.f;
        }
        const int len = s.hi - s.lo, groups = (len + kG - 1) / kG;
        if (len > 0) {
            __syncthreads();       // the span before is done with s_bc
            for (int e = threadIdx.x; e < groups * kG * 2 * NP; e += 256) {
                const int k = e / (2 * NP), j = e % (2 * NP), n = j % NP;
                float v = 0.f;
                if (n < a.d_state && k < len) {
                    const bool is_c = j >= NP;
                    const T *p = static_cast<const T *>(is_c ? a.C : a.B);
                    v = io<T>::ld(p + (s.lo + k) * (is_c ? a.c_stride : a.b_stride) + l.g * a.d_state + n);
                }
                s_bc[e] = v;
            }
            __syncthreads();
        }
        // back, group by group
        for (int q = groups - 1; q >= 0; --q) {
            const int m = len - q * kG < kG ? len - q * kG : kG;
            const int64_t t = s.lo + q * kG;
            float x[kG], d[kG], raw[kG], gt[kG], go[kG], hist[kG][NS];
            T xr[kG], dr[kG], gr[kG];
            TG yr[kG];
            fetch_rows(static_cast<const T *>(a.dt) + t * a.dt_stride, a.dt_stride, c, m, dr);
            fetch_rows(static_cast<const T *>(a.x) + t * a.x_stride, a.x_stride, c, m, xr);
            fetch_rows(static_cast<const TG *>(a.dO) + t * a.channels, a.channels, c, m, yr);
            if (gated) fetch_rows(static_cast<const T *>(a.gate) + t * a.gate_stride, a.gate_stride, c, m, gr);
            widen(dr, d);
            widen(xr, x);
            widen(yr, go);
            if (gated) widen(gr, gt);
#pragma unroll
            for (int k = 0; k < kG; ++k) raw[k] = d[k] += bias;
            steps(d, m);
            if (m < kG || !l.on)
#pragma unroll
                for (int k = 0; k < kG; ++k)
                    if (k >= m || !l.on) x[k] = go[k] = 0.f;
            // the state entering the group: the one that enters the span, or what launch 1 kept
            // and, where that was reached from zero, what is left of the one that enters the tile
            float h[NS];
            if (!s.starts) {
                load_tile(a, l, a.tiles_h, tile, h);
            } else if (a.S0 && q == 0) {
                load_state<false>(a, l, a.S0, s.i, h);
            } else {
#pragma unroll
                for (int n = 0; n < NS; ++n) h[n] = 0.f;
            }
            if (q > 0) {
                float kept[NS];
                load_tile(a, l, a.kept_h, t / kG, kept);
                const float cum = s.starts ? 0.f : a.kept_dt[(t / kG) * a.channels + c];
#pragma unroll
                for (int n = 0; n < NS; ++n) h[n] = fmaf(__builtin_amdgcn_exp2f(A2[n] * cum), h[n], kept[n]);
            }
            const float *bc = s_bc + q * kG * 2 * NP + l.n0;
#pragma unroll
            for (int k = 0; k < kG; ++k) {
                const float u = d[k] * x[k];
                float b[NS];
                lds_row<NS>(bc + k * 2 * NP, b);
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    // kept: a_t h_{t-1}, from which h_t follows by one operation
                    hist[k][n] = __builtin_amdgcn_exp2f(d[k] * A2[n]) * h[n];
                    h[n] = fmaf(u, b[n], hist[k][n]);
                }
                pin(hist[k]);
            }
            float *red = my_red + turn * other;
            pin(d);        // the decays are formed again below: kept, they would take kG * NS registers
#pragma unroll
            for (int k = kG - 1; k >= 0; --k) {
                // what is kept of the group's tokens takes most registers, so the two products
                // that are summed over channels are formed one after the other
                const float u = d[k] * x[k];
                float sg = 1.f, dy = go[k];
                if (gated) {
                    sg = sigmoid_hw(gt[k]);
                    dy *= gt[k] * sg;
                }
                float y = 0.f, sB = 0.f, sA = 0.f;
                {
                    float b[NS], cv[NS], p[NS];
                    lds_row<NS>(bc + k * 2 * NP, b);
                    lds_row<NS>(bc + k * 2 * NP + NP, cv);
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        const float ht = fmaf(u, b[n], hist[k][n]);
                        y = fmaf(cv[n], ht, y);
                        p[n] = dy * ht;
                        g[n] = fmaf(cv[n], dy, g[n]);        // gh_t
                        sB = fmaf(g[n], b[n], sB);
                    }
                    reduce_spread<TOP, NS>(p);
#pragma unroll
                    for (int i = 0; i < LEFT; ++i) red[k * 2 * NP + NP + i] = p[i];
                }
                {
                    float p[NS];
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        p[n] = g[n] * u;
                        const float r = g[n] * hist[k][n];
                        sA = fmaf(r, A2[n], sA);
                        dA[n] = fmaf(r, d[k], dA[n]);
                        g[n] *= __builtin_amdgcn_exp2f(d[k] * A2[n]);
                    }
                    reduce_spread<TOP, NS>(p);
#pragma unroll
                    for (int i = 0; i < LEFT; ++i) red[k * 2 * NP + i] = p[i];
                }
                sB = sum_parts<S>(sB);
                float dd = fmaf(x[k], sB, sum_parts<S>(sA) * (1.f / kLog2e));
                if (a.softplus) {       // a masked step, of no slope, takes none of a product beyond fp32
                    const float slope = sigmoid_hw(raw[k]);
                    dd = slope == 0.f ? 0.f : dd * slope;
                }
                dD = fmaf(dy, x[k], dD);
                dbias += k < m ? dd : 0.f;
                if (gated) {        // dgate, dx and ddt take the places of gate, dO and raw
                    y = fmaf(skip, x[k], sum_parts<S>(y));
                    gt[k] = go[k] * y * (sg * fmaf(gt[k], 1.f - sg, 1.f));
                }
                go[k] = fmaf(skip, dy, d[k] * sB);
                raw[k] = dd;
                float out[5] = {go[k], raw[k], gated ? gt[k] : 0.f, dD, dbias};
                pin(out);
                go[k] = out[0];
                raw[k] = out[1];
                gt[k] = out[2];
                dD = out[3];
                dbias = out[4];
                pin(g);
                pin(dA);
            }
            if (l.on && l.part == 0) {
                TG *px = static_cast<TG *>(a.dx) + t * a.channels, *pd = static_cast<TG *>(a.ddt) + t * a.channels;
#pragma unroll
                for (int k = 0; k < kG; ++k) {
                    if (k < m) {
                        io<TG>::st(elem(px, c), go[k]);
                        io<TG>::st(elem(pd, c), raw[k]);
                    }
                    px += a.channels;
                    pd += a.channels;
                }
                if (gated) {
                    TG *pg = static_cast<TG *>(a.dgate) + t * a.channels;
#pragma unroll
                    for (int k = 0; k < kG; ++k) {
                        if (k < m) io<TG>::st(elem(pg, c), gt[k]);
                        pg += a.channels;
                    }
                }
            }
            __syncthreads();
            // the waves' shares of dB and dC, added in their order
            for (int e = threadIdx.x; e < m * 2 * NP; e += 256) {
                const int k = e / (2 * NP), j = e % (2 * NP), n = j % NP;
                if (n >= a.d_state) continue;
                float v = 0.f;
#pragma unroll
                for (int w = 0; w < kScanWaves; ++w) v += s_red[(turn * kScanWaves + w) * RED + e];
                a.part_bc[((static_cast<int64_t>(blockIdx.x) * a.map.total + t + k) * 2 + (j >= NP)) * a.d_state + n] = v;
            }
            turn ^= 1;
        }
        if (s.starts && a.dS0) store_state(a, l, a.dS0, s.i, g);
    });
    // the tile's sums for dA, dD and ddt_bias, where its state and sum of dt were
    store_tile(a, l, a.tiles_h, tile, dA);
    if (l.on && l.part == 0) {
        a.tiles_dt[tile * a.channels + c] = dD;
        a.tiles_db[tile * a.channels + c] = dbias;
    }
}

// Over the tiles: a column per lane, four waves taking every fourth tile. Columns: d_state *
// channels of dA, then channels of dD, then channels of ddt_bias.
__device__ __forceinline__ void sum_tiles(const ScanArgs &a, int tiles) {
    __shared__ float s[4][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t cols = static_cast<int64_t>(a.d_state) * a.channels;
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
    const float *p = nullptr;
    int64_t step = a.channels;
    if (col < cols) { p = a.tiles_h + col; step = cols; }
    else if (col < cols + a.channels) p = a.dD ? a.tiles_dt + (col - cols) : nullptr;
    else if (col < cols + 2 * a.channels) p = a.ddt_bias ? a.tiles_db + (col - cols - a.channels) : nullptr;
    float sum = 0.f;
    if (p)
#pragma unroll 8
        for (int i = wave; i < tiles; i += 4) sum += p[i * step];
    s[wave][lane] = sum;
    __syncthreads();
    if (wave != 0 || !p) return;
    sum += s[1][lane] + s[2][lane] + s[3][lane];
    if (col < cols) {
        const int n = static_cast<int>(col / a.channels);
        a.dA[(col - static_cast<int64_t>(n) * a.channels) * a.d_state + n] = sum;
    } else if (col < cols + a.channels) {
        a.dD[col - cols] = sum;
    } else {
        a.ddt_bias[col - cols - a.channels] = sum;
    }
}

// Over the workgroups of a group's channels: dB and dC, one value per thread. Tokens behind the
// last sequence are left as they were. This is workgroup `wg` of `wgs`.
template <typename TG>
__device__ __forceinline__ void sum_blocks(const ScanArgs &a, int blocks, int wg, int wgs) {
    const int end = seq_begin(a.map, a.map.n);
    const int64_t row = 2 * static_cast<int64_t>(a.d_state), n = a.groups * row * end;
    for (int64_t e = wg * static_cast<int64_t>(256) + threadIdx.x; e < n;
         e += static_cast<int64_t>(wgs) * 256) {
        const int64_t tg = e / row;
        const int j = static_cast<int>(e - tg * row);
        const int64_t t = tg / a.groups;
        const int g = static_cast<int>(tg - t * a.groups);
        float v = 0.f;
        for (int b = 0; b < blocks; ++b)
            v += a.part_bc[(static_cast<int64_t>(g * blocks + b) * a.map.total + t) * row + j];
        TG *out = static_cast<TG *>(j < a.d_state ? a.dB : a.dC);
        io<TG>::st(out + tg * a.d_state + (j < a.d_state ? j : j - a.d_state), v);
    }
}

// Launch 4: the first `first` workgroups add over the tiles, the others over workgroups. (One
// launch: as two they took 4.6 and 4.4 us behind each other, mostly latency.)
template <typename TG>
__global__ __launch_bounds__(256) void scan_bwd_sums_kernel(ScanArgs a, int tiles, int blocks, int first) {
    const int wg = blockIdx.x;
    if (wg < first) sum_tiles(a, tiles);
    else sum_blocks<TG>(a, blocks, wg - first, static_cast<int>(gridDim.x) - first);
}

template <typename T, typename TG, int NS, int S>
hipError_t launch_bwd(const ScanArgs &a, hipStream_t st) {
    const int tiles = scan_tiles(a.map.total, a.tile), blocks = scan_blocks(a.channels, a.groups, S);
    const dim3 grid = scan_grid(blocks, tiles);
    const int64_t cols = static_cast<int64_t>(a.d_state) * a.channels;
    if (a.chained || a.tile > kG) {
        // sixteen states per lane where two waves per SIMD are left (a channel's step and gate are
        // then formed by half the lanes: 62.4 against 70.7 us on 4,096 tokens x 2,048 channels x 16
        // states; with one wave 34.5 against 28.8 us, 1,011 x 1,002 x 24). Above 16 states the instance
        // spills 84-116 bytes per lane and is the faster all the same: whole calls of 16, 24, 32, 64 and 128
        // states, bf16 and fp32, 512 to 4,096 channels, take 1.6 to 4 % more without it.
        constexpr int N1 = S > 1 ? 2 * NS : NS, S1 = S > 1 ? S / 2 : 1;
        const int wide = scan_blocks(a.channels, a.groups, S1);
        if (static_cast<int64_t>(wide) * tiles * kScanWaves >= 2 * kSimds)
            hipLaunchKernelGGL((scan_bwd_tile_kernel<T, TG, N1, S1>), scan_grid(wide, tiles), dim3(256), 0, st, a);
        else
            hipLaunchKernelGGL((scan_bwd_tile_kernel<T, TG, NS, S>), grid, dim3(256), 0, st, a);
    }
    if (a.chained) {
        hipLaunchKernelGGL(scan_bwd_chain_kernel, dim3(static_cast<unsigned>((cols + 255) / 256), 2),
                           dim3(256), 0, st, a, tiles);
    }
    constexpr int RED = kG * 2 * NS * S, FIXED = (2 * kScanWaves + 1) * RED + 64;
    const size_t lds = sizeof(float) * (static_cast<size_t>((a.tile + kG - 1) / kG) * RED + FIXED);
    static_assert(kB == kG, "what launch 1 keeps at its batches is what launch 3 reads at its groups");
    static_assert(sizeof(float) * (kScanMaxBwdTile / kG * RED + FIXED) <= 160 * 1024, "a tile fits the LDS");
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(scan_bwd_kernel<T, TG, NS, S>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(lds));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((scan_bwd_kernel<T, TG, NS, S>), grid, dim3(256), lds, st, a);
    const int64_t all = cols + 2 * static_cast<int64_t>(a.channels);
    const int64_t n = 2 * static_cast<int64_t>(a.d_state) * a.groups * a.map.total;
    const int first = static_cast<int>((all + 63) / 64), rest = static_cast<int>((n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096);
    hipLaunchKernelGGL(scan_bwd_sums_kernel<TG>, dim3(static_cast<unsigned>(first + rest)), dim3(256), 0, st, a,
                       tiles, blocks / a.groups, first);
    return hipGetLastError();
}

template <typename T, typename TG>
hipError_t launch_bwd_t(const ScanArgs &a, hipStream_t st) {
    switch (scan_bwd_parts(a.d_state)) {
    case 1: return launch_bwd<T, TG, 8, 1>(a, st);
    case 2: return launch_bwd<T, TG, 8, 2>(a, st);
    case 4: return launch_bwd<T, TG, 8, 4>(a, st);
    case 8: return launch_bwd<T, TG, 8, 8>(a, st);
    default: return launch_bwd<T, TG, 8, 16>(a, st);
    }
}

}  // namespace

// Eight states per lane: a group's kept states are 64 registers, so that two waves fit a SIMD, with
// 28-44 bytes per lane spilled (none up to 8 states). Sixteen, as in the forward, need 350: on 4,096 tokens x 2,048 channels x 16
// states 209.6 us at one wave per SIMD against 197.6 us, although a channel's step, gate and
// loads are then done by twice the lanes.
int scan_bwd_parts(int d_state) {
    return d_state <= 8 ? 1 : d_state <= 16 ? 2 : d_state <= 32 ? 4 : d_state <= 64 ? 8 : 16;
}

// Tokens per tile: about two waves per SIMD, between 8 tokens (16 where that would be more than 64
// tiles to chain) and what LDS holds; whole sequences where they are no longer than that. Few waves
// take 10 us per eight tokens, so short sequences are cut too: 64 tokens x 768 channels x 16 states
// 31 us in 8 tiles against 87 us whole, 16 x 64 tokens 66 against 92 us; 64 x 16 tokens x 256
// channels 35 us whole against 46 us in halves.
int scan_bwd_tile(int channels, int groups, int d_state, int batch, int seqlen, bool packed) {
    const int64_t total = static_cast<int64_t>(batch) * seqlen;
    const int64_t waves = static_cast<int64_t>(kScanWaves) * scan_blocks(channels, groups, scan_bwd_parts(d_state));
    const int64_t t = (total * waves / (2 * kSimds) + kG - 1) / kG * kG;
    const int least = total <= 64 * kG ? kG : 2 * kG;
    const int tile = t < least ? least : t > kScanMaxBwdTile ? kScanMaxBwdTile : static_cast<int>(t);
    return !packed && seqlen <= tile ? (seqlen > 0 ? seqlen : 1) : tile;
}

hipError_t launch_scan_bwd(const ScanArgs &a, hipStream_t st) {
    if (!a.bf16) return launch_bwd_t<float, float>(a, st);
    return a.grad_bf16 ? launch_bwd_t<bf16_t, bf16_t>(a, st) : launch_bwd_t<bf16_t, float>(a, st);
}

}  // namespace gdn2
