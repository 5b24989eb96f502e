// gdn2_scan_bwd.hip -- gradients of the selective scan.
//
// With dy = dO silu(gate), a_t = exp(dt_t A), and gh_t the gradient of the state h_t:
//     gh_t   = C_t dy_t + a_{t+1} gh_{t+1}          (dS_T after a sequence's last token)
//     dC_t   = sum_d dy h_t,                        dB_t = sum_d gh_t dt_t x_t
//     dx_t   = D dy + dt_t sum_n gh_t B_t,          dD = sum_t dy x
//     ddt_t  = x_t sum_n gh_t B_t + sum_n gh_t a_t h_{t-1} A,   through softplus' for the input
//     dA     = sum_t gh_t a_t h_{t-1} dt_t,         dS0 = a_0 gh_0,   dgate = dO y silu'(gate)
// Nothing but the inputs is kept from the forward. Four launches:
//   1. per tile of tokens: the state it reaches from zero, its sum of dt, and what its outputs
//      alone give back to the state that enters it (sum_t prod_{s<=t} a_s C_t dy_t);
//   2. both chained over the tiles, one from the front, one from the back;
//   3. per tile: the states forward once, every eighth into LDS; then back over groups of eight
//      tokens: their states again into registers, and the gradients from the last to the first;
//   4. the sums over tiles (dA, dD, ddt_bias) and over workgroups of channels (dB, dC).
// Every sum has a fixed order: the same bits at every call.
//
// dB and dC sum over channels, which lie across the lanes. A wave reduces and spreads at once:
// each step sends half of a lane's values to the partner lane and adds the other half, so 16
// values over 64 lanes cost about 35 operations instead of 96 (reduce_spread).
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

// Launch 1. See the head of the file; `chain` is the running product of decays.
template <typename T, typename TG, int NS, int S>
__global__ __launch_bounds__(256) void scan_bwd_tile_kernel(ScanArgs a) {
    using Lane = ScanLane<NS, S>;
    constexpr int NP = Lane::NP;
    __shared__ __align__(16) float s_bc[2][kB * 2 * NP];
    const Lane l(a, blockIdx.x);
    const int64_t tile = tile_index();
    if (tile * a.tile >= a.map.total && tile > 0) return;      // the whole workgroup
    const int t0 = static_cast<int>(tile * a.tile);
    const int t1 = a.map.total - t0 < a.tile ? a.map.total : t0 + a.tile;
    const T *x = static_cast<const T *>(a.x) + l.c, *dt = static_cast<const T *>(a.dt) + l.c;
    const T *gate = a.gate ? static_cast<const T *>(a.gate) + l.c : nullptr;
    const TG *dO = static_cast<const TG *>(a.dO) + l.c;
    float A2[NS], h[NS], back[NS], chain[NS];
    load_rates(a, l, A2);
    const float bias = a.dt_bias ? a.dt_bias[l.c] : 0.f;
    float sum = 0.f;
    bool pass = false;
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
        if (s.lo < s.hi) {
            Stage<T, NP, true> st;
            T xr[kB], dr[kB], gr[kB];
            TG yr[kB];
            auto fetch = [&](int t) {
                st.take(a, l.g, t, s.hi);
#pragma unroll
                for (int k = 0; k < kB; ++k)
                    if (t + k < s.hi) {
                        xr[k] = x[(t + k) * a.x_stride];
                        dr[k] = dt[(t + k) * a.dt_stride];
                        yr[k] = dO[(t + k) * static_cast<int64_t>(a.channels)];
                        if (gate) gr[k] = gate[(t + k) * a.gate_stride];
                    }
            };
            fetch(s.lo);
            st.put(s_bc[0]);
            __syncthreads();
            int buf = 0;
            for (int t = s.lo; t < s.hi; t += kB, buf ^= 1) {
                float xv[kB], dv[kB], yv[kB];
#pragma unroll
                for (int k = 0; k < kB; ++k) {
                    xv[k] = io<T>::val(xr[k]);
                    dv[k] = io<T>::val(dr[k]);
                    yv[k] = io<TG>::val(yr[k]);
                    if (gate) yv[k] *= silu(io<T>::val(gr[k]));
                }
                const bool more = t + kB < s.hi;
                if (more) fetch(t + kB);
                const int m = s.hi - t;
#pragma unroll
                for (int k = 0; k < kB; ++k) {
                    if (k >= m) break;
                    float d = dv[k] + bias;
                    if (a.softplus) d = softplus(d);
                    const float u = d * xv[k];
                    const float *row = s_bc[buf] + k * 2 * NP + l.n0;
                    float b[NS];
                    lds_row<NS>(row, b);
                    if (!s.starts) {
                        float c[NS];
                        lds_row<NS>(row + NP, c);
#pragma unroll
                        for (int n = 0; n < NS; ++n) {
                            const float decay = __builtin_amdgcn_exp2f(d * A2[n]);
                            h[n] = fmaf(decay, h[n], u * b[n]);
                            chain[n] *= decay;
                            back[n] = fmaf(chain[n], c[n] * yv[k], back[n]);
                        }
                    } else {
#pragma unroll
                        for (int n = 0; n < NS; ++n)
                            h[n] = fmaf(__builtin_amdgcn_exp2f(d * A2[n]), h[n], u * b[n]);
                    }
                    sum += d;
                }
                if (more) st.put(s_bc[buf ^ 1]);
                __syncthreads();
            }
        }
        if (!s.starts && s.ends && a.dS_T) {
            float g[NS];
            load_state(a, l, a.dS_T, s.i, g);
#pragma unroll
            for (int n = 0; n < NS; ++n) back[n] = fmaf(chain[n], g[n], back[n]);
        }
    });
    store_tile(a, l, a.tiles_h, tile, h);
    store_tile(a, l, a.tiles_g, tile, back);
    if (l.on && l.part == 0) a.tiles_dt[tile * a.channels + l.c] = sum;
    if (blockIdx.x == 0 && threadIdx.x == 0) a.tiles_pass[tile] = pass ? 1 : 0;
}

// Launch 2: the states from the front, the gradients from the back.
__global__ __launch_bounds__(256) void scan_bwd_chain_kernel(ScanArgs a, int tiles) {
    if (blockIdx.y == 0) chain_tiles<1>(a, a.tiles_h, tiles);
    else chain_tiles<-1>(a, a.tiles_g, tiles);
}

// Launch 3.
template <typename T, typename TG, int NS, int S>
__global__ __launch_bounds__(256) void scan_bwd_kernel(ScanArgs a) {
    using Lane = ScanLane<NS, S>;
    constexpr int NP = Lane::NP, CW = Lane::CW, TOP = CW == 64 ? 5 : CW == 32 ? 4 : CW == 16 ? 3 : 2;
    extern __shared__ __align__(16) float lds[];
    // B and C of the tile [tile][2][NP]; states every kG tokens [waves][groups][NS][64];
    // the waves' dB and dC [waves][kG][2][NP]
    float *s_bc = lds, *s_h = s_bc + a.tile * 2 * NP;
    const int tile_groups = (a.tile + kG - 1) / kG;
    float *s_red = s_h + kScanWaves * tile_groups * NS * 64;
    const Lane l(a, blockIdx.x);
    const int lane = threadIdx.x & 63;
    const int64_t tile = tile_index();
    if (tile * a.tile >= a.map.total && tile > 0) return;      // the whole workgroup
    const int t0 = static_cast<int>(tile * a.tile);
    const int t1 = a.map.total - t0 < a.tile ? a.map.total : t0 + a.tile;
    const T *x = static_cast<const T *>(a.x) + l.c, *dt = static_cast<const T *>(a.dt) + l.c;
    const T *gate = a.gate ? static_cast<const T *>(a.gate) + l.c : nullptr;
    const TG *dO = static_cast<const TG *>(a.dO) + l.c;
    TG *dx = static_cast<TG *>(a.dx) + l.c, *ddt = static_cast<TG *>(a.ddt) + l.c;
    TG *dgate = a.gate ? static_cast<TG *>(a.dgate) + l.c : nullptr;
    float *my_h = s_h + l.wave * tile_groups * NS * 64 + lane;
    float *my_red = s_red + l.wave * kG * 2 * NP;
    float A2[NS], dA[NS];
    load_rates(a, l, A2);
#pragma unroll
    for (int n = 0; n < NS; ++n) dA[n] = 0.f;
    const float bias = a.dt_bias ? a.dt_bias[l.c] : 0.f, skip = a.D ? a.D[l.c] : 0.f;
    float dD = 0.f, dbias = 0.f;
    bool writes;
    const int red_n = l.n0 + spread_index<CW, NS>(&writes);
    // inputs of a token; zero in lanes without a channel, so that they add nothing to any sum
    auto in = [&](const T *p, int64_t at) { return l.on ? io<T>::ld(p + at) : 0.f; };
    auto step = [&](float raw) { return a.softplus ? softplus(raw) : raw; };
    for_spans(a.map, t0, t1, [&](const Span &s) {
        float h[NS], g[NS];        // g: the gradient that comes to h_t from behind, a_{t+1} gh_{t+1}
        if (s.ends) {
            if (a.dS_T) load_state(a, l, a.dS_T, s.i, g);
            else
#pragma unroll
                for (int n = 0; n < NS; ++n) g[n] = 0.f;
        } else {
            load_tile(a, l, a.tiles_g, tile, g);
        }
        if (s.starts) {
            if (a.S0) load_state(a, l, a.S0, s.i, h);
            else
#pragma unroll
                for (int n = 0; n < NS; ++n) h[n] = 0.f;
        } else {
            load_tile(a, l, a.tiles_h, tile, h);
        }
        const int len = s.hi - s.lo;
        if (len > 0) {
            __syncthreads();       // the span before is done with s_bc
            for (int e = threadIdx.x; e < len * 2 * NP; e += 256) {
                const int k = e / (2 * NP), j = e % (2 * NP), n = j % NP;
                float v = 0.f;
                if (n < a.d_state) {
                    const bool c = j >= NP;
                    const T *p = static_cast<const T *>(c ? a.C : a.B);
                    v = io<T>::ld(p + (s.lo + k) * (c ? a.c_stride : a.b_stride) + l.g * a.d_state + n);
                }
                s_bc[e] = v;
            }
            __syncthreads();
            const int groups = (len + kG - 1) / kG;
            // forward: the state entering every group of kG tokens
            for (int q = 0; q < groups; ++q) {
#pragma unroll
                for (int n = 0; n < NS; ++n) my_h[(q * NS + n) * 64] = h[n];
                if (q == groups - 1) break;
                float xv[kG], dv[kG];
#pragma unroll
                for (int k = 0; k < kG; ++k) {
                    const int64_t t = s.lo + q * kG + k;
                    xv[k] = in(x, t * a.x_stride);
                    dv[k] = in(dt, t * a.dt_stride);
                }
#pragma unroll
                for (int k = 0; k < kG; ++k) {
                    const float d = l.on ? step(dv[k] + bias) : 0.f, u = d * xv[k];
                    float b[NS];
                    lds_row<NS>(s_bc + (q * kG + k) * 2 * NP + l.n0, b);
#pragma unroll
                    for (int n = 0; n < NS; ++n)
                        h[n] = fmaf(__builtin_amdgcn_exp2f(d * A2[n]), h[n], u * b[n]);
                }
            }
            // back, group by group
            for (int q = groups - 1; q >= 0; --q) {
                const int m = len - q * kG < kG ? len - q * kG : kG;
                float xv[kG], dv[kG], rv[kG], gv[kG], yv[kG], hist[kG][NS];
#pragma unroll
                for (int k = 0; k < kG; ++k) {
                    xv[k] = dv[k] = gv[k] = yv[k] = 0.f;
                    if (k < m) {
                        const int64_t t = s.lo + q * kG + k;
                        xv[k] = in(x, t * a.x_stride);
                        dv[k] = in(dt, t * a.dt_stride);
                        if (l.on) yv[k] = io<TG>::ld(dO + t * a.channels);
                        if (gate) gv[k] = in(gate, t * a.gate_stride);
                    }
                }
#pragma unroll
                for (int n = 0; n < NS; ++n) h[n] = my_h[(q * NS + n) * 64];
#pragma unroll
                for (int k = 0; k < kG; ++k) {
                    rv[k] = dv[k] + bias;
                    dv[k] = l.on ? step(rv[k]) : 0.f;
                    if (k >= m) break;
                    const float u = dv[k] * xv[k];
                    const float *row = s_bc + (q * kG + k) * 2 * NP + l.n0;
                    float b[NS];
                    lds_row<NS>(row, b);
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        // kept: a_t h_{t-1}, from which h_t follows by one operation
                        hist[k][n] = __builtin_amdgcn_exp2f(dv[k] * A2[n]) * h[n];
                        h[n] = fmaf(u, b[n], hist[k][n]);
                    }
                }
                __syncthreads();       // the group behind is done with s_red
#pragma unroll
                for (int k = kG - 1; k >= 0; --k) {
                    if (k >= m) continue;
                    const int64_t t = s.lo + q * kG + k;
                    const float d = dv[k], u = d * xv[k];
                    const float *row = s_bc + (q * kG + k) * 2 * NP + l.n0;
                    float b[NS], c[NS];
                    lds_row<NS>(row, b);
                    lds_row<NS>(row + NP, c);
                    const float sg = gate ? sigmoid_hw(gv[k]) : 1.f;
                    const float dy = gate ? yv[k] * (gv[k] * sg) : yv[k];
                    float y = 0.f, sB = 0.f, sA = 0.f, pb[NS], pc[NS];
#pragma unroll
                    for (int n = 0; n < NS; ++n) {
                        const float ah = hist[k][n], ht = fmaf(u, b[n], ah);
                        y = fmaf(c[n], ht, y);
                        pc[n] = dy * ht;
                        const float gh = fmaf(c[n], dy, g[n]);
                        pb[n] = gh * u;
                        sB = fmaf(gh, b[n], sB);
                        const float r = gh * ah;
                        sA = fmaf(r, A2[n], sA);
                        dA[n] = fmaf(r, d, dA[n]);
                        g[n] = __builtin_amdgcn_exp2f(d * A2[n]) * gh;
                    }
                    reduce_spread<TOP, NS>(pb);
                    reduce_spread<TOP, NS>(pc);
                    if (writes)
#pragma unroll
                        for (int i = 0; i < spread_left(CW, NS); ++i) {
                            my_red[k * 2 * NP + red_n + i] = pb[i];
                            my_red[k * 2 * NP + NP + red_n + i] = pc[i];
                        }
                    sB = sum_parts<S>(sB);
                    sA = sum_parts<S>(sA);
                    if (gate) {
                        y = fmaf(skip, xv[k], sum_parts<S>(y));
                        if (l.on && l.part == 0)
                            io<TG>::st(dgate + t * a.channels,
                                       yv[k] * y * (sg * fmaf(gv[k], 1.f - sg, 1.f)));
                    }
                    float dd = fmaf(xv[k], sB, sA * (1.f / kLog2e));
                    if (a.softplus) dd *= sigmoid_hw(rv[k]);
                    dD = fmaf(dy, xv[k], dD);
                    dbias += dd;
                    if (l.on && l.part == 0) {
                        io<TG>::st(dx + t * a.channels, fmaf(skip, dy, d * sB));
                        io<TG>::st(ddt + t * a.channels, dd);
                    }
                }
                __syncthreads();
                // the waves' shares of dB and dC, added in their order
                for (int e = threadIdx.x; e < m * 2 * NP; e += 256) {
                    const int k = e / (2 * NP), j = e % (2 * NP), n = j % NP;
                    if (n >= a.d_state) continue;
                    float v = 0.f;
#pragma unroll
                    for (int w = 0; w < kScanWaves; ++w) v += s_red[w * kG * 2 * NP + e];
                    const int64_t t = s.lo + q * kG + k;
                    a.part_bc[((static_cast<int64_t>(blockIdx.x) * a.map.total + t) * 2 + (j >= NP)) * a.d_state + n] = v;
                }
            }
        }
        if (s.starts && a.dS0) store_state(a, l, a.dS0, s.i, g);
    });
    // the tile's sums for dA, dD and ddt_bias, where its state and sum of dt were
    store_tile(a, l, a.tiles_h, tile, dA);
    if (l.on && l.part == 0) {
        a.tiles_dt[tile * a.channels + l.c] = dD;
        a.tiles_db[tile * a.channels + l.c] = dbias;
    }
}

// Launch 4, over the tiles: a column per lane, four waves taking every fourth tile.
// Columns: d_state * channels of dA, then channels of dD, then channels of ddt_bias.
__global__ __launch_bounds__(256) void scan_bwd_params_kernel(ScanArgs a, int tiles) {
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

// Launch 4, over the workgroups of a group's channels: dB and dC, one value per thread. Tokens
// behind the last sequence are left as they were.
template <typename TG>
__global__ __launch_bounds__(256) void scan_bwd_bc_kernel(ScanArgs a, int blocks) {
    const int end = seq_begin(a.map, a.map.n);
    const int64_t row = 2 * static_cast<int64_t>(a.d_state), n = a.groups * row * end;
    for (int64_t e = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x; e < n;
         e += static_cast<int64_t>(gridDim.x) * 256) {
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

template <typename T, typename TG, int NS, int S>
hipError_t launch_bwd(const ScanArgs &a, hipStream_t st) {
    const int tiles = scan_tiles(a.map.total, a.tile), blocks = scan_blocks(a.channels, a.groups, S);
    const dim3 grid = scan_grid(blocks, tiles);
    const int64_t cols = static_cast<int64_t>(a.d_state) * a.channels;
    if (a.chained) {
        hipLaunchKernelGGL((scan_bwd_tile_kernel<T, TG, NS, S>), grid, dim3(256), 0, st, a);
        hipLaunchKernelGGL(scan_bwd_chain_kernel, dim3(static_cast<unsigned>((cols + 255) / 256), 2),
                           dim3(256), 0, st, a, tiles);
    }
    const size_t lds = sizeof(float) * (static_cast<size_t>(a.tile) * 2 * NS * S +
                                        kScanWaves * ((a.tile + kG - 1) / kG) * NS * 64 +
                                        kScanWaves * kG * 2 * NS * S);
    static_assert(kScanMaxBwdTile % kG == 0, "whole groups of tokens in a tile");
    static_assert(sizeof(float) * (kScanMaxBwdTile * 2 * NS * S + kScanWaves * (kScanMaxBwdTile / kG) * NS * 64 +
                                   kScanWaves * kG * 2 * NS * S) <= 160 * 1024, "a tile fits the LDS");
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(scan_bwd_kernel<T, TG, NS, S>),
                                             hipFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(lds));
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL((scan_bwd_kernel<T, TG, NS, S>), grid, dim3(256), lds, st, a);
    const int64_t all = cols + 2 * static_cast<int64_t>(a.channels);
    hipLaunchKernelGGL(scan_bwd_params_kernel, dim3(static_cast<unsigned>((all + 63) / 64)), dim3(256), 0, st,
                       a, tiles);
    const int64_t n = 2 * static_cast<int64_t>(a.d_state) * a.groups * a.map.total;
    if (n > 0) {
        const int64_t wg = (n + 255) / 256;
        hipLaunchKernelGGL(scan_bwd_bc_kernel<TG>, dim3(static_cast<unsigned>(wg < 4096 ? wg : 4096)),
                           dim3(256), 0, st, a, blocks / a.groups);
    }
    return hipGetLastError();
}

template <typename T, typename TG>
hipError_t launch_bwd_t(const ScanArgs &a, hipStream_t st) {
    switch (scan_parts(a.d_state)) {
    case 1: return a.d_state <= 8 ? launch_bwd<T, TG, 8, 1>(a, st) : launch_bwd<T, TG, 16, 1>(a, st);
    case 2: return launch_bwd<T, TG, 16, 2>(a, st);
    case 4: return launch_bwd<T, TG, 16, 4>(a, st);
    default: return launch_bwd<T, TG, 16, 8>(a, st);
    }
}

}  // namespace

// Tokens per tile: whole sequences where they are short enough, else about 2,048 waves, between
// 8 tokens and what LDS holds.
int scan_bwd_tile(int channels, int groups, int d_state, int batch, int seqlen, bool packed) {
    if (!packed && seqlen <= kScanMaxBwdTile) return seqlen > 0 ? seqlen : 1;
    const int64_t total = static_cast<int64_t>(batch) * seqlen;
    const int64_t waves = static_cast<int64_t>(kScanWaves) * scan_blocks(channels, groups, scan_parts(d_state));
    const int64_t t = (total * waves / 2048 + kG - 1) / kG * kG;
    return t < kG ? kG : t > kScanMaxBwdTile ? kScanMaxBwdTile : static_cast<int>(t);
}

hipError_t launch_scan_bwd(const ScanArgs &a, hipStream_t st) {
    if (!a.bf16) return launch_bwd_t<float, float>(a, st);
    return a.grad_bf16 ? launch_bwd_t<bf16_t, bf16_t>(a, st) : launch_bwd_t<bf16_t, float>(a, st);
}

}  // namespace gdn2
