// gdn2_conv.hip -- the short causal depthwise convolution over prompts, its gradients, and its
// form for single tokens against a pool of conv states.
//
// Per channel c, with W taps (2, 3 or 4) and x before the sequence taken from the conv state:
//     a_t = bias + sum_{j < W} w_j x_{t - W + 1 + j},        y_t = silu(a_t) or a_t.
// Gradients, with e_t = dy_t act'(a_t) (a_t formed again from x) and e = 0 outside the sequence:
//     dx_t = sum_j w_j e_{t + W - 1 - j},   dw_j = sum_t e_t x_{t - W + 1 + j},   dbias = sum_t e_t.
// The same sum at the W - 1 positions before the sequence is the gradient of the conv state.
//
// All three are bound by memory: 2 W operations per element against 2 or 3 element accesses. A
// lane owns V neighbouring channels (4 forward, where 8 left too few waves: 28 against 22 us on
// 4,096 tokens x 6,144 bf16 channels; 2 backward, where 4 take 200 registers and two waves per
// SIMD hide neither memory nor arithmetic: 52 against 39 us) and walks a tile of tokens with the last
// W - 1 inputs (and, backward, the last W values of e) in registers, so every element is read
// from memory once; only the W - 1 rows next to a tile are read again by its neighbour. Tiles cut
// the token axis without regard to sequences: a wave walks the sequences inside its tile, so the
// work per wave does not depend on how a packed batch is cut.
//
// Measured: prompt of 4,096 x 6,144 bf16 22 us (101 MB, 4.6 TB/s; a large copy reaches 5.1), its
// gradients 41 us (151 MB, 3.7 TB/s: the vector unit is as busy as memory), 64 single tokens x
// 10,240 channels 5.7 us of GPU time (18.5 MB).
#include <type_traits>

#include "gdn2_internal.h"
#include "gdn2_layer.h"

namespace gdn2 {

namespace {

constexpr int kBatch = 4;    // rows whose loads are in flight together

// The W - 1 inputs before token t of a span, oldest first.
template <typename T, int W, int V>
__device__ __forceinline__ void load_history(const ConvArgs &a, const T *x, const Span &s, int t,
                                             uint32_t c, float (&h)[W - 1][V]) {
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
        const int at = t - (W - 1) + r;
        if (at >= s.first) {
            ldv<T, V>(x + at * a.x_stride + c, h[r]);
        } else if (a.state0) {
            const int64_t row = static_cast<int64_t>(s.i) * (W - 1) + (at - s.first + W - 1);
            ldv<float, V>(a.state0 + row * a.channels + c, h[r]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) h[r][v] = 0.f;
        }
    }
}

// The taps ([C][W], so a lane's are V * W consecutive floats) and biases of V channels.
template <int W, int V>
__device__ __forceinline__ void load_taps(const float *weight, const float *bias, int c,
                                          float (&w)[W][V], float (&b)[V]) {
    float flat[V * W];
    const float *p = weight + static_cast<int64_t>(c) * W;
    if constexpr (V == 1) {
#pragma unroll
        for (int j = 0; j < W; ++j) flat[j] = p[j];
    } else {
        ldv<float, V * W>(p, flat);
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][v] = flat[v * W + j];
        b[v] = 0.f;
    }
    if (bias) ldv<float, V>(bias + c, b);
}

template <typename T, int W, int V, bool SILU>
__global__ __launch_bounds__(256) void conv_fwd_kernel(ConvArgs a) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t t0l = (static_cast<int64_t>(blockIdx.y) * 4 + wave) * a.tile;
    if (t0l >= a.map.total && t0l > 0) return;
    const int t0 = static_cast<int>(t0l);
    const int t1 = a.map.total - t0 < a.tile ? a.map.total : t0 + a.tile;
    const int64_t c0 = (static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63)) * V;
    const bool on = c0 < a.channels;
    const uint32_t c = on ? static_cast<uint32_t>(c0) : 0;
    const T *x = static_cast<const T *>(a.x);
    float w[W][V], bias[V];
    load_taps<W, V>(a.weight, a.bias, c, w, bias);
    for_spans(a.map, t0, t1, [&](const Span &s) {
        float h[W - 1 + kBatch][V];      // the last W - 1 inputs, then a batch of new ones
        {
            float old[W - 1][V];
            load_history<T, W, V>(a, x, s, s.lo, c, old);
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) h[r][v] = old[r][v];
        }
        Raw<T, V> raw[kBatch];
        if (s.lo < s.hi) load_rows(x + s.lo * a.x_stride, a.x_stride, c, s.hi - s.lo, raw);
        for (int t = s.lo; t < s.hi; t += kBatch) {
            const int m = s.hi - t;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) raw[k].get(h[W - 1 + k]);
            if (m > kBatch) load_rows(x + (t + kBatch) * a.x_stride, a.x_stride, c, m - kBatch, raw);
            T *row = static_cast<T *>(a.y) + static_cast<int64_t>(t) * a.channels;
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float acc = bias[v];
#pragma unroll
                    for (int j = 0; j < W; ++j) acc = fmaf(w[j][v], h[k + j][v], acc);
                    o[v] = SILU ? silu(acc) : acc;
                }
                if (k < m && on) stv<T, V>(elem(row, c), o);
                row += a.channels;
            }
            // the last W - 1 inputs move to the front
            if (m < kBatch) {
#pragma unroll
                for (int r = 0; r < W - 1; ++r)
#pragma unroll
                    for (int v = 0; v < V; ++v)
#pragma unroll
                        for (int q = 1; q < kBatch; ++q) h[r][v] = m == q ? h[r + q][v] : h[r][v];
                break;
            }
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) h[r][v] = h[r + kBatch][v];
        }
        if (s.ends && a.state_T && on) {
            float *st = a.state_T + static_cast<int64_t>(s.i) * (W - 1) * a.channels + c;
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
                stv<float, V>(st + static_cast<int64_t>(r) * a.channels, h[r]);
        }
    });
}

// One tile's dx (and dstate0), and its partial sums of dweight and dbias. The wave walks the
// tile's tokens and W - 1 more, forming e_t once per token, and writes dx W - 1 tokens behind.
// Batches inside a sequence, nearly all of a long one, take a path without the conditions of its
// ends.
template <typename T, typename TG, int W, int V, bool SILU>
__global__ __launch_bounds__(256) void conv_bwd_kernel(ConvArgs a) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t tile = static_cast<int64_t>(blockIdx.y) * 4 + wave;
    const int64_t t0l = tile * a.tile;
    if (t0l >= a.map.total && t0l > 0) return;
    const int t0 = static_cast<int>(t0l);
    const int t1 = a.map.total - t0 < a.tile ? a.map.total : t0 + a.tile;
    const int64_t c0 = (static_cast<int64_t>(blockIdx.x) * 64 + (threadIdx.x & 63)) * V;
    const bool on = c0 < a.channels;
    const uint32_t c = on ? static_cast<uint32_t>(c0) : 0;
    const T *x = static_cast<const T *>(a.x);
    const TG *dy = static_cast<const TG *>(a.dy);
    float w[W][V], bias[V], dw[W][V], db[V];
    load_taps<W, V>(a.weight, a.bias, c, w, bias);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][v] = 0.f;
    }
    for_spans(a.map, t0, t1, [&](const Span &s) {
        // the last W - 1 inputs and values of e, then a batch of new ones
        float h[W - 1 + kBatch][V], e[W - 1 + kBatch][V];
        {
            float old[W - 1][V];
            load_history<T, W, V>(a, x, s, s.lo, c, old);
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) { h[r][v] = old[r][v]; e[r][v] = 0.f; }
        }
        const int last = s.hi + W - 1;       // one past the last step; e = 0 from s.end on
        Raw<T, V> rx[kBatch];
        Raw<TG, V> rg[kBatch];
        auto fetch = [&](int t) {
            if (t >= s.end || t >= last) return;
            load_rows(x + t * a.x_stride, a.x_stride, c, s.end - t, rx);
            load_rows(dy + static_cast<int64_t>(t) * a.channels, a.channels, c, s.end - t, rg);
        };
        auto batch = [&](auto inner, int t) {
            constexpr bool INNER = decltype(inner)::value;
            float g[kBatch][V];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                rx[k].get(h[W - 1 + k]);
                rg[k].get(g[k]);
            }
            if (t + kBatch < last) fetch(t + kBatch);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int tk = t + k;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float ek = g[k][v];
                    if (SILU) {
                        float acc = bias[v];
#pragma unroll
                        for (int j = 0; j < W; ++j) acc = fmaf(w[j][v], h[k + j][v], acc);
                        ek *= silu_slope(acc);
                    }
                    e[W - 1 + k][v] = INNER || tk < s.end ? ek : 0.f;
                }
                if (tk < s.hi)               // each token counts in one tile
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        db[v] += e[W - 1 + k][v];
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][v] = fmaf(e[W - 1 + k][v], h[k + j][v], dw[j][v]);
                    }
                float o[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    o[v] = 0.f;
#pragma unroll
                    for (int j = 0; j < W; ++j) o[v] = fmaf(w[j][v], e[W - 1 + k - j][v], o[v]);
                }
                const int at = tk - (W - 1);             // the token whose gradient is whole now
                if constexpr (INNER) {
                    if (at < s.lo || at >= s.hi) continue;
                } else {
                    if (tk >= last) continue;
                    const bool before = at < s.first;    // a row of the conv state
                    if (before ? !(s.starts && a.dstate0) : at < s.lo) continue;
                    const int r = at - (s.end - (W - 1));     // the row of state_T that is this input
                    if (a.dstate_T && r >= 0) {
                        float d[V];
                        ldv<float, V>(a.dstate_T + (static_cast<int64_t>(s.i) * (W - 1) + r) * a.channels + c, d);
#pragma unroll
                        for (int v = 0; v < V; ++v) o[v] += d[v];
                    }
                    if (before) {
                        const int64_t row = static_cast<int64_t>(s.i) * (W - 1) + (at - s.first + W - 1);
                        if (on) stv<float, V>(a.dstate0 + row * a.channels + c, o);
                        continue;
                    }
                }
                if (on) stv<TG, V>(elem(static_cast<TG *>(a.dx) + static_cast<int64_t>(at) * a.channels, c), o);
            }
#pragma unroll
            for (int r = 0; r < W - 1; ++r)
#pragma unroll
                for (int v = 0; v < V; ++v) { h[r][v] = h[r + kBatch][v]; e[r][v] = e[r + kBatch][v]; }
        };
        fetch(s.lo);
        for (int t = s.lo; t < last; t += kBatch) {
            const bool rows = s.starts && a.dstate0 && t - (W - 1) < s.first;    // of the conv state
            if (t + kBatch <= s.end && !rows) batch(std::true_type{}, t);
            else batch(std::false_type{}, t);
        }
    });
    if (!on) return;
    // partial sums: [tile][W + 1][channels], the bias last
    float *part = a.partial + tile * (W + 1) * a.channels + c;
#pragma unroll
    for (int j = 0; j < W; ++j) stv<float, V>(part + static_cast<int64_t>(j) * a.channels, dw[j]);
    stv<float, V>(part + static_cast<int64_t>(W) * a.channels, db);
}

// dweight [C][W] and dbias [C]: the tiles' partial sums, added in a fixed order (the same bits
// at every call). 64 columns per workgroup; its sixteen waves take every sixteenth tile.
__global__ __launch_bounds__(1024) void conv_reduce_kernel(const float *part, int tiles, int channels,
                                                           int width, float *dweight, float *dbias) {
    __shared__ float s[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int64_t cols = static_cast<int64_t>(channels) * (width + 1);
    const int64_t col = static_cast<int64_t>(blockIdx.x) * 64 + lane;
    float sum = 0.f;
    if (col < cols)
#pragma unroll 4
        for (int i = wave; i < tiles; i += 16) sum += part[i * cols + col];
    s[wave][lane] = sum;
    __syncthreads();
    if (wave != 0 || col >= cols) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) sum += s[i][lane];
    const int j = static_cast<int>(col / channels);
    const int64_t c = col - static_cast<int64_t>(j) * channels;
    if (j < width) dweight[c * width + j] = sum;
    else if (dbias) dbias[c] = sum;
}

// T tokens of every sequence against its slot of the pool: one lane per sequence and V channels,
// the state row read once and written once. A slot index outside the pool marks padding.
template <typename T, int W, int V, bool SILU>
__global__ __launch_bounds__(256) void conv_step_kernel(ConvStepArgs a) {
    const int64_t c0 = (static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x) * V;
    if (c0 >= a.channels) return;
    const int c = static_cast<int>(c0);
    for (int64_t n = blockIdx.y; n < a.num_seqs; n += gridDim.y) {
        const int slot = a.idx ? a.idx[n] : static_cast<int>(n);
        const T *x = static_cast<const T *>(a.x) + n * a.ntok * a.x_stride + c;
        T *y = static_cast<T *>(a.y) + n * a.ntok * static_cast<int64_t>(a.channels) + c;
        if (slot < 0 || slot >= a.num_slots) {
            const float zero[V] = {};
            for (int t = 0; t < a.ntok; ++t) stv<T, V>(y + static_cast<int64_t>(t) * a.channels, zero);
            continue;
        }
        float *st = a.state + static_cast<int64_t>(slot) * (W - 1) * a.channels + c;
        float h[W][V], w[W][V], bias[V];
#pragma unroll
        for (int r = 0; r < W - 1; ++r) ldv<float, V>(st + static_cast<int64_t>(r) * a.channels, h[r]);
        load_taps<W, V>(a.weight, a.bias, c, w, bias);
        for (int t = 0; t < a.ntok; ++t) {
            ldv<T, V>(x + t * a.x_stride, h[W - 1]);
            float o[V];
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float acc = bias[v];
#pragma unroll
                for (int j = 0; j < W; ++j) acc = fmaf(w[j][v], h[j][v], acc);
                o[v] = SILU ? silu(acc) : acc;
            }
            stv<T, V>(y + static_cast<int64_t>(t) * a.channels, o);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) h[j][v] = h[j + 1][v];
        }
#pragma unroll
        for (int r = 0; r < W - 1; ++r) stv<float, V>(st + static_cast<int64_t>(r) * a.channels, h[r]);
    }
}

// Whether V channels per lane can be read and written in whole pieces: V elements of the token
// tensors, up to 16 bytes of the fp32 ones.
bool whole(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % (bytes < 16 ? bytes : 16) == 0; }
bool vector_ok(const ConvArgs &a, int V) {
    const int t = V * (a.bf16 ? 2 : 4), g = V * (a.grad_bf16 ? 2 : 4), f = V * 4;
    return a.channels % V == 0 && a.x_stride % V == 0 && whole(a.x, t) && whole(a.y, t) &&
           whole(a.dy, g) && whole(a.dx, g) && whole(a.state0, f) && whole(a.state_T, f) &&
           whole(a.dstate0, f) && whole(a.dstate_T, f) && whole(a.weight, 16) && whole(a.bias, f);
}

dim3 tile_grid(const ConvArgs &a, int V) {
    const int64_t tiles = conv_tiles(a.map.total, a.tile);
    return dim3(static_cast<unsigned>((a.channels + 64 * V - 1) / (64 * V)),
                static_cast<unsigned>((tiles + 3) / 4));
}

template <typename T, int V, bool SILU>
hipError_t launch_fwd_s(const ConvArgs &a, hipStream_t st) {
    const dim3 grid = tile_grid(a, V);
    switch (a.width) {
    case 2: hipLaunchKernelGGL((conv_fwd_kernel<T, 2, V, SILU>), grid, dim3(256), 0, st, a); break;
    case 3: hipLaunchKernelGGL((conv_fwd_kernel<T, 3, V, SILU>), grid, dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL((conv_fwd_kernel<T, 4, V, SILU>), grid, dim3(256), 0, st, a); break;
    }
    return hipGetLastError();
}

template <typename T, int V>
hipError_t launch_fwd(const ConvArgs &a, hipStream_t st) {
    return a.silu ? launch_fwd_s<T, V, true>(a, st) : launch_fwd_s<T, V, false>(a, st);
}

template <typename T, typename TG, int V, bool SILU>
hipError_t launch_bwd_s(const ConvArgs &a, hipStream_t st) {
    const dim3 grid = tile_grid(a, V);
    switch (a.width) {
    case 2: hipLaunchKernelGGL((conv_bwd_kernel<T, TG, 2, V, SILU>), grid, dim3(256), 0, st, a); break;
    case 3: hipLaunchKernelGGL((conv_bwd_kernel<T, TG, 3, V, SILU>), grid, dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL((conv_bwd_kernel<T, TG, 4, V, SILU>), grid, dim3(256), 0, st, a); break;
    }
    return hipGetLastError();
}

template <typename T, typename TG, int V>
hipError_t launch_bwd(const ConvArgs &a, hipStream_t st) {
    const hipError_t e = a.silu ? launch_bwd_s<T, TG, V, true>(a, st) : launch_bwd_s<T, TG, V, false>(a, st);
    if (e != hipSuccess) return e;
    const int64_t cols = static_cast<int64_t>(a.channels) * (a.width + 1);
    hipLaunchKernelGGL(conv_reduce_kernel, dim3(static_cast<unsigned>((cols + 63) / 64)), dim3(1024),
                       0, st, a.partial, static_cast<int>(conv_tiles(a.map.total, a.tile)), a.channels,
                       a.width, a.dweight, a.dbias);
    return hipGetLastError();
}

template <typename T, int V, bool SILU>
hipError_t launch_step_s(const ConvStepArgs &a, hipStream_t st) {
    const dim3 grid(static_cast<unsigned>((a.channels + 256 * V - 1) / (256 * V)),
                    static_cast<unsigned>(a.num_seqs < 65535 ? a.num_seqs : 65535));
    switch (a.width) {
    case 2: hipLaunchKernelGGL((conv_step_kernel<T, 2, V, SILU>), grid, dim3(256), 0, st, a); break;
    case 3: hipLaunchKernelGGL((conv_step_kernel<T, 3, V, SILU>), grid, dim3(256), 0, st, a); break;
    default: hipLaunchKernelGGL((conv_step_kernel<T, 4, V, SILU>), grid, dim3(256), 0, st, a); break;
    }
    return hipGetLastError();
}

template <typename T, int V>
hipError_t launch_step(const ConvStepArgs &a, hipStream_t st) {
    return a.silu ? launch_step_s<T, V, true>(a, st) : launch_step_s<T, V, false>(a, st);
}

}  // namespace

// Tokens per tile: about six waves of the forward's 256 channels or three of the backward's 128 on
// each SIMD, and at least 8 tokens, where the rows next to a tile are nearly half of what a wave
// reads. On 4,096 tokens x 6,144 channels: 16 tokens forward (21.1 us; 24 tokens
// 22.0, 48 tokens 25.4), 64 backward (39.0 us; 24 tokens 45.0). Where channels are taken one by one a
// wave has 64, and there are four (backward two) times as many: 2,311 tokens x 1,537 bf16 channels
// take 9.1 us forward, 1,536 channels 6.5.
int conv_tile(int64_t tokens, int channels, bool backward) {
    const int per = backward ? 128 : 256;
    const int64_t waves = (static_cast<int64_t>(channels) + per - 1) / per;
    int64_t t = (tokens * waves / ((backward ? 3 : 6) * kSimds) + kBatch - 1) / kBatch * kBatch;
    if (t < 8) t = 8;
    if (t > 64) t = 64;
    // the grid's second dimension holds at most 65,535 workgroups of four tiles
    while ((tokens + t - 1) / t > 4 * 65535) t *= 2;
    return static_cast<int>(t);
}

int64_t conv_tiles(int64_t tokens, int tile) {
    const int64_t n = (tokens + tile - 1) / tile;
    return n > 0 ? n : 1;
}

hipError_t launch_conv_fwd(const ConvArgs &a, hipStream_t st) {
    if (a.bf16) return vector_ok(a, 4) ? launch_fwd<bf16_t, 4>(a, st) : launch_fwd<bf16_t, 1>(a, st);
    return vector_ok(a, 4) ? launch_fwd<float, 4>(a, st) : launch_fwd<float, 1>(a, st);
}

hipError_t launch_conv_bwd(const ConvArgs &a, hipStream_t st) {
    if (!a.bf16)
        return vector_ok(a, 2) ? launch_bwd<float, float, 2>(a, st) : launch_bwd<float, float, 1>(a, st);
    const bool v = vector_ok(a, 2);
    if (a.grad_bf16) return v ? launch_bwd<bf16_t, bf16_t, 2>(a, st) : launch_bwd<bf16_t, bf16_t, 1>(a, st);
    return v ? launch_bwd<bf16_t, float, 2>(a, st) : launch_bwd<bf16_t, float, 1>(a, st);
}

hipError_t launch_conv_step(const ConvStepArgs &a, hipStream_t st) {
    const int t = a.bf16 ? 8 : 16;
    const bool v = a.channels % 4 == 0 && a.x_stride % 4 == 0 && whole(a.x, t) && whole(a.y, t) &&
                   whole(a.state, 16) && whole(a.weight, 16) && whole(a.bias, 16);
    if (a.bf16) return v ? launch_step<bf16_t, 4>(a, st) : launch_step<bf16_t, 1>(a, st);
    return v ? launch_step<float, 4>(a, st) : launch_step<float, 1>(a, st);
}

}  // namespace gdn2
