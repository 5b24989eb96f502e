// gdn2_scan.h -- shared by the selective scan's kernels: the lane layout and the step size.
//
// A wave holds CW = 64 / S channels: lane l owns channel l % CW and the NS states
// [NS (l / CW), NS (l / CW) + NS) of it, so a channel's d_state <= NS * S states lie in S lanes.
// The four waves of a workgroup take neighbouring channels of one group (which share B and C)
// and the same tile of tokens. Lanes past a group's last channel run along on its first one and
// store nothing, so groups of fewer channels than a workgroup's cost a whole one each: gradients of
// 64 x 512 tokens x 128 channels x 16 states, bf16, take 206 us in one group and 558 us in four.
#pragma once
#include "gdn2_internal.h"
#include "gdn2_layer.h"

namespace gdn2 {

constexpr int kScanWaves = 4;

template <int NS, int S>
struct ScanLane {
    static constexpr int CW = 64 / S, NP = NS * S;
    int wave, c, part, n0, g;
    bool on;
    __device__ __forceinline__ ScanLane(const ScanArgs &a, int block) {
        const int lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        const int per = a.channels / a.groups;                       // channels of a group
        const int blocks = (per + kScanWaves * CW - 1) / (kScanWaves * CW);
        g = block / blocks;
        const int in = (block - g * blocks) * kScanWaves * CW + wave * CW + (lane & (CW - 1));
        on = in < per;
        c = g * per + (on ? in : 0);
        part = lane / CW;
        n0 = part * NS;
    }
};

// Sum over the S lanes of a channel.
template <int S>
__device__ __forceinline__ float sum_parts(float x) {
#pragma unroll
    for (int m = 64 / S; m < 64; m <<= 1) x += __shfl_xor(x, m);
    return x;
}

// softplus(x) = max(x, 0) + log(1 + e), e = e^-|x| in [0, 1]. log(1 + e) / e is a polynomial of
// degree 8, fitted for the least relative error on [0, 1], so that a small e, a usual step of 0.001,
// keeps its relative precision. With its coefficients rounded to fp32 it is within 6.5e-8, and with
// fp32 Horner steps within 1.4e-7 (2.3 * 2^-24), taken over every fp32 e from 1e-12 to 1.
__device__ __forceinline__ float softplus(float x) {
    const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(x));
    float p = 0.005232692696154118f;
    p = fmaf(p, e, -0.029505232349038124f);
    p = fmaf(p, e, 0.07822594046592712f);
    p = fmaf(p, e, -0.13663244247436523f);
    p = fmaf(p, e, 0.19106006622314453f);
    p = fmaf(p, e, -0.2484298199415207f);
    p = fmaf(p, e, 0.3331909775733948f);
    p = fmaf(p, e, -0.4999949336051941f);
    p = fmaf(p, e, 0.9999999403953552f);
    return fmaf(p, e, fmaxf(x, 0.f));
}

// softplus of K values that are the same in the S lanes of a channel: with S > 1 the lanes of either
// half of the wave form half of them, and the halves are exchanged.
template <int S, int K>
__device__ __forceinline__ void softplus_shared(float (&d)[K]) {
    if constexpr (S == 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) d[k] = softplus(d[k]);
    } else {
        const bool up = threadIdx.x & 32;
#pragma unroll
        for (int k = 0; k < K / 2; ++k) {
            const uint32_t v = __float_as_uint(softplus(up ? d[k + K / 2] : d[k]));
            const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
            d[k] = __uint_as_float(r[0]);
            d[k + K / 2] = __uint_as_float(r[1]);
        }
    }
}

// A decay rate times log2(e), so that a decay is exp2(dt * rate2(A)). A rate of -inf becomes the
// lowest value, so that a step of zero keeps the state (0 * -inf would not).
__device__ __forceinline__ float rate2(float A) {
    const float r = kLog2e * A;
    return r == -__builtin_inff() ? -3.4e38f : r;
}

// A lane's states of one channel's row of d_state floats: zero where there is none, in whole pieces
// of four where ScanArgs::vec allows. PIECES false: value by value, where the
// pieces' registers would spill.
template <bool PIECES, int NS, int S>
__device__ __forceinline__ void load_row(const ScanArgs &a, const ScanLane<NS, S> &l, const float *row,
                                         float (&h)[NS]) {
    if constexpr (!PIECES) {
#pragma unroll
        for (int n = 0; n < NS; ++n) h[n] = l.on && l.n0 + n < a.d_state ? row[l.n0 + n] : 0.f;
        return;
    }
    if (a.vec) {
#pragma unroll
        for (int n = 0; n < NS; n += 4) {
            const f32x4 v = *reinterpret_cast<const f32x4 *>(row + (l.n0 + n < a.d_state ? l.n0 + n : 0));
            h[n] = v.x; h[n + 1] = v.y; h[n + 2] = v.z; h[n + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int n = 0; n < NS; ++n) h[n] = row[l.n0 + n < a.d_state ? l.n0 + n : 0];
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = l.on && l.n0 + n < a.d_state ? h[n] : 0.f;
}

// The decay rates of a lane's states.
template <int NS, int S>
__device__ __forceinline__ void load_rates(const ScanArgs &a, const ScanLane<NS, S> &l, float (&A2)[NS]) {
    load_row<true>(a, l, a.A + static_cast<int64_t>(l.c) * a.d_state, A2);
#pragma unroll
    for (int n = 0; n < NS; ++n) A2[n] = rate2(A2[n]);
}

// A lane's states of sequence i from / to [num_seqs][channels][d_state].
template <bool PIECES = true, int NS, int S>
__device__ __forceinline__ void load_state(const ScanArgs &a, const ScanLane<NS, S> &l, const float *s,
                                           int i, float (&h)[NS]) {
    load_row<PIECES>(a, l, s + (static_cast<int64_t>(i) * a.channels + l.c) * a.d_state, h);
}
template <int NS, int S>
__device__ __forceinline__ void store_state(const ScanArgs &a, const ScanLane<NS, S> &l, float *s, int i,
                                            const float (&h)[NS]) {
    float *p = s + (static_cast<int64_t>(i) * a.channels + l.c) * a.d_state;
    if (a.vec) {
#pragma unroll
        for (int n = 0; n < NS; n += 4)
            if (l.on && l.n0 + n < a.d_state)
                *reinterpret_cast<f32x4 *>(p + l.n0 + n) = f32x4{h[n], h[n + 1], h[n + 2], h[n + 3]};
    } else {
#pragma unroll
        for (int n = 0; n < NS; ++n)
            if (l.on && l.n0 + n < a.d_state) p[l.n0 + n] = h[n];
    }
}

// The same from / to a tile's row of a workspace [tiles][d_state][channels] (neighbouring lanes
// next to each other).
template <int NS, int S>
__device__ __forceinline__ void load_tile(const ScanArgs &a, const ScanLane<NS, S> &l, const float *s,
                                          int64_t tile, float (&h)[NS]) {
    const float *p = s + tile * a.d_state * a.channels + l.c;
#pragma unroll
    for (int n = 0; n < NS; ++n)
        h[n] = l.on && l.n0 + n < a.d_state ? p[static_cast<int64_t>(l.n0 + n) * a.channels] : 0.f;
}
template <int NS, int S>
__device__ __forceinline__ void store_tile(const ScanArgs &a, const ScanLane<NS, S> &l, float *s,
                                           int64_t tile, const float (&h)[NS]) {
    float *p = s + tile * a.d_state * a.channels + l.c;
#pragma unroll
    for (int n = 0; n < NS; ++n)
        if (l.on && l.n0 + n < a.d_state) p[static_cast<int64_t>(l.n0 + n) * a.channels] = h[n];
}

// The state that enters a tile, chained here from the tiles that sequence `s` reaches through
// before it: what chain_tiles leaves in the workspace.
template <int NS, int S>
__device__ __forceinline__ void walk_tiles(const ScanArgs &a, const ScanLane<NS, S> &l, const Span &s,
                                           int64_t tile, const float (&A2)[NS], float (&h)[NS]) {
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = 0.f;
    constexpr int U = 8;       // tiles whose loads are in flight together
    const int64_t first = s.first / a.tile;
    for (int64_t i0 = first; i0 < tile; i0 += U) {
        float hl[U][NS], dl[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            const int64_t i = i0 + k < tile ? i0 + k : tile - 1;
            const float *p = a.tiles_h + i * a.d_state * a.channels + l.c;
            dl[k] = a.tiles_dt[i * a.channels + l.c];
#pragma unroll
            for (int n = 0; n < NS; ++n)
                hl[k][n] = p[static_cast<int64_t>(l.n0 + n < a.d_state ? l.n0 + n : 0) * a.channels];
        }
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i0 + k < tile)
#pragma unroll
                for (int n = 0; n < NS; ++n) {
                    // the first tile's sum of dt is also of sequences before this one
                    const float on = fmaf(__builtin_amdgcn_exp2f(A2[n] * dl[k]), h[n], hl[k][n]);
                    h[n] = i0 + k > first ? on : hl[k][n];
                }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = l.on && l.n0 + n < a.d_state ? h[n] : 0.f;
}

constexpr int kB = 8;        // tokens whose inputs are in flight and whose B and C are staged together

// B (and C) of the m <= kB tokens from t on, staged as fp32 [kB][NP] each, zero where there is
// none. take() loads this thread's share of a batch into registers, put() writes it to LDS.
template <typename T, int NP, bool WITH_C>
struct Stage {
    static constexpr int ROW = WITH_C ? 2 * NP : NP, PER = (kB * ROW + 255) / 256;
    T r[PER];
    __device__ __forceinline__ void take(const ScanArgs &a, int g, int t, int m) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = threadIdx.x + 256 * i, k = e / ROW, j = e % ROW, n = j % NP;
            r[i] = T{};
            if (k < m && n < a.d_state) {
                const bool c = WITH_C && j >= NP;
                const T *p = static_cast<const T *>(c ? a.C : a.B);
                r[i] = p[(t + k) * (c ? a.c_stride : a.b_stride) + g * a.d_state + n];
            }
        }
    }
    __device__ __forceinline__ void put(float *s) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = threadIdx.x + 256 * i;
            if (PER * 256 == kB * ROW || e < kB * ROW) s[e] = io<T>::val(r[i]);
        }
    }
};

// Element c of the K rows from `row` on; rows from m on repeat row m - 1, so no access is
// conditional.
template <typename T, int K>
__device__ __forceinline__ void fetch_rows(const T *row, int64_t stride, uint32_t c, int m, T (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k] = *elem(row, c);
        row += k + 1 < m ? stride : 0;
    }
}
template <typename T, int K>
__device__ __forceinline__ void widen(const T (&r)[K], float (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = io<T>::val(r[k]);
}

// NS floats from LDS, the same address in all lanes of a part.
template <int NS>
__device__ __forceinline__ void lds_row(const float *s, float (&v)[NS]) {
#pragma unroll
    for (int n = 0; n < NS; n += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4 *>(s + n);
        v[n] = x.x; v[n + 1] = x.y; v[n + 2] = x.z; v[n + 3] = x.w;
    }
}

// Holds values where they are computed, at no cost: behind an unrolled batch of tokens it keeps the
// compiler from moving most of the batch into the next block, with all its LDS reads live until
// there.
template <int N>
__device__ __forceinline__ void pin(float (&v)[N]) {
#pragma unroll
    for (int n = 0; n < N; ++n) asm volatile("" : "+v"(v[n]));
}

// Tiles are spread over the grid's second and third dimension.
inline dim3 scan_grid(int blocks, int tiles) {
    const int y = tiles < 32768 ? tiles : 32768;
    return dim3(blocks, y, (tiles + y - 1) / y);
}
__device__ __forceinline__ int64_t tile_index() {
    return static_cast<int64_t>(blockIdx.z) * gridDim.y + blockIdx.y;
}

// Chains the tiles, from the front (DIR 1) or the back (DIR -1): what comes into tile i from the
// tile before it replaces what tile i reached from zero. One thread per (state, channel), sixteen
// tiles' loads in flight together.
template <int DIR>
__device__ __forceinline__ void chain_tiles(const ScanArgs &a, float *states, int tiles) {
    const int64_t col = blockIdx.x * static_cast<int64_t>(256) + threadIdx.x;
    const int64_t cols = static_cast<int64_t>(a.d_state) * a.channels;
    if (col >= cols) return;
    const int n = static_cast<int>(col / a.channels);
    const int c = static_cast<int>(col - static_cast<int64_t>(n) * a.channels);
    const float A2 = rate2(a.A[static_cast<int64_t>(c) * a.d_state + n]);
    float run = 0.f;
    constexpr int U = 16;
    for (int i0 = 0; i0 < tiles; i0 += U) {
        float hl[U], dl[U];
        int pl[U];
#pragma unroll
        for (int k = 0; k < U; ++k)
            if (i0 + k < tiles) {
                const int64_t i = DIR > 0 ? i0 + k : tiles - 1 - i0 - k;
                hl[k] = states[i * cols + col];
                dl[k] = a.tiles_dt[i * a.channels + c];
                pl[k] = a.tiles_pass[i];
            }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (i0 + k < tiles) {
                const int64_t i = DIR > 0 ? i0 + k : tiles - 1 - i0 - k;
                states[i * cols + col] = run;
                run = pl[k] ? fmaf(__builtin_amdgcn_exp2f(A2 * dl[k]), run, hl[k]) : hl[k];
            }
        }
    }
}

}  // namespace gdn2
