// gdn2_scan.h -- shared by the selective scan's kernels: the lane layout and the step size.
//
// A wave holds CW = 64 / S channels: lane l owns channel l % CW and the NS states
// [NS (l / CW), NS (l / CW) + NS) of it, so a channel's d_state <= NS * S states lie in S lanes.
// The four waves of a workgroup take neighbouring channels of one group (which share B and C)
// and the same tile of tokens.
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

// log(1 + e), 0 <= e <= 1, as 2 atanh(e / (2 + e)): the series in s^2 <= 1/9, cut where the next
// term is below 2^-26 of the value, so small e keep their relative precision (log(1 + e) of the
// rounded sum would lose it: steps of 0.001 are usual).
__device__ __forceinline__ float log1p_unit(float e) {
    const float s = e * __builtin_amdgcn_rcpf(2.f + e), q = s * s;
    float p = 1.f / 15.f;
    p = fmaf(p, q, 1.f / 13.f);
    p = fmaf(p, q, 1.f / 11.f);
    p = fmaf(p, q, 1.f / 9.f);
    p = fmaf(p, q, 1.f / 7.f);
    p = fmaf(p, q, 1.f / 5.f);
    p = fmaf(p, q, 1.f / 3.f);
    return 2.f * fmaf(p * q, s, s);
}

// softplus(x) = max(x, 0) + log(1 + e^-|x|)
__device__ __forceinline__ float softplus(float x) {
    return fmaxf(x, 0.f) + log1p_unit(__builtin_amdgcn_exp2f(-kLog2e * fabsf(x)));
}

// The decay rates of a lane's states times log2(e), so that a decay is exp2(dt * A2).
template <int NS, int S>
__device__ __forceinline__ void load_rates(const ScanArgs &a, const ScanLane<NS, S> &l, float (&A2)[NS]) {
    const float *A = a.A + static_cast<int64_t>(l.c) * a.d_state;
#pragma unroll
    for (int n = 0; n < NS; ++n)
        A2[n] = l.on && l.n0 + n < a.d_state ? kLog2e * A[l.n0 + n] : 0.f;
}

// A lane's states from / to a row of [N][channels][d_state].
template <int NS, int S>
__device__ __forceinline__ void load_state(const ScanArgs &a, const ScanLane<NS, S> &l, const float *s,
                                           int i, float (&h)[NS]) {
    const float *p = s + (static_cast<int64_t>(i) * a.channels + l.c) * a.d_state;
#pragma unroll
    for (int n = 0; n < NS; ++n) h[n] = l.on && l.n0 + n < a.d_state ? p[l.n0 + n] : 0.f;
}
template <int NS, int S>
__device__ __forceinline__ void store_state(const ScanArgs &a, const ScanLane<NS, S> &l, float *s, int i,
                                            const float (&h)[NS]) {
    float *p = s + (static_cast<int64_t>(i) * a.channels + l.c) * a.d_state;
#pragma unroll
    for (int n = 0; n < NS; ++n)
        if (l.on && l.n0 + n < a.d_state) p[l.n0 + n] = h[n];
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

constexpr int kB = 8;        // tokens whose inputs are in flight and whose B and C are staged together

// B (and C) of tokens [t, hi) of a group, staged as fp32 [kB][NP] each, zero where there is none.
// take() loads this thread's share of a batch into registers, put() writes it to LDS.
template <typename T, int NP, bool WITH_C>
struct Stage {
    static constexpr int ROW = WITH_C ? 2 * NP : NP, PER = (kB * ROW + 255) / 256;
    float r[PER];
    __device__ __forceinline__ void take(const ScanArgs &a, int g, int t, int hi) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = threadIdx.x + 256 * i, k = e / ROW, j = e % ROW, n = j % NP;
            r[i] = 0.f;
            if (k < kB && t + k < hi && n < a.d_state) {
                const bool c = WITH_C && j >= NP;
                const T *p = static_cast<const T *>(c ? a.C : a.B);
                r[i] = io<T>::ld(p + (t + k) * (c ? a.c_stride : a.b_stride) + g * a.d_state + n);
            }
        }
    }
    __device__ __forceinline__ void put(float *s) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int e = threadIdx.x + 256 * i;
            if (PER * 256 == kB * ROW || e < kB * ROW) s[e] = r[i];
        }
    }
};

// NS floats from LDS, the same address in all lanes of a part.
template <int NS>
__device__ __forceinline__ void lds_row(const float *s, float (&v)[NS]) {
#pragma unroll
    for (int n = 0; n < NS; n += 4) {
        const f32x4 x = *reinterpret_cast<const f32x4 *>(s + n);
        v[n] = x.x; v[n + 1] = x.y; v[n + 2] = x.z; v[n + 3] = x.w;
    }
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
    const float A2 = kLog2e * a.A[static_cast<int64_t>(c) * a.d_state + n];
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
