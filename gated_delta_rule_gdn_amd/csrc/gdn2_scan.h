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

}  // namespace gdn2
