// gdn2_layer.h -- device helpers of the operators around the recurrence (short convolution,
// selective scan, block norm): vector element access, the SiLU, and the walk of a wave over
// the sequences that share a tile of the token axis.
#pragma once
#include "gdn2_common.h"
#include "gdn2_internal.h"

namespace gdn2 {

constexpr int kSimds = 1024;     // 256 CUs of four

// V consecutive elements of T as floats, in accesses of up to 16 bytes. The caller sees to the
// alignment (V * sizeof(T), at most 16 bytes); V = 1 needs none beyond the element's own.
template <typename T, int V>
__device__ __forceinline__ void ldv(const T *p, float (&x)[V]) {
    if constexpr (V == 1) {
        x[0] = io<T>::ld(p);
    } else if constexpr (V % 4 == 2 && sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(p + i);
            x[i] = v.x; x[i + 1] = v.y;
        }
    } else if constexpr (V == 2) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
        x[0] = __uint_as_float(w << 16);
        x[1] = __uint_as_float(w & 0xffff0000u);
    } else if constexpr (sizeof(T) == 4) {
        static_assert(V % 4 == 0, "whole 16-byte pieces");
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const f32x4 v = io<T>::ld4(p + i);
            x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
        }
    } else if constexpr (V == 4) {
        const f32x4 v = io<T>::ld4(p);
        x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
    } else {
        static_assert(V == 8, "bf16 vectors have 1, 2, 4 or 8 elements");
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x[2 * i] = __uint_as_float(w[i] << 16);
            x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
}

template <typename T, int V>
__device__ __forceinline__ void stv(T *p, const float (&x)[V]) {
    if constexpr (V == 1) {
        io<T>::st(p, x[0]);
    } else if constexpr (V == 2 && sizeof(T) == 4) {
        *reinterpret_cast<float2 *>(p) = float2{x[0], x[1]};
    } else if constexpr (V == 2) {
        *reinterpret_cast<uint32_t *>(p) = static_cast<uint32_t>(f32_to_bf16_bits(x[0])) |
                                           (static_cast<uint32_t>(f32_to_bf16_bits(x[1])) << 16);
    } else if constexpr (sizeof(T) == 4 || V == 4) {
#pragma unroll
        for (int i = 0; i < V; i += 4) io<T>::st4(p + i, f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]});
    } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            w[i] = static_cast<uint32_t>(f32_to_bf16_bits(x[2 * i])) |
                   (static_cast<uint32_t>(f32_to_bf16_bits(x[2 * i + 1])) << 16);
        *reinterpret_cast<uint4 *>(p) = uint4{w[0], w[1], w[2], w[3]};
    }
}

// Element c of a row: one pointer for the wave and 32 bits of offset per lane (c < 2^20), the
// form that global memory instructions take without address arithmetic.
template <typename T>
__device__ __forceinline__ const T *elem(const T *row, uint32_t c) {
    return reinterpret_cast<const T *>(reinterpret_cast<const char *>(row) + c * static_cast<uint32_t>(sizeof(T)));
}
template <typename T>
__device__ __forceinline__ T *elem(T *row, uint32_t c) {
    return reinterpret_cast<T *>(reinterpret_cast<char *>(row) + c * static_cast<uint32_t>(sizeof(T)));
}

// V elements as they are in memory: loaded now, widened when they are used, so that the load does
// not have to be waited for before.
template <typename T, int V>
struct Raw {
    static constexpr int N = V * sizeof(T) / 4;
    typedef uint32_t words __attribute__((ext_vector_type(N), aligned(N * 4 < 16 ? N * 4 : 16)));
    words w;
    __device__ __forceinline__ void load(const T *p) { w = *reinterpret_cast<const words *>(p); }
    __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if constexpr (sizeof(T) == 4) {
                x[i] = __uint_as_float(w[i]);
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
};
template <typename T>
struct Raw<T, 1> {
    T w;
    __device__ __forceinline__ void load(const T *p) { w = *p; }
    __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = io<T>::val(w); }
};

// Element c of the K rows from `row` on, V of them; rows from m on repeat row m - 1, so no access
// is conditional (m >= 1).
template <typename T, int V, int K>
__device__ __forceinline__ void load_rows(const T *row, int64_t stride, uint32_t c, int m, Raw<T, V> (&v)[K]) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
        v[k].load(elem(row, c));
        row += k + 1 < m ? stride : 0;
    }
}

constexpr float kLog2e = 1.44269504088896340736f;

// 1 / (1 + e^-a): exp2 and reciprocal of the transcendental unit, each within 1 ulp.
__device__ __forceinline__ float sigmoid_hw(float a) {
    return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(-kLog2e * a));
}
__device__ __forceinline__ float silu(float a) { return a * sigmoid_hw(a); }
// d silu(a) / da = s (1 + a (1 - s)), s = sigmoid(a)
__device__ __forceinline__ float silu_slope(float a) {
    const float s = sigmoid_hw(a);
    return s * fmaf(a, 1.f - s, 1.f);
}

// Offset of sequence i of a SeqMap (i = n: the end of the last one). Offsets are held inside
// [0, total], so a wrong table never makes an access leave the tensors.
__host__ __device__ __forceinline__ int seq_begin(const SeqMap &m, int i) {
    if (!m.cu) return i * m.seqlen;
    const int v = m.cu[i];
    return v < 0 ? 0 : (v > m.total ? m.total : v);
}

// The first i in [0, n] with seq_begin(i) >= t, or n + 1. 64 offsets are looked at a time, so a
// search takes one load per factor of 64 in n: count(lo, step, hi) says how many of the offsets
// i = lo + l * step < hi, l < 64, are below t. (Split from seq_first_at so that it runs on a host.)
template <typename Count>
__host__ __device__ __forceinline__ int seq_search(const SeqMap &m, int t, Count &&count) {
    if (!m.cu) {
        if (t <= 0) return 0;
        if (m.seqlen <= 0) return m.n + 1;
        const int i = (t - 1) / m.seqlen + 1;
        return i > m.n ? m.n + 1 : i;
    }
    int lo = 0, hi = m.n + 1;
    while (lo < hi) {
        const int step = (hi - lo + 63) >> 6;
        const int c = count(lo, step, hi);
        if (c == 0) break;
        if (step == 1) return lo + c;
        const int64_t end = lo + static_cast<int64_t>(c) * step;
        lo += (c - 1) * step + 1;
        if (end < hi) hi = static_cast<int>(end);
    }
    return lo;
}

// The search by a whole wave, an offset per lane.
__device__ __forceinline__ int seq_first_at(const SeqMap &m, int t) {
    const int lane = threadIdx.x & 63;
    return seq_search(m, t, [&](int lo, int step, int hi) {
        const int64_t i = lo + static_cast<int64_t>(lane) * step;
        const bool before = i < hi && seq_begin(m, static_cast<int>(i)) < t;
        return __popcll(__ballot(before));
    });
}

// One sequence's share [lo, hi) of a tile: sequence i covers tokens [first, end).
struct Span {
    int i, first, end, lo, hi;
    bool starts, ends;     // the tile holds the sequence's first position; its end
};

// Calls f(Span) for every sequence that has tokens in [t0, t1), in order, from i on, which
// seq_search found for t0. Empty sequences come too, once each: with the tile that holds their
// position, those at the very end (t1 == total) with the last tile. Tokens behind the last sequence
// belong to no span. With offsets that decrease, spans are wrong, but 0 <= first <= lo <= hi <= total
// and t0 <= lo, hi <= t1 hold for any table, which is what keeps every access inside the tensors.
template <typename F>
__host__ __device__ __forceinline__ void walk_spans(const SeqMap &m, int t0, int t1, int i, F &&f) {
    bool inside = i > 0 && i <= m.n && seq_begin(m, i) > t0;    // t0 lies inside sequence i - 1
    if (inside) --i;
    for (; i < m.n; ++i) {
        const int first = seq_begin(m, i);
        if (!inside && first >= t1 && t1 < m.total) return;
        int end = seq_begin(m, i + 1);
        if (end < first) end = first;
        const int lo = inside || first < t0 ? t0 : first, hi = end < t1 ? end : t1;
        // (first > lo: a sequence taken as entered that a decreasing table puts behind the tile's start)
        f(Span{i, first < lo ? first : lo, end, lo, hi < lo ? lo : hi, !inside, end <= t1});
        if (end > t1) return;
        inside = false;
    }
}

// The same for a tile of a wave: every lane takes part, and everything in the span is the same in
// all of them.
template <typename F>
__device__ __forceinline__ void for_spans(const SeqMap &m, int t0, int t1, F &&f) {
    walk_spans(m, t0, t1, __builtin_amdgcn_readfirstlane(seq_first_at(m, t0)), static_cast<F &&>(f));
}

}  // namespace gdn2
