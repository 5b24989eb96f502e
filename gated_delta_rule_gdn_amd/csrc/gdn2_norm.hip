// gdn2_norm.hip -- the norms after and before a block, fused with the block's gate, the residual
// and its scale, and their gradients.
//
// Per row of d values, with rstd(v) = 1 / sqrt(mean(v^2) + eps) and every stage but the last
// optional:
//     p = x rstd(x) norm_weight,   u = p silu(gate),   h = residual + scale u,
//     y = h rstd(h) next_weight.
// Gradients, from dh and dy: with w = dy next_weight and r = rstd(h),
//     g = dh + r w - h r^3 mean(w h),        dresidual = g,        dscale = sum_rows g u,
//     dnext_weight = sum_rows dy h r,        g1 = g scale,         dgate = g1 p silu'(gate),
//     g2 = g1 silu(gate),                    dnorm_weight = sum_rows g2 x rstd(x),
//     dx = r_x w_x - x r_x^3 mean(w_x x),    w_x = g2 norm_weight, r_x = rstd(x).
//
// Both are bound by memory: one pass, each input read once, each output written once. A row
// lives in the registers of L lanes (16 to 1,024), 8 values each (16 above 8,192 columns), so
// both statistics are sums over registers and lanes. The statistics and every value between the
// loads and the stores are fp32; h is normalised before it is rounded to its type.
//
// Measured: 8,192 x 2,048 bf16 with every stage 25.4 us of GPU time (134 MB, 5.3 TB/s, what a large
// copy reaches); gradients of 4,096 x 2,048 bf16 with an fp32 residual 52.6 us (185 MB; 48 for the
// pass, 3.9 TB/s behind four row sums with a barrier each, and 4.6 for the parameters' sums). Far
// from the bytes' time are gradients of short rows (see norm_reduce_kernel) and of rows above 4,096
// columns (see launch_rows).
#include "gdn2_internal.h"
#include "gdn2_layer.h"

namespace gdn2 {

namespace {

// Threads of a workgroup: four waves where rows fit in waves, else one row's lanes (a row's sum
// then goes through LDS and barriers, which the workgroup shares).
constexpr int norm_threads(int lanes) { return lanes <= 64 ? 256 : lanes; }

// Sum over the L lanes of a row: inside a wave by exchanges, across waves through LDS. `slot`
// alternates between the two halves of s, so one barrier per sum is enough.
template <int L>
__device__ __forceinline__ float row_sum(float x, float (*s)[16], int slot) {
#pragma unroll
    for (int m = 1; m < (L < 64 ? L : 64); m <<= 1) x += __shfl_xor(x, m);
    if constexpr (L > 64) {
        const int wave = threadIdx.x >> 6;
        if ((threadIdx.x & 63) == 0) s[slot][wave] = x;
        __syncthreads();
        x = 0.f;
#pragma unroll
        for (int w = 0; w < L / 64; ++w) x += s[slot][w];
    }
    return x;
}

// Values a lane holds: P pieces of V neighbouring values, pieces L * V apart.
template <int V, int P>
struct Cols {
    int c0, step, d;
    __device__ __forceinline__ int at(int i) const { return c0 + i * step; }
    __device__ __forceinline__ bool in(int i) const { return at(i) < d; }
};

template <typename T, int V, int P>
__device__ __forceinline__ void load_row(const T *p, const Cols<V, P> &k, float (&x)[P][V], float fill) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (k.in(i)) {
            ldv<T, V>(p + k.at(i), x[i]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) x[i][v] = fill;
        }
    }
}

// The same in two steps: loaded as it is in memory, widened when it is used.
template <typename T, int V, int P>
struct RawRow {
    Raw<T, V> r[P];
    __device__ __forceinline__ void load(const T *p, const Cols<V, P> &k) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (k.in(i)) r[i].load(p + k.at(i));
    }
    __device__ __forceinline__ void get(const Cols<V, P> &k, float (&x)[P][V]) const {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            r[i].get(x[i]);
#pragma unroll
            for (int v = 0; v < V; ++v) x[i][v] = k.in(i) ? x[i][v] : 0.f;
        }
    }
};

template <typename T, int V, int P>
__device__ __forceinline__ void store_row(T *p, const Cols<V, P> &k, const float (&x)[P][V]) {
#pragma unroll
    for (int i = 0; i < P; ++i)
        if (k.in(i)) stv<T, V>(p + k.at(i), x[i]);
}

template <typename T, typename TR, int L, int V, int P>
__global__ __launch_bounds__(norm_threads(L)) void norm_fwd_kernel(NormArgs a) {
    constexpr int ROWS = norm_threads(L) / L;          // rows of a workgroup
    __shared__ float s_sum[2][16];
    const int64_t set = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    const int64_t row = set * ROWS + threadIdx.x / L;
    if (row >= a.rows) return;                          // L > 64: ROWS is 1, whole workgroups
    const Cols<V, P> k{static_cast<int>(threadIdx.x % L) * V, L * V, a.d};
    const float inv = 1.f / a.d;
    float x[P][V], t[P][V];
    load_row<T>(static_cast<const T *>(a.x) + row * a.x_stride, k, x, 0.f);
    float g[P][V], res[P][V];
    if (a.gate) load_row<T>(static_cast<const T *>(a.gate) + row * a.gate_stride, k, g, 0.f);
    if (a.residual) load_row<TR>(static_cast<const TR *>(a.residual) + row * a.d, k, res, 0.f);
    if (a.norm_weight) {
        float q = 0.f;
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) q = fmaf(x[i][v], x[i][v], q);
        const float r = rsqrtf(row_sum<L>(q, s_sum, 0) * inv + a.eps);
        load_row<float>(a.norm_weight, k, t, 0.f);
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) x[i][v] *= r * t[i][v];
    }
    if (a.gate)
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) x[i][v] *= silu(g[i][v]);
    if (a.scale) {
        load_row<float>(a.scale, k, t, 0.f);
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) x[i][v] *= t[i][v];
    }
    if (a.residual)
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) x[i][v] += res[i][v];
    store_row<TR>(static_cast<TR *>(a.h) + row * a.d, k, x);
    if (!a.next_weight) return;
    float q = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) q = fmaf(x[i][v], x[i][v], q);
    const float r = rsqrtf(row_sum<L>(q, s_sum, 1) * inv + a.eps);
    load_row<float>(a.next_weight, k, t, 0.f);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) x[i][v] *= r * t[i][v];
    store_row<T>(static_cast<T *>(a.y) + row * a.d, k, x);
}

// A workgroup takes every gridDim.x-th set of rows and keeps its columns' sums of the parameter
// gradients in registers; they leave as one row of a.partial per row slot.
template <typename T, typename TR, typename TG, typename TGR, int L, int V, int P>
__global__ __launch_bounds__(norm_threads(L)) void norm_bwd_kernel(NormArgs a) {
    constexpr int ROWS = norm_threads(L) / L;
    __shared__ float s_sum[2][16];
    const Cols<V, P> k{static_cast<int>(threadIdx.x % L) * V, L * V, a.d};
    const float inv = 1.f / a.d;
    float dnw[P][V], dsc[P][V], dxw[P][V];
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) dnw[i][v] = dsc[i][v] = dxw[i][v] = 0.f;
    int slot = 0;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * ROWS + threadIdx.x / L;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * ROWS;
    // the next row's inputs are loaded while a row is worked on, where registers allow
    constexpr bool AHEAD = L < 1024;
    RawRow<T, V, P> nx, ngate;
    RawRow<TR, V, P> nres;
    RawRow<TGR, V, P> ndh;
    RawRow<TG, V, P> ndy;
    auto fetch = [&](int64_t row) {
        nx.load(static_cast<const T *>(a.x) + row * a.x_stride, k);
        if (a.gate) ngate.load(static_cast<const T *>(a.gate) + row * a.gate_stride, k);
        if (a.dh) ndh.load(static_cast<const TGR *>(a.dh) + row * a.d, k);
        if (a.next_weight) {
            ndy.load(static_cast<const TG *>(a.dy) + row * a.d, k);
            if (a.residual) nres.load(static_cast<const TR *>(a.residual) + row * a.d, k);
        }
    };
    if (AHEAD && first < a.rows) fetch(first);
    for (int64_t row = first; row < a.rows; row += stride) {
        // p: x through the first norm; u: through the gate; h: the new residual
        float x[P][V], p[P][V], t[P][V], g[P][V], sl[P][V], h[P][V], w[P][V];
        if (!AHEAD) fetch(row);
        nx.get(k, x);
        if (a.gate) ngate.get(k, sl);
        if (a.dh) ndh.get(k, g);
        else
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) g[i][v] = 0.f;
        if (a.next_weight) {
            ndy.get(k, w);
            if (a.residual) nres.get(k, h);
            else
#pragma unroll
                for (int i = 0; i < P; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v) h[i][v] = 0.f;
        }
        if (AHEAD && row + stride < a.rows) fetch(row + stride);
        float rx = 1.f;
        if (a.norm_weight) {
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) q = fmaf(x[i][v], x[i][v], q);
            rx = rsqrtf(row_sum<L>(q, s_sum, slot) * inv + a.eps);
            slot ^= 1;
            load_row<float>(a.norm_weight, k, t, 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) p[i][v] = x[i][v] * rx * t[i][v];
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) p[i][v] = x[i][v];
        }
        if (a.next_weight) {
            if (a.scale) load_row<float>(a.scale, k, t, 0.f);
            float q = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float u = a.gate ? p[i][v] * silu(sl[i][v]) : p[i][v];
                    if (a.scale) u *= t[i][v];
                    h[i][v] += u;
                    q = fmaf(h[i][v], h[i][v], q);
                }
            const float r = rsqrtf(row_sum<L>(q, s_sum, slot) * inv + a.eps);
            slot ^= 1;
            load_row<float>(a.next_weight, k, t, 0.f);
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    dnw[i][v] = fmaf(w[i][v], h[i][v] * r, dnw[i][v]);
                    w[i][v] *= t[i][v];
                    m = fmaf(w[i][v], h[i][v], m);
                }
            m = row_sum<L>(m, s_sum, slot) * inv * r * r;
            slot ^= 1;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) g[i][v] += r * (w[i][v] - h[i][v] * m);
        }
        if (a.dresidual) store_row<TGR>(static_cast<TGR *>(a.dresidual) + row * a.d, k, g);
        if (a.scale) {
            load_row<float>(a.scale, k, t, 0.f);
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float u = a.gate ? p[i][v] * silu(sl[i][v]) : p[i][v];
                    dsc[i][v] = fmaf(g[i][v], u, dsc[i][v]);
                    g[i][v] *= t[i][v];
                }
        }
        if (a.gate) {
            float dg[P][V];
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float s = sigmoid_hw(sl[i][v]), z = sl[i][v];
                    dg[i][v] = g[i][v] * p[i][v] * (s * fmaf(z, 1.f - s, 1.f));
                    g[i][v] *= z * s;
                }
            store_row<TG>(static_cast<TG *>(a.dgate) + row * a.d, k, dg);
        }
        if (a.norm_weight) {
            load_row<float>(a.norm_weight, k, t, 0.f);
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    dxw[i][v] = fmaf(g[i][v], x[i][v] * rx, dxw[i][v]);
                    g[i][v] *= t[i][v];
                    m = fmaf(g[i][v], x[i][v], m);
                }
            m = row_sum<L>(m, s_sum, slot) * inv * rx * rx;
            slot ^= 1;
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) g[i][v] = rx * (g[i][v] - x[i][v] * m);
        }
        store_row<TG>(static_cast<TG *>(a.dx) + row * a.d, k, g);
    }
    // [gridDim.x * ROWS][3][d]: dnorm_weight, dscale, dnext_weight
    float *part = a.partial + first * 3 * a.d;
    if (a.norm_weight) store_row<float>(part, k, dxw);
    if (a.scale) store_row<float>(part + a.d, k, dsc);
    if (a.next_weight) store_row<float>(part + 2 * static_cast<int64_t>(a.d), k, dnw);
}

// The parameter gradients: the rows of a.partial added in a fixed order. 32 columns per
// workgroup, whose 32 halves of waves each take every 32nd row. Rows of at most 128 columns leave 16
// partial rows per workgroup of the pass for few columns: of 65,536 x 128 bf16 four workgroups add
// 12,288 rows in 21 us, behind a pass of 20 us (84 MB, 16 us at a copy's rate).
__global__ __launch_bounds__(1024) void norm_reduce_kernel(NormArgs a, int parts) {
    __shared__ float s[32][33];
    const int lane = threadIdx.x & 31, half = threadIdx.x >> 5;
    const int which = blockIdx.y;
    float *out = which == 0 ? a.dnorm_weight : which == 1 ? a.dscale : a.dnext_weight;
    if (!(which == 0 ? a.norm_weight : which == 1 ? a.scale : a.next_weight)) return;
    const int col = blockIdx.x * 32 + lane;
    float sum = 0.f;
    if (col < a.d) {
        const float *p = a.partial + static_cast<int64_t>(which) * a.d + col;
#pragma unroll 8
        for (int i = half; i < parts; i += 32) sum += p[static_cast<int64_t>(i) * 3 * a.d];
    }
    s[half][lane] = sum;
    __syncthreads();
    if (half != 0 || col >= a.d) return;
#pragma unroll
    for (int i = 1; i < 32; ++i) sum += s[i][lane];
    out[col] = sum;
}

constexpr int kNormGridX = 1 << 20;
// Workgroups of a backward pass: three per CU, as many as bf16 rows' instances of 256 threads have
// there (148-168 registers). fp32 rows (170-177) have two, so that their last third runs alone.
constexpr int kNormGroups = 768;

template <typename T, typename TR, typename TG, typename TGR, int L, int V, int P>
hipError_t launch(const NormArgs &a, bool backward, hipStream_t st) {
    constexpr int THREADS = norm_threads(L), ROWS = THREADS / L;
    const int64_t sets = norm_sets(a.rows, a.d);
    if (!backward) {
        // one dimension of a grid holds less than 2^32 threads
        const unsigned gx = static_cast<unsigned>(sets < kNormGridX ? sets : kNormGridX);
        const unsigned gy = static_cast<unsigned>((sets + gx - 1) / gx);
        hipLaunchKernelGGL((norm_fwd_kernel<T, TR, L, V, P>), dim3(gx, gy), dim3(THREADS), 0, st, a);
        return hipGetLastError();
    }
    const unsigned groups = static_cast<unsigned>(sets < kNormGroups ? sets : kNormGroups);
    hipLaunchKernelGGL((norm_bwd_kernel<T, TR, TG, TGR, L, V, P>), dim3(groups), dim3(THREADS), 0, st, a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(a.norm_weight || a.scale || a.next_weight)) return e;
    hipLaunchKernelGGL(norm_reduce_kernel, dim3(static_cast<unsigned>((a.d + 31) / 32), 3), dim3(1024), 0,
                       st, a, static_cast<int>(groups) * ROWS);
    return hipGetLastError();
}

// Eight values per lane: a lane's piece of a bf16 row is one 16-byte access, and the backward's
// row-sized arrays take 148-195 registers up to 4,096 columns (value by value up to 256, with 44-76
// bytes spilled at 512 lanes), for two or three waves per SIMD. Rows above 4,096 columns take 1,024
// threads, which have 128 registers: the backward spills 84-176 bytes per lane there (value by value
// 284-320), and above 8,192 columns, where a lane has 16 values, 528-736 (968-1,040). With every
// stage and an fp32 residual the pass over 4,096 rows of 5,120 bf16 columns takes 325 us against 90
// for its bytes, 8,192 418 against 144, 16,384 1,585 against 288. The forward spills nothing.
template <typename T, typename TR, typename TG, typename TGR, int V>
hipError_t launch_rows(const NormArgs &a, bool backward, hipStream_t st) {
    constexpr int P = 8 / V;
    switch (norm_lanes(a.d)) {
    case 16: return launch<T, TR, TG, TGR, 16, V, P>(a, backward, st);
    case 64: return launch<T, TR, TG, TGR, 64, V, P>(a, backward, st);
    case 128: return launch<T, TR, TG, TGR, 128, V, P>(a, backward, st);
    case 256: return launch<T, TR, TG, TGR, 256, V, P>(a, backward, st);
    case 512: return launch<T, TR, TG, TGR, 512, V, P>(a, backward, st);
    default:
        return a.d <= 8192 ? launch<T, TR, TG, TGR, 1024, V, P>(a, backward, st)
                           : launch<T, TR, TG, TGR, 1024, V, 2 * P>(a, backward, st);
    }
}

bool al16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

template <typename T, typename TR, typename TG, typename TGR>
hipError_t launch_types(const NormArgs &a, bool backward, hipStream_t st) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
    const bool vec = a.d % V == 0 && a.x_stride % V == 0 && (!a.gate || a.gate_stride % V == 0) &&
                     al16(a.x) && al16(a.gate) && al16(a.residual) && al16(a.h) && al16(a.y) &&
                     al16(a.dh) && al16(a.dy) && al16(a.dx) && al16(a.dgate) && al16(a.dresidual) &&
                     al16(a.norm_weight) && al16(a.scale) && al16(a.next_weight);
    return vec ? launch_rows<T, TR, TG, TGR, V>(a, backward, st) : launch_rows<T, TR, TG, TGR, 1>(a, backward, st);
}

}  // namespace

int norm_lanes(int d) {
    return d <= 128 ? 16 : d <= 512 ? 64 : d <= 1024 ? 128 : d <= 2048 ? 256 : d <= 4096 ? 512 : 1024;
}

int64_t norm_sets(int64_t rows, int d) {
    const int l = norm_lanes(d), per = norm_threads(l) / l;
    const int64_t sets = (rows + per - 1) / per;
    return sets > 1 ? sets : 1;
}

int64_t norm_parts(int64_t rows, int d) {
    const int l = norm_lanes(d), per = norm_threads(l) / l;
    const int64_t sets = norm_sets(rows, d);
    return (sets < kNormGroups ? sets : kNormGroups) * per;
}

hipError_t launch_norm(const NormArgs &a, bool backward, hipStream_t st) {
    if (!a.bf16) return launch_types<float, float, float, float>(a, backward, st);
    if (a.residual_f32)       // a residual stream in fp32, and its gradients
        return a.grad_bf16 ? launch_types<bf16_t, float, bf16_t, float>(a, backward, st)
                           : launch_types<bf16_t, float, float, float>(a, backward, st);
    return a.grad_bf16 ? launch_types<bf16_t, bf16_t, bf16_t, bf16_t>(a, backward, st)
                       : launch_types<bf16_t, bf16_t, float, float>(a, backward, st);
}

}  // namespace gdn2
