// gdn2_rotary.hip -- norms of queries and keys per head with the rotation by position in one pass,
// into plain tensors or into the pages of a cache, and their gradients.
//
// Per token at position p and per head, with r = 1 / sqrt(mean(x^2) + eps) and R = d_rot:
//     y = x r w,   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)  for the R/2 pairs (a, b),
// c and s the cosine and sine of the pair's angle at p, taken from a table; pairs are (i, i + R/2)
// or (2i, 2i + 1), values from R on stay. Without w there is no norm. Gradients, from g = dy turned
// back by the same angles (a rotation's transpose):
//     dw = sum over tokens and heads of g x r,     dx = r (g w - x r^2 mean(g w x)).
//
// Bound by memory (every value is read once and written once), the forward as much by the vector unit:
// at 4,096 x 20 bf16 heads of 128 that issues in 83 % of the busy cycles, 11 us. A head's row lives in
// the registers of L lanes. A lane holds P units of 2 V values, the two members of V pairs (V neighbours each, so
// a unit is two accesses of up to 16 bytes), and the rotation needs no exchange between lanes; the
// values that are not rotated are cut into pairs in the same way. A wave takes a token's heads,
// 64 / L at a time, with the token's cosines and sines and the weights in registers. Sums and
// rotation are fp32, rounded once at the store.
#include <initializer_list>

#include "gdn2_internal.h"
#include "gdn2_layer.h"

namespace gdn2 {

namespace {

// Where a lane's units lie in a row: unit u = lane + i L holds values a(u) .. a(u) + V - 1 and
// b(u) .. b(u) + V - 1, whose angles are the table's columns pair(u) .. pair(u) + V - 1. INTER: pairs
// (2i, 2i + 1), a unit being 2 V neighbours.
template <int V, int L, int P, bool INTER>
struct Units {
    int lane, half, rest;        // half = R / 2; rest = (d - R) / 2
    __device__ __forceinline__ explicit Units(const RotaryArgs &r)
        : lane(static_cast<int>(threadIdx.x) % L), half(r.d_rot / 2), rest((r.d - r.d_rot) / 2) {}
    __device__ __forceinline__ int pair(int i) const { return (lane + i * L) * V; }
    __device__ __forceinline__ bool in(int i) const { return pair(i) < half + rest; }
    __device__ __forceinline__ bool turns(int i) const { return pair(i) < half; }
    __device__ __forceinline__ int a(int i) const {
        return INTER ? 2 * pair(i) : turns(i) ? pair(i) : half + pair(i);
    }
    __device__ __forceinline__ int b(int i) const {
        return INTER ? 2 * pair(i) + V : turns(i) ? half + pair(i) : half + rest + pair(i);
    }
};

// The two members of a lane's pairs: x[i][0][v] and x[i][1][v].
template <int V, int P>
using Pairs = float[P][2][V];

// Two runs of V neighbours, as they are in memory, into members: in the interleaved order member m
// of pair v is value 2 v + m of both runs together.
template <int V, bool INTER>
__device__ __forceinline__ void to_members(const float (&lo)[V], const float (&hi)[V], float (&x)[2][V]) {
#pragma unroll
    for (int v = 0; v < V; ++v) {
        x[0][v] = !INTER ? lo[v] : 2 * v < V ? lo[2 * v % V] : hi[2 * v % V];
        x[1][v] = !INTER ? hi[v] : 2 * v + 1 < V ? lo[(2 * v + 1) % V] : hi[(2 * v + 1) % V];
    }
}

template <typename T, int V, int L, int P, bool INTER>
__device__ __forceinline__ void load_pairs(const T *row, const Units<V, L, P, INTER> &k, Pairs<V, P> &x) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        float lo[V] = {}, hi[V] = {};
        if (k.in(i)) {
            ldv<T, V>(row + k.a(i), lo);
            ldv<T, V>(row + k.b(i), hi);
        }
        to_members<V, INTER>(lo, hi, x[i]);
    }
}

template <typename T, int V, int L, int P, bool INTER>
__device__ __forceinline__ void store_pairs(T *row, const Units<V, L, P, INTER> &k, const Pairs<V, P> &x) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        float lo[V], hi[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            lo[v] = INTER ? x[i][v & 1][v / 2] : x[i][0][v];
            hi[v] = INTER ? x[i][(V + v) & 1][(V + v) / 2] : x[i][1][v];
        }
        if (k.in(i)) {
            stv<T, V>(row + k.a(i), lo);
            stv<T, V>(row + k.b(i), hi);
        }
    }
}

// The same loads in two steps: what is in memory now, its members when they are used.
template <typename T, int V, int P>
struct RawPairs {
    Raw<T, V> lo[P], hi[P];
    template <int L, bool INTER>
    __device__ __forceinline__ void load(const T *row, const Units<V, L, P, INTER> &k) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (k.in(i)) {
                lo[i].load(row + k.a(i));
                hi[i].load(row + k.b(i));
            }
    }
    template <int L, bool INTER>
    __device__ __forceinline__ void get(const Units<V, L, P, INTER> &k, bool used, Pairs<V, P> &x) const {
#pragma unroll
        for (int i = 0; i < P; ++i) {
            float a[V], b[V];
            lo[i].get(a);
            hi[i].get(b);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                a[v] = used && k.in(i) ? a[v] : 0.f;
                b[v] = used && k.in(i) ? b[v] : 0.f;
            }
            to_members<V, INTER>(a, b, x[i]);
        }
    }
};

// Cosines and sines of a lane's pairs; 1 and 0 where nothing turns.
template <int V, int L, int P, bool INTER>
__device__ __forceinline__ void load_turn(const float *row, const Units<V, L, P, INTER> &k, bool used, Pairs<V, P> &t) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
        if (used && k.turns(i)) {
            ldv<float, V>(row + k.pair(i), t[i][0]);
            ldv<float, V>(row + k.half + k.pair(i), t[i][1]);
        } else {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                t[i][0][v] = 1.f;
                t[i][1][v] = 0.f;
            }
        }
    }
}

// Sum over the L lanes of a row.
template <int L>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int m = 1; m < L; m <<= 1) x += __shfl_xor(x, m);
    return x;
}

template <int V, int P>
__device__ __forceinline__ float dot(const Pairs<V, P> &x, const Pairs<V, P> &y) {
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int v = 0; v < V; ++v) s = fmaf(x[i][0][v], y[i][0][v], fmaf(x[i][1][v], y[i][1][v], s));
    return s;
}

// The row of cos_sin of a token, or a negative number for padding.
__device__ __forceinline__ int position_of(const RotaryArgs &a, int token) {
    const int p = a.positions ? a.positions[token] : token % a.seqlen;
    return p >= 0 && (p < a.num_positions || a.d_rot == 0) ? p : -1;
}

// The rows that a wave takes at once: 64 / L of them, a.row_heads heads of as many tokens as that leaves
// room for. They come in sets: all heads of q, then of k, then (in front of a cache) of v.
template <int L>
struct Rows {
    int head, token;             // the lane's first head, and its token among the wave's
    int sets_q, sets;
    __device__ __forceinline__ explicit Rows(const RotaryArgs &a) {
        const int row = (threadIdx.x & 63) / L;
        head = row & (a.row_heads - 1);
        token = row / a.row_heads;
        sets_q = (a.h_q + a.row_heads - 1) / a.row_heads;
        sets = sets_q + (a.slots ? 2 : 1) * ((a.h_k + a.row_heads - 1) / a.row_heads);
    }
    static __device__ __forceinline__ int tokens(const RotaryArgs &a) { return 64 / L / a.row_heads; }
};

// A wave takes its tokens and every gridDim.y-th set of their rows; v is copied.
template <typename T, int V, int L, int P, bool INTER>
__global__ __launch_bounds__(256) void rotary_fwd_kernel(RotaryArgs a) {
    const Rows<L> rows(a);
    const int64_t block = static_cast<int64_t>(blockIdx.z) * gridDim.x + blockIdx.x;
    const int64_t token = (block * 4 + (threadIdx.x >> 6)) * Rows<L>::tokens(a) + rows.token;
    const bool real = token < a.tokens;
    const Units<V, L, P, INTER> k(a);
    const int at = real ? position_of(a, static_cast<int>(token)) : -1;
    Pairs<V, P> turn;
    load_turn<V, L, P, INTER>(a.cos_sin + static_cast<int64_t>(at) * a.d_rot, k, at >= 0, turn);
    int64_t place = -1, page = 0;
    int within = 0;
    if (a.slots && at >= 0) {
        place = a.slots[token];
        if (place >= a.num_places) place = -1;
        page = place / a.page_size;
        within = static_cast<int>(place % a.page_size);
    }
    const int sets_k = rows.sets_q + (a.h_k + a.row_heads - 1) / a.row_heads;      // where k's sets end
    for (int set = blockIdx.y; set < rows.sets; set += gridDim.y) {
        const int kind = set < rows.sets_q ? 0 : set < sets_k ? 1 : 2;
        const int head = (set - (kind == 0 ? 0 : kind == 1 ? rows.sets_q : sets_k)) * a.row_heads + rows.head;
        const int heads = kind == 0 ? a.h_q : a.h_k;
        const bool cached = kind && a.slots;
        const bool mine = real && head < heads && !(cached && place < 0);
        const T *src = static_cast<const T *>(kind == 0 ? a.q : kind == 1 ? a.k : a.v) +
                       token * (kind == 0 ? a.q_stride : kind == 1 ? a.k_stride : a.v_stride) +
                       static_cast<int64_t>(head) * a.d;
        T *dst = static_cast<T *>(kind == 0 ? a.q_out : kind == 1 ? a.k_out : a.v_out) +
                 (cached ? (page * a.h_k + head) * a.page_size + within : token * heads + head) * a.d;
        Pairs<V, P> x;
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) x[i][0][v] = x[i][1][v] = 0.f;
        if (mine && at >= 0) load_pairs<T, V, L, P, INTER>(src, k, x);
        if (kind < 2) {
            const float *weight = kind == 0 ? a.q_weight : a.k_weight;
            if (weight) {
                Pairs<V, P> w;
                load_pairs<float, V, L, P, INTER>(weight, k, w);
                const float r = rsqrtf(lanes_sum<L>(dot<V, P>(x, x)) * a.inv_d + a.eps);
#pragma unroll
                for (int i = 0; i < P; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        x[i][0][v] *= r * w[i][0][v];
                        x[i][1][v] *= r * w[i][1][v];
                    }
            }
            if (at < 0) {        // (0 / 0 with an eps of 0)
#pragma unroll
                for (int i = 0; i < P; ++i)
#pragma unroll
                    for (int v = 0; v < V; ++v) x[i][0][v] = x[i][1][v] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float c = turn[i][0][v], s = turn[i][1][v], p = x[i][0][v], q = x[i][1][v];
                    // (what does not turn is kept as it is: 0 * an infinite partner would be NaN)
                    x[i][0][v] = k.turns(i) ? fmaf(p, c, -q * s) : p;
                    x[i][1][v] = k.turns(i) ? fmaf(q, c, p * s) : q;
                }
        }
        if (mine) store_pairs<T, V, L, P, INTER>(dst, k, x);
    }
}

// A wave takes its tokens, then those 4 gridDim.x waves on, with every gridDim.y-th set of their rows one
// after the other, the next set's rows under way while one is worked on. It keeps its columns' sums of the
// weights' gradients in registers; a workgroup's leave as one row of a.partial, [2][d].
template <typename T, typename TG, int V, int L, int P, bool INTER>
__global__ __launch_bounds__(256, 3) void rotary_bwd_kernel(RotaryArgs a) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const Rows<L> rows(a);
    const Units<V, L, P, INTER> k(a);
    const int per = Rows<L>::tokens(a);
    const int64_t first = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * per + rows.token;
    const int64_t stride = static_cast<int64_t>(gridDim.x) * 4 * per;
    Pairs<V, P> dw[2];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int v = 0; v < V; ++v) dw[n][i][0][v] = dw[n][i][1][v] = 0.f;

    RawPairs<T, V, P> nx;
    RawPairs<TG, V, P> ng;
    Pairs<V, P> turn, nturn;
    // the rows of a set of the tokens, if they are there
    auto fetch = [&](int64_t token, bool real, int set) {
        const int kind = set < rows.sets_q ? 0 : 1, heads = kind ? a.h_k : a.h_q;
        const int head = (set - (kind ? rows.sets_q : 0)) * a.row_heads + rows.head;
        if (!real || head >= heads) return;
        ng.load(static_cast<const TG *>(kind ? a.dk_out : a.dq_out) + (token * heads + head) * a.d, k);
        if (kind ? a.k_weight : a.q_weight)
            nx.load(static_cast<const T *>(kind ? a.k : a.q) + token * (kind ? a.k_stride : a.q_stride) +
                        static_cast<int64_t>(head) * a.d, k);
    };
    const int set0 = blockIdx.y, sets_on = gridDim.y;
    int at = first < a.tokens ? position_of(a, static_cast<int>(first)) : -1;
    load_turn<V, L, P, INTER>(a.cos_sin + static_cast<int64_t>(at) * a.d_rot, k, at >= 0, turn);
    fetch(first, at >= 0, set0);
    for (int64_t base = 0; first - rows.token + base < a.tokens; base += stride) {
        const int64_t token = first + base, next = token + stride;
        const bool real = token < a.tokens;
        const int next_at = next < a.tokens ? position_of(a, static_cast<int>(next)) : -1;
        for (int set = set0; set < rows.sets; set += sets_on) {
            const int kind = set < rows.sets_q ? 0 : 1, heads = kind ? a.h_k : a.h_q;
            const int head = (set - (kind ? rows.sets_q : 0)) * a.row_heads + rows.head;
            const bool mine = real && head < heads, used = mine && at >= 0;
            const float *weight = kind ? a.k_weight : a.q_weight;
            Pairs<V, P> g, x;
            ng.get(k, used, g);
            if (weight) nx.get(k, used, x);
            const bool last = set + sets_on >= rows.sets;
            fetch(last ? next : token, last ? next_at >= 0 : at >= 0, last ? set0 : set + sets_on);
            if (last) load_turn<V, L, P, INTER>(a.cos_sin + static_cast<int64_t>(next_at) * a.d_rot, k, next_at >= 0, nturn);
#pragma unroll
            for (int i = 0; i < P; ++i)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float c = turn[i][0][v], s = turn[i][1][v], p = g[i][0][v], q = g[i][1][v];
                    g[i][0][v] = k.turns(i) ? fmaf(p, c, q * s) : p;
                    g[i][1][v] = k.turns(i) ? fmaf(q, c, -p * s) : q;
                }
            if (weight) {
                Pairs<V, P> w;
                load_pairs<float, V, L, P, INTER>(weight, k, w);
                // (a row that is not there has a sum of 0, and no gradient even with an eps of 0)
                const float r = used ? rsqrtf(lanes_sum<L>(dot<V, P>(x, x)) * a.inv_d + a.eps) : 0.f;
#pragma unroll
                for (int i = 0; i < P; ++i)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            const float e = g[i][m][v] * (x[i][m][v] * r);
                            if (kind) dw[1][i][m][v] += e;
                            else dw[0][i][m][v] += e;
                            g[i][m][v] *= w[i][m][v];
                        }
                const float mean = lanes_sum<L>(dot<V, P>(g, x)) * a.inv_d * r * r;
#pragma unroll
                for (int i = 0; i < P; ++i)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int v = 0; v < V; ++v) g[i][m][v] = r * (g[i][m][v] - x[i][m][v] * mean);
            }
            if (mine)
                store_pairs<TG, V, L, P, INTER>(static_cast<TG *>(kind ? a.dk : a.dq) + (token * heads + head) * a.d, k, g);
        }
        at = next_at;
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int v = 0; v < V; ++v) turn[i][m][v] = nturn[i][m][v];
    }
    if (!a.q_weight && !a.k_weight) return;
    // the lanes that hold the same columns, then the four waves
    __shared__ float s_sum[4][2 * 512];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float x = dw[n][i][m][v];
#pragma unroll
                    for (int s = L; s < 64; s <<= 1) x += __shfl_xor(x, s);
                    dw[n][i][m][v] = x;
                }
    if (lane < L)
#pragma unroll
        for (int n = 0; n < 2; ++n) store_pairs<float, V, L, P, INTER>(s_sum[wave] + n * a.d, k, dw[n]);
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * a.d; c += 256)
        a.partial[(static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * 2 * a.d + c] =
            (s_sum[0][c] + s_sum[1][c]) + (s_sum[2][c] + s_sum[3][c]);
}

// The weights' gradients: the rows of a.partial added in a fixed order, 16 columns per workgroup. Lane
// l of wave w takes rows 4 w + l / 16, 64 on and so forth of column l % 16; then the four rows of a wave
// are added by exchanges, and the 16 waves in the first one.
constexpr int kReduceCols = 16;
__global__ __launch_bounds__(1024) void rotary_reduce_kernel(RotaryArgs a, int parts) {
    __shared__ float s[16][kReduceCols];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = lane % kReduceCols;
    const int col = blockIdx.x * kReduceCols + c;
    float sum = 0.f;
    if (col < 2 * a.d)
#pragma unroll 8
        for (int i = threadIdx.x / kReduceCols; i < parts; i += 64) sum += a.partial[static_cast<int64_t>(i) * 2 * a.d + col];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (lane < kReduceCols) s[wave][c] = sum;
    __syncthreads();
    if (wave != 0) return;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) sum += s[lane / kReduceCols * 4 + i][c];
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (lane >= kReduceCols || col >= 2 * a.d) return;
    if (col < a.d) {
        if (a.q_weight) a.dq_weight[col] = sum;
    } else if (a.k_weight) {
        a.dk_weight[col - a.d] = sum;
    }
}

// Waves that fill the chip. A call of fewer gives the sets of a token's rows to waves of their own
// (forward: 64 tokens x 20 heads of 256 into pages 8.6 -> 3.9 us; gradients of 584 x (66 + 11) fp32
// heads of 256 48 -> 27), and heads of several tokens go side by side only above that (16,384 x (16 + 4)
// of 64: gradients 37.5 -> 30.3).
constexpr int kRotaryWaves = 4096;

int next_pow2(int x) {
    int p = 1;
    while (p < x) p *= 2;
    return p;
}

// Heads of a token that a wave takes at once, of the `rows` that it has room for. As many as there are
// leaves places empty where the last set of q or of k is not full (16 and 4 heads in sets of 16); with
// enough tokens for all workgroups, the number that leaves the fewest empty.
int heads_at_once(const RotaryArgs &a, int rows) {
    const int most = next_pow2(a.h_q > a.h_k ? a.h_q : a.h_k);
    int best = most < rows ? most : rows;
    auto taken = [&](int n) { return (a.h_q + n - 1) / n * n + (a.h_k + n - 1) / n * n; };
    for (int n = best / 2; n >= 1; n /= 2)
        if (taken(n) < taken(best) && a.tokens / (rows / n) >= kRotaryWaves) best = n;
    return best;
}

template <typename T, typename TG, int V, int L, int P, bool INTER>
hipError_t launch(RotaryArgs a, bool backward, hipStream_t st) {
    a.row_heads = heads_at_once(a, 64 / L);
    a.inv_d = 1.f / a.d;
    const int per = 4 * (64 / L / a.row_heads);          // tokens of a workgroup
    const int groups = a.tokens / per + (a.tokens % per != 0);
    const int sets = (a.h_q + a.row_heads - 1) / a.row_heads + (a.slots ? 2 : 1) * ((a.h_k + a.row_heads - 1) / a.row_heads);
    auto split = [&](int n) { return n < 1 ? 1 : n < sets ? n : sets; };
    if (!backward) {
        // one dimension of a grid holds less than 2^32 threads
        const unsigned gx = static_cast<unsigned>(groups < (1 << 20) ? groups : 1 << 20);
        const unsigned gy = static_cast<unsigned>(split(kRotaryWaves / (4 * groups)));
        const unsigned gz = (static_cast<unsigned>(groups) + gx - 1) / gx;
        hipLaunchKernelGGL((rotary_fwd_kernel<T, V, L, P, INTER>), dim3(gx, gy, gz), dim3(256), 0, st, a);
        return hipGetLastError();
    }
    // as many as run at once: instances of eight values per access have 161-168 registers, others 96-122
    constexpr int AT_ONCE = V == 8 ? 3 * 256 : kRotaryParts;
    const int gx = groups < 1 ? 1 : groups < AT_ONCE ? groups : AT_ONCE, gy = split(AT_ONCE / gx);
    hipLaunchKernelGGL((rotary_bwd_kernel<T, TG, V, L, P, INTER>), dim3(gx, gy), dim3(256), 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !(a.q_weight || a.k_weight)) return e;
    hipLaunchKernelGGL(rotary_reduce_kernel, dim3((2 * a.d + kReduceCols - 1) / kReduceCols), dim3(1024), 0, st, a,
                       gx * gy);
    return hipGetLastError();
}

template <typename T, typename TG, int V, bool INTER>
hipError_t launch_rows(const RotaryArgs &a, bool backward, hipStream_t st) {
    const int units = a.d / (2 * V);
    if constexpr (V <= 2) {
        if (units <= 64 / V) return launch<T, TG, V, 16, 4 / V, INTER>(a, backward, st);
        return launch<T, TG, V, 64, 4 / V, INTER>(a, backward, st);
    } else {
        if (units <= 4) return launch<T, TG, V, 4, 1, INTER>(a, backward, st);
        if (units <= 8) return launch<T, TG, V, 8, 1, INTER>(a, backward, st);
        if (units <= 16) return launch<T, TG, V, 16, 1, INTER>(a, backward, st);
        if (units <= 32) return launch<T, TG, V, 32, 1, INTER>(a, backward, st);
        return launch<T, TG, V, 64, 1, INTER>(a, backward, st);
    }
}

// Whether every run of V pairs' members can be taken in whole accesses, at most 16 bytes each.
bool whole(const RotaryArgs &a, int V) {
    const int half = a.d_rot / 2, rest = (a.d - a.d_rot) / 2;
    uintptr_t low = 0;
    for (const void *p : {a.q, a.k, a.v, static_cast<const void *>(a.cos_sin), static_cast<const void *>(a.q_weight),
                          static_cast<const void *>(a.k_weight), static_cast<const void *>(a.q_out),
                          static_cast<const void *>(a.k_out), static_cast<const void *>(a.v_out), a.dq_out, a.dk_out,
                          static_cast<const void *>(a.dq), static_cast<const void *>(a.dk)})
        low |= reinterpret_cast<uintptr_t>(p);
    return half % V == 0 && rest % V == 0 && a.q_stride % V == 0 && a.k_stride % V == 0 && a.v_stride % V == 0 &&
           low % (V == 2 ? 8 : 16) == 0;
}

template <typename T, typename TG, bool INTER>
hipError_t launch_types(const RotaryArgs &a, bool backward, hipStream_t st) {
    constexpr int V = sizeof(T) == 2 ? 8 : 4;
    if (whole(a, V)) return launch_rows<T, TG, V, INTER>(a, backward, st);
    return whole(a, 2) ? launch_rows<T, TG, 2, INTER>(a, backward, st) : launch_rows<T, TG, 1, INTER>(a, backward, st);
}

template <typename T, typename TG>
hipError_t launch_types(const RotaryArgs &a, bool backward, hipStream_t st) {
    return a.interleaved ? launch_types<T, TG, true>(a, backward, st) : launch_types<T, TG, false>(a, backward, st);
}

}  // namespace

hipError_t launch_rotary(const RotaryArgs &a, hipStream_t st) {
    return a.bf16 ? launch_types<bf16_t, bf16_t>(a, false, st) : launch_types<float, float>(a, false, st);
}

hipError_t launch_rotary_bwd(const RotaryArgs &a, hipStream_t st) {
    if (!a.bf16) return launch_types<float, float>(a, true, st);
    return a.grad_bf16 ? launch_types<bf16_t, bf16_t>(a, true, st) : launch_types<bf16_t, float>(a, true, st);
}

}  // namespace gdn2
