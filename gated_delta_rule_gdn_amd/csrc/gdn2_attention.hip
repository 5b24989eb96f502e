// gdn2_attention.hip -- attention of the newest tokens of every sequence over a paged cache.
//
// The rows of one key head are its T new tokens times the G query heads that read it, row r being
// token r / G. For a row at place p and the keys j that it sees,
//     o = sum_j e^(s_j - m) v_j / l,   m = max_j s_j,   l = sum_j e^(s_j - m),   s_j = scale q . k_j
// in one pass over the keys: m, l and the unnormalised o are kept and rescaled when m grows, and
// parts of a sequence (m, l, o) join the same way. Exponentials are taken to base 2.
//
// Bound by memory: every key and value is read once for all rows of its head. Each of the two
// products is made on the matrix cores, 16 rows at a time, with the cache in registers only:
//   S^T = K Q^T    A operand: 16 keys, a lane 8 (fp32: 4) neighbouring values of its key's row
//   O^T = V^T P^T  B operand: the output tiles of S^T as they are (their rows are the keys); A
//                  operand: a lane loads the rows of the 8 (fp32: 4) keys whose scores it holds,
//                  VE neighbouring values of each, so that value j of every row makes the operand
//                  of product j (its 16 rows are the values j, VE + j, 2 VE + j ...)
// so neither operand goes through LDS. The four waves of a workgroup take every fourth tile of keys
// of its part of a sequence and join at its end; a second kernel joins the parts.
#include "gdn2_internal.h"
#include "gdn2_layer.h"
#include "gdn2_mfma.h"

namespace gdn2 {

namespace {

constexpr int kWaves = 4;

// Workgroups that a call is cut into, about, and steps (a tile per wave) below which a part is not cut.
constexpr int kTargetGroups = 1024;
constexpr int kLeastSteps = 4;

__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) x += __shfl_xor(x, m);
    return x;
}

__device__ __forceinline__ int seq_len(const AttentionArgs &a, int n) {
    const int most = a.max_pages * a.page_size, len = a.seq_lens[n];
    return len < 0 ? 0 : len > most ? most : len;
}

// Steps of a workgroup (kWaves tiles) over the places that a sequence's new tokens see.
template <int KT>
__device__ __forceinline__ int seq_steps(const AttentionArgs &a, int len) {
    const int64_t first = static_cast<int64_t>(len) - a.new_tokens - a.window + 1;
    const int lo = a.window > 0 && first > 0 ? static_cast<int>(first) / KT * KT : 0;
    return (len - lo + kWaves * KT - 1) / (kWaves * KT);
}

// Steps of a part: all parts together come to at most groups / heads + num_seqs.
template <int KT>
__device__ __forceinline__ int part_steps(const AttentionArgs &a, int heads) {
    const int lane = threadIdx.x & 63;
    int64_t all = 0;
    for (int base = 0; base < a.num_seqs; base += 64)
        if (base + lane < a.num_seqs) all += seq_steps<KT>(a, seq_len(a, base + lane));
#pragma unroll
    for (int m = 1; m < 64; m <<= 1) all += __shfl_xor(all, m);
    const int64_t per = (all * heads + kTargetGroups - 1) / kTargetGroups;
    return per > kLeastSteps ? static_cast<int>(per) : kLeastSteps;
}

__device__ __forceinline__ int num_parts(int steps, int per) {
    const int n = (steps + per - 1) / per;
    return n > 1 ? n : 1;
}

// A part of a sequence: number `part` of `parts`, of which `before` belong to earlier sequences.
struct Part {
    int n, part, parts, before;
};

// The sequence that holds part `id`, or n < 0 behind the last.
template <int KT>
__device__ __forceinline__ Part find_part(const AttentionArgs &a, int per, int id) {
    const int lane = threadIdx.x & 63;
    int before = 0;
    for (int base = 0; base < a.num_seqs; base += 64) {
        const int mine = base + lane < a.num_seqs ? num_parts(seq_steps<KT>(a, seq_len(a, base + lane)), per) : 0;
        int sum = mine;                              // inclusive sum over the lanes
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const int x = __shfl_up(sum, m);
            if (lane >= m) sum += x;
        }
        const uint64_t hit = __ballot(mine > 0 && id < before + sum);
        if (hit) {
            const int l = __ffsll(static_cast<unsigned long long>(hit)) - 1;
            const int parts = __shfl(mine, l), first = before + __shfl(sum, l) - parts;
            return Part{base + l, id - first, parts, first};
        }
        before += __shfl(sum, 63);
    }
    return Part{-1, 0, 0, 0};
}

// Weights of keys as B operands of the second product. bf16 holds a weight as the sum of two (8 bits
// each, 2^-17 of the weight off at most): one alone would put an error of the size of the output's
// own rounding into every weight.
template <typename O>
struct Split {
    O hi, lo;
};
__device__ __forceinline__ f32x4 rest_of(f32x4 p, uint32_t a, uint32_t b) {
    return f32x4{p.x - bf16_lo(a), p.y - bf16_hi(a), p.z - bf16_lo(b), p.w - bf16_hi(b)};
}
__device__ __forceinline__ Split<u32x4> operand(const f32x4 (&p)[2], bf16_t) {
    const u32x4 hi = dpair_to_b32(p[0], p[1]);
    return Split<u32x4>{hi, dpair_to_b32(rest_of(p[0], hi.x, hi.y), rest_of(p[1], hi.z, hi.w))};
}
__device__ __forceinline__ Split<u32x2> operand(const f32x4 (&p)[1], bf16_t) {
    const u32x2 hi = f4_to_b16(p[0]);
    return Split<u32x2>{hi, f4_to_b16(rest_of(p[0], hi.x, hi.y))};
}
__device__ __forceinline__ f32x4 operand(const f32x4 (&p)[1], float) { return p[0]; }

// Keys of a tile: what a wave holds of keys and values at once, 64 registers (fp32 of 256 values: 128).
template <typename T> constexpr int tile_keys(int d) { return sizeof(T) == 2 && d <= 128 ? 32 : 16; }

// Waves per SIMD that the registers are held to.
template <typename T, int D, int MT> constexpr int waves_per_simd() {
    return sizeof(T) == 4 && D == 256 ? 1 : D == 128 && MT == 1 ? 3 : 2;
}

// The first product: QW values of a head per operand of a lane's 16 bytes.
template <typename T> struct Ops;
template <> struct Ops<bf16_t> {
    static constexpr int QW = 32;
    typedef u32x4 Frag;                          // 8 values of a q or k row
    static __device__ __forceinline__ f32x4 qk(Frag k, Frag q, f32x4 c) { return mma_k32(k, q, c); }
    static __device__ __forceinline__ Frag each(const bf16_t *p) {      // value by value
        Frag f;
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = p[2 * i].bits | static_cast<uint32_t>(p[2 * i + 1].bits) << 16;
        return f;
    }
};
template <> struct Ops<float> {
    static constexpr int QW = 16;
    typedef f32x4 Frag;
    static __device__ __forceinline__ f32x4 qk(Frag k, Frag q, f32x4 c) { return mma_k16_f32(k, q, c); }
    static __device__ __forceinline__ Frag each(const float *p) { return Frag{p[0], p[1], p[2], p[3]}; }
};

// Rows of v that a lane holds: VR keys, VE neighbouring values of each of S sets of 16 VE values.
template <typename T, int D> struct VRows;

template <int D> struct VRows<bf16_t, D> {
    static constexpr int VR = tile_keys<bf16_t>(D) / 4, VE = D < 128 ? D / 16 : 8, S = D / (16 * VE), W = VE / 2;
    typedef uint32_t words __attribute__((ext_vector_type(W)));
    typedef uint32_t Oper __attribute__((ext_vector_type(VR / 2)));
    typedef Split<Oper> Weights;
    words w[VR][S];
    __device__ __forceinline__ void load(int r, const bf16_t *row, int li) {
#pragma unroll
        for (int s = 0; s < S; ++s) w[r][s] = *reinterpret_cast<const words *>(row + (s * 16 + li) * VE);
    }
    __device__ __forceinline__ bool finite() const {
        bool f = true;
#pragma unroll
        for (int r = 0; r < VR; ++r)
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < W; ++i)
                    f &= (w[r][s][i] & 0x7f80u) != 0x7f80u && (w[r][s][i] & 0x7f800000u) != 0x7f800000u;
        return f;
    }
    // the key of a lane's row r within the tile: those of the output tiles' rows
    static __device__ __forceinline__ int key(int lg, int r) { return perm_k<true>(lg, r); }
    // bits of the operand that belong to row r, if it is seen
    static __device__ __forceinline__ void see(int r, bool seen, Oper &bits) {
        if (r % 2 == 0) bits[r / 2] = 0;
        if (seen) bits[r / 2] |= r % 2 ? 0xffff0000u : 0xffffu;
    }
    static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) { return mma_k32(a, b, c); }
    static __device__ __forceinline__ f32x4 mma(u32x2 a, u32x2 b, f32x4 c) { return mma_k16_bf16(a, b, c); }
    // o += V^T P^T for value j of set s, of the rows in `bits`
    __device__ __forceinline__ f32x4 pv(int s, int j, const Weights &p, f32x4 o, const Oper *bits = nullptr) const {
        Oper v;
#pragma unroll
        for (int i = 0; i < VR / 2; ++i)      // the same half of two rows' words
            v[i] = __builtin_amdgcn_perm(w[2 * i + 1][s][j / 2], w[2 * i][s][j / 2], j % 2 ? 0x07060302u : 0x05040100u);
        if (bits) v &= *bits;
        return mma(v, p.lo, mma(v, p.hi, o));
    }
};

template <int D> struct VRows<float, D> {
    static constexpr int VR = 4, VE = 4, S = D / 64;
    typedef u32x4 Oper;
    typedef f32x4 Weights;
    f32x4 w[VR][S];
    __device__ __forceinline__ void load(int r, const float *row, int li) {
#pragma unroll
        for (int s = 0; s < S; ++s) w[r][s] = *reinterpret_cast<const f32x4 *>(row + (s * 16 + li) * VE);
    }
    __device__ __forceinline__ bool finite() const {
        bool f = true;
#pragma unroll
        for (int r = 0; r < VR; ++r)
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int i = 0; i < 4; ++i) f &= (__float_as_uint(w[r][s][i]) & 0x7f800000u) != 0x7f800000u;
        return f;
    }
    static __device__ __forceinline__ int key(int lg, int r) { return 4 * lg + r; }
    static __device__ __forceinline__ void see(int r, bool seen, u32x4 &bits) { bits[r] = seen ? ~0u : 0u; }
    __device__ __forceinline__ f32x4 pv(int s, int j, f32x4 p, f32x4 o, const u32x4 *bits = nullptr) const {
        f32x4 v = {w[0][s][j], w[1][s][j], w[2][s][j], w[3][s][j]};
        if (bits) v = __builtin_bit_cast(f32x4, __builtin_bit_cast(u32x4, v) & *bits);
        return mma_k16_f32(v, p, o);
    }
};

template <typename T, int D, int MT>
__global__ __launch_bounds__(64 * kWaves, (waves_per_simd<T, D, MT>())) void paged_attention_kernel(AttentionArgs a, int row_blocks) {
    using Op = Ops<T>;
    using V = VRows<T, D>;
    constexpr int KT = tile_keys<T>(D), ST = KT / 16, QF = D / Op::QW, ROWS = 16 * MT;
    constexpr int LV = 16 / sizeof(T);           // values of a 16-byte access
    typedef typename Op::Frag Frag;
    __shared__ Frag s_q[MT * QF * 64];
    __shared__ float s_ml[kWaves][2][ROWS];
    __shared__ f32x4 s_o[2][V::S * V::VE * 64];
    const int lane = threadIdx.x & 63, lg = lane >> 4, li = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int heads = a.h_k * row_blocks;
    const int sub = static_cast<int>(blockIdx.x % heads), h = sub / row_blocks, rb = sub % row_blocks;
    const int G = a.h_q / a.h_k, R = a.new_tokens * G;
    const int per = part_steps<KT>(a, heads);
    const Part part = find_part<KT>(a, per, static_cast<int>(blockIdx.x / heads));
    if (part.n < 0) return;
    const int len = seq_len(a, part.n);

    // the places that this workgroup's rows see: row r those of [lo_r, hi_r)
    const int r0 = rb * ROWS, r1 = r0 + ROWS < R ? r0 + ROWS : R;
    const int t0 = r0 / G, t1 = (r1 - 1) / G;
    const int base = len - a.new_tokens;         // place of token 0, below 0 if there are too few
    auto first_of = [&](int t) {
        const int64_t f = a.window > 0 ? static_cast<int64_t>(base) + t - a.window + 1 : 0;
        return f > 0 ? static_cast<int>(f) : 0;
    };
    auto end_of = [&](int t) { return base + t + 1 > 0 ? base + t + 1 : 0; };
    // the part's steps: an even share of the sequence's, cut to what these rows see
    const int steps = seq_steps<KT>(a, len);
    const int lo_seq = first_of(0) / KT * KT;
    const int s0 = static_cast<int>(static_cast<int64_t>(steps) * part.part / part.parts);
    const int s1 = static_cast<int>(static_cast<int64_t>(steps) * (part.part + 1) / part.parts);
    const int lo = max(first_of(t0), lo_seq + s0 * kWaves * KT);
    const int hi = min(end_of(t1), min(len, lo_seq + s1 * kWaves * KT));
    // between these, every row sees every key
    const int lo_all = first_of(t1), hi_all = end_of(t0);

    // q as the first product's B operands, in LDS: [MT][QF][64 lanes]
    int row_t[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = r0 + mt * 16 + li, rr = r < R ? r : R - 1;
        row_t[mt] = rr / G;
        const T *p = static_cast<const T *>(a.q) +
                     (static_cast<int64_t>(part.n) * a.new_tokens + row_t[mt]) * a.q_stride +
                     static_cast<int64_t>(h * G + rr % G) * D;
        for (int f = wave; f < QF; f += kWaves) {
            const T *at = p + f * Op::QW + lg * LV;
            s_q[(mt * QF + f) * 64 + lane] = a.q_whole ? *reinterpret_cast<const Frag *>(at) : Op::each(at);
        }
    }
    __syncthreads();

    f32x4 o[MT][V::S][V::VE];
    float m[MT], l[MT];                          // l: this lane's keys only
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        m[mt] = -INFINITY;
        l[mt] = 0.f;
#pragma unroll
        for (int s = 0; s < V::S; ++s)
#pragma unroll
            for (int j = 0; j < V::VE; ++j) o[mt][s][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    }

    const int32_t *table = a.page_table + static_cast<int64_t>(part.n) * a.max_pages;
    const T *const kp = static_cast<const T *>(a.k_pages), *const vp = static_cast<const T *>(a.v_pages);
    // the row of the pools that holds place j of the sequence
    auto pool_row = [&](int j) {
        const int pg = static_cast<int>((static_cast<uint64_t>(j) * a.page_mul) >> a.page_shift);
        int id = table[pg];
        id = id < a.num_pages ? id : a.num_pages - 1;
        id = id > 0 ? id : 0;
        return static_cast<uint32_t>((id * a.h_k + h) * a.page_size + (j - pg * a.page_size));
    };
    const float to2 = a.scale * kLog2e;
    Frag k[ST][QF];
    V v;
    f32x4 s[MT][ST];
    typename V::Weights pb[MT];

    auto products = [&]() {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int t = 0; t < ST; ++t) s[mt][t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < QF; ++f)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const Frag q = s_q[(mt * QF + f) * 64 + lane];
#pragma unroll
                for (int t = 0; t < ST; ++t) s[mt][t] = Op::qk(k[t][f], q, s[mt][t]);
            }
    };
    auto softmax = [&](int mt) {
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = fmaxf(top, s[mt][t][i]);
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        top = fmaxf(top, m[mt]);
        const float at = top == -INFINITY ? 0.f : top;      // nothing seen so far: all weights 0
        const float keep = __builtin_amdgcn_exp2f(m[mt] - at);
        m[mt] = top;
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][t][i] = __builtin_amdgcn_exp2f(s[mt][t][i] - at);
        l[mt] *= keep;
#pragma unroll
        for (int t = 0; t < ST; ++t) l[mt] += (s[mt][t].x + s[mt][t].y) + (s[mt][t].z + s[mt][t].w);
        pb[mt] = operand(s[mt], T{});
        if (!__all(keep == 1.f))
#pragma unroll
            for (int c = 0; c < V::S; ++c)
#pragma unroll
                for (int j = 0; j < V::VE; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) o[mt][c][j][i] *= keep;
    };
    auto add_values = [&]() {
#pragma unroll
        for (int c = 0; c < V::S; ++c)
#pragma unroll
            for (int j = 0; j < V::VE; ++j)
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) o[mt][c][j] = v.pv(c, j, pb[mt], o[mt][c][j]);
    };

    // A tile whose keys every row sees, in pages of whole sixteens: each 16 keys lie in one page, so
    // their rows are the same for all lanes but for a fixed offset.
    const int k_at = li * D + lg * LV, v_at = 4 * lg * D + li * V::VE;
    uint32_t row[ST];
    auto find_rows = [&](int tile, uint32_t (&to)[ST]) {
#pragma unroll
        for (int t = 0; t < ST; ++t) to[t] = __builtin_amdgcn_readfirstlane(pool_row(tile + 16 * t));
    };
    auto load_keys = [&]() {
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            const T *p = kp + static_cast<int64_t>(row[t]) * D;
#pragma unroll
            for (int f = 0; f < QF; ++f) k[t][f] = *reinterpret_cast<const Frag *>(p + k_at + f * Op::QW);
        }
    };
    auto load_values = [&]() {
#pragma unroll
        for (int r = 0; r < V::VR; ++r)
            v.load(r, vp + static_cast<int64_t>(row[r / 4]) * D + v_at + r % 4 * D, 0);
    };
    // Any other tile. Keys outside [lo, hi) take the nearest one inside, which is read instead and masked.
    auto edge = [&](int tile) {
        int at = tile + lane % KT;
        at = at < hi ? at : hi - 1;
        at = at > lo ? at : lo;
        const uint32_t mine = pool_row(at);
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            const T *p = kp + static_cast<int64_t>(__shfl(mine, t * 16 + li)) * D + lg * LV;
#pragma unroll
            for (int f = 0; f < QF; ++f) k[t][f] = *reinterpret_cast<const Frag *>(p + f * Op::QW);
        }
#pragma unroll
        for (int r = 0; r < V::VR; ++r) v.load(r, vp + static_cast<int64_t>(__shfl(mine, V::key(lg, r))) * D, li);
        products();
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int first = max(lo, first_of(row_t[mt])), end = min(hi, end_of(row_t[mt]));
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int j = tile + t * 16 + 4 * lg + i;
                    s[mt][t][i] = j >= first && j < end ? s[mt][t][i] * to2 : -INFINITY;
                }
            softmax(mt);
        }
        // Where rows see different keys of a tile, a weight of zero would still take in a value that
        // is not finite (0 * NaN): token by token then, without the values it does not see.
        const bool once = t0 == t1 || __all(v.finite());
        for (int t = once ? t1 : t0; t <= t1; ++t) {
            const int first = max(lo, first_of(t)), end = min(hi, end_of(t));
            typename V::Oper bits;
#pragma unroll
            for (int r = 0; r < V::VR; ++r) {
                const int j = tile + V::key(lg, r);
                V::see(r, once || (j >= first && j < end), bits);
            }
#pragma unroll
            for (int c = 0; c < V::S; ++c)
#pragma unroll
                for (int j = 0; j < V::VE; ++j) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const f32x4 x = v.pv(c, j, pb[mt], o[mt][c][j], &bits);
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[mt][c][j][i] = once || row_t[mt] == t ? x[i] : o[mt][c][j][i];
                    }
                    __builtin_amdgcn_sched_barrier(0);      // one product's registers at a time
                }
        }
    };

    constexpr int NEXT = kWaves * KT;
    const int full_lo = max(lo, lo_all), full_hi = min(hi, hi_all);
    const bool whole_pages = a.page_size % 16 == 0;
    int tile = lo < hi ? lo / KT * KT + wave * KT : hi;
    while (tile < hi) {
        if (!whole_pages || tile < full_lo || tile + KT > full_hi) {
            edge(tile);
            tile += NEXT;
            continue;
        }
        // The next tile's keys are under way while this one's weights and values are worked on, its
        // values while its products are. (The last tile loads its own keys again instead: a load that
        // is not always made would have to be waited for at once.)
        find_rows(tile, row);
        load_keys();
        bool more;
        do {
            more = tile + NEXT + KT <= full_hi;
            uint32_t ahead[ST];
            find_rows(more ? tile + NEXT : tile, ahead);
            load_values();
            __builtin_amdgcn_sched_barrier(0);
            products();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int t = 0; t < ST; ++t) row[t] = ahead[t];
            load_keys();
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
                for (int t = 0; t < ST; ++t)
#pragma unroll
                    for (int i = 0; i < 4; ++i) s[mt][t][i] *= to2;
                softmax(mt);
            }
            __builtin_amdgcn_sched_barrier(0);
            add_values();
            tile += NEXT;
        } while (more);
    }

    // the waves' rows join: every wave scales its sums to the common maximum, then 2 + 2 and 1 + 1
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16);
        l[mt] += __shfl_xor(l[mt], 32);
        if (lg == 0) {
            s_ml[wave][0][mt * 16 + li] = m[mt];
            s_ml[wave][1][mt * 16 + li] = l[mt];
        }
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_ml[w][0][mt * 16 + li]);
        const float at = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            sum += s_ml[w][1][mt * 16 + li] * __builtin_amdgcn_exp2f(s_ml[w][0][mt * 16 + li] - at);
        const float keep = __builtin_amdgcn_exp2f(m[mt] - at);
#pragma unroll
        for (int c = 0; c < V::S; ++c)
#pragma unroll
            for (int j = 0; j < V::VE; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][c][j][i] *= keep;
        m[mt] = top;
        l[mt] = sum;
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int half = kWaves / 2; half > 0; half >>= 1) {
            if (wave >= half && wave < 2 * half)
#pragma unroll
                for (int c = 0; c < V::S; ++c)
#pragma unroll
                    for (int j = 0; j < V::VE; ++j) s_o[wave - half][(c * V::VE + j) * 64 + lane] = o[mt][c][j];
            __syncthreads();
            if (wave < half)
#pragma unroll
                for (int c = 0; c < V::S; ++c)
#pragma unroll
                    for (int j = 0; j < V::VE; ++j) o[mt][c][j] += s_o[wave][(c * V::VE + j) * 64 + lane];
            __syncthreads();
        }
    if (wave != 0) return;

    // value j of row i of set c's product j is value (16 c + 4 lg + i) VE + j of the head
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = r0 + mt * 16 + li;
        if (r >= R) continue;
        if (part.parts == 1) {
            const int64_t at = (static_cast<int64_t>(part.n) * a.new_tokens + row_t[mt]) * a.h_q + h * G + r % G;
            const float inv = l[mt] == 0.f ? 0.f : 1.f / l[mt];
            T *out = static_cast<T *>(a.o) + at * D;
#pragma unroll
            for (int c = 0; c < V::S; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x[V::VE];
#pragma unroll
                    for (int j = 0; j < V::VE; ++j) x[j] = o[mt][c][j][i] * inv;
                    stv<T, V::VE>(out + (16 * c + 4 * lg + i) * V::VE, x);
                }
            if (a.lse && lg == 0)
                a.lse[at] = l[mt] == 0.f ? -INFINITY : (m[mt] + log2f(l[mt])) * (1.f / kLog2e);
        } else {
            const int64_t at = static_cast<int64_t>(blockIdx.x) * ROWS + mt * 16 + li;
            float *out = a.part_o + at * D;
#pragma unroll
            for (int c = 0; c < V::S; ++c)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float x[V::VE];
#pragma unroll
                    for (int j = 0; j < V::VE; ++j) x[j] = o[mt][c][j][i];
                    stv<float, V::VE>(out + (16 * c + 4 * lg + i) * V::VE, x);
                }
            if (lg == 0) {
                a.part_ml[2 * at] = m[mt];
                a.part_ml[2 * at + 1] = l[mt];
            }
        }
    }
}

// Joins the parts of a sequence: a workgroup per row, its D / 4 lanes per value times JW groups of
// threads that take every JW-th part.
template <typename T, int D, int MT>
__global__ __launch_bounds__(256) void paged_attention_join_kernel(AttentionArgs a, int row_blocks) {
    constexpr int KT = tile_keys<T>(D), ROWS = 16 * MT, LANES = D / 4, JW = 256 / LANES;
    __shared__ f32x4 s_o[JW][LANES];
    __shared__ float s_l[JW];
    const int G = a.h_q / a.h_k, heads = a.h_k * row_blocks;
    const int64_t at = static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x;
    if (at >= static_cast<int64_t>(a.num_seqs) * a.new_tokens * a.h_q) return;
    const int n = static_cast<int>(at / (static_cast<int64_t>(a.new_tokens) * a.h_q));
    const int t = static_cast<int>(at / a.h_q % a.new_tokens), hq = static_cast<int>(at % a.h_q);
    const int per = part_steps<KT>(a, heads);
    const int parts = num_parts(seq_steps<KT>(a, seq_len(a, n)), per);
    if (parts == 1) return;                      // written by the first kernel
    int before = 0;
    for (int base = 0; base < n; base += 64) {
        const int i = base + static_cast<int>(threadIdx.x & 63);
        before += wave_sum(i < n ? num_parts(seq_steps<KT>(a, seq_len(a, i)), per) : 0);
    }
    const int h = hq / G, r = t * G + hq % G;
    const int64_t step = static_cast<int64_t>(heads) * ROWS;
    const int64_t first = (static_cast<int64_t>(before) * heads + h * row_blocks + r / ROWS) * ROWS + r % ROWS;
    float top = -INFINITY;
    for (int p = threadIdx.x & 63; p < parts; p += 64) top = fmaxf(top, a.part_ml[2 * (first + p * step)]);
#pragma unroll
    for (int x = 1; x < 64; x <<= 1) top = fmaxf(top, __shfl_xor(top, x));
    const float ref = top == -INFINITY ? 0.f : top;
    const int c = threadIdx.x % LANES, g = threadIdx.x / LANES;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f;
#pragma unroll 4
    for (int p = g; p < parts; p += JW) {
        const int64_t i = first + p * step;
        const float w = __builtin_amdgcn_exp2f(a.part_ml[2 * i] - ref);
        l = fmaf(w, a.part_ml[2 * i + 1], l);
        const f32x4 x = *reinterpret_cast<const f32x4 *>(a.part_o + i * D + 4 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(w, x[e], o[e]);
    }
    s_o[g][c] = o;
    if (c == 0) s_l[g] = l;
    __syncthreads();
    if (g != 0) return;
#pragma unroll
    for (int x = 1; x < JW; ++x) {
        o += s_o[x][c];
        l += s_l[x];
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    io<T>::st4(static_cast<T *>(a.o) + at * D + 4 * c, o * inv);
    if (a.lse && c == 0) a.lse[at] = l == 0.f ? -INFINITY : (top + log2f(l)) * (1.f / kLog2e);
}

template <typename T, int D, int MT>
hipError_t launch(const AttentionArgs &a, const AttentionPlan &p, hipStream_t st) {
    const unsigned groups = static_cast<unsigned>(p.max_parts) * static_cast<unsigned>(a.h_k * p.row_blocks);
    hipLaunchKernelGGL((paged_attention_kernel<T, D, MT>), dim3(groups), dim3(64 * kWaves), 0, st, a, p.row_blocks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !p.split) return e;
    const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.new_tokens * a.h_q;
    const unsigned gx = static_cast<unsigned>(rows < (1 << 20) ? rows : (1 << 20));
    hipLaunchKernelGGL((paged_attention_join_kernel<T, D, MT>), dim3(gx, static_cast<unsigned>((rows + gx - 1) / gx)),
                       dim3(256), 0, st, a, p.row_blocks);
    return hipGetLastError();
}

template <typename T, int D>
hipError_t launch_rows(const AttentionArgs &a, const AttentionPlan &p, hipStream_t st) {
    return p.row_tiles == 1 ? launch<T, D, 1>(a, p, st) : launch<T, D, 2>(a, p, st);
}

template <typename T>
hipError_t launch_dims(const AttentionArgs &a, const AttentionPlan &p, hipStream_t st) {
    return a.d == 64 ? launch_rows<T, 64>(a, p, st) : a.d == 128 ? launch_rows<T, 128>(a, p, st)
                                                                 : launch_rows<T, 256>(a, p, st);
}

}  // namespace

// Tiles of 16 rows per workgroup, and blocks of them, for a key head's rows.
static int row_tiles(int64_t rows) { return rows <= 16 ? 1 : 2; }
static int64_t row_blocks(int64_t rows) { return (rows + 16 * row_tiles(rows) - 1) / (16 * row_tiles(rows)); }
static bool may_split(const gdn2_attention_dims &d) {
    const int step = kWaves * (d.dtype == GDN2_BF16 ? tile_keys<bf16_t>(d.d) : tile_keys<float>(d.d));
    return static_cast<int64_t>(d.max_pages) * d.page_size > kLeastSteps * step;
}

int64_t attention_groups(const gdn2_attention_dims &d) {
    const int64_t heads = d.h_k * row_blocks(static_cast<int64_t>(d.new_tokens) * (d.h_q / d.h_k));
    return (d.num_seqs + (may_split(d) ? kTargetGroups / heads : 0)) * heads;
}

AttentionPlan attention_plan(const gdn2_attention_dims &d) {
    const int64_t rows = static_cast<int64_t>(d.new_tokens) * (d.h_q / d.h_k);
    AttentionPlan p;
    p.row_tiles = row_tiles(rows);
    p.row_blocks = static_cast<int>(row_blocks(rows));
    p.split = may_split(d);
    p.max_parts = static_cast<int>(attention_groups(d) / (static_cast<int64_t>(d.h_k) * p.row_blocks));
    return p;
}

hipError_t launch_attention(const AttentionArgs &a, const AttentionPlan &p, hipStream_t st) {
    return a.bf16 ? launch_dims<bf16_t>(a, p, st) : launch_dims<float>(a, p, st);
}

}  // namespace gdn2
