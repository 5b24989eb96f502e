// gdn2_attention.hip -- attention of the newest tokens of every sequence over a paged cache.
//
// The rows of one key head are its T new tokens times the G query heads that read it, row r being
// token r / G. For a row at place p and the keys j that it sees,
//     o = sum_j e^(s_j - m) v_j / l,   m = max_j s_j,   l = sum_j e^(s_j - m),   s_j = scale q . k_j
// in one pass over the keys: m, l and the unnormalised o are kept and rescaled when m grows, and
// parts of a sequence (m, l, o) join the same way. Exponentials are taken to base 2, of differences of
// the products as they are (m is one of them): (q . k_j - m) times to_base2 is 0 for the largest and -inf
// for a product of -inf, whatever their size, and off by its own roundings only. (A scaled product less a
// rounded scaled maximum is off by the rounding of the larger one: 2^100 at the lowest value of bf16.) For
// a scale below 0 the queries change their sign, so that the largest product has the largest weight.
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

constexpr int kWaves = 4;           // of a workgroup: as many as an output tile has rows in a lane

// Steps (a tile per wave) of a call that is never cut, of one with a window, whose sequences are about
// as long as each other, that is not if every CU has a sequence then, and of the shortest part that a
// sequence is cut into. The second launch takes 4 us, a step 1 to 2. (64 sequences, 4 key heads of 128, a
// window of 512 keys: 15 us whole, 22 cut; of 1,024 24.4 and 28.7; 1,500 32.1 and 37.3; two sequences of
// 768 14.2 and 11.3.)
constexpr int kWholeSteps = 4;
constexpr int kWindowSteps = 12;
constexpr int kLeastSteps = 1;
// Shares of all steps, in parts that run at once, that a part is held to where sequences outnumber those
// (256 sequences of 32,768 tokens together, 8 key heads of 128: 44.8 us with 2, 47.8 with 1, 56.4 with 8;
// 300 of 150,000: 125, 132, 148).
constexpr int kTurns = 2;

// Inclusive sum over the lanes of a wave, by the rows of 16 that DPP shifts in and across them.
__device__ __forceinline__ int lane_sums(int x) {
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, true);     // row_shr 1, 2, 4, 8
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, true);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);    // lane 15 to row 1, 47 to row 3
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);    // lane 31 to rows 2 and 3
    return x;
}
__device__ __forceinline__ int last_lane(int x) { return __builtin_amdgcn_readlane(x, 63); }

// The factor of differences of products: |scale| log2 e, but held inside the range of fp32, so that neither
// 0 nor -inf makes NaN with it. (A scale of 0 gives weights that are equal to 1e-6 at least.)
__device__ __forceinline__ float to_base2(const AttentionArgs &a) {
    return fminf(fmaxf(fabsf(a.scale) * kLog2e, 0x1p-149f), 0x1.fffffep127f);
}
// The log-sum-exp of a row whose largest product is `top`.
__device__ __forceinline__ float row_lse(const AttentionArgs &a, float top, float sum) {
    return sum == 0.f ? -INFINITY : fmaf(top, fabsf(a.scale), log2f(sum) * (1.f / kLog2e));
}

__device__ __forceinline__ int seq_len(const AttentionArgs &a, int n) {
    const int most = a.max_pages * a.page_size, len = a.seq_lens[n];
    return len < 0 ? 0 : len > most ? most : len;
}

// Steps of a workgroup over the places that a sequence's new tokens see.
template <int KT>
__device__ __forceinline__ int seq_steps(const AttentionArgs &a, int len) {
    const int64_t first = static_cast<int64_t>(len) - a.new_tokens - a.window + 1;
    const int lo = a.window > 0 && first > 0 ? static_cast<int>(first) / KT * KT : 0;
    return (len - lo + kWaves * KT - 1) / (kWaves * KT);
}

// Parts of `per` steps, about: the quotient is taken with a reciprocal that is held too small by 2^-21
// (it is off by 2^-23 itself, and conversion, product and factor by 2^-24 each), so that there is never
// a part more than steps / per rounded up: the workspace has room for no more.
struct Parts {
    float inv;
    int less;
    __device__ __forceinline__ explicit Parts(int per)
        : inv(__builtin_amdgcn_rcpf(static_cast<float>(per)) * (1.f - 0x1p-21f)), less(per - 1) {}
    __device__ __forceinline__ int of(int steps) const {
        const int n = static_cast<int>(static_cast<float>(static_cast<uint32_t>(steps) + less) * inv);
        return n > 1 ? n : 1;
    }
};

// A part of a sequence: number `part` of `parts`, of which `before` belong to earlier sequences.
struct Part {
    int n, part, parts, before;
};

// How a call's sequences are cut. Workgroups that run at once, a.budget parts of a sequence with all
// its heads, end together if no part is longer than another's and none has to wait, so the steps of a
// part are the fewest that give at most `budget` parts, or near them. More sequences than that run
// in turn, and only those longer than a share of the whole are cut. (64 sequences of 262,144 tokens
// together, 4 key heads of 128: 103 us with at most 768 workgroups for 768 places, 106 with about 1,024.)
// Every workgroup works this out by itself, in loops: what is not repeated has its code fetched
// first, which takes longer than running it (four tries side by side: 0.6 us more than in turn).
template <int KT>
__device__ __forceinline__ Part find_part(const AttentionArgs &a, int id, int (&s_steps)[64 * kWaves]) {
    const int lane = threadIdx.x & 63;
    auto load = [&](int n) { return n < a.num_seqs ? seq_steps<KT>(a, seq_len(a, n)) : 0; };
    // up to 64 sequences are in registers, up to 256 in LDS, a load per wave
    const int mine = load(a.num_seqs <= 64 ? lane : threadIdx.x);
    if (a.num_seqs > 64) {
        s_steps[threadIdx.x] = mine;
        __syncthreads();
    }
    auto steps_of = [&](int n) { return a.num_seqs <= 64 ? mine : n < 64 * kWaves ? s_steps[n] : load(n); };
    const float shares = static_cast<float>(a.budget - a.num_seqs);
    int low = 0, per = 0, next = 0;
#pragma unroll 1
    for (int tries = 0; tries < 5; ++tries) {
        // first all steps, then the parts that `next` steps give
        const Parts p(next);
        int64_t sum = 0;
#pragma unroll 1
        for (int base = 0; base < a.num_seqs; base += 64) {
            const int steps = steps_of(base + lane);
            sum += last_lane(lane_sums(next == 0 ? steps : base + lane < a.num_seqs ? p.of(steps) : 0));
        }
        if (next == 0) {
            // Steps per part that are enough in any case: all / (budget - num_seqs), rounded up. In
            // fp32, held too large by 2^-20 and one.
            const float all = static_cast<float>(sum);
            auto share = [&](float among) {
                const float x = all * __builtin_amdgcn_rcpf(among);
                return x < 0x1p24f ? static_cast<int>(x * (1.f + 0x1p-20f)) : 1 << 24;
            };
            low = share(static_cast<float>(shares > 0.f ? a.budget : kTurns * a.budget));
            low = low > kLeastSteps ? low : kLeastSteps;
            per = shares > 0.f ? share(shares) + 1 : low + 1;
            if (shares <= 0.f || a.num_seqs > 256) break;
        } else if (sum <= a.budget) {
            per = next;
        } else {
            low = next + 1;
        }
        if (low >= per) break;
        next = (low + per) / 2;
    }
    const Parts p(per);
    int before = 0;
#pragma unroll 1
    for (int base = 0; base < a.num_seqs; base += 64) {
        const int steps = steps_of(base + lane);
        const int parts = base + lane < a.num_seqs ? p.of(steps) : 0;
        const int sum = lane_sums(parts);
        const uint64_t hit = __ballot(parts > 0 && id < before + sum);
        if (hit) {
            const int l = __builtin_ctzll(hit), n = __builtin_amdgcn_readlane(parts, l);
            const int first = before + __builtin_amdgcn_readlane(sum, l) - n;
            return Part{base + l, id - first, n, first};
        }
        before += last_lane(sum);
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
    if (D == 64) return MT == 2 ? 3 : 4;
    return D == 128 ? (MT == 1 ? 3 : 2) : sizeof(T) == 4 ? 1 : 2;
}

// The first product: QW values of a head per operand of a lane's 16 bytes.
template <typename T> struct Ops;
template <> struct Ops<bf16_t> {
    static constexpr int QW = 32;
    typedef u32x4 Frag;                          // 8 values of a q or k row
    static constexpr int CHAINS = 1;
    static __device__ __forceinline__ void qk(Frag k, Frag q, f32x4 (&c)[1]) { c[0] = mma_k32(k, q, c[0]); }
    static __device__ __forceinline__ Frag turned(Frag f) { return f ^ 0x80008000u; }
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
    static constexpr int CHAINS = 4;
    static __device__ __forceinline__ void qk(Frag k, Frag q, f32x4 (&c)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = __builtin_amdgcn_mfma_f32_16x16x4f32(k[i], q[i], c[i], 0, 0, 0);
    }
    static __device__ __forceinline__ Frag turned(Frag f) { return -f; }
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
    __device__ __forceinline__ void clear(int r, bool seen) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < W; ++i) w[r][s][i] = seen ? w[r][s][i] : 0;
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
    __device__ __forceinline__ void clear(int r, bool seen) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) w[r][s][i] = seen ? w[r][s][i] : 0.f;
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

// PB: 8 for pages of whole eights that are not of whole sixteens, 16 for those and any others. (Pages of 8,
// 32 sequences x 4 new tokens, 65,536 keys of 2 x 8 heads of 256: 44 us, as any others 58; 16 sequences
// of 65,536, 4 key heads of 256 in fp32: 115 and 182.)
template <typename T, int D, int MT, int PB>
__global__ __launch_bounds__(64 * kWaves, (waves_per_simd<T, D, MT>())) void paged_attention_kernel(AttentionArgs a, int row_blocks) {
    using Op = Ops<T>;
    using V = VRows<T, D>;
    constexpr int KT = tile_keys<T>(D), ST = KT / 16, QF = D / Op::QW, ROWS = 16 * MT;
    constexpr int LV = 16 / sizeof(T);           // values of a 16-byte access
    typedef typename Op::Frag Frag;
    // q while the keys are worked on, one tile of rows of the waves' sums after that
    constexpr int QB = MT * QF * 64 * sizeof(Frag), OB = kWaves * 4 * V::S * V::VE * 64 * sizeof(float);
    __shared__ __align__(16) char s_mem[QB > OB ? QB : OB];
    __shared__ float s_ml[kWaves][2][ROWS];
    __shared__ int s_steps[64 * kWaves];
    Frag *const s_q = reinterpret_cast<Frag *>(s_mem);
    float *const s_o = reinterpret_cast<float *>(s_mem);
    const int lane = threadIdx.x & 63, lg = lane >> 4, li = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    // The blocks of rows that share keys are 8 apart: workgroups go round the 8 XCDs, so they find them in
    // one XCD's cache. (Fewer than 8 pairs of a part and a key head leave the other XCDs without work: a prompt
    // of 4,096 tokens runs at 393 TFLOP/s with 8 key heads of 128, at 105 with 2.) `group` is the workgroup's number without that.
    const int eight = static_cast<int>(blockIdx.x) / (8 * row_blocks), among = static_cast<int>(blockIdx.x) % (8 * row_blocks);
    const int rb = among / 8, pair = 8 * eight + among % 8, group = pair * row_blocks + rb;
    const int h = pair % a.h_k;
    const int G = a.h_q / a.h_k, R = a.new_tokens * G;
    const int id = pair / a.h_k;
    Part part{id, 0, 1, id};
    if (a.budget == 0) {
        if (id >= a.num_seqs) return;
    } else {
        part = find_part<KT>(a, id, s_steps);
        if (part.n < 0) return;
        if (part.part == 0 && h == 0 && rb == 0 && threadIdx.x == 0) {
            a.part_info[2 * part.n] = part.before;
            a.part_info[2 * part.n + 1] = part.parts;
        }
    }
    part.n = __builtin_amdgcn_readfirstlane(part.n);
    part.part = __builtin_amdgcn_readfirstlane(part.part);
    part.parts = __builtin_amdgcn_readfirstlane(part.parts);
    const int len = __builtin_amdgcn_readfirstlane(seq_len(a, part.n));

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

    // q as the first product's B operands: in LDS as [MT][QF][64 lanes], a share per wave
    constexpr int QS = (MT * QF + kWaves - 1) / kWaves;
    Frag q[QS];
    int row_t[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int r = r0 + mt * 16 + li;
        row_t[mt] = (r < R ? r : R - 1) / G;
    }
#pragma unroll
    for (int i = 0; i < QS; ++i) {
        const int f = wave + i * kWaves, mt = f / QF;
        if (f >= MT * QF) continue;
        const int t = MT == 1 || mt == 0 ? row_t[0] : row_t[MT - 1], r = r0 + mt * 16 + li;
        const T *p = static_cast<const T *>(a.q) +
                     (static_cast<int64_t>(part.n) * a.new_tokens + t) * a.q_stride +
                     static_cast<int64_t>(h * G + (r < R ? r : R - 1) - t * G) * D + f % QF * Op::QW + lg * LV;
        q[i] = a.q_whole ? *reinterpret_cast<const Frag *>(p) : Op::each(p);
        if (a.scale < 0.f) q[i] = Op::turned(q[i]);
    }

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
    const float to2 = to_base2(a);
    Frag k[ST][QF];
    V v;
    f32x4 s[MT][ST];
    typename V::Weights pb[MT];

    // fp32: four chains of d / 16 instructions, joined at the end, in place of one of d / 4. A score's
    // error goes into every weight, and it is the largest (1.1e-6 of o at 64 values with one chain).
    constexpr int CH = Op::CHAINS;
    auto products = [&]() {
        f32x4 part[MT][ST][CH];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int c = 0; c < CH; ++c) part[mt][t][c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int f = 0; f < QF; ++f)
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const Frag q = s_q[(mt * QF + f) * 64 + lane];
#pragma unroll
                for (int t = 0; t < ST; ++t) Op::qk(k[t][f], q, part[mt][t]);
            }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int t = 0; t < ST; ++t)
                s[mt][t] = CH == 1 ? part[mt][t][0]
                                   : (part[mt][t][0] + part[mt][t][1 % CH]) + (part[mt][t][2 % CH] + part[mt][t][3 % CH]);
    };
    // Of a tile's products, those that seen(t, i) says.
    auto softmax = [&](int mt, auto &&seen) {
        float top = -INFINITY;
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s[mt][t][i] = seen(t, i) ? s[mt][t][i] : -INFINITY;
                top = fmaxf(top, s[mt][t][i]);
            }
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        top = fmaxf(top, m[mt]);
        const float at = top == -INFINITY ? 0.f : top;      // nothing seen so far: all weights 0
        const float keep = __builtin_amdgcn_exp2f((m[mt] - at) * to2);
        m[mt] = top;
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[mt][t][i] = __builtin_amdgcn_exp2f((s[mt][t][i] - at) * to2);
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

    // Pages of whole PB: each PB keys lie in one page, so their rows follow the first, whose row is the same
    // for all lanes. PB keys outside [lo, hi) (a tile has some inside) are the nearest ones inside instead.
    constexpr int NB = KT / PB, OF = 16 / PB;            // blocks of a tile, and of sixteen keys
    const int k_at = li % PB * D + lg * LV, v_at = 4 * lg % PB * D + li * V::VE;
    uint32_t row[NB];
    auto find_rows = [&](int tile, uint32_t (&to)[NB]) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            int at = tile + PB * b;
            if (b > 0) at = min(at, (hi - 1) / PB * PB);
            if (b + 1 < NB) at = max(at, lo / PB * PB);
            to[b] = __builtin_amdgcn_readfirstlane(pool_row(at));
        }
    };
    auto load_keys = [&]() {
#pragma unroll
        for (int t = 0; t < ST; ++t) {
            const uint32_t mine = li < PB ? row[OF * t] : row[OF * t + OF - 1];
            const T *p = kp + static_cast<int64_t>(mine) * D;
#pragma unroll
            for (int f = 0; f < QF; ++f) k[t][f] = *reinterpret_cast<const Frag *>(p + k_at + f * Op::QW);
        }
    };
    auto load_values = [&]() {
#pragma unroll
        for (int r = 0; r < V::VR; ++r) {
            const uint32_t mine = 4 * lg < PB ? row[OF * (r / 4)] : row[OF * (r / 4) + OF - 1];
            v.load(r, vp + static_cast<int64_t>(mine) * D + v_at + r % 4 * D, 0);
        }
    };
    // Other pages. Keys outside [lo, hi) take the nearest one inside, which is read instead and masked.
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
            softmax(mt, [&](int t, int i) {
                const int j = tile + t * 16 + 4 * lg + i;
                return j >= first && j < end;
            });
        }
        // Where rows see different keys of a tile, a weight of zero would still take in a value that
        // is not finite: token by token then, without the values it does not see.
        int once = t0 == t1 || __all(v.finite());
        for (int t = once ? t1 : t0; t <= t1; ++t) {
            asm volatile("" : "+v"(once));       // else the loop is built twice, with the sums copied between
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

    // This wave's tiles are first, first + NEXT .. below hi.
    constexpr int NEXT = kWaves * KT;
    const int first = lo < hi ? lo / KT * KT + wave * KT : hi;
    const int full_lo = max(lo, lo_all), full_hi = min(hi, hi_all);
    const int piped = a.page_size % PB == 0 ? hi : first;
    if (first < piped) {
        find_rows(first, row);
        load_keys();
    }
#pragma unroll
    for (int i = 0; i < QS; ++i)
        if (wave + i * kWaves < MT * QF) s_q[(wave + i * kWaves) * 64 + lane] = q[i];
    __syncthreads();
    // The next tile's keys are under way while this one's weights and values are worked on, its values
    // while its products are. (The last tile loads its own keys again instead: a load that is not
    // always made would have to be waited for at once.) Places that no row sees are in the pool too, and
    // masked: in the loop of other pages, tiles with such places take longer (both kernels of 4 sequences of
    // 611 tokens together 8.5 us in place of 8.0, of 32 x 4 new tokens with a window 42 in place of 40.7).
    int tile = first;
    for (; tile < piped; tile += NEXT) {
        uint32_t ahead[NB];
        find_rows(tile + NEXT < hi ? tile + NEXT : tile, ahead);
        load_values();
        __builtin_amdgcn_sched_barrier(0);
        products();
        __builtin_amdgcn_sched_barrier(0);
        if (tile < full_lo || tile + KT > full_hi) {      // not every row sees all of it
#pragma unroll
            for (int r = 0; r < V::VR; ++r) {
                const int j = tile + V::key(lg, r);
                v.clear(r, j >= lo && j < hi);
            }
            if (t0 < t1 && !__all(v.finite())) break;      // it and what follows: as other pages
        }
#pragma unroll
        for (int b = 0; b < NB; ++b) row[b] = ahead[b];
        load_keys();
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int from = max(lo, first_of(row_t[mt])), many = max(min(hi, end_of(row_t[mt])) - from, 0);
            const int at = tile + 4 * lg - from;
            softmax(mt, [&](int t, int i) { return static_cast<uint32_t>(at + t * 16 + i) < static_cast<uint32_t>(many); });
        }
        __builtin_amdgcn_sched_barrier(0);
        add_values();
    }
    for (; tile < hi; tile += NEXT) edge(tile);

    // The waves' rows join: every wave scales its sums to the common maximum, then wave i adds row i of
    // every output tile over the waves, and writes it.
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        l[mt] += __shfl_xor(l[mt], 16);
        l[mt] += __shfl_xor(l[mt], 32);
        if (lg == 0) {
            s_ml[wave][0][mt * 16 + li] = m[mt];
            s_ml[wave][1][mt * 16 + li] = l[mt];
        }
    }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        __syncthreads();                         // the first: all waves have done with q
        float top = -INFINITY, sum = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) top = fmaxf(top, s_ml[w][0][mt * 16 + li]);
        const float at = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int w = 0; w < kWaves; ++w)
            sum += s_ml[w][1][mt * 16 + li] * __builtin_amdgcn_exp2f((s_ml[w][0][mt * 16 + li] - at) * to2);
        const float keep = __builtin_amdgcn_exp2f((m[mt] - at) * to2);
#pragma unroll
        for (int c = 0; c < V::S; ++c)
#pragma unroll
            for (int j = 0; j < V::VE; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    s_o[(((wave * 4 + i) * V::S + c) * V::VE + j) * 64 + lane] = o[mt][c][j][i] * keep;
        __syncthreads();
        const int r = r0 + mt * 16 + li;
        const bool cut = part.parts > 1;
        const float inv = cut ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
        const int64_t part_at = static_cast<int64_t>(group) * ROWS + mt * 16 + li;
        const int64_t row_at = (static_cast<int64_t>(part.n) * a.new_tokens + row_t[mt]) * a.h_q + h * G + r - row_t[mt] * G;
#pragma unroll
        for (int c = 0; c < V::S; ++c) {
            float x[V::VE];
#pragma unroll
            for (int j = 0; j < V::VE; ++j) {
                x[j] = 0.f;
#pragma unroll
                for (int w = 0; w < kWaves; ++w) x[j] += s_o[(((w * 4 + wave) * V::S + c) * V::VE + j) * 64 + lane];
                x[j] *= inv;
            }
            // value j of row i of set c's product j is value (16 c + 4 lg + i) VE + j of the head
            const int to = (16 * c + 4 * lg + wave) * V::VE;
            if (r >= R) continue;
            if (cut) stv<float, V::VE>(a.part_o + part_at * D + to, x);
            else stv<T, V::VE>(static_cast<T *>(a.o) + row_at * D + to, x);
        }
        if (r < R && lg == 0 && wave == 0) {
            if (cut) *reinterpret_cast<float2 *>(a.part_ml + 2 * part_at) = float2{top, sum};
            else if (a.lse) a.lse[row_at] = row_lse(a, top, sum);
        }
    }
}

// Joins the parts of a sequence: a row has D / 4 lanes per part, and the rest of its THREADS other
// parts. Many rows take a wave each (8,192 rows of whole sequences: 4.6 us in place of 15), few a
// workgroup (5.1 us for 32 rows of 93 parts).
template <typename T, int D, int MT, int THREADS>
__global__ __launch_bounds__(256) void paged_attention_join_kernel(AttentionArgs a, int row_blocks) {
    constexpr int ROWS = 16 * MT, LANES = D / 4, JW = THREADS / LANES, PER = 256 / THREADS;
    __shared__ f32x4 s_o[PER][JW][LANES];
    __shared__ float2 s_ml[PER][JW];
    const int G = a.h_q / a.h_k, heads = a.h_k * row_blocks;
    const float to2 = to_base2(a);
    const int slot = threadIdx.x / THREADS, thread = threadIdx.x % THREADS;
    const int64_t at = (static_cast<int64_t>(blockIdx.y) * gridDim.x + blockIdx.x) * PER + slot;
    const bool mine = at < static_cast<int64_t>(a.num_seqs) * a.new_tokens * a.h_q;
    int parts = 1, before = 0, n = 0;
    if (mine) {
        n = static_cast<int>(at / (static_cast<int64_t>(a.new_tokens) * a.h_q));
        before = a.part_info[2 * n];
        parts = a.part_info[2 * n + 1];
    }
    const bool cut = parts > 1;                  // whole sequences are written by the first kernel
    const int c = thread % LANES, g = thread / LANES;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    float l = 0.f, top = -INFINITY;
    if (cut) {
        const int t = static_cast<int>(at / a.h_q % a.new_tokens), hq = static_cast<int>(at % a.h_q);
        const int h = hq / G, r = t * G + hq % G;
        const int64_t step = static_cast<int64_t>(heads) * ROWS;
        const int64_t first = (static_cast<int64_t>(before) * heads + h * row_blocks + r / ROWS) * ROWS + r % ROWS;
        // parts g, JW + g .., four of them under way at a time, with a running maximum as in a part
        constexpr int U = 4;
        for (int p = g; p < parts; p += U * JW) {
            float2 ml[U];
            f32x4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int64_t i = first + (p + u * JW < parts ? p + u * JW : p) * step;
                ml[u] = *reinterpret_cast<const float2 *>(a.part_ml + 2 * i);
                x[u] = *reinterpret_cast<const f32x4 *>(a.part_o + i * D + 4 * c);
            }
            float high = top;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (p + u * JW >= parts) ml[u].x = -INFINITY;
                high = fmaxf(high, ml[u].x);
            }
            const float ref = high == -INFINITY ? 0.f : high, keep = __builtin_amdgcn_exp2f((top - ref) * to2);
            top = high;
            l *= keep;
            o *= keep;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const float w = __builtin_amdgcn_exp2f((ml[u].x - ref) * to2);
                l = fmaf(w, ml[u].y, l);
#pragma unroll
                for (int e = 0; e < 4; ++e) o[e] = fmaf(w, x[u][e], o[e]);
            }
        }
    }
    if constexpr (JW > 1) {
        s_o[slot][g][c] = o;
        if (c == 0) s_ml[slot][g] = float2{top, l};
        __syncthreads();
        if (g != 0) return;
        float high = top;
#pragma unroll
        for (int x = 1; x < JW; ++x) high = fmaxf(high, s_ml[slot][x].x);
        const float ref = high == -INFINITY ? 0.f : high, keep = __builtin_amdgcn_exp2f((top - ref) * to2);
        top = high;
        l *= keep;
        o *= keep;
#pragma unroll
        for (int x = 1; x < JW; ++x) {
            const float w = __builtin_amdgcn_exp2f((s_ml[slot][x].x - ref) * to2);
            l = fmaf(w, s_ml[slot][x].y, l);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(w, s_o[slot][x][c][e], o[e]);
        }
    }
    if (!cut) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    io<T>::st4(static_cast<T *>(a.o) + at * D + 4 * c, o * inv);
    if (a.lse && c == 0) a.lse[at] = row_lse(a, top, l);
}

constexpr int kJoinRows = 2048;      // most rows that take a workgroup each

template <typename T, int D, int MT>
hipError_t launch(const AttentionArgs &a, const AttentionPlan &p, hipStream_t st) {
    const int blocks_of_rows = static_cast<int>(p.row_blocks);
    const dim3 groups(static_cast<unsigned>(p.groups)), threads(64 * kWaves);
    if (a.page_size % 16 == 8) hipLaunchKernelGGL((paged_attention_kernel<T, D, MT, 8>), groups, threads, 0, st, a, blocks_of_rows);
    else hipLaunchKernelGGL((paged_attention_kernel<T, D, MT, 16>), groups, threads, 0, st, a, blocks_of_rows);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || p.budget == 0) return e;
    const int64_t rows = static_cast<int64_t>(a.num_seqs) * a.new_tokens * a.h_q;
    const int64_t blocks = rows <= kJoinRows ? rows : (rows + 3) / 4;
    const unsigned gx = static_cast<unsigned>(blocks < (1 << 20) ? blocks : (1 << 20));
    const dim3 grid(gx, static_cast<unsigned>((blocks + gx - 1) / gx));
    if (rows <= kJoinRows)
        hipLaunchKernelGGL((paged_attention_join_kernel<T, D, MT, 256>), grid, dim3(256), 0, st, a, blocks_of_rows);
    else
        hipLaunchKernelGGL((paged_attention_join_kernel<T, D, MT, 64>), grid, dim3(256), 0, st, a, blocks_of_rows);
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
static int step_keys(const gdn2_attention_dims &d) {
    return kWaves * (d.dtype == GDN2_BF16 ? tile_keys<bf16_t>(d.d) : tile_keys<float>(d.d));
}
// Workgroups that the chip holds at once.
static int places(const gdn2_attention_dims &d, int tiles) {
    auto of = [&](auto type) {
        using T = decltype(type);
        return d.d == 64 ? (tiles == 1 ? waves_per_simd<T, 64, 1>() : waves_per_simd<T, 64, 2>())
             : d.d == 128 ? (tiles == 1 ? waves_per_simd<T, 128, 1>() : waves_per_simd<T, 128, 2>())
                          : (tiles == 1 ? waves_per_simd<T, 256, 1>() : waves_per_simd<T, 256, 2>());
    };
    return kSimds / 4 * (d.dtype == GDN2_BF16 ? of(bf16_t{}) : of(float{}));
}

AttentionPlan attention_plan(const gdn2_attention_dims &d) {
    const int64_t rows = static_cast<int64_t>(d.new_tokens) * (d.h_q / d.h_k);
    AttentionPlan p;
    p.row_tiles = row_tiles(rows);
    p.row_blocks = row_blocks(rows);
    const int64_t heads = d.h_k * p.row_blocks, keys = static_cast<int64_t>(d.max_pages) * d.page_size;
    const int64_t seen = static_cast<int64_t>(d.window) + d.new_tokens - 1;
    const bool short_window = d.window > 0 && seen < keys;
    int whole = kWholeSteps;
    // Steps of 3 us: fp32 of 256 values, and two tiles of rows of them in pages whose rows are looked up
    // lane by lane (32 sequences x 2 key heads, a window of 200: 23 us cut, 26 whole; 1 x 7, 7 new tokens,
    // 248: 18, 23).
    if (d.d == 256 && (d.dtype == GDN2_F32 || (p.row_tiles == 2 && d.page_size % 8 != 0))) whole /= 2;
    if (short_window && d.num_seqs * heads >= kSimds / 4) whole = kWindowSteps;
    const bool cut = (short_window ? seen : keys) > static_cast<int64_t>(whole) * step_keys(d);
    p.budget = cut ? places(d, p.row_tiles) / heads : 0;
    // Two tiles of rows in bf16: the sums of a part are so large (32 KB at 256 values, for 256 KB of keys
    // and values where the chip is just filled) that one workgroup per CU does better, as long as that
    // leaves four parts per sequence (32 sequences x 4 new tokens, 65,536 keys of 2 x 8 heads of 256:
    // 42.3 -> 40.3 us, one of 200,000 97 -> 91; with two per sequence, 64 of 200,000 together 101 -> 105).
    // It does worse where its one wave per SIMD is busy rather than waiting: workgroups that share keys
    // (32 x 8 new tokens, 200,000 keys of 4 x 8 heads of 128: 112 -> 126), 64 values (42 -> 45), fp32
    // (32 x 8 new tokens, 4 x 8 heads of 128: 109 -> 120).
    if (p.budget > 0 && p.row_tiles == 2 && p.row_blocks == 1 && d.dtype == GDN2_BF16 && d.d > 64 &&
        kSimds / 4 / heads >= 4 * static_cast<int64_t>(d.num_seqs))
        p.budget = kSimds / 4 / heads;
    if (p.budget == 1 && d.num_seqs >= 1) p.budget = 0;      // every sequence whole
    p.max_parts = p.budget > d.num_seqs ? p.budget : d.num_seqs + kTurns * p.budget;
    p.groups = (p.max_parts * d.h_k + 7) / 8 * 8 * p.row_blocks;
    return p;
}

hipError_t launch_attention(const AttentionArgs &a, const AttentionPlan &p, hipStream_t st) {
    return a.bf16 ? launch_dims<bf16_t>(a, p, st) : launch_dims<float>(a, p, st);
}

}  // namespace gdn2
