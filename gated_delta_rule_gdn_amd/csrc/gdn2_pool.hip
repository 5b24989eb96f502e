// gdn2_pool.hip -- slots of pools copied: dst[i] takes the bytes of src[i] in every pool.
//
// Bound by memory: every byte is read once and written once, from the registers, with no staging copy
// between. The stores are non-temporal, straight to memory: 64 pages of 16 KB in 48 pools take 18.9 us
// (101 MB moved, 5.3 TB/s) and 24 states of 3.3 MB 25.7 (157 MB, 6.1), in place of 31.1 and 40.8 through
// the caches. What reads a copy next finds it in memory, though: a kernel that reads all of it at once
// takes 9 us longer behind the first, 3 behind the second. A fork's pages are read layer by layer
// between everything else that a layer moves, which would have put them out of the caches by then.
#include "gdn2_internal.h"

namespace gdn2 {

namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

// 256 x 8 accesses per workgroup cost 0.5 us less or more at large slots, but 5 us more for 400 slots of
// 80 bytes in 96 pools, of which a workgroup has one.
constexpr int kCopyThreads = 128;
constexpr int kCopyUnits = 4;        // accesses that a thread has in flight

// A workgroup copies pieces of slots, kCopyThreads * kCopyUnits accesses each: every gridDim.x-th of all
// pools' pieces one after the other, of every gridDim.y-th pair.
template <typename W>
__global__ __launch_bounds__(kCopyThreads) void pool_copy_kernel(CopyArgs a) {
    for (int id = static_cast<int>(blockIdx.x); id < a.pieces; id += gridDim.x) {
        int p, piece;
        if (a.same_pieces) {
            p = id / a.same_pieces;
            piece = id - p * a.same_pieces;
        } else {
            // the last pool whose pieces begin at or before this one
            const int lane = threadIdx.x & 63;
            const int begin = lane < a.num_pools ? a.first_piece[lane] : INT32_MAX;
            p = __popcll(__ballot(begin <= id)) - 1;
            piece = id - a.first_piece[p];
        }
        char *pool = static_cast<char *>(a.pool[p]);
        const int64_t units = a.bytes[p] / static_cast<int64_t>(sizeof(W));
        const int64_t first = static_cast<int64_t>(piece) * kCopyThreads * kCopyUnits + threadIdx.x;
        for (int i = blockIdx.y; i < a.count; i += gridDim.y) {
            const int from = a.src[i], to = a.dst[i];
            if (from < 0 || from >= a.num_slots || to < 0 || to >= a.num_slots || from == to) continue;
            const W *s = reinterpret_cast<const W *>(pool) + from * units;
            W *t = reinterpret_cast<W *>(pool) + to * units;
            W x[kCopyUnits];
#pragma unroll
            for (int u = 0; u < kCopyUnits; ++u)
                if (first + u * kCopyThreads < units) x[u] = s[first + u * kCopyThreads];
#pragma unroll
            for (int u = 0; u < kCopyUnits; ++u)
                if (first + u * kCopyThreads < units) __builtin_nontemporal_store(x[u], t + first + u * kCopyThreads);
        }
    }
}

template <typename W>
hipError_t launch(CopyArgs a, hipStream_t st) {
    constexpr int64_t PIECE = static_cast<int64_t>(sizeof(W)) * kCopyThreads * kCopyUnits;
    int64_t pieces = 0;
    a.same_pieces = static_cast<int>((a.bytes[0] + PIECE - 1) / PIECE);
    for (int p = 0; p < a.num_pools; ++p) {
        const int64_t n = (a.bytes[p] + PIECE - 1) / PIECE;
        if (n != a.same_pieces) a.same_pieces = 0;
        a.first_piece[p] = static_cast<int>(pieces);
        pieces += n;
    }
    a.pieces = static_cast<int>(pieces);       // 64 slots of 2^32 bytes, one by one: 2^29
    // one dimension of a grid holds less than 2^32 threads
    const unsigned gx = static_cast<unsigned>(pieces < (1 << 20) ? pieces : 1 << 20);
    const unsigned gy = static_cast<unsigned>(a.count < 32768 ? a.count : 32768);
    hipLaunchKernelGGL((pool_copy_kernel<W>), dim3(gx, gy), dim3(kCopyThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace

// The widest access that suits all pools of the launch. (64 pages of 16 KB in 48 pools, the same ones again:
// 15.4 us; with a pool of slots of 4 bytes beside them 18.5, of 6 32, of one 66.)
hipError_t launch_pool_copy(const CopyArgs &a, hipStream_t st) {
    uint64_t low = 0;                // bits of every address and size: their common alignment
    for (int p = 0; p < a.num_pools; ++p)
        low |= reinterpret_cast<uintptr_t>(a.pool[p]) | static_cast<uint64_t>(a.bytes[p]);
    if (low % 16 == 0) return launch<u32x4>(a, st);
    if (low % 4 == 0) return launch<uint32_t>(a, st);
    if (low % 2 == 0) return launch<uint16_t>(a, st);
    return launch<uint8_t>(a, st);
}

}  // namespace gdn2
