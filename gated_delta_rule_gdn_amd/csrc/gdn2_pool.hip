// gdn2_pool.hip -- slots of pools copied: dst[i] takes the bytes of src[i] in every pool.
//
// Bound by memory: every byte is read once and written once, from the registers, with no
// staging copy between.
#include "gdn2_internal.h"

namespace gdn2 {

namespace {

constexpr int kCopyThreads = 256;
constexpr int kCopyUnits = 4;        // accesses a thread has in flight

template <typename W>
__global__ __launch_bounds__(kCopyThreads) void pool_copy_kernel(CopyArgs a) {
    char *pool = static_cast<char *>(a.pool[blockIdx.z]);
    const int64_t units = a.bytes[blockIdx.z] / static_cast<int64_t>(sizeof(W));
    const int64_t first = static_cast<int64_t>(blockIdx.x) * kCopyThreads * kCopyUnits + threadIdx.x;
    if (first >= units) return;
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
            if (first + u * kCopyThreads < units) t[first + u * kCopyThreads] = x[u];
    }
}

template <typename W>
hipError_t launch(const CopyArgs &a, int64_t most, hipStream_t st) {
    const int64_t units = most / static_cast<int64_t>(sizeof(W));
    const int64_t pieces = (units + kCopyThreads * kCopyUnits - 1) / (kCopyThreads * kCopyUnits);
    const unsigned rows = static_cast<unsigned>(a.count < 32768 ? a.count : 32768);
    hipLaunchKernelGGL((pool_copy_kernel<W>), dim3(static_cast<unsigned>(pieces), rows, static_cast<unsigned>(a.num_pools)),
                       dim3(kCopyThreads), 0, st, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_pool_copy(const CopyArgs &a, hipStream_t st) {
    uint64_t low = 0;                // bits of every address and size: their common alignment
    int64_t most = 0;
    for (int p = 0; p < a.num_pools; ++p) {
        low |= reinterpret_cast<uintptr_t>(a.pool[p]) | static_cast<uint64_t>(a.bytes[p]);
        most = a.bytes[p] > most ? a.bytes[p] : most;
    }
    if (low % 16 == 0) return launch<uint4>(a, most, st);
    if (low % 4 == 0) return launch<uint32_t>(a, most, st);
    if (low % 2 == 0) return launch<uint16_t>(a, most, st);
    return launch<uint8_t>(a, most, st);
}

}  // namespace gdn2
