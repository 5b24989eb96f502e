// gdn2_checks.h -- host checks of arguments shared by the calls around the recurrence and of the
// attention layer.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn2.h"
#include "gdn2_internal.h"

namespace gdn2 {
namespace checks {

constexpr int64_t kMaxElems = (int64_t{1} << 40);    // bound on any tensor's element count
constexpr int64_t kMaxTokens = (int64_t{1} << 30);   // token arithmetic stays in 32 bits
constexpr int32_t kMaxChannels = 1 << 20;
constexpr size_t kAlign = 256;                       // of workspaces and their parts

inline gdn2_status ok() { return report(GDN2_OK, ""); }

inline gdn2_status done(hipError_t e, const char *where) {
    return e == hipSuccess ? ok() : report_hip(e, where);
}

inline bool dtype_ok(int32_t t) { return t == GDN2_F32 || t == GDN2_BF16; }

// An output that is the same buffer as an input or as another output. NULLs are not compared.
template <int NO, int NI>
bool aliases(const void *const (&outs)[NO], const void *const (&ins)[NI]) {
    for (int i = 0; i < NO; ++i) {
        if (!outs[i]) continue;
        for (int j = 0; j < NI; ++j)
            if (outs[i] == ins[j]) return true;
        for (int j = i + 1; j < NO; ++j)
            if (outs[i] == outs[j]) return true;
    }
    return false;
}

// A token stride: 0 means contiguous. False if it is too small or the tensor too large.
inline bool take_stride(int64_t given, int64_t row, int64_t tokens, int64_t *out) {
    *out = given == 0 ? row : given;
    return *out >= row && *out <= kMaxElems && (tokens <= 0 || *out <= kMaxElems / tokens);
}

inline size_t padded(size_t bytes) { return (bytes + kAlign - 1) / kAlign * kAlign; }

inline gdn2_status check_workspace(const void *ws, size_t bytes, size_t need) {
    if (need == 0) return GDN2_OK;
    if (!ws) return report(GDN2_ERR_WORKSPACE, "workspace is NULL");
    if (bytes < need) return report(GDN2_ERR_WORKSPACE, "workspace is too small");
    if (reinterpret_cast<uintptr_t>(ws) % kAlign != 0)
        return report(GDN2_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    return GDN2_OK;
}

}  // namespace checks
}  // namespace gdn2
