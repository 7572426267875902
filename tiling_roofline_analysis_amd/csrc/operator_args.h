// operator_args.h -- what the C-ABI entry points of the operators share on the host:
// views of their operands, checks of them, status codes.
#pragma once

#include <cstddef>
#include <cstdint>

#include "gemm_internal.h"
#include "tra_gemm.h"

namespace tra {
namespace host {

// M, N, K: indices along an axis, rounded up to whole tiles and doubled for a gated
// result, fit 32 bits.
constexpr int64_t kMaxSize = int64_t{1} << 30;
constexpr size_t kAlign = 256;              // of the workspace's parts

inline size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

inline int64_t elem_bytes(int dtype) { return dtype == TRA_DTYPE_F32 ? 4 : 2; }

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Rows of a matrix at p start 16-byte aligned.
inline bool rows16(const void *p, int64_t ld, int64_t bytes) {
    return aligned16(p) && ld * bytes % 16 == 0;
}

// A row-major view: rows x cols elements of `bytes` bytes.
struct View {
    const void *p;
    int64_t rows, cols, ld, bytes;

    bool empty() const { return rows <= 0 || cols <= 0; }
    // A view the kernels may touch: aligned to its elements, rows that do not
    // overlap, extent in the address space.
    bool valid() const {
        if (empty()) return true;
        if (p == nullptr || ld < cols) return false;
        const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
        if (lo % static_cast<uintptr_t>(bytes) != 0) return false;
        const __int128 extent = (static_cast<__int128>(rows - 1) * ld + cols) * bytes;
        return extent <= static_cast<__int128>(INT64_MAX) &&
               static_cast<__int128>(lo) + extent <= static_cast<__int128>(UINTPTR_MAX);
    }
    uintptr_t lo() const { return reinterpret_cast<uintptr_t>(p); }
    uintptr_t hi() const {
        return lo() + static_cast<uintptr_t>(((rows - 1) * ld + cols) * bytes);
    }
};

// True if the two (valid) views share an element, or might: column ranges of
// one row-major buffer (same row pitch) interleave without sharing any.
inline bool share(const View &a, const View &b) {
    if (a.empty() || b.empty() || a.hi() <= b.lo() || b.hi() <= a.lo()) return false;
    if (a.rows == 1 || b.rows == 1 || a.ld * a.bytes != b.ld * b.bytes) return true;
    const View &x = a.lo() <= b.lo() ? a : b, &y = a.lo() <= b.lo() ? b : a;
    const int64_t pitch = x.ld * x.bytes;
    const int64_t at = static_cast<int64_t>((y.lo() - x.lo()) % static_cast<uintptr_t>(pitch));
    return at < x.cols * x.bytes || at + y.cols * y.bytes > pitch;
}

inline bool same(const View &a, const View &b) { return a.p == b.p && (a.ld == b.ld || a.rows <= 1); }

inline bool valid_act(int act) { return act >= TRA_ACT_NONE && act < TRA_ACT_COUNT; }
inline bool valid_dtype(int d) { return d >= TRA_DTYPE_F32 && d < TRA_DTYPE_COUNT; }

inline tra_status status_of(hipError_t err) {
    if (err == hipSuccess) return TRA_OK;
    record_hip_error(err);
    return TRA_ERR_HIP;
}

inline bool workspace_ok(const void *ws, uint64_t have, size_t need) {
    return need == 0 || (ws != nullptr && have >= need &&
                         (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1)) == 0);
}

}  // namespace host
}  // namespace tra
