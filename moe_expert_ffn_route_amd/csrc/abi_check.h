// Host checks of the operators' arguments, shared by the ABI's sources.
#pragma once
#include "../../include/moe_w8a8.h"
#include "ops.h"

namespace moe {

constexpr int kMaxHidden = 16384;
constexpr int kMaxExperts = 1024;

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

struct Range {
    const void *p;
    size_t bytes;
};
inline bool overlap(const Range &a, const Range &b) {
    if (!a.p || !b.p || !a.bytes || !b.bytes) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}

inline size_t dtype_bytes(int dt) { return dt == MOE_DTYPE_FP32 ? 4 : dt == MOE_DTYPE_INT8 ? 1 : 2; }
inline bool is_float_dtype(int dt) { return dt == MOE_DTYPE_BF16 || dt == MOE_DTYPE_FP16 || dt == MOE_DTYPE_FP32; }

inline moe_status_t of_launch(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

}  // namespace moe
