// Shared by the operators around the block: arguments, launches, element types.
#pragma once

#include "internal.h"

namespace moe {

// Operators around the block: arguments after validation (see the header for
// the formulas).
struct NormArgs {
    const void *x, *residual, *weight;
    void *residual_out, *y, *q;
    float *q_scale;
    int T, H, dtype, weight_dtype, quant;
    int group;  // elements per scale, 0 = one per row
    float rms_eps, amax_eps;
};
struct GateArgs {
    const void *x, *weight;
    const float *bias;
    int32_t *ids;
    float *scales;
    double *logits;  // workspace: [parts, T, E]
    float *x_norms, *w_norms;  // workspace behind them: squares of the rows, [parts, T] and [parts, E]
    int T, H, E, K, score, normalize, dtype, weight_dtype;
    float route_scale;
};
struct LinearW4Args {
    const void *x;
    const float *x_scale;
    const uint8_t *codes;    // packed weight: codes, then scales, then zero points
    const float *scale;
    const uint8_t *zero;     // null: all 8
    const float *bias;
    void *out;
    int T, N, K, group, act, gated;
    int n_tiles, k_tiles;    // 16 rows, 128 k
};
hipError_t launch_norm_quant(const NormArgs &a, hipStream_t s);
size_t gate_workspace(int T, int E, int H);
hipError_t launch_gate(const GateArgs &a, hipStream_t s);
hipError_t launch_pack_w4(const uint8_t *codes, const float *scale, const uint8_t *zero, uint8_t *dst_codes,
                          float *dst_scale, uint8_t *dst_zero, const LinearW4Args &a, hipStream_t s);
hipError_t launch_linear_w4(const LinearW4Args &a, hipStream_t s);

// One element of a MOE_DTYPE_* array to fp32, and back with one rounding to
// nearest even (fp16 overflow to infinity).
struct Bf16 { uint16_t bits; };
struct Fp16 { uint16_t bits; };
__device__ __forceinline__ float to_f32(Bf16 v) { return bf16_to_f32(v.bits); }
__device__ __forceinline__ float to_f32(Fp16 v) { return static_cast<float>(__builtin_bit_cast(_Float16, v.bits)); }
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ void from_f32(float f, Bf16 &v) { v.bits = f32_to_bf16(f); }
__device__ __forceinline__ void from_f32(float f, Fp16 &v) {
    v.bits = __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
}
__device__ __forceinline__ void from_f32(float f, float &v) { v = f; }

}  // namespace moe
