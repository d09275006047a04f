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
struct LinearW8Args {
    const int8_t *x;
    const float *x_scale;
    const int8_t *codes;     // packed weight: codes, then scales
    const float *scale;
    const float *bias;
    void *out;
    int T, N, K, out_dtype, gated, streamed;
    int n_tiles, k_tiles;    // 16 rows, 128 k
};
struct QuantArgs {
    const void *x;
    const float *smooth;
    void *q;
    float *q_scale;
    int T, H, dtype, quant, streamed;
    int group;  // elements per scale, 0 = one per row
    float amax_eps;
};
struct JoinNormArgs {
    const void *block, *share, *residual, *post_weight, *gate, *weight;
    const float *share_scale;
    void *residual_out, *y, *q;
    float *q_scale;
    int T, H, dtype, weight_dtype, quant, group, post_norm, streamed;
    size_t gate_stride;  // elements between the tokens' rows of gate
    float residual_scale, branch_scale, post_eps, rms_eps, amax_eps;
};
struct DispatchArgs {
    const int32_t *ids;
    const void *x;
    const float *x_scale;
    const uint8_t *mask;
    void *rows;
    float *row_scale;
    int32_t *counts, *offset, *row_of_pair, *pair_of_row;
    int32_t *workspace;
    int T, K, E, H, elem, groups, align, streamed;  // elem: bytes of an element
    int64_t R;                            // rows of `rows` and pair_of_row
};
struct RowsArgs {  // sorted rows back to tokens, and the gradient
    const void *rows, *addend, *dout;
    const int32_t *row_of_pair, *pair_of_row;
    const float *scales;
    void *out, *drows;
    float *dscales;
    int T, K, H, R, dtype, out_dtype, streamed;
};
hipError_t launch_norm_quant(const NormArgs &a, hipStream_t s);
size_t gate_workspace(int T, int E, int H);
hipError_t launch_gate(const GateArgs &a, hipStream_t s);
hipError_t launch_pack_w4(const uint8_t *codes, const float *scale, const uint8_t *zero, uint8_t *dst_codes,
                          float *dst_scale, uint8_t *dst_zero, const LinearW4Args &a, hipStream_t s);
hipError_t launch_linear_w4(const LinearW4Args &a, hipStream_t s);
hipError_t launch_pack_w8(const int8_t *codes, const float *scale, int8_t *dst_codes, float *dst_scale,
                          const LinearW8Args &a, hipStream_t s);
hipError_t launch_linear_w8(const LinearW8Args &a, hipStream_t s);
hipError_t launch_quant(const QuantArgs &a, hipStream_t s);
hipError_t launch_join_norm(const JoinNormArgs &a, hipStream_t s);
size_t dispatch_workspace(int T, int K, int E);
hipError_t launch_dispatch(const DispatchArgs &a, hipStream_t s);
hipError_t launch_combine_rows(const RowsArgs &a, hipStream_t s);
hipError_t launch_combine_grad(const RowsArgs &a, hipStream_t s);

// Calls that write much store it as a stream (non-temporal): it does not push
// out of L2 what is still being read. In us, plain / streamed: int8 product T
// 4096, N 8192, K 4096 134 / 123, joining norm T 4001, H 5003 56 / 44, quantiser T
// 8192, H 4096 19.9 / 16.1, dispatch T 4096, K 8, H 4096 66 / 53, combine T 4096
// 68.0 / 64.9. What the next launch could still find in the cache behind the
// L2s is stored plainly: joining norm, product (N 8192) and quantiser in a row, T
// 512 (4 to 8 MB each) 34.6 / 38.1, T 2048 (16 to 32 MB) 96 / 91, T 8192 329 / 328.
constexpr size_t kStreamBytes = 16u << 20;
// 8 or 16-byte stores to any address.
template <typename V>
__device__ __forceinline__ void store_out(void *p, const V &v, bool streamed) {
    static_assert(sizeof(V) == 8 || sizeof(V) % 16 == 0, "whole stores");
    typedef int v4 __attribute__((ext_vector_type(4), aligned(1)));
    typedef int v2 __attribute__((ext_vector_type(2), aligned(1)));
    if (!streamed) {
        __builtin_memcpy(p, &v, sizeof(V));
        return;
    }
    asm volatile("");  // with nothing before and behind it, the compiler makes one plain store of both
    if constexpr (sizeof(V) == 8) {
        v2 w;
        __builtin_memcpy(&w, &v, 8);
        __builtin_nontemporal_store(w, static_cast<v2 *>(p));
    } else {
        v4 w[sizeof(V) / 16];
        __builtin_memcpy(w, &v, sizeof(V));
#pragma unroll
        for (unsigned i = 0; i < sizeof(V) / 16; ++i) __builtin_nontemporal_store(w[i], static_cast<v4 *>(p) + i);
    }
    asm volatile("");
}

// One element of a MOE_DTYPE_* array to fp32, and back with one rounding to
// nearest even (fp16 overflow to infinity).
struct Bf16 { uint16_t bits; };
struct Fp16 { uint16_t bits; };
__device__ __forceinline__ float to_f32(Bf16 v) { return bf16_to_f32(v.bits); }
__device__ __forceinline__ float to_f32(Fp16 v) { return static_cast<float>(__builtin_bit_cast(_Float16, v.bits)); }
__device__ __forceinline__ float to_f32(float v) { return v; }
// (The hardware's conversion to bf16 gives the bits of f32_to_bf16 for every
// one of the 2^32 inputs, as tests/test_gpu_conversions.py checks; in six
// instructions less.)
__device__ __forceinline__ void from_f32(float f, Bf16 &v) {
    v.bits = __builtin_bit_cast(uint16_t, static_cast<__bf16>(f));
}
__device__ __forceinline__ void from_f32(float f, Fp16 &v) {
    v.bits = __builtin_bit_cast(uint16_t, static_cast<_Float16>(f));
}
__device__ __forceinline__ void from_f32(float f, float &v) { v = f; }

}  // namespace moe
