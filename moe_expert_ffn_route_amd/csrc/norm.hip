// Residual addition, root-mean-square norm and 8-bit quantisation of a row in
// one pass.
//
//   r = x + residual;  p = r * w;  rstd = 1 / sqrt(mean(r^2) + rms_eps)
//   y = p * rstd
//   codes of y by the block's rule (rowquant.h): a' = max(max|y|, amax_eps),
//   scale = a' / Q, q = rint((y * Q) / a'), Q = 127 or 448.
// y is p times one positive number per row, so (y * Q) / max|y| equals
// (p * Q) / max|p|: the codes come from p and max|p| alone, both single IEEE
// operations per element and a maximum, and do not depend on the order in
// which the squares are summed. rstd enters only the scale, and the codes of
// rows (or groups) whose amax lies under the floor.
//
// A row (of up to 16384 elements) is held as fp32 p in the registers of its
// kTPR threads between the one read of x, residual and w and the writes.
#include "internal.h"
#include "rowquant.h"

#include "../../include/moe_w8a8.h"

namespace moe {
namespace {

constexpr int kVec = 8;  // elements per thread and chunk

// kVec consecutive elements; rows of odd length start at any element, so
// nothing is assumed about the address but the element's own alignment (the
// hardware takes such 16-byte accesses).
template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[kVec]) {
    T raw[kVec];
    __builtin_memcpy(raw, p, sizeof raw);
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = to_f32(raw[e]);
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[kVec]) {
    T raw[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) from_f32(v[e], raw[e]);
    __builtin_memcpy(p, raw, sizeof raw);
}
// The last chunk of a row whose length is no multiple of kVec: n < kVec.
template <typename T>
__device__ __forceinline__ void load_tail(const T *p, int n, float (&v)[kVec]) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = e < n ? to_f32(p[e]) : 0.0f;
}
template <typename T>
__device__ __forceinline__ void store_tail(T *p, int n, const float (&v)[kVec]) {
#pragma unroll
    for (int e = 0; e < kVec; ++e)
        if (e < n) from_f32(v[e], p[e]);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
    return v;
}

// One workgroup of TPR threads per row, CH chunks of kVec elements per
// thread: H <= TPR * CH * kVec.
template <typename T, typename W, int TPR, int CH>
__global__ __launch_bounds__(TPR) void norm_kernel(NormArgs a) {
    constexpr int kWaves = TPR / kWave;
    __shared__ float s_sum[kWaves], s_max[kWaves];
    const int tr = threadIdx.x;
    const size_t base = static_cast<size_t>(blockIdx.x) * a.H;
    const T *x = static_cast<const T *>(a.x) + base;
    const T *res = a.residual ? static_cast<const T *>(a.residual) + base : nullptr;
    const W *w = static_cast<const W *>(a.weight);
    T *res_out = a.residual_out ? static_cast<T *>(a.residual_out) + base : nullptr;

    float p[CH][kVec];
    float sum = 0.0f, mx = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = (tr + j * TPR) * kVec, left = a.H - i;
        if (left <= 0) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) p[j][e] = 0.0f;
            continue;
        }
        float g[kVec];
        if (left >= kVec) {
            load8(x + i, p[j]);
            if (res) {
                load8(res + i, g);
#pragma unroll
                for (int e = 0; e < kVec; ++e) p[j][e] = p[j][e] + g[e];
            }
            if (w) load8(w + i, g);
        } else {
            load_tail(x + i, left, p[j]);
            if (res) {
                load_tail(res + i, left, g);
#pragma unroll
                for (int e = 0; e < kVec; ++e) p[j][e] = p[j][e] + g[e];
            }
            if (w) load_tail(w + i, left, g);
        }
        if (res_out) {
            if (left >= kVec) store8(res_out + i, p[j]);
            else store_tail(res_out + i, left, p[j]);
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            sum += p[j][e] * p[j][e];
            if (w) p[j][e] = p[j][e] * g[e];
            mx = fmaxf(mx, fabsf(p[j][e]));
        }
    }
    sum = wave_sum(sum);
    mx = wave_max(mx);
    if ((tr & (kWave - 1)) == 0) {
        s_sum[tr / kWave] = sum;
        s_max[tr / kWave] = mx;
    }
    __syncthreads();
    sum = 0.0f;
    mx = 0.0f;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        sum += s_sum[i];
        mx = fmaxf(mx, s_max[i]);
    }
    const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.H) + a.rms_eps);

    if (a.y) {
        T *y = static_cast<T *>(a.y) + base;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            const int i = (tr + j * TPR) * kVec, left = a.H - i;
            if (left <= 0) break;
            float v[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] = p[j][e] * rstd;
            if (left >= kVec) store8(y + i, v);
            else store_tail(y + i, left, v);
        }
    }
    if (!a.q) return;
    const bool fp8 = a.quant == MOE_QUANT_E4M3;
    const float top_inv = fp8 ? 1.0f / kQMax<true> : 1.0f / kQMax<false>;
    uint8_t *q = static_cast<uint8_t *>(a.q) + base;
    const int gl = a.group / kVec;  // lanes per group
    float *scale = a.q_scale + static_cast<size_t>(blockIdx.x) * (a.group ? a.H / a.group : 1);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int i = (tr + j * TPR) * kVec, left = a.H - i;
        if (j * TPR * kVec >= a.H) break;  // uniform
        float pm = mx;
        if (gl) {  // a group is gl neighbouring lanes' chunks and never straddles the row's end
            pm = 0.0f;
#pragma unroll
            for (int e = 0; e < kVec; ++e) pm = fmaxf(pm, fabsf(p[j][e]));
            for (int d = gl / 2; d > 0; d >>= 1) pm = fmaxf(pm, __shfl_xor(pm, d, kWave));
        }
        if (left <= 0) continue;
        const float am = pm * rstd;
        const float inv = am >= a.amax_eps ? 1.0f / pm : rstd * (1.0f / a.amax_eps);
        uint32_t lo, hi;
        if (fp8) {
            lo = quant4<true>(p[j][0], p[j][1], p[j][2], p[j][3], inv);
            hi = quant4<true>(p[j][4], p[j][5], p[j][6], p[j][7], inv);
        } else {
            lo = quant4<false>(p[j][0], p[j][1], p[j][2], p[j][3], inv);
            hi = quant4<false>(p[j][4], p[j][5], p[j][6], p[j][7], inv);
        }
        const uint64_t code = lo | (static_cast<uint64_t>(hi) << 32);
        if (left >= kVec) {
            __builtin_memcpy(q + i, &code, sizeof code);
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e < left) q[i + e] = static_cast<uint8_t>(code >> (8 * e));
        }
        if (gl ? (tr & (gl - 1)) == 0 : (j == 0 && tr == 0))
            scale[gl ? i / a.group : 0] = fmaxf(am, a.amax_eps) * top_inv;
    }
}

template <typename T, typename W>
hipError_t launch(const NormArgs &a, hipStream_t s) {
    const dim3 grid(a.T), blk(256);
    if (a.H <= 256 * kVec * 2)
        hipLaunchKernelGGL((norm_kernel<T, W, 256, 2>), grid, blk, 0, s, a);
    else
        hipLaunchKernelGGL((norm_kernel<T, W, 256, 8>), grid, blk, 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_norm_quant(const NormArgs &a, hipStream_t s) {
    switch (a.dtype) {
        case MOE_DTYPE_BF16:
            return a.weight_dtype == MOE_DTYPE_FP32 ? launch<Bf16, float>(a, s) : launch<Bf16, Bf16>(a, s);
        case MOE_DTYPE_FP16:
            return a.weight_dtype == MOE_DTYPE_FP32 ? launch<Fp16, float>(a, s) : launch<Fp16, Fp16>(a, s);
        default: return launch<float, float>(a, s);
    }
}

}  // namespace moe
