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
// A row (of up to 16384 elements) is held as fp32 p in the registers of one
// workgroup between the one read of x, residual and w and the writes. What
// that costs is set by memory: T 8192, H 4096, bf16 with residual, y and int8
// codes (302 MB, half of it written) takes 57 us, 5.3 TB/s; the library's
// read-and-write probe with as much written as read moves 5.5 TB/s.
//
// Every load is issued before anything waits for one: none stands behind a
// branch. Lanes past the row's end read its last chunk again and count nothing.
// A row whose length is no multiple of kVec ends in up to seven elements more,
// one per thread.
#include "ops.h"
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
// Sum and maximum over the wave: DPP shifts within rows of 16 lanes, then the
// row ends to the following rows; lane 63 holds the result.
template <int CTRL>
__device__ __forceinline__ float dpp_or(float v, float absent) {
    return __int_as_float(__builtin_amdgcn_update_dpp(__float_as_int(absent), __float_as_int(v), CTRL, 0xF, 0xF, false));
}
__device__ __forceinline__ float last_lane_sum(float v) {
    v += dpp_or<0x111>(v, 0.0f);
    v += dpp_or<0x112>(v, 0.0f);
    v += dpp_or<0x114>(v, 0.0f);
    v += dpp_or<0x118>(v, 0.0f);
    // lanes 15, 31, 47, 63 hold their rows' sums; rows 1 and 3, then 2 and 3, take what is before them
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x142, 0xA, 0xF, false));
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x143, 0xC, 0xF, false));
    return v;
}
__device__ __forceinline__ float last_lane_max(float v) {  // of magnitudes
    v = fmaxf(v, dpp_or<0x111>(v, 0.0f));
    v = fmaxf(v, dpp_or<0x112>(v, 0.0f));
    v = fmaxf(v, dpp_or<0x114>(v, 0.0f));
    v = fmaxf(v, dpp_or<0x118>(v, 0.0f));
    v = fmaxf(v, dpp_or<0x142>(v, 0.0f));
    v = fmaxf(v, dpp_or<0x143>(v, 0.0f));
    return v;
}

// TPR threads per row, CH chunks of kVec elements per thread: H <= TPR * CH *
// kVec. A workgroup is one row, or four rows of one wave each. TAIL: H is no
// multiple of kVec.
template <int TPR>
constexpr int kRows = TPR == kWave ? 4 : 1;
template <typename T, typename W, int TPR, int CH, bool TAIL>
__global__ __launch_bounds__(TPR *kRows<TPR>) void norm_kernel(NormArgs a) {
    constexpr int kWaves = TPR / kWave;
    const int tr = threadIdx.x % TPR, row = blockIdx.x * kRows<TPR> + threadIdx.x / TPR;
    if (kRows<TPR> > 1 && row >= a.T) return;  // whole waves, and such a row has no barrier
    const size_t base = static_cast<size_t>(row) * a.H;
    const T *x = static_cast<const T *>(a.x) + base;
    const T *res = static_cast<const T *>(a.residual) + base;
    const W *w = static_cast<const W *>(a.weight);
    T *res_out = static_cast<T *>(a.residual_out) + base;
    const int chunks = a.H / kVec, rest = a.H % kVec;  // whole chunks, and the elements after them
    const bool tail = TAIL && tr < rest;
    const int it = TAIL ? chunks * kVec + min(tr, rest - 1) : 0;

    // chunk j of the thread, or the row's last one (a row without a whole chunk: nothing is read)
    auto at = [&](int j) { return min(tr + j * TPR, chunks - 1) * kVec; };
    float p[CH][kVec], g[CH][kVec], pt = 0.0f, gt = 1.0f;
    if (!TAIL || chunks > 0) {
        float r[CH][kVec];
#pragma unroll
        for (int j = 0; j < CH; ++j) load8(x + at(j), p[j]);
        if (a.residual) {
#pragma unroll
            for (int j = 0; j < CH; ++j) load8(res + at(j), r[j]);
        }
        if (w) {
#pragma unroll
            for (int j = 0; j < CH; ++j) load8(w + at(j), g[j]);
        }
        if (a.residual) {
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int e = 0; e < kVec; ++e) p[j][e] = p[j][e] + r[j][e];
        }
    }
    if (TAIL) {
        pt = to_f32(x[it]);
        if (a.residual) pt = pt + to_f32(res[it]);
        if (w) gt = to_f32(w[it]);
    }
    float sum = 0.0f, mx = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const bool in = tr + j * TPR < chunks;
        if (in && a.residual_out) store8(res_out + at(j), p[j]);
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            if (!in) p[j][e] = 0.0f;
            sum += p[j][e] * p[j][e];
            if (in && w) p[j][e] = p[j][e] * g[j][e];
            mx = fmaxf(mx, fabsf(p[j][e]));
        }
    }
    if (TAIL) {
        if (tail && a.residual_out) from_f32(pt, res_out[it]);
        if (!tail) pt = 0.0f;
        sum += pt * pt;
        if (tail && w) pt = pt * gt;
        mx = fmaxf(mx, fabsf(pt));
    }
    sum = last_lane_sum(sum);
    mx = last_lane_max(mx);
    if constexpr (kWaves == 1) {  // the wave has read every element: y may lie where x or residual did
        sum = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(sum), kWave - 1));
        mx = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(mx), kWave - 1));
    } else {
        __shared__ float s_sum[kWaves], s_max[kWaves];
        if ((tr & (kWave - 1)) == kWave - 1) {
            s_sum[tr / kWave] = sum;
            s_max[tr / kWave] = mx;
        }
        __syncthreads();  // the same, for the workgroup
        sum = 0.0f;
        mx = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) {
            sum += s_sum[i];
            mx = fmaxf(mx, s_max[i]);
        }
    }
    const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.H) + a.rms_eps);

    if (a.y) {
        T *y = static_cast<T *>(a.y) + base;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            if (tr + j * TPR >= chunks) break;
            float v[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] = p[j][e] * rstd;
            store8(y + at(j), v);
        }
        if (tail) from_f32(pt * rstd, y[it]);
    }
    if (!a.q) return;
    const bool fp8 = a.quant == MOE_QUANT_E4M3;
    const float top_inv = fp8 ? 1.0f / kQMax<true> : 1.0f / kQMax<false>;
    uint8_t *q = static_cast<uint8_t *>(a.q) + base;
    float *scale = a.q_scale + static_cast<size_t>(row) * (a.group ? a.H / a.group : 1);
    auto inv_of = [&](float pm, float am) {
        return am >= a.amax_eps ? 1.0f / pm : rstd * (1.0f / a.amax_eps);
    };
    auto quant8 = [&](const float (&v)[kVec], float inv) -> uint64_t {
        uint32_t lo, hi;
        if (fp8) {
            lo = quant4<true>(v[0], v[1], v[2], v[3], inv);
            hi = quant4<true>(v[4], v[5], v[6], v[7], inv);
        } else {
            lo = quant4<false>(v[0], v[1], v[2], v[3], inv);
            hi = quant4<false>(v[4], v[5], v[6], v[7], inv);
        }
        return lo | (static_cast<uint64_t>(hi) << 32);
    };
    if (a.group) {  // a group is gl neighbouring lanes' chunks; groups divide H, so there is no tail
        const int gl = a.group / kVec;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            if (j * TPR >= chunks) break;  // uniform
            float pm = 0.0f;
#pragma unroll
            for (int e = 0; e < kVec; ++e) pm = fmaxf(pm, fabsf(p[j][e]));
            for (int d = gl / 2; d > 0; d >>= 1) pm = fmaxf(pm, __shfl_xor(pm, d, kWave));
            if (tr + j * TPR >= chunks) continue;
            const float am = pm * rstd;
            const uint64_t code = quant8(p[j], inv_of(pm, am));
            __builtin_memcpy(q + at(j), &code, sizeof code);
            if ((tr & (gl - 1)) == 0) scale[at(j) / a.group] = fmaxf(am, a.amax_eps) * top_inv;
        }
        return;
    }
    const float am = mx * rstd, inv = inv_of(mx, am);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if (tr + j * TPR >= chunks) break;
        const uint64_t code = quant8(p[j], inv);
        __builtin_memcpy(q + at(j), &code, sizeof code);
    }
    if (tail) q[it] = static_cast<uint8_t>(fp8 ? quant4<true>(pt, 0.0f, 0.0f, 0.0f, inv) : quant4<false>(pt, 0.0f, 0.0f, 0.0f, inv));
    if (tr == 0) *scale = fmaxf(am, a.amax_eps) * top_inv;
}

template <typename T, typename W, int TPR, int CH>
hipError_t launch_rows(const NormArgs &a, hipStream_t s) {
    const dim3 grid((a.T + kRows<TPR> - 1) / kRows<TPR>), blk(TPR * kRows<TPR>);
    if (a.H % kVec) hipLaunchKernelGGL((norm_kernel<T, W, TPR, CH, true>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((norm_kernel<T, W, TPR, CH, false>), grid, blk, 0, s, a);
    return hipGetLastError();
}

// Short rows: one wave. Else 256 threads, or for long rows 1024 while they are
// few. In us, 1024 / 256 threads (in a captured graph): T 64, H 7168, groups of
// 128 5.8 / 7.3; T 300, H 16384 13.9 / 16.0; T 512, H 7168 13.7 / 10.8; T 777,
// H 5003, fp16 to E4M3 14.4 / 10.6; T 1000, H 16384 34 / 39; T 2000, H 7168 36
// / 32, H 5003 33 / 27.
template <typename T, typename W>
hipError_t launch(const NormArgs &a, hipStream_t s) {
    if (a.H <= 64 * kVec) return launch_rows<T, W, 64, 1>(a, s);
    if (a.H <= 256 * kVec) return launch_rows<T, W, 256, 1>(a, s);
    if (a.H <= 512 * kVec) return launch_rows<T, W, 256, 2>(a, s);
    if (a.T < 512) return a.H <= 1024 * kVec ? launch_rows<T, W, 1024, 1>(a, s) : launch_rows<T, W, 1024, 2>(a, s);
    return a.H <= 1024 * kVec ? launch_rows<T, W, 256, 4>(a, s) : launch_rows<T, W, 256, 8>(a, s);
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
