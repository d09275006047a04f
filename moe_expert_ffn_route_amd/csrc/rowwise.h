// A row in the registers of one workgroup: loads and stores of eight elements,
// and reductions over a wave. Shared by the norms and the quantiser.
#pragma once
#include "ops.h"
#include "rowquant.h"

namespace moe {

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

// The same for the workgroup of a row: WAVES waves, `slot` its WAVES words of
// LDS. One wave needs no barrier.
template <int WAVES, typename V, typename Join>
__device__ __forceinline__ V join_waves(V v, V *slot, int tr, Join join) {  // v: lane 63's
    if ((tr & (kWave - 1)) == kWave - 1) slot[tr / kWave] = v;
    __syncthreads();
    v = slot[0];
#pragma unroll
    for (int i = 1; i < WAVES; ++i) v = join(v, slot[i]);
    return v;
}

// Eight codes of a row.
__device__ __forceinline__ uint64_t quant8(const float (&v)[kVec], float inv, bool fp8) {
    uint32_t lo, hi;
    if (fp8) {
        lo = quant4<true>(v[0], v[1], v[2], v[3], inv);
        hi = quant4<true>(v[4], v[5], v[6], v[7], inv);
    } else {
        lo = quant4<false>(v[0], v[1], v[2], v[3], inv);
        hi = quant4<false>(v[4], v[5], v[6], v[7], inv);
    }
    return lo | (static_cast<uint64_t>(hi) << 32);
}

// Rows per workgroup: four of one wave each, or one.
template <int TPR>
constexpr int kRows = TPR == kWave ? 4 : 1;

// Codes and scales of the row's p (zero behind its end) times rstd, mx = max|p|.
// Thread tr holds chunk tr + j * TPR and, TAIL, element `it` if `tail`.
template <int TPR, int CH, bool TAIL>
__device__ __forceinline__ void write_codes(const float (&p)[CH][kVec], float pt, float mx, float rstd, float eps,
                                            bool fp8, int group, int H, int tr, bool tail, int it, uint8_t *q,
                                            float *scale) {
    const int chunks = H / kVec;
    const float top_inv = fp8 ? 1.0f / kQMax<true> : 1.0f / kQMax<false>;
    auto inv_of = [&](float pm, float am) { return am >= eps ? 1.0f / pm : rstd * (1.0f / eps); };
    if (group) {  // a group is gl neighbouring lanes' chunks; groups divide H, so there is no tail
        const int gl = group / kVec;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            if (j * TPR >= chunks) break;  // uniform
            float pm = 0.0f;
#pragma unroll
            for (int e = 0; e < kVec; ++e) pm = fmaxf(pm, fabsf(p[j][e]));
            for (int d = gl / 2; d > 0; d >>= 1) pm = fmaxf(pm, __shfl_xor(pm, d, kWave));
            const int c = tr + j * TPR;
            if (c >= chunks) continue;
            const float am = pm * rstd;
            const uint64_t code = quant8(p[j], inv_of(pm, am), fp8);
            __builtin_memcpy(q + c * kVec, &code, sizeof code);
            if ((tr & (gl - 1)) == 0) scale[c * kVec / group] = fmaxf(am, eps) * top_inv;
        }
        return;
    }
    const float am = mx * rstd, inv = inv_of(mx, am);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = tr + j * TPR;
        if (c >= chunks) break;
        const uint64_t code = quant8(p[j], inv, fp8);
        __builtin_memcpy(q + c * kVec, &code, sizeof code);
    }
    if (TAIL && tail)
        q[it] = static_cast<uint8_t>(fp8 ? quant4<true>(pt, 0.0f, 0.0f, 0.0f, inv) : quant4<false>(pt, 0.0f, 0.0f, 0.0f, inv));
    if (tr == 0) *scale = fmaxf(am, eps) * top_inv;
}

}  // namespace moe
