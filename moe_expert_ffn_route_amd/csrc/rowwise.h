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
__device__ __forceinline__ void store8(T *p, const float (&v)[kVec], bool streamed = false) {
    T raw[kVec];
#pragma unroll
    for (int e = 0; e < kVec; ++e) from_f32(v[e], raw[e]);
    store_out(p, raw, streamed);
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
// DPP on both words of an fp64; lanes that nothing reaches take zero.
template <int CTRL, int ROWS = 0xF>
__device__ __forceinline__ double dpp_or_zero(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xF, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xF, false);
    return __builtin_bit_cast(double, lo | (static_cast<uint64_t>(hi) << 32));
}
__device__ __forceinline__ double last_lane_sum(double v) {
    v += dpp_or_zero<0x111>(v);
    v += dpp_or_zero<0x112>(v);
    v += dpp_or_zero<0x114>(v);
    v += dpp_or_zero<0x118>(v);
    v += dpp_or_zero<0x142, 0xA>(v);
    v += dpp_or_zero<0x143, 0xC>(v);
    return v;
}

// The join of the values of a row of 16 lanes, in each of them: mirrors of the
// row and of its halves, pairs, neighbours.
template <int CTRL>
__device__ __forceinline__ float swapped(float v) { return dpp_or<CTRL>(v, 0.0f); }
template <int CTRL>
__device__ __forceinline__ double swapped(double v) { return dpp_or_zero<CTRL>(v); }
template <typename V, typename Join>
__device__ __forceinline__ V join_lanes(V v, Join join) {
    v = join(v, swapped<0x140>(v));
    v = join(v, swapped<0x141>(v));
    v = join(v, swapped<0x4E>(v));
    return join(v, swapped<0xB1>(v));
}

// The same for the workgroup of a row, of `waves` waves (at most 16): lane 63's
// values meet in `slot`, and each lane of a row of 16 takes one. With a barrier.
template <typename V, typename Join>
__device__ __forceinline__ V join_waves(V v, V *slot, int tr, int waves, V none, Join join) {
    if ((tr & (kWave - 1)) == kWave - 1) slot[tr / kWave] = v;
    __syncthreads();
    const int i = tr & 15;
    return join_lanes(i < waves ? slot[i] : none, join);
}

// Eight codes of a row, quant4's bits: t = (v * Q) * inv, brought to [-Q, Q]
// (where v * Q leaves fp32) and rounded to nearest even, int8 by an addition
// whose sum's last bits are the integer, E4M3 by the hardware's conversion,
// which gives e4m3_code's bits for every fp32 of up to 464 (the codes of all
// fp32 up to a row's largest are checked by tests/test_gpu_conversions.py). A NaN gives -127 (the median of three is the smaller one then), or
// E4M3's NaN without a sign, for which a lane that has one takes quant4.
__device__ __forceinline__ uint64_t quant8(const float (&v)[kVec], float inv, bool fp8) {
    uint32_t w[2];
    if (fp8) {
        float t[kVec];
        bool nan = false;
#pragma unroll
        for (int e = 0; e < kVec; ++e) t[e] = v[e] * kQMax<true> * inv;
#pragma unroll
        for (int e = 0; e < kVec; e += 2) nan |= __builtin_isunordered(t[e], t[e + 1]);
#pragma unroll
        for (int e = 0; e < kVec; ++e) t[e] = __builtin_amdgcn_fmed3f(t[e], -kQMax<true>, kQMax<true>);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(t[4 * h], t[4 * h + 1], 0, false);
            w[h] = static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(t[4 * h + 2], t[4 * h + 3], lo, true));
        }
        if (nan) {
#pragma unroll
            for (int h = 0; h < 2; ++h) w[h] = quant4<true>(v[4 * h], v[4 * h + 1], v[4 * h + 2], v[4 * h + 3], inv);
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t b[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float t = __builtin_amdgcn_fmed3f(v[4 * h + e] * kQMax<false> * inv, -kQMax<false>, kQMax<false>);
                b[e] = __float_as_uint(t + 12582912.0f);  // 1.5 * 2^23
            }
            const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0C);
            w[h] = lo | hi;
        }
    }
    return w[0] | (static_cast<uint64_t>(w[1]) << 32);
}

// Maximum over aligned runs of 8, 16 or 32 lanes, in all of them: DPP swaps of
// neighbours and of pairs, the mirrors of half rows and rows, and one shuffle.
template <int CTRL>
__device__ __forceinline__ float dpp_max(float v) {
    return fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xF, 0xF, true)));
}
__device__ __forceinline__ float run_max(float v, int lanes) {
    v = dpp_max<0xB1>(v);
    v = dpp_max<0x4E>(v);
    v = dpp_max<0x141>(v);
    if (lanes >= 16) v = dpp_max<0x140>(v);
    if (lanes >= 32) v = fmaxf(v, __shfl_xor(v, 16, kWave));
    return v;
}

// Rows per workgroup: four of one wave each, or one.
template <int TPR>
constexpr int kRows = TPR == kWave ? 4 : 1;

// Codes and scales of the row's p (zero behind its end) times rstd, mx = max|p|.
// Thread tr of tpr holds chunks tr + j * tpr and, TAIL, element `it` if `tail`.
template <int CH, bool TAIL>
__device__ __forceinline__ void write_codes(const float (&p)[CH][kVec], float pt, float mx, float rstd, float eps,
                                            bool fp8, int group, int H, int tr, int tpr, bool tail, int it, uint8_t *q,
                                            float *scale, bool streamed = false) {
    const int chunks = H / kVec;
    const float top_inv = fp8 ? 1.0f / kQMax<true> : 1.0f / kQMax<false>;
    auto inv_of = [&](float pm, float am) { return am >= eps ? 1.0f / pm : rstd * (1.0f / eps); };
    if (group) {  // a group is gl neighbouring lanes' chunks; groups divide H, so there is no tail
        const int gl = group / kVec;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            if (j * tpr >= chunks) break;  // uniform
            float pm = 0.0f;
#pragma unroll
            for (int e = 0; e < kVec; ++e) pm = fmaxf(pm, fabsf(p[j][e]));
            pm = run_max(pm, gl);
            const int c = tr + j * tpr;
            if (c >= chunks) continue;
            const float am = pm * rstd;
            const uint64_t code = quant8(p[j], inv_of(pm, am), fp8);
            store_out(q + c * kVec, code, streamed);
            if ((tr & (gl - 1)) == 0) scale[c * kVec / group] = fmaxf(am, eps) * top_inv;
        }
        return;
    }
    const float am = mx * rstd, inv = inv_of(mx, am);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        const int c = tr + j * tpr;
        if (c >= chunks) break;
        const uint64_t code = quant8(p[j], inv, fp8);
        store_out(q + c * kVec, code, streamed);

    }
    if (TAIL && tail)
        q[it] = static_cast<uint8_t>(fp8 ? quant4<true>(pt, 0.0f, 0.0f, 0.0f, inv) : quant4<false>(pt, 0.0f, 0.0f, 0.0f, inv));
    if (tr == 0) *scale = fmaxf(am, eps) * top_inv;
}

}  // namespace moe
