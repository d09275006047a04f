// Two operators on rows: the quantiser of an activation, and the norm that
// joins a block's outputs to the residual stream.
//
// Codes follow the block's rule (rowquant.h). As in norm.hip, those of y = p *
// rstd come from p and max|p| alone, so that rstd enters only the scales (and
// the codes of rows under the amax floor). The branch's own norm does enter p.
// Both mean squares are summed in fp64 and 1 / sqrt rounded once to fp32, so
// that every output is the same whatever the order of these sums, which is the
// batch's (it decides only sums within 2^-50 or so of a rounding border of
// 1 / sqrt). An fp32 sum of the second changed y with the batch and was no
// faster than by 2 % (us, fp64 / fp32, H 4096: T 8 3.6 / 3.7, T 500 7.0 / 6.9, T
// 8192 64.8 / 64.8).
//
// A row of up to 16384 elements stays in the registers of one workgroup
// between the one read of its inputs and the writes: what bounds both
// operators is memory. In us: quantiser T 8192, H 4096, bf16, groups of 128 16.5
// (6.1 TB/s of reads and writes); joining norm T 4001, H 5003, fp16, post norm
// and gate, y and E4M3 codes 43.9 to 45.7 (3.9 to 4.1 TB/s: rows start at odd
// addresses); at T 8 both 4 to 4.5, a launch and its round trips.
#include "rowwise.h"

#include <type_traits>

#include "../../include/moe_w8a8.h"

namespace moe {
namespace {

__device__ __forceinline__ float lane63(float v) {
    return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), kWave - 1));
}
__device__ __forceinline__ double lane63(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), kWave - 1);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), kWave - 1);
    return __builtin_bit_cast(double, lo | (static_cast<uint64_t>(hi) << 32));
}
// 1 / sqrt(v), rounded once to fp32: the hardware's fp64 estimate y, off by
// some 2^-23, and with e = 1 - v y^2 three terms of y (1 - e)^(-1/2), whose rest
// (5/16 e^3) is under 2^-65: what is left are fp64 roundings. (With a root and a
// division, and sums by shuffles instead of DPP: T 8, H 4096 4.03 us, now 3.65.)
__device__ __forceinline__ float root_of(double v) {
    const double y = __builtin_amdgcn_rsq(v), e = __builtin_fma(-v * y, y, 1.0);
    return static_cast<float>(__builtin_fma(y * e, __builtin_fma(e, 0.375, 0.5), y));
}
__device__ __forceinline__ void add_squares(const float (&v)[kVec], double &sum) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) sum = __builtin_fma(static_cast<double>(v[e]), static_cast<double>(v[e]), sum);
}

// A workgroup is one row, its threads as many whole waves as CH chunks of kVec
// elements each need, or (ONE) four rows of one wave each. TAIL: H is no
// multiple of kVec. Loads stand behind no branch: lanes past the row's end
// read its last chunk again and count nothing.
template <int CH, bool ONE>
constexpr int kMost = ONE ? 4 * kWave : 1024;
template <typename T, int CH, bool TAIL, bool ONE>
__global__ __launch_bounds__((kMost<CH, ONE>)) void quant_kernel(QuantArgs a) {
    const int tpr = ONE ? kWave : static_cast<int>(blockDim.x), waves = tpr / kWave;
    const int tr = ONE ? threadIdx.x % kWave : threadIdx.x, row = ONE ? blockIdx.x * 4 + threadIdx.x / kWave : blockIdx.x;
    if (ONE && row >= a.T) return;  // whole waves, and such a row has no barrier
    const size_t base = static_cast<size_t>(row) * a.H;
    const T *x = static_cast<const T *>(a.x) + base;
    const int chunks = a.H / kVec, rest = a.H % kVec;
    const bool tail = TAIL && tr < rest;
    const int it = TAIL ? chunks * kVec + min(tr, rest - 1) : 0;
    auto at = [&](int j) { return min(tr + j * tpr, chunks - 1) * kVec; };
    float p[CH][kVec] = {}, pt = 0.0f;
    if (!TAIL || chunks > 0) {
        float g[CH][kVec];
#pragma unroll
        for (int j = 0; j < CH; ++j) load8(x + at(j), p[j]);
        if (a.smooth) {
#pragma unroll
            for (int j = 0; j < CH; ++j) load8(a.smooth + at(j), g[j]);
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int e = 0; e < kVec; ++e) p[j][e] = p[j][e] * g[j][e];
        }
    }
    if (TAIL) {
        pt = to_f32(x[it]);
        if (a.smooth) pt = pt * a.smooth[it];
        if (!tail) pt = 0.0f;
    }
    float mx = fabsf(pt);
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if (tr + j * tpr >= chunks) {  // a branch that most waves do not take, not eight selections
#pragma unroll
            for (int e = 0; e < kVec; ++e) p[j][e] = 0.0f;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) mx = fmaxf(mx, fabsf(p[j][e]));
    }
    if (!a.group) {
        mx = last_lane_max(mx);
        __shared__ float s_max[16];
        if constexpr (ONE) mx = lane63(mx);
        else mx = join_waves(mx, s_max, tr, waves, 0.0f, [](float u, float v) { return fmaxf(u, v); });
    }
    write_codes<CH, TAIL>(p, pt, mx, 1.0f, a.amax_eps, a.quant == MOE_QUANT_E4M3, a.group, a.H, tr, tpr, tail, it,
                          static_cast<uint8_t *>(a.q) + base,
                          a.q_scale + static_cast<size_t>(row) * (a.group ? a.H / a.group : 1), a.streamed);
}

template <typename T, typename W, int CH, bool TAIL, bool ONE>
__global__ __launch_bounds__((kMost<CH, ONE>)) void join_norm_kernel(JoinNormArgs a) {
    __shared__ double s_sq[2][16];
    __shared__ float s_max[16];
    const int tpr = ONE ? kWave : static_cast<int>(blockDim.x), waves = tpr / kWave;
    const int tr = ONE ? threadIdx.x % kWave : threadIdx.x, row = ONE ? blockIdx.x * 4 + threadIdx.x / kWave : blockIdx.x;
    if (ONE && row >= a.T) return;  // whole waves, and such a row has no barrier
    const size_t base = static_cast<size_t>(row) * a.H;
    const T *block = static_cast<const T *>(a.block) + base, *share = static_cast<const T *>(a.share) + base;
    const T *res = static_cast<const T *>(a.residual) + base;
    const W *pw = static_cast<const W *>(a.post_weight), *w = static_cast<const W *>(a.weight);
    const W *gate = static_cast<const W *>(a.gate) + row * a.gate_stride;
    const int chunks = a.H / kVec, rest = a.H % kVec;
    const bool tail = TAIL && tr < rest, whole = !TAIL || chunks > 0;
    const int it = TAIL ? chunks * kVec + min(tr, rest - 1) : 0;
    auto at = [&](int j) { return min(tr + j * tpr, chunks - 1) * kVec; };

    // b, and what will be needed later on its way
    float p[CH][kVec] = {}, r[CH][kVec] = {}, pt = 0.0f, rt = 0.0f;
    const double inv_h = 1.0 / a.H;  // while the loads are under way
    const float ss = a.share_scale ? a.share_scale[row] : 1.0f;
    if (whole) {
#pragma unroll
        for (int j = 0; j < CH; ++j) load8(block + at(j), p[j]);
        if (a.share) {
            float v[CH][kVec];
#pragma unroll
            for (int j = 0; j < CH; ++j) load8(share + at(j), v[j]);
            if (a.residual) {
#pragma unroll
                for (int j = 0; j < CH; ++j) load8(res + at(j), r[j]);
            }
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int e = 0; e < kVec; ++e) p[j][e] = p[j][e] + v[j][e] * ss;
        } else if (a.residual) {
#pragma unroll
            for (int j = 0; j < CH; ++j) load8(res + at(j), r[j]);
        }
    }
    if (TAIL) {
        pt = to_f32(block[it]);
        if (a.share) pt = pt + to_f32(share[it]) * ss;
        if (a.residual) rt = to_f32(res[it]);
    }
    if (a.post_norm) {
        double sq = tail ? static_cast<double>(pt) * pt : 0.0;
#pragma unroll
        for (int j = 0; j < CH; ++j)
            if (tr + j * tpr < chunks) add_squares(p[j], sq);
        sq = last_lane_sum(sq);
        if constexpr (ONE) sq = lane63(sq);
        else sq = join_waves(sq, s_sq[0], tr, waves, 0.0, [](double u, double v) { return u + v; });
        const float rstd = root_of(sq * inv_h + static_cast<double>(a.post_eps));
        if (pw && whole) {
            float v[CH][kVec];
#pragma unroll
            for (int j = 0; j < CH; ++j) load8(pw + at(j), v[j]);
#pragma unroll
            for (int j = 0; j < CH; ++j)
#pragma unroll
                for (int e = 0; e < kVec; ++e) p[j][e] = p[j][e] * v[j][e];
        }
        if (TAIL && pw) pt = pt * to_f32(pw[it]);
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) p[j][e] = p[j][e] * rstd;
        pt = pt * rstd;
    }
    // r = residual * residual_scale + n * (gate * branch_scale), in p
    if (a.gate && whole) {
        float v[CH][kVec];
#pragma unroll
        for (int j = 0; j < CH; ++j) load8(gate + at(j), v[j]);
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) p[j][e] = p[j][e] * (v[j][e] * a.branch_scale);
    } else {
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) p[j][e] = p[j][e] * a.branch_scale;
    }
    if (TAIL) pt = pt * (a.gate ? to_f32(gate[it]) * a.branch_scale : a.branch_scale);
    if (a.residual) {
#pragma unroll
        for (int j = 0; j < CH; ++j)
#pragma unroll
            for (int e = 0; e < kVec; ++e) p[j][e] = r[j][e] * a.residual_scale + p[j][e];
        pt = rt * a.residual_scale + pt;
    }
    if (a.residual_out) {  // its row has been read by the threads that write it
        T *out = static_cast<T *>(a.residual_out) + base;
#pragma unroll
        for (int j = 0; j < CH; ++j)
            if (tr + j * tpr < chunks) store8(out + at(j), p[j], a.streamed);
        if (tail) from_f32(pt, out[it]);
    }
    if (!a.y && !a.q) return;  // uniform
    if (w && whole) {
#pragma unroll
        for (int j = 0; j < CH; ++j) load8(w + at(j), r[j]);
    }
    double sum = 0.0;
    float mx = 0.0f;
#pragma unroll
    for (int j = 0; j < CH; ++j) {
        if (tr + j * tpr >= chunks) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) p[j][e] = 0.0f;
        }
        add_squares(p[j], sum);
        if (w) {
#pragma unroll
            for (int e = 0; e < kVec; ++e) p[j][e] = p[j][e] * r[j][e];
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) mx = fmaxf(mx, fabsf(p[j][e]));
    }
    if (TAIL) {
        if (!tail) pt = 0.0f;
        sum = __builtin_fma(static_cast<double>(pt), static_cast<double>(pt), sum);
        if (tail && w) pt = pt * to_f32(w[it]);
        mx = fmaxf(mx, fabsf(pt));
    }
    sum = last_lane_sum(sum);
    mx = last_lane_max(mx);
    if constexpr (ONE) {
        sum = lane63(sum);
        mx = lane63(mx);
    } else {
        if ((tr & (kWave - 1)) == kWave - 1) s_max[tr / kWave] = mx;
        sum = join_waves(sum, s_sq[1], tr, waves, 0.0, [](double u, double v) { return u + v; });
        mx = join_lanes((tr & 15) < waves ? s_max[tr & 15] : 0.0f, [](float u, float v) { return fmaxf(u, v); });
    }
    const float rstd = root_of(sum * inv_h + static_cast<double>(a.rms_eps));
    if (a.y) {
        T *y = static_cast<T *>(a.y) + base;
#pragma unroll
        for (int j = 0; j < CH; ++j) {
            if (tr + j * tpr >= chunks) break;
            float v[kVec];
#pragma unroll
            for (int e = 0; e < kVec; ++e) v[e] = p[j][e] * rstd;
            store8(y + at(j), v, a.streamed);
        }
        if (tail) from_f32(pt * rstd, y[it]);
    }
    if (!a.q) return;
    write_codes<CH, TAIL>(p, pt, mx, rstd, a.amax_eps, a.quant == MOE_QUANT_E4M3, a.group, a.H, tr, tpr, tail, it,
                          static_cast<uint8_t *>(a.q) + base,
                          a.q_scale + static_cast<size_t>(row) * (a.group ? a.H / a.group : 1), a.streamed);
}

// f(CH, ONE) as constants, and the grid and workgroup that go with them. Short
// rows: one wave. Else as many waves as the row needs with one chunk a thread
// (few rows: the shortest way through) or two (many: more rows in flight for
// their registers). In us, one / two / four chunks: joining norm without post
// norm, bf16, H 4096, T 8 3.6 / 4.0 / 4.9, T 500 6.7 / 6.9 / 8.1, T 8192 68.1 /
// 67.3 / 73.4; with post norm and gate, fp16 to E4M3, H 5003, T 700 13.8 / 11.2 /
// 12.2, T 4001 68 / 56 / 59; quantiser, H 8192, T 3000 13.9 / 13.7 / 13.8.
template <typename F>
hipError_t by_length(int T, int H, F f) {
    const int chunks = H / kVec;
    if (chunks <= kWave) return f(std::integral_constant<int, 1>{}, std::true_type{}, dim3((T + 3) / 4), dim3(4 * kWave));
    auto wide = [&](auto ch) {
        const int threads = ((chunks + ch - 1) / ch + kWave - 1) / kWave * kWave;
        return f(ch, std::false_type{}, dim3(T), dim3(threads));
    };
    return T < 512 && chunks <= 1024 ? wide(std::integral_constant<int, 1>{}) : wide(std::integral_constant<int, 2>{});
}

template <typename T>
hipError_t quant_of(const QuantArgs &a, hipStream_t s) {
    return by_length(a.T, a.H, [&](auto ch, auto one, dim3 grid, dim3 blk) {
        if (a.H % kVec) hipLaunchKernelGGL((quant_kernel<T, ch, true, one>), grid, blk, 0, s, a);
        else hipLaunchKernelGGL((quant_kernel<T, ch, false, one>), grid, blk, 0, s, a);
        return hipGetLastError();
    });
}
template <typename T, typename W>
hipError_t join_of(const JoinNormArgs &a, hipStream_t s) {
    return by_length(a.T, a.H, [&](auto ch, auto one, dim3 grid, dim3 blk) {
        if (a.H % kVec) hipLaunchKernelGGL((join_norm_kernel<T, W, ch, true, one>), grid, blk, 0, s, a);
        else hipLaunchKernelGGL((join_norm_kernel<T, W, ch, false, one>), grid, blk, 0, s, a);
        return hipGetLastError();
    });
}

}  // namespace

hipError_t launch_quant(const QuantArgs &a, hipStream_t s) {
    switch (a.dtype) {
        case MOE_DTYPE_BF16: return quant_of<Bf16>(a, s);
        case MOE_DTYPE_FP16: return quant_of<Fp16>(a, s);
        default: return quant_of<float>(a, s);
    }
}

hipError_t launch_join_norm(const JoinNormArgs &a, hipStream_t s) {
    switch (a.dtype) {
        case MOE_DTYPE_BF16: return a.weight_dtype == MOE_DTYPE_FP32 ? join_of<Bf16, float>(a, s) : join_of<Bf16, Bf16>(a, s);
        case MOE_DTYPE_FP16: return a.weight_dtype == MOE_DTYPE_FP32 ? join_of<Fp16, float>(a, s) : join_of<Fp16, Fp16>(a, s);
        default: return join_of<float, float>(a, s);
    }
}

}  // namespace moe
