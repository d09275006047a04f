// Router: logits, scores and top-k choice of experts.
//
//   l[t,e] = sum_h x[t,h] * W[e,h];  s = score(l)
//   ids: the K largest of s + bias (of l without bias), ties to the lowest id
//   scales: s of the chosen, normalised, times route_scale
//
// Ids are whole numbers that decide which experts run: a sum whose last bit
// depends on its order would make them depend on the tiling, the batch size
// and the split of H. Products and sums are therefore fp64 (a product of two
// fp32 values is exact in it), where neighbouring logits of real inputs never
// lie within rounding of each other, and rounded once, to fp32 weights.
//
// Two launches: the logits, into the workspace, and one wave per token for
// scores and choice.
#include "internal.h"

#include "../../include/moe_w8a8.h"

namespace moe {
namespace {

constexpr int kVec = 8;
constexpr int kBlock = 256;

template <typename T>
__device__ __forceinline__ void load8(const T *p, int left, float (&v)[kVec]) {
    T raw[kVec];
    if (left >= kVec) {
        __builtin_memcpy(raw, p, sizeof raw);
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = to_f32(raw[e]);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) v[e] = e < left ? to_f32(p[e]) : 0.0f;
    }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
    return v;
}
__device__ __forceinline__ double wave_max(double v) {
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) v = fmax(v, __shfl_xor(v, d, kWave));
    return v;
}

// One wave per (token, expert).
template <typename T, typename W>
__global__ __launch_bounds__(kBlock) void logits_kernel(GateArgs a) {
    const int lane = threadIdx.x & (kWave - 1);
    const int e = blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave;
    if (e >= a.E) return;
    for (int t = blockIdx.y; t < a.T; t += gridDim.y) {
        const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(t) * a.H;
        const W *w = static_cast<const W *>(a.weight) + static_cast<size_t>(e) * a.H;
        double sum = 0.0;
        for (int i = lane * kVec; i < a.H; i += kWave * kVec) {
            float u[kVec], v[kVec];
            load8(x + i, a.H - i, u);
            load8(w + i, a.H - i, v);
#pragma unroll
            for (int j = 0; j < kVec; ++j) sum = fma(static_cast<double>(u[j]), static_cast<double>(v[j]), sum);
        }
        sum = wave_sum(sum);
        if (lane == 0) a.logits[static_cast<size_t>(t) * a.E + e] = sum;
    }
}

// Score of a logit (softmax: before the division by the sum; m = the largest
// logit).
__device__ __forceinline__ double score_of(int score, double l, double m) {
    if (score == MOE_SCORE_SOFTMAX) return exp(l - m);
    if (score == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
    return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}

// One wave per token; lane l holds experts l, l + 64, ... (NPL of them).
template <int NPL>
__global__ __launch_bounds__(kBlock) void choose_kernel(GateArgs a) {
    const int lane = threadIdx.x & (kWave - 1);
    const int t = blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave;
    if (t >= a.T) return;
    const double none = -__builtin_inf();
    double s[NPL], c[NPL];  // scores, and what the choice goes by
    double m = none;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const int e = j * kWave + lane;
        s[j] = e < a.E ? a.logits[static_cast<size_t>(t) * a.E + e] : none;
        m = fmax(m, s[j]);
    }
    if (a.score == MOE_SCORE_SOFTMAX) m = wave_max(m);
    double total = 0.0;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const int e = j * kWave + lane;
        const double l = s[j];
        s[j] = e < a.E ? score_of(a.score, l, m) : 0.0;
        total += s[j];
        c[j] = l;
    }
    if (a.score == MOE_SCORE_SOFTMAX) {
        total = wave_sum(total);
#pragma unroll
        for (int j = 0; j < NPL; ++j) s[j] = s[j] / total;
    }
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const int e = j * kWave + lane;
        if (a.bias && e < a.E) c[j] = s[j] + static_cast<double>(a.bias[e]);
        if (e >= a.E || !(c[j] > none)) c[j] = none;  // NaN is never chosen
    }
    double w_mine = 0.0, w_sum = 0.0;  // lane k keeps the k-th choice
    int id_mine = -1;
    for (int k = 0; k < a.K; ++k) {
        double best = none, best_s = 0.0;
        int best_e = 0x7FFFFFFF;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            if (c[j] > best) {
                best = c[j];
                best_s = s[j];
                best_e = j * kWave + lane;
            }
        }
#pragma unroll
        for (int d = kWave / 2; d > 0; d >>= 1) {
            const double oc = __shfl_xor(best, d, kWave), os = __shfl_xor(best_s, d, kWave);
            const int oe = __shfl_xor(best_e, d, kWave);
            if (oc > best || (oc == best && oe < best_e)) {
                best = oc;
                best_s = os;
                best_e = oe;
            }
        }
        if (!(best > none)) break;  // uniform: nothing is left
#pragma unroll
        for (int j = 0; j < NPL; ++j)
            if (j * kWave + lane == best_e) c[j] = none;
        w_sum += best_s;
        if (lane == k) {
            w_mine = best_s;
            id_mine = best_e;
        }
    }
    if (lane < a.K) {
        double w = w_mine;
        if (a.normalize && w_sum > 0.0) w = w / w_sum;
        w = w * static_cast<double>(a.route_scale);
        const size_t o = static_cast<size_t>(t) * a.K + lane;
        a.ids[o] = id_mine;
        a.scales[o] = id_mine < 0 ? 0.0f : static_cast<float>(w);
    }
}

template <typename T, typename W>
hipError_t launch_logits(const GateArgs &a, hipStream_t s) {
    const dim3 grid((a.E + kBlock / kWave - 1) / (kBlock / kWave), a.T < 4096 ? a.T : 4096);
    hipLaunchKernelGGL((logits_kernel<T, W>), grid, dim3(kBlock), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t gate_workspace(int T, int E, int H) {
    (void)H;
    return static_cast<size_t>(T) * E * sizeof(double);
}

hipError_t launch_gate(const GateArgs &a, hipStream_t s) {
    hipError_t e;
    if (a.dtype == MOE_DTYPE_BF16)
        e = a.weight_dtype == MOE_DTYPE_BF16 ? launch_logits<Bf16, Bf16>(a, s) : launch_logits<Bf16, float>(a, s);
    else if (a.dtype == MOE_DTYPE_FP16)
        e = a.weight_dtype == MOE_DTYPE_FP16   ? launch_logits<Fp16, Fp16>(a, s)
            : a.weight_dtype == MOE_DTYPE_BF16 ? launch_logits<Fp16, Bf16>(a, s)
                                               : launch_logits<Fp16, float>(a, s);
    else
        e = a.weight_dtype == MOE_DTYPE_BF16 ? launch_logits<float, Bf16>(a, s) : launch_logits<float, float>(a, s);
    if (e != hipSuccess) return e;
    const dim3 grid((a.T + kBlock / kWave - 1) / (kBlock / kWave)), blk(kBlock);
    if (a.E <= kWave) hipLaunchKernelGGL((choose_kernel<1>), grid, blk, 0, s, a);
    else if (a.E <= 4 * kWave) hipLaunchKernelGGL((choose_kernel<4>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((choose_kernel<16>), grid, blk, 0, s, a);
    return hipGetLastError();
}

}  // namespace moe
