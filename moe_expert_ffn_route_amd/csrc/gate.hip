// Router: logits, scores and top-k choice of experts.
//
//   l[t,e] = sum_h x[t,h] * W[e,h];  s = score(l)
//   ids: the K largest of s + bias (of l without bias), ties to the lowest id
//   scales: s of the chosen, normalised, times route_scale
//
// Ids are whole numbers that decide which experts run: a sum whose last bits
// depend on its order would make them depend on the tiling, the batch size
// and the split of H. They are therefore those of 64-bit logits, in one of
// two ways:
//   - x and W both bf16, or both fp16: MFMA with fp32 sums over 128 products,
//     which are added up in fp64. Beside them the MFMA makes the sums of
//     |x * w|, which bound how far such a logit is off (kGamma). Where the
//     bound leaves open which of two experts comes first, the choice kernel
//     computes the logits of those experts again, in fp64.
//   - other types: fp64 MFMA throughout (their products are exact in it).
//
// Two launches: the logits, in up to kMaxSplit parts of H, into the
// workspace; and one wave per token, which adds the parts in order, for
// scores and choice.
#include "internal.h"

#include "../../include/moe_w8a8.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef double v4d __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));

constexpr int kVec = 8;      // elements per lane and load
constexpr int kStep = 32;    // h per load of a 16-row tile
constexpr int kChunk = 128;  // products per fp32 sum
constexpr int kBlock = 256;
constexpr int kMaxSplit = 16;
// An fp32 sum of 128 products that are themselves exact, in any order, with
// every addition off by at most one unit in the last place (an adder that
// truncates): 128 * 2^-23 of the sum of magnitudes.
constexpr double kGamma = 1.0 / 65536.0;
// Products under the smallest normal fp32 may be dropped: 16384 of them.
constexpr double kTiny = 0x1p-110;

// Eight elements from h = k of a row of H.
template <typename T>
__device__ __forceinline__ void load8(const T *row, int k, int H, T (&raw)[kVec]) {
    if (k + kVec <= H) {
        __builtin_memcpy(raw, row + k, sizeof raw);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            raw[e] = T{};
            if (k + e < H) raw[e] = row[k + e];
        }
    }
}

template <typename T>
constexpr bool kIs16 = sizeof(T) == 2;
template <typename T, typename W>
constexpr bool kFast = false;
template <>
constexpr bool kFast<Bf16, Bf16> = true;
template <>
constexpr bool kFast<Fp16, Fp16> = true;

template <typename T>
__device__ __forceinline__ v4f mfma32(v4i a, v4i b, v4f c) {
    if constexpr (__is_same(T, Bf16))
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
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

// Part blockIdx.z of the logits of 16 * TM * WM tokens (A rows) and
// 16 * TN * WN experts (B columns). The four waves of a workgroup are WM x WN
// tiles, and WK slices of the part's H, joined in LDS. Lane l loads row
// l % 16, eight h from 8 * (l / 16) of each step.
template <typename T, typename W, int TM, int TN, int WM, int WN, int WK>
__global__ __launch_bounds__(kBlock) void logits_kernel(GateArgs a, int chunks_per_part) {
    static_assert(WM * WN * WK * kWave == kBlock, "four waves");
    constexpr bool FAST = kFast<T, W>;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int r = lane & 15, kq = lane >> 4;
    const int wk = wave % WK, wn = wave / WK % WN, wm = wave / (WK * WN);
    const int t0 = (blockIdx.y * WM + wm) * 16 * TM, e0 = (blockIdx.x * WN + wn) * 16 * TN;
    // rows past the end read the last one; their results are not stored
    const T *xr[TM];
    const W *wr[TN];
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int t = t0 + i * 16 + r;
        xr[i] = static_cast<const T *>(a.x) + static_cast<size_t>(t < a.T ? t : a.T - 1) * a.H;
    }
#pragma unroll
    for (int j = 0; j < TN; ++j) {
        const int e = e0 + j * 16 + r;
        wr[j] = static_cast<const W *>(a.weight) + static_cast<size_t>(e < a.E ? e : a.E - 1) * a.H;
    }
    v4d sum[TM][TN];
    v4f mag[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) {
            sum[i][j] = v4d{0.0, 0.0, 0.0, 0.0};
            mag[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        }
    const int c_end = min((static_cast<int>(blockIdx.z) + 1) * chunks_per_part, (a.H + kChunk - 1) / kChunk);
    for (int c = blockIdx.z * chunks_per_part + wk; c < c_end; c += WK) {
        if constexpr (FAST) {
            v4i xf[TM][kChunk / kStep], wf[TN][kChunk / kStep];
#pragma unroll
            for (int s = 0; s < kChunk / kStep; ++s) {
                const int k = c * kChunk + s * kStep + kq * kVec;
#pragma unroll
                for (int i = 0; i < TM; ++i) {
                    T raw[kVec];
                    load8(xr[i], k, a.H, raw);
                    __builtin_memcpy(&xf[i][s], raw, sizeof raw);
                }
#pragma unroll
                for (int j = 0; j < TN; ++j) {
                    W raw[kVec];
                    load8(wr[j], k, a.H, raw);
                    __builtin_memcpy(&wf[j][s], raw, sizeof raw);
                }
            }
            v4f acc[TM][TN];
#pragma unroll
            for (int s = 0; s < kChunk / kStep; ++s)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = mfma32<T>(xf[i][s], wf[j][s], s == 0 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j]);
#pragma unroll
            for (int s = 0; s < kChunk / kStep; ++s) {
#pragma unroll
                for (int i = 0; i < TM; ++i) xf[i][s] &= 0x7FFF7FFF;
#pragma unroll
                for (int j = 0; j < TN; ++j) wf[j][s] &= 0x7FFF7FFF;
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j) mag[i][j] = mfma32<T>(xf[i][s], wf[j][s], mag[i][j]);
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
#pragma unroll
                    for (int q = 0; q < 4; ++q) sum[i][j][q] += static_cast<double>(acc[i][j][q]);
        } else {
#pragma unroll
            for (int s = 0; s < kChunk / kStep; ++s) {
                const int k = c * kChunk + s * kStep + kq * kVec;
                T xv[TM][kVec];
                W wv[TN][kVec];
#pragma unroll
                for (int i = 0; i < TM; ++i) load8(xr[i], k, a.H, xv[i]);
#pragma unroll
                for (int j = 0; j < TN; ++j) load8(wr[j], k, a.H, wv[j]);
                // the MFMA takes four h, one per lane quarter: h = 8 kq + e for step e
#pragma unroll
                for (int e = 0; e < kVec; ++e)
#pragma unroll
                    for (int i = 0; i < TM; ++i)
#pragma unroll
                        for (int j = 0; j < TN; ++j)
                            sum[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(
                                static_cast<double>(to_f32(xv[i][e])), static_cast<double>(to_f32(wv[j][e])),
                                sum[i][j], 0, 0, 0);
            }
        }
    }
    if constexpr (WK > 1) {
        __shared__ v4d s_sum[WK - 1][kWave];
        __shared__ v4f s_mag[WK - 1][kWave];
        static_assert(WM * WN * TM * TN == 1, "one tile per wave");
        if (wk > 0) {
            s_sum[wk - 1][lane] = sum[0][0];
            s_mag[wk - 1][lane] = mag[0][0];
        }
        __syncthreads();
        if (wk > 0) return;
#pragma unroll
        for (int w = 0; w < WK - 1; ++w) {
            sum[0][0] += s_sum[w][lane];
            mag[0][0] += s_mag[w][lane];
        }
    }
    const size_t part = static_cast<size_t>(blockIdx.z) * a.T * a.E;
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // result registers: fp32 D rows 4 * (l / 16) + q, fp64 D rows l / 16 + 4 * q
                const int t = t0 + i * 16 + (FAST ? 4 * kq + q : kq + 4 * q), e = e0 + j * 16 + r;
                if (t < a.T && e < a.E) {
                    const size_t o = part + static_cast<size_t>(t) * a.E + e;
                    a.logits[o] = sum[i][j][q];
                    if (FAST) a.mags[o] = mag[i][j][q];
                }
            }
}

// The logit of expert e in fp64, by the whole wave.
template <typename T, typename W>
__device__ double exact_logit(const GateArgs &a, int t, int e, int lane) {
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(t) * a.H;
    const W *w = static_cast<const W *>(a.weight) + static_cast<size_t>(e) * a.H;
    double sum = 0.0;
    for (int i = lane * kVec; i < a.H; i += kWave * kVec) {
        T u[kVec];
        W v[kVec];
        load8(x, i, a.H, u);
        load8(w, i, a.H, v);
#pragma unroll
        for (int j = 0; j < kVec; ++j)
            sum = fma(static_cast<double>(to_f32(u[j])), static_cast<double>(to_f32(v[j])), sum);
    }
    return wave_sum(sum);
}

// Score of a logit (softmax: before the division by the sum; m = the largest
// logit).
__device__ __forceinline__ double score_of(int score, double l, double m) {
    if (score == MOE_SCORE_SOFTMAX) return exp(l - m);
    if (score == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
    return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}

// Largest value of the wave and its lowest expert (0x7FFFFFFF: all -infinity).
template <int NPL>
__device__ __forceinline__ void wave_best(const double (&c)[NPL], int lane, double &best, int &best_e) {
    best = -__builtin_inf();
    best_e = 0x7FFFFFFF;
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        if (c[j] > best) {
            best = c[j];
            best_e = j * kWave + lane;
        }
    }
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) {
        const double oc = __shfl_xor(best, d, kWave);
        const int oe = __shfl_xor(best_e, d, kWave);
        if (oc > best || (oc == best && oe < best_e)) {
            best = oc;
            best_e = oe;
        }
    }
}

// One wave per token; lane l holds experts l, l + 64, ... (NPL of them).
template <typename T, typename W, int NPL>
__global__ __launch_bounds__(kBlock) void choose_kernel(GateArgs a, int parts) {
    constexpr bool FAST = kFast<T, W>;
    const int lane = threadIdx.x & (kWave - 1);
    const int t = blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave;
    if (t >= a.T) return;
    const double none = -__builtin_inf();
    double l[NPL], s[NPL], c[NPL];  // logits, scores, and what the choice goes by
    float mag = 0.0f;               // largest sum of |x * w|
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const int e = j * kWave + lane;
        double v = 0.0;
        float b = 0.0f;
        if (e < a.E) {
            for (int p = 0; p < parts; ++p) {
                const size_t o = (static_cast<size_t>(p) * a.T + t) * a.E + e;
                v += a.logits[o];
                if (FAST) b += a.mags[o];
            }
        }
        l[j] = e < a.E ? v : none;
        mag = fmaxf(mag, b);
    }
    // choice values of every expert, from the logits
    auto values = [&] {
        double m = none, total = 0.0;
        if (a.score == MOE_SCORE_SOFTMAX) {
#pragma unroll
            for (int j = 0; j < NPL; ++j) m = fmax(m, l[j]);
            m = wave_max(m);
        }
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            s[j] = j * kWave + lane < a.E ? score_of(a.score, l[j], m) : 0.0;
            total += s[j];
        }
        if (a.score == MOE_SCORE_SOFTMAX) {
            total = wave_sum(total);
#pragma unroll
            for (int j = 0; j < NPL; ++j) s[j] = s[j] / total;
        }
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            const int e = j * kWave + lane;
            c[j] = a.bias && e < a.E ? s[j] + static_cast<double>(a.bias[e]) : l[j];
            if (e >= a.E || !(c[j] > none)) c[j] = none;  // NaN is never chosen
        }
    };
    values();
    if constexpr (FAST) {
        // How far two choice values may be off together. Slopes: sigmoid 1/4,
        // sqrt(softplus) under 1/3; a softmax share moves by at most twice its
        // logits' error.
        double off = 2.0 * (kGamma * 1.01 * wave_max(static_cast<double>(mag)) + kTiny);
        if (a.bias) off *= a.score == MOE_SCORE_SOFTMAX ? 2.5 : a.score == MOE_SCORE_SIGMOID ? 0.25 : 0.34;
        off += 1e-13;
        // K + 1 choices in order; an expert that is closer than `off` to one of
        // them is marked, and so is that one
        double left[NPL];
        uint32_t marked = 0;  // bit j: expert j * 64 + lane
#pragma unroll
        for (int j = 0; j < NPL; ++j) left[j] = c[j];
        for (int k = 0; k < a.K; ++k) {
            double best;
            int best_e;
            wave_best(left, lane, best, best_e);
            if (!(best > none)) break;
            bool close = false;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                if (j * kWave + lane == best_e) {
                    left[j] = none;
                } else if (left[j] > best - off) {
                    marked |= 1u << j;
                    close = true;
                }
            }
            if (__ballot(close)) {
#pragma unroll
                for (int j = 0; j < NPL; ++j)
                    if (j * kWave + lane == best_e) marked |= 1u << j;
            }
        }
        if (__ballot(marked != 0)) {
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                unsigned long long todo = __ballot((marked >> j) & 1u);
                while (todo) {
                    const int who = __builtin_ctzll(todo);
                    todo &= todo - 1;
                    const double v = exact_logit<T, W>(a, t, j * kWave + who, lane);
                    if (lane == who) l[j] = v;
                }
            }
            values();
        }
    }
    double w_mine = 0.0, w_sum = 0.0;  // lane k keeps the k-th choice
    int id_mine = -1;
    for (int k = 0; k < a.K; ++k) {
        double best;
        int best_e;
        wave_best(c, lane, best, best_e);
        if (!(best > none)) break;  // uniform: nothing is left
        double v = 0.0;
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            if (best_e / kWave == j) v = s[j];
            if (j * kWave + lane == best_e) c[j] = none;
        }
        v = __shfl(v, best_e & (kWave - 1), kWave);
        w_sum += v;
        if (lane == k) {
            w_mine = v;
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

// Parts of H: enough workgroups to give every CU one, of at least two chunks
// per wave slice each.
struct Plan {
    int small;  // up to 16 tokens: one 16 x 16 tile per workgroup, its waves split H
    dim3 grid;
    int chunks_per_part, parts;
};
Plan plan_of(int T, int E, int H) {
    Plan p;
    p.small = T <= 16;
    const int tile = p.small ? 16 : 64, slices = p.small ? 4 : 1;
    p.grid = dim3((E + tile - 1) / tile, (T + tile - 1) / tile);
    const int chunks = (H + kChunk - 1) / kChunk;
    const int blocks = static_cast<int>(p.grid.x * p.grid.y);
    int parts = (256 + blocks - 1) / blocks;
    if (parts > kMaxSplit) parts = kMaxSplit;
    if (parts > chunks / (2 * slices)) parts = chunks / (2 * slices);
    if (parts < 1) parts = 1;
    p.chunks_per_part = (chunks + parts - 1) / parts;
    p.parts = (chunks + p.chunks_per_part - 1) / p.chunks_per_part;
    p.grid.z = p.parts;
    return p;
}

template <typename T, typename W>
hipError_t launch(const GateArgs &a, hipStream_t s) {
    const Plan p = plan_of(a.T, a.E, a.H);
    GateArgs g = a;
    g.mags = reinterpret_cast<float *>(a.logits + static_cast<size_t>(p.parts) * a.T * a.E);
    if (p.small)
        hipLaunchKernelGGL((logits_kernel<T, W, 1, 1, 1, 1, 4>), p.grid, dim3(kBlock), 0, s, g, p.chunks_per_part);
    else
        hipLaunchKernelGGL((logits_kernel<T, W, 2, 2, 2, 2, 1>), p.grid, dim3(kBlock), 0, s, g, p.chunks_per_part);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const dim3 grid((a.T + kBlock / kWave - 1) / (kBlock / kWave)), blk(kBlock);
    if (a.E <= kWave) hipLaunchKernelGGL((choose_kernel<T, W, 1>), grid, blk, 0, s, g, p.parts);
    else if (a.E <= 4 * kWave) hipLaunchKernelGGL((choose_kernel<T, W, 4>), grid, blk, 0, s, g, p.parts);
    else hipLaunchKernelGGL((choose_kernel<T, W, 16>), grid, blk, 0, s, g, p.parts);
    return hipGetLastError();
}

}  // namespace

size_t gate_workspace(int T, int E, int H) {
    if (T == 0) return 0;
    return static_cast<size_t>(plan_of(T, E, H).parts) * T * E * (sizeof(double) + sizeof(float));
}

hipError_t launch_gate(const GateArgs &a, hipStream_t s) {
    if (a.dtype == MOE_DTYPE_BF16)
        return a.weight_dtype == MOE_DTYPE_BF16 ? launch<Bf16, Bf16>(a, s) : launch<Bf16, float>(a, s);
    if (a.dtype == MOE_DTYPE_FP16)
        return a.weight_dtype == MOE_DTYPE_FP16   ? launch<Fp16, Fp16>(a, s)
               : a.weight_dtype == MOE_DTYPE_BF16 ? launch<Fp16, Bf16>(a, s)
                                                  : launch<Fp16, float>(a, s);
    return a.weight_dtype == MOE_DTYPE_BF16 ? launch<float, Bf16>(a, s) : launch<float, float>(a, s);
}

}  // namespace moe
