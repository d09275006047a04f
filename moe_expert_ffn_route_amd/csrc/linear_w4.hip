// Dense product with 4-bit weights on MFMA:
//
//   o[t,n] = xs[t] * sum_g s[n,g] * (sum_{k in g} (c[n,k] - z[n,g]) * x[t,k]) + bias[n]
//
// Weight rows are the MFMA's A rows, tokens its B columns: one 16 x 16 tile of
// D covers 16 output rows and 16 tokens, lane l holding rows 4 * (l / 16) ..+3
// of token l % 16. The 4-bit codes go to the matrix operand in few operations
// per eight of them:
//   fp16:  0x6400 | c is 1024 + c; minus (1024 + z), exact
//   bf16:  0x4300 | c is 128 + c, exact; the group's sum then carries
//          (128 + z) * sum(x), which is subtracted with the sum of x that one
//          more MFMA with a matrix of ones makes (per token tile, shared by
//          the weight tiles). bf16 has no packed subtraction here. The fp32
//          cancellation costs at most a factor of about 2^5 of fp32 rounding.
//   int8:  codes are packed as the nibble of c - 8; kept in a byte's high half
//          it is 16 * (c - 8) as int8. Zero points other than 8 are subtracted
//          with the int32 sum of x, as for bf16; the 16 divides out at the end,
//          exactly.
// A group's products are summed in the MFMA's fp32 (int8: exactly, in int32),
// scaled, and the groups are added in fp32.
//
// A workgroup takes 16 weight rows and all of K, its waves every kWaves-th tile of
// 128 k; their sums meet in LDS. No workspace, no atomics: results do not
// depend on timing.
#include "internal.h"

#include "../../include/moe_w8a8.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kTileK = 128;

// Position in a 128-k tile of element j (0..7) of code word d (0..3) of lane
// quarter kq: what the MFMA K steps of that group size read from the lane.
__host__ __device__ __forceinline__ int w4_k(int group, int kq, int d, int j) {
    return group == 32 ? d * 32 + kq * 8 + j : (d >> 1) * 64 + kq * 16 + (d & 1) * 8 + j;
}

// ------------------------------------------------------------------ packing
// One thread per 32-bit word of codes: tile (nt, kt), lane l, word d.
__global__ __launch_bounds__(256) void pack_codes_kernel(const uint8_t *__restrict__ src, uint32_t *__restrict__ dst,
                                                         LinearW4Args a) {
    const int64_t o = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // grid covers the words exactly
    const int d = static_cast<int>(o & 3), l = static_cast<int>(o >> 2) & 63;
    const int64_t tile = o >> 8;
    const int kt = static_cast<int>(tile % a.k_tiles), nt = static_cast<int>(tile / a.k_tiles);
    const int r = l & 15, kq = l >> 4;
    const int half = a.N / 2;
    const int unit = a.gated ? nt * 8 + r / 2 : nt * 16 + r;
    const bool row_ok = unit < (a.gated ? half : a.N);
    const int64_t row = a.gated && (r & 1) ? half + unit : unit;
    const bool i8 = a.act == MOE_DTYPE_INT8;
    uint32_t w = 0;
    for (int j = 0; j < 8; ++j) {
        const int k = kt * kTileK + w4_k(a.group, kq, d, j);
        uint32_t c = 0;  // padded rows have scale 0, padded k meet x = 0
        if (row_ok && k < a.K) {
            const uint8_t b = src[row * (a.K / 2) + k / 2];
            c = k & 1 ? b >> 4 : b & 15u;
        }
        // 16-bit x: element pairs (2i, 2i + 1) in nibbles i and i + 4; int8:
        // elements 0..3 in the low nibbles of the bytes, 4..7 in the high ones
        const int nib = i8 ? (j & 3) * 2 + (j >> 2) : (j >> 1) + 4 * (j & 1);
        w |= (i8 ? c ^ 8u : c) << (4 * nib);
    }
    dst[o] = w;
}

// One thread per (tile, group, row).
__global__ __launch_bounds__(256) void pack_scales_kernel(const float *__restrict__ scale,
                                                          const uint8_t *__restrict__ zero, float *__restrict__ dst,
                                                          uint8_t *__restrict__ dst_zero, LinearW4Args a, int64_t n) {
    const int64_t o = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (o >= n) return;
    const int gpt = kTileK / a.group;
    const int r = static_cast<int>(o & 15), g = static_cast<int>((o >> 4) % gpt);
    const int64_t tile = (o >> 4) / gpt;
    const int kt = static_cast<int>(tile % a.k_tiles), nt = static_cast<int>(tile / a.k_tiles);
    const int half = a.N / 2;
    const int unit = a.gated ? nt * 8 + r / 2 : nt * 16 + r;
    const int64_t row = a.gated && (r & 1) ? half + unit : unit;
    const int gk = kt * gpt + g, groups = a.K / a.group;
    const bool ok = unit < (a.gated ? half : a.N) && gk < groups;
    dst[o] = ok ? scale[row * groups + gk] : 0.0f;
    if (dst_zero) dst_zero[o] = ok ? zero[row * groups + gk] : 8;
}

// ------------------------------------------------------------------ product
// X: 0 bf16, 1 fp16, 2 int8. G: group. Z: zero points given. MT: 16-token
// tiles per workgroup.
constexpr int kWaves = 8;

template <int X>
struct Acc { typedef v4f type; };
template <>
struct Acc<2> { typedef v4i type; };

__device__ __forceinline__ v4i load16(const void *p) { return *static_cast<const v4i *>(p); }

template <int X, int G, bool Z, int MT>
__global__ __launch_bounds__(kWaves *kWave) void linear_w4_kernel(LinearW4Args a) {
    typedef typename Acc<X>::type acc_t;
    constexpr int kGroups = kTileK / G;
    constexpr bool kSums = X == 0 || (X == 2 && Z);  // sums of x are needed
    constexpr int kElem = X == 2 ? 1 : 2;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int col = lane & 15, kq = lane >> 4;
    const int nt = blockIdx.x;
    const int t0 = blockIdx.y * 16 * MT;
    const uint8_t *codes = a.codes + static_cast<size_t>(nt) * a.k_tiles * 1024 + lane * 16;
    const float *scale = a.scale + static_cast<size_t>(nt) * a.k_tiles * kGroups * 16 + kq * 4;
    const uint8_t *zero = Z ? a.zero + static_cast<size_t>(nt) * a.k_tiles * kGroups * 16 : nullptr;
    const uint8_t *x = static_cast<const uint8_t *>(a.x);

    v4f total[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) total[m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

    for (int kt = wave; kt < a.k_tiles; kt += kWaves) {
        const v4i cw = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(codes + static_cast<size_t>(kt) * 1024));
        // x fragments: word d of the codes meets 8 elements
        v4i xr[MT][X == 2 ? 2 : 4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int t = t0 + m * 16 + col;
            const uint8_t *xp = x + (static_cast<size_t>(t) * a.K + static_cast<size_t>(kt) * kTileK) * kElem;
#pragma unroll
            for (int i = 0; i < (X == 2 ? 2 : 4); ++i) {
                v4i v = {0, 0, 0, 0};
                if (X == 2 && G == 32) {  // words 2i and 2i + 1, 8 bytes each
                    const int k0 = w4_k(G, kq, 2 * i, 0), k1 = w4_k(G, kq, 2 * i + 1, 0);
                    if (t < a.T && kt * kTileK + k0 < a.K) {
                        const int2 b = *reinterpret_cast<const int2 *>(xp + k0);
                        v.x = b.x;
                        v.y = b.y;
                    }
                    if (t < a.T && kt * kTileK + k1 < a.K) {
                        const int2 b = *reinterpret_cast<const int2 *>(xp + k1);
                        v.z = b.x;
                        v.w = b.y;
                    }
                } else {
                    const int k0 = w4_k(G, kq, X == 2 ? 2 * i : i, 0);
                    if (t < a.T && kt * kTileK + k0 < a.K) v = load16(xp + k0 * kElem);
                }
                xr[m][i] = v;
            }
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
            const size_t go = (static_cast<size_t>(kt) * kGroups + g) * 16;
            const v4f sc = *reinterpret_cast<const v4f *>(scale + go);
            v4f zf = {8.0f, 8.0f, 8.0f, 8.0f};
            v4i zi = {0, 0, 0, 0};
            v2h zh = {static_cast<_Float16>(1032.0f), static_cast<_Float16>(1032.0f)};
            if (Z && X == 1) {
                const _Float16 h = static_cast<_Float16>(1024.0f + static_cast<float>(zero[go + col]));
                zh = v2h{h, h};
            } else if (Z) {
                const uint32_t zw = *reinterpret_cast<const uint32_t *>(zero + go + kq * 4);
                zf = v4f{static_cast<float>(zw & 255u), static_cast<float>((zw >> 8) & 255u),
                         static_cast<float>((zw >> 16) & 255u), static_cast<float>(zw >> 24)};
                zi = v4i{static_cast<int>(zw & 255u) * 16 - 128, static_cast<int>((zw >> 8) & 255u) * 16 - 128,
                         static_cast<int>((zw >> 16) & 255u) * 16 - 128, static_cast<int>(zw >> 24) * 16 - 128};
            }
            acc_t acc[MT], sx[MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                acc[m] = acc_t{0, 0, 0, 0};
                sx[m] = acc_t{0, 0, 0, 0};
            }
            constexpr int kWords = G / 32;  // code words of the group
            if constexpr (X != 2) {
#pragma unroll
                for (int i = 0; i < kWords; ++i) {
                    const int d = g * kWords + i;
                    const uint32_t w = static_cast<uint32_t>(cw[d]);
                    constexpr uint32_t kBase = X == 1 ? 0x64006400u : 0x43004300u;
                    v4i av;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        uint32_t u = ((w >> (4 * e)) & 0x000F000Fu) | kBase;
                        if (X == 1) u = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, u) - zh);
                        av[e] = static_cast<int>(u);
                    }
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        if constexpr (X == 1) {
                            acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_f16(
                                __builtin_bit_cast(v8h, av), __builtin_bit_cast(v8h, xr[m][d]), acc[m], 0, 0, 0);
                        } else {
                            const v4i ones = {0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80};
                            acc[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(v8bf, av), __builtin_bit_cast(v8bf, xr[m][d]), acc[m], 0, 0, 0);
                            sx[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                __builtin_bit_cast(v8bf, ones), __builtin_bit_cast(v8bf, xr[m][d]), sx[m], 0, 0, 0);
                        }
                    }
                }
            } else if constexpr (G == 32) {
                const uint32_t w = static_cast<uint32_t>(cw[g]);
                const long av = static_cast<long>((static_cast<uint64_t>(w & 0xF0F0F0F0u) << 32) |
                                                  ((w << 4) & 0xF0F0F0F0u));
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const v4i xv = xr[m][g / 2];
                    const long b = static_cast<long>(
                        (static_cast<uint64_t>(static_cast<uint32_t>(g & 1 ? xv.w : xv.y)) << 32) |
                        static_cast<uint32_t>(g & 1 ? xv.z : xv.x));
                    acc[m] = __builtin_amdgcn_mfma_i32_16x16x32_i8(av, b, acc[m], 0, 0, 0);
                    if (Z) sx[m] = __builtin_amdgcn_mfma_i32_16x16x32_i8(0x0101010101010101L, b, sx[m], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int i = 0; i < G / 64; ++i) {
                    const int u = g * (G / 64) + i;
                    const uint32_t w0 = static_cast<uint32_t>(cw[2 * u]), w1 = static_cast<uint32_t>(cw[2 * u + 1]);
                    const v4i av = {static_cast<int>((w0 << 4) & 0xF0F0F0F0u), static_cast<int>(w0 & 0xF0F0F0F0u),
                                    static_cast<int>((w1 << 4) & 0xF0F0F0F0u), static_cast<int>(w1 & 0xF0F0F0F0u)};
                    const v4i ones = {0x01010101, 0x01010101, 0x01010101, 0x01010101};
#pragma unroll
                    for (int m = 0; m < MT; ++m) {
                        acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, xr[m][u], acc[m], 0, 0, 0);
                        if (Z) sx[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(ones, xr[m][u], sx[m], 0, 0, 0);
                    }
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float v;
                    if constexpr (X == 2) v = static_cast<float>(Z ? acc[m][i] - zi[i] * sx[m][0] : acc[m][i]);
                    else if constexpr (X == 0) v = __builtin_fmaf(-(128.0f + zf[i]), sx[m][0], acc[m][i]);
                    else v = acc[m][i];
                    total[m][i] = __builtin_fmaf(v, sc[i], total[m][i]);
                }
            }
        }
    }
    (void)kSums;

    __shared__ v4f red[kWaves][MT][kWave];
#pragma unroll
    for (int m = 0; m < MT; ++m) red[wave][m][lane] = total[m];
    __syncthreads();
    for (int m = wave; m < MT; m += kWaves) {  // uniform per wave
        v4f o = red[0][m][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) o += red[w][m][lane];
        const int t = t0 + m * 16 + col;
        if (t >= a.T) continue;
        if (X == 2) {
            const float xs = a.x_scale[t] * 0.0625f;  // the codes were 16 * (c - 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = o[i] * xs;
        }
        uint16_t *out = static_cast<uint16_t *>(a.out);
        auto put = [&](int n, int width, float v) {
            if (n >= width) return;
            uint16_t b;
            if (X == 1) b = __builtin_bit_cast(uint16_t, static_cast<_Float16>(v));
            else b = f32_to_bf16(v);
            out[static_cast<size_t>(t) * width + n] = b;
        };
        if (a.gated) {
            const int half = a.N / 2;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int n = nt * 8 + kq * 2 + i;
                float g = o[2 * i], u = o[2 * i + 1];
                if (a.bias && n < half) {
                    g += a.bias[n];
                    u += a.bias[half + n];
                }
                put(n, half, swiglu_y(g, u));
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = nt * 16 + kq * 4 + i;
                put(n, a.N, a.bias && n < a.N ? o[i] + a.bias[n] : o[i]);
            }
        }
    }
}

template <int X, int G, bool Z>
hipError_t launch_tokens(const LinearW4Args &a, hipStream_t s) {
    const dim3 blk(kWaves * kWave);
    auto grid = [&](int mt) { return dim3(a.n_tiles, (a.T + 16 * mt - 1) / (16 * mt)); };
    if (a.T <= 16) hipLaunchKernelGGL((linear_w4_kernel<X, G, Z, 1>), grid(1), blk, 0, s, a);
    else if (a.T <= 32) hipLaunchKernelGGL((linear_w4_kernel<X, G, Z, 2>), grid(2), blk, 0, s, a);
    else hipLaunchKernelGGL((linear_w4_kernel<X, G, Z, 4>), grid(4), blk, 0, s, a);
    return hipGetLastError();
}

template <int X>
hipError_t launch_act(const LinearW4Args &a, hipStream_t s) {
    if (a.group == 32) return a.zero ? launch_tokens<X, 32, true>(a, s) : launch_tokens<X, 32, false>(a, s);
    if (a.group == 64) return a.zero ? launch_tokens<X, 64, true>(a, s) : launch_tokens<X, 64, false>(a, s);
    return a.zero ? launch_tokens<X, 128, true>(a, s) : launch_tokens<X, 128, false>(a, s);
}

}  // namespace

hipError_t launch_pack_w4(const uint8_t *codes, const float *scale, const uint8_t *zero, uint8_t *dst_codes,
                          float *dst_scale, uint8_t *dst_zero, const LinearW4Args &a, hipStream_t s) {
    const int64_t tiles = static_cast<int64_t>(a.n_tiles) * a.k_tiles;  // <= 2^26: the grid below fits
    const int64_t n = tiles * (kTileK / a.group) * 16;
    hipLaunchKernelGGL(pack_codes_kernel, dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s, codes,
                       reinterpret_cast<uint32_t *>(dst_codes), a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(pack_scales_kernel, dim3(static_cast<unsigned>((n + 255) / 256)), dim3(256), 0, s, scale, zero,
                       dst_scale, dst_zero, a, n);
    return hipGetLastError();
}

hipError_t launch_linear_w4(const LinearW4Args &a, hipStream_t s) {
    if (a.act == MOE_DTYPE_BF16) return launch_act<0>(a, s);
    if (a.act == MOE_DTYPE_FP16) return launch_act<1>(a, s);
    return launch_act<2>(a, s);
}

}  // namespace moe
