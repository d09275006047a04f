// Dense product with 4-bit weights on MFMA:
//
//   o[t,n] = xs[t] * sum_g s[n,g] * (sum_{k in g} (c[n,k] - z[n,g]) * x[t,k]) + bias[n]
//
// Weight rows are the MFMA's A rows, tokens its B columns: one 16 x 16 tile of
// D covers 16 output rows and 16 tokens, lane l holding rows 4 * (l / 16) ..+3
// of token l % 16. The 4-bit codes go to the matrix operand in few operations
// per eight of them:
//   fp16:  0x5800 | c << 3 is 128 + c; minus (128 + z), exact
//   bf16:  0x4180 | c << 3 is 16 + c, exact; the group's sum then carries
//          (16 + z) * sum(x), which is subtracted with the sum of x that one
//          more MFMA with a matrix of ones makes (per token tile, shared by
//          the weight tiles). bf16 has no packed subtraction here. 16 is the
//          smallest base with all codes in one binade: products of up to 31 x
//          stand for up to 15 x, one bit of fp32. (128 + c, three more: T 512,
//          N 8192, K 4096, outputs that are not the rounded 64-bit value:
//          0.12 %, with 16 + c 0.016 %, an fp32 product of whole rows 0.072 %.)
//   For both, codes are packed rotated by 3, so that c << 3 costs no shift.
//   int8:  codes are packed as the nibble of c - 8; kept in a byte's high half
//          it is 16 * (c - 8) as int8. Zero points other than 8 are subtracted
//          with the int32 sum of x, as for bf16; the 16 divides out at the end,
//          exactly.
// A group's products are summed in the MFMA's fp32 (int8: exactly, in int32),
// scaled, and the groups are added in fp32.
//
// Two kernels: few tokens, whose time is the weight stream, and many, whose
// time is the matrix products (below). Sums over K are split over waves and
// joined in LDS in a fixed order: no workspace, no atomics, and results do not
// depend on timing.
#include "ops.h"

#include <type_traits>

#include "../../include/moe_w8a8.h"

namespace moe {
namespace {

typedef int v2i __attribute__((ext_vector_type(2)));
typedef int v4i __attribute__((ext_vector_type(4)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

constexpr int kTileK = 128;

__device__ __forceinline__ v4i load16(const void *p) { return *static_cast<const v4i *>(p); }

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
    // the word's eight elements are consecutive: four bytes of the row
    const int k0 = kt * kTileK + w4_k(a.group, kq, d, 0);
    uint32_t raw = 0;  // padded rows have scale 0, padded k too
    if (row_ok && k0 < a.K) __builtin_memcpy(&raw, src + row * (a.K / 2) + k0 / 2, 4);
    uint32_t w = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t c = (raw >> (4 * j)) & 15u;
        // 16-bit x: element pairs (2i, 2i + 1) in nibbles i and i + 4; int8:
        // elements 0..3 in the low nibbles of the bytes, 4..7 in the high ones
        const int nib = i8 ? (j & 3) * 2 + (j >> 2) : (j >> 1) + 4 * (j & 1);
        w |= (i8 ? c ^ 8u : c) << (4 * nib);
    }
    dst[o] = i8 ? w : w << 3 | w >> 29;
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
// X: 0 bf16, 1 fp16, 2 int8. G: group. Z: zero points given.

template <int X>
struct Acc { typedef v4f type; };
template <>
struct Acc<2> { typedef v4i type; };

// x of 16 tokens and one 128-k tile in LDS: rows of kSlots 16-byte slots, slot
// c of row r at place c ^ swizzle(r). Whole rows are written, 16 rows' slots of
// one k are read: both meet every bank equally often.
template <int X>
struct XTile {
    static constexpr int kElem = X == 2 ? 1 : 2;
    static constexpr int kSlots = kTileK * kElem / 16;
    static constexpr int kBytes = 16 * kSlots * 16;
    static __device__ __forceinline__ int at(int row, int slot) {
        const int sw = kSlots == 16 ? row & 15 : (row >> 1) & 7;
        return (row * kSlots + (slot ^ sw)) * 16;
    }
};

// The lane's x operands of one 16-token tile: for 16-bit x one per code word,
// for int8 one per two words.
template <int X>
constexpr int kFrags = X == 2 ? 2 : 4;

// LDS that one wave writes and reads, its lanes what others wrote, without a
// barrier: the LDS unit takes a wave's accesses in order, and volatile keeps
// the compiler from changing it (to its alias analysis a lane is a thread of
// its own). Fences at wave scope do so too, but hold back the loads of the
// next tiles: T 2, N 28672, K 8192 29.0 us instead of 27.2.
template <typename V>
using OwnLds = __attribute__((address_space(3))) volatile V;
template <bool OWN, typename V>
__device__ __forceinline__ V read_lds(const char *p) {
    if constexpr (OWN) return *(const OwnLds<V> *)p;
    else return *reinterpret_cast<const V *>(p);
}

template <int X, int G, bool OWN>
__device__ __forceinline__ void read_frags(const char *lds, int r, int kq, v4i (&f)[kFrags<X>]) {
#pragma unroll
    for (int i = 0; i < kFrags<X>; ++i) {
        if constexpr (X == 2 && G == 32) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = w4_k(G, kq, 2 * i + h, 0);
                const v2i b = read_lds<OWN, v2i>(lds + XTile<X>::at(r, k / 16) + k % 16);
                f[i][2 * h] = b.x;
                f[i][2 * h + 1] = b.y;
            }
        } else {
            const int k = w4_k(G, kq, X == 2 ? 2 * i : i, 0);
            f[i] = read_lds<OWN, v4i>(lds + XTile<X>::at(r, k * XTile<X>::kElem / 16));
        }
    }
}

// One group's scales and zero points for the lane: its four D rows, and (fp16,
// whose codes are made exact before the product) its A row.
template <int X, bool Z>
struct GroupScale {
    v4f sc;
    uint32_t z;
    __device__ __forceinline__ void load(const float *scale, const uint8_t *zero, size_t o, int r, int kq) {
        sc = *reinterpret_cast<const v4f *>(scale + o + kq * 4);
        if (Z) z = X == 1 ? zero[o + r] : *reinterpret_cast<const uint32_t *>(zero + o + kq * 4);
    }
    __device__ __forceinline__ v2h half_zero() const {
        const _Float16 h = static_cast<_Float16>(Z ? 128.0f + static_cast<float>(z) : 136.0f);
        return v2h{h, h};
    }
    // what one unit of the sum of x takes off the group's product of row i
    __device__ __forceinline__ float offset(int i) const {
        return Z ? 16.0f + static_cast<float>((z >> (8 * i)) & 255u) : 24.0f;
    }
    __device__ __forceinline__ int offset8(int i) const {
        return Z ? static_cast<int>((z >> (8 * i)) & 255u) * 16 - 128 : 0;
    }
};

// The mask and base of expand16 in registers: as literals they would take an
// instruction each, in registers one v_and_or_b32 takes both.
template <int X>
struct ExpandConst {
    uint32_t mask, base;
    __device__ __forceinline__ ExpandConst() {
        asm("s_mov_b32 %0, 0x00780078" : "=s"(mask));
        if (X == 1) asm("v_mov_b32 %0, 0x58005800" : "=v"(base));
        else asm("v_mov_b32 %0, 0x41804180" : "=v"(base));
    }
};

// Eight codes to an A operand of 16-bit elements.
template <int X>
__device__ __forceinline__ v4i expand16(const ExpandConst<X> &c, uint32_t w, v2h zh) {
    v4i a;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        // the last pair's upper code reaches around the word's end
        uint32_t u = ((e < 3 ? w >> (4 * e) : __builtin_rotateright32(w, 12)) & c.mask) | c.base;
        if (X == 1) u = __builtin_bit_cast(uint32_t, __builtin_bit_cast(v2h, u) - zh);
        a[e] = static_cast<int>(u);
    }
    return a;
}
// Sixteen codes to an A operand of int8: 16 * (c - 8).
__device__ __forceinline__ v4i expand8(uint32_t w0, uint32_t w1) {
    return v4i{static_cast<int>((w0 << 4) & 0xF0F0F0F0u), static_cast<int>(w0 & 0xF0F0F0F0u),
               static_cast<int>((w1 << 4) & 0xF0F0F0F0u), static_cast<int>(w1 & 0xF0F0F0F0u)};
}
__device__ __forceinline__ long low8(v4i v) {
    return static_cast<long>((static_cast<uint64_t>(static_cast<uint32_t>(v.y)) << 32) | static_cast<uint32_t>(v.x));
}
__device__ __forceinline__ long high8(v4i v) {
    return static_cast<long>((static_cast<uint64_t>(static_cast<uint32_t>(v.w)) << 32) | static_cast<uint32_t>(v.z));
}

// acc += (codes of group g, expanded) x (x fragments); `ones` instead of codes
// gives the sums of x.
template <int X, int G>
__device__ __forceinline__ void group_mfma(typename Acc<X>::type &acc, const v4i (&a)[4], const v4i (&x)[kFrags<X>], int g) {
    if constexpr (X == 2 && G == 32) {
        const v4i av = a[g / 2], xv = x[g / 2];
        acc = __builtin_amdgcn_mfma_i32_16x16x32_i8(g & 1 ? high8(av) : low8(av), g & 1 ? high8(xv) : low8(xv), acc, 0, 0, 0);
    } else if constexpr (X == 2) {
#pragma unroll
        for (int i = 0; i < G / 64; ++i)
            acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[g * (G / 64) + i], x[g * (G / 64) + i], acc, 0, 0, 0);
    } else {
#pragma unroll
        for (int i = 0; i < G / 32; ++i) {
            const int d = g * (G / 32) + i;
            if constexpr (X == 1)
                acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a[d]), __builtin_bit_cast(v8h, x[d]), acc, 0, 0, 0);
            else
                acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a[d]), __builtin_bit_cast(v8bf, x[d]), acc, 0, 0, 0);
        }
    }
}

// total += scale * (acc - offset * sum of x), row by row
template <int X, bool Z>
__device__ __forceinline__ void add_group(v4f &total, typename Acc<X>::type acc, typename Acc<X>::type sx,
                                          const GroupScale<X, Z> &s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float v;
        if constexpr (X == 2) v = static_cast<float>(Z ? acc[i] - s.offset8(i) * sx[0] : acc[i]);
        else if constexpr (X == 0) v = __builtin_fmaf(-s.offset(i), sx[0], acc[i]);
        else v = acc[i];
        total[i] = __builtin_fmaf(v, s.sc[i], total[i]);
    }
}

// The finished sums of rows 4 * kq ..+3 of tile nt for token t.
template <int X>
__device__ __forceinline__ void finish(const LinearW4Args &a, int nt, int kq, int t, v4f o) {
    if (X == 2) {
        const float xs = a.x_scale[t] * 0.0625f;  // the codes were 16 * (c - 8)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = o[i] * xs;
    }
    auto bits = [](float v) -> uint16_t {
        return X == 1 ? __builtin_bit_cast(uint16_t, static_cast<_Float16>(v)) : f32_to_bf16(v);
    };
    uint16_t *out = static_cast<uint16_t *>(a.out);
    if (a.gated) {
        const int half = a.N / 2, n = nt * 8 + kq * 2;
        uint16_t *p = out + static_cast<size_t>(t) * half + n;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            if (n + i >= half) break;
            float g = o[2 * i], u = o[2 * i + 1];
            if (a.bias) {
                g += a.bias[n + i];
                u += a.bias[half + n + i];
            }
            p[i] = bits(swiglu_y(g, u));
        }
    } else {
        const int n = nt * 16 + kq * 4;
        uint16_t *p = out + static_cast<size_t>(t) * a.N + n;
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N) o[i] += a.bias[n + i];
        }
        if (a.N % 4 == 0) {  // then whole quadruples, 8-byte aligned
            if (n < a.N) {
                const uint64_t v = bits(o[0]) | static_cast<uint64_t>(bits(o[1])) << 16 |
                                   static_cast<uint64_t>(bits(o[2])) << 32 | static_cast<uint64_t>(bits(o[3])) << 48;
                *reinterpret_cast<uint64_t *>(p) = v;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (n + i < a.N) p[i] = bits(o[i]);
        }
    }
}

// Few tokens (MT tiles of 16): the weight stream is what counts. A workgroup
// takes 16 weight rows, its WAVES waves every WAVES-th tile of 128 k, whose
// codes and scales are loaded DEPTH tiles ahead; the waves' sums meet in LDS.
//
// MFMA operands are one row per lane, so loading x straight into them is 64
// requests of 16 bytes per instruction, and four instructions per tile kept
// the load units busier than the weights did (T 2, N 28672, K 8192: 41 us).
// Whole rows of the ROWS tokens there may be are loaded instead, and turned in
// LDS, in a place of the wave's own (no barrier).
//
// Nothing is masked: loads of tokens past the end read the last token's x, and
// columns of rows that were never loaded work on whatever LDS holds: a column
// is one token's, and these are not stored. Lanes of k past the end read the
// row's last k, which meets scales that the packing set to zero.
template <int X, int G, bool Z, int ROWS, int R, int WAVES>
__global__ __launch_bounds__(WAVES *kWave) void linear_w4_few_kernel(LinearW4Args a) {
    typedef typename Acc<X>::type acc_t;
    typedef XTile<X> XT;
    constexpr int kGroups = kTileK / G, kF = kFrags<X>;
    constexpr int DEPTH = 2;                         // tiles in flight; 3 and 4 lose more to registers than they hide
    constexpr bool kSums = X == 0 || (X == 2 && Z);  // the sums of x are needed
    constexpr int MT = (ROWS + 15) / 16;             // tiles of 16 tokens
    static_assert(MT * R <= WAVES, "one wave per tile finishes");
    constexpr int kRowsPerLoad = kWave / XT::kSlots;
    constexpr int kL = ROWS >= 16 ? kF : (ROWS + kRowsPerLoad - 1) / kRowsPerLoad;  // loads of x per tile
    constexpr int kBufs = MT > 1 ? 2 : 1;            // places per wave
    constexpr int kPer16 = 16 / XT::kElem;           // elements per 16 bytes
    constexpr int kStageBytes = WAVES * kBufs * XT::kBytes, kRedBytes = WAVES * MT * R * kWave * 16;
    __shared__ __attribute__((aligned(16))) char lds[kStageBytes > kRedBytes ? kStageBytes : kRedBytes];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, kq = lane >> 4;
    const int nt0 = blockIdx.x * R, t0 = blockIdx.y * ROWS;
    char *place = lds + wave * kBufs * XT::kBytes;
    const uint8_t *x = static_cast<const uint8_t *>(a.x) + static_cast<size_t>(t0) * a.K * XT::kElem;

    uint32_t xrow[MT][kL];  // where the lane's loads of a tile begin: at most 64 rows of 2^18 bytes
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int i = 0; i < kL; ++i) {
            const int t = m * 16 + (i * kWave + lane) / XT::kSlots;
            xrow[m][i] = static_cast<uint32_t>(min(t, a.T - 1 - t0)) * static_cast<uint32_t>(a.K * XT::kElem);
        }
    const ExpandConst<X> konst;
    struct Tile {
        v4i codes[R];
        GroupScale<X, Z> s[R][kGroups];
        v4i x[MT][kL];
    };
    const int count = (a.k_tiles - wave + WAVES - 1) / WAVES;  // the wave's tiles; <= 0: none
    auto fetch = [&](int i, Tile &f) {
        const int kt = wave + min(i, count - 1) * WAVES;  // past the end: the last one again
#pragma unroll
        for (int j = 0; j < R; ++j) {  // rows past the end: the last ones, not stored
            const size_t tile = static_cast<size_t>(min(nt0 + j, a.n_tiles - 1)) * a.k_tiles + kt;
            f.codes[j] = __builtin_nontemporal_load(reinterpret_cast<const v4i *>(a.codes + tile * 1024 + lane * 16));
#pragma unroll
            for (int g = 0; g < kGroups; ++g) f.s[j][g].load(a.scale, a.zero, (tile * kGroups + g) * 16, r, kq);
        }
        const int k = min(kt * kTileK + lane % XT::kSlots * kPer16, a.K - kPer16);
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int j = 0; j < kL; ++j) f.x[m][j] = load16(x + (xrow[m][j] + static_cast<uint32_t>(k * XT::kElem)));
    };
    v4f total[R][MT];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) total[j][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    auto multiply = [&](const Tile &f) {
        v4i av[R][4], ones[4];
#pragma unroll
        for (int j = 0; j < R; ++j) {
            if constexpr (X == 2) {
                av[j][0] = expand8(f.codes[j].x, f.codes[j].y);
                av[j][1] = expand8(f.codes[j].z, f.codes[j].w);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d)
                    av[j][d] = expand16<X>(konst, f.codes[j][d], f.s[j][d * 32 / G].half_zero());
            }
        }
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int one = X == 2 ? 0x01010101 : 0x3F803F80;
            ones[d] = v4i{one, one, one, one};
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            v4i xf[kF];
            char *buf = place + (m % kBufs) * XT::kBytes;
#pragma unroll
            for (int j = 0; j < kL; ++j) {
                const int slot = j * kWave + lane;
                *(OwnLds<v4i> *)(buf + XT::at(slot / XT::kSlots, slot % XT::kSlots)) = f.x[m][j];
            }
            read_frags<X, G, true>(buf, r, kq, xf);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                acc_t sx = {0, 0, 0, 0};
                if constexpr (kSums) group_mfma<X, G>(sx, ones, xf, g);
#pragma unroll
                for (int j = 0; j < R; ++j) {
                    acc_t acc = {0, 0, 0, 0};
                    group_mfma<X, G>(acc, av[j], xf, g);
                    add_group<X, Z>(total[j][m], acc, sx, f.s[j][g]);
                }
            }
        }
    };
    // Loads complete in the order of their issue, and the compiler counts them
    // exactly only where none is conditional: the loop refills all DEPTH tiles,
    // and the last round, which refills none, stands behind it.
    if (count > 0) {
        Tile ring[DEPTH];
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) fetch(d, ring[d]);
        int i = 0;
        for (; i + DEPTH < count; i += DEPTH) {
#pragma unroll
            for (int d = 0; d < DEPTH; ++d) {
                multiply(ring[d]);
                fetch(i + DEPTH + d, ring[d]);
            }
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (i + d < count) multiply(ring[d]);
    }
    v4f(*red)[R * MT][kWave] = reinterpret_cast<v4f(*)[R * MT][kWave]>(lds);
    __syncthreads();  // the places are read until here
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) red[wave][j * MT + m][lane] = total[j][m];
    __syncthreads();
    if (wave >= R * MT) return;
    v4f o = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) o += red[w][wave][lane];
    const int nt = nt0 + wave / MT, t = t0 + wave % MT * 16 + r;
    if (nt < a.n_tiles && t < a.T) finish<X>(a, nt, kq, t, o);
}

// Many tokens: the matrix rate is what counts. A workgroup takes 128 weight
// rows (each of its four waves two tiles; half of that with groups of 32) and
// 64 tokens; x of one 128-k
// tile lies in LDS for all of them, the next two tiles' on their way in registers;
// codes go from memory straight to the wave that expands them. The sums of x
// that bf16 codes and zero points need are made once, by the threads that
// bring x in, not by every wave.
//
// Workgroups of the same rows get numbers that are equal modulo 8: their
// codes come from one XCD's L2.
constexpr int kManyWaves = 4, kManyTokens = 64;
// Row tiles per wave. Four groups' scales and zero points of two row tiles do
// not fit the registers.
template <int G>
constexpr int kManyRows = G == 32 ? 1 : 2;

// Sum over aligned runs of N lanes, in all of them: DPP swaps of neighbours
// and of pairs, then the mirrors of half rows and rows.
template <int N, typename V>
__device__ __forceinline__ V run_sum(V v) {
    auto step = [&](auto ctrl) {
        const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(ctrl)::value, 0xF, 0xF, true);
        v += __builtin_bit_cast(V, o);
    };
    if constexpr (N >= 2) step(std::integral_constant<int, 0xB1>{});
    if constexpr (N >= 4) step(std::integral_constant<int, 0x4E>{});
    if constexpr (N >= 8) step(std::integral_constant<int, 0x141>{});
    if constexpr (N >= 16) step(std::integral_constant<int, 0x140>{});
    return v;
}

template <int X, int G, bool Z>
__global__ __launch_bounds__(kManyWaves *kWave, 2) void linear_w4_many_kernel(LinearW4Args a, int token_blocks,
                                                                          int row_blocks) {
    typedef typename Acc<X>::type acc_t;
    typedef XTile<X> XT;
    typedef decltype(acc_t{}[0] + acc_t{}[0]) sum_t;
    constexpr int MT = kManyTokens / 16, kRowTiles = kManyRows<G>;
    constexpr int kGroups = kTileK / G, kF = kFrags<X>, kThreads = kManyWaves * kWave;
    constexpr bool kSums = X == 0 || (X == 2 && Z);
    constexpr int kPer16 = 16 / XT::kElem;
    constexpr int kLoads = MT * 16 * XT::kSlots / kThreads;  // 16-byte loads of x per thread and tile
    constexpr int kRun = G / kPer16;                         // neighbouring slots of one group
    __shared__ __attribute__((aligned(16))) char s_x[2][MT * XT::kBytes];
    __shared__ sum_t s_sum[2][kSums ? MT : 1][kGroups][16];
    const int rb = static_cast<int>(blockIdx.x >> 3) / token_blocks * 8 + static_cast<int>(blockIdx.x & 7);
    if (rb >= row_blocks) return;
    const int t0 = static_cast<int>(blockIdx.x >> 3) % token_blocks * 16 * MT;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int r = lane & 15, kq = lane >> 4;

    // rows past the end: the last tile's weights, not stored
    int nt[kRowTiles];
    const uint8_t *codes[kRowTiles];
    size_t so[kRowTiles];
#pragma unroll
    for (int j = 0; j < kRowTiles; ++j) {
        nt[j] = (rb * kManyWaves + wave) * kRowTiles + j;
        const size_t tile = static_cast<size_t>(min(nt[j], a.n_tiles - 1)) * a.k_tiles;
        codes[j] = a.codes + tile * 1024 + lane * 16;
        so[j] = tile * kGroups * 16;
    }
    const uint8_t *x = static_cast<const uint8_t *>(a.x) + static_cast<size_t>(t0) * a.K * XT::kElem;
    static_assert(kThreads % XT::kSlots == 0, "a thread's slots are one column");
    const int xk = static_cast<int>(threadIdx.x) % XT::kSlots * kPer16;
    uint32_t xrow[kLoads];  // 64 rows of at most 2^18 bytes
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
        const int t = (static_cast<int>(threadIdx.x) + i * kThreads) / XT::kSlots;
        xrow[i] = static_cast<uint32_t>(min(t, a.T - 1 - t0)) * static_cast<uint32_t>(a.K * XT::kElem);
    }
    auto fetch_x = [&](int kt, v4i (&xr)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i)
            xr[i] = load16(x + (xrow[i] + static_cast<uint32_t>(min(kt * kTileK + xk, a.K - kPer16) * XT::kElem)));
    };
    auto put_x = [&](int buf, const v4i (&xr)[kLoads]) {
#pragma unroll
        for (int i = 0; i < kLoads; ++i) {
            const int slot = static_cast<int>(threadIdx.x) + i * kThreads;
            const int row = slot / XT::kSlots, c = slot % XT::kSlots;
            *reinterpret_cast<v4i *>(s_x[buf] + row / 16 * XT::kBytes + XT::at(row % 16, c)) = xr[i];
            if constexpr (kSums) {
                sum_t v = 0;
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int e = xr[i][q];  // a vector's element has no address to cast from
                    if constexpr (X == 2) {
                        v = __builtin_amdgcn_sdot4(e, 0x01010101, v, false);
                    } else {
                        typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
                        v = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(v2bf, e),
                                                            __builtin_bit_cast(v2bf, 0x3F803F80), v, false);
                    }
                }
                v = run_sum<kRun>(v);
                s_sum[buf][row / 16][c / kRun][row % 16] = v;  // the same from every lane of the run: no branch
            }
        }
    };
    struct Weights {
        v4i codes[kRowTiles];
        GroupScale<X, Z> s[kRowTiles][kGroups];
    };
    auto fetch_w = [&](int kt, Weights &f) {
#pragma unroll
        for (int j = 0; j < kRowTiles; ++j) {
            f.codes[j] = load16(codes[j] + static_cast<size_t>(kt) * 1024);
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
                f.s[j][g].load(a.scale, a.zero, so[j] + (static_cast<size_t>(kt) * kGroups + g) * 16, r, kq);
        }
    };
    v4f total[kRowTiles][MT];
#pragma unroll
    for (int j = 0; j < kRowTiles; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) total[j][m] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    const ExpandConst<X> konst;
    auto multiply = [&](int buf, const Weights &f) {
        v4i av[kRowTiles][4];
#pragma unroll
        for (int j = 0; j < kRowTiles; ++j) {
            if constexpr (X == 2) {
                av[j][0] = expand8(f.codes[j].x, f.codes[j].y);
                av[j][1] = expand8(f.codes[j].z, f.codes[j].w);
            } else {
#pragma unroll
                for (int d = 0; d < 4; ++d) av[j][d] = expand16<X>(konst, f.codes[j][d], f.s[j][d * 32 / G].half_zero());
            }
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            v4i xf[kF];
            read_frags<X, G, false>(s_x[buf] + m * XT::kBytes, r, kq, xf);
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                acc_t sx = {0, 0, 0, 0};
                if constexpr (kSums) sx[0] = s_sum[buf][m][g][r];
#pragma unroll
                for (int j = 0; j < kRowTiles; ++j) {
                    acc_t acc = {0, 0, 0, 0};
                    group_mfma<X, G>(acc, av[j], xf, g);
                    add_group<X, Z>(total[j][m], acc, sx, f.s[j][g]);
                }
            }
            // several groups: token tile by token tile, else the scheduler
            // draws all of them together and spills
            if constexpr (kGroups > 1) __builtin_amdgcn_sched_barrier(0);
        }
    };
    // Everything is loaded two tiles ahead, and past the end the last tile
    // again: no load is conditional, so the compiler's wait counts are exact.
    const int last = a.k_tiles - 1;
    Weights w0, w1;
    v4i x0[kLoads], x1[kLoads];
    fetch_x(0, x0);
    fetch_w(0, w0);
    fetch_x(min(1, last), x1);
    fetch_w(min(1, last), w1);
    put_x(0, x0);
    __syncthreads();
    auto step = [&](int kt, Weights &w, v4i (&x_later)[kLoads], const v4i (&x_next)[kLoads]) {
        fetch_x(min(kt + 2, last), x_later);
        multiply(kt & 1, w);
        fetch_w(min(kt + 2, last), w);
        put_x((kt + 1) & 1, x_next);  // that place was read in the step before, which every wave has left
        __syncthreads();
    };
    int kt = 0;
    for (; kt + 1 < a.k_tiles; kt += 2) {
        step(kt, w0, x0, x1);
        step(kt + 1, w1, x1, x0);
    }
    if (kt < a.k_tiles) multiply(kt & 1, w0);
#pragma unroll
    for (int j = 0; j < kRowTiles; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int t = t0 + m * 16 + r;
            if (nt[j] < a.n_tiles && t < a.T) finish<X>(a, nt[j], kq, t, total[j][m]);
        }
}

template <int X, int G, bool Z>
hipError_t launch_many(const LinearW4Args &a, hipStream_t s) {
    const int token_blocks = (a.T + kManyTokens - 1) / kManyTokens, rows = kManyWaves * kManyRows<G>;
    const int row_blocks = (a.n_tiles + rows - 1) / rows;
    const dim3 grid(static_cast<unsigned>((row_blocks + 7) / 8 * 8) * token_blocks);
    hipLaunchKernelGGL((linear_w4_many_kernel<X, G, Z>), grid, dim3(kManyWaves * kWave), 0, s, a, token_blocks,
                       row_blocks);
    return hipGetLastError();
}

template <int X, int G, bool Z, int ROWS, int R, int WAVES>
hipError_t launch_few(const LinearW4Args &a, hipStream_t s) {
    const dim3 grid((a.n_tiles + R - 1) / R, (a.T + ROWS - 1) / ROWS);
    hipLaunchKernelGGL((linear_w4_few_kernel<X, G, Z, ROWS, R, WAVES>), grid, dim3(WAVES * kWave), 0, s, a);
    return hipGetLastError();
}
// Which kernel: linear_w4_many_kernel needs workgroups to fill the chip, the
// other re-reads x for every 16 rows. In microseconds (in a captured graph),
// few / many, bf16, groups of 128, K 4096:
//   T 32, N 28672: 32 / 34      T 40, N 28672: 46 / 33    T 40, N 14336: 27 / 33
//   T 64, N 4096: 12 / 33       T 64, N 14336: 33 / 33    T 128, N 4096: 18 / 33
//   T 256, N 4096: 32 / 33      T 300, N 4096: 39 / 33    T 512, N 8192: 121 / 49
// so it goes by 16-row tiles x 64-token tiles. (int8 x: 22 / 24 at T 256, 24 /
// 24 at T 300; groups of 32: 52 / 42 at T 300.)
// Two row tiles per workgroup halve what x costs, and four halve it again,
// where there are enough of them and registers hold their scales: T 16, N
// 28672, K 8192, one / two / four 43 / 37 / 33 us; T 8, N 8192, K 4096, one /
// two 6.7 / 5.9; T 64, N 8192, K 4096, int8 x, one / two 12.4 / 9.2 (bf16 19.6
// / 20.5). N 4096 would fill half the chip.
template <int X, int G, bool Z>
hipError_t launch_tokens(const LinearW4Args &a, hipStream_t s) {
    const bool wide = G != 32 && a.n_tiles >= 512;
    if (a.T > 32 && a.n_tiles * static_cast<int64_t>((a.T + 63) / 64) > 1024) return launch_many<X, G, Z>(a, s);
    constexpr int kTwo = G != 32 ? 2 : 1;
    if (a.T <= 4) return wide ? launch_few<X, G, Z, 4, kTwo, 8>(a, s) : launch_few<X, G, Z, 4, 1, 8>(a, s);
    if (a.T <= 8) return wide ? launch_few<X, G, Z, 8, kTwo, 8>(a, s) : launch_few<X, G, Z, 8, 1, 8>(a, s);
    if constexpr (G == 128 && !(X == 1 && Z)) {
        if (a.T <= 16 && a.n_tiles >= 1024) return launch_few<X, G, Z, 16, 4, 8>(a, s);
    }
    if (a.T <= 16) return wide ? launch_few<X, G, Z, 16, kTwo, 8>(a, s) : launch_few<X, G, Z, 16, 1, 8>(a, s);
    if (a.T <= 32) return wide ? launch_few<X, G, Z, 32, kTwo, 8>(a, s) : launch_few<X, G, Z, 32, 1, 8>(a, s);
    if constexpr (X == 2 && G != 32) {
        if (wide) return a.T <= 48 ? launch_few<X, G, Z, 48, 2, 8>(a, s) : launch_few<X, G, Z, 64, 2, 8>(a, s);
    }
    if (a.T <= 48) return launch_few<X, G, Z, 48, 1, 4>(a, s);
    return launch_few<X, G, Z, 64, 1, 4>(a, s);
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
    const int64_t tiles = static_cast<int64_t>(a.n_tiles) * a.k_tiles;  // <= 2^23: the grid below fits
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
