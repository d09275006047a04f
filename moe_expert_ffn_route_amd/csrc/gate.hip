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
//   - large products of x and W both bf16, or both fp16, or bf16 x and fp32 W
//     (W is split into three bf16 parts, which hold its 24 bits): MFMA with
//     fp32 sums over 64 h, which are added up in fp64. |x| |w| (2-norms),
//     which is no less than the sum of |x * w|, bounds how far such a logit is
//     off. Where the bound leaves open which of two experts comes first, the
//     choice kernel computes the logits of those experts again, in fp64.
//   - small products, other types, and softmax with a bias: fp64 MFMA
//     throughout (products are exact in it).
//
// Two launches: the logits, in up to kMaxSplit parts of H, into the
// workspace; and one wave per token, which adds the parts in order, for
// scores and choice.
#include "ops.h"

#include <type_traits>

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
constexpr int kChunk = 128;  // h per stage
constexpr int kBlock = 256;
constexpr int kMaxSplit = 8;
// An fp32 sum of n products that are themselves exact, in any order, with
// every addition off by at most one unit in the last place (an adder that
// truncates): n * 2^-23 of the sum of magnitudes, which Cauchy's inequality
// bounds by the norms.
constexpr double kUnit = 0x1p-23;
// Numbers under the smallest normal fp32 may be dropped. Products, and sums of
// them: at most 16384 of each for every plane of W. Squares: the norms' (at
// most 16384 of them) may lack their share of it, which also covers inputs
// that are dropped: 2^-126 of each is under kUnit * 2^-56.
constexpr int kMaxPlanes = 3, kMaxTerms = 16384;
constexpr double kTiny = 0x1p-109, kTinySquares = 0x1p-112;
static_assert(kTiny >= 2.0 * kMaxPlanes * kMaxTerms * 0x1p-126 && kTinySquares >= kMaxTerms * 0x1p-126,
              "what is dropped is inside the bound");

// Eight elements from h = k of a row of H. WHOLE: they are known to be there
// (no branch, so that loads can be issued in a row).
template <bool WHOLE, typename T>
__device__ __forceinline__ void load8(const T *row, int k, int H, T (&raw)[kVec]) {
    if (WHOLE || k + kVec <= H) {
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
// Planes of W that the fp32 sums may be made of, else 0.
template <typename T, typename W>
constexpr int kPlanes = kFast<T, W> ? 1 : 0;
template <>
constexpr int kPlanes<Bf16, float> = kMaxPlanes;
// Three planes pay where the fp64 MFMA is the time: bf16 x, fp32 W, E 256, H
// 4096, logits and choice together, planes / fp64: T 4096 64 / 153 us, T 1024
// 34 / 48, T 520 31 / 47; under the border they gain 10 % (T 512 30 / 33, T 400
// 29 / 32).
constexpr int64_t kPlanesFrom = int64_t(1) << 29;  // products

template <typename T>
__device__ __forceinline__ v4f mfma32(v4i a, v4i b, v4f c) {
    if constexpr (__is_same(T, Bf16))
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8bf, a), __builtin_bit_cast(v8bf, b), c, 0, 0, 0);
    else
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
}

// n += the squares of 16 bytes of elements.
template <typename T>
__device__ __forceinline__ void add_squares(v4i v, float &n) {
    if constexpr (__is_same(T, float)) {  // four elements
#pragma unroll
        for (int i = 0; i < 4; ++i) n = __builtin_fmaf(__int_as_float(v[i]), __int_as_float(v[i]), n);
    } else if constexpr (__is_same(T, Bf16)) {
        typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = v[i];  // a vector's element has no address to cast from
            const v2bf p = __builtin_bit_cast(v2bf, e);
            n = __builtin_amdgcn_fdot2_f32_bf16(p, p, n, false);
        }
    } else {
        typedef _Float16 v2h __attribute__((ext_vector_type(2)));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int e = v[i];
            const v2h p = __builtin_bit_cast(v2h, e);
            n = __builtin_amdgcn_fdot2(p, p, n, false);
        }
    }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
    for (int d = kWave / 2; d > 0; d >>= 1) v += __shfl_xor(v, d, kWave);
    return v;
}
// Largest value of the wave, in every lane (a scalar): DPP shifts by 1, 2, 4
// and 8 within rows of 16 lanes, the row ends to the next row, row 1's end to
// rows 2 and 3; lane 63 then holds it. `low` is what an absent lane counts as.
template <typename I>
__device__ __forceinline__ I wave_max_int(I v, I low) {
    auto step = [&](auto ctrl) {
        const I o = static_cast<I>(__builtin_amdgcn_update_dpp(static_cast<int>(low), static_cast<int>(v),
                                                               decltype(ctrl)::value, 0xF, 0xF, false));
        v = v > o ? v : o;
    };
    step(std::integral_constant<int, 0x111>{});
    step(std::integral_constant<int, 0x112>{});
    step(std::integral_constant<int, 0x114>{});
    step(std::integral_constant<int, 0x118>{});
    step(std::integral_constant<int, 0x142>{});
    step(std::integral_constant<int, 0x143>{});
    return static_cast<I>(__builtin_amdgcn_readlane(static_cast<int>(v), kWave - 1));
}
__device__ __forceinline__ int64_t wave_max(int64_t v) {
    const int32_t hi = wave_max_int<int32_t>(static_cast<int32_t>(v >> 32), INT32_MIN);
    const uint32_t lo = wave_max_int<uint32_t>(static_cast<int32_t>(v >> 32) == hi ? static_cast<uint32_t>(v) : 0u, 0u);
    return (static_cast<int64_t>(hi) << 32) | lo;
}
// A double as an integer of the same order; NaN and -infinity are the least.
constexpr int64_t kNone = INT64_MIN;
__device__ __forceinline__ int64_t key_of(double v) {
    const int64_t b = __builtin_bit_cast(int64_t, v);
    return v > -__builtin_inf() ? b ^ (b >> 63 & INT64_MAX) : kNone;
}
__device__ __forceinline__ double value_of(int64_t k) {
    return __builtin_bit_cast(double, k ^ (k >> 63 & INT64_MAX));
}

// Fragments of 32 h, in the two ways that the logits are summed: `sum` += in
// fp64; fast(): FOLD steps are summed in fp32 first.
template <typename T, typename W, bool FAST, int TM, int TN>
struct Tiles {
    v4d sum[TM][TN];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j) sum[i][j] = v4d{0.0, 0.0, 0.0, 0.0};
    }
    // The planes of W come smallest first: what their sums are off by is then
    // 2^-7 of a plane's, and with a plane more or less the bound stays n * kUnit
    // (times 1.05, which the choice takes).
    template <int FOLD, int PLANES>
    __device__ __forceinline__ void fast(const v4i (&x)[FOLD][TM], const v4i (&w)[PLANES][FOLD][TN]) {
        v4f acc[TM][TN];
#pragma unroll
        for (int p = PLANES - 1; p >= 0; --p)
#pragma unroll
            for (int s = 0; s < FOLD; ++s)
#pragma unroll
                for (int i = 0; i < TM; ++i)
#pragma unroll
                    for (int j = 0; j < TN; ++j)
                        acc[i][j] = mfma32<T>(x[s][i], w[p][s][j],
                                              p == PLANES - 1 && s == 0 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : acc[i][j]);
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) sum[i][j][q] += static_cast<double>(acc[i][j][q]);
    }
    // the MFMA takes four h, one per lane quarter: h = 8 kq + e for step e
    __device__ __forceinline__ void full(const T (&x)[TM][kVec], const W (&w)[TN][kVec]) {
#pragma unroll
        for (int e = 0; e < kVec; ++e)
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j)
                    sum[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(static_cast<double>(to_f32(x[i][e])),
                                                                     static_cast<double>(to_f32(w[j][e])), sum[i][j],
                                                                     0, 0, 0);
    }
    // into part `part` of the workspace; token tiles from t0, expert tiles from e0
    __device__ __forceinline__ void store(const GateArgs &a, int part, int t0, int e0, int lane) {
#pragma unroll
        for (int i = 0; i < TM; ++i)
#pragma unroll
            for (int j = 0; j < TN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    // result registers: fp32 D rows 4 * (l / 16) + q, fp64 D rows l / 16 + 4 * q
                    const int t = t0 + i * 16 + (FAST ? 4 * (lane >> 4) + q : (lane >> 4) + 4 * q);
                    const int e = e0 + j * 16 + (lane & 15);
                    if (t < a.T && e < a.E) {
                        const size_t o = (static_cast<size_t>(part) * a.T + t) * a.E + e;
                        a.logits[o] = sum[i][j][q];
                    }
                }
    }
};

// Small products: workgroup (16 experts, part, 16 tokens), its four waves take
// every fourth chunk of the part. Lane l loads row l % 16, eight h from 8 * (l
// / 16) of each step, straight from memory: there is too little of it for LDS
// to pay, and 16 x 16 tiles are enough workgroups. fp64 MFMA, also for bf16 and
// fp16: at these sizes its time is less than that of computing the one doubtful
// choice again that a batch of fp32 sums has as a rule (T 64, E 256, H 4096:
// 11 us against 15).
constexpr int kSlices = 4;
template <typename T, typename W>
__global__ __launch_bounds__(kBlock) void logits_few_kernel(GateArgs a, int chunks_per_part) {
    static_assert(kSlices * kWave == kBlock, "one slice per wave");
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int r = lane & 15, kq = lane >> 4;
    const int e0 = blockIdx.x * 16, part = blockIdx.y, t0 = blockIdx.z * 16;
    // rows past the end read the last one; their results are not stored
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(min(t0 + r, a.T - 1)) * a.H;
    const W *w = static_cast<const W *>(a.weight) + static_cast<size_t>(min(e0 + r, a.E - 1)) * a.H;
    Tiles<T, W, false, 1, 1> tile;
    tile.clear();
    const int c_end = min((part + 1) * chunks_per_part, (a.H + kChunk - 1) / kChunk);
    auto chunk = [&](auto whole, int c) {
        T xv[kChunk / kStep][1][kVec];
        W wv[kChunk / kStep][1][kVec];
#pragma unroll
        for (int s = 0; s < kChunk / kStep; ++s) {
            const int k = c * kChunk + s * kStep + kq * kVec;
            load8<decltype(whole)::value>(x, k, a.H, xv[s][0]);
            load8<decltype(whole)::value>(w, k, a.H, wv[s][0]);
        }
#pragma unroll
        for (int s = 0; s < kChunk / kStep; ++s) tile.full(xv[s], wv[s]);
    };
    for (int c = part * chunks_per_part + wave; c < c_end; c += kSlices) {
        if ((c + 1) * kChunk <= a.H) chunk(std::true_type{}, c);
        else chunk(std::false_type{}, c);
    }
    __shared__ v4d s_sum[kSlices - 1][kWave];
    if (wave > 0) s_sum[wave - 1][lane] = tile.sum[0][0];
    __syncthreads();
    if (wave > 0) return;
#pragma unroll
    for (int i = 0; i < kSlices - 1; ++i) tile.sum[0][0] += s_sum[i][lane];
    tile.store(a, part, t0, e0, lane);
}

// Large products: workgroups of 64 tokens x 64 experts, a wave 32 x 32 of them.
// Lanes that load MFMA fragments straight from rows touch 16 rows with 16
// bytes each, four times the requests of whole lines, which is what bound such
// a kernel (66 us at T 4096, E 256, H 4096); so 128 h of the 128 rows go
// through LDS, the next ones on their way in registers meanwhile. 16-byte slot
// c of a row lies at slot c ^ (row % 16): writes of a row and reads of 16
// rows' fragments both meet every bank once.
constexpr int kTileRows = 64;
template <typename T>
struct Stage {  // kTileRows rows of kChunk elements
    static constexpr int kSlots = kChunk * sizeof(T) / 16;           // per row
    static constexpr int kPer = kTileRows * kSlots / kBlock;         // per thread
    static constexpr int kBytes = kTileRows * kSlots * 16;
    static constexpr int kElems = 16 / sizeof(T);
    const T *p[kPer];  // where the thread's slots of the first chunk lie
    int k;             // and their element (the same for all of them)
    static_assert(kBlock % kSlots == 0, "a thread's slots are one column");
    // rows past the end read the last one
    __device__ __forceinline__ void start(const T *base, int row0, int rows, int H) {
        k = static_cast<int>(threadIdx.x) % kSlots * kElems;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int row = min(row0 + static_cast<int>(threadIdx.x + i * kBlock) / kSlots, rows - 1);
            p[i] = base + static_cast<size_t>(row) * H + k;
        }
    }
    template <bool WHOLE>
    __device__ __forceinline__ void fetch(int c, int H, v4i (&v)[kPer]) const {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            if (WHOLE || c * kChunk + k + kElems <= H) {
                __builtin_memcpy(&v[i], p[i] + c * kChunk, 16);
            } else {
                T raw[kElems];
#pragma unroll
                for (int e = 0; e < kElems; ++e) {
                    raw[e] = T{};
                    if (c * kChunk + k + e < H) raw[e] = p[i][c * kChunk + e];
                }
                __builtin_memcpy(&v[i], raw, 16);
            }
        }
    }
    static __device__ __forceinline__ void put(char *lds, const v4i (&v)[kPer]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int slot = threadIdx.x + i * kBlock, row = slot / kSlots, c = slot % kSlots;
            *reinterpret_cast<v4i *>(lds + (row * kSlots + (c ^ (row & 15))) * 16) = v[i];
        }
    }
    // fp32 slots as three planes of bf16: the upper 8 of the 24 bits, the next
    // and the last (a truncation and an exact difference each)
    static constexpr int kPlaneBytes = kTileRows * kChunk * 2;
    static __device__ __forceinline__ void put_planes(char *lds, const v4i (&v)[kPer]) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int slot = threadIdx.x + i * kBlock, row = slot / kSlots, c = slot % kSlots;
            float f[4];
            __builtin_memcpy(f, &v[i], 16);
#pragma unroll
            for (int p = 0; p < kMaxPlanes; ++p) {
                uint32_t b[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    b[e] = __float_as_uint(f[e]);
                    f[e] = f[e] - __uint_as_float(b[e] & 0xFFFF0000u);
                }
                const uint64_t pair = __builtin_amdgcn_perm(b[1], b[0], 0x07060302) |
                                      static_cast<uint64_t>(__builtin_amdgcn_perm(b[3], b[2], 0x07060302)) << 32;
                *reinterpret_cast<uint64_t *>(lds + p * kPlaneBytes + (row * 16 + ((c / 2) ^ (row & 15))) * 16 + c % 2 * 8) = pair;
            }
        }
    }
    // eight elements of a row from element k (a multiple of 8)
    static __device__ __forceinline__ void get(const char *lds, int row, int k, T (&out)[kVec]) {
#pragma unroll
        for (int i = 0; i < static_cast<int>(kVec * sizeof(T) / 16); ++i) {
            const int c = k / kElems + i;
            __builtin_memcpy(&out[i * kElems], lds + (row * kSlots + (c ^ (row & 15))) * 16, 16);
        }
    }
};

// Steps that are summed in fp32 before the fp64 sum: 64 products. Logits and
// choice at E 256, two / four steps: T 4096, H 4096 48 / 50 us, T 8192, H 7168
// 100 / 104 (a wider bound leaves more tokens open); one step: fewer open
// tokens, but 3 us more in all.
constexpr int kFold = 2;

// Registers for three workgroups per CU where their LDS fits: T 8192, H 7168,
// with the choice 95 us instead of 100.
template <typename T, typename W, int PLANES>
constexpr int kPerCu = sizeof(T) + (PLANES > 1 ? 2 * PLANES : sizeof(W)) > 6 ? 2 : 3;
template <typename T, typename W, int PLANES>
__global__ __launch_bounds__(kBlock, (kPerCu<T, W, PLANES>)) void logits_many_kernel(GateArgs a, int chunks_per_part, int e_tiles, int units) {
    constexpr bool FAST = PLANES > 0;
    __shared__ __attribute__((aligned(16))) char s_x[Stage<T>::kBytes];
    __shared__ __attribute__((aligned(16))) char s_w[PLANES > 1 ? PLANES * Stage<T>::kBytes : Stage<W>::kBytes];
    // The expert tiles of one unit (token tile, part) read the same x: they
    // get block numbers that are equal modulo 8, so that one XCD's L2 serves
    // them all.
    const int unit = static_cast<int>(blockIdx.x >> 3) / e_tiles * 8 + static_cast<int>(blockIdx.x & 7);
    if (unit >= units) return;
    const int t_tiles = (a.T + kTileRows - 1) / kTileRows;
    const int t0 = unit % t_tiles * kTileRows, part = unit / t_tiles;
    const int e0 = static_cast<int>(blockIdx.x >> 3) % e_tiles * kTileRows;
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int r = lane & 15, kq = lane >> 4;
    const int tm = (wave >> 1) * 32, en = (wave & 1) * 32;
    Tiles<T, W, FAST, 2, 2> tile;
    tile.clear();
    Stage<T> sx;
    Stage<W> sw;
    sx.start(static_cast<const T *>(a.x), t0, a.T, a.H);
    sw.start(static_cast<const W *>(a.weight), e0, a.E, a.H);
    float xn[Stage<T>::kPer] = {}, wn[Stage<W>::kPer] = {};  // squares of the thread's slots
    struct Chunk {
        v4i x[Stage<T>::kPer], w[Stage<W>::kPer];
    };
    auto fetch = [&](auto whole, int c, Chunk &f) {
        sx.template fetch<decltype(whole)::value>(c, a.H, f.x);
        sw.template fetch<decltype(whole)::value>(c, a.H, f.w);
    };
    auto put = [&](const Chunk &f) {
        __syncthreads();
        Stage<T>::put(s_x, f.x);
        if constexpr (PLANES > 1) Stage<W>::put_planes(s_w, f.w);
        else Stage<W>::put(s_w, f.w);
        if constexpr (FAST) {
#pragma unroll
            for (int i = 0; i < Stage<T>::kPer; ++i) add_squares<T>(f.x[i], xn[i]);
#pragma unroll
            for (int i = 0; i < Stage<W>::kPer; ++i) add_squares<W>(f.w[i], wn[i]);
        }
        __syncthreads();
    };
    auto multiply = [&] {
        if constexpr (FAST) {
#pragma unroll
            for (int s = 0; s < kChunk / kStep; s += kFold) {
                v4i xf[kFold][2], wf[PLANES][kFold][2];
#pragma unroll
                for (int f = 0; f < kFold; ++f) {
                    const int k = (s + f) * kStep + kq * kVec;
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        T v[kVec];
                        Stage<T>::get(s_x, tm + i * 16 + r, k, v);
                        __builtin_memcpy(&xf[f][i], v, 16);
#pragma unroll
                        for (int p = 0; p < PLANES; ++p) {  // a plane lies as 16-bit elements do
                            Stage<T>::get(s_w + p * Stage<T>::kBytes, en + i * 16 + r, k, v);
                            __builtin_memcpy(&wf[p][f][i], v, 16);
                        }
                    }
                }
                tile.template fast<kFold, PLANES>(xf, wf);
            }
        } else {
#pragma unroll
            for (int s = 0; s < kChunk / kStep; ++s) {
                T xv[2][kVec];
                W wv[2][kVec];
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    Stage<T>::get(s_x, tm + i * 16 + r, s * kStep + kq * kVec, xv[i]);
                    Stage<W>::get(s_w, en + i * 16 + r, s * kStep + kq * kVec, wv[i]);
                }
                tile.full(xv, wv);
            }
        }
    };
    // The next whole chunk is loaded meanwhile, and past the last one that one
    // again: no load is conditional, so the compiler's wait counts are exact
    // (T 8192, H 7168, with the choice 117 -> 100 us; two ahead 106).
    const int c0 = part * chunks_per_part, c_end = min(c0 + chunks_per_part, (a.H + kChunk - 1) / kChunk);
    const int whole_end = min(c_end, a.H / kChunk);
    Chunk chunk;
    if (c0 < whole_end) fetch(std::true_type{}, c0, chunk);
    for (int c = c0; c < whole_end; ++c) {
        put(chunk);
        fetch(std::true_type{}, min(c + 1, whole_end - 1), chunk);
        multiply();
    }
    if (whole_end < c_end) {
        fetch(std::false_type{}, whole_end, chunk);
        put(chunk);
        multiply();
    }
    tile.store(a, part, t0 + tm, e0 + en, lane);
    if constexpr (FAST) {  // a row's slots lie in neighbouring lanes, 16 of them or 32
        auto put = [&](float n, int lanes, int i, bool mine, int row0, int rows, float *out) {
            for (int d = lanes / 2; d > 0; d >>= 1) n += __shfl_xor(n, d, kWave);
            const int row = row0 + static_cast<int>(threadIdx.x + i * kBlock) / lanes;
            if (mine && (lane & (lanes - 1)) == 0 && row < rows) out[part * rows + row] = n;
        };
#pragma unroll
        for (int i = 0; i < Stage<T>::kPer; ++i) put(xn[i], Stage<T>::kSlots, i, e0 == 0, t0, a.T, a.x_norms);
#pragma unroll
        for (int i = 0; i < Stage<W>::kPer; ++i) put(wn[i], Stage<W>::kSlots, i, t0 == 0, e0, a.E, a.w_norms);
    }
}

// The logits of experts e0 and e1 in fp64, by the whole wave: two at a time,
// since a doubt is between two as a rule, and both rows' loads overlap.
template <typename T, typename W>
__device__ __forceinline__ void exact_logits(const GateArgs &a, int t, int e0, int e1, int lane, double &l0, double &l1) {
    const T *x = static_cast<const T *>(a.x) + static_cast<size_t>(t) * a.H;
    const W *w0 = static_cast<const W *>(a.weight) + static_cast<size_t>(e0) * a.H;
    const W *w1 = static_cast<const W *>(a.weight) + static_cast<size_t>(e1) * a.H;
    double s0 = 0.0, s1 = 0.0;
    constexpr int kBatch = 2;  // loads in flight, written out: a loop that adds as it loads waits for each
    auto add = [&](auto whole, int i) {
        T u[kBatch][kVec];
        W v0[kBatch][kVec], v1[kBatch][kVec];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int k = i + (b * kWave + lane) * kVec;
            load8<decltype(whole)::value>(x, k, a.H, u[b]);
            load8<decltype(whole)::value>(w0, k, a.H, v0[b]);
            load8<decltype(whole)::value>(w1, k, a.H, v1[b]);
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                const double xv = static_cast<double>(to_f32(u[b][j]));
                s0 = fma(xv, static_cast<double>(to_f32(v0[b][j])), s0);
                s1 = fma(xv, static_cast<double>(to_f32(v1[b][j])), s1);
            }
    };
    int i0 = 0;
    for (; i0 + kBatch * kWave * kVec <= a.H; i0 += kBatch * kWave * kVec) add(std::true_type{}, i0);
    if (i0 < a.H) add(std::false_type{}, i0);
    l0 = wave_sum(s0);
    l1 = wave_sum(s1);
}

template <typename T>
__device__ __forceinline__ bool row_is_zero(const GateArgs &a, const T *x, int lane) {
    uint32_t any = 0;
    for (int k = lane * kVec; k < a.H; k += kWave * kVec) {
        T u[kVec];
        load8<false>(x, k, a.H, u);
#pragma unroll
        for (int e = 0; e < kVec; ++e) any |= u[e].bits & 0x7FFFu;
    }
    return __ballot(any != 0) == 0;
}

// Score of a logit (softmax: before the division by the sum; m = the largest
// logit, finite). NaN of NaN.
template <int SCORE>
__device__ __forceinline__ double score_of(double l, double m) {
    if constexpr (SCORE == MOE_SCORE_SOFTMAX) return exp(l - m);
    if constexpr (SCORE == MOE_SCORE_SIGMOID) return 1.0 / (1.0 + exp(-l));
    return sqrt(fmax(l, 0.0) + log1p(exp(-fabs(l))));
}

// One wave per token; lane l holds experts l, l + 64, ... (NPL of them).
// FAST: the logits are bounded fp32 sums of T and W; else they are 64-bit sums,
// and T and W do not matter.
//
// K choices in order. FAST, an expert that lies closer than `off` below a
// choice is marked, and so is that choice (all experts, where an fp32 sum is
// not finite); the marked ones' logits are then computed in fp64 and the choice
// is made again. An unmarked expert is further than `off` from all that it was
// compared with, so its place stands.
//
// A token is a chain of reductions, and few tokens are a single wave's
// latency, most of it instruction fetches of a kernel that runs once: scores
// are a template parameter and the second choice shares the first one's code
// (13 -> 6 us at 8 tokens, 256 experts, with the loads issued together).
template <bool FAST, typename T, typename W, int SCORE, int NPL>
__global__ __launch_bounds__(kBlock) void choose_kernel(GateArgs a, int parts, double gamma) {
    const int lane = threadIdx.x & (kWave - 1);
    const int t = blockIdx.x * (kBlock / kWave) + threadIdx.x / kWave;
    if (t >= a.T) return;
    double l[NPL];  // logits
    float n[NPL];   // squares of the experts' rows
    float xn = 0.0f;
    float bias[NPL];
    // Loads without branches between them: lanes past the end read the last
    // expert, and without a bias the workspace's first words are read instead.
    const float *bp = a.bias ? a.bias : reinterpret_cast<const float *>(a.logits);
    const size_t row = static_cast<size_t>(t) * a.E, stride = static_cast<size_t>(a.T) * a.E;
    constexpr int kBatch = NPL > 4 ? 1 : 4;  // parts in flight
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        l[j] = 0.0;
        n[j] = 0.0f;
        bias[j] = bp[min(j * kWave + lane, a.E - 1)];
    }
    for (int p = 0; p < parts; p += kBatch) {
        double lv[kBatch][NPL];
        float nv[kBatch][NPL], xv[kBatch];
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            const int q = min(p + b, parts - 1);  // past the last part: read it again, add nothing
            const size_t o = q * stride + row;
            if (FAST) xv[b] = a.x_norms[q * a.T + t];
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                const int e = min(j * kWave + lane, a.E - 1);
                lv[b][j] = a.logits[o + e];
                if (FAST) nv[b][j] = a.w_norms[q * a.E + e];
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
            if (p + b >= parts) continue;
            if (FAST) xn += xv[b];
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                l[j] += lv[b][j];
                if (FAST) n[j] += nv[b][j];
            }
        }
    }
    // How far two choice values may be off together. Slopes: sigmoid 1/4,
    // sqrt(softplus) under 1/3. (Softmax goes by the logit: with a bias its
    // logits are in 64 bits.)
    double off = 0.0;
    uint32_t overflowed = 0;  // bit j: expert j * 64 + lane
    if constexpr (FAST) {
        float wn = 0.0f;  // squares order like their bits; rows with a NaN have no logit to be told from others
#pragma unroll
        for (int j = 0; j < NPL; ++j) wn = n[j] > wn ? n[j] : wn;
        wn = __uint_as_float(wave_max_int<uint32_t>(__float_as_uint(wn), 0u));
        off = 2.0 * (gamma * 1.05 * sqrt((xn + kTinySquares) * (wn + kTinySquares)) + kTiny);
        if (a.bias) off *= SCORE == MOE_SCORE_SIGMOID ? 0.25 : 0.34;
        // and the 64-bit roundings of score + bias
        float bm = 1.0f;
#pragma unroll
        for (int j = 0; j < NPL; ++j) bm = a.bias && fabsf(bias[j]) < __builtin_inff() ? fmaxf(bm, fabsf(bias[j])) : bm;
        bm = __uint_as_float(wave_max_int<uint32_t>(__float_as_uint(bm), 0u));
        off += 0x1p-50 * static_cast<double>(bm);
        // A row of zeros (a padded batch): its logits are 0, all of them equal
        // and right. Without this 243 us instead of 10 for two such rows of 8.
        if (xn == 0.0f && row_is_zero(a, static_cast<const T *>(a.x) + static_cast<size_t>(t) * a.H, lane)) {
            off = -__builtin_inf();
        } else {
            // An fp32 sum that is infinite or NaN says nothing, it may have
            // overflowed, and key_of would leave its expert out: then every
            // logit is computed again. (Not where x or the expert's row hold a
            // NaN, which their squares show: that logit is NaN. Nor where the
            // bias leaves the expert out.)
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (j * kWave + lane < a.E && !(fabs(l[j]) < __builtin_inf()) && xn == xn && n[j] == n[j] &&
                    (!a.bias || bias[j] > -__builtin_inff()))
                    overflowed |= 1u << j;
            if (__ballot(overflowed != 0)) off = __builtin_inf();
        }
    }
    double s[NPL], total;  // scores (softmax: undivided, `total` their sum)
    int id_mine;           // lane k keeps the k-th choice
    for (bool again = false;; again = true) {
        double top = 0.0;
        total = 1.0;
        if constexpr (SCORE == MOE_SCORE_SOFTMAX) {
            int64_t k = kNone;
#pragma unroll
            for (int j = 0; j < NPL; ++j) {
                if (j * kWave + lane >= a.E) l[j] = -__builtin_inf();
                k = max(k, key_of(l[j]));
            }
            top = value_of(wave_max(k));
            total = 0.0;
            if (top > __DBL_MAX__) {  // the infinite ones share alike, the others have nothing
#pragma unroll
                for (int j = 0; j < NPL; ++j) l[j] = l[j] > __DBL_MAX__ ? __DBL_MAX__ : l[j];
                top = __DBL_MAX__;
            }
        }
        int64_t c[NPL];  // what the choice goes by
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            s[j] = score_of<SCORE>(l[j], top);
            if (SCORE == MOE_SCORE_SOFTMAX && s[j] == s[j]) total += s[j];  // an expert with a NaN logit is not there
        }
        if (SCORE == MOE_SCORE_SOFTMAX) total = wave_sum(total);
#pragma unroll
        for (int j = 0; j < NPL; ++j) {
            double v = l[j];
            if (a.bias) v = (SCORE == MOE_SCORE_SOFTMAX ? s[j] / total : s[j]) + static_cast<double>(bias[j]);
            c[j] = j * kWave + lane < a.E ? key_of(v) : kNone;
        }
        id_mine = -1;
        int64_t c_mine = kNone;
        for (int k = 0; k < a.K; ++k) {
            int64_t best = c[0];
#pragma unroll
            for (int j = 1; j < NPL; ++j) best = max(best, c[j]);
            best = wave_max(best);
            if (best == kNone) break;  // nothing is left
            int id = 0;                // its lowest expert
#pragma unroll
            for (int j = NPL - 1; j >= 0; --j) {
                const unsigned long long equal = __ballot(c[j] == best);
                if (equal) id = j * kWave + __builtin_ctzll(equal);
            }
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (j * kWave + lane == id) c[j] = kNone;
            if (lane == k) {
                c_mine = best;
                id_mine = id;
            }
        }
        if constexpr (!FAST) {
            break;
        } else {
            if (again) break;
            // neighbours in the order that are closer than `off`: lane k
            // against lane k + 1, the last choice against all that are left
            const double mine = value_of(c_mine);
            const bool chosen = id_mine >= 0;
            const int count = __popcll(__ballot(chosen));
            const double next = value_of(__shfl_down(c_mine, 1, kWave));
            const double last = value_of(__shfl(c_mine, max(count - 1, 0), kWave));
            uint32_t marked = 0;  // bit j: expert j * 64 + lane
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (c[j] != kNone && !(last - value_of(c[j]) > off)) marked |= 1u << j;
            const unsigned long long left = __ballot(marked != 0);
            const unsigned long long near = __ballot(chosen && lane + 1 < count && !(mine - next > off)) |
                                            (left && count > 0 ? 1ull << (count - 1) : 0);
#pragma unroll
            for (int j = 0; j < NPL; ++j)
                if (overflowed >> j & 1) marked |= 1u << j;
            if (!__ballot(marked != 0) && !near) break;
            unsigned long long todo = near | near << 1;  // both of a pair
            todo &= (1ull << count) - 1;                 // count <= kMaxTopK
            while (todo) {
                const int id = __builtin_amdgcn_readlane(id_mine, __builtin_ctzll(todo));
                todo &= todo - 1;
                if (lane == (id & (kWave - 1))) marked |= 1u << (id / kWave);
            }
            for (;;) {
                int e[2] = {-1, -1};  // the next two marked experts
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const unsigned long long some = __ballot(marked != 0);
                    if (!some) continue;  // uniform
                    const int lo = __builtin_ctzll(some);
                    const int j = __builtin_ctz(__builtin_amdgcn_readlane(marked, lo));
                    e[i] = j * kWave + lo;
                    if (lane == lo) marked &= ~(1u << j);
                }
                if (e[0] < 0) break;
                double v[2];
                exact_logits<T, W>(a, t, e[0], e[1] < 0 ? e[0] : e[1], lane, v[0], v[1]);
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int j = 0; j < NPL; ++j)
                        if (j * kWave + lane == e[i]) l[j] = v[i];
            }
        }
    }
    double w = 0.0;  // the score of lane k's choice
#pragma unroll
    for (int j = 0; j < NPL; ++j) {
        const double v = __shfl(s[j], id_mine & (kWave - 1), kWave);
        if (id_mine >= 0 && id_mine / kWave == j) w = v;
    }
    if (a.normalize) {
        double sum = w;
#pragma unroll
        for (int d = kMaxTopK / 2; d > 0; d >>= 1) sum += __shfl_xor(sum, d, kWave);
        if (sum > 0.0) w = w / sum;
    } else if (SCORE == MOE_SCORE_SOFTMAX) {
        w = w / total;
    }
    if (lane < a.K) {
        const size_t o = static_cast<size_t>(t) * a.K + lane;
        a.ids[o] = id_mine;
        a.scales[o] = id_mine < 0 ? 0.0f : static_cast<float>(w * static_cast<double>(a.route_scale));
    }
}

// Experts per lane: the fewest that hold E (E 384, H 7168, logits and choice, 8
// / 16 per lane: T 8 14.2 / 18.4 us, T 2048 61 / 70).
template <bool FAST, typename T, typename W, int SCORE>
void choose_score(const GateArgs &a, int parts, double gamma, hipStream_t s) {
    const dim3 grid((a.T + kBlock / kWave - 1) / (kBlock / kWave)), blk(kBlock);
    if (a.E <= kWave) hipLaunchKernelGGL((choose_kernel<FAST, T, W, SCORE, 1>), grid, blk, 0, s, a, parts, gamma);
    else if (a.E <= 2 * kWave) hipLaunchKernelGGL((choose_kernel<FAST, T, W, SCORE, 2>), grid, blk, 0, s, a, parts, gamma);
    else if (a.E <= 4 * kWave) hipLaunchKernelGGL((choose_kernel<FAST, T, W, SCORE, 4>), grid, blk, 0, s, a, parts, gamma);
    else if (a.E <= 8 * kWave) hipLaunchKernelGGL((choose_kernel<FAST, T, W, SCORE, 8>), grid, blk, 0, s, a, parts, gamma);
    else hipLaunchKernelGGL((choose_kernel<FAST, T, W, SCORE, 16>), grid, blk, 0, s, a, parts, gamma);
}
template <bool FAST, typename T, typename W>
void choose(const GateArgs &a, int parts, double gamma, hipStream_t s) {
    if (a.score == MOE_SCORE_SOFTMAX) choose_score<FAST, T, W, MOE_SCORE_SOFTMAX>(a, parts, gamma, s);
    else if (a.score == MOE_SCORE_SIGMOID) choose_score<FAST, T, W, MOE_SCORE_SIGMOID>(a, parts, gamma, s);
    else choose_score<FAST, T, W, MOE_SCORE_SQRT_SOFTPLUS>(a, parts, gamma, s);
}

// Which kernel, by the products T * E * H. Logits and choice together, H 4096,
// 16 x 16 / 64 x 64 tiles, in us: bf16, E 256, T 32 10 / 20, T 256 19 / 23, T
// 300 23.7 / 23.2, T 512 31 / 26; E 128, T 509 19 / 21.5. fp64 MFMA in both: E
// 256, T 128 15 / 29, T 512 36 / 32; T 509, E 72, H 2501 15 / 23. Rows under a
// chunk per wave leave waves idle: T 1024, E 1024, H 256 35 / 32.
constexpr int64_t kFewUpTo = int64_t(1) << 28;

// Parts of H: two workgroups per CU where that takes no more than kMaxSplit
// parts (T 4096, E 256, with the choice: 48 us, three 49, four 51), of at least
// one chunk per wave (small products; two: T 8 10.1 us instead of 9.2) or two
// per workgroup.
struct Plan {
    bool few;
    int t_tiles, e_tiles, parts, chunks_per_part;
};
Plan plan_of(int T, int E, int H) {
    Plan p;
    p.few = T <= 16 || (H >= kSlices * kChunk && static_cast<int64_t>(T) * E * H <= kFewUpTo);
    const int rows = p.few ? 16 : kTileRows, chunks = (H + kChunk - 1) / kChunk;
    p.t_tiles = (T + rows - 1) / rows;
    p.e_tiles = (E + rows - 1) / rows;
    int parts = (512 + p.t_tiles * p.e_tiles - 1) / (p.t_tiles * p.e_tiles);
    parts = min(min(parts, kMaxSplit), chunks / (p.few ? kSlices : 2));
    parts = max(parts, 1);
    p.chunks_per_part = (chunks + parts - 1) / parts;
    p.parts = (chunks + p.chunks_per_part - 1) / p.chunks_per_part;
    return p;
}

template <typename T, typename W>
hipError_t launch(const GateArgs &a, hipStream_t s) {
    const Plan p = plan_of(a.T, a.E, a.H);
    GateArgs g = a;
    g.x_norms = reinterpret_cast<float *>(a.logits + static_cast<size_t>(p.parts) * a.T * a.E);
    g.w_norms = g.x_norms + static_cast<size_t>(p.parts) * a.T;
    // Whether the logits are bounded fp32 sums. Not for softmax with a bias:
    // what is ordered there, share + bias, holds the sum over all experts, so
    // that exact logits of the doubtful ones alone would not decide (a bias can
    // cancel the difference of two shares to any number of bits). T 4096, E
    // 256, H 4096 takes 157 us so (72 without certainty), T 512 31 (39).
    const bool fast = !p.few && !(a.score == MOE_SCORE_SOFTMAX && a.bias) &&
                      (kPlanes<T, W> == 1 ||
                       (kPlanes<T, W> > 1 && static_cast<int64_t>(a.T) * a.E * a.H > kPlanesFrom));
    if (p.few) {
        hipLaunchKernelGGL((logits_few_kernel<T, W>), dim3(p.e_tiles, p.parts, p.t_tiles), dim3(kBlock), 0, s, g,
                           p.chunks_per_part);
    } else {
        const int units = p.t_tiles * p.parts;
        const dim3 grid((units + 7) / 8 * 8 * p.e_tiles);
        if (fast)
            hipLaunchKernelGGL((logits_many_kernel<T, W, kPlanes<T, W>>), grid, dim3(kBlock), 0, s, g,
                               p.chunks_per_part, p.e_tiles, units);
        else
            hipLaunchKernelGGL((logits_many_kernel<T, W, 0>), grid, dim3(kBlock), 0, s, g, p.chunks_per_part,
                               p.e_tiles, units);
    }
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const double gamma = kStep * kFold * kUnit;
    if constexpr (kPlanes<T, W> > 0) {
        if (fast) choose<true, T, W>(g, p.parts, gamma, s);
    }
    if (!fast) choose<false, float, float>(g, p.parts, gamma, s);
    return hipGetLastError();
}

}  // namespace

// What plan_of's parts take, or more, so that the size never falls as T grows
// (a workspace for the largest batch serves all): parts are at most kMaxSplit
// and chunks / 2, and there is one, or parts * t_tiles * e_tiles < 2 * 512.
size_t gate_workspace(int T, int E, int H) {
    if (T == 0) return 0;
    const size_t parts = max(1, min(kMaxSplit, (H + kChunk - 1) / kChunk / 2)), logits = static_cast<size_t>(T) * E;
    const size_t split = min(parts * logits, size_t(2 * 512) * kTileRows * kTileRows);
    return max(logits, split) * sizeof(double) + parts * (static_cast<size_t>(T) + E) * sizeof(float);
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
