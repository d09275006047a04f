// Dense product in 8-bit integers on MFMA:
//
//   o[t,n] = (float(sum_k x[t,k] * w[n,k]) * ws[n]) * xs[t] + bias[n]
//
// The sum is exact in int32 (|x w| <= 2^14, K <= 2^16), so no split or order
// of it changes a bit. Weight rows are the MFMA's A rows, tokens its B columns:
// one 16 x 16 tile of D covers 16 output rows and 16 tokens, lane l holding
// rows 4 * (l / 16) ..+3 of token l % 16.
//
// The weights are packed in the order in which the lanes take them, 1 KB per
// 16 rows and 64 k, k padded with zeros to whole tiles of 128: whatever x holds
// behind a row's end (the next row's codes) meets zeros.
#include "ops.h"

#include <type_traits>
#include <utility>
#include "../../include/moe_w8a8.h"

namespace moe {
namespace {

typedef int v4i __attribute__((ext_vector_type(4)));

constexpr int kTileK = 128;
constexpr int kTileBytes = 16 * kTileK;  // of weights: two 1 KB blocks of 64 k

// ------------------------------------------------------------------ packing
__device__ __forceinline__ int64_t source_row(const LinearW8Args &a, int nt, int r, bool &ok) {
    const int half = a.N / 2;
    const int unit = a.gated ? nt * 8 + r / 2 : nt * 16 + r;
    ok = unit < (a.gated ? half : a.N);
    return a.gated && (r & 1) ? half + unit : unit;
}
// One thread per 16 bytes: tile, block, lane.
__global__ __launch_bounds__(256) void pack_codes8_kernel(const int8_t *__restrict__ src, int8_t *__restrict__ dst,
                                                          LinearW8Args a) {
    const int64_t o = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    const int64_t tile = o >> 7;
    if (tile >= static_cast<int64_t>(a.n_tiles) * a.k_tiles) return;
    const int l = static_cast<int>(o) & 63, h = static_cast<int>(o >> 6) & 1;
    const int kt = static_cast<int>(tile % a.k_tiles), nt = static_cast<int>(tile / a.k_tiles);
    bool ok;
    const int64_t row = source_row(a, nt, l & 15, ok);
    const int k0 = kt * kTileK + h * 64 + (l >> 4) * 16;
    int8_t v[16] = {};
    const int8_t *from = src + row * a.K + k0;
    if (ok && k0 + 16 <= a.K) {
        __builtin_memcpy(v, from, 16);
    } else if (ok) {
#pragma unroll
        for (int b = 0; b < 16; ++b)
            if (k0 + b < a.K) v[b] = from[b];
    }
    __builtin_memcpy(dst + o * 16, v, 16);
}
__global__ __launch_bounds__(256) void pack_scales8_kernel(const float *__restrict__ scale, float *__restrict__ dst,
                                                           LinearW8Args a) {
    const int o = blockIdx.x * 256 + threadIdx.x;
    if (o >= a.n_tiles * 16) return;
    bool ok;
    const int64_t row = source_row(a, o >> 4, o & 15, ok);
    dst[o] = ok ? scale[row] : 0.0f;
}

// ------------------------------------------------------------------ product

// x of 16 tokens and one 128-k tile in LDS: rows of eight 16-byte slots, slot c
// of row r at place c ^ ((r >> 1) & 7). Whole rows are written, 16 rows' slots
// of one k are read: both meet every bank equally often.
__device__ __forceinline__ int x_at(int row, int slot) { return (row * 8 + (slot ^ ((row >> 1) & 7))) * 16; }

// 16 bytes of x from any address (the hardware takes such accesses).
__device__ __forceinline__ v4i load16(const int8_t *p) {
    v4i v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
__device__ __forceinline__ v4i shift_down(v4i v, int bytes) {
    uint64_t q[2];
    __builtin_memcpy(q, &v, 16);
    const unsigned __int128 w = ((static_cast<unsigned __int128>(q[1]) << 64) | q[0]) >> (min(bytes, 15) * 8);
    q[0] = static_cast<uint64_t>(w);
    q[1] = static_cast<uint64_t>(w >> 64);
    __builtin_memcpy(&v, q, 16);
    return v;
}
// Rows whose length is no multiple of 16 begin anywhere, and the last 16 bytes
// of the last ones may end behind x. The load is moved back to x's last 16
// bytes then, and its bytes back to their places where they are used: only
// the last tile of k needs that. Offsets are from token t0's row.
struct RowEnd {
    int last;   // of the offsets with 16 bytes of x behind them (may be negative)
    int bytes;  // of x, where they are fewer than 16
    __device__ __forceinline__ RowEnd(const LinearW8Args &a, int t0) {
        const int64_t behind = static_cast<int64_t>(a.T - t0) * a.K - 16, all = static_cast<int64_t>(a.T) * a.K;
        last = static_cast<int>(behind < 0x7FFFFFFF ? behind : 0x7FFFFFFF);
        bytes = all < 16 ? static_cast<int>(all) : 0;
    }
    __device__ __forceinline__ v4i load(const int8_t *x, int off) const {
        if (bytes == 0) return load16(x + min(off, last));
        int8_t b[16] = {};
        for (int i = 0; i < bytes; ++i) b[i] = x[i];  // then t0 is 0
        v4i v;
        __builtin_memcpy(&v, b, 16);
        return v;
    }
    __device__ __forceinline__ v4i place(v4i v, int off) const {
        return shift_down(v, max(off - (bytes == 0 ? last : 0), 0));
    }
};

__device__ __forceinline__ uint16_t bits16(float v, bool fp16) {
    return fp16 ? __builtin_bit_cast(uint16_t, static_cast<_Float16>(v)) : __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
}
// Two outputs of type O (MOE_DTYPE_BF16 or FP16) in a word.
template <int O>
__device__ __forceinline__ int pair16(float u, float v) {
    typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
    typedef _Float16 v2h __attribute__((ext_vector_type(2)));
    typedef float v2f __attribute__((ext_vector_type(2)));
    if constexpr (O == MOE_DTYPE_FP16) return __builtin_bit_cast(int, v2h{static_cast<_Float16>(u), static_cast<_Float16>(v)});
    else return __builtin_bit_cast(int, __builtin_convertvector((v2f{u, v}), v2bf));
}

// The finished sums of rows 4 * kq ..+3 of tile nt for token t.
__device__ __forceinline__ void finish(const LinearW8Args &a, int nt, int kq, int t, v4i acc) {
    const float xs = a.x_scale[t];
    float o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = dequant(acc[i], a.scale[nt * 16 + kq * 4 + i], xs);
    const bool wide = a.out_dtype == MOE_DTYPE_FP32, fp16 = a.out_dtype == MOE_DTYPE_FP16;
    const int units = a.gated ? a.N / 2 : a.N, n = a.gated ? nt * 8 + kq * 2 : nt * 16 + kq * 4;
    const int per = a.gated ? 2 : 4;
    if (a.bias) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int unit = a.gated ? n + i / 2 : n + i;
            if (unit < units) o[i] += a.bias[a.gated && (i & 1) ? units + unit : unit];
        }
    }
    if (a.gated) {
        o[0] = swiglu_y(o[0], o[1]);
        o[1] = swiglu_y(o[2], o[3]);
    }
    const size_t at = static_cast<size_t>(t) * units + n;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (i >= per || n + i >= units) break;
        if (wide) static_cast<float *>(a.out)[at + i] = o[i];
        else static_cast<uint16_t *>(a.out)[at + i] = bits16(o[i], fp16);
    }
}

// What bounds it: the weights' bytes, in the few us that a launch and its first
// loads leave of that. T 1, N 4096, K 4096 4.6 us (3.6 TB/s), T 64 6.5; odd rows
// take one shift of the last tile more: T 37, N 5006, K 4251, gated 7.8.
// More waves or tiles ahead are no faster: T 128, N 1383, K 9470 12.1 us, with 16
// waves 12.7; one / two / four tiles ahead (in a captured graph) T 37, N 5006, K
// 4251 8.3 / 8.3 / 8.9, T 1, N 4096, K 4096 5.1 / 5.1 / 5.1, T 8, N 2048, K 16384
// 9.2 / 7.9 / 7.8, T 8, N 28672, K 4096 23.5 / 22.9 / 24.4.
constexpr int kFewWaves = 8;

// Few tokens: a workgroup takes R tiles of 16 weight rows and ROWS tokens, its
// WAVES waves every WAVES-th tile of 128 k, loaded DEPTH tiles ahead; the waves'
// sums meet in LDS.
//
// Whole rows of x are loaded and turned to operands in LDS, in a place of the
// wave's own. Nothing is masked: tokens past the end read the last token's x
// (columns that are not stored), k past the end meets zero weights.
template <int ROWS, int R, bool ODD>
__global__ __launch_bounds__(kFewWaves *kWave) void linear_w8_few_kernel(LinearW8Args a, int token_blocks) {
    constexpr int WAVES = kFewWaves, DEPTH = 2, MT = (ROWS + 15) / 16;
    constexpr int kL = (ROWS + 7) / 8;               // loads of x per tile: 8 rows each
    constexpr int kPer = kL > 1 ? 2 : 1;             // of them per token tile
    constexpr int kBufs = MT > 1 ? 2 : 1;            // token tiles in a wave's place
    constexpr int kSums = R * MT, kJoin = kSums < 8 ? kSums : 8;  // tiles of sums, and those joined at once
    constexpr int kStage = WAVES * kBufs * 2048, kRed = WAVES * kJoin * kWave * 16;
    __shared__ __attribute__((aligned(16))) char lds[kStage > kRed ? kStage : kRed];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, kq = lane >> 4;
    // Workgroups b, b + 8, ... run on one XCD: each gets consecutive pairs of a
    // row block and a token block, token blocks first, so that the weights of a
    // row block come from one XCD's L2. With one token block nothing is shared,
    // and there is no division to wait for.
    const int row_blocks = (a.n_tiles + R - 1) / R, b = static_cast<int>(blockIdx.x);
    int row_block = b, token_block = 0;
    if (token_blocks > 1) {
        const int pair = (b & 7) * static_cast<int>(gridDim.x >> 3) + (b >> 3);
        row_block = pair / token_blocks;
        token_block = pair - row_block * token_blocks;
    }
    if (row_block >= row_blocks) return;
    const int nt0 = row_block * R, t0 = token_block * ROWS;
    char *place = lds + wave * kBufs * 2048;
    const int8_t *x = a.x + static_cast<size_t>(t0) * a.K;
    const RowEnd end(a, t0);
    const int count = (a.k_tiles - wave + WAVES - 1) / WAVES;  // the wave's tiles; <= 0: none
    struct Tile {
        v4i codes[R][2];
        v4i x[kL];
    };
    int row_off[kL];  // at most 64 rows of 2^16 bytes
#pragma unroll
    for (int j = 0; j < kL; ++j) row_off[j] = min(j * 8 + lane / 8, a.T - 1 - t0) * a.K;
    auto tile_of = [&](int i) { return wave + min(i, count - 1) * WAVES; };  // past the end: the last one again
    auto offset = [&](int kt, int j) { return row_off[j] + min(kt * kTileK + lane % 8 * 16, ODD ? a.K - 1 : a.K - 16); };
    auto fetch = [&](int i, Tile &f) {
        const int kt = tile_of(i);
#pragma unroll
        for (int j = 0; j < R; ++j) {  // rows past the end: the last tile, not stored
            const int8_t *w = a.codes + (static_cast<size_t>(min(nt0 + j, a.n_tiles - 1)) * a.k_tiles + kt) * kTileBytes + lane * 16;
#pragma unroll
            for (int h = 0; h < 2; ++h) f.codes[j][h] = load16(w + h * 1024);
        }
#pragma unroll
        for (int j = 0; j < kL; ++j) f.x[j] = ODD ? end.load(x, offset(kt, j)) : load16(x + offset(kt, j));
    };
    v4i acc[R][MT];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[j][m] = v4i{0, 0, 0, 0};
    typedef __attribute__((address_space(3))) volatile v4i own_lds;  // one wave's own: in order without a barrier
    auto multiply = [&](int i, Tile &f) {
        if (ODD && tile_of(i) == a.k_tiles - 1) {  // the only tile that reaches behind x
#pragma unroll
            for (int j = 0; j < kL; ++j) f.x[j] = end.place(f.x[j], offset(tile_of(i), j));
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            char *buf = place + m % kBufs * 2048;
#pragma unroll
            for (int j = 0; j < kPer; ++j) *(own_lds *)(buf + x_at(j * 8 + lane / 8, lane % 8)) = f.x[m * kPer + j];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4i xf = *(own_lds *)(buf + x_at(r, h * 4 + kq));
#pragma unroll
                for (int j = 0; j < R; ++j)
                    acc[j][m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.codes[j][h], xf, acc[j][m], 0, 0, 0);
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
                multiply(i + d, ring[d]);
                fetch(i + DEPTH + d, ring[d]);
            }
        }
#pragma unroll
        for (int d = 0; d < DEPTH; ++d)
            if (i + d < count) multiply(i + d, ring[d]);
    }
    v4i(*red)[kJoin][kWave] = reinterpret_cast<v4i(*)[kJoin][kWave]>(lds);
#pragma unroll
    for (int p = 0; p < kSums; p += kJoin) {
        __syncthreads();  // the places, or the sums before, are read until here
#pragma unroll
        for (int i = 0; i < kJoin; ++i) red[wave][i][lane] = acc[(p + i) / MT][(p + i) % MT];
        __syncthreads();
        if (wave >= kJoin) continue;
        v4i sum = red[0][wave][lane];
#pragma unroll
        for (int w = 1; w < WAVES; ++w) sum += red[w][wave][lane];
        const int nt = nt0 + (p + wave) / MT, t = t0 + (p + wave) % MT * 16 + r;
        if (nt < a.n_tiles && t < a.T && (ROWS >= 16 || r < ROWS)) finish(a, nt, kq, t, sum);
    }
}

// Many tokens: the matrix rate is what counts. A workgroup takes 16 MT tokens
// and 64 NW weight rows, NW tiles of 16 for each of its four waves. Only x goes
// through LDS, where all waves read it, one tile of 128 k (a stage) at a time;
// weights come packed in operand order and go from memory to the wave's
// registers, a stage ahead. Per stage a wave reads 2 MT KB of LDS for 2 MT NW
// products of 16 cycles: four waves take 32 MT of their 32 MT NW cycles at 256
// bytes a cycle (a loop of such reads alone reached 208), a quarter of the time
// with NW = 4. (With both operands in LDS and 64 x 64 sums per wave it would be
// half.)
//
// x lies in NB buffers, stage s in buffer s % NB, copied straight to LDS NB - 2
// stages ahead (into a buffer whose operands every wave has multiplied by the
// last barrier, not only asked for), eight rows of 128 bytes an instruction: a lane fetches the
// 16-byte chunk that belongs at its place (x_at). Rows of ODD length are not
// aligned for such copies: they go through registers.
//
// Measured (T, N, K 8192, bf16 out): 2.44 POP/s, the library's int8 product 2.13;
// the matrix units are busy 67 % of the cycles, at the 1.75 GHz that the clock
// falls to under this load; LDS is busy 18 % of them (SQ_LDS_IDX_ACTIVE: a
// quarter of the matrix units' time, and the writes of the end), and what is
// loaded is 30 bytes a cycle and CU. With one workgroup a CU (T 256, N 8192, K
// 4096 or T 512, N 4096: 15.3 us, the operations' 8.1) a SIMD has one wave:
// waves wait for loads and barriers 55 % of their cycles, the matrix units are
// busy 22 %, and L2 gives 13 TB/s where plain reads by as many waves get 28:
// latency. 256 tokens a workgroup (one wave per SIMD) was 35 %
// slower.
typedef __attribute__((address_space(3))) void lds_void;
typedef __attribute__((address_space(1))) void glb_void;
constexpr int kManyWaves = 4;

// The sums of a wave, NW row tiles from nt0 by MT token tiles from t0, to out
// of type O. Lanes hold up to four neighbouring outputs of a token
// each; through LDS of the wave's own (its lanes' accesses in order, for the
// compiler too) they become 16 bytes of a row that neighbouring lanes continue.
template <int NW>
constexpr int kPlaceBytes = 16 * (NW * 16 * 4 + 16);
template <int MT, int NW, int O, bool GATED>
__device__ __forceinline__ void write_sums(const LinearW8Args &a, const v4i (&acc)[NW][MT], int nt0, int t0, int lane,
                                           char *place) {
    typedef int v2i __attribute__((ext_vector_type(2)));
    constexpr int E = O == MOE_DTYPE_FP32 ? 4 : 2;
    constexpr int kUnits = NW * (GATED ? 8 : 16), kRow = kUnits * E + 16;  // outputs of a token, and their bytes in LDS
    constexpr int kPer = 16 / E, kLanes = kUnits / kPer, kTokens = kWave / kLanes;
    const int r = lane & 15, kq = lane >> 4;
    const int units = GATED ? a.N / 2 : a.N, n0 = nt0 * (GATED ? 8 : 16);
    float ws[NW][4], bias[NW][4] = {};
#pragma unroll
    for (int j = 0; j < NW; ++j) {
        const int nt = min(nt0 + j, a.n_tiles - 1);
        __builtin_memcpy(ws[j], a.scale + nt * 16 + kq * 4, 16);
        if (a.bias) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int n = GATED ? nt * 8 + kq * 2 + i / 2 : nt * 16 + kq * 4 + i;
                bias[j][i] = a.bias[min(n, units - 1) + (GATED && (i & 1) ? units : 0)];
            }
        }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const float xs = a.x_scale[min(t0 + m * 16 + r, a.T - 1)];
#pragma unroll
        for (int j = 0; j < NW; ++j) {
            float o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[i] = dequant(acc[j][m][i], ws[j][i], xs);
                if (a.bias) o[i] += bias[j][i];
            }
            char *at = place + r * kRow;
            if constexpr (GATED) {
                const float u = swiglu_y(o[0], o[1]), v = swiglu_y(o[2], o[3]);
                if constexpr (E == 4) {
                    *(__attribute__((address_space(3))) volatile v2i *)(at + j * 32 + kq * 8) =
                        v2i{__float_as_int(u), __float_as_int(v)};
                } else {
                    *(__attribute__((address_space(3))) volatile int *)(at + j * 16 + kq * 4) =
                        pair16<O>(u, v);
                }
            } else if constexpr (E == 4) {
                *(__attribute__((address_space(3))) volatile v4i *)(at + j * 64 + kq * 16) =
                    v4i{__float_as_int(o[0]), __float_as_int(o[1]), __float_as_int(o[2]), __float_as_int(o[3])};
            } else {
                *(__attribute__((address_space(3))) volatile v2i *)(at + j * 32 + kq * 8) =
                    v2i{pair16<O>(o[0], o[1]), pair16<O>(o[2], o[3])};
            }
        }
#pragma unroll
        for (int i = 0; i < (16 + kTokens - 1) / kTokens; ++i) {
            const int row = i * kTokens + lane / kLanes, n = lane % kLanes * kPer, t = t0 + m * 16 + row;
            if (row >= 16 || t >= a.T) continue;
            const v4i v = *(__attribute__((address_space(3))) volatile v4i *)(place + row * kRow + n * E);
            char *p = static_cast<char *>(a.out) + (static_cast<size_t>(t) * units + n0 + n) * E;
            const int left = units - n0 - n;
            if (left >= kPer) store_out(p, v, a.streamed);
            else if (left > 0) {
                char b[16];
                __builtin_memcpy(b, &v, 16);
#pragma unroll
                for (int e = 0; e < kPer; ++e)
                    if (e < left) __builtin_memcpy(p + e * E, b + e * E, E);
            }
        }
    }
}

template <int... I, typename F>
__device__ __forceinline__ void unrolled(std::integer_sequence<int, I...>, F f) {
    (f(std::integral_constant<int, I>{}), ...);
}

template <int MT, int NW, int NB, int WR, bool ODD>
__global__ __launch_bounds__(kManyWaves *kWave, 2) void linear_w8_many_kernel(LinearW8Args a, int token_blocks,
                                                                            int row_blocks) {
    static_assert((NB == 4 && WR == 2) || (NB == 8 && WR == 4), "");
    constexpr int XA = NB - 2;           // stages that x is copied ahead
    constexpr int XO = WR == 4 ? 4 : 2;  // ODD: that it is loaded ahead, to be put two ahead
    constexpr int XR = XO == 4 ? 4 : 1;  // sets of registers for that
    constexpr auto kGroup = std::make_integer_sequence<int, NB>{};
    constexpr int kStage = MT * 2048, kCopies = MT / 2;  // copies of 1 KB per wave and stage
    constexpr int kAhead = MT >= 4 ? 4 : 2;              // operands of x on their way from LDS
    constexpr int kBuffer = kStage > kPlaceBytes<NW> ? kStage : kPlaceBytes<NW>;
    constexpr int kMore = NB == 8 ? kBuffer : 16;
    // arrays of their own, by which the compiler tells copies into one from reads of another
    __shared__ __attribute__((aligned(16))) char s_x0[kBuffer], s_x1[kBuffer], s_x2[kBuffer], s_x3[kBuffer];
    __shared__ __attribute__((aligned(16))) char s_x4[kMore], s_x5[kMore], s_x6[kMore], s_x7[kMore];
    auto buffer = [&](auto i) -> char * {
        constexpr int n = decltype(i)::value % NB;
        if constexpr (n == 0) return s_x0;
        else if constexpr (n == 1) return s_x1;
        else if constexpr (n == 2) return s_x2;
        else if constexpr (n == 3) return s_x3;
        else if constexpr (n == 4) return s_x4;
        else if constexpr (n == 5) return s_x5;
        else if constexpr (n == 6) return s_x6;
        else return s_x7;
    };
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, kq = lane >> 4;

    // Workgroups b, b + 8, ... run on one XCD: each gets consecutive tiles, in
    // groups of 8 token blocks, so that those in flight share both operands in its L2.
    const int total = token_blocks * row_blocks, b8 = total & ~7;
    int b = blockIdx.x;
    if (b < b8) b = (b & 7) * (b8 >> 3) + (b >> 3);
    const int group = b / (8 * row_blocks), in = b - group * 8 * row_blocks;
    const int wide = min(8, token_blocks - group * 8);
    const int t0 = (group * 8 + in % wide) * MT * 16, nt0 = (in / wide * kManyWaves + wave) * NW;

    uint32_t row_off[kCopies];  // of x's rows from token t0's: at most 256 of 2^16 bytes
    int chunk[kCopies];
    const int8_t *x = a.x + static_cast<size_t>(t0) * a.K;
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
        const int row = (wave * kCopies + i) * 8 + lane / 8;  // rows past the end: the last one, not stored
        row_off[i] = static_cast<uint32_t>(min(row, a.T - 1 - t0)) * static_cast<uint32_t>(a.K);
        chunk[i] = ((lane & 7) ^ ((row >> 1) & 7)) * 16;
    }
    const int last = a.k_tiles - 1;
    auto x_off = [&](int s, int i) {  // k past the end: the row's last, which meets zero weights
        return row_off[i] + static_cast<uint32_t>(min(s * kTileK + chunk[i], ODD ? a.K - 1 : a.K - 16));
    };
    auto copy_x = [&](int s, char *buf) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
            __builtin_amdgcn_global_load_lds((glb_void *)(x + x_off(s, i)), (lds_void *)(buf + (wave * kCopies + i) * 1024),
                                             16, 0, 0);
    };
    // ODD: loads that would end behind x are moved back (RowEnd); only the last
    // stage's bytes are moved in turn, by `place`, so that the loop has none of it.
    const RowEnd end(a, t0);
    auto fetch_x = [&](int s, v4i (&v)[kCopies]) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) v[i] = load16(x + min(static_cast<int>(x_off(s, i)), end.last));
    };
    auto put_x = [&](const v4i (&v)[kCopies], char *buf) {
#pragma unroll
        for (int i = 0; i < kCopies; ++i) *reinterpret_cast<v4i *>(buf + (wave * kCopies + i) * 1024 + lane * 16) = v[i];
    };
    auto bring_x = [&](int s, char *buf) {
        v4i v[kCopies];
        fetch_x(s, v);
#pragma unroll
        for (int i = 0; i < kCopies; ++i) v[i] = end.place(v[i], static_cast<int>(x_off(s, i)));
        put_x(v, buf);
    };
    const int8_t *w[NW];  // rows past the end: the last tile, not stored
#pragma unroll
    for (int j = 0; j < NW; ++j)
        w[j] = a.codes + static_cast<size_t>(min(nt0 + j, a.n_tiles - 1)) * a.k_tiles * kTileBytes + lane * 16;
    auto fetch_w = [&](int s, v4i (&f)[NW][2]) {
#pragma unroll
        for (int j = 0; j < NW; ++j)
#pragma unroll
            for (int h = 0; h < 2; ++h) f[j][h] = load16(w[j] + static_cast<size_t>(s) * kTileBytes + h * 1024);
    };
    v4i acc[NW][MT];
#pragma unroll
    for (int j = 0; j < NW; ++j)
#pragma unroll
        for (int m = 0; m < MT; ++m) acc[j][m] = v4i{0, 0, 0, 0};
    v4i xf[kAhead];
    auto read_x = [&](const char *buf, int q) {  // operand q = half * MT + token tile
        xf[q % kAhead] = *reinterpret_cast<const v4i *>(buf + (q % MT) * 2048 + x_at(r, q / MT * 4 + kq));
    };
    // What a wave waits for before the barrier that lets others read stage s + 1.
    // Copies: of the XA - 1 steps since, nothing crosses the barriers between, but
    // within a step the compiler may put the weights' loads before or after the
    // copies: only those steps' loads may be left. ODD: every write to LDS, since
    // the barrier by itself waits for none.
    constexpr int kLeft = (XA - 1) * (kCopies + 2 * NW);
    static_assert(kLeft <= 63 && 2 * MT > kAhead, "");
    constexpr int kWait = ODD ? 15 | (3 << 14) | (7 << 4)                                    // lgkmcnt(0)
                              : (kLeft & 15) | ((kLeft >> 4) << 14) | (7 << 4) | (15 << 8);  // vmcnt(kLeft)
    v4i wr[WR][NW][2], xr[XR][kCopies];
    // Stage s, the group's u-th, whose first kAhead operands have been read; the
    // next stage's are read at its end.
    auto step = [&](auto at, int s) {
        constexpr int u = decltype(at)::value;
        const char *cur = buffer(at), *later = buffer(std::integral_constant<int, u + 1>{});
        if constexpr (ODD) fetch_x(min(s + XO, last), xr[(u + XO) % XR]);
        else copy_x(min(s + XA, last), buffer(std::integral_constant<int, u + XA>{}));
        fetch_w(min(s + WR - 1, last), wr[(u + WR - 1) % WR]);
#pragma unroll
        for (int q = 0; q < 2 * MT; ++q) {
            if (q == 2 * MT - kAhead) {
                __builtin_amdgcn_sched_barrier(0);
                __builtin_amdgcn_s_waitcnt(kWait);
                asm volatile("" ::: "memory");  // for the compiler
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int j = 0; j < NW; ++j)
                acc[j][q % MT] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wr[u % WR][j][q / MT], xf[q % kAhead], acc[j][q % MT], 0, 0, 0);
            if (q + kAhead < 2 * MT) read_x(cur, q + kAhead);
            else read_x(later, q + kAhead - 2 * MT);
            // as written: the scheduler would draw the reads together and wait for all of them
            __builtin_amdgcn_sched_group_barrier(0x8, NW, 0);    // MFMA
            __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);   // LDS read
        }
        if constexpr (ODD) put_x(xr[(u + 2) % XR], buffer(std::integral_constant<int, u + 2>{}));
    };
    // A stage of the last ones, all of whose x lies in LDS.
    auto multiply = [&](const char *buf, const v4i (&w)[NW][2]) {
#pragma unroll
        for (int q = 0; q < 2 * MT; ++q) {
            const v4i v = *reinterpret_cast<const v4i *>(buf + (q % MT) * 2048 + x_at(r, q / MT * 4 + kq));
#pragma unroll
            for (int j = 0; j < NW; ++j)
                acc[j][q % MT] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[j][q / MT], v, acc[j][q % MT], 0, 0, 0);
        }
    };
    unrolled(kGroup, [&](auto at) {
        constexpr int u = decltype(at)::value;
        if constexpr (ODD) {
            if constexpr (u < XO) fetch_x(min(u, last), xr[u % XR]);
            if constexpr (u < 2) put_x(xr[u % XR], buffer(at));
        } else if constexpr (u < XA) {
            copy_x(min(u, last), buffer(at));
        }
        if constexpr (u < WR - 1) fetch_w(min(u, last), wr[u]);
    });
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kAhead; ++q) read_x(s_x0, q);
    // Groups of NB stages, then the few that are left (an exit inside the group
    // would cost the sums their registers); for ODD the last stage is always
    // among these.
    int s = 0;
    for (; s + NB + (ODD ? 1 : 0) <= a.k_tiles; s += NB) unrolled(kGroup, [&](auto at) { step(at, s + decltype(at)::value); });
    if (s < a.k_tiles) {
        if constexpr (ODD) {
            __syncthreads();  // the buffers are read until here
            unrolled(kGroup, [&](auto at) {
                if (s + decltype(at)::value < a.k_tiles) bring_x(s + decltype(at)::value, buffer(at));
            });
        } else {  // the group's last buffer but one: what was read of it has been multiplied
            copy_x(min(s + NB - 2, last), buffer(std::integral_constant<int, NB - 2>{}));
        }
        __builtin_amdgcn_s_waitcnt(0x0070);
        __syncthreads();
        if constexpr (NB == 8) {
            unrolled(kGroup, [&](auto at) {
                constexpr int u = decltype(at)::value;
                if (s + u < a.k_tiles) {
                    fetch_w(min(s + u + WR - 1, last), wr[(u + WR - 1) % WR]);
                    multiply(buffer(at), wr[u % WR]);
                }
            });
        } else {
            for (int i = 0; s + i < a.k_tiles; ++i) {
                fetch_w(min(s + i + 1, last), wr[1]);
                multiply(i == 0 ? s_x0 : i == 1 ? s_x1 : i == 2 ? s_x2 : s_x3, wr[0]);
#pragma unroll
                for (int j = 0; j < NW; ++j)
#pragma unroll
                    for (int h = 0; h < 2; ++h) wr[0][j][h] = wr[1][j][h];
            }
        }
    }
    __builtin_amdgcn_s_waitcnt(0x0070);  // copies past the last stage have landed before the LDS is used again
    __syncthreads();
    char *place = wave == 0 ? s_x0 : wave == 1 ? s_x1 : wave == 2 ? s_x2 : s_x3;
    auto write = [&](auto type) {
        if (a.gated) write_sums<MT, NW, decltype(type)::value, true>(a, acc, nt0, t0, lane, place);
        else write_sums<MT, NW, decltype(type)::value, false>(a, acc, nt0, t0, lane, place);
    };
    if (a.out_dtype == MOE_DTYPE_FP32) write(std::integral_constant<int, MOE_DTYPE_FP32>{});
    else if (a.out_dtype == MOE_DTYPE_FP16) write(std::integral_constant<int, MOE_DTYPE_FP16>{});
    else write(std::integral_constant<int, MOE_DTYPE_BF16>{});
}

template <int MT, int NW, int NB = 4, int WR = 2>
hipError_t launch_many(const LinearW8Args &a, hipStream_t s) {
    const int token_blocks = (a.T + MT * 16 - 1) / (MT * 16), rows = kManyWaves * NW;
    const int row_blocks = (a.n_tiles + rows - 1) / rows;
    const dim3 grid(static_cast<unsigned>(row_blocks) * token_blocks), blk(kManyWaves * kWave);
    if (a.K % 16) hipLaunchKernelGGL((linear_w8_many_kernel<MT, NW, NB, WR, true>), grid, blk, 0, s, a, token_blocks, row_blocks);
    else hipLaunchKernelGGL((linear_w8_many_kernel<MT, NW, NB, WR, false>), grid, blk, 0, s, a, token_blocks, row_blocks);
    return hipGetLastError();
}

template <int ROWS, int R>
hipError_t launch_few(const LinearW8Args &a, hipStream_t s) {
    const int token_blocks = (a.T + ROWS - 1) / ROWS, row_blocks = (a.n_tiles + R - 1) / R;
    const dim3 grid((static_cast<unsigned>(row_blocks) * token_blocks + 7) / 8 * 8), blk(kFewWaves * kWave);
    if (a.K % 16) hipLaunchKernelGGL((linear_w8_few_kernel<ROWS, R, true>), grid, blk, 0, s, a, token_blocks);
    else hipLaunchKernelGGL((linear_w8_few_kernel<ROWS, R, false>), grid, blk, 0, s, a, token_blocks);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_pack_w8(const int8_t *codes, const float *scale, int8_t *dst_codes, float *dst_scale,
                          const LinearW8Args &a, hipStream_t s) {
    const int64_t tiles = static_cast<int64_t>(a.n_tiles) * a.k_tiles;  // <= 2^23: the grids below fit
    hipLaunchKernelGGL(pack_codes8_kernel, dim3(static_cast<unsigned>((tiles * 128 + 255) / 256)), dim3(256), 0, s, codes,
                       dst_codes, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(pack_scales8_kernel, dim3(static_cast<unsigned>((a.n_tiles * 16 + 255) / 256)), dim3(256), 0, s,
                       scale, dst_scale, a);
    return hipGetLastError();
}

// Which kernel: the few-token one splits K over a workgroup's waves, so it fills
// the chip where there are few tiles of outputs, but it reads x for every 16 R
// weight rows and joins eight sums; it wants one workgroup for each CU, of the
// least x and weights (16 R rows, ROWS tokens). The other wants two large
// workgroups a CU, or more small ones; with a short K, small ones, whose ends
// overlap others' products; with less than two a CU, eight stages under way
// instead of four. In us (bf16 out; few tokens / many, * taken):
//   T 64, N 4096, K 4096: 32 x 2 *6.5, 64 x 4 10.7 / 10.0   T 128, N 8192: 64 x 4 *11.7 / 12.0
//   T 37, N 5006, K 4256, gated: 16 x 4 *6.9, 64 x 4 10.5 / 11.2    T 512, N 4096: 19.9 / 64 x 8 *15.1
//   T 1000, N 1000, K 1000: 7.8 / 32 x 4 *5.5              T 64, N 28672: 33.3 / 64 x 8 *28.1
// many, tokens x row tiles 128 x 16, 128 x 8, 64 x 8, 64 x 4, 32 x 4, K 4096 (eight stages in brackets: 64 x 8, 32 x 4):
//   T 4096, N 8192 *111 128 148 193 249 (161 257)   T 2048, N 4096 33.4 *33.2 39 49 64 (42 67)
//   T 512, N 8192 31.8 25.1 *21.3 25.0 33.2 (22.1 35.0)   T 256, N 8192 31.0 24.1 18.8 19.2 17.6 (*15.2 19.7)
//   K 700, T 2500, N 5000: 20.8 25.5 *21.5 30.1 30.8 (30.7 37.9)   K 8429, T 636, N 2332: 73 50 34 38 36 (*29.6 36)
hipError_t launch_linear_w8(const LinearW8Args &a, hipStream_t s) {
    auto blocks = [&](int tokens, int tiles) {
        return static_cast<int64_t>((a.T + tokens - 1) / tokens) * ((a.n_tiles + tiles - 1) / tiles);
    };
    if (a.T <= 8) return launch_few<8, 1>(a, s);
    if (a.T <= 16) return a.n_tiles < 512 ? launch_few<16, 1>(a, s) : launch_few<16, 2>(a, s);
    if (blocks(64, 4) <= 256 && (a.T <= 64 || a.k_tiles >= 16)) {
        if (blocks(16, 1) <= 256) return launch_few<16, 1>(a, s);
        if (blocks(16, 2) <= 256) return launch_few<16, 2>(a, s);
        if (blocks(32, 2) <= 256) return launch_few<32, 2>(a, s);
        if (blocks(16, 4) <= 256) return launch_few<16, 4>(a, s);
        if (blocks(32, 4) <= 256) return launch_few<32, 4>(a, s);
        return launch_few<64, 4>(a, s);
    }
    // more than 16 tokens from here: x has the 16 bytes that the kernel for many takes for granted
    if (a.k_tiles >= 16 && blocks(128, 16) >= 512) return launch_many<8, 4>(a, s);
    if (a.k_tiles >= 16 && blocks(128, 8) >= 400) return launch_many<8, 2>(a, s);
    if (blocks(64, 8) >= 384) return launch_many<4, 2>(a, s);
    if (a.k_tiles >= 16) return blocks(64, 8) >= 160 ? launch_many<4, 2, 8, 4>(a, s) : launch_many<2, 1, 8, 4>(a, s);
    return blocks(64, 4) >= 384 ? launch_many<4, 1>(a, s) : launch_many<2, 1>(a, s);
}

}  // namespace moe
