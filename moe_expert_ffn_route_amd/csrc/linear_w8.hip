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
    int8_t v[16];
#pragma unroll
    for (int b = 0; b < 16; ++b) v[b] = ok && k0 + b < a.K ? src[row * a.K + k0 + b] : static_cast<int8_t>(0);
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
// Rows whose length is no multiple of 16 begin anywhere, and the last 16 bytes
// of the last ones may end behind x. The load is moved back to x's last 16
// bytes then, and its bytes back to their places where they are used.
struct OddX {
    int64_t total;  // T * K
    __device__ __forceinline__ int64_t from(int64_t off) const {
        const int64_t last = total - 16;
        return off < last ? off : last < 0 ? 0 : last;
    }
    __device__ __forceinline__ v4i load(const int8_t *x, int64_t off) const {
        if (total >= 16) return load16(x + from(off));
        int8_t b[16] = {};
        for (int i = 0; i < static_cast<int>(total); ++i) b[i] = x[i];
        v4i v;
        __builtin_memcpy(&v, b, 16);
        return v;
    }
    __device__ __forceinline__ v4i place(v4i v, int64_t off) const {
        const int64_t by = off - from(off);  // 0 but behind the end
        if (by == 0) return v;
        uint64_t q[2];
        __builtin_memcpy(q, &v, 16);
        const int s = static_cast<int>(by < 15 ? by : 15) * 8;
        const unsigned __int128 w = ((static_cast<unsigned __int128>(q[1]) << 64) | q[0]) >> s;
        q[0] = static_cast<uint64_t>(w);
        q[1] = static_cast<uint64_t>(w >> 64);
        __builtin_memcpy(&v, q, 16);
        return v;
    }
};

__device__ __forceinline__ uint16_t bits16(float v, bool fp16) {
    return fp16 ? __builtin_bit_cast(uint16_t, static_cast<_Float16>(v)) : f32_to_bf16(v);
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

// Few tokens: a workgroup takes 16 weight rows, its WAVES waves every WAVES-th
// tile of 128 k, loaded DEPTH tiles ahead; the waves' sums meet in LDS.
//
// Whole rows of x are loaded and turned to operands in LDS, in a place of the
// wave's own. Nothing is masked: tokens past the end read the last token's x
// (columns that are not stored), k past the end meets zero weights.
template <int ROWS, bool ODD>
__global__ __launch_bounds__(8 * kWave) void linear_w8_few_kernel(LinearW8Args a) {
    constexpr int WAVES = 8, DEPTH = 2;
    constexpr int MT = (ROWS + 15) / 16;
    constexpr int kL = (ROWS + 7) / 8;  // loads of x per tile: 8 rows each
    constexpr int kStage = WAVES * MT * 2048, kRed = WAVES * MT * kWave * 16;
    __shared__ __attribute__((aligned(16))) char lds[kStage > kRed ? kStage : kRed];
    const int lane = threadIdx.x & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int r = lane & 15, kq = lane >> 4;
    const int nt = blockIdx.x, t0 = blockIdx.y * ROWS;
    char *place = lds + wave * MT * 2048;
    const OddX odd{static_cast<int64_t>(a.T) * a.K};
    const int count = (a.k_tiles - wave + WAVES - 1) / WAVES;  // the wave's tiles; <= 0: none
    struct Tile {
        v4i codes[2];
        v4i x[kL];
    };
    auto offset = [&](int i, int j) -> int64_t {  // of the lane's j-th load of its i-th tile
        const int kt = wave + min(i, count - 1) * WAVES;
        const int t = min(t0 + j * 8 + lane / 8, a.T - 1);
        int k = kt * kTileK + lane % 8 * 16;
        k = ODD ? min(k, a.K - 1) : min(k, a.K - 16);
        return static_cast<int64_t>(t) * a.K + k;
    };
    auto fetch = [&](int i, Tile &f) {
        const int kt = wave + min(i, count - 1) * WAVES;
        const int8_t *w = a.codes + (static_cast<size_t>(nt) * a.k_tiles + kt) * kTileBytes + lane * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h) f.codes[h] = load16(w + h * 1024);
#pragma unroll
        for (int j = 0; j < kL; ++j) f.x[j] = ODD ? odd.load(a.x, offset(i, j)) : load16(a.x + offset(i, j));
    };
    v4i acc[MT];
#pragma unroll
    for (int m = 0; m < MT; ++m) acc[m] = v4i{0, 0, 0, 0};
    typedef __attribute__((address_space(3))) volatile v4i own_lds;  // one wave's own: in order without a barrier
    auto multiply = [&](int i, const Tile &f) {
#pragma unroll
        for (int j = 0; j < kL; ++j) {
            const int row = j * 8 + lane / 8;
            *(own_lds *)(place + row / 16 * 2048 + x_at(row % 16, lane % 8)) = ODD ? odd.place(f.x[j], offset(i, j)) : f.x[j];
        }
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4i xf = *(own_lds *)(place + m * 2048 + x_at(r, h * 4 + kq));
                acc[m] = __builtin_amdgcn_mfma_i32_16x16x64_i8(f.codes[h], xf, acc[m], 0, 0, 0);
            }
    };
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
    v4i(*red)[MT][kWave] = reinterpret_cast<v4i(*)[MT][kWave]>(lds);
    __syncthreads();  // the places are read until here
#pragma unroll
    for (int m = 0; m < MT; ++m) red[wave][m][lane] = acc[m];
    __syncthreads();
    if (wave >= MT) return;
    v4i sum = red[0][wave][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) sum += red[w][wave][lane];
    const int t = t0 + wave * 16 + r;
    if (t < a.T) finish(a, nt, kq, t, sum);
}

template <int ROWS>
hipError_t launch_few(const LinearW8Args &a, hipStream_t s) {
    const dim3 grid(a.n_tiles, (a.T + ROWS - 1) / ROWS), blk(8 * kWave);
    if (a.K % 16) hipLaunchKernelGGL((linear_w8_few_kernel<ROWS, true>), grid, blk, 0, s, a);
    else hipLaunchKernelGGL((linear_w8_few_kernel<ROWS, false>), grid, blk, 0, s, a);
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

hipError_t launch_linear_w8(const LinearW8Args &a, hipStream_t s) {
    if (a.T <= 8) return launch_few<8>(a, s);
    if (a.T <= 16) return launch_few<16>(a, s);
    return launch_few<64>(a, s);
}

}  // namespace moe
