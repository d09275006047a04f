// Tokens sorted by expert, back again with their weights, and the gradient.
//
// Dispatch is a stable counting sort of the pairs (t, k) by expert:
//   row(p) = first(e) + #{pairs q < p of expert e},
//   first(e) = sum over e' < e of the counts rounded up to row_align
// and a copy of x's rows. Batches of up to kSmallPairs pairs take one launch,
// whose workgroups (one per token) each count all ids; larger ones count by
// blocks of pairs, scan, and place, and copy in a launch of its own. Counts are
// integers: the order of the LDS atomics does not reach a result.
//
// Combine sums a token's rows in fp32, k ascending, one rounding per product
// and sum. The gradient reads a token's dout once for its K rows.
//
// All of it is bounded by memory: rows in, rows out.
#include "rowwise.h"

#include "../../include/moe_w8a8.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kSmallPairs = 2048;
constexpr int kBlockPairs = 1024;  // pairs per block of the counting pass

// The pair's expert, -1 if it is dropped.
__device__ __forceinline__ int expert_of(const DispatchArgs &a, int p) {
    const int e = a.ids[p];
    const bool kept = static_cast<unsigned>(e) < static_cast<unsigned>(a.E) && (!a.mask || a.mask[p / a.K]);
    return kept ? e : -1;
}
__device__ __forceinline__ int round_up(int n, int align) { return (n + align - 1) & -align; }

// s_first[e] = exclusive sum of s_count rounded up to align, e in [0, E].
// Whole workgroup of NT threads, 1024 / NT experts each; s_wave: NT / kWave
// words. Ends in a barrier.
template <int NT>
__device__ __forceinline__ void scan_counts(const int *s_count, int *s_first, int *s_wave, int E, int align) {
    constexpr int kPer = 1024 / NT;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    int n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        n[i] = e < E ? round_up(s_count[e], align) : 0;
        sum += n[i];
    }
    int incl = sum;
#pragma unroll
    for (int d = 1; d < kWave; d <<= 1) {
        const int up = __shfl_up(incl, d, kWave);
        if (lane >= d) incl += up;
    }
    if (lane == kWave - 1) s_wave[wave] = incl;
    __syncthreads();
    int at = incl - sum;
    for (int w = 0; w < wave; ++w) at += s_wave[w];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int e = tid * kPer + i;
        if (e <= E) s_first[e] = at;
        at += n[i];
    }
    if (tid == NT - 1 && E == 1024) s_first[E] = at;
    __syncthreads();
}

// Bytes of a row, 16 at a time from its start wherever that is, and the bytes
// after them one by one. By `n` threads, of which this is number i.
__device__ __forceinline__ void copy_row(uint8_t *dst, const uint8_t *src, size_t bytes, int i, int n) {
    const int chunks = static_cast<int>(bytes / 16), rest = static_cast<int>(bytes % 16);
    for (int c = i; c < chunks; c += n) __builtin_memcpy(dst + c * 16, src + c * 16, 16);
    if (i < rest) dst[chunks * 16 + i] = src[chunks * 16 + i];
}
__device__ __forceinline__ void zero_row(uint8_t *dst, size_t bytes, int i, int n) {
    const int chunks = static_cast<int>(bytes / 16), rest = static_cast<int>(bytes % 16);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int c = i; c < chunks; c += n) __builtin_memcpy(dst + c * 16, &zero, 16);
    if (i < rest) dst[chunks * 16 + i] = 0;
}
// Rows [from, to) that fill an expert's last row_align.
__device__ __forceinline__ void fill_rows(const DispatchArgs &a, int from, int to) {
    const size_t bytes = static_cast<size_t>(a.H) * a.elem;
    for (int r = from; r < to; ++r) {
        if (!a.rows) break;
        zero_row(static_cast<uint8_t *>(a.rows) + r * bytes, bytes, threadIdx.x, blockDim.x);
        for (int g = threadIdx.x; g < a.groups; g += blockDim.x) a.row_scale[static_cast<size_t>(r) * a.groups + g] = 0.0f;
    }
}
// x's row t and its scales to `row`.
__device__ __forceinline__ void move_row(const DispatchArgs &a, int t, int row) {
    const size_t bytes = static_cast<size_t>(a.H) * a.elem;
    copy_row(static_cast<uint8_t *>(a.rows) + row * bytes, static_cast<const uint8_t *>(a.x) + t * bytes, bytes,
             threadIdx.x, blockDim.x);
    for (int g = threadIdx.x; g < a.groups; g += blockDim.x)
        a.row_scale[static_cast<size_t>(row) * a.groups + g] = a.x_scale[static_cast<size_t>(t) * a.groups + g];
}

// No token: nothing but the counts.
__global__ __launch_bounds__(kThreads) void dispatch_none_kernel(DispatchArgs a) {
    for (int e = threadIdx.x; e <= a.E; e += kThreads) {
        if (e < a.E) a.counts[e] = 0;
        a.offset[e] = 0;
    }
}

// One workgroup per token, each of which counts every pair.
__global__ __launch_bounds__(kThreads) void dispatch_small_kernel(DispatchArgs a) {
    __shared__ int s_count[1024], s_first[1025], s_wave[kThreads / kWave], s_mine[kMaxTopK], s_rank[kMaxTopK];
    const int t = blockIdx.x, tid = threadIdx.x, P = a.T * a.K;
    for (int e = tid; e < a.E; e += kThreads) s_count[e] = 0;
    if (tid < a.K) {
        s_mine[tid] = expert_of(a, t * a.K + tid);
        s_rank[tid] = 0;
    }
    __syncthreads();
    for (int p = tid; p < P; p += kThreads) {
        const int e = expert_of(a, p);
        if (e < 0) continue;
        atomicAdd(&s_count[e], 1);
        for (int k = 0; k < a.K; ++k)
            if (s_mine[k] == e && p < t * a.K + k) atomicAdd(&s_rank[k], 1);
    }
    __syncthreads();
    scan_counts<kThreads>(s_count, s_first, s_wave, a.E, a.align);
    if (tid < a.K) {
        const int e = s_mine[tid], p = t * a.K + tid, row = e < 0 ? -1 : s_first[e] + s_rank[tid];
        a.row_of_pair[p] = row;
        if (row >= 0) a.pair_of_row[row] = p;
    }
    if (t == 0)
        for (int e = tid; e <= a.E; e += kThreads) {
            if (e < a.E) a.counts[e] = s_count[e];
            a.offset[e] = s_first[e];
        }
    for (int64_t r = s_first[a.E] + t * kThreads + tid; r < a.R; r += static_cast<int64_t>(a.T) * kThreads)
        a.pair_of_row[r] = -1;
    if (a.align > 1)
        for (int e = t; e < a.E; e += a.T) {
            const int from = s_first[e] + s_count[e], to = s_first[e + 1];
            for (int r = from + tid; r < to; r += kThreads) a.pair_of_row[r] = -1;
            fill_rows(a, from, to);
        }
    if (a.rows)
        for (int k = 0; k < a.K; ++k)
            if (s_mine[k] >= 0) move_row(a, t, s_first[s_mine[k]] + s_rank[k]);
}

// ws[b][e] = pairs of expert e in block b of kBlockPairs pairs
__global__ __launch_bounds__(kThreads) void dispatch_count_kernel(DispatchArgs a) {
    __shared__ int s_count[1024];
    const int P = a.T * a.K;
    for (int e = threadIdx.x; e < a.E; e += kThreads) s_count[e] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < kBlockPairs; i += kThreads) {
        const int p = blockIdx.x * kBlockPairs + i;
        const int e = p < P ? expert_of(a, p) : -1;
        if (e >= 0) atomicAdd(&s_count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < a.E; e += kThreads) a.workspace[static_cast<size_t>(blockIdx.x) * a.E + e] = s_count[e];
}
// ws[b][e] = pairs of e in the blocks before b, and counts[e] = all of them
__global__ __launch_bounds__(kWave) void dispatch_scan_kernel(DispatchArgs a, int blocks) {
    const int e = blockIdx.x * kWave + threadIdx.x;
    if (e >= a.E) return;
    int sum = 0;
    for (int b = 0; b < blocks; ++b) {
        int *at = a.workspace + static_cast<size_t>(b) * a.E + e;
        const int n = *at;
        *at = sum;
        sum += n;
    }
    a.counts[e] = sum;
}
// The maps. One thread per pair of the block.
__global__ __launch_bounds__(kBlockPairs) void dispatch_place_kernel(DispatchArgs a) {
    constexpr int kWaves = kBlockPairs / kWave;
    __shared__ int s_count[1024], s_first[1025], s_wave[kWaves];
    __shared__ uint16_t s_here[kWaves][1024];  // pairs of an expert in each wave
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave, P = a.T * a.K;
    const int p = blockIdx.x * kBlockPairs + tid;
    for (int e = tid; e < a.E; e += kBlockPairs) s_count[e] = a.counts[e];
    for (int i = tid; i < kWaves * a.E; i += kBlockPairs) s_here[i / a.E][i % a.E] = 0;
    const int e = p < P ? expert_of(a, p) : -1;
    __syncthreads();
    scan_counts<kBlockPairs>(s_count, s_first, s_wave, a.E, a.align);
    uint64_t same = __ballot(e >= 0);  // the wave's lanes with this expert
    for (int bit = 1; bit < a.E; bit <<= 1) {
        const uint64_t set = __ballot(e >= 0 && (e & bit));
        same &= (e & bit) ? set : ~set;
    }
    const uint64_t before = same & ((1ull << lane) - 1);
    if (e >= 0 && before == 0) s_here[wave][e] = static_cast<uint16_t>(__popcll(same));
    __syncthreads();
    if (p < P) {
        int row = -1;
        if (e >= 0) {
            row = s_first[e] + a.workspace[static_cast<size_t>(blockIdx.x) * a.E + e] + __popcll(before);
            for (int w = 0; w < wave; ++w) row += s_here[w][e];
            a.pair_of_row[row] = p;
        }
        a.row_of_pair[p] = row;
    }
    if (blockIdx.x == 0)
        for (int i = tid; i <= a.E; i += kBlockPairs) a.offset[i] = s_first[i];
    for (int64_t r = s_first[a.E] + static_cast<int64_t>(blockIdx.x) * kBlockPairs + tid; r < a.R;
         r += static_cast<int64_t>(gridDim.x) * kBlockPairs)
        a.pair_of_row[r] = -1;
    if (a.align > 1)
        for (int i = blockIdx.x * kWaves + wave; i < a.E; i += gridDim.x * kWaves)
            for (int r = s_first[i] + s_count[i] + lane; r < s_first[i + 1]; r += kWave) a.pair_of_row[r] = -1;
}
// Workgroups [0, T): the rows of a token; the others: the rows that fill an
// expert's last row_align.
__global__ __launch_bounds__(kThreads) void dispatch_move_kernel(DispatchArgs a) {
    const int b = blockIdx.x;
    if (b >= a.T) {
        const int e = b - a.T;
        fill_rows(a, a.offset[e] + a.counts[e], a.offset[e + 1]);
        return;
    }
    for (int k = 0; k < a.K; ++k) {
        const int row = a.row_of_pair[b * a.K + k];
        if (row >= 0) move_row(a, b, row);
    }
}

// ------------------------------------------------------------------ back

// Thread c of a token's takes elements [8 c, 8 c + 8), or, behind the row's
// whole chunks, one element each.
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void combine_rows_kernel(RowsArgs a) {
    constexpr int kAhead = 8;  // rows on their way at once
    const int t = blockIdx.x, c = blockIdx.y * kThreads + threadIdx.x;
    const int chunks = a.H / kVec, rest = a.H % kVec;
    if (c >= chunks + rest) return;
    const T *rows = static_cast<const T *>(a.rows);
    const size_t out_at = static_cast<size_t>(t) * a.H;
    const O *addend = static_cast<const O *>(a.addend) + out_at;
    O *out = static_cast<O *>(a.out) + out_at;
    auto sum = [&](auto load, auto &acc) {
        for (int k0 = 0; k0 < a.K && a.R > 0; k0 += kAhead) {
            decltype(load(rows)) v[kAhead];
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {  // dropped pairs, and k past the end: some row, not counted
                const int r = a.row_of_pair[t * a.K + min(k0 + j, a.K - 1)];
                v[j] = load(rows + static_cast<size_t>(static_cast<unsigned>(r) < static_cast<unsigned>(a.R) ? r : 0) * a.H);
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                if (k0 + j >= a.K) break;
                const int r = a.row_of_pair[t * a.K + k0 + j];
                if (static_cast<unsigned>(r) >= static_cast<unsigned>(a.R)) continue;
                acc(v[j], a.scales ? a.scales[t * a.K + k0 + j] : 1.0f);
            }
        }
    };
    struct Eight { T v[kVec]; };
    if (c < chunks) {
        float acc[kVec] = {}, add[kVec];
        if (a.addend) load8(addend + c * kVec, add);
        auto load = [&](const T *row) {
            Eight e;
            __builtin_memcpy(&e, row + c * kVec, sizeof e);
            return e;
        };
        auto take = [&](const Eight &e, float w) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) acc[i] = acc[i] + (a.scales ? to_f32(e.v[i]) * w : to_f32(e.v[i]));
        };
        sum(load, take);
        if (a.addend) {
#pragma unroll
            for (int i = 0; i < kVec; ++i) acc[i] = acc[i] + add[i];
        }
        store8(out + c * kVec, acc);
    } else {
        const int i = chunks * kVec + c - chunks;
        float acc = 0.0f;
        auto load = [&](const T *row) { return row[i]; };
        auto take = [&](T e, float w) { acc = acc + (a.scales ? to_f32(e) * w : to_f32(e)); };
        sum(load, take);
        if (a.addend) acc = acc + to_f32(addend[i]);
        from_f32(acc, out[i]);
    }
}

// The row that pair p has by both maps, or -1.
__device__ __forceinline__ int own_row(const RowsArgs &a, int p) {
    const int r = a.row_of_pair[p];
    return static_cast<unsigned>(r) < static_cast<unsigned>(a.R) && a.pair_of_row[r] == p ? r : -1;
}

// A product rounded to fp32. Without the barrier the compiler makes it and its
// conversion to fp16 one instruction, of one rounding, in some places only.
__device__ __forceinline__ float product(float d, float w) {
    float p = d * w;
    asm("" : "+v"(p));
    return p;
}

// Workgroups [0, T): a token's K rows. The others: rows without a pair.
template <typename T, typename O>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(RowsArgs a) {
    constexpr int kWaves = kThreads / kWave;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int chunks = a.H / kVec, rest = a.H % kVec;
    if (static_cast<int>(blockIdx.x) >= a.T) {
        const size_t bytes = static_cast<size_t>(a.H) * sizeof(T);
        const int waves = (gridDim.x - a.T) * kWaves, first = (blockIdx.x - a.T) * kWaves + wave;
        for (int64_t r0 = static_cast<int64_t>(first) * kWave; r0 < a.R; r0 += static_cast<int64_t>(waves) * kWave) {
            const int r = static_cast<int>(r0) + lane;
            bool none = false;
            if (r < a.R) {
                const int p = a.pair_of_row[r];
                none = static_cast<unsigned>(p) >= static_cast<unsigned>(a.T * a.K) || a.row_of_pair[p] != r;
            }
            for (uint64_t left = __ballot(none); left; left &= left - 1)
                zero_row(static_cast<uint8_t *>(a.drows) + (r0 + __builtin_ctzll(left)) * bytes, bytes, lane, kWave);
        }
        return;
    }
    __shared__ float s_dot[kWaves][kMaxTopK];
    const int t = blockIdx.x;
    const O *dout = static_cast<const O *>(a.dout) + static_cast<size_t>(t) * a.H;
    const T *rows = static_cast<const T *>(a.rows);
    T *drows = static_cast<T *>(a.drows);
    for (int k = 0; k < a.K; ++k) {
        const int r = own_row(a, t * a.K + k);
        float dot = 0.0f;
        if (r >= 0) {
            const size_t at = static_cast<size_t>(r) * a.H;
            const float w = a.scales ? a.scales[t * a.K + k] : 1.0f;
            for (int c = tid; c < chunks; c += kThreads) {
                float d[kVec], v[kVec];
                load8(dout + c * kVec, d);
                if (a.dscales) {
                    load8(rows + at + c * kVec, v);
#pragma unroll
                    for (int i = 0; i < kVec; ++i) dot += v[i] * d[i];
                }
                if (a.drows) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) d[i] = product(d[i], w);
                    store8(drows + at + c * kVec, d);
                }
            }
            if (tid < rest) {
                const int i = chunks * kVec + tid;
                const float d = to_f32(dout[i]);
                if (a.dscales) dot += to_f32(rows[at + i]) * d;
                if (a.drows) from_f32(product(d, w), drows[at + i]);
            }
        }
        dot = last_lane_sum(dot);
        if (lane == kWave - 1) s_dot[wave][k] = dot;
    }
    __syncthreads();
    if (a.dscales && tid < a.K) {
        float dot = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) dot += s_dot[w][tid];
        a.dscales[t * a.K + tid] = dot;
    }
}

template <typename T, typename O>
hipError_t combine_of(const RowsArgs &a, hipStream_t s) {
    const int items = a.H / kVec + a.H % kVec;
    hipLaunchKernelGGL((combine_rows_kernel<T, O>), dim3(a.T, (items + kThreads - 1) / kThreads), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}
template <typename T, typename O>
hipError_t grad_of(const RowsArgs &a, hipStream_t s) {
    const int others = a.drows ? (a.R + kThreads - 1) / kThreads : 0;
    hipLaunchKernelGGL((combine_grad_kernel<T, O>), dim3(a.T + (others < 2048 ? others : 2048)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t dispatch_workspace(int T, int K, int E) {
    const int64_t P = static_cast<int64_t>(T) * K;
    return P <= kSmallPairs ? 0 : static_cast<size_t>((P + kBlockPairs - 1) / kBlockPairs) * E * sizeof(int32_t);
}

hipError_t launch_dispatch(const DispatchArgs &a, hipStream_t s) {
    if (a.T == 0) {
        hipLaunchKernelGGL(dispatch_none_kernel, dim3(1), dim3(kThreads), 0, s, a);
        return hipGetLastError();
    }
    const int P = a.T * a.K;
    if (P <= kSmallPairs) {
        hipLaunchKernelGGL(dispatch_small_kernel, dim3(a.T), dim3(kThreads), 0, s, a);
        return hipGetLastError();
    }
    const int blocks = (P + kBlockPairs - 1) / kBlockPairs;
    hipLaunchKernelGGL(dispatch_count_kernel, dim3(blocks), dim3(kThreads), 0, s, a);
    hipLaunchKernelGGL(dispatch_scan_kernel, dim3((a.E + kWave - 1) / kWave), dim3(kWave), 0, s, a, blocks);
    hipLaunchKernelGGL(dispatch_place_kernel, dim3(blocks), dim3(kBlockPairs), 0, s, a);
    if (a.rows)
        hipLaunchKernelGGL(dispatch_move_kernel, dim3(a.T + (a.align > 1 ? a.E : 0)), dim3(kThreads), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_combine_rows(const RowsArgs &a, hipStream_t s) {
    const bool wide = a.out_dtype == MOE_DTYPE_FP32;
    switch (a.dtype) {
        case MOE_DTYPE_BF16: return wide ? combine_of<Bf16, float>(a, s) : combine_of<Bf16, Bf16>(a, s);
        case MOE_DTYPE_FP16: return wide ? combine_of<Fp16, float>(a, s) : combine_of<Fp16, Fp16>(a, s);
        default: return combine_of<float, float>(a, s);
    }
}

hipError_t launch_combine_grad(const RowsArgs &a, hipStream_t s) {
    const bool wide = a.out_dtype == MOE_DTYPE_FP32;
    switch (a.dtype) {
        case MOE_DTYPE_BF16: return wide ? grad_of<Bf16, float>(a, s) : grad_of<Bf16, Bf16>(a, s);
        case MOE_DTYPE_FP16: return wide ? grad_of<Fp16, float>(a, s) : grad_of<Fp16, Fp16>(a, s);
        default: return grad_of<float, float>(a, s);
    }
}

}  // namespace moe
