// Tokens sorted by expert, back again with their weights, and the gradient.
//
// Dispatch is a stable counting sort of the pairs (t, k) by expert:
//   row(p) = first(e) + #{pairs q < p of expert e},
//   first(e) = sum over e' < e of the counts rounded up to row_align
// and a copy of x's rows: x's bytes read once, K times as many written, which
// is what bounds large batches. For small ones it is latency: batches of up to
// 64 pairs (a decode step) hold all ids in the lanes of every wave and need
// no LDS and no barrier; up to kSmallPairs one launch still does it, every
// workgroup counting all pairs. More pairs are counted by blocks in a launch
// of its own, and each workgroup of the second places and moves the rows of
// its few tokens from the blocks' counts. Counts are integers: the order of
// the LDS atomics does not reach a result.
//
// Combine sums a token's rows in fp32, k ascending, one rounding per product
// and sum. The gradient reads a token's dout once for its K rows.
//
// In us, with the rate of what has to be read and written (a copy: 4.9 TB/s):
// dispatch T 4096, E 256, K 8, H 4096, bf16, row_align 16 54 (4.7), T 8 4.8,
// a launch; combine T 2047, K 6, H 5003, bf16 to fp32 28.2 (5.0), T 8 4.1; the
// gradient T 4096, K 8, H 4096 118 (4.9).
//
// Both ways rows are moved by 16 bytes from their first element, whatever its
// address (the hardware takes such accesses).
#include "rowwise.h"

#include <type_traits>

#include "../../include/moe_w8a8.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / kWave;
// One launch up to here. In us, one / two (int8, H 4096, E 256; E 8 in brackets):
//   512 pairs: K 8 6.7 / 13.4 (6.6 / 13.1), K 2 4.8 / 15.4 (4.9 / 15.2), K 1 4.7 / 18.1 (5.1 / 17.9)
//   2048: K 8 9.1 / 14.6 (9.1 / 14.4), K 2 8.9 / 19.2 (11.5 / 18.9), K 1 11.6 / 21.8 (19.0 / 21.9)
//   4096: K 8 10.5 / 14.3 (10.8 / 14.1), K 2 14.2 / 18.7 (23.7 / 18.8), K 1 25.2 / 23.9 (52.4 / 23.9)
// Each of T workgroups counts all pairs, so with K 1 and few experts, whose LDS
// counters are few too, the last row's border is too far.
constexpr int kSmallPairs = 4096;
constexpr int kParts = 16;        // workgroups of the second launch per block of the first
constexpr int kScanBlocks = 64;   // more blocks are summed in a launch of their own

// The pair's expert, -1 if it is dropped.
__device__ __forceinline__ int expert_of(const DispatchArgs &a, int p) {
    const int e = a.ids[p];
    const bool kept = static_cast<unsigned>(e) < static_cast<unsigned>(a.E) && (!a.mask || a.mask[p / a.K]);
    return kept ? e : -1;
}
__device__ __forceinline__ int round_up(int n, int align) { return (n + align - 1) & -align; }

// The wave's lanes whose expert is the lane's; of no use where e < 0.
__device__ __forceinline__ uint64_t same_expert(int e, int E) {
    uint64_t same = __ballot(e >= 0);
    for (int bit = 1; bit < E; bit <<= 1) {
        const uint64_t set = __ballot(e >= 0 && (e & bit));
        same &= (e & bit) ? set : ~set;
    }
    return same;
}

// s_first[e] = exclusive sum of s_count rounded up to align, e in [0, E], by a
// whole workgroup; s_wave: kWaves words. Ends in a barrier.
__device__ __forceinline__ void scan_counts(const int *s_count, int *s_first, int *s_wave, int E, int align) {
    constexpr int kPer = 1024 / kThreads;
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
    if (tid == kThreads - 1 && E == 1024) s_first[E] = at;
    __syncthreads();
}

__device__ __forceinline__ uint4 load16(const uint8_t *p) {
    uint4 v;
    __builtin_memcpy(&v, p, 16);
    return v;
}
__device__ __forceinline__ void zero_row(uint8_t *dst, size_t bytes, int i, int n, bool streamed) {
    const int chunks = static_cast<int>(bytes / 16), rest = static_cast<int>(bytes % 16);
    const uint4 zero = make_uint4(0, 0, 0, 0);
    for (int c = i; c < chunks; c += n) store_out(dst + c * 16, zero, streamed);
    if (i < rest) dst[chunks * 16 + i] = 0;
}
// Row r fills an expert's last row_align: by n threads, of which this is number i.
__device__ __forceinline__ void fill_row(const DispatchArgs &a, int r, int i, int n) {
    if (i == 0) a.pair_of_row[r] = -1;
    if (!a.rows) return;
    const size_t bytes = static_cast<size_t>(a.H) * a.elem;
    zero_row(static_cast<uint8_t *>(a.rows) + r * bytes, bytes, i, n, a.streamed);
    for (int g = i; g < a.groups; g += n) a.row_scale[static_cast<size_t>(r) * a.groups + g] = 0.0f;
}
// The rows that fill the experts' last row_align, by workgroup f of F: where
// there are more workgroups than experts, several an expert.
__device__ __forceinline__ void fill_share(const DispatchArgs &a, const int *s_count, const int *s_first, int f, int F) {
    const int each = F > a.E ? F / a.E : 1, experts = F / each, wave = threadIdx.x / kWave;
    if (f >= experts * each) return;
    for (int e = f / each; e < a.E; e += experts)
        for (int r = s_first[e] + s_count[e] + f % each * kWaves + wave; r < s_first[e + 1]; r += each * kWaves)
            fill_row(a, r, threadIdx.x & (kWave - 1), kWave);
}
// x's row t and its scales to the rows row(k) >= 0, k < K: 16 bytes at a time,
// kAhead loads before the first store, and the bytes after them one by one.
constexpr int kAhead = 4;
struct Ahead { uint4 v[kAhead]; };
// The token's chunks c0, c0 + n, ...; none of a row without a whole chunk.
__device__ __forceinline__ Ahead load_token(const DispatchArgs &a, int t, int c0, int n) {
    const size_t bytes = static_cast<size_t>(a.H) * a.elem;
    const int chunks = static_cast<int>(bytes / 16);
    const uint8_t *x = static_cast<const uint8_t *>(a.x) + t * bytes;
    Ahead f = {};
    if (chunks > 0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) f.v[j] = load16(x + min(c0 + j * n, chunks - 1) * 16);
    }
    return f;
}
template <typename Row>
__device__ __forceinline__ void move_token(const DispatchArgs &a, int t, Ahead f, Row row, int i, int n) {
    const size_t bytes = static_cast<size_t>(a.H) * a.elem;
    const int chunks = static_cast<int>(bytes / 16), rest = static_cast<int>(bytes % 16);
    const uint8_t *x = static_cast<const uint8_t *>(a.x) + t * bytes;
    uint8_t *rows = static_cast<uint8_t *>(a.rows);
    for (int c0 = i; c0 < chunks; c0 += kAhead * n) {
        if (c0 != i) f = load_token(a, t, c0, n);
        for (int k = 0; k < a.K; ++k) {
            const int r = row(k);
            if (r < 0) continue;
#pragma unroll
            for (int j = 0; j < kAhead; ++j)
                if (c0 + j * n < chunks) store_out(rows + r * bytes + (c0 + j * n) * 16, f.v[j], a.streamed);
        }
    }
    const uint8_t tail = i < rest ? x[chunks * 16 + i] : 0;
    for (int k = 0; k < a.K; ++k) {
        const int r = row(k);
        if (r < 0) continue;
        if (i < rest) rows[r * bytes + chunks * 16 + i] = tail;
        for (int g = i; g < a.groups; g += n)
            a.row_scale[static_cast<size_t>(r) * a.groups + g] = a.x_scale[static_cast<size_t>(t) * a.groups + g];
    }
}

// No token: nothing but the counts.
__global__ __launch_bounds__(kThreads) void dispatch_none_kernel(DispatchArgs a) {
    for (int e = threadIdx.x; e <= a.E; e += kThreads) {
        if (e < a.E) a.counts[e] = 0;
        a.offset[e] = 0;
    }
}

// Up to 64 pairs: lane p of every wave holds pair p's expert. Workgroups [0,
// T): a token's rows. The next `count_blocks`: the counts and offsets of kThreads
// experts each, and what pair_of_row holds behind the last row. The others:
// the rows that fill an expert's last row_align. In loops where it can be: a
// short launch pays for fetching its code (unrolled, 6.1 us instead of 4.8).
__global__ __launch_bounds__(kThreads) void dispatch_tiny_kernel(DispatchArgs a, int count_blocks) {
    const int P = a.T * a.K, lane = threadIdx.x & (kWave - 1), b = blockIdx.x;
    Ahead ahead = {};
    if (a.rows && b < a.T) ahead = load_token(a, b, threadIdx.x, kThreads);  // on its way beside the ids
    const int e = lane < P ? expert_of(a, lane) : -1;
    const uint64_t kept = __ballot(e >= 0);
    const int top = 1 << (31 - __builtin_clz(a.E));
    // the pairs of experts below `value`, and of `value`: by bits, from the highest
    auto compare = [&](int value, uint64_t &less, uint64_t &same) {
        less = 0;
        same = kept;
#pragma unroll 1
        for (int bit = top; bit > 0; bit >>= 1) {
            const uint64_t set = __ballot(e & bit), want = value & bit ? ~0ull : 0ull;
            less |= same & want & ~set;
            same &= ~(set ^ want);
        }
    };
    // an expert's rows are counted at its first pair
    uint64_t less, same, firsts = kept;
    int takes = e >= 0 ? 1 : 0;
    if (a.align > 1) {
        compare(max(e, 0), less, same);
        takes = e >= 0 && (same & ((1ull << lane) - 1)) == 0 ? round_up(__popcll(same), a.align) : 0;
        firsts = __ballot(takes > 0);
    }
    auto rows_of = [&](uint64_t pairs) {  // those that the experts of these pairs take
        if (a.align == 1) return static_cast<int>(__popcll(pairs));
        int n = 0;
#pragma unroll 1
        for (uint64_t left = firsts; left; left &= left - 1) {
            const int q = __builtin_ctzll(left);
            n += (pairs >> q) & 1 ? __builtin_amdgcn_readlane(takes, q) : 0;
        }
        return n;
    };
    if (b < a.T) {
        compare(max(e, 0), less, same);
        const int row = e < 0 ? -1 : rows_of(less) + static_cast<int>(__popcll(same & ((1ull << lane) - 1)));
        if (threadIdx.x < kWave && lane / a.K == b && lane < P) {
            a.row_of_pair[lane] = row;
            if (row >= 0) a.pair_of_row[row] = lane;
        }
        if (a.rows)
            move_token(a, b, ahead, [&](int k) { return __builtin_amdgcn_readlane(row, b * a.K + k); }, threadIdx.x, kThreads);
        return;
    }
    const int total = rows_of(kept);
    if (b < a.T + count_blocks) {
        const int mine = (b - a.T) * kThreads + threadIdx.x;
        compare(min(mine, a.E), less, same);
        const int at = rows_of(less);
        if (mine < a.E) a.counts[mine] = static_cast<int>(__popcll(same));
        if (mine <= a.E) a.offset[mine] = at;
        for (int64_t r = total + mine; r < a.R; r += count_blocks * kThreads) a.pair_of_row[r] = -1;
        return;
    }
    compare(max(e, 0), less, same);
    const int at = rows_of(less), used = static_cast<int>(__popcll(same));
    const int first = b - a.T - count_blocks, step = gridDim.x - a.T - count_blocks;
    for (uint64_t left = firsts; left; left &= left - 1) {
        const int q = __builtin_ctzll(left);
        const int from = __builtin_amdgcn_readlane(at, q), n = __builtin_amdgcn_readlane(takes, q);
        for (int r = from + __builtin_amdgcn_readlane(used, q) + first; r < from + n; r += step)
            fill_row(a, r, threadIdx.x, kThreads);
    }
}

// One workgroup per token, each of which counts every pair, and apart those of
// the tokens before its own; the workgroups behind them share the rows that
// fill an expert's last row_align.
template <int kPairs>  // of a thread, at most
__global__ __launch_bounds__(kThreads) void dispatch_small_kernel(DispatchArgs a) {
    __shared__ int s_count[1024], s_before[1024], s_first[1025], s_wave[kWaves], s_mine[kMaxTopK], s_row[kMaxTopK];
    const int t = blockIdx.x, tid = threadIdx.x, P = a.T * a.K, p0 = t * a.K;
    Ahead ahead = {};
    if (a.rows && t < a.T) ahead = load_token(a, t, tid, kThreads);
    int e[kPairs];  // loaded together
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int p = i * kThreads + tid;
        e[i] = p < P ? expert_of(a, p) : -1;
    }
    for (int i = tid; i < a.E; i += kThreads) {
        s_count[i] = 0;
        s_before[i] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int p = i * kThreads + tid;
        if (e[i] >= 0) {
            atomicAdd(&s_count[e[i]], 1);
            if (p < p0) atomicAdd(&s_before[e[i]], 1);
        }
        if (p >= p0 && p < p0 + a.K) s_mine[p - p0] = e[i];
    }
    __syncthreads();
    scan_counts(s_count, s_first, s_wave, a.E, a.align);
    if (t >= a.T) {
        fill_share(a, s_count, s_first, t - a.T, gridDim.x - a.T);
        return;
    }
    if (tid < a.K) {
        const int of = s_mine[tid];
        int row = -1;
        if (of >= 0) {
            row = s_first[of] + s_before[of];
            for (int k = 0; k < tid; ++k) row += s_mine[k] == of;
            a.pair_of_row[row] = p0 + tid;
        }
        a.row_of_pair[p0 + tid] = row;
        s_row[tid] = row;
    }
    if (t == 0)
        for (int i = tid; i <= a.E; i += kThreads) {
            if (i < a.E) a.counts[i] = s_count[i];
            a.offset[i] = s_first[i];
        }
    for (int64_t r = s_first[a.E] + t * kThreads + tid; r < a.R; r += static_cast<int64_t>(a.T) * kThreads)
        a.pair_of_row[r] = -1;
    __syncthreads();
    if (a.rows) move_token(a, t, ahead, [&](int k) { return s_row[k]; }, tid, kThreads);
}

// Larger batches: tokens of a workgroup of the second launch (at most 64
// pairs), and of a block of kParts of them, which the first one counts.
__host__ __device__ __forceinline__ int tokens_of(int K) { return kWave / K; }

// ws[b][e] = pairs of expert e in block b
__global__ __launch_bounds__(kThreads) void dispatch_count_kernel(DispatchArgs a) {
    __shared__ int s_count[1024];
    const int P = a.T * a.K, pairs = kParts * tokens_of(a.K) * a.K, from = blockIdx.x * pairs;
    for (int e = threadIdx.x; e < a.E; e += kThreads) s_count[e] = 0;
    __syncthreads();
    constexpr int kPairs = kParts * kWave / kThreads;  // at most, of a thread: loaded together
    int e[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int p = i * kThreads + threadIdx.x;
        e[i] = p < pairs && from + p < P ? expert_of(a, from + p) : -1;
    }
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
        if (e[i] >= 0) atomicAdd(&s_count[e[i]], 1);
    __syncthreads();
    for (int i = threadIdx.x; i < a.E; i += kThreads) a.workspace[static_cast<size_t>(blockIdx.x) * a.E + i] = s_count[i];
}
// ws[b][e] = pairs of e in the blocks before b, and counts[e] = all of them.
// A wave per quarter of the blocks, a lane per expert.
__global__ __launch_bounds__(kThreads) void dispatch_scan_kernel(DispatchArgs a, int blocks) {
    constexpr int kBatch = 8;
    __shared__ int s_sum[kWaves][kWave];
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave, e = blockIdx.x * kWave + lane;
    const int per = (blocks + kWaves - 1) / kWaves, lo = min(wave * per, blocks), hi = min(lo + per, blocks);
    int *ws = a.workspace + min(e, a.E - 1);
    int sum = 0;
#pragma unroll 8
    for (int b = lo; b < hi; ++b) sum += ws[static_cast<size_t>(b) * a.E];
    s_sum[wave][lane] = sum;
    __syncthreads();
    if (e >= a.E) return;
    int at = 0;
    for (int w = 0; w < wave; ++w) at += s_sum[w][lane];
    if (wave == kWaves - 1) a.counts[e] = at + sum;
    for (int b0 = lo; b0 < hi; b0 += kBatch) {
        int n[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) n[i] = ws[static_cast<size_t>(min(b0 + i, hi - 1)) * a.E];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            if (b0 + i < hi) ws[static_cast<size_t>(b0 + i) * a.E] = at;
            at += n[i];
        }
    }
}
// The maps, and the rows. SCANNED: ws and counts are dispatch_scan_kernel's;
// else ws is the counting launch's.
template <bool SCANNED>
__global__ __launch_bounds__(kThreads) void dispatch_place_kernel(DispatchArgs a, int blocks) {
    __shared__ int s_count[1024], s_first[1025], s_before[1024], s_wave[kWaves], s_row[kWave];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave, P = a.T * a.K;
    const int tokens = tokens_of(a.K), t0 = blockIdx.x * tokens, p0 = t0 * a.K;
    const int block = blockIdx.x / kParts, from = block * kParts * tokens * a.K;
    // what comes before in the block: at most kParts * kWave pairs
    constexpr int kPairs = kParts * kWave / kThreads;
    int early[kPairs];
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
        const int p = from + i * kThreads + tid;
        early[i] = p < p0 ? expert_of(a, p) : -1;
    }
    for (int e = tid; e < a.E; e += kThreads) {
        int all = 0, before = 0;
        if (SCANNED) {
            all = a.counts[e];
            before = a.workspace[static_cast<size_t>(block) * a.E + e];
        } else {
            constexpr int kBatch = 16;
            for (int b0 = 0; b0 < blocks; b0 += kBatch) {
                int n[kBatch];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) n[i] = a.workspace[static_cast<size_t>(min(b0 + i, blocks - 1)) * a.E + e];
#pragma unroll
                for (int i = 0; i < kBatch; ++i) {
                    all += b0 + i < blocks ? n[i] : 0;
                    before += b0 + i < block ? n[i] : 0;
                }
            }
        }
        s_count[e] = all;
        s_before[e] = before;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPairs; ++i)
        if (early[i] >= 0) atomicAdd(&s_before[early[i]], 1);
    scan_counts(s_count, s_first, s_wave, a.E, a.align);
    if (wave == 0) {
        const int p = p0 + lane;
        const bool here = lane < tokens * a.K && p < P;
        const int e = here ? expert_of(a, p) : -1;
        const uint64_t same = same_expert(e, a.E);
        int row = -1;
        if (e >= 0) {
            row = s_first[e] + s_before[e] + __popcll(same & ((1ull << lane) - 1));
            a.pair_of_row[row] = p;
        }
        if (here) a.row_of_pair[p] = row;
        s_row[lane] = row;
    }
    if (blockIdx.x == 0)
        for (int e = tid; e <= a.E; e += kThreads) {
            if (!SCANNED && e < a.E) a.counts[e] = s_count[e];
            a.offset[e] = s_first[e];
        }
    for (int64_t r = s_first[a.E] + static_cast<int64_t>(blockIdx.x) * kThreads + tid; r < a.R;
         r += static_cast<int64_t>(gridDim.x) * kThreads)
        a.pair_of_row[r] = -1;
    if (a.align > 1) fill_share(a, s_count, s_first, blockIdx.x, gridDim.x);
    __syncthreads();
    if (a.rows)
        for (int i = wave; i < tokens && t0 + i < a.T; i += kWaves)
            move_token(a, t0 + i, load_token(a, t0 + i, lane, kWave), [&](int k) { return s_row[i * a.K + k]; }, lane, kWave);
}

// ------------------------------------------------------------------ back

// Thread c of a token's takes elements [8 c, 8 c + 8), or, behind the row's
// whole chunks, one element each. SHORT rows: `tokens` tokens a workgroup (else a
// wave's token is one, and its rows are found by scalar loads).
// kG rows are on their way at once.
template <typename T, typename O, int kG, bool SHORT>
__global__ __launch_bounds__(kThreads) void combine_rows_kernel(RowsArgs a, int tokens) {
    const int chunks = a.H / kVec, rest = a.H % kVec, items = chunks + rest;
    int t = blockIdx.x, c = blockIdx.y * kThreads + threadIdx.x;
    if constexpr (SHORT) {
        const int mine = threadIdx.x / items;
        if (mine >= tokens) return;
        t = t * tokens + mine;
        c = threadIdx.x - mine * items;
    }
    if (c >= items || t >= a.T) return;
    const T *rows = static_cast<const T *>(a.rows);
    const size_t out_at = static_cast<size_t>(t) * a.H;
    const O *addend = static_cast<const O *>(a.addend) + out_at;
    O *out = static_cast<O *>(a.out) + out_at;
    auto sum = [&](auto load, auto &acc) {
        for (int k0 = 0; k0 < a.K && a.R > 0; k0 += kG) {
            decltype(load(rows)) v[kG];
            bool kept[kG];
            float w[kG];
#pragma unroll
            for (int j = 0; j < kG; ++j) {  // dropped pairs, and k past the end: some row, not counted
                const int p = t * a.K + min(k0 + j, a.K - 1), r = a.row_of_pair[p];
                w[j] = a.scales ? a.scales[p] : 1.0f;
                kept[j] = k0 + j < a.K && static_cast<unsigned>(r) < static_cast<unsigned>(a.R);
                v[j] = load(rows + static_cast<size_t>(kept[j] ? r : 0) * a.H);
            }
#pragma unroll
            for (int j = 0; j < kG; ++j)
                if (kept[j]) acc(v[j], w[j]);
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
        store8(out + c * kVec, acc, a.streamed);
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

constexpr int kLook = 16;
// Workgroups [0, T * parts): KM of a token's K rows, kAhead of them on their way
// at once. The others: rows without a pair.
template <typename T, typename O, int KM>
__global__ __launch_bounds__(kThreads) void combine_grad_kernel(RowsArgs a) {
    const int parts = (a.K + KM - 1) / KM, working = a.T * parts;
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave;
    const int chunks = a.H / kVec, rest = a.H % kVec;
    if (static_cast<int>(blockIdx.x) >= working) {
        // every wave looks at kLook rows and takes each kWaves-th of those without a pair
        const size_t bytes = static_cast<size_t>(a.H) * sizeof(T);
        for (int64_t r0 = static_cast<int64_t>(blockIdx.x - working) * kLook; r0 < a.R;
             r0 += static_cast<int64_t>(gridDim.x - working) * kLook) {
            const int r = static_cast<int>(r0) + lane;
            bool none = false;
            if (a.T == 0) {  // no maps either
                none = lane < kLook && r < a.R;
            } else if (lane < kLook && r < a.R) {
                const int p = a.pair_of_row[r];
                none = static_cast<unsigned>(p) >= static_cast<unsigned>(a.T * a.K) || a.row_of_pair[p] != r;
            }
            int i = 0;
            for (uint64_t left = __ballot(none); left; left &= left - 1, ++i)
                if (i % kWaves == wave)
                    zero_row(static_cast<uint8_t *>(a.drows) + (r0 + __builtin_ctzll(left)) * bytes, bytes, lane, kWave, a.streamed);
        }
        return;
    }
    __shared__ float s_dot[kWaves][KM], s_scale[KM];
    __shared__ int s_row[KM];
    const int t = blockIdx.x / parts, k_first = blockIdx.x % parts * KM, count = min(a.K - k_first, KM);
    const int p0 = t * a.K + k_first;
    if (tid < count) {
        s_row[tid] = own_row(a, p0 + tid);
        s_scale[tid] = a.scales ? a.scales[p0 + tid] : 1.0f;
    }
    __syncthreads();
    const O *dout = static_cast<const O *>(a.dout) + static_cast<size_t>(t) * a.H;
    const T *rows = static_cast<const T *>(a.rows);
    T *drows = static_cast<T *>(a.drows);
    float dot[KM] = {};
    struct Eight { T v[kVec]; };
    for (int c = tid; c < chunks; c += kThreads) {
        float d[kVec];
        load8(dout + c * kVec, d);
#pragma unroll
        for (int k0 = 0; k0 < KM; k0 += kAhead) {
            if (k0 >= count) break;
            Eight v[kAhead];
            if (a.dscales) {
#pragma unroll
                for (int j = 0; j < kAhead; ++j) {  // dropped pairs, and k past the end: some row, not counted
                    const int r = max(s_row[min(k0 + j, count - 1)], 0);
                    if (a.R > 0) __builtin_memcpy(&v[j], rows + static_cast<size_t>(r) * a.H + c * kVec, sizeof v[j]);
                }
            }
#pragma unroll
            for (int j = 0; j < kAhead; ++j) {
                const int k = k0 + j, r = __builtin_amdgcn_readfirstlane(k < count ? s_row[k] : -1);
                if (r < 0) continue;
                if (a.dscales) {
#pragma unroll
                    for (int i = 0; i < kVec; ++i) dot[k] += to_f32(v[j].v[i]) * d[i];
                }
                if (a.drows) {
                    const float w = s_scale[k];
                    float o[kVec];
#pragma unroll
                    for (int i = 0; i < kVec; ++i) o[i] = product(d[i], w);
                    store8(drows + static_cast<size_t>(r) * a.H + c * kVec, o, a.streamed);
                }
            }
        }
    }
    const int at = chunks * kVec + tid;
    const float dt = tid < rest ? to_f32(dout[at]) : 0.0f;
#pragma unroll
    for (int k = 0; k < KM; ++k) {
        if (k >= count) break;
        const int r = s_row[k];
        if (r >= 0 && tid < rest) {
            if (a.dscales) dot[k] += to_f32(rows[static_cast<size_t>(r) * a.H + at]) * dt;
            if (a.drows) from_f32(product(dt, s_scale[k]), drows[static_cast<size_t>(r) * a.H + at]);
        }
        if (a.dscales) {
            const float sum = last_lane_sum(dot[k]);
            if (lane == kWave - 1) s_dot[wave][k] = sum;
        }
    }
    __syncthreads();
    if (a.dscales && tid < count) {
        float sum = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) sum += s_dot[w][tid];
        a.dscales[p0 + tid] = sum;
    }
}

template <typename T, typename O>
hipError_t combine_of(const RowsArgs &a, hipStream_t s) {
    const int items = a.H / kVec + a.H % kVec, passes = (a.K + 7) / 8;
    const int tokens = kThreads / items > 1 ? kThreads / items : 1;
    const dim3 grid((a.T + tokens - 1) / tokens, (items + kThreads - 1) / kThreads), blk(kThreads);
    auto launch = [&](auto g) {
        if (tokens > 1) hipLaunchKernelGGL((combine_rows_kernel<T, O, g, true>), grid, blk, 0, s, a, tokens);
        else hipLaunchKernelGGL((combine_rows_kernel<T, O, g, false>), grid, blk, 0, s, a, tokens);
    };
    switch ((a.K + passes - 1) / passes) {
        case 1: launch(std::integral_constant<int, 1>{}); break;
        case 2: launch(std::integral_constant<int, 2>{}); break;
        case 3: launch(std::integral_constant<int, 3>{}); break;
        case 4: launch(std::integral_constant<int, 4>{}); break;
        case 5: launch(std::integral_constant<int, 5>{}); break;
        case 6: launch(std::integral_constant<int, 6>{}); break;
        case 7: launch(std::integral_constant<int, 7>{}); break;
        default: launch(std::integral_constant<int, 8>{}); break;
    }
    return hipGetLastError();
}
// Few tokens: four rows a workgroup, for a shorter way through.
template <typename T, typename O>
hipError_t grad_of(const RowsArgs &a, hipStream_t s) {
    const int looks = a.drows ? (a.R + kLook - 1) / kLook : 0, others = looks < 8192 ? looks : 8192;
    const dim3 blk(kThreads);
    if (a.T < 512) hipLaunchKernelGGL((combine_grad_kernel<T, O, 4>), dim3(a.T * ((a.K + 3) / 4) + others), blk, 0, s, a);
    else hipLaunchKernelGGL((combine_grad_kernel<T, O, kMaxTopK>), dim3(a.T + others), blk, 0, s, a);
    return hipGetLastError();
}

}  // namespace

size_t dispatch_workspace(int T, int K, int E) {
    if (static_cast<int64_t>(T) * K <= kSmallPairs) return 0;
    const int per = kParts * tokens_of(K);
    return static_cast<size_t>((T + per - 1) / per) * E * sizeof(int32_t);
}

hipError_t launch_dispatch(const DispatchArgs &a, hipStream_t s) {
    const dim3 blk(kThreads);
    if (a.T == 0) {
        hipLaunchKernelGGL(dispatch_none_kernel, dim3(1), blk, 0, s, a);
        return hipGetLastError();
    }
    const int P = a.T * a.K;
    if (P <= kWave) {
        const int count_blocks = (a.E + kThreads) / kThreads;  // of E + 1 offsets
        hipLaunchKernelGGL(dispatch_tiny_kernel, dim3(a.T + count_blocks + (a.align > 1 ? 128 : 0)), blk, 0, s, a, count_blocks);
        return hipGetLastError();
    }
    if (P <= kSmallPairs) {
        const dim3 grid(a.T + (a.align > 1 ? 512 : 0));
        if (P <= 4 * kThreads) hipLaunchKernelGGL(dispatch_small_kernel<4>, grid, blk, 0, s, a);
        else hipLaunchKernelGGL(dispatch_small_kernel<kSmallPairs / kThreads>, grid, blk, 0, s, a);
        return hipGetLastError();
    }
    const int tokens = tokens_of(a.K), blocks = (a.T + kParts * tokens - 1) / (kParts * tokens);
    const dim3 grid((a.T + tokens - 1) / tokens);
    hipLaunchKernelGGL(dispatch_count_kernel, dim3(blocks), blk, 0, s, a);
    if (blocks <= kScanBlocks) {
        hipLaunchKernelGGL(dispatch_place_kernel<false>, grid, blk, 0, s, a, blocks);
    } else {
        hipLaunchKernelGGL(dispatch_scan_kernel, dim3((a.E + kWave - 1) / kWave), blk, 0, s, a, blocks);
        hipLaunchKernelGGL(dispatch_place_kernel<true>, grid, blk, 0, s, a, blocks);
    }
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
