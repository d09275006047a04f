// C ABI of the operators between the block and the rest of a program: argument
// validation of the int8 dense product, the quantiser, the joining norm, and
// tokens sorted by expert and back, and their launches. Nothing here allocates
// or synchronises.
#include <math.h>

#include "abi_check.h"

using namespace moe;

namespace {

constexpr int kMaxOut = 1 << 20;
constexpr int kMaxIn8 = 1 << 16;               // 2^16 products of at most 2^14: an int32 sum
constexpr int64_t kMaxW8Tiles = 1 << 23;       // 16 x 128 weights each: 16 G weights, and a packing grid under 2^31 threads
constexpr int kMaxRows = 1 << 22;
constexpr int kMaxScaleGroups = 256;

bool is_flag(int v) { return v == 0 || v == 1; }
bool is_eps(float v, float least) { return v >= least && isfinite(v); }

moe_status_t check_w8(const moe_w8a8_linear_w8_dims_t *d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->num_tokens < 0 || d->out_features <= 0 || d->in_features <= 0 || !is_float_dtype(d->out_dtype) ||
        !is_flag(d->gated) || (d->gated && d->out_features % 2))
        return MOE_ERR_INVALID_ARG;
    if (d->num_tokens > kMaxTokens || d->out_features > kMaxOut || d->in_features > kMaxIn8) return MOE_ERR_UNSUPPORTED;
    if (((d->out_features + 15ll) / 16 + 1) * ((d->in_features + 127ll) / 128) > kMaxW8Tiles) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Parts of a packed int8 weight: codes, scales.
struct W8Layout {
    int n_tiles, k_tiles;
    size_t scale_off, total;
};
W8Layout w8_layout(const moe_w8a8_linear_w8_dims_t *d) {
    W8Layout L;
    // 16 rows per tile: 8 gate and 8 up rows when gated
    L.n_tiles = d->gated ? (d->out_features / 2 + 7) / 8 : (d->out_features + 15) / 16;
    L.k_tiles = (d->in_features + 127) / 128;
    L.scale_off = static_cast<size_t>(L.n_tiles) * L.k_tiles * 2048;
    L.total = L.scale_off + static_cast<size_t>(L.n_tiles) * 16 * sizeof(float);
    return L;
}
LinearW8Args w8_args(const moe_w8a8_linear_w8_dims_t *d, const W8Layout &L, const void *weight) {
    LinearW8Args a = {};
    a.codes = static_cast<const int8_t *>(weight);
    a.scale = reinterpret_cast<const float *>(a.codes + L.scale_off);
    a.T = d->num_tokens;
    a.N = d->out_features;
    a.K = d->in_features;
    a.out_dtype = d->out_dtype;
    a.gated = d->gated;
    a.n_tiles = L.n_tiles;
    a.k_tiles = L.k_tiles;
    return a;
}

// hidden, and the groups of an 8-bit output
moe_status_t check_rows(int T, int H, int dtype, int group) {
    if (T < 0 || H <= 0 || !is_float_dtype(dtype)) return MOE_ERR_INVALID_ARG;
    if (T > kMaxTokens || H > kMaxHidden) return MOE_ERR_UNSUPPORTED;
    if (group != 0 && ((group != 64 && group != 128 && group != 256) || H % group)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status_t check_quant(const moe_w8a8_quant_dims_t *d) {
    if (!d || (d->quant != MOE_QUANT_INT8 && d->quant != MOE_QUANT_E4M3) || !is_eps(d->amax_eps, 1e-20f))
        return MOE_ERR_INVALID_ARG;
    return check_rows(d->num_tokens, d->hidden, d->dtype, d->quant_group);
}

moe_status_t check_join(const moe_w8a8_join_norm_dims_t *d) {
    if (!d || d->quant < MOE_QUANT_NONE || d->quant > MOE_QUANT_E4M3 || !is_float_dtype(d->weight_dtype) ||
        !is_flag(d->post_norm) || !is_eps(d->post_eps, 1e-30f) || !is_eps(d->rms_eps, 1e-30f) ||
        !is_eps(d->amax_eps, 1e-20f) || !isfinite(d->residual_scale) || !isfinite(d->branch_scale))
        return MOE_ERR_INVALID_ARG;
    if (d->quant_group != 0 && d->quant == MOE_QUANT_NONE) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_rows(d->num_tokens, d->hidden, d->dtype, d->quant_group);
    if (st != MOE_OK) return st;
    if (d->weight_dtype != d->dtype && d->weight_dtype != MOE_DTYPE_FP32) return MOE_ERR_UNSUPPORTED;
    if (d->num_tokens > 0 && d->gate_rows != 0 && d->gate_rows != 1 && d->gate_rows != d->num_tokens)
        return MOE_ERR_INVALID_ARG;
    return MOE_OK;
}

moe_status_t check_dispatch(const moe_w8a8_dispatch_dims_t *d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->num_tokens < 0 || d->topk <= 0 || d->moe_expert_num <= 0 || d->hidden <= 0 || d->dtype < MOE_DTYPE_BF16 ||
        d->dtype > MOE_DTYPE_INT8 || d->scale_groups < 0 || d->row_align <= 0 || (d->row_align & (d->row_align - 1)))
        return MOE_ERR_INVALID_ARG;
    if (d->num_tokens > kMaxTokens || d->topk > kMaxTopK || d->moe_expert_num > kMaxExperts || d->hidden > kMaxHidden ||
        d->scale_groups > kMaxScaleGroups || d->row_align > 256)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
// Every expert that has a pair may end in a row_align of which it fills one row.
int64_t dispatch_rows(const moe_w8a8_dispatch_dims_t *d) {
    const int64_t pairs = static_cast<int64_t>(d->num_tokens) * d->topk;
    return pairs + (pairs < d->moe_expert_num ? pairs : d->moe_expert_num) * (d->row_align - 1);
}

moe_status_t check_combine(const moe_w8a8_combine_dims_t *d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->num_tokens < 0 || d->topk <= 0 || d->hidden <= 0 || d->num_rows < 0 || !is_float_dtype(d->dtype) ||
        !is_float_dtype(d->out_dtype))
        return MOE_ERR_INVALID_ARG;
    if (d->num_tokens > kMaxTokens || d->topk > kMaxTopK || d->hidden > kMaxHidden || d->num_rows > kMaxRows ||
        (d->out_dtype != d->dtype && d->out_dtype != MOE_DTYPE_FP32))
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}
RowsArgs rows_args(const moe_w8a8_combine_dims_t *d) {
    RowsArgs a = {};
    a.T = d->num_tokens;
    a.K = d->topk;
    a.H = d->hidden;
    a.R = d->num_rows;
    a.dtype = d->dtype;
    a.out_dtype = d->out_dtype;
    return a;
}

template <int N>
bool all_aligned(const void *const (&p)[N], size_t to) {
    for (const void *q : p)
        if (!aligned(q, to)) return false;
    return true;
}
// What a call writes is stored as a stream (ops.h).
template <int O>
bool is_much(const Range (&out)[O]) {
    size_t bytes = 0;
    for (const Range &o : out) bytes += o.p ? o.bytes : 0;
    return bytes >= kStreamBytes;
}
// No output meets an input or another output.
template <int O, int I>
bool apart(const Range (&out)[O], const Range (&in)[I]) {
    for (int o = 0; o < O; ++o) {
        for (const Range &i : in)
            if (overlap(out[o], i)) return false;
        for (int p = 0; p < o; ++p)
            if (overlap(out[o], out[p])) return false;
    }
    return true;
}

}  // namespace

extern "C" moe_status_t moe_w8a8_packed_w8_bytes(const moe_w8a8_linear_w8_dims_t *d, size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_w8(d);
    if (st != MOE_OK) return st;
    *bytes = w8_layout(d).total;
    return MOE_OK;
}

extern "C" moe_status_t moe_w8a8_pack_weights_w8(const moe_w8a8_linear_w8_dims_t *d, const int8_t *codes,
                                                 const float *scale, void *dst, void *stream) {
    const moe_status_t st = check_w8(d);
    if (st != MOE_OK) return st;
    if (!codes || !scale || !dst || !aligned(scale, 4) || !aligned(dst, 16)) return MOE_ERR_INVALID_ARG;
    const W8Layout L = w8_layout(d);
    const size_t n = d->out_features;
    const Range to = {dst, L.total};
    if (overlap(to, {codes, n * d->in_features}) || overlap(to, {scale, n * sizeof(float)})) return MOE_ERR_INVALID_ARG;
    int8_t *w = static_cast<int8_t *>(dst);
    return of_launch(launch_pack_w8(codes, scale, w, reinterpret_cast<float *>(w + L.scale_off), w8_args(d, L, dst),
                                    static_cast<hipStream_t>(stream)));
}

extern "C" moe_status_t moe_w8a8_linear_w8(const moe_w8a8_linear_w8_dims_t *d, const int8_t *x, const float *x_scale,
                                           const void *weight, const float *bias, void *out, void *stream) {
    const moe_status_t st = check_w8(d);
    if (st != MOE_OK) return st;
    if (d->num_tokens == 0) return MOE_OK;
    if (!x || !x_scale || !weight || !out || !all_aligned({x, weight, static_cast<const void *>(out)}, 16) ||
        !aligned(x_scale, 4) || !aligned(bias, 4))
        return MOE_ERR_INVALID_ARG;
    const W8Layout L = w8_layout(d);
    const size_t T = d->num_tokens, N = d->out_features;
    const Range to[] = {{out, T * (d->gated ? N / 2 : N) * dtype_bytes(d->out_dtype)}};
    const Range in[] = {{x, T * d->in_features}, {x_scale, T * sizeof(float)}, {weight, L.total}, {bias, N * sizeof(float)}};
    if (!apart(to, in)) return MOE_ERR_INVALID_ARG;
    LinearW8Args a = w8_args(d, L, weight);
    a.x = x;
    a.x_scale = x_scale;
    a.bias = bias;
    a.out = out;
    a.streamed = is_much(to);
    return of_launch(launch_linear_w8(a, static_cast<hipStream_t>(stream)));
}

extern "C" moe_status_t moe_w8a8_quant(const moe_w8a8_quant_dims_t *d, const void *x, const float *smooth, void *q,
                                       float *q_scale, void *stream) {
    const moe_status_t st = check_quant(d);
    if (st != MOE_OK) return st;
    if (d->num_tokens == 0) return MOE_OK;
    if (!x || !q || !q_scale || !all_aligned({x, static_cast<const void *>(smooth), static_cast<const void *>(q)}, 16) ||
        !aligned(q_scale, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t T = d->num_tokens, H = d->hidden;
    const Range in[] = {{x, T * H * dtype_bytes(d->dtype)}, {smooth, H * sizeof(float)}};
    const Range out[] = {{q, T * H}, {q_scale, sizeof(float) * T * (d->quant_group ? H / d->quant_group : 1)}};
    if (!apart(out, in)) return MOE_ERR_INVALID_ARG;
    QuantArgs a;
    a.x = x;
    a.smooth = smooth;
    a.q = q;
    a.q_scale = q_scale;
    a.T = d->num_tokens;
    a.H = d->hidden;
    a.dtype = d->dtype;
    a.quant = d->quant;
    a.group = d->quant_group;
    a.amax_eps = d->amax_eps;
    a.streamed = is_much(out);
    return of_launch(launch_quant(a, static_cast<hipStream_t>(stream)));
}

extern "C" moe_status_t moe_w8a8_join_norm(const moe_w8a8_join_norm_dims_t *d, const void *block, const void *share,
                                           const float *share_scale, const void *residual, const void *post_weight,
                                           const void *gate, const void *weight, void *residual_out, void *y, void *q,
                                           float *q_scale, void *stream) {
    const moe_status_t st = check_join(d);
    if (st != MOE_OK) return st;
    if (d->num_tokens == 0) return MOE_OK;
    if (!block || (share_scale && !share) || (post_weight && !d->post_norm) || (gate != nullptr) != (d->gate_rows != 0) ||
        (q != nullptr) != (d->quant != MOE_QUANT_NONE) || (q != nullptr) != (q_scale != nullptr) ||
        (!residual_out && !y && !q))
        return MOE_ERR_INVALID_ARG;
    if (!all_aligned({block, share, residual, post_weight, gate, weight, static_cast<const void *>(residual_out),
                      static_cast<const void *>(y), static_cast<const void *>(q)}, 16) ||
        !aligned(share_scale, 4) || !aligned(q_scale, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t T = d->num_tokens, H = d->hidden, tensor = T * H * dtype_bytes(d->dtype);
    const size_t row = H * dtype_bytes(d->weight_dtype);
    // the first three: residual_out and y may be one of them, whose elements
    // are read by the thread that writes them, before it does
    const Range in[] = {{block, tensor},    {share, tensor},          {residual, tensor}, {share_scale, T * sizeof(float)},
                        {post_weight, row}, {gate, row * d->gate_rows}, {weight, row}};
    const Range out[] = {{residual_out, tensor},
                         {y, tensor},
                         {q, T * H},
                         {q_scale, sizeof(float) * T * (d->quant_group ? H / d->quant_group : 1)}};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 7; ++i) {
            if (o < 2 && i < 3 && out[o].p == in[i].p) continue;
            if (overlap(out[o], in[i])) return MOE_ERR_INVALID_ARG;
        }
        for (int p = 0; p < o; ++p)
            if (overlap(out[o], out[p])) return MOE_ERR_INVALID_ARG;
    }
    JoinNormArgs a;
    a.block = block;
    a.share = share;
    a.residual = residual;
    a.post_weight = post_weight;
    a.gate = gate;
    a.weight = weight;
    a.share_scale = share_scale;
    a.residual_out = residual_out;
    a.y = y;
    a.q = q;
    a.q_scale = q_scale;
    a.T = d->num_tokens;
    a.H = d->hidden;
    a.dtype = d->dtype;
    a.weight_dtype = d->weight_dtype;
    a.quant = d->quant;
    a.group = d->quant_group;
    a.post_norm = d->post_norm;
    a.gate_stride = d->gate_rows > 1 ? H : 0;
    a.residual_scale = d->residual_scale;
    a.branch_scale = d->branch_scale;
    a.post_eps = d->post_eps;
    a.rms_eps = d->rms_eps;
    a.amax_eps = d->amax_eps;
    a.streamed = is_much(out);
    return of_launch(launch_join_norm(a, static_cast<hipStream_t>(stream)));
}

extern "C" moe_status_t moe_w8a8_dispatch_rows(const moe_w8a8_dispatch_dims_t *d, int64_t *rows) {
    if (!rows) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_dispatch(d);
    if (st != MOE_OK) return st;
    *rows = dispatch_rows(d);
    return MOE_OK;
}

extern "C" moe_status_t moe_w8a8_dispatch_workspace_size(const moe_w8a8_dispatch_dims_t *d, size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_dispatch(d);
    if (st != MOE_OK) return st;
    *bytes = dispatch_workspace(d->num_tokens, d->topk, d->moe_expert_num);
    return MOE_OK;
}

extern "C" moe_status_t moe_w8a8_dispatch(const moe_w8a8_dispatch_dims_t *d, const int32_t *expert_ids, const void *x,
                                          const float *x_scale, const uint8_t *x_active_mask, void *rows,
                                          float *row_scale, int32_t *expert_token_nums, int32_t *expert_offset,
                                          int32_t *row_of_pair, int32_t *pair_of_row, void *workspace,
                                          size_t workspace_bytes, void *stream) {
    const moe_status_t st = check_dispatch(d);
    if (st != MOE_OK) return st;
    if (!expert_token_nums || !expert_offset || !aligned(expert_token_nums, 4) || !aligned(expert_offset, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t T = d->num_tokens, pairs = T * d->topk, E = d->moe_expert_num, R = dispatch_rows(d);
    const size_t need = dispatch_workspace(d->num_tokens, d->topk, d->moe_expert_num);
    if (T > 0) {
        const bool scales = rows && d->scale_groups > 0;
        if (!expert_ids || !row_of_pair || !pair_of_row || (x != nullptr) != (rows != nullptr) ||
            (x_scale != nullptr) != scales || (row_scale != nullptr) != scales)
            return MOE_ERR_INVALID_ARG;
        if (!all_aligned({x, static_cast<const void *>(rows)}, 16) ||
            !all_aligned({static_cast<const void *>(expert_ids), static_cast<const void *>(x_scale),
                          static_cast<const void *>(row_scale), static_cast<const void *>(row_of_pair),
                          static_cast<const void *>(pair_of_row)}, 4))
            return MOE_ERR_INVALID_ARG;
        if (need && (!workspace || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
        if (need && !aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
    }
    const size_t row = d->hidden * dtype_bytes(d->dtype), scale_row = sizeof(float) * d->scale_groups;
    const Range in[] = {{expert_ids, pairs * 4}, {x, T * row}, {x_scale, T * scale_row}, {x_active_mask, T}};
    const Range out[] = {{rows, R * row},         {row_scale, R * scale_row}, {expert_token_nums, E * 4},
                         {expert_offset, E * 4 + 4}, {row_of_pair, pairs * 4},   {pair_of_row, R * 4},
                         {need ? workspace : nullptr, need}};
    if (!apart(out, in)) return MOE_ERR_INVALID_ARG;
    DispatchArgs a;
    a.ids = expert_ids;
    a.x = x;
    a.x_scale = x_scale;
    a.mask = x_active_mask;
    a.rows = rows;
    a.row_scale = row_scale;
    a.counts = expert_token_nums;
    a.offset = expert_offset;
    a.row_of_pair = row_of_pair;
    a.pair_of_row = pair_of_row;
    a.workspace = static_cast<int32_t *>(workspace);
    a.T = d->num_tokens;
    a.K = d->topk;
    a.E = d->moe_expert_num;
    a.H = d->hidden;
    a.elem = static_cast<int>(dtype_bytes(d->dtype));
    a.groups = rows ? d->scale_groups : 0;
    a.align = d->row_align;
    a.R = static_cast<int64_t>(R);
    a.streamed = is_much(out);
    return of_launch(launch_dispatch(a, static_cast<hipStream_t>(stream)));
}

extern "C" moe_status_t moe_w8a8_combine(const moe_w8a8_combine_dims_t *d, const void *rows, const int32_t *row_of_pair,
                                         const float *expert_scales, const void *addend, void *out, void *stream) {
    const moe_status_t st = check_combine(d);
    if (st != MOE_OK) return st;
    if (d->num_tokens == 0) return MOE_OK;
    if ((!rows && d->num_rows > 0) || !row_of_pair || !out || !all_aligned({rows, addend, static_cast<const void *>(out)}, 16) ||
        !aligned(row_of_pair, 4) || !aligned(expert_scales, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t T = d->num_tokens, H = d->hidden, pairs = T * d->topk, tensor = T * H * dtype_bytes(d->out_dtype);
    const Range to[] = {{out, tensor}};
    const Range in[] = {{rows, d->num_rows * H * dtype_bytes(d->dtype)},
                        {row_of_pair, pairs * 4},
                        {expert_scales, pairs * 4},
                        {addend == out ? nullptr : addend, tensor}};
    if (!apart(to, in)) return MOE_ERR_INVALID_ARG;
    RowsArgs a = rows_args(d);
    a.rows = rows;
    a.row_of_pair = row_of_pair;
    a.scales = expert_scales;
    a.addend = addend;
    a.out = out;
    a.streamed = is_much(to);
    return of_launch(launch_combine_rows(a, static_cast<hipStream_t>(stream)));
}

extern "C" moe_status_t moe_w8a8_combine_grad(const moe_w8a8_combine_dims_t *d, const void *dout,
                                              const int32_t *row_of_pair, const int32_t *pair_of_row, const void *rows,
                                              const float *expert_scales, void *drows, float *dscales, void *stream) {
    const moe_status_t st = check_combine(d);
    if (st != MOE_OK) return st;
    if (d->num_tokens == 0) {  // no row has a pair
        if (!drows || d->num_rows == 0) return MOE_OK;
        if (!aligned(drows, 16)) return MOE_ERR_INVALID_ARG;
        RowsArgs a = rows_args(d);
        a.drows = drows;
        a.streamed = is_much({Range{drows, d->num_rows * static_cast<size_t>(d->hidden) * dtype_bytes(d->dtype)}});
        return of_launch(launch_combine_grad(a, static_cast<hipStream_t>(stream)));
    }
    if (!dout || !row_of_pair || (d->num_rows > 0 && (!pair_of_row || (rows != nullptr) != (dscales != nullptr))) ||
        (!drows && !dscales) || !all_aligned({dout, rows, static_cast<const void *>(drows)}, 16) ||
        !all_aligned({static_cast<const void *>(row_of_pair), static_cast<const void *>(pair_of_row),
                      static_cast<const void *>(expert_scales), static_cast<const void *>(dscales)}, 4))
        return MOE_ERR_INVALID_ARG;
    const size_t T = d->num_tokens, H = d->hidden, R = d->num_rows, pairs = T * d->topk;
    const size_t tensor = R * H * dtype_bytes(d->dtype);
    const Range to[] = {{drows, tensor}, {dscales, pairs * 4}};
    const Range in[] = {{dout, T * H * dtype_bytes(d->out_dtype)}, {row_of_pair, pairs * 4}, {pair_of_row, R * 4},
                        {rows, tensor}, {expert_scales, pairs * 4}};
    if (!apart(to, in)) return MOE_ERR_INVALID_ARG;
    RowsArgs a = rows_args(d);
    a.dout = dout;
    a.row_of_pair = row_of_pair;
    a.pair_of_row = pair_of_row;
    a.rows = rows;
    a.scales = expert_scales;
    a.drows = drows;
    a.dscales = dscales;
    a.streamed = is_much(to);
    return of_launch(launch_combine_grad(a, static_cast<hipStream_t>(stream)));
}
