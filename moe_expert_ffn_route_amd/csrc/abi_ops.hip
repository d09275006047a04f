// C ABI of the operators around the expert block: argument validation of the
// pre-norm, the router and the 4-bit dense product, and their launches.
// Nothing here allocates or synchronises.
#include <math.h>

#include "abi_check.h"

using namespace moe;

namespace {

constexpr int kMaxOut = 1 << 20;
constexpr int kMaxIn = 1 << 17;
constexpr int64_t kMaxW4Tiles = 1 << 23;  // 16 x 128 weights each: 17 G weights, and a packing grid under 2^31 threads

moe_status_t check_norm(const moe_w8a8_norm_dims_t *d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->num_tokens < 0 || d->hidden <= 0 || !is_float_dtype(d->dtype) || !is_float_dtype(d->weight_dtype) ||
        d->quant < MOE_QUANT_NONE || d->quant > MOE_QUANT_E4M3)
        return MOE_ERR_INVALID_ARG;
    if (!(d->rms_eps >= 1e-30f) || !isfinite(d->rms_eps) || !(d->amax_eps >= 1e-20f) || !isfinite(d->amax_eps))
        return MOE_ERR_INVALID_ARG;
    if (d->num_tokens > kMaxTokens || d->hidden > kMaxHidden) return MOE_ERR_UNSUPPORTED;
    if (d->weight_dtype != d->dtype && d->weight_dtype != MOE_DTYPE_FP32) return MOE_ERR_UNSUPPORTED;
    if (d->quant_group != 0) {
        const int g = d->quant_group;
        if ((g != 64 && g != 128 && g != 256) || d->hidden % g) return MOE_ERR_UNSUPPORTED;
        if (d->quant == MOE_QUANT_NONE) return MOE_ERR_INVALID_ARG;
    }
    return MOE_OK;
}

moe_status_t check_gate(const moe_w8a8_gate_dims_t *d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->num_tokens < 0 || d->hidden <= 0 || d->moe_expert_num <= 0 || d->topk <= 0 ||
        d->topk > d->moe_expert_num || d->score < MOE_SCORE_SOFTMAX || d->score > MOE_SCORE_SQRT_SOFTPLUS ||
        (d->normalize != 0 && d->normalize != 1) || !is_float_dtype(d->dtype) || !is_float_dtype(d->weight_dtype) ||
        !isfinite(d->route_scale))
        return MOE_ERR_INVALID_ARG;
    if (d->num_tokens > kMaxTokens || d->hidden > kMaxHidden || d->moe_expert_num > kMaxExperts ||
        d->topk > kMaxTopK)
        return MOE_ERR_UNSUPPORTED;
    if (d->weight_dtype == MOE_DTYPE_FP16 && d->dtype != MOE_DTYPE_FP16) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

moe_status_t check_w4(const moe_w8a8_linear_w4_dims_t *d) {
    if (!d) return MOE_ERR_INVALID_ARG;
    if (d->num_tokens < 0 || d->out_features <= 0 || d->in_features <= 0 || (d->gated != 0 && d->gated != 1) ||
        (d->has_zeros != 0 && d->has_zeros != 1) || (d->gated && d->out_features % 2))
        return MOE_ERR_INVALID_ARG;
    if (d->group != 32 && d->group != 64 && d->group != 128) return MOE_ERR_UNSUPPORTED;
    if (d->act_dtype != MOE_DTYPE_BF16 && d->act_dtype != MOE_DTYPE_FP16 && d->act_dtype != MOE_DTYPE_INT8)
        return MOE_ERR_UNSUPPORTED;
    if (d->in_features % d->group) return MOE_ERR_INVALID_ARG;
    if (d->num_tokens > kMaxTokens || d->out_features > kMaxOut || d->in_features > kMaxIn)
        return MOE_ERR_UNSUPPORTED;
    if (((d->out_features + 15ll) / 16 + 1) * ((d->in_features + 127ll) / 128) > kMaxW4Tiles)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

// Parts of a packed 4-bit weight: codes, scales, zero points.
struct W4Layout {
    int n_tiles, k_tiles;
    size_t scale_off, zero_off, total;
};
W4Layout w4_layout(const moe_w8a8_linear_w4_dims_t *d) {
    W4Layout L;
    // 16 rows per tile: 8 gate and 8 up rows when gated
    L.n_tiles = d->gated ? (d->out_features / 2 + 7) / 8 : (d->out_features + 15) / 16;
    L.k_tiles = (d->in_features + 127) / 128;
    const size_t tiles = static_cast<size_t>(L.n_tiles) * L.k_tiles;
    const size_t groups = tiles * (128 / d->group) * 16;  // (row, group) pairs
    L.scale_off = tiles * 1024;
    L.zero_off = L.scale_off + groups * sizeof(float);
    L.total = L.zero_off + (d->has_zeros ? groups : 0);
    return L;
}

LinearW4Args w4_args(const moe_w8a8_linear_w4_dims_t *d, const W4Layout &L, const void *weight) {
    LinearW4Args a = {};
    const uint8_t *w = static_cast<const uint8_t *>(weight);
    a.codes = w;
    a.scale = reinterpret_cast<const float *>(w + L.scale_off);
    a.zero = d->has_zeros ? w + L.zero_off : nullptr;
    a.T = d->num_tokens;
    a.N = d->out_features;
    a.K = d->in_features;
    a.group = d->group;
    a.act = d->act_dtype;
    a.gated = d->gated;
    a.n_tiles = L.n_tiles;
    a.k_tiles = L.k_tiles;
    return a;
}

}  // namespace

extern "C" moe_status_t moe_w8a8_norm_quant(const moe_w8a8_norm_dims_t *d, const void *x, const void *residual,
                                            const void *weight, void *residual_out, void *y, void *q, float *q_scale,
                                            void *stream) {
    const moe_status_t st = check_norm(d);
    if (st != MOE_OK) return st;
    if (d->num_tokens == 0) return MOE_OK;
    if ((d->quant == MOE_QUANT_NONE) != (q == nullptr) || (q == nullptr) != (q_scale == nullptr))
        return MOE_ERR_INVALID_ARG;
    if ((residual_out && !residual) || (!y && !q)) return MOE_ERR_INVALID_ARG;
    for (const void *p : {x, residual, weight, static_cast<const void *>(residual_out), static_cast<const void *>(y),
                          static_cast<const void *>(q)})
        if (p && !aligned(p, 16)) return MOE_ERR_INVALID_ARG;
    if (q_scale && !aligned(q_scale, 4)) return MOE_ERR_INVALID_ARG;
    if (!x) return MOE_ERR_INVALID_ARG;
    const size_t T = d->num_tokens, H = d->hidden, tensor = T * H * dtype_bytes(d->dtype);
    const Range in[] = {{x, tensor}, {residual, tensor}, {weight, H * dtype_bytes(d->weight_dtype)}};
    const Range out[] = {{residual_out, tensor},
                         {y, tensor},
                         {q, T * H},
                         {q_scale, sizeof(float) * T * (d->quant_group ? H / d->quant_group : 1)}};
    for (int o = 0; o < 4; ++o) {
        for (int i = 0; i < 3; ++i) {
            // residual_out and y may be x or residual themselves: every
            // element is read by the thread that writes it, before it does
            if (o < 2 && i < 2 && out[o].p == in[i].p) continue;
            if (overlap(out[o], in[i])) return MOE_ERR_INVALID_ARG;
        }
        for (int p = 0; p < o; ++p)
            if (overlap(out[o], out[p])) return MOE_ERR_INVALID_ARG;
    }
    NormArgs a;
    a.x = x;
    a.residual = residual;
    a.weight = weight;
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
    a.rms_eps = d->rms_eps;
    a.amax_eps = d->amax_eps;
    return of_launch(launch_norm_quant(a, static_cast<hipStream_t>(stream)));
}

extern "C" moe_status_t moe_w8a8_gate_workspace_size(const moe_w8a8_gate_dims_t *d, size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_gate(d);
    if (st != MOE_OK) return st;
    *bytes = gate_workspace(d->num_tokens, d->moe_expert_num, d->hidden);
    return MOE_OK;
}

extern "C" moe_status_t moe_w8a8_gate(const moe_w8a8_gate_dims_t *d, const void *x, const void *weight,
                                      const float *bias, int32_t *expert_ids, float *expert_scales, void *workspace,
                                      size_t workspace_bytes, void *stream) {
    const moe_status_t st = check_gate(d);
    if (st != MOE_OK) return st;
    if (d->num_tokens == 0) return MOE_OK;
    if (!aligned(x, 16) || !aligned(weight, 16) || !aligned(bias, 4) || !aligned(expert_ids, 4) ||
        !aligned(expert_scales, 4))
        return MOE_ERR_INVALID_ARG;
    if (!x || !weight || !expert_ids || !expert_scales) return MOE_ERR_INVALID_ARG;
    const size_t need = gate_workspace(d->num_tokens, d->moe_expert_num, d->hidden);
    if (!workspace || workspace_bytes < need) return MOE_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return MOE_ERR_INVALID_ARG;
    const size_t T = d->num_tokens, H = d->hidden, E = d->moe_expert_num, TK = T * d->topk;
    const Range in[] = {{x, T * H * dtype_bytes(d->dtype)},
                        {weight, E * H * dtype_bytes(d->weight_dtype)},
                        {bias, E * sizeof(float)}};
    const Range out[] = {{expert_ids, TK * 4}, {expert_scales, TK * 4}, {workspace, need}};
    for (int o = 0; o < 3; ++o) {
        for (const Range &i : in)
            if (overlap(out[o], i)) return MOE_ERR_INVALID_ARG;
        for (int p = 0; p < o; ++p)
            if (overlap(out[o], out[p])) return MOE_ERR_INVALID_ARG;
    }
    GateArgs a;
    a.x = x;
    a.weight = weight;
    a.bias = bias;
    a.ids = expert_ids;
    a.scales = expert_scales;
    a.logits = static_cast<double *>(workspace);
    a.T = d->num_tokens;
    a.H = d->hidden;
    a.E = d->moe_expert_num;
    a.K = d->topk;
    a.score = d->score;
    a.normalize = d->normalize;
    a.dtype = d->dtype;
    a.weight_dtype = d->weight_dtype;
    a.route_scale = d->route_scale;
    return of_launch(launch_gate(a, static_cast<hipStream_t>(stream)));
}

extern "C" moe_status_t moe_w8a8_packed_w4_bytes(const moe_w8a8_linear_w4_dims_t *d, size_t *bytes) {
    if (!bytes) return MOE_ERR_INVALID_ARG;
    const moe_status_t st = check_w4(d);
    if (st != MOE_OK) return st;
    *bytes = w4_layout(d).total;
    return MOE_OK;
}

extern "C" moe_status_t moe_w8a8_pack_weights_w4(const moe_w8a8_linear_w4_dims_t *d, const uint8_t *codes,
                                                 const float *scale, const uint8_t *zero, void *dst, void *stream) {
    const moe_status_t st = check_w4(d);
    if (st != MOE_OK) return st;
    if (!codes || !scale || !dst || (zero != nullptr) != (d->has_zeros != 0) || !aligned(scale, 4) ||
        !aligned(dst, 16))
        return MOE_ERR_INVALID_ARG;
    const W4Layout L = w4_layout(d);
    const size_t n = d->out_features, groups = d->in_features / d->group;
    const Range to = {dst, L.total};
    if (overlap(to, {codes, n * (d->in_features / 2)}) || overlap(to, {scale, n * groups * sizeof(float)}) ||
        overlap(to, {zero, n * groups}))
        return MOE_ERR_INVALID_ARG;
    const LinearW4Args a = w4_args(d, L, dst);
    uint8_t *w = static_cast<uint8_t *>(dst);
    return of_launch(launch_pack_w4(codes, scale, zero, w, reinterpret_cast<float *>(w + L.scale_off),
                                    d->has_zeros ? w + L.zero_off : nullptr, a, static_cast<hipStream_t>(stream)));
}

extern "C" moe_status_t moe_w8a8_linear_w4(const moe_w8a8_linear_w4_dims_t *d, const void *x, const float *x_scale,
                                           const void *weight, const float *bias, void *out, void *stream) {
    const moe_status_t st = check_w4(d);
    if (st != MOE_OK) return st;
    const bool int8 = d->act_dtype == MOE_DTYPE_INT8;
    if (d->num_tokens == 0) return MOE_OK;
    if (!x || !weight || !out || !aligned(x, 16) || !aligned(x_scale, 4) || !aligned(weight, 16) || !aligned(bias, 4) ||
        !aligned(out, 16) || int8 != (x_scale != nullptr))
        return MOE_ERR_INVALID_ARG;
    const W4Layout L = w4_layout(d);
    const size_t T = d->num_tokens, N = d->out_features;
    const Range to = {out, T * (d->gated ? N / 2 : N) * 2};
    const Range in[] = {{x, T * d->in_features * dtype_bytes(d->act_dtype)},
                        {x_scale, T * sizeof(float)},
                        {weight, L.total},
                        {bias, N * sizeof(float)}};
    for (const Range &i : in)
        if (overlap(to, i)) return MOE_ERR_INVALID_ARG;
    LinearW4Args a = w4_args(d, L, weight);
    a.x = x;
    a.x_scale = x_scale;
    a.bias = bias;
    a.out = out;
    return of_launch(launch_linear_w4(a, static_cast<hipStream_t>(stream)));
}
