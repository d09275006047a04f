"""What is measured of the operators around the expert block: the pre-norm with its 8-bit output, the router, and dense
products with 4-bit weights.

`own = False` computes their plain form in torch; `own = True` calls the library. Both take the same `prepare` state;
only the 4-bit weights are re-laid there for the library, as a program does once when it loads a model."""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
SCORES = ("softmax", "sigmoid", "sqrtsoftplus")


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token between two blocks: nothing but latency. Hidden size of the decode workload.
        dict(name="norm_t1", op="norm", T=1, H=4096, dtype="bf16", residual=True, y=True, quant="int8", group=0),
        # a serving batch at the widest hidden size of the pages, codes for the group-wise block
        dict(name="norm_t64_g128", op="norm", T=64, H=7168, dtype="bf16", residual=True, y=True, quant="int8", group=128),
        # ragged batch, odd width, FP8 codes for the FP4-weight block, first layer (no residual yet)
        dict(name="norm_odd_fp8", op="norm", T=777, H=5003, dtype="fp16", residual=False, y=True, quant="fp8", group=0),
        # a long prompt: memory rate
        dict(name="norm_t8192", op="norm", T=8192, H=4096, dtype="bf16", residual=True, y=True, quant="int8", group=0),
        # attention output projection of one token
        dict(name="w4_t1", op="w4", T=1, N=4096, K=4096, G=128, x="bf16", zeros=False, gated=False, bias=False),
        # dense gated block of a decode batch on the norm's int8 codes (the shared expert's sizes)
        dict(name="w4_t8_int8_gated", op="w4", T=8, N=4096, K=4096, G=64, x="int8", zeros=True, gated=True, bias=False),
        # odd output width, a contraction that ends inside a tile, smallest groups, three token tiles
        dict(name="w4_t33_odd", op="w4", T=33, N=5003, K=4256, G=32, x="fp16", zeros=True, gated=False, bias=True),
        # the widest dense layer, two tokens: weight stream
        dict(name="w4_t2_wide", op="w4", T=2, N=28672, K=8192, G=128, x="bf16", zeros=False, gated=True, bias=False),
        # the same weights on a prompt: matrix rate
        dict(name="w4_t512", op="w4", T=512, N=8192, K=4096, G=128, x="bf16", zeros=False, gated=False, bias=False),
        # router of the decode workload
        dict(name="gate_t8", op="gate", T=8, E=256, H=4096, k=8, score="softmax", bias=False, norm=True, x="bf16", w="bf16"),
        # odd sizes, fp32 router weights, selection bias
        dict(name="gate_odd_bias", op="gate", T=509, E=72, H=2501, k=6, score="sigmoid", bias=True, norm=True, x="bf16", w="fp32"),
        # router of a prompt
        dict(name="gate_t4096", op="gate", T=4096, E=256, H=4096, k=8, score="sqrtsoftplus", bias=True, norm=True, x="bf16", w="bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm", "w4", "gate"])
    if op == "norm":
        quant = rng.choice(["int8", "int8", "fp8", "none"])
        group = rng.choice([0, 0, 64, 128, 256]) if quant != "none" else 0
        h = _log(rng, 64, 16384)
        if group:
            h = max(group, h // group * group)
        t = _log(rng, 1, max(1, min(16384, 8192 * 4096 // h)))
        return dict(op=op, T=t, H=h, dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]), residual=rng.random() < 0.7,
                    y=quant == "none" or rng.random() < 0.7, quant=quant, group=group)
    if op == "w4":
        g = rng.choice([32, 64, 128])
        gated = rng.random() < 0.4
        k = max(g, _log(rng, 256, 16384) // g * g)
        n = _log(rng, 16, min(28672, 28672 * 8192 // k))
        n = n // 2 * 2 if gated else n
        t = min(_log(rng, 1, 600), max(1, 512 * 8192 * 4096 // (n * k)))
        return dict(op=op, T=t, N=n, K=k, G=g, x=rng.choice(["bf16", "bf16", "fp16", "int8"]), zeros=rng.random() < 0.5,
                    gated=gated, bias=rng.random() < 0.3)
    e = _log(rng, 8, 512)
    h = _log(rng, 128, 8192)
    t = _log(rng, 1, max(1, min(4096, 4096 * 256 * 4096 // (e * h))))
    return dict(op=op, T=t, E=e, H=h, k=rng.randint(1, min(e, 12)), score=rng.choice(SCORES), bias=rng.random() < 0.5,
                norm=rng.random() < 0.7, x=rng.choice(["bf16", "bf16", "fp32"]), w=rng.choice(["bf16", "fp32"]))


# ------------------------------------------------------------------ inputs

def _inputs(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + 13)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    if c["op"] == "norm":
        T, H, dt = c["T"], c["H"], DT[c["dtype"]]
        wide = torch.exp(0.5 * n(H))  # channels of unlike size, as a residual stream has them
        return dict(x=n(T, H).to(dt), residual=(n(T, H) * wide * 2).to(dt) if c["residual"] else None,
                    weight=(0.5 + u(H)).to(dt))
    if c["op"] == "w4":
        T, N, K, G = c["T"], c["N"], c["K"], c["G"]
        codes = torch.randint(0, 256, (N, K // 2), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8)
        scale = (0.5 + u(N, K // G)) * (0.25 / math.sqrt(K))
        zero = torch.randint(5, 11, (N, K // G), generator=g, device=DEV, dtype=torch.int32).to(torch.uint8) if c["zeros"] else None
        if c["x"] == "int8":
            x = torch.clamp(torch.round(n(T, K) * 32), -127, 127).to(torch.int8)
            xs = (0.5 + u(T)) / 32
        else:
            x, xs = n(T, K).to(DT[c["x"]]), None
        return dict(x=x, x_scale=xs, codes=codes, scale=scale, zero=zero, bias=n(N) * 0.1 if c["bias"] else None)
    T, E, H = c["T"], c["E"], c["H"]
    return dict(x=n(T, H).to(DT[c["x"]]), weight=(n(E, H) / math.sqrt(H)).to(DT[c["w"]]),
                bias=n(E) * 0.02 if c["bias"] else None)


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    """What a program keeps beside its tensors: the sizes, the output buffers, the workspace, and the re-laid weights."""
    import moe_expert_ffn_route_amd as moe
    c = s["case"]
    s["moe"] = moe
    if c["op"] == "norm":
        T, H, dt = c["T"], c["H"], DT[c["dtype"]]
        d = moe.make_norm_dims(T, H, dtype=dt, weight_dtype=dt,
                               quant={"none": moe.MOE_QUANT_NONE, "int8": moe.MOE_QUANT_INT8, "fp8": moe.MOE_QUANT_E4M3}[c["quant"]],
                               quant_group=c["group"], rms_eps=1e-6, amax_eps=1e-6)
        s["dims"] = d
        s["out"] = dict(residual_out=torch.empty(T, H, dtype=dt, device=DEV) if c["residual"] else None,
                        y=torch.empty(T, H, dtype=dt, device=DEV) if c["y"] else None)
        if c["quant"] != "none":
            s["out"]["q"] = torch.empty(T, H, dtype=torch.int8 if c["quant"] == "int8" else torch.float8_e4m3fn, device=DEV)
            s["out"]["q_scale"] = torch.empty((T, H // c["group"]) if c["group"] else (T,), dtype=torch.float32, device=DEV)
    elif c["op"] == "w4":
        act = torch.int8 if c["x"] == "int8" else DT[c["x"]]
        d = moe.make_linear_w4_dims(c["T"], c["N"], c["K"], group=c["G"], act_dtype=act, gated=c["gated"], has_zeros=c["zeros"])
        s["dims"] = d
        s["packed"] = moe.moe_w8a8_pack_weights_w4(d, s["codes"], s["scale"], s["zero"])
        s["out"] = torch.empty(c["T"], c["N"] // 2 if c["gated"] else c["N"],
                               dtype=torch.float16 if c["x"] == "fp16" else torch.bfloat16, device=DEV)
    else:
        d = moe.make_gate_dims(c["T"], c["H"], c["E"], c["k"], score={"softmax": moe.MOE_SCORE_SOFTMAX, "sigmoid": moe.MOE_SCORE_SIGMOID,
                               "sqrtsoftplus": moe.MOE_SCORE_SQRT_SOFTPLUS}[c["score"]], normalize=c["norm"], route_scale=2.5,
                               dtype=DT[c["x"]], weight_dtype=DT[c["w"]])
        s["dims"] = d
        s["workspace"] = torch.empty(max(256, moe.moe_w8a8_gate_workspace_size(d)), dtype=torch.uint8, device=DEV)
        s["ids"] = torch.empty(c["T"], c["k"], dtype=torch.int32, device=DEV)
        s["scales"] = torch.empty(c["T"], c["k"], dtype=torch.float32, device=DEV)


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        moe, d = s["moe"], s["dims"]
        if c["op"] == "norm":
            moe.moe_w8a8_norm_quant(d, s["x"], s["weight"], residual=s["residual"], **s["out"])
            return s["out"]
        if c["op"] == "w4":
            moe.moe_w8a8_linear_w4(d, s["x"], s["packed"], x_scale=s["x_scale"], bias=s["bias"], out=s["out"])
            return {"out": s["out"]}
        moe.moe_w8a8_gate(d, s["x"], s["weight"], bias=s["bias"], expert_ids=s["ids"], expert_scales=s["scales"],
                          workspace=s["workspace"])
        return {"ids": s["ids"], "scales": s["scales"]}
    return {"norm": _norm, "w4": _w4, "gate": _gate}[c["op"]](s)


def _norm(s):
    """r = x + residual, y = r * weight / rms(r). The codes are those of y under a = max(max|y|, eps): with p = r * weight,
    y / max|y| = p / max|p|, so they are taken from p, and rms(r) enters the scales alone."""
    c = s["case"]
    r = s["x"].float()
    out = {"residual_out": None}
    if s["residual"] is not None:
        r = r + s["residual"].float()
        out["residual_out"] = r.to(s["x"].dtype)
    rstd = torch.rsqrt((r * r).mean(-1, keepdim=True) + 1e-6)
    p = r * s["weight"].float()
    out["y"] = (p * rstd).to(s["x"].dtype) if c["y"] else None
    if c["quant"] != "none":
        top = 127.0 if c["quant"] == "int8" else 448.0
        T, H = p.shape
        grouped = p.view(T, H // c["group"], c["group"]) if c["group"] else p.view(T, 1, H)
        rstd = rstd.view(T, 1, 1)
        pm = grouped.abs().amax(-1, keepdim=True)
        a = pm * rstd
        inv = torch.where(a >= 1e-6, 1.0 / pm, rstd / 1e-6)  # rows below the floor keep their rms
        v = grouped * top * inv
        out["q"] = (torch.round(v).clamp(-127, 127).to(torch.int8) if c["quant"] == "int8" else v.to(torch.float8_e4m3fn)).view(T, H)
        scale = torch.clamp(a, min=1e-6) * (1.0 / top)
        out["q_scale"] = scale.view(T, H // c["group"]) if c["group"] else scale.view(T)
    return out


def _w4(s):
    c = s["case"]
    N, K, G = c["N"], c["K"], c["G"]
    q = torch.stack((s["codes"] & 15, s["codes"] >> 4), -1).view(N, K // G, G).float()
    q = q - (s["zero"].float()[..., None] if s["zero"] is not None else 8.0)
    w = (q * s["scale"][..., None]).view(N, K)
    o = s["x"].float() @ w.t()
    if s["x_scale"] is not None:
        o = o * s["x_scale"][:, None]
    if s["bias"] is not None:
        o = o + s["bias"]
    if c["gated"]:
        g, u = o[:, :N // 2], o[:, N // 2:]
        o = g / (1 + torch.exp(-g)) * u
    return {"out": o.to(torch.float16 if c["x"] == "fp16" else torch.bfloat16)}


def _gate(s):
    """Logits in 64 bits: which experts a token takes is decided between neighbouring values."""
    c = s["case"]
    l = s["x"].double() @ s["weight"].double().t()
    if c["score"] == "softmax":
        v = torch.exp(l - l.amax(-1, keepdim=True))
        v = v / v.sum(-1, keepdim=True)
    elif c["score"] == "sigmoid":
        v = 1 / (1 + torch.exp(-l))
    else:
        v = torch.sqrt(torch.clamp(l, min=0) + torch.log1p(torch.exp(-l.abs())))
    choice = l if s["bias"] is None else v + s["bias"].double()
    ids = torch.sort(choice, dim=-1, descending=True, stable=True)[1][:, :c["k"]]
    w = torch.gather(v, 1, ids)
    if c["norm"]:
        w = w / w.sum(-1, keepdim=True)
    return {"ids": ids.int(), "scales": (w * 2.5).float()}


# ------------------------------------------------------------------ work and exact values

def work(case):
    c = case
    if c["op"] == "norm":
        e = DT[c["dtype"]].itemsize
        n = c["T"] * c["H"]
        b = n * e * (1 + (2 if c["residual"] else 0) + (1 if c["y"] else 0)) + c["H"] * e
        if c["quant"] != "none":
            b += n + 4 * c["T"] * (c["H"] // c["group"] if c["group"] else 1)
        return {"bytes": b, "flops": 8 * n}
    if c["op"] == "w4":
        nk = c["N"] * c["K"]
        b = nk // 2 + 4 * nk // c["G"] + (nk // c["G"] if c["zeros"] else 0) + (4 * c["N"] if c["bias"] else 0)
        b += c["T"] * c["K"] * (1 if c["x"] == "int8" else 2) + (4 * c["T"] if c["x"] == "int8" else 0)
        b += 2 * c["T"] * (c["N"] // 2 if c["gated"] else c["N"])
        return {"bytes": b, "flops": 2 * c["T"] * nk}
    b = c["T"] * c["H"] * DT[c["x"]].itemsize + c["E"] * c["H"] * DT[c["w"]].itemsize + 8 * c["T"] * c["k"]
    return {"bytes": b + (4 * c["E"] if c["bias"] else 0), "flops": 2 * c["T"] * c["E"] * c["H"]}


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "norm":
        r = s["x"].double() + (s["residual"].double() if s["residual"] is not None else 0)
        y = r / torch.sqrt(torch.linalg.vector_norm(r, dim=1, keepdim=True) ** 2 / c["H"] + 1e-6) * s["weight"].double()
        out = {"residual_out": r if s["residual"] is not None else None, "y": y if c["y"] else None}
        if c["quant"] != "none":  # codes are whole numbers or 8-bit values: compared with the plain form's
            top = 127 if c["quant"] == "int8" else 448
            a = torch.linalg.vector_norm(y.unflatten(1, (-1, c["group"] or c["H"])), float("inf"), dim=-1)
            out["q"] = None
            out["q_scale"] = torch.clamp(a if c["group"] else a[:, 0], min=1e-6) / top
        return out
    if c["op"] == "w4":
        parts = []
        for i in range(0, c["N"], 4096):
            b = s["codes"][i:i + 4096].long()
            w = torch.empty(b.shape[0], c["K"], dtype=torch.float64, device=DEV)
            w[:, 0::2], w[:, 1::2] = b % 16, b // 16
            z = s["zero"][i:i + 4096].double() if s["zero"] is not None else torch.full_like(s["scale"][i:i + 4096], 8).double()
            w -= z.repeat_interleave(c["G"], 1)
            w *= s["scale"][i:i + 4096].double().repeat_interleave(c["G"], 1)
            parts.append(torch.mm(w, s["x"].double().t().contiguous()))
        o = torch.cat(parts).t()
        if s["x_scale"] is not None:
            o = o * s["x_scale"].double()[:, None]
        if s["bias"] is not None:
            o = o + s["bias"].double()
        if c["gated"]:
            h = c["N"] // 2
            o = o[:, :h] * torch.sigmoid(o[:, :h]) * o[:, h:]
        return {"out": o}
    l = torch.mm(s["weight"].double(), s["x"].double().t().contiguous()).t()
    v = {"softmax": lambda: torch.softmax(l, 1), "sigmoid": lambda: torch.sigmoid(l),
         "sqrtsoftplus": lambda: torch.nn.functional.softplus(l, threshold=50).sqrt()}[c["score"]]()
    order = v + s["bias"].double() if s["bias"] is not None else l
    ids = torch.topk(order, c["k"], dim=1).indices
    w = v.gather(1, ids)
    if c["norm"]:
        w = w / w.sum(1, keepdim=True)
    return {"ids": None, "scales": 2.5 * w}
