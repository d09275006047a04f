"""What is measured of the operators that join the expert block to the rest of a W8A8 program: dense int8 products, the
quantiser of an activation, the norm that joins a block's outputs to the residual stream, and tokens sorted by expert and
back with the gradient.

`own = False` computes their plain form in torch; `own = True` calls the library. Both take the same `prepare` state;
only the int8 weights are re-laid there for the library, as a program does once when it loads a model."""
import math

import torch

own = False

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8}
EPS = 1e-6


# ------------------------------------------------------------------ cases

def listed():
    return [
        # attention output projection of one token: launch latency and a weight stream that fits the caches
        dict(name="w8_t1", op="w8", T=1, N=4096, K=4096, out="bf16", gated=False, bias=False),
        # dense gated block of a ragged decode batch; the contraction is no multiple of anything
        dict(name="w8_t37_odd_gated", op="w8", T=37, N=5006, K=4251, out="fp16", gated=True, bias=True),
        # a prompt through a projection: matrix rate
        dict(name="w8_t4096", op="w8", T=4096, N=8192, K=4096, out="bf16", gated=False, bias=False),
        # input of the down projection in a decode batch (the shared expert's width)
        dict(name="quant_t8", op="quant", T=8, H=2048, dtype="bf16", quant="int8", group=0, smooth=True),
        # a long prompt, codes for the group-wise block: memory rate
        dict(name="quant_t8192_g128", op="quant", T=8192, H=4096, dtype="bf16", quant="int8", group=128, smooth=False),
        # between two layers of a decode step: routed and shared outputs into the stream, codes for the next layer
        dict(name="join_t8", op="join", T=8, H=4096, dtype="bf16", wdtype="bf16", share=True, post=False, gate="none", y=True,
             quant="int8", group=0),
        # a prompt with odd width, norms on both sides and a gate for each channel, FP8 codes
        dict(name="join_t4001_odd", op="join", T=4001, H=5003, dtype="fp16", wdtype="fp32", share=False, post=True, gate="row",
             y=True, quant="fp8", group=0),
        # a decode batch's codes and scales sorted by expert before they are sent to the experts' ranks
        dict(name="dispatch_t8", op="dispatch", T=8, E=256, K=8, H=4096, dtype="int8", groups=1, align=1, drop=False),
        # a prompt's rows for a program's own expert products, segments aligned to their tiles, padded tokens masked
        dict(name="dispatch_t4096", op="dispatch", T=4096, E=256, K=8, H=4096, dtype="bf16", groups=0, align=16, drop=True),
        # what came back of a decode batch, weighted, with the shared expert's output added
        dict(name="combine_t8", op="combine", T=8, E=256, K=8, H=4096, dtype="bf16", out="bf16", weights=True, addend=True,
             drop=False, align=1, grad=False),
        # a ragged prompt, summed for a fp32 residual stream
        dict(name="combine_t2047_odd", op="combine", T=2047, E=72, K=6, H=5003, dtype="bf16", out="fp32", weights=True,
             addend=False, drop=True, align=1, grad=False),
        # its backward pass in training: gradients of the experts' rows and of the routing weights
        dict(name="combine_grad_t4096", op="combine", T=4096, E=64, K=8, H=4096, dtype="bf16", out="bf16", weights=True,
             addend=False, drop=False, align=16, grad=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["w8", "w8", "quant", "join", "dispatch", "combine"])
    if op == "w8":
        gated = rng.random() < 0.4
        k = _log(rng, 64, 16384)
        n = _log(rng, 16, 28672)
        n = n // 2 * 2 if gated else n
        t = _log(rng, 1, max(1, min(8192, 4096 * 8192 * 4096 // (n * k))))
        return dict(op=op, T=t, N=n, K=k, out=rng.choice(["bf16", "bf16", "fp16", "fp32"]), gated=gated, bias=rng.random() < 0.3)
    if op in ("quant", "join"):
        group = rng.choice([0, 0, 64, 128, 256])
        h = _log(rng, 64, 16384)
        quant = rng.choice(["int8", "int8", "fp8"] + (["none"] if op == "join" else []))
        group = group if quant != "none" else 0
        h = max(group, h // group * group) if group else h
        t = _log(rng, 1, max(1, min(16384, 8192 * 4096 // h)))
        dt = rng.choice(["bf16", "bf16", "fp16", "fp32"])
        if op == "quant":
            return dict(op=op, T=t, H=h, dtype=dt, quant=quant, group=group, smooth=rng.random() < 0.5)
        return dict(op=op, T=t, H=h, dtype=dt, wdtype=rng.choice([dt, "fp32"]), share=rng.random() < 0.5, post=rng.random() < 0.5,
                    gate=rng.choice(["none", "row", "token"]), y=quant == "none" or rng.random() < 0.5, quant=quant, group=group)
    e = _log(rng, 8, 512)
    k = rng.randint(1, min(e, 12))
    h = _log(rng, 64, 8192)
    t = _log(rng, 1, max(1, min(16384, 4096 * 8 * 4096 // (k * h))))
    align = rng.choice([1, 1, 16, 64])
    drop = rng.random() < 0.4
    if op == "dispatch":
        dt = rng.choice(["int8", "int8", "bf16", "fp16", "fp32"])
        groups = rng.choice([0, 1, max(1, h // 128)]) if dt == "int8" else 0
        return dict(op=op, T=t, E=e, K=k, H=h, dtype=dt, groups=groups, align=align, drop=drop)
    dt = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    grad = rng.random() < 0.5
    return dict(op=op, T=t, E=e, K=k, H=h, dtype=dt, out=rng.choice([dt, "fp32"]), weights=rng.random() < 0.8,
                addend=not grad and rng.random() < 0.5, drop=drop, align=align, grad=grad)


# ------------------------------------------------------------------ inputs

def _rows(c):
    """Rows that sorted pairs may need: a segment of every expert that has one may end in a padded tile."""
    n = c["T"] * c["K"]
    return n + min(c["E"], n) * (c["align"] - 1)


def _inputs(c, seed):
    g = torch.Generator(device=DEV).manual_seed(seed * 7919 + 29)
    n = lambda *s: torch.randn(*s, generator=g, device=DEV)  # noqa: E731
    u = lambda *s: torch.rand(*s, generator=g, device=DEV)  # noqa: E731
    codes = lambda *s: torch.clamp(torch.round(n(*s) * 32), -127, 127).to(torch.int8)  # noqa: E731
    if c["op"] == "w8":
        T, N, K = c["T"], c["N"], c["K"]
        return dict(x=codes(T, K), x_scale=(0.5 + u(T)) / 32, codes=codes(N, K), scale=(0.5 + u(N)) / (32 * math.sqrt(K)),
                    bias=n(N) * 0.1 if c["bias"] else None)
    if c["op"] == "quant":
        T, H = c["T"], c["H"]
        return dict(x=(n(T, H) * torch.exp(0.5 * n(H))).to(DT[c["dtype"]]), smooth=0.5 + 1.5 * u(H) if c["smooth"] else None)
    if c["op"] == "join":
        T, H, dt, wt = c["T"], c["H"], DT[c["dtype"]], DT[c["wdtype"]]
        wide = torch.exp(0.5 * n(H))  # channels of unlike size, as a residual stream has them
        return dict(block=n(T, H).to(dt), share=n(T, H).to(dt) if c["share"] else None,
                    share_scale=1 / (1 + torch.exp(-n(T))) if c["share"] else None, residual=(n(T, H) * wide * 2).to(dt),
                    post_weight=(0.5 + u(H)).to(wt) if c["post"] else None,
                    gate=None if c["gate"] == "none" else (0.2 * n(*((T, H) if c["gate"] == "token" else (H,)))).to(wt),
                    weight=(0.5 + u(H)).to(wt))
    T, E, K, H = c["T"], c["E"], c["K"], c["H"]
    ids = torch.sort(n(T, E) + 0.7 * n(E), dim=1, descending=True)[1][:, :K].int().contiguous()  # some experts are busier
    mask = None
    if c["drop"]:  # pairs of other ranks' experts, and the tokens that pad a batch
        ids = torch.where(u(T, K) < 0.1, torch.full_like(ids, -1), ids)
        mask = (u(T) < 0.9).to(torch.uint8)
    s = dict(ids=ids, mask=mask)
    if c["op"] == "dispatch":
        s["x"] = codes(T, H) if c["dtype"] == "int8" else n(T, H).to(DT[c["dtype"]])
        s["x_scale"] = (0.5 + u(T, c["groups"])) / 32 if c["groups"] else None
        return s
    s["row_of_pair"], s["pair_of_row"], _, _ = _sort(c, ids, mask)
    s["rows"] = n(_rows(c), H).to(DT[c["dtype"]])
    w = torch.exp(n(T, K))
    s["weights"] = w / w.sum(1, keepdim=True) if c["weights"] else None
    s["addend"] = n(T, H).to(DT[c["out"]]) if c["addend"] else None
    s["dout"] = n(T, H).to(DT[c["out"]]) if c["grad"] else None
    return s


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
    new = lambda *shape, dt: torch.empty(*shape, dtype=dt, device=DEV)  # noqa: E731
    quant = {"none": moe.MOE_QUANT_NONE, "int8": moe.MOE_QUANT_INT8, "fp8": moe.MOE_QUANT_E4M3}
    if c["op"] == "w8":
        d = moe.make_linear_w8_dims(c["T"], c["N"], c["K"], out_dtype=DT[c["out"]], gated=c["gated"])
        s["packed"] = moe.moe_w8a8_pack_weights_w8(d, s["codes"], s["scale"])
        s["out"] = new(c["T"], c["N"] // 2 if c["gated"] else c["N"], dt=DT[c["out"]])
    elif c["op"] in ("quant", "join"):
        T, H, dt = c["T"], c["H"], DT[c["dtype"]]
        s["out"] = {}
        if c["quant"] != "none":
            s["out"]["q"] = new(T, H, dt=torch.int8 if c["quant"] == "int8" else torch.float8_e4m3fn)
            s["out"]["q_scale"] = new(*((T, H // c["group"]) if c["group"] else (T,)), dt=torch.float32)
        if c["op"] == "quant":
            d = moe.make_quant_dims(T, H, dtype=dt, quant=quant[c["quant"]], quant_group=c["group"], amax_eps=EPS)
        else:
            d = moe.make_join_norm_dims(T, H, dtype=dt, weight_dtype=DT[c["wdtype"]], post_norm=c["post"],
                                        gate_rows={"none": 0, "row": 1, "token": T}[c["gate"]], quant=quant[c["quant"]],
                                        quant_group=c["group"], residual_scale=0.75, branch_scale=1.25, post_eps=EPS,
                                        rms_eps=EPS, amax_eps=EPS)
            s["out"]["residual_out"] = new(T, H, dt=dt)
            s["out"]["y"] = new(T, H, dt=dt) if c["y"] else None
    elif c["op"] == "dispatch":
        d = moe.make_dispatch_dims(c["T"], c["H"], c["E"], c["K"], dtype=DT[c["dtype"]], scale_groups=c["groups"],
                                   row_align=c["align"])
        R = moe.moe_w8a8_dispatch_rows(d)
        s["out"] = dict(rows=torch.zeros(R, c["H"], dtype=DT[c["dtype"]], device=DEV),
                        row_scale=torch.zeros(R, c["groups"], device=DEV) if c["groups"] else None,
                        expert_token_nums=new(c["E"], dt=torch.int32), expert_offset=new(c["E"] + 1, dt=torch.int32),
                        row_of_pair=new(c["T"], c["K"], dt=torch.int32), pair_of_row=new(R, dt=torch.int32))
        s["workspace"] = new(max(256, moe.moe_w8a8_dispatch_workspace_size(d)), dt=torch.uint8)
    else:
        d = moe.make_combine_dims(c["T"], c["H"], c["K"], _rows(c), dtype=DT[c["dtype"]], out_dtype=DT[c["out"]])
        if c["grad"]:
            s["out"] = dict(drows=new(_rows(c), c["H"], dt=DT[c["dtype"]]),
                            dscales=new(c["T"], c["K"], dt=torch.float32) if c["weights"] else None)
        else:
            s["out"] = dict(out=new(c["T"], c["H"], dt=DT[c["out"]]))
    s["dims"] = d


# ------------------------------------------------------------------ one pass

def run(s):
    c = s["case"]
    if own:
        moe, d = s["moe"], s["dims"]
        if c["op"] == "w8":
            moe.moe_w8a8_linear_w8(d, s["x"], s["x_scale"], s["packed"], bias=s["bias"], out=s["out"])
            return {"out": s["out"]}
        if c["op"] == "quant":
            moe.moe_w8a8_quant(d, s["x"], smooth=s["smooth"], **s["out"])
        elif c["op"] == "join":
            moe.moe_w8a8_join_norm(d, s["block"], residual=s["residual"], share=s["share"], share_scale=s["share_scale"],
                                   post_weight=s["post_weight"], gate=s["gate"], weight=s["weight"], **s["out"])
        elif c["op"] == "dispatch":
            moe.moe_w8a8_dispatch(d, s["ids"], x=s["x"], x_scale=s["x_scale"], x_active_mask=s["mask"], **s["out"],
                                  workspace=s["workspace"])
        elif c["grad"]:
            moe.moe_w8a8_combine_grad(d, s["dout"], s["row_of_pair"], s["pair_of_row"], rows=s["rows"] if c["weights"] else None,
                                      expert_scales=s["weights"], **s["out"])
        else:
            moe.moe_w8a8_combine(d, s["rows"], s["row_of_pair"], expert_scales=s["weights"], addend=s["addend"], **s["out"])
        return s["out"]
    if c["op"] == "combine":
        return _combine_grad(s) if c["grad"] else _combine(s)
    return {"w8": _w8, "quant": _quant, "join": _join, "dispatch": _dispatch}[c["op"]](s)


def _w8(s):
    c = s["case"]
    o = (s["x"].float() @ s["codes"].float().t()) * s["scale"] * s["x_scale"][:, None]
    if s["bias"] is not None:
        o = o + s["bias"]
    if c["gated"]:
        g, u = o[:, :c["N"] // 2], o[:, c["N"] // 2:]
        o = g / (1 + torch.exp(-g)) * u
    return {"out": o.to(DT[c["out"]])}


def _codes(c, p, rstd):
    """Codes and scales of p * rstd under a = max(max|p| rstd, eps), taken from p: rstd, of any order of sums, enters the
    scales and the rows below the floor alone."""
    top = 127.0 if c["quant"] == "int8" else 448.0
    T, H = p.shape
    p = p.view(T, -1, c["group"] or H)
    pm = p.abs().amax(-1, keepdim=True)
    a = pm if rstd is None else pm * rstd.view(T, 1, 1)
    inv = torch.where(a >= EPS, 1.0 / pm, 1.0 / EPS if rstd is None else rstd.view(T, 1, 1) / EPS)
    v = p * top * inv
    q = (torch.round(v).clamp(-127, 127).to(torch.int8) if c["quant"] == "int8" else v.to(torch.float8_e4m3fn)).view(T, H)
    scale = torch.clamp(a, min=EPS) * (1.0 / top)
    return {"q": q, "q_scale": scale.view(T, -1) if c["group"] else scale.view(T)}


def _quant(s):
    v = s["x"].float()
    if s["smooth"] is not None:
        v = v * s["smooth"]
    return _codes(s["case"], v, None)


def _join(s):
    """The norm of the branch enters r, and r the codes: its mean square is summed in 64 bits, so that codes next to a
    border do not go by the order of a sum."""
    c = s["case"]
    n = s["block"].float()
    if c["share"]:
        n = n + s["share"].float() * s["share_scale"][:, None]
    if c["post"]:
        ms = (n.double() * n.double()).mean(-1, keepdim=True)
        n = n * s["post_weight"].float() * (1 / torch.sqrt(ms + EPS)).float()
    n = n * (s["gate"].float() * 1.25 if s["gate"] is not None else 1.25)
    r = s["residual"].float() * 0.75 + n
    rstd = (1 / torch.sqrt((r.double() * r.double()).mean(-1, keepdim=True) + EPS)).float()
    p = r * s["weight"].float()
    out = {"residual_out": r.to(s["block"].dtype), "y": (p * rstd).to(s["block"].dtype) if c["y"] else None}
    if c["quant"] != "none":
        out.update(_codes(c, p, rstd))
    return out


def _sort(c, ids, mask):
    """Rows of the pairs in the order of (expert, token, k), every expert's at a multiple of `align`: row_of_pair,
    pair_of_row, the experts' counts and the offsets of their rows."""
    T, E, K, R = c["T"], c["E"], c["K"], _rows(c)
    kept = (ids >= 0) & (ids < E)
    if mask is not None:
        kept = kept & (mask[:, None] != 0)
    key = torch.where(kept, ids, E).view(-1).long()
    key, order = torch.sort(key, stable=True)
    counts = torch.zeros(E + 1, dtype=torch.long, device=DEV).index_add_(0, key, torch.ones_like(key))
    before = torch.cumsum(counts, 0) - counts
    padded = (counts + c["align"] - 1) // c["align"] * c["align"]
    offset = torch.cumsum(padded, 0) - padded
    row = offset[key] + torch.arange(T * K, device=DEV) - before[key]
    row = torch.where(key < E, row, torch.full_like(row, R))  # dropped pairs: behind the rows
    row_of_pair = torch.empty(T * K, dtype=torch.long, device=DEV).index_copy_(0, order, row)
    pair_of_row = torch.full((R + 1,), -1, dtype=torch.long, device=DEV).index_copy_(0, row, order)[:R]
    row_of_pair = torch.where(row_of_pair < R, row_of_pair, torch.full_like(row_of_pair, -1)).view(T, K)
    return row_of_pair.int(), pair_of_row.int(), counts[:E].int(), offset.int()


def _dispatch(s):
    c = s["case"]
    row_of_pair, pair_of_row, counts, offset = _sort(c, s["ids"], s["mask"])
    token = (torch.clamp(pair_of_row, min=0) // c["K"]).long()
    some = (pair_of_row >= 0)[:, None]  # padded rows, and those behind the last segment, hold zeros
    return dict(rows=s["x"][token] * some.to(s["x"].dtype), row_scale=s["x_scale"][token] * some if c["groups"] else None,
                expert_token_nums=counts, expert_offset=offset, row_of_pair=row_of_pair, pair_of_row=pair_of_row)


def _combine(s):
    kept = (s["row_of_pair"] >= 0)[..., None]
    z = s["rows"][torch.clamp(s["row_of_pair"], min=0).long()].float() * kept
    if s["weights"] is not None:
        z = z * s["weights"][..., None]
    z = z.sum(1)
    if s["addend"] is not None:
        z = z + s["addend"].float()
    return {"out": z.to(DT[s["case"]["out"]])}


def _combine_grad(s):
    c = s["case"]
    pair = torch.clamp(s["pair_of_row"], min=0).long()
    d = s["dout"].float()[pair // c["K"]] * (s["pair_of_row"] >= 0)[:, None]
    dscales = None
    if s["weights"] is not None:
        dot = (d * s["rows"].float()).sum(1)
        dscales = dot[torch.clamp(s["row_of_pair"], min=0).long()] * (s["row_of_pair"] >= 0)
        d = d * s["weights"].view(-1)[pair][:, None]
    return {"drows": d.to(DT[c["dtype"]]), "dscales": dscales}


# ------------------------------------------------------------------ work and exact values

def work(case):
    c = case
    if c["op"] == "w8":
        T, N, K = c["T"], c["N"], c["K"]
        b = N * K + 4 * N + T * K + 4 * T + (4 * N if c["bias"] else 0) + T * (N // 2 if c["gated"] else N) * DT[c["out"]].itemsize
        return {"bytes": b, "flops": 2 * T * N * K}
    if c["op"] in ("quant", "join"):
        n, e = c["T"] * c["H"], DT[c["dtype"]].itemsize
        b = n + 4 * c["T"] * (c["H"] // c["group"] if c["group"] else 1) if c["quant"] != "none" else 0
        if c["op"] == "quant":
            return {"bytes": b + n * e + (4 * c["H"] if c["smooth"] else 0), "flops": 3 * n}
        w = DT[c["wdtype"]].itemsize
        b += n * e * (3 + (1 if c["share"] else 0) + (1 if c["y"] else 0)) + c["H"] * w * (2 if c["post"] else 1)
        b += {"none": 0, "row": c["H"] * w, "token": n * w}[c["gate"]] + (4 * c["T"] if c["share"] else 0)
        return {"bytes": b, "flops": 14 * n}
    T, E, K, H = c["T"], c["E"], c["K"], c["H"]
    kept = int(T * K * (0.81 if c["drop"] else 1.0))  # pairs
    e = DT[c["dtype"]].itemsize
    if c["op"] == "dispatch":
        return {"bytes": (T + kept) * (H * e + 4 * c["groups"]) + 8 * E + 4 * (2 * T * K + _rows(c)), "flops": 0}
    o = DT[c["out"]].itemsize
    b = (kept * H * e + T * H * o) + T * K * (8 if c["weights"] else 4)
    if c["grad"]:
        b += (kept * H * e if c["weights"] else 0) + 4 * _rows(c) + (4 * T * K if c["weights"] else 0)
        return {"bytes": b, "flops": 3 * kept * H}
    return {"bytes": b + (T * H * o if c["addend"] else 0), "flops": 2 * kept * H}


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "w8":
        xt = s["x"].double().t().contiguous()
        o = torch.cat([torch.mm(w.double(), xt) * f.double()[:, None]
                       for w, f in zip(s["codes"].split(4096), s["scale"].split(4096))]).t() * s["x_scale"].double()[:, None]
        if s["bias"] is not None:
            o = o + s["bias"].double()
        if c["gated"]:
            h = c["N"] // 2
            o = o[:, :h] * torch.sigmoid(o[:, :h]) * o[:, h:]
        return {"out": o}
    if c["op"] in ("quant", "join"):
        out = {}
        if c["op"] == "quant":
            y = s["x"].double() if s["smooth"] is None else s["x"].double() * s["smooth"].double()
        else:
            r = s["block"].double()
            if c["share"]:
                r = r + s["share"].double() * s["share_scale"].double()[:, None]
            if c["post"]:
                r = r / torch.sqrt(torch.linalg.vector_norm(r, dim=1, keepdim=True) ** 2 / c["H"] + EPS) * s["post_weight"].double()
            r = 0.75 * s["residual"].double() + 1.25 * (r if s["gate"] is None else r * s["gate"].double())
            y = r / torch.sqrt(torch.linalg.vector_norm(r, dim=1, keepdim=True) ** 2 / c["H"] + EPS) * s["weight"].double()
            out.update(residual_out=r, y=y if c["y"] else None)
        if c["quant"] != "none":  # codes are whole numbers or 8-bit values: compared with the plain form's
            a = torch.linalg.vector_norm(y.unflatten(1, (-1, c["group"] or c["H"])), float("inf"), dim=-1)
            out.update(q=None, q_scale=torch.clamp(a if c["group"] else a[:, 0], min=EPS) / (127 if c["quant"] == "int8" else 448))
        return out
    if c["op"] == "dispatch":  # what is moved; the maps are whole numbers, compared with the plain form's
        n = c["T"] * c["K"]
        expert = s["ids"].view(-1).long() if s["mask"] is None else torch.where(s["mask"].repeat_interleave(c["K"]) > 0, s["ids"].view(-1).long(), -1)
        pair = torch.argsort(expert * n + torch.arange(n, device=DEV))[int((expert < 0).sum()):]
        first = torch.searchsorted(expert[pair], torch.arange(c["E"] + 1, device=DEV))
        tiles = -(-(first[1:] - first[:-1]) // c["align"])
        at = (torch.cumsum(tiles, 0) - tiles)[expert[pair]] * c["align"] + torch.arange(len(pair), device=DEV) - first[expert[pair]]
        out = {}
        for name, x in (("rows", s["x"]), ("row_scale", s["x_scale"])):
            out[name] = None if x is None else torch.zeros(_rows(c), *x.shape[1:], dtype=x.dtype, device=DEV)
            if x is not None:
                out[name][at] = x[pair // c["K"]]
        return out
    at = s["row_of_pair"].long()
    w = s["weights"].double() if s["weights"] is not None else torch.ones(at.shape, dtype=torch.float64, device=DEV)
    w = torch.where(at >= 0, w, torch.zeros_like(w))
    if not c["grad"]:
        out = s["addend"].double() if s["addend"] is not None else torch.zeros(c["T"], c["H"], dtype=torch.float64, device=DEV)
        for k in range(c["K"]):
            out = torch.addcmul(out, w[:, k:k + 1], s["rows"][at[:, k]].double())
        return {"out": out}
    rows, d = s["rows"], s["dout"].double()
    drows, ds = torch.zeros(rows.shape[0] + 1, c["H"], dtype=torch.float64, device=DEV), torch.zeros_like(w)
    for k in range(c["K"]):
        i = torch.where(at[:, k] >= 0, at[:, k], rows.shape[0])
        drows[i] = d * w[:, k:k + 1]
        ds[:, k] = torch.linalg.vecdot(d, rows[at[:, k]].double()) * (at[:, k] >= 0)
    return {"drows": drows[:-1], "dscales": ds if s["weights"] is not None else None}
