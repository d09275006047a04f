"""moe_w8a8_quant and moe_w8a8_join_norm on the GPU.

Both are chains of fp32 operations whose order the header fixes, but for two
sums. Codes and scales of the quantiser, and everything the joining norm makes
before its second norm, equal the same operations in torch bit for bit (each a
kernel of its own, so none is fused); the branch's mean square is taken in fp64
there too, where the order decides nothing short of a rounding border of
1 / sqrt(...), 2^-28 wide or less.

Against 64 bits, with u = 2^-24:
  b: a product and a sum, u (|share ss| + |b|) =: e_b.
  n: e_b scaled by |pw| rstd, and 4 u |n| (three roundings, and that of rstd);
     rstd is that of the fp32 b, whose root mean square is off by at most the
     root mean square of e_b.
  r: n's error times |g|, two roundings of g and one of n g (3 u |n g|), 2 u
     |residual rs|, u |r|.
  y: rstd of a sum of at most 64 squares a thread joined over 6 + 16 more
     (100 u with the squares' and the chain's roundings, halved by the root),
     3 u for division, root and product, and r's error twice (through r, and
     through rstd, as above).
  q_scale: y's bound for the largest element, and u for the product with
     1 / Q, u for that constant.
"""
import pytest
import torch

import moe_expert_ffn_route_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
F8 = torch.float8_e4m3fn
EPS = 1e-6
NAMES = {BF: "bf16", FP: "fp16", F32: "fp32"}


def gen(seed):
    return torch.Generator().manual_seed(seed)


def buf(shape, dt):
    """A tensor with a guard behind it."""
    n = 1
    for s in shape:
        n *= s
    b = torch.full((n + 64,), 7.0, device="cuda").to(dt)
    return b, b[:n].view(shape)


def guards(*bufs):
    for b in bufs:
        if b is not None:
            assert bool((b[-64:].float() == 7).all()), "written past the end"


def codes_of(p, rstd, quant, group, eps=EPS):
    """The rule, in fp32 operations: codes from p, scales of p * rstd."""
    T, H = p.shape
    top = torch.tensor(127.0 if quant == "int8" else 448.0, device=p.device)
    eps = torch.tensor(eps, dtype=F32, device=p.device)
    p = p.view(T, -1, group or H)
    pm = p.abs().amax(-1, keepdim=True)
    a = pm * rstd.view(T, 1, 1)
    inv = torch.where(a >= eps, 1.0 / pm, rstd.view(T, 1, 1) * (1.0 / eps))
    v = (p * top * inv).view(T, H)
    q = torch.round(v).clamp(-127, 127).to(torch.int8) if quant == "int8" else v.to(F8)
    s = torch.maximum(a, eps) * (1.0 / top)
    return q, s.view(T, -1) if group else s.view(T)


def same_codes(q, want):
    return torch.equal(q.view(torch.int8), want.view(torch.int8))


# ------------------------------------------------------------------ quantiser

QSHAPES = [(1, 1), (1, 8), (3, 5), (2, 63), (5, 64), (4, 65), (7, 511), (6, 512), (9, 513), (8, 2048), (17, 2051), (3, 4096),
           (10, 5003), (2, 8192), (5, 8200), (3, 9001), (2, 16384), (1, 16383), (700, 5003), (600, 12000), (530, 16384),
           (1000, 640), (2051, 72), (65, 4104)]


def quantise(x, quant="int8", group=0, smooth=None, eps=EPS, stream=None):
    T, H = x.shape
    qb, q = buf((T, H), torch.int8 if quant == "int8" else F8)
    sb, s = buf((T, H // group) if group else (T,), F32)
    d = moe.make_quant_dims(T, H, dtype=x.dtype, quant=moe.MOE_QUANT_INT8 if quant == "int8" else moe.MOE_QUANT_E4M3,
                            quant_group=group, amax_eps=eps)
    moe.moe_w8a8_quant(d, x, smooth=smooth, q=q, q_scale=s, stream=stream)
    torch.cuda.synchronize()
    guards(qb, sb)
    return q, s


def check_quant(x, q, s, quant, group, smooth, eps=EPS):
    v = x.float() if smooth is None else x.float() * smooth
    wq, ws = codes_of(v, torch.ones(x.shape[0], device="cuda"), quant, group, eps)
    assert same_codes(q, wq)
    assert torch.equal(s, ws)
    # the formula in 64 bits: half a step of the code, and the roundings of v Q / a'
    y = x.double() if smooth is None else x.double() * smooth.double()
    sc = (s.double().repeat_interleave(group, 1) if group else s.double()[:, None])
    c = q.float().double()
    half = 0.5 if quant == "int8" else torch.clamp(c.abs() * 2.0 ** -4, min=2.0 ** -10)
    assert bool(((c - y / sc).abs() <= half + 8 * U * (y / sc).abs() + 1e-30).all())


@pytest.mark.parametrize("T,H", QSHAPES)
@pytest.mark.parametrize("dt", [BF, FP, F32], ids=NAMES.get)
def test_quant_shapes(T, H, dt):
    g = gen(T * 31 + H)
    x = (torch.randn(T, H, generator=g) * torch.exp(torch.randn(H, generator=g))).clamp(-3e4, 3e4).to(dt).cuda()
    sm = (0.5 + torch.rand(H, generator=g)).cuda()
    check_quant(x, *quantise(x, "int8", smooth=sm), "int8", 0, sm)
    check_quant(x, *quantise(x, "e4m3"), "e4m3", 0, None)


@pytest.mark.parametrize("T,H,group", [(1, 64, 64), (3, 128, 64), (5, 640, 128), (2, 2048, 256), (9, 4096, 128), (4, 8192, 64),
                                       (3, 16384, 256), (600, 4608, 128), (513, 12544, 64), (70, 1280, 256)])
@pytest.mark.parametrize("dt", [BF, F32], ids=NAMES.get)
def test_quant_groups(T, H, group, dt):
    g = gen(T + H + group)
    x = torch.randn(T, H, generator=g).to(dt).cuda()
    x[:, group // 2] *= 40  # a group with an outlier
    sm = (0.5 + torch.rand(H, generator=g)).cuda()
    check_quant(x, *quantise(x, "int8", group), "int8", group, None)
    check_quant(x, *quantise(x, "e4m3", group, sm), "e4m3", group, sm)


@pytest.mark.parametrize("H", [40, 77, 2048, 9000])
def test_quant_floor_zeros_and_ties(H):
    x = torch.zeros(6, H)
    x[1] = 1e-9
    x[2, 0], x[2, 1:4] = 127, torch.tensor([0.5, 2.5, -62.5])  # scale 1: exact ties, to even
    x[3, -1] = 1e-6 * 0.999
    x[4, H // 2] = -3.0
    x[5] = torch.linspace(-1, 1, H)
    x = x.cuda()
    q, s = quantise(x)
    check_quant(x, q, s, "int8", 0, None)
    eps = torch.tensor(EPS, dtype=F32)
    assert bool((q[0] == 0).all()) and float(s[0]) == float(eps * (1 / torch.tensor(127.0)))
    assert q[2, 1:4].tolist() == [0, 2, -62]
    assert int(q[4, H // 2]) == -127


def test_quant_other_rows_of_a_row_that_is_not_finite():
    x = torch.randn(9, 300, generator=gen(1)).cuda()
    want = quantise(x)
    x[4, 7], x[6, 299] = float("nan"), float("inf")
    got = quantise(x)
    rows = [0, 1, 2, 3, 5, 7, 8]
    assert torch.equal(got[0][rows], want[0][rows]) and torch.equal(got[1][rows], want[1][rows])


def codes_by_the_rule(v, inv, quant):
    """(v * Q) * inv in fp32 as the block's quantiser takes it, any v."""
    t = (v * (127.0 if quant == "int8" else 448.0)) * inv
    if quant == "int8":
        return torch.where(t.isnan(), -127.0, t.round().clamp(-127, 127)).to(torch.int8).view(torch.uint8)
    c = t.nan_to_num(0.0, 448.0, -448.0).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.where(t.isnan(), torch.tensor(0x7F, dtype=torch.uint8), c)


@pytest.mark.parametrize("quant", ["int8", "fp8"])
def test_codes_of_any_value_follow_the_rule(quant):
    """NaN, infinities and values whose product with 127 or 448 leaves fp32: the
    same codes within whole chunks and behind them, from the quantiser and from
    a norm whose weights are that large."""
    nan, inf, top = float("nan"), float("inf"), 3.0e38
    special = [nan, -nan, inf, -inf, top, -top, 1e36, -1e36, 1.0, -1.0, 0.0, 5e35, -4e36]
    x = torch.randn(len(special) + 1, 205, generator=gen(2)) * 1e35
    for i, v in enumerate(special):
        x[i, 11] = x[i, 131] = x[i, 203] = v
    x[-1, :13] = x[-1, 192:205] = torch.tensor(special)
    q, s = quantise(x.cuda(), quant)
    am = torch.where(x.isnan(), 0.0, x.abs()).amax(1, keepdim=True).clamp(min=EPS)
    assert torch.equal(q.cpu().view(torch.uint8), codes_by_the_rule(x, 1.0 / am, quant))

    # x = 1 and x^2 an exact sum: rstd = 1 / sqrt(1 + eps), y = w * rstd
    T, H = 3, 256
    w = torch.randn(H, generator=gen(3)) * 1e36
    w[9], w[77], w[200] = 3e38, -2e38, 1e37
    qd = moe.MOE_QUANT_INT8 if quant == "int8" else moe.MOE_QUANT_E4M3
    out = torch.empty(T, H, dtype=torch.int8 if quant == "int8" else torch.float8_e4m3fn, device="cuda")
    moe.moe_w8a8_norm_quant(moe.make_norm_dims(T, H, dtype=F32, quant=qd), torch.ones(T, H, device="cuda"), w.cuda(), q=out,
                            q_scale=torch.empty(T, device="cuda"))
    want = codes_by_the_rule(w, 1.0 / w.abs().max(), quant)
    assert bool((out.cpu().view(torch.uint8) == want).all())


# --------------------------------------------------------------- joining norm

def inputs(T, H, dt, wt, share=True, ss=True, residual=True, post=True, pw=True, gate="row", weight=True, seed=0):
    g = gen(seed + T * 17 + H)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    c = lambda t, d: None if t is None else t.to(d).cuda()  # noqa: E731
    return dict(block=c(n(T, H), dt), share=c(n(T, H), dt) if share else None,
                share_scale=c(torch.rand(T, generator=g) * 2, F32) if share and ss else None,
                residual=c(n(T, H) * torch.exp(0.5 * n(H)) * 2, dt) if residual else None,
                post_weight=c(0.5 + torch.rand(H, generator=g), wt) if post and pw else None,
                gate=None if not gate else c(0.3 * n(*((T, H) if gate == "token" else (H,))), wt),
                weight=c(0.5 + torch.rand(H, generator=g), wt) if weight else None)


def join(c, post, quant="int8", group=0, rs=0.75, bs=1.25, eps=(1e-5, 1e-6, EPS), want=("residual_out", "y"), stream=None,
         over=None):
    T, H = c["block"].shape
    dt = c["block"].dtype
    wt = next((c[k].dtype for k in ("post_weight", "gate", "weight") if c[k] is not None), dt)
    gate_rows = 0 if c["gate"] is None else 1 if c["gate"].dim() == 1 else T
    d = moe.make_join_norm_dims(T, H, dtype=dt, weight_dtype=wt, post_norm=post, gate_rows=gate_rows,
                                quant=dict(none=0, int8=1, e4m3=2)[quant], quant_group=group, residual_scale=rs,
                                branch_scale=bs, post_eps=eps[0], rms_eps=eps[1], amax_eps=eps[2])
    out, bufs = {}, []
    for k in want:
        b, out[k] = buf((T, H), dt)
        bufs.append(b)
    if quant != "none":
        b, out["q"] = buf((T, H), torch.int8 if quant == "int8" else F8)
        bufs.append(b)
        b, out["q_scale"] = buf((T, H // group) if group else (T,), F32)
        bufs.append(b)
    out.update(over or {})
    torch.cuda.synchronize()
    moe.moe_w8a8_join_norm(d, stream=stream, **c, **out)
    torch.cuda.synchronize()
    guards(*bufs)
    return out


def f32(v):
    return torch.tensor(v, dtype=F32, device="cuda")


def check_join(c, out, post, quant="int8", group=0, rs=0.75, bs=1.25, eps=(1e-5, 1e-6, EPS), dt=None):
    T, H = c["block"].shape
    dt = c["block"].dtype
    up = lambda k: None if c[k] is None else c[k].float()  # noqa: E731
    # the header's operations, one by one
    b = up("block")
    if c["share"] is not None:
        b = b + (up("share") * c["share_scale"][:, None] if c["share_scale"] is not None else up("share"))
    n = b
    if post:
        rstd = (1 / torch.sqrt((b.double() ** 2).mean(1, keepdim=True) + f32(eps[0]).double())).float()
        n = (b * up("post_weight") if c["post_weight"] is not None else b) * rstd
    ng = n * (up("gate") * f32(bs) if c["gate"] is not None else f32(bs))
    r = up("residual") * f32(rs) + ng if c["residual"] is not None else ng
    p = r * up("weight") if c["weight"] is not None else r
    if "residual_out" in out:
        assert torch.equal(out["residual_out"], r.to(dt))
    # in 64 bits
    D = lambda k: None if c[k] is None else c[k].double()  # noqa: E731
    rms = lambda t: (t ** 2).mean(1, keepdim=True).sqrt()  # noqa: E731
    b6, e_b = D("block"), 0
    if c["share"] is not None:
        s6 = D("share") * (c["share_scale"].double()[:, None] if c["share_scale"] is not None else 1)
        b6 = b6 + s6
        e_b = U * (s6.abs() + b6.abs())
    n6, e_n = b6, e_b
    if post:
        k6 = 1 / torch.sqrt((b6 ** 2).mean(1, keepdim=True) + float(f32(eps[0])))
        w6 = D("post_weight") if c["post_weight"] is not None else 1.0
        n6 = b6 * w6 * k6
        e_n = e_b * abs(w6) * k6 + 4 * U * n6.abs()
        if c["share"] is not None:
            e_n = e_n + n6.abs() * rms(e_b) * k6
    g6 = (D("gate") if c["gate"] is not None else 1.0) * float(f32(bs))
    r6 = n6 * g6
    e_r = e_n * abs(g6) + 3 * U * r6.abs()
    if c["residual"] is not None:
        q6 = D("residual") * float(f32(rs))
        r6 = r6 + q6
        e_r = e_r + 2 * U * q6.abs()
    e_r = e_r + U * r6.abs()
    h = torch.finfo(dt).eps / 2
    tiny = torch.finfo(dt).smallest_normal * h
    near = lambda got, want, tol: bool(((got.double() - want).abs() <= tol * (1 + h) + h * want.abs() + tiny).all())  # noqa: E731
    if "residual_out" in out:
        assert near(out["residual_out"], r6, e_r)
    k6 = 1 / torch.sqrt((r6 ** 2).mean(1, keepdim=True) + float(f32(eps[1])))
    w6 = D("weight") if c["weight"] is not None else 1.0
    y6 = r6 * w6 * k6
    e_y = e_r * abs(w6) * k6 + y6.abs() * (rms(e_r) * k6 + 54 * U)
    if "y" in out:
        assert near(out["y"], y6, e_y)
    if quant == "none":
        return
    a6 = y6.view(T, -1, group or H).abs().amax(-1)
    e_a = e_y.view(T, -1, group or H).amax(-1)
    top = 127 if quant == "int8" else 448
    e6 = float(f32(eps[2]))
    s = out["q_scale"].view(T, -1).double()
    assert bool(((s - torch.clamp(a6, min=e6) / top).abs() <= (e_a + 2 * U * torch.clamp(a6, min=e6)) / top * (1 + U)).all())
    wq, _ = codes_of(p, k6.float(), quant, group, eps[2])
    floored = ((s * top) <= e6 * (1 + 4 * U)).any(1)  # their codes go by the second norm's sum: one step of a code
    assert same_codes(out["q"][~floored], wq[~floored])
    assert bool(((out["q"][floored].float() - wq[floored].float()).abs() <= 1).all())


JSHAPES = [(1, 1), (1, 7), (3, 8), (2, 63), (6, 512), (5, 520), (7, 513), (1, 4096), (9, 2048), (4, 2055), (3, 4100), (2, 8192),
           (5, 7168), (3, 9001), (1, 16384), (2, 16381), (600, 5003), (530, 8192), (520, 16384), (513, 12001), (1000, 640),
           (2100, 100)]


@pytest.mark.parametrize("T,H", JSHAPES)
@pytest.mark.parametrize("dt,wt", [(BF, BF), (BF, F32), (FP, FP), (FP, F32), (F32, F32)],
                         ids=["bf16", "bf16_w32", "fp16", "fp16_w32", "fp32"])
def test_join_shapes(T, H, dt, wt):
    c = inputs(T, H, dt, wt)
    check_join(c, join(c, True), True)
    c = inputs(T, H, dt, wt, post=False, gate=None, seed=1)
    check_join(c, join(c, False, "e4m3"), False, "e4m3")


OPTIONS = [dict(share=False), dict(ss=False), dict(residual=False), dict(pw=False), dict(gate="token"), dict(gate=None),
           dict(weight=False), dict(share=False, residual=False, gate=None, weight=False, pw=False)]


@pytest.mark.parametrize("H", [96, 1000, 4096, 5003])
@pytest.mark.parametrize("over", OPTIONS, ids=lambda o: "_".join(f"{k}_{v}" for k, v in o.items()))
def test_join_options(H, over):
    for post in (False, True):
        c = inputs(11, H, BF, F32, post=post, seed=3, **over)
        check_join(c, join(c, post), post)
        check_join(c, join(c, post, "none", want=("y",)), post, "none")
        out = join(c, post, "none", want=("residual_out",))
        check_join(c, out, post, "none")
        check_join(c, join(c, post, "int8", want=()), post, "int8")


@pytest.mark.parametrize("T,H,group", [(1, 64, 64), (5, 640, 128), (2, 2048, 256), (9, 4096, 128), (3, 7168, 64),
                                       (2, 16384, 256), (520, 4608, 128), (515, 8448, 256)])
def test_join_groups(T, H, group):
    for quant in ("int8", "e4m3"):
        c = inputs(T, H, BF, BF, seed=7)
        check_join(c, join(c, True, quant, group), True, quant, group)


@pytest.mark.parametrize("H", [64, 501, 4096])
def test_join_floor_and_zero_rows(H):
    c = inputs(5, H, F32, F32, post=False, gate=None, share=False)
    c["block"][0] = 0
    c["residual"][0] = 0
    c["block"][1] *= 1e-12
    c["residual"][1] *= 1e-12
    c["block"][2] *= 1e-8
    c["residual"][2] *= 1e-8
    eps = (1e-5, 1e-6, 1e-3)
    out = join(c, False, eps=eps)
    check_join(c, out, False, eps=eps)
    assert bool((out["q"][0] == 0).all())
    for quant, top in (("int8", 127.0), ("e4m3", 448.0)):
        s = join(c, False, quant, eps=eps)["q_scale"]
        assert float(s[0]) == float(f32(1e-3) * (1 / f32(top)))


@pytest.mark.parametrize("T,H", [(7, 513), (40, 4096), (600, 5003), (3, 9000)])
def test_join_in_place(T, H):
    """residual_out and y where an input was: the same bits."""
    for ro, y in (("residual", None), ("block", "share"), ("share", "block"), ("residual", "block"), (None, "residual")):
        c = inputs(T, H, BF, BF, seed=13)
        want = join(c, True)
        mine = {k: v if v is None else v.clone() for k, v in c.items()}
        got = join(mine, True, want=tuple(k for k, v in (("residual_out", ro), ("y", y)) if v is None),
                   over={k: mine[v] for k, v in (("residual_out", ro), ("y", y)) if v})
        for k in want:
            assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), (k, ro, y)


def test_join_is_the_norm_where_the_branch_is_nothing():
    """Without a branch it is moe_w8a8_norm_quant of x + residual: the stream
    and the codes bit for bit; y and the scales but for the order of the sum of
    squares, each side's rstd off by at most 54 u (see above): 108 u, after
    which two roundings to bf16 are at most one step (2 eps / 2) apart."""
    for T, H in ((5, 512), (9, 5003), (3, 16384)):
        c = inputs(T, H, BF, BF, share=False, post=False, gate=None, seed=2)
        got = join(c, False, rs=1.0, bs=1.0, eps=(1e-5, 1e-6, EPS))
        want = {k: torch.empty_like(v) for k, v in got.items()}
        moe.moe_w8a8_norm_quant(moe.make_norm_dims(T, H), c["block"], c["weight"], residual=c["residual"], **want)
        for k in ("residual_out", "q"):
            assert torch.equal(got[k].view(torch.uint8), want[k].view(torch.uint8)), k
        for k, step in (("y", torch.finfo(BF).eps), ("q_scale", 0)):
            a, b = got[k].double(), want[k].double()
            assert bool(((a - b).abs() <= (108 * U + step) * torch.maximum(a.abs(), b.abs())).all()), k


def test_join_other_rows_of_a_row_that_is_not_finite():
    c = inputs(9, 700, BF, F32, seed=4)
    want = join(c, True)
    c["block"][2, 5], c["share"][5, 1], c["residual"][7, 699] = float("nan"), float("inf"), float("-inf")
    got = join(c, True)
    rows = [0, 1, 3, 4, 6, 8]
    for k in want:
        assert torch.equal(got[k][rows].view(torch.uint8), want[k][rows].view(torch.uint8)), k


def test_a_row_is_the_same_in_every_batch():
    """Codes do not depend on the launch that a batch size takes."""
    for H in (4200, 9000):
        c = inputs(700, H, BF, F32, seed=5)
        whole = join(c, True)
        part = {k: v if v is None or v.shape[0] != 700 else v[:100].contiguous() for k, v in c.items()}
        few = join(part, True)
        assert torch.equal(whole["q"][:100], few["q"]) and torch.equal(whole["residual_out"][:100], few["residual_out"])
        x = c["block"]
        assert torch.equal(quantise(x)[0][:100], quantise(x[:100].contiguous())[0])


def test_rows_captured():
    c = inputs(33, 4104, BF, BF, seed=6)
    d = moe.make_join_norm_dims(33, 4104, post_norm=True, gate_rows=1)
    qd = moe.make_quant_dims(33, 4104)
    out = dict(residual_out=torch.empty_like(c["block"]), y=torch.empty_like(c["block"]),
               q=torch.empty(33, 4104, dtype=torch.int8, device="cuda"), q_scale=torch.empty(33, device="cuda"))
    q2, s2 = torch.empty_like(out["q"]), torch.empty_like(out["q_scale"])

    def step():
        moe.moe_w8a8_join_norm(d, **c, **out)
        moe.moe_w8a8_quant(qd, out["y"], q=q2, q_scale=s2)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        n = inputs(33, 4104, BF, BF, seed=50 + seed)
        for k in c:
            c[k].copy_(n[k])
        graph.replay()
        torch.cuda.synchronize()
        check_join(c, out, True, rs=1.0, bs=1.0, eps=(1e-6, 1e-6, EPS))
        check_quant(out["y"], q2, s2, "int8", 0, None)
        eager = [v.clone() for v in out.values()]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(eager, out.values()))


def test_no_token():
    x = torch.empty(0, 64, dtype=BF, device="cuda")
    q, s = moe.moe_w8a8_quant(moe.make_quant_dims(0, 64), x)
    assert q.shape == (0, 64) and s.shape == (0,)
    moe.moe_w8a8_join_norm(moe.make_join_norm_dims(0, 64), x, y=x)


@pytest.mark.parametrize("H", [4200, 5003, 9000])
@pytest.mark.parametrize("post", [False, True])
def test_every_output_is_the_same_in_every_batch(H, post):
    """fp32, so that the last bit of 1 / sqrt of either mean square shows in y
    and in q_scale; a third of the rows lie under the floor, and their codes go
    by that root too. 100 and 700 rows take unlike workgroups."""
    c = inputs(700, H, F32, F32, post=post, gate=None if post else "token", seed=23)
    for k in ("block", "share", "residual"):
        c[k][::3] *= 1e-8
    part = {k: v if v is None or v.shape[0] != 700 else v[:100].contiguous() for k, v in c.items()}
    for quant, group in (("int8", 0), ("e4m3", 0)):
        eps = (1e-5, 1e-6, 1e-3)
        whole, few = join(c, post, quant, group, eps=eps), join(part, post, quant, group, eps=eps)
        for k in whole:
            assert torch.equal(whole[k][:100].view(torch.uint8), few[k].view(torch.uint8)), (k, quant)


@pytest.mark.parametrize("T,H", [(5, 512), (33, 5003), (600, 4096), (520, 16384), (3, 16381)])
def test_the_norm_of_the_stream_is_rounded_once(T, H):
    """r = block exactly. In units of u = 2^-24: y is a product by the weight,
    one by 1 / sqrt(...) and that root, each rounded once: 3 u. q_scale is the
    largest of these times 1 / Q, one product and one constant more: 5 u. (And
    what is summed in 64 bits, under 2^-40.)"""
    c = inputs(T, H, F32, F32, share=False, residual=False, post=False, gate=None, seed=29)
    out = join(c, False, rs=1.0, bs=1.0)
    r, w = c["block"].double(), c["weight"].double()
    y = r * w / torch.sqrt((r * r).mean(1, keepdim=True) + float(f32(1e-6)))
    more = 1 + 2.0 ** -16  # products of the bounds
    assert bool(((out["y"].double() - y).abs() <= 3 * U * more * y.abs()).all())
    s = y.abs().amax(1) / 127
    assert bool(((out["q_scale"].double() - s).abs() <= 5 * U * more * s).all())


@pytest.mark.parametrize("T,H,group", [(4200, 4096, 128), (4001, 5003, 0), (40000, 500, 0), (40000, 448, 64), (1100, 16381, 0),
                                       (1030, 16384, 256)])
@pytest.mark.parametrize("dt", [BF, FP, F32], ids=NAMES.get)
def test_rows_streamed(T, H, group, dt):
    """16 MB of codes or more."""
    assert T * H >= 16 << 20
    g = torch.Generator("cuda").manual_seed(T + H)
    x = (torch.randn(T, H, generator=g, device="cuda") * 3).to(dt)
    sm = 0.5 + torch.rand(H, generator=g, device="cuda")
    check_quant(x, *quantise(x, "int8", group, sm), "int8", group, sm)
    check_quant(x, *quantise(x, "e4m3", group), "e4m3", group, None)


@pytest.mark.parametrize("T,H,group", [(1100, 5003, 0), (1030, 8192, 128), (20000, 500, 0), (400, 16381, 0)])
@pytest.mark.parametrize("dt", [BF, FP, F32], ids=NAMES.get)
def test_join_streamed(T, H, group, dt):
    for quant, gate in (("int8", "row"), ("e4m3", "token")):
        c = inputs(T, H, dt, F32, gate=gate, seed=31)
        check_join(c, join(c, True, quant, group), True, quant, group)
