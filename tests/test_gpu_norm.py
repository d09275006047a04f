"""moe_w8a8_norm_quant on the GPU, against the formula in 64 bits and, for the
codes, against the same IEEE operations on the CPU.

Tolerances. u = 2^-24, h = half a step of the output type (eps / 2).
  residual_out: the fp32 sum and its rounding: h + u relative.
  rstd: the squares are positive, so a sum with at most 80 additions in a row
    (64 in a thread, 6 in a wave, at most 16 over waves; fewer elements in a
    thread where more waves share a row) is off by 80 u at most, the squares
    by 3 u, the division, the eps and the root by 4 u more; the root halves
    what goes in: 46 u.
  y: rstd, two products, the sum: 50 u, and h.  scale: 50 u.
  codes: equal to those of the same fp32 operations; against 64 bits, off by
    half a step and Q * 6 u (products and 1 / max). A row under the amax floor
    is scaled by rstd: Q * 60 u."""
import numpy as np
import pytest
import torch

import moe_expert_ffn_route_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
Q8, E4, NO = moe.MOE_QUANT_INT8, moe.MOE_QUANT_E4M3, moe.MOE_QUANT_NONE


def make(T, H, dt, wdt, residual, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(dt)
    res = (torch.randn(T, H, generator=g) * torch.exp(torch.randn(H, generator=g))).to(dt) if residual else None
    w = None if wdt is None else (0.5 + torch.rand(H, generator=g)).to(wdt)
    return x, res, w


def run(x, res, w, quant, group, want_y=True, eps=1e-6, amax_eps=1e-6, pad=3):
    """The call with every output behind and before guard rows."""
    T, H = x.shape
    d = moe.make_norm_dims(T, H, dtype=x.dtype, weight_dtype=None if w is None else w.dtype, quant=quant,
                           quant_group=group, rms_eps=eps, amax_eps=amax_eps)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    ns = H // group if group else 1
    full = lambda n, dt: torch.full((T * n + pad * 16,), 7, dtype=dt, device="cuda")  # noqa: E731
    bufs = {}
    if res is not None:
        bufs["residual_out"] = full(H, x.dtype)
    if want_y:
        bufs["y"] = full(H, x.dtype)
    if quant != NO:
        bufs["q"] = full(H, torch.uint8)
        bufs["q_scale"] = full(ns, torch.float32)
    code_t = torch.int8 if quant == Q8 else torch.float8_e4m3fn
    views = {k: v[:T * (ns if k == "q_scale" else H)] for k, v in bufs.items()}
    if quant != NO:
        views["q"] = views["q"].view(code_t)
    moe.moe_w8a8_norm_quant(d, cu(x), cu(w), residual=cu(res), **views)
    torch.cuda.synchronize()
    for k, v in bufs.items():
        n = T * (ns if k == "q_scale" else H)
        assert bool((v[n:] == 7).all()), f"{k}: written past its end"
    out = {k: v.cpu().view(T, -1) for k, v in views.items()}
    return out


def check(x, res, w, quant, group, out, eps=1e-6, amax_eps=1e-6):
    T, H = x.shape
    h = torch.finfo(x.dtype).eps / 2
    tiny = torch.finfo(x.dtype).smallest_normal * h
    r = x.double() + (res.double() if res is not None else 0)
    rstd = 1 / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
    y = r * (w.double() if w is not None else 1) * rstd
    if "residual_out" in out:
        assert bool(((out["residual_out"].double() - r).abs() <= (h + 2 * U) * r.abs() + tiny).all())
    if "y" in out:
        assert bool(((out["y"].double() - y).abs() <= (h + 52 * U) * y.abs() + tiny).all())
    if quant == NO:
        return
    Q = 127.0 if quant == Q8 else 448.0
    n = group or H
    yg = y.view(T, H // n, n)
    a = yg.abs().amax(-1)
    floored = a < amax_eps
    s = torch.clamp(a, min=amax_eps) / Q
    assert bool(((out["q_scale"].double() - s).abs() <= 54 * U * s).all())
    got = out["q"].float().double().view(T, H // n, n) if quant == E4 else out["q"].double().view(T, H // n, n)
    v = yg / s[..., None]
    if quant == Q8:
        slack = torch.where(floored[..., None], 60.0 * Q * U, 6.0 * Q * U)
        assert bool(((got - v).abs() <= 0.5 + slack).all())
    # the same fp32 operations on the CPU
    p = x.float() + (res.float() if res is not None else 0.0)
    if w is not None:
        p = p * w.float()
    pg = p.view(T, H // n, n)
    inv = 1.0 / pg.abs().amax(-1, keepdim=True)
    t = (pg * Q) * inv
    want = torch.round(t).clamp(-127, 127) if quant == Q8 else t.to(torch.float8_e4m3fn).float()
    same = (got.float() == want) | floored[..., None]
    assert bool(same.all()), f"{int((~same).sum())} codes differ"


SIZES = [(1, 1), (3, 2), (2, 7), (5, 8), (1, 9), (4, 63), (3, 64), (2, 65), (7, 200), (1, 512), (5, 1000), (3, 2047),
         (2, 2048), (3, 2049), (1, 4096), (64, 4096), (3, 4097), (300, 4096), (5, 5003), (2, 7168), (600, 7168), (3, 8192), (2, 12345),
         (1, 16383), (2, 16384), (300, 16384), (1100, 640)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("dt", [BF, FP, F32], ids=["bf16", "fp16", "fp32"])
def test_sizes(T, H, dt):
    for i, (quant, residual, wdt) in enumerate([(Q8, True, dt), (E4, False, F32), (NO, True, None)]):
        x, res, w = make(T, H, dt, wdt, residual, seed=H * 10 + i)
        check(x, res, w, quant, 0, run(x, res, w, quant, 0))


@pytest.mark.parametrize("group", [64, 128, 256])
@pytest.mark.parametrize("T,H", [(1, 256), (3, 768), (2, 4096), (70, 7168), (2, 16384), (400, 2304)])
@pytest.mark.parametrize("quant", [Q8, E4], ids=["int8", "e4m3"])
def test_groups(T, H, group, quant):
    x, res, w = make(T, H, BF, BF, True, seed=H + group)
    x[0, :group] = 0  # one group under the floor beside ordinary ones
    res[0, :group] = 0
    out = run(x, res, w, quant, group, want_y=False)
    assert float(out["q"].float()[0, :group].abs().max()) == 0
    check(x, res, w, quant, group, out)


@pytest.mark.parametrize("quant", [Q8, E4], ids=["int8", "e4m3"])
def test_floor_rows(quant):
    x, _, w = make(6, 1000, F32, F32, False, seed=3)
    x[1] = 0
    x[2] *= 1e-12  # y about 1e-9 at most: under the floor of 1e-6
    x[3] *= 1e-25
    x[4] *= 1e5
    out = run(x, None, w, quant, 0)
    check(x, None, w, quant, 0, out)
    Q = np.float32(127 if quant == Q8 else 448)
    floor = np.float32(1e-6) * (np.float32(1) / Q)
    for t in (1, 3):
        assert float(out["q"].float()[t].abs().max()) == 0 and out["q_scale"][t, 0].item() == floor
    # the smallest floors that are accepted: nothing overflows on the way
    out = run(x, None, w, quant, 0, eps=1e-30, amax_eps=1e-20)
    assert bool(torch.isfinite(out["y"]).all()) and bool(torch.isfinite(out["q_scale"]).all())
    assert float(out["q"].float()[1].abs().max()) == 0
    check(x, None, w, quant, 0, out, eps=1e-30, amax_eps=1e-20)


def test_ties_round_to_even():
    # max 127: t = v exactly, so x.5 is a tie
    v = torch.tensor([127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5, -126.5])
    out = run(v.view(1, -1), None, None, Q8, 0)
    t = (v * 127) * (torch.tensor(1.0) / 127)
    assert out["q"][0].tolist() == torch.round(t).to(torch.int8).tolist()


def test_codes_do_not_depend_on_the_norm():
    x, res, w = make(9, 4096, BF, BF, True, seed=11)
    a, b = run(x, res, w, Q8, 0), run(x, res, w, Q8, 0, eps=100.0)
    assert torch.equal(a["q"], b["q"]) and not torch.equal(a["q_scale"], b["q_scale"])


@pytest.mark.parametrize("T,H", [(3, 4096), (40, 5003), (500, 4096), (3, 16384)])
def test_in_place(T, H):
    x, res, w = make(T, H, BF, BF, True, seed=5)
    ref = run(x, res, w, Q8, 0)
    d = moe.make_norm_dims(T, H)
    for where in ((0, 1), (1, 0), (0, None), (None, 1)):
        xs, rs = x.cuda(), res.cuda()
        y = (xs, rs)[where[0]] if where[0] is not None else torch.empty_like(xs)
        ro = (xs, rs)[where[1]] if where[1] is not None else torch.empty_like(xs)
        q, s = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        moe.moe_w8a8_norm_quant(d, xs, w.cuda(), residual=rs, residual_out=ro, y=y, q=q, q_scale=s)
        assert torch.equal(y.cpu(), ref["y"]) and torch.equal(ro.cpu(), ref["residual_out"])
        assert torch.equal(q.cpu(), ref["q"]) and torch.equal(s.cpu().view(-1, 1), ref["q_scale"])


@pytest.mark.parametrize("T", [5, 700])
def test_non_finite_row_leaves_the_others(T):
    x, res, w = make(T, 4096, BF, BF, True, seed=6)
    ref = run(x, res, w, Q8, 0)
    bad = x.clone()
    bad[2, 17], bad[3, 0], bad[4, 4095] = float("nan"), float("inf"), -float("inf")
    out = run(bad, res, w, Q8, 0)
    rows = [t for t in range(T) if t not in (2, 3, 4)]
    for k in ref:
        assert torch.equal(out[k][rows], ref[k][rows]), k


def test_row_alone_equals_row_in_a_batch():
    # the split of a row over threads goes by the batch: values may differ in
    # rstd's last bits, codes may not
    x, res, w = make(900, 4096, BF, BF, True, seed=8)
    a, b = run(x, res, w, Q8, 0), run(x[41:42], res[41:42], w, Q8, 0)
    assert torch.equal(a["q"][41:42], b["q"])


def test_zero_tokens_and_side_stream():
    d = moe.make_norm_dims(0, 64)
    e = torch.empty(0, 64, dtype=BF, device="cuda")
    moe.moe_w8a8_norm_quant(d, e, y=e.clone(), q=torch.empty(0, 64, dtype=torch.int8, device="cuda"),
                            q_scale=torch.empty(0, device="cuda"))
    x, res, w = make(33, 4096, BF, BF, True, seed=9)
    ref = run(x, res, w, Q8, 0)
    st = torch.cuda.Stream()
    xs, rs, ws = x.cuda(), res.cuda(), w.cuda()
    y, q, s = torch.empty_like(xs), torch.empty(33, 4096, dtype=torch.int8, device="cuda"), torch.empty(33, device="cuda")
    torch.cuda.synchronize()
    moe.moe_w8a8_norm_quant(moe.make_norm_dims(33, 4096), xs, ws, residual=rs, y=y, q=q, q_scale=s, stream=st)
    st.synchronize()
    assert torch.equal(y.cpu(), ref["y"]) and torch.equal(q.cpu(), ref["q"])


def test_offsets_past_32_bits():
    T, H = 65536, 16384  # 2^30 elements, 4 GiB in, 1 GiB of codes
    x = torch.ones(T, H, dtype=F32, device="cuda")
    x[-1] = torch.randn(H, generator=torch.Generator().manual_seed(1)).cuda()
    q, s = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
    moe.moe_w8a8_norm_quant(moe.make_norm_dims(T, H, dtype=F32), x, q=q, q_scale=s)
    ref = run(x[-1:].cpu(), None, None, Q8, 0)
    assert torch.equal(q[-1:].cpu(), ref["q"]) and bool((q[:-1:997] == 127).all())


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("T,H", [(4, 1024), (600, 5120)])
def test_e4m3_codes_against_64_bits(T, H, group):
    """Rows over the amax floor and under it. The value that is rounded is off by at most 60 u, so its code lies between
    the codes of the 64-bit value moved by 64 u (one more rounding, to fp32) either way."""
    x, res, w = make(T, H, BF, BF, True, seed=61)
    eps = 100.0 if group else 1e4  # amax of groups on both sides of 1, of rows under it
    for amax_eps in (1e-6, 1.0):
        out = run(x, res, w, E4, group, eps=eps, amax_eps=amax_eps)
        r = x.double() + res.double()
        y = r * w.double() / torch.sqrt((r * r).mean(1, keepdim=True) + eps)
        n = group or H
        a = y.view(T, H // n, n).abs().amax(-1, keepdim=True)
        assert bool((a < amax_eps).any()) == (amax_eps == 1.0) and (amax_eps < 1 or group == 0 or bool((a > 1).any()))
        v = y.view(T, H // n, n) / (torch.clamp(a, min=amax_eps) / 448)
        code = lambda f: (v * (1 + f * v.sign() * 64 * U)).float().to(torch.float8_e4m3fn).float()  # noqa: E731
        got = out["q"].float().view(T, H // n, n)
        assert float(got.abs().max()) > 8
        assert bool(((got >= code(-1)) & (got <= code(1))).all())
