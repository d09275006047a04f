"""moe_w8a8_gate on the GPU against the formula in 64 bits on the CPU.

Ids are equal: the inputs are random, so two choice values lie within the
1e-14 that a 64-bit sum may be off only by design (equal rows, checked for the
lowest id).

Weights. Types that are not both bf16, both fp16, or bf16 x and fp32 weights:
everything before the
rounding to fp32 is in 64 bits, so 2^-24 relative, and 1e-10 for the sums and
exp. Both 16-bit: a logit is a sum of fp32 sums of at most 128 exact products, each
addition off by at most 2^-23 of the magnitudes so far, so off by at most
B = 128 * 2^-23 * sum |x w|. A score moves by at most B relative (softmax 2 B,
with its sum), the sum of the chosen ones by as much: 4 B, and 2^-24.
That is with all roundings agreeing. As they do not, the 2-norm is held to
4e-6: H additions, each off by 2^-24 of a partial sum that for these inputs is
at most about 6 * 1.5 * sqrt(128 / H), add up to sqrt(H) * 2^-24 * 102 /
sqrt(H) = 6e-6 in the worst token and under half of it over all."""
import pytest
import torch

import moe_expert_ffn_route_amd as moe

pytestmark = pytest.mark.gpu
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32
SOFTMAX, SIGMOID, SQRTSP = moe.MOE_SCORE_SOFTMAX, moe.MOE_SCORE_SIGMOID, moe.MOE_SCORE_SQRT_SOFTPLUS


def make(T, H, E, dt=BF, wdt=BF, bias=False, seed=0):
    g = torch.Generator().manual_seed(seed + 31 * T + 7 * H + E)
    x = torch.randn(T, H, generator=g).to(dt)
    w = (torch.randn(E, H, generator=g) * (1.5 / H ** 0.5)).to(wdt)
    return x, w, torch.randn(E, generator=g) * 0.05 if bias else None


def formula(x, w, b, K, score, normalize, route_scale):
    l = x.double() @ w.double().t()
    s = {SOFTMAX: lambda: torch.softmax(l, 1), SIGMOID: lambda: torch.sigmoid(l),
         SQRTSP: lambda: (torch.clamp(l, min=0) + torch.log1p(torch.exp(-l.abs()))).sqrt()}[score]()
    c = l if b is None else s + b.double()
    ids = torch.sort(c, dim=1, descending=True, stable=True)[1][:, :K]
    v = s.gather(1, ids)
    if normalize:
        v = v / v.sum(1, keepdim=True)
    return ids, v * route_scale


def run(x, w, b, K, score=SOFTMAX, normalize=True, route_scale=1.0, stream=None):
    d = moe.make_gate_dims(x.shape[0], x.shape[1], w.shape[0], K, score=score, normalize=normalize,
                           route_scale=route_scale, dtype=x.dtype, weight_dtype=w.dtype)
    n = x.shape[0] * K
    ids = torch.full((n + 64,), -7, dtype=torch.int32, device="cuda")
    sc = torch.full((n + 64,), -7.0, device="cuda")
    ws = torch.full((moe.moe_w8a8_gate_workspace_size(d) + 256,), 0xA5, dtype=torch.uint8, device="cuda")
    need = ws.numel() - 256
    moe.moe_w8a8_gate(d, x.cuda(), w.cuda(), bias=None if b is None else b.cuda(), expert_ids=ids[:n],
                      expert_scales=sc[:n], workspace=ws[:need], stream=stream)
    torch.cuda.synchronize()
    assert bool((ids[n:] == -7).all()) and bool((sc[n:] == -7).all()) and bool((ws[need:] == 0xA5).all())
    return ids[:n].view(-1, K).cpu(), sc[:n].view(-1, K).cpu()


def check(got, want, x, w):
    assert torch.equal(got[0].long(), want[0])
    err = (got[1].double() - want[1]).abs()
    tol = torch.full((x.shape[0], 1), 2.0 ** -24 + 1e-10, dtype=torch.float64)
    if (x.dtype == w.dtype and x.dtype != F32) or (x.dtype == BF and w.dtype == F32):
        tol += 4 * 2.0 ** -16 * (x.double().abs() @ w.double().abs().t()).amax(1, keepdim=True)
    assert bool((err <= tol * want[1].abs() + 1e-45).all())
    assert float(err.norm()) <= 4e-6 * float(want[1].norm())


SIZES = [(1, 1, 1, 1), (1, 4096, 256, 8), (8, 4096, 256, 8), (3, 7, 5, 5), (2, 8, 64, 16), (5, 130, 65, 6), (16, 1000, 128, 4),
         (17, 2501, 72, 6), (33, 512, 256, 8), (64, 7168, 384, 8), (100, 640, 1024, 16), (129, 1024, 257, 9),
         (300, 2048, 160, 6), (509, 2501, 72, 6), (1000, 333, 30, 3), (1, 16384, 1024, 16), (2, 16383, 511, 2), (700, 4096, 256, 8),
         (250, 4095, 255, 8), (1100, 2501, 130, 6), (40, 511, 70, 4), (7, 600, 512, 16), (900, 2048, 500, 8)]


@pytest.mark.parametrize("T,H,E,K", SIZES)
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID, SQRTSP], ids=["softmax", "sigmoid", "sqrtsoftplus"])
def test_sizes(T, H, E, K, score):
    for bias in (False, True):
        x, w, b = make(T, H, E, bias=bias)
        check(run(x, w, b, K, score, normalize=bias or K > 3, route_scale=2.5),
              formula(x, w, b, K, score, bias or K > 3, 2.5), x, w)


@pytest.mark.parametrize("dt,wdt", [(BF, F32), (FP, FP), (FP, BF), (FP, F32), (F32, BF), (F32, F32)], ids=str)
@pytest.mark.parametrize("T,H,E,K", [(1, 4096, 256, 8), (7, 1001, 40, 4), (64, 2048, 256, 8), (200, 515, 130, 8), (600, 1024, 64, 6),
                                     (1100, 2501, 130, 6)])
def test_types(T, H, E, K, dt, wdt):
    x, w, b = make(T, H, E, dt, wdt, bias=True)
    check(run(x, w, b, K, SIGMOID), formula(x, w, b, K, SIGMOID, True, 1.0), x, w)


@pytest.mark.parametrize("T", [3, 40, 600, 1400])
def test_ties_go_to_the_lowest_id(T):
    x, w, _ = make(T, 1024, 200)
    w[60:120] = w[0:60]     # every expert of 60..119 ties with one of 0..59
    w[199] = w[3]
    l = x.double() @ w.double().t()
    l[:, 60:120], l[:, 199] = l[:, 0:60], l[:, 3]  # whatever order the library sums each column in
    want = torch.sort(l, dim=1, descending=True, stable=True)[1][:, :8]
    ids, sc = run(x, w, None, 8)
    assert torch.equal(ids.long(), want)
    check((ids, sc), (want, torch.softmax(l.gather(1, want), 1)), x, w)
    zero = torch.zeros_like(w)
    ids, sc = run(x, zero, None, 8)
    assert ids.tolist() == [list(range(8))] * T and bool((sc == 0.125).all())


@pytest.mark.parametrize("T", [5, 200, 1500])
@pytest.mark.parametrize("keep", [None, 0, 3, 7], ids=lambda k: "all" if k is None else f"element{k}")
@pytest.mark.parametrize("bias", [False, True], ids=["logit", "bias"])
@pytest.mark.parametrize("dt", [BF, FP], ids=["bf16", "fp16"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID, SQRTSP])
def test_close_logits_are_told_apart(T, bias, dt, score, keep):
    """Experts in pairs and triples whose rows differ in one last bit of one
    element: logits that fp32 sums cannot order. `keep`: only that one of every
    eight elements of x is not zero, so that a bound that misses it is zero."""
    x, w, b = make(T, 2048, 96, dt, dt, bias=bias, seed=17)
    if keep is not None:
        x = torch.where(torch.arange(2048) % 8 == keep, 3 * x.float(), torch.zeros(1)).to(dt)
    step = 2.0 ** -8 if dt == BF else 2.0 ** -11
    for e in range(0, 96, 3):
        w[e + 1], w[e + 2] = w[e], w[e]
        k = 7 * e + 5 if keep is None else 8 * e + keep
        w[e + 1, k], w[e + 2, k] = w[e, k] * (1 + 2 * step), w[e, k] * (1 - 4 * step)
        if bias:
            b[e + 1] = b[e + 2] = b[e]
    w[:, 1000:] *= 16  # sums whose terms dwarf the difference
    l = x.double() @ w.double().t()
    gaps = torch.sort(l, dim=1)[0].diff(dim=1)
    mag = (x.double().abs() @ w.double().abs().t()).amax(1, keepdim=True)
    assert float(gaps.min()) < 2.0 ** -23 * float(mag.max()) and float(gaps.min()) > 0  # under fp32's last bit; no ties
    ids, sc = run(x, w, b, 9, score)
    want, v = formula(x, w, b, 9, score, True, 1.0)
    # A softmax share of 1e-18 beside a bias of 0.05 is under the bias' last
    # bit: there the 64-bit sums themselves, off by 2048 * 2^-53 of the
    # magnitudes in a logit (relative to the share) and by 4 * 2^-53 of the
    # value, leave the order open. Everywhere else ids are equal.
    s64 = {SOFTMAX: lambda: torch.softmax(l, 1), SIGMOID: lambda: torch.sigmoid(l),
           SQRTSP: lambda: (torch.clamp(l, min=0) + torch.log1p(torch.exp(-l.abs()))).sqrt()}[score]()
    c = l if b is None else s64 + b.double()
    slope = 1.0 if b is None else 2 * s64.gather(1, want) if score == SOFTMAX else 0.34
    open_ = 2 * 2.0 ** -53 * (2048 * mag * slope + 4 * c.gather(1, want).abs())
    same = ids.long() == want
    assert bool((same | ((c.gather(1, ids.long()) - c.gather(1, want)).abs() <= open_)).all())
    if b is None:
        assert bool(same.all())
    check((want.int(), sc), (want, v), x, w)


@pytest.mark.parametrize("T", [7, 150, 3000])
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (FP, FP), (BF, F32)], ids=["bf16", "fp16", "bf16-fp32"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID, SQRTSP])
def test_large_biases(T, dt, wdt, score):
    """score + bias is rounded at the bias' size: 64-bit values that tie there go to the lowest id."""
    x, w, b = make(T, 1500, 130, dt, wdt, bias=True, seed=5)
    for size in (1e3, 1e6):
        bb = (torch.randint(0, 3, (130,)).float() + 1) * size
        bb[7] = -float("inf")
        check(run(x, w, bb, 8, score), formula(x, w, bb, 8, score, True, 1.0), x, w)


@pytest.mark.parametrize("T", [7, 150])
def test_subnormal_and_tiny_inputs(T):
    x, w, _ = make(T, 1024, 64, FP, FP, seed=6)
    x = (x.float() * 2.0 ** -20).to(FP)  # fp16 subnormals
    assert 0 < float(x.abs().max()) < torch.finfo(FP).smallest_normal
    check(run(x, w, None, 6), formula(x, w, None, 6, SOFTMAX, True, 1.0), x, w)
    x, w, _ = make(T, 1024, 64, BF, F32, seed=7)
    x = x.repeat(1 + 60 * (T > 100), 8)
    w = torch.cat([w.roll(i, 1) for i in range(8)], 1)  # 9150 x 64 x 8192 products: the split
    check(run(x, (w * 2.0 ** -60), None, 6), formula(x, w * 2.0 ** -60, None, 6, SOFTMAX, True, 1.0), x, w * 2.0 ** -60)
    check(run((x.float() * 2.0 ** -50).to(BF), w, None, 6), formula((x.float() * 2.0 ** -50).to(BF), w, None, 6, SOFTMAX, True, 1.0), x, w)


@pytest.mark.parametrize("T", [7, 150, 1500])
@pytest.mark.parametrize("dt,wdt,xs,ws", [(BF, BF, -82, 60), (BF, BF, 56, -76), (FP, FP, -20, 4), (BF, F32, -82, 60)],
                         ids=["bf16-x", "bf16-w", "fp16", "fp32-w"])
def test_close_logits_of_inputs_whose_squares_vanish(T, dt, wdt, xs, ws):
    """Pairs of experts with the same products in another order, and one small
    element's last bit more: fp32 sums order them by their roundings. The
    elements are fp16 subnormals, or so small that their squares are not even
    fp32 subnormals: the bound still has to see them."""
    g = torch.Generator().manual_seed(23 + T)
    x, w, _ = make(T, 2048, 96, dt, wdt, seed=23)
    x, w = (x.float() * 2.0 ** xs).to(dt), (w.float() * 2.0 ** ws).to(wdt)
    x[x == 0] = 2.0 ** (xs - 4)  # a zero would tie
    x = x[:, :16].repeat(1 if wdt == dt else 1 + 2900 // T, 128)  # fp32 w: products enough for the split
    for e in range(0, 96, 2):
        w[e, 5] *= {BF: 2.0 ** -14, FP: 2.0 ** -7, F32: 1.0}[wdt]
        w[e + 1] = w[e].view(128, 16)[torch.randperm(128, generator=g)].view(-1)
        w[e, 5] *= 1 + {BF: 2.0 ** -7, FP: 2.0 ** -10, F32: 2.0 ** -23}[wdt]
    want, v = formula(x, w, None, 9, SIGMOID, True, 1.0)
    check(run(x, w, None, 9, SIGMOID), (want, v), x, w)


@pytest.mark.parametrize("T", [9, 130, 3000])
@pytest.mark.parametrize("bias", [False, True], ids=["logit", "bias"])
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (FP, FP), (BF, F32)], ids=["bf16", "fp16", "fp32-w"])
def test_padded_batch(T, dt, wdt, bias):
    """Rows of zeros (both signs) among others: every logit is 0, so the bias or the ids decide."""
    x, w, b = make(T, 2047, 90, dt, wdt, bias=bias, seed=29)
    x[T // 2:] = 0.0
    x[T // 2, ::3] = -0.0
    x[T - 1, 2046] = 2.0 ** -24  # not quite zero
    check(run(x, w, b, 7, SIGMOID), formula(x, w, b, 7, SIGMOID, True, 1.0), x, w)


@pytest.mark.parametrize("T", [60, 2900])
@pytest.mark.parametrize("bias", [False, True], ids=["logit", "bias"])
def test_fp32_weights_to_their_last_bit(T, bias):
    """bf16 x and fp32 weights whose rows differ in one last bit of 24: every part of the split counts."""
    x, w, b = make(T, 2048, 96, BF, F32, bias=bias, seed=21)
    for e in range(0, 96, 2):
        w[e + 1] = w[e]
        k = 5 * e + 3
        w[e + 1, k] = torch.nextafter(w[e, k], torch.tensor(9.0))
        if bias:
            b[e + 1] = b[e]
    l = x.double() @ w.double().t()
    assert float((l[:, 0::2] - l[:, 1::2]).abs().min()) > 0
    check(run(x, w, b, 10, SIGMOID), formula(x, w, b, 10, SIGMOID, True, 1.0), x, w)


def test_choice_between_values_that_fp32_sums_cannot_tell_apart():
    # logits of two experts that differ by 2^-40 of their size: large terms
    # that cancel, and one small one
    x = torch.ones(4, 2048, dtype=F32)
    w = torch.zeros(8, 2048, dtype=F32)
    w[:, 0::2], w[:, 1::2] = 1024.0, -1024.0
    w[5, 77] += 2.0 ** -13
    w[2, 1500] += 2.0 ** -12
    ids, _ = run(x, w, None, 3)
    assert ids.tolist() == [[2, 5, 0]] * 4


@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID, SQRTSP])
@pytest.mark.parametrize("T", [2, 300])
def test_excluded_experts_and_empty_places(score, T):
    x, w, b = make(T, 512, 64, bias=True)
    b[:] = -float("inf")
    b[[5, 9, 40]] = 0.01
    ids, sc = run(x, w, b, 6, score)
    want, v = formula(x, w, b, 3, score, True, 1.0)
    assert torch.equal(ids[:, :3].long(), want) and bool((ids[:, 3:] == -1).all()) and bool((sc[:, 3:] == 0).all())
    check((ids[:, :3], sc[:, :3]), (want, v), x, w)
    b[:] = -float("inf")
    ids, sc = run(x, w, b, 6, score)
    assert bool((ids == -1).all()) and bool((sc == 0).all())


@pytest.mark.parametrize("T", [6, 400])
def test_non_finite_token_leaves_the_others(T):
    x, w, b = make(T, 4096, 256, bias=True)
    ref = run(x, w, b, 8, SIGMOID)
    x[1, 5], x[4, 4000] = float("nan"), float("inf")
    ids, sc = run(x, w, b, 8, SIGMOID)
    rows = [t for t in range(T) if t not in (1, 4)]
    assert torch.equal(ids[rows], ref[0][rows]) and torch.equal(sc[rows], ref[1][rows])
    assert ids.min() >= -1 and ids.max() < 256
    assert bool((ids[1] == -1).all())  # every logit NaN: no expert


def test_extreme_logits():
    # scores that saturate: the choice without bias still goes by the logit
    x = torch.full((2, 64), 8.0)
    x[1] = -8.0
    w = torch.arange(1, 33, dtype=F32).view(32, 1).repeat(1, 64)
    for score in (SOFTMAX, SIGMOID, SQRTSP):
        ids, sc = run(x, w, None, 4, score)
        assert ids.tolist() == [[31, 30, 29, 28], [0, 1, 2, 3]]
        assert bool(torch.isfinite(sc).all())
    ids, sc = run(x, w, None, 4, SIGMOID, normalize=False)
    assert sc[0].tolist() == [1.0] * 4


def test_batch_does_not_change_a_token():
    x, w, b = make(700, 4096, 256, bias=True)
    ids, sc = run(x, w, b, 8, SQRTSP)
    for n in (1, 9, 40, 200):
        i2, s2 = run(x[:n], w, b, 8, SQRTSP)
        assert torch.equal(i2, ids[:n])
        # 64-bit sums, or fp32 sums of 64 products joined in 64 bits
        assert bool(((s2 - sc[:n]).abs() <= 2.0 ** -23 * sc[:n]).all())


def test_defaults_zero_tokens_and_side_stream():
    x, w, b = make(12, 1024, 64)
    want = run(x, w, None, 4)
    st = torch.cuda.Stream()
    d = moe.make_gate_dims(12, 1024, 64, 4)
    xs, ws = x.cuda(), w.cuda()
    torch.cuda.synchronize()
    ids, sc = torch.empty(12, 4, dtype=torch.int32, device="cuda"), torch.empty(12, 4, device="cuda")
    work = torch.empty(moe.moe_w8a8_gate_workspace_size(d), dtype=torch.uint8, device="cuda")
    moe.moe_w8a8_gate(d, xs, ws, expert_ids=ids, expert_scales=sc, workspace=work, stream=st)
    st.synchronize()
    assert torch.equal(ids.cpu(), want[0]) and torch.equal(sc.cpu(), want[1])
    ids, sc = moe.moe_w8a8_gate(d, xs, ws)
    assert torch.equal(ids.cpu(), want[0]) and torch.equal(sc.cpu(), want[1])
    ids, sc = moe.moe_w8a8_gate(moe.make_gate_dims(0, 1024, 64, 4), xs[:0], ws)
    assert ids.shape == (0, 4) and sc.shape == (0, 4)


def test_largest_batch():
    T, H, E = 65536, 64, 1024  # a workspace of 512 MiB
    x, w, _ = make(T, H, E, F32, F32, seed=3)
    ids, sc = run(x, w, None, 2)
    rows = torch.arange(0, T, 1021)
    want = formula(x[rows], w, None, 2, SOFTMAX, True, 1.0)
    check((ids[rows], sc[rows]), want, x[rows], w)


@pytest.mark.parametrize("T,dt,wdt", [(9, BF, BF), (300, BF, BF), (9, BF, F32), (600, BF, F32)], ids=str)
@pytest.mark.parametrize("sign", [-1, 0, 1], ids=["all-negative", "mixed", "all-positive"])
def test_finite_inputs_whose_fp32_sums_overflow(T, dt, wdt, sign):
    """Products of 2^130: the 64-bit logits are finite, sums in fp32 would be infinite or NaN. All logits of one sign,
    and rows whose terms cancel."""
    x, w, _ = make(T, 4096, 256, dt, wdt, seed=41)
    if sign:
        x, w = x.abs(), sign * w.abs()
    x, w = (x.float() * 2.0 ** 100).to(dt), (w.float() * 2.0 ** 36).to(wdt)
    want = formula(x, w, None, 8, SOFTMAX, True, 1.0)
    assert bool(torch.isfinite(want[1]).all())
    ids, sc = run(x, w, None, 8, SOFTMAX)
    assert torch.equal(ids.long(), want[0])
    assert bool(((sc.double() - want[1]).abs() <= 2.0 ** -24 * want[1]).all())  # logits lie far apart: shares are 1 and 0
    b = torch.zeros(256)
    b[want[0][:, 0].unique()] = -float("inf")  # an expert that the bias takes out stays out
    ids, _ = run(x, w, b, 8, SIGMOID)
    want = formula(x, w, b, 8, SIGMOID, False, 1.0)
    assert torch.equal(ids.long(), want[0])


@pytest.mark.parametrize("T,dt,wdt", [(5, BF, BF), (300, BF, BF), (300, FP, FP), (600, BF, F32)], ids=str)
def test_softmax_shares_whose_difference_the_bias_all_but_cancels(T, dt, wdt):
    """Two experts of unlike shares p0 > p1 and biases that differ by p0 - p1, but for 2e-11 either way: every other
    expert's logit counts, through the softmax's sum, in which comes first. 64-bit values are 1e-15 apart at most."""
    x, w, _ = make(T, 4096, 256, dt, wdt, seed=43)
    x[:] = x[0].clone()
    n = float((x[0].double() ** 2).sum())
    w[3], w[200] = (x[0].float() * (8.0 / n)).to(wdt), (x[0].float() * (7.4 / n)).to(wdt)
    p = torch.softmax(torch.mv(w.double(), x[0].double()), 0)
    d = float(p[3] - p[200])
    assert d > 0.1
    for side in (-1, 1):
        b = torch.zeros(256)
        b[200] = d + 2e-5
        b[3] = float(b[200].double()) - d + side * 2e-11
        gap = float(p[3] + b[3].double() - p[200] - b[200].double())
        assert 1e-11 < side * gap < 4e-11
        ids, sc = run(x, w, b, 2)
        assert torch.equal(ids, torch.tensor([[3, 200] if side > 0 else [200, 3]], dtype=torch.int32).expand(T, 2))
        check((ids, sc), formula(x, w, b, 2, SOFTMAX, True, 1.0), x, w)
        assert bool((run(x, w, b, 1)[0] == (3 if side > 0 else 200)).all())


@pytest.mark.parametrize("T", [9, 300])
@pytest.mark.parametrize("bias", [False, True], ids=["logit", "bias"])
@pytest.mark.parametrize("normalize", [False, True], ids=["plain", "normalized"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID, SQRTSP], ids=["softmax", "sigmoid", "sqrtsoftplus"])
def test_nan_logit_takes_its_own_expert_out(score, normalize, bias, T):
    """As a row of weights that was never filled gives: the other experts are chosen and weighted as if it were not there."""
    x, w, b = make(T, 4096, 256, bias=bias, seed=47)
    rest = [e for e in range(256) if e not in (17, 130)]
    w[17], w[130, 40] = float("nan"), float("nan")
    ids, sc = run(x, w, b, 6, score, normalize)
    want, v = formula(x, w[rest], None if b is None else b[rest], 6, score, normalize, 1.0)
    check((ids, sc), (torch.tensor(rest)[want], v), x, w[rest])
    w3 = w.clone()
    w3[:] = float("nan")
    w3[:3] = w[:3]
    ids, sc = run(x, w3, b, 6, score, normalize)
    assert bool((ids[:, 3:] == -1).all()) and bool((sc[:, 3:] == 0).all())
    want, v = formula(x, w[:3], None if b is None else b[:3], 3, score, normalize, 1.0)
    check((ids[:, :3], sc[:, :3]), (want, v), x, w[:3])


@pytest.mark.parametrize("T", [9, 300])
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (BF, F32)], ids=["bf16", "fp32-w"])
def test_infinite_logit_comes_first(T, dt, wdt):
    x, w, b = make(T, 4096, 256, dt, wdt, bias=True, seed=53)
    x[:, 5] = x[:, 5].abs() + 1
    w[9, 5] = float("inf")
    w[77, 5] = -float("inf")
    l = torch.nan_to_num(x.double() @ w.double().t(), posinf=1e300, neginf=-1e300)
    for bias, score in ((None, SOFTMAX), (b, SOFTMAX), (None, SIGMOID)):
        ids, sc = run(x, w, bias, 4, score)
        s = torch.softmax(l, 1) if score == SOFTMAX else torch.sigmoid(l)
        want = torch.sort(l if bias is None else s + bias.double(), dim=1, descending=True, stable=True)[1][:, :4]
        v = s.gather(1, want)
        assert torch.equal(ids.long(), want) and bool((want[:, 0] == 9).all())
        v = v / v.sum(1, keepdim=True)
        assert bool(((sc.double() - v).abs() <= 2.0 ** -20 * v + 1e-45).all())


@pytest.mark.parametrize("T,H,E,K", [(1, 4096, 256, 8), (16, 1000, 128, 4), (64, 4096, 256, 8), (200, 2048, 500, 8)])
@pytest.mark.parametrize("dt,wdt", [(BF, BF), (FP, FP), (BF, F32)], ids=str)
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID, SQRTSP], ids=["softmax", "sigmoid", "sqrtsoftplus"])
def test_weights_of_small_products_are_rounded_once(T, H, E, K, dt, wdt, score):
    """Up to 2^28 products T * E * H the logits are in 64 bits whatever the types: 2^-24 relative, and 1e-10."""
    x, w, b = make(T, H, E, dt, wdt, bias=True, seed=59)
    want, v = formula(x, w, b, K, score, True, 2.5)
    ids, sc = run(x, w, b, K, score, route_scale=2.5)
    assert torch.equal(ids.long(), want)
    assert bool(((sc.double() - v).abs() <= (2.0 ** -24 + 1e-10) * v).all())


@pytest.mark.parametrize("dt,wdt", [(BF, BF), (FP, FP), (BF, F32)], ids=str)
@pytest.mark.parametrize("bias", [False, True], ids=["logit", "bias"])
@pytest.mark.parametrize("score", [SOFTMAX, SIGMOID, SQRTSP], ids=["softmax", "sigmoid", "sqrtsoftplus"])
def test_batch_does_not_change_the_experts(score, bias, dt, wdt):
    """Every kernel that a batch size leads to, among them the split of fp32 weights (from 513 tokens on)."""
    x, w, b = make(700, 4096, 256, dt, wdt, bias=bias, seed=67)
    ids = run(x, w, b, 8, score)[0]
    for n in (1, 17, 64, 257, 520):
        assert torch.equal(run(x[:n], w, b, 8, score)[0], ids[:n])
