"""moe_w8a8_linear_w4 and its packing on the GPU against the formula in 64 bits.

Tolerances, with u = 2^-24, h = half a step of the output (bf16 2^-9 of a
power of two, so 2^-8 relative at worst: eps / 2), per output:
  int8 x: a group's sum is exact; K / group scaled sums are added in fp32, each
    with two roundings, over at most 16 waves, then x_scale: (K / group + 20) u
    times the sum of the groups' magnitudes.
  fp16 x: products are exact, a group is summed in fp32 with at most `group`
    roundings of at most 2 u (an adder may truncate): 2 group u times the sum
    of |w x|, and the groups as above.
  bf16 x: as fp16 with 128 + code for code - zero, and the sum of x likewise:
    4 group u times the sum of 143 scale |x|.
  The bf16 bound is wide because all roundings would have to agree; so the
  2-norm of the error is held to h of the 2-norm too, plus a sixteenth: the
  roundings of the fp32 sums, which are as often up as down, add about
  31 sqrt(group) u = 2e-5 relative, far below h / 16.
  SwiGLU: the slope of silu is under 1.1 and |silu(g)| <= |g|."""
import pytest
import torch

import moe_expert_ffn_route_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP, I8 = torch.bfloat16, torch.float16, torch.int8


def make(T, N, K, G, act, zeros, bias, seed=0):
    g = torch.Generator().manual_seed(seed + T * 7 + N * 13 + K * 3 + G)
    code = torch.randint(0, 16, (N, K), generator=g, dtype=torch.uint8)
    scale = (0.5 + torch.rand(N, K // G, generator=g)) * (0.25 / K ** 0.5)
    zero = torch.randint(0, 16, (N, K // G), generator=g, dtype=torch.uint8) if zeros else None
    if act == I8:
        x = torch.randint(-128, 128, (T, K), generator=g, dtype=torch.int32).to(I8)
        xs = (0.5 + torch.rand(T, generator=g)) / 64
    else:
        x, xs = torch.randn(T, K, generator=g).to(act), None
    b = torch.randn(N, generator=g) * 0.1 if bias else None
    return dict(code=code, scale=scale, zero=zero, x=x, xs=xs, bias=b)


def run(c, G, gated=False, stream=None, packed=None):
    T, K = c["x"].shape
    N = c["code"].shape[0]
    d = moe.make_linear_w4_dims(T, N, K, group=G, act_dtype=c["x"].dtype, gated=gated, has_zeros=c["zero"] is not None)
    cu = lambda t: None if t is None else t.cuda()  # noqa: E731
    if packed is None:
        packed = moe.moe_w8a8_pack_weights_w4(d, (c["code"][:, 0::2] | (c["code"][:, 1::2] << 4)).contiguous().cuda(),
                                              cu(c["scale"]), cu(c["zero"]))
    width = N // 2 if gated else N
    dt = FP if c["x"].dtype == FP else BF
    buf = torch.full((T * width + 64,), 7.0, dtype=dt, device="cuda")
    torch.cuda.synchronize()
    moe.moe_w8a8_linear_w4(d, cu(c["x"]), packed, x_scale=cu(c["xs"]), bias=cu(c["bias"]), out=buf[:T * width],
                           stream=stream)
    torch.cuda.synchronize()
    assert bool((buf[T * width:] == 7).all()), "written past the end"
    return buf[:T * width].view(T, width).cpu()


def check(c, G, gated, out, tokens=None):
    """Against 64 bits (on the GPU: plain matrix products of contiguous operands)."""
    x = c["x"].cuda().double()
    K = x.shape[1]
    s = c["scale"].cuda().double()
    z = c["zero"].cuda().double() if c["zero"] is not None else torch.full_like(s, 8.0)
    q = c["code"].cuda().double() - z.repeat_interleave(G, 1)
    w = q * s.repeat_interleave(G, 1)
    xs = c["xs"].cuda().double()[:, None] if c["xs"] is not None else 1.0
    xt = x.t().contiguous()
    o = torch.mm(w, xt).t() * xs
    ng = K // G
    if c["x"].dtype == I8:
        mag = torch.zeros_like(o)
        for i in range(ng):
            k = slice(i * G, (i + 1) * G)
            mag += torch.mm(w[:, k].contiguous(), xt[k].contiguous()).t().abs()
        tol = (ng + 20) * U * mag * xs
    elif c["x"].dtype == FP:
        tol = (2 * G + ng + 20) * U * torch.mm(w.abs(), xt.abs()).t()
    else:
        tol = (4 * G + ng + 20) * U * torch.mm(143 * s.repeat_interleave(G, 1), xt.abs()).t()
    if c["bias"] is not None:
        o = o + c["bias"].cuda().double()
        tol = tol + U * o.abs()
    if gated:
        n = o.shape[1] // 2
        g, u, tg, tu = o[:, :n], o[:, n:], tol[:, :n], tol[:, n:]
        silu = g * torch.sigmoid(g)
        o = silu * u
        tol = (1.1 * tg + 8 * U * silu.abs()) * (u.abs() + tu) + silu.abs() * tu + 8 * U * o.abs()
    h = torch.finfo(out.dtype).eps / 2
    tiny = torch.finfo(out.dtype).smallest_normal * h
    err = (out.cuda().double() - o).abs()
    assert bool((err <= tol * (1 + h) + h * o.abs() + tiny).all()), float((err - tol - h * o.abs()).max())
    assert float(err.norm()) <= h * (1 + 2.0 ** -4) * float(o.norm()) + tiny * err.numel() ** 0.5


SHAPES = [(1, 1, 32, 32), (1, 16, 128, 128), (2, 17, 64, 64), (3, 33, 96, 32), (1, 4096, 4096, 128), (5, 100, 320, 64),
          (16, 256, 1152, 128), (17, 48, 2048, 64), (31, 130, 544, 32), (33, 200, 4256, 32), (64, 64, 1024, 128),
          (65, 1000, 512, 64), (128, 96, 256, 32), (130, 520, 1408, 128), (200, 2000, 640, 64), (300, 1024, 1024, 128),
          (515, 272, 192, 32), (1, 8, 16384, 128), (4, 12000, 256, 64),
          # over 1024 pairs of 16 rows and 64 tokens: the kernel for many tokens; one, two, three k tiles and more
          (33, 16500, 128, 128), (1030, 1100, 96, 32), (65, 8300, 320, 64), (600, 1999, 1152, 128), (515, 2320, 160, 32),
          (128, 8208, 256, 128), (700, 1600, 1088, 64), (64, 16400, 544, 32),
          # two and four row tiles per workgroup, their last ones past the end
          (3, 8200, 256, 128), (6, 8210, 320, 32), (12, 8200, 320, 64), (12, 16400, 1280, 128), (30, 8201, 256, 128),
          (40, 8200, 384, 128), (60, 8205, 320, 64)]


@pytest.mark.parametrize("T,N,K,G", SHAPES)
@pytest.mark.parametrize("act", [BF, FP, I8], ids=["bf16", "fp16", "int8"])
def test_shapes(T, N, K, G, act):
    for zeros, bias in ((False, True), (True, False)):
        c = make(T, N, K, G, act, zeros, bias)
        check(c, G, False, run(c, G))


@pytest.mark.parametrize("T,N,K,G", [(1, 2, 32, 32), (1, 4096, 1024, 128), (7, 34, 192, 64), (20, 512, 2048, 128),
                                     (64, 258, 416, 32), (100, 1040, 512, 128), (260, 640, 768, 64),
                                     (514, 1270, 320, 64), (100, 4500, 416, 32), (40, 9000, 384, 128)])
@pytest.mark.parametrize("act", [BF, FP, I8], ids=["bf16", "fp16", "int8"])
@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
def test_gated(T, N, K, G, act, zeros):
    c = make(T, N, K, G, act, zeros, bias=True, seed=5)
    c["scale"] = c["scale"] * 4  # gates over a few units
    check(c, G, True, run(c, G, gated=True))


@pytest.mark.parametrize("act", [BF, I8], ids=["bf16", "int8"])
@pytest.mark.parametrize("G", [32, 64, 128])
@pytest.mark.parametrize("N", [40, 4120], ids=["few", "many"])
def test_every_code_and_position(act, G, N):
    """x = unit vectors: every element of W comes out by itself, exactly rounded once."""
    K = 256
    c = make(K, N, K, G, act, True, False)
    c["x"] = torch.eye(K).to(act)
    c["xs"] = torch.ones(K) if act == I8 else None
    c["scale"] = torch.exp2(torch.randint(-4, 5, (N, K // G)).float())
    want = (c["code"].double() - c["zero"].double().repeat_interleave(G, 1)) * c["scale"].double().repeat_interleave(G, 1)
    for lo, hi in ((0, K), (37, 38), (100, 117), (3, 40), (0, 64)):  # every tile count
        c2 = dict(c, x=c["x"][lo:hi].contiguous(), xs=c["xs"][lo:hi] if act == I8 else None)
        assert torch.equal(run(c2, G).double(), want.t()[lo:hi])


def test_one_packing_serves_bf16_and_fp16_and_every_batch():
    N, K, G = 272, 1024, 128
    c = make(70, N, K, G, BF, False, False)
    d = moe.make_linear_w4_dims(1, N, K, group=G)
    packed = moe.moe_w8a8_pack_weights_w4(d, (c["code"][:, 0::2] | (c["code"][:, 1::2] << 4)).contiguous().cuda(),
                                          c["scale"].cuda())
    d16 = moe.make_linear_w4_dims(9, N, K, group=G, act_dtype=FP)
    other = moe.moe_w8a8_pack_weights_w4(d16, (c["code"][:, 0::2] | (c["code"][:, 1::2] << 4)).contiguous().cuda(),
                                         c["scale"].cuda())
    assert torch.equal(packed, other)
    for t in (1, 16, 17, 40, 70):
        for act in (BF, FP):
            c2 = dict(c, x=c["x"][:t].to(act).contiguous())
            check(c2, G, False, run(c2, G, packed=packed))


@pytest.mark.parametrize("act", [BF, I8], ids=["bf16", "int8"])
@pytest.mark.parametrize("T", [9, 150])
def test_non_finite_token_leaves_the_others(T, act):
    c = make(T, 96, 512, 64, act, True, False)
    ref = run(c, 64)
    if act == I8:
        c["xs"][4] = float("nan")
    else:
        c["x"][4, 100], c["x"][4, 101] = float("nan"), float("inf")
    out = run(c, 64)
    rows = [t for t in range(T) if t != 4]
    assert torch.equal(out[rows], ref[rows])


def test_zero_scale_and_zero_rows():
    c = make(3, 32, 256, 64, BF, True, False)
    c["scale"][5] = 0
    c["x"][1] = 0
    out = run(c, 64)
    assert float(out[1].abs().max()) == 0 and float(out[:, 5].abs().max()) == 0
    check(c, 64, False, out)


def test_large_activations():
    c = make(5, 64, 1024, 128, BF, False, False)
    c["x"] = (c["x"].float() * 2.0 ** 60).to(BF)
    c["scale"] = c["scale"] * 2.0 ** -60
    check(c, 128, False, run(c, 128))
    c = make(5, 64, 1024, 128, FP, False, False)
    c["x"] = (torch.sign(c["x"].float()) * 60000).to(FP)
    c["scale"] = c["scale"] / 4096
    check(c, 128, False, run(c, 128))


def test_side_stream_repeat_and_zero_tokens():
    c = make(12, 1000, 2048, 128, BF, False, True)
    a = run(c, 128)
    assert torch.equal(a, run(c, 128, stream=torch.cuda.Stream())) and torch.equal(a, run(c, 128))
    d = moe.make_linear_w4_dims(0, 1000, 2048)
    w = torch.empty(moe.moe_w8a8_packed_w4_bytes(d), dtype=torch.uint8, device="cuda")
    assert moe.moe_w8a8_linear_w4(d, torch.empty(0, 2048, dtype=BF, device="cuda"), w).shape == (0, 1000)


def test_weights_past_32_bits():
    """Codes of more than 4 GiB; the last rows, against the formula."""
    N, K, G = 589_840, 16384, 128
    codes = torch.randint(0, 256, (N, K // 2), dtype=torch.uint8, device="cuda",
                          generator=torch.Generator("cuda").manual_seed(4))
    scale = torch.full((N, K // G), 0.002, device="cuda")
    d = moe.make_linear_w4_dims(2, N, K, group=G)
    packed = moe.moe_w8a8_pack_weights_w4(d, codes, scale)
    x = torch.randn(2, K, generator=torch.Generator().manual_seed(2)).to(BF)
    out = moe.moe_w8a8_linear_w4(d, x.cuda(), packed)
    for rows in (slice(0, 64), slice(N - 64, N), slice(N // 2 + 7, N // 2 + 71)):
        b = codes[rows].cpu()
        c = dict(code=torch.stack((b & 15, b >> 4), -1).view(64, K), scale=scale[rows].cpu(), zero=None, x=x, xs=None,
                 bias=None)
        check(c, G, False, out[:, rows].cpu().contiguous())


@pytest.mark.parametrize("T,N,K,G", [(1, 48, 1024, 128), (7, 4100, 512, 128), (20, 260, 320, 64), (50, 130, 416, 32),
                                     (130, 8300, 512, 128), (600, 2000, 320, 64), (515, 2320, 160, 32)])
@pytest.mark.parametrize("zeros", [False, True], ids=["sym", "zeros"])
@pytest.mark.parametrize("act", [BF, FP], ids=["bf16", "fp16"])
def test_whole_numbers_come_out_exactly(T, N, K, G, zeros, act):
    """Whole x up to 2^24 / (32 G), positive as activations may be, and small whole outputs: every partial sum of
    (16 + code) * x and of 31 * x is a whole number under 2^24, so fp32 holds all of them and nothing may be lost."""
    g = torch.Generator().manual_seed(3 * T + N + K + G)
    top = 2 ** 24 // (32 * G)
    x = torch.randint(top // 2, top, (T, K // 2), generator=g).float()
    mant = {BF: 2.0 ** 8, FP: 2.0 ** 11}[act]
    step = torch.exp2(torch.floor(torch.log2(x)) + 1) / mant  # whole, or x is exact already
    x = torch.where(step > 1, torch.floor(x / step) * step, x)
    x = torch.stack((x, x), -1).view(T, K)  # equal neighbours: opposite codes cancel
    x[:, 0::G] = torch.randint(1, 4, (T, K // G), generator=g).float()
    x[:, 1::G] = 1.0
    zero = torch.randint(5, 12, (N, K // G), generator=g, dtype=torch.uint8) if zeros else None
    z = zero.repeat_interleave(G, 1) if zeros else torch.full((N, K), 8, dtype=torch.uint8)
    d = torch.randint(0, 5, (N, K // 2), generator=g).to(torch.int16)
    code = z.to(torch.int16) + torch.stack((d, -d), -1).view(N, K)
    few = torch.zeros(K, dtype=torch.bool)
    few[0::G], few[1::G] = True, True
    live = (torch.arange(K // G) == K // G - 1).repeat_interleave(G)  # one group whose pair does not cancel
    code[:, few & live] = (z.to(torch.int16) + torch.randint(0, 3, (N, K), generator=g, dtype=torch.int16))[:, few & live]
    code[:, few & ~live] = z.to(torch.int16)[:, few & ~live]
    c = dict(code=code.to(torch.uint8), scale=torch.ones(N, K // G), zero=zero, x=x.to(act), xs=None, bias=None)
    assert torch.equal(c["x"].float(), x) and bool((code >= 0).all()) and bool((code <= 15).all())
    want = torch.mm(x.double(), (code.double() - z.double()).t().contiguous())
    assert float(want.abs().max()) <= 8 and float((x.view(T, K // G, G).sum(-1)).max()) * 31 < 2 ** 24
    assert torch.equal(run(c, G).double(), want)
