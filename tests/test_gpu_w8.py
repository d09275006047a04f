"""moe_w8a8_linear_w8 and its packing on the GPU.

The sums are exact, and each step after them is one fp32 operation in a fixed
order, so without SwiGLU the outputs equal, bit for bit, those operations on
the exact sums (fp64 products of integers below 2^53). They are also held to
the formula in 64 bits: the sum's conversion to fp32, two products and the
bias's addition are at most four roundings of u = 2^-24 relative to |o - bias|
and |o|, then half a step h of the output (bf16 and fp16: eps / 2).
SwiGLU: the slope of silu is under 1.1 and |silu(g)| <= |g|; exp, the
division, the addition and the product add 8 u."""
import pytest
import torch

import moe_expert_ffn_route_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


def make(T, N, K, bias, seed=0):
    g = torch.Generator().manual_seed(seed + T * 7 + N * 13 + K * 3)
    i8 = lambda *s: torch.randint(-128, 128, s, generator=g, dtype=torch.int32).to(torch.int8)  # noqa: E731
    return dict(x=i8(T, K), xs=(0.5 + torch.rand(T, generator=g)) / 64, w=i8(N, K),
                ws=(0.5 + torch.rand(N, generator=g)) / (64 * K ** 0.5), bias=torch.randn(N, generator=g) * 0.1 if bias else None)


def pack(c, gated=False, **kw):
    d = moe.make_linear_w8_dims(1, *c["w"].shape, gated=gated)
    return moe.moe_w8a8_pack_weights_w8(d, c["w"].cuda(), c["ws"].cuda(), **kw)


def run(c, dt=BF, gated=False, packed=None, stream=None):
    T, K = c["x"].shape
    N = c["w"].shape[0]
    packed = pack(c, gated) if packed is None else packed
    width = N // 2 if gated else N
    buf = torch.full((T * width + 64,), 7.0, dtype=dt, device="cuda")
    xs = [c["x"].cuda(), c["xs"].cuda(), None if c["bias"] is None else c["bias"].cuda()]
    torch.cuda.synchronize()
    moe.moe_w8a8_linear_w8(moe.make_linear_w8_dims(T, N, K, out_dtype=dt, gated=gated), xs[0], xs[1], packed, bias=xs[2],
                           out=buf[:T * width], stream=stream)
    torch.cuda.synchronize()
    assert bool((buf[T * width:] == 7).all()), "written past the end"
    return buf[:T * width].view(T, width)


def sums(c):
    """The exact sums, in fp64 (a plain matrix product of contiguous operands)."""
    return torch.mm(c["w"].cuda().double(), c["x"].cuda().double().t().contiguous()).t().contiguous()


def check(c, out, gated=False, acc=None):
    acc = sums(c) if acc is None else acc
    ws, xs = c["ws"].cuda(), c["xs"].cuda()[:, None]
    if not gated:
        o = acc.float() * ws * xs
        if c["bias"] is not None:
            o = o + c["bias"].cuda()
        assert torch.equal(out, o.to(out.dtype))
    o = acc * ws.double() * xs.double()
    tol = 4 * U * o.abs()
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
    err = (out.double() - o).abs()
    assert bool((err <= tol * (1 + h) + h * o.abs() + tiny).all()), float((err - tol - h * o.abs()).max())


SHAPES = [(1, 1, 1), (1, 16, 64), (1, 17, 15), (2, 31, 17), (3, 33, 100), (5, 7, 3), (1, 4096, 4096), (7, 100, 129),
          (8, 256, 1152), (9, 48, 2048), (15, 130, 545), (16, 64, 128), (17, 200, 4251), (31, 80, 255), (33, 250, 640),
          (48, 1000, 96), (63, 65, 1000), (64, 512, 512), (65, 96, 272), (100, 300, 1009), (127, 129, 128),
          (129, 257, 384), (130, 2000, 640), (255, 256, 256), (257, 520, 1408), (300, 1024, 1024), (515, 272, 191),
          (1000, 1000, 1000), (600, 1999, 1152), (2049, 130, 200), (700, 4100, 72), (1, 8, 65536), (3, 24, 65521),
          (40, 8, 16400), (16, 16400, 48), (1024, 2048, 16), (4, 12000, 257), (260, 4096, 130), (1030, 515, 2050)]


@pytest.mark.parametrize("T,N,K", SHAPES)
def test_shapes(T, N, K):
    c = make(T, N, K, bias=True)
    acc, packed = sums(c), pack(c)
    check(c, run(c, BF, packed=packed), acc=acc)
    c["bias"] = None
    check(c, run(c, F32, packed=packed), acc=acc)
    check(c, run(c, FP, packed=packed), acc=acc)


# long contractions: the large tiles, eight stages under way, and row tiles of four; odd and even, K just past a group of stages
LARGE = [(4096, 4096, 2064), (4100, 4100, 2053), (2050, 4100, 2064), (2060, 4090, 2181), (512, 4096, 2048), (520, 4090, 2065),
         (1100, 1000, 2176), (1100, 1000, 3001), (256, 4096, 2064), (250, 4090, 3071), (128, 4096, 1920), (100, 3000, 4000)]


@pytest.mark.parametrize("T,N,K", LARGE)
def test_large(T, N, K):
    c = make(T, N, K, bias=True)
    acc, packed = sums(c), pack(c)
    check(c, run(c, F32, packed=packed), acc=acc)
    c["bias"] = None
    check(c, run(c, BF, packed=packed), acc=acc)
    check(c, run(c, FP, gated=True), gated=True, acc=acc)


def test_a_token_is_the_same_in_every_kernel():
    for K in (2064, 2069):
        c = make(4200, 4112, K, bias=False, seed=19)
        packed = pack(c)
        whole = run(c, F32, packed=packed)
        for T in (1, 16, 40, 100, 300, 700, 2100):
            assert torch.equal(run(dict(c, x=c["x"][-T:], xs=c["xs"][-T:]), F32, packed=packed), whole[-T:]), (T, K)


@pytest.mark.parametrize("T,N,K", [(1, 2, 1), (1, 4096, 1024), (7, 34, 193), (20, 512, 2048), (64, 258, 416), (100, 1042, 515),
                                   (260, 640, 768), (513, 1026, 1000), (1029, 2048, 260), (2000, 18, 48)])
@pytest.mark.parametrize("dt", [BF, FP, F32], ids=["bf16", "fp16", "fp32"])
def test_gated(T, N, K, dt):
    c = make(T, N, K, bias=T % 2 == 0, seed=5)
    check(c, run(c, dt, gated=True), gated=True)


@pytest.mark.parametrize("T", [1, 16, 40, 300])
@pytest.mark.parametrize("K", [65536, 65521])
def test_largest_sums_do_not_overflow(T, K):
    c = make(T, 20, K, bias=False)
    c["x"].fill_(-128)
    c["w"].fill_(-128)  # 2^30 each
    c["w"][3] = 127
    check(c, run(c, F32))


def test_a_token_is_the_same_in_every_batch():
    """Whichever kernel a batch takes, a row's outputs are the same bits."""
    for gated in (False, True):
        c = make(2100, 1030, 1000, bias=True, seed=9)
        packed = pack(c, gated)
        whole = run(c, F32, gated=gated, packed=packed)
        for T in (1, 3, 8, 9, 16, 17, 33, 64, 65, 128, 200, 257, 512, 1024):
            part = dict(c, x=c["x"][-T:], xs=c["xs"][-T:])
            assert torch.equal(run(part, F32, gated=gated, packed=packed), whole[-T:]), (T, gated)


def test_packing():
    for N, K, gated in ((33, 200, False), (16, 128, False), (34, 65, True)):
        c = make(1, N, K, bias=False, seed=3)
        d = moe.make_linear_w8_dims(1, N, K, gated=gated)
        n = moe.moe_w8a8_packed_w8_bytes(d)
        buf = torch.full((n + 16,), 7, dtype=torch.uint8, device="cuda")
        moe.moe_w8a8_pack_weights_w8(d, c["w"].cuda(), c["ws"].cuda(), dst=buf[:n])
        got = buf.cpu()
        assert bool((got[n:] == 7).all())
        kt, tiles = -(-K // 128), -(-(N // 2) // 8) if gated else -(-N // 16)
        rows = torch.zeros(tiles * 16, kt * 128, dtype=torch.int8)
        scale = torch.zeros(tiles * 16)
        if gated:
            h = N // 2
            pick = lambda t: torch.stack((t[:h], t[h:]), 1).flatten(0, 1)  # noqa: E731  gate and up rows in turn
            rows[:N, :K], scale[:N] = pick(c["w"]), pick(c["ws"])
        else:
            rows[:N, :K], scale[:N] = c["w"], c["ws"]
        # [tile, row, block of 64 k, quarter, byte] -> [tile, block, quarter, row, byte]
        want = rows.view(tiles, 16, kt * 2, 4, 16).permute(0, 2, 3, 1, 4).contiguous().view(torch.uint8).flatten()
        assert torch.equal(got[:want.numel()], want)
        assert torch.equal(got[want.numel():n].view(torch.float32), scale)


def test_scales_of_any_size_and_zero():
    """Row scales from subnormal to large, zero rows, and bias alone."""
    c = make(40, 100, 200, bias=True, seed=11)
    c["xs"][:4] = torch.tensor([0.0, 2.0 ** -100, 2.0 ** 60, 1.0])
    c["ws"][:3] = torch.tensor([0.0, 2.0 ** -60, 2.0 ** 20])
    c["x"][5] = 0
    check(c, run(c, F32))


def test_allocates_its_output_and_runs_on_a_stream():
    c = make(20, 300, 500, bias=True, seed=2)
    packed = pack(c)
    want = run(c, BF, packed=packed)
    side = torch.cuda.Stream()
    x, xs, b = c["x"].cuda(), c["xs"].cuda(), c["bias"].cuda()
    torch.cuda.synchronize()
    got = moe.moe_w8a8_linear_w8(moe.make_linear_w8_dims(20, 300, 500), x, xs, packed, bias=b, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    with torch.cuda.stream(side):
        got = moe.moe_w8a8_linear_w8(moe.make_linear_w8_dims(20, 300, 500), x, xs, packed, bias=b)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("T,K", [(4, 512), (40, 500), (300, 1024)])
def test_captured(T, K):
    """Replays on new inputs, with eager work between them."""
    c = make(T, 500, K, bias=False, seed=4)
    packed, d = pack(c), moe.make_linear_w8_dims(T, 500, K)
    x, xs, out = c["x"].cuda(), c["xs"].cuda(), torch.empty(T, 500, dtype=BF, device="cuda")
    moe.moe_w8a8_linear_w8(d, x, xs, packed, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_w8a8_linear_w8(d, x, xs, packed, out=out)
    for seed in range(4):
        n = make(T, 500, K, bias=False, seed=20 + seed)
        x.copy_(n["x"])
        xs.copy_(n["xs"])
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        check(dict(n, w=c["w"], ws=c["ws"]), got)
        assert torch.equal(moe.moe_w8a8_linear_w8(d, x, xs, packed), got)


def test_no_token():
    c = make(1, 32, 64, bias=False)
    out = moe.moe_w8a8_linear_w8(moe.make_linear_w8_dims(0, 32, 64), c["x"][:0].cuda(), c["xs"][:0].cuda(), pack(c))
    assert out.shape == (0, 32)


# One shape at least for every kernel that a product can take, with whole and odd rows (test_w8_rule.py checks that they do)
EVERY = [(5, 100, 512), (7, 90, 515), (12, 200, 1024), (16, 330, 1001), (9, 8300, 256), (14, 8202, 263), (40, 500, 2000),
         (33, 610, 777), (40, 2000, 640), (45, 2018, 1037), (64, 4096, 4096), (64, 4096, 4099), (40, 4800, 2048),
         (37, 4810, 1155), (64, 6000, 512), (100, 3000, 3999), (64, 10000, 528), (63, 9990, 531), (4096, 4096, 1936),
         (4090, 4102, 1933), (2048, 3200, 2064), (2040, 3206, 2061), (1088, 2944, 208), (1080, 2950, 201),
         (1088, 2944, 2064), (1080, 2950, 2071), (2500, 5000, 704), (2500, 5000, 700), (640, 2048, 2064), (630, 2050, 2057),
         (640, 1920, 2064), (630, 1910, 2059), (640, 2560, 272), (630, 2570, 261), (100, 1000, 112), (90, 1010, 101)]


@pytest.mark.parametrize("T,N,K", EVERY)
def test_every_kernel(T, N, K):
    c = make(T, N, K, bias=True, seed=31)
    acc, packed, gated = sums(c), pack(c), pack(c, True)
    for dt in (BF, FP, F32):
        check(c, run(c, dt, packed=packed), acc=acc)
        check(c, run(c, dt, gated=True, packed=gated), gated=True, acc=acc)
        c["bias"] = None


def test_short_rows_and_a_wide_output():
    """Outputs of 240 MB, streamed, of two tiles of k."""
    c = make(6000, 20000, 100, bias=True, seed=37)
    out = run(c, BF)
    for t in range(0, 6000, 2000):  # fp64 values of a part at a time
        part = dict(c, x=c["x"][t:t + 2000], xs=c["xs"][t:t + 2000])
        check(part, out[t:t + 2000])
