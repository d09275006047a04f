"""moe_w8a8_dispatch, moe_w8a8_combine and moe_w8a8_combine_grad on the GPU.

The maps are whole numbers and the rows are copies: equal to a plain stable
sort. Combine's sum has one order (k ascending, fp32), so it equals the same
operations in torch bit for bit; so do the gradient's rows (one product, one
rounding). The gradient of a routing weight is an fp32 dot product over H of
exact-to-u products: a thread adds at most 64 + 8 of them (256 threads or more
share a row of 16384), six shuffles and 16 waves' sums follow, the product is
rounded: under 128 u of the sum of magnitudes, u = 2^-24."""
import pytest
import torch

import moe_expert_ffn_route_amd as moe

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
BF, FP, F32, I8 = torch.bfloat16, torch.float16, torch.float32, torch.int8
F8 = torch.float8_e4m3fn


def ids_of(T, E, K, seed=0, kind="random"):
    g = torch.Generator().manual_seed(seed + T * 7 + E * 3 + K)
    if kind == "one":
        return torch.full((T, K), E // 2, dtype=torch.int32)
    ids = torch.argsort(torch.rand(T, E, generator=g) + 0.3 * torch.rand(E, generator=g), 1)[:, :K].int() if K <= E else \
        torch.randint(0, E, (T, K), generator=g, dtype=torch.int32)
    if kind == "dropped":
        junk = torch.tensor([-1, E, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32)[torch.randint(0, 4, (T, K), generator=g)]
        ids = torch.where(torch.rand(T, K, generator=g) < 0.3, junk, ids)
    if kind == "none":
        ids = torch.full((T, K), -1, dtype=torch.int32)
    return ids.contiguous()


def plain(ids, E, align, mask=None):
    """row_of_pair, pair_of_row without its end, counts, offsets: a loop over
    the experts."""
    T, K = ids.shape
    flat = ids.flatten().long()
    if mask is not None:
        flat = torch.where(mask.repeat_interleave(K) != 0, flat, -1)
    row_of_pair, pair_of_row = torch.full((T * K,), -1), []
    counts, offset = [], [0]
    by = torch.argsort(flat, stable=True)
    key = flat[by]
    for e in range(E):
        lo, hi = torch.searchsorted(key, e).item(), torch.searchsorted(key, e, right=True).item()
        pairs = by[lo:hi]
        row_of_pair[pairs] = offset[-1] + torch.arange(hi - lo)
        fill = -(hi - lo) % align
        pair_of_row += [pairs, torch.full((fill,), -1)]
        counts.append(hi - lo)
        offset.append(offset[-1] + hi - lo + fill)
    return row_of_pair.view(T, K), torch.cat(pair_of_row), torch.tensor(counts), torch.tensor(offset)


def data(T, H, dt, seed=0):
    g = torch.Generator().manual_seed(seed + T + H)
    if dt in (I8, F8):
        return torch.randint(-128, 128, (T, H), generator=g, dtype=torch.int32).to(I8).view(dt).cuda()
    return torch.randn(T, H, generator=g).to(dt).cuda()


def check_dispatch(ids, E, H, dt=BF, groups=0, align=1, mask=None, x=True, stream=None):
    T, K = ids.shape
    d = moe.make_dispatch_dims(T, H, E, K, dtype=I8 if dt == F8 else dt, scale_groups=groups, row_align=align)
    R = moe.moe_w8a8_dispatch_rows(d)
    xs = data(T, H, dt) if x else None
    sc = torch.rand(T, groups, generator=torch.Generator().manual_seed(T)).cuda() if x and groups else None
    guard = lambda n, t: torch.full((n + 32,), 77, dtype=t, device="cuda")  # noqa: E731
    bufs = dict(expert_token_nums=guard(E, torch.int32), expert_offset=guard(E + 1, torch.int32),
                row_of_pair=guard(T * K, torch.int32), pair_of_row=guard(R, torch.int32))
    sizes = dict(expert_token_nums=E, expert_offset=E + 1, row_of_pair=T * K, pair_of_row=R)
    if x:
        bufs["rows"], sizes["rows"] = guard(R * H, I8 if dt == F8 else dt), R * H
        if groups:
            bufs["row_scale"], sizes["row_scale"] = guard(R * groups, F32), R * groups
    n = moe.moe_w8a8_dispatch_workspace_size(d)
    ws = torch.full((max(256, n) + 64,), 77, dtype=torch.uint8, device="cuda")
    given = {k: b[:sizes[k]] for k, b in bufs.items()}
    if dt == F8:
        given["rows"] = given["rows"].view(F8)
    ic, mc = ids.cuda(), None if mask is None else mask.cuda()
    torch.cuda.synchronize()
    out = moe.moe_w8a8_dispatch(d, ic, x=xs, x_scale=sc, x_active_mask=mc, workspace=ws[:max(256, n)],
                                stream=stream, **given)
    torch.cuda.synchronize()
    for k, b in bufs.items():
        assert bool((b[sizes[k]:].float() == 77).all()), (k, "written past the end")
    assert bool((ws[max(256, n):] == 77).all())
    row_of_pair, pair_of_row, counts, offset = plain(ids, E, align, mask)
    used = len(pair_of_row)
    assert used <= R
    assert torch.equal(out["row_of_pair"].view(T, K).cpu().long(), row_of_pair)
    assert torch.equal(out["pair_of_row"][:used].cpu().long(), pair_of_row)
    assert bool((out["pair_of_row"][used:] == -1).all())
    assert torch.equal(out["expert_token_nums"].cpu().long(), counts)
    assert torch.equal(out["expert_offset"].cpu().long(), offset)
    if x:
        def moved(got, src, width, untouched):
            got = got.view(R, width)
            want = torch.zeros(used, width, dtype=src.dtype, device="cuda")
            some = (pair_of_row >= 0).cuda()
            want[some] = src[(pair_of_row[pair_of_row >= 0] // K).cuda()]
            assert torch.equal(got[:used], want)
            assert bool((got[used:].float() == untouched).all()), "rows behind the last"
        bytes_of = (lambda t: t.view(I8)) if dt == F8 else (lambda t: t)
        moved(bytes_of(out["rows"]), bytes_of(xs), H, 77)
        if groups:
            moved(out["row_scale"], sc, groups, 77)
    return d, out


SHAPES = [(1, 1, 1, 1), (1, 8, 2, 17), (3, 4, 4, 64), (8, 256, 8, 4096), (7, 72, 6, 5003), (64, 256, 8, 512), (17, 1024, 16, 33),
          (128, 3, 2, 100), (200, 5, 1, 2500), (256, 64, 8, 96), (257, 64, 8, 40), (2048, 100, 1, 24), (2049, 100, 1, 24),
          (1000, 256, 8, 200), (3000, 1024, 6, 31), (4096, 512, 16, 16), (9, 2, 5, 16384), (700, 1, 7, 12), (5001, 33, 3, 65)]


@pytest.mark.parametrize("T,E,K,H", SHAPES)
@pytest.mark.parametrize("align", [1, 16])
def test_dispatch_shapes(T, E, K, H, align):
    check_dispatch(ids_of(T, E, K), E, H, BF, align=align)
    check_dispatch(ids_of(T, E, K, kind="dropped"), E, H, I8, groups=1, align=align)


@pytest.mark.parametrize("T,E,K", [(1, 5, 3), (40, 16, 4), (500, 70, 6), (1500, 300, 2)])
@pytest.mark.parametrize("kind", ["random", "dropped", "one", "none"])
def test_dispatch_ids(T, E, K, kind):
    ids = ids_of(T, E, K, kind=kind)
    mask = (torch.rand(T, generator=torch.Generator().manual_seed(T)) < 0.6).to(torch.uint8) * 3
    for align in (1, 2, 64, 256):
        check_dispatch(ids, E, 72, FP, align=align)
        check_dispatch(ids, E, 72, FP, align=align, mask=mask)
    check_dispatch(ids, E, 72, F32, mask=torch.zeros(T, dtype=torch.uint8), align=8)


@pytest.mark.parametrize("dt", [BF, FP, F32, I8, F8], ids=str)
def test_dispatch_types(dt):
    for T, H in ((5, 129), (700, 1000)):
        check_dispatch(ids_of(T, 9, 3), 9, H, dt, groups=0 if dt in (BF, FP, F32) else 7, align=4)


@pytest.mark.parametrize("T,groups", [(4, 1), (4, 256), (600, 32), (1200, 3)])
def test_dispatch_scales(T, groups):
    check_dispatch(ids_of(T, 20, 4), 20, 256, I8, groups=groups, align=32)


def test_dispatch_maps_alone():
    check_dispatch(ids_of(50, 20, 4), 20, 256, BF, x=False, align=8)
    check_dispatch(ids_of(5000, 20, 4), 20, 256, BF, x=False, groups=2, align=8)


def test_dispatch_allocates():
    ids = ids_of(33, 12, 3)
    x = data(33, 100, I8)
    s = torch.rand(33, 2, device="cuda")
    d = moe.make_dispatch_dims(33, 100, 12, 3, dtype=I8, scale_groups=2)
    out = moe.moe_w8a8_dispatch(d, ids.cuda(), x=x, x_scale=s)
    torch.cuda.synchronize()
    token = out["pair_of_row"].long() // 3
    assert torch.equal(out["rows"], x[token]) and torch.equal(out["row_scale"], s[token])
    maps = moe.moe_w8a8_dispatch(moe.make_dispatch_dims(33, 100, 12, 3), ids.cuda())
    assert maps["rows"] is None and torch.equal(maps["row_of_pair"], out["row_of_pair"])


def test_dispatch_no_token():
    d = moe.make_dispatch_dims(0, 64, 5, 2, row_align=4)
    out = moe.moe_w8a8_dispatch(d, torch.empty(0, 2, dtype=torch.int32, device="cuda"))
    assert out["expert_token_nums"].tolist() == [0] * 5 and out["expert_offset"].tolist() == [0] * 6
    assert out["pair_of_row"].shape == (0,)


def test_dispatch_largest_number_of_pairs():
    check_dispatch(ids_of(65536, 1024, 16), 1024, 3, I8, align=256)


def test_dispatch_offsets_past_32_bits():
    """Rows whose bytes end behind 2^32."""
    T, K, H = 4300, 16, 16384
    ids = ids_of(T, 40, K)
    d = moe.make_dispatch_dims(T, H, 40, K, dtype=F32)
    x = torch.randn(T, H, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    out = moe.moe_w8a8_dispatch(d, ids.cuda(), x=x)
    row_of_pair, _, _, _ = plain(ids, 40, 1)
    assert out["rows"].numel() * 4 > 2 ** 32
    for k in (0, 7, 15):
        assert torch.equal(out["rows"][row_of_pair[:, k].cuda()], x)
    cd = moe.make_combine_dims(T, H, K, T * K, dtype=F32)
    back = moe.moe_w8a8_combine(cd, out["rows"], out["row_of_pair"])
    want = torch.zeros_like(x)
    for k in range(K):
        want = want + x
    assert torch.equal(back, want)
    dr = torch.empty_like(out["rows"])
    moe.moe_w8a8_combine_grad(cd, back, out["row_of_pair"], out["pair_of_row"], drows=dr)
    assert torch.equal(dr[row_of_pair[:, 9].cuda()], back) and torch.equal(dr[row_of_pair[:, 0].cuda()], back)


# ------------------------------------------------------------ combine and back

def case(T, E, K, H, dt, out_dt, kind="random", align=1, seed=0):
    g = torch.Generator().manual_seed(seed + T + H * 3)
    ids = ids_of(T, E, K, seed, kind)
    rp, pr, _, _ = plain(ids, E, align)
    R = T * K + min(E, T * K) * (align - 1)
    pair_of_row = torch.full((R,), -1)
    pair_of_row[:len(pr)] = pr
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(rows=n(R, H).to(dt).cuda(), row_of_pair=rp.int().cuda(), pair_of_row=pair_of_row.int().cuda(),
                w=torch.rand(T, K, generator=g).cuda(), addend=n(T, H).to(out_dt).cuda(), dout=n(T, H).to(out_dt).cuda())


def combined(c, out_dt, weights=True, addend=True):
    """The operations of the header in torch, one by one."""
    T, K = c["row_of_pair"].shape
    R = c["rows"].shape[0]
    o = torch.zeros(T, c["rows"].shape[1], device="cuda")
    for k in range(K):
        r = c["row_of_pair"][:, k].long()
        some = (r >= 0) & (r < R)
        z = c["rows"][r.clamp(0, R - 1)].float()
        if weights:
            z = z * c["w"][:, k:k + 1]
        o = torch.where(some[:, None], o + z, o)
    if addend:
        o = o + c["addend"].float()
    return o.to(out_dt)


def combine(c, out_dt, weights=True, addend=True, in_place=False, stream=None):
    T, K = c["row_of_pair"].shape
    R, H = c["rows"].shape
    buf = torch.full((T * H + 64,), 7.0, device="cuda").to(out_dt)
    if in_place:
        buf[:T * H] = c["addend"].flatten()
    out = buf[:T * H].view(T, H)
    torch.cuda.synchronize()
    moe.moe_w8a8_combine(moe.make_combine_dims(T, H, K, R, dtype=c["rows"].dtype, out_dtype=out_dt), c["rows"],
                         c["row_of_pair"], expert_scales=c["w"] if weights else None,
                         addend=(out if in_place else c["addend"]) if addend else None, out=out, stream=stream)
    torch.cuda.synchronize()
    assert bool((buf[T * H:].float() == 7).all()), "written past the end"
    return out


def grads(c, weights=True, drows=True, dscales=True, stream=None):
    T, K = c["row_of_pair"].shape
    R, H = c["rows"].shape
    db = torch.full((R * H + 64,), 7.0, device="cuda").to(c["rows"].dtype)
    sb = torch.full((T * K + 64,), 7.0, device="cuda")
    dr, ds = db[:R * H].view(R, H), sb[:T * K].view(T, K)
    torch.cuda.synchronize()
    moe.moe_w8a8_combine_grad(moe.make_combine_dims(T, H, K, R, dtype=c["rows"].dtype, out_dtype=c["dout"].dtype), c["dout"],
                              c["row_of_pair"], c["pair_of_row"], rows=c["rows"] if dscales else None,
                              expert_scales=c["w"] if weights else None, drows=dr if drows else None,
                              dscales=ds if dscales else None, stream=stream)
    torch.cuda.synchronize()
    assert bool((db[R * H:].float() == 7).all()) and bool((sb[T * K:] == 7).all()), "written past the end"
    return dr, ds


def check_grads(c, dr, ds, weights=True):
    T, K = c["row_of_pair"].shape
    R, H = c["rows"].shape
    p = c["pair_of_row"].long()
    some = p >= 0
    want = torch.zeros(R, H, device="cuda")
    want[some] = c["dout"].float()[p[some] // K]
    if weights:
        want[some] = want[some] * c["w"].flatten()[p[some], None]
    if dr is not None:
        assert torch.equal(dr, want.to(dr.dtype))
    if ds is not None:
        r = c["row_of_pair"].long()
        rows, d = c["rows"].double(), c["dout"].double()
        for k in range(K):
            t = rows[r[:, k].clamp(min=0)] * d
            kept = r[:, k] >= 0
            err = (ds[:, k].double() - t.sum(1)).abs()
            assert bool((err <= 128 * U * t.abs().sum(1))[kept].all())
            assert bool((ds[:, k][~kept] == 0).all())


CSHAPES = [(1, 1, 1, 1), (1, 8, 2, 7), (2, 16, 3, 8), (8, 256, 8, 4096), (5, 72, 6, 5003), (64, 64, 16, 520), (3, 4, 4, 16384),
           (300, 40, 5, 2501), (1000, 256, 8, 96), (2047, 72, 6, 33), (4000, 16, 1, 64), (70, 9, 9, 8200), (33, 300, 12, 2056)]
TYPES = [(BF, BF), (BF, F32), (FP, FP), (FP, F32), (F32, F32)]
TYPE_IDS = ["bf16", "bf16_fp32", "fp16", "fp16_fp32", "fp32"]


@pytest.mark.parametrize("T,E,K,H", CSHAPES)
@pytest.mark.parametrize("dt,out_dt", TYPES, ids=TYPE_IDS)
def test_combine_shapes(T, E, K, H, dt, out_dt):
    c = case(T, E, K, H, dt, out_dt)
    assert torch.equal(combine(c, out_dt), combined(c, out_dt))
    c = case(T, E, K, H, dt, out_dt, "dropped", align=16, seed=1)
    assert torch.equal(combine(c, out_dt, weights=False, addend=False), combined(c, out_dt, False, False))
    assert torch.equal(combine(c, out_dt, in_place=True), combined(c, out_dt))


@pytest.mark.parametrize("T,E,K,H", CSHAPES)
@pytest.mark.parametrize("dt,out_dt", TYPES, ids=TYPE_IDS)
def test_grad_shapes(T, E, K, H, dt, out_dt):
    c = case(T, E, K, H, dt, out_dt)
    check_grads(c, *grads(c))
    c = case(T, E, K, H, dt, out_dt, "dropped", align=8, seed=1)
    check_grads(c, *grads(c))
    dr, _ = grads(c, weights=False, dscales=False)
    check_grads(c, dr, None, weights=False)
    _, ds = grads(c, drows=False)
    check_grads(c, None, ds)


@pytest.mark.parametrize("T", [3, 700])
def test_all_dropped(T):
    c = case(T, 10, 4, 100, BF, BF, "none")
    assert torch.equal(combine(c, BF), c["addend"])
    assert bool((combine(c, BF, addend=False).view(torch.int16) == 0).all())  # +0
    dr, ds = grads(c)
    assert bool((dr == 0).all()) and bool((ds == 0).all())


def test_no_rows():
    c = case(5, 10, 4, 100, BF, BF, "none")
    d = moe.make_combine_dims(5, 100, 4, 0)
    none = torch.empty(0, 100, dtype=BF, device="cuda")
    assert torch.equal(moe.moe_w8a8_combine(d, none, c["row_of_pair"], addend=c["addend"]), c["addend"])
    ds = torch.ones(5, 4, device="cuda")
    moe.moe_w8a8_combine_grad(d, c["dout"], c["row_of_pair"], torch.empty(0, dtype=torch.int32, device="cuda"), rows=none,
                              expert_scales=c["w"], drows=torch.empty_like(none), dscales=ds)
    assert bool((ds == 0).all())


@pytest.mark.parametrize("dt", [BF, torch.float32])
@pytest.mark.parametrize("R,H", [(1, 5), (50, 100), (2100, 4096)])
def test_no_tokens(R, H, dt):
    """No row has a pair: zeros, whatever the maps hold."""
    buf = torch.full((R + 2, H), 3, dtype=dt, device="cuda")
    if H % 8 == 0:
        dr = buf[1:R + 1]
    else:
        dr = torch.full((R, H), 3, dtype=dt, device="cuda")
    maps = torch.zeros(R, dtype=torch.int32, device="cuda")
    ids = torch.empty(0, 4, dtype=torch.int32, device="cuda")
    moe.moe_w8a8_combine_grad(moe.make_combine_dims(0, H, 4, R, dtype=dt), torch.empty(0, H, dtype=dt, device="cuda"), ids, maps,
                              drows=dr)
    assert bool((dr == 0).all())
    assert bool((buf[0] == 3).all()) and bool((buf[R + 1] == 3).all())


@pytest.mark.parametrize("T", [6, 600])
def test_rows_outside_are_dropped(T):
    """Rows past the end or below 0 add nothing; a row that two pairs claim is
    the pair's that pair_of_row names."""
    c = case(T, 10, 4, 200, BF, BF)
    c["row_of_pair"][1, 2], c["row_of_pair"][2, 0], c["row_of_pair"][3, 3] = T * 4, 2 ** 31 - 1, -2 ** 31
    c["rows"][0] = float("nan")  # where dropped pairs might look
    c["row_of_pair"][c["row_of_pair"] == 0] = -7
    assert torch.equal(combine(c, BF), combined(c, BF))
    gone = torch.zeros(T * 4, dtype=torch.bool, device="cuda")
    for p, r in enumerate(c["row_of_pair"].flatten().tolist()):
        if not 0 <= r < T * 4:
            gone[p] = True
    first, second = 4, 5
    c["row_of_pair"].view(-1)[second] = c["row_of_pair"].view(-1)[first]
    dr, ds = grads(c)
    lost = c["pair_of_row"].long()
    gone[second] = True
    want = c["dout"].float()[lost // 4] * c["w"].flatten()[lost, None]
    want[gone[lost]] = 0
    assert torch.equal(dr, want.to(BF))
    assert bool((ds.flatten()[gone] == 0).all())


def test_gradients_against_differences():
    """Combine is linear in its rows and in its weights: with fp32 and steps of
    a power of two the difference quotient is the gradient, but for roundings
    (each of the K sums' two: 2 K u of the magnitudes, twice, over 2 delta)."""
    T, E, K, H = 40, 12, 4, 300
    c = case(T, E, K, H, F32, F32, "dropped", align=4)
    dr, ds = grads(c)
    g = torch.Generator().manual_seed(3)
    delta = 0.25
    d6 = c["dout"].double()
    mag = float((combined(dict(c, rows=c["rows"].abs()), F32).double().abs() * d6.abs()).sum()) * 2
    for name in ("rows", "w"):
        step = torch.randn(c[name].shape, generator=g).cuda()
        up, down = dict(c, **{name: c[name] + delta * step}), dict(c, **{name: c[name] - delta * step})
        quotient = float(((combine(up, F32).double() - combine(down, F32).double()) * d6).sum()) / (2 * delta)
        moved = (up[name].double() - down[name].double()) / (2 * delta)  # the step that was taken
        want = float(((dr if name == "rows" else ds).double() * moved).sum())
        assert abs(quotient - want) <= (4 * K * U * mag / delta + 128 * U * mag) * 4, (name, quotient, want)


def test_dispatch_gradient_is_combine_without_weights():
    """<dispatch(x), d> = <x, combine(d)>, and the rows that fill a tile take
    no part."""
    T, E, K, H = 50, 12, 3, 128
    ids = ids_of(T, E, K, kind="dropped")
    d = moe.make_dispatch_dims(T, H, E, K, dtype=F32, row_align=8)
    x = data(T, H, F32)
    out = moe.moe_w8a8_dispatch(d, ids.cuda(), x=x, rows=torch.zeros(moe.moe_w8a8_dispatch_rows(d), H, device="cuda"))
    R = out["rows"].shape[0]
    grad = data(R, H, F32, seed=9)
    dx = moe.moe_w8a8_combine(moe.make_combine_dims(T, H, K, R, dtype=F32), grad, out["row_of_pair"])
    a, b = (out["rows"].double() * grad.double()).sum(), (x.double() * dx.double()).sum()
    mag = float((out["rows"].double() * grad.double()).abs().sum())
    assert abs(float(a - b)) <= K * U * mag


@pytest.mark.parametrize("T,K", [(20, 4), (3000, 2)])
def test_captured(T, K):
    """Dispatch, combine and the gradient in one graph, replayed on other ids."""
    E, H = 24, 264
    d = moe.make_dispatch_dims(T, H, E, K, row_align=4)
    R = moe.moe_w8a8_dispatch_rows(d)
    new = lambda *s, dt: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    i32 = torch.int32
    out = dict(rows=new(R, H, dt=BF), expert_token_nums=new(E, dt=i32), expert_offset=new(E + 1, dt=i32),
               row_of_pair=new(T, K, dt=i32), pair_of_row=new(R, dt=i32))
    ws = new(max(256, moe.moe_w8a8_dispatch_workspace_size(d)), dt=torch.uint8)
    ids, x, w, back = new(T, K, dt=i32), new(T, H, dt=BF), torch.rand(T, K, device="cuda"), new(T, H, dt=BF)
    dr, ds, cd = new(R, H, dt=BF), new(T, K, dt=F32), moe.make_combine_dims(T, H, K, R)

    def step():
        moe.moe_w8a8_dispatch(d, ids, x=x, workspace=ws, **out)
        moe.moe_w8a8_combine(cd, out["rows"], out["row_of_pair"], expert_scales=w, out=back)
        moe.moe_w8a8_combine_grad(cd, back, out["row_of_pair"], out["pair_of_row"], rows=out["rows"], expert_scales=w,
                                  drows=dr, dscales=ds)
    ids.copy_(ids_of(T, E, K))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        kind = "dropped" if seed % 2 else "random"
        i = ids_of(T, E, K, seed=seed, kind=kind)
        ids.copy_(i)
        x.copy_(data(T, H, BF, seed))
        out["rows"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        rp, pr, counts, offset = plain(i, E, 4)
        assert torch.equal(out["row_of_pair"].cpu().long(), rp) and torch.equal(out["expert_offset"].cpu().long(), offset)
        c = dict(rows=out["rows"], row_of_pair=out["row_of_pair"], pair_of_row=out["pair_of_row"], w=w, dout=back)
        assert torch.equal(back, combined(c, BF, addend=False))
        check_grads(c, dr, ds)
        kept = [t.clone() for t in (*out.values(), back, dr, ds)]
        step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, (*out.values(), back, dr, ds)))


@pytest.mark.parametrize("T,K", [(1500, 4), (40000, 2)])
def test_two_graphs_share_a_workspace(T, K):
    """Batches that use it; replayed in turn, with other ids each time."""
    E, H = 40, 24
    d = moe.make_dispatch_dims(T, H, E, K, dtype=I8, row_align=8)
    need = moe.moe_w8a8_dispatch_workspace_size(d)
    assert need > 0
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    R = moe.moe_w8a8_dispatch_rows(d)
    x = data(T, H, I8)
    sides = []
    for _ in range(2):
        ids = ids_of(T, E, K).cuda()
        out = dict(rows=torch.zeros(R, H, dtype=I8, device="cuda"), expert_token_nums=torch.empty(E, dtype=torch.int32, device="cuda"),
                   expert_offset=torch.empty(E + 1, dtype=torch.int32, device="cuda"),
                   row_of_pair=torch.empty(T, K, dtype=torch.int32, device="cuda"),
                   pair_of_row=torch.empty(R, dtype=torch.int32, device="cuda"))
        moe.moe_w8a8_dispatch(d, ids, x=x, workspace=ws, **out)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_w8a8_dispatch(d, ids, x=x, workspace=ws, **out)
        sides.append((ids, out, graph))
    for seed in range(3):
        new = [ids_of(T, E, K, seed=10 * seed + i, kind="dropped" if seed else "random") for i in range(2)]
        for (ids, _, _), i in zip(sides, new):
            ids.copy_(i)
        for _, _, graph in sides:
            graph.replay()
        torch.cuda.synchronize()
        for (_, out, _), i in zip(sides, new):
            rp, _, counts, offset = plain(i, E, 8)
            assert torch.equal(out["row_of_pair"].cpu().long(), rp)
            assert torch.equal(out["expert_token_nums"].cpu().long(), counts)
            assert torch.equal(out["expert_offset"].cpu().long(), offset)
            at = out["row_of_pair"].view(-1).long()
            kept = at >= 0
            assert torch.equal(out["rows"][at[kept]], x.repeat_interleave(K, 0)[kept])


@pytest.mark.parametrize("T,K", [(8, 8), (16, 4), (17, 4), (33, 2), (500, 8), (513, 8), (70, 16)])
def test_dispatch_at_the_borders_of_its_launches(T, K):
    """64 and 4096 pairs, and one more, with and without padded tiles."""
    for align in (1, 16):
        for kind in ("random", "dropped"):
            check_dispatch(ids_of(T, 48, K, kind=kind), 48, 200, I8, groups=3, align=align)
            check_dispatch(ids_of(T, 48, K, kind=kind), 48, 1, I8, align=align)


# Calls that write 16 MB or more, whose stores are streamed: every launch of dispatch, rows that end inside 16 bytes

@pytest.mark.parametrize("T,E,K,H,dt,groups,align", [
    (8, 64, 8, 4100, I8, 3, 256), (12, 40, 5, 8200, BF, 0, 256), (500, 20, 8, 5003, BF, 0, 16), (480, 70, 8, 5003, I8, 2, 16),
    (2100, 20, 4, 1003, BF, 0, 16), (2100, 20, 4, 2051, I8, 1, 16), (17000, 60, 4, 515, FP, 0, 16), (17000, 60, 4, 517, I8, 5, 1),
    (4100, 33, 6, 333, F32, 0, 64), (1030, 8, 4, 4096, F8, 32, 16)])
def test_dispatch_streamed(T, E, K, H, dt, groups, align):
    for kind in ("random", "dropped"):
        d, out = check_dispatch(ids_of(T, E, K, kind=kind), E, H, dt, groups=groups, align=align)
    assert out["rows"].numel() * out["rows"].element_size() >= 16 << 20


@pytest.mark.parametrize("T,E,K,H", [(2047, 72, 6, 5003), (2048, 64, 8, 4104), (4100, 20, 1, 2501), (1100, 40, 12, 8200),
                                     (40000, 50, 2, 217), (1030, 30, 3, 8193)])
@pytest.mark.parametrize("dt,out_dt", TYPES, ids=TYPE_IDS)
def test_combine_streamed(T, E, K, H, dt, out_dt):
    assert T * H * out_dt.itemsize >= 16 << 20
    c = case(T, E, K, H, dt, out_dt, "dropped", seed=3)
    assert torch.equal(combine(c, out_dt, addend=False), combined(c, out_dt, addend=False))
    assert torch.equal(combine(c, out_dt, in_place=True), combined(c, out_dt))
    assert torch.equal(combine(c, out_dt, weights=False), combined(c, out_dt, weights=False))


@pytest.mark.parametrize("T,E,K,H", [(600, 40, 8, 2003), (520, 30, 5, 4104), (300, 50, 12, 4099), (400, 20, 16, 2056),
                                     (9000, 20, 2, 501)])
@pytest.mark.parametrize("dt,out_dt", TYPES, ids=TYPE_IDS)
def test_grad_streamed(T, E, K, H, dt, out_dt):
    c = case(T, E, K, H, dt, out_dt, "dropped", align=16, seed=4)
    assert c["rows"].numel() * dt.itemsize >= 16 << 20
    check_grads(c, *grads(c))
    dr, _ = grads(c, weights=False, dscales=False)
    check_grads(c, dr, None, weights=False)


class Dispatched(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, d, ids):
        out = moe.moe_w8a8_dispatch(d, ids, x=x, rows=torch.zeros(moe.moe_w8a8_dispatch_rows(d), x.shape[1], device="cuda"))
        ctx.row_of_pair = out["row_of_pair"]
        ctx.mark_non_differentiable(out["row_of_pair"], out["pair_of_row"])
        return out["rows"], out["row_of_pair"], out["pair_of_row"]

    @staticmethod
    def backward(ctx, drows, *_):
        (T, K), (R, H) = ctx.row_of_pair.shape, drows.shape
        return moe.moe_w8a8_combine(moe.make_combine_dims(T, H, K, R, dtype=F32), drows.contiguous(), ctx.row_of_pair), None, None


class Combined(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rows, weights, addend, row_of_pair, pair_of_row):
        ctx.save_for_backward(rows, weights, row_of_pair, pair_of_row)
        T, K = row_of_pair.shape
        d = moe.make_combine_dims(T, rows.shape[1], K, rows.shape[0], dtype=F32)
        return moe.moe_w8a8_combine(d, rows, row_of_pair, expert_scales=weights, addend=addend)

    @staticmethod
    def backward(ctx, dout):
        rows, weights, row_of_pair, pair_of_row = ctx.saved_tensors
        T, K = row_of_pair.shape
        d = moe.make_combine_dims(T, rows.shape[1], K, rows.shape[0], dtype=F32)
        drows, dweights, dout = torch.empty_like(rows), torch.empty_like(weights), dout.contiguous()
        moe.moe_w8a8_combine_grad(d, dout, row_of_pair, pair_of_row, rows=rows, expert_scales=weights, drows=drows,
                                  dscales=dweights)
        return drows, dweights, dout, None, None


def test_inside_autograd():
    """A layer of a program's own experts (scales by expert) that trains, and
    the same by torch's indexing in 64 bits. A gradient is a sum of products of
    three factors, of at most T = 70 terms (scales: an expert's pairs; rows that
    fill a tile add zeros) or H = 130 (weights): in any order 130 u of the terms'
    magnitudes, and 3 u for the products."""
    T, E, K, H = 70, 11, 4, 130
    ids = ids_of(T, E, K, kind="dropped")
    g = torch.Generator().manual_seed(8)
    leaf = lambda *s: torch.randn(*s, generator=g).cuda().requires_grad_()  # noqa: E731
    x, w, a, scale = leaf(T, H), leaf(T, K), leaf(T, H), leaf(E, H)
    dout = torch.randn(T, H, generator=g).cuda()
    d = moe.make_dispatch_dims(T, H, E, K, dtype=F32, row_align=4)
    rows, row_of_pair, pair_of_row = Dispatched.apply(x, d, ids.cuda())
    expert = ids.cuda().flatten().long()[pair_of_row.long().clamp(min=0)].clamp(0, E - 1)
    out = Combined.apply(rows * scale[expert], w, a, row_of_pair, pair_of_row)
    got = torch.autograd.grad(out, (x, w, a, scale), dout)

    def plain_layer(x, w, a, scale):
        kept = ((ids >= 0) & (ids < E)).cuda()
        z = x[:, None] * scale[ids.cuda().long().clamp(0, E - 1)]
        return (z * (w * kept)[..., None]).sum(1) + a
    wide = [t.detach().double().requires_grad_() for t in (x, w, a, scale)]
    want = torch.autograd.grad(plain_layer(*wide), wide, dout.double())
    size = [t.detach().double().abs().requires_grad_() for t in (x, w, a, scale)]
    mag = torch.autograd.grad(plain_layer(*size), size, dout.double().abs())
    for one, two, m in zip(got, want, mag):
        assert bool(((one.double() - two).abs() <= 133 * U * (1 + 2.0 ** -14) * m).all())
