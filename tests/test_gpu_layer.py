"""The feed-forward half of a layer as a program runs it: norm (with residual
and 8-bit output) -> router -> expert block on the norm's codes, and the norm's
codes through a dense gated pair of 4-bit products. Also
moe_w8a8_forward_quantized by itself: bit for bit moe_w8a8_forward on an x
whose codes it is given."""
import threading

import numpy as np
import pytest
import torch

import moe_expert_ffn_route_amd as moe
import oracle
from moe_expert_ffn_route_amd import synth

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
ERR = pytest.raises


def codes_of(case):
    """The block's own codes of x, by the oracle's quantiser."""
    s = case.spec
    x = synth.bf16_bits_to_f32(case.x).astype(np.float32)
    if s.quant_group:
        q, sc = zip(*(oracle.quant_row_groups(r, s.quant_group) for r in x))
    elif s.weight_format == "mxfp4":
        q, sc = zip(*(oracle.quant_row_fp8(r) for r in x))
    else:
        q, sc = zip(*(oracle.quant_row(r) for r in x))
    q = torch.from_numpy(np.ascontiguousarray(np.stack(q)).view(np.int8)).cuda()
    return q, torch.from_numpy(np.asarray(sc, dtype=np.float32)).cuda()


def spec(**kw):
    base = dict(name="q", T=12, H=512, I=256, E_g=8, K=2, I_s=256, seed=811)
    base.update(kw)
    return synth.Spec(**base)


CASES = {
    "decode": spec(active=10),
    "decode_fused_route_scale": spec(fuse_route_scale=True, I_s=0),
    "requant_in_epilogue": spec(requant_in_epilogue=True, I_s=512),
    "wide": spec(T=40, active=33),
    "wide_ep_share": spec(T=70, E_g=16, ep_size=2, ep_rank=1, K=4),
    "tall": spec(T=300, E_g=2),
    "group128": spec(quant_group=128),
    "group64_wide": spec(quant_group=64, T=80, E_g=4),
    "mxfp4": spec(weight_format="mxfp4"),
    "mxfp4_wide": spec(weight_format="mxfp4", T=90, E_g=4),
    "one_token": spec(T=1),
}


@pytest.mark.parametrize("name", list(CASES))
def test_forward_quantized_equals_forward(name):
    case = synth.make_case(CASES[name])
    dims = moe.dims_of_case(case)
    t = moe.upload(case)
    if CASES[name].weight_format == "int8":
        t = moe.pack_weights(t)
        dims.weight_layout = moe.MOE_WEIGHT_PACKED
    ref = moe.Runner(dims)
    ref(t)
    q, s = codes_of(case)
    t2 = {k: v for k, v in t.items() if k not in ("x", "expert_smooth_scales", "share_smooth_scales")}
    got = moe.Runner(dims)
    got.workspace.fill_(0xA5)
    got.output.fill_(7)
    moe.moe_w8a8_forward_quantized(dims, q, s, output=got.output, share_output=got.share_output,
                                   expert_token_nums=got.expert_token_nums, workspace=got.workspace, **t2)
    torch.cuda.synchronize()
    assert torch.equal(got.output.view(torch.int16), ref.output.view(torch.int16))
    assert torch.equal(got.expert_token_nums, ref.expert_token_nums)
    if ref.share_output is not None:
        assert torch.equal(got.share_output.view(torch.int16), ref.share_output.view(torch.int16))


def test_forward_quantized_debug_rows_and_zero_tokens():
    case = synth.make_case(CASES["wide"])
    dims, t = moe.dims_of_case(case), moe.upload(case)
    q, s = codes_of(case)
    t = {k: v for k, v in t.items() if k not in ("x", "expert_smooth_scales", "share_smooth_scales")}
    r = moe.Runner(dims)
    d, bufs = moe.debug_buffers(dims)
    moe.moe_w8a8_forward_quantized(dims, q, s, output=r.output, share_output=r.share_output, dbg=d,
                                   expert_token_nums=r.expert_token_nums, workspace=r.workspace, **t)
    torch.cuda.synchronize()
    P = int(bufs["num_rows"][0])
    tok = (bufs["sorted_pair"][:P] // dims.topk).long()
    assert P > 0 and torch.equal(bufs["q_x"][:P], q[tok]) and torch.equal(bufs["xs"][:P], s[tok])
    dims.num_tokens = 0
    none = dict(t, expert_ids=None, expert_scales=None, x_active_mask=None)
    moe.moe_w8a8_forward_quantized(dims, None, None, expert_token_nums=r.expert_token_nums, workspace=r.workspace,
                                   **none)
    torch.cuda.synchronize()
    assert int(r.expert_token_nums.sum()) == 0


class Layer:
    """One feed-forward half with every buffer that its calls keep."""

    def __init__(self, T, H=512, I=256, E=16, K=4, dense=768, seed=0):
        g = torch.Generator().manual_seed(seed)
        rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.T, self.H, self.I, self.E, self.K, self.D = T, H, I, E, K, dense
        cu = lambda t: t.cuda()  # noqa: E731
        self.x, self.res, self.w = cu(rn(T, H).to(BF)), cu((3 * rn(T, H)).to(BF)), cu((0.5 + torch.rand(H, generator=g)).to(BF))
        self.wg, self.bias = cu((rn(E, H) / H ** 0.5).to(BF)), cu(0.02 * rn(E))
        i8 = lambda *s: torch.clamp(torch.round(32 * rn(*s)), -127, 127).to(torch.int8)  # noqa: E731
        sc = lambda *s: (1 + torch.rand(*s, generator=g)) * 1e-3  # noqa: E731
        self.w1, self.w1s, self.w2, self.w2s = i8(E, 2 * I, H), sc(E, 2 * I), i8(E, H, I), sc(E, H)
        self.dims = moe.make_dims(T, H, I, K, E)
        self.run_ = moe.Runner(self.dims)
        self.gpu = [cu(t) for t in (self.w1, self.w1s, self.w2, self.w2s)]
        self.nd = moe.make_norm_dims(T, H)
        self.r, self.y = torch.empty_like(self.x), torch.empty_like(self.x)
        self.q, self.s = torch.empty(T, H, dtype=torch.int8, device="cuda"), torch.empty(T, device="cuda")
        self.gd = moe.make_gate_dims(T, H, E, K, score=moe.MOE_SCORE_SIGMOID, route_scale=1.5)
        self.ids, self.sc = torch.empty(T, K, dtype=torch.int32, device="cuda"), torch.empty(T, K, device="cuda")
        self.gws = torch.empty(max(256, moe.moe_w8a8_gate_workspace_size(self.gd)), dtype=torch.uint8, device="cuda")
        # dense gated pair: up to D, back to H
        self.c1, self.c2 = torch.randint(0, 16, (2 * dense, H), generator=g, dtype=torch.uint8), \
            torch.randint(0, 16, (H, dense), generator=g, dtype=torch.uint8)
        self.s1, self.s2 = (0.5 + torch.rand(2 * dense, H // 128, generator=g)) * 0.02, \
            (0.5 + torch.rand(H, dense // 64, generator=g)) * 0.01
        self.ld1 = moe.make_linear_w4_dims(T, 2 * dense, H, group=128, act_dtype=torch.int8, gated=True)
        self.ld2 = moe.make_linear_w4_dims(T, H, dense, group=64)
        pair = lambda c: (c[:, 0::2] | (c[:, 1::2] << 4)).contiguous().cuda()  # noqa: E731
        self.p1 = moe.moe_w8a8_pack_weights_w4(self.ld1, pair(self.c1), cu(self.s1))
        self.p2 = moe.moe_w8a8_pack_weights_w4(self.ld2, pair(self.c2), cu(self.s2))
        self.h, self.o = torch.empty(T, dense, dtype=BF, device="cuda"), torch.empty(T, H, dtype=BF, device="cuda")

    def __call__(self):
        moe.moe_w8a8_norm_quant(self.nd, self.x, self.w, residual=self.res, residual_out=self.r, y=self.y, q=self.q,
                                q_scale=self.s)
        moe.moe_w8a8_gate(self.gd, self.y, self.wg, bias=self.bias, expert_ids=self.ids, expert_scales=self.sc,
                          workspace=self.gws)
        w1, w1s, w2, w2s = self.gpu
        moe.moe_w8a8_forward_quantized(self.dims, self.q, self.s, self.ids, self.sc, w1, w1s, w2, w2s,
                                       output=self.run_.output, expert_token_nums=self.run_.expert_token_nums,
                                       workspace=self.run_.workspace)
        moe.moe_w8a8_linear_w4(self.ld1, self.q, self.p1, x_scale=self.s, out=self.h)
        moe.moe_w8a8_linear_w4(self.ld2, self.h, self.p2, out=self.o)

    def outputs(self):
        return [self.r, self.y, self.q, self.s, self.ids, self.sc, self.run_.output, self.run_.expert_token_nums,
                self.h, self.o]

    def clear(self):
        for t in self.outputs():
            t.fill_(3)
        self.gws.fill_(0x5A)
        self.run_.workspace.fill_(0x5A)


@pytest.mark.parametrize("T", [1, 9, 40, 300])
def test_layer_against_64_bits(T):
    L = Layer(T)
    L.clear()
    L()
    torch.cuda.synchronize()
    d = lambda t: t.cpu().double()  # noqa: E731
    r = d(L.x) + d(L.res)
    y = r / torch.sqrt((r * r).mean(1, keepdim=True) + 1e-6) * d(L.w)
    assert float((d(L.y) - y).abs().max()) <= (2.0 ** -8 + 1e-5) * float(y.abs().max())
    # the router works on the bf16 rows it is given
    sig = torch.sigmoid(torch.mm(d(L.y), d(L.wg).t().contiguous()))
    ids = torch.sort(sig + d(L.bias), dim=1, descending=True, stable=True)[1][:, :L.K]
    assert torch.equal(L.ids.cpu().long(), ids)
    wt = sig.gather(1, ids)
    wt = 1.5 * wt / wt.sum(1, keepdim=True)
    assert float((d(L.sc) - wt).abs().max()) <= 2e-7
    # the experts on the norm's codes: h is requantised to 8 bits a row, the
    # rows are bf16, both inside the block's own bar
    xq = d(L.q) * d(L.s)[:, None]
    assert float((xq - y).abs().max()) <= 0.51 * float(L.s.max())
    out = torch.zeros(T, L.H, dtype=torch.float64)
    for e in range(L.E):
        tk, kk = (ids == e).nonzero(as_tuple=True)
        if len(tk):
            a = torch.mm(xq[tk], (L.w1[e].double() * L.w1s[e].double()[:, None]).t().contiguous())
            h = a[:, :L.I] * torch.sigmoid(a[:, :L.I]) * a[:, L.I:]
            hs = h.abs().amax(1, keepdim=True) / 127
            h = torch.round(h / hs) * hs
            z = torch.mm(h, (L.w2[e].double() * L.w2s[e].double()[:, None]).t().contiguous())
            out.index_add_(0, tk, z * wt[tk, kk][:, None])
    err = (d(L.run_.output) - out).abs()
    assert float(err.max()) <= 2e-2 * float(out.abs().max()) and float(err.sum()) <= 5e-3 * float(out.abs().sum())
    # the dense pair, each product on what it was given
    deq = lambda c, s, G: (c.double() - 8) * s.double().repeat_interleave(G, 1)  # noqa: E731
    a = torch.mm(xq, deq(L.c1, L.s1, 128).t().contiguous())
    h = a[:, :L.D] * torch.sigmoid(a[:, :L.D]) * a[:, L.D:]
    assert float((d(L.h) - h).norm()) <= 2.0 ** -8 * 1.1 * float(h.norm())
    o = torch.mm(d(L.h), deq(L.c2, L.s2, 64).t().contiguous())
    assert float((d(L.o) - o).norm()) <= 2.0 ** -8 * 1.1 * float(o.norm())


@pytest.mark.parametrize("T", [1, 9, 40, 300])
def test_layer_captured_and_replayed(T):
    a, b = Layer(T, seed=1), Layer(T, seed=2)
    eager = []
    for L in (a, b):
        L.clear()
        L()
        torch.cuda.synchronize()
        eager.append([t.clone() for t in L.outputs()])
    st = torch.cuda.Stream()
    graphs = []
    for L in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            L()
        graphs.append(g)
    for i in range(4):
        for L in (a, b):
            L.clear()
        torch.cuda.synchronize()
        graphs[i % 2].replay()
        graphs[1 - i % 2].replay()
        torch.cuda.synchronize()
        for L, e in zip((a, b), eager):
            for got, want in zip(L.outputs(), e):
                assert torch.equal(got.view(torch.uint8), want.view(torch.uint8)), i


def test_two_layers_at_once_on_two_streams():
    a, b = Layer(40, seed=3), Layer(9, seed=4)
    want = []
    for L in (a, b):
        L()
        torch.cuda.synchronize()
        want.append([t.clone() for t in L.outputs()])
        L.clear()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for L, st in zip((a, b), streams):
            with torch.cuda.stream(st):
                L()
    torch.cuda.synchronize()
    for L, w in zip((a, b), want):
        for got, x in zip(L.outputs(), w):
            assert torch.equal(got.view(torch.uint8), x.view(torch.uint8))


def test_two_threads_call_at_once():
    """A thread and a stream each: the calls release the interpreter's lock."""
    layers = [Layer(40, seed=3), Layer(9, seed=4)]
    want = []
    for L in layers:
        L()
        torch.cuda.synchronize()
        want.append([t.clone() for t in L.outputs()])
        L.clear()
    torch.cuda.synchronize()
    errors = []

    def work(L):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    L()
        except Exception as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(L,)) for L in layers]
    for t in threads:
        t.start()
    for t in threads:
        t.join(60)
    torch.cuda.synchronize()
    assert not errors and not any(t.is_alive() for t in threads)
    for L, w in zip(layers, want):
        for got, x in zip(L.outputs(), w):
            assert torch.equal(got.view(torch.uint8), x.view(torch.uint8))


def test_buffers_that_a_call_allocates_belong_to_its_stream():
    """On a stream of their own, with the current stream taking and filling
    memory as fast as it can: a workspace freed to the wrong pool would be
    overwritten under the kernels."""
    g = torch.Generator().manual_seed(12)
    x, w = torch.randn(700, 2048, generator=g).to(BF).cuda(), torch.randn(128, 2048, generator=g).to(BF).cuda()
    d = moe.make_gate_dims(700, 2048, 128, 6)
    want = moe.moe_w8a8_gate(d, x, w)
    n = moe.moe_w8a8_gate_workspace_size(d)
    torch.cuda.synchronize()
    for stream in (torch.cuda.Stream(), torch.cuda.Stream().cuda_stream):
        for _ in range(10):
            ids, sc = moe.moe_w8a8_gate(d, x, w, stream=stream)
            junk = [torch.empty(n, dtype=torch.uint8, device="cuda").fill_(0xFF) for _ in range(3)]
            torch.cuda.synchronize()
            assert torch.equal(ids, want[0]) and torch.equal(sc, want[1])
            del junk
    ld = moe.make_linear_w4_dims(5, 64, 256)
    codes = torch.randint(0, 256, (64, 128), dtype=torch.uint8, generator=g).cuda()
    scale = torch.rand(64, 2, generator=g).cuda()
    x5 = torch.randn(5, 256, generator=g).to(BF).cuda()
    ref = moe.moe_w8a8_linear_w4(ld, x5, moe.moe_w8a8_pack_weights_w4(ld, codes, scale))
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    out = moe.moe_w8a8_linear_w4(ld, x5, moe.moe_w8a8_pack_weights_w4(ld, codes, scale, stream=st), stream=st)
    st.synchronize()
    assert torch.equal(out, ref)


def test_allocating_calls_captured_and_on_the_null_stream():
    """Outputs and workspaces that calls allocate under capture are the graph's own; handle 0 is a stream."""
    g = torch.Generator().manual_seed(14)
    x, w = torch.randn(70, 1024, generator=g).to(BF).cuda(), torch.randn(128, 1024, generator=g).to(BF).cuda()
    d, ld = moe.make_gate_dims(70, 1024, 128, 6), moe.make_linear_w4_dims(70, 64, 1024)
    codes = torch.randint(0, 256, (64, 512), dtype=torch.uint8, generator=g).cuda()
    packed = moe.moe_w8a8_pack_weights_w4(ld, codes, torch.rand(64, 8, generator=g).cuda())
    call = lambda **kw: [*moe.moe_w8a8_gate(d, x, w, **kw), moe.moe_w8a8_linear_w4(ld, x, packed, **kw)]  # noqa: E731
    want = call()
    torch.cuda.synchronize()
    got = call(stream=0)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(4):
        for t in got:
            t.fill_(1)
        call()  # eager work in between
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_binding_refuses_tensors_that_do_not_fit():
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    d = moe.make_norm_dims(4, 64, quant=moe.MOE_QUANT_NONE)
    with ERR(ValueError, match="contiguous"):
        moe.moe_w8a8_norm_quant(d, torch.zeros(64, 4, dtype=BF, device="cuda").t(), y=x)
    with ERR(ValueError, match="y: expected"):
        moe.moe_w8a8_norm_quant(d, x, y=x.float())
    with ERR(ValueError, match="residual: expected"):
        moe.moe_w8a8_norm_quant(d, x, residual=x[:3], y=x)
    with ERR(ValueError, match="weight: .*GPU"):
        moe.moe_w8a8_norm_quant(d, x, torch.ones(64, dtype=BF), y=x)
    with ERR(moe.MoeError):  # 8 bytes off
        buf = torch.zeros(4 * 64 + 8, dtype=BF, device="cuda")
        moe.moe_w8a8_norm_quant(d, buf[4:4 + 256].view(4, 64), y=x)
    g = moe.make_gate_dims(4, 64, 8, 2)
    with ERR(moe.MoeError):
        moe.moe_w8a8_gate(g, x, x[:0].new_zeros(8, 64), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    ld = moe.make_linear_w4_dims(4, 32, 64, group=64)
    with ERR(ValueError, match="weight: expected"):
        moe.moe_w8a8_linear_w4(ld, x, torch.zeros(100, dtype=torch.uint8, device="cuda"))
    with ERR(ValueError, match="x_scale: expected"):
        ld8 = moe.make_linear_w4_dims(4, 32, 64, group=64, act_dtype=torch.int8)
        w = torch.zeros(moe.moe_w8a8_packed_w4_bytes(ld8), dtype=torch.uint8, device="cuda")
        moe.moe_w8a8_linear_w4(ld8, x.to(torch.int8), w, x_scale=torch.ones(3, device="cuda"))
    bd = moe.make_dims(num_tokens=4, hidden=512, inter=256, topk=2, moe_expert_num=8)
    q, s = torch.zeros(4, 512, dtype=torch.int8, device="cuda"), torch.ones(4, device="cuda")
    with ERR(ValueError, match="q_x: expected"):
        moe.moe_w8a8_forward_quantized(bd, q[:3], s, *[None] * 6)
    with ERR(ValueError, match="q_x: expected"):
        moe.moe_w8a8_forward_quantized(bd, q.to(BF), s, *[None] * 6)
    with ERR(ValueError, match="x_scale: expected"):
        moe.moe_w8a8_forward_quantized(bd, q, s[:3], *[None] * 6)
    with ERR(moe.MoeError):
        moe.moe_w8a8_forward_quantized(bd, q, s, *[None] * 6)
