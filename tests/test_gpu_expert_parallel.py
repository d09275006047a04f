"""The operators between the block and the rest of a program as a program runs
them together: an expert-parallel layer on one GPU, its ranks one after the
other. Norm with codes -> router -> dispatch -> each rank's block on the rows
of its experts -> combine -> joining norm -> a dense gated pair of int8
products -> the stream."""
import threading

import pytest
import torch

import moe_expert_ffn_route_amd as moe

pytestmark = pytest.mark.gpu
BF, F32, I8 = torch.bfloat16, torch.float32, torch.int8
U = 2.0 ** -24


class Layer:
    def __init__(self, T, H=512, inter=256, E=16, K=4, ranks=4, dense=768, seed=0):
        g = torch.Generator().manual_seed(seed)
        i8 = lambda *s: torch.randint(-127, 128, s, generator=g, dtype=torch.int32).to(I8).cuda()  # noqa: E731
        u = lambda *s: (torch.rand(*s, generator=g) + 0.5).cuda()  # noqa: E731
        n = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
        self.T, self.H, self.inter, self.E, self.K, self.ranks, self.dense = T, H, inter, E, K, ranks, dense
        self.norm, self.next_norm, self.post = u(H).to(BF), u(H).to(BF), u(H).to(BF)
        self.router = (n(E, H) / H ** 0.5).to(BF)
        self.w1, self.w1s, self.w2, self.w2s = i8(E, 2 * inter, H), u(E, 2 * inter) * 4e-4, i8(E, H, inter), u(E, H) * 1e-3
        self.s1, self.s1s, self.s2, self.s2s = i8(2 * inter, H), u(2 * inter) * 4e-4, i8(H, inter), u(H) * 1e-3
        self.d1, self.d1s, self.d2, self.d2s = i8(2 * dense, H), u(2 * dense) * 4e-4, i8(H, dense), u(H) * 4e-4
        self.p1 = moe.moe_w8a8_pack_weights_w8(moe.make_linear_w8_dims(T, 2 * dense, H, gated=True), self.d1, self.d1s)
        self.p2 = moe.moe_w8a8_pack_weights_w8(moe.make_linear_w8_dims(T, H, dense), self.d2, self.d2s)

    def block(self, q, s, ids, w, rank=None, shared=False):
        """The block on codes: all experts, or a rank's share. Its outputs."""
        T, K = ids.shape
        ep = 1 if rank is None else self.ranks
        loc = self.E // ep
        lo = 0 if rank is None else rank * loc
        d = moe.make_dims(T, self.H, self.inter, K, self.E, share_inter=self.inter if shared else 0, ep_rank_size=ep,
                          ep_rank_id=0 if rank is None else rank)
        out, sout = (torch.empty(T, self.H, dtype=BF, device="cuda") for _ in range(2))
        nums = torch.empty(loc, dtype=torch.int32, device="cuda")
        ws = torch.empty(max(256, moe.moe_w8a8_workspace_size(d)), dtype=torch.uint8, device="cuda")
        share = (self.s1, self.s1s, self.s2, self.s2s) if shared else (None,) * 4
        moe.moe_w8a8_forward_quantized(d, q, s, ids, w, self.w1[lo:lo + loc], self.w1s[lo:lo + loc], self.w2[lo:lo + loc],
                                       self.w2s[lo:lo + loc], *share, output=out, share_output=sout if shared else None,
                                       expert_token_nums=nums, workspace=ws)
        return out, sout, nums

    def front(self, x, res):
        T, H = self.T, self.H
        q, s, stream = torch.empty(T, H, dtype=I8, device="cuda"), torch.empty(T, device="cuda"), torch.empty_like(x)
        y = torch.empty_like(x)
        moe.moe_w8a8_norm_quant(moe.make_norm_dims(T, H), x, self.norm, residual=res, residual_out=stream, y=y, q=q, q_scale=s)
        ids, w = moe.moe_w8a8_gate(moe.make_gate_dims(T, H, self.E, self.K), y, self.router)
        return stream, q, s, ids, w

    def back(self, stream, out, share):
        """From the block's outputs to the dense pair's."""
        T, H = self.T, self.H
        d = moe.make_join_norm_dims(T, H, post_norm=True, residual_scale=0.5)
        o = dict(residual_out=torch.empty_like(stream), q=torch.empty(T, H, dtype=I8, device="cuda"),
                 q_scale=torch.empty(T, device="cuda"))
        moe.moe_w8a8_join_norm(d, out, residual=stream, share=share, post_weight=self.post, weight=self.next_norm, **o)
        h = moe.moe_w8a8_linear_w8(moe.make_linear_w8_dims(T, 2 * self.dense, H, gated=True), o["q"], o["q_scale"], self.p1)
        hq, hs = moe.moe_w8a8_quant(moe.make_quant_dims(T, self.dense), h)
        z = moe.moe_w8a8_linear_w8(moe.make_linear_w8_dims(T, H, self.dense, out_dtype=BF), hq, hs, self.p2)
        return dict(o, h=h, hq=hq, hs=hs, z=z)

    def split(self, q, s, ids, w):
        """The block over the ranks: dispatch, each rank's share, combine."""
        T, H = self.T, self.H
        d = moe.make_dispatch_dims(T, H, self.E, self.K, dtype=I8, scale_groups=1)
        sent = moe.moe_w8a8_dispatch(d, ids, x=q, x_scale=s)
        at = sent["expert_offset"].tolist()
        loc = self.E // self.ranks
        back = torch.full((T * self.K, H), 7.0, dtype=BF, device="cuda")
        for r in range(self.ranks):
            a, b = at[r * loc], at[(r + 1) * loc]
            if a == b:
                continue
            mine = torch.repeat_interleave(torch.arange(r * loc, (r + 1) * loc, device="cuda"),
                                           sent["expert_token_nums"][r * loc:(r + 1) * loc].long()).int().view(-1, 1)
            got, _, nums = self.block(sent["rows"][a:b].clone(), sent["row_scale"][a:b, 0].clone(), mine,
                                      torch.ones(b - a, 1, device="cuda"), rank=r)
            assert torch.equal(nums, sent["expert_token_nums"][r * loc:(r + 1) * loc])
            back[a:b] = got
        return moe.moe_w8a8_combine(moe.make_combine_dims(T, H, self.K, T * self.K), back, sent["row_of_pair"], expert_scales=w)


def inputs(T, H, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(T, H, generator=g).to(BF).cuda(), (torch.randn(T, H, generator=g) * 2).to(BF).cuda()


@pytest.mark.parametrize("T", [1, 8, 40, 300])
def test_ranks_together_are_the_whole_block(T):
    """Bit for bit: a rank's rows are the block's own z rows (weight 1), and
    combine is the block's."""
    m = Layer(T, seed=T)
    stream, q, s, ids, w = m.front(*inputs(T, m.H, T))
    whole, share, _ = m.block(q, s, ids, w, shared=True)
    split = m.split(q, s, ids, w)
    torch.cuda.synchronize()
    assert torch.equal(whole, split)
    one, other = m.back(stream, whole, share), m.back(stream, split, share)
    for k in one:
        assert torch.equal(one[k].view(torch.uint8), other[k].view(torch.uint8)), k


@pytest.mark.parametrize("T", [1, 8, 70])
def test_dense_pair_against_64_bits(T):
    """The int8 products of the pair, each from its own codes."""
    m = Layer(T, seed=T + 1)
    stream, q, s, ids, w = m.front(*inputs(T, m.H, T))
    out, share, _ = m.block(q, s, ids, w, shared=True)
    o = m.back(stream, out, share)
    torch.cuda.synchronize()
    mm = lambda a, b: torch.mm(b.double(), a.double().t().contiguous()).t()  # noqa: E731
    z = (mm(o["hq"], m.d2).float() * m.d2s * o["hs"][:, None]).to(BF)
    assert torch.equal(o["z"], z)
    h = mm(o["q"], m.d1) * m.d1s.double() * o["q_scale"].double()[:, None]
    gate, up = h[:, :m.dense], h[:, m.dense:]
    want = gate * torch.sigmoid(gate) * up
    # half a step of bf16; gate and up are off by 3 u, silu's slope is under 1.1, exp and its division add 8 u
    tol = 2.0 ** -8 * want.abs() * (1 + 2.0 ** -8) + 16 * U * (want.abs() + gate.abs() * up.abs()) + 1e-38
    assert bool(((o["h"].double() - want).abs() <= tol).all())
    # the codes of h: half a step, and the roundings of v * 127 / a'
    v = o["h"].double() / o["hs"].double()[:, None]
    assert bool(((o["hq"].double() - v).abs() <= 0.5 + 8 * U * v.abs()).all())


def test_two_streams_at_once():
    """Two layers from two threads, each on its own stream."""
    layers = [Layer(24, seed=31), Layer(60, seed=32)]
    ins = [inputs(m.T, m.H, 33 + i) for i, m in enumerate(layers)]

    def whole(i):
        m = layers[i]
        stream, q, s, ids, w = m.front(*ins[i])
        _, share, _ = m.block(q, s, ids, w, shared=True)
        return m.back(stream, m.split(q, s, ids, w), share)
    want = [whole(i) for i in range(2)]
    torch.cuda.synchronize()
    got, errors = [None, None], []

    def work(i):
        try:
            side = torch.cuda.Stream()
            with torch.cuda.stream(side):
                for _ in range(5):
                    got[i] = whole(i)
            side.synchronize()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors, errors
    for a, b in zip(want, got):
        for k in a:
            assert torch.equal(a[k].view(torch.uint8), b[k].view(torch.uint8)), k


def test_decode_step_captured():
    """The back half of a decode step in one graph; two graphs share a
    workspace and run in turn."""
    m = Layer(8, seed=41)
    T, H, K = m.T, m.H, m.K
    stream, q, s, ids, w = m.front(*inputs(T, H, 42))
    out, share, _ = m.block(q, s, ids, w, shared=True)
    d = moe.make_dispatch_dims(T, H, m.E, K, dtype=I8, scale_groups=1)
    ws = torch.empty(256, dtype=torch.uint8, device="cuda")
    cd = moe.make_combine_dims(T, H, K, T * K)
    rows = torch.randn(T * K, H, device="cuda").to(BF)
    results, graphs = [], []
    for seed in (0, 1):
        buf = dict(rows=torch.empty(T * K, H, dtype=I8, device="cuda"), row_scale=torch.empty(T * K, 1, device="cuda"),
                   expert_token_nums=torch.empty(m.E, dtype=torch.int32, device="cuda"),
                   expert_offset=torch.empty(m.E + 1, dtype=torch.int32, device="cuda"),
                   row_of_pair=torch.empty(T, K, dtype=torch.int32, device="cuda"),
                   pair_of_row=torch.empty(T * K, dtype=torch.int32, device="cuda"))
        back = torch.empty(T, H, dtype=BF, device="cuda")

        def step():
            moe.moe_w8a8_dispatch(d, ids, x=q, x_scale=s, workspace=ws, **buf)
            moe.moe_w8a8_combine(cd, rows, buf["row_of_pair"], expert_scales=w, addend=share, out=back)
            return m.back(stream, back, share)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = step()
        results.append(got)
        graphs.append(graph)
    for seed in range(3):
        g = torch.Generator().manual_seed(60 + seed)
        ids.copy_(torch.argsort(torch.rand(T, m.E, generator=g), 1)[:, :K].int())
        rows.copy_(torch.randn(T * K, H, generator=g).to(BF))
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        a = [t.clone() for r in results for t in r.values()]
        dd = moe.moe_w8a8_dispatch(d, ids, x=q, x_scale=s)
        back = moe.moe_w8a8_combine(cd, rows, dd["row_of_pair"], expert_scales=w, addend=share)
        want = m.back(stream, back, share)
        torch.cuda.synchronize()
        half = len(a) // 2
        for i, t in enumerate(want.values()):
            assert torch.equal(a[i].view(torch.uint8), t.view(torch.uint8))
            assert torch.equal(a[half + i].view(torch.uint8), t.view(torch.uint8))
