"""The operators between the block and the rest of a program without a GPU:
struct layouts, and the calls that the library or the binding refuses before
anything is launched."""
import ctypes
import os
import subprocess

import pytest
import torch

import moe_expert_ffn_route_amd as moe
from moe_expert_ffn_route_amd import binding

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INV, UNS, WSP, OK = (binding.MOE_ERR_INVALID_ARG, binding.MOE_ERR_UNSUPPORTED, binding.MOE_ERR_WORKSPACE,
                     binding.MOE_OK)
MB = 1 << 20  # fake, 256-aligned device addresses are multiples of it; never dereferenced
NAN = float("nan")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from moe_expert_ffn_route_amd import build
        build.build()
    return binding.library()


@pytest.mark.parametrize("struct,name", [(binding.LinearW8Dims, "moe_w8a8_linear_w8_dims_t"),
                                         (binding.QuantDims, "moe_w8a8_quant_dims_t"),
                                         (binding.JoinNormDims, "moe_w8a8_join_norm_dims_t"),
                                         (binding.DispatchDims, "moe_w8a8_dispatch_dims_t"),
                                         (binding.CombineDims, "moe_w8a8_combine_dims_t")])
def test_struct_layout_matches_header(tmp_path, struct, name):
    fields = [f for f, _ in struct._fields_]
    prog = ['#include <stdio.h>', '#include <stddef.h>', '#include "moe_w8a8.h"', 'int main(void){',
            f'printf("%zu\\n", sizeof({name}));']
    prog += [f'printf("%zu\\n", offsetof({name}, {f}));' for f in fields] + ['return 0;}']
    src = tmp_path / "layout.c"
    src.write_text("\n".join(prog))
    subprocess.check_call(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "layout")])
    vals = [int(v) for v in subprocess.check_output([str(tmp_path / "layout")]).split()]
    assert vals[0] == ctypes.sizeof(struct)
    assert vals[1:] == [getattr(struct, f).offset for f in fields]


def changed(d, over):
    for k, v in (over or {}).items():
        setattr(d, k, v)
    return d


# ------------------------------------------------------------- int8 products

def w8_dims(**over):
    return changed(moe.make_linear_w8_dims(4, 64, 256), over)


@pytest.mark.parametrize("over,code", [
    (dict(num_tokens=-1), INV), (dict(out_features=0), INV), (dict(in_features=0), INV), (dict(gated=2), INV),
    (dict(gated=1, out_features=63), INV), (dict(out_dtype=3), INV), (dict(out_dtype=-1), INV),
    (dict(num_tokens=65537), UNS), (dict(out_features=(1 << 20) + 1), UNS), (dict(in_features=(1 << 16) + 1), UNS),
    (dict(out_features=1 << 20, in_features=1 << 16), UNS)])
def test_w8_refuses_bad_dims(lib, over, code):
    d, n = w8_dims(**over), ctypes.c_size_t(0)
    assert lib.moe_w8a8_packed_w8_bytes(ctypes.byref(d), ctypes.byref(n)) == code
    assert lib.moe_w8a8_linear_w8(ctypes.byref(d), MB, 2 * MB, 3 * MB, None, 4 * MB, None) == code
    assert lib.moe_w8a8_pack_weights_w8(ctypes.byref(d), MB, 2 * MB, 3 * MB, None) == code


def test_w8_packed_bytes(lib):
    # 2048 bytes of codes per 16 rows x 128 k, 4 bytes of scale per row
    assert moe.moe_w8a8_packed_w8_bytes(w8_dims()) == 4 * 2 * 2048 + 64 * 4
    assert moe.moe_w8a8_packed_w8_bytes(w8_dims(out_features=65, in_features=129)) == 5 * (2 * 2048 + 64)
    assert moe.moe_w8a8_packed_w8_bytes(w8_dims(out_features=34, gated=1, in_features=1)) == 3 * (2048 + 64)
    assert lib.moe_w8a8_packed_w8_bytes(ctypes.byref(w8_dims()), None) == INV
    assert lib.moe_w8a8_packed_w8_bytes(None, ctypes.byref(ctypes.c_size_t())) == INV


@pytest.mark.parametrize("kw", [dict(x=None), dict(x_scale=None), dict(weight=None), dict(out=None), dict(x=MB + 8),
                                dict(x_scale=2 * MB + 2), dict(weight=3 * MB + 8), dict(out=4 * MB + 2),
                                dict(bias=5 * MB + 1), dict(out=MB), dict(out=2 * MB), dict(out=3 * MB + 16384),
                                dict(bias=4 * MB + 64)])
def test_w8_refuses_bad_pointers(lib, kw):
    a = dict(x=MB, x_scale=2 * MB, weight=3 * MB, bias=None, out=4 * MB)
    a.update(kw)
    assert lib.moe_w8a8_linear_w8(ctypes.byref(w8_dims()), *a.values(), None) == INV


@pytest.mark.parametrize("kw", [dict(codes=None), dict(scale=None), dict(dst=None), dict(dst=3 * MB + 8),
                                dict(scale=2 * MB + 2), dict(dst=MB), dict(dst=2 * MB)])
def test_w8_pack_refuses_bad_pointers(lib, kw):
    a = dict(codes=MB, scale=2 * MB, dst=3 * MB)
    a.update(kw)
    assert lib.moe_w8a8_pack_weights_w8(ctypes.byref(w8_dims()), *a.values(), None) == INV


# ------------------------------------------------------------------ quantiser

def quant(lib, over=None, **kw):
    d = changed(moe.make_quant_dims(4, 512), over)
    a = dict(x=MB, smooth=2 * MB, q=3 * MB, q_scale=4 * MB)
    a.update(kw)
    return lib.moe_w8a8_quant(ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(num_tokens=-1), INV), (dict(hidden=0), INV), (dict(dtype=3), INV), (dict(quant=0), INV), (dict(quant=3), INV),
    (dict(amax_eps=1e-30), INV), (dict(amax_eps=NAN), INV), (dict(num_tokens=65537), UNS), (dict(hidden=16385), UNS),
    (dict(quant_group=32), UNS), (dict(quant_group=256, hidden=640), UNS), (dict(num_tokens=0), OK)])
def test_quant_refuses_bad_dims(lib, over, code):
    assert quant(lib, over) == code


@pytest.mark.parametrize("kw", [dict(x=None), dict(q=None), dict(q_scale=None), dict(x=MB + 8), dict(smooth=2 * MB + 4),
                                dict(q=3 * MB + 8), dict(q_scale=4 * MB + 2), dict(q=MB), dict(q_scale=3 * MB + 2044),
                                dict(q=2 * MB), dict(q_scale=2 * MB)])
def test_quant_refuses_bad_pointers(lib, kw):
    assert quant(lib, **kw) == INV


# --------------------------------------------------------------- joining norm

def join(lib, over=None, **kw):
    d = changed(moe.make_join_norm_dims(4, 512, post_norm=True, gate_rows=1), over)
    a = dict(block=MB, share=2 * MB, share_scale=3 * MB, residual=4 * MB, post_weight=5 * MB, gate=6 * MB, weight=7 * MB,
             residual_out=8 * MB, y=9 * MB, q=10 * MB, q_scale=11 * MB)
    a.update(kw)
    return lib.moe_w8a8_join_norm(ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(num_tokens=-1), INV), (dict(hidden=0), INV), (dict(dtype=3), INV), (dict(weight_dtype=3), INV),
    (dict(weight_dtype=1), UNS), (dict(post_norm=2), INV), (dict(gate_rows=2), INV), (dict(gate_rows=-1), INV),
    (dict(quant=3), INV), (dict(post_eps=0.0), INV), (dict(rms_eps=NAN), INV), (dict(amax_eps=0.0), INV),
    (dict(residual_scale=float("inf")), INV), (dict(branch_scale=NAN), INV), (dict(num_tokens=65537), UNS),
    (dict(hidden=16385), UNS), (dict(quant_group=100), UNS), (dict(num_tokens=0), OK), (dict(num_tokens=0, gate_rows=7), OK),
    (dict(post_norm=0), INV),            # a post weight without the norm
    (dict(gate_rows=0), INV),            # a gate that gate_rows denies
    (dict(quant=0), INV),                # codes that quant denies
    (dict(quant=0, quant_group=64), INV)])
def test_join_refuses_bad_dims(lib, over, code):
    assert join(lib, over) == code


@pytest.mark.parametrize("kw", [
    dict(block=None), dict(share=None), dict(gate=None), dict(q=None), dict(q_scale=None), dict(block=MB + 8),
    dict(share_scale=3 * MB + 2), dict(residual=4 * MB + 4), dict(gate=6 * MB + 2), dict(q=10 * MB + 8),
    dict(residual_out=MB + 1024), dict(y=8 * MB), dict(residual_out=4 * MB, y=4 * MB), dict(y=6 * MB), dict(q=MB),
    dict(q_scale=3 * MB), dict(residual_out=7 * MB), dict(q=9 * MB + 2048)])
def test_join_refuses_bad_pointers(lib, kw):
    assert join(lib, **kw) == INV


def test_join_refuses_nothing_to_write(lib):
    assert join(lib, dict(quant=0), q=None, q_scale=None, y=None, residual_out=None) == INV
    assert lib.moe_w8a8_join_norm(None, *[MB] * 11, None) == INV


# ------------------------------------------------------------------- dispatch

def dispatch(lib, over=None, ws_bytes=1 << 40, **kw):
    d = changed(moe.make_dispatch_dims(4, 512, 16, 2, scale_groups=2), over)
    a = dict(ids=MB, x=2 * MB, x_scale=3 * MB, mask=4 * MB, rows=5 * MB, row_scale=6 * MB, nums=7 * MB, offset=8 * MB,
             row_of_pair=9 * MB, pair_of_row=10 * MB, workspace=11 * MB)
    a.update(kw)
    return lib.moe_w8a8_dispatch(ctypes.byref(d), *a.values(), ws_bytes, None)


@pytest.mark.parametrize("over,code", [
    (dict(num_tokens=-1), INV), (dict(topk=0), INV), (dict(moe_expert_num=0), INV), (dict(hidden=0), INV),
    (dict(dtype=4), INV), (dict(dtype=-1), INV), (dict(scale_groups=-1), INV), (dict(row_align=0), INV),
    (dict(row_align=3), INV), (dict(row_align=-4), INV), (dict(num_tokens=65537), UNS), (dict(topk=17), UNS),
    (dict(moe_expert_num=1025), UNS), (dict(hidden=16385), UNS), (dict(scale_groups=257), UNS), (dict(row_align=512), UNS)])
def test_dispatch_refuses_bad_dims(lib, over, code):
    assert dispatch(lib, over) == code
    d = changed(moe.make_dispatch_dims(4, 512, 16, 2), over)
    assert lib.moe_w8a8_dispatch_rows(ctypes.byref(d), ctypes.byref(ctypes.c_int64())) == code
    assert lib.moe_w8a8_dispatch_workspace_size(ctypes.byref(d), ctypes.byref(ctypes.c_size_t())) == code


@pytest.mark.parametrize("over,kw,code", [
    ({}, dict(ids=None), INV), ({}, dict(x=None), INV), ({}, dict(rows=None), INV), ({}, dict(x_scale=None), INV),
    ({}, dict(row_scale=None), INV), (dict(scale_groups=0), {}, INV), ({}, dict(x=None, rows=None), INV),
    ({}, dict(nums=None), INV), ({}, dict(offset=None), INV), ({}, dict(row_of_pair=None), INV),
    ({}, dict(pair_of_row=None), INV), ({}, dict(x=2 * MB + 8), INV), ({}, dict(rows=5 * MB + 8), INV),
    ({}, dict(ids=MB + 2), INV), ({}, dict(offset=8 * MB + 1), INV), ({}, dict(rows=2 * MB), INV),
    ({}, dict(nums=MB), INV), ({}, dict(offset=7 * MB), INV), ({}, dict(pair_of_row=9 * MB), INV),
    ({}, dict(row_scale=5 * MB + 512), INV), ({}, dict(nums=4 * MB), INV),
    (dict(num_tokens=4096), dict(workspace=None, x=None, rows=None, x_scale=None, row_scale=None), WSP),
    (dict(num_tokens=4096), dict(ws_bytes=16, x=None, rows=None, x_scale=None, row_scale=None), WSP),
    (dict(num_tokens=4096), dict(workspace=11 * MB + 16, x=None, rows=None, x_scale=None, row_scale=None), INV)])
def test_dispatch_refuses_bad_pointers(lib, over, kw, code):
    assert dispatch(lib, over, **kw) == code


def test_dispatch_rows(lib):
    rows = lambda **kw: moe.moe_w8a8_dispatch_rows(changed(moe.make_dispatch_dims(4, 512, 16, 2), kw))  # noqa: E731
    assert rows() == 8
    assert rows(row_align=16) == 8 + 8 * 15                  # every pair an expert of its own
    assert rows(row_align=16, num_tokens=100) == 200 + 16 * 15
    assert rows(num_tokens=0, row_align=64) == 0
    assert rows(num_tokens=65536, topk=16, moe_expert_num=1024, row_align=256) == (1 << 20) + 1024 * 255


def test_dispatch_workspace_for_the_largest_batch_serves_all(lib):
    for E in (1, 72, 1024):
        for K in (1, 6, 16):
            last = 0
            for T in [*range(0, 3000, 7), *range(3000, 65537, 613), 65536]:
                n = moe.moe_w8a8_dispatch_workspace_size(moe.make_dispatch_dims(T, 64, E, K))
                assert n >= last
                last = n


# ------------------------------------------------------------ combine and back

def combine(lib, over=None, **kw):
    d = changed(moe.make_combine_dims(4, 512, 2, 8), over)
    a = dict(rows=MB, row_of_pair=2 * MB, scales=3 * MB, addend=4 * MB, out=5 * MB)
    a.update(kw)
    return lib.moe_w8a8_combine(ctypes.byref(d), *a.values(), None)


def grad(lib, over=None, **kw):
    d = changed(moe.make_combine_dims(4, 512, 2, 8), over)
    a = dict(dout=MB, row_of_pair=2 * MB, pair_of_row=3 * MB, rows=4 * MB, scales=5 * MB, drows=6 * MB, dscales=7 * MB)
    a.update(kw)
    return lib.moe_w8a8_combine_grad(ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(num_tokens=-1), INV), (dict(topk=0), INV), (dict(hidden=0), INV), (dict(num_rows=-1), INV), (dict(dtype=3), INV),
    (dict(out_dtype=3), INV), (dict(out_dtype=1), UNS), (dict(dtype=2), UNS), (dict(topk=17), UNS),
    (dict(num_tokens=65537), UNS), (dict(hidden=16385), UNS), (dict(num_rows=(1 << 22) + 1), UNS), (dict(num_tokens=0), OK)])
def test_combine_refuses_bad_dims(lib, over, code):
    assert combine(lib, over) == code
    # (without tokens drows is written all the same: zeros)
    assert grad(lib, over, **({} if code != OK else dict(drows=None))) == code
    if code == OK:
        assert grad(lib, dict(over, num_rows=0)) == OK
        assert grad(lib, over, drows=6 * MB + 8) == INV


@pytest.mark.parametrize("kw", [dict(rows=None), dict(row_of_pair=None), dict(out=None), dict(rows=MB + 8),
                                dict(row_of_pair=2 * MB + 2), dict(scales=3 * MB + 1), dict(addend=4 * MB + 8),
                                dict(out=5 * MB + 4), dict(out=MB), dict(out=2 * MB), dict(out=3 * MB), dict(out=4 * MB + 64)])
def test_combine_refuses_bad_pointers(lib, kw):
    assert combine(lib, **kw) == INV


@pytest.mark.parametrize("kw", [dict(dout=None), dict(row_of_pair=None), dict(pair_of_row=None), dict(rows=None),
                                dict(dscales=None), dict(drows=None, dscales=None), dict(dout=MB + 8),
                                dict(drows=6 * MB + 8), dict(dscales=7 * MB + 2), dict(drows=4 * MB), dict(drows=MB),
                                dict(dscales=5 * MB), dict(dscales=6 * MB), dict(drows=2 * MB), dict(dscales=3 * MB)])
def test_combine_grad_refuses_bad_pointers(lib, kw):
    assert grad(lib, **kw) == INV


# --------------------------------------------------------------- the binding

def test_binding_refuses_host_tensors_and_misfits(lib):
    x = torch.zeros(2, 64, dtype=torch.int8)
    s = torch.zeros(2)
    w = torch.zeros(moe.moe_w8a8_packed_w8_bytes(moe.make_linear_w8_dims(2, 16, 64)), dtype=torch.uint8)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_w8a8_linear_w8(moe.make_linear_w8_dims(2, 16, 64), x, s, w)
    with pytest.raises(ValueError, match="x: expected 128 elements"):
        moe.moe_w8a8_linear_w8(moe.make_linear_w8_dims(2, 16, 64), x.float(), s, w)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_w8a8_quant(moe.make_quant_dims(2, 64), x.bfloat16())
    with pytest.raises(ValueError, match="dims"):
        moe.moe_w8a8_quant(moe.make_linear_w8_dims(2, 16, 64), x.bfloat16(), q=x, q_scale=s)
    with pytest.raises(ValueError, match="block: expected 128 elements"):
        moe.moe_w8a8_join_norm(moe.make_join_norm_dims(2, 64), x, y=x)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_w8a8_dispatch(moe.make_dispatch_dims(2, 64, 4, 2), torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_w8a8_combine(moe.make_combine_dims(2, 64, 2, 4), torch.zeros(4, 64, dtype=torch.bfloat16),
                             torch.zeros(2, 2, dtype=torch.int32))
    with pytest.raises(ValueError, match="dout: expected 128 elements"):
        moe.moe_w8a8_combine_grad(moe.make_combine_dims(2, 64, 2, 4), x, None, None)
    for t in (None, 4096, [1.0]):
        for call in (lambda: moe.moe_w8a8_linear_w8(moe.make_linear_w8_dims(2, 16, 64), t, s, w),
                     lambda: moe.moe_w8a8_quant(moe.make_quant_dims(2, 64), t),
                     lambda: moe.moe_w8a8_join_norm(moe.make_join_norm_dims(2, 64), t),
                     lambda: moe.moe_w8a8_dispatch(moe.make_dispatch_dims(2, 64, 4, 2), t),
                     lambda: moe.moe_w8a8_combine(moe.make_combine_dims(2, 64, 2, 4), t, s),
                     lambda: moe.moe_w8a8_combine_grad(moe.make_combine_dims(2, 64, 2, 4), t, s, s),
                     lambda: moe.moe_w8a8_pack_weights_w8(moe.make_linear_w8_dims(2, 16, 64), t, s)):
            with pytest.raises(ValueError, match="expected a tensor"):
                call()


def test_binding_reports_bad_dims_where_outputs_are_allocated(lib):
    x, ids = torch.zeros(2, 64, dtype=torch.int8), torch.zeros(2, 2, dtype=torch.int32)
    for call in (lambda: moe.moe_w8a8_linear_w8(moe.make_linear_w8_dims(-1, 16, 64), x, x, x),
                 lambda: moe.moe_w8a8_linear_w8(changed(moe.make_linear_w8_dims(2, 16, 64), dict(out_dtype=9)), x, x, x),
                 lambda: moe.moe_w8a8_quant(moe.make_quant_dims(-1, 64), x),
                 lambda: moe.moe_w8a8_quant(moe.make_quant_dims(2, 64, quant_group=60), x),
                 lambda: moe.moe_w8a8_dispatch(moe.make_dispatch_dims(2, 64, 4, 2, row_align=3), ids),
                 lambda: moe.moe_w8a8_combine(moe.make_combine_dims(-1, 64, 2, 4), x, ids)):
        with pytest.raises(moe.MoeError):
            call()
