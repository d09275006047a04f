"""The operators around the block without a GPU: struct layouts, and the calls
that the library or the binding refuses before anything is launched."""
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


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from moe_expert_ffn_route_amd import build
        build.build()
    return binding.library()


@pytest.mark.parametrize("struct,name", [(binding.NormDims, "moe_w8a8_norm_dims_t"),
                                         (binding.GateDims, "moe_w8a8_gate_dims_t"),
                                         (binding.LinearW4Dims, "moe_w8a8_linear_w4_dims_t")])
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


# ------------------------------------------------------------------- norm

def norm(lib, over=None, **kw):
    d = moe.make_norm_dims(4, 512)
    for k, v in (over or {}).items():
        setattr(d, k, v)
    a = dict(x=MB, residual=2 * MB, weight=3 * MB, residual_out=4 * MB, y=5 * MB, q=6 * MB, q_scale=7 * MB)
    a.update(kw)
    return lib.moe_w8a8_norm_quant(ctypes.byref(d), *a.values(), None)


@pytest.mark.parametrize("over,code", [
    (dict(num_tokens=-1), INV), (dict(hidden=0), INV), (dict(dtype=3), INV), (dict(weight_dtype=-1), INV),
    (dict(quant=3), INV), (dict(rms_eps=0.0), INV), (dict(rms_eps=float("nan")), INV), (dict(amax_eps=1e-30), INV),
    (dict(amax_eps=float("inf")), INV), (dict(num_tokens=65537), UNS), (dict(hidden=16385), UNS),
    (dict(weight_dtype=1), UNS), (dict(quant_group=32), UNS), (dict(quant_group=256, hidden=640), UNS),
    (dict(quant_group=-64), UNS)])
def test_norm_refuses_bad_dims(lib, over, code):
    assert norm(lib, over) == code


@pytest.mark.parametrize("kw", [
    dict(x=None), dict(q=None), dict(q_scale=None), dict(residual=None), dict(x=MB + 8), dict(weight=3 * MB + 2),
    dict(q=6 * MB + 8), dict(q_scale=7 * MB + 2),
    dict(residual_out=MB + 512),        # overlaps x without being it
    dict(y=4 * MB), dict(residual_out=2 * MB, y=2 * MB),   # two outputs in one place
    dict(q=MB), dict(q_scale=3 * MB), dict(q=5 * MB + 1024), dict(y=3 * MB)])
def test_norm_refuses_bad_pointers(lib, kw):
    assert norm(lib, **kw) == INV


def test_norm_refuses_codes_without_quant_and_nothing_to_write(lib):
    assert norm(lib, dict(quant=0)) == INV                       # q given
    assert norm(lib, dict(quant=0), q=None, q_scale=None, y=None) == INV
    assert norm(lib, dict(quant=0, quant_group=64), q=None, q_scale=None) == INV
    assert lib.moe_w8a8_norm_quant(None, *[MB] * 7, None) == INV
    assert norm(lib, dict(num_tokens=0), x=None) == OK            # nothing to do


# ------------------------------------------------------------------- gate

def gate(lib, over=None, ws_bytes=1 << 40, **kw):
    d = moe.make_gate_dims(4, 512, 16, 2)
    for k, v in (over or {}).items():
        setattr(d, k, v)
    a = dict(x=MB, weight=2 * MB, bias=3 * MB, ids=4 * MB, scales=5 * MB, workspace=6 * MB)
    a.update(kw)
    return lib.moe_w8a8_gate(ctypes.byref(d), *a.values(), ws_bytes, None)


@pytest.mark.parametrize("over,code", [
    (dict(num_tokens=-1), INV), (dict(hidden=0), INV), (dict(moe_expert_num=0), INV), (dict(topk=0), INV),
    (dict(topk=17), INV), (dict(topk=17, moe_expert_num=32), UNS), (dict(moe_expert_num=1025), UNS),
    (dict(score=3), INV), (dict(score=-1), INV), (dict(normalize=2), INV), (dict(dtype=3), INV),
    (dict(weight_dtype=1), UNS), (dict(hidden=16385), UNS), (dict(num_tokens=65537), UNS),
    (dict(route_scale=float("nan")), INV), (dict(num_tokens=0), OK)])
def test_gate_refuses_bad_dims(lib, over, code):
    assert gate(lib, over) == code
    if code != OK:
        d = moe.make_gate_dims(4, 512, 16, 2)
        for k, v in over.items():
            setattr(d, k, v)
        n = ctypes.c_size_t(0)
        assert lib.moe_w8a8_gate_workspace_size(ctypes.byref(d), ctypes.byref(n)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INV), (dict(weight=None), INV), (dict(ids=None), INV), (dict(scales=None), INV),
    (dict(workspace=None), WSP), (dict(ws_bytes=16), WSP), (dict(workspace=6 * MB + 16), INV), (dict(x=MB + 8), INV),
    (dict(weight=2 * MB + 4), INV), (dict(ids=4 * MB + 2), INV), (dict(bias=3 * MB + 1), INV),
    (dict(ids=MB), INV), (dict(scales=4 * MB), INV), (dict(workspace=2 * MB), INV), (dict(scales=3 * MB), INV)])
def test_gate_refuses_bad_pointers(lib, kw, code):
    assert gate(lib, **kw) == code


def test_gate_workspace_size(lib):
    assert lib.moe_w8a8_gate_workspace_size(None, ctypes.byref(ctypes.c_size_t())) == INV
    assert lib.moe_w8a8_gate_workspace_size(ctypes.byref(moe.make_gate_dims(4, 512, 16, 2)), None) == INV
    assert moe.moe_w8a8_gate_workspace_size(moe.make_gate_dims(8, 4096, 256, 8)) >= 8 * 256 * 8
    assert moe.moe_w8a8_gate_workspace_size(moe.make_gate_dims(0, 4096, 256, 8)) >= 0


@pytest.mark.parametrize("H,E", [(1, 1), (4096, 256), (2501, 72), (16384, 1024), (700, 1024)])
def test_gate_workspace_for_the_largest_batch_serves_all(lib, H, E):
    """Its size grows with T, and holds plan_of's parts of the logits and norms."""
    last = 0
    for T in [*range(0, 5000), *range(5000, 65537, 53), 65536]:
        n = moe.moe_w8a8_gate_workspace_size(moe.make_gate_dims(T, H, E, 1))
        assert n >= last
        few = T <= 16 or (H >= 512 and T * E * H <= 2 ** 28)
        rows, chunks = 16 if few else 64, -(-H // 128)
        tiles = -(-T // rows) * -(-E // rows)
        if T:
            parts = max(1, min(8, -(-512 // tiles), chunks // (8 if few else 2)))
            parts = -(-chunks // -(-chunks // parts))
            assert n >= parts * (8 * T * E + 4 * (T + E))
        last = n


# ------------------------------------------------------------- 4-bit linear

def w4_dims(**over):
    d = moe.make_linear_w4_dims(4, 64, 256)
    for k, v in over.items():
        setattr(d, k, v)
    return d


@pytest.mark.parametrize("over,code", [
    (dict(num_tokens=-1), INV), (dict(out_features=0), INV), (dict(in_features=0), INV), (dict(gated=2), INV),
    (dict(has_zeros=-1), INV), (dict(gated=1, out_features=63), INV), (dict(group=16), UNS), (dict(group=256), UNS),
    (dict(act_dtype=2), UNS), (dict(act_dtype=-1), UNS), (dict(in_features=320), INV),
    (dict(num_tokens=65537), UNS), (dict(out_features=(1 << 20) + 1), UNS), (dict(in_features=1 << 18), UNS),
    (dict(out_features=1 << 20, in_features=1 << 17), UNS)])
def test_w4_refuses_bad_dims(lib, over, code):
    d, n = w4_dims(**over), ctypes.c_size_t(0)
    assert lib.moe_w8a8_packed_w4_bytes(ctypes.byref(d), ctypes.byref(n)) == code
    assert lib.moe_w8a8_linear_w4(ctypes.byref(d), MB, None, 2 * MB, None, 3 * MB, None) == code
    assert lib.moe_w8a8_pack_weights_w4(ctypes.byref(d), MB, 2 * MB, None, 3 * MB, None) == code


def test_w4_packed_bytes(lib):
    # 1024 bytes of codes per 16 rows x 128 k, 4 bytes of scale (and 1 of zero point) per row and group
    assert moe.moe_w8a8_packed_w4_bytes(w4_dims()) == 4 * 2 * (1024 + 16 * 4)
    assert moe.moe_w8a8_packed_w4_bytes(w4_dims(group=32, has_zeros=1)) == 4 * 2 * (1024 + 4 * 16 * 5)
    assert moe.moe_w8a8_packed_w4_bytes(w4_dims(out_features=65, in_features=128)) == 5 * (1024 + 64)
    assert moe.moe_w8a8_packed_w4_bytes(w4_dims(out_features=34, gated=1, group=32, in_features=96)) == 3 * (1024 + 256)
    assert lib.moe_w8a8_packed_w4_bytes(ctypes.byref(w4_dims()), None) == INV
    assert lib.moe_w8a8_packed_w4_bytes(None, ctypes.byref(ctypes.c_size_t())) == INV


@pytest.mark.parametrize("over,kw", [
    ({}, dict(x=None)), ({}, dict(weight=None)), ({}, dict(out=None)), ({}, dict(x=MB + 8)),
    ({}, dict(weight=2 * MB + 8)), ({}, dict(out=3 * MB + 2)), ({}, dict(bias=4 * MB + 1)),
    ({}, dict(x_scale=5 * MB)),                       # scales without int8 x
    (dict(act_dtype=3), {}),                          # int8 x without scales
    ({}, dict(out=MB)), ({}, dict(out=2 * MB + 1024)), ({}, dict(bias=3 * MB))])
def test_w4_refuses_bad_pointers(lib, over, kw):
    a = dict(x=MB, x_scale=None, weight=2 * MB, bias=None, out=3 * MB)
    a.update(kw)
    assert lib.moe_w8a8_linear_w4(ctypes.byref(w4_dims(**over)), *a.values(), None) == INV


def test_w4_nothing_to_do(lib):
    assert lib.moe_w8a8_linear_w4(ctypes.byref(w4_dims(num_tokens=0)), None, None, MB, None, None, None) == OK


@pytest.mark.parametrize("over,kw", [
    ({}, dict(codes=None)), ({}, dict(scale=None)), ({}, dict(dst=None)), ({}, dict(zero=3 * MB)),
    (dict(has_zeros=1), {}), ({}, dict(dst=4 * MB + 8)), ({}, dict(scale=2 * MB + 2)), ({}, dict(dst=MB)),
    ({}, dict(dst=2 * MB)), (dict(has_zeros=1), dict(zero=4 * MB))])
def test_w4_pack_refuses_bad_pointers(lib, over, kw):
    a = dict(codes=MB, scale=2 * MB, zero=None, dst=4 * MB)
    a.update(kw)
    assert lib.moe_w8a8_pack_weights_w4(ctypes.byref(w4_dims(**over)), *a.values(), None) == INV


# ------------------------------------------------------- block on given codes

@pytest.mark.parametrize("kw,code", [
    (dict(q_x=None), INV), (dict(x_scale=None), INV), (dict(x_scale=MB + 4), INV), (dict(q_x=MB + 8), INV),
    (dict(expert_ids=None), INV), (dict(output=None), INV), (dict(workspace=None), WSP)])
def test_forward_quantized_refuses_bad_arguments(lib, kw, code):
    d = moe.make_dims(num_tokens=8, hidden=512, inter=256, topk=2, moe_expert_num=8)
    names = ["q_x", "x_scale", "expert_ids", "expert_scales", "w1", "w1s", "w2", "w2s", "s1", "s1s", "s2", "s2s",
             "mask", "output", "share_output", "expert_token_nums", "workspace"]
    a = {n: None if n in ("s1", "s1s", "s2", "s2s", "mask", "share_output") else MB for n in names}
    a.update(kw)
    assert lib.moe_w8a8_forward_quantized(ctypes.byref(d), *a.values(), 1 << 40, None, None) == code
    assert lib.moe_w8a8_forward_quantized(None, *a.values(), 1 << 40, None, None) == INV


# --------------------------------------------------------------- the binding

def test_binding_refuses_host_tensors_and_misfits(lib):
    d = moe.make_norm_dims(2, 64)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_w8a8_norm_quant(d, x, y=x)
    with pytest.raises(ValueError, match="x: expected 128 elements"):
        moe.moe_w8a8_norm_quant(d, x.float(), y=x)
    with pytest.raises(ValueError, match="x: expected 128 elements"):
        moe.moe_w8a8_norm_quant(d, x[:1], y=x)
    with pytest.raises(ValueError, match="element type"):
        moe.make_norm_dims(2, 64, dtype=torch.float64)
    with pytest.raises(ValueError, match="GPU"):
        moe.moe_w8a8_linear_w4(moe.make_linear_w4_dims(2, 16, 64, group=64), x, torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(moe.MoeError):
        moe.moe_w8a8_packed_w4_bytes(moe.make_linear_w4_dims(2, 16, 64, group=0))
    with pytest.raises(moe.MoeError):
        moe.moe_w8a8_gate(moe.make_gate_dims(2, 64, 4, 5), x, x)
    with pytest.raises(ValueError, match="expected a tensor"):
        moe.moe_w8a8_norm_quant(d, x.data_ptr(), y=x)
    with pytest.raises(ValueError, match="dims"):
        moe.moe_w8a8_norm_quant(moe.make_gate_dims(2, 64, 4, 2), x, y=x)


def test_binding_refuses_what_is_no_tensor_where_outputs_are_allocated(lib):
    g, ld = moe.make_gate_dims(2, 64, 4, 2), moe.make_linear_w4_dims(2, 16, 64, group=64)
    for x in (None, 4096, [1.0]):
        with pytest.raises(ValueError, match="expected a tensor"):
            moe.moe_w8a8_gate(g, x, x)
        with pytest.raises(ValueError, match="expected a tensor"):
            moe.moe_w8a8_linear_w4(ld, x, x)
        with pytest.raises(ValueError, match="expected a tensor"):
            moe.moe_w8a8_pack_weights_w4(ld, x, x)
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="expected a tensor"):
        moe.moe_w8a8_gate(g, x, x, workspace=4096)
    with pytest.raises(ValueError, match="expected a tensor"):
        moe.moe_w8a8_pack_weights_w4(ld, torch.zeros(16, 32, dtype=torch.uint8), 4096)


def test_binding_reports_bad_dims_where_outputs_are_allocated(lib):
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError):
        moe.moe_w8a8_gate(moe.make_gate_dims(-1, 64, 4, 2), x, x)
    with pytest.raises(moe.MoeError):
        moe.moe_w8a8_linear_w4(moe.make_linear_w4_dims(-1, 16, 64, group=64), x, x)


def test_missing_python_entry_says_how_to_build_it(lib, monkeypatch):
    import sys
    monkeypatch.setattr(binding, "_pycall", None)
    monkeypatch.setitem(sys.modules, "moe_expert_ffn_route_amd._pycall", None)
    monkeypatch.delattr(moe, "_pycall", raising=False)
    with pytest.raises(ImportError, match="python -m moe_expert_ffn_route_amd.build"):
        moe.moe_w8a8_norm_quant(moe.make_norm_dims(2, 64), torch.zeros(2, 64, dtype=torch.bfloat16))
