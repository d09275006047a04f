"""ctypes binding of libmoe_w8a8 (include/moe_w8a8.h).

The entry points keep the C names: `moe_w8a8_workspace_size`,
`moe_w8a8_forward`, `moe_w8a8_status_string`. This module only marshals
arguments (torch device tensors -> device pointers, the current HIP stream);
every step of the block runs in the library's HIP kernels. There is no other
backend: if the library is missing, loading raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_w8a8.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = 0, -1, -2, -3, -4
MOE_ERR_SCRATCH_LIMIT = -5
NOALLOC_SCRATCH_BYTES = 32 << 20  # MOE_W8A8_NOALLOC_SCRATCH_BYTES

EXPORTS = ("moe_w8a8_workspace_size", "moe_w8a8_forward", "moe_w8a8_forward_noalloc", "moe_w8a8_pack_weights",
           "moe_w8a8_packed_mx_bytes", "moe_w8a8_pack_weights_mx", "moe_w8a8_warm", "moe_w8a8_read_probe",
           "moe_w8a8_read_write_probe", "moe_w8a8_status_string", "moe_w8a8_forward_quantized", "moe_w8a8_norm_quant",
           "moe_w8a8_gate_workspace_size", "moe_w8a8_gate", "moe_w8a8_packed_w4_bytes", "moe_w8a8_pack_weights_w4",
           "moe_w8a8_linear_w4", "moe_w8a8_packed_w8_bytes", "moe_w8a8_pack_weights_w8", "moe_w8a8_linear_w8",
           "moe_w8a8_quant", "moe_w8a8_join_norm", "moe_w8a8_dispatch_rows", "moe_w8a8_dispatch_workspace_size",
           "moe_w8a8_dispatch", "moe_w8a8_combine", "moe_w8a8_combine_grad")
MOE_WEIGHT_ROW_MAJOR, MOE_WEIGHT_PACKED = 0, 1
MOE_WEIGHT_INT8, MOE_WEIGHT_MXFP4 = 0, 1
MOE_PACK_GMM1, MOE_PACK_GMM2 = 1, 2
MOE_DTYPE_BF16, MOE_DTYPE_FP16, MOE_DTYPE_FP32, MOE_DTYPE_INT8 = 0, 1, 2, 3
MOE_QUANT_NONE, MOE_QUANT_INT8, MOE_QUANT_E4M3 = 0, 1, 2
MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID, MOE_SCORE_SQRT_SOFTPLUS = 0, 1, 2
_DTYPE_CODE = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_FP16, torch.float32: MOE_DTYPE_FP32,
               torch.int8: MOE_DTYPE_INT8}


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {moe_w8a8_status_string(code)} ({code})")
        self.code = code


class Dims(ctypes.Structure):
    """moe_w8a8_dims_t"""
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("inter", ctypes.c_int32),
                ("share_inter", ctypes.c_int32), ("topk", ctypes.c_int32), ("moe_expert_num", ctypes.c_int32),
                ("ep_rank_size", ctypes.c_int32), ("ep_rank_id", ctypes.c_int32), ("quant_mode", ctypes.c_int32),
                ("amax_eps", ctypes.c_float), ("weight_layout", ctypes.c_int32),
                ("fuse_route_scale", ctypes.c_int32), ("weight_format", ctypes.c_int32),
                ("quant_group", ctypes.c_int32), ("requant_in_epilogue", ctypes.c_int32)]

    @property
    def e_loc(self) -> int:
        return self.moe_expert_num // self.ep_rank_size


class NormDims(ctypes.Structure):
    """moe_w8a8_norm_dims_t"""
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("quant", ctypes.c_int32), ("quant_group", ctypes.c_int32),
                ("rms_eps", ctypes.c_float), ("amax_eps", ctypes.c_float)]


class GateDims(ctypes.Structure):
    """moe_w8a8_gate_dims_t"""
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("moe_expert_num", ctypes.c_int32),
                ("topk", ctypes.c_int32), ("score", ctypes.c_int32), ("normalize", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("weight_dtype", ctypes.c_int32), ("route_scale", ctypes.c_float)]


class LinearW4Dims(ctypes.Structure):
    """moe_w8a8_linear_w4_dims_t"""
    _fields_ = [("num_tokens", ctypes.c_int32), ("out_features", ctypes.c_int32), ("in_features", ctypes.c_int32),
                ("group", ctypes.c_int32), ("act_dtype", ctypes.c_int32), ("gated", ctypes.c_int32),
                ("has_zeros", ctypes.c_int32)]


class LinearW8Dims(ctypes.Structure):
    """moe_w8a8_linear_w8_dims_t"""
    _fields_ = [("num_tokens", ctypes.c_int32), ("out_features", ctypes.c_int32), ("in_features", ctypes.c_int32),
                ("out_dtype", ctypes.c_int32), ("gated", ctypes.c_int32)]


class QuantDims(ctypes.Structure):
    """moe_w8a8_quant_dims_t"""
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("quant", ctypes.c_int32), ("quant_group", ctypes.c_int32), ("amax_eps", ctypes.c_float)]


class JoinNormDims(ctypes.Structure):
    """moe_w8a8_join_norm_dims_t"""
    _fields_ = [("num_tokens", ctypes.c_int32), ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("weight_dtype", ctypes.c_int32), ("post_norm", ctypes.c_int32), ("gate_rows", ctypes.c_int32),
                ("quant", ctypes.c_int32), ("quant_group", ctypes.c_int32), ("residual_scale", ctypes.c_float),
                ("branch_scale", ctypes.c_float), ("post_eps", ctypes.c_float), ("rms_eps", ctypes.c_float),
                ("amax_eps", ctypes.c_float)]


class DispatchDims(ctypes.Structure):
    """moe_w8a8_dispatch_dims_t"""
    _fields_ = [("num_tokens", ctypes.c_int32), ("topk", ctypes.c_int32), ("moe_expert_num", ctypes.c_int32),
                ("hidden", ctypes.c_int32), ("dtype", ctypes.c_int32), ("scale_groups", ctypes.c_int32),
                ("row_align", ctypes.c_int32)]


class CombineDims(ctypes.Structure):
    """moe_w8a8_combine_dims_t"""
    _fields_ = [("num_tokens", ctypes.c_int32), ("topk", ctypes.c_int32), ("hidden", ctypes.c_int32),
                ("num_rows", ctypes.c_int32), ("dtype", ctypes.c_int32), ("out_dtype", ctypes.c_int32)]


DEBUG_FIELDS = ("sorted_pair", "row_of_pair", "group_offset", "shared_token", "num_rows", "q_x", "xs", "acc1",
                "h", "q_h", "hs", "acc2", "z", "stage_events", "kernel_events")
STAGES = ("route_quant", "gemm1", "requant", "gemm2", "combine")


class Debug(ctypes.Structure):
    """moe_w8a8_debug_t"""
    _fields_ = [(n, ctypes.c_void_p) for n in DEBUG_FIELDS]


_lib = None


def library() -> ctypes.CDLL:
    """Open libmoe_w8a8.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with `python -m moe_expert_ffn_route_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        P = ctypes.c_void_p
        L.moe_w8a8_workspace_size.restype = ctypes.c_int
        L.moe_w8a8_workspace_size.argtypes = [ctypes.POINTER(Dims), ctypes.POINTER(ctypes.c_size_t)]
        L.moe_w8a8_forward.restype = ctypes.c_int
        L.moe_w8a8_forward.argtypes = ([ctypes.POINTER(Dims)] + [P] * 18 + [ctypes.c_size_t, ctypes.POINTER(Debug), P])
        L.moe_w8a8_forward_noalloc.restype = ctypes.c_int
        L.moe_w8a8_forward_noalloc.argtypes = [ctypes.POINTER(Dims)] + [P] * 17 + [ctypes.POINTER(Debug), P]
        L.moe_w8a8_pack_weights.restype = ctypes.c_int
        L.moe_w8a8_pack_weights.argtypes = [P, P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, P]
        L.moe_w8a8_packed_mx_bytes.restype = ctypes.c_int
        L.moe_w8a8_packed_mx_bytes.argtypes = [ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                               ctypes.POINTER(ctypes.c_size_t)]
        L.moe_w8a8_pack_weights_mx.restype = ctypes.c_int
        L.moe_w8a8_pack_weights_mx.argtypes = [P, P, P, ctypes.c_int64, ctypes.c_int32, ctypes.c_int32,
                                               ctypes.c_int32, P]
        L.moe_w8a8_warm.restype = ctypes.c_int
        L.moe_w8a8_warm.argtypes = [P, ctypes.c_size_t, P]
        L.moe_w8a8_read_probe.restype = ctypes.c_int
        L.moe_w8a8_read_probe.argtypes = [P, ctypes.c_size_t, P]
        L.moe_w8a8_read_write_probe.restype = ctypes.c_int
        L.moe_w8a8_read_write_probe.argtypes = [P, ctypes.c_size_t, P, ctypes.c_size_t, P]
        L.moe_w8a8_forward_quantized.restype = ctypes.c_int
        L.moe_w8a8_forward_quantized.argtypes = ([ctypes.POINTER(Dims)] + [P] * 17
                                                 + [ctypes.c_size_t, ctypes.POINTER(Debug), P])
        L.moe_w8a8_norm_quant.restype = ctypes.c_int
        L.moe_w8a8_norm_quant.argtypes = [ctypes.POINTER(NormDims)] + [P] * 8
        L.moe_w8a8_gate_workspace_size.restype = ctypes.c_int
        L.moe_w8a8_gate_workspace_size.argtypes = [ctypes.POINTER(GateDims), ctypes.POINTER(ctypes.c_size_t)]
        L.moe_w8a8_gate.restype = ctypes.c_int
        L.moe_w8a8_gate.argtypes = [ctypes.POINTER(GateDims)] + [P] * 6 + [ctypes.c_size_t, P]
        L.moe_w8a8_packed_w4_bytes.restype = ctypes.c_int
        L.moe_w8a8_packed_w4_bytes.argtypes = [ctypes.POINTER(LinearW4Dims), ctypes.POINTER(ctypes.c_size_t)]
        L.moe_w8a8_pack_weights_w4.restype = ctypes.c_int
        L.moe_w8a8_pack_weights_w4.argtypes = [ctypes.POINTER(LinearW4Dims)] + [P] * 5
        L.moe_w8a8_linear_w4.restype = ctypes.c_int
        L.moe_w8a8_linear_w4.argtypes = [ctypes.POINTER(LinearW4Dims)] + [P] * 6
        L.moe_w8a8_packed_w8_bytes.restype = ctypes.c_int
        L.moe_w8a8_packed_w8_bytes.argtypes = [ctypes.POINTER(LinearW8Dims), ctypes.POINTER(ctypes.c_size_t)]
        L.moe_w8a8_pack_weights_w8.restype = ctypes.c_int
        L.moe_w8a8_pack_weights_w8.argtypes = [ctypes.POINTER(LinearW8Dims)] + [P] * 4
        L.moe_w8a8_linear_w8.restype = ctypes.c_int
        L.moe_w8a8_linear_w8.argtypes = [ctypes.POINTER(LinearW8Dims)] + [P] * 6
        L.moe_w8a8_quant.restype = ctypes.c_int
        L.moe_w8a8_quant.argtypes = [ctypes.POINTER(QuantDims)] + [P] * 5
        L.moe_w8a8_join_norm.restype = ctypes.c_int
        L.moe_w8a8_join_norm.argtypes = [ctypes.POINTER(JoinNormDims)] + [P] * 12
        L.moe_w8a8_dispatch_rows.restype = ctypes.c_int
        L.moe_w8a8_dispatch_rows.argtypes = [ctypes.POINTER(DispatchDims), ctypes.POINTER(ctypes.c_int64)]
        L.moe_w8a8_dispatch_workspace_size.restype = ctypes.c_int
        L.moe_w8a8_dispatch_workspace_size.argtypes = [ctypes.POINTER(DispatchDims), ctypes.POINTER(ctypes.c_size_t)]
        L.moe_w8a8_dispatch.restype = ctypes.c_int
        L.moe_w8a8_dispatch.argtypes = [ctypes.POINTER(DispatchDims)] + [P] * 11 + [ctypes.c_size_t, P]
        L.moe_w8a8_combine.restype = ctypes.c_int
        L.moe_w8a8_combine.argtypes = [ctypes.POINTER(CombineDims)] + [P] * 6
        L.moe_w8a8_combine_grad.restype = ctypes.c_int
        L.moe_w8a8_combine_grad.argtypes = [ctypes.POINTER(CombineDims)] + [P] * 8
        L.moe_w8a8_status_string.restype = ctypes.c_char_p
        L.moe_w8a8_status_string.argtypes = [ctypes.c_int]
        _lib = L
    return _lib


def make_dims(num_tokens, hidden, inter, topk, moe_expert_num, share_inter=0, ep_rank_size=1, ep_rank_id=0,
              quant_mode=1, amax_eps=1e-6, weight_layout=MOE_WEIGHT_ROW_MAJOR, fuse_route_scale=0,
              weight_format=MOE_WEIGHT_INT8, quant_group=0, requant_in_epilogue=0) -> Dims:
    return Dims(num_tokens, hidden, inter, share_inter, topk, moe_expert_num, ep_rank_size, ep_rank_id, quant_mode,
                amax_eps, weight_layout, fuse_route_scale, weight_format, quant_group, requant_in_epilogue)


def moe_w8a8_status_string(code: int) -> str:
    return library().moe_w8a8_status_string(code).decode()


def moe_w8a8_workspace_size(dims: Dims) -> int:
    n = ctypes.c_size_t(0)
    rc = library().moe_w8a8_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_workspace_size")
    return int(n.value)


def _stream(stream):
    """The HIP stream handle to pass: torch's current stream when None."""
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else stream


def moe_w8a8_pack_weights(src, which, dst=None, stream=None):
    """Pack an int8 weight tensor [groups, n, k] or [n, k] (device) into the
    kernels' streaming order; `which` is MOE_PACK_GMM1 for a gmm1 tensor and
    MOE_PACK_GMM2 for a gmm2 tensor. Returns dst (allocated like src if None)."""
    if dst is None:
        dst = torch.empty_like(src)
    shape = src.shape if src.dim() == 3 else (1, *src.shape)
    rc = library().moe_w8a8_pack_weights(_ptr(src), _ptr(dst), shape[0], shape[1], shape[2], which, _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_pack_weights")
    return dst


def moe_w8a8_warm(t, nbytes: Optional[int] = None, stream=None) -> None:
    """Warm the caches with a device tensor's bytes (or its first nbytes)."""
    n = t.numel() * t.element_size() if nbytes is None else nbytes
    rc = library().moe_w8a8_warm(_ptr(t), n, _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_warm")


def moe_w8a8_read_probe(t, nbytes: Optional[int] = None, stream=None) -> None:
    """Stream a device tensor's bytes (or its first nbytes) once and discard
    them (the read-bandwidth probe)."""
    n = t.numel() * t.element_size() if nbytes is None else nbytes
    rc = library().moe_w8a8_read_probe(_ptr(t), n, _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_read_probe")


def moe_w8a8_read_write_probe(src, src_bytes: int, dst=None, dst_bytes: int = 0, stream=None) -> None:
    """Read src_bytes of a device tensor in 256 KB work items and write dst_bytes
    of another (arbitrary values) in equal shares at the items' ends: the
    larger-batch GEMMs' read and write mix, for measurement."""
    rc = library().moe_w8a8_read_write_probe(_ptr(src), src_bytes, _ptr(dst), dst_bytes, _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_read_write_probe")


def moe_w8a8_packed_mx_bytes(groups: int, n: int, k: int) -> int:
    b = ctypes.c_size_t(0)
    rc = library().moe_w8a8_packed_mx_bytes(groups, n, k, ctypes.byref(b))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_packed_mx_bytes")
    return int(b.value)


def moe_w8a8_pack_weights_mx(data, block_scale, which, dst=None, stream=None):
    """Pack FP4 weights (uint8 E2M1 pairs [groups, n, k/2] or [n, k/2], E8M0
    block scales [.., n, k/32], device tensors) into one buffer for
    weight_format MOE_WEIGHT_MXFP4. Returns dst (uint8, allocated if None)."""
    shape = data.shape if data.dim() == 3 else (1, *data.shape)
    groups, n, k = shape[0], shape[1], 2 * shape[2]
    if dst is None:
        dst = torch.empty(moe_w8a8_packed_mx_bytes(groups, n, k), dtype=torch.uint8, device=data.device)
    rc = library().moe_w8a8_pack_weights_mx(_ptr(data), _ptr(block_scale), _ptr(dst), groups, n, k, which,
                                            _stream(stream))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_pack_weights_mx")
    return dst


def pack_weights(tensors: dict, stream=None) -> dict:
    """Return a copy of an upload() dict whose four weight tensors are packed."""
    out = dict(tensors)
    for k in ("gmm1_weight", "gmm2_weight", "share_gmm1_weight", "share_gmm2_weight"):
        if out.get(k) is not None:
            out[k] = moe_w8a8_pack_weights(out[k], MOE_PACK_GMM1 if "gmm1" in k else MOE_PACK_GMM2, stream=stream)
    return out


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensors passed to libmoe_w8a8 must be device tensors")
    if not t.is_contiguous():
        raise ValueError("tensors passed to libmoe_w8a8 must be contiguous")
    return t.data_ptr()


def moe_w8a8_forward(dims: Dims, x, expert_ids, expert_scales, gmm1_weight, gmm1_weight_scale, gmm2_weight,
                     gmm2_weight_scale, share_gmm1_weight=None, share_gmm1_weight_scale=None,
                     share_gmm2_weight=None, share_gmm2_weight_scale=None, expert_smooth_scales=None,
                     share_smooth_scales=None, x_active_mask=None, output=None, share_output=None,
                     expert_token_nums=None, workspace=None, workspace_bytes: Optional[int] = None,
                     dbg: Optional[Debug] = None, stream=None, check: bool = True) -> int:
    """Call the C entry point with device tensors (or raw device addresses).
    Returns the status code; raises MoeError on failure when check=True."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = [x, expert_ids, expert_scales, gmm1_weight, gmm1_weight_scale, gmm2_weight, gmm2_weight_scale,
            share_gmm1_weight, share_gmm1_weight_scale, share_gmm2_weight, share_gmm2_weight_scale,
            expert_smooth_scales, share_smooth_scales, x_active_mask, output, share_output, expert_token_nums,
            workspace]
    rc = library().moe_w8a8_forward(ctypes.byref(dims), *[_ptr(a) for a in args], workspace_bytes,
                                    ctypes.byref(dbg) if dbg is not None else None, _stream(stream))
    if check and rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_forward")
    return rc


def moe_w8a8_forward_noalloc(dims: Dims, x, expert_ids, expert_scales, gmm1_weight, gmm1_weight_scale,
                             gmm2_weight, gmm2_weight_scale, share_gmm1_weight=None, share_gmm1_weight_scale=None,
                             share_gmm2_weight=None, share_gmm2_weight_scale=None, expert_smooth_scales=None,
                             share_smooth_scales=None, x_active_mask=None, output=None, share_output=None,
                             expert_token_nums=None, dbg: Optional[Debug] = None, stream=None,
                             check: bool = True) -> int:
    """Call the entry point that takes no workspace (the library's built-in
    per-device scratch array). Returns the status code; raises MoeError on
    failure when check=True."""
    args = [x, expert_ids, expert_scales, gmm1_weight, gmm1_weight_scale, gmm2_weight, gmm2_weight_scale,
            share_gmm1_weight, share_gmm1_weight_scale, share_gmm2_weight, share_gmm2_weight_scale,
            expert_smooth_scales, share_smooth_scales, x_active_mask, output, share_output, expert_token_nums]
    rc = library().moe_w8a8_forward_noalloc(ctypes.byref(dims), *[_ptr(a) for a in args],
                                            ctypes.byref(dbg) if dbg is not None else None, _stream(stream))
    if check and rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_forward_noalloc")
    return rc


def moe_w8a8_forward_quantized(dims: Dims, q_x, x_scale, expert_ids, expert_scales, gmm1_weight, gmm1_weight_scale,
                               gmm2_weight, gmm2_weight_scale, share_gmm1_weight=None, share_gmm1_weight_scale=None,
                               share_gmm2_weight=None, share_gmm2_weight_scale=None, x_active_mask=None, output=None,
                               share_output=None, expert_token_nums=None, workspace=None,
                               workspace_bytes: Optional[int] = None, dbg: Optional[Debug] = None, stream=None,
                               check: bool = True) -> int:
    """moe_w8a8_forward on codes and scales that moe_w8a8_norm_quant (or the
    caller) made of x: q_x [T, H] int8 (float8_e4m3fn for FP4 weights), x_scale
    fp32 [T] or [T, H / quant_group]. int8 and uint8 tensors are also taken as
    the raw bytes of E4M3 codes, so norm codes for FP4 weights have to be made
    with MOE_QUANT_E4M3 (the default is int8). Runs on q_x's device. Returns
    the status code; raises MoeError on failure when check=True."""
    T, H = dims.num_tokens, dims.hidden
    if isinstance(q_x, torch.Tensor):
        want = torch.float8_e4m3fn if dims.weight_format == MOE_WEIGHT_MXFP4 else torch.int8
        if q_x.numel() != T * H or q_x.dtype not in (want, torch.uint8, torch.int8):
            raise ValueError(f"q_x: expected {T * H} codes of {want} (or their bytes), got {tuple(q_x.shape)} of {q_x.dtype}")
        if q_x.is_cuda and q_x.get_device() != torch.cuda.current_device():
            with torch.cuda.device(q_x.get_device()):
                return moe_w8a8_forward_quantized(
                    dims, q_x, x_scale, expert_ids, expert_scales, gmm1_weight, gmm1_weight_scale, gmm2_weight,
                    gmm2_weight_scale, share_gmm1_weight, share_gmm1_weight_scale, share_gmm2_weight,
                    share_gmm2_weight_scale, x_active_mask, output, share_output, expert_token_nums, workspace,
                    workspace_bytes, dbg, stream, check)
    if isinstance(x_scale, torch.Tensor):
        n = T * (H // dims.quant_group if dims.quant_mode == 2 and dims.quant_group > 0 else 1)
        if x_scale.dtype is not torch.float32 or x_scale.numel() != n:
            raise ValueError(f"x_scale: expected {n} elements of torch.float32, got {tuple(x_scale.shape)} of "
                             f"{x_scale.dtype}")
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    args = [q_x, x_scale, expert_ids, expert_scales, gmm1_weight, gmm1_weight_scale, gmm2_weight, gmm2_weight_scale,
            share_gmm1_weight, share_gmm1_weight_scale, share_gmm2_weight, share_gmm2_weight_scale, x_active_mask,
            output, share_output, expert_token_nums, workspace]
    rc = library().moe_w8a8_forward_quantized(ctypes.byref(dims), *[_ptr(a) for a in args], workspace_bytes,
                                              ctypes.byref(dbg) if dbg is not None else None, _stream(stream))
    if check and rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_forward_quantized")
    return rc


# ------------------------------------------- operators around the block
# These take tensors only, and check their types, sizes and device: a call
# whose tensors do not fit its dims raises ValueError before the library sees
# it. They run on the tensors' device, whichever device is current. The checks
# and the call are in csrc/pycall.cpp.

_pycall = None


def _native():
    """The compiled argument checks (raises if they have not been built)."""
    global _pycall
    if _pycall is None:
        library()
        try:
            from . import _pycall as module
        except ImportError as e:
            raise ImportError(f"_pycall.so ({e}): build it with `python -m moe_expert_ffn_route_amd.build`") from e
        _pycall = module
    return _pycall


def _tensor(t, name: str) -> None:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name}: expected a tensor, got {type(t).__name__}")


def _call(where: str, fn, first, stream, *args) -> None:
    """fn(*args, stream handle) with the device of tensor `first` current; the
    stream defaults to that device's current one (its handle: the stream
    object costs a microsecond)."""
    _tensor(first, where)
    device = first.get_device()
    if device < 0:  # refused by fn
        handle = 0
    elif device != torch._C._cuda_getDevice():
        with torch.cuda.device(device):
            return _call(where, fn, first, stream, *args)
    else:
        handle = torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)
    rc = fn(*args, handle)
    if rc != MOE_OK:
        raise MoeError(rc, where)


def _arg(t, name: str, dtype, numel: int, device: int) -> Optional[int]:
    """The device pointer of an argument of `numel` elements (None: NULL)."""
    if t is None:
        return None
    _tensor(t, name)
    if t.dtype is not dtype or t.numel() != numel:
        raise ValueError(f"{name}: expected {numel} elements of {dtype}, got {tuple(t.shape)} of {t.dtype}")
    if t.get_device() != device or device < 0:
        raise ValueError(f"{name}: expected a tensor on the GPU that holds the call's first tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors passed to libmoe_w8a8 must be contiguous")
    return t.data_ptr()


def _empty(shape, dtype, device, stream):
    """A tensor that the call allocates: from the pool of the stream that the
    call runs on, so that memory freed after the call is not handed to another
    stream while the kernels still use it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _code(dt) -> int:
    if dt not in _DTYPE_CODE:
        raise ValueError(f"unsupported element type {dt}")
    return _DTYPE_CODE[dt]


def _torch_type(code: int):
    for dt, c in _DTYPE_CODE.items():
        if c == code:
            return dt
    raise ValueError(f"unsupported element type code {code}")


def make_norm_dims(num_tokens, hidden, dtype=torch.bfloat16, weight_dtype=None, quant=MOE_QUANT_INT8, quant_group=0,
                   rms_eps=1e-6, amax_eps=1e-6) -> NormDims:
    return NormDims(num_tokens, hidden, _code(dtype), _code(dtype if weight_dtype is None else weight_dtype), quant,
                    quant_group, rms_eps, amax_eps)


def moe_w8a8_norm_quant(dims: NormDims, x, weight=None, residual=None, residual_out=None, y=None, q=None,
                        q_scale=None, stream=None) -> None:
    """Residual addition, RMS norm and 8-bit quantisation of x [T, H] in one
    pass; writes those of residual_out, y, q and q_scale that are given (see
    the header). residual_out and y may be x or residual themselves."""
    _call("moe_w8a8_norm_quant", _native().norm_quant, x, stream, dims, x, residual, weight, residual_out, y, q,
          q_scale)


def make_gate_dims(num_tokens, hidden, moe_expert_num, topk, score=MOE_SCORE_SOFTMAX, normalize=True,
                   route_scale=1.0, dtype=torch.bfloat16, weight_dtype=None) -> GateDims:
    return GateDims(num_tokens, hidden, moe_expert_num, topk, score, int(normalize), _code(dtype),
                    _code(dtype if weight_dtype is None else weight_dtype), route_scale)


def moe_w8a8_gate_workspace_size(dims: GateDims) -> int:
    n = ctypes.c_size_t(0)
    rc = library().moe_w8a8_gate_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_gate_workspace_size")
    return int(n.value)


def moe_w8a8_gate(dims: GateDims, x, weight, bias=None, expert_ids=None, expert_scales=None, workspace=None,
                  stream=None):
    """Router: top-k experts of x [T, H] and their weights. Returns
    (expert_ids int32 [T, K], expert_scales fp32 [T, K]), allocated if None,
    as is the workspace."""
    if expert_ids is None or expert_scales is None or workspace is None:
        _tensor(x, "x")
        n = moe_w8a8_gate_workspace_size(dims)  # dims that no buffer can have raise here
        if expert_ids is None:
            expert_ids = _empty((dims.num_tokens, dims.topk), torch.int32, x.device, stream)
        if expert_scales is None:
            expert_scales = _empty((dims.num_tokens, dims.topk), torch.float32, x.device, stream)
        if workspace is None:
            workspace = _empty(max(256, n), torch.uint8, x.device, stream)
    _tensor(workspace, "workspace")
    _call("moe_w8a8_gate", _native().gate, x, stream, dims, x, weight, bias, expert_ids, expert_scales, workspace,
          workspace.numel())
    return expert_ids, expert_scales


def make_linear_w4_dims(num_tokens, out_features, in_features, group=128, act_dtype=torch.bfloat16, gated=False,
                        has_zeros=False) -> LinearW4Dims:
    return LinearW4Dims(num_tokens, out_features, in_features, group, _code(act_dtype), int(gated), int(has_zeros))


def moe_w8a8_packed_w4_bytes(dims: LinearW4Dims) -> int:
    b = ctypes.c_size_t(0)
    rc = library().moe_w8a8_packed_w4_bytes(ctypes.byref(dims), ctypes.byref(b))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_packed_w4_bytes")
    return int(b.value)


def moe_w8a8_pack_weights_w4(dims: LinearW4Dims, codes, scale, zero=None, dst=None, stream=None):
    """Pack 4-bit weights (codes uint8 [N, K/2], scale fp32 [N, K/group], zero
    uint8 [N, K/group] if has_zeros) for moe_w8a8_linear_w4 with these dims
    (num_tokens aside). Returns dst (uint8, allocated if None)."""
    _tensor(codes, "codes")
    nbytes, dev = moe_w8a8_packed_w4_bytes(dims), codes.get_device()
    if dst is None:
        dst = _empty(nbytes, torch.uint8, codes.device, stream)
    N, K = dims.out_features, dims.in_features
    groups = N * (K // dims.group)
    _call("moe_w8a8_pack_weights_w4", library().moe_w8a8_pack_weights_w4, codes, stream, ctypes.byref(dims),
          _arg(codes, "codes", torch.uint8, N * (K // 2), dev), _arg(scale, "scale", torch.float32, groups, dev),
          _arg(zero, "zero", torch.uint8, groups, dev), _arg(dst, "dst", torch.uint8, nbytes, dev))
    return dst


def moe_w8a8_linear_w4(dims: LinearW4Dims, x, weight, x_scale=None, bias=None, out=None, stream=None):
    """Dense product of x [T, K] (bf16, fp16, or int8 with x_scale fp32 [T])
    with packed 4-bit weights. Returns out (bf16, fp16 for fp16 x; [T, N], or
    [T, N/2] when gated), allocated if None."""
    if out is None:
        _tensor(x, "x")
        moe_w8a8_packed_w4_bytes(dims)  # dims that no buffer can have raise here
        width = dims.out_features // 2 if dims.gated else dims.out_features
        out = _empty((dims.num_tokens, width), torch.float16 if dims.act_dtype == MOE_DTYPE_FP16 else torch.bfloat16,
                     x.device, stream)
    _call("moe_w8a8_linear_w4", _native().linear_w4, x, stream, dims, x, x_scale, weight, bias, out)
    return out


# ------------------------- operators between the block and the rest of a program

def make_linear_w8_dims(num_tokens, out_features, in_features, out_dtype=torch.bfloat16, gated=False) -> LinearW8Dims:
    return LinearW8Dims(num_tokens, out_features, in_features, _code(out_dtype), int(gated))


def moe_w8a8_packed_w8_bytes(dims: LinearW8Dims) -> int:
    b = ctypes.c_size_t(0)
    rc = library().moe_w8a8_packed_w8_bytes(ctypes.byref(dims), ctypes.byref(b))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_packed_w8_bytes")
    return int(b.value)


def moe_w8a8_pack_weights_w8(dims: LinearW8Dims, codes, scale, dst=None, stream=None):
    """Pack int8 weights (codes int8 [N, K], scale fp32 [N]) for
    moe_w8a8_linear_w8 with these dims (num_tokens and out_dtype aside).
    Returns dst (uint8, allocated if None)."""
    _tensor(codes, "codes")
    nbytes, dev = moe_w8a8_packed_w8_bytes(dims), codes.get_device()
    if dst is None:
        dst = _empty(nbytes, torch.uint8, codes.device, stream)
    N = dims.out_features
    _call("moe_w8a8_pack_weights_w8", library().moe_w8a8_pack_weights_w8, codes, stream, ctypes.byref(dims),
          _arg(codes, "codes", torch.int8, N * dims.in_features, dev), _arg(scale, "scale", torch.float32, N, dev),
          _arg(dst, "dst", torch.uint8, nbytes, dev))
    return dst


def moe_w8a8_linear_w8(dims: LinearW8Dims, x, x_scale, weight, bias=None, out=None, stream=None):
    """Dense product of int8 codes x [T, K] with scales x_scale fp32 [T] by
    packed int8 weights. Returns out (dims.out_dtype; [T, N], or [T, N/2] when
    gated), allocated if None."""
    if out is None:
        _tensor(x, "x")
        moe_w8a8_packed_w8_bytes(dims)  # dims that no buffer can have raise here
        width = dims.out_features // 2 if dims.gated else dims.out_features
        out = _empty((dims.num_tokens, width), _torch_type(dims.out_dtype), x.device, stream)
    _call("moe_w8a8_linear_w8", _native().linear_w8, x, stream, dims, x, x_scale, weight, bias, out)
    return out


def make_quant_dims(num_tokens, hidden, dtype=torch.bfloat16, quant=MOE_QUANT_INT8, quant_group=0,
                    amax_eps=1e-6) -> QuantDims:
    return QuantDims(num_tokens, hidden, _code(dtype), quant, quant_group, amax_eps)


def moe_w8a8_quant(dims: QuantDims, x, smooth=None, q=None, q_scale=None, stream=None):
    """Codes and scales of x [T, H], times smooth fp32 [H] if given. Returns
    (q int8 or float8_e4m3fn [T, H], q_scale fp32 [T] or [T, H / quant_group]),
    allocated if None."""
    if q is None or q_scale is None:
        _tensor(x, "x")
        T, H, g = dims.num_tokens, dims.hidden, dims.quant_group
        if T < 0 or H <= 0 or g < 0 or (g and H % g):  # dims that no buffer can have
            raise MoeError(MOE_ERR_INVALID_ARG, "moe_w8a8_quant")
        if q is None:
            q = _empty((T, H), torch.float8_e4m3fn if dims.quant == MOE_QUANT_E4M3 else torch.int8, x.device, stream)
        if q_scale is None:
            q_scale = _empty((T, H // g) if g else (T,), torch.float32, x.device, stream)
    _call("moe_w8a8_quant", _native().quant, x, stream, dims, x, smooth, q, q_scale)
    return q, q_scale


def make_join_norm_dims(num_tokens, hidden, dtype=torch.bfloat16, weight_dtype=None, post_norm=False, gate_rows=0,
                        quant=MOE_QUANT_INT8, quant_group=0, residual_scale=1.0, branch_scale=1.0, post_eps=1e-6,
                        rms_eps=1e-6, amax_eps=1e-6) -> JoinNormDims:
    return JoinNormDims(num_tokens, hidden, _code(dtype), _code(dtype if weight_dtype is None else weight_dtype),
                        int(post_norm), gate_rows, quant, quant_group, residual_scale, branch_scale, post_eps, rms_eps,
                        amax_eps)


def moe_w8a8_join_norm(dims: JoinNormDims, block, residual=None, share=None, share_scale=None, post_weight=None,
                       gate=None, weight=None, residual_out=None, y=None, q=None, q_scale=None, stream=None) -> None:
    """The block's outputs (share times share_scale fp32 [T]), normed if
    dims.post_norm, gated and scaled, onto the residual stream, and the next
    norm with its codes; writes those of residual_out, y, q and q_scale that
    are given (see the header). residual_out and y may be block, share or
    residual themselves."""
    _call("moe_w8a8_join_norm", _native().join_norm, block, stream, dims, block, share, share_scale, residual,
          post_weight, gate, weight, residual_out, y, q, q_scale)


def make_dispatch_dims(num_tokens, hidden, moe_expert_num, topk, dtype=torch.bfloat16, scale_groups=0,
                       row_align=1) -> DispatchDims:
    """dtype of x and its rows; torch.int8 stands for any 8-bit codes."""
    return DispatchDims(num_tokens, topk, moe_expert_num, hidden, _code(dtype), scale_groups, row_align)


def moe_w8a8_dispatch_rows(dims: DispatchDims) -> int:
    n = ctypes.c_int64(0)
    rc = library().moe_w8a8_dispatch_rows(ctypes.byref(dims), ctypes.byref(n))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_dispatch_rows")
    return int(n.value)


def moe_w8a8_dispatch_workspace_size(dims: DispatchDims) -> int:
    n = ctypes.c_size_t(0)
    rc = library().moe_w8a8_dispatch_workspace_size(ctypes.byref(dims), ctypes.byref(n))
    if rc != MOE_OK:
        raise MoeError(rc, "moe_w8a8_dispatch_workspace_size")
    return int(n.value)


def moe_w8a8_dispatch(dims: DispatchDims, expert_ids, x=None, x_scale=None, x_active_mask=None, rows=None,
                      row_scale=None, expert_token_nums=None, expert_offset=None, row_of_pair=None, pair_of_row=None,
                      workspace=None, stream=None) -> dict:
    """Sort the pairs of expert_ids int32 [T, K] by expert, and with them the
    rows of x [T, H] and its scales x_scale fp32 [T, scale_groups]. Returns a
    dict of rows, row_scale, expert_token_nums, expert_offset, row_of_pair and
    pair_of_row (see the header), allocated if None, as is the workspace.
    Without x the maps are made alone (rows and row_scale None)."""
    if (expert_token_nums is None or expert_offset is None or row_of_pair is None or pair_of_row is None
            or workspace is None or x is not None and (rows is None or row_scale is None and dims.scale_groups)):
        _tensor(expert_ids, "expert_ids")
        R, need = moe_w8a8_dispatch_rows(dims), moe_w8a8_dispatch_workspace_size(dims)  # impossible dims raise here

        def new(t, shape, dtype):
            return _empty(shape, dtype, expert_ids.device, stream) if t is None else t
        i32 = torch.int32
        expert_token_nums = new(expert_token_nums, (dims.moe_expert_num,), i32)
        expert_offset = new(expert_offset, (dims.moe_expert_num + 1,), i32)
        row_of_pair = new(row_of_pair, (dims.num_tokens, dims.topk), i32)
        pair_of_row = new(pair_of_row, (R,), i32)
        workspace = new(workspace, (max(256, need),), torch.uint8)
        if x is not None:
            _tensor(x, "x")
            rows = new(rows, (R, dims.hidden), x.dtype)
            if dims.scale_groups:
                row_scale = new(row_scale, (R, dims.scale_groups), torch.float32)
    _tensor(workspace, "workspace")
    _call("moe_w8a8_dispatch", _native().dispatch, expert_ids, stream, dims, expert_ids, x, x_scale, x_active_mask, rows,
          row_scale, expert_token_nums, expert_offset, row_of_pair, pair_of_row, workspace, workspace.numel())
    return dict(rows=rows, row_scale=row_scale, expert_token_nums=expert_token_nums, expert_offset=expert_offset,
                row_of_pair=row_of_pair, pair_of_row=pair_of_row)


def make_combine_dims(num_tokens, hidden, topk, num_rows, dtype=torch.bfloat16, out_dtype=None) -> CombineDims:
    return CombineDims(num_tokens, topk, hidden, num_rows, _code(dtype), _code(dtype if out_dtype is None else out_dtype))


def moe_w8a8_combine(dims: CombineDims, rows, row_of_pair, expert_scales=None, addend=None, out=None, stream=None):
    """Sorted rows [R, H] back to their tokens, weighted by expert_scales fp32
    [T, K] if given, plus addend [T, H] if given (may be out). Returns out
    [T, H] (dims.out_dtype), allocated if None. Without expert_scales it is
    the gradient of moe_w8a8_dispatch. As with every call here, autograd does
    not record it: out is detached from rows, expert_scales and addend, and a
    program that trains calls moe_w8a8_combine_grad in its own backward."""
    if out is None:
        _tensor(rows, "rows")
        if dims.num_tokens < 0 or dims.hidden <= 0:  # dims that no buffer can have
            raise MoeError(MOE_ERR_INVALID_ARG, "moe_w8a8_combine")
        out = _empty((dims.num_tokens, dims.hidden), _torch_type(dims.out_dtype), rows.device, stream)
    _call("moe_w8a8_combine", _native().combine, rows, stream, dims, rows, row_of_pair, expert_scales, addend, out)
    return out


def moe_w8a8_combine_grad(dims: CombineDims, dout, row_of_pair, pair_of_row, rows=None, expert_scales=None, drows=None,
                          dscales=None, stream=None) -> None:
    """The gradient of moe_w8a8_combine: writes those of drows [R, H] (of its
    rows) and dscales fp32 [T, K] (of expert_scales; needs rows) that are
    given. The maps are those of moe_w8a8_dispatch."""
    _call("moe_w8a8_combine_grad", _native().combine_grad, dout, stream, dims, dout, row_of_pair, pair_of_row, rows,
          expert_scales, drows, dscales)


# ---------------------------------------------------------------- helpers

def dims_of_case(case) -> Dims:
    """Dims of a moe_expert_ffn_route_amd.synth.Case."""
    return Dims(**case.dims)


def upload(case, device="cuda", weights=None) -> dict:
    """Copy a synth.Case's arrays to the device (weights may be passed in to
    reuse already resident tensors). Returns a dict of tensors keyed by the
    C argument names."""
    def t(a, dtype=None):
        if a is None:
            return None
        x = torch.from_numpy(a)
        if dtype is not None:
            x = x.view(dtype)
        return x.to(device, non_blocking=False).contiguous()

    d = dict(x=t(case.x, torch.bfloat16) if case.x.size else torch.empty(case.x.shape, dtype=torch.bfloat16,
                                                                          device=device),
             expert_ids=t(case.expert_ids), expert_scales=t(case.expert_scales),
             expert_smooth_scales=t(case.smooth), share_smooth_scales=t(case.share_smooth),
             x_active_mask=t(case.mask))
    if weights is None and case.w1b is None:
        weights = dict(gmm1_weight=t(case.w1), gmm1_weight_scale=t(case.w1s), gmm2_weight=t(case.w2),
                       gmm2_weight_scale=t(case.w2s), share_gmm1_weight=t(case.sw1),
                       share_gmm1_weight_scale=t(case.sw1s), share_gmm2_weight=t(case.sw2),
                       share_gmm2_weight_scale=t(case.sw2s))
    if weights is None and case.w1b is not None:
        # FP4 weights: element pairs and block scales packed into one buffer each
        weights = {}
        for name, data, bs in (("gmm1_weight", case.w1, case.w1b), ("gmm2_weight", case.w2, case.w2b),
                               ("share_gmm1_weight", case.sw1, case.sw1b),
                               ("share_gmm2_weight", case.sw2, case.sw2b)):
            if data is not None:
                weights[name] = moe_w8a8_pack_weights_mx(t(data), t(bs),
                                                         MOE_PACK_GMM1 if "gmm1" in name else MOE_PACK_GMM2)
        weights.update(gmm1_weight_scale=t(case.w1s), gmm2_weight_scale=t(case.w2s),
                       share_gmm1_weight_scale=t(case.sw1s), share_gmm2_weight_scale=t(case.sw2s))
        for k in ("share_gmm1_weight", "share_gmm2_weight"):
            weights.setdefault(k, None)
    d.update(weights)
    return d


class Runner:
    """Owns the outputs and workspace for repeated calls of one shape."""

    def __init__(self, dims: Dims, device="cuda"):
        self.dims = dims
        T, H = dims.num_tokens, dims.hidden
        self.output = torch.empty((T, H), dtype=torch.bfloat16, device=device)
        self.share_output = torch.empty((T, H), dtype=torch.bfloat16, device=device) if dims.share_inter else None
        self.expert_token_nums = torch.empty(dims.e_loc, dtype=torch.int32, device=device)
        self.workspace_bytes = moe_w8a8_workspace_size(dims)
        self.workspace = torch.empty(max(256, self.workspace_bytes), dtype=torch.uint8, device=device)
        assert self.workspace.data_ptr() % 256 == 0

    def __call__(self, tensors: dict, dbg: Optional[Debug] = None, stream=None):
        moe_w8a8_forward(self.dims, output=self.output, share_output=self.share_output,
                         expert_token_nums=self.expert_token_nums, workspace=self.workspace,
                         workspace_bytes=self.workspace_bytes, dbg=dbg, stream=stream, **tensors)
        return self.output, self.share_output, self.expert_token_nums


def debug_buffers(dims: Dims, device="cuda") -> tuple[Debug, dict]:
    """Allocate every intermediate buffer of moe_w8a8_debug_t."""
    T, K, H, E = dims.num_tokens, dims.topk, dims.hidden, dims.e_loc
    imax = max(dims.inter, dims.share_inter)
    R = T * K + T
    G = dims.quant_group if dims.quant_mode == 2 else 0
    ngx, ngh = (H // G, imax // G) if G else (1, 1)  # activation scales per row
    z = lambda *s, dt: torch.zeros(s, dtype=dt, device=device)
    bufs = dict(sorted_pair=z(max(1, T * K), dt=torch.int32), row_of_pair=z(max(1, T * K), dt=torch.int32),
                group_offset=z(E + 1, dt=torch.int32), shared_token=z(max(1, T), dt=torch.int32),
                num_rows=z(4, dt=torch.int32), q_x=z(max(1, R), H, dt=torch.int8),
                xs=z(max(1, R), ngx, dt=torch.float32) if G else z(max(1, R), dt=torch.float32),
                acc1=z(max(1, R), 2 * imax, dt=torch.int32), h=z(max(1, R), imax, dt=torch.float32),
                q_h=z(max(1, R), imax, dt=torch.int8),
                hs=z(max(1, R), ngh, dt=torch.float32) if G else z(max(1, R), dt=torch.float32),
                acc2=z(max(1, R), H, dt=torch.int32), z=z(max(1, R), H, dt=torch.int16))
    dbg = Debug(**{k: v.data_ptr() for k, v in bufs.items()})
    return dbg, bufs
