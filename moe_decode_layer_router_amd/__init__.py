"""moe_decode_layer_router_amd -- local-expert MoE block for AMD MI355X (gfx950).

A thin ctypes binding of ``libmoeblk.so`` (C ABI: ``include/moeblk.h``). The
functions below carry the C entry points' names and only marshal arguments:
torch tensors supply device memory and the current HIP stream, every step of
the block runs in the library's HIP kernels. There is no fallback: without the
built library (or without a GPU) the calls raise.
"""

from __future__ import annotations

import ctypes
import os

from ._build import LIB as _LIB_PATH

__all__ = [
    "MoeDims",
    "MoeError",
    "lib",
    "dims_from",
    "moe_abi_version",
    "moe_status_string",
    "moe_check_dims",
    "moe_packed_mxfp4_bytes",
    "moe_pack_mxfp4",
    "moe_packed_bf16_bytes",
    "moe_pack_bf16",
    "moe_route",
    "moe_route_workspace_bytes",
    "moe_bucket",
    "moe_ffn_workspace_bytes",
    "moe_expert_ffn",
    "moe_combine",
    "moe_forward_workspace_bytes",
    "moe_forward",
    "moe_forward_static",
    "moe_forward_one_launch",
    "MOE_STATIC_SCRATCH_BYTES",
    "MoeProjDims",
    "proj_dims_from",
    "moe_check_proj_dims",
    "moe_packed_dense_bytes",
    "moe_pack_dense",
    "moe_proj_workspace_bytes",
    "moe_pre_expert",
    "moe_latent_norm",
    "moe_post_expert",
    "moe_topk",
    "MOE_W13",
    "MOE_W2",
    "MoeFp8Dims",
    "fp8_dims_from",
    "moe_check_fp8_dims",
    "moe_fp8_quant",
    "moe_packed_fp8_bytes",
    "moe_pack_fp8",
    "moe_fp8_gemm_workspace_bytes",
    "moe_fp8_gemm",
    "moe_fp8_proj_workspace_bytes",
    "moe_fp8_proj",
    "moe_packed_fp8_expert_bytes",
    "moe_pack_fp8_expert",
    "moe_fp8_ffn_workspace_bytes",
    "moe_fp8_expert_ffn",
    "MOE_WS13",
    "MOE_WS2",
    "MOE_BF16",
    "MOE_FP32",
    "MoeBalanceDims",
    "balance_dims_from",
    "moe_check_balance_dims",
    "moe_balance_workspace_bytes",
    "moe_expert_counts",
    "moe_balance_loss",
    "moe_balance_backward",
    "MOE_SCORE_SIGMOID",
    "MOE_SCORE_SOFTMAX",
    "MoeGateDims",
    "gate_dims_from",
    "moe_check_gate_dims",
    "moe_gate",
    "moe_gate_backward",
    "MoeRowsDims",
    "rows_dims_from",
    "moe_check_rows_dims",
    "moe_sort_workspace_bytes",
    "moe_sort",
    "moe_dispatch",
    "moe_return",
    "moe_return_backward",
    "MoeMxDims",
    "mx_dims_from",
    "moe_check_mx_dims",
    "moe_mx_quant",
    "moe_mx_dequant",
    "moe_packed_mx_bytes",
    "moe_pack_mx",
    "moe_mx_gemm_workspace_bytes",
    "moe_mx_gemm",
    "moe_mx_proj_workspace_bytes",
    "moe_mx_proj",
    "MoeMxGroupDims",
    "mx_group_dims_from",
    "moe_check_mx_group_dims",
    "moe_mx_gate_up",
    "moe_mx_down",
    "MOE_MXFP4",
]

MOE_OK = 0
MOE_ERR_NULL = -1
MOE_ERR_SHAPE = -2
MOE_ERR_ALIGN = -3
MOE_ERR_UNSUPPORTED = -4
MOE_ERR_WORKSPACE = -5
MOE_ERR_HIP = -6
MOE_W13 = 0
MOE_W2 = 1
MOE_WS13 = 2
MOE_WS2 = 3
MOE_BF16 = 0
MOE_FP32 = 1
MOE_MXFP4 = 2
MOE_SCORE_SIGMOID = 0
MOE_SCORE_SOFTMAX = 1
MOE_STATIC_SCRATCH_BYTES = 16 << 20  # moe_forward_static's static scratch a GPU


# the layout of moe_dims and the entry points below (MOEBLK_ABI_VERSION)
ABI_VERSION = 4


class MoeDims(ctypes.Structure):
    _fields_ = [
        ("S", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("n_local", ctypes.c_int32),
        ("local_base", ctypes.c_int32),
        ("I", ctypes.c_int32),
        ("renorm", ctypes.c_int32),
        ("eps", ctypes.c_float),
        ("shared_I", ctypes.c_int32),
        ("bias_mode", ctypes.c_int32),
    ]

    @property
    def r_max(self) -> int:
        return self.S * min(self.topk, self.n_local)


class MoeProjDims(ctypes.Structure):
    _fields_ = [
        ("S", ctypes.c_int32),
        ("K", ctypes.c_int32),
        ("N", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("bias_mode", ctypes.c_int32),
        ("eps", ctypes.c_float),
    ]


class MoeFp8Dims(ctypes.Structure):
    _fields_ = [
        ("M", ctypes.c_int32),
        ("N", ctypes.c_int32),
        ("K", ctypes.c_int32),
        ("in_type", ctypes.c_int32),
        ("out_type", ctypes.c_int32),
    ]


class MoeBalanceDims(ctypes.Structure):
    _fields_ = [
        ("T", ctypes.c_int32),
        ("E", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("n_seq", ctypes.c_int32),
        ("score", ctypes.c_int32),
        ("coef", ctypes.c_float),
    ]


class MoeGateDims(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("T", "E", "topk", "score", "renorm", "bias_mode")]


class MoeRowsDims(ctypes.Structure):
    _fields_ = [
        (f, ctypes.c_int32) for f in ("T", "E", "topk", "n_local", "local_base", "d", "tok_type", "row_type")
    ]


class MoeMxDims(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("M", "N", "K", "in_type", "out_type")]


class MoeMxGroupDims(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int32) for f in ("T", "E", "topk", "n_local", "d", "I", "h_type", "out_type")]


class MoeError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn}: {moe_status_string(code)} (status {code})")
        self.code = code


_lib = None
_P = ctypes.c_void_p
_DP = ctypes.POINTER(MoeDims)


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it is not built."""
    global _lib
    if _lib is None:
        if not os.path.exists(_LIB_PATH):
            raise RuntimeError(
                f"{_LIB_PATH} is not built: run __graft_entry__.build() or "
                "python -m moe_decode_layer_router_amd._build"
            )
        L = ctypes.CDLL(_LIB_PATH)
        L.moe_abi_version.restype = ctypes.c_int
        if L.moe_abi_version() != ABI_VERSION:
            raise RuntimeError(
                f"{_LIB_PATH} has ABI version {L.moe_abi_version()}, this binding expects "
                f"{ABI_VERSION}: rebuild it"
            )
        L.moe_status_string.argtypes = [ctypes.c_int]
        L.moe_status_string.restype = ctypes.c_char_p
        L.moe_check_dims.argtypes = [_DP]
        L.moe_check_dims.restype = ctypes.c_int
        for f in ("moe_packed_mxfp4_bytes", "moe_packed_bf16_bytes"):
            getattr(L, f).argtypes = [_DP, ctypes.c_int]
            getattr(L, f).restype = ctypes.c_size_t
        L.moe_ffn_workspace_bytes.argtypes = [_DP]
        L.moe_ffn_workspace_bytes.restype = ctypes.c_size_t
        L.moe_pack_mxfp4.argtypes = [_DP, ctypes.c_int, _P, _P, _P, _P]
        L.moe_pack_bf16.argtypes = [_DP, ctypes.c_int, _P, _P, _P]
        L.moe_route_workspace_bytes.argtypes = [_DP]
        L.moe_route_workspace_bytes.restype = ctypes.c_size_t
        L.moe_route.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P, ctypes.c_size_t, _P]
        L.moe_bucket.argtypes = [_DP, _P, _P, _P, _P, _P, _P, _P]
        L.moe_expert_ffn.argtypes = [_DP] + [_P] * 11 + [ctypes.c_size_t, _P]
        L.moe_combine.argtypes = [_DP, _P, _P, _P, _P, _P, _P]
        L.moe_forward_workspace_bytes.argtypes = [_DP]
        L.moe_forward_workspace_bytes.restype = ctypes.c_size_t
        L.moe_forward.argtypes = [_DP] + [_P] * 19 + [ctypes.c_size_t, _P]
        L.moe_forward_static.argtypes = [_DP] + [_P] * 19 + [_P]
        L.moe_forward_one_launch.argtypes = [_DP] + [_P] * 17 + [ctypes.c_size_t, _P]
        _PD = ctypes.POINTER(MoeProjDims)
        L.moe_check_proj_dims.argtypes = [_PD]
        for f in ("moe_packed_dense_bytes", "moe_proj_workspace_bytes"):
            getattr(L, f).argtypes = [_PD]
            getattr(L, f).restype = ctypes.c_size_t
        L.moe_pack_dense.argtypes = [_PD, _P, _P, _P]
        L.moe_pre_expert.argtypes = [_PD] + [_P] * 7 + [ctypes.c_size_t, _P]
        L.moe_latent_norm.argtypes = [_PD, _P, _P, _P, _P]
        L.moe_post_expert.argtypes = [_PD] + [_P] * 4 + [ctypes.c_size_t, _P]
        L.moe_topk.argtypes = [_DP, _P, _P, _P, _P, _P]
        _FD, _BD, _Z = ctypes.POINTER(MoeFp8Dims), ctypes.POINTER(MoeBalanceDims), ctypes.c_size_t
        _GD, _RD = ctypes.POINTER(MoeGateDims), ctypes.POINTER(MoeRowsDims)
        _XD, _XG = ctypes.POINTER(MoeMxDims), ctypes.POINTER(MoeMxGroupDims)
        for f, dims in (
            ("moe_packed_fp8_bytes", _FD), ("moe_fp8_gemm_workspace_bytes", _FD),
            ("moe_fp8_proj_workspace_bytes", _FD), ("moe_fp8_ffn_workspace_bytes", _DP),
            ("moe_balance_workspace_bytes", _BD), ("moe_sort_workspace_bytes", _RD),
            ("moe_packed_mx_bytes", _XD), ("moe_mx_gemm_workspace_bytes", _XD), ("moe_mx_proj_workspace_bytes", _XD),
        ):
            getattr(L, f).argtypes = [dims]
            getattr(L, f).restype = _Z
        L.moe_packed_fp8_expert_bytes.argtypes = [_DP, ctypes.c_int]
        L.moe_packed_fp8_expert_bytes.restype = _Z
        for f, args in (
            ("moe_check_fp8_dims", [_FD]),
            ("moe_fp8_quant", [_FD] + [_P] * 4),
            ("moe_pack_fp8", [_FD] + [_P] * 4),
            ("moe_fp8_gemm", [_FD] + [_P] * 5 + [_Z, _P]),
            ("moe_fp8_proj", [_FD] + [_P] * 4 + [_Z, _P]),
            ("moe_pack_fp8_expert", [_DP, ctypes.c_int] + [_P] * 4),
            ("moe_fp8_expert_ffn", [_DP] + [_P] * 11 + [_Z, _P]),
            ("moe_check_balance_dims", [_BD]),
            ("moe_expert_counts", [_BD] + [_P] * 4 + [_Z, _P]),
            ("moe_balance_loss", [_BD] + [_P] * 7 + [_Z, _P]),
            ("moe_balance_backward", [_BD] + [_P] * 6),
            ("moe_check_gate_dims", [_GD]),
            ("moe_gate", [_GD] + [_P] * 5),
            ("moe_gate_backward", [_GD] + [_P] * 6),
            ("moe_check_rows_dims", [_RD]),
            ("moe_sort", [_RD] + [_P] * 6 + [_Z, _P]),
            ("moe_dispatch", [_RD] + [_P] * 4),
            ("moe_return", [_RD] + [_P] * 5),
            ("moe_return_backward", [_RD] + [_P] * 7),
            ("moe_check_mx_dims", [_XD]),
            ("moe_mx_quant", [_XD] + [_P] * 4),
            ("moe_mx_dequant", [_XD] + [_P] * 4),
            ("moe_pack_mx", [_XD] + [_P] * 4),
            ("moe_mx_gemm", [_XD] + [_P] * 5 + [_Z, _P]),
            ("moe_mx_proj", [_XD] + [_P] * 4 + [_Z, _P]),
            ("moe_check_mx_group_dims", [_XG]),
            ("moe_mx_gate_up", [_XG] + [_P] * 8),
            ("moe_mx_down", [_XG] + [_P] * 6),
        ):
            getattr(L, f).argtypes = args
            getattr(L, f).restype = ctypes.c_int
        for f in (
            "moe_pack_mxfp4", "moe_pack_bf16", "moe_route", "moe_bucket", "moe_expert_ffn", "moe_combine",
            "moe_forward", "moe_forward_static", "moe_forward_one_launch", "moe_check_proj_dims", "moe_pack_dense", "moe_pre_expert", "moe_latent_norm",
            "moe_post_expert", "moe_topk",
        ):
            getattr(L, f).restype = ctypes.c_int
        _lib = L
    return _lib


def dims_from(cfg) -> MoeDims:
    """MoeDims from an object or dict with the moe_dims field names."""
    get = cfg.get if isinstance(cfg, dict) else (lambda k, dflt=None: getattr(cfg, k, dflt))
    return MoeDims(
        S=get("S"), d=get("d"), E=get("E"), topk=get("topk"), n_local=get("n_local"),
        local_base=get("local_base"), I=get("I"), renorm=get("renorm"), eps=get("eps"),
        shared_I=get("shared_I"), bias_mode=get("bias_mode", 0),
    )


# ---------------------------------------------------------------- marshalling


def _ptr(t) -> int | None:
    """A tensor's device pointer (None -> NULL). Raw ints pass through."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise ValueError("tensor is not on a GPU device")
    if not t.is_contiguous():
        raise ValueError("tensor is not contiguous")
    return t.data_ptr()


def _stream(stream) -> int | None:
    if stream is None:
        import torch

        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _call(fn: str, *args) -> None:
    rc = getattr(lib(), fn)(*args)
    if rc != MOE_OK:
        raise MoeError(fn, rc)


def _d(dims) -> MoeDims:
    return dims if isinstance(dims, MoeDims) else dims_from(dims)


def moe_abi_version() -> int:
    return lib().moe_abi_version()


def moe_status_string(code: int) -> str:
    return lib().moe_status_string(int(code)).decode()


def moe_check_dims(dims) -> int:
    return lib().moe_check_dims(ctypes.byref(_d(dims)))


def moe_packed_mxfp4_bytes(dims, which: int) -> int:
    return lib().moe_packed_mxfp4_bytes(ctypes.byref(_d(dims)), int(which))


def moe_packed_bf16_bytes(dims, which: int) -> int:
    return lib().moe_packed_bf16_bytes(ctypes.byref(_d(dims)), int(which))


def moe_ffn_workspace_bytes(dims) -> int:
    return lib().moe_ffn_workspace_bytes(ctypes.byref(_d(dims)))


def moe_pack_mxfp4(dims, which, q, scales, packed, stream=None) -> None:
    _call("moe_pack_mxfp4", ctypes.byref(_d(dims)), int(which), _ptr(q), _ptr(scales), _ptr(packed), _stream(stream))


def moe_pack_bf16(dims, which, w, packed, stream=None) -> None:
    _call("moe_pack_bf16", ctypes.byref(_d(dims)), int(which), _ptr(w), _ptr(packed), _stream(stream))


def moe_route_workspace_bytes(dims) -> int:
    return int(lib().moe_route_workspace_bytes(ctypes.byref(_d(dims))))


def moe_route(dims, x, w_router, bias, logits, topk_ids, topk_w, workspace=None, stream=None) -> None:
    """``workspace``: a device tensor of at least moe_route_workspace_bytes
    (None when that is 0)."""
    nbytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _call(
        "moe_route", ctypes.byref(_d(dims)), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(logits),
        _ptr(topk_ids), _ptr(topk_w), _ptr(workspace), ctypes.c_size_t(nbytes), _stream(stream),
    )


def moe_bucket(dims, topk_ids, counts, offsets, rows, pick_pos, active, stream=None) -> None:
    _call(
        "moe_bucket", ctypes.byref(_d(dims)), _ptr(topk_ids), _ptr(counts), _ptr(offsets), _ptr(rows),
        _ptr(pick_pos), _ptr(active), _stream(stream),
    )


def moe_expert_ffn(dims, x, w13_packed, w2_packed, counts, offsets, rows, active, ws13_packed,
                   ws2_packed, y, workspace, workspace_bytes=None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _call(
        "moe_expert_ffn", ctypes.byref(_d(dims)), _ptr(x), _ptr(w13_packed), _ptr(w2_packed), _ptr(counts),
        _ptr(offsets), _ptr(rows), _ptr(active), _ptr(ws13_packed), _ptr(ws2_packed), _ptr(y),
        _ptr(workspace), int(workspace_bytes), _stream(stream),
    )


def moe_combine(dims, y, topk_w, pick_pos, gamma, out, stream=None) -> None:
    _call(
        "moe_combine", ctypes.byref(_d(dims)), _ptr(y), _ptr(topk_w), _ptr(pick_pos), _ptr(gamma), _ptr(out),
        _stream(stream),
    )


def moe_forward_workspace_bytes(dims) -> int:
    return lib().moe_forward_workspace_bytes(ctypes.byref(_d(dims)))


def moe_forward(dims, x, w_router, bias, w13_packed, w2_packed, ws13_packed, ws2_packed, gamma, logits,
                topk_ids, topk_w, counts, offsets, rows, pick_pos, active, y, out, workspace,
                workspace_bytes=None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _call(
        "moe_forward", ctypes.byref(_d(dims)), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(w13_packed),
        _ptr(w2_packed), _ptr(ws13_packed), _ptr(ws2_packed), _ptr(gamma), _ptr(logits), _ptr(topk_ids),
        _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(rows), _ptr(pick_pos), _ptr(active), _ptr(y), _ptr(out),
        _ptr(workspace), int(workspace_bytes), _stream(stream),
    )


def moe_forward_one_launch(dims, x, w_router, bias, w13_packed, w2_packed, gamma, logits, topk_ids, topk_w,
                           counts, offsets, rows, pick_pos, active, y, out, workspace, workspace_bytes=None,
                           stream=None) -> None:
    """moe_forward as one launch (S <= 16, d <= 4096, no shared expert)."""
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _call(
        "moe_forward_one_launch", ctypes.byref(_d(dims)), _ptr(x), _ptr(w_router), _ptr(bias),
        _ptr(w13_packed), _ptr(w2_packed), _ptr(gamma), _ptr(logits), _ptr(topk_ids), _ptr(topk_w),
        _ptr(counts), _ptr(offsets), _ptr(rows), _ptr(pick_pos), _ptr(active), _ptr(y), _ptr(out),
        _ptr(workspace), int(workspace_bytes), _stream(stream),
    )


def moe_forward_static(dims, x, w_router, bias, w13_packed, w2_packed, ws13_packed, ws2_packed, gamma,
                       logits, topk_ids, topk_w, counts, offsets, rows, pick_pos, active, y, out,
                       wait_error=None, stream=None) -> None:
    """moe_forward on the library's static per-GPU scratch (no workspace)."""
    _call(
        "moe_forward_static", ctypes.byref(_d(dims)), _ptr(x), _ptr(w_router), _ptr(bias), _ptr(w13_packed),
        _ptr(w2_packed), _ptr(ws13_packed), _ptr(ws2_packed), _ptr(gamma), _ptr(logits), _ptr(topk_ids),
        _ptr(topk_w), _ptr(counts), _ptr(offsets), _ptr(rows), _ptr(pick_pos), _ptr(active), _ptr(y), _ptr(out),
        _ptr(wait_error), _stream(stream),
    )


# ---------------------------------------------------------------- around the block


def proj_dims_from(cfg) -> MoeProjDims:
    """MoeProjDims from an object or dict with the moe_proj_dims field names."""
    get = cfg.get if isinstance(cfg, dict) else (lambda k, dflt=None: getattr(cfg, k, dflt))
    return MoeProjDims(
        S=get("S"), K=get("K"), N=get("N"), E=get("E", 0), bias_mode=get("bias_mode", 0), eps=get("eps", 1e-6),
    )


def _pd(dims) -> MoeProjDims:
    return dims if isinstance(dims, MoeProjDims) else proj_dims_from(dims)


def moe_check_proj_dims(dims) -> int:
    return lib().moe_check_proj_dims(ctypes.byref(_pd(dims)))


def moe_packed_dense_bytes(dims) -> int:
    return lib().moe_packed_dense_bytes(ctypes.byref(_pd(dims)))


def moe_pack_dense(dims, w, packed, stream=None) -> None:
    _call("moe_pack_dense", ctypes.byref(_pd(dims)), _ptr(w), _ptr(packed), _stream(stream))


def moe_proj_workspace_bytes(dims) -> int:
    return lib().moe_proj_workspace_bytes(ctypes.byref(_pd(dims)))


def moe_pre_expert(dims, ffn_in, w_packed, w_router, bias, logits, h_raw, workspace, workspace_bytes=None,
                   stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _call(
        "moe_pre_expert", ctypes.byref(_pd(dims)), _ptr(ffn_in), _ptr(w_packed), _ptr(w_router), _ptr(bias),
        _ptr(logits), _ptr(h_raw), _ptr(workspace), int(workspace_bytes), _stream(stream),
    )


def moe_latent_norm(dims, h_raw, gamma, h, stream=None) -> None:
    _call("moe_latent_norm", ctypes.byref(_pd(dims)), _ptr(h_raw), _ptr(gamma), _ptr(h), _stream(stream))


def moe_post_expert(dims, partial, w_packed, out, workspace, workspace_bytes=None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    _call(
        "moe_post_expert", ctypes.byref(_pd(dims)), _ptr(partial), _ptr(w_packed), _ptr(out), _ptr(workspace),
        int(workspace_bytes), _stream(stream),
    )


def moe_topk(dims, logits, bias, topk_ids, topk_w, stream=None) -> None:
    _call(
        "moe_topk", ctypes.byref(_d(dims)), _ptr(logits), _ptr(bias), _ptr(topk_ids), _ptr(topk_w),
        _stream(stream),
    )


# ---------------------------------------------------------------- FP8 weights


class _Torch:
    """What the calls below ask of torch on every call, looked up once (these
    calls take a few microseconds on the GPU, so the marshalling counts)."""

    def __init__(self):
        import torch

        self.device = torch.cuda.current_device
        self.raw_stream = torch._C._cuda_getCurrentRawStream  # of a device, as an int
        self.f32, self.bf16, self.i32 = (torch.float32,), (torch.bfloat16,), (torch.int32,)
        self.bytes = (torch.uint8,)
        self.e4m3 = (torch.float8_e4m3fn, torch.uint8)
        self.rows = {MOE_BF16: self.bf16, MOE_FP32: self.f32}


_torch = None


def _t() -> _Torch:
    global _torch, _buf
    if _torch is None:
        _torch = _Torch()
        _buf = _check_in_c(_python_buf)
    return _torch


def _check_in_c(python_buf):
    """The same check in C (csrc/marshal.cpp), where it is built for this torch: it reads
    tensors by the layout it was compiled with."""
    import torch

    try:
        from . import _marshal
    except ImportError:
        return python_buf
    if getattr(_marshal, "torch_build", None) != f"{torch.__version__} {torch.version.git_version}":
        return python_buf
    _marshal.set_python(python_buf)  # for what it leaves to it
    return _marshal.buf


def _buf(t, name: str, n: int, kinds, device: int):
    """The pointer of a tensor of ``n`` elements or more (None -> NULL) of one
    of the dtypes ``kinds`` (None: dims the library refuses) on GPU ``device``:
    the calls below launch on the current device."""
    if t is None or type(t) is int:  # a raw pointer passes through
        return t
    if t.get_device() != device:
        raise ValueError(f"{name}: tensor is not on the current GPU device")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensor is not contiguous")
    if kinds is not None and t.dtype not in kinds:
        raise ValueError(f"{name}: dtype {t.dtype}, expected one of {kinds}")
    if t.numel() < n:
        raise ValueError(f"{name}: {t.numel()} elements, {n} are needed")
    return t.data_ptr()


_python_buf = _buf  # _t() may put the check in C in _buf's place


def _on(stream, T: _Torch, device: int) -> int:
    if stream is None:
        return T.raw_stream(device)
    if not isinstance(stream, int) and stream.device_index != device:
        raise ValueError("stream: not on the current GPU device")
    return _stream(stream)


def _fp8_bytes(N: int, K: int) -> int:
    """Packed bytes of one [N, K] matrix: whole 64 x 128 blocks, then the scales."""
    kb = -(-K // 128)
    return -(-N // 64) * 64 * kb * 128 + -(-(-(-N // 128) * kb) // 4) * 16


def _workspace(ws, workspace_bytes, T: _Torch, device: int):
    """The workspace's pointer and bytes (``workspace_bytes`` may state fewer
    than the tensor has; a raw pointer needs it)."""
    if workspace_bytes is None:
        if type(ws) is int:
            raise ValueError("workspace: a raw pointer needs workspace_bytes")
        workspace_bytes = 0 if ws is None else ws.numel()
    elif workspace_bytes < 0:  # would be a huge size_t
        raise ValueError(f"workspace_bytes: {workspace_bytes}")
    return _buf(ws, "workspace", workspace_bytes, T.bytes, device), workspace_bytes


def fp8_dims_from(cfg) -> MoeFp8Dims:
    """MoeFp8Dims from an object or dict with the moe_fp8_dims field names."""
    get = cfg.get if isinstance(cfg, dict) else (lambda k, dflt=None: getattr(cfg, k, dflt))
    return MoeFp8Dims(
        M=get("M"), N=get("N", 1), K=get("K"), in_type=get("in_type", MOE_BF16), out_type=get("out_type", MOE_BF16),
    )


def _fd(dims) -> MoeFp8Dims:
    return dims if isinstance(dims, MoeFp8Dims) else fp8_dims_from(dims)


def moe_check_fp8_dims(dims) -> int:
    return lib().moe_check_fp8_dims(ctypes.byref(_fd(dims)))


def moe_packed_fp8_bytes(dims) -> int:
    return lib().moe_packed_fp8_bytes(ctypes.byref(_fd(dims)))


def moe_fp8_gemm_workspace_bytes(dims) -> int:
    return lib().moe_fp8_gemm_workspace_bytes(ctypes.byref(_fd(dims)))


def moe_fp8_proj_workspace_bytes(dims) -> int:
    return lib().moe_fp8_proj_workspace_bytes(ctypes.byref(_fd(dims)))


def moe_fp8_quant(dims, x, xq, xs, stream=None) -> None:
    """x [M, K] -> xq [M, Kp] e4m3 (torch.float8_e4m3fn or uint8), xs [Kb, M] fp32."""
    d, T = _fd(dims), _t()
    dev = T.device()
    kb = -(-d.K // 128)
    _call(
        "moe_fp8_quant", ctypes.byref(d), _buf(x, "x", d.M * d.K, T.rows.get(d.in_type), dev),
        _buf(xq, "xq", d.M * kb * 128, T.e4m3, dev), _buf(xs, "xs", d.M * kb, T.f32, dev), _on(stream, T, dev),
    )


def moe_pack_fp8(dims, q, scales, packed, stream=None) -> None:
    d, T = _fd(dims), _t()
    dev = T.device()
    _call(
        "moe_pack_fp8", ctypes.byref(d), _buf(q, "q", d.N * d.K, T.e4m3, dev),
        _buf(scales, "scales", -(-d.N // 128) * -(-d.K // 128), T.f32, dev),
        _buf(packed, "packed", moe_packed_fp8_bytes(d), T.bytes, dev), _on(stream, T, dev),
    )


def moe_fp8_gemm(dims, xq, xs, w_packed, out, workspace, workspace_bytes=None, stream=None) -> None:
    d, T = _fd(dims), _t()
    dev = T.device()
    kb = -(-d.K // 128)
    ws, n = _workspace(workspace, workspace_bytes, T, dev)
    _call(
        "moe_fp8_gemm", ctypes.byref(d), _buf(xq, "xq", d.M * kb * 128, T.e4m3, dev),
        _buf(xs, "xs", d.M * kb, T.f32, dev), _buf(w_packed, "w_packed", _fp8_bytes(d.N, d.K), T.bytes, dev),
        _buf(out, "out", d.M * d.N, T.rows.get(d.out_type), dev), ws, n, _on(stream, T, dev),
    )


def moe_fp8_proj(dims, x, w_packed, out, workspace, workspace_bytes=None, stream=None) -> None:
    """moe_fp8_quant of x and moe_fp8_gemm in one call."""
    d, T = _fd(dims), _t()
    dev = T.device()
    ws, n = _workspace(workspace, workspace_bytes, T, dev)
    _call(
        "moe_fp8_proj", ctypes.byref(d), _buf(x, "x", d.M * d.K, T.rows.get(d.in_type), dev),
        _buf(w_packed, "w_packed", _fp8_bytes(d.N, d.K), T.bytes, dev), _buf(out, "out", d.M * d.N, T.rows.get(d.out_type), dev),
        ws, n, _on(stream, T, dev),
    )


def moe_packed_fp8_expert_bytes(dims, which: int) -> int:
    return lib().moe_packed_fp8_expert_bytes(ctypes.byref(_d(dims)), int(which))


def moe_pack_fp8_expert(dims, which, q, scales, packed, stream=None) -> None:
    d, T = _d(dims), _t()
    dev = T.device()
    need = moe_packed_fp8_expert_bytes(d, which)
    if need == 0:  # invalid dims, or a selector they do not have
        raise MoeError("moe_pack_fp8_expert", moe_check_dims(d) or MOE_ERR_UNSUPPORTED)
    n = d.n_local if which in (MOE_W13, MOE_W2) else 1
    size = d.d * (d.I if which in (MOE_W13, MOE_W2) else d.shared_I) * n * (2 if which in (MOE_W13, MOE_WS13) else 1)
    _call(
        "moe_pack_fp8_expert", ctypes.byref(d), int(which), _buf(q, "q", size, T.e4m3, dev),
        _buf(scales, "scales", size // 16384, T.f32, dev), _buf(packed, "packed", need, T.bytes, dev), _on(stream, T, dev),
    )


def moe_fp8_ffn_workspace_bytes(dims) -> int:
    return lib().moe_fp8_ffn_workspace_bytes(ctypes.byref(_d(dims)))


def moe_fp8_expert_ffn(dims, x, w13_packed, w2_packed, counts, offsets, rows, active, ws13_packed, ws2_packed, y,
                       workspace, workspace_bytes=None, stream=None) -> None:
    """moe_expert_ffn on FP8 weights (moe_pack_fp8_expert)."""
    d, T = _d(dims), _t()
    dev = T.device()
    S, dd, I, Is, n_loc = d.S, d.d, d.I, d.shared_I, d.n_local  # noqa: E741
    r_max = d.r_max
    ws, nb = _workspace(workspace, workspace_bytes, T, dev)
    _call(
        "moe_fp8_expert_ffn", ctypes.byref(d), _buf(x, "x", S * dd, T.bf16, dev),
        _buf(w13_packed, "w13_packed", n_loc * _fp8_bytes(2 * I, dd), T.bytes, dev),
        _buf(w2_packed, "w2_packed", n_loc * _fp8_bytes(dd, I), T.bytes, dev),
        _buf(counts, "counts", n_loc, T.i32, dev), _buf(offsets, "offsets", n_loc + 1, T.i32, dev),
        _buf(rows, "rows", r_max, T.i32, dev), _buf(active, "active", n_loc + 1, T.i32, dev),
        _buf(ws13_packed, "ws13_packed", _fp8_bytes(2 * Is, dd), T.bytes, dev),
        _buf(ws2_packed, "ws2_packed", _fp8_bytes(dd, Is), T.bytes, dev),
        _buf(y, "y", (r_max + (S if Is else 0)) * dd, T.bf16, dev), ws, nb, _on(stream, T, dev),
    )


# ---------------------------------------------------------------- the router's balance


def balance_dims_from(cfg) -> MoeBalanceDims:
    """MoeBalanceDims from an object or dict with the moe_balance_dims field names."""
    get = cfg.get if isinstance(cfg, dict) else (lambda k, dflt=None: getattr(cfg, k, dflt))
    return MoeBalanceDims(
        T=get("T"), E=get("E"), topk=get("topk"), n_seq=get("n_seq", 1), score=get("score", MOE_SCORE_SIGMOID),
        coef=get("coef", 1.0),
    )


def _bd(dims) -> MoeBalanceDims:
    return dims if isinstance(dims, MoeBalanceDims) else balance_dims_from(dims)


def moe_check_balance_dims(dims) -> int:
    return lib().moe_check_balance_dims(ctypes.byref(_bd(dims)))


def moe_balance_workspace_bytes(dims) -> int:
    return lib().moe_balance_workspace_bytes(ctypes.byref(_bd(dims)))


def moe_expert_counts(dims, topk_ids, seq_starts, counts, workspace, workspace_bytes=None, stream=None) -> None:
    d, T = _bd(dims), _t()
    dev = T.device()
    ws, n = _workspace(workspace, workspace_bytes, T, dev)
    _call(
        "moe_expert_counts", ctypes.byref(d), _buf(topk_ids, "topk_ids", d.T * d.topk, T.i32, dev),
        _buf(seq_starts, "seq_starts", d.n_seq + 1, T.i32, dev), _buf(counts, "counts", d.n_seq * d.E, T.i32, dev),
        ws, n, _on(stream, T, dev),
    )


def moe_balance_loss(dims, logits, topk_ids, seq_starts, counts, probs, loss, workspace, workspace_bytes=None,
                     stream=None) -> None:
    d, T = _bd(dims), _t()
    dev = T.device()
    ws, n = _workspace(workspace, workspace_bytes, T, dev)
    _call(
        "moe_balance_loss", ctypes.byref(d), _buf(logits, "logits", d.T * d.E, T.f32, dev),
        _buf(topk_ids, "topk_ids", d.T * d.topk, T.i32, dev), _buf(seq_starts, "seq_starts", d.n_seq + 1, T.i32, dev),
        _buf(counts, "counts", d.n_seq * d.E, T.i32, dev), _buf(probs, "probs", d.n_seq * d.E, T.f32, dev),
        _buf(loss, "loss", 1, T.f32, dev), ws, n, _on(stream, T, dev),
    )


def moe_balance_backward(dims, logits, counts, seq_starts, dloss, dlogits, stream=None) -> None:
    """``dloss``: a one-element device tensor, or None for 1."""
    d, T = _bd(dims), _t()
    dev = T.device()
    _call(
        "moe_balance_backward", ctypes.byref(d), _buf(logits, "logits", d.T * d.E, T.f32, dev),
        _buf(counts, "counts", d.n_seq * d.E, T.i32, dev), _buf(seq_starts, "seq_starts", d.n_seq + 1, T.i32, dev),
        _buf(dloss, "dloss", 1, T.f32, dev), _buf(dlogits, "dlogits", d.T * d.E, T.f32, dev), _on(stream, T, dev),
    )


# ---------------------------------------------------------------- many rows: top-k


def gate_dims_from(cfg) -> MoeGateDims:
    """MoeGateDims from an object or dict with the moe_gate_dims field names."""
    get = cfg.get if isinstance(cfg, dict) else (lambda k, dflt=None: getattr(cfg, k, dflt))
    return MoeGateDims(
        T=get("T"), E=get("E"), topk=get("topk"), score=get("score", MOE_SCORE_SIGMOID), renorm=get("renorm", 1),
        bias_mode=get("bias_mode", 0),
    )


def _gd(dims) -> MoeGateDims:
    return dims if isinstance(dims, MoeGateDims) else gate_dims_from(dims)


def moe_check_gate_dims(dims) -> int:
    return lib().moe_check_gate_dims(ctypes.byref(_gd(dims)))


def moe_gate(dims, logits, bias, topk_ids, topk_w, stream=None) -> None:
    """Top-k of the rows' logits and the routing weights (``bias``: None, or what
    steers the selection under bias_mode 1)."""
    d, T = _gd(dims), _t()
    dev = T.device()
    _call(
        "moe_gate", ctypes.byref(d), _buf(logits, "logits", d.T * d.E, T.f32, dev), _buf(bias, "bias", d.E, T.f32, dev),
        _buf(topk_ids, "topk_ids", d.T * d.topk, T.i32, dev), _buf(topk_w, "topk_w", d.T * d.topk, T.f32, dev),
        _on(stream, T, dev),
    )


def moe_gate_backward(dims, logits, topk_ids, dtopk_w, dadd, dlogits, stream=None) -> None:
    """``dadd``: None, or a gradient of the logits that is added (it may be ``dlogits``)."""
    d, T = _gd(dims), _t()
    dev = T.device()
    _call(
        "moe_gate_backward", ctypes.byref(d), _buf(logits, "logits", d.T * d.E, T.f32, dev),
        _buf(topk_ids, "topk_ids", d.T * d.topk, T.i32, dev), _buf(dtopk_w, "dtopk_w", d.T * d.topk, T.f32, dev),
        _buf(dadd, "dadd", d.T * d.E, T.f32, dev), _buf(dlogits, "dlogits", d.T * d.E, T.f32, dev),
        _on(stream, T, dev),
    )


# ---------------------------------------------------------------- many rows: sorted by expert and back


def rows_dims_from(cfg) -> MoeRowsDims:
    """MoeRowsDims from an object or dict with the moe_rows_dims field names."""
    get = cfg.get if isinstance(cfg, dict) else (lambda k, dflt=None: getattr(cfg, k, dflt))
    return MoeRowsDims(
        T=get("T"), E=get("E"), topk=get("topk"), n_local=get("n_local"), local_base=get("local_base", 0),
        d=get("d", 1), tok_type=get("tok_type", MOE_BF16), row_type=get("row_type", MOE_BF16),
    )


def _rd(dims) -> MoeRowsDims:
    return dims if isinstance(dims, MoeRowsDims) else rows_dims_from(dims)


def moe_check_rows_dims(dims) -> int:
    return lib().moe_check_rows_dims(ctypes.byref(_rd(dims)))


def moe_sort_workspace_bytes(dims) -> int:
    return lib().moe_sort_workspace_bytes(ctypes.byref(_rd(dims)))


def moe_sort(dims, topk_ids, counts, offsets, rows, pick_pos, workspace, workspace_bytes=None, stream=None) -> None:
    d, T = _rd(dims), _t()
    dev = T.device()
    ws, n = _workspace(workspace, workspace_bytes, T, dev)
    picks = d.T * d.topk
    _call(
        "moe_sort", ctypes.byref(d), _buf(topk_ids, "topk_ids", picks, T.i32, dev),
        _buf(counts, "counts", d.n_local, T.i32, dev), _buf(offsets, "offsets", d.n_local + 1, T.i32, dev),
        _buf(rows, "rows", picks, T.i32, dev), _buf(pick_pos, "pick_pos", picks, T.i32, dev), ws, n,
        _on(stream, T, dev),
    )


def moe_dispatch(dims, x, pick_pos, xs, stream=None) -> None:
    """x [T, d] -> xs [T * topk, d], the picks' rows sorted by expert."""
    d, T = _rd(dims), _t()
    dev = T.device()
    picks = d.T * d.topk
    _call(
        "moe_dispatch", ctypes.byref(d), _buf(x, "x", d.T * d.d, T.rows.get(d.tok_type), dev),
        _buf(pick_pos, "pick_pos", picks, T.i32, dev), _buf(xs, "xs", picks * d.d, T.rows.get(d.row_type), dev),
        _on(stream, T, dev),
    )


def moe_return(dims, y, topk_w, pick_pos, out, stream=None) -> None:
    """The weighted sums of sorted rows (``topk_w`` None: plain sums, moe_dispatch's gradient)."""
    d, T = _rd(dims), _t()
    dev = T.device()
    picks = d.T * d.topk
    _call(
        "moe_return", ctypes.byref(d), _buf(y, "y", picks * d.d, T.rows.get(d.row_type), dev),
        _buf(topk_w, "topk_w", picks, T.f32, dev), _buf(pick_pos, "pick_pos", picks, T.i32, dev),
        _buf(out, "out", d.T * d.d, T.rows.get(d.tok_type), dev), _on(stream, T, dev),
    )


def moe_return_backward(dims, dout, y, topk_w, pick_pos, dy, dtopk_w, stream=None) -> None:
    d, T = _rd(dims), _t()
    dev = T.device()
    picks = d.T * d.topk
    row = T.rows.get(d.row_type)
    _call(
        "moe_return_backward", ctypes.byref(d), _buf(dout, "dout", d.T * d.d, T.rows.get(d.tok_type), dev),
        _buf(y, "y", picks * d.d, row, dev), _buf(topk_w, "topk_w", picks, T.f32, dev),
        _buf(pick_pos, "pick_pos", picks, T.i32, dev), _buf(dy, "dy", picks * d.d, row, dev),
        _buf(dtopk_w, "dtopk_w", picks, T.f32, dev), _on(stream, T, dev),
    )


# ---------------------------------------------------------------- many rows: MXFP4


def mx_dims_from(cfg) -> MoeMxDims:
    """MoeMxDims from an object or dict with the moe_mx_dims field names."""
    get = cfg.get if isinstance(cfg, dict) else (lambda k, dflt=None: getattr(cfg, k, dflt))
    return MoeMxDims(
        M=get("M", 1), N=get("N", 1), K=get("K"), in_type=get("in_type", MOE_BF16), out_type=get("out_type", MOE_BF16),
    )


def _xd(dims) -> MoeMxDims:
    return dims if isinstance(dims, MoeMxDims) else mx_dims_from(dims)


def moe_check_mx_dims(dims) -> int:
    return lib().moe_check_mx_dims(ctypes.byref(_xd(dims)))


def moe_packed_mx_bytes(dims) -> int:
    return lib().moe_packed_mx_bytes(ctypes.byref(_xd(dims)))


def moe_mx_gemm_workspace_bytes(dims) -> int:
    return lib().moe_mx_gemm_workspace_bytes(ctypes.byref(_xd(dims)))


def moe_mx_proj_workspace_bytes(dims) -> int:
    return lib().moe_mx_proj_workspace_bytes(ctypes.byref(_xd(dims)))


def moe_mx_quant(dims, x, q, scales, stream=None) -> None:
    """x [M, K] -> q [M, Kp / 2] uint8 (two codes a byte), scales [M, Kp / 32] uint8."""
    d, T = _xd(dims), _t()
    dev = T.device()
    kc = -(-d.K // 128)
    _call(
        "moe_mx_quant", ctypes.byref(d), _buf(x, "x", d.M * d.K, T.rows.get(d.in_type), dev),
        _buf(q, "q", d.M * kc * 64, T.bytes, dev), _buf(scales, "scales", d.M * kc * 4, T.bytes, dev),
        _on(stream, T, dev),
    )


def moe_mx_dequant(dims, q, scales, x, stream=None) -> None:
    """The values of MXFP4 rows: x [M, K] of dims.out_type."""
    d, T = _xd(dims), _t()
    dev = T.device()
    kc = -(-d.K // 128)
    _call(
        "moe_mx_dequant", ctypes.byref(d), _buf(q, "q", d.M * kc * 64, T.bytes, dev),
        _buf(scales, "scales", d.M * kc * 4, T.bytes, dev), _buf(x, "x", d.M * d.K, T.rows.get(d.out_type), dev),
        _on(stream, T, dev),
    )


def _mx_bytes(N: int, K: int) -> int:
    """Packed bytes of one [N, K] matrix: 64 x 128 tiles of 4352 bytes."""
    return -(-N // 64) * -(-K // 128) * 4352


def moe_pack_mx(dims, q, scales, packed, stream=None) -> None:
    d, T = _xd(dims), _t()
    dev = T.device()
    kc = -(-d.K // 128)
    _call(
        "moe_pack_mx", ctypes.byref(d), _buf(q, "q", d.N * kc * 64, T.bytes, dev),
        _buf(scales, "scales", d.N * kc * 4, T.bytes, dev), _buf(packed, "packed", _mx_bytes(d.N, d.K), T.bytes, dev),
        _on(stream, T, dev),
    )


def moe_mx_gemm(dims, xq, xs, w_packed, out, workspace, workspace_bytes=None, stream=None) -> None:
    d, T = _xd(dims), _t()
    dev = T.device()
    kc = -(-d.K // 128)
    ws, n = _workspace(workspace, workspace_bytes, T, dev)
    _call(
        "moe_mx_gemm", ctypes.byref(d), _buf(xq, "xq", d.M * kc * 64, T.bytes, dev),
        _buf(xs, "xs", d.M * kc * 4, T.bytes, dev), _buf(w_packed, "w_packed", _mx_bytes(d.N, d.K), T.bytes, dev),
        _buf(out, "out", d.M * d.N, T.rows.get(d.out_type), dev), ws, n, _on(stream, T, dev),
    )


def moe_mx_proj(dims, x, w_packed, out, workspace, workspace_bytes=None, stream=None) -> None:
    """moe_mx_quant of x and moe_mx_gemm in one call."""
    d, T = _xd(dims), _t()
    dev = T.device()
    ws, n = _workspace(workspace, workspace_bytes, T, dev)
    _call(
        "moe_mx_proj", ctypes.byref(d), _buf(x, "x", d.M * d.K, T.rows.get(d.in_type), dev),
        _buf(w_packed, "w_packed", _mx_bytes(d.N, d.K), T.bytes, dev),
        _buf(out, "out", d.M * d.N, T.rows.get(d.out_type), dev), ws, n, _on(stream, T, dev),
    )


def mx_group_dims_from(cfg) -> MoeMxGroupDims:
    """MoeMxGroupDims from an object or dict with the moe_mx_group_dims field names."""
    get = cfg.get if isinstance(cfg, dict) else (lambda k, dflt=None: getattr(cfg, k, dflt))
    return MoeMxGroupDims(
        T=get("T"), E=get("E"), topk=get("topk"), n_local=get("n_local"), d=get("d"), I=get("I"),
        h_type=get("h_type", MOE_MXFP4), out_type=get("out_type", MOE_BF16),
    )


def _xg(dims) -> MoeMxGroupDims:
    return dims if isinstance(dims, MoeMxGroupDims) else mx_group_dims_from(dims)


def moe_check_mx_group_dims(dims) -> int:
    return lib().moe_check_mx_group_dims(ctypes.byref(_xg(dims)))


def moe_mx_gate_up(dims, xq, xs, offsets, rows, w13_packed, h, hs=None, stream=None) -> None:
    """gate_up with SwiGLU of sorted rows: h bf16 [T * topk, I], or (h_type MOE_MXFP4)
    codes [T * topk, I / 2] with scale bytes hs [T * topk, I / 32]."""
    d, T = _xg(dims), _t()
    dev = T.device()
    picks, mx = d.T * d.topk, d.h_type == MOE_MXFP4
    _call(
        "moe_mx_gate_up", ctypes.byref(d), _buf(xq, "xq", d.T * d.d // 2, T.bytes, dev),
        _buf(xs, "xs", d.T * d.d // 32, T.bytes, dev), _buf(offsets, "offsets", d.n_local + 1, T.i32, dev),
        _buf(rows, "rows", picks, T.i32, dev),
        _buf(w13_packed, "w13_packed", d.n_local * _mx_bytes(2 * d.I, d.d), T.bytes, dev),
        _buf(h, "h", picks * d.I // 2 if mx else picks * d.I, T.bytes if mx else T.bf16, dev),
        _buf(hs, "hs", picks * d.I // 32 if mx else 0, T.bytes, dev), _on(stream, T, dev),
    )


def moe_mx_down(dims, hq, hs, offsets, w2_packed, y, stream=None) -> None:
    """down of sorted MXFP4 rows: y [T * topk, d] of dims.out_type."""
    d, T = _xg(dims), _t()
    dev = T.device()
    picks = d.T * d.topk
    _call(
        "moe_mx_down", ctypes.byref(d), _buf(hq, "hq", picks * d.I // 2, T.bytes, dev),
        _buf(hs, "hs", picks * d.I // 32, T.bytes, dev), _buf(offsets, "offsets", d.n_local + 1, T.i32, dev),
        _buf(w2_packed, "w2_packed", d.n_local * _mx_bytes(d.d, d.I), T.bytes, dev),
        _buf(y, "y", picks * d.d, T.rows.get(d.out_type), dev), _on(stream, T, dev),
    )
