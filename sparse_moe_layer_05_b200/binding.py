"""ctypes binding of ``libmoe_b200.so`` (the C ABI in ``include/moe_b200.h``).

Argument marshalling only: every step of the layer runs in the library's CUDA
kernels. Tensors are torch CUDA tensors (torch provides device memory and
streams); functions keep the C names. There is no CPU fallback: if the
library or a CUDA device is missing, the calls raise.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libmoe_b200.so")

STATUS = {
    0: "MOE_OK",
    1: "MOE_ERR_INVALID_ARG",
    2: "MOE_ERR_UNSUPPORTED",
    3: "MOE_ERR_WORKSPACE",
    4: "MOE_ERR_CUDA",
    5: "MOE_ERR_TIMEOUT",
    6: "MOE_ERR_NO_DEVICE",
}

EXPORTS = [
    "moe_status_string", "moe_version", "moe_workspace_size", "moe_forward",
    "moe_workspace_size_hostio", "moe_forward_hostio", "moe_route_workspace_size",
    "moe_route", "moe_workspace_layout", "moe_mxfp4_to_bf16", "moe_mx_split_e4m3", "moe_sync_status",
    "moe_selftest_wait_timeout", "moe_forward_launch_count", "moe_forward_timed",
    "moe_set_tile_policy", "moe_route_noalloc",
    "moe_workspace_size_block", "moe_forward_block", "moe_rms_norm", "moe_forward_biased",
    "moe_forward_timed_events", "moe_forward_ex", "moe_mx_quantize", "moe_forward_timed_ex",
    "moe_balance_loss_workspace_size", "moe_balance_loss", "moe_balance_loss_backward",
    "moe_gate_backward", "moe_router_backward_workspace_size", "moe_router_backward",
    "moe_rms_norm_checkpoint", "moe_rms_norm_backward_workspace_size", "moe_rms_norm_backward",
    "moe_forward_block_checkpoint",
]
# the measurement library (libmoe_b200_probe.so, include/moe_b200_probe.h)
PROBE_EXPORTS = ["moe_probe_tensor_rate", "moe_probe_error_string", "moe_probe_error_site"]
PROBE_LIB_PATH = os.path.join(PKG, "libmoe_b200_probe.so")

# moe_forward_opts.act_quant
ACT_BF16, ACT_MXFP8, ACT_MXFP4 = 0, 1, 2
ACT_MODES = {"bf16": ACT_BF16, "mxfp8": ACT_MXFP8, "mxfp4": ACT_MXFP4}

STAGES = ["router_logits", "topk_softmax", "perm_hist", "perm_scan", "perm_scatter",
          "gather_rows", "transpose_scales_gu", "transpose_scales_d", "gemm_gateup_swiglu",
          "gemm_down_combine", "combine"]


class MoEError(RuntimeError):
    def __init__(self, fn: str, code: int):
        super().__init__(f"{fn} returned {STATUS.get(code, code)}")
        self.code = code


class ForwardOpts(ctypes.Structure):
    """moe_forward_opts (include/moe_b200.h)."""
    _fields_ = [("tile_policy", ctypes.c_int), ("act_quant", ctypes.c_int),
                ("gu_bias_dev", ctypes.c_void_p), ("down_bias_dev", ctypes.c_void_p)]


class WsLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("logits", "topk_idx", "topk_w", "counts", "offsets", "perm", "xp", "h", "yw",
                 "status", "total", "x_scales", "h_scales")]


_lib = None


def load(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the library (once). Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m sparse_moe_layer_05_b200.build`")
    lib = ctypes.CDLL(p)
    vp, sz, i32, u8p, fp = (ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int,
                            ctypes.c_void_p, ctypes.c_void_p)
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_status_string.argtypes = [i32]
    lib.moe_version.restype = i32
    lib.moe_workspace_size.restype = sz
    lib.moe_workspace_size.argtypes = [i32] * 5
    lib.moe_workspace_size_hostio.restype = sz
    lib.moe_workspace_size_hostio.argtypes = [i32] * 5
    lib.moe_route_workspace_size.restype = sz
    lib.moe_route_workspace_size.argtypes = [i32] * 4
    fwd = [vp, fp, fp, u8p, u8p, u8p, u8p, i32, i32, i32, i32, i32, vp, vp, sz, vp]
    lib.moe_forward.restype = i32
    lib.moe_forward.argtypes = fwd
    lib.moe_forward_hostio.restype = i32
    lib.moe_forward_hostio.argtypes = fwd
    lib.moe_forward_timed.restype = i32
    lib.moe_forward_timed.argtypes = fwd + [ctypes.POINTER(ctypes.c_float)]
    lib.moe_forward_timed_events.restype = i32
    lib.moe_forward_timed_events.argtypes = fwd + [ctypes.c_uint, ctypes.POINTER(ctypes.c_float)]
    lib.moe_route.restype = i32
    lib.moe_route.argtypes = [vp, fp, fp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_route_noalloc.restype = i32
    lib.moe_route_noalloc.argtypes = [vp, fp, fp, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp]
    lib.moe_workspace_layout.restype = i32
    lib.moe_workspace_layout.argtypes = [i32] * 5 + [ctypes.POINTER(WsLayout)]
    lib.moe_mxfp4_to_bf16.restype = i32
    lib.moe_mxfp4_to_bf16.argtypes = [u8p, u8p, i32, i32, vp, vp]
    lib.moe_workspace_size_block.restype = sz
    lib.moe_workspace_size_block.argtypes = [i32] * 5
    lib.moe_forward_block.restype = i32
    # the biased forms: gate/up bias after the gate/up weights, down bias after the down ones
    fwd_b = fwd[:5] + [fp] + fwd[5:7] + [fp] + fwd[7:]
    lib.moe_forward_biased.restype = i32
    lib.moe_forward_biased.argtypes = fwd_b
    lib.moe_forward_block.argtypes = [vp, fp, ctypes.c_float] + fwd_b[1:]
    lib.moe_rms_norm.restype = i32
    lib.moe_rms_norm.argtypes = [vp, fp, ctypes.c_float, i32, i32, vp, vp]
    lib.moe_forward_ex.restype = i32
    lib.moe_forward_ex.argtypes = fwd[:15] + [ctypes.POINTER(ForwardOpts), vp]
    lib.moe_forward_timed_ex.restype = i32
    lib.moe_forward_timed_ex.argtypes = fwd[:15] + [ctypes.POINTER(ForwardOpts), vp, ctypes.c_uint,
                                                    ctypes.POINTER(ctypes.c_float)]
    lib.moe_mx_quantize.restype = i32
    lib.moe_mx_quantize.argtypes = [vp, i32, i32, i32, u8p, u8p, vp]
    lib.moe_mx_split_e4m3.restype = i32
    lib.moe_mx_split_e4m3.argtypes = [vp, i32, i32, u8p, u8p, u8p, vp]
    lib.moe_sync_status.restype = i32
    lib.moe_sync_status.argtypes = [vp, sz, vp]
    lib.moe_selftest_wait_timeout.restype = i32
    lib.moe_selftest_wait_timeout.argtypes = [vp, vp]
    lib.moe_set_tile_policy.restype = i32
    lib.moe_set_tile_policy.argtypes = [i32]
    lib.moe_forward_launch_count.restype = i32
    lib.moe_forward_launch_count.argtypes = [i32] * 5
    f32 = ctypes.c_float
    lib.moe_balance_loss_workspace_size.restype = sz
    lib.moe_balance_loss_workspace_size.argtypes = [i32] * 3
    lib.moe_balance_loss.restype = i32
    lib.moe_balance_loss.argtypes = [vp, vp, vp, i32, i32, i32, f32, f32, vp, vp, vp, vp, vp, sz, vp]
    lib.moe_balance_loss_backward.restype = i32
    lib.moe_balance_loss_backward.argtypes = [vp] * 5 + [i32, i32, i32, f32, f32, vp, i32, vp, vp]
    lib.moe_gate_backward.restype = i32
    lib.moe_gate_backward.argtypes = [vp] * 5 + [i32] * 5 + [vp, vp]
    lib.moe_router_backward_workspace_size.restype = sz
    lib.moe_router_backward_workspace_size.argtypes = [i32] * 3
    lib.moe_router_backward.restype = i32
    lib.moe_router_backward.argtypes = ([vp] * 8 + [i32] * 3 + [vp, i32] + [vp] * 4 + [sz, vp])
    lib.moe_rms_norm_checkpoint.restype = i32
    lib.moe_rms_norm_checkpoint.argtypes = [vp, vp, f32, i32, i32, vp, vp, vp, vp, vp]
    lib.moe_rms_norm_backward_workspace_size.restype = sz
    lib.moe_rms_norm_backward_workspace_size.argtypes = [i32] * 2
    lib.moe_rms_norm_backward.restype = i32
    lib.moe_rms_norm_backward.argtypes = [vp] * 7 + [i32, i32, vp, i32, vp, vp, vp, sz, vp]
    lib.moe_forward_block_checkpoint.restype = i32
    lib.moe_forward_block_checkpoint.argtypes = ([vp, fp, f32] + fwd_b[1:15] + [vp, vp, vp]
                                                 + fwd_b[15:])
    _lib = lib
    return lib


_probe_lib = None


def load_probe(path: Optional[str] = None) -> ctypes.CDLL:
    """Load the tensor-core rate probe library (measurement tooling)."""
    global _probe_lib
    if _probe_lib is not None:
        return _probe_lib
    p = path or PROBE_LIB_PATH
    if not os.path.exists(p):
        raise RuntimeError(f"{p} is missing: build it with `python -m sparse_moe_layer_05_b200.build`")
    lib = ctypes.CDLL(p)
    lib.moe_probe_tensor_rate.restype = ctypes.c_int
    lib.moe_probe_tensor_rate.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                          ctypes.POINTER(ctypes.c_double), ctypes.c_void_p]
    lib.moe_probe_error_string.restype = ctypes.c_char_p
    lib.moe_probe_error_site.restype = ctypes.c_char_p
    _probe_lib = lib
    return lib


def _check(fn: str, code: int) -> None:
    if code != 0:
        raise MoEError(fn, code)


def _ptr(t) -> int:
    if t is None:
        return 0
    return int(t.data_ptr())


def _stream(stream) -> int:
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream)


def _require_cuda(*ts) -> None:
    for t in ts:
        if t is not None and not t.is_cuda:
            raise ValueError("expected CUDA tensors")
        if t is not None and not t.is_contiguous():
            raise ValueError("expected contiguous tensors")


# element types of the training calls' tensors: names, resolved to torch dtypes
# on first use (torch is imported where it is needed only)
_F32, _F16, _I32, _U8, _E4M3, _E8M0 = range(6)
_KINDS = ("f32", "bf16", "i32", "u8", "e4m3", "e8m0")
_DTYPES = None
_torch_c = None


def _device() -> int:
    """Index of the current CUDA device."""
    global _DTYPES, _torch_c
    if _DTYPES is None:
        import torch
        torch.cuda.init()
        _torch_c = torch._C
        _DTYPES = ((torch.float32,), (torch.bfloat16, torch.uint16), (torch.int32,),
                   (torch.uint8, torch.bool), (torch.uint8, torch.float8_e4m3fn),
                   (torch.uint8, torch.float8_e8m0fnu))
    return _torch_c._cuda_getDevice()


def _args(cur: int, specs) -> list:
    """Pointers of the tensors of a training call, checked: on device ``cur`` (the
    current one), contiguous, and of the type and number of elements that each
    (name, tensor, type, elements) asks for; a None tensor gives a null pointer.
    Without these checks a wrong size would be read past its end."""
    ptrs = []
    for name, t, kind, n in specs:
        if t is None:
            ptrs.append(None)
        elif (t.get_device() == cur and t.dtype in _DTYPES[kind] and t.numel() == n
              and t.is_contiguous()):
            ptrs.append(t.data_ptr())
        elif t.get_device() != cur:
            raise ValueError(f"{name}: expected a tensor on the current CUDA device")
        elif t.dtype not in _DTYPES[kind]:
            raise ValueError(f"{name}: expected {_KINDS[kind]} elements, got {t.dtype}")
        elif t.numel() != n:
            raise ValueError(f"{name}: expected {n} elements, got {t.numel()}")
        else:
            raise ValueError(f"{name}: expected a contiguous tensor")
    return ptrs


def _raw_stream(stream, cur: int) -> int:
    return int(stream.cuda_stream) if stream is not None else _torch_c._cuda_getCurrentRawStream(cur)


# ---------------------------------------------------------------- sizes ----

def moe_workspace_size(E: int, k: int, T: int, d: int, I: int) -> int:
    return int(load().moe_workspace_size(E, k, T, d, I))


def moe_workspace_size_hostio(E: int, k: int, T: int, d: int, I: int) -> int:
    return int(load().moe_workspace_size_hostio(E, k, T, d, I))


def moe_route_workspace_size(E: int, k: int, T: int, d: int) -> int:
    return int(load().moe_route_workspace_size(E, k, T, d))


def moe_workspace_layout(E: int, k: int, T: int, d: int, I: int) -> dict:
    L = WsLayout()
    _check("moe_workspace_layout", load().moe_workspace_layout(E, k, T, d, I, ctypes.byref(L)))
    return {n: getattr(L, n) for n, _ in WsLayout._fields_}


def moe_forward_launch_count(E: int, k: int, T: int, d: int, I: int) -> int:
    return int(load().moe_forward_launch_count(E, k, T, d, I))


# ---------------------------------------------------------------- calls ----

def moe_forward(x, W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes, Wd_scales, E, k, T, d, I,
                out, workspace, stream=None) -> None:
    """Enqueue the forward pass (see include/moe_b200.h). x/out: uint16 or bf16 [T, d]."""
    _require_cuda(x, W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes, Wd_scales, out, workspace)
    _check("moe_forward", load().moe_forward(
        _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(Wgu_codes), _ptr(Wgu_scales), _ptr(Wd_codes),
        _ptr(Wd_scales), E, k, T, d, I, _ptr(out), _ptr(workspace), workspace.numel(),
        _stream(stream)))


def moe_forward_biased(x, W_r, b_r, Wgu_codes, Wgu_scales, gu_bias, Wd_codes, Wd_scales, down_bias,
                       E, k, T, d, I, out, workspace, stream=None) -> None:
    """moe_forward with per-expert biases: gu_bias f32 [E, 2I] (gate then up),
    down_bias f32 [E, d]; either may be None."""
    _require_cuda(x, W_r, b_r, Wgu_codes, Wgu_scales, gu_bias, Wd_codes, Wd_scales, down_bias, out,
                  workspace)
    _check("moe_forward_biased", load().moe_forward_biased(
        _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(Wgu_codes), _ptr(Wgu_scales), _ptr(gu_bias),
        _ptr(Wd_codes), _ptr(Wd_scales), _ptr(down_bias), E, k, T, d, I, _ptr(out),
        _ptr(workspace), workspace.numel(), _stream(stream)))


def moe_forward_ex(x, W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes, Wd_scales, E, k, T, d, I,
                   out, workspace, tile_policy: int = 0, act_quant=ACT_BF16, gu_bias=None,
                   down_bias=None, stream=None) -> None:
    """moe_forward with per-call options: tile_policy (-1 process default, 0 by
    shape, 1..4 forced), act_quant (ACT_BF16, ACT_MXFP8, ACT_MXFP4 or their
    names), optional expert biases."""
    _require_cuda(x, W_r, b_r, Wgu_codes, Wgu_scales, gu_bias, Wd_codes, Wd_scales, down_bias, out,
                  workspace)
    if isinstance(act_quant, str):
        act_quant = ACT_MODES[act_quant]
    o = ForwardOpts(tile_policy, act_quant, _ptr(gu_bias) or None, _ptr(down_bias) or None)
    _check("moe_forward_ex", load().moe_forward_ex(
        _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(Wgu_codes), _ptr(Wgu_scales), _ptr(Wd_codes),
        _ptr(Wd_scales), E, k, T, d, I, _ptr(out), _ptr(workspace), workspace.numel(),
        ctypes.byref(o), _stream(stream)))


def moe_forward_timed(x, W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes, Wd_scales, E, k, T, d, I,
                      out, workspace, stream=None) -> list:
    """Forward pass with per-launch CUDA-event timing; returns len(STAGES)+1
    floats (ms): one per launch in the order of STAGES, then the whole span.
    Blocks."""
    _require_cuda(x, W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes, Wd_scales, out, workspace)
    ms = (ctypes.c_float * (len(STAGES) + 1))()
    _check("moe_forward_timed", load().moe_forward_timed(
        _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(Wgu_codes), _ptr(Wgu_scales), _ptr(Wd_codes),
        _ptr(Wd_scales), E, k, T, d, I, _ptr(out), _ptr(workspace), workspace.numel(),
        _stream(stream), ms))
    return list(ms)


def moe_forward_timed_events(x, W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes, Wd_scales, E, k, T, d,
                             I, out, workspace, event_mask: int, stream=None) -> list:
    """moe_forward_timed recording only the boundaries in event_mask (bit i:
    before launch i, bit len(STAGES): after the last); entries of unrecorded
    boundaries are 0, each recorded one spans to the next recorded. Blocks."""
    _require_cuda(x, W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes, Wd_scales, out, workspace)
    ms = (ctypes.c_float * (len(STAGES) + 1))()
    _check("moe_forward_timed_events", load().moe_forward_timed_events(
        _ptr(x), _ptr(W_r), _ptr(b_r), _ptr(Wgu_codes), _ptr(Wgu_scales), _ptr(Wd_codes),
        _ptr(Wd_scales), E, k, T, d, I, _ptr(out), _ptr(workspace), workspace.numel(),
        _stream(stream), event_mask, ms))
    return list(ms)


def moe_forward_hostio(x_host, W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes, Wd_scales, E, k, T, d,
                       I, out_host, workspace, stream=None) -> None:
    """Forward pass with x and out in host memory (pinned for async copies); synchronises."""
    _require_cuda(W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes, Wd_scales, workspace)
    if x_host.is_cuda or out_host.is_cuda:
        raise ValueError("x_host and out_host must be host tensors")
    _check("moe_forward_hostio", load().moe_forward_hostio(
        _ptr(x_host), _ptr(W_r), _ptr(b_r), _ptr(Wgu_codes), _ptr(Wgu_scales), _ptr(Wd_codes),
        _ptr(Wd_scales), E, k, T, d, I, _ptr(out_host), _ptr(workspace), workspace.numel(),
        _stream(stream)))


def moe_route(x, W_r, b_r, E, k, T, d, topk_idx, topk_w, counts=None, offsets=None, perm=None,
              workspace=None, stream=None) -> None:
    _require_cuda(x, W_r, b_r, topk_idx, topk_w, counts, offsets, perm, workspace)
    _check("moe_route", load().moe_route(
        _ptr(x), _ptr(W_r), _ptr(b_r), E, k, T, d, _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
        _ptr(offsets), _ptr(perm), _ptr(workspace), workspace.numel(), _stream(stream)))


def moe_route_noalloc(x, W_r, b_r, E, k, T, d, topk_idx, topk_w, counts, offsets, perm,
                      stream=None) -> None:
    """moe_route with the library's own fixed device scratch (no workspace):
    for callers that cannot allocate; T * E <= 1,048,576."""
    _require_cuda(x, W_r, b_r, topk_idx, topk_w, counts, offsets, perm)
    _check("moe_route_noalloc", load().moe_route_noalloc(
        _ptr(x), _ptr(W_r), _ptr(b_r), E, k, T, d, _ptr(topk_idx), _ptr(topk_w), _ptr(counts),
        _ptr(offsets), _ptr(perm), _stream(stream)))


def moe_workspace_size_block(E: int, k: int, T: int, d: int, I: int) -> int:
    return int(load().moe_workspace_size_block(E, k, T, d, I))


def moe_rms_norm(h, g, eps: float, T: int, d: int, x, stream=None) -> None:
    _require_cuda(h, g, x)
    _check("moe_rms_norm", load().moe_rms_norm(_ptr(h), _ptr(g), eps, T, d, _ptr(x), _stream(stream)))


def moe_forward_block(h, g, eps: float, W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes, Wd_scales,
                      E: int, k: int, T: int, d: int, I: int, out, workspace, stream=None,
                      gu_bias=None, down_bias=None) -> None:
    """out = h + MoE(RMSNorm(h)) (bf16 rows; g f32 gain; optional expert biases)."""
    _require_cuda(h, g, W_r, b_r, Wgu_codes, Wgu_scales, gu_bias, Wd_codes, Wd_scales, down_bias,
                  out, workspace)
    _check("moe_forward_block", load().moe_forward_block(
        _ptr(h), _ptr(g), eps, _ptr(W_r), _ptr(b_r), _ptr(Wgu_codes), _ptr(Wgu_scales),
        _ptr(gu_bias), _ptr(Wd_codes), _ptr(Wd_scales), _ptr(down_bias), E, k, T, d, I,
        _ptr(out), _ptr(workspace), workspace.numel(), _stream(stream)))


def moe_probe_tensor_rate(kind: int, N: int, per_commit: int, stream=None) -> float:
    """MACs per SM clock of back-to-back UMMAs (kind 0 bf16, 1 block-scaled
    E2M1 x E4M3, 2 block-scaled E2M1 x E2M1), from the probe library."""
    out = ctypes.c_double(0.0)
    lib = load_probe()
    code = lib.moe_probe_tensor_rate(kind, N, per_commit, ctypes.byref(out), _stream(stream))
    if code == 4:        # MOE_ERR_CUDA: say which call failed and how
        raise MoEError(f"moe_probe_tensor_rate ({lib.moe_probe_error_site().decode()}: "
                       f"{lib.moe_probe_error_string().decode()})", code)
    _check("moe_probe_tensor_rate", code)
    return out.value


def moe_mx_quantize(x, rows: int, K: int, act_quant, q, scales, stream=None) -> None:
    """The quantised modes' activation conversion on plain bf16 rows: q [rows, K]
    E4M3 (ACT_MXFP8) or [rows, K/2] packed E2M1 (ACT_MXFP4), scales [rows, K/32]."""
    _require_cuda(x, q, scales)
    if isinstance(act_quant, str):
        act_quant = ACT_MODES[act_quant]
    _check("moe_mx_quantize", load().moe_mx_quantize(
        _ptr(x), rows, K, act_quant, _ptr(q), _ptr(scales), _stream(stream)))


def moe_mx_split_e4m3(x, rows: int, K: int, hi, lo, scales, stream=None) -> None:
    _require_cuda(x, hi, lo, scales)
    _check("moe_mx_split_e4m3", load().moe_mx_split_e4m3(
        _ptr(x), rows, K, _ptr(hi), _ptr(lo), _ptr(scales), _stream(stream)))


def moe_mxfp4_to_bf16(codes, scales, rows: int, K: int, out, stream=None) -> None:
    _require_cuda(codes, scales, out)
    _check("moe_mxfp4_to_bf16", load().moe_mxfp4_to_bf16(
        _ptr(codes), _ptr(scales), rows, K, _ptr(out), _stream(stream)))


# ------------------------------------------------- training the router ----

def moe_balance_loss_workspace_size(E: int, k: int, T: int) -> int:
    return int(load().moe_balance_loss_workspace_size(E, k, T))


def moe_router_backward_workspace_size(E: int, T: int, d: int) -> int:
    return int(load().moe_router_backward_workspace_size(E, T, d))


def moe_rms_norm_backward_workspace_size(T: int, d: int) -> int:
    return int(load().moe_rms_norm_backward_workspace_size(T, d))


def moe_balance_loss(logits, topk_idx, E: int, k: int, T: int, balance_coef: float, z_coef: float,
                     stats, counts, mean_probs, lse, workspace, token_mask=None,
                     stream=None) -> None:
    """Load-balance and z loss of logits [T, E] f32 with the per-expert counts:
    stats f32 [4] (loss, balance, z, live tokens), counts i32 [E], mean_probs
    f32 [E], lse f32 [T]. token_mask u8 or bool [T]: 0 leaves a token out."""
    cur = _device()
    lo, ix, mk, sa, co, mp, ls, ws = _args(cur, (
        ("logits", logits, _F32, T * E),
        ("topk_idx", topk_idx, _I32, T * k),
        ("token_mask", token_mask, _U8, T),
        ("stats", stats, _F32, 4),
        ("counts", counts, _I32, E),
        ("mean_probs", mean_probs, _F32, E),
        ("lse", lse, _F32, T),
        ("workspace", workspace, _U8, workspace.numel())))
    _check("moe_balance_loss", load().moe_balance_loss(
        lo, ix, mk, E, k, T, balance_coef, z_coef, sa, co, mp, ls, ws, workspace.numel(),
        _raw_stream(stream, cur)))


def moe_balance_loss_backward(logits, lse, counts, stats, E: int, k: int, T: int,
                              balance_coef: float, z_coef: float, dlogits, dloss=None,
                              token_mask=None, accumulate: bool = False, stream=None) -> None:
    """dlogits [T, E] f32 (+)= gradient of moe_balance_loss; dloss f32 [1] on the
    device (None: 1)."""
    cur = _device()
    lo, ls, co, sa, mk, dv, dl = _args(cur, (
        ("logits", logits, _F32, T * E),
        ("lse", lse, _F32, T),
        ("counts", counts, _I32, E),
        ("stats", stats, _F32, 4),
        ("token_mask", token_mask, _U8, T),
        ("dloss", dloss, _F32, 1),
        ("dlogits", dlogits, _F32, T * E)))
    _check("moe_balance_loss_backward", load().moe_balance_loss_backward(
        lo, ls, co, sa, mk, E, k, T, balance_coef, z_coef, dv, int(accumulate), dl,
        _raw_stream(stream, cur)))


def moe_gate_backward(dout, yw, topk_idx, topk_w, E: int, k: int, T: int, d: int, dlogits,
                      token_mask=None, accumulate: bool = False, stream=None) -> None:
    """dlogits [T, E] f32 (+)= gradient through the selected-set softmax, from
    dout bf16 [T, d] and the weighted expert rows yw f32 [T*k, d]."""
    cur = _device()
    do, yp, ix, wp, mk, dl = _args(cur, (
        ("dout", dout, _F16, T * d),
        ("yw", yw, _F32, T * k * d),
        ("topk_idx", topk_idx, _I32, T * k),
        ("topk_w", topk_w, _F32, T * k),
        ("token_mask", token_mask, _U8, T),
        ("dlogits", dlogits, _F32, T * E)))
    _check("moe_gate_backward", load().moe_gate_backward(
        do, yp, ix, wp, mk, E, k, T, d, int(accumulate), dl, _raw_stream(stream, cur)))


def moe_router_backward(dlogits, W_r, E: int, T: int, d: int, dW, db, dx, workspace, x=None,
                        q=None, scales=None, rstd=None, g=None, dx_in=None, token_mask=None,
                        accumulate: bool = False, stream=None) -> None:
    """dW f32 [E, d], db f32 [E], dx bf16 [T, d] (each may be None) from dlogits
    f32 [T, E]; the input rows as x bf16 [T, d], or as the checkpoint q, scales,
    rstd with the norm's gain g."""
    cur = _device()
    dl, wr, xp, qp, sp, rp, gp, mk, di, dw, bp, dp, ws = _args(cur, (
        ("dlogits", dlogits, _F32, T * E),
        ("W_r", W_r, _F32, E * d),
        ("x", x, _F16, T * d),
        ("q", q, _E4M3, T * d),
        ("scales", scales, _E8M0, T * (d // 32)),
        ("rstd", rstd, _F32, T),
        ("g", g, _F32, d),
        ("token_mask", token_mask, _U8, T),
        ("dx_in", dx_in, _F16, T * d),
        ("dW", dW, _F32, E * d),
        ("db", db, _F32, E),
        ("dx", dx, _F16, T * d),
        ("workspace", workspace, _U8, workspace.numel())))
    _check("moe_router_backward", load().moe_router_backward(
        dl, wr, xp, qp, sp, rp, gp, mk, E, T, d, di, int(accumulate), dw, bp, dp, ws,
        workspace.numel(), _raw_stream(stream, cur)))


def moe_rms_norm_checkpoint(h, g, eps: float, T: int, d: int, x, q, scales, rstd,
                            stream=None) -> None:
    """moe_rms_norm that also leaves h as an 8-bit checkpoint: q E4M3 [T, d],
    scales E8M0 [T, d/32], and rstd f32 [T]; x may be None."""
    cur = _device()
    hp, gp, xp, qp, sp, rp = _args(cur, (
        ("h", h, _F16, T * d),
        ("g", g, _F32, d),
        ("x", x, _F16, T * d),
        ("q", q, _E4M3, T * d),
        ("scales", scales, _E8M0, T * (d // 32)),
        ("rstd", rstd, _F32, T)))
    _check("moe_rms_norm_checkpoint", load().moe_rms_norm_checkpoint(
        hp, gp, eps, T, d, xp, qp, sp, rp, _raw_stream(stream, cur)))


def moe_rms_norm_backward(dx, g, rstd, T: int, d: int, dh, dg, workspace, h=None, q=None,
                          scales=None, dh_in=None, token_mask=None, accumulate: bool = False,
                          stream=None) -> None:
    """dh bf16 [T, d] and dg f32 [d] of the norm, from its bf16 input rows h or
    their checkpoint q, scales."""
    cur = _device()
    dp, hp, qp, sp, rp, gp, mk, di, oh, og, ws = _args(cur, (
        ("dx", dx, _F16, T * d),
        ("h", h, _F16, T * d),
        ("q", q, _E4M3, T * d),
        ("scales", scales, _E8M0, T * (d // 32)),
        ("rstd", rstd, _F32, T),
        ("g", g, _F32, d),
        ("token_mask", token_mask, _U8, T),
        ("dh_in", dh_in, _F16, T * d),
        ("dh", dh, _F16, T * d),
        ("dg", dg, _F32, d),
        ("workspace", workspace, _U8, workspace.numel())))
    _check("moe_rms_norm_backward", load().moe_rms_norm_backward(
        dp, hp, qp, sp, rp, gp, mk, T, d, di, int(accumulate), oh, og, ws, workspace.numel(),
        _raw_stream(stream, cur)))


def moe_forward_block_checkpoint(h, g, eps: float, W_r, b_r, Wgu_codes, Wgu_scales, Wd_codes,
                                 Wd_scales, E: int, k: int, T: int, d: int, I: int, out, q, scales,
                                 rstd, workspace, stream=None, gu_bias=None,
                                 down_bias=None) -> None:
    """moe_forward_block that also leaves the norm's 8-bit checkpoint."""
    _require_cuda(h, g, W_r, b_r, Wgu_codes, Wgu_scales, gu_bias, Wd_codes, Wd_scales, down_bias,
                  out, workspace)
    qp, sp, rp = _args(_device(), (("q", q, _E4M3, T * d), ("scales", scales, _E8M0, T * (d // 32)),
                                   ("rstd", rstd, _F32, T)))
    _check("moe_forward_block_checkpoint", load().moe_forward_block_checkpoint(
        _ptr(h), _ptr(g), eps, _ptr(W_r), _ptr(b_r), _ptr(Wgu_codes), _ptr(Wgu_scales),
        _ptr(gu_bias), _ptr(Wd_codes), _ptr(Wd_scales), _ptr(down_bias), E, k, T, d, I,
        _ptr(out), qp, sp, rp, _ptr(workspace), workspace.numel(), _stream(stream)))


TILE_AUTO, TILE_SINGLE, TILE_PAIR, TILE_SWAP, TILE_MX, TILE_MX_PAIR = 0, 1, 2, 3, 4, 5


def moe_set_tile_policy(policy: int) -> None:
    """0 = by shape, 1 = single-CTA, 2 = CTA-pair, 3 = swapped-operand,
    4 = block-scaled tiles, 5 = block-scaled tiles on a CTA pair: the process
    default of the calls without options (moe_forward_ex takes one per call)."""
    _check("moe_set_tile_policy", load().moe_set_tile_policy(policy))


def moe_sync_status(workspace, stream=None) -> int:
    """Synchronise, then return (and clear) the device status code."""
    return int(load().moe_sync_status(_ptr(workspace), workspace.numel(), _stream(stream)))


def moe_selftest_wait_timeout(workspace, stream=None) -> None:
    _check("moe_selftest_wait_timeout",
           load().moe_selftest_wait_timeout(_ptr(workspace), _stream(stream)))


# ----------------------------------------------------------- convenience ----

def _result(T: int, d: int, device, stream):
    """Room for a bf16 [T, d] result that kernels on `stream` (None: the current one)
    write. The allocator hands a block out again in the order of the stream that it
    was allocated on, so the block is `stream`'s; the current stream, where the caller
    goes on with the tensor, is recorded with it."""
    import torch
    if stream is None:
        return torch.empty((T, d), dtype=torch.uint16, device=device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(int(stream.cuda_stream), device)
    current = torch.cuda.current_stream(device)
    with torch.cuda.stream(stream):
        out = torch.empty((T, d), dtype=torch.uint16, device=device)
    if current != stream:
        out.record_stream(current)
    return out


class NormCheckpoint:
    """What moe_forward_block_checkpoint leaves of its norm's input: E4M3 codes,
    E8M0 scales and the rows' inverse roots, for up to T tokens."""

    def __init__(self, T: int, d: int, device="cuda"):
        import torch
        self.q = torch.empty((T, d), dtype=torch.uint8, device=device)
        self.scales = torch.empty((T, d // 32), dtype=torch.uint8, device=device)
        self.rstd = torch.empty(T, dtype=torch.float32, device=device)

    def rows(self, T: int):
        return self.q[:T], self.scales[:T], self.rstd[:T]


class RouterGrads:
    """Gradients of a layer's router and norm (dW_r, db_r, dg), the auxiliary loss's
    values (stats: loss, balance, z, live tokens; counts; mean_probs), and the
    buffers and workspace that MoELayer.backward_block uses, for up to T tokens."""

    def __init__(self, E: int, k: int, T: int, d: int, device="cuda"):
        import torch
        f = lambda *s: torch.zeros(s, dtype=torch.float32, device=device)
        self.T = T
        self.dW_r, self.db_r, self.dg = f(E, d), f(E), f(d)
        self.stats, self.mean_probs = f(4), f(E)
        self.counts = torch.zeros(E, dtype=torch.int32, device=device)
        self.dlogits, self.lse = f(T, E), f(T)
        self.dx = torch.empty((T, d), dtype=torch.uint16, device=device)
        # the calls run one after another, so they share the largest one's workspace
        nbytes = max(moe_balance_loss_workspace_size(E, k, T),
                     moe_router_backward_workspace_size(E, T, d),
                     moe_rms_norm_backward_workspace_size(T, d))
        if nbytes == 0:
            raise ValueError("unsupported shape")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)


class MoELayer:
    """Device-resident MoE layer: weights uploaded once, workspace owned here."""

    def __init__(self, inp, device="cuda", T_max: Optional[int] = None, hostio: bool = False,
                 block: bool = False):
        import torch
        self.d, self.I, self.E, self.k = inp.d, inp.I, inp.E, inp.k
        to = lambda a: torch.from_numpy(a).to(device)
        self.W_r = to(inp.W_r)
        self.b_r = to(inp.b_r)
        self.Wgu_codes = to(inp.Wgu_codes)
        self.Wgu_scales = to(inp.Wgu_scales)
        self.Wd_codes = to(inp.Wd_codes)
        self.Wd_scales = to(inp.Wd_scales)
        self.T_max = T_max if T_max is not None else inp.T
        size_fn = (moe_workspace_size_hostio if hostio else
                   moe_workspace_size_block if block else moe_workspace_size)
        nbytes = size_fn(self.E, self.k, self.T_max, self.d, self.I)
        if nbytes == 0:
            raise ValueError("unsupported shape")
        self.workspace = torch.empty(nbytes, dtype=torch.uint8, device=device)

    def forward(self, x, out=None, stream=None):
        T = x.shape[0]
        if T > self.T_max:
            raise ValueError("more tokens than the workspace was sized for")
        if out is None:
            out = _result(T, self.d, x.device, stream)
        moe_forward(x, self.W_r, self.b_r, self.Wgu_codes, self.Wgu_scales, self.Wd_codes,
                    self.Wd_scales, self.E, self.k, T, self.d, self.I, out, self.workspace, stream)
        return out

    def forward_block(self, h, g, eps: float, out=None, checkpoint: Optional[NormCheckpoint] = None,
                      stream=None):
        """out = h + MoE(RMSNorm(h)) (a layer made with block=True); with a
        checkpoint, the training form, whose backward pass is backward_block."""
        T = h.shape[0]
        if T > self.T_max:
            raise ValueError("more tokens than the workspace was sized for")
        if out is None:
            out = _result(T, self.d, h.device, stream)
        args = (h, g, eps, self.W_r, self.b_r, self.Wgu_codes, self.Wgu_scales, self.Wd_codes,
                self.Wd_scales, self.E, self.k, T, self.d, self.I, out)
        if checkpoint is None:
            moe_forward_block(*args, self.workspace, stream)
        else:
            moe_forward_block_checkpoint(*args, *checkpoint.rows(T), self.workspace, stream)
        return out

    def backward_block(self, dout, g, checkpoint: NormCheckpoint, grads: RouterGrads,
                       balance_coef: float = 0.0, z_coef: float = 0.0, dloss=None, dx_in=None,
                       token_mask=None, accumulate: bool = False, dh=None, stream=None):
        """The backward pass of forward_block with a checkpoint, right after it (what
        it reads lies in the layer's workspace): fills grads from dout bf16 [T, d],
        the gradient of out, and returns dh bf16 [T, d]. The auxiliary loss
        balance_coef * balance + z_coef * z is weighted by dloss (f32 [1]; None: 1).
        dW_r and db_r are complete. The experts are frozen, and their share of the
        gradient that reaches RMSNorm(h) is not computed here: dh and grads.dg are the
        sublayer's only if the caller passes it as dx_in bf16 [T, d]; without it they
        hold the residual's gradient (dh) and the path through the logits."""
        T = dout.shape[0]
        if T > grads.T:
            raise ValueError("more tokens than the gradients' buffers were sized for")
        if dh is None:
            dh = _result(T, self.d, dout.device, stream)
        E, k, d, mask = self.E, self.k, self.d, token_mask
        logits, idx = self.intermediate("logits", T), self.intermediate("topk_idx", T)
        dlogits, dx, ws = grads.dlogits[:T], grads.dx[:T], grads.workspace
        q, scales, rstd = checkpoint.rows(T)
        moe_gate_backward(dout, self.intermediate("yw", T), idx, self.intermediate("topk_w", T), E, k,
                          T, d, dlogits, token_mask=mask, stream=stream)
        moe_balance_loss(logits, idx, E, k, T, balance_coef, z_coef, grads.stats, grads.counts,
                         grads.mean_probs, grads.lse[:T], ws, token_mask=mask, stream=stream)
        if balance_coef or z_coef:
            moe_balance_loss_backward(logits, grads.lse[:T], grads.counts, grads.stats, E, k, T,
                                      balance_coef, z_coef, dlogits, dloss=dloss, token_mask=mask,
                                      accumulate=True, stream=stream)
        moe_router_backward(dlogits, self.W_r, E, T, d, grads.dW_r, grads.db_r, dx, ws, q=q,
                            scales=scales, rstd=rstd, g=g, dx_in=dx_in, token_mask=mask,
                            accumulate=accumulate, stream=stream)
        moe_rms_norm_backward(dx, g, rstd, T, d, dh, grads.dg, ws, q=q, scales=scales, dh_in=dout,
                              token_mask=mask, accumulate=accumulate, stream=stream)
        return dh

    def forward_timed(self, x, out, stream=None):
        T = x.shape[0]
        return moe_forward_timed(x, self.W_r, self.b_r, self.Wgu_codes, self.Wgu_scales,
                                 self.Wd_codes, self.Wd_scales, self.E, self.k, T, self.d,
                                 self.I, out, self.workspace, stream)

    def forward_timed_events(self, x, out, event_mask: int, stream=None, tile_policy=None,
                             act_quant=None):
        """moe_forward_timed_events; with tile_policy or act_quant given, the
        per-call options form (moe_forward_timed_ex)."""
        T = x.shape[0]
        if tile_policy is None and act_quant is None:
            return moe_forward_timed_events(x, self.W_r, self.b_r, self.Wgu_codes,
                                            self.Wgu_scales, self.Wd_codes, self.Wd_scales,
                                            self.E, self.k, T, self.d, self.I, out,
                                            self.workspace, event_mask, stream)
        if isinstance(act_quant, str):
            act_quant = ACT_MODES[act_quant]
        o = ForwardOpts(-1 if tile_policy is None else tile_policy,
                        ACT_BF16 if act_quant is None else act_quant, None, None)
        ms = (ctypes.c_float * (len(STAGES) + 1))()
        _check("moe_forward_timed_ex", load().moe_forward_timed_ex(
            _ptr(x), _ptr(self.W_r), _ptr(self.b_r), _ptr(self.Wgu_codes), _ptr(self.Wgu_scales),
            _ptr(self.Wd_codes), _ptr(self.Wd_scales), self.E, self.k, T, self.d, self.I, _ptr(out),
            _ptr(self.workspace), self.workspace.numel(), ctypes.byref(o), _stream(stream),
            event_mask, ms))
        return list(ms)

    def forward_hostio(self, x_host, out_host, stream=None):
        T = x_host.shape[0]
        moe_forward_hostio(x_host, self.W_r, self.b_r, self.Wgu_codes, self.Wgu_scales,
                           self.Wd_codes, self.Wd_scales, self.E, self.k, T, self.d, self.I,
                           out_host, self.workspace, stream)
        return out_host

    def layout(self, T: int) -> dict:
        return moe_workspace_layout(self.E, self.k, T, self.d, self.I)

    def intermediate(self, name: str, T: int):
        """View of an intermediate buffer inside the workspace after a forward."""
        import torch
        L = self.layout(T)
        P = T * self.k
        spec = {
            "logits": (torch.float32, (T, self.E)), "topk_idx": (torch.int32, (T, self.k)),
            "topk_w": (torch.float32, (T, self.k)), "counts": (torch.int32, (self.E,)),
            "offsets": (torch.int32, (self.E + 1,)), "perm": (torch.int32, (P,)),
            "xp": (torch.uint16, (P, self.d)), "h": (torch.uint16, (P, self.I)),
            "yw": (torch.float32, (P, self.d)),
        }[name]
        dt, shape = spec
        n = 1
        for s in shape:
            n *= s
        nbytes = n * torch.empty((), dtype=dt).element_size()
        raw = self.workspace[L[name]:L[name] + nbytes]
        return raw.view(dt).view(shape)
