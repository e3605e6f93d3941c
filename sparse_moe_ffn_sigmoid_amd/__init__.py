"""Python binding of the MI355X Stable LatentMoE library (``libmoe_mi355x.so``).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, their device pointers and the current HIP stream are passed to
the C ABI declared in ``include/moe_mi355x.h``, and every step of the layer
runs in the library's HIP kernels.  There is no fallback: if the library is
missing or fails to load, importing this package raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_mi355x.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python sparse_moe_ffn_sigmoid_amd/build.py`")
_lib = ctypes.CDLL(LIB_PATH)

MOE_F32, MOE_BF16, MOE_MXFP4, MOE_MXFP4_A8, MOE_MXFP4_A4 = 0, 1, 2, 3, 4
MOE_F16 = 5
MOE_QB_FROZEN, MOE_QB_BATCH = 0, 1
EXPORTED = ("moe_route_workspace_bytes", "moe_route_qb", "moe_route_sign",
            "moe_forward_workspace_bytes",
            "moe_latent_forward", "moe_status_str", "moe_stage_timing", "moe_stage_times",
            "moe_stage_name", "moe_mxfp8_quantize", "moe_mxfp4_quantize",
            "moe_route_qb_noalloc", "moe_backward_workspace_bytes", "moe_latent_backward",
            "moe_sgd_step", "moe_latent_backward_sgd", "moe_saved_activations_bytes",
            "moe_latent_forward_train", "moe_latent_backward_train",
            "moe_balance_loss_workspace_bytes", "moe_balance_loss", "moe_balance_loss_backward",
            "moe_router_backward_workspace_bytes", "moe_router_backward",
            "moe_mxfp4_padded_rows", "moe_mxfp4_pack", "moe_mxfp4_unpack", "moe_mxfp4_matmul",
            "moe_mxfp4_matmul_kgroup", "moe_mxfp4_linear_workspace_bytes", "moe_mxfp4_linear")


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("d", ctypes.c_int32), ("latent", ctypes.c_int32),
                ("n_experts", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("inter", ctypes.c_int32), ("shared_inter", ctypes.c_int32),
                ("act_dtype", ctypes.c_int32), ("routed_dtype", ctypes.c_int32),
                ("rms_eps", ctypes.c_float), ("qb_mode", ctypes.c_int32),
                ("qb_max_rounds", ctypes.c_int32)]


class MoeWeights(ctypes.Structure):
    _fields_ = [(name, ctypes.c_void_p) for name in (
        "w_router", "router_logit_offset", "w_down", "w_up", "w_gate", "w_uproj", "w_dn",
        "s_gate", "s_uproj", "s_dn", "rms_gamma", "ws_gate", "ws_up", "ws_down")]


_vp, _i32, _sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
class MoeGrads(ctypes.Structure):
    _fields_ = [(f, ctypes.c_void_p) for f in (
        "dx", "d_w_router", "d_router_logit_offset", "d_w_down", "d_w_up", "d_w_gate",
        "d_w_uproj", "d_w_dn", "d_rms_gamma", "d_ws_gate", "d_ws_up", "d_ws_down")]


_lib.moe_route_workspace_bytes.argtypes = [_i32, _i32, _i32]
_lib.moe_route_workspace_bytes.restype = _sz
_lib.moe_route_qb.argtypes = [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp,
                              _sz, _vp]
_lib.moe_route_qb.restype = ctypes.c_int
_lib.moe_route_sign.argtypes = [_vp, _i32, _i32, _i32, ctypes.c_double, _i32, _vp, _vp, _vp, _vp,
                                _vp, _vp, _sz, _vp]
_lib.moe_route_sign.restype = ctypes.c_int
_lib.moe_forward_workspace_bytes.argtypes = [ctypes.POINTER(MoeShape)]
_lib.moe_forward_workspace_bytes.restype = _sz
_lib.moe_latent_forward.argtypes = [ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeights), _vp,
                                    _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.moe_latent_forward.restype = ctypes.c_int
_lib.moe_status_str.argtypes = [ctypes.c_int]
_lib.moe_status_str.restype = ctypes.c_char_p
_lib.moe_stage_timing.argtypes = [ctypes.c_int]
_lib.moe_stage_timing.restype = ctypes.c_int
_lib.moe_stage_times.argtypes = [_vp, _vp, _i32]
_lib.moe_stage_times.restype = ctypes.c_int
_lib.moe_stage_name.argtypes = [ctypes.c_int]
_lib.moe_stage_name.restype = ctypes.c_char_p
_lib.moe_route_qb_noalloc.argtypes = [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp,
                                      _vp]
_lib.moe_route_qb_noalloc.restype = ctypes.c_int
_lib.moe_backward_workspace_bytes.argtypes = [ctypes.POINTER(MoeShape)]
_lib.moe_backward_workspace_bytes.restype = _sz
_lib.moe_latent_backward.argtypes = [ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeights), _vp, _vp,
                                     _vp, _vp, _vp, ctypes.POINTER(MoeGrads), _vp, _sz, _vp]
_lib.moe_latent_backward.restype = ctypes.c_int
_lib.moe_sgd_step.argtypes = [ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeights),
                              ctypes.POINTER(MoeGrads), ctypes.c_float, _vp]
_lib.moe_sgd_step.restype = ctypes.c_int
_lib.moe_latent_backward_sgd.argtypes = [ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeights), _vp,
                                         _vp, _vp, _vp, _vp, ctypes.POINTER(MoeGrads),
                                         ctypes.c_float, _vp, _sz, _vp]
_lib.moe_latent_backward_sgd.restype = ctypes.c_int
_lib.moe_saved_activations_bytes.argtypes = [ctypes.POINTER(MoeShape)]
_lib.moe_saved_activations_bytes.restype = _sz
_lib.moe_latent_forward_train.argtypes = [ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeights),
                                          _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                          _vp, _sz, _vp]
_lib.moe_latent_forward_train.restype = ctypes.c_int
_lib.moe_latent_backward_train.argtypes = [ctypes.POINTER(MoeShape), ctypes.POINTER(MoeWeights),
                                           _vp, _vp, _vp, _vp, _vp, _vp, _sz,
                                           ctypes.POINTER(MoeGrads), ctypes.c_int, ctypes.c_float,
                                           _vp, _sz, _vp]
_lib.moe_latent_backward_train.restype = ctypes.c_int
_lib.moe_mxfp4_quantize.argtypes = [_vp, ctypes.c_int64, ctypes.c_int64, _vp, _vp, _vp]
_lib.moe_mxfp4_quantize.restype = ctypes.c_int
_lib.moe_mxfp8_quantize.argtypes = [_vp, ctypes.c_int64, ctypes.c_int64, _vp, _vp, _vp]
_lib.moe_mxfp8_quantize.restype = ctypes.c_int
_i64 = ctypes.c_int64
for _name, _res, _args in (
        ("moe_balance_loss_workspace_bytes", _sz, [_i32, _i32]),
        ("moe_balance_loss", ctypes.c_int, [_vp, _i64, _i32, _i32, _i32, _vp, _vp, _i32, _vp, _vp,
                                            _vp, _vp, _vp, _vp, _vp, _sz, _vp]),
        ("moe_balance_loss_backward", ctypes.c_int, [_vp, _i64, _i32, _i32, _i32, _vp, _vp, _vp,
                                                     _i32, _vp, _vp, _vp, _vp]),
        ("moe_router_backward_workspace_bytes", _sz, [_i32, _i32, _i32]),
        ("moe_router_backward", ctypes.c_int, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, ctypes.c_int,
                                               _vp, _vp, _vp, _vp, _sz, _vp]),
        ("moe_mxfp4_padded_rows", _i64, [_i64, _i32]),
        ("moe_mxfp4_pack", ctypes.c_int, [_vp, _i32, _i64, _i64, _i64, _i64, _i64, _vp, _vp, _vp,
                                          _vp, _vp, _i32, _vp, _vp]),
        ("moe_mxfp4_unpack", ctypes.c_int, [_vp, _vp, _i64, _i64, _i32, _vp, _i64, _vp]),
        ("moe_mxfp4_matmul", ctypes.c_int, [_vp, _vp, _i64, _vp, _vp, _i64, _i64, _i64, _vp, _i32,
                                            _vp, _vp, _i32, _i64, _vp]),
        ("moe_mxfp4_matmul_kgroup", ctypes.c_int, [_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _i32,
                                                   _vp, _i32, _vp]),
        ("moe_mxfp4_linear_workspace_bytes", _sz, [_i64, _i64]),
        ("moe_mxfp4_linear", ctypes.c_int, [_vp, _i32, _i64, _i64, _vp, _vp, _i64, _i64, _i64, _vp,
                                            _i32, _vp, _vp, _i32, _i64, _vp, _sz, _vp])):
    getattr(_lib, _name).argtypes = _args
    getattr(_lib, _name).restype = _res


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {_lib.moe_status_str(status).decode()} ({status})")
        self.status = status


def lib() -> ctypes.CDLL:
    return _lib


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(t, name, dtype, shape, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def route_workspace_bytes(T: int, n: int, k: int) -> int:
    return int(_lib.moe_route_workspace_bytes(T, n, k))


def route_qb(scores: torch.Tensor, k: int, bias: torch.Tensor | None = None,
             mode: int = MOE_QB_BATCH, max_rounds: int = 64, workspace=None):
    """Route fp32 scores [T, n] (device) to k experts per token.

    Returns dict(idx [T,k] int32, w [T,k] fp32, loads [n] int32, bias [n] fp64,
    info [4] int32) -- info = (quantile rounds, status, max |load-target|,
    augmenting-path moves).  ``bias`` (fp64 [n]) is the start / frozen bias.
    """
    dev = scores.device
    T, n = scores.shape
    _check(scores, "scores", torch.float32, (T, n), dev)
    b = torch.zeros(n, dtype=torch.float64, device=dev) if bias is None else bias.clone()
    _check(b, "bias", torch.float64, (n,), dev)
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    loads = torch.empty(n, dtype=torch.int32, device=dev)
    info = torch.zeros(4, dtype=torch.int32, device=dev)
    need = route_workspace_bytes(T, n, k)
    ws = workspace if workspace is not None else torch.empty(max(need, 256), dtype=torch.uint8,
                                                             device=dev)
    st = _lib.moe_route_qb(_ptr(scores), T, n, k, mode, max_rounds, _ptr(b), _ptr(idx), _ptr(w),
                           _ptr(loads), _ptr(info), _ptr(ws), ws.numel(), _stream())
    if st != 0:
        raise MoeError(st, "moe_route_qb")
    return dict(idx=idx, w=w, loads=loads, bias=b, info=info)


def route_qb_noalloc(scores: torch.Tensor, k: int, bias: torch.Tensor | None = None,
                     mode: int = MOE_QB_BATCH, max_rounds: int = 64):
    """:func:`route_qb` through moe_route_qb_noalloc: the library's own
    per-device scratch array instead of a workspace (outputs are still
    allocated here, by torch)."""
    dev = scores.device
    T, n = scores.shape
    _check(scores, "scores", torch.float32, (T, n), dev)
    b = torch.zeros(n, dtype=torch.float64, device=dev) if bias is None else bias.clone()
    _check(b, "bias", torch.float64, (n,), dev)
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    loads = torch.empty(n, dtype=torch.int32, device=dev)
    info = torch.zeros(4, dtype=torch.int32, device=dev)
    st = _lib.moe_route_qb_noalloc(_ptr(scores), T, n, k, mode, max_rounds, _ptr(b), _ptr(idx),
                                   _ptr(w), _ptr(loads), _ptr(info), _stream())
    if st != 0:
        raise MoeError(st, "moe_route_qb_noalloc")
    return dict(idx=idx, w=w, loads=loads, bias=b, info=info)


def route_sign(scores: torch.Tensor, k: int, step: float, max_rounds: int,
               bias: torch.Tensor | None = None, workspace=None):
    """DeepSeek-V3's fixed-step sign update of the bias on fp32 scores [T, n]
    (device), the baseline for Quantile Balancing.  Returns the dict of
    :func:`route_qb` with info = (updates, status, max |load-target|, 0)."""
    dev = scores.device
    T, n = scores.shape
    _check(scores, "scores", torch.float32, (T, n), dev)
    b = torch.zeros(n, dtype=torch.float64, device=dev) if bias is None else bias.clone()
    _check(b, "bias", torch.float64, (n,), dev)
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    loads = torch.empty(n, dtype=torch.int32, device=dev)
    info = torch.zeros(4, dtype=torch.int32, device=dev)
    need = route_workspace_bytes(T, n, k)
    ws = workspace if workspace is not None else torch.empty(max(need, 256), dtype=torch.uint8,
                                                             device=dev)
    st = _lib.moe_route_sign(_ptr(scores), T, n, k, float(step), max_rounds, _ptr(b), _ptr(idx),
                             _ptr(w), _ptr(loads), _ptr(info), _ptr(ws), ws.numel(), _stream())
    if st != 0:
        raise MoeError(st, "moe_route_sign")
    return dict(idx=idx, w=w, loads=loads, bias=b, info=info)


def mxfp8_quantize(x: torch.Tensor):
    """bf16 rows [rows, K] (device, K a multiple of 32) -> (E4M3 codes uint8
    [rows, K], E8M0 scales uint8 [rows, K/32]), one scale per 32 elements."""
    rows, K = x.shape
    _check(x, "x", torch.bfloat16, (rows, K), x.device)
    codes = torch.empty((rows, K), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, K // 32), dtype=torch.uint8, device=x.device)
    st = _lib.moe_mxfp8_quantize(_ptr(x), rows, K, _ptr(codes), _ptr(scales), _stream())
    if st != 0:
        raise MoeError(st, "moe_mxfp8_quantize")
    return codes, scales


def mxfp4_quantize(x: torch.Tensor):
    """bf16 rows [rows, K] (device, K a multiple of 32) -> (E2M1 codes uint8
    [rows, K/2], two per byte, element 2i in the low nibble; E8M0 scales uint8
    [rows, K/32])."""
    rows, K = x.shape
    _check(x, "x", torch.bfloat16, (rows, K), x.device)
    codes = torch.empty((rows, K // 2), dtype=torch.uint8, device=x.device)
    scales = torch.empty((rows, K // 32), dtype=torch.uint8, device=x.device)
    st = _lib.moe_mxfp4_quantize(_ptr(x), rows, K, _ptr(codes), _ptr(scales), _stream())
    if st != 0:
        raise MoeError(st, "moe_mxfp4_quantize")
    return codes, scales


# --------------------------------------------------------------------------
# Balance loss and the dense gradient of the router's scores
# --------------------------------------------------------------------------
def _device_of(t, name):
    """The GPU that a call runs on: that of its first tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be on a GPU, got {t.device}")
    return t.device


def _addr(t):
    return None if t is None else t.data_ptr()


def _status(fn, dev, *args):
    """fn(*args, stream) on the device's current stream."""
    stream = torch._C._cuda_getCurrentRawStream(dev.index)
    if dev.index == torch.cuda.current_device():
        return fn(*args, stream)
    with torch.cuda.device(dev):
        return fn(*args, stream)


def _call(fn, dev, *args):
    """As _status; raises MoeError."""
    st = _status(fn, dev, *args)
    if st != 0:
        raise MoeError(st, fn.__name__)


def _call_scratch(fn, dev, few, need, workspace, *args):
    """fn(*args, workspace, its bytes, stream).  Calls with few tokens may need
    no workspace: they are made without one first, and the library asks for it
    with MOE_EWORKSPACE before it launches anything.  need: (query, arguments)."""
    if workspace is None and few:
        st = _status(fn, dev, *args, None, 0)
        if st == 0:
            return
        if st != -3:
            raise MoeError(st, fn.__name__)
    if workspace is None:
        workspace = torch.empty(max(need[0](*need[1:]), 256), dtype=torch.uint8, device=dev)
    else:
        _check(workspace, "workspace", torch.uint8, (workspace.numel(),), dev)
    _call(fn, dev, *args, _addr(workspace), workspace.numel())


def _score_rows(scores, name="scores"):
    """Device, T, n and row stride of fp32 scores [T, n] with unit column stride."""
    dev = _device_of(scores, name)
    if scores.dim() != 2 or scores.dtype != torch.float32:
        raise ValueError(f"{name} must be fp32 [T, n], got {scores.dtype} {tuple(scores.shape)}")
    T, n = scores.shape
    if n > 1 and scores.stride(1) != 1 or T > 1 and scores.stride(0) < n:
        raise ValueError(f"{name} must have unit column stride and rows that do not overlap")
    return dev, T, n, (scores.stride(0) if T > 1 else n)


def _sequences(seq_offsets, token_mask, dloss, T, dev):
    """(number of sequences, mask as uint8), the arguments checked."""
    S = 1
    if seq_offsets is not None:
        S = seq_offsets.numel() - 1
        _check(seq_offsets, "seq_offsets", torch.int32, (S + 1,), dev)
    if token_mask is not None:
        if token_mask.dtype == torch.bool:
            token_mask = token_mask.view(torch.uint8)
        _check(token_mask, "token_mask", torch.uint8, (T,), dev)
    if dloss is not None:
        _check(dloss, "dloss", torch.float32, (S,), dev)
    return S, token_mask


def balance_loss(scores: torch.Tensor, idx: torch.Tensor, seq_offsets=None, token_mask=None,
                 dloss=None, want_grad: bool = False, workspace=None):
    """Balance loss of the routing idx [T, k] (int32; an index outside [0, n),
    such as -1, is not counted) per sequence, with per-expert counts.

    ``scores`` fp32 [T, n] >= 0 (rows may be strided); ``seq_offsets`` int32
    [S + 1] (device) or None for one sequence; ``token_mask`` bool or uint8
    [T], false for padding.  Over the N counted tokens of a sequence
    loss = n / (k N^2) sum_i c_i sum_t s_ti / sum_j s_tj, 1 for even counts.
    Returns dict(loss [S] fp32, counts [S, n] int32, tokens [S] int32), and
    with ``want_grad`` dscores [T, n] fp32, the gradient of sum(loss * dloss)
    (``dloss`` fp32 [S], None for ones) with the choices held fixed, from the
    same pass over the scores.
    """
    dev, T, n, ld = _score_rows(scores)
    if not isinstance(idx, torch.Tensor) or idx.dim() != 2:
        raise ValueError("idx must be a tensor [T, k]")
    k = idx.shape[1]
    _check(idx, "idx", torch.int32, (T, k), dev)
    S, mask = _sequences(seq_offsets, token_mask, dloss, T, dev)
    out = dict(loss=torch.empty(S, dtype=torch.float32, device=dev),
               counts=torch.empty((S, n), dtype=torch.int32, device=dev),
               tokens=torch.empty(S, dtype=torch.int32, device=dev))
    if want_grad:
        out["dscores"] = torch.empty((T, n), dtype=torch.float32, device=dev)
    _call_scratch(_lib.moe_balance_loss, dev, T <= 256,
                  (_lib.moe_balance_loss_workspace_bytes, T, S), workspace, _addr(scores), ld, T,
                  n, k, _addr(idx), _addr(seq_offsets), S, _addr(mask), _addr(dloss),
                  _addr(out["loss"]), _addr(out["counts"]), _addr(out["tokens"]),
                  _addr(out.get("dscores")))
    return out


def balance_loss_backward(scores: torch.Tensor, counts: torch.Tensor, tokens: torch.Tensor, k: int,
                          seq_offsets=None, token_mask=None, dloss=None):
    """dscores [T, n] of :func:`balance_loss` from the counts and tokens it
    returned; the other arguments as it took them."""
    dev, T, n, ld = _score_rows(scores)
    S, mask = _sequences(seq_offsets, token_mask, dloss, T, dev)
    _check(counts, "counts", torch.int32, (S, n), dev)
    _check(tokens, "tokens", torch.int32, (S,), dev)
    dscores = torch.empty((T, n), dtype=torch.float32, device=dev)
    _call(_lib.moe_balance_loss_backward, dev, _addr(scores), ld, T, n, k, _addr(counts),
          _addr(tokens), _addr(seq_offsets), S, _addr(mask), _addr(dloss), _addr(dscores))
    return dscores


def router_backward(x: torch.Tensor, w_router: torch.Tensor, scores: torch.Tensor,
                    dscores: torch.Tensor, into: dict | None = None, workspace=None):
    """A gradient of all router scores (such as the balance loss's dscores)
    taken to x [T, d] bf16, w_router [n, d] fp32 and the logit offset, for
    scores = sigmoid(x w_router^T + offset) [T, n] fp32.

    Returns dict(dx bf16, d_w_router fp32, d_router_logit_offset fp32).  With
    ``into`` (a dict of :func:`latent_backward`) the gradients are added to
    the tensors it holds under those names (entries that are None are left
    out) and it is returned.
    """
    dev = _device_of(x, "x")
    T, d = x.shape
    n = w_router.shape[0]
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(w_router, "w_router", torch.float32, (n, d), dev)
    _check(scores, "scores", torch.float32, (T, n), dev)
    _check(dscores, "dscores", torch.float32, (T, n), dev)
    names = dict(dx=(torch.bfloat16, (T, d)), d_w_router=(torch.float32, (n, d)),
                 d_router_logit_offset=(torch.float32, (n,)))
    out = into
    if into is None:
        out = {f: torch.empty(shape, dtype=dt, device=dev) for f, (dt, shape) in names.items()}
    else:
        for f, (dt, shape) in names.items():
            if into.get(f) is not None:
                _check(into[f], f, dt, shape, dev)
    _call_scratch(_lib.moe_router_backward, dev, T <= 1024,
                  (_lib.moe_router_backward_workspace_bytes, T, d, n), workspace, _addr(x),
                  _addr(w_router), _addr(scores), _addr(dscores), T, d, n,
                  0 if into is None else 1, *[_addr(out.get(f)) for f in names])
    return out


# --------------------------------------------------------------------------
# MXFP4 packing and products
# --------------------------------------------------------------------------
_MX_TYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16, torch.float16: MOE_F16}


def _mx_type(dtype, name):
    if dtype not in _MX_TYPES:
        raise ValueError(f"{name} must be fp32, bf16 or fp16, got {dtype}")
    return _MX_TYPES[dtype]


def _mx_operand(codes, scales, name, dim, dev):
    """Shape [.., rows, K] of packed codes [.., rows, K/2] and their scales."""
    if not isinstance(codes, torch.Tensor) or codes.dim() != dim:
        raise ValueError(f"{name}codes must be a tensor of {dim} dimensions")
    shape = tuple(codes.shape)
    if shape[-1] == 0 or shape[-1] % 16:
        raise ValueError(f"{name}codes must hold whole blocks of 32 elements (16 bytes)")
    _check(codes, f"{name}codes", torch.uint8, shape, dev)
    _check(scales, f"{name}scales", torch.uint8, shape[:-1] + (shape[-1] // 16,), dev)
    return shape[:-1] + (2 * shape[-1],)


def mxfp4_pack(x: torch.Tensor, rows: bool = True, cols: bool = False, offsets=None):
    """MXFP4 rounding of x [rows, K] or [batch, rows, K] (fp32, bf16 or fp16,
    unit column stride) along rows and/or columns, from one read.

    Returns a dict: with ``rows`` codes uint8 [.., rows, 16 ceil(K/32)] and
    scales uint8 [.., rows, ceil(K/32)]; with ``cols`` codes_t uint8 [.., K,
    16 R] and scales_t uint8 [.., K, R], R = ceil(rows/32).  Tails are filled
    up with zeros.  With ``offsets`` int32 [G + 1] (2-D x, ``cols``) no block
    of a column crosses from one row group to the next, each group starts at a
    multiple of 32 padded rows, offsets_t int32 [G + 1], and R covers
    rows + 31 G; rows outside every group are not touched.  A block with an
    infinity or NaN becomes NaN.
    """
    dev = _device_of(x, "x")
    if x.dim() not in (2, 3):
        raise ValueError(f"x must be [rows, K] or [batch, rows, K], got {tuple(x.shape)}")
    dt = _mx_type(x.dtype, "x")
    B = x.shape[0] if x.dim() == 3 else 1
    R, K = x.shape[-2:]
    rs = x.stride(-2) if R > 1 else max(K, 1)
    bs = x.stride(0) if x.dim() == 3 and B > 1 else R * rs
    if K < 1 or (K > 1 and x.stride(-1) != 1) or rs < K:
        raise ValueError("x must have at least one column, unit column stride and rows that do "
                         "not overlap")
    if not rows and not cols:
        raise ValueError("mxfp4_pack: neither rows nor cols asked for")
    G = 0
    if offsets is not None:
        if not cols or x.dim() != 2:
            raise ValueError("offsets need a matrix and cols=True")
        G = offsets.numel() - 1
        _check(offsets, "offsets", torch.int32, (G + 1,), dev)
    lead = tuple(x.shape[:-2])
    cb = (K + 31) // 32
    out = {}
    if rows:
        out["codes"] = torch.empty(lead + (R, cb * 16), dtype=torch.uint8, device=dev)
        out["scales"] = torch.empty(lead + (R, cb), dtype=torch.uint8, device=dev)
    if cols:
        padded = _lib.moe_mxfp4_padded_rows(R, G)
        if padded < 0:
            raise MoeError(-2, "moe_mxfp4_padded_rows")
        out["codes_t"] = torch.empty(lead + (K, padded // 2), dtype=torch.uint8, device=dev)
        out["scales_t"] = torch.empty(lead + (K, padded // 32), dtype=torch.uint8, device=dev)
    if offsets is not None:
        out["offsets_t"] = torch.empty(G + 1, dtype=torch.int32, device=dev)
    _call(_lib.moe_mxfp4_pack, dev, _addr(x), dt, B, R, K, rs, bs,
          *[_addr(out.get(f)) for f in ("codes", "scales", "codes_t", "scales_t")], _addr(offsets),
          G, _addr(out.get("offsets_t")))
    return out


def mxfp4_unpack(codes: torch.Tensor, scales: torch.Tensor, K: int, dtype=torch.bfloat16):
    """Values [.., rows, K] of packed rows (codes [.., rows, 16 ceil(K/32)]);
    bf16 and fp32 hold them exactly, fp16 rounds them."""
    dev = _device_of(codes, "codes")
    dt = _mx_type(dtype, "dtype")
    shape = _mx_operand(codes, scales, "", codes.dim(), dev)
    if len(shape) < 2 or not shape[-1] - 32 < K <= shape[-1]:
        raise ValueError(f"K = {K} does not fit codes of {shape[-1]} elements")
    out = torch.empty(shape[:-1] + (K,), dtype=dtype, device=dev)
    _call(_lib.moe_mxfp4_unpack, dev, _addr(codes), _addr(scales), out.numel() // K, K, dt,
          _addr(out), K)
    return out


def _groups(offsets, b_dim, dev):
    if offsets is None:
        if b_dim != 2:
            raise ValueError("a matrix per group needs offsets")
        return 1
    _check(offsets, "offsets", torch.int32, (offsets.numel(),), dev)
    return offsets.numel() - 1


def _mx_out(out, M, N, dtype, dev):
    """The output [M, N] and its row stride: given (rows may be strided) or new."""
    if out is None:
        return torch.empty((M, N), dtype=dtype, device=dev), N
    if out.device != dev or out.dtype != dtype or tuple(out.shape) != (M, N):
        raise ValueError(f"out must be {dtype} {(M, N)} on {dev}")
    if (N > 1 and out.stride(1) != 1) or (M > 1 and out.stride(0) < N):
        raise ValueError("out must have unit column stride and rows that do not overlap")
    return out, out.stride(0) if M > 1 else N


def mxfp4_matmul(a_codes, a_scales, b_codes, b_scales, offsets=None, rows=None,
                 out_dtype=torch.bfloat16, out=None):
    """C [M, N] = A B^T of MXFP4 operands A [R, K] and B [N, K], packed along K.

    With ``offsets`` int32 [G + 1] (device) and B [G, N, K] rows [offsets[g],
    offsets[g + 1]) of C meet B[g]; rows outside every group stay as they were
    (undefined unless ``out`` is given).  ``rows`` int32 [M] (device): row r of
    C is made from row rows[r] of A, M = R without it.
    """
    dev = _device_of(a_codes, "a_codes")
    R, K = _mx_operand(a_codes, a_scales, "a_", 2, dev)
    G = _groups(offsets, b_codes.dim(), dev)
    b = _mx_operand(b_codes, b_scales, "b_", 2 if offsets is None else 3, dev)
    if b[-1] != K or (offsets is not None and b[0] != G):
        raise ValueError(f"b is {b}: K = {K} and {G} groups are wanted")
    M, N = R, b[-2]
    if rows is not None:
        M = rows.numel()
        _check(rows, "rows", torch.int32, (M,), dev)
    dt = _mx_type(out_dtype, "out_dtype")
    out, ldo = _mx_out(out, M, N, out_dtype, dev)
    _call(_lib.moe_mxfp4_matmul, dev, _addr(a_codes), _addr(a_scales), R, _addr(b_codes),
          _addr(b_scales), M, N, K, _addr(offsets), G, _addr(rows), _addr(out), dt, ldo)
    return out


def mxfp4_matmul_kgroup(a_codes, a_scales, b_codes, b_scales, offsets=None,
                        out_dtype=torch.float32):
    """Products over ranges of the contraction, the weight gradients of a
    linear layer or of experts: out[g] = A[:, range g] B[:, range g]^T of
    A [M, K] and B [N, K] (codes_t and scales_t of :func:`mxfp4_pack`), ranges
    from ``offsets`` (its offsets_t).  Returns [G, M, N], or [M, N] over all of
    K without ``offsets``."""
    dev = _device_of(a_codes, "a_codes")
    M, K = _mx_operand(a_codes, a_scales, "a_", 2, dev)
    N, Kb = _mx_operand(b_codes, b_scales, "b_", 2, dev)
    if Kb != K:
        raise ValueError(f"the operands' K differ: {K} and {Kb}")
    dt = _mx_type(out_dtype, "out_dtype")
    G = 1
    if offsets is not None:
        G = offsets.numel() - 1
        _check(offsets, "offsets", torch.int32, (G + 1,), dev)
    out = torch.empty(((G,) if offsets is not None else ()) + (M, N), dtype=out_dtype, device=dev)
    _call(_lib.moe_mxfp4_matmul_kgroup, dev, _addr(a_codes), _addr(a_scales), _addr(b_codes),
          _addr(b_scales), M, N, K, _addr(offsets), G, _addr(out), dt)
    return out


def mxfp4_linear(x: torch.Tensor, w_codes: torch.Tensor, w_scales: torch.Tensor, offsets=None,
                 rows=None, out_dtype=None, out=None, workspace=None):
    """:func:`mxfp4_matmul` of activations x [R, K] (fp32, bf16 or fp16, K a
    multiple of 32) that are packed on the way, against packed weights [N, K],
    or [G, N, K] with ``offsets``.  ``out_dtype`` defaults to x's."""
    dev = _device_of(x, "x")
    if x.dim() != 2:
        raise ValueError(f"x must be [R, K], got {tuple(x.shape)}")
    xt = _mx_type(x.dtype, "x")
    R, K = x.shape
    rs = x.stride(0) if R > 1 else K
    if x.stride(1) != 1 and K > 1 or rs < K:
        raise ValueError("x must have unit column stride and rows that do not overlap")
    G = _groups(offsets, w_codes.dim(), dev)
    w = _mx_operand(w_codes, w_scales, "w_", 2 if offsets is None else 3, dev)
    if w[-1] != K or (offsets is not None and w[0] != G):
        raise ValueError(f"the weights are {w}: K = {K} and {G} groups are wanted")
    M, N = R, w[-2]
    if rows is not None:
        M = rows.numel()
        _check(rows, "rows", torch.int32, (M,), dev)
    out_dtype = x.dtype if out_dtype is None else out_dtype
    dt = _mx_type(out_dtype, "out_dtype")
    out, ldo = _mx_out(out, M, N, out_dtype, dev)
    _call_scratch(_lib.moe_mxfp4_linear, dev, M <= 16,
                  (_lib.moe_mxfp4_linear_workspace_bytes, R, K), workspace, _addr(x), xt, R, rs,
                  _addr(w_codes), _addr(w_scales), M, N, K, _addr(offsets), G, _addr(rows),
                  _addr(out), dt, ldo)
    return out


GRAD_SHAPES = {  # gradient name -> (weight key, shape from (T, d, L, n, k, m, ms))
    "d_w_router": ("w_router", lambda T, d, L, n, k, m, ms: (n, d)),
    "d_router_logit_offset": ("router_logit_offset", lambda T, d, L, n, k, m, ms: (n,)),
    "d_w_down": ("w_down", lambda T, d, L, n, k, m, ms: (L, d)),
    "d_w_up": ("w_up", lambda T, d, L, n, k, m, ms: (d, L)),
    "d_w_gate": ("w_gate", lambda T, d, L, n, k, m, ms: (n, m, L)),
    "d_w_uproj": ("w_uproj", lambda T, d, L, n, k, m, ms: (n, m, L)),
    "d_w_dn": ("w_dn", lambda T, d, L, n, k, m, ms: (n, L, m)),
    "d_rms_gamma": ("rms_gamma", lambda T, d, L, n, k, m, ms: (L,)),
    "d_ws_gate": ("ws_gate", lambda T, d, L, n, k, m, ms: (ms, d)),
    "d_ws_up": ("ws_up", lambda T, d, L, n, k, m, ms: (ms, d)),
    "d_ws_down": ("ws_down", lambda T, d, L, n, k, m, ms: (d, ms)),
}


def latent_backward(shape: MoeShape, weights: dict, x: torch.Tensor, scores: torch.Tensor,
                    idx: torch.Tensor, w: torch.Tensor, dout: torch.Tensor, workspace=None,
                    dscores=None):
    """Gradients of sum(out * dout) for a forward call with routing (scores
    [T,n] f32, idx [T,k] i32, w [T,k] f32), the selection held fixed.  Returns
    dict(dx, d_w_router, ...): fp32 weight gradients, dx in the activation
    dtype (bf16 layers only).  ``dscores`` [T,n] f32: a further gradient of
    the scores, such as the balance loss's, that :func:`router_backward` adds
    to dx, d_w_router and d_router_logit_offset."""
    dev = x.device
    T, d, l, n, k = shape.T, shape.d, shape.latent, shape.n_experts, shape.top_k
    m, ms = shape.inter, shape.shared_inter
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(dout, "dout", torch.bfloat16, (T, d), dev)
    _check(scores, "scores", torch.float32, (T, n), dev)
    _check(idx, "idx", torch.int32, (T, k), dev)
    _check(w, "w", torch.float32, (T, k), dev)
    if dscores is not None:  # refused before anything runs
        _check(dscores, "dscores", torch.float32, (T, n), dev)
    wts = MoeWeights(*[None if weights.get(f) is None else weights[f].data_ptr()
                       for f, _ in MoeWeights._fields_])
    out = {"dx": torch.empty((T, d), dtype=torch.bfloat16, device=dev)}
    for name, (key, fn) in GRAD_SHAPES.items():
        if weights.get(key) is None:
            out[name] = None
        else:
            out[name] = torch.empty(fn(T, d, l, n, k, m, ms), dtype=torch.float32, device=dev)
    grads = MoeGrads(*[None if out[f] is None else out[f].data_ptr() for f, _ in MoeGrads._fields_])
    need = _lib.moe_backward_workspace_bytes(ctypes.byref(shape))
    if need == 0:
        raise MoeError(-2, "moe_backward_workspace_bytes")
    ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8, device=dev)
    st = _lib.moe_latent_backward(ctypes.byref(shape), ctypes.byref(wts), _ptr(x), _ptr(scores),
                                  _ptr(idx), _ptr(w), _ptr(dout), ctypes.byref(grads), _ptr(ws),
                                  ws.numel(), _stream())
    if st != 0:
        raise MoeError(st, "moe_latent_backward")
    if dscores is not None:
        router_backward(x, weights["w_router"], scores, dscores, into=out)
    return out


EXPERT_GRADS = ("d_w_gate", "d_w_uproj", "d_w_dn")


def latent_backward_sgd(shape: MoeShape, weights: dict, x: torch.Tensor, scores: torch.Tensor,
                        idx: torch.Tensor, w: torch.Tensor, dout: torch.Tensor, lr: float,
                        workspace=None):
    """latent_backward followed by sgd_step in one call, the routed experts'
    weight gradients applied in place without being stored.  Updates every
    weight tensor of `weights`; returns the other gradients (dx, d_w_router,
    ...; the three expert entries are None)."""
    dev = x.device
    T, d, l, n, k = shape.T, shape.d, shape.latent, shape.n_experts, shape.top_k
    m, ms = shape.inter, shape.shared_inter
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(dout, "dout", torch.bfloat16, (T, d), dev)
    _check(scores, "scores", torch.float32, (T, n), dev)
    _check(idx, "idx", torch.int32, (T, k), dev)
    _check(w, "w", torch.float32, (T, k), dev)
    wts = MoeWeights(*[None if weights.get(f) is None else weights[f].data_ptr()
                       for f, _ in MoeWeights._fields_])
    out = {"dx": torch.empty((T, d), dtype=torch.bfloat16, device=dev)}
    for name, (key, fn) in GRAD_SHAPES.items():
        if weights.get(key) is None or name in EXPERT_GRADS:
            out[name] = None
        else:
            out[name] = torch.empty(fn(T, d, l, n, k, m, ms), dtype=torch.float32, device=dev)
    grads = MoeGrads(*[None if out[f] is None else out[f].data_ptr() for f, _ in MoeGrads._fields_])
    need = _lib.moe_backward_workspace_bytes(ctypes.byref(shape))
    if need == 0:
        raise MoeError(-2, "moe_backward_workspace_bytes")
    ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8, device=dev)
    st = _lib.moe_latent_backward_sgd(ctypes.byref(shape), ctypes.byref(wts), _ptr(x),
                                      _ptr(scores), _ptr(idx), _ptr(w), _ptr(dout),
                                      ctypes.byref(grads), ctypes.c_float(lr), _ptr(ws),
                                      ws.numel(), _stream())
    if st != 0:
        raise MoeError(st, "moe_latent_backward_sgd")
    return out


def latent_backward_train(shape: MoeShape, weights: dict, x: torch.Tensor, scores: torch.Tensor,
                          idx: torch.Tensor, w: torch.Tensor, dout: torch.Tensor,
                          saved: torch.Tensor, lr=None, workspace=None, dscores=None):
    """The backward of a training forward (latent_forward with `saved`),
    reading the activations it kept.  lr None: every gradient, as
    latent_backward; else the SGD step is applied as in latent_backward_sgd
    (the experts' gradients in place, not returned).  ``dscores`` as for
    latent_backward; not with lr, whose step comes before it could be added."""
    if dscores is not None and lr is not None:
        raise ValueError("dscores needs lr=None (apply sgd_step to the gradients)")
    dev = x.device
    T, d, l, n, k = shape.T, shape.d, shape.latent, shape.n_experts, shape.top_k
    m, ms = shape.inter, shape.shared_inter
    _check(x, "x", torch.bfloat16, (T, d), dev)
    _check(dout, "dout", torch.bfloat16, (T, d), dev)
    _check(scores, "scores", torch.float32, (T, n), dev)
    _check(idx, "idx", torch.int32, (T, k), dev)
    _check(w, "w", torch.float32, (T, k), dev)
    if dscores is not None:  # refused before anything runs
        _check(dscores, "dscores", torch.float32, (T, n), dev)
    _check(saved, "saved", torch.uint8, (saved.numel(),), dev)
    wts = MoeWeights(*[None if weights.get(f) is None else weights[f].data_ptr()
                       for f, _ in MoeWeights._fields_])
    out = {"dx": torch.empty((T, d), dtype=torch.bfloat16, device=dev)}
    for name, (key, fn) in GRAD_SHAPES.items():
        if weights.get(key) is None or (lr is not None and name in EXPERT_GRADS):
            out[name] = None
        else:
            out[name] = torch.empty(fn(T, d, l, n, k, m, ms), dtype=torch.float32, device=dev)
    grads = MoeGrads(*[None if out[f] is None else out[f].data_ptr() for f, _ in MoeGrads._fields_])
    need = _lib.moe_backward_workspace_bytes(ctypes.byref(shape))
    if need == 0:
        raise MoeError(-2, "moe_backward_workspace_bytes")
    ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8, device=dev)
    st = _lib.moe_latent_backward_train(ctypes.byref(shape), ctypes.byref(wts), _ptr(x),
                                        _ptr(scores), _ptr(idx), _ptr(w), _ptr(dout),
                                        _ptr(saved), saved.numel(), ctypes.byref(grads),
                                        0 if lr is None else 1,
                                        ctypes.c_float(0.0 if lr is None else lr), _ptr(ws),
                                        ws.numel(), _stream())
    if st != 0:
        raise MoeError(st, "moe_latent_backward_train")
    if dscores is not None:
        router_backward(x, weights["w_router"], scores, dscores, into=out)
    return out


def sgd_step(shape: MoeShape, weights: dict, grads: dict, lr: float):
    """One gradient-descent step in place on the weight tensors of `weights`
    (w <- w - lr * g, fp32 operations, stored in each weight's type) from
    `grads` as returned by latent_backward (dx is not used)."""
    wts = MoeWeights(*[None if weights.get(f) is None else weights[f].data_ptr()
                       for f, _ in MoeWeights._fields_])
    gr = MoeGrads(*[None if f == "dx" or grads.get(f) is None else grads[f].data_ptr()
                    for f, _ in MoeGrads._fields_])
    for name, (key, _) in GRAD_SHAPES.items():
        wt, g = weights.get(key), grads.get(name)
        if (wt is None) != (g is None) or (g is not None and (
                g.dtype != torch.float32 or g.shape != wt.shape or not g.is_contiguous()
                or not wt.is_contiguous() or g.device != wt.device)):
            raise ValueError(f"sgd_step: {name} does not match {key}")
    st = _lib.moe_sgd_step(ctypes.byref(shape), ctypes.byref(wts), ctypes.byref(gr),
                           ctypes.c_float(lr), _stream())
    if st != 0:
        raise MoeError(st, "moe_sgd_step")


def make_shape(T, d, latent, n, k, inter, shared_inter, act_dtype, routed_dtype,
               rms_eps=1e-6, qb_mode=MOE_QB_BATCH, qb_max_rounds=64) -> MoeShape:
    return MoeShape(T, d, latent, n, k, inter, shared_inter, act_dtype, routed_dtype, rms_eps,
                    qb_mode, qb_max_rounds)


def forward_workspace_bytes(shape: MoeShape) -> int:
    return int(_lib.moe_forward_workspace_bytes(ctypes.byref(shape)))


_DT = {MOE_F32: torch.float32, MOE_BF16: torch.bfloat16}


def saved_activations_bytes(shape: MoeShape) -> int:
    return int(_lib.moe_saved_activations_bytes(ctypes.byref(shape)))


def latent_forward(shape: MoeShape, weights: dict, x: torch.Tensor, bias=None,
                   scores_in=None, want_scores=False, workspace=None, saved=None):
    """One forward pass of the layer.

    ``saved``: a device uint8 buffer of saved_activations_bytes(shape) bytes;
    when given, the training forward also keeps there what
    latent_backward_train needs (bf16 layers).

    ``weights`` holds device tensors keyed as in ``moe_weights_t`` (MXFP4
    routed weights as uint8 codes plus ``s_gate``/``s_uproj``/``s_dn``).
    Returns dict(out, idx, w, loads, bias, info[, scores]).
    """
    dev = x.device
    T, d, l, n, k = shape.T, shape.d, shape.latent, shape.n_experts, shape.top_k
    m, ms = shape.inter, shape.shared_inter
    adt = _DT[shape.act_dtype]
    _check(x, "x", adt, (T, d), dev)
    _check(weights["w_router"], "w_router", torch.float32, (n, d), dev)
    if weights.get("router_logit_offset") is not None:
        _check(weights["router_logit_offset"], "router_logit_offset", torch.float32, (n,), dev)
    _check(weights["w_down"], "w_down", adt, (l, d), dev)
    _check(weights["w_up"], "w_up", adt, (d, l), dev)
    if shape.routed_dtype in (MOE_MXFP4, MOE_MXFP4_A8, MOE_MXFP4_A4):
        for nm, sn, rows, K in (("w_gate", "s_gate", m, l), ("w_uproj", "s_uproj", m, l),
                                ("w_dn", "s_dn", l, m)):
            _check(weights[nm], nm, torch.uint8, (n, rows, K // 2), dev)
            _check(weights[sn], sn, torch.uint8, (n, rows, K // 32), dev)
    else:
        rdt = _DT[shape.routed_dtype]
        _check(weights["w_gate"], "w_gate", rdt, (n, m, l), dev)
        _check(weights["w_uproj"], "w_uproj", rdt, (n, m, l), dev)
        _check(weights["w_dn"], "w_dn", rdt, (n, l, m), dev)
    _check(weights["rms_gamma"], "rms_gamma", torch.float32, (l,), dev)
    _check(weights["ws_gate"], "ws_gate", adt, (ms, d), dev)
    _check(weights["ws_up"], "ws_up", adt, (ms, d), dev)
    _check(weights["ws_down"], "ws_down", adt, (d, ms), dev)
    if scores_in is not None:
        _check(scores_in, "scores_in", torch.float32, (T, n), dev)
    wts = MoeWeights(*[None if weights.get(f) is None else weights[f].data_ptr()
                       for f, _ in MoeWeights._fields_])
    out = torch.empty((T, d), dtype=adt, device=dev)
    b = torch.zeros(n, dtype=torch.float64, device=dev) if bias is None else bias.clone()
    _check(b, "bias", torch.float64, (n,), dev)
    idx = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), dtype=torch.float32, device=dev)
    loads = torch.empty(n, dtype=torch.int32, device=dev)
    info = torch.zeros(4, dtype=torch.int32, device=dev)
    scores = torch.empty((T, n), dtype=torch.float32, device=dev) if want_scores else None
    need = forward_workspace_bytes(shape)
    if need == 0:
        raise MoeError(-1, "moe_forward_workspace_bytes")
    ws = workspace if workspace is not None else torch.empty(need, dtype=torch.uint8, device=dev)
    if saved is not None:
        _check(saved, "saved", torch.uint8, (saved.numel(),), dev)
        st = _lib.moe_latent_forward_train(ctypes.byref(shape), ctypes.byref(wts), _ptr(x),
                                           _ptr(out), _ptr(b), _ptr(scores_in), _ptr(scores),
                                           _ptr(idx), _ptr(w), _ptr(loads), _ptr(info),
                                           _ptr(saved), saved.numel(), _ptr(ws), ws.numel(),
                                           _stream())
        if st != 0:
            raise MoeError(st, "moe_latent_forward_train")
    else:
        st = _lib.moe_latent_forward(ctypes.byref(shape), ctypes.byref(wts), _ptr(x), _ptr(out),
                                     _ptr(b), _ptr(scores_in), _ptr(scores), _ptr(idx), _ptr(w),
                                     _ptr(loads), _ptr(info), _ptr(ws), ws.numel(), _stream())
        if st != 0:
            raise MoeError(st, "moe_latent_forward")
    res = dict(out=out, idx=idx, w=w, loads=loads, bias=b, info=info)
    if want_scores:
        res["scores"] = scores
    return res


def stage_timing(enable: bool) -> None:
    """Start (and reset) or stop per-stage HIP-event timing in the library."""
    _lib.moe_stage_timing(1 if enable else 0)


def stage_times() -> dict:
    """{stage name: (total ms, launches)} since the last stage_timing(True);
    synchronise the streams first."""
    tot = (ctypes.c_double * 16)()
    cnt = (ctypes.c_int32 * 16)()
    n = _lib.moe_stage_times(ctypes.cast(tot, ctypes.c_void_p), ctypes.cast(cnt, ctypes.c_void_p), 16)
    if n < 0:
        raise MoeError(n, "moe_stage_times")
    return {_lib.moe_stage_name(i).decode(): (tot[i], cnt[i]) for i in range(n)}
