"""Training operators of the block's dense branch: Python binding of include/moe_train.h.

Norms (RMS and layer) and the gated MLP with their backward passes, and the 8-bit
checkpoints of activations that the backward passes read in place of the activations:

    from mixture_experts_ffn_05_b200 import train

    ncfg = train.NormConfig(cols=H)                    # RMS norm, bf16
    mcfg = train.MlpConfig(hidden=H, inter=D)          # gelu_tanh, bf16
    kx, kxn = train.act8(T, H), train.act8(T, H)       # int8 codes and scales
    kgu = train.act8(T, D, parts=2)                    # gate and up halves
    ws, nws = train.mlp_workspace(mcfg, T), train.norm_workspace(ncfg, T)

    train.moe_norm_forward(ncfg, x, gain, None, xn, None, rstd, kept=kx)
    train.moe_act_encode(xn, kxn)
    train.moe_mlp_forward(mcfg, xn, w_gate_up, w_down, y, ws, kept_gu=kgu)
    ...
    train.moe_mlp_backward(mcfg, kxn, kgu, w_gate_up, w_down, dy, dxn, dw_gate_up, dw_down, ws)
    train.moe_norm_backward(ncfg, kx, gain, None, rstd, dxn, dx, d_gain, None, nws)

As in the package's other functions, every call checks and marshals its tensors and enqueues
the library's kernels on a stream (the tensors' device's current one by default).
Activations are 2-D tensors whose rows are contiguous and may lie further apart than their
length.  Nothing is recorded for autograd: outputs that require a gradient are refused outside
torch.no_grad(), and a written tensor's version goes up, so that a backward pass that had saved
it raises.  The header states formulas, layouts, limits and errors.
"""
from __future__ import annotations

import ctypes
import dataclasses

import torch

from . import MOE_ERR_INVALID_ARG, MoeError, _check, lib

F_BF16, F_F16, F_F32, F_INT8, F_E4M3 = range(5)
_FORMATS = {torch.bfloat16: F_BF16, torch.float16: F_F16, torch.float32: F_F32,
            torch.int8: F_INT8, torch.uint8: F_E4M3}
_KINDS = {"rms": 0, "layer": 1}
_ACTS = {"gelu_tanh": 0, "silu": 1}
GROUP = 32  # values of a row that share an 8-bit checkpoint's scale

# Entry points of include/moe_train.h (the CPU tests check the header declares exactly these).
ENTRY_POINTS = ("moe_act_encode", "moe_act_decode", "moe_norm_forward",
                "moe_norm_workspace_size", "moe_norm_backward", "moe_mlp_workspace_size",
                "moe_mlp_forward", "moe_mlp_backward")

_P, _I32, _I64, _SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t


class CAct(ctypes.Structure):
    _fields_ = [("data", _P), ("scales", _P), ("ld", _I64), ("format", _I32)]


class CNormConfig(ctypes.Structure):
    _fields_ = [("kind", _I32), ("cols", _I32), ("eps", ctypes.c_float), ("format", _I32),
                ("param_format", _I32)]


class CMlpConfig(ctypes.Structure):
    _fields_ = [("hidden", _I32), ("inter", _I32), ("act", _I32), ("format", _I32)]


_A, _N, _M = (ctypes.POINTER(c) for c in (CAct, CNormConfig, CMlpConfig))
_SIG = {
    "moe_act_encode": (_I32, [_I64, _I32, _A, _A, _P]),
    "moe_act_decode": (_I32, [_I64, _I32, _A, _A, _P]),
    "moe_norm_forward": (_I32, [_N, _I32, _A, _P, _P, _A, _P, _P, _A, _P]),
    "moe_norm_workspace_size": (_SZ, [_N, _I32]),
    "moe_norm_backward": (_I32, [_N, _I32, _A, _P, _P, _P, _A, _A, _P, _P, _I32, _P, _SZ, _P]),
    "moe_mlp_workspace_size": (_SZ, [_M, _I32]),
    "moe_mlp_forward": (_I32, [_M, _I32, _A, _P, _P, _A, _A, _P, _SZ, _P]),
    "moe_mlp_backward": (_I32, [_M, _I32, _A, _A, _P, _P, _A, _A, _P, _P, _I32, _I32, _P, _SZ,
                                _P]),
}

_fns = None


def _lib():
    """The library's functions with this interface's signatures."""
    global _fns
    if _fns is None:
        l = lib()
        for name, (res, args) in _SIG.items():
            f = getattr(l, name)
            f.restype, f.argtypes = res, args
        _fns = l
    return _fns


# ------------------------------------------------------------------ tensors

@dataclasses.dataclass(frozen=True)
class Act8:
    """An 8-bit checkpoint of an activation: codes [rows][parts * cols] (int8, or E4M3 codes
    as uint8) and scale bytes [rows][parts * ceil(cols / 32)] (uint8)."""
    codes: torch.Tensor
    scales: torch.Tensor
    parts: int = 1


def act8(rows: int, cols: int, fmt: str = "int8", parts: int = 1, device=None) -> Act8:
    """A new checkpoint for [rows][cols] (fmt: int8 or e4m3).  parts = 2: for the gated MLP's
    pre-activations, gate and up halves of cols columns each, with scales of their own."""
    dt = {"int8": torch.int8, "e4m3": torch.uint8}[fmt]
    device = device or "cuda"
    return Act8(torch.empty(rows, parts * cols, dtype=dt, device=device),
                torch.empty(rows, parts * (-(-cols // GROUP)), dtype=torch.uint8, device=device),
                parts)


# A device's current stream as a handle, and the current device: torch.cuda.current_stream alone
# takes longer than the rest of a call, and at one token the host's time is the call's time.
_get_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream
_Tensor = torch.Tensor


def _first(t, name):
    """(device index, rows, columns) of a call's first tensor, whose device the others share."""
    if isinstance(t, Act8):
        t = t.codes
    if not isinstance(t, _Tensor):
        raise TypeError(f"{name} must be a torch.Tensor or an Act8")
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(shape)}")
    return t.get_device(), shape[0], shape[1]


def _i32(n):
    """A size as an int32 argument.  ctypes would take it modulo 2^32; one that does not fit
    becomes the largest, which the library refuses as unsupported."""
    return n if -0x80000000 <= n <= 0x7FFFFFFF else 0x7FFFFFFF


def _wrong_device(t, name, index):
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    raise ValueError(f"{name} is on {t.device}, the call's first tensor on cuda:{index}")


def _ptr(t, name, index, dtype, numel):
    """The address of a contiguous tensor of `numel` elements (None: any number)."""
    if not isinstance(t, _Tensor):
        if t is None:
            raise ValueError(f"{name} is required")
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        _wrong_device(t, name, index)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must hold {numel} elements, got {t.numel()}")
    return t.data_ptr()


def _act(t, name, index, rows, cols, dtype, parts=1):
    """The C description of an activation [rows][parts * cols]: a tensor of `dtype` (None: bf16,
    fp16 or fp32) or an Act8."""
    width = parts * cols
    scales = None
    if isinstance(t, _Tensor):
        fmt = _FORMATS.get(t.dtype, 9)
        if (fmt > F_F32) if dtype is None else (t.dtype is not dtype):
            raise TypeError(f"{name} must be {dtype or 'bf16, fp16 or fp32'}, got {t.dtype}")
    elif isinstance(t, Act8):
        if t.parts != parts:
            raise ValueError(f"{name} must be a checkpoint of {parts} part(s)")
        scales = _ptr(t.scales, f"{name}.scales", index, torch.uint8,
                      rows * parts * (-(-cols // GROUP)))
        t = t.codes
        fmt = _FORMATS.get(t.dtype, 9)
        if fmt != F_INT8 and fmt != F_E4M3:
            raise TypeError(f"{name}: codes must be torch.int8 or torch.uint8 (E4M3)")
    elif t is None:
        raise ValueError(f"{name} is required")
    else:
        raise TypeError(f"{name} must be a torch.Tensor or an Act8")
    if t.get_device() != index:
        _wrong_device(t, name, index)
    if t.shape != (rows, width):
        raise ValueError(f"{name} must be [{rows}, {width}], got {tuple(t.shape)}")
    ld, inner = t.stride()
    if inner != 1 and width > 1:
        raise ValueError(f"{name} must have contiguous rows")
    # of one row the stride says nothing
    return CAct(t.data_ptr(), scales, ld if rows > 1 else width, fmt)


def _plain(t, name):
    """A value that must not be an Act8."""
    if isinstance(t, Act8):
        raise TypeError(f"{name} must be a torch.Tensor")
    return t


_recording = torch.is_grad_enabled
# Tells autograd that tensors were written, so that a backward pass that had saved one raises
# and does not use the new values (torch.autograd.graph.increment_version, without its checks).
_written = torch._C._increment_version


def _no_grad(*outputs):
    """Nothing here is recorded for autograd, so an output that requires a gradient is refused
    while autograd records, as torch refuses it as an `out` argument."""
    if _recording():
        for t in outputs:
            if getattr(t, "requires_grad", False):
                raise ValueError("an output requires a gradient, and these calls record none: "
                                 "pass a detached tensor or call under torch.no_grad()")


def _run(name, index, stream, *args):
    if index < 0:
        raise ValueError(f"{name}: the tensors must be on a CUDA device")
    fn = getattr(_fns or _lib(), name)
    s = _raw_stream(index) if stream is None else stream.cuda_stream
    if index == _get_device():
        st = fn(*args, s)
    else:
        with torch.cuda.device(index):
            st = fn(*args, s)
    if st:
        _check(name, st)


def _zeros(n, fn, device):
    if n == 0:
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


# ------------------------------------------------------------------ 8-bit checkpoints

def _checkpoint(kept):
    if not isinstance(kept, Act8):
        raise TypeError("kept must be an Act8")
    return kept


def moe_act_encode(x, kept: Act8, stream=None) -> None:
    """Write the 8-bit checkpoint of x [rows][cols] (bf16, fp16 or fp32)."""
    i, rows, cols = _first(_plain(x, "x"), "x")
    _run("moe_act_encode", i, stream, rows, _i32(cols), _act(x, "x", i, rows, cols, None),
         _act(_checkpoint(kept), "kept", i, rows, cols, None))
    _written((kept.codes, kept.scales))


def moe_act_decode(kept: Act8, out, stream=None) -> None:
    """Read an 8-bit checkpoint back into out [rows][cols] (bf16, fp16 or fp32)."""
    i, rows, cols = _first(_plain(out, "out"), "out")
    _no_grad(out)
    _run("moe_act_decode", i, stream, rows, _i32(cols),
         _act(_checkpoint(kept), "kept", i, rows, cols, None),
         _act(out, "out", i, rows, cols, None))
    _written((out,))


# ------------------------------------------------------------------ norms

@dataclasses.dataclass(frozen=True)
class NormConfig:
    cols: int
    kind: str = "rms"  # or "layer"
    eps: float = 1e-6
    dtype: torch.dtype = torch.bfloat16        # of x, y, dy and dx
    param_dtype: torch.dtype = torch.bfloat16  # of gain and bias

    def __post_init__(self):
        object.__setattr__(self, "_c", CNormConfig(
            _KINDS[self.kind], _i32(self.cols), self.eps, _FORMATS[self.dtype],
            _FORMATS[self.param_dtype]))

    def c(self) -> CNormConfig:
        return self._c


def norm_workspace(cfg: NormConfig, T: int, device=None) -> torch.Tensor:
    """A zeroed workspace for moe_norm_backward over T rows."""
    n = int(_lib().moe_norm_workspace_size(cfg._c, _i32(int(T))))
    return _zeros(n, "moe_norm_workspace_size", device)


def moe_norm_forward(cfg, x, gain, bias, y, mean, rstd, kept: Act8 | None = None,
                     stream=None) -> None:
    """y = norm(x) * gain + bias with the row statistics the backward pass needs (mean: layer
    norm only), and on request the 8-bit checkpoint of x.  gain and bias may be None."""
    i, T, _ = _first(_plain(x, "x"), "x")
    n, dt, pt, f32 = cfg.cols, cfg.dtype, cfg.param_dtype, torch.float32
    _no_grad(y, mean, rstd)
    _run("moe_norm_forward", i, stream, cfg._c, _i32(T), _act(x, "x", i, T, n, dt),
         None if gain is None else _ptr(gain, "gain", i, pt, n),
         None if bias is None else _ptr(bias, "bias", i, pt, n),
         _act(_plain(y, "y"), "y", i, T, n, dt),
         None if mean is None else _ptr(mean, "mean", i, f32, T), _ptr(rstd, "rstd", i, f32, T),
         None if kept is None else _act(_checkpoint(kept), "kept", i, T, n, None))
    _written((y, rstd) if mean is None else (y, mean, rstd))
    if kept is not None:
        _written((kept.codes, kept.scales))


def moe_norm_backward(cfg, x, gain, mean, rstd, dy, dx, d_gain, d_bias, ws,
                      accumulate: bool = False, stream=None) -> None:
    """dx and the fp32 gradients of gain and bias (either may be None), from x or its 8-bit
    checkpoint and the forward pass's statistics.  accumulate adds to d_gain and d_bias."""
    i, T, _ = _first(x, "x")
    n, dt, f32 = cfg.cols, cfg.dtype, torch.float32
    _no_grad(dx, d_gain, d_bias)
    _run("moe_norm_backward", i, stream, cfg._c, _i32(T), _act(x, "x", i, T, n, dt),
         None if gain is None else _ptr(gain, "gain", i, cfg.param_dtype, n),
         None if mean is None else _ptr(mean, "mean", i, f32, T), _ptr(rstd, "rstd", i, f32, T),
         _act(_plain(dy, "dy"), "dy", i, T, n, dt), _act(_plain(dx, "dx"), "dx", i, T, n, dt),
         None if d_gain is None else _ptr(d_gain, "d_gain", i, f32, n),
         None if d_bias is None else _ptr(d_bias, "d_bias", i, f32, n), 1 if accumulate else 0,
         _ptr(ws, "ws", i, torch.uint8, None), ws.numel())
    _written([t for t in (dx, d_gain, d_bias) if t is not None])


# ------------------------------------------------------------------ the gated MLP

@dataclasses.dataclass(frozen=True)
class MlpConfig:
    hidden: int
    inter: int
    act: str = "gelu_tanh"  # or "silu"
    dtype: torch.dtype = torch.bfloat16  # or torch.float16

    def __post_init__(self):
        object.__setattr__(self, "_c", CMlpConfig(
            _i32(self.hidden), _i32(self.inter), _ACTS[self.act], _FORMATS[self.dtype]))

    def c(self) -> CMlpConfig:
        return self._c


def mlp_workspace(cfg: MlpConfig, T: int, device=None) -> torch.Tensor:
    """A zeroed workspace for moe_mlp_forward and moe_mlp_backward over T rows."""
    n = int(_lib().moe_mlp_workspace_size(cfg._c, _i32(int(T))))
    return _zeros(n, "moe_mlp_workspace_size", device)


def moe_mlp_forward(cfg, x, w_gate_up, w_down, y, ws, kept_gu=None, stream=None) -> None:
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T.  kept_gu: None, or what the backward pass needs of
    it, a [T][2D] tensor or an Act8 of two parts."""
    i, T, _ = _first(_plain(x, "x"), "x")
    H, D, dt = cfg.hidden, cfg.inter, cfg.dtype
    _no_grad(y, kept_gu)
    _run("moe_mlp_forward", i, stream, cfg._c, _i32(T), _act(x, "x", i, T, H, dt),
         _ptr(w_gate_up, "w_gate_up", i, dt, 2 * D * H), _ptr(w_down, "w_down", i, dt, D * H),
         _act(_plain(y, "y"), "y", i, T, H, dt),
         None if kept_gu is None else _act(kept_gu, "kept_gu", i, T, D, dt, 2),
         _ptr(ws, "ws", i, torch.uint8, None), ws.numel())
    _written((y,) if kept_gu is None else (y, kept_gu.codes, kept_gu.scales)
             if isinstance(kept_gu, Act8) else (y, kept_gu))


def moe_mlp_backward(cfg, x, gu, w_gate_up, w_down, dy, dx, dw_gate_up, dw_down, ws,
                     accumulate: bool = False, stream=None) -> None:
    """The gradients of x and the weights from x and gu as kept (tensors or Act8).  dx,
    dw_gate_up and dw_down may be None; the weight gradients are in cfg's dtype or fp32, both
    the same, and accumulate adds to what they hold."""
    i, T, _ = _first(_plain(dy, "dy"), "dy")
    H, D, dt = cfg.hidden, cfg.inter, cfg.dtype
    grad = next((g.dtype for g in (dw_gate_up, dw_down) if g is not None), dt)
    if grad not in (dt, torch.float32):
        raise TypeError(f"weight gradients must be {dt} or torch.float32, got {grad}")
    _no_grad(dx, dw_gate_up, dw_down)
    _run("moe_mlp_backward", i, stream, cfg._c, _i32(T),
         None if x is None and dw_gate_up is None else _act(x, "x", i, T, H, dt),
         _act(gu, "gu", i, T, D, dt, 2),
         None if w_gate_up is None and dx is None else
         _ptr(w_gate_up, "w_gate_up", i, dt, 2 * D * H),
         _ptr(w_down, "w_down", i, dt, D * H), _act(dy, "dy", i, T, H, dt),
         None if dx is None else _act(_plain(dx, "dx"), "dx", i, T, H, dt),
         None if dw_gate_up is None else _ptr(dw_gate_up, "dw_gate_up", i, grad, 2 * D * H),
         None if dw_down is None else _ptr(dw_down, "dw_down", i, grad, D * H), _FORMATS[grad],
         1 if accumulate else 0, _ptr(ws, "ws", i, torch.uint8, None), ws.numel())
    _written([t for t in (dx, dw_gate_up, dw_down) if t is not None])
