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
length.  The header states formulas, layouts, limits and errors.
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


# The device's index of a tensor (-1: CPU) and a device's current stream as a handle: the calls
# of one token take a few microseconds, of which torch.cuda.current_stream alone would be half.
_get_device = torch._C._cuda_getDevice
_raw_stream = torch._C._cuda_getCurrentRawStream


class _Call:
    """One call's tensors: all on one device, which is current while the call is made."""
    __slots__ = ("index", "stream")

    def __init__(self, first, stream):
        if isinstance(first, Act8):
            first = first.codes
        if not isinstance(first, torch.Tensor):
            raise TypeError("an activation must be a torch.Tensor or an Act8")
        self.index, self.stream = first.get_device(), stream

    def _on_device(self, t, name):
        if t.get_device() != self.index or self.index < 0:
            if not t.is_cuda:
                raise ValueError(f"{name} must be on a CUDA device")
            raise ValueError(f"{name} is on {t.device}, the call's first tensor on "
                             f"{f'cuda:{self.index}' if self.index >= 0 else 'the CPU'}")

    def ptr(self, t, name, dtype=None, numel=None, nullable=False):
        if t is None:
            if nullable:
                return None
            raise ValueError(f"{name} is required")
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if dtype is not None and t.dtype != dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        self._on_device(t, name)
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if numel is not None and t.numel() != numel:
            raise ValueError(f"{name} must hold {numel} elements, got {t.numel()}")
        return t.data_ptr()

    def act(self, t, name, rows, cols, dtype=None, parts=1, nullable=False):
        """The C description of an activation [rows][parts * cols], a tensor or an Act8;
        dtype None takes any format."""
        if t is None:
            if nullable:
                return None
            raise ValueError(f"{name} is required")
        scales = None
        width = parts * cols
        if isinstance(t, Act8):
            data = t.codes
            if data.dtype not in (torch.int8, torch.uint8):
                raise TypeError(f"{name}: codes must be torch.int8 or torch.uint8 (E4M3)")
            if t.parts != parts:
                raise ValueError(f"{name} must be a checkpoint of {parts} part(s)")
            scales = self.ptr(t.scales, f"{name}.scales", torch.uint8,
                              rows * parts * (-(-cols // GROUP)))
        elif not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor or an Act8")
        else:
            data = t
            if (t.dtype != dtype) if dtype is not None else (_FORMATS.get(t.dtype, 9) > F_F32):
                raise TypeError(f"{name} must be {dtype or 'bf16, fp16 or fp32'}, got {t.dtype}")
        self._on_device(data, name)
        if data.shape != (rows, width):
            raise ValueError(f"{name} must be [{rows}, {width}], got {tuple(data.shape)}")
        strides = data.stride()
        if width > 1 and strides[1] != 1:
            raise ValueError(f"{name} must have contiguous rows")
        # of one row the stride says nothing
        return CAct(data.data_ptr(), scales, strides[0] if rows > 1 else width,
                    _FORMATS[data.dtype])

    def run(self, name, *args):
        fn = getattr(_fns or _lib(), name)
        index = self.index
        s = _raw_stream(index) if self.stream is None else self.stream.cuda_stream
        if index == _get_device():
            st = fn(*args, s)
        else:
            with torch.cuda.device(index):
                st = fn(*args, s)
        if st:
            _check(name, st)


def _shape(t, name):
    t = t.codes if isinstance(t, Act8) else t
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor or an Act8")
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D, got {tuple(t.shape)}")
    return t.shape


def _zeros(n, fn, device):
    if n == 0:
        raise MoeError(fn, MOE_ERR_INVALID_ARG)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


# ------------------------------------------------------------------ 8-bit checkpoints

def moe_act_encode(x, kept: Act8, stream=None) -> None:
    """Write the 8-bit checkpoint of x [rows][cols] (bf16, fp16 or fp32)."""
    rows, cols = _shape(x, "x")
    if not isinstance(kept, Act8):
        raise TypeError("kept must be an Act8")
    c = _Call(x, stream)
    c.run("moe_act_encode", rows, cols, c.act(x, "x", rows, cols),
          c.act(kept, "kept", rows, cols))


def moe_act_decode(kept: Act8, out, stream=None) -> None:
    """Read an 8-bit checkpoint back into out [rows][cols] (bf16, fp16 or fp32)."""
    rows, cols = _shape(out, "out")
    if not isinstance(kept, Act8):
        raise TypeError("kept must be an Act8")
    c = _Call(out, stream)
    c.run("moe_act_decode", rows, cols, c.act(kept, "kept", rows, cols),
          c.act(out, "out", rows, cols))


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
            _KINDS[self.kind], self.cols, self.eps, _FORMATS[self.dtype],
            _FORMATS[self.param_dtype]))

    def c(self) -> CNormConfig:
        return self._c


def norm_workspace(cfg: NormConfig, T: int, device=None) -> torch.Tensor:
    """A zeroed workspace for moe_norm_backward over T rows."""
    n = int(_lib().moe_norm_workspace_size(cfg._c, int(T)))
    return _zeros(n, "moe_norm_workspace_size", device)


def moe_norm_forward(cfg, x, gain, bias, y, mean, rstd, kept: Act8 | None = None,
                     stream=None) -> None:
    """y = norm(x) * gain + bias with the row statistics the backward pass needs (mean: layer
    norm only), and on request the 8-bit checkpoint of x.  gain and bias may be None."""
    T, n = _shape(x, "x")
    c = _Call(x, stream)
    if kept is not None and not isinstance(kept, Act8):
        raise TypeError("kept must be an Act8")
    f32 = torch.float32
    c.run("moe_norm_forward", cfg._c, T, c.act(x, "x", T, cfg.cols, cfg.dtype),
          c.ptr(gain, "gain", cfg.param_dtype, cfg.cols, True),
          c.ptr(bias, "bias", cfg.param_dtype, cfg.cols, True),
          c.act(y, "y", T, cfg.cols, cfg.dtype), c.ptr(mean, "mean", f32, T, True),
          c.ptr(rstd, "rstd", f32, T), c.act(kept, "kept", T, cfg.cols, nullable=True))


def moe_norm_backward(cfg, x, gain, mean, rstd, dy, dx, d_gain, d_bias, ws,
                      accumulate: bool = False, stream=None) -> None:
    """dx and the fp32 gradients of gain and bias (either may be None), from x or its 8-bit
    checkpoint and the forward pass's statistics.  accumulate adds to d_gain and d_bias."""
    T, n = _shape(x, "x")
    c = _Call(x, stream)
    f32 = torch.float32
    c.run("moe_norm_backward", cfg._c, T, c.act(x, "x", T, cfg.cols, cfg.dtype),
          c.ptr(gain, "gain", cfg.param_dtype, cfg.cols, True),
          c.ptr(mean, "mean", f32, T, True), c.ptr(rstd, "rstd", f32, T),
          c.act(dy, "dy", T, cfg.cols, cfg.dtype), c.act(dx, "dx", T, cfg.cols, cfg.dtype),
          c.ptr(d_gain, "d_gain", f32, cfg.cols, True),
          c.ptr(d_bias, "d_bias", f32, cfg.cols, True), int(bool(accumulate)),
          c.ptr(ws, "ws", torch.uint8), ws.numel())


# ------------------------------------------------------------------ the gated MLP

@dataclasses.dataclass(frozen=True)
class MlpConfig:
    hidden: int
    inter: int
    act: str = "gelu_tanh"  # or "silu"
    dtype: torch.dtype = torch.bfloat16  # or torch.float16

    def __post_init__(self):
        object.__setattr__(self, "_c", CMlpConfig(self.hidden, self.inter, _ACTS[self.act],
                                                  _FORMATS[self.dtype]))

    def c(self) -> CMlpConfig:
        return self._c


def mlp_workspace(cfg: MlpConfig, T: int, device=None) -> torch.Tensor:
    """A zeroed workspace for moe_mlp_forward and moe_mlp_backward over T rows."""
    n = int(_lib().moe_mlp_workspace_size(cfg._c, int(T)))
    return _zeros(n, "moe_mlp_workspace_size", device)


def moe_mlp_forward(cfg, x, w_gate_up, w_down, y, ws, kept_gu=None, stream=None) -> None:
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T.  kept_gu: None, or what the backward pass needs of
    it, a [T][2D] tensor or an Act8 of two parts."""
    T, n = _shape(x, "x")
    H, D = cfg.hidden, cfg.inter
    c = _Call(x, stream)
    c.run("moe_mlp_forward", cfg._c, T, c.act(x, "x", T, H, cfg.dtype),
          c.ptr(w_gate_up, "w_gate_up", cfg.dtype, 2 * D * H),
          c.ptr(w_down, "w_down", cfg.dtype, D * H), c.act(y, "y", T, H, cfg.dtype),
          c.act(kept_gu, "kept_gu", T, D, cfg.dtype, 2, True), c.ptr(ws, "ws", torch.uint8),
          ws.numel())


def moe_mlp_backward(cfg, x, gu, w_gate_up, w_down, dy, dx, dw_gate_up, dw_down, ws,
                     accumulate: bool = False, stream=None) -> None:
    """The gradients of x and the weights from x and gu as kept (tensors or Act8).  dx,
    dw_gate_up and dw_down may be None; the weight gradients are in cfg's dtype or fp32, both
    the same, and accumulate adds to what they hold."""
    T, n = _shape(dy, "dy")
    H, D = cfg.hidden, cfg.inter
    c = _Call(dy, stream)
    grad = next((g.dtype for g in (dw_gate_up, dw_down) if g is not None), cfg.dtype)
    if grad not in (cfg.dtype, torch.float32):
        raise TypeError(f"weight gradients must be {cfg.dtype} or torch.float32, got {grad}")
    c.run("moe_mlp_backward", cfg._c, T,
          c.act(x, "x", T, H, cfg.dtype, nullable=dw_gate_up is None),
          c.act(gu, "gu", T, D, cfg.dtype, 2),
          c.ptr(w_gate_up, "w_gate_up", cfg.dtype, 2 * D * H, dx is None),
          c.ptr(w_down, "w_down", cfg.dtype, D * H),
          c.act(dy, "dy", T, H, cfg.dtype), c.act(dx, "dx", T, H, cfg.dtype, nullable=True),
          c.ptr(dw_gate_up, "dw_gate_up", grad, 2 * D * H, True),
          c.ptr(dw_down, "dw_down", grad, D * H, True), _FORMATS[grad], int(bool(accumulate)),
          c.ptr(ws, "ws", torch.uint8), ws.numel())
