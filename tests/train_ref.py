"""Plain 64-bit forms of the training operators for the tests, and the helpers they share.

Rounding allowances count half steps, torch.finfo(t).eps / 2 relative to the value, and for
fp32 sums the number of additions on a value's path times 2^-24 of the terms' magnitudes."""
from __future__ import annotations

import math

import torch

GROUP = 32
U32 = 2.0 ** -24


def half(dtype) -> float:
    return torch.finfo(dtype).eps / 2


def rel2(got, ref) -> float:
    """2-norm of the difference over the 2-norm of the reference."""
    d = (got.double() - ref).norm()
    n = ref.norm()
    return float(d / n) if n > 0 else float(d)


# ------------------------------------------------------------------ 8-bit checkpoints

def scales8(v, fmt):
    """(scale exponents k [rows][groups], bad [rows][groups]) of v [rows][cols] double."""
    rows, cols = v.shape
    g = -(-cols // GROUP)
    w = torch.nn.functional.pad(v, (0, g * GROUP - cols)).reshape(rows, g, GROUP)
    bad = ~torch.isfinite(w).all(dim=2)
    top = torch.where(torch.isfinite(w), w, 0.0).abs().amax(dim=2)
    m, e = torch.frexp(top)
    f, n = (127 / 128, 7) if fmt == "int8" else (448 / 512, 9)
    k = (e - n + (m > f)).clamp_min(-126)
    return torch.where(top == 0, -126, k).long(), bad


def codes8(v, fmt):
    """(codes as values, scale bytes) of an 8-bit checkpoint of v, exactly."""
    k, bad = scales8(v.double(), fmt)
    ke = k.repeat_interleave(GROUP, dim=1)[:, : v.shape[1]]
    r = torch.ldexp(v.double(), -ke)
    if fmt == "int8":
        q = r.round()  # half to even
    else:
        a = r.abs().clamp_min(2.0 ** -6)
        step = torch.ldexp(torch.ones_like(r), torch.frexp(a)[1] - 4)
        q = (r / step).round() * step
    q = torch.where(bad.repeat_interleave(GROUP, dim=1)[:, : v.shape[1]], 0.0, q)
    return q, torch.where(bad, 255, k + 127).to(torch.uint8)


def code_values(codes):
    """The values that int8 or E4M3 (uint8) codes stand for, as double."""
    if codes.dtype == torch.int8:
        return codes.double()
    return codes.view(torch.float8_e4m3fn).float().double()


def decode8(kept):
    """What an Act8 stands for, as double."""
    rows, width = kept.codes.shape
    cols = width // kept.parts
    g = -(-cols // GROUP)
    k = kept.scales.long() - 127
    out = code_values(kept.codes)
    for p in range(kept.parts):
        ke = k[:, p * g:(p + 1) * g].repeat_interleave(GROUP, dim=1)[:, :cols]
        part = torch.ldexp(out[:, p * cols:(p + 1) * cols], ke)
        out[:, p * cols:(p + 1) * cols] = torch.where(ke == 128, math.nan, part)
    return out


# ------------------------------------------------------------------ norms

def norm_forward(x, gain, bias, kind, eps):
    x = x.double()
    mean = x.mean(1) if kind == "layer" else torch.zeros_like(x[:, 0])
    rstd = 1 / torch.sqrt(((x - mean[:, None]) ** 2).mean(1) + eps)
    z = (x - mean[:, None]) * rstd[:, None]
    y = z * (1.0 if gain is None else gain.double())
    return y if bias is None else y + bias.double(), mean, rstd


def norm_backward(x, gain, mean, rstd, dy, kind):
    """dx, d_gain, d_bias by the operator's formulas."""
    x, dy = x.double(), dy.double()
    z = (x - mean[:, None]) * rstd[:, None]
    a = dy * (1.0 if gain is None else gain.double())
    dx = a - z * (a * z).mean(1, keepdim=True)
    if kind == "layer":
        dx = dx - a.mean(1, keepdim=True)
    return dx * rstd[:, None], (dy * z).sum(0), dy.sum(0)


# ------------------------------------------------------------------ the gated MLP

def gate(g, act):
    """act(g) and its derivative."""
    if act == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    k0, k1 = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(k0 * (g + k1 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * k0 * (1 + 3 * k1 * g * g)


def mlp_forward(x, wgu, wd, act):
    """y and the pre-activations [T][2D]."""
    gu = x.double() @ wgu.double().t()
    g, u = gu.chunk(2, dim=1)
    return (gate(g, act)[0] * u) @ wd.double().t(), gu


def mlp_backward(x, gu, wgu, wd, dy, act):
    """dx, dw_gate_up, dw_down by the operator's formulas from x and gu as kept."""
    x, gu, dy, wgu, wd = (t.double() for t in (x, gu, dy, wgu, wd))
    g, u = gu.chunk(2, dim=1)
    a, da = gate(g, act)
    dh = dy @ wd
    dgu = torch.cat((dh * u * da, dh * a), dim=1)
    return dgu @ wgu, dgu.t() @ x, dy.t() @ (a * u)


# ------------------------------------------------------------------ inputs

def normal(gen, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=gen, device=gen.device) * std).to(dtype)


def gen(seed, device="cuda"):
    return torch.Generator(device=device).manual_seed(seed)


def padded(t, extra, fill=7.0):
    """t's values in rows `extra` elements longer, the gaps filled: (view, base)."""
    base = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    base[:, : t.shape[1]] = t
    return base[:, : t.shape[1]], base
