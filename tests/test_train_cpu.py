"""The training operators' interface on the CPU: the header's entry points, the workspace
sizes, every refusal (found on the host before anything is launched), and the plain forms
that the GPU tests compare with, against automatic differentiation and differences."""
import ctypes
import os
import re
import subprocess

import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import build as mbuild
from mixture_experts_ffn_05_b200 import train
from tests import train_ref as ref

HEADER = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include",
                      "moe_train.h")
FAKE = 1 << 20  # an aligned address that is never dereferenced
OK, INVALID, UNSUPPORTED, WORKSPACE = (mf.MOE_OK, mf.MOE_ERR_INVALID_ARG, mf.MOE_ERR_UNSUPPORTED,
                                       mf.MOE_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return train._lib()


def test_header_declares_and_library_exports_the_entry_points(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    names = sorted(set(re.findall(r"^[A-Za-z_][\w \*]*?\b(\w+)\s*\(", text, flags=re.M)))
    assert names == sorted(train.ENTRY_POINTS)
    out = subprocess.run(["nm", "-D", "--defined-only", mf.LIB_PATH], capture_output=True,
                         text=True, check=True).stdout
    exported = {l.split()[-1] for l in out.splitlines() if l.strip()}
    assert set(names) <= exported


def act(fmt=train.F_BF16, ld=64, data=FAKE, scales=None):
    if scales is None and fmt in (train.F_INT8, train.F_E4M3):
        scales = FAKE
    return train.CAct(data, scales or None, ld, fmt)


def test_act8_refusals(lib):
    enc, dec = lib.moe_act_encode, lib.moe_act_decode

    def both(rows, cols, vals, codes):
        a = enc(rows, cols, vals, codes, None)
        b = dec(rows, cols, codes, vals, None)
        assert a == b
        return a

    good, good8 = act(), act(train.F_INT8)
    assert both(0, 64, good, good8) == OK  # no rows: nothing to do
    assert both(-1, 64, good, good8) == INVALID
    assert both(4, 0, good, good8) == INVALID
    assert both(4, 65537, act(ld=70000), act(train.F_INT8, ld=70000)) == UNSUPPORTED
    assert both((1 << 46) // 64, 64, good, good8) == UNSUPPORTED
    assert both(4, 64, good8, good) == INVALID          # the formats exchanged
    assert both(4, 64, good, good) == INVALID           # not an 8-bit checkpoint
    assert both(4, 64, act(7), good8) == INVALID
    assert both(4, 64, good, act(9)) == INVALID
    assert both(4, 64, act(ld=63), good8) == INVALID    # rows overlap
    assert both(4, 64, good, act(train.F_E4M3, ld=63)) == INVALID
    assert both(4, 64, act(data=None), good8) == INVALID
    assert both(4, 64, act(data=FAKE + 8), good8) == INVALID
    assert both(4, 64, act(scales=FAKE), good8) == INVALID
    assert both(4, 64, good, train.CAct(FAKE, None, 64, train.F_INT8)) == INVALID
    assert enc(4, 64, None, good8, None) == INVALID and enc(4, 64, good, None, None) == INVALID


def norm_cfg(kind=0, cols=64, eps=1e-6, fmt=0, pfmt=0):
    return train.CNormConfig(kind, cols, eps, fmt, pfmt)


def test_norm_refusals(lib):
    f, b, size = lib.moe_norm_forward, lib.moe_norm_backward, lib.moe_norm_workspace_size
    n = size(norm_cfg(), 4)
    assert n > 0 and size(norm_cfg(), 1 << 20) >= n and size(norm_cfg(), 0) > 0

    def fwd(c=norm_cfg(), T=4, x=act(), gain=FAKE, bias=None, y=act(data=2 * FAKE), mean=None,
            rstd=FAKE, kept=None):
        return f(c, T, x, gain, bias, y, mean, rstd, kept, None)

    def bwd(c=norm_cfg(), T=4, x=act(), gain=FAKE, mean=None, rstd=FAKE, dy=act(),
            dx=act(data=2 * FAKE), dg=FAKE, db=None, ws=FAKE, n=n):
        return b(c, T, x, gain, mean, rstd, dy, dx, dg, db, 0, ws, n, None)

    layer = norm_cfg(kind=1)
    for c, want in ((norm_cfg(kind=2), INVALID), (norm_cfg(cols=0), UNSUPPORTED),
                    (norm_cfg(cols=16385), UNSUPPORTED), (norm_cfg(eps=0.0), INVALID),
                    (norm_cfg(eps=float("nan")), INVALID), (norm_cfg(eps=float("inf")), INVALID),
                    (norm_cfg(fmt=3), INVALID), (norm_cfg(pfmt=4), INVALID)):
        assert fwd(c) == want and bwd(c) == want and size(c, 4) == 0
    assert f(None, 4, act(), None, None, act(), None, FAKE, None, None) == INVALID
    assert fwd(T=-1) == INVALID and bwd(T=-1) == INVALID and size(norm_cfg(), -1) == 0
    assert fwd(T=2 ** 31 - 1) == UNSUPPORTED
    assert fwd(T=0) == OK and bwd(T=0, dg=None) == OK
    assert fwd(bias=FAKE) == INVALID and fwd(mean=FAKE) == INVALID  # RMS has neither
    assert bwd(db=FAKE) == INVALID and bwd(mean=FAKE) == INVALID
    assert fwd(layer) == INVALID and bwd(layer) == INVALID          # layer needs the mean
    for bad in (None, act(ld=63), act(data=None), act(data=FAKE + 2), act(1), act(scales=FAKE)):
        assert fwd(x=bad) == INVALID and fwd(y=bad) == INVALID
        assert bwd(x=bad) == INVALID and bwd(dy=bad) == INVALID and bwd(dx=bad) == INVALID
    assert fwd(x=act(3)) == INVALID                # forward takes no checkpoint
    assert bwd(x=train.CAct(FAKE, None, 64, 3)) == INVALID
    assert fwd(kept=act()) == INVALID and fwd(kept=act(3, ld=32)) == INVALID
    assert fwd(gain=FAKE + 4) == INVALID and bwd(gain=FAKE + 4) == INVALID
    assert fwd(rstd=None) == INVALID and bwd(rstd=None) == INVALID
    assert bwd(dg=FAKE + 4) == INVALID
    # in place only with the same rows
    assert fwd(x=act(ld=64), y=act(ld=72)) == INVALID
    assert bwd(dy=act(ld=64), dx=act(ld=72)) == INVALID
    assert bwd(ws=None) == WORKSPACE and bwd(ws=FAKE + 16) == WORKSPACE
    assert bwd(n=n - 1) == WORKSPACE


def mlp_cfg(H=64, D=72, a=0, fmt=0):
    return train.CMlpConfig(H, D, a, fmt)


def test_mlp_refusals(lib):
    f, b, size = lib.moe_mlp_forward, lib.moe_mlp_backward, lib.moe_mlp_workspace_size
    n = size(mlp_cfg(), 4)
    assert n > 0 and size(mlp_cfg(), 4096) > n and size(mlp_cfg(), 0) > 0
    kept16, kept8 = act(ld=144), act(3, ld=144)

    def fwd(c=mlp_cfg(), T=4, x=act(), wgu=FAKE, wd=FAKE, y=act(), kept=None, ws=FAKE, n=n):
        return f(c, T, x, wgu, wd, y, kept, ws, n, None)

    def bwd(c=mlp_cfg(), T=4, x=act(), gu=kept16, wgu=FAKE, wd=FAKE, dy=act(), dx=act(),
            dwgu=FAKE, dwd=FAKE, gf=0, ws=FAKE, n=n):
        return b(c, T, x, gu, wgu, wd, dy, dx, dwgu, dwd, gf, 0, ws, n, None)

    for c, want in ((mlp_cfg(H=0), UNSUPPORTED), (mlp_cfg(H=60), UNSUPPORTED),
                    (mlp_cfg(D=16392), UNSUPPORTED), (mlp_cfg(D=4), UNSUPPORTED),
                    (mlp_cfg(a=2), INVALID), (mlp_cfg(fmt=2), INVALID)):
        assert fwd(c) == want and bwd(c) == want and size(c, 4) == 0
    assert f(None, 4, act(), FAKE, FAKE, act(), None, FAKE, n, None) == INVALID
    assert fwd(T=-1) == INVALID and fwd(T=2 ** 31 - 1) == UNSUPPORTED
    assert fwd(T=0) == OK and bwd(T=0, dwgu=None, dwd=None) == OK
    for bad in (None, act(ld=60), act(ld=68), act(data=None), act(data=FAKE + 8), act(1), act(3)):
        assert fwd(x=bad) == INVALID and fwd(y=bad) == INVALID and bwd(dy=bad) == INVALID
        if bad is not None:
            assert bwd(dx=bad) == INVALID
    assert fwd(wgu=None) == INVALID and fwd(wd=FAKE + 4) == INVALID
    for bad in (act(ld=136), act(3, ld=136), act(ld=148), act(1, ld=144),
                train.CAct(FAKE, None, 144, 4)):
        assert fwd(kept=bad) == INVALID and bwd(gu=bad) == INVALID
    assert bwd(gu=None) == INVALID and bwd(x=None) == INVALID and bwd(x=act(1)) == INVALID
    assert bwd(x=act(3, ld=68)) == INVALID
    assert bwd(wd=None) == INVALID and bwd(wgu=None) == INVALID
    assert bwd(dwgu=FAKE + 4) == INVALID and bwd(dwd=FAKE + 4) == INVALID
    assert bwd(gf=1) == INVALID and bwd(gf=3) == INVALID  # cfg's format or fp32
    for kw in ({"ws": None}, {"ws": FAKE + 16}, {"n": n - 1}):
        assert fwd(**kw) == WORKSPACE and fwd(kept=kept8, **kw) == WORKSPACE
        assert bwd(**kw) == WORKSPACE and bwd(gu=kept8, x=act(4), **kw) == WORKSPACE
    # nothing asked for: nothing launched
    assert bwd(x=None, dx=None, dwgu=None, dwd=None, wgu=None) == OK


def test_binding_refuses_before_the_library(lib):
    cfg = train.MlpConfig(64, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(128, 64, dtype=torch.bfloat16)
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA"):
        train.moe_mlp_forward(cfg, x, w, w[:64], x, ws)
    with pytest.raises(TypeError, match="must be"):
        train.moe_mlp_forward(cfg, x.float(), w, w[:64], x, ws)
    with pytest.raises(TypeError, match="Act8"):
        train.moe_act_encode(x, x)
    with pytest.raises(ValueError, match="2-D"):
        train.moe_norm_forward(train.NormConfig(64), x[0], None, None, x, None, x)
    with pytest.raises(TypeError, match="gradients"):
        train.moe_mlp_backward(cfg, x, x, w, w, x, x, w.double(), w, ws)
    with pytest.raises(mf.MoeError):
        train.mlp_workspace(train.MlpConfig(60, 64), 4)
    with pytest.raises(mf.MoeError):
        train.norm_workspace(train.NormConfig(0), 4)
    for bad in (dict(act="relu"), dict(dtype=torch.int32)):
        with pytest.raises(KeyError):
            train.MlpConfig(64, 64, **bad)


# ------------------------------------------------------------------ the plain forms

@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_plain_norm_gradients(kind):
    g = ref.gen(3, "cpu")
    x, dy = (ref.normal(g, 5, 33, dtype=torch.float64) for _ in range(2))
    gain = ref.normal(g, 33, dtype=torch.float64)
    bias = ref.normal(g, 33, dtype=torch.float64) if kind == "layer" else None
    leaves = [t.clone().requires_grad_() for t in (x, gain)] + \
        ([bias.clone().requires_grad_()] if bias is not None else [])

    def f(x, gain, bias=None):
        return ref.norm_forward(x, gain, bias, kind, 1e-6)[0]

    (f(*leaves) * dy).sum().backward()
    _, mean, rstd = ref.norm_forward(x, gain, bias, kind, 1e-6)
    got = ref.norm_backward(x, gain, mean, rstd, dy, kind)
    for a, t in zip(got, leaves):
        assert torch.allclose(a, t.grad, rtol=1e-10, atol=1e-12)
    h = 1e-6  # against differences
    d = torch.zeros_like(x)
    d[2, 7] = h
    num = ((f(x + d, gain, bias) - f(x - d, gain, bias)) * dy).sum() / (2 * h)
    assert abs(float(num - got[0][2, 7])) < 1e-7


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_plain_mlp_gradients(act):
    g = ref.gen(4, "cpu")
    x, wgu, wd, dy = (ref.normal(g, *s, dtype=torch.float64)
                      for s in ((6, 16), (40, 16), (16, 20), (6, 16)))
    leaves = [t.clone().requires_grad_() for t in (x, wgu, wd)]
    y, gu = ref.mlp_forward(*leaves, act)
    (y * dy).sum().backward()
    got = ref.mlp_backward(x, gu.detach(), wgu, wd, dy, act)
    for a, t in zip(got, leaves):
        assert torch.allclose(a, t.grad, rtol=1e-10, atol=1e-12)
    h = 1e-6
    d = torch.zeros_like(wgu)
    d[25, 3] = h
    num = ((ref.mlp_forward(x, wgu + d, wd, act)[0] - ref.mlp_forward(x, wgu - d, wd, act)[0]) *
           dy).sum() / (2 * h)
    assert abs(float(num - got[1][25, 3])) < 1e-6


def test_plain_codes_are_the_nearest():
    """The checkpoint's plain form: smallest fitting power of two, nearest code."""
    g = ref.gen(5, "cpu")
    v = ref.normal(g, 7, 45, dtype=torch.float64) * torch.exp2(
        torch.randint(-20, 20, (7, 1), generator=g).double())
    v[3, :32] = 0
    for fmt, top in (("int8", 127.0), ("e4m3", 448.0)):
        q, b = ref.codes8(v, fmt)
        grid = torch.arange(-127.0, 128.0, dtype=torch.float64) if fmt == "int8" else \
            torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().double()
        grid = grid[torch.isfinite(grid)]
        for r in range(7):
            for lo in (0, 32):
                w = v[r, lo:lo + 32]
                k = int(b[r, lo // 32]) - 127
                assert w.abs().max() <= top * 2.0 ** k
                assert k == -126 or w.abs().max() > top * 2.0 ** (k - 1)
                best = (w[:, None] / 2.0 ** k - grid).abs().amin(1)
                assert torch.equal((w / 2.0 ** k - q[r, lo:lo + 32]).abs(), best)
