"""Norms and gated MLPs whose tensors have more than 2^31 elements: the rows at the end, where
offsets pass 32 bits, and the gradients' sums, against plain 64-bit forms.  Only the last rows
are drawn; the others are zero and must give exactly what zero rows give."""
import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import train
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
TAIL = 200


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    train._lib()
    yield
    torch.cuda.empty_cache()


def with_tail(rows, cols, seed):
    t = torch.zeros(rows, cols, dtype=BF, device="cuda")
    t[-TAIL:] = ref.normal(ref.gen(seed), TAIL, cols, dtype=BF)
    return t


@pytest.mark.parametrize("kind,n,keep", [("rms", 16384, "int8"), ("layer", 16383, None)])
def test_norm(kind, n, keep):
    T = (1 << 31) // n + 1000
    cfg = train.NormConfig(cols=n, kind=kind)
    x, dy = with_tail(T, n, 1), with_tail(T, n, 2)
    assert x.numel() > 1 << 31
    gain = (torch.rand(n, generator=ref.gen(3), device="cuda") + 0.5).to(BF)
    y, dx = torch.ones_like(x), torch.ones_like(x)
    mean = torch.empty(T, device="cuda") if kind == "layer" else None
    rstd, d_gain = torch.empty(T, device="cuda"), torch.empty(n, device="cuda")
    kept = train.act8(T, n, keep) if keep else None
    train.moe_norm_forward(cfg, x, gain, None, y, mean, rstd, kept=kept)
    train.moe_norm_backward(cfg, kept or x, gain, mean, rstd, dy, dx, d_gain, None,
                            train.norm_workspace(cfg, T))
    for t in (y, dx):
        assert not t[:-TAIL].any()
    want, mu, r = ref.norm_forward(x[-TAIL:], gain, None, kind, cfg.eps)
    # one rounding of a value, at most half a step, unrelated to the others' (and fp32 sums)
    lim = ref.half(BF) + 1e-5
    assert ref.rel2(y[-TAIL:], want) <= lim
    assert ref.rel2(rstd[-TAIL:], r) <= 1e-5
    back = x[-TAIL:]
    if keep:
        assert (kept.scales[:-TAIL] == 1).all() and not kept.codes[:-TAIL].any()
        back = ref.decode8(train.Act8(kept.codes[-TAIL:], kept.scales[-TAIL:]))
    wdx, wdg, _ = ref.norm_backward(back, gain, mu, r, dy[-TAIL:], kind)
    assert ref.rel2(dx[-TAIL:], wdx) <= lim
    assert ref.rel2(d_gain, wdg) <= 1e-5


@pytest.mark.parametrize("H,D,keep", [(16384, 8, "int8"), (8, 16384, "16"), (8, 16384, "e4m3")])
def test_mlp(H, D, keep):
    """x, y, dy and dx (H = 16384), or the pre-activations and the workspace's rows (D)."""
    T = (1 << 31) // max(H, 2 * D if D > H else H) + 1000
    cfg = train.MlpConfig(H, D)
    x, dy = with_tail(T, H, 4), with_tail(T, H, 5)
    g = ref.gen(6)
    wgu = ref.normal(g, 2 * D, H, std=1.5 / H ** 0.5, dtype=BF)
    wd = ref.normal(g, H, D, std=1.5 / D ** 0.5, dtype=BF)
    y, dx = torch.ones_like(x), torch.ones_like(x)
    gu = torch.ones(T, 2 * D, dtype=BF, device="cuda") if keep == "16" else \
        train.act8(T, D, keep, parts=2)
    assert max(x.numel(), T * 2 * D) > 1 << 31
    kx = x if keep == "16" else train.act8(T, H, keep)
    dwgu, dwd = torch.empty_like(wgu), torch.empty_like(wd)
    ws = train.mlp_workspace(cfg, T)
    train.moe_mlp_forward(cfg, x, wgu, wd, y, ws, kept_gu=gu)
    if kx is not x:
        train.moe_act_encode(x, kx)
    train.moe_mlp_backward(cfg, kx, gu, wgu, wd, dy, dx, dwgu, dwd, ws)
    assert mf.moe_check_device_status(ws) == mf.MOE_OK
    for t in (y, dx):
        assert not t[:-TAIL].any()
    # h and y, or dg, du, h and the results: two roundings, as in the tests of smaller sizes
    lim = 2 ** 0.5 * ref.half(BF) + 1e-5
    want, pre = ref.mlp_forward(x[-TAIL:], wgu, wd, cfg.act)
    assert ref.rel2(y[-TAIL:], want) <= lim
    back = x[-TAIL:]
    if keep == "16":
        assert not gu[:-TAIL].any()
        assert ref.rel2(gu[-TAIL:], pre) <= ref.half(BF) + 1e-5
        kgu = gu[-TAIL:]
    else:
        kgu = ref.decode8(train.Act8(gu.codes[-TAIL:], gu.scales[-TAIL:], 2))
        back = ref.decode8(train.Act8(kx.codes[-TAIL:], kx.scales[-TAIL:]))
        assert not gu.codes[:-TAIL].any()
    for got, w in zip((dx[-TAIL:], dwgu, dwd),
                      ref.mlp_backward(back, kgu, wgu, wd, dy[-TAIL:], cfg.act)):
        assert ref.rel2(got, w) <= lim
