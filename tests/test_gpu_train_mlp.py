"""The gated MLP's forward and backward passes against plain 64-bit forms."""
import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import train
from tests import train_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    train._lib()


class Case:
    """keep: None, "16", "int8" or "e4m3" (x and the pre-activations both)."""

    def __init__(self, T, H, D, act="gelu_tanh", dtype=torch.bfloat16, keep="16", pad=0, seed=1,
                 grad=None):
        g = ref.gen(seed)
        self.T, self.H, self.D, self.act, self.dtype = T, H, D, act, dtype
        self.cfg = train.MlpConfig(H, D, act, dtype)
        self.x, _ = ref.padded(ref.normal(g, T, H, dtype=dtype), pad)
        self.dy, _ = ref.padded(ref.normal(g, T, H, dtype=dtype), pad)
        self.wgu = ref.normal(g, 2 * D, H, std=1.5 / H ** 0.5, dtype=dtype)
        self.wd = ref.normal(g, H, D, std=1.5 / D ** 0.5, dtype=dtype)
        self.y, self.ybase = ref.padded(torch.zeros_like(self.x), pad)
        self.dx, self.dxbase = ref.padded(torch.zeros_like(self.x), pad)
        self.gubase = None
        if keep == "16":
            self.gu, self.gubase = ref.padded(
                torch.zeros(T, 2 * D, dtype=dtype, device="cuda"), pad)
        else:
            self.gu = train.act8(T, D, keep, parts=2) if keep else None
        self.kx = train.act8(T, H, keep) if keep in ("int8", "e4m3") else self.x
        grad = grad or dtype
        self.dwgu = torch.full((2 * D, H), 2.0, dtype=grad, device="cuda")
        self.dwd = torch.full((H, D), 2.0, dtype=grad, device="cuda")
        self.ws = train.mlp_workspace(self.cfg, T)

    def forward(self):
        train.moe_mlp_forward(self.cfg, self.x, self.wgu, self.wd, self.y, self.ws,
                              kept_gu=self.gu)
        if self.kx is not self.x:
            train.moe_act_encode(self.x, self.kx)
        return self

    def backward(self, **kw):
        a = dict(dx=self.dx, dw_gate_up=self.dwgu, dw_down=self.dwd)
        a.update(kw)
        train.moe_mlp_backward(self.cfg, self.kx, self.gu, self.wgu, self.wd, self.dy, a.pop("dx"),
                               a.pop("dw_gate_up"), a.pop("dw_down"), self.ws, **a)
        return self

    def check_forward(self):
        """y: one rounding of h and one of y, so sqrt(2) half steps in the 2-norm (a rounding's
        error is at most half a step and unrelated to the others), and per element at most
        half a step of y and of every h that enters it.  fp32 sums add 64 2^-24 of their
        terms."""
        assert mf.moe_check_device_status(self.ws) == mf.MOE_OK
        y, gu = ref.mlp_forward(self.x, self.wgu, self.wd, self.act)
        g, u = gu.chunk(2, dim=1)
        h = half = ref.half(self.dtype)
        assert torch.isfinite(self.y).all()
        assert ref.rel2(self.y, y) <= 2 ** 0.5 * half + 1e-5
        mid = (ref.gate(g, self.act)[0] * u).abs() @ self.wd.double().abs().t()
        noise = 64 * ref.U32 * (self.x.double().abs() @ self.wgu.double().abs().t())
        gn, un = noise.chunk(2, dim=1)
        # a gate is at most 1.13 |g| steep; act(g) at most |g|
        mid32 = (1.13 * gn * u.abs() + un * g.abs()) @ self.wd.double().abs().t()
        tiny = 2.0 ** -24 * (1 + self.wd.double().abs().sum(1)) if self.dtype == torch.float16 else 0
        tol = half * y.abs() + (h + 64 * ref.U32) * 1.01 * mid + 1.01 * mid32 + tiny
        assert ((self.y.double() - y).abs() <= tol).all()
        if self.gu is None:
            return
        if isinstance(self.gu, torch.Tensor):
            tol = half * gu.abs() + noise + (2.0 ** -25 if self.dtype == torch.float16 else 0)
            assert ((self.gu.double() - gu).abs() <= tol).all()
            return
        # 8 bits: half a code step of the checkpoint's own scale, which is the smallest fitting
        # one wherever the group's maximum is not next to a border
        fmt = "int8" if self.gu.codes.dtype == torch.int8 else "e4m3"
        got, n = ref.decode8(self.gu), -(-self.D // ref.GROUP)
        for p, (v, nz) in enumerate(((g, gn), (u, un))):
            byte = self.gu.scales[:, p * n:(p + 1) * n].long()
            s = torch.ldexp(torch.ones_like(byte, dtype=torch.float64), byte - 127)
            s = s.repeat_interleave(ref.GROUP, dim=1)[:, : self.D]
            step = s if fmt == "int8" else \
                torch.maximum(s * 2.0 ** -9, v.abs() * 2.0 ** -3)  # at most |v| / 8 a step
            assert ((got[:, p * self.D:(p + 1) * self.D] - v).abs() <= step / 2 + 2 * nz).all()
            k = ref.scales8(v, fmt)[0]
            near = sum((ref.scales8(v * f, fmt)[0] != k) for f in (1 - 1e-4, 1 + 1e-4)) > 0
            assert torch.equal(byte[~near], (k + 127)[~near])

    def check_backward(self, base=0.0, what=("dx", "dwgu", "dwd")):
        """From what was kept: dg, du and h are rounded once, the results once, so sqrt(2) half
        steps in the 2-norm.  A 16-bit gradient that accumulates is rounded on top of base."""
        assert mf.moe_check_device_status(self.ws) == mf.MOE_OK
        x = self.kx if isinstance(self.kx, torch.Tensor) else ref.decode8(self.kx)
        gu = self.gu if isinstance(self.gu, torch.Tensor) else ref.decode8(self.gu)
        want = ref.mlp_backward(x, gu, self.wgu, self.wd, self.dy, self.act)
        half = ref.half(self.dtype)
        for name, w in zip(("dx", "dwgu", "dwd"), want):
            if name not in what:
                continue
            got = getattr(self, name)
            b = base if name != "dx" else 0.0
            assert torch.isfinite(got).all(), name
            tol = 2 ** 0.5 * half + 1e-5
            if b and got.dtype != torch.float32:
                tol = half * (1 + float((w + b).norm() / w.norm()))
            elif b:
                tol += ref.U32 * float((w + b).norm() / w.norm())
            assert ref.rel2(got.double() - b, w) <= tol, name
        return self


SIZES = [(1, 8, 8), (1, 2816, 2112), (2, 64, 64), (7, 72, 40), (33, 264, 136), (128, 128, 128),
         (129, 512, 384), (300, 1000, 1352), (257, 2816, 2112), (515, 136, 2056), (1000, 512, 384),
         (2049, 264, 200)]


@pytest.mark.parametrize("act,dtype", [("gelu_tanh", torch.bfloat16), ("silu", torch.float16)])
@pytest.mark.parametrize("keep", [None, "16", "int8", "e4m3"])
@pytest.mark.parametrize("T,H,D", SIZES)
def test_forward(T, H, D, keep, act, dtype):
    Case(T, H, D, act, dtype, keep).forward().check_forward()


@pytest.mark.parametrize("act,dtype", [("silu", torch.bfloat16), ("gelu_tanh", torch.float16)])
@pytest.mark.parametrize("keep", ["16", "int8", "e4m3"])
@pytest.mark.parametrize("T,H,D", SIZES)
def test_backward(T, H, D, keep, act, dtype):
    Case(T, H, D, act, dtype, keep, seed=2).forward().backward().check_backward()


@pytest.mark.parametrize("T", [5000, 16384])
def test_long_batches(T):
    c = Case(T, 512, 384, keep="int8", seed=3).forward()
    c.check_forward()
    c.backward().check_backward()


@pytest.mark.parametrize("keep", ["16", "int8"])
def test_the_widest_sizes(keep):
    c = Case(40, 16384, 64, keep=keep).forward()
    c.check_forward()
    c.backward().check_backward()
    c = Case(40, 64, 16384, keep=keep).forward()
    c.check_forward()
    c.backward().check_backward()


@pytest.mark.parametrize("T", [9, 700])
def test_strided_rows_leave_the_gaps(T):
    c = Case(T, 264, 136, pad=8).forward()
    c.check_forward()
    c.backward().check_backward()
    for b, n in ((c.ybase, 264), (c.dxbase, 264), (c.gubase, 272)):
        assert (b[:, n:] == 7.0).all()


@pytest.mark.parametrize("T", [5, 600])
@pytest.mark.parametrize("grad", [torch.bfloat16, torch.float32])
def test_accumulated_gradients(T, grad):
    c = Case(T, 264, 136, grad=grad).forward().backward(accumulate=True)
    c.check_backward(base=2.0)
    c.backward()  # overwritten, not added to
    c.check_backward()


@pytest.mark.parametrize("T", [5, 600])
def test_gradients_not_asked_for(T):
    c = Case(T, 264, 136).forward().backward()
    full = [t.clone() for t in (c.dx, c.dwgu, c.dwd)]
    for skip in range(3):
        names = ("dx", "dw_gate_up", "dw_down")
        bufs = [torch.zeros_like(t) for t in full]
        c.backward(**{n: None if i == skip else bufs[i] for i, n in enumerate(names)})
        for i in range(3):
            if i != skip:
                assert torch.equal(bufs[i], full[i])


def test_no_tokens():
    c = Case(3, 64, 64)
    e = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    gu = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    train.moe_mlp_forward(c.cfg, e, c.wgu, c.wd, e, c.ws)
    train.moe_mlp_backward(c.cfg, e, gu, c.wgu, c.wd, e, e, c.dwgu, c.dwd, c.ws, accumulate=True)
    assert (c.dwgu == 2).all() and (c.dwd == 2).all()
    train.moe_mlp_backward(c.cfg, e, gu, c.wgu, c.wd, e, e, c.dwgu, c.dwd, c.ws)
    assert (c.dwgu == 0).all() and (c.dwd == 0).all()


@pytest.mark.parametrize("act", ["gelu_tanh", "silu"])
def test_large_pre_activations_are_finite(act):
    """Gates far outside exp's range: act and its derivative go to 0 or to the identity."""
    c = Case(40, 64, 64, act, keep="16").forward()
    vals = torch.tensor([-1e30, -3e4, -300.0, -90.0, -20.0, 20.0, 90.0, 300.0, 3e4, 1e30],
                        device="cuda").to(torch.bfloat16)
    c.gu[:, :60] = vals.repeat(6)
    c.dy.mul_(1e-3)
    c.backward()
    gu = c.gu.double()
    # the formulas with the gates' limits (a' of the plain form meets 0 * inf there)
    big = gu[:, :64].abs() > 16
    cap = gu.clone()
    cap[:, :64] = torch.where(big, gu[:, :64].clamp(-600, 600), gu[:, :64])
    a, da = ref.gate(cap[:, :64], act)
    a = torch.where(big, gu[:, :64].clamp_min(0) if act == "gelu_tanh" else a, a)
    a = torch.where(gu[:, :64] > 600, gu[:, :64], torch.where(gu[:, :64] < -600, 0.0, a))
    dh = c.dy.double() @ c.wd.double()
    dgu = torch.cat((dh * gu[:, 64:] * da, dh * a), dim=1)
    assert torch.isfinite(c.dx).all() and torch.isfinite(c.dwgu).all()
    assert ref.rel2(c.dx, dgu @ c.wgu.double()) <= 2 ** 0.5 * ref.half(torch.bfloat16) + 1e-5


def test_non_finite_rows_stay_in_their_rows():
    c = Case(200, 72, 40, keep="int8")
    c.x[17, 3] = float("inf")
    c.x[190, 0] = float("nan")
    c.forward().backward()
    rows = [i for i in range(200) if i not in (17, 190)]
    assert torch.isfinite(c.y[rows]).all() and torch.isfinite(c.dx[rows]).all()
    assert torch.isnan(c.y[190]).all() and torch.isnan(c.dx[190]).all()
    assert torch.isnan(c.dwgu).any()


def test_same_bits_every_time():
    c = Case(777, 512, 384, keep="e4m3").forward().backward()
    first = [t.clone() for t in (c.y, c.dx, c.dwgu, c.dwd, c.gu.codes, c.gu.scales)]
    for _ in range(3):
        c.forward().backward()
        for t, f in zip((c.y, c.dx, c.dwgu, c.dwd, c.gu.codes, c.gu.scales), first):
            assert torch.equal(t, f)


def test_one_row_agrees_with_the_inference_mlp():
    """The block's own dense MLP and this one on the same tokens: both within their rounding
    of the same definition."""
    T, H, D = 5, 512, 384
    c = Case(T, H, D, keep=None).forward()
    cfg = mf.Config(hidden=H, num_experts=16, top_k=4, expert_inter=128, dense_inter=D)
    out = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    mf.dense_mlp_forward(cfg, c.x.contiguous(), c.wgu, c.wd, out, mf.workspace(cfg, T))
    assert ref.rel2(c.y, out.double()) <= 2 * 2 ** 0.5 * ref.half(torch.bfloat16)
