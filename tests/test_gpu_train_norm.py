"""RMS and layer norm, forward and backward, against plain 64-bit forms."""
import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import train
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    train._lib()


class Case:
    def __init__(self, T, n, kind="rms", dtype=torch.bfloat16, pdtype=None, bias=True, keep=None,
                 pad=0, seed=1, spread=True, gain=True):
        g = ref.gen(seed)
        pdtype = pdtype or dtype
        self.T, self.n, self.kind = T, n, kind
        self.cfg = train.NormConfig(cols=n, kind=kind, dtype=dtype, param_dtype=pdtype)
        s = 1 + 4 * (torch.rand(n, generator=g, device="cuda") < 0.05) if spread else 1.0
        self.x, _ = ref.padded((ref.normal(g, T, n) * s + 0.5).to(dtype), pad)
        self.dy, _ = ref.padded(ref.normal(g, T, n, dtype=dtype), pad)
        self.gain = (torch.rand(n, generator=g, device="cuda") + 0.5).to(pdtype) if gain else None
        self.bias = ref.normal(g, n, dtype=pdtype) if bias and kind == "layer" else None
        self.y, self.ybase = ref.padded(torch.zeros_like(self.x), pad)
        self.dx, self.dxbase = ref.padded(torch.zeros_like(self.x), pad)
        f32 = dict(dtype=torch.float32, device="cuda")
        self.rstd = torch.empty(T, **f32)
        self.mean = torch.empty(T, **f32) if kind == "layer" else None
        self.d_gain = torch.full((n,), 3.0, **f32)
        self.d_bias = torch.full((n,), 5.0, **f32) if kind == "layer" else None
        self.kept = train.act8(T, n, keep) if keep else None
        self.ws = train.norm_workspace(self.cfg, T)

    def run(self, accumulate=False):
        train.moe_norm_forward(self.cfg, self.x, self.gain, self.bias, self.y, self.mean,
                               self.rstd, kept=self.kept)
        train.moe_norm_backward(self.cfg, self.kept or self.x, self.gain, self.mean, self.rstd,
                                self.dy, self.dx, self.d_gain, self.d_bias, self.ws,
                                accumulate=accumulate)
        return self

    def check(self, base=0.0):
        """A row's sums run through at most 32 additions in a thread, 5 shuffles and 16 warps,
        so a mean of terms is off by K 2^-24 of their mean magnitude with K = 64; a few such
        means meet in each output (4 K)."""
        x, dy = self.x.double(), self.dy.double()
        y, mean, rstd = ref.norm_forward(x, self.gain, self.bias, self.kind, self.cfg.eps)
        K = 64 * ref.U32
        g = 1.0 if self.gain is None else self.gain.double().abs()
        far = x.abs().mean(1, keepdim=True) * rstd[:, None]  # magnitude behind the mean, in z
        z = (x - mean[:, None]) * rstd[:, None]
        h = ref.half(self.x.dtype)
        tiny = 2.0 ** -25 if self.x.dtype == torch.float16 else 0.0  # half the smallest step
        fine = torch.finfo(torch.float32).tiny
        tol = h * y.abs() + 4 * K * (z.abs() + far) * g + tiny + fine
        if self.bias is not None:
            tol = tol + K * self.bias.double().abs()
        assert ((self.y.double() - y).abs() <= tol).all()
        assert ((self.rstd.double() - rstd).abs() <= 4 * K * rstd).all()
        if self.mean is not None:
            assert ((self.mean.double() - mean).abs() <= K * x.abs().mean(1) + fine).all()
        if self.kept is not None:
            fmt = "int8" if self.kept.codes.dtype == torch.int8 else "e4m3"
            q, b = ref.codes8(x, fmt)
            assert torch.equal(self.kept.scales, b)
            assert torch.equal(ref.code_values(self.kept.codes), q)
            x = ref.decode8(self.kept)
            z = (x - mean[:, None]) * rstd[:, None]
        dx, dg, db = ref.norm_backward(x, self.gain, mean, rstd, dy, self.kind)
        a = dy.abs() * g
        zz = z.abs() + far
        mag = a + zz * (a * zz).mean(1, keepdim=True) + a.mean(1, keepdim=True)
        tol = h * dx.abs() + 4 * K * rstd[:, None] * mag + tiny + fine
        assert ((self.dx.double() - dx).abs() <= tol).all()
        # sums over rows: a thread adds its rows one by one, then the CTAs' sums are added
        adds = min(self.T, 2048) + 64
        tol = (adds * ref.U32 + 4 * K) * (dy.abs() * zz).sum(0) + ref.U32 * abs(base) * 4
        assert ((self.d_gain.double() - base - dg).abs() <= tol).all()
        if self.d_bias is not None:
            tol = adds * ref.U32 * dy.abs().sum(0) + ref.U32 * abs(base) * 4
            assert ((self.d_bias.double() - base - db).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n", [(1, 1), (1, 2816), (2, 7), (5, 33), (3, 256), (37, 264),
                                 (1000, 96), (129, 1001), (300, 2816), (65, 4096), (9, 4100),
                                 (33, 6144), (4, 8192), (5, 8200), (7, 16384), (3, 16383)])
def test_norm(T, n, dtype, kind):
    Case(T, n, kind, dtype).run().check()


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("keep", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n", [(1, 5), (11, 40), (77, 2816), (40, 1001), (9, 6144), (3, 16384)])
def test_norm_from_a_checkpoint(T, n, dtype, keep, kind):
    Case(T, n, kind, dtype, keep=keep).run().check()


@pytest.mark.parametrize("T", [4097, 40000])
@pytest.mark.parametrize("n", [128, 1000])
def test_many_rows(T, n):
    Case(T, n, "layer", torch.bfloat16, keep="int8").run().check()


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_mixed_parameter_types_and_no_parameters(kind):
    Case(20, 264, kind, torch.bfloat16, pdtype=torch.float32).run().check()
    Case(20, 264, kind, torch.float32, pdtype=torch.float16).run().check()
    Case(20, 264, kind, torch.bfloat16, gain=False, bias=False).run().check()


@pytest.mark.parametrize("pad", [8, 3])
def test_strided_rows_leave_the_gaps(pad):
    c = Case(21, 264, "layer", pad=pad).run()
    c.check()
    for b in (c.ybase, c.dxbase):
        assert (b[:, 264:] == 7.0).all()


@pytest.mark.parametrize("T", [3, 500])
def test_accumulated_gradients(T):
    c = Case(T, 264, "layer")
    c.d_gain.fill_(2.0)
    c.d_bias.fill_(2.0)
    c.run(accumulate=True).check(base=2.0)


def test_gradients_not_asked_for_and_in_place():
    c = Case(50, 264, "layer").run()
    y, dx = c.y.clone(), c.dx.clone()
    x2, dy2 = c.x.clone(), c.dy.clone()
    train.moe_norm_forward(c.cfg, x2, c.gain, c.bias, x2, c.mean, c.rstd)
    assert torch.equal(x2, y)
    train.moe_norm_backward(c.cfg, c.x, c.gain, c.mean, c.rstd, dy2, dy2, None, None, c.ws)
    assert torch.equal(dy2, dx)
    only = torch.zeros_like(c.d_bias)
    train.moe_norm_backward(c.cfg, c.x, c.gain, c.mean, c.rstd, c.dy, c.dx, None, only, c.ws)
    assert torch.equal(only, c.d_bias)


def test_no_rows():
    c = Case(4, 264, "layer")
    e = torch.empty(0, 264, dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, dtype=torch.float32, device="cuda")
    train.moe_norm_forward(c.cfg, e, c.gain, c.bias, e, s, s)
    train.moe_norm_backward(c.cfg, e, c.gain, s, s, e, e, c.d_gain, c.d_bias, c.ws, accumulate=True)
    assert (c.d_gain == 3.0).all()
    train.moe_norm_backward(c.cfg, e, c.gain, s, s, e, e, c.d_gain, c.d_bias, c.ws)
    assert (c.d_gain == 0).all() and (c.d_bias == 0).all()


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_rows_of_one_value_and_non_finite_rows(kind):
    """Constant and zero rows (variance 0: rstd = eps^-1/2) are finite; an infinity or NaN
    stays in its own row of y and dx."""
    c = Case(12, 264, kind, torch.float32)
    c.x[0] = 0
    c.x[1] = 3.0
    c.run().check()
    c.x[2, 5], c.x[3, 7] = float("inf"), float("nan")
    c.run()
    keep = [i for i in range(12) if i not in (2, 3)]
    assert torch.isfinite(c.y[keep]).all() and torch.isfinite(c.dx[keep]).all()
    assert torch.isnan(c.y[3]).all() and torch.isnan(c.dx[3]).all()


def test_same_bits_every_time():
    a = Case(3001, 2816, "layer", keep="int8").run()
    first = [t.clone() for t in (a.y, a.dx, a.d_gain, a.d_bias, a.rstd)]
    for _ in range(3):
        a.run()
        for t, f in zip((a.y, a.dx, a.d_gain, a.d_bias, a.rstd), first):
            assert torch.equal(t, f)
    assert mf.moe_check_device_status(a.ws) == mf.MOE_OK
