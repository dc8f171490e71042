"""8-bit checkpoints of the largest finite values: what was finite in 16 bits reads back finite,
and so do the gradients that are formed from it."""
import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import train
from tests import train_ref as ref
from tests.test_gpu_train_mlp import Case

pytestmark = pytest.mark.gpu
FMTS = ["int8", "e4m3"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    train._lib()


def read_back(x, fmt, dtype):
    kept = train.act8(*x.shape, fmt)
    train.moe_act_encode(x, kept)
    back = torch.empty(x.shape, dtype=dtype, device="cuda")
    train.moe_act_decode(kept, back)
    return kept, back


def nearest_finite(v, dtype):
    """v (double) rounded to dtype, at most its largest finite value."""
    top = torch.finfo(dtype).max
    return v.clamp(-top, top).to(dtype)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("cols", [72, 70])  # rows that 16-byte accesses fit, and others
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_largest_values_of_a_format(dtype, cols, fmt):
    """Every one of the format's highest values (down to an eighth of the largest), alone in its
    group and beside the others, and its negative."""
    top = torch.finfo(dtype).max
    bits = torch.tensor([top], dtype=dtype).view(torch.int16).item()
    step = 1 << (10 if dtype == torch.float16 else 7)  # values of one exponent
    high = torch.arange(bits - 3 * step, bits + 1, dtype=torch.int16).view(dtype)
    x = torch.zeros(2 * len(high) + 4, cols, dtype=dtype)
    x[:len(high), 3] = high
    x[len(high):2 * len(high), 40] = -high
    x[-4:] = high[-4 * cols:].reshape(4, cols)
    x = x.cuda()
    kept, back = read_back(x, fmt, dtype)
    q, b = ref.codes8(x, fmt)
    assert torch.equal(kept.scales, b) and torch.equal(ref.code_values(kept.codes), q)
    assert torch.isfinite(back).all()
    assert torch.equal(back, nearest_finite(ref.decode8(kept), dtype))
    # at most half a step of the codes: s / 2 (int8), 1/16 of the value (E4M3)
    s = torch.exp2(b.double() - 127).repeat_interleave(ref.GROUP, dim=1)[:, :cols]
    lim = s / 2 if fmt == "int8" else torch.maximum(x.double().abs() / 16, s * 2.0 ** -10)
    assert ((back.double() - x.double()).abs() <= lim).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("cols", [64, 33])
def test_values_past_the_largest(cols, fmt):
    """A wide checkpoint read into a narrower type: the largest finite value, and NaN for groups
    that held an infinity or NaN."""
    x = torch.zeros(6, cols, device="cuda")
    x[0, 1], x[1, 2], x[2, 3] = 1e5, -3e38, torch.finfo(torch.float32).max
    x[3, 4], x[4, 5] = float("inf"), float("nan")
    for dtype in (torch.float16, torch.bfloat16):
        kept, back = read_back(x, fmt, dtype)
        v = ref.decode8(kept)
        bad = torch.isnan(v)
        assert bad[3, :32].all() and bad[4, :32].all() and int(bad.sum()) == 64
        assert torch.equal(torch.isnan(back), bad)
        assert torch.equal(back[~bad], nearest_finite(v[~bad], dtype))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [40, 600])
def test_gradients_from_the_largest_inputs(T, fmt):
    """fp16: an input of 65504 whose weights are zero reaches the weights' gradient alone."""
    c = Case(T, 72, 40, "silu", torch.float16, keep=fmt, grad=torch.float32)
    c.x[3, 5], c.x[7, 5] = 65504.0, -65504.0
    c.wgu[:, 5] = 0
    c.forward().backward()
    assert mf.moe_check_device_status(c.ws) == mf.MOE_OK
    x = ref.decode8(c.kx).clamp(-65504.0, 65504.0)
    want = ref.mlp_backward(x, ref.decode8(c.gu), c.wgu, c.wd, c.dy, c.act)
    # dg and du are rounded once: half a step each, as in the other tests of the gradients
    for got, w in zip((c.dx, c.dwgu, c.dwd), want):
        assert torch.isfinite(got).all()
        assert ref.rel2(got, w) <= 2 ** 0.5 * ref.half(torch.float16) + 1e-5
