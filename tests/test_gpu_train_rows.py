"""Norms and 8-bit checkpoints over more rows than the GPU holds at one time: every width of a
thread's share, rings that go round, teams that share a CTA, rows that no 16-byte access fits."""
import pytest
import torch

from mixture_experts_ffn_05_b200 import train
from tests import train_ref as ref
from tests.test_gpu_train_norm import Case

pytestmark = pytest.mark.gpu
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    train._lib()


@pytest.mark.parametrize("kind,keep", [("rms", None), ("layer", None), ("rms", "int8"),
                                       ("layer", "e4m3")])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("T,n", [(20011, 31), (20000, 256), (6001, 700), (6001, 1001),
                                 (6000, 2816), (6001, 2819), (3000, 4104), (3001, 6144),
                                 (1003, 6145), (700, 12288), (601, 13000), (600, 16384)])
def test_norm(T, n, dtype, kind, keep):
    Case(T, n, kind, dtype, keep=keep, seed=n).run().check()


@pytest.mark.parametrize("T", [149, 296, 297, 1777])
@pytest.mark.parametrize("n,pad", [(264, 8), (2817, 3), (1000, 1)])
def test_norm_rows_apart(T, n, pad):
    c = Case(T, n, "layer", keep="int8", pad=pad, seed=T)
    c.run().check()
    for b in (c.ybase, c.dxbase):
        assert (b[:, n:] == 7.0).all()


def test_norm_in_place_over_many_rows():
    for n in (1001, 2816):  # rows share their 16-byte pieces with their neighbours, or not
        c = Case(5003, n, "rms", torch.float16, seed=n).run()
        x, dy = c.x.clone(), c.dy.clone()
        train.moe_norm_forward(c.cfg, x, c.gain, None, x, None, c.rstd)
        assert torch.equal(x, c.y)
        train.moe_norm_backward(c.cfg, c.x, c.gain, None, c.rstd, dy, dy, c.d_gain, None, c.ws)
        assert torch.equal(dy, c.dx)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,cols,pad", [(70001, 40, 0), (50000, 64, 0), (9000, 1000, 8),
                                           (9001, 1001, 0), (3001, 4224, 0), (400, 65528, 0)])
def test_checkpoint(rows, cols, pad, dtype, fmt):
    g = ref.gen(cols)
    x, _ = ref.padded(ref.normal(g, rows, cols, dtype=dtype), pad)
    kept = train.act8(rows, cols, fmt)
    train.moe_act_encode(x, kept)
    q, b = ref.codes8(x, fmt)
    assert torch.equal(kept.scales, b)
    assert torch.equal(ref.code_values(kept.codes), q)
    back, base = ref.padded(torch.zeros_like(x), pad)
    train.moe_act_decode(kept, back)
    assert torch.equal(back, ref.decode8(kept).to(dtype))
    assert (base[:, cols:] == 7.0).all()
