"""The gated MLP at sizes for which every tiling of its products is chosen in turn (CTA pairs,
128 x 128, 128 x 64, and few-token tiles split 1, 2, 4 and 8 ways), with rows, columns and K
that no tile divides, in every kept format: against plain 64-bit forms."""
import pytest
import torch

from mixture_experts_ffn_05_b200 import train
from tests.test_gpu_train_mlp import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    train._lib()


SIZES = [(1, 72, 8), (1, 200, 8), (3, 328, 16), (21, 680, 264), (31, 1240, 136), (69, 776, 88),
         (48, 72, 1416), (303, 2488, 48), (327, 1368, 8), (438, 2408, 712), (734, 2456, 1496),
         (704, 960, 824), (2453, 8, 1432), (3149, 440, 152), (2248, 744, 1024), (3537, 1152, 608),
         (4769, 1392, 104), (7056, 128, 120), (7049, 792, 1376)]


@pytest.mark.parametrize("keep,act,dtype", [("16", "gelu_tanh", torch.bfloat16),
                                            ("int8", "silu", torch.bfloat16),
                                            ("e4m3", "gelu_tanh", torch.float16)])
@pytest.mark.parametrize("T,H,D", SIZES)
def test_step(T, H, D, keep, act, dtype):
    c = Case(T, H, D, act, dtype, keep, seed=T)
    c.forward().check_forward()
    c.backward().check_backward()


@pytest.mark.parametrize("T,H,D", [(48, 72, 1416), (438, 2408, 712), (3537, 1152, 608)])
def test_summed_gradients(T, H, D):
    """fp32 gradients added to what the buffers hold, on each tiling's own epilogue."""
    c = Case(T, H, D, grad=torch.float32, seed=T)
    c.forward()
    c.backward(accumulate=True).check_backward(base=2.0)


@pytest.mark.parametrize("T", [1, 60, 200, 1500])
def test_same_bits_every_time(T):
    c = Case(T, 1000, 1352, seed=T)
    c.forward().backward()
    first = [t.clone() for t in (c.y, c.gu, c.dx, c.dwgu, c.dwd)]
    for _ in range(3):
        c.forward().backward()
        for t, f in zip((c.y, c.gu, c.dx, c.dwgu, c.dwd), first):
            assert torch.equal(t, f)


def test_one_workspace_for_many_sizes():
    """Batches of every size in turn on the workspace of the largest, nothing left over."""
    H, D = 520, 392
    big = Case(3000, H, D)
    for T in (3000, 1, 128, 129, 700, 16, 2000, 5):
        c = Case(T, H, D, seed=T)
        c.ws = big.ws
        c.forward().check_forward()
        c.backward().check_backward()
