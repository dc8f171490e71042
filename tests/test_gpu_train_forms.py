"""Every form of every launch of the gated MLP (the CPU tests hold that the sizes reach them all),
each with every epilogue that it has: gradients in 16 bits and in fp32, written and added to what
the buffers hold, with dx in the same launch and without, against plain 64-bit forms."""
import pytest
import torch

from mixture_experts_ffn_05_b200 import train
from tests import train_forms
from tests.test_gpu_train_mlp import Case

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    train._lib()


@pytest.mark.parametrize("act,dtype,keep", [("gelu_tanh", BF, "16"), ("silu", HF, "e4m3")])
@pytest.mark.parametrize("T,H,D", train_forms.SIZES)
def test_forward(T, H, D, act, dtype, keep):
    Case(T, H, D, act, dtype, keep, seed=T).forward().check_forward()


@pytest.mark.parametrize("grad", ["16", "fp32"])
@pytest.mark.parametrize("act,dtype,keep", [("silu", BF, "int8"), ("gelu_tanh", HF, "16")])
@pytest.mark.parametrize("T,H,D", train_forms.SIZES)
def test_gradients(T, H, D, act, dtype, keep, grad):
    c = Case(T, H, D, act, dtype, keep, seed=T + 1, grad=F32 if grad == "fp32" else dtype).forward()
    c.backward(accumulate=True).check_backward(base=2.0)  # the buffers hold 2
    c.backward().check_backward()
    for t in (c.dwgu, c.dwd):
        t.fill_(2.0)
    c.backward(dx=None, accumulate=True).check_backward(base=2.0, what=("dwgu", "dwd"))
    c.backward(dx=None).check_backward(what=("dwgu", "dwd"))
    c.dwd.fill_(2.0)  # one gradient alone
    c.backward(dx=None, dw_gate_up=None, accumulate=True).check_backward(base=2.0, what=("dwd",))
