"""Calls whose tensors are not on the current device are refused before the library is reached
(its kernels run on the current device and would not find the tensors' memory there)."""
import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import build as mbuild

BF, I32, F32, U8 = torch.bfloat16, torch.int32, torch.float32, torch.uint8


class Elsewhere(torch.Tensor):
    """A tensor that says it is on cuda:1."""
    is_cuda = True
    device = torch.device("cuda", 1)

    def get_device(self):
        return 1


def t(dtype, *shape):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Elsewhere)


CFG = mf.Config(hidden=512, num_experts=16, top_k=4, expert_inter=128, dense_inter=384)


def calls():
    x, ws = t(BF, 8, 512), t(U8, 4096)
    idx, off, srt = t(I32, 8, 4), t(I32, 17), t(I32, 32)
    w = mf.BlockWeights(CFG, {n: t(BF, 8) for n in mf.BlockWeights.NAMES + ("w_gate_up", "w_down")
                              if n != "logit_bias"})
    e = {"w_gate_up": t(BF, 8), "w_down": t(BF, 8)}
    g = t(BF, 512)
    return {
        "moe_router": lambda: mf.moe_router(CFG, x, g, g, None, g, g, g, idx, t(F32, 8, 4), x, x, ws),
        "moe_permute": lambda: mf.moe_permute(CFG, idx, off, srt, srt, ws),
        "moe_permute_noalloc": lambda: mf.moe_permute_noalloc(CFG, idx, off, srt, srt),
        "moe_ffn_forward": lambda: mf.moe_ffn_forward(CFG, x, t(F32, 8, 4), off, srt, srt, e, x, ws),
        "dense_mlp_forward": lambda: mf.dense_mlp_forward(CFG, x, g, g, x, ws),
        "moe_block_forward": lambda: mf.moe_block_forward(CFG, x, w, x, ws),
        "moe_stack_forward": lambda: mf.moe_stack_forward(CFG, x, [w], x, ws),
        "moe_quantize_int8": lambda: mf.moe_quantize_int8(x, t(torch.int8, 8, 512), t(F32, 8)),
        "moe_quantize_fp8": lambda: mf.moe_quantize_fp8(x, t(U8, 8, 512), t(F32, 8)),
        "moe_quantize_nvfp4": lambda: mf.moe_quantize_nvfp4(x, t(U8, 8, 256), t(U8, 8, 32), t(F32, 1)),
        "moe_wait_selftest": lambda: mf.moe_wait_selftest(ws, 10000),
    }


@pytest.mark.parametrize("name", sorted(calls()))
def test_tensors_of_another_device_are_refused(name, monkeypatch):
    mbuild.build()
    monkeypatch.setattr(mf, "_current_device", lambda: 0)
    reached = []
    monkeypatch.setattr(mf, "lib", lambda: type("L", (), {"__getattr__": lambda s, n: (
        lambda *a: reached.append(n))})())
    with pytest.raises(ValueError, match="the current device is cuda:0"):
        calls()[name]()
    assert not reached


def test_the_status_is_read_on_the_workspaces_device(monkeypatch):
    """Training calls run on their tensors' device, whichever is current; so does this."""
    at = [0]

    class Device:
        def __init__(self, i):
            self.i = i

        def __enter__(self):
            at.append(self.i)

        def __exit__(self, *a):
            at.pop()

    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(mf, "_current_device", lambda: at[-1])
    monkeypatch.setattr(torch.cuda, "current_stream", lambda: type("S", (), {"cuda_stream": at[-1]})())
    seen = []
    monkeypatch.setattr(mf, "lib", lambda: type("L", (), {
        "moe_check_device_status": staticmethod(lambda *a: seen.append((at[-1], a[2])) or 0)}))
    assert mf.moe_check_device_status(t(U8, 4096)) == 0
    assert seen == [(1, 1)] and at == [0]
