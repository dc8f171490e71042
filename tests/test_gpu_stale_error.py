"""A call reports its own launch: an error that an earlier call left on the thread (and reported)
does not make a later one fail."""
import ctypes

import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import train

pytestmark = pytest.mark.gpu


def cuda_runtime():
    with open("/proc/self/maps") as f:
        path = next(l.split()[-1] for l in f if "libcudart.so" in l)
    return ctypes.CDLL(path)


def leave_an_error(ws):
    """A refused call: the status word cannot be waited for on a stream that is being captured
    (the capture becomes invalid and is dropped; nothing of it runs)."""
    rt = cuda_runtime()
    s = ctypes.c_void_p(torch.cuda.Stream().cuda_stream)
    assert rt.cudaStreamBeginCapture(s, 2) == 0  # relaxed mode
    assert mf.lib().moe_check_device_status(ws.data_ptr(), ws.numel(), s) == mf.MOE_ERR_CUDA
    graph = ctypes.c_void_p()
    assert rt.cudaStreamEndCapture(s, ctypes.byref(graph)) != 0
    rt.cudaGetLastError()  # torch's runtime keeps an error of its own


def test_calls_after_a_refused_one():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    ws = torch.zeros(4096, dtype=torch.uint8, device="cuda")
    x = torch.randn(64, 64, device="cuda").bfloat16()
    kept, back = train.act8(64, 64), torch.empty_like(x)
    q8, s8 = torch.empty(64, 64, dtype=torch.uint8, device="cuda"), torch.empty(64, device="cuda")
    qi = torch.empty(64, 64, dtype=torch.int8, device="cuda")
    q4, b4 = (torch.empty(1, 64, n, dtype=torch.uint8, device="cuda") for n in (32, 4))
    t4 = torch.empty(1, device="cuda")
    torch.cuda.synchronize()
    for call in (lambda: train.moe_act_encode(x, kept), lambda: train.moe_act_decode(kept, back),
                 lambda: mf.moe_quantize_int8(x, qi, s8), lambda: mf.moe_quantize_fp8(x, q8, s8),
                 lambda: mf.moe_quantize_nvfp4(x[None], q4, b4, t4)):
        leave_an_error(ws)
        call()
    torch.cuda.synchronize()
    assert (back.float() - x.float()).abs().max() <= x.float().abs().max() / 127
