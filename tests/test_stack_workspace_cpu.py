"""The stack's workspace holds every chunk that a prompt may end with."""
import ctypes

import pytest

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import build as mbuild

FAKE = 1 << 20  # an aligned address that is never dereferenced


@pytest.fixture(scope="module")
def lib():
    mbuild.build()
    return mf.lib()


@pytest.mark.parametrize("flag", [None, "int8", "fp8", "nvfp4"])
@pytest.mark.parametrize("H,E,k,I,D", [(128, 16, 1, 16384, 128), (256, 4, 4, 128, 16384),
                                       (2816, 128, 8, 704, 2112)])
def test_every_last_chunk_fits(lib, H, E, k, I, D, flag):
    cfg = mf.Config(H, E, k, I, D, **({flag: True} if flag else {}))
    c = 1024
    size = lib.moe_stack_workspace_size(ctypes.byref(cfg.c()), c)
    most = max(mf.workspace_size(cfg, T) for T in range(1, c + 1))
    assert size >= most + 2 * c * H * 2
    arr = (mf.CBlockWeights * 1)()
    for rest in (1, 17, 128, 256, 888, 1023):  # refused for the weights (none), not the space
        st = lib.moe_stack_forward(ctypes.byref(cfg.c()), c + rest, FAKE, arr, 1, FAKE, c, FAKE,
                                   size, None)
        assert st == mf.MOE_ERR_INVALID_ARG
        need = max(mf.workspace_size(cfg, T) for T in (c, rest)) + 2 * c * H * 2
        st = lib.moe_stack_forward(ctypes.byref(cfg.c()), c + rest, FAKE, arr, 1, FAKE, c, FAKE,
                                   need - 1, None)
        assert st == mf.MOE_ERR_WORKSPACE
