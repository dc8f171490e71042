"""Sizes at and past the limits of the training operators' interface, on the CPU: found on the
host, before anything is launched or touched."""
import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import build as mbuild
from mixture_experts_ffn_05_b200 import train

BF = torch.bfloat16
PAST = (1 << 32) + 4  # modulo 2^32: 4


@pytest.fixture()
def refused(monkeypatch):
    """Runs a call of the binding on CPU tensors through to the library, whose status must be
    `unsupported`."""
    mbuild.build()
    train._lib()

    def run(name, index, stream, *args):
        mf._check(name, getattr(train._lib(), name)(*args, None))

    monkeypatch.setattr(train, "_run", run)

    def check(call):
        with pytest.raises(mf.MoeError) as e:
            call()
        assert e.value.status == mf.MOE_ERR_UNSUPPORTED

    return check


def many(rows, cols, dtype=BF):
    """[rows][cols] for any number of rows, in the memory of one: the calls never read it."""
    return torch.empty(1, cols, dtype=dtype).expand(rows, cols)


def test_rows_past_32_bits_are_refused(refused, monkeypatch):
    """ctypes takes an int modulo 2^32, so such a call would do 4 rows and leave the others as
    they were."""
    ws = torch.zeros(4096, dtype=torch.uint8)
    stat = torch.empty(1).expand(PAST)
    ptr = train._ptr  # wants contiguous statistics, which would take 16 GB
    monkeypatch.setattr(train, "_ptr", lambda t, *a: t.data_ptr() if t is stat else ptr(t, *a))
    n, x = train.NormConfig(1), many(PAST, 1)
    refused(lambda: train.moe_norm_forward(n, x, None, None, x, None, stat))
    refused(lambda: train.moe_norm_backward(n, x, None, None, stat, x, x, None, None, ws))
    m, x, gu = train.MlpConfig(8, 8), many(PAST, 8), many(PAST, 16)
    w = torch.zeros(16, 8, dtype=BF)
    refused(lambda: train.moe_mlp_forward(m, x, w, w[:8], x, ws))
    refused(lambda: train.moe_mlp_backward(m, x, gu, w, w[:8], x, x, w, w[:8], ws))


def test_columns_past_32_bits_are_refused(refused, monkeypatch):
    """The same for a checkpoint's columns."""
    shape = torch.empty(1, 1, dtype=BF).expand(2, PAST)  # rows of no tensor that would fit here
    codes = torch.empty(1, 1, dtype=torch.int8).expand(2, PAST)
    kept = train.Act8(codes, torch.zeros(2, 1, dtype=torch.uint8))
    monkeypatch.setattr(train, "_act", lambda t, *a: train.CAct(
        1 << 20, 1 << 20 if isinstance(t, train.Act8) else None, PAST,
        train.F_INT8 if isinstance(t, train.Act8) else train.F_BF16))
    refused(lambda: train.moe_act_encode(shape, kept))
    refused(lambda: train.moe_act_decode(kept, shape))


@pytest.mark.parametrize("past", [PAST, (1 << 31), -(1 << 32) + 8, (1 << 32) + 64])
def test_workspaces_and_configurations_past_32_bits(past):
    mbuild.build()
    for f, c in ((train.norm_workspace, train.NormConfig(64)),
                 (train.mlp_workspace, train.MlpConfig(64, 64))):
        with pytest.raises(mf.MoeError):
            f(c, past, device="cpu")
    for f, c in ((train.norm_workspace, train.NormConfig(past)),
                 (train.mlp_workspace, train.MlpConfig(past, 64)),
                 (train.mlp_workspace, train.MlpConfig(64, past))):
        with pytest.raises(mf.MoeError):
            f(c, 4, device="cpu")


def test_the_most_rows():
    """2^31 - 512 rows, as the header says, and not one more (the tiles' rows stay int32)."""
    mbuild.build()
    most = (1 << 31) - 512
    l = train._lib()
    for f, c in ((l.moe_norm_workspace_size, train.NormConfig(8).c()),
                 (l.moe_mlp_workspace_size, train.MlpConfig(8, 8).c())):
        assert f(c, most) > 0 and f(c, most + 1) == 0
    act = train.CAct(1 << 20, None, 8, train.F_BF16)
    n, m = train.NormConfig(8).c(), train.MlpConfig(8, 8).c()
    ptr = 1 << 20
    # up to the limit it is the tensors (here: none) that are refused, past it the size
    for T, want in ((most, mf.MOE_ERR_INVALID_ARG), (most + 1, mf.MOE_ERR_UNSUPPORTED)):
        assert l.moe_norm_forward(n, T, None, None, None, act, None, ptr, None, None) == want
        assert l.moe_norm_backward(n, T, None, None, None, ptr, act, act, None, None, 0, ptr,
                                   1 << 40, None) == want
        assert l.moe_mlp_forward(m, T, None, ptr, ptr, act, None, ptr, 1 << 50, None) == want
        assert l.moe_mlp_backward(m, T, act, None, ptr, ptr, act, act, ptr, ptr, 0, 0, ptr,
                                  1 << 50, None) == want
