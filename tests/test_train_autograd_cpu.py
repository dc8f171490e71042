"""The training calls and autograd, on the CPU with the library's part left out: outputs that
require a gradient are refused, and writing a tensor that autograd has saved is noticed."""
import pytest
import torch

from mixture_experts_ffn_05_b200 import train

BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture()
def calls(monkeypatch):
    """Every entry point as (name, function of its outputs, the outputs)."""
    monkeypatch.setattr(train, "_run", lambda *a: None)
    n, m = train.NormConfig(8, "layer"), train.MlpConfig(8, 16)
    x, ws = torch.zeros(4, 8, dtype=BF), torch.zeros(64, dtype=torch.uint8)
    g, st = torch.zeros(8, dtype=BF), torch.zeros(4)
    wgu, wd, gu = (torch.zeros(*s, dtype=BF) for s in ((32, 8), (8, 16), (4, 32)))

    def e(*s, dtype=BF):
        return torch.zeros(*s, dtype=dtype)

    kx = lambda: train.act8(4, 8, device="cpu")  # noqa: E731
    return [
        ("encode", lambda k: train.moe_act_encode(x, k), [kx()]),
        ("decode", lambda o: train.moe_act_decode(kx(), o), [e(4, 8)]),
        ("norm_forward", lambda y, mu, r, k: train.moe_norm_forward(n, x, g, g, y, mu, r, kept=k),
         [e(4, 8), e(4, dtype=F32), e(4, dtype=F32), kx()]),
        ("norm_backward",
         lambda dx, a, b: train.moe_norm_backward(n, x, g, st, st, x, dx, a, b, ws),
         [e(4, 8), e(8, dtype=F32), e(8, dtype=F32)]),
        ("mlp_forward", lambda y, k: train.moe_mlp_forward(m, x, wgu, wd, y, ws, kept_gu=k),
         [e(4, 8), e(4, 32)]),
        ("mlp_forward_8", lambda y, k: train.moe_mlp_forward(m, x, wgu, wd, y, ws, kept_gu=k),
         [e(4, 8), train.act8(4, 16, device="cpu", parts=2)]),
        ("mlp_backward",
         lambda dx, a, b: train.moe_mlp_backward(m, x, gu, wgu, wd, x, dx, a, b, ws),
         [e(4, 8), e(32, 8), e(8, 16)]),
    ]


def tensors(t):
    return [t.codes, t.scales] if isinstance(t, train.Act8) else [t]


def test_written_tensors_count_a_version(calls):
    for name, call, outs in calls:
        before = [t._version for o in outs for t in tensors(o)]
        call(*outs)
        after = [t._version for o in outs for t in tensors(o)]
        assert all(b > a for a, b in zip(before, after)), name


def test_outputs_that_require_a_gradient_are_refused(calls):
    for name, call, outs in calls:
        for i, o in enumerate(outs):
            if isinstance(o, train.Act8):
                continue
            leaf = o.clone().requires_grad_()
            args = [leaf if j == i else t for j, t in enumerate(outs)]
            with pytest.raises(ValueError, match="requires a gradient"):
                call(*args)
            assert leaf._version == 0
            with torch.no_grad():  # where torch lets a leaf be written too
                call(*args)
            args[i] = leaf.detach()
            call(*args)


def test_inputs_may_require_gradients(monkeypatch):
    monkeypatch.setattr(train, "_run", lambda *a: None)
    x, w = torch.zeros(4, 8, dtype=BF), torch.zeros(16, 8, dtype=BF)
    for t in (x, w):
        t.requires_grad_()
    y, ws = torch.zeros(4, 8, dtype=BF), torch.zeros(64, dtype=torch.uint8)
    with torch.no_grad():
        wd = w[:8].clone().requires_grad_()
    train.moe_mlp_forward(train.MlpConfig(8, 8), x, w, wd, y, ws)
    assert x._version == w._version == wd._version == 0 and y._version == 1


def test_a_saved_tensor_that_is_overwritten_raises(calls):
    a = torch.ones(4, 8, dtype=BF, requires_grad=True)
    name, call, (y, mu, r, kept) = calls[2]
    out = (a * y).sum()  # saves y
    call(y, mu, r, kept)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        out.backward()


def test_wrong_outputs_still_name_themselves(calls):
    x = torch.zeros(4, 8, dtype=BF)
    with pytest.raises(TypeError, match="y must be"):
        train.moe_norm_forward(train.NormConfig(8), x, None, None, 3, None, torch.zeros(4))
    with pytest.raises(ValueError, match="y is required"):
        train.moe_norm_forward(train.NormConfig(8), x, None, None, None, None, torch.zeros(4))


def test_tensors_of_inference_mode(monkeypatch):
    monkeypatch.setattr(train, "_run", lambda *a: None)
    with torch.inference_mode():
        x, y = torch.zeros(4, 8, dtype=BF), torch.zeros(4, 8, dtype=BF)
        r = torch.zeros(4)
        train.moe_norm_forward(train.NormConfig(8), x, None, None, y, None, r)
    train.moe_norm_forward(train.NormConfig(8), x, None, None, y, None, r)
