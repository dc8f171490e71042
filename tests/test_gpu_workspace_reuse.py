"""One workspace for batches of every size in turn: whatever a call left in it, the next one
gives the bits that it gives on a workspace of its own."""
import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
import synth
from mixture_experts_ffn_05_b200 import train
from tests import cases
from tests.gpu_util import (config, device_layer, fp8_experts, int8_experts, nvfp4_experts, to_dev)

pytestmark = pytest.mark.gpu

# split K, no split, pieces from a counter, pairs; both routers, sorts in the router, in one
# block and in many: sizes up and down past each border
BATCHES = (4, 3, 2, 1, 8, 5, 64, 16, 3, 200, 64, 129, 7, 512, 33, 1024, 128, 300, 1, 513, 6)
SMALL = synth.Shape(T=8, H=512, E=16, k=4, I=128, D=384)
LAYER = synth.Shape(T=8, H=2816, E=128, k=8, I=704, D=2112)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mf.lib()


def experts(c, fmt):
    if fmt == "bf16":
        return {}
    return {"int8": int8_experts, "fp8": fp8_experts, "nvfp4": nvfp4_experts}[fmt](c)[0]


def block(cfg, bw, x, ws):
    out = torch.empty_like(x)
    moe = torch.empty_like(x)
    mf.moe_block_forward(cfg, x, bw, out, ws, moe_out=moe)
    assert mf.moe_check_device_status(ws) == mf.MOE_OK
    return out, moe


@pytest.mark.parametrize("shape,fmt", [(SMALL, "bf16"), (LAYER, "bf16"), (SMALL, "int8"),
                                       (SMALL, "fp8"), (SMALL, "nvfp4")],
                         ids=["small_bf16", "layer_bf16", "int8", "fp8", "nvfp4"])
def test_blocks_of_every_size(shape, fmt):
    c = cases.make_case(shape, seed=41, gap=False)
    base = config(shape)
    cfg = mf.Config(**{**base.__dict__, fmt: True}) if fmt != "bf16" else base
    bw = mf.BlockWeights(cfg, {**device_layer(c), **experts(c, fmt)})
    x = to_dev(synth.x_rows(42, shape.H, max(BATCHES)))
    shared = torch.zeros(max(mf.workspace_size(cfg, T) for T in BATCHES), dtype=torch.uint8,
                         device="cuda")
    for T in BATCHES:
        want = block(cfg, bw, x[:T], mf.workspace(cfg, T))
        got = block(cfg, bw, x[:T], shared)
        for a, b in zip(got, want):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16)), T


def test_dense_mlps_and_layers_of_two_shapes():
    """The dense MLP alone, and two layers of other sizes, in turn with blocks."""
    pair = []
    for seed, shape in ((43, SMALL), (44, synth.Shape(T=8, H=768, E=8, k=2, I=256, D=512))):
        c = cases.make_case(shape, seed=seed, gap=False)
        cfg = config(shape)
        pair.append((cfg, mf.BlockWeights(cfg, device_layer(c)),
                     to_dev(synth.x_rows(seed, shape.H, 512))))
    sizes = (3, 300, 16, 1, 512, 40, 2)
    shared = torch.zeros(max(mf.workspace_size(p[0], T) for p in pair for T in sizes),
                         dtype=torch.uint8, device="cuda")
    for T in sizes:
        for cfg, bw, x in pair:
            outs = []
            for ws in (mf.workspace(cfg, T), shared):
                d = torch.empty_like(x[:T])
                mf.dense_mlp_forward(cfg, x[:T], bw.tensors["w_dense_gate_up"],
                                     bw.tensors["w_dense_down"], d, ws)
                outs.append((d, *block(cfg, bw, x[:T], ws)))
            for a, b in zip(*outs):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16)), T


@pytest.mark.parametrize("rest", [1, 3, 16, 128, 452])
def test_stack_whose_last_chunk_is_short(rest):
    """Two chunks through two layers, the last of `rest` tokens, then the whole once more."""
    cfg = config(SMALL)
    layers = []
    for l in range(2):
        c = cases.make_case(SMALL, seed=45 + l, gap=False)
        layers.append(mf.BlockWeights(cfg, device_layer(c)))
    x = to_dev(synth.x_rows(47, SMALL.H, 1024 + rest))
    ws = mf.stack_workspace(cfg, 1024)
    want = torch.empty_like(x)
    for t0, n in ((0, 1024), (1024, rest)):
        cur = x[t0:t0 + n]
        for bw in layers:
            cur = block(cfg, bw, cur, mf.workspace(cfg, n))[0]
        want[t0:t0 + n] = cur
    for _ in range(2):
        out = torch.zeros_like(x)
        mf.moe_stack_forward(cfg, x, layers, out, ws, chunk_tokens=1024)
        assert mf.moe_check_device_status(ws) == mf.MOE_OK
        assert torch.equal(out.view(torch.int16), want.view(torch.int16))


def test_blocks_and_training_calls_in_turn():
    """Inference of a block and training passes of its dense branch on one workspace."""
    from tests.test_gpu_train_mlp import Case as MlpCase
    from tests.test_gpu_train_norm import Case as NormCase

    c = cases.make_case(SMALL, seed=48, gap=False)
    cfg = config(SMALL)
    bw = mf.BlockWeights(cfg, device_layer(c))
    x = to_dev(synth.x_rows(49, SMALL.H, 300))
    sizes = (8, 300, 3, 64)
    mcfg, ncfg = train.MlpConfig(SMALL.H, SMALL.D), train.NormConfig(SMALL.H, "layer")
    need = max(max(mf.workspace_size(cfg, T), train.mlp_workspace(mcfg, T).numel(),
                   train.norm_workspace(ncfg, T).numel()) for T in sizes)
    ws = torch.zeros(need, dtype=torch.uint8, device="cuda")
    for T in sizes:
        want = block(cfg, bw, x[:T], mf.workspace(cfg, T))
        m = MlpCase(T, SMALL.H, SMALL.D, keep="int8", seed=T).forward().backward()
        n = NormCase(T, SMALL.H, "layer", seed=T).run()
        outs = (m.y, m.dx, m.dwgu, m.dwd, n.y, n.dx, n.d_gain, n.d_bias)
        first = [t.clone() for t in outs]
        m.ws = n.ws = ws
        for _ in range(2):
            m.forward().backward()
            n.run()
            for a, b in zip(outs, first):
                assert torch.equal(a, b)
            for a, b in zip(block(cfg, bw, x[:T], ws), want):
                assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("start", [-16, -1000000, 5])
def test_a_piece_counter_that_is_not_zero(start):
    """A workspace that was not zeroed gives wrong results at most: pieces below zero or past the
    end are nobody's."""
    c = cases.make_case(SMALL, seed=50, gap=False)
    cfg = config(SMALL)
    bw = mf.BlockWeights(cfg, device_layer(c))
    T = 100  # tiles of 64 tokens, whose pieces come from the counter
    x = to_dev(synth.x_rows(51, SMALL.H, T))
    ws = mf.workspace(cfg, T)
    want = block(cfg, bw, x, ws)
    ws[256 + 1024:256 + 1024 + 12].view(torch.int32)[[0, 2]] = start
    out = torch.empty_like(x)
    mf.moe_block_forward(cfg, x, bw, out, ws)
    torch.cuda.synchronize()
    ws.zero_()
    for a, b in zip(block(cfg, bw, x, ws), want):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
