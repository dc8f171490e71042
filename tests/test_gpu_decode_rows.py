"""Few (token, slot) pairs: the expert matmuls read each routed row of xn_moe where it lies.
Experts that get one token, some of them or all of them, tokens that are not neighbours,
captured and replayed: against the oracle."""
import dataclasses

import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
import synth
from tests import cases
from tests.gpu_util import bf16_np, config, device_layer, oracle_block, to_dev

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    mf.lib()


SHAPES = [synth.Shape(T=4, H=512, E=8, k=8, I=128, D=384),   # every expert gets every token
          synth.Shape(T=8, H=512, E=5, k=2, I=128, D=384),   # three or so of the eight
          synth.Shape(T=8, H=640, E=16, k=4, I=192, D=128),
          synth.Shape(T=4, H=2816, E=128, k=8, I=704, D=2112),
          synth.Shape(T=1, H=512, E=32, k=1, I=128, D=128)]
IDS = [f"T{s.T}_E{s.E}_k{s.k}" for s in SHAPES]


def check(cfg, c, bw, ws, x):
    out = torch.empty(c.shape.T, cfg.hidden, dtype=torch.bfloat16, device="cuda")
    moe = torch.empty_like(out)
    mf.moe_block_forward(cfg, x, bw, out, ws, moe_out=moe)
    assert mf.moe_check_device_status(ws) == mf.MOE_OK
    ref = oracle_block(c)
    cases.check_bar(bf16_np(out), ref["out"], cases.FRAC_BF16, "out")
    cases.check_bar(bf16_np(moe), ref["moe"], cases.FRAC_BF16, "moe_out")
    return out


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_every_batch_up_to_the_limit(shape):
    """T tokens, then the first T - 1 of them, and so on down to one."""
    c = cases.make_case(shape, seed=77)
    cfg = config(shape)
    bw = mf.BlockWeights(cfg, device_layer(c))
    x = to_dev(c.x)
    for T in range(shape.T, 0, -1):
        assert mf.moe_block_launch_count(cfg, T) == 4
        part = dataclasses.replace(c, shape=dataclasses.replace(shape, T=T), x=c.x[:T])
        check(cfg, part, bw, mf.workspace(cfg, T), x[:T])


@pytest.mark.parametrize("shape", SHAPES[:3], ids=IDS[:3])
def test_a_few_rows_more_than_the_limit_agree(shape):
    """The same tokens in a larger batch, whose rows are gathered: both within the bar, and off
    from one another by no more than two roundings of the output."""
    c = cases.make_case(shape, seed=78)
    cfg = config(shape)
    bw = mf.BlockWeights(cfg, device_layer(c))
    x = to_dev(c.x)
    few = check(cfg, c, bw, mf.workspace(cfg, shape.T), x)
    many = x.repeat(9, 1)
    out = torch.empty_like(many)
    mf.moe_block_forward(cfg, many, bw, out, mf.workspace(cfg, len(many)))
    cases.check_bar(bf16_np(out[-shape.T:]), oracle_block(c)["out"], cases.FRAC_BF16, "gathered")
    cases.check_bar(bf16_np(out[-shape.T:]), bf16_np(few), cases.FRAC_BF16, "both")


def test_captured_and_replayed():
    """Other tokens, and so other experts, in the buffers of a captured call."""
    shape = SHAPES[1]
    c = cases.make_case(shape, seed=79)
    cfg = config(shape)
    bw, ws = mf.BlockWeights(cfg, device_layer(c)), mf.workspace(cfg, shape.T)
    x = to_dev(c.x)
    out = torch.empty_like(x)
    mf.moe_block_forward(cfg, x, bw, out, ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for _ in range(3):  # back to back: no call may read the tables of the one before
            mf.moe_block_forward(cfg, x, bw, out, ws)
    for order in ([3, 1, 0, 2, 7, 6, 5, 4], [7, 7, 7, 7, 0, 0, 0, 0], list(range(8))):
        x.copy_(to_dev(c.x[order]))
        g.replay()
        torch.cuda.synchronize()
        ref = oracle_block(dataclasses.replace(c, x=c.x[order]))["out"]
        cases.check_bar(bf16_np(out), ref, cases.FRAC_BF16, str(order))
