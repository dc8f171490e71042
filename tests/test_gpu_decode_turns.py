"""Single tokens one after another on one workspace, nothing waited for in between: each
call must route, gather and multiply by its own routing tables, never by the ones that the
call before left in the workspace."""
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


@pytest.mark.parametrize("shape", [synth.TINY, synth.DECODE], ids=["tiny", "decode"])
def test_tokens_in_turn(shape):
    c = cases.make_case(shape, seed=1234)
    cfg = config(c.shape)
    bw = mf.BlockWeights(cfg, device_layer(c))
    x = to_dev(c.x)
    rounds = 8
    out = torch.zeros(rounds, c.shape.T, cfg.hidden, dtype=torch.bfloat16, device="cuda")
    ws = mf.workspace(cfg, 1)
    for r in range(rounds):
        for t in range(c.shape.T):
            mf.moe_block_forward(cfg, x[t:t + 1], bw, out[r, t:t + 1], ws)
    assert mf.moe_check_device_status(ws) == mf.MOE_OK
    ref = oracle_block(c)["out"]
    for r in range(rounds):
        cases.check_bar(bf16_np(out[r]), ref, cases.FRAC_BF16, f"round {r}")
        assert torch.equal(out[r], out[0])
