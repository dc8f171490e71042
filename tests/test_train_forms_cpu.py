"""The sizes at which the GPU tests run the gated MLP reach every form of every launch.  A new
estimate of a tiling's time may move sizes from one form to another: then this fails, and the
sizes are to be chosen again."""
import pytest

from mixture_experts_ffn_05_b200 import build as mbuild
from tests import train_forms


@pytest.fixture(scope="module", autouse=True)
def _lib():
    mbuild.build()


def test_every_form_of_every_launch_is_run():
    run = set().union(*(train_forms.forms(*s) for s in train_forms.SIZES))
    can = train_forms.reachable()
    few = {10 + n for n in (1, 2, 4, 8)}
    tiles = {train_forms.PAIRS, train_forms.ONE128, train_forms.ONE64}
    for launch in ("gate_up", "down", "dh"):
        assert {f for l, f in can if l == launch} == tiles | few
    assert {f for l, f in can if l == "dx"} == few
    for launch in ("gradients", "dx and gradients", "gradients alone"):
        assert {f for l, f in can if l == launch} == tiles
    assert can <= run
