"""The training operators together, as a training step of the dense branch uses them:
out = x + N_post(MLP(N_pre(x))), forward and backward, from 16-bit activations and from 8-bit
checkpoints, on streams, captured and replayed."""
import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import train
from tests import train_ref as ref

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    train._lib()


class Branch:
    """Weights, buffers and workspaces of one dense branch over T tokens."""

    def __init__(self, T, H, D, keep, seed=1):
        g = ref.gen(seed)
        bf = torch.bfloat16
        self.T, self.H, self.D, self.keep = T, H, D, keep
        self.ncfg = train.NormConfig(cols=H)
        self.mcfg = train.MlpConfig(hidden=H, inter=D)
        self.x = ref.normal(g, T, H, dtype=bf)
        self.dout = ref.normal(g, T, H, dtype=bf)
        self.g1, self.g2 = ((torch.rand(H, generator=g, device="cuda") + 0.5).to(bf)
                            for _ in range(2))
        self.wgu = ref.normal(g, 2 * D, H, std=1 / H ** 0.5, dtype=bf)
        self.wd = ref.normal(g, H, D, std=1 / D ** 0.5, dtype=bf)
        row = lambda: torch.zeros(T, H, dtype=bf, device="cuda")  # noqa: E731
        self.xn, self.m, self.out, self.dm, self.dxn, self.dx = (row() for _ in range(6))
        self.r1, self.r2 = (torch.zeros(T, device="cuda") for _ in range(2))
        self.dg1, self.dg2 = (torch.zeros(H, device="cuda") for _ in range(2))
        self.dwgu, self.dwd = torch.zeros_like(self.wgu), torch.zeros_like(self.wd)
        if keep == "16":
            self.kx, self.kxn, self.km = self.x, self.xn, self.m
            self.kgu = torch.zeros(T, 2 * D, dtype=bf, device="cuda")
        else:
            self.kx, self.kxn, self.km = (train.act8(T, H, keep) for _ in range(3))
            self.kgu = train.act8(T, D, keep, parts=2)
        self.ws, self.nws = train.mlp_workspace(self.mcfg, T), train.norm_workspace(self.ncfg, T)

    def step(self, stream=None):
        n, m, kw = self.ncfg, self.mcfg, {"stream": stream}
        eight = self.keep != "16"
        train.moe_norm_forward(n, self.x, self.g1, None, self.xn, None, self.r1,
                               kept=self.kx if eight else None, **kw)
        if eight:
            train.moe_act_encode(self.xn, self.kxn, **kw)
        train.moe_mlp_forward(m, self.xn, self.wgu, self.wd, self.m, self.ws, kept_gu=self.kgu,
                              **kw)
        train.moe_norm_forward(n, self.m, self.g2, None, self.out, None, self.r2,
                               kept=self.km if eight else None, **kw)
        train.moe_norm_backward(n, self.km, self.g2, None, self.r2, self.dout, self.dm, self.dg2,
                                None, self.nws, **kw)
        train.moe_mlp_backward(m, self.kxn, self.kgu, self.wgu, self.wd, self.dm, self.dxn,
                               self.dwgu, self.dwd, self.ws, **kw)
        train.moe_norm_backward(n, self.kx, self.g1, None, self.r1, self.dxn, self.dx, self.dg1,
                                None, self.nws, **kw)
        return self

    def results(self):
        return {n: getattr(self, n) for n in ("out", "dx", "dg1", "dg2", "dwgu", "dwd")}

    def exact(self):
        """By automatic differentiation of the definition in 64 bits."""
        leaves = [t.double().requires_grad_() for t in (self.x, self.g1, self.g2, self.wgu, self.wd)]
        x, g1, g2, wgu, wd = leaves
        xn = ref.norm_forward(x, g1, None, "rms", 1e-6)[0]
        m = ref.mlp_forward(xn, wgu, wd, "gelu_tanh")[0]
        out = ref.norm_forward(m, g2, None, "rms", 1e-6)[0]
        (out * self.dout.double()).sum().backward()
        return dict(zip(("out", "dx", "dg1", "dg2", "dwgu", "dwd"),
                        [out.detach()] + [t.grad for t in leaves]))


# Each 16-bit tensor on the way (at most 9: xn, g u, h, m, dm, dg du, dxn and the result) is
# rounded once, half a step each, unrelated to the others: 3 half steps, and twice that where
# a norm's projection or a product of two rounded factors passes on more than it is given.
# An 8-bit tensor's error is at most s / sqrt(12) per value in the root mean square, s <= 2
# max / 127: max / 220, where a group's max is at most 4 times its root mean square here
# (normal values): 0.018 for int8.  E4M3 is off by at most 2^-4 / sqrt(3) = 0.036.  Three such
# tensors (gu twice, and x, xn or m) meet in a gradient: sqrt(3) times that.
LIMIT = {"16": 6 * 2.0 ** -8, "int8": 6 * 2.0 ** -8 + 3 ** 0.5 * 0.018,
         "e4m3": 6 * 2.0 ** -8 + 3 ** 0.5 * 0.036}


@pytest.mark.parametrize("keep", ["16", "int8", "e4m3"])
@pytest.mark.parametrize("T,H,D", [(1, 512, 384), (37, 512, 384), (700, 264, 200),
                                   (300, 2816, 2112)])
def test_training_step(T, H, D, keep):
    b = Branch(T, H, D, keep).step()
    want = b.exact()
    for n, got in b.results().items():
        lim = LIMIT["16"] if n == "out" else LIMIT[keep]
        assert ref.rel2(got, want[n]) <= lim, n
    for w in (b.ws, b.nws):
        assert mf.moe_check_device_status(w) == mf.MOE_OK


def test_two_streams_at_once():
    """Two branches with workspaces of their own, enqueued side by side."""
    pairs = [Branch(300, 512, 384, k, seed=s) for s, k in ((1, "int8"), (2, "16"))]
    alone = [{n: t.clone() for n, t in b.step().results().items()} for b in pairs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pairs]
    for _ in range(10):
        for b, s in zip(pairs, streams):
            b.step(stream=s)
    torch.cuda.synchronize()
    for b, want in zip(pairs, alone):
        for n, t in b.results().items():
            assert torch.equal(t, want[n]), n


@pytest.mark.parametrize("keep", ["16", "e4m3"])
def test_captured_and_replayed(keep):
    """A captured step gives the bits of the eager one, on new values in the same buffers, and
    two captures that share a workspace may be replayed in turn."""
    b = Branch(130, 512, 384, keep)
    b.step()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for g in graphs:
        with torch.cuda.graph(g):
            b.step()
    for seed, g in ((5, graphs[0]), (6, graphs[1]), (7, graphs[0])):
        b.x.copy_(ref.normal(ref.gen(seed), 130, 512))
        b.dout.copy_(ref.normal(ref.gen(seed + 50), 130, 512))
        b.step()
        want = {n: t.clone() for n, t in b.results().items()}
        for t in b.results().values():
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        for n, t in b.results().items():
            assert torch.equal(t, want[n]), n


def test_workspace_of_a_larger_batch_serves_smaller_ones():
    big, small = Branch(700, 512, 384, "int8"), Branch(37, 512, 384, "int8", seed=9)
    small.step()
    want = {n: t.clone() for n, t in small.results().items()}
    small.ws, small.nws = big.ws, big.nws
    big.step()
    small.step()
    for n, t in small.results().items():
        assert torch.equal(t, want[n]), n


def test_tensors_of_two_devices_are_refused():
    """A tensor that is not where the call's first one is never reaches the library."""
    b = Branch(4, 64, 64, "16")
    with pytest.raises(ValueError, match="CUDA"):
        train.moe_mlp_forward(b.mcfg, b.x, b.wgu.cpu(), b.wd, b.m, b.ws)
    with pytest.raises(ValueError, match=r"must be \[4, 64\]"):
        train.moe_mlp_forward(b.mcfg, b.x, b.wgu, b.wd, b.m[:3], b.ws)
    with pytest.raises(ValueError, match="contiguous rows"):
        train.moe_norm_forward(b.ncfg, torch.zeros(64, 4, dtype=torch.bfloat16, device="cuda").t(),
                               b.g1, None, b.out, None, b.r1)
    with pytest.raises(ValueError, match="part"):
        train.moe_mlp_forward(b.mcfg, b.x, b.wgu, b.wd, b.m, b.ws, kept_gu=train.act8(4, 128))
    with pytest.raises(mf.MoeError):  # rows that overlap
        train.moe_norm_forward(b.ncfg, b.x[:1].expand(4, 64), b.g1, None, b.out, None, b.r1)
