"""Calls from several host threads at once, each with tensors, workspaces and a stream of its own."""
import ctypes
import threading

import pytest
import torch

import mixture_experts_ffn_05_b200 as mf
from mixture_experts_ffn_05_b200 import train
from tests.test_gpu_train_mlp import Case as MlpCase
from tests.test_gpu_train_norm import Case as NormCase

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    train._lib()


def norm_calls(c, stream):
    """A norm's two calls as ready arguments of the library's functions, so that threads spend
    their time in the library, where the interpreter's lock does not part them."""
    l, n, dt = train._lib(), c.n, c.x.dtype

    def act(t):
        return train._act(t, "t", t.get_device(), c.T, n, dt)

    def ptr(t):
        return None if t is None else t.data_ptr()

    s = stream.cuda_stream
    return ((l.moe_norm_forward, (c.cfg.c(), c.T, act(c.x), ptr(c.gain), ptr(c.bias), act(c.y),
                                  ptr(c.mean), ptr(c.rstd), None, s)),
            (l.moe_norm_backward, (c.cfg.c(), c.T, act(c.x), ptr(c.gain), ptr(c.mean),
                                   ptr(c.rstd), act(c.dy), act(c.dx), ptr(c.d_gain),
                                   ptr(c.d_bias), 0, ptr(c.ws), c.ws.numel(), s)))


@pytest.mark.parametrize("which", [0, 1], ids=["forward", "backward"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norms_of_few_and_many_rows(kind, which):
    """The same kernel with little shared memory (few rows: two teams a CTA) and with much of it
    (many rows): no call may lower the limit that another one is about to launch with."""
    cases = [NormCase(T, 2816, kind, seed=T + i).run() for i, T in enumerate((296, 3000) * 2)]
    outs = lambda c: (c.y, c.dx, c.d_gain, c.rstd)  # noqa: E731
    want = [[t.clone() for t in outs(c)] for c in cases]
    torch.cuda.synchronize()
    start, refused = threading.Barrier(len(cases)), []

    def work(c, stream):
        fn, args = norm_calls(c, stream)[which]
        start.wait()
        refused.append(sum(fn(*args) != 0 for _ in range(4000)))

    streams = [torch.cuda.Stream() for _ in cases]
    threads = [threading.Thread(target=work, args=a) for a in zip(cases, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(cases)
    for c, w in zip(cases, want):
        for t, f in zip(outs(c), w):
            assert torch.equal(t, f)


@pytest.mark.parametrize("T", [8, 200])
def test_routers_of_narrow_and_wide_layers(T):
    """The routers' kernels with the shared memory of two layer widths (T = 8) and of two expert
    counts (T = 200, the tensor-core router)."""
    sizes = [(512, 32), (2816, 128)] * 2
    calls, outs = [], []
    for i, (H, E) in enumerate(sizes):
        cfg = mf.Config(hidden=H, num_experts=E, top_k=4, expert_inter=128, dense_inter=128)
        g = torch.Generator(device="cuda").manual_seed(i)
        t = {n: torch.randn(*sh, generator=g, device="cuda").bfloat16()
             for n, sh in (("x", (T, H)), ("rs", (H,)), ("wr", (E, H)), ("pes", (E,)),
                           ("gm", (H,)), ("gd", (H,)))}
        idx = torch.zeros(T, 4, dtype=torch.int32, device="cuda")
        w = torch.zeros(T, 4, device="cuda")
        xm, xd = torch.zeros_like(t["x"]), torch.zeros_like(t["x"])
        ws = mf.workspace(cfg, T)
        mf.moe_router(cfg, t["x"], t["rs"], t["wr"], None, t["pes"], t["gm"], t["gd"], idx, w, xm,
                      xd, ws)
        outs.append([(o, o.clone()) for o in (idx, w, xm, xd)] + [(ws, None), (t, None)])
        calls.append((cfg.c(), T, *(p.data_ptr() for p in (t["x"], t["rs"], t["wr"])), None,
                      *(p.data_ptr() for p in (t["pes"], t["gm"], t["gd"], idx, w, xm, xd, ws)),
                      ws.numel()))
    torch.cuda.synchronize()
    start, refused = threading.Barrier(len(calls)), []
    fn = mf.lib().moe_router

    def work(args, stream):
        args = (ctypes.byref(args[0]), *args[1:], stream.cuda_stream)
        start.wait()
        refused.append(sum(fn(*args) != 0 for _ in range(3000)))

    streams = [torch.cuda.Stream() for _ in calls]
    threads = [threading.Thread(target=work, args=a) for a in zip(calls, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert refused == [0] * len(calls)
    for o in outs:
        for got, want in o[:4]:
            assert torch.equal(got, want)


def on_a_new_thread(body):
    """body on a host thread that has not used the GPU before; what it raised."""
    raised = []

    def work():
        try:
            body()
        except Exception as e:  # noqa: BLE001 - reported by the test
            raised.append(repr(e))

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    return raised


@pytest.mark.parametrize("T", [5, 700])
def test_first_call_of_a_thread(T):
    """Each entry point as a thread's very first use of the GPU."""
    H, D = 512, 384
    c = MlpCase(T, H, D, keep="int8").forward().backward()
    cfg = mf.Config(hidden=H, num_experts=16, top_k=4, expert_inter=128, dense_inter=D)
    out, ws = torch.empty(T, H, dtype=torch.bfloat16, device="cuda"), mf.workspace(cfg, T)
    x = c.x.contiguous()
    mf.dense_mlp_forward(cfg, x, c.wgu, c.wd, out, ws)
    results = (c.y, c.gu.codes, c.dx, c.dwgu, c.dwd, out)
    want = [t.clone() for t in results]
    for t in results:
        t.zero_()
    torch.cuda.synchronize()
    s = torch.cuda.current_stream()
    assert on_a_new_thread(c.forward) == []
    assert on_a_new_thread(c.backward) == []
    assert on_a_new_thread(
        lambda: mf.dense_mlp_forward(cfg, x, c.wgu, c.wd, out, ws, stream=s)) == []
    for t, f in zip(results, want):
        assert torch.equal(t, f)
    n = NormCase(T, H, "layer").run()
    want = n.dx.clone()
    n.dx.zero_()
    torch.cuda.synchronize()
    assert on_a_new_thread(n.run) == []
    assert torch.equal(n.dx, want)


def test_mlps_of_few_and_many_tokens():
    """Forward and backward passes of two sizes on two threads, over and over."""
    cases = [MlpCase(T, 512, 384, keep="int8", seed=T).forward().backward() for T in (40, 1000)]
    outs = lambda c: (c.y, c.dx, c.dwgu, c.dwd)  # noqa: E731
    want = [[t.clone() for t in outs(c)] for c in cases]
    torch.cuda.synchronize()
    start, raised = threading.Barrier(len(cases)), []

    def work(c):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                start.wait()
                for _ in range(500):
                    c.forward().backward()
        except Exception as e:  # noqa: BLE001 - reported below
            raised.append(repr(e))

    threads = [threading.Thread(target=work, args=(c,)) for c in cases]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert raised == []
    for c, w in zip(cases, want):
        assert mf.moe_check_device_status(c.ws) == mf.MOE_OK
        for t, f in zip(outs(c), w):
            assert torch.equal(t, f)
