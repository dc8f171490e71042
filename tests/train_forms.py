"""How the library tiles the gated MLP's launches, asked from the library itself, and sizes that
between them reach every form of every launch."""
import ctypes
import random

from mixture_experts_ffn_05_b200 import train

LAUNCHES = ("gate_up", "down", "dh", "dx", "gradients")
PAIRS, ONE128, ONE64 = 0, 1, 2  # 10 + n: few tokens, n CTAs a tile

SIZES = [(300, 2816, 2112), (1500, 1000, 1352), (5000, 512, 384), (2, 208, 1544), (2, 496, 352),
         (388, 2432, 32), (2, 72, 32), (2, 336, 480), (5108, 1432, 120), (1882, 1224, 1240)]


def forms(T, H, D):
    """{(launch, form)} of a call at this size; the gradients' launch with dx in it, without it,
    and in a call that wants no dx are launches of their own here."""
    f = train._lib().moe_mlp_tilings
    f.restype = ctypes.c_int32
    f.argtypes = [ctypes.POINTER(train.CMlpConfig), ctypes.c_int32, ctypes.c_int32,
                  ctypes.POINTER(ctypes.c_int32)]
    cfg = train.MlpConfig(H, D).c()
    out, alone = (ctypes.c_int32 * 5)(), (ctypes.c_int32 * 5)()
    assert f(cfg, T, 1, out) and f(cfg, T, 0, alone)
    got = dict(zip(LAUNCHES, out))
    if got["dx"] < 0:
        del got["dx"]
        got["dx and gradients"] = got.pop("gradients")
    got["gradients alone"] = alone[4]
    return set(got.items())


def reachable(n=30000):
    """Every (launch, form) that n random sizes meet."""
    rng = random.Random(1)
    seen = set()
    for _ in range(n):
        seen |= forms(int(2 ** rng.uniform(0, 14)), 8 * int(2 ** rng.uniform(0, 11)),
                      8 * int(2 ** rng.uniform(0, 11)))
    return seen
