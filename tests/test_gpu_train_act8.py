"""8-bit activation checkpoints against their definition, code by code."""
import math

import pytest
import torch

from mixture_experts_ffn_05_b200 import train
from tests import train_ref as ref

pytestmark = pytest.mark.gpu
FMTS = ["int8", "e4m3"]
DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    train._lib()


def check(x, kept, fmt):
    q, b = ref.codes8(x, fmt)
    assert torch.equal(kept.scales, b)
    assert torch.equal(ref.code_values(kept.codes), q)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 31), (2, 32), (5, 33), (1, 257), (7, 1000),
                                       (33, 264), (4, 2112), (1000, 8), (2, 65536)])
def test_encode_and_decode(rows, cols, fmt, dtype):
    g = ref.gen(rows * 1000 + cols)
    x = ref.normal(g, rows, cols)
    x = (x * torch.exp2(torch.randint(-12, 8, (rows, cols), generator=g, device="cuda")
                        .float())).to(dtype)
    kept = train.act8(rows, cols, fmt)
    train.moe_act_encode(x, kept)
    check(x, kept, fmt)
    back = torch.empty_like(x)
    train.moe_act_decode(kept, back)
    assert torch.equal(back, ref.decode8(kept).to(dtype))
    if dtype == torch.bfloat16:  # a checkpoint's values are bf16 values: kept again, the same
        again = train.act8(rows, cols, fmt)
        train.moe_act_encode(back, again)
        assert torch.equal(ref.decode8(again), ref.decode8(kept))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("cols,pad_x,pad_c", [(64, 8, 16), (64, 1, 0), (40, 3, 5), (96, 0, 8)])
def test_strided_rows_leave_the_gaps(cols, pad_x, pad_c, fmt):
    rows = 9
    g = ref.gen(11)
    x, _ = ref.padded(ref.normal(g, rows, cols, dtype=torch.bfloat16), pad_x)
    k = train.act8(rows, cols, fmt)
    codes, cbase = ref.padded(k.codes.zero_(), pad_c, 77)
    kept = train.Act8(codes, k.scales)
    train.moe_act_encode(x, kept)
    check(x, kept, fmt)
    assert (cbase[:, cols:] == 77).all()
    out, obase = ref.padded(torch.zeros(rows, cols, device="cuda"), pad_x)
    train.moe_act_decode(kept, out)
    assert torch.equal(out.double(), ref.decode8(kept))
    assert (obase[:, cols:] == 7.0).all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("cols", [70, 72])
def test_borders_zeros_and_non_finite(fmt, cols):
    """Scales at and next to their borders, halfway codes, zero groups, the extremes of fp32,
    and groups with infinities or NaN (which mark their own group only)."""
    q = 127.0 if fmt == "int8" else 448.0
    x = torch.zeros(10, cols, device="cuda")
    x[0, 3] = q
    x[1, 3] = torch.nextafter(torch.tensor(q), torch.tensor(1e9))  # one step above the border
    x[2, :9] = torch.tensor([q, 0.5, 1.5, 2.5, -0.5, -1.5, 2 ** -10, 3 * 2 ** -10, 17.0])
    x[3, 0], x[3, 40] = math.inf, 1.0
    x[4, 31], x[4, 32] = math.nan, 1.0
    x[5, -1] = -math.inf
    x[6] = torch.finfo(torch.float32).max
    x[7] = 1e-42  # subnormal
    x[8, 0] = torch.finfo(torch.float32).tiny
    kept = train.act8(10, cols, fmt)
    train.moe_act_encode(x, kept)
    check(x, kept, fmt)
    back = torch.empty_like(x)
    train.moe_act_decode(kept, back)
    assert torch.equal(torch.isnan(back), torch.isnan(ref.decode8(kept)))
    assert torch.isnan(back[3, :32]).all() and torch.isfinite(back[3, 32:]).all()
    assert torch.isnan(back[4, :32]).all() and torch.isfinite(back[4, 32:]).all()
    assert torch.isfinite(back[5, :64]).all() and torch.isnan(back[5, 64:]).all()
    fin = torch.isfinite(x) & torch.isfinite(back)
    assert torch.equal(back[fin].double(), ref.decode8(kept)[fin])


def test_offsets_past_32_bits():
    """Elements past 2^31 of a tensor (rows beyond 32-bit offsets)."""
    rows, cols = 66000, 32800  # 2.16e9 codes
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    g = ref.gen(2)
    tail = ref.normal(g, 300, cols, dtype=torch.bfloat16)
    x[-300:] = tail
    kept = train.act8(rows, cols)
    train.moe_act_encode(x, kept)
    assert (kept.scales[:-300] == 1).all()
    check(tail, train.Act8(kept.codes[-300:], kept.scales[-300:]), "int8")
    train.moe_act_decode(kept, x)
    assert torch.equal(x[-300:].double(),
                       ref.decode8(train.Act8(kept.codes[-300:], kept.scales[-300:])))
