"""Block-scaled e4m3 on the GPU at the ends of the values' range: gates of any
size in the gated product."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw
from oracle import block as ob

pytestmark = pytest.mark.gpu

# silu's exp leaves fp32 beyond 88.7 (large), 87.3 .. 103.9 (small); its argument's
# product with log2(e) leaves it beyond 2.36e38
GATES = [3.4e38, 3e38, 2.4e38, 2.36e38, 1e38, 1e20, 200.0, 104.0, 89.0, 88.72, 88.0, 87.0, 44.5, 44.3, 17.0, 1.0, 1e-3, 1e-30, 0.0]
GATES = GATES + [-g for g in GATES] + [-87.3, -87.34, -87.5, -88.4, -88.7, -88.73, -90.0, -92.0, -95.0, -100.0, -103.0, -130.0, -133.0]


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("up", [1.0, -3.0, 2.0 ** 20])
def test_gates_of_any_size(dtype, up):
    """A row of one value is a block whose scale holds that value's 24 bits."""
    g = torch.tensor(GATES, dtype=torch.float64).clamp(-torch.finfo(dtype).max, torch.finfo(dtype).max)
    h = torch.stack([g, torch.full_like(g, up)], 1).to(dtype).cuda()
    rec = qw.block_quantize_swiglu(h)
    s = rec["scales"].cpu().numpy().astype(np.float64)[:, 0]
    hd = h.double().cpu().numpy()
    want = ob.swiglu(hd)[:, 0]
    silu = ob.swiglu(np.stack([hd[:, 0], np.ones(len(hd))], 1))[:, 0]
    over = np.abs(want) >= 2.0 ** 128 * (1 - 2.0 ** -25)
    assert np.all(np.isinf(s[over])) and np.all(np.isfinite(s[~over])), list(zip(hd[:, 0], s))
    codes = np.where(over, 0, rec["codes"].view(torch.uint8).cpu().numpy()[:, 0])
    got = ob.values(codes[:, None], np.where(over, 0, s)[:, None].astype(np.float32), 1, 1)[:, 0]
    # exp 2 ulp, sum and reciprocal 1.5, two products 1, the scale's division 0.5, its product
    # with the code, which has no error here: 5 ulp of 2^-23; and where silu or the
    # scale is subnormal half of 2^-149, times up or times 448
    ok = np.abs(got - want) <= 5 * 2.0 ** -23 * np.abs(want) + 2.0 ** -150 * (abs(up) + 1)
    # a subnormal scale: off by half of 2^-149, so that the code is not the largest one: half a step of it
    small = np.abs(want) < 448 * 2.0 ** -126
    ok |= small & (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + 450 * 2.0 ** -150 + 2.0 ** -150 * abs(up))
    assert np.all(ok | over), [v for v in zip(hd[:, 0], silu, got, want, ok) if not v[-1]]


@pytest.mark.parametrize("t", [2, 40, 700])
@pytest.mark.parametrize("gate", [3e38, -80.0, -88.5, -3e38])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_expert_mlp_with_far_gates(t, gate, dtype):
    """The same in the products that gate their input or their output: every hidden
    value of a token is one number, which codes hold exactly."""
    d, f = 128, 128
    x = torch.full((t, d), 2.0 ** 60 if abs(gate) > 1e3 else 1.0, device="cuda")
    scale = float(x[0, 0]) * d
    up = 1.0 if abs(gate) > 1e3 else 2.0 ** 100
    w = torch.cat([torch.full((2, f, d), gate / scale), torch.full((2, f, d), up / scale)], 1)
    down = torch.full((2, d, f), 2.0 ** -90, device="cuda")
    ids = torch.arange(t, device="cuda")[:, None] % 2
    y = qw.moe_mlp(qw.block_quantize(w.cuda(), 128), qw.block_quantize(down, 128), x, ids, out_dtype=dtype)
    held = float(w[0, 0, 0]) * scale
    want = float(ob.swiglu(np.array([[held, up]]))[0, 0]) * f * 2.0 ** -90
    # an error of the gate is multiplied by |gate| where silu falls off: quantizer, product
    # and sum are off by 2^-23 each; then a few ulp, and half a step of y's type
    steep = 3 * abs(gate) if -1e3 < gate < 0 else 3
    bar = (steep + 8) * 2.0 ** -23 + (0 if dtype is torch.float32 else 2.0 ** -8)
    assert bool(((y.double() - want).abs() <= bar * abs(want)).all()), (y[0, 0], want)
