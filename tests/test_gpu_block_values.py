"""Block-scaled e4m3 on the GPU at the ends of the values' range: gates of any
size in the gated product, and blocks with NaN or infinities in them."""

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


def poisoned(rows, k, size, poison, dtype):
    """Values up to `size`, the same with one value replaced, and where: row 2, column 130."""
    rng = np.random.default_rng([rows, k])
    w = (rng.uniform(-1, 1, (rows, k)) * size).astype(np.float32)
    w[:, ::128] = size
    clean = torch.from_numpy(w).to(dtype)
    clean[2, 130] = 0.0
    dirty = clean.clone()
    dirty[2, 130] = poison
    return clean.cuda(), dirty.cuda()


def codes_of(rec):
    return rec["codes"].view(torch.uint8).cpu().numpy()


# scales of 1, below 2^-60, of a subnormal value, and above 2^100
SCALES = [448.0, 1e-18, 1e-40, 1e35]


@pytest.mark.parametrize("size", SCALES)
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype,k", [(torch.float32, 384), (torch.float32, 301), (torch.bfloat16, 384)])
def test_a_block_with_a_value_that_is_no_number(size, poison, block_rows, dtype, k):
    clean, dirty = poisoned(5, k, size, poison, dtype)
    a, b = qw.block_quantize(clean, block_rows), qw.block_quantize(dirty, block_rows)
    ca, cb = codes_of(a), codes_of(b)
    sa, sb = a["scales"].cpu().numpy(), b["scales"].cpu().numpy()
    assert cb[2, 130] & 127 == 127
    rows = slice(2, 3) if block_rows == 1 else slice(0, 5)
    hit = (2 if block_rows == 1 else 0, 1)
    if np.isnan(poison):      # its own code, and nothing else
        ca[2, 130] = cb[2, 130]
        assert np.array_equal(ca, cb) and np.array_equal(sa.view(np.uint32), sb.view(np.uint32))
    else:                     # the block's scale is infinite
        assert np.isposinf(sb[hit])
        sb[hit] = sa[hit]
        assert np.array_equal(sa, sb)
        block = cb[rows, 128:256].copy()
        block[2 - rows.start, 2] &= 0
        assert not (block & 127).any()
        cb[rows, 128:256] = ca[rows, 128:256]
        assert np.array_equal(ca, cb)
        assert bool(torch.isnan(qw.block_unpack(b)[rows, 128:256]).all())


@pytest.mark.parametrize("size", SCALES)
@pytest.mark.parametrize("poison", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("m", [4, 12, 40, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_products_of_what_is_no_number(size, poison, m, dtype):
    """The poisoned row's outputs are NaN, for every way that x is quantized, and the others as they were."""
    clean, dirty = poisoned(m, 384, size, poison, dtype)
    rec = qw.block_quantize(torch.rand(70, 384, device="cuda") + 0.5, 128)
    a, b = qw.block_matmul(rec, clean), qw.block_matmul(rec, dirty)
    keep = torch.arange(m, device="cuda") != 2
    assert bool(torch.isnan(b[2]).all()) and torch.equal(a[keep], b[keep])
    # as rows of an expert's tokens: gathered as codes
    pos = torch.arange(m, dtype=torch.int32, device="cuda")[:, None]
    c, d = qw.moe_gather_block(dirty, dict(pos=pos)), qw.block_quantize(dirty, 1)
    assert np.array_equal(codes_of(c), codes_of(d)) and np.array_equal(c["scales"].cpu().numpy(), d["scales"].cpu().numpy())


@pytest.mark.parametrize("t", [2, 40, 700])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_expert_mlp_of_a_token_that_is_no_number(t, dtype):
    """Tiny tokens, one of them with a NaN: its output is NaN (quantized in the product, gathered, gated)."""
    gate_up = qw.block_quantize(torch.rand(2, 256, 256, device="cuda") + 0.5, 128)
    down = qw.block_quantize(torch.rand(2, 256, 128, device="cuda") + 0.5, 128)
    x = (torch.rand(t, 256, device="cuda") * 1e-18).to(dtype)
    ids = torch.arange(t, device="cuda")[:, None] % 2
    clean = qw.moe_mlp(gate_up, down, x, ids)
    x[1, 130] = float("nan")
    y = qw.moe_mlp(gate_up, down, x, ids)
    keep = torch.arange(t, device="cuda") != 1
    assert bool(torch.isnan(y[1]).all()) and torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("m", [4, 40, 300])
def test_weights_that_are_no_number(block_rows, m):
    """A NaN in a tiny weight reaches its own column of y, and only that."""
    clean, dirty = poisoned(140, 384, 1e-18, float("nan"), torch.float32)
    x = torch.rand(m, 384, device="cuda") + 0.5
    for dtype in (torch.float32, torch.bfloat16):
        a = qw.block_matmul(qw.block_quantize(clean, block_rows), x, out_dtype=dtype)
        b = qw.block_matmul(qw.block_quantize(dirty, block_rows), x, out_dtype=dtype)
        keep = torch.arange(140, device="cuda") != 2
        assert bool(torch.isnan(b[:, 2]).all()) and torch.equal(a[:, keep], b[:, keep])
