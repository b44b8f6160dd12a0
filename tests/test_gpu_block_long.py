"""Products with long sums and with scales far from 1, within qw.h's bounds."""

import pytest
import torch

from int8_int4_dequant_amd import qw

pytestmark = pytest.mark.gpu

BAR = {torch.float32: 1e-5, torch.bfloat16: 1e-3}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def check(y, xrec, rec, k):
    """In float64 on the GPU; block_unpack rounds each value once (2^-24)."""
    xv, wv = qw.block_unpack(xrec).double(), qw.block_unpack(rec).double()
    ref, base = xv @ wv.T, xv.abs() @ wv.abs().T
    bar = (BAR[y.dtype] + -(-k // 128) * 2.0 ** -24 + 2.0 ** -23) * base
    err = (y.double() - ref).abs()
    assert bool((err <= bar + HALF[y.dtype] * (ref.abs() + bar)).all())
    return float((err / base).max())


# direct kernels, whose waves share k, and a tiled one, whose waves do not
SIZES = [(12, 200), (40, 200), (600, 1000)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("k", [65600, 262144])
@pytest.mark.parametrize("br,dtype", [(128, torch.float32), (1, torch.float32), (128, torch.bfloat16), (1, torch.bfloat16)])
def test_long_sums_of_one_sign(m, n, k, br, dtype):
    g = torch.Generator(device="cuda").manual_seed(m + k)
    rec = qw.block_quantize(torch.rand(n, k, generator=g, device="cuda"), br)
    xrec = qw.block_quantize(torch.rand(m, k, generator=g, device="cuda"), 1)
    check(qw.block_gemm(rec, xrec, out_dtype=dtype), xrec, rec, k)


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("br", [1, 128])
def test_long_sums_that_lose_every_block(m, n, br):
    """A first block of 25690112 and 2047 of 0.76, less than half of fp32's step of
    2 there: one after another they are all lost, 6e-5 of the sum."""
    k = 262144
    w = torch.full((n, k), 448.0, device="cuda")
    x = torch.full((m, k), 448 * 0.99 * 2.0 ** -25, device="cuda")
    x[:, :128] = 448.0
    rec, xrec = qw.block_quantize(w, br), qw.block_quantize(x, 1)
    worst = check(qw.block_gemm(rec, xrec), xrec, rec, k)
    print("error of the sum", worst, flush=True)


@pytest.mark.parametrize("m", [3, 12, 40, 300])
@pytest.mark.parametrize("xs,ws", [(2.0 ** -50, 2.0 ** -50), (2.0 ** -120, 2.0 ** 20), (2.0 ** 55, 2.0 ** 55), (2.0 ** 120, 2.0 ** -30)])
def test_scales_far_from_1(m, xs, ws):
    g = torch.Generator(device="cuda").manual_seed(m)
    w, x = torch.randn(200, 700, generator=g, device="cuda") * ws, torch.randn(m, 700, generator=g, device="cuda") * xs
    rec, xrec = qw.block_quantize(w, 128), qw.block_quantize(x, 1)
    for dtype in (torch.float32, torch.bfloat16):
        check(qw.block_gemm(rec, xrec, out_dtype=dtype), xrec, rec, 700)
        check(qw.block_matmul(rec, x, out_dtype=dtype), xrec, rec, 700)
