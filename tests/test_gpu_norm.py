"""RMS norm with the residual's addition on the GPU, its quantized outputs and its
gradients, against 64 bits.

Tolerances in units of 2^-24: a lane adds 8 values of every 8 LANES (at most 64 one
after another while a row fits the registers, d / 256 beyond) and the lanes' sums meet
in 8 steps; the sum of squares is off by that at most and its root by half."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw
from oracle import mx as om
from tests.test_gpu_mx import HALF, as_type, host

pytestmark = pytest.mark.gpu

SHAPES = [(1, 1), (3, 7), (5, 64), (4, 500), (2, 513), (9, 1000), (7, 1030), (6, 2048), (5, 2049), (3, 4096), (4, 5003), (2, 8200),
          (3, 16384), (2, 16392), (2, 40001), (1030, 96), (2100, 33)]
TYPES = [torch.float32, torch.bfloat16]


def chain(d):
    return max(64, d / 256) + 8


def inputs(rows, d, dtype, offset=0, seed=0):
    rng = np.random.default_rng([rows, d, seed])
    big = 1 + 15 * (rng.random(d) < 0.02)
    x = as_type((rng.standard_normal((rows, d)) * big).astype(np.float32), dtype, offset)
    res = as_type((rng.standard_normal((rows, d)) * 3).astype(np.float32), dtype, offset)
    w = as_type((1 + 0.1 * rng.standard_normal(d)).astype(np.float32), torch.float32, offset)
    return x, res, w


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("res,weight,offset", [(False, torch.float32, 0), (True, torch.bfloat16, 1), (True, None, 0)])
def test_norm(rows, d, dtype, res, weight, offset):
    print("norm", rows, d, dtype, res, weight, flush=True)
    x, r, w = inputs(rows, d, dtype, offset)
    w = None if weight is None else w.to(weight)
    yt = dtype if offset else torch.float32
    y = as_type(np.full((rows + 1, d), 7, np.float32), yt, offset)
    got, s = qw.rms_norm(x, w, residual=r if res else None, eps=1e-5, out=y[:rows])
    want_s = (x.float() + r.float()).to(dtype) if res else x
    assert torch.equal(s, want_s)
    want = om.norm(host(want_s), None if w is None else host(w), 1e-5)
    tol = (chain(d) / 2 + 8) * 2.0 ** -24 * np.abs(want)
    assert np.all(np.abs(host(got) - want) <= tol + HALF[yt] * (np.abs(want) + tol))
    assert bool((y[rows] == 7).all())


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
def test_quantized_outputs_are_the_codes_of_the_values(rows, d, dtype):
    """The norm's fp32 values, quantized by the calls of their own: the same bits."""
    print("norm codes", rows, d, dtype, flush=True)
    x, r, w = inputs(rows, d, dtype)
    y, s = qw.rms_norm(x, w, residual=r, out_dtype=torch.float32)
    for form, quantize in (("block", lambda v: qw.block_quantize(v, 1)), ("mx", qw.mx_quantize)):
        rec, s2 = qw.rms_norm(x, w, residual=r, quantize=form)
        want = quantize(y)
        assert torch.equal(s, s2) and rec["shape"] == want["shape"]
        assert torch.equal(rec["codes"].view(torch.uint8), want["codes"].view(torch.uint8))
        assert torch.equal(rec["scales"], want["scales"])


@pytest.mark.parametrize("d", [200, 3000, 20000])
def test_the_sum_may_take_an_inputs_place(d):
    for dtype in TYPES:
        x, r, w = inputs(6, d, dtype)
        y, s = qw.rms_norm(x, w, residual=r)
        for place in (0, 1):
            a, b = x.clone(), r.clone()
            y2, s2 = qw.rms_norm(a, w, residual=b, sum=(a, b)[place])
            assert s2 is (a, b)[place] and torch.equal(s2, s) and torch.equal(y2, y)
            assert torch.equal((b, a)[place], (r, x)[place])
        copy = torch.zeros_like(x)
        assert qw.rms_norm(x, w, sum=copy)[1] is copy and torch.equal(copy, x)


@pytest.mark.parametrize("d", [100, 2000, 17000])
def test_rows_of_zeros_infinities_and_nan(d):
    x, _, w = inputs(6, d, torch.float32)
    clean = qw.rms_norm(x, w)[0]
    x[1] = 0.0
    x[2, d // 2] = float("nan")
    x[4, 3] = float("inf")
    y = qw.rms_norm(x, w, eps=1e-6)[0]
    assert torch.equal(y[[0, 3, 5]], clean[[0, 3, 5]]) and not bool(y[1].any())
    assert bool(torch.isnan(y[2]).all()) and bool(torch.isnan(y[4, 3]))
    for form in ("block", "mx"):
        rec = qw.rms_norm(x, w, eps=0.0, quantize=form)[0]  # a row of zeros without eps is NaN, its padding not
        want = qw.rms_norm(x, w, eps=0.0)[0]
        want = qw.block_quantize(want, 1) if form == "block" else qw.mx_quantize(want)
        assert torch.equal(rec["codes"].view(torch.uint8)[:, d:], want["codes"].view(torch.uint8)[:, d:])
        assert torch.equal(rec["scales"].view(torch.uint8), want["scales"].view(torch.uint8))


@pytest.mark.parametrize("d", [100, 2000, 17000])
@pytest.mark.parametrize("by", [2.0 ** -90, 2.0 ** 100])
def test_squares_beyond_fp32(d, by):
    """By a power of two, without eps: the same values."""
    x, _, w = inputs(3, d, torch.float32)
    want, _ = qw.rms_norm(x, w, eps=0.0)
    got, _ = qw.rms_norm(x * by, w, eps=0.0)
    assert bool(want.isfinite().all()) and torch.equal(got, want)


@pytest.mark.parametrize("d", [100, 2000, 17000])
def test_infinite_weights(d):
    """Infinities of the values' sign, NaN for a value of 0, and no harm to others."""
    x, _, w = inputs(3, d, torch.float32)
    x[1, 4], x[2] = 0.0, 1.0
    plain, _ = qw.rms_norm(x, w, out_dtype=torch.float32)
    w[4], w[d - 1] = np.inf, -np.inf
    y, _ = qw.rms_norm(x, w, out_dtype=torch.float32)
    assert torch.equal(y[:, :4], plain[:, :4]) and torch.equal(y[:, 5:-1], plain[:, 5:-1])
    assert np.array_equal(host(y[:, [4, d - 1]]), host(x[:, [4, d - 1]] * w[[4, d - 1]]), equal_nan=True)


@pytest.mark.parametrize("rows,d", SHAPES)
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dsum,weight,offset", [(False, torch.float32, 0), (True, torch.bfloat16, 1), (True, None, 0)])
def test_backward(rows, d, dtype, dsum, weight, offset):
    print("norm backward", rows, d, dtype, dsum, weight, flush=True)
    s, t, w = inputs(rows, d, dtype, offset)
    w = None if weight is None else w.to(weight)
    dy = as_type(np.random.default_rng(d).standard_normal((rows, d)).astype(np.float32), dtype, offset)
    t = t if dsum else None
    ds = as_type(np.full((rows + 1, d), 7, np.float32), dtype, offset)
    got, dw = qw.rms_norm_backward(dy, s, w, eps=1e-5, dsum=t, ds=ds[:rows], dweight=torch.full((d,), 7.0, device="cuda"))
    hy, hs, hw, ht = host(dy), host(s), None if w is None else host(w), None if t is None else host(t)
    want, want_w = om.norm_backward(hy, hs, hw, 1e-5, ht)
    r = 1 / np.sqrt((hs * hs).mean(1, keepdims=True) + 1e-5)
    u = hy if hw is None else hy * hw
    # the mean of u s is off by its chain of the mean of |u s|, r by half, r^3 by 1.5 of it
    tol = (3 * chain(d) + 16) * 2.0 ** -24 * (np.abs(r * u) + np.abs(hs) * r ** 3 * np.abs(u * hs).mean(1, keepdims=True))
    if ht is not None:
        tol = tol + 2.0 ** -24 * np.abs(want)
    assert np.all(np.abs(host(got) - want) <= tol + HALF[dtype] * (np.abs(want) + tol))
    assert bool((ds[rows] == 7).all())
    # every row's term within its r, and at most rows + 8 additions one after another
    tol = (chain(d) / 2 + 16 + rows) * 2.0 ** -24 * np.abs(hy * hs * r).sum(0)
    assert np.all(np.abs(host(dw) - want_w) <= tol)
    again, dw2 = qw.rms_norm_backward(dy, s, w, eps=1e-5, dsum=t)
    assert torch.equal(again, got) and (dw2 is None if w is None else torch.equal(dw2, dw))


@pytest.mark.parametrize("d", [70, 1500, 17000])
def test_backward_in_place(d):
    s, t, w = inputs(5, d, torch.bfloat16)
    dy = torch.randn(5, d, device="cuda").bfloat16()
    want, _ = qw.rms_norm_backward(dy, s, w, dsum=t)
    for place in (0, 1):
        a, b = dy.clone(), t.clone()
        got, _ = qw.rms_norm_backward(a, s, w, dsum=b, ds=(a, b)[place])
        assert torch.equal(got, want)


def test_backward_against_differences():
    """In 64 bits' differences of the definition, along a few directions."""
    s, t, w = inputs(4, 300, torch.float32)
    dy = torch.randn(4, 300, device="cuda")
    ds, dw = qw.rms_norm_backward(dy, s, w, eps=1e-5)
    hs, hw, hy = host(s), host(w), host(dy)
    rng = np.random.default_rng(1)
    for _ in range(5):
        v, e = rng.standard_normal(hs.shape), 1e-5
        diff = (hy * (om.norm(hs + e * v, hw, 1e-5) - om.norm(hs - e * v, hw, 1e-5))).sum() / (2 * e)
        assert abs((host(ds) * v).sum() - diff) <= 1e-5 * np.abs(host(ds) * v).sum()
        v = rng.standard_normal(hw.shape)
        diff = (hy * (om.norm(hs, hw + e * v, 1e-5) - om.norm(hs, hw - e * v, 1e-5))).sum() / (2 * e)
        assert abs((host(dw) * v).sum() - diff) <= 1e-5 * np.abs(host(dw) * v).sum()


def test_empty():
    x = torch.zeros(0, 40, device="cuda")
    assert qw.rms_norm(x)[0].shape == (0, 40) and qw.rms_norm(x, quantize="mx")[0]["shape"] == [0, 40]
    ds, dw = qw.rms_norm_backward(x, x, torch.ones(40, device="cuda"))
    assert ds.shape == (0, 40) and not bool(dw.any())
    x = torch.zeros(5, 0, device="cuda")
    assert qw.rms_norm(x)[0].shape == (5, 0)
    ds, dw = qw.rms_norm_backward(x, x, torch.ones(0, device="cuda"))
    assert ds.shape == (5, 0) and dw.shape == (0,)
