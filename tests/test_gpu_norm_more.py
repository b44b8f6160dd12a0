"""RMS norm and its gradients on the GPU where tests/test_gpu_norm.py says nothing: blocks
that take many rows, large rows past the caches, values rounded once, rows of any
magnitude.

Bars of the gradients: those of tests/test_gpu_norm.py."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw
from oracle import mx as om
from tests.test_gpu_mx import HALF, as_type, host
from tests.test_gpu_norm import TYPES, chain, inputs

pytestmark = pytest.mark.gpu


def check_backward(dy, s, w, t, eps, got, dw):
    rows, d = s.shape
    hy, hs, hw, ht = host(dy), host(s), None if w is None else host(w), None if t is None else host(t)
    want, want_w = om.norm_backward(hy, hs, hw, eps, ht)
    r = 1 / np.sqrt((hs * hs).mean(1, keepdims=True) + eps)
    u = hy if hw is None else hy * hw
    tol = (3 * chain(d) + 16) * 2.0 ** -24 * (np.abs(r * u) + np.abs(hs) * r ** 3 * np.abs(u * hs).mean(1, keepdims=True))
    if ht is not None:
        tol = tol + 2.0 ** -24 * np.abs(want)
    # below 2^-126 a step is the type's smallest value, 2^-149 or 2^-133, however small the result
    step = 2.0 ** -149 if s.dtype == torch.float32 else 2.0 ** -133
    assert np.all(np.abs(host(got) - want) <= tol + HALF[s.dtype] * (np.abs(want) + tol) + step / 2)
    tol = (chain(d) / 2 + 16 + rows) * 2.0 ** -24 * np.abs(hy * hs * r).sum(0)
    assert np.all(np.abs(host(dw) - want_w) <= tol)


# more rows than the 768 or 1024 blocks, so that a block adds up the weight gradients of some
@pytest.mark.parametrize("rows,d", [(2500, 1030), (1700, 1030), (1600, 2049), (1600, 5003), (900, 8192), (1600, 8200), (1100, 16392), (4099, 600)])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("dsum,offset", [(False, 0), (True, 1)])
def test_backward_of_many_rows(rows, d, dtype, dsum, offset):
    print("norm backward", rows, d, dtype, dsum, flush=True)
    s, t, w = inputs(rows, d, dtype, offset)
    dy = as_type(np.random.default_rng(d).standard_normal((rows, d)).astype(np.float32), dtype, offset)
    t = t if dsum else None
    ds = as_type(np.full((rows + 1, d), 7, np.float32), dtype, offset)
    got, dw = qw.rms_norm_backward(dy, s, w, eps=1e-5, dsum=t, ds=ds[:rows], dweight=torch.full((d,), 7.0, device="cuda"))
    check_backward(dy, s, w, t, 1e-5, got, dw)
    assert bool((ds[rows] == 7).all())
    again, dw2 = qw.rms_norm_backward(dy, s, w, eps=1e-5, dsum=t)
    assert torch.equal(again, got) and torch.equal(dw2, dw)


@pytest.mark.parametrize("rows,d", [(65600, 256), (16400, 1024), (8200, 2056), (4100, 4104), (2100, 8200), (1030, 16384)])
def test_large_bf16_rows_as_their_parts(rows, d):
    """16 million values and more, which go past the caches: the results of some rows in calls
    of their own."""
    print("norm", rows, d, flush=True)
    assert rows * d >= 16 << 20
    g = torch.Generator(device="cuda").manual_seed(d)
    x, res = (torch.randn(rows, d, generator=g, device="cuda").mul_(3).bfloat16() for _ in range(2))
    w = 1 + 0.1 * torch.randn(d, generator=g, device="cuda")
    for form in (None, "block", "mx"):
        y, s = qw.rms_norm(x, w, residual=res, quantize=form)
        for i in range(0, rows, rows // 5):
            part = slice(i, i + rows // 5)
            yp, sp = qw.rms_norm(x[part], w, residual=res[part], quantize=form)
            assert torch.equal(s[part], sp)
            if form is None:
                assert torch.equal(y[part], yp)
            else:
                assert torch.equal(y["codes"][part].view(torch.uint8), yp["codes"].view(torch.uint8)) and torch.equal(y["scales"][part], yp["scales"])


@pytest.mark.parametrize("rows,d", [(3, 7), (5, 500), (4, 1000), (7, 1030), (3, 4096), (4, 5003), (2, 16384), (2, 40001), (1030, 96)])
@pytest.mark.parametrize("dtype", TYPES)
def test_values_are_rounded_once(rows, d, dtype):
    """y in fp32: half a step of it, and what s r's rest and its product with the weight leave, 2^-47."""
    x, res, w = inputs(rows, d, dtype)
    for weight in (w, w.bfloat16(), None):
        y, s = qw.rms_norm(x, weight, residual=res, eps=1e-5, out_dtype=torch.float32)
        want = om.norm(host(s), None if weight is None else host(weight), 1e-5)
        assert np.all(np.abs(host(y) - want) <= 2.0 ** -24 * (1 + 2.0 ** -20) * np.abs(want))


def rows_of_any_size(d, dtype, powers, seed):
    """Rows of normal values times a power of two each, as dtype holds them."""
    rng = np.random.default_rng([d, seed])
    return torch.from_numpy((rng.standard_normal((len(powers), d)) * 2.0 ** np.array(powers, float)[:, None]).astype(np.float32)).cuda().to(dtype)


# fp32's subnormal values begin below 2^-126; normal ones times 2^125 end below its largest
POWERS = [0, -146, -140, -132, -128, -120, -90, -60, -30, 30, 60, 90, 124, 125]


@pytest.mark.parametrize("d", [100, 900, 2000, 17000])
@pytest.mark.parametrize("dtype", TYPES)
def test_rows_over_the_range_of_r(d, dtype):
    """Without eps, so that y has no magnitude of its own left.  Rounded once up to 2^100; beyond, r's
    second part and then bits of its first are below fp32's smallest value, 2^-150 of 2^-128 at
    most; below 2^-128 r is infinite."""
    x = rows_of_any_size(d, dtype, POWERS, 1)
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    y, _ = qw.rms_norm(x, w, eps=0.0, out_dtype=torch.float32)
    with np.errstate(divide="ignore", invalid="ignore"):  # bf16 has no values in the smallest rows
        want = om.norm(host(x), host(w), 0.0)
    for i, p in enumerate(POWERS):
        if -126 < p < 128:
            bar = (2.0 ** -24 + (2.0 ** -22 if p > 100 else 0.0)) * (1 + 2.0 ** -20) * np.abs(want[i])
            assert np.all(np.abs(host(y[i]) - want[i]) <= bar)
        elif p < -130:
            assert not bool(y[i].isfinite().any())
    for form, quantize in (("block", lambda v: qw.block_quantize(v, 1)), ("mx", qw.mx_quantize)):
        got, want = qw.rms_norm(x, w, eps=0.0, quantize=form)[0], quantize(y)
        assert torch.equal(got["scales"].view(torch.uint8), want["scales"].view(torch.uint8))
        assert torch.equal(got["codes"].view(torch.uint8), want["codes"].view(torch.uint8))


@pytest.mark.parametrize("d", [100, 900, 2000, 5003, 17000])
@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("times", [1, 100])
def test_gradients_of_rows_of_any_magnitude(d, dtype, times):
    """dy 2^-12 of normal values, so that the gradients of the smallest rows are in fp32's range.  A
    row's squares as fp32 holds them would be zero from 2^-75 down and infinite from 2^64 up."""
    powers = [p for p in POWERS if p >= -120] * times
    s = rows_of_any_size(d, dtype, powers, 2)
    dy = rows_of_any_size(d, dtype, [-12] * len(powers), 3)
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    got, dw = qw.rms_norm_backward(dy, s, w, eps=0.0)
    check_backward(dy, s, w, None, 0.0, got, dw)
    # the gradient past the norm of the gradient's own size, in its place
    t = (got.float() * 0.75).to(dtype)
    want, _ = qw.rms_norm_backward(dy, s, w, eps=0.0, dsum=t)
    check_backward(dy, s, w, t, 0.0, want, dw)
    again, dw2 = qw.rms_norm_backward(dy, s, w, eps=0.0, dsum=t, ds=t)
    assert again is t and torch.equal(again, want) and torch.equal(dw2, dw)


@pytest.mark.parametrize("d", [100, 2000, 17000])
@pytest.mark.parametrize("eps", [2.0 ** -100, 2.0 ** -149, 2.0 ** 120])
def test_gradients_with_eps_of_any_magnitude(d, eps):
    """Rows of zeros, rows whose squares are far below eps, near it and above it."""
    e = int(np.log2(eps)) // 2
    powers = [e - 40, e - 3, e, e + 3, e + 40] if e > -70 else [e - 10, e - 3, e, e + 3, e + 40]
    s = rows_of_any_size(d, torch.float32, powers + [0], 4)
    s[-1] = 0.0
    dy = rows_of_any_size(d, torch.float32, [-12] * len(s), 5)
    w = torch.linspace(0.5, 1.5, d, device="cuda")
    got, dw = qw.rms_norm_backward(dy, s, w, eps=eps)
    check_backward(dy, s, w, None, eps, got, dw)


@pytest.mark.parametrize("d", [100, 2000, 17000])
def test_gradients_of_rows_without_values_of_their_own(d):
    """A row of zeros without eps, of an infinity, of a NaN: NaN as the definition has it, and no harm to others."""
    s, _, w = inputs(6, d, torch.float32)
    dy = torch.randn(6, d, device="cuda")
    clean, _ = qw.rms_norm_backward(dy, s, w, eps=0.0)
    s[1], s[2, d // 2], s[4, 3] = 0.0, float("nan"), float("inf")
    got, _ = qw.rms_norm_backward(dy, s, w, eps=0.0)
    assert torch.equal(got[[0, 3, 5]], clean[[0, 3, 5]]) and bool(torch.isnan(got[[1, 2, 4]]).all())
