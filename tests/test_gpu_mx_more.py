"""4-bit codes and gated products on the GPU where tests/test_gpu_mx.py says nothing: rows of
codes behind NaN, large weights of the quantizer, the gated product's sums beyond 32-bit
offsets, gates far from zero within a few ulp."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw
from oracle import mx as om
from tests.test_gpu_mx import HALF, bar_of, bytes_of, host, value

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,f,k", [(5, 700, 300), (9, 1, 40), (70, 33, 640), (300, 700, 513), (1030, 600, 260), (700, 1300, 1100), (2500, 4200, 70), (2051, 515, 2100)])
def test_gated_codes_of_rows_with_nan(m, f, k):
    """A row of NaN, one of infinities: NaN blocks up to f, and the padding that every row has."""
    print("gated codes", m, f, k, qw.qw_mx_debug_path(2, m, f, k), flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + f + k)
    rec = qw.mx_quantize(torch.randn(2 * f, k, generator=g, device="cuda") * k ** -0.5)
    x = torch.randn(m, k, generator=g, device="cuda")
    x[1, ::32] = float("nan")
    x[m - 1, 3] = float("inf")
    xrec = qw.mx_quantize(x)
    got = qw.mx_gated(rec, xrec, quantize=True)
    scales, codes, blocks = bytes_of(got["scales"]), bytes_of(got["codes"]), -(-f // 32)
    for row in (1, m - 1):
        assert np.all(scales[row, :blocks] == 255) and not codes[row].any()
    assert np.all(scales[:, blocks:] == 127) and not codes[:, 16 * blocks:].any()
    if m > 64:  # the same sums as the values'
        want = qw.mx_quantize(qw.mx_gated(rec, xrec))
        assert torch.equal(got["scales"], want["scales"]) and torch.equal(got["codes"], want["codes"])


@pytest.mark.parametrize("n,k", [(4100, 4100), (1030, 16388), (131101, 132)])
def test_large_weights_as_their_parts(n, k):
    """fp32 weights of 16 million values and more, whose rows go past the caches: the codes of
    the rows in calls of their own."""
    g = torch.Generator(device="cuda").manual_seed(n)
    w = torch.randn(n, k, generator=g, device="cuda") * torch.exp2(torch.randint(-30, 30, (n, 1), generator=g, device="cuda").float())
    w[n // 2, k // 2], w[n - 1, k - 1], w[7] = float("nan"), float("inf"), 0.0
    assert n * k >= 16 << 20
    rec = qw.mx_quantize(w)
    step = n // 5
    for i in range(0, n, step):
        part = qw.mx_quantize(w[i:i + step])
        assert torch.equal(rec["codes"][i:i + step], part["codes"]) and torch.equal(rec["scales"][i:i + step], part["scales"])
    codes, scales = om.quantize(w[-3:].cpu().numpy())
    assert np.array_equal(bytes_of(rec["codes"][-3:]), codes) and np.array_equal(bytes_of(rec["scales"][-3:]), scales)


def test_gated_products_behind_4_gib():
    """gate and up rows beyond 2^32 bytes of codes: the last 200 of each, all others zero."""
    n, k = 1 << 20, 9000
    f, kp = n // 2, om.pitch(k)
    codes = torch.zeros(n, kp // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, kp // 32), 127, dtype=torch.uint8, device="cuda")
    part = qw.mx_quantize(torch.randn(400, k, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") * k ** -0.5)
    for half in (0, 1):
        rows = slice(half * f + f - 200, half * f + f)
        codes[rows], scales[rows] = part["codes"][200 * half:200 * half + 200], part["scales"][200 * half:200 * half + 200]
    assert codes.numel() > 1 << 32
    rec, wv = dict(bits=4, block=32, shape=[n, k], codes=codes, scales=scales), qw.mx_unpack(part).double()
    for m in (3, 70, 300):
        print("gated behind 4 GiB", m, [qw.qw_mx_debug_path(op, m, f, k) for op in (1, 2, 3)], flush=True)
        xrec = qw.mx_quantize(torch.randn(m, k, device="cuda"))
        xv = qw.mx_unpack(xrec).double()
        p, bar = xv @ wv.T, bar_of(k) * (xv.abs() @ wv.abs().T)
        gate, up, eg, eu = p[:, :200], p[:, 200:], bar[:, :200], bar[:, 200:]
        t = torch.sigmoid(gate)
        silu, want = gate * t, gate * t * up
        tol = 1.1 * eg * (up.abs() + eu) + silu.abs() * eu + 8 * 2.0 ** -23 * want.abs()
        near = lambda got, ref, tol: bool(((got.double() - ref).abs() <= tol + HALF[got.dtype] * (ref.abs() + tol)).all())  # noqa: E731
        h = qw.mx_gated(rec, xrec, out_dtype=torch.bfloat16)
        assert not bool(h[:, :-200].any()) and near(h[:, -200:], want, tol)
        del h
        got = qw.mx_gated(rec, xrec, quantize=True)
        assert not bool((got["codes"][:, :-128] & 0x77).any())
        last = dict(bits=4, block=32, shape=[m, 512], codes=got["codes"][:, -256:].contiguous(), scales=got["scales"][:, -16:].contiguous())
        s = torch.exp2(last["scales"].double() - 127).repeat_interleave(32, 1)[:, -200:]
        assert bool(((qw.mx_unpack(last)[:, -200:].double() - want).abs() <= torch.maximum(want.abs(), s) / 4 * (1 + 1e-4) + tol).all())
        del got
        dh = torch.randn(m, f, device="cuda").bfloat16()
        d, h = qw.mx_gated_backward(rec, xrec, dh)
        a = dh[:, -200:].double()
        tg = a.abs() * (1.1 * eu + 0.5 * eg * (up.abs() + eu) + 10 * 2.0 ** -23 * up.abs())
        tu = a.abs() * (1.1 * eg + 8 * 2.0 ** -23 * gate.abs())
        assert near(h[:, -200:], want, tol) and near(d[:, f - 200:f], a * up * t * (1 + gate * (1 - t)), tg) and near(d[:, -200:], a * silu, tu)
        assert not bool(d[:, :f - 200].any()) and not bool(d[:, f:-200].any())
        del d, h, dh


@pytest.mark.parametrize("m", [5, 300])
def test_far_gates_within_a_few_ulp(m):
    """In units of 2^-23: 2^x 1, its second part 0.5, the sum 0.5 and the reciprocal 1, products
    0.5 each.  The forward's silu 4 with the product by up; the gradients' t = e / (1 + e) 4.5, so
    silu 5 and what it is multiplied with 5.5; of 1 + gate (1 - t) the second term 3, which at
    gate = -1 is 2.7 times the result: 4.5 + 8.5 and three products."""
    gates = np.array([0.0, 1e-30, 1e-3, -1e-3, 1.0, -1.0, 6.0, -6.0, 12.0, -12.0, 24.0, -24.0, 32.0, -32.0, 48.0, -48.0, 64.0, -64.0, -80.0, 96.0,
                      1e4, -1e4, 1e30, -1e30], np.float32)
    f = len(gates)
    w = np.zeros((2 * f, 128), np.float32)
    for at, part in ((0, 1.0), (64, 2.0 ** -5), (96, 2.0 ** -11)):  # gates that no code is: sums of three, exact in fp32
        w[:f, at] = gates * np.float32(part)
    w[f:, 32] = 2.0
    rec = qw.mx_quantize(torch.from_numpy(w).cuda())
    x = torch.zeros(m, 128, device="cuda")
    x[:, ::32] = 1.0
    xrec = qw.mx_quantize(x)
    gate, up = value(rec)[:f].sum(1), np.full(f, 2.0)
    dh = torch.full((m, f), 3.0, device="cuda")
    got, h = qw.mx_gated_backward(rec, xrec, dh)
    dg, du = om.gated_backward(gate, up, np.full(f, 3.0))
    for a, want, ulps in ((host(got)[:, :f], dg, 15), (host(got)[:, f:], du, 5.5), (host(h), om.gated(gate, up), 5.5),
                          (host(qw.mx_gated(rec, xrec)), om.gated(gate, up), 4)):
        assert np.all(np.abs(a - want) <= np.abs(want) * 2.0 ** -23 * ulps)
