"""The tiled 4-bit products where a block takes tile after tile: more than four steps of
256 values of k, and more tiles than the chip holds at once, so that the copies of the
next tile run while the results of this one are written.  Every tile that the library
reports, every result, both types, rows and columns that end inside a tile.

Bars: those of tests/test_gpu_mx.py."""

import pytest
import torch

from int8_int4_dequant_amd import qw
from tests.test_gpu_mx import HALF, bar_of, gpu_check

pytestmark = pytest.mark.gpu

# weight rows, tokens and tiles of a compute unit, by the reported kernel
TILES = {256256: (256, 256, 1), 128256: (128, 256, 1), 128128: (128, 128, 2), 128064: (128, 64, 2)}
UNITS = 256
PAIRS = [(257, 11009), (515, 20001), (765, 5435), (777, 5003), (1027, 11009), (1541, 5003), (2051, 515), (2051, 4097), (4099, 515),
         (4099, 6001), (5117, 1595), (5117, 3195), (5629, 1467), (5629, 2939), (8197, 1003), (9469, 827), (9469, 1659)]
KS = (1100, 1285, 2100, 2309, 3333, 4096, 11008, 20000)


def rounds(op, path, m, n):
    """How many tiles there are for every one that the chip holds."""
    bn, bm, each = TILES[path]
    width = bn if op == 0 else bn // 2
    cols = -(-n // 512) * 512 if op == 2 else n  # codes: whole rows of them
    return -(-m // bm) * -(-cols // width) / (UNITS * each)


def sizes(op):
    """The cheapest call of more than a round for every tile, steps of the last chunk of scales and
    parity of the chunks."""
    found = {}
    for m, n, k in sorted(((m, n, k) for m, n in PAIRS for k in KS), key=lambda s: s[0] * s[1] * s[2]):
        path, kb = qw.qw_mx_debug_path(op, m, n, k), -(-k // 256)
        if path in TILES and rounds(op, path, m, n) > 1:
            found.setdefault((path, kb % 4, (kb + 3) // 4 % 2), (m, n, k))
    assert {key[0] for key in found} == set(TILES) and {key[1] for key in found} == {0, 1, 2, 3}
    assert {key[::2] for key in found} >= {(path, p) for path in TILES if path != 128256 for p in (0, 1)}
    return found


def operands(m, n, k):
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    spread = torch.rand(k, generator=g, device="cuda").mul(2).exp()
    rec = qw.mx_quantize(torch.randn(n, k, generator=g, device="cuda") * k ** -0.5 * spread)
    return rec, qw.mx_quantize(torch.randn(m, k, generator=g, device="cuda")), g


def test_products_tile_after_tile():
    for (path, _, _), (m, n, k) in sizes(0).items():
        rec, xrec, _ = operands(m, n, k)
        for dtype in (torch.float32, torch.bfloat16):
            print("product", path, m, n, k, dtype, flush=True)
            y = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
            qw.mx_gemm(rec, xrec, out=y[:m], out_dtype=dtype)
            gpu_check(y[:m], xrec, rec)
            assert bool((y[m] == 7).all())
            assert torch.equal(qw.mx_gemm(rec, xrec, out_dtype=dtype), y[:m])


def terms(rec, xrec, f, k):
    """gate, up and their bars in 64 bits."""
    xv, wv = qw.mx_unpack(xrec).double(), qw.mx_unpack(rec).double()
    p, bar = xv @ wv.T, bar_of(k) * (xv.abs() @ wv.abs().T)
    return p[:, :f], p[:, f:], bar[:, :f], bar[:, f:]


def near(got, want, tol):
    h = HALF[got.dtype]
    return bool(((got.double() - want).abs() <= tol + h * (want.abs() + tol) + 2.0 ** -149).all())


def check_gated(m, f, k):
    rec, xrec, _ = operands(m, 2 * f, k)
    gate, up, eg, eu = terms(rec, xrec, f, k)
    silu = gate * torch.sigmoid(gate)
    want = silu * up
    tol = 1.1 * eg * (up.abs() + eu) + silu.abs() * eu + 8 * 2.0 ** -23 * want.abs()
    for dtype in (torch.float32, torch.bfloat16):
        h = torch.full((m + 1, f), 7.0, dtype=dtype, device="cuda")
        qw.mx_gated(rec, xrec, out=h[:m])
        assert near(h[:m], want, tol) and bool((h[m] == 7).all())


def test_gated_values_tile_after_tile():
    for (path, _, _), (m, f, k) in sizes(1).items():
        print("gated", path, m, f, k, flush=True)
        check_gated(m, f, k)


def test_gated_codes_tile_after_tile():
    """The codes of the values, which are checked beside them: the same bits."""
    for (path, _, _), (m, f, k) in sizes(2).items():
        print("gated codes", path, m, f, k, flush=True)
        check_gated(m, f, k)
        rec, xrec, _ = operands(m, 2 * f, k)
        got, want = qw.mx_gated(rec, xrec, quantize=True), qw.mx_quantize(qw.mx_gated(rec, xrec))
        assert torch.equal(got["scales"], want["scales"]) and torch.equal(got["codes"], want["codes"])


def test_gated_gradients_tile_after_tile():
    for (path, _, _), (m, f, k) in sizes(3).items():
        rec, xrec, g = operands(m, 2 * f, k)
        gate, up, eg, eu = terms(rec, xrec, f, k)
        t = torch.sigmoid(gate)
        silu, want_h = gate * t, gate * t * up
        th = 1.1 * eg * (up.abs() + eu) + silu.abs() * eu + 8 * 2.0 ** -23 * want_h.abs()
        for dtype in (torch.float32, torch.bfloat16):
            print("gated gradients", path, m, f, k, dtype, flush=True)
            dh = torch.randn(m, f, generator=g, device="cuda").to(dtype)
            out = torch.full((m + 1, 2 * f), 7.0, dtype=dtype, device="cuda")
            h = torch.full((m + 1, f), 7.0, dtype=dtype, device="cuda")
            qw.mx_gated_backward(rec, xrec, dh, out=out[:m], h=h[:m])
            a = dh.double()
            tg = a.abs() * (1.1 * eu + 0.5 * eg * (up.abs() + eu) + 10 * 2.0 ** -23 * up.abs())
            tu = a.abs() * (1.1 * eg + 8 * 2.0 ** -23 * gate.abs())
            assert near(out[:m, :f], a * up * t * (1 + gate * (1 - t)), tg)
            assert near(out[:m, f:], a * silu, tu) and near(h[:m], want_h, th)
            assert bool((out[m] == 7).all()) and bool((h[m] == 7).all())
            again, none = qw.mx_gated_backward(rec, xrec, dh, h=False)
            assert none is None and torch.equal(again, out[:m])
