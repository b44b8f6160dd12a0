"""Microscaled 4-bit codes and products on the GPU: codes and scales bit for bit,
products within qw_mx.h's bound, (4 + k / 64) 2^-23 of sum |x w|, and half a step of
y's type.

The bound: every matrix instruction adds 64 products to the accumulator with an error
of at most 2^-23 of all their magnitudes, k / 64 of them one after the other, and
where waves share k their few sums are added up."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw
from oracle import mx as om

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def host(t):
    return t.detach().cpu().double().numpy()


def bytes_of(t):
    return t.view(torch.uint8).cpu().numpy()


def wide(seed, n, k):
    """Values over many magnitudes, with zero blocks and large channels."""
    rng = np.random.default_rng(seed)
    w = rng.standard_normal((n, k)) * np.exp(rng.uniform(-8, 8, (n, 1))) * np.exp(2 * rng.standard_normal((1, k)))
    w[rng.random((n, k)) < 0.05] = 0.0
    if n > 2:
        w[1] = 0.0
    return w.astype(np.float32)


def as_type(a, dtype, offset=0):
    """A contiguous device tensor of `dtype`, `offset` elements into its memory."""
    t = torch.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)
    m = torch.empty(t.numel() + offset, dtype=dtype, device="cuda")
    m[offset:] = t.reshape(-1)
    return m[offset:].view(t.shape)


def same_codes(rec, w):
    codes, scales = om.quantize(w)
    assert rec["shape"] == list(w.shape)
    assert np.array_equal(bytes_of(rec["scales"]), scales)
    assert np.array_equal(bytes_of(rec["codes"]), codes)


def value(rec):
    return om.values(bytes_of(rec["codes"]), bytes_of(rec["scales"]), rec["shape"][1])


# ---------------------------------------------------------------- codes


@pytest.mark.parametrize("size", [2.0 ** -126, 2.0 ** -100, 1.0, 2.0 ** 40, 2.0 ** 125])
def test_every_code(size):
    """Codes, their midpoints with neighbours, values beyond the largest code; both signs."""
    mid = ((om.VALUES[1:] + om.VALUES[:-1]) / 2).astype(np.float32)
    v = np.concatenate([om.VALUES, mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(9)),
                        [6.5, 7.0, np.nextafter(np.float32(8), np.float32(0)), 0.2, 1e-3, 1e-30]]).astype(np.float32)
    v = np.concatenate([v, -v])
    v = np.pad(v, (0, -len(v) % 31)).reshape(-1, 31)
    w = np.concatenate([np.full((len(v), 1), 4, np.float32), v], axis=1) * np.float32(size)
    w = w.reshape(1, -1)
    rec = qw.mx_quantize(torch.from_numpy(w).cuda())
    same_codes(rec, w)
    assert np.array_equal(host(qw.mx_unpack(rec)), value(rec))


SHAPES = [(1, 1), (1, 31), (3, 33), (5, 512), (7, 513), (130, 1000), (257, 72), (64, 2056), (513, 130), (300, 4101)]


@pytest.mark.parametrize("n,k", SHAPES)
@pytest.mark.parametrize("transpose", [False, True])
@pytest.mark.parametrize("dtype,offset", [(torch.float32, 0), (torch.float32, 1), (torch.bfloat16, 0), (torch.bfloat16, 3)])
def test_quantize_and_unpack(n, k, transpose, dtype, offset):
    w = as_type(wide([n, k], n, k), dtype, offset)
    rec = qw.mx_quantize(w, transpose=transpose)
    v = w.float().cpu().numpy()
    same_codes(rec, v.T if transpose else v)
    out = as_type(np.full(rec["shape"], np.nan, np.float32), torch.float32, offset)
    assert qw.mx_unpack(rec, out=out) is out
    assert np.array_equal(host(out), value(rec))


@pytest.mark.parametrize("size", [3.4e38, 1.0, 1e-30, 2.0 ** -124, 2.0 ** -126, 1e-40, 2.0 ** -149])
def test_quantize_extreme_magnitudes(size):
    rng = np.random.default_rng(3)
    w = (rng.uniform(-1, 1, (4, 256)) * size).astype(np.float32)
    w[:, ::32] = size
    rec = qw.mx_quantize(torch.from_numpy(w).cuda())
    same_codes(rec, w)
    assert np.array_equal(host(qw.mx_unpack(rec)), value(rec))
    same_codes(qw.mx_quantize(torch.from_numpy(w).cuda(), transpose=True), w.T)


def test_infinities_and_nan_take_their_block():
    w = wide(4, 70, 200)
    w[3, 40], w[5, 64], w[9, 199], w[60, 0] = np.nan, np.inf, -np.inf, np.nan
    for transpose in (False, True):
        rec = qw.mx_quantize(torch.from_numpy(w).cuda(), transpose=transpose)
        same_codes(rec, w.T if transpose else w)
        got = host(qw.mx_unpack(rec))
        assert np.array_equal(np.isnan(got), np.isnan(value(rec))) and np.isnan(got).sum() >= 3 * 8
    y = qw.mx_matmul(qw.mx_quantize(torch.randn(50, 200, device="cuda")), torch.from_numpy(w).cuda())
    assert torch.isnan(y).all(1).nonzero()[:, 0].tolist() == [3, 5, 9, 60] and int(torch.isnan(y).sum()) == 200


def test_scales_at_the_ends():
    """Scale bytes that the quantizer never writes are read as what they stand for."""
    codes = torch.randint(0, 256, (256, 256), dtype=torch.uint8, device="cuda")
    scales = torch.arange(256, device="cuda").to(torch.uint8)[:, None].repeat(1, 16).contiguous()
    rec = dict(bits=4, block=32, shape=[256, 512], codes=codes, scales=scales)
    got, want = qw.mx_unpack(rec).cpu().numpy(), value(rec)
    with np.errstate(over="ignore"):
        assert np.array_equal(got, want.astype(np.float32), equal_nan=True)
    typed = dict(rec, codes=codes.view(torch.float4_e2m1fn_x2), scales=scales.view(torch.float8_e8m0fnu))
    assert np.array_equal(qw.mx_unpack(typed).cpu().numpy(), got, equal_nan=True)


# ---------------------------------------------------------------- products


def bar_of(k):
    return (4 + k / 64) * 2.0 ** -23


def check_product(y, xv, wv):
    """y against 64-bit values, within the bar and half a step of its type."""
    ref, base = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    err, bar = np.abs(host(y) - ref), bar_of(xv.shape[1]) * base
    assert np.all(err <= bar + HALF[y.dtype] * (np.abs(ref) + bar)), float((err - bar).max())


SIZES = [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 17, 129), (3, 1000, 300), (5, 16, 5000), (7, 4096, 130), (8, 333, 1024),
         (15, 128, 4096), (16, 257, 2048), (17, 96, 640), (31, 200, 1000), (32, 100, 512), (33, 513, 256), (63, 64, 1152), (64, 1000, 384),
         (65, 65, 257), (100, 4096, 512), (127, 300, 128), (128, 256, 896), (129, 1025, 1000), (200, 2048, 640), (256, 256, 128),
         (257, 511, 384), (300, 2304, 1280), (1000, 130, 100), (513, 4097, 333), (4, 50, 13000), (20, 40, 9001), (12, 9, 40000)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gemm(m, n, k, dtype):
    print("gemm", m, n, k, dtype, flush=True)
    big = n * k > 1 << 21
    w = np.random.default_rng(n + k).standard_normal((n, k), dtype=np.float32) if big else wide([m, n, k], n, k)
    rec = qw.mx_quantize(torch.from_numpy(w).cuda())
    x = torch.from_numpy(wide([k, m], m, k)).cuda()
    xrec = qw.mx_quantize(x)
    y = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
    qw.mx_gemm(rec, xrec, out=y[:m], out_dtype=dtype)
    check_product(y[:m], value(xrec), value(rec))
    assert bool((y[m] == 7).all())
    assert torch.equal(qw.mx_gemm(rec, xrec, out_dtype=dtype), y[:m])


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("xt,yt,offset", [(torch.float32, torch.float32, 0), (torch.bfloat16, torch.bfloat16, 0),
                                          (torch.float32, torch.bfloat16, 1), (torch.bfloat16, torch.float32, 1)])
def test_matmul(m, n, k, xt, yt, offset):
    print("matmul", m, n, k, xt, yt, flush=True)
    w = np.random.default_rng(n + k).standard_normal((n, k), dtype=np.float32)
    rec = qw.mx_quantize(torch.from_numpy(w).cuda())
    x = as_type(wide([k, m], m, k), xt, offset)
    y = as_type(np.full((m, n), np.nan, np.float32), yt, offset)
    assert qw.mx_matmul(rec, x, out=y) is y
    check_product(y, value(qw.mx_quantize(x)), value(rec))
    assert qw.mx_matmul(rec, x).dtype == xt


# whole and ragged large tiles, a last round that is partly filled
LARGE = [(600, 3000, 260), (1000, 5000, 500), (4096, 4096, 256), (2100, 4000, 200), (2048, 8300, 1000), (40, 4096, 1000), (60, 2048, 4000),
         (1025, 16385, 513)]


@pytest.mark.parametrize("m,n,k", LARGE)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gemm_large(m, n, k, dtype):
    print("gemm", m, n, k, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    make = lambda r, c: torch.randn(r, c, generator=g, device="cuda") * torch.rand(c, generator=g, device="cuda").exp()  # noqa: E731
    rec, x = qw.mx_quantize(make(n, k)), make(m, k)
    xrec = qw.mx_quantize(x)
    y = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
    qw.mx_gemm(rec, xrec, out=y[:m], out_dtype=dtype)
    xv, wv = qw.mx_unpack(xrec).double(), qw.mx_unpack(rec).double()
    ref, bar = xv @ wv.T, bar_of(k) * (xv.abs() @ wv.abs().T)
    assert bool(((y[:m].double() - ref).abs() <= bar + HALF[dtype] * (ref.abs() + bar)).all())
    assert bool((y[m] == 7).all())
    assert torch.equal(qw.mx_matmul(rec, x, out_dtype=dtype), y[:m])


@pytest.mark.parametrize("m", [1, 9, 40, 150, 300])
def test_empty_sums_and_empty_sides(m):
    for dtype in (torch.float32, torch.bfloat16):
        rec = qw.mx_quantize(torch.zeros(70, 0, device="cuda"))
        y = torch.full((m, 70), 7.0, dtype=dtype, device="cuda")
        qw.mx_matmul(rec, torch.zeros(m, 0, device="cuda"), out=y)
        assert not bool(y.any())
    rec = qw.mx_quantize(torch.zeros(0, 40, device="cuda"))
    assert qw.mx_matmul(rec, torch.zeros(m, 40, device="cuda")).shape == (m, 0)
    rec = qw.mx_quantize(torch.ones(30, 40, device="cuda"))
    assert qw.mx_matmul(rec, torch.zeros(0, 40, device="cuda")).shape == (0, 30)


def test_rows_do_not_influence_each_other():
    """A row of infinities and NaN leaves the others as they are, and a row has the same
    bits alone as among others of the same call size."""
    rec = qw.mx_quantize(torch.from_numpy(wide(1, 300, 700)).cuda())
    for m in (4, 16, 50, 200, 400):
        x = torch.randn(m, 700, device="cuda")
        y = qw.mx_matmul(rec, x)
        x[m // 2, ::3] = float("nan")
        x[m // 2, 1::3] = float("inf")
        z = qw.mx_matmul(rec, x)
        rest = torch.arange(m, device="cuda") != m // 2
        assert torch.equal(y[rest], z[rest]) and bool(torch.isnan(z[m // 2]).all())


def test_gradients_by_the_documented_calls():
    """dx with the transposed weight's codes, dw of transposed dy and x, against 64 bits."""
    m, n, k = 200, 333, 450
    w, x, dy = (torch.from_numpy(wide(i, *s)).cuda() for i, s in ((1, (n, k)), (2, (m, k)), (3, (m, n))))
    wt, d = qw.mx_quantize(w, transpose=True), qw.mx_quantize(dy)
    check_product(qw.mx_gemm(wt, d), value(d), value(wt))
    xt, dt = qw.mx_quantize(x, transpose=True), qw.mx_quantize(dy, transpose=True)
    dw = qw.mx_gemm(xt, dt)
    assert dw.shape == w.shape
    check_product(dw, value(dt), value(xt))


# ---------------------------------------------------------------- gated product


def gated_case(m, f, k, seed=0):
    rng = np.random.default_rng([m, f, k, seed])
    w = (rng.standard_normal((2 * f, k)) * k ** -0.5).astype(np.float32)
    x = (rng.standard_normal((m, k)) * (1 + 15 * (rng.random(k) < 0.01))).astype(np.float32)
    rec, xrec = qw.mx_quantize(torch.from_numpy(w).cuda()), qw.mx_quantize(torch.from_numpy(x).cuda())
    wv, xv = value(rec), value(xrec)
    gate, up = xv @ wv[:f].T, xv @ wv[f:].T
    base = bar_of(k) * (np.abs(xv) @ np.abs(wv).T)
    return rec, xrec, gate, up, base[:, :f], base[:, f:]


GATED = [(1, 1, 1), (1, 128, 256), (3, 33, 100), (4, 1408, 1024), (16, 65, 520), (17, 200, 300), (33, 96, 640), (70, 130, 1000),
         (128, 512, 256), (200, 1000, 333), (300, 700, 513), (1030, 600, 260), (513, 2600, 300), (2, 40, 9001)]


@pytest.mark.parametrize("m,f,k", GATED)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gated(m, f, k, dtype):
    print("gated", m, f, k, dtype, flush=True)
    rec, xrec, gate, up, eg, eu = gated_case(m, f, k)
    h = torch.full((m + 1, f), 7.0, dtype=dtype, device="cuda")
    assert qw.mx_gated(rec, xrec, out=h[:m]).dtype == dtype
    want, silu = om.gated(gate, up), gate * om.sigmoid(gate)
    # |silu'| <= 1.1; silu and the product with up within 8 ulp
    tol = 1.1 * eg * (np.abs(up) + eu) + np.abs(silu) * eu + 8 * 2.0 ** -23 * np.abs(want)
    assert np.all(np.abs(host(h[:m]) - want) <= tol + HALF[dtype] * (np.abs(want) + tol))
    assert bool((h[m] == 7).all())


@pytest.mark.parametrize("m,f,k", GATED)
def test_gated_codes(m, f, k):
    """The codes of the values: of more than 64 rows, whose floats have the same sums, bit
    for bit; of fewer, whose floats are summed in another order, within half a step."""
    print("gated codes", m, f, k, flush=True)
    rec, xrec = gated_case(m, f, k)[:2]
    got, h = qw.mx_gated(rec, xrec, quantize=True), qw.mx_gated(rec, xrec)
    want = qw.mx_quantize(h)
    assert got["shape"] == [m, f]
    if m > 64:
        assert torch.equal(got["scales"], want["scales"]) and torch.equal(got["codes"], want["codes"])
    s = np.repeat(2.0 ** (bytes_of(got["scales"]).astype(np.float64) - 127), 32, 1)[:, :f]
    assert np.all(np.abs(value(got) - host(h)) <= np.maximum(np.abs(host(h)), s) / 4 * (1 + 1e-4))
    kp = om.pitch(f)
    assert not bytes_of(got["codes"])[:, -(-f // 32) * 16:].any() and np.all(bytes_of(got["scales"])[:, -(-f // 32):kp // 32] == 127)


@pytest.mark.parametrize("m,f,k", GATED)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_gated_backward(m, f, k, dtype):
    print("gated backward", m, f, k, dtype, flush=True)
    rec, xrec, gate, up, eg, eu = gated_case(m, f, k)
    dh = torch.from_numpy(wide([f, m], m, f)).cuda().to(dtype)
    out = torch.full((m + 1, 2 * f), 7.0, dtype=dtype, device="cuda")
    got, h = qw.mx_gated_backward(rec, xrec, dh, out=out[:m])
    d, (dg, du) = np.abs(host(dh)), om.gated_backward(gate, up, host(dh))
    # |silu'| <= 1.1, |silu''| <= 0.5; the gate's factor within 8 ulp of its terms (1.2 at most)
    tg = d * (1.1 * eu + 0.5 * eg * (np.abs(up) + eu) + 10 * 2.0 ** -23 * np.abs(up))
    tu = d * (1.1 * eg + 8 * 2.0 ** -23 * np.abs(gate))
    for a, want, tol in ((got[:, :f], dg, tg), (got[:, f:], du, tu)):
        assert np.all(np.abs(host(a) - want) <= tol + HALF[dtype] * (np.abs(want) + tol) + 2.0 ** -149)
    assert bool((out[m] == 7).all())
    # h: within half a step of the forward's fp32 values, which have the same sums
    want = qw.mx_gated(rec, xrec)
    assert bool(((h.double() - want.double()).abs() <= (HALF[dtype] + 10 * 2.0 ** -23) * want.double().abs() + 2.0 ** -140).all())
    again, none = qw.mx_gated_backward(rec, xrec, dh, h=False)
    assert none is None and torch.equal(again, got)


@pytest.mark.parametrize("m", [5, 300])
def test_far_gates(m):
    """Gates of every size up to 1e30: no overflow inside, gradients zero or exact where silu is flat or a line."""
    gates = np.array([0.0, 1e-30, 1.0, -1.0, 30.0, -30.0, 88.0, -88.0, -104.0, 120.0, -120.0, 1e4, -1e4, 1e30, -1e30], np.float32)
    f = len(gates)
    w = np.zeros((2 * f, 64), np.float32)
    w[:f, 0], w[f:, 32] = gates, 2.0
    rec = qw.mx_quantize(torch.from_numpy(w).cuda())
    x = torch.zeros(m, 64, device="cuda")
    x[:, 0] = x[:, 32] = 1.0
    xrec = qw.mx_quantize(x)
    gate, up = value(rec)[:f, 0], np.full(f, 2.0)
    dh = torch.full((m, f), 3.0, device="cuda")
    got, h = qw.mx_gated_backward(rec, xrec, dh)
    dg, du = om.gated_backward(gate, up, np.full(f, 3.0))
    tiny = 2.0 ** -140
    for a, want in ((host(got)[:, :f], dg), (host(got)[:, f:], du), (host(h), om.gated(gate, up)), (host(qw.mx_gated(rec, xrec)), om.gated(gate, up))):
        # exp's argument is rounded: |gate| half ulps more where exp decides, up to 104
        assert np.all(np.abs(a - want) <= np.abs(want) * 2.0 ** -23 * (16 + np.minimum(np.abs(gate), 104)) + tiny)


@pytest.mark.parametrize("m,d,f", [(1, 64, 40), (4, 512, 1408), (8, 1000, 333), (17, 256, 700), (40, 520, 96), (200, 700, 513), (600, 512, 1300)])
@pytest.mark.parametrize("xt,yt", [(torch.float32, torch.float32), (torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32)])
def test_mlp(m, d, f, xt, yt):
    """Against the calls one by one: the same codes of x; h's codes where its value is
    not within the sums' error of a border."""
    print("mlp", m, d, f, xt, yt, flush=True)
    rng = np.random.default_rng([m, d, f])
    gu = qw.mx_quantize(torch.from_numpy((rng.standard_normal((2 * f, d)) * d ** -0.5).astype(np.float32)).cuda())
    dn = qw.mx_quantize(torch.from_numpy((rng.standard_normal((d, f)) * f ** -0.5).astype(np.float32)).cuda())
    x = torch.from_numpy(rng.standard_normal((m, d)).astype(np.float32)).cuda().to(xt)
    y = torch.full((m + 1, d), 7.0, dtype=yt, device="cuda")
    qw.mx_mlp(gu, dn, x, out=y[:m])
    assert bool((y[m] == 7).all())
    xr = qw.mx_quantize(x)
    hr = qw.mx_gated(gu, xr, quantize=True)
    xv, wv, hv, dv = value(xr), value(gu), value(hr), value(dn)
    gate, up = xv @ wv[:f].T, xv @ wv[f:].T
    base = bar_of(d) * (np.abs(xv) @ np.abs(wv).T)
    tol = 1.1 * base[:, :f] * (np.abs(up) + base[:, f:]) + np.abs(gate) * base[:, f:] + 8 * 2.0 ** -23 * np.abs(om.gated(gate, up))
    # a value may go to the next code if it is that near to a border: a step of its block at most
    s = np.repeat(2.0 ** (bytes_of(hr["scales"]).astype(np.float64) - 127), 32, 1)[:, :f]
    v = np.abs(om.gated(gate, up)) / s
    near = np.min(np.abs(v[..., None] - np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])), -1) <= 2 * tol / s
    top = np.pad(v, ((0, 0), (0, -f % 32))).reshape(m, -1, 32).max(-1)
    edge = np.minimum(np.abs(top - 4), np.abs(top - 8)) <= 1e-3   # another scale: the whole block
    near |= np.repeat(edge, 32, 1)[:, :f]
    ref, base = hv @ dv.T, np.abs(hv) @ np.abs(dv).T
    bar = bar_of(f) * base + (near * 4.0 * s) @ np.abs(dv).T
    assert np.all(np.abs(host(y[:m]) - ref) <= bar + HALF[yt] * (np.abs(ref) + bar))
    assert near.mean() < 0.02


def test_mlp_without_hidden_values():
    gu, dn = qw.mx_quantize(torch.zeros(0, 40, device="cuda")), qw.mx_quantize(torch.zeros(40, 0, device="cuda"))
    for m in (1, 20, 300):
        y = torch.full((m, 40), 7.0, device="cuda")
        qw.mx_mlp(gu, dn, torch.randn(m, 40, device="cuda"), out=y)
        assert not bool(y.any())


# ---------------------------------------------------------------- every kernel

MS = (1, 2, 8, 9, 16, 17, 32, 33, 64, 65, 130, 300, 700, 1500, 2500)
NS = (5, 33, 300, 1100, 2300, 4200, 9000)
KS = (70, 600, 1500, 4097, 8300, 12400, 17000, 21000)


def sizes_of_paths(op):
    """One call (m, n, k) for every kernel that the library reports, the cheapest first."""
    found = {}
    for m, n, k in sorted(((m, n, k) for m in MS for n in NS for k in KS), key=lambda s: s[0] * s[1] * s[2] + s[1] * s[2]):
        found.setdefault(qw.qw_mx_debug_path(op, m, n, k), (m, n, k))
    return found


def gpu_check(y, xrec, rec, bar=None):
    k = rec["shape"][1]
    xv, wv = qw.mx_unpack(xrec).double(), qw.mx_unpack(rec).double()
    ref, bar = xv @ wv.T, bar_of(k) * (xv.abs() @ wv.abs().T)
    assert bool(((y.double() - ref).abs() <= bar + HALF[y.dtype] * (ref.abs() + bar)).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_every_kernel_of_the_product(dtype):
    found = sizes_of_paths(0)
    assert {2, 128064, 128128, 256256} <= set(found) and {101, 102, 103, 104, 105, 201, 202, 203, 401, 402} <= set(found)
    for path, (m, n, k) in found.items():
        print("product", path, m, n, k, dtype, flush=True)
        g = torch.Generator(device="cuda").manual_seed(path)
        w = torch.randn(n, k, generator=g, device="cuda") * torch.rand(k, generator=g, device="cuda").mul(3).exp()
        x = torch.randn(m, k, generator=g, device="cuda")
        rec, xrec = qw.mx_quantize(w), qw.mx_quantize(x)
        y = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
        qw.mx_gemm(rec, xrec, out=y[:m], out_dtype=dtype)
        gpu_check(y[:m], xrec, rec)
        assert bool((y[m] == 7).all())
        z = qw.mx_matmul(rec, x.to(dtype), out_dtype=dtype)
        gpu_check(z, qw.mx_quantize(x.to(dtype)), rec)


@pytest.mark.parametrize("op", [1, 2, 3])
def test_every_kernel_of_the_gated_product(op):
    found = sizes_of_paths(op)
    assert {2, 128064, 128128, 256256} <= set(found)
    assert op > 1 or {101, 102, 103, 104, 201, 202, 401} <= set(found)
    for path, (m, f, k) in found.items():
        print("gated", op, path, m, f, k, flush=True)
        g = torch.Generator(device="cuda").manual_seed(path)
        rec = qw.mx_quantize(torch.randn(2 * f, k, generator=g, device="cuda") * k ** -0.5)
        xrec = qw.mx_quantize(torch.randn(m, k, generator=g, device="cuda"))
        xv, wv = qw.mx_unpack(xrec).double(), qw.mx_unpack(rec).double()
        p, bar = xv @ wv.T, bar_of(k) * (xv.abs() @ wv.abs().T)
        gate, up, eg, eu = p[:, :f], p[:, f:], bar[:, :f], bar[:, f:]
        t = torch.sigmoid(gate)
        silu = gate * t
        want = silu * up
        tol = 1.1 * eg * (up.abs() + eu) + silu.abs() * eu + 8 * 2.0 ** -23 * want.abs()
        if op == 1:
            h = qw.mx_gated(rec, xrec).double()
            assert bool(((h - want).abs() <= tol + HALF[torch.float32] * want.abs()).all())
        elif op == 2:
            got = qw.mx_gated(rec, xrec, quantize=True)
            s = torch.exp2(got["scales"].double() - 127).repeat_interleave(32, 1)[:, :f]
            assert bool(((qw.mx_unpack(got).double() - want).abs() <= torch.maximum(want.abs(), s) / 4 * (1 + 1e-4) + tol).all())
        else:
            dh = torch.randn(m, f, generator=g, device="cuda")
            d, h = qw.mx_gated_backward(rec, xrec, dh)
            a = dh.double().abs()
            assert bool(((h.double() - want).abs() <= tol + HALF[torch.float32] * want.abs()).all())
            dg = dh.double() * up * t * (1 + gate * (1 - t))
            tg = a * (1.1 * eu + 0.5 * eg * (up.abs() + eu) + 10 * 2.0 ** -23 * up.abs())
            assert bool(((d[:, :f].double() - dg).abs() <= tg + HALF[torch.float32] * dg.abs()).all())
            tu = a * (1.1 * eg + 8 * 2.0 ** -23 * gate.abs())
            assert bool(((d[:, f:].double() - dh.double() * silu).abs() <= tu + HALF[torch.float32] * (dh.double() * silu).abs()).all())


def test_matmul_quantizes_on_the_way_or_before():
    """Both sides of the choice give the product of the same codes."""
    found = {qw.qw_mx_debug_path(4, m, 300, k): (m, k) for m in (16, 9, 8, 4, 1) for k in (700, 4096, 9000)}
    assert set(found) == {1, 2}
    for m, k in ((1, 700), (8, 700), (9, 700), (16, 4096), (3, 9000), (4, 9000)):
        rec, x = qw.mx_quantize(torch.randn(300, k, device="cuda")), torch.randn(m, k, device="cuda")
        a, b = qw.mx_matmul(rec, x), qw.mx_gemm(rec, qw.mx_quantize(x))
        assert torch.equal(a, b)


# ---------------------------------------------------------------- values far apart


@pytest.mark.parametrize("m", [3, 20, 60, 100, 500])
def test_far_scales(m):
    """Blocks whose scales are up to 2^40 apart, and products near both ends of fp32."""
    g = torch.Generator(device="cuda").manual_seed(m)
    for shift in (0, -60, 50):
        w = torch.randn(200, 1000, generator=g, device="cuda") * torch.exp2(torch.randint(-20, 21, (200, 1000 // 40), generator=g, device="cuda").float() + shift).repeat_interleave(40, 1)
        x = torch.randn(m, 1000, generator=g, device="cuda") * 2.0 ** shift
        rec, xrec = qw.mx_quantize(w), qw.mx_quantize(x)
        gpu_check(qw.mx_gemm(rec, xrec), xrec, rec)


def test_products_are_exact_where_fp32_holds_them():
    """Integer codes whose sums need 20 bits: exact in every kernel."""
    rng = np.random.default_rng(8)
    for m in (1, 20, 60, 100, 600):
        w, x = (rng.choice([-6, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], s).astype(np.float32) for s in ((400, 3100), (m, 3100)))
        w[:, ::32] = 6
        x[:, ::32] = 6
        y = qw.mx_matmul(qw.mx_quantize(torch.from_numpy(w).cuda()), torch.from_numpy(x).cuda())
        assert np.array_equal(host(y), x.astype(np.float64) @ w.T.astype(np.float64))
