"""Block-scaled e4m3 on the GPU: codes and scales bit for bit, products within
qw.h's bounds (1e-5 of sum |x w| for fp32 y, 1e-3 for bf16 y) plus half a step
of y's type.

The 8-bit cores' bound: they add 8 products at a time, each cut off 2^-13 below
the largest of the 8, so that 7 products lose 7 * 2^-13 = 8.6e-4 of it at most,
and the largest is at most the 8 products' sum of magnitudes."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw
from oracle import block as ob

pytestmark = pytest.mark.gpu

BAR = {torch.float32: 1e-5, torch.bfloat16: 1e-3}
HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def host(t):
    return t.detach().cpu().double().numpy()


def codes_of(rec):
    return rec["codes"].view(torch.uint8).cpu().numpy()


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
    t = torch.from_numpy(a).cuda().to(dtype)
    m = torch.empty(t.numel() + offset, dtype=dtype, device="cuda")
    m[offset:] = t.reshape(-1)
    return m[offset:].view(t.shape)


def test_every_code():
    """All bf16 values up to 448 and the midpoints of the codes with their neighbours,
    in blocks whose scale is 1."""
    bits = np.arange(1 << 16, dtype=np.uint32) << 16
    v = bits.view(np.float32)
    v = v[np.isfinite(v) & (np.abs(v) <= 448)]
    mid = ((ob.VALUES[1:] + ob.VALUES[:-1]) / 2).astype(np.float32)
    mid = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(500))])
    v = np.concatenate([v, mid, -mid])
    v = np.pad(v, (0, -len(v) % 127)).reshape(-1, 127)
    w = np.concatenate([np.full((len(v), 1), 448, np.float32), v], axis=1)
    rec = qw.block_quantize(torch.from_numpy(w).cuda(), 1)
    assert np.all(rec["scales"].cpu().numpy() == 1)
    assert np.array_equal(codes_of(rec), ob.encode(w))
    want = ob.decode(ob.encode(w))
    assert np.array_equal(host(qw.block_unpack(rec)), want)


@pytest.mark.parametrize("n,k", [(1, 1), (3, 127), (130, 128), (5, 129), (257, 1000), (128, 4104), (300, 77)])
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype,offset", [(torch.float32, 0), (torch.float32, 1), (torch.bfloat16, 0), (torch.bfloat16, 3)])
def test_quantize_and_unpack(n, k, block_rows, dtype, offset):
    w = as_type(wide([n, k], n, k), dtype, offset)
    rec = qw.block_quantize(w, block_rows)
    codes, scales = ob.quantize(w.float().cpu().numpy(), block_rows)
    assert np.array_equal(rec["scales"].cpu().numpy().view(np.uint32), scales.view(np.uint32))
    assert np.array_equal(codes_of(rec), codes)
    out = as_type(np.full((n, k), np.nan, np.float32), torch.float32, offset)
    qw.block_unpack(rec, out=out)
    s = np.repeat(np.repeat(scales, 128, 1), block_rows, 0)[:n, :k]
    want = ob.decode(codes)[:, :k].astype(np.float32) * s
    assert np.array_equal(out.cpu().numpy().view(np.uint32), want.view(np.uint32))


@pytest.mark.parametrize("size", [3e38, 1.0, 1e-30, 2.0 ** -120, 1e-40, 2.0 ** -149])
def test_quantize_extreme_magnitudes(size):
    """Scales near the ends of fp32's range, subnormal ones and ones that become zero."""
    rng = np.random.default_rng(3)
    w = (rng.uniform(-1, 1, (4, 256)) * size).astype(np.float32)
    w[:, 0] = size
    for br in (1, 128):
        codes, scales = ob.quantize(w, br)
        rec = qw.block_quantize(torch.from_numpy(w).cuda(), br)
        assert np.array_equal(rec["scales"].cpu().numpy().view(np.uint32), scales.view(np.uint32))
        assert np.array_equal(codes_of(rec), codes)


def test_quantize_experts_one_after_another():
    w = wide(5, 3 * 150, 200).reshape(3, 150, 200)
    rec = qw.block_quantize(torch.from_numpy(w).cuda(), 128)
    for e in range(3):
        codes, scales = ob.quantize(w[e], 128)
        assert np.array_equal(codes_of(rec)[e], codes)
        assert np.array_equal(rec["scales"][e].cpu().numpy(), scales)


def test_quantize_transposed_moves_the_blocks():
    w = torch.from_numpy(wide(6, 300, 260)).cuda()
    a, b = qw.block_quantize(w, 128), qw.block_quantize(w.t().contiguous(), 128)
    assert torch.equal(a["scales"], b["scales"].t())
    assert np.array_equal(codes_of(a)[:, :260], codes_of(b)[:, :300].T)


@pytest.mark.parametrize("rows,f,dtype,offset", [(1, 1, torch.float32, 0), (7, 200, torch.float32, 0), (5, 131, torch.float32, 0),
                                                 (9, 256, torch.bfloat16, 0), (9, 136, torch.bfloat16, 5)])
def test_swiglu(rows, f, dtype, offset):
    rng = np.random.default_rng([rows, f])
    h = (rng.standard_normal((rows, 2 * f)) * 4).astype(np.float32)
    h[0, 0] = -120.0     # exp(-gate) beyond fp32: the value is 0
    h = as_type(h, dtype, offset)
    rec = qw.block_quantize_swiglu(h)
    want = ob.swiglu(host(h))
    got = ob.values(codes_of(rec), rec["scales"].cpu().numpy(), 1, f)
    s = np.repeat(rec["scales"].cpu().numpy().astype(np.float64), 128, 1)[:, :f]
    top = np.abs(np.pad(want, ((0, 0), (0, -f % 128)))).reshape(rows, -1, 128).max(-1)
    # the fp32 value is a few ulp off (exp, add, divide, multiply: 6 at most), and so is the scale;
    # it is 1 where it has no fp32 value but zero (silu(-120) is -9e-51, fp32 ends at 2^-149 = 1.4e-45)
    step = np.where((top / 448).astype(np.float32) > 0, top / 448, 1)
    assert np.all(np.abs(s[:, ::128] - step) <= 8 * 2.0 ** -23 * step)
    assert np.all(np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-5))
    assert not codes_of(rec)[:, f:].any()


def test_swiglu_leaves_unused_rows():
    h = torch.randn(40, 256, device="cuda")
    full = qw.block_quantize_swiglu(h)
    for used in (0, 1, 17, 40, 1000, -3):
        codes = torch.full((40, 128), 77, dtype=torch.uint8, device="cuda")
        scales = torch.full((40, 1), -1.0, device="cuda")
        u = torch.tensor([used], dtype=torch.int32, device="cuda")
        assert qw.qw_block_quantize_swiglu(40, 128, 0, h, u, codes, scales) == 0
        n = min(max(used, 0), 40)
        assert torch.equal(codes[:n], full["codes"].view(torch.uint8)[:n]) and torch.equal(scales[:n], full["scales"][:n])
        assert bool((codes[n:] == 77).all()) and bool((scales[n:] == -1).all())


def check_product(y, xv, wv):
    """y against 64-bit values, within the bar and half a step of its type."""
    ref, base = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    err, bar = np.abs(host(y) - ref), BAR[y.dtype] * base
    assert np.all(err <= bar + HALF[y.dtype] * (np.abs(ref) + bar)), float((err - bar).max())


def record(seed, n, k, br):
    w = wide(seed, n, k) if n * k < 1 << 21 else np.random.default_rng(seed).standard_normal((n, k), dtype=np.float32)
    rec = qw.block_quantize(torch.from_numpy(w).cuda(), br)
    return rec, ob.values(codes_of(rec), rec["scales"].cpu().numpy(), br, k)


SIZES = [(1, 1, 1), (1, 128, 128), (1, 4096, 4096), (2, 17, 129), (3, 1000, 300), (5, 16, 5000), (7, 4096, 130), (8, 333, 1024),
         (15, 128, 4096), (16, 257, 2048), (17, 96, 640), (31, 200, 1000), (33, 513, 256), (63, 64, 1152), (64, 1000, 384),
         (65, 65, 257), (100, 4096, 512), (127, 300, 128), (128, 256, 896), (129, 1025, 1000), (200, 2048, 640), (256, 256, 128),
         (257, 511, 384), (300, 2304, 1280), (1000, 130, 100), (513, 4097, 333)]


# the larger tiles, a last round that is cut off, waves with many blocks of k, and
# more of them than a wave holds
LARGE = [(2, 60, 9000), (8, 60, 9000), (3, 40, 13000), (16, 70, 13000), (600, 3000, 260), (1000, 5000, 500), (4096, 4096, 256),
         (2100, 4000, 200), (2048, 8300, 1000), (40, 4096, 1000), (60, 2048, 4000)]


def on_gpu(xrec, rec, k, y):
    """check_product for large sizes, in float64 on the GPU, piece by piece."""
    val = lambda r, br: qw.block_unpack(r).double()  # noqa: E731  (fl32(code * S): 2^-24 of each value)
    xv, wv = val(xrec, 1), val(rec, rec["block_rows"])
    ref, base = xv @ wv.T, xv.abs() @ wv.abs().T
    bar = (BAR[y.dtype] + 2.0 ** -23) * base
    assert bool(((y.double() - ref).abs() <= bar + HALF[y.dtype] * (ref.abs() + bar)).all())


@pytest.mark.parametrize("m,n,k", LARGE)
@pytest.mark.parametrize("br,dtype", [(128, torch.float32), (1, torch.float32), (128, torch.bfloat16), (1, torch.bfloat16)])
def test_gemm_large(m, n, k, br, dtype):
    print("gemm", m, n, k, br, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    make = lambda r, c: torch.randn(r, c, generator=g, device="cuda") * torch.rand(c, generator=g, device="cuda").exp()  # noqa: E731
    rec, x = qw.block_quantize(make(n, k), br), make(m, k)
    xrec = qw.block_quantize(x, 1)
    y = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
    qw.block_gemm(rec, xrec, out=y[:m], out_dtype=dtype)
    on_gpu(xrec, rec, k, y[:m])
    assert bool((y[m] == 7).all())
    on_gpu(xrec, rec, k, qw.block_matmul(rec, x, out_dtype=dtype))


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("br,dtype", [(128, torch.float32), (1, torch.float32), (128, torch.bfloat16), (1, torch.bfloat16)])
def test_gemm(m, n, k, br, dtype):
    print("gemm", m, n, k, br, dtype, flush=True)
    rec, wv = record([m, n, k], n, k, br)
    xrec, xv = record([k, m], m, k, 1)
    y = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
    qw.block_gemm(rec, xrec, out=y[:m], out_dtype=dtype)
    check_product(y[:m], xv, wv)
    assert bool((y[m] == 7).all())
    again = qw.block_gemm(rec, xrec, out_dtype=dtype)
    assert torch.equal(again, y[:m])


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("xt,yt,offset", [(torch.float32, torch.float32, 0), (torch.bfloat16, torch.bfloat16, 0),
                                          (torch.float32, torch.bfloat16, 1), (torch.bfloat16, torch.float32, 1)])
def test_matmul(m, n, k, xt, yt, offset):
    print("matmul", m, n, k, xt, yt, flush=True)
    rec, wv = record([m, n, k], n, k, 128)
    x = as_type(wide([k, m], m, k), xt, offset)
    xv = ob.values(*ob.quantize(x.float().cpu().numpy(), 1), 1, k)
    y = as_type(np.full((m, n), np.nan, np.float32), yt, offset)
    qw.block_matmul(rec, x, out=y)
    check_product(y, xv, wv)
    assert qw.block_matmul(rec, x).dtype == xt


def test_products_that_bf16_would_lose():
    """Integer codes whose sums need all of fp32's bits: exact results."""
    rng = np.random.default_rng(8)
    for m in (1, 40, 300):
        w = rng.integers(-16, 17, (200, 512)).astype(np.float32)
        x = rng.integers(-16, 17, (m, 512)).astype(np.float32)
        w[:, ::128] = 448.0
        x[:, ::128] = 448.0
        y = qw.block_matmul(qw.block_quantize(torch.from_numpy(w).cuda(), 128), torch.from_numpy(x).cuda())
        assert np.array_equal(host(y), x.astype(np.float64) @ w.T.astype(np.float64))


@pytest.mark.parametrize("m", [1, 9, 40, 150, 300])
def test_empty_sums_and_empty_sides(m):
    for dtype in (torch.float32, torch.bfloat16):
        rec = qw.block_quantize(torch.zeros(70, 0, device="cuda"), 128)
        y = torch.full((m, 70), 7.0, dtype=dtype, device="cuda")
        qw.block_matmul(rec, torch.zeros(m, 0, device="cuda"), out=y)
        assert not bool(y.any())
    rec = qw.block_quantize(torch.zeros(0, 40, device="cuda"), 128)
    assert qw.block_matmul(rec, torch.zeros(m, 40, device="cuda")).shape == (m, 0)
    rec = qw.block_quantize(torch.ones(30, 40, device="cuda"), 128)
    assert qw.block_matmul(rec, torch.zeros(0, 40, device="cuda")).shape == (0, 30)


def test_rows_do_not_influence_each_other():
    """A row of infinities and NaN leaves the others as they are."""
    rec, _ = record(1, 300, 700, 128)
    for m in (4, 16, 50, 200, 400):
        x = torch.randn(m, 700, device="cuda")
        clean = qw.block_matmul(rec, x)
        x[m // 2] = float("nan")
        x[m // 2, ::3] = float("inf")
        dirty = qw.block_matmul(rec, x)
        keep = torch.arange(m, device="cuda") != m // 2
        assert torch.equal(clean[keep], dirty[keep])


def test_gradients_of_a_product():
    """Both gradients by the calls that qw.h names, against the formula on the
    values the codes stand for, and the input's against differences."""
    m, n, k = 70, 260, 390
    rng = np.random.default_rng(9)
    w = torch.from_numpy(rng.standard_normal((n, k)).astype(np.float32)).cuda()
    x = torch.from_numpy(rng.standard_normal((m, k)).astype(np.float32)).cuda()
    dy = torch.from_numpy(rng.standard_normal((m, n)).astype(np.float32)).cuda()
    rec = qw.block_quantize(w, 128)
    wv = ob.values(codes_of(rec), rec["scales"].cpu().numpy(), 128, k)
    dyr = qw.block_quantize(dy, 1)
    dyv = ob.values(codes_of(dyr), dyr["scales"].cpu().numpy(), 1, n)
    dx = qw.block_gemm(qw.block_quantize(w.t().contiguous(), 128), dyr)
    check_product(dx, dyv, wv.T)
    a, b = qw.block_quantize(dy.t().contiguous(), 1), qw.block_quantize(x.t().contiguous(), 1)
    av = ob.values(codes_of(a), a["scales"].cpu().numpy(), 1, m)
    bv = ob.values(codes_of(b), b["scales"].cpu().numpy(), 1, m)
    check_product(qw.block_gemm(b, a), av, bv)
    # <dy, f(x + e) - f(x)> = <dx, e> for the product of unquantized x with the codes' values
    e = rng.standard_normal((m, k))
    xd = host(x)
    diff = (dyv * ((xd + e) @ wv.T - xd @ wv.T)).sum()
    assert abs(diff - (host(dx) * e).sum()) <= 1e-4 * (np.abs(dyv) @ np.abs(wv) * np.abs(e)).sum()


# ------------------------------------------------------------ grouped


GROUPS = [([0], 5, 130), ([3], 100, 200), ([0, 0, 1, 0], 64, 128), ([1, 2, 3, 4, 5], 260, 300), ([17, 0, 64, 1, 65, 0, 130], 200, 257),
          ([300, 1, 0, 257, 128], 513, 384), ([40] * 70, 96, 256), ([1] * 130, 130, 129), ([0] * 99 + [700], 300, 200), ([2, 1], 40, 9000), ([5] * 8, 100, 5000), ([1, 3], 40, 13000), ([20] * 4, 64, 13000)]


@pytest.mark.parametrize("counts,n,k", GROUPS)
@pytest.mark.parametrize("br,dtype", [(128, torch.float32), (1, torch.bfloat16)])
def test_grouped(counts, n, k, br, dtype):
    print("grouped", counts, n, k, br, dtype, flush=True)
    e, used = len(counts), sum(counts)
    rows = used + 37
    rng = np.random.default_rng([e, n, k])
    w = rng.standard_normal((e, n, k), dtype=np.float32)
    x = rng.standard_normal((rows, k), dtype=np.float32)
    rec, xrec = qw.block_quantize(torch.from_numpy(w).cuda(), br), qw.block_quantize(torch.from_numpy(x).cuda(), 1)
    # codes behind the last expert's rows are never looked at
    xrec["codes"].view(torch.uint8)[used:] = 0x7F
    xrec["scales"][used:] = float("nan")
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = torch.full((rows, n), 7.0, dtype=dtype, device="cuda")
    qw.block_gemm_grouped(rec, xrec, torch.from_numpy(off).cuda(), out=y, out_dtype=dtype)
    assert bool((y[used:] == 7).all())
    xv = ob.values(codes_of(xrec)[:used] & 0xFF, xrec["scales"].cpu().numpy()[:used], 1, k)
    for i in range(e):
        if counts[i]:
            wv = ob.values(codes_of(rec)[i], rec["scales"].cpu().numpy()[i], br, k)
            check_product(y[off[i]:off[i + 1]], xv[off[i]:off[i + 1]], wv)


@pytest.mark.parametrize("counts,n,k", [([900, 0, 1500], 4000, 300), ([300] * 8, 2000, 256), ([150] * 30, 1000, 128), ([700] * 12, 2000, 128),
                                        ([20] * 8, 600, 2000), ([257, 1, 511, 256, 128, 0, 640], 2050, 640)])
@pytest.mark.parametrize("br,dtype", [(128, torch.float32), (1, torch.float32), (128, torch.bfloat16), (1, torch.bfloat16)])
def test_grouped_large(counts, n, k, br, dtype):
    print("grouped", len(counts), sum(counts), n, k, br, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(n + k)
    rows = sum(counts) + 37
    rec = qw.block_quantize(torch.randn(len(counts), n, k, generator=g, device="cuda"), br)
    xrec = qw.block_quantize(torch.randn(rows, k, generator=g, device="cuda"), 1)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    y = torch.full((rows, n), 7.0, dtype=dtype, device="cuda")
    qw.block_gemm_grouped(rec, xrec, torch.from_numpy(off).cuda(), out=y, out_dtype=dtype)
    assert bool((y[off[-1]:] == 7).all())
    part = lambda r, at, shape: dict(r, shape=shape, codes=r["codes"][at].contiguous(), scales=r["scales"][at].contiguous())  # noqa: E731
    for e, c in enumerate(counts):
        if c:
            at = slice(int(off[e]), int(off[e + 1]))
            on_gpu(part(xrec, at, [c, k]), part(rec, e, [n, k]), k, y[at])


def test_grouped_clamps_offsets():
    """Offsets outside [0, rows] end at the rows there are."""
    rec = qw.block_quantize(torch.randn(3, 80, 128, device="cuda"), 128)
    x = qw.block_quantize(torch.randn(50, 128, device="cuda"), 1)
    good = qw.block_gemm_grouped(rec, x, torch.tensor([0, 20, 20, 50], dtype=torch.int32, device="cuda"))
    wild = qw.block_gemm_grouped(rec, x, torch.tensor([-9, 20, 20, 1 << 30], dtype=torch.int32, device="cuda"))
    assert torch.equal(good, wild)


# ------------------------------------------------------ streams and graphs


def test_side_stream():
    rec = qw.block_quantize(torch.randn(500, 600, device="cuda"), 128)
    x = torch.randn(100, 600, device="cuda")
    want = qw.block_matmul(rec, x)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream):
        got = qw.block_matmul(rec, x, stream=stream)
        s.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("m", [1, 16, 60, 300])
def test_graph_replays(m):
    rec = qw.block_quantize(torch.randn(700, 900, device="cuda"), 128)
    x = torch.randn(m, 900, device="cuda")
    y = qw.block_matmul(rec, x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qw.block_matmul(rec, x, out=y)
    for i in range(4):
        x.copy_(torch.randn(m, 900, device="cuda"))
        want = qw.block_matmul(rec, x)
        y.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i
