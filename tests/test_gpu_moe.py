"""Tokens sorted by expert and back on the GPU, against the oracle's loops."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw
from oracle import block as ob

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def host(t):
    return t.detach().cpu().double().numpy()


def routing(seed, t, topk, experts, drop=0.2, dtype=np.int64):
    rng = np.random.default_rng(seed)
    ids = rng.integers(0, experts, (t, topk)) if topk > experts else np.argsort(rng.random((t, experts)), axis=1)[:, :topk]
    if drop:
        bad = rng.random((t, topk)) < drop
        ids = np.where(bad, rng.choice([-1, experts, 2 ** 31 - 1, -2 ** 31], (t, topk)), ids)
    return ids.astype(dtype)


@pytest.mark.parametrize("t,topk,experts", [(0, 2, 8), (1, 1, 1), (1, 8, 64), (5, 3, 7), (63, 1, 2), (64, 1, 64), (65, 4, 512),
                                            (1000, 8, 128), (1024, 8, 256), (1025, 8, 256), (3000, 3, 511), (20000, 8, 60), (300000, 1, 3)])
@pytest.mark.parametrize("drop", [0.0, 0.3, 1.0])
@pytest.mark.parametrize("dtype", [np.int32, np.int64])
def test_sort(t, topk, experts, drop, dtype):
    print("sort", t, topk, experts, drop, dtype, flush=True)
    ids = routing([t, topk], t, topk, experts, drop, dtype)
    if dtype is np.int64 and drop:
        ids[ids < 0] = -2 ** 63
        ids[ids == 2 ** 31 - 1] = 2 ** 40 + 1      # low half in range
    r = qw.moe_sort(torch.from_numpy(ids).cuda(), experts)
    pos, order, off = ob.sort(ids, experts)
    assert np.array_equal(r["offsets"].cpu().numpy(), off)
    assert np.array_equal(r["pos"].cpu().numpy(), pos)
    assert np.array_equal(r["order"].cpu().numpy(), order)
    r = qw.moe_sort(torch.from_numpy(ids).cuda(), experts, order=False)
    assert r["order"] is None and np.array_equal(r["pos"].cpu().numpy(), pos)


def test_sort_one_expert_takes_all():
    ids = torch.full((9000, 2), 5, device="cuda")
    r = qw.moe_sort(ids, 8)
    assert torch.equal(r["order"], torch.arange(18000, dtype=torch.int32, device="cuda"))
    assert r["offsets"].tolist() == [0] * 6 + [18000] * 3


SHAPES = [(1, 1, 1, 8), (3, 2, 5, 8), (9, 8, 16, 1003), (40, 3, 7, 130), (33, 9, 20, 256), (5, 17, 4, 64), (130, 4, 8, 4096), (64, 2, 4, 5000)]


def as_type(a, dtype, offset=0):
    t = torch.from_numpy(a).cuda().to(dtype)
    m = torch.empty(t.numel() + offset, dtype=dtype, device="cuda")
    m[offset:] = t.reshape(-1)
    return m[offset:].view(t.shape)


@pytest.mark.parametrize("t,topk,experts,d", SHAPES)
@pytest.mark.parametrize("dtype,offset", [(torch.float32, 0), (torch.bfloat16, 0), (torch.bfloat16, 1), (torch.float32, 1)])
def test_gather_combine_and_gradients(t, topk, experts, d, dtype, offset):
    print("moe", t, topk, experts, d, dtype, offset, flush=True)
    rng = np.random.default_rng([t, topk, d])
    ids = routing([d, t], t, topk, experts)
    pos, order, off = ob.sort(ids, experts)
    rows = t * topk
    route = dict(pos=torch.from_numpy(pos).cuda())
    x = as_type(rng.standard_normal((t, d)).astype(np.float32), dtype, offset)
    xs = as_type(np.full((rows, d), 7, np.float32), dtype, offset)
    qw.moe_gather(x, route, out=xs)
    want = np.full((rows, d), 7.0)
    have = order >= 0
    want[have] = host(x)[order[have] // topk]
    assert np.array_equal(host(xs), want)

    # weights and rows of slots that are out are never looked at
    w = rng.standard_normal((t, topk)).astype(np.float32)
    w[pos < 0] = np.nan
    ys = rng.standard_normal((rows, d)).astype(np.float32)
    ys[off[-1]:] = np.nan
    ys = as_type(ys, dtype, offset)
    wt = torch.from_numpy(w).cuda()
    for weights in (wt, None):
        wn = None if weights is None else w
        ref = ob.combine(host(ys), pos, wn)
        mag = ob.combine(np.abs(host(ys)), pos, None if wn is None else np.abs(wn))
        for yt in (torch.float32, torch.bfloat16):
            y = as_type(np.full((t, d), np.nan, np.float32), yt, offset)
            qw.moe_combine(ys, route, weights, out=y)
            # topk fused multiply-adds in fp32, then one rounding
            assert np.all(np.abs(host(y) - ref) <= topk * 2.0 ** -24 * mag * (1 + 2.0 ** -8) + HALF[yt] * np.abs(ref))

    dy = as_type(rng.standard_normal((t, d)).astype(np.float32), dtype, offset)
    dys = as_type(np.full((rows, d), 7, np.float32), dtype, offset)
    dw = torch.full((t, topk), float("nan"), device="cuda")
    qw.moe_combine_backward(dy, ys, route, wt, dys=dys, dweights=dw)
    rdys, rdw = ob.combine_backward(host(dy), host(ys), pos, w, np.full((rows, d), 7.0))
    assert np.all(np.abs(host(dys) - rdys) <= (HALF[dtype] + 2.0 ** -24 * (dtype != torch.float32)) * np.abs(rdys))
    _, mag = ob.combine_backward(np.abs(host(dy)), np.abs(host(ys)), pos, w, rdys)
    # a lane sums d / 256 + 8 products, then 8 partial sums are joined in pairs
    assert np.all(np.abs(host(dw) - rdw) <= (d / 256 + 16) * 2.0 ** -24 * mag)

    # dys holds 7 behind the rows; the gather's gradient does not look there
    dx = qw.moe_gather_backward(dys, route)
    ref = ob.combine(host(dys), pos, None)
    mag = ob.combine(np.abs(host(dys)), pos, None)
    assert np.all(np.abs(host(dx) - ref) <= topk * 2.0 ** -24 * mag * (1 + 2.0 ** -8) + HALF[dtype] * np.abs(ref))


def test_gradients_against_differences():
    """<dy, f(p + e) - f(p)> = <gradient, e>: gather and combine are linear in
    rows and weights, so a step of 1 has no error of its own."""
    t, topk, e, d = 40, 3, 6, 72
    rng = np.random.default_rng(4)
    ids = routing(3, t, topk, e)
    pos, order, off = ob.sort(ids, e)
    n = off[-1]
    route = dict(pos=torch.from_numpy(pos).cuda())
    make = lambda *s: torch.from_numpy(rng.integers(-8, 9, s).astype(np.float32)).cuda()  # noqa: E731
    ys, ey, w, ew, dy = make(t * topk, d), make(t * topk, d), make(t, topk), make(t, topk), make(t, d)
    dys, dw = qw.moe_combine_backward(dy, ys, route, w, dys=torch.zeros_like(ys))
    f = lambda r, v: host(qw.moe_combine(r, route, v))  # noqa: E731
    # small whole numbers: every sum is exact
    assert (host(dy) * (f(ys + ey, w) - f(ys, w))).sum() == (host(dys)[:n] * host(ey)[:n]).sum()
    assert (host(dy) * (f(ys, w + ew) - f(ys, w))).sum() == (host(dw) * host(ew)).sum()
    x, ex, dxs = make(t, d), make(t, d), make(t * topk, d)
    g = lambda v: host(qw.moe_gather(v, route, out=torch.zeros_like(dxs)))  # noqa: E731
    assert (host(dxs) * (g(x + ex) - g(x))).sum() == (host(qw.moe_gather_backward(dxs, route)) * host(ex)).sum()


def test_either_gradient_alone():
    t, topk, d = 20, 2, 136
    pos = torch.arange(t * topk, dtype=torch.int32, device="cuda").view(t, topk)
    dy, ys, w = torch.randn(t, d, device="cuda"), torch.randn(t * topk, d, device="cuda"), torch.randn(t, topk, device="cuda")
    dys, dw = qw.moe_combine_backward(dy, ys, dict(pos=pos), w)
    a, b = torch.empty_like(dys), torch.empty_like(dw)
    assert qw.qw_moe_combine_backward(t, topk, d, t * topk, 0, dy, None, pos, w, a, None) == 0
    assert qw.qw_moe_combine_backward(t, topk, d, t * topk, 0, dy, ys, pos, w, None, b) == 0
    assert torch.equal(a, dys) and torch.equal(b, dw)


def test_positions_beyond_the_rows_are_skipped():
    t, topk, d, rows = 30, 2, 128, 40
    pos = torch.arange(t * topk, dtype=torch.int32, device="cuda").view(t, topk)
    x, w = torch.randn(t, d, device="cuda"), torch.rand(t, topk, device="cuda")
    xs = torch.full((rows, d), 7.0, device="cuda")
    qw.moe_gather(x, dict(pos=pos), out=xs)
    assert torch.equal(xs, x.repeat_interleave(topk, 0)[:rows])
    rec = qw.moe_gather_block(x, dict(pos=pos), rows=rows)
    full = qw.block_quantize(xs, 1)
    assert torch.equal(rec["codes"].view(torch.uint8), full["codes"].view(torch.uint8)) and torch.equal(rec["scales"], full["scales"])
    y = qw.moe_combine(xs, dict(pos=pos), w)
    kept = torch.where(pos < rows, w, 0.0)
    assert torch.allclose(y, x * kept.sum(1, keepdim=True), rtol=1e-6, atol=1e-6)
    dys, dw = qw.moe_combine_backward(x, xs, dict(pos=pos), w)
    assert dys.shape == (rows, d) and not bool(dw[pos >= rows].any())


@pytest.mark.parametrize("t,topk,experts,d,dtype,offset", [(1, 2, 4, 5, torch.float32, 0), (50, 3, 8, 300, torch.float32, 0),
                                                           (50, 8, 8, 512, torch.bfloat16, 0), (33, 2, 6, 264, torch.bfloat16, 1)])
def test_gather_block_is_quantize_of_the_gathered(t, topk, experts, d, dtype, offset):
    ids = routing([t, d], t, topk, experts)
    r = qw.moe_sort(torch.from_numpy(ids).cuda(), experts)
    n = int(r["offsets"][-1])
    x = as_type(np.random.default_rng(t).standard_normal((t, d)).astype(np.float32), dtype, offset)
    rec = qw.moe_gather_block(x, r)
    want = qw.block_quantize(qw.moe_gather(x, r), 1)
    assert torch.equal(rec["codes"].view(torch.uint8)[:n], want["codes"].view(torch.uint8)[:n])
    assert torch.equal(rec["scales"][:n], want["scales"][:n])


# ------------------------------------------------------------ expert MLP


def mlp_reference(gate_up, down, x, ids, weights, f):
    """The definition in 64 bits on the codes' values; x and the hidden values quantized by the oracle."""
    val = lambda r, e: ob.values(r["codes"].view(torch.uint8)[e].cpu().numpy(), r["scales"][e].cpu().numpy(),  # noqa: E731
                                 r["block_rows"], r["shape"][2])
    d = x.shape[1]
    xv = ob.values(*ob.quantize(x.float().cpu().numpy(), 1), 1, d)
    y = np.zeros((len(x), d))
    for e in range(gate_up["shape"][0]):
        at, slot = np.nonzero(ids == e)
        if len(at) == 0:
            continue
        h = ob.swiglu(xv[at] @ val(gate_up, e).T)
        h = ob.values(*ob.quantize(h.astype(np.float32), 1), 1, f)
        ye = h @ val(down, e).T
        for i, a in enumerate(at):
            y[a] += (1.0 if weights is None else float(weights[a, slot[i]])) * ye[i]
    return y


MLP = [(1, 1, 1, 128, 128), (1, 4, 8, 512, 384), (3, 2, 5, 200, 70), (7, 2, 4, 130, 257), (40, 2, 8, 256, 128), (130, 4, 6, 300, 200),
       (300, 2, 3, 264, 136), (600, 1, 2, 128, 300), (200, 2, 4, 260, 128), (333, 3, 5, 128, 384), (900, 2, 6, 700, 256), (2, 2, 3, 1300, 600), (16, 2, 8, 136, 1100),
       (2, 1, 2, 4200, 300), (1, 1, 1, 9000, 128), (1, 1, 1, 128, 4200), (3, 1, 1, 200, 9100)]


@pytest.mark.parametrize("t,topk,experts,d,f", MLP)
@pytest.mark.parametrize("br,dtype,weighted", [(128, torch.bfloat16, True), (1, torch.float32, True), (128, torch.float32, False)])
def test_mlp(t, topk, experts, d, f, br, dtype, weighted):
    print("mlp", t, topk, experts, d, f, br, dtype, flush=True)
    rng = np.random.default_rng([t, d, f])
    make = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).cuda()  # noqa: E731
    gate_up = qw.block_quantize(make(experts, 2 * f, d) * d ** -0.5, br)
    down = qw.block_quantize(make(experts, d, f) * f ** -0.5, br)
    x = make(t, d).to(dtype)
    ids = routing([t, f], t, topk, experts, 0.1)
    w = rng.random((t, topk)).astype(np.float32) if weighted else None
    wt = torch.from_numpy(w).cuda() if weighted else None
    y = qw.moe_mlp(gate_up, down, x, torch.from_numpy(ids).cuda(), wt, out_dtype=torch.float32)
    ref = mlp_reference(gate_up, down, x, ids, w, f)
    # The 8-bit cores cut products off at 2^-13 of the largest of 8: uniform in [0, 2^-13)
    # of it for either sign, 2^-13 / sqrt(3) for one in 8 of the sums' own square root of
    # terms: about 2e-5 of h's size, so a share of up to 2 * 2e-5 / 2^-4 = 6.4e-4 of the
    # codes may be the next one, off by at most 2^-3: sqrt(6.4e-4) / 8 = 3.2e-3 in the 2-norm,
    # on top of 2e-5 of the second product.
    norm = np.linalg.norm(ref)
    assert np.linalg.norm(host(y) - ref) <= 3.3e-3 * norm + 1e-30
    # the calls one by one give the same up to the order of fp32 sums
    r = qw.moe_sort(torch.from_numpy(ids).cuda(), experts)
    xr = qw.moe_gather_block(x, r)
    h = qw.block_gemm_grouped(gate_up, xr, r["offsets"])
    hr = qw.block_quantize_swiglu(h, r["offsets"][-1:])
    y2 = qw.moe_combine(qw.block_gemm_grouped(down, hr, r["offsets"]), r, wt)
    assert np.linalg.norm(host(y2) - ref) <= 3.3e-3 * norm + 1e-30
    yb = qw.moe_mlp(gate_up, down, x, torch.from_numpy(ids).cuda(), wt, out_dtype=torch.bfloat16)
    assert np.linalg.norm(host(yb) - host(y)) <= 2.0 ** -8 * norm + 1e-30


@pytest.mark.parametrize("t", [1, 9, 300])
def test_mlp_with_no_slot_in(t):
    gate_up = qw.block_quantize(torch.randn(4, 256, 128, device="cuda"), 128)
    down = qw.block_quantize(torch.randn(4, 128, 128, device="cuda"), 128)
    y = torch.full((t, 128), 7.0, device="cuda")
    qw.moe_mlp(gate_up, down, torch.randn(t, 128, device="cuda"), torch.full((t, 2), -1, device="cuda"),
               torch.full((t, 2), float("nan"), device="cuda"), out=y)
    assert not bool(y.any())
    assert qw.moe_mlp(gate_up, down, torch.zeros(0, 128, device="cuda"), torch.zeros(0, 2, dtype=torch.int64, device="cuda")).shape == (0, 128)


@pytest.mark.parametrize("t", [1, 9, 400])
def test_mlp_without_hidden_values(t):
    """f = 0 is an empty sum: zeros, for few and for many rows an expert."""
    gate_up = qw.block_quantize(torch.zeros(2, 0, 128, device="cuda"), 128)
    down = qw.block_quantize(torch.zeros(2, 128, 0, device="cuda"), 128)
    y = torch.full((t, 128), 7.0, device="cuda")
    qw.moe_mlp(gate_up, down, torch.randn(t, 128, device="cuda"), torch.zeros(t, 2, dtype=torch.int64, device="cuda"), out=y)
    assert not bool(y.any())


@pytest.mark.parametrize("t", [3, 400])
def test_mlp_graph_replays(t):
    d, f, e, topk = 256, 192, 8, 2
    gate_up = qw.block_quantize(torch.randn(e, 2 * f, d, device="cuda") * 0.06, 128)
    down = qw.block_quantize(torch.randn(e, d, f, device="cuda") * 0.06, 128)
    x, w = torch.randn(t, d, device="cuda"), torch.rand(t, topk, device="cuda")
    ids = torch.randint(0, e, (t, topk), device="cuda")
    y = qw.moe_mlp(gate_up, down, x, ids, w)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        qw.moe_mlp(gate_up, down, x, ids, w, out=y)
    for i in range(4):
        x.copy_(torch.randn(t, d, device="cuda"))
        ids.copy_(torch.randint(-1, e, (t, topk), device="cuda"))
        want = qw.moe_mlp(gate_up, down, x, ids, w)
        y.zero_()
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want), i


def test_layer_forward_and_backward_together():
    """Sort, gather, experts' product, combine, and back to the tokens: the
    whole chain's gradient against the formula in 64 bits."""
    t, topk, e, d, n = 90, 2, 5, 260, 140
    rng = np.random.default_rng(12)
    ids = routing(11, t, topk, e)
    w = rng.random((t, topk)).astype(np.float32)
    x = rng.standard_normal((t, d)).astype(np.float32)
    dy = rng.standard_normal((t, n)).astype(np.float32)
    weights = torch.from_numpy(rng.standard_normal((e, n, d), dtype=np.float32)).cuda()
    rec = qw.block_quantize(weights, 128)
    back = qw.block_quantize(weights.transpose(1, 2).contiguous(), 128)
    cu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    r = qw.moe_sort(cu(ids), e)
    ys = qw.block_gemm_grouped(rec, qw.moe_gather_block(cu(x), r), r["offsets"])
    y = qw.moe_combine(ys, r, cu(w))
    dys, dw = qw.moe_combine_backward(cu(dy), ys, r, cu(w), dys=torch.zeros_like(ys))
    dyr = qw.block_quantize(dys, 1)
    dxs = qw.block_gemm_grouped(back, dyr, r["offsets"])
    dx = qw.moe_gather_backward(dxs, r)

    wv = [ob.values(rec["codes"].view(torch.uint8)[i].cpu().numpy(), rec["scales"][i].cpu().numpy(), 128, d) for i in range(e)]
    xv = ob.values(*ob.quantize(x, 1), 1, d)
    dyv = ob.values(dyr["codes"].view(torch.uint8).cpu().numpy(), dyr["scales"].cpu().numpy(), 1, n)
    pos = r["pos"].cpu().numpy()
    ry, rdx, rdw = np.zeros((t, n)), np.zeros((t, d)), np.zeros((t, topk))
    my, mdx, mdw = np.zeros((t, n)), np.zeros((t, d)), np.zeros((t, topk))
    for i in range(t):
        for j in range(topk):
            if pos[i, j] >= 0:
                a = wv[ids[i, j]]
                ry[i] += w[i, j] * (a @ xv[i])
                my[i] += w[i, j] * (np.abs(a) @ np.abs(xv[i]))
                rdw[i, j] = dy[i].astype(np.float64) @ (a @ xv[i])
                mdw[i, j] = np.abs(dy[i]).astype(np.float64) @ (np.abs(a) @ np.abs(xv[i]))
                rdx[i] += dyv[pos[i, j]] @ a
                mdx[i] += np.abs(dyv[pos[i, j]]) @ np.abs(a)
    # the products' bar, and a few fp32 roundings behind it
    assert np.all(np.abs(host(y) - ry) <= 1.1e-5 * my)
    assert np.all(np.abs(host(dw) - rdw) <= 1.2e-5 * mdw)
    assert np.all(np.abs(host(dx) - rdx) <= 1.1e-5 * mdx)
