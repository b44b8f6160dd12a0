"""Every tile of the block-scaled products and every way of the expert MLP, with more
blocks of k than a wave's buffers hold and with more tiles than compute units; the
sizes are searched for by the kernel that the choice reports, so that they follow
it.  And sizes whose offsets pass 32 bits."""

import random

import pytest
import torch

from int8_int4_dequant_amd import qw

pytestmark = pytest.mark.gpu

F32, BF16 = torch.float32, torch.bfloat16
BAR = {F32: 1e-5, BF16: 1e-3}
HALF = {F32: 2.0 ** -24, BF16: 2.0 ** -8}


@pytest.fixture(autouse=True)
def free_afterwards():
    yield
    torch.cuda.empty_cache()


def path(op, m, n, k, dtype, experts=0):
    return qw.qw_block_debug_path(op, experts, m, n, k, qw.TYPES[dtype])


def rand(g, *shape):
    """Normal values, some channels larger."""
    return torch.randn(*shape, generator=g, device="cuda") * torch.rand(shape[-1], generator=g, device="cuda").exp()


def check(y, xv, wv):
    """y against float64 values (of block_unpack: rounded once, 2^-24 each)."""
    ref, base = xv @ wv.T, xv.abs() @ wv.abs().T
    bar = (BAR[y.dtype] + -(-xv.shape[1] // 128) * 2.0 ** -24 + 2.0 ** -23) * base
    assert bool(((y.double() - ref).abs() <= bar + HALF[y.dtype] * (ref.abs() + bar)).all())


def examples(dtype, grouped):
    """{(tile, tile of the rest): the smallest size that takes them}, of 6000 drawn."""
    rng = random.Random(3)
    found = {}
    for _ in range(6000):
        m, n = int(2 ** rng.uniform(4.2, 13)), int(2 ** rng.uniform(4, 13.2))
        k = rng.choice([700, 1100, 1300, 2100, 2432])
        tiles = (path(2, m, n, k, dtype, 7), 0) if grouped else (path(0, m, n, k, dtype), path(1, m, n, k, dtype))
        if tiles not in found or m * n * k < found[tiles][0]:
            found[tiles] = (m * n * k, m, n, k)
    return {tiles: size[1:] for tiles, size in found.items()}


def cases(grouped):
    return [(*size, dtype, *tiles) for dtype in (F32, BF16) for tiles, size in sorted(examples(dtype, grouped).items())]


# the largest tile with fewer blocks of k and, starting at different ones, with 16, 17, 19, 64
LARGEST = [(769, 9288, 700), (2048, 8192, 2048), (2048, 8192, 2100), (2011, 8190, 2432), (2048, 8192, 8192), (2048, 28672, 2100)]
TILES = cases(False) + [(m, n, k, BF16, path(0, m, n, k, BF16), path(1, m, n, k, BF16)) for m, n, k in LARGEST]


def test_the_cases_take_many_tiles():
    for dtype, most in ((F32, 128 * 256), (BF16, 256 * 256)):
        tiles = {c[4] for c in TILES if c[3] is dtype}
        sizes = {(t // 1000) * (t % 1000) for t in tiles}
        assert len(tiles) > 4 and most in sizes and any(c[5] for c in TILES if c[3] is dtype)
    assert sum(c[4] == 256256 and c[2] >= 2048 and c[3] is BF16 for c in TILES) > 3


@pytest.mark.parametrize("m,n,k,dtype,tile,rest", TILES)
@pytest.mark.parametrize("br", [1, 128])
def test_every_tile(m, n, k, dtype, tile, rest, br):
    print("tile", m, n, k, dtype, tile, rest, br, flush=True)
    g = torch.Generator(device="cuda").manual_seed(m + n + k)
    rec, xrec = qw.block_quantize(rand(g, n, k), br), qw.block_quantize(rand(g, m, k), 1)
    y = torch.full((m + 1, n), 7.0, dtype=dtype, device="cuda")
    qw.block_gemm(rec, xrec, out=y[:m])
    assert bool((y[m] == 7).all())
    check(y[:m], qw.block_unpack(xrec).double(), qw.block_unpack(rec).double())
    assert torch.equal(qw.block_gemm(rec, xrec, out_dtype=dtype), y[:m])


@pytest.mark.parametrize("rows,n,k,dtype,tile,rest", cases(True))
@pytest.mark.parametrize("br", [1, 128])
def test_every_grouped_tile(rows, n, k, dtype, tile, rest, br):
    """Seven experts, one with most of the rows and two without any."""
    print("grouped tile", rows, n, k, dtype, tile, br, flush=True)
    counts = [rows // 5, 1, 0, rows // 7, 0, rows // 9]
    counts.append(rows - sum(counts))
    e, used, rows = 7, rows, rows + 5
    g = torch.Generator(device="cuda").manual_seed(n + k)
    rec, xrec = qw.block_quantize(rand(g, e, n, k), br), qw.block_quantize(rand(g, rows, k), 1)
    xrec = dict(xrec, shape=[used, k], codes=xrec["codes"][:used], scales=xrec["scales"][:used])
    off = torch.tensor([sum(counts[:i]) for i in range(e + 1)], dtype=torch.int32, device="cuda")
    y = torch.full((rows, n), 7.0, dtype=dtype, device="cuda")
    qw.block_gemm_grouped(rec, xrec, off, out=y[:used])
    assert bool((y[used:] == 7).all())
    xv, wv, at = qw.block_unpack(xrec).double(), qw.block_unpack(rec), off.tolist()
    for i in range(e):
        if counts[i]:
            check(y[at[i]:at[i + 1]], xv[at[i]:at[i + 1]], wv[i].double())


def mlp_reference(gate_up, down, x, ids, weights):
    """The definition in float64 on the codes' values; codes by block_quantize."""
    e, d, f = down["shape"]
    xv = qw.block_unpack(qw.block_quantize(x, 1)).double()
    gu, dn = qw.block_unpack(gate_up), qw.block_unpack(down)
    y = torch.zeros(len(x), d, dtype=torch.float64, device="cuda")
    for i in range(e):
        at, slot = torch.nonzero(ids == i, as_tuple=True)
        if len(at) == 0:
            continue
        h = xv[at] @ gu[i].double().T
        h = h[:, :f] / (1 + torch.exp(-h[:, :f])) * h[:, f:]
        hv = qw.block_unpack(qw.block_quantize(h.float(), 1)).double()
        y.index_add_(0, at, weights[at, slot].double()[:, None] * (hv @ dn[i].double().T))
    return y


# few rows an expert; more; many, with hidden values in whole blocks and not, and fp32 results
MLP = [
    (40, 6, 64, 520, 1408, BF16), (40, 6, 64, 520, 1408, F32), (500, 4, 64, 520, 1408, BF16), (500, 4, 64, 520, 1408, F32),
    (4099, 2, 6, 520, 1408, BF16), (2600, 4, 8, 2048, 1408, BF16), (4099, 6, 64, 2048, 1408, BF16), (1500, 4, 8, 1003, 512, BF16),
    (3000, 2, 5, 520, 1000, BF16), (4099, 2, 6, 520, 1408, F32),
]


def test_the_cases_take_every_way():
    ways = [(path(3, t * topk, f, d, dtype, e), t * topk * f / 128 ** 2) for t, topk, e, d, f, dtype in MLP]
    assert {w for w, _ in ways} == {1, 2, 3}
    assert sum(w == 3 and tiles > 512 for w, tiles in ways) > 1       # blocks with a second tile
    assert any(path(2, t * topk, d, f, dtype, e) == 256256 for t, topk, e, d, f, dtype in MLP)


@pytest.mark.parametrize("t,topk,experts,d,f,dtype", MLP)
@pytest.mark.parametrize("br", [1, 128])
def test_expert_mlp_ways(t, topk, experts, d, f, dtype, br):
    print("mlp", t, topk, experts, d, f, dtype, br, flush=True)
    g = torch.Generator(device="cuda").manual_seed(t + d)
    gate_up = qw.block_quantize(torch.randn(experts, 2 * f, d, generator=g, device="cuda") * d ** -0.5, br)
    down = qw.block_quantize(torch.randn(experts, d, f, generator=g, device="cuda") * f ** -0.5, br)
    x = torch.randn(t, d, generator=g, device="cuda").to(dtype)
    w = torch.rand(t, topk, generator=g, device="cuda")
    # distinct experts a token, one of them popular, one without tokens, and slots that are out
    score = torch.rand(t, experts, generator=g, device="cuda")
    score[:, 0] += 0.5
    score[:, 1] = -1
    ids = score.topk(topk, 1).indices
    ids[torch.rand(t, topk, generator=g, device="cuda") < 0.05] = -1
    y = qw.moe_mlp(gate_up, down, x, ids, w)
    ref = mlp_reference(gate_up, down, x, ids, w)
    # as in the layer's other test: codes flipped by the 8-bit cores' sums, 3.3e-3 of the norm, and y's rounding
    err = (y.double() - ref).norm(dim=1)
    assert float(err.norm()) <= (3.3e-3 + HALF[dtype]) * float(ref.norm())
    # a row: about one flipped code a slot, by 2^-3 of a value of up to 15 times the f values'
    # root mean square (a product of two normal ones); 128 wrong values would be sqrt(128 / f)
    assert bool((err <= (2 * f ** -0.5 + HALF[dtype]) * ref.norm(dim=1)).all())
    assert torch.equal(qw.moe_mlp(gate_up, down, x, ids, w), y)


@pytest.mark.parametrize("t,topk,d,dtype", [(8500, 4, 4096, BF16), (4300, 4, 4096, F32), (9000, 9, 2048, BF16)])
def test_rows_beyond_the_caches(t, topk, d, dtype):
    """Gather, combine and its gradients on more than 256 MiB of rows."""
    rows = t * topk
    assert rows * d * (4 if dtype is F32 else 2) > 256 << 20
    g = torch.Generator(device="cuda").manual_seed(t)
    ids = torch.randint(-1, 32, (t, topk), generator=g, device="cuda")
    r = qw.moe_sort(ids, 32)
    n, pos, order = int(r["offsets"][-1]), r["pos"].long(), r["order"].long()
    x = torch.randn(t, d, generator=g, device="cuda").to(dtype)
    xs = qw.moe_gather(x, r, out=torch.full((rows, d), 7.0, dtype=dtype, device="cuda"))
    assert torch.equal(xs[:n], x[order[:n] // topk]) and bool((xs[n:] == 7).all())
    ys = torch.randn(rows, d, generator=g, device="cuda").to(dtype)
    ys[n:] = float("nan")
    w = torch.rand(t, topk, generator=g, device="cuda")
    dy = torch.randn(t, d, generator=g, device="cuda").to(dtype)
    dys, dw = qw.moe_combine_backward(dy, ys, r, w, dys=torch.full((rows, d), 7.0, dtype=dtype, device="cuda"))
    y, y32, dx = qw.moe_combine(ys, r, w), qw.moe_combine(ys, r, w, out_dtype=F32), qw.moe_gather_backward(dys, r)
    ref, mag = torch.zeros(t, d, dtype=torch.float64, device="cuda"), torch.zeros(t, d, dtype=torch.float64, device="cuda")
    rdx, mdx = torch.zeros_like(ref), torch.zeros_like(ref)
    for j in range(topk):
        have = pos[:, j] >= 0
        at = torch.where(have, pos[:, j], 0)
        v = torch.where(have[:, None], ys[at].double(), 0.0)
        a = torch.where(have, w[:, j], 0.0).double()[:, None]
        ref += a * v
        mag += a * v.abs()
        dot, base = (dy.double() * v).sum(1), (dy.double() * v).abs().sum(1)
        # a lane's 8 d / 2048 products, then lanes and waves in pairs
        assert bool(((dw[:, j].double() - dot).abs() <= (d / 256 + 16) * 2.0 ** -24 * base).all())
        want = a * dy.double()
        got = dys[at].double()
        assert bool(((got - want).abs() <= (HALF[dtype] + 2.0 ** -24) * want.abs())[have].all())
        rdx += torch.where(have[:, None], got, 0.0)
        mdx += torch.where(have[:, None], got.abs(), 0.0)
    for got, want, m in ((y, ref, mag), (y32, ref, mag), (dx, rdx, mdx)):
        assert bool(((got.double() - want).abs() <= topk * 2.0 ** -24 * m * (1 + 2.0 ** -8) + HALF[got.dtype] * want.abs()).all())
    assert bool((dys[n:] == 7).all())


def test_more_than_2_to_32_elements():
    """Quantizer, unpack, gather and combine on 1.1 million rows of 4096."""
    rows, d, topk = 1_100_000, 4096, 8
    t = rows // topk
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(t, d, generator=g, device="cuda").bfloat16()
    pos = torch.randperm(rows, generator=g, device="cuda").to(torch.int32).view(t, topk)
    xs = qw.moe_gather(x, dict(pos=pos))
    some = torch.tensor([0, 1, 524288, 1048575, 1048576, 1048577, rows - 1], device="cuda")
    back = torch.empty(rows, dtype=torch.int64, device="cuda")
    back[pos.view(-1).long()] = torch.arange(rows, device="cuda") // topk
    assert torch.equal(xs[some], x[back[some]])
    y = qw.moe_combine(xs, dict(pos=pos))
    assert torch.equal(y, (x.float() * 8).bfloat16())      # eight copies: exact
    for br, first in ((1, rows - 300), (128, rows // 128 * 128 - 256)):
        rec = qw.block_quantize(xs, br)
        part = qw.block_quantize(xs[first:].contiguous(), br)
        assert torch.equal(rec["codes"].view(torch.uint8)[first:], part["codes"].view(torch.uint8))
        assert torch.equal(rec["scales"][first // br:], part["scales"])
        out = qw.block_unpack(rec)
        assert torch.equal(out[first:], qw.block_unpack(part))
        del rec, out


def test_product_with_more_than_2_to_32_outputs():
    """131072 x 131400 outputs, 17 billion, and more tiles of 64 x 64 than a launch holds."""
    m, n, k = 131072, 131400, 300
    assert path(0, m, n, k, BF16) > 33000      # tiled
    g = torch.Generator(device="cuda").manual_seed(2)
    rec, xrec = qw.block_quantize(rand(g, n, k), 128), qw.block_quantize(rand(g, m, k), 1)
    y = qw.block_gemm(rec, xrec, out_dtype=BF16)
    xv, wv = qw.block_unpack(xrec), qw.block_unpack(rec).double()
    for rows in (slice(0, 300), slice(32640, 32840), slice(65400, 65700), slice(m - 300, m)):
        check(y[rows], xv[rows].double(), wv)
    cols = torch.tensor([0, 1, 255, 256, 65535, 65536, n - 1], device="cuda")
    check(y[:, cols], xv.double(), wv[cols])
