"""The feed-forward half of a layer in 4 bits as a program runs it: residual and norm,
the block, its gradients; on other streams, captured into graphs, with buffers of the
caller's, and beyond 32-bit offsets."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw
from oracle import mx as om
from tests.test_gpu_mx import bytes_of, host, value, wide

pytestmark = pytest.mark.gpu


def layer(d, f, seed=0):
    rng = np.random.default_rng(seed)
    gu = torch.from_numpy((rng.standard_normal((2 * f, d)) * d ** -0.5).astype(np.float32)).cuda()
    dn = torch.from_numpy((rng.standard_normal((d, f)) * f ** -0.5).astype(np.float32)).cuda()
    return dict(gu=gu, dn=dn, gate_up=qw.mx_quantize(gu), down=qw.mx_quantize(dn), gu_t=qw.mx_quantize(gu, transpose=True),
                dn_t=qw.mx_quantize(dn, transpose=True), gain=torch.from_numpy((1 + 0.1 * rng.standard_normal(d)).astype(np.float32)).cuda())


def forward(p, x, res):
    """(block's output, residual stream, codes of the norm)."""
    c, s = qw.rms_norm(x, p["gain"], residual=res, quantize="mx")
    h = qw.mx_gated(p["gate_up"], c, quantize=True)
    return qw.mx_gemm(p["down"], h, out_dtype=x.dtype), s, c


def backward(p, s, c, dy, ds):
    """Gradients of x (and of the residual), of the gain and of both weights, for the
    gradient dy of the block's output and ds of the residual stream."""
    dh = qw.mx_matmul(p["dn_t"], dy)
    dgu, h = qw.mx_gated_backward(p["gate_up"], c, dh)
    dn = qw.mx_matmul(p["gu_t"], dgu)
    dx, dgain = qw.rms_norm_backward(dn, s, p["gain"], dsum=ds)
    y = qw.rms_norm(s, p["gain"])[0]
    t = lambda v: qw.mx_quantize(v, transpose=True)  # noqa: E731
    return dx, dgain, qw.mx_gemm(t(y), t(dgu)), qw.mx_gemm(t(h), t(dy))


@pytest.mark.parametrize("m,d,f", [(1, 256, 500), (5, 512, 1408), (40, 300, 700), (130, 1000, 333), (600, 512, 1100)])
def test_a_layer_forward(m, d, f):
    """Every call's result from the values that the call before it gave."""
    p = layer(d, f)
    x, res = torch.randn(m, d, device="cuda").bfloat16(), torch.randn(m, d, device="cuda").bfloat16()
    y, s, c = forward(p, x, res)
    assert torch.equal(s, (x.float() + res.float()).bfloat16())
    n = om.norm(host(s), host(p["gain"]), 1e-6)
    assert np.all(np.abs(value(c) - n) <= np.maximum(np.abs(n), np.repeat(2.0 ** (bytes_of(c["scales"]).astype(float) - 127), 32, 1)[:, :d]) / 4 * (1 + 1e-4))
    gate, up = np.split(value(c) @ value(p["gate_up"]).T, 2, axis=1)
    h = qw.mx_gated(p["gate_up"], c, quantize=True)
    g = om.gated(gate, up)
    assert np.all(np.abs(value(h) - g) <= np.maximum(np.abs(g), np.repeat(2.0 ** (bytes_of(h["scales"]).astype(float) - 127), 32, 1)[:, :f]) / 4 * (1 + 1e-3) + 1e-5)
    ref, base = value(h) @ value(p["down"]).T, np.abs(value(h)) @ np.abs(value(p["down"])).T
    assert np.all(np.abs(host(y) - ref) <= 1e-5 * base + 2.0 ** -8 * np.abs(ref))
    assert torch.equal(qw.mx_mlp(p["gate_up"], p["down"], qw.mx_unpack(c)), qw.mx_mlp(p["gate_up"], p["down"], qw.mx_unpack(c)))


def test_a_layers_gradients_against_the_unquantized_layer():
    """4 bits' rounding is a quarter of a value at most and 11 in a hundred of a normal
    one on average; five of them lie in a row here, so that gradients keep their direction:
    a cosine of 0.9 leaves twice the angle that five independent errors of 0.13 make."""
    m, d, f = 512, 512, 1024
    p = layer(d, f)
    x, res, dy, ds = (torch.randn(m, d, device="cuda") for _ in range(4))
    y, s, c = forward(p, x, res)
    got = backward(p, s, c, dy, ds)
    leaves = [t.clone().double().requires_grad_() for t in (s, p["gain"], p["gu"], p["dn"])]
    ls, lg, lgu, ldn = leaves
    n = ls * torch.rsqrt((ls * ls).mean(1, keepdim=True) + 1e-6) * lg
    gate, up = (n @ lgu.T).chunk(2, 1)
    out = (torch.nn.functional.silu(gate) * up) @ ldn.T
    want = torch.autograd.grad([out, ls], leaves, [dy.double(), ds.double()])
    for a, b in zip(got, want):
        cos = torch.nn.functional.cosine_similarity(a.double().flatten(), b.flatten(), dim=0)
        assert a.shape == b.shape and float(cos) > 0.9, float(cos)


def all_calls(p, x, res, dy):
    y, s, c = forward(p, x, res)
    return [y, s, c["codes"], c["scales"], qw.mx_mlp(p["gate_up"], p["down"], x), qw.mx_matmul(p["gate_up"], x), qw.rms_norm(x, p["gain"])[0],
            qw.rms_norm(x, p["gain"], quantize="block")[0]["codes"].view(torch.uint8), *backward(p, s, c, dy, None)]


@pytest.mark.parametrize("m", [1, 4, 40, 300])
def test_on_another_stream(m):
    p = layer(512, 700)
    x, res, dy = (torch.randn(m, 512, device="cuda").bfloat16() for _ in range(3))
    want = all_calls(p, x, res, dy)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = all_calls(p, x, res, dy)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    y = qw.mx_matmul(p["gate_up"], x, stream=side)
    z = qw.mx_mlp(p["gate_up"], p["down"], x, stream=side.cuda_stream)
    side.synchronize()
    assert torch.equal(y, want[5]) and torch.equal(z, want[4])


@pytest.mark.parametrize("m", [1, 40, 300])
def test_two_streams_at_once(m):
    """Calls that overlap in time share nothing."""
    p = layer(512, 1400)
    xs = [torch.randn(m, 512, device="cuda").bfloat16() for _ in range(2)]
    want = [qw.mx_mlp(p["gate_up"], p["down"], x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            got[i].append(qw.mx_mlp(p["gate_up"], p["down"], xs[i], stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


@pytest.mark.parametrize("m", [1, 4, 40, 300])
def test_captured_and_replayed(m):
    """A graph of a whole step, replayed with new inputs between eager work."""
    p = layer(512, 700)
    x, res, dy = (torch.randn(m, 512, device="cuda").bfloat16() for _ in range(3))
    all_calls(p, x, res, dy)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = all_calls(p, x, res, dy)
    for i in range(4):
        for t in (x, res, dy):
            t.copy_(torch.randn(m, 512, device="cuda"))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = all_calls(p, x, res, dy)
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_buffers_of_the_callers():
    """One work buffer for the largest call serves all smaller ones, and nothing behind the
    stated size is touched."""
    L = qw.lib()
    p = layer(700, 900)
    for m in (1, 5, 17, 40, 64, 65, 300):
        for need, call in ((L.qw_mx_mlp_work_bytes(m, 700, 900), lambda w: qw.mx_mlp(p["gate_up"], p["down"], x, work=w)),
                           (L.qw_mx_matmul_work_bytes(m, 700), lambda w: qw.mx_matmul(p["gate_up"], x, work=w)),
                           (L.qw_rms_norm_backward_work_bytes(m, 700), lambda w: qw.rms_norm_backward(x, x, p["gain"], work=w)[1])):
            x = torch.randn(m, 700, device="cuda")
            big = torch.full((need + 4096,), 77, dtype=torch.uint8, device="cuda")
            y = call(big[:need])
            assert bool((big[need:] == 77).all())
            assert torch.equal(y, call(None)) and torch.equal(y, call(torch.zeros(need * 4 + 64, dtype=torch.uint8, device="cuda")))
            if need:
                with pytest.raises(qw.QwError):
                    call(torch.zeros(need - 1, dtype=torch.uint8, device="cuda"))


def test_codes_behind_4_gib():
    """Offsets beyond 32 bits: the last rows of a weight of 2^33 codes, and of its values."""
    n, k = 1 << 20, 9000
    kp = om.pitch(k)
    codes = torch.zeros(n, kp // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, kp // 32), 127, dtype=torch.uint8, device="cuda")
    assert codes.numel() > 1 << 32
    part = qw.mx_quantize(torch.from_numpy(wide(3, 200, k)).cuda())
    codes[-200:], scales[-200:] = part["codes"], part["scales"]
    rec = dict(bits=4, block=32, shape=[n, k], codes=codes, scales=scales)
    for m in (1, 3, 40, 100):
        x = torch.randn(m, k, device="cuda")
        y = qw.mx_matmul(rec, x, out_dtype=torch.bfloat16)
        assert not bool(y[:, :-200].any())
        ref = qw.mx_matmul(dict(part), x)
        tol = (4 + k / 64) * 2.0 ** -22 * (qw.mx_unpack(qw.mx_quantize(x)).abs() @ qw.mx_unpack(part).abs().T) + 2.0 ** -8 * ref.abs()
        assert bool(((y[:, -200:].float() - ref).abs() <= tol).all())
    del y
    h = qw.mx_gated(rec, qw.mx_quantize(torch.randn(70, k, device="cuda")), out_dtype=torch.bfloat16)
    assert h.shape == (70, n // 2) and not bool(h[:, : n // 2 - 200].any())


def test_rows_behind_4_gib():
    """The quantizers and the norm on rows beyond 2^32 bytes."""
    rows, d = 140000, 16384
    x = torch.zeros(rows, d, dtype=torch.bfloat16, device="cuda")
    tail = torch.randn(3, d, device="cuda").bfloat16()
    x[-3:] = tail
    w = torch.ones(d, device="cuda")
    y, s = qw.rms_norm(x, w)
    want = qw.rms_norm(tail.clone(), w)[0]
    assert torch.equal(y[-3:], want) and not bool(y[:1000].any())
    del y, s
    rec = qw.mx_quantize(x)
    assert torch.equal(rec["codes"][-3:], qw.mx_quantize(tail)["codes"])
    rec = qw.mx_quantize(x, transpose=True)
    last = qw.mx_quantize(x[-32 * 5:].clone(), transpose=True)   # 140000 rows are 4375 whole blocks
    assert torch.equal(rec["codes"][:, : rows // 2][:, -80:], last["codes"][:, :80])
