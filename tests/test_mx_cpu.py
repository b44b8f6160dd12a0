"""4-bit codes, RMS norm and gated products without a GPU: the oracle's own pins and the
refusals of the C ABI and of the binding, before anything is enqueued."""

import ctypes
import inspect
import os
import re

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw
from oracle import mx as om

MAXE = 1 << 36
I64 = (1 << 63) - 1
P = 4096  # an aligned address that no refused call reads
OK, ESHAPE, EM, ENULL, EWORK, EARG = 0, -3, -4, -5, -8, -9
NAN, INF = float("nan"), float("inf")


def test_header_and_binding_agree():
    txt = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "qw_mx.h")).read()
    txt = re.sub(r"/\*.*?\*/", "", txt, flags=re.S)
    assert sorted(set(re.findall(r"\b(qw_[a-z_]+)\s*\(", txt))) == sorted(qw.EXPORTS_MX)
    raw = ctypes.CDLL(qw.LIB_PATH)
    for name in qw.EXPORTS_MX:
        assert ctypes.cast(getattr(raw, name), ctypes.c_void_p).value and callable(getattr(qw, name))
    assert re.search(r"#define QW_MX_BLOCK 32\b", txt) and qw.MX_BLOCK == 32


# ---------------------------------------------------------------- the oracle


def test_oracle_codes():
    """Nearest value, ties to the even code, clipped; by comparison with every code."""
    v = np.concatenate([np.linspace(-8, 8, 4097), (om.VALUES[1:] + om.VALUES[:-1]) / 2])
    got = om.VALUES[om.encode(v) & 7]
    best = np.abs(np.abs(v)[:, None] - om.VALUES).min(1)
    assert np.array_equal(np.abs(np.abs(v) - got), best)
    assert om.encode([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.0]).tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 8]


def test_oracle_scales():
    tops = [0.0, 1.0, 1.999, 2.0, 3.9, 4.0, 7.9, 2.0 ** -125, 2.0 ** -126, 2.0 ** -149, 3.4e38, np.inf, np.nan]
    assert [om.scale_byte(t) for t in tops] == [127, 125, 125, 126, 126, 127, 127, 0, 0, 0, 252, 255, 255]


def test_oracle_quantize_within_a_quarter():
    """Half a step is at most a quarter of a value of a scale or more, and a quarter of a scale below."""
    w = np.random.default_rng(1).standard_normal((5, 300))
    codes, scales = om.quantize(w)
    assert codes.shape == (5, 256) and scales.shape == (5, 16)
    assert not codes[:, 150:].any() and np.all(scales[:, 10:] == 127)
    s = np.repeat(2.0 ** (scales.astype(float) - 127), 32, 1)[:, :300]
    assert np.all(np.abs(om.values(codes, scales, 300) - w) <= np.maximum(np.abs(w) / 4, s / 4))


def test_oracle_gradients_against_differences():
    rng = np.random.default_rng(2)
    gate, up, dh, e = rng.standard_normal(200) * 4, rng.standard_normal(200), rng.standard_normal(200), 1e-6
    dg, du = om.gated_backward(gate, up, dh)
    assert np.allclose(dg, dh * (om.gated(gate + e, up) - om.gated(gate - e, up)) / (2 * e), rtol=1e-6, atol=1e-8)
    assert np.allclose(du, dh * (om.gated(gate, up + e) - om.gated(gate, up - e)) / (2 * e), rtol=1e-6, atol=1e-8)
    s, w, dy, v = rng.standard_normal((3, 50)), rng.standard_normal(50), rng.standard_normal((3, 50)), rng.standard_normal((3, 50))
    ds, dw = om.norm_backward(dy, s, w, 1e-5, None)
    diff = (dy * (om.norm(s + e * v, w, 1e-5) - om.norm(s - e * v, w, 1e-5))).sum() / (2 * e)
    assert abs((ds * v).sum() - diff) < 1e-6
    assert np.allclose(dw, (dy * om.norm(s, None, 1e-5)).sum(0))


# ---------------------------------------------------------------- the C ABI


def test_sizes():
    L = qw.lib()
    assert [L.qw_mx_pitch(k) for k in (0, 1, 512, 513, MAXE)] == [0, 512, 512, 1024, MAXE]
    assert L.qw_mx_pitch(-1) == L.qw_mx_pitch(I64) == L.qw_mx_pitch(MAXE + 1) == -1
    assert L.qw_mx_matmul_work_bytes(100, 513) >= 100 * (512 + 32) and L.qw_mx_matmul_work_bytes(1, 4096) == L.qw_mx_matmul_work_bytes(0, 513) == 0
    for a in ((-1, 8), (8, -1), (8, I64), (I64, 8), (1, (1 << 22) + 1), (MAXE // 512 + 1, 1)):
        assert L.qw_mx_matmul_work_bytes(*a) == -1
    assert L.qw_rms_norm_backward_work_bytes(3, 100) >= 3 * 400
    assert L.qw_rms_norm_backward_work_bytes(-1, 4) == L.qw_rms_norm_backward_work_bytes(2, I64) == -1
    for a in ((-1, 4, 4), (4, -1, 4), (4, 4, -1), (I64, 4, 4), (4, I64, 4), (4, 4, I64), (4, (1 << 22) + 1, 4), (4, 4, (1 << 22) + 1)):
        assert L.qw_mx_mlp_work_bytes(*a) == -1


def test_work_sizes_grow_with_every_argument():
    L = qw.lib()
    for f, steps in ((L.qw_mx_matmul_work_bytes, ((1, 8, 9, 16, 17, 300), (1, 511, 512, 513, 9000, 13000, 40000))),
                     (L.qw_rms_norm_backward_work_bytes, ((1, 4, 1023, 1024, 1025, 9000), (1, 64, 512, 5000, 20000))),
                     (lambda m, d: L.qw_mx_mlp_work_bytes(m, d, 700), ((1, 8, 16, 17, 33, 300), (1, 512, 513, 20000))),
                     (lambda m, f: L.qw_mx_mlp_work_bytes(m, 700, f), ((1, 8, 16, 17, 33, 300), (1, 512, 513, 20000)))):
        got = np.array([[f(a, b) for b in steps[1]] for a in steps[0]])
        assert np.all(np.diff(got, axis=0) >= 0) and np.all(np.diff(got, axis=1) >= 0)


@pytest.mark.parametrize("want,args", [
    (EARG, (2, 4, 64, 0, P, P, P)), (EARG, (-1, 4, 64, 0, P, P, P)), (EARG, (0, 4, 64, 2, P, P, P)),
    (ESHAPE, (0, -1, 64, 0, P, P, P)), (ESHAPE, (0, 4, -64, 0, P, P, P)), (ESHAPE, (1, 4, I64, 0, P, P, P)),
    (ESHAPE, (0, MAXE, 1, 0, P, P, P)),            # a row of codes holds 512 values
    (ESHAPE, (1, 1, MAXE, 0, P, P, P)),
    (ENULL, (0, 4, 64, 0, None, P, P)), (ENULL, (0, 4, 64, 0, P, None, P)), (ENULL, (1, 4, 64, 0, P, P, None)),
    (EARG, (0, 4, 64, 0, P, P + 8, P)), (EARG, (0, 4, 64, 0, P, P, P + 8)),
    (OK, (0, 0, 64, 0, None, None, None)), (OK, (1, 4, 0, 0, None, None, None)),
])
def test_quantize_refusals(want, args):
    assert qw.lib().qw_mx_quantize(*args, None) == want


def test_unpack_refusals():
    f = qw.lib().qw_mx_unpack
    assert f(-1, 4, P, P, P, None) == f(4, I64, P, P, P, None) == f(MAXE, 1, P, P, P, None) == ESHAPE
    assert f(4, 4, None, P, P, None) == f(4, 4, P, None, P, None) == f(4, 4, P, P, None, None) == ENULL
    assert f(4, 4, P + 8, P, P, None) == f(4, 4, P, P + 8, P, None) == EARG
    assert f(0, 4, None, None, None, None) == OK


PRODUCT = [
    (EARG, dict(t=2)), (EARG, dict(c=P + 8)), (EARG, dict(s=P + 8)), (EARG, dict(xc=P + 4)), (EARG, dict(xs=P + 4)),
    (ESHAPE, dict(n=-1)), (ESHAPE, dict(k=-1)), (ESHAPE, dict(k=I64)), (ESHAPE, dict(n=I64)), (ESHAPE, dict(k=(1 << 22) + 1)),
    (EM, dict(m=-1)), (EM, dict(m=I64)), (EM, dict(n=1 << 20, m=1 << 20)), (EM, dict(k=1, m=MAXE // 512 + 1)),
    (ENULL, dict(c=None)), (ENULL, dict(s=None)), (ENULL, dict(xc=None)), (ENULL, dict(xs=None)), (ENULL, dict(y=None)),
    (ENULL, dict(k=0, y=None)), (OK, dict(m=0, c=None, s=None, xc=None, xs=None, y=None)),
    (OK, dict(n=0, c=None, s=None, xc=None, xs=None, y=None)),
]


@pytest.mark.parametrize("want,over", PRODUCT)
def test_product_refusals(want, over):
    a = dict(n=8, k=64, c=P, s=P, m=4, xc=P, xs=P, t=0, y=P) | over
    L = qw.lib()
    head = (a["n"], a["k"], a["c"], a["s"], a["m"], a["xc"], a["xs"])
    assert L.qw_mx_gemm(*head, a["t"], a["y"], None) == want
    assert L.qw_mx_gated(*head, a["t"], a["y"], None) == want
    assert L.qw_mx_gated_backward(*head, a["t"], P, a["y"], None, None) == want
    if "t" not in over:
        assert L.qw_mx_gated_codes(*head, a["y"], P, None) == want
    if not {"xc", "xs"} & set(over) or a["m"] * a["n"] == 0:
        work = lambda w, b: L.qw_mx_matmul(a["n"], a["k"], a["c"], a["s"], a["m"], 1, a["xc"], a["t"], a["y"], w, b, None)  # noqa: E731
        assert work(P, 1 << 40) == want


@pytest.mark.parametrize("want,n,m", [(ESHAPE, MAXE // 512 + 2, 1), (ESHAPE, MAXE, 1), (EM, 2, MAXE // 512 + 1), (EM, 1, MAXE)])
def test_sides_too_long_for_a_launch_without_any_k(want, n, m):
    L = qw.lib()
    assert L.qw_mx_gemm(n, 0, P, P, m, P, P, 0, P, None) == want
    assert L.qw_mx_matmul(n, 0, P, P, m, 1, P, 0, P, P, 1 << 40, None) == want
    assert L.qw_mx_gated(max(n // 2, 1), 0, P, P, m, P, P, 0, P, None) == want
    assert L.qw_mx_debug_path(0, m, n, 0) == want


def test_more_product_refusals():
    L = qw.lib()
    assert L.qw_mx_gated_backward(8, 64, P, P, 4, P, P, 0, None, P, P, None) == ENULL
    assert L.qw_mx_gated_codes(8, 64, P, P, 4, P, P, P, None, None) == ENULL
    assert L.qw_mx_gated_codes(8, 64, P, P, 4, P, P, P + 8, P, None) == EARG
    assert L.qw_mx_gated_codes(8, 64, P, P, 4, P, P, P, P + 8, None) == EARG
    mm = lambda m=400, x=P, xt=0, w=P, b=1 << 30: L.qw_mx_matmul(8, 64, P, P, m, xt, x, 0, P, w, b, None)  # noqa: E731
    assert mm(xt=5) == EARG and mm(x=None) == ENULL
    assert mm(w=None) == mm(b=400) == mm(w=P + 8) == EWORK
    mlp = lambda d=8, f=8, g=P, gs=P, dn=P, dsc=P, m=400, xt=0, x=P, yt=0, y=P, w=P, b=1 << 30: L.qw_mx_mlp(  # noqa: E731
        d, f, g, gs, dn, dsc, m, xt, x, yt, y, w, b, None)
    assert mlp(xt=2) == mlp(yt=2) == mlp(g=P + 8) == mlp(gs=P + 8) == mlp(dn=P + 8) == mlp(dsc=P + 8) == EARG
    assert mlp(d=-1) == mlp(f=-1) == mlp(d=I64) == mlp(f=I64) == mlp(d=(1 << 22) + 1) == mlp(f=(1 << 22) + 1) == ESHAPE
    assert mlp(m=-1) == mlp(m=I64) == EM
    assert mlp(g=None) == mlp(gs=None) == mlp(dn=None) == mlp(dsc=None) == mlp(x=None) == mlp(y=None) == ENULL
    assert mlp(w=None) == mlp(b=64) == mlp(w=P + 8) == EWORK
    assert mlp(m=0, x=None, y=None, w=None) == mlp(d=0, x=None, y=None, w=None) == OK


NORM = [
    (EARG, dict(t=2)), (EARG, dict(wt=7)), (EARG, dict(eps=-1e-6)), (EARG, dict(eps=NAN)), (EARG, dict(eps=INF)),
    (ESHAPE, dict(rows=-1)), (ESHAPE, dict(d=-1)), (ESHAPE, dict(d=I64)), (ESHAPE, dict(rows=I64)), (ESHAPE, dict(rows=1 << 20, d=1 << 20)),
    (ENULL, dict(x=None)), (ENULL, dict(y=None)), (OK, dict(rows=0, x=None, y=None)), (OK, dict(d=0, x=None, y=None)),
]


@pytest.mark.parametrize("want,over", NORM)
def test_norm_refusals(want, over):
    a = dict(rows=4, d=64, t=0, x=P, res=None, sum=None, wt=0, w=P, eps=1e-6, y=P) | over
    L = qw.lib()
    head = (a["rows"], a["d"], a["t"], a["x"], a["res"], a["sum"], a["wt"], a["w"], a["eps"])
    assert L.qw_rms_norm(*head, 0, a["y"], None) == want
    assert L.qw_rms_norm_block(*head, a["y"], P, None) == want
    assert L.qw_rms_norm_mx(*head, a["y"], P, None) == want
    back = L.qw_rms_norm_backward(a["rows"], a["d"], a["t"], a["x"], a["y"], a["wt"], a["w"], a["eps"], None, P, None, None, 0, None)
    assert back == want


def test_more_norm_refusals():
    L = qw.lib()
    head = (4, 64, 0, P, None, None, 0, P, 1e-6)
    assert L.qw_rms_norm(*head, 2, P, None) == EARG
    assert L.qw_rms_norm_block(*head, P + 8, P, None) == L.qw_rms_norm_mx(*head, P + 8, P, None) == L.qw_rms_norm_mx(*head, P, P + 8, None) == EARG
    assert L.qw_rms_norm_block(*head, P, None, None) == L.qw_rms_norm_mx(*head, P, None, None) == ENULL
    one = (MAXE, 1, 0, P, None, None, 0, P, 1e-6)    # a row of codes holds 128 or 512 values
    assert L.qw_rms_norm_block(*one, P, P, None) == L.qw_rms_norm_mx(*one, P, P, None) == ESHAPE
    back = lambda rows=4, ds=P, dw=P, w=P, b=1 << 20: L.qw_rms_norm_backward(rows, 64, 0, P, P, 0, P, 1e-6, None, ds, dw, w, b, None)  # noqa: E731
    assert back(w=None) == back(b=100) == back(w=P + 8) == EWORK
    assert back(ds=None, dw=None, w=None) == back(rows=0, dw=None, w=None) == OK


# ---------------------------------------------------------------- the binding


def _rec(n, k):
    kp = om.pitch(k)
    return dict(bits=4, block=32, shape=[n, k], codes=torch.zeros(n, kp // 2, dtype=torch.uint8), scales=torch.zeros(n, kp // 32, dtype=torch.uint8))


Z = torch.zeros


@pytest.mark.parametrize("call", [
    lambda: qw.mx_quantize(Z(4, 8, dtype=torch.float16)),
    lambda: qw.mx_quantize(Z(8, 4).t()),
    lambda: qw.mx_quantize(Z(2, 8, 4)),
    lambda: qw.mx_quantize(Z(4, 8)),                                # a host tensor
    lambda: qw.mx_unpack(dict(_rec(4, 8), shape=[5, 8])),
    lambda: qw.mx_unpack(dict(_rec(4, 8), bits=8)),
    lambda: qw.mx_unpack(dict(_rec(4, 8), block=16)),
    lambda: qw.mx_unpack(dict(_rec(4, 8), scales=Z(4, 16))),
    lambda: qw.mx_unpack(_rec(4, 8), out=Z(4, 9)),
    lambda: qw.mx_gemm(_rec(4, 8), _rec(3, 9)),
    lambda: qw.mx_gemm(_rec(4, 8), _rec(3, 8), out_dtype=torch.float16),
    lambda: qw.mx_gemm(_rec(4, 8), _rec(3, 8), out=Z(3, 5)),
    lambda: qw.mx_gemm(_rec(4, 8), _rec(3, 8)),                     # host tensors
    lambda: qw.mx_matmul(_rec(4, 8), Z(3, 9)),
    lambda: qw.mx_matmul(_rec(4, 8), Z(3, 8, dtype=torch.int8)),
    lambda: qw.mx_matmul(_rec(4, 8), Z(3, 16)[:, ::2]),
    lambda: qw.mx_gated(_rec(5, 8), _rec(3, 8)),                    # an odd number of rows
    lambda: qw.mx_gated(_rec(4, 8), _rec(3, 8), out=Z(3, 2), quantize=True),
    lambda: qw.mx_gated(_rec(4, 8), _rec(3, 8), out=Z(3, 4)),
    lambda: qw.mx_gated_backward(_rec(4, 8), _rec(3, 8), Z(3, 4)),
    lambda: qw.mx_gated_backward(_rec(4, 8), _rec(3, 8), Z(3, 2), out=Z(3, 2)),
    lambda: qw.mx_gated_backward(_rec(4, 8), _rec(3, 8), Z(3, 2), h=Z(3, 2).bfloat16()),
    lambda: qw.mx_mlp(_rec(8, 8), _rec(8, 5), Z(3, 8)),
    lambda: qw.mx_mlp(_rec(8, 8), _rec(7, 4), Z(3, 8)),
    lambda: qw.mx_mlp(_rec(8, 8), _rec(8, 4), Z(3, 7)),
    lambda: qw.rms_norm(Z(3, 8, dtype=torch.float16)),
    lambda: qw.rms_norm(Z(3, 16)[:, ::2]),
    lambda: qw.rms_norm(Z(8)),
    lambda: qw.rms_norm(Z(3, 8), Z(7)),
    lambda: qw.rms_norm(Z(3, 8), Z(8, dtype=torch.float16)),
    lambda: qw.rms_norm(Z(3, 8), residual=Z(2, 8)),
    lambda: qw.rms_norm(Z(3, 8), residual=Z(3, 8).bfloat16()),
    lambda: qw.rms_norm(Z(3, 8), sum=Z(3, 9)),
    lambda: qw.rms_norm(Z(3, 8), quantize="fp8"),
    lambda: qw.rms_norm(Z(3, 8), quantize="mx", out=Z(3, 8)),
    lambda: qw.rms_norm(Z(3, 8)),                                   # a host tensor
    lambda: qw.rms_norm_backward(Z(3, 8), Z(3, 9)),
    lambda: qw.rms_norm_backward(Z(3, 8).bfloat16(), Z(3, 8)),
    lambda: qw.rms_norm_backward(Z(3, 8), Z(3, 8), Z(8), dweight=Z(8).bfloat16()),
    lambda: qw.rms_norm_backward(Z(3, 8), Z(3, 8), dsum=Z(3, 7)),
    lambda: qw.rms_norm_backward(Z(3, 8), Z(3, 8), ds=Z(3, 8).bfloat16()),
])
def test_binding_refuses_before_any_call(call):
    with pytest.raises(ValueError):
        call()


def test_every_call_takes_its_stream_last():
    for name in ("mx_quantize", "mx_unpack", "mx_gemm", "mx_matmul", "rms_norm", "rms_norm_backward", "mx_gated", "mx_gated_backward", "mx_mlp"):
        f = getattr(qw, name)
        parameters = list(inspect.signature(f).parameters)
        assert parameters[-1] == "stream" and f.__wrapped__.__code__.co_varnames.index("stream") == len(parameters) - 1
