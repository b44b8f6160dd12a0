"""Block-scaled e4m3 and expert calls without a GPU: the oracle's own pins and
the refusals of the C ABI and of the binding, before anything is enqueued."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw
from oracle import block as ob

MAXE = 1 << 36
I64 = (1 << 63) - 1
P = 4096  # an aligned address that no refused call reads
OK, EGROUP, ESHAPE, EM, ENULL, EWORK, EARG = 0, -2, -3, -4, -5, -8, -9


def test_oracle_codes_are_torch_codes():
    """Every bf16 value in range against torch's own conversion, and the midpoints."""
    bits = np.arange(1 << 16, dtype=np.uint32) << 16
    v = bits.view(np.float32)
    v = v[np.isfinite(v) & (np.abs(v) <= 448)]
    mid = ((ob.VALUES[1:] + ob.VALUES[:-1]) / 2).astype(np.float32)
    mid = np.concatenate([mid, np.nextafter(mid, np.float32(0)), np.nextafter(mid, np.float32(500))])
    v = np.concatenate([v, mid, -mid])
    want = torch.from_numpy(v).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ob.encode(v), want)
    assert np.array_equal(ob.decode(want), torch.from_numpy(want).view(torch.float8_e4m3fn).double().numpy())


def test_oracle_quantize_halves_a_step():
    rng = np.random.default_rng(1)
    w = rng.standard_normal((130, 300)).astype(np.float32)
    for br in (1, 128):
        codes, scales = ob.quantize(w, br)
        assert codes.shape == (130, 384) and not codes[:, 300:].any()
        v = ob.values(codes, scales, br, 300)
        s = np.repeat(np.repeat(scales, 128, 1), br, 0)[:130, :300]
        # half a step: 2^-4 of the value, or half of 2^-9 scales below the normal range
        assert np.all(np.abs(v - w) <= np.maximum(np.abs(w) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 1e-6))


def test_oracle_sort():
    pos, order, off = ob.sort(np.array([[2, 0], [5, 2], [0, -1]]), 3)
    assert pos.tolist() == [[2, 0], [-1, 3], [1, -1]]
    assert order.tolist() == [1, 4, 0, 3, -1, -1] and off.tolist() == [0, 2, 2, 4]


def test_sizes():
    L = qw.lib()
    assert [L.qw_block_pitch(k) for k in (0, 1, 128, 129, MAXE)] == [0, 128, 128, 256, MAXE]
    assert L.qw_block_pitch(-1) == L.qw_block_pitch(I64) == -1
    assert L.qw_block_num_scales(128, 129, 300) == 6
    assert L.qw_block_num_scales(1, 129, 300) == 387
    for br, n, k in ((0, 4, 4), (2, 4, 4), (128, -1, 4), (1, 4, I64), (1, MAXE, 2)):
        assert L.qw_block_num_scales(br, n, k) == -1
    assert L.qw_block_matmul_work_bytes(1, 4096) == 0
    assert L.qw_block_matmul_work_bytes(100, 129) >= 100 * 256 + 100 * 8
    assert L.qw_block_matmul_work_bytes(-1, 8) == L.qw_block_matmul_work_bytes(8, I64) == -1
    assert L.qw_moe_sort_work_bytes(10, 2, 8) == 0
    assert L.qw_moe_sort_work_bytes(1 << 20, 8, 64) > 0
    for a in ((-1, 2, 8), (2, 0, 8), (2, 2, 0), (2, 2, 513), (1 << 30, 2, 8), (I64, I64, 8)):
        assert L.qw_moe_sort_work_bytes(*a) == -1
    assert L.qw_moe_mlp_work_bytes(4, 2, 8, 256, 128) > 0
    for a in ((-1, 2, 8, 4, 4), (4, 2, 8, -4, 4), (4, 2, 8, I64, 4), (4, 2, 8, 4, I64), (4, 2, 8, 4, -1)):
        assert L.qw_moe_mlp_work_bytes(*a) == -1


@pytest.mark.parametrize("want,args", [
    (EARG, (64, 1, 4, 128, 0, P, P, P)), (EARG, (1, 1, 4, 128, 2, P, P, P)),
    (ESHAPE, (1, -1, 4, 128, 0, P, P, P)), (ESHAPE, (1, 1, -4, 128, 0, P, P, P)),
    (ESHAPE, (1, 1, 4, I64, 0, P, P, P)), (ESHAPE, (1, MAXE, 2, 1, 0, P, P, P)),
    (ESHAPE, (1, 1, MAXE, 1, 0, P, P, P)),        # a row of codes has 128 bytes
    (ENULL, (1, 1, 4, 128, 0, None, P, P)), (ENULL, (1, 1, 4, 128, 0, P, None, P)),
    (ENULL, (1, 1, 4, 128, 0, P, P, None)), (EARG, (1, 1, 4, 128, 0, P, P + 8, P)),
    (OK, (1, 0, 4, 128, 0, None, None, None)), (OK, (128, 1, 0, 128, 0, None, None, None)),
    (OK, (128, 1, 4, 0, 0, None, None, None)),
])
def test_quantize_refusals(want, args):
    assert qw.lib().qw_block_quantize(*args, None) == want


def test_unpack_and_swiglu_refusals():
    L = qw.lib()
    assert L.qw_block_unpack(3, 1, 4, 4, P, P, P, None) == EARG
    assert L.qw_block_unpack(1, 1, 4, -4, P, P, P, None) == ESHAPE
    assert L.qw_block_unpack(1, 1, 4, 4, P + 1, P, P, None) == EARG
    assert L.qw_block_unpack(1, 1, 4, 4, P, P, None, None) == ENULL
    assert L.qw_block_quantize_swiglu(4, 4, 3, P, None, P, P, None) == EARG
    assert L.qw_block_quantize_swiglu(-4, 4, 0, P, None, P, P, None) == ESHAPE
    assert L.qw_block_quantize_swiglu(4, 4, 0, None, None, P, P, None) == ENULL
    assert L.qw_block_quantize_swiglu(0, 4, 0, None, None, None, None, None) == OK


@pytest.mark.parametrize("want,args", [
    (EARG, (2, 8, 128, P, P, 4, P, P, 0, P)), (EARG, (1, 8, 128, P, P, 4, P, P, 5, P)),
    (EARG, (1, 8, 128, P + 4, P, 4, P, P, 0, P)), (EARG, (1, 8, 128, P, P, 4, P + 4, P, 0, P)),
    (ESHAPE, (1, -8, 128, P, P, 4, P, P, 0, P)), (ESHAPE, (1, 8, I64, P, P, 4, P, P, 0, P)),
    (EM, (1, 8, 128, P, P, -4, P, P, 0, P)), (EM, (1, 8, 128, P, P, I64, P, P, 0, P)),
    (EM, (1, 1 << 20, 0, P, P, 1 << 20, P, P, 0, P)), (ESHAPE, (1, 8, (1 << 22) + 1, P, P, 4, P, P, 0, P)),
    (ENULL, (1, 8, 128, None, P, 4, P, P, 0, P)), (ENULL, (1, 8, 128, P, None, 4, P, P, 0, P)),
    (ENULL, (1, 8, 128, P, P, 4, None, P, 0, P)), (ENULL, (1, 8, 128, P, P, 4, P, None, 0, P)),
    (ENULL, (1, 8, 128, P, P, 4, P, P, 0, None)), (ENULL, (1, 8, 0, None, None, 4, None, None, 0, None)),
    (OK, (1, 8, 128, None, None, 0, None, None, 0, None)), (OK, (1, 0, 128, None, None, 4, None, None, 0, None)),
])
def test_gemm_refusals(want, args):
    assert qw.lib().qw_block_gemm(*args, None) == want


@pytest.mark.parametrize("want,args", [
    (EARG, (1, 8, 128, P, P, 4, 7, P, 0, P, None, 0)), (EARG, (1, 8, 128, P, P, 4, 0, P, 7, P, None, 0)),
    (EARG, (1, 8, 128, P + 2, P, 4, 0, P, 0, P, None, 0)),
    (EM, (1, 8, 128, P, P, -1, 0, P, 0, P, None, 0)), (ENULL, (1, 8, 128, P, P, 4, 0, None, 0, P, None, 0)),
    (EWORK, (1, 8, 128, P, P, 400, 0, P, 0, P, None, 1 << 30)), (EWORK, (1, 8, 128, P, P, 400, 0, P, 0, P, P, 400)),
    (EWORK, (1, 8, 128, P, P, 400, 0, P, 0, P, P + 4, 1 << 30)),
    (OK, (1, 8, 128, None, None, 0, 0, None, 0, None, None, 0)),
])
def test_matmul_refusals(want, args):
    assert qw.lib().qw_block_matmul(*args, None) == want


@pytest.mark.parametrize("want,args", [
    (EARG, (1, 0, 8, 128, P, P, 4, P, P, P, 0, P)), (EARG, (1, 513, 8, 128, P, P, 4, P, P, P, 0, P)),
    (EARG, (4, 2, 8, 128, P, P, 4, P, P, P, 0, P)), (EARG, (1, 2, 8, 128, P, P, 4, P, P, P, 9, P)),
    (ESHAPE, (1, 2, -8, 128, P, P, 4, P, P, P, 0, P)), (ESHAPE, (1, 512, 1 << 30, 128, P, P, 4, P, P, P, 0, P)),
    (EM, (1, 2, 8, 128, P, P, -4, P, P, P, 0, P)), (EM, (1, 2, 8, 128, P, P, (1 << 30) + 1, P, P, P, 0, P)),
    (ENULL, (1, 2, 8, 128, P, P, 4, P, P, None, 0, P)), (ENULL, (1, 2, 8, 128, P, P, 4, P, P, P, 0, None)),
    (OK, (1, 2, 8, 128, None, None, 0, None, None, None, 0, None)),
])
def test_grouped_refusals(want, args):
    assert qw.lib().qw_block_gemm_grouped(*args, None) == want


def test_moe_refusals():
    L = qw.lib()
    sort = lambda t=4, k=2, e=8, b=4, ids=P, pos=P, order=P, off=P, w=None, wb=0: L.qw_moe_sort(  # noqa: E731
        t, k, e, b, ids, pos, order, off, w, wb, None)
    assert sort(k=0) == sort(e=0) == sort(e=513) == sort(b=2) == EARG
    assert sort(t=-1) == sort(t=1 << 30) == sort(t=I64, k=I64) == ESHAPE
    assert sort(ids=None) == sort(pos=None) == sort(off=None) == ENULL
    assert sort(t=1 << 20) == sort(t=1 << 20, w=P, wb=8) == EWORK
    gather = lambda t=4, k=2, d=8, r=8, ty=0, x=P, pos=P, xs=P: L.qw_moe_gather(  # noqa: E731
        t, k, d, r, ty, x, pos, xs, None)
    assert gather(k=0) == gather(ty=2) == EARG
    assert gather(t=-1) == gather(d=-1) == gather(d=I64) == gather(r=-1) == gather(r=1 << 31) == ESHAPE
    assert gather(x=None) == gather(pos=None) == gather(xs=None) == ENULL
    assert gather(t=0, x=None, pos=None, xs=None) == gather(r=0, xs=None) == OK
    block = lambda c=P, k=2, ty=0: L.qw_moe_gather_block(4, k, 8, 8, ty, P, P, c, P, None)  # noqa: E731
    assert block(k=0) == block(ty=-1) == block(c=P + 8) == EARG and block(c=None) == ENULL
    comb = lambda t=4, k=2, ys=P, ty=0, yt=0, y=P: L.qw_moe_combine(t, k, 8, 8, ty, ys, P, None, yt, y, None)  # noqa: E731
    assert comb(k=0) == comb(ty=4) == comb(yt=4) == EARG and comb(t=-4) == ESHAPE
    assert comb(ys=None) == comb(y=None) == ENULL and comb(t=0, ys=None, y=None) == OK
    back = lambda k=2, dy=P, ys=P, dys=P, dw=P, ty=1: L.qw_moe_combine_backward(  # noqa: E731
        4, k, 8, 8, ty, dy, ys, P, None, dys, dw, None)
    assert back(k=0) == back(ty=9) == EARG
    assert back(dy=None) == back(ys=None) == ENULL and back(dys=None, dw=None) == OK
    mlp = lambda br=1, e=2, d=8, f=8, g=P, t=4, k=2, xt=0, x=P, b=4, ids=P, yt=0, y=P, w=P, wb=1 << 30: L.qw_moe_mlp(  # noqa: E731
        br, e, d, f, g, P, P, P, t, k, xt, x, b, ids, None, yt, y, w, wb, None)
    assert mlp(br=0) == mlp(e=0) == mlp(k=0) == mlp(xt=2) == mlp(yt=2) == mlp(b=1) == mlp(g=P + 4) == EARG
    assert mlp(t=-1) == mlp(d=-1) == mlp(f=-1) == mlp(d=I64) == mlp(f=I64) == ESHAPE
    assert mlp(x=None) == mlp(ids=None) == mlp(y=None) == mlp(g=None) == ENULL
    assert mlp(w=None) == mlp(wb=64) == mlp(w=P + 8) == EWORK
    assert mlp(t=0, x=None, ids=None, y=None, w=None) == OK


def _rec(n, k, br=128, e=None):
    lead = () if e is None else (e,)
    kp = ob.pitch(k)
    return dict(block_rows=br, shape=[*lead, n, k], codes=torch.zeros(*lead, n, kp, dtype=torch.uint8),
                scales=torch.ones(*lead, -(-n // br), kp // 128))


@pytest.mark.parametrize("call", [
    lambda: qw.block_quantize(torch.zeros(4, 8, dtype=torch.float16)),
    lambda: qw.block_quantize(torch.zeros(8, 4).t()),
    lambda: qw.block_quantize(torch.zeros(4, 8), 64),
    lambda: qw.block_quantize(torch.zeros(8)),
    lambda: qw.block_quantize(torch.zeros(4, 8)),                       # a host tensor
    lambda: qw.block_quantize_swiglu(torch.zeros(4, 7)),
    lambda: qw.block_quantize_swiglu(torch.zeros(4, 8), torch.zeros(2, dtype=torch.int32)),
    lambda: qw.block_unpack(dict(_rec(4, 8), shape=[5, 8])),
    lambda: qw.block_unpack(dict(_rec(4, 8), block_rows=16)),
    lambda: qw.block_unpack(_rec(4, 8), out=torch.zeros(4, 9)),
    lambda: qw.block_gemm(_rec(4, 8), _rec(3, 8, 128)),                  # x with 128-row blocks
    lambda: qw.block_gemm(_rec(4, 8), _rec(3, 9, 1)),
    lambda: qw.block_gemm(_rec(4, 8, e=2), _rec(3, 8, 1)),
    lambda: qw.block_gemm(_rec(4, 8), _rec(3, 8, 1), out_dtype=torch.float16),
    lambda: qw.block_gemm(_rec(4, 8), _rec(3, 8, 1)),                    # host tensors
    lambda: qw.block_matmul(_rec(4, 8), torch.zeros(3, 9)),
    lambda: qw.block_matmul(_rec(4, 8), torch.zeros(3, 8, dtype=torch.int8)),
    lambda: qw.block_matmul(_rec(4, 8), torch.zeros(3, 8), out=torch.zeros(3, 5)),
    lambda: qw.block_matmul(_rec(4, 8), torch.zeros(3, 16)[:, ::2]),
    lambda: qw.block_gemm_grouped(_rec(4, 8, e=2), _rec(3, 8, 1), torch.zeros(2, dtype=torch.int32)),
    lambda: qw.block_gemm_grouped(_rec(4, 8), _rec(3, 8, 1), torch.zeros(3, dtype=torch.int32)),
    lambda: qw.moe_sort(torch.zeros(4, 2), 8),
    lambda: qw.moe_sort(torch.zeros(4, 2, dtype=torch.int64).t(), 8),
    lambda: qw.moe_gather(torch.zeros(4, 8), dict(pos=torch.zeros(5, 2, dtype=torch.int32))),
    lambda: qw.moe_gather(torch.zeros(4, 8), dict(pos=torch.zeros(4, 2, dtype=torch.int64))),
    lambda: qw.moe_gather(torch.zeros(4, 8), dict(pos=torch.zeros(4, 2, dtype=torch.int32)), out=torch.zeros(8, 9)),
    lambda: qw.moe_gather_block(torch.zeros(4, 8), dict(pos=torch.zeros(4, 2, dtype=torch.int32)), rows=-1),
    lambda: qw.moe_combine(torch.zeros(8, 8), dict(pos=torch.zeros(4, 2, dtype=torch.int32)), torch.zeros(4, 3)),
    lambda: qw.moe_combine(torch.zeros(8, 8), dict(pos=torch.zeros(4, 2, dtype=torch.int32)),
                           torch.zeros(4, 2, dtype=torch.bfloat16)),
    lambda: qw.moe_combine_backward(torch.zeros(4, 9), torch.zeros(8, 8), dict(pos=torch.zeros(4, 2, dtype=torch.int32))),
    lambda: qw.moe_combine_backward(torch.zeros(4, 8).bfloat16(), torch.zeros(8, 8),
                                    dict(pos=torch.zeros(4, 2, dtype=torch.int32))),
    lambda: qw.moe_mlp(_rec(8, 8, e=2), _rec(8, 5, e=2), torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64)),
    lambda: qw.moe_mlp(_rec(8, 8, e=2), _rec(8, 4, 1, e=2), torch.zeros(4, 8), torch.zeros(4, 2, dtype=torch.int64)),
    lambda: qw.moe_mlp(_rec(8, 8, e=2), _rec(8, 4, e=2), torch.zeros(5, 8), torch.zeros(4, 2, dtype=torch.int64)),
])
def test_binding_refuses_before_any_call(call):
    with pytest.raises(ValueError):
        call()
