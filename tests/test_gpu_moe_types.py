"""The expert MLP's precision follows y's type, and products take the type of `out`."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,topk,experts,d,f", [(1, 4, 8, 512, 384), (7, 2, 4, 130, 257), (2, 2, 3, 1300, 600), (3, 1, 1, 200, 9100),
                                                (40, 2, 8, 256, 128), (130, 4, 6, 300, 200), (300, 2, 3, 264, 136), (333, 3, 5, 128, 384), (900, 2, 6, 700, 256)])
@pytest.mark.parametrize("br", [1, 128])
def test_fp32_mlp_is_the_calls_one_by_one(t, topk, experts, d, f, br):
    """y in fp32: the products of the one call have fp32 sums, as the grouped
    product has for fp32 y; the same kernels, so the same bits."""
    print("mlp", t, topk, experts, d, f, br, flush=True)
    rng = np.random.default_rng([t, d, f])
    make = lambda *s: torch.from_numpy(rng.standard_normal(s, dtype=np.float32)).cuda()  # noqa: E731
    gate_up = qw.block_quantize(make(experts, 2 * f, d) * d ** -0.5, br)
    down = qw.block_quantize(make(experts, d, f) * f ** -0.5, br)
    x, w = make(t, d), torch.from_numpy(rng.random((t, topk), dtype=np.float32)).cuda()
    ids = torch.from_numpy(rng.integers(-1, experts, (t, topk))).cuda()
    y = qw.moe_mlp(gate_up, down, x, ids, w)
    r = qw.moe_sort(ids, experts)
    h = qw.block_gemm_grouped(gate_up, qw.moe_gather_block(x, r), r["offsets"])
    hr = qw.block_quantize_swiglu(h, r["offsets"][-1:])
    want = qw.moe_combine(qw.block_gemm_grouped(down, hr, r["offsets"]), r, w)
    assert y.dtype == torch.float32 and torch.equal(y, want)



def test_products_take_the_type_of_out():
    rec = qw.block_quantize(torch.randn(130, 300, device="cuda"), 128)
    x = qw.block_quantize(torch.randn(20, 300, device="cuda"), 1)
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.empty(20, 130, dtype=dtype, device="cuda")
        assert qw.block_gemm(rec, x, out=out) is out
        assert torch.equal(out, qw.block_gemm(rec, x, out_dtype=dtype))
        with pytest.raises(ValueError):
            qw.block_gemm(rec, x, out=out, out_dtype=torch.float32 if dtype is torch.bfloat16 else torch.bfloat16)
    assert qw.block_gemm(rec, x).dtype == torch.float32
    experts = qw.block_quantize(torch.randn(3, 130, 300, device="cuda"), 128)
    off = torch.tensor([0, 5, 5, 20], dtype=torch.int32, device="cuda")
    for dtype in (torch.float32, torch.bfloat16):
        out = torch.empty(20, 130, dtype=dtype, device="cuda")
        assert qw.block_gemm_grouped(experts, x, off, out=out) is out
        assert torch.equal(out, qw.block_gemm_grouped(experts, x, off, out_dtype=dtype))
    assert qw.block_gemm_grouped(experts, x, off).dtype == torch.float32
