"""The expert MLP's precision follows y's type."""

import numpy as np
import pytest
import torch

from int8_int4_dequant_amd import qw

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t,topk,experts,d,f", [(40, 2, 8, 256, 128), (130, 4, 6, 300, 200), (300, 2, 3, 264, 136), (333, 3, 5, 128, 384), (900, 2, 6, 700, 256)])
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
