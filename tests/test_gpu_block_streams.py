"""Block-scaled calls on a stream given as a handle, or as the last positional argument."""

import pytest
import torch

from int8_int4_dequant_amd import qw

pytestmark = pytest.mark.gpu


def test_streams_by_handle_and_by_place():
    w, x = torch.randn(300, 500, device="cuda"), torch.randn(70, 500, device="cuda")
    want = qw.block_matmul(qw.block_quantize(w), x)
    ids = torch.randint(0, 4, (70, 2), device="cuda")
    order = qw.moe_sort(ids, 4)["order"]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for stream in (s, s.cuda_stream, 0):
        rec = qw.block_quantize(w, 128, stream)
        y = qw.block_matmul(rec, x, None, None, None, stream)
        r = qw.moe_sort(ids, 4, True, None, stream)
        z = qw.block_matmul(rec, x, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(y, want) and torch.equal(z, want) and torch.equal(r["order"], order)
