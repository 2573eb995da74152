"""Attention repeats itself bit for bit, whatever order its warps and copies
come in: every unit shape (8, 16, 64 and 256 query rows), split and whole."""
import pytest
import torch

from gpu_cases import dev
from sparse_weight_b200 import hyb
from test_gpu_cache import check_attention, dev32, queries, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim,type_", [(64, "i8"), (128, "e4m3")])
@pytest.mark.parametrize("lens,new,heads,kvh,kw", [
    ([2500, 31, 1200], 1, 12, 2, {}), ([2500, 900], 2, 16, 2, dict(window=700, sinks=5)),
    ([2100, 60, 1300], 5, 20, 2, {}), ([2100, 200], 8, 14, 2, dict(window=300, sinks=40)),
    ([900, 128], 90, 4, 2, {})])
def test_repeats(lens, new, heads, kvh, kw, dim, type_):
    C, table, off = setup(lens, [new] * len(lens), kvh, dim, 32, type_, seed=new)
    q = queries(int(off[-1]), heads, dim, 5)
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, len(lens), heads, new, table.shape[1] * 32), dev())
    args = (C, q.to(dev()), dev32(table), dev32(lens))
    o, lse = hyb.cache_attention(*args, return_lse=True, ws=ws, **kw)
    check_attention(C, table, lens, off, q, o, lse, **kw)
    noise = torch.randn(4096, 4096, device=dev())
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(20):  # (other work beside it: warps and copies come in another order)
            noise = noise * 1.0001
    for _ in range(40):
        o2, lse2 = hyb.cache_attention(*args, return_lse=True, ws=ws, **kw)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)
    side.synchronize()
    assert hyb.check_status(ws) == 0
