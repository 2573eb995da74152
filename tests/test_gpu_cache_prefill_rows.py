"""Prompt attention whose query rows end inside a warp: the lanes without a row
take part in the warp's reads of tensor memory and write nothing."""
import pytest
import torch

from gpu_cases import dev
from sparse_weight_b200 import hyb
from test_gpu_cache import check_attention, dev32, queries, setup

pytestmark = pytest.mark.gpu


# lens, new, query heads, kv heads, page, type: rows of a unit 67, 65 and 64 + 1, 256 + 137, 95, 129 and 127
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("lens,new,heads,kvh,size,type_", [
    ([400], [67], 1, 1, 16, "e4m3"), ([3000], [67], 1, 1, 64, "i8"), ([70, 66, 0], [65, 1, 0], 1, 1, 32, "i8"),
    ([300], [131], 3, 1, 64, "e4m3"), ([2500, 95], [95, 95], 2, 2, 32, "e4m3"), ([900, 130], [43, 127], 6, 2, 16, "i8")])
def test_rows_that_end_inside_a_warp(lens, new, heads, kvh, size, type_, dim):
    C, table, off = setup(lens, new, kvh, dim, size, type_, seed=dim)
    rows = int(off[-1])
    q = queries(rows, heads, dim, 7)
    out = torch.full((rows + 3, heads, dim), 3.0, dtype=torch.bfloat16, device=dev())
    qd = torch.cat([q, torch.full((3, heads, dim), float("nan"), dtype=torch.bfloat16)]).to(dev())
    o, lse = hyb.cache_attention(C, qd, dev32(table), dev32(lens), off=dev32(off), max_new=max(new), out=out,
                                 return_lse=True)
    assert (o[rows:] == 3).all()
    check_attention(C, table, lens, off, q, o[:rows], lse[:rows])
