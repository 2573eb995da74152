"""Attention whose page table is much wider than its sequences are long (a table of
fixed width, as a captured step has), and of more units than are ever split."""
import numpy as np
import pytest
import torch

from gpu_cases import dev
from sparse_weight_b200 import hyb
from test_gpu_cache import check_attention, dev32, queries, setup

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("lens,new,heads,kvh,dim,size,type_", [
    ([700], 1, 8, 2, 128, 64, "e4m3"), ([700, 31, 0], 3, 8, 2, 64, 16, "i8"), ([900, 64], 4, 16, 2, 128, 32, "e4m3"),
    ([900, 128], 40, 4, 2, 128, 64, "i8"), ([1], 1, 1, 1, 64, 16, "e4m3")])
def test_wide_table(lens, new, heads, kvh, dim, size, type_):
    C, table, off = setup(lens, [new] * len(lens), kvh, dim, size, type_, seed=new)
    wide = np.full((len(lens), 131072 // size), -1, np.int32)  # entries behind a sequence are not used
    wide[:, :table.shape[1]] = table
    for b, t in enumerate(lens):
        wide[b, -(-t // size):] = -1 - b
    q = queries(int(off[-1]), heads, dim, new)
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, len(lens), heads, new, 131072), dev())
    for kw in ({}, dict(window=100, sinks=3)):
        o, lse = hyb.cache_attention(C, q.to(dev()), dev32(wide), dev32(lens), return_lse=True, ws=ws, **kw)
        assert hyb.check_status(ws) == 0
        check_attention(C, table, lens, off, q, o, lse, **kw)
        # a view of the same table that is just wide enough
        cut = dev32(wide)[:, :table.shape[1]]
        o2, lse2 = hyb.cache_attention(C, q.to(dev()), cut, dev32(lens), return_lse=True, ws=ws, **kw)
        assert hyb.check_status(ws) == 0
        check_attention(C, table, lens, off, q, o2, lse2, **kw)


@pytest.mark.parametrize("batch", [147, 148, 300])
def test_batches_around_the_last_split_one(batch):
    """8 key heads x 148 sequences: from there on units stay whole."""
    lens = [17 + 5 * (b % 23) for b in range(batch)]
    lens[3], lens[70] = 2500, 0
    C, table, off = setup(lens, [1] * batch, 8, 64, 16, "i8", seed=batch)
    q = queries(batch, 16, 64, batch)
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, batch, 16, 1, table.shape[1] * 16), dev())
    o, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32(lens), return_lse=True, ws=ws)
    assert hyb.check_status(ws) == 0
    part = [0, 3, 70, 71, batch - 1]
    check_attention(C, table[part], [lens[b] for b in part], np.arange(len(part) + 1), q[part], o[part], lse[part])
