"""Attention of 17 to 64 query rows per sequence and key head (the kernel whose
warps have rows of their own and share one ring of keys and values) against the
plain 64-bit form."""
import numpy as np
import pytest
import torch

import ref8
from gpu_cases import dev
from sparse_weight_b200 import hyb
from test_gpu_cache import behind_a_page, check_attention, dev32, host_cache, queries, setup

pytestmark = pytest.mark.gpu

# lens (with the new tokens), new tokens, query heads, kv heads, dim, page, type; rows = most new x heads / kv heads
MID = [
    ([300, 40, 0], [5, 5, 5], 16, 2, 128, 16, "e4m3"),          # 40 rows, an empty slot
    ([1500], [16], 4, 1, 128, 64, "i8"),                        # 64 rows, split
    ([33, 17, 16, 1], [17, 17, 0, 1], 1, 1, 64, 16, "i8"),      # 17 rows; sequences of 1 and no row
    ([2100, 3, 64], [7, 3, 1], 9, 1, 64, 64, "e4m3"),           # 63 rows; 27 and 9: warps without a row
    ([64, 128, 129, 65], [12, 12, 12, 12], 10, 2, 128, 32, "e4m3"),
    ([5000, 700], [4, 4], 32, 2, 128, 16, "i8"),                # 64 rows, split unevenly
    ([31, 32, 33, 63, 64, 65, 0, 20], [20] * 6 + [20, 20], 6, 2, 64, 32, "e4m3"),
    ([1000, 50], [33, 2], 2, 2, 128, 64, "e4m3"),
]



@pytest.mark.parametrize("order", ["pht", "pth"])
@pytest.mark.parametrize("i", range(len(MID)))
def test_rows_17_to_64(i, order):
    lens, new, heads, kvh, dim, size, type_ = MID[i]
    assert 17 <= max(new) * heads // kvh <= 64
    C, table, off = setup(lens, new, kvh, dim, size, type_, order, seed=i)
    rows = int(off[-1])
    q = queries(rows, heads, dim, i)
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, len(lens), heads, max(new), table.shape[1] * size), dev())
    out = torch.full((rows + 2, heads, dim), 3.0, dtype=torch.bfloat16, device=dev())
    qd = torch.cat([q, torch.full((2, heads, dim), float("nan"), dtype=torch.bfloat16)]).to(dev())
    o, lse = hyb.cache_attention(C, qd, dev32(table), dev32(lens), off=dev32(off), max_new=max(new), out=out,
                                 return_lse=True, ws=ws)
    assert hyb.check_status(ws) == 0 and (o[rows:] == 3).all()
    check_attention(C, table, lens, off, q, o[:rows], lse[:rows])
    if len(set(new)) == 1:
        o2, lse2 = hyb.cache_attention(C, qd[:rows], dev32(table), dev32(lens), max_new=max(new), return_lse=True, ws=ws)
        assert torch.equal(o2, o[:rows]) and torch.equal(lse2, lse[:rows])


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (31, 0), (33, 40), (100, 20), (5000, 3), (64, 5000)])
@pytest.mark.parametrize("i", range(len(MID)))
def test_window(i, window, sinks):
    lens, new, heads, kvh, dim, size, type_ = MID[i]
    C, table, off = setup(lens, new, kvh, dim, size, type_, seed=i)
    q = queries(int(off[-1]), heads, dim, i)
    kw = dict(window=window, sinks=sinks)
    # pages that no query sees are given back
    given = table.copy()
    for b, t in enumerate(lens):
        for j in range(given.shape[1]):
            if j * size >= sinks and (j + 1) * size <= t - new[b] - window + 1:
                given[b, j] = -1
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, len(lens), heads, max(new), table.shape[1] * size), dev())
    o, lse = hyb.cache_attention(C, q.to(dev()), dev32(given), dev32(lens), off=dev32(off), max_new=max(new),
                                 return_lse=True, ws=ws, **kw)
    assert hyb.check_status(ws) == 0
    check_attention(C, table, lens, off, q, o, lse, **kw)


@pytest.mark.parametrize("scales", [(0.0, 0.0), (float("nan"), float("nan")), (float("inf"), float("inf"))])
@pytest.mark.parametrize("i", [0, 1, 3, 6])
def test_pages_of_no_sequence(i, scales):
    lens, new, heads, kvh, dim, size, type_ = MID[i]
    C, table, off = setup(lens, new, kvh, dim, size, type_, seed=i)
    q = queries(int(off[-1]), heads, dim, i)
    for kw in ({}, dict(window=21, sinks=3)):
        o, lse = hyb.cache_attention(behind_a_page(C, *scales), q.to(dev()), dev32(table + 1), dev32(lens),
                                     off=dev32(off), max_new=max(new), return_lse=True, **kw)
        check_attention(C, table, lens, off, q, o, lse, **kw)


@pytest.mark.parametrize("i", [0, 1, 3, 5])
def test_zero_scales(i):
    lens, new, heads, kvh, dim, size, type_ = MID[i]
    C, table, off = setup(lens, new, kvh, dim, size, type_, seed=i, poison=False)
    q = queries(int(off[-1]), heads, dim, i)
    g = torch.Generator().manual_seed(i)
    for x in (C.k_scale, C.v_scale):
        x.copy_(torch.where(torch.rand(x.shape, generator=g) < 0.3, 0.0, x.cpu()))
    o, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32(lens), off=dev32(off), max_new=max(new), return_lse=True)
    O, L, bO, bl = ref8.attention(host_cache(C), q.double().numpy(), table, lens, off, dim ** -0.5)
    # scales below 2^-64 count as 2^-64: values of at most 448 * 2^-64
    assert (np.abs(o.double().cpu().numpy() - O) <= bO + 448 * 2.0 ** -64 * (1 + 2.0 ** -8)).all()
    z, f = lse.double().cpu().numpy(), ~np.isinf(L)
    assert np.array_equal(np.isinf(z), ~f) and (np.abs(z[f] - L[f]) <= bl[f]).all()


@pytest.mark.parametrize("type_", ["e4m3", "i8"])
@pytest.mark.parametrize("dim", [64, 128])
def test_growing_scores(dim, type_):
    """Scores that grow by many binades along the tokens: what was summed against an earlier maximum is rescaled."""
    T, new = 700, 12
    C, table, off = setup([T], [new], 1, dim, 32, type_, seed=3, poison=False)
    g = torch.Generator().manual_seed(2)
    u = torch.sign(torch.randn(dim, generator=g))
    q = (queries(new, 4, dim, 1).abs() * u).to(torch.bfloat16)
    for page in range(-(-T // 32)):
        i = int(table[0, page])
        ramp = (page + torch.arange(32) / 32.0) % 5 / 5 * (127 if type_ == "i8" else 256)
        C.k[i, 0].copy_((ramp[:, None] * u).to(dev()).to(C.k.dtype))
        C.k_scale[i, 0] = 2.0 ** (-9 + page % 3)
    o, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32([T]), return_lse=True)
    check_attention(C, table, [T], off, q, o, lse)


def test_nan_query_spoils_its_own_row_only():
    lens, new = [90, 33], [6, 6]
    C, table, off = setup(lens, new, 2, 128, 32, "i8", seed=3)
    q = queries(12, 8, 128, 2)
    args = (dev32(table), dev32(lens))
    plain = hyb.cache_attention(C, q.to(dev()), *args)
    q[7, 5, 100] = float("nan")
    o = hyb.cache_attention(C, q.to(dev()), *args)
    assert o[7, 5].isnan().all()
    o[7, 5] = plain[7, 5]
    assert torch.equal(o, plain)
