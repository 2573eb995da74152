"""hyb_cache_append and hyb_cache_attention against their plain 64-bit forms."""
import numpy as np
import pytest
import torch

import ref8
from gpu_cases import dev
from sparse_weight_b200 import hyb

pytestmark = pytest.mark.gpu
TYPES = {"e4m3": torch.float8_e4m3fn, "i8": torch.int8}


def host(t):
    """Stored 8-bit values as float64."""
    if t.dtype == torch.int8:
        return t.cpu().numpy().astype(np.float64)
    return ref8.e4m3_decode(t.view(torch.uint8).cpu().numpy())


def host_cache(C):
    return dict(k=host(C.k), v=host(C.v), k_scale=C.k_scale.cpu().numpy().copy(),
                v_scale=C.v_scale.cpu().numpy().copy())


def layout(pages, heads, size, dim, dtype, order, device):
    """A cache of zeros, [page][head][token] or [page][token][head] in memory."""
    shape = {"pht": (pages, heads, size, dim), "pth": (pages, size, heads, dim)}[order]
    kv = [torch.zeros(shape, dtype=torch.uint8, device=device).view(dtype) for _ in range(2)]
    if order == "pth":
        kv = [x.transpose(1, 2) for x in kv]
    return hyb.Cache(kv[0], kv[1], torch.zeros(pages, heads, device=device), torch.zeros(pages, heads, device=device))


def setup(lens, new, heads, dim, size, type_, order="pht", seed=0, poison=True):
    """A filled cache, scattered pages; places behind every sequence and pages of none hold NaN bytes (e4m3)."""
    rng = np.random.default_rng(seed)
    need = [-(-t // size) for t in lens]
    pages, width = sum(need) + 2, max(1, max(need)) + 1
    perm = rng.permutation(pages)
    table = np.zeros((len(lens), width), np.int32)
    at = 0
    for b, c in enumerate(need):
        table[b, :c] = perm[at:at + c]
        table[b, c:] = 10 ** 6  # never looked at
        at += c
    C = layout(pages, heads, size, dim, TYPES[type_], order, dev())
    raw = rng.standard_normal((2, pages, heads, size, dim))
    sc = np.exp2(rng.integers(-9, -3, (2, pages, heads))).astype(np.float32)
    top = 127 if type_ == "i8" else 448
    for x, r, s, sd in ((C.k, raw[0], C.k_scale, sc[0]), (C.v, raw[1], C.v_scale, sc[1])):
        y = np.clip(r / np.abs(r).max(axis=(2, 3), keepdims=True) * top, -top, top)
        x.copy_(torch.from_numpy(np.rint(y) if type_ == "i8" else y).to(dev()).to(TYPES[type_]))
        s.copy_(torch.from_numpy(sd))
    if poison:
        bad = 0x7F if type_ == "e4m3" else 0x80
        live = np.zeros((pages, size), bool)
        for b, t in enumerate(lens):
            for j in range(t):
                live[table[b, j // size], j % size] = True
        dead = torch.from_numpy(~live).to(dev())
        for x in (C.k, C.v):
            u = x.view(torch.uint8)
            u.copy_(torch.where(dead[:, None, :, None], torch.tensor(bad, dtype=torch.uint8, device=dev()), u))
    off = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
    return C, table, off


def dev32(x):
    return torch.from_numpy(np.asarray(x, np.int32)).to(dev())


def queries(rows, heads, dim, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(rows, heads, dim, generator=g) * 1.5).to(torch.bfloat16)


def check_attention(C, table, lens, off, q, got, lse, **kw):
    O, L, bO, bl = ref8.attention(host_cache(C), q.double().numpy(), table, lens, off,
                                  kw.pop("scale", q.shape[2] ** -0.5), **kw)
    e = np.abs(got.double().cpu().numpy() - O)
    assert (e <= bO + 1e-30).all(), ("O", float((e / (bO + 1e-30)).max()))
    z = lse.double().cpu().numpy()
    assert np.array_equal(np.isinf(z), np.isinf(L)) and not np.isnan(z).any()
    f = ~np.isinf(L)
    assert (np.abs(z - np.where(f, L, 0))[f] <= bl[f]).all(), float((np.abs(z[f] - L[f]) / bl[f]).max())


# lens (with the new tokens), new tokens, query heads, kv heads, dim, page, type
ATT = [
    ([1], [1], 1, 1, 64, 16, "e4m3"),
    ([1], [1], 8, 2, 128, 64, "i8"),
    ([300], [1], 32, 8, 128, 16, "e4m3"),
    ([15, 16, 17, 31, 32, 33, 0, 64, 65], [1] * 9, 8, 2, 128, 16, "e4m3"),
    ([63, 64, 65, 127, 128, 129], [1] * 6, 10, 2, 64, 32, "i8"),
    ([2000, 3, 700], [1] * 3, 16, 2, 128, 64, "i8"),
    ([4500], [1], 4, 1, 64, 32, "e4m3"),
    ([100, 5, 0, 64], [5, 5, 5, 5], 12, 4, 128, 32, "e4m3"),
    ([40, 0, 129, 7], [7, 3, 1, 7], 8, 4, 64, 16, "i8"),
    ([90, 33], [33, 33], 3, 1, 128, 64, "e4m3"),
    ([200, 64, 1], [200, 17, 0], 16, 2, 128, 32, "e4m3"),
    ([257], [130], 40, 8, 64, 64, "i8"),
    ([700, 300], [70, 70], 4, 1, 128, 16, "i8"),
    ([600, 0, 90, 64], [100, 40, 90, 1], 6, 2, 64, 16, "e4m3"),
    ([1500], [20], 8, 1, 128, 32, "e4m3"),
    ([129, 65], [129, 65], 2, 1, 128, 64, "e4m3"),
]


@pytest.mark.parametrize("order", ["pht", "pth"])
@pytest.mark.parametrize("i", range(len(ATT)))
def test_attention(i, order):
    lens, new, heads, kvh, dim, size, type_ = ATT[i]
    C, table, off = setup(lens, new, kvh, dim, size, type_, order, seed=i)
    q = queries(int(off[-1]), heads, dim, i)
    uniform = len(set(new)) == 1
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, len(lens), heads, max(new), table.shape[1] * size),
                           dev())
    args = (C, q.to(dev()), dev32(table), dev32(lens))
    o, lse = hyb.cache_attention(*args, off=None if uniform else dev32(off), max_new=max(new), return_lse=True, ws=ws)
    assert hyb.check_status(ws) == 0
    check_attention(C, table, lens, off, q, o, lse)
    o2, lse2 = hyb.cache_attention(*args, off=dev32(off), max_new=max(new), return_lse=True, ws=ws)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (31, 0), (33, 40), (100, 20), (5000, 3), (64, 5000)])
@pytest.mark.parametrize("i", [2, 3, 5, 7, 8, 10, 11, 12, 13, 14])
def test_attention_window(i, window, sinks):
    lens, new, heads, kvh, dim, size, type_ = ATT[i]
    C, table, off = setup(lens, new, kvh, dim, size, type_, seed=i)
    if type_ == "e4m3" and max(new) == 1:
        # what the window hides must not count, whatever it holds
        for b, t in enumerate(lens):
            for j in range(min(sinks, t), max(0, t - window)):
                for x in (C.k, C.v):
                    x.view(torch.uint8)[table[b, j // size], :, j % size] = 0x7F
    q = queries(int(off[-1]), heads, dim, i)
    o, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32(lens), off=dev32(off), max_new=max(new),
                                 window=window, sinks=sinks, return_lse=True)
    check_attention(C, table, lens, off, q, o, lse, window=window, sinks=sinks)


def test_attention_long():
    """Many steps per warp, splits and their merge, one sequence and a ragged batch."""
    for lens, heads, kvh, type_, size, kw in (
            ([9000], 8, 1, "e4m3", 64, {}),
            ([9000, 20, 3000], 4, 1, "i8", 16, {}),
            ([9000, 5000], 4, 1, "e4m3", 32, dict(window=3000, sinks=70))):
        C, table, off = setup(lens, [2] * len(lens), kvh, 128, size, type_, seed=len(lens))
        q = queries(int(off[-1]), heads, 128, 3)
        o, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32(lens), return_lse=True, **kw)
        check_attention(C, table, lens, off, q, o, lse, **kw)


def test_attention_many_units():
    """More units than are split: no partial results."""
    lens = [37 + 3 * i for i in range(40)]
    C, table, off = setup(lens, [30] * 40, 8, 64, 16, "e4m3", seed=4)
    q = queries(int(off[-1]), 64, 64, 4)
    o, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32(lens), return_lse=True)
    part = [0, 19, 39]
    rows = np.concatenate([np.arange(off[b], off[b + 1]) for b in part])
    sub = np.concatenate([[0], np.cumsum([30] * 3)])
    check_attention(C, table[part], [lens[b] for b in part], sub, q[rows], o[rows], lse[rows])


@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0])
def test_attention_scales(scale):
    """Other softmax scales, and pages whose value scales lie far apart."""
    C, table, off = setup([200, 77], [3, 3], 2, 128, 16, "e4m3", seed=9)
    g = torch.Generator().manual_seed(1)
    C.v_scale.copy_(torch.exp2(torch.randint(-40, 10, C.v_scale.shape, generator=g).float()))
    q = queries(6, 4, 128, 5)
    q[0] *= 1e-12
    q[1] *= 100
    q[2] = 0
    o, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32([200, 77]), scale=scale, return_lse=True)
    check_attention(C, table, [200, 77], off, q, o, lse, scale=scale)


def test_attention_rows_strides_and_nan_query():
    """Strided Q and O; rows of no sequence stay; a NaN query spoils its own row only."""
    lens, new = [50, 20, 9], [4, 0, 3]
    C, table, off = setup(lens, new, 2, 128, 32, "i8", seed=3)
    q = queries(10, 8, 128, 2)
    buf = torch.zeros(10, 10, 160, dtype=torch.bfloat16, device=dev())
    buf[:, 1:9, 16:144] = q.to(dev())
    out = torch.full((10, 9, 136), 3.0, dtype=torch.bfloat16, device=dev())
    hyb.cache_attention(C, buf[:, 1:9, 16:144], dev32(table), dev32(lens), off=dev32(off), max_new=4,
                        out=out[:, :8, :128])
    plain, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32(lens), off=dev32(off), max_new=4,
                                     return_lse=True)
    assert torch.equal(out[:7, :8, :128], plain[:7])
    assert (out[7:] == 3).all() and (out[:, 8:] == 3).all() and (out[:, :, 128:] == 3).all()
    check_attention(C, table, lens, off, q[:7], plain[:7], lse[:7])
    bad = q.clone()
    bad[2, 5, 7] = float("nan")
    o = hyb.cache_attention(C, bad.to(dev()), dev32(table), dev32(lens), off=dev32(off), max_new=4)
    assert o[2, 5].isnan().all()
    o[2, 5] = plain[2, 5]
    assert torch.equal(o[:7], plain[:7])


def test_attention_shared_pages_graph_stream_workspace():
    """Two sequences on the same pages; captured and replayed; side stream; shapes sharing one workspace."""
    lens = [700, 700, 40]
    C, table, off = setup(lens, [1] * 3, 2, 128, 32, "e4m3", seed=6)
    table[1] = table[0]
    q = queries(3, 8, 128, 1).to(dev())
    q2 = queries(60, 8, 128, 2).to(dev())
    q[1] = q[0]
    a = (dev32(table), dev32(lens))
    n = max(hyb.cache_attention_workspace_bytes(C, 3, 8, m, table.shape[1] * 32) for m in (1, 20))
    ws = hyb.new_workspace(n, dev())
    o = hyb.cache_attention(C, q, *a)
    assert torch.equal(o[0], o[1])
    p = hyb.cache_attention(C, q2, *a)
    for _ in range(3):
        assert torch.equal(hyb.cache_attention(C, q, *a, ws=ws), o)
        assert torch.equal(hyb.cache_attention(C, q2, *a, ws=ws), p)
        assert torch.equal(hyb.cache_attention(C, q, *a, ws=ws, window=100, sinks=2),
                           hyb.cache_attention(C, q, *a, window=100, sinks=2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s = hyb.cache_attention(C, q, *a, stream=side)
    side.synchronize()
    assert torch.equal(s, o)
    gq, go = torch.zeros_like(q), torch.empty_like(o)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hyb.cache_attention(C, gq, *a, out=go, ws=ws)
    gq.copy_(q)
    for _ in range(2):
        graph.replay()
        assert torch.equal(go, o)
    assert hyb.check_status(ws) == 0


# lens, new, kv heads, dim, page, type
APP = [
    ([1], [1], 1, 64, 16, "e4m3"),
    ([16, 17, 33, 0, 5], [1] * 5, 2, 128, 16, "e4m3"),
    ([16, 17, 33, 0, 5], [1] * 5, 2, 64, 32, "i8"),
    ([64, 65, 130], [64, 1, 70], 3, 128, 64, "i8"),
    ([100, 37, 9, 20], [100, 30, 0, 5], 2, 64, 32, "e4m3"),
    ([20, 90], [7, 81], 4, 128, 16, "i8"),
]


@pytest.mark.parametrize("big", [1.0, 60.0, 1e-3])
@pytest.mark.parametrize("order", ["pht", "pth"])
@pytest.mark.parametrize("i", range(len(APP)))
def test_append(i, order, big):
    """Bit-exact values and scales; everything else in the cache untouched; a second identical call changes nothing."""
    lens, new, heads, dim, size, type_ = APP[i]
    C, table, off = setup(lens, new, heads, dim, size, type_, order, seed=i, poison=False)
    rows = int(off[-1])
    g = torch.Generator().manual_seed(i)
    kv = (torch.randn(rows + 2, 2 * heads, dim, generator=g) * big).to(torch.bfloat16)
    d = kv.to(dev())
    uniform = len(set(new)) == 1
    ref = host_cache(C)
    ref8.append(ref, dict(k=kv[:rows, :heads].double().numpy(), v=kv[:rows, heads:].double().numpy()),
                table, lens, off, type_ == "i8")
    ws = hyb.new_workspace(256, dev())
    n = rows if uniform else rows + 2  # rows of no sequence are ignored
    for _ in range(2):
        hyb.cache_append(C, d[:n, :heads], d[:n, heads:], dev32(table), dev32(lens),
                         off=None if uniform else dev32(off), max_new=max(new), ws=ws)
        assert hyb.check_status(ws) == 0
        got = host_cache(C)
        for w in ref:
            assert np.array_equal(got[w], ref[w]), w


@pytest.mark.parametrize("type_", ["e4m3", "i8"])
def test_append_token_by_token(type_):
    """Values that grow and shrink along a page: the scale only grows, a page's first token resets it."""
    size, heads, dim, T = 16, 2, 64, 40
    C, table, _ = setup([T], [1], heads, dim, size, type_, seed=2, poison=False)
    ref = host_cache(C)
    g = torch.Generator().manual_seed(3)
    for t in range(1, T + 1):
        x = (torch.randn(1, 2 * heads, dim, generator=g) * float(2.0 ** ((t * 7) % 11 - 5))).to(torch.bfloat16)
        if t == 20:
            x.zero_()
        d = x.to(dev())
        hyb.cache_append(C, d[:, :heads], d[:, heads:], dev32(table), dev32([t]))
        ref8.append(ref, dict(k=x[:, :heads].double().numpy(), v=x[:, heads:].double().numpy()), table, [t], [0, 1],
                    type_ == "i8")
    got = host_cache(C)
    for w in ref:
        assert np.array_equal(got[w], ref[w]), w


@pytest.mark.parametrize("type_", ["e4m3", "i8"])
def test_append_nan_inf_extremes(type_):
    C, table, off = setup([40], [40], 1, 64, 16, type_, seed=2, poison=False)
    x = queries(40, 2, 64, 4)
    x[3, 0, 5], x[4, 1, 6], x[5, 0, 7] = float("nan"), float("inf"), -float("inf")
    x[16:32] = 0
    x[33] *= 1e37
    ref = host_cache(C)
    ref8.append(ref, dict(k=x[:, :1].double().numpy(), v=x[:, 1:].double().numpy()), table, [40], off, type_ == "i8")
    ws = hyb.new_workspace(256, dev())
    hyb.cache_append(C, x[:, :1].to(dev()), x[:, 1:].to(dev()), dev32(table), dev32([40]), ws=ws)
    with pytest.raises(hyb.HybError) as ei:
        hyb.check_status(ws)
    assert ei.value.flags == hyb.STATUS_NAN
    got = host_cache(C)
    for w in ref:
        assert np.array_equal(got[w], ref[w]), w


def _flags(ws):
    with pytest.raises(hyb.HybError) as ei:
        hyb.check_status(ws)
    return ei.value.flags


BAD = [
    dict(lens=[40, 33]),             # beyond the table (2 pages of 16)
    dict(lens=[-1, 20]),
    dict(lens=[2, 20]),              # fewer tokens than new ones
    dict(off=[0, 5, 3]),             # decreasing
    dict(off=[0, 3, 7]),             # beyond the rows
    dict(off=[-1, 3, 6]),
    dict(off=[0, 5, 6]),             # more than max_new
    dict(table=[[0, 99], [2, 3]]),
    dict(table=[[0, -1], [2, 3]]),
]


@pytest.mark.parametrize("i", range(len(BAD)))
def test_bad_sequences_are_flagged(i):
    """Contradictory device data: reported, the other sequence served, nothing outside touched."""
    good = dict(lens=[20, 20], off=[0, 3, 6], table=[[0, 1], [2, 3]])
    bad = {**good, **BAD[i]}
    C, _, _ = setup([64], [1], 2, 64, 16, "i8", poison=False)  # 6 pages
    q = queries(6, 4, 64, 1)
    kv = queries(6, 2, 64, 2)
    args = lambda d: (dev32(d["table"]), dev32(d["lens"]))  # noqa: E731
    before = [x.clone() for x in (C.k, C.v, C.k_scale, C.v_scale)]
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, 2, 4, 3, 32), dev())
    out = torch.full((6, 4, 64), 3.0, dtype=torch.bfloat16, device=dev())
    hyb.cache_attention(C, q.to(dev()), *args(bad), off=dev32(bad["off"]), max_new=3, out=out, ws=ws)
    assert _flags(ws) == hyb.STATUS_BAD_SEQ
    assert all(torch.equal(x, y) for x, y in zip(before, (C.k, C.v, C.k_scale, C.v_scale)))
    # the workspace serves the next call
    o = hyb.cache_attention(C, q.to(dev()), *args(good), off=dev32(good["off"]), max_new=3, ws=ws)
    assert hyb.check_status(ws) == 0
    assert torch.equal(o, hyb.cache_attention(C, q.to(dev()), *args(good), off=dev32(good["off"]), max_new=3))
    hyb.cache_append(C, kv.to(dev()), kv.to(dev()), *args(bad), off=dev32(bad["off"]), max_new=3, ws=ws)
    assert _flags(ws) == hyb.STATUS_BAD_SEQ
    assert torch.equal(C.k[4:], before[0][4:]) and torch.equal(C.v_scale[4:], before[3][4:])


def behind_a_page(C, k_scale, v_scale):
    """The same cache behind one more page of zeros with these scales; page p becomes p + 1."""
    kv = [torch.cat([torch.zeros_like(x.view(torch.uint8)[:1]), x.view(torch.uint8)]).view(x.dtype) for x in (C.k, C.v)]
    sc = [torch.cat([torch.full_like(x[:1], s), x]) for x, s in ((C.k_scale, k_scale), (C.v_scale, v_scale))]
    return hyb.Cache(kv[0], kv[1], sc[0], sc[1])


@pytest.mark.parametrize("scales", [(0.0, 0.0), (float("nan"), float("nan")), (float("inf"), float("inf"))])
@pytest.mark.parametrize("i", range(len(ATT)))
def test_attention_pages_of_no_sequence(i, scales):
    """A page that no sequence holds (page 0 of a fresh cache, say) has no part in any result, whatever its scales."""
    lens, new, heads, kvh, dim, size, type_ = ATT[i]
    C, table, off = setup(lens, new, kvh, dim, size, type_, seed=i)
    q = queries(int(off[-1]), heads, dim, i)
    for kw in ({}, dict(window=21, sinks=3)):
        o, lse = hyb.cache_attention(behind_a_page(C, *scales), q.to(dev()), dev32(table + 1), dev32(lens),
                                     off=dev32(off), max_new=max(new), return_lse=True, **kw)
        check_attention(C, table, lens, off, q, o, lse, **kw)


@pytest.mark.parametrize("window,sinks", [(1, 0), (16, 4), (40, 17), (100, 0)])
@pytest.mark.parametrize("i", [2, 5, 6, 11, 12, 14])
def test_attention_pages_behind_the_window(i, window, sinks):
    """Table entries of pages that no query sees are not used: a program may give those pages back."""
    lens, new, heads, kvh, dim, size, type_ = ATT[i]
    C, table, off = setup(lens, new, kvh, dim, size, type_, seed=i)
    q = queries(int(off[-1]), heads, dim, i)
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, len(lens), heads, max(new), table.shape[1] * size), dev())
    kw = dict(window=window, sinks=sinks)
    given = table.copy()
    for b, t in enumerate(lens):
        lowest = t - new[b] - window + 1
        for j in range(given.shape[1]):
            if j * size >= sinks and (j + 1) * size <= lowest:
                given[b, j] = -1
    o, lse = hyb.cache_attention(C, q.to(dev()), dev32(given), dev32(lens), off=dev32(off), max_new=max(new),
                                 return_lse=True, ws=ws, **kw)
    assert hyb.check_status(ws) == 0
    check_attention(C, table, lens, off, q, o, lse, **kw)


@pytest.mark.parametrize("i", [2, 5, 9, 11, 12, 15])
def test_attention_zero_scales(i):
    """Pages whose scale is 0 (a page of zeros, as some quantisers write it) count with values of 0."""
    lens, new, heads, kvh, dim, size, type_ = ATT[i]
    C, table, off = setup(lens, new, kvh, dim, size, type_, seed=i, poison=False)
    q = queries(int(off[-1]), heads, dim, i)
    g = torch.Generator().manual_seed(i)
    for x in (C.k_scale, C.v_scale):
        x.copy_(torch.where(torch.rand(x.shape, generator=g) < 0.3, 0.0, x.cpu()))
    o, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32(lens), off=dev32(off), max_new=max(new), return_lse=True)
    # scales below 2^-64 count as 2^-64: values of at most 448 * 2^-64
    O, L, bO, bl = ref8.attention(host_cache(C), q.double().numpy(), table, lens, off, dim ** -0.5)
    assert (np.abs(o.double().cpu().numpy() - O) <= bO + 448 * 2.0 ** -64 * (1 + 2.0 ** -8)).all()
    assert (np.abs(lse.double().cpu().numpy() - L) <= bl).all()


def test_attention_workspace_of_the_largest_step():
    """A workspace sized for the largest step serves smaller ones, with the results of one of their own."""
    rng = np.random.default_rng(5)
    for kvh, group, size in ((2, 4, 16), (8, 1, 32), (1, 20, 64)):
        C = layout(3, kvh, size, 64, torch.int8, "pht", dev())
        need = lambda b, n, pg: hyb.cache_attention_workspace_bytes(C, b, kvh * group, n, pg * size)  # noqa: E731
        for _ in range(300):
            B, N, W = (int(x) for x in np.exp(rng.uniform(0, np.log([64, 200, 500]))))
            top = need(B, N, W)
            assert need(int(rng.integers(1, B + 1)), int(rng.integers(1, N + 1)), int(rng.integers(1, W + 1))) <= top
    lens, new = [200] * 11, [12] * 11
    C, table, off = setup(lens, new, 2, 64, 16, "e4m3", seed=1)
    q = queries(132, 8, 64, 1).to(dev())
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, 13, 8, 21, 22 * 16), dev())
    for n, rows in ((12, 132), (1, 11), (3, 33)):
        a = (C, q[:rows], dev32(table), dev32(lens))
        assert torch.equal(hyb.cache_attention(*a, ws=ws), hyb.cache_attention(*a))
    assert hyb.check_status(ws) == 0


@pytest.mark.parametrize("type_", ["e4m3", "i8"])
@pytest.mark.parametrize("dim", [64, 128])
def test_attention_growing_scores(dim, type_):
    """Scores that grow by many binades along the tokens, within a step and from step to step: what was summed
    against an earlier, smaller maximum is rescaled."""
    T, new = 700, 80
    C, table, off = setup([T], [new], 1, dim, 32, type_, seed=3, poison=False)
    g = torch.Generator().manual_seed(2)
    q = queries(new, 4, dim, 1)
    # all keys along one direction, longer and longer, in ramps of different steepness; queries share its sign
    u = torch.sign(torch.randn(dim, generator=g))
    q = (q.abs() * u).to(torch.bfloat16)
    for page in range(-(-T // 32)):
        i = int(table[0, page])
        ramp = (page + torch.arange(32) / 32.0) % 5 / 5 * (127 if type_ == "i8" else 256)
        C.k[i, 0].copy_((ramp[:, None] * u).to(dev()).to(TYPES[type_]))
        C.k_scale[i, 0] = 2.0 ** (-9 + page % 3)
    o, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32([T]), return_lse=True)
    check_attention(C, table, [T], off, q, o, lse)


def test_both_bindings_agree():
    """The C++ binding and the Python code (which a given stream takes) make the same calls, errors among them."""
    from sparse_weight_b200.hyb import _load_native
    nat = _load_native()
    here = torch.cuda.current_stream()
    lens, new = [90, 33, 0], [4, 2, 1]
    C, table, off = setup(lens, new, 2, 64, 16, "i8", seed=1, poison=False)
    D, _, _ = setup(lens, new, 2, 64, 16, "i8", seed=1, poison=False)
    q, t, n, o = queries(7, 8, 64, 1).to(dev()), dev32(table), dev32(lens), dev32(off)
    kv = queries(7, 4, 64, 2).to(dev())
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, 3, 8, 4, table.shape[1] * 16), dev())
    for X, st in ((C, None), (D, here)):
        hyb.cache_append(X, kv[:, :2], kv[:, 2:], t, n, o, 4, ws=ws, stream=st)
    for w in ("k", "v", "k_scale", "v_scale"):
        assert torch.equal(getattr(C, w), getattr(D, w)), w
    for kw in ({}, dict(window=9, sinks=2), dict(scale=0.3), dict(return_lse=True)):
        for a in ((C, q, t, n, o, 4), (C, q[:3], t, n), (C, q[:1], t[:1], n[:1]), (C, q[:, ::2], t, n, o, 4)):
            u, v = hyb.cache_attention(*a, ws=ws, **kw), hyb.cache_attention(*a, ws=ws, stream=here, **kw)
            u, v = (u, v) if kw.get("return_lse") else ((u,), (v,))
            for x, y in zip(u, v):
                assert x.shape == y.shape and x.stride() == y.stride() and torch.equal(x, y)
    out = torch.zeros(7, 9, 72, dtype=torch.bfloat16, device=dev())[:, :8, :64]
    assert hyb.cache_attention(C, q, t, n, o, 4, out=out, ws=ws) is out
    assert torch.equal(out, hyb.cache_attention(C, q, t, n, o, 4))
    at = (C._at, C._index)
    for args in ((*at, q.float(), t, n, o, 4), (*at, q, t.long(), n, o, 4), (*at, q, t, n[:2], o, 4), (*at, q, t, n, o, None),
                 (*at, q, t[:1].expand(3, table.shape[1]), n, o, 4), (*at, q, t, n, None, 4), (*at, q.cpu(), t, n, o, 4),
                 (*at, q[:, :, :32], t, n, o, 4), (C._at, -1, q, t, n, o, 4)):
        assert nat.cache_attention(*args, None, 0, 0, None, False, ws) is None
    assert nat.cache_attention(*at, q, t, n, o, 4, None, 0, 0, out[:, :7], False, ws) is None
    assert nat.cache_append(*at, kv[:, :2], kv[:6, 2:], t, n, o, 4, ws) is None
    assert nat.cache_append(*at, kv[:, :3], kv[:, :3], t, n, o, 4, ws) is None
    for st in (None, here):
        with pytest.raises(hyb.HybError) as ei:
            hyb.cache_attention(C, q[:, :7], t, n, o, 4, ws=ws, stream=st)
        assert ei.value.status == hyb.HYB_ERR_INVALID_ARG
        with pytest.raises(hyb.HybError) as ei:
            hyb.cache_append(C, kv[:, :2], kv[:, 2:], t, n, o, 4, ws=ws[:100], stream=st)
        assert ei.value.status == hyb.HYB_ERR_WORKSPACE
