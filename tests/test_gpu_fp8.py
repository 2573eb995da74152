"""hyb_fp8_quant and hyb_fp8_matmul against their plain 64-bit forms."""
import numpy as np
import pytest
import torch

import ref8
from gpu_cases import dev
from sparse_weight_b200 import hyb

pytestmark = pytest.mark.gpu


def values(rows, cols, seed, dtype=torch.bfloat16, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g) * std
    x *= torch.where(torch.rand(cols, generator=g) < 0.02, 20.0, 1.0)
    return x.to(dtype)


def decoded(q):
    return ref8.e4m3_decode(q.view(torch.uint8).cpu().numpy())


@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 128), (5, 130), (129, 257), (128, 1024), (300, 1000)])
def test_quant(shape, dtype, block_rows):
    x = values(*shape, seed=sum(shape), dtype=dtype)
    ld = -(-shape[1] // 8) * 8
    buf = torch.full((shape[0], ld), float("nan"), dtype=dtype, device=dev())  # not read behind the row
    buf[:, :shape[1]] = x.to(dev())
    ws = hyb.new_workspace(256, dev())
    q, s = hyb.quant_fp8(buf[:, :shape[1]], block_rows, ws=ws)
    assert hyb.check_status(ws) == 0
    rq, rs = ref8.quant(x.double().numpy(), block_rows)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(decoded(q), rq)
    # rows that do not start on 16 bytes
    odd = torch.zeros(shape[0], ld + 3, dtype=dtype, device=dev())
    odd[:, 1:shape[1] + 1] = x.to(dev())
    q2, s2 = hyb.quant_fp8(odd[:, 1:shape[1] + 1], block_rows)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quant_extremes(block_rows):
    """Zeros, tiny and huge blocks, ties, NaN and infinities."""
    x = values(6, 128 * 6, 1, torch.float32)
    x[:, :128] = 0
    x[:, 128:256] *= 1e-30
    x[:, 256:384] = x[:, 256:384].sign() * 3e38
    x[1, 384:512] = torch.linspace(-448, 448, 128)
    x[0, 512], x[2, 513], x[3, 514] = float("nan"), float("inf"), -float("inf")
    x[4, 640:] = float("inf")
    ws = hyb.new_workspace(256, dev())
    q, s = hyb.quant_fp8(x.to(dev()), block_rows, ws=ws)
    with pytest.raises(hyb.HybError) as ei:
        hyb.check_status(ws)
    assert ei.value.flags == hyb.STATUS_NAN
    rq, rs = ref8.quant(x.double().numpy(), block_rows)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(decoded(q), rq, equal_nan=True)


def weight(n, k, seed):
    W = values(n, k, seed, std=0.02)
    A = hyb.pack_fp8(W.to(dev()))
    rq, rs = ref8.quant(W.double().numpy(), 128)
    assert np.array_equal(decoded(A.q), rq) and np.array_equal(A.scale.cpu().numpy(), rs)
    return A, rq, rs


def check(Y, x, wq, ws, k):
    xq, xs = ref8.quant(x.double().numpy(), 1)
    y, env = ref8.matmul(xq, xs, wq, ws)
    bound = ref8.matmul_bound(env, k) + 1e-30
    if Y.dtype == torch.bfloat16:
        bound = bound + 2.0 ** -8 * np.abs(y)
    err = np.abs(Y.double().cpu().numpy() - y)
    assert (err <= bound).all(), float((err / bound).max())


MNK = [(1, 1, 1), (1, 128, 128), (1, 17, 130), (2, 200, 1000), (7, 1024, 512), (8, 129, 4096), (9, 256, 384),
       (16, 1000, 1100), (17, 256, 256), (33, 384, 640), (64, 130, 2000), (65, 300, 129), (127, 128, 512),
       (130, 512, 1040), (257, 390, 700), (300, 128, 1), (1, 4096, 4096)]


@pytest.mark.parametrize("ydt", [hyb.HYB_F32, hyb.HYB_BF16])
@pytest.mark.parametrize("m,n,k", MNK)
def test_matmul(m, n, k, ydt):
    """bf16 X (quantised inside) and e4m3 X give the same bits, within the bound."""
    A, wq, ws = weight(n, k, m + n + k)
    x = values(m, -(-k // 8) * 8, 7 * m + k)
    xd = x.to(dev())
    xd[:, k:] = float("nan")  # what lies behind a row is not used
    xd, x = xd[:, :k], x[:, :k]
    w = hyb.new_workspace(hyb.fp8_workspace_bytes(m, n, k), dev())
    Y = hyb.matmul_fp8(A, xd, ydt=ydt, ws=w)
    assert hyb.check_status(w) == 0
    check(Y, x, wq, ws, k)
    q, s = hyb.quant_fp8(xd)
    assert torch.equal(hyb.matmul_fp8(A, q, xs=s, ydt=ydt, ws=w), Y)


@pytest.mark.parametrize("m", [1, 5, 16, 40, 200])
def test_matmul_strides_and_untouched(m):
    """Row strides of every operand; what lies outside Y, and behind the rows of X and W, stays or is not used."""
    n, k = 200, 300
    A, wq, ws = weight(n, k, 5)
    qbuf = torch.full((n, 352), 0x7F, dtype=torch.uint8, device=dev())
    qbuf[:, :k] = A.q.view(torch.uint8)
    sbuf = torch.full((2, 5), float("nan"), device=dev())
    sbuf[:, :3] = A.scale
    B = hyb.Fp8Matrix(n, k, qbuf.view(torch.float8_e4m3fn)[:, :k], sbuf[:, :3])
    x = values(m, k, 6)
    xbuf = torch.full((m + 1, 336), float("nan"), dtype=torch.bfloat16, device=dev())
    xbuf[:m, :k] = x.to(dev())
    Y = torch.full((m + 2, 256), 7.0, device=dev())
    hyb.matmul_fp8(B, xbuf[:m, :k], Y=Y[:m, :n])
    torch.cuda.synchronize()
    check(Y[:m, :n], x, wq, ws, k)
    assert (Y[m:] == 7).all() and (Y[:, n:] == 7).all()
    xq, xs = hyb.quant_fp8(xbuf[:m, :k])
    qx = torch.full((m, 400), 0x7F, dtype=torch.uint8, device=dev())
    qx[:, :k] = xq.view(torch.uint8)
    sx = torch.full((m, 9), float("nan"), device=dev())
    sx[:, :3] = xs
    Z = hyb.matmul_fp8(B, qx.view(torch.float8_e4m3fn)[:, :k], xs=sx[:, :3])
    assert torch.equal(Z, Y[:m, :n])


@pytest.mark.parametrize("m", [1, 16, 40, 300])
def test_matmul_nan_and_inf(m):
    """A NaN in a token makes that token's outputs NaN and no other's; an infinity saturates; both are flagged."""
    n, k = 256, 384
    A, wq, ws = weight(n, k, 8)
    x = values(m, k, 9)
    x[0, 200] = float("inf")
    if m > 1:
        x[m - 1, 3] = float("nan")
    w = hyb.new_workspace(hyb.fp8_workspace_bytes(m, n, k), dev())
    Y = hyb.matmul_fp8(A, x.to(dev()), ws=w)
    with pytest.raises(hyb.HybError) as ei:
        hyb.check_status(w)
    assert ei.value.flags == hyb.STATUS_NAN
    if m > 1:
        assert Y[m - 1].isnan().all()
        Y, x = Y[:m - 1], x[:m - 1]
    check(Y, x, wq, ws, k)


def test_matmul_streams_graphs_and_shared_workspace():
    """Captured, replayed with new inputs, on a side stream, shapes sharing one workspace: always the same bits."""
    A, _, _ = weight(512, 1024, 11)
    B, _, _ = weight(300, 520, 12)
    ms = (1, 12, 50, 260)
    ws = hyb.new_workspace(max(hyb.fp8_workspace_bytes(m, C.n, C.k) for m in ms for C in (A, B)), dev())
    for m in ms:
        xa, xb = values(m, 1024, m).to(dev()), values(m, 520, m + 1).to(dev())
        ya, yb = hyb.matmul_fp8(A, xa), hyb.matmul_fp8(B, xb)
        for _ in range(3):
            za, zb = hyb.matmul_fp8(A, xa, ws=ws), hyb.matmul_fp8(B, xb, ws=ws)
            assert torch.equal(za, ya) and torch.equal(zb, yb)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        zs = hyb.matmul_fp8(A, xa, stream=side)
        side.synchronize()
        assert torch.equal(zs, ya)
        gx, gy = torch.zeros_like(xa), torch.empty_like(ya)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            hyb.matmul_fp8(A, gx, Y=gy, ws=ws)
        gx.copy_(xa)
        g.replay()
        assert torch.equal(gy, ya)
        f = hyb.matmul_fp8(A, xa, ws=ws, flags=hyb.LAUNCH_OVERLAP_PREV)
        f2 = hyb.matmul_fp8(A, xa, ws=ws, flags=hyb.LAUNCH_OVERLAP_PREV)
        assert torch.equal(f, ya) and torch.equal(f2, ya)
    assert hyb.check_status(ws) == 0


def test_both_bindings_agree():
    """The C++ binding and the Python code (which a given stream takes) make the same calls, errors among them."""
    from sparse_weight_b200.hyb import _load_native
    nat = _load_native()
    here = torch.cuda.current_stream()
    x = values(20, 300, 1)
    ws = hyb.new_workspace(hyb.fp8_workspace_bytes(20, 130, 300), dev())
    for X in (x, x.float(), x[:1], x[::2], x[:, 8:40], x.t()[:1]):
        X = X.to(dev())
        for block_rows in (1, 128):
            a, b = hyb.quant_fp8(X, block_rows, ws), hyb.quant_fp8(X, block_rows, ws, stream=here)
            for u, v in zip(a, b):
                assert u.shape == v.shape and u.stride() == v.stride() and u.dtype == v.dtype
                assert torch.equal(u.view(torch.uint8), v.view(torch.uint8))
    A = hyb.pack_fp8(values(130, 300, 2).to(dev()))
    pad = torch.zeros(20, 304, dtype=torch.bfloat16, device=dev())
    pad[:, :300] = x.to(dev())
    X = pad[:, :300]
    xq, xs = hyb.quant_fp8(X, 1, ws)
    for ydt, yt in ((hyb.HYB_F32, torch.float32), (hyb.HYB_BF16, torch.bfloat16)):
        for u, s in ((X, None), (X[:1], None), (xq, xs), (xq[:7], xs[:7]), (xq[::3], xs[::3])):
            a = hyb.matmul_fp8(A, u, s, ydt=ydt, ws=ws)
            assert a.dtype == yt and torch.equal(a, hyb.matmul_fp8(A, u, s, ydt=ydt, ws=ws, stream=here))
            Y = torch.zeros(u.shape[0], 140, dtype=yt, device=dev())
            assert hyb.matmul_fp8(A, u, s, Y=Y[:, 3:133], ydt=ydt, ws=ws).data_ptr() == Y[:, 3:133].data_ptr()
            assert torch.equal(Y[:, 3:133], a)
    # what the C++ binding does not serve it leaves alone
    bf = torch.bfloat16
    for args in ((A._at, A._index, X.float(), None, None, 0, 0, ws), (A._at, A._index, X.cpu(), None, None, 0, 0, ws),
                 (A._at, A._index, X, None, None, 2, 0, ws), (A._at, A._index, X, None, None, 0, -1, ws),
                 (A._at, A._index, X[0], None, None, 0, 0, ws), (A._at, A._index, xq, None, None, 0, 0, ws),
                 (A._at, A._index, X, None, Y.to(bf), 0, 0, ws), (A._at, -1, X, None, None, 0, 0, ws),
                 (A._at, A._index, xq, xs[:1].expand(20, 3), None, 0, 0, ws)):
        assert nat.matmul_fp8(*args) is None
    for args in ((X.half(), 1, ws), (X, 2, ws), (X[:1].expand(4, 300), 1, ws), (X[0], 1, ws), (X.t(), 1, ws), (X, 1, None)):
        assert nat.quant_fp8(*args) is None
    with pytest.raises(hyb.HybError) as one:
        hyb.matmul_fp8(A, X, flags=6, ws=ws)
    with pytest.raises(hyb.HybError) as two:
        hyb.matmul_fp8(A, X, flags=6, ws=ws, stream=here)
    assert str(one.value) == str(two.value) and one.value.status == two.value.status
    with pytest.raises(hyb.HybError):
        hyb.quant_fp8(X, 1, ws[:100])


@pytest.mark.parametrize("ydt", [hyb.HYB_F32, hyb.HYB_BF16])
@pytest.mark.parametrize("m,n,k", [(257, 12900, 300), (500, 9400, 260), (640, 12992, 128), (385, 14336, 513),
                                   (2200, 2560, 130)])
def test_matmul_wide(m, n, k, ydt):
    """Products whose tiles fill the GPU: CTAs of 256 columns, two blocks of W's scales each."""
    A, wq, ws = weight(n, k, m + n + k)
    x = values(m, -(-k // 8) * 8, 7 * m + k)[:, :k]
    xd = torch.zeros(m, -(-k // 8) * 8, dtype=torch.bfloat16, device=dev())[:, :k]
    xd.copy_(x)
    w = hyb.new_workspace(hyb.fp8_workspace_bytes(m, n, k), dev())
    Y = torch.full((m + 1, n + 8), 3.0, dtype=torch.float32 if ydt == hyb.HYB_F32 else torch.bfloat16, device=dev())
    hyb.matmul_fp8(A, xd, Y=Y[:m, :n], ydt=ydt, ws=w)
    assert hyb.check_status(w) == 0
    assert (Y[m] == 3).all() and (Y[:, n:] == 3).all()
    check(Y[:m, :n], x, wq, ws, k)
