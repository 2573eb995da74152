"""Argument checks of the 8-bit operators: every one is made on the host before
any CUDA call, so these run without a GPU and launch nothing."""
import ctypes

import pytest
import torch

from sparse_weight_b200 import hyb

P = ctypes.c_void_p
INV, UNS, ALI, WSP = (hyb.HYB_ERR_INVALID_ARG, hyb.HYB_ERR_UNSUPPORTED, hyb.HYB_ERR_ALIGNMENT,
                      hyb.HYB_ERR_WORKSPACE)
A = 4096  # an aligned address that nothing reads


@pytest.fixture(scope="module")
def L():
    from sparse_weight_b200 import build
    build.build()
    return hyb.lib()


def quant(L, rows=4, cols=100, X=A, ldx=104, xdt=hyb.HYB_BF16, br=1, Q=A, ldq=112, s=A, lds=1, ws=A, n=256):
    return L.hyb_fp8_quant(rows, cols, P(X), ldx, xdt, br, P(Q), ldq, P(s), lds, P(ws), n, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(rows=0), INV), (dict(cols=0), INV), (dict(X=None), INV), (dict(Q=None), INV), (dict(s=None), INV),
    (dict(xdt=hyb.HYB_E4M3), INV), (dict(xdt=7), INV), (dict(br=2), INV), (dict(br=0), INV), (dict(ldx=96), INV),
    (dict(ldq=96), INV), (dict(lds=0), INV), (dict(X=A + 1), ALI), (dict(xdt=hyb.HYB_F32, X=A + 2), ALI),
    (dict(Q=A + 8), ALI), (dict(ldq=120), ALI), (dict(ws=None), WSP), (dict(n=255), WSP),
    (dict(ws=A + 16), ALI), (dict(rows=1 << 31), UNS), (dict(cols=1 << 31, ldx=1 << 31, ldq=1 << 31, lds=1 << 30), UNS)])
def test_quant(L, kw, rc):
    assert quant(L, **kw) == rc


def matmul(L, n=64, k=100, q=A, ldq=112, scale=A, lds=1, m=4, X=A, ldx=112, xdt=hyb.HYB_BF16, xs=None, ldxs=0, Y=A,
           ldy=64, ydt=hyb.HYB_F32, flags=0, ws=A, nb=1 << 30):
    a = hyb.HybFp8Matrix(n, k, q, ldq, scale, lds)
    return L.hyb_fp8_matmul(ctypes.byref(a), m, P(X), ldx, xdt, P(xs), ldxs, P(Y), ldy, ydt, flags, P(ws), nb, None)


@pytest.mark.parametrize("kw,rc", [
    (dict(n=0), INV), (dict(k=0), INV), (dict(q=None), INV), (dict(scale=None), INV), (dict(ldq=96), INV),
    (dict(lds=0), INV), (dict(m=0), INV), (dict(X=None), INV), (dict(Y=None), INV), (dict(xdt=hyb.HYB_F32), INV),
    (dict(xdt=hyb.HYB_I8), INV), (dict(xs=A, ldxs=1), INV), (dict(xdt=hyb.HYB_E4M3), INV),
    (dict(xdt=hyb.HYB_E4M3, xs=A, ldxs=0), INV), (dict(ydt=hyb.HYB_E4M3), INV), (dict(flags=2), INV),
    (dict(ldx=96), INV), (dict(ldy=63), INV), (dict(q=A + 8), ALI), (dict(ldq=104), ALI), (dict(X=A + 2), ALI),
    (dict(ldx=108), ALI), (dict(xdt=hyb.HYB_E4M3, xs=A, ldxs=1, ldx=104), ALI), (dict(Y=A + 2), ALI),
    (dict(ydt=hyb.HYB_BF16, Y=A + 1), ALI), (dict(ws=None), WSP), (dict(nb=255), WSP), (dict(ws=A + 128), ALI),
    (dict(m=1 << 31), UNS), (dict(n=1 << 31), UNS)])
def test_matmul(L, kw, rc):
    assert matmul(L, **kw) == rc


def test_matmul_null(L):
    assert L.hyb_fp8_matmul(None, 1, P(A), 16, 1, None, 0, P(A), 16, 0, 0, P(A), 1 << 20, None) == INV
    assert L.hyb_fp8_workspace_bytes(0, 1, 1) == 0 and L.hyb_fp8_workspace_bytes(1, 0, 1) == 0
    assert L.hyb_fp8_workspace_bytes(1, 1, 0) == 0 and L.hyb_fp8_workspace_bytes(1, 1, 1) >= 256


def structs(**kw):
    c = dict(k=A, v=A, k_scale=A, v_scale=A, type=hyb.HYB_E4M3, num_pages=8, kv_heads=2, page_size=16, head_dim=64,
             stride_page=2048, stride_head=1024, stride_token=64)
    s = dict(batch=2, max_new=3, rows=6, lens=A, off=None, page_table=A, max_pages=4, table_stride=4)
    for name, value in kw.items():
        (c if name in c else s)[name] = value
    return hyb.HybCache(*c.values()), hyb.HybSequences(*s.values())


CACHE = [
    (dict(k=None), INV), (dict(v=None), INV), (dict(k_scale=None), INV), (dict(v_scale=None), INV),
    (dict(type=hyb.HYB_BF16), INV), (dict(num_pages=0), INV), (dict(kv_heads=0), INV), (dict(page_size=0), UNS),
    (dict(page_size=24), UNS), (dict(page_size=128), UNS), (dict(head_dim=96), UNS), (dict(head_dim=256), UNS),
    (dict(stride_page=0), INV), (dict(stride_head=-64), INV), (dict(stride_token=32), INV), (dict(k=A + 8), ALI),
    (dict(v=A + 4), ALI), (dict(stride_token=72), ALI), (dict(stride_page=2056), ALI), (dict(stride_page=1 << 40), UNS),
    (dict(batch=0), INV), (dict(max_new=0), INV), (dict(rows=-1), INV), (dict(rows=5), INV), (dict(lens=None), INV),
    (dict(page_table=None), INV), (dict(max_pages=0), INV), (dict(table_stride=3), INV), (dict(batch=65536), UNS),
    (dict(lens=A + 2), ALI), (dict(off=A + 1), ALI)]


def append(L, K=A, ldk=128, hsk=64, V=A, ldv=128, hsv=64, ws=A, n=256, **kw):
    c, s = structs(**kw)
    return L.hyb_cache_append(ctypes.byref(c), ctypes.byref(s), P(K), ldk, hsk, P(V), ldv, hsv, P(ws), n, None)


@pytest.mark.parametrize("kw,rc", CACHE + [
    (dict(K=None), INV), (dict(V=None), INV), (dict(ldk=32), INV), (dict(hsv=8), INV), (dict(K=A + 2), ALI),
    (dict(ldv=130), ALI), (dict(hsk=68), ALI), (dict(ws=None), WSP), (dict(n=100), WSP), (dict(ws=A + 64), ALI)])
def test_append(L, kw, rc):
    assert append(L, **kw) == rc


def attention(L, Q=A, ldq=256, hsq=64, O=A, ldo=256, hso=64, lse=None, ldl=4, heads=4, scale=0.125, window=0, sinks=0,
              ws=None, n=0, **kw):
    c, s = structs(**kw)
    return L.hyb_cache_attention(ctypes.byref(c), ctypes.byref(s), P(Q), ldq, hsq, P(O), ldo, hso, P(lse), ldl, heads,
                                 scale, window, sinks, P(ws), n, None)


@pytest.mark.parametrize("kw,rc", CACHE + [
    (dict(Q=None), INV), (dict(O=None), INV), (dict(heads=0), INV), (dict(heads=3), INV), (dict(window=-1), INV),
    (dict(sinks=-1), INV), (dict(scale=float("nan")), INV), (dict(ldq=8), INV), (dict(hso=8), INV),
    (dict(lse=A, ldl=3), INV), (dict(Q=A + 2), ALI), (dict(hsq=68), ALI), (dict(ldo=260), ALI), (dict(lse=A + 1), ALI),
    (dict(), WSP)])
def test_attention(L, kw, rc):
    assert attention(L, **kw) == rc


def test_null_structs(L):
    c, s = structs()
    assert L.hyb_cache_append(None, ctypes.byref(s), P(A), 128, 64, P(A), 128, 64, P(A), 256, None) == INV
    assert L.hyb_cache_append(ctypes.byref(c), None, P(A), 128, 64, P(A), 128, 64, P(A), 256, None) == INV
    assert L.hyb_cache_attention_workspace_bytes(None, 1, 1, 1, 2) == 0
    assert L.hyb_cache_attention_workspace_bytes(ctypes.byref(c), 1, 1, 1, 3) == 0
    assert L.hyb_cache_attention_workspace_bytes(ctypes.byref(c), 0, 1, 1, 2) == 0


def test_products_refuse_the_8_bit_output_types(L):
    """The new hyb_dtype values are no output type of the products."""
    m = hyb.HybMatrix(128, 128, 128, 128, 1, A, A, A, A, A, 128 * 128, 0, None, 0)
    for ydt in (hyb.HYB_E4M3, hyb.HYB_I8):
        assert L.hyb_spmv(ctypes.byref(m), P(A), 128, P(A), 128, ydt, None, P(A), 1 << 20, None) == INV
        assert L.hyb_gemv_dense(128, 128, 1, P(A), 128, P(A), 128, P(A), 128, ydt, P(A), 1 << 20, None) == INV


def test_binding_checks():
    """The binding's own checks: types, shapes, devices, strides (CPU tensors: nothing is launched)."""
    e4 = torch.zeros(4, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        hyb.Fp8Matrix(4, 128, e4, torch.zeros(2, 1))
    with pytest.raises(ValueError):
        hyb.Fp8Matrix(4, 128, e4.float(), torch.zeros(1, 1))
    a = hyb.Fp8Matrix(4, 128, e4, torch.zeros(1, 1))
    for x, xs in ((torch.zeros(2, 100, dtype=torch.bfloat16), None), (torch.zeros(2, 128), None),
                  (e4, None), (e4, torch.zeros(4, 2)), (torch.zeros(2, 128, dtype=torch.bfloat16), None)):
        with pytest.raises(ValueError):
            hyb.matmul_fp8(a, x, xs=xs)
    with pytest.raises(ValueError):
        hyb.quant_fp8(torch.zeros(2, 128, dtype=torch.float16))
    kv = torch.zeros(3, 2, 16, 64, dtype=torch.int8)
    s = torch.zeros(3, 2)
    with pytest.raises(ValueError):
        hyb.Cache(kv, kv.float(), s, s)
    with pytest.raises(ValueError):
        hyb.Cache(kv, kv[:2], s, s)
    with pytest.raises(ValueError):
        hyb.Cache(kv, kv, s, s.double())
    C = hyb.Cache(kv, kv, s, s)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    t, lens = torch.zeros(2, 3, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        hyb.cache_attention(C, q, t, lens)
    with pytest.raises(ValueError, match="CUDA"):
        hyb.cache_append(C, q[:, :2], q[:, 2:], t, lens)
    for bad in (dict(Q=q.float()), dict(Q=q[:, :, :32]), dict(Q=q[:1])):
        with pytest.raises(ValueError):
            hyb.cache_attention(C, bad["Q"], t, lens)


def test_expanded_rows_are_refused():
    """Rows that lie on one another (expand) would be read past their tensor's end; one row may have any stride."""
    e4 = torch.zeros(4, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    a = hyb.Fp8Matrix(4, 128, e4, torch.zeros(1, 1))
    q300 = torch.zeros(300, 128, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(ValueError, match="overlap"):
        hyb.Fp8Matrix(300, 128, q300, torch.zeros(1, 1).expand(3, 1))
    with pytest.raises(ValueError, match="overlap"):
        hyb.Fp8Matrix(300, 128, q300[:1].view(torch.uint8).expand(300, 128), torch.zeros(3, 1))
    for block_rows in (1, 128):
        for x in (torch.zeros(1, 128).expand(5, 128), torch.zeros(200).as_strided((3, 128), (16, 1))):
            with pytest.raises(ValueError, match="overlap"):
                hyb.quant_fp8(x, block_rows)
    with pytest.raises(ValueError, match="overlap"):
        hyb.matmul_fp8(a, e4, xs=torch.zeros(1, 1).expand(4, 1))
    with pytest.raises(ValueError, match="CUDA"):
        hyb.matmul_fp8(a, e4[:1], xs=torch.zeros(1, 1).expand(1, 1))
    kv, s = torch.zeros(3, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2)
    C = hyb.Cache(kv, kv, s, s)
    q, lens = torch.zeros(2, 4, 64, dtype=torch.bfloat16), torch.ones(2, dtype=torch.int32)
    for t in (torch.zeros(1, 3, dtype=torch.int32).expand(2, 3), torch.zeros(8, dtype=torch.int32).as_strided((2, 3), (2, 1))):
        with pytest.raises(ValueError, match="overlap"):
            hyb.cache_attention(C, q, t, lens)
        with pytest.raises(ValueError, match="overlap"):
            hyb.cache_append(C, q[:, :2], q[:, 2:], t, lens)
    with pytest.raises(ValueError, match="CUDA"):
        hyb.cache_attention(C, q[:1], torch.zeros(1, 1, dtype=torch.int32).expand(1, 3).contiguous()[:, :3], lens[:1])


def test_largest_sizes(L):
    """Columns that the quantiser could not count in 31 bits are refused."""
    big = (1 << 31) - 2048
    assert quant(L, cols=big, ldx=big, ldq=big, lds=1 << 30) == UNS
    assert matmul(L, k=big, ldq=big, lds=1 << 30, ldx=big) == UNS
    assert L.hyb_fp8_workspace_bytes(1, 1, big) == 0 and L.hyb_fp8_workspace_bytes(1, 1, big - 1) > 0


def test_stream_of_another_device():
    class Stream:
        device_index, cuda_stream = 1, 0
    with pytest.raises(ValueError, match="device 1"):
        hyb._scope(0, Stream())
