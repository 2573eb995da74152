"""An 8-bit weight or cache whose tensors get another storage (Tensor.data, a
module that is moved or cloned): every call reads where the values are now."""
import copy
import io
import pickle

import pytest
import torch

from gpu_cases import dev
from sparse_weight_b200 import hyb


def matrix(n=200, k=300, device="cpu", seed=0):
    g = torch.Generator().manual_seed(seed)
    ld = -(-k // 16) * 16
    q = torch.randint(0, 120, (n, ld), generator=g, dtype=torch.uint8).to(device)
    s = (torch.rand(-(-n // 128), -(-k // 128), generator=g) + 0.5).to(device)
    return hyb.Fp8Matrix(n, k, q.view(torch.float8_e4m3fn)[:, :k], s)


def cache(device="cpu", seed=0):
    g = torch.Generator().manual_seed(seed)
    kv = [torch.randint(-127, 128, (4, 2, 16, 64), generator=g, dtype=torch.int8).to(device) for _ in range(2)]
    sc = [(torch.rand(4, 2, generator=g) + 0.5).to(device) for _ in range(2)]
    return hyb.Cache(*kv, *sc)


def swap(t, to):
    """t's storage becomes another one; returns a tensor that keeps the old one."""
    old = t.detach()[:]
    t.data = to
    return old


def test_structs_follow_the_tensors():
    A, C = matrix(), cache()
    for _ in range(2):
        keep = [swap(A.q, A.q.view(torch.uint8).clone().view(A.q.dtype)), swap(A.scale, A.scale.clone())]
        s = A.struct()
        assert (s.q, s.scale, s.ldq) == (A.q.data_ptr(), A.scale.data_ptr(), A.q.stride(0))
        assert s.q != keep[0].data_ptr() and s.scale != keep[1].data_ptr()
        keep = [swap(t, t.clone()) for t in (C.k, C.v, C.k_scale, C.v_scale)]
        s = C.struct()
        for at, t, old in zip((s.k, s.v, s.k_scale, s.v_scale), (C.k, C.v, C.k_scale, C.v_scale), keep):
            assert at == t.data_ptr() != old.data_ptr()


def test_another_layout_is_refused():
    """A storage of another shape, type or stride is no longer the weight or the cache."""
    x = torch.zeros(2, 300, dtype=torch.bfloat16)
    for t, to in (("q", torch.zeros(100, 304, dtype=torch.uint8)), ("q", torch.zeros(200, 300)),
                  ("q", torch.zeros(300, 200, dtype=torch.uint8).t()), ("scale", torch.zeros(2, 2)),
                  ("scale", torch.zeros(2, 1).expand(2, 3))):
        A = matrix()
        swap(getattr(A, t), to)
        with pytest.raises(ValueError, match="Fp8Matrix"):
            hyb.matmul_fp8(A, x)
    q = torch.zeros(1, 4, 64, dtype=torch.bfloat16)
    args = (torch.zeros(1, 2, dtype=torch.int32), torch.ones(1, dtype=torch.int32))
    for t, to in (("v", torch.zeros(3, 2, 16, 64, dtype=torch.int8)), ("k", torch.zeros(4, 16, 2, 64).transpose(1, 2)),
                  ("k_scale", torch.zeros(4, 3)), ("v_scale", torch.zeros(2, 4).t())):
        C = cache()
        swap(getattr(C, t), to)
        with pytest.raises(ValueError, match="Cache"):
            hyb.cache_attention(C, q, *args)
        with pytest.raises(ValueError, match="Cache"):
            hyb.cache_append(C, q[:, :2], q[:, 2:], *args)


def test_copies():
    """deepcopy and torch.save give weights and caches of their own storage, pickle too (but for e4m3
    tensors, which torch does not unpickle outside torch.load)."""
    for X in (matrix(), cache()):
        names = ("q", "scale") if isinstance(X, hyb.Fp8Matrix) else ("k", "v", "k_scale", "v_scale")
        buf = io.BytesIO()
        torch.save(X, buf)
        buf.seek(0)
        copies = [copy.deepcopy(X), torch.load(buf, weights_only=False)]
        if isinstance(X, hyb.Cache):
            copies.append(pickle.loads(pickle.dumps(X)))
        for Y in copies:
            s = Y.struct()
            for w in names:
                a, b = getattr(X, w), getattr(Y, w)
                assert getattr(s, w) == b.data_ptr() != a.data_ptr() and a.dtype == b.dtype
                assert torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))
                assert any(t is b for t in Y._at)  # the C++ binding's view of it, too


def value(A, x):
    """The product in 64 bits from what A holds, for x of small whole numbers (exact in e4m3 with any scale)."""
    q = A.q.float().double()
    s = A.scale.double().repeat_interleave(128, 0)[:A.n].repeat_interleave(128, 1)[:, :A.k]
    return x.double() @ (q * s).t()


@pytest.mark.gpu
@pytest.mark.parametrize("k", [300, 304])
@pytest.mark.parametrize("m", [3, 20, 70])
def test_product_reads_the_new_storage(m, k):
    """Through both bindings, with the weight a module's parameter that is moved.  A move packs the rows: where k
    is no multiple of 16 bytes they then lie where no product reads them, and the call is refused."""
    class Holder(torch.nn.Module):
        def __init__(self, A):
            super().__init__()
            self.q = torch.nn.Parameter(A.q, requires_grad=False)
            self.scale = torch.nn.Parameter(A.scale, requires_grad=False)

    a, b = matrix(k=k, device=dev(), seed=1), matrix(k=k, device=dev(), seed=2)
    h = Holder(a)
    A = hyb.Fp8Matrix(a.n, a.k, h.q, h.scale)
    g = torch.Generator().manual_seed(m)
    # every block of 128 holds a 448: its scale is 1 and the values are exact
    x = torch.randint(-8, 9, (m, 304), generator=g).to(torch.bfloat16)
    x[:, ::128] = 448
    x = x.to(dev())[:, :k]
    ws = hyb.new_workspace(hyb.fp8_workspace_bytes(m, A.n, A.k), dev())
    here = torch.cuda.current_stream()

    def check(want):
        for st in (None, here):
            y = hyb.matmul_fp8(A, x, ws=ws, stream=st)
            ref = value(want, x)
            # fp32 sums of some 300 exact products: within 2^-14 of the sum of magnitudes
            env = value(hyb.Fp8Matrix(want.n, want.k, want.q.float().abs().to(want.q.dtype).contiguous()
                                      .view(torch.uint8).reshape(want.n, want.k).view(want.q.dtype), want.scale), x.abs())
            assert ((y.double() - ref).abs() <= env * 2.0 ** -14).all()

    check(a)
    keep = [swap(h.q, b.q), swap(h.scale, b.scale)]
    check(b)
    del keep
    h.cpu()
    with pytest.raises(ValueError, match="tensors"):
        hyb.matmul_fp8(A, x, ws=ws)
    h.cuda(dev())
    if k % 16:
        with pytest.raises(hyb.HybError, match="aligned"):
            hyb.matmul_fp8(A, x, ws=ws)
    else:
        check(b)


@pytest.mark.gpu
def test_cache_calls_read_the_new_storage():
    C, D = cache(dev(), 1), cache(dev(), 2)
    table = torch.tensor([[2, 0, 3]], dtype=torch.int32, device=dev())
    lens = torch.tensor([37], dtype=torch.int32, device=dev())
    g = torch.Generator().manual_seed(3)
    x = torch.randn(1, 8, 64, generator=g).to(torch.bfloat16).to(dev())
    ws = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, 1, 4, 1, 48), dev())
    here = torch.cuda.current_stream()
    names = ("k", "v", "k_scale", "v_scale")
    first = hyb.cache_attention(C, x[:, :4], table, lens, ws=ws)
    old = [swap(getattr(C, w), getattr(D, w).clone()) for w in names]
    before = [t.clone() for t in old]
    for st in (None, here):
        o = hyb.cache_attention(C, x[:, :4], table, lens, ws=ws, stream=st)
        assert torch.equal(o, hyb.cache_attention(D, x[:, :4], table, lens, ws=ws)) and not torch.equal(o, first)
        for X in (C, D):
            hyb.cache_append(X, x[:, 4:6], x[:, 6:], table, lens, ws=ws, stream=st)
        for w in names:
            assert torch.equal(getattr(C, w), getattr(D, w)), w
    assert all(torch.equal(t, u) for t, u in zip(old, before))
