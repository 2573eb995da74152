"""The 8-bit operators where offsets pass 32 bits, as a process's first (captured)
calls, and on two streams at once."""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import ref8
from gpu_cases import dev
from sparse_weight_b200 import hyb
from test_gpu_cache import TYPES, check_attention, dev32, queries

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("type_,order", [("e4m3", "pht"), ("i8", "pth")])
def test_a_cache_of_more_than_4_gib(type_, order):
    """Pages at both ends of keys and values of 4.6 GB each: appended, then read by 1, 5 and 90 new tokens."""
    pages, heads, size, dim = 70001, 8, 64, 128
    shape = {"pht": (pages, heads, size, dim), "pth": (pages, size, heads, dim)}[order]
    kv = [torch.zeros(shape, dtype=torch.uint8, device=dev()).view(TYPES[type_]) for _ in range(2)]
    kv = [x.transpose(1, 2) if order == "pth" else x for x in kv]
    C = hyb.Cache(*kv, *(torch.zeros(pages, heads, device=dev()) for _ in range(2)))
    far = [70000, 0, 69999, 32768, 32769, 65536, 1]  # 32768 and 65536 pages: 2^31 and 2^32 bytes
    table = np.array([far], np.int32)
    T = 6 * size + 9
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, 2 * heads, dim, generator=g).to(torch.bfloat16)
    d = x.to(dev())
    ref = dict(k=np.zeros((7, heads, size, dim)), v=np.zeros((7, heads, size, dim)),
               k_scale=np.zeros((7, heads), np.float32), v_scale=np.zeros((7, heads), np.float32))
    near = np.arange(7, dtype=np.int32).reshape(1, -1)
    ref8.append(ref, dict(k=x[:, :heads].double().numpy(), v=x[:, heads:].double().numpy()), near, [T], [0, T], type_ == "i8")
    ws = hyb.new_workspace(256, dev())
    hyb.cache_append(C, d[:, :heads], d[:, heads:], dev32(table), dev32([T]), ws=ws)
    assert hyb.check_status(ws) == 0
    small = hyb.Cache(*(t[far].contiguous() if t.dtype == torch.int8 else
                        t.view(torch.uint8)[far].contiguous().view(t.dtype) for t in (C.k, C.v)),
                      C.k_scale[far].contiguous(), C.v_scale[far].contiguous())
    from test_gpu_cache import host_cache
    got = host_cache(small)
    for w in ref:
        assert np.array_equal(got[w], ref[w]), w
    # nothing else was written (the pages beside the used ones stand for all)
    for p in (2, 32767, 32770, 65535, 65537, 69998):
        assert not C.k.view(torch.uint8)[p].any() and not C.v.view(torch.uint8)[p].any()
    for new in (1, 5, 90):
        q = queries(new, 16, dim, new)
        for kw in ({}, dict(window=70, sinks=66)):
            o, lse = hyb.cache_attention(C, q.to(dev()), dev32(table), dev32([T]), return_lse=True, **kw)
            check_attention(small, near, [T], [0, new], q, o, lse, **kw)


def test_rows_far_apart():
    """Rows of inputs and outputs 2^30 elements apart."""
    far = 1 << 30
    buf = torch.empty(2 * far + 512, dtype=torch.bfloat16, device=dev())
    g = torch.Generator().manual_seed(4)
    x = torch.randn(3, 400, generator=g).to(torch.bfloat16).to(dev())
    X = buf.as_strided((3, 400), (far, 1))
    X.copy_(x)
    q, s = hyb.quant_fp8(X)
    q0, s0 = hyb.quant_fp8(x)
    assert torch.equal(q.view(torch.uint8), q0.view(torch.uint8)) and torch.equal(s, s0)
    n = 300
    A = hyb.pack_fp8((torch.randn(n, 400, generator=g) / 20).to(dev()))
    out = torch.empty(2 * far + 512, device=dev()).as_strided((3, n), (far, 1))
    assert torch.equal(hyb.matmul_fp8(A, X, Y=out), hyb.matmul_fp8(A, x))
    for m in (20, 70):  # the same rows for the kernels of more tokens
        step = (2 * far) // (m - 1) // 16 * 16
        xm = torch.randn(m, 400, generator=g).to(torch.bfloat16).to(dev())
        X = buf.as_strided((m, 400), (step, 1))
        X.copy_(xm)
        out = torch.empty(step * (m - 1) + 512, device=dev()).as_strided((m, n), (step, 1))
        assert torch.equal(hyb.matmul_fp8(A, X, Y=out), hyb.matmul_fp8(A, xm))
    # attention: query and output rows
    C = hyb.new_cache(2, 1, 64, 64, torch.int8, dev())
    C.k.copy_(torch.randint(-127, 128, C.k.shape, generator=g, dtype=torch.int8))
    C.v.copy_(torch.randint(-127, 128, C.v.shape, generator=g, dtype=torch.int8))
    for sc in (C.k_scale, C.v_scale):
        sc.fill_(2.0 ** -6)
    t, n = dev32([[1, 0]]), dev32([100])
    for new in (3, 12, 80):
        step = (2 * far) // (new - 1) // 16 * 16
        qd = torch.randn(new, 2, 64, generator=g).to(torch.bfloat16).to(dev())
        Q = buf.as_strided((new, 2, 64), (step, 64, 1))
        Q.copy_(qd)
        O = torch.empty(step * (new - 1) + 512, dtype=torch.bfloat16, device=dev()).as_strided((new, 2, 64), (step, 64, 1))
        assert torch.equal(hyb.cache_attention(C, Q, t, n, out=O), hyb.cache_attention(C, qd, t, n))


SCRIPT = """
import torch
from sparse_weight_b200 import hyb
dev = "cuda:0"
g = torch.Generator().manual_seed(1)
W = (torch.randn(700, 1100, generator=g) / 30).to(dev)
C = hyb.new_cache(12, 2, 16, {dim}, {dtype}, dev)
x = torch.randn({m}, 1104, generator=g).to(torch.bfloat16).to(dev)[:, :1100]
kv = torch.randn({m}, 4, {dim}, generator=g).to(torch.bfloat16).to(dev)
q = torch.randn({m}, 8, {dim}, generator=g).to(torch.bfloat16).to(dev)
table = torch.arange(12, dtype=torch.int32, device=dev).view(1, 12)
lens = torch.tensor([190], dtype=torch.int32, device=dev)
wq = hyb.new_workspace(256, dev)
wm = hyb.new_workspace(hyb.fp8_workspace_bytes({m}, 700, 1100), dev)
wa = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, 1, 8, {m}, 192), dev)
torch.cuda.synchronize()
def calls():
    A = hyb.Fp8Matrix(700, 1100, *hyb.quant_fp8(W, 128, ws=wq))
    y = hyb.matmul_fp8(A, x, ws=wm)
    hyb.cache_append(C, kv[:, :2], kv[:, 2:], table, lens, ws=wq)
    return y, hyb.cache_attention(C, q, table, lens, ws=wa)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y, o = calls()
graph.replay()
torch.cuda.synchronize()
first = y.clone(), o.clone(), C.k.clone()
for _ in range(3):
    graph.replay()
y2, o2 = calls()
for a, b in zip(first, (y2, o2, C.k)):
    assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
assert torch.equal(y, y2) and torch.equal(o, o2) and not y.isnan().any() and y.abs().max() > 0 and o.abs().max() > 0
for w in (wq, wm, wa):
    assert hyb.check_status(w) == 0
print("same")
"""


@pytest.mark.parametrize("m,dim,dtype", [(1, 128, "torch.int8"), (12, 64, "torch.float8_e4m3fn"), (90, 128, "torch.float8_e4m3fn")])
def test_first_calls_of_a_process_are_captured(m, dim, dtype):
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(m=m, dim=dim, dtype=dtype)], cwd=ROOT, capture_output=True,
                       text=True, timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stderr[-2000:]


def test_two_streams_at_once():
    """Calls of every kind beside one another, each stream with workspaces of its own: the bits of a call alone."""
    g = torch.Generator().manual_seed(2)
    A = hyb.pack_fp8((torch.randn(1500, 2000, generator=g) / 40).to(dev()))
    C = hyb.new_cache(200, 2, 32, 128, torch.float8_e4m3fn, dev())
    for t in (C.k, C.v):
        t.copy_(torch.randn(t.shape, generator=g).to(dev()).to(t.dtype))
    for t in (C.k_scale, C.v_scale):
        t.fill_(0.25)
    table = dev32(np.arange(200).reshape(2, 100))
    lens = dev32([3100, 1700])
    work = []
    for m, new in ((1, 1), (16, 4), (100, 10), (300, 100)):
        x = torch.randn(m, 2000, generator=g).to(torch.bfloat16).to(dev())
        q = torch.randn(2 * new, 16, 128, generator=g).to(torch.bfloat16).to(dev())
        work.append((x, q, new))
    want = [(hyb.matmul_fp8(A, x), hyb.cache_attention(C, q, table, lens)) for x, q, _ in work]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [(hyb.new_workspace(hyb.fp8_workspace_bytes(300, 1500, 2000), dev()),
               hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, 2, 16, 100, 3200), dev())) for _ in streams]
    torch.cuda.synchronize()
    got = [[], []]
    for turn in range(12):
        for i, st in enumerate(streams):
            x, q, _ = work[(turn + 2 * i) % 4]
            with torch.cuda.stream(st):
                got[i].append(((turn + 2 * i) % 4, hyb.matmul_fp8(A, x, ws=spaces[i][0]),
                               hyb.cache_attention(C, q, table, lens, ws=spaces[i][1])))
    torch.cuda.synchronize()
    for i in range(2):
        for j, y, o in got[i]:
            assert torch.equal(y, want[j][0]) and torch.equal(o, want[j][1])
        for w in spaces[i]:
            assert hyb.check_status(w) == 0
