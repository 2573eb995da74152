"""The attention block: projections, append, attention and output projection as
a decode loop runs them, with hybrid and 8-bit weights."""
import numpy as np
import pytest
import torch

import ref8
from gpu_cases import dev
from sparse_weight_b200 import decode, hyb, inputs
from test_gpu_cache import TYPES, dev32, host_cache

pytestmark = pytest.mark.gpu
HID, HEADS, KVH, DIM, SIZE = 512, 8, 2, 64, 16


def weight(kind, n, k, seed):
    """(library weight, the float64 matrix it stands for)."""
    W = inputs.weight(n, k, 0.05, seed)
    if kind == "fp8":
        A = hyb.pack_fp8(W.to(dev()))
        q, s = ref8.quant(W.double().numpy(), 128)
        return A, q * np.repeat(np.repeat(s, 128, 0)[:n], 128, 1)[:, :k]
    tmap = inputs.tile_map_fraction((n // 128) * (k // 128), 0.5, seed)
    return hyb.pack(W.to(dev()), tmap, 128, 128), None


def block(kinds, type_, pages, batch, width, **kw):
    wq, wk, wv, wo = (weight(c, n, k, 10 + i)[0] for i, (c, n, k) in enumerate(zip(
        kinds, (HEADS * DIM, KVH * DIM, KVH * DIM, HID), (HID, HID, HID, HEADS * DIM))))
    C = hyb.new_cache(pages, KVH, SIZE, DIM, TYPES[type_], dev())
    return decode.AttentionBlock(wq, wk, wv, wo, HEADS, C, batch, width, **kw)


@pytest.mark.parametrize("type_", ["e4m3", "i8"])
@pytest.mark.parametrize("kinds,window", [(("fp8",) * 4, 0), (("hyb", "fp8", "hyb", "hyb"), 0), (("fp8",) * 3 + ("hyb",), 24)])
def test_prompt_and_decode_steps(kinds, window, type_):
    B, width = 3, 6
    blk = block(kinds, type_, B * width + 1, B, width, max_new=40, max_rows=75, window=window, sinks=2 if window else 0)
    rng = np.random.default_rng(1)
    table = rng.permutation(B * width).reshape(B, width).astype(np.int32)
    lens = np.zeros(B, int)
    for step, new in enumerate(([40, 5, 30], [1, 1, 1], [1, 1, 1], [3, 0, 17], [1, 1, 1])):
        lens = lens + new
        off = np.concatenate([[0], np.cumsum(new)])
        x = inputs.activations(int(off[-1]), HID, 50 + step).to(dev())
        before = host_cache(blk.cache)
        y = blk.step(x, dev32(table), dev32(lens), dev32(off), max(new))
        rows = x.shape[0]
        # the same products on their own give the projections bit for bit
        q, k, v = (blk._product(w, x).view(rows, -1, DIM) for w in (blk.wq, blk.wk, blk.wv))
        ref8.append(before, dict(k=k.double().cpu().numpy(), v=v.double().cpu().numpy()), table, lens, off, type_ == "i8")
        got = host_cache(blk.cache)
        for w in got:
            assert np.array_equal(got[w], before[w]), (step, w)
        a, lse = hyb.cache_attention(blk.cache, q, dev32(table), dev32(lens), dev32(off), max(new), window=window,
                                     sinks=blk.sinks, return_lse=True)
        O, L, bO, bl = ref8.attention(got, q.double().cpu().numpy(), table, lens, off, DIM ** -0.5, window, blk.sinks)
        assert (np.abs(a.double().cpu().numpy() - O) <= bO + 1e-30).all()
        assert (np.abs(lse.double().cpu().numpy() - L) <= bl).all()
        assert torch.equal(y, blk._product(blk.wo, a.view(rows, -1)))
    blk.check()


def test_captured_step():
    """A captured decode step, replayed with new tokens, equals eager steps."""
    B, width = 2, 4
    one, two = (block(("fp8",) * 4, "e4m3", B * width, B, width) for _ in range(2))
    table = dev32(np.arange(B * width).reshape(B, width))
    x, lens = torch.zeros(B, HID, dtype=torch.bfloat16, device=dev()), dev32([1, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        two.step(x, table, lens)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = two.step(x, table, lens)
    for t in range(20):
        z = inputs.activations(B, HID, t).to(dev())
        n = dev32([t + 1, t + 1])
        want = one.step(z, table, n)
        x.copy_(z)
        lens.copy_(n)
        g.replay()
        assert torch.equal(y, want), t
    for w in ("k", "v"):
        assert torch.equal(getattr(one.cache, w).view(torch.uint8), getattr(two.cache, w).view(torch.uint8))
    one.check()
    two.check()


def test_step_refuses_what_it_was_not_made_for():
    blk = block(("fp8",) * 4, "e4m3", 8, 2, 4)
    table = dev32(np.zeros((2, 4)))
    x = torch.zeros(2, HID, dtype=torch.bfloat16, device=dev())
    with pytest.raises(ValueError):
        blk.step(torch.zeros(4, HID, dtype=torch.bfloat16, device=dev()), table, dev32([2, 2]))
    with pytest.raises(ValueError):
        blk.step(x, dev32(np.zeros((2, 5))), dev32([1, 1]))
    with pytest.raises(ValueError):
        decode.AttentionBlock(blk.wk, blk.wk, blk.wv, blk.wo, HEADS, blk.cache, 2, 4)


@pytest.mark.parametrize("batch,new,width", [(11, 12, 22), (13, 1, 5), (1, 21, 22), (4, 3, 9)])
def test_smaller_steps_fit(batch, new, width):
    """A block serves every step within its sizes, as one made for just that step does."""
    B, N, W = 13, 21, 22
    big = block(("fp8",) * 4, "e4m3", B * W, B, W, max_new=N)
    own = block(("fp8",) * 4, "e4m3", B * W, batch, width, max_new=new)
    table = dev32(np.arange(batch * width).reshape(batch, width))
    lens = dev32([max(new, (37 * b) % (width * SIZE)) for b in range(batch)])
    x = inputs.activations(batch * new, HID, 3).to(dev())
    assert torch.equal(big.step(x, table, lens), own.step(x, table, lens))
    big.check()
    own.check()


def test_ragged_step_without_max_new():
    """off without max_new: any sequence may have as many new tokens as the block allows."""
    one, two = (block(("fp8",) * 4, "i8", 8, 2, 4, max_new=30) for _ in range(2))
    table, lens, off = dev32([[0, 1, 2, 3], [4, 5, 6, 7]]), dev32([30, 4]), dev32([0, 30, 32])
    x = inputs.activations(32, HID, 9).to(dev())
    assert torch.equal(one.step(x, table, lens, off), two.step(x, table, lens, off, 30))
    one.check()


def test_check_reports_the_shared_quantiser():
    blk = block(("fp8",) * 4, "i8", 8, 1, 4, max_new=30)
    x = inputs.activations(30, HID, 9).to(dev())
    x[3, 7] = float("nan")
    blk.step(x, dev32([[0, 1, 2, 3]]), dev32([30]))
    # the append and the last product flag it too: their words are cleared first
    for ws in (blk._ws_append, blk._ws_fp8, blk._ws_attention):
        try:
            hyb.check_status(ws)
        except hyb.HybError:
            pass
    with pytest.raises(hyb.HybError) as ei:
        blk.check()
    assert ei.value.flags == hyb.STATUS_NAN
