"""A step whose rows end with padding (off[batch] < rows, as a captured step of a
fixed size has them): the rows of no sequence give what a zero attention gives,
and nothing that lies in fresh memory is read or reported."""
import pytest
import torch

from gpu_cases import dev
from sparse_weight_b200 import hyb, inputs
from test_gpu_cache import dev32
from test_gpu_decode import HID, block

pytestmark = pytest.mark.gpu


def soil(shapes):
    """Leave NaN in the blocks that the allocator hands out next."""
    for _ in range(3):
        keep = [torch.full(s, float("nan"), dtype=torch.bfloat16, device=dev()) for s in shapes]
        torch.cuda.synchronize()
        del keep


@pytest.mark.parametrize("kinds", [("fp8",) * 4, ("hyb", "fp8", "fp8", "hyb")])
@pytest.mark.parametrize("new,rows", [([3, 1, 0], 12), ([20, 5, 1], 40), ([1, 1, 1], 4), ([0, 0, 0], 5)])
def test_padded_step(kinds, new, rows):
    B, width = 3, 4
    one, two = (block(kinds, "e4m3", B * width, B, width, max_new=40, max_rows=64) for _ in range(2))
    table = dev32([[4 * b + j for j in range(width)] for b in range(B)])
    lens = [n + 2 if n else 0 for n in new]
    off = [0]
    for n in new:
        off.append(off[-1] + n)
    x = inputs.activations(rows, HID, 3).to(dev())
    x[off[-1]:] = 0
    # two tokens in the cache of every sequence that has new ones
    pre, poff = inputs.activations(6, HID, 4).to(dev()), dev32([0, 2, 4, 6])
    for blk in (one, two):
        blk.step(pre, table, dev32([2] * B), poff, 2)
    soil([(rows, 8, 64), (rows, HID), (rows, 2, 64), (rows, 8 * 64)])
    y = one.step(x, table, dev32(lens), dev32(off), 40)
    one.check()
    assert (y[off[-1]:] == 0).all() and not y.isnan().any()
    if off[-1]:
        # the live rows: what a step without padding gives, up to the products' own choice of kernel by rows
        q = one._product(one.wq, x).view(rows, 8, 64)
        a = hyb.cache_attention(one.cache, q, table, dev32(lens), dev32(off), 40, out=torch.zeros_like(q))
        assert torch.equal(y, one._product(one.wo, a.view(rows, -1)))


def test_padded_step_captured():
    """One captured step of 6 rows serves fewer live ones."""
    B, width, rows = 3, 4, 6
    blk, ref = (block(("fp8",) * 4, "i8", B * width, B, width, max_new=2, max_rows=rows) for _ in range(2))
    table = dev32([[4 * b + j for j in range(width)] for b in range(B)])
    x = torch.zeros(rows, HID, dtype=torch.bfloat16, device=dev())
    lens, off = dev32([0] * B), dev32([0] * (B + 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        blk.step(x, table, lens, off)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = blk.step(x, table, lens, off)
    had = [0] * B
    for t, new in enumerate(([2, 2, 2], [1, 0, 2], [0, 1, 0], [2, 1, 1])):
        had = [h + n for h, n in zip(had, new)]
        offs = [0]
        for n in new:
            offs.append(offs[-1] + n)
        z = inputs.activations(rows, HID, t).to(dev())
        z[offs[-1]:] = 0
        x.copy_(z)
        lens.copy_(dev32(had))
        off.copy_(dev32(offs))
        g.replay()
        soil([(rows, 8, 64)])
        want = ref.step(z, table, lens, off)
        assert torch.equal(y, want) and (y[offs[-1]:] == 0).all()
    blk.check()
    ref.check()
