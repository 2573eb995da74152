"""Numbers that a 32-bit field of the C structs would cut off are refused, not
wrapped (CPU tensors: nothing is launched)."""
import pytest
import torch

from sparse_weight_b200 import hyb

WIDE = [1 << 31, 1 << 32, (1 << 32) + 16, (1 << 63) - 1, -(1 << 31) - 1]


def parts():
    kv, s = torch.zeros(3, 2, 16, 64, dtype=torch.int8), torch.zeros(3, 2)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    return (hyb.Cache(kv, kv.clone(), s, s.clone()), q, torch.zeros(2, 3, dtype=torch.int32),
            torch.ones(2, dtype=torch.int32), torch.tensor([0, 1, 2], dtype=torch.int32))


@pytest.mark.parametrize("v", WIDE)
def test_attention_and_append(v):
    C, q, table, lens, off = parts()
    for kw in (dict(window=v), dict(sinks=v), dict(window=16, sinks=v), dict(off=off, max_new=v)):
        with pytest.raises(ValueError, match="32 bits"):
            hyb.cache_attention(C, q, table, lens, **kw)
    with pytest.raises(ValueError, match="32 bits"):
        hyb.cache_append(C, q[:, :2], q[:, 2:], table, lens, off=off, max_new=v)


@pytest.mark.parametrize("v", [x for x in WIDE if x > 0])
def test_workspace(v):
    C = parts()[0]
    for a in ((v, 4, 1, 48), (2, v, 1, 48), (2, 4, v, 48), (2, 4, 1, 16 * v)):
        with pytest.raises(ValueError, match="32 bits"):
            hyb.cache_attention_workspace_bytes(C, *a)


@pytest.mark.parametrize("v", [-1, 1 << 32, (1 << 32) + 1])
def test_product_flags(v):
    A = hyb.Fp8Matrix(4, 128, torch.zeros(4, 128, dtype=torch.uint8), torch.zeros(1, 1))
    with pytest.raises(ValueError, match="32 bits"):
        hyb.matmul_fp8(A, torch.zeros(2, 128, dtype=torch.bfloat16), flags=v)


def test_more_pages_than_32_bits():
    kv = torch.zeros(1, 1, 16, 64, dtype=torch.int8).expand((1 << 31) + 5, 1, 16, 64)
    s = torch.empty((1 << 31) + 5, 1, device="meta")
    with pytest.raises(ValueError, match="32 bits"):
        hyb.Cache(kv.to("meta"), kv.to("meta"), s, s)


def test_the_largest_numbers_stay_open():
    """What fits goes on to the next check (here the device's)."""
    C, q, table, lens, off = parts()
    top = (1 << 31) - 1
    with pytest.raises(ValueError, match="CUDA"):
        hyb.cache_attention(C, q, table, lens, window=top, sinks=top)
    with pytest.raises(ValueError, match="CUDA"):
        hyb.cache_attention(C, q, table, lens, off=off, max_new=top)
