"""The append's scale where the largest value is a power of two times the format's
largest, exactly, and one bf16 step to either side: the smallest 2^e that holds it."""
import numpy as np
import pytest
import torch

import ref8
from gpu_cases import dev
from sparse_weight_b200 import hyb
from test_gpu_cache import TYPES, dev32, host_cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("type_", ["e4m3", "i8"])
def test_borders(type_, dim):
    size, exps = 16, range(-50, 62)
    border = torch.tensor([(1.75 if type_ == "e4m3" else 127.0 / 64) * 2.0 ** (e + (8 if type_ == "e4m3" else 6))
                           for e in exps]).to(torch.bfloat16)
    bits = border.view(torch.int16)
    tops = torch.stack([(bits + d).view(torch.bfloat16) for d in (-1, 0, 1)], 1).reshape(-1)  # a page each
    T = size * len(tops)
    g = torch.Generator().manual_seed(dim)
    x = torch.rand(len(tops), size, 2, dim, generator=g) * 2 - 1
    x = (x * tops.float()[:, None, None, None] * 0.99).to(torch.bfloat16)
    at = torch.randint(0, size * dim, (len(tops), 2), generator=g)
    for w in range(2):
        for p in range(len(tops)):
            x[p, at[p, w] // dim, w, at[p, w] % dim] = tops[p] if p % 2 else -tops[p]
    x = x.reshape(T, 2, dim)
    C = hyb.new_cache(len(tops), 1, size, dim, TYPES[type_], dev())
    table = np.random.default_rng(1).permutation(len(tops)).astype(np.int32).reshape(1, -1)
    ref = host_cache(C)
    ref8.append(ref, dict(k=x[:, :1].double().numpy(), v=x[:, 1:].double().numpy()), table, [T], [0, T], type_ == "i8")
    ws = hyb.new_workspace(256, dev())
    d = x.to(dev())
    hyb.cache_append(C, d[:, :1], d[:, 1:], dev32(table), dev32([T]), ws=ws)
    assert hyb.check_status(ws) == 0
    got = host_cache(C)
    for w in ref:
        assert np.array_equal(got[w], ref[w]), w
    # the rule itself, in whole numbers of bf16's exponent and fraction
    most = 448 if type_ == "e4m3" else 127
    for p, top in enumerate(tops.double().tolist()):
        s = float(got["k_scale"][table[0, p], 0])
        assert s == 2.0 ** -40 or most * s / 2 < top
        assert s == 2.0 ** 60 or most * s >= top
