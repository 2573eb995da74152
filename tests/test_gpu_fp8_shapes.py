"""Quantiser and products at sizes that choose each variant: four blocks per
half-warp (prompts), 9 to 32 tokens over wide weights (one or several CTAs per
cluster, ragged columns, any alignment of Y), few tokens over long rows."""
import numpy as np
import pytest
import torch

import ref8
from gpu_cases import dev
from sparse_weight_b200 import hyb
from test_gpu_fp8 import check, decoded, values, weight

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("shape", [(1300, 1100), (3, 500000), (9473, 100), (1185, 1024), (149, 8200)])
def test_quant_of_many_blocks(shape, dtype):
    """Rows x blocks around and beyond 9472, where a warp takes 8 blocks: lanes, divisions and the ragged last block."""
    x = values(*shape, seed=sum(shape), dtype=dtype)
    x[0, :min(128, shape[1])] = 0
    x[-1, -1] = 5000
    ws = hyb.new_workspace(256, dev())
    q, s = hyb.quant_fp8(x.to(dev()), 1, ws=ws)
    assert hyb.check_status(ws) == 0
    rq, rs = ref8.quant(x.double().numpy(), 1)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(decoded(q), rq)
    # rows that do not start on 16 bytes, and what lies behind them
    odd = torch.full((shape[0], shape[1] + 3), float("nan"), dtype=dtype, device=dev())
    odd[:, 1:shape[1] + 1] = x.to(dev())
    q2, s2 = hyb.quant_fp8(odd[:, 1:shape[1] + 1], 1, ws=ws)
    assert hyb.check_status(ws) == 0
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(s2, s)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_of_many_blocks_with_nan_and_inf(dtype):
    x = values(1300, 1100, 1, dtype)
    for i, v in enumerate((float("nan"), float("inf"), -float("inf"))):
        x[400 * i + 7, 130 * i + 5] = v
    x[1299, 1024:] = float("inf")
    ws = hyb.new_workspace(256, dev())
    q, s = hyb.quant_fp8(x.to(dev()), 1, ws=ws)
    with pytest.raises(hyb.HybError) as ei:
        hyb.check_status(ws)
    assert ei.value.flags == hyb.STATUS_NAN
    rq, rs = ref8.quant(x.double().numpy(), 1)
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(decoded(q), rq, equal_nan=True)


@pytest.mark.parametrize("ydt", [hyb.HYB_F32, hyb.HYB_BF16])
@pytest.mark.parametrize("m,n,k", [(16, 2500, 1100), (31, 4099, 700), (32, 4096, 2000), (32, 20000, 300), (32, 200, 900),
                                   (9, 2433, 129), (1, 100, 8200), (8, 500, 16384), (5, 17, 12345), (8, 333, 16000),
                                   (9, 40, 16384), (1, 8192, 1030), (33, 2500, 1100), (64, 4099, 700)])
def test_product_variants(m, n, k, ydt):
    A, wq, ws = weight(n, k, m + n + k)
    x = values(m, -(-k // 8) * 8, 7 * m + k)
    xd = x.to(dev())
    xd[:, k:] = float("nan")
    xd, x = xd[:, :k], x[:, :k]
    w = hyb.new_workspace(hyb.fp8_workspace_bytes(m, n, k), dev())
    Y = hyb.matmul_fp8(A, xd, ydt=ydt, ws=w)
    assert hyb.check_status(w) == 0
    check(Y, x, wq, ws, k)
    q, s = hyb.quant_fp8(xd)
    assert torch.equal(hyb.matmul_fp8(A, q, xs=s, ydt=ydt, ws=w), Y)
    # rows of Y that start anywhere; what lies around it stays
    for shift, pad in ((1, 2), (3, 4), (4, 8)):
        Z = torch.full((m + 1, n + shift + pad), 7.0, dtype=Y.dtype, device=dev())
        hyb.matmul_fp8(A, xd, Y=Z[:m, shift:shift + n], ydt=ydt, ws=w)
        assert torch.equal(Z[:m, shift:shift + n], Y)
        assert (Z[m] == 7).all() and (Z[:, :shift] == 7).all() and (Z[:, shift + n:] == 7).all()
    assert hyb.check_status(w) == 0
