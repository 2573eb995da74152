"""A product that starts beside a long kernel: its bounded waits count its own
pipeline's time, not the time that the kernel before it takes."""
import pytest
import torch

from gpu_cases import dev
from sparse_weight_b200 import hyb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("m,flags", [(16, hyb.LAUNCH_OVERLAP_PREV), (100, 0), (100, hyb.LAUNCH_OVERLAP_PREV)])
def test_product_behind_a_long_kernel(m, flags):
    g = torch.Generator().manual_seed(m)
    A = hyb.pack_fp8(torch.randn(300, 1500, generator=g).to(dev()))
    x, xs = hyb.quant_fp8(torch.randn(m, 1504, generator=g).to(dev())[:, :1500])
    ws = hyb.new_workspace(hyb.fp8_workspace_bytes(m, 300, 1500), dev())
    want = hyb.matmul_fp8(A, x, xs=xs, ws=ws)
    # 128 units of 256 query rows, each over 80 million tokens (the same few pages again
    # and again): some 3.2e9 clocks on 128 of the SMs, and a wait is bounded by 2.1e9
    C = hyb.new_cache(8, 1, 64, 128, torch.int8, dev())
    C.k.copy_(torch.randint(-20, 21, C.k.shape, generator=g, dtype=torch.int8))
    C.k_scale.fill_(2.0 ** -7)
    C.v_scale.fill_(2.0 ** -7)
    pages = 1_250_000
    table = (torch.arange(pages, dtype=torch.int32, device=dev()) % 8).view(1, -1)
    lens = torch.tensor([64 * pages], dtype=torch.int32, device=dev())
    q = torch.randn(512, 64, 128, generator=g).to(torch.bfloat16).to(dev())
    wa = hyb.new_workspace(hyb.cache_attention_workspace_bytes(C, 1, 64, 512, 64 * pages), dev())
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    out = torch.empty_like(q)
    torch.cuda.synchronize()
    begin.record()
    hyb.cache_attention(C, q, table, lens, out=out, ws=wa)
    y = hyb.matmul_fp8(A, x, xs=xs, ws=ws, flags=flags)
    end.record()
    torch.cuda.synchronize()
    print(f"{begin.elapsed_time(end):.0f} ms")
    assert hyb.check_status(wa) == 0 and hyb.check_status(ws) == 0
    assert torch.equal(y, want)
