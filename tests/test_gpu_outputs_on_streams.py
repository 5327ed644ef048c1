"""Outputs that the 4-bit and routing calls make themselves, on another stream
than the current one: their memory has to be that stream's.  Memory that was freed
on the current stream may still be read by what is queued there."""
import numpy as np
import pytest
import torch

from trellis_coded_bit_b200 import exl3

pytestmark = pytest.mark.gpu
ROWS, K, TOPK, EXPERTS = 4096, 512, 2, 4


@pytest.fixture(scope="module")
def inputs():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    exl3.load()
    g = torch.Generator("cuda")
    g.manual_seed(1)
    x = torch.randn((ROWS, K), generator=g, device="cuda").half()
    ids = torch.randint(0, EXPERTS, (ROWS, TOPK), generator=g, device="cuda", dtype=torch.int32)
    ws = exl3.new_workspace(64 << 20)
    codes, scales = exl3.exl3_mx4_quantize(x)
    offsets, positions = exl3.exl3_moe_sort(ids, EXPERTS, workspace=ws)
    w = torch.rand((ROWS, TOPK), generator=g, device="cuda")
    return dict(x=x, ids=ids, ws=ws, codes=codes, scales=scales, offsets=offsets, positions=positions, w=w,
                half=offsets // TOPK,
                xs=exl3.exl3_moe_gather(x, positions))


CALLS = {
    "quantize": lambda t, s: exl3.exl3_mx4_quantize(t["x"], stream=s),
    "dequantize": lambda t, s: exl3.exl3_mx4_dequantize(t["codes"], t["scales"], stream=s),
    "matmul": lambda t, s: exl3.exl3_mx4_matmul(t["codes"], t["scales"], t["codes"][:256], t["scales"][:256],
                                                workspace=t["ws"], stream=s),
    "linear": lambda t, s: exl3.exl3_mx4_linear(t["x"], t["codes"][:256], t["scales"][:256], workspace=t["ws"], stream=s),
    "experts": lambda t, s: exl3.exl3_mx4_matmul_experts(
        t["codes"], t["scales"], t["half"], t["codes"][:1024].view(EXPERTS, 256, -1),
        t["scales"][:1024].view(EXPERTS, 256, -1), workspace=t["ws"], stream=s),
    "sort": lambda t, s: exl3.exl3_moe_sort(t["ids"], EXPERTS, workspace=t["ws"], stream=s),
    "gather": lambda t, s: exl3.exl3_moe_gather(t["x"], t["positions"], stream=s),
    "combine": lambda t, s: exl3.exl3_moe_combine(t["xs"], t["positions"], stream=s),
    "combine_grad": lambda t, s: exl3.exl3_moe_combine_grad(t["x"], t["xs"], t["positions"], t["w"], stream=s),
}


@pytest.mark.parametrize("name", sorted(CALLS))
def test_output_is_not_memory_in_use(name, inputs):
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = CALLS[name](inputs, side)
    torch.cuda.synchronize()
    outs = outs if isinstance(outs, tuple) else (outs,)
    sizes = [o.numel() * o.element_size() for o in outs]
    plain = [o.clone() for o in outs]
    del outs
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    busy = torch.randn((8192, 8192), device="cuda")
    product = torch.empty_like(busy)
    blocks = [torch.full((n,), 0x5A, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
    kept = [torch.empty_like(b) for b in blocks]
    for _ in range(10):  # some 100 ms of work before the blocks are read
        torch.matmul(busy, busy, out=product)
    for b, c in zip(blocks, kept):
        c.copy_(b)
    del blocks, b
    outs = CALLS[name](inputs, side)
    outs = outs if isinstance(outs, tuple) else (outs,)
    torch.cuda.synchronize()
    assert all(bool((c == 0x5A).all()) for c in kept)
    assert all(torch.equal(a, o) for a, o in zip(plain, outs))
